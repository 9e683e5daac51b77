"""The 64-bit definition of the 4-bit cache, at the end of the range."""
import numpy as np
import torch

from oracle import requests_oracle as RO

BF16_MAX = float(torch.finfo(torch.bfloat16).max)
F32_MAX = float(torch.finfo(torch.float32).max)


def test_held_values_round_to_finite_numbers_or_are_marked():
    x = np.linspace(0.0, 1.0, 64)
    ones = np.ones((1, 1, 64))
    for vec, marked in ((3.0e38 * x, False), (-3.3e38 * x, False), (np.full(64, BF16_MAX), False), (BF16_MAX * x, False),
                        (1e36 + (BF16_MAX - 1e36) * x, True), (F32_MAX * x, True), (-F32_MAX * x, True),
                        (BF16_MAX * (2 * x - 1), True), (np.where(x == 1, np.inf, x), True), (np.where(x == 0, np.nan, x), True)):
        vec = vec.astype(np.float32).astype(np.float64)[None, None]
        for k, v in ((vec, ones), (ones, vec)):
            hk, hv = RO.held(k, v)
            assert np.isnan(hk).all() == marked and (hv == 0).all() == marked
            if not marked:
                for h in (hk, hv):
                    assert torch.isfinite(torch.as_tensor(h).to(torch.float32).to(torch.bfloat16)).all()
                assert np.abs(hk - k).max() <= np.ptp(k) / 15 and np.abs(hv - v).max() <= np.ptp(v) / 15
