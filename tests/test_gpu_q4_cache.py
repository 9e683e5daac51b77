"""The 4-bit cache's writes: tokens at the end of bf16's range."""
import numpy as np
import pytest
import torch

import block_sparse_attention_pbsa_b200 as P
from oracle import requests_oracle as RO
from tests._requests import DEV, Filled, t_dtype

pytestmark = pytest.mark.gpu


def _expand(geom, pool, slots, H, d, dt):
    ko = torch.zeros((H, slots, 64, d), dtype=dt, device=DEV)
    vo = torch.zeros_like(ko)
    P.pbsa_expand_q4(geom, pool, slots, torch.arange(slots, dtype=torch.int32, device=DEV), ko, vo)
    return [t.permute(1, 2, 0, 3).reshape(-1, H, d).cpu() for t in (ko, vo)]


BF16_MAX = float(torch.finfo(torch.bfloat16).max)


def _end_of_range(dt):
    """Finite vectors of 64 channels at the end of the range, by name, and whether their held values, their minimum or
    their range pass the largest number (of bf16; of fp32)."""
    x = torch.linspace(0.0, 1.0, 64, dtype=torch.float64)
    f = torch.finfo(dt).max
    return {k: (t.to(dt), marked) for k, (t, marked) in {
        "large": (3.0e38 * x, False), "large and negative": (-3.3e38 * x, False),
        "all the largest": (torch.full((64,), BF16_MAX).double(), False),
        # 15 steps of 17 * 2^120 above 1e36
        "15 steps pass the largest": (1e36 + (BF16_MAX - 1e36) * x, True),
        # 15 steps of 17 * 2^120 are 255 * 2^120, bf16's largest; a step for fp32's is rounded up to 17.125 * 2^120
        "from zero": (f * x, dt == torch.float32),
        "range above fp32's": (f * (2 * x - 1), True),
    }.items()}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tokens_at_the_end_of_the_range(dtype):
    """Whatever is read back is finite, or the token is marked as one that is not."""
    dt = t_dtype(dtype)
    cases = _end_of_range(dt)
    T, H, d = 2 * len(cases), 1, 64
    k, v = torch.ones((T, H, d), dtype=dt), torch.ones((T, H, d), dtype=dt)
    for i, (x, _) in enumerate(cases.values()):
        k[2 * i, 0] = x
        v[2 * i + 1, 0] = x
    g = P.make_req_geom(H, H, d, d ** -0.5, dtype)
    pool = torch.zeros((H, 1, P.pbsa_q4_block_bytes(g)), dtype=torch.uint8, device=DEV)
    P.pbsa_append_q4(g, k.to(DEV), v.to(DEV), torch.arange(T, dtype=torch.int32, device=DEV), pool, 1)
    ko, vo = (t[:T] for t in _expand(g, pool, 1, H, d, dt))
    for i, (name, (_, marked)) in enumerate(cases.items()):
        for t in (2 * i, 2 * i + 1):
            assert bool(torch.isnan(ko[t]).all()) == marked and not torch.isinf(ko[t]).any(), name
            assert torch.isfinite(vo[t]).all() and bool((vo[t] == 0).all()) == marked, name
    for got, want in zip((ko, vo), RO.held(k.double().numpy(), v.double().numpy())):
        np.testing.assert_array_equal(got.double().numpy(), torch.as_tensor(want).to(torch.float32).to(dt).double().numpy())


@pytest.mark.parametrize("lens,heavy", [([(1, 70), (1, 100)], False), ([(40, 50), (130, 5)], False), ([(90, 50), (130, 5)], True)])
def test_values_past_the_range_reach_only_the_rows_that_see_them(lens, heavy):
    """A finite token whose held values would pass bf16's largest number is one that is not finite: NaN for the rows that
    attend it, nothing for the others."""
    def edit(f):
        n, p = f.lens[0]
        f.v[p + n - 1, 0] = 1e36
        f.v[p + n - 1, 0, 5] = BF16_MAX

    f = Filled(lens, 4, 2, 128, "bf16", seed=8, edit=edit, heavy=heavy)
    o, lse = f.attend(True)
    f.check(o, lse, True)
    n = lens[0][0]
    assert torch.isnan(o[n - 1, :2]).all() and torch.isfinite(o[:n - 1]).all() and torch.isfinite(o[n:]).all()
