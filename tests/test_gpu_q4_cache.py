"""The 4-bit cache's writes, bit for bit: both forms of the append (a token at a time, and pairs of neighbouring tokens
from 4096 token-heads on), and tokens at the end of bf16's range."""
import numpy as np
import pytest
import torch

import block_sparse_attention_pbsa_b200 as P
from oracle import requests_oracle as RO
from tests._requests import DEV, Filled, t_dtype

pytestmark = pytest.mark.gpu


def _maps(T, rng):
    """(name, slot map, slots): how neighbouring tokens of a call may lie in the pool."""
    slots = T // 64 + 4
    perm = rng.permutation(slots)

    def along(first):
        pos = np.arange(T) + first
        return perm[pos // 64] * 64 + pos % 64
    even, odd = along(0), along(1)
    holes = along(37).copy()
    holes[rng.random(T) < 0.3] = -1
    # every pair's first token, or its second, is skipped
    first, second = even.copy(), even.copy()
    first[0::2] = -1
    second[1::2] = -1
    anywhere = rng.permutation(slots * 64)[:T]
    swapped = even.copy()                               # the later token of a pair in the earlier row
    swapped[0:T - 1:2], swapped[1::2] = even[1::2], even[0:T - 1:2]
    return slots, dict(even=even, odd=odd, holes=holes, first=first, second=second, anywhere=anywhere, swapped=swapped)


def _expand(geom, pool, slots, H, d, dt):
    ko = torch.zeros((H, slots, 64, d), dtype=dt, device=DEV)
    vo = torch.zeros_like(ko)
    P.pbsa_expand_q4(geom, pool, slots, torch.arange(slots, dtype=torch.int32, device=DEV), ko, vo)
    return [t.permute(1, 2, 0, 3).reshape(-1, H, d).cpu() for t in (ko, vo)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,d,T", [
    (8, 128, 511), (8, 128, 512), (8, 128, 515),         # 8 below, at and 24 above 4096 token-heads
    (8, 64, 511), (8, 64, 512), (5, 64, 821), (1, 64, 4097), (1, 128, 4095),
    (8, 128, 2047), (12, 128, 1367), (1, 64, 16385),
])
def test_append_of_many_tokens_bit_for_bit(H, d, T, dtype):
    """Rows that the map names hold the definition's values, tokens that are not finite their marks, other rows what they
    held."""
    dt = t_dtype(dtype)
    rng = np.random.default_rng(T * H + d)
    gen = torch.Generator().manual_seed(T + d)
    k, v = (torch.randn((T, H, d), generator=gen).to(dt) for _ in range(2))
    # one token of a pair is not finite, in K or in V, first or second; both of a pair
    k[10, 0, 3] = float("nan")
    k[21, H - 1, d - 1] = float("inf")
    v[30, 0, 0] = -float("inf")
    v[T - 1, H - 1, 5] = float("nan")
    k[40, :, 1] = float("nan")
    v[41, :, 2] = float("inf")
    want = [torch.as_tensor(x).to(torch.float32).to(dt) for x in RO.held(k.double().numpy(), v.double().numpy())]
    g = P.make_req_geom(H, H, d, d ** -0.5, dtype)
    slots, maps = _maps(T, rng)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    kd, vd = k.to(DEV), v.to(DEV)
    for name, rows in maps.items():
        pool = torch.randint(0, 64, (H, slots, P.pbsa_q4_block_bytes(g)), dtype=torch.uint8, generator=gen).to(DEV)
        before = _expand(g, pool, slots, H, d, dt)
        P.pbsa_append_q4(g, kd, vd, torch.as_tensor(rows.astype(np.int32)).to(DEV), pool, slots, ws=ws)
        live = rows >= 0
        for b, w, got in zip(before, want, _expand(g, pool, slots, H, d, dt)):
            b[rows[live]] = w[torch.as_tensor(live)]
            assert torch.equal(got.isnan(), b.isnan()), name
            assert torch.equal(got.nan_to_num(0.0), b.nan_to_num(0.0)), name
        assert P.pbsa_get_device_error(ws) == 0


@pytest.mark.parametrize("T", [100, 600])
def test_append_skips_bad_rows_beside_good_ones(T):
    """A row outside the pool is recorded and skipped whichever of two neighbours it is."""
    H, d, slots = 8, 128, T // 64 + 1
    gen = torch.Generator().manual_seed(T)
    k, v = (torch.randn((T, H, d), generator=gen).to(torch.bfloat16) for _ in range(2))
    g = P.make_req_geom(H, H, d, d ** -0.5, "bf16")
    rows = np.arange(T)
    rows[[6, 13, 20, 21]] = [slots * 64, -2, 2 ** 31 - 1, -2 ** 31]
    pool = torch.zeros((H, slots, P.pbsa_q4_block_bytes(g)), dtype=torch.uint8, device=DEV)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    P.pbsa_append_q4(g, k.to(DEV), v.to(DEV), torch.as_tensor(rows.astype(np.int32)).to(DEV), pool, slots, ws=ws)
    assert P.pbsa_get_device_error(ws) == 5
    live = np.ones(T, bool)
    live[[6, 13, 20, 21]] = False
    for w, got in zip(RO.held(k.double().numpy(), v.double().numpy()), _expand(g, pool, slots, H, d, torch.bfloat16)):
        full = torch.zeros((slots * 64, H, d), dtype=torch.bfloat16)
        full[:T][torch.as_tensor(live)] = torch.as_tensor(w[live]).to(torch.float32).to(torch.bfloat16)
        assert torch.equal(got, full)


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


def test_expand_rounds_to_fp32_and_from_there_to_bf16():
    """Code 3 of a token from -2^-30 to 15.0625 (s = 129/128) stands for 3.0234375 - 2^-30, next to the middle of two bf16
    numbers: fp32 rounds it to the middle, which goes to the even one above."""
    x = torch.full((1, 1, 64), 15.0625, dtype=torch.bfloat16)
    x[0, 0, 0], x[0, 0, 1] = -2.0 ** -30, 3.015625
    g = P.make_req_geom(1, 1, 64, 0.125, "bf16")
    pool = torch.zeros((1, 1, P.pbsa_q4_block_bytes(g)), dtype=torch.uint8, device=DEV)
    P.pbsa_append_q4(g, x.to(DEV), x.to(DEV), torch.zeros(1, dtype=torch.int32, device=DEV), pool, 1)
    for t in _expand(g, pool, 1, 1, 64, torch.bfloat16):
        assert float(t[0, 0, 1]) == 3.03125
    f = P.make_req_geom(1, 1, 64, 0.125, "f32")
    for t in _expand(f, pool, 1, 1, 64, torch.float32):
        assert float(t[0, 0, 1]) == 3.0234375
