"""Requests over a 4-bit paged cache: tables, append, expand and attention against their definitions
in float64."""
import numpy as np
import pytest
import torch

import block_sparse_attention_pbsa_b200 as P
from oracle import requests_oracle as RO
from tests._requests import DEV, Filled, t_dtype

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------- tables
def _tables_state(step, seq, ld, free, seed=0, slots=None):
    nb = [RO.blocks(max(q, 0)) if q <= 64 * ld else 0 for q in seq]
    slots = slots or sum(nb) + free + 2
    rng = np.random.default_rng(seed)
    perm = rng.permutation(slots).astype(np.int32)
    table = np.full((len(seq), ld), -7, np.int32)
    at = 0
    for r, n in enumerate(nb):
        table[r, :n] = perm[at:at + n]
        at += n
    stack = np.full(slots, -9, np.int32)
    stack[:free] = perm[at:at + free]
    return table, stack, slots


def _run_tables(step, seq, table, stack, cnt, tokens, in_place=False, position=True):
    c = lambda a: torch.as_tensor(np.asarray(a, np.int32)).to(DEV)  # noqa: E731
    e = lambda n: torch.full((n,), -5, dtype=torch.int32, device=DEV)  # noqa: E731
    R = len(step)
    st, sq, tb, sk, ct = c(step), c(seq), c(table), c(stack), c([cnt])
    out = dict(q_start=e(R + 1), q_len=e(R), kv_len=sq if in_place else e(R), cnt=ct if in_place else e(1),
               slot_map=e(tokens), position=e(tokens), table=tb, stack=sk)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    P.pbsa_request_tables(st, sq, tb, sk, ct, out["q_start"], out["q_len"], out["kv_len"], out["cnt"], out["slot_map"],
                          out["position"] if position else None, ws=ws)
    return {k: v.cpu().numpy() for k, v in out.items()}, P.pbsa_get_device_error(ws)


def _same(got, want):
    for k in ("q_start", "q_len", "kv_len", "slot_map", "position", "table", "stack"):
        np.testing.assert_array_equal(got[k], want[k], err_msg=k)
    assert got["cnt"][0] == want["cnt"]


TABLES = {
    "one request, first token": ([1], [0], 4, 3, 1),
    "one request, into a new block": ([1], [64], 4, 3, 1),
    "one request, within its block": ([1], [63], 4, 0, 1),
    "nothing to do": ([0, 0], [5, 0], 2, 1, 0),
    "only ended requests": ([-1, -1, -3], [130, 0, 64], 3, 0, 0),
    "given back blocks serve the same step": ([-1, 100, 1], [200, 60, 64], 4, 0, 101),
    "a request is refused, a later one needs none": ([65, 1, 1, 70], [64, 64, 10, 0], 4, 2, 137),
    "exactly the free blocks": ([64, 64, 64], [0, 0, 0], 2, 3, 192),
    "rows run out": ([5, 6, 1, 0, 2], [0, 0, 9, 0, 0], 2, 9, 12),
    "a table row runs out": ([1, 1], [128, 127], 2, 9, 2),
    "rows behind the last request": ([3, 2], [1, 2], 2, 9, 70),
}


@pytest.mark.parametrize("name", TABLES)
@pytest.mark.parametrize("in_place", [False, True])
def test_tables_by_hand(name, in_place):
    step, seq, ld, free, tokens = TABLES[name]
    table, stack, slots = _tables_state(step, seq, ld, free)
    got, err = _run_tables(step, seq, table, stack, free, tokens, in_place)
    assert err == 0
    _same(got, RO.tables(step, seq, table, stack, free, slots, tokens))


@pytest.mark.parametrize("R,tokens,seed", [(1, 5000, 1), (3, 1024, 2), (3, 1025, 3), (100, 3000, 4), (1023, 9000, 5),
                                           (1025, 2049, 6), (8192, 20000, 7)])
def test_tables_random_steps(R, tokens, seed):
    """Chains of three steps: state in place, ended requests, refusals by rows and by blocks."""
    rng = np.random.default_rng(seed)
    ld = 20
    seq = rng.integers(0, 64 * ld // 2, R)
    table, stack, slots = _tables_state(None, seq.tolist(), ld, max(1, R // 4), seed)
    cnt = max(1, R // 4)
    for i in range(3):
        step = np.where(rng.random(R) < 0.15, -1, rng.integers(0, max(2, 2 * tokens // R), R))
        want = RO.tables(step, seq, table, stack, cnt, slots, tokens)
        got, err = _run_tables(step, seq, table, stack, cnt, tokens, in_place=bool(i & 1))
        assert err == 0
        _same(got, want)
        seq, table, stack, cnt = want["kv_len"], want["table"], want["stack"], want["cnt"]


def test_tables_bad_numbers_are_recorded_and_not_served():
    # a length past the table, a negative one, a slot outside the pool
    step, seq, ld = [1, 1, 1, 1], [64 * 3 + 1, -4, 10, 20], 3
    table, stack, slots = _tables_state(step, [0, 0, 10, 20], ld, 4)
    table[2, 0] = slots + 5
    got, err = _run_tables(step, seq, table, stack, 4, 4)
    assert err == 5
    _same(got, RO.tables(step, seq, table, stack, 4, slots, 4))
    assert got["slot_map"][2] == -1 and got["slot_map"][3] >= 0
    # a free count above the stack
    got, err = _run_tables([1], [0], table[:1], stack, slots + 1, 1)
    assert err == 5


def test_tables_can_be_repeated_with_inputs_kept_apart():
    step, seq, ld, free, tokens = TABLES["given back blocks serve the same step"]
    table, stack, slots = _tables_state(step, seq, ld, free)
    once, _ = _run_tables(step, seq, table, stack, free, tokens)
    twice, _ = _run_tables(step, seq, once["table"], once["stack"], free, tokens)
    for k in once:
        np.testing.assert_array_equal(once[k], twice[k], err_msg=k)


# ------------------------------------------------------------------------------- append and expand
def _expand(f, slots):
    src = torch.as_tensor(np.asarray(slots, np.int32)).to(DEV)
    ko = torch.full((f.hk, len(slots), 64, f.d), 3.0, dtype=t_dtype(f.dtype), device=DEV)
    vo = torch.full_like(ko, 3.0)
    P.pbsa_expand_q4(f.geom, f.pool, f.slots, src, ko, vo, ws=f.ws)
    return ko.cpu(), vo.cpu()


def _held_as(x, dt):
    """float64 values in the dtype they are read back as (one rounding: the values are exact fp32 sums' inputs)."""
    return torch.as_tensor(x).to(torch.float32).to(dt) if dt == torch.float32 else torch.as_tensor(x).to(torch.float32).to(dt)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hk,lens", [(1, [(0, 1)]), (3, [(5, 60), (0, 64), (0, 129), (1, 0)]), (12, [(0, 1000)])])
def test_append_then_expand_gives_the_held_values(d, dtype, hk, lens):
    """Bit for bit: s, m and the codes have one definition, and s*c + m is rounded once to fp32 (and once more
    to bf16 when that is the type)."""
    f = Filled(lens, hk, hk, d, dtype, seed=d + hk)
    kk, vv = RO.held(f.k.double().numpy(), f.v.double().numpy())
    ko, vo = _expand(f, range(f.slots))
    rows = f.every.cpu().long()
    for got, want in ((ko, kk), (vo, vv)):
        got = got.permute(1, 2, 0, 3).reshape(-1, hk, d)[rows]
        assert torch.equal(got, torch.as_tensor(want).to(torch.float32).to(t_dtype(dtype)))
    assert P.pbsa_get_device_error(f.ws) == 0


def test_append_extremes():
    """Equal channels, huge and tiny ranges, values that are not finite (in K, in V, NaN and infinities)."""
    H, d = 2, 128

    def edit(f):
        f.k[0, 0] = 1.5                       # range 0
        f.v[0, 0] = 0.0
        f.k[1, 0] *= 1e30
        f.v[1, 1] *= 1e-30
        f.k[2, 0] = f.k[2, 0] * 0 + 1.0
        f.k[2, 0, 5] = 1.0078125              # one step of bf16 above the rest
        f.k[3, 1, 7] = float("nan")
        f.v[4, 0, 100] = float("inf")
        f.k[5, 0, 0] = -float("inf")
        f.v[6] = 1e-40                        # below the smallest normal number
        f.v[6, :, 3] = 0.0

    f = Filled([(0, 70)], H, H, d, "bf16", seed=5, edit=edit)
    kk, vv = RO.held(f.k.double().numpy(), f.v.double().numpy())
    ko, vo = _expand(f, range(f.slots))
    rows = f.every.cpu().long()
    for got, want in ((ko, kk), (vo, vv)):
        got = got.permute(1, 2, 0, 3).reshape(-1, H, d)[rows].float().numpy()
        np.testing.assert_array_equal(got, torch.as_tensor(want).to(torch.float32).to(torch.bfloat16).float().numpy())
    assert np.isnan(kk[3, 1]).all() and (vv[4, 0] == 0).all() and np.isnan(kk[5, 0]).all()


def test_append_strided_tokens_and_skipped_rows():
    """K and V as slices of one projection's output; -1 rows are skipped (their values are not read into the
    cache), rows of the pool that no token names stay as they were."""
    H, d, T = 4, 128, 37
    gen = torch.Generator().manual_seed(3)
    qkv = torch.randn((T, 3 * H, d), generator=gen).to(torch.bfloat16).to(DEV)
    k, v = qkv[:, H:2 * H], qkv[:, 2 * H:]
    g = P.make_req_geom(H, H, d, d ** -0.5, "bf16")
    smap = torch.randperm(5 * 64, generator=gen)[:T].to(torch.int32)
    smap[[0, 7, 36]] = -1
    qkv[[0, 7, 36]] = float("nan")
    pool = torch.zeros((H, 5, P.pbsa_q4_block_bytes(g)), dtype=torch.uint8, device=DEV)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    P.pbsa_append_q4(g, k, v, smap.to(DEV), pool, 5, ws=ws)
    ko = torch.zeros((H, 5, 64, d), dtype=torch.bfloat16, device=DEV)
    vo = torch.zeros_like(ko)
    P.pbsa_expand_q4(g, pool, 5, torch.arange(5, dtype=torch.int32, device=DEV), ko, vo, ws=ws)
    assert P.pbsa_get_device_error(ws) == 0
    kk, vv = RO.held(np.nan_to_num(k.double().cpu().numpy()), np.nan_to_num(v.double().cpu().numpy()))
    for got, want in ((ko, kk), (vo, vv)):
        full = torch.zeros((5 * 64, H, d), dtype=torch.bfloat16)
        live = smap >= 0
        full[smap[live].long()] = torch.as_tensor(want[live.numpy()]).float().to(torch.bfloat16)
        assert torch.equal(got.cpu().permute(1, 2, 0, 3).reshape(-1, H, d), full)


def test_append_and_expand_record_bad_slots():
    f = Filled([(0, 64)], 1, 1, 64, "f32")
    before = f.pool.clone()
    bad = torch.tensor([f.slots * 64, -2], dtype=torch.int32, device=DEV)
    P.pbsa_append_q4(f.geom, f.k[:2].to(DEV), f.v[:2].to(DEV), bad, f.pool, f.slots, ws=f.ws)
    assert P.pbsa_get_device_error(f.ws) == 5 and torch.equal(before, f.pool)
    ko, vo = _expand(f, [f.slots, -1])
    assert P.pbsa_get_device_error(f.ws) == 5
    assert (ko == 3).all() and (vo == 3).all()          # blocks without a source stay as they were
    ko, vo = _expand(f, [-1])
    assert P.pbsa_get_device_error(f.ws) == 0 and (ko == 3).all()


# ------------------------------------------------------------------------------- attention
SINGLE = [(1, 0), (1, 1), (1, 14), (1, 15), (1, 16), (1, 62), (1, 63), (1, 64), (1, 200), (1, 511)]
FEW = [(3, 0), (0, 9), (2, 62), (8, 57), (5, 300), (1, 128), (7, 1)]
MANY = [(70, 0), (1, 500), (129, 64), (33, 190), (0, 5), (64, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hk", [(1, 1), (2, 2), (6, 2), (8, 1), (15, 3), (16, 1), (20, 1)])
def test_single_tokens(hq, hk, d, dtype):
    f = Filled(SINGLE, hq, hk, d, dtype, seed=hq)
    f.check(*f.attend(True), True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hk", [(1, 1), (4, 2), (6, 1), (8, 8)])
@pytest.mark.parametrize("causal", [True, False])
def test_a_few_tokens(hq, hk, d, dtype, causal):
    f = Filled(FEW, hq, hk, d, dtype, seed=3, rows_after=4)
    f.check(*f.attend(causal), causal)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hk,d", [(2, 2, 128), (4, 1, 128), (3, 1, 64), (10, 2, 64)])
@pytest.mark.parametrize("causal", [True, False])
def test_prompts_and_decodes_together(hq, hk, d, dtype, causal):
    f = Filled(MANY, hq, hk, d, dtype, seed=4, rows_after=3)
    f.check(*f.attend(causal), causal)


@pytest.mark.parametrize("lens,hq,hk,d,causal", [
    ([(700, 0)], 4, 2, 128, True),                     # a prompt from nothing: row tiles see more and more
    ([(300, 1500), (1, 90), (40, 0), (257, 31)], 6, 2, 128, True),
    ([(130, 2000), (129, 63)], 8, 8, 64, False),
    ([(33, 5000)], 1, 1, 128, True),                   # one row tile over every CTA
    ([(513, 700), (0, 3), (2, 4000)], 3, 1, 64, True),
    ([(5, 333), (4, 100)], 64, 1, 128, True),          # 64 heads share one
    ([(25, 900), (130, 300), (20, 5), (300, 0)], 4, 2, 128, True),   # tiles with and without a second half
    ([(60, 64), (120, 10), (64, 900), (70, 1)], 2, 1, 64, False),
])
def test_long_prompts(lens, hq, hk, d, causal):
    f = Filled(lens, hq, hk, d, "bf16", seed=14, rows_after=2)
    f.check(*f.attend(causal), causal)


@pytest.mark.parametrize("hq,hk,d", [(2, 2, 128), (4, 1, 128), (3, 1, 64), (10, 2, 64)])
@pytest.mark.parametrize("causal", [True, False])
def test_prompts_and_decodes_beside_a_heavy_request(hq, hk, d, causal):
    f = Filled(MANY, hq, hk, d, "bf16", seed=4, rows_after=3, heavy=True)
    f.check(*f.attend(causal), causal)


@pytest.mark.parametrize("lens,hq,hk,d,causal", [
    ([(700, 0)], 4, 2, 128, True),
    ([(300, 1500), (1, 90), (90, 0), (257, 31)], 6, 2, 128, True),
    ([(130, 2000), (129, 63)], 8, 8, 64, False),
    ([(513, 700), (0, 3), (2, 4000)], 3, 1, 64, True),
    ([(5, 333), (4, 100), (1, 700)], 96, 1, 128, True),   # 96 heads share one: a single token fills a half
    ([(25, 900), (130, 300), (64, 5), (300, 0)], 4, 2, 128, True),   # tiles with and without a second half
    ([(60, 64), (120, 10), (64, 900), (70, 1), (90, 2)], 2, 1, 64, False),
])
def test_long_prompts_beside_a_heavy_request(lens, hq, hk, d, causal):
    f = Filled(lens, hq, hk, d, "bf16", seed=14, rows_after=2, heavy=True)
    f.check(*f.attend(causal), causal)


@pytest.mark.parametrize("past", [3000, 4000, 4500, 5000, 6000])
def test_either_side_of_the_choice_of_kernel(past):
    """From a little less work than the tensor-core kernel is chosen for to a little more: the same sums, to rounding."""
    f = Filled([(256, past), (1, 70), (90, 10)], 8, 4, 128, "bf16", seed=18)
    f.heavy = True                                     # (the looser of the two bounds)
    f.check(*f.attend(True), True)


@pytest.mark.parametrize("heavy", [False, True])
def test_tiles_without_keys_among_others(heavy):
    """Prompts of which only a few tokens are cached: whole row tiles see nothing, in the middle of a CTA's share
    and at its ends."""
    lens = [(200, 0), (140, 60), (300, 0), (200, 100)]
    f = Filled(lens, 4, 1, 128, "bf16", seed=15, heavy=heavy)
    full = f.kv_len.clone()
    f.kv_len[0] = 3
    f.kv_len[2] = 0
    o, lse = f.attend(True)
    assert P.pbsa_get_device_error(f.ws) == 0
    assert (o[:197] == 0).all() and torch.isneginf(lse[:, :197]).all() and torch.isfinite(lse[:, 197:200]).all()
    assert (o[340:640] == 0).all() and torch.isneginf(lse[:, 340:640]).all()
    f.kv_len = full
    want, wl = f.attend(True)
    assert torch.equal(o[200:340], want[200:340]) or (o[200:340] - want[200:340]).abs().max() <= 2.0 ** -6
    f.check(want, wl, True)


def test_long_cache_is_split_and_joined():
    """One request over hundreds of blocks (every CTA holds a piece), and beside short ones."""
    for lens in ([(1, 40000)], [(1, 3), (1, 20000), (2, 64), (1, 9000)]):
        f = Filled(lens, 4, 2, 128, "bf16", seed=6)
        f.check(*f.attend(True), True)


@pytest.mark.parametrize("lens", [[(1, i % 3) for i in range(8192)], [(0, 1)] * 8190 + [(60, 70), (1, 64)]])
def test_the_most_requests(lens):
    f = Filled(lens, 1, 1, 64, "bf16", seed=17)
    f.check(*f.attend(True), True)


def test_rows_without_keys():
    """More step tokens than cached ones: the causal rule leaves the first rows no key; and no cache at all."""
    f = Filled([(5, 0), (4, 3)], 4, 2, 128, "bf16", seed=7)
    f.kv_len[0] = 2                  # only 2 of the 5 tokens are in the cache: rows 0..2 see nothing
    f.kv_len[1] = 0
    o, lse = f.attend(True)
    assert (o[:3] == 0).all() and torch.isneginf(lse[:, :3]).all()
    assert (o[5:] == 0).all() and torch.isneginf(lse[:, 5:]).all()
    q, k, v = (t.double().numpy() for t in (f.q, f.k, f.v))
    kk, vv = RO.held(k[:2], v[:2])
    wo, wl, _ = RO.attend(q[3:5], kk, vv, float(np.float32(128 ** -0.5)), True)
    assert np.abs(o[3:5].double().cpu().numpy() - wo).max() <= 2.0 ** -6 * np.abs(vv).max()
    o, lse = f.attend(False)
    assert (o[5:] == 0).all() and torch.isneginf(lse[:, 5:]).all() and torch.isfinite(lse[:, :5]).all()


@pytest.mark.parametrize("lens", [[(1, 700), (4, 300)], [(40, 900), (130, 300)]])
@pytest.mark.parametrize("factor", [30.0, 1e4, 1e9, 1e20, 1e34])
@pytest.mark.parametrize("heavy", [False, True])
def test_large_scores(lens, factor, heavy):
    """Scores from hundreds to the end of fp32's range: the softmax picks one key, whose value is the output (where
    two keys' scores are nearer than fp32 can tell, any mix of theirs), and nothing overflows."""
    f = Filled(lens, 4, 2, 128, "bf16", seed=16, q_scale=factor, heavy=heavy)
    o, lse = f.attend(True)
    assert P.pbsa_get_device_error(f.ws) == 0
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    at = kv = 0
    q, k, v = (t.double().numpy() for t in (f.q, f.k, f.v))
    for n, p in lens:
        kk, vv = RO.held(k[kv:kv + n + p], v[kv:kv + n + p])
        for i in range(n):
            for h in range(4):
                L = p + i + 1
                z = 128 ** -0.5 * (kk[:L, h // 2] @ q[at + i, h])
                # a score's error as in Filled._bounds: 2^-18 of the products it sums, the codes' offset included
                _, ks, km = RO.quantise(k[kv:kv + L, h // 2])
                dx = 2.0 ** -18 * 128 ** -0.5 * (136.0 * ks.max() * np.abs(q[at + i, h]).sum()
                                                 + np.abs(km).max() * abs(q[at + i, h].sum()))
                near = z >= z.max() - 2.0 * dx - 30.0        # (e^-30 of the largest weight and less is nothing)
                lo, hi = vv[:L, h // 2][near].min(0), vv[:L, h // 2][near].max(0)
                got = o[at + i, h].double().cpu().numpy()
                slack = 2.0 ** -6 * np.abs(vv).max()
                assert (got >= lo - slack).all() and (got <= hi + slack).all()
                # log of a sum of at most L weights, in fp32
                assert abs(float(lse[h, at + i]) - z.max()) <= dx + np.log(L) + 2.0 ** -20 * abs(z.max()) + 1e-3
        at += n
        kv += n + p


@pytest.mark.parametrize("lens,heavy", [([(1, 70), (1, 100)], False), ([(40, 50), (130, 5)], False), ([(90, 50), (130, 5)], True)])
def test_values_that_are_not_finite_reach_only_the_rows_that_see_them(lens, heavy):
    """A token that is not finite makes the rows that attend it NaN, and no others: not those it is masked for
    (later step tokens), not other requests."""
    def edit(f):
        n, p = f.lens[0]
        f.k[p + n - 1, 0, 3] = float("nan")      # request 0's last token, head 0
        f.v[n + p, 1, 0] = float("inf")          # request 1's first token, head 1

    f = Filled(lens, 4, 2, 128, "bf16", seed=8, edit=edit, heavy=heavy)
    o, lse = f.attend(True)
    f.check(o, lse, True)
    n = lens[0][0]
    assert torch.isnan(o[n - 1, :2]).all() and torch.isfinite(o[:n - 1]).all() and torch.isfinite(o[n:, :2]).all()


def test_bad_requests_are_left_out():
    f = Filled([(2, 100), (3, 50), (1, 60), (2, 10)], 2, 2, 64, "bf16", seed=9)
    want, _ = f.attend(True)
    f.kv_len[0] = 64 * f.ld + 1
    f.q_len[1] = 4                                  # above max_q
    f.q_start[2] = 100000
    o, lse = f.attend(True, max_q=3)
    assert P.pbsa_get_device_error(f.ws) == 5
    assert (o[:6] == 7).all() and (lse[:, :6] == 7).all()
    assert torch.equal(o[6:], want[6:])


def test_bad_slots_and_requests_beside_a_heavy_request():
    """The tensor-core kernel: a slot outside the pool is recorded and its tokens left out, a bad request is left out."""
    f = Filled([(100, 150), (120, 40)], 2, 2, 64, "bf16", seed=19, heavy=True)
    want, _ = f.attend(True)
    f.table[0, 1] = f.slots + 3
    f.kv_len[1] = 64 * f.ld + 1
    o, lse = f.attend(True)
    assert P.pbsa_get_device_error(f.ws) == 5
    assert (o[100:220] == 7).all() and (lse[:, 100:220] == 7).all()
    assert torch.equal(o[220:], want[220:]) or (o[220:] - want[220:]).abs().max() <= 2.0 ** -6   # (shares lie otherwise)
    keep = np.r_[0:64, 128:250]
    k, v = f.k[:250].double().numpy(), f.v[:250].double().numpy()
    kk, vv = RO.held(k[keep], v[keep])
    wo, wl, _ = RO.attend(f.q[:100].double().numpy(), kk, vv, float(np.float32(64 ** -0.5)), True)
    assert np.abs(o[:100].double().cpu().numpy() - wo).max() <= 2.0 ** -6 * np.abs(vv).max()
    assert np.abs(lse[:, :100].double().cpu().numpy() - wl).max() <= 1e-4


def test_bad_slot_is_left_out_of_the_sums():
    f = Filled([(1, 150)], 2, 2, 128, "bf16", seed=10)
    f.table[0, 1] = f.slots + 3
    o, lse = f.attend(True)
    assert P.pbsa_get_device_error(f.ws) == 5
    keep = np.r_[0:64, 128:151]
    kk, vv = RO.held(f.k.double().numpy()[keep], f.v.double().numpy()[keep])
    wo, wl, _ = RO.attend(f.q.double().numpy(), kk, vv, float(np.float32(128 ** -0.5)), True)
    assert np.abs(o.double().cpu().numpy() - wo).max() <= 2.0 ** -6 * np.abs(vv).max()
    assert np.abs(lse.double().cpu().numpy() - wl).max() <= 1e-4


@pytest.mark.parametrize("lens,causal,heavy", [(FEW, True, False), (MANY, False, False), (MANY, True, True)])
def test_strided_queries_and_outputs(lens, causal, heavy):
    """q as a slice of a projection's output, o inside a wider buffer."""
    f = Filled(lens, 4, 2, 128, "bf16", seed=11, heavy=heavy)
    T = f.tokens
    wide = torch.zeros((T, 8, 128), dtype=torch.bfloat16, device=DEV)
    wide[:, :4] = f.q.to(DEV)
    out = torch.full((T, 6, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    o, lse = f.attend(causal, q=wide[:, :4], o=out[:, 1:5])
    f.check(o, lse, causal)
    assert (out[:, 0] == 7).all() and (out[:, 5] == 7).all()


@pytest.mark.parametrize("lens,heavy", [(FEW, False), (MANY, False), (MANY, True)])
def test_same_bits_every_time_and_without_lse(lens, heavy):
    f = Filled(lens, 8, 2, 128, "bf16", seed=12, heavy=heavy)
    o, lse = f.attend(True)
    for _ in range(3):
        o2, lse2 = f.attend(True)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    o3 = torch.zeros_like(o)
    P.pbsa_attend_q4(f.geom, f.q.to(DEV), f.q_start, f.q_len, f.kv_len, f.max_q, f.pool, f.slots, f.table, True, o3,
                     None, ws=f.ws)
    assert torch.equal(o, o3)


@pytest.mark.parametrize("heavy", [False, True])
def test_the_workspace_may_hold_anything_behind_its_error_word(heavy):
    f = Filled(FEW + [(1, 3000)], 8, 2, 128, "bf16", seed=13, heavy=heavy)
    o, lse = f.attend(True)
    f.ws[256:] = 0xFF
    o2, lse2 = f.attend(True)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
