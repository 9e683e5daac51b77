"""Calls of the request operators that the documentation allows at its edges: the most query heads, generous bounds, rows in
any order, slots past 32 bits of bytes, slots that several requests list, one pool for both types."""
import numpy as np
import pytest
import torch

import block_sparse_attention_pbsa_b200 as P
from oracle import requests_oracle as RO
from tests._requests import DEV, Filled

pytestmark = pytest.mark.gpu
MIXED = [(1, 70), (3, 200), (1, 0), (0, 9), (90, 130), (1, 1000)]


@pytest.mark.parametrize("lens,hq,hk,dtype", [([(1, 100)], 4096, 1, "bf16"), ([(3, 4000)], 4096, 1, "bf16"), ([(1, 70)], 4096, 1, "f32"),
                                              ([(2, 100), (1, 5)], 4096, 4096, "bf16")])
def test_the_most_query_heads(lens, hq, hk, dtype):
    f = Filled(lens, hq, hk, 64, dtype, seed=31)
    f.heavy = dtype == "bf16" and hk == 1              # (the looser bound, where the second goes to the tensor-core kernel)
    f.check(*f.attend(True), True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("max_q", [91, 5000, 2 ** 31 - 1])
def test_a_bound_above_every_length(dtype, max_q):
    f = Filled(MIXED, 4, 2, 128, dtype, seed=32, rows_after=2)
    f.check(*f.attend(True, max_q=max_q), True)


@pytest.mark.parametrize("heavy", [False, True])
def test_rows_in_another_order_than_the_requests(heavy):
    """Each request's rows at a place of its own, with gaps that stay as they were."""
    f = Filled(MIXED, 4, 2, 128, "bf16", seed=33, heavy=heavy)
    want, wl = f.attend(True)
    order = np.random.default_rng(1).permutation(len(f.lens))
    start, at = [0] * len(f.lens), 3
    for r in order:
        start[r] = at
        at += f.lens[r][0] + 2
    old = f.q_start.cpu().tolist()
    q = torch.full((at, 4, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
    for r, (n, _) in enumerate(f.lens):
        q[start[r]:start[r] + n] = f.q[old[r]:old[r] + n].to(DEV)
    o, lse = torch.full_like(q, 7.0), torch.full((4, at), 7.0, device=DEV)
    P.pbsa_attend_q4(f.geom, q, torch.tensor(start, dtype=torch.int32, device=DEV), f.q_len, f.kv_len, f.max_q, f.pool, f.slots,
                     f.table, True, o, lse, ws=f.ws)
    gap = torch.ones(at, dtype=torch.bool)
    for r, (n, _) in enumerate(f.lens):
        assert torch.equal(o[start[r]:start[r] + n], want[old[r]:old[r] + n])
        assert torch.equal(lse[:, start[r]:start[r] + n], wl[:, old[r]:old[r] + n])
        gap[start[r]:start[r] + n] = False
    assert (o[gap.to(DEV)] == 7).all() and (lse[:, gap.to(DEV)] == 7).all()
    assert P.pbsa_get_device_error(f.ws) == 0


@pytest.mark.parametrize("heavy", [False, True])
def test_a_pool_past_32_bits(heavy):
    """6 GB of slots, of which a batch's lie at the end: append, expand and attention reach them."""
    f = Filled(MIXED, 4, 2, 128, "bf16", seed=34, heavy=heavy)
    want, wl = f.attend(True)
    slots = 360_000
    shift = slots - f.slots
    small, f.pool = f.pool, torch.full((2, slots, P.pbsa_q4_block_bytes(f.geom)), 0xFF, dtype=torch.uint8, device=DEV)
    assert f.pool.numel() > 6 * 10 ** 9
    P.pbsa_append_q4(f.geom, f.k.to(DEV), f.v.to(DEV), f.every + shift * 64, f.pool, slots, ws=f.ws)
    assert torch.equal(f.pool[:, shift:], small) and (f.pool[:, shift - 2:shift] == 0xFF).all()
    used = f.table[f.table >= 0].contiguous()
    blocks = [torch.zeros((2, used.numel(), 64, 128), dtype=torch.bfloat16, device=DEV) for _ in range(4)]
    P.pbsa_expand_q4(f.geom, small, f.slots, used, *blocks[:2], ws=f.ws)
    P.pbsa_expand_q4(f.geom, f.pool, slots, used + shift, *blocks[2:], ws=f.ws)
    assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(blocks[:2], blocks[2:]))
    f.table = torch.where(f.table >= 0, f.table + shift, f.table)
    f.slots = slots
    o, lse = f.attend(True)
    assert torch.equal(o, want) and torch.equal(lse, wl)
    assert P.pbsa_get_device_error(f.ws) == 0


def test_requests_that_list_the_same_slots():
    """Reading is shared freely: two requests over one's cache give the same rows as one."""
    f = Filled([(2, 300), (2, 300)], 4, 2, 128, "bf16", seed=35)
    f.table[1] = f.table[0]
    q = f.q.to(DEV)
    q[2:4] = q[:2]
    o, lse = f.attend(True, q=q)
    # (the shares may cut them in other places: sums of weights rounded to bf16, each rounded to bf16 at the end)
    assert (o[2:4] - o[:2]).abs().max() <= 2.0 ** -7 * o.abs().max() and (lse[:, 2:] - lse[:, :2]).abs().max() <= 2.0 ** -17
    kk, vv = RO.held(f.k[:302].double().numpy(), f.v[:302].double().numpy())
    wo, _, _ = RO.attend(f.q[:2].double().numpy(), kk, vv, float(np.float32(128 ** -0.5)), True)
    assert np.abs(o[:2].double().cpu().numpy() - wo).max() <= 2.0 ** -6 * np.abs(vv).max()


def test_one_pool_for_both_types():
    """The pool's format does not depend on the token tensors' type: what fp32 tokens wrote, bf16 queries attend."""
    f = Filled([(3, 200), (1, 64)], 4, 2, 128, "f32", seed=36)
    g = P.make_req_geom(4, 2, 128, 128 ** -0.5, "bf16")
    q = f.q.to(torch.bfloat16)
    o = torch.zeros(q.shape, dtype=torch.bfloat16, device=DEV)
    P.pbsa_attend_q4(g, q.to(DEV), f.q_start, f.q_len, f.kv_len, f.max_q, f.pool, f.slots, f.table, True, o, ws=f.ws)
    f.q = q.float()
    want, _ = f.attend(True)
    v = np.abs(f.v.double().numpy()).max()
    assert (o.float() - want).abs().max() <= 2.0 ** -6 * v and P.pbsa_get_device_error(f.ws) == 0


@pytest.mark.parametrize("lens,heavy", [(MIXED, False), (MIXED, True), ([(1, 40)] * 9, False)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf"), 3e38])
def test_a_query_that_is_not_finite_stays_in_its_row(lens, heavy, value):
    """Queries share tiles and products; the other rows stay within the bounds of their sums.  (Not always to the bit: in the
    tensor-core form 32 rows take one pass over their scores or two together, and the second rounds a score before the
    reference is taken from it, where the first rounds once.  The bounds count many more roundings than that one.)"""
    f = Filled(lens, 6, 2, 128, "bf16", seed=37, heavy=heavy)
    want, wl = f.attend(True)
    q = f.q.to(DEV)
    rows = [0, 2, f.lens[0][0] + f.lens[1][0] + 1, f.tokens - 1]
    for i, t in enumerate(rows):
        q[t, i, 7 * i] = value
    o, lse = f.attend(True, q=q)
    other = torch.ones((f.tokens, 6), dtype=torch.bool, device=DEV)
    for i, t in enumerate(rows):
        other[t, i] = False
        assert not torch.isfinite(o[t, i]).all() or abs(value) < float("inf")
    if not heavy:
        assert torch.equal(o[other], want[other]) and torch.equal(lse[other.t()], wl[other.t()])
    at, got, gl = 0, o.double().cpu().numpy(), lse.double().cpu().numpy()
    for (n, _), (wo, wlse, ob, lb) in zip(f.lens, f.expected(True)):
        keep = other[at:at + n].cpu().numpy()
        assert (np.abs(got[at:at + n] - wo) <= ob)[keep].all()
        assert (np.abs(gl[:, at:at + n] - wlse) <= lb)[keep.T].all()
        at += n
    assert P.pbsa_get_device_error(f.ws) == 0


@pytest.mark.parametrize("heavy", [False, True])
@pytest.mark.parametrize("value", [0.0, 0.5, -3.0, 1e-39])
def test_keys_with_equal_channels(heavy, value):
    """Keys whose channels are all one number (zeros, above all) have a scale of 0 and their score from the minimum alone, beside
    small keys and queries with one large channel."""
    def edit(f):
        n, p = f.lens[0]
        f.k[:n + p] *= 1e-3
        f.k[:n + p][torch.arange(n + p) % 3 > 0] = value

    f = Filled([(90, 50), (1, 60)], 4, 2, 128, "bf16", seed=38, edit=edit, heavy=heavy)
    f.q[:, :, 0] *= 1e5
    f.check(*f.attend(True), True)


FIRST = """
import sys, torch
sys.path.insert(0, sys.argv[1])
import block_sparse_attention_pbsa_b200 as P
heavy = sys.argv[2] == "heavy"
T = 600 if heavy else 4
batch = P.RequestBatch(P.RequestConfig(requests=2, blocks=200, tokens=T, pool_slots=400))
cache = P.Q4LayerCache(batch, 8, 2, 128)
gen = torch.Generator(device="cuda").manual_seed(0)
q, k, v = (torch.randn((T, h, 128), generator=gen, device="cuda").to(torch.bfloat16) for h in (8, 2, 2))
o, kv = torch.zeros_like(q), [torch.zeros((2, 1, 64, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
slots = torch.zeros(1, dtype=torch.int32, device="cuda")
batch.step_len.copy_(torch.tensor([T - 1, 1], dtype=torch.int32))
start = batch.state_dict(device="cuda")
def run():
    batch.step(None, T)
    cache.append(k, v)
    cache.attend(q, o=o)
    cache.blocks(slots, *kv)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    run()                       # the first calls of the process
g.replay()
torch.cuda.synchronize()
got = [t.clone() for t in (o, *kv, batch.kv_len)]
batch.load_state_dict(start)
batch.step_len.copy_(torch.tensor([T - 1, 1], dtype=torch.int32))
o.zero_()
run()
assert all(torch.equal(a, b) for a, b in zip(got, (o, *kv, batch.kv_len))) and got[-1].tolist() == [T - 1, 1]
assert P.pbsa_get_device_error(cache.ws) == 0 and P.pbsa_get_device_error(batch.ws) == 0
"""


@pytest.mark.parametrize("work", ["little", "heavy"])
def test_the_first_calls_of_a_process_may_be_captured(tmp_path, work):
    import os
    import subprocess
    import sys
    code = tmp_path / "first.py"
    code.write_text(FIRST)
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, str(code), root, work], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


@pytest.mark.parametrize("in_place", [False, True])
def test_a_bad_slot_given_back_is_recorded(in_place):
    """An ended request's table lists a slot outside the pool: it goes back on the stack as it is, recorded."""
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    for bad in (9, -1, 2 ** 31 - 1):
        table, stack, seq, cnt = i(3, bad, 5, 6).view(2, 2), i(0, 1, 2, 4, 7, 7, 7, 7, 7), i(100, 70), i(4)
        out, ws = [torch.zeros(n, dtype=torch.int32, device=DEV) for n in (3, 2, 2, 1, 3)], torch.zeros(256, dtype=torch.uint8, device=DEV)
        kv, left = (seq, cnt) if in_place else (out[2], out[3])
        P.pbsa_request_tables(i(-1, 3), seq, table, stack, cnt, out[0], out[1], kv, left, out[4], ws=ws)
        assert stack.tolist() == [0, 1, 2, 4, 3, bad, 7, 7, 7] and left.tolist() == [6] and kv.tolist() == [0, 73]
        assert out[4].tolist() == [6 * 64 + 6 + j for j in range(3)]
        assert P.pbsa_get_device_error(ws) == 5
