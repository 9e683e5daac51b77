"""A batch saved with its caches and resumed in new ones; steps whose numbers the host does not see; streams and
tensors of another place; captured attentions that overlap."""
import pytest
import torch

import block_sparse_attention_pbsa_b200 as P

pytestmark = pytest.mark.gpu
DEV = "cuda"
CFG = P.RequestConfig(requests=3, blocks=4, tokens=100, pool_slots=8)


def _step(batch, cache, step, seed):
    gen = torch.Generator().manual_seed(seed)
    q, k, v = (torch.randn((CFG.tokens, h, 64), generator=gen).to(torch.bfloat16).to(DEV) for h in (4, 2, 2))
    batch.step(step, max(step))
    cache.append(k, v)
    return cache.attend(q)


def test_a_resumed_batch_attends_as_the_one_that_ran_on():
    a = P.RequestBatch(CFG)
    ca = P.Q4LayerCache(a, 4, 2, 64)
    _step(a, ca, [70, 1, 29], 1)
    saved = a.state_dict(), ca.state_dict()
    b = P.RequestBatch(CFG)
    cb = P.Q4LayerCache(b, 4, 2, 64)
    b.load_state_dict(saved[0])
    cb.load_state_dict(saved[1])
    for seed, step in ((2, [1, 1, 1]), (3, [-1, 64, 30])):
        assert torch.equal(_step(a, ca, step, seed), _step(b, cb, step, seed))
    for cache in (ca, cb):
        assert P.pbsa_get_device_error(cache.ws) == 0


def test_a_loaded_state_has_no_step_yet():
    """What the target's own last step left does not go on: nothing is written or attended before the next step."""
    a, b = P.RequestBatch(CFG), P.RequestBatch(CFG)
    ca, cb = P.Q4LayerCache(a, 4, 2, 64), P.Q4LayerCache(b, 4, 2, 64)
    _step(a, ca, [70, 1, 29], 1)
    _step(b, cb, [1, 90, 2], 2)
    b.load_state_dict(a.state_dict())
    cb.load_state_dict(ca.state_dict())
    x = torch.ones((CFG.tokens, 4, 64), dtype=torch.bfloat16, device=DEV)
    cb.append(x[:, :2], x[:, 2:])
    assert torch.equal(cb.pool, ca.pool)
    assert (cb.attend(x) == 0).all()
    assert (b.slot_map == -1).all() and (b.position == -1).all() and (b.q_len == 0).all() and b.max_q_len == 0


def test_a_state_is_taken_on_the_stream_of_its_steps():
    a = P.RequestBatch(CFG)
    ca = P.Q4LayerCache(a, 4, 2, 64)
    x = torch.ones((CFG.tokens, 4, 64), dtype=torch.bfloat16, device=DEV)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        torch.cuda._sleep(20_000_000)
    a.step(torch.tensor([70, 1, 29], dtype=torch.int32, device=DEV), 70, stream=st)
    ca.append(x[:, :2], x[:, 2:], stream=st)
    saved = a.state_dict(stream=st), ca.state_dict(stream=st)
    torch.cuda.synchronize()
    assert saved[0]["kv_len"].tolist() == [70, 1, 29] and torch.equal(saved[1]["pool"], ca.pool.cpu())
    b = P.RequestBatch(CFG)
    cb = P.Q4LayerCache(b, 4, 2, 64)
    with torch.cuda.stream(st):
        torch.cuda._sleep(20_000_000)
    b.load_state_dict(saved[0], stream=st)
    cb.load_state_dict(saved[1], stream=st)
    o = torch.zeros_like(x)
    b.step([1, 1, 1], 1, stream=st)
    cb.attend(x, o=o, stream=st)
    a.step([1, 1, 1], 1, stream=st)
    want = ca.attend(x, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(b.kv_len, a.kv_len) and torch.equal(o, want)


def test_states_of_other_caches_are_refused():
    a = P.RequestBatch(CFG)
    st = P.Q4LayerCache(a, 4, 2, 64).state_dict()
    for other in (P.Q4LayerCache(a, 4, 1, 64), P.Q4LayerCache(a, 4, 2, 128), P.Q4LayerCache(a, 4, 2, 64, dtype="f32"),
                  P.Q4LayerCache(P.RequestBatch(P.RequestConfig(3, 4, 100, 9)), 4, 2, 64)):
        before = other.pool.clone()
        with pytest.raises(ValueError):
            other.load_state_dict(st)
        assert torch.equal(other.pool, before)
    bst = a.state_dict()
    bst["free_slot"] = bst["free_slot"][:3]
    before = a.state_dict()
    with pytest.raises(ValueError):
        a.load_state_dict(bst)
    assert all(torch.equal(before[n], a.state_dict()[n]) for n in ("kv_len", "block_table", "free_slot", "free_cnt"))


def test_an_entry_above_the_bound_is_recorded():
    """A tensor's entries are not looked at on the host: a request above max_q_len is left out of the attention, which
    the layer's error word tells."""
    a = P.RequestBatch(CFG)
    c = P.Q4LayerCache(a, 4, 2, 64)
    x = torch.ones((CFG.tokens, 4, 64), dtype=torch.bfloat16, device=DEV)
    a.step(torch.tensor([5, 2, 0], dtype=torch.int32), 4)
    c.append(x[:, :2], x[:, 2:])
    o = c.attend(x)
    assert (o[:5] == 0).all() and (o[5:7] != 0).all()
    assert P.pbsa_get_device_error(a.ws) == 0 and P.pbsa_get_device_error(c.ws) == 5


def test_a_stream_of_another_device_is_refused():
    class Elsewhere:
        cuda_stream, device_index = 0, torch.cuda.current_device() + 1

    a = P.RequestBatch(CFG)
    c = P.Q4LayerCache(a, 4, 2, 64)
    x = torch.ones((CFG.tokens, 4, 64), dtype=torch.bfloat16, device=DEV)
    slots = torch.zeros(1, dtype=torch.int32, device=DEV)
    kv = torch.zeros((2, 1, 64, 64), dtype=torch.bfloat16, device=DEV)
    s = Elsewhere()
    for call in (
            lambda: P.pbsa_request_tables(a.step_len, a.kv_len, a.block_table, a.free_slot, a.free_cnt, a.q_start, a.q_len,
                                          a.kv_len, a.free_cnt, a.slot_map, stream=s),
            lambda: P.pbsa_append_q4(c.geom, x[:, :2], x[:, 2:], a.slot_map, c.pool, CFG.pool_slots, stream=s),
            lambda: P.pbsa_expand_q4(c.geom, c.pool, CFG.pool_slots, slots, kv, kv.clone(), stream=s),
            lambda: P.pbsa_attend_q4(c.geom, x, a.q_start, a.q_len, a.kv_len, 1, c.pool, CFG.pool_slots, a.block_table, True,
                                     torch.zeros_like(x), ws=c.ws, stream=s)):
        with pytest.raises(ValueError, match="stream"):
            call()


def test_the_binding_names_what_lies_on_the_host():
    """The refusals are the binding's own, not torch's."""
    g = P.make_req_geom(2, 2, 64, 0.1, "bf16")
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    i, pool = torch.zeros(4, dtype=torch.int32), torch.zeros(2 * 3 * 4608, dtype=torch.uint8)
    dev = lambda *t: [y.to(DEV) for y in t]  # noqa: E731
    for name, args in (("k", (x, *dev(x, i, pool))), ("v", (*dev(x), x, *dev(i, pool))), ("slot_map", (*dev(x, x), i, *dev(pool))),
                       ("pool", (*dev(x, x, i), pool))):
        with pytest.raises(ValueError, match=f"^{name} must be a tensor of the current CUDA device"):
            P.pbsa_append_q4(g, *args, 3)


@pytest.mark.parametrize("heavy", [False, True])
def test_every_replay_of_two_graphs_at_once_gives_the_same(heavy):
    """Two captured attentions with workspaces of their own on two streams: the outputs of each of the replays are kept."""
    from tests._requests import Filled
    f = Filled([(1, 9000), (2, 3000), (70, 500)], 4, 2, 128, "bf16", seed=21, heavy=heavy)
    want, wl = f.attend(True)
    q, runs, streams = f.q.to(DEV), [], [torch.cuda.Stream() for _ in range(2)]
    for st in streams:
        ws, o, lse = torch.zeros_like(f.ws), torch.zeros_like(want), torch.zeros_like(wl)
        st.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            P.pbsa_attend_q4(f.geom, q, f.q_start, f.q_len, f.kv_len, f.max_q, f.pool, f.slots, f.table, True, o, lse, ws=ws)
        runs.append((g, o, lse, ws, torch.zeros((20, *o.shape), dtype=o.dtype, device=DEV), torch.zeros((20, *lse.shape), device=DEV)))
    torch.cuda.synchronize()
    for i in range(20):
        for st, (g, o, lse, _, keep_o, keep_l) in zip(streams, runs):
            with torch.cuda.stream(st):
                o.zero_()
                lse.zero_()
                g.replay()
                keep_o[i].copy_(o)
                keep_l[i].copy_(lse)
    torch.cuda.synchronize()
    for _, _, _, ws, keep_o, keep_l in runs:
        for i in range(20):
            assert torch.equal(keep_o[i], want) and torch.equal(keep_l[i], wl), i
        assert P.pbsa_get_device_error(ws) == 0
