"""States of batches and caches on the host (tensors on the CPU: nothing is launched)."""
import pytest
import torch

import block_sparse_attention_pbsa_b200 as P

CFG = P.RequestConfig(requests=3, blocks=4, tokens=10, pool_slots=8)


def _pair():
    b = P.RequestBatch(CFG, device="cpu")
    return b, P.Q4LayerCache(b, 4, 2, 64)


def test_states_are_copies_and_come_back_whole():
    b, c = _pair()
    b.kv_len.copy_(torch.tensor([5, 0, 70]))
    c.pool.random_(0, 255, generator=torch.Generator().manual_seed(0))
    saved, bytes_ = (b.state_dict(), c.state_dict()), c.pool.clone()
    b.kv_len.zero_()
    c.pool.zero_()
    assert saved[0]["kv_len"].tolist() == [5, 0, 70] and torch.equal(saved[1]["pool"], bytes_)
    b2, c2 = _pair()
    for t in (b2.q_len, b2.slot_map, b2.position, b2.q_start, b2.step_len):
        t.fill_(3)
    b2.max_q_len = 3
    b2.load_state_dict(saved[0])
    c2.load_state_dict(saved[1])
    assert b2.kv_len.tolist() == [5, 0, 70] and torch.equal(c2.pool, bytes_)
    # between two steps
    assert (b2.slot_map == -1).all() and (b2.position == -1).all() and b2.max_q_len == 0
    assert not b2.q_len.any() and not b2.q_start.any() and not b2.step_len.any()


def test_a_state_that_does_not_fit_changes_nothing():
    b, c = _pair()
    b.kv_len.fill_(9)
    for drop in ({"kv_len": None}, {"free_slot": b.free_slot[:3]}, {"block_table": b.block_table.long()}, {"config": None}):
        other, _ = _pair()
        with pytest.raises(ValueError):
            other.load_state_dict({**b.state_dict(), **drop})
        assert not other.kv_len.any()
    for args in ((4, 1, 64), (2, 2, 64), (4, 2, 128), (4, 2, 64, "f32"), (4, 2, 64, "bf16", 0.5)):
        with pytest.raises(ValueError):
            P.Q4LayerCache(b, *args).load_state_dict(c.state_dict())
    with pytest.raises(ValueError):
        c.load_state_dict(b.state_dict())


def test_a_step_that_is_refused_keeps_the_bound():
    b, _ = _pair()
    b.max_q_len = 2
    with pytest.raises((ValueError, RuntimeError)):
        b.step([1, 1, 1], 1)                 # the tables are on the CPU
    assert b.max_q_len == 2
