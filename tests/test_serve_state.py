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
    b2.load_state_dict(saved[0])
    c2.load_state_dict(saved[1])
    assert b2.kv_len.tolist() == [5, 0, 70] and torch.equal(c2.pool, bytes_)


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
