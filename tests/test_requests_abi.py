"""Host-side rules of the entry points for requests over a 4-bit cache: status codes, and the binding's
refusals.  Every case fails before any CUDA call."""
import ctypes

import pytest
import torch

import block_sparse_attention_pbsa_b200 as P
from block_sparse_attention_pbsa_b200 import _lib, build

host_only = pytest.mark.skipif(torch.cuda.is_available(), reason="fake device pointers: CPU-only check")


@pytest.fixture(scope="module")
def L():
    build.build()
    return _lib.load()


def test_sizes(L):
    g = P.make_req_geom(32, 8, 128, 0.1, "bf16")
    # 64 tokens x (K, V) x (128 / 2 code bytes + 4 bytes of scale and minimum)
    assert P.pbsa_q4_block_bytes(g) == 64 * 2 * (64 + 4)
    assert P.pbsa_q4_block_bytes(P.make_req_geom(1, 1, 64, 0.1, "f32")) == 64 * 2 * (32 + 4)
    assert P.pbsa_attend_q4_workspace_bytes(g) > 256
    for bad in (P.make_req_geom(3, 2, 128, 0.1, "bf16"), P.make_req_geom(2, 2, 96, 0.1, "bf16"),
                P.make_req_geom(2, 2, 128, 0.0, "bf16"), P.make_req_geom(2, 2, 128, float("nan"), "bf16"),
                P.make_req_geom(2, 0, 128, 0.1, "bf16"), P.make_req_geom(2, 2, 128, 0.1, 5)):
        assert P.pbsa_q4_block_bytes(bad) == 0 and P.pbsa_attend_q4_workspace_bytes(bad) == 0


@host_only
def test_status_codes(L):
    f, m = 0x10000, 0x10004      # aligned / misaligned, never dereferenced
    g = P.make_req_geom(32, 8, 128, 0.1, "bf16")

    def tables(step=f, R=4, ld=8, slots=100, tokens=16, smap=f):
        return L.pbsa_request_tables(step, f, R, f, ld, f, f, slots, tokens, f, f, f, f, smap, None, None, None)
    assert tables(step=None) == 1
    assert tables(R=0) == 1
    assert tables(ld=0) == 1
    assert tables(slots=0) == 1
    assert tables(tokens=-1) == 1
    assert tables(smap=None) == 1
    assert tables(slots=1 << 25) == 1             # slot * 64 + row would pass 31 bits
    assert tables(R=8193) == 2
    assert tables(tokens=(1 << 28) + 1) == 2

    def append(geom=g, k=f, k_ld=1024, v_ld=1024, T=4, smap=f, pool=f, slots=100):
        return L.pbsa_append_q4(geom, k, k_ld, f, v_ld, T, smap, pool, slots, None, None)
    assert append(geom=P.make_req_geom(3, 2, 128, 0.1, "bf16")) == 1
    assert append(geom=P.make_req_geom(2, 2, 32, 0.1, "bf16")) == 2
    assert append(k=None) == 1
    assert append(k=m) == 1
    assert append(k_ld=1016) == 1                 # tokens would overlap
    assert append(v_ld=1028) == 1                 # rows that are not 16-byte aligned
    assert append(T=-1) == 1
    assert append(smap=None) == 1
    assert append(pool=m) == 1
    assert append(slots=0) == 1
    assert append(slots=(1 << 31) // (8 * 64) + 1) == 1
    assert append(T=0) == 0                       # nothing to do

    def expand(n=4, src=f, k=f, pool=f):
        return L.pbsa_expand_q4(g, pool, 100, src, n, k, f, None, None)
    assert expand(n=-1) == 1
    assert expand(src=None) == 1
    assert expand(k=m) == 1
    assert expand(pool=None) == 1
    assert expand(n=0) == 0

    def attend(geom=g, q=f, q_ld=4096, T=16, R=4, max_q=4, slots=100, ld=8, flags=1, o_ld=4096, ws=f, table=f):
        return L.pbsa_attend_q4(geom, q, q_ld, T, f, f, f, R, max_q, f, slots, table, ld, flags, f, o_ld, None, ws, None)
    assert attend(q=None) == 1
    assert attend(q=m) == 1
    assert attend(q_ld=4088) == 1
    assert attend(o_ld=4100) == 1
    assert attend(T=-1) == 1
    assert attend(R=0) == 1
    assert attend(max_q=-1) == 1
    assert attend(slots=0) == 1
    assert attend(ld=0) == 1
    assert attend(flags=2) == 1
    assert attend(ws=None) == 1
    assert attend(ws=m) == 1
    assert attend(table=None) == 1
    assert attend(geom=P.make_req_geom(33, 8, 128, 0.1, "bf16")) == 1
    assert attend(R=8193) == 2
    assert attend(T=0) == 0
    assert attend(max_q=0) == 0


def test_binding_refuses_host_tensors():
    g = P.make_req_geom(2, 2, 64, 0.1, "bf16")
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        P.pbsa_append_q4(g, torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(4, 2, 64, dtype=torch.bfloat16), i,
                         torch.zeros(2 * 3 * 4608, dtype=torch.uint8), 3)


def test_batch_refusals_on_the_host():
    """Checks of serve.RequestBatch that come before any device work (a batch on the CPU: nothing is launched)."""
    b = P.RequestBatch(P.RequestConfig(requests=2, blocks=2, tokens=10, pool_slots=3), device="cpu")
    with pytest.raises(ValueError):
        b.step([1, 1], 11)               # more than the rows
    with pytest.raises(ValueError):
        b.step([5, 1], 4)                # an entry above the bound
    with pytest.raises(ValueError):
        b.step([1, 1, 1], 4)             # another number of requests
    with pytest.raises(ValueError):
        P.Q4LayerCache(b, 3, 2, 128)     # heads that do not divide
    with pytest.raises(ValueError):
        P.Q4LayerCache(b, 2, 2, 96)
    c = P.Q4LayerCache(b, 2, 2, 64)
    assert c.kv_bytes == 2 * 3 * 4608
    with pytest.raises(ValueError):
        c.append(torch.zeros(9, 2, 64), torch.zeros(9, 2, 64))
    with pytest.raises(ValueError):
        c.attend(torch.zeros(9, 2, 64))


@host_only
def test_misaligned_workspaces_are_refused(L):
    f, m = 0x10000, 0x10004      # aligned / misaligned, never dereferenced
    g = P.make_req_geom(32, 8, 128, 0.1, "bf16")
    assert L.pbsa_request_tables(f, f, 4, f, 8, f, f, 100, 16, f, f, f, f, f, None, m, None) == 1
    assert L.pbsa_append_q4(g, f, 1024, f, 1024, 4, f, f, 100, m, None) == 1
    assert L.pbsa_expand_q4(g, f, 100, f, 4, f, f, m, None) == 1


@host_only
def test_a_scale_of_zero_is_refused(L):
    batch = P.RequestBatch(P.RequestConfig(requests=1, blocks=1, tokens=1, pool_slots=1), device="cpu")
    with pytest.raises(ValueError, match="scale"):
        P.Q4LayerCache(batch, 2, 2, 64, scale=0.0)
