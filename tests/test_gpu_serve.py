"""A batch of requests served step by step over 4-bit caches: tables, append and attention together, as a
program runs them -- prompts, decodes, ended requests whose blocks others take, graphs, streams."""
import numpy as np
import pytest
import torch

import block_sparse_attention_pbsa_b200 as P
from oracle import requests_oracle as RO

pytestmark = pytest.mark.gpu
DEV = "cuda"
SCALE = lambda d: float(np.float32(d ** -0.5))  # noqa: E731


class Served:
    """The batch beside a plain record of every request's tokens."""

    def __init__(self, cfg, hq, hk, d, dtype, layers=1, seed=0):
        self.batch = P.RequestBatch(cfg)
        self.caches = [P.Q4LayerCache(self.batch, hq, hk, d, dtype) for _ in range(layers)]
        for c in self.caches:
            c.pool.fill_(0xFF)
        self.hq, self.hk, self.d = hq, hk, d
        self.dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.gen = torch.Generator().manual_seed(seed)
        R = cfg.requests
        self.k = [[np.zeros((0, hk, d)) for _ in range(R)] for _ in range(layers)]
        self.v = [[np.zeros((0, hk, d)) for _ in range(R)] for _ in range(layers)]
        self.state = dict(seq=[0] * R, table=np.full((R, cfg.blocks), -1, np.int32),
                          stack=np.arange(cfg.pool_slots - 1, -1, -1, dtype=np.int32), cnt=cfg.pool_slots)

    def draw(self):
        T = self.batch.cfg.tokens
        r = lambda h: torch.randn((T, h, self.d), generator=self.gen).to(self.dt)  # noqa: E731
        return r(self.hq), r(self.hk), r(self.hk)

    def expect(self, step):
        """The oracle's step; returns its tables."""
        c, s = self.batch.cfg, self.state
        want = RO.tables(step, s["seq"], s["table"], s["stack"], s["cnt"], c.pool_slots, c.tokens)
        self.state = dict(seq=want["kv_len"].tolist(), table=want["table"], stack=want["stack"], cnt=want["cnt"])
        return want

    def check_tables(self, want):
        b = self.batch
        for name, got in (("q_start", b.q_start), ("q_len", b.q_len), ("kv_len", b.kv_len), ("slot_map", b.slot_map),
                          ("position", b.position), ("table", b.block_table), ("stack", b.free_slot)):
            np.testing.assert_array_equal(got.cpu().numpy(), want[name], err_msg=name)
        assert int(b.free_cnt) == want["cnt"]

    def check_layer(self, i, want, step, q, k, v, o, causal=True):
        q, k, v, o = (t.double().cpu().numpy() for t in (q, k, v, o))
        u = 2.0 ** -8 if self.dt == torch.bfloat16 else 2.0 ** -24
        covered = np.zeros(len(o), bool)
        for r, n in enumerate(want["q_len"]):
            if step[r] < 0:
                self.k[i][r], self.v[i][r] = self.k[i][r][:0], self.v[i][r][:0]
            if n == 0:
                continue
            a = want["q_start"][r]
            covered[a:a + n] = True
            self.k[i][r] = np.concatenate([self.k[i][r], k[a:a + n]])
            self.v[i][r] = np.concatenate([self.v[i][r], v[a:a + n]])
            kk, vv = RO.held(self.k[i][r], self.v[i][r])
            wo, _, w = RO.attend(q[a:a + n], kk, vv, SCALE(self.d), causal)
            g = self.hq // self.hk
            # p s rounded against codes up to 8 off the middle, V rounded (tensor-core form) and o rounded: each at
            # most half a step of the type, against |v| + 8 s <= 3 max |v| (s <= range / 15); fp32 sums add 2^-15
            for h in range(self.hq):
                mag = w[h] @ np.abs(vv[:, h // g]) + 8.0 * w[h] @ np.ptp(self.v[i][r][:, h // g], axis=-1)[:, None] / 15
                bound = 2.0 * u * mag + u * np.abs(wo[:, h]) + 2.0 ** -15 * mag
                assert (np.abs(o[a:a + n, h] - wo[:, h]) <= bound).all(), (r, h, np.abs(o[a:a + n, h] - wo[:, h]).max())
        assert (o[~covered] == 0).all()


STEPS = [
    [37, 0, 130, 1, 0],          # prompts
    [1, 5, 1, 64, 0],            # decodes, a late prompt
    [1, 1, -1, 1, 90],           # one has ended; another takes its blocks in the same step
    [1, 1, 70, 1, 1],            # its row serves a new request
    [0, -1, 1, 200, 1],          # a prompt too long for the rows: not served
    [1, 3, 1, 1, 1],
]


@pytest.mark.parametrize("dtype,hq,hk,d", [("bf16", 4, 2, 128), ("bf16", 16, 1, 64), ("f32", 3, 3, 64)])
def test_steps_of_a_batch(dtype, hq, hk, d):
    s = Served(P.RequestConfig(requests=5, blocks=5, tokens=170, pool_slots=9), hq, hk, d, dtype, layers=2)
    for step in STEPS:
        want = s.expect(step)
        # (a tensor is not looked at on the host, so a prompt longer than the rows reaches the tables)
        s.batch.step(step if max(step) <= 170 else torch.tensor(step, dtype=torch.int32), min(max(step), 170))
        for i, c in enumerate(s.caches):
            q, k, v = s.draw()
            c.append(k.to(DEV), v.to(DEV))
            s.check_layer(i, want, step, q, k, v, c.attend(q.to(DEV)))
            assert P.pbsa_get_device_error(c.ws) == 0
        s.check_tables(want)
        assert P.pbsa_get_device_error(s.batch.ws) == 0


def test_captured_decode_step_follows_the_lengths():
    """A step of two layers in one CUDA graph: replayed while the requests grow over block boundaries, end, and start
    again, with other inputs in the captured buffers each time."""
    cfg = P.RequestConfig(requests=4, blocks=4, tokens=6, pool_slots=11)
    s = Served(cfg, 6, 2, 128, "bf16", layers=2, seed=1)
    q = torch.zeros((6, 6, 128), dtype=torch.bfloat16, device=DEV)
    k = torch.zeros((6, 2, 128), dtype=torch.bfloat16, device=DEV)
    v, o = torch.zeros_like(k), [torch.zeros_like(q) for _ in range(2)]

    def run():
        s.batch.step(None, max_q_len=3)
        for c, out in zip(s.caches, o):
            c.append(k, v)
            c.attend(q, o=out)

    # a first run, with no request, sets kernel attributes; then capture
    run()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        run()
    steps = [[3, 0, 1, 0], [1, 3, 1, 1]] + [[1, 1, 1, 1]] * 62 + [[1, -1, 1, 3], [3, 1, 1, 1], [-1, 1, 1, 1], [2, 1, 1, 1]]
    for n, step in enumerate(steps):
        want = s.expect(step)
        hq, hk, hv = s.draw()
        q.copy_(hq)
        k.copy_(hk)
        v.copy_(hv)
        for out in o:
            out.zero_()
        s.batch.step_len.copy_(torch.tensor(step, dtype=torch.int32))
        graph.replay()
        for i in range(2):
            s.check_layer(i, want, step, hq, hk, hv, o[i])
        if n % 16 == 0 or n > 60:
            s.check_tables(want)
    assert P.pbsa_get_device_error(s.batch.ws) == 0


@pytest.mark.parametrize("heavy", [False, True])
def test_two_graphs_with_workspaces_of_their_own_run_at_once(heavy):
    """Two captured attentions over the same cache, each with its own workspace, on two streams at the same time."""
    from tests._requests import Filled
    f = Filled([(1, 9000), (2, 3000), (70, 500)], 4, 2, 128, "bf16", seed=21, heavy=heavy)
    want, _ = f.attend(True)
    q = f.q.to(DEV)
    outs, graphs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for st in streams:
        ws = torch.zeros_like(f.ws)
        o = torch.zeros_like(want)
        st.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            P.pbsa_attend_q4(f.geom, q, f.q_start, f.q_len, f.kv_len, f.max_q, f.pool, f.slots, f.table, True, o, None, ws=ws)
        outs.append((o, ws))
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(20):
        for st, g in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for o, ws in outs:
        assert torch.equal(o, want) and P.pbsa_get_device_error(ws) == 0


def test_calls_one_after_another_share_a_workspace():
    """Attentions that are much and little work, of many and of few rows, in turn over one workspace, eager and captured."""
    from tests._requests import Filled
    fs = [Filled([(1, 5000), (90, 300)], 4, 2, 128, "bf16", seed=23, heavy=True), Filled([(1, 700)] * 5, 8, 2, 128, "bf16", seed=24),
          Filled([(200, 100), (3, 9)], 4, 2, 128, "bf16", seed=25), Filled([(20, 400)], 4, 2, 128, "f32", seed=26)]
    want = [f.attend(True)[0] for f in fs]
    for f in fs[1:]:
        f.ws = fs[0].ws
    qs = [f.q.to(DEV) for f in fs]
    outs = [torch.zeros_like(w) for w in want]

    def run():
        for f, q, o in zip(fs, qs, outs):
            P.pbsa_attend_q4(f.geom, q, f.q_start, f.q_len, f.kv_len, f.max_q, f.pool, f.slots, f.table, True, o, None, ws=f.ws)
    run()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)
        o.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        run()
        run()
    for _ in range(10):
        graph.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)
    assert P.pbsa_get_device_error(fs[0].ws) == 0


def test_a_stream_argument_is_used():
    """The calls run on the stream given: work queued there before is seen, on the default stream nothing is awaited."""
    from tests._requests import Filled
    f = Filled([(3, 200), (60, 64)], 4, 2, 128, "bf16", seed=22)
    want, _ = f.attend(True)
    st = torch.cuda.Stream()
    q = torch.zeros_like(f.q, device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        torch.cuda._sleep(20_000_000)
        q.copy_(f.q.to(DEV, non_blocking=True))
    o, _ = f.attend(True, q=q, stream=st)
    st.synchronize()
    assert torch.equal(o, want)


def test_outputs_made_by_a_call_belong_to_its_stream():
    """Outputs that attend and blocks make are cleared on the stream given, not on a current one that lags behind."""
    batch = P.RequestBatch(P.RequestConfig(requests=1, blocks=2, tokens=70, pool_slots=2))
    cache = P.Q4LayerCache(batch, 4, 2, 128)
    gen = torch.Generator().manual_seed(6)
    q, k, v = (torch.randn((70, h, 128), generator=gen).to(torch.bfloat16).to(DEV) for h in (4, 2, 2))
    batch.step([70], 70)
    cache.append(k, v)
    slots = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    want, (wk, wv) = cache.attend(q), cache.blocks(slots)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    torch.cuda._sleep(20_000_000)
    o, (kp, vp) = cache.attend(q, stream=st), cache.blocks(slots, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(kp, wk) and torch.equal(vp, wv)


def test_expanded_blocks_feed_the_block_attention():
    """4-bit blocks expanded into pools and attended by pbsa_attend: the result over the held values."""
    batch = P.RequestBatch(P.RequestConfig(requests=2, blocks=8, tokens=300, pool_slots=10))
    cache = P.Q4LayerCache(batch, 2, 2, 128)
    gen = torch.Generator().manual_seed(4)
    k, v = (torch.randn((300, 2, 128), generator=gen).to(torch.bfloat16) for _ in range(2))
    batch.step([128, 172], 172)
    cache.append(k.to(DEV), v.to(DEV))
    table = batch.block_table.cpu()
    slots = torch.cat([table[1, :2], table[0, :2]]).to(DEV)            # four full blocks
    k_pool, v_pool = cache.blocks(slots)
    g = P.make_geom(2, 128, 8, 8, 8, 8, 128 ** -0.5, "bf16")            # a frame of one block
    q = torch.randn((64, 2, 128), generator=gen).to(torch.bfloat16)
    o = torch.zeros_like(q, device=DEV)
    lists = torch.arange(4, dtype=torch.int32, device=DEV).expand(2, 1, 4).contiguous()
    cnt = torch.full((2, 1), 4, dtype=torch.int32, device=DEV)
    P.pbsa_attend(g, q.to(DEV), 1, k_pool, v_pool, 4, lists, cnt, 4, o, ws=cache.ws)
    kk, vv = RO.held(k.double().numpy(), v.double().numpy())
    rows = np.r_[128:256, 0:128]
    wo, _, _ = RO.attend(q.double().numpy(), kk[rows], vv[rows], SCALE(128), False)
    err = np.abs(o.double().cpu().numpy() - wo)
    assert err.max() <= 2e-2 and err.mean() <= 2e-3
    assert P.pbsa_get_device_error(cache.ws) == 0


def test_batch_state_can_be_saved_and_resumed():
    cfg = P.RequestConfig(requests=3, blocks=4, tokens=100, pool_slots=8)
    a = P.RequestBatch(cfg)
    a.step([70, 1, 0], 70)
    st = a.state_dict()
    b = P.RequestBatch(cfg)
    b.load_state_dict(st)
    for x in (a, b):
        x.step([-1, 64, 30], 64)
    for name in ("kv_len", "block_table", "free_slot", "free_cnt", "slot_map", "q_len"):
        assert torch.equal(getattr(a, name), getattr(b, name)), name
    with pytest.raises(ValueError):
        P.RequestBatch(P.RequestConfig(3, 4, 100, 9)).load_state_dict(st)


def test_the_binding_refuses_what_the_calls_do_not_take():
    """Types, shapes, layouts, devices and sizes that are refused before anything is launched."""
    g = P.make_req_geom(4, 2, 64, 0.1, "bf16")
    i = lambda n: torch.zeros(n, dtype=torch.int32, device=DEV)  # noqa: E731
    x = lambda h, t=8, dt=torch.bfloat16: torch.zeros((t, h, 64), dtype=dt, device=DEV)  # noqa: E731
    pool = torch.zeros(2 * 3 * 4608, dtype=torch.uint8, device=DEV)
    ws = torch.zeros(P.pbsa_attend_q4_workspace_bytes(g), dtype=torch.uint8, device=DEV)

    def tables(**kw):
        a = dict(step_len=i(3), seq_len=i(3), block_table=i(6).view(3, 2), free_slot=i(5), free_cnt=i(1), q_start=i(4), q_len=i(3),
                 kv_len=i(3), free_cnt_out=i(1), slot_map=i(9), position=i(9))
        P.pbsa_request_tables(*{**a, **kw}.values(), ws=None)
    tables()
    for kw in (dict(step_len=i(4)), dict(seq_len=i(3).cpu()), dict(block_table=i(6)), dict(q_start=i(3)), dict(position=i(8)),
               dict(free_cnt=i(2)), dict(slot_map=i(18)[::2]), dict(kv_len=i(3).long()), dict(q_len=None)):
        with pytest.raises(ValueError):
            tables(**kw)
    with pytest.raises(P.PBSAError):
        tables(free_slot=i(0))                                   # a pool without slots

    def append(k=None, v=None, m=None, p=pool, slots=3, w=None):
        P.pbsa_append_q4(g, x(2) if k is None else k, x(2) if v is None else v, i(8) - 1 if m is None else m, p, slots, ws=w)
    append()
    for kw in (dict(k=x(3)), dict(k=x(2, dt=torch.float32)), dict(k=x(2, 7)), dict(v=x(4)[:, ::2]), dict(m=i(7)), dict(slots=4),
               dict(p=pool.view(torch.int8)), dict(w=ws[:100]), dict(k=x(2).cpu())):
        with pytest.raises(ValueError):
            append(**kw)
    with pytest.raises(P.PBSAError):
        append(k=torch.zeros((8, 2 * 64 + 4), dtype=torch.bfloat16, device=DEV)[:, :128].unflatten(1, (2, 64)))   # 8-byte rows
    with pytest.raises(P.PBSAError):
        append(k=x(2)[:1].expand(8, 2, 64))                      # every token the same memory
    with pytest.raises(TypeError):
        append(slots="3")

    def attend(q=None, o=None, start=None, n=1, table=None, lse=None, w=ws, slots=3):
        P.pbsa_attend_q4(g, x(4) if q is None else q, i(4) if start is None else start, i(3), i(3), n, pool, slots,
                         i(6).view(3, 2) if table is None else table, True, x(4) if o is None else o, lse, ws=w)
    attend()
    attend(start=i(3))
    for kw in (dict(q=x(2)), dict(o=x(4, 9)), dict(start=i(5)), dict(table=i(6)), dict(table=i(8).view(4, 2)), dict(w=None),
               dict(w=ws[:-16]), dict(lse=torch.zeros(31, device=DEV)), dict(lse=x(4)), dict(slots=2), dict(n=1 << 40)):
        with pytest.raises(ValueError):
            attend(**kw)
    with pytest.raises(P.PBSAError):
        attend(w=torch.zeros(ws.numel() + 8, dtype=torch.uint8, device=DEV)[8:])        # 8-byte aligned

    def expand(src=None, k=None, v=None):
        d = torch.zeros((2, 2, 64, 64), dtype=torch.bfloat16, device=DEV)
        P.pbsa_expand_q4(g, pool, 3, i(2) if src is None else src, d if k is None else k, d.clone() if v is None else v)
    expand()
    for kw in (dict(src=i(3)), dict(k=torch.zeros((2, 2, 64, 64), device=DEV)), dict(v=x(2)), dict(src=i(2).float())):
        with pytest.raises(ValueError):
            expand(**kw)
    torch.cuda.synchronize()
