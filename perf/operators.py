"""Operators for serving requests over a paged cache held in 4 bits, as measured cases.

Four operators that are used together, layer by layer, in a step of a serving program:

``tables``  block tables and slot maps of a step, from the requests' lengths (once a step)
``append``  K and V of the step's tokens enter the 4-bit cache through the slot map; the blocks
            they entered are read back (``expand``) into the 64-token block pools of the
            block-sparse attention
``attend``  attention of the step's queries over the cache: single tokens, a few tokens, long
            chunks, causal or over everything cached

The 4-bit form of the channels x of one token and head (K and V alike, one s and m each):

    m = the largest bf16 <= min x             s = the smallest bf16 >= (max x - m) / 15
    c_i = round((x_i - m) / s), 0 .. 15       x_i is held as  s * c_i + m

``(max x - m) / 15`` is the fp32 product with the fp32 constant 1/15, ``(x_i - m) / s`` the fp32
product with the fp32 reciprocal of s, rounded to the even integer on ties; s = 0 where max x = m,
and never below 2**-126 otherwise.  ``own = False`` computes everything with elementary torch
operations in fp32, ``own = True`` calls this repository's kernels.
"""
import math
import random

import numpy as np
import torch

own = False

B = 64      # tokens of a cache block


# ------------------------------------------------------------------------------- the cases
def listed():
    return [
        # a decode step of 64 requests: one new token each, one request in 64 opens a new block
        dict(name="tables_decode", op="tables", requests=64, tokens=64, max_seq=8192, mix="decode", shape=11),
        # a full step under load: prompts, decodes, ended requests, idle rows, too few free blocks
        dict(name="tables_mixed", op="tables", requests=1024, tokens=49152, max_seq=4096, mix="mixed", shape=12),
        # the K and V of a decode step of 64 requests
        dict(name="append_decode", op="append", kv_heads=8, dim=128, dtype="bf16", requests=64, q_min=1, q_max=1,
             past_min=1, past_max=4000, shape=21),
        # a chunk of 3 frames of 1536 tokens, the heads of the 5 s decode
        dict(name="append_chunk", op="append", kv_heads=12, dim=128, dtype="bf16", requests=1, q_min=4608, q_max=4608,
             past_min=1536, past_max=1536, shape=22),
        # odd prompts in fp32, the small head size
        dict(name="append_f32", op="append", kv_heads=4, dim=64, dtype="f32", requests=7, q_min=3, q_max=301,
             past_min=0, past_max=200, shape=23),
        # one request, one token, a short cache: latency
        dict(name="decode_one", op="attend", q_heads=12, kv_heads=12, dim=128, dtype="bf16", requests=1, q_min=1,
             q_max=1, past_min=1536, past_max=1536, causal=True, shape=31),
        # an ordinary decode batch with shared heads
        dict(name="decode_batch", op="attend", q_heads=32, kv_heads=8, dim=128, dtype="bf16", requests=48, q_min=1,
             q_max=1, past_min=300, past_max=8192, causal=True, shape=32),
        # long caches: what the 4-bit cache is for
        dict(name="decode_long", op="attend", q_heads=32, kv_heads=8, dim=128, dtype="bf16", requests=32, q_min=1,
             q_max=1, past_min=16000, past_max=60000, causal=True, shape=33),
        # a few drafted tokens a request are checked at once; 6 query heads a key head
        dict(name="verify_few", op="attend", q_heads=24, kv_heads=4, dim=128, dtype="bf16", requests=16, q_min=1,
             q_max=8, past_min=200, past_max=6000, causal=True, shape=34),
        # prompt chunks over caches that hold their earlier chunks
        dict(name="prefill_chunk", op="attend", q_heads=32, kv_heads=8, dim=128, dtype="bf16", requests=3, q_min=700,
             q_max=2048, past_min=1000, past_max=14000, causal=True, shape=35),
        # a chunk of 3 frames attends 6 frames of history and itself, both ways: the 5 s decode's heads
        dict(name="chunk_full", op="attend", q_heads=12, kv_heads=12, dim=128, dtype="bf16", requests=1, q_min=4608,
             q_max=4608, past_min=9216, past_max=9216, causal=False, shape=36),
        # fp32, small heads, odd lengths, prompts and decodes in one call
        dict(name="ragged_f32", op="attend", q_heads=8, kv_heads=2, dim=64, dtype="f32", requests=9, q_min=0, q_max=90,
             past_min=0, past_max=700, causal=True, shape=37),
    ]


def _log(rng, a, b):
    return max(a, min(b, int(round(math.exp(rng.uniform(math.log(max(a, 1)), math.log(b)))))))


def draw(rng):
    kind = rng.choice(["tables", "append", "append", "decode", "decode", "few", "prefill", "f32"])
    shape = rng.randrange(1 << 30)
    if kind == "tables":
        r = _log(rng, 1, 2000)
        mix = rng.choice(["decode", "mixed"])
        return dict(op="tables", requests=r, tokens=r + rng.randrange(5) if mix == "decode" else _log(rng, max(r, 64), 49152),
                    max_seq=_log(rng, 100, 8192), mix=mix, shape=shape)
    dim = rng.choice([64, 128])
    hk = rng.choice([1, 2, 4, 8, 12])
    if kind == "append":
        r = _log(rng, 1, 64)
        q = _log(rng, 1, max(1, 4608 // r))
        return dict(op="append", kv_heads=hk, dim=dim, dtype=rng.choice(["bf16", "bf16", "f32"]), requests=r,
                    q_min=rng.randrange(q + 1) if r > 1 else q, q_max=q, past_min=0, past_max=_log(rng, 1, 3000),
                    shape=shape)
    if kind == "decode":
        g = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        r = _log(rng, 1, 64)
        past = _log(rng, 60, min(60000, max(64, 6000000 // (r * hk))))
        return dict(op="attend", q_heads=hk * g, kv_heads=hk, dim=dim, dtype="bf16", requests=r, q_min=1, q_max=1,
                    past_min=rng.randrange(past + 1), past_max=past, causal=True, shape=shape)
    if kind == "few":
        g = rng.choice([1, 2, 4, 6, 8])
        r = _log(rng, 1, 32)
        past = _log(rng, 1, min(20000, max(64, 1500000 // (r * hk))))
        return dict(op="attend", q_heads=hk * g, kv_heads=hk, dim=dim, dtype="bf16", requests=r, q_min=rng.randrange(3),
                    q_max=rng.randrange(2, 40), past_min=0, past_max=past, causal=rng.random() < 0.8, shape=shape)
    if kind == "prefill":
        g = rng.choice([1, 2, 3, 4, 8])
        hk = rng.choice([1, 2, 4, 8])
        r = rng.randrange(1, 4)
        q = _log(rng, 64, 2048)
        return dict(op="attend", q_heads=hk * g, kv_heads=hk, dim=dim, dtype="bf16", requests=r,
                    q_min=rng.randrange(1, q + 1), q_max=q, past_min=0, past_max=_log(rng, 1, 12000 // g),
                    causal=rng.random() < 0.7, shape=shape)
    g = rng.choice([1, 2, 3, 4])
    hk = rng.choice([1, 2, 3])
    return dict(op="attend", q_heads=hk * g, kv_heads=hk, dim=dim, dtype="f32", requests=_log(rng, 1, 12),
                q_min=0, q_max=_log(rng, 1, 120), past_min=0, past_max=_log(rng, 1, 1500), causal=rng.random() < 0.7,
                shape=shape)


def _blocks(n):
    return (n + B - 1) // B


def _lens(case):
    """(new tokens, cached tokens before them) of every request, from the case alone."""
    rng = random.Random(case["shape"])
    return [(rng.randint(case["q_min"], case["q_max"]), rng.randint(case["past_min"], case["past_max"]))
            for _ in range(case["requests"])]


def _step(case):
    """Tables: (step_len, seq_len) of every request (-1: the request has ended) and the free blocks."""
    rng = random.Random(case["shape"])
    R, T = case["requests"], case["tokens"]
    step, seq = [], []
    left = T
    for r in range(R):
        seq.append(rng.randint(0, case["max_seq"]))
        if case["mix"] == "decode":
            step.append(1)
            continue
        u = rng.random()
        if u < 0.1:
            step.append(-1)
        elif u < 0.2:
            step.append(0)
        elif u < 0.7 or left < R:
            step.append(1)
        else:
            step.append(min(rng.randint(2, max(2, 6 * T // R)), max(1, left - (R - r))))
        left -= max(step[-1], 0)
    need = sum(_blocks(q + n) - _blocks(q) for q, n in zip(seq, step) if n > 0)
    free = need + 64 if case["mix"] == "decode" else max(1, int(0.6 * need))
    return step, seq, free


def work(case):
    if case["op"] == "tables":
        step, seq, _ = _step(case)
        R, T = case["requests"], case["tokens"]
        new = sum(_blocks(q + n) - _blocks(q) for q, n in zip(seq, step) if n > 0)
        gone = sum(_blocks(q) for q, n in zip(seq, step) if n < 0)
        # lengths in, starts and lengths out; slots taken or given back read and written; the maps out
        return {"bytes": 4 * (5 * R + 1 + 2 * new + 2 * gone + 2 * T + 2), "flops": 8 * T}
    lens = _lens(case)
    H, d = case["kv_heads"], case["dim"]
    es = 2 if case["dtype"] == "bf16" else 4
    token = 2 * H * (d // 2 + 4)                         # bytes of one token's K and V in the cache
    T = sum(n for n, _ in lens)
    if case["op"] == "append":
        full = sum(_blocks(p + n) - p // B for n, p in lens if n)
        return {"bytes": T * (2 * H * d * es + 4 + token) + full * B * (token + 2 * H * d * es),
                "flops": 8 * T * 2 * H * d}
    Hq = case["q_heads"]
    kv = sum(n + p for n, p in lens if n)
    pairs = sum(n * p + (n * (n + 1) // 2 if case["causal"] else n * n) for n, p in lens)
    return {"bytes": kv * token + T * Hq * (2 * d * es + 4), "flops": 4 * d * Hq * pairs}


# ------------------------------------------------------------------------------- the inputs
def _dt(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _tokens(gen, n, H, d, dt, spread):
    """Keys or values: every channel of a head has its own offset and size, as projections have."""
    x = torch.randn((n, H, d), generator=gen, device="cuda")
    off = torch.randn((H, d), generator=gen, device="cuda") * spread
    size = 0.5 + torch.rand((H, d), generator=gen, device="cuda")
    return (x * size + off).to(dt)


def _layout(case, gen):
    """Block table of the requests (before the step and after it hold the same slots), the slot map of
    the step's tokens and the number of slots: a pool that long use has shuffled."""
    lens = _lens(case)
    nb = [_blocks(n + p) for n, p in lens]
    slots = sum(nb) + 5
    perm = torch.randperm(slots, generator=gen, device="cuda").to(torch.int32).cpu()
    ld = max(max(nb), 1) + 2
    table = torch.full((len(lens), ld), -1, dtype=torch.int32)
    at, q_start, smap, every = 0, [0], [], []
    for r, (n, p) in enumerate(lens):
        table[r, :nb[r]] = perm[at:at + nb[r]]
        at += nb[r]
        pos = torch.arange(n + p)
        rows = table[r, pos // B] * B + (pos % B).to(torch.int32)
        smap.append(rows[p:])
        every.append(rows)
        q_start.append(q_start[-1] + n)
    cat = lambda l: torch.cat(l).to(torch.int32).cuda()  # noqa: E731
    return dict(lens=lens, slots=slots, table=table.cuda(), q_start=torch.tensor(q_start, dtype=torch.int32).cuda(),
                smap=cat(smap), every=cat(every), q_len=torch.tensor([n for n, _ in lens], dtype=torch.int32).cuda(),
                kv_len=torch.tensor([n + p for n, p in lens], dtype=torch.int32).cuda())


def _inputs(case, seed):
    """Everything that the seed decides, as plain tensors."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "tables":
        step, seq, free = _step(case)
        nb = [_blocks(q) for q in seq]
        ld = max(_blocks(q + max(n, 0)) for q, n in zip(seq, step)) + 1
        slots = sum(nb) + free
        perm = torch.randperm(slots, generator=gen, device="cuda").to(torch.int32).cpu()
        table = torch.full((len(seq), ld), -1, dtype=torch.int32)
        at = 0
        for r, n in enumerate(nb):
            table[r, :n] = perm[at:at + n]
            at += n
        stack = torch.full((slots,), -1, dtype=torch.int32)
        stack[:free] = perm[at:]
        c = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
        return dict(step=c(step), seq=c(seq), table=table.cuda(), stack=stack.cuda(), cnt=c([free]), slots=slots,
                    tokens=case["tokens"])
    x = _layout(case, gen)
    H, d, dt = case["kv_heads"], case["dim"], _dt(case)
    if case["op"] == "append":
        T = sum(n for n, _ in x["lens"])
        x["k"], x["v"] = _tokens(gen, T, H, d, dt, 1.0), _tokens(gen, T, H, d, dt, 0.2)
        touched = [x["table"][r, p // B:_blocks(n + p)] for r, (n, p) in enumerate(x["lens"]) if n]
        x["touched"] = (torch.cat(touched) if touched else x["table"][:0, 0]).contiguous()
        return x
    T, kv = sum(n for n, _ in x["lens"]), sum(n + p for n, p in x["lens"])
    x["k"], x["v"] = _tokens(gen, kv, H, d, dt, 1.0), _tokens(gen, kv, H, d, dt, 0.2)
    x["q"] = _tokens(gen, T, case["q_heads"], d, dt, 0.5)
    return x


def _bf16_down(x):
    y = x.to(torch.bfloat16).float()
    return torch.where(y > x, torch.nextafter(y.to(torch.bfloat16), torch.full_like(y, -math.inf).to(torch.bfloat16)).float(), y)


def _bf16_up(x):
    return -_bf16_down(-x)


def _quantise(x):
    """The 4-bit form of x [..., d]: codes uint8 [..., d], s and m fp32 [..., 1]."""
    x = x.float()
    hi = x.amax(-1, keepdim=True)
    m = _bf16_down(x.amin(-1, keepdim=True))
    s = _bf16_up((hi - m) * torch.tensor(1.0 / 15.0, dtype=torch.float32, device=x.device)).clamp(min=2.0 ** -126)
    s = torch.where(hi == m, torch.zeros_like(s), s)
    inv = torch.where(s > 0, torch.ones_like(s) / s, torch.zeros_like(s))
    return torch.round((x - m) * inv).clamp(max=15).to(torch.uint8), s, m


def _value(c, s, m):
    return c.float() * s + m


def _empty_cache(slots, H, d):
    z = lambda n, dt: torch.zeros((slots * B, H, n), dtype=dt, device="cuda")  # noqa: E731
    return [(z(d, torch.uint8), z(1, torch.float32), z(1, torch.float32)) for _ in range(2)]


def _store(cache, rows, k, v, step=1 << 16):
    for i in range(0, rows.numel(), step):
        r = rows[i:i + step].long()
        for part, x in zip(cache, (k, v)):
            for dst, src in zip(part, _quantise(x[i:i + step])):
                dst[r] = src


def prepare(case, seed):
    x = _inputs(case, seed)
    st = dict(case=case, **x)
    if case["op"] == "tables":
        R, T = case["requests"], case["tokens"]
        e = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
        st.update(q_start=e(R + 1), q_len=e(R), kv_len=e(R), smap=e(T), pos=e(T), cnt_out=e(1))
        if own:
            st["ws"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
        return st
    H, d, dt = case["kv_heads"], case["dim"], _dt(case)
    if own:
        import block_sparse_attention_pbsa_b200 as P
        st["geom"] = P.make_req_geom(case.get("q_heads", H), H, d, d ** -0.5, case["dtype"])
        st["pool"] = torch.zeros((H, x["slots"], P.pbsa_q4_block_bytes(st["geom"])), dtype=torch.uint8, device="cuda")
        st["ws"] = torch.zeros(P.pbsa_attend_q4_workspace_bytes(st["geom"]), dtype=torch.uint8, device="cuda")
    else:
        st["cache"] = _empty_cache(x["slots"], H, d)
    if case["op"] == "append":
        n = x["touched"].numel()
        st["k_out"] = torch.zeros((H, n, B, d), dtype=dt, device="cuda")
        st["v_out"] = torch.zeros_like(st["k_out"])
        return st
    if own:
        P.pbsa_append_q4(st["geom"], x["k"], x["v"], x["every"], st["pool"], x["slots"], ws=st["ws"])
    else:
        _store(st["cache"], x["every"], x["k"], x["v"])
    del st["k"], st["v"], st["every"]
    st["max_q"] = max(n for n, _ in x["lens"])
    st["o"] = torch.zeros_like(x["q"])
    st["lse"] = torch.zeros((case["q_heads"], x["q"].shape[0]), device="cuda")
    return st


# ------------------------------------------------------------------------------- one pass
def run(st):
    return _own(st) if own else _plain(st)


def _own(st):
    import block_sparse_attention_pbsa_b200 as P
    op = st["case"]["op"]
    if op == "tables":
        P.pbsa_request_tables(st["step"], st["seq"], st["table"], st["stack"], st["cnt"], st["q_start"], st["q_len"],
                              st["kv_len"], st["cnt_out"], st["smap"], st["pos"], ws=st["ws"])
        return [st[k] for k in ("q_start", "q_len", "kv_len", "smap", "pos", "table", "stack", "cnt_out")]
    if op == "append":
        P.pbsa_append_q4(st["geom"], st["k"], st["v"], st["smap"], st["pool"], st["slots"], ws=st["ws"])
        P.pbsa_expand_q4(st["geom"], st["pool"], st["slots"], st["touched"], st["k_out"], st["v_out"], ws=st["ws"])
        return [st["k_out"], st["v_out"]]
    P.pbsa_attend_q4(st["geom"], st["q"], st["q_start"], st["q_len"], st["kv_len"], st["max_q"], st["pool"],
                     st["slots"], st["table"], st["case"]["causal"], st["o"], st["lse"], ws=st["ws"])
    return [st["o"], st["lse"]]


def _plain_tables(st):
    step, seq, table, stack, T = (st[k] for k in ("step", "seq", "table", "stack", "tokens"))
    step, seq, cnt = step.long(), seq.long(), st["cnt"].long()
    R, ld = table.shape
    dev = table.device
    n = step.clamp(min=0)
    end = torch.cumsum(n, 0)
    start = end - n
    before, after = (seq + B - 1) // B, (seq + n + B - 1) // B
    fits = (step >= 0) & (end <= T) & (after <= ld)
    need = torch.where(fits, after - before, 0)
    upto = torch.cumsum(need, 0)
    gone = torch.where(step < 0, before, 0)
    avail = cnt + gone.sum()
    ok = fits & ((need == 0) | (upto <= avail))
    take = torch.where(ok, need, 0)
    col = torch.arange(ld, device=dev)
    back = table[col[None, :] < gone[:, None]]                       # blocks given back, in request order
    chain = torch.cat([stack, back])                                 # ... lie on top of the free ones
    place = lambda v: torch.where(v < cnt, v, stack.numel() + v - cnt)  # noqa: E731
    i = (upto - need)[:, None] + col[None, :] - before[:, None]
    fresh = (col[None, :] >= before[:, None]) & (col[None, :] < (before + take)[:, None])
    v = torch.where(fresh, avail - 1 - i, 0)
    table.copy_(torch.where(fresh, chain[place(v)], table))
    left = avail - take.sum()
    p = torch.arange(stack.numel(), device=dev)
    put = (p >= cnt) & (p < left)
    stack.copy_(torch.where(put, chain[place(torch.where(put, p, 0))], stack))
    t = torch.arange(T, device=dev)
    r = torch.searchsorted(end, t, right=True)
    live = r < R
    r = r.clamp(max=R - 1)
    live &= ok[r]
    pos = torch.where(live, seq[r] + t - start[r], 0)
    rows = table[r, pos // B].long() * B + pos % B
    st["smap"].copy_(torch.where(live, rows, -1))
    st["pos"].copy_(torch.where(live, pos, -1))
    st["q_start"].copy_(torch.cat([start, end[-1:]]).clamp(max=T))
    st["q_len"].copy_(torch.where(ok, n, 0))
    st["kv_len"].copy_(torch.where(step < 0, 0, seq + torch.where(ok, n, 0)))
    st["cnt_out"].copy_(left)
    return [st[k] for k in ("q_start", "q_len", "kv_len", "smap", "pos", "table", "stack", "cnt_out")]


def _plain(st):
    case = st["case"]
    if case["op"] == "tables":
        return _plain_tables(st)
    H, d, dt = case["kv_heads"], case["dim"], _dt(case)
    if case["op"] == "append":
        _store(st["cache"], st["smap"], st["k"], st["v"])
        out = []
        rows = (st["touched"].long()[:, None] * B + torch.arange(B, device="cuda")).reshape(-1)
        for part in st["cache"]:
            x = _value(*(a[rows] for a in part))
            out.append(x.reshape(-1, B, H, d).permute(2, 0, 1, 3).to(dt).contiguous())
        return out
    Hq, g, scale = case["q_heads"], case["q_heads"] // H, d ** -0.5
    dev, lens = "cuda", st["lens"]
    i = 0
    while i < len(lens):
        # as many requests at once, padded to their longest, as 2^29 values of K and V or of scores hold
        j, N, L = i, 1, 1
        while j < len(lens):
            n, l = max(N, lens[j][0]), max(L, sum(lens[j]))
            if j > i and (j + 1 - i) * l * max(2 * H * d, Hq * n) > 1 << 29:
                break
            j, N, L = j + 1, n, l
        q_len = st["q_len"][i:j, None]
        kv_len = st["kv_len"][i:j, None]
        rows = st["table"][i:j, :_blocks(L)].long().clamp(min=0)[:, :, None] * B + torch.arange(B, device=dev)
        rows = rows.flatten(1)[:, :L]
        k, v = (_value(*(a[rows] for a in part)).permute(0, 2, 1, 3) for part in st["cache"])      # [R, H, L, d]
        behind = torch.arange(L, device=dev) >= kv_len                                              # [R, L]
        v = torch.where(behind[:, None, :, None], 0.0, v)
        part = max(1, (1 << 29) // ((j - i) * Hq * L))
        for t0 in range(0, N, part):
            t = torch.arange(t0, min(t0 + part, N), device=dev)                                     # tokens of the step
            c = t.numel()
            live = t[None, :] < q_len                                                               # [R, c]
            src = torch.where(live, st["q_start"][i:j, None] + t, 0).long()
            q = st["q"][src].float().reshape(j - i, c, H, g, d).permute(0, 2, 1, 3, 4).reshape(j - i, H, c * g, d)
            s = ((q @ k.transpose(2, 3)) * scale).reshape(j - i, H, c, g, L)
            hide = behind[:, None, :].expand(-1, c, -1)
            if case["causal"]:
                hide = hide | (torch.arange(L, device=dev) > (kv_len - q_len + t)[:, :, None])
            s = torch.where(hide[:, None, :, None, :], -math.inf, s)
            top = s.amax(-1, keepdim=True).clamp(min=-3e38)
            e = torch.exp(s - top)
            den = e.sum(-1, keepdim=True)
            o = (e.reshape(j - i, H, c * g, L) @ v).reshape(j - i, H, c, g, d) / den
            lse = (top + torch.log(den))[..., 0]
            to = src[live]
            st["o"][to] = o.permute(0, 2, 1, 3, 4).reshape(j - i, c, Hq, d)[live].to(dt)
            st["lse"][:, to] = lse.permute(0, 2, 1, 3).reshape(j - i, c, Hq)[live].t()
        i = j
    return [st["o"], st["lse"]]


# ------------------------------------------------------------------------------- in 64 bits
def _held64(x):
    """What the cache holds for x [..., d], in 64 bits.  The format fixes the roundings of m, s, of
    (max x - m) / 15, of 1 / s and of their products; they are done here one by one."""
    f32 = lambda t: t.to(torch.float32).to(torch.float64)  # noqa: E731
    shape = x.shape
    g = x.to(torch.float64).flatten(0, -2)
    lo, hi = g.min(1).values, g.max(1).values

    def outward(t, up):
        """The nearest bf16 on the asked side: 8 significant bits of t."""
        mant, ex = torch.frexp(t)
        n = torch.ceil(mant * 256) if up else torch.floor(mant * 256)
        return torch.ldexp(n / 256, ex)

    m = outward(lo, False)
    span = f32(hi - m)
    s = outward(f32(span * float(np.float32(1.0 / 15.0))), True)
    s = torch.where(span == 0, torch.zeros_like(s), torch.clamp(s, min=2.0 ** -126))
    inv = torch.where(s > 0, f32(1.0 / torch.where(s > 0, s, torch.ones_like(s))), torch.zeros_like(s))
    c = torch.clamp(torch.round(f32(f32(g - m[:, None]) * inv[:, None])), max=15.0)
    return (c * s[:, None] + m[:, None]).reshape(shape)


def _exact_tables(x, T):
    """The step, request by request."""
    step, seq, table = x["step"].tolist(), x["seq"].tolist(), x["table"].cpu().numpy().copy()
    stack, cnt = x["stack"].cpu().numpy().copy(), int(x["cnt"])
    R, ld = table.shape
    free = stack[:cnt].tolist()
    for r in range(R):
        if step[r] < 0:
            free += table[r, :_blocks(seq[r])].tolist()
    room = len(free)
    asked, at = 0, 0
    q_start, q_len, kv_len = [], [], []
    smap, pos = np.full(T, -1, np.int32), np.full(T, -1, np.int32)
    for r in range(R):
        n, old = max(step[r], 0), seq[r]
        q_start.append(min(at, T))
        took = 0
        if step[r] >= 0 and at + n <= T and _blocks(old + n) <= ld:
            need = _blocks(old + n) - _blocks(old)
            asked += need
            if need == 0 or asked <= room:
                for b in range(need):
                    table[r, _blocks(old) + b] = free.pop()
                for i in range(n):
                    pos[at + i] = old + i
                    smap[at + i] = table[r, (old + i) // B] * B + (old + i) % B
                took = n
        q_len.append(took)
        kv_len.append(0 if step[r] < 0 else old + took)
        at += n
    q_start.append(min(at, T))
    if len(free) > cnt:
        stack[cnt:len(free)] = free[cnt:]
    c = lambda a: torch.as_tensor(np.asarray(a, np.int32))  # noqa: E731
    return [c(q_start), c(q_len), c(kv_len), c(smap), c(pos), c(table), c(stack), c([len(free)])]


def exact(case, seed):
    x = _inputs(case, seed)
    if case["op"] == "tables":
        return _exact_tables(x, case["tokens"])
    H, d = case["kv_heads"], case["dim"]
    if case["op"] == "append":
        place = {int(s): i for i, s in enumerate(x["touched"].tolist())}
        rows = x["smap"].tolist()
        j = torch.tensor([place[r // B] for r in rows], dtype=torch.long, device="cuda")
        w = torch.tensor([r % B for r in rows], dtype=torch.long, device="cuda")
        out = []
        for t in (x["k"], x["v"]):
            full = torch.zeros((len(place), B, H, d), dtype=torch.float64, device="cuda")
            full[j, w] = _held64(t)
            out.append(full.permute(2, 0, 1, 3).contiguous())
        return out
    Hq = case["q_heads"]
    pairs = sum(n * (n + p) for n, p in x["lens"])
    if 4.0 * d * Hq * pairs > 5e13:
        return None
    T = x["q"].shape[0]
    o = torch.zeros((T, Hq, d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((Hq, T), dtype=torch.float64, device="cuda")
    at = kv = 0
    for n, p in x["lens"]:
        L = n + p
        for h in range(H if n else 0):
            k, v = _held64(x["k"][kv:kv + L, h]), _held64(x["v"][kv:kv + L, h])
            for head in range(h * (Hq // H), (h + 1) * (Hq // H)):
                for i in range(0, n, 1024):
                    q = x["q"][at + i:at + min(i + 1024, n), head].double()
                    z = torch.matmul(q, k.t()) / math.sqrt(d)
                    if case["causal"]:
                        ahead = torch.ones_like(z, dtype=torch.bool).triu(p + i + 1)
                        z = z.masked_fill(ahead, -math.inf)
                    l = torch.logsumexp(z, 1)
                    o[at + i:at + i + q.shape[0], head] = torch.matmul(torch.exp(z - l[:, None]), v)
                    lse[head, at + i:at + i + q.shape[0]] = l
        at += n
        kv += L
    return [o, lse]
