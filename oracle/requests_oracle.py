"""Plain definitions, in float64, of the operators for requests over a 4-bit paged cache: tables of a
step, the 4-bit form of a token, attention over cached tokens.  Numpy only; shares no code with the
CUDA path (test infrastructure)."""
from __future__ import annotations

import numpy as np

B = 64


def blocks(n: int) -> int:
    return -(-n // B)


def tables(step, seq, table, stack, cnt, slots, tokens):
    """One step of the requests' tables, request by request.  Returns a dict of the outputs; ``table`` and
    ``stack`` are copied.  A length outside [0, 64 ld] counts as 0 and its request is not served."""
    table, stack = table.copy(), stack.copy()
    R, ld = table.shape
    ok_seq = [0 <= int(q) <= B * ld for q in seq]
    seq = [int(q) if g else 0 for q, g in zip(seq, ok_seq)]
    free = stack[:cnt].tolist()
    for r in range(R):
        if step[r] < 0:
            free += table[r, :blocks(seq[r])].tolist()
    room, asked, at = len(free), 0, 0
    q_start, q_len, kv_len = [], [], []
    smap, pos = np.full(tokens, -1, np.int32), np.full(tokens, -1, np.int32)
    for r in range(R):
        n, old, took = max(int(step[r]), 0), seq[r], 0
        q_start.append(min(at, tokens))
        if step[r] >= 0 and ok_seq[r] and at + n <= tokens and blocks(old + n) <= ld:
            need = blocks(old + n) - blocks(old)
            asked += need
            if need == 0 or asked <= room:
                for b in range(need):
                    table[r, blocks(old) + b] = free.pop()
                for i in range(n):
                    slot = int(table[r, (old + i) // B])
                    pos[at + i] = old + i
                    smap[at + i] = slot * B + (old + i) % B if 0 <= slot < slots else -1
                took = n
        q_len.append(took)
        kv_len.append(0 if step[r] < 0 else old + took)
        at += n
    q_start.append(min(at, tokens))
    if len(free) > cnt:
        stack[cnt:len(free)] = free[cnt:]
    i32 = lambda a: np.asarray(a, np.int32)  # noqa: E731
    return dict(q_start=i32(q_start), q_len=i32(q_len), kv_len=i32(kv_len), slot_map=smap, position=pos, table=table,
                stack=stack, cnt=len(free))


def _f32(x):
    return np.asarray(x, np.float64).astype(np.float32).astype(np.float64)


def _bf16_side(x, up):
    """The nearest bf16 at or above (below) x: 8 significant bits."""
    m, e = np.frexp(x)
    r = (np.ceil if up else np.floor)(m * 256.0)
    return np.ldexp(r / 256.0, e)


def quantise(x):
    """(codes, s, m) of vectors x [..., d] (finite), float64."""
    x = np.asarray(x, np.float64)
    hi = x.max(-1, keepdims=True)
    m = _bf16_side(x.min(-1, keepdims=True), False)
    span = _f32(hi - m)
    s = _bf16_side(_f32(span * float(np.float32(1.0 / 15.0))), True)
    s = np.where(span == 0, 0.0, np.maximum(s, 2.0 ** -126))
    inv = np.where(s > 0, _f32(1.0 / np.where(s > 0, s, 1.0)), 0.0)
    c = np.minimum(np.rint(_f32(_f32(x - m) * inv)), 15.0)
    return c, s, m


def held(k, v):
    """The values that the cache holds for k, v [..., d], float64: a token and head with a value that is not
    finite in k or v, or whose minimum, range or uppermost held value bf16 or fp32 would round to infinity, holds
    NaN as k and 0 as v."""
    bad = ~(np.isfinite(k).all(-1, keepdims=True) & np.isfinite(v).all(-1, keepdims=True))
    past = 2.0 ** 128 - 2.0 ** 119                       # half a step above bf16's largest number, 2^128 - 2^120
    for x in (k, v):
        x = np.where(bad, 0.0, x)
        lo, hi = x.min(-1, keepdims=True), x.max(-1, keepdims=True)
        wide = (_bf16_side(lo, False) < -past) | (hi - _bf16_side(lo, False) >= 2.0 ** 128 - 2.0 ** 103)
        _, s, m = quantise(np.where(wide, 0.0, x))
        bad = bad | wide | (_f32(np.minimum(15.0 * s + m, past)) >= past)
    out = []
    for x, mark in ((k, np.nan), (v, 0.0)):
        c, s, m = quantise(np.where(bad, 0.0, x))
        out.append(np.where(bad, mark, s * c + m))
    return out


def attend(q, k, v, scale, causal):
    """One request: q [n, Hq, d], held k, v [L, H, d] -> o [n, Hq, d], lse [Hq, n], and the weights
    [Hq, n, L] (for error bounds)."""
    n, Hq, d = q.shape
    L, H = k.shape[:2]
    g = Hq // H
    o, lse, w = np.zeros((n, Hq, d)), np.full((Hq, n), -np.inf), np.zeros((Hq, n, L))
    seen = np.arange(L)[None, :] < ((L - n + np.arange(n) + 1)[:, None] if causal else np.full((n, 1), L))
    for h in range(Hq):
        z = scale * (q[:, h] @ k[:, h // g].T) if L else np.zeros((n, 0))
        for i in range(n):
            js = np.nonzero(seen[i])[0]
            if not len(js):
                continue
            zi = z[i, js]
            top = zi.max()
            e = np.exp(zi - top)
            lse[h, i] = top + np.log(e.sum())
            w[h, i, js] = e / e.sum()
            o[i, h] = w[h, i, js] @ v[js, h // g]
    return o, lse, w
