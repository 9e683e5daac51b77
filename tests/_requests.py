"""Shared pieces of the tests of requests over a 4-bit cache: a filled cache, and the error bounds of
its attention."""
from __future__ import annotations

import random

import numpy as np
import torch

import block_sparse_attention_pbsa_b200 as P
from oracle import requests_oracle as RO

DEV = "cuda"
# half a step of rounding, relative to the value
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def t_dtype(dtype):
    return torch.bfloat16 if dtype == "bf16" else torch.float32


class Filled:
    """Requests of ``lens`` = [(step tokens, cached tokens before them)] whose whole K and V are in a 4-bit pool,
    in shuffled slots; queries of the step.  ``rows_after``: rows of no request behind the last one.  ``heavy``: one more
    request, enough work for the batch's requests of more than 80 rows (bf16) to go to the tensor-core kernel."""

    def __init__(self, lens, q_heads, kv_heads, d, dtype, seed=0, rows_after=0, edit=None, slack=3, q_scale=1.0, heavy=False):
        if heavy:
            # 16-row tiles of 125 blocks of 8000 tokens (and 3 for their own start and end), times heads: above 32 for
            # each of the 2 * 148 CTAs of the few-rows kernel
            tiles = -(-33 * 296 // (128 * kv_heads))
            lens = list(lens) + [(max(16 * tiles * kv_heads // q_heads, 81), 8000)]
        self.heavy = heavy
        self.lens, self.hq, self.hk, self.d, self.dtype = lens, q_heads, kv_heads, d, dtype
        dt = t_dtype(dtype)
        gen = torch.Generator().manual_seed(seed)
        rng = random.Random(seed)
        nb = [RO.blocks(n + p) for n, p in lens]
        self.slots = sum(nb) + slack
        perm = list(range(self.slots))
        rng.shuffle(perm)
        self.ld = max(max(nb), 1) + 1
        table = torch.full((len(lens), self.ld), -1, dtype=torch.int32)
        at, maps = 0, []
        for r, (n, p) in enumerate(lens):
            table[r, :nb[r]] = torch.tensor(perm[at:at + nb[r]], dtype=torch.int32)
            at += nb[r]
            pos = torch.arange(n + p)
            maps.append(table[r, pos // 64] * 64 + (pos % 64).to(torch.int32))
        total = sum(n + p for n, p in lens)
        off = torch.randn((2, kv_heads, d), generator=gen)
        self.k = (torch.randn((total, kv_heads, d), generator=gen) + off[0]).to(dt)
        self.v = (torch.randn((total, kv_heads, d), generator=gen) + 0.3 * off[1]).to(dt)
        if edit is not None:
            edit(self)
        T = sum(n for n, _ in lens)
        self.tokens = T + rows_after
        self.q = (q_scale * torch.randn((self.tokens, q_heads, d), generator=gen)).to(dt)
        starts = np.cumsum([0] + [n for n, _ in lens])
        self.table = table.to(DEV)
        self.q_start = torch.tensor(starts, dtype=torch.int32, device=DEV)
        self.q_len = torch.tensor([n for n, _ in lens], dtype=torch.int32, device=DEV)
        self.kv_len = torch.tensor([n + p for n, p in lens], dtype=torch.int32, device=DEV)
        self.max_q = max(n for n, _ in lens)
        self.geom = P.make_req_geom(q_heads, kv_heads, d, d ** -0.5, dtype)
        bb = P.pbsa_q4_block_bytes(self.geom)
        # rows that no token was written to hold bytes whose scales are NaN
        self.pool = torch.full((kv_heads, self.slots, bb), 0xFF, dtype=torch.uint8, device=DEV)
        self.ws = torch.zeros(P.pbsa_attend_q4_workspace_bytes(self.geom), dtype=torch.uint8, device=DEV)
        self.every = torch.cat(maps).to(torch.int32).to(DEV) if total else torch.zeros(0, dtype=torch.int32, device=DEV)
        P.pbsa_append_q4(self.geom, self.k.to(DEV), self.v.to(DEV), self.every, self.pool, self.slots, ws=self.ws)

    def attend(self, causal, q=None, o=None, lse=None, max_q=None, stream=None):
        q = self.q.to(DEV) if q is None else q
        if o is None:
            o = torch.full(q.shape, 7.0, dtype=q.dtype, device=DEV)
        if lse is None:
            lse = torch.full((self.hq, self.tokens), 7.0, device=DEV)
        P.pbsa_attend_q4(self.geom, q, self.q_start, self.q_len, self.kv_len, self.max_q if max_q is None else max_q,
                         self.pool, self.slots, self.table, causal, o, lse, ws=self.ws, stream=stream)
        return o, lse

    def expected(self, causal):
        """Per request: o, lse, bound of o's error, bound of lse's."""
        q, k, v = (t.double().numpy() for t in (self.q, self.k, self.v))
        scale = float(np.float32(self.d ** -0.5))
        out, at, kv = [], 0, 0
        for n, p in self.lens:
            L = n + p
            kk, vv = RO.held(k[kv:kv + L], v[kv:kv + L])
            o, lse, w = RO.attend(q[at:at + n], kk, vv, scale, causal)
            ob, lb = self._bounds(q[at:at + n], k[kv:kv + L], v[kv:kv + L], o, lse, w, scale)
            if self.heavy and n * self.hq // self.hk > 80:
                # the tensor-core form: p is rounded to bf16 (instead of p s), and so is each value: half a step of |v| each
                g = self.hq // self.hk
                for h in range(self.hq):
                    ob[:, h] += 2.0 * U[self.q.dtype] * (w[h] @ np.abs(np.nan_to_num(vv[:, h // g])))
            out.append((o, lse, ob, lb))
            at += n
            kv += L
        return out

    def _bounds(self, q, k, v, o, lse, w, scale):
        """fp32 arithmetic on exact codes: a score sums products up to 136 s |q| (the codes' offset) and m sum(q),
        with fewer than 2^5 roundings of 2^-24 (one more bit for truncating adders): dx.  The exponential and
        the logarithm are good to 2^-21.  Each weight is then off by 2 dx relative, on top of which p s is rounded
        to the query's type (fp32: three bf16 terms, 2^-24) against the centred codes, |c - 8| s, and o once at the
        end.  The sums over keys add 2^-19 of their absolute values (at most 2^5 partial sums meet in a chain that
        keeps growing; a term's share shrinks with it)."""
        n, Hq, d = q.shape
        if not k.shape[0] or not n:
            return np.zeros_like(o), np.zeros_like(lse)
        fin = np.isfinite(k).all(-1, keepdims=True) & np.isfinite(v).all(-1, keepdims=True)
        _, ks, km = RO.quantise(np.where(fin, k, 0.0))
        vc, vs, vm = RO.quantise(np.where(fin, v, 0.0))
        g = Hq // k.shape[1]
        ob, lb = np.zeros_like(o), np.zeros_like(lse)
        u = U[self.q.dtype]
        for h in range(Hq):
            big = 136.0 * ks[:, h // g, 0].max() * np.abs(q[:, h]).sum(-1) + np.abs(km[:, h // g, 0]).max() * np.abs(q[:, h].sum(-1))
            dx = 2.0 ** -18 * scale * big + 2.0 ** -21                                  # [n]
            cent = np.abs(vc[:, h // g] - 8.0) * vs[:, h // g]
            mag = cent + np.abs(vm[:, h // g] + 8.0 * vs[:, h // g])
            ob[:, h] = (u * (w[h] @ cent) + u * np.abs(o[:, h])
                        + (2.0 * dx[:, None] + 2.0 ** -19) * (w[h] @ mag) + 1e-30)
            lb[h] = dx + 2.0 ** -20 * np.abs(np.where(np.isfinite(lse[h]), lse[h], 0.0)) + 2.0 ** -20
        return ob, lb

    def check(self, o, lse, causal):
        o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
        at = 0
        for r, ((n, p), (wo, wl, ob, lb)) in enumerate(zip(self.lens, self.expected(causal))):
            go, gl = o[at:at + n], lse[:, at:at + n]
            assert np.array_equal(np.isnan(go), np.isnan(wo)), f"request {r}: NaN in other places"
            assert np.array_equal(np.isneginf(gl), np.isneginf(wl)), f"request {r}: rows without keys"
            bad = ~(np.abs(go - wo) <= ob) & ~np.isnan(wo)
            assert not bad.any(), f"request {r}: o off by {np.abs(go - wo)[bad].max():.3e} where {ob[bad].min():.3e} is allowed"
            fin = np.isfinite(wl)
            assert (np.abs(gl - wl)[fin] <= lb[fin]).all(), f"request {r}: lse off by {np.abs(gl - wl)[fin].max():.3e}"
            at += n
        # rows of no request are left as they were
        assert (o[at:] == 7.0).all() and (lse[:, at:] == 7.0).all()
        assert P.pbsa_get_device_error(self.ws) == 0
