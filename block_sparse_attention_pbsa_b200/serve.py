"""Requests of different lengths over 4-bit paged caches: the device state of a batch and of its layers.

``RequestBatch`` holds what all layers of a model share -- the requests' lengths, block tables and the
stack of free slots -- and builds a step's tables from the number of tokens that each request adds.
``Q4LayerCache`` holds one layer's 4-bit pool, writes a step's K and V into it and attends over it.
Both only sequence the C-ABI calls; every number, the lengths included, stays on the device, so a
step (or a step of every layer) can be captured in a CUDA graph and replayed while the lengths move:

    batch.step(step_len, max_q_len)        # once a step
    for layer, cache in ...:
        cache.append(k, v)                 # K, V of the step's tokens [tokens, kv_heads, head_dim]
        o = cache.attend(q)                # Q of the step's tokens [tokens, q_heads, head_dim]
"""
from __future__ import annotations

import contextlib
import dataclasses

import torch

from . import _lib as L


@dataclasses.dataclass(frozen=True)
class RequestConfig:
    """Sizes of a batch: ``requests`` rows of a table of ``blocks`` slots each (64 tokens a slot), ``tokens`` rows
    of a step's token tensors, ``pool_slots`` slots that the requests share."""
    requests: int
    blocks: int
    tokens: int
    pool_slots: int


def _on(stream):
    """The context in which a call makes its own tensors: the stream that its kernels run on."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _saved(owner, config: dict, device, stream) -> dict:
    with _on(stream):
        st = {name: getattr(owner, name).to(device, copy=True) for name in owner._STATE}
    return {**st, "config": config}


def _load(owner, st: dict, config: dict, stream):
    """All of a state, or nothing where any of it does not fit."""
    what = type(owner).__name__
    if st.get("config") != config:
        raise ValueError(f"the state was taken from a {what} of another configuration")
    for name in owner._STATE:
        dst, src = getattr(owner, name), st.get(name)
        if not isinstance(src, torch.Tensor) or src.shape != dst.shape or src.dtype != dst.dtype:
            raise ValueError(f"{name}: shape or dtype does not match the {what}")
    with _on(stream):
        for name in owner._STATE:
            getattr(owner, name).copy_(st[name])


class RequestBatch:
    def __init__(self, cfg: RequestConfig, device="cuda"):
        self.cfg = cfg
        self.device = torch.device(device)
        new = lambda n, v=0: torch.full((n,), v, dtype=torch.int32, device=self.device)  # noqa: E731
        R, T = cfg.requests, cfg.tokens
        self.kv_len = new(R)                   # tokens cached of each request, the step's own included
        self.block_table = torch.full((R, cfg.blocks), -1, dtype=torch.int32, device=self.device)
        # slots are handed out from the end: the first request gets the first slots
        self.free_slot = torch.arange(cfg.pool_slots - 1, -1, -1, dtype=torch.int32, device=self.device)
        self.free_cnt = new(1, cfg.pool_slots)
        self.step_len = new(R)
        self.q_start, self.q_len = new(R + 1), new(R)
        self.slot_map, self.position = new(T, -1), new(T, -1)
        self.ws = torch.zeros(256, dtype=torch.uint8, device=self.device)
        self.max_q_len = 0

    def step(self, step_len, max_q_len: int, stream=None):
        """The tables of a step: request r adds ``step_len[r]`` tokens (0: none, negative: it has ended and its
        blocks are free again).  ``step_len`` is a device tensor (None: what ``self.step_len`` holds, as in a captured
        step) or a list; no entry is above ``max_q_len`` (a tensor's are not looked at here: the attention leaves such a
        request out and records it, see ``Q4LayerCache``).  Afterwards ``q_len`` tells which requests were served
        (a request that found no room has 0), ``slot_map`` and ``position`` where the step's tokens go."""
        if not 0 <= max_q_len <= self.cfg.tokens:
            raise ValueError(f"max_q_len must lie in [0, {self.cfg.tokens}], got {max_q_len}")
        if step_len is not None and not isinstance(step_len, torch.Tensor):
            if max(step_len, default=0) > max_q_len:
                raise ValueError(f"a request adds {max(step_len)} tokens, more than max_q_len = {max_q_len}")
            step_len = torch.tensor(step_len, dtype=torch.int32)
        if step_len is not None and step_len is not self.step_len:
            if step_len.shape != self.step_len.shape:
                raise ValueError(f"step_len must have {self.cfg.requests} entries, got {list(step_len.shape)}")
            with _on(stream):
                self.step_len.copy_(step_len)
        L.pbsa_request_tables(self.step_len, self.kv_len, self.block_table, self.free_slot, self.free_cnt, self.q_start,
                              self.q_len, self.kv_len, self.free_cnt, self.slot_map, self.position, ws=self.ws,
                              stream=stream)
        self.max_q_len = max_q_len

    # ------------------------------------------------------------------ checkpoint / resume
    _STATE = ("kv_len", "block_table", "free_slot", "free_cnt")

    def state_dict(self, device="cpu", stream=None) -> dict:
        """The lengths, block tables and free slots (copied to ``device`` on ``stream``, that of the steps).  With the
        ``state_dict`` of each layer's cache, which holds the K and V, it is everything that the next step needs."""
        return _saved(self, dataclasses.asdict(self.cfg), device, stream)

    def load_state_dict(self, st: dict, stream=None):
        """Restore a ``state_dict`` of a batch of the same configuration.  The batch is then between two steps: until
        the next one no row has a place in the cache and no request has tokens."""
        _load(self, st, dataclasses.asdict(self.cfg), stream)
        with _on(stream):
            for t in (self.step_len, self.q_start, self.q_len):
                t.zero_()
            for t in (self.slot_map, self.position):
                t.fill_(-1)
        self.max_q_len = 0


class Q4LayerCache:
    """One layer's 4-bit pool for the requests of ``batch``.  ``ws`` may be shared by the layers of a model, whose
    calls follow one another (see pbsa_attend_q4_workspace_bytes).  What the calls find wrong on the device -- slots
    outside the pool, requests whose numbers are out of range -- is in the error words of ``ws`` and ``batch.ws``, which
    ``pbsa_get_device_error`` reads and clears."""

    def __init__(self, batch: RequestBatch, q_heads: int, kv_heads: int, head_dim: int, dtype="bf16", scale=None, ws=None):
        self.batch = batch
        self.geom = L.make_req_geom(q_heads, kv_heads, head_dim, head_dim ** -0.5 if scale is None else scale,
                                    dtype)
        block = L.pbsa_q4_block_bytes(self.geom)
        if block == 0:
            raise ValueError("heads, head size, scale or type that the 4-bit cache is not built for")
        self.pool = torch.zeros((kv_heads, batch.cfg.pool_slots, block), dtype=torch.uint8, device=batch.device)
        need = L.pbsa_attend_q4_workspace_bytes(self.geom)
        if ws is not None and ws.numel() * ws.element_size() < need:
            raise ValueError(f"the workspace must hold {need} bytes")
        self.ws = torch.zeros(need, dtype=torch.uint8, device=batch.device) if ws is None else ws

    @property
    def kv_bytes(self) -> int:
        """Bytes of the pool."""
        return self.pool.numel()

    def append(self, k, v, stream=None):
        """K and V of the step's tokens [tokens, kv_heads, head_dim] into the cache."""
        b = self.batch
        if k.shape[0] != b.cfg.tokens:
            raise ValueError(f"a step has {b.cfg.tokens} token rows, got {k.shape[0]}")
        L.pbsa_append_q4(self.geom, k, v, b.slot_map, self.pool, b.cfg.pool_slots, ws=self.ws, stream=stream)

    def attend(self, q, causal=True, o=None, lse=None, stream=None):
        """Attention of the step's tokens over the cache (their own K and V included).  Rows of ``o`` (and ``lse``)
        that belong to no served request are left as they are (zeros where ``o`` is made here)."""
        b = self.batch
        if q.shape[0] != b.cfg.tokens:
            raise ValueError(f"a step has {b.cfg.tokens} token rows, got {q.shape[0]}")
        if o is None:
            with _on(stream):
                o = torch.zeros(q.shape, dtype=q.dtype, device=q.device)
        L.pbsa_attend_q4(self.geom, q, b.q_start, b.q_len, b.kv_len, b.max_q_len, self.pool, b.cfg.pool_slots,
                         b.block_table, causal, o, lse, ws=self.ws, stream=stream)
        return o

    def blocks(self, slots, k_pool=None, v_pool=None, stream=None):
        """Slots (int32 device tensor) as dense blocks [kv_heads, len(slots), 64, head_dim], the pools that
        pbsa_attend reads."""
        if k_pool is None or v_pool is None:
            dt = torch.bfloat16 if self.geom.dtype == L.PBSA_BF16 else torch.float32
            shape = (self.geom.kv_heads, slots.numel(), 64, self.geom.head_dim)
            with _on(stream):
                k_pool = torch.zeros(shape, dtype=dt, device=self.batch.device) if k_pool is None else k_pool
                v_pool = torch.zeros(shape, dtype=dt, device=self.batch.device) if v_pool is None else v_pool
        L.pbsa_expand_q4(self.geom, self.pool, self.batch.cfg.pool_slots, slots, k_pool, v_pool, ws=self.ws, stream=stream)
        return k_pool, v_pool

    # ------------------------------------------------------------------ checkpoint / resume
    _STATE = ("pool",)

    def _config(self) -> dict:
        g = self.geom
        return dict(q_heads=g.q_heads, kv_heads=g.kv_heads, head_dim=g.head_dim, scale=g.scale, dtype=g.dtype,
                    pool_slots=self.batch.cfg.pool_slots)

    def state_dict(self, device="cpu", stream=None) -> dict:
        """The cached K and V (copied to ``device`` on ``stream``, that of the steps), beside the batch's own state."""
        return _saved(self, self._config(), device, stream)

    def load_state_dict(self, st: dict, stream=None):
        """Restore a ``state_dict`` of a cache of the same heads, head size, scale, type and number of slots."""
        _load(self, st, self._config(), stream)
