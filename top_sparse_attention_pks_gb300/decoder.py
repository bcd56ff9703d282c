"""Owning wrapper around one decode-step shape: outputs, workspace, arguments."""

from __future__ import annotations

import torch

from . import pks


class SparseDecodeStep:
    """Device tensors of one batch plus the output, top-k and workspace buffers.

    ``tensors`` holds device tensors named like the C arguments: seq_lens,
    block_table, q, q_idx, w_idx, kv_k, kv_v, idx_k.  Calling the object runs
    ``pks_decode_step`` on ``stream`` (default: torch's current stream).
    """

    def __init__(self, tensors: dict, k: int, attn_splits: int = 0, topk_mode: int = 0,
                 stream=None, wait_limit: int = 0):
        t = dict(tensors)
        q = t["q"]
        dev = q.device
        self.tensors = t
        self.k = int(k)
        # q: [B, Hq, D], or [B, Nq, Hq, D] with Nq query tokens per request
        self.out = torch.empty(q.shape, dtype=torch.bfloat16, device=dev)
        self.topk_idx = torch.empty(tuple(q.shape[:-2]) + (self.k,), dtype=torch.int32, device=dev)
        probe = pks.make_args(k=self.k, topk_idx=self.topk_idx, out=self.out,
                              attn_splits=attn_splits, topk_mode=topk_mode,
                              wait_limit=wait_limit, **t)
        nbytes = pks.pks_decode_workspace_size(probe)
        self.workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=dev)
        if self.workspace.data_ptr() % 256:
            raise RuntimeError("workspace allocation is not 256-byte aligned")
        self.args = pks.make_args(k=self.k, topk_idx=self.topk_idx, out=self.out,
                                  workspace=self.workspace, attn_splits=attn_splits,
                                  topk_mode=topk_mode, wait_limit=wait_limit, **t)
        pks.pks_decode_workspace_init(self.args, stream)

    def __call__(self, stream=None):
        pks.pks_decode_step(self.args, stream)
        return self.out, self.topk_idx

    def timed(self, events, stream=None):
        pks.pks_decode_step_timed(self.args, events, stream)

    def attention_only(self, stream=None):
        pks.pks_sparse_attention(self.args, stream)

    def scores(self, stream=None) -> torch.Tensor:
        B = self.args.B * max(1, self.args.n_queries)  # one row per query token
        ld = self.args.max_pages * self.args.page_size
        out = torch.zeros((B, ld), dtype=torch.int32, device=self.out.device)
        pks.pks_indexer_scores(self.args, out, stream)
        return out

    def launches(self) -> int:
        """Kernels one step enqueues on the current device."""
        return pks.pks_decode_launches(self.args)

    def device_error(self, stream=None) -> int:
        return pks.pks_decode_device_error(self.args, stream)


class ResidentDecodeStep:
    """The decode step with the KV cache in host memory and an LRU cache of
    its pages in HBM: select (scan + top-k), residency update (miss list),
    fetch of the admitted misses into their slots, attention through the
    table.  ``host_k`` / ``host_v`` are device-accessible (pinned) host tensors
    [num_pages, P, Hkv, D]; ``tensors`` holds the other inputs on the device.
    The slots start with ``init_pages`` (copied in here, as a loader would)."""

    def __init__(self, tensors: dict, host_k: torch.Tensor, host_v: torch.Tensor, k: int,
                 capacity: int, init_pages=(), stream=None):
        t = dict(tensors)
        t["kv_k"], t["kv_v"] = host_k, host_v
        self.step = SparseDecodeStep(t, k, stream=stream)
        self.args = self.step.args
        dev = t["q"].device
        num_pages = host_k.shape[0]
        self.capacity = int(capacity)
        self.slot_k = torch.empty((max(1, capacity),) + tuple(host_k.shape[1:]),
                                  dtype=torch.bfloat16, device=dev)
        self.slot_v = torch.empty_like(self.slot_k)
        self.table = pks.ResidencyTable(num_pages, capacity, init_pages, device=dev, stream=stream)
        init = sorted(set(int(p) for p in init_pages))
        if init:
            idx = torch.tensor(init, dtype=torch.long)
            self.slot_k[: len(init)].copy_(host_k.index_select(0, idx))
            self.slot_v[: len(init)].copy_(host_v.index_select(0, idx))
        self.host_k, self.host_v = host_k, host_v
        self.block_table = t["block_table"]
        self.page_size = host_k.shape[1]
        self.miss = torch.empty(num_pages, dtype=torch.int32, device=dev)
        self.n_miss = torch.zeros(1, dtype=torch.int32, device=dev)

    # the step's four calls, in order
    def select(self, stream=None):
        pks.pks_decode_select(self.args, stream)

    def update(self, stream=None):
        self.table.update(self.step.topk_idx, self.block_table, self.page_size, self.miss,
                          self.n_miss, stream)

    def fetch(self, stream=None):
        self.table.fetch(self.miss, self.n_miss, self.host_k, self.host_v, self.slot_k,
                         self.slot_v, stream)

    def attend(self, stream=None):
        pks.pks_sparse_attention_resident(self.args, self.table.state, self.capacity, self.slot_k,
                                          self.slot_v, stream)

    def __call__(self, stream=None):
        self.select(stream)
        self.update(stream)
        self.fetch(stream)
        self.attend(stream)
        return self.step.out, self.step.topk_idx


class ResidentLayers:
    """Several layers of the decode step through HBM residency tables, the
    miss fetch overlapped layer by layer ("Sparse Attention on GLM5.3 and
    HBM", HiSparse paragraph: the KV cache lives in host memory, an LRU cache
    of it in HBM, misses of the top-k are loaded, the loads overlapped across
    layers).  Every layer has its own KV pools in pinned host memory, its own
    slot table and slot pools, and its own inputs (``tensors`` per layer).

    With ``overlap`` the fetch of layer l runs on a side stream: it waits for
    layer l's residency update (an event) and runs while the main stream
    selects layer l+1 and attends layer l-1; layer l's attention waits for its
    own fetch (a second event).  Without it the four calls of every layer run
    one after the other on the main stream.  Both orders compute the same
    values: each layer's fetch writes only that layer's slots, which only that
    layer's attention reads."""

    def __init__(self, layers: list, k: int, capacity: int, stream=None):
        # layers: dicts with "tensors" (device inputs), "host_k", "host_v"
        # (pinned [num_pages, P, Hkv, D]) and "init_pages"
        self.layers = [ResidentDecodeStep(L["tensors"], L["host_k"], L["host_v"], k, capacity,
                                          L["init_pages"], stream=stream) for L in layers]
        dev = layers[0]["tensors"]["q"].device
        self.side = torch.cuda.Stream(device=dev)
        n = len(self.layers)
        self.updated = [torch.cuda.Event() for _ in range(n)]
        self.fetched = [torch.cuda.Event() for _ in range(n)]

    def __call__(self, stream=None, overlap: bool = True):
        main = stream if stream is not None else torch.cuda.current_stream()
        if not overlap:
            for L in self.layers:
                L(main)
            return [(L.step.out, L.step.topk_idx) for L in self.layers]
        side = self.side
        n = len(self.layers)
        for l in range(n + 1):
            if l < n:
                L = self.layers[l]
                L.select(main)
                L.update(main)
                self.updated[l].record(main)
                side.wait_event(self.updated[l])
                L.fetch(side)
                self.fetched[l].record(side)
            if l > 0:  # the previous layer's attention, once its own fetch is done
                main.wait_event(self.fetched[l - 1])
                self.layers[l - 1].attend(main)
        return [(L.step.out, L.step.topk_idx) for L in self.layers]


class MlaAttention:
    """Sparse MLA in MQA mode over given selections: ``pks_mla_sparse_attention``
    with its own output and workspace.  q [B, H, d + r], kv [num_pages, P, d + r]
    (bf16), topk_idx [B, k] (int32), d = 512 latent values."""

    def __init__(self, seq_lens, block_table, topk_idx, q, kv, sm_scale: float = 0.0,
                 trim: bool = False, splits: int = 0, stream=None, wait_limit: int = 0):
        dev = q.device
        self.out = torch.empty((q.shape[0], q.shape[1], 512), dtype=torch.bfloat16, device=dev)
        probe = pks.make_mla_args(seq_lens=seq_lens, block_table=block_table, topk_idx=topk_idx,
                                  q=q, kv=kv, out=self.out, sm_scale=sm_scale, trim=trim,
                                  splits=splits)
        nbytes = pks.pks_mla_workspace_size(probe)
        self.workspace = torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=dev)
        self.args = pks.make_mla_args(seq_lens=seq_lens, block_table=block_table,
                                      topk_idx=topk_idx, q=q, kv=kv, out=self.out,
                                      workspace=self.workspace, sm_scale=sm_scale, trim=trim,
                                      splits=splits, wait_limit=wait_limit)
        self._keep = (seq_lens, block_table, topk_idx, q, kv)

    def __call__(self, stream=None):
        pks.pks_mla_sparse_attention(self.args, stream)
        return self.out

    def device_error(self, stream=None) -> int:
        return pks.pks_mla_device_error(self.args, stream)


def _select_args(t: dict, topk_idx, num_pages: int, page_size: int, topk_mode: int):
    """Selection arguments: the indexer and top-k fields of pks_decode_args (the GQA
    attention fields stay unset; select does not read them)."""
    a = pks.pks_decode_args()
    B = t["seq_lens"].shape[0]
    q_idx = t["q_idx"]
    if q_idx.dim() != topk_idx.dim() + 1:
        raise ValueError("q_idx must be [B, Hi, Di], or [B, Nq, Hi, Di] where q has Nq")
    Hi, Di = q_idx.shape[-2:]
    a.B, a.Hq, a.Hkv, a.D, a.Hi, a.Di = int(B), 1, 1, 64, int(Hi), int(Di)
    a.page_size, a.max_pages = int(page_size), int(t["block_table"].shape[1])
    a.num_pages, a.k = int(num_pages), int(topk_idx.shape[-1])
    a.seq_lens = pks._dptr(t["seq_lens"], torch.int32, "seq_lens")
    a.block_table = pks._dptr(t["block_table"], torch.int32, "block_table")
    f8 = torch.float8_e4m3fn  # (taken by their bit patterns, as in make_args)
    q_idx, idx_k = (x.view(torch.int8) if x.dtype == f8 else x for x in (q_idx, t["idx_k"]))
    a.q_idx = pks._dptr(q_idx, torch.int8, "q_idx")
    a.w_idx = pks._dptr(t.get("w_idx"), torch.int32, "w_idx")
    a.idx_k = pks._dptr(idx_k, torch.int8, "idx_k")
    a.topk_idx = pks._dptr(topk_idx, torch.int32, "topk_idx")
    a.topk_mode = int(topk_mode)
    # real-valued head weights and FP8 e4m3 queries/keys (DSA's indexer)
    if t.get("w_idx_f") is not None:
        a.w_idx_f = pks._dptr(t["w_idx_f"], torch.float32, "w_idx_f")
    a.idx_fp8 = 1 if t.get("idx_fp8") else 0
    return a


def _select_workspace(a, device, stream) -> torch.Tensor:
    nbytes = pks.pks_decode_workspace_size(a)
    with pks._on_stream(stream):
        ws = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
    a.workspace = ws.data_ptr()
    a.workspace_bytes = ws.numel()
    pks.pks_decode_workspace_init(a, stream)
    return ws


class MlaDecodeStep:
    """The DSA decode step with MLA attention (``pks_mla_decode_step``): indexer
    scan and top-k, then the sparse MLA over the selected tokens.
    ``tensors``: seq_lens, block_table, q_idx, w_idx, idx_k as for the GQA
    step, plus q [B, H, d + r] and kv [num_pages, P, d + r] (bf16)."""

    def __init__(self, tensors: dict, k: int, topk_mode: int = 0, splits: int = 0,
                 sm_scale: float = 0.0, stream=None):
        t = dict(tensors)
        q, kv = t["q"], t["kv"]
        dev = q.device
        B = q.shape[0]
        self.k = int(k)
        self.topk_idx = torch.empty((B, self.k), dtype=torch.int32, device=dev)
        npages, P, _ = kv.shape
        a = _select_args(t, self.topk_idx, npages, P, topk_mode)
        self.select_workspace = _select_workspace(a, dev, stream)
        self.select_args = a
        self.attention = MlaAttention(t["seq_lens"], t["block_table"], self.topk_idx, q, kv,
                                      sm_scale=sm_scale, trim=True, splits=splits)
        self.out = self.attention.out
        self.tensors = t

    def select(self, stream=None):
        pks.pks_decode_select(self.select_args, stream)
        return self.topk_idx

    def __call__(self, stream=None):
        pks.pks_mla_decode_step(self.select_args, self.attention.args, stream)
        return self.out, self.topk_idx


class PrefixAttention:
    """Dense decode attention of a batch whose requests alias the pages of shared
    prefixes (``pks_prefix_plan`` and ``pks_prefix_attention``): a prefix's K/V
    take part once for all requests of its group.  q [B, Hq, D] or
    [B, Nq, Hq, D] (query tokens at the end of each request, ``causal`` among
    themselves), kv_k / kv_v [num_pages, P, Hkv, D] (bf16), prefix_group [B]
    (int32, negative: none) or None, min_shared: tokens from which on a prefix is
    taken once (0: when that is expected to be faster).  Owns ``out``, ``lse`` (when
    asked for) and the workspace, allocated and cleared on ``stream`` (default: torch's
    current stream): calls on another stream have to wait for that one.

    Calling the object plans and attends.  ``plan`` alone is needed whenever
    lengths, table or groups have changed; ``attend`` serves further layers,
    ``attend(q, kv_k, kv_v)`` with tensors of the same shapes, which later calls
    keep to (a call that is refused leaves those before it in place).  One object's calls run one after another: their workspace is one."""

    def __init__(self, seq_lens, block_table, q, kv_k, kv_v, prefix_group=None,
                 causal: bool = False, sm_scale: float = 0.0, lse: bool = False,
                 wait_limit: int = 0, min_shared: int = 0, stream=None):
        pks._on_current_device(seq_lens, block_table, q, kv_k, kv_v, prefix_group)
        dev = q.device
        with pks._on_stream(stream):
            self.out = torch.empty(q.shape, dtype=torch.bfloat16, device=dev)
            self.lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=dev) if lse else None
        kw = dict(seq_lens=seq_lens, block_table=block_table, q=q, kv_k=kv_k, kv_v=kv_v,
                  prefix_group=prefix_group, causal=causal, sm_scale=sm_scale, out=self.out,
                  lse=self.lse, wait_limit=wait_limit, min_shared=min_shared)
        nbytes = pks.pks_prefix_workspace_size(pks.make_prefix_args(**kw))
        with pks._on_stream(stream):
            self.workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=dev)
            self.workspace[:256].zero_()
        self.args = pks.make_prefix_args(workspace=self.workspace, **kw)
        self._keep = [seq_lens, block_table, prefix_group, q, kv_k, kv_v]

    def plan(self, stream=None):
        pks._on_current_device(self.out)
        pks.pks_prefix_plan(self.args, stream)

    def attend(self, q=None, kv_k=None, kv_v=None, stream=None):
        new = {}  # all of them are looked at before any is taken over
        for at, (name, t) in enumerate((("q", q), ("kv_k", kv_k), ("kv_v", kv_v)), 3):
            if t is None:
                continue
            was = self._keep[at]
            if t.shape != was.shape or t.device != was.device:
                raise ValueError(f"{name} must have the shape and device it was planned with")
            new[name] = at, t, pks._dptr(t, torch.bfloat16, name)
        pks._on_current_device(self.out)
        old = {name: getattr(self.args, name) for name in new}
        for name, (_, _, ptr) in new.items():
            setattr(self.args, name, ptr)
        try:
            pks.pks_prefix_attention(self.args, stream)
        except BaseException:
            for name, ptr in old.items():
                setattr(self.args, name, ptr)
            raise
        for at, t, _ in new.values():
            self._keep[at] = t
        return self.out

    def __call__(self, stream=None):
        pks._on_current_device(self.out)
        pks.pks_prefix_plan(self.args, stream)
        pks.pks_prefix_attention(self.args, stream)
        return self.out

    def device_error(self, stream=None) -> int:
        return pks.pks_prefix_device_error(self.args, stream)


class PageTable:
    """A block table whose page sharing is kept on the device (``pks_pages_*``):
    holders of every page and the free pages.  ``seq_lens`` [B] and
    ``block_table`` [B, max_pages] (int32, e.g. from ``Pool.build_block_table``)
    stay the caller's tensors and are updated in place; ``pools`` are the paged
    tensors [num_pages, page_size, ...] whose rows move with the pages.  All
    calls run on ``stream`` (default: torch's current stream), one after another;
    calls on another stream than the one it was built on have to wait for that one.

    ``refs`` [num_pages], ``n_free`` and ``granted`` (0-dim) are views of the
    state and ``page_map`` [num_pages] is what the last ``compact`` wrote."""

    def __init__(self, seq_lens, block_table, num_pages: int, page_size: int, pools=(),
                 state=None, stream=None):
        pks._on_current_device(seq_lens, block_table, state, *pools)
        dev = block_table.device
        nbytes = pks.pks_pages_state_bytes(num_pages)
        with pks._on_stream(stream):
            if state is None:
                state = torch.empty(nbytes, dtype=torch.uint8, device=dev)
            self.page_map = torch.empty(int(num_pages), dtype=torch.int32, device=dev)
        self.state = state
        self.seq_lens, self.block_table, self.pools = seq_lens, block_table, list(pools)
        self.args = pks.make_pages_args(seq_lens=seq_lens, block_table=block_table,
                                        num_pages=num_pages, page_size=page_size, state=state,
                                        pools=self.pools)
        off = pks.pks_pages_offsets(num_pages)["ref"]
        header = state[:256].view(torch.int32)
        self.n_free, self.granted = header[2], header[6]
        self.refs = state[off: off + 4 * int(num_pages)].view(torch.int32)
        pks.pks_pages_init(self.args, stream)

    def fork(self, src_rows, dst_rows, n_tokens=None, stream=None):
        """Rows ``dst_rows`` (empty) become aliases of ``src_rows``' first tokens."""
        pks._on_current_device(self.state, src_rows, dst_rows, n_tokens)
        pks.pks_pages_fork(self.args, src_rows, dst_rows, n_tokens, stream)

    def extend(self, add, stream=None):
        """Every row grows by ``add`` [B] tokens, or none does (``granted`` is 0)."""
        pks._on_current_device(self.state, add)
        pks.pks_pages_extend(self.args, add, stream)

    def free(self, rows, keep=None, stream=None):
        """Truncate ``rows`` to ``keep`` tokens (default 0: give them back)."""
        pks._on_current_device(self.state, rows, keep)
        pks.pks_pages_free(self.args, rows, keep, stream)

    def compact(self, stream=None):
        """Move the held pages to the lowest ids; returns the map of page ids."""
        pks._on_current_device(self.state)
        pks.pks_pages_compact(self.args, self.page_map, stream)
        return self.page_map

    def device_error(self, stream=None) -> int:
        return pks.pks_pages_device_error(self.args, stream)


class Q4Cache:
    """A paged K/V cache held in 4 bits (``pks_q4_write`` and ``pks_q4_read``): the pools
    ``k`` and ``v``, uint8 [num_pages, page_size, token_bytes], which move with the pages of a
    ``PageTable(pools=[cache.k, cache.v])``.  Allocated, with zeros, on ``stream`` (default:
    torch's current stream): calls on another stream have to wait for that one.

    Rows come packed: rows starts[b] .. starts[b + 1] of k and v [n, Hkv, D] (bfloat16,
    float16 or float32, any row and head strides of 16 bytes) are the last tokens of request
    b, whose length counts them.  Rows from starts[B] on are left alone."""

    def __init__(self, num_pages: int, page_size: int, Hkv: int, D: int, device=None, stream=None):
        row = pks.pks_q4_token_bytes(Hkv, D)
        if device is None:
            device = torch.device("cuda", torch.cuda.current_device())
        with pks._on_stream(stream):
            shape = (int(num_pages), int(page_size), row)
            self._k = torch.zeros(shape, dtype=torch.uint8, device=device)
            self._v = torch.zeros(shape, dtype=torch.uint8, device=device)
            self._error = torch.zeros(1, dtype=torch.int32, device=device)
        self.Hkv, self.D = int(Hkv), int(D)
        pks._on_current_device(self.k)
        self._base = pks._q4_rows_base(self.k, self.v, Hkv, D, self.error)

    # (read-only, as _base holds their addresses)
    k = property(lambda self: self._k)
    v = property(lambda self: self._v)
    error = property(lambda self: self._error)

    def _args(self, k, v, seq_lens, block_table, starts):
        pks._on_current_device(self.k, k, v, seq_lens, block_table, starts)
        a = pks.pks_q4_rows_args.from_buffer_copy(self._base)  # (calls may come from two threads)
        return pks._q4_rows_fill(a, k, v, seq_lens, block_table, starts)

    def write(self, k, v, seq_lens, block_table, starts, stream=None):
        """Quantise the rows of k and v into their pages."""
        pks.pks_q4_write(self._args(k, v, seq_lens, block_table, starts), stream)

    def read(self, seq_lens, block_table, starts, k, v, stream=None):
        """Fill k and v with the values that the cached rows stand for."""
        pks.pks_q4_read(self._args(k, v, seq_lens, block_table, starts), stream)
        return k, v

    def device_error(self, stream=None) -> int:
        """The last row's fault since this was last asked (1 page, 2 starts, 3 length), or 0;
        synchronises the stream."""
        with pks._on_stream(stream):
            code = int(self.error.item())
            if code:
                self.error.zero_()
        return code


class Q4Attention:
    """Dense decode attention over a ``Q4Cache`` (``pks_q4_attention``): q [B, Hq, D] or
    [B, Nq, Hq, D] (query tokens at the end of each request, ``causal`` among themselves).
    Owns ``out``, ``lse`` (when asked for) and the workspace, allocated and cleared on
    ``stream`` (default: torch's current stream): calls on another stream have to wait for
    that one.  ``attend(q, cache)`` serves further layers with tensors of the same shapes,
    which later calls keep to (a call that is refused leaves those before it in place).  One
    object's calls run one after another: their workspace is one."""

    _entry = staticmethod(pks.pks_q4_attention)

    def __init__(self, seq_lens, block_table, q, cache: Q4Cache, causal: bool = False,
                 sm_scale: float = 0.0, lse: bool = False, wait_limit: int = 0, stream=None):
        self._build(stream, lse, cache, q, seq_lens=seq_lens, block_table=block_table,
                    causal=causal, sm_scale=sm_scale, wait_limit=wait_limit)

    def _build(self, stream, lse, cache, q, **kw):
        pks._on_current_device(q, cache.k, kw["seq_lens"], kw["block_table"], kw.get("topk_idx"))
        if q.shape[-1] != cache.D:
            raise ValueError("q and the cache differ in D")
        dev = q.device
        with pks._on_stream(stream):
            self.out = torch.empty(q.shape, dtype=torch.bfloat16, device=dev)
            self.lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=dev) if lse else None
        kw.update(q=q, pool_k=cache.k, pool_v=cache.v, Hkv=cache.Hkv, out=self.out, lse=self.lse)
        nbytes = pks.pks_q4_workspace_size(pks.make_q4_attention_args(**kw))
        with pks._on_stream(stream):
            self.workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=dev)
            self.workspace[:256].zero_()
        self.args = pks.make_q4_attention_args(workspace=self.workspace, **kw)
        self._keep = [q, cache, kw["seq_lens"], kw["block_table"], kw.get("topk_idx")]

    def attend(self, q=None, cache=None, stream=None):
        was_q, was = self._keep[:2]
        if q is not None and (q.shape != was_q.shape or q.device != was_q.device):
            raise ValueError("q must have the shape and device it was built with")
        if cache is not None and (cache.k.shape != was.k.shape or cache.k.device != was.k.device
                                  or (cache.Hkv, cache.D) != (was.Hkv, was.D)):
            raise ValueError("the cache must have the shape and device it was built with")
        new = {}
        if q is not None:
            new["q"] = pks._dptr(q, torch.bfloat16, "q")
        if cache is not None:
            new["pool_k"] = pks._dptr(cache.k, torch.uint8, "pool_k")
            new["pool_v"] = pks._dptr(cache.v, torch.uint8, "pool_v")
        pks._on_current_device(self.out)
        old = {name: getattr(self.args, name) for name in new}
        for name, ptr in new.items():
            setattr(self.args, name, ptr)
        try:
            self._entry(self.args, stream)
        except BaseException:
            for name, ptr in old.items():
                setattr(self.args, name, ptr)
            raise
        if q is not None:
            self._keep[0] = q
        if cache is not None:
            self._keep[1] = cache
        return self.out

    def __call__(self, stream=None):
        pks._on_current_device(self.out)
        self._entry(self.args, stream)
        return self.out

    def device_error(self, stream=None) -> int:
        return pks.pks_q4_device_error(self.args, stream)


class Q4SparseAttention(Q4Attention):
    """Attention over selected tokens of a ``Q4Cache`` (``pks_q4_sparse_attention``): topk_idx
    [B, k], or [B, Nq, k] with q [B, Nq, Hq, D] (int32 positions, -1: none).  ``trim``: every
    list holds its entries first, and no more than its request has tokens."""

    _entry = staticmethod(pks.pks_q4_sparse_attention)

    def __init__(self, seq_lens, block_table, topk_idx, q, cache: Q4Cache, sm_scale: float = 0.0,
                 trim: bool = False, lse: bool = False, wait_limit: int = 0, stream=None):
        self._build(stream, lse, cache, q, seq_lens=seq_lens, block_table=block_table,
                    topk_idx=topk_idx, trim=trim, sm_scale=sm_scale, wait_limit=wait_limit)


class Q4DecodeStep:
    """The sparse decode step over a ``Q4Cache`` (``pks_q4_decode_step``): indexer scan and
    top-k, then attention over the selected tokens.  ``tensors``: seq_lens, block_table, q,
    q_idx, w_idx (or w_idx_f), idx_k, idx_fp8 as for ``SparseDecodeStep``."""

    def __init__(self, tensors: dict, cache: Q4Cache, k: int, topk_mode: int = 0,
                 sm_scale: float = 0.0, lse: bool = False, stream=None):
        t = dict(tensors)
        q = t["q"]
        self.k = int(k)
        with pks._on_stream(stream):
            self.topk_idx = torch.empty(tuple(q.shape[:-2]) + (self.k,), dtype=torch.int32,
                                        device=q.device)
        num_pages, page_size = cache.k.shape[:2]
        if t["q_idx"].shape[:-2] != q.shape[:-2]:
            raise ValueError("q_idx must be [B, Hi, Di] or [B, Nq, Hi, Di] like q")
        Hi, Di = t["q_idx"].shape[-2:]
        if tuple(t["idx_k"].shape) != (num_pages, page_size, Di):
            raise ValueError("idx_k must be [num_pages, page_size, Di] of the cache's pages")
        if t["seq_lens"].shape != q.shape[:1] or t["block_table"].dim() != 2 or \
                t["block_table"].shape[0] != q.shape[0]:
            raise ValueError("block_table must be [B, max_pages] and seq_lens [B]")
        if t.get("w_idx") is not None and t["w_idx"].numel() != Hi:
            raise ValueError("w_idx must be [Hi]")
        if t.get("w_idx_f") is not None and \
                t["w_idx_f"].numel() != t["q_idx"].shape[:-1].numel():
            raise ValueError("w_idx_f must be [B, Hi]")
        a = _select_args(t, self.topk_idx, num_pages, page_size, topk_mode)
        if q.dim() == 4:
            a.n_queries = int(q.shape[1])
        pks._on_current_device(q, cache.k, *(t.get(x) for x in (
            "seq_lens", "block_table", "q_idx", "idx_k", "w_idx", "w_idx_f")))
        self.select_workspace = _select_workspace(a, q.device, stream)
        self.select_args = a
        self.attention = Q4SparseAttention(t["seq_lens"], t["block_table"], self.topk_idx, q,
                                           cache, sm_scale=sm_scale, trim=True, lse=lse,
                                           stream=stream)
        self.out, self.lse = self.attention.out, self.attention.lse
        self.tensors = t

    def select(self, stream=None):
        pks._on_current_device(self.topk_idx)
        pks.pks_decode_select(self.select_args, stream)
        return self.topk_idx

    def __call__(self, stream=None):
        pks._on_current_device(self.out)
        pks.pks_q4_decode_step(self.select_args, self.attention.args, stream)
        return self.out, self.topk_idx

    def device_error(self, stream=None) -> int:
        """Of the selection, else of the attention."""
        return pks.pks_decode_device_error(self.select_args, stream) or \
            self.attention.device_error(stream)
