"""Device state of one IndexShare group and its per-step schedule.

The schedule is the one of the GLM-5.2 shared-Indexer KV Cache Offload page,
§4.4 (SFA first, refill later) and §5.1 (one plan per group, per-layer serve,
refill on a side stream synchronised by events, metadata update at the group's
last layer). It is enqueued by the library's dsa_group_step in one native call
per step:

  main stream   : ts_topk -> [wait refilled of the previous step] -> dsa_plan
                  -> signal planned
                  -> for each layer l: [wait gathered[l]] -> sfa_mla_decode(l)
  gather stream : [wait planned] -> one gather launch for layers 0..3; the
                  kernel signals gathered[l] as soon as layer l's rows are in
  side stream   : for each layer l: [wait gathered[l]] -> dsa_refill_pool(l)
                  (the last layer also updates tags and FIFO pointers)
                  -> signal refilled

Waits are stream memory operations on device words (the library's `sync`
words), polled by the GPU's front end in HBM; no kernel waits on another.

The plan is shared by the group, so every layer's gather can start as soon as
it exists: the host-link transfers of layer l+1 overlap the attention of
layer l, and each layer's attention still starts the moment its own rows are
in (SFA first); each refill runs beside its layer's attention on a few SMs. Memory and streams come from PyTorch; this module only fills
the descriptor; the arithmetic runs in libdsakv's kernels.
"""
from __future__ import annotations

import ctypes
import math

import numpy as np
import torch

from . import _abi as abi

D = 576
DV = 512


def plan_metrics(miss_rows, miss_count, miss_ids, install, k: int, S: int) -> dict:
    """Per-request counts of one step's plan, from its outputs as host arrays
    ([B], [B], [B][k], [B][k] or None): positions that hit (k minus the
    positions that miss, repeats included), distinct misses, misses installed
    (install code 1 or 2) and overflow sets (sets that missed more tokens than
    they have ways: their earliest misses are not installed). Each a list of
    B ints; installs and overflow sets are None without an install array
    (the reuse policy installs nothing)."""
    miss_rows = np.asarray(miss_rows)
    miss_count = np.asarray(miss_count)
    B = miss_count.shape[0]
    out = {"hits": [int(k - miss_rows[b]) for b in range(B)],
           "misses": [int(miss_count[b]) for b in range(B)],
           "installs": None, "overflow_sets": None}
    if install is not None:
        install = np.asarray(install)
        miss_ids = np.asarray(miss_ids)
        out["installs"], out["overflow_sets"] = [], []
        for b in range(B):
            M = int(miss_count[b])
            codes = install[b, :M]
            out["installs"].append(int(np.count_nonzero(codes)))
            dropped = miss_ids[b, :M][codes == 0]
            out["overflow_sets"].append(int(np.unique(dropped % S).size))
    return out


class PinnedHost:
    """A page-locked host buffer the device reads and writes in place, seen as
    a numpy array (zero-filled). kind="alloc" (default): ts_host_alloc memory,
    which the SMs read and write fastest (ts_copy, gathers); kind="register":
    numpy memory registered with ts_host_register, for buffers that DMA copies
    read (on GB300, zero-copy reads stalled for a while after a large DMA from
    ts_host_alloc memory; not after one from registered memory)."""

    def __init__(self, shape, dtype, kind: str = "alloc"):
        nbytes = int(np.prod(shape)) * np.dtype(dtype).itemsize
        self.kind = kind
        self._host = 0
        self.dev = 0
        if nbytes == 0:
            self.array = np.zeros(shape, dtype=dtype)
        elif kind == "alloc":
            self._host, self.dev = abi.ts_host_alloc(nbytes)
            buf = (ctypes.c_uint8 * nbytes).from_address(self._host)
            self.array = np.frombuffer(buf, dtype=dtype).reshape(shape)
            self.array[...] = 0
        elif kind == "register":
            self.array = np.zeros(shape, dtype=dtype)
            self._host = self.array.ctypes.data
            self.dev = abi.ts_host_register(self._host, nbytes)
        else:
            raise ValueError(kind)

    def tensor(self) -> torch.Tensor:
        return torch.from_numpy(self.array)

    def close(self):
        if self._host:
            if self.kind == "alloc":
                self.array = None
                abi.ts_host_free(self._host)
            else:
                abi.ts_host_unregister(self._host)
        self._host = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class HostKV:
    """Full latent KV of a group in pinned host memory, read in place by the
    gather: uint16 (bf16 bits) [layers][B][ctx_stride][576]. By default the
    memory comes from ts_host_alloc (the gathers read it fastest); a caller's
    own C-contiguous array is registered instead."""

    def __init__(self, layers: int, B: int, ctx_stride: int, array: np.ndarray | None = None):
        shape = (layers, B, ctx_stride, D)
        self.layers, self.B, self.ctx_stride = layers, B, ctx_stride
        self.layer_bytes = B * ctx_stride * D * 2
        nbytes = layers * self.layer_bytes
        if array is None:
            self._host, self.dev = abi.ts_host_alloc(nbytes)
            self._owned = True
            buf = (ctypes.c_uint16 * (nbytes // 2)).from_address(self._host)
            self.array = np.frombuffer(buf, dtype=np.uint16).reshape(shape)
        else:
            assert array.shape == shape and array.dtype == np.uint16
            assert array.flags["C_CONTIGUOUS"]
            self.array = array
            self._host = array.ctypes.data
            self.dev = abi.ts_host_register(self._host, array.nbytes)
            self._owned = False

    def layer_ptr(self, l: int) -> int:
        return self.dev + l * self.layer_bytes

    def close(self):
        if self._host:
            self.array = None
            if self._owned:
                abi.ts_host_free(self._host)
            else:
                abi.ts_host_unregister(self._host)
            self._host = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class StepTiming:
    """CUDA timing events for the launches of one step, created (and recorded
    once, which makes them valid) ahead of use, in the order dsa_group_step
    fills them: top-k, plan, gather (every layer), sfa[l], refill[l].
    light=True hands the step only the top-k's start, the gather's start and
    end and the last attention's end (the step's span and the gather's time);
    the other entries stay unrecorded."""

    def __init__(self, layers: int, stream=None, refills: bool = True, light: bool = False):
        self.layers = layers
        self.refills = refills  # the reuse policy runs no refill
        self.light = light
        n = 2 * (3 + 2 * layers)
        st = torch.cuda.current_stream() if stream is None else stream
        self.events = [torch.cuda.Event(enable_timing=True) for _ in range(n)]
        for e in self.events:
            e.record(st)
        keep = {0, 4, 5, 2 * (3 + layers - 1) + 1} if light else set(range(n))
        self.array = (ctypes.c_void_p * n)(*[e.cuda_event if i in keep else None
                                             for i, e in enumerate(self.events)])
        self.with_topk = True

    def ms(self) -> dict:
        """name -> per-launch milliseconds (after the step completed); with
        light timing the gather only."""
        L = self.layers
        ev = self.events

        def pair(i):
            return ev[2 * i].elapsed_time(ev[2 * i + 1])

        if self.light:
            return {"gather": [pair(2)]}

        out = {"topk": [pair(0)] if self.with_topk else [], "plan": [pair(1)]}
        out["gather"] = [pair(2)]
        out["sfa"] = [pair(3 + l) for l in range(L)]
        out["refill"] = [pair(3 + L + l) for l in range(L)] if self.refills else []
        return out

    def spans(self, t0) -> dict:
        """name -> [(start, end)] in microseconds after event t0."""
        L = self.layers
        ev = self.events

        def span(i):
            return (t0.elapsed_time(ev[2 * i]) * 1e3, t0.elapsed_time(ev[2 * i + 1]) * 1e3)

        out = {"topk": [span(0)] if self.with_topk else [], "plan": [span(1)]}
        out["gather"] = [span(2)]
        out["sfa"] = [span(3 + l) for l in range(L)]
        out["refill"] = [span(3 + L + l) for l in range(L)] if self.refills else []
        return out


class DecodeGroup:
    """Pool state and buffers for B requests of one IndexShare group.

    policy "fifo": the set-associative FIFO pool of S sets x W ways;
    policy "lru": a fully associative pool of S x W entries, least recently
    used first (tags and the slots' recency order per request);
    policy "reuse": the base design's adjacent-step reuse, where the device
    keeps only the previous step's selection (S and W are then unused).
    After a step, `ids` and `sel` hold that step's ids and selection.

    layout "selection": every layer's rows are gathered into `sel`, which the
    attention reads; layout "staged" (FIFO or LRU): the attention reads its rows
    straight from the pool, which then holds P + k rows per request (rows P..
    stage the step's misses at their first positions) and `sel` is None.
    With `streamed` (staged only; B <= 1024) each layer's attention starts
    while the gather runs, every CTA waiting for its own request's rows, each
    layer on a stream of its own (launched once the previous layer's CTAs all
    run); otherwise each layer's attention waits for the whole layer."""

    def __init__(self, B: int, layers: int, k: int, S: int, W: int, H: int,
                 ctx_len, ctx_stride: int, host: HostKV, scale: float | None = None,
                 device: str = "cuda", max_ctx: int | None = None, policy: str = "fifo",
                 layout: str = "selection", streamed: bool = True):
        if policy not in ("fifo", "reuse", "lru"):
            raise ValueError(policy)
        if layout not in ("selection", "staged") or (layout == "staged" and policy == "reuse"):
            raise ValueError(layout)
        self.policy = policy
        self.layout = layout
        self.B, self.L, self.k, self.S, self.W, self.H = B, layers, k, S, W, H
        self.P = S * W
        self.ctx_stride = ctx_stride
        self.scale = 1.0 / math.sqrt(D) if scale is None else scale
        self.host = host
        dev = torch.device(device)
        i32 = dict(dtype=torch.int32, device=dev)
        self.ctx_len = torch.as_tensor(np.asarray(ctx_len, np.int32), **i32)
        self.max_ctx = int(np.max(ctx_len)) if max_ctx is None else max_ctx
        # pool state: data per (layer, request), metadata per request (the
        # reuse policy keeps the previous step's ids and selection instead)
        reuse = policy == "reuse"
        P = 1 if reuse else self.P
        rows = P + k if layout == "staged" else P
        self.pool = torch.zeros((layers, B, rows, D), dtype=torch.int16, device=dev)
        self.tags = torch.full((B, P), -1, **i32)
        self.fifo_ptr = torch.zeros((B, S if policy == "fifo" else 1), **i32)
        # LRU pool: each request's slots from least to most recently used
        # (the identity order of a cold pool)
        self.lru_order = (torch.arange(P, **i32).repeat(B, 1) if policy == "lru"
                          else torch.zeros((1,), **i32))
        # plan outputs
        self.ids = torch.empty((B, k), **i32)
        self.src_map = torch.empty((B, k), **i32)
        self.miss_ids = torch.empty((B, k), **i32)
        self.miss_pos = torch.empty((B, k), **i32)
        self.victim = torch.empty((B, k), **i32)
        self.install = torch.empty((B, k), dtype=torch.uint8, device=dev)
        self.miss_count = torch.zeros((B,), **i32)
        self.miss_rows = torch.zeros((B,), **i32)
        self.ptr_next = torch.empty((B, S if policy == "fifo" else 1), **i32)
        # per-layer selection buffers and attention outputs
        self.sel = (None if layout == "staged"
                    else torch.empty((layers, B, k, D), dtype=torch.int16, device=dev))
        if reuse:
            self.prev_ids = torch.full((B, k), -1, **i32)
            self.prev_sel = torch.zeros((layers, B, k, D), dtype=torch.int16, device=dev)
            self._bufs = {t.data_ptr(): t for t in (self.ids, self.prev_ids, self.sel,
                                                    self.prev_sel)}
        self.out = torch.empty((layers, B, H, DV), dtype=torch.bfloat16, device=dev)
        self.lse = torch.empty((layers, B, H), dtype=torch.float32, device=dev)
        # workspaces and the device error word
        self.topk_ws_bytes = abi.ts_topk_workspace_size(B, self.max_ctx, k)
        streamed = layout == "staged" and streamed
        # streamed: one attention workspace per layer and a stream per layer
        # (the library runs the layers' attention side by side where one
        # layer's CTAs fill at most half of the SMs, else on the main stream)
        self.sfa_ws_bytes = abi.sfa_workspace_size(B, H, k) * (layers if streamed else 1)
        self.topk_ws = torch.empty(self.topk_ws_bytes, dtype=torch.uint8, device=dev)
        self.sfa_ws = torch.empty(self.sfa_ws_bytes, dtype=torch.uint8, device=dev)
        self.err = torch.zeros((1,), **i32)
        # streams and events
        # the critical path (top-k, plan, attention) has the higher priority:
        # when CTAs of several kernels wait for SMs, its CTAs go first
        self.main = torch.cuda.Stream(device=dev, priority=-1)
        self.gstream = torch.cuda.Stream(device=dev, priority=0)
        self.side = torch.cuda.Stream(device=dev, priority=0)
        self.lstreams = ([torch.cuda.Stream(device=dev, priority=-1) for _ in range(layers)]
                         if streamed else [])
        self._lstream_handles = (ctypes.c_void_p * max(1, layers))(
            *[st.cuda_stream for st in self.lstreams])
        # cross-stream signals: device words written and waited on by the
        # streams themselves (zero before the first step)
        self.sync = torch.zeros((5 + 3 * layers,), **i32)
        # staged layout: per (layer, request) arrival counts of the gather, so
        # that each attention CTA starts once its own request's rows are in;
        # the gather's start words; each layer's started attention CTAs
        self.arrived = (torch.zeros((layers * B + 3 + layers,), **i32)
                        if streamed else None)
        # device staging of dsa_group_step_host (made on first use)
        self._io_scores = None
        self._io_q = None
        self.desc = self._descriptor()

    def staged_rows(self, l: int, b: int):
        """Staged layout: the rows the step staged for request b of layer l
        (int16 [k][576]; row j holds the host row of a miss first selected at
        position j, the other rows are stale)."""
        return self.pool[l, b, self.P:]

    def timing(self, light: bool = False) -> StepTiming:
        """Timing events for one step of this group (see StepTiming)."""
        return StepTiming(self.L, self.main, refills=self.policy == "fifo", light=light)

    def _descriptor(self):
        d = abi.DsaGroup()
        d.B, d.layers, d.k, d.S, d.W, d.H = self.B, self.L, self.k, self.S, self.W, self.H
        d.max_ctx, d.ctx_stride, d.scale = self.max_ctx, self.ctx_stride, self.scale
        d.ctx_len = self.ctx_len.data_ptr()
        d.pool, d.pool_tags, d.fifo_ptr = (self.pool.data_ptr(), self.tags.data_ptr(),
                                           self.fifo_ptr.data_ptr())
        d.host_kv = self.host.dev
        for name in ("ids", "src_map", "miss_ids", "miss_pos", "victim", "install",
                     "miss_count", "miss_rows", "ptr_next", "sel", "out", "lse"):
            t = getattr(self, name)
            setattr(d, name, 0 if t is None else t.data_ptr())
        d.layout = abi.DSA_LAYOUT_STAGED if self.layout == "staged" else abi.DSA_LAYOUT_SELECTION
        d.topk_ws, d.topk_ws_bytes = self.topk_ws.data_ptr(), self.topk_ws_bytes
        d.sfa_ws, d.sfa_ws_bytes = self.sfa_ws.data_ptr(), self.sfa_ws_bytes
        d.err = self.err.data_ptr()
        d.arrived = 0 if self.arrived is None else self.arrived.data_ptr()
        d.layer_streams = (ctypes.addressof(self._lstream_handles) if self.lstreams else 0)
        if self.policy == "lru":
            d.policy = abi.DSA_POLICY_LRU
            d.lru_order = self.lru_order.data_ptr()
        if self.policy == "reuse":
            d.policy = abi.DSA_POLICY_REUSE
            d.prev_ids = self.prev_ids.data_ptr()
            d.prev_sel = self.prev_sel.data_ptr()
        d.main_stream = self.main.cuda_stream
        d.gather_stream = self.gstream.cuda_stream
        d.side_stream = self.side.cuda_stream
        d.sync = self.sync.data_ptr()
        d.step = 0
        return d

    # -- the step --------------------------------------------------------
    def step(self, scores: torch.Tensor, q: torch.Tensor, ids: torch.Tensor | None = None,
             timing: StepTiming | None = None) -> None:
        """Enqueue one decode step (one native call). scores: float32
        [B][ctx_stride] (device); q: bf16 bits [layers][B][H][576] (device).
        With `ids` given (int32 [B][k]), the top-k is skipped and those ids are
        planned. `timing`, when given, receives (start, end) events around
        every launch."""
        if timing is not None:
            timing.with_topk = ids is None
        abi.check(abi.dsa_group_step(self.desc, scores, q, ids,
                                     None if timing is None else timing.array),
                  "dsa_group_step")
        if self.policy == "reuse":
            # the step swapped its buffers: this step's ids and selection are
            # now the descriptor's previous ones
            self.ids = self._bufs[self.desc.prev_ids]
            self.sel = self._bufs[self.desc.prev_sel]

    def step_host(self, scores_h: int, q_h: int, out_h: int,
                  timing: StepTiming | None = None) -> None:
        """Enqueue one decode step whose inputs and output live in page-locked
        host memory (device-accessible addresses of float32 [B][ctx_stride]
        scores, bf16 [layers][B][H][576] queries and bf16 [layers][B][H][512]
        output): the library copies them inside the step (dsa_group_step_host).
        The output also lands in `out`."""
        if self._io_scores is None:
            dev = self.out.device
            self._io_scores = torch.empty((self.B, self.ctx_stride), dtype=torch.float32,
                                          device=dev)
            self._io_q = torch.empty((2, self.L, self.B, self.H, D), dtype=torch.int16,
                                     device=dev)
        if timing is not None:
            timing.with_topk = True
        abi.check(abi.dsa_group_step_host(self.desc, scores_h, q_h, out_h, self._io_scores,
                                          self._io_q,
                                          None if timing is None else timing.array),
                  "dsa_group_step_host")
        if self.policy == "reuse":
            self.ids = self._bufs[self.desc.prev_ids]
            self.sel = self._bufs[self.desc.prev_sel]

    def join(self, stream=None) -> None:
        """Make `stream` (default: the current stream) wait for all step work."""
        st = torch.cuda.current_stream() if stream is None else stream
        st.wait_stream(self.main)
        st.wait_stream(self.gstream)
        st.wait_stream(self.side)
        for ls in self.lstreams:
            st.wait_stream(ls)

    def metrics(self) -> dict:
        """plan_metrics of the last step's plan (after synchronize())."""
        install = None if self.policy == "reuse" else self.install.cpu().numpy()
        return plan_metrics(self.miss_rows.cpu().numpy(), self.miss_count.cpu().numpy(),
                            self.miss_ids.cpu().numpy(), install, self.k, self.S)

    # -- checkpoint / resume ---------------------------------------------
    def state(self) -> dict:
        """The pool's state after the steps so far, as host arrays (numpy): its
        metadata (tags, FIFO pointers, LRU order) and every layer's slot rows;
        with the reuse policy the previous step's ids and selection instead of
        the pool. Waits for the group's streams first (raises if the device
        reported an error). load_state puts it into a group of the same
        shapes, after which that group continues as this one would; a test
        resumes the oracle from the same arrays (tags, pointers and rows of
        one request)."""
        if self.synchronize():
            raise RuntimeError("device error bits set before the checkpoint")
        st = {"tags": self.tags.cpu().numpy(), "fifo_ptr": self.fifo_ptr.cpu().numpy(),
              "lru_order": self.lru_order.cpu().numpy()}
        if self.policy == "reuse":
            st["prev_ids"] = self._bufs[self.desc.prev_ids].cpu().numpy()
            st["prev_sel"] = self._bufs[self.desc.prev_sel].cpu().numpy()
        else:
            st["pool"] = self.pool[:, :, :self.P].cpu().numpy()
        return st

    def load_state(self, st: dict) -> None:
        """Put a state from state() into this group (its streams idle); the
        group's own step count and ordering words carry on as they are."""
        self.synchronize()

        def put(t: torch.Tensor, a: np.ndarray):
            if tuple(t.shape) != a.shape:
                raise ValueError(f"state of shape {a.shape} for a buffer of {tuple(t.shape)}")
            t.copy_(torch.from_numpy(np.ascontiguousarray(a)))

        put(self.tags, st["tags"])
        put(self.fifo_ptr, st["fifo_ptr"])
        put(self.lru_order, st["lru_order"])
        if self.policy == "reuse":
            put(self._bufs[self.desc.prev_ids], st["prev_ids"])
            put(self._bufs[self.desc.prev_sel], st["prev_sel"])
        else:
            put(self.pool[:, :, :self.P], st["pool"])
        torch.cuda.synchronize(self.pool.device)

    def synchronize(self) -> int:
        """Wait for everything and return (and clear) the device error bits."""
        self.main.synchronize()
        self.gstream.synchronize()
        self.side.synchronize()
        for ls in self.lstreams:
            ls.synchronize()
        return abi.ts_read_error(self.err, self.main)


class PagedKV:
    """The paged latent cache of one layer (dsa_cache_write, dsa_cache_append,
    dsa_cache_read, sfa_mla_chunk, sfa_mla_tree, dsa_cache_keep,
    dsa_cache_fork): num_pages pages of page_size rows, as bf16 or quantised to
    8 bits (fmt "e4m3"). The caller deals out the pages; a request's position t
    lies in slot block_table[b][t // page_size] * page_size + t % page_size.
    `data` are the rows (uint8 [num_pages * page_size][row bytes]), `err` the
    device error word; making one waits until both are zero. Calls enqueue on
    `stream` (default: the current stream of the cache's device) and do not
    wait."""

    def __init__(self, num_pages: int, page_size: int = 64, fmt: str = "bf16",
                 device: str = "cuda"):
        if fmt not in ("bf16", "e4m3"):
            raise ValueError(fmt)
        self.num_pages, self.page_size, self.fmt = num_pages, page_size, fmt
        self._fmt = abi.DSA_CACHE_BF16 if fmt == "bf16" else abi.DSA_CACHE_E4M3
        self.num_slots = num_pages * page_size
        dev = torch.device(device)
        self.data = torch.zeros((self.num_slots, abi.dsa_cache_row_bytes(self._fmt)),
                                dtype=torch.uint8, device=dev)
        self.err = torch.zeros((1,), dtype=torch.int32, device=dev)
        # the zeros are there before the first call, whatever its stream (inside
        # a capture there is nothing to wait for: they are part of the graph)
        if self.data.is_cuda:
            with torch.cuda.device(self.data.device):
                if not torch.cuda.is_current_stream_capturing():
                    torch.cuda.current_stream().synchronize()

    def _int32(self, t: torch.Tensor, name: str, dims: int) -> torch.Tensor:
        if t.dtype != torch.int32 or t.dim() != dims or t.device != self.data.device:
            raise ValueError(f"{name}: expected {dims} int32 dimensions on {self.data.device}")
        if t.numel() and t.stride(-1) != 1:
            raise ValueError(f"{name}: its last dimension must be contiguous")
        return t

    def _bf16(self, t: torch.Tensor, name: str, shape) -> torch.Tensor:
        if (t.dtype not in (torch.bfloat16, torch.int16) or t.device != self.data.device
                or tuple(t.shape) != tuple(shape)):
            raise ValueError(f"{name}: expected bf16 {tuple(shape)} on {self.data.device}")
        return t

    @staticmethod
    def _stream(stream, device):
        return torch.cuda.current_stream(device) if stream is None else stream

    def write(self, latent: torch.Tensor, rope: torch.Tensor, slots: torch.Tensor,
              stream=None) -> None:
        """Put rows latent [n][512], rope [n][64] (bf16, rows of any stride)
        into slots [n] (negative: skipped)."""
        n = latent.shape[0]
        self._bf16(latent, "latent", (n, DV))
        self._bf16(rope, "rope", (n, D - DV))
        if self._int32(slots, "slots", 1).shape[0] != n:
            raise ValueError("slots: one for each row")
        if n == 0:
            return
        if latent.stride(1) != 1 or rope.stride(1) != 1:
            raise ValueError("latent, rope: rows must be contiguous")
        with torch.cuda.device(self.data.device):
            abi.check(abi.dsa_cache_write(
                latent, latent.stride(0) if n > 1 else DV, rope,
                rope.stride(0) if n > 1 else D - DV, slots, n, self.data, self.num_slots,
                self._fmt, self.err, self._stream(stream, self.data.device)), "dsa_cache_write")

    def append(self, latent: torch.Tensor, rope: torch.Tensor, pos: torch.Tensor,
               slots: torch.Tensor, freq: torch.Tensor, q_rope: torch.Tensor | None = None,
               q: torch.Tensor | None = None, interleaved: bool = True, stream=None) -> None:
        """write, with the rope parts turned by their positions on the way: pos
        int32 [n], freq float64 [32] (radians a position), pairs of values side by
        side (interleaved) or half the part apart. With q_rope [n][H][64] (bf16,
        tokens and heads of any stride) the queries' rope parts are turned too,
        into q[..., 512:] (bf16 [n][H][576], a token's heads contiguous); q_rope
        may be that part itself."""
        n = latent.shape[0]
        rope_dim = D - DV
        self._bf16(latent, "latent", (n, DV))
        self._bf16(rope, "rope", (n, rope_dim))
        for t, name in ((pos, "pos"), (slots, "slots")):
            if self._int32(t, name, 1).shape[0] != n:
                raise ValueError(f"{name}: one for each row")
        if (freq.dtype != torch.float64 or tuple(freq.shape) != (rope_dim // 2,)
                or not freq.is_contiguous() or freq.device != self.data.device):
            raise ValueError(f"freq: expected contiguous float64 {(rope_dim // 2,)} on "
                             f"{self.data.device}")
        if (q_rope is None) != (q is None):
            raise ValueError("q_rope, q: both or neither")
        H, strides = 0, (0, 0, 0)
        if q is not None:
            H = q.shape[1] if q.dim() == 3 else 0
            self._bf16(q, "q", (n, H, D))
            self._bf16(q_rope, "q_rope", (n, H, rope_dim))
            if n and H and (q.stride(2) != 1 or (H > 1 and q.stride(1) != D)):
                raise ValueError("q: a token's heads must be contiguous")
            if n and H and q_rope.stride(2) != 1:
                raise ValueError("q_rope: a head's values must be contiguous")
            # (a dimension of one may have any stride)
            head = q_rope.stride(1) if H > 1 else rope_dim
            strides = (q_rope.stride(0) if n > 1 else rope_dim, head,
                       q.stride(0) if n > 1 else H * D)
        if n == 0:
            return
        if latent.stride(1) != 1 or rope.stride(1) != 1:
            raise ValueError("latent, rope: rows must be contiguous")
        if H == 0:
            q_rope = None
        with torch.cuda.device(self.data.device):
            abi.check(abi.dsa_cache_append(
                latent, latent.stride(0) if n > 1 else DV, rope,
                rope.stride(0) if n > 1 else rope_dim, pos, slots, n, freq, interleaved,
                self.data, self.num_slots, self._fmt, q_rope, strides[0], strides[1], H, q,
                strides[2], self.err, self._stream(stream, self.data.device)), "dsa_cache_append")

    def plan_tree(self, parent: torch.Tensor | None, cu_q: torch.Tensor,
                  block_table: torch.Tensor, ctx_len: torch.Tensor, T: int, most: int,
                  stream=None):
        """What append and attend need of a step's drafted trees (dsa_tree_plan):
        parent int32 [T] (a node's parent's number within its request, -1 for a
        root; None: chains), at most `most` nodes a request. Returns (pos int32
        [T], slots int32 [T], mask int32 [T][ceil(most / 32)]); the same for every
        layer's cache of these pages."""
        B = ctx_len.shape[0]
        if T < 0 or not 1 <= most <= abi.TS_MAX_TREE:
            raise ValueError(f"T, most: at least 0, and 1 to {abi.TS_MAX_TREE}")
        if parent is not None and self._int32(parent, "parent", 1).shape[0] != T:
            raise ValueError("parent: one for each token")
        if self._int32(cu_q, "cu_q", 1).shape[0] != B + 1:
            raise ValueError("cu_q: one more than the requests")
        self._table(block_table, ctx_len, B)
        dev, words = self.data.device, -(-most // 32)
        if T == 0:
            new = dict(dtype=torch.int32, device=dev)
            return torch.empty(0, **new), torch.empty(0, **new), torch.empty((0, words), **new)
        st = self._stream(stream, dev)
        with torch.cuda.device(dev), torch.cuda.stream(st):
            pos = torch.empty((T,), dtype=torch.int32, device=dev)
            slots = torch.empty((T,), dtype=torch.int32, device=dev)
            mask = torch.empty((T, words), dtype=torch.int32, device=dev)
            if B:
                abi.check(abi.dsa_tree_plan(parent, cu_q, T, B, ctx_len, block_table,
                                            self._table_stride(block_table), self.page_size,
                                            self.num_slots, pos, slots, mask, words, self.err, st),
                          "dsa_tree_plan")
            else:  # tokens that no request has
                pos.zero_(), slots.fill_(-1), mask.zero_()
        return pos, slots, mask

    def keep(self, path: torch.Tensor, accepted: torch.Tensor, cu_q: torch.Tensor, T: int,
             block_table: torch.Tensor, ctx_len: torch.Tensor, new_len: torch.Tensor | None = None,
             stream=None) -> torch.Tensor:
        """The rows of verify_tree's accepted paths moved together behind each
        request's context (dsa_cache_keep): path int32 [B][depth + 1], accepted
        int32 [B]; cu_q, T and ctx_len as in the step's attention. Returns the
        requests' lengths afterwards (new_len int32 [B], a fresh one unless given;
        it may be ctx_len)."""
        dev, B = self.data.device, ctx_len.shape[0]
        self._table(block_table, ctx_len, B)
        if not self._int32(path, "path", 2).is_contiguous() or path.shape[0] != B or \
                path.shape[1] < 1:
            raise ValueError("path: a contiguous row for each request")
        if self._int32(cu_q, "cu_q", 1).shape[0] != B + 1:
            raise ValueError("cu_q: one more than the requests")
        if T < 0:
            raise ValueError("T: at least 0")
        for t, name in ((accepted, "accepted"), (new_len, "new_len")):
            if t is not None and self._int32(t, name, 1).shape[0] != B:
                raise ValueError(f"{name}: one for each request")
        if B == 0:
            return torch.empty(0, dtype=torch.int32, device=dev) if new_len is None else new_len
        st = self._stream(stream, dev)
        with torch.cuda.device(dev), torch.cuda.stream(st):
            if new_len is None:
                new_len = torch.empty((B,), dtype=torch.int32, device=dev)
            abi.check(abi.dsa_cache_keep(
                self.data, self.num_slots, self._fmt, block_table,
                self._table_stride(block_table), self.page_size, cu_q, T, ctx_len, B, path,
                path.shape[1] - 1, accepted, new_len, self.err, st), "dsa_cache_keep")
        return new_len

    def fork(self, parents: torch.Tensor, spare: torch.Tensor, block_table: torch.Tensor,
             ctx_len: torch.Tensor, tables: bool = True, stream=None):
        """The sequences' states in beam_select's new order (dsa_cache_fork):
        parents int32 [B][n] (the beam each continues, -1: none) over the B * K
        sequences of block_table and ctx_len; spare int32 [B * n]: a page of its own
        for each new sequence, which gets the rows of its parent's partial last page
        and the rows to come. Returns (block_table int32 [B * n][..], ctx_len int32
        [B * n]) of the new sequences; `tables` False: the rows alone (the other
        layers' caches), and None."""
        dev = self.data.device
        B, n = self._int32(parents, "parents", 2).shape
        old = ctx_len.shape[0]
        self._table(block_table, ctx_len, old)
        if not parents.is_contiguous():
            raise ValueError("parents must be contiguous")
        if self._int32(spare, "spare", 1).shape[0] != B * n:
            raise ValueError("spare: one for each new sequence")
        if B and old % B:
            raise ValueError("block_table, ctx_len: equally many sequences for each request")
        def made():
            if not tables:
                return None, None
            new = dict(dtype=torch.int32, device=dev)
            return torch.empty((B * n, block_table.shape[1]), **new), torch.empty(B * n, **new)

        if B == 0 or n == 0:
            return made() if tables else None
        st = self._stream(stream, dev)
        with torch.cuda.device(dev), torch.cuda.stream(st):
            table, length = made()
            abi.check(abi.dsa_cache_fork(
                self.data, self.num_slots, self._fmt, block_table,
                self._table_stride(block_table), self.page_size, ctx_len, parents, spare, B,
                old // B, n, table, length, self.err, st), "dsa_cache_fork")
        return (table, length) if tables else None

    def read(self, block_table: torch.Tensor, ctx_len: torch.Tensor, pos: torch.Tensor,
             out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """The rows of positions pos [B][k] as bf16 [B][k][576]: sfa_mla_decode's
        selection buffer. block_table int32 [B][pages a request], contiguous."""
        B, k = self._int32(pos, "pos", 2).shape
        self._table(block_table, ctx_len, B)
        if not pos.is_contiguous():
            raise ValueError("pos must be contiguous")
        if out is not None and not self._bf16(out, "out", (B, k, D)).is_contiguous():
            raise ValueError("out must be contiguous")
        if B == 0 or k == 0:
            return torch.empty((B, k, D), dtype=torch.bfloat16,
                               device=self.data.device) if out is None else out
        st = self._stream(stream, self.data.device)
        if out is None:
            with torch.cuda.stream(st):
                out = torch.empty((B, k, D), dtype=torch.bfloat16, device=self.data.device)
        with torch.cuda.device(self.data.device):
            abi.check(abi.dsa_cache_read(self.data, self.num_slots, self._fmt, block_table,
                                         self._table_stride(block_table), self.page_size, pos,
                                         ctx_len, B, k, out, self.err, st), "dsa_cache_read")
        return out

    def _table(self, block_table, ctx_len, B):
        self._int32(block_table, "block_table", 2)
        self._int32(ctx_len, "ctx_len", 1)
        if block_table.shape[0] != B or ctx_len.shape[0] != B:
            raise ValueError("block_table, ctx_len: one row for each request")
        if B > 1 and block_table.stride(0) != block_table.shape[1]:
            raise ValueError("block_table must be contiguous")

    @staticmethod
    def _table_stride(block_table):
        return block_table.shape[1]

    def attend(self, q: torch.Tensor, cu_q: torch.Tensor, block_table: torch.Tensor,
               ctx_len: torch.Tensor, causal: bool = True, scale: float | None = None,
               out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
               ws: torch.Tensor | None = None, stream=None, tree: torch.Tensor | None = None):
        """Attention of the newest tokens q [T][H][576] (request b's are rows
        cu_q[b] .. cu_q[b + 1]) over the cached positions below ctx_len[b];
        block_table int32 [B][pages a request], contiguous. Returns (out bf16
        [T][H][512], lse float [T][H]), fresh ones unless given; rows that no
        request has are left as they were. `ws`: a workspace of
        `workspace(T, B, H)` kept by the caller (contiguous uint8 on the cache's
        device); without one the call takes its own from PyTorch's allocator, on
        its stream. `tree`: the new tokens are drafted trees, and of the new
        positions each sees those of its row of plan_tree's masks (int32
        [T][words], sfa_mla_tree; `causal` is not used then)."""
        dev = self.data.device
        T, H = q.shape[0], q.shape[1]
        B = ctx_len.shape[0]
        self._bf16(q, "q", (T, H, D))
        if T and (q.stride(2) != 1 or (H > 1 and q.stride(1) != D)):
            raise ValueError("q: a token's heads must be contiguous")
        if self._int32(cu_q, "cu_q", 1).shape[0] != B + 1:
            raise ValueError("cu_q: one more than the requests")
        self._table(block_table, ctx_len, B)
        # (its size and alignment are the library's to check)
        if ws is not None and (ws.dtype != torch.uint8 or ws.device != dev
                               or not ws.is_contiguous()):
            raise ValueError(f"ws: expected contiguous uint8 on {dev}")
        if out is not None and not self._bf16(out, "out", (T, H, DV)).is_contiguous():
            raise ValueError("out must be contiguous")
        if lse is not None and (lse.dtype != torch.float32 or tuple(lse.shape) != (T, H)
                                or not lse.is_contiguous() or lse.device != dev):
            raise ValueError(f"lse: expected contiguous float32 {(T, H)} on {dev}")
        if tree is not None and (self._int32(tree, "tree", 2).shape[0] != T
                                 or not tree.is_contiguous() or not tree.shape[1]):
            raise ValueError("tree: a contiguous row of masks for each token")
        if (T == 0 or B == 0) and out is not None and lse is not None:
            return out, lse
        st = self._stream(stream, dev)
        with torch.cuda.device(dev), torch.cuda.stream(st):
            if out is None:
                out = torch.empty((T, H, DV), dtype=torch.bfloat16, device=dev)
            if lse is None:
                lse = torch.empty((T, H), dtype=torch.float32, device=dev)
            if T == 0 or B == 0:  # no rows, or nobody's
                return out, lse
            if ws is None:
                ws = self.workspace(T, B, H)
            first = (q, q.stride(0) if T > 1 else H * D, cu_q, T, B, H, self.data,
                     self.num_slots, self._fmt, block_table, self._table_stride(block_table),
                     self.page_size, ctx_len)
            last = (1.0 / math.sqrt(D) if scale is None else scale, out, lse, ws, ws.numel(),
                    self.err, st)
            if tree is None:
                abi.check(abi.sfa_mla_chunk(*first, causal, *last), "sfa_mla_chunk")
            else:
                abi.check(abi.sfa_mla_tree(*first, tree, tree.shape[1], *last), "sfa_mla_tree")
        return out, lse

    def workspace(self, T: int, B: int, H: int) -> torch.Tensor:
        """A workspace of attend for up to T tokens of B requests."""
        return torch.empty((max(256, abi.sfa_chunk_workspace_size(T, B, H)),), dtype=torch.uint8,
                           device=self.data.device)

    def synchronize(self, stream=None) -> int:
        """Wait for the stream and return (and clear) the device error bits."""
        with torch.cuda.device(self.data.device):
            return abi.ts_read_error(self.err, self._stream(stream, self.data.device))


def verify_drafts(drafts: torch.Tensor, target: torch.Tensor, draft: torch.Tensor | None,
                  u: torch.Tensor, n_draft: torch.Tensor | None = None,
                  err: torch.Tensor | None = None, stream=None):
    """ts_verify_drafts on tensors: drafts int32 [B][n], target float [B][n + 1][V],
    draft float [B][n][V] or None (certain drafts), u float [B][n + 1], n_draft
    int32 [B] or None. Returns (tokens int32 [B][n + 1], accepted int32 [B]).
    `err`: a device error word (int32 [1], read with ts_read_error); without one
    bad ids and probabilities are not reported."""
    dev = target.device
    B, n = drafts.shape
    V = target.shape[2]

    def rows(t, name, count):
        if t.dtype != torch.float32 or t.device != dev or tuple(t.shape) != (B, count, V):
            raise ValueError(f"{name}: expected float32 {(B, count, V)} on {dev}")
        if t.numel() == 0:
            return V
        # (a dimension of one may have any stride)
        step = t.stride(1) if count > 1 else t.stride(0) if B > 1 else V
        if ((V > 1 and t.stride(2) != 1) or step < V
                or (B > 1 and count > 1 and t.stride(0) != count * step)):
            raise ValueError(f"{name}: its rows must be evenly spaced, V floats or more apart")
        return step

    ts = rows(target, "target", n + 1)
    ds = V if draft is None else rows(draft, "draft", n)
    for t, name, dtype, shape in ((drafts, "drafts", torch.int32, (B, n)),
                                  (u, "u", torch.float32, (B, n + 1)),
                                  (n_draft, "n_draft", torch.int32, (B,)),
                                  (err, "err", torch.int32, (1,))):
        if t is not None and (t.dtype != dtype or tuple(t.shape) != shape or t.device != dev
                              or not t.is_contiguous()):
            raise ValueError(f"{name}: expected contiguous {dtype} {shape} on {dev}")
    st = torch.cuda.current_stream(dev) if stream is None else stream
    with torch.cuda.device(dev), torch.cuda.stream(st):
        tokens = torch.empty((B, n + 1), dtype=torch.int32, device=dev)
        accepted = torch.empty((B,), dtype=torch.int32, device=dev)
        abi.check(abi.ts_verify_drafts(drafts, n_draft, target, ts, draft, ds, u, B, n, V, tokens,
                                       accepted, err, st), "ts_verify_drafts")
    return tokens, accepted


def verify_tree(tokens: torch.Tensor, parent: torch.Tensor | None, cu_q: torch.Tensor,
                target: torch.Tensor, u: torch.Tensor | None, depth: int | None = None,
                err: torch.Tensor | None = None, stream=None):
    """ts_verify_tree on tensors: drafted trees, tokens int32 [T] and parent int32
    [T] (None: chains), packed by cu_q int32 [B + 1], against target float [T][V],
    by u float [B][depth + 1], or (u None, with depth) by the largest value. Returns
    (path int32 [B][depth + 1], tokens int32 [B][depth + 1], accepted int32 [B]).
    `err`: a device error word (int32 [1], read with ts_read_error); without one bad
    probabilities are not reported."""
    dev = target.device
    if target.dim() != 2 or cu_q.dim() != 1 or cu_q.shape[0] < 1:
        raise ValueError("target, cu_q: expected [T][V] and [B + 1]")
    (T, V), B = target.shape, cu_q.shape[0] - 1
    if u is not None and (u.dim() != 2 or u.shape[1] < 1):
        raise ValueError("u: expected [B][depth + 1]")
    if depth is None:
        if u is None:
            raise ValueError("depth: needed without u")
        depth = u.shape[1] - 1
    if depth < 0:
        raise ValueError("depth: at least 0")
    if (target.dtype != torch.float32 or (V > 1 and T and target.stride(1) != 1)
            or (T > 1 and target.stride(0) < V)):
        raise ValueError("target: expected float32 rows, V floats or more apart")
    for t, name, dtype, shape in ((tokens, "tokens", torch.int32, (T,)),
                                  (parent, "parent", torch.int32, (T,)),
                                  (cu_q, "cu_q", torch.int32, (B + 1,)),
                                  (u, "u", torch.float32, (B, depth + 1)),
                                  (err, "err", torch.int32, (1,))):
        if t is not None and (t.dtype != dtype or tuple(t.shape) != shape or t.device != dev
                              or not t.is_contiguous()):
            raise ValueError(f"{name}: expected contiguous {dtype} {shape} on {dev}")
    st = torch.cuda.current_stream(dev) if stream is None else stream
    with torch.cuda.device(dev), torch.cuda.stream(st):
        path = torch.empty((B, depth + 1), dtype=torch.int32, device=dev)
        out = torch.empty((B, depth + 1), dtype=torch.int32, device=dev)
        accepted = torch.empty((B,), dtype=torch.int32, device=dev)
        abi.check(abi.ts_verify_tree(tokens, parent, cu_q, T, B, target,
                                     target.stride(0) if T > 1 else V, u, V, depth, path, out,
                                     accepted, err, st), "ts_verify_tree")
    return path, out, accepted


def beam_select(logits: torch.Tensor, cum: torch.Tensor, n: int, ws: torch.Tensor | None = None,
                err: torch.Tensor | None = None, stream=None):
    """ts_beam_select on tensors: the n best continuations of each request's K
    beams, logits float32 or bf16 [B][K][V] (rows evenly spaced), cum float [B][K].
    Returns (tokens int32 [B][n], parents int32 [B][n], scores float [B][n]).
    `ws`: a workspace of ts_beam_workspace_size(B, K, V, n) bytes kept by the
    caller (contiguous uint8); `err`: a device error word (int32 [1])."""
    dev = logits.device
    if logits.dim() != 3 or logits.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("logits: expected float32 or bf16 [B][K][V]")
    B, K, V = logits.shape
    # (a dimension of one may have any stride)
    step = logits.stride(1) if K > 1 else logits.stride(0) if B > 1 else V
    if logits.numel() and ((V > 1 and logits.stride(2) != 1) or step < V
                           or (B > 1 and K > 1 and logits.stride(0) != K * step)):
        raise ValueError("logits: its rows must be evenly spaced, V values or more apart")
    for t, name, dtype, shape in ((cum, "cum", torch.float32, (B, K)),
                                  (err, "err", torch.int32, (1,))):
        if t is not None and (t.dtype != dtype or tuple(t.shape) != shape or t.device != dev
                              or not t.is_contiguous()):
            raise ValueError(f"{name}: expected contiguous {dtype} {shape} on {dev}")
    # (its size and alignment are the library's to check)
    if ws is not None and (ws.dtype != torch.uint8 or ws.device != dev or not ws.is_contiguous()):
        raise ValueError(f"ws: expected contiguous uint8 on {dev}")
    st = torch.cuda.current_stream(dev) if stream is None else stream
    with torch.cuda.device(dev), torch.cuda.stream(st):
        tokens = torch.empty((B, n), dtype=torch.int32, device=dev)
        parents = torch.empty((B, n), dtype=torch.int32, device=dev)
        scores = torch.empty((B, n), dtype=torch.float32, device=dev)
        if ws is None:
            ws = torch.empty((max(256, abi.ts_beam_workspace_size(B, K, V, n)),),
                             dtype=torch.uint8, device=dev)
        abi.check(abi.ts_beam_select(logits, abi.TS_FP32 if logits.dtype == torch.float32
                                     else abi.TS_BF16, step, cum, B, K, V, n, tokens, parents,
                                     scores, ws, ws.numel(), err, st), "ts_beam_select")
    return tokens, parents, scores
