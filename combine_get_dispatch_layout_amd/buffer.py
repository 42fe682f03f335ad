"""Python front end with the call shapes of the pages, over libmoedx.so.

``Buffer`` mirrors the normal and low-latency usage examples of the
EnflameTechnology/DeepEP README (get_dispatch_layout, dispatch, combine,
low_latency_dispatch, low_latency_combine, capture); ``EventOverlap`` mirrors
the event wrapper of "How DeepEP Achieves Communication-Computation
Overlapping with EventOverlap" (current_stream_wait and the context manager).
PyTorch only provides device memory and the current stream; every step runs in
the library's HIP kernels.
"""

from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _capi as C


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    p = t.data_ptr()
    if p == 0 and t.numel() == 0:  # an empty view still names its allocation
        p = t.untyped_storage().data_ptr()
    return ctypes.c_void_p(p or None)


def _stream() -> int:
    return torch.cuda.current_stream().cuda_stream


def _addr(t: Optional[torch.Tensor]):
    """_ptr as a plain int (or None)."""
    if t is None:
        return None
    return t.data_ptr() or (t.untyped_storage().data_ptr() or None)


# The handle of a device's current stream: torch's own accessor for callers of
# raw kernels where it has one (a tenth of the Stream object's cost).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _contiguous(t: Optional[torch.Tensor], previous_event) -> Optional[torch.Tensor]:
    """`t`, or its contiguous copy, which is made on the current stream of t's
    device: like the call it is for, behind `previous_event` (the call's own
    wait comes later, and may be another stream's)."""
    if t is None or t.is_contiguous():
        return t
    if previous_event is not None and previous_event.event is not None:
        C.check(C.moedx_event_wait(previous_event.event, _raw_stream(t.get_device())))
    return t.contiguous()


# Releases that must wait until no stream capture is running.  Destroying a
# context synchronises its stream and frees device and pinned memory, and an
# event destroy is not a capturable call either; any of them during a capture
# invalidates the graph being recorded.  A finalizer can run at any point (the
# garbage collector may collect an old Buffer in the middle of someone else's
# capture), so while the current stream is capturing the release is queued and
# done by the next call that runs outside a capture.
_deferred: list = []


def _capturing() -> bool:
    try:
        return torch.cuda.is_available() and torch.cuda.is_current_stream_capturing()
    except Exception:  # interpreter shutdown: torch may already be gone
        return False


def _flush_deferred(_deferred=_deferred, _capturing=_capturing) -> None:
    while _deferred and not _capturing():
        fn, ptr = _deferred.pop()
        fn(ptr)


# Finalizers reach these through default arguments and class attributes: at
# interpreter exit the module's globals may already be gone.
def _release(fn, ptr, _deferred=_deferred, _capturing=_capturing,
             _flush=_flush_deferred) -> None:
    if _capturing():
        _deferred.append((fn, ptr))
        return
    fn(ptr)
    _flush()


class EventOverlap:
    """Owns one library event.  ``event is None`` means "already complete"
    (what a call with async_finish=False hands back, for tuple arity)."""

    def __init__(self, event: Optional[int] = None):
        self.event = event

    def current_stream_wait(self) -> None:
        if self.event is not None:
            C.check(C.moedx_event_wait(self.event, _stream()))

    def synchronize(self) -> None:
        if self.event is not None:
            C.check(C.moedx_event_synchronize(self.event))

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.current_stream_wait()

    # Held by the class: at interpreter exit module globals may already be gone.
    _destroy = staticmethod(C.moedx_event_destroy)
    _release = staticmethod(_release)

    def __del__(self):
        if getattr(self, "event", None) is not None:
            self._release(self._destroy, self.event)
            self.event = None


_MATRICES = {C.MOEDX_T_CHANNEL_PREFIX_MATRIX, C.MOEDX_T_RECV_CHANNEL_PREFIX_MATRIX,
             C.MOEDX_T_IS_TOKEN_IN_RANK, C.MOEDX_T_SEND_HEAD, C.MOEDX_T_LL_SRC_IDX,
             C.MOEDX_T_LL_SLOT_OF}


class Handle:
    """A prepared layout: the library handle plus the device workspace that
    holds its arrays (kept alive as long as the handle)."""

    def __init__(self, ptr: int, workspace: torch.Tensor, T: int, K: int, low_latency: bool,
                 capacity: int = 0, buffer: "Optional[Buffer]" = None):
        self.ptr = ptr
        self.workspace = workspace
        self.T, self.K = T, K
        self.low_latency = low_latency
        self.capacity = capacity
        self.buffer = buffer  # the Buffer whose ctx prepared it (normal handles)

    def finish(self) -> None:
        """Write a capacity-mode handle's prefixes, totals and N on the current
        stream now rather than on its first dispatch or combine (nothing runs
        when they are already written)."""
        if self.low_latency or self.buffer is None:
            return
        ex = C.make_exec(_stream(), None, None, C.MOEDX_ASYNC)
        C.check(C.moedx_handle_finish(self.buffer.ctx, self.ptr, ctypes.byref(ex)))

    def tensor(self, which: int, dtype: torch.dtype) -> torch.Tensor:
        """View of one handle array (MOEDX_T_*) inside the workspace."""
        dev = ctypes.c_void_p()
        shape = (ctypes.c_int64 * 2)()
        C.check(C.moedx_handle_tensor(self.ptr, which, ctypes.byref(dev), shape))
        n0, n1 = int(shape[0]), int(shape[1])
        off = (dev.value or 0) - self.workspace.data_ptr()
        nbytes = n0 * n1 * torch.empty((), dtype=dtype).element_size()
        assert 0 <= off and off + nbytes <= self.workspace.numel()
        v = self.workspace[off: off + nbytes].view(dtype)
        return v.view(n0, n1) if which in _MATRICES else v

    @property
    def num_recv(self) -> int:
        n = ctypes.c_int64()
        C.check(C.moedx_handle_num_recv(self.ptr, ctypes.byref(n)))
        return int(n.value)

    def recv_tokens_per_expert(self, num_experts: int) -> list:
        a = (ctypes.c_int32 * num_experts)()
        C.check(C.moedx_handle_recv_tokens_per_expert(self.ptr, a))
        return list(a)

    # handle fields named on the handle-reuse page
    def fields(self) -> dict:
        self.finish()
        if self.low_latency:
            return {"src_idx": self.tensor(C.MOEDX_T_LL_SRC_IDX, torch.int32),
                    "slot_of": self.tensor(C.MOEDX_T_LL_SLOT_OF, torch.int32)}
        return {
            "rank_prefix_matrix": self.tensor(C.MOEDX_T_RANK_PREFIX_MATRIX, torch.int32),
            "channel_prefix_matrix": self.tensor(C.MOEDX_T_CHANNEL_PREFIX_MATRIX, torch.int32),
            "recv_channel_prefix_matrix": self.tensor(C.MOEDX_T_RECV_CHANNEL_PREFIX_MATRIX, torch.int32),
            "recv_src_idx": self.tensor(C.MOEDX_T_RECV_SRC_IDX, torch.int32),
            "is_token_in_rank": self.tensor(C.MOEDX_T_IS_TOKEN_IN_RANK, torch.uint8),
            "send_head": self.tensor(C.MOEDX_T_SEND_HEAD, torch.int32),
            "num_tokens_per_rank": self.tensor(C.MOEDX_T_NUM_TOKENS_PER_RANK, torch.int32),
            "num_tokens_per_expert": self.tensor(C.MOEDX_T_NUM_TOKENS_PER_EXPERT, torch.int32),
            "num_recv": self.tensor(C.MOEDX_T_NUM_RECV, torch.int32),
        }

    _destroy = staticmethod(C.moedx_handle_destroy)

    def __del__(self):
        if getattr(self, "ptr", None):
            self._destroy(self.ptr)
            self.ptr = None


_DTYPES = {torch.bfloat16: C.MOEDX_BF16, torch.float16: C.MOEDX_F16, torch.float32: C.MOEDX_F32}
_PRODUCT_DTYPES = (torch.bfloat16, torch.float16)
_INT8, _FP32 = (torch.int8,), (torch.float32,)
# What every call takes beside its own arguments.
_OPTIONS = ("previous_event", "async_finish", "allocate_on_comm_stream", "no_sync")
_SCORES = {"softmax": C.MOEDX_GATE_SOFTMAX, "sigmoid": C.MOEDX_GATE_SIGMOID}


class ExpertOrder:
    """Rows in expert order (Buffer.expert_order): expert e has rows
    [expert_offsets[e], expert_offsets[e + 1]); ``row_of_slot`` [T, K] is the
    row of each pair (-1 = empty slot) and ``slot_of_row`` [T * K] its inverse
    (t * K + k, -1 past the last row).  All int32 on the device."""

    def __init__(self, expert_offsets: torch.Tensor, row_of_slot: torch.Tensor,
                 slot_of_row: torch.Tensor):
        self.expert_offsets = expert_offsets
        self.row_of_slot = row_of_slot
        self.slot_of_row = slot_of_row


class Buffer:
    """One GPU's share of the expert-parallel exchange: ``num_ranks`` logical
    ranks are buckets of ``num_experts / num_ranks`` experts in this GPU's HBM."""

    def __init__(self, num_experts: int, num_ranks: int, num_channels: int = 24,
                 max_tokens: int = 16384, device: Optional[int] = None):
        self.device = torch.cuda.current_device() if device is None else device
        self.num_experts, self.num_ranks, self.num_channels = num_experts, num_ranks, num_channels
        self.max_tokens = max_tokens
        _flush_deferred()
        ctx = ctypes.c_void_p()
        C.check(C.moedx_create(ctypes.byref(ctx), self.device, num_experts, num_ranks,
                               num_channels, max_tokens, 0))
        self.ctx = ctx.value
        # The comm stream (allocate_on_comm_stream) is one of PyTorch's own
        # pool streams, which live as long as the process: tensors an op used
        # there record it (_keep), and the caching allocator records an event
        # on it when such a tensor is freed, possibly after this Buffer is gone.
        self._ctx_stream = torch.cuda.Stream(device=self.device)
        C.check(C.moedx_ctx_set_stream(self.ctx, self._ctx_stream.cuda_stream))
        self._torch_device = torch.device("cuda", self.device)
        self._index = self._torch_device.index
        self._order_size = (None, None, 0)  # the last expert_order's T, K and workspace bytes

    _destroy = staticmethod(C.moedx_destroy)
    _release = staticmethod(_release)

    def __del__(self):
        if getattr(self, "ctx", None):
            self._release(self._destroy, self.ctx)
            self.ctx = None

    # -- plumbing ---------------------------------------------------------------
    def ctx_stream(self) -> "torch.cuda.Stream":
        """The ctx's own stream (where allocate_on_comm_stream runs an op)."""
        return self._ctx_stream

    def _keep(self, on_ctx_stream: bool, *tensors) -> None:
        """An op on the ctx stream uses memory that PyTorch's caching allocator
        handed out on the caller's stream: record the ctx stream on every such
        tensor, so that no block is given to a new allocation before the ctx
        stream's work on it has finished (even when the tensor is a temporary
        dropped as the call returns)."""
        if not on_ctx_stream:
            return
        s = self.ctx_stream()
        for t in tensors:
            if isinstance(t, torch.Tensor) and t.is_cuda and t.numel() > 0:
                t.record_stream(s)

    def _exec(self, previous_event, async_finish, allocate_on_comm_stream, no_sync=False):
        if _deferred:
            _flush_deferred()
        done = ctypes.c_void_p() if async_finish else None
        flags = (C.MOEDX_ON_CTX_STREAM if allocate_on_comm_stream else 0) | (
            C.MOEDX_ASYNC if no_sync else 0)
        prev = previous_event.event if previous_event is not None else None
        return C.make_exec(_stream(), prev, done, flags), done

    @staticmethod
    def _event(done) -> EventOverlap:
        return EventOverlap(done.value if done is not None else None)

    def stats(self) -> dict:
        s = C.moedx_stats()
        C.check(C.moedx_ctx_stats(self.ctx, ctypes.byref(s)))
        return {f: getattr(s, f) for f, _ in C.moedx_stats._fields_}

    @staticmethod
    def capture() -> EventOverlap:
        ev = ctypes.c_void_p()
        C.check(C.moedx_event_record(ctypes.byref(ev), _stream()))
        return EventOverlap(ev.value)

    # -- layout -----------------------------------------------------------------
    def get_dispatch_layout(self, topk_idx: torch.Tensor, num_experts: int,
                            previous_event: Optional[EventOverlap] = None,
                            async_finish: bool = False, allocate_on_comm_stream: bool = False,
                            no_sync: bool = False):
        """Returns (num_tokens_per_rank, None, num_tokens_per_expert,
        is_token_in_rank, event); the None stands for the per-RDMA-rank counts,
        which do not exist on one GPU.  ``no_sync`` returns without blocking
        (stream order only), as under graph capture."""
        assert num_experts == self.num_experts
        topk_idx = _contiguous(topk_idx, previous_event)
        T, K = topk_idx.shape
        dev = topk_idx.device
        ntr = torch.empty(self.num_ranks, dtype=torch.int32, device=dev)
        nte = torch.empty(num_experts, dtype=torch.int32, device=dev)
        itr = torch.empty(T, self.num_ranks, dtype=torch.bool, device=dev)
        ex, done = self._exec(previous_event, async_finish, allocate_on_comm_stream, no_sync)
        C.check(C.moedx_get_dispatch_layout(self.ctx, _ptr(topk_idx), T, K, _ptr(ntr), _ptr(nte),
                                            _ptr(itr), ctypes.byref(ex)))
        self._keep(allocate_on_comm_stream, topk_idx, ntr, nte, itr)
        return ntr, None, nte, itr, self._event(done)

    # -- normal dispatch / combine --------------------------------------------------
    def prepare(self, topk_idx: torch.Tensor, num_worst_tokens: int = 0,
                previous_event=None, async_finish=False, allocate_on_comm_stream=False,
                no_sync=False, num_tokens_per_rank=None, is_token_in_rank=None,
                num_tokens_per_expert=None):
        """Layout + scan into a new handle (exact mode, or capacity mode with
        ``num_worst_tokens`` receive rows; a capacity-mode handle's prefixes,
        totals and N are written by its first dispatch or combine).  Given
        get_dispatch_layout's ``is_token_in_rank`` and ``num_tokens_per_expert``
        (and optionally ``num_tokens_per_rank``), no layout runs: the handle is
        scanned from them."""
        topk_idx = _contiguous(topk_idx, previous_event)
        T, K = topk_idx.shape
        from_layout = is_token_in_rank is not None or num_tokens_per_expert is not None
        if from_layout:
            assert is_token_in_rank is not None and num_tokens_per_expert is not None, \
                "is_token_in_rank and num_tokens_per_expert go together"
            assert tuple(is_token_in_rank.shape) == (T, self.num_ranks)
            assert is_token_in_rank.dtype in (torch.bool, torch.uint8)
            assert tuple(num_tokens_per_expert.shape) == (self.num_experts,)
            assert num_tokens_per_expert.dtype == torch.int32
            is_token_in_rank = _contiguous(is_token_in_rank, previous_event)
            num_tokens_per_expert = _contiguous(num_tokens_per_expert, previous_event)
            if num_tokens_per_rank is not None:
                assert tuple(num_tokens_per_rank.shape) == (self.num_ranks,)
                num_tokens_per_rank = _contiguous(num_tokens_per_rank, previous_event)
        else:
            num_tokens_per_rank = None
        nbytes = ctypes.c_size_t()
        C.check(C.moedx_handle_workspace_bytes(self.ctx, T, K, num_worst_tokens, ctypes.byref(nbytes)))
        ws = torch.empty(nbytes.value, dtype=torch.uint8, device=topk_idx.device)
        h = ctypes.c_void_p()
        ex, done = self._exec(previous_event, async_finish, allocate_on_comm_stream, no_sync)
        C.check(C.moedx_dispatch_prepare(self.ctx, _ptr(topk_idx), T, K, _ptr(num_tokens_per_rank),
                                         _ptr(is_token_in_rank), _ptr(num_tokens_per_expert),
                                         _ptr(ws), nbytes.value, num_worst_tokens,
                                         ctypes.byref(h), ctypes.byref(ex)))
        self._keep(allocate_on_comm_stream, topk_idx, ws, is_token_in_rank, num_tokens_per_expert)
        return Handle(h.value, ws, T, K, False, num_worst_tokens, self), self._event(done)

    def dispatch(self, x, handle: Optional[Handle] = None, num_tokens_per_rank=None,
                 num_tokens_per_rdma_rank=None, is_token_in_rank=None, num_tokens_per_expert=None,
                 topk_idx: Optional[torch.Tensor] = None, topk_weights: Optional[torch.Tensor] = None,
                 previous_event: Optional[EventOverlap] = None, async_finish: bool = False,
                 allocate_on_comm_stream: bool = False, num_worst_tokens: int = 0,
                 fp8: bool = False, round_scale: bool = False, use_ue8m0: bool = False,
                 fp8_quant_scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                 out_scales: Optional[torch.Tensor] = None, no_sync: bool = False):
        """Returns (recv_x, recv_topk_idx, recv_topk_weights,
        num_recv_tokens_per_expert_list, handle, event); recv_x is
        (codes, scales) for FP8 (scales None with a per-tensor scale).  ``x``
        may be a pre-quantised (codes uint8 [T, H], scales) pair, dispatched
        unchanged.  FP8 scales: per 1x128 block amax / 448 by default;
        ``round_scale`` rounds them up to powers of two; ``use_ue8m0`` stores
        them as UE8M0 exponent bytes (and implies ``round_scale``);
        ``fp8_quant_scale`` is one scale for the whole tensor (exclusive with
        ``use_ue8m0``).  With ``handle`` (cached dispatch) topk_idx and
        topk_weights must be None and only recv_x is produced.  On a first
        dispatch, get_dispatch_layout's outputs (``is_token_in_rank`` and
        ``num_tokens_per_expert``, with ``num_tokens_per_rank`` if at hand) are
        reused: the handle is scanned from them and no layout runs again."""
        prequant = isinstance(x, tuple)
        x_scales = None
        if prequant:
            x, x_scales = x
            x_scales = _contiguous(x_scales, previous_event)
            fp8 = True
        assert not (use_ue8m0 and fp8_quant_scale is not None), \
            "fp8_quant_scale and use_ue8m0 are exclusive"
        fp8 = fp8 or round_scale or use_ue8m0 or fp8_quant_scale is not None
        x = _contiguous(x, previous_event)
        T, H = x.shape
        first = handle is None
        inputs_ready = previous_event
        if first:
            assert topk_idx is not None, "a first dispatch needs topk_idx"
            reuse = is_token_in_rank is not None and num_tokens_per_expert is not None
            handle, _ = self.prepare(
                topk_idx, num_worst_tokens, previous_event, False, allocate_on_comm_stream,
                no_sync=True, num_tokens_per_rank=num_tokens_per_rank if reuse else None,
                is_token_in_rank=is_token_in_rank if reuse else None,
                num_tokens_per_expert=num_tokens_per_expert if reuse else None)
            previous_event = None
        else:
            assert topk_idx is None and topk_weights is None, \
                "a cached dispatch takes no topk_idx / topk_weights"
        rows = handle.capacity if handle.capacity > 0 else handle.num_recv
        K = handle.K
        dev = x.device
        # At least one row is allocated so that an empty receive side still
        # passes a valid device pointer; the returned views have `rows` rows.
        alloc = max(rows, 1)
        mode = (C.MOEDX_FP8_SCALE_TENSOR if fp8_quant_scale is not None else
                C.MOEDX_FP8_SCALE_UE8M0 if use_ue8m0 else
                C.MOEDX_FP8_SCALE_POW2 if round_scale else C.MOEDX_FP8_SCALE_AMAX)
        if fp8:
            recv_x = out if out is not None else torch.empty(alloc, H, dtype=torch.uint8, device=dev)
            sdt = torch.uint8 if mode == C.MOEDX_FP8_SCALE_UE8M0 else torch.float32
            recv_s = None if mode == C.MOEDX_FP8_SCALE_TENSOR else (
                out_scales if out_scales is not None else
                torch.empty(alloc, H // 128, dtype=sdt, device=dev))
        else:
            recv_x = out if out is not None else torch.empty(alloc, H, dtype=torch.bfloat16, device=dev)
            recv_s = None
        rti = rtw = None
        if first and not fp8:
            rti = torch.empty(alloc, K, dtype=torch.int64, device=dev)
            if topk_weights is not None:
                rtw = torch.empty(alloc, K, dtype=torch.float32, device=dev)
        ex, done = self._exec(previous_event, async_finish, allocate_on_comm_stream, no_sync)
        if fp8 and (mode != C.MOEDX_FP8_SCALE_AMAX or prequant):
            opts = C.moedx_fp8(mode, int(prequant),
                               float(fp8_quant_scale) if fp8_quant_scale is not None else 0.0,
                               _ptr(x_scales))
            C.check(C.moedx_dispatch_fp8(self.ctx, handle.ptr, _ptr(x), T, H, ctypes.byref(opts),
                                         _ptr(recv_x), _ptr(recv_s), ctypes.byref(ex)))
        else:
            tw = _contiguous(topk_weights, inputs_ready)
            ti = _contiguous(topk_idx, inputs_ready) if (first and not fp8) else None
            C.check(C.moedx_dispatch(self.ctx, handle.ptr, _ptr(x), T, H,
                                     C.MOEDX_QUANT_FP8_E4M3_1X128 if fp8 else C.MOEDX_QUANT_NONE,
                                     _ptr(ti), _ptr(tw if (first and not fp8) else None),
                                     _ptr(recv_x), _ptr(recv_s), _ptr(rti), _ptr(rtw),
                                     ctypes.byref(ex)))
            self._keep(allocate_on_comm_stream, ti, tw)
        self._keep(allocate_on_comm_stream, x, x_scales, recv_x, recv_s, rti, rtw, topk_idx,
                   topk_weights if first else None)
        per_expert = handle.recv_tokens_per_expert(self.num_experts) if (
            first and handle.capacity == 0) else None
        if out is None:
            recv_x = recv_x[:rows]
        if recv_s is not None and out_scales is None:
            recv_s = recv_s[:rows]
        rti = rti[:rows] if rti is not None else None
        rtw = rtw[:rows] if rtw is not None else None
        rx = (recv_x, recv_s) if fp8 else recv_x
        return rx, rti, rtw, per_expert, handle, self._event(done)

    def combine(self, x: torch.Tensor, handle: Handle, topk_weights: Optional[torch.Tensor] = None,
                gate_weights: Optional[torch.Tensor] = None,
                previous_event: Optional[EventOverlap] = None, async_finish: bool = False,
                allocate_on_comm_stream: bool = False, out: Optional[torch.Tensor] = None,
                no_sync: bool = False):
        """Returns (combined_x, combined_topk_weights, event).  ``topk_weights``
        is the per-row weight payload ([rows, K]) reduced like the rows;
        ``gate_weights`` ([T, K]) scales each bucket's row by its summed gate
        weight."""
        x = _contiguous(x, previous_event)
        H = x.shape[1]
        T, K = handle.T, handle.K
        combined = out if out is not None else torch.empty(T, H, dtype=torch.bfloat16, device=x.device)
        cw = torch.empty(T, K, dtype=torch.float32, device=x.device) if topk_weights is not None else None
        ex, done = self._exec(previous_event, async_finish, allocate_on_comm_stream, no_sync)
        gw = _contiguous(gate_weights, previous_event)
        tw = _contiguous(topk_weights, previous_event)
        C.check(C.moedx_combine(self.ctx, handle.ptr, _ptr(x), H, _ptr(gw), _ptr(tw),
                                _ptr(combined), _ptr(cw), ctypes.byref(ex)))
        self._keep(allocate_on_comm_stream, x, gw, tw, combined, cw)
        return combined, cw, self._event(done)

    # -- low-latency ------------------------------------------------------------
    def low_latency_dispatch(self, x: torch.Tensor, topk_idx: torch.Tensor,
                             num_max_dispatch_tokens_per_rank: int, num_experts: int,
                             previous_event=None, async_finish: bool = False,
                             return_recv_hook: bool = False, no_sync: bool = False):
        """Returns (recv_x [E, cap, H], recv_count [E] int32, handle, event, hook).
        With return_recv_hook the call fills counts and the handle only, and
        the rows arrive when hook() runs (a second kernel launch on the
        current stream); otherwise hook is None."""
        assert num_experts == self.num_experts
        x = _contiguous(x, previous_event)
        topk_idx = _contiguous(topk_idx, previous_event)
        T, H = x.shape
        K = topk_idx.shape[1]
        cap = num_max_dispatch_tokens_per_rank
        dev = x.device
        nbytes = ctypes.c_size_t()
        C.check(C.moedx_ll_workspace_bytes(self.ctx, T, K, cap, ctypes.byref(nbytes)))
        ws = torch.empty(nbytes.value, dtype=torch.uint8, device=dev)
        recv_x = torch.empty(num_experts, cap, H, dtype=torch.bfloat16, device=dev)
        cnt = torch.empty(num_experts, dtype=torch.int32, device=dev)
        h = ctypes.c_void_p()
        ex, done = self._exec(previous_event, async_finish, False, no_sync)
        C.check(C.moedx_ll_dispatch(self.ctx, _ptr(x), _ptr(topk_idx), T, K, H, cap,
                                    None if return_recv_hook else _ptr(recv_x), _ptr(cnt),
                                    _ptr(ws), nbytes.value, ctypes.byref(h), ctypes.byref(ex)))
        handle = Handle(h.value, ws, T, K, True)
        hook = None
        if return_recv_hook:
            def hook():
                rex = C.make_exec(_stream(), None, None, C.MOEDX_ASYNC)
                C.check(C.moedx_ll_dispatch_recv(self.ctx, handle.ptr, _ptr(x), _ptr(topk_idx), H,
                                                 _ptr(recv_x), ctypes.byref(rex)))
        return recv_x, cnt, handle, self._event(done), hook

    def low_latency_combine(self, x: torch.Tensor, topk_idx: torch.Tensor,
                            topk_weights: torch.Tensor, handle: Handle, previous_event=None,
                            async_finish: bool = False, return_recv_hook: bool = False,
                            out: Optional[torch.Tensor] = None, no_sync: bool = False):
        """Returns (combined [T, H] bf16, event, hook).  With return_recv_hook
        the reduction runs when hook() is called (on the current stream) and
        event is None; otherwise hook is None."""
        x = _contiguous(x, previous_event)
        H = x.shape[-1]
        T = handle.T
        combined = out if out is not None else torch.empty(T, H, dtype=torch.bfloat16, device=x.device)
        ti = _contiguous(topk_idx, previous_event)
        tw = _contiguous(topk_weights, previous_event)

        def run(ex):
            C.check(C.moedx_ll_combine(self.ctx, _ptr(x), _ptr(ti), _ptr(tw), handle.ptr, H,
                                       _ptr(combined), ctypes.byref(ex)))

        if return_recv_hook:
            prev = previous_event.event if previous_event is not None else None

            def hook():
                run(C.make_exec(_stream(), prev, None, C.MOEDX_ASYNC))
            return combined, EventOverlap(None), hook
        ex, done = self._exec(previous_event, async_finish, False, no_sync)
        run(ex)
        return combined, self._event(done), None

    # -- router, rows in expert order, the experts' products -----------------------
    def _check(self, name: str, t, dtypes, shape, previous_event=None) -> torch.Tensor:
        """`t` is a tensor on this Buffer's device, of one of `dtypes` and of
        `shape` (None = any size); made contiguous behind `previous_event`."""
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"{name} must be a tensor")
        if not t.is_cuda or t.get_device() != self._index:
            raise ValueError(f"{name} is on {t.device}, the Buffer on {self._torch_device}")
        if t.dtype not in dtypes:
            raise ValueError(f"{name} has dtype {t.dtype}, expected one of {list(dtypes)}")
        got = t.shape
        bad = len(got) != len(shape)
        if not bad:
            for n, m in zip(shape, got):
                if n is not None and n != m:
                    bad = True
        if bad:
            raise ValueError(f"{name} has shape {tuple(got)}, expected {tuple(shape)}")
        return t if t.is_contiguous() else _contiguous(t, previous_event)

    def _out(self, name: str, out, dtype, shape) -> torch.Tensor:
        """`out` checked (it must be contiguous), or a new tensor."""
        if out is None:
            return torch.empty(shape, dtype=dtype, device=self._torch_device)
        if isinstance(out, torch.Tensor) and not out.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        return self._check(name, out, (dtype,), shape)

    def _exec_here(self, previous_event, async_finish, allocate_on_comm_stream, no_sync):
        """As _exec, on the current stream of this Buffer's device."""
        if _deferred:
            _flush_deferred()
        done = ctypes.c_void_p() if async_finish else None
        flags = (C.MOEDX_ON_CTX_STREAM if allocate_on_comm_stream else 0) | (
            C.MOEDX_ASYNC if no_sync else 0)
        ex = C.moedx_exec()  # zeroed
        ex.stream = _raw_stream(self._index)
        ex.flags = flags
        if previous_event is not None:
            ex.prev = previous_event.event
        if done is not None:
            ex.done = ctypes.addressof(done)
        return ex, done

    def _gate_options(self, score, num_groups, groups_kept, renormalize, scale, bias,
                      previous_event):
        if score not in _SCORES:
            raise ValueError(f"score={score!r} must be one of {sorted(_SCORES)}")
        if bias is not None:
            bias = self._check("bias", bias, (torch.float32,), (self.num_experts,), previous_event)
        return C.moedx_gate(_SCORES[score], num_groups,
                            num_groups if groups_kept is None else groups_kept,
                            1 if renormalize else 0, scale, _addr(bias)), bias

    def gate_topk(self, logits: torch.Tensor, topk: int, score: str = "softmax",
                  num_groups: int = 1, groups_kept: Optional[int] = None,
                  renormalize: bool = False, scale: float = 1.0,
                  bias: Optional[torch.Tensor] = None,
                  previous_event: Optional[EventOverlap] = None, async_finish: bool = False,
                  allocate_on_comm_stream: bool = False, no_sync: bool = False):
        """Returns (topk_idx [T, topk] int64, topk_weights [T, topk] fp32,
        event) from the router's ``logits`` [T, E] (fp32, bf16 or fp16): what
        get_dispatch_layout and dispatch take.  ``score``: "softmax" or
        "sigmoid"; ``bias`` [E] fp32 is added to the scores for the choice
        only; with ``num_groups`` > 1 only the ``groups_kept`` groups with the
        best two-expert sums are chosen from; ``renormalize`` divides the
        chosen scores by their sum; ``scale`` multiplies the weights.  Experts
        with a logit of -inf or NaN are never chosen; slots that stay empty
        are -1 with weight 0."""
        logits = self._check("logits", logits, _DTYPES, (None, self.num_experts), previous_event)
        T = logits.shape[0]
        opts, bias = self._gate_options(score, num_groups, groups_kept, renormalize, scale, bias,
                                        previous_event)
        dev = self._torch_device
        idx = torch.empty(T, max(topk, 0), dtype=torch.int64, device=dev)
        w = torch.empty(T, max(topk, 0), dtype=torch.float32, device=dev)
        ex, done = self._exec_here(previous_event, async_finish, allocate_on_comm_stream, no_sync)
        C.check(C.moedx_gate_topk(self.ctx, _addr(logits), _DTYPES[logits.dtype], T, topk,
                                  ctypes.byref(opts), _addr(idx), _addr(w), ctypes.byref(ex)))
        self._keep(allocate_on_comm_stream, logits, bias, idx, w)
        return idx, w, self._event(done)

    def gate_topk_backward(self, d_topk_weights: torch.Tensor, logits: torch.Tensor,
                           topk_idx: torch.Tensor, score: str = "softmax", num_groups: int = 1,
                           groups_kept: Optional[int] = None, renormalize: bool = False,
                           scale: float = 1.0, bias: Optional[torch.Tensor] = None,
                           previous_event: Optional[EventOverlap] = None,
                           async_finish: bool = False, allocate_on_comm_stream: bool = False,
                           no_sync: bool = False):
        """Returns (d_logits [T, E] of the logits' dtype, event): the gradient
        of gate_topk's weights for its choice ``topk_idx`` with the same
        options (the choice, and so ``bias``, has no gradient)."""
        logits = self._check("logits", logits, _DTYPES, (None, self.num_experts), previous_event)
        T = logits.shape[0]
        topk_idx = self._check("topk_idx", topk_idx, (torch.int64,), (T, None), previous_event)
        K = topk_idx.shape[1]
        dw = self._check("d_topk_weights", d_topk_weights, (torch.float32,), (T, K), previous_event)
        opts, bias = self._gate_options(score, num_groups, groups_kept, renormalize, scale, bias,
                                        previous_event)
        d = torch.empty_like(logits)
        ex, done = self._exec_here(previous_event, async_finish, allocate_on_comm_stream, no_sync)
        C.check(C.moedx_gate_topk_backward(self.ctx, _addr(logits), _DTYPES[logits.dtype], T, K,
                                           ctypes.byref(opts), _addr(topk_idx), _addr(dw), _addr(d),
                                           ctypes.byref(ex)))
        self._keep(allocate_on_comm_stream, logits, bias, topk_idx, dw, d)
        return d, self._event(done)

    def expert_order(self, topk_idx: torch.Tensor, handle: Optional[Handle] = None,
                     previous_event: Optional[EventOverlap] = None, async_finish: bool = False,
                     allocate_on_comm_stream: bool = False, no_sync: bool = False):
        """Returns (ExpertOrder, event): the filled (token, slot) pairs of
        ``topk_idx`` [T, K] sorted by expert, then token, then slot.  With
        ``handle``, ``topk_idx`` is the recv_topk_idx of its first dispatch
        (ids local to the row's bucket; rows past N are empty).  Nothing is
        read on the host."""
        topk_idx = self._check("topk_idx", topk_idx, (torch.int64,), (None, None), previous_event)
        T, K = topk_idx.shape
        size = self._order_size  # read once: another thread may replace it
        if size[:2] != (T, K):
            nbytes = ctypes.c_size_t()
            C.check(C.moedx_expert_order_workspace_bytes(self.ctx, T, K, ctypes.byref(nbytes)))
            size = self._order_size = (T, K, nbytes.value)
        nbytes = size[2]
        dev = self._torch_device
        offsets = torch.empty(self.num_experts + 1, dtype=torch.int32, device=dev)
        row_of_slot = torch.empty(T, K, dtype=torch.int32, device=dev)
        slot_of_row = torch.empty(T * K, dtype=torch.int32, device=dev)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
        ex, done = self._exec_here(previous_event, async_finish, allocate_on_comm_stream, no_sync)
        C.check(C.moedx_expert_order(self.ctx, _addr(topk_idx), T, K,
                                     handle.ptr if handle is not None else None, _addr(offsets),
                                     _addr(row_of_slot), _addr(slot_of_row), _addr(ws), nbytes,
                                     ctypes.byref(ex)))
        self._keep(allocate_on_comm_stream, topk_idx, offsets, row_of_slot, slot_of_row, ws,
                   handle.workspace if handle is not None else None)
        return ExpertOrder(offsets, row_of_slot, slot_of_row), self._event(done)

    def expert_sort(self, x: torch.Tensor, order: ExpertOrder, out: Optional[torch.Tensor] = None,
                    previous_event: Optional[EventOverlap] = None, async_finish: bool = False,
                    allocate_on_comm_stream: bool = False, no_sync: bool = False):
        """Returns (rows [T * K, H], event): every filled pair's row of ``x``
        [T, H] (bf16, fp16 or fp32) in expert order.  Rows past the last pair
        are left as they were (unspecified without ``out``)."""
        T, K = order.row_of_slot.shape
        x = self._check("x", x, _DTYPES, (T, None), previous_event)
        H = x.shape[1]
        ros = self._check("row_of_slot", order.row_of_slot, (torch.int32,), (T, K), previous_event)
        rows = self._out("out", out, x.dtype, (T * K, H))
        ex, done = self._exec_here(previous_event, async_finish, allocate_on_comm_stream, no_sync)
        C.check(C.moedx_expert_sort(self.ctx, _addr(x), _DTYPES[x.dtype], T, K, H, _addr(ros),
                                    _addr(rows), ctypes.byref(ex)))
        self._keep(allocate_on_comm_stream, x, ros, rows)
        return rows, self._event(done)

    def expert_unsort(self, rows: torch.Tensor, order: ExpertOrder,
                      topk_weights: Optional[torch.Tensor] = None,
                      out: Optional[torch.Tensor] = None,
                      previous_event: Optional[EventOverlap] = None, async_finish: bool = False,
                      allocate_on_comm_stream: bool = False, no_sync: bool = False):
        """Returns (out [T, H], event): each token's rows back from expert
        order, scaled by ``topk_weights`` [T, K] fp32 (None = 1) and summed in
        fp32 over its filled slots; zero for a token without any."""
        T, K = order.row_of_slot.shape
        rows = self._check("rows", rows, _DTYPES, (T * K, None), previous_event)
        H = rows.shape[1]
        ros = self._check("row_of_slot", order.row_of_slot, (torch.int32,), (T, K), previous_event)
        w = None if topk_weights is None else self._check(
            "topk_weights", topk_weights, (torch.float32,), (T, K), previous_event)
        out = self._out("out", out, rows.dtype, (T, H))
        ex, done = self._exec_here(previous_event, async_finish, allocate_on_comm_stream, no_sync)
        C.check(C.moedx_expert_unsort(self.ctx, _addr(rows), _DTYPES[rows.dtype], T, K, H,
                                      _addr(ros), _addr(w), _addr(out), ctypes.byref(ex)))
        self._keep(allocate_on_comm_stream, rows, ros, w, out)
        return out, self._event(done)

    def expert_sort_backward(self, d_rows: torch.Tensor, order: ExpertOrder,
                             out: Optional[torch.Tensor] = None,
                             previous_event: Optional[EventOverlap] = None,
                             async_finish: bool = False, allocate_on_comm_stream: bool = False,
                             no_sync: bool = False):
        """Returns (d_x [T, H], event), the gradient of expert_sort: each
        token's row gradients summed (expert_unsort without weights)."""
        return self.expert_unsort(d_rows, order, None, out, previous_event, async_finish,
                                  allocate_on_comm_stream, no_sync)

    def expert_unsort_backward(self, d_out: torch.Tensor, rows: torch.Tensor, order: ExpertOrder,
                               topk_weights: torch.Tensor, out: Optional[torch.Tensor] = None,
                               previous_event: Optional[EventOverlap] = None,
                               async_finish: bool = False, allocate_on_comm_stream: bool = False,
                               no_sync: bool = False):
        """Returns (d_rows [T * K, H], d_topk_weights [T, K] fp32, event), the
        gradients of expert_unsort.  ``out``: where d_rows goes; rows past the
        last pair are left as they were."""
        T, K = order.row_of_slot.shape
        rows = self._check("rows", rows, _DTYPES, (T * K, None), previous_event)
        H = rows.shape[1]
        d_out = self._check("d_out", d_out, (rows.dtype,), (T, H), previous_event)
        ros = self._check("row_of_slot", order.row_of_slot, (torch.int32,), (T, K), previous_event)
        sor = self._check("slot_of_row", order.slot_of_row, (torch.int32,), (T * K,), previous_event)
        w = self._check("topk_weights", topk_weights, (torch.float32,), (T, K), previous_event)
        d_rows = self._out("out", out, rows.dtype, (T * K, H))
        d_w = torch.empty(T, K, dtype=torch.float32, device=rows.device)
        ex, done = self._exec_here(previous_event, async_finish, allocate_on_comm_stream, no_sync)
        C.check(C.moedx_expert_unsort_backward(self.ctx, _addr(d_out), _addr(rows),
                                               _DTYPES[rows.dtype], T, K, H, _addr(ros), _addr(sor),
                                               _addr(w), _addr(d_rows), _addr(d_w),
                                               ctypes.byref(ex)))
        self._keep(allocate_on_comm_stream, d_out, rows, ros, sor, w, d_rows, d_w)
        return d_rows, d_w, self._event(done)

    def _expert_rows(self, rows, x: torch.Tensor, previous_event):
        """The moedx_expert_rows of x's leading dimensions: an ExpertOrder or
        int32 offsets [E + 1] for [M, *], int32 counts [E] for [E, cap, *]."""
        E = self.num_experts
        t = rows.expert_offsets if isinstance(rows, ExpertOrder) else rows
        if x.dim() == 3:
            t = self._check("recv_count", t, (torch.int32,), (E,), previous_event)
            return C.moedx_expert_rows(None, _addr(t), x.shape[0] * x.shape[1]), t
        t = self._check("expert_offsets", t, (torch.int32,), (E + 1,), previous_event)
        return C.moedx_expert_rows(_addr(t), None, x.shape[0]), t

    def _lead(self, name: str, x) -> tuple:
        """Leading dimensions of a row buffer: (M,) or (E, cap)."""
        if not isinstance(x, torch.Tensor) or x.dim() not in (2, 3):
            raise ValueError(f"{name} must be a [M, *] or [num_experts, cap, *] tensor")
        if x.dim() == 3 and x.shape[0] != self.num_experts:
            raise ValueError(f"{name} has {x.shape[0]} experts, expected {self.num_experts}")
        return tuple(x.shape[:-1])

    def expert_linear(self, x: torch.Tensor, w: torch.Tensor, rows, swiglu: bool = False,
                      return_pre: bool = False, out: Optional[torch.Tensor] = None,
                      previous_event: Optional[EventOverlap] = None, async_finish: bool = False,
                      allocate_on_comm_stream: bool = False, no_sync: bool = False):
        """Returns (y, pre, event): every row of ``x`` times its expert's
        matrix, y[m] = w[e] x[m], for ``w`` [E, N, K] (bf16 or fp16).  ``x`` is
        [M, K] with ``rows`` an ExpertOrder (or its int32 expert_offsets
        [E + 1]), or low_latency_dispatch's [E, cap, K] with ``rows`` its int32
        recv_count [E].  With ``swiglu``, ``w`` is [E, 2N, K] (gate rows, then
        up rows) and y = silu(gate) * up; ``return_pre`` also gives the rounded
        (gate, up) values [*, 2N] that expert_swiglu_backward takes, else pre
        is None.  Rows of no expert are left as they were (unspecified without
        ``out``).  Weights that are not contiguous are copied on every call."""
        lead = self._lead("x", x)
        x = self._check("x", x, _PRODUCT_DTYPES, lead + (None,), previous_event)
        K = x.shape[-1]
        w = self._check("w", w, (x.dtype,), (self.num_experts, None, K), previous_event)
        N = w.shape[1]
        if swiglu:
            if N % 2 != 0:
                raise ValueError(f"w has {N} rows per expert, expected gate and up halves")
            N //= 2
        elif return_pre:
            raise ValueError("return_pre needs swiglu")
        er, t = self._expert_rows(rows, x, previous_event)
        y = self._out("out", out, x.dtype, lead + (N,))
        pre = torch.empty(lead + (2 * N,), dtype=x.dtype, device=x.device) if return_pre else None
        ex, done = self._exec_here(previous_event, async_finish, allocate_on_comm_stream, no_sync)
        C.check(C.moedx_expert_linear(self.ctx, _addr(x), _addr(w), _DTYPES[x.dtype], K, N,
                                      ctypes.byref(er), 1 if swiglu else 0, _addr(y), _addr(pre),
                                      ctypes.byref(ex)))
        self._keep(allocate_on_comm_stream, x, w, t, y, pre)
        return y, pre, self._event(done)

    def expert_linear_backward(self, d_y: torch.Tensor, x: Optional[torch.Tensor],
                               w: Optional[torch.Tensor], rows,
                               out: Optional[torch.Tensor] = None,
                               d_w: Optional[torch.Tensor] = None, d_w_dtype=None,
                               previous_event: Optional[EventOverlap] = None,
                               async_finish: bool = False, allocate_on_comm_stream: bool = False,
                               no_sync: bool = False):
        """Returns (d_x, d_w, event), the gradients of expert_linear without
        its activation: d_x[m] = w[e]^T d_y[m] (rows of no expert left as they
        were in ``out``) and d_w[e] = the sum of d_y[m] x[m]^T over e's rows
        (zero without any), written to ``d_w`` (of w's dtype or fp32) or to a
        new tensor of ``d_w_dtype`` (w's dtype by default).  ``w`` None leaves
        d_x out, ``x`` None d_w (each is then None): where x is computed again
        from d_x, as with expert_swiglu_backward_int8, the two are asked for
        one after the other."""
        lead = self._lead("d_y" if x is None else "x", d_y if x is None else x)
        if x is not None:
            x = self._check("x", x, _PRODUCT_DTYPES, lead + (None,), previous_event)
            K, dtype = x.shape[-1], x.dtype
            if w is not None:
                w = self._check("w", w, (dtype,), (self.num_experts, None, K), previous_event)
        elif w is None:
            raise ValueError("x or w is needed")
        else:
            w = self._check("w", w, _PRODUCT_DTYPES, (self.num_experts, None, None), previous_event)
            K, dtype = w.shape[2], w.dtype
        N = None if w is None else w.shape[1]
        d_y = self._check("d_y", d_y, (dtype,), lead + (N,), previous_event)
        N = d_y.shape[-1]
        if x is None and (d_w is not None or d_w_dtype is not None):
            raise ValueError("d_w needs x")
        if w is None and out is not None:
            raise ValueError("out needs w")
        if d_w_dtype is None:
            d_w_dtype = dtype if d_w is None else d_w.dtype
        if d_w_dtype not in (dtype, torch.float32):
            raise ValueError(f"d_w_dtype={d_w_dtype} must be {dtype} or torch.float32")
        er, t = self._expert_rows(rows, d_y, previous_event)
        d_x = None if w is None else self._out("out", out, dtype, lead + (K,))
        if x is not None:
            d_w = self._out("d_w", d_w, d_w_dtype, (self.num_experts, N, K))
        ex, done = self._exec_here(previous_event, async_finish, allocate_on_comm_stream, no_sync)
        C.check(C.moedx_expert_linear_backward(self.ctx, _addr(d_y), _addr(x), _addr(w),
                                               _DTYPES[dtype], K, N, ctypes.byref(er), _addr(d_x),
                                               _addr(d_w), _DTYPES[d_w_dtype], ctypes.byref(ex)))
        self._keep(allocate_on_comm_stream, d_y, x, w, t, d_x, d_w)
        return d_x, d_w, self._event(done)

    def expert_swiglu_backward(self, d_h: torch.Tensor, pre: torch.Tensor, rows,
                               out: Optional[torch.Tensor] = None,
                               previous_event: Optional[EventOverlap] = None,
                               async_finish: bool = False, allocate_on_comm_stream: bool = False,
                               no_sync: bool = False):
        """Returns (d_pre [*, 2N], event): the gradient of expert_linear's
        swiglu at ``pre`` = (gate, up) for ``d_h`` [*, N]; expert_linear_backward
        takes d_pre as its d_y.  Rows of no expert are left as they were."""
        lead = self._lead("d_h", d_h)
        d_h = self._check("d_h", d_h, _PRODUCT_DTYPES, lead + (None,), previous_event)
        N = d_h.shape[-1]
        pre = self._check("pre", pre, (d_h.dtype,), lead + (2 * N,), previous_event)
        er, t = self._expert_rows(rows, d_h, previous_event)
        d_pre = self._out("out", out, d_h.dtype, lead + (2 * N,))
        ex, done = self._exec_here(previous_event, async_finish, allocate_on_comm_stream, no_sync)
        C.check(C.moedx_expert_swiglu_backward(self.ctx, _addr(d_h), _addr(pre), _DTYPES[d_h.dtype],
                                               N, ctypes.byref(er), _addr(d_pre),
                                               ctypes.byref(ex)))
        self._keep(allocate_on_comm_stream, d_h, pre, t, d_pre)
        return d_pre, self._event(done)

    # -- the experts' rows in int8 -----------------------------------------------------
    # These calls take the options of every call by name: previous_event,
    # async_finish, allocate_on_comm_stream, no_sync.
    @staticmethod
    def _options(options: dict) -> tuple:
        for name in options:
            if name not in _OPTIONS:
                raise TypeError(f"unexpected argument {name!r}, expected one of {_OPTIONS}")
        get = options.get
        return (get("previous_event"), get("async_finish", False),
                get("allocate_on_comm_stream", False), get("no_sync", False))

    def _any_rows(self, rows, x: torch.Tensor, previous_event):
        """_expert_rows, or every row of x where `rows` is None."""
        if rows is not None:
            return self._expert_rows(rows, x, previous_event)
        return C.moedx_expert_rows(None, None, x.numel() // max(x.shape[-1], 1)), None

    @staticmethod
    def _scale_shape(lead: tuple, H: int, block: int) -> tuple:
        if block not in (0, 128):
            raise ValueError(f"block={block} must be 0 (a scale per row) or 128")
        return lead if block == 0 else lead + ((H + block - 1) // block,)

    def _codes(self, name: str, codes, scales, width, previous_event):
        """(codes, scales, block) checked: int8 rows [*, width] with their scales."""
        lead = self._lead(name, codes)
        codes = self._check(name, codes, _INT8, lead + (width,), previous_event)
        if not isinstance(scales, torch.Tensor):
            raise ValueError(f"{name}_scales must be a tensor")
        if scales.dim() == len(lead):
            block, shape = 0, lead
        else:
            block, shape = 128, lead + ((codes.shape[-1] + 127) // 128,)
        return codes, self._check(f"{name}_scales", scales, _FP32, shape, previous_event), block

    def expert_quantize(self, x: torch.Tensor, rows=None, block: int = 0,
                        out: Optional[torch.Tensor] = None,
                        scales: Optional[torch.Tensor] = None, **options):
        """Returns (codes int8, scales fp32, event) of ``x`` [M, H] with ``rows``
        an ExpertOrder (or its int32 expert_offsets), or [E, cap, H] with
        ``rows`` int32 recv_count (bf16, fp16 or fp32); ``rows`` None takes every
        row (weights [E, N, K]).  ``block`` 0: a scale per row (scales [M] or
        [E, cap]: what expert_linear_int8 takes); 128: one per 128 values
        (scales [*, ceil(H / 128)]: finer, for saved rows).  A value is code *
        scale; codes are in [-127, 127], a scale is the largest magnitude /
        127.  Rows with an inf or NaN stay NaN.  Rows of no expert are left as
        they were in ``out`` and ``scales`` (unspecified without).  The backward
        calls in int8 and expert_dequantize take codes and scales as they are."""
        prev, async_finish, comm, no_sync = self._options(options)
        lead = self._lead("x", x)
        x = self._check("x", x, _DTYPES, lead + (None,), prev)
        H = x.shape[-1]
        er, t = self._any_rows(rows, x, prev)
        codes = self._out("out", out, torch.int8, lead + (H,))
        scales = self._out("scales", scales, torch.float32, self._scale_shape(lead, H, block))
        ex, done = self._exec_here(prev, async_finish, comm, no_sync)
        C.check(C.moedx_expert_quantize(self.ctx, _addr(x), _DTYPES[x.dtype], H, block,
                                        ctypes.byref(er), _addr(codes), _addr(scales),
                                        ctypes.byref(ex)))
        self._keep(comm, x, t, codes, scales)
        return codes, scales, self._event(done)

    def expert_dequantize(self, codes: torch.Tensor, scales: torch.Tensor, rows=None,
                          dtype: torch.dtype = torch.bfloat16,
                          out: Optional[torch.Tensor] = None, **options):
        """Returns (x, event): expert_quantize's rows restored in ``dtype``, code *
        scale rounded once.  Rows of no expert are left as they were."""
        prev, async_finish, comm, no_sync = self._options(options)
        codes, scales, block = self._codes("codes", codes, scales, None, prev)
        if dtype not in _DTYPES:
            raise ValueError(f"dtype={dtype} must be one of {list(_DTYPES)}")
        er, t = self._any_rows(rows, codes, prev)
        x = self._out("out", out, dtype, tuple(codes.shape))
        ex, done = self._exec_here(prev, async_finish, comm, no_sync)
        C.check(C.moedx_expert_dequantize(self.ctx, _addr(codes), _addr(scales), codes.shape[-1],
                                          block, ctypes.byref(er), _addr(x), _DTYPES[dtype],
                                          ctypes.byref(ex)))
        self._keep(comm, codes, scales, t, x)
        return x, self._event(done)

    def expert_sort_int8(self, x: torch.Tensor, order: ExpertOrder,
                         out: Optional[torch.Tensor] = None,
                         scales: Optional[torch.Tensor] = None, **options):
        """Returns (codes [T * K, H] int8, scales [T * K] fp32, event): expert_sort
        and expert_quantize in one: each row of ``x`` [T, H] is quantised once,
        with one scale, and put at its filled slots' rows in expert order.
        Rows past the last pair are left as they were."""
        prev, async_finish, comm, no_sync = self._options(options)
        T, K = order.row_of_slot.shape
        x = self._check("x", x, _DTYPES, (T, None), prev)
        H = x.shape[1]
        ros = self._check("row_of_slot", order.row_of_slot, (torch.int32,), (T, K), prev)
        codes = self._out("out", out, torch.int8, (T * K, H))
        scales = self._out("scales", scales, torch.float32, (T * K,))
        ex, done = self._exec_here(prev, async_finish, comm, no_sync)
        C.check(C.moedx_expert_sort_int8(self.ctx, _addr(x), _DTYPES[x.dtype], T, K, H, _addr(ros),
                                         _addr(codes), _addr(scales), ctypes.byref(ex)))
        self._keep(comm, x, ros, codes, scales)
        return codes, scales, self._event(done)

    def expert_linear_int8(self, x: torch.Tensor, x_scales: torch.Tensor, w: torch.Tensor,
                           w_scales: torch.Tensor, rows, swiglu: bool = False,
                           dtype: torch.dtype = torch.bfloat16,
                           out: Optional[torch.Tensor] = None, **options):
        """Returns (y, event): expert_linear in int8.  ``x`` and its scales are
        expert_quantize's (or expert_sort_int8's) with a scale per row, ``w``
        [E, N, K] int8 with ``w_scales`` [E, N] a model's weights, quantised once
        (expert_quantize(w)).  y is of ``dtype`` (bf16 or fp16): the exact
        integer sum times both scales, with ``swiglu`` as expert_linear.  A
        row's results do not depend on its place or on other rows."""
        prev, async_finish, comm, no_sync = self._options(options)
        x, x_scales, block = self._codes("x", x, x_scales, None, prev)
        if block:
            raise ValueError("x's scales must be one per row (block=0)")
        lead, K = tuple(x.shape[:-1]), x.shape[-1]
        w = self._check("w", w, _INT8, (self.num_experts, None, K), prev)
        N = w.shape[1]
        w_scales = self._check("w_scales", w_scales, _FP32, (self.num_experts, N), prev)
        if dtype not in _PRODUCT_DTYPES:
            raise ValueError(f"dtype={dtype} must be one of {list(_PRODUCT_DTYPES)}")
        if swiglu:
            if N % 2 != 0:
                raise ValueError(f"w has {N} rows per expert, expected gate and up halves")
            N //= 2
        er, t = self._expert_rows(rows, x, prev)
        y = self._out("out", out, dtype, lead + (N,))
        ex, done = self._exec_here(prev, async_finish, comm, no_sync)
        C.check(C.moedx_expert_linear_int8(self.ctx, _addr(x), _addr(x_scales), _addr(w),
                                           _addr(w_scales), K, N, ctypes.byref(er),
                                           1 if swiglu else 0, _addr(y), _DTYPES[dtype],
                                           ctypes.byref(ex)))
        self._keep(comm, x, x_scales, w, w_scales, t, y)
        return y, self._event(done)

    def expert_linear_backward_int8(self, d_y: torch.Tensor, x: torch.Tensor,
                                    x_scales: torch.Tensor, w: Optional[torch.Tensor], rows,
                                    out: Optional[torch.Tensor] = None,
                                    d_w: Optional[torch.Tensor] = None, d_w_dtype=None, **options):
        """Returns (d_x, d_w, event): expert_linear_backward of rows that were
        saved in int8 (expert_quantize, either block): d_w is that of
        expert_dequantize(x) in d_y's dtype, without the restored rows in
        memory.  ``w`` None leaves d_x out (None)."""
        prev, async_finish, comm, no_sync = self._options(options)
        x, x_scales, block = self._codes("x", x, x_scales, None, prev)
        lead, K = tuple(x.shape[:-1]), x.shape[-1]
        d_y = self._check("d_y", d_y, _PRODUCT_DTYPES, lead + (None,), prev)
        N = d_y.shape[-1]
        if w is not None:
            w = self._check("w", w, (d_y.dtype,), (self.num_experts, N, K), prev)
        elif out is not None:
            raise ValueError("out needs w")
        if d_w_dtype is None:
            d_w_dtype = d_y.dtype if d_w is None else d_w.dtype
        if d_w_dtype not in (d_y.dtype, torch.float32):
            raise ValueError(f"d_w_dtype={d_w_dtype} must be {d_y.dtype} or torch.float32")
        er, t = self._expert_rows(rows, x, prev)
        d_x = None if w is None else self._out("out", out, d_y.dtype, lead + (K,))
        d_w = self._out("d_w", d_w, d_w_dtype, (self.num_experts, N, K))
        ex, done = self._exec_here(prev, async_finish, comm, no_sync)
        C.check(C.moedx_expert_linear_backward_int8(
            self.ctx, _addr(d_y), _addr(x), _addr(x_scales), block, _addr(w), _DTYPES[d_y.dtype], K,
            N, ctypes.byref(er), _addr(d_x), _addr(d_w), _DTYPES[d_w_dtype], ctypes.byref(ex)))
        self._keep(comm, d_y, x, x_scales, w, t, d_x, d_w)
        return d_x, d_w, self._event(done)

    def expert_swiglu_backward_int8(self, d_h: torch.Tensor, pre: torch.Tensor,
                                    pre_scales: torch.Tensor, rows, return_h: bool = False,
                                    out: Optional[torch.Tensor] = None,
                                    h: Optional[torch.Tensor] = None, **options):
        """Returns (d_pre [*, 2N], h, event): expert_swiglu_backward at (gate, up)
        values saved in int8 (expert_quantize of expert_linear's pre).  With
        ``return_h`` (or ``h`` to write to) also the activation's output [*, N] at
        them, which the next weight gradient takes: neither pre nor h need be
        kept in 16 bits.  Rows of no expert are left as they were."""
        prev, async_finish, comm, no_sync = self._options(options)
        lead = self._lead("d_h", d_h)
        d_h = self._check("d_h", d_h, _PRODUCT_DTYPES, lead + (None,), prev)
        N = d_h.shape[-1]
        pre, pre_scales, block = self._codes("pre", pre, pre_scales, 2 * N, prev)
        if tuple(pre.shape[:-1]) != lead:
            raise ValueError(f"pre has shape {tuple(pre.shape)}, expected {lead + (2 * N,)}")
        er, t = self._expert_rows(rows, d_h, prev)
        d_pre = self._out("out", out, d_h.dtype, lead + (2 * N,))
        if return_h or h is not None:
            h = self._out("h", h, d_h.dtype, lead + (N,))
        ex, done = self._exec_here(prev, async_finish, comm, no_sync)
        C.check(C.moedx_expert_swiglu_backward_int8(
            self.ctx, _addr(d_h), _addr(pre), _addr(pre_scales), block, _DTYPES[d_h.dtype], N,
            ctypes.byref(er), _addr(d_pre), _addr(h), ctypes.byref(ex)))
        self._keep(comm, d_h, pre, pre_scales, t, d_pre, h)
        return d_pre, h, self._event(done)
