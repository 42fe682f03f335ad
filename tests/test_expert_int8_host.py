"""The int8 calls without a GPU: a null ctx, strided inputs behind previous_event,
and what the Python methods refuse (on a Buffer without a device, with CPU
tensors that pass for device memory)."""

import ctypes

import pytest
import torch

from tests.test_capi_host import capi  # noqa: F401
from tests.test_event_order_host import (E, EVENT, H, K, N, STREAM, T, bench, dense,  # noqa: F401
                                         strided)

P = ctypes.c_void_p(256)  # never read: the calls are refused first
M = T * K
I8, I32, F32, BF16 = torch.int8, torch.int32, torch.float32, torch.bfloat16


@pytest.mark.parametrize("call", [
    lambda C, e: C.moedx_expert_quantize(None, P, 0, 16, 0, e, P, P, None),
    lambda C, e: C.moedx_expert_dequantize(None, P, P, 16, 0, e, P, 0, None),
    lambda C, e: C.moedx_expert_sort_int8(None, P, 0, 4, 2, 16, P, P, P, None),
    lambda C, e: C.moedx_expert_linear_int8(None, P, P, P, P, 16, 8, e, 0, P, 0, None),
    lambda C, e: C.moedx_expert_linear_backward_int8(None, P, P, P, 0, P, 0, 16, 8, e, P, P, 0, None),
    lambda C, e: C.moedx_expert_swiglu_backward_int8(None, P, P, P, 0, 0, 8, e, P, P, None),
], ids=["quantize", "dequantize", "sort", "linear", "linear_backward", "swiglu_backward"])
def test_null_ctx(capi, call):  # noqa: F811
    er = capi.moedx_expert_rows(P, None, 8)
    assert call(capi, ctypes.byref(er)) == capi.MOEDX_EINVAL
    assert capi.last_error()


def calls(buf, make):
    """Every method with its tensors from make(shape, dtype)."""
    from combine_get_dispatch_layout_amd import ExpertOrder
    order = ExpertOrder(None, make((T, K), I32), None)
    rows, counts = make((E + 1,), I32), make((E,), I32)
    return {
        "expert_quantize": lambda **k: buf.expert_quantize(make((M, H), BF16), rows, **k),
        "expert_quantize, all": lambda **k: buf.expert_quantize(make((E, N, H), F32), **k),
        "expert_quantize, counts": lambda **k: buf.expert_quantize(dense((E, 3, H), BF16), counts, **k),
        "expert_dequantize": lambda **k: buf.expert_dequantize(make((M, H), I8), make((M,), F32), rows,
                                                               **k),
        "expert_dequantize, scales": lambda **k: buf.expert_dequantize(
            dense((M, H), I8), make((M, 1), F32), None, **k),
        "expert_sort_int8": lambda **k: buf.expert_sort_int8(make((T, H), BF16), order, **k),
        "expert_linear_int8": lambda **k: buf.expert_linear_int8(
            make((M, H), I8), make((M,), F32), make((E, 2 * N, H), I8), make((E, 2 * N), F32), rows,
            swiglu=True, **k),
        "expert_linear_int8, counts": lambda **k: buf.expert_linear_int8(
            dense((E, 3, H), I8), dense((E, 3), F32), dense((E, N, H), I8), make((E, N), F32), counts,
            **k),
        "expert_linear_backward_int8": lambda **k: buf.expert_linear_backward_int8(
            make((M, N), BF16), make((M, H), I8), make((M,), F32), make((E, N, H), BF16), rows, **k),
        "expert_linear_backward_int8, d_w": lambda **k: buf.expert_linear_backward_int8(
            dense((M, N), BF16), dense((M, H), I8), make((M, 1), F32), None, rows, **k),
        "expert_swiglu_backward_int8": lambda **k: buf.expert_swiglu_backward_int8(
            make((M, N), BF16), make((M, 2 * N), I8), make((M,), F32), rows, return_h=True, **k),
        "expert_linear_backward, d_x": lambda **k: buf.expert_linear_backward(
            make((M, N), BF16), None, make((E, N, H), BF16), rows, **k),
        "expert_linear_backward, d_w": lambda **k: buf.expert_linear_backward(
            make((M, N), BF16), make((M, H), BF16), None, rows, **k),
    }


NAMES = ["expert_quantize", "expert_quantize, all", "expert_quantize, counts", "expert_dequantize",
         "expert_dequantize, scales", "expert_sort_int8", "expert_linear_int8",
         "expert_linear_int8, counts", "expert_linear_backward_int8",
         "expert_linear_backward_int8, d_w", "expert_swiglu_backward_int8",
         "expert_linear_backward, d_x", "expert_linear_backward, d_w"]


@pytest.mark.parametrize("name", NAMES)
def test_copies_wait_for_the_event(bench, name):  # noqa: F811
    from combine_get_dispatch_layout_amd import EventOverlap
    buf, log = bench
    event = EventOverlap()
    event.event = EVENT
    call = calls(buf, strided)[name]
    try:
        call(previous_event=event)
    finally:
        event.event = None
    assert "copy" in log and log[0] == (EVENT, STREAM), log
    del log[:]
    call()
    call(previous_event=EventOverlap())
    assert set(log) == {"copy"}
    del log[:]
    event.event = EVENT
    try:
        calls(buf, dense)[name](previous_event=event)
    finally:
        event.event = None
    assert log == []


def test_every_method_is_here(bench):  # noqa: F811
    import inspect
    buf, _ = bench
    methods = {n for n in dir(type(buf)) if not n.startswith("_") and callable(getattr(type(buf), n))
               and any(p.kind is p.VAR_KEYWORD
                       for p in inspect.signature(getattr(type(buf), n)).parameters.values())}
    assert set(calls(buf, dense)) == set(NAMES)
    assert methods == {n.split(",")[0] for n in NAMES} - {"expert_linear_backward"}


def test_refusals(bench):  # noqa: F811
    buf, _ = bench
    x, rows, order = dense((M, H), BF16), dense((E + 1,), I32), None
    c, s, s128 = dense((M, H), I8), dense((M,), F32), dense((M, 1), F32)
    w, ws = dense((E, N, H), I8), dense((E, N), F32)
    w16, d_y = dense((E, N, H), BF16), dense((M, N), BF16)
    pre = dense((M, 2 * N), I8)
    slots = dense((E, 3, H), BF16)
    from combine_get_dispatch_layout_amd import ExpertOrder
    order = ExpertOrder(None, dense((T, K), I32), None)
    for f in (
        lambda: buf.expert_quantize(x.double(), rows), lambda: buf.expert_quantize(x[0], rows),
        lambda: buf.expert_quantize(x, rows, block=64), lambda: buf.expert_quantize(x, rows[:E]),
        lambda: buf.expert_quantize(x, rows.long()), lambda: buf.expert_quantize(slots, rows),
        lambda: buf.expert_quantize(slots[:2]), lambda: buf.expert_quantize(x, rows, out=x),
        lambda: buf.expert_quantize(x, rows, scales=s128), lambda: buf.expert_quantize(x, rows, 128, scales=s),
        lambda: buf.expert_quantize(x, rows, out=strided((M, H), I8)), lambda: buf.expert_quantize(None),
        lambda: buf.expert_dequantize(x, s, rows), lambda: buf.expert_dequantize(c, None, rows),
        lambda: buf.expert_dequantize(c, s[:5], rows), lambda: buf.expert_dequantize(c, s.double(), rows),
        lambda: buf.expert_dequantize(c, dense((M, 2), F32), rows),
        lambda: buf.expert_dequantize(c, s, rows, dtype=torch.float64),
        lambda: buf.expert_dequantize(c, s, rows, out=dense((M, H), F32)),
        lambda: buf.expert_sort_int8(x, order), lambda: buf.expert_sort_int8(dense((T, H), I8), order),
        lambda: buf.expert_linear_int8(c, s128, w, ws, rows), lambda: buf.expert_linear_int8(x, s, w, ws, rows),
        lambda: buf.expert_linear_int8(c, s, w16, ws, rows), lambda: buf.expert_linear_int8(c, s, w, ws[0], rows),
        lambda: buf.expert_linear_int8(c, s, w[:, :, :8], ws, rows),
        lambda: buf.expert_linear_int8(c, s, w[:2], ws[:2], rows),
        lambda: buf.expert_linear_int8(c, s, w, ws, rows, dtype=F32),
        lambda: buf.expert_linear_int8(c, s, w, ws, None),
        lambda: buf.expert_linear_int8(c, s, w[:, :7].contiguous(), ws[:, :7].contiguous(), rows, swiglu=True),
        lambda: buf.expert_linear_int8(c, s, w, ws, rows, out=dense((M, N), torch.float16)),
        lambda: buf.expert_linear_backward_int8(d_y[:5], c, s, w16, rows),
        lambda: buf.expert_linear_backward_int8(d_y.float(), c, s, w16, rows),
        lambda: buf.expert_linear_backward_int8(d_y, c, s, w16.half(), rows),
        lambda: buf.expert_linear_backward_int8(d_y, c, s, None, rows, out=x),
        lambda: buf.expert_linear_backward_int8(d_y, c, s, w16, rows, d_w_dtype=torch.float16),
        lambda: buf.expert_linear_backward_int8(d_y, c, s, w16, rows, d_w=w16[:2]),
        lambda: buf.expert_swiglu_backward_int8(d_y, pre[:, :N].contiguous(), s, rows),
        lambda: buf.expert_swiglu_backward_int8(d_y[:5], pre, s, rows),
        lambda: buf.expert_swiglu_backward_int8(d_y, pre, s, rows, h=pre),
        lambda: buf.expert_swiglu_backward_int8(d_y, pre.float(), s, rows),
        lambda: buf.expert_linear_backward(d_y, None, None, rows),
        lambda: buf.expert_linear_backward(d_y, None, w16, rows, d_w=w16),
        lambda: buf.expert_linear_backward(d_y, None, w16, rows, d_w_dtype=F32),
        lambda: buf.expert_linear_backward(d_y, x, None, rows, out=x),
        lambda: buf.expert_linear_backward(d_y[:5], x, None, rows),
        lambda: buf.expert_linear_backward(d_y[:, :5].contiguous(), None, w16, rows),
    ):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: buf.expert_quantize(x, rows, prev=None),
              lambda: buf.expert_linear_int8(c, s, w, ws, rows, return_pre=True)):
        with pytest.raises(TypeError):
            f()
