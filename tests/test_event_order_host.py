"""Strided inputs and previous_event without a GPU: every method of Buffer copies
a strided input only behind the event that orders it.  The library's calls are
replaced by ones that return OK and record themselves, the tensors by CPU ones
that pass for device memory and record their copies."""

import inspect

import pytest
import torch

from tests.test_capi_host import capi  # noqa: F401

E, T, K, H, N, R = 4, 6, 2, 16, 8, 2
EVENT, STREAM = 0x1230, 77


class DeviceTensor(torch.Tensor):
    is_cuda = True
    log = []

    def get_device(self):
        return 0

    def contiguous(self, *args, **kw):
        if not self.is_contiguous():
            self.log.append("copy")
        return super().contiguous(*args, **kw)


def dense(shape, dtype):
    return torch.zeros(shape, dtype=dtype).as_subclass(DeviceTensor)


def strided(shape, dtype):
    return dense(tuple(shape) + (2,), dtype)[..., 0]


@pytest.fixture
def bench(capi, monkeypatch):  # noqa: F811
    """(a Buffer without a device, the record of events waited for and copies)"""
    from combine_get_dispatch_layout_amd import buffer as b

    log = DeviceTensor.log = []

    def record(name):
        def call(*args):
            if name == "moedx_event_wait":
                log.append((args[0], args[1]))
            elif name == "moedx_handle_num_recv":
                args[1]._obj.value = T
            return capi.MOEDX_OK
        return call

    for name in capi.SIGNATURES:
        monkeypatch.setattr(capi, name, record(name))
    monkeypatch.setattr(b, "_stream", lambda: STREAM)
    monkeypatch.setattr(b, "_raw_stream", lambda index: STREAM)
    buf = object.__new__(b.Buffer)
    buf.device, buf.num_experts, buf.num_ranks, buf.ctx = 0, E, R, None
    buf._torch_device, buf._index, buf._order_size = torch.device("cpu"), 0, (None, None, 0)
    buf._keep = lambda *args: None
    return buf, log


def calls(buf, make):
    """Every method with its tensors from make(shape, dtype)."""
    from combine_get_dispatch_layout_amd import ExpertOrder
    from combine_get_dispatch_layout_amd.buffer import Handle
    bf16, f32, i32, i64 = torch.bfloat16, torch.float32, torch.int32, torch.int64
    M = T * K
    h = Handle(None, dense((1,), torch.uint8), T, K, False)
    order = ExpertOrder(make((E + 1,), i32), make((T, K), i32), make((M,), i32))
    rows = make((E + 1,), i32)
    return {
        "get_dispatch_layout": lambda ev: buf.get_dispatch_layout(make((T, K), i64), E,
                                                                  previous_event=ev),
        "prepare": lambda ev: buf.prepare(make((T, K), i64), 0, ev),
        "prepare from a layout": lambda ev: buf.prepare(
            dense((T, K), i64), 0, ev, num_tokens_per_rank=make((R,), i32),
            is_token_in_rank=make((T, R), torch.bool), num_tokens_per_expert=make((E,), i32)),
        "dispatch": lambda ev: buf.dispatch(make((T, H), bf16), topk_idx=make((T, K), i64),
                                            topk_weights=make((T, K), f32), previous_event=ev),
        "dispatch, weights": lambda ev: buf.dispatch(dense((T, H), bf16),
                                                     topk_idx=dense((T, K), i64),
                                                     topk_weights=make((T, K), f32),
                                                     previous_event=ev,
                                                     allocate_on_comm_stream=True),
        "dispatch of codes": lambda ev: buf.dispatch(
            (make((T, 128), torch.uint8), make((T, 2), f32)), h, previous_event=ev),
        "cached dispatch": lambda ev: buf.dispatch(make((T, H), bf16), h, previous_event=ev),
        "combine": lambda ev: buf.combine(make((T, H), bf16), h, make((T, K), f32),
                                          make((T, K), f32), previous_event=ev),
        "combine, weights": lambda ev: buf.combine(dense((T, H), bf16), h, make((T, K), f32),
                                                   make((T, K), f32), previous_event=ev),
        "low_latency_dispatch": lambda ev: buf.low_latency_dispatch(
            make((T, H), bf16), make((T, K), i64), 8, E, ev),
        "low_latency_combine": lambda ev: buf.low_latency_combine(
            make((E, 8, H), bf16), make((T, K), i64), make((T, K), f32), h, ev),
        "low_latency_combine, hook": lambda ev: buf.low_latency_combine(
            dense((E, 8, H), bf16), make((T, K), i64), make((T, K), f32), h, ev,
            return_recv_hook=True),
        "gate_topk": lambda ev: buf.gate_topk(make((T, E), f32), K, bias=make((E,), f32),
                                              previous_event=ev),
        "gate_topk, bias": lambda ev: buf.gate_topk(dense((T, E), f32), K, bias=make((E,), f32),
                                                    previous_event=ev),
        "gate_topk_backward": lambda ev: buf.gate_topk_backward(
            make((T, K), f32), make((T, E), f32), make((T, K), i64), bias=make((E,), f32),
            previous_event=ev),
        "expert_order": lambda ev: buf.expert_order(make((T, K), i64), previous_event=ev),
        "expert_sort": lambda ev: buf.expert_sort(make((T, H), bf16), order, previous_event=ev),
        "expert_unsort": lambda ev: buf.expert_unsort(make((M, H), bf16), order,
                                                      make((T, K), f32), previous_event=ev),
        "expert_sort_backward": lambda ev: buf.expert_sort_backward(make((M, H), bf16), order,
                                                                    previous_event=ev),
        "expert_unsort_backward": lambda ev: buf.expert_unsort_backward(
            make((T, H), bf16), make((M, H), bf16), order, make((T, K), f32), previous_event=ev),
        "expert_linear": lambda ev: buf.expert_linear(
            make((M, H), bf16), make((E, 2 * N, H), bf16), rows, swiglu=True, return_pre=True,
            previous_event=ev),
        "expert_linear, offsets": lambda ev: buf.expert_linear(
            dense((M, H), bf16), dense((E, N, H), bf16), rows, previous_event=ev),
        "expert_linear, counts": lambda ev: buf.expert_linear(
            dense((E, 3, H), bf16), dense((E, N, H), bf16), make((E,), i32), previous_event=ev),
        "expert_linear_backward": lambda ev: buf.expert_linear_backward(
            make((M, N), bf16), make((M, H), bf16), make((E, N, H), bf16), rows,
            previous_event=ev),
        "expert_swiglu_backward": lambda ev: buf.expert_swiglu_backward(
            make((M, N), bf16), make((M, 2 * N), bf16), rows, previous_event=ev),
    }


NAMES = ["get_dispatch_layout", "prepare", "prepare from a layout", "dispatch", "dispatch, weights",
         "dispatch of codes", "cached dispatch", "combine", "combine, weights",
         "low_latency_dispatch", "low_latency_combine", "low_latency_combine, hook", "gate_topk",
         "gate_topk, bias", "gate_topk_backward", "expert_order", "expert_sort", "expert_unsort",
         "expert_sort_backward", "expert_unsort_backward", "expert_linear",
         "expert_linear, offsets", "expert_linear, counts", "expert_linear_backward",
         "expert_swiglu_backward"]


def test_every_method_is_here(bench):
    buf, _ = bench
    cls = type(buf)
    methods = {n for n in dir(cls) if not n.startswith("_") and callable(getattr(cls, n))
               and "previous_event" in inspect.signature(getattr(cls, n)).parameters}
    here = calls(buf, dense)
    assert set(here) == set(NAMES)
    assert methods == {n.split(",")[0].split(" ")[0] for n in here} - {"cached"}


@pytest.mark.parametrize("name", NAMES)
def test_copies_wait_for_the_event(bench, name):
    from combine_get_dispatch_layout_amd import EventOverlap
    buf, log = bench
    event = EventOverlap()
    event.event = EVENT
    call = calls(buf, strided)[name]
    try:
        call(event)
    finally:
        event.event = None
    # each copy runs on the current stream, behind a wait of that stream
    assert "copy" in log and log[0] == (EVENT, STREAM), log
    del log[:]
    call(None)
    call(EventOverlap())  # an event that is already complete
    assert set(log) == {"copy"}
    del log[:]
    event.event = EVENT
    try:
        calls(buf, dense)[name](event)
    finally:
        event.event = None
    assert log == []  # nothing is copied, and only the call's own stream waits
