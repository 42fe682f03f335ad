"""Strided inputs that another stream is still writing, ordered by
previous_event alone: each call gives what it gives for finished, contiguous
ones, on the caller's stream and on the comm stream."""

import pytest
import torch

from tests.gpu_common import device, make_buffer

pytestmark = pytest.mark.gpu

T, H, F, E, R, K = 96, 128, 72, 16, 4, 3


@pytest.fixture(scope="module")
def side():
    dev = device()
    stream = torch.cuda.Stream()
    load = torch.randn(4096, 4096, device=dev)
    with torch.cuda.stream(stream):
        load @ load  # the library's set-up
    torch.cuda.synchronize()
    return stream, load


def late(side, *tensors):
    """(strided tensors of zeros that get these values on the side stream behind
    products of some milliseconds, the event that marks them ready)"""
    from combine_get_dispatch_layout_amd import Buffer
    stream, load = side
    out = [torch.zeros(*t.shape, 2, dtype=t.dtype, device=t.device)[..., 0] for t in tensors]
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        for _ in range(12):
            load @ load
        for o, t in zip(out, tensors):
            o.copy_(t)
        ready = Buffer.capture()
    return out, ready


def outputs(result):
    """The tensors of a call's result, ExpertOrder's among them."""
    from combine_get_dispatch_layout_amd import ExpertOrder
    flat = []
    for r in result:
        if isinstance(r, ExpertOrder):
            flat += [r.expert_offsets, r.row_of_slot, r.slot_of_row]
        elif isinstance(r, torch.Tensor):
            flat.append(r)
    return flat


@pytest.mark.parametrize("comm", [False, True], ids=["caller", "comm"])
def test_late_strided_inputs(side, comm):
    from combine_get_dispatch_layout_amd import ExpertOrder
    dev = device()
    buf = make_buffer(E, R, 2, T)
    bf16 = dict(device=dev, dtype=torch.bfloat16)
    x, logits = torch.randn(T, H, **bf16), torch.randn(T, E, device=dev)
    bias = torch.randn(E, device=dev)
    idx, gates, _ = buf.gate_topk(logits, K, bias=bias)
    order, _ = buf.expert_order(idx)
    w1, w2 = torch.randn(E, 2 * F, H, **bf16), torch.randn(E, H, F, **bf16)
    rows, _ = buf.expert_sort(x, order)
    h, pre, _ = buf.expert_linear(rows, w1, order, swiglu=True, return_pre=True)
    y, _, _ = buf.expert_linear(h, w2, order)
    off = order.expert_offsets
    kw = dict(allocate_on_comm_stream=comm)
    cases = {
        "gate_topk": ((logits, bias), lambda l, b, **k: buf.gate_topk(l, K, bias=b, **k)),
        "gate_topk_backward": ((gates, logits, idx), buf.gate_topk_backward),
        "expert_order": ((idx,), buf.expert_order),
        "expert_sort": ((x, order.row_of_slot), lambda v, r, **k: buf.expert_sort(
            v, ExpertOrder(None, r, None), **k)),
        "expert_unsort": ((y, gates), lambda v, g, **k: buf.expert_unsort(v, order, g, **k)),
        "expert_unsort_backward": ((x, y, gates, order.slot_of_row),
                                   lambda d, v, g, s, **k: buf.expert_unsort_backward(
                                       d, v, ExpertOrder(off, order.row_of_slot, s), g, **k)),
        "expert_linear": ((rows, w1, off), lambda v, w, o, **k: buf.expert_linear(
            v, w, o, swiglu=True, return_pre=True, **k)),
        "expert_linear_backward": ((y, h, w2), lambda d, v, w, **k: buf.expert_linear_backward(
            d, v, w, order, **k)),
        "expert_swiglu_backward": ((h, pre, off), buf.expert_swiglu_backward),
        "get_dispatch_layout": ((idx,), lambda i, **k: buf.get_dispatch_layout(i, E, **k)),
        "dispatch": ((x, idx, gates), lambda v, i, g, **k: buf.dispatch(
            v, topk_idx=i, topk_weights=g, num_worst_tokens=T * R, **k)),
    }
    n = int(off[-1])
    assert n == T * K  # every row of every buffer is somebody's
    for name, (tensors, call) in cases.items():
        print(f"[events] late strided inputs: {name} comm={comm}", flush=True)
        want = outputs(call(*tensors, **kw))
        strided, ready = late(side, *tensors)
        got = outputs(call(*strided, previous_event=ready, **kw))
        torch.cuda.synchronize()
        m = int(call(*tensors)[4].tensor(8, torch.int32)[0]) if name == "dispatch" else None
        for a, b in zip(got, want):
            assert torch.equal(a[:m], b[:m]), name
    handle = buf.dispatch(x, topk_idx=idx, topk_weights=gates)[4]
    recv = buf.dispatch(x, handle)[0]
    want = buf.combine(recv, handle, gate_weights=gates)[0]
    strided, ready = late(side, recv, gates)
    got = buf.combine(strided[0], handle, gate_weights=strided[1], previous_event=ready, **kw)[0]
    assert torch.equal(got, want)


def test_late_strided_slots(side):
    dev = device()
    buf = make_buffer(E, R, 2, T)
    x = torch.randn(T, H, device=dev, dtype=torch.bfloat16)
    idx, gates, _ = buf.gate_topk(torch.randn(T, E, device=dev), K)
    recv, cnt, handle, _, _ = buf.low_latency_dispatch(x, idx, T, E)
    want = buf.low_latency_combine(recv, idx, gates, handle)[0]
    (xs, ids), ready = late(side, x, idx)
    got = buf.low_latency_dispatch(xs, ids, T, E, ready)
    assert torch.equal(got[1], cnt)
    for e in range(E):
        assert torch.equal(got[0][e, :int(cnt[e])], recv[e, :int(cnt[e])])
    strided, ready = late(side, recv, idx, gates)
    out = buf.low_latency_combine(*strided, handle, ready)[0]
    assert torch.equal(out, want)
