"""The int8 calls in a row, as they are used: a layer served in int8 (over expert
order and in the low-latency slots), a training step whose rows are saved in
int8; captured and replayed, on the comm stream, on two streams and from host
threads.

A value held in int8 is off by at most half its scale (and 4 fp32 roundings of
127 steps: 0.5 + 127 * 4 * 2^-24 < 0.5001 scales).  The bounds below carry that
through the products' sums of sizes, as fp64 computes them."""

import threading

import pytest
import torch

from tests.gpu_common import device, make_buffer
from tests.test_gpu_expert_int8 import product, quantized, values
from tests.test_gpu_expert_linear import V, check, swiglu_reference
from tests.test_gpu_strided_events import late, outputs, side  # noqa: F401

pytestmark = pytest.mark.gpu

T, H, F, E, K = 203, 256, 144, 16, 4
HALF = 0.5001
EPS = 2.0 ** -8


def weights(dev, seed=0):
    g = torch.Generator(dev).manual_seed(seed)
    w1 = (torch.randn(E, 2 * F, H, generator=g, device=dev) * H ** -0.5).to(torch.bfloat16)
    w2 = (torch.randn(E, H, F, generator=g, device=dev) * F ** -0.5).to(torch.bfloat16)
    return w1, w2


def inputs(dev, seed, n=T):
    g = torch.Generator(dev).manual_seed(seed)
    x = torch.randn(n, H, generator=g, device=dev).to(torch.bfloat16)
    return x, torch.randn(n, E, generator=g, device=dev)


def in_int8(buf, *ws):
    out = []
    for w in ws:
        out += buf.expert_quantize(w)[:2]
    return out


def serve(buf, x, logits, q, **kw):
    w1, s1, w2, s2 = q
    idx, gates, _ = buf.gate_topk(logits, K, renormalize=True, **kw)
    order, _ = buf.expert_order(idx, **kw)
    rows, xs, _ = buf.expert_sort_int8(x, order, **kw)
    h, _ = buf.expert_linear_int8(rows, xs, w1, s1, order, swiglu=True, **kw)
    hq, hs, _ = buf.expert_quantize(h, order, **kw)
    y, _ = buf.expert_linear_int8(hq, hs, w2, s2, order, **kw)
    out, _ = buf.expert_unsort(y, order, gates, **kw)
    return idx, gates, order, rows, xs, h, hq, hs, y, out


def test_served_layer():
    dev = device()
    w1, w2 = weights(dev)
    x, logits = inputs(dev, 1)
    buf = make_buffer(E, 1, 1, T)
    q = in_int8(buf, w1, w2)
    idx, gates, order, rows, xs, h, hq, hs, y, out = serve(buf, x, logits, q)
    off, token = order.expert_offsets.tolist(), order.slot_of_row.long() // K
    want = torch.zeros(T * K, H, dtype=torch.float64, device=dev)
    bound = torch.zeros_like(want)
    for e in range(E):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        # each stage is its definition, from the stage before
        t = token[a:b]
        c, s = quantized(x[t], 0)
        assert torch.equal(rows[a:b].cpu(), c) and torch.equal(xs[a:b].cpu(), s)
        p = product(rows[a:b], xs[a:b], q[0][e], q[1][e])
        g, u = p[:, :F].double(), p[:, F:].double()
        act = g * torch.sigmoid(g) * u
        check("h", h[a:b], act, 8 * V * act.abs(), torch.bfloat16)
        c, s = quantized(h[a:b], 0)
        assert torch.equal(hq[a:b].cpu(), c) and torch.equal(hs[a:b].cpu(), s)
        assert torch.equal(y[a:b], product(hq[a:b], hs[a:b], q[2][e], q[3][e]).to(y.dtype))
        # the layer itself in fp64, and what its int8 values may be off
        xd, v1, v2 = x[t].double(), w1[e].double(), w2[e].double()
        dx, d1 = HALF * xs[a:b, None].double(), HALF * q[1][e].double()
        t1, t2 = v1.t().contiguous(), v2.t().contiguous()
        pre = xd @ t1
        d_pre = dx * t1.abs().sum(0) + xd.abs().sum(1, keepdim=True) * d1 + H * dx * d1
        act, d_act = swiglu_reference(pre[:, :F], pre[:, F:], d_pre[:, :F], d_pre[:, F:])
        d_act = d_act + EPS * (act.abs() + d_act) + HALF * hs[a:b, None].double()
        d2 = HALF * q[3][e].double()
        want[a:b] = act @ t2
        bound[a:b] = d_act @ t2.abs() + (act.abs() + d_act).sum(1, keepdim=True) * d2
        bound[a:b] += EPS * (want[a:b].abs() + bound[a:b])
    row = order.row_of_slot.long()
    layer = (want[row] * gates[..., None].double()).sum(1)
    size = (bound[row] * gates[..., None].double().abs()).sum(1) + EPS * layer.abs() + 1e-6
    assert ((out.double() - layer).abs() <= size * (1 + EPS)).all()


@pytest.mark.parametrize("n", [1, 37, T])
def test_decode_slots_equal_expert_order(n):
    """A row's results do not depend on where it lies: the low-latency slots give
    the same bits as rows in expert order."""
    dev = device()
    x, logits = inputs(dev, 2, n)
    buf = make_buffer(E, 1, 1, T)
    q = in_int8(buf, *weights(dev))
    idx, gates, order, *_, y, out = serve(buf, x, logits, q)
    slots, counts, handle, _, _ = buf.low_latency_dispatch(x, idx, T, E)
    c, s, _ = buf.expert_quantize(slots, counts)
    h, _ = buf.expert_linear_int8(c, s, q[0], q[1], counts, swiglu=True)
    c, s, _ = buf.expert_quantize(h, counts)
    z, _ = buf.expert_linear_int8(c, s, q[2], q[3], counts)
    off = order.expert_offsets.tolist()
    for e in range(E):
        assert torch.equal(z[e, :off[e + 1] - off[e]], y[off[e]:off[e + 1]])
    got, _, _ = buf.low_latency_combine(z, idx, gates, handle)
    # the sums are fused multiply-adds in the same order
    assert torch.equal(got, out)


def test_through_dispatch():
    """The received rows of a dispatch, quantised as they are sorted."""
    dev = device()
    R = 4
    x, logits = inputs(dev, 3)
    buf = make_buffer(E, R, 2, T)
    q = in_int8(buf, *weights(dev))
    idx, gates, *_, out = serve(buf, x, logits, q)
    recv, ri, rw, _, handle, _ = buf.dispatch(x, topk_idx=idx, topk_weights=gates)
    order, _ = buf.expert_order(ri, handle=handle)
    c, s, _ = buf.expert_sort_int8(recv, order)
    h, _ = buf.expert_linear_int8(c, s, q[0], q[1], order, swiglu=True)
    c, s, _ = buf.expert_quantize(h, order)
    y, _ = buf.expert_linear_int8(c, s, q[2], q[3], order)
    got, _, _ = buf.combine(buf.expert_unsort(y, order, rw)[0], handle)
    # the same expert rows, summed by bucket with one rounding more each
    row_sum, _ = buf.expert_unsort(y.abs(), order, rw.abs())
    size, _, _ = buf.combine(row_sum, handle)
    assert ((got.double() - out.double()).abs() <= 3 * EPS * size.double() + 1e-6).all()


def forward(buf, x, logits, w1, w2, block, **kw):
    """The layer's output and what the backward pass needs: rows, (gate, up) and
    outputs of the experts in int8."""
    idx, gates, _ = buf.gate_topk(logits, K, renormalize=True, **kw)
    order, _ = buf.expert_order(idx, **kw)
    rows, _ = buf.expert_sort(x, order, **kw)
    h, pre, _ = buf.expert_linear(rows, w1, order, swiglu=True, return_pre=True, **kw)
    y, _, _ = buf.expert_linear(h, w2, order, **kw)
    out, _ = buf.expert_unsort(y, order, gates, **kw)
    saved = [buf.expert_quantize(v, order, block=block, **kw)[:2] for v in (rows, pre, y)]
    return out, (idx, gates, order, saved), (rows, pre, h, y)


def backward(buf, d_out, logits, w1, w2, kept, **kw):
    idx, gates, order, ((rq, rs), (pq, ps), (yq, ys)) = kept
    y, _ = buf.expert_dequantize(yq, ys, order, **kw)
    d_y, d_gates, _ = buf.expert_unsort_backward(d_out, y, order, gates, **kw)
    d_h, _, _ = buf.expert_linear_backward(d_y, None, w2, order, **kw)
    d_pre, h, _ = buf.expert_swiglu_backward_int8(d_h, pq, ps, order, return_h=True, **kw)
    _, d_w2, _ = buf.expert_linear_backward(d_y, h, None, order, **kw)
    d_rows, d_w1, _ = buf.expert_linear_backward_int8(d_pre, rq, rs, w1, order, **kw)
    d_x, _ = buf.expert_sort_backward(d_rows, order, **kw)
    d_logits, _ = buf.gate_topk_backward(d_gates, logits, idx, renormalize=True, **kw)
    return (d_x, d_logits, d_w1, d_w2), (y, d_y, d_h, d_pre, h)


@pytest.mark.parametrize("block", [0, 128])
def test_training_step_from_saved_rows(block):
    dev = device()
    w1, w2 = weights(dev)
    x, logits = inputs(dev, 4)
    d_out = torch.randn(T, H, device=dev).to(torch.bfloat16)
    buf = make_buffer(E, 1, 1, T)
    _, kept, (rows, pre, h16, y16) = forward(buf, x, logits, w1, w2, block)
    grads, (y, d_y, d_h, d_pre, h) = backward(buf, d_out, logits, w1, w2, kept)
    order = kept[2]
    off = order.expert_offsets.tolist()
    n = off[-1]
    (rq, rs), (pq, ps), (yq, ys) = kept[3]
    # what is saved is near what it stands for
    for v, c, s in ((rows, rq, rs), (pre, pq, ps), (y16, yq, ys)):
        each = values(torch.ones_like(c), s)[:n].double()
        assert ((values(c, s)[:n].double() - v[:n].double()).abs() <= HALF * each).all()
    # both halves of a gradient asked for alone are those of the whole call
    full_h, full_w2, _ = buf.expert_linear_backward(d_y, h, w2, order)
    assert torch.equal(full_h[:n], d_h[:n]) and torch.equal(full_w2, grads[3])
    # the saved rows' gradients, and how far from those of the rows themselves
    d_rows16, d_w1_16, _ = buf.expert_linear_backward(d_pre, rows, w1, order, d_w_dtype=torch.float32)
    for e in range(E):
        a, b = off[e], off[e + 1]
        d = d_pre[a:b].double().t().contiguous()
        xs = values(rq, rs)[a:b].to(torch.bfloat16).double()
        check("d_w1", grads[2][e], d @ xs, (b - a + 1) * V * (d.abs() @ xs.abs()), torch.bfloat16)
        each = HALF * values(torch.ones_like(rq), rs)[a:b].double()
        each = each + EPS * (xs.abs() + each)
        off_by = (grads[2][e].double() - d_w1_16[e].double()).abs()
        assert (off_by <= d.abs() @ each + EPS * d_w1_16[e].double().abs() + 1e-6
                + 2 * (b - a + 1) * V * (d.abs() @ xs.abs())).all()
    assert torch.equal(grads[0], buf.expert_sort_backward(d_rows16, order)[0])
    assert torch.isfinite(grads[1]).all()


def same(a, b, n):
    assert torch.equal(a[:n], b[:n])


def test_hip_graph_replays():
    """The served layer and the training step, captured once; each replay sees new
    tokens and logits, with eager work of another Buffer between."""
    dev = device()
    w1, w2 = weights(dev)
    buf, other = make_buffer(E, 1, 1, T), make_buffer(E, 1, 1, T)
    q = in_int8(buf, w1, w2)
    x, logits = inputs(dev, 5)
    d_out = torch.randn(T, H, device=dev).to(torch.bfloat16)
    kw = dict(no_sync=True)

    def step(b, x, logits):
        served = serve(b, x, logits, q, **kw)[-1]
        out, kept, _ = forward(b, x, logits, w1, w2, 128, **kw)
        return served, out, backward(b, d_out, logits, w1, w2, kept, **kw)[0]

    step(buf, x, logits)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            served, out, grads = step(buf, x, logits)
    torch.cuda.current_stream().wait_stream(s)
    for rep in range(4):
        nx, nl = inputs(dev, 50 + rep)
        if rep == 2:
            nl[:, 3:] = float("-inf")  # three experts take every token, one slot stays empty
        x.copy_(nx)
        logits.copy_(nl)
        print(f"[graph] int8 replay {rep}", flush=True)
        graph.replay()
        w_served, w_out, w_grads = step(other, nx, nl)
        torch.cuda.synchronize()
        assert torch.equal(served, w_served) and torch.equal(out, w_out)
        for a, b in zip(grads, w_grads):
            assert torch.equal(a, b)


def test_comm_stream_and_events():
    """On the ctx stream, ordered by events, with temporaries dropped at once."""
    dev = device()
    w1, w2 = weights(dev)
    x, logits = inputs(dev, 6)
    buf = make_buffer(E, 1, 1, T)
    q = in_int8(buf, w1, w2)
    _, gates, order, *_, want = serve(buf, x, logits, q)
    kw = dict(async_finish=True, allocate_on_comm_stream=True)
    c, s, ev = buf.expert_sort_int8(x.clone(), order, **kw)
    h, ev = buf.expert_linear_int8(c, s, q[0], q[1], order, swiglu=True, previous_event=ev, **kw)
    del c, s
    c, s, ev = buf.expert_quantize(h, order, previous_event=ev, **kw)
    del h
    y, ev = buf.expert_linear_int8(c, s, q[2], q[3], order, previous_event=ev, **kw)
    del c, s
    out, ev = buf.expert_unsort(y, order, gates, previous_event=ev, **kw)
    ev.current_stream_wait()
    assert torch.equal(out, want)

    d_y = torch.randn(T * K, H, device=dev).to(torch.bfloat16)
    _, kept, _ = forward(buf, x, logits, w1, w2, 128)
    order, ((rq, rs), (pq, ps), (yq, ys)) = kept[2], kept[3]
    n = int(order.expert_offsets[-1])
    d_h, _, _ = buf.expert_linear_backward(d_y, None, w2, order)
    want_y, _ = buf.expert_dequantize(yq, ys, order)
    want_p, want_h, _ = buf.expert_swiglu_backward_int8(d_h, pq, ps, order, return_h=True)
    want_x, want_w, _ = buf.expert_linear_backward_int8(want_p, rq, rs, w1, order)
    got_y, ev = buf.expert_dequantize(yq, ys, order, **kw)
    p, got_h, ev = buf.expert_swiglu_backward_int8(d_h.clone(), pq.clone(), ps.clone(), order,
                                                   return_h=True, previous_event=ev, **kw)
    got_x, got_w, ev = buf.expert_linear_backward_int8(p, rq.clone(), rs.clone(), w1, order,
                                                       previous_event=ev, **kw)
    ev.current_stream_wait()
    same(got_y, want_y, n)
    same(p, want_p, n)
    same(got_h, want_h, n)
    same(got_x, want_x, n)
    assert torch.equal(got_w, want_w)


@pytest.mark.parametrize("comm", [False, True], ids=["caller", "comm"])
def test_late_strided_inputs(side, comm):  # noqa: F811
    """Strided inputs that are written behind previous_event are copied behind it."""
    from combine_get_dispatch_layout_amd import ExpertOrder
    dev = device()
    w1, w2 = weights(dev)
    x, logits = inputs(dev, 12)
    buf = make_buffer(E, 1, 1, T)
    q1, s1, q2, s2 = in_int8(buf, w1, w2)
    order, _ = buf.expert_order(buf.gate_topk(logits, K)[0])
    off = order.expert_offsets
    assert int(off[-1]) == T * K  # every row of every buffer is somebody's
    rq, rs, _ = buf.expert_sort_int8(x, order)
    r16, _ = buf.expert_dequantize(rq, rs, order)
    bq, bs, _ = buf.expert_quantize(r16, order, block=128)
    h, pre, _ = buf.expert_linear(r16, w1, order, swiglu=True, return_pre=True)
    pq, ps, _ = buf.expert_quantize(pre, order, block=128)
    kw = dict(allocate_on_comm_stream=comm)
    cases = {
        "expert_quantize": ((r16, off), buf.expert_quantize),
        "expert_dequantize": ((bq, bs, off), buf.expert_dequantize),
        "expert_sort_int8": ((x, order.row_of_slot), lambda v, r, **k: buf.expert_sort_int8(
            v, ExpertOrder(None, r, None), **k)),
        "expert_linear_int8": ((rq, rs, q1, s1, off), lambda *a, **k: buf.expert_linear_int8(
            *a, swiglu=True, **k)),
        "expert_swiglu_backward_int8": ((h, pq, ps, off),
                                        lambda *a, **k: buf.expert_swiglu_backward_int8(
                                            *a, return_h=True, **k)),
        "expert_linear_backward_int8": ((pre, bq, bs, w1, off), buf.expert_linear_backward_int8),
        "d_x alone": ((pre, w1, off), lambda d, w, o, **k: buf.expert_linear_backward(
            d, None, w, o, **k)),
        "d_w alone": ((pre, r16, off), lambda d, v, o, **k: buf.expert_linear_backward(
            d, v, None, o, **k)),
    }
    for name, (tensors, call) in cases.items():
        print(f"[int8] late strided inputs: {name} comm={comm}", flush=True)
        want = outputs(call(*tensors, **kw))
        strided, ready = late(side, *tensors)
        got = outputs(call(*strided, previous_event=ready, **kw))
        torch.cuda.synchronize()
        assert len(got) == len(want) > 0
        for a, b in zip(got, want):
            assert torch.equal(a, b), name


def test_two_streams_and_threads():
    """Layers of one Buffer on streams and host threads of their own share nothing."""
    dev = device()
    w1, w2 = weights(dev)
    buf = make_buffer(E, 1, 1, 2048)
    q = in_int8(buf, w1, w2)
    sizes = [1, 64, 203, 1500]
    ins = [inputs(dev, 70 + i, n) for i, n in enumerate(sizes)]
    d_outs = [torch.randn(n, H, device=dev).to(torch.bfloat16) for n in sizes]

    def run(i, **kw):
        out, kept, _ = forward(buf, *ins[i], w1, w2, 128, **kw)
        grads, _ = backward(buf, d_outs[i], ins[i][1], w1, w2, kept, **kw)
        return (serve(buf, *ins[i], q, **kw)[-1], out) + grads

    want = [run(i) for i in range(len(sizes))]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sizes]
    got = [None] * len(sizes)
    for _ in range(2):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = run(i, no_sync=True)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(u, v) for u, v in zip(a, b))
    got, errors = [None] * len(sizes), []

    def work(i):
        try:
            with torch.cuda.stream(streams[i]):
                for _ in range(3):
                    got[i] = run(i, no_sync=True)
            streams[i].synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(sizes))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for a, b in zip(got, want):
        assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_buffers_past_4_gib():
    """Rows, codes, scales and weights whose offsets pass 32 bits."""
    dev = device()
    buf = make_buffer(2, 1, 1, 1)
    g = torch.Generator(dev).manual_seed(7)
    Kd, N, dt = 8192, 16, torch.bfloat16
    M = (1 << 32) // Kd + 1000  # codes past 4 GiB, rows past 8
    x = torch.zeros(M, Kd, device=dev, dtype=dt)
    x[-40:] = torch.randn(40, Kd, generator=g, device=dev).to(dt)
    rows = torch.tensor([0, 7, M], dtype=torch.int32, device=dev)
    for block in (128, 0):
        print(f"[int8] rows past 4 GiB, block={block}", flush=True)
        codes, scales, _ = buf.expert_quantize(x, rows, block=block)
        want_c, want_s = quantized(x[-40:], block)
        assert torch.equal(codes[-40:].cpu(), want_c) and torch.equal(scales[-40:].cpu(), want_s)
        assert not codes[:-40].any()
        back, _ = buf.expert_dequantize(codes, scales, rows)
        assert torch.equal(back[-40:].cpu(), values(want_c, want_s).to(dt))
        assert not back[:-40].any()
        del back
        d_y = torch.zeros(M, N, device=dev, dtype=dt)
        d_y[-40:] = torch.randn(40, N, generator=g, device=dev).to(dt)
        _, d_w, _ = buf.expert_linear_backward_int8(d_y, codes, scales, None, rows,
                                                    d_w_dtype=torch.float32)
        d, xs = d_y[-40:].double().t().contiguous(), values(codes[-40:], scales[-40:]).to(dt).double()
        check("d_w", d_w[1], d @ xs, 41 * V * (d.abs() @ xs.abs()), torch.float32)
        assert not d_w[0].any()
    del x
    w = torch.randint(-127, 128, (2, N, Kd), generator=g, device=dev, dtype=torch.int8)
    ws = torch.rand(2, N, generator=g, device=dev) * 1e-3
    y, _ = buf.expert_linear_int8(codes, scales, w, ws, rows)
    assert torch.equal(y[-40:], product(codes[-40:], scales[-40:], w[1], ws[1]).to(y.dtype))
    assert not y[:-40].any()
    del codes, y
    # (gate, up) codes past 4 GiB
    N2 = 8192
    M = (1 << 32) // (2 * N2) + 100
    pre = torch.zeros(M, 2 * N2, device=dev, dtype=torch.int8)
    pre[-5:] = torch.randint(-127, 128, (5, 2 * N2), generator=g, device=dev, dtype=torch.int8)
    ps = torch.full((M, 128), 0.02, device=dev)
    d_h = torch.ones(M, N2, device=dev, dtype=dt)
    rows = torch.tensor([0, 7, M], dtype=torch.int32, device=dev)
    d_pre, h, _ = buf.expert_swiglu_backward_int8(d_h, pre, ps, rows, return_h=True)
    p2, h2, _ = buf.expert_swiglu_backward_int8(
        d_h[-5:], pre[-5:].contiguous(), ps[-5:].contiguous(),
        torch.tensor([0, 1, 5], dtype=torch.int32, device=dev), return_h=True)
    assert torch.equal(d_pre[-5:], p2) and torch.equal(h[-5:], h2)
    assert not h[:-5].any()
    del pre, d_h, d_pre, h
    # weights past 4 GiB
    E2, N2 = 80, 8192
    buf = make_buffer(E2, 1, 1, 1)
    w = torch.zeros(E2, N2, Kd, device=dev, dtype=torch.int8)
    w[-1] = torch.randint(-127, 128, (N2, Kd), generator=g, device=dev, dtype=torch.int8)
    ws = torch.full((E2, N2), 1e-3, device=dev)
    c = torch.randint(-127, 128, (5, Kd), generator=g, device=dev, dtype=torch.int8)
    cs = torch.rand(5, device=dev)
    rows = torch.zeros(E2 + 1, dtype=torch.int32, device=dev)
    rows[-1] = 5
    y, _ = buf.expert_linear_int8(c, cs, w, ws, rows)
    assert torch.equal(y, product(c, cs, w[-1], ws[-1]).to(y.dtype))
    d_y = torch.randn(5, N2, generator=g, device=dev).to(dt)
    del w
    _, d_w, _ = buf.expert_linear_backward_int8(d_y, c, cs, None, rows)
    d, xs = d_y.double().t().contiguous(), values(c, cs).to(dt).double()
    check("d_w", d_w[-1], d @ xs, 6 * V * (d.abs() @ xs.abs()), dt)
    assert not d_w[:-1].any()


def test_readme_example():
    """The README's example as written runs, and its served, decoded and trained
    parts are what the same calls give here."""
    import os
    import re
    device()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "README.md")).read()
    m = re.search(r"## The experts in 8 bits.*?```python\n(.*?)```", text, re.S)
    print("[int8] README example", flush=True)
    torch.manual_seed(0)
    ns = {}
    exec(compile(m.group(1), "README.md", "exec"), ns)
    torch.cuda.synchronize()
    buf, idx, gates, order = ns["buf"], ns["idx"], ns["gates"], ns["order"]
    q = [ns[k] for k in ("q1", "s1", "q2", "s2")]
    hq, hs, _ = buf.expert_quantize(
        buf.expert_linear_int8(ns["rows"], ns["scales"], q[0], q[1], order, swiglu=True)[0], order)
    y, _ = buf.expert_linear_int8(hq, hs, q[2], q[3], order)
    assert torch.equal(ns["served"], buf.expert_unsort(y, order, gates)[0])
    # rows do not depend on their place: the slots give the same sums
    assert torch.equal(ns["decoded"], ns["served"][:128])
    for leaf, grad in (("x", "d_x"), ("w1", "d_w1"), ("w2", "d_w2"), ("logits", "d_logits")):
        assert ns[grad].shape == ns[leaf].shape and bool(torch.isfinite(ns[grad]).all())


def test_many_tiles_captured_and_at_once():
    """Products whose workgroups go through several tiles: replayed with other rows in
    each expert, and by two streams at the same time."""
    dev = device()
    E_, Kd = 8, 272
    buf = make_buffer(E_, 1, 1, 1)
    g = torch.Generator(dev).manual_seed(31)
    counts = [[1024] * 8, [0, 3000, 1, 700, 65, 0, 4000, 300], [0] * 8, [8192] + [0] * 7]
    offsets = [torch.tensor([0] + c, device=dev).cumsum(0).int() for c in counts]
    for N in (2056, 392):  # 256 x 256 and 128 x 128 tiles
        x = torch.randint(-128, 128, (8192, Kd), generator=g, device=dev, dtype=torch.int8)
        xs = torch.rand(8192, generator=g, device=dev) * 0.01
        w = torch.randint(-128, 128, (E_, 2 * N, Kd), generator=g, device=dev, dtype=torch.int8)
        ws = torch.rand(E_, 2 * N, generator=g, device=dev) * 0.01
        out = lambda: torch.full((8192, N), 7.0, dtype=torch.bfloat16, device=dev)  # noqa: E731
        call = lambda o, y: buf.expert_linear_int8(x, xs, w, ws, o, swiglu=True, out=y,  # noqa: E731
                                                   no_sync=True)
        want = []
        for o in offsets:
            want.append(call(o, out())[0])
        o, y = offsets[0].clone(), out()
        graph = torch.cuda.CUDAGraph()
        call(o, y)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            call(o, y)
        for turn in range(2):
            for v, expected in zip(offsets, want):
                o.copy_(v)
                y.fill_(7.0)
                graph.replay()
                assert torch.equal(y, expected)
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        torch.cuda.synchronize()
        got = [[], []]
        ys = [[out() for _ in range(6)] for _ in streams]
        torch.cuda.synchronize()
        for i in range(6):
            for k, s in enumerate(streams):
                with torch.cuda.stream(s):
                    got[k].append(call(offsets[(i + k) % 4], ys[k][i])[0])
        torch.cuda.synchronize()
        for i in range(6):
            for k in range(2):
                assert torch.equal(got[k][i], want[(i + k) % 4])
