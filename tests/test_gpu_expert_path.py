"""The whole layer in a row: router, dispatch, expert order, the experts' two
products, the way back and the combine; its gradients; the decode form in the
low-latency slots; captured and replayed; and on the comm stream.

Each stage is within its own rounding of the definition (the other files of
these operators check that), so the chain is compared with the layer in fp64:
h, y, a bucket's sum and the output are each rounded once to bf16 (2^-8
relative), so an output is within 5 * 2^-8 of the sum of its terms' sizes."""

import pytest
import torch

from tests.gpu_common import device, make_buffer

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -8
T, H, F, E, R, K = 203, 256, 136, 16, 4, 4


def weights(dev, seed=0):
    g = torch.Generator(dev).manual_seed(seed)
    w1 = (torch.randn(E, 2 * F, H, generator=g, device=dev) * H ** -0.5).to(torch.bfloat16)
    w2 = (torch.randn(E, H, F, generator=g, device=dev) * F ** -0.5).to(torch.bfloat16)
    return w1, w2


def inputs(dev, seed, n=T):
    g = torch.Generator(dev).manual_seed(seed)
    x = torch.randn(n, H, generator=g, device=dev).to(torch.bfloat16)
    logits = torch.randn(n, E, generator=g, device=dev)
    return x, logits


def layer(x, idx, gates, w1, w2):
    """(output, sum of its terms' sizes) in fp64."""
    out = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    size = torch.zeros_like(out)
    for e in range(E):
        t, k = torch.nonzero(idx == e, as_tuple=True)
        if t.numel() == 0:
            continue
        p = x[t].double() @ w1[e].double().t().contiguous()
        h = p[:, :F] * torch.sigmoid(p[:, :F]) * p[:, F:]
        w = w2[e].double().t().contiguous()
        a = gates[t, k].double()[:, None]
        out.index_add_(0, t, a * (h @ w))
        size.index_add_(0, t, a.abs() * (h.abs() @ w.abs()))
    return out, size


def close(got, want, size, n=5):
    bad = (got.double() - want).abs() > n * EPS * size + 1e-6
    assert not bad.any(), int(bad.sum())


def on_tokens(buf, x, logits, w1, w2, **kw):
    idx, gates, _ = buf.gate_topk(logits, K, renormalize=True, **kw)
    order, _ = buf.expert_order(idx, **kw)
    rows, _ = buf.expert_sort(x, order, **kw)
    h, pre, _ = buf.expert_linear(rows, w1, order, swiglu=True, return_pre=True, **kw)
    y, _, _ = buf.expert_linear(h, w2, order, **kw)
    out, _ = buf.expert_unsort(y, order, gates, **kw)
    return idx, gates, order, rows, h, pre, y, out


def backward(buf, d_out, logits, w1, w2, saved, **kw):
    idx, gates, order, rows, h, pre, y, _ = saved
    d_y, d_gates, _ = buf.expert_unsort_backward(d_out, y, order, gates, **kw)
    d_h, d_w2, _ = buf.expert_linear_backward(d_y, h, w2, order, **kw)
    d_pre, _ = buf.expert_swiglu_backward(d_h, pre, order, **kw)
    d_rows, d_w1, _ = buf.expert_linear_backward(d_pre, rows, w1, order, **kw)
    d_x, _ = buf.expert_sort_backward(d_rows, order, **kw)
    d_logits, _ = buf.gate_topk_backward(d_gates, logits, idx, renormalize=True, **kw)
    return d_x, d_logits, d_w1, d_w2


@pytest.mark.parametrize("capacity", [False, True], ids=["exact", "capacity"])
def test_layer_through_dispatch(capacity):
    dev = device()
    w1, w2 = weights(dev)
    x, logits = inputs(dev, 1)
    buf = make_buffer(E, R, 4, T)
    idx, gates, _ = buf.gate_topk(logits, K, num_groups=4, groups_kept=2, renormalize=True)
    ntr, _, nte, itr, _ = buf.get_dispatch_layout(idx, E)
    recv, rti, rtw, _, handle, _ = buf.dispatch(
        x, topk_idx=idx, topk_weights=gates, num_tokens_per_rank=ntr, is_token_in_rank=itr,
        num_tokens_per_expert=nte, num_worst_tokens=T * R if capacity else 0)
    order, _ = buf.expert_order(rti, handle=handle)
    rows, _ = buf.expert_sort(recv, order)
    h, _, _ = buf.expert_linear(rows, w1, order, swiglu=True)
    y, _, _ = buf.expert_linear(h, w2, order)
    back, _ = buf.expert_unsort(y, order, rtw)
    out, _, _ = buf.combine(back, handle)
    close(out, *layer(x, idx, gates, w1, w2))


def test_layer_and_gradients():
    """On the tokens themselves, and every gradient against autograd through
    the fp64 layer for the same choice.  A gradient passes up to 8 roundings
    (d_y, d_h, d_pre, d_rows, its sum; h, y, pre), each at most 2^-8 of its
    terms: compared in norm, where they average, at 8 * 2^-8."""
    dev = device()
    w1, w2 = weights(dev)
    x, logits = inputs(dev, 2)
    buf = make_buffer(E, 1, 1, T)
    saved = on_tokens(buf, x, logits, w1, w2)
    idx, gates = saved[0], saved[1]
    close(saved[-1], *layer(x, idx, gates, w1, w2))
    g = torch.Generator(dev).manual_seed(9)
    d_out = torch.randn(T, H, generator=g, device=dev).to(torch.bfloat16)
    got = backward(buf, d_out, logits, w1, w2, saved)
    leaves = [v.cpu().double().requires_grad_() for v in (x, logits, w1, w2)]
    xd, ld, w1d, w2d = leaves
    ic = idx.cpu()
    gt = torch.softmax(torch.gather(ld, 1, ic), 1)
    out = torch.zeros(T, H, dtype=torch.float64)
    for e in range(E):
        t, k = torch.nonzero(ic == e, as_tuple=True)
        p = xd[t] @ w1d[e].t()
        hh = p[:, :F] * torch.sigmoid(p[:, :F]) * p[:, F:]
        out = out.index_add(0, t, gt[t, k][:, None] * (hh @ w2d[e].t()))
    want = torch.autograd.grad((out * d_out.cpu().double()).sum(), leaves)
    for name, a, b in zip(("d_x", "d_logits", "d_w1", "d_w2"), got, want):
        rel = float((a.cpu().double() - b).norm() / b.norm())
        assert rel < 8 * EPS, (name, rel)


@pytest.mark.parametrize("n", [1, 5, 64])
def test_decode_layer_in_slots(n):
    dev = device()
    w1, w2 = weights(dev)
    x, logits = inputs(dev, 3, n)
    buf = make_buffer(E, R, 1, 64)
    idx, gates, _ = buf.gate_topk(logits, K, score="sigmoid", renormalize=True)
    recv, cnt, handle, _, _ = buf.low_latency_dispatch(x, idx, 64, E)
    h, _, _ = buf.expert_linear(recv, w1, cnt, swiglu=True)
    y, _, _ = buf.expert_linear(h, w2, cnt)
    out, _, _ = buf.low_latency_combine(y, idx, gates, handle)
    close(out, *layer(x, idx, gates, w1, w2))


def test_training_step_hip_graph_replays():
    """The layer and its gradients captured once; each replay sees new tokens
    and logits, with eager work of another Buffer between, and equals the
    eager calls on the same inputs bit for bit."""
    dev = device()
    w1, w2 = weights(dev)
    buf, other = make_buffer(E, 1, 1, T), make_buffer(E, 1, 1, T)
    x, logits = inputs(dev, 4)
    d_out = torch.randn(T, H, device=dev).to(torch.bfloat16)
    kw = dict(no_sync=True)

    def step(b, x, logits):
        saved = on_tokens(b, x, logits, w1, w2, **kw)
        return saved[-1], backward(b, d_out, logits, w1, w2, saved, **kw), saved[2]

    step(buf, x, logits)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            out, grads, order = step(buf, x, logits)
    torch.cuda.current_stream().wait_stream(s)
    for rep in range(4):
        nx, nl = inputs(dev, 50 + rep)
        if rep == 2:
            nl[:, 3:] = float("-inf")  # three experts take every token, one slot stays empty
        x.copy_(nx)
        logits.copy_(nl)
        print(f"[graph] training step replay {rep}", flush=True)
        graph.replay()
        w_out, w_grads, w_order = step(other, nx, nl)
        torch.cuda.synchronize()
        n = int(w_order.expert_offsets[-1])
        assert torch.equal(order.slot_of_row, w_order.slot_of_row)
        assert n == (T * 3 if rep == 2 else T * K)
        assert torch.equal(out, w_out)
        for a, b in zip(grads, w_grads):
            assert torch.equal(a, b)


def test_comm_stream_and_events():
    """On the ctx stream, ordered by events, with temporaries dropped at once."""
    dev = device()
    w1, w2 = weights(dev)
    x, logits = inputs(dev, 5)
    buf = make_buffer(E, 1, 1, T)
    want = on_tokens(buf, x, logits, w1, w2)[-1]
    idx, gates, ev = buf.gate_topk(logits.clone(), K, renormalize=True, async_finish=True,
                                   allocate_on_comm_stream=True)
    order, ev = buf.expert_order(idx, previous_event=ev, async_finish=True,
                                 allocate_on_comm_stream=True)
    rows, ev = buf.expert_sort(x.clone(), order, previous_event=ev, async_finish=True,
                               allocate_on_comm_stream=True)
    h, _, ev = buf.expert_linear(rows, w1, order, swiglu=True, previous_event=ev,
                                 async_finish=True, allocate_on_comm_stream=True)
    del rows
    y, _, ev = buf.expert_linear(h, w2, order, previous_event=ev, async_finish=True,
                                 allocate_on_comm_stream=True)
    out, ev = buf.expert_unsort(y, order, gates, previous_event=ev, async_finish=True,
                                allocate_on_comm_stream=True)
    ev.current_stream_wait()
    assert torch.equal(out, want)


def test_two_streams_at_once():
    """Two orders and layers of one Buffer on two streams share nothing."""
    dev = device()
    w1, w2 = weights(dev)
    buf = make_buffer(E, 1, 1, T)
    ins = [inputs(dev, 60 + i) for i in range(2)]
    want = [on_tokens(buf, x, l, w1, w2)[-1] for x, l in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(3):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(on_tokens(buf, *ins[i], w1, w2, no_sync=True)[-1])
    torch.cuda.synchronize()
    for i in range(2):
        for out in got[i]:
            assert torch.equal(out, want[i])


def test_threads_share_a_buffer():
    """Host threads ordering batches of different sizes on one Buffer, each on a
    stream of its own."""
    import threading
    dev = device()
    w1, w2 = weights(dev)
    buf = make_buffer(E, 1, 1, 4096)
    sizes = [64, 203, 1500, 3000]
    ins = [inputs(dev, 70 + i, n) for i, n in enumerate(sizes)]
    want = [on_tokens(buf, x, l, w1, w2)[-1] for x, l in ins]
    torch.cuda.synchronize()
    got, errors = [None] * len(ins), []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(5):
                    got[i] = on_tokens(buf, *ins[i], w1, w2, no_sync=True)[-1]
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(ins))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_readme_example():
    """The README's example as written: the layer through the dispatch and in the
    decode slots gives the layer on the tokens, each rounded a few times."""
    import os
    import re
    dev = device()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "README.md")).read()
    m = re.search(r"## From the router to the output.*?```python\n(.*?)```", text, re.S)
    print("[path] README example", flush=True)
    torch.manual_seed(0)
    ns = {}
    exec(compile(m.group(1), "README.md", "exec"), ns)
    torch.cuda.synchronize()
    out = ns["out"].double()
    scale = float(out.norm())
    assert float((ns["out2"].double() - out).norm()) < 8 * EPS * scale
    n = ns["out3"].shape[0]
    assert float((ns["out3"].double() - out[:n]).norm()) < 8 * EPS * float(out[:n].norm())
    assert ns["x"].device.type == dev.type
    for leaf, grad in (("x", "d_x"), ("w1", "d_w1"), ("w2", "d_w2"), ("logits", "d_logits")):
        assert ns[grad].shape == ns[leaf].shape and bool(torch.isfinite(ns[grad]).all())
