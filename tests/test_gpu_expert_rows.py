"""Rows in expert order and back (expert_order, expert_sort, expert_unsort and
their gradients) against plain fp64 forms.  Indexes and copies are equal; a
sum of n fp32 products differs by at most (n + 1) 2^-24 of the sum of their
sizes, and by half a step of the output's type."""

import numpy as np
import pytest
import torch

from combine_get_dispatch_layout_amd import workloads as wl
from tests.gpu_common import device, make_buffer

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def routing(kind, T, E, K, seed):
    rng = np.random.default_rng(seed)
    if kind == "one":  # every pair goes to the last expert
        idx = np.full((T, K), -1, np.int64)
        if T:
            idx[:, K - 1] = E - 1
        return torch.from_numpy(idx)
    if kind == "none":
        return torch.full((T, K), -1, dtype=torch.int64)
    idx = torch.from_numpy(wl.random_routing(rng, T, E, K, p_empty=0.0 if kind == "full" else 0.3))
    if kind == "wild" and T:  # ids out of range count as empty
        idx[0, 0] = E
        idx[T - 1, 0] = -7
        idx[T // 2, K - 1] = 1 << 40
    return idx


def order_reference(idx, E):
    T, K = idx.shape
    flat = idx.reshape(-1).tolist()
    lists = [[] for _ in range(E)]
    for p, e in enumerate(flat):
        if 0 <= e < E:
            lists[e].append(p)
    offsets = [0]
    for ps in lists:
        offsets.append(offsets[-1] + len(ps))
    slot = [p for ps in lists for p in ps]
    row = [-1] * (T * K)
    for r, p in enumerate(slot):
        row[p] = r
    slot += [-1] * (T * K - len(slot))
    i32 = torch.int32
    return (torch.tensor(offsets, dtype=i32), torch.tensor(row, dtype=i32).view(T, K),
            torch.tensor(slot, dtype=i32))


ORDERS = [(0, 16, 2, "full"), (1, 1, 1, "full"), (1, 256, 8, "full"), (2, 1024, 16, "some"),
          (127, 16, 2, "some"), (128, 16, 2, "full"), (129, 60, 7, "wild"), (513, 256, 8, "some"),
          (700, 1024, 3, "wild"), (1000, 64, 6, "one"), (300, 64, 6, "none"), (4097, 256, 8, "some"),
          (2500, 65, 5, "wild")]


@pytest.mark.parametrize("case", ORDERS, ids=lambda c: "-".join(map(str, c)))
def test_expert_order(case):
    T, E, K, kind = case
    dev = device()
    idx = routing(kind, T, E, K, 7)
    buf = make_buffer(E, 1, 1, max(T, 1))
    print(f"[order] {case}", flush=True)
    order, _ = buf.expert_order(idx.to(dev))
    want = order_reference(idx, E)
    assert torch.equal(order.expert_offsets.cpu(), want[0])
    assert torch.equal(order.row_of_slot.cpu(), want[1])
    assert torch.equal(order.slot_of_row.cpu(), want[2])


@pytest.mark.parametrize("capacity", [False, True])
def test_expert_order_of_received_rows(capacity):
    """recv_topk_idx of a dispatch: local ids become global by the row's
    bucket, and a capacity-mode buffer's rows past N stay out."""
    dev = device()
    T, E, R, K, H = 333, 64, 8, 6, 64
    idx = routing("some", T, E, K, 3)
    w = torch.rand(T, K)
    x = torch.randn(T, H).to(torch.bfloat16)
    buf = make_buffer(E, R, 4, T)
    cap = T * min(K, R) if capacity else 0
    _, rti, rtw, _, h, _ = buf.dispatch(x.to(dev), topk_idx=idx.to(dev), topk_weights=w.to(dev),
                                        num_worst_tokens=cap)
    # the rows past N of a capacity buffer hold whatever was there
    n = int(h.fields()["num_recv"].cpu()[0])
    if capacity:
        assert n < rti.shape[0]
        rti[n:] = 3
    order, _ = buf.expert_order(rti, handle=h)
    P = E // R
    prefix = h.fields()["rank_prefix_matrix"].cpu().tolist()
    glob = rti.cpu().clone()
    for row in range(rti.shape[0]):
        bucket = sum(row >= p for p in prefix)
        glob[row] = -1 if row >= n else torch.where(glob[row] >= 0, glob[row] + bucket * P, -1)
    want = order_reference(glob, E)
    assert torch.equal(order.expert_offsets.cpu(), want[0])
    assert torch.equal(order.row_of_slot.cpu(), want[1])
    assert torch.equal(order.slot_of_row.cpu(), want[2])
    # every pair of the routing is there once
    counts = torch.bincount(idx[idx >= 0], minlength=E)
    assert torch.equal((order.expert_offsets[1:] - order.expert_offsets[:-1]).cpu().long(), counts)


MOVES = [(1, 16, 2, 8, "full"), (3, 16, 4, 520, "some"), (127, 64, 6, 1416, "some"),
         (65, 256, 8, 7168, "some"), (33, 8, 8, 24, "wild"), (20, 64, 16, 4104, "full"),
         (9, 64, 6, 256, "none"), (2, 4, 2, 20008, "full")]
TYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.mark.parametrize("dt", TYPES, ids=lambda d: str(d)[6:])
@pytest.mark.parametrize("case", MOVES, ids=lambda c: "-".join(map(str, c)))
def test_sort_unsort_and_gradients(case, dt):
    T, E, K, H, kind = case
    dev = device()
    g = torch.Generator().manual_seed(T * 31 + H)
    idx = routing(kind, T, E, K, 11)
    buf = make_buffer(E, 1, 1, T)
    offsets, row, slot = order_reference(idx, E)
    n = int(offsets[-1])
    order, _ = buf.expert_order(idx.to(dev))
    x = torch.randn(T, H, generator=g).to(dt)
    print(f"[moves] {case} {dt}", flush=True)
    rows, _ = buf.expert_sort(x.to(dev), order, out=torch.full((T * K, H), 7.0, dtype=dt, device=dev))
    rows = rows.cpu()
    assert torch.equal(rows[:n], x[slot[:n].long() // K])
    assert (rows[n:] == 7.0).all()  # rows behind the last pair are left alone

    y = torch.randn(T * K, H, generator=g).to(dt)
    y[n:] = float("nan")  # never read
    w = torch.randn(T, K, generator=g)
    half = torch.finfo(dt).eps / 2 if dt != torch.float32 else 0.0
    tiny = torch.finfo(dt).tiny
    for weights in (w, None):
        out, _ = buf.expert_unsort(y.to(dev), order, None if weights is None else weights.to(dev))
        ww = torch.ones(T, K) if weights is None else weights
        want, size = torch.zeros(T, H, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
        for k in range(K):
            t = torch.nonzero(row[:, k] >= 0)[:, 0]
            v = y[row[t, k].long()].double() * ww[t, k, None].double()
            want[t] += v
            size[t] += v.abs()
        err = (out.cpu().double() - want).abs()
        acc = (K + 1) * U * size
        assert (err <= acc + half * (want.abs() + acc) + tiny).all()
    back, _ = buf.expert_sort_backward(y.to(dev), order)
    assert torch.equal(back, out)

    d_out = torch.randn(T, H, generator=g).to(dt)
    y[n:] = 5.0
    d_rows, d_w, _ = buf.expert_unsort_backward(
        d_out.to(dev), y.to(dev), order, w.to(dev),
        out=torch.full((T * K, H), 7.0, dtype=dt, device=dev))
    d_rows, d_w = d_rows.cpu(), d_w.cpu()
    assert (d_rows[n:] == 7.0).all()
    t, k = slot[:n].long() // K, slot[:n].long() % K
    want = d_out[t].double() * w[t, k, None].double()
    assert ((d_rows[:n].double() - want).abs() <= (half + 2 * U) * want.abs() + tiny).all()
    prod = d_out[t].double() * y[:n].double()
    want_w, size_w = torch.zeros(T, K, dtype=torch.float64), torch.zeros(T, K, dtype=torch.float64)
    want_w[t, k], size_w[t, k] = prod.sum(1), prod.abs().sum(1)
    assert ((d_w.double() - want_w).abs() <= (H + 8) * U * size_w).all()
    assert (d_w[row < 0] == 0).all()


def test_long_order():
    """More pairs than one pass of tiles holds (2^20), counted in longer tiles."""
    dev = device()
    T, E, K = 150_000, 12, 8
    g = torch.Generator().manual_seed(1)
    idx = torch.randint(-1, E, (T, K), generator=g)
    buf = make_buffer(E, 1, 1, 1)
    order, _ = buf.expert_order(idx.to(dev))
    flat = idx.reshape(-1)
    key = torch.where(flat < 0, E, flat)
    slot = torch.sort(key, stable=True).indices
    n = int((flat >= 0).sum())
    got = order.slot_of_row.cpu()
    assert torch.equal(got[:n].long(), slot[:n]) and (got[n:] == -1).all()
    row = torch.full((T * K,), -1, dtype=torch.int64)
    row[slot[:n]] = torch.arange(n)
    assert torch.equal(order.row_of_slot.cpu().long().reshape(-1), row)
    counts = torch.bincount(key, minlength=E + 1)[:E]
    assert torch.equal(order.expert_offsets.cpu().long()[1:], torch.cumsum(counts, 0))


def test_rows_past_4_gib():
    """Row offsets pass 32 bits: 70,000 rows of 65,536 bytes."""
    dev = device()
    T, E, K, H = 35_000, 4, 2, 32_768
    idx = torch.stack([torch.arange(T) % E, (torch.arange(T) + 1) % E], 1).to(dev)
    buf = make_buffer(E, 1, 1, T)
    order, _ = buf.expert_order(idx)
    x = torch.randint(-100, 100, (T, H), device=dev, dtype=torch.int16).to(torch.bfloat16)
    rows, _ = buf.expert_sort(x, order)
    probe = torch.arange(0, T * K, 997, device=dev)
    assert torch.equal(rows[probe], x[(order.slot_of_row[probe] // K).long()])
    out, _ = buf.expert_unsort(rows, order)
    assert torch.equal(out, x * 2)


def test_strided_inputs():
    """Views with other strides give what their copies give."""
    dev = device()
    T, E, K, H = 37, 16, 3, 40
    buf = make_buffer(E, 1, 1, T)
    idx = routing("some", T, E, K, 5).to(dev)
    wide = torch.full((T, 2 * K), -7, dtype=torch.int64, device=dev)
    wide[:, ::2] = idx
    order, _ = buf.expert_order(idx)
    again, _ = buf.expert_order(wide[:, ::2])
    assert torch.equal(order.row_of_slot, again.row_of_slot)
    x = torch.randn(H, T, device=dev).to(torch.bfloat16).t()
    w = torch.rand(K, T, device=dev).t()
    rows, _ = buf.expert_sort(x, order)
    want, _ = buf.expert_sort(x.contiguous(), order)
    n = int(order.expert_offsets[-1])
    assert torch.equal(rows[:n], want[:n])
    out, _ = buf.expert_unsort(rows, order, w)
    want, _ = buf.expert_unsort(rows, order, w.contiguous())
    assert torch.equal(out, want)


def test_refusals():
    from combine_get_dispatch_layout_amd import ExpertOrder
    from combine_get_dispatch_layout_amd import _capi as C
    dev = device()
    buf = make_buffer(16, 4, 2, 8)
    idx = torch.zeros(4, 2, dtype=torch.int64, device=dev)
    idx[:, 1] = 5
    order, _ = buf.expert_order(idx)
    x = torch.zeros(4, 16, device=dev, dtype=torch.bfloat16)
    bad = [lambda: buf.expert_order(idx.int()), lambda: buf.expert_order(idx.cpu()),
           lambda: buf.expert_order(idx[0]),
           lambda: buf.expert_sort(x[:3], order), lambda: buf.expert_sort(x.double(), order),
           lambda: buf.expert_sort(x.cpu(), order),
           lambda: buf.expert_sort(x, order, out=torch.zeros(7, 16, device=dev, dtype=x.dtype)),
           lambda: buf.expert_sort(x, order, out=torch.zeros(8, 16, device=dev)),
           lambda: buf.expert_sort(x, order, out=torch.zeros(16, 8, device=dev, dtype=x.dtype).t()),
           lambda: buf.expert_sort(x, ExpertOrder(None, order.row_of_slot.long(), None)),
           lambda: buf.expert_unsort(x, order),
           lambda: buf.expert_unsort(torch.zeros(8, 16, device=dev), order,
                                     torch.zeros(4, 2, device=dev, dtype=torch.float64)),
           lambda: buf.expert_unsort_backward(x, torch.zeros(8, 16, device=dev), order,
                                              torch.zeros(4, 2, device=dev))]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    odd = torch.zeros(4, 12, device=dev, dtype=torch.bfloat16)
    wide = torch.zeros(2, 17, dtype=torch.int64, device=dev)
    for f in (lambda: buf.expert_sort(odd, order), lambda: buf.expert_order(wide)):
        with pytest.raises(C.MoedxError) as e:
            f()
        assert e.value.code == C.MOEDX_EINVAL
    # outputs on their inputs, and more rows than a grid has waves
    flat = torch.zeros(12, 16, device=dev, dtype=torch.bfloat16)
    p = flat.data_ptr()
    big = [(1 << 26, 1, 8), (1 << 22, 16, 8), (1 << 24, 4, 4096)]
    for f in [lambda: buf.expert_sort(flat[:4], order, out=flat[3:11]),
              lambda: buf.expert_unsort(flat[:8], order, out=flat[7:11]),
              lambda: buf.expert_sort(flat.view(-1)[1:65].view(4, 16), order),
              lambda: buf.expert_unsort(flat.view(-1)[1:129].view(8, 16), order),
              lambda: buf.expert_unsort_backward(flat[:4], x.repeat(2, 1), order,
                                                 torch.zeros(4, 2, device=dev), out=flat[2:10]),
              lambda: buf.expert_unsort_backward(x, flat[:8], order,
                                                 torch.zeros(4, 2, device=dev), out=flat[:8])] + [
            lambda n=n: C.check(C.moedx_expert_sort(buf.ctx, p, C.MOEDX_BF16, *n, p, p, None))
            for n in big]:
        with pytest.raises(C.MoedxError) as e:
            f()
        assert e.value.code == C.MOEDX_EINVAL
    # a handle of other rows, and a low-latency handle
    _, _, _, _, h, _ = buf.dispatch(x, topk_idx=idx)
    with pytest.raises(C.MoedxError) as e:
        buf.expert_order(torch.zeros(3, 2, dtype=torch.int64, device=dev), handle=h)
    assert e.value.code == C.MOEDX_ESTATE
    _, _, ll, _, _ = buf.low_latency_dispatch(x, idx, 8, 16)
    with pytest.raises(C.MoedxError) as e:
        buf.expert_order(idx, handle=ll)
    assert e.value.code == C.MOEDX_EINVAL


def test_gradients_with_index_outside():
    """A row index outside [0, T * K) is an empty slot for every call: its
    weight's gradient is zero."""
    import ctypes

    from combine_get_dispatch_layout_amd import _capi as C
    dev = device()
    T, E, K, H = 9, 4, 3, 40
    buf = make_buffer(E, 1, 1, T)
    order, _ = buf.expert_order(routing("full", T, E, K, 11).to(dev))
    ros, sor = order.row_of_slot.clone(), order.slot_of_row.clone()
    outside = {5: T * K, 11: (1 << 31) - 1, 20: -9}
    for slot, row in outside.items():
        sor[ros.view(-1)[slot].long()] = -1
        ros.view(-1)[slot] = row
    y, d_out = torch.randn(T * K, H, device=dev), torch.randn(T, H, device=dev)
    w = torch.rand(T, K, device=dev)
    d_rows, d_w = torch.full_like(y, 7.0), torch.full_like(w, 7.0)
    ex = C.moedx_exec(stream=torch.cuda.current_stream().cuda_stream)
    C.check(C.moedx_expert_unsort_backward(
        buf.ctx, d_out.data_ptr(), y.data_ptr(), C.MOEDX_F32, T, K, H, ros.data_ptr(), sor.data_ptr(),
        w.data_ptr(), d_rows.data_ptr(), d_w.data_ptr(), ctypes.byref(ex)))
    torch.cuda.synchronize()
    want_rows, want_w, _ = buf.expert_unsort_backward(d_out, y, order, w)
    for slot in range(T * K):
        row = int(order.row_of_slot.view(-1)[slot])
        if slot in outside:
            assert float(d_w.view(-1)[slot]) == 0.0 and (d_rows[row] == 7.0).all()
        else:
            assert torch.equal(d_w.view(-1)[slot], want_w.view(-1)[slot])
            assert torch.equal(d_rows[row], want_rows[row])
