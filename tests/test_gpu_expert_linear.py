"""The experts' products (expert_linear and its gradients) against fp64
products of the same inputs.  A sum of n products in fp32, in any order,
differs by at most (n + 1) 2^-23 of the sum of their sizes (2^-23: the matrix
instructions' own additions may truncate), and an output by half a step of its
type more."""

import pytest
import torch

from tests.gpu_common import device, make_buffer

pytestmark = pytest.mark.gpu

V = 2.0 ** -23


def half_step(want, acc, dt):
    if dt == torch.float32:
        return torch.finfo(dt).tiny
    return torch.finfo(dt).eps / 2 * (want.abs() + acc) + 2.0 ** -24 * (dt == torch.float16) + 1e-37


def spans(counts, gap=0):
    """Offsets of experts with these row counts."""
    out = [gap]
    for c in counts:
        out.append(out[-1] + c)
    return out


def check(name, got, want, acc, dt):
    err = (got.double() - want).abs()
    bad = err > acc + half_step(want, acc, dt)
    assert not bad.any(), (name, int(bad.sum()), torch.nonzero(bad)[0].tolist(),
                           float(err[bad].max()), float(want[bad].abs().max()))


def swiglu_reference(g, u, dg, du):
    """silu(g) * u and its error for errors dg, du of g and u (|silu'| <= 1.1)
    and 8 roundings of fp32 in the activation."""
    s = g * torch.sigmoid(g)
    h = s * u
    acc = 1.1 * dg * (u.abs() + du) + s.abs() * du + 8 * V * h.abs()
    return h, acc


CASES = [
    # counts per expert, K, N
    ([1], 8, 8),
    ([0, 1, 0, 0], 64, 16),
    ([3, 0, 17, 16, 1, 33], 40, 24),
    ([0, 0, 0], 72, 40),
    ([65, 1, 64, 127], 136, 264),
    ([300, 0, 129, 255, 257, 1], 328, 520),
    ([5] * 16, 1416, 136),
    ([700, 30], 520, 1032),
    ([2, 2, 1, 0, 3, 1, 1, 6], 7168, 64),
    ([1100], 128, 256),
    ([40, 0, 90, 61, 33, 20, 70, 9], 256, 512),
    ([20, 33, 64, 0, 31, 17], 520, 72),
    ([16, 31, 1, 47], 4104, 48),
]
# Enough rows and outputs for 256 x 256 tiles on every compute unit: tiles of
# 256 rows, of 20, 44, 63, 68, 108, 128 and 192, outputs past the last tile,
# reductions of 1 to 17 stages of 64.
CASES += [([2000, 0, 300, 831, 260, 740, 128], k, 4104) for k in (8, 72, 200, 328)]
CASES += [([2000, 0, 300, 831, 260, 740, 128], 4104, n) for n in (16, 136, 192, 1032)]
# Reductions that workgroups enter at scattered places, in each tile size.
CASES += [([2, 1, 0, 17, 3], 4096, 72), ([9, 12, 30], 2048, 136),
          ([60, 70, 0, 55, 61, 90, 33, 64], 2048, 4096)]
TYPES = [torch.bfloat16, torch.float16]


def make(counts, K, N, dt, dev, seed, cols):
    g = torch.Generator(dev).manual_seed(seed)
    off = spans(counts)
    M = off[-1] + 5  # rows behind the last expert's
    x = torch.randn(M, K, generator=g, device=dev).to(dt)
    w = (torch.randn(len(counts), cols, K, generator=g, device=dev) * K ** -0.5).to(dt)
    return off, M, x, w, g


@pytest.mark.parametrize("dt", TYPES, ids=lambda d: str(d)[6:])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}e{sum(c[0])}r-{c[1]}-{c[2]}")
def test_forward(case, dt):
    counts, K, N = case
    dev = device()
    E = len(counts)
    buf = make_buffer(E, 1, 1, 1)
    off, M, x, w, _ = make(counts, K, N, dt, dev, 1, 2 * N)
    x[off[-1]:] = float("nan")  # never read into a result
    rows = torch.tensor(off, dtype=torch.int32, device=dev)
    print(f"[linear] {case} {dt}", flush=True)
    y, none, _ = buf.expert_linear(x, w[:, :N].contiguous(), rows,
                                   out=torch.full((M, N), 7.0, dtype=dt, device=dev))
    assert none is None
    h, pre, _ = buf.expert_linear(x, w, rows, swiglu=True, return_pre=True,
                                  out=torch.full((M, N), 7.0, dtype=dt, device=dev))
    h2, _, _ = buf.expert_linear(x, w, rows, swiglu=True)
    assert (y[off[-1]:] == 7.0).all() and (h[off[-1]:] == 7.0).all()
    assert torch.equal(h[:off[-1]], h2[:off[-1]])
    for e in range(E):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        xs, ws = x[a:b].double(), w[e].double().t().contiguous()
        p = xs @ ws
        acc = (K + 1) * V * (xs.abs() @ ws.abs())
        check("y", y[a:b], p[:, :N], acc[:, :N], dt)
        check("pre", pre[a:b], p, acc, dt)
        want, err = swiglu_reference(p[:, :N], p[:, N:], acc[:, :N], acc[:, N:])
        check("h", h[a:b], want, err, dt)


@pytest.mark.parametrize("wide", [False, True], ids=["same", "fp32"])
@pytest.mark.parametrize("dt", TYPES, ids=lambda d: str(d)[6:])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}e{sum(c[0])}r-{c[1]}-{c[2]}")
def test_backward(case, dt, wide):
    counts, K, N = case
    dev = device()
    E = len(counts)
    buf = make_buffer(E, 1, 1, 1)
    off, M, x, w, g = make(counts, K, N, dt, dev, 2, N)
    d_y = torch.randn(M, N, generator=g, device=dev).to(dt)
    x[off[-1]:] = float("inf")
    d_y[off[-1]:] = float("nan")
    rows = torch.tensor(off, dtype=torch.int32, device=dev)
    wt = torch.float32 if wide else dt
    print(f"[linear backward] {case} {dt} {wt}", flush=True)
    d_x, d_w, _ = buf.expert_linear_backward(d_y, x, w, rows, d_w_dtype=wt,
                                             out=torch.full((M, K), 7.0, dtype=dt, device=dev))
    assert (d_x[off[-1]:] == 7.0).all() and d_w.dtype == wt
    for e in range(E):
        a, b = off[e], off[e + 1]
        if a == b:
            assert (d_w[e] == 0).all()
            continue
        d, xs, ws = d_y[a:b].double(), x[a:b].double(), w[e].double()
        check("d_x", d_x[a:b], d @ ws, (N + 1) * V * (d.abs() @ ws.abs()), dt)
        dt_ = d.t().contiguous()
        check("d_w", d_w[e], dt_ @ xs, (b - a + 1) * V * (dt_.abs() @ xs.abs()), wt)


@pytest.mark.parametrize("dt", TYPES, ids=lambda d: str(d)[6:])
@pytest.mark.parametrize("N", [8, 24, 2056])
def test_swiglu_backward(N, dt):
    dev = device()
    counts = [3, 0, 5, 1]
    buf = make_buffer(4, 1, 1, 1)
    off = spans(counts)
    M = off[-1] + 3
    g = torch.Generator(dev).manual_seed(3)
    pre = (torch.randn(M, 2 * N, generator=g, device=dev) * 4).to(dt)
    pre[0, :4] = torch.tensor([80.0, -80.0, 0.0, -1.2785], device=dev).to(dt)
    d_h = torch.randn(M, N, generator=g, device=dev).to(dt)
    rows = torch.tensor(off, dtype=torch.int32, device=dev)
    d_pre, _ = buf.expert_swiglu_backward(d_h, pre, rows,
                                          out=torch.full((M, 2 * N), 7.0, dtype=dt, device=dev))
    n = off[-1]
    assert (d_pre[n:] == 7.0).all()
    gg, u, d = pre[:n, :N].double(), pre[:n, N:].double(), d_h[:n].double()
    s, s1 = torch.sigmoid(gg), torch.sigmoid(-gg)
    want = torch.cat([d * u * s * (1 + gg * s1), d * gg * s], 1)
    # 16 roundings of each term; the two terms of d_gate may cancel
    acc = 16 * V * torch.cat([(d * u * s).abs() * (1 + (gg * s1).abs()), (d * gg * s).abs()], 1)
    check("d_pre", d_pre[:n], want, acc, dt)


def test_swiglu_backward_of_many_rows():
    """More rows than workgroups."""
    dev = device()
    M, N, dt = (1 << 20) + 77, 8, torch.bfloat16
    buf = make_buffer(2, 1, 1, 1)
    rows = torch.tensor([1, 1 << 19, M - 1], dtype=torch.int32, device=dev)
    pre = torch.randn(M, 2 * N, device=dev).to(dt)
    d_h = torch.randn(M, N, device=dev).to(dt)
    d_pre, _ = buf.expert_swiglu_backward(d_h, pre, rows,
                                          out=torch.full((M, 2 * N), 7.0, dtype=dt, device=dev))
    assert (d_pre[0] == 7.0).all() and (d_pre[-1] == 7.0).all()
    part = slice(M - 100, M - 1)
    again, _ = buf.expert_swiglu_backward(d_h[part], pre[part],
                                          torch.tensor([0, 9, 99], dtype=torch.int32, device=dev))
    assert torch.equal(d_pre[part], again)
    assert not (d_pre[1:-1] == 7.0).all(1).any()


@pytest.mark.parametrize("cap", [1, 7, 130])
def test_slots_with_counts(cap):
    """[E, cap, *] buffers with counts (the low-latency layout); counts beyond
    the capacity or below zero are clamped."""
    dev = device()
    E, K, N, dt = 5, 72, 40, torch.bfloat16
    counts = [cap, 0, min(3, cap), cap + 9, -4]
    held = [cap, 0, min(3, cap), cap, 0]
    buf = make_buffer(E, 1, 1, 1)
    g = torch.Generator(dev).manual_seed(4)
    x = torch.randn(E, cap, K, generator=g, device=dev).to(dt)
    w = (torch.randn(E, N, K, generator=g, device=dev) * K ** -0.5).to(dt)
    d_y = torch.randn(E, cap, N, generator=g, device=dev).to(dt)
    rows = torch.tensor(counts, dtype=torch.int32, device=dev)
    y, _, _ = buf.expert_linear(x, w, rows, out=torch.full((E, cap, N), 7.0, dtype=dt, device=dev))
    d_x, d_w, _ = buf.expert_linear_backward(
        d_y, x, w, rows, out=torch.full((E, cap, K), 7.0, dtype=dt, device=dev))
    for e in range(E):
        c = held[e]
        assert (y[e, c:] == 7.0).all() and (d_x[e, c:] == 7.0).all()
        if c == 0:
            assert (d_w[e] == 0).all()
            continue
        xs, ws, d = x[e, :c].double(), w[e].double(), d_y[e, :c].double()
        wt, dtr = ws.t().contiguous(), d.t().contiguous()
        check("y", y[e, :c], xs @ wt, (K + 1) * V * (xs.abs() @ wt.abs()), dt)
        check("d_x", d_x[e, :c], d @ ws, (N + 1) * V * (d.abs() @ ws.abs()), dt)
        check("d_w", d_w[e], dtr @ xs, (c + 1) * V * (dtr.abs() @ xs.abs()), dt)


def test_wide_slots():
    """Slots whose live rows fill 256 x 256 tiles, a prefix of each expert's."""
    dev = device()
    E, cap, K, N, dt = 3, 1500, 136, 4096, torch.bfloat16
    held = [1500, 257, 1024]
    buf = make_buffer(E, 1, 1, 1)
    g = torch.Generator(dev).manual_seed(5)
    x = torch.randn(E, cap, K, generator=g, device=dev).to(dt)
    w = (torch.randn(E, N, K, generator=g, device=dev) * K ** -0.5).to(dt)
    for e in range(E):
        x[e, held[e]:] = float("nan")
    rows = torch.tensor(held, dtype=torch.int32, device=dev)
    y, _, _ = buf.expert_linear(x, w, rows, out=torch.full((E, cap, N), 7.0, dtype=dt, device=dev))
    for e, c in enumerate(held):
        assert (y[e, c:] == 7.0).all()
        xs, wt = x[e, :c].double(), w[e].double().t().contiguous()
        check("y", y[e, :c], xs @ wt, (K + 1) * V * (xs.abs() @ wt.abs()), dt)


def test_one_gradient_at_a_time():
    """The C call leaves out the gradient whose pointer is null."""
    import ctypes

    from combine_get_dispatch_layout_amd import _capi as C
    dev = device()
    counts, K, N, dt = [30, 0, 65], 72, 40, torch.bfloat16
    E = len(counts)
    buf = make_buffer(E, 1, 1, 1)
    off, M, x, w, g = make(counts, K, N, dt, dev, 8, N)
    d_y = torch.randn(M, N, generator=g, device=dev).to(dt)
    rows = torch.tensor(off, dtype=torch.int32, device=dev)
    d_x, d_w, _ = buf.expert_linear_backward(d_y, x, w, rows,
                                             out=torch.zeros(M, K, dtype=dt, device=dev))
    a, b = torch.zeros_like(d_x), torch.full_like(d_w, 7.0)
    er = C.moedx_expert_rows(rows.data_ptr(), None, M)
    ex = C.moedx_exec(stream=torch.cuda.current_stream().cuda_stream)

    def call(px, pw, pdx, pdw):
        C.check(C.moedx_expert_linear_backward(
            buf.ctx, d_y.data_ptr(), px, pw, C.MOEDX_BF16, K, N, ctypes.byref(er), pdx, pdw,
            C.MOEDX_BF16, ctypes.byref(ex)))

    call(None, w.data_ptr(), a.data_ptr(), None)
    call(x.data_ptr(), None, None, b.data_ptr())
    torch.cuda.synchronize()
    assert torch.equal(a, d_x) and torch.equal(b, d_w)
    for bad in ((x.data_ptr(), None, a.data_ptr(), None), (None, w.data_ptr(), None, b.data_ptr()),
                (x.data_ptr(), w.data_ptr(), None, None)):
        with pytest.raises(C.MoedxError) as err:
            call(*bad)
        assert err.value.code == C.MOEDX_EINVAL


def test_buffers_past_4_gib():
    """Rows, gradients and weights whose offsets pass 32 bits."""
    dev = device()
    dt, K, N = torch.bfloat16, 8192, 8
    M = (1 << 32) // (K * 2) + 1000
    buf = make_buffer(2, 1, 1, 1)
    g = torch.Generator(dev).manual_seed(9)
    x = torch.zeros(M, K, device=dev, dtype=dt)
    d_y = torch.zeros(M, N, device=dev, dtype=dt)
    x[-40:] = torch.randn(40, K, generator=g, device=dev).to(dt)
    d_y[-40:] = torch.randn(40, N, generator=g, device=dev).to(dt)
    w = (torch.randn(2, N, K, generator=g, device=dev) * K ** -0.5).to(dt)
    rows = torch.tensor([0, 7, M], dtype=torch.int32, device=dev)
    print("[linear] rows past 4 GiB", flush=True)
    y, _, _ = buf.expert_linear(x, w, rows)
    d_x, d_w, _ = buf.expert_linear_backward(d_y, x, w, rows, d_w_dtype=torch.float32)
    xs, ws, d = x[-40:].double(), w[1].double(), d_y[-40:].double()
    wt, dtr = ws.t().contiguous(), d.t().contiguous()
    check("y", y[-40:], xs @ wt, (K + 1) * V * (xs.abs() @ wt.abs()), dt)
    check("d_x", d_x[-40:], d @ ws, (N + 1) * V * (d.abs() @ ws.abs()), dt)
    check("d_w", d_w[1], dtr @ xs, 41 * V * (dtr.abs() @ xs.abs()), torch.float32)
    assert (y[:-40] == 0).all() and (d_x[7:-40] == 0).all() and (d_w[0] == 0).all()
    del x, y, d_x

    E, N = 40, 8192
    buf = make_buffer(E, 1, 1, 1)
    w = torch.zeros(E, N, K, device=dev, dtype=dt)
    w[-1] = (torch.randn(N, K, generator=g, device=dev) * K ** -0.5).to(dt)
    x = torch.randn(5, K, generator=g, device=dev).to(dt)
    rows = torch.zeros(E + 1, dtype=torch.int32, device=dev)
    rows[-1] = 5
    print("[linear] weights past 4 GiB", flush=True)
    y, _, _ = buf.expert_linear(x, w, rows)
    d_x, d_w, _ = buf.expert_linear_backward(y, x, w, rows)
    ws = w[-1].double()
    wt = ws.t().contiguous()
    check("y", y, x.double() @ wt, (K + 1) * V * (x.double().abs() @ wt.abs()), dt)
    check("d_x", d_x, y.double() @ ws, (N + 1) * V * (y.double().abs() @ ws.abs()), dt)
    dtr = y.double().t().contiguous()
    check("d_w", d_w[-1], dtr @ x.double(), 6 * V * (dtr.abs() @ x.double().abs()), dt)
    assert (d_w[:-1] == 0).all()


def test_no_rows_at_all():
    dev = device()
    E, K, N, dt = 3, 16, 24, torch.bfloat16
    buf = make_buffer(E, 1, 1, 1)
    w = torch.ones(E, N, K, device=dev, dtype=dt)
    off = torch.zeros(E + 1, dtype=torch.int32, device=dev)
    x, d_y = torch.empty(0, K, device=dev, dtype=dt), torch.empty(0, N, device=dev, dtype=dt)
    y, pre, _ = buf.expert_linear(x, w, off, swiglu=False)
    assert y.shape == (0, N) and pre is None
    d_x, d_w, _ = buf.expert_linear_backward(d_y, x, w, off, d_w=torch.full_like(w, 7.0))
    assert d_x.shape == (0, K) and (d_w == 0).all()
    slots = torch.empty(E, 0, K, device=dev, dtype=dt)
    y, _, _ = buf.expert_linear(slots, w, off[:E].contiguous())
    assert y.shape == (E, 0, N)
    d_pre, _ = buf.expert_swiglu_backward(d_y, torch.empty(0, 2 * N, device=dev, dtype=dt), off)
    assert d_pre.shape == (0, 2 * N)


def test_offsets_are_clamped():
    """Offsets outside the buffer, or falling, touch nothing outside it."""
    dev = device()
    E, K, N, M, dt = 3, 16, 16, 20, torch.bfloat16
    buf = make_buffer(E, 1, 1, 1)
    x = torch.ones(M, K, device=dev, dtype=dt)
    w = torch.ones(E, N, K, device=dev, dtype=dt)
    for off, live in (([-5, 4, 1 << 30, 1 << 30], (0, 20)), ([2, 6, 5, 9], (2, 9)),
                      ([0, 0, 0, 0], (0, 0))):
        y, _, _ = buf.expert_linear(x, w, torch.tensor(off, dtype=torch.int32, device=dev),
                                    out=torch.full((M, N), 7.0, dtype=dt, device=dev))
        want = torch.full((M, N), 7.0, dtype=dt, device=dev)
        want[live[0]:live[1]] = K
        assert torch.equal(y, want)


def test_special_values_stay_in_their_rows():
    """An infinity or NaN in one row or one expert reaches no other."""
    dev = device()
    E, K, N, dt = 3, 136, 72, torch.bfloat16
    off = [0, 20, 60, 75]
    buf = make_buffer(E, 1, 1, 1)
    g = torch.Generator(dev).manual_seed(6)
    x = torch.randn(75, K, generator=g, device=dev).to(dt)
    w = torch.randn(E, N, K, generator=g, device=dev).to(dt)
    d_y = torch.randn(75, N, generator=g, device=dev).to(dt)
    rows = torch.tensor(off, dtype=torch.int32, device=dev)
    clean, _, _ = buf.expert_linear(x, w, rows)
    c_dx, c_dw, _ = buf.expert_linear_backward(d_y, x, w, rows)
    x2, w2, d2 = x.clone(), w.clone(), d_y.clone()
    x2[30] = float("inf")
    w2[2] = float("nan")
    d2[19] = float("nan")
    y, _, _ = buf.expert_linear(x2, w2, rows)
    same = [m for m in range(60) if m != 30]
    assert torch.equal(y[same], clean[same])
    assert torch.isnan(y[60:]).all() and not torch.isfinite(y[30]).any()
    d_x, d_w, _ = buf.expert_linear_backward(d2, x2, w2, rows)
    same = [m for m in range(60) if m != 19]
    assert torch.equal(d_x[same], c_dx[same])
    assert torch.isnan(d_w[0]).all() and torch.equal(d_w[2], c_dw[2])


def test_refusals():
    from combine_get_dispatch_layout_amd import _capi as C
    dev = device()
    E, K, N, dt = 4, 16, 24, torch.bfloat16
    buf = make_buffer(E, 1, 1, 1)
    x = torch.zeros(10, K, device=dev, dtype=dt)
    w = torch.zeros(E, N, K, device=dev, dtype=dt)
    off = torch.tensor([0, 2, 4, 6, 10], dtype=torch.int32, device=dev)
    d_y = torch.zeros(10, N, device=dev, dtype=dt)
    slots = torch.zeros(E, 3, K, device=dev, dtype=dt)
    bad = [lambda: buf.expert_linear(x, w.half(), off), lambda: buf.expert_linear(x.float(), w.float(), off),
           lambda: buf.expert_linear(x, w[:3], off), lambda: buf.expert_linear(x, w[:, :, :8], off),
           lambda: buf.expert_linear(x, w, off[:4]), lambda: buf.expert_linear(x, w, off.long()),
           lambda: buf.expert_linear(x, w, off, return_pre=True),
           lambda: buf.expert_linear(x, w.cpu(), off), lambda: buf.expert_linear(x[0], w, off),
           lambda: buf.expert_linear(slots, w, off), lambda: buf.expert_linear(slots[:3], w, off[:3]),
           lambda: buf.expert_linear(x, w, off, out=torch.zeros(9, N, device=dev, dtype=dt)),
           lambda: buf.expert_linear_backward(d_y[:9], x, w, off),
           lambda: buf.expert_linear_backward(d_y, x, w, off, d_w_dtype=torch.float16),
           lambda: buf.expert_linear_backward(d_y, x, w, off, d_w=w[:2]),
           lambda: buf.expert_swiglu_backward(d_y, d_y, off)]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    flat = torch.zeros(4096, device=dev, dtype=dt)
    sq = torch.zeros(E, K, K, device=dev, dtype=dt)
    pre = torch.zeros(10, 2 * K, device=dev, dtype=dt)
    over = [lambda: buf.expert_linear(x, sq, off, out=x),
            lambda: buf.expert_linear(flat[:10 * K].view(10, K), sq, off,
                                      out=flat[9 * K:19 * K].view(10, K)),
            lambda: buf.expert_linear(x, sq, off, out=sq.view(-1, K)[:10]),
            lambda: buf.expert_linear_backward(x, x.clone(), sq, off, out=x),
            lambda: buf.expert_linear_backward(x, x.clone(), sq, off, d_w=sq),
            lambda: buf.expert_swiglu_backward(x, pre, off, out=pre)]
    # contiguous views that start inside 16 bytes
    off_x, off_w = flat[1:1 + 10 * K].view(10, K), flat[1:1 + E * N * K].view(E, N, K)
    over += [lambda: buf.expert_linear(off_x, w, off), lambda: buf.expert_linear(x, off_w, off),
             lambda: buf.expert_linear(x, w, off, out=flat[1:1 + 10 * N].view(10, N)),
             lambda: buf.expert_linear_backward(d_y, off_x, w, off),
             lambda: buf.expert_swiglu_backward(off_x, pre, off)]
    for f in over:
        with pytest.raises(C.MoedxError) as e:
            f()
        assert e.value.code == C.MOEDX_EINVAL
    odd = torch.zeros(10, 12, device=dev, dtype=dt)
    for f in (lambda: buf.expert_linear(odd, torch.zeros(E, N, 12, device=dev, dtype=dt), off),
              lambda: buf.expert_linear(x, torch.zeros(E, 12, K, device=dev, dtype=dt), off),
              lambda: buf.expert_linear(x, w, off, swiglu=True)):  # halves of 12 rows
        with pytest.raises(C.MoedxError) as e:
            f()
        assert e.value.code == C.MOEDX_EINVAL


def test_slots_of_many_experts():
    """1024 experts' slots of which few rows are likely: 32-row tiles of the
    whole capacity would be 2^24 workgroups, more than a grid has threads for."""
    dev = device()
    E, cap, K, N, dt = 1024, 1024, 8, 8192, torch.bfloat16
    held = {0: 3, 17: 40, 511: 1024, 1023: 129}
    buf = make_buffer(E, 1, 1, 1)
    g = torch.Generator(dev).manual_seed(12)
    counts = torch.zeros(E, dtype=torch.int32, device=dev)
    x = torch.full((E, cap, K), float("nan"), device=dev, dtype=dt)
    w = torch.randn(E, 2 * N, K, generator=g, device=dev, dtype=torch.float32).to(dt)
    for e, c in held.items():
        counts[e] = c
        x[e, :c] = torch.randn(c, K, generator=g, device=dev).to(dt)
    out = torch.full((E, cap, N), 7.0, dtype=dt, device=dev)
    print("[linear] slots of 1024 experts", flush=True)
    h, _, _ = buf.expert_linear(x, w, counts, swiglu=True, out=out)
    for e, c in held.items():
        xs, ws = x[e, :c].double(), w[e].double().t().contiguous()
        p, acc = xs @ ws, (K + 1) * V * (xs.abs() @ ws.abs())
        want, err = swiglu_reference(p[:, :N], p[:, N:], acc[:, :N], acc[:, N:])
        check("h", h[e, :c], want, err, dt)
        assert (h[e, c:] == 7.0).all() and (e == 1023 or (h[e + 1] == 7.0).all())


def test_more_rows_than_a_grid_has():
    """Buffers whose tiles no grid covers are refused before anything runs."""
    from combine_get_dispatch_layout_amd import _capi as C
    dev = device()
    M, dt = (1 << 31) - 1, torch.bfloat16
    buf = make_buffer(1, 1, 1, 1)
    x, y = torch.empty(M, 8, device=dev, dtype=dt), torch.empty(M, 8, device=dev, dtype=dt)
    w = torch.zeros(1, 8, 8, device=dev, dtype=dt)
    rows = torch.zeros(2, dtype=torch.int32, device=dev)
    for f in (lambda: buf.expert_linear(x, w, rows, out=y),
              lambda: buf.expert_linear_backward(y, x, w, rows, out=torch.empty_like(x))):
        with pytest.raises(C.MoedxError) as e:
            f()
        assert e.value.code == C.MOEDX_EINVAL and "grid" in str(e.value)


def test_rows_near_2_31():
    """One expert whose rows reach 2^31: every one of them is written, forward
    and input gradient, and the products are exact (powers of two)."""
    import ctypes

    from combine_get_dispatch_layout_amd import _capi as C
    dev = device()
    M, dt = (1 << 31) - 1024, torch.bfloat16
    buf = make_buffer(1, 1, 1, 1)
    powers = 2.0 ** torch.arange(8, device=dev)
    w = torch.zeros(1, 8, 8, device=dev, dtype=dt)
    w[0, :, 0] = powers.to(dt)  # y[m, n] = 2^n x[m, 0]
    x, y = torch.zeros(M, 8, device=dev, dtype=dt), torch.zeros(M, 8, device=dev, dtype=dt)
    step = 1 << 27
    for a in range(0, M, step):
        b = min(a + step, M)
        x[a:b, 0] = (torch.arange(a, b, device=dev) % 251 + 1).to(dt)
    live = (5, M - 3)
    rows = torch.tensor(live, dtype=torch.int32, device=dev)

    def check_rows(got, weights):
        for a in range(0, M, step):
            b = min(a + step, M)
            for n in range(8):
                want = x[a:b, 0] * weights[n].to(dt)
                if a < live[0]:
                    want[:live[0] - a] = 0
                if b > live[1]:
                    want[live[1] - a:] = 0
                assert torch.equal(got[a:b, n], want), (a, n)

    print("[linear] rows near 2^31", flush=True)
    buf.expert_linear(x, w, rows, out=y)
    check_rows(y, powers)
    y.zero_()
    wt = w.transpose(1, 2).contiguous()  # d_x[m, k] = 2^k d_y[m, 0]
    er = C.moedx_expert_rows(rows.data_ptr(), None, M)
    ex = C.moedx_exec(stream=torch.cuda.current_stream().cuda_stream)
    print("[linear backward] rows near 2^31", flush=True)
    C.check(C.moedx_expert_linear_backward(buf.ctx, x.data_ptr(), None, wt.data_ptr(), C.MOEDX_BF16,
                                           8, 8, ctypes.byref(er), y.data_ptr(), None, C.MOEDX_BF16,
                                           ctypes.byref(ex)))
    check_rows(y, powers)


@pytest.mark.parametrize("E,cap", [(65, 32), (128, 32), (200, 128), (512, 300), (1024, 1), (1024, 130)])
@pytest.mark.parametrize("dense", [False, True], ids=["few live", "all live"])
def test_many_experts(E, cap, dense):
    """More experts than a wave has lanes, in slots and in expert order: a tile's
    expert is found past others, whichever tiles the buffer's size picks."""
    dev = device()
    K, N, dt = 72, 40, torch.bfloat16
    buf = make_buffer(E, 1, 1, 1)
    g = torch.Generator().manual_seed(E + cap)
    counts = torch.randint(0 if cap > 1 else 1, min(cap, 3) + 1, (E,), generator=g)
    if not dense:
        counts *= (torch.rand(E, generator=g) < 0.03).long()
        counts[E - 1] = min(cap, 2)
    if cap > 64:
        counts[E // 2], counts[63], counts[64] = cap, cap - 1, 33
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)])
    M = int(offsets[-1])
    ex = torch.repeat_interleave(torch.arange(E), counts)  # the expert of each row
    slot = (torch.arange(M) - offsets[ex]).to(dev)
    ex = ex.to(dev)
    x = torch.randn(M, K, generator=g).to(dev).to(dt)
    w = (torch.randn(E, N, K, generator=g) * K ** -0.5).to(dev).to(dt)
    d_y = torch.randn(M, N, generator=g).to(dev).to(dt)
    rows, cnt = offsets.int().to(dev), counts.int().to(dev)
    slots_x = torch.full((E, cap, K), float("nan"), dtype=dt, device=dev)
    slots_d = torch.full((E, cap, N), float("nan"), dtype=dt, device=dev)
    slots_x[ex, slot], slots_d[ex, slot] = x, d_y
    print(f"[linear] {E} experts, slots of {cap}, {M} rows", flush=True)
    y, _, _ = buf.expert_linear(x, w, rows)
    sy, _, _ = buf.expert_linear(slots_x, w, cnt,
                                 out=torch.full((E, cap, N), 7.0, dtype=dt, device=dev))
    d_x, d_w, _ = buf.expert_linear_backward(d_y, x, w, rows)
    s_dx, s_dw, _ = buf.expert_linear_backward(
        slots_d, slots_x, w, cnt, out=torch.full((E, cap, K), 7.0, dtype=dt, device=dev))
    we, xd, dd = w.double()[ex], x.double(), d_y.double()
    want = (we * xd[:, None, :]).sum(2)
    acc = (K + 1) * V * (we.abs() * xd.abs()[:, None, :]).sum(2)
    check("y", y, want, acc, dt)
    check("y in slots", sy[ex, slot], want, acc, dt)
    want = (we * dd[:, :, None]).sum(1)
    acc = (N + 1) * V * (we.abs() * dd.abs()[:, :, None]).sum(1)
    check("d_x", d_x, want, acc, dt)
    check("d_x in slots", s_dx[ex, slot], want, acc, dt)
    want = torch.zeros(E, N, K, dtype=torch.float64, device=dev)
    size = torch.zeros_like(want)
    outer = dd[:, :, None] * xd[:, None, :]
    want.index_add_(0, ex, outer)
    size.index_add_(0, ex, outer.abs())
    n = counts.to(dev).double()[:, None, None] + 1
    check("d_w", d_w, want, n * V * size, dt)
    check("d_w in slots", s_dw, want, n * V * size, dt)
    empty = torch.ones(E, cap, dtype=torch.bool, device=dev)
    empty[ex, slot] = False
    assert (sy[empty] == 7.0).all() and (s_dx[empty] == 7.0).all()
