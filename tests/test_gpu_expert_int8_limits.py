"""The int8 calls at their limits: offsets outside the buffer, many experts, the
most rows, strided and misaligned inputs, refusals."""

import ctypes

import pytest
import torch

from tests.gpu_common import device, make_buffer
from tests.test_gpu_expert_int8 import product, quantized, swiglu_gradients, values
from tests.test_gpu_expert_linear import V, check

pytestmark = pytest.mark.gpu


def test_offsets_are_clamped():
    """Offsets outside the buffer, or falling, touch nothing outside it."""
    dev = device()
    E, K, N, M = 3, 16, 16, 20
    buf = make_buffer(E, 1, 1, 1)
    x = torch.ones(M, K, device=dev, dtype=torch.bfloat16)
    w, ws, _ = buf.expert_quantize(torch.ones(E, N, K, device=dev))
    for off, live in (([-5, 4, 1 << 30, 1 << 30], (0, 20)), ([2, 6, 5, 9], (2, 9)),
                      ([0, 0, 0, 0], (0, 0)), ([25, 30, 31, 40], (0, 0))):
        rows = torch.tensor(off, dtype=torch.int32, device=dev)
        inside = torch.zeros(M, dtype=torch.bool, device=dev)
        inside[live[0]:live[1]] = True
        for block in (0, 128):
            shape = (M,) if block == 0 else (M, 1)
            codes, scales, _ = buf.expert_quantize(
                x, rows, block=block, out=torch.full((M, K), 7, dtype=torch.int8, device=dev),
                scales=torch.full(shape, 9.0, device=dev))
            assert ((codes == 127).all(1) == inside).all() and ((codes == 7).all(1) == ~inside).all()
            assert ((scales.view(M) == 9.0) == ~inside).all()
            back, _ = buf.expert_dequantize(codes, scales, rows, dtype=torch.float32,
                                            out=torch.full((M, K), 5.0, device=dev))
            assert ((back == 5.0).all(1) == ~inside).all()
        codes, scales, _ = buf.expert_quantize(x)
        y, _ = buf.expert_linear_int8(codes, scales, w, ws, rows,
                                      out=torch.full((M, N), 7.0, dtype=torch.bfloat16, device=dev))
        assert ((y == K).all(1) == inside).all() and ((y == 7.0).all(1) == ~inside).all()
        pre, ps, _ = buf.expert_quantize(torch.ones(M, 2 * N, device=dev))
        d_pre, h, _ = buf.expert_swiglu_backward_int8(
            x, pre, ps, rows, out=torch.full((M, 2 * N), 7.0, dtype=x.dtype, device=dev),
            h=torch.full((M, N), 7.0, dtype=x.dtype, device=dev))
        assert ((h == 7.0).all(1) == ~inside).all() and ((d_pre == 7.0).all(1) == ~inside).all()
        # of falling offsets, the rows of each expert
        _, d_w, _ = buf.expert_linear_backward_int8(x, codes, scales, None, rows)
        lo = [min(max(o, 0), M) for o in off]
        for e in range(E):
            assert (d_w[e] == max(lo[e + 1] - lo[e], 0)).all()


@pytest.mark.parametrize("E,cap", [(65, 32), (128, 32), (200, 128), (512, 300), (1024, 1), (1024, 130)])
@pytest.mark.parametrize("dense", [False, True], ids=["few live", "all live"])
def test_many_experts(E, cap, dense):
    """More experts than a wave has lanes, in slots and in expert order."""
    dev = device()
    K, N, dt = 80, 40, torch.bfloat16
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
    d_y = torch.randn(M, N, generator=g).to(dev).to(dt)
    w = torch.randint(-127, 128, (E, 2 * N, K), generator=g, dtype=torch.int8).to(dev)
    ws = (torch.rand(E, 2 * N, generator=g) * 0.01).to(dev)
    rows, cnt = offsets.int().to(dev), counts.int().to(dev)
    sx = torch.full((E, cap, K), float("nan"), dtype=dt, device=dev)
    sd = torch.full((E, cap, N), float("nan"), dtype=dt, device=dev)
    sx[ex, slot], sd[ex, slot] = x, d_y
    print(f"[int8] {E} experts, slots of {cap}, {M} rows", flush=True)
    for block in (128, 0):
        codes, scales, _ = buf.expert_quantize(x, rows, block=block)
        c, s = quantized(x, block)
        assert torch.equal(codes.cpu(), c) and torch.equal(scales.cpu(), s)
        sc, ss, _ = buf.expert_quantize(sx, cnt, block=block)
        assert torch.equal(sc[ex, slot], codes) and torch.equal(ss[ex, slot], scales)
        back, _ = buf.expert_dequantize(sc, ss, cnt, dtype=dt,
                                        out=torch.full((E, cap, K), 5.0, dtype=dt, device=dev))
        saved = values(codes, scales).to(dt)
        assert torch.equal(back[ex, slot], saved)
        assert int((back == 5.0).all(2).sum()) == E * cap - M
        _, d_w, _ = buf.expert_linear_backward_int8(d_y, codes, scales, None, rows)
        _, s_dw, _ = buf.expert_linear_backward_int8(sd, sc, ss, None, cnt)
        outer = d_y.double()[:, :, None] * saved.double()[:, None, :]
        want = torch.zeros(E, N, K, dtype=torch.float64, device=dev)
        size = torch.zeros_like(want)
        want.index_add_(0, ex, outer)
        size.index_add_(0, ex, outer.abs())
        acc = (counts.max().item() + 1) * V * size
        check("d_w", d_w, want, acc, dt)
        check("d_w of slots", s_dw, want, acc, dt)
    total = (w.double()[ex] * codes.double()[:, None, :]).sum(2).float()
    want = total * scales[:, None] * ws[ex]
    for swiglu in (False, True):
        wv, wsv = (w, ws) if swiglu else (w[:, :N].contiguous(), ws[:, :N].contiguous())
        y, _ = buf.expert_linear_int8(codes, scales, wv, wsv, rows, swiglu=swiglu)
        sy, _ = buf.expert_linear_int8(sc, ss, wv, wsv, cnt, swiglu=swiglu,
                                       out=torch.full((E, cap, N), 7.0, dtype=dt, device=dev))
        assert torch.equal(sy[ex, slot], y)
        assert int((sy == 7.0).all(2).sum()) == E * cap - M
        if swiglu:
            gd, u = want[:, :N].double(), want[:, N:].double()
            h = gd * torch.sigmoid(gd) * u
            check("h", y, h, 8 * V * h.abs(), dt)
        else:
            assert torch.equal(y, want[:, :N].to(dt))
    pre, ps = codes[:, :2 * N].contiguous(), scales
    d_pre, h, _ = buf.expert_swiglu_backward_int8(sd, sc, ss, cnt, return_h=True)
    p = values(pre, ps).double()
    want, want_h = swiglu_gradients(p[:, :N], p[:, N:], d_y.double())
    gd, u, d = p[:, :N], p[:, N:], d_y.double()
    sg = torch.sigmoid(gd)
    acc = 16 * V * torch.cat([(d * u * sg).abs() * (1 + (gd * (1 - sg)).abs()), (d * gd * sg).abs()], 1)
    check("d_pre", d_pre[ex, slot], want, acc, dt)
    check("h of slots", h[ex, slot], want_h, 8 * V * want_h.abs(), dt)


@pytest.mark.parametrize("K", [16, 160, 400, 1040])
def test_wide_tiles_of_many_experts(K):
    """256 x 256 tiles, several to a workgroup, among more experts than a wave has
    lanes: runs of experts without rows, a few rows and many, in expert order
    and in slots."""
    dev = device()
    E, N, cap, dt = 200, 1032, 2048, torch.bfloat16
    g = torch.Generator().manual_seed(K)
    counts = torch.randint(0, 40, (E,), generator=g)
    counts[60:140] = 0
    for e, c in ((0, 700), (63, 1), (64, 513), (65, 256), (127, 2048), (128, 300), (139, 0),
                 (140, 1900), (191, 255), (192, 257), (199, 2000)):
        counts[e] = c
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)])
    M = int(offsets[-1]) + 9000  # rows behind the last expert's: more than 72 an expert
    assert M >= 73 * E
    buf = make_buffer(E, 1, 1, 1)
    gd = torch.Generator(dev).manual_seed(K)
    x = torch.randint(-128, 128, (M, K), generator=gd, device=dev, dtype=torch.int8)
    w = torch.randint(-128, 128, (E, 2 * N, K), generator=gd, device=dev, dtype=torch.int8)
    xs = torch.rand(M, generator=gd, device=dev) * 0.02
    ws = torch.rand(E, 2 * N, generator=gd, device=dev) * K ** -0.5 * 0.02
    xs[int(offsets[-1]):] = float("nan")
    wn, wsn = w[:, :N].contiguous(), ws[:, :N].contiguous()
    rows, cnt = offsets.int().to(dev), counts.int().to(dev)
    print(f"[int8] wide tiles of many experts, K={K}", flush=True)
    sevens = lambda *s: torch.full(s + (N,), 7.0, dtype=dt, device=dev)  # noqa: E731
    y, _ = buf.expert_linear_int8(x, xs, wn, wsn, rows, out=sevens(M))
    h, _ = buf.expert_linear_int8(x, xs, w, ws, rows, swiglu=True, out=sevens(M))
    assert (y[int(offsets[-1]):] == 7.0).all() and (h[int(offsets[-1]):] == 7.0).all()
    sx = torch.zeros(E, cap, K, dtype=torch.int8, device=dev)
    ss = torch.full((E, cap), float("nan"), device=dev)
    for e in range(E):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if a == b:
            continue
        p = product(x[a:b], xs[a:b], w[e], ws[e])
        assert torch.equal(y[a:b], p[:, :N].to(dt)), e
        gt, u = p[:, :N].double(), p[:, N:].double()
        want = gt * torch.sigmoid(gt) * u
        check("h", h[a:b], want, 8 * V * want.abs(), dt)
        sx[e, :b - a], ss[e, :b - a] = x[a:b], xs[a:b]
    sy, _ = buf.expert_linear_int8(sx, ss, wn, wsn, cnt, out=sevens(E, cap))
    sh, _ = buf.expert_linear_int8(sx, ss, w, ws, cnt, swiglu=True, out=sevens(E, cap))
    for e in range(E):
        a, c = int(offsets[e]), int(counts[e])
        assert torch.equal(sy[e, :c], y[a:a + c]) and torch.equal(sh[e, :c], h[a:a + c]), e
        assert (sy[e, c:] == 7.0).all() and (sh[e, c:] == 7.0).all(), e


def test_slots_of_many_experts():
    """1024 experts' slots of which few rows are likely."""
    dev = device()
    E, cap, K, N = 1024, 1024, 16, 8192
    held = {0: 3, 17: 40, 511: 1024, 1023: 129}
    buf = make_buffer(E, 1, 1, 1)
    g = torch.Generator(dev).manual_seed(12)
    counts = torch.zeros(E, dtype=torch.int32, device=dev)
    for e, c in held.items():
        counts[e] = c
    x = torch.randint(-128, 128, (E, cap, K), generator=g, device=dev, dtype=torch.int8)
    xs = torch.rand(E, cap, generator=g, device=dev)
    w = torch.randint(-128, 128, (E, N, K), generator=g, device=dev, dtype=torch.int8)
    ws = torch.rand(E, N, generator=g, device=dev)
    out = torch.full((E, cap, N), 7.0, dtype=torch.bfloat16, device=dev)
    print("[int8] slots of 1024 experts", flush=True)
    y, _ = buf.expert_linear_int8(x, xs, w, ws, counts, out=out)
    for e, c in held.items():
        assert torch.equal(y[e, :c], product(x[e, :c], xs[e, :c], w[e], ws[e]).to(y.dtype))
        assert (y[e, c:] == 7.0).all() and (e == 1023 or (y[e + 1] == 7.0).all())


def test_rows_near_2_31():
    """One expert whose rows reach 2^31: every one of them is quantised,
    multiplied and restored, exactly (a row's one value is a power of two times
    127, its scale that power)."""
    dev = device()
    M, K, N, dt = (1 << 31) - 1024, 16, 8, torch.bfloat16
    buf = make_buffer(1, 1, 1, 1)
    x = torch.zeros(M, K, device=dev, dtype=dt)
    step = 1 << 27
    powers = torch.tensor([2.0 ** (i - 48) for i in range(97)], device=dev)  # exact, unlike pow
    power = lambda a, b: powers[torch.arange(a, b, device=dev) % 97]  # noqa: E731
    for a in range(0, M, step):
        b = min(a + step, M)
        x[a:b, 3] = (127 * power(a, b)).to(dt)
    live = (5, M - 3)
    rows = torch.tensor(live, dtype=torch.int32, device=dev)
    codes = torch.full((M, K), 7, device=dev, dtype=torch.int8)
    scales = torch.full((M,), 3.0, device=dev)
    print("[int8] quantise rows near 2^31", flush=True)
    buf.expert_quantize(x, rows, out=codes, scales=scales)
    w = torch.zeros(1, N, K, device=dev, dtype=torch.int8)
    w[0, :, 3] = torch.arange(1, N + 1, device=dev).to(torch.int8)
    ws = torch.ones(1, N, device=dev)
    y = torch.zeros(M, N, device=dev, dtype=dt)
    print("[int8] product of rows near 2^31", flush=True)
    buf.expert_linear_int8(codes, scales, w, ws, rows, out=y)
    x.fill_(9.0)
    print("[int8] restore rows near 2^31", flush=True)
    buf.expert_dequantize(codes, scales, rows, out=x)
    torch.cuda.synchronize()
    for a in range(0, M, step):
        b = min(a + step, M)
        p = power(a, b)
        inside = torch.ones(b - a, dtype=torch.bool, device=dev)
        inside[:max(live[0] - a, 0)] = False
        inside[max(live[1] - a, 0):] = False
        assert torch.equal(scales[a:b], torch.where(inside, p, 3.0))
        assert torch.equal(codes[a:b, 3], torch.where(inside, 127, 7).to(torch.int8))
        assert torch.equal(codes[a:b, 4], torch.where(inside, 0, 7).to(torch.int8))
        assert torch.equal(x[a:b, 3], torch.where(inside, 127 * p, 9.0).to(dt))
        assert torch.equal(x[a:b, 15], torch.where(inside, 0.0, 9.0).to(dt))
        for n in range(N):
            want = torch.where(inside, 127 * (n + 1) * p, 0.0).to(dt)
            assert torch.equal(y[a:b, n], want), (a, n)


def test_more_rows_than_a_grid_has():
    """Buffers whose tiles no grid covers are refused before anything runs."""
    from combine_get_dispatch_layout_amd import _capi as C
    dev = device()
    M = (1 << 31) - 1
    buf = make_buffer(1, 1, 1, 1)
    x, y = torch.empty(M, 16, device=dev, dtype=torch.int8), torch.empty(M, 8, device=dev, dtype=torch.bfloat16)
    w, ws = torch.zeros(1, 8, 16, device=dev, dtype=torch.int8), torch.ones(1, 8, device=dev)
    rows = torch.zeros(2, dtype=torch.int32, device=dev)
    with pytest.raises(C.MoedxError) as e:
        buf.expert_linear_int8(x, torch.empty(M, device=dev), w, ws, rows, out=y)
    assert e.value.code == C.MOEDX_EINVAL and "grid" in str(e.value)


def test_strided_inputs():
    dev = device()
    E, M, K, N, dt = 3, 20, 32, 24, torch.bfloat16
    buf = make_buffer(E, 1, 1, 1)
    g = torch.Generator(dev).manual_seed(1)
    rows = torch.tensor([0, 7, 7, 20], dtype=torch.int32, device=dev)
    x = torch.randn(M, K, generator=g, device=dev).to(dt)
    d_y = torch.randn(M, N, generator=g, device=dev).to(dt)
    w16 = torch.randn(E, N, K, generator=g, device=dev).to(dt)
    codes, scales, _ = buf.expert_quantize(x, rows, block=128)
    rc, rs, _ = buf.expert_quantize(x, rows)
    w, ws, _ = buf.expert_quantize(w16)
    pre, ps, _ = buf.expert_quantize(torch.randn(M, 2 * N, generator=g, device=dev))
    s = lambda t: torch.stack([t, t], -1)[..., 0]  # noqa: E731
    assert not s(x).is_contiguous()
    pairs = [
        (buf.expert_quantize(s(x), s(rows), block=128)[:2], (codes, scales)),
        (buf.expert_quantize(s(w16))[:2], (w, ws)),
        (buf.expert_dequantize(s(codes), s(scales), s(rows))[:1],
         buf.expert_dequantize(codes, scales, rows)[:1]),
        (buf.expert_linear_int8(s(rc), s(rs), s(w), s(ws), s(rows))[:1],
         buf.expert_linear_int8(rc, rs, w, ws, rows)[:1]),
        (buf.expert_linear_backward_int8(s(d_y), s(codes), s(scales), s(w16), s(rows))[:2],
         buf.expert_linear_backward_int8(d_y, codes, scales, w16, rows)[:2]),
        (buf.expert_swiglu_backward_int8(s(d_y), s(pre), s(ps), s(rows), return_h=True)[:2],
         buf.expert_swiglu_backward_int8(d_y, pre, ps, rows, return_h=True)[:2]),
        (buf.expert_linear_backward(s(d_y), None, s(w16), s(rows))[:1],
         buf.expert_linear_backward(d_y, x, w16, rows)[:1]),
        (buf.expert_linear_backward(s(d_y), s(x), None, s(rows))[1:2],
         buf.expert_linear_backward(d_y, x, w16, rows)[1:2]),
    ]
    for got, want in pairs:
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals():
    """What the library itself refuses, with its message."""
    from combine_get_dispatch_layout_amd import _capi as C
    dev = device()
    E, M, K, N = 4, 10, 32, 40
    buf = make_buffer(E, 1, 1, 1)
    mem = torch.zeros(1 << 16, dtype=torch.uint8, device=dev)
    off = torch.tensor([0, 2, 4, 6, 10], dtype=torch.int32, device=dev)
    at = lambda k: mem.data_ptr() + 4096 * k  # noqa: E731
    ex = C.moedx_exec(stream=torch.cuda.current_stream().cuda_stream)
    x = ctypes.byref(ex)

    def er(rows=M, offsets=True, counts=False):
        return ctypes.byref(C.moedx_expert_rows(off.data_ptr() if offsets else None,
                                                off.data_ptr() if counts else None, rows))

    def quantize(dtype=C.MOEDX_BF16, H=K, block=0, rows=None, xp=at(1), cp=at(2), sp=at(3)):
        return C.moedx_expert_quantize(buf.ctx, xp, dtype, H, block, rows or er(), cp, sp, x)

    def dequantize(dtype=C.MOEDX_BF16, H=K, block=0, rows=None, xp=at(1), cp=at(2), sp=at(3)):
        return C.moedx_expert_dequantize(buf.ctx, cp, sp, H, block, rows or er(), xp, dtype, x)

    def sort(dtype=C.MOEDX_BF16, T=5, k=2, H=K, xp=at(1), rp=at(5), cp=at(2), sp=at(3)):
        return C.moedx_expert_sort_int8(buf.ctx, xp, dtype, T, k, H, rp, cp, sp, x)

    def linear(k=K, n=N, rows=None, swiglu=0, dtype=C.MOEDX_BF16, xp=at(1), xs=at(2), wp=at(3),
               ws=at(6), yp=at(7)):
        return C.moedx_expert_linear_int8(buf.ctx, xp, xs, wp, ws, k, n, rows or er(), swiglu, yp,
                                          dtype, x)

    def backward(k=K, n=N, rows=None, dtype=C.MOEDX_BF16, block=0, dp=at(1), xp=at(2), xs=at(3),
                 wp=at(4), dx=at(7), dw=at(8), dwt=C.MOEDX_BF16):
        return C.moedx_expert_linear_backward_int8(buf.ctx, dp, xp, xs, block, wp, dtype, k, n,
                                                   rows or er(), dx, dw, dwt, x)

    def swiglu(n=N, rows=None, dtype=C.MOEDX_BF16, block=0, dp=at(1), pp=at(2), ps=at(3), op=at(4),
               hp=at(5)):
        return C.moedx_expert_swiglu_backward_int8(buf.ctx, dp, pp, ps, block, dtype, n,
                                                   rows or er(), op, hp, x)

    calls = [quantize, dequantize, sort, linear, backward, swiglu]
    for call in calls:
        assert call() == C.MOEDX_OK, (call.__name__, C.last_error())
    torch.cuda.synchronize()
    null = {"rows": None}  # noqa: F841
    bad = []
    for call in (quantize, dequantize):
        bad += [lambda c=call, v=v: c(H=v) for v in (0, 8, 24, 33, -16, (1 << 20) + 16)]
        bad += [lambda c=call, v=v: c(block=v) for v in (1, 64, 256, -128)]
        bad += [lambda c=call, v=v: c(dtype=v) for v in (3, -1)]
        bad += [lambda c=call, v=v: c(rows=er(v)) for v in (-1, 1 << 31)]
        bad += [lambda c=call: c(rows=er(offsets=True, counts=True)),
                lambda c=call: c(rows=er(9, False, True)), lambda c=call: c(xp=None),
                lambda c=call: c(cp=None), lambda c=call: c(sp=None), lambda c=call: c(xp=at(1) + 8),
                lambda c=call: c(cp=at(2) + 8), lambda c=call: c(sp=at(3) + 2)]
    bad += [lambda v=v: sort(H=v) for v in (0, 8, 24)]
    bad += [lambda v=v: sort(k=v) for v in (0, 17)]
    bad += [lambda: sort(T=-1), lambda: sort(T=1 << 26), lambda: sort(dtype=3), lambda: sort(xp=None),
            lambda: sort(rp=None), lambda: sort(cp=None), lambda: sort(sp=None),
            lambda: sort(cp=at(2) + 8), lambda: sort(rp=at(5) + 2), lambda: sort(sp=at(3) + 2)]
    bad += [lambda v=v: linear(k=v) for v in (0, 8, 24, (1 << 17), (1 << 20))]
    bad += [lambda v=v: linear(n=v) for v in (0, 4, 12, (1 << 20) + 8)]
    bad += [lambda v=v: linear(dtype=v) for v in (C.MOEDX_F32, 3)]
    bad += [lambda: linear(swiglu=2), lambda: linear(rows=er(offsets=False)), lambda: linear(xp=None),
            lambda: linear(xs=None), lambda: linear(wp=None), lambda: linear(ws=None),
            lambda: linear(yp=None), lambda: linear(k=1 << 16, n=1 << 16),
            lambda: linear(ws=at(6) + 4), lambda: linear(xp=at(1) + 8), lambda: linear(xs=at(2) + 2),
            lambda: linear(yp=at(7) + 8), lambda: linear(wp=at(3) + 8)]
    bad += [lambda v=v: backward(k=v) for v in (0, 8, 24)] + [lambda: backward(n=12)]
    bad += [lambda: backward(block=64), lambda: backward(dtype=C.MOEDX_F32),
            lambda: backward(dwt=C.MOEDX_F16), lambda: backward(dx=None, dw=None),
            lambda: backward(xp=None), lambda: backward(xs=None), lambda: backward(wp=None),
            lambda: backward(dp=None), lambda: backward(rows=er(offsets=False)),
            lambda: backward(dx=at(7) + 8), lambda: backward(xs=at(3) + 2)]
    bad += [lambda: swiglu(n=12), lambda: swiglu(n=(1 << 19) + 8), lambda: swiglu(block=32),
            lambda: swiglu(dtype=C.MOEDX_F32), lambda: swiglu(dp=None), lambda: swiglu(pp=None),
            lambda: swiglu(ps=None), lambda: swiglu(op=None), lambda: swiglu(hp=at(5) + 8),
            lambda: swiglu(rows=er(offsets=False))]
    for i, f in enumerate(bad):
        assert f() == C.MOEDX_EINVAL and C.last_error(), i
    # left out, as documented
    assert backward(dw=None, xp=None, xs=None) == C.MOEDX_OK
    assert backward(dx=None, wp=None) == C.MOEDX_OK
    assert swiglu(hp=None) == C.MOEDX_OK
    assert quantize(rows=er(offsets=False)) == C.MOEDX_OK
    assert dequantize(rows=er(offsets=False)) == C.MOEDX_OK
    torch.cuda.synchronize()
