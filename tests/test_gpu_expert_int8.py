"""The experts' rows in int8 (expert_quantize, expert_sort_int8,
expert_dequantize, expert_linear_int8 and the backward calls from saved rows).

Codes, scales, restored values and products without an activation are defined to
the last bit: they are compared with the definition in IEEE fp32 on the CPU (a
product's sum is an integer below 2^31, which fp64 holds exactly).  Activations
and gradients are compared with fp64; the tolerances are those of
test_gpu_expert_linear.py, from the restored values."""

import ctypes

import pytest
import torch

from tests.gpu_common import device, make_buffer
from tests.test_gpu_expert_linear import V, check, spans

pytestmark = pytest.mark.gpu

FLOOR = 2.0 ** -100
TYPES = [torch.bfloat16, torch.float16, torch.float32]
PRODUCTS = TYPES[:2]
name = lambda d: str(d)[6:]  # noqa: E731


def quantized(x, block):
    """The definition: (codes, scales) of x [n, H] in fp32 on the CPU."""
    f = x.detach().cpu().float()
    n, H = f.shape
    width = block or H
    groups = (H + width - 1) // width
    f = torch.nn.functional.pad(f, (0, groups * width - H)).view(n, groups, width)
    m = torch.clamp_min(f.abs().amax(-1), FLOOR)
    top = torch.full_like(m, 127.0)
    codes = torch.round(f * (top / m)[..., None]).view(n, groups * width)[:, :H]
    scales = m / top
    return codes.to(torch.int8), scales[:, 0] if block == 0 else scales


def values(codes, scales):
    """code * scale in fp32, of rows [..., H] with a scale per row or per 128."""
    if scales.dim() == codes.dim() - 1:
        return codes.float() * scales[..., None]
    return codes.float() * scales.repeat_interleave(128, -1)[..., :codes.shape[-1]]


def rows_of(n, H, dt, dev, seed):
    g = torch.Generator(dev).manual_seed(seed)
    x = torch.randn(n, H, generator=g, device=dev)
    x *= torch.exp(3 * torch.randn(n, 1, generator=g, device=dev))
    return x.to(dt)


WIDTHS = [16, 32, 112, 128, 144, 512, 528, 1040, 2064, 4112, 7168, 8192, 8208, 20496]


@pytest.mark.parametrize("dt", TYPES, ids=name)
@pytest.mark.parametrize("block", [0, 128])
@pytest.mark.parametrize("H", WIDTHS)
def test_quantize_and_back(H, block, dt):
    dev = device()
    counts = [3, 0, 130, 1]
    buf = make_buffer(4, 1, 1, 1)
    off = spans(counts, gap=2)
    M, a, b = off[-1] + 3, off[0], off[-1]
    x = rows_of(M, H, dt, dev, 1)
    x[a] = 0
    x[a + 1, 1:] = 0
    x[:a], x[b:] = float("nan"), float("inf")
    rows = torch.tensor(off, dtype=torch.int32, device=dev)
    shape = (M,) if block == 0 else (M, (H + 127) // 128)
    print(f"[int8] quantize H={H} block={block} {dt}", flush=True)
    codes, scales, _ = buf.expert_quantize(
        x, rows, block=block, out=torch.full((M, H), 77, dtype=torch.int8, device=dev),
        scales=torch.full(shape, 7.0, device=dev))
    want_c, want_s = quantized(x[a:b], block)
    assert torch.equal(codes[a:b].cpu(), want_c) and torch.equal(scales[a:b].cpu(), want_s)
    for outside in (slice(0, a), slice(b, M)):
        assert (codes[outside] == 77).all() and (scales[outside] == 7.0).all()
    for to in TYPES:
        back, _ = buf.expert_dequantize(codes, scales, rows, dtype=to,
                                        out=torch.full((M, H), 5.0, dtype=to, device=dev))
        assert torch.equal(back[a:b].cpu(), values(want_c, want_s).to(to))
        assert (back[:a] == 5.0).all() and (back[b:] == 5.0).all()
    # every row, and new outputs
    codes2, scales2, _ = buf.expert_quantize(x[a:b].contiguous(), block=block)
    assert torch.equal(codes2, codes[a:b]) and torch.equal(scales2, scales[a:b])
    back2, _ = buf.expert_dequantize(codes2, scales2)
    assert torch.equal(back2.cpu(), values(want_c, want_s).to(torch.bfloat16))
    # half a scale, and the roundings of the scale, its inverse and three products
    f = x[a:b].double().cpu()
    off_by = (values(want_c, want_s).double() - f).abs()
    each = values(torch.ones_like(want_c), want_s).double()
    assert (off_by <= each * (0.5 + 127 * 4 * 2.0 ** -24)).all()


@pytest.mark.parametrize("dt", TYPES, ids=name)
@pytest.mark.parametrize("block", [0, 128])
def test_extremes(block, dt):
    """Groups of zeros, the smallest and largest values, and inf or NaN, which
    stay in their group."""
    dev = device()
    buf = make_buffer(1, 1, 1, 1)
    H = 272
    info = torch.finfo(dt)
    x = torch.zeros(9, H, dtype=dt, device=dev)
    x[1, ::2], x[1, 1::2] = info.max, -info.max
    x[2, 3] = info.smallest_normal
    x[3, 5] = info.smallest_normal * 2 ** -4 if dt != torch.float16 else 2.0 ** -24
    x[4] = torch.linspace(-1, 1, H, device=dev).to(dt)
    x[5] = x[4]
    x[5, 200] = float("inf")
    x[6] = x[4]
    x[6, 7] = float("nan")
    x[7] = x[4]
    x[7, 130] = float("-inf")
    x[8, 0] = 2.0 ** -20
    codes, scales, _ = buf.expert_quantize(x, block=block)
    back, _ = buf.expert_dequantize(codes, scales, dtype=torch.float32)
    fine = [0, 1, 2, 3, 4, 8]
    want_c, want_s = quantized(x[fine], block)
    assert torch.equal(codes[fine].cpu(), want_c) and torch.equal(scales[fine].cpu(), want_s)
    width = block or H
    for row, at in ((5, 200), (6, 7), (7, 130)):
        bad = torch.zeros(H, dtype=torch.bool, device=dev)
        bad[at // width * width:(at // width + 1) * width] = True
        assert torch.isnan(back[row][bad]).all(), row
        others = buf.expert_dequantize(codes[4:5], scales[4:5], dtype=torch.float32)[0][0]
        assert torch.equal(back[row][~bad], others[~bad]), row
    # such rows make their own outputs NaN, and no other row's
    if block == 0:
        w = torch.randint(-127, 128, (1, 24, H), device=dev, dtype=torch.int8)
        y, _ = buf.expert_linear_int8(codes, scales, w, torch.ones(1, 24, device=dev),
                                      torch.tensor([0, 9], dtype=torch.int32, device=dev))
        assert torch.isnan(y[5:8]).all() and torch.isfinite(y[[0, 2, 3, 4, 8]]).all()


def test_quantize_slots():
    """[E, cap, H] buffers with counts; counts outside [0, cap] are clamped."""
    dev = device()
    E, cap, H = 5, 7, 144
    counts, held = [7, 0, 3, 16, -4], [7, 0, 3, 7, 0]
    buf = make_buffer(E, 1, 1, 1)
    x = rows_of(E * cap, H, torch.bfloat16, dev, 2).view(E, cap, H)
    n = torch.tensor(counts, dtype=torch.int32, device=dev)
    for block in (0, 128):
        shape = (E, cap) if block == 0 else (E, cap, 2)
        codes, scales, _ = buf.expert_quantize(
            x, n, block=block, out=torch.full((E, cap, H), 77, dtype=torch.int8, device=dev),
            scales=torch.full(shape, 7.0, device=dev))
        back, _ = buf.expert_dequantize(codes, scales, n, dtype=torch.float32,
                                        out=torch.full((E, cap, H), 5.0, device=dev))
        for e in range(E):
            c = held[e]
            assert (codes[e, c:] == 77).all() and (scales[e, c:] == 7.0).all()
            assert (back[e, c:] == 5.0).all()
            want_c, want_s = quantized(x[e, :c], block)
            assert torch.equal(codes[e, :c].cpu(), want_c)
            assert torch.equal(scales[e, :c].cpu(), want_s)
            assert torch.equal(back[e, :c].cpu(), values(want_c, want_s))


@pytest.mark.parametrize("dt", TYPES, ids=name)
@pytest.mark.parametrize("H", [16, 528, 2064, 4112, 7168, 8208])
def test_sort_int8(H, dt):
    dev = device()
    T, K, E = 41, 5, 8
    buf = make_buffer(E, 1, 1, T)
    g = torch.Generator().manual_seed(3)
    idx = torch.stack([torch.randperm(E, generator=g)[:K] for _ in range(T)])
    idx[torch.rand(T, K, generator=g) < 0.2] = -1
    idx[7] = -1
    order, _ = buf.expert_order(idx.to(dev))
    x = rows_of(T, H, dt, dev, 4)
    out = torch.full((T * K, H), 77, dtype=torch.int8, device=dev)
    codes, scales, _ = buf.expert_sort_int8(x, order, out=out,
                                            scales=torch.full((T * K,), 7.0, device=dev))
    n = int(order.expert_offsets[-1])
    want_c, want_s = quantized(x, 0)
    token = order.slot_of_row[:n].cpu().long() // K
    assert torch.equal(codes[:n].cpu(), want_c[token]) and torch.equal(scales[:n].cpu(), want_s[token])
    assert (codes[n:] == 77).all() and (scales[n:] == 7.0).all()
    # the same as quantising sorted rows
    rows, _ = buf.expert_sort(x, order)
    c2, s2, _ = buf.expert_quantize(rows, order)
    assert torch.equal(c2[:n], codes[:n]) and torch.equal(s2[:n], scales[:n])


CASES = [
    # counts per expert, K, N
    ([1], 16, 8),
    ([0, 1, 0, 0], 64, 16),
    ([3, 0, 17, 16, 1, 33], 80, 24),
    ([0, 0, 0], 144, 40),
    ([65, 1, 64, 127], 272, 264),
    ([300, 0, 129, 255, 257, 1], 656, 520),
    ([5] * 16, 1424, 136),
    ([700, 30], 1040, 1032),
    ([2, 2, 1, 0, 3, 1, 1, 6], 7168, 64),
    ([1100], 256, 256),
    ([40, 0, 90, 61, 33, 20, 70, 9], 512, 512),
    ([20, 33, 64, 0, 31, 17], 1040, 72),
    ([16, 31, 1, 47], 4112, 48),
]
# 256 x 256 tiles with 1 to 33 stages of 128 codes
CASES += [([2000, 0, 300, 831, 260, 740, 128], k, 4104) for k in (16, 144, 400, 656, 4112)]
CASES += [([2000, 0, 300, 831, 260, 740, 128], 4112, n) for n in (16, 136, 192, 1032)]
# reductions that workgroups enter at scattered places, in each tile size
CASES += [([2, 1, 0, 17, 3], 8192, 72), ([9, 12, 30], 4096, 136),
          ([60, 70, 0, 55, 61, 90, 33, 64], 4096, 4096)]
# 128 x 128 tiles, two and three stages deep, the weights through the caches and
# past them
CASES += [([256, 100, 0, 300, 280, 511, 256, 200], k, 2056) for k in (16, 272, 1040, 4112)]
CASES += [([60, 70, 0, 129, 61, 90, 33, 64], k, 4104) for k in (16, 272, 4096)]
CASES += [([60, 70, 0, 129, 61, 90, 33, 64] * 2, k, 4104) for k in (80, 4096)]
# a few rows in each expert, about 32 and 64; stages fewer and more than a ring has
CASES += [([33, 40, 0, 64, 38, 65, 36, 30], k, 136) for k in (16, 272, 400, 4096, 7168)]
CASES += [([5, 0, 17, 64, 33, 1] * 11, 400, 1032)]
CASES += [([64, 0, 1, 33, 0, 0, 2, 0, 0, 65, 0, 0, 16, 0, 5, 3] * 4, k, 1032) for k in (16, 272, 400, 8192)]
# 256 x 256 tiles that start at scattered places, more than a workgroup's first
CASES += [([100, 90, 120, 81] * 16, 4096, 1032), ([100, 90, 120, 81] * 16, 112, 1032)]
ids = lambda c: f"{len(c[0])}e{sum(c[0])}r-{c[1]}-{c[2]}"  # noqa: E731


def int8_inputs(counts, K, cols, dev, seed):
    g = torch.Generator(dev).manual_seed(seed)
    off = spans(counts)
    M = off[-1] + 5  # rows behind the last expert's
    x = torch.randint(-128, 128, (M, K), generator=g, device=dev, dtype=torch.int8)
    w = torch.randint(-128, 128, (len(counts), cols, K), generator=g, device=dev, dtype=torch.int8)
    xs = torch.rand(M, generator=g, device=dev) * 0.02
    ws = torch.rand(len(counts), cols, generator=g, device=dev) * K ** -0.5 * 0.02
    return off, M, x, xs, w, ws


def product(x, xs, w, ws):
    """(sum, scaled in fp32): the definition."""
    total = (x.double() @ w.double().t().contiguous()).float()  # exact, then one rounding
    return total * xs[:, None] * ws


@pytest.mark.parametrize("dt", PRODUCTS, ids=name)
@pytest.mark.parametrize("case", CASES, ids=ids)
def test_linear_int8(case, dt):
    counts, K, N = case
    dev = device()
    E = len(counts)
    buf = make_buffer(E, 1, 1, 1)
    off, M, x, xs, w, ws = int8_inputs(counts, K, 2 * N, dev, 5)
    xs[off[-1]:] = float("nan")  # never read into a result
    rows = torch.tensor(off, dtype=torch.int32, device=dev)
    print(f"[int8] linear {case} {dt}", flush=True)
    y, _ = buf.expert_linear_int8(x, xs, w[:, :N].contiguous(), ws[:, :N].contiguous(), rows,
                                  dtype=dt, out=torch.full((M, N), 7.0, dtype=dt, device=dev))
    h, _ = buf.expert_linear_int8(x, xs, w, ws, rows, swiglu=True, dtype=dt,
                                  out=torch.full((M, N), 7.0, dtype=dt, device=dev))
    assert (y[off[-1]:] == 7.0).all() and (h[off[-1]:] == 7.0).all()
    for e in range(E):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        p = product(x[a:b], xs[a:b], w[e], ws[e])
        assert torch.equal(y[a:b], p[:, :N].to(dt))
        g, u = p[:, :N].double(), p[:, N:].double()
        want = g * torch.sigmoid(g) * u
        check("h", h[a:b], want, 8 * V * want.abs(), dt)


@pytest.mark.parametrize("cap", [1, 7, 130])
def test_linear_int8_slots(cap):
    dev = device()
    E, K, N, dt = 5, 144, 40, torch.bfloat16
    counts, held = [cap, 0, min(3, cap), cap + 9, -4], [cap, 0, min(3, cap), cap, 0]
    buf = make_buffer(E, 1, 1, 1)
    _, _, x, xs, w, ws = int8_inputs([cap] * E, K, N, dev, 6)
    x, xs = x[:E * cap].view(E, cap, K), xs[:E * cap].view(E, cap)
    y, _ = buf.expert_linear_int8(x, xs, w, ws, torch.tensor(counts, dtype=torch.int32, device=dev),
                                  out=torch.full((E, cap, N), 7.0, dtype=dt, device=dev))
    for e in range(E):
        c = held[e]
        assert (y[e, c:] == 7.0).all()
        assert torch.equal(y[e, :c], product(x[e, :c], xs[e, :c], w[e], ws[e]).to(dt))


def test_linear_int8_rows_alone():
    """A row's outputs are the same bits in any buffer, by any of the tiles."""
    dev = device()
    E, K, N = 4, 4096, 1032
    buf = make_buffer(E, 1, 1, 1)
    off, M, x, xs, w, ws = int8_inputs([700, 1200, 300, 900], K, N, dev, 7)
    y, _ = buf.expert_linear_int8(x, xs, w, ws, torch.tensor(off, dtype=torch.int32, device=dev))
    for row, e in ((0, 0), (699, 0), (700, 1), (1899, 1), (2100, 2), (3099, 3)):
        for n in (1, 40, 300):
            a = max(off[e], min(row, off[e + 1] - n))
            part = slice(a, min(a + n, off[e + 1]))
            k = part.stop - part.start
            rows = torch.tensor([0] * (e + 1) + [k] * (E - e), dtype=torch.int32, device=dev)
            z, _ = buf.expert_linear_int8(x[part].contiguous(), xs[part].contiguous(), w, ws, rows)
            assert torch.equal(z, y[part])


def test_linear_int8_largest_sums():
    """The longest reduction of the largest codes: 2^31 - 2^18 and its negative."""
    dev = device()
    K, N = (1 << 17) - 16, 16
    buf = make_buffer(1, 1, 1, 1)
    x = torch.full((3, K), -128, dtype=torch.int8, device=dev)
    x[1] = 127
    w = torch.full((1, N, K), -128, dtype=torch.int8, device=dev)
    w[:, 1::2] = 127
    xs, ws = torch.ones(3, device=dev), torch.ones(1, N, device=dev)
    rows = torch.tensor([0, 3], dtype=torch.int32, device=dev)
    y, _ = buf.expert_linear_int8(x, xs, w, ws, rows)
    assert torch.equal(y, product(x, xs, w[0], ws[0]).to(y.dtype))
    from combine_get_dispatch_layout_amd import _capi as C
    with pytest.raises(C.MoedxError, match="2\\^17"):
        buf.expert_linear_int8(torch.zeros(3, K + 16, dtype=torch.int8, device=dev), xs,
                               torch.zeros(1, N, K + 16, dtype=torch.int8, device=dev), ws, rows)


@pytest.mark.parametrize("wide", [False, True], ids=["same", "fp32"])
@pytest.mark.parametrize("dt", PRODUCTS, ids=name)
@pytest.mark.parametrize("block", [0, 128])
@pytest.mark.parametrize("case", CASES, ids=ids)
def test_linear_backward_int8(case, block, dt, wide):
    counts, K, N = case
    dev = device()
    E = len(counts)
    buf = make_buffer(E, 1, 1, 1)
    g = torch.Generator(dev).manual_seed(8)
    off = spans(counts, gap=3)
    M, a0, b0 = off[-1] + 5, off[0], off[-1]
    x = torch.randn(M, K, generator=g, device=dev).to(dt)
    d_y = torch.randn(M, N, generator=g, device=dev).to(dt)
    w = (torch.randn(E, N, K, generator=g, device=dev) * N ** -0.5).to(dt)
    codes, scales, _ = buf.expert_quantize(x, block=block)
    saved = values(codes, scales).to(dt)
    for outside in (slice(0, a0), slice(b0, M)):  # never read into a result
        codes[outside], scales[outside], d_y[outside] = 99, float("nan"), float("inf")
    rows = torch.tensor(off, dtype=torch.int32, device=dev)
    wt = torch.float32 if wide else dt
    print(f"[int8] backward {case} block={block} {dt} {wt}", flush=True)
    d_x, d_w, _ = buf.expert_linear_backward_int8(
        d_y, codes, scales, w, rows, d_w_dtype=wt, out=torch.full((M, K), 7.0, dtype=dt, device=dev))
    none, d_w2, _ = buf.expert_linear_backward_int8(d_y, codes, scales, None, rows,
                                                    d_w=torch.full((E, N, K), 7.0, dtype=wt, device=dev))
    assert none is None and d_w.dtype == wt and torch.equal(d_w, d_w2)
    want_x, _, _ = buf.expert_linear_backward(d_y, saved, w, rows)
    assert torch.equal(d_x[a0:b0], want_x[a0:b0])
    assert (d_x[:a0] == 7.0).all() and (d_x[b0:] == 7.0).all()
    for e in range(E):
        a, b = off[e], off[e + 1]
        if a == b:
            assert (d_w[e] == 0).all()
            continue
        dtr, xs = d_y[a:b].double().t().contiguous(), saved[a:b].double()
        check("d_w", d_w[e], dtr @ xs, (b - a + 1) * V * (dtr.abs() @ xs.abs()), wt)


def test_linear_backward_int8_slots():
    dev = device()
    E, cap, K, N, dt = 5, 130, 144, 136, torch.bfloat16
    counts, held = [cap, 0, 3, cap + 9, -4], [cap, 0, 3, cap, 0]
    buf = make_buffer(E, 1, 1, 1)
    g = torch.Generator(dev).manual_seed(9)
    x = torch.randn(E, cap, K, generator=g, device=dev).to(dt)
    d_y = torch.randn(E, cap, N, generator=g, device=dev).to(dt)
    n = torch.tensor(counts, dtype=torch.int32, device=dev)
    for block in (0, 128):
        codes, scales, _ = buf.expert_quantize(x, block=block)
        saved = values(codes, scales).to(dt)
        for e in range(E):
            scales[e, held[e]:] = float("nan")
        _, d_w, _ = buf.expert_linear_backward_int8(d_y, codes, scales, None, n)
        for e in range(E):
            c = held[e]
            if c == 0:
                assert (d_w[e] == 0).all()
                continue
            dtr, xs = d_y[e, :c].double().t().contiguous(), saved[e, :c].double()
            check("d_w", d_w[e], dtr @ xs, (c + 1) * V * (dtr.abs() @ xs.abs()), dt)


def test_weight_gradient_against_differences():
    """d_w of the loss sum(y * d_y) over y = saved x w^T, by central differences of
    the loss in fp64 (it is linear in w: the step is 1) at some weights."""
    dev = device()
    E, K, N, dt = 3, 144, 40, torch.bfloat16
    counts = [5, 0, 70]
    buf = make_buffer(E, 1, 1, 1)
    g = torch.Generator(dev).manual_seed(21)
    off = spans(counts)
    x = torch.randn(off[-1], K, generator=g, device=dev).to(dt)
    d_y = torch.randn(off[-1], N, generator=g, device=dev).to(dt)
    w = torch.randn(E, N, K, generator=g, device=dev).double()
    rows = torch.tensor(off, dtype=torch.int32, device=dev)
    for block in (0, 128):
        codes, scales, _ = buf.expert_quantize(x, rows, block=block)
        saved = values(codes, scales).to(dt).double()
        _, d_w, _ = buf.expert_linear_backward_int8(d_y, codes, scales, None, rows,
                                                    d_w_dtype=torch.float32)

        def terms(v):
            return torch.cat([saved[off[e]:off[e + 1]] @ v[e].t() for e in range(E)]) * d_y.double()

        # the loss is a sum of n terms, each of a sum of K: fp64 roundings
        noise = 2 ** -52 * K * d_y.numel() * terms(w.abs()).abs().sum().item()
        for e, n, k in ((0, 0, 0), (0, 39, 143), (1, 7, 9), (2, 0, 128), (2, 17, 66), (2, 39, 127)):
            up, down = w.clone(), w.clone()
            up[e, n, k] += 1
            down[e, n, k] -= 1
            diff = (terms(up).sum() - terms(down).sum()) / 2
            a, b = off[e], off[e + 1]
            each = (d_y[a:b, n].double() * saved[a:b, k]).abs().sum()
            check("d_w", d_w[e, n, k].view(1), diff.view(1),
                  ((b - a + 1) * V * each + noise).view(1), torch.float32)


def swiglu_gradients(g, u, d):
    s, s1 = torch.sigmoid(g), torch.sigmoid(-g)
    return torch.cat([d * u * s * (1 + g * s1), d * g * s], 1), g * s * u


@pytest.mark.parametrize("dt", PRODUCTS, ids=name)
@pytest.mark.parametrize("block", [0, 128])
@pytest.mark.parametrize("N", [8, 24, 136, 712, 2056, 4104])
def test_swiglu_backward_int8(N, block, dt):
    dev = device()
    counts = [3, 0, 5, 1]
    buf = make_buffer(4, 1, 1, 1)
    off = spans(counts, gap=1)
    M, a, b = off[-1] + 3, off[0], off[-1]
    g = torch.Generator(dev).manual_seed(10)
    pre = torch.randn(M, 2 * N, generator=g, device=dev) * 4
    pre[a, :4] = torch.tensor([80.0, -80.0, 0.0, -1.2785], device=dev)
    d_h = torch.randn(M, N, generator=g, device=dev).to(dt)
    codes, scales, _ = buf.expert_quantize(pre, block=block)
    rows = torch.tensor(off, dtype=torch.int32, device=dev)
    print(f"[int8] swiglu backward N={N} block={block} {dt}", flush=True)
    sevens = lambda n: torch.full((M, n), 7.0, dtype=dt, device=dev)  # noqa: E731
    d_pre, h, _ = buf.expert_swiglu_backward_int8(d_h, codes, scales, rows, out=sevens(2 * N),
                                                  h=sevens(N))
    only, none, _ = buf.expert_swiglu_backward_int8(d_h, codes, scales, rows)
    assert none is None and torch.equal(only[a:b], d_pre[a:b])
    for outside in (slice(0, a), slice(b, M)):
        assert (d_pre[outside] == 7.0).all() and (h[outside] == 7.0).all()
    p, d = values(codes, scales)[a:b].double(), d_h[a:b].double()
    gg, u = p[:, :N], p[:, N:]
    want, want_h = swiglu_gradients(gg, u, d)
    s = torch.sigmoid(gg)
    # 16 roundings of each term; the two terms of d_gate may cancel
    acc = 16 * V * torch.cat([(d * u * s).abs() * (1 + (gg * (1 - s)).abs()), (d * gg * s).abs()], 1)
    check("d_pre", d_pre[a:b], want, acc, dt)
    check("h", h[a:b], want_h, 8 * V * want_h.abs(), dt)
    # and against differences of the activation in fp64
    step = 1e-5
    f = lambda g_, u_: (g_ * torch.sigmoid(g_) * u_ * d)  # noqa: E731
    diff = torch.cat([f(gg + step, u) - f(gg - step, u), f(gg, u + step) - f(gg, u - step)], 1) / (2 * step)
    check("difference", d_pre[a:b], diff, acc + 1e-8 * (1 + d.abs().max() * p.abs().max()), dt)


def test_no_rows_at_all():
    dev = device()
    E, K, N = 3, 16, 24
    buf = make_buffer(E, 1, 1, 1)
    off = torch.zeros(E + 1, dtype=torch.int32, device=dev)
    x = torch.empty(0, K, device=dev, dtype=torch.bfloat16)
    codes, scales, _ = buf.expert_quantize(x, off)
    c128, s128, _ = buf.expert_quantize(x, block=128)
    assert codes.shape == (0, K) and scales.shape == (0,) and s128.shape == (0, 1)
    assert buf.expert_dequantize(c128, s128)[0].shape == (0, K)
    w, ws, _ = buf.expert_quantize(torch.ones(E, N, K, device=dev))
    assert buf.expert_linear_int8(codes, scales, w, ws, off)[0].shape == (0, N)
    d_y = torch.empty(0, N, device=dev, dtype=torch.bfloat16)
    _, d_w, _ = buf.expert_linear_backward_int8(d_y, codes, scales, None, off)
    assert (d_w == 0).all() and d_w.shape == (E, N, K)
    p, ps, _ = buf.expert_quantize(torch.empty(0, 2 * N, device=dev))
    d_pre, h, _ = buf.expert_swiglu_backward_int8(d_y, p, ps, off, return_h=True)
    assert d_pre.shape == (0, 2 * N) and h.shape == (0, N)
    idx = torch.full((5, 2), -1, dtype=torch.int64, device=dev)
    order, _ = buf.expert_order(idx)
    out = torch.full((10, K), 77, dtype=torch.int8, device=dev)
    codes, scales, _ = buf.expert_sort_int8(torch.ones(5, K, device=dev), order, out=out,
                                            scales=torch.full((10,), 7.0, device=dev))
    assert (codes == 77).all() and (scales == 7.0).all()
    order, _ = buf.expert_order(idx[:0])
    assert buf.expert_sort_int8(torch.ones(0, K, device=dev), order)[0].shape == (0, K)
