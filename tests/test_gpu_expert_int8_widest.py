"""The int8 calls at the widest rows and outputs that moedx.h allows, against the
definitions (tolerances as in test_gpu_expert_int8.py)."""

import pytest
import torch

from tests.gpu_common import device, make_buffer
from tests.test_gpu_expert_int8 import (PRODUCTS, TYPES, name, product, quantized, rows_of,
                                        swiglu_gradients, values)
from tests.test_gpu_expert_linear import V, check

pytestmark = pytest.mark.gpu

WIDEST = 1 << 20


def offsets(*rows):
    return torch.tensor(rows, dtype=torch.int32, device=device())


@pytest.mark.parametrize("dt", TYPES, ids=name)
@pytest.mark.parametrize("block", [0, 128])
def test_widest_rows(block, dt):
    dev = device()
    M, H = 5, WIDEST
    buf = make_buffer(2, 1, 1, 1)
    x = rows_of(M, H, dt, dev, 51)
    rows = offsets(1, 2, 4)
    shape = (M,) if block == 0 else (M, H // 128)
    print(f"[int8] quantize {H} values a row, block={block} {dt}", flush=True)
    codes, scales, _ = buf.expert_quantize(
        x, rows, block=block, out=torch.full((M, H), 77, dtype=torch.int8, device=dev),
        scales=torch.full(shape, 7.0, device=dev))
    want_c, want_s = quantized(x[1:4], block)
    assert torch.equal(codes[1:4].cpu(), want_c) and torch.equal(scales[1:4].cpu(), want_s)
    back, _ = buf.expert_dequantize(codes, scales, rows, dtype=dt,
                                    out=torch.full((M, H), 5.0, dtype=dt, device=dev))
    assert torch.equal(back[1:4].cpu(), values(want_c, want_s).to(dt))
    for v, filled in ((codes, 77), (scales, 7.0), (back, 5.0)):
        assert (v[0] == filled).all() and (v[4] == filled).all()
    if block:
        return
    idx = torch.tensor([[0, 1], [1, -1], [-1, -1], [1, 0], [0, -1]], device=dev)
    order, _ = buf.expert_order(idx)
    sc, ss, _ = buf.expert_sort_int8(x, order)
    n = int(order.expert_offsets[-1])
    token = order.slot_of_row[:n].long().cpu() // 2
    want_c, want_s = quantized(x, 0)
    assert torch.equal(sc[:n].cpu(), want_c[token]) and torch.equal(ss[:n].cpu(), want_s[token])


@pytest.mark.parametrize("dt", PRODUCTS, ids=name)
@pytest.mark.parametrize("block", [0, 128])
def test_widest_activation(block, dt):
    dev = device()
    M, N = 3, WIDEST // 2
    buf = make_buffer(1, 1, 1, 1)
    g = torch.Generator(dev).manual_seed(52)
    codes, scales, _ = buf.expert_quantize(torch.randn(M, 2 * N, generator=g, device=dev) * 4, block=block)
    d_h = torch.randn(M, N, generator=g, device=dev).to(dt)
    print(f"[int8] swiglu backward N={N} block={block} {dt}", flush=True)
    d_pre, h, _ = buf.expert_swiglu_backward_int8(d_h, codes, scales, offsets(0, M), return_h=True)
    p, d = values(codes, scales).double(), d_h.double()
    gate, u = p[:, :N], p[:, N:]
    want, want_h = swiglu_gradients(gate, u, d)
    s = torch.sigmoid(gate)
    acc = 16 * V * torch.cat([(d * u * s).abs() * (1 + (gate * (1 - s)).abs()), (d * gate * s).abs()], 1)
    check("d_pre", d_pre, want, acc, dt)
    check("h", h, want_h, 8 * V * want_h.abs(), dt)


@pytest.mark.parametrize("counts", [[0, 1], [3, 70], [0, 300]], ids=str)
def test_most_outputs(counts):
    dev = device()
    N, K, dt = WIDEST, 16, torch.bfloat16
    buf = make_buffer(2, 1, 1, 1)
    g = torch.Generator(dev).manual_seed(53)
    M = sum(counts) + 1
    x = torch.randint(-128, 128, (M, K), generator=g, device=dev, dtype=torch.int8)
    w = torch.randint(-128, 128, (2, 2 * N, K), generator=g, device=dev, dtype=torch.int8)
    xs, ws = torch.rand(M, generator=g, device=dev) * 0.02, torch.rand(2, 2 * N, generator=g, device=dev) * 0.02
    rows = offsets(0, counts[0], sum(counts))
    for gated in (False, True):
        print(f"[int8] {N} outputs, rows {counts}, gated={gated}", flush=True)
        wv, wsv = (w, ws) if gated else (w[:, :N].contiguous(), ws[:, :N].contiguous())
        y, _ = buf.expert_linear_int8(x, xs, wv, wsv, rows, swiglu=gated,
                                      out=torch.full((M, N), 7.0, dtype=dt, device=dev))
        assert (y[-1] == 7.0).all()
        for e, (a, b) in enumerate(((0, counts[0]), (counts[0], sum(counts)))):
            for m in {a, (a + b) // 2, b - 1} if b > a else ():
                p = product(x[m:m + 1], xs[m:m + 1], wv[e], wsv[e])
                if not gated:
                    assert torch.equal(y[m:m + 1], p.to(dt)), m
                    continue
                gate, u = p[:, :N].double(), p[:, N:].double()
                want = gate * torch.sigmoid(gate) * u
                check("h", y[m:m + 1], want, 8 * V * want.abs(), dt)


@pytest.mark.parametrize("wide", [False, True], ids=["same", "fp32"])
@pytest.mark.parametrize("block", [0, 128])
def test_widest_weight_gradient(block, wide):
    dev = device()
    K, N, dt = WIDEST, 24, torch.bfloat16
    counts = [37, 0, 66]
    buf = make_buffer(3, 1, 1, 1)
    g = torch.Generator(dev).manual_seed(54)
    M = sum(counts)
    x = torch.randn(M, K, generator=g, device=dev).to(dt)
    d_y = torch.randn(M, N, generator=g, device=dev).to(dt)
    codes, scales, _ = buf.expert_quantize(x, block=block)
    wt = torch.float32 if wide else dt
    print(f"[int8] weight gradient of {K} columns, block={block} {wt}", flush=True)
    _, d_w, _ = buf.expert_linear_backward_int8(d_y, codes, scales, None, offsets(0, 37, 37, M),
                                                d_w_dtype=wt)
    saved = values(codes, scales).to(dt)
    assert (d_w[1] == 0).all()
    for e, (a, b) in ((0, (0, 37)), (2, (37, M))):
        dtr, xs = d_y[a:b].double().t().contiguous(), saved[a:b].double()
        check("d_w", d_w[e], dtr @ xs, (b - a + 1) * V * (dtr.abs() @ xs.abs()), wt)
