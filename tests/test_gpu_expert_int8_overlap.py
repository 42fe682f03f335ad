"""Outputs of the int8 calls that overlap another buffer of the call, and buffers
that are not aligned, are refused; outputs right behind another buffer are not.
All buffers lie in one allocation of zeros, so that every call stays inside it."""

import ctypes

import pytest
import torch

from tests.gpu_common import device, make_buffer
from tests.test_gpu_expert_overlap import place, up

pytestmark = pytest.mark.gpu

E, T, K, H, N = 8, 600, 2, 32, 24
SLOTS = T * K


def calls(C, ctx):
    """name -> (buffers as (name, bytes, alignment, is an output), the call)"""
    ex = C.moedx_exec(stream=torch.cuda.current_stream().cuda_stream)
    x = ctypes.byref(ex)

    def rows(off):
        return ctypes.byref(C.moedx_expert_rows(off, None, SLOTS))

    def slots(cnt):
        return ctypes.byref(C.moedx_expert_rows(None, cnt, SLOTS))

    tokens, rows16, codes = (T * H * 2, 16), (SLOTS * H * 2, 16), (SLOTS * H, 16)
    one, off, cnt = (SLOTS * 4, 4), ((E + 1) * 4, 4), (E * 4, 4)
    outs, both, pre = (SLOTS * N * 2, 16), (SLOTS * N * 4, 16), (SLOTS * 2 * N, 16)
    w, ws = (E * 2 * N * H, 16), (E * 2 * N * 4, 16)
    w16, dw = (E * N * H * 2, 16), (E * N * H * 4, 16)

    def b(name, size, out=False):
        return (name, size[0], size[1], out)

    return {
        "quantize": ([b("x", rows16), b("offsets", off), b("codes", codes, True), b("scales", one, True)],
                     lambda v, o, c, s: C.moedx_expert_quantize(ctx, v, C.MOEDX_BF16, H, 128, rows(o),
                                                                c, s, x)),
        "quantize all": ([b("x", rows16), b("codes", codes, True), b("scales", one, True)],
                         lambda v, c, s: C.moedx_expert_quantize(ctx, v, C.MOEDX_F16, H, 0, rows(None),
                                                                 c, s, x)),
        "dequantize": ([b("codes", codes), b("scales", one), b("counts", cnt), b("x", rows16, True)],
                       lambda c, s, n, v: C.moedx_expert_dequantize(ctx, c, s, H, 0, slots(n), v,
                                                                    C.MOEDX_BF16, x)),
        "sort": ([b("x", tokens), b("row_of_slot", one), b("codes", codes, True), b("scales", one, True)],
                 lambda v, r, c, s: C.moedx_expert_sort_int8(ctx, v, C.MOEDX_BF16, T, K, H, r, c, s, x)),
        "linear": ([b("x", codes), b("x_scales", one), b("w", w), b("w_scales", ws), b("offsets", off),
                    b("y", outs, True)],
                   lambda v, s, wp, wsp, o, y: C.moedx_expert_linear_int8(
                       ctx, v, s, wp, wsp, H, N, rows(o), 1, y, C.MOEDX_BF16, x)),
        "linear_backward": ([b("d_y", outs), b("x", codes), b("x_scales", one), b("w", w16),
                             b("counts", cnt), b("d_x", rows16, True), b("d_w", dw, True)],
                            lambda d, v, s, wp, n, dx, dwp: C.moedx_expert_linear_backward_int8(
                                ctx, d, v, s, 128, wp, C.MOEDX_BF16, H, N, slots(n), dx, dwp,
                                C.MOEDX_F32, x)),
        "swiglu_backward": ([b("d_h", outs), b("pre", pre), b("pre_scales", one), b("offsets", off),
                             b("d_pre", both, True), b("h", outs, True)],
                            lambda d, p, s, o, dp, h: C.moedx_expert_swiglu_backward_int8(
                                ctx, d, p, s, 0, C.MOEDX_BF16, N, rows(o), dp, h, x)),
    }


NAMES = ["quantize", "quantize all", "dequantize", "sort", "linear", "linear_backward",
         "swiglu_backward"]


@pytest.fixture(scope="module")
def arena():
    from combine_get_dispatch_layout_amd import _capi as C
    dev = device()
    return C, make_buffer(E, 1, 1, T), torch.zeros(4 << 20, dtype=torch.uint8, device=dev)


def runner(arena, name):
    C, buf, mem = arena
    buffers, call = calls(C, buf.ctx)[name]

    def run(at):
        mem.zero_()
        assert all(0 <= p and p + b[1] <= mem.numel() for p, b in zip(at, buffers))
        rc = call(*[mem.data_ptr() + p for p in at])
        torch.cuda.synchronize()
        return rc

    return buffers, place(mem, buffers), run


@pytest.mark.parametrize("name", NAMES)
def test_overlaps(arena, name):
    C, _, mem = arena
    buffers, apart, run = runner(arena, name)
    assert run(apart) == C.MOEDX_OK, C.last_error()
    for i, (_, n, a, out) in enumerate(buffers):
        for j, (other, m, _, _) in enumerate(buffers):
            if i == j or not out:
                continue
            print(f"[overlap] int8 {name}: {buffers[i][0]} and {other}", flush=True)
            for p in (apart[j] + (m - 1) // a * a, apart[j] - (n - 1) // a * a, apart[j]):
                at = list(apart)
                at[i] = p
                assert run(at) == C.MOEDX_EINVAL and "overlap" in C.last_error(), (other, p)
            at = [mem.numel() // 2 - up(m, 256) - up(n, 256) - 512 if k == j else p
                  for k, p in enumerate(apart)]
            at[i] = up(at[j] + m, a)
            assert run(at) == C.MOEDX_OK, (other, C.last_error())


@pytest.mark.parametrize("name", NAMES)
def test_alignment(arena, name):
    C = arena[0]
    buffers, apart, run = runner(arena, name)
    for i, (b, _, a, _) in enumerate(buffers):
        at = list(apart)
        at[i] += a // 2
        assert run(at) == C.MOEDX_EINVAL and "aligned" in C.last_error(), b
