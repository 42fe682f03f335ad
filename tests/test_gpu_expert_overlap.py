"""Outputs of the router, expert-order and expert-product calls that overlap
another buffer of the call, and buffers that are not aligned to their type, are
refused; outputs right behind another buffer are not.  All buffers lie in one
allocation of zeros (indexes and offsets of zero are valid), so that every call
stays inside it."""

import ctypes

import pytest
import torch

from tests.gpu_common import device, make_buffer

pytestmark = pytest.mark.gpu

E, T, K, H, N = 8, 600, 2, 16, 24  # more than 1024 slots: the order needs its workspace
SLOTS = T * K


def calls(C, ctx, h, ws):
    """name -> (buffers as (name, bytes, alignment, is an output), the call)"""
    gate = C.moedx_gate(C.MOEDX_GATE_SOFTMAX, 1, 1, 0, 1.0, None)
    ex = C.moedx_exec(stream=torch.cuda.current_stream().cuda_stream)
    x = ctypes.byref(ex)

    def with_bias(p):
        gate.bias = p
        return ctypes.byref(gate)

    def rows(off):
        return ctypes.byref(C.moedx_expert_rows(off, None, SLOTS))

    def slots(cnt):
        return ctypes.byref(C.moedx_expert_rows(None, cnt, SLOTS))

    tokens, sorted_rows = (T * H * 2, 16), (SLOTS * H * 2, 16)
    idx, f32, i32 = (SLOTS * 8, 8), (SLOTS * 4, 4), (SLOTS * 4, 4)
    logits, bias = (T * E * 4, 4), (E * 4, 4)
    off, cnt = ((E + 1) * 4, 4), (E * 4, 4)
    wide, both = (SLOTS * N * 2, 16), (SLOTS * N * 4, 16)
    w, w2, w32 = (E * N * H * 2, 16), (E * 2 * N * H * 2, 16), (E * N * H * 4, 16)

    def b(name, size, out=False):
        return (name, size[0], size[1], out)

    return {
        "gate_topk": ([b("logits", logits), b("bias", bias), b("idx", idx, True),
                       b("weights", f32, True)],
                      lambda l, bi, i, g: C.moedx_gate_topk(ctx, l, C.MOEDX_F32, T, K, with_bias(bi),
                                                            i, g, x)),
        "gate_topk_backward": (
            [b("logits", logits), b("bias", bias), b("idx", idx), b("d_weights", f32),
             b("d_logits", logits, True)],
            lambda l, bi, i, g, d: C.moedx_gate_topk_backward(ctx, l, C.MOEDX_F32, T, K,
                                                              with_bias(bi), i, g, d, x)),
        "expert_order": (
            [b("idx", idx), b("offsets", off, True), b("row_of_slot", i32, True),
             b("slot_of_row", i32, True), b("workspace", (ws, 256), True)],
            lambda i, o, r, s, wk: C.moedx_expert_order(ctx, i, T, K, h, o, r, s, wk, ws, x)),
        "expert_sort": (
            [b("x", tokens), b("row_of_slot", i32), b("rows", sorted_rows, True)],
            lambda v, r, o: C.moedx_expert_sort(ctx, v, C.MOEDX_BF16, T, K, H, r, o, x)),
        "expert_unsort": (
            [b("rows", sorted_rows), b("row_of_slot", i32), b("weights", f32),
             b("out", tokens, True)],
            lambda v, r, g, o: C.moedx_expert_unsort(ctx, v, C.MOEDX_BF16, T, K, H, r, g, o, x)),
        "expert_unsort_backward": (
            [b("d_out", tokens), b("rows", sorted_rows), b("row_of_slot", i32),
             b("slot_of_row", i32), b("weights", f32), b("d_rows", sorted_rows, True),
             b("d_weights", f32, True)],
            lambda d, v, r, s, g, o, dg: C.moedx_expert_unsort_backward(
                ctx, d, v, C.MOEDX_BF16, T, K, H, r, s, g, o, dg, x)),
        "expert_linear": (
            [b("x", sorted_rows), b("w", w2), b("offsets", off), b("y", wide, True),
             b("pre", both, True)],
            lambda v, wp, o, y, p: C.moedx_expert_linear(ctx, v, wp, C.MOEDX_BF16, H, N, rows(o), 1,
                                                         y, p, x)),
        "expert_linear of slots": (
            [b("x", sorted_rows), b("w", w), b("counts", cnt), b("y", wide, True)],
            lambda v, wp, o, y: C.moedx_expert_linear(ctx, v, wp, C.MOEDX_BF16, H, N, slots(o), 0, y,
                                                      None, x)),
        "expert_linear_backward": (
            [b("d_y", wide), b("x", sorted_rows), b("w", w), b("offsets", off),
             b("d_x", sorted_rows, True), b("d_w", w32, True)],
            lambda d, v, wp, o, dx, dw: C.moedx_expert_linear_backward(
                ctx, d, v, wp, C.MOEDX_BF16, H, N, rows(o), dx, dw, C.MOEDX_F32, x)),
        "expert_swiglu_backward": (
            [b("d_h", wide), b("pre", both), b("counts", cnt), b("d_pre", both, True)],
            lambda d, p, o, dp: C.moedx_expert_swiglu_backward(ctx, d, p, C.MOEDX_BF16, N, slots(o),
                                                               dp, x)),
    }


NAMES = ["gate_topk", "gate_topk_backward", "expert_order", "expert_sort", "expert_unsort",
         "expert_unsort_backward", "expert_linear", "expert_linear of slots",
         "expert_linear_backward", "expert_swiglu_backward"]


def up(n, a):
    return (n + a - 1) // a * a


@pytest.fixture(scope="module")
def arena():
    from combine_get_dispatch_layout_amd import _capi as C
    dev = device()
    buf = make_buffer(E, 1, 1, T)
    mem = torch.zeros(4 << 20, dtype=torch.uint8, device=dev)
    ws = ctypes.c_size_t()
    C.check(C.moedx_expert_order_workspace_bytes(buf.ctx, T, K, ctypes.byref(ws)))
    assert ws.value > 0
    return C, buf, mem, ws.value


def place(mem, buffers):
    """Offsets of the buffers, apart from each other, from the middle on."""
    at, out = mem.numel() // 2, []
    for _, n, a, _ in buffers:
        at = up(at, 256)
        out.append(at)
        at += n + 256
    assert at <= mem.numel()
    return out


def runner(arena, name):
    """(the call's buffers, offsets apart from each other, the call at offsets)"""
    C, buf, mem, ws = arena
    buffers, call = calls(C, buf.ctx, None, ws)[name]

    def run(at):
        mem.zero_()
        assert all(0 <= p and p + b[1] <= mem.numel() for p, b in zip(at, buffers))
        rc = call(*[mem.data_ptr() + p for p in at])
        torch.cuda.synchronize()
        return rc

    return buffers, place(mem, buffers), run


@pytest.mark.parametrize("name", NAMES)
def test_overlaps(arena, name):
    C, _, mem, _ = arena
    buffers, apart, run = runner(arena, name)
    assert run(apart) == C.MOEDX_OK, C.last_error()
    for i, (_, n, a, out) in enumerate(buffers):
        for j, (other, m, _, _) in enumerate(buffers):
            if i == j or not out:
                continue
            print(f"[overlap] {name}: {buffers[i][0]} and {other}", flush=True)
            # the output's first bytes on the other's last, its last on the
            # other's first, inside it or around it, and right behind it
            for p in (apart[j] + (m - 1) // a * a, apart[j] - (n - 1) // a * a, apart[j]):
                at = list(apart)
                at[i] = p
                assert run(at) == C.MOEDX_EINVAL and "overlap" in C.last_error(), (other, p)
            at = [mem.numel() // 2 - up(m, 256) - up(n, 256) - 512 if k == j else p
                  for k, p in enumerate(apart)]
            at[i] = up(at[j] + m, a)
            assert run(at) == C.MOEDX_OK, (other, C.last_error())


def test_order_and_its_handle(arena):
    """The order of received rows reads the handle's prefixes: no output on them."""
    C, buf, mem, ws = arena
    dev = device()
    x = torch.zeros(T, H, device=dev, dtype=torch.bfloat16)
    idx = torch.zeros(T, K, dtype=torch.int64, device=dev)
    idx[:, 1] = 1
    _, rti, _, _, handle, _ = buf.dispatch(x, topk_idx=idx, num_worst_tokens=T)
    prefix = handle.tensor(C.MOEDX_T_RANK_PREFIX_MATRIX, torch.int32)
    base = mem.data_ptr()
    buffers, call = calls(C, buf.ctx, handle.ptr, ws)["expert_order"]
    at = [base + p for p in place(mem, buffers)]
    at[0] = rti.data_ptr()
    assert call(*at) == C.MOEDX_OK, C.last_error()
    torch.cuda.synchronize()
    for i in (1, 2, 3):
        bad = list(at)
        bad[i] = prefix.data_ptr()
        assert call(*bad) == C.MOEDX_EINVAL and "overlap" in C.last_error()


def test_empty_buffers_overlap_nothing(arena):
    """No rows: an output of no bytes may lie anywhere."""
    C, buf, mem, _ = arena
    p = mem.data_ptr()
    ex = C.moedx_exec(stream=torch.cuda.current_stream().cuda_stream)
    er = C.moedx_expert_rows(p, None, 0)
    assert C.moedx_expert_linear(buf.ctx, p + 4096, p + 8192, C.MOEDX_BF16, H, N, ctypes.byref(er), 0,
                                 p + 8192 + 16, None, ctypes.byref(ex)) == C.MOEDX_OK
    assert C.moedx_expert_sort(buf.ctx, p, C.MOEDX_BF16, 0, K, H, p, p, ctypes.byref(ex)) == C.MOEDX_OK


@pytest.mark.parametrize("name", NAMES)
def test_alignment(arena, name):
    """A buffer that is not aligned to its type is refused."""
    C = arena[0]
    buffers, apart, run = runner(arena, name)
    for i, (b, _, a, _) in enumerate(buffers):
        at = list(apart)
        at[i] += a // 2
        assert run(at) == C.MOEDX_EINVAL and "aligned" in C.last_error(), b
