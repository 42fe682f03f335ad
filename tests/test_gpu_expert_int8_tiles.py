"""expert_linear_int8 by each of its kernels whose workgroups go through several
tiles (int8_tile_cases.py): with and without an activation, in both types, over
one reduction stage and many, of 64 and 256 experts; captured and replayed with
other rows in each expert, and on two streams at once.

Products are compared with the definition for equality, activations with fp64
(the tolerance of test_gpu_expert_int8.py)."""

import pytest
import torch

from tests.gpu_common import device, make_buffer
from tests.int8_tile_cases import CASES, CHANGING
from tests.test_gpu_expert_int8 import PRODUCTS, product
from tests.test_gpu_expert_linear import V, check, spans

pytestmark = pytest.mark.gpu


def codes(shape, g, dev):
    return torch.randint(-128, 128, shape, generator=g, device=dev, dtype=torch.int8)


def layout(counts, cap, M):
    """(rows argument, first row of each expert, which of the M rows are live)."""
    first = [e * cap for e in range(len(counts))] if cap else spans(counts)[:-1]
    rows = torch.tensor(counts if cap else spans(counts), dtype=torch.int32, device=device())
    live = torch.zeros(M, dtype=torch.bool, device=device())
    for a, c in zip(first, counts):
        live[a:a + c] = True
    return rows, first, live


@pytest.mark.parametrize("case", CASES, ids=repr)
def test_several_tiles(case):
    dev = device()
    E, K, outs, M = case.E, case.K, case.outs, case.rows
    buf = make_buffer(E, 1, 1, 1)
    g = torch.Generator(dev).manual_seed(41)
    rows, first, live = layout(case.counts, case.cap, M)
    x, w = codes((M, K), g, dev), codes((E, outs, K), g, dev)
    xs = torch.rand(M, generator=g, device=dev) * 0.02
    xs[~live] = float("nan")  # never read into a result
    ws = torch.rand(E, outs, generator=g, device=dev) * K ** -0.5 * 0.02
    lead = (E, case.cap) if case.cap else (M,)
    got = {}
    for dt in PRODUCTS:
        for gated in (False, True):
            N = outs // 2 if gated else outs
            print(f"[int8] {case} {dt} gated={gated}", flush=True)
            y, _ = buf.expert_linear_int8(
                x.view(*lead, K), xs.view(lead), w, ws, rows, swiglu=gated, dtype=dt,
                out=torch.full((*lead, N), 7.0, dtype=dt, device=dev))
            got[dt, gated] = y.view(M, N)
            assert (got[dt, gated][~live] == 7.0).all()
    for e in range(E):
        a, b = first[e], first[e] + case.counts[e]
        if a == b:
            continue
        p = product(x[a:b], xs[a:b], w[e], ws[e])
        gate, up = p[:, :outs // 2].double(), p[:, outs // 2:].double()
        h = gate * torch.sigmoid(gate) * up
        for dt in PRODUCTS:
            assert torch.equal(got[dt, False][a:b], p.to(dt)), (e, dt)
            check("h", got[dt, True][a:b], h, 8 * V * h.abs(), dt)


@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("case", CHANGING, ids=lambda c: f"{c[0]}-{c[1]}-{c[2]}")
def test_several_tiles_captured_and_at_once(case, gated):
    """Each replay finds other rows in each expert, also none at all; two streams take
    several tiles to a workgroup at the same time."""
    dev = device()
    kind, cap, outs, M, counts = case
    E, K = len(counts[0]), 272
    N = outs // 2 if gated else outs
    buf = make_buffer(E, 1, 1, 1)
    g = torch.Generator(dev).manual_seed(43)
    x, w = codes((M, K), g, dev), codes((E, outs, K), g, dev)
    xs = torch.rand(M, generator=g, device=dev) * 0.01
    ws = torch.rand(E, outs, generator=g, device=dev) * 0.01
    lead = (E, cap) if cap else (M,)
    sevens = lambda: torch.full((*lead, N), 7.0, dtype=torch.bfloat16, device=dev)  # noqa: E731

    def call(rows, out):
        return buf.expert_linear_int8(x.view(*lead, K), xs.view(lead), w, ws, rows, swiglu=gated,
                                      out=out, no_sync=True)[0]

    rows, want = [], []
    for v in counts:
        r, first, live = layout(v, cap, M)
        print(f"[int8] {kind} {sum(v)} rows gated={gated}", flush=True)
        y = call(r, sevens())
        flat = y.view(M, N)
        assert (flat[~live] == 7.0).all()
        for e, c in enumerate(v if not gated else []):
            a = first[e]
            assert torch.equal(flat[a:a + c], product(x[a:a + c], xs[a:a + c], w[e], ws[e]).to(y.dtype))
        rows.append(r)
        want.append(y)
    held, y = rows[0].clone(), sevens()
    graph = torch.cuda.CUDAGraph()
    call(held, y)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call(held, y)
    for turn in range(2):
        for r, expected in zip(rows, want):
            held.copy_(r)
            y.fill_(7.0)
            print(f"[graph] int8 {kind} turn {turn}", flush=True)
            graph.replay()
            assert torch.equal(y, expected)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs_of = [[sevens() for _ in rows] for _ in streams]
    torch.cuda.synchronize()
    for i in range(len(rows)):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                call(rows[(i + k) % len(rows)], outs_of[k][i])
    torch.cuda.synchronize()
    for i in range(len(rows)):
        for k in range(2):
            assert torch.equal(outs_of[k][i], want[(i + k) % len(rows)])
