"""The experts' rows in 8 bits, as cases that can be timed: int8 products with
a scale per row and per weight row (expert_sort_int8, expert_quantize,
expert_linear_int8), and saved rows in int8 with their use in the backward pass
(expert_quantize, expert_dequantize, expert_swiglu_backward_int8,
expert_linear_backward_int8).

``run`` computes a case in plain torch while ``own`` is false, and with the
library's calls, as a user's program makes them, while it is true.

A group of values (a row, or 128 values of it) is held as codes and a scale:
m = max(largest magnitude, 2^-100), scale = m / 127, code = x * (127 / m) to
nearest even, in fp32.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
FLOOR = 2.0 ** -100


# ---- cases --------------------------------------------------------------------

def listed():
    """Widths, expert counts and top-k are those of the package's workloads
    (128 x 256, decode 128 x 7168, prefill 4096 x 7168, reuse 16384 x 4096);
    the experts' inner widths are generic."""
    return [
        # A small batch from its routing to its experts' first product: order,
        # rows sorted and quantised, product. The smallest call, latency counts.
        dict(name="serve_tiny", op="serve", T=128, E=16, K=2, Kd=256, N=256, dtype="bf16", routing="uniform",
             empty=0.0, swiglu=False),
        # A prefill's rows the same way, with the gated activation: the largest.
        dict(name="serve_prefill", op="serve", T=4096, E=64, K=8, Kd=7168, N=2048, dtype="bf16",
             routing="uniform", empty=0.0, swiglu=True),
        # One token's experts: eight experts' weights are read once, in 8 bits.
        dict(name="product_one_token", op="product", T=1, E=64, K=8, Kd=7168, N=2048, dtype="bf16",
             routing="uniform", empty=0.0, swiglu=True),
        # A decode batch in the low-latency layout ([E, cap, Kd] slots with counts).
        dict(name="product_decode", op="product_slots", T=128, E=64, K=6, Kd=4096, N=2048, cap=128, dtype="bf16",
             routing="uniform", empty=0.0, swiglu=True),
        # A skewed batch's second product, half precision, odd sizes.
        dict(name="product_skewed", op="product", T=2047, E=64, K=6, Kd=1424, N=4096, dtype="f16",
             routing="zipf", empty=0.05, swiglu=False),
        # Saving and restoring the rows of a small training batch, one scale per row.
        dict(name="saved_small", op="saved", T=128, E=16, K=2, H=256, block=0, dtype="bf16", routing="uniform",
             empty=0.0),
        # The same for the (gate, up) values of a long one, a scale per 128 values.
        dict(name="saved_long", op="saved", T=8191, E=64, K=6, H=4096, block=128, dtype="bf16",
             routing="uniform", empty=0.0),
        # The activation's gradient from saved (gate, up) values, with its output
        # computed again for the next weight gradient: the same training step.
        dict(name="act_grad_long", op="act_grad", T=8191, E=64, K=6, N=2048, block=128, dtype="bf16",
             routing="uniform", empty=0.0),
        # A short odd batch of it in half precision, a scale per row.
        dict(name="act_grad_odd", op="act_grad", T=333, E=12, K=3, N=712, block=0, dtype="f16", routing="zipf",
             empty=0.05),
        # The weight gradient from saved rows: the same training step.
        dict(name="w_grad_long", op="w_grad", T=8192, E=64, K=6, Kd=4096, N=2048, block=128, dtype="bf16",
             wide=False, routing="uniform", empty=0.0),
        # A skewed one, half precision, odd sizes, gradients in fp32.
        dict(name="w_grad_skewed", op="w_grad", T=2047, E=64, K=6, Kd=1424, N=1032, block=0, dtype="f16",
             wide=True, routing="zipf", empty=0.05),
    ]


def draw(rng):
    def log(lo, hi, step=1):
        v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
        return max(lo, min(hi, int(v) // step * step))

    op = rng.choice(["serve", "serve", "product", "product", "product_slots", "saved", "act_grad", "w_grad", "w_grad"])
    E = rng.choice([8, 12, 16, 32, 64])
    case = dict(op=op, T=log(1, 4096), E=E, K=rng.randint(1, 8), dtype=rng.choice(["bf16", "bf16", "f16"]),
                routing=rng.choice(["uniform", "zipf"]), empty=rng.choice([0.0, 0.05, 0.5]))
    if op in ("serve", "product", "product_slots"):
        case.update(Kd=log(64, 7168, 16), N=log(64, 2048, 8), swiglu=rng.random() < 0.5)
        if op == "product_slots":
            case["T"] = log(1, 256)
            case["cap"] = case["T"] + rng.randint(0, 64)
        return case
    case["block"] = rng.choice([0, 128])
    case["T"] = log(1, 8191)
    case["K"] = min(case["K"], 6)
    if op == "saved":
        case.update(dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), H=log(64, 4096, 16))
    elif op == "act_grad":
        case.update(N=log(64, 2048, 8))
    else:
        case.update(Kd=log(64, 4096, 16), N=log(64, 2048, 8), wide=rng.random() < 0.5)
    return case


# ---- inputs -------------------------------------------------------------------

def _route(g, case, dev):
    """topk_idx [T, K] int64: distinct experts of a token, some slots empty."""
    T, E, K = case["T"], case["E"], case["K"]
    noise = torch.rand(T, E, generator=g, device=dev, dtype=torch.float64).clamp(1e-12, 1 - 1e-12)
    noise = -torch.log(-torch.log(noise))
    if case["routing"] == "zipf":  # expert e drawn with weight (e + 1)^-1.2
        noise = noise - 1.2 * torch.log(torch.arange(1, E + 1, device=dev, dtype=torch.float64))
    idx = torch.topk(noise, K, dim=1).indices
    if case["empty"] > 0:
        idx = torch.where(torch.rand(T, K, generator=g, device=dev) < case["empty"], -1, idx)
    return idx.contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(dev)
    g.manual_seed(seed)
    op, T, E, K = case["op"], case["T"], case["E"], case["K"]
    dt = DTYPES[case["dtype"]]

    def randn(*shape, scale=1.0, dtype=dt):
        return torch.randn(*shape, generator=g, device=dev, dtype=dtype).mul_(scale)

    def activations(*shape, dtype=dt):
        """Rows of different sizes with a few columns that stand out."""
        x = randn(*shape, dtype=dtype)
        x *= torch.exp(randn(*shape[:-1], 1, scale=0.5, dtype=torch.float32)).to(dtype)
        x[..., 5::397] *= 8
        return x

    s = dict(case=case)
    if own:
        from combine_get_dispatch_layout_amd import Buffer
        s["buf"] = Buffer(num_experts=E, num_ranks=1, num_channels=1, max_tokens=max(T, 1))
    idx = _route(g, case, dev)
    flat = idx.reshape(-1)
    by = torch.sort(torch.where(flat >= 0, flat, E)).values
    offsets = torch.searchsorted(by, torch.arange(E + 1, device=dev)).to(torch.int32)
    s["offsets"], s["bounds"] = offsets, offsets.tolist()  # the plain forms go expert by expert
    M = T * K
    if op == "saved":
        s["x"] = activations(M, case["H"])
        s["codes"] = torch.zeros(M, case["H"], device=dev, dtype=torch.int8)
        s["scales"] = torch.zeros(_scale_shape((M,), case["H"], case["block"]), device=dev)
        s["out"] = torch.zeros_like(s["x"])
        return s
    if op == "act_grad":
        s["codes"], s["scales"] = _quantize(activations(M, 2 * case["N"]), case["block"])
        s["d_h"] = randn(M, case["N"])
        s["out"] = torch.zeros(M, 2 * case["N"], device=dev, dtype=dt)
        s["h"] = torch.zeros(M, case["N"], device=dev, dtype=dt)
        return s
    Kd, N = case["Kd"], case["N"]
    if op == "w_grad":
        s["codes"], s["scales"] = _quantize(activations(M, Kd), case["block"])
        s["d_y"] = randn(M, N)
        s["wide"] = torch.float32 if case["wide"] else dt
        return s
    # the weights of a model in 8 bits: quantised once, a scale per output
    cols = 2 * N if case["swiglu"] else N
    s["w"] = torch.empty(E, cols, Kd, device=dev, dtype=torch.int8)
    s["w_scales"] = torch.empty(E, cols, device=dev)
    for e in range(E):
        s["w"][e], s["w_scales"][e] = _quantize(randn(cols, Kd, scale=Kd ** -0.5), 0)
    if op == "product_slots":
        s["counts"] = (offsets[1:] - offsets[:-1]).contiguous()
        s["x"] = activations(E, case["cap"], Kd)
        s["out"] = torch.zeros(E, case["cap"], N, device=dev, dtype=dt)
        return s
    s["out"] = torch.zeros(M, N, device=dev, dtype=dt)
    if op == "serve":
        s["topk_idx"] = idx
        s["x"] = activations(T, Kd)
    else:
        s["x"] = activations(M, Kd)
    return s


# ---- one pass -----------------------------------------------------------------

def run(state):
    if own:
        return _OWN[state["case"]["op"]](state)
    return _PLAIN[state["case"]["op"]](state)


def _own_serve(s):
    buf, c = s["buf"], s["case"]
    order, _ = buf.expert_order(s["topk_idx"], no_sync=True)
    codes, scales, _ = buf.expert_sort_int8(s["x"], order, no_sync=True)
    y, _ = buf.expert_linear_int8(codes, scales, s["w"], s["w_scales"], order, swiglu=c["swiglu"],
                                  dtype=s["out"].dtype, out=s["out"], no_sync=True)
    return y


def _own_product(s):
    buf, c = s["buf"], s["case"]
    rows = s["counts"] if c["op"] == "product_slots" else s["offsets"]
    codes, scales, _ = buf.expert_quantize(s["x"], rows, no_sync=True)
    y, _ = buf.expert_linear_int8(codes, scales, s["w"], s["w_scales"], rows, swiglu=c["swiglu"],
                                  dtype=s["out"].dtype, out=s["out"], no_sync=True)
    return y


def _own_saved(s):
    buf = s["buf"]
    codes, scales, _ = buf.expert_quantize(s["x"], s["offsets"], block=s["case"]["block"], out=s["codes"],
                                           scales=s["scales"], no_sync=True)
    x, _ = buf.expert_dequantize(codes, scales, s["offsets"], dtype=s["out"].dtype, out=s["out"], no_sync=True)
    return x, scales


def _own_act_grad(s):
    d_pre, h, _ = s["buf"].expert_swiglu_backward_int8(s["d_h"], s["codes"], s["scales"], s["offsets"], return_h=True,
                                                       out=s["out"], h=s["h"], no_sync=True)
    return d_pre, h


def _own_w_grad(s):
    _, d_w, _ = s["buf"].expert_linear_backward_int8(s["d_y"], s["codes"], s["scales"], None, s["offsets"],
                                                     d_w_dtype=s["wide"], no_sync=True)
    return d_w


_OWN = {"serve": _own_serve, "product": _own_product, "product_slots": _own_product, "saved": _own_saved,
        "act_grad": _own_act_grad, "w_grad": _own_w_grad}


# ---- plain forms --------------------------------------------------------------

def _scale_shape(lead, H, block):
    return lead if block == 0 else lead + ((H + block - 1) // block,)


def _grouped(x, block):
    """x [..., H] as [..., groups, values], zeros behind the row's end."""
    if block == 0:
        return x.unsqueeze(-2)
    H = x.shape[-1]
    groups = (H + block - 1) // block
    return torch.nn.functional.pad(x, (0, groups * block - H)).unflatten(-1, (groups, block))


def _quantize(x, block):
    f = _grouped(x.float(), block)
    m = f.abs().amax(-1, keepdim=True).clamp_min(FLOOR)
    top = torch.full_like(m, 127.0)  # by a tensor: torch multiplies by the inverse of a number
    codes = torch.round(f * (top / m)).to(torch.int8).flatten(-2)[..., :x.shape[-1]]
    scales = (m / top).squeeze(-1)
    return codes.contiguous(), scales.squeeze(-1) if block == 0 else scales


def _restored(codes, scales, block):
    """fp32 values of codes."""
    if block == 0:
        return codes.float() * scales[..., None]
    return codes.float() * scales.repeat_interleave(block, -1)[..., :codes.shape[-1]]


def _swiglu(pre):
    g, u = pre.chunk(2, dim=-1)
    return g / (1.0 + torch.exp(-g)) * u


def _spans(s):
    """(expert, first row, row past its last) of the experts that have rows."""
    b = s["bounds"]
    return [(e, b[e], b[e + 1]) for e in range(len(b) - 1) if b[e + 1] > b[e]]


def _plain_product(s):
    c, w, ws = s["case"], s["w"], s["w_scales"]
    codes, scales = _quantize(s["x"], 0)
    if c["op"] == "serve":  # rows by expert
        flat = s["topk_idx"].reshape(-1)
        slots = torch.sort(torch.where(flat >= 0, flat, c["E"]), stable=True).indices
        codes, scales = codes[slots // c["K"]], scales[slots // c["K"]]
    out = torch.zeros_like(s["out"])
    for e, a, b in _spans(s):
        at = (e, slice(0, b - a)) if c["op"] == "product_slots" else slice(a, b)
        y = codes[at].float() @ w[e].float().t() * scales[at][:, None] * ws[e]
        out[at] = (_swiglu(y) if c["swiglu"] else y).to(out.dtype)
    return out


def _plain_saved(s):
    n, block = s["bounds"][-1], s["case"]["block"]
    codes, scales = _quantize(s["x"][:n], block)
    x, kept = torch.zeros_like(s["out"]), torch.zeros_like(s["scales"])
    x[:n] = _restored(codes, scales, block).to(x.dtype)
    kept[:n] = scales
    return x, kept


def _plain_act_grad(s):
    n, block = s["bounds"][-1], s["case"]["block"]
    g, u = _restored(s["codes"][:n], s["scales"][:n], block).chunk(2, dim=-1)
    d = s["d_h"][:n].float()
    sg = 1.0 / (1.0 + torch.exp(-g))
    d_pre, h = torch.zeros_like(s["out"]), torch.zeros_like(s["h"])
    d_pre[:n] = torch.cat([d * u * sg * (1.0 + g * (1.0 - sg)), d * g * sg], -1).to(d_pre.dtype)
    h[:n] = (g * sg * u).to(h.dtype)
    return d_pre, h


def _plain_w_grad(s):
    c, d_y = s["case"], s["d_y"]
    d_w = torch.zeros(c["E"], c["N"], c["Kd"], device=d_y.device, dtype=s["wide"])
    for e, a, b in _spans(s):
        # the operator's definition: saved rows come back in the gradient's type
        x = _restored(s["codes"][a:b], s["scales"][a:b], c["block"]).to(d_y.dtype)
        d_w[e] = (d_y[a:b].float().t() @ x.float()).to(d_w.dtype)
    return d_w


_PLAIN = {"serve": _plain_product, "product": _plain_product, "product_slots": _plain_product,
          "saved": _plain_saved, "act_grad": _plain_act_grad, "w_grad": _plain_w_grad}


# ---- work ---------------------------------------------------------------------

def work(case):
    op, T, E, K, b = case["op"], case["T"], case["E"], case["K"], BYTES[case["dtype"]]
    M = int(round(T * K * (1.0 - case["empty"])))
    groups = lambda width: 1 if case["block"] == 0 else (width + 127) // 128  # noqa: E731
    if op == "saved":  # the codes are kept: written, and read again
        H = case["H"]
        return {"bytes": M * (2 * H * b + 2 * H + 8 * groups(H)), "flops": 5 * M * H}
    N = case["N"]
    if op == "act_grad":
        return {"bytes": M * (N * b + 2 * N + 4 * groups(2 * N) + 3 * N * b), "flops": 16 * M * N}
    Kd = case["Kd"]
    if op == "w_grad":
        return {"bytes": M * (N * b + Kd + 4 * groups(Kd)) + E * N * Kd * (4 if case["wide"] else b),
                "flops": 2 * M * N * Kd}
    cols = 2 * N if case["swiglu"] else N
    used = min(E, M) if case["routing"] == "zipf" else E * (1.0 - (1.0 - K * (1.0 - case["empty"]) / E) ** T) \
        if K < E else E
    rows = (T if op == "serve" else M) * Kd * b + (T * K * 8 if op == "serve" else 0)
    return {"bytes": int(rows + M * N * b + used * cols * (Kd + 4)), "flops": 2 * M * cols * Kd}


# ---- the definitions in 64 bits --------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op, E, K = case["op"], case["E"], case["K"]
    ends, dev = s["offsets"].tolist(), s["offsets"].device
    f64 = dict(dtype=torch.float64, device=dev)

    def codes_of(x, width):
        """(codes, scales per value, scales) of x in 64 bits, `width` values to a group."""
        cols = torch.arange(x.shape[-1], device=dev) // width
        n = int(cols[-1]) + 1
        top = torch.zeros(*x.shape[:-1], n, **f64).scatter_reduce_(-1, cols.expand(x.shape), x.abs(), "amax")
        top = torch.maximum(top, torch.tensor(FLOOR, **f64))
        # codes and scales are defined with three fp32 roundings, each of an exact or a 64-bit value
        scale, factor = (top / 127).float().double(), (127 / top).float().double()
        return torch.round((x * factor[..., cols]).float().double()), scale[..., cols], scale

    def values(codes, scales):
        if case["block"] == 0:
            return codes.double() * scales.double()[:, None]
        cols = torch.arange(codes.shape[-1], device=dev) // case["block"]
        return codes.double() * scales.double()[:, cols]

    n = ends[-1]
    if op == "saved":
        H = case["H"]
        c, each, scale = codes_of(s["x"][:n].double(), case["block"] or H)
        x, kept = torch.zeros(s["x"].shape, **f64), torch.zeros(s["scales"].shape, **f64)
        x[:n] = c * each
        kept[:n] = scale if case["block"] else scale[:, 0]
        return x, kept
    if op == "act_grad":
        N = case["N"]
        pre = values(s["codes"][:n], s["scales"][:n])
        g, u, d = pre[:, :N], pre[:, N:], s["d_h"][:n].double()
        sg = torch.sigmoid(g)
        d_pre, h = torch.zeros(s["out"].shape, **f64), torch.zeros(s["h"].shape, **f64)
        d_pre[:n, :N] = d * u * (sg + g * sg * (1 - sg))
        d_pre[:n, N:] = d * g * sg
        h[:n] = g * sg * u
        return d_pre, h
    if op == "w_grad":
        d_w = torch.zeros(E, case["N"], case["Kd"], **f64)
        for e in range(E):
            a, b = ends[e], ends[e + 1]
            if b > a:  # the definition rounds restored rows to the gradient's type
                x = values(s["codes"][a:b], s["scales"][a:b]).to(s["d_y"].dtype).double()
                torch.matmul(s["d_y"][a:b].double().t().contiguous(), x, out=d_w[e])
        return d_w
    x, N = s["x"], case["N"]
    out = torch.zeros(s["out"].shape, **f64)
    if op == "serve":
        t, k = torch.nonzero(s["topk_idx"] >= 0, as_tuple=True)
        by = torch.argsort(s["topk_idx"][t, k] * s["topk_idx"].numel() + t * K + k)
        token = t[by]
    for e in range(E):
        a, b = ends[e], ends[e + 1]
        if a == b:
            continue
        xs = x[e, :b - a] if op == "product_slots" else x[token[a:b]] if op == "serve" else x[a:b]
        c, each, _ = codes_of(xs.double(), case["Kd"])
        w = s["w"][e].double() * s["w_scales"][e].double()[:, None]
        y = torch.matmul(c * each, w.t().contiguous())
        if case["swiglu"]:
            y = y[:, :N] * torch.sigmoid(y[:, :N]) * y[:, N:]
        if op == "product_slots":
            out[e, :b - a] = y
        else:
            out[a:b] = y
    return out
