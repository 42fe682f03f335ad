"""The operators beside the dispatch path, as cases that can be timed: the
router (gate_topk), tokens sorted by expert and back (expert_order,
expert_sort, expert_unsort) and the experts' products (expert_linear), with
their gradients.

``run`` computes a case in plain torch while ``own`` is false, and with the
library's calls, as a user's program makes them, while it is true.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


# ---- cases --------------------------------------------------------------------

def listed():
    """Widths, expert counts and top-k are those of the package's workloads
    (128 x 256, decode 128 x 7168, prefill 4096 x 7168, skewed 8192 x 7168,
    reuse 16384 x 4096); the experts' inner widths are generic."""
    return [
        # Router of a decode batch: grouped sigmoid scores with a selection bias.
        dict(name="gate_decode", op="gate", T=128, E=256, K=8, dtype="f32", score="sigmoid", groups=8, kept=4,
             renorm=True, bias=True, masked=0.0, grad=False),
        # Router of a training step over a long batch, forward and backward, some
        # experts masked out per token (and a few tokens with every expert masked).
        dict(name="gate_train", op="gate", T=16384, E=256, K=8, dtype="bf16", score="softmax", groups=1, kept=1,
             renorm=False, bias=False, masked=0.1, grad=True),
        # One decode batch put in expert order: the smallest call, latency counts.
        dict(name="sort_tiny", op="sort", T=128, E=16, K=2, H=256, dtype="bf16", routing="uniform", empty=0.0),
        # A long skewed prefill, an odd token count, in expert order.
        dict(name="sort_skewed", op="sort", T=8191, E=256, K=8, H=7168, dtype="bf16", routing="zipf", empty=0.05),
        # The way back with the gate weights, the package's longest batch.
        dict(name="unsort_long", op="unsort", T=16384, E=64, K=6, H=4096, dtype="bf16", routing="uniform",
             empty=0.0),
        # The same call's gradients in a training step (rows and weights).
        dict(name="unsort_grad", op="unsort_grad", T=4095, E=256, K=8, H=7168, dtype="bf16", routing="uniform",
             empty=0.05),
        # One token's experts: eight experts' weights are read once.
        dict(name="linear_one_token", op="linear", T=1, E=64, K=8, Kd=7168, N=2048, dtype="bf16", routing="uniform",
             empty=0.0, swiglu=True),
        # A decode batch in the low-latency layout ([E, cap, H] slots with counts).
        dict(name="linear_decode", op="linear_slots", T=128, E=64, K=6, Kd=4096, N=2048, cap=128, dtype="bf16",
             routing="uniform", empty=0.0, swiglu=True),
        # A prefill's first product with its gated activation.
        dict(name="linear_prefill", op="linear", T=4096, E=64, K=8, Kd=7168, N=2048, dtype="bf16",
             routing="uniform", empty=0.0, swiglu=True),
        # A skewed batch's second product, half precision, odd sizes.
        dict(name="linear_skewed", op="linear", T=2047, E=64, K=6, Kd=1416, N=4096, dtype="f16", routing="zipf",
             empty=0.05, swiglu=False),
        # Both gradients of a product in a training step.
        dict(name="linear_grad", op="linear_grad", T=8192, E=64, K=6, Kd=4096, N=2048, dtype="bf16",
             routing="uniform", empty=0.0),
        # The activation's gradient between the two products of that step.
        dict(name="swiglu_grad", op="swiglu_grad", T=8191, E=64, K=6, N=2048, dtype="bf16", routing="uniform",
             empty=0.0),
    ]


def draw(rng):
    def log(lo, hi, step=1):
        v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
        return max(lo, min(hi, int(v) // step * step))

    op = rng.choice(["gate", "sort", "unsort", "unsort_grad", "linear", "linear", "linear_slots", "linear_grad",
                     "linear_grad", "swiglu_grad"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    if op == "gate":
        E = rng.choice([8, 16, 60, 64, 128, 160, 256, 512])
        groups = rng.choice([g for g in (1, 1, 2, 4, 8) if E % g == 0 and E // g >= 2])
        kept = rng.randint(1, groups)
        K = rng.randint(1, min(8, kept * (E // groups)))
        return dict(op=op, T=log(1, 16384), E=E, K=K, dtype=rng.choice(["f32", "bf16", "f16"]),
                    score=rng.choice(["softmax", "sigmoid"]), groups=groups, kept=kept,
                    renorm=rng.random() < 0.5, bias=rng.random() < 0.5, masked=rng.choice([0.0, 0.1]),
                    grad=rng.random() < 0.5)
    routing = rng.choice(["uniform", "zipf"])
    empty = rng.choice([0.0, 0.05, 0.5])
    if op in ("sort", "unsort", "unsort_grad"):
        E = rng.choice([16, 60, 64, 128, 256, 1024])
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        H = log(64, 7168 if dtype != "f32" else 3584, 8)
        return dict(op=op, T=log(1, 8191), E=E, K=rng.randint(1, 8), H=H, dtype=dtype, routing=routing, empty=empty)
    E = rng.choice([8, 12, 16, 32, 64])
    K = rng.randint(1, 8)
    if op == "swiglu_grad":
        return dict(op=op, T=log(1, 8191), E=E, K=min(K, 6), N=log(64, 2048, 8), dtype=dtype, routing=routing,
                    empty=empty)
    case = dict(op=op, T=log(1, 4096), E=E, K=K, Kd=log(64, 7168, 8), N=log(64, 2048, 8), dtype=dtype,
                routing=routing, empty=empty)
    if op == "linear_slots":
        case["T"] = log(1, 256)
        case["cap"] = case["T"] + rng.randint(0, 64)
        case["swiglu"] = rng.random() < 0.5
    elif op == "linear":
        case["swiglu"] = rng.random() < 0.5
    else:
        case["Kd"] = min(case["Kd"], 4096)
    return case


# ---- inputs -------------------------------------------------------------------

def _route(g, case, dev):
    """topk_idx [T, K] int64: distinct experts of a token, some slots empty."""
    T, E, K = case["T"], case["E"], case["K"]
    noise = -torch.log(-torch.log(torch.rand(T, E, generator=g, device=dev, dtype=torch.float64).clamp(1e-12, 1 - 1e-12)))
    if case["routing"] == "zipf":  # expert e drawn with weight (e + 1)^-1.2
        noise = noise - 1.2 * torch.log(torch.arange(1, E + 1, device=dev, dtype=torch.float64))
    idx = torch.topk(noise, K, dim=1).indices
    if case["empty"] > 0:
        idx = torch.where(torch.rand(T, K, generator=g, device=dev) < case["empty"], -1, idx)
    return idx.contiguous()


def _buffer(case):
    from combine_get_dispatch_layout_amd import Buffer
    return Buffer(num_experts=case["E"], num_ranks=1, num_channels=1, max_tokens=max(case["T"], 1))


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(dev)
    g.manual_seed(seed)
    op, T, E, K = case["op"], case["T"], case["E"], case["K"]
    dt = DTYPES[case["dtype"]]

    def randn(*shape, scale=1.0, dtype=dt):
        return torch.randn(*shape, generator=g, device=dev, dtype=dtype).mul_(scale)

    s = dict(case=case)
    if own:
        s["buf"] = _buffer(case)
    if op == "gate":
        logits = randn(T, E, scale=1.5)
        if case["masked"] > 0:
            logits.masked_fill_(torch.rand(T, E, generator=g, device=dev) < case["masked"], float("-inf"))
            logits[T // 2::97] = float("-inf")
        s["logits"] = logits
        s["bias"] = randn(E, scale=0.1, dtype=torch.float32) if case["bias"] else None
        s["scale"] = 2.5
        s["d_weights"] = randn(T, K, dtype=torch.float32) if case["grad"] else None
        return s
    idx = _route(g, case, dev)
    s["topk_idx"] = idx
    order = _order_plain(idx, E)
    if op == "sort":
        s["x"] = randn(T, case["H"])
        s["out"] = torch.zeros(T * K, case["H"], device=dev, dtype=dt)
        return s
    if op in ("unsort", "unsort_grad"):
        s["order"] = s["buf"].expert_order(idx)[0] if own else order
        s["rows"] = randn(T * K, case["H"])
        s["weights"] = torch.softmax(randn(T, K, dtype=torch.float32), -1)
        if op == "unsort_grad":
            s["d_out"] = randn(T, case["H"])
            s["out"] = torch.zeros(T * K, case["H"], device=dev, dtype=dt)
        return s
    offsets = order[0]
    counts = (offsets[1:] - offsets[:-1]).contiguous()
    s["offsets"], s["counts"] = offsets, counts
    s["bounds"] = offsets.tolist()  # the plain forms go expert by expert
    M = T * K
    if op == "swiglu_grad":
        s["pre"] = randn(M, 2 * case["N"])
        s["d_h"] = randn(M, case["N"])
        s["out"] = torch.zeros(M, 2 * case["N"], device=dev, dtype=dt)
        return s
    Kd, N = case["Kd"], case["N"]
    cols = 2 * N if case.get("swiglu") else N
    s["w"] = randn(E, cols, Kd, scale=Kd ** -0.5)
    if op == "linear_slots":
        s["x"] = randn(E, case["cap"], Kd)
        s["out"] = torch.zeros(E, case["cap"], N, device=dev, dtype=dt)
    else:
        s["x"] = randn(M, Kd)
        if op == "linear":
            s["out"] = torch.zeros(M, N, device=dev, dtype=dt)
        else:
            s["d_y"] = randn(M, N)
            s["out"] = torch.zeros(M, Kd, device=dev, dtype=dt)
    return s


# ---- one pass -----------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _gate_options(c, s):
    return dict(score=c["score"], num_groups=c["groups"], groups_kept=c["kept"], renormalize=c["renorm"],
                scale=s["scale"], bias=s["bias"])


def _own_gate(s):
    c = s["case"]
    opts = _gate_options(c, s)
    idx, w, _ = s["buf"].gate_topk(s["logits"], c["K"], no_sync=True, **opts)
    if not c["grad"]:
        return idx, w
    d, _ = s["buf"].gate_topk_backward(s["d_weights"], s["logits"], idx, no_sync=True, **opts)
    return idx, w, d


def _own_sort(s):
    order, _ = s["buf"].expert_order(s["topk_idx"], no_sync=True)
    rows, _ = s["buf"].expert_sort(s["x"], order, out=s["out"], no_sync=True)
    return rows, order.expert_offsets, order.row_of_slot, order.slot_of_row


def _own_unsort(s):
    out, _ = s["buf"].expert_unsort(s["rows"], s["order"], topk_weights=s["weights"], no_sync=True)
    return out


def _own_unsort_grad(s):
    d_rows, d_w, _ = s["buf"].expert_unsort_backward(s["d_out"], s["rows"], s["order"], s["weights"], out=s["out"],
                                                     no_sync=True)
    return d_rows, d_w


def _own_linear(s):
    slots = s["case"]["op"] == "linear_slots"
    y, _, _ = s["buf"].expert_linear(s["x"], s["w"], s["counts"] if slots else s["offsets"],
                                     swiglu=s["case"]["swiglu"], out=s["out"], no_sync=True)
    return y


def _own_linear_grad(s):
    d_x, d_w, _ = s["buf"].expert_linear_backward(s["d_y"], s["x"], s["w"], s["offsets"], out=s["out"], no_sync=True)
    return d_x, d_w


def _own_swiglu_grad(s):
    d_pre, _ = s["buf"].expert_swiglu_backward(s["d_h"], s["pre"], s["offsets"], out=s["out"], no_sync=True)
    return d_pre


_OWN = {"gate": _own_gate, "sort": _own_sort, "unsort": _own_unsort, "unsort_grad": _own_unsort_grad,
        "linear": _own_linear, "linear_slots": _own_linear, "linear_grad": _own_linear_grad,
        "swiglu_grad": _own_swiglu_grad}


# ---- plain forms --------------------------------------------------------------

def _best(keys, n):
    """The n best of the last axis, ties to the lower index."""
    return torch.sort(keys, dim=-1, descending=True, stable=True).indices[..., :n]


def _plain_gate(s):
    c = s["case"]
    T, E = s["logits"].shape
    K, scale = c["K"], s["scale"]
    l = s["logits"].double()  # scores next to a border: selection in 64 bits
    none = torch.isinf(l) & (l < 0)
    top = torch.clamp_min(l.amax(-1, keepdim=True), -1e300)
    if c["score"] == "softmax":
        e = torch.exp(l - top)
        score = e / e.sum(-1, keepdim=True).clamp_min(1e-300)
    else:
        score = 1.0 / (1.0 + torch.exp(-l))
    keys = score + s["bias"].double() if s["bias"] is not None else score
    keys = torch.where(none, float("-inf"), keys)
    if c["groups"] > 1:
        by = keys.view(T, c["groups"], E // c["groups"])
        two = torch.sort(by, dim=-1, descending=True).values[..., :2]
        group = torch.where(torch.isinf(two), 0.0, two).sum(-1)
        group = torch.where(torch.isinf(two[..., 0]), float("-inf"), group)
        keep = torch.zeros_like(group, dtype=torch.bool).scatter_(1, _best(group, c["kept"]), True)
        keys = torch.where(keep[..., None], by, float("-inf")).reshape(T, E)
    idx = _best(keys, K)
    filled = ~torch.isinf(torch.gather(keys, 1, idx))
    at = torch.gather(score, 1, idx) * filled
    v = at / at.sum(-1, keepdim=True).clamp_min(1e-300) if c["renorm"] else at
    out_idx = torch.where(filled, idx, -1)
    out_w = (scale * v).float()
    if not c["grad"]:
        return out_idx, out_w
    gr = s["d_weights"].double() * filled
    if c["renorm"]:
        d = scale * v * (gr - (gr * v).sum(-1, keepdim=True))
        if c["score"] == "sigmoid":
            d = d * (1.0 - at)
        dl = torch.zeros_like(l).scatter_add_(1, idx, d * filled)
    elif c["score"] == "sigmoid":
        dl = torch.zeros_like(l).scatter_add_(1, idx, scale * gr * at * (1.0 - at))
    else:
        dl = torch.zeros_like(l).scatter_add_(1, idx, gr) - (gr * at).sum(-1, keepdim=True)
        dl = scale * score * dl
    return out_idx, out_w, dl.to(s["logits"].dtype)


def _order_plain(idx, E):
    """(expert_offsets [E + 1], row_of_slot [T, K], slot_of_row [T * K])."""
    flat = idx.reshape(-1)
    n = flat.numel()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    by, slots = torch.sort(key, stable=True)
    offsets = torch.searchsorted(by, torch.arange(E + 1, device=idx.device)).to(torch.int32)
    filled = by < E
    slot_of_row = torch.where(filled, slots, -1).to(torch.int32)
    row = torch.empty(n, dtype=torch.int32, device=idx.device)
    row[slots] = torch.where(filled, torch.arange(n, device=idx.device), -1).to(torch.int32)
    return offsets, row.view(idx.shape), slot_of_row


def _plain_sort(s):
    x, K = s["x"], s["case"]["K"]
    offsets, row_of_slot, slot_of_row = _order_plain(s["topk_idx"], s["case"]["E"])
    src = slot_of_row.long()
    rows = torch.where((src >= 0)[:, None], x[src.clamp_min(0) // K], 0.0)
    return rows.to(x.dtype), offsets, row_of_slot, slot_of_row


def _plain_unsort(s):
    rows, w = s["rows"], s["weights"]
    row = s["order"][1].long()
    acc = torch.zeros(row.shape[0], rows.shape[1], device=rows.device)
    for k in range(row.shape[1]):
        here = row[:, k] >= 0
        y = rows[row[:, k].clamp_min(0)].float() * w[:, k:k + 1]
        acc += torch.where(here[:, None], y, 0.0)
    return acc.to(rows.dtype)


def _plain_unsort_grad(s):
    rows, w, d_out = s["rows"], s["weights"], s["d_out"].float()
    row = s["order"][1].long()
    d_rows = torch.zeros(rows.shape, device=rows.device, dtype=rows.dtype)
    d_w = torch.zeros_like(w)
    for k in range(row.shape[1]):
        t = torch.nonzero(row[:, k] >= 0).squeeze(1)
        r = row[t, k]
        d_rows[r] = (d_out[t] * w[t, k:k + 1]).to(rows.dtype)
        d_w[t, k] = (d_out[t].double() * rows[r].double()).sum(-1).float()
    return d_rows, d_w


def _spans(s):
    """(expert, first row, row past its last) of the experts that have rows."""
    b = s["bounds"]
    return [(e, b[e], b[e + 1]) for e in range(len(b) - 1) if b[e + 1] > b[e]]


def _swiglu(pre):
    g, u = pre.chunk(2, dim=-1)
    return g / (1.0 + torch.exp(-g)) * u


def _plain_linear(s):
    x, w, c = s["x"], s["w"], s["case"]
    out = torch.zeros_like(s["out"])
    for e, a, b in _spans(s):
        at = (e, slice(0, b - a)) if c["op"] == "linear_slots" else slice(a, b)
        y = x[at].float() @ w[e].float().t()
        out[at] = (_swiglu(y) if c["swiglu"] else y).to(x.dtype)
    return out


def _plain_linear_grad(s):
    x, w, d_y = s["x"], s["w"], s["d_y"]
    d_x = torch.zeros_like(s["out"])
    d_w = torch.zeros_like(w)
    for e, a, b in _spans(s):
        d = d_y[a:b].float()
        d_x[a:b] = (d @ w[e].float()).to(x.dtype)
        d_w[e] = (d.t() @ x[a:b].float()).to(w.dtype)
    return d_x, d_w


def _plain_swiglu_grad(s):
    n = s["bounds"][-1]
    g, u = s["pre"][:n].float().chunk(2, dim=-1)
    d = s["d_h"][:n].float()
    sg = 1.0 / (1.0 + torch.exp(-g))
    d_pre = torch.zeros_like(s["out"])
    d_pre[:n] = torch.cat([d * u * sg * (1.0 + g * (1.0 - sg)), d * g * sg], -1).to(d_pre.dtype)
    return d_pre


_PLAIN = {"gate": _plain_gate, "sort": _plain_sort, "unsort": _plain_unsort, "unsort_grad": _plain_unsort_grad,
          "linear": _plain_linear, "linear_slots": _plain_linear, "linear_grad": _plain_linear_grad,
          "swiglu_grad": _plain_swiglu_grad}


# ---- work ---------------------------------------------------------------------

def work(case):
    op, T, E, K, b = case["op"], case["T"], case["E"], case["K"], BYTES[case["dtype"]]
    if op == "gate":
        n = T * E * b + T * K * 12
        if case["grad"]:
            n += 2 * T * E * b + T * K * 12
        return {"bytes": n, "flops": T * E * (12 if case["grad"] else 6)}
    M = int(round(T * K * (1.0 - case["empty"])))
    if op == "sort":
        return {"bytes": (T + M) * case["H"] * b + T * K * 16 + 4 * (E + 1), "flops": T * K}
    if op == "unsort":
        return {"bytes": (T + M) * case["H"] * b + T * K * 8, "flops": 2 * M * case["H"]}
    if op == "unsort_grad":
        return {"bytes": (T + 2 * M) * case["H"] * b + T * K * 12, "flops": 3 * M * case["H"]}
    N = case["N"]
    if op == "swiglu_grad":
        return {"bytes": 5 * M * N * b, "flops": 12 * M * N}
    Kd = case["Kd"]
    cols = 2 * N if case.get("swiglu") else N
    used = min(E, M) if case["routing"] == "zipf" else E * (1.0 - (1.0 - K * (1.0 - case["empty"]) / E) ** T) \
        if K < E else E
    if op == "linear_grad":
        return {"bytes": int(M * (2 * Kd + N) + (used + E) * N * Kd) * b, "flops": 4 * M * N * Kd}
    return {"bytes": int(M * (Kd + N) + used * cols * Kd) * b, "flops": 2 * M * cols * Kd}


# ---- the definitions in 64 bits --------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "gate":
        return _exact_gate(case, s)
    idx, E, K = s["topk_idx"], case["E"], case["K"]
    # rows by expert, then token, then slot
    t, k = torch.nonzero(idx >= 0, as_tuple=True)
    e = idx[t, k]
    by = torch.argsort(e * idx.numel() + t * K + k)
    t, k, e = t[by], k[by], e[by]
    n = t.numel()
    starts = [0] + torch.cumsum(torch.bincount(e, minlength=E), 0).tolist()
    if op == "sort":
        rows = torch.zeros(idx.numel(), case["H"], dtype=torch.float64, device=idx.device)
        rows[:n] = s["x"].double()[t]
        ros = torch.full_like(idx, -1)
        ros[t, k] = torch.arange(n, device=idx.device)
        sor = torch.full((idx.numel(),), -1, dtype=torch.int64, device=idx.device)
        sor[:n] = t * K + k
        return rows, torch.tensor(starts, device=idx.device).to(torch.int32), ros.to(torch.int32), sor.to(torch.int32)
    if op in ("unsort", "unsort_grad"):
        w = s["weights"].double()[t, k]
        y = s["rows"][:n].double()
        if op == "unsort":
            out = torch.zeros(case["T"], case["H"], dtype=torch.float64, device=idx.device)
            return out.index_add_(0, t, y * w[:, None])
        d = s["d_out"].double()[t]
        d_rows = torch.zeros(idx.numel(), case["H"], dtype=torch.float64, device=idx.device)
        d_rows[:n] = d * w[:, None]
        d_w = torch.zeros(idx.shape, dtype=torch.float64, device=idx.device)
        d_w[t, k] = (d * y).sum(1)
        return d_rows, d_w
    if op == "swiglu_grad":
        pre = s["pre"][:n].double()
        N = case["N"]
        g, u, d = pre[:, :N], pre[:, N:], s["d_h"][:n].double()
        sg = torch.sigmoid(g)
        out = torch.zeros(idx.numel(), 2 * N, dtype=torch.float64, device=idx.device)
        out[:n, :N] = d * u * (sg + g * sg * (1 - sg))
        out[:n, N:] = d * g * sg
        return out
    if op == "linear_grad":
        d_x = torch.zeros(s["x"].shape, dtype=torch.float64, device=idx.device)
        d_w = torch.zeros(s["w"].shape, dtype=torch.float64, device=idx.device)
        for i in range(E):
            a, b = starts[i], starts[i + 1]
            d = s["d_y"][a:b].double()
            torch.matmul(d, s["w"][i].double(), out=d_x[a:b])
            torch.matmul(d.t().contiguous(), s["x"][a:b].double(), out=d_w[i])
        return d_x, d_w
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=idx.device)
    N = case["N"]
    for i in range(E):
        a, b = starts[i], starts[i + 1]
        if a == b:
            continue
        xs = s["x"][i, :b - a] if op == "linear_slots" else s["x"][a:b]
        y = torch.matmul(xs.double(), s["w"][i].double().t().contiguous())
        if case["swiglu"]:
            y = y[:, :N] * torch.sigmoid(y[:, :N]) * y[:, N:]
        if op == "linear_slots":
            out[i, :b - a] = y
        else:
            out[a:b] = y
    return out


def _exact_gate(c, s):
    """Selection one expert at a time; gradients from the Jacobian of the chosen weights."""
    l = s["logits"].double()
    T, E = l.shape
    K, G, scale = c["K"], c["groups"], s["scale"]
    ok = l > float("-inf")
    some = ok.any(1, keepdim=True)
    if c["score"] == "softmax":
        p = torch.where(some, torch.softmax(torch.where(some, l, 0.0), 1), 0.0)
    else:
        p = torch.sigmoid(l)
    low = torch.tensor(-1e30, dtype=torch.float64, device=l.device)
    key = torch.where(ok, p + (0 if s["bias"] is None else s["bias"].double()), low)
    cols = torch.arange(E, device=l.device)

    def first_max(v):  # lowest index among the largest
        m = v.max(1, keepdim=True).values
        return torch.where(v == m, torch.arange(v.shape[1], device=v.device), v.shape[1]).min(1).values

    if G > 1:
        gk = key.view(T * G, E // G)
        a = first_max(gk)
        one = gk.gather(1, a[:, None])[:, 0]
        rest = gk.scatter(1, a[:, None], -1e30)
        two = rest.max(1).values
        gs = torch.where(one > -1e29, one + torch.where(two > -1e29, two, 0.0), low).view(T, G)
        keep = torch.zeros(T, G, dtype=torch.bool, device=l.device)
        for _ in range(c["kept"]):
            j = first_max(gs)
            keep[torch.arange(T, device=l.device), j] = True
            gs = gs.scatter(1, j[:, None], -2e30)
        key = torch.where(keep[:, cols // (E // G)], key, low)
    chosen, filled = [], []
    for _ in range(K):
        j = first_max(key)
        filled.append(key.gather(1, j[:, None])[:, 0] > -1e29)
        chosen.append(j)
        key = key.scatter(1, j[:, None], -2e30)
    idx, filled = torch.stack(chosen, 1), torch.stack(filled, 1)
    sc = torch.where(filled, p.gather(1, idx), 0.0)
    total = sc.sum(1, keepdim=True)
    w = scale * (sc / torch.where(total > 0, total, 1.0) if c["renorm"] else sc)
    out_idx = torch.where(filled, idx, -1)
    if not c["grad"]:
        return out_idx, w
    gw = torch.where(filled, s["d_weights"].double(), 0.0) * scale
    d_sc = gw
    if c["renorm"]:
        den = torch.where(total > 0, total, 1.0)
        d_sc = torch.where(filled, gw / den - (gw * sc).sum(1, keepdim=True) / den ** 2, 0.0)
    d_p = torch.zeros_like(p).scatter_add_(1, idx, d_sc)
    if c["score"] == "softmax":
        return out_idx, w, p * (d_p - (d_p * p).sum(1, keepdim=True))
    return out_idx, w, d_p * p * (1 - p)
