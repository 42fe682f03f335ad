"""The router (gate_topk and its gradient) against its definition in fp64 on
the CPU.  The choice must be equal; a weight may differ by its fp32 roundings:
the argument of exp is rounded once (relative error |l - max| 2^-24 of exp),
exp and the division are within a few units, and the sum over E experts adds
at most log2(64) + E / 64 roundings."""

import pytest
import torch

from tests.gpu_common import device, make_buffer

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def reference(logits, K, score, groups, kept, renorm, scale, bias, d_w=None):
    """(idx, weights, d_logits) in fp64, one token at a time."""
    T, E = logits.shape
    l = logits.double()
    idx = torch.full((T, K), -1, dtype=torch.int64)
    w = torch.zeros(T, K, dtype=torch.float64)
    d = torch.zeros(T, E, dtype=torch.float64)
    for t in range(T):
        ok = l[t] > float("-inf")
        if not ok.any():
            continue
        p = torch.zeros(E, dtype=torch.float64)
        if score == "softmax":
            p[ok] = torch.softmax(l[t][ok], 0)
        else:
            p[ok] = torch.sigmoid(l[t][ok])
        key = p + (0.0 if bias is None else bias.double())
        cand = [e for e in range(E) if ok[e] and key[e] > float("-inf")]
        if groups > 1:
            per = E // groups
            sums = []
            for g in range(groups):
                best = sorted((float(key[e]) for e in cand if e // per == g), reverse=True)[:2]
                sums.append(sum(best) if best else float("-inf"))
            keep = sorted(range(groups), key=lambda g: (-sums[g], g))[:kept]
            cand = [e for e in cand if e // per in keep]
        # without a bias the logits order as the scores do, exactly
        rank = l[t] if bias is None else key
        cand = sorted(cand, key=lambda e: (-float(rank[e]), e))[:K]
        n = len(cand)
        if n == 0:
            continue
        c = torch.tensor(cand)
        idx[t, :n] = c
        if renorm:
            s = l[t][c] if score == "softmax" else torch.nn.functional.logsigmoid(l[t][c])
            v = torch.softmax(s, 0)
        else:
            v = p[c]
        w[t, :n] = scale * v
        if d_w is None:
            continue
        g = d_w[t, :n].double()
        if renorm:
            own = scale * v * (g - (g * v).sum())
            if score == "sigmoid":
                own = own * torch.sigmoid(-l[t][c])
            d[t, c] = own
        elif score == "sigmoid":
            d[t, c] = scale * g * p[c] * torch.sigmoid(-l[t][c])
        else:
            e = torch.zeros(E, dtype=torch.float64)
            e[c] = g
            d[t] = scale * p * (e - (g * v).sum())
    return idx, w, d


def relative(logits, E):
    """The relative error that the fp32 exps, the sum and the division allow."""
    finite = logits[logits > float("-inf")].double()
    span = float(finite.max() - finite.min()) if finite.numel() else 0.0
    return (2.0 * span + 2.0 * (6 + E / 64.0) + 24.0) * U


CASES = [
    # T, E, K, dtype, score, groups, kept, renorm, bias, masked
    (1, 1, 1, torch.float32, "softmax", 1, 1, False, False, 0.0),
    (1, 256, 8, torch.float32, "sigmoid", 8, 4, True, True, 0.0),
    (5, 16, 2, torch.bfloat16, "softmax", 1, 1, True, False, 0.3),
    (67, 60, 6, torch.float16, "softmax", 4, 2, False, False, 0.1),
    (129, 256, 8, torch.bfloat16, "softmax", 8, 4, False, True, 0.2),
    (33, 64, 8, torch.bfloat16, "sigmoid", 1, 1, False, False, 0.0),
    (33, 65, 16, torch.float32, "sigmoid", 5, 2, False, True, 0.5),
    (7, 1024, 16, torch.float32, "softmax", 64, 3, True, True, 0.1),
    (9, 1000, 3, torch.float16, "sigmoid", 1, 1, True, True, 0.0),
    (3, 512, 1, torch.float32, "softmax", 2, 2, False, False, 0.9),
    (40, 8, 8, torch.float32, "softmax", 4, 1, True, False, 0.4),
    (40, 12, 5, torch.float32, "sigmoid", 12, 3, True, True, 0.4),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v).replace("torch.", "") for v in c))
def test_gate_and_gradient(case):
    T, E, K, dt, score, groups, kept, renorm, use_bias, masked = case
    dev = device()
    g = torch.Generator().manual_seed(hash(case[:3]) % 1000)
    logits = (torch.randn(T, E, generator=g) * 2.0).to(dt)
    if masked:
        logits[torch.rand(T, E, generator=g) < masked] = float("-inf")
        logits[T // 2] = float("-inf")  # a token that no expert may take
        logits[0, 0] = float("nan")
    bias = torch.randn(E, generator=g) * 0.2 if use_bias else None
    d_w = torch.randn(T, K, generator=g)
    opts = dict(score=score, num_groups=groups, groups_kept=kept, renormalize=renorm, scale=2.5)
    want_idx, want_w, want_d = reference(logits, K, score, groups, kept, renorm, 2.5, bias, d_w)
    buf = make_buffer(E, 1, 1, T)
    bd = None if bias is None else bias.to(dev)
    print(f"[gate] {case}", flush=True)
    idx, w, _ = buf.gate_topk(logits.to(dev), K, bias=bd, **opts)
    d, _ = buf.gate_topk_backward(d_w.to(dev), logits.to(dev), idx, bias=bd, **opts)
    assert torch.equal(idx.cpu(), want_idx)
    rel = relative(logits, E)
    assert ((w.cpu().double() - want_w).abs() <= rel * want_w.abs() + 1e-37).all()
    assert (w.cpu()[want_idx < 0] == 0).all()
    # every product of the gradient carries the weights' error; |g| and the
    # weighted mean of g bound both terms, and the sum over K adds K roundings
    gmax = d_w.abs().amax(1, keepdim=True).double()
    p = want_d.new_zeros(T, E)
    l = logits.double()
    ok = l > float("-inf")
    p[ok] = 1.0
    if score == "softmax" and not renorm:
        lm = torch.where(ok, l, -1e300)
        p = torch.softmax(lm, 1) * ok
    bound = 2.5 * 2 * gmax * p * (2 * rel + (K + 8) * U)
    half = torch.finfo(dt).eps / 2
    err = (d.cpu().double() - want_d).abs()
    assert (err <= bound + half * (want_d.abs() + bound) + torch.finfo(dt).tiny).all()


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gate_gradient_by_differences(score, renorm):
    """sum(weights * d_w) moves by d_logits * h where a logit moves by h (the
    choice stays): central differences of the definition in fp64, whose own
    error is O(h^2) = 1e-8."""
    dev = device()
    T, E, K, h = 3, 16, 4, 1e-4
    g = torch.Generator().manual_seed(5)
    logits = torch.stack([torch.randperm(E, generator=g) for _ in range(T)]).float() * 0.25
    d_w = torch.randn(T, K, generator=g)
    buf = make_buffer(E, 1, 1, T)
    idx, _, _ = buf.gate_topk(logits.to(dev), K, score=score, renormalize=renorm, scale=1.5)
    d, _ = buf.gate_topk_backward(d_w.to(dev), logits.to(dev), idx, score=score, renormalize=renorm,
                                  scale=1.5)
    d = d.cpu().double()
    for t in range(T):
        for e in range(E):
            v = []
            for s in (h, -h):
                moved = logits.double().clone()
                moved[t, e] += s
                _, w, _ = reference(moved, K, score, 1, 1, renorm, 1.5, None)
                v.append(float((w * d_w.double()).sum()))
            assert abs((v[0] - v[1]) / (2 * h) - float(d[t, e])) < 1e-6


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_gate_extremes(dt):
    """Ties go to the lower index; the type's lowest value is a candidate like
    any other and renormalised weights stay finite and sum to 1."""
    dev = device()
    E, K = 64, 4
    low, big = torch.finfo(dt).min, torch.finfo(dt).max
    rows = torch.stack([torch.zeros(E), torch.full((E,), low), torch.full((E,), big),
                        torch.full((E,), -200.0)]).to(dt)
    rows[3, 10] = -100.0
    buf = make_buffer(E, 1, 1, 4)
    for score in ("softmax", "sigmoid"):
        idx, w, _ = buf.gate_topk(rows.to(dev), K, score=score, renormalize=True)
        idx, w = idx.cpu(), w.cpu()
        for t in (0, 1, 2):
            assert idx[t].tolist() == [0, 1, 2, 3]
            assert (w[t] == 0.25).all()
        assert idx[3].tolist() == [10, 0, 1, 2] and float(w[3, 0]) == 1.0
        d, _ = buf.gate_topk_backward(torch.ones(4, K, device=dev), rows.to(dev), idx.to(dev),
                                      score=score, renormalize=True)
        assert torch.isfinite(d).all()


def test_gate_close_scores():
    """Scores that differ by less than an fp32 rounding are told apart: logits
    one fp32 step apart, in every order, through a bias of zero."""
    dev = device()
    T, E, K = 64, 128, 8
    g = torch.Generator().manual_seed(9)
    ladder = torch.full((E,), 1.0)
    for e in range(1, E):
        ladder[e] = torch.nextafter(ladder[e - 1], torch.tensor(2.0))
    perm = torch.stack([torch.randperm(E, generator=g) for _ in range(T)])
    logits = ladder[perm]
    want = torch.argsort(perm, dim=1, descending=True)[:, :K]
    buf = make_buffer(E, 1, 1, T)
    zero = torch.zeros(E, device=dev)
    for score in ("softmax", "sigmoid"):
        for bias in (None, zero):
            idx, _, _ = buf.gate_topk(logits.to(dev), K, score=score, bias=bias)
            assert torch.equal(idx.cpu(), want), (score, bias is None)


def test_gate_empty_batch_and_refusals():
    from combine_get_dispatch_layout_amd import _capi as C
    dev = device()
    buf = make_buffer(16, 4, 1, 8)
    idx, w, _ = buf.gate_topk(torch.empty(0, 16, device=dev), 2)
    assert idx.shape == (0, 2) and w.shape == (0, 2)
    x = torch.zeros(3, 16, device=dev)
    for bad in (dict(topk=0), dict(topk=17), dict(topk=2, num_groups=3), dict(topk=2, num_groups=0),
                dict(topk=2, num_groups=4, groups_kept=5), dict(topk=2, num_groups=4, groups_kept=0)):
        with pytest.raises(C.MoedxError) as e:
            buf.gate_topk(x, **bad)
        assert e.value.code == C.MOEDX_EINVAL
    for args, kw in (((x[:, :8], 2), {}), ((x.double(), 2), {}), ((x.cpu(), 2), {}),
                     ((x, 2), dict(score="relu")), ((x, 2), dict(bias=torch.zeros(8, device=dev))),
                     ((x, 2), dict(bias=torch.zeros(16, device=dev, dtype=torch.float16)))):
        with pytest.raises(ValueError):
            buf.gate_topk(*args, **kw)
    idx, w, _ = buf.gate_topk(x, 2)
    with pytest.raises(ValueError):
        buf.gate_topk_backward(w[:2], x, idx)
    with pytest.raises(ValueError):
        buf.gate_topk_backward(w, x, idx.int())


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16, torch.float16], ids=lambda d: str(d)[6:])
@pytest.mark.parametrize("renorm", [False, True], ids=["plain", "renorm"])
@pytest.mark.parametrize("form", ["logits", "bias", "groups", "odd groups", "groups and bias"])
@pytest.mark.parametrize("E", [60, 512])
def test_gate_infinite_logits(E, form, renorm, dt):
    """A logit of +inf: the softmax scores are those of the limit (the experts
    with +inf share 1, the others have 0) where they choose, and the token's
    weights are NaN; sigmoid scores are 1.  Other tokens see nothing of it."""
    dev = device()
    K, groups, kept = 4, 1, 1
    if "groups" in form:
        groups, kept = (E // 5, 3) if form == "odd groups" and E == 60 else (4, 2)
    inf = float("inf")
    g = torch.Generator().manual_seed(3)
    plain = torch.randn(E, generator=g) * 2.0
    rows = [plain.clone() for _ in range(6)]
    rows[0][5] = inf
    rows[1][[3, 40]] = inf
    rows[2][:] = inf
    rows[4][:] = -inf  # three candidates only
    rows[4][[7, 2, 50]] = torch.tensor([inf, 0.5, 1.5])
    rows[5][20] = inf  # the bias keeps it from being chosen
    logits = torch.stack(rows).to(dt)
    bias = None
    if "bias" in form:
        bias = torch.randn(E, generator=g) * 0.2
        bias[20] = -30.0
    opts = dict(num_groups=groups, groups_kept=kept, renormalize=renorm, scale=1.5)
    buf = make_buffer(E, 1, 1, 6)
    bd = None if bias is None else bias.to(dev)
    print(f"[gate] infinite logits {E} {form} {renorm} {dt}", flush=True)
    idx, w, _ = buf.gate_topk(logits.to(dev), K, score="softmax", bias=bd, **opts)
    d, _ = buf.gate_topk_backward(torch.ones(6, K, device=dev), logits.to(dev), idx,
                                  score="softmax", bias=bd, **opts)
    idx, w, d = idx.cpu(), w.cpu(), d.cpu()
    l = logits.double()
    for t in range(6):
        if t == 3:
            continue
        ok, top = l[t] > -inf, l[t] == inf
        p = top.double() / top.sum()
        key = l[t] if form == "logits" else p if bias is None else p + bias.double()
        cand = [e for e in range(E) if ok[e]]
        if groups > 1:
            per = E // groups
            sums = []
            for q in range(groups):
                best = sorted((float(key[e]) for e in cand if e // per == q), reverse=True)[:2]
                sums.append(sum(best) if best else -inf)
            keep = sorted(range(groups), key=lambda q: (-sums[q], q))[:kept]
            cand = [e for e in cand if e // per in keep]
        cand = sorted(cand, key=lambda e: (-float(key[e]), e))[:K]
        n = len(cand)
        assert idx[t].tolist() == cand + [-1] * (K - n), t
        assert torch.isnan(w[t, :n]).all() and (w[t, n:] == 0).all(), t
        # the gradient of plain scores is NaN for every candidate, that of
        # renormalised ones where one with +inf was chosen
        if not renorm:
            assert torch.isnan(d[t][ok]).all() and (d[t][~ok] == 0).all(), t
        elif top[cand].any():
            assert torch.isnan(d[t, cand]).all(), t
    alone = [v.cpu() for v in buf.gate_topk(logits[3:4].to(dev), K, score="softmax", bias=bd, **opts)[:2]]
    assert torch.equal(idx[3:4], alone[0]) and torch.equal(w[3:4], alone[1])
    assert torch.isfinite(w[3]).all() and torch.isfinite(d[3]).all()
    idx, w, _ = buf.gate_topk(logits.to(dev), K, score="sigmoid", bias=bd, **opts)
    want_idx, want_w, _ = reference(logits, K, "sigmoid", groups, kept, renorm, 1.5, bias)
    assert torch.equal(idx.cpu(), want_idx)
    assert ((w.cpu().double() - want_w).abs() <= 64 * U * want_w).all()


DTYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.mark.parametrize("renorm", [False, True], ids=["plain", "renorm"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dt", DTYPES, ids=lambda d: str(d)[6:])
@pytest.mark.parametrize("K", [1, 8, 16])
@pytest.mark.parametrize("E", [257, 300, 512, 1000, 1024])
def test_gate_many_experts(E, K, dt, score, renorm):
    """More than 256 experts without bias and groups: their own kernel.  16-bit
    logits have many ties."""
    test_gate_and_gradient((6, E, K, dt, score, 1, 1, renorm, False, 0.1))


@pytest.mark.parametrize("renorm", [False, True], ids=["plain", "renorm"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dt", DTYPES, ids=lambda d: str(d)[6:])
@pytest.mark.parametrize("E", [16, 33, 64, 200, 256])
def test_gate_sixteen_choices(E, dt, score, renorm):
    """The most choices, up to as many as there are experts, and few candidates."""
    test_gate_and_gradient((21, E, 16, dt, score, 1, 1, renorm, False, 0.2))
    test_gate_and_gradient((22, E, 16, dt, score, 1, 1, renorm, False, 0.95))


@pytest.mark.parametrize("E", [512, 1000, 1024])
def test_gate_ties_of_many_experts(E):
    """As test_gate_extremes and test_gate_close_scores, past 256 experts: ties
    within a lane's experts and across lanes go to the lower index, round by
    round, and fp32 neighbours are told apart."""
    dev = device()
    K = 16
    buf = make_buffer(E, 1, 1, 64)
    for dt in DTYPES:
        low, big = torch.finfo(dt).min, torch.finfo(dt).max
        rows = torch.stack([torch.zeros(E), torch.full((E,), low), torch.full((E,), big),
                            torch.full((E,), -3.0)]).to(dt)
        tied = [E - 1, 0, E // 2, E // 2 + 1, 17, 100, 101, 102, 103]
        rows[3, tied] = 1.0
        want3 = sorted(tied) + [e for e in range(E) if e not in tied][:K - len(tied)]
        for score in ("softmax", "sigmoid"):
            idx, w, _ = buf.gate_topk(rows.to(dev), K, score=score, renormalize=True)
            idx, w = idx.cpu(), w.cpu()
            for t in (0, 1, 2):
                assert idx[t].tolist() == list(range(K))
                assert (w[t] == 1.0 / K).all()
            assert idx[3].tolist() == want3
            d, _ = buf.gate_topk_backward(torch.ones(4, K, device=dev), rows.to(dev), idx.to(dev),
                                          score=score, renormalize=True)
            assert torch.isfinite(d).all()
    g = torch.Generator().manual_seed(9)
    ladder = torch.full((E,), 1.0)
    for e in range(1, E):
        ladder[e] = torch.nextafter(ladder[e - 1], torch.tensor(2.0))
    perm = torch.stack([torch.randperm(E, generator=g) for _ in range(64)])
    logits = ladder[perm]
    want = torch.argsort(perm, dim=1, descending=True)[:, :K]
    zero = torch.zeros(E, device=dev)
    for score in ("softmax", "sigmoid"):
        for bias in (None, zero):
            idx, _, _ = buf.gate_topk(logits.to(dev), K, score=score, bias=bias)
            assert torch.equal(idx.cpu(), want), (score, bias is None)
