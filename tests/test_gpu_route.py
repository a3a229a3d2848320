"""The router against its definition in 64 bits: the choice equal, the weights and
the gradient within bounds.

Tolerances. Weights: the header's 16 units of 2^-23 (exponential, sum, division,
the sum over the chosen and its division, the scale), softmax weights that
are not renormalised E / 32 units more for the sum over the experts. The gradient
is a difference of products of such weights and g: 40 units of 2^-23 (and E / 32)
of the magnitudes p |g| and p sum |g| p that it is the difference of, and half a
step of bf16 (2^-8) where that is its type.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
f64, INF = torch.float64, float("inf")


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    from combine_movement_gb300 import build
    build.build()
    from combine_movement_gb300 import ep as mod
    return mod


def order(values):
    """Indices of a list by value, descending; NaN first, equal ones by index."""
    nan = lambda v: v != v
    return sorted(range(len(values)), key=lambda i: (0 if nan(values[i]) else 1,
                                                     0 if nan(values[i]) else -values[i], i))


def scores64(l, score):
    l = l.to(f64).cpu()
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-l))
    m = l.amax(dim=1, keepdim=True)
    p = torch.where(l == -INF, 0.0, torch.exp(l - m))
    return p / p.sum(dim=1, keepdim=True)


def reference(logits, K, bias, score, groups, kept, worth, renorm, scale):
    """(idx, weights in 64 bits) as lists' order gives them."""
    s = scores64(logits, score)
    l = logits.to(f64).cpu()
    b = None if bias is None else bias.to(f64).cpu()
    idx, w = [], []
    for t in range(l.shape[0]):
        E = l.shape[1]
        st, lt = s[t].tolist(), l[t].tolist()
        c = lt if b is None else (s[t] + b).tolist()
        live = [lt[e] != -INF and (b is None or float(b[e]) != -INF) for e in range(E)]
        if groups > 1:
            size, value = E // groups, []
            for g in range(groups):
                of = [c[e] if worth == "max" or b is not None else st[e]
                      for e in range(g * size, (g + 1) * size) if live[e]]
                of = [of[i] for i in order(of)]
                value.append((of[0] if worth == "max" or len(of) < 2 else of[0] + of[1]) if of else None)
            on = [g for g in range(groups) if value[g] is not None]
            stay = {on[i] for i in order([value[g] for g in on])[:kept]}
            live = [live[e] and e // size in stay for e in range(E)]
        es = [e for e in range(E) if live[e]]
        chosen = [es[i] for i in order([c[e] for e in es])[:K]]
        wt = [st[e] for e in chosen]
        if renorm:
            if score == "softmax":  # by the chosen alone: scores below 64 bits keep their ratios
                top = max([lt[e] for e in chosen], default=0.0)
                wt = torch.exp(torch.tensor([lt[e] for e in chosen], dtype=f64) - top).tolist()
            total = sum(wt)
            wt = [v / total for v in wt]
        idx.append(chosen + [-1] * (K - len(chosen)))
        w.append([v * scale for v in wt] + [0.0] * (K - len(chosen)))
    return torch.tensor(idx), torch.tensor(w, dtype=f64)


def logits_of(T, E, dtype, seed, masked=0.0, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    l = torch.randn((T, E), generator=g) * spread
    if masked:
        l[torch.rand((T, E), generator=g) < masked] = -INF
        l[::5] = -INF
    return l.to(dtype).cuda()


def check(ep, logits, K, bias=None, score="softmax", groups=1, kept=1, worth="max", renorm=True,
          scale=1.0):
    idx, w = ep.route(logits, K, bias, score, groups, kept, worth, renorm, scale)
    ref_idx, ref_w = reference(logits, K, bias, score, groups, kept, worth, renorm, scale)
    assert torch.equal(idx.cpu(), ref_idx)
    units = 16 + (0 if renorm else logits.shape[1] / 32)
    err = (w.cpu().to(f64) - ref_w).abs()
    assert bool((err <= units * 2.0 ** -23 * ref_w.abs() + 2.0 ** -140)[~ref_w.isnan()].all())
    assert torch.equal(w.cpu().isnan(), ref_w.isnan())
    return idx, w


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (3, 5, 5), (9, 32, 8), (7, 33, 4), (33, 60, 4),
                                   (2, 64, 32), (17, 100, 6), (64, 256, 8), (5, 500, 3),
                                   (4, 1000, 32), (3, 1025, 8), (2, 4096, 16)])
@pytest.mark.parametrize("biased,renorm", [(False, True), (True, False), (True, True), (False, False)])
def test_sizes(ep, dtype, score, T, E, K, biased, renorm):
    bias = torch.randn(E, generator=torch.Generator().manual_seed(E)).cuda() * 0.1 if biased else None
    check(ep, logits_of(T, E, dtype, T + E), K, bias, score, renorm=renorm, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("worth", ["max", "top2"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("E,groups,kept,K", [(256, 8, 4, 8), (64, 8, 1, 8), (60, 4, 2, 6), (32, 32, 5, 5),
                                             (256, 2, 1, 8), (160, 8, 3, 6), (512, 16, 4, 8),
                                             (36, 3, 2, 7), (64, 16, 16, 4), (1024, 32, 2, 32)])
@pytest.mark.parametrize("masked", [0.0, 0.6])
def test_groups(ep, score, worth, biased, E, groups, kept, K, masked):
    bias = torch.randn(E, generator=torch.Generator().manual_seed(3)).cuda() * 0.1 if biased else None
    check(ep, logits_of(24, E, torch.float32, E + groups, masked), K, bias, score, groups, kept, worth)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [None, "zero", "equal", "random"])
@pytest.mark.parametrize("groups,worth", [(1, "max"), (8, "max"), (8, "top2")])
def test_ties_go_to_the_lower_index(ep, score, bias, groups, worth):
    E, g = 64, torch.Generator().manual_seed(1)
    l = torch.randint(-2, 3, (40, E), generator=g).float()  # five values, most of them equal
    l[0] = 0.0
    l[1, ::2], l[1, 1::2] = 0.0, -0.0
    b = {None: None, "zero": torch.zeros(E), "equal": torch.full((E,), -0.3),
         "random": torch.randint(-1, 2, (E,), generator=g) * 0.25}[bias]
    check(ep, l.cuda(), 8, None if b is None else b.cuda(), score, groups, max(1, groups // 2), worth)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,worth", [(1, "max"), (4, "top2")])
def test_orders_that_32_bits_cannot_settle(ep, score, groups, worth):
    """Biases that make up for the scores' differences up to parts in 10^9 to 10^12."""
    E, T = 64, 24
    g = torch.Generator().manual_seed(5)
    l = torch.randn(E, generator=g)
    s = scores64(l[None], score)[0]
    for step in (1e-9, 1e-12):
        l2 = l[None].repeat(T, 1)
        bias = (s.max() + 0.5 - s).float()  # rounded: c differs by up to 2^-25
        check(ep, l2.cuda(), 8, bias.cuda(), score, groups, max(1, groups // 2), worth)
        near = (torch.arange(E) % 7) * step
        check(ep, l2.cuda(), 8, (s.max() + 0.5 - s + near).float().cuda(), score, groups,
              max(1, groups // 2), worth)


@pytest.mark.parametrize("E,K", [(256, 8), (64, 4), (60, 7), (500, 3), (32, 32), (1000, 32)])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("groups,worth", [(1, "max"), (4, "max"), (4, "top2")])
def test_values_a_few_units_apart(ep, E, K, biased, groups, worth):
    """Logits (with a bias, their scores' neighbours too) one to forty units of 2^-23 apart,
    so that integers without their last bits put them in a wrong order, at the border
    of what is chosen too."""
    g = torch.Generator().manual_seed(E)
    l = 1.0 + torch.randint(0, 40, (48, E), generator=g).float() * 2.0 ** -23
    l[::3] = 1.0 + torch.randint(0, 3, (16, E), generator=g).float() * 2.0 ** -23
    l[1::6, ::2] += 0.5
    b = torch.randint(0, 3, (E,), generator=g).float() * 2.0 ** -24 if biased else None
    kept = groups if E // groups * (groups // 2) < K else max(1, groups // 2)
    check(ep, l.cuda(), K, None if b is None else b.cuda(), "sigmoid", groups, kept, worth)
    check(ep, l.cuda(), K, None if b is None else b.cuda(), "softmax", groups, kept, worth)


def test_scores_beyond_32_bits(ep):
    """Logits whose scores underflow keep their order and their ratios."""
    l = torch.tensor([[-200.0, -201.0, -199.5, -300.0], [-120.0, -90.0, -104.0, -119.0],
                      [90.0, 88.0, 100.0, -100.0], [3e38, -3e38, 0.0, 1.0]]).cuda()
    for score in ("softmax", "sigmoid"):
        for bias in (None, torch.zeros(4).cuda()):
            check(ep, l, 2, bias, score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_nothing_left(ep, score):
    l = torch.full((3, 8), -INF).cuda()
    l[1, 5] = 0.0
    idx, w = check(ep, l, 3, None, score)
    assert idx.tolist() == [[-1] * 3, [5, -1, -1], [-1] * 3] and w[0].tolist() == [0.0] * 3
    bias = torch.full((8,), -INF).cuda()
    bias[2] = -1e30
    idx, _ = check(ep, torch.zeros(2, 8).cuda(), 3, bias, score)
    assert idx.tolist() == [[2, -1, -1]] * 2
    idx, w = ep.route(torch.zeros(0, 8).cuda(), 3)
    assert idx.shape == (0, 3) and w.shape == (0, 3)


def test_many_tokens(ep):
    """More tokens than warps at a time; the choice as torch sorts logits, the weights
    as torch's softmax over them."""
    l = logits_of(70001, 128, torch.float32, 12)
    idx, w = ep.route(l, 6)
    top, want = l.sort(dim=1, descending=True, stable=True)
    assert torch.equal(idx, want[:, :6])
    ref = torch.softmax(top[:, :6].to(f64), dim=1)
    assert bool(((w.to(f64) - ref).abs() <= 16 * 2.0 ** -23 * ref).all())


@pytest.mark.parametrize("groups", [1, 4])
def test_nan_is_chosen_and_shows(ep, groups):
    l = logits_of(6, 32, torch.float32, 9)
    l[1, 17] = float("nan")
    l[3, 4] = INF
    for bias in (None, torch.rand(32).cuda() * 0.1):
        idx, w = check(ep, l, 4, bias, "sigmoid", groups, max(1, groups // 2), "top2", True)
        assert int(idx[1, 0]) == 17 and bool(w[1].isnan().all())
        assert not bool(w[[0, 2, 3, 4, 5]].isnan().any())
        _, w = ep.route(l, 4, bias, "softmax", renormalize=False)
        assert bool(w[1].isnan().all()) and not bool(w[[0, 2, 4, 5]].isnan().any())


# -- the gradient ---------------------------------------------------------------

def grad64(dw, logits, idx, score, renorm, scale):
    """The definition's, by torch's own differentiation in 64 bits, and the
    magnitudes that it is the difference of."""
    l = logits.to(f64).cpu().requires_grad_(True)
    idx, dw = idx.cpu(), dw.to(f64).cpu()
    live = (idx >= 0) & (l.detach().gather(1, idx.clamp_min(0)) != -INF)
    at = idx.clamp_min(0)
    ok = torch.where(l == -INF, -1e4, l)  # (its score is 0 all the same)
    if score == "sigmoid":
        s = torch.sigmoid(ok)
    else:
        s = torch.softmax(ok, dim=1)
    p = torch.where(live, s.gather(1, at), 0.0)
    if renorm and score == "softmax":
        # the same weights from the chosen logits alone: through every expert's
        # score the others' gradients, which are 0, come out as 64 bits' rounding
        # of a difference of equal numbers
        p = torch.where(live, torch.softmax(torch.where(live, ok.gather(1, at), -1e4), dim=1), 0.0)
    total = p.sum(dim=1, keepdim=True)
    if renorm:
        p = torch.where(live, p / torch.where(total == 0, 1.0, total), 0.0)
    (torch.where(live, p * dw, 0.0).sum() * scale).backward()
    g = torch.where(live, dw * scale, 0.0).abs()
    pd, sd = p.detach(), s.detach()
    size = torch.zeros_like(sd).scatter_add_(1, at, torch.where(live, pd * g, 0.0))
    dot = (pd * g).sum(dim=1, keepdim=True)
    if renorm:
        size.scatter_add_(1, at, torch.where(live, pd * dot, 0.0))
    elif score == "softmax":
        size = sd * (torch.zeros_like(sd).scatter_add_(1, at, g) + dot)
    return torch.where(logits.cpu() == -INF, 0.0, l.grad), size


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,E,K,masked", [(1, 1, 1, 0.0), (5, 33, 7, 0.0), (64, 256, 8, 0.0),
                                          (40, 60, 4, 0.5), (3, 4096, 32, 0.1), (129, 128, 1, 0.2)])
def test_gradient(ep, dtype, score, renorm, T, E, K, masked):
    l = logits_of(T, E, dtype, T * E, masked)
    idx, _ = ep.route(l, K, None, score, renormalize=renorm)
    dw = torch.randn((T, K), generator=torch.Generator().manual_seed(T)).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    d = torch.full_like(l, float("nan"))
    ep.ep_route_grad(dw, l, idx, d, score, renorm, 2.5, status)
    assert ep.ep_get_status(status) == ep.EP_OK
    want, size = grad64(dw, l, idx, score, renorm, 2.5)
    half = 2.0 ** -8 if dtype is torch.bfloat16 else 0.0
    bound = (40 + E / 32) * 2.0 ** -23 * size + half * want.abs() + 2.0 ** -130
    assert bool(((d.cpu().to(f64) - want).abs() <= bound).all())


def test_gradient_by_differences(ep):
    """(w(l + h) - w(l - h)) / 2h, in the direction of a random change of the
    logits that leaves the choice as it is."""
    l = logits_of(16, 64, torch.float32, 2).cpu().to(f64)
    g = torch.Generator().manual_seed(8)
    step = torch.randn(l.shape, generator=g, dtype=f64)
    dw = torch.randn((16, 6), generator=g)
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            lf = l.float().cuda()
            idx, _ = ep.route(lf, 6, None, score, renormalize=renorm)
            d = ep.route_grad(dw.cuda(), lf, idx, score, renorm).cpu().to(f64)

            def weights(x):
                s = scores64(x, score).gather(1, idx.cpu())
                return s / s.sum(dim=1, keepdim=True) if renorm else s
            h = 1e-5
            slope = ((weights(l.float().to(f64) + h * step) - weights(l.float().to(f64) - h * step))
                     / (2 * h) * dw).sum(dim=1)
            assert torch.allclose((d * step).sum(dim=1), slope, rtol=1e-4, atol=2e-5)


def test_gradient_skips_and_reports_bad_entries(ep):
    l = logits_of(4, 16, torch.float32, 4)
    idx = torch.tensor([[1, 2], [1, 16], [-2, 3], [-1, -1]]).cuda()
    dw = torch.ones((4, 2)).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    d = ep.route_grad(dw, l, idx, "sigmoid", False, status=status)
    assert ep.ep_get_status(status) == ep.EP_ERR_BAD_EXPERT
    clean = ep.route_grad(dw, l, torch.where((idx < 0) | (idx > 15), -1, idx), "sigmoid", False)
    assert torch.equal(d, clean) and not bool(d[3].any())
    ep.route_grad(dw, l, torch.full_like(idx, 1 << 40), status=status)  # far outside


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_of_an_expert_chosen_twice(ep, score, renorm):
    l = logits_of(5, 40, torch.float32, 6)
    idx = torch.randint(0, 3, (5, 6), generator=torch.Generator().manual_seed(2)).cuda()
    dw = torch.randn((5, 6), generator=torch.Generator().manual_seed(3)).cuda()
    d = ep.route_grad(dw, l, idx, score, renorm)
    want, size = grad64(dw, l, idx, score, renorm, 1.0)
    assert bool(((d.cpu().to(f64) - want).abs() <= 48 * 2.0 ** -23 * size).all())


def test_route_feeds_layout_and_survives_a_graph(ep):
    l = logits_of(300, 64, torch.float32, 7, masked=0.3)
    bias = torch.rand(64).cuda() * 0.1
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        idx, w = ep.route(l, 4, bias, "sigmoid")
        ep.get_dispatch_layout(idx, 64)
    torch.cuda.synchronize()
    idx2, w2 = torch.empty_like(idx), torch.empty_like(w)
    d = torch.empty_like(l)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        ep.ep_route(l, idx2, w2, bias, "sigmoid")
        ep.ep_route_grad(w2, l, idx2, d, "sigmoid")
        counts, _, slot = ep.get_dispatch_layout(idx2, 64)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(idx, idx2) and torch.equal(w, w2)
    assert torch.equal(d, ep.route_grad(w, l, idx, "sigmoid"))
    assert torch.equal(slot < 0, idx < 0) and int(counts.sum()) == int((idx >= 0).sum())
    l.copy_(logits_of(300, 64, torch.float32, 11))
    graph.replay()
    torch.cuda.synchronize()
    again, _ = ep.route(l, 4, bias, "sigmoid")
    assert torch.equal(idx2, again)
