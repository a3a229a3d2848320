"""Dense products and their gradients against the formulas in 64 bits.

Tolerances. A sum of K products takes at most K + 8 additions (the tensor core's,
those of a tile's parts, the bias), each of which may lose one unit of 2^-23 of the sum
of magnitudes so far: e = (K + 8) 2^-23 (sum |p| + |bias|). The activations have
slopes of at most 1.13, and errors of their own: silu (8 + 2 |z|) 2^-23 of its
value, gelu (16 + z^2) 2^-23 (the argument's rounding, times z^2 in the tail), and
the spacing of fp32's subnormals. swiglu takes e through both factors. The residual's
addition and the products add 4 units of 2^-23. bf16 results are off by half a step,
2^-8 of their value. Sums of dz in bf16 take its rounding, 2^-8 |dz|, through
the product's magnitudes.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
f64, bf = torch.float64, torch.bfloat16
U = 2.0 ** -23
ACTS = ["none", "relu", "gelu", "silu", "swiglu"]


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    from combine_movement_gb300 import build
    build.build()
    from combine_movement_gb300 import ep as mod
    return mod


def rand(*shape, seed=0, dtype=bf, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def act64(z, act):
    """(act(z), bound on the activation's own error, largest slope times |.|)."""
    if act == "relu":
        return z.clamp_min(0), 0 * z
    if act == "gelu":
        y = z * 0.5 * torch.special.erfc(-z * 0.5 ** 0.5)
        return y, (16 + z * z) * U * y.abs()
    if act == "silu":
        y = z * torch.sigmoid(z)
        return y, (8 + 2 * z.abs()) * U * y.abs()
    return z, 0 * z


def linear64(x, w, bias, act, residual):
    """(y, z, bounds on the errors of y and z before bf16)."""
    K = x.shape[1]
    z = x.to(f64) @ w.to(f64).T
    size = x.to(f64).abs() @ w.to(f64).abs().T
    if bias is not None:
        z, size = z + bias.to(f64), size + bias.to(f64).abs()
    e = (K + 8) * U * size
    if act == "swiglu":
        n = w.shape[0] // 2
        g, u, eg, eu = z[:, :n], z[:, n:], e[:, :n], e[:, n:]
        s, es = act64(g, "silu")
        y = s * u
        ey = (1.13 * eg + es) * (u.abs() + eu) + s.abs() * eu + 4 * U * y.abs()
    else:
        y, ey = act64(z, act)
        ey = ey + 1.13 * e
    if residual is not None:
        y = y + residual.to(f64)
    return y, z, ey + 4 * U * y.abs() + 2.0 ** -126, e


def close(got, want, err):
    half = 2.0 ** -8 if got.dtype is bf else 0.0
    bad = (got.to(f64) - want).abs() > err + half * (want.abs() + err)
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:4].tolist())


def case(ep, M, N, K, act="none", bias=False, residual=False, out=bf, keep=False, seed=0):
    wide = 2 * N if act == "swiglu" else N
    x, w = rand(M, K, seed=seed), rand(wide, K, seed=seed + 1, scale=K ** -0.5)
    b = rand(wide, seed=seed + 2, dtype=torch.float32) if bias else None
    r = rand(M, N, seed=seed + 3, dtype=out) if residual else None
    guard = 64  # what lies behind the results stays
    flat = torch.full((M * N + guard,), 7.0, dtype=out, device="cuda")
    zflat = torch.full((M * wide + guard,), 7.0, dtype=bf, device="cuda")
    y, z = flat[:M * N].view(M, N), zflat[:M * wide].view(M, wide) if keep else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ep.ep_linear(x, w, y, b, act, r, z, status)
    assert ep.ep_get_status(status) == ep.EP_OK
    want, wz, err, ez = linear64(x, w, b, act, r)
    close(y, want, err)
    assert bool((flat[M * N:] == 7.0).all()) and bool((zflat[M * wide:] == 7.0).all())
    if keep:
        close(z, wz, ez)
    return x, w, b, r, y


@pytest.mark.parametrize("M", [1, 2, 3, 8, 15, 17, 33, 64, 65, 127, 128, 129, 300])
@pytest.mark.parametrize("N,K", [(256, 512), (8, 8), (60, 1000), (1075, 264), (130, 2056)])
def test_sizes(ep, M, N, K):
    case(ep, M, N, K, out=torch.float32, seed=M)
    case(ep, M, N, K, bias=True, residual=True, seed=M)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K", [(5, 192, 128), (130, 300, 200), (70, 77, 72), (1, 1, 8),
                                   (257, 512, 2048), (16, 1030, 4096)])
@pytest.mark.parametrize("out", [bf, torch.float32])
def test_epilogues(ep, act, M, N, K, out):
    case(ep, M, N, K, act, True, True, out, True, seed=N)
    case(ep, M, N, K, act, False, False, out, True, seed=N + 9)


def test_many_tiles(ep):
    """More tiles than SMs, so that CTAs take several, with odd edges."""
    case(ep, 3001, 4100, 136, "silu", True, True, bf, True)
    case(ep, 2050, 2100, 72, "swiglu", True, True, bf, True)
    case(ep, 9000, 1000, 1048, residual=True, out=torch.float32)


# Shapes that tiles of each kind are made for, by which CTAs and with which sums (a CTA
# alone, 2 to 16 that share one, pairs; long k in fp32).
@pytest.mark.parametrize("M,N,K", [(1000, 1000, 1000), (600, 1030, 1096), (16, 256, 7168), (130, 260, 4104),
                                   (512, 250, 2056), (2000, 256, 1544), (3001, 2100, 1100 + 4),
                                   (5000, 1000, 72), (9000, 260, 2056)])
@pytest.mark.parametrize("act,out", [("none", bf), ("none", torch.float32), ("swiglu", torch.float32),
                                     ("gelu", bf)])
def test_tiles_of_every_kind(ep, M, N, K, act, out):
    case(ep, M, N, K, act, out=out, seed=K)
    case(ep, M, N, K, act, True, True, out, True, seed=K + 1)


# Sums of positive numbers: what the tensor cores' steps lose adds up. A step takes at
# least 8 products and loses at most a unit of the sum so far, which grows evenly: of
# 1024 products at most 64.5 units of 2^-23 of their sum. Adding P parts loses at most
# half a unit of the sum so far each time, (P + 1) / 4 in all. (The numbers lie in 1 to 2,
# so that no sum of 8 is further than a quarter from the others: 1.25 times that.) In one
# sum of K products it would be up to K / 16 units.
@pytest.mark.parametrize("M,N,K", [(128, 256, 32768), (2000, 256, 7168), (1000, 1000, 7168), (512, 512, 16384),
                                   (300, 2048, 16384), (4096, 4096, 8192), (5000, 64, 8192)])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_fp32_results_are_of_short_sums(ep, M, N, K, act):
    x, w = rand(M, K).uniform_(1, 2), rand(N, K, seed=1).uniform_(1, 2)
    units = 1.25 * (64.5 + (K / 1024 + 1) / 4)
    if act == "swiglu":  # gates of 1, by the first product; silu and products: 10 + 4
        N, units = N // 2, units + 14
        w[:N], w[:N, 0], x[:, 0] = 0, 1, 1
    y = torch.empty(M, N, device="cuda")
    ep.ep_linear(x, w, y, activation=act)
    want = x.to(f64) @ w[-N:].to(f64).T
    if act == "swiglu":
        want = want * torch.sigmoid(torch.ones((), dtype=f64, device="cuda"))
    assert float(((y.to(f64) - want).abs() / want).max()) < units * U


@pytest.mark.parametrize("M,N,K", [(8192, 256, 2048), (16384, 256, 1024), (16384, 64, 512), (9000, 1000, 520)])
def test_fp32_weight_gradients_are_of_short_sums(ep, M, N, K):
    dz, x = rand(M, ep.linear_pitch(N)).uniform_(1, 2), rand(M, K, seed=1).uniform_(1, 2)
    d_w = torch.empty(N, K, device="cuda")
    ep.ep_linear_grad_weight(dz, x, d_w)
    want = dz[:, :N].to(f64).T @ x.to(f64)
    units = 1.25 * (64.5 + (M / 1024 + 1) / 4)
    assert float(((d_w.to(f64) - want).abs() / want).max()) < units * U


@pytest.mark.parametrize("act", ACTS)
def test_infinities_and_nan_pass_through(ep, act):
    x, w = rand(40, 64), rand(96, 64, seed=1)
    x[3, 5], x[7, 9] = float("nan"), float("inf")
    y = torch.empty(40, 96 // (2 if act == "swiglu" else 1), device="cuda")
    ep.ep_linear(x, w, y, activation=act)
    assert bool(y[3].isnan().all()) and not bool(y[7].isfinite().all())
    rest = [i for i in range(40) if i not in (3, 7)]
    assert bool(y[rest].isfinite().all())


def test_the_residual_may_be_the_result(ep):
    x, w, r = rand(200, 128), rand(264, 128, seed=1), rand(200, 264, seed=2)
    want = ep.linear(x, w, residual=r)
    ep.ep_linear(x, w, r, residual=r)
    assert torch.equal(r, want)


def test_equal_calls_give_equal_bits(ep):
    for M, N, K in ((1, 512, 7168), (128, 256, 4096), (700, 900, 1024)):
        x, w = rand(M, K), rand(N, K, seed=1)
        first = ep.linear(x, w, out_dtype=torch.float32)
        for _ in range(3):
            assert torch.equal(first, ep.linear(x, w, out_dtype=torch.float32))


def test_no_rows(ep):
    assert ep.linear(rand(0, 64), rand(8, 64)).shape == (0, 8)
    d_w = torch.full((8, 64), 3.0, device="cuda")
    ep.ep_linear_grad_weight(rand(0, 8), rand(0, 64), d_w, accumulate=True)
    assert bool((d_w == 3.0).all())
    ep.ep_linear_grad_weight(rand(0, 8), rand(0, 64), d_w)
    assert not bool(d_w.any())
    d_b = torch.full((8,), 3.0, device="cuda")
    ep.ep_linear_act_grad(rand(0, 8), rand(0, 8), rand(0, 8), d_b, "silu")
    assert not bool(d_b.any())


def test_results_past_32_bit_offsets(ep):
    M, N, K = 33000, 65544, 8  # 2.16e9 results
    x, w = rand(M, K), rand(N, K, seed=1)
    y = ep.linear(x, w)
    for rows in (slice(0, 3), slice(M - 5, M)):
        want, _, err, _ = linear64(x[rows], w, None, "none", None)
        close(y[rows], want, err)


# -- gradients ------------------------------------------------------------------

def slopes64(z, dy, act):
    """dz in 64 bits."""
    z, dy = z.to(f64), dy.to(f64)
    if act == "swiglu":
        n = dy.shape[1]
        g, u = z[:, :n], z[:, n:]
        s = torch.sigmoid(g)
        return torch.cat([dy * u * (s + g * s * (1 - s)), dy * g * s], dim=1)
    if act == "relu":
        return dy * (z > 0)
    if act == "gelu":
        return dy * (0.5 * torch.special.erfc(-z * 0.5 ** 0.5)
                     + z * torch.exp(-z * z / 2) * (2 * torch.pi) ** -0.5)
    if act == "silu":
        s = torch.sigmoid(z)
        return dy * (s + z * s * (1 - s))
    return dy


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [bf, torch.float32])
@pytest.mark.parametrize("M,N", [(1, 8), (3, 60), (129, 57), (1000, 264), (77, 1), (4097, 130)])
def test_act_grad(ep, act, dtype, M, N):
    """slopes: (40 + 4 z^2) units of 2^-23 of their terms' magnitudes, at most 1 + |z|
    of dy (and |u| of it); the sums (M + 16) units more."""
    wide = 2 * N if act == "swiglu" else N
    pitch = ep.linear_pitch(wide)
    dy, z = rand(M, N, dtype=dtype), rand(M, wide, seed=1, scale=2.0)
    dz = torch.full((M, pitch), 7.0, dtype=bf, device="cuda")
    d_b = torch.full((wide,), float("nan"), device="cuda")
    ep.ep_linear_act_grad(dy, z if act != "none" else None, dz, d_b, act)
    want = slopes64(z, dy, act)
    a = z.to(f64).abs()
    terms = dy.to(f64).abs()
    if act == "swiglu":
        g, u = a[:, :N], a[:, N:]
        terms = torch.cat([terms * u * (1 + g), terms * g], dim=1)
        a = torch.cat([g, g], dim=1)
    elif act != "none":
        terms = terms * (1 + a)
    err = (40 + 4 * a * a) * U * terms + 2.0 ** -126 if act != "none" else 0 * terms
    close(dz[:, :wide], want, err)
    assert bool((dz[:, wide:] == 7.0).all())
    sums = (d_b.to(f64) - want.sum(dim=0)).abs()
    assert bool((sums <= err.sum(dim=0) + (M + 16) * U * (want.abs() + err).sum(dim=0)).all())
    dz2 = torch.empty_like(dz)
    ep.ep_linear_act_grad(dy, z if act != "none" else None, dz2, None, act)
    assert torch.equal(dz[:, :wide], dz2[:, :wide])


@pytest.mark.parametrize("M,N,K", [(1, 8, 8), (5, 60, 64), (130, 57, 136), (300, 256, 1000),
                                   (64, 2050, 72), (1000, 33, 520), (2049, 300, 2056),
                                   (1500, 2050, 2056), (4100, 60, 2048)])
def test_grad_products(ep, M, N, K):
    dz = torch.full((M, ep.linear_pitch(N)), float("nan"), dtype=bf, device="cuda")
    dz[:, :N] = rand(M, N)
    x, w = rand(M, K, seed=1), rand(N, K, seed=2)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    d, dabs = dz[:, :N].to(f64), dz[:, :N].to(f64).abs()
    flat = torch.full((M * K + 64,), 7.0, dtype=bf, device="cuda")
    ep.ep_linear_grad_input(dz, w, flat[:M * K].view(M, K), status)
    close(flat[:M * K].view(M, K), d @ w.to(f64), (N + 8) * U * (dabs @ w.to(f64).abs()))
    assert bool((flat[M * K:] == 7.0).all())
    size = (M + 8) * U * (dabs.T @ x.to(f64).abs())
    for dtype in (bf, torch.float32):
        d_w = torch.full((N, K), float("nan"), dtype=dtype, device="cuda")
        ep.ep_linear_grad_weight(dz, x, d_w, status=status)
        close(d_w, d.T @ x.to(f64), size)
        start = rand(N, K, seed=3, dtype=dtype)
        d_w = start.clone()
        ep.ep_linear_grad_weight(dz, x, d_w, accumulate=True, status=status)
        total = d.T @ x.to(f64) + start.to(f64)
        close(d_w, total, size + 2 * U * total.abs())
    assert ep.ep_get_status(status) == ep.EP_OK


def test_calls_on_a_stream_and_in_a_graph(ep):
    """Two captured graphs and a second stream give the first call's bits."""
    x, w, r = rand(130, 2048), rand(520, 2048, seed=1), rand(130, 520, seed=2)
    want = ep.linear(x, w, activation="gelu", residual=r)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    assert torch.equal(ep.linear(x, w, activation="gelu", residual=r, stream=s), want)
    s.synchronize()
    outs, graphs = [], []
    for _ in range(2):
        y, d_w = torch.empty_like(want), torch.empty_like(w)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ep.ep_linear(x, w, y, activation="gelu", residual=r)
            ep.ep_linear_grad_weight(y, x, d_w)
        outs.append((y, d_w))
        graphs.append(graph)
    for graph in graphs + graphs:
        graph.replay()
    torch.cuda.synchronize()
    d_w = torch.empty_like(w)
    ep.ep_linear_grad_weight(want, x, d_w)
    for y, d in outs:
        assert torch.equal(y, want) and torch.equal(d, d_w)


def test_two_streams_at_once(ep):
    """Calls that run beside each other, on tiles of different kinds."""
    shapes = [(128, 256, 7168), (700, 512, 2048), (1, 2048, 7168), (3000, 1024, 512)]
    args = [(rand(M, K, seed=i), rand(N, K, seed=i + 9)) for i, (M, N, K) in enumerate(shapes)]
    want = [ep.linear(x, w, out_dtype=torch.float32) for x, w in args]
    streams = [torch.cuda.Stream() for _ in args]
    torch.cuda.synchronize()
    for _ in range(4):
        got = [ep.linear(x, w, out_dtype=torch.float32, stream=s) for (x, w), s in zip(args, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_in_a_partition(ep):
    """On a partition's stream, where tiles are not shared between CTAs: the same
    values within the sums' error."""
    raw, _, sms, _ = ep.ep_sm_partition(24)
    s = torch.cuda.ExternalStream(raw)
    x, w = rand(64, 4096), rand(512, 4096, seed=1, scale=1 / 64)
    torch.cuda.synchronize()
    y = ep.linear(x, w, out_dtype=torch.float32, stream=s)
    d_b = torch.empty(512, device="cuda")
    ep.ep_linear_act_grad(y, None, None, d_b, stream=s)
    s.synchronize()
    want, _, err, _ = linear64(x, w, None, "none", None)
    close(y, want, err)
    assert torch.allclose(d_b.to(f64), y.to(f64).sum(dim=0), rtol=0,
                          atol=float(80 * U * y.abs().sum(dim=0).max()))


@pytest.mark.parametrize("M,N", [(5000, 512), (3000, 57), (700, 6000)])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_act_grad_in_a_partition(ep, M, N, act):
    """Sums over many rows where a partition's SMs may hold no cluster (bounds: those of
    test_act_grad)."""
    raw, _, sms, _ = ep.ep_sm_partition(8)
    s = torch.cuda.ExternalStream(raw)
    wide = 2 * N if act == "swiglu" else N
    dy, z = rand(M, N), rand(M, wide, seed=1)
    dz = torch.empty(M, ep.linear_pitch(wide), dtype=bf, device="cuda")
    d_b = torch.full((wide,), float("nan"), device="cuda")
    torch.cuda.synchronize()
    ep.ep_linear_act_grad(dy, z if act != "none" else None, dz, d_b, act, stream=s)
    s.synchronize()
    want = slopes64(z, dy, act)
    err = 0 * want
    if act == "swiglu":
        g, u, d = z[:, :N].to(f64).abs(), z[:, N:].to(f64).abs(), dy.to(f64).abs()
        err = (40 + 4 * torch.cat([g, g], 1) ** 2) * U * torch.cat([d * u * (1 + g), d * g], 1) + 2.0 ** -126
    close(dz[:, :wide], want, err)
    sums = (d_b.to(f64) - want.sum(dim=0)).abs()
    assert bool((sums <= err.sum(dim=0) + (M + 16) * U * (want.abs() + err).sum(dim=0)).all())
