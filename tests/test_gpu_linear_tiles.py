"""Every way in which a dense product's tiles are made: the rule is asked for a grid of
sizes what it would do, and the smallest sizes of each answer (who works on a tile, how
many CTAs share it, whether its sums are added up from parts, gated or not, how many
values of a row are stored at once, rounded sums alone or with an epilogue) are run
against the formula in 64 bits, with the tolerances of test_gpu_linear.py."""
import functools

import pytest
import torch

from test_gpu_linear import U, case, close, rand

pytestmark = pytest.mark.gpu
f64, bf, f32 = torch.float64, torch.bfloat16, torch.float32

ROWS = [1, 2, 3, 4, 5, 8, 17, 33, 64, 65, 100, 128, 129, 200, 256, 300, 400, 512, 700, 1000, 1500, 2000,
        3000, 4000, 5000, 8000, 9000, 16000, 32000]
COLS = [8, 30, 33, 60, 64, 77, 128, 130, 200, 256, 301, 400, 512, 514, 700, 1000, 1030, 1075, 2000, 2050,
        3001, 4000, 4100, 7000, 8000, 16000]
LONG = [8, 64, 72, 128, 136, 256, 264, 512, 1000, 1024, 1096, 2048, 2056, 3200, 4096, 5000, 7000, 8192, 8200,
        16000, 16400, 33000, 66000, 132000, 263000]
MOST = 6e10  # products of a run


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    from combine_movement_gb300 import build
    build.build()
    from combine_movement_gb300 import ep as mod
    return mod


def width(n):
    return 4 if n % 4 == 0 else 2 if n % 2 == 0 else 1


@functools.lru_cache(None)
def ways(ep, product):
    """{way: the smallest (M, N, K, activation, out type, epilogue) that it is taken for}"""
    found = {}
    for M in (ROWS if product != "grad_weight" else LONG):
        for N in (COLS if product != "grad_input" else [8 * n for n in LONG if n < 4000] + COLS):
            for K in (LONG if product == "linear" else [n for n in COLS if n % 8 == 0]):
                if M * N * K > MOST or max(M * K, N * K, M * N) > 3e8:
                    continue
                for act in (("none", "swiglu") if product == "linear" else ("none",)):
                    for out in ((bf, f32) if product != "grad_input" else (bf,)):
                        for epilogue in ((False, True) if product != "grad_input" else (False,)):
                            way = ep.ep_linear_tiles(product, M, N, K, act, out, epilogue)
                            assert way is not None
                            cols = N if product == "linear" else K
                            key = way + (act == "swiglu", width(cols), epilogue)
                            cost = M * N * K * (2 if act == "swiglu" else 1)
                            if key not in found or cost < found[key][0]:
                                found[key] = (cost, M, N, K, act, out, epilogue)
    return {k: v[1:] for k, v in sorted(found.items())}


def test_the_grid_reaches_all(ep):
    """Each kind of tile, each number of CTAs to one, in parts and not, gated and not."""
    found = ways(ep, "linear")
    kinds = {(k[0], k[1]) for k in found}
    assert {k for k, _ in kinds} == set(ep.TILES)
    assert {n for k, n in kinds if k == "shared 64"} == {2, 4, 8, 16}
    for kind in ep.TILES[1:]:
        for in_parts in (False, True):
            for gated in (False, True):
                assert any(k[0] == kind and k[2] == in_parts and k[3] == gated for k in found), (
                    kind, in_parts, gated)


def test_products(ep):
    for way, (M, N, K, act, out, epilogue) in ways(ep, "linear").items():
        try:
            case(ep, M, N, K, act, epilogue, epilogue, out, epilogue, seed=M + K)
            if epilogue and act == "none":
                case(ep, M, N, K, "silu", True, False, out, False, seed=M)
        except AssertionError as e:
            raise AssertionError(f"{way}: {M} x {N} x {K} {act} {out}") from e


def test_input_gradients(ep):
    for way, (M, N, K, _, _, _) in ways(ep, "grad_input").items():
        dz = torch.full((M, ep.linear_pitch(N)), float("nan"), dtype=bf, device="cuda")
        dz[:, :N] = rand(M, N)
        w = rand(N, K, seed=1)
        dx = torch.empty(M, K, dtype=bf, device="cuda")
        ep.ep_linear_grad_input(dz, w, dx)
        d = dz[:, :N].to(f64)
        try:
            close(dx, d @ w.to(f64), (N + 8) * U * (d.abs() @ w.to(f64).abs()))
        except AssertionError as e:
            raise AssertionError(f"{way}: {M} x {N} x {K}") from e


def test_weight_gradients(ep):
    for way, (M, N, K, _, out, epilogue) in ways(ep, "grad_weight").items():
        dz = torch.full((M, ep.linear_pitch(N)), float("nan"), dtype=bf, device="cuda")
        dz[:, :N] = rand(M, N)
        x = rand(M, K, seed=1)
        start = rand(N, K, seed=2, dtype=out)
        d_w = start.clone()
        ep.ep_linear_grad_weight(dz, x, d_w, accumulate=epilogue)
        d = dz[:, :N].to(f64)
        want = d.T @ x.to(f64) + (start.to(f64) if epilogue else 0)
        try:
            close(d_w, want, (M + 8) * U * (d.abs().T @ x.to(f64).abs()) + 2 * U * want.abs())
        except AssertionError as e:
            raise AssertionError(f"{way}: {M} x {N} x {K} {out}") from e
