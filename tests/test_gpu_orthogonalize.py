"""Orthogonalised updates on the GPU against the fp64 iteration."""
import pytest
import torch

import routing_util as U
from ragged_util import DT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from round_dropless_expert_amd import binding
    binding.load()
    binding.check_runtime()
    return binding


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def update(B, g, **kw):
    E, N, K = (1, *g.shape) if g.dim() == 2 else g.shape
    ws = torch.full((B.orthogonalize_workspace_size(E, N, K),), 255, dtype=torch.uint8,
                    device="cuda")  # every value of it a NaN
    buf = torch.full((g.numel() + 8,), 77.0, dtype=torch.bfloat16, device="cuda")
    y = buf[: g.numel()].view(g.shape)
    B.moe_orthogonalize(g, y, ws, **kw)
    assert (buf[g.numel():] == 77.0).all()
    return y


def check(y, g, coefficients, scale=1.0):
    for e in range(g.shape[0]):
        ref, bound = U.orthogonalize(g[e].double().cpu(), coefficients, scale)
        err = float(torch.linalg.matrix_norm(y[e].double().cpu() - ref))
        norm = float(torch.linalg.matrix_norm(ref))
        assert err <= bound, f"matrix {e}: {err:.4g} of {norm:.4g}, bound {bound:.4g}"


SIZES = [(1, 1, 1), (2, 1, 40), (3, 40, 1), (2, 7, 5), (3, 64, 64), (3, 201, 77), (2, 77, 201),
         (2, 128, 256), (1, 130, 129), (4, 256, 512), (2, 512, 256), (1, 300, 1000), (1, 515, 390)]


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("E,N,K", SIZES)
def test_update(B, dt, E, N, K):
    g = (torch.randn(E, N, K, generator=gen(N + K), device="cuda") * 1e-2).to(DT[dt])
    check(update(B, g), g, [U.USUAL] * 5)


@pytest.mark.parametrize("N,K", [(96, 160), (160, 96), (256, 256), (300, 260)])
def test_spectra(B, N, K):
    """A few strong directions; a matrix of low rank; rows and columns of zeros;
    gradients of any size."""
    r = gen(5)
    g = torch.randn(6, N, K, generator=r, device="cuda") * 0.05
    g[0] += torch.randn(N, 1, generator=r, device="cuda") * torch.randn(1, K, generator=r,
                                                                      device="cuda")
    g[1] = torch.randn(N, 3, generator=r, device="cuda") @ torch.randn(3, K, generator=r,
                                                                     device="cuda")
    g[2, N // 3:] = 0
    g[3, :, K // 3:] = 0
    g[4] *= 1e30
    g[5] *= 1e-14
    check(update(B, g), g, [U.USUAL] * 5)


def test_steps_and_coefficients(B):
    g = torch.randn(2, 100, 140, generator=gen(6), device="cuda")
    for steps in (1, 2, 7):
        check(update(B, g, steps=steps), g, [U.USUAL] * steps)
    own = [(3.0, -3.2, 1.2), (2.5, -2.0, 0.5), (1.875, -1.25, 0.375)]
    check(update(B, g, steps=3, coefficients=own, scale=-0.2), g, own, -0.2)
    # the odd cubic iteration converges to the orthogonal factor
    y = update(B, g, steps=20, coefficients=[(1.5, -0.5, 0.0)] * 20)
    q = y.double() @ y.double().transpose(1, 2)
    eye = torch.eye(100, dtype=torch.float64, device="cuda")
    # each element of y is within bf16's half step and fp16's of the factor's
    assert float(torch.linalg.matrix_norm(q - eye, 2).max()) <= 2 * 100 ** 0.5 * (2.0 ** -8 + 2.0 ** -10)


# a matrix a workgroup, and tiles of both kinds
@pytest.mark.parametrize("N,K", [(70, 50), (50, 70), (261, 300), (300, 261), (1300, 1400)])
def test_zeros_and_non_numbers(B, N, K):
    g = torch.randn(5, N, K, generator=gen(7), device="cuda")
    good = update(B, g)
    g2 = g.clone()
    g2[0] = 0
    g2[2, 3, 4] = float("inf")
    g2[4, N - 1, K - 1] = float("nan")
    y = update(B, g2)
    assert (y[0] == 0).all()
    assert torch.isnan(y[2]).all() and torch.isnan(y[4]).all()
    assert torch.equal(y[1], good[1]) and torch.equal(y[3], good[3])


def test_one_matrix_and_unaligned_output(B):
    g = torch.randn(64, 96, generator=gen(8), device="cuda")
    y = update(B, g)
    assert torch.equal(y, update(B, g.unsqueeze(0))[0])
    buf = torch.zeros(64 * 96 + 1, dtype=torch.bfloat16, device="cuda")
    z = buf[1:].view(64, 96)
    ws = torch.empty(B.orthogonalize_workspace_size(1, 64, 96), dtype=torch.uint8, device="cuda")
    B.moe_orthogonalize(g, z, ws)
    assert torch.equal(z, y)


@pytest.mark.parametrize("E,N,K", [(2, 1024, 1536), (40, 512, 520)])
def test_large_tiles(B, E, N, K):
    """Sizes that take the 256 x 256 tiles; checked against fp64 on the GPU by the
    singular values' own polynomial."""
    g = torch.randn(E, N, K, generator=gen(9), device="cuda")
    y = update(B, g)
    for e in (0, E - 1):
        check(y[e:e + 1], g[e:e + 1], [U.USUAL] * 5)


@pytest.mark.parametrize("N,K", [(16384, 200), (30, 16384), (64, 1100), (1100, 64), (193, 193)])
def test_long_sides(B, N, K):
    g = torch.randn(1, N, K, generator=gen(10), device="cuda") * 1e-3
    check(update(B, g), g, [U.USUAL] * 5)


def test_updates_repeat(B):
    """The same bits again, with other matrices around them."""
    for N, K in ((100, 120), (260, 400), (1024, 512)):
        g = torch.randn(6, N, K, generator=gen(11), device="cuda")
        y = update(B, g)
        assert torch.equal(y, update(B, g))
        assert torch.equal(y[2:3], update(B, g[2:3].contiguous()))


@pytest.mark.parametrize("E,N,K", [
    (3, 16, 16), (2, 40, 100), (2, 100, 40), (3, 77, 201), (3, 201, 77), (2, 192, 190),
    (1, 193, 60), (2, 257, 300), (2, 300, 257), (1, 129, 1000), (1, 1000, 130), (3, 640, 520),
    (2, 1024, 1536), (2, 1536, 1024), (2, 1411, 1297), (2, 2048, 2048)])
def test_whole_numbers(B, E, N, K):
    """Every value exact, so every element of y is known: 4^p elements of +-1 and
    zeros have the norm 2^p, A and A A are whole numbers over powers of two, and
    with coefficients that are powers of two Q = (8 I + 2 n1 + n2) / 256 and X' need
    at most 11 and 24 bits. A first step with Q = I passes X on."""
    m = min(N, K)
    p = 1
    while 4 ** (p + 1) <= min(16 * m, N * K // 2):
        p += 1
    g = torch.zeros(E, N * K)
    r = torch.Generator().manual_seed(N + K)
    for e in range(E):
        at = torch.randperm(N * K, generator=r)[: 4 ** p]
        g[e, at] = torch.randint(0, 2, (4 ** p,), generator=r).float() * 2 - 1
    g = g.view(E, N, K)
    x = (g if N <= K else g.transpose(1, 2)).double()
    n1 = x @ x.transpose(1, 2)
    q = 8 * torch.eye(m, dtype=torch.float64) + 2 * n1 + n1 @ n1
    assert q.abs().max() < 2048 and n1.abs().max() < 2048
    y = q @ x  # 256 2^p times the result
    assert y.abs().max() < 2 ** 24
    want = (y if N <= K else y.transpose(1, 2)).float().bfloat16()
    c = [(8 / 256, 2 * 4.0 ** p / 256, 16.0 ** p / 256)]
    for dt in (torch.float32, torch.bfloat16):
        for steps in ([(1.0, 0.0, 0.0)] + c, c):
            got = update(B, g.to(dt).cuda(), steps=len(steps), coefficients=steps,
                         scale=256.0 * 2 ** p)
            assert torch.equal(got.cpu(), want), (dt, len(steps))
