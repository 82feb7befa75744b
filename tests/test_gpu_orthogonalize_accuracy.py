"""How near the orthogonalised updates come to the fp64 iteration, for gradients
of full and of low rank, on limits that are a small part of the answer.

A value y rounded to bf16 is off by at most 2^-8 of it, so all of them by at most 2^-8
of their norm, and by 2^-8 / sqrt(6) = 1.6e-3 of it where roundings spread evenly over
a binade. On top come the fp16 values between the products. An error of the
polynomial P in X' = d X + P X keeps X's null spaces: of five steps, each with
roundings of A and P that are at most 2^-11, typically 2^-11 / sqrt(6), of products two
to three times X', it leaves 3 sqrt(10) 2^-11 / sqrt(6) = 1.9e-3 if none decays. An
error of X that lies in both null spaces grows by a factor a a step, which 22 bits of
X leave room for: a^5 2^-23 is 6e-5. Together 2.5e-3. LIMIT, bf16's half step, is 1.6
times that, a sixth of what fp16 values alone make of rank 64 (0.024) and 1/38 of what
they make of rank 1 (0.15)."""
import pytest
import torch

import routing_util as U

pytestmark = pytest.mark.gpu

LIMIT = 2.0 ** -8


@pytest.fixture(scope="module")
def B():
    from round_dropless_expert_amd import binding
    binding.load()
    binding.check_runtime()
    return binding


def gen(seed):
    return torch.Generator().manual_seed(seed)


def exact(g, coefficients, scale=1.0):
    """The iteration in fp64 on the host."""
    x = g.double()
    tall = x.shape[0] > x.shape[1]
    x = x.t() if tall else x
    x = x / (torch.linalg.matrix_norm(x) + 1e-20)
    for a, b, c in coefficients:
        p = x @ x.t()
        x = a * x + (b * p + c * (p @ p)) @ x
    return scale * (x.t() if tall else x)


def error(B, g, coefficients=None, **kw):
    """Errors of the matrices g [E, N, K], as parts of the answers' norms."""
    E, N, K = g.shape
    ws = torch.full((B.orthogonalize_workspace_size(E, N, K),), 255, dtype=torch.uint8,
                    device="cuda")
    y = torch.empty(E, N, K, dtype=torch.bfloat16, device="cuda")
    steps = kw.get("steps", 5)
    B.moe_orthogonalize(g.cuda(), y, ws, coefficients=coefficients, **kw)
    y = y.double().cpu()
    out = []
    for e in range(E):
        want = exact(g[e], coefficients or [U.USUAL] * steps, kw.get("scale", 1.0))
        out.append(float(torch.linalg.matrix_norm(y[e] - want) / torch.linalg.matrix_norm(want)))
    return out


def low_rank(shape, rank, seed):
    E, N, K = shape
    r = gen(seed)
    return torch.randn(E, N, rank, generator=r) @ torch.randn(E, rank, K, generator=r)


# a workgroup a matrix at every number of row blocks, both tiles, both orientations
SIZES = [(2, 20, 31), (2, 64, 64), (2, 201, 77), (2, 90, 720), (2, 128, 256), (2, 256, 128),
         (2, 150, 300), (2, 190, 192), (2, 31, 1000), (2, 1000, 60), (2, 515, 390), (2, 260, 512),
         (40, 512, 520), (2, 1024, 1536)]


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N,K", [(64, 64), (201, 77), (256, 128), (300, 260)])
def test_types(B, dt, N, K):
    g = torch.cat([low_rank((2, N, K), 2, N), torch.randn(2, N, K, generator=gen(K))]).to(dt)
    assert max(error(B, g)) <= LIMIT


@pytest.mark.parametrize("E,N,K", SIZES)
def test_full_rank(B, E, N, K):
    e = error(B, torch.randn(E, N, K, generator=gen(N + K)) * 1e-2)
    assert max(e) <= LIMIT, e


@pytest.mark.parametrize("rank", [1, 3, 8, 64])
@pytest.mark.parametrize("E,N,K", SIZES)
def test_low_rank(B, E, N, K, rank):
    """The gradient of an expert that got `rank` tokens."""
    e = error(B, low_rank((min(E, 3), N, K), min(rank, N, K), N + rank) * 1e-3)
    assert max(e) <= LIMIT, e


@pytest.mark.parametrize("N,K", [(96, 160), (160, 96), (256, 256), (300, 260), (1024, 512)])
def test_strong_directions(B, N, K):
    """A few singular values far above the others, and rows that are few."""
    r = gen(5)
    g = torch.randn(3, N, K, generator=r) * 0.05
    g[0] += torch.randn(N, 1, generator=r) @ torch.randn(1, K, generator=r)
    g[1] += 100 * torch.randn(N, 2, generator=r) @ torch.randn(2, K, generator=r)
    g[2] = 0
    g[2, :3] = torch.randn(3, 1, generator=r) @ torch.randn(1, K, generator=r)
    e = error(B, g)
    assert max(e) <= LIMIT, e


@pytest.mark.parametrize("N,K", [(64, 64), (300, 200), (512, 512)])
def test_more_steps(B, N, K):
    """Eight steps multiply an error in both null spaces by a^8 = 2e4: X's 2^-23 / sqrt(6)
    by 1e-3, a quarter of the limit."""
    e = error(B, low_rank((2, N, K), 4, 8), steps=8)
    assert max(e) <= LIMIT, e


@pytest.mark.parametrize("N,K", [(64, 96), (300, 200)])
def test_one_step_and_other_coefficients(B, N, K):
    g = torch.cat([low_rank((1, N, K), 2, 9), torch.randn(1, N, K, generator=gen(10))])
    for steps in (1, 2, 3):
        assert max(error(B, g, steps=steps)) <= LIMIT
    own = [(3.0, -3.2, 1.2), (2.5, -2.0, 0.5), (1.875, -1.25, 0.375)]
    assert max(error(B, g, own, steps=3, scale=-0.2)) <= LIMIT
    assert max(error(B, g, [(1.5, -0.5, 0.0)] * 12, steps=12)) <= LIMIT


# the longest sides that fit in LDS (half of it, all of it) by blocks of 32 rows, and
# one more column, which does not
@pytest.mark.parametrize("m,n", [(32, 960), (30, 2496), (32, 2497), (64, 416), (61, 1184), (64, 1185),
                                 (96, 224), (90, 736), (96, 737), (128, 480), (120, 481),
                                 (160, 320), (155, 321), (192, 192), (192, 193)])
def test_longest_in_lds(B, m, n):
    g = torch.cat([torch.randn(2, m, n, generator=gen(m)), low_rank((2, m, n), 2, n)])
    wide = error(B, g)
    tall = error(B, g.transpose(1, 2).contiguous())
    assert max(wide + tall) <= LIMIT, (wide, tall)


@pytest.mark.parametrize("N,K", [(77, 201), (260, 512)])
def test_graph_and_repeats(B, N, K):
    """Captured and replayed with other gradients between eager updates, on one
    workspace: the bits of the eager call each time."""
    g = low_rank((3, N, K), 2, 11).cuda()
    ws = torch.empty(B.orthogonalize_workspace_size(3, N, K), dtype=torch.uint8, device="cuda")
    y, z = (torch.empty(3, N, K, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    B.moe_orthogonalize(g, y, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.moe_orthogonalize(g, y, ws)
    for seed in range(4):
        g.copy_(low_rank((3, N, K), 1 + seed, 20 + seed))
        B.moe_orthogonalize(g, z, ws)
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, z) and bool(torch.isfinite(y).all())


def test_past_4_gib(B):
    """Matrices whose X^T and its rest lie past 4 GiB of the workspace."""
    E, N, K = 520, 2048, 2048
    g = torch.zeros(E, N, K, dtype=torch.bfloat16, device="cuda")
    few = torch.cat([low_rank((1, N, K), 2, 1), torch.randn(1, N, K, generator=gen(2))])
    for e in (0, 1):
        g[e] = g[E - 2 + e] = few[e].cuda()
    y = torch.full((E, N, K), 3.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((B.orthogonalize_workspace_size(E, N, K),), 255, dtype=torch.uint8,
                    device="cuda")
    B.moe_orthogonalize(g, y, ws)
    assert torch.equal(y[0], y[E - 2]) and torch.equal(y[1], y[E - 1])
    assert (y[2:E - 2] == 0).all()
    want = exact(g[0].float().cpu(), [U.USUAL] * 5)
    assert torch.linalg.matrix_norm(y[0].double().cpu() - want) <= LIMIT * torch.linalg.matrix_norm(want)
