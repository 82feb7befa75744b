"""Routing and sort where the sizes or values are extreme, compared with what is known
exactly."""
import numpy as np
import pytest
import torch

import routing_util as U

pytestmark = pytest.mark.gpu

MOST = torch.finfo(torch.float32).max


@pytest.fixture(scope="module")
def B():
    from round_dropless_expert_amd import binding
    binding.load()
    binding.check_runtime()
    return binding


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


@pytest.mark.parametrize("mode", ["even", "skewed", "one", "padded"])
@pytest.mark.parametrize("n,E", [(1048576, 256), (1048577, 256), (1048577, 1024), (2000003, 256),
                                 (2000003, 1024), (5000011, 40)])
def test_sort_long_runs(B, n, E, mode):
    """More than 2^20 assignments: a wavefront's run is longer than what it keeps, so it
    reads the rest twice."""
    idx = torch.randint(0, E, (n,), generator=gen(n + E), device="cuda", dtype=torch.int32)
    if mode == "skewed":
        idx = torch.where(torch.rand(n, generator=gen(1), device="cuda") < 0.6, idx % 3, idx)
    if mode == "one":
        idx[:] = E - 1
    if mode == "padded":
        m = torch.rand(n, generator=gen(3), device="cuda")
        idx[m < 0.2] = -1
        idx[m > 0.9] = E
        idx[m > 0.95] = 2 ** 31 - 1
        idx[-70000:] = -1
    perm, pos = (torch.full((n + 1,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    off = torch.full((E + 2,), -9, dtype=torch.int32, device="cuda")
    ws = torch.full((B.sort_workspace_size(n, E),), 255, dtype=torch.uint8, device="cuda")
    B.moe_sort(idx, E, perm, pos, off, ws)
    want = U.sort(idx.cpu().numpy(), E)
    for got, ref, name in zip((perm[:n], pos[:n], off[: E + 1]), want, ("perm", "pos", "offsets")):
        assert np.array_equal(got.cpu().numpy(), ref), name
    assert perm[n] == -9 and pos[n] == -9 and off[E + 1] == -9


def test_gradient_past_4_gib(B):
    """Each row against its closed form: with sigmoids s of the chosen two, weights w =
    s / sum s and dweight g, dl_j = w_j (1 - s_j) (g_j - sum w g), zeros elsewhere. Some
    ten fp32 roundings of values up to 1 and of g up to 2: 20 2^-24."""
    T, E = 4_300_000, 256  # 4.4 GB of fp32
    logits = torch.zeros(T, E, device="cuda")
    logits[-1, 200], logits[-1, 7], logits[-2, 3] = 3.0, 2.0, 1.0
    idx = torch.tensor([0, 1], dtype=torch.int32, device="cuda").repeat(T, 1)
    idx[-1] = torch.tensor([200, 7], dtype=torch.int32)
    idx[-2] = torch.tensor([3, 0], dtype=torch.int32)
    dweight = torch.tensor([1.0, -2.0], device="cuda").repeat(T, 1)
    dweight[-1, 0] = 0.5
    dl = torch.full((T + 1, E), 7.0, device="cuda")
    B.moe_route_backward(B.router(T, E, 2, "f32", "sigmoid"), logits, idx, dweight, dl[:T])

    def want(l, g):
        s = torch.sigmoid(torch.tensor(l, dtype=torch.float64))
        g = torch.tensor(g, dtype=torch.float64)
        w = s / s.sum()
        return (w * (1 - s) * (g - (w * g).sum())).tolist()

    near = lambda got, ref: abs(float(got) - ref) <= 20 * 2.0 ** -24
    for row, experts, l, g in ((-1, (200, 7), (3.0, 2.0), (0.5, -2.0)),
                               (-2, (3, 0), (1.0, 0.0), (1.0, -2.0))):
        got = dl[:T][row]
        for e, v in zip(experts, want(l, g)):
            assert abs(v) > 0.01 and near(got[e], v), (row, e, float(got[e]), v)
        assert int((got != 0).sum()) == 2
    first, second = want((0.0, 0.0), (1.0, -2.0))
    for part in dl[: T - 2].split(500_000):
        assert near(part[:, 0].min(), first) and near(part[:, 0].max(), first)
        assert near(part[:, 1].min(), second) and near(part[:, 1].max(), second)
        assert int((part[:, 2:] != 0).sum()) == 0
    assert (dl[T] == 7.0).all()


# kernels of 8 and 16 lanes a token, of few and many choices, and the exact one
@pytest.mark.parametrize("E,k", [(8, 4), (64, 6), (128, 8), (256, 8), (256, 12), (512, 16), (40, 20),
                                 (1024, 8), (1024, 33)])
@pytest.mark.parametrize("biased", [False, True])
def test_weights_of_extreme_logits(B, E, k, biased):
    """Rows whose weights are known: equal shares, all of it, or nothing. A share is a
    sum of ones (exact), a division and a product with the scale: 2^-22 of it covers
    their three roundings."""
    inf, nan, scale = float("inf"), float("nan"), 2.5
    rows = []  # logits, and sigmoids of the chosen ones in the order of the choice

    def row(base, s, *changes):
        l = torch.full((E,), base)
        for at, v in changes:
            l[at] = v
        rows.append((l, s))

    row(MOST, [1.0] * k)
    row(-MOST, [0.0] * k)
    row(inf, [1.0] * k)
    row(0.0, [0.5] * k)
    row(-MOST, [1.0] + [0.0] * (k - 1), (E - 1, MOST))
    row(-inf, [1.0] + [0.0] * (k - 1), (E // 2, MOST))
    row(nan, [0.0] * k)
    row(-inf, [1.0, 1.0] + [0.0] * (k - 2), (1, inf), (E - 2, inf))
    logits = torch.stack([l for l, _ in rows])
    if biased:  # it is added to scores, and the same for all: no choice changes
        bias = torch.full((E,), 0.25, device="cuda")
    T = len(rows)
    for score in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            r = B.router(T, E, k, "f32", score, renormalize=renormalize, scale=scale)
            idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
            w = torch.full((T, k), nan, device="cuda")
            B.moe_route(r, logits.cuda(), idx, w, bias=bias if biased else None)
            for t, (l, s) in enumerate(rows):
                what = (score, renormalize, t)
                chosen = l[idx[t].cpu().long()]
                live = chosen > -inf
                top = (chosen == chosen[live].max()) if live.any() else torch.zeros(k).bool()
                if score == "sigmoid" and not renormalize:
                    want = torch.tensor(s, dtype=torch.float64)
                elif renormalize:
                    want = top.double() / max(int(top.sum()), 1)
                else:  # the softmax's share of every expert with the largest logit
                    want = top.double() / max(int((l == chosen[0]).sum()), 1)
                want = scale * want
                err = (w[t].double().cpu() - want).abs()
                assert (err <= 2.0 ** -22 * want).all(), (what, w[t].tolist(), want.tolist())


@pytest.mark.parametrize("dt", [torch.float32])
@pytest.mark.parametrize("E,k", [(64, 6), (256, 8), (700, 17)])
def test_softmax_of_shifted_logits(B, E, k, dt):
    """A large number added to all of a token's logits (exactly: all are multiples of
    1/4 below 2^22) changes no weight by more than the rounding of differences of at most
    20: an exponent is off by 20 2^-24, a sum of E terms by E 2^-24, and a few steps."""
    T = 50
    l = torch.randint(-40, 41, (T, E), generator=gen(E), device="cuda").to(dt) / 4
    ref = torch.softmax(l.double(), dim=1)
    for shift in (-3e6, 3e6):
        for renormalize in (True, False):
            r = B.router(T, E, k, dt, renormalize=renormalize)
            idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
            w = torch.empty(T, k, device="cuda")
            B.moe_route(r, l + shift, idx, w)
            want = ref.gather(1, idx.long())
            if renormalize:
                want = want / want.sum(dim=1, keepdim=True)
            assert ((w.double() - want).abs() <= (20 + E + 8) * 2.0 ** -24 * want).all()
