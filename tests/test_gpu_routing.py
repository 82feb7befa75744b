"""Routing, its gradient, the sort and the collection on the GPU against plain
fp64 forms (routing_util)."""
import numpy as np
import pytest
import torch

import ragged_util as R
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


def randn(shape, dtype, seed, pad=0, scale=1.0):
    t = torch.randn(*shape[:-1], shape[-1] + pad, generator=gen(seed), device="cuda") * scale
    return t.to(dtype)[..., : shape[-1]]


def check(got, ref, bound, what):
    err = np.abs(np.asarray(got, dtype=np.float64) - ref)
    bad = ~(err <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} past the bound, first at "
                           f"{tuple(np.argwhere(bad)[0])}, worst {np.nanmax(err / bound):.3f}")


def route(B, logits, k, score, bias=None, groups=1, top_groups=1, group_top=2, renormalize=True,
          scale=1.0):
    T, E = logits.shape
    r = B.router(T, E, k, logits.dtype, score, groups, top_groups, group_top, renormalize, scale,
                 ld=logits.stride(0) if T > 1 else 0)
    idx = torch.full((T + 1, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T + 1, k), 77.0, device="cuda")
    B.moe_route(r, logits, idx[:T], w[:T], bias=bias)
    assert (idx[T:] == -7).all() and (w[T:] == 77.0).all()
    return r, idx[:T], w[:T]


def check_route(B, logits, k, score, bias=None, groups=1, top_groups=1, group_top=2,
                renormalize=True, scale=1.0):
    _, idx, w = route(B, logits, k, score, bias, groups, top_groups, group_top, renormalize, scale)
    l = logits.double().cpu().numpy()
    b = None if bias is None else bias.double().cpu().numpy()
    want = U.choose(l, b, k, score, groups, top_groups, group_top)
    got = idx.cpu().numpy()
    assert np.array_equal(got, want), (
        f"{(got != want).any(axis=1).sum()} of {len(got)} tokens, first "
        f"{np.argwhere((got != want).any(axis=1))[0]}")
    ref, bound = U.weights(l, got, score, renormalize, scale)
    check(w.cpu().numpy(), ref, bound, "weight")


# E, k, groups, top_groups
SHAPES = [(1, 1, 1, 1), (4, 2, 1, 1), (8, 3, 4, 2), (16, 8, 2, 1), (17, 5, 1, 1), (64, 6, 1, 1),
          (64, 8, 8, 4), (60, 4, 5, 3), (96, 6, 12, 5), (100, 8, 1, 1), (128, 4, 16, 3),
          (160, 6, 8, 3), (192, 8, 6, 2), (256, 8, 8, 4), (256, 1, 1, 1), (256, 8, 256 // 4, 9),
          (384, 8, 1, 1), (512, 8, 16, 4), (513, 10, 27, 20), (1024, 64, 32, 8), (1024, 7, 1, 1),
          (40, 40, 1, 1), (64, 64, 1, 1), (48, 16, 48, 30), (12, 4, 12, 5), (16, 2, 16, 2),
          (96, 8, 3, 1), (512, 8, 2, 1), (192, 1, 12, 1)]


@pytest.mark.parametrize("E,k,groups,top", SHAPES)
def test_route(B, E, k, groups, top):
    for i, (score, dt, biased) in enumerate([("sigmoid", "f32", True), ("softmax", "f32", False),
                                             ("sigmoid", "bf16", False), ("softmax", "f16", True),
                                             ("softmax", "bf16", True)]):
        T, pad = [1, 67, 130, 33, 5][i], [0, 0, 3, 8, 16][i]
        logits = randn((T, E), DT[dt], 10 * i + E, pad, 1.5)
        bias = randn((E,), torch.float32, 3, scale=0.05) if biased else None
        check_route(B, logits, k, score, bias, groups, top, 1 + i % 2, i % 3 != 1, 2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top", [(256, 8, 4), (256, 1, 1), (160, 8, 3)])
def test_route_many_tokens(B, score, E, groups, top):
    """Near ties among many tokens: the choice is that of fp64."""
    logits = randn((20011, E), torch.float32, 5, scale=1.5)
    check_route(B, logits, 8, score, randn((E,), torch.float32, 6, scale=0.05), groups, top)
    check_route(B, logits, 8, score, None, groups, top, renormalize=False)


@pytest.mark.parametrize("groups,top", [(1, 1), (4, 2)])
def test_route_close_values(B, groups, top):
    """Choices that fp32 cannot tell apart, and true ties."""
    T, E, k = 512, 64, 6
    l = randn((T, E), torch.float32, 8)
    l = l[:, :1] + 1e-7 * torch.randint(0, 6, (T, E), generator=gen(9), device="cuda").float()
    bias = 1e-7 * torch.randint(0, 3, (E,), generator=gen(10), device="cuda").float()
    for score in ("softmax", "sigmoid"):
        check_route(B, l, k, score, bias, groups, top)
        check_route(B, l, k, score, None, groups, top)
    # ties: one of few values, and a bias that evens out two experts' scores
    l = torch.randint(0, 3, (T, E), generator=gen(11), device="cuda").float()
    for score in ("softmax", "sigmoid"):
        check_route(B, l, k, score, torch.zeros(E, device="cuda"), groups, top)
        check_route(B, l, k, score, None, groups, top)
        check_route(B, torch.zeros_like(l), k, score, None, groups, top)
        check_route(B, l.bfloat16(), k, score, torch.zeros(E, device="cuda"), groups, top)


@pytest.mark.parametrize("E,k,groups,top", [(32, 4, 1, 1), (64, 6, 8, 2), (300, 8, 1, 1),
                                            (64, 20, 1, 1)])
def test_route_masked(B, E, k, groups, top):
    """Experts and rows that a mask leaves nothing of; large and infinite logits."""
    T = 96
    l = randn((T, E), torch.float32, 12, scale=2.0)
    m = torch.rand(T, E, generator=gen(13), device="cuda")
    l[m < 0.3] = U.NINF
    l[m > 0.95] = float("nan")
    l[0] = U.NINF
    l[1] = float("nan")
    l[2] = U.NINF
    l[2, E // 2] = 3.0            # one is left
    l[3] = torch.finfo(torch.float32).min
    l[4] = -200.0 - torch.arange(E, device="cuda")   # every sigmoid vanishes in fp32
    l[5] = 200.0 + torch.arange(E, device="cuda")
    l[6, 0] = float("inf")
    l[7, :2] = float("inf")
    l[8] = torch.finfo(torch.float32).max
    for score in ("softmax", "sigmoid"):
        for ren in (True, False):
            check_route(B, l, k, score, None, groups, top, renormalize=ren)
    bias = randn((E,), torch.float32, 14, scale=0.1)
    bias[1] = U.NINF
    bias[2] = float("nan")
    live = torch.ones(T, dtype=torch.bool)
    live[5] = False  # sigmoids of 1 that fp64 cannot tell apart
    for score in ("softmax", "sigmoid"):
        check_route(B, l[live], k, score, bias, groups, top)


# E, k, groups, top_groups: both numbers of lanes a token, up to 16 choices, the
# widest rows without a bias
WIDE = [(33, 8, 1, 1), (50, 7, 1, 1), (65, 8, 1, 1), (127, 3, 1, 1), (128, 8, 1, 1),
        (16, 16, 1, 1), (33, 9, 1, 1), (64, 16, 8, 3), (100, 12, 1, 1), (128, 16, 4, 1),
        (256, 9, 8, 4), (255, 16, 5, 3), (300, 11, 1, 1), (512, 16, 16, 5), (600, 3, 1, 1),
        (1000, 16, 1, 1), (1023, 8, 1, 1)]


@pytest.mark.parametrize("E,k,groups,top", WIDE)
def test_route_wide(B, E, k, groups, top):
    T = 333
    l = randn((T, E), torch.float32, E, 3, 1.5)
    l[5] = U.NINF
    l[6, : E - k // 2] = U.NINF
    l[7] = float("nan")
    bias = randn((E,), torch.float32, 17, scale=0.05)
    for i, score in enumerate(("softmax", "sigmoid")):
        check_route(B, l, k, score, None, groups, top, 1 + i, renormalize=i == 0)
        check_route(B, l, k, score, bias, groups, top, 2 - i)
        check_route(B, l.bfloat16(), k, score, None, groups, top, renormalize=i == 1)


@pytest.mark.parametrize("E,k,groups,top", [(64, 8, 1, 1), (128, 8, 1, 1), (128, 16, 1, 1),
                                            (256, 16, 8, 4), (256, 8, 8, 4)])
def test_route_close_values_wide(B, E, k, groups, top):
    """Near and true ties where each token is chosen again, alone or with three more
    of its wavefront."""
    T = 400
    l = randn((T, E), torch.float32, 18)
    l[::3] = l[::3, :1] + 1e-7 * torch.randint(0, 6, (134, E), generator=gen(19),
                                               device="cuda").float()
    bias = 1e-7 * torch.randint(0, 3, (E,), generator=gen(20), device="cuda").float()
    for score in ("softmax", "sigmoid"):
        check_route(B, l, k, score, bias, groups, top)
        check_route(B, l, k, score, None, groups, top)
    l = torch.randint(0, 4, (T, E), generator=gen(21), device="cuda").float()
    for score in ("softmax", "sigmoid"):
        check_route(B, l, k, score, torch.zeros(E, device="cuda"), groups, top)


def test_route_more_tokens_than_a_grid(B):
    """Past 2^32 threads: two launches."""
    T = (32 << 23) + 1001
    l = torch.empty(T, 2, dtype=torch.bfloat16, device="cuda")
    l.normal_(generator=gen(22))
    r = B.router(T, 2, 1, l.dtype, "softmax")
    idx = torch.full((T, 1), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, 1), 77.0, device="cuda")
    B.moe_route(r, l, idx, w)
    assert torch.equal(idx[:, 0], (l[:, 1] > l[:, 0]).int())
    assert (w == 1.0).all()


def test_route_infinite_bias(B):
    """An expert that every token takes, one that none does."""
    l = randn((70, 64), torch.float32, 15)
    bias = randn((64,), torch.float32, 16, scale=0.05)
    bias[9] = float("inf")
    bias[11] = U.NINF
    for groups, top in ((1, 1), (8, 2)):
        for score in ("softmax", "sigmoid"):
            check_route(B, l, 4, score, bias, groups, top)


def backward(B, r, logits, idx, dw):
    T, E = logits.shape
    ld = r.ld or E
    out = torch.full((T + 1, ld), 77.0, dtype=logits.dtype, device="cuda")
    B.moe_route_backward(r, logits, idx, dw, out[:T, :E])
    assert (out[T] == 77.0).all() and (out[:T, E:] == 77.0).all()
    return out[:T, :E]


def grad_bound(l, idx, dw, score, renormalize, scale, dtype):
    """Formula's gradient and bound: the sums over the chosen (or all) experts and
    the exponents cost the weights' steps; both terms of g - dot count in full."""
    l = l.double().cpu().requires_grad_()
    dw = dw.double().cpu()
    w = U.weights_of(l, idx.cpu(), score, renormalize, scale)
    g, = torch.autograd.grad((w * dw).sum(), l)
    with torch.no_grad():
        s = torch.from_numpy(U.scores(l.detach().numpy(), score))
        sj = s.gather(1, idx.cpu().long())
        share = w / scale
        full = score == "softmax" and not renormalize
        mag = torch.zeros_like(l)
        dot = (share * dw.abs()).sum(dim=1, keepdim=True)
        if full:
            mag += s * dot
            mag.scatter_add_(1, idx.cpu().long(), sj * dw.abs())
        elif renormalize:
            f = 1.0 if score == "softmax" else 1 - sj
            mag.scatter_add_(1, idx.cpu().long(), share * (dw.abs() + dot) * f)
        else:
            mag.scatter_add_(1, idx.cpu().long(), sj * (1 - sj) * dw.abs())
        steps = 2 * l.abs().max() + (l.shape[1] if full else 0) + 2 * idx.shape[1] + 20
        b = abs(scale) * mag * steps * 2.0 ** -23
        # the fp64 reference's own steps: what cancels there (an expert that was not
        # chosen) leaves up to as many times 2^-52 of the whole
        b = b + abs(scale) * dw.abs().sum(dim=1, keepdim=True) * (steps + l.shape[1]) * 2.0 ** -52
        return g, b * (1 + torch.finfo(dtype).eps) + R.rounding(g, dtype)


@pytest.mark.parametrize("E,k", [(1, 1), (4, 2), (8, 8), (17, 5), (64, 6), (100, 8), (160, 6),
                                 (256, 8), (384, 3), (1024, 64), (40, 40)])
@pytest.mark.parametrize("score,renormalize", [("softmax", True), ("softmax", False),
                                               ("sigmoid", True), ("sigmoid", False)])
def test_route_backward(B, E, k, score, renormalize):
    for i, (T, dt, pad) in enumerate([(1, "f32", 0), (129, "f32", 5), (70, "bf16", 8),
                                      (33, "f16", 1)]):
        logits = randn((T, E), DT[dt], i + E, pad, 1.5)
        r, idx, _ = route(B, logits, k, score, renormalize=renormalize, scale=2.5)
        dw = randn((T, k), torch.float32, 50 + i)
        got = backward(B, r, logits, idx, dw)
        ref, bound = grad_bound(logits, idx, dw, score, renormalize, 2.5, DT[dt])
        check(got.double().cpu().numpy(), ref.numpy(), bound.numpy(), "dlogits")


@pytest.mark.parametrize("score,renormalize", [("softmax", True), ("softmax", False),
                                               ("sigmoid", True), ("sigmoid", False)])
def test_route_backward_is_the_forwards_difference(B, score, renormalize):
    T, E, k, h = 16, 12, 4, 1e-5
    logits = randn((T, E), torch.float32, 21)
    r, idx, _ = route(B, logits, k, score, renormalize=renormalize)
    dw = randn((T, k), torch.float32, 22)
    got = backward(B, r, logits, idx, dw).double().cpu()
    l, ic, d = logits.double().cpu(), idx.cpu(), dw.double().cpu()
    f = lambda x: (U.weights_of(x, ic, score, renormalize, 1.0) * d).sum(dim=1)
    for e in range(E):
        step = torch.zeros_like(l)
        step[:, e] = h
        diff = (f(l + step) - f(l - step)) / (2 * h)
        # central differences: h^2 / 6 times a third derivative (below 10 here),
        # 2^-52 / h of cancellation, and fp32's steps of the kernel
        tol = 10 * h * h + 2.0 ** -50 / h + 60 * 2.0 ** -23 * d.abs().sum(dim=1)
        assert ((got[:, e] - diff).abs() <= tol).all()


def test_route_backward_masked(B):
    """Nothing flows to masked experts or from padded choices; values far out."""
    T, E, k = 6, 16, 4
    for score in ("softmax", "sigmoid"):
        for ren in (True, False):
            l = randn((T, E), torch.float32, 23)
            l[:, 3] = U.NINF
            l[0] = U.NINF
            l[1] = -300.0 - torch.arange(E, device="cuda")
            l[2] = 300.0
            r, idx, w = route(B, l, k, score, renormalize=ren)
            idx[4, 2] = -1
            idx[5] = E + 5
            dw = randn((T, k), torch.float32, 24)
            got = backward(B, r, l, idx, dw)
            assert torch.isfinite(got).all()
            assert (got[torch.isneginf(l)] == 0).all()
            assert (got[0] == 0).all() and (got[5] == 0).all()
            if ren and score == "sigmoid":  # ratios of vanishing sigmoids still have a gradient
                lw = torch.softmax(l[1, idx[1].long()].double(), 0)
                g = dw[1].double()
                ref = lw * (g - (lw * g).sum())
                err = (got[1, idx[1].long()].double() - ref).abs()
                assert (err <= 2.0 ** -23 * 700 * g.abs().max()).all()


# E with 1 and 2 vectors a lane, rows that are read on past what a lane keeps, and
# rows of no whole vectors
@pytest.mark.parametrize("E,pad", [(64, 0), (128, 0), (256, 0), (512, 0), (1024, 0), (62, 5),
                                   (130, 1), (250, 3), (1000, 5), (1021, 0)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_route_backward_rows(B, E, pad, dt):
    T, k = 77, min(E, 20)
    logits = randn((T, E), DT[dt], E, pad, 1.5)
    for score in ("softmax", "sigmoid"):
        for ren in (False, True):
            r, idx, _ = route(B, logits, k, score, renormalize=ren)
            dw = randn((T, k), torch.float32, 25)
            g, bound = grad_bound(logits, idx, dw, score, ren, 1.0, DT[dt])
            check(backward(B, r, logits, idx, dw).double().cpu().numpy(), g.numpy(),
                  bound.numpy(), f"{score} {ren}")


@pytest.mark.parametrize("score,renormalize", [("softmax", True), ("softmax", False),
                                               ("sigmoid", True), ("sigmoid", False)])
def test_route_backward_subnormal(B, score, renormalize):
    """Gradients below fp32's normal numbers are kept: each product and sum of them
    (one for each choice and four of an expert's own) is off by 2^-150 at most, and
    what multiplies it afterwards is at most 1."""
    T, E, k = 9, 64, 6
    logits = randn((T, E), torch.float32, 26)
    r, idx, _ = route(B, logits, k, score, renormalize=renormalize)
    dw = 3e-39 * torch.arange(1, k + 1, device="cuda").float().expand(T, k).contiguous()
    g, bound = grad_bound(logits, idx, dw, score, renormalize, 1.0, torch.float32)
    check(backward(B, r, logits, idx, dw).double().cpu().numpy(), g.numpy(),
          bound.numpy() + (k + 4) * 2.0 ** -150, "dlogits")


@pytest.mark.parametrize("n,E", [(1, 1), (5, 8), (64, 64), (63, 1024), (1000, 7), (4096, 256),
                                 (4097, 256), (4096, 1024), (30000, 1024), (131072, 64),
                                 (600001, 300), (2100, 1023)])
def test_sort(B, n, E):
    for mode in ("even", "skewed", "one", "padded"):
        idx = torch.randint(0, E, (n,), generator=gen(n + E), device="cuda", dtype=torch.int32)
        if mode == "skewed":
            idx = idx * idx // max(E, 1) // 2
        if mode == "one":
            idx[:] = E - 1
        if mode == "padded":
            m = torch.rand(n, generator=gen(3), device="cuda")
            idx[m < 0.2] = -1
            idx[m > 0.9] = E
            idx[m > 0.95] = 2 ** 31 - 1
        perm, pos = (torch.full((n + 1,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
        off = torch.full((E + 2,), -9, dtype=torch.int32, device="cuda")
        size = B.sort_workspace_size(n, E)
        ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda") if size else None
        B.moe_sort(idx, E, perm, pos, off, ws)
        want = U.sort(idx.cpu().numpy(), E)
        assert np.array_equal(perm[:n].cpu().numpy(), want[0]), mode
        assert np.array_equal(pos[:n].cpu().numpy(), want[1]), mode
        assert np.array_equal(off[:E + 1].cpu().numpy(), want[2]), mode
        assert perm[n] == -9 and pos[n] == -9 and off[E + 1] == -9


def test_sort_nothing(B):
    off = torch.full((9,), -9, dtype=torch.int32, device="cuda")
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    assert B.load().moe_sort(0, 8, None, None, None, off.data_ptr(), None, 0,
                             torch.cuda.current_stream().cuda_stream) == B.MOE_OK
    assert (off == 0).all() and e.numel() == 0


@pytest.mark.parametrize("T,k,d,pad,dt,behind", [
    (1, 1, 1, 0, "f32", 0), (1, 8, 7168, 0, "bf16", 0), (5, 3, 1001, 3, "f16", 2),
    (33, 2, 64, 8, "bf16", 5), (17, 5, 519, 1, "f32", 0), (100, 6, 2048, 0, "bf16", 9),
    (64, 4, 1024, 16, "f16", 0), (9, 64, 40, 0, "f32", 1), (3, 2, 20000, 0, "bf16", 0),
    (130, 8, 7, 0, "bf16", 3)])
def test_collect(B, T, k, d, pad, dt, behind):
    el, rows = DT[dt], T * k + behind
    order = torch.randperm(rows, generator=gen(T), device="cuda")[: T * k].to(torch.int32)
    pos = order.view(T, k).contiguous()
    if T > 4:  # padding and rows that are not there
        pos[2] = -1
        pos[3, 0] = rows
        pos[3, k - 1] = -2 ** 31
    z, dy = randn((rows, d), el, 1, pad), randn((T, d), el, 2, pad)
    w = randn((T, k), torch.float32, 3)
    ok = (pos >= 0) & (pos < rows)
    at = torch.where(ok, pos, 0).long().cpu()
    used = torch.zeros(rows, dtype=torch.bool)
    used[pos[ok].long().cpu()] = True
    z[~used.cuda()] = float("nan")  # of nobody: not read
    zc = torch.nan_to_num(z.double()).cpu()
    okc, wc, dyc = ok.cpu(), w.double().cpu(), dy.double().cpu()
    for weighted in (True, False):
        wj = torch.where(okc, wc if weighted else torch.ones_like(wc), 0.0)
        terms = wj.unsqueeze(2) * zc[at]
        ref, mag = terms.sum(dim=1), terms.abs().sum(dim=1)
        buf = torch.full((T + 1, d + pad), 77.0, dtype=el, device="cuda")
        y = buf[:T, :d]
        B.moe_collect(z, pos, y, weight=w if weighted else None)
        check(y.double().cpu().numpy(), ref.numpy(), R.sum_bound(ref, mag, k, el).numpy(), "y")
        assert (buf[T] == 77.0).all() and (buf[:, d:] == 77.0).all()

        ref = torch.full((rows, d), 77.0, dtype=torch.float64)
        ref[at[okc]] = (wj.unsqueeze(2) * dyc.unsqueeze(1))[okc]
        bound = R.sum_bound(ref, ref.abs(), 1, el)
        dref = torch.where(okc, (zc[at] * dyc.unsqueeze(1)).sum(dim=2), 0.0)
        dmag = (zc[at] * dyc.unsqueeze(1)).abs().sum(dim=2)
        for what in ("both", "dz", "dweight"):
            buf = torch.full((rows, d + pad), 77.0, dtype=el, device="cuda")
            dz = buf[:, :d] if what != "dweight" else None
            dw = torch.full((T, k), 77.0, device="cuda") if what != "dz" else None
            B.moe_collect_backward(dy, pos, dz, weight=w if weighted else None,
                                   z=z if dw is not None else None, dweight=dw)
            if dz is not None:
                check(dz.double().cpu().numpy(), ref.numpy(), bound.numpy(), "dz")
                assert (buf[~used.cuda()] == 77.0).all() and (buf[:, d:] == 77.0).all()
            if dw is not None:
                check(dw.cpu().numpy(), dref.numpy(),
                      R.sum_bound(dref, dmag, d, torch.float32).numpy(), "dweight")
