"""The ragged expert operators where bounds from the arithmetic say little: small
whole numbers, whose sums fp32 holds exactly, compared for equality, at widths
below 16 bytes and over experts of many rows."""
import pytest
import torch

import ragged_util as R
from ragged_util import DT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from round_dropless_expert_amd import binding
    binding.load()
    binding.check_runtime()
    return binding


def whole(shape, dtype, seed):
    """Whole numbers from -2 to 2: a sum of n products is exact in fp32 for
    4 n <= 2^24, in any order."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-2, 3, shape, generator=gen, device="cuda").to(dtype)


def dev_off(off):
    return torch.from_numpy(off).cuda()


# matrices of rows shorter than 16 bytes, one after the other, with few rows
# behind the last whole stage (of 32 to 256 values of c)
@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("rows", [129, 257, 513])
@pytest.mark.parametrize("narrow", [1, 2, 3, 5])
def test_rows_shorter_than_16_bytes(B, dt, rows, narrow):
    el = DT[dt]
    for N, K in [(narrow, 512), (512, narrow), (narrow, 257), (257, narrow), (513, narrow)]:
        off = R.offsets_of([rows])
        x, dy, w = whole((rows, K), el, 1), whole((rows, N), el, 2), whole((1, N, K), el, 3)
        g = B.grouped(rows, 1, N, K, el)
        y, dx = torch.empty(rows, N, dtype=el, device="cuda"), torch.empty_like(x)
        dw = torch.empty(1, N, K, device="cuda")
        ws = torch.empty(B.grouped_dw_workspace_size(g), dtype=torch.uint8, device="cuda")
        B.moe_grouped_gemm(g, dev_off(off), x, w, y)
        B.moe_grouped_gemm_dx(g, dev_off(off), dy, w, dx)
        B.moe_grouped_gemm_dw(g, dev_off(off), x, dy, dw, ws)
        assert torch.equal(y.cpu(), R.product(off, x, w, rows)[0].to(el)), (N, K)
        assert torch.equal(dx.cpu(), R.product(off, dy, w, rows, transpose=True)[0].to(el)), (N, K)
        assert torch.equal(dw.double().cpu(), R.weight_grad(off, x, dy, 1)[0]), (N, K)


def mm(a, b):
    """fp64 product on the device: exact for these numbers."""
    return torch.mm(a.double().contiguous(), b.double().contiguous())


def expect(off, a, w, el):
    """a[i] w[e]^T, rounded once; rows of nobody are 0."""
    y = torch.zeros(a.shape[0], w.shape[1], dtype=el, device="cuda")
    for e, b, t in R.segments(off):
        if t > b:
            y[b:t] = mm(a[b:t], w[e].t()).to(el)
    return y


# experts of many rows over many chunks, whose sums a bound over all their terms
# could not tell from one with a row lost, in rows that start at 16 bytes (the
# ring for 16-bit types where it has the tiles) and in others
@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("counts,N,K", [
    ([20000, 0, 1, 129, 14000, 640], 200, 256), ([127, 128, 9000, 513, 0, 8191], 520, 264),
    ([3000, 1, 0, 2000], 1024, 2048)])
def test_weight_gradient_misses_and_doubles_no_row(B, dt, pad, counts, N, K):
    el, off = DT[dt], R.offsets_of(counts, 2)
    rows, E = int(off[-1]) + 3, len(counts)
    x, dy = whole((rows, K + pad), el, 1)[:, :K], whole((rows, N + pad), el, 2)[:, :N]
    g = B.grouped(rows, E, N, K, el, ld_x=K + pad, ld_y=N + pad)
    ws = torch.full((B.grouped_dw_workspace_size(g),), 255, dtype=torch.uint8, device="cuda")
    dw = torch.full((E, N, K), float("nan"), device="cuda")
    ref = torch.stack([mm(dy[b:t].t(), x[b:t]) for _, b, t in R.segments(off)])
    B.moe_grouped_gemm_dw(g, dev_off(off), x, dy, dw, ws)
    assert torch.equal(dw.double(), ref)
    was = whole((E, N, K), torch.float32, 3)
    dw.copy_(was)
    B.moe_grouped_gemm_dw(g, dev_off(off), x, dy, dw, ws, accumulate=True)
    assert torch.equal(dw.double(), ref + was.double())


def test_weight_gradient_past_4_gib_misses_and_doubles_no_row(B):
    """One expert with nearly all rows of a buffer of 4.9 GB, in many chunks:
    columns at both ends and in the middle."""
    rows, N, K, el = 300_000, 256, 8192, torch.bfloat16
    off = R.offsets_of([5, rows - 135, 130])
    x, dy = whole((rows, K), torch.int8, 1).to(el), whole((rows, N), el, 2)
    g = B.grouped(rows, 3, N, K, el)
    ws = torch.full((B.grouped_dw_workspace_size(g),), 255, dtype=torch.uint8, device="cuda")
    dw = torch.empty(3, N, K, device="cuda")
    B.moe_grouped_gemm_dw(g, dev_off(off), x, dy, dw, ws)
    cols = [0, 1, 255, 256, 4095, 8190, 8191]
    for e, b, t in R.segments(off):
        assert torch.equal(dw[e][:, cols].double(), mm(dy[b:t].t(), x[b:t][:, cols])), e


# every tile of the products, with sums too long for a bound to see one term:
# the ring's 256 x 256, 256 x 128 and 128 x 64, the skinny kernel, and (3 more
# elements a row) the general kernel; K ends inside a stage and inside a slot
@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("counts,N,K,pad", [
    ([4000, 0, 4192], 4096, 2088, 0), ([1500, 260], 2048, 4104, 0), ([70, 0, 300, 64], 2000, 7168, 0),
    ([1], 4096, 4112, 0), ([3, 0, 30], 1000, 7160, 0), ([700, 0, 33], 520, 4099, 3),
    ([2], 300, 4099, 3)])
def test_products_miss_and_double_no_term(B, dt, counts, N, K, pad):
    el, off = DT[dt], R.offsets_of(counts, 1)
    rows, E = int(off[-1]) + 2, len(counts)
    x, dy = whole((rows, K + pad), el, 1)[:, :K], whole((rows, N + pad), el, 2)[:, :N]
    w = whole((E, N, K), el, 3)
    g = B.grouped(rows, E, N, K, el, ld_x=K + pad, ld_y=N + pad)
    y = torch.zeros(rows, N + pad, dtype=el, device="cuda")[:, :N]
    dx = torch.zeros(rows, K + pad, dtype=el, device="cuda")[:, :K]
    B.moe_grouped_gemm(g, dev_off(off), x, w, y)
    assert torch.equal(y, expect(off, x, w, el))
    B.moe_grouped_gemm_dx(g, dev_off(off), dy, w, dx)
    assert torch.equal(dx, expect(off, dy, w.transpose(1, 2), el))


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("counts,N,K", [
    ([4000, 0, 4192], 4096, 2080), ([1500, 260], 2048, 4128), ([70, 0, 300, 64], 2000, 7168),
    ([1], 4096, 4096), ([3, 0, 30], 1000, 7136)])
def test_mxfp4_products_miss_and_double_no_term(B, dt, counts, N, K):
    """Values of 1/4 to 12 in steps that make every product a multiple of 1/16
    of at most 144: sums of 7168 of them are exact in fp32."""
    el, off = DT[dt], R.offsets_of(counts, 1)
    rows, E, S = int(off[-1]) + 2, len(counts), B.mxfp4_scale_stride(K)
    gen = torch.Generator(device="cuda").manual_seed(1)
    levels = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
    levels = torch.cat([levels, -levels]).cuda()

    def operand(n):
        c = torch.randint(0, 16, (n, K), generator=gen, device="cuda", dtype=torch.uint8)
        s = torch.randint(126, 129, (n, S), generator=gen, device="cuda", dtype=torch.uint8)
        f = torch.exp2(s[:, : K // 32].double() - 127).repeat_interleave(32, dim=1)
        s[:, K // 32:] = 255  # the padding is never used
        return c[:, 0::2] | (c[:, 1::2] << 4), s, levels[c.int()] * f

    xq, xs, xv = operand(rows)
    wq, wsc, wv = operand(E * N)
    y = torch.zeros(rows, N, dtype=el, device="cuda")
    B.moe_mxfp4_grouped_gemm(B.grouped(rows, E, N, K, el), dev_off(off), xq, xs, wq, wsc, y)
    ref = torch.zeros(rows, N, dtype=torch.float64, device="cuda")
    for e, b, t in R.segments(off):
        if t > b:
            ref[b:t] = mm(xv[b:t], wv.view(E, N, K)[e].t())
    assert torch.equal(y, ref.float().to(el))


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("f,pad", [(2048, 0), (37, 3)])
def test_swiglu_where_the_gate_is_below_fp32(B, dt, f, pad):
    """s(g) down to and below 2^-126 against u and dh that bring the outputs back
    into range: nothing is flushed."""
    el = DT[dt]
    fi = torch.finfo(el)
    gs = [-60.0, -80.0, -85.5, -86.0, -86.5, -87.0, -87.5, -88.0, -90.0, -100.0, -103.5, -104.0,
          -120.0, -150.0, -200.0, -250.0, -280.0, -300.0, -500.0, -1000.0, -1023.0, -1024.0,
          -1032.0, -3000.0]
    gs = gs + [30.0, 100.0, -1.0, 0.0]
    vals = [1.0, -1e30, 3e38, -1e36, 1e4, 1e-3]
    rows = len(vals) ** 2
    gen = torch.Generator().manual_seed(1)
    g = torch.tensor(gs)[torch.randint(0, len(gs), (rows, f), generator=gen)].to(el)
    u = torch.tensor(vals).clamp(-fi.max, fi.max).repeat_interleave(len(vals))
    d = torch.tensor(vals).clamp(-fi.max, fi.max).repeat(len(vals))
    u, d = (v.to(el).unsqueeze(1).expand(rows, f) for v in (u, d))

    def padded(t):
        b = torch.zeros(rows, t.shape[1] + pad, dtype=el, device="cuda")[:, :t.shape[1]]
        b.copy_(t)
        return b

    gu, dh = padded(torch.cat([g, u], dim=1)), padded(d)
    h, dgu = padded(torch.zeros_like(d)), padded(torch.zeros(rows, 2 * f, dtype=el))
    B.moe_swiglu(gu, h)
    B.moe_swiglu_backward(gu, dh, dgu)
    g, u, d = g.double(), u.double(), d.double()
    s, r = torch.sigmoid(g), torch.sigmoid(-g)
    # exponential, reciprocal and products, each within an ulp or two (2^-21
    # covers eight roundings); of 16-bit types the exponent's argument from -86
    # on is rounded to fp32, off by |g| 2^-24 in all
    rel = 2.0 ** -21 + (0.0 if dt == "f32" else torch.where(g < -86, 0.0, g.abs() * 2.0 ** -23))

    def near(got, ref, tol, what):
        ok = ref.abs() < fi.max / 4  # no partial product overflows either
        # fp32 subnormals on the way to the output: 2^-149
        bound = tol + R.rounding(ref.abs() + tol, el) + 2.0 ** -149
        err = (got.double().cpu() - ref).abs()
        bad = ok & ~(err <= bound)
        assert not bad.any(), (what, int(bad.sum()), g[bad][0], u[bad][0], d[bad][0],
                               got.double().cpu()[bad][0], ref[bad][0])

    href = g * s * u
    near(h, href, href.abs() * rel, "h")
    du = d * g * s
    near(dgu[:, f:], du, du.abs() * rel, "du")
    # from -86 on dh s (1 + g (1 - s)) is fp32 before u comes in, so that half a
    # step of its subnormals counts u times
    dg = d * u * s * (1 + g * r)
    tol = (d * u).abs() * s * (1 + (g * r).abs()) * 2 * rel
    near(dgu[:, :f], dg, tol + torch.where(g < -86, 0.0, u.abs() * 2.0 ** -149), "dg")


def test_transposed_weights_are_refused(B):
    """Layouts that have the right number of elements and other rows."""
    el, rows, E, N, K = torch.bfloat16, 8, 2, 16, 64
    zeros = lambda *n, dtype=el: torch.zeros(*n, dtype=dtype, device="cuda")
    g, off = B.grouped(rows, E, N, K, el), torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    x, y, S = zeros(rows, K), zeros(rows, N), B.mxfp4_scale_stride(K)
    u8 = lambda *n: zeros(*n, dtype=torch.uint8)
    ops = [u8(rows, K // 2), u8(rows, S), u8(E, N, K // 2), u8(E, N, S)]
    calls = [
        lambda w: B.moe_grouped_gemm(g, off, x, w, y),
        lambda w: B.moe_grouped_gemm_dx(g, off, y, w, x),
        lambda w: B.moe_grouped_gemm_dw(g, off, x, y, w.float()),
        lambda w: B.moe_mxfp4_quantize(w, u8(E, K, N // 2), u8(E, N, S)),
        lambda w: B.moe_mxfp4_quantize(w, u8(E, N, K // 2), u8(E, S, N)),
    ]
    for i in range(4):
        t = [*ops]
        t[i] = t[i].reshape(*t[i].shape[:-2], t[i].shape[-1], t[i].shape[-2])
        calls.append(lambda w, t=t: B.moe_mxfp4_grouped_gemm(g, off, *t, y))
    for f in calls[:3]:
        f(zeros(E, N, K)), f(zeros(E * N, K)), f(zeros(E, 2, N // 2, K)), f(zeros(E * N * K))
        with pytest.raises(ValueError, match="shape"):
            f(zeros(E, K, N))
    for f in calls[3:]:
        with pytest.raises(ValueError, match="shape"):
            f(zeros(E, N, K))


def test_dequantised_values_are_exact_or_infinite(B):
    """Every code under every scale byte against fp64: bf16 and fp32 hold all
    values but those past their largest, which are infinite; fp16 rounds."""
    import numpy as np
    c = np.tile(np.arange(16, dtype=np.uint8), (255, 2))
    codes = torch.from_numpy(R.pack(c)).cuda()
    scales = torch.zeros(255, 4, dtype=torch.uint8, device="cuda")
    scales[:, 0] = torch.arange(255, dtype=torch.uint8)
    ref = torch.from_numpy(R.values_of(c, np.arange(255, dtype=np.uint8)[:, None]))
    for el in DT.values():
        y = torch.empty(255, 32, dtype=el, device="cuda")
        B.moe_mxfp4_dequantize(codes, scales, y)
        y = y.double().cpu()
        past = ref.abs() > torch.finfo(el).max
        if el != torch.float16:
            assert past.nonzero()[:, 0].unique().tolist() == [253, 254]
            assert torch.equal(y[~past], ref[~past])
        else:
            assert torch.equal(y[~past], ref[~past].to(el).double())
        assert torch.equal(y[past], torch.copysign(torch.full_like(ref[past], torch.inf), ref[past]))


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("N,K,pad", [(16, 2 ** 20, 0), (2 ** 20, 16, 0), (5, 2 ** 20 - 3, 3),
                                     (2 ** 20 - 8, 3, 8)])
def test_the_widest_rows(B, dt, N, K, pad):
    """Rows of 2^20 elements, the limit: a few of two experts, every product."""
    el, off = DT[dt], R.offsets_of([2, 0, 70])
    rows, E = int(off[-1]), 3
    ld_x, ld_y = (K + pad, N) if K > N else (K, N + pad)
    x = whole((rows, ld_x), torch.int8, 1).to(el)[:, :K]
    dy = whole((rows, ld_y), torch.int8, 2).to(el)[:, :N]
    w = whole((E, N, K), torch.int8, 3).to(el)
    g = B.grouped(rows, E, N, K, el, ld_x=ld_x, ld_y=ld_y)
    y = torch.zeros(rows, ld_y, dtype=el, device="cuda")[:, :N]
    dx = torch.zeros(rows, ld_x, dtype=el, device="cuda")[:, :K]
    dw = torch.empty(E, N, K, device="cuda")
    ws = torch.empty(B.grouped_dw_workspace_size(g), dtype=torch.uint8, device="cuda")
    B.moe_grouped_gemm(g, dev_off(off), x, w, y)
    B.moe_grouped_gemm_dx(g, dev_off(off), dy, w, dx)
    B.moe_grouped_gemm_dw(g, dev_off(off), x, dy, dw, ws)
    assert torch.equal(y, expect(off, x, w, el))
    assert torch.equal(dx, expect(off, dy, w.transpose(1, 2), el))
    for e, b, t in R.segments(off):
        assert torch.equal(dw[e].double(), mm(dy[b:t].t(), x[b:t])), e


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_the_widest_rows_elementwise(B, dt):
    el, rows, K = DT[dt], 3, 2 ** 20
    gen = torch.Generator(device="cuda").manual_seed(1)
    gu = torch.randn(rows, K, generator=gen, device="cuda").to(el)
    dh = torch.randn(rows, K // 2, generator=gen, device="cuda").to(el)
    h, dgu = torch.empty_like(dh), torch.empty_like(gu)
    B.moe_swiglu(gu, h)
    B.moe_swiglu_backward(gu, dh, dgu)
    g, u, d = gu[:, : K // 2].double(), gu[:, K // 2:].double(), dh.double()
    s, r = torch.sigmoid(g), torch.sigmoid(-g)
    # as for narrow rows: 2^-20 covers the fp32 arithmetic of |g| < 8
    for got, ref, size in ((h, g * s * u, g * s * u), (dgu[:, K // 2:], d * g * s, d * g * s),
                           (dgu[:, : K // 2], d * u * s * (1 + g * r),
                            d * u * s * (1 + (g * r).abs()))):
        tol = size.abs() * 2.0 ** -20
        assert ((got.double() - ref).abs() <= tol + R.rounding(ref.abs() + tol, el)).all()
    codes = torch.empty(rows, K // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(rows, K // 32, dtype=torch.uint8, device="cuda")
    B.moe_mxfp4_quantize(gu, codes, scales)
    c, sc = R.codes_of(gu.double().cpu().numpy())
    assert (R.unpack(codes.cpu().numpy()) == c).all() and (scales.cpu().numpy() == sc).all()


def test_three_hundred_million_rows(B):
    """Row numbers past 2^28 and element numbers past 2^31 in every operator."""
    rows, K, N, el = 300_000_007, 8, 8, torch.bfloat16
    off = R.offsets_of([5, 0, rows - 1000, 990], 2)
    d_off, E, end = dev_off(off), 4, int(off[-1])
    x = whole((rows, K), torch.int8, 1).to(el)
    w = whole((E, N, K), el, 2)
    y = torch.full((rows, N), 77.0, dtype=el, device="cuda")
    g = B.grouped(rows, E, N, K, el)

    def same(got, a, m):  # got[i] = a[i] m[e]^T, in parts
        for e, b, t in R.segments(off):
            for i in range(b, t, 1 << 24):
                j = min(t, i + (1 << 24))
                assert torch.equal(got[i:j], (a[i:j].float() @ m[e].float().t()).to(el)), (e, i)
        assert (got[:2] == 77.0).all() and (got[end:] == 77.0).all()

    B.moe_grouped_gemm(g, d_off, x, w, y)
    same(y, x, w)
    y.fill_(77.0)
    B.moe_grouped_gemm_dx(g, d_off, x, w, y)
    same(y, x, w.transpose(1, 2).contiguous())
    # a few rows of dy that are not 0, at both ends of every expert and between
    y.zero_()
    some = [2, 6, 7, 8, 2 ** 28 - 1, 2 ** 28, end - 991, end - 990, end - 1]
    y[some] = whole((len(some), N), el, 3)
    y[:2] = y[end:] = float("nan")
    dw = torch.empty(E, N, K, device="cuda")
    ws = torch.empty(B.grouped_dw_workspace_size(g), dtype=torch.uint8, device="cuda")
    B.moe_grouped_gemm_dw(g, d_off, x, y, dw, ws)
    ref = torch.zeros(E, N, K, dtype=torch.float64, device="cuda")
    for i in some:
        e = 0 if i < 7 else 2 if i < end - 990 else 3
        ref[e] += y[i].double().unsqueeze(1) * x[i].double()
    assert torch.equal(dw.double(), ref)
    # x as [g, u] of four features
    h = torch.full((rows, 4), 77.0, dtype=el, device="cuda")
    B.moe_swiglu(x, h, n_rows=d_off[E:])
    B.moe_swiglu_backward(x, h, y, n_rows=d_off[E:])
    for i in (0, 2 ** 28 - 2, end - 64):
        gg, u, d = (t[i:i + 64].double().cpu() for t in (x[:, :4], x[:, 4:], h))
        href, du = gg * torch.sigmoid(gg) * u, d * gg * torch.sigmoid(gg)
        for got, want in ((d, href), (y[i:i + 64, 4:].double().cpu(), du)):
            tol = want.abs() * 2.0 ** -20
            assert ((got - want).abs() <= tol + R.rounding(want.abs() + tol, el)).all(), i
    assert (h[end:] == 77.0).all() and torch.isnan(y[end:]).all()
    del h, y
    # the same values as rows of 32, in four bits and back
    n = rows * K // 32
    xq = torch.empty(n, 16, dtype=torch.uint8, device="cuda")
    xs = torch.empty(n, 4, dtype=torch.uint8, device="cuda")
    x = x.view(-1)[: n * 32].view(n, 32)
    B.moe_mxfp4_quantize(x, xq, xs)
    back = torch.empty_like(x)
    B.moe_mxfp4_dequantize(xq, xs, back)
    assert torch.equal(back, x)  # -2 to 2 are 4-bit values under the scale 2^-1


def test_two_threads_on_two_streams(B):
    """Calls that overlap in time, each with outputs and a workspace of its own."""
    import threading
    el, c, N, K = torch.bfloat16, [3000, 0, 1500, 4], 264, 520
    off = R.offsets_of(c)
    rows, E, d_off = int(off[-1]), len(c), dev_off(off)
    g = B.grouped(rows, E, N, K, el)
    size = B.grouped_dw_workspace_size(g)
    sets = []
    for seed in (1, 2):
        sets.append(dict(
            x=whole((rows, K), el, seed), dy=whole((rows, N), el, seed + 2),
            w=whole((E, N, K), el, seed + 4), y=torch.zeros(rows, N, dtype=el, device="cuda"),
            dx=torch.zeros(rows, K, dtype=el, device="cuda"), dw=torch.zeros(E, N, K, device="cuda"),
            ws=torch.empty(size, dtype=torch.uint8, device="cuda"), st=torch.cuda.Stream()))
    torch.cuda.synchronize()

    def calls(s):
        with torch.cuda.stream(s["st"]):
            for _ in range(20):
                B.moe_grouped_gemm(g, d_off, s["x"], s["w"], s["y"])
                B.moe_grouped_gemm_dx(g, d_off, s["dy"], s["w"], s["dx"])
                B.moe_grouped_gemm_dw(g, d_off, s["x"], s["dy"], s["dw"], s["ws"])

    threads = [threading.Thread(target=calls, args=(s,)) for s in sets]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for s in sets:
        assert torch.equal(s["y"], expect(off, s["x"], s["w"], el))
        assert torch.equal(s["dx"], expect(off, s["dy"], s["w"].transpose(1, 2), el))
        for e, b, t in R.segments(off):
            assert torch.equal(s["dw"][e].double(), mm(s["dy"][b:t].t(), s["x"][b:t]))
