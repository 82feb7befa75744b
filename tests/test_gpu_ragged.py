"""The ragged expert operators on the GPU against plain fp64 forms: grouped
products and their gradients, SwiGLU, MXFP4 quantisation and product, and a
run of them together. Every bound follows from the arithmetic
(ragged_util.sum_bound, rounding)."""
import numpy as np
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


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(shape, dtype, seed, pad=0, scale=1.0):
    t = torch.randn(*shape[:-1], shape[-1] + pad, generator=gen(seed), device="cuda") * scale
    return t.to(dtype)[..., : shape[-1]]


def dev_off(off):
    return torch.from_numpy(off).cuda()


def check(got, ref, bound, what):
    err = (got.double().cpu() - ref).abs()
    bad = ~(err <= bound)
    assert not bad.any(), (
        f"{what}: {int(bad.sum())} of {bad.numel()} past the bound, first at "
        f"{tuple(bad.nonzero()[0].tolist())}, worst {(err / bound).max():.3f} of it")


SENTINEL = 77.0


def filled(rows, cols, dtype, pad):
    return torch.full((rows, cols + pad), SENTINEL, dtype=dtype, device="cuda")[:, :cols]


# counts per expert, rows before the first and behind the last sequence
COUNTS = {
    "one_row": ([1], 0, 0),
    "one_of_four": ([0, 0, 1, 0], 0, 3),
    "empty": ([0, 0, 0], 0, 5),
    "few": ([3, 0, 17, 1, 40], 2, 1),
    "hot": ([5, 700, 0, 9], 0, 64),
    "long": ([0, 1500, 64, 2, 300], 7, 0),
    "many": ([i % 5 for i in range(130)], 0, 9),
}
SIZES = [(1, 1), (7, 5), (64, 64), (33, 200), (256, 128), (520, 72), (264, 1000), (1024, 512)]


def case_list():
    out = []
    for i, (name, _) in enumerate(COUNTS.items()):
        for j, (N, K) in enumerate(SIZES):
            if name == "many" and N * K > 8192:
                continue
            dt = ["bf16", "f16", "f32"][(i + j) % 3]
            out.append((dt, name, N, K, [0, 8, 3][(i + 2 * j) % 3]))
    # every type on the aligned sizes that the wide tiles take
    for dt in DT:
        out += [(dt, "long", 512, 512, 0), (dt, "hot", 768, 256, 64), (dt, "few", 2048, 1024, 0)]
    return sorted(set(out))


@pytest.mark.parametrize("dt,counts,N,K,pad", case_list())
def test_product_and_gradients(B, dt, counts, N, K, pad):
    c, before, behind = COUNTS[counts]
    off = R.offsets_of(c, before)
    rows, E, el = int(off[-1]) + behind, len(c), DT[dt]
    x, w = randn((rows, K), el, 1, pad), randn((E, N, K), el, 2, 0, K ** -0.5)
    dy = randn((rows, N), el, 3, pad)
    # nothing of what belongs to nobody may be read
    nan = float("nan")
    for t in (x, dy):
        t[:before] = nan
        t[int(off[-1]):] = nan
    for e, n in enumerate(c):
        if n == 0:
            w[e] = nan
    g = B.grouped(rows, E, N, K, el, ld_x=K + pad, ld_y=N + pad)
    d_off = dev_off(off)
    wc = torch.nan_to_num(w.double()).cpu()
    live = torch.zeros(rows, dtype=torch.bool)
    live[before:int(off[-1])] = True

    y = filled(rows, N, el, pad)
    B.moe_grouped_gemm(g, d_off, x, w, y)
    ref, s = R.product(off, x, wc, rows)
    check(y[live], ref[live], R.sum_bound(ref, s, K, el)[live], "y")
    assert (y[~live] == SENTINEL).all()

    dx = filled(rows, K, el, pad)
    B.moe_grouped_gemm_dx(g, d_off, dy, w, dx)
    ref, s = R.product(off, dy, wc, rows, transpose=True)
    check(dx[live], ref[live], R.sum_bound(ref, s, N, el)[live], "dx")
    assert (dx[~live] == SENTINEL).all()

    ws = torch.full((B.grouped_dw_workspace_size(g),), 255, dtype=torch.uint8, device="cuda")
    dw = torch.full((E, N, K), nan, device="cuda")
    B.moe_grouped_gemm_dw(g, d_off, x, dy, dw, ws)
    ref, s = R.weight_grad(off, x, dy, E)
    check(dw, ref, R.sum_bound(ref, s, max(c), torch.float32), "dw")
    # added to what is there
    dw0 = dw.clone()
    B.moe_grouped_gemm_dw(g, d_off, x, dy, dw, ws, accumulate=True)
    check(dw, 2 * ref, R.sum_bound(2 * ref, 2 * s, 2 * max(c) + 1, torch.float32), "dw added")
    # and the same bits again
    dw1 = torch.empty_like(dw0)
    B.moe_grouped_gemm_dw(g, d_off, x, dy, dw1, ws)
    assert torch.equal(dw0, dw1)
    # padding of the rows is nobody's either
    if pad:
        for t in (y, dx):
            base = torch.as_strided(t, (rows, t.shape[1] + pad), (t.shape[1] + pad, 1))
            assert (base[:, t.shape[1]:] == SENTINEL).all()


@pytest.mark.parametrize("dt", list(DT))
def test_rows_do_not_depend_on_the_call(B, dt):
    """The same row gives the same bits whatever the other rows are, as long
    as the buffers' sizes choose the same kernel, and from call to call."""
    el, N, K = DT[dt], 512, 512
    c = [600, 0, 424]
    off = R.offsets_of(c)
    x, w = randn((1024, K), el, 5), randn((3, N, K), el, 6, 0, K ** -0.5)
    g = B.grouped(1024, 3, N, K, el)
    y = filled(1024, N, el, 0)
    B.moe_grouped_gemm(g, dev_off(off), x, w, y)
    # expert 2's rows alone, at the start of the buffer
    x2 = torch.zeros_like(x)
    x2[:424] = x[600:]
    y2 = filled(1024, N, el, 0)
    B.moe_grouped_gemm(g, dev_off(R.offsets_of([0, 0, 424])), x2, w, y2)
    assert torch.equal(y2[:424], y[600:])


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("N,K", [(72, 40), (512, 256)])
def test_infinities_and_nan_stay_in_their_rows(B, dt, N, K):
    el = DT[dt]
    off = R.offsets_of([130, 70])
    x, w = randn((200, K), el, 1), randn((2, N, K), el, 2)
    x[5, 3] = float("inf")
    x[140, K - 1] = float("nan")
    g = B.grouped(200, 2, N, K, el)
    y = filled(200, N, el, 0)
    B.moe_grouped_gemm(g, dev_off(off), x, w, y)
    ok = torch.isfinite(y).all(dim=1).cpu()
    assert (~ok).nonzero().flatten().tolist() == [5, 140]
    assert torch.isinf(y[5]).all() and torch.isnan(y[140]).all()
    assert torch.equal(torch.signbit(y[5]), torch.signbit(w[0, :, 3]))


@pytest.mark.parametrize("dt", list(DT))
def test_weight_gradient_over_many_chunks(B, dt):
    """An expert with most of the rows: its sum goes through the workspace."""
    el, N, K, rows = DT[dt], 128, 192, 9000
    off = R.offsets_of([8000, 0, 600, 400])
    x, dy = randn((rows, K), el, 1), randn((rows, N), el, 2)
    g = B.grouped(rows, 4, N, K, el)
    need = B.grouped_dw_workspace_size(g)
    assert need > 0
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    dw = torch.empty(4, N, K, device="cuda")
    B.moe_grouped_gemm_dw(g, dev_off(off), x, dy, dw, ws)
    ref, s = R.weight_grad(off, x, dy, 4)
    check(dw, ref, R.sum_bound(ref, s, 8000, torch.float32), "dw")
    assert (dw[1] == 0).all()
    # added to what is there, at an address that is only four-byte aligned
    buf = torch.full((4 * N * K + 1,), 2.0, device="cuda")
    dw2 = buf[1:].view(4, N, K)
    B.moe_grouped_gemm_dw(g, dev_off(off), x, dy, dw2, ws, accumulate=True)
    check(dw2, ref + 2, R.sum_bound(ref + 2, s + 2, 8001, torch.float32), "dw added")
    assert buf[0] == 2.0 and (dw2[1] == 2.0).all()
    # a width that ends inside 16 bytes, and too small a workspace
    g3 = B.grouped(rows, 4, N, 190, el, ld_x=K)
    ws3 = torch.empty(B.grouped_dw_workspace_size(g3), dtype=torch.uint8, device="cuda")
    dw3 = torch.empty(4, N, 190, device="cuda")
    B.moe_grouped_gemm_dw(g3, dev_off(off), x[:, :190], dy, dw3, ws3)
    check(dw3, ref[:, :, :190], R.sum_bound(ref, s, 8000, torch.float32)[:, :, :190], "dw narrow")
    with pytest.raises(B.MoeError):
        B.moe_grouped_gemm_dw(g, dev_off(off), x, dy, dw, ws[:-1])
    with pytest.raises(B.MoeError):
        B.moe_grouped_gemm_dw(g, dev_off(off), x, dy, dw)


def test_no_rows(B):
    g = B.grouped(0, 3, 16, 8, "bf16")
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    e = torch.empty(0, 8, dtype=torch.bfloat16, device="cuda")
    y = torch.empty(0, 16, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(3, 16, 8, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((3, 16, 8), 5.0, device="cuda")
    B.moe_grouped_gemm(g, off, e, w, y)
    B.moe_grouped_gemm_dx(g, off, y, w, e)
    B.moe_grouped_gemm_dw(g, off, e, y, dw, accumulate=True)
    assert (dw == 5.0).all()
    B.moe_grouped_gemm_dw(g, off, e, y, dw)
    assert (dw == 0).all()
    B.moe_swiglu(torch.empty(0, 8, device="cuda"), torch.empty(0, 4, device="cuda"))
    q = torch.empty(0, 16, dtype=torch.uint8, device="cuda")
    B.moe_mxfp4_quantize(torch.empty(0, 32, device="cuda"), q, q)
    B.moe_mxfp4_dequantize(q, q, torch.empty(0, 32, device="cuda"))


@pytest.mark.parametrize("rows,N,K,raw", [
    (8, 64, 64, [-5, 3, 2, 9]), (8, 64, 64, [0, 100, 100, 100]), (8, 64, 64, [9, 4, 0, -1]),
    (8, 64, 64, [-(2 ** 31), 2 ** 31 - 1, -(2 ** 31), 2 ** 31 - 1]),
    (2000, 512, 512, [0, 2000, 0, 2000]), (2000, 512, 512, [2000, 0, 1500, 100]),
    (2000, 512, 512, [-7, 5000, 3, 1999])])
def test_wrong_offsets_stay_inside_the_buffers(B, rows, N, K, raw):
    """Offsets outside [0, rows] or out of order: no result is promised, but
    nothing outside the outputs is written (guard rows around them)."""
    E = 3
    off = torch.tensor(raw, dtype=torch.int32, device="cuda")
    x, w = randn((rows, K), torch.bfloat16, 1), randn((E, N, K), torch.bfloat16, 2)
    buf = torch.full((rows + 512, N), SENTINEL, dtype=torch.bfloat16, device="cuda")
    y = buf[256:256 + rows]
    g = B.grouped(rows, E, N, K, "bf16")
    B.moe_grouped_gemm(g, off, x, w, y)
    B.moe_grouped_gemm_dx(g, off, x, w, y)
    assert (buf[:256] == SENTINEL).all() and (buf[256 + rows:] == SENTINEL).all()
    dw = torch.full((E + 2, N, K), SENTINEL, device="cuda")
    ws = torch.empty(B.grouped_dw_workspace_size(g), dtype=torch.uint8, device="cuda")
    B.moe_grouped_gemm_dw(g, off, x, x, dw[1:1 + E], ws)
    assert (dw[0] == SENTINEL).all() and (dw[-1] == SENTINEL).all()
    _, _, xq, xsc = mx_operand(rows, K, 1)
    _, _, wq, wsc = mx_operand(E * N, K, 2)
    B.moe_mxfp4_grouped_gemm(g, off, xq, xsc, wq, wsc, y)
    assert (buf[:256] == SENTINEL).all() and (buf[256 + rows:] == SENTINEL).all()


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("rows,f,pad", [(1, 1, 0), (5, 1001, 3), (9, 64, 8), (300, 256, 0),
                                        (64, 2048, 16)])
def test_swiglu_and_gradient(B, dt, rows, f, pad):
    el = DT[dt]
    gu, dh = randn((rows, 2 * f), el, 1, pad, 3.0), randn((rows, f), el, 2, pad)
    ext = torch.tensor([0.0, -0.0, 100.0, -100.0, 3e3, -3e3, 1e-6, -1e-6, -1.278, 20.0, -20.0,
                        88.8, -88.8])
    n = min(f, ext.numel())
    gu[0, :n] = ext[:n].to(el)
    live = max(1, rows - 2)
    n_rows = torch.tensor([live], dtype=torch.int32, device="cuda")
    h, dgu = filled(rows, f, el, pad), filled(rows, 2 * f, el, pad)
    B.moe_swiglu(gu, h, n_rows=n_rows)
    B.moe_swiglu_backward(gu, dh, dgu, n_rows=n_rows)
    g, u, d = (t.double().cpu() for t in (gu[:, :f], gu[:, f:], dh))
    s, r = torch.sigmoid(g), torch.sigmoid(-g)
    # s and 1 - s: exponential, sum, reciprocal and product, each within an
    # ulp or two (2^-21 covers eight roundings), and for 16-bit types the
    # exponent's argument |g| log2 e rounded to fp32, off by |g| 2^-24 in all;
    # s below 2^-126 may lose bits or vanish
    rel = 2.0 ** -21 + (g.abs() * 2.0 ** -23 if dt != "f32" else 0.0)
    tiny = 2.0 ** -125
    href = g * s * u
    hb = href.abs() * rel + (g * u).abs() * tiny
    check(h[:live], href[:live], (hb + R.rounding(href.abs() + hb, el))[:live], "h")
    t = s * (1 + g * r)
    dg, du = d * u * t, d * g * s
    # 1 + g r cancels near g = -1.278: the error is relative to 1 + |g r|
    gb = (d * u).abs() * (s * (1 + (g * r).abs()) * 2 * rel + (1 + g.abs()) * tiny)
    ub = du.abs() * rel + (d * g).abs() * tiny
    check(dgu[:live, :f], dg[:live], (gb + R.rounding(dg.abs() + gb, el))[:live], "dg")
    check(dgu[:live, f:], du[:live], (ub + R.rounding(du.abs() + ub, el))[:live], "du")
    assert (h[live:] == SENTINEL).all() and (dgu[live:] == SENTINEL).all()


def test_swiglu_gradient_against_differences(B):
    gu = randn((4, 32), torch.float32, 1).contiguous()
    dh = randn((4, 16), torch.float32, 2).contiguous()
    dgu = torch.empty_like(gu)
    B.moe_swiglu_backward(gu, dh, dgu)
    step, f = 2.0 ** -7, 16
    for i, j in [(0, 0), (1, 5), (2, 15), (3, 16), (0, 31)]:
        hs = []
        for sgn in (1, -1):
            v = gu.clone()
            v[i, j] += sgn * step
            h = torch.empty(4, f, device="cuda")
            B.moe_swiglu(v, h)
            hs.append((h.double() * dh.double()).sum().item())
        # central difference: third derivative of g s(g) is below 1, times
        # |u dh| < 10 over 6, step^2; plus fp32 errors of h over the step
        assert abs((hs[0] - hs[1]) / (2 * step) - dgu[i, j].item()) < 10 / 6 * step ** 2 + 1e-3


SPECIAL = [0.0, -0.0, 1.0, 6.0, 7.99, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -5.0, -2.5]


def special_rows(el, K):
    """Blocks of zeros, ties, tiny and huge values, infinities and NaN."""
    fi = torch.finfo(el)
    x = torch.randn(12, K, generator=torch.Generator().manual_seed(3)).double()
    x[0] = 0.0
    x[1, :15] = torch.tensor(SPECIAL, dtype=torch.float64)
    x[2] = x[2] * 2.0 ** -12
    x[3] = x[3] * fi.smallest_normal           # subnormals among them
    x[4] = torch.where(x[4] > 0, fi.max, -fi.max)
    x[5, 3] = float("inf")
    x[6, K - 1] = float("-inf")
    x[7, 0] = float("nan")
    x[8] = fi.smallest_normal * fi.eps         # the least magnitude
    x[9, :32] = 0.0
    x[9, 31] = fi.smallest_normal
    x[10] = torch.arange(K).double() % 33 / 4
    x[11] = -4.0 - torch.arange(K).double() % 16 / 4
    return x.to(el)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("K,pad", [(32, 0), (96, 4), (160, 3), (2048, 8)])
def test_quantize_and_dequantize(B, dt, K, pad):
    el = DT[dt]
    x = torch.zeros(12, K + pad, dtype=el, device="cuda")
    x[:, :K] = special_rows(el, K).cuda()
    x = x[:, :K]
    S = B.mxfp4_scale_stride(K)
    codes = torch.full((12, K // 2), 99, dtype=torch.uint8, device="cuda")
    scales = torch.full((12, S), 99, dtype=torch.uint8, device="cuda")
    B.moe_mxfp4_quantize(x, codes, scales)
    c, s = R.codes_of(x.double().cpu().numpy())
    assert np.array_equal(scales.cpu().numpy()[:, : K // 32], s)
    assert np.array_equal(R.unpack(codes.cpu().numpy()), c)
    assert (scales[:, K // 32:] == 0).all()
    y = filled(12, K, el, pad)
    B.moe_mxfp4_dequantize(codes, scales, y)
    ref = torch.from_numpy(R.values_of(c, s)).to(el)
    assert torch.equal(torch.nan_to_num(y.cpu(), nan=1e3), torch.nan_to_num(ref, nan=1e3))
    assert torch.equal(torch.isnan(y.cpu()), torch.isnan(ref))


def test_dequantize_every_code_and_scale(B):
    """All 16 codes under every scale byte: fp32 and bf16 hold each value."""
    c = np.tile(np.arange(16, dtype=np.uint8), (256, 2))
    codes = torch.from_numpy(R.pack(c)).cuda()
    scales = torch.zeros(256, 4, dtype=torch.uint8, device="cuda")
    scales[:, 0] = torch.arange(256, dtype=torch.uint8)
    ref = R.values_of(c, np.arange(256, dtype=np.uint8)[:, None])
    for el in DT.values():
        y = torch.empty(256, 32, dtype=el, device="cuda")
        B.moe_mxfp4_dequantize(codes, scales, y)
        want = torch.from_numpy(ref).to(torch.float32).to(el)
        assert torch.equal(torch.nan_to_num(y.cpu(), nan=1e3), torch.nan_to_num(want, nan=1e3))


@pytest.mark.parametrize("dt", list(DT))
def test_quantize_gathers_rows(B, dt):
    el, K, T, k = DT[dt], 96, 7, 3
    x = randn((T, K), el, 1, 5)
    idx = [20, 0, 4, 4, -1, 9, 21, 2 ** 31 - 1, -(2 ** 31), 13]
    index = torch.tensor(idx, dtype=torch.int32, device="cuda")
    codes = torch.full((10, K // 2), 99, dtype=torch.uint8, device="cuda")
    scales = torch.full((10, 4), 99, dtype=torch.uint8, device="cuda")
    n_rows = torch.tensor([9], dtype=torch.int32, device="cuda")
    B.moe_mxfp4_quantize(x, codes, scales, index=index, index_div=k, n_rows=n_rows)
    rows = np.zeros((10, K))
    for i, a in enumerate(idx):
        if 0 <= a < T * k:
            rows[i] = x[a // k].double().cpu().numpy()
    c, s = R.codes_of(rows)
    assert np.array_equal(R.unpack(codes.cpu().numpy())[:9], c[:9])
    assert np.array_equal(scales.cpu().numpy()[:9, :3], s[:9])
    assert (codes[9] == 99).all() and (scales[9] == 99).all()


def mx_operand(rows, K, seed, spread=0):
    """Random codes and scales (exponents within 2^+-spread of 2^-2)."""
    rng = np.random.default_rng(seed)
    c = rng.integers(0, 16, (rows, K)).astype(np.uint8)
    s = (125 + rng.integers(-spread, spread + 1, (rows, K // 32))).astype(np.uint8)
    S = (K // 32 + 3) // 4 * 4
    sp = rng.integers(0, 256, (rows, S)).astype(np.uint8)  # the padding is never used
    sp[:, : K // 32] = s
    return c, s, torch.from_numpy(R.pack(c)).cuda(), torch.from_numpy(sp).cuda()


@pytest.mark.parametrize("dt,counts,N,K,pad", [
    ("bf16", "one_row", 16, 32, 0), ("f16", "one_of_four", 33, 64, 3), ("f32", "empty", 16, 96, 0),
    ("f32", "few", 130, 224, 0), ("bf16", "few", 512, 1024, 8), ("f16", "hot", 200, 160, 1),
    ("bf16", "hot", 768, 512, 0), ("f32", "long", 512, 2048, 0), ("bf16", "long", 260, 1056, 0),
    ("bf16", "many", 64, 128, 0), ("f32", "hot", 1, 128, 5), ("f16", "long", 1024, 256, 0)])
def test_mxfp4_product(B, dt, counts, N, K, pad):
    c, before, behind = COUNTS[counts]
    off = R.offsets_of(c, before)
    rows, E, el = int(off[-1]) + behind, len(c), DT[dt]
    xc, xs, xq, xsc = mx_operand(rows, K, 1, 3)
    wc, wsb, wq, wsc = mx_operand(E * N, K, 2, 3)
    # what belongs to nobody holds NaN scales
    xsc[:before] = 255
    xsc[int(off[-1]):] = 255
    g = B.grouped(rows, E, N, K, el, ld_y=N + pad)
    y = filled(rows, N, el, pad)
    B.moe_mxfp4_grouped_gemm(g, dev_off(off), xq, xsc, wq, wsc, y)
    xv = torch.from_numpy(R.values_of(xc, xs))
    wv = torch.from_numpy(R.values_of(wc, wsb)).view(E, N, K)
    ref, s = R.product(off, xv, wv, rows)
    live = torch.zeros(rows, dtype=torch.bool)
    live[before:int(off[-1])] = True
    check(y[live], ref[live], R.sum_bound(ref, s, K, el)[live], "y")
    assert (y[~live] == SENTINEL).all()


@pytest.mark.parametrize("rows,N,K", [(40, 48, 96), (700, 512, 512)])
def test_mxfp4_product_scales(B, rows, N, K):
    """Scales at both ends of their range, and NaN blocks in their rows only."""
    off = R.offsets_of([rows])
    xc, xs, xq, xsc = mx_operand(rows, K, 1)
    wc, wsb, wq, wsc = mx_operand(N, K, 2)
    xs, wsb = xs.copy(), wsb.copy()
    xs[0], xs[1], xs[2] = 1, 254, 0
    wsb[0], wsb[1] = 250, 2
    xs[7, 1] = 255
    wsb[9, 2] = 255
    xsc[:, : K // 32] = torch.from_numpy(xs).cuda()
    wsc[:, : K // 32] = torch.from_numpy(wsb).cuda()
    y = torch.empty(rows, N, device="cuda")
    g = B.grouped(rows, 1, N, K, "f32")
    B.moe_mxfp4_grouped_gemm(g, dev_off(off), xq, xsc, wq, wsc, y)
    nan = torch.isnan(y).cpu()
    want = torch.zeros(rows, N, dtype=torch.bool)
    want[7] = True
    want[:, 9] = True
    ref, s = R.product(off, torch.from_numpy(np.nan_to_num(R.values_of(xc, xs))),
                       torch.from_numpy(np.nan_to_num(R.values_of(wc, wsb))).view(1, N, K), rows)
    # where the sum of magnitudes leaves fp32 an output may be infinite
    fits = s < 2.0 ** 126
    assert torch.equal(nan & fits, want & fits)
    ok = ~want & fits
    # products below 2^-126 may be flushed: K of them
    bound = R.sum_bound(ref, s, K, torch.float32) + K * 2.0 ** -126
    check(y[ok], ref[ok], bound[ok], "y")


def test_streams_and_graph_replays(B):
    """A captured training pass on a stream of its own: replayed with other
    data in its buffers, every replay equals the eager calls."""
    E, N, K, rows, f = 4, 256, 128, 700, 128
    el = torch.bfloat16
    g1, g2 = B.grouped(rows, E, N, K, el), B.grouped(rows, E, K, f, el)
    w1, w2 = randn((E, N, K), el, 1, 0, K ** -0.5), randn((E, K, f), el, 2, 0, f ** -0.5)
    mk = lambda n, dt=el: torch.zeros(rows, n, dtype=dt, device="cuda")
    S = B.mxfp4_scale_stride(K)
    u8 = lambda *n: torch.zeros(*n, dtype=torch.uint8, device="cuda")
    w1q, w1s = u8(E, N, K // 2), u8(E, N, S)
    B.moe_mxfp4_quantize(w1.contiguous(), w1q, w1s)

    def bufs():
        return dict(x=mk(K), off=torch.zeros(E + 1, dtype=torch.int32, device="cuda"), gu=mk(N),
                    h=mk(f), y=mk(K), dh=mk(f), dgu=mk(N), dx=mk(K),
                    dw=torch.zeros(E, N, K, device="cuda"),
                    ws=torch.zeros(max(1, B.grouped_dw_workspace_size(g1)), dtype=torch.uint8,
                                   device="cuda"),
                    q=torch.zeros(rows, K // 2, dtype=torch.uint8, device="cuda"),
                    s=torch.zeros(rows, S, dtype=torch.uint8, device="cuda"), v=mk(K),
                    gu4=mk(N))

    def run(b):
        B.moe_grouped_gemm(g1, b["off"], b["x"], w1, b["gu"])
        B.moe_swiglu(b["gu"], b["h"], n_rows=b["off"][E:])
        B.moe_grouped_gemm(g2, b["off"], b["h"], w2, b["y"])
        B.moe_grouped_gemm_dx(g2, b["off"], b["y"], w2, b["dh"])
        B.moe_swiglu_backward(b["gu"], b["dh"], b["dgu"], n_rows=b["off"][E:])
        B.moe_grouped_gemm_dx(g1, b["off"], b["dgu"], w1, b["dx"])
        B.moe_grouped_gemm_dw(g1, b["off"], b["x"], b["dgu"], b["dw"], b["ws"])
        B.moe_mxfp4_quantize(b["y"], b["q"], b["s"], n_rows=b["off"][E:])
        B.moe_mxfp4_dequantize(b["q"], b["s"], b["v"], n_rows=b["off"][E:])
        B.moe_mxfp4_grouped_gemm(g1, b["off"], b["q"], b["s"], w1q, w1s, b["gu4"])

    def fill(b, seed, counts):
        b["x"].copy_(randn((rows, K), el, seed))
        b["off"].copy_(dev_off(R.offsets_of(counts)))

    cap, eager = bufs(), bufs()
    st = torch.cuda.Stream()
    fill(cap, 1, [100, 200, 300, 100])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        run(cap)  # every kernel loaded before the capture
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=st):
        run(cap)
    outs = ("gu", "h", "y", "dh", "dgu", "dx", "dw", "q", "s", "v", "gu4")
    for seed, counts in ((2, [700, 0, 0, 0]), (3, [0, 0, 1, 0]), (4, [0, 0, 0, 0]),
                         (5, [5, 600, 5, 90])):
        for b in (cap, eager):
            fill(b, seed, counts)
            for o in outs:
                b[o].zero_()
        torch.cuda.synchronize()
        graph.replay()
        run(eager)
        torch.cuda.synchronize()
        for o in outs:
            assert torch.equal(cap[o], eager[o]), (seed, o)


def layer(B, T, E, k, d, f, seed=0):
    """A planned layer: its config, workspace views and bf16 inputs."""
    cfg = B.config(T, E, k, d, f, max(1, T * k // E), "bf16")
    el = torch.bfloat16
    logits = torch.randn(T, E, generator=gen(seed), device="cuda")
    x = randn((T, d), el, seed + 1)
    wg, wu = (randn((E, f, d), el, seed + i, 0, d ** -0.5) for i in (2, 3))
    wd = randn((E, d, f), el, seed + 4, 0, f ** -0.5)
    ws = torch.empty(B.workspace_size(cfg), dtype=torch.uint8, device="cuda")
    return cfg, logits, x, wg.contiguous(), wu.contiguous(), wd.contiguous(), ws


@pytest.mark.parametrize("T,E,k,d,f", [(1, 8, 2, 64, 128), (333, 8, 2, 128, 192),
                                       (1024, 16, 4, 512, 256)])
def test_a_layer_of_ragged_products(B, T, E, k, d, f):
    """plan, product, SwiGLU, product into z, combine: the layer's forward
    without rounds, against moe_forward (same roundings, so z differs by the
    order of sums only) and in 4 bits against its own definition."""
    cfg, logits, x, wg, wu, wd, ws = layer(B, T, E, k, d, f)
    el = torch.bfloat16
    want = torch.empty(T, d, dtype=el, device="cuda")
    ws_f = torch.empty_like(ws)
    B.moe_forward(cfg, logits, x, wg, wu, wd, want, ws_f)

    B.moe_plan(cfg, logits, ws, read_rounds=False)
    v = B.workspace_views(cfg, ws)
    off, rows = v["offsets"], T * k
    xs = x[(v["perm"] // k).long()].contiguous()
    w1 = torch.cat([wg, wu], dim=1).contiguous()
    g1, g2 = B.grouped(rows, E, 2 * f, d, el), B.grouped(rows, E, d, f, el)
    gu = torch.empty(rows, 2 * f, dtype=el, device="cuda")
    h = torch.empty(rows, f, dtype=el, device="cuda")
    B.moe_grouped_gemm(g1, off, xs, w1, gu)
    B.moe_swiglu(gu, h, n_rows=off[E:])
    B.moe_grouped_gemm(g2, off, h, wd, v["z"])
    y = torch.empty(T, d, dtype=el, device="cuda")
    B.moe_combine(cfg, ws, y)
    # g and u are rounded to bf16 here and not there (2^-8 each way on g and
    # u, 2^-8 on h again), the sum of f terms and y's own rounding: the
    # layer's own tolerance
    scale = want.abs().max().item()
    assert (y.float() - want.float()).abs().max().item() <= 2e-2 * scale

    # the same in 4 bits
    S = B.mxfp4_scale_stride
    u8 = lambda *s: torch.empty(*s, dtype=torch.uint8, device="cuda")
    xq, xsc = u8(rows, d // 2), u8(rows, S(d))
    hq, hsc = u8(rows, f // 2), u8(rows, S(f))
    w1q, w1s = u8(E, 2 * f, d // 2), u8(E, 2 * f, S(d))
    wdq, wds = u8(E, d, f // 2), u8(E, d, S(f))
    B.moe_mxfp4_quantize(w1, w1q, w1s)
    B.moe_mxfp4_quantize(wd, wdq, wds)
    B.moe_mxfp4_quantize(x, xq, xsc, index=v["perm"], index_div=k)
    B.moe_mxfp4_grouped_gemm(g1, off, xq, xsc, w1q, w1s, gu)
    B.moe_swiglu(gu, h, n_rows=off[E:])
    B.moe_mxfp4_quantize(h, hq, hsc, n_rows=off[E:])
    B.moe_mxfp4_grouped_gemm(g2, off, hq, hsc, wdq, wds, v["z"])
    host = off.cpu().numpy()

    def vals(codes, scales, K):
        c = R.unpack(codes.reshape(-1, K // 2).cpu().numpy())
        return torch.from_numpy(
            R.values_of(c, scales.reshape(-1, S(K)).cpu().numpy()[:, : K // 32]))

    ref, s = R.product(host, vals(xq, xsc, d), vals(w1q, w1s, d).view(E, 2 * f, d), rows)
    check(gu, ref, R.sum_bound(ref, s, d, el), "gate and up in 4 bits")
    ref, s = R.product(host, vals(hq, hsc, f), vals(wdq, wds, f).view(E, d, f), rows)
    check(v["z"], ref, R.sum_bound(ref, s, f, el), "down in 4 bits")


def test_gradients_of_a_ragged_ffn_against_differences(B):
    """loss = sum c . (w2 swiglu(w1 x)) in fp32: the gradients of x, w1 and
    w2 from the library's calls against central differences of its forward."""
    E, d, f = 3, 24, 16
    off = R.offsets_of([7, 0, 12])
    rows, el = 19, torch.float32
    d_off = dev_off(off)
    g1, g2 = B.grouped(rows, E, 2 * f, d, el), B.grouped(rows, E, d, f, el)
    x = randn((rows, d), el, 1).contiguous()
    w1, w2 = randn((E, 2 * f, d), el, 2, 0, 0.3), randn((E, d, f), el, 3, 0, 0.3)
    c = randn((rows, d), el, 4).contiguous()
    gu, h, y = (torch.zeros(rows, n, device="cuda") for n in (2 * f, f, d))

    def loss(x, w1, w2):
        B.moe_grouped_gemm(g1, d_off, x, w1, gu)
        B.moe_swiglu(gu, h)
        B.moe_grouped_gemm(g2, d_off, h, w2, y)
        return (c.double() * y.double()).sum().item()

    loss(x, w1, w2)
    dh, dgu, dx = torch.zeros_like(h), torch.zeros_like(gu), torch.zeros_like(x)
    dw1, dw2 = torch.empty_like(w1), torch.empty_like(w2)
    B.moe_grouped_gemm_dx(g2, d_off, c, w2, dh)
    B.moe_grouped_gemm_dw(g2, d_off, h, c, dw2)
    B.moe_swiglu_backward(gu, dh, dgu)
    B.moe_grouped_gemm_dx(g1, d_off, dgu, w1, dx)
    B.moe_grouped_gemm_dw(g1, d_off, x, dgu, dw1)
    args, grads = [x, w1.contiguous(), w2.contiguous()], [dx, dw1, dw2]
    step = 2.0 ** -6
    for a in range(3):
        for pos in (0, args[a].numel() // 2 + 3, args[a].numel() - 1):
            v = []
            for sgn in (1, -1):
                p = [t.clone() for t in args]
                p[a].view(-1)[pos] += sgn * step
                v.append(loss(*p))
            num = (v[0] - v[1]) / (2 * step)
            # truncation: |third derivative| step^2 / 6, the third derivative
            # of a sum of a few SwiGLU terms with weights of order 0.3 well
            # below 50; rounding: fp32 errors of y (24 terms) over the step
            assert abs(num - grads[a].view(-1)[pos].item()) <= 50 / 6 * step ** 2 + 1e-3, (a, pos)


@pytest.mark.parametrize("K", [544, 608, 1056, 2080, 4128])
def test_mxfp4_product_reads_no_scales_past_its_arrays(B, K):
    """Scale rows that do not end at 16 bytes, arrays of exactly their size:
    the last row's scales count, what lies behind the array (NaN scales, in
    the same allocation) does not."""
    rows, N, S = 1500, 512, B.mxfp4_scale_stride(K)
    off = R.offsets_of([rows])
    xc, xs, xq, xsc = mx_operand(rows, K, 1, 3)
    wc, wsb, wq, wsc = mx_operand(N, K, 2, 3)

    def behind(t, fill):
        buf = torch.full((t.shape[0] + 64, t.shape[1]), fill, dtype=torch.uint8, device="cuda")
        buf[: t.shape[0]] = t
        return buf[: t.shape[0]]

    xsc, wsc, xq, wq = behind(xsc, 255), behind(wsc, 255), behind(xq, 0x77), behind(wq, 0x77)
    y = torch.empty(rows, N, device="cuda")
    B.moe_mxfp4_grouped_gemm(B.grouped(rows, 1, N, K, "f32"), dev_off(off), xq, xsc, wq, wsc, y)
    ref, s = R.product(off, torch.from_numpy(R.values_of(xc, xs)),
                       torch.from_numpy(R.values_of(wc, wsb)).view(1, N, K), rows)
    check(y, ref, R.sum_bound(ref, s, K, torch.float32), "y")


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("N,K,ld_y,ld_x", [(777, 333, 784, 336), (65, 513, 72, 520),
                                           (259, 261, 264, 264)])
def test_odd_widths_in_aligned_rows(B, dt, N, K, ld_y, ld_x):
    """Rows that start at 16 bytes and end at an odd element, in buffers that
    end with the last row's last element."""
    el, off = DT[dt], R.offsets_of([70, 0, 601, 30])
    rows = int(off[-1])

    def exact(rows, cols, ld, seed):
        n = (rows - 1) * ld + cols
        flat = torch.full((n,), float("nan"), dtype=el, device="cuda")
        t = flat.as_strided((rows, cols), (ld, 1))
        t.copy_(randn((rows, cols), el, seed))
        return t

    x, dy = exact(rows, K, ld_x, 1), exact(rows, N, ld_y, 2)
    w = randn((4, N, K), el, 3, 0, K ** -0.5)
    g = B.grouped(rows, 4, N, K, el, ld_x=ld_x, ld_y=ld_y)
    ws = torch.empty(max(16, B.grouped_dw_workspace_size(g)), dtype=torch.uint8, device="cuda")
    dw = torch.empty(4, N, K, device="cuda")
    B.moe_grouped_gemm_dw(g, dev_off(off), x, dy, dw, ws)
    ref, s = R.weight_grad(off, x, dy, 4)
    check(dw, ref, R.sum_bound(ref, s, 601, torch.float32), "dw")
    y, dx = exact(rows, N, ld_y, 4), exact(rows, K, ld_x, 5)
    B.moe_grouped_gemm(g, dev_off(off), x, w, y)
    ref, s = R.product(off, x, w, rows)
    check(y, ref, R.sum_bound(ref, s, K, el), "y")
    B.moe_grouped_gemm_dx(g, dev_off(off), dy, w, dx)
    ref, s = R.product(off, dy, w, rows, transpose=True)
    check(dx, ref, R.sum_bound(ref, s, N, el), "dx")


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("E,lo,hi", [(65, 0, 3), (200, 0, 40), (1024, 0, 9)])
def test_many_experts(B, dt, E, lo, hi):
    el, N, K = DT[dt], 192, 128
    c = np.random.default_rng(E).integers(lo, hi, E)
    c[[0, E // 2]] = 0
    c[E - 1] = 300
    off = R.offsets_of(c)
    rows = int(off[-1])
    x, dy = randn((rows, K), el, 1), randn((rows, N), el, 2)
    w = randn((E, N, K), el, 3, 0, K ** -0.5)
    g = B.grouped(rows, E, N, K, el)
    d_off = dev_off(off)
    y, dx = filled(rows, N, el, 0), filled(rows, K, el, 0)
    dw = torch.full((E, N, K), float("nan"), device="cuda")
    ws = torch.empty(max(16, B.grouped_dw_workspace_size(g)), dtype=torch.uint8, device="cuda")
    B.moe_grouped_gemm(g, d_off, x, w, y)
    B.moe_grouped_gemm_dx(g, d_off, dy, w, dx)
    B.moe_grouped_gemm_dw(g, d_off, x, dy, dw, ws)
    ref, s = R.product(off, x, w, rows)
    check(y, ref, R.sum_bound(ref, s, K, el), "y")
    ref, s = R.product(off, dy, w, rows, transpose=True)
    check(dx, ref, R.sum_bound(ref, s, N, el), "dx")
    ref, s = R.weight_grad(off, x, dy, E)
    check(dw, ref, R.sum_bound(ref, s, 300, torch.float32), "dw")
    xc, xs, xq, xsc = mx_operand(rows, K, 1, 3)
    wc, wsb, wq, wsc = mx_operand(E * N, K, 2, 3)
    B.moe_mxfp4_grouped_gemm(g, d_off, xq, xsc, wq, wsc, y)
    ref, s = R.product(off, torch.from_numpy(R.values_of(xc, xs)),
                       torch.from_numpy(R.values_of(wc, wsb)).view(E, N, K), rows)
    check(y, ref, R.sum_bound(ref, s, K, el), "MXFP4 y")


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("rows", [1, 15, 16, 17, 31, 32, 33, 50])
def test_one_expert_with_few_rows(B, dt, rows):
    """Every split of a few rows into blocks of 16, at widths that end inside
    a block and a K that ends inside a step and inside a scale group."""
    el = DT[dt]
    for N, K in [(40, 96), (264, 544), (1000, 2080)]:
        off = R.offsets_of([0, rows, 0])
        x, w = randn((rows, K), el, 1), randn((3, N, K), el, 2, 0, K ** -0.5)
        w[0] = w[2] = float("nan")
        g = B.grouped(rows, 3, N, K, el)
        y = filled(rows, N, el, 0)
        B.moe_grouped_gemm(g, dev_off(off), x, w, y)
        ref, s = R.product(off, x, torch.nan_to_num(w.double()), rows)
        check(y, ref, R.sum_bound(ref, s, K, el), (N, K))
        xc, xs, xq, xsc = mx_operand(rows, K, 1, 3)
        wc, wsb, wq, wsc = mx_operand(3 * N, K, 2, 3)
        B.moe_mxfp4_grouped_gemm(g, dev_off(off), xq, xsc, wq, wsc, y)
        ref, s = R.product(off, torch.from_numpy(R.values_of(xc, xs)),
                           torch.from_numpy(R.values_of(wc, wsb)).view(3, N, K), rows)
        check(y, ref, R.sum_bound(ref, s, K, el), ("MXFP4", N, K))


def test_overlapping_offsets_on_a_large_buffer(B):
    """Half of the experts claim all rows: far more tiles, chunks and slots than
    the shape has. No result is promised; the calls stay inside their outputs."""
    rows, E, N, K = 1 << 14, 1024, 64, 64
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[1::2] = rows
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(E, N, K, dtype=torch.bfloat16, device="cuda")
    guard = torch.full((rows + 512, N), SENTINEL, dtype=torch.bfloat16, device="cuda")
    y = guard[256:256 + rows]
    g = B.grouped(rows, E, N, K, "bf16")
    B.moe_grouped_gemm(g, off, x, w, y)
    B.moe_grouped_gemm_dx(g, off, x, w, y)
    dw = torch.full((E + 2, N, K), SENTINEL, device="cuda")
    ws = torch.empty(B.grouped_dw_workspace_size(g), dtype=torch.uint8, device="cuda")
    B.moe_grouped_gemm_dw(g, off, x, x, dw[1:1 + E], ws)
    torch.cuda.synchronize()
    assert (guard[:256] == SENTINEL).all() and (guard[256 + rows:] == SENTINEL).all()
    assert (dw[0] == SENTINEL).all() and (dw[-1] == SENTINEL).all()


def test_buffers_past_4_gib(B):
    """Rows whose byte offsets pass 32 bits: products, gradients, SwiGLU and
    quantisation, checked on rows at both ends."""
    rows, E, N, K = 300_000, 3, 256, 8192
    el = torch.bfloat16
    off = R.offsets_of([5, rows - 135, 130])
    x = torch.empty(rows, K, dtype=el, device="cuda")
    for a in range(0, rows, 50_000):
        x[a:a + 50_000] = randn((min(50_000, rows - a), K), el, a)
    w = randn((E, N, K), el, 2, 0, K ** -0.5)
    g, d_off = B.grouped(rows, E, N, K, el), dev_off(off)
    y = torch.empty(rows, N, dtype=el, device="cuda")
    B.moe_grouped_gemm(g, d_off, x, w, y)
    pick = [0, 4, 5, 131_071, 131_072, 262_143, 262_144, rows - 131, rows - 130, rows - 1]
    e_of = [0 if i < 5 else (1 if i < rows - 130 else 2) for i in pick]
    for i, e in zip(pick, e_of):
        ref, s = R.product(np.array([0, 1]), x[i:i + 1], w[e:e + 1], 1)
        check(y[i:i + 1], ref, R.sum_bound(ref, s, K, el), i)
    dx = torch.empty(rows, K, dtype=el, device="cuda")
    B.moe_grouped_gemm_dx(g, d_off, y, w, dx)
    for i, e in zip(pick, e_of):
        ref, s = R.product(np.array([0, 1]), y[i:i + 1], w[e:e + 1], 1, transpose=True)
        check(dx[i:i + 1], ref, R.sum_bound(ref, s, N, el), i)
    # the last expert's rows are the buffer's end
    ws = torch.empty(max(16, B.grouped_dw_workspace_size(g)), dtype=torch.uint8, device="cuda")
    dw = torch.empty(E, N, K, device="cuda")
    B.moe_grouped_gemm_dw(g, d_off, x, y, dw, ws)
    last = R.offsets_of([130])
    ref, s = R.weight_grad(last, x[-130:], y[-130:], 1)
    check(dw[2:], ref, R.sum_bound(ref, s, 130, torch.float32), "dw")
    # x as [g, u] of 4096 features each
    h = torch.empty(rows, K // 2, dtype=el, device="cuda")
    B.moe_swiglu(x, h)
    B.moe_swiglu_backward(x, h, dx)
    codes = torch.empty(rows, K // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(rows, K // 32, dtype=torch.uint8, device="cuda")
    B.moe_mxfp4_quantize(x, codes, scales)
    for i in pick:
        gg, u = x[i, : K // 2].double().cpu(), x[i, K // 2:].double().cpu()
        ref = gg * torch.sigmoid(gg) * u
        check(h[i], ref, ref.abs() * 2.0 ** -20 + R.rounding(ref * (1 + 2.0 ** -20), el), i)
        d = h[i].double().cpu()
        ref = d * gg * torch.sigmoid(gg)
        check(dx[i, K // 2:], ref, ref.abs() * 2.0 ** -20 + R.rounding(ref * (1 + 2.0 ** -20), el), i)
        c, s = R.codes_of(x[i:i + 1].double().cpu().numpy())
        assert np.array_equal(R.unpack(codes[i:i + 1].cpu().numpy()), c)
        assert np.array_equal(scales[i:i + 1].cpu().numpy(), s)
    B.moe_mxfp4_dequantize(codes, scales, dx)
    for i in pick:
        c, s = R.codes_of(x[i:i + 1].double().cpu().numpy())
        assert torch.equal(dx[i:i + 1].double().cpu(), torch.from_numpy(R.values_of(c, s)))


def test_calls_on_a_given_stream_wait_for_it(B):
    """stream= is where the work goes: it sees what was queued there before."""
    st = torch.cuda.Stream()
    x = torch.zeros(4096, 512, device="cuda")
    y = torch.zeros(4096, 256, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        torch.cuda._sleep(20_000_000)
        x.fill_(1.0)
    B.moe_swiglu(x, y, stream=st)
    st.synchronize()
    assert torch.allclose(y, torch.full_like(y, 1 / (1 + np.exp(-1.0))))
    B.moe_swiglu(x, y, stream=st.cuda_stream)
    st.synchronize()


def test_wrong_tensors_are_refused(B):
    el = torch.bfloat16
    g = B.grouped(8, 2, 16, 32, el)
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    x, w = torch.zeros(8, 32, dtype=el, device="cuda"), torch.zeros(2, 16, 32, dtype=el, device="cuda")
    y = torch.zeros(8, 16, dtype=el, device="cuda")
    bad = [(off.long(), x, w, y), (off[:2], x, w, y), (off.cpu(), x, w, y), (off, x.float(), w, y),
           (off, x[:7], w, y), (off, x[:, :16], w, y), (off, x.t(), w, y), (off, x, w[:1], y),
           (off, x, w.transpose(1, 2), y), (off, x, w, y[:, :8]), (off, x, w, x),
           (off, x[:1].expand(8, 32), w, y)]
    for a in bad:
        with pytest.raises(ValueError):
            B.moe_grouped_gemm(g, *a)
    with pytest.raises(ValueError):
        B.moe_swiglu(x, y[:, :8])
    with pytest.raises(ValueError):
        B.moe_swiglu(x, y.float())
    with pytest.raises(ValueError):
        B.moe_swiglu(x, y[:1].expand(8, 16))
    with pytest.raises(ValueError):
        B.moe_mxfp4_quantize(x.int(), off, off)
    u8 = torch.zeros(8, 16, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError):
        B.moe_mxfp4_quantize(x, u8, u8[:1])
    with pytest.raises(ValueError):
        B.moe_mxfp4_quantize(x, u8, u8, index=off.long())
    with pytest.raises(B.MoeError):
        B.moe_mxfp4_quantize(x, u8, u8, index=off, index_div=0)
    with pytest.raises(ValueError):
        B.moe_mxfp4_quantize(x[:, :16], u8, u8)


# around 16 bytes and a 128-byte stage of every type, where the ends of rows
# are loaded in another way than the rest
@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,K", [(2, 3), (3, 9), (9, 2), (8, 7), (33, 31), (65, 71), (66, 130),
                                 (129, 63), (135, 129), (5, 1031)])
def test_widths_around_vectors_and_stages(B, dt, N, K):
    el, c = DT[dt], [70, 0, 1, 131, 8]
    off = R.offsets_of(c, 1)
    rows, E, nan = int(off[-1]) + 2, len(c), float("nan")

    def framed(shape, seed, scale=1.0):  # NaN around every row and matrix
        n = int(np.prod(shape))
        flat = torch.full((n + 64,), nan, dtype=el, device="cuda")
        t = flat[33:33 + n].view(shape)
        t.copy_(randn((n // shape[-1], shape[-1]), el, seed, 0, scale).view(shape))
        return t

    def rows_of(width, seed):  # behind every row, and before it, NaN
        t = torch.full((rows, width + 11), nan, dtype=el, device="cuda")[:, 5:5 + width]
        t[1:int(off[-1])] = randn((int(off[-1]) - 1, width), el, seed)
        return t

    x, dy, w = rows_of(K, 1), rows_of(N, 2), framed((E, N, K), 3, K ** -0.5)
    g = B.grouped(rows, E, N, K, el, ld_x=K + 11, ld_y=N + 11)
    d_off, live = dev_off(off), slice(1, int(off[-1]))
    y, dx = filled(rows, N, el, 11), filled(rows, K, el, 11)
    dw = torch.empty(E, N, K, device="cuda")
    ws = torch.empty(B.grouped_dw_workspace_size(g), dtype=torch.uint8, device="cuda")
    B.moe_grouped_gemm(g, d_off, x, w, y)
    B.moe_grouped_gemm_dx(g, d_off, dy, w, dx)
    B.moe_grouped_gemm_dw(g, d_off, x, dy, dw, ws)
    ref, s = R.product(off, x, w, rows)
    check(y[live], ref[live], R.sum_bound(ref, s, K, el)[live], "y")
    ref, s = R.product(off, dy, w, rows, transpose=True)
    check(dx[live], ref[live], R.sum_bound(ref, s, N, el)[live], "dx")
    ref, s = R.weight_grad(off, x, dy, E)
    check(dw, ref, R.sum_bound(ref, s, max(c), torch.float32), "dw")
    for t in (y, dx):
        assert (t[0] == SENTINEL).all() and (t[int(off[-1]):] == SENTINEL).all()


# few outputs with long sums, where a tile's wavefronts share the sum
@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,K", [(40, 1031), (1031, 40), (129, 4095), (32, 128), (33, 127)])
def test_few_outputs_with_long_sums(B, dt, N, K):
    el, c = DT[dt], [3, 33, 0, 300]
    off = R.offsets_of(c, 2)
    rows, E = int(off[-1]) + 1, len(c)
    x, dy = randn((rows, K), el, 1, 3), randn((rows, N), el, 2, 3)
    w = randn((E, N, K), el, 3, 0, K ** -0.5)
    g = B.grouped(rows, E, N, K, el, ld_x=K + 3, ld_y=N + 3)
    d_off, live = dev_off(off), slice(2, int(off[-1]))
    y, dx = filled(rows, N, el, 3), filled(rows, K, el, 3)
    dw = randn((E, N, K), torch.float32, 4)
    was = dw.double().cpu()
    ws = torch.empty(B.grouped_dw_workspace_size(g), dtype=torch.uint8, device="cuda")
    B.moe_grouped_gemm(g, d_off, x, w, y)
    B.moe_grouped_gemm_dx(g, d_off, dy, w, dx)
    B.moe_grouped_gemm_dw(g, d_off, x, dy, dw, ws, accumulate=True)
    ref, s = R.product(off, x, w, rows)
    check(y[live], ref[live], R.sum_bound(ref, s, K, el)[live], "y")
    ref, s = R.product(off, dy, w, rows, transpose=True)
    check(dx[live], ref[live], R.sum_bound(ref, s, N, el)[live], "dx")
    ref, s = R.weight_grad(off, x, dy, E)
    check(dw, ref + was, R.sum_bound(ref + was, s + was.abs(), max(c) + 1, torch.float32), "dw")
    for t in (y, dx):
        assert (t[:2] == SENTINEL).all() and (t[int(off[-1]):] == SENTINEL).all()


# a 256 x 256 tile for every CU: the weight gradient's ring
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("E,hi,N,K,ld_y,ld_x", [
    (64, 40, 520, 264, 520, 264), (130, 5, 264, 72, 272, 72), (4, 700, 2048, 2048, 2048, 2056),
    (60, 33, 777, 333, 784, 336), (300, 3, 65, 130, 72, 136), (5, 1, 1921, 2050, 1928, 2056)])
def test_weight_gradient_with_many_tiles(B, dt, E, hi, N, K, ld_y, ld_x):
    el = DT[dt]
    c = np.random.default_rng(E + hi).integers(0, hi + 1, E).tolist()
    c[E // 2] = 0
    off = R.offsets_of(c, 3)
    rows, nan = int(off[-1]) + 5, float("nan")
    x, dy = randn((rows, K), el, 1, ld_x - K), randn((rows, N), el, 2, ld_y - N)
    for t in (x, dy):
        t[:3] = nan
        t[int(off[-1]):] = nan
    g = B.grouped(rows, E, N, K, el, ld_x=ld_x, ld_y=ld_y)
    ws = torch.full((B.grouped_dw_workspace_size(g),), 255, dtype=torch.uint8, device="cuda")
    dw = torch.full((E, N, K), nan, device="cuda")
    B.moe_grouped_gemm_dw(g, dev_off(off), x, dy, dw, ws)
    ref, s = R.weight_grad(off, x, dy, E)
    bound = R.sum_bound(ref, s, max(c), torch.float32)
    check(dw, ref, bound, "dw")
    dw0 = dw.clone()
    B.moe_grouped_gemm_dw(g, dev_off(off), x, dy, dw, ws, accumulate=True)
    check(dw, 2 * ref, R.sum_bound(2 * ref, 2 * s, 2 * max(c) + 1, torch.float32), "dw added")
    dw1 = torch.empty_like(dw0)
    B.moe_grouped_gemm_dw(g, dev_off(off), x, dy, dw1, ws)
    assert torch.equal(dw0, dw1)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_weight_gradient_with_many_chunks_and_tiles(B, dt):
    """Experts of very different sizes over many chunks of 128 rows, their
    sums joined from the slots; overlapping offsets store no slot twice."""
    el, N, K = DT[dt], 200, 256
    c = [20000, 0, 1, 129, 14000, 640]
    off = R.offsets_of(c)
    rows, E = int(off[-1]), len(c)
    x, dy = randn((rows, K), el, 1), randn((rows, N), el, 2)
    g = B.grouped(rows, E, N, K, el)
    size = B.grouped_dw_workspace_size(g)
    ws = torch.full((size + 4096,), 255, dtype=torch.uint8, device="cuda")
    dw = torch.empty(E, N, K, device="cuda")
    B.moe_grouped_gemm_dw(g, dev_off(off), x, dy, dw, ws)
    ref, s = R.weight_grad(off, x, dy, E)
    check(dw, ref, R.sum_bound(ref, s, max(c), torch.float32), "dw")
    raw = torch.tensor([0, rows, -5, rows + 9, 7, rows, 0], dtype=torch.int32, device="cuda")
    B.moe_grouped_gemm_dw(g, raw, x, dy, dw, ws)
    torch.cuda.synchronize()
    assert (ws[size:] == 255).all()


# outputs enough for the input gradient's ring: every one of its tiles
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("E,hi,N,K,pad", [
    (130, 5, 264, 1000, 0), (4, 700, 72, 1000, 8), (3, 2000, 40, 2056, 8), (2, 3000, 520, 520, 0),
    (60, 33, 1032, 333 * 8, 3), (8, 400, 8, 1032, 0)])
def test_input_gradient_with_many_tiles(B, dt, E, hi, N, K, pad):
    el, nan = DT[dt], float("nan")
    c = np.random.default_rng(E + hi).integers(hi // 2, hi + 1, E).tolist()
    c[E // 2] = 0
    off = R.offsets_of(c, 3)
    rows = int(off[-1]) + 5
    dy, w = randn((rows, N), el, 1, 8), randn((E, N, K), el, 2, 0, N ** -0.5)
    dy[:3] = nan
    dy[int(off[-1]):] = nan
    w[E // 2] = nan
    dx = filled(rows, K, el, pad)
    B.moe_grouped_gemm_dx(B.grouped(rows, E, N, K, el, ld_x=K + pad, ld_y=N + 8), dev_off(off), dy,
                          w, dx)
    live = slice(3, int(off[-1]))
    ref, s = R.product(off, dy, torch.nan_to_num(w.double()), rows, transpose=True)
    check(dx[live], ref[live], R.sum_bound(ref, s, N, el)[live], "dx")
    assert (dx[:3] == SENTINEL).all() and (dx[int(off[-1]):] == SENTINEL).all()
