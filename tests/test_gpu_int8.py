"""8-bit integers on the GPU: quantisation, its inverse and the product."""
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


def quantize(B, x, **kw):
    rows = kw["index"].numel() if "index" in kw else x.shape[0]
    S = B.int8_stride(x.shape[1])
    q = torch.full((rows, S), 55, dtype=torch.int8, device="cuda")
    s = torch.full((rows + 1,), 55.0, device="cuda")
    B.moe_int8_quantize(x, q, s[:rows], **kw)
    assert s[rows] == 55.0
    return q, s[:rows]


def check_codes(q, s, x, what=""):
    K = x.shape[1]
    want, ws = U.int8_codes(x.double().cpu().numpy())
    got = q.cpu().numpy()
    assert np.array_equal(got[:, :K], want), what
    assert (got[:, K:] == 0).all(), what
    assert np.array_equal(s.cpu().numpy(), ws, equal_nan=True), what


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("rows,K,pad", [(1, 1, 0), (3, 15, 1), (5, 16, 0), (7, 33, 8), (64, 128, 0),
                                        (9, 1111, 5), (33, 2048, 0), (130, 4104, 8), (17, 7168, 0),
                                        (2, 16400, 0), (2, 40000, 3)])
def test_quantize(B, dt, rows, K, pad):
    x = randn((rows, K), DT[dt], rows + K, pad)
    if rows > 2:
        x[1] = 0
        x[2, 0] = float("inf")
    if rows > 4:
        x[3, K // 2] = float("nan")
        x[4] = x[4] * (1e-6 if dt == "f16" else 1e-38)  # small: quotients by a subnormal
    q, s = quantize(B, x)
    check_codes(q, s, x)
    y = torch.full((rows, K + pad), 77.0, dtype=DT[dt], device="cuda")
    B.moe_int8_dequantize(q, s, y[:, :K])
    v = q[:, :K].double().cpu() * s.double().cpu().unsqueeze(1)
    # one fp32 product, one rounding
    bound = R.sum_bound(v, v.abs(), 1, DT[dt])
    got = y[:, :K].double().cpu()
    bad = torch.isnan(s.cpu())
    assert torch.isnan(got[bad]).all()
    assert ((got - v).abs() <= bound)[~bad].all()
    assert (y[:, K:] == 77.0).all()


@pytest.mark.parametrize("dt", list(DT))
def test_quantize_borders(B, dt):
    """Quotients that are ties, or next to one."""
    el = DT[dt]
    a = torch.arange(1, 128, dtype=torch.float64)
    rows = []
    for top in (127.0, 254.0, 1.0, 0.375, 3.0, 96.0):
        x = (a - 0.5) * top / 127.0
        x = torch.cat([x, -x]).to(el)
        steps = [x]
        if el is torch.float32:
            inf = torch.tensor(float("inf"))
            steps += [torch.nextafter(x, inf), torch.nextafter(x, -inf)]
        for v in steps:
            rows.append(torch.cat([torch.tensor([top], dtype=el), v]))
    x = torch.stack(rows).cuda()
    q, s = quantize(B, x)
    check_codes(q, s, x)


@pytest.mark.parametrize("dt", list(DT))
def test_quantize_gathers(B, dt):
    src, K, div = 11, 200, 3
    x = randn((src, K), DT[dt], 4, 8)
    index = torch.tensor([0, 32, 33, 5, -1, 7, 31, -2 ** 31, 2 ** 31 - 1, 4], dtype=torch.int32)
    q, s = quantize(B, x, index=index.cuda(), index_div=div)
    t = [i // div if i >= 0 else -1 for i in index.tolist()]
    want = torch.stack([x[i] if 0 <= i < src else torch.zeros_like(x[0]) for i in t])
    check_codes(q, s, want)
    # rows from n_rows on are left alone
    for n in (0, 4, 10, 99):
        q2 = torch.full_like(q, 55)
        s2 = torch.full_like(s, 55.0)
        nr = torch.tensor([n], dtype=torch.int32, device="cuda")
        B.moe_int8_quantize(x, q2, s2, index=index.cuda(), index_div=div, n_rows=nr)
        m = min(n, 10)
        assert torch.equal(q2[:m], q[:m]) and torch.equal(s2[:m], s[:m])
        assert (q2[m:] == 55).all() and (s2[m:] == 55.0).all()
        y = torch.full((10, K), 77.0, dtype=DT[dt], device="cuda")
        B.moe_int8_dequantize(q, s, y, n_rows=nr)
        assert (y[m:] == 77.0).all() and torch.isfinite(y).all()


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


def cases():
    out = []
    for i, name in enumerate(COUNTS):
        for j, (N, K) in enumerate(SIZES):
            out.append((["bf16", "f16", "f32"][(i + j) % 3], name, N, K, [0, 8, 3][(i + 2 * j) % 3]))
    for dt in DT:  # the tiles of every shape
        out += [(dt, "long", 512, 640, 0), (dt, "hot", 768, 256, 64), (dt, "few", 2048, 1040, 0),
                (dt, "long", 2050, 100, 1)]
    return out


@pytest.mark.parametrize("dt,counts,N,K,pad", cases())
def test_product(B, dt, counts, N, K, pad):
    c, before, behind = COUNTS[counts]
    off = R.offsets_of(c, before)
    rows, E, el, S = int(off[-1]) + behind, len(c), DT[dt], B.int8_stride(K)
    xq = torch.randint(-127, 128, (rows, S), generator=gen(1), device="cuda", dtype=torch.int8)
    wq = torch.randint(-127, 128, (E, N, S), generator=gen(2), device="cuda", dtype=torch.int8)
    xq[:, K:] = 0
    wq[..., K:] = 0
    xs = torch.rand(rows, generator=gen(3), device="cuda") * 1e-2
    ws = torch.rand(E, N, generator=gen(4), device="cuda") * 1e-2
    nobody = torch.ones(rows, dtype=torch.bool)
    nobody[before:int(off[-1])] = False
    xs[nobody.cuda()] = float("nan")
    for e, n in enumerate(c):
        if n == 0:
            ws[e] = float("nan")
    g = B.grouped(rows, E, N, K, el, ld_y=N + pad)
    buf = torch.full((rows, N + pad), 77.0, dtype=el, device="cuda")
    y = buf[:, :N]
    d_off = torch.from_numpy(off).cuda()
    B.moe_int8_grouped_gemm(g, d_off, xq, xs, wq, ws, y)
    ref = torch.zeros(rows, N, dtype=torch.float64)
    for e, a, b in R.segments(off):
        if b > a:
            s = xq[a:b, :K].double().cpu() @ wq[e, :, :K].double().cpu().t()  # exact
            ref[a:b] = s * xs[a:b].double().cpu()[:, None] * ws[e].double().cpu()[None]
    # the sum to fp32 and two products: three roundings; then one to el
    b = 3 * 2.0 ** -24 * ref.abs() * (1 + 2.0 ** -20)
    bound = b * (1 + torch.finfo(el).eps) + R.rounding(ref, el)
    got = y.double().cpu()
    assert ((got - ref).abs() <= bound)[~nobody].all()
    assert (buf[nobody.cuda()] == 77.0).all() and (buf[:, N:] == 77.0).all()
    # the same bits again, a NaN where a scale is one
    again = torch.full_like(buf, 77.0)
    live = torch.nonzero(~nobody).flatten()
    if live.numel():
        xs[live[0]] = float("nan")
    B.moe_int8_grouped_gemm(g, d_off, xq, xs, wq, ws, again[:, :N])
    if live.numel():
        assert torch.isnan(again[live[0], :N]).all()
        assert torch.equal(again[live[1:]], buf[live[1:]])


def test_product_extremes(B):
    """The largest sums: all codes at an end, the widest row."""
    K, N, rows = 2 ** 17 - 1, 32, 40
    S = B.int8_stride(K)
    for a, b in ((127, 127), (-127, 127), (-128, -128)):
        xq = torch.full((rows, S), a, dtype=torch.int8, device="cuda")
        wq = torch.full((1, N, S), b, dtype=torch.int8, device="cuda")
        xq[:, K:] = 0
        wq[..., K:] = 0
        one = torch.ones(rows, device="cuda")
        y = torch.zeros(rows, N, device="cuda")
        g = B.grouped(rows, 1, N, K, "f32")
        off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
        B.moe_int8_grouped_gemm(g, off, xq, one, wq, torch.ones(1, N, device="cuda"), y)
        assert (y.double() == float(np.float32(a * b * K))).all()


def test_quantize_from_nothing(B):
    """An index into no rows: zeros and scales of 0."""
    q, s = quantize(B, torch.empty(0, 40, device="cuda"),
                    index=torch.zeros(5, dtype=torch.int32, device="cuda"))
    assert (q == 0).all() and (s == 0).all()


@pytest.mark.parametrize("dt", list(DT))
def test_quantize_the_widest_rows(B, dt):
    x = randn((2, 2 ** 20), DT[dt], 9)
    q, s = quantize(B, x)
    check_codes(q, s, x)


def test_product_of_many_experts(B):
    """1024 experts, most of them without rows."""
    E, N, K = 1024, 40, 80
    counts = [(7 * e) % 5 if e % 9 == 0 else 0 for e in range(E)]
    off = R.offsets_of(counts, 3)
    rows = int(off[-1]) + 4
    xq = torch.randint(-127, 128, (rows, K), generator=gen(1), device="cuda", dtype=torch.int8)
    wq = torch.randint(-127, 128, (E, N, K), generator=gen(2), device="cuda", dtype=torch.int8)
    one, ws = torch.ones(rows, device="cuda"), torch.ones(E, N, device="cuda")
    y = torch.full((rows, N), 77.0, device="cuda")
    B.moe_int8_grouped_gemm(B.grouped(rows, E, N, K, "f32"), torch.from_numpy(off).cuda(), xq, one,
                            wq, ws, y)
    ref = torch.full((rows, N), 77.0, dtype=torch.float64)
    for e, a, b in R.segments(off):
        ref[a:b] = xq[a:b].double().cpu() @ wq[e].double().cpu().t()
    assert torch.equal(y.double().cpu(), ref)  # whole numbers below 2^24
