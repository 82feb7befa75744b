"""The operators around the experts' products as a program uses them: a training
step and its gradients, 8-bit serving captured and replayed, several streams,
and buffers past 4 GiB."""
import numpy as np
import pytest
import torch

import routing_util as U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from round_dropless_expert_amd import binding
    binding.load()
    binding.check_runtime()
    return binding


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(shape, dtype, seed, scale=1.0):
    return (torch.randn(*shape, generator=gen(seed), device="cuda") * scale).to(dtype)


def u8(n):
    return torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")


class Step:
    """Buffers and calls of a layer's forward and backward in one element type."""

    def __init__(self, B, T, E, k, d, f, dtype, **router):
        self.B, self.dims = B, (T, E, k, d, f)
        rows, dev = T * k, "cuda"
        e = lambda *s, dt=dtype: torch.full(s, float("nan"), dtype=dt, device=dev)
        i = lambda *s: torch.full(s, -5, dtype=torch.int32, device=dev)
        self.r = B.router(T, E, k, "f32", scale=1.5, **router)
        self.g1 = B.grouped(rows, E, 2 * f, d, dtype)
        self.g2 = B.grouped(rows, E, d, f, dtype)
        self.idx, self.pos, self.perm, self.off = i(T, k), i(T, k), i(rows), i(E + 1)
        self.weight, self.dweight = e(T, k, dt=torch.float32), e(T, k, dt=torch.float32)
        self.xs, self.gu, self.h, self.z, self.y = (e(rows, d), e(rows, 2 * f), e(rows, f),
                                                    e(rows, d), e(T, d))
        self.dz, self.dh, self.dgu, self.dxs, self.dx = (e(rows, d), e(rows, f), e(rows, 2 * f),
                                                         e(rows, d), e(T, d))
        self.dw1, self.dw2 = e(E, 2 * f, d, dt=torch.float32), e(E, d, f, dt=torch.float32)
        self.dl = e(T, E, dt=torch.float32)
        self.sort_ws = u8(B.sort_workspace_size(rows, E))
        self.ws1, self.ws2 = (u8(B.grouped_dw_workspace_size(g)) for g in (self.g1, self.g2))
        self.u1 = torch.empty_like(self.dw1, dtype=torch.bfloat16)
        self.ows = u8(B.orthogonalize_workspace_size(E, 2 * f, d))

    def forward(self, logits, bias, x, w1, w2):
        B, E = self.B, self.dims[1]
        B.moe_route(self.r, logits, self.idx, self.weight, bias=bias)
        B.moe_sort(self.idx, E, self.perm, self.pos, self.off, self.sort_ws)
        B.moe_collect_backward(x, self.pos, self.xs)  # tokens into expert order
        B.moe_grouped_gemm(self.g1, self.off, self.xs, w1, self.gu)
        B.moe_swiglu(self.gu, self.h, n_rows=self.off[E:])
        B.moe_grouped_gemm(self.g2, self.off, self.h, w2, self.z)
        B.moe_collect(self.z, self.pos, self.y, weight=self.weight)

    def backward(self, logits, dy, w1, w2):
        B, E = self.B, self.dims[1]
        B.moe_collect_backward(dy, self.pos, self.dz, weight=self.weight, z=self.z,
                               dweight=self.dweight)
        B.moe_grouped_gemm_dw(self.g2, self.off, self.h, self.dz, self.dw2, self.ws2)
        B.moe_grouped_gemm_dx(self.g2, self.off, self.dz, w2, self.dh)
        B.moe_swiglu_backward(self.gu, self.dh, self.dgu, n_rows=self.off[E:])
        B.moe_grouped_gemm_dw(self.g1, self.off, self.xs, self.dgu, self.dw1, self.ws1)
        B.moe_grouped_gemm_dx(self.g1, self.off, self.dgu, w1, self.dxs)
        B.moe_collect(self.dxs, self.pos, self.dx)  # the gather's gradient
        B.moe_route_backward(self.r, logits, self.idx, self.dweight, self.dl)
        B.moe_orthogonalize(self.dw1, self.u1, self.ows)

    def results(self):
        return [self.idx, self.weight, self.y, self.dx, self.dl, self.dw1, self.dw2, self.u1]


def plain(logits, idx, x, w1, w2, score, renormalize, dy):
    """y and the gradients in fp64 for a given choice, and the same sums over
    magnitudes (|silu'| <= 1.1, |silu(g)| <= |g|, weights and their derivatives by
    their scores at most 1.5 each)."""
    l, x, w1, w2 = (t.double().cpu().requires_grad_() for t in (logits, x, w1, w2))
    dy, idx = dy.double().cpu(), idx.cpu().long()
    w = U.weights_of(l, idx, score, renormalize, 1.5)
    gu = torch.einsum("td,tjfd->tjf", x, w1[idx])
    g, u = gu.chunk(2, dim=2)
    h = torch.nn.functional.silu(g) * u
    z = torch.einsum("tjf,tjdf->tjd", h, w2[idx])
    y = (w.unsqueeze(2) * z).sum(dim=1)
    grads = torch.autograd.grad((y * dy).sum(), (l, x, w1, w2))
    with torch.no_grad():
        ax, a1, a2, ad = x.abs(), w1.abs()[idx], w2.abs()[idx], dy.abs()
        agu = torch.einsum("td,tjfd->tjf", ax, a1)
        ag, au = agu.chunk(2, dim=2)
        ah = ag * au
        az = torch.einsum("tjf,tjdf->tjd", ah, a2)
        aw = 1.5
        ay = aw * az.sum(dim=1)
        adz = aw * ad.unsqueeze(1).expand_as(az)
        adh = torch.einsum("tjd,tjdf->tjf", adz, a2)
        adgu = torch.cat([1.1 * adh * au, adh * ag], dim=2)
        adx = torch.einsum("tjf,tjfd->td", adgu, a1)
        adw = (az * ad.unsqueeze(1)).sum(dim=2)
        adl = 1.5 * adw.sum(dim=1, keepdim=True).expand_as(l)
        d1, d2 = torch.zeros_like(w1), torch.zeros_like(w2)
        t1 = adgu.unsqueeze(3) * ax[:, None, None, :]
        t2 = adz.unsqueeze(3) * ah.unsqueeze(2)
        for j in range(idx.shape[1]):
            d1.index_add_(0, idx[:, j], t1[:, j])
            d2.index_add_(0, idx[:, j], t2[:, j])
    return [y.detach(), grads[1], grads[0], grads[2], grads[3]], [ay, adx, adl, d1, d2]


@pytest.mark.parametrize("T,E,k,d,f,kw", [
    (96, 8, 2, 48, 40, dict(score="softmax")),
    (70, 16, 3, 64, 32, dict(score="sigmoid", groups=4, top_groups=2)),
    (33, 24, 4, 40, 24, dict(score="softmax", renormalize=False))])
def test_training_step(B, T, E, k, d, f, kw):
    """Forward, backward and update, fp32, against autograd in fp64."""
    logits, x = randn((T, E), torch.float32, 1), randn((T, d), torch.float32, 2)
    w1, w2 = randn((E, 2 * f, d), torch.float32, 3, d ** -0.5), randn((E, d, f), torch.float32, 4, f ** -0.5)
    dy, bias = randn((T, d), torch.float32, 5), randn((E,), torch.float32, 6, 0.05)
    s = Step(B, T, E, k, d, f, torch.float32, **kw)
    s.forward(logits, bias, x, w1, w2)
    s.backward(logits, dy, w1, w2)
    want = U.choose(logits.double().cpu().numpy(), bias.double().cpu().numpy(), k, kw["score"],
                    kw.get("groups", 1), kw.get("top_groups", 1))
    assert np.array_equal(s.idx.cpu().numpy(), want)
    ref, mag = plain(logits, s.idx, x, w1, w2, kw["score"], kw.get("renormalize", True), dy)
    # Every value is reached through at most two products of d and f terms each way,
    # sums over k, and the scores' E and their exponents (|l| below 5): as many
    # roundings, each 2^-23 of the magnitudes
    steps = 2 * (d + 2 * f) + T + 2 * k + E + 60
    for name, got, r, m in zip(("y", "dx", "dlogits", "dw1", "dw2"),
                               (s.y, s.dx, s.dl, s.dw1, s.dw2), ref, mag):
        err = (got.double().cpu() - r).abs()
        assert (err <= steps * 2.0 ** -23 * m + 1e-30).all(), name
    for e in range(E):
        r, bound = U.orthogonalize(s.dw1[e].double().cpu(), [U.USUAL] * 5)
        assert float(torch.linalg.matrix_norm(s.u1[e].double().cpu() - r)) <= bound


def serve(B, st):
    """A token batch through a layer in 8 bits."""
    B.moe_route(st["r"], st["logits"], st["idx"], st["weight"], bias=st["bias"])
    B.moe_sort(st["idx"], st["E"], st["perm"], st["pos"], st["off"], st["sort_ws"])
    end = st["off"][st["E"]:]
    B.moe_int8_quantize(st["x"], st["xq"], st["xsc"], index=st["perm"], index_div=st["k"])
    B.moe_int8_grouped_gemm(st["g1"], st["off"], st["xq"], st["xsc"], st["w1q"], st["w1s"], st["gu"])
    B.moe_swiglu(st["gu"], st["h"], n_rows=end)
    B.moe_int8_quantize(st["h"], st["hq"], st["hsc"], n_rows=end)
    B.moe_int8_grouped_gemm(st["g2"], st["off"], st["hq"], st["hsc"], st["w2q"], st["w2s"], st["z"])
    B.moe_collect(st["z"], st["pos"], st["y"], weight=st["weight"])


def serving_state(B, T, E, k, d, f, seed):
    rows = T * k
    st = dict(E=E, k=k, T=T, r=B.router(T, E, k, "f32", "sigmoid", groups=4, top_groups=2))
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")
    i32, i8, f32 = torch.int32, torch.int8, torch.float32
    st.update(logits=randn((T, E), f32, seed), bias=randn((E,), f32, seed + 1, 0.05),
              x=randn((T, d), torch.bfloat16, seed + 2), idx=z(T, k, dt=i32), pos=z(T, k, dt=i32),
              perm=z(rows, dt=i32), off=z(E + 1, dt=i32), weight=z(T, k, dt=f32), gu=z(rows, 2 * f),
              h=z(rows, f), z=z(rows, d), y=z(T, d), sort_ws=u8(B.sort_workspace_size(rows, E)),
              g1=B.grouped(rows, E, 2 * f, d, "bf16"), g2=B.grouped(rows, E, d, f, "bf16"))
    for n, r, c in (("x", rows, d), ("h", rows, f), ("w1", E * 2 * f, d), ("w2", E * d, f)):
        st[n + "q"] = z(r, B.int8_stride(c), dt=i8)
        st[n + ("s" if n[0] == "w" else "sc")] = z(r, dt=f32)
    for n, s in (("w1", (E * 2 * f, d)), ("w2", (E * d, f))):
        w = randn(s, torch.bfloat16, seed + 3, s[1] ** -0.5)
        st[n] = w
        B.moe_int8_quantize(w, st[n + "q"], st[n + "s"])
        st[n + "s"] = st[n + "s"].view(E, -1)
    return st


def test_serving_in_8_bits(B):
    """Against the same layer in fp64 on unquantised weights: each of the four
    quantisations is off by half a step, 1/254 of its row's largest value."""
    T, E, k, d, f = 50, 16, 3, 200, 136
    st = serving_state(B, T, E, k, d, f, 7)
    serve(B, st)
    idx = st["idx"].cpu().long()
    x, w1, w2 = st["x"].double().cpu(), st["w1"].double().cpu().view(E, 2 * f, d), st["w2"].double().cpu().view(E, d, f)
    w = U.weights(st["logits"].double().cpu().numpy(), idx.numpy(), "sigmoid", True, 1.0)[0]
    w = torch.from_numpy(w)
    q = lambda t: t.abs().amax(dim=-1, keepdim=True) / 254
    gu = torch.einsum("td,tjfd->tjf", x, w1[idx])
    ex, e1 = q(x).expand_as(x), q(w1).expand_as(w1)
    egu = torch.einsum("td,tjfd->tjf", ex, (w1.abs() + e1)[idx]) + torch.einsum("td,tjfd->tjf", x.abs(), e1[idx])
    egu = egu + gu.abs() * 2.0 ** -8
    g, u = gu.chunk(2, dim=2)
    eg, eu = egu.chunk(2, dim=2)
    h = torch.nn.functional.silu(g) * u
    eh = 1.1 * eg * (u.abs() + eu) + g.abs() * eu + h.abs() * 2.0 ** -8
    eh = eh + (h.abs() + eh).amax(dim=2, keepdim=True) / 254
    e2 = q(w2).expand_as(w2)
    z = torch.einsum("tjf,tjdf->tjd", h, w2[idx])
    ez = torch.einsum("tjf,tjdf->tjd", eh, (w2.abs() + e2)[idx]) + torch.einsum("tjf,tjdf->tjd", h.abs(), e2[idx])
    ez = ez + z.abs() * 2.0 ** -8
    y = (w.unsqueeze(2) * z).sum(dim=1)
    bound = ((w.unsqueeze(2) * ez).sum(dim=1) + y.abs() * 2.0 ** -8) * 1.02  # second orders
    assert ((st["y"].double().cpu() - y).abs() <= bound).all()


@pytest.mark.parametrize("T", [1, 64, 700])
def test_serving_captured(B, T):
    """Captured once, replayed on new inputs with eager work in between."""
    st = serving_state(B, T, 16, 4, 256, 128, 11)
    serve(B, st)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        serve(B, st)
    other = serving_state(B, T, 16, 4, 256, 128, 50)
    for n in range(4):
        st["logits"].copy_(randn(st["logits"].shape, torch.float32, 100 + n))
        st["x"].copy_(randn(st["x"].shape, torch.bfloat16, 200 + n))
        for t in ("y", "z", "weight"):
            st[t].fill_(float("nan"))
        graph.replay()
        serve(B, other)  # eager, its own buffers
        torch.cuda.synchronize()
        got = {t: st[t].clone() for t in ("idx", "weight", "perm", "pos", "off", "y")}
        serve(B, st)
        torch.cuda.synchronize()
        for t, v in got.items():
            assert torch.equal(v, st[t]), (n, t)


def test_training_captured(B):
    """A whole step captured and replayed while eager tensors of the same sizes
    live; every replay equals the eager step."""
    T, E, k, d, f = 200, 8, 2, 128, 64
    logits, x = randn((T, E), torch.float32, 1), randn((T, d), torch.bfloat16, 2)
    w1, w2 = randn((E, 2 * f, d), torch.bfloat16, 3, d ** -0.5), randn((E, d, f), torch.bfloat16, 4, f ** -0.5)
    dy, bias = randn((T, d), torch.bfloat16, 5), randn((E,), torch.float32, 6, 0.05)
    s, eager = (Step(B, T, E, k, d, f, torch.bfloat16, score="sigmoid") for _ in range(2))

    def run(step):
        step.forward(logits, bias, x, w1, w2)
        step.backward(logits, dy, w1, w2)

    run(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(s)
    for n in range(3):
        logits.copy_(randn((T, E), torch.float32, 60 + n))
        dy.copy_(randn((T, d), torch.bfloat16, 70 + n))
        graph.replay()
        run(eager)
        torch.cuda.synchronize()
        for a, b in zip(s.results(), eager.results()):
            assert torch.equal(a, b)


def test_streams(B):
    """Two streams, each with its buffers and workspaces, interleaved."""
    states = [serving_state(B, 300, 16, 4, 256, 128, 20 + i) for i in range(2)]
    gs = [torch.randn(3, 300, 200, generator=gen(i), device="cuda") for i in range(2)]
    want = []
    for st, g in zip(states, gs):
        serve(B, st)
        y = torch.empty(3, 300, 200, dtype=torch.bfloat16, device="cuda")
        B.moe_orthogonalize(g, y, u8(B.orthogonalize_workspace_size(3, 300, 200)))
        torch.cuda.synchronize()
        want.append((st["y"].clone(), y))
        st["y"].zero_()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty(3, 300, 200, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    wss = [u8(B.orthogonalize_workspace_size(3, 300, 200)) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for st, g, y, ws, s in zip(states, gs, outs, wss, streams):
            with torch.cuda.stream(s):
                serve(B, st)
            B.moe_orthogonalize(g, y, ws, stream=s)
    torch.cuda.synchronize()
    for st, y, (a, b) in zip(states, outs, want):
        assert torch.equal(st["y"], a) and torch.equal(y, b)


def test_buffers_past_4_gib(B):
    """The last rows of buffers whose offsets pass 32 bits."""
    rows, d = 700_001, 3200  # 4.48 GB of bf16, 2.24 GB of codes
    z = torch.zeros(rows, d, dtype=torch.bfloat16, device="cuda")
    last = randn((4, d), torch.bfloat16, 31)
    z[-4:] = last
    pos = torch.tensor([[rows - 1, rows - 4], [0, rows - 2]], dtype=torch.int32, device="cuda")
    y = torch.empty(2, d, dtype=torch.bfloat16, device="cuda")
    B.moe_collect(z, pos, y)
    assert torch.equal(y[0], (last[3].float() + last[0].float()).bfloat16())
    assert torch.equal(y[1], last[2])
    dz = torch.zeros_like(z)
    dw = torch.empty(2, 2, device="cuda")
    B.moe_collect_backward(y, pos, dz, z=z, dweight=dw)
    assert torch.equal(dz[rows - 1], y[0]) and torch.equal(dz[rows - 4], y[0])
    assert torch.equal(dz[rows - 2], y[1]) and dz[rows - 3].abs().max() == 0
    del dz
    codes = torch.empty(rows, d, dtype=torch.int8, device="cuda")
    scales = torch.empty(rows, device="cuda")
    B.moe_int8_quantize(z, codes, scales)
    want, ws = U.int8_codes(last.double().cpu().numpy())
    assert np.array_equal(codes[-4:].cpu().numpy(), want)
    assert np.array_equal(scales[-4:].cpu().numpy(), ws)
    B.moe_int8_dequantize(codes, scales, z)
    assert torch.equal(z[-4:], (codes[-4:].float() * scales[-4:, None]).bfloat16())
    del z
    # codes past 2^31: the product of the last rows
    wq = torch.randint(-9, 10, (1, 48, d), generator=gen(3), device="cuda", dtype=torch.int8)
    out = torch.zeros(rows, 48, dtype=torch.float32, device="cuda")
    off = torch.tensor([rows - 300, rows], dtype=torch.int32, device="cuda")
    scales[-300:-4] = 0
    B.moe_int8_grouped_gemm(B.grouped(rows, 1, 48, d, "f32"), off, codes, scales, wq,
                            torch.ones(1, 48, device="cuda"), out)
    ref = (codes[-4:].double() @ wq[0].double().t()) * scales[-4:, None].double()
    assert ((out[-4:].double() - ref).abs() <= 3 * 2.0 ** -24 * ref.abs()).all()
    assert out[:-4].abs().max() == 0


def test_logits_past_4_gib(B):
    T, E, k = 4_300_000, 256, 2  # 4.4 GB of fp32
    logits = torch.zeros(T, E, device="cuda")
    logits[-1, 200], logits[-1, 7], logits[-2, 3] = 3.0, 2.0, 1.0
    idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, k, device="cuda")
    r = B.router(T, E, k, "f32", "sigmoid", groups=8, top_groups=2)
    B.moe_route(r, logits, idx, w, bias=torch.zeros(E, device="cuda"))
    assert idx[-1].tolist() == [200, 7] and idx[-2].tolist() == [3, 0]
    assert (idx[:-2] == torch.tensor([0, 1], dtype=torch.int32, device="cuda")).all()
    perm, pos = (torch.empty(T * k, dtype=torch.int32, device="cuda") for _ in range(2))
    off = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    ws = u8(B.sort_workspace_size(T * k, E))
    B.moe_sort(idx, E, perm, pos, off, ws)
    assert perm[-1] == 2 * (T - 1) and off[E] == T * k and off[1] == T - 1
    dl = logits  # gradients over the logits' own size
    dl2 = torch.empty_like(logits)
    B.moe_route_backward(r, dl, idx, torch.ones(T, k, device="cuda"), dl2)
    assert dl2[-1].abs().max() <= 2.0 ** -20 and torch.isfinite(dl2[-1]).all()


def test_empty_calls(B):
    e = lambda *s, dt=torch.float32: torch.empty(*s, dtype=dt, device="cuda")
    i32 = torch.int32
    B.moe_route(B.router(0, 8, 2), e(0, 8), e(0, 2, dt=i32), e(0, 2))
    B.moe_route_backward(B.router(0, 8, 2), e(0, 8), e(0, 2, dt=i32), e(0, 2), e(0, 8))
    off = torch.full((9,), 5, dtype=i32, device="cuda")
    B.moe_sort(e(0, 2, dt=i32), 8, e(0, dt=i32), e(0, dt=i32), off)
    assert (off == 0).all()
    B.moe_collect(e(0, 16), e(0, 2, dt=i32), e(0, 16))
    y = e(3, 16).fill_(7)
    B.moe_collect(e(0, 16), torch.zeros(3, 2, dtype=i32, device="cuda"), y)  # no rows: zeros
    assert (y == 0).all()
    B.moe_collect_backward(e(0, 16), e(0, 2, dt=i32), e(4, 16))
    B.moe_int8_quantize(e(0, 40), e(0, 48, dt=torch.int8), e(0))
    B.moe_int8_dequantize(e(0, 48, dt=torch.int8), e(0), e(0, 40))
