"""Cases of the ragged expert operators: what is timed and compared.

The operators work on rows sorted by expert, expert e owning the rows
offsets[e] .. offsets[e + 1] - 1 (the order and the offsets of moe_plan):

  product    y[i] = W[e] x[i]
  gradients  its backward: dx[i] = W[e]^T dy[i], dW[e] = sum_i dy[i] x[i]^T
  swiglu     h = silu(g) u for rows [g, u], with its gradient
  quantize   rows to microscaled 4-bit floating point (blocks of 32 values,
             one power of two each), gathered into expert order, and back
  mxfp4      the product with both operands in that format

Where `own` is false the operators run in plain torch, in 32 bits, rounded
once; where it is true they are the library's calls.
"""
import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BLOCK = 32


def listed():
    return [
        # one token through the balanced layer's gate and up weights: the
        # call is a read of four experts' weights and a launch
        dict(name="product_one_token_bf16", kind="product", dtype="bf16", T=1, k=4, E=32,
             N=2048, K=2048, pad=0, empty=0, behind=0),
        # a serving batch of 64 tokens on the down weights of the layer with
        # 64 experts: every expert has a few rows, the weights are streamed
        dict(name="product_serving_batch_bf16", kind="product", dtype="bf16", T=64, k=8, E=64,
             N=4096, K=1536, pad=0, empty=0, behind=0),
        # odd sizes, strided rows, experts without rows and buffer rows
        # behind the last sequence
        dict(name="product_odd_f16", kind="product", dtype="f16", T=2501, k=2, E=7,
             N=777, K=1111, pad=3, empty=2, behind=37),
        # a long prompt through gate and up of the largest layer (d 7168,
        # two times 2048 features, 64 experts, 6 a token)
        dict(name="product_prompt_bf16", kind="product", dtype="bf16", T=16384, k=6, E=64,
             N=4096, K=7168, pad=0, empty=0, behind=0),
        # the backward of a training step's gate and up product, balanced
        # layer
        dict(name="gradients_step_bf16", kind="gradients", dtype="bf16", T=8192, k=4, E=32,
             N=2048, K=2048, pad=0, empty=0, behind=0),
        # the same at the smallest layer, in fp32, with an expert that no
        # token chose: latency and exactness
        dict(name="gradients_small_f32", kind="gradients", dtype="f32", T=512, k=2, E=8,
             N=256, K=64, pad=0, empty=1, behind=0),
        # the activation between the products of a long prompt's training
        # step, forward and backward
        dict(name="swiglu_step_bf16", kind="swiglu", dtype="bf16", T=16384, k=6, E=64,
             N=2048, K=0, pad=0, empty=0, behind=0),
        # an odd width and a few rows, one of them behind the last sequence
        dict(name="swiglu_few_rows_f32", kind="swiglu", dtype="f32", T=3, k=2, E=8,
             N=1001, K=0, pad=5, empty=0, behind=1),
        # a long prompt's tokens into expert order and 4 bits
        dict(name="quantize_prompt_bf16", kind="quantize", dtype="bf16", T=16384, k=6, E=64,
             N=0, K=7168, pad=0, empty=0, behind=0),
        # a few tokens, an odd number of blocks
        dict(name="quantize_few_tokens_f16", kind="quantize", dtype="f16", T=5, k=3, E=8,
             N=0, K=2080, pad=16, empty=0, behind=2),
        # the serving batch in 4 bits: a quarter of the weight bytes
        dict(name="mxfp4_serving_batch", kind="mxfp4", dtype="bf16", T=64, k=8, E=64,
             N=4096, K=1536, pad=0, empty=0, behind=0),
        # the long prompt in 4 bits
        dict(name="mxfp4_prompt", kind="mxfp4", dtype="bf16", T=16384, k=6, E=64,
             N=4096, K=7168, pad=0, empty=0, behind=0),
    ]


def _log_int(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    kind = rng.choice(["product", "product", "gradients", "swiglu", "quantize", "mxfp4"])
    E = _log_int(rng, 1, 64)
    k = rng.randint(1, min(E, 8))
    T = _log_int(rng, 1, 16384)
    case = dict(kind=kind, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), T=T, k=k, E=E,
                N=0, K=0, pad=rng.choice([0, 0, 8, rng.randint(1, 31)]),
                empty=rng.randint(0, max(0, min(E - k, 3))), behind=rng.choice([0, 0, rng.randint(1, 65)]))

    def width():
        n = _log_int(rng, 40, 4096)
        return n if rng.random() < 0.3 else (n + 63) // 64 * 64

    if kind in ("product", "gradients"):
        case["N"], case["K"] = width(), width()
    elif kind == "swiglu":
        case["N"] = width()
    elif kind == "quantize":
        case["K"] = (_log_int(rng, 32, 7168) + 31) // 32 * 32
    else:
        case["N"], case["K"] = width(), (_log_int(rng, 64, 7168) + 31) // 32 * 32
        case["dtype"] = rng.choice(["bf16", "bf16", "f16", "f32"])
    if case["dtype"] == "f32" and kind in ("product", "gradients"):
        case["T"] = min(T, 4096)  # the training parity runs in fp32 are short ones
    return case


def _rows(case):
    return case["T"] * case["k"] + case["behind"]


def work(case):
    r, N, K = case["T"] * case["k"], case["N"], case["K"]
    es = 4 if case["dtype"] == "f32" else 2
    active = min(case["E"] - case["empty"], r)
    kind = case["kind"]
    if kind == "product":
        return {"bytes": es * (r * (N + K) + active * N * K), "flops": 2 * r * N * K}
    if kind == "gradients":  # x, dy and the weights read, dx and dW (fp32) written
        return {"bytes": es * (r * (N + 2 * K) + active * N * K) + 4 * case["E"] * N * K,
                "flops": 4 * r * N * K}
    if kind == "swiglu":  # gu and dh read, h and dgu written
        return {"bytes": es * r * (2 * N + N + N + 2 * N), "flops": 20 * r * N}
    if kind == "quantize":  # tokens read once, codes, scales and values written
        rows = _rows(case)
        return {"bytes": es * case["T"] * K + rows * (K // 2 + K // BLOCK + es * K),
                "flops": 4 * rows * K}
    kb = K // 2 + K // BLOCK
    return {"bytes": r * (kb + es * N) + active * N * kb, "flops": 2 * r * N * K}


# ---------------------------------------------------------------- inputs


def _route(case, seed):
    """Expert-sorted assignments as moe_plan makes them: every token picks k
    distinct experts (a skewed choice; `empty` of the experts get none).
    Returns perm (assignment ids sorted by expert) and the offsets."""
    rng = np.random.default_rng([seed, 17])
    T, k, E = case["T"], case["k"], case["E"]
    bias = -0.8 * np.log(np.arange(1, E + 1))[rng.permutation(E)]
    if case["empty"]:
        bias[rng.permutation(E)[: case["empty"]]] = -np.inf
    score = bias + rng.gumbel(size=(T, E))
    idx = np.argsort(-score, axis=1, kind="stable")[:, :k].reshape(-1)
    perm = np.argsort(idx, kind="stable").astype(np.int32)
    off = np.zeros(E + 1, dtype=np.int32)
    off[1:] = np.cumsum(np.bincount(idx, minlength=E))
    return perm, off


def _normal(gen, shape, dtype, scale=1.0, pad=0):
    """N(0, scale^2) values; with pad the rows of a wider buffer."""
    t = torch.empty(*shape[:-1], shape[-1] + pad, dtype=dtype, device="cuda")
    flat = t.view(-1, t.shape[-1])
    step = max(1, (1 << 26) // t.shape[-1])
    for i in range(0, flat.shape[0], step):
        b = flat[i:i + step]
        b.copy_(torch.randn(b.shape, generator=gen, device="cuda") * scale)
    return t[..., : shape[-1]]


def _zeros(rows, cols, dtype, pad):
    return torch.zeros(rows, cols + pad, dtype=dtype, device="cuda")[:, :cols]


def _packed(gen, rows, K, scale):
    """Codes and scales of N(0, scale^2) rows: two codes a byte (the lower
    one first), the scale rows padded to whole groups of four."""
    q = torch.empty(rows, K // 2, dtype=torch.uint8, device="cuda")
    s = torch.zeros(rows, (K // BLOCK + 3) // 4 * 4, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 25) // K)
    for i in range(0, rows, step):
        n = min(step, rows - i)
        codes, e = _to_codes(torch.randn(n, K, generator=gen, device="cuda") * scale)
        q[i:i + n] = codes[:, 0::2] | (codes[:, 1::2] << 4)
        s[i:i + n, : K // BLOCK] = e
    return q, s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 7919 + 13)
    perm, off = _route(case, seed)
    dt, rows, pad = DTYPES[case["dtype"]], _rows(case), case["pad"]
    E, N, K = case["E"], case["N"], case["K"]
    st = dict(case=case, off=off.tolist(), offsets=torch.from_numpy(off).cuda())
    kind = case["kind"]
    if kind in ("product", "gradients"):
        st["x"] = _normal(gen, (rows, K), dt, pad=pad)
        st["w"] = _normal(gen, (E, N, K), dt, K ** -0.5)
        if kind == "product":
            st["y"] = _zeros(rows, N, dt, pad)
        else:
            st["dy"] = _normal(gen, (rows, N), dt, pad=pad)
            st["dx"] = _zeros(rows, K, dt, pad)
            st["dw"] = torch.zeros(E, N, K, device="cuda")
    elif kind == "swiglu":
        st["gu"] = _normal(gen, (rows, 2 * N), dt, pad=pad)
        st["dh"] = _normal(gen, (rows, N), dt, pad=pad)
        st["h"] = _zeros(rows, N, dt, pad)
        st["dgu"] = _zeros(rows, 2 * N, dt, pad)
    elif kind == "quantize":
        st["x"] = _normal(gen, (case["T"], K), dt, pad=pad)
        # buffer rows behind the last sequence hold no token
        idx = np.full(rows, -1, dtype=np.int32)
        idx[: perm.size] = perm
        st["index"] = torch.from_numpy(idx).cuda()
        st["codes"] = torch.zeros(rows, K // 2, dtype=torch.uint8, device="cuda")
        st["scales"] = torch.zeros(rows, (K // BLOCK + 3) // 4 * 4, dtype=torch.uint8,
                                   device="cuda")
        st["values"] = _zeros(rows, K, dt, pad)
    else:
        st["xq"], st["xs"] = _packed(gen, rows, K, 1.0)
        wq, ws = _packed(gen, E * N, K, K ** -0.5)
        st["wq"], st["ws"] = wq.view(E, N, -1), ws.view(E, N, -1)
        st["y"] = _zeros(rows, N, dt, pad)
    if own:
        _plan(st)
    return st


def _plan(st):
    """What a program of the library keeps: the call's shape and workspace."""
    from round_dropless_expert_amd import binding as B
    case = st["case"]
    pad = case["pad"]
    if case["kind"] in ("product", "gradients", "mxfp4"):
        st["g"] = B.grouped(_rows(case), case["E"], case["N"], case["K"], case["dtype"],
                            ld_x=0 if case["kind"] == "mxfp4" else case["K"] + pad,
                            ld_y=case["N"] + pad)
    if case["kind"] == "gradients":
        st["bws"] = torch.empty(B.grouped_dw_workspace_size(st["g"]), dtype=torch.uint8,
                                device="cuda")


# ---------------------------------------------------------------- plain forms


def _to_codes(x):
    """Codes (sign bit and three bits of magnitude) and scale bytes of fp32
    rows, block by block: the scale is the power of two that brings the
    block's largest magnitude into [4, 8), the codes are rounded to nearest,
    ties to even, and end at 6."""
    r, K = x.shape
    b = x.reshape(r, K // BLOCK, BLOCK)
    top = b.abs().amax(dim=-1)
    e = torch.where(top > 0, torch.frexp(top)[1] - 3, -127).clamp(-127, 127)
    a = torch.ldexp(b.abs(), -e.unsqueeze(-1))
    c = (a > 0.25).to(torch.uint8)
    for border, up in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True),
                       (5.0, False)):
        c += (a >= border) if up else (a > border)
    c |= (torch.signbit(b).to(torch.uint8) << 3)
    bad = ~torch.isfinite(top)
    s = torch.where(bad, 255, e + 127).to(torch.uint8)
    c = torch.where(bad.unsqueeze(-1), 0, c)
    return c.reshape(r, K), s


def _levels(dtype):
    half = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    return torch.tensor(half + [-v for v in half], dtype=dtype, device="cuda")


def _values(codes, s, dtype=torch.float32):
    """The values that codes [r][K] and scale bytes [r][K/32] stand for."""
    r, K = codes.shape
    v = _levels(dtype)[codes.to(torch.int32)].view(r, K // BLOCK, BLOCK)
    f = torch.ldexp(torch.ones((), dtype=dtype, device="cuda"), s.to(torch.int32) - 127)
    f = torch.where(s == 255, float("nan"), f)
    return (v * f.unsqueeze(-1)).view(r, K)


def _unpack(q):
    return torch.stack((q & 15, q >> 4), dim=-1).view(q.shape[0], -1)


def _silu_parts(gu, n):
    g, u = gu[:, :n], gu[:, n:]
    s = 1.0 / (1.0 + torch.exp(-g))
    return g, u, s


def _segments(st):
    off = st["off"]
    return [(e, off[e], off[e + 1]) for e in range(len(off) - 1) if off[e + 1] > off[e]]


def _run_plain(st):
    case = st["case"]
    kind, N, K = case["kind"], case["N"], case["K"]
    dt, end = DTYPES[case["dtype"]], st["off"][-1]
    if kind == "product":
        y = torch.zeros_like(st["y"])
        for e, a, b in _segments(st):
            y[a:b] = (st["x"][a:b].float() @ st["w"][e].float().t()).to(dt)
        return y
    if kind == "gradients":
        dx = torch.zeros_like(st["dx"])
        dw = torch.zeros_like(st["dw"])
        for e, a, b in _segments(st):
            dy = st["dy"][a:b].float()
            dx[a:b] = (dy @ st["w"][e].float()).to(dt)
            dw[e] = dy.t() @ st["x"][a:b].float()
        return dx, dw
    if kind == "swiglu":
        h, dgu = torch.zeros_like(st["h"]), torch.zeros_like(st["dgu"])
        g, u, s = _silu_parts(st["gu"][:end].float(), N)
        d = st["dh"][:end].float()
        h[:end] = (g * s * u).to(dt)
        dgu[:end, :N] = (d * u * s * (1.0 + g * (1.0 - s))).to(dt)
        dgu[:end, N:] = (d * g * s).to(dt)
        return h, dgu
    if kind == "quantize":
        t = torch.div(st["index"], case["k"], rounding_mode="floor")
        rows = st["x"].float()[t.clamp(min=0)]
        rows = torch.where((t >= 0).unsqueeze(-1), rows, 0.0)
        codes, s = _to_codes(rows)
        return _values(codes, s).to(dt), s
    y = torch.zeros_like(st["y"])
    nb = K // BLOCK
    for e, a, b in _segments(st):
        x = _values(_unpack(st["xq"][a:b]), st["xs"][a:b, :nb])
        w = _values(_unpack(st["wq"][e]), st["ws"][e][:, :nb])
        y[a:b] = (x @ w.t()).to(dt)
    return y


def _run_own(st):
    from round_dropless_expert_amd import binding as B
    case = st["case"]
    kind = case["kind"]
    if kind == "product":
        B.moe_grouped_gemm(st["g"], st["offsets"], st["x"], st["w"], st["y"])
        return st["y"]
    if kind == "gradients":
        B.moe_grouped_gemm_dx(st["g"], st["offsets"], st["dy"], st["w"], st["dx"])
        B.moe_grouped_gemm_dw(st["g"], st["offsets"], st["x"], st["dy"], st["dw"], st["bws"])
        return st["dx"], st["dw"]
    if kind == "swiglu":
        end = st["offsets"][-1:]
        B.moe_swiglu(st["gu"], st["h"], n_rows=end)
        B.moe_swiglu_backward(st["gu"], st["dh"], st["dgu"], n_rows=end)
        return st["h"], st["dgu"]
    if kind == "quantize":
        B.moe_mxfp4_quantize(st["x"], st["codes"], st["scales"], index=st["index"],
                             index_div=case["k"])
        B.moe_mxfp4_dequantize(st["codes"], st["scales"], st["values"])
        return st["values"], st["scales"][:, : case["K"] // BLOCK]
    B.moe_mxfp4_grouped_gemm(st["g"], st["offsets"], st["xq"], st["xs"], st["wq"], st["ws"],
                             st["y"])
    return st["y"]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------- 64 bits


def _exact_round(x):
    """The nearest 4-bit values of fp64 rows and their scale bytes, by
    distance to every level (ties to the even code)."""
    r, K = x.shape
    b = x.view(r, K // BLOCK, BLOCK)
    top = b.abs().amax(dim=-1, keepdim=True)
    two = torch.pow(2.0, torch.arange(-130, 129, dtype=torch.float64, device="cuda"))
    # floor(log2(top)) = the number of powers of two at most top
    e = (torch.searchsorted(two, top.reshape(-1), right=True).view_as(top) - 131).double()
    e = torch.where(top > 0, e - 2, -127.0).clamp(min=-127.0)
    a = b.abs() / torch.pow(2.0, e)
    level = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64,
                         device="cuda")
    best = torch.full_like(a, 1e300)
    val = torch.zeros_like(a)
    for c in (0, 2, 4, 6, 1, 3, 5, 7):  # even codes first: they keep a tie
        d = (a - level[c]).abs()
        near = d < best
        best = torch.where(near, d, best)
        val = torch.where(near, level[c], val)
    val = torch.copysign(val, b) * torch.pow(2.0, e)
    return val.view(r, K), (e + 127).squeeze(-1).to(torch.uint8)


def exact(case, seed):
    st = prepare(case, seed)
    kind, N, K, rows = case["kind"], case["N"], case["K"], _rows(case)
    f64 = dict(dtype=torch.float64, device="cuda")
    off = st["off"]
    if kind in ("product", "mxfp4"):
        y = torch.zeros(rows, N, **f64)
        nb = K // BLOCK
        for e in range(case["E"]):
            part = slice(off[e], off[e + 1])
            if kind == "product":
                y[part] = torch.mm(st["x"][part].double(), st["w"][e].double().t())
            else:
                xv = _values(_unpack(st["xq"][part]), st["xs"][part, :nb], torch.float64)
                wv = _values(_unpack(st["wq"][e]), st["ws"][e][:, :nb], torch.float64)
                y[part] = torch.mm(xv, wv.t())
        return y
    if kind == "gradients":
        dx, dw = torch.zeros(rows, K, **f64), torch.zeros(case["E"], N, K, **f64)
        for e in range(case["E"]):
            part = slice(off[e], off[e + 1])
            dy = st["dy"][part].double()
            dx[part] = torch.mm(dy, st["w"][e].double())
            dw[e] = torch.mm(dy.t().contiguous(), st["x"][part].double())
        return dx, dw
    if kind == "swiglu":
        n = off[-1]
        h, dgu = torch.zeros(rows, N, **f64), torch.zeros(rows, 2 * N, **f64)
        for a in range(0, n, 8192):
            c = slice(a, min(a + 8192, n))
            g = st["gu"][c, :N].double()
            u = st["gu"][c, N:].double()
            d = st["dh"][c].double()
            s = torch.sigmoid(g)
            h[c] = g * s * u
            dgu[c, :N] = d * u * (s + g * s * torch.sigmoid(-g))
            dgu[c, N:] = d * g * s
        return h, dgu
    vals = torch.zeros(rows, K, **f64)
    sc = torch.zeros(rows, K // BLOCK, dtype=torch.uint8, device="cuda")
    idx = st["index"].tolist()
    tok = torch.tensor([i // case["k"] if i >= 0 else -1 for i in idx], device="cuda")
    step = max(1, (1 << 26) // K)
    for a in range(0, rows, step):
        t = tok[a:a + step]
        x = st["x"][t.clamp(min=0)].double() * (t >= 0).double().unsqueeze(-1)
        vals[a:a + step], sc[a:a + step] = _exact_round(x)
    return vals, sc
