"""Cases of the operators around the experts' products: what is timed and
compared.

  route           scores, choice and weights of each token's experts, and its
                  assignments sorted by expert (the order of the products)
  route_backward  the gradient of the weights with respect to the logits
  collect         the experts' outputs summed back to tokens, with the
                  gradients with respect to the outputs and the weights
  int8_quantize   rows to 8-bit integers with a scale each, gathered into
                  expert order, and the values they stand for
  int8            the experts' product of such rows and weights
  orthogonalize   an update of every expert's matrix made orthogonal by
                  Newton-Schulz products

Where `own` is false the operators run in plain torch, in 32 bits (64 where a
border decides), rounded once; where it is true they are the library's calls.
"""
import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
# of the orthogonalising iteration, every step
COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def listed():
    return [
        # one token's choice when serving: 8 of 256 experts out of 4 of 8
        # groups, sigmoid scores and a bias; two launches of latency
        dict(name="route_one_token", kind="route", dtype="f32", T=1, E=256, k=8,
             score="sigmoid", groups=8, top_groups=4, renormalize=True, bias=True, pad=0),
        # a long prompt's through the same router
        dict(name="route_prompt", kind="route", dtype="f32", T=16384, E=256, k=8,
             score="sigmoid", groups=8, top_groups=4, renormalize=True, bias=True, pad=0),
        # a training step of the layer with 64 experts, 6 a token: softmax
        # over all experts, weights not renormalised, so every logit has a
        # gradient
        dict(name="route_backward_step", kind="route_backward", dtype="f32", T=16384, E=64, k=6,
             score="softmax", groups=1, top_groups=1, renormalize=False, bias=False, pad=0),
        # logits of 16 bits, an odd number of tokens, experts that are no
        # power of two, rows apart
        dict(name="route_backward_odd_bf16", kind="route_backward", dtype="bf16", T=2501, E=160,
             k=6, score="sigmoid", groups=1, top_groups=1, renormalize=True, bias=True, pad=8),
        # a training step of the widest layer: outputs of 6 experts a token
        # summed, and the gradients back to the experts
        dict(name="collect_step_bf16", kind="collect", dtype="bf16", T=16384, E=64, k=6, d=7168,
             pad=0),
        # a few tokens of an odd width
        dict(name="collect_few_tokens_f16", kind="collect", dtype="f16", T=5, E=8, k=3, d=1001,
             pad=3),
        # a long prompt's tokens into expert order and 8 bits
        dict(name="int8_quantize_prompt_bf16", kind="int8_quantize", dtype="bf16", T=16384, E=64,
             k=6, K=7168, pad=0, behind=0),
        # a few tokens, a width that is no multiple of anything
        dict(name="int8_quantize_few_tokens_f32", kind="int8_quantize", dtype="f32", T=5, E=8,
             k=3, K=1111, pad=5, behind=2),
        # a serving batch of 64 tokens on the down weights of the layer with
        # 64 experts: the weights are streamed, at half the bytes of 16 bits
        dict(name="int8_serving_batch", kind="int8", dtype="bf16", T=64, E=64, k=8, N=4096,
             K=1536, pad=0, behind=0),
        # a long prompt through gate and up of the largest layer
        dict(name="int8_prompt", kind="int8", dtype="bf16", T=16384, E=64, k=6, N=4096, K=7168,
             pad=0, behind=0),
        # the update of the balanced layer's gate and up weights from their
        # fp32 gradients
        dict(name="orthogonalize_layer_f32", kind="orthogonalize", dtype="f32", E=32, N=2048,
             K=2048, steps=5),
        # a few small matrices, taller than wide and odd, from bf16
        dict(name="orthogonalize_small_bf16", kind="orthogonalize", dtype="bf16", E=3, N=201,
             K=77, steps=5),
    ]


def _log_int(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    kind = rng.choice(["route", "route", "route_backward", "collect", "int8_quantize", "int8",
                       "int8", "orthogonalize"])
    dt = rng.choice(["bf16", "f16", "f32"])
    pad = rng.choice([0, 0, 8, rng.randint(1, 31)])
    if kind in ("route", "route_backward"):
        if rng.random() < 0.5:
            groups = rng.choice([2, 4, 8])
            E = groups * rng.randint(4, 32)
            top = rng.randint(1, groups)
        else:
            groups, top, E = 1, 1, _log_int(rng, 4, 384)
        k = rng.randint(1, min(8, top * (E // groups)))
        return dict(kind=kind, dtype=rng.choice(["f32", "f32", "bf16", "f16"]),
                    T=_log_int(rng, 1, 32768), E=E, k=k, score=rng.choice(["softmax", "sigmoid"]),
                    groups=groups, top_groups=top, renormalize=rng.random() < 0.6,
                    bias=rng.random() < 0.5, pad=pad)
    if kind == "orthogonalize":
        def side():
            n = _log_int(rng, 48, 2048)
            return n if rng.random() < 0.4 else (n + 63) // 64 * 64
        return dict(kind=kind, dtype=dt, E=_log_int(rng, 1, 32), N=side(), K=side(),
                    steps=rng.choice([4, 5, 5]))
    E = _log_int(rng, 1, 64)
    case = dict(kind=kind, dtype=dt, T=_log_int(rng, 1, 16384), E=E, k=rng.randint(1, min(E, 8)),
                pad=pad)
    n = _log_int(rng, 40, 4096)
    wide = n if rng.random() < 0.4 else (n + 63) // 64 * 64
    if kind == "collect":
        case["d"] = wide
    else:
        case["K"] = wide
        case["behind"] = rng.choice([0, 0, rng.randint(1, 65)])
    if kind == "int8":
        n = _log_int(rng, 40, 4096)
        case["N"] = n if rng.random() < 0.4 else (n + 63) // 64 * 64
    return case


def work(case):
    kind, es = case["kind"], 4 if case["dtype"] == "f32" else 2
    if kind == "orthogonalize":
        m, n = sorted((case["N"], case["K"]))
        # both factors of A = X X^T and of A A are the same: half of a
        # symmetric product's values suffice
        return {"bytes": case["E"] * m * n * (es + 2),
                "flops": case["E"] * case["steps"] * (m * m * n + m * m * m + 2 * m * m * n)}
    T, E, k = case["T"], case["E"], case["k"]
    if kind == "route":  # logits and bias read; experts, weights, order written
        return {"bytes": T * E * es + E * 8 + T * k * 16, "flops": 8 * T * E}
    if kind == "route_backward":
        full = case["score"] == "softmax" and not case["renormalize"]
        return {"bytes": T * E * es * (2 if full else 1) + T * k * (8 + (0 if full else es)),
                "flops": 8 * T * E}
    rows = T * k
    if kind == "collect":  # forward: z, y; backward: dy, z, dz
        d = case["d"]
        return {"bytes": es * d * (rows + T + T + rows + rows) + rows * 12, "flops": 5 * rows * d}
    if kind == "int8_quantize":  # tokens read, codes, scales and values written
        K = case["K"]
        rows += case["behind"]
        return {"bytes": es * T * K + rows * (K + 4 + es * K), "flops": 4 * rows * K}
    N, K = case["N"], case["K"]
    return {"bytes": rows * (K + 4 + es * N) + min(E, rows) * N * (K + 4), "flops": 2 * rows * N * K}


# ---------------------------------------------------------------- inputs


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


def _ints(n, dtype=torch.int32):
    return torch.zeros(n, dtype=dtype, device="cuda")


def _assign(gen, case):
    """idx [T][k], distinct experts of a token, some chosen more often."""
    T, E, k = case["T"], case["E"], case["k"]
    score = torch.randn(T, E, generator=gen, device="cuda")
    score += 0.4 * torch.randn(E, generator=gen, device="cuda")
    return score.topk(k, dim=1).indices.to(torch.int32)


def _codes(gen, rows, K, scale):
    """Codes and scales of N(0, scale^2) rows; code rows padded to whole 16
    bytes."""
    q = torch.zeros(rows, (K + 15) // 16 * 16, dtype=torch.int8, device="cuda")
    s = torch.empty(rows, device="cuda")
    step = max(1, (1 << 25) // K)
    for i in range(0, rows, step):
        x = torch.randn(min(step, rows - i), K, generator=gen, device="cuda") * scale
        q[i:i + step, :K], s[i:i + step] = _to_int8(x)
    return q, s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 7919 + 29)
    kind, dt = case["kind"], DTYPES[case["dtype"]]
    st = dict(case=case)
    if kind == "orthogonalize":
        E, N, K = case["E"], case["N"], case["K"]
        # a gradient: a few strong directions over many weak ones
        g = _normal(gen, (E, N, K), torch.float32, 1e-3)
        u = torch.randn(E, N, 4, generator=gen, device="cuda")
        v = torch.randn(E, 4, K, generator=gen, device="cuda") * 5e-4
        for r in range(4):
            g += u[:, :, r:r + 1] * v[:, r:r + 1, :]
        st["g"] = g.to(dt)
        st["y"] = torch.zeros(E, N, K, dtype=torch.bfloat16, device="cuda")
        return _plan(st) if own else st
    T, E, k = case["T"], case["E"], case["k"]
    rows = T * k
    if kind in ("route", "route_backward"):
        st["logits"] = _normal(gen, (T, E), dt, 1.5, case["pad"])
        # what a balancing rule leaves: experts often chosen are held back
        st["bias"] = torch.randn(E, generator=gen, device="cuda") * 0.05 if case["bias"] else None
        if kind == "route":
            st["idx"] = _ints((T, k))
            st["weight"] = torch.zeros(T, k, device="cuda")
            st["perm"], st["pos"], st["offsets"] = _ints(rows), _ints((T, k)), _ints(E + 1)
        else:
            st["idx"] = _assign(gen, case)
            st["dweight"] = torch.randn(T, k, generator=gen, device="cuda")
            st["dlogits"] = _zeros(T, E, dt, case["pad"])
        return _plan(st) if own else st
    idx = _assign(gen, case)
    perm, pos, offsets = _order(idx, E)
    if kind == "collect":
        d = case["d"]
        st["pos"] = pos
        st["weight"] = torch.softmax(torch.randn(T, k, generator=gen, device="cuda"), dim=1)
        st["z"], st["dy"] = (_normal(gen, (n, d), dt, 1.0, case["pad"]) for n in (rows, T))
        st["y"], st["dz"] = (_zeros(n, d, dt, case["pad"]) for n in (T, rows))
        st["dweight"] = torch.zeros(T, k, device="cuda")
        return st
    K = case["K"]
    if kind == "int8_quantize":
        # buffer rows behind the last sequence hold no token
        st["index"] = torch.cat([perm, _ints(case["behind"]) - 1])
        rows += case["behind"]
        st["x"] = _normal(gen, (T, K), dt, 1.0, case["pad"])
        st["codes"] = _ints((rows, (K + 15) // 16 * 16), torch.int8)
        st["scales"] = torch.zeros(rows, device="cuda")
        st["values"] = _zeros(rows, K, dt, case["pad"])
        return st
    N = case["N"]
    st["offsets"], st["off"] = offsets, offsets.tolist()
    st["xq"], st["xs"] = _codes(gen, rows + case["behind"], K, 1.0)
    wq, ws = _codes(gen, E * N, K, K ** -0.5)
    st["wq"], st["ws"] = wq.view(E, N, -1), ws.view(E, N)
    st["y"] = _zeros(rows + case["behind"], N, dt, case["pad"])
    return _plan(st) if own else st


def _plan(st):
    """What a program of the library keeps: the calls' shapes and workspaces."""
    from round_dropless_expert_amd import binding as B
    case = st["case"]
    kind = case["kind"]
    if kind == "orthogonalize":
        size = B.orthogonalize_workspace_size(case["E"], case["N"], case["K"])
        st["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    elif kind == "int8":
        st["g"] = B.grouped(st["y"].shape[0], case["E"], case["N"], case["K"], case["dtype"],
                            ld_y=case["N"] + case["pad"])
    else:
        st["router"] = B.router(case["T"], case["E"], case["k"], case["dtype"], case["score"],
                                groups=case["groups"], top_groups=case["top_groups"],
                                renormalize=case["renormalize"], scale=2.5,
                                ld=case["E"] + case["pad"])
        if kind == "route":
            size = B.sort_workspace_size(case["T"] * case["k"], case["E"])
            st["sort_ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return st


# ---------------------------------------------------------------- plain forms


def _scores(logits, kind):
    if kind == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-logits))
    e = torch.exp(logits - logits.amax(dim=1, keepdim=True))
    return e / e.sum(dim=1, keepdim=True)


def _choose(case, logits, bias):
    """idx [T][k] from fp64 scores: descending, ties to the lowest index."""
    T, E, groups = case["T"], case["E"], case["groups"]
    s = _scores(logits.double(), case["score"])
    c = s if bias is None else s + bias.double()
    if groups > 1:
        best = c.view(T, groups, E // groups).topk(2, dim=2).values.sum(dim=2)
        order = best.sort(dim=1, descending=True, stable=True).indices[:, : case["top_groups"]]
        keep = torch.zeros_like(best, dtype=torch.bool).scatter_(1, order, True)
        c = c.masked_fill(~keep.repeat_interleave(E // groups, dim=1), float("-inf"))
    idx = c.sort(dim=1, descending=True, stable=True).indices[:, : case["k"]]
    return idx, s.gather(1, idx)


def _order(idx, E):
    """Assignments sorted by expert (stable), where each went, and where each
    expert's begin."""
    flat = idx.reshape(-1)
    perm = flat.sort(stable=True).indices
    pos = torch.empty_like(perm)
    pos[perm] = torch.arange(perm.numel(), device="cuda")
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[1:] = torch.bincount(flat, minlength=E).cumsum(0)
    return perm.to(torch.int32), pos.to(torch.int32).view_as(idx), off


def _to_int8(x):
    """Codes and scales of fp32 rows: the largest magnitude becomes 127,
    rounded to nearest, ties to even (in 64 bits: a border decides)."""
    top = x.abs().amax(dim=1, keepdim=True)
    q = torch.round(x.double() * 127.0 / torch.where(top > 0, top, 1.0).double())
    return q.to(torch.int8), (top / 127.0).squeeze(1)


def _run_plain(st):
    case = st["case"]
    kind, dt = case["kind"], DTYPES[case["dtype"]]
    if kind == "route":
        idx, s = _choose(case, st["logits"], st["bias"])
        w = s / s.sum(dim=1, keepdim=True) if case["renormalize"] else s
        return (idx.to(torch.int32), (2.5 * w).float(), *_order(idx, case["E"]))
    if kind == "route_backward":
        idx, g = st["idx"].long(), 2.5 * st["dweight"]
        s = _scores(st["logits"].float(), case["score"])
        sj = s.gather(1, idx)
        if case["renormalize"]:
            w = sj / sj.sum(dim=1, keepdim=True)
            g = w * (g - (w * g).sum(dim=1, keepdim=True))
            if case["score"] == "sigmoid":
                g = g * (1.0 - sj)
            return torch.zeros_like(s).scatter_(1, idx, g).to(dt)
        if case["score"] == "sigmoid":
            return torch.zeros_like(s).scatter_(1, idx, g * sj * (1.0 - sj)).to(dt)
        full = torch.zeros_like(s).scatter_(1, idx, g)
        return (s * (full - (sj * g).sum(dim=1, keepdim=True))).to(dt)
    if kind == "collect":
        pos = st["pos"].long()
        z = st["z"].float()[pos]  # [T][k][d]
        dy = st["dy"].float().unsqueeze(1)
        w = st["weight"].unsqueeze(2)
        dz = torch.zeros_like(st["dz"])
        dz[pos] = (w * dy).to(dt)
        return (w * z).sum(dim=1).to(dt), dz, (z * dy).sum(dim=2)
    if kind == "int8_quantize":
        t = torch.div(st["index"], case["k"], rounding_mode="floor")
        q, s = _to_int8(st["x"].float())
        q, s = q[t.clamp(min=0)], s[t.clamp(min=0)]
        v = torch.where((t >= 0).unsqueeze(1), q.float() * s.unsqueeze(1), 0.0)
        return v.to(dt), torch.where(t >= 0, s, 0.0)
    if kind == "int8":
        # every expert's rows in a block of the most rows that one has
        E, N, K, off = case["E"], case["N"], case["K"], st["offsets"].long()
        count = off[1:] - off[:-1]
        most = int(np.diff(st["off"]).max())
        row = off[:-1, None] + torch.arange(most, device="cuda")
        live = torch.arange(most, device="cuda") < count[:, None]
        row = torch.where(live, row, 0)
        x = st["xq"][row][..., :K].float()
        y = torch.bmm(x, st["wq"][..., :K].float().transpose(1, 2).contiguous())
        y *= st["xs"][row].unsqueeze(2)
        y *= st["ws"].unsqueeze(1)
        out = torch.zeros_like(st["y"])
        out[row[live]] = y[live].to(dt)
        return out
    x = st["g"].float()
    tall = case["N"] > case["K"]
    if tall:
        x = x.transpose(1, 2).contiguous()
    norm = x.double().square().sum(dim=(1, 2), keepdim=True).sqrt()
    x = (x / (norm + 1e-20)).float()
    a, b, c = COEFFICIENTS
    for _ in range(case["steps"]):
        p = torch.bmm(x, x.transpose(1, 2).contiguous())
        x = a * x + torch.bmm(b * p + c * torch.bmm(p, p), x)
    return (x.transpose(1, 2) if tall else x).to(torch.bfloat16).contiguous()


def _run_own(st):
    from round_dropless_expert_amd import binding as B
    case = st["case"]
    kind = case["kind"]
    if kind == "route":
        B.moe_route(st["router"], st["logits"], st["idx"], st["weight"], bias=st["bias"])
        B.moe_sort(st["idx"], case["E"], st["perm"], st["pos"], st["offsets"], st["sort_ws"])
        return st["idx"], st["weight"], st["perm"], st["pos"], st["offsets"]
    if kind == "route_backward":
        B.moe_route_backward(st["router"], st["logits"], st["idx"], st["dweight"], st["dlogits"])
        return st["dlogits"]
    if kind == "collect":
        B.moe_collect(st["z"], st["pos"], st["y"], weight=st["weight"])
        B.moe_collect_backward(st["dy"], st["pos"], st["dz"], weight=st["weight"], z=st["z"],
                               dweight=st["dweight"])
        return st["y"], st["dz"], st["dweight"]
    if kind == "int8_quantize":
        B.moe_int8_quantize(st["x"], st["codes"], st["scales"], index=st["index"],
                            index_div=case["k"])
        B.moe_int8_dequantize(st["codes"], st["scales"], st["values"])
        return st["values"], st["scales"]
    if kind == "int8":
        B.moe_int8_grouped_gemm(st["g"], st["offsets"], st["xq"], st["xs"], st["wq"], st["ws"],
                                st["y"])
        return st["y"]
    B.moe_orthogonalize(st["g"], st["y"], st["ws"], steps=case["steps"])
    return st["y"]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------- 64 bits


def _exact_scores(case, logits, idx):
    """ln of the scores, and the chosen ones'."""
    l = logits.double()
    if case["score"] == "softmax":
        ln = l - torch.logsumexp(l, dim=1, keepdim=True)
    else:
        ln = -torch.logaddexp(torch.zeros_like(l), -l)
    return ln, ln.gather(1, idx.long())


def exact(case, seed):
    st = prepare(case, seed)
    kind = case["kind"]
    f64 = dict(dtype=torch.float64, device="cuda")
    if kind == "route":
        T, E, k, groups = case["T"], case["E"], case["k"], case["groups"]
        ln, _ = _exact_scores(case, st["logits"], torch.zeros(T, 1, device="cuda"))
        choice = ln.exp() + (0.0 if st["bias"] is None else st["bias"].double())
        if groups > 1:
            parts = choice.reshape(T, groups, -1).sort(dim=2).values
            total = parts[:, :, -1] + parts[:, :, -2]
            # a group's place: how many are before it
            ahead = (total[:, None, :] > total[:, :, None]).sum(dim=2)
            drop = (ahead >= case["top_groups"])[:, :, None].expand(T, groups, E // groups)
            choice = choice.masked_fill(drop.reshape(T, E), -1e9)
        best = choice.topk(k, dim=1).indices
        chosen = ln.gather(1, best)
        w = torch.softmax(chosen, dim=1) if case["renormalize"] else chosen.exp()
        return None, 2.5 * w, None, None, None
    if kind == "route_backward":
        l = st["logits"].double().clone().requires_grad_()
        _, chosen = _exact_scores(case, l, st["idx"])
        w = torch.softmax(chosen, dim=1) if case["renormalize"] else chosen.exp()
        return torch.autograd.grad((2.5 * w * st["dweight"].double()).sum(), l)[0]
    if kind == "collect":
        T, k, d = case["T"], case["k"], case["d"]
        y, dz = torch.zeros(T, d, **f64), torch.zeros(T * k, d, **f64)
        dw = torch.zeros(T, k, **f64)
        for j in range(k):
            for a in range(0, T, 4096):
                c = slice(a, a + 4096)
                at, wj = st["pos"][c, j].long(), st["weight"][c, j].double().unsqueeze(1)
                zj, dy = st["z"].index_select(0, at).double(), st["dy"][c].double()
                y[c].addcmul_(wj, zj)
                dz.index_copy_(0, at, wj * dy)
                dw[c, j] = (zj * dy).sum(dim=1)
        return y, dz, dw
    if kind == "int8_quantize":
        rows, K = st["values"].shape
        vals, sc = torch.zeros(rows, K, **f64), torch.zeros(rows, **f64)
        tok = [i // case["k"] if i >= 0 else -1 for i in st["index"].tolist()]
        tok = torch.tensor(tok, device="cuda")
        for a in range(0, rows, 8192):
            t = tok[a:a + 8192]
            x = st["x"][t.clamp(min=0)].double() * (t >= 0).unsqueeze(1)
            s = x.abs().max(dim=1).values / 127.0
            # nearest whole number of steps by distance, ties to even
            n = torch.where(s > 0, s, 1.0).unsqueeze(1)
            lo = torch.floor(x / n)
            up = (x / n - lo > 0.5) | ((x / n - lo == 0.5) & (lo % 2 != 0))
            vals[a:a + 8192], sc[a:a + 8192] = (lo + up) * s.unsqueeze(1), s
        return vals, sc
    if kind == "int8":
        y = torch.zeros(st["y"].shape, **f64)
        K = case["K"]
        for e in range(case["E"]):
            part = slice(st["off"][e], st["off"][e + 1])
            v = st["xq"][part, :K].double() * st["xs"][part].double().unsqueeze(1)
            w = st["wq"][e, :, :K].double() * st["ws"][e].double().unsqueeze(1)
            y[part] = torch.mm(v, w.t())
        return y
    y = torch.zeros(st["y"].shape, **f64)
    a, b, c = COEFFICIENTS
    for e in range(case["E"]):
        # the polynomial of the singular values, by the smaller Gram matrix's
        # powers on the left or the right
        x = st["g"][e].double()
        x = x / (torch.linalg.matrix_norm(x) + 1e-20)
        eye = torch.eye(min(x.shape), **f64)
        for _ in range(case["steps"]):
            if x.shape[0] <= x.shape[1]:
                q = torch.mm(x, x.t())
                x = torch.mm(a * eye + torch.mm(q, b * eye + c * q), x)
            else:
                q = torch.mm(x.t(), x)
                x = torch.mm(x, a * eye + torch.mm(q, b * eye + c * q))
        y[e] = x
    return y
