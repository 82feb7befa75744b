"""Plain fp64 forms of the operators around the experts' products, and the
error bounds that follow from their arithmetic."""
import numpy as np
import torch

NINF = float("-inf")


def scores(l, kind):
    """fp64 scores of logits [T, E]; -inf and NaN score 0."""
    l = np.asarray(l, dtype=np.float64)
    dead = ~(l > NINF)
    if kind == "sigmoid":
        with np.errstate(over="ignore"):
            s = 1.0 / (1.0 + np.exp(-np.where(dead, 0.0, l)))
        return np.where(dead, 0.0, s)
    top = np.max(np.where(dead, NINF, l), axis=1, keepdims=True)
    with np.errstate(invalid="ignore"):
        e = np.where(dead, 0.0, np.where(l == top, 1.0, np.exp(l - top)))
    return e / np.maximum(e.sum(axis=1, keepdims=True), 1e-300)


def choose(l, bias, k, kind, groups=1, top_groups=1, group_top=2):
    """idx [T, k]: the choice by fp64 values, ties to the lower index."""
    l = np.asarray(l, dtype=np.float64)
    T, E = l.shape
    dead = ~(l > NINF)
    c = scores(l, kind)
    if bias is not None:
        c = c + np.asarray(bias, dtype=np.float64)
    c = np.where(dead | np.isnan(c), NINF, c)
    closed = np.zeros((T, E), dtype=bool)
    g = E // groups
    if groups > 1 and top_groups < groups:
        part = -np.sort(-c.reshape(T, groups, g), axis=2)
        with np.errstate(invalid="ignore"):
            best = part[:, :, 0] + part[:, :, 1] if group_top == 2 and g > 1 else part[:, :, 0]
        best = np.where(np.isnan(best), NINF, best)
        order = np.argsort(-best, axis=1, kind="stable")
        keep = np.zeros((T, groups), dtype=bool)
        np.put_along_axis(keep, order[:, :top_groups], True, axis=1)
        closed = ~np.repeat(keep, g, axis=1)
    rank = c if bias is not None else np.where(dead, NINF, l)
    # closed experts behind the dead ones of open groups
    key = np.lexsort((np.broadcast_to(np.arange(E), (T, E)), -rank, closed), axis=1)
    return key[:, :k].astype(np.int32)


def weights(l, idx, kind, renormalize, scale):
    """fp64 weights and a bound of their fp32 errors: every elementary step (a
    subtraction in an exponent, an exponential, an addition, a division) is off by
    at most 2^-23 of its result, or of the exponent."""
    l = np.asarray(l, dtype=np.float64)
    E = l.shape[1]
    lj = np.take_along_axis(l, idx, axis=1)
    dead = ~(lj > NINF)
    s = np.take_along_axis(scores(l, kind), idx, axis=1)
    k = idx.shape[1]
    fin = np.where(np.isfinite(lj), lj, 0.0)
    span = np.abs(fin).max(axis=1, keepdims=True) * 2
    if renormalize:
        if kind == "softmax":
            ln = np.where(dead, NINF, lj)
        else:
            ln = np.where(dead, NINF, -np.logaddexp(0.0, -np.where(dead, 0.0, lj)))
        top = np.max(ln, axis=1, keepdims=True)
        with np.errstate(invalid="ignore"):
            e = np.where(dead, 0.0, np.where(ln == top, 1.0, np.exp(ln - top)))
        w = e / np.maximum(e.sum(axis=1, keepdims=True), 1e-300)
        steps = span + k + 10
    else:
        w = np.where(dead, 0.0, s)
        steps = span + (E if kind == "softmax" else 0) + 10
    return scale * w, np.abs(scale * w) * steps * 2.0 ** -23 + abs(scale) * 2.0 ** -126


def weights_of(l, idx, kind, renormalize, scale):
    """The weights as a differentiable fp64 torch function of finite logits."""
    if kind == "softmax":
        ln = torch.log_softmax(l, dim=1)
    else:
        ln = torch.nn.functional.logsigmoid(l)
    chosen = ln.gather(1, idx.long())
    return scale * (torch.softmax(chosen, dim=1) if renormalize else chosen.exp())


def sort(idx, E):
    """perm, pos, offsets; assignments of no expert last, as -1."""
    flat = np.asarray(idx).reshape(-1).astype(np.int64)
    b = np.where((flat >= 0) & (flat < E), flat, E)
    perm = np.argsort(b, kind="stable")
    pos = np.empty_like(perm)
    pos[perm] = np.arange(perm.size)
    off = np.zeros(E + 1, dtype=np.int64)
    off[1:] = np.cumsum(np.bincount(b, minlength=E + 1)[:E])
    perm[off[E]:] = -1
    return perm.astype(np.int32), np.where(b < E, pos, -1).astype(np.int32), off.astype(np.int32)


def int8_codes(x):
    """Codes and scales of rows. 127 x is exact in fp64 for x of 24 bits, and a
    quotient by the row's largest magnitude that is no tie lies 2^-33 or more
    from one, so the fp64 division's rounding changes no code."""
    x = np.asarray(x, dtype=np.float64)
    top = np.abs(x).max(axis=1, keepdims=True) if x.shape[1] else np.zeros((x.shape[0], 1))
    bad = ~np.isfinite(top)
    safe = np.where(bad | (top == 0), 1.0, top)
    with np.errstate(invalid="ignore"):
        q = np.rint(127.0 * x / safe)
    q = np.where(bad, 0, q).astype(np.int8)
    s = (top.astype(np.float32) / np.float32(127)).astype(np.float32)[:, 0]
    return q, np.where(bad[:, 0], np.float32(np.nan), s)


USUAL = (3.4445, -4.7750, 2.0315)


def orthogonalize(g, coefficients, scale=1.0):
    """The iteration in fp64 for one matrix, and a bound of the Frobenius norm
    of the error of one with fp16 values between its products.

    With u = 2^-11 (fp16's half step, relative; 2^-25 below its normal numbers),
    every value stored is off by u of it, every fp32 sum of t products by t 2^-23 of
    the product of the factors' norms. An error of X before the remaining steps
    is multiplied by their derivative: for an odd polynomial f of the singular
    values its norm is the largest divided difference (f(s) - f(t)) / (s - t), for
    s, t among the singular values and their negatives. First order; the
    triangle inequalities used leave far more room than the second needs.
    """
    x = g.double()
    tall = x.shape[0] > x.shape[1]
    x = x.t() if tall else x
    norm = torch.linalg.matrix_norm(x)
    x = x / (norm + 1e-20)
    m, n = x.shape
    up = 2.0 ** max(0, int(np.floor(np.log2(np.sqrt(m * n)))) - 4)
    u, tiny, acc = 2.0 ** -11, 2.0 ** -25, 2.0 ** -23
    fro = lambda a: float(torch.linalg.matrix_norm(a))
    two = lambda a: float(torch.linalg.matrix_norm(a, 2))
    xs, errs = [x], [u * fro(x) + tiny * np.sqrt(m * n) / up]
    for a, b, c in coefficients:
        p = x @ x.t()
        q = a * torch.eye(m, dtype=x.dtype) + b * p + c * (p @ p)
        nx = q @ x
        e_p = u * fro(p) + tiny * m + n * acc * fro(x) ** 2
        e_q = (u * fro(q) + tiny * m + abs(b) * e_p + abs(c) * (2 * two(p) * e_p
                                                               + m * acc * fro(p) ** 2))
        errs.append(u * fro(nx) + tiny * np.sqrt(m * n) / up + e_q * two(x)
                    + m * acc * fro(q) * fro(x))
        x = nx
        xs.append(x)
    total = 0.0
    for i, e in enumerate(errs[:-1]):
        s = torch.linalg.svdvals(xs[i])
        s = torch.cat([s, -s])
        f, d = s.clone(), torch.ones_like(s)
        for a, b, c in coefficients[i:]:
            d = d * (a + 3 * b * f ** 2 + 5 * c * f ** 4)
            f = a * f + b * f ** 3 + c * f ** 5
        ds = s[:, None] - s[None]
        near = ds.abs() < 1e-6
        dd = torch.where(near, d[:, None].abs(), ((f[:, None] - f[None]) / torch.where(near, 1.0, ds)).abs())
        total += e * float(dd.max())
    total += errs[-1]
    y = scale * (x.t() if tall else x)
    eps = 2.0 ** -8  # bf16's half step
    return y, abs(scale) * total * (1 + eps) + eps * fro(y)
