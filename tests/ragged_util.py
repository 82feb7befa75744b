"""Plain fp64 forms of the ragged expert operators and the error bounds that
follow from their arithmetic."""
import numpy as np
import torch

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BLOCK = 32
LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def offsets_of(counts, first=0):
    off = np.zeros(len(counts) + 1, dtype=np.int32)
    off[0] = first
    off[1:] = first + np.cumsum(counts)
    return off


def segments(off):
    return [(e, int(off[e]), int(off[e + 1])) for e in range(len(off) - 1)]


def rounding(ref, dtype):
    """Half a step of `dtype` at ref: relative, and half a subnormal step."""
    fi = torch.finfo(dtype)
    return ref.abs() * (fi.eps / 2) + fi.smallest_normal * fi.eps / 2


def product(off, a, w, rows, transpose=False):
    """out[i] = a[i] w[e]^T (or a[i] w[e]) and sum |a||w|, fp64 on the CPU."""
    w = w.double().cpu()
    a = a.double().cpu()
    n = w.shape[2] if transpose else w.shape[1]
    y = torch.zeros(rows, n, dtype=torch.float64)
    s = torch.zeros_like(y)
    for e, b, t in segments(off):
        m = w[e] if transpose else w[e].t()
        y[b:t] = a[b:t] @ m
        s[b:t] = a[b:t].abs() @ m.abs()
    return y, s


def weight_grad(off, x, dy, E):
    x, dy = x.double().cpu(), dy.double().cpu()
    dw = torch.zeros(E, dy.shape[1], x.shape[1], dtype=torch.float64)
    s = torch.zeros_like(dw)
    for e, b, t in segments(off):
        dw[e] = dy[b:t].t() @ x[b:t]
        s[e] = dy[b:t].t().abs() @ x[b:t].abs()
    return dw, s


def sum_bound(ref, s, terms, dtype):
    """A sum of `terms` products in fp32, in any order: every product and
    every addition is off by at most 2^-23 of a partial sum of magnitudes
    (2^-24 where it rounds to nearest), so the sum by (terms + 1) 2^-23
    sum|p|; then one rounding to dtype, of the sum with its error."""
    acc = (terms + 1) * 2.0 ** -23 * s
    return acc * (1 + torch.finfo(dtype).eps / 2) + rounding(ref, dtype)


def codes_of(x):
    """(codes, scale bytes) of fp64 rows by distance to every level, ties to
    the even code; x of any float type that fp64 holds exactly."""
    x = np.asarray(x, dtype=np.float64)
    r, K = x.shape
    b = x.reshape(r, K // BLOCK, BLOCK)
    top = np.abs(b).max(axis=-1)
    bad = ~np.isfinite(top)
    safe = np.where(bad | (top == 0), 1.0, top)
    e = np.floor(np.log2(safe)).astype(int)
    e = np.where(np.exp2(e.astype(float)) > safe, e - 1, e)
    e = np.where(np.exp2(e.astype(float) + 1) <= safe, e + 1, e)
    e = np.where(top == 0, -127, np.maximum(e - 2, -127))
    with np.errstate(invalid="ignore"):
        a = np.abs(b) / np.exp2(e.astype(float))[..., None]
        d = np.abs(a[..., None] - LEVELS)
    best = d.min(axis=-1, keepdims=True)
    tie = d == best
    # of two equally near levels the one with the even code
    order = np.where(tie, np.array([0, 1, 0, 1, 0, 1, 0, 1]), 2)
    code = order.argmin(axis=-1)
    code = code | (np.signbit(b).astype(int) << 3)
    code = np.where(bad[..., None], 0, code)
    return (code.reshape(r, K).astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8))


def values_of(codes, scales):
    """fp64 values of unpacked codes [r, K] and scale bytes [r, K / 32]."""
    v = np.where(codes & 8, -1.0, 1.0) * LEVELS[codes & 7]
    f = np.where(scales == 255, np.nan, np.exp2(scales.astype(float) - 127))
    return (v.reshape(*scales.shape, BLOCK) * f[..., None]).reshape(codes.shape)


def unpack(q):
    q = np.asarray(q)
    return np.stack((q & 15, q >> 4), axis=-1).reshape(q.shape[0], -1)


def pack(codes):
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)
