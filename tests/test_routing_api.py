"""Argument checks of the operators around the experts' products: exact status
codes before any GPU call (no GPU needed), and the plain forms' own pins."""
import ctypes
import math
import os

import numpy as np
import pytest
import torch

import routing_util as U


@pytest.fixture(scope="module")
def B():
    from round_dropless_expert_amd import binding
    if not os.path.exists(binding.LIB_PATH):
        from round_dropless_expert_amd.csrc import build
        build.build()
    binding.load()
    return binding


P = 0x10000  # an aligned address that no call may touch


def err(B, fn, *args):
    with pytest.raises(B.MoeError) as e:
        B._check(getattr(B.load(), fn)(*args))
    return e.value.status


def router(B, **kw):
    a = dict(T=10, E=64, k=6, dtype=B.MOE_F32, score=0, groups=8, top_groups=4, group_top=2,
             renormalize=1, scale=1.0, ld=0)
    a.update(kw)
    return ctypes.byref(B.MoeRouter(*(a[n] for n, _ in B.MoeRouter._fields_)))


BAD = [
    (dict(T=-1), "INVALID"), (dict(E=0), "INVALID"), (dict(k=0), "INVALID"),
    (dict(k=65), "INVALID"), (dict(dtype=3), "INVALID"), (dict(score=2), "INVALID"),
    (dict(score=-1), "INVALID"), (dict(groups=7), "INVALID"), (dict(groups=-1), "INVALID"),
    (dict(top_groups=9), "INVALID"), (dict(top_groups=-1), "INVALID"),
    (dict(group_top=3), "INVALID"), (dict(group_top=-1), "INVALID"),
    (dict(renormalize=2), "INVALID"), (dict(scale=math.nan), "INVALID"),
    (dict(scale=math.inf), "INVALID"), (dict(ld=63), "INVALID"), (dict(ld=-1), "INVALID"),
    (dict(k=33), "INVALID"),  # four groups of eight hold 32
    (dict(E=1032), "UNSUPPORTED"), (dict(E=128, groups=1, top_groups=1, k=65), "UNSUPPORTED"),
    (dict(E=130, groups=65, top_groups=8), "UNSUPPORTED"), (dict(T=2 ** 31), "UNSUPPORTED"),
    (dict(T=2 ** 30), "UNSUPPORTED"), (dict(ld=2 ** 20 + 1), "UNSUPPORTED"),
]


@pytest.mark.parametrize("kw,status", BAD)
def test_routers_are_refused(B, kw, status):
    want = {"INVALID": B.MOE_ERR_INVALID_ARGUMENT, "UNSUPPORTED": B.MOE_ERR_UNSUPPORTED}[status]
    assert err(B, "moe_route", router(B, **kw), P, P, P, P, None) == want
    assert err(B, "moe_route_backward", router(B, **kw), P, P, P, P, None) == want


def test_pointers_are_checked(B):
    inv = B.MOE_ERR_INVALID_ARGUMENT
    assert err(B, "moe_route", None, P, P, P, P, None) == inv
    for fn, alone in (("moe_route", (0, 2, 3)), ("moe_route_backward", (0, 1, 2, 3))):
        for i in range(4):
            for bad in (None, P + 2):
                if bad is None and i not in alone:
                    continue
                a = [P] * 4
                a[i] = bad
                assert err(B, fn, router(B), *a, None) == inv
    L = B.load()
    assert L.moe_route(router(B, T=0), None, None, None, None, None) == B.MOE_OK
    assert L.moe_route_backward(router(B, T=0), None, None, None, None, None) == B.MOE_OK


def test_sort_is_checked(B):
    inv, uns, small = (B.MOE_ERR_INVALID_ARGUMENT, B.MOE_ERR_UNSUPPORTED,
                       B.MOE_ERR_WORKSPACE_TOO_SMALL)
    ok = [100, 8, P, P, P, P, None, 0, None]

    def bad(i, v, n=100):
        a = list(ok)
        a[0], a[i] = n, v
        return err(B, "moe_sort", *a)

    assert bad(0, -1, -1) == inv and bad(1, 0) == inv
    assert bad(0, 2 ** 31, 2 ** 31) == uns and bad(1, 1025) == uns
    for i in (2, 3, 4, 5):
        assert bad(i, None) == inv and bad(i, P + 1) == inv
    assert B.sort_workspace_size(0, 8) == 0 and B.sort_workspace_size(100, 1024) == 0
    need = B.sort_workspace_size(100000, 64)
    assert need > 0
    a = [100000, 64, P, P, P, P]
    assert err(B, "moe_sort", *a, None, need, None) == inv
    assert err(B, "moe_sort", *a, P + 4, need, None) == inv
    assert err(B, "moe_sort", *a, P, need - 1, None) == small
    # a small share of what it sorts, also at the largest sizes
    assert B.sort_workspace_size(2 ** 31 - 1, 1024) <= 2 ** 21
    n = ctypes.c_size_t(0)
    assert err(B, "moe_sort_workspace_size", 5, 0, ctypes.byref(n)) == inv
    assert err(B, "moe_sort_workspace_size", 5, 5, None) == inv


def test_collect_is_checked(B):
    inv, uns = B.MOE_ERR_INVALID_ARGUMENT, B.MOE_ERR_UNSUPPORTED
    bf = B.MOE_BF16
    #     dtype T k rows d z ld pos w y ld
    ok = [bf, 4, 2, 9, 8, P, 0, P, P, P, 0, None]
    for i, v, want in [(0, 7, inv), (1, -1, inv), (2, 0, inv), (3, -1, inv), (4, 0, inv),
                       (5, None, inv), (5, P + 1, inv), (6, 7, inv), (7, None, inv),
                       (7, P + 2, inv), (8, P + 2, inv), (9, None, inv), (9, P + 1, inv),
                       (10, 7, inv), (1, 2 ** 30, uns), (3, 2 ** 31, uns), (4, 2 ** 20 + 1, uns),
                       (6, 2 ** 20 + 1, uns)]:
        a = list(ok)
        a[i] = v
        assert err(B, "moe_collect", *a) == want, i
    #     dtype T k rows d dy ld z ld pos w dz ld dw
    ok = [bf, 4, 2, 9, 8, P, 0, P, 0, P, P, P, 0, P, None]
    for i, v, want in [(0, -1, inv), (5, None, inv), (6, 7, inv), (7, None, inv), (8, 7, inv),
                       (9, None, inv), (10, P + 2, inv), (11, P + 1, inv), (12, 7, inv),
                       (13, P + 2, inv), (2, 2 ** 30, uns), (12, 2 ** 21, uns)]:
        a = list(ok)
        a[i] = v
        assert err(B, "moe_collect_backward", *a) == want, i
    a = list(ok)
    a[11] = a[13] = None
    assert err(B, "moe_collect_backward", *a) == inv
    L = B.load()
    assert L.moe_collect(bf, 0, 2, 0, 8, None, 0, None, None, None, 0, None) == B.MOE_OK
    assert L.moe_collect_backward(bf, 0, 2, 9, 8, None, 0, None, 0, None, None, P, 0, None,
                                  None) == B.MOE_OK


def test_int8_is_checked(B):
    inv, uns = B.MOE_ERR_INVALID_ARGUMENT, B.MOE_ERR_UNSUPPORTED
    bf = B.MOE_BF16
    q = lambda *a: err(B, "moe_int8_quantize", *a)
    assert q(9, 4, 33, P, 0, 4, None, 1, None, P, P, None) == inv
    assert q(bf, -1, 33, P, 0, 4, None, 1, None, P, P, None) == inv
    assert q(bf, 4, 0, P, 0, 4, None, 1, None, P, P, None) == inv
    assert q(bf, 4, 33, P, 32, 4, None, 1, None, P, P, None) == inv
    assert q(bf, 4, 33, P, 0, 4, P, 0, None, P, P, None) == inv
    assert q(bf, 4, 33, P, 0, -1, P, 1, None, P, P, None) == inv
    assert q(bf, 4, 33, P, 0, 4, P + 1, 1, None, P, P, None) == inv
    assert q(bf, 4, 33, None, 0, 4, None, 1, None, P, P, None) == inv
    assert q(bf, 4, 33, P, 0, 4, None, 1, P + 2, P, P, None) == inv
    assert q(bf, 4, 33, P, 0, 4, None, 1, None, P + 8, P, None) == inv
    assert q(bf, 4, 33, P, 0, 4, None, 1, None, P, P + 2, None) == inv
    assert q(bf, 4, 2 ** 20 + 1, P, 0, 4, None, 1, None, P, P, None) == uns
    d = lambda *a: err(B, "moe_int8_dequantize", *a)
    assert d(bf, 4, 33, P + 8, P, P, 0, None, None) == inv
    assert d(bf, 4, 33, P, None, P, 0, None, None) == inv
    assert d(bf, 4, 33, P, P, P + 1, 0, None, None) == inv
    assert d(bf, 4, 33, P, P, P, 32, None, None) == inv
    g = lambda **kw: ctypes.byref(B.MoeGrouped(*({**dict(rows=10, E=4, N=32, K=64, dtype=bf,
                                                         ld_x=0, ld_y=0), **kw}).values()))
    for i in range(6):
        for bad in (None, P + 1):
            a = [P] * 6
            a[i] = bad
            assert err(B, "moe_int8_grouped_gemm", g(), *a, None) == inv
    assert err(B, "moe_int8_grouped_gemm", g(ld_x=80), *[P] * 6, None) == inv
    assert err(B, "moe_int8_grouped_gemm", g(K=2 ** 17), *[P] * 6, None) == uns
    assert err(B, "moe_int8_grouped_gemm", g(E=1025), *[P] * 6, None) == uns
    assert B.load().moe_int8_grouped_gemm(g(rows=0), *[None] * 7) == B.MOE_OK
    for k in (1, 15, 16, 17, 7168, 2 ** 20):
        assert B.load().moe_int8_stride(k) == B.int8_stride(k) == -(-k // 16) * 16
    for k in (0, -5, 2 ** 20 + 1):
        assert B.load().moe_int8_stride(k) == -1
        with pytest.raises(ValueError):
            B.int8_stride(k)


def test_orthogonalize_is_checked(B):
    inv, uns, small = (B.MOE_ERR_INVALID_ARGUMENT, B.MOE_ERR_UNSUPPORTED,
                       B.MOE_ERR_WORKSPACE_TOO_SMALL)
    need = B.orthogonalize_workspace_size(3, 40, 70)
    #     dtype E N K g y steps c scale ws bytes
    ok = [B.MOE_F32, 3, 40, 70, P, P, 5, None, 1.0, P, need, None]
    for i, v, want in [(0, 5, inv), (1, 0, inv), (2, 0, inv), (3, -1, inv), (4, None, inv),
                       (4, P + 2, inv), (5, None, inv), (5, P + 1, inv), (6, 0, inv), (6, 33, uns),
                       (8, math.inf, inv), (9, None, inv), (9, P + 8, inv), (10, need - 1, small),
                       (1, 1025, uns), (2, 16385, uns), (3, 16385, uns)]:
        a = list(ok)
        a[i] = v
        assert err(B, "moe_orthogonalize", *a) == want, i
    a = list(ok)
    a[7] = (ctypes.c_float * 15)(*([1.0] * 14 + [math.nan]))
    assert err(B, "moe_orthogonalize", *a) == inv
    assert B.orthogonalize_workspace_size(3, 70, 40) == need  # of the shape's sides alone
    n = ctypes.c_size_t(0)
    assert err(B, "moe_orthogonalize_workspace_size", 0, 4, 4, ctypes.byref(n)) == inv
    assert err(B, "moe_orthogonalize_workspace_size", 4, 4, 4, None) == inv


def test_host_tensors_and_wrong_shapes_are_refused(B, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    f, i = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    r = B.router(4, 8, 2)
    for call in (lambda: B.moe_route(r, f, i, f), lambda: B.moe_route_backward(r, f, i, f, f),
                 lambda: B.moe_sort(i, 8, i, i, i), lambda: B.moe_collect(f, i, f),
                 lambda: B.moe_collect_backward(f, i, f),
                 lambda: B.moe_int8_quantize(f, f, f), lambda: B.moe_int8_dequantize(f, f, f),
                 lambda: B.moe_orthogonalize(f, f, f)):
        with pytest.raises(ValueError):
            call()
    monkeypatch.setattr(B, "_on_device", lambda t, name, dev: None)
    monkeypatch.setattr(B, "_arg", lambda t, *a: t.data_ptr())
    with pytest.raises(ValueError, match="y"):
        B.moe_orthogonalize(f, f, None)  # an update is bfloat16
    with pytest.raises(ValueError, match="triples"):
        B.moe_orthogonalize(f, f.bfloat16(), None, steps=2, coefficients=[(1, 2, 3)])
    with pytest.raises(ValueError, match="dweight needs z"):
        B.moe_collect_backward(f, i, None, dweight=f)
    with pytest.raises(ValueError, match="neither"):
        B.moe_collect_backward(f, i)
    with pytest.raises(ValueError, match="32 bits"):
        B.router(4, 2 ** 32 + 8, 2)


def test_plain_choice_is_the_definition():
    l = np.array([[1.0, 3.0, 3.0, -np.inf, np.nan, 2.0]])
    assert U.choose(l, None, 6, "softmax")[0].tolist() == [1, 2, 5, 0, 3, 4]
    b = np.array([0.9, 0, 0, 5, 5, 0])
    assert U.choose(l, b, 3, "sigmoid")[0].tolist() == [0, 1, 2]
    # groups of two: sums of sigmoids .73 + .95, .95, .88
    assert U.choose(l, None, 2, "sigmoid", 3, 1)[0].tolist() == [1, 0]
    # the best alone: a tie of groups 0 and 1
    assert U.choose(l, None, 2, "sigmoid", 3, 1, 1)[0].tolist() == [1, 0]
    assert U.choose(l, None, 2, "sigmoid", 3, 2, 1)[0].tolist() == [1, 2]
    w, _ = U.weights(l, np.array([[1, 0, 3]]), "softmax", True, 2.0)
    assert np.allclose(w, 2 * np.array([[math.e ** 2, 1, 0]]) / (math.e ** 2 + 1))
    perm, pos, off = U.sort(np.array([[1, 0], [-1, 1], [2, 0]]), 3)
    assert perm.tolist() == [1, 5, 0, 3, 4, -1] and off.tolist() == [0, 2, 4, 5]
    assert pos.tolist() == [2, 0, -1, 3, 4, 1]


def test_plain_codes_are_the_definition():
    x = np.array([[127.0, 0.5, 1.5, -0.5, 126.5, -127], [0] * 6, [1, np.inf, 0, 0, 0, 0]])
    q, s = U.int8_codes(x)
    assert q[0].tolist() == [127, 0, 2, 0, 126, -127] and s[0] == 1 and s[1] == 0
    assert (q[1:] == 0).all() and np.isnan(s[2])


def test_plain_iteration_is_the_polynomial():
    g = torch.randn(5, 8, dtype=torch.float64, generator=torch.Generator().manual_seed(1))
    y, bound = U.orthogonalize(g, [U.USUAL] * 5)
    u, s, v = torch.linalg.svd(g, full_matrices=False)
    s = s / torch.linalg.vector_norm(s)
    for _ in range(5):
        a, b, c = U.USUAL
        s = a * s + b * s ** 3 + c * s ** 5
    assert torch.allclose(y, u @ torch.diag(s) @ v) and 0 < bound < 2.3
