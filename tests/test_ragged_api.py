"""The ragged expert operators' argument checks and host functions: exact
status codes before any GPU call (no GPU needed)."""
import ctypes
import os

import numpy as np
import pytest
import torch

import ragged_util as R


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
    return e.value.status, str(e.value)


BAD = [
    (dict(rows=-1), "INVALID"), (dict(E=0), "INVALID"), (dict(N=0), "INVALID"),
    (dict(K=0), "INVALID"), (dict(dtype=3), "INVALID"), (dict(dtype=-1), "INVALID"),
    (dict(ld_x=63), "INVALID"), (dict(ld_y=-4), "INVALID"), (dict(E=1025), "UNSUPPORTED"),
    (dict(rows=2 ** 31), "UNSUPPORTED"), (dict(ld_y=2 ** 20 + 1), "UNSUPPORTED"),
    (dict(N=2 ** 15, K=2 ** 14, E=1), "UNSUPPORTED"),
    (dict(rows=2 ** 31 - 1, N=2 ** 16), "UNSUPPORTED"),
]


def grouped(B, **kw):
    a = dict(rows=10, E=4, N=32, K=64, dtype=B.MOE_BF16, ld_x=0, ld_y=0)
    a.update(kw)
    return B.MoeGrouped(*(a[n] for n, _ in B.MoeGrouped._fields_))


@pytest.mark.parametrize("kw,status", BAD)
def test_shapes_are_refused(B, kw, status):
    want = {"INVALID": B.MOE_ERR_INVALID_ARGUMENT, "UNSUPPORTED": B.MOE_ERR_UNSUPPORTED}[status]
    g = ctypes.byref(grouped(B, **kw))
    assert err(B, "moe_grouped_gemm", g, P, P, P, P, None)[0] == want
    assert err(B, "moe_grouped_gemm_dx", g, P, P, P, P, None)[0] == want
    assert err(B, "moe_grouped_gemm_dw", g, P, P, P, P, 0, P, 1 << 40, None)[0] == want
    assert err(B, "moe_mxfp4_grouped_gemm", g, P, P, P, P, P, P, None)[0] == want
    n = ctypes.c_size_t(0)
    assert err(B, "moe_grouped_dw_workspace_size", g, ctypes.byref(n))[0] == want


def test_pointers_are_checked(B):
    inv = B.MOE_ERR_INVALID_ARGUMENT
    g = ctypes.byref(grouped(B))
    for fn in ("moe_grouped_gemm", "moe_grouped_gemm_dx"):
        for i, bad in [(0, None), (1, None), (2, None), (3, None), (0, P + 2), (1, P + 1),
                       (2, P + 1), (3, P + 1)]:
            a = [P, P, P, P]
            a[i] = bad
            assert err(B, fn, g, *a, None)[0] == inv
    for i in range(6):
        for bad in (None, P + 1):
            a = [P] * 6
            a[i] = bad
            assert err(B, "moe_mxfp4_grouped_gemm", g, *a, None)[0] == inv
    for i in range(4):
        a = [P] * 4
        a[i] = None
        assert err(B, "moe_grouped_gemm_dw", g, *a, 0, None, 0, None)[0] == inv
    assert err(B, "moe_grouped_gemm_dw", g, P, P, P, P + 2, 0, None, 0, None)[0] == inv
    assert err(B, "moe_grouped_gemm_dw", g, P, P, P, P, 2, None, 0, None)[0] == inv
    assert err(B, "moe_grouped_gemm", None, P, P, P, P, None)[0] == inv
    # fp32 elements need four-byte addresses
    g32 = ctypes.byref(grouped(B, dtype=B.MOE_F32))
    assert err(B, "moe_grouped_gemm", g32, P, P + 2, P, P, None)[0] == inv


def test_weight_gradient_workspace(B):
    g = B.grouped(9000, 4, 128, 192, "bf16")
    need = B.grouped_dw_workspace_size(g)
    assert need > 0 and need % (128 * 192 * 4) == 0
    assert need == B.grouped_dw_workspace_size(B.grouped(9000, 64, 128, 192, "f32", ld_x=200))
    a = [ctypes.byref(g), P, P, P, P, 0]
    assert err(B, "moe_grouped_gemm_dw", *a, None, 1 << 40, None)[0] == B.MOE_ERR_INVALID_ARGUMENT
    assert err(B, "moe_grouped_gemm_dw", *a, P + 8, 1 << 40, None)[0] == B.MOE_ERR_INVALID_ARGUMENT
    st, msg = err(B, "moe_grouped_gemm_dw", *a, P, need - 1, None)
    assert st == B.MOE_ERR_WORKSPACE_TOO_SMALL and "workspace" in msg
    assert B.grouped_dw_workspace_size(B.grouped(0, 4, 128, 192, "bf16")) == 0
    assert B.grouped_dw_workspace_size(B.grouped(100, 4, 128, 192, "bf16")) == 0


def test_elementwise_calls_are_checked(B):
    inv, uns = B.MOE_ERR_INVALID_ARGUMENT, B.MOE_ERR_UNSUPPORTED
    bf = B.MOE_BF16
    sw = lambda *a: err(B, "moe_swiglu", *a)[0]
    assert sw(5, 4, 8, P, 0, P, 0, None, None) == inv
    assert sw(bf, -1, 8, P, 0, P, 0, None, None) == inv
    assert sw(bf, 4, 0, P, 0, P, 0, None, None) == inv
    assert sw(bf, 4, 8, P, 15, P, 0, None, None) == inv
    assert sw(bf, 4, 8, P, 0, P, 7, None, None) == inv
    assert sw(bf, 4, 8, None, 0, P, 0, None, None) == inv
    assert sw(bf, 4, 8, P, 0, P + 1, 0, None, None) == inv
    assert sw(bf, 4, 8, P, 0, P, 0, P + 1, None) == inv
    assert sw(bf, 2 ** 31, 8, P, 0, P, 0, None, None) == uns
    assert sw(bf, 4, 2 ** 20, P, 0, P, 0, None, None) == uns
    assert sw(bf, 4, 2 ** 62, P, 0, P, 0, None, None) == uns
    bw = lambda *a: err(B, "moe_swiglu_backward", *a)[0]
    assert bw(bf, 4, 8, P, 0, P, 0, P, 15, None, None) == inv
    assert bw(bf, 4, 8, P, 0, None, 0, P, 0, None, None) == inv
    assert bw(bf, 4, 8, P, 0, P, 0, None, 0, None, None) == inv
    q = lambda *a: err(B, "moe_mxfp4_quantize", *a)[0]
    assert q(bf, 4, 33, P, 0, 4, None, 1, None, P, P, None) == inv
    assert q(bf, 4, 32, P, 31, 4, None, 1, None, P, P, None) == inv
    assert q(bf, 4, 32, P, 0, 4, P, 0, None, P, P, None) == inv
    assert q(bf, 4, 32, P, 0, -1, P, 1, None, P, P, None) == inv
    assert q(bf, 4, 32, P, 0, 4, P + 2, 1, None, P, P, None) == inv
    assert q(bf, 4, 32, P, 0, 4, None, 1, None, P + 4, P, None) == inv
    assert q(bf, 4, 32, P, 0, 4, None, 1, None, P, None, None) == inv
    assert q(bf, 4, 32, None, 0, 4, None, 1, None, P, P, None) == inv
    dq = lambda *a: err(B, "moe_mxfp4_dequantize", *a)[0]
    assert dq(bf, 4, 40, P, P, P, 0, None, None) == inv
    assert dq(bf, 4, 32, P, P, P, 16, None, None) == inv
    assert dq(bf, 4, 32, P, P + 8, P, 0, None, None) == inv
    assert dq(9, 4, 32, P, P, P, 0, None, None) == inv
    g = ctypes.byref(grouped(B, K=48))
    assert err(B, "moe_mxfp4_grouped_gemm", g, P, P, P, P, P, P, None)[0] == inv
    g = ctypes.byref(grouped(B, K=64, ld_x=128))
    assert err(B, "moe_mxfp4_grouped_gemm", g, P, P, P, P, P, P, None)[0] == inv


def test_scale_rows(B):
    assert [B.mxfp4_scale_stride(k) for k in (32, 64, 128, 160, 256, 7168)] == [4, 4, 4, 8, 8, 224]
    for k in (32, 64, 128, 160, 1056, 7168):
        assert B.load().moe_mxfp4_scale_stride(k) == B.mxfp4_scale_stride(k)
    for k in (0, -32, 31, 48):
        assert B.load().moe_mxfp4_scale_stride(k) == -1
        with pytest.raises(ValueError):
            B.mxfp4_scale_stride(k)


def test_calls_without_rows_launch_nothing(B):
    g = ctypes.byref(grouped(B, rows=0))
    L = B.load()
    assert L.moe_grouped_gemm(g, None, None, None, None, None) == B.MOE_OK
    assert L.moe_grouped_gemm_dx(g, None, None, None, None, None) == B.MOE_OK
    assert L.moe_mxfp4_grouped_gemm(g, None, None, None, None, None, None, None) == B.MOE_OK
    assert L.moe_swiglu(B.MOE_F16, 0, 8, None, 0, None, 0, None, None) == B.MOE_OK
    assert L.moe_mxfp4_quantize(B.MOE_F16, 0, 32, None, 0, 0, None, 1, None, None, None,
                                None) == B.MOE_OK


def test_host_tensors_are_refused(B, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    g = B.grouped(4, 1, 8, 32, "bf16")
    t = torch.zeros(4, 32, dtype=torch.bfloat16)
    off = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        B.moe_grouped_gemm(g, off, t, t, t)
    with pytest.raises(ValueError):
        B.moe_swiglu(t, t)
    with pytest.raises(ValueError):
        B.moe_mxfp4_quantize(t, t, t)


def test_plain_codes_are_the_definition():
    """The tests' own quantiser: borders, ties and special blocks."""
    x = np.zeros((1, 32))
    x[0, :12] = [4.0, 0.25, 0.26, 0.75, 1.25, 1.26, 1.75, 2.5, 2.51, 3.5, 5.0, 5.01]
    c, s = R.codes_of(x)
    assert s[0, 0] == 127
    assert c[0, :12].tolist() == [6, 0, 1, 2, 2, 3, 4, 4, 5, 6, 6, 7]
    x[0, 0] = 7.99
    assert R.codes_of(x)[0][0, 0] == 7 and R.codes_of(x)[1][0, 0] == 127
    x[0, 0] = 8.0
    assert R.codes_of(x)[1][0, 0] == 128
    x[0, 3] = np.nan
    assert R.codes_of(x)[1][0, 0] == 255
    assert R.codes_of(np.zeros((1, 32)))[1][0, 0] == 0
    v = R.values_of(*R.codes_of(np.full((1, 32), 3.0)))
    assert (v == 3.0).all()
    q = np.arange(32, dtype=np.uint8).reshape(1, 32) % 16
    assert np.array_equal(R.unpack(R.pack(q)), q)


@pytest.mark.parametrize("kw", [dict(E=2**32 + 1), dict(N=2**31), dict(K=-2**31 - 1)])
def test_sizes_past_32_bits_are_refused(B, kw):
    with pytest.raises(ValueError, match="32 bits"):
        B.grouped(**{**dict(rows=4, E=1, N=8, K=8, dtype="bf16"), **kw})


@pytest.mark.parametrize("shape,have,ok", [
    ((4, 16, 8), (4, 16, 8), True), ((4, 16, 8), (5, 16, 8), True), ((4, 16, 8), (64, 8), True),
    ((4, 16, 8), (4, 128), True), ((4, 16, 8), (512,), True), ((4, 16, 8), (4, 2, 8, 8), True),
    ((4, 16, 8), (4, 16, 2, 4), True), ((8, 4), (2, 4, 4), True), ((3, 4), (8, 16), True),
    ((0, 4), (0, 16), True), ((4, 16, 8), (4, 8, 16), False), ((4, 4, 16), (4, 16, 4), False),
    ((4, 16, 8), (8, 64), False), ((4, 16, 8), (3, 16, 8), False), ((8, 12), (8, 16), False),
    ((8, 12), (24, 4), False)])
def test_layouts_of_matrices_are_checked(B, monkeypatch, shape, have, ok):
    """Tensors of other shapes are taken where their rows are the shape's."""
    monkeypatch.setattr(B, "_on_device", lambda t, name, dev: None)

    def address(t, name, dtype, numel):
        if t.numel() < numel:
            raise ValueError(name)
        return t.data_ptr()

    monkeypatch.setattr(B, "_arg", address)
    t = torch.zeros(have)
    if ok:
        assert B._matrices(t, "w", torch.float32, shape, 0) == t.data_ptr()
    else:
        with pytest.raises(ValueError, match="w"):
            B._matrices(t, "w", torch.float32, shape, 0)


def test_weight_gradient_workspace_is_small_beside_the_operands(B):
    """Few slots where many rows meet small matrices: a chunk has 512 rows, or in
    fp32 128 where there are at most 4096."""
    size = lambda rows, dt: B.grouped_dw_workspace_size(B.grouped(rows, 64, 256, 256, dt))
    for rows in (4097, 65536, 131072):
        for dt in ("bf16", "f16", "f32"):
            assert size(rows, dt) <= rows // 512 * 256 * 256 * 4
    assert size(4096, "bf16") == 8 * 256 * 256 * 4 and size(4096, "f32") == 32 * 256 * 256 * 4


@pytest.mark.parametrize("n", [0, 8, 64, 2**31 - 1, True])
def test_numbers_of_rows_are_not_taken_for_addresses(B, n):
    with pytest.raises(TypeError, match="n_rows"):
        B._n_rows(n, 0)
    assert B._n_rows(None, 0) is None and B._n_rows(1 << 46, 0) == 1 << 46
