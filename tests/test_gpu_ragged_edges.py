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
