"""Routing and sort where the sizes or values are extreme, compared with what is known
exactly."""
import numpy as np
import pytest
import torch

import routing_util as U

pytestmark = pytest.mark.gpu

MOST = torch.finfo(torch.float32).max


@pytest.fixture(scope="module")
def B():
    from round_dropless_expert_amd import binding
    binding.load()
    binding.check_runtime()
    return binding


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


@pytest.mark.parametrize("mode", ["even", "skewed", "one", "padded"])
@pytest.mark.parametrize("n,E", [(1048576, 256), (1048577, 256), (1048577, 1024), (2000003, 256),
                                 (2000003, 1024), (5000011, 40)])
def test_sort_long_runs(B, n, E, mode):
    """More than 2^20 assignments: a wavefront's run is longer than what it keeps, so it
    reads the rest twice."""
    idx = torch.randint(0, E, (n,), generator=gen(n + E), device="cuda", dtype=torch.int32)
    if mode == "skewed":
        idx = torch.where(torch.rand(n, generator=gen(1), device="cuda") < 0.6, idx % 3, idx)
    if mode == "one":
        idx[:] = E - 1
    if mode == "padded":
        m = torch.rand(n, generator=gen(3), device="cuda")
        idx[m < 0.2] = -1
        idx[m > 0.9] = E
        idx[m > 0.95] = 2 ** 31 - 1
        idx[-70000:] = -1
    perm, pos = (torch.full((n + 1,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    off = torch.full((E + 2,), -9, dtype=torch.int32, device="cuda")
    ws = torch.full((B.sort_workspace_size(n, E),), 255, dtype=torch.uint8, device="cuda")
    B.moe_sort(idx, E, perm, pos, off, ws)
    want = U.sort(idx.cpu().numpy(), E)
    for got, ref, name in zip((perm[:n], pos[:n], off[: E + 1]), want, ("perm", "pos", "offsets")):
        assert np.array_equal(got.cpu().numpy(), ref), name
    assert perm[n] == -9 and pos[n] == -9 and off[E + 1] == -9
