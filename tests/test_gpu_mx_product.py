"""Products of microscaled tensors: the ways in which the two kernels join,
add up and store their sums."""
import numpy as np
import pytest
import torch

import mx_ref as ref
from test_gpu_mx import U23, fill, mx, random_bits  # noqa: F401  (mx is the module's fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K", [(1, 100, 8192), (1, 4, 16384), (3, 4000, 8192), (1, 8192, 8192), (2, 9001, 520),
                                   (200, 1, 8192), (300, 33, 8200), (130, 64, 2100), (100, 1100, 4096)])
@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_few_results_joined_from_a_cluster(mx, fmt, M, N, K):
    """K cut over 1, 2, 4 and 8 CTAs, C by rows and across them, with fewer results
    than a round of loads takes: right, and the same bits in every one of many calls
    that follow one another without a pause."""
    rng = np.random.default_rng(M + 3 * N + K)
    a, va = fill(mx, fmt, random_bits(rng, M, K, 0.5))
    b, vb = fill(mx, fmt, random_bits(rng, N, K, 0.5))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = [torch.full((M, N), float("nan"), device="cuda") for _ in range(50)]
    for c in out:
        mx.matmul(a, b, out=c, status=status)
    assert int(status.item()) == 0
    got = out[0].cpu().numpy().astype(np.float64)
    assert (np.abs(got - va @ vb.T) <= (K + 2) * U23 * (np.abs(va) @ np.abs(vb).T)).all()
    assert all(torch.equal(c, out[0]) for c in out)
