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


# ---------------------------------------------------------- waits that give up

def check_give_up(mx, fmt, M, N, K, out, limits):
    """Products whose waits give up at once, or some of them in the middle: each
    call ends by itself and says so in its status word or is right, and nothing of it
    is left to those that follow."""
    from lossless_bf16_exponent_codec_gb300 import binding as B
    rng = np.random.default_rng(M + N + K)
    a, _ = fill(mx, fmt, random_bits(rng, M, K, 0.5))
    b, _ = fill(mx, fmt, random_bits(rng, N, K, 0.5))
    kind = torch.bfloat16 if out == "bf16" else torch.float32
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    good = mx.matmul(a, b, dtype=kind, status=status)
    assert int(status.item()) == 0
    c = torch.empty_like(good)
    try:
        for limit in limits:
            B.ez_mx_wait_limit(limit)
            status.zero_()
            mx.matmul(a, b, out=c, status=status)
            word = int(status.item())
            assert word == 8 or (word == 0 and limit > 0 and torch.equal(c, good)), (limit, word)
    finally:
        B.ez_mx_wait_limit()
    for _ in range(3):
        status.zero_()
        mx.matmul(a, b, out=c, status=status)
        assert int(status.item()) == 0 and torch.equal(c, good)


LIMITS = [0, 1, 2, 3, 5, 8, 12, 20, 40, 70, 100, 150, 300, 1000, 5000]


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("M,N,K", [(1, 100, 8192), (1, 4096, 8192), (1, 8192, 8192), (48, 10240, 5120), (200, 33, 8200),
                                   (3, 20, 100), (128, 1024, 4096)])
def test_cluster_product_that_gives_up(mx, fmt, M, N, K):
    check_give_up(mx, fmt, M, N, K, "f32", LIMITS)


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("M,N,K,out", [(700, 904, 8200, "f32"), (2304, 1920, 4400, "f32"), (4096, 4096, 2048, "bf16"),
                                       (300, 4096, 256, "bf16")])
def test_pair_product_that_gives_up(mx, fmt, M, N, K, out):
    check_give_up(mx, fmt, M, N, K, out, LIMITS)


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("M,N,K,out", [(700, 901, 8200, "f32"), (1411, 1701, 1000, "bf16"), (2304, 4101, 4400, "f32"),
                                       (300, 4097, 256, "bf16")])
def test_pair_product_across_the_lanes_that_gives_up(mx, fmt, M, N, K, out):
    """Odd rows of C leave through memory that four warps share: each of them may
    give up by itself, none may be left waiting for another."""
    check_give_up(mx, fmt, M, N, K, out, LIMITS)


# ------------------------------------------------------------------- long sums

@pytest.mark.parametrize("place", ["apart", "in place"])
@pytest.mark.parametrize("M,N", [(1300, 1040), (1300, 1041), (1300, 1044)])
@pytest.mark.parametrize("fmt,K", [("e4m3", 8 * 24 * 128), ("e2m1", 8 * 24 * 256), ("e4m3", 700)])
def test_addend_is_added_once(mx, fmt, K, M, N, place):
    """C is the product, to which the addend is added in one FP32 addition, also
    when the parts of the sum are each lost beside it: 3/4 from each eighth of K
    (times a power of two of the row) under addends whose steps are from 1/8 to 4
    times that."""
    g = torch.Generator(device="cuda")
    g.manual_seed(K + N)
    x, y = torch.zeros(M, K, device="cuda"), torch.zeros(N, K, device="cuda")
    at = torch.arange(8, device="cuda") * (K // 8) + 5
    row = torch.exp2(torch.randint(-3, 3, (M, 1), generator=g, device="cuda").float())
    x[:, at], y[:, at] = row, 0.75
    a, b = mx.MxTensor.empty(fmt, M, K), mx.MxTensor.empty(fmt, N, K)
    mx.quantize(x.to(torch.bfloat16), row=a)
    mx.quantize(y.to(torch.bfloat16), row=b)
    add = 2.0 ** 23 * (1 + torch.rand(M, N, generator=g, device="cuda"))
    want = (add.double() + 6 * row.double()).float()
    c = mx.matmul(a, b, out=add if place == "in place" else None, add=add)
    assert torch.equal(c, want)


@pytest.mark.parametrize("sign", ["random", "one"])
@pytest.mark.parametrize("M,N", [(1300, 1344), (16, 12800)])
@pytest.mark.parametrize("fmt,K", [("e4m3", 16384), ("e2m1", 32768)])
def test_long_sums_in_fp32(mx, fmt, K, M, N, sign):
    """The tensor core cuts off where FP32 rounds: over the 512 additions of these
    sums that costs 8-bit operands 3e-6 of the result and more where all terms have one
    sign (root mean square of the errors over that of the results); in segments of 96
    additions, which are added with rounding, 0.5e-6 to 0.6e-6.  The bound lies between.
    (1300 x 1344 takes pairs of CTAs, 16 x 12800 one CTA to a tile and all of K.)"""
    g = torch.Generator(device="cuda")
    g.manual_seed(K + N)
    x, y = (torch.randn(r, K, generator=g, device="cuda") for r in (M, N))
    if sign == "one":
        x, y = x.abs(), y.abs()
    a, b = mx.MxTensor.empty(fmt, M, K), mx.MxTensor.empty(fmt, N, K)
    mx.quantize(x.to(torch.bfloat16), row=a)
    mx.quantize(y.to(torch.bfloat16), row=b)
    want = mx.dequantize(a).double() @ mx.dequantize(b).double().t()
    got = mx.matmul(a, b, dtype=torch.float32).double()
    assert float((got - want).norm() / want.norm()) < 1e-6
