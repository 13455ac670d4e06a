"""Few rows by NVFP4 weights where the elements of one row of x differ by many powers of two:
outliers, subnormal numbers, infinities and NaN, against the decoded weights in 64 bits.

Every element of x counts with its own bits, so the error is one of fp32 sums alone, in units
of the terms' absolute values, whatever the largest element is.  Digits: an element's eight bits
lie in four digits between -4 and 3, whose places add up to at most 4 times the element (8^3 - 4
8^2 - 4 8 - 4 = 220 against 804).  Of a plane's sum a step of 64 products may drop bits below 2^-23
of its largest term, at most 24 steps an accumulator at these sizes: 96 * 2^-23; then 3 + 11 + 8
additions at 4 * 2^-24: 44 * 2^-23.  Elements multiplied one by one: 256 in a chain for a k-block,
then at most 20 k-blocks, at 2^-24 each: 138 * 2^-23.  In all under 280 * 2^-23; then eps / 2 of
the stored type.  Results below 2^-126 are rounded at 2^-149 or become 0.
"""

import pytest
import torch

from tests.gpu_common import lib
from tests.test_gpu_matvec import done, gen, weights

pytestmark = pytest.mark.gpu

SUM = 280 * 2.0 ** -23
TINY = 2.0 ** -126


@pytest.fixture(scope="module")
def ig4(cuda_device):
    return lib()


def check(out, x, ref):
    want = x.double() @ ref.T
    size = x.double().abs() @ ref.abs().T
    err = (out.double() - want).abs()
    assert torch.all(err <= torch.finfo(out.dtype).eps / 2 * want.abs() + SUM * size + TINY)


@pytest.mark.parametrize("M,N,K", [(1, 512, 4608), (3, 256, 1088), (8, 256, 12288)])
@pytest.mark.parametrize("big", [1e5, -1e6, 1e9, 1e30])
def test_outliers(ig4, M, N, K, big):
    """One huge channel: an output whose weight there is zero does not see it."""
    g = gen(M + N + K)
    codes, sf, scale, ref = weights(ig4, g, N, K)
    x = torch.randn(M, K, device="cuda", generator=g).to(torch.bfloat16)
    x[:, K // 3] = big
    assert (ref[:, K // 3] == 0).sum() > N // 16
    out = torch.full((M, N), float("nan"), device="cuda")
    ig4.ig4_nvfp4_matvec(x, codes, sf, scale, None, out)
    done(ig4)
    check(out, x, ref)


# places around the ends of what digits hold, then every power of two there is; shapes with one and
# many CTAs in a cluster, several rounds of row tiles, and the longest rows
@pytest.mark.parametrize("M,N,K", [(1, 100, 64), (2, 300, 1088), (5, 20000, 320), (8, 129, 4608),
                                   (4, 300, 24576), (7, 130, 24576), (8, 130, 24576)])
@pytest.mark.parametrize("low,high", [(-40, 0), (-133, 110)])
def test_every_power_of_two(ig4, M, N, K, low, high):
    g = gen(M + N + K - low)
    codes, sf, scale, ref = weights(ig4, g, N, K)
    power = torch.randint(low, high + 1, (M, K), device="cuda", generator=g)
    x = torch.ldexp(torch.randn(M, K, device="cuda", generator=g, dtype=torch.float64), power)
    x = x.to(torch.bfloat16)
    out, again = (torch.full((M, N), float("nan"), device="cuda") for _ in range(2))
    ig4.ig4_nvfp4_matvec(x, codes, sf, scale, None, out)
    ig4.ig4_nvfp4_matvec(x, codes, sf, scale, None, again)
    done(ig4)
    check(out, x, ref)
    assert torch.equal(out, again)


@pytest.mark.parametrize("M,I,K", [(1, 300, 1088), (8, 300, 24576), (3, 12288, 320)])
def test_gated_outliers(ig4, M, I, K):
    g = gen(M + I + K)
    (gc, gs, gf, gw), (uc, us, uf, uw) = weights(ig4, g, I, K), weights(ig4, g, I, K)
    gf *= K ** -0.5 / 100
    gw *= K ** -0.5 / 100
    x = torch.randn(M, K, device="cuda", generator=g).to(torch.bfloat16)
    x[:, 5::97] *= 2.0 ** -30
    x[:, K // 2] = 1e9
    zero = (gw[:, K // 2] == 0) & (uw[:, K // 2] == 0)
    assert zero.sum() > 0
    out = torch.full((M, I), float("nan"), dtype=torch.bfloat16, device="cuda")
    ig4.ig4_nvfp4_swiglu_matvec(x, gc, gs, gf, uc, us, uf, out)
    done(ig4)
    x = x.double()
    G, U = x @ gw.T, x @ uw.T
    want = G * torch.sigmoid(G) * U
    # |silu'| <= 1.1, its evaluation good to 2^-20, as in test_gpu_matvec.py
    tol = SUM * (1.1 * (x.abs() @ gw.abs().T) * U.abs() + G.abs() * (x.abs() @ uw.abs().T))
    ok = (out.double() - want).abs() <= (2.0 ** -8 + 2.0 ** -19) * want.abs() + 1.2 * tol + TINY
    assert torch.all(ok[:, zero])


def test_infinities_and_nan(ig4):
    """As in the formula: an infinity where the weight is not zero, NaN where it is, and where
    infinities of both signs or a NaN meet; other rows of x do not notice."""
    M, N, K = 5, 384, 1088
    g = gen(77)
    codes, sf, scale, ref = weights(ig4, g, N, K)
    x = torch.randn(M, K, device="cuda", generator=g).to(torch.bfloat16)
    x[0, 3], x[1, 1000], x[3, 9] = float("inf"), float("-inf"), float("nan")
    x[2, 40], x[2, 700] = float("inf"), float("inf")
    out = torch.empty(M, N, device="cuda")
    ig4.ig4_nvfp4_matvec(x, codes, sf, scale, None, out)
    done(ig4)
    want = x.double() @ ref.T
    assert torch.isinf(want[0]).any() and torch.isnan(want[2]).any() and torch.isinf(want[2]).any()
    bad = ~torch.isfinite(want)
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    assert torch.equal(out[bad].nan_to_num(nan=0.0).sign().double(),
                       want[bad].nan_to_num(nan=0.0).sign())
    assert torch.equal(torch.isinf(out), torch.isinf(want))
    check(out[4:], x[4:], ref)
    x[0] = float("inf")  # a row without a finite element
    ig4.ig4_nvfp4_matvec(x, codes, sf, scale, None, out)
    done(ig4)
    assert not torch.isfinite(out[0]).any()
    check(out[4:], x[4:], ref)


def test_captured_with_outliers(ig4):
    g = gen(6)
    codes, sf, scale, ref = weights(ig4, g, 2816, 4608)
    x = torch.randn(4, 4608, device="cuda", generator=g).to(torch.bfloat16)
    out = torch.empty(4, 2816, device="cuda")
    graph = torch.cuda.CUDAGraph()
    ig4.ig4_nvfp4_matvec(x, codes, sf, scale, None, out)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        ig4.ig4_nvfp4_matvec(x, codes, sf, scale, None, out)
    for big in (1e9, 1.0, float("inf"), 1e30):  # strays come and go between the replays
        x[:, 1234] = big
        graph.replay()
        done(ig4)
        if big != float("inf"):
            check(out, x, ref)
