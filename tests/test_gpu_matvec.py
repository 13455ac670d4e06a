"""Few bf16 rows times NVFP4 weights against the decoded weights in 64 bits.

The products are exact.  x is rounded at 2^-22 of its slice's largest element, which
for normal numbers is under 6 of the mean magnitude: 12 * 2^-23 of the terms'
absolute values.  In the fp32 sum a tensor-core step of 64 products may drop bits
below 2^-23 of its largest term, at most 36 steps an accumulator at these sizes, then
at most 3 + 7 + 8 additions: under 64 * 2^-23 of the terms' absolute values in all;
then eps / 2 of the stored type.
"""

import pytest
import torch

import oracle as O
from tests.gpu_common import lib

pytestmark = pytest.mark.gpu

SUM = 64 * 2.0 ** -23


@pytest.fixture(scope="module")
def ig4(cuda_device):
    return lib()


def weights(ig4, g, N, K):
    """codes, packed scales, fp32 scale, and the weights they stand for (64 bits)."""
    codes = torch.randint(0, 256, (N, K // 2), device="cuda", generator=g, dtype=torch.uint8)
    # every finite non-negative E4M3 value, subnormal ones too
    sf = torch.randint(0, 127, (N, K // 16), device="cuda", generator=g, dtype=torch.uint8)
    scale = torch.rand(N, device="cuda", generator=g) + 0.5
    packed = torch.empty(ig4.ig4_nvfp4_scale_bytes(N, K), dtype=torch.uint8, device="cuda")
    ig4.ig4_nvfp4_pack_scales(sf, packed)
    ref = torch.from_numpy(O.dequant_nvfp4(codes.cpu().numpy(), sf.cpu().numpy(),
                                           scale.cpu().numpy())).cuda()
    return codes, packed, scale, ref


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def done(ig4):
    torch.cuda.synchronize()
    assert ig4.ig4_last_device_error() == ig4.IG4_OK


# one weight row to many, rows that end inside a tile and a block, one k-block to the longest K,
# odd halves of the last 128-element chunk, every cluster size
@pytest.mark.parametrize("M,N,K", [(1, 1, 64), (1, 16, 128), (3, 100, 192), (8, 129, 1088),
                                   (2, 4608, 1024), (1, 4608, 12288), (8, 640, 12288),
                                   (5, 33, 24576), (7, 300, 8256), (4, 20000, 576),
                                   (8, 2816, 4608), (6, 257, 6208)])
@pytest.mark.parametrize("odt", [torch.float32, torch.bfloat16])
def test_matvec(ig4, M, N, K, odt):
    g = gen(M + N + K)
    codes, sf, scale, ref = weights(ig4, g, N, K)
    x = torch.randn(M, K, device="cuda", generator=g).to(torch.bfloat16)
    bias = torch.randn(N, device="cuda", generator=g)
    for b in (bias, None):
        out = torch.full((M, N), float("nan"), dtype=odt, device="cuda")
        ig4.ig4_nvfp4_matvec(x, codes, sf, scale, b, out)
        done(ig4)
        want = x.double() @ ref.T + (0 if b is None else b.double())
        size = x.double().abs() @ ref.abs().T + want.abs()
        assert torch.all((out.double() - want).abs() <=
                         torch.finfo(odt).eps / 2 * want.abs() + SUM * size)


@pytest.mark.parametrize("M,I,K", [(1, 1, 64), (8, 384, 1024), (2, 12288, 4608), (5, 700, 12352),
                                   (3, 4100, 640)])
def test_swiglu_matvec(ig4, M, I, K):
    g = gen(M + I + K)
    (gc, gs, gf, gw), (uc, us, uf, uw) = weights(ig4, g, I, K), weights(ig4, g, I, K)
    # gates of order one: the scales above reach 448 * 6
    gf *= K ** -0.5 / 100
    gw *= K ** -0.5 / 100
    x = torch.randn(M, K, device="cuda", generator=g).to(torch.bfloat16)
    out = torch.full((M, I), float("nan"), dtype=torch.bfloat16, device="cuda")
    ig4.ig4_nvfp4_swiglu_matvec(x, gc, gs, gf, uc, us, uf, out)
    done(ig4)
    x = x.double()
    G, U = x @ gw.T, x @ uw.T
    want = G * torch.sigmoid(G) * U
    # |silu'| <= 1.1; its own evaluation (exponential, divide) is good to 2^-20
    tol = SUM * (1.1 * (x.abs() @ gw.abs().T) * U.abs() + G.abs() * (x.abs() @ uw.abs().T))
    assert torch.all((out.double() - want).abs() <= (2.0 ** -8 + 2.0 ** -19) * want.abs() + 1.2 * tol)


@pytest.mark.parametrize("power", [-120, -40, 40, 100])
def test_rows_of_very_different_size(ig4, power):
    """Every row has its own power of two: tiny and huge rows next to one another."""
    M, N, K = 4, 256, 2048
    g = gen(power + 500)
    codes, sf, scale, ref = weights(ig4, g, N, K)
    x = torch.randn(M, K, device="cuda", generator=g).to(torch.bfloat16)
    x[1] *= 2.0 ** power
    x[2] = 0
    out = torch.empty(M, N, device="cuda")
    ig4.ig4_nvfp4_matvec(x, codes, sf, scale, None, out)
    done(ig4)
    want = x.double() @ ref.T
    size = x.double().abs() @ ref.abs().T
    # results under the smallest normal fp32 number are rounded at 2^-149
    assert torch.all((out.double() - want).abs() <= 2.0 ** -24 * want.abs() + SUM * size + 2.0 ** -126)
    assert torch.all(out[2] == 0)


def test_infinity_and_nan_stay_in_their_row(ig4):
    M, N, K = 3, 128, 512
    g = gen(9)
    codes, sf, scale, ref = weights(ig4, g, N, K)
    codes |= 0x11  # no zero weight: infinity times zero is NaN in the formula too
    x = torch.randn(M, K, device="cuda", generator=g).to(torch.bfloat16)
    x[0, 3], x[2, 400] = float("inf"), float("nan")
    out = torch.empty(M, N, device="cuda")
    ig4.ig4_nvfp4_matvec(x, codes, sf, scale, None, out)
    done(ig4)
    assert torch.all(torch.isfinite(out[1])) and torch.all(torch.isnan(out[2]))
    assert not torch.any(torch.isfinite(out[0]))


def test_captured_on_another_stream_and_side_by_side(ig4):
    """Two calls at once on two streams, then captured and replayed: the same bits."""
    g = gen(4)
    codes, sf, scale, _ = weights(ig4, g, 2816, 4608)
    x = torch.randn(4, 4608, device="cuda", generator=g).to(torch.bfloat16)
    want, out, other = (torch.empty(4, 2816, device="cuda") for _ in range(3))
    ig4.ig4_nvfp4_matvec(x, codes, sf, scale, None, want)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        ig4.ig4_nvfp4_matvec(x, codes, sf, scale, None, out, stream=a)
        ig4.ig4_nvfp4_matvec(x, codes, sf, scale, None, other, stream=b)
    done(ig4)
    assert torch.equal(out, want) and torch.equal(other, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ig4.ig4_nvfp4_matvec(x, codes, sf, scale, None, out)
    out.zero_()
    graph.replay()
    done(ig4)
    assert torch.equal(out, want)


def test_binding_refuses(ig4):
    g = gen(1)
    codes, sf, scale, _ = weights(ig4, g, 128, 256)
    x = torch.zeros(2, 256, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(2, 128, device="cuda")
    for bad in ((x.float(), codes, sf, scale, None, out),
                (x[:, ::2], codes, sf, scale, None, out),
                (x, codes[:, :64], sf, scale, None, out),
                (x, codes, sf[:-1], scale, None, out),
                (x, codes, sf, scale[:5], None, out),
                (x, codes, sf, scale, scale[:5], out),
                (x, codes, sf, scale, None, out.t()),
                (x.cpu(), codes, sf, scale, None, out)):
        with pytest.raises(ig4.Ig4Error) as e:
            ig4.ig4_nvfp4_matvec(*bad)
        assert e.value.status == ig4.IG4_ERR_INVALID_ARG


@pytest.mark.parametrize("M,N,K", [(1, 16384, 12288), (8, 16384, 12288), (3, 9216, 24576),
                                   (5, 40000, 2048)])
def test_more_row_tiles_than_the_device_takes_at_once(ig4, M, N, K):
    """Several rounds of row tiles: every buffer used again and again, in step over a cluster.
    Up to 48 steps an accumulator: 12 + 48 + 9 = 69, under 80 * 2^-23."""
    g = gen(M + N + K)
    codes = torch.randint(0, 256, (N, K // 2), device="cuda", generator=g, dtype=torch.uint8)
    sf = torch.randint(0, 127, (N, K // 16), device="cuda", generator=g, dtype=torch.uint8)
    scale = torch.rand(N, device="cuda", generator=g) + 0.5
    packed = torch.empty(ig4.ig4_nvfp4_scale_bytes(N, K), dtype=torch.uint8, device="cuda")
    ig4.ig4_nvfp4_pack_scales(sf, packed)
    x = torch.randn(M, K, device="cuda", generator=g).to(torch.bfloat16)
    out, again = (torch.full((M, N), float("nan"), device="cuda") for _ in range(2))
    ig4.ig4_nvfp4_matvec(x, codes, packed, scale, None, out)
    for _ in range(20):
        ig4.ig4_nvfp4_matvec(x, codes, packed, scale, None, again)
    done(ig4)
    assert torch.equal(out, again)
    value = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6],
                         dtype=torch.float64, device="cuda")
    for rows in torch.arange(N, device="cuda").split(2048):
        c = codes[rows].long()
        w = torch.stack([value[c & 15], value[c >> 4]], -1).reshape(len(rows), K)
        w *= sf[rows].view(torch.float8_e4m3fn).double().repeat_interleave(16, 1)
        w *= scale[rows, None].double()
        want, size = x.double() @ w.T, x.double().abs() @ w.abs().T
        assert torch.all((out[:, rows].double() - want).abs() <= 2.0 ** -24 * want.abs() + 80 * 2.0 ** -23 * size)
