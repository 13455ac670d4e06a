"""Residual addition + RMSNorm and its gradients against the formulas in 64 bits.

Tolerances count roundings: eps / 2 of the stored type relative to the value,
and in fp32 the sums of squares (at most 16 terms per thread, 5 shuffles and 16
warps in a chain of positive terms: 37 roundings, halved by the root), the root
(2 ulp) and the products: under 40 * 2^-24 relative to y in all.
"""

import pytest
import torch

from tests.gpu_common import lib

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
C32 = 40 * U32
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def ig4(cuda_device):
    return lib()


def half(dt):
    return torch.finfo(dt).eps / 2


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return lambda *shape, dt=torch.float32, std=1.0: (
        torch.randn(*shape, device="cuda", generator=g) * std).to(dt)


def reference(x, r, g, eps):
    t = x.double() + (0 if r is None else r.double())
    y = t / (t.pow(2).mean(-1, keepdim=True) + eps).sqrt()
    return t, y if g is None else y * g.double()


def done(ig4):
    torch.cuda.synchronize()
    assert ig4.ig4_last_device_error() == ig4.IG4_OK


# every launch form: a warp per row (D <= 512), one to sixteen warps per row, one row to more
# rows than a grid has CTAs; widths that end inside a thread's vectors and inside a warp
SHAPES = [(1, 8), (1, 4608), (3, 512), (5, 520), (700, 264), (2, 8192), (37, 1032), (1500, 4608),
          (33, 8184), (5000, 16)]


@pytest.mark.parametrize("M,D", SHAPES)
@pytest.mark.parametrize("xdt", ["bf16", "f32"])
@pytest.mark.parametrize("ydt", ["bf16", "f32"])
def test_add_rms_norm(ig4, M, D, xdt, ydt):
    rn = gen(M * 10007 + D)
    x = rn(M, D, dt=DT[xdt]) * torch.exp(rn(M, 1, dt=DT[xdt]))
    r, g = rn(M, D, dt=DT[xdt], std=0.5), 1 + rn(D, std=0.3)
    s, y = torch.empty_like(x), torch.empty(M, D, dtype=DT[ydt], device="cuda")
    ig4.ig4_add_rms_norm(x, r, g, 1e-6, s, y)
    done(ig4)
    t64, y64 = reference(x, r, g, 1e-6)
    assert torch.all((s.double() - t64).abs() <= (half(s.dtype) + U32) * t64.abs())
    assert torch.all((y.double() - y64).abs() <= (half(y.dtype) + C32) * y64.abs())


@pytest.mark.parametrize("with_r,with_g,with_s", [(False, True, True), (True, False, False),
                                                  (False, False, False)])
def test_optional_parts(ig4, with_r, with_g, with_s):
    M, D = 9, 1280
    rn = gen(5)
    x = rn(M, D, dt=torch.bfloat16)
    r = rn(M, D, dt=torch.bfloat16) if with_r else None
    g = rn(D) if with_g else None
    s = torch.empty_like(x) if with_s else None
    y = torch.empty(M, D, device="cuda")
    ig4.ig4_add_rms_norm(x, r, g, 1e-5, s, y)
    done(ig4)
    t64, y64 = reference(x, r, g, 1e-5)
    assert torch.all((y.double() - y64).abs() <= (half(y.dtype) + C32) * y64.abs())
    if with_s and r is None:
        assert torch.equal(s, x)


@pytest.mark.parametrize("which", ["x", "r"])
def test_sum_in_place(ig4, which):
    M, D = 401, 4608
    rn = gen(6)
    x, r, g = rn(M, D, dt=torch.bfloat16), rn(M, D, dt=torch.bfloat16), rn(D)
    s, y, y2 = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    ig4.ig4_add_rms_norm(x, r, g, 1e-6, s, y)
    ig4.ig4_add_rms_norm(x, r, g, 1e-6, x if which == "x" else r, y2)
    done(ig4)
    assert torch.equal(x if which == "x" else r, s) and torch.equal(y, y2)


@pytest.mark.parametrize("M,D", [(1, 128), (130, 512), (7, 640), (257, 4608), (3, 8192)])
@pytest.mark.parametrize("xdt", ["bf16", "f32"])
def test_row_scaled_fp8(ig4, M, D, xdt):
    rn = gen(M + D)
    x, r, g = rn(M, D, dt=DT[xdt]), rn(M, D, dt=DT[xdt]), rn(D)
    x[0] = 0
    r[0] = 0  # a zero row: scale 1, codes 0
    y = torch.empty(M, D, dtype=torch.float8_e4m3fn, device="cuda")
    sc = torch.empty(M, device="cuda")
    ig4.ig4_add_rms_norm(x, r, g, 1e-6, None, y, y_scale_out=sc)
    done(ig4)
    _, y64 = reference(x, r, g, 1e-6)
    top = y64.abs().amax(1)
    want = torch.where(top > 0, top / 448, 1.0)
    assert torch.all((sc.double() - want).abs() <= (C32 + U32) * want)
    got = y.double() * sc.double()[:, None]
    # half a step of E4M3 (2^-4 relative, 2^-10 of the scale below the normal range), and the
    # fp32 arithmetic in front of it
    assert torch.all((got - y64).abs() <= (2.0 ** -4 + 2 * C32) * y64.abs() +
                     2.0 ** -10 * (1 + C32) * want[:, None])
    assert sc[0] == 1 and torch.all(y[0].float() == 0)


@pytest.mark.parametrize("M,D", [(1, 128), (129, 384), (300, 512), (257, 4608), (31, 8192)])
@pytest.mark.parametrize("xdt", ["bf16", "f32"])
def test_block_scaled_fp8_is_the_quantised_bf16_output(ig4, M, D, xdt):
    rn = gen(M * D)
    x, r, g = rn(M, D, dt=DT[xdt]), rn(M, D, dt=DT[xdt]), rn(D)
    x[M // 2, :64] = 0
    r[M // 2, :64] = 0  # zero blocks
    n = ig4.ig4_mx8_scale_bytes(M, D)
    y, yb = (torch.empty(M, D, dtype=dt, device="cuda")
             for dt in (torch.float8_e4m3fn, torch.bfloat16))
    q = torch.empty_like(y)
    # padding rows' scale bytes are not written: they keep the caller's fill
    sf, sq = (torch.full((n,), 77, dtype=torch.uint8, device="cuda") for _ in range(2))
    ig4.ig4_add_rms_norm(x, r, g, 1e-6, None, y, y_sf_out=sf)
    ig4.ig4_add_rms_norm(x, r, g, 1e-6, None, yb)
    ig4.ig4_quantize_mx8(M, D, yb, q, sq)
    done(ig4)
    assert torch.equal(y.view(torch.uint8), q.view(torch.uint8)) and torch.equal(sf, sq)


def test_infinities_and_nan_stay_in_their_rows(ig4):
    M, D = 8, 1024
    rn = gen(8)
    x, g = rn(M, D, dt=torch.bfloat16), rn(D)
    x[2, 5], x[5, 0] = float("nan"), float("inf")
    y = torch.empty(M, D, device="cuda")
    ig4.ig4_add_rms_norm(x, None, g, 1e-6, None, y)
    done(ig4)
    _, y64 = reference(x, None, g, 1e-6)
    fine = [0, 1, 3, 4, 6, 7]
    assert torch.all((y.double() - y64)[fine].abs() <= C32 * y64[fine].abs())
    assert torch.equal(torch.isnan(y), torch.isnan(y64))


# ------------------------------------------------------------------ gradients

def reference_grad(s, g, eps, dy, ds):
    s, dy = s.double(), dy.double()
    g = torch.ones_like(s[0]) if g is None else g.double()
    rstd = 1 / (s.pow(2).mean(1, keepdim=True) + eps).sqrt()
    n, dn = s * rstd, dy * g
    dx = rstd * (dn - n * (dn * n).mean(1, keepdim=True)) + (0 if ds is None else ds.double())
    # what the terms' roundings are relative to
    size = rstd * (dn.abs() + n.abs() * (dn * n).abs().mean(1, keepdim=True))
    return dx, (dy * n).sum(0), size + (0 if ds is None else ds.double().abs()), (dy * n).abs().sum(0)


def run_grad(ig4, s, g, eps, dy, ds, want_dg=True, dx=None):
    M, D = s.shape
    dx = torch.empty_like(s) if dx is None else dx
    dg = torch.empty(D, device="cuda") if want_dg else None
    ws = torch.empty(ig4.ig4_add_rms_norm_backward_workspace_size(M, D), dtype=torch.uint8,
                     device="cuda") if want_dg else None
    ig4.ig4_add_rms_norm_backward(s, g, eps, dy, ds, dx, dg, ws)
    done(ig4)
    return dx, dg


@pytest.mark.parametrize("M,D", SHAPES)
@pytest.mark.parametrize("sdt,ydt", [("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32"),
                                     ("f32", "f32")])
def test_backward(ig4, M, D, sdt, ydt):
    rn = gen(M + 3 * D)
    s = rn(M, D, dt=DT[sdt]) * torch.exp(rn(M, 1, dt=DT[sdt]))
    g, dy, ds = 1 + rn(D, std=0.3), rn(M, D, dt=DT[ydt]), rn(M, D, dt=DT[sdt])
    dx, dg = run_grad(ig4, s, g, 1e-6, dy, ds)
    dx64, dg64, size, dgsize = reference_grad(s, g, 1e-6, dy, ds)
    assert torch.all((dx.double() - dx64).abs() <= half(dx.dtype) * dx64.abs() + 2 * C32 * size)
    # dg adds M rounded terms in fp32 in some fixed order
    assert torch.all((dg.double() - dg64).abs() <= (M * U32 + C32) * dgsize)


@pytest.mark.parametrize("with_g,with_ds,with_dg", [(False, True, True), (True, False, True),
                                                    (True, True, False), (False, False, False)])
def test_backward_optional_parts(ig4, with_g, with_ds, with_dg):
    M, D = 311, 2304
    rn = gen(11)
    s, dy = rn(M, D), rn(M, D)
    g = rn(D) if with_g else None
    ds = rn(M, D) if with_ds else None
    dx, dg = run_grad(ig4, s, g, 1e-5, dy, ds, with_dg)
    dx64, dg64, size, dgsize = reference_grad(s, g, 1e-5, dy, ds)
    assert torch.all((dx.double() - dx64).abs() <= half(dx.dtype) * dx64.abs() + 2 * C32 * size)
    if with_dg:
        assert torch.all((dg.double() - dg64).abs() <= (M * U32 + C32) * dgsize)


def test_backward_in_place_repeats_bit_for_bit(ig4):
    M, D = 1000, 4608
    rn = gen(12)
    s, dy, ds, g = (rn(M, D, dt=torch.bfloat16), rn(M, D, dt=torch.bfloat16),
                    rn(M, D, dt=torch.bfloat16), rn(D))
    dx, dg = run_grad(ig4, s, g, 1e-6, dy, ds)
    dx2, dg2 = run_grad(ig4, s, g, 1e-6, dy, ds, dx=ds)
    assert torch.equal(dx, dx2) and torch.equal(dg, dg2)


@pytest.mark.parametrize("D", [24, 1544])
def test_gradient_against_differences(ig4, D):
    """<dx, v> and <dg, w> against central differences of the forward in 64 bits: the step's own
    error is h^2 times a third derivative, h = 1e-4; fp32 rounding of the gradients is the rest."""
    M, h = 6, 1e-4
    rn = gen(13)
    x, r, g, dy, ds = rn(M, D), rn(M, D), 1 + rn(D, std=0.2), rn(M, D), rn(M, D)
    s, y = torch.empty_like(x), torch.empty_like(x)
    ig4.ig4_add_rms_norm(x, r, g, 1e-6, s, y)
    dx, dg = run_grad(ig4, s, g, 1e-6, dy, ds)
    v, w = rn(M, D).double(), rn(D).double()

    def loss(a):
        t, y = reference(x.double() + a * v, r, g.double() + a * w, 1e-6)
        return (y * dy.double()).sum() + (t * ds.double()).sum()
    want = (loss(h) - loss(-h)) / (2 * h)
    got = (dx.double() * v).sum() + (dg.double() * w).sum()
    size = (dx.double() * v).abs().sum() + (dg.double() * w).abs().sum()
    assert (got - want).abs() <= 1e-6 * size


def test_capture_and_another_stream(ig4):
    """One captured forward + backward, replayed on new inputs, gives the eager bits."""
    M, D = 77, 4608
    rn = gen(14)
    x, r, dy = (rn(M, D, dt=torch.bfloat16) for _ in range(3))
    g = rn(D)
    s, y, dx = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    dg = torch.empty(D, device="cuda")
    ws = torch.empty(ig4.ig4_add_rms_norm_backward_workspace_size(M, D), dtype=torch.uint8,
                     device="cuda")

    def both(stream=None):
        ig4.ig4_add_rms_norm(x, r, g, 1e-6, s, y, stream=stream)
        ig4.ig4_add_rms_norm_backward(s, g, 1e-6, dy, None, dx, dg, ws, stream=stream)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    both(side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    x.copy_(rn(M, D, dt=torch.bfloat16))
    dy.copy_(rn(M, D, dt=torch.bfloat16))
    both()
    torch.cuda.synchronize()
    want = [t.clone() for t in (s, y, dx, dg)]
    for t in (s, y, dx, dg):
        t.zero_()
    graph.replay()
    done(ig4)
    assert all(torch.equal(a, b) for a, b in zip(want, (s, y, dx, dg)))


@pytest.mark.parametrize("D", [128, 1280])
def test_tiny_rows_keep_finite_codes(ig4, D):
    """Rows so small that max|y| / 448 has no finite reciprocal: codes of y / 2^-126, half a step
    of E4M3's smallest numbers (2^-10) off at most, and zeros stay zeros."""
    x = torch.zeros(5, D, device="cuda")
    x[1, ::3], x[2, 7], x[3, ::2], x[4, 5] = 1e-40, -1e-42, 3e-38, 2.0 ** -120
    y = torch.empty(5, D, dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty(5, device="cuda")
    ig4.ig4_add_rms_norm(x, None, None, 1.0, None, y, y_scale_out=scale)
    done(ig4)
    amax = x.double().abs().amax(-1)
    least = torch.where(amax > 0, (amax / 448).clamp(min=2.0 ** -126), 1.0)
    assert torch.all((scale.double() - least).abs() <= 2.0 ** -23 * least)
    got = y.double() * scale.double()[:, None]
    # eps / 2 of the code, half its smallest step, and the fp32 subnormals of y itself
    tol = (2.0 ** -4 + 2.0 ** -20) * x.double().abs() + 2.0 ** -10 * scale.double()[:, None] + 2.0 ** -149
    assert torch.all((got - x.double()).abs() <= tol)


@pytest.mark.parametrize("D", [256, 1280])
def test_rows_whose_squares_overflow(ig4, D):
    """|t| up to 2^57 is exact as any; a row whose squares overflow comes out as zero."""
    x = torch.randn(3, D, device="cuda")
    x[0] *= 2.0 ** 54
    x[1] *= 2.0 ** 70
    y = torch.empty_like(x)
    ig4.ig4_add_rms_norm(x, None, None, 1e-6, None, y)
    done(ig4)
    _, y64 = reference(x, None, None, 1e-6)
    assert torch.all((y[::2].double() - y64[::2]).abs() <= (half(y.dtype) + C32) * y64[::2].abs())
    assert torch.all(y[1] == 0)


def test_offsets_past_32_bits(ig4):
    """More than 2^31 elements: the last rows come out as those rows alone."""
    D = 512
    M = (1 << 31) // D + 700
    x = torch.zeros(M, D, dtype=torch.bfloat16, device="cuda")
    x[-300:] = torch.randn(300, D, device="cuda").to(x.dtype)
    y, tail = torch.empty_like(x), torch.empty_like(x[-300:])
    ig4.ig4_add_rms_norm(x, None, None, 1e-6, None, y)
    ig4.ig4_add_rms_norm(x[-300:], None, None, 1e-6, None, tail)
    done(ig4)
    assert torch.equal(y[-300:], tail) and not y[:300].any()


def test_binding_refuses(ig4):
    x, g = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda"), torch.ones(256, device="cuda")
    y, f8 = torch.empty_like(x), torch.empty(4, 256, dtype=torch.float8_e4m3fn, device="cuda")
    sc, dg = torch.empty(4, device="cuda"), torch.empty(256, device="cuda")
    sf = torch.empty(64, dtype=torch.uint8, device="cuda")
    ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    forward = [(x[:0], None, g, 1e-6, None, y[:0]), (x, x[:2], g, 1e-6, None, y),
               (x, x.float(), g, 1e-6, None, y), (x, None, g.bfloat16(), 1e-6, None, y),
               (x, None, g[:128], 1e-6, None, y), (x, None, g, 1e-6, y.float(), y),
               (x.half(), None, g, 1e-6, None, y), (x, None, g, 1e-6, None, y.half()),
               (x, None, g, 1e-6, None, y.t().contiguous().t()), (x[:, :200], None, None, 1e-6, None, y),
               (x, None, g, 1e-6, None, f8, sc[:2]), (x, None, g, 1e-6, None, f8, None, sf),
               (x, None, g, 1e-6, None, f8, sc, sf), (x, None, g.cpu(), 1e-6, None, y)]
    backward = [(x, g, 1e-6, x[:2], None, y, dg, ws), (x, g, 1e-6, x.half(), None, y, dg, ws),
                (x, g, 1e-6, x, x.float(), y, dg, ws), (x, g, 1e-6, x, None, y.float(), dg, ws),
                (x, g, 1e-6, x, None, y, dg.bfloat16(), ws), (x, g, 1e-6, x, None, x, dg, ws),
                (x, g, 1e-6, x, None, y, dg, ws.cpu())]
    for call, cases in ((ig4.ig4_add_rms_norm, forward), (ig4.ig4_add_rms_norm_backward, backward)):
        for args in cases:
            with pytest.raises(ig4.Ig4Error) as e:
                call(*args)
            assert e.value.status == ig4.IG4_ERR_INVALID_ARG
    with pytest.raises(ig4.Ig4Error) as e:
        ig4.ig4_add_rms_norm_backward(x, g, 1e-6, x, None, y, dg, ws[:256])
    assert e.value.status == ig4.IG4_ERR_WORKSPACE
