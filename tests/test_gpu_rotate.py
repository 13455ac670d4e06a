"""Rotary positions on strided heads against the formula in 64 bits.

An angle is formed in turns in fp64 and rounded to fp32 after it is reduced to
half a turn: 2^-25 of a half turn is pi 2^-25 = 9.4e-8; sincospi adds 2 ulp
(2.4e-7), the two products and the sum 2^-24 each: under 5e-7 of |x1| + |x2|,
then eps / 2 of the stored type.
"""

import pytest
import torch

from tests.gpu_common import lib

pytestmark = pytest.mark.gpu

ANGLE = 5e-7
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def ig4(cuda_device):
    return lib()


def axes_of(sections, interleaved):
    if not interleaved:
        return [a for a in range(3) for _ in range(sections[a])]
    return [a for _, a in sorted((i, a) for a in range(3) for i in range(sections[a]))]


def reference(x, pos, theta, sections, interleaved, adjacent, inverse):
    """(rotated, |x1| + |x2| of each element's pair) in 64 bits."""
    P = sum(sections)
    out, size = x.double().clone(), torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    for j, a in enumerate(axes_of(sections, interleaved)):
        lo, hi = (2 * j, 2 * j + 1) if adjacent else (j, j + P)
        ang = pos[..., a, :].double() * theta ** (-j / P) * (-1 if inverse else 1)
        c, s = ang.cos()[..., None], ang.sin()[..., None]
        x1, x2 = x[..., lo].double(), x[..., hi].double()
        out[..., lo], out[..., hi] = x1 * c - x2 * s, x2 * c + x1 * s
        size[..., lo] = size[..., hi] = x1.abs() + x2.abs()
    return out, size


def check(got, x, pos, *how):
    want, size = reference(x, pos, *how)
    tol = torch.finfo(x.dtype).eps / 2 * want.abs() + ANGLE * size
    assert torch.all((got.double() - want).abs() <= tol)


def make(seed, view, B, L, H, d, dt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def rn(*shape):
        return torch.randn(*shape, device="cuda", generator=g).to(dt)
    if view == "bhld":
        return rn(B, H, L, d).transpose(1, 2)
    if view == "padded":  # heads of a wider row, at an odd offset
        return rn(B, L, H * d + 7)[:, :, 3:3 + H * d].unflatten(2, (H, d))
    if view == "broadcast":  # one sample for all
        return rn(1, L, H, d).expand(B, L, H, d)
    return rn(B, L, H, d)


CASES = [
    # sections, head_dim: the block's own, whole heads, odd widths, one pair, the widest
    ((24, 20, 20), 256), ((24, 20, 20), 128), ((3, 2, 4), 21), ((0, 1, 0), 2), ((1, 0, 6), 14),
    ((16, 24, 24), 136), ((100, 78, 78), 1024), ((5, 5, 6), 40),
]


@pytest.mark.parametrize("sections,d", CASES)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotate(ig4, sections, d, dt, adjacent, interleaved):
    B, L, H, Hk = 2, 37, 5, 2
    q, k = make(1, "blhd", B, L, H, d, DT[dt]), make(2, "bhld", B, L, Hk, d, DT[dt])
    pos = torch.randint(0, 500, (B, 3, L), dtype=torch.int32, device="cuda")
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    for inverse in (False, True):
        ig4.ig4_mrope_rotate(q, k, pos, 5e6, sections, qo, ko, interleaved=interleaved,
                             adjacent=adjacent, inverse=inverse)
        torch.cuda.synchronize()
        check(qo, q, pos, 5e6, sections, interleaved, adjacent, inverse)
        check(ko, k, pos, 5e6, sections, interleaved, adjacent, inverse)
        R = 2 * sum(sections)
        assert torch.equal(qo[..., R:], q[..., R:]) and torch.equal(ko[..., R:], k[..., R:])


@pytest.mark.parametrize("B,L,H", [(1, 1, 1), (8, 1, 18), (1, 4608, 18), (3, 700, 1), (1, 3001, 33)])
@pytest.mark.parametrize("view", ["blhd", "bhld", "padded", "broadcast"])
def test_sizes_and_views(ig4, B, L, H, view):
    q = make(3, view, B, L, H, 256, torch.bfloat16)
    pos = ig4.ig4_mrope_positions(L, 0, 0, 0, device="cuda")
    out = torch.empty(B, L, H, 256, dtype=q.dtype, device="cuda")
    ig4.ig4_mrope_rotate(q, None, pos, 5e6, (24, 20, 20), out, None)
    torch.cuda.synchronize()
    check(out, q, pos, 5e6, (24, 20, 20), False, False, False)


def test_matches_the_rotary_table_of_the_block(ig4):
    """The block's own tables turn a head the same way (both round fp64 angles to fp32)."""
    pos = ig4.ig4_mrope_positions(32, 1, 8, 8, device="cuda")
    L = pos.shape[1]
    c, s = (torch.empty(L, 64, device="cuda") for _ in range(2))
    ig4.ig4_rope_table(pos, 5e6, (24, 20, 20), c, s)
    x = make(4, "blhd", 1, L, 3, 256, torch.float32)
    out = torch.empty_like(x)
    ig4.ig4_mrope_rotate(x, None, pos, 5e6, (24, 20, 20), out, None)
    a, b, c, s = x[..., :64], x[..., 64:128], c[:, None], s[:, None]
    size = a.abs() + b.abs()
    assert torch.all((out[..., :64] - (a * c - b * s)).abs() <= 2 * ANGLE * size)
    assert torch.all((out[..., 64:128] - (b * c + a * s)).abs() <= 2 * ANGLE * size)


def test_far_and_negative_positions(ig4):
    """Positions up to 2^30: 2^-53 relative in the turns is still under 2^-24 of a turn."""
    pos = torch.tensor([0, 1, -1, -77, 2 ** 20 + 1, 2 ** 30 - 3], dtype=torch.int32, device="cuda")
    pos = pos.expand(3, -1).contiguous()
    x = make(5, "blhd", 1, 6, 2, 128, torch.float32)
    out = torch.empty_like(x)
    ig4.ig4_mrope_rotate(x, None, pos, 1e4, (24, 20, 20), out, None)
    torch.cuda.synchronize()
    # 64-bit reference angles are themselves off by 2^-53 * 2^30: add 2e-7
    want, size = reference(x, pos, 1e4, (24, 20, 20), False, False, False)
    assert torch.all((out.double() - want).abs() <= 2.0 ** -24 * want.abs() + (ANGLE + 2e-7) * size)
    assert torch.equal(out[:, 0], x[:, 0])


@pytest.mark.parametrize("adjacent", [False, True])
def test_in_place_on_a_fused_projection_touches_nothing_else(ig4, adjacent):
    B, L, H, Hk, d = 2, 50, 4, 2, 256
    qkv = make(6, "blhd", B, L, H + 2 * Hk, d, torch.bfloat16)
    before = qkv.clone()
    pos = torch.randint(0, 99, (3, L), dtype=torch.int32, device="cuda")
    q, k = qkv[:, :, :H], qkv[:, :, H:H + Hk]
    ig4.ig4_mrope_rotate(q, k, pos, 5e6, (24, 20, 20), q, k, adjacent=adjacent)
    torch.cuda.synchronize()
    check(q, before[:, :, :H], pos, 5e6, (24, 20, 20), False, adjacent, False)
    check(k, before[:, :, H:H + Hk], pos, 5e6, (24, 20, 20), False, adjacent, False)
    assert torch.equal(qkv[:, :, H + Hk:], before[:, :, H + Hk:])
    assert torch.equal(qkv[..., 128:], before[..., 128:])


def test_gradient_is_the_inverse_rotation(ig4):
    """<rotate(v), w> = <v, rotate_back(w)> for the linear map, and back after forth is the
    identity, each up to the roundings of both passes."""
    pos = torch.randint(0, 4000, (3, 129), dtype=torch.int32, device="cuda")
    v, w = (make(s, "blhd", 1, 129, 3, 256, torch.float32) for s in (7, 8))
    rv, rw, back = torch.empty_like(v), torch.empty_like(v), torch.empty_like(v)
    ig4.ig4_mrope_rotate(v, None, pos, 5e6, (24, 20, 20), rv, None, interleaved=True)
    ig4.ig4_mrope_rotate(w, None, pos, 5e6, (24, 20, 20), rw, None, interleaved=True, inverse=True)
    ig4.ig4_mrope_rotate(rv, None, pos, 5e6, (24, 20, 20), back, None, interleaved=True,
                         inverse=True)
    torch.cuda.synchronize()
    a, b = (rv.double() * w.double()), (v.double() * rw.double())
    assert (a.sum() - b.sum()).abs() <= 4 * ANGLE * (a.abs().sum() + b.abs().sum())
    assert torch.all((back - v).abs() <= 4 * ANGLE * (v.abs().max() * 2))


def test_offsets_past_32_bits(ig4):
    """A strided view whose last sample starts past 2^31 elements."""
    L, H, d = 3, 2, 128
    far = (1 << 31) + 4096
    buf = torch.zeros(far + L * H * d, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(buf, (2, L, H, d), (far, H * d, d, 1))
    src = make(9, "blhd", 2, L, H, d, torch.bfloat16)
    x.copy_(src)
    pos = torch.randint(0, 99, (3, L), dtype=torch.int32, device="cuda")
    ig4.ig4_mrope_rotate(x, None, pos, 5e6, (24, 20, 20), x, None)
    torch.cuda.synchronize()
    check(x, src, pos, 5e6, (24, 20, 20), False, False, False)


def test_capture_and_another_stream(ig4):
    q = make(10, "bhld", 2, 333, 4, 256, torch.bfloat16)
    pos = torch.randint(0, 99, (2, 3, 333), dtype=torch.int32, device="cuda")
    out, want = torch.empty_like(q), torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ig4.ig4_mrope_rotate(q, None, pos, 5e6, (24, 20, 20), want, None, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ig4.ig4_mrope_rotate(q, None, pos, 5e6, (24, 20, 20), out, None)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_views_of_one_buffer_interleave(ig4):
    """q into the place of another part of the same rows, k in place beside it."""
    B, L, d = 2, 33, 256
    buf = make(11, "blhd", B, L, 10, d, torch.bfloat16)
    before = buf.clone()
    pos = torch.randint(0, 99, (3, L), dtype=torch.int32, device="cuda")
    q, k, qo = buf[:, :, :4], buf[:, :, 4:6], buf[:, :, 6:]
    ig4.ig4_mrope_rotate(q, k, pos, 5e6, (24, 20, 20), qo, k)
    torch.cuda.synchronize()
    check(qo, before[:, :, :4], pos, 5e6, (24, 20, 20), False, False, False)
    check(k, before[:, :, 4:6], pos, 5e6, (24, 20, 20), False, False, False)
    assert torch.equal(q, before[:, :, :4])


def test_binding_refuses(ig4):
    q = make(12, "blhd", 2, 5, 3, 256, torch.bfloat16)
    out, pos = torch.empty_like(q), torch.zeros(3, 5, dtype=torch.int32, device="cuda")
    sec = (24, 20, 20)
    for args in ((q[0], None, pos, 5e6, sec, out[0], None),
                 (q, None, pos.long(), 5e6, sec, out, None),
                 (q, None, pos[:, :4], 5e6, sec, out, None),
                 (q, None, pos.cpu(), 5e6, sec, out, None),
                 (q, None, pos.t().contiguous().t(), 5e6, sec, out, None),
                 (q, None, pos, 5e6, sec, out.float(), None),
                 (q, None, pos, 5e6, sec, out[:, :4], None),
                 (q.half(), None, pos, 5e6, sec, out.half(), None),
                 (q, q, pos, 5e6, sec, out, None),
                 (q, None, pos, 5e6, sec, q[:, :, :1].expand(2, 5, 3, 256), None),
                 (q, None, pos, 5e6, (24, 20, 200), out, None),
                 (q.transpose(2, 3), None, pos, 5e6, (1, 0, 0), out.transpose(2, 3), None)):
        with pytest.raises(ig4.Ig4Error) as e:
            ig4.ig4_mrope_rotate(*args)
        assert e.value.status == ig4.IG4_ERR_INVALID_ARG
