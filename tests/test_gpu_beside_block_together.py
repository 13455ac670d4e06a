"""The operators beside the block, run together as a layer would run them.

Each reference is 64-bit arithmetic that rounds to bf16 where the operators
store bf16.  Then only elements whose 64-bit and fp32 values lie on two sides of
a rounding border differ, by one step (2^-7 relative): fp32 errors are under
2^-18 of a value, a border every 2^-8, so at most one element in 2^9, and the
2-norm of the difference is under 2^-7 / sqrt(2^9) = 3.5e-4 of the result's.
Later stages pass such differences on with gains of order one: 2e-3 is asked.
"""

import pytest
import torch

import oracle as O
from tests.gpu_common import lib

pytestmark = pytest.mark.gpu

TOL = 2e-3
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def ig4(cuda_device):
    return lib()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return lambda *shape, dt=BF16, std=1.0: (
        torch.randn(*shape, device="cuda", generator=g) * std).to(dt)


def b16(t):
    return t.to(BF16).double()


def norm64(t, g):
    return t / (t.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * g.double()


def near(got, want):
    rel = ((got.double() - want).norm() / want.norm()).item()
    assert rel <= TOL, rel


@pytest.mark.parametrize("M", [5, 300])
def test_gradients_through_a_feed_forward_layer(ig4, M):
    """s = x + r; y = norm(s); u = swiglu(y); loss = <u, du> + <s, ds>: gradients of x, the norm's
    weight and both projections, eager and from one captured graph."""
    D, I = 512, 1280
    rn = gen(M)
    x, r, g = rn(M, D), rn(M, D), 1 + rn(D, dt=torch.float32, std=0.2)
    wg, wu, du, ds = rn(I, D, std=D ** -0.5), rn(I, D, std=D ** -0.5), rn(M, I), rn(M, D)
    s, y, dy, dx = (torch.empty(M, D, dtype=BF16, device="cuda") for _ in range(4))
    u = torch.empty(M, I, dtype=BF16, device="cuda")
    dwg, dwu, dg = torch.empty_like(wg), torch.empty_like(wu), torch.empty(D, device="cuda")
    ws = torch.empty(ig4.ig4_swiglu_backward_workspace_size(M, I, D), dtype=torch.uint8,
                     device="cuda")
    ws2 = torch.empty(ig4.ig4_add_rms_norm_backward_workspace_size(M, D), dtype=torch.uint8,
                      device="cuda")

    def layer():
        ig4.ig4_add_rms_norm(x, r, g, 1e-6, s, y)
        ig4.ig4_swiglu(M, I, D, y, None, wg, wu, None, None, u)
        ig4.ig4_swiglu_backward(y, wg, wu, du, dy, dwg, dwu, ws)
        ig4.ig4_add_rms_norm_backward(s, g, 1e-6, dy, ds, dx, dg, ws2)
    layer()
    torch.cuda.synchronize()
    assert ig4.ig4_last_device_error() == ig4.IG4_OK

    t = x.double() + r.double()
    y64 = b16(norm64(t, g))
    s64 = b16(t)
    G, U = y64 @ wg.double().T, y64 @ wu.double().T
    sig = torch.sigmoid(G)
    dU, dG = b16(du.double() * G * sig), b16(du.double() * U * sig * (1 + G * (1 - sig)))
    dy64 = b16(dG @ wg.double() + dU @ wu.double())
    rstd = 1 / (s64.pow(2).mean(1, keepdim=True) + 1e-6).sqrt()
    n, dn = s64 * rstd, dy64 * g.double()
    near(y, y64)
    near(u, b16(G * sig * U))
    near(dwg, b16(dG.T @ y64))
    near(dwu, b16(dU.T @ y64))
    near(dy, dy64)
    near(dx, rstd * (dn - n * (dn * n).mean(1, keepdim=True)) + ds.double())
    near(dg, (dy64 * n).sum(0))

    graph = torch.cuda.CUDAGraph()
    outs = (s, y, u, dy, dwg, dwu, dx, dg)
    want = [o.clone() for o in outs]
    with torch.cuda.graph(graph):
        layer()
    for o in outs:
        o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs))


@pytest.mark.parametrize("M", [1, 8])
def test_single_tokens_through_a_4_bit_feed_forward_layer(ig4, M):
    """norm -> gated 4-bit projections -> 4-bit down projection -> residual addition and norm."""
    D, I = 1024, 2816
    rn = gen(40 + M)
    g = torch.Generator(device="cuda")
    g.manual_seed(M)

    def weights(N, K):
        codes = torch.randint(0, 256, (N, K // 2), device="cuda", generator=g, dtype=torch.uint8)
        sf = torch.randint(40, 72, (N, K // 16), device="cuda", generator=g, dtype=torch.uint8)
        scale = (torch.rand(N, device="cuda", generator=g) + 0.5) * K ** -0.5 / 3
        packed = torch.empty(ig4.ig4_nvfp4_scale_bytes(N, K), dtype=torch.uint8, device="cuda")
        ig4.ig4_nvfp4_pack_scales(sf, packed)
        ref = torch.from_numpy(O.dequant_nvfp4(codes.cpu().numpy(), sf.cpu().numpy(),
                                               scale.cpu().numpy())).cuda()
        return (codes, packed, scale), ref
    (gate, gate64), (up, up64), (down, down64) = weights(I, D), weights(I, D), weights(D, I)
    x, r = rn(M, D), rn(M, D)
    g1, g2 = (1 + rn(D, dt=torch.float32, std=0.2) for _ in range(2))
    s, y, h, s2, y2 = (torch.empty(M, D, dtype=BF16, device="cuda") for _ in range(5))
    u = torch.empty(M, I, dtype=BF16, device="cuda")
    ig4.ig4_add_rms_norm(x, r, g1, 1e-6, s, y)
    ig4.ig4_nvfp4_swiglu_matvec(y, *gate, *up, u)
    ig4.ig4_nvfp4_matvec(u, *down, None, h)
    ig4.ig4_add_rms_norm(s, h, g2, 1e-6, s2, y2)
    torch.cuda.synchronize()
    assert ig4.ig4_last_device_error() == ig4.IG4_OK
    t = x.double() + r.double()
    y64 = b16(norm64(t, g1))
    G, U = y64 @ gate64.T, y64 @ up64.T
    u64 = b16(G * torch.sigmoid(G) * U)
    h64 = b16(u64 @ down64.T)
    t2 = b16(t) + h64
    for got, want in ((y, y64), (u, u64), (h, h64), (s2, b16(t2)), (y2, b16(norm64(t2, g2)))):
        near(got, want)


def test_rotated_heads_into_the_joint_attention(ig4):
    """q and k of a fused projection, normed elsewhere, rotated in place in the attention's own
    layout, against attention over heads rotated in 64 bits."""
    B, H, L, T, side = 1, 2, 164, 20, 12
    rn = gen(77)
    q, k = rn(B, H, L, 256), rn(B, H, L, 256)
    vt = torch.zeros(B, H, 256, 168, dtype=BF16, device="cuda")
    vt[..., :L] = rn(B, H, 256, L)
    pos = ig4.ig4_mrope_positions(T, 1, side, side, device="cuda")
    want = []
    for x in (q, k):
        out = x.double().clone()
        axes = [0] * 24 + [1] * 20 + [2] * 20
        for j, a in enumerate(axes):
            ang = pos[a].double() * 5e6 ** (-j / 64)
            c, s = ang.cos(), ang.sin()
            lo, hi = x[..., j].double(), x[..., j + 64].double()
            out[..., j], out[..., j + 64] = lo * c - hi * s, hi * c + lo * s
        want.append(b16(out))
    ig4.ig4_mrope_rotate(q.transpose(1, 2), k.transpose(1, 2), pos, 5e6, (24, 20, 20),
                         q.transpose(1, 2), k.transpose(1, 2))
    o = torch.empty(B * L, H * 256, dtype=BF16, device="cuda")
    ig4.ig4_joint_attention(B, H, L, q, k, vt, 168, o)
    torch.cuda.synchronize()
    assert ig4.ig4_last_device_error() == ig4.IG4_OK
    near(q, want[0])
    near(k, want[1])
    p = torch.softmax(want[0] @ want[1].transpose(-1, -2) / 16, -1)
    ref = (p @ vt[..., :L].double().transpose(-1, -2)).transpose(1, 2).reshape(B * L, H * 256)
    # the attention itself rounds its probabilities and its output to bf16: 2.3e-3 each
    rel = ((o.double() - ref).norm() / ref.norm()).item()
    assert rel <= TOL + 2 * 2.3e-3, rel
