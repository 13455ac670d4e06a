"""SwiGLU gradients against the formulas in 64 bits on the same bf16 inputs.

Roundings: dG and dU once to bf16 (at most 2^-8 relative) in front of the
products, the results once more; G and U carry fp32 sums of K terms, which
move dG and dU by far less.  Element by element the products' error is at most
2^-8 of the sum of the terms' absolute values (2^-10 of it added for the fp32
parts).  Over a whole matrix the roundings are independent: each has a root
mean square of at most 2^-8 / sqrt(3) = 2.3e-3 relative, so dh and dW, with two
of them, stay under 4.5e-3 in the 2-norm.
"""

import pytest
import torch

from tests.gpu_common import lib

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8


@pytest.fixture(scope="module")
def ig4(cuda_device):
    return lib()


def make(M, I, K, seed=0, gain=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + M + 7 * I + 13 * K)

    def rn(*shape, std=1.0):
        return (torch.randn(*shape, device="cuda", generator=g) * std).to(torch.bfloat16)
    return rn(M, K, std=gain), rn(I, K, std=K ** -0.5), rn(I, K, std=K ** -0.5), rn(M, I, std=0.3)


def reference(h, wg, wu, du):
    h, wg, wu, du = (t.double() for t in (h, wg, wu, du))
    G, U = h @ wg.T, h @ wu.T
    sig = torch.sigmoid(G)
    dU, dG = du * G * sig, du * U * sig * (1 + G * (1 - sig))
    want = (dG @ wg + dU @ wu, dG.T @ h, dU.T @ h)
    size = (dG.abs() @ wg.abs() + dU.abs() @ wu.abs(), dG.abs().T @ h.abs(), dU.abs().T @ h.abs())
    return want, size


def run(ig4, h, wg, wu, du, dh=True, dw=True):
    (M, K), I = h.shape, wg.shape[0]
    ws = torch.empty(ig4.ig4_swiglu_backward_workspace_size(M, I, K), dtype=torch.uint8,
                     device="cuda")
    out = [torch.full_like(h, float("nan")) if dh else None,
           torch.full_like(wg, float("nan")) if dw else None,
           torch.full_like(wu, float("nan")) if dw else None]
    ig4.ig4_swiglu_backward(h, wg, wu, du, *out, ws)
    torch.cuda.synchronize()
    assert ig4.ig4_last_device_error() == ig4.IG4_OK
    return out


def check(got, want, size):
    for g, w, s in zip(got, want, size):
        if g is None:
            continue
        err = (g.double() - w).abs()
        rel = (err.norm() / w.norm()).item()
        print(f"rel {rel:.2e}")
        assert torch.all(err <= HALF * w.abs() + (HALF + 2.0 ** -10) * s)
        assert rel <= 4.5e-3


# one token; ragged rows on both sides of the one-CTA and pair forms of the recomputation; widths
# that end inside a 256-wide tile; contraction shares of every count the rule gives
@pytest.mark.parametrize("M,I,K", [(1, 128, 64), (1, 2816, 1024), (17, 256, 192), (96, 2816, 1024),
                                   (127, 640, 320), (128, 128, 4608), (129, 384, 448),
                                   (255, 1152, 512), (257, 256, 64), (300, 12288, 576),
                                   (1153, 1408, 1088), (2500, 512, 1600)])
def test_swiglu_backward(ig4, M, I, K):
    t = make(M, I, K)
    check(run(ig4, *t), *reference(*t))


@pytest.mark.parametrize("dh,dw", [(True, False), (False, True)])
def test_only_what_is_wanted(ig4, dh, dw):
    t = make(200, 384, 256)
    full = run(ig4, *t)
    part = run(ig4, *t, dh=dh, dw=dw)
    for a, b in zip(full, part):
        assert b is None or torch.equal(a, b)


def test_saturated_gates(ig4):
    """Gates far out on both sides: sig(G) 0 or 1, no overflow in its exponential."""
    h, wg, wu, du = make(140, 256, 128, gain=200.0)
    got = run(ig4, h, wg, wu, du)
    check(got, *reference(h, wg, wu, du))


def test_zero_gradient_gives_zero(ig4):
    h, wg, wu, du = make(33, 256, 128)
    for g in run(ig4, h, wg, wu, torch.zeros_like(du)):
        assert torch.all(g == 0)


def test_gradient_against_differences(ig4):
    """<dh, v> + <dWg, a> + <dWu, b> against central differences of the loss in 64 bits."""
    h, wg, wu, du = make(40, 256, 192)
    got = run(ig4, h, wg, wu, du)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    v = [torch.randn(t.shape, device="cuda", generator=g, dtype=torch.float64) for t in (h, wg, wu)]

    def loss(e):
        a, b, c = (t.double() + e * d for t, d in zip((h, wg, wu), v))
        G, U = a @ b.T, a @ c.T
        return (G * torch.sigmoid(G) * U * du.double()).sum()
    step = 1e-5
    want = (loss(step) - loss(-step)) / (2 * step)
    terms = [x.double() * d for x, d in zip(got, v)]
    # independent errors of 4.5e-3 at most: relative to the root of the sum of squares, five
    # standard deviations
    spread = sum(t.pow(2).sum() for t in terms).sqrt()
    assert (sum(t.sum() for t in terms) - want).abs() <= 5 * 4.5e-3 * spread


def test_same_bits_again_captured_and_on_another_stream(ig4):
    h, wg, wu, du = make(300, 1152, 640)
    want = run(ig4, h, wg, wu, du)
    ws = torch.empty(ig4.ig4_swiglu_backward_workspace_size(300, 1152, 640), dtype=torch.uint8,
                     device="cuda")
    out = [torch.empty_like(t) for t in want]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ig4.ig4_swiglu_backward(h, wg, wu, du, *out, ws, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, out))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ig4.ig4_swiglu_backward(h, wg, wu, du, *out, ws)
    for t in out:
        t.zero_()
    ws.fill_(255)  # nothing of the workspace has to start at zero
    graph.replay()
    torch.cuda.synchronize()
    assert ig4.ig4_last_device_error() == ig4.IG4_OK
    assert all(torch.equal(a, b) for a, b in zip(want, out))


def test_binding_refuses(ig4):
    h, wg, wu, du = make(8, 256, 128)
    ws = torch.empty(ig4.ig4_swiglu_backward_workspace_size(8, 256, 128), dtype=torch.uint8,
                     device="cuda")
    dh, dg, du_w = torch.empty_like(h), torch.empty_like(wg), torch.empty_like(wu)
    good = [h, wg, wu, du, dh, dg, du_w, ws]
    for i, bad in ((0, h.float()), (0, h[:, :64]), (1, wg[:128]), (2, wu.t()), (2, wu.half()),
                   (3, du[:4]), (3, du.float()), (4, dh[:, ::2]), (4, h), (5, dg.float()), (5, None),
                   (6, du_w.cpu()), (6, dg), (7, ws[::2])):
        with pytest.raises(ig4.Ig4Error) as e:
            ig4.ig4_swiglu_backward(*good[:i], bad, *good[i + 1:])
        assert e.value.status == ig4.IG4_ERR_INVALID_ARG
    for bad in (None, ws[:-1]):
        with pytest.raises(ig4.Ig4Error) as e:
            ig4.ig4_swiglu_backward(*good[:7], bad)
        assert e.value.status == ig4.IG4_ERR_WORKSPACE
