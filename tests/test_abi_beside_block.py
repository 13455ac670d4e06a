"""Argument checks of the operators beside the block, on the host: each refusal
returns before anything is launched, so none of this needs a GPU.  Addresses
are made up; nothing reads them."""

import ctypes
import os
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F32, BF16, E4M3 = 0, 1, 2


@pytest.fixture(scope="module")
def ig4():
    from stream_diffusion_transformer_fwd_b200.build import build
    build()
    from stream_diffusion_transformer_fwd_b200 import ig4 as m
    return m


def at(i, off=0):
    """The i-th of a row of made-up buffers, 4 GiB apart."""
    return ctypes.c_void_p((1 << 44) + (i << 32) + off)


def test_struct_layouts_match_header(ig4, tmp_path):
    src = tmp_path / "layout.c"
    src.write_text(
        '#include <stddef.h>\n#include <stdio.h>\n#include "ig4.h"\n'
        'int main(void) { printf("%zu %zu %zu %zu %zu %zu\\n", sizeof(ig4_rotary),'
        ' offsetof(ig4_rotary, theta), offsetof(ig4_rotary, dtype), sizeof(ig4_heads),'
        ' offsetof(ig4_heads, H), offsetof(ig4_heads, stride_h)); return 0; }\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    R, H = ig4.Rotary, ig4.Heads
    assert [int(v) for v in got] == [ctypes.sizeof(R), R.theta.offset, R.dtype.offset,
                                     ctypes.sizeof(H), H.H.offset, H.stride_h.offset]


# ------------------------------------------------------------ add + RMSNorm

def norm(ig4, M=4, D=256, x=at(0), r=at(1), xd=BF16, g=at(2), eps=1e-6, s=at(3), y=at(4), yd=BF16,
         sc=None, sf=None):
    return ig4.library().ig4_add_rms_norm(M, D, x, r, xd, g, eps, s, y, yd, sc, sf, None)


@pytest.mark.parametrize("bad", [
    dict(M=0), dict(M=-1), dict(D=0), dict(D=12), dict(D=8200), dict(x=None), dict(y=None),
    dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(xd=E4M3), dict(xd=3), dict(yd=3),
    dict(x=at(0, 8)), dict(r=at(1, 2)), dict(g=at(2, 4)), dict(s=at(3, 8)), dict(y=at(4, 8)),
    dict(sc=at(5)),                                     # a scale for a bf16 output
    dict(yd=E4M3),                                      # no scale form chosen
    dict(yd=E4M3, sc=at(5), sf=at(6)),                  # both
    dict(yd=E4M3, sf=at(6), D=264),                     # block scales need D % 128 == 0
    dict(yd=E4M3, sc=at(5, 2)), dict(yd=E4M3, sf=at(6, 2)),
    dict(s=at(0, 16)), dict(s=at(1, 512)),              # overlaps x or r but is neither
    dict(y=at(0)), dict(y=at(1)), dict(y=at(2)), dict(y=at(3)), dict(y=at(3, 2032)),
    dict(yd=E4M3, sc=at(4)), dict(yd=E4M3, sf=at(0, 64)), dict(s=at(2))])
def test_add_rms_norm_refuses(ig4, bad):
    assert norm(ig4, **bad) == ig4.IG4_ERR_INVALID_ARG


def grad(ig4, M=4, D=256, s=at(0), sd=BF16, g=at(1), eps=1e-6, dy=at(2), dyd=BF16, ds=at(3),
         dx=at(4), dg=at(5), ws=at(6), nbytes=1 << 24):
    return ig4.library().ig4_add_rms_norm_backward(M, D, s, sd, g, eps, dy, dyd, ds, dx, dg, ws,
                                                   nbytes, None)


@pytest.mark.parametrize("bad", [
    dict(M=0), dict(D=4), dict(D=8200), dict(s=None), dict(dy=None), dict(dx=None), dict(eps=0.0),
    dict(sd=E4M3), dict(dyd=E4M3), dict(s=at(0, 8)), dict(g=at(1, 8)), dict(dy=at(2, 8)),
    dict(ds=at(3, 8)), dict(dx=at(4, 8)), dict(dg=at(5, 2)), dict(dx=at(0)), dict(dx=at(2)),
    dict(dx=at(3, 16)), dict(dg=at(1)), dict(dg=at(4, 64)), dict(ws=at(0)), dict(ws=at(4, 256))])
def test_add_rms_norm_backward_refuses(ig4, bad):
    assert grad(ig4, **bad) == ig4.IG4_ERR_INVALID_ARG


def test_add_rms_norm_backward_workspace(ig4):
    need = ig4.ig4_add_rms_norm_backward_workspace_size(4, 256)
    assert need > 0 and need % 256 == 0
    assert grad(ig4, nbytes=need - 1) == ig4.IG4_ERR_WORKSPACE
    assert grad(ig4, ws=None) == ig4.IG4_ERR_WORKSPACE
    assert grad(ig4, ws=at(6, 128)) == ig4.IG4_ERR_WORKSPACE
    for M, D in ((0, 256), (4, 12), (4, 8200), (-3, 8)):
        assert ig4.ig4_add_rms_norm_backward_workspace_size(M, D) == 0


# ------------------------------------------------------------------- rotary

def rotate(ig4, q=None, qo=None, k=None, ko=None, pos=at(9), pos_stride=0, **kw):
    rot = dict(B=2, L=16, head_dim=256, rotary_dim=128, theta=5e6, sections=(24, 20, 20),
               interleaved=0, adjacent=0, inverse=0, dtype=BF16)
    rot.update(kw)
    rot["sections"] = (ctypes.c_int * 3)(*rot["sections"])
    q = q or (at(0), 4, 16 * 1024, 1024, 256)
    qo = qo or (at(1), 4, 16 * 1024, 1024, 256)
    views = [None if v is None else ig4.Heads(v[0], *v[1:]) for v in (q, qo, k, ko)]
    return ig4.library().ig4_mrope_rotate(
        ctypes.byref(ig4.Rotary(**rot)), pos, pos_stride,
        *(None if v is None else ctypes.byref(v) for v in views), None)


QK = (at(2), 2, 16 * 512, 512, 256)


@pytest.mark.parametrize("bad", [
    dict(B=0), dict(L=0), dict(B=1 << 16, L=1 << 15), dict(head_dim=1), dict(head_dim=1026),
    dict(rotary_dim=0), dict(rotary_dim=127), dict(head_dim=64), dict(rotary_dim=126),
    dict(sections=(24, 20, 21)), dict(sections=(-1, 45, 20)), dict(theta=0.0),
    dict(theta=float("inf")), dict(theta=float("nan")), dict(dtype=E4M3), dict(pos=None),
    dict(pos=at(9, 2)), dict(pos_stride=-1),
    dict(head_dim=1024, rotary_dim=514, sections=(257, 0, 0)),
    dict(q=(None, 4, 16 * 1024, 1024, 256)), dict(q=(at(0), 0, 16 * 1024, 1024, 256)),
    dict(q=(at(0, 1), 4, 16 * 1024, 1024, 256)), dict(q=(at(0), 4, -1, 1024, 256)),
    dict(qo=(at(1), 5, 16 * 1024, 1024, 256)),          # another number of heads
    dict(qo=(at(1), 4, 0, 1024, 256)),                  # samples on top of one another
    dict(qo=(at(1), 4, 16 * 1024, 1024, 128)),          # heads that overlap
    dict(qo=(at(0), 4, 16 * 2048, 2048, 256)),          # in place with other strides
    dict(k=QK), dict(ko=QK),                            # one of k and its output
    dict(k=QK, ko=(at(1), 2, 16 * 512, 512, 256))])     # q's and k's output the same
def test_mrope_rotate_refuses(ig4, bad):
    assert rotate(ig4, **bad) == ig4.IG4_ERR_INVALID_ARG


# ------------------------------------------------------------ SwiGLU gradients

def swiglu(ig4, M=8, I=256, K=128, h=at(0), wg=at(1), wu=at(2), du=at(3), dh=at(4), dwg=at(5),
           dwu=at(6), ws=at(7), nbytes=1 << 30):
    return ig4.library().ig4_swiglu_backward(M, I, K, h, wg, wu, du, dh, dwg, dwu, ws, nbytes, None)


@pytest.mark.parametrize("bad", [
    dict(M=0), dict(I=0), dict(K=-64), dict(h=None), dict(wg=None), dict(wu=None), dict(du=None),
    dict(dwg=None), dict(dwu=None), dict(dh=None, dwg=None, dwu=None), dict(h=at(0, 8)),
    dict(wg=at(1, 8)), dict(wu=at(2, 8)), dict(du=at(3, 8)), dict(dh=at(4, 8)), dict(dwg=at(5, 8)),
    dict(dwu=at(6, 8)), dict(dh=at(0)), dict(dwg=at(1)), dict(dwu=at(5)), dict(dh=at(3, 16)),
    dict(ws=at(1)), dict(ws=at(4, 256))])
def test_swiglu_backward_refuses(ig4, bad):
    assert swiglu(ig4, **bad) == ig4.IG4_ERR_INVALID_ARG


def test_swiglu_backward_sizes_and_workspace(ig4):
    for bad in (dict(I=192), dict(K=96), dict(M=(1 << 20) + 1), dict(K=1 << 18)):
        assert swiglu(ig4, **bad) == ig4.IG4_ERR_UNSUPPORTED
    need = ig4.ig4_swiglu_backward_workspace_size(8, 256, 128)
    assert need >= 8 * 512 * 2 and need % 256 == 0
    assert swiglu(ig4, nbytes=need - 1) == ig4.IG4_ERR_WORKSPACE
    assert swiglu(ig4, ws=None) == ig4.IG4_ERR_WORKSPACE
    assert swiglu(ig4, ws=at(7, 128)) == ig4.IG4_ERR_WORKSPACE
    for sizes in ((0, 256, 128), (8, 100, 128), (8, 256, 32)):
        assert ig4.ig4_swiglu_backward_workspace_size(*sizes) == 0


# ------------------------------------------------------ few rows x NVFP4 weights

def matvec(ig4, M=2, N=256, K=128, x=at(0), c=at(1), sf=at(2), sc=at(3), b=at(4), out=at(5),
           od=BF16):
    return ig4.library().ig4_nvfp4_matvec(M, N, K, x, c, sf, sc, b, out, od, None)


@pytest.mark.parametrize("bad", [
    dict(M=0), dict(M=9), dict(N=0), dict(K=0), dict(K=96), dict(K=24640), dict(x=None),
    dict(c=None), dict(sf=None), dict(sc=None), dict(out=None), dict(od=E4M3), dict(x=at(0, 8)),
    dict(c=at(1, 8)), dict(sf=at(2, 8)), dict(sc=at(3, 2)), dict(b=at(4, 2)), dict(out=at(5, 1)),
    dict(out=at(5, 2), od=F32), dict(out=at(0)), dict(out=at(1, 64)), dict(out=at(2)),
    dict(out=at(3)), dict(out=at(4))])
def test_nvfp4_matvec_refuses(ig4, bad):
    assert matvec(ig4, **bad) == ig4.IG4_ERR_INVALID_ARG


def gated(ig4, M=2, I=256, K=128, x=at(0), gc=at(1), gs=at(2), gf=at(3), uc=at(4), us=at(5),
          uf=at(6), out=at(7)):
    return ig4.library().ig4_nvfp4_swiglu_matvec(M, I, K, x, gc, gs, gf, uc, us, uf, out, None)


@pytest.mark.parametrize("bad", [
    dict(M=0), dict(M=9), dict(I=0), dict(K=32), dict(x=None), dict(gc=None), dict(gs=None),
    dict(gf=None), dict(uc=None), dict(us=None), dict(uf=None), dict(out=None), dict(uc=at(4, 8)),
    dict(us=at(5, 8)), dict(uf=at(6, 2)), dict(out=at(7, 1)), dict(out=at(4)), dict(out=at(6))])
def test_nvfp4_swiglu_matvec_refuses(ig4, bad):
    assert gated(ig4, **bad) == ig4.IG4_ERR_INVALID_ARG


# ------------------------------------------------------------------- binding

def test_binding_refuses_host_tensors(ig4):
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    h = torch.zeros(1, 4, 2, 256, dtype=torch.bfloat16)
    calls = [lambda: ig4.ig4_add_rms_norm(x, None, None, 1e-6, None, x),
             lambda: ig4.ig4_add_rms_norm_backward(x, None, 1e-6, x, None, x, None),
             lambda: ig4.ig4_mrope_rotate(h, None, torch.zeros(3, 4, dtype=torch.int32), 5e6,
                                          (24, 20, 20), h, None),
             lambda: ig4.ig4_swiglu_backward(x, x, x, x, x, None, None, x)]
    for call in calls:
        with pytest.raises(ig4.Ig4Error) as e:
            call()
        assert e.value.status == ig4.IG4_ERR_INVALID_ARG


# ------------------------------------------------- outputs on other operands

PACKED = 10 * 256                                        # a row of 10 heads: q 0-3, k 4-5, v 6-9


def packed(buffer, head, H, l=PACKED):
    return at(buffer, head * 512), H, 16 * l, l, 256


@pytest.mark.parametrize("bad", [
    dict(q=packed(0, 0, 4), qo=packed(0, 2, 4)),         # its own heads, shifted by two
    dict(q=packed(0, 0, 4), qo=packed(0, 0, 4)[:1] + (4, 16 * 1024, 1024, 256)),
    dict(q=packed(0, 0, 4), qo=packed(0, 10, 4)),        # shifted by a token
    dict(q=packed(0, 0, 4), qo=(at(0, 20 * 256 * 15), 4, 16 * 1024, 1024, 256)),
    dict(q=packed(0, 0, 4), qo=packed(1, 0, 4), k=packed(0, 4, 2), ko=packed(0, 3, 2)),
    dict(q=packed(0, 0, 4), qo=packed(1, 0, 4), k=packed(0, 4, 2), ko=packed(1, 3, 2)),
    dict(q=packed(0, 0, 4), qo=packed(0, 4, 4), k=packed(0, 4, 2), ko=packed(1, 0, 2)),
    dict(qo=(at(9, -4 * 1024), 4, 16 * 1024, 1024, 256)),             # the positions
    dict(q=(at(0), 4, 1 << 39, 1 << 39, 1 << 39), B=1 << 15, L=1 << 15)])
def test_mrope_rotate_refuses_outputs_on_other_operands(ig4, bad):
    assert rotate(ig4, **bad) == ig4.IG4_ERR_INVALID_ARG


def test_norms_refuse_an_infinite_eps(ig4):
    for call in (norm, grad):
        assert call(ig4, eps=float("inf")) == ig4.IG4_ERR_INVALID_ARG


@pytest.mark.parametrize("rows", [2 ** 31, 2 ** 32 + 4])
def test_binding_refuses_more_rows_than_an_int(ig4, monkeypatch, rows):
    class Rows:
        is_cuda, shape, dtype = True, (rows, 8), torch.bfloat16
        get_device, numel, is_contiguous, data_ptr = (
            lambda s: 0, lambda s: rows * 8, lambda s: True, lambda s: 1 << 44)

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(ig4, "_stream_on", lambda dev, stream: 0)
    monkeypatch.setattr(ig4._lib, "ig4_add_rms_norm", None)   # the library is not reached
    monkeypatch.setattr(ig4._lib, "ig4_add_rms_norm_backward", None)
    x = Rows()
    for call in (lambda: ig4.ig4_add_rms_norm(x, None, None, 1e-6, None, x),
                 lambda: ig4.ig4_add_rms_norm_backward(x, None, 1e-6, x, None, x, None)):
        with pytest.raises(ig4.Ig4Error) as e:
            call()
        assert e.value.status == ig4.IG4_ERR_INVALID_ARG
