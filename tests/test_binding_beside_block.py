"""The binding of the operators beside the block: what it refuses before the library is called, and
the bytes that it hands over.  Nothing here needs a GPU: host tensors stand in for the device's."""

import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def built():
    from stream_diffusion_transformer_fwd_b200.build import build
    build()
    from stream_diffusion_transformer_fwd_b200 import ig4 as m
    return m


@pytest.fixture
def ig4(built, monkeypatch):
    """The binding with host tensors taken for the device's and no library behind it."""
    check = built._device_of
    monkeypatch.setattr(built, "_device_of",
                        lambda where, t: check(where, t) if t is None else t.get_device())
    monkeypatch.setattr(built, "_stream_on", lambda dev, stream: 0)
    for name in ("ig4_add_rms_norm", "ig4_add_rms_norm_backward", "ig4_mrope_rotate",
                 "ig4_nvfp4_matvec", "ig4_nvfp4_swiglu_matvec", "ig4_swiglu_backward"):
        monkeypatch.setattr(built._lib, name, None)
    return built


B16 = torch.bfloat16


def arguments(ig4, name):
    x, h = torch.zeros(4, 256, dtype=B16), torch.zeros(1, 4, 2, 256, dtype=B16)
    codes, scale = torch.zeros(64, 128, dtype=torch.uint8), torch.ones(64)
    sf = torch.zeros(ig4.ig4_nvfp4_scale_bytes(64, 256), dtype=torch.uint8)
    w = torch.zeros(128, 256, dtype=B16)
    return {
        "ig4_add_rms_norm": (x, x, torch.ones(256), 1e-6, x, x),
        "ig4_add_rms_norm_backward": (x, torch.ones(256), 1e-6, x, x, x, None),
        "ig4_mrope_rotate": (h, h, torch.zeros(3, 4, dtype=torch.int32), 5e6, (24, 20, 20), h, h),
        "ig4_nvfp4_matvec": (x, codes, sf, scale, None, torch.empty(4, 64)),
        "ig4_nvfp4_swiglu_matvec": (x, codes, sf, scale, codes, sf, scale,
                                    torch.empty(4, 64, dtype=B16)),
        "ig4_swiglu_backward": (x, w, w, torch.zeros(4, 128, dtype=B16), x, None, None, x),
    }[name]


def refuses(ig4, name, args):
    with pytest.raises(ig4.Ig4Error) as e:
        getattr(ig4, name)(*args)
    assert e.value.status == ig4.IG4_ERR_INVALID_ARG


@pytest.mark.parametrize("name,required", [
    ("ig4_add_rms_norm", (0, 5)), ("ig4_add_rms_norm_backward", (0, 3, 5)),
    ("ig4_mrope_rotate", (0, 1, 2, 3, 4, 5, 6)), ("ig4_nvfp4_matvec", (0, 1, 2, 3, 5)),
    ("ig4_nvfp4_swiglu_matvec", (0, 1, 2, 4, 5)), ("ig4_swiglu_backward", (0, 1))])
def test_a_missing_operand_is_refused(ig4, name, required):
    for i in required:
        args = list(arguments(ig4, name))
        args[i] = None
        refuses(ig4, name, args)


@pytest.mark.parametrize("sections", [(24, 20), (24, 20, 20, 0), (2 ** 40, 20, 20), (24, "20", 20),
                                      64, None])
def test_sections_that_are_not_three_small_numbers(ig4, sections):
    args = list(arguments(ig4, "ig4_mrope_rotate"))
    args[4] = sections
    refuses(ig4, "ig4_mrope_rotate", args)


def test_more_weight_rows_than_an_int(ig4):
    """The library takes an int: 2^32 + 64 rows would arrive as 64."""
    class Rows:
        shape, dtype = torch.Size((2 ** 32 + 64, 128)), torch.uint8
        dim, get_device, is_contiguous, data_ptr = (
            lambda s: 2, lambda s: -1, lambda s: True, lambda s: 1 << 44)

    class Many:
        dtype = torch.uint8
        shape = torch.Size((2 ** 40,))
        numel, get_device, is_contiguous, data_ptr = (
            lambda s: 2 ** 40, lambda s: -1, lambda s: True, lambda s: 1 << 44)

    class Scale(Many):
        shape, dtype = torch.Size((2 ** 32 + 64,)), torch.float32

    class Out(Rows):
        shape, dtype = torch.Size((4, 2 ** 32 + 64)), torch.float32

    args = list(arguments(ig4, "ig4_nvfp4_matvec"))
    args[1:4], args[5] = (Rows(), Many(), Scale()), Out()
    refuses(ig4, "ig4_nvfp4_matvec", args)

def test_packed_structures_are_the_header_s(built):
    """The bytes that ig4_mrope_rotate hands over against the C structures' own layout (which
    test_abi_beside_block.py compares with the header)."""
    rotary = built.Rotary(B=3, L=5, head_dim=7, rotary_dim=11, theta=1.5,
                          sections=(ctypes.c_int * 3)(13, 17, 19), interleaved=23, adjacent=29,
                          inverse=31, dtype=37)
    packed = built._pack_rotary(3, 5, 7, 11, 1.5, 13, 17, 19, 23, 29, 31, 37)
    assert len(packed) == ctypes.sizeof(built.Rotary)
    assert bytes(rotary) == packed
    heads = built.Heads(data=1 << 44, H=3, stride_b=1 << 41, stride_l=5, stride_h=7)
    packed = built._pack_heads(1 << 44, 3, 1 << 41, 5, 7)
    assert bytes(heads) == packed and len(packed) == ctypes.sizeof(built.Heads)


def test_heads_are_packed_from_a_view(ig4):
    buffer = torch.zeros(2, 6, 5, 64, dtype=B16)
    view = buffer.transpose(1, 2)[:, :, 1:4]  # [2, 5, 3, 64]
    got = ig4.Heads.from_buffer_copy(ig4._heads("heads", -1, view, 2, 5, 64, B16))
    assert (got.data, got.H) == (view.data_ptr(), 3)
    assert (got.stride_b, got.stride_l, got.stride_h) == view.stride()[:3]
