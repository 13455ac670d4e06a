"""SwiGLU gradients on the paths between the sizes of test_gpu_ffn_grad.py, against the same
formulas in 64 bits with the same tolerances (derived there)."""

import pytest
import torch

from tests.gpu_common import lib
from tests.test_gpu_ffn_grad import check, make, reference, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ig4(cuda_device):
    return lib()


# Warps whose lanes are partly past the last row or the tile's weight rows, over several chunks of
# columns read from tensor memory by the whole warp: up to 128 tokens with 24, 88 and 8 weight rows
# a tile, then ragged tokens in the recomputation and in the split tiles of dh
@pytest.mark.parametrize("M,I,K", [(100, 2816, 192), (128, 12288, 256), (65, 128, 4672),
                                   (131, 384, 192), (290, 640, 704)])
def test_partly_idle_warps(ig4, M, I, K):
    t = make(M, I, K)
    check(run(ig4, *t), *reference(*t))
