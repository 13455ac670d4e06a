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


# dh of 90 and 85 tiles on 74 pairs: whole tiles and split ones together, some pairs with a second
# item; the second shape's dG | dU exceeds 64 MiB, where tiles are walked in groups of ten rows of
# them, with a group left over
@pytest.mark.parametrize("M,I,K", [(1153, 512, 4608), (4200, 4096, 1216)])
def test_whole_and_split_tiles_together(ig4, M, I, K):
    t = make(M, I, K)
    check(run(ig4, *t), *reference(*t))


# more weight rows (columns) than 148 CTAs take at once: the few-token products' second item each
@pytest.mark.parametrize("M,I,K", [(17, 19072, 128), (17, 128, 19072), (70, 38016, 64)])
def test_more_weight_rows_than_the_device_takes_at_once(ig4, M, I, K):
    t = make(M, I, K)
    check(run(ig4, *t), *reference(*t))
