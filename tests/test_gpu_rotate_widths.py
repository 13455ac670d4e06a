"""Head widths whose elements past the rotary ones do not split into equal runs of a CTA's threads
(primes above 256, alone or with the vectors that alignment leaves), with the tolerances of
test_gpu_rotate.py; what is not rotated arrives bit by bit, and nothing is written beside a head."""

import pytest
import torch

from tests.gpu_common import lib
from tests.test_gpu_rotate import check, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ig4(cuda_device):
    return lib()


@pytest.mark.parametrize("sections,d", [((2, 1, 1), 265), ((1, 0, 0), 1021), ((1, 0, 0), 771),
                                        ((3, 0, 0), 1024), ((2, 1, 1), 522), ((2, 1, 1), 1012),
                                        ((1, 1, 1), 1024)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("B,L,H", [(1, 1, 1), (2, 37, 5), (1, 1500, 3)])
def test_rest_of_any_length(ig4, sections, d, dt, adjacent, B, L, H):
    q = make(d, "blhd", B, L, H, d, dt)
    pos = torch.randint(0, 500, (B, 3, L), dtype=torch.int32, device="cuda")
    room = torch.full((B, L, H, d + 16), 7.0, dtype=dt, device="cuda")
    out = room[..., 8:8 + d]
    ig4.ig4_mrope_rotate(q, None, pos, 5e6, sections, out, None, adjacent=adjacent)
    torch.cuda.synchronize()
    check(out, q, pos, 5e6, sections, False, adjacent, False)
    R = 2 * sum(sections)
    assert torch.equal(out[..., R:], q[..., R:])
    assert torch.all(room[..., :8] == 7) and torch.all(room[..., 8 + d:] == 7)
