"""Calls from threads other than the one that set things up."""

import threading

import pytest
import torch

from tests.gpu_common import lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ig4(cuda_device):
    return lib()


def norm(ig4, M):
    x, y, st = torch.ones(M, 8192, device="cuda"), torch.empty(M, 8192, device="cuda"), torch.cuda.Stream()
    return lambda: ig4.ig4_add_rms_norm(x, x, None, 1e-6, None, y, stream=st)


def norm_backward(ig4, M):
    x, y, st = torch.ones(M, 8192, device="cuda"), torch.empty(M, 8192, device="cuda"), torch.cuda.Stream()
    return lambda: ig4.ig4_add_rms_norm_backward(x, None, 1e-6, x, x, y, None, stream=st)


def swiglu_backward(ig4, M, I=128, K=1024):
    h, wg, wu, du, dh = (torch.ones(*s, dtype=torch.bfloat16, device="cuda")
                         for s in ((M, K), (I, K), (I, K), (M, I), (M, K)))
    ws = torch.empty(ig4.ig4_swiglu_backward_workspace_size(M, I, K), dtype=torch.uint8,
                     device="cuda")
    st = torch.cuda.Stream()
    return lambda: ig4.ig4_swiglu_backward(h, wg, wu, du, dh, None, None, ws, stream=st)


def matvec(ig4, M, N=256, K=512):
    x, out = torch.ones(M, K, dtype=torch.bfloat16, device="cuda"), torch.empty(M, N, device="cuda")
    codes = torch.zeros(N, K // 2, dtype=torch.uint8, device="cuda")
    sf = torch.zeros(ig4.ig4_nvfp4_scale_bytes(N, K), dtype=torch.uint8, device="cuda")
    scale, st = torch.ones(N, device="cuda"), torch.cuda.Stream()
    return lambda: ig4.ig4_nvfp4_matvec(x, codes, sf, scale, None, out, stream=st)


def rotate(ig4, L):
    q, st = torch.ones(1, L, 2, 128, device="cuda"), torch.cuda.Stream()
    pos = torch.zeros(3, L, dtype=torch.int32, device="cuda")
    return lambda: ig4.ig4_mrope_rotate(q, None, pos, 5e6, (24, 20, 20), q, None, stream=st)


def run_in_threads(ig4, calls, times):
    failed = []

    def work(call):
        for i in range(times):
            try:
                call()
            except ig4.Ig4Error as e:
                failed.append(e.status)
            if i % 256 == 255:
                torch.cuda.synchronize()

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert ig4.ig4_last_device_error() == ig4.IG4_OK
    assert failed == []


@pytest.mark.parametrize("make,M", [(norm, 3), (norm_backward, 3), (swiglu_backward, 3),
                                    (swiglu_backward, 200), (matvec, 3), (rotate, 3)])
def test_the_first_call_of_a_thread(ig4, make, M):
    run_in_threads(ig4, [make(ig4, M)], 1)


@pytest.mark.parametrize("make,sizes", [(norm, (1, 500)), (norm_backward, (1, 500)),
                                        (swiglu_backward, (17, 128))])
def test_two_threads_with_sizes_of_different_shared_memory(ig4, make, sizes):
    run_in_threads(ig4, [make(ig4, M) for M in sizes], 8000)
