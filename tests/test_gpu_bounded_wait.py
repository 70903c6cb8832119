"""A warp's wait on a barrier has one outcome for all its lanes, also where the limit runs out for some of them only."""
import ctypes
import subprocess

import pytest
import torch

pytestmark = pytest.mark.gpu

# Warp 0 waits, lane l for (100 + 20 l) ms; warp 1 arrives once `arrive` ns have passed (0: never).
SOURCE = r"""
#include "gda_device.cuh"
__global__ void wait_kernel(int *got, unsigned long long arrive) {
    __shared__ __align__(8) uint64_t bar;
    if (threadIdx.x == 0) {
        gda::mbar_init(&bar, 1);
        gda::fence_mbar_init();
    }
    __syncthreads();
    const uint64_t t0 = gda::global_timer_ns();
    if (threadIdx.x < 32) {
        got[threadIdx.x] = gda::mbar_wait_warp(gda::smem_u32(&bar), 0, (100 + 20 * threadIdx.x) * 1000000ull);
    } else if (threadIdx.x == 32 && arrive > 0) {
        while (gda::global_timer_ns() - t0 < arrive) __nanosleep(1000);
        gda::mbar_arrive(&bar);
    }
}
extern "C" int run_wait(int *got, unsigned long long arrive, cudaStream_t stream) {
    wait_kernel<<<1, 64, 0, stream>>>(got, arrive);
    return static_cast<int>(cudaGetLastError());
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    from grouped_differential_attention_gb300 import build
    build.build()
    at = tmp_path_factory.mktemp("wait")
    (at / "wait.cu").write_text(SOURCE)
    subprocess.run([build.nvcc_path(), "-shared", "-o", str(at / "wait.so"), str(at / "wait.cu"), *build.compile_flags()],
                   check=True)
    lib = ctypes.CDLL(str(at / "wait.so"))
    lib.run_wait.argtypes = [ctypes.c_void_p, ctypes.c_ulonglong, ctypes.c_void_p]
    return lib


@pytest.mark.parametrize("arrive_ms,want", [
    (1, 1), (50, 1),                       # in time for all
    (400, 0), (600, 0),                    # after some lanes' limit: none may go on
    (0, 0),                                # never
])
def test_one_outcome_for_the_warp(lib, arrive_ms, want):
    got = torch.full((32,), -1, dtype=torch.int32, device="cuda")
    assert lib.run_wait(got.data_ptr(), arrive_ms * 1000000, torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert got.tolist() == [want] * 32
