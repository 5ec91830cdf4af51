"""The bounded wait of the latent-attention kernels' roles, run by one warp in a kernel of its own."""
import ctypes
import subprocess

import pytest
import torch

import paged_kv_cache_232_gb300 as pa
from paged_kv_cache_232_gb300 import _build

pytestmark = pytest.mark.gpu

SOURCE = r"""
#include "latent_kernel.cuh"

// Lane `late` waits for a barrier that nothing arrives on, the others for one whose phase is complete.
__global__ void wait_kernel(unsigned* err, int* result, int late) {
    __shared__ __align__(8) unsigned long long bars[2];
    const uint32_t done = pa::smem_addr(bars), open = pa::smem_addr(bars + 1);
    if (threadIdx.x == 0) {
        pa::mbar_init(done, 1);
        pa::mbar_init(open, 1);
        pa::fence_barrier_init();
        pa::mbar_arrive(done);
    }
    __syncwarp();
    result[threadIdx.x] = pa::lat::warp_wait((int)threadIdx.x == late ? open : done, 0u, err);
}

extern "C" int run_wait(unsigned* err, int* result, int late) {
    wait_kernel<<<1, 32>>>(err, result, late);
    return (int)cudaGetLastError();
}
"""


@pytest.fixture(scope="module")
def wait_lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("wait")
    src, so = d / "wait.cu", d / "wait.so"
    src.write_text(SOURCE)
    r = subprocess.run([_build._nvcc(), *_build.ARCH, *_build.NVCC_FLAGS, "-shared", "-I", _build.INCLUDE, "-I", _build.CSRC,
                        str(src), "-o", str(so)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    lib = ctypes.CDLL(str(so))
    lib.run_wait.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int]
    return lib


@pytest.mark.parametrize("late", [-1, 0, 13])
def test_a_wait_that_runs_out_is_the_whole_warps(wait_lib, late):
    """One lane's time limit expires while the others' waits are over: every lane gets the same answer (the wait ends
    by its limit, one second)."""
    err = torch.zeros(1, device="cuda", dtype=torch.int32)
    result = torch.full((32,), -1, device="cuda", dtype=torch.int32)
    torch.cuda.synchronize()
    assert wait_lib.run_wait(err.data_ptr(), result.data_ptr(), late) == 0
    torch.cuda.synchronize()
    assert result.tolist() == [1 if late < 0 else 0] * 32
    assert err.item() == (0 if late < 0 else pa.PA_DEVERR_TIMEOUT)
