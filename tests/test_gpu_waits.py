"""The bounded wait of a whole warp (kvc_tc.cuh) whose lanes would come to different answers: half of them wait for
barriers that are complete, the others for some that nothing completes, with the flag that ends waits set before."""
import ctypes
import os
import subprocess

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = r"""
#include <cuda.h>
#include <type_traits>
#include "kvc_common.cuh"
#include "kvc_tc.cuh"

// out[0 .. 31] the lanes' answers alone, [32 .. 63] the warp's, [64 .. 95] the warp's where all are complete
__global__ void waits(int *out, int32_t *status)
{
    __shared__ uint64_t bar[32], done;
    __shared__ int flag;
    const int lane = threadIdx.x;
    kvc::mbar_init(&bar[lane], 1);
    if (lane == 0) {
        kvc::mbar_init(&done, 1);
        flag = 1;
    }
    kvc::fence_mbar_init();
    __syncwarp();
    if (lane % 2 == 0)
        kvc::mbar_arrive(&bar[lane]);
    if (lane == 0)
        kvc::mbar_arrive(&done);
    __syncwarp();
    out[lane] = kvc_tc::wait_or_abort(&bar[lane], 0, &flag, status);
    __syncwarp();
    out[32 + lane] = kvc_tc::warp_wait_or_abort(&bar[lane], 0, &flag, status);
    out[64 + lane] = kvc_tc::warp_wait_or_abort(&done, 0, &flag, status);
}

extern "C" __attribute__((visibility("default"))) int run(int *out, int32_t *status)
{
    waits<<<1, 32>>>(out, status);
    return cudaDeviceSynchronize();
}
"""


def test_lanes_with_different_answers(tmp_path):
    from persistent_kv_cache_gb300 import build as B
    src, lib = tmp_path / "waits.cu", tmp_path / "waits.so"
    src.write_text(CODE)
    subprocess.run([B._nvcc(), *B.ARCH, "-O3", "-std=c++17", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC", "-shared", "-cudart", "static",
                    "-I", B.CSRC, "-I", os.path.join(ROOT, "include"), "-o", str(lib), str(src)], check=True, capture_output=True, text=True)
    out, st = torch.full((96,), -1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    assert ctypes.CDLL(str(lib)).run(ctypes.c_void_p(out.data_ptr()), ctypes.c_void_p(st.data_ptr())) == 0
    alone, warp, complete = out.cpu().reshape(3, 32).tolist()
    assert alone == [1, 0] * 16 and warp == [0] * 32 and complete == [1] * 32
    assert st.item() == 0  # (the flag ended the waits, not their limit)
