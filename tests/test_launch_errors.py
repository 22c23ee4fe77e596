"""A launch that fails is the failure of its call: nothing of it is left for the next call to find."""
import ctypes
import os
import subprocess

import tensor_train_compressed_embeddingbag_gb300._nvcc_build as b

SHIM = r"""
#include <cuda_runtime.h>
// A runtime whose launches fail, and which keeps the last error as the real one does.
static cudaError_t g_last = cudaSuccess;
template <class... A>
cudaError_t failing_launch(A&&...) { return g_last = cudaErrorInvalidConfiguration; }
static cudaError_t last_error() { const cudaError_t e = g_last; g_last = cudaSuccess; return e; }
#define cudaLaunchKernelEx failing_launch
#define cudaGetLastError last_error
#include "tt_units.cuh"
namespace ttemb {
__global__ void k_nothing(int) {}
}
extern "C" int launch(int* left) {
    const bool ok = ttemb::launch_ahead(ttemb::k_nothing, dim3(1), 32, 0, nullptr, 1);
    *left = (int)g_last;
    return ok;
}
"""


def test_a_launch_that_fails_leaves_no_error(tmp_path):
    src, so = tmp_path / "shim.cu", tmp_path / "shim.so"
    src.write_text(SHIM)
    subprocess.run([b.nvcc(), *b.ARCH, *b.FLAGS, "-shared", str(src), "-o", str(so)], check=True, capture_output=True)
    left = ctypes.c_int(-1)
    assert not ctypes.CDLL(str(so)).launch(ctypes.byref(left))
    assert left.value == 0
