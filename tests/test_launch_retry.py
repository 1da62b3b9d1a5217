"""The launch helpers' second attempt, on the CPU: a program with its own stand-ins for the five runtime calls
that they make.  The stand-ins keep a failed call's error until it is asked for, as the runtime's
documentation has it, whatever succeeds in between."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

STAND_INS = r"""
#include <cuda_runtime_api.h>

int limit = 49152, launches = 0, refusals = 0;
static cudaError_t last = cudaSuccess;
static cudaError_t done(cudaError_t e) { if (e != cudaSuccess) last = e; return e; }

extern "C" {
cudaError_t cudaGetDevice(int *d) { *d = 0; return done(cudaSuccess); }
cudaError_t cudaFuncSetAttribute(const void *, cudaFuncAttribute a, int v) {
    if (a == cudaFuncAttributeMaxDynamicSharedMemorySize) limit = v;
    return done(cudaSuccess);
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *c, const void *, void **) {
    if ((int)c->dynamicSmemBytes > limit) { ++refusals; return done(cudaErrorInvalidValue); }
    ++launches;
    return done(cudaSuccess);
}
cudaError_t cudaGetLastError() { const cudaError_t e = last; last = cudaSuccess; return e; }
cudaError_t cudaPeekAtLastError() { return last; }
}
"""

PROGRAM = r"""
#include <cstdio>
#include "paged_kv_attention_write_gb300/csrc/common.cuh"

extern int limit, launches, refusals;
static void kernel(int) {}
static std::atomic<int> a[pa::kMaxDevices], b[pa::kMaxDevices];
static int bad = 0;
static void expect(const char *what, int got, int want) {
    if (got != want) { std::printf("%s: %d, not %d\n", what, got, want); bad = 1; }
}

int main() {
    const dim3 one(1);
    // the limit is raised by the first launch, to what the caller names
    expect("smem", pa::launch_pdl_smem(kernel, a, one, one, 60000, 0, 1), cudaSuccess);
    expect("cluster", pa::launch_pdl_cluster(kernel, b, one, one, 30000, 90000, 2, 0, 1), cudaSuccess);
    expect("limit", limit, 90000);
    expect("deeper", pa::launch_pdl_cluster(kernel, b, one, one, 80000, 90000, 2, 0, 1), cudaSuccess);
    expect("refusals", refusals, 0);
    // the limit is lost: one refused launch, and the next one's success is the call's
    limit = 49152;
    expect("smem again", pa::launch_pdl_smem(kernel, a, one, one, 60000, 0, 1), cudaSuccess);
    limit = 49152;
    expect("cluster again", pa::launch_pdl_cluster(kernel, b, one, one, 80000, 90000, 2, 0, 1), cudaSuccess);
    expect("refusals", refusals, 2);
    expect("launches", launches, 5);
    expect("nothing is left behind", cudaPeekAtLastError(), cudaSuccess);
    // a launch that fails for good says so, and its error can be asked for
    expect("too much", pa::launch_pdl_cluster(kernel, b, one, one, 99000, 90000, 2, 0, 1), cudaErrorInvalidValue);
    expect("its error", cudaGetLastError(), cudaErrorInvalidValue);
    return bad;
}
"""


def test_second_attempt(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("no nvcc")
    (tmp_path / "retry.cu").write_text(PROGRAM)
    (tmp_path / "stand_ins.cpp").write_text(STAND_INS)
    exe = str(tmp_path / "retry")
    r = subprocess.run([nvcc, "-std=c++17", "-cudart", "shared", "-gencode", "arch=compute_103a,code=sm_103a", "-I", ROOT,
                        "-I", os.path.join(ROOT, "include"), "-o", exe, str(tmp_path / "retry.cu"),
                        str(tmp_path / "stand_ins.cpp")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    lib = os.path.join(os.path.dirname(os.path.dirname(nvcc)), "lib64")
    r = subprocess.run([exe], capture_output=True, text=True,
                       env={**os.environ, "LD_LIBRARY_PATH": lib + ":" + os.environ.get("LD_LIBRARY_PATH", "")})
    assert r.returncode == 0, r.stdout + r.stderr
