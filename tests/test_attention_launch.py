"""How the attention side's kernels are launched, with the CUDA runtime's calls replaced by ones that keep account (no GPU)."""
import os
import subprocess

import lora_co_serving_gb300 as lm
from lora_co_serving_gb300 import _build

CUDA_INCLUDE = os.path.join(os.path.dirname(os.path.dirname(_build._nvcc())), "include")

# A runtime that keeps each kernel's limit of dynamic shared memory and refuses a launch above it, as CUDA does
RUNTIME = r'''
#include <cuda_runtime_api.h>
#include <cstdio>
#include <functional>
#include <map>
#include "lora_attention.h"
std::map<const void*, size_t> limits;
std::function<void()> other_thread;      // what another thread does between a call's attribute and its launch
int launches = 0;
extern "C" {
cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute, int value) {
    limits[f] = value;
    if (other_thread) {
        auto other = other_thread;
        other_thread = nullptr;
        other();
    }
    return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**) {
    ++launches;
    const size_t limit = limits.count(f) ? limits[f] : 48 * 1024;
    return c->dynamicSmemBytes <= limit ? cudaSuccess : cudaErrorInvalidValue;
}
const char* cudaGetErrorString(cudaError_t) { return "refused"; }
static void* handle;
void** __cudaRegisterFatBinary(void*) { return &handle; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction() {}
void __cudaRegisterVar() {}
cudaError_t __cudaGetKernel() { return cudaErrorUnknown; }
cudaError_t __cudaLaunchKernel() { return cudaErrorUnknown; }
cudaError_t __cudaPopCallConfiguration() { return cudaErrorUnknown; }
}
namespace lora { void set_last_error(const char* s) { printf("%s\n", s); } }
'''


def run(tmp_path, source, body):
    """Builds the object of `source` and a main() into a program, runs it, and returns what it printed."""
    lm.build()
    obj = os.path.join(_build.OBJDIR, source + ".o")
    if not os.path.exists(obj):
        lm.build(force=True)
    src, exe = tmp_path / "t.cpp", str(tmp_path / "t")
    src.write_text(RUNTIME + body)
    subprocess.run(["g++", "-std=c++17", "-I", CUDA_INCLUDE, "-I", _build.INCLUDE, str(src), obj, "-o", exe], check=True)
    res = subprocess.run([exe], capture_output=True, text=True)
    assert res.returncode == 0, res.stdout + res.stderr
    return res.stdout


def test_two_threads_leave_each_other_the_shared_memory(tmp_path):
    """A decode batch of any number of rows, launched by another thread between a long batch's attribute and its launch."""
    run(tmp_path, "rotary.cu", r'''
int main() {
    char* const p = (char*)(1 << 20);
    for (int D : {64, 128, 256})
        for (int dt : {LORA_BF16, LORA_F32})
            for (int rows = 1; rows <= 12; ++rows) {
                lora_rotary_t r = {(int64_t*)p, p, p, 8, 2, D, D, 0, 1e-6f};
                auto forward = [&](int T) {
                    return lora_rotary_forward(T, (lora_dtype_t)dt, &r, p, 10 * D, (int64_t*)p, p + (1 << 24), 10 * D,
                                               nullptr, 0, nullptr, nullptr, 0, nullptr);
                };
                auto backward = [&](int T) {
                    return lora_rotary_backward(T, (lora_dtype_t)dt, &r, p, 10 * D, (int64_t*)p, p, 10 * D, p + (1 << 24),
                                                10 * D, (float*)p, (float*)p, p, 1 << 30, nullptr);
                };
                int rc = 0;
                other_thread = [&] { rc |= forward(rows); };
                rc |= forward(5000);
                if (rc || other_thread) return printf("forward, %d rows of heads of %d\n", rows, D), 1;
                other_thread = [&] { rc |= backward(rows); };
                rc |= backward(5000);
                if (rc || other_thread) return printf("backward, %d rows of heads of %d\n", rows, D), 1;
            }
    return launches > 0 ? 0 : 1;
}
''')
