"""A process that calls the library on one device and then on another (no GPU needed: the host code is linked with a
stand-in for the CUDA runtime that has two devices and keeps each kernel's shared-memory limit per device, as CUDA does)."""
import ctypes
import os
import subprocess

import pytest

import bit_matvec_lb_gb300 as lb
from bit_matvec_lb_gb300 import build

RUNTIME = r"""
#include <cuda_runtime.h>
#include <cstdlib>
#include <map>
#include <new>
#include <utility>
static int device = 0;
static bool no_memory = false;
void *operator new(size_t n) {
    void *p = no_memory ? nullptr : std::malloc(n);
    if (!p) throw std::bad_alloc();
    return p;
}
void operator delete(void *p) noexcept { std::free(p); }
void operator delete(void *p, size_t) noexcept { std::free(p); }
static std::map<std::pair<int, const void *>, int> limit;   // dynamic shared memory, 48 KB unless it was raised
extern "C" {
cudaError_t cudaGetDevice(int *d) { *d = device; return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaPeekAtLastError() { return cudaSuccess; }
const char *cudaGetErrorName(cudaError_t) { return ""; }
cudaError_t cudaDeviceGetAttribute(int *v, cudaDeviceAttr a, int) {
    *v = a == cudaDevAttrMaxSharedMemoryPerBlockOptin ? 227 * 1024 : a == cudaDevAttrComputeCapabilityMajor ? 10
         : a == cudaDevAttrComputeCapabilityMinor ? 3 : 152;
    return cudaSuccess;
}
cudaError_t cudaFuncGetAttributes(cudaFuncAttributes *a, const void *) { a->sharedSizeBytes = 1024; return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void *k, cudaFuncAttribute, int v) {
    limit[{device, k}] = v;
    return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int *n, const void *, int, size_t, unsigned) {
    *n = 1;
    return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessor(int *n, const void *, int, size_t) { *n = 1; return cudaSuccess; }
cudaError_t cudaGetSymbolAddress(void **, const void *) { return cudaErrorUnknown; }
cudaError_t cudaGetDriverEntryPointByVersion(const char *, void **, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult *) { return cudaErrorUnknown; }
cudaError_t cudaMemcpyAsync(void *, const void *, size_t, cudaMemcpyKind, cudaStream_t) { return cudaErrorUnknown; }
cudaError_t cudaMemsetAsync(void *, int, size_t, cudaStream_t) { return cudaErrorUnknown; }
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaErrorUnknown; }
void **__cudaRegisterFatBinary(void *) { static void *p; return &p; }
void __cudaRegisterFatBinaryEnd(void **) {}
void __cudaUnregisterFatBinary(void **) {}
void __cudaRegisterVar(void **, char *, char *, const char *, int, size_t, int, int) {}
void __cudaRegisterFunction(void **, const char *, char *, const char *, int, void *, void *, void *, void *, int *) {}
char __cudaInitModule(void **) { return 0; }
}
namespace lb { int prepare_kernel(const void *kernel, int threads, size_t smem, int *blocks_per_sm); }
extern "C" __attribute__((visibility("default"))) int prepare_without_memory(const void *kernel) {
    int per_sm = 0;
    device = 0;
    no_memory = true;
    const int status = lb::prepare_kernel(kernel, 256, 1024, &per_sm);   // (an exception would end the process)
    no_memory = false;
    return status;
}
extern "C" __attribute__((visibility("default"))) int prepare_on(int dev, const void *kernel, size_t smem) {
    int per_sm = 0;
    device = dev;
    const int status = lb::prepare_kernel(kernel, 256, smem, &per_sm);
    if (status != 0) return status;
    const auto at = limit.find({dev, kernel});
    return (at == limit.end() ? 48 * 1024 : at->second) >= (int)smem ? 0 : 1;   // 1: the launch would be refused
}
"""


@pytest.fixture(scope="module")
def runtime(tmp_path_factory):
    lb.load()   # (the objects are there and up to date)
    at = tmp_path_factory.mktemp("devices")
    (at / "runtime.cpp").write_text(RUNTIME)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(build._nvcc())))
    subprocess.run(["g++", "-shared", "-fPIC", "-O1", "-I", os.path.join(cuda, "include"), str(at / "runtime.cpp"),
                    os.path.join(build.BUILD, "lb_capi.o"), "-Wl,-Bsymbolic", "-o", str(at / "devices.so")], check=True)
    return ctypes.CDLL(str(at / "devices.so"))


@pytest.fixture(scope="module")
def prepare_on(runtime):
    runtime.prepare_on.argtypes = [ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t]
    return runtime.prepare_on


def test_shared_memory_limit_of_every_device(prepare_on):
    """Products take about 200 KB of shared memory; without its own limit the second device refuses the launch."""
    for kernel in (0x1000, 0x2000):
        for dev in (0, 1, 0, 1, 63):
            assert prepare_on(dev, kernel, 200 * 1024) == 0, (dev, kernel)


def test_a_device_beyond_the_last(prepare_on):
    assert prepare_on(64, 0x3000, 1024) == -5


def test_no_memory_on_the_host(runtime):
    """An error, not an exception through a C entry; the next call finds its way."""
    runtime.prepare_without_memory.argtypes = [ctypes.c_void_p]
    assert runtime.prepare_without_memory(0x4000) == -6
    assert runtime.prepare_on(0, 0x4000, 1024) == 0
