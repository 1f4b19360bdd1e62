"""mxfp8_device_status tells every wait that a kernel gave up, once.  On the CPU: csrc/status.cu over a stand-in
for the CUDA runtime, in which another stream's kernel counts itself at the worst moment.  On the GPU: a small
kernel waits, with the library's own wait and count, for an arrival that never comes."""
import ctypes
import os
import shutil
import subprocess

import pytest

from mxfp8_master_weight_gb300 import _capi, build

FAKE_RUNTIME = r"""
#pragma once
#include <cstddef>
#include <cstring>
#define __device__
enum cudaError_t { cudaSuccess, cudaErrorInvalidDevice };
enum cudaMemcpyKind { cudaMemcpyDeviceToHost, cudaMemcpyHostToDevice };
typedef void* cudaStream_t;
extern int fake_device;
void fake_synchronized();  // what the GPU does between a call's synchronisation and its next step
inline cudaError_t cudaGetDevice(int* d) { *d = fake_device; return cudaSuccess; }
template <class T> cudaError_t cudaGetSymbolAddress(void** p, T& s) { *p = &s; return cudaSuccess; }
template <class T> cudaError_t cudaMemcpyFromSymbolAsync(void* dst, const T& s, size_t n, size_t, cudaMemcpyKind, cudaStream_t) {
  std::memcpy(dst, &s, n);
  return cudaSuccess;
}
template <class T> cudaError_t cudaMemcpyToSymbolAsync(T& s, const void* src, size_t n, size_t, cudaMemcpyKind, cudaStream_t) {
  std::memcpy(&s, src, n);
  return cudaSuccess;
}
inline cudaError_t cudaStreamSynchronize(cudaStream_t) { fake_synchronized(); return cudaSuccess; }
"""

PROGRAM = r"""
#include "status.cu"
#include <cassert>
#include <thread>
#include <vector>

int fake_device = 0;
static unsigned* counter;
static unsigned meanwhile = 0;
void fake_synchronized() { *counter += meanwhile; meanwhile = 0; }

static unsigned told() {
  unsigned n = 77;
  assert(mxfp8::waits_given_up(nullptr, &n) == cudaSuccess);
  return n;
}

int main() {
  assert(mxfp8::given_up_address(0, &counter) == cudaSuccess);
  assert(told() == 0);
  *counter += 3;
  assert(told() == 3 && told() == 0);
  // another stream's kernel counts itself while this call reads: told by the next call, not lost
  *counter += 1;
  meanwhile = 2;
  assert(told() == 1);
  assert(told() == 2 && told() == 0);
  // the count wraps
  mxfp8::Told t;
  assert(t.news(0x7fffffffu) == 0x7fffffffu && t.news(0xfffffffeu) == 0x7fffffffu && t.news(2) == 4 && t.news(2) == 0);
  // an older reading that comes late adds nothing
  assert(t.news(9) == 7 && t.news(5) == 0 && t.news(9) == 0 && t.news(10) == 1);
  // many threads: the sum of what they are told is what was added
  mxfp8::Told shared;
  std::atomic<unsigned> count{0}, sum{0};
  std::vector<std::thread> threads;
  for (int i = 0; i < 8; ++i)
    threads.emplace_back([&] {
      for (int k = 0; k < 20000; ++k) {
        count.fetch_add(1);
        sum.fetch_add(shared.news(count.load()));
      }
    });
  for (auto& th : threads) th.join();
  assert(sum.load() == 160000u && count.load() == 160000u);
  fake_device = 1000;
  unsigned n;
  assert(mxfp8::waits_given_up(nullptr, &n) == cudaErrorInvalidDevice);
  return 0;
}
"""


def test_every_count_is_told_once(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    (tmp_path / "cuda_runtime.h").write_text(FAKE_RUNTIME)
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-pthread", f"-I{tmp_path}", f"-I{build.CSRC}", str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stderr


# One warp waits on a barrier of its own that expects one arrival, which nothing makes.
PROBE = r"""
#include "status.h"
#include "tensor_core.cuh"

using namespace mxfp8;

__global__ void k_wait_in_vain(unsigned* given_up, long long* cycles) {
  __shared__ uint64_t bar;
  __shared__ uint32_t s_gave_up;
  if (threadIdx.x == 0) {
    tc::mbar_init(tc::smem_addr(&bar), 1);
    s_gave_up = 0;
    tc::mbar_init_fence();
  }
  __syncthreads();
  const long long t0 = clock64();
  const bool landed = tc::mbar_wait(tc::smem_addr(&bar), 0, &s_gave_up);
  __syncthreads();
  if (threadIdx.x == 0) {
    *cycles = landed ? -1 : clock64() - t0;
    if (s_gave_up != 0) tc::report_given_up(given_up);
  }
}

extern "C" __attribute__((visibility("default"))) int wait_in_vain(int blocks, long long* cycles, void* stream) {
  unsigned* at = nullptr;
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess || given_up_address(device, &at) != cudaSuccess) return 1;
  k_wait_in_vain<<<blocks, 32, 0, static_cast<cudaStream_t>(stream)>>>(at, cycles);
  return cudaGetLastError() != cudaSuccess;
}
"""


@pytest.mark.gpu
def test_a_wait_in_vain_is_told_once(tmp_path):
    """The wait ends by itself, the next status call says so, the one after is clean, and the context works on."""
    import torch
    build.build()
    objects = [os.path.join(build.BUILD_DIR, u.replace(".cu", ".o")) for u in build.UNITS]
    if not all(map(os.path.exists, objects)):
        build.build(force=True)
    src, lib = tmp_path / "probe.cu", tmp_path / "probe.so"
    src.write_text(PROBE)
    subprocess.run([build._nvcc(), *build.cflags(), "-shared", "-cudart", "static", str(src), *objects, "-o", str(lib)], check=True)
    so = ctypes.CDLL(str(lib))
    vp, i64 = ctypes.c_void_p, ctypes.c_int64
    so.wait_in_vain.argtypes, so.mxfp8_device_status.argtypes = [ctypes.c_int, vp, vp], [vp]
    so.mxfp8_last_error.restype = ctypes.c_char_p
    cycles = torch.zeros(1, dtype=torch.int64, device="cuda")
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    status = lambda st: so.mxfp8_device_status(vp(st.cuda_stream))  # noqa: E731
    assert status(one) == 0
    assert so.wait_in_vain(2, vp(cycles.data_ptr()), vp(one.cuda_stream)) == 0
    assert status(one) == 6 and b"gave up" in so.mxfp8_last_error()
    assert status(one) == 0 and so.mxfp8_last_error() == b""
    # the limit and one interval between looks, and the time that the last look itself took
    assert 4.0e9 < cycles.item() < 3 * 4.0e9
    # on another stream: told to whoever asks after it completed
    assert so.wait_in_vain(1, vp(cycles.data_ptr()), vp(two.cuda_stream)) == 0
    two.synchronize()
    assert status(one) == 6 and status(two) == 0
    # the context is usable, and so are the operators
    T = _capi.Tensor
    x, w = torch.randn(4, 64, device="cuda"), torch.ones(64, device="cuda")
    y, mean, rstd = torch.empty_like(x), torch.empty(4, device="cuda"), torch.empty(4, device="cuda")
    t = lambda v: ctypes.byref(T(vp(v.data_ptr()), _capi.DTYPE_F32, v.dim(), (i64 * 2)(*(list(v.shape) + [0])[:2])))  # noqa: E731
    so.mxfp8_layer_norm_forward.argtypes = [ctypes.POINTER(T)] * 6 + [i64, i64, ctypes.c_float, vp]
    empty = _capi.empty_tensor()
    torch.cuda.synchronize()
    assert so.mxfp8_layer_norm_forward(t(x), t(w), ctypes.byref(empty), t(y), t(mean), t(rstd), 4, 64, 1e-5, vp(one.cuda_stream)) == 0
    assert status(one) == 0
    assert torch.allclose(y, torch.nn.functional.layer_norm(x, (64,)), atol=1e-5)
