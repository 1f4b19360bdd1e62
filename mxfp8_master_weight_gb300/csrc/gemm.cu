// Block-scaled product out = A B^T (+ addend) on the tensor cores.
//
//   out[i][j] = sum_p 2^(ea - 127) 2^(eb - 127) A(i, p) B(j, p)
//
// with E4M3 codes and one E8M0 scale per 32 or 128 values of p in each operand.  The scales are
// powers of two, so the block-scaled matrix instruction (tcgen05.mma kind::mxf8f6f4) takes them
// as they are: it multiplies each 32-value partial product by both scales and adds into F32 sums
// in tensor memory, with no pass over the sums in between.  A scale column in tensor memory
// holds four bytes per row; with 32 values per scale the four instructions of a 128-value stage
// take bytes 0..3, with 128 values they all take byte (stage % 4), so both block sizes read the
// same 128x4-tile layout and may meet in one product.
//
// An operand is read as it lies: a box of 128 stored rows by 128 bytes goes to shared memory under
// the 128-byte swizzle whether its rows run along k or across it, and the instruction descriptor
// says which.  Rows and bytes past the matrix are zeros, which add nothing (a scale is never
// infinite; padding scales are finite).
//
// k_gemm_any: operands whose base or row stride is not a multiple of 16 bytes, which no TMA map
// can describe.  256 threads fetch the boxes with whatever loads the addresses allow and store
// them swizzled; one thread issues the matrix instructions.
#include <atomic>

#include "gemm_impl.cuh"
#include "gemm_maps.h"

namespace mxfp8 {
namespace {

__device__ unsigned g_given_up = 0;

// ------------------------------------------------------------------------------ any alignment
constexpr int kAnyStages = 3;
constexpr int kAnyLoaders = 256;
constexpr int kAnyStageBytes = 2 * kBoxBytes + 2 * kScaleTile;  // A, B and their scales
constexpr int kAnySmem = kAnyStages * kAnyStageBytes + 1024 + 256;
constexpr int kAnyTmemCols = 256;  // 128 of sums, then two buffers of 4 + 4 scale columns

// 16 bytes at p of which the first n belong to the row (zeros past them).  [lo, hi) are the
// matrix's bytes: no load leaves them.
__device__ __forceinline__ uint4 load16(const uint8_t* p, int n, const uint8_t* lo, const uint8_t* hi) {
  if (n <= 0) return make_uint4(0, 0, 0, 0);
  const uintptr_t at = reinterpret_cast<uintptr_t>(p);
  if (n >= 16) {
    if (at % 16 == 0) return *reinterpret_cast<const uint4*>(p);
    const uint32_t* w = reinterpret_cast<const uint32_t*>(at & ~uintptr_t(3));
    if (at % 4 == 0) return make_uint4(w[0], w[1], w[2], w[3]);
    if (reinterpret_cast<const uint8_t*>(w) >= lo && reinterpret_cast<const uint8_t*>(w) + 20 <= hi) {
      const uint32_t sh = uint32_t(at & 3) * 8;
      const uint32_t a = w[0], b = w[1], c = w[2], d = w[3], e = w[4];
      return make_uint4(__funnelshift_r(a, b, sh), __funnelshift_r(b, c, sh), __funnelshift_r(c, d, sh),
                        __funnelshift_r(d, e, sh));
    }
  }
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (i < n) w[i >> 2] |= uint32_t(p[i]) << (8 * (i & 3));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// This thread's four 16-byte units of an operand's box at (mn0, k0): unit t % 8 of rows
// t / 8 + 32 i of the stored matrix.
__device__ __forceinline__ void fetch_box(const GemmOperand& o, int64_t k, int64_t mn0, int64_t k0, int t,
                                          uint4 (&v)[4]) {
  const int64_t rows = o.colwise ? k : o.mn, cols = o.colwise ? o.mn : k;
  const int64_t row0 = o.colwise ? k0 : mn0, col = (o.colwise ? mn0 : k0) + 16 * (t & 7);
  const int64_t left = cols - col;
  const int n = left >= 16 ? 16 : (left > 0 ? int(left) : 0);
  const uint8_t* hi = o.codes + (rows - 1) * o.ld + cols;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = row0 + (t >> 3) + 32 * i;
    v[i] = load16(o.codes + row * o.ld + col, row < rows ? n : 0, o.codes, hi);
  }
}

__device__ __forceinline__ void store_box(char* smem, int t, const uint4 (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = (t >> 3) + 32 * i;
    *reinterpret_cast<uint4*>(smem + row * 128 + (((t & 7) ^ (row & 7)) << 4)) = v[i];
  }
}

__global__ void __launch_bounds__(kAnyLoaders + 32) k_gemm_any(const __grid_constant__ GemmParams p) {
  extern __shared__ char raw[];
  char* smem = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kAnyStages * kAnyStageBytes);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kAnyStages + 1);
  volatile uint32_t* gave_up = tmem_slot + 1;
  const int t = threadIdx.x, warp = t >> 5;
  const uint32_t full = tc::smem_addr(bars), empty = full + 8 * kAnyStages, done = empty + 8 * kAnyStages;
  if (t == 0) {
    for (int s = 0; s < kAnyStages; ++s) {
      tc::mbar_init(full + 8 * s, kAnyLoaders);
      tc::mbar_init(empty + 8 * s, 1);
    }
    tc::mbar_init(done, 1);
    *gave_up = 0;
    tc::mbar_init_fence();
  }
  if (warp == 8) tc::tmem_alloc<1>(tc::smem_addr(tmem_slot), kAnyTmemCols);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  tc::grid_wait_then_release();
  const uint32_t tmem = *tmem_slot;
  int64_t tm, tn;
  tile_at(blockIdx.x, (p.m + 127) / 128, (p.n + 127) / 128, tm, tn);
  const int64_t nk = (p.k + kBlockK - 1) / kBlockK;

  if (warp < 8) {
    const GemmOperand& mine = t < 32 ? p.a : p.b;  // whose scales threads 0..63 fetch
    const uint8_t* scales = mine.scale + (t < 32 ? tm : tn) * scale_tiles_along_k(p.k, mine.block) * kScaleTile;
    for (int64_t kb = 0; kb < nk; ++kb) {
      const int s = int(kb % kAnyStages);
      uint4 a[4], b[4], sc = make_uint4(0, 0, 0, 0);
      fetch_box(p.a, p.k, tm * 128, kb * kBlockK, t, a);
      fetch_box(p.b, p.k, tn * 128, kb * kBlockK, t, b);
      if (t < 64)
        sc = *reinterpret_cast<const uint4*>(scales + scale_tile_of(kb, mine.block) * kScaleTile + 16 * (t & 31));
      if (!tc::mbar_wait(empty + 8 * s, uint32_t((kb / kAnyStages) & 1) ^ 1, gave_up)) break;
      char* st = smem + s * kAnyStageBytes;
      store_box(st, t, a);
      store_box(st + kBoxBytes, t, b);
      if (t < 64) *reinterpret_cast<uint4*>(st + 2 * kBoxBytes + 16 * t) = sc;
      tc::fence_async_proxy();
      tc::mbar_arrive(full + 8 * s);
    }
  } else if (t == kAnyLoaders) {
    const uint32_t idesc = tc::instr_desc(128, 128, p.a.colwise, p.b.colwise);
    const uint32_t astep = p.a.colwise ? 4096 : 32, bstep = p.b.colwise ? 4096 : 32;  // bytes per 32 values of k
    for (int64_t kb = 0; kb < nk; ++kb) {
      const int s = int(kb % kAnyStages);
      if (!tc::mbar_wait(full + 8 * s, uint32_t((kb / kAnyStages) & 1), gave_up)) break;
      tc::fence_after_sync();
      const uint32_t st = tc::smem_addr(smem + s * kAnyStageBytes);
      const uint32_t sa = tmem + 128 + 8 * uint32_t(kb & 1), sb = sa + 4;
      tc::copy_scales<1>(sa, tc::scale_desc(st + 2 * kBoxBytes));
      tc::copy_scales<1>(sb, tc::scale_desc(st + 2 * kBoxBytes + kScaleTile));
#pragma unroll
      for (int j = 0; j < 4; ++j)
        tc::mma_scaled<1>(tmem, tc::operand_desc(st + j * astep), tc::operand_desc(st + kBoxBytes + j * bstep),
                          tc::with_scale_ids(idesc, scale_id_of(kb, j, p.a.block), scale_id_of(kb, j, p.b.block)), sa,
                          sb, kb > 0 || j > 0);
      tc::commit(empty + 8 * s);
    }
    tc::commit(done);
  }
  __syncwarp();
  if (warp < 8) {
    tc::mbar_wait(done, 0, gave_up);
    tc::fence_after_sync();
    // the stages are free again: every copy into them has been used
    const int width = p.out_f32 ? 32 : 64;
    for (int c = 64 * (warp >> 2); c < 64 * (warp >> 2) + 64; c += width) {
      write_rows(p, smem + warp * 4096, tm * 128 + 32 * (warp & 3), tn * 128 + c, [&](int e, float(&v)[32]) {
        if (nk > 0) {
          tc::tmem_load32(tmem + (uint32_t(32 * (warp & 3)) << 16) + c + e, v);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0.0f;
        }
      });
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (t == 0 && *gave_up != 0) tc::report_given_up(&g_given_up);
  if (warp == 8) tc::tmem_free<1>(tmem, kAnyTmemCols);
}

}  // namespace

// Device address of g_given_up for the current device, looked up once per device.
cudaError_t given_up_address(int device, unsigned** out) {
  constexpr int kMaxDevices = 64;
  static std::atomic<unsigned*> known[kMaxDevices];
  unsigned* p = device < kMaxDevices ? known[device].load() : nullptr;
  if (p == nullptr) {
    const cudaError_t e = cudaGetSymbolAddress(reinterpret_cast<void**>(&p), g_given_up);
    if (e != cudaSuccess) return e;
    if (device < kMaxDevices) known[device].store(p);
  }
  *out = p;
  return cudaSuccess;
}

cudaError_t launch_gemm(const GemmParams& p, const DeviceInfo& dev, cudaStream_t stream, const char** what) {
  if (p.a.aligned && p.b.aligned) {
    unsigned* given_up = nullptr;
    const cudaError_t e = given_up_address(dev.device, &given_up);
    if (e != cudaSuccess) return e;
    // Split over k: outputs of at most 64 rows or columns (a tile of the pair kernel would stay mostly
    // empty: 64 x 4096 x 4096 8.6 us split, 10.3 us by pairs), and few tiles with a long k, where it
    // finds work for every SM (160 x 96 x 2048 7.5 / 11.0 us).  Everything else by pairs
    // (1024^3 9.4 / 6.0 us, 256 x 4096 x 4096 14.8 / 10.5 us, 2048^3 12.4 / 10.8 us).
    const int64_t halves = ((p.m + 255) / 256) * ((p.n + 127) / 128);
    const bool split = p.m <= 64 || p.n <= 64 || (8 * halves <= dev.sms && p.k >= 16 * kBlockK);
    return split ? launch_gemm_split(p, given_up, dev, stream, what) : launch_gemm_pair(p, given_up, dev, stream, what);
  }
  const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(k_gemm_any),
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, kAnySmem);
  if (e != cudaSuccess) return e;
  const int64_t tiles = ((p.m + 127) / 128) * ((p.n + 127) / 128);
  if (tiles > 0x7fffffff) {
    *what = "gemm: too many output tiles";
    return cudaErrorInvalidValue;
  }
  return launch_kernel(k_gemm_any, dim3(static_cast<unsigned>(tiles)), dim3(kAnyLoaders + 32), kAnySmem, stream, p);
}

cudaError_t waits_given_up(cudaStream_t stream, unsigned* count) {
  cudaError_t e = cudaMemcpyFromSymbolAsync(count, g_given_up, sizeof(unsigned), 0, cudaMemcpyDeviceToHost, stream);
  if (e != cudaSuccess) return e;
  e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess || *count == 0) return e;
  static const unsigned zero = 0;
  return cudaMemcpyToSymbolAsync(g_given_up, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, stream);
}

}  // namespace mxfp8
