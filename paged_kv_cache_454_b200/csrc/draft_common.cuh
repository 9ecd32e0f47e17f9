// Helpers shared by the kernels that walk a line of key tiles (tree attention,
// accumulated attention weight).
#pragma once

#include "tc_common.cuh"

namespace pa {

// (Not the read-only path: what is read here may have been written by a kernel that
// still ran when this one was set up.)
__device__ __forceinline__ int ld_i32(const int32_t* ptr) {
  int x;
  asm volatile("ld.global.b32 %0, [%1];" : "=r"(x) : "l"(ptr));
  return x;
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// One lane of a converged warp, always the same.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// A wait of a unit ring: several times as long as the waits for data, and heeding
// no abort flag (every role takes every unit).
__device__ __forceinline__ bool ring_wait(uint64_t* bar, uint32_t parity, unsigned* err) {
  for (int i = 0; i < 8; ++i)
    if (mbar_wait(bar, parity, nullptr, err)) return true;
  return false;
}

// A sequence of the batch, as the lengths on the device describe it.
struct SeqRaw {
  int q0, q1, L;
};

// Division by a number from 1 to 256 that the host knows, of numbers below 2^24: the
// product with m = floor(2^32 / d) + 1 exceeds n 2^32 / d by less than n, hence the
// quotient by less than 2^-8 <= 1/d.
struct Divisor {
  uint64_t m;
  Divisor() = default;
  explicit Divisor(uint32_t d) : m((1ull << 32) / d + 1) {}
  __device__ __forceinline__ int quotient(uint32_t n) const {
    return static_cast<int>((n * m) >> 32);
  }
};

__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)),
               "r"(bytes)
               : "memory");
}

// Quotient of two non-negative numbers; a 64-bit division is ten times a 32-bit
// one, and the numbers here rarely need it.
__device__ __forceinline__ long long quotient(long long a, long long b) {
  if (((a | b) >> 32) == 0)
    return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// Exclusive scan of one number per thread over a CTA of `warps` warps (`slots`: as
// many words of shared memory); `total` is the sum of all.
template <int kWarps>
__device__ __forceinline__ long long cta_scan(long long mine, long long* slots, long long& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  long long scan = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += v;
  }
  if (lane == 31) slots[warp] = scan;
  __syncthreads();
  long long before = scan - mine;
  total = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += slots[w];
    total += slots[w];
  }
  return before;
}

// Launch of a kernel that may be set up while the one before it on the stream ends
// (it waits for that one's end itself, before it reads anything).
template <typename P>
inline int launch_overlapped(void (*kernel)(P), dim3 grid, int threads, int smem, const P& p,
                             cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess) return PA_OK;
  cudaGetLastError();
  return PA_ERR_CUDA;
}

}  // namespace pa
