// Helpers shared by the kernels that walk a line of key tiles (tree attention,
// accumulated attention weight).
#pragma once

#include "tc_common.cuh"

namespace pa {

// (Not the read-only path: what is read here may have been written by a kernel that
// still ran when this one was set up, before griddepcontrol.wait.)
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

// A page of one head (16 rows of D dims) moved by one copy, as rows of an operand
// whose dims run along its 128-byte rows: 8-row groups kGroup bytes apart from page to
// page, and for D = 128 the 64-dim halves of a group next to each other.  (Two copies
// of 64 dims each, all 128 rows of a half together, hold a kernel that reads pages to
// 5.6 TB/s: a copy costs its SM some 90 cycles, and the K of a decode step waited for
// them, 84 against 77 us on 470 MB.)
template <int D>
struct KPage {
  static constexpr int kBytes = 32 * D;
  static constexpr int kGroup = 16 * D;
  static constexpr int kHalf = 1024;
  // of 16 dims i of a row
  static __host__ __device__ constexpr uint32_t dims16(int i) {
    return (i >> 2) * kHalf + (i & 3) * 32;
  }
  static bool encode(CUtensorMap* map, const void* pool, uint64_t rows) {
    if (D == 128) {  // dims of a half, rows of a group, halves, groups
      const uint64_t dims[4] = {64, 8, 2, rows / 8};
      const uint64_t strides[3] = {D * 2, 128, D * 16};
      const uint32_t box[4] = {64, 8, 2, 2};
      return encode_bf16_map(map, pool, 4, dims, strides, box);
    }
    const uint64_t dims[2] = {D, rows};
    const uint64_t strides[1] = {D * 2};
    const uint32_t box[2] = {64, 16};
    return encode_bf16_map(map, pool, 2, dims, strides, box);
  }
  // The page whose first pool row is `row`.
  static __device__ __forceinline__ void load(uint32_t dst, const CUtensorMap* map, int row,
                                              uint64_t* bar) {
    if (D == 64) {
      tc::tma_load_2d(dst, map, 0, row, bar);
      return;
    }
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%2, %2, %2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row >> 3), "r"(smem_u32(bar))
        : "memory");
  }
};

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

// Launch of a kernel that may be set up while the one before it on the stream ends.
// Before its griddepcontrol.wait it may only prepare its own shared and tensor memory:
// it reads no global memory (the lengths included) and writes none.
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
