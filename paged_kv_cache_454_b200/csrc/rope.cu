// Rotary positions, norms per head and the cache write of the prepared K and V.
//
// A row of D dims belongs to D/8 neighbouring lanes, 16 bytes each, so a row is
// read and written with one coalesced access per lane and its norm is a
// shuffle reduction inside those lanes.  A CTA works on four tokens, 64 threads
// each, and on one part of their rows: the q heads (split further where there
// are few tokens), the K heads or the V heads, so no part waits for another's
// loads.  The tokens' cos and sin are computed once per CTA, a pair per thread,
// and met in shared memory.  A lane always has the same dims whatever the head,
// so it then keeps its cos and sin, times the norm's weights, in registers, and
// a row is
//     y = r (x A + x' B),   r = 1 / sqrt(mean x^2 + eps) or 1,
// with x' the partner dims: rot/16 lanes away in the half layout (shuffled as
// packed bf16 pairs), inside the lane in the interleaved one.
//
// Bound: HBM for many tokens (every row is read once and written once), the
// launch for few.
#include <math.h>

#include <algorithm>

#include "../../include/pa_rope.h"
#include "common.cuh"
#include "internal.h"

namespace pa {
namespace {

// Measured (graph replays; 32768 tokens of 64/8 heads, 1.34 GB | 4288 of 40/8 |
// 128 of 64/8): four tokens of a CTA 231 | 28.1 | 3.8 us (5.8 TB/s at the
// largest), two 271 | 35 | 4.3, one 401 | 63 | 5.2 -- a CTA's angles and its
// wait for them cost as much as a dozen rows.  Three rows in flight 231 | 28.1,
// two 238 | 28.1, four 236 | 28.2; four CTAs resident per SM 231, three 251.
constexpr int kRopeThreads = 256;
constexpr int kRopeTokens = 4;  // tokens of a CTA
constexpr int kRopeTokenThreads = kRopeThreads / kRopeTokens;
// Fewer q CTAs than this per SM: the q heads are split (two 28.3 | 3.8 us on 4288 and
// 128 tokens, sixteen 30.3 | 4.2).
constexpr int kRopeCtasPerSm = 2;
constexpr int kRopeRows = 3;       // rows of a lane group in flight

struct RopeParams {
  const uint4* q;
  const uint4* k;
  const uint4* v;
  uint4* q_out;
  uint4* k_out;    // without the cache write
  uint4* k_pool;   // with it
  uint4* v_pool;
  int64_t q_stride, k_stride, v_stride, q_out_stride, k_out_stride;  // 16-byte chunks
  const uint4* q_weight;
  const uint4* k_weight;
  const int64_t* positions;
  const double* inv_freq;
  const int64_t* slots;
  int hq, hkv;
  int num_tokens;
  int q_parts, parts;  // CTAs of four tokens: for their q heads, in all
  int rot;
  int num_blocks;
  float factor, eps;
  unsigned int* err;
};

// cos and sin of position * inv_freq.  The product and its reduction to within
// half a turn are fp64: at position 10^6 an fp32 product would be off by 0.06
// rad in the fastest pair.
__device__ __forceinline__ float2 turn_of(int64_t position, double inv_freq, float factor) {
  constexpr double kTurnsPerRad = 0.15915494309189533577;
  const double turns = static_cast<double>(position) * inv_freq * kTurnsPerRad;
  const float r = static_cast<float>(turns - rint(turns));
  float s, c;
  sincospif(2.f * r, &s, &c);
  return make_float2(c * factor, s * factor);
}

__device__ __forceinline__ float2 unpack2(uint32_t w) { return make_float2(bf16lo(w), bf16hi(w)); }

__device__ __forceinline__ uint32_t pack2(float2 x) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(x.x, x.y);
  return *reinterpret_cast<const uint32_t*>(&b);
}

__device__ __forceinline__ uint32_t word(const uint4& w, int j) {
  return j == 0 ? w.x : j == 1 ? w.y : j == 2 ? w.z : w.w;
}

template <int D, bool kInterleaved, bool kCache>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kLanes = D / 8;                       // lanes of a row
  constexpr int kGroups = kRopeTokenThreads / kLanes;  // rows of a token in work at once
  __shared__ float2 turn[kRopeTokens][D / 2];
  // a decode plan launched after this kernel may start now (it reads only the
  // tables and lengths before this grid has ended, and writes nothing)
  if (kCache) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int mine = threadIdx.x / kRopeTokenThreads;  // which of the CTA's tokens
  const int at = threadIdx.x % kRopeTokenThreads;
  const int part = blockIdx.x % p.parts;
  const int64_t t = static_cast<int64_t>(blockIdx.x / p.parts) * kRopeTokens + mine;
  const bool live = t < p.num_tokens;  // alike in a warp
  const int lane = at % kLanes;
  const bool is_q = part < p.q_parts;
  const int lead = is_q ? part * kGroups : 0;  // the first head of the token's first group
  const int first = lead + at / kLanes;        // and of this thread's group
  const int step = kGroups * (is_q ? p.q_parts : 1);
  const int heads = is_q ? p.hq : p.hkv;
  const int half = p.rot >> 1;

  // K and V of the cache write go to head h of the slot's page; a padding
  // token's go nowhere
  int64_t page_row = -1;
  if (kCache && !is_q && live) {
    const int64_t slot = p.slots[t];
    if (slot >= static_cast<int64_t>(p.num_blocks) * 16) {
      if (at == 0) raise_error(p.err, PA_DEV_ERR_SLOT);
    } else if (slot >= 0) {
      page_row = ((slot >> 4) * p.hkv * 16 + (slot & 15)) * kLanes + lane;
    }
  }
  if (kCache && part == p.q_parts + 1) {  // V: the rows as they are
    if (page_row < 0) return;
    const uint4* src = p.v + t * p.v_stride + lane;
    for (int h = first; h < heads; h += kRopeRows * step) {
      uint4 x[kRopeRows];
#pragma unroll
      for (int u = 0; u < kRopeRows; ++u)
        if (h + u * step < heads) x[u] = src[(h + u * step) * kLanes];
#pragma unroll
      for (int u = 0; u < kRopeRows; ++u)
        if (h + u * step < heads)
          p.v_pool[page_row + static_cast<int64_t>(h + u * step) * 16 * kLanes] = x[u];
    }
    return;
  }

  const uint4* src = (is_q ? p.q + t * p.q_stride : p.k + t * p.k_stride) + lane;
  uint4* dst = is_q ? p.q_out + t * p.q_out_stride + lane
               : !kCache ? p.k_out + t * p.k_out_stride + lane
               : page_row >= 0 ? p.k_pool + page_row : nullptr;
  const int64_t dst_step = kCache && !is_q ? 16 * kLanes : kLanes;
  const uint4* weight = is_q ? p.q_weight : p.k_weight;

  // the first rows are on their way while cos and sin are computed
  uint4 raw[kRopeRows];
  auto load = [&](int h) {
#pragma unroll
    for (int u = 0; u < kRopeRows; ++u)
      if (h + u * step < heads) raw[u] = src[(h + u * step) * kLanes];
  };
  if (live) {
    load(first);
    if (at < half) turn[mine][at] = turn_of(p.positions[t], p.inv_freq[at], p.factor);
  }
  const int e = lane * 8;
  const bool low = e < half;
  const bool rotated = e < p.rot;
  const int partner = rotated ? (low ? lane + half / 8 : lane - half / 8) : lane;
  const uint4 none = make_uint4(0, 0, 0, 0);
  const uint4 w = weight ? weight[lane] : none;
  const uint4 wp = weight ? weight[partner] : none;
  __syncthreads();
  if (!live) return;  // whole warps: none takes part in a shuffle below

  // A and B of this lane's dims; dims past rot go through with A = the weight, or as
  // they are (a product would flush subnormals and not keep a NaN's bits)
  const bool as_is = !rotated && !weight;
  float2 A[4], B[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 ws = weight ? unpack2(word(w, j)) : make_float2(1.f, 1.f);
    if (!rotated) {
      A[j] = ws;
      B[j] = make_float2(-0.f, -0.f);  // adding -0 keeps the sign of a zero
    } else if (kInterleaved) {  // a pair of dims, one angle
      const float2 cs = turn[mine][e / 2 + j];
      A[j] = make_float2(cs.x * ws.x, cs.x * ws.y);
      B[j] = make_float2(-cs.y * ws.y, cs.y * ws.x);
    } else {  // two dims, two angles; the sine's sign is that of the lane's half
      const float2 wo = weight ? unpack2(word(wp, j)) : make_float2(1.f, 1.f);
      const int i = (low ? e : e - half) + 2 * j;
      const float2 c0 = turn[mine][i], c1 = turn[mine][i + 1];
      A[j] = make_float2(c0.x * ws.x, c1.x * ws.y);
      B[j] = low ? make_float2(-c0.y * wo.x, -c1.y * wo.y) : make_float2(c0.y * wo.x, c1.y * wo.y);
    }
  }
  // every lane of a warp takes the same number of turns (shuffles)
  for (int base = 0; lead + base < heads; base += kRopeRows * step) {
    uint4 now[kRopeRows];
#pragma unroll
    for (int u = 0; u < kRopeRows; ++u) now[u] = raw[u];
    load(first + base + kRopeRows * step);
#pragma unroll
    for (int u = 0; u < kRopeRows; ++u) {
      if (lead + base + u * step >= heads) break;
      const int h = first + base + u * step;
      const uint4 x4 = h < heads ? now[u] : none;
      float r = 1.f;
      if (weight) {
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 x = unpack2(word(x4, j));
          sum = __ffma2_rn(x, x, sum);
        }
        float ss = sum.x + sum.y;
#pragma unroll
        for (int m = kLanes / 2; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
        r = rsqrtf(ss * (1.f / D) + p.eps);
      }
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t own = word(x4, j);
        uint32_t other = own;
        if (kInterleaved)
          other = __byte_perm(own, own, 0x1032);  // the pair's other dim
        else
          other = __shfl_sync(0xffffffffu, own, partner, kLanes);
        const float2 x = unpack2(own);
        // a product with 0 would turn an infinity past rot into NaN
        const float2 xo = rotated ? unpack2(other) : make_float2(0.f, 0.f);
        float2 y = __ffma2_rn(x, A[j], __fmul2_rn(xo, B[j]));
        if (weight) y = __fmul2_rn(y, make_float2(r, r));
        o[j] = as_is ? own : pack2(y);
      }
      if (h < heads && dst) dst[h * dst_step] = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

template <int D>
void launch_rope(const RopeParams& p, bool interleaved, bool cache, int grid, cudaStream_t st) {
  if (interleaved) {
    if (cache)
      rope_kernel<D, true, true><<<grid, kRopeThreads, 0, st>>>(p);
    else
      rope_kernel<D, true, false><<<grid, kRopeThreads, 0, st>>>(p);
  } else {
    if (cache)
      rope_kernel<D, false, true><<<grid, kRopeThreads, 0, st>>>(p);
    else
      rope_kernel<D, false, false><<<grid, kRopeThreads, 0, st>>>(p);
  }
}

// The q heads are split over CTAs while there are few of these, down to one row
// per lane group.
int run_rope(RopeParams& p, int head_dim, int layout, bool cache, int num_tokens, void* stream) {
  p.num_tokens = num_tokens;
  const int groups = kRopeTokenThreads / (head_dim / 8);
  const int most = (p.hq + groups - 1) / groups;
  const int blocks = (num_tokens + kRopeTokens - 1) / kRopeTokens;
  const int want = num_sms() * kRopeCtasPerSm / blocks;
  p.q_parts = std::max(1, std::min(want, most));
  p.parts = p.q_parts + (p.hkv > 0 ? 1 : 0) + (cache ? 1 : 0);
  const int64_t grid = static_cast<int64_t>(blocks) * p.parts;
  if (grid > 0x7fffffff) return PA_ERR_UNSUPPORTED;
  if (head_dim == 128)
    launch_rope<128>(p, layout == PA_ROPE_INTERLEAVED, cache, static_cast<int>(grid), as_stream(stream));
  else
    launch_rope<64>(p, layout == PA_ROPE_INTERLEAVED, cache, static_cast<int>(grid), as_stream(stream));
  return launch_status();
}

// Heads of a token times head_dim stay below 2^31, so a row's offset within a
// token is an int.
bool bad_rows(const void* x, int64_t stride, int heads, int head_dim) {
  return !x || !aligned16(x) || stride < static_cast<int64_t>(heads) * head_dim || stride % 8;
}

bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

int check_rotation(int head_dim, const int64_t* positions, const double* inv_freq, int rot_dim,
                   int layout) {
  if (layout != PA_ROPE_HALF && layout != PA_ROPE_INTERLEAVED) return PA_ERR_ARG;
  if (rot_dim < 0) return PA_ERR_ARG;
  if (rot_dim > head_dim) return PA_ERR_SHAPE;
  if (rot_dim % 16) return PA_ERR_UNSUPPORTED;
  // read an element at a time: the types' own alignment is enough
  if (rot_dim > 0 && (!positions || !inv_freq || !aligned8(positions) || !aligned8(inv_freq)))
    return PA_ERR_ARG;
  return PA_OK;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" {

int pa_rope(const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride,
            int32_t num_q_heads, const void* k, int64_t k_stride, void* k_out,
            int64_t k_out_stride, int32_t num_kv_heads, int32_t head_dim,
            const int64_t* positions, const double* inv_freq, int32_t rot_dim, int32_t layout,
            float factor, int32_t num_tokens, void* stream) {
  PA_NVTX_RANGE("pa_rope");
  if (head_dim != 64 && head_dim != 128) return PA_ERR_UNSUPPORTED;
  if (num_tokens < 0 || num_q_heads <= 0 || num_kv_heads < 0) return PA_ERR_ARG;
  if (num_q_heads > PA_ROPE_MAX_HEADS || num_kv_heads > PA_ROPE_MAX_HEADS)
    return PA_ERR_UNSUPPORTED;
  if (num_tokens == 0) return PA_OK;
  const int st = check_rotation(head_dim, positions, inv_freq, rot_dim, layout);
  if (st != PA_OK) return st;
  if (bad_rows(q, q_stride, num_q_heads, head_dim) ||
      bad_rows(q_out, q_out_stride, num_q_heads, head_dim))
    return PA_ERR_ARG;
  if (num_kv_heads > 0 && (bad_rows(k, k_stride, num_kv_heads, head_dim) ||
                           bad_rows(k_out, k_out_stride, num_kv_heads, head_dim)))
    return PA_ERR_ARG;
  RopeParams p = {};
  p.q = static_cast<const uint4*>(q);
  p.k = static_cast<const uint4*>(k);
  p.q_out = static_cast<uint4*>(q_out);
  p.k_out = static_cast<uint4*>(k_out);
  p.q_stride = q_stride / 8;
  p.k_stride = k_stride / 8;
  p.q_out_stride = q_out_stride / 8;
  p.k_out_stride = k_out_stride / 8;
  p.positions = positions;
  p.inv_freq = inv_freq;
  p.hq = num_q_heads;
  p.hkv = num_kv_heads;
  p.rot = rot_dim;
  p.factor = factor;
  return run_rope(p, head_dim, layout, false, num_tokens, stream);
}

int pa_rope_and_cache(const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride,
                      int32_t num_q_heads, const void* key, int64_t k_stride, const void* value,
                      int64_t v_stride, const void* q_weight, const void* k_weight, float eps,
                      const int64_t* positions, const double* inv_freq, int32_t rot_dim,
                      int32_t layout, float factor, void* k_pool, void* v_pool,
                      pa_pool_desc pool, const int64_t* slot_mapping, int32_t num_tokens,
                      void* stream) {
  PA_NVTX_RANGE("pa_rope_and_cache");
  int st = check_pool(pool);
  if (st != PA_OK) return st;
  if (num_tokens < 0 || num_q_heads <= 0) return PA_ERR_ARG;
  if (num_q_heads > PA_ROPE_MAX_HEADS || pool.num_kv_heads > PA_ROPE_MAX_HEADS)
    return PA_ERR_UNSUPPORTED;
  if (num_q_heads % pool.num_kv_heads) return PA_ERR_SHAPE;
  if (num_tokens == 0) return PA_OK;
  st = check_rotation(pool.head_dim, positions, inv_freq, rot_dim, layout);
  if (st != PA_OK) return st;
  if (bad_rows(q, q_stride, num_q_heads, pool.head_dim) ||
      bad_rows(q_out, q_out_stride, num_q_heads, pool.head_dim) ||
      bad_rows(key, k_stride, pool.num_kv_heads, pool.head_dim) ||
      bad_rows(value, v_stride, pool.num_kv_heads, pool.head_dim))
    return PA_ERR_ARG;
  if (!k_pool || !v_pool || !slot_mapping || !aligned16(k_pool) || !aligned16(v_pool) ||
      !aligned8(slot_mapping) || !aligned16(q_weight) || !aligned16(k_weight))
    return PA_ERR_ARG;
  if ((q_weight || k_weight) && !(eps >= 0.f)) return PA_ERR_ARG;
  RopeParams p = {};
  p.err = device_error_word();
  if (!p.err) return PA_ERR_CUDA;
  p.q = static_cast<const uint4*>(q);
  p.k = static_cast<const uint4*>(key);
  p.v = static_cast<const uint4*>(value);
  p.q_out = static_cast<uint4*>(q_out);
  p.k_pool = static_cast<uint4*>(k_pool);
  p.v_pool = static_cast<uint4*>(v_pool);
  p.q_stride = q_stride / 8;
  p.k_stride = k_stride / 8;
  p.v_stride = v_stride / 8;
  p.q_out_stride = q_out_stride / 8;
  p.q_weight = static_cast<const uint4*>(q_weight);
  p.k_weight = static_cast<const uint4*>(k_weight);
  p.positions = positions;
  p.inv_freq = inv_freq;
  p.slots = slot_mapping;
  p.hq = num_q_heads;
  p.hkv = pool.num_kv_heads;
  p.rot = rot_dim;
  p.num_blocks = pool.num_blocks;
  p.factor = factor;
  p.eps = eps;
  return run_rope(p, pool.head_dim, layout, true, num_tokens, stream);
}

int pa_rope_frequencies(int32_t rot_dim, double base, int32_t scaling, double scale,
                        double original_max_position, double low_turns, double high_turns,
                        double* inv_freq_host, double* factor_host) {
  if (rot_dim <= 0 || rot_dim % 2 || !inv_freq_host || !(base > 1.0)) return PA_ERR_ARG;
  if (scaling < PA_ROPE_SCALE_NONE || scaling > PA_ROPE_SCALE_RAMP) return PA_ERR_ARG;
  if (scaling != PA_ROPE_SCALE_NONE && !(scale > 0.0)) return PA_ERR_ARG;
  if (scaling == PA_ROPE_SCALE_BASE) {
    if (rot_dim == 2) return PA_ERR_ARG;
    base *= pow(scale, static_cast<double>(rot_dim) / (rot_dim - 2));
  }
  if (scaling == PA_ROPE_SCALE_RAMP && (!(high_turns > low_turns) || !(original_max_position > 0.0)))
    return PA_ERR_ARG;
  constexpr double kTwoPi = 6.283185307179586;
  for (int i = 0; i < rot_dim / 2; ++i) {
    const double f = pow(base, -2.0 * i / rot_dim);
    double out = f;
    if (scaling == PA_ROPE_SCALE_LINEAR) out = f / scale;
    if (scaling == PA_ROPE_SCALE_RAMP) {
      const double r = original_max_position * f / kTwoPi;
      const double keep = std::min(1.0, std::max(0.0, (r - low_turns) / (high_turns - low_turns)));
      out = f * keep + f / scale * (1.0 - keep);
    }
    inv_freq_host[i] = out;
  }
  if (factor_host)
    *factor_host = scaling == PA_ROPE_SCALE_RAMP && scale > 1.0 ? 0.1 * log(scale) + 1.0 : 1.0;
  return PA_OK;
}

}  // extern "C"
