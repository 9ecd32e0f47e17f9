// Rotary positions, norms per head and the cache write of the prepared K and V.
//
// One CTA works on the head rows of one token (or a part of them: blockIdx.y).
// A row of D dims belongs to D/8 neighbouring lanes, 16 bytes each, so a row is
// read and written with one coalesced access per lane and its norm is a
// shuffle reduction inside those lanes.  The token's cos and sin are computed
// once per CTA (one pair per thread) and then stay in registers, a lane always
// having the same dims whatever the head: per row there is nothing left but the
// load, the norm, the products and the store.  In the half layout a lane's
// partner dims are rot/16 lanes away and come by shuffle, in the interleaved
// layout a pair is inside the lane.
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

constexpr int kRopeThreads = 256;
constexpr int kRopeUnroll = 2;  // rows of a lane group in flight

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
  int hq, hkv, rows;  // rows of a token: q heads, K heads and, with the cache write, V heads
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

__device__ __forceinline__ void unpack8(uint4 w, float (&x)[8]) {
  x[0] = bf16lo(w.x);
  x[1] = bf16hi(w.x);
  x[2] = bf16lo(w.y);
  x[3] = bf16hi(w.y);
  x[4] = bf16lo(w.z);
  x[5] = bf16hi(w.z);
  x[6] = bf16lo(w.w);
  x[7] = bf16hi(w.w);
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

template <int D, bool kInterleaved, bool kCache>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kLanes = D / 8;                       // lanes of a row
  constexpr int kGroups = kRopeThreads / kLanes;      // rows in work at once
  __shared__ float2 turn[D / 2];
  // a decode plan launched after this kernel may start now (it reads only the
  // tables and lengths, and waits for this grid before it completes)
  if (kCache) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x % kLanes;
  const int group = threadIdx.x / kLanes;
  const int step = kGroups * gridDim.y;
  const int half = p.rot >> 1;

  int64_t slot = -1;
  if (kCache) {
    slot = p.slots[t];
    if (slot >= static_cast<int64_t>(p.num_blocks) * 16) {
      if (threadIdx.x == 0 && blockIdx.y == 0) raise_error(p.err, PA_DEV_ERR_SLOT);
      slot = -1;
    }
  }
  auto source = [&](int r) -> const uint4* {
    if (r < p.hq) return p.q + t * p.q_stride + r * kLanes + lane;
    if (!kCache || r < p.hq + p.hkv) return p.k + t * p.k_stride + (r - p.hq) * kLanes + lane;
    return p.v + t * p.v_stride + (r - p.hq - p.hkv) * kLanes + lane;
  };
  // Row r of the token goes to q_out, k_out or, in a pool, head g of its slot's
  // page; nullptr: a padding token's K and V.
  auto target = [&](int r) -> uint4* {
    if (r < p.hq) return p.q_out + t * p.q_out_stride + r * kLanes + lane;
    if (!kCache) return p.k_out + t * p.k_out_stride + (r - p.hq) * kLanes + lane;
    if (slot < 0) return nullptr;
    const bool is_k = r < p.hq + p.hkv;
    const int g = r - p.hq - (is_k ? 0 : p.hkv);
    const int64_t at = (((slot >> 4) * p.hkv + g) * 16 + (slot & 15)) * kLanes + lane;
    return (is_k ? p.k_pool : p.v_pool) + at;
  };

  // the first rows are on their way while cos and sin are computed
  int r0 = blockIdx.y * kGroups + group;
  uint4 raw[kRopeUnroll];
#pragma unroll
  for (int u = 0; u < kRopeUnroll; ++u)
    if (r0 + u * step < p.rows) raw[u] = *source(r0 + u * step);
  if (threadIdx.x < half)
    turn[threadIdx.x] = turn_of(p.positions[t], p.inv_freq[threadIdx.x], p.factor);
  __syncthreads();

  // This lane's cos and sin: eight pairs in the half layout (the sine's sign is
  // that of the lane's half), four in the interleaved one; (1, 0) past rot.
  constexpr int kPairs = kInterleaved ? 4 : 8;
  float c[kPairs], s[kPairs];
  const int e = lane * 8;
  const bool low = e < half;
  const bool rotated = e < p.rot;
  const int partner = rotated ? (low ? lane + half / 8 : lane - half / 8) : lane;
#pragma unroll
  for (int j = 0; j < kPairs; ++j) {
    const int i = kInterleaved ? e / 2 + j : (low ? e : e - half) + j;
    const float2 cs = rotated ? turn[i] : make_float2(1.f, 0.f);
    c[j] = cs.x;
    s[j] = kInterleaved || !low ? cs.y : -cs.y;
  }
  const uint4 none = make_uint4(0, 0, 0, 0);
  const uint4 wq = p.q_weight ? p.q_weight[lane] : none;
  const uint4 wk = p.k_weight ? p.k_weight[lane] : none;

  // every lane of a warp takes the same number of turns (shuffles)
  const int first = blockIdx.y * kGroups;
  for (int base = first; base < p.rows; base += kRopeUnroll * step, r0 += kRopeUnroll * step) {
    uint4 now[kRopeUnroll];
#pragma unroll
    for (int u = 0; u < kRopeUnroll; ++u) {
      now[u] = raw[u];
      const int next = r0 + (kRopeUnroll + u) * step;
      if (next < p.rows) raw[u] = *source(next);
    }
#pragma unroll
    for (int u = 0; u < kRopeUnroll; ++u) {
      const int r = r0 + u * step;
      const bool live = r < p.rows;
      const bool is_q = r < p.hq;
      const bool is_v = kCache && r >= p.hq + p.hkv;
      float x[8];
      unpack8(live ? now[u] : none, x);
      if (p.q_weight || p.k_weight) {
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = fmaf(x[j], x[j], sum);
#pragma unroll
        for (int m = kLanes / 2; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
        if (is_q ? p.q_weight != nullptr : p.k_weight != nullptr) {
          const float inv = rsqrtf(sum * (1.f / D) + p.eps);
          float w[8];
          unpack8(is_q ? wq : wk, w);
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] *= inv * w[j];
        }
      }
      float y[8];
      if (kInterleaved) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          y[2 * j] = x[2 * j] * c[j] - x[2 * j + 1] * s[j];
          y[2 * j + 1] = x[2 * j + 1] * c[j] + x[2 * j] * s[j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float other = __shfl_sync(0xffffffffu, x[j], partner, kLanes);
          y[j] = x[j] * c[j % kPairs] + other * s[j % kPairs];
        }
      }
      // dims past rot go through as they are: a product with 0 would turn an
      // infinity into NaN
      if (!rotated) {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = x[j];
      }
      uint4 o;
      o.x = pack2(y[0], y[1]);
      o.y = pack2(y[2], y[3]);
      o.z = pack2(y[4], y[5]);
      o.w = pack2(y[6], y[7]);
      if (is_v) o = now[u];  // V's bits, untouched
      if (live) {
        uint4* dst = target(r);
        if (dst) *dst = o;
      }
    }
  }
}

template <int D>
void launch_rope(const RopeParams& p, bool interleaved, bool cache, dim3 grid, cudaStream_t st) {
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

// A token's rows are split over CTAs while there are fewer CTAs than the device
// holds at once, down to one row per lane group.
int run_rope(RopeParams& p, int head_dim, int layout, bool cache, int num_tokens, void* stream) {
  p.rows = p.hq + (cache ? 2 : 1) * p.hkv;
  const int groups = kRopeThreads / (head_dim / 8);
  const int most = (p.rows + groups - 1) / groups;
  const int64_t want = (static_cast<int64_t>(num_sms()) * 8 + num_tokens - 1) / num_tokens;
  const dim3 grid(num_tokens, static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(want, most))));
  if (head_dim == 128)
    launch_rope<128>(p, layout == PA_ROPE_INTERLEAVED, cache, grid, as_stream(stream));
  else
    launch_rope<64>(p, layout == PA_ROPE_INTERLEAVED, cache, grid, as_stream(stream));
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
