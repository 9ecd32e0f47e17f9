// Eviction: choosing the heaviest cached tokens of every KV head and packing
// them.
//
// Choice (evict_select_kernel, one CTA per (sequence, head)): the weights become
// unsigned keys of the same order and stay in registers (up to 32 per thread);
// the key of the last token that fits is found bit by bit from the top -- a
// candidate threshold, a count of the keys at or above it, one barrier -- until
// a count hits the wanted number exactly or the bits run out.  As soon as no more
// keys share the threshold's bits than there are threads (after a dozen bits of a
// spread row), only those are looked at, one each.  Then every token above the
// threshold is kept, and of those at it the lowest indices.  A warp owns a run of
// tokens, so counts of ballots give each kept token its place in order without
// sorting.  A small CTA takes a row of up to 8192 tokens, so that several rows
// share an SM.  Longer rows, and any where there are few, are shared by a cluster
// of eight CTAs (evict_select_cluster_kernel): the same steps, two bits at a time,
// the counts of all warps sent through distributed shared memory.  Rows past
// 131072 tokens (evict_select_long_kernel) are read again for every eight bits,
// with a histogram per warp.
//
// Move (compact): rows of 16-byte chunks.  Into fresh blocks all rows move at
// once; in place a CTA takes one slice of the columns of one (sequence, head),
// K or V, and goes through its rows in order, a chunk of rows read before it is
// written: sources are never below their destinations, so a chunk's writes can
// only hit rows that were read.
//
// Bound: HBM for the move (each kept row read and written once); the choice is
// bound by its steps' latency.
#include <cooperative_groups.h>

#include <algorithm>

#include "../../include/pa_evict.h"
#include "common.cuh"
#include "internal.h"

namespace pa {
namespace {

// ---------------------------------------------------------------------------
// Choice
// ---------------------------------------------------------------------------
constexpr int kSelThreads = 1024;  // of the long rows' kernel
constexpr int kSelWarps = kSelThreads / 32;

struct SelectParams {
  const float* mass;
  int64_t mass_stride;
  const int32_t* context_lens;
  const int32_t* budgets;
  int sink, recent;
  int32_t* kept;
  int kept_stride;
  int32_t* new_lens;
  float* mass_out;
  int64_t mass_out_stride;
  int hkv;
  int most_len;   // tokens of a table
  unsigned int* err;
};

// What a row keeps: [0, sink) and [len - recent, len) whatever their weight, and
// `need` of the tokens between.
struct Choice {
  int len, keep, sink, recent, need;
};

__device__ __forceinline__ Choice choice_of(const SelectParams& p, int s, bool flag) {
  Choice c;
  c.len = p.context_lens[s];
  if (c.len < 0 || c.len > p.most_len || c.len > p.mass_stride) {
    if (flag) raise_error(p.err, PA_DEV_ERR_CONTEXT);
    c.len = 0;
  }
  const int64_t most = min(static_cast<int64_t>(p.kept_stride), p.mass_out_stride);
  c.keep = max(0, min(c.len, p.budgets[s]));
  if (c.keep > most) c.keep = static_cast<int>(most);
  c.sink = min(p.sink, c.keep);
  c.recent = min(p.recent, c.keep - c.sink);
  c.need = c.keep - c.sink - c.recent;
  return c;
}

// Keys in the order of the weights: NaN is the least (0), both zeros are alike.
// On the bits alone: comparisons of floats would take denormal weights for zeros.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x), size = b & 0x7fffffffu;
  if (size > 0x7f800000u) return 0;
  if (size == 0) return 0x80000000u;
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float weight_of(uint32_t key) {
  if (key == 0) return __uint_as_float(0x7fc00000u);
  return __uint_as_float((key & 0x80000000u) ? key & 0x7fffffffu : ~key);
}

// Sum over a CTA of `kWarps` warps of one number per thread; `slots` alternates
// between two arrays so that one barrier is enough.
template <int kWarps>
__device__ __forceinline__ int cta_sum(int x, int* slots, int warp, int lane) {
  const int w = __reduce_add_sync(0xffffffffu, x);
  if (lane == 0) slots[warp] = w;
  __syncthreads();
  return __reduce_add_sync(0xffffffffu, lane < kWarps ? slots[lane] : 0);
}

// Where this warp's kept tokens and ties begin: sums over the warps before it; and
// the sums over all.
template <int kWarps>
__device__ __forceinline__ int2 warps_before(int2 x, int2* slots, int warp, int lane, int2& all) {
  if (lane == 0) slots[warp] = x;
  __syncthreads();
  const int2 v = lane < kWarps ? slots[lane] : make_int2(0, 0);
  all = make_int2(__reduce_add_sync(0xffffffffu, v.x), __reduce_add_sync(0xffffffffu, v.y));
  return make_int2(__reduce_add_sync(0xffffffffu, lane < warp ? v.x : 0),
                   __reduce_add_sync(0xffffffffu, lane < warp ? v.y : 0));
}

// The kept tokens of a row, in order, from per-thread flags of one token each
// (`sure`: forced or above the threshold; `at`: at it), for tokens that follow
// one another along the lanes.  place and tie are the warp's running counts: kept
// tokens, and ties, before these.  `no_ties`: no token is at it.
__device__ __forceinline__ int place_of(bool sure, bool at, bool no_ties, int ties, int lane,
                                        int& place, int& tie) {
  const uint32_t below = (1u << lane) - 1u;
  bool keep = sure;
  if (!no_ties) {
    const uint32_t ats = __ballot_sync(0xffffffffu, at);
    keep = sure || (at && tie + __popc(ats & below) < ties);
    tie += __popc(ats);
  }
  const uint32_t keeps = __ballot_sync(0xffffffffu, keep);
  const int i = place + __popc(keeps & below);
  place += __popc(keeps);
  return keep ? i : -1;
}

// ITEMS: tokens per lane at most.  Lane l's item k of warp w is token
// (w * items + k) * 32 + l, items = ceil(len / THREADS).
template <int THREADS, int ITEMS>
__global__ void __launch_bounds__(THREADS, 768 / THREADS)
    evict_select_kernel(const __grid_constant__ SelectParams p) {
  constexpr int kWarps = THREADS / 32;
  __shared__ int sums[2][kWarps];
  __shared__ int2 bases[kWarps];
  __shared__ uint32_t close[THREADS];  // the keys that share the threshold's bits
  __shared__ int n_close;
  // the move may be set up now (it waits for this grid's end)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int row = blockIdx.x;
  const int s = row / p.hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Choice c = choice_of(p, s, row % p.hkv == 0 && tid == 0);
  if (row % p.hkv == 0 && tid == 0) p.new_lens[s] = c.keep;
  if (c.keep == 0) return;
  const float* mass = p.mass + row * p.mass_stride;
  const int items = (c.len + THREADS - 1) / THREADS;
  const int first = warp * items * 32 + lane;
  const int lo = c.sink, hi = c.len - c.recent;  // the tokens with a choice
  int32_t* kept = p.kept + static_cast<int64_t>(row) * p.kept_stride;
  float* out = p.mass_out + row * p.mass_out_stride;
  if (tid == 0) n_close = 0;
  // (every load is made, of the last token where there is none: then they all are
  // on their way at once)
  uint32_t key[ITEMS];
#pragma unroll
  for (int k = 0; k < ITEMS; ++k)
    key[k] = __float_as_uint(mass[min(first + 32 * min(k, items - 1), c.len - 1)]);
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) key[k] = key_of(__uint_as_float(key[k]));
  __syncthreads();  // all weights are read: in place, theirs may be overwritten
  // Tokens kept anyway have their places already; `open`: the others, whose key
  // counts (a key of 0 reaches no threshold).  Most warps have none of the former.
  uint32_t open = 0xffffffffu >> (32 - min(items, 32));
  if (warp * items * 32 < lo || (warp + 1) * items * 32 > hi) {
    open = 0;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
      const int t = first + 32 * k;
      if (k < items && t >= lo && t < hi) {
        open |= 1u << k;
      } else {
        if (k < items && t < c.len) {
          const int i = t < lo ? t : c.keep - (c.len - t);
          kept[i] = t;
          out[i] = weight_of(key[k]);
        }
        key[k] = 0;
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < ITEMS; ++k)
      if (k >= items) key[k] = 0;
  }
  if (c.need == 0) return;
  // The largest threshold that at least `need` keys reach.
  uint32_t bar = 0;
  int above = hi - lo;  // keys at or above the threshold (0: all with a choice)
  int over = 0;         // keys above all that share its bits so far
  if (c.need < hi - lo) {
    int b = 31;
    for (; b >= 0 && above != c.need && above - over > THREADS; --b) {
      const uint32_t cand = bar | (1u << b);
      int mine = 0;
#pragma unroll
      for (int k = 0; k < ITEMS; ++k) mine += key[k] >= cand;
      const int n = cta_sum<kWarps>(mine, sums[b & 1], warp, lane);
      if (n >= c.need) {
        bar = cand;
        above = n;
      } else {
        over = n;
      }
    }
    if (b >= 0 && above != c.need) {
      // the keys in [bar, bar + 2^(b + 1)), in any order: a warp's share of the
      // list at a time
      const uint32_t span = b == 31 ? 0xffffffffu : (2u << b) - 1u;
      uint32_t in = 0;
#pragma unroll
      for (int k = 0; k < ITEMS; ++k)
        if (key[k] - bar <= span) in |= open & (1u << k);
      const int n_in = __popc(in);
      int upto = n_in;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
      }
      int base = 0;
      if (lane == 31) base = atomicAdd(&n_close, upto);
      base = __shfl_sync(0xffffffffu, base, 31) + upto - n_in;
#pragma unroll
      for (int k = 0; k < ITEMS; ++k)
        if ((in >> k) & 1u) close[base++] = key[k];
      __syncthreads();
      const uint32_t mine = tid < n_close ? close[tid] : 0u;
      for (; b >= 0 && above != c.need; --b) {
        const uint32_t cand = bar | (1u << b);
        const int n = over + cta_sum<kWarps>(mine >= cand, sums[b & 1], warp, lane);
        if (n >= c.need) {
          bar = cand;
          above = n;
        }
      }
    }
  }
  // Above the threshold: kept; at it: the first ones in order, as many as fit (all
  // of them where the count was hit exactly: then they count as above).
  const bool exact = above == c.need;
  const uint32_t least = exact ? bar : bar + 1;  // (bar + 1 is 0 for no key there is)
  uint32_t sure = 0, at = 0;
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    if (key[k] >= least) sure |= 1u << k;
    if (key[k] == bar) at |= 1u << k;
  }
  sure &= open;
  at = exact ? 0u : at & open;
  const int2 mine = make_int2(__reduce_add_sync(0xffffffffu, __popc(sure)),
                              __reduce_add_sync(0xffffffffu, __popc(at)));
  int2 all;
  const int2 before = warps_before<kWarps>(mine, bases, warp, lane, all);
  const int ties = c.need - all.x;
  int place = c.sink + before.x + min(before.y, ties), tie = before.y;
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    if (k < items) {
      const int i = place_of((sure >> k) & 1u, (at >> k) & 1u, exact, ties, lane, place, tie);
      if (i >= 0) {
        kept[i] = first + 32 * k;
        out[i] = weight_of(key[k]);
      }
    }
  }
}

// A row shared by a cluster of eight CTAs: lane l's item k of the cluster's warp w
// is token (w * items + k) * 32 + l.
//
// Every warp sends its word of counts to every CTA and waits on an mbarrier of its
// own CTA for all warps' words: no fence, and no barrier of the cluster, in a step.
// Measured on 8 rows of 31337 tokens: 13.4 us; with the words stored and a barrier of
// the cluster in every step 17.8, the fences of those the largest stall.
// Two sets of words and mbarriers in turn are enough: a warp sends its word of step
// i + 2 when it has all words of step i + 1, and a warp sent that only after it read
// the words of step i.  No word is on its way to a CTA that ended: a CTA's last
// words are the last that are sent.
constexpr int kSelCluster = 8;

__device__ __forceinline__ uint32_t map_rank(uint32_t addr, int rank) {
  uint32_t x;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(x) : "r"(addr), "r"(rank));
  return x;
}
__device__ __forceinline__ void send_word(uint32_t dst, uint32_t word, uint32_t bar) {
  asm volatile(
      "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.u32 [%0], %1, [%2];" ::"r"(dst),
      "r"(word), "r"(bar)
      : "memory");
}

template <int THREADS, int ITEMS>
__global__ void __cluster_dims__(kSelCluster, 1, 1) __launch_bounds__(THREADS, 1)
    evict_select_cluster_kernel(const __grid_constant__ SelectParams p) {
  namespace cg = cooperative_groups;
  constexpr int kWarps = THREADS / 32 * kSelCluster;  // of the cluster
  static_assert(32 * ITEMS < 1024, "three counts of a warp share a word");
  __shared__ uint32_t counts[2][kWarps];  // every warp's, in every CTA; in turn
  __shared__ uint64_t arrived[2];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank());
  const int row = blockIdx.x / kSelCluster;
  const int s = row / p.hkv;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = rank * (THREADS / 32) + (tid >> 5);
  const bool lead = row % p.hkv == 0 && rank == 0 && tid == 0;
  const Choice c = choice_of(p, s, lead);
  if (lead) p.new_lens[s] = c.keep;
  if (c.keep == 0) return;  // the whole cluster
  const float* mass = p.mass + row * p.mass_stride;
  const int items = (c.len + 32 * kWarps - 1) / (32 * kWarps);
  const int first = warp * items * 32 + lane;
  const int lo = c.sink, hi = c.len - c.recent;
  int32_t* kept = p.kept + static_cast<int64_t>(row) * p.kept_stride;
  float* out = p.mass_out + row * p.mass_out_stride;
  if (tid == 0) {
    mbar_init(&arrived[0], 1);
    mbar_init(&arrived[1], 1);
    fence_barrier_init();
  }
  uint32_t key[ITEMS];
#pragma unroll
  for (int k = 0; k < ITEMS; ++k)
    key[k] = __float_as_uint(mass[min(first + 32 * min(k, items - 1), c.len - 1)]);
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) key[k] = key_of(__uint_as_float(key[k]));
  cluster.sync();  // all weights are read, and all CTAs have their mbarriers
  uint32_t open = 0;
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    const int t = first + 32 * k;
    if (k < items && t >= lo && t < hi) {
      open |= 1u << k;
    } else {
      if (k < items && t < c.len) {
        const int i = t < lo ? t : c.keep - (c.len - t);
        kept[i] = t;
        out[i] = weight_of(key[k]);
      }
      key[k] = 0;
    }
  }
  if (c.need == 0) return;
  // Every warp's word in every CTA (lane j sends to CTA j); null after a time-out.
  int turn = 0;
  auto exchange = [&](uint32_t mine) -> const uint32_t* {
    const int set = turn & 1;
    if (tid == 0) mbar_arrive_expect_tx(&arrived[set], kWarps * 4);
    if (lane < kSelCluster)
      send_word(map_rank(smem_u32(&counts[set][warp]), lane), mine,
                map_rank(smem_u32(&arrived[set]), lane));
    const bool ok = mbar_wait(&arrived[set], (turn >> 1) & 1, nullptr, p.err);
    ++turn;
    if (__all_sync(0xffffffffu, ok)) return counts[set];
    cluster.sync();  // nobody ends while another may still send
    return nullptr;
  };
  uint32_t bar = 0;
  int above = hi - lo;
  if (c.need < hi - lo) {
    for (int b = 30; b >= 0 && above != c.need; b -= 2) {
      const uint32_t cand = bar | (1u << b);
      int n1 = 0, n2 = 0, n3 = 0;
#pragma unroll
      for (int k = 0; k < ITEMS; ++k) {
        n1 += key[k] >= cand;
        n2 += key[k] >= cand + (1u << b);
        n3 += key[k] >= cand + (2u << b);
      }
      const uint32_t* words =
          exchange(__reduce_add_sync(0xffffffffu, n1 | n2 << 10 | n3 << 20));
      if (!words) return;
      n1 = n2 = n3 = 0;
      for (int w = lane; w < kWarps; w += 32) {
        const uint32_t x = words[w];
        n1 += x & 1023u;
        n2 += (x >> 10) & 1023u;
        n3 += x >> 20;
      }
      n1 = __reduce_add_sync(0xffffffffu, n1);
      n2 = __reduce_add_sync(0xffffffffu, n2);
      n3 = __reduce_add_sync(0xffffffffu, n3);
      const int steps = n3 >= c.need ? 3 : n2 >= c.need ? 2 : n1 >= c.need ? 1 : 0;
      bar += static_cast<uint32_t>(steps) << b;
      above = steps == 3 ? n3 : steps == 2 ? n2 : steps == 1 ? n1 : above;
    }
  }
  const bool exact = above == c.need;
  const uint32_t least = exact ? bar : bar + 1;
  uint32_t sure = 0, at = 0;
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    if (key[k] >= least) sure |= 1u << k;
    if (key[k] == bar) at |= 1u << k;
  }
  sure &= open;
  at = exact ? 0u : at & open;
  const uint32_t* words =
      exchange(__reduce_add_sync(0xffffffffu, __popc(sure) | __popc(at) << 16));
  if (!words) return;
  int before_sure = 0, before_at = 0, all_sure = 0;
  for (int w = lane; w < kWarps; w += 32) {
    const int x = words[w];
    all_sure += x & 0xffff;
    if (w < warp) {
      before_sure += x & 0xffff;
      before_at += x >> 16;
    }
  }
  all_sure = __reduce_add_sync(0xffffffffu, all_sure);
  before_sure = __reduce_add_sync(0xffffffffu, before_sure);
  before_at = __reduce_add_sync(0xffffffffu, before_at);
  const int ties = c.need - all_sure;
  int place = c.sink + before_sure + min(before_at, ties), tie = before_at;
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    if (k < items) {
      const int i = place_of((sure >> k) & 1u, (at >> k) & 1u, exact, ties, lane, place, tie);
      if (i >= 0) {
        kept[i] = first + 32 * k;
        out[i] = weight_of(key[k]);
      }
    }
  }
}

// Rows of any length: token k * 1024 + tid is thread tid's in turn k.
__global__ void __launch_bounds__(kSelThreads, 1) evict_select_long_kernel(
    const __grid_constant__ SelectParams p) {
  __shared__ int hist[kSelWarps][256];
  __shared__ int2 bases[2][kSelWarps];
  __shared__ uint32_t found[2];  // the digit, what is still needed within it
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int row = blockIdx.x;
  const int s = row / p.hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Choice c = choice_of(p, s, row % p.hkv == 0 && tid == 0);
  if (row % p.hkv == 0 && tid == 0) p.new_lens[s] = c.keep;
  if (c.keep == 0) return;
  const float* mass = p.mass + row * p.mass_stride;
  const int lo = c.sink, hi = c.len - c.recent;
  uint32_t bar = 0;
  int rem = c.need;  // still needed among the keys that share the digits so far
  if (c.need > 0 && c.need < hi - lo) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < kSelWarps * 256; i += kSelThreads) (&hist[0][0])[i] = 0;
      __syncthreads();
#pragma unroll 4
      for (int t = lo + tid; t < hi; t += kSelThreads) {
        const uint32_t k = key_of(mass[t]);
        if (shift == 24 || (k >> (shift + 8)) == (bar >> (shift + 8)))
          atomicAdd(&hist[warp][(k >> shift) & 255u], 1);
      }
      __syncthreads();
      if (tid < 256) {
        int n = 0;
        for (int w = 0; w < kSelWarps; ++w) n += hist[w][tid];
        hist[0][tid] = n;
      }
      __syncthreads();
      if (warp == 0) {
        // lane l: digits 255 - 8 l down to 248 - 8 l
        int n = 0;
        for (int j = 0; j < 8; ++j) n += hist[0][255 - 8 * lane - j];
        int upto = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += v;
        }
        int over = upto - n;  // keys of larger digits
        if (over < rem && upto >= rem) {
          for (int j = 0; j < 8; ++j) {
            const int d = 255 - 8 * lane - j, h = hist[0][d];
            if (over + h >= rem) {
              found[0] = d;
              found[1] = rem - over;
              break;
            }
            over += h;
          }
        }
      }
      __syncthreads();
      bar |= found[0] << shift;
      rem = static_cast<int>(found[1]);
    }
  }
  // Ties that fit: what the tokens surely kept leave of keep.
  int n_sure = 0;
  for (int t = lo + tid; t < hi; t += kSelThreads) n_sure += c.need > 0 && key_of(mass[t]) > bar;
  __syncthreads();
  n_sure = cta_sum<kSelWarps>(n_sure, hist[0], warp, lane);
  const int ties = c.need - n_sure;
  int32_t* kept = p.kept + static_cast<int64_t>(row) * p.kept_stride;
  float* out = p.mass_out + row * p.mass_out_stride;
  int done = 0, ties_done = 0;  // before this turn
  for (int t0 = 0, turn = 0; t0 < c.len; t0 += kSelThreads, ++turn) {
    const int t = t0 + tid;
    const uint32_t k = t < c.len ? key_of(mass[t]) : 0u;
    const bool open = t >= lo && t < hi && c.need > 0;
    const bool sure = t < c.len && (t < lo || t >= hi || (open && k > bar));
    const bool at = open && k == bar;
    const int2 mine = make_int2(__popc(__ballot_sync(0xffffffffu, sure)),
                                __popc(__ballot_sync(0xffffffffu, at)));
    int2 all;
    const int2 before = warps_before<kSelWarps>(mine, bases[turn & 1], warp, lane, all);
    int tie = ties_done + before.y;
    int place = done + before.x + min(tie, ties);
    const int i = place_of(sure, at, false, ties, lane, place, tie);
    if (i >= 0) {  // (i <= t: this turn's weights are read, later ones lie beyond)
      kept[i] = t;
      out[i] = weight_of(k);
    }
    done += all.x;
    ties_done += all.y;
  }
}

// ---------------------------------------------------------------------------
// Move
// ---------------------------------------------------------------------------
struct MoveParams {
  uint4* k_pool;
  uint4* v_pool;
  int num_blocks, hkv;
  const int32_t* tables;
  int max_blocks;
  const int32_t* new_tables;
  int new_max_blocks;
  const int32_t* base;
  const int32_t* kept;
  int64_t kept_seq, kept_head;  // strides
  int kept_stride;
  const int32_t* counts;
  int num_seqs;
  int parts;  // CTAs per (sequence, head)
  unsigned int* err;
};

// Flat pool row of a sequence's row `pos` for KV head g, or -1.
__device__ __forceinline__ int64_t pool_row(const MoveParams& p, const int32_t* table, int blocks,
                                            int64_t pos, int g) {
  if (pos < 0 || pos >= static_cast<int64_t>(blocks) * 16) {
    raise_error(p.err, PA_DEV_ERR_CONTEXT);
    return -1;
  }
  const int b = table[pos >> 4];
  if (b < 0 || b >= p.num_blocks) {
    raise_error(p.err, PA_DEV_ERR_BLOCK_ID);
    return -1;
  }
  return (static_cast<int64_t>(b) * p.hkv + g) * 16 + (pos & 15);
}

__device__ __forceinline__ int move_count(const MoveParams& p, int s, bool flag) {
  const int n = p.counts[s];
  if (n >= 0 && n <= p.kept_stride) return n;
  if (flag) raise_error(p.err, PA_DEV_ERR_CONTEXT);
  return n < 0 ? 0 : p.kept_stride;
}

// Into other blocks: a warp takes as many rows as two accesses of 16 bytes a lane
// cover; their first lanes look them up, then every row's K and V go at once.
// Measured on 48 sequences brought down to 1531 tokens (602 MB moved): four rows of
// D = 128 per warp 123 us with the choice, eight 136, sixteen 133; small CTAs (128
// threads) and many of them (64 per SM) 123, 16 per SM 129; a lane looking up a row
// each for 32 rows at a time 122, but 24 against 21 us on one long sequence.
constexpr int kMoveThreads = 128;
constexpr int kMoveSteps = 2;
__host__ __device__ constexpr int move_rows(int head_dim) {  // of a warp
  return kMoveSteps * 32 / (head_dim / 8);
}
__host__ __device__ constexpr int move_cta_rows(int head_dim) {
  return move_rows(head_dim) * (kMoveThreads / 32);
}

template <int D>
__global__ void __launch_bounds__(kMoveThreads) move_out_kernel(const __grid_constant__ MoveParams p) {
  constexpr int kLanes = D / 8;           // chunks of a row
  constexpr int kAtOnce = 32 / kLanes;    // rows a warp covers with one access
  constexpr int kSteps = kMoveSteps;
  constexpr int kMoveRows = move_rows(D), kMoveCtaRows = move_cta_rows(D);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int sg = blockIdx.x / p.parts, part = blockIdx.x % p.parts;
  const int s = sg / p.hkv, g = sg % p.hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = move_count(p, s, g == 0 && part == 0 && threadIdx.x == 0);
  const int base = p.base ? p.base[s] : 0;
  const int32_t* kept = p.kept + s * p.kept_seq + g * p.kept_head;
  const int32_t* table = p.tables + static_cast<int64_t>(s) * p.max_blocks;
  const int32_t* new_table = p.new_tables + static_cast<int64_t>(s) * p.new_max_blocks;
  for (int i0 = part * kMoveCtaRows + warp * kMoveRows; i0 < n; i0 += p.parts * kMoveCtaRows) {
    int64_t src = -1, dst = -1;
    const int i = i0 + lane;
    if (lane < kMoveRows && i < n) {
      src = pool_row(p, table, p.max_blocks, static_cast<int64_t>(base) + kept[i], g);
      dst = pool_row(p, new_table, p.new_max_blocks, static_cast<int64_t>(base) + i, g);
      if (src < 0 || dst < 0) src = dst = -1;
    }
    uint4 k[kSteps], v[kSteps];
    int64_t to[kSteps];
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      const int r = j * kAtOnce + lane / kLanes;
      const int64_t from = __shfl_sync(0xffffffffu, src, r);
      to[j] = __shfl_sync(0xffffffffu, dst, r);
      if (from >= 0) {
        k[j] = p.k_pool[from * kLanes + lane % kLanes];
        v[j] = p.v_pool[from * kLanes + lane % kLanes];
      }
    }
#pragma unroll
    for (int j = 0; j < kSteps; ++j)
      if (to[j] >= 0) {
        p.k_pool[to[j] * kLanes + lane % kLanes] = k[j];
        p.v_pool[to[j] * kLanes + lane % kLanes] = v[j];
      }
  }
}

// In place: blockIdx.x = ((sequence, head), slice); a slice is four 16-byte
// chunks of K's or V's rows.  Thread i of a turn takes rows i / 4, + 64, ...
// Measured with the choice: 48 sequences brought down to 1531 tokens 157 us (into other
// blocks 123), one of 31337 to 4096 57 us (19): a (sequence, head) has eight CTAs at
// D = 128, and a turn is a chain of dependent loads (list, table, row).
constexpr int kPlaceThreads = 256;
constexpr int kSliceLanes = 4;
constexpr int kPlaceUnroll = 4;

template <int D>
__global__ void __launch_bounds__(kPlaceThreads) move_in_place_kernel(
    const __grid_constant__ MoveParams p) {
  constexpr int kRowChunks = D / 8;
  constexpr int kSlices = kRowChunks / kSliceLanes;  // of K, and as many of V
  constexpr int kRows = kPlaceThreads / kSliceLanes;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int sg = blockIdx.x / (2 * kSlices), slice = blockIdx.x % (2 * kSlices);
  const int s = sg / p.hkv, g = sg % p.hkv;
  const int n = move_count(p, s, g == 0 && slice == 0 && threadIdx.x == 0);
  const int base = p.base ? p.base[s] : 0;
  const int32_t* kept = p.kept + s * p.kept_seq + g * p.kept_head;
  const int32_t* table = p.tables + static_cast<int64_t>(s) * p.max_blocks;
  uint4* pool = (slice < kSlices ? p.k_pool : p.v_pool) + (slice % kSlices) * kSliceLanes +
                threadIdx.x % kSliceLanes;
  const int r = threadIdx.x / kSliceLanes;
  for (int i0 = 0; i0 < n; i0 += kRows * kPlaceUnroll) {
    uint4 x[kPlaceUnroll];
    int64_t to[kPlaceUnroll];
#pragma unroll
    for (int u = 0; u < kPlaceUnroll; ++u) {
      const int i = i0 + u * kRows + r;
      to[u] = -1;
      if (i < n) {
        const int t = kept[i];
        if (t != i) {  // a token that stays is not touched
          const int64_t from = pool_row(p, table, p.max_blocks, static_cast<int64_t>(base) + t, g);
          to[u] = pool_row(p, table, p.max_blocks, static_cast<int64_t>(base) + i, g);
          if (from < 0) to[u] = -1;
          if (to[u] >= 0) x[u] = pool[from * kRowChunks];
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kPlaceUnroll; ++u)
      if (to[u] >= 0) pool[to[u] * kRowChunks] = x[u];
  }
}

template <typename F>
int launch_dependent(F kernel, int grid, int threads, const MoveParams& p, bool dependent,
                     cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = dependent ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, kernel, p) != cudaSuccess) {
    cudaGetLastError();
    return PA_ERR_CUDA;
  }
  return PA_OK;
}

// `dependent`: the kernel before is the choice, whose end the move waits for
// itself.
int run_move(MoveParams& p, int head_dim, bool dependent, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(p.num_seqs) * p.hkv;
  if (p.new_tables) {
    // enough CTAs to fill the device several times over, no more than the rows need
    const int cta_rows = move_cta_rows(head_dim);
    const int64_t most = (static_cast<int64_t>(p.kept_stride) + cta_rows - 1) / cta_rows;
    const int64_t want = (static_cast<int64_t>(num_sms()) * 64 + rows - 1) / rows;
    p.parts = static_cast<int>(std::max<int64_t>(1, std::min(most, want)));
    if (rows * p.parts > 0x7fffffff) return PA_ERR_UNSUPPORTED;
    const int grid = static_cast<int>(rows * p.parts);
    return head_dim == 128
               ? launch_dependent(move_out_kernel<128>, grid, kMoveThreads, p, dependent, stream)
               : launch_dependent(move_out_kernel<64>, grid, kMoveThreads, p, dependent, stream);
  }
  const int64_t grid = rows * 2 * (head_dim / 8 / kSliceLanes);
  if (grid > 0x7fffffff) return PA_ERR_UNSUPPORTED;
  return head_dim == 128
             ? launch_dependent(move_in_place_kernel<128>, static_cast<int>(grid), kPlaceThreads, p,
                                dependent, stream)
             : launch_dependent(move_in_place_kernel<64>, static_cast<int>(grid), kPlaceThreads, p,
                                dependent, stream);
}

template <int THREADS, int ITEMS>
int launch_select(const SelectParams& p, int rows, cudaStream_t stream) {
  evict_select_kernel<THREADS, ITEMS><<<rows, THREADS, 0, stream>>>(p);
  return launch_status();
}

template <int THREADS, int ITEMS>
int launch_select_cluster(const SelectParams& p, int rows, cudaStream_t stream) {
  evict_select_cluster_kernel<THREADS, ITEMS><<<rows * kSelCluster, THREADS, 0, stream>>>(p);
  return launch_status();
}

// Tokens of a table, an int.
int64_t table_tokens(int max_blocks) { return static_cast<int64_t>(max_blocks) * 16; }

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" {

int pa_evict(const float* mass, int64_t mass_stride, void* k_pool, void* v_pool, pa_pool_desc pool,
             const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* context_lens,
             const int32_t* budgets, int32_t sink, int32_t recent, const int32_t* new_tables,
             int32_t new_max_blocks, int32_t* kept, int32_t kept_stride, int32_t* new_lens,
             float* mass_out, int64_t mass_out_stride, int32_t num_seqs, void* stream) {
  PA_NVTX_RANGE("pa_evict");
  int st = check_pool(pool);
  if (st != PA_OK) return st;
  if (num_seqs < 0 || max_blocks_per_seq <= 0 || sink < 0 || recent < 0 || kept_stride <= 0 ||
      mass_stride < 0 || mass_out_stride < 0)
    return PA_ERR_ARG;
  if (num_seqs == 0) return PA_OK;
  if (!mass || !k_pool || !v_pool || !block_tables || !context_lens || !budgets || !kept ||
      !new_lens || !mass_out || new_lens == context_lens)
    return PA_ERR_ARG;
  if (!aligned16(k_pool) || !aligned16(v_pool)) return PA_ERR_ARG;
  if (new_tables && (new_max_blocks <= 0 || new_tables == block_tables)) return PA_ERR_ARG;
  if (mass_out == mass && mass_out_stride != mass_stride) return PA_ERR_ARG;
  const int64_t rows = static_cast<int64_t>(num_seqs) * pool.num_kv_heads;
  if (rows > 0x7fffffff / kSelCluster || table_tokens(max_blocks_per_seq) > (1 << 30)) return PA_ERR_UNSUPPORTED;
  SelectParams p = {};
  p.err = device_error_word();
  if (!p.err) return PA_ERR_CUDA;
  p.mass = mass;
  p.mass_stride = mass_stride;
  p.context_lens = context_lens;
  p.budgets = budgets;
  p.sink = sink;
  p.recent = recent;
  p.kept = kept;
  p.kept_stride = kept_stride;
  p.new_lens = new_lens;
  p.mass_out = mass_out;
  p.mass_out_stride = mass_out_stride;
  p.hkv = pool.num_kv_heads;
  p.most_len = static_cast<int>(table_tokens(max_blocks_per_seq));
  // the longest row there can be, and whether one CTA per row leaves most of the
  // device idle, decide the kernel
  const int64_t longest = std::min<int64_t>(p.most_len, mass_stride);
  const int r = static_cast<int>(rows);
  cudaStream_t cs = as_stream(stream);
  if (longest <= 8192 && rows * kSelCluster > 2 * num_sms())
    st = longest <= 2048 ? launch_select<256, 8>(p, r, cs) : launch_select<256, 32>(p, r, cs);
  else if (longest <= 8192)
    st = launch_select_cluster<256, 4>(p, r, cs);
  else if (longest <= 32768)
    st = launch_select_cluster<256, 16>(p, r, cs);
  else if (longest <= 131072)
    st = launch_select_cluster<1024, 16>(p, r, cs);
  else {
    evict_select_long_kernel<<<r, kSelThreads, 0, cs>>>(p);
    st = launch_status();
  }
  if (st != PA_OK) return st;
  MoveParams m = {};
  m.k_pool = static_cast<uint4*>(k_pool);
  m.v_pool = static_cast<uint4*>(v_pool);
  m.num_blocks = pool.num_blocks;
  m.hkv = pool.num_kv_heads;
  m.tables = block_tables;
  m.max_blocks = max_blocks_per_seq;
  m.new_tables = new_tables;
  m.new_max_blocks = new_max_blocks;
  m.kept = kept;
  m.kept_head = kept_stride;
  m.kept_seq = static_cast<int64_t>(kept_stride) * pool.num_kv_heads;
  m.kept_stride = kept_stride;
  m.counts = new_lens;
  m.num_seqs = num_seqs;
  m.err = p.err;
  return run_move(m, pool.head_dim, true, as_stream(stream));
}

int pa_compact_tokens(void* k_pool, void* v_pool, pa_pool_desc pool, const int32_t* block_tables,
                      int32_t max_blocks_per_seq, const int32_t* new_tables,
                      int32_t new_max_blocks, const int32_t* base, const int32_t* kept,
                      int32_t kept_heads, int32_t kept_stride, const int32_t* counts,
                      int32_t num_seqs, void* stream) {
  PA_NVTX_RANGE("pa_compact_tokens");
  const int st = check_pool(pool);
  if (st != PA_OK) return st;
  if (num_seqs < 0 || max_blocks_per_seq <= 0 || kept_stride < 0) return PA_ERR_ARG;
  if (kept_heads != 1 && kept_heads != pool.num_kv_heads) return PA_ERR_SHAPE;
  if (num_seqs == 0 || kept_stride == 0) return PA_OK;
  if (!k_pool || !v_pool || !block_tables || !kept || !counts) return PA_ERR_ARG;
  if (!aligned16(k_pool) || !aligned16(v_pool)) return PA_ERR_ARG;
  if (new_tables && (new_max_blocks <= 0 || new_tables == block_tables)) return PA_ERR_ARG;
  // a row's number within a list, and a turn's step past it, stay an int
  if (kept_stride > (1 << 30)) return PA_ERR_UNSUPPORTED;
  MoveParams m = {};
  m.err = device_error_word();
  if (!m.err) return PA_ERR_CUDA;
  m.k_pool = static_cast<uint4*>(k_pool);
  m.v_pool = static_cast<uint4*>(v_pool);
  m.num_blocks = pool.num_blocks;
  m.hkv = pool.num_kv_heads;
  m.tables = block_tables;
  m.max_blocks = max_blocks_per_seq;
  m.new_tables = new_tables;
  m.new_max_blocks = new_max_blocks;
  m.base = base;
  m.kept = kept;
  m.kept_head = kept_heads == 1 ? 0 : kept_stride;
  m.kept_seq = static_cast<int64_t>(kept_stride) * kept_heads;
  m.kept_stride = kept_stride;
  m.counts = counts;
  m.num_seqs = num_seqs;
  return run_move(m, pool.head_dim, false, as_stream(stream));
}

}  // extern "C"
