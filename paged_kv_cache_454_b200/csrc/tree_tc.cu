// Attention of drafted trees over the paged cache, on the 5th-generation tensor
// cores.
//
// The G = Hq/Hkv query heads of a sequence's n drafted tokens form rows (token,
// head), token-major; floor(128/G) tokens make one 128-row tile, and an item is
// (sequence, KV head, pass of up to two row tiles) over the sequence's key tiles
// of 128, half a tile (64 keys) per step:
//     S [128 x 64] = Q . K^T             (D/16 MMAs)
//     O [128 x D] += P . V               (4 MMAs of P_hi, 4 of P_lo)
// with fp32 accumulators in tensor memory; P = P_hi + P_lo, the weight rounded to
// bf16 and what that leaves rounded likewise, replaces its scores in
// tensor memory (per 16 keys: 8 columns of P_hi, 8 of P_lo) and is read there by
// the second product.
//
// Two streams of (row tile, key tile) run side by side, each with its own scores,
// accumulator and softmax warpgroup (a thread owns a row):
//   pair mode    (two row tiles): stream h takes row tile h, both take every key
//                tile; K and V are read once for up to 256 rows.
//   split mode   (one row tile): both take the same rows, stream h the key tiles
//                h, h+2, ...; their results meet by log-sum-exp at the end.
// A stream has two buffers of scores, one per half of a tile: while the softmax
// works on one half, the other's weights are multiplied and the half after that
// is scored (with one buffer of a whole tile, scores, softmax and product follow
// each other and the tensor cores idle half the time).  K and V have five slots of a
// tile at D = 128 (four: 111 against 96 us on 24 sequences of 32/32 heads, 480 against
// 407 on 48 of 64/8).  A thread takes its 64 scores into registers once and puts the
// weights back once: tensor memory answers between products, so every round trip to it
// waits.
//
// Work split: all items' key tiles, in order, are one line, on which a tile has
// places for its time and an item more in front of them for what it costs besides,
// and every CTA takes an equal stretch of it (each finds its start from the lengths
// by a scan of its own: no plan kernel, no queue).  An item inside one CTA's stretch
// is finished there; one that crosses a border leaves normalised fp32 partial
// rows and base-2 log-sum-exps in the workspace -- at most two items per CTA --
// and a second kernel, a programmatic dependent, merges them.
//
// Bound: for many rows the tensor cores (48 sequences of 64/8 heads and 7 to 63 drafted
// tokens over 300 to 16001: 406 to 430 us, 711 TFLOP/s without P_lo; their pipe is busy
// for 62% of the active cycles); for few the padding of their 128-row tiles (24
// sequences of 32/32 heads, 3 to 25 drafted: 95 us against 43 of HBM; tensor pipe 32%,
// DRAM 37%, one softmax warp of four at work); for one sequence the latency of two
// kernels (17 to 19 us).
//
// Roles (one CTA per SM): warp 0 copies K and V pages (one ring, K and V of a
// tile in turn), warps 1 and 2 issue the MMAs of one stream each (one warp for
// both left the tensor cores idle for a third of the time: what it does between
// two products is short, but every instruction of it waits among those of the
// softmax warps), warp 3 walks the stretch, publishes its units in a ring and
// copies their q, warps 4-11 are the two streams' softmax warpgroups.
// Every wait on an mbarrier is bounded.  The named barriers join softmax warps
// that go through the same units and steps whatever happens: after a time-out
// the data waits return at once and the unit ring still runs to its end.
#include <math_constants.h>

#include "../../include/pa_tree.h"
#include "draft_common.cuh"
#include "internal.h"

namespace pa {
namespace {

using namespace tc;

constexpr int kThreads = 384;
constexpr int kMaxCtas = 160;      // partial results are sized for this many
// Places on the line, near a fit of the CTAs' cycles to what they had, over six batches
// (a tile 3570 in split mode, 3950 in pair mode; an item 4100 and 12100 besides).  Five
// other ratios, the fit's own (9, 10; 10, 30) among them, time alike on seven batches
// within two runs' scatter: 93 to 98 us on 24 sequences of 32/32 heads and 358 to 403 on
// 48 of 64/8, these 93 to 94 and 361 to 366.
constexpr int kSplitTile = 5, kPairTile = 6;
constexpr int kSplitItem = 7, kPairItem = 22;  // in front of an item's tiles
constexpr int kMinPlaces = 10;                 // of a stretch
constexpr int kRegion = 128 * 128; // 128 rows x 128 bytes
constexpr int kQSlots = 2;
constexpr int kUnits = 4;          // ring of units
constexpr int kUnitReaders = 3 + 8;  // K/V, MMA and softmax warps
constexpr int kMaskRing = 16;
constexpr float kRaiseLog2 = 16.f; // raise the maximum in use only past 2^16
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kOCol = 256;    // S of stream h, half b at column 128 h + 64 b; O_h at 256 + 128 h

// Named barriers.
constexpr int kBarBoth = 1;    // all softmax warps
constexpr int kBarStream = 2;  // + h: the warps of one stream

template <int D>
struct Cfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kTileBytes = kHalves * kRegion;
  static constexpr int kSlots = D == 128 ? 5 : 8;  // K/V ring
  static constexpr int kPage = kHalves * 2048;     // bytes of a page
  static constexpr int kOffQ = 0;
  static constexpr int kOffKV = kQSlots * kTileBytes;
  static constexpr int kOffUnit = kOffKV + kSlots * kTileBytes;  // [kUnits] x 48 bytes
  static constexpr int kOffX = kOffUnit + kUnits * 48;  // [4][128] floats: exchanges of a row
  static constexpr int kOffBar = kOffX + 4 * 128 * 4;
  static constexpr int kNumBars = 2 * kQSlots + 2 * kSlots + 2 * kUnits + 12 + 3;
  // tensor-memory slot, abort flag, plan (seven words)
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kOffMask = kOffMisc + 40;
  static constexpr int kOffPoison = kOffMask + 4 * kMaskRing;  // [3 sets][2][4 words]
  static constexpr int kSmem = kOffPoison + 3 * 2 * 16;
  static_assert(kSmem <= 232448, "shared memory per CTA");
};

struct __align__(64) TreeParams {
  CUtensorMap tm_k;
  CUtensorMap tm_v;
  CUtensorMap tm_q;
  const int32_t* cu_q;
  const uint32_t* mask;  // the int64 words as pairs of 32-bit ones
  const int32_t* block_tables;
  const int32_t* context_lens;
  uint16_t* out;
  float* lse;
  int4* border;     // per CTA: the item that begins there and ends in a later CTA
  float* part_lse;  // [2 * CTA + (begun there)][part_rows]
  float* part_o;    // the same, [D]
  unsigned int* err;
  int total_q;
  int max_n;        // drafted tokens of a sequence at most
  int mask_words;   // 32-bit words of a mask row
  int max_blocks;
  int num_blocks;
  int hkv;
  int hq;
  int group;
  int tpt;          // tokens of a row tile
  Divisor by_pass;  // division by 2 tpt
  int num_seqs;
  int part_rows;    // 128 or 256
  float scale_log2;
};

// ---------------------------------------------------------------------------
// Sequences, items and units
// ---------------------------------------------------------------------------
struct Seq {
  int q0, n, L;
  int tiles, passes;  // tiles 0: nothing to do
};

__device__ __forceinline__ SeqRaw fetch_seq(const TreeParams& p, int s) {
  SeqRaw r;
  r.q0 = ld_i32(p.cu_q + s);
  r.q1 = ld_i32(p.cu_q + s + 1);
  r.L = ld_i32(p.context_lens + s);
  return r;
}

__device__ __forceinline__ Seq decode_seq(const TreeParams& p, const SeqRaw& r, unsigned* err) {
  Seq q;
  q.q0 = r.q0;
  q.n = r.q1 - r.q0;
  q.L = r.L;
  q.tiles = q.passes = 0;
  const bool ok = r.q0 >= 0 && r.q1 >= r.q0 && r.q1 <= p.total_q && q.n <= p.max_n &&
                  r.L >= q.n && r.L <= p.max_blocks * 16;
  if (!ok && err) raise_error(err, PA_DEV_ERR_CONTEXT);
  if (!ok || q.n == 0) return q;
  q.tiles = (r.L + 127) >> 7;
  q.passes = p.by_pass.quotient(q.n + 2 * p.tpt - 1);
  return q;
}

// Places on the line of one item of pass rp, as what lies in front of its tiles and
// each of them; and of a head (all passes but the last have two row tiles).
struct Places {
  int front, each;
};
__device__ __forceinline__ Places places_of(const Seq& q, int rp, int tpt) {
  return q.n - rp * 2 * tpt > tpt ? Places{kPairItem, kPairTile} : Places{kSplitItem, kSplitTile};
}
__device__ __forceinline__ int item_places(const Seq& q, const Places& w) {
  return w.front + w.each * q.tiles;
}
__device__ __forceinline__ long long head_places(const Seq& q, int tpt) {
  if (!q.tiles) return 0;
  return static_cast<long long>(q.passes - 1) * item_places(q, Places{kPairItem, kPairTile}) +
         item_places(q, places_of(q, q.passes - 1, tpt));
}
// Key tiles of an item that begin before a place of it.
__device__ __forceinline__ int tiles_before(int place, const Places& w) {
  return place <= w.front ? 0 : (place - w.front + w.each - 1) / w.each;
}

// A unit: one CTA's key tiles [tile0, tile0 + nt) of one item; nt 0: no more.
struct __align__(16) UnitWords {
  int s, g, rp, q0;
  int n, L, tile0, nt;
  int tiles, pad0, pad1, pad2;
};
static_assert(sizeof(UnitWords) == 48, "three 16-byte words");

struct Unit {
  int s, g, rp, q0, n, L, c;
  int i0;       // first token of the pass
  int tile0, nt, tiles;
  bool pair;    // two row tiles
};

// 32 keys' visibility for one row, from key c + rel on: cached ones (rel < 0) are
// seen, drafted ones by the row's mask (its first two words are at hand), ones
// past the context are not.
__device__ __forceinline__ uint32_t mask_word(const uint32_t* row, uint2 head, int j, int n) {
  if (j < 0) return 0xffffffffu;
  const int have = n - 32 * j;
  if (have <= 0) return 0;
  const uint32_t w = j == 0 ? head.x : j == 1 ? head.y : row[j];
  return have >= 32 ? w : w & ((1u << have) - 1u);
}
__device__ __forceinline__ uint32_t visible32(const uint32_t* row, uint2 head, int rel, int n) {
  const int j = rel >> 5;  // floor
  return __funnelshift_r(mask_word(row, head, j, n), mask_word(row, head, j + 1, n), rel & 31);
}

// 8 consecutive fp32 columns of this thread's TMEM lane, waits included.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float (&v)[8]) {
  uint32_t r[8];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n\t"
      "tcgen05.wait::st.sync.aligned;" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
      : "memory");
}

// Transposes, within every four lanes, the 4 x 4 16-byte words that are v[0..3] of
// each: lane j's v[i] becomes lane i's v[j].
__device__ __forceinline__ void transpose4(uint4 (&v)[4], int lane) {
#pragma unroll
  for (int b = 1; b <= 2; b <<= 1) {
    const bool up = lane & b;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k & b) continue;
      const uint4 x = up ? v[k] : v[k | b];
      uint4 y;
      y.x = __shfl_xor_sync(0xffffffffu, x.x, b);
      y.y = __shfl_xor_sync(0xffffffffu, x.y, b);
      y.z = __shfl_xor_sync(0xffffffffu, x.z, b);
      y.w = __shfl_xor_sync(0xffffffffu, x.w, b);
      if (up)
        v[k] = y;
      else
        v[k | b] = y;
    }
  }
}

__device__ __forceinline__ bool nonfinite_pair(uint32_t w) {
  return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

// ---------------------------------------------------------------------------
// The kernel
// ---------------------------------------------------------------------------
template <int D>
__global__ void __launch_bounds__(kThreads, 1) tree_tc_kernel(const __grid_constant__ TreeParams p) {
  using C = Cfg<D>;
  // (bit 13 of the instruction descriptor: the first operand is negated)
  const uint32_t idesc_s = idesc_bf16_f32(128, 64, false, false) | (p.scale_log2 < 0.f ? 1u << 13 : 0u);
  constexpr uint32_t kIdescO = idesc_bf16_f32(128, D, false, true);
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t sbase = smem_u32(smem);
  UnitWords* units = reinterpret_cast<UnitWords*>(smem + C::kOffUnit);
  float* xbuf = reinterpret_cast<float*>(smem + C::kOffX);
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* q_empty = q_full + kQSlots;
  uint64_t* kv_full = q_empty + kQSlots;   // ring position 2t: K of tile t, 2t + 1: V
  uint64_t* kv_empty = kv_full + C::kSlots;
  uint64_t* u_full = kv_empty + C::kSlots;
  uint64_t* u_empty = u_full + kUnits;
  uint64_t* s_full = u_empty + kUnits;  // [stream][half]: scores ready
  uint64_t* p_full = s_full + 4;        // weights written back
  uint64_t* pv_done = p_full + 4;       // P.V complete
  uint64_t* o_free = pv_done + 4;       // both accumulators of a unit read out, and
                                        // both MMA warps past the unit's wait for it
  uint64_t* drain = o_free + 1;         // per stream
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  // where this CTA begins: sequence, its q0, q1 and length, head, pass, place
  volatile int* plan = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 8);
  // loaded pages of key tile t, in slot t % kMaskRing
  volatile uint32_t* kmask = reinterpret_cast<volatile uint32_t*>(smem + C::kOffMask);
  // drafted tokens of a tile whose V is not finite: [set: stream 0, stream 1,
  // both][in turn][key / 32]
  volatile uint32_t* poison_s = reinterpret_cast<volatile uint32_t*>(smem + C::kOffPoison);
  static_assert(C::kOffUnit % 16 == 0 && C::kOffMisc % 8 == 0, "alignment of the words");

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (sbase & 1023u) {  // the swizzled tiles need it, and the compiler gives it
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (tid == 0) {
      raise_error(p.err, PA_DEV_ERR_TIMEOUT);
      p.border[blockIdx.x] = make_int4(-1, 0, 0, 0);
    }
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < kQSlots; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 2);  // one arrival per stream
    }
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 2);
    }
    for (int i = 0; i < kUnits; ++i) {
      mbar_init(&u_full[i], 1);
      mbar_init(&u_empty[i], kUnitReaders);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);  // one arrival per warp of the stream
      mbar_init(&pv_done[i], 1);
    }
    mbar_init(&drain[0], 1);
    mbar_init(&drain[1], 1);
    mbar_init(o_free, 8 + 2);  // softmax warps, and the MMA warps past their wait
    *abort_flag = 0;
    prefetch_tmap(&p.tm_k);
    prefetch_tmap(&p.tm_v);
    prefetch_tmap(&p.tm_q);
  }
  if (warp == 1) tmem_alloc(tmem_slot, kTmemCols);
  // This kernel may have been set up while the one before it ran; it reads nothing
  // before that one's end, the lengths among it (without the wait their last write need
  // not be visible, and CTAs that read different ones would not agree on the line).  The
  // merge kernel may be set up now, not sooner: whatever starts early overlaps one
  // kernel only, the one before it.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // Where this CTA's stretch begins.  Thread i sums a run of sequences, a scan
  // over the threads places the runs on the line, and the thread whose run holds
  // the CTA's first place finds it there.
  long long chunk, total;
  {
    const int per = (p.num_seqs + kThreads - 1) / kThreads;
    const int s_lo = min(tid * per, p.num_seqs), s_hi = min(s_lo + per, p.num_seqs);
    long long mine = 0;
    SeqRaw raw = {};
    Seq q = {};
    for (int s = s_lo; s < s_hi; ++s) {
      raw = fetch_seq(p, s);
      q = decode_seq(p, raw, blockIdx.x == 0 ? p.err : nullptr);
      mine += p.hkv * head_places(q, p.tpt);
    }
    const long long before =
        cta_scan<kThreads / 32>(mine, reinterpret_cast<long long*>(xbuf), total);
    chunk = quotient(total + gridDim.x - 1, gridDim.x);
    if (chunk < kMinPlaces) chunk = kMinPlaces;
    const long long begin = chunk * blockIdx.x;
    if (begin >= before && begin < before + mine) {
      long long at = begin - before;
      int s = s_lo;
      if (per > 1)
        for (; s < s_hi; ++s) {
          raw = fetch_seq(p, s);
          q = decode_seq(p, raw, nullptr);
          const long long places = p.hkv * head_places(q, p.tpt);
          if (at < places) break;
          at -= places;
        }
      const long long head = head_places(q, p.tpt);
      const int g = static_cast<int>(quotient(at, head));
      const long long rest = at - g * head;
      const int whole = item_places(q, Places{kPairItem, kPairTile});
      const int rp = static_cast<int>(min(quotient(rest, whole), static_cast<long long>(q.passes - 1)));
      plan[0] = s;
      plan[1] = raw.q0;
      plan[2] = raw.q1;
      plan[3] = raw.L;
      plan[4] = g;
      plan[5] = rp;
      plan[6] = static_cast<int>(rest - static_cast<long long>(rp) * whole);
    }
  }
  fence_barrier_init();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int rows_box = p.tpt * p.group;

  // The next unit of the ring, for a whole warp.  Its waits do
  // not heed the abort flag (every role takes every unit) and outlast those that
  // set it.
  uint32_t u_at = 0;
  Unit u;
  auto next_unit = [&]() -> bool {
    const int slot = u_at % kUnits;
    if (!ring_wait(&u_full[slot], (u_at / kUnits) & 1, p.err)) return false;
    const int4* src = reinterpret_cast<const int4*>(&units[slot]);
    const int4 a = src[0], b = src[1];
    u.s = a.x;
    u.g = a.y;
    u.rp = a.z;
    u.q0 = a.w;
    u.n = b.x;
    u.L = b.y;
    u.tile0 = b.z;
    u.nt = b.w;
    u.tiles = units[slot].tiles;
    u.c = u.L - u.n;
    u.i0 = u.rp * 2 * p.tpt;
    u.pair = u.n - u.i0 > p.tpt;
    __syncwarp();
    if (lane == 0) mbar_arrive(&u_empty[slot]);
    ++u_at;
    return u.nt > 0;
  };

  if (warp == 3) {
    // ====== the walk along the stretch, its border, and the q producer ======
    uint32_t qi = 0;
    const long long begin = chunk * blockIdx.x;
    long long left = total - begin < chunk ? total - begin : chunk;  // places still to take
    long long at = begin;
    int4 border = make_int4(-1, 0, 0, 0);
    int s = 0, g = 0, rp = 0, place = 0;
    Seq cur = {};
    SeqRaw next = {};
    auto enter = [&](const SeqRaw& r) {
      cur = decode_seq(p, r, nullptr);
      if (s + 1 < p.num_seqs) next = fetch_seq(p, s + 1);
    };
    if (left > 0) {
      s = plan[0];
      enter(SeqRaw{plan[1], plan[2], plan[3]});
      g = plan[4];
      rp = plan[5];
      place = plan[6];
    }
    while (true) {
      UnitWords w = {};
      while (left > 0) {  // the next stretch of places with a key tile among them
        const Places w_of = places_of(cur, rp, p.tpt);
        const int all = item_places(cur, w_of), each = w_of.each;
        const int take = left < all - place ? static_cast<int>(left) : all - place;
        const int t0 = tiles_before(place, w_of), t1 = tiles_before(place + take, w_of);
        w.s = s;
        w.g = g;
        w.rp = rp;
        w.q0 = cur.q0;
        w.n = cur.n;
        w.L = cur.L;
        w.tile0 = t0;
        w.nt = t1 - t0;
        w.tiles = cur.tiles;
        if (t0 == 0 && t1 > 0 && t1 < cur.tiles)  // ends in a later CTA
          border = make_int4(s, g, rp, min(static_cast<int>(gridDim.x) - 1,
                                           static_cast<int>(quotient(at - place + all - each, chunk))));
        left -= take;
        at += take;
        place += take;
        if (place == all) {
          place = 0;
          if (++rp == cur.passes) {
            rp = 0;
            if (++g == p.hkv) {
              g = 0;
              while (left > 0 && s + 1 < p.num_seqs) {
                const SeqRaw r = next;
                ++s;
                enter(r);
                if (cur.tiles > 0) break;
              }
            }
          }
        }
        if (w.nt > 0) break;
      }
      const int slot = u_at % kUnits;
      if (!ring_wait(&u_empty[slot], ((u_at / kUnits) & 1) ^ 1, p.err)) break;
      if (lane == 0) {
        units[slot] = w;
        mbar_arrive(&u_full[slot]);
      }
      __syncwarp();
      ++u_at;
      if (w.nt == 0) break;
      const int i0 = w.rp * 2 * p.tpt;
      const int tiles = w.n - i0 > p.tpt ? 2 : 1;
      for (int h = 0; h < tiles; ++h) {
        const int qs = qi % kQSlots;
        mbar_wait(&q_empty[qs], ((qi / kQSlots) & 1) ^ 1, abort_flag, p.err);
        if (__any_sync(0xffffffffu, *abort_flag)) break;
        if (lane == 0) {
          const uint32_t dst = sbase + C::kOffQ + qs * C::kTileBytes;
          const int token = w.q0 + i0 + h * p.tpt;
          mbar_arrive_expect_tx(&q_full[qs], C::kHalves * rows_box * 128);
          tma_load_3d(dst, &p.tm_q, 0, w.g * p.group, token, &q_full[qs]);
          if (D == 128) tma_load_3d(dst + kRegion, &p.tm_q, 64, w.g * p.group, token, &q_full[qs]);
        }
        __syncwarp();
        ++qi;
      }
    }
    if (lane == 0) p.border[blockIdx.x] = border;
    if (*abort_flag && lane == 0)
      for (uint32_t w = qi > kQSlots ? qi - kQSlots : 0; w < qi; ++w)
        mbar_wait(&q_full[w % kQSlots], (w / kQSlots) & 1, nullptr, p.err);
  } else if (warp == 0) {
    // ======================== K and V producer ========================
    const uint32_t ubase = __shfl_sync(0xffffffffu, sbase, 0);
    uint32_t pos = 0, kt = 0;
    int slot = 0;
    uint32_t phase = 0;
    while (next_unit()) {
      const int32_t* table = p.block_tables + static_cast<int64_t>(u.s) * p.max_blocks;
      const int blocks = (u.L + 15) >> 4;
      // block-table entries, four tiles at a time: this group's and the next's
      auto entries = [&](int tile) {
        const int b = tile * 8 + lane;
        return b < blocks ? ld_i32(table + b) : -1;
      };
      int ent = entries(u.tile0), ent_next = entries(u.tile0 + 4);
      for (int j = 0; j < u.nt; ++j, ++kt) {
        if (j > 0 && (j & 3) == 0) {
          ent = ent_next;
          ent_next = entries(u.tile0 + j + 4);
        }
        int pb = __shfl_sync(0xffffffffu, ent, (j & 3) * 8 + (lane & 7));
        const bool wanted = lane < 8 && (u.tile0 + j) * 8 + lane < blocks;
        if (wanted && (pb < 0 || pb >= p.num_blocks)) {
          raise_error(p.err, PA_DEV_ERR_BLOCK_ID);
          pb = -1;
        }
        const unsigned vm = __ballot_sync(0xffffffffu, wanted && pb >= 0);
        const int row = (pb * p.hkv + u.g) * 16;
        int y[8];
#pragma unroll
        for (int pg = 0; pg < 8; ++pg) y[pg] = __shfl_sync(0xffffffffu, row, pg);
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          mbar_wait(&kv_empty[slot], phase ^ 1, abort_flag, p.err);
          if (!__any_sync(0xffffffffu, *abort_flag)) {
            if (lane == 0) {
              if (v == 0) kmask[kt % kMaskRing] = vm;
              mbar_arrive_expect_tx(&kv_full[slot], __popc(vm) * C::kPage);
            }
            __syncwarp();
            const uint32_t dst = ubase + C::kOffKV + slot * C::kTileBytes;
            if (elect_one()) {
#pragma unroll
              for (int pg = 0; pg < 8; ++pg) {
                if ((vm >> pg) & 1u) {
                  if (v == 0) {
                    KPage<D>::load(dst + pg * C::kPage, &p.tm_k, y[pg], &kv_full[slot]);
                  } else {  // a page's 64-dim halves next to each other, 16 rows each
                    if (D == 128)
                      tma_load_3d(dst + pg * C::kPage, &p.tm_v, 0, y[pg], 0, &kv_full[slot]);
                    else
                      tma_load_2d(dst + pg * C::kPage, &p.tm_v, 0, y[pg], &kv_full[slot]);
                  }
                }
              }
            }
            __syncwarp();
            ++pos;
          }
          if (++slot == C::kSlots) {
            slot = 0;
            phase ^= 1;
          }
        }
      }
    }
    if (*abort_flag && lane == 0)  // the copies in flight land before the CTA ends
      for (uint32_t w = pos > C::kSlots ? pos - C::kSlots : 0; w < pos; ++w)
        mbar_wait(&kv_full[w % C::kSlots], (w / C::kSlots) & 1, nullptr, p.err);
  } else if (warp < 3) {
    // ============================= MMA ==============================
    // Warp 1 + h issues stream h's products.  Step x (half x % 2 of the stream's
    // tile x / 2) is scored when the P.V of step x - 2 has read its weights:
    //     S(0), S(1), P.V(0), S(2), P.V(1), S(3), ...
    // The whole warp goes along with the same values and one lane issues, so the
    // descriptors stay in uniform registers.
    const int h = warp - 1;
    const uint32_t ubase = __shfl_sync(0xffffffffu, sbase, 0);
    const uint32_t utmem = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t dq0 = smem_desc_sw128(ubase + C::kOffQ, 16, 1024);
    const uint64_t dk0 = smem_desc_sw128(ubase + C::kOffKV, 16, KPage<D>::kGroup);
    const uint64_t dv0 = smem_desc_sw128(ubase + C::kOffKV, 2048, 1024);
    const uint32_t s_col = utmem + h * 128, o_col = utmem + kOCol + h * 128;
    uint32_t cnt = 0;   // this stream's tiles before the unit
    uint32_t qi = 0, unit = 0, kt0 = 0;
    // Both streams wait for every ring position and every q tile, in order, and both
    // arrive for each: with a commit for what they read, at once for what is the other
    // stream's.  A stream that left the other's out could find a slot's barrier still
    // in the phase before its own, whose parity is that of the phase before that one:
    // its wait would end at once.
    uint32_t kv_at = 0;  // positions waited for
    auto kv_wait = [&](uint32_t pos) {
      mbar_wait(&kv_full[pos % C::kSlots], (pos / C::kSlots) & 1, abort_flag, p.err);
    };
    auto kv_pass = [&](uint32_t pos) {  // up to pos, which are the other stream's
      for (; kv_at < pos; ++kv_at) {
        kv_wait(kv_at);
        if (lane == 0) mbar_arrive(&kv_empty[kv_at % C::kSlots]);
      }
    };
    auto kv_take = [&](uint32_t pos) {
      kv_pass(pos);
      kv_wait(pos);
      kv_at = pos + 1;
    };
    auto q_wait = [&](uint32_t q) {
      mbar_wait(&q_full[q % kQSlots], (q / kQSlots) & 1, abort_flag, p.err);
    };
    auto q_pass = [&](uint32_t q) {
      q_wait(q);
      if (lane == 0) mbar_arrive(&q_empty[q % kQSlots]);
    };
    while (next_unit()) {
      const bool pair = __shfl_sync(0xffffffffu, u.pair ? 1 : 0, 0);
      const int nt = __shfl_sync(0xffffffffu, u.nt, 0);
      const int tiles = pair ? nt : (nt - h + 1) >> 1;
      const uint32_t qq = pair ? qi + h : qi;
      const int qs = qq % kQSlots;
      const uint64_t qa = desc_add(dq0, qs * C::kTileBytes);
      auto position = [&](int x) -> uint32_t {  // ring position of a step's K
        return 2 * (kt0 + (pair ? x >> 1 : 2 * (x >> 1) + h));
      };
      auto scores = [&](int x) {
        const int half = x & 1;
        const uint32_t kpos = position(x);
        const int ks = kpos % C::kSlots;
        if (half == 0) kv_take(kpos);
        // the buffer's last weights are read: P.V of step x - 2
        mbar_wait(&pv_done[2 * h + half], ((cnt + (x >> 1)) & 1) ^ 1, abort_flag, p.err);
        if (__any_sync(0xffffffffu, *abort_flag)) return;
        tc_fence_after();
        const uint64_t kb = desc_add(dk0, ks * C::kTileBytes + half * 4 * C::kPage);
        if (elect_one()) {
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            const uint32_t off = (i >> 2) * kRegion + (i & 3) * 32;
            umma_ss(s_col + 64 * half, desc_add(qa, off), desc_add(kb, KPage<D>::dims16(i)), idesc_s,
                    i > 0 ? 1u : 0u);
          }
          umma_commit(&s_full[2 * h + half]);
          if (half) umma_commit(&kv_empty[ks]);
          if (x == 2 * tiles - 1) umma_commit(&q_empty[qs]);
        }
        __syncwarp();
      };
      if (pair && h == 1) q_pass(qi);
      if (tiles == 0) q_pass(qq);
      if (tiles > 0) {
        q_wait(qq);
        scores(0);
        scores(1);
      }
      // Every unit's, and the next phase ends only when both MMA warps have passed this
      // wait: a stream without a tile in a unit is not waited for otherwise, and one that
      // came a unit late would take the parity of the phase it waits for for that of the
      // next and wait for a unit that needs it.
      mbar_wait(o_free, (unit & 1) ^ 1, abort_flag, p.err);
      if (lane == 0) mbar_arrive(o_free);
      for (int x = 0; x < 2 * tiles; ++x) {
        const int half = x & 1;
        const uint32_t vpos = position(x) + 1;
        const int vs = vpos % C::kSlots;
        if (half == 0) kv_take(vpos);
        mbar_wait(&p_full[2 * h + half], (cnt + (x >> 1)) & 1, abort_flag, p.err);
        if (__any_sync(0xffffffffu, *abort_flag)) continue;
        tc_fence_after();
        const uint64_t vb = desc_add(dv0, vs * C::kTileBytes + half * 4 * C::kPage);
        const uint32_t pc = s_col + 64 * half;
        if (elect_one()) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            umma_ts(o_col, pc + 16 * i, desc_add(vb, i * C::kPage), kIdescO,
                    x == 0 && i == 0 ? 0u : 1u);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            umma_ts(o_col, pc + 16 * i + 8, desc_add(vb, i * C::kPage), kIdescO, 1u);
          umma_commit(&pv_done[2 * h + half]);
          if (half) umma_commit(&kv_empty[vs]);
        }
        __syncwarp();
        if (x + 2 < 2 * tiles) scores(x + 2);
      }
      kv_pass(2 * (kt0 + nt));
      if (pair && h == 0) q_pass(qi + 1);
      qi += pair ? 2 : 1;
      cnt += tiles;
      ++unit;
      kt0 += nt;
    }
    if (elect_one()) umma_commit(&drain[h]);
    __syncwarp();
    mbar_wait(&drain[h], 0, nullptr, p.err);
  } else {
    // ============================ softmax ============================
    const int h = (warp - 4) >> 2;  // stream
    const int q4 = warp & 3;
    const int r = q4 * 32 + lane;  // row of the tile, TMEM lane
    const uint32_t lane_addr = static_cast<uint32_t>(q4 * 32) << 16;
    const uint32_t srow = tmem + lane_addr + h * 128;
    const uint32_t ocol = tmem + lane_addr + kOCol + h * 128;
    const int ti = r / p.group;  // token of this row within its tile
    // (a negative scale's sign is in the scores; 0 becomes the smallest number there
    // is, which keeps infinities)
    const float sc = p.scale_log2 == 0.f ? 1.2e-38f : fabsf(p.scale_log2);
    const float2 sc2 = make_float2(sc, sc);
    const float2 neg1 = make_float2(-1.f, -1.f);
    uint32_t cnt = 0;  // this stream's tiles
    uint32_t kt0 = 0;  // ring number of the unit's first tile
    // Tail tiles so far: two records of them are in use in turn, so one is only
    // written again when everybody has passed the other's barrier.
    uint32_t split_tails = 0, pair_tails = 0;
    while (true) {
      // (the unit's slot is kept to the unit's end, and what is seldom needed is
      // read there when it is: the registers are the scores')
      const int slot = u_at % kUnits;
      if (!ring_wait(&u_full[slot], (u_at / kUnits) & 1, p.err)) break;
      const volatile UnitWords* U = &units[slot];
      const int nt = U->nt;
      if (nt == 0) break;
      ++u_at;
      const int n = U->n, c = U->L - n, tile0 = U->tile0;
      const int pass0 = U->rp * 2 * p.tpt;
      const bool pair = n - pass0 > p.tpt;
      const int token = pass0 + (pair ? h * p.tpt : 0) + ti;  // this row's, in its sequence
      const bool row_ok = r < rows_box && token < n;
      const bool warp_ok = __any_sync(0xffffffffu, row_ok);
      // the row's first mask words, on their way long before they are needed
      const uint32_t* mrow = p.mask + static_cast<int64_t>(U->q0 + token) * p.mask_words;
      uint2 mhead = make_uint2(0, 0);
      if (row_ok) {
        mhead.x = mrow[0];
        if (n > 32) mhead.y = mrow[1];
      }
      const int tiles = pair ? nt : (nt - h + 1) >> 1;
      float m = -CUDART_INF_F, l = 0.f;
      bool bad = false;  // this row sees a drafted token whose V is not finite
#pragma unroll 1
      for (int x = 0; x < 2 * tiles; ++x) {
        const int half = x & 1;
        const int tl = pair ? x >> 1 : 2 * (x >> 1) + h;
        const uint32_t kt = kt0 + tl;
        const int kv0 = (tile0 + tl) * 128 + 64 * half;  // the step's first key
        const uint32_t scol = srow + 64 * half;
        mbar_wait(&s_full[2 * h + half], (cnt + (x >> 1)) & 1, abort_flag, p.err);
        tc_fence_after();
        const uint32_t vm = (kmask[kt % kMaskRing] >> (4 * half)) & 15u;
        // A tail step holds drafted tokens or the context's end (the lengths alone
        // say so: all warps take its barrier, or none).  In any other step whose
        // pages were all loaded every row sees every key.
        const bool tail = kv0 + 64 > c;
        if (tail || vm != 15u) {
          const int L = U->L;
          volatile uint32_t* pw =
              poison_s + ((pair ? 4 : 2 * h) + ((pair ? pair_tails : split_tails) & 1)) * 4;
          // (in pair mode stream 0 does, behind the barrier, and both do where there
          // is none: the same zeros)
          if (!pair || h == 0 || !tail) {
            // Two threads look after a key row of V, a 64-dim half each: zero past
            // the context and in pages that were not loaded (their weights are 0,
            // and 0 times what is there could be NaN), and zero, on record, where
            // a drafted token's V is not finite (rows that do not see it have
            // weight 0).  Each row begins at a chunk of its own: at the same one,
            // eight rows' would lie in the same banks.
            const int kr = r & 63, part = r >> 6;
            const int key = kv0 + kr;
            const uint32_t vpos = 2 * kt + 1;
            const int vs = vpos % C::kSlots;
            mbar_wait(&kv_full[vs], (vpos / C::kSlots) & 1, abort_flag, p.err);
            const bool dead = key >= L || !((vm >> (kr >> 4)) & 1u);
            const uint32_t vrow = sbase + C::kOffKV + vs * C::kTileBytes +
                                  (4 * half + (kr >> 4)) * C::kPage + part * 2048 + (kr & 15) * 128;
            bool odd = false;
            if (part < C::kHalves) {
              if (!dead && key >= c) {
#pragma unroll 4
                for (int j = 0; j < 8; ++j) {
                  const uint4 y = lds128(vrow + ((j + kr) & 7) * 16);
                  odd |= nonfinite_pair(y.x) | nonfinite_pair(y.y) | nonfinite_pair(y.z) |
                         nonfinite_pair(y.w);
                }
              }
              if (dead || odd) {
#pragma unroll 4
                for (int j = 0; j < 8; ++j) sts128_zero(vrow + ((j + kr) & 7) * 16);
                fence_proxy_async_smem();
              }
            }
            const uint32_t word = __ballot_sync(0xffffffffu, odd);
            if (tail && lane == 0) pw[q4] = word;  // [64-dim half][key / 32]
          }
          if (tail) {
            named_bar_sync(pair ? kBarBoth : kBarStream + h, pair ? 256 : 128);
            if (pair)
              ++pair_tails;
            else
              ++split_tails;
          }
          // Scores of keys that are not seen become -inf in place: from here on
          // every step is alike.
          if (warp_ok) {
#pragma unroll 1
            for (int j = 0; j < 2; ++j) {
              const uint32_t two = vm >> (2 * j);
              const uint32_t pages =
                  ((two & 1u) ? 0x0000ffffu : 0u) | ((two & 2u) ? 0xffff0000u : 0u);
              const uint32_t vis = row_ok ? visible32(mrow, mhead, kv0 + 32 * j - c, n) & pages : 0u;
              if (tail) bad |= (vis & (pw[j] | pw[2 + j])) != 0;
              if (__any_sync(0xffffffffu, row_ok && vis != 0xffffffffu)) {
                float y[32];
                tmem_ld32(scol + 32 * j, y);
                uint32_t w[32];
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  w[i] = __float_as_uint(((vis >> i) & 1u) ? y[i] : -CUDART_INF_F);
                tmem_st32_nowait(scol + 32 * j, w);
              }
            }
            tmem_wait_st();
          }
        }
        if (warp_ok) {
          // The row's scores and their maximum (scaled).
          float s[64];
          tmem_ld64(scol, s);
          float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
          for (int i = 4; i < 60; i += 8)
#pragma unroll
            for (int j = 0; j < 4; ++j) mx[j] = fmaxf(fmaxf(mx[j], s[i + j]), s[i + 4 + j]);
#pragma unroll
          for (int j = 0; j < 4; ++j) mx[j] = fmaxf(mx[j], s[60 + j]);
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc;
          // The maximum in use is raised (and the row of O_h and l rescaled) only
          // when the step's exceeds it by 2^16: weights up to that cannot overflow
          // fp32 sums, and the division by l makes the result exact either way.
          const bool raise = m == -CUDART_INF_F ? top != -CUDART_INF_F : top > m + kRaiseLog2;
          if (__any_sync(0xffffffffu, raise)) {
            const float f = !raise ? 1.f : m == -CUDART_INF_F ? 0.f : exp2f(m - top);
            if (raise) m = top;
            l *= f;
            if (x > 0) {  // once the P.V of the step before is done
              mbar_wait(&pv_done[2 * h + (half ^ 1)], (cnt + ((x - 1) >> 1)) & 1, abort_flag, p.err);
              tc_fence_after();
#pragma unroll 1
              for (int cc = 0; cc < D / 8; ++cc) {
                float ov[8];
                tmem_ld8(ocol + cc * 8, ov);
                uint32_t ow[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) ow[i] = __float_as_uint(ov[i] * f);
                tmem_st8(ocol + cc * 8, ow);
              }
            }
          }
          // Weights, in place of the scores: per 16 keys 8 columns of P_hi and 8 of
          // P_lo.  Both parts are rounded to nearest (cut off instead, which takes as
          // long, they made every output smaller by some 2^-17 of itself: l sums the
          // whole weights).
          const float nm = m == -CUDART_INF_F ? 0.f : -m;
          const float2 nm2 = make_float2(nm, nm);
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              const float2 y =
                  __ffma2_rn(make_float2(s[16 * j + i], s[16 * j + i + 1]), sc2, nm2);
              const float2 e = make_float2(exp2f(y.x), exp2f(y.y));
              sum[(i >> 1) & 1] = __fadd2_rn(sum[(i >> 1) & 1], e);
              const uint32_t h2 = pack_bf16x2(e.x, e.y);
              w[i >> 1] = h2;
              const float2 hi = make_float2(bf16lo(h2), bf16hi(h2));
              const float2 lo = __ffma2_rn(hi, neg1, e);  // e - P_hi, exact
              w[8 + (i >> 1)] = pack_bf16x2(lo.x, lo.y);
            }
            tmem_st16_nowait(scol + 16 * j, w);
          }
          l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[2 * h + half]);
      }
      cnt += tiles;

      // End of the unit: this row's output and log-sum-exp of the unit's keys.  In
      // split mode the two streams' maxima and sums (a sum's sign is set where the
      // row is bad) meet first.
      // (the last step's P.V: it and all before it are done)
      if (tiles > 0) mbar_wait(&pv_done[2 * h + 1], (cnt - 1) & 1, abort_flag, p.err);
      float m0 = m, l0 = l, m1 = -CUDART_INF_F, l1 = 0.f;
      if (!pair) {
        tc_fence_before();
        xbuf[256 * h + r] = m;  // [stream][m, l][row]
        xbuf[256 * h + 128 + r] = bad ? -l : l;
        named_bar_sync(kBarBoth, 256);
        m0 = xbuf[r];
        l0 = xbuf[128 + r];
        m1 = xbuf[256 + r];
        l1 = xbuf[384 + r];
        bad = signbit(l0) | signbit(l1);
        l0 = fabsf(l0);
        l1 = fabsf(l1);
        named_bar_sync(kBarBoth, 256);  // read by all before either stream writes again
      }
      tc_fence_after();
      const float M = fmaxf(m0, m1);
      const float e0 = m0 == -CUDART_INF_F ? 0.f : exp2f(m0 - M);
      const float e1 = m1 == -CUDART_INF_F ? 0.f : exp2f(m1 - M);
      const float L = l0 * e0 + l1 * e1;
      // l > 0, or NaN where a score was
      const bool live = !(L == 0.f);
      const float inv = bad ? CUDART_NAN_F : live ? 1.f / L : 0.f;
      const float f0 = e0 * inv, f1 = e1 * inv;
      const bool full = nt == U->tiles;
      const int64_t orow = static_cast<int64_t>(U->q0 + token) * p.hq + U->g * p.group +
                           (r - ti * p.group);
      const int64_t prow = static_cast<int64_t>(2 * blockIdx.x + (tile0 == 0 ? 1 : 0)) *
                               p.part_rows + (pair ? h * 128 : 0) + r;
      __syncwarp();
      if (lane == 0) mbar_arrive(&u_empty[slot]);
      // pair mode: all dims of the stream's row; split mode: this stream's half of
      // the dims, from both accumulators
      const int d0 = pair ? 0 : h * (D / 2);
      const int dims = pair ? D : D / 2;
      const uint32_t src = pair ? ocol : tmem + lane_addr + kOCol + d0;
      const bool two = !pair && nt > 1;  // stream 1 had a tile
      // (nothing seen: the accumulator of all-zero weights is zero, and stays so)
      if (warp_ok && full) {
#pragma unroll 1
        for (int cc = 0; cc < dims; cc += 16) {
          float a[16];
          tmem_ld16(src + cc, a);
#pragma unroll
          for (int i = 0; i < 16; ++i) a[i] *= f0;
          if (two) {
            float b[16];
            tmem_ld16(src + 128 + cc, b);
#pragma unroll
            for (int i = 0; i < 16; ++i) a[i] = fmaf(b[i], f1, a[i]);
          }
          if (row_ok) {
            uint4* dst = reinterpret_cast<uint4*>(p.out + orow * D + d0 + cc);
#pragma unroll
            for (int i = 0; i < 2; ++i)
              dst[i] = make_uint4(pack_bf16x2(a[8 * i], a[8 * i + 1]),
                                  pack_bf16x2(a[8 * i + 2], a[8 * i + 3]),
                                  pack_bf16x2(a[8 * i + 4], a[8 * i + 5]),
                                  pack_bf16x2(a[8 * i + 6], a[8 * i + 7]));
          }
        }
      } else if (warp_ok) {
        // Partial rows, four lanes' transposed before they are stored: a lane then
        // holds the same 16-byte chunk of four rows, and the lanes' chunks of a row
        // lie next to each other (a store of 32 rows' chunks takes 32 turns of the
        // load-store unit, 4000 cycles of a small call in all).
        const int q = lane & 3;
        const uint32_t oks = __ballot_sync(0xffffffffu, row_ok) >> (lane & ~3);
#pragma unroll 1
        for (int cc = 0; cc < dims; cc += 16) {
          float a[16];
          tmem_ld16(src + cc, a);
          float b[16] = {};
          if (two) tmem_ld16(src + 128 + cc, b);
          uint4 v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = fmaf(b[4 * i + j], two ? f1 : 0.f, a[4 * i + j] * f0);
            v[i] = make_uint4(__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]),
                              __float_as_uint(y[3]));
          }
          transpose4(v, lane);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if ((oks >> i) & 1u)
              *reinterpret_cast<uint4*>(p.part_o + (prow - q + i) * D + d0 + cc + 4 * q) = v[i];
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_free);
      if (row_ok && (pair || h == 0)) {
        const float lse2 = live ? M + log2f(L) : -CUDART_INF_F;
        if (!full)
          p.part_lse[prow] = lse2;
        else if (p.lse)
          p.lse[orow] = live ? lse2 * kLn2 : -CUDART_INF_F;
      }
      kt0 += nt;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ---------------------------------------------------------------------------
// Merge: block (c, y) takes rows of the item that begins in CTA c and ends in a
// later one; a warp per row.  part i of the item is CTA c's "begun there" part
// for i = 0 and CTA c + i's other part after that.
// ---------------------------------------------------------------------------
constexpr int kMergeWarps = 4;

template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps) tree_merge_kernel(
    const __grid_constant__ TreeParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int4 b = p.border[blockIdx.x];
  if (b.x < 0) return;
  const int lane = threadIdx.x & 31;
  const int q0 = p.cu_q[b.x], n = p.cu_q[b.x + 1] - q0;
  const int parts = b.w - static_cast<int>(blockIdx.x) + 1;
  constexpr int kPer = D / 32;  // dims of a lane
  for (int row = blockIdx.y * kMergeWarps + (threadIdx.x >> 5); row < p.part_rows;
       row += gridDim.y * kMergeWarps) {
    const int h = row >> 7, r = row & 127;
    const int ti = r / p.group, head = r - ti * p.group;
    const int token = b.z * 2 * p.tpt + h * p.tpt + ti;
    if (ti >= p.tpt || token >= n) continue;
    auto at = [&](int i) {
      const int64_t cta = blockIdx.x + i;
      return (2 * cta + (i == 0 ? 1 : 0)) * p.part_rows + row;
    };
    float top = -CUDART_INF_F;
    for (int i = lane; i < parts; i += 32) top = fmaxf(top, p.part_lse[at(i)]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float ref = top == -CUDART_INF_F ? 0.f : top;
    float z = 0.f;
    float acc[kPer];
#pragma unroll
    for (int d = 0; d < kPer; ++d) acc[d] = 0.f;
#pragma unroll 4
    for (int i = 0; i < parts; ++i) {
      const int64_t a = at(i);
      const float w = exp2f(p.part_lse[a] - ref);  // 0 for an empty part
      z += w;
      const float* o = p.part_o + a * D + lane * kPer;
#pragma unroll
      for (int d = 0; d < kPer; ++d) acc[d] = fmaf(w, o[d], acc[d]);
    }
    const bool live = !(z == 0.f);
    const float inv = live ? 1.f / z : 0.f;
    const int64_t orow = static_cast<int64_t>(q0 + token) * p.hq + b.y * p.group + head;
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + orow * D) + lane * (kPer / 2);
#pragma unroll
    for (int d = 0; d < kPer; d += 2) dst[d / 2] = pack_bf16x2(acc[d] * inv, acc[d + 1] * inv);
    if (p.lse && lane == 0) p.lse[orow] = live ? (ref + log2f(z)) * kLn2 : -CUDART_INF_F;
  }
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

int rows_of(int max_q_len, int group) { return max_q_len > 128 / group ? 256 : 128; }

template <int D>
int launch_tree(TreeParams& p, const void* q, int64_t q_stride, const void* k_pool,
                const void* v_pool, const pa_pool_desc& pool, int64_t most_tiles,
                cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(pool.num_blocks) * pool.num_kv_heads * 16;
  {
    const uint64_t dims[2] = {static_cast<uint64_t>(D), static_cast<uint64_t>(rows)};
    const uint64_t strides[1] = {D * 2};
    const uint32_t box[2] = {64, 16};
    if (!KPage<D>::encode(&p.tm_k, k_pool, rows)) return PA_ERR_CUDA;
    if (D == 64 && !encode_bf16_map(&p.tm_v, v_pool, 2, dims, strides, box)) return PA_ERR_CUDA;
  }
  if (D == 128) {
    // V: (dim within a 64-dim half, pool row, half): one copy moves both halves
    const uint64_t dims[3] = {64, static_cast<uint64_t>(rows), 2};
    const uint64_t strides[2] = {D * 2, 128};
    const uint32_t box[3] = {64, 16, 2};
    if (!encode_bf16_map(&p.tm_v, v_pool, 3, dims, strides, box)) return PA_ERR_CUDA;
  }
  {
    const uint64_t dims[3] = {static_cast<uint64_t>(D), static_cast<uint64_t>(p.hq),
                              static_cast<uint64_t>(p.total_q)};
    const uint64_t strides[2] = {D * 2, static_cast<uint64_t>(q_stride) * 2};
    const uint32_t box[3] = {64, static_cast<uint32_t>(p.group), static_cast<uint32_t>(p.tpt)};
    if (!encode_bf16_map(&p.tm_q, q, 3, dims, strides, box)) return PA_ERR_CUDA;
  }
  static KernelLaunchCache cache;
  if (cache.blocks_per_sm(reinterpret_cast<const void*>(tree_tc_kernel<D>), kThreads,
                          Cfg<D>::kSmem) < 1)
    return PA_ERR_CUDA;
  const int sms = num_sms() < kMaxCtas ? num_sms() : kMaxCtas;
  const int grid = static_cast<int>(most_tiles < sms ? most_tiles : sms);
  const int st =
      launch_overlapped(tree_tc_kernel<D>, dim3(grid), kThreads, Cfg<D>::kSmem, p, stream);
  if (st != PA_OK) return st;
  return launch_overlapped(tree_merge_kernel<D>, dim3(grid, p.part_rows / (2 * kMergeWarps)),
                           32 * kMergeWarps, 0, p, stream);
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" {

size_t pa_tree_workspace_size(int32_t max_q_len, int32_t num_q_heads, pa_pool_desc pool) {
  if (max_q_len <= 0 || num_q_heads <= 0 || pool.num_kv_heads <= 0 || pool.head_dim <= 0 ||
      num_q_heads < pool.num_kv_heads || num_q_heads / pool.num_kv_heads > 16)
    return 0;
  const size_t rows = size_t(2) * kMaxCtas * rows_of(max_q_len, num_q_heads / pool.num_kv_heads);
  return align256(sizeof(int4) * kMaxCtas) + align256(sizeof(float) * rows) +
         sizeof(float) * rows * pool.head_dim;
}

int pa_tree_attention(const void* q, int64_t q_stride, const int32_t* cu_q_lens, int32_t total_q,
                      int32_t max_q_len, const int64_t* tree_mask, int32_t mask_words,
                      const void* k_pool, const void* v_pool, pa_pool_desc pool,
                      const int32_t* block_tables, int32_t max_blocks_per_seq,
                      const int32_t* context_lens, int32_t num_seqs, int32_t num_q_heads,
                      float scale, void* out, float* lse, void* workspace, size_t workspace_bytes,
                      void* stream) {
  PA_NVTX_RANGE("pa_tree_attention");
  const int st = check_pool(pool);
  if (st != PA_OK) return st;
  if (num_seqs < 0 || total_q < 0 || num_q_heads <= 0 || max_blocks_per_seq <= 0)
    return PA_ERR_ARG;
  if (num_q_heads % pool.num_kv_heads) return PA_ERR_SHAPE;
  const int group = num_q_heads / pool.num_kv_heads;
  if (group > 16) return PA_ERR_UNSUPPORTED;
  if (num_seqs == 0 || total_q == 0) return PA_OK;
  if (max_q_len < 1 || mask_words < 1 || static_cast<int64_t>(mask_words) * 64 < max_q_len)
    return PA_ERR_ARG;
  // the context limit keeps a sequence's positions, and a pool's rows, in an int
  const int64_t rows = static_cast<int64_t>(pool.num_blocks) * pool.num_kv_heads * 16;
  if (max_q_len > PA_TREE_MAX_TOKENS || mask_words > (1 << 20) || total_q >= (1 << 30) ||
      rows >= (1LL << 31) || max_blocks_per_seq > (1 << 26))
    return PA_ERR_UNSUPPORTED;
  if (!q || !cu_q_lens || !tree_mask || !k_pool || !v_pool || !block_tables || !context_lens ||
      !out)
    return PA_ERR_ARG;
  if (!aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(out))
    return PA_ERR_ARG;
  if (q_stride < static_cast<int64_t>(num_q_heads) * pool.head_dim || q_stride % 8)
    return PA_ERR_ARG;
  if (!workspace || !aligned16(workspace) ||
      workspace_bytes < pa_tree_workspace_size(max_q_len, num_q_heads, pool))
    return PA_ERR_WORKSPACE;
  TreeParams p = {};
  p.err = device_error_word();
  if (!p.err) return PA_ERR_CUDA;
  p.cu_q = cu_q_lens;
  p.mask = reinterpret_cast<const uint32_t*>(tree_mask);
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.total_q = total_q;
  p.max_n = max_q_len;
  p.mask_words = 2 * mask_words;
  p.max_blocks = max_blocks_per_seq;
  p.num_blocks = pool.num_blocks;
  p.hkv = pool.num_kv_heads;
  p.hq = num_q_heads;
  p.group = group;
  p.tpt = 128 / group;
  p.by_pass = Divisor(2 * p.tpt);
  p.num_seqs = num_seqs;
  p.part_rows = rows_of(max_q_len, group);
  p.scale_log2 = scale * kLog2e;
  char* ws = static_cast<char*>(workspace);
  p.border = reinterpret_cast<int4*>(ws);
  ws += align256(sizeof(int4) * kMaxCtas);
  p.part_lse = reinterpret_cast<float*>(ws);
  ws += align256(sizeof(float) * 2 * kMaxCtas * p.part_rows);
  p.part_o = reinterpret_cast<float*>(ws);
  const int64_t passes = (max_q_len + 2 * p.tpt - 1) / (2 * p.tpt);
  const int64_t tiles = (static_cast<int64_t>(max_blocks_per_seq) * 16 + 127) / 128;
  const int64_t most = tiles > kMaxCtas ? kMaxCtas : tiles * passes * num_seqs * p.hkv;
  if (pool.head_dim == 128)
    return launch_tree<128>(p, q, q_stride, k_pool, v_pool, pool, most, as_stream(stream));
  return launch_tree<64>(p, q, q_stride, k_pool, v_pool, pool, most, as_stream(stream));
}

}  // extern "C"
