// kv_attention.cuh -- attention over the paged 8-bit key/value cache.
//
//   z_j = softmax_scale * sK(block of j) * sum_d q_d kcode_j,d      for the tokens j that the row sees
//   out = sum_j w_j sV(block of j) vcode_j, w = softmax(z);  lse = log sum_j exp z_j
//
// Query i of a request with L cached tokens and Q queries stands at position p = L - Q + i and sees
// j < L, with j <= p (causal) and j > p - window (a window).  A row that sees nothing gives 0 and
// lse = -inf.
#pragma once

#include <cmath>

#include "kv_cache.cuh"
#include "kv_ring.cuh"

namespace mxgb {

struct KvAttnArgs {
  const uint16_t* q;  // [tokens][heads][D], bf16 or fp16
  int64_t stride_t, stride_h;
  const uint8_t* k_codes;
  const uint8_t* v_codes;
  const float* k_scale;
  const float* v_scale;
  const int32_t* tables;   // [requests][max_blocks]
  const int32_t* lengths;  // [requests]
  const int32_t* q_start;  // [requests + 1]
  uint16_t* out;           // [tokens][heads][D]
  float* lse;              // [tokens][heads]
  float scale_log2;        // softmax scale * log2(e)
  int64_t num_blocks;
  int tokens, heads, kv_heads, requests, max_blocks, shift;
  int causal, window;
  int f16;                 // q and out are FP16, else bf16
};

constexpr float kLn2 = 0.69314718055994531f;

// mbar_wait by a whole warp, whose lanes all get the same answer: one that went on while another gave up would wait
// for it for ever at the next operation of the whole warp.  The waiting loop is out of line: the roles' loops stay
// short, which prompts gain 1% and drafts 3% by.
__device__ __noinline__ bool kv_wait_on(uint64_t* bar, uint32_t parity, volatile int* abort_flag, unsigned int site) {
  return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, abort_flag, site));
}
__device__ __forceinline__ bool kv_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, unsigned int site) {
  return __all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity)) || kv_wait_on(bar, parity, abort_flag, site);
}

// ================================================================== few rows for each kv head
// Queries of one request that share a kv head (query heads of the group x query tokens, at most 16 rows)
// meet the same keys, and the cache is read once for all of them: the call is bound by the cache's
// bytes.  What the kernel does about it:
//
//  * The work is the list of (request, kv head) units, each a row of 64-token tiles; all tiles of all
//    units, in order, are cut into gridDim.x equal ranges, one for each resident CTA, whatever the
//    lengths are.  A range is a few segments of units; a unit that one CTA has whole is finished
//    there, else each segment leaves (O, m, l) in the workspace and the CTA that finishes last joins them, in order.
//  * One warp keeps a ring of tiles in flight: TMA boxes of a block's rows of codes (128 or 64 bytes,
//    swizzled), so a tile's codes cross the SM once, and the scales of its four 16-token slices.  It walks
//    the units, tells the other warps of the next segment and brings its queries while the present one runs.
//    (16-token blocks are 8 boxes a tile.  16-byte copies by every lane instead: 39 us against 36 us for
//    33 requests of 3000 tokens at D = 64.)
//  * Four warps take one 16-token slice of the tile each, all rows, with running (m, l, O) of their own
//    and no barrier between them until the segment's end.  Codes become FP16 in registers, exactly.
//      S^T (16 tokens x 8 rows) = K Q^T and O^T (16 of D x 8 rows) += V^T P^T on m16n8k16 products:
//    the small side of both is the rows, so 8 rows cost one product's n = 8 where a 128-row tensor-memory
//    tile would be 1/16 full.  A slice's 16 products take 32 cycles of an SM (measured rate: one in two
//    cycles), its 4 KB of codes 174 cycles of the SM's share of the memory's rate; the conversions (a pair of
//    codes: 2.2 cycles of a quarter of the SM from the low half of a register, 4 from the high) take 50.
//    The order of d inside K Q^T, and of d among the rows of V^T, is free: each lane takes 16-byte words.
//  * Queries become FP16 with a power of two for each row, exact to 2^-29 of the row's largest.
//  * Softmax in base 2.  sV is folded into the exponent: p' = 2^(z + log2 sV - m), l = sum p' / sV, so
//    the weights of all blocks are rounded to FP16 (2^-11, or 2^-25 of the reference below 2^-14 of it; the
//    output's own type is no finer) relative to the same reference m.  m is renewed when a score passes it
//    by 8 (p' <= 2^8 stays well inside FP16), not at each new maximum.
//  * Tiles that some row does not see whole are masked; codes there that no row sees are cleared, and
//    NaN codes of V (0 * NaN) are taken out and put into the rows that see them at the end.
//
// Measured (D = 128, E4M3): 8 requests of up to 65536 tokens, 8 kv heads, 8 rows each: 130 us, 6.0 TB/s, 0.90
// of the measured copy rate.  64 of up to 4096, 4 rows: 62 us, 5.4 TB/s; about 10 us of that is what a call of any
// size takes (1 request, 777 tokens: 13 us), the join among it.  What bounds it: memory latency where a CTA's ring
// runs dry at a segment's first tiles.  Three CTAs of three 16 KB stages a SM: two CTAs 63 us, four of two
// stages 72 us (64 x 4096); at D = 64 four CTAs of five 8 KB stages: 36 us, two 39, five of three stages 45.
constexpr int kKvTile = 64;
constexpr int kKvWarps = 4;
constexpr int kKvFewThreads = 32 * (kKvWarps + 1);
constexpr int kKvMaxCtas = 608;

struct KvJob {  // a range of the list, and the unit that it begins in
  long long begin, end, unit;
  int tiles, head, q0, row0, rows, request, q_tile;  // rows row0 .. row0 + rows - 1 of the request's head group
};

// Workspace: counters of the cut units (zero between calls), the jobs (many rows), then parts.
constexpr size_t kKvJobsAt = 4096;
static_assert(4 * kKvMaxCtas <= kKvJobsAt, "a counter for each range");
constexpr size_t kKvSlotsAt = kKvJobsAt + sizeof(KvJob) * kKvMaxCtas;

// A segment as the loading warp tells the others of it, with its queries; count = 0: no more.
struct alignas(16) KvFewSegment {
  int count, token;            // tiles, and the first one's first token
  int rows, q0, len, head;
  int any_lo, all_lo, all_hi;  // tokens from any_lo on are seen by some row, [all_lo, all_hi) by all
  int part;                    // 0: the whole unit; 1 + slot: a part of it
  int parts, first, first_slot;  // a cut unit: how many ranges have tiles of it, the first of them and its slot
  long long place;             // and where its tiles begin in the list
};

template <int D, int NT>
struct KvFewCfg {
  static constexpr int ROWS = 8 * NT;
  static constexpr int STAGES = D == 128 ? 3 : 5;
  static constexpr int HALF = kKvTile * D;          // codes of K, or of V, in a tile
  static constexpr int O_STRIDE = D + 4;
  static constexpr int OFF_O = STAGES * 2 * HALF;   // float [warps][ROWS][O_STRIDE]
  static constexpr int OFF_ML = OFF_O + 4 * kKvWarps * ROWS * O_STRIDE;  // float2 [warps][ROWS]
  // two segments' queries
  static constexpr int OFF_Q = OFF_ML + 8 * kKvWarps * ROWS;        // uint2 [2][D / 16][NT][32]
  static constexpr int OFF_QF = OFF_Q + 2 * (D / 16) * NT * 32 * 8;     // float [2][ROWS]
  static constexpr int OFF_SEEN = OFF_QF + 2 * 4 * ROWS;                // int2 [2][ROWS]
  static constexpr int OFF_NAN = OFF_SEEN + 2 * 8 * ROWS;               // u32 [2][ROWS][D / 32], bits of d
  static constexpr int OFF_SEG = OFF_NAN + 2 * 4 * ROWS * (D / 32);     // KvFewSegment [2]
  static constexpr int OFF_SC = OFF_SEG + 2 * sizeof(KvFewSegment);     // float4 [STAGES][4]: sK, log2 sV, 1 / sV, how codes are taken
  static constexpr int OFF_BAR = OFF_SC + 16 * 4 * STAGES;
  static constexpr int SMEM = OFF_BAR + 8 * (2 * STAGES + 5) + 16 + 1024;
  static constexpr int CTAS = NT == 1 ? (D == 64 ? 4 : 3) : 2;
  static constexpr size_t SLOT = static_cast<size_t>(ROWS) * (D + 2) * 4;  // (O, m, l) of a segment
};

__device__ __forceinline__ void kv_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t kv_transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ float kv_exp2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t kv_pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// 0x80 in each byte that is a NaN code (E5M2: or an infinity)
template <int FMT>
__device__ __forceinline__ uint32_t kv_nan_bytes(uint32_t w) {
  return ((w & 0x7F7F7F7Fu) + (FMT == 0 ? 0x01010101u : 0x04040404u)) & 0x80808080u;
}

// Scales are 0 or in [2^-48, 2^48]: within it 2^(z + log2 sV - m) and its quotient by sV stay numbers of FP32 that
// count (two blocks' are at most 2^96 apart).  The codes of a block of scale 0 are taken as zeros; those of one of any
// other scale as NaN, which reaches the rows that see it as a NaN in the cache does.
// What a V scale of 0 counts as, beside codes that are zeros: below other blocks' scales, which then keep the bits of
// their weights, but no further from 1 than lse bears (log2 sV is in its reference: 2^-48 cost it a bit).
constexpr float kKvZeroAs = 1.f / (1 << 24);
constexpr int kKvTakeZero = 1, kKvTakeNan = 0x80;  // 1 + the byte that each code is taken as; 0: as it is

// What a scale says of its block's codes; the scale itself becomes one in range.
__device__ __forceinline__ int kv_check_scale(float& s, float for_zero) {
  if (s >= kKvLeastScale && s <= kKvMostScale) return 0;
  const bool zero = s == 0.f;
  s = zero ? for_zero : 1.f;
  return zero ? kKvTakeZero : kKvTakeNan;
}
// Both scales of a block; of K, and of V << 8.  tell: some row sees the block.
__device__ __forceinline__ int kv_check_scales(float& sk, float& sv, bool tell) {
  const int take = kv_check_scale(sk, 1.f) | kv_check_scale(sv, kKvZeroAs) << 8;
  if (tell && take & (kKvTakeNan | kKvTakeNan << 8)) atomicOr(&g_mx_error_word, kSiteBadCache);
  return take;
}
__device__ __forceinline__ uint32_t kv_four_taken(int take) { return static_cast<uint32_t>(take - 1) * 0x01010101u; }
// A warp's slice of 16 tokens whose codes are not taken as they are: K, and V `half` behind it.  (Rare.)
template <int D>
__device__ __noinline__ void kv_take_slice(uint8_t* at, int half, int take) {
  for (int i = 16 * (threadIdx.x & 31); i < 16 * D; i += 512) {
    const uint32_t k = kv_four_taken(take & 0xFF), v = kv_four_taken(take >> 8);
    if (take & 0xFF) *reinterpret_cast<uint4*>(at + i) = make_uint4(k, k, k, k);
    if (take >> 8) *reinterpret_cast<uint4*>(at + half + i) = make_uint4(v, v, v, v);
  }
  fence_proxy_async_smem();  // (copies come to the same place next)
  __syncwarp();
}
// Block and scales of a table entry.  A number out of range has no block, and scales that are none.
__device__ __forceinline__ void kv_look_up(const KvAttnArgs& a, int request, int page, int head, int& block, float& sk,
                                           float& sv) {
  block = a.tables[static_cast<int64_t>(request) * a.max_blocks + page];
  if (block < 0 || block >= a.num_blocks) {
    block = -1;
    sk = sv = NAN;
  } else {
    const int64_t at = static_cast<int64_t>(block) * a.kv_heads + head;
    sk = a.k_scale[at];
    sv = a.v_scale[at];
  }
}

// A request as the kernels go through it.
struct KvRequest {
  int q0, rows_q, len, first_tile, tiles;  // tiles = 0: no queries
  __device__ int cost() const;
};

__device__ __forceinline__ KvRequest kv_request(const KvAttnArgs& a, int r, int most_q, bool tell) {
  KvRequest v;
  v.q0 = a.q_start[r];
  const int end = a.q_start[r + 1];
  v.len = a.lengths[r];
  // (compared before they are subtracted: differences of any two 32-bit numbers do not fit)
  const bool ok = v.q0 >= 0 && v.q0 <= end && end <= a.tokens && end - v.q0 <= most_q && v.len >= 0 &&
                  v.len <= a.max_blocks << a.shift;
  if (!ok && tell) atomicOr(&g_mx_error_word, kSiteBadCache);
  v.rows_q = ok ? end - v.q0 : 0;
  v.len = ok ? v.len : 0;
  const int lo = a.window ? max(0, v.len - v.rows_q - a.window + 1) : 0;
  v.first_tile = lo / kKvTile;
  v.tiles = v.rows_q ? max(1, (v.len + kKvTile - 1) / kKvTile - v.first_tile) : 0;
  return v;
}

// The list of all units' work, in 64-token tiles, is cut into equal ranges.  A unit costs its tiles and
// kKvUnitCost more, for its queries' fetch and the join of the warps, so that many short units are not
// one CTA's (64 x 4096 tokens and 3 empty places: 110 us with no such cost, 67 with 1, 61 with 3 and 5; prompts
// of 6 x 1500: 246 us with 1, 227 with 3 and 5); a range that begins inside those first places begins at the unit's first tile.
constexpr int kKvUnitCost = 3;

__device__ __forceinline__ int KvRequest::cost() const { return tiles ? tiles + kKvUnitCost : 0; }

// the range, of n, that place p of a list of `total` places is in
__device__ __forceinline__ int kv_range_of(long long total, long long p, int n) {
  if (total < (1 << 21)) return static_cast<int>((static_cast<unsigned>(p + 1) * static_cast<unsigned>(n) - 1) / static_cast<unsigned>(total));
  return static_cast<int>(((p + 1) * n - 1) / total);
}
// place i n-ths into a list of `total` places
__device__ __forceinline__ long long kv_cut(long long total, int i, int n) {
  if (total < (1 << 21)) return static_cast<unsigned>(total) * static_cast<unsigned>(i) / static_cast<unsigned>(n);
  return total * i / n;
}

// The walk over a range's segments.
struct KvWalk {
  long long pos, end, base;  // base: where the current unit begins in the list
  int r, h;
  KvRequest req;
  int tile, count;  // the current segment: tiles of the unit, from the unit's first one on
};

// Finds where this CTA's range begins and ends: every thread sums a stretch of the requests, the sums are
// scanned, and the thread that holds the range's first place finds its unit.
struct KvPlanSmem {
  long long warp_sum[kKvWarps + 1];
  long long pos, end, base, total;
  int r, h;
};
__device__ __forceinline__ void kv_plan(const KvAttnArgs& a, int most_q, KvPlanSmem& sm, KvWalk& w) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.requests + kKvFewThreads - 1) / kKvFewThreads;
  const int r0 = min(tid * per, a.requests), r1 = min(r0 + per, a.requests);
  long long mine = 0;
  for (int r = r0; r < r1; ++r) mine += kv_request(a, r, most_q, blockIdx.x == 0).cost();
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) sm.warp_sum[warp] = incl;
  __syncthreads();
  long long before = incl - mine, total = 0;
#pragma unroll
  for (int i = 0; i <= kKvWarps; ++i) {
    if (i < warp) before += sm.warp_sum[i];
    total += sm.warp_sum[i];
  }
  total *= a.kv_heads;
  before *= a.kv_heads;
  mine *= a.kv_heads;
  const long long pos = kv_cut(total, blockIdx.x, gridDim.x);
  if (pos >= before && pos < before + mine) {
    long long at = before;
    for (int r = r0; r < r1; ++r) {
      const int cost = kv_request(a, r, most_q, false).cost();
      const long long all = static_cast<long long>(cost) * a.kv_heads;
      if (pos < at + all) {
        sm.r = r;
        sm.h = static_cast<int>(pos - at < (1ll << 31) ? static_cast<unsigned>(pos - at) / static_cast<unsigned>(cost)
                                                       : (pos - at) / cost);
        sm.base = at + static_cast<long long>(sm.h) * cost;
        break;
      }
      at += all;
    }
  }
  if (tid == 0) {
    sm.pos = pos;
    sm.end = kv_cut(total, blockIdx.x + 1, gridDim.x);
    sm.total = total;
  }
  __syncthreads();
  w.pos = sm.pos;
  w.end = sm.end;
  w.base = sm.base;
  w.r = sm.r;
  w.h = sm.h;
  if (w.pos < sm.total) w.req = kv_request(a, w.r, most_q, false);
}
// tiles of a unit in front of place x of its cost
__device__ __forceinline__ int kv_tiles_before(long long x, int tiles) {
  return static_cast<int>(min(max(x - kKvUnitCost, 0ll), static_cast<long long>(tiles)));
}
// The next segment that has tiles, from w.pos on; false at the range's end.
__device__ __forceinline__ bool kv_next_segment(const KvAttnArgs& a, int most_q, KvWalk& w) {
  while (w.pos < w.end) {
    const long long unit_end = w.base + w.req.cost();
    if (w.pos == unit_end) {
      w.base = unit_end;
      if (++w.h == a.kv_heads) {
        w.h = 0;
        while (++w.r < a.requests) {
          w.req = kv_request(a, w.r, most_q, false);
          if (w.req.tiles) break;
        }
        if (w.r >= a.requests) return false;
      }
      continue;
    }
    const long long to = min(w.end, unit_end);
    w.tile = kv_tiles_before(w.pos - w.base, w.req.tiles);
    w.count = kv_tiles_before(to - w.base, w.req.tiles) - w.tile;
    w.pos = to;
    if (w.count) return true;
  }
  return false;
}

// Rows that no request has: 0 and -inf.
__device__ __forceinline__ void kv_clear_rest(const KvAttnArgs& a, int head_dim, int first, int step) {
  const int end = a.q_start[a.requests], used = end >= 0 && end <= a.tokens ? end : a.tokens;
  const int64_t rows = static_cast<int64_t>(a.tokens - used) * a.heads, words = rows * head_dim / 8;
  uint4* out = reinterpret_cast<uint4*>(a.out + static_cast<int64_t>(used) * a.heads * head_dim);
  for (int64_t i = first; i < words; i += step) out[i] = make_uint4(0, 0, 0, 0);
  for (int64_t i = first; i < rows; i += step) a.lse[static_cast<int64_t>(used) * a.heads + i] = -INFINITY;
}

__device__ __forceinline__ float2 kv_unpack2(uint32_t w, int f16) {
  return f16 ? kv_unpack2<true>(w) : kv_unpack2<false>(w);
}
__device__ __forceinline__ uint32_t kv_pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t kv_pack_out(float lo, float hi, int f16) {
  return f16 ? kv_pack_f16(lo, hi) : kv_pack_bf16(lo, hi);
}

// (m, l, O) and a further part's, joined
__device__ __forceinline__ void kv_join(float& m, float& l, float4& o, float2 ml, float4 x) {
  const float most = fmaxf(m, ml.x), ref = most == -INFINITY ? 0.f : most;
  const float f0 = kv_exp2(m - ref), f1 = kv_exp2(ml.x - ref);
  l = l * f0 + ml.y * f1;
  o.x = o.x * f0 + x.x * f1;
  o.y = o.y * f0 + x.y * f1;
  o.z = o.z * f0 + x.z * f1;
  o.w = o.w * f0 + x.w * f1;
  m = most;
}
// Four elements of a row's output from d on, and the row's lse.  row: of the head group, from token q0 on.
template <int D>
__device__ __forceinline__ void kv_finish(const KvAttnArgs& a, int q0, int row, int group, int head, int d, float m, float l,
                                          float4 o) {
  const int qi = row / group, hg = row - qi * group;
  const int64_t at_row = static_cast<int64_t>(q0 + qi) * a.heads + head * group + hg;
  const float inv = 1.f / l;
  *reinterpret_cast<uint2*>(a.out + at_row * D + d) =
      l == 0.f ? make_uint2(0, 0) : make_uint2(kv_pack_out(o.x * inv, o.y * inv, a.f16), kv_pack_out(o.z * inv, o.w * inv, a.f16));
  if (d == 0) a.lse[at_row] = l == 0.f ? -INFINITY : ((m == -INFINITY ? 0.f : m) + log2f(l)) * kLn2;
}

template <int FMT, int D, int NT>
__global__ void __launch_bounds__(kKvFewThreads, KvFewCfg<D, NT>::CTAS)
    kv_attention_few_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                            const KvAttnArgs a, int most_q, uint8_t* workspace) {
  using Cfg = KvFewCfg<D, NT>;
  constexpr int KS = D / 16;      // k-steps of K Q^T
  constexpr int VW = D / 32;      // 32-bit words of V that a lane takes from each token
  constexpr int LD = D / 4;       // elements of d that a lane takes from each key
  extern __shared__ uint8_t kv_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(kv_smem_raw) + 1023) & ~uintptr_t(1023));
  float* sO = reinterpret_cast<float*>(smem + Cfg::OFF_O);
  float2* sML = reinterpret_cast<float2*>(smem + Cfg::OFF_ML);
  uint2* sQ = reinterpret_cast<uint2*>(smem + Cfg::OFF_Q);
  float* sQF = reinterpret_cast<float*>(smem + Cfg::OFF_QF);
  int2* sSeen = reinterpret_cast<int2*>(smem + Cfg::OFF_SEEN);
  uint32_t* sNan = reinterpret_cast<uint32_t*>(smem + Cfg::OFF_NAN);
  KvFewSegment* sSeg = reinterpret_cast<KvFewSegment*>(smem + Cfg::OFF_SEG);
  float4* sSC = reinterpret_cast<float4*>(smem + Cfg::OFF_SC);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Cfg::OFF_BAR);
  uint64_t* empty = full + Cfg::STAGES;
  uint64_t* seg_full = empty + Cfg::STAGES;  // [2]
  uint64_t* seg_empty = seg_full + 2;        // [2]
  uint64_t* join_bar = seg_empty + 2;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(join_bar + 1);
  volatile int* last_part = abort_flag + 1;
  __shared__ KvPlanSmem plan;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int group = a.heads / a.kv_heads;

  if (tid == 0) {
    for (int i = 0; i < Cfg::STAGES; ++i) {
      mbar_init(&full[i], 2);  // the boxes' bytes; the scales
      mbar_init(&empty[i], kKvWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&seg_full[i], 1);
      mbar_init(&seg_empty[i], kKvWarps);
    }
    mbar_init(join_bar, kKvWarps);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  pdl_wait();  // (no early trigger: CTAs of the next kernel would take the places of this one's last CTAs)
  KvWalk w;
  kv_plan(a, most_q, plan, w);  // (its barriers also publish the mbarriers)
  kv_clear_rest(a, D, blockIdx.x * kKvFewThreads + tid, gridDim.x * kKvFewThreads);

  if (warp == kKvWarps) {
    // ------------------------------------------------------------------ loads
    // A chunk is up to 32 blocks of a segment: lane i holds block i and its scales, read while the chunk
    // before it is loaded.
    struct Chunk {
      int token, tiles, h, block, take;
      float sk, sv;
    };
    const int P = 1 << a.shift, rows_box = min(P, kKvTile), boxes = kKvTile / rows_box;
    const int most_tiles = P > kKvTile ? 32 * P / kKvTile - 1 : 32 * P / kKvTile;  // (a segment may start inside a block)
    const long long range_start = w.pos;
    int left = 0;
    uint32_t seg = 0;
    // tells the others of the next segment and brings its queries, as the fragments of Q^T
    auto next_segment = [&]() {
      const bool more = kv_next_segment(a, most_q, w);
      const int buf = seg & 1;
      if (!kv_wait(&seg_empty[buf], ((seg >> 1) & 1) ^ 1, abort_flag, kSiteProducerEmpty)) return false;
      ++seg;
      const int rows = w.req.rows_q * group, pos0 = w.req.len - w.req.rows_q;  // (pos0: the first query's position)
      if (lane == 0) {
        KvFewSegment v;
        v.count = more ? w.count : 0;
        v.token = (w.req.first_tile + w.tile) * kKvTile;
        v.rows = rows;
        v.q0 = w.req.q0;
        v.len = w.req.len;
        v.head = w.h;
        v.any_lo = a.window ? pos0 - a.window + 1 : 0;
        v.all_lo = a.window ? w.req.len - a.window : 0;
        v.all_hi = a.causal ? min(w.req.len, pos0 + 1) : w.req.len;
        v.part = w.count == w.req.tiles ? 0 : w.base < range_start ? 1 : 2;
        if (v.part) {
          const long long total = plan.total;
          const int n = gridDim.x;
          v.place = w.base + kKvUnitCost;
          v.first = kv_range_of(total, v.place, n);
          // (fewer places than ranges: a range has one or none)
          v.parts = total < n ? w.req.tiles : kv_range_of(total, v.place + w.req.tiles - 1, n) - v.first + 1;
          v.first_slot = w.base < kv_cut(total, v.first, n) ? 0 : 1;
        }
        sSeg[buf] = v;
      }
      if (more) {
        for (int i = lane; i < Cfg::ROWS * (D / 32); i += 32) sNan[buf * Cfg::ROWS * (D / 32) + i] = 0;
        const int g = lane >> 2, c = lane & 3;
#pragma unroll 1
        for (int nt = 0; nt < NT; ++nt) {
          const int row = nt * 8 + g;
          uint4 x[LD / 8];
          float amax = 0.f;
          const int qi = row / group, hg = row - qi * group;
          const uint16_t* src = a.q + (w.req.q0 + qi) * a.stride_t + (w.h * group + hg) * a.stride_h + c * LD;
#pragma unroll
          for (int i = 0; i < LD / 8; ++i) x[i] = row < rows ? *reinterpret_cast<const uint4*>(src + 8 * i) : make_uint4(0, 0, 0, 0);
          float f[LD];
#pragma unroll
          for (int i = 0; i < LD / 8; ++i) {
            const uint32_t u[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 y = kv_unpack2(u[j], a.f16);
              f[8 * i + 2 * j] = y.x;
              f[8 * i + 2 * j + 1] = y.y;
              amax = fmaxf(amax, fmaxf(fabsf(y.x), fabsf(y.y)));
            }
          }
          amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
          amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
          // 2^e with amax 2^e in [2^14, 2^15)
          const int e = min(14 - (static_cast<int>(__float_as_uint(amax) >> 23) - 127), 120);
          const float mul = amax > 0.f ? __uint_as_float(static_cast<uint32_t>(e + 127) << 23) : 1.f;
#pragma unroll
          for (int i = 0; i < KS; ++i)
            sQ[((buf * KS + i) * NT + nt) * 32 + lane] = make_uint2(kv_pack_f16(f[4 * i] * mul, f[4 * i + 1] * mul),
                                                                    kv_pack_f16(f[4 * i + 2] * mul, f[4 * i + 3] * mul));
          if (c == 0) {
            sQF[buf * Cfg::ROWS + row] = a.scale_log2 / mul;
            const int p = pos0 + (row < rows ? qi : 0);
            sSeen[buf * Cfg::ROWS + row] =
                make_int2(a.window ? p - a.window + 1 : 0, a.causal ? min(w.req.len, p + 1) : w.req.len);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&seg_full[buf]);
      return more;
    };
    auto fetch = [&](Chunk& ch) {
      ch.tiles = 0;
      if (!left) {
        if (!next_segment()) return;
        left = w.count;
      }
      ch.tiles = min(left, most_tiles);
      ch.token = (w.req.first_tile + w.tile + w.count - left) * kKvTile;
      ch.h = w.h;
      left -= ch.tiles;
      const int page = (ch.token >> a.shift) + lane, any_lo = a.window ? w.req.len - w.req.rows_q - a.window + 1 : 0;
      ch.block = -1;
      ch.sk = 1.f;
      ch.sv = 1.f;
      if (page << a.shift < w.req.len && (page + 1) << a.shift > any_lo)  // (what is in front of every row's window is not read)
        kv_look_up(a, w.r, page, ch.h, ch.block, ch.sk, ch.sv);
    };
    int stage = 0;
    uint32_t phase = 0;
    uint32_t issued = 0;
    bool ok = true;
    Chunk cur, next;
    fetch(cur);
    while (cur.tiles && ok) {
      for (int i = 0; i < cur.tiles; ++i) {
        const int token = cur.token + i * kKvTile, first = (token >> a.shift) - (cur.token >> a.shift);
        if (!kv_wait(&empty[stage], phase ^ 1, abort_flag, kSiteProducerEmpty)) {
          ok = false;
          break;
        }
        const int box_block = __shfl_sync(0xFFFFFFFFu, cur.block, min(first + lane, 31));
        const bool load = lane < boxes && box_block >= 0;
        const uint32_t loads = __popc(__ballot_sync(0xFFFFFFFFu, load));
        if (lane == 0) mbar_arrive_expect_tx(&full[stage], loads * 2 * rows_box * D);
        __syncwarp();
        if (load) {
          const int row = ((box_block * a.kv_heads + cur.h) << a.shift) + (token & (P - 1));
          uint8_t* dst = smem + stage * 2 * Cfg::HALF + lane * rows_box * D;
          tma_load_2d(dst, &tmK, &full[stage], 0, row);
          tma_load_2d(dst + Cfg::HALF, &tmV, &full[stage], 0, row);
        }
        const int from = ((token + 16 * (lane & 3)) >> a.shift) - (cur.token >> a.shift);  // lanes 0..3: the slices' scales
        if (i == 0) cur.take = kv_check_scales(cur.sk, cur.sv, true);  // (here, where the first boxes are on their way)
        const float slice_k = __shfl_sync(0xFFFFFFFFu, cur.sk, from), slice_v = __shfl_sync(0xFFFFFFFFu, cur.sv, from);
        const int take = __shfl_sync(0xFFFFFFFFu, cur.take, from);
        if (lane < 4) sSC[stage * 4 + lane] = make_float4(slice_k, log2f(slice_v), 1.f / slice_v, __int_as_float(take));
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[stage]);
        ++issued;
        if (++stage == Cfg::STAGES) {
          stage = 0;
          phase ^= 1;
        }
        if (i == min(Cfg::STAGES, cur.tiles) - 1) fetch(next);
      }
      cur = next;
    }
    // every copy has landed before the CTA's shared memory goes
    for (uint32_t i = 0; i < Cfg::STAGES; ++i)
      if (issued > i) mbar_drain(&full[i], kv_ring_last_parity(issued, i, Cfg::STAGES), kWaitBudgetNs);
    return;
  }

  // -------------------------------------------------------------------- products and softmax
  const int g = lane >> 2, c = lane & 3;
  int stage = 0;
  uint32_t phase = 0, joins = 0;
  auto warps_meet = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(join_bar);
    return kv_wait(join_bar, joins++ & 1, abort_flag, kSiteEpiTmemFull);
  };
  for (uint32_t seg = 0;; ++seg) {
    const int buf = seg & 1;
    if (!kv_wait(&seg_full[buf], (seg >> 1) & 1, abort_flag, kSiteMmaFull)) break;
    const KvFewSegment v = sSeg[buf];
    if (v.count == 0) break;
    const uint2* q_frag = sQ + buf * KS * NT * 32 + lane;
    const float* q_mul = sQF + buf * Cfg::ROWS;
    const int2* q_seen = sSeen + buf * Cfg::ROWS;
    uint32_t* q_nan = sNan + buf * Cfg::ROWS * (D / 32);
    uint2 qf[NT == 1 ? KS : 1];
    if (NT == 1) {
#pragma unroll
      for (int i = 0; i < KS; ++i) qf[i] = q_frag[i * 32];
    }
    float m[2 * NT], l[2 * NT];
#pragma unroll
    for (int i = 0; i < 2 * NT; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
    }
    float acc[2 * VW][NT][4];
#pragma unroll
    for (int i = 0; i < 2 * VW; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][n][j] = 0.f;

    bool ok = true;
    for (int i = 0; i < v.count; ++i) {
      const int token = v.token + i * kKvTile;
      ok = kv_wait(&full[stage], phase, abort_flag, kSiteMmaFull);
      const uint8_t* sK = smem + stage * 2 * Cfg::HALF + warp * 16 * D;
      const uint8_t* sV = sK + Cfg::HALF;
      const float4 sc = sSC[stage * 4 + warp];
      const bool edge = token < v.all_lo || token + kKvTile > v.all_hi;
      const int t0 = token + 16 * warp;
      if (!ok) break;
      if (const int take = __float_as_int(sc.w)) kv_take_slice<D>(smem + stage * 2 * Cfg::HALF + warp * 16 * D, Cfg::HALF, take);
      {
        // S^T
        float s[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
        uint4 ka[LD / 16], kb[LD / 16];
#pragma unroll
        for (int j = 0; j < LD / 16; ++j) {
          const int at = D == 128 ? g * 128 + (((2 * c + j) ^ g) << 4) : g * 64 + ((c ^ ((g >> 1) & 3)) << 4);
          ka[j] = *reinterpret_cast<const uint4*>(sK + at);
          kb[j] = *reinterpret_cast<const uint4*>(sK + 8 * D + at);
        }
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const uint4 x = ka[k / 4], y = kb[k / 4];
          const uint32_t wa = k % 4 == 0 ? x.x : k % 4 == 1 ? x.y : k % 4 == 2 ? x.z : x.w;
          const uint32_t wb = k % 4 == 0 ? y.x : k % 4 == 1 ? y.y : k % 4 == 2 ? y.z : y.w;
          uint32_t a0, a1, a2, a3;
          kv_codes4_to_f16<FMT>(wa, a0, a2);
          kv_codes4_to_f16<FMT>(wb, a1, a3);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const uint2 b = NT == 1 ? qf[NT == 1 ? k : 0] : q_frag[(k * NT + n) * 32];
            kv_mma(s[n], a0, a1, a2, a3, b.x, b.y);
          }
        }
        // z + log2 sV, the reference, the weights
        bool past = false;
        float mx[2 * NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int j = 0; j < 4; ++j) s[n][j] = fmaf(s[n][j], q_mul[n * 8 + 2 * c + (j & 1)] * sc.x, sc.y);
          if (edge) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int t = t0 + g + 8 * (j >> 1);
              const int2 seen = q_seen[n * 8 + 2 * c + (j & 1)];
              if (t < seen.x || t >= seen.y) s[n][j] = -INFINITY;
            }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            mx[2 * n + e] = fmaxf(s[n][e], s[n][2 + e]);
            past = past || mx[2 * n + e] > m[2 * n + e] + 8.f;
          }
        }
        if (__any_sync(0xFFFFFFFFu, past)) {
#pragma unroll
          for (int j = 0; j < 2 * NT; ++j) {
            float x = mx[j];
            x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 8));
            x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 16));
            x = fmaxf(x, m[j]);
            const float keep = kv_exp2(m[j] - (x == -INFINITY ? 0.f : x));
            m[j] = x;
            l[j] *= keep;
#pragma unroll
            for (int k = 0; k < 2 * VW; ++k) {
              acc[k][j >> 1][j & 1] *= keep;
              acc[k][j >> 1][2 + (j & 1)] *= keep;
            }
          }
        }
        uint32_t pb[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float m0 = m[2 * n] == -INFINITY ? 0.f : m[2 * n], m1 = m[2 * n + 1] == -INFINITY ? 0.f : m[2 * n + 1];
          const float p0 = kv_exp2(s[n][0] - m0), p1 = kv_exp2(s[n][1] - m1), p2 = kv_exp2(s[n][2] - m0),
                      p3 = kv_exp2(s[n][3] - m1);
          l[2 * n] = fmaf(p0 + p2, sc.z, l[2 * n]);
          l[2 * n + 1] = fmaf(p1 + p3, sc.z, l[2 * n + 1]);
          pb[n][0] = kv_transpose8x8(kv_pack_f16(p0, p1));
          pb[n][1] = kv_transpose8x8(kv_pack_f16(p2, p3));
        }
        // V: tokens 2c, 2c + 1, 2c + 8, 2c + 9, this lane's D / 8 values of each
        uint32_t vw[4][VW];
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) {
          const int t = 2 * c + (tt & 1) + 8 * (tt >> 1);
          if (D == 128) {
            const uint4 x = *reinterpret_cast<const uint4*>(sV + t * 128 + ((g ^ (t & 7)) << 4));
            vw[tt][0] = x.x;
            vw[tt][1] = x.y;
            vw[tt][VW - 2] = x.z;
            vw[tt][VW - 1] = x.w;
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(sV + t * 64 + (((g >> 1) ^ ((t >> 1) & 3)) << 4) + (g & 1) * 8);
            vw[tt][0] = x.x;
            vw[tt][1] = x.y;
          }
        }
        if (edge) {
          uint32_t bad = 0;
#pragma unroll
          for (int tt = 0; tt < 4; ++tt) {
            const int t = t0 + 2 * c + (tt & 1) + 8 * (tt >> 1);
#pragma unroll
            for (int j = 0; j < VW; ++j) {
              if (t < v.any_lo || t >= v.len) vw[tt][j] = 0;
              bad |= kv_nan_bytes<FMT>(vw[tt][j]);
            }
          }
          if (bad) {  // (rare) for each NaN: note the rows that see it, clear the code
#pragma unroll
            for (int tt = 0; tt < 4; ++tt)
#pragma unroll
              for (int j = 0; j < VW; ++j) {
                const uint32_t x = kv_nan_bytes<FMT>(vw[tt][j]);
                vw[tt][j] &= ~((x >> 7) * 0xFFu);
                const int t = t0 + 2 * c + (tt & 1) + 8 * (tt >> 1), d = (D / 8) * g + 4 * j;
                if (x)
                  for (int row = 0; row < Cfg::ROWS; ++row)
                    if (t >= q_seen[row].x && t < q_seen[row].y)
                      atomicOr(&q_nan[row * (D / 32) + (d >> 5)],
                               ((x >> 7 & 1) | (x >> 14 & 2) | (x >> 21 & 4) | (x >> 28 & 8)) << (d & 31));
              }
          }
        }
        // O^T
#pragma unroll
        for (int j = 0; j < VW; ++j) {
          const uint32_t x01 = __byte_perm(vw[0][j], vw[1][j], 0x5140), y01 = __byte_perm(vw[0][j], vw[1][j], 0x7362);
          const uint32_t x23 = __byte_perm(vw[2][j], vw[3][j], 0x5140), y23 = __byte_perm(vw[2][j], vw[3][j], 0x7362);
          uint32_t a0, a1, a2, a3, b0, b1, b2, b3;
          kv_codes4_to_f16<FMT>(x01, a0, a1);
          kv_codes4_to_f16<FMT>(x23, a2, a3);
          kv_codes4_to_f16<FMT>(y01, b0, b1);
          kv_codes4_to_f16<FMT>(y23, b2, b3);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            kv_mma(acc[2 * j][n], a0, a1, a2, a3, pb[n][0], pb[n][1]);
            kv_mma(acc[2 * j + 1][n], b0, b1, b2, b3, pb[n][0], pb[n][1]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[stage]);
      if (++stage == Cfg::STAGES) {
        stage = 0;
        phase ^= 1;
      }
    }

    if (!ok) break;

    // the four warps' (m, l, O) through shared memory
#pragma unroll
    for (int j = 0; j < 2 * NT; ++j)
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) l[j] += __shfl_xor_sync(0xFFFFFFFFu, l[j], o);
    float* part = reinterpret_cast<float*>(workspace + kKvSlotsAt + (2 * blockIdx.x + max(v.part - 1, 0)) * Cfg::SLOT);
    if (!warps_meet()) break;  // what was joined before has been read
#pragma unroll
    for (int j = 0; j < 2 * NT; ++j) {
      const int at = warp * Cfg::ROWS + (j >> 1) * 8 + 2 * c + (j & 1);
      if (g == 0) sML[at] = make_float2(m[j], l[j]);
#pragma unroll
      for (int k = 0; k < VW; ++k)
        *reinterpret_cast<float4*>(&sO[at * Cfg::O_STRIDE + (D / 8) * g + 4 * k]) =
            make_float4(acc[2 * k][j >> 1][j & 1], acc[2 * k][j >> 1][2 + (j & 1)], acc[2 * k + 1][j >> 1][j & 1],
                        acc[2 * k + 1][j >> 1][2 + (j & 1)]);
    }
    if (!warps_meet()) break;
    for (int i = tid; i < v.rows * (D / 4); i += 32 * kKvWarps) {
      const int row = i / (D / 4), d = i % (D / 4) * 4;
      float2 ml[kKvWarps];
      float most = -INFINITY;
#pragma unroll
      for (int k = 0; k < kKvWarps; ++k) {
        ml[k] = sML[k * Cfg::ROWS + row];
        most = fmaxf(most, ml[k].x);
      }
      const float ref = most == -INFINITY ? 0.f : most;
      float sum = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kKvWarps; ++k) {
        const float f = kv_exp2(ml[k].x - ref);
        const float4 x = *reinterpret_cast<const float4*>(&sO[(k * Cfg::ROWS + row) * Cfg::O_STRIDE + d]);
        sum = fmaf(ml[k].y, f, sum);
        o.x = fmaf(x.x, f, o.x);
        o.y = fmaf(x.y, f, o.y);
        o.z = fmaf(x.z, f, o.z);
        o.w = fmaf(x.w, f, o.w);
      }
      if (const uint32_t nan = q_nan[row * (D / 32) + (d >> 5)] >> (d & 31) & 15) {
        if (nan & 1) o.x = NAN;
        if (nan & 2) o.y = NAN;
        if (nan & 4) o.z = NAN;
        if (nan & 8) o.w = NAN;
      }
      if (v.part == 0) {
        kv_finish<D>(a, v.q0, row, group, v.head, d, most, sum, o);
      } else {
        *reinterpret_cast<float4*>(part + row * D + d) = o;
        if (d == 0) *reinterpret_cast<float2*>(part + Cfg::ROWS * D + 2 * row) = make_float2(most, sum);
      }
    }
    if (v.part) {
      // A part of a unit that range boundaries cut: the CTA that writes the last part joins them, in order.
      __threadfence();
      if (!warps_meet()) break;
      unsigned int* counter = reinterpret_cast<unsigned int*>(workspace) + v.first;
      if (tid == 0) {
        *last_part = atomicAdd(counter, 1u) == static_cast<unsigned>(v.parts) - 1;
        __threadfence();
      }
      if (!warps_meet()) break;
      if (*last_part) {
        const long long total = plan.total;
        for (int i = tid; i < v.rows * (D / 4); i += 32 * kKvWarps) {
          const int row = i / (D / 4), d = i % (D / 4) * 4;
          float most = -INFINITY, sum = 0.f;
          float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
          for (int k = 0; k < v.parts; ++k) {
            const int range = total < gridDim.x ? kv_range_of(total, v.place + k, gridDim.x) : v.first + k;
            const float* from = reinterpret_cast<const float*>(workspace + kKvSlotsAt + (2 * range + (k ? 0 : v.first_slot)) * Cfg::SLOT);
            const float2 ml = __ldcg(reinterpret_cast<const float2*>(from + Cfg::ROWS * D + 2 * row));
            const float4 x = __ldcg(reinterpret_cast<const float4*>(from + row * D + d));
            kv_join(most, sum, o, ml, x);
          }
          kv_finish<D>(a, v.q0, row, group, v.head, d, most, sum, o);
        }
        if (tid == 0) *counter = 0;
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&seg_empty[buf]);
  }
}

}  // namespace mxgb
