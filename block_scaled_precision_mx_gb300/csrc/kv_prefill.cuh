// kv_prefill.cuh -- attention over the paged 8-bit cache for more than 16 query rows a kv head (prompts,
// their chunks, drafts): the products are the bound, so both run on the tensor cores' own memory.
//
// A unit is 256 rows (query tokens x query heads of the group) of one request and kv head against the
// tokens that any of them sees, in tiles of 128.  One CTA a SM, persistent over an equal range of all
// units' tiles (found by the kernel itself for few requests, else by kv_plan_kernel); a unit cut by a range
// boundary leaves (O, m, l) in parts, which kv_join_kernel joins in order.  Roles:
//
//   warps 0-3, 4-7   softmax of rows 0-127 and 128-255, a row a thread.  They bring their queries into
//                    shared memory as FP16 (a power of two for each row, exact to 2^-29 of its largest),
//                    read S from tensor memory, write the weights back as FP16 over it, and keep m, l.
//                    Where a unit has at most 128 rows both work on them, on alternate tiles, with an O each.
//   warps 8-11       codes -> FP16 (exact) in the layout that the products read.
//   warp 12          walks the range, tells the others of its segments, and loads: TMA boxes of blocks' codes
//                    of K and V, tile by tile, and the scales of their 16-token slices.
//   warp 13          products:  S_w = Q_w K^T (M = 128, N = 128, K = D),  O_w += P_w V (P from tensor memory).
//
// The two row halves take turns: while one's softmax runs, the other's products do.  FP16 keeps every code
// exactly, so the only roundings are the weights' (2^-11) and the FP32 sums'.  As for few rows: sV is
// folded into the exponent, and the reference m is renewed only when a score passes it by 8; the row's O in
// tensor memory is then rescaled by its own thread, between two products.
//
// Measured (D = 128, 32 query and 8 kv heads, E4M3): 4096 queries over 32768 tokens 1.60 ms, 1.29 PFLOP/s, 0.66 of the
// measured bf16 rate; 6 prompts of 711 to 1500 tokens 193 us (872 units of 11 tiles; 75 us of products).
// What bounds it: a tile's products are 2048 cycles, but a half's chain of softmax (~2300 cycles: maximum 560,
// weights 1260, waits), its P V and its next S is ~3700, because S and P share tensor memory (O and S of two halves fill it) and S(i + 1) has to follow P(i) V; and shared memory carries 320 KB a tile (2560
// cycles: Q 64, K and V 64 each, the codes in, out and back as FP16 128).  Tried and slower: one pass over the
// scores with the weights held in registers until their maximum is known (2.2 ms), P V started at half of the
// weights (1.68 ms), 16 scores a step (1.82 ms), one row half's tiles split in columns (1.69 ms).
// Instruction supply decides much of this: with every role unrolled the same work took 3.0 ms, so each
// role's loop is short and rolled, and code that runs once a segment is short too (a segment's queries by an
// unrolled load of 16 rows a lane: 20000 cycles; by the present loops: 5000).
//
// Trees (TREE) of 17 rows a kv head and more take the same kernel with their own masks and a few changes that
// KvManyCfg names.  Their tiles are bound by chains, not by a pipe: of one row half a tile is ~2200 cycles (its codes'
// conversion by two warps 1500, softmax 1900 on alternate tiles, the products' handing over 500 each), of two ~3400.  Tried
// there and slower: scores of 64 tokens in two buffers a half with a tile's weights unrolled (98 us for 71, 387 for 257), codes
// brought to L2 ahead of their loads (92), the next 32 scores read while the present ones become weights (81), a warp
// for each of the two products (262 for 257), weights apart from the scores (256, not worth its code), and with them the
// maximum beside the weights in one pass, made again where the reference was too low (303).
#pragma once

#include "kv_attention.cuh"

namespace mxgb {

constexpr int kKvManyThreads = 512;
constexpr int kKvManyTile = 128;
constexpr int kKvManyRows = 256;
constexpr int kKvPlanThreads = 512;
constexpr int kKvManyMaxCtas = 160;

// A segment as the loading warp tells the others of it; count = 0: no more.
struct alignas(16) KvSegment {
  int count, token;           // tiles, and the first one's first token
  int rows, row0, q0, rows_q; // as in KvUnit
  int len, any_lo, all_lo, all_hi;
  int head;
  int part;                   // 0: the whole unit; 1 + slot: a part of it
};
static_assert(sizeof(KvSegment) <= 64, "a segment's place in shared memory");
constexpr int kKvManySegments = 4;

// TREE: a tree's rows, few for many tokens, so that a tile's way through the CTA counts: three groups of warps convert items
// in turn, D = 64 has twice the buffers, of one row half K and V come in the order of the products, a tile's mask bits are
// fetched at once, and the half that does not write brings the next queries (32 trees of 16 to 32 nodes, 4 query heads a kv
// head, up to 4096 tokens: 87 us without all that, 71 with it; 9 of 61 nodes, D = 64, windows of 20000: 272 and 257).  ONE: no unit has more than 128 rows, so that the place of the other half's queries is free.
template <int D, bool TREE, bool ONE>
struct KvManyCfg {
  static constexpr int RAW_SLOTS = !TREE ? 4 : D == 64 ? 8 : ONE ? 6 : 4, F16_SLOTS = TREE && D == 64 ? 6 : 3;
  // Tiles whose scales are kept: a tile's are written when its codes have a place, so RAW_SLOTS + F16_SLOTS items behind
  // what the products have done with; two more tiles may be under a softmax.
  static constexpr int SCALES = TREE && D == 64 ? 16 : 8;
  static_assert(SCALES >= (RAW_SLOTS + F16_SLOTS + 1) / 2 + 3, "scales");
  static constexpr int RAW = kKvManyTile * D;      // codes of K or V of a tile
  static constexpr int WIDE = 2 * RAW;             // the same in FP16; also 128 rows of Q
  static constexpr int OFF_F16 = (ONE ? 1 : 2) * WIDE;
  static constexpr int OFF_RAW = OFF_F16 + F16_SLOTS * WIDE;
  static constexpr int OFF_SC = OFF_RAW + RAW_SLOTS * RAW;          // float2 [tiles][8 slices]: sK, log2 sV
  static constexpr int OFF_MUL = OFF_SC + SCALES * 8 * 8;    // float [128], for one row half
  static constexpr int OFF_NAN = OFF_MUL + 4 * 128;                 // int [tiles]
  static constexpr int OFF_BAR = OFF_NAN + 4 * SCALES;
  static constexpr int BARS = 2 * RAW_SLOTS + 2 * F16_SLOTS + 4 * 2 + SCALES + 2 * kKvManySegments + 4;
  static constexpr int OFF_SEG = (OFF_BAR + 8 * BARS + 15) / 16 * 16;  // KvSegment [segments]
  static constexpr int SMEM = OFF_SEG + 64 * kKvManySegments + 16 + 1024;
  static constexpr size_t SLOT = static_cast<size_t>(kKvManyRows) * (D + 2) * 4;
  // warps that convert an item, and how many such groups there are
  static constexpr int CONVERT = TREE ? 2 : 4, GROUPS = TREE ? 3 : 1;
  static constexpr size_t NAN_BYTES = 4 * kKvManyTile * (D / 8);    // u16 [4 tiles][128 tokens][D / 16] a CTA
};

// workspace: jobs, the requests' places (8 bytes each), NaN notes, segments
__host__ __device__ constexpr size_t kv_many_nan_at(int64_t requests) {
  return kKvSlotsAt + static_cast<size_t>((8 * (requests + 1) + 31) / 32 * 32);
}
__host__ __device__ constexpr size_t kv_many_slots_at(int64_t requests, int head_dim) {
  return kv_many_nan_at(requests) + static_cast<size_t>(kKvManyMaxCtas) * 4 * kKvManyTile * (head_dim / 8);
}

struct KvUnit {
  int q0, rows_q, len;                // the request
  int row0, rows;                     // this unit's rows of its head group
  int first_tile, tiles;
  int any_lo, any_hi, all_lo, all_hi; // tokens [any_lo, any_hi) are seen by some row; [all_lo, all_hi) by all
  __device__ __forceinline__ int cost() const { return tiles + kKvUnitCost; }
};

template <bool TREE>
__device__ __forceinline__ KvUnit kv_unit(const KvAttnArgs& a, const KvRequest& req, int group, int q_tile) {
  KvUnit u;
  u.q0 = req.q0;
  u.rows_q = req.rows_q;
  u.len = req.len;
  u.row0 = q_tile * kKvManyRows;
  u.rows = min(kKvManyRows, req.rows_q * group - u.row0);
  // (a tree's rows may stand at any of its positions)
  const int p0 = req.len - req.rows_q + (TREE ? 0 : u.row0 / group);
  const int p1 = TREE ? req.len - 1 : req.len - req.rows_q + (u.row0 + u.rows - 1) / group;
  u.any_lo = a.window ? max(0, p0 - a.window + 1) : 0;
  u.all_lo = a.window ? max(0, p1 - a.window + 1) : 0;
  u.all_hi = TREE ? p0 : a.causal ? min(req.len, p0 + 1) : req.len;
  u.any_hi = a.causal ? min(req.len, p1 + 1) : req.len;
  u.first_tile = u.any_lo / kKvManyTile;
  u.tiles = max(1, (max(u.any_hi, 0) + kKvManyTile - 1) / kKvManyTile - u.first_tile);
  return u;
}
__device__ __forceinline__ int kv_units_of(const KvRequest& req, int group) {
  return (req.rows_q * group + kKvManyRows - 1) / kKvManyRows;
}

// The unit of request r, whose units begin at place x, that job.begin falls into.
template <bool TREE>
__device__ __forceinline__ void kv_first_unit(const KvAttnArgs& a, const KvRequest& req, int r, int group, long long x,
                                              KvJob& job) {
#pragma unroll 1
  for (int q_tile = 0;; ++q_tile) {
    const KvUnit u = kv_unit<TREE>(a, req, group, q_tile);
    const long long all = static_cast<long long>(u.cost()) * a.kv_heads;
    if (job.begin < x + all) {
      job.head = static_cast<int>((job.begin - x) / u.cost());
      job.unit = x + static_cast<long long>(job.head) * u.cost();
      job.tiles = u.tiles;
      job.q0 = u.q0;
      job.row0 = u.row0;
      job.rows = u.rows;
      job.request = r;
      job.q_tile = q_tile;
      return;
    }
    x += all;
  }
}

// Ranges of the list of all units (request by request, then 256 rows by 256 rows, then head by head): one
// CTA sums the requests' costs, scans them and finds each range's first unit.  A request's units are summed
// by a thread while they are few, by a warp otherwise.
template <bool TREE>
__global__ void __launch_bounds__(kKvPlanThreads) kv_plan_kernel(const KvAttnArgs a, int most_q, int ranges,
                                                                 uint8_t* workspace) {
  pdl_prologue();
  __shared__ long long warp_sum[kKvPlanThreads / 32];
  long long* place = reinterpret_cast<long long*>(workspace + kKvSlotsAt);  // [requests + 1]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, group = a.heads / a.kv_heads;
  if (static_cast<long long>(most_q) * group <= 8 * kKvManyRows) {
    for (int r = tid; r < a.requests; r += kKvPlanThreads) {
      const KvRequest req = kv_request<TREE>(a, r, most_q, true);
      const int units = kv_units_of(req, group);
      long long sum = 0;
      for (int i = 0; i < units; ++i) sum += kv_unit<TREE>(a, req, group, i).cost();
      place[r] = sum * a.kv_heads;
    }
  } else {
    for (int r = warp; r < a.requests; r += kKvPlanThreads / 32) {
      const KvRequest req = kv_request<TREE>(a, r, most_q, lane == 0);
      const int units = kv_units_of(req, group);
      long long sum = 0;
      for (int i = lane; i < units; i += 32) sum += kv_unit<TREE>(a, req, group, i).cost();
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
      if (lane == 0) place[r] = sum * a.kv_heads;
    }
  }
  __syncthreads();
  const int per = (a.requests + kKvPlanThreads - 1) / kKvPlanThreads;
  const int r0 = min(tid * per, a.requests), r1 = min(r0 + per, a.requests);
  long long mine = 0;
  for (int r = r0; r < r1; ++r) mine += place[r];
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  long long at = incl - mine, total = 0;
  for (int i = 0; i < kKvPlanThreads / 32; ++i) {
    if (i < warp) at += warp_sum[i];
    total += warp_sum[i];
  }
  for (int r = r0; r < r1; ++r) {
    const long long c = place[r];
    place[r] = at;
    at += c;
  }
  if (tid == 0) place[a.requests] = total;
  __syncthreads();
  KvJob* jobs = reinterpret_cast<KvJob*>(workspace + kKvJobsAt);
  for (int c = tid; c < ranges; c += kKvPlanThreads) {
    KvJob job{kv_cut(total, c, ranges), kv_cut(total, c + 1, ranges), 0, 0, 0, 0, 0, 0, 0, 0};
    if (job.begin < total) {
      int lo = 0, hi = a.requests;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (place[mid] <= job.begin) lo = mid;
        else hi = mid;
      }
      kv_first_unit<TREE>(a, kv_request<TREE>(a, lo, most_q, false), lo, group, place[lo], job);
    }
    jobs[c] = job;
  }
}

struct KvManyWalk {
  long long pos, end, base;
  int r, h, q_tile;
  KvRequest req;
  KvUnit u;
  int tile, count;  // the current segment
};
template <bool TREE>
__device__ __forceinline__ void kv_many_begin(const KvAttnArgs& a, int most_q, int group, const KvJob& job, KvManyWalk& w) {
  w.pos = job.begin;
  w.end = job.end;
  w.base = job.unit;
  w.r = job.request;
  w.h = job.head;
  w.q_tile = job.q_tile;
  if (w.pos < w.end) {
    w.req = kv_request<TREE>(a, w.r, most_q, false);
    w.u = kv_unit<TREE>(a, w.req, group, w.q_tile);
  }
}
template <bool TREE>
__device__ __noinline__ bool kv_many_next(const KvAttnArgs& a, int most_q, int group, KvManyWalk& w) {
  while (w.pos < w.end) {
    const long long unit_end = w.base + w.u.cost();
    if (w.pos == unit_end) {
      w.base = unit_end;
      if (++w.h == a.kv_heads) {
        w.h = 0;
        if (++w.q_tile >= kv_units_of(w.req, group)) {
          w.q_tile = 0;
          do {
            if (++w.r >= a.requests) return false;
            w.req = kv_request<TREE>(a, w.r, most_q, false);
          } while (w.req.rows_q == 0);
        }
        w.u = kv_unit<TREE>(a, w.req, group, w.q_tile);
      }
      continue;
    }
    const long long to = min(w.end, unit_end);
    w.tile = kv_tiles_before(w.pos - w.base, w.u.tiles);
    w.count = kv_tiles_before(to - w.base, w.u.tiles) - w.tile;
    w.pos = to;
    if (w.count) return true;
  }
  return false;
}

// kind::f16: FP16 operands, FP32 accumulator; B K-major or N-major
__host__ __device__ constexpr uint32_t kv_idesc_f16(uint32_t M, uint32_t N, bool b_n_major) {
  return (1u << 4) | (b_n_major ? 1u << 16 : 0u) | ((N >> 3) << 17) | ((M >> 4) << 24);
}
__device__ __forceinline__ void umma_f16_ss(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// 32 bytes a thread, a whole sector: a warp's threads write rows apart from each other.  (Two stores of 16: 6 x 1500
// 202 us against 193.)  What fills the registers is straight code, with the type known to the compiler: filled in two
// branches, FP16 or bf16, such a store once wrote wrong pairs, and why is not known.
__device__ __forceinline__ void kv_store32(void* to, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]),
               "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// one thread of a converged warp
__device__ __forceinline__ bool kv_elect() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ uint64_t kv_fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

__device__ __forceinline__ uint64_t kv_add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// The items of a segment of n tiles, in the order in which the products take them: K and V of each tile; of a tree's one
// row half, whose halves take alternate tiles, K0 K1 V0 K2 V1 .. V(n-1), so that a K's buffer is that of the V two
// tiles before the one whose product comes first.
__device__ __forceinline__ uint32_t kv_item_k(bool apart, uint32_t tile) { return apart && tile ? 2 * tile - 1 : 2 * tile; }
__device__ __forceinline__ uint32_t kv_item_v(bool apart, uint32_t tile, uint32_t n) {
  return apart && tile + 1 < n ? 2 * tile + 2 : 2 * tile + 1;
}
// the tile of item i, and whether it is a V
__device__ __forceinline__ uint32_t kv_item_tile(bool apart, uint32_t i, uint32_t n, bool& is_v) {
  is_v = apart ? i == 2 * n - 1 || (i && !(i & 1)) : i & 1;
  return !apart || i == 2 * n - 1 ? i >> 1 : is_v ? (i >> 1) - 1 : (i + 1) >> 1;
}

// One lane's box of codes in place of a load.  (Rare.)
__device__ __noinline__ void kv_fill_box(uint8_t* to, int bytes, uint32_t four) {
  for (int i = 0; i < bytes; i += 16) *reinterpret_cast<uint4*>(to + i) = make_uint4(four, four, four, four);
  fence_proxy_async_smem();  // (a copy may come to the same place next)
}

// Which of a tile's 128 tokens, from `token` on, a row of a tree sees, as bits: `nodes` is its row of the mask (null: none of
// the nodes), first the first token that it sees of those in front of the nodes, n how many nodes there are.
struct KvTreeBits {
  uint64_t b[2];
};
__device__ __forceinline__ KvTreeBits kv_tree_bits(const uint64_t* nodes, int words, int n, int context, int first, int token) {
  const int o = token - context, w0 = o >> 6, sh = o & 63;
  uint64_t x[3];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    const int w = w0 + k, left = n - 64 * w;  // (w < 0: what is in front of the nodes)
    uint64_t word = w < 0 ? ~0ull : 0;
    if (w >= 0 && left > 0 && w < words && nodes) word = nodes[w] & (left < 64 ? (1ull << left) - 1 : ~0ull);
    x[k] = word;
  }
  KvTreeBits v;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    v.b[k] = sh ? x[k] >> sh | x[k + 1] << (64 - sh) : x[k];
    const int hidden = first - token - 64 * k;
    if (hidden > 0) v.b[k] = hidden < 64 ? v.b[k] & (~0ull << hidden) : 0;
  }
  return v;
}

template <int FMT, int D, bool F16, bool TREE, bool ONE>
__global__ void __launch_bounds__(kKvManyThreads, 1)
    kv_attention_many_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                             const KvAttnArgs a, int most_q, int planned, uint8_t* workspace) {
  using Cfg = KvManyCfg<D, TREE, ONE>;
  extern __shared__ uint8_t kv_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(kv_smem_raw) + 1023) & ~uintptr_t(1023));
  float2* sSC = reinterpret_cast<float2*>(smem + Cfg::OFF_SC);
  float* sMul = reinterpret_cast<float*>(smem + Cfg::OFF_MUL);
  volatile int* sNan = reinterpret_cast<volatile int*>(smem + Cfg::OFF_NAN);
  KvSegment* sSeg = reinterpret_cast<KvSegment*>(smem + Cfg::OFF_SEG);
  uint64_t* raw_full = reinterpret_cast<uint64_t*>(smem + Cfg::OFF_BAR);
  uint64_t* raw_empty = raw_full + Cfg::RAW_SLOTS;
  uint64_t* f_full = raw_empty + Cfg::RAW_SLOTS;
  uint64_t* f_empty = f_full + Cfg::F16_SLOTS;
  uint64_t* q_full = f_empty + Cfg::F16_SLOTS;  // [2] each
  uint64_t* s_full = q_full + 2;
  uint64_t* p_full = s_full + 2;
  uint64_t* o_full = p_full + 2;
  uint64_t* sc_full = o_full + 2;               // [Cfg::SCALES]
  uint64_t* seg_full = sc_full + Cfg::SCALES; // [kKvManySegments]
  uint64_t* seg_empty = seg_full + kKvManySegments;
  uint64_t* join_full = seg_empty + kKvManySegments;
  uint64_t* join_empty = join_full + 1;
  uint64_t* drain_bar = join_empty + 1;
  uint64_t* turn = drain_bar + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::OFF_SEG + 64 * kKvManySegments);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;
  const int group = a.heads / a.kv_heads;
  if (tid == 0) {
    for (int i = 0; i < Cfg::RAW_SLOTS; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], Cfg::CONVERT);
    }
    for (int i = 0; i < Cfg::F16_SLOTS; ++i) {
      mbar_init(&f_full[i], Cfg::CONVERT);
      mbar_init(&f_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 4);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&o_full[i], 1);
    }
    for (int i = 0; i < Cfg::SCALES; ++i) mbar_init(&sc_full[i], 1);
    for (int i = 0; i < kKvManySegments; ++i) {
      mbar_init(&seg_full[i], 1);
      mbar_init(&seg_empty[i], 9 + Cfg::CONVERT * Cfg::GROUPS);  // all that walk the segments but the loading warp
    }
    mbar_init(join_full, 4);
    mbar_init(join_empty, 4);
    mbar_init(drain_bar, 1);
    mbar_init(turn, 4);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  if (warp == 13) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);
  pdl_wait();
  kv_clear_rest(a, D, blockIdx.x * kKvManyThreads + tid, gridDim.x * kKvManyThreads);
  __shared__ KvJob job;
  if (planned) {
    if (tid == 0) job = reinterpret_cast<const KvJob*>(workspace + kKvJobsAt)[blockIdx.x];
  } else {
    // Few requests of few units: every CTA finds its own range, a request a thread (a launch of kv_plan_kernel less).
    __shared__ long long warp_sum[kKvManyThreads / 32];
    KvRequest req{};
    long long mine = 0;
    if (tid < a.requests) {
      req = kv_request<TREE>(a, tid, most_q, blockIdx.x == 0);
      const int units = kv_units_of(req, group);
#pragma unroll 1
      for (int i = 0; i < units; ++i) mine += kv_unit<TREE>(a, req, group, i).cost();
    }
    mine *= a.kv_heads;
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += u;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    long long before = incl - mine, total = 0;
#pragma unroll 1
    for (int i = 0; i < kKvManyThreads / 32; ++i) {
      if (i < warp) before += warp_sum[i];
      total += warp_sum[i];
    }
    KvJob mine_job{kv_cut(total, blockIdx.x, gridDim.x), kv_cut(total, blockIdx.x + 1, gridDim.x), 0, 0, 0, 0, 0, 0, 0, 0};
    const bool here = mine_job.begin >= before && mine_job.begin < before + mine;
    if (here) kv_first_unit<TREE>(a, req, tid, group, before, mine_job);
    if (here || (total == 0 && tid == 0)) {
      job = mine_job;
      reinterpret_cast<KvJob*>(workspace + kKvJobsAt)[blockIdx.x] = mine_job;
    }
  }
  __syncthreads();
  uint8_t* nan_notes = workspace + kv_many_nan_at(a.requests) + blockIdx.x * Cfg::NAN_BYTES;

  // the next segment, for every warp but the loading one; false at the end
  uint32_t seg = 0;
  auto next_segment = [&](KvSegment& v) {
    const uint32_t i = seg % kKvManySegments;
    const bool ok = kv_wait(&seg_full[i], (seg / kKvManySegments) & 1, abort_flag, kSiteMmaFull);
    v = sSeg[i];
    __syncwarp();
    if (lane == 0) mbar_arrive(&seg_empty[i]);
    ++seg;
    return ok && v.count > 0;
  };

  if (warp == 12) {
    // ------------------------------------------------------------------ loads
    KvManyWalk w;
    kv_many_begin<TREE>(a, most_q, group, job, w);
    const long long range_start = w.pos;
    const int P = 1 << a.shift, rows_box = min(P, kKvTile), boxes = kKvManyTile / rows_box;
    const int most_tiles = 32 * P / kKvManyTile;
    uint32_t tiles_done = 0, issued = 0;  // issued: items
    int row_before = -1, take_before = 0;  // this lane's box of the tile before
    bool ok = true, odd_before = false;
    // the next item: this lane's box from `row` on (-1: none), or codes that are taken as something else
    auto load_item = [&](int v, int row, int taken, bool odd) {
      const uint32_t slot = issued % Cfg::RAW_SLOTS;
      if (!kv_wait(&raw_empty[slot], ((issued / Cfg::RAW_SLOTS) & 1) ^ 1, abort_flag, kSiteProducerEmpty)) {
        ok = false;
        return false;
      }
      uint8_t* dst = smem + Cfg::OFF_RAW + slot * Cfg::RAW + lane * rows_box * D;
      const bool load = lane < boxes && row >= 0 && !taken;
      const uint32_t bytes = __popc(__ballot_sync(0xFFFFFFFFu, load)) * rows_box * D;
      if (odd) {
        if (lane < boxes && taken) kv_fill_box(dst, rows_box * D, kv_four_taken(taken));
        __syncwarp();
      }
      ++issued;
      if (lane == 0) mbar_arrive_expect_tx(&raw_full[slot], bytes);
      __syncwarp();
      if (load) tma_load_2d(dst, v ? &tmV : &tmK, &raw_full[slot], 0, row);
      return true;
    };
    while (ok) {
      const bool more = kv_many_next<TREE>(a, most_q, group, w);
      const uint32_t sl = seg % kKvManySegments;
      if (!kv_wait(&seg_empty[sl], ((seg / kKvManySegments) & 1) ^ 1, abort_flag, kSiteProducerEmpty)) break;
      if (lane == 0) {
        const int part = w.count == w.u.tiles ? 0 : w.base < range_start ? 1 : 2;
        KvSegment v{more ? w.count : 0, (w.u.first_tile + w.tile) * kKvManyTile, w.u.rows, w.u.row0, w.u.q0, w.u.rows_q,
                    w.u.len, w.u.any_lo, w.u.all_lo, w.u.all_hi, w.h, part};
        sSeg[sl] = v;
        mbar_arrive(&seg_full[sl]);
      }
      ++seg;
      if (!more) break;
      for (int i0 = 0; i0 < w.count && ok; i0 += most_tiles) {  // up to 32 blocks at a time
        const int n = min(most_tiles, w.count - i0), token0 = (w.u.first_tile + w.tile + i0) * kKvManyTile;
        const int page = (token0 >> a.shift) + lane;
        int block = -1;
        float sk = 1.f, sv = 1.f;
        const bool told = page << a.shift < w.u.any_hi;  // (behind any_hi another unit's rows may see it)
        if (page << a.shift < w.u.len && (page + 1) << a.shift > w.u.any_lo)  // (in front of any_lo no row sees it)
          kv_look_up(a, w.r, page, w.h, block, sk, sv);
        const int take = kv_check_scales(sk, sv, told);
        const bool odd = __any_sync(0xFFFFFFFFu, take != 0);  // some block's codes are not taken as they are
        for (int i = 0; i < n && ok; ++i, ++tiles_done) {
          const int token = token0 + i * kKvManyTile, from = (token - token0) >> a.shift;
          const int my = token + lane * rows_box;
          const int box_at = min((my - token0) >> a.shift, 31), box_block = __shfl_sync(0xFFFFFFFFu, block, box_at);
          const int box_take = odd ? __shfl_sync(0xFFFFFFFFu, take, box_at) : 0;
          const int slice = ((lane & 7) * 16) >> a.shift;
          const float slice_k = __shfl_sync(0xFFFFFFFFu, sk, from + slice), slice_v = __shfl_sync(0xFFFFFFFFu, sv, from + slice);
          const int box_row = box_block >= 0 ? ((box_block * a.kv_heads + w.h) << a.shift) + (my & (P - 1)) : -1;
          const bool apart = TREE && (ONE || w.u.rows <= 128), last = i0 + i + 1 == w.count;
          // K of this tile; V of this one, or of the one before
          if (!load_item(0, box_row, box_take & 0xFF, odd)) break;
          const uint32_t st = tiles_done % Cfg::SCALES;
          if (lane < 8) sSC[st * 8 + lane] = make_float2(slice_k, log2f(slice_v));
          if (lane == 0) sNan[st] = 0;
          __syncwarp();
          if (lane == 0) mbar_arrive(&sc_full[st]);
          if (!apart) {
            load_item(1, box_row, box_take >> 8, odd);
          } else {
            if (i0 + i) load_item(1, row_before, take_before, odd || odd_before);
            if (last && ok) load_item(1, box_row, box_take >> 8, odd);
            row_before = box_row;
            take_before = box_take >> 8;
            odd_before = odd;
          }
        }
      }
    }
    // every copy has landed before the CTA's shared memory goes
    for (uint32_t i = 0; i < Cfg::RAW_SLOTS; ++i)
      if (issued > i) mbar_drain(&raw_full[i], kv_ring_last_parity(issued, i, Cfg::RAW_SLOTS), kWaitBudgetNs);
  } else if (warp == 13) {
    // ------------------------------------------------------------------ products (the whole warp keeps step, one thread issues)
    constexpr uint32_t kHi = smem_desc_hi(1024, kSwizzle128B);
    constexpr uint32_t kLoK = smem_desc_lo_lbo(16), kLoN = smem_desc_lo_lbo(kKvManyTile * 128);
    constexpr uint32_t kIdS = kv_idesc_f16(128, kKvManyTile, false), kIdO = kv_idesc_f16(128, D, true);
    const uint32_t q_lo = (smem_u32(smem) >> 4) | kLoK, f_lo = smem_u32(smem + Cfg::OFF_F16) >> 4;
    uint32_t tiles_done = 0, segments[2] = {0, 0}, weights[2] = {0, 0};
    bool ok = true;
    KvSegment v;
    while (ok && next_segment(v)) {
      const int count = __shfl_sync(0xFFFFFFFFu, v.count, 0);
      const bool single = ONE || v.rows <= 128, apart = TREE && single;
      const int steps = single ? count + 2 : 2 * (count + 1);
      for (int step = 0; step < steps && ok; ++step) {
        // half h: V of an earlier tile, then K of the next.  Two row halves: both take every tile; one: every second.
        const int h = step & 1, pv = single ? step - 2 : (step >> 1) - 1, sc = single ? step : step >> 1;
        const bool frees = single || h == 1;
        if (pv >= 0) {
          const uint32_t item = 2 * tiles_done + kv_item_v(apart, pv, count), slot = item % Cfg::F16_SLOTS;
          ok = kv_wait(&f_full[slot], (item / Cfg::F16_SLOTS) & 1, abort_flag, kSiteMmaFull) &&
               kv_wait(&p_full[h], weights[h]++ & 1, abort_flag, kSiteMmaTmemEmpty);
          if (!ok) break;
          tc_fence_after();
          const uint32_t v_lo = __shfl_sync(0xFFFFFFFFu, (f_lo + slot * (Cfg::WIDE / 16)) | kLoN, 0);
          const bool first = single ? pv < 2 : pv == 0;
          if (kv_elect()) {
#pragma unroll
            for (int k = 0; k < kKvManyTile / 16; ++k)  // O_h += P_h V, 16 tokens at a time
              umma_f16_ts(tmem + 256 + h * 128, tmem + h * 128 + k * 8, desc_from_words(v_lo + k * (16 * 128 / 16), kHi), kIdO,
                          !first || k > 0);
            if (pv >= count - (single ? 2 : 1)) umma_commit(&o_full[h]);
            if (frees) umma_commit(&f_empty[slot]);
          }
          __syncwarp();
        }
        if (sc < count) {
          const uint32_t item = 2 * tiles_done + kv_item_k(apart, sc), slot = item % Cfg::F16_SLOTS;
          ok = kv_wait(&f_full[slot], (item / Cfg::F16_SLOTS) & 1, abort_flag, kSiteMmaFull);
          if (ok && sc == 0) ok = kv_wait(&q_full[h], segments[h]++ & 1, abort_flag, kSiteMmaFull);
          if (!ok) break;
          tc_fence_after();
          const uint32_t k_lo = __shfl_sync(0xFFFFFFFFu, (f_lo + slot * (Cfg::WIDE / 16)) | kLoK, 0);
          const uint32_t qh_lo = q_lo + (single ? 0 : h) * (Cfg::WIDE / 16);
          if (kv_elect()) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {  // S_h = Q_h K^T
              const uint32_t at = (k / 4) * (kKvManyTile * 128 / 16) + (k % 4) * 2;
              umma_f16_ss(tmem + h * 128, desc_from_words(qh_lo + at, kHi), desc_from_words(k_lo + at, kHi), kIdS, k > 0);
            }
            umma_commit(&s_full[h]);
            if (frees) umma_commit(&f_empty[slot]);
          }
          __syncwarp();
        }
      }
      tiles_done += count;
    }
    // every product has ended before the tensor memory goes
    if (kv_elect()) {
      umma_commit(drain_bar);
      mbar_drain(drain_bar, 0, kWaitBudgetNs);
    }
    __syncwarp();
  } else if (warp >= 8 && warp < (TREE ? 16 : 12)) {
    // ------------------------------------------------------------------ codes -> FP16
    constexpr int CH = D / 16;  // 16-code words of a token
    constexpr int WORDS = CH * 4 / Cfg::CONVERT, STEP = TREE ? 4 : 2;  // words of a lane, and those taken at once
    const int wq = (warp - 8) % Cfg::CONVERT, tl = lane & 7;
    const uint32_t mine = warp < 12 ? (warp - 8) / Cfg::CONVERT : 2;  // warps 14 and 15 are the last group
    uint32_t tiles_done = 0;
    bool ok = true;
    KvSegment v;
    while (ok && next_segment(v)) {
      const uint32_t items = 2 * (tiles_done + v.count);
      const bool apart = TREE && (ONE || v.rows <= 128);
#pragma unroll 1
      for (uint32_t item = 2 * tiles_done; item < items; ++item) {
        if (Cfg::GROUPS > 1 && item % Cfg::GROUPS != mine) continue;
        const uint32_t slot = item % Cfg::RAW_SLOTS, fs = item % Cfg::F16_SLOTS;
        ok = kv_wait(&raw_full[slot], (item / Cfg::RAW_SLOTS) & 1, abort_flag, kSiteMmaFull) &&
             kv_wait(&f_empty[fs], ((item / Cfg::F16_SLOTS) & 1) ^ 1, abort_flag, kSiteProducerEmpty);
        if (!ok) break;
        uint8_t* src = smem + Cfg::OFF_RAW + slot * Cfg::RAW;
        uint8_t* dst = smem + Cfg::OFF_F16 + fs * Cfg::WIDE;
        // lane: row tl of 8, word lane / 8 of 4; D = 128 has two groups of 4 words
        auto raw_at = [&](int n, int& row, int& word) {
          row = 128 / Cfg::CONVERT * wq + 8 * (n / (CH / 4)) + tl;
          word = (n % (CH / 4)) * 4 + (lane >> 3);
          return reinterpret_cast<uint4*>(src + (D == 128 ? row * 128 + ((word ^ (row & 7)) << 4)
                                                          : row * 64 + ((word ^ ((row >> 1) & 3)) << 4)));
        };
        bool is_v;
        const uint32_t nth = kv_item_tile(apart, item - 2 * tiles_done, v.count, is_v), tile = tiles_done + nth;
        const int token = v.token + static_cast<int>(nth) * kKvManyTile;
        if (is_v && (token < v.all_lo || token + kKvManyTile > v.all_hi)) {
          // V of a tile that some row does not see whole: clear what no row sees; take NaN codes out and note them
          uint32_t any = 0;
#pragma unroll 1
          for (int n = 0; n < WORDS; ++n) {
            int row, word;
            uint4* at = raw_at(n, row, word);
            const uint4 x = *at;
            const bool out = token + row < v.any_lo || token + row >= v.len;
            uint32_t c[4] = {x.x, x.y, x.z, x.w}, bits = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (out) c[j] = 0;
              const uint32_t y = kv_nan_bytes<FMT>(c[j]);
              c[j] &= ~((y >> 7) * 0xFFu);
              bits |= ((y >> 7 & 1) | (y >> 14 & 2) | (y >> 21 & 4) | (y >> 28 & 8)) << (4 * j);
            }
            *at = make_uint4(c[0], c[1], c[2], c[3]);
            reinterpret_cast<uint16_t*>(nan_notes)[((tile & 3) * kKvManyTile + row) * CH + word] = static_cast<uint16_t>(bits);
            any |= bits;
          }
          if (any) sNan[tile % Cfg::SCALES] = 1;
          __threadfence_block();
        }
#pragma unroll 1
        for (int n0 = 0; n0 < WORDS; n0 += STEP) {
          uint4 x[STEP];
          int row[STEP], word[STEP];
#pragma unroll
          for (int n = 0; n < STEP; ++n) x[n] = *raw_at(n0 + n, row[n], word[n]);
#pragma unroll
          for (int n = 0; n < STEP; ++n) {
            const uint32_t c[4] = {x[n].x, x[n].y, x[n].z, x[n].w};
            uint32_t f[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) kv_codes4_to_f16<FMT>(c[j], f[2 * j], f[2 * j + 1]);
            uint8_t* to = dst + (word[n] >> 2) * (kKvManyTile * 128) + row[n] * 128;
            const int ch = (word[n] & 3) * 2;
            *reinterpret_cast<uint4*>(to + ((ch ^ (row[n] & 7)) << 4)) = make_uint4(f[0], f[1], f[2], f[3]);
            *reinterpret_cast<uint4*>(to + (((ch + 1) ^ (row[n] & 7)) << 4)) = make_uint4(f[4], f[5], f[6], f[7]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&raw_empty[slot]);
          mbar_arrive(&f_full[fs]);
        }
      }
      tiles_done += v.count;
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------------ softmax, a row a thread
    const int half = warp >> 2, row = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + half * 128 + lanes, tO = tmem + 256 + half * 128 + lanes;
    uint32_t tiles_done = 0, my_tiles = 0, segments = 0, joins = 0;
    uint32_t other_segments = 0;  // half 1's segments with tiles, as half 0 counts them
    bool ok = true;
    // A segment's queries as FP16; returns what this thread's row of scores is to be multiplied with.  The rows
    // are copied to their places as they are, D / 8 lanes a row, and converted there, a row a thread.  (Short
    // loops: code that runs once a segment is not in the instruction cache, and costs by its length.)
    // Of one row half `by` brings the rows of both.
    auto bring = [&](const KvSegment& v, int by) {
      constexpr int LANES = D / 8, AT_ONCE = 32 / LANES;
      const bool single = ONE || v.rows <= 128;
      uint8_t* sQ = smem + (single ? 0 : half) * Cfg::WIDE;
      const int rows_at = single ? 0 : half * 128;
      if (single && half != by) {
        ok = kv_wait(&q_full[0], (seg - 1) & 1, abort_flag, kSiteEpiTmemFull);
        return sMul[row];
      }
      const int word = lane % LANES, sub = lane / LANES, row0 = 32 * (warp & 3);
      int r = row0 + sub, qi = (v.row0 + rows_at + r) / group, hg = v.row0 + rows_at + r - qi * group;
      const int qi_step = AT_ONCE / group, hg_step = AT_ONCE % group;
      const uint32_t to = smem_u32(sQ) + (word >> 3) * (128 * 128);
#pragma unroll 1
      for (; r < row0 + 32; r += AT_ONCE) {
        const uint16_t* src = a.q + (v.q0 + qi) * a.stride_t + (v.head * group + hg) * a.stride_h + 8 * word;
        const uint32_t bytes = rows_at + r < v.rows ? 16 : 0;  // (the rest of the 16 is zeros)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + r * 128 + (((word & 7) ^ (r & 7)) << 4)),
                     "l"(bytes ? src : a.q), "r"(bytes)
                     : "memory");
        qi += qi_step;
        hg += hg_step;
        if (hg >= group) {
          hg -= group;
          ++qi;
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncwarp();
      auto chunk = [&](int i) {
        return reinterpret_cast<uint4*>(sQ + (i >> 3) * (128 * 128) + row * 128 + (((i & 7) ^ (row & 7)) << 4));
      };
      uint32_t most2 = 0;
#pragma unroll 4
      for (int i = 0; i < D / 8; ++i) {
        const uint4 x = *chunk(i);
        most2 = __vmaxu2(most2, __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu), __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu)));
      }
      const uint32_t most1 = max(most2 & 0xFFFFu, most2 >> 16);
      const float amax = F16 ? __half2float(__ushort_as_half(static_cast<unsigned short>(most1))) : __uint_as_float(most1 << 16);
      // 2^e with amax 2^e in [2^14, 2^15)
      const int e = min(14 - (static_cast<int>(__float_as_uint(amax) >> 23) - 127), 120);
      const float mul = most1 ? __uint_as_float(static_cast<uint32_t>(e + 127) << 23) : 1.f;
#pragma unroll 2
      for (int i = 0; i < D / 8; ++i) {
        const uint4 x = *chunk(i);
        const uint32_t u[4] = {x.x, x.y, x.z, x.w};
        uint32_t f[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 y = kv_unpack2<F16>(u[j]);
          f[j] = kv_pack_f16(y.x * mul, y.y * mul);
        }
        *chunk(i) = make_uint4(f[0], f[1], f[2], f[3]);
      }
      // Times a block's scale (2^-48 at least) it is not to become 0: masked scores are -inf before that product, and
      // -inf * 0 is no mask.  At 2^-101 and below, every score (below 2^38 before it, times 2^48 at most) is 0 to 2^-15.
      const float row_mul = fmaxf(a.scale_log2 / mul, 1.f / (1ull << 50) / (1ull << 51));
      if (single) sMul[row] = row_mul;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[single ? 0 : half]);
      return row_mul;
    };
    KvSegment v;
    bool more = next_segment(v);
    float row_mul = more ? bring(v, 0) : 0.f;
    while (ok && more) {
      const bool single = ONE || v.rows <= 128;  // both halves work on the same rows, on every second tile
      const int my_row = single ? row : 128 * half + row;
      const bool live = my_row < v.rows;
      const int qi = (v.row0 + my_row) / group, hg = v.row0 + my_row - qi * group;
      const int context = v.len - v.rows_q, p = context + qi;
      const uint64_t* nodes = TREE && live ? a.tree_mask + static_cast<int64_t>(v.q0 + qi) * a.tree_words : nullptr;
      const int lo = TREE ? (live ? kv_tree_first(a, v.q0 + qi, context, v.rows_q) : 0) : a.window ? max(0, p - a.window + 1) : 0;
      const int hi = TREE ? context : a.causal ? min(v.len, p + 1) : v.len;
      const uint32_t width = static_cast<uint32_t>(max(hi - lo, 0));
      const int first = single ? half : 0;
      float m = -INFINITY, l = 0.f;
      uint32_t nan_d[D / 32];
#pragma unroll
      for (int i = 0; i < D / 32; ++i) nan_d[i] = 0;
#pragma unroll 1
      for (int i = first; i < v.count; i += single ? 2 : 1, ++my_tiles) {
        const int token = v.token + i * kKvManyTile;
        const uint32_t tile = tiles_done + i, st = tile % Cfg::SCALES;
        KvTreeBits seen{};
        if (TREE && (token < v.all_lo || token + kKvManyTile > v.all_hi))
          seen = kv_tree_bits(nodes, a.tree_words, v.rows_q, context, lo, token);
        ok = kv_wait(&sc_full[st], (tile / Cfg::SCALES) & 1, abort_flag, kSiteEpiTmemFull) &&
             kv_wait(&s_full[half], my_tiles & 1, abort_flag, kSiteEpiTmemFull);
        if (!ok) break;
        tc_fence_after();
        const float2* scales = sSC + st * 8;
        const bool edge = token < v.all_lo || token + kKvManyTile > v.all_hi;
        if (edge) {  // what the row does not see becomes -inf in place
#pragma unroll 1
          for (int g = 0; g < 8; ++g) {
            const int t = token + 16 * g;
            const uint32_t bits = static_cast<uint32_t>((g < 4 ? seen.b[0] : seen.b[1]) >> (16 * (g & 3))) & 0xFFFFu;
            if (!__any_sync(0xFFFFFFFFu, TREE ? bits != 0xFFFFu : t < lo || t + 16 > hi)) continue;
            uint32_t x[16];
            tmem_ld_32x32b_x16(tS + 16 * g, x);
            tmem_ld_wait();
            tmem_regs_ready16(x);
            if (TREE) {
#pragma unroll
              for (int j = 0; j < 16; ++j)
                if (!(bits >> j & 1)) x[j] = 0xFF800000u;
            } else {
#pragma unroll
              for (int j = 0; j < 16; ++j)
                if (static_cast<uint32_t>(token + 16 * g + j - lo) >= width) x[j] = 0xFF800000u;
            }
            tmem_st_32x32b_x16(tS + 16 * g, x);
          }
          tmem_st_wait();
        }
        // the row's largest z + log2 sV
        float most = -INFINITY;
#pragma unroll 1
        for (int g2 = 0; g2 < 4; g2 += 2) {
          uint32_t xx[2][32];
          tmem_ld_32x32b_x32(tS + 32 * g2, xx[0]);
          tmem_ld_32x32b_x32(tS + 32 * g2 + 32, xx[1]);
          tmem_ld_wait();
          tmem_regs_ready(xx[0]);
          tmem_regs_ready(xx[1]);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const int g = g2 + kk / 2, k = kk & 1;
            uint32_t (&x)[32] = xx[kk / 2];
            float y0 = __uint_as_float(x[16 * k]), y1 = __uint_as_float(x[16 * k + 1]);
#pragma unroll
            for (int j = 2; j < 16; j += 4) {
              y0 = fmaxf(fmaxf(y0, __uint_as_float(x[16 * k + j])), __uint_as_float(x[16 * k + (j + 1) % 16]));
              if (j + 2 < 16) y1 = fmaxf(fmaxf(y1, __uint_as_float(x[16 * k + j + 2])), __uint_as_float(x[16 * k + j + 3]));
            }
            const float2 sc = scales[2 * g + k];
            most = fmaxf(most, fmaf(fmaxf(y0, y1), row_mul * sc.x, sc.y));
          }
        }
        const bool past = most > m + 8.f;
        if (__any_sync(0xFFFFFFFFu, past)) {
          const float keep = past && m > -INFINITY ? kv_exp2(m - most) : 1.f;  // (at m = -inf O and l are 0, or NaN)
          l *= keep;
          m = past ? most : m;
          if (i > first) {
#pragma unroll 1
            for (int j = 0; j < D / 16; ++j) {
              uint32_t o[16];
              tmem_ld_32x32b_x16(tO + 16 * j, o);
              tmem_ld_wait();
              tmem_regs_ready16(o);
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * keep);
              tmem_st_32x32b_x16(tO + 16 * j, o);
            }
          }
        }
        const float ref = m == -INFINITY ? 0.f : m;
        // the weights, over the scores that were read before them
#pragma unroll 1
        for (int g = 0; g < 4; ++g) {
          uint32_t x[32], packed[16];
          tmem_ld_32x32b_x32(tS + 32 * g, x);
          tmem_ld_wait();
          tmem_regs_ready(x);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float2 sc = scales[2 * g + k];
            const float mul = row_mul * sc.x, add = sc.y - ref;
            const uint64_t mul2 = pack_f32x2(mul, mul), add2 = pack_f32x2(add, add);
            uint64_t sum2[2] = {0, 0};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const uint32_t* y = &x[16 * k + 2 * j];
              float z0, z1;
              unpack_f32x2(kv_fma2(pack_f32x2(__uint_as_float(y[0]), __uint_as_float(y[1])), mul2, add2), z0, z1);
              const float p0 = kv_exp2(z0), p1 = kv_exp2(z1);
              sum2[j & 1] = kv_add2(sum2[j & 1], pack_f32x2(p0, p1));
              packed[8 * k + j] = kv_pack_f16(p0, p1);
            }
            float sum0, sum1;
            unpack_f32x2(kv_add2(sum2[0], sum2[1]), sum0, sum1);
            l = fmaf(sum0 + sum1, kv_exp2(-sc.y), l);
          }
          tmem_st_32x32b_x16(tS + 16 * g, packed);
        }
        tmem_st_wait();
        tc_fence_before();
        if (edge) {  // NaN codes of V in tokens that this row sees
          const uint32_t v_item = 2 * tiles_done + kv_item_v(TREE && single, i, v.count);
          ok = kv_wait(&f_full[v_item % Cfg::F16_SLOTS], (v_item / Cfg::F16_SLOTS) & 1, abort_flag, kSiteEpiTmemFull);
          if (!ok) break;
          if (sNan[st]) {
            const int j0 = max(lo - token, 0), j1 = min((TREE ? v.len : hi) - token, kKvManyTile);
            for (int j = j0; j < j1; ++j) {
              if (TREE && !((j < 64 ? seen.b[0] : seen.b[1]) >> (j & 63) & 1)) continue;
              const volatile uint32_t* note =
                  reinterpret_cast<const volatile uint32_t*>(nan_notes + ((tile & 3) * kKvManyTile + j) * (D / 8));
#pragma unroll
              for (int k = 0; k < D / 32; ++k) nan_d[k] |= note[k];
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[half]);
      }
      if (!ok) break;
      tiles_done += v.count;
      if (!single) ++other_segments;
      // The queries of the next segment, so that its first products run under this one's output.  (This half's
      // products with the present ones have ended: its last scores have come.)
      KvSegment next;
      more = next_segment(next);
      if (more && !single) row_mul = bring(next, 0);
      const bool any = first < v.count;  // whether this half had a tile
      if (any) ok = kv_wait(&o_full[half], segments++ & 1, abort_flag, kSiteEpiTmemFull);
      if (!ok) break;
      tc_fence_after();
      if (single && half == 1) {
        uint32_t told[16];  // (m, l) and the NaN notes, where its scores were
#pragma unroll
        for (int j = 0; j < 16; ++j) told[j] = j >= 2 && j < 2 + D / 32 ? nan_d[j >= 2 && j < 2 + D / 32 ? j - 2 : 0] : 0;
        told[0] = __float_as_uint(m);
        told[1] = __float_as_uint(l);
        tmem_st_32x32b_x16(tS, told);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(join_full);
        if (TREE) {  // while half 0 joins and writes
          ok = kv_wait(turn, joins & 1, abort_flag, kSiteEpiTmemFull);
          if (!ok) break;
          if (more) row_mul = bring(next, 1);
        }
        ok = kv_wait(join_empty, joins++ & 1, abort_flag, kSiteEpiTmemFull);
      } else {
        float f0 = 1.f, f1 = 0.f;  // O = f0 O_half + f1 O_1
        if (single) {
          ok = kv_wait(join_full, joins++ & 1, abort_flag, kSiteEpiTmemFull);
          if (ok && v.count > 1) {
            tc_fence_after();
            uint32_t told[16];
            tmem_ld_32x32b_x16(tmem + 128 + lanes, told);
            tmem_ld_wait();
            tmem_regs_ready16(told);
            const float2 other = make_float2(__uint_as_float(told[0]), __uint_as_float(told[1]));
            const float most = fmaxf(m, other.x), ref = most == -INFINITY ? 0.f : most;
            f0 = kv_exp2(m - ref);
            f1 = kv_exp2(other.x - ref);
            l = l * f0 + other.y * f1;
            m = most;
#pragma unroll
            for (int j = 0; j < D / 32; ++j) nan_d[j] |= told[2 + j];
            tc_fence_before();
          }
          if (TREE) {  // half 1 may bring the next queries: the last scores with these have come, and it is read what it told
            __syncwarp();
            if (lane == 0) mbar_arrive(turn);
          }
        }
        if (!ok) break;
        const bool two = single && v.count > 1;
        const bool whole = v.part == 0;
        const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
        f0 *= inv;
        f1 *= inv;
        const int64_t at_row = static_cast<int64_t>(v.q0 + qi) * a.heads + v.head * group + hg;
        float* part = reinterpret_cast<float*>(workspace + kv_many_slots_at(a.requests, D) + (2 * blockIdx.x + max(v.part - 1, 0)) * Cfg::SLOT);
        if (two) {
          ok = kv_wait(&o_full[1], (other_segments++) & 1, abort_flag, kSiteEpiTmemFull);
          if (!ok) break;
          tc_fence_after();
        }
#pragma unroll 1
        for (int j = 0; j < D / 16; ++j) {
          uint32_t o[16];
          float f[16];
          tmem_ld_32x32b_x16(tO + 16 * j, o);
          tmem_ld_wait();
          tmem_regs_ready16(o);
#pragma unroll
          for (int k = 0; k < 16; ++k) f[k] = __uint_as_float(o[k]) * f0;
          if (two) {
            tmem_ld_32x32b_x16(tO + 128 + 16 * j, o);
            tmem_ld_wait();
            tmem_regs_ready16(o);
#pragma unroll
            for (int k = 0; k < 16; ++k) f[k] = fmaf(__uint_as_float(o[k]), f1, f[k]);
          }
          const uint32_t nan = nan_d[0] & 0xFFFFu;  // (the notes move along)
#pragma unroll
          for (int k = 0; k < D / 32; ++k) nan_d[k] = (nan_d[k] >> 16) | (k + 1 < D / 32 ? nan_d[k + 1 < D / 32 ? k + 1 : k] << 16 : 0);
#pragma unroll
          for (int k = 0; k < 16; ++k) f[k] = nan >> k & 1 ? NAN : l == 0.f ? 0.f : f[k];
          if (live && whole) {
            uint32_t h[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) h[k] = F16 ? kv_pack_f16(f[2 * k], f[2 * k + 1]) : kv_pack_bf16(f[2 * k], f[2 * k + 1]);
            kv_store32(a.out + at_row * D + 16 * j, h);
          } else if (live) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              uint32_t h[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) h[i] = __float_as_uint(f[8 * k + i]);
              kv_store32(part + my_row * D + 16 * j + 8 * k, h);
            }
          }
        }
        if (live && whole) a.lse[at_row] = l == 0.f ? -INFINITY : ((m == -INFINITY ? 0.f : m) + log2f(l)) * kLn2;
        else if (live) *reinterpret_cast<float2*>(part + kKvManyRows * D + 2 * my_row) = make_float2(m, l);
        tc_fence_before();
        if (single) {
          __syncwarp();
          if (lane == 0) mbar_arrive(join_empty);
        }
      }
      if (!ok) break;
      if (more && single && !(TREE && half == 1)) row_mul = bring(next, TREE ? 1 : 0);
      v = next;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 13) tmem_dealloc(tmem, 512);
}

// Joins the segments of the units that range boundaries cut.  CTA c looks at the boundary where range c
// begins; the first boundary inside a unit takes the unit.  Segments are added in order: the range that
// the unit begins in left its one in slot 1, the others in slot 0.
template <int D>
__global__ void __launch_bounds__(128) kv_join_kernel(const KvAttnArgs a, const uint8_t* workspace, size_t slots_at) {
  pdl_prologue();
  constexpr size_t kSlot = static_cast<size_t>(kKvManyRows) * (D + 2) * 4;
  __shared__ int list[kKvMaxCtas];
  __shared__ int listed;
  const KvJob* jobs = reinterpret_cast<const KvJob*>(workspace + kKvJobsAt);
  const int c = blockIdx.x + 1, ranges = gridDim.x + 1;
  const KvJob job = jobs[c];
  const long long before = jobs[c - 1].begin, total = jobs[ranges - 1].end;
  if (job.begin >= total || job.unit == job.begin || before > job.unit) return;
  const long long unit_end = job.unit + job.tiles + kKvUnitCost;
  if (threadIdx.x < 32) {
    int n = 0;
    for (int k0 = c - 1; k0 < ranges; k0 += 32) {
      const int k = k0 + threadIdx.x;
      bool has = false, over = true;
      if (k < ranges) {
        const long long b = jobs[k].begin, e = jobs[k].end;
        over = b >= unit_end;
        const int from = kv_tiles_before(b - job.unit, job.tiles), to = kv_tiles_before(e - job.unit, job.tiles);
        has = !over && to > from && to - from < job.tiles;  // (a range that has all of it has finished it)
      }
      const uint32_t m = __ballot_sync(0xFFFFFFFFu, has);
      if (has) list[n + __popc(m & ((1u << threadIdx.x) - 1))] = 2 * k + (k == c - 1 ? 1 : 0);
      n += __popc(m);
      if (__any_sync(0xFFFFFFFFu, over)) break;
    }
    if (threadIdx.x == 0) listed = n;
  }
  __syncthreads();
  const int n = listed;
  if (n == 0) return;
  const int group = a.heads / a.kv_heads;
  for (int i = blockIdx.y * 128 + threadIdx.x; i < job.rows * (D / 4); i += 128 * gridDim.y) {
    const int row = i / (D / 4), d = i % (D / 4) * 4;
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < n; ++k) {
      const float* part = reinterpret_cast<const float*>(workspace + slots_at + list[k] * kSlot);
      const float2 ml = *reinterpret_cast<const float2*>(part + kKvManyRows * D + 2 * row);
      const float4 x = *reinterpret_cast<const float4*>(part + row * D + d);
      kv_join(m, l, o, ml, x);
    }
    kv_finish<D>(a, job.q0, job.row0 + row, group, job.head, d, m, l, o);
  }
}

}  // namespace mxgb
