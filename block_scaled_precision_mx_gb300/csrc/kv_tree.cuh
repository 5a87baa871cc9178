// kv_tree.cuh -- attention of a tree's queries over the paged 8-bit cache, for more than 16 rows a kv head.
//
// Units, ranges, parts and roles are those of the kernel for prompts (kv_prefill.cuh).  Trees differ in that all rows of
// a unit see nearly all of its tokens and that there are few units' rows for many tokens, so that a tile's way through the
// CTA is what counts, and not the products.  What is done about it:
//
//  * Scores come in pieces of 64 tokens, two buffers of them for each row half: the products of the next piece are there
//    when a half has finished its softmax, so that it does not wait for P V and the next S in turn.  A piece's
//    scores stay in registers from their maximum to their weights.
//  * Units of at most 128 rows: both halves work on the same rows, on the two pieces of each tile, with an O each; S
//    is one product for both.  (On alternate tiles, as prompts have it, a tile's S waits for the P V of the one before.)
//  * The loading warp has the next 32 blocks of the table, and their scales, in hand before it needs them, and brings
//    their codes from memory to L2 some tiles ahead: what is in flight then is not bound by shared memory, where the
//    codes take up 32 KB (D = 128), and a load of them takes an L2's latency.
//  * Four buffers of FP16 codes: with three, a tile's K waits for the P V of the one before.
#pragma once

#include "kv_prefill.cuh"

namespace mxgb {

constexpr int kKvTreeSegments = 3;

template <int D>
struct KvTreeCfg {
  static constexpr int RAW_SLOTS = D == 128 ? 4 : 12, F16_SLOTS = 4;
  // Tiles whose scales are kept.  A tile's are written when its codes have a place, so that the codes R = RAW_SLOTS / 4
  // tiles before it have been converted, the K two tiles before those is done with, and the softmax two before that.
  static constexpr int SCALES = D == 128 ? 6 : 8;
  static_assert(SCALES >= RAW_SLOTS / 4 + 4, "a tile's scales are read until its softmax has ended");
  static constexpr int RAW = 64 * D;                   // codes of K or V of half a tile
  static constexpr int WIDE = 2 * kKvManyTile * D;     // a tile's K or V in FP16; also 128 rows of Q
  static constexpr int OFF_F16 = 2 * WIDE;
  static constexpr int OFF_RAW = OFF_F16 + F16_SLOTS * WIDE;
  static constexpr int OFF_SC = OFF_RAW + RAW_SLOTS * RAW;            // float2 [tiles][8 slices]: sK, log2 sV
  static constexpr int OFF_MUL = OFF_SC + SCALES * 8 * 8;      // float [128], for units of one row half
  static constexpr int OFF_NAN = OFF_MUL + 4 * 128;               // int [tiles]
  static constexpr int OFF_BAR = OFF_NAN + 4 * SCALES;
  static constexpr int BARS = 2 * RAW_SLOTS + 2 * F16_SLOTS + 2 + 4 + 4 + 4 + SCALES + 2 * kKvTreeSegments + 3;
  static constexpr int OFF_SEG = (OFF_BAR + 8 * BARS + 15) / 16 * 16;  // KvSegment [segments]
  static constexpr int SMEM = OFF_SEG + 64 * kKvTreeSegments + 16 + 1024;
  static constexpr int AHEAD = 512 / D;                               // tiles that L2 is told of ahead
  static constexpr size_t SLOT = KvManyCfg<D>::SLOT, NAN_BYTES = KvManyCfg<D>::NAN_BYTES;
};
static_assert(KvTreeCfg<128>::SMEM <= 232448 && KvTreeCfg<64>::SMEM <= 232448, "a CTA's shared memory");
static_assert(KvTreeCfg<128>::OFF_BAR % 8 == 0 && KvTreeCfg<64>::OFF_BAR % 8 == 0, "barriers");

__device__ __forceinline__ void kv_prefetch_2d(const CUtensorMap* map, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(map), "r"(x), "r"(y) : "memory");
}

// Which of the 16 tokens from t on a row of a tree sees, as bits: `nodes` is its row of the mask (null: none of the nodes),
// first the first token that it sees of those in front of the nodes, n how many nodes there are.
__device__ __forceinline__ uint32_t kv_tree_sees16(const uint64_t* nodes, int words, int n, int context, int first, int t) {
  const int o = t - context;
  uint32_t b = 0xFFFFu;
  if (o > -16) {
    const int w = o >> 6, sh = o & 63;  // (w = -1: what is in front of the nodes)
    const uint64_t at = w < 0 ? ~0ull : nodes && w < words ? nodes[w] : 0;
    const uint64_t behind = sh > 48 && nodes && w + 1 < words ? nodes[w + 1] : 0;
    b &= static_cast<uint32_t>(at >> sh) | (sh > 48 ? static_cast<uint32_t>(behind << (64 - sh)) : 0);
    if (n - o < 16) b &= (1u << max(n - o, 0)) - 1;
  }
  if (first > t) b &= ~0u << min(first - t, 16);
  return b;
}

// Where piece g of half h has its scores, and then its weights, in tensor memory.
__device__ __forceinline__ uint32_t kv_tree_scores(bool single, uint32_t h, uint32_t g) {
  return single ? (g & 1) * 128 + h * 64 : h * 128 + (g & 1) * 64;
}

template <int FMT, int D, bool F16>
__global__ void __launch_bounds__(kKvManyThreads, 1)
    kv_tree_many_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                        const KvAttnArgs a, int most_q, int planned, uint8_t* workspace) {
  using Cfg = KvTreeCfg<D>;
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
  uint64_t* q_full = f_empty + Cfg::F16_SLOTS;  // [2]
  uint64_t* s_full = q_full + 2;                // [2 halves][2 buffers]
  uint64_t* p_full = s_full + 4;                // [2][2]
  // [2][2]; as p_full: a wait tells a phase from the one before it, not from two before, and the scores of a piece say
  // only that the products two pieces back, in the same buffer, have ended
  uint64_t* pv_done = p_full + 4;
  uint64_t* sc_full = pv_done + 4;              // [Cfg::SCALES]
  uint64_t* seg_full = sc_full + Cfg::SCALES; // [kKvTreeSegments]
  uint64_t* seg_empty = seg_full + kKvTreeSegments;
  uint64_t* join_full = seg_empty + kKvTreeSegments;
  uint64_t* join_empty = join_full + 1;
  uint64_t* drain_bar = join_empty + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::OFF_SEG + 64 * kKvTreeSegments);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  // (where the range is planned, in front of the loads)
  KvJob& job = *reinterpret_cast<KvJob*>(smem + Cfg::OFF_F16);
  long long* warp_sum = reinterpret_cast<long long*>(smem + Cfg::OFF_F16 + 256);
  const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;
  const int group = a.heads / a.kv_heads;
  if (tid == 0) {
    for (int i = 0; i < Cfg::RAW_SLOTS; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], 4);
    }
    for (int i = 0; i < Cfg::F16_SLOTS; ++i) {
      mbar_init(&f_full[i], 4);
      mbar_init(&f_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) mbar_init(&q_full[i], 4);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&pv_done[i], 1);
    }
    for (int i = 0; i < Cfg::SCALES; ++i) mbar_init(&sc_full[i], 1);
    for (int i = 0; i < kKvTreeSegments; ++i) {
      mbar_init(&seg_full[i], 1);
      mbar_init(&seg_empty[i], 13);  // warps 0-11 and 13
    }
    mbar_init(join_full, 4);
    mbar_init(join_empty, 4);
    mbar_init(drain_bar, 1);
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
  if (planned) {
    if (tid == 0) job = reinterpret_cast<const KvJob*>(workspace + kKvJobsAt)[blockIdx.x];
  } else {
    // Few requests of few units: every CTA finds its own range, a request a thread (a launch of kv_plan_kernel less).
    KvRequest req{};
    long long mine = 0;
    if (tid < a.requests) {
      req = kv_request<true>(a, tid, most_q, blockIdx.x == 0);
      const int units = kv_units_of(req, group);
#pragma unroll 1
      for (int i = 0; i < units; ++i) mine += kv_unit<true>(a, req, group, i).cost();
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
    if (here) kv_first_unit<true>(a, req, tid, group, before, mine_job);
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
    const uint32_t i = seg % kKvTreeSegments;
    const bool ok = kv_wait(&seg_full[i], (seg / kKvTreeSegments) & 1, abort_flag, kSiteMmaFull);
    v = sSeg[i];
    __syncwarp();
    if (lane == 0) mbar_arrive(&seg_empty[i]);
    ++seg;
    return ok && v.count > 0;
  };

  if (warp == 12) {
    // ------------------------------------------------------------------ loads: item 2i = K, 2i + 1 = V of tile i, in halves
    // A chunk is up to 32 blocks of a segment: lane i holds block i and its scales, read while the chunk before it is loaded.
    struct Chunk {
      int token, tiles, h, block, take;
      float sk, sv;
      bool odd;  // some block's codes are not taken as they are
    };
    KvManyWalk w;
    kv_many_begin<true>(a, most_q, group, job, w);
    const long long range_start = w.pos;
    const int P = 1 << a.shift, rows_box = min(P, kKvTile), boxes = kKvTile / rows_box;
    const int most_tiles = 32 * P / kKvManyTile;
    int left = 0;
    bool ok = true;
    auto row_of = [&](int block, int h) { return (block * a.kv_heads + h) << a.shift; };
    auto prefetch = [&](const Chunk& ch, int from, int to) {  // codes of the chunk's tiles [from, to), to L2
      const int tile = (lane << a.shift) / kKvManyTile;
      if (tile >= from && tile < min(to, ch.tiles) && ch.block >= 0)
        for (int row = 0; row < P; row += rows_box) {
          kv_prefetch_2d(&tmK, 0, row_of(ch.block, ch.h) + row);
          kv_prefetch_2d(&tmV, 0, row_of(ch.block, ch.h) + row);
        }
    };
    auto fetch = [&](Chunk& ch) {
      ch.tiles = 0;
      if (!left) {
        const bool more = kv_many_next<true>(a, most_q, group, w);
        const uint32_t sl = seg % kKvTreeSegments;
        if (!kv_wait(&seg_empty[sl], ((seg / kKvTreeSegments) & 1) ^ 1, abort_flag, kSiteProducerEmpty)) {
          ok = false;
          return;
        }
        if (lane == 0) {
          const int part = w.count == w.u.tiles ? 0 : w.base < range_start ? 1 : 2;
          sSeg[sl] = KvSegment{more ? w.count : 0, (w.u.first_tile + w.tile) * kKvManyTile, w.u.rows, w.u.row0, w.u.q0,
                               w.u.rows_q, w.u.len, w.u.any_lo, w.u.all_lo, w.u.all_hi, w.h, part};
          mbar_arrive(&seg_full[sl]);
        }
        ++seg;
        if (!more) return;
        left = w.count;
      }
      ch.tiles = min(most_tiles, left);
      ch.token = (w.u.first_tile + w.tile + w.count - left) * kKvManyTile;
      ch.h = w.h;
      left -= ch.tiles;
      const int page = (ch.token >> a.shift) + lane;
      ch.block = -1;
      ch.sk = ch.sv = 1.f;
      const bool told = page << a.shift < w.u.any_hi;
      if (page << a.shift < w.u.len && (page + 1) << a.shift > w.u.any_lo)  // (in front of any_lo no row sees it)
        kv_look_up(a, w.r, page, w.h, ch.block, ch.sk, ch.sv);
      prefetch(ch, 0, Cfg::AHEAD);
      ch.take = kv_check_scales(ch.sk, ch.sv, told);
      ch.odd = __any_sync(0xFFFFFFFFu, ch.take != 0);
    };
    uint32_t tiles_done = 0, issued = 0;
    Chunk cur, next;
    fetch(cur);
    while (ok && cur.tiles) {
      for (int i = 0; i < cur.tiles && ok; ++i, ++tiles_done) {
        const int token = cur.token + i * kKvManyTile, first = token - cur.token;
        prefetch(cur, i + Cfg::AHEAD, i + Cfg::AHEAD + 1);
        const int slice = (first + (lane & 7) * 16) >> a.shift;
        const float slice_k = __shfl_sync(0xFFFFFFFFu, cur.sk, slice), slice_v = __shfl_sync(0xFFFFFFFFu, cur.sv, slice);
#pragma unroll 1
        for (int part = 0; part < 4; ++part) {  // K's halves, V's halves
          const uint32_t item = 4 * tiles_done + part, slot = item % Cfg::RAW_SLOTS;
          const int my = first + 64 * (part & 1) + lane * rows_box, box_at = min(my >> a.shift, 31);
          const int box_block = __shfl_sync(0xFFFFFFFFu, cur.block, box_at);
          const int box_take = cur.odd ? __shfl_sync(0xFFFFFFFFu, cur.take, box_at) : 0;
          if (!kv_wait(&raw_empty[slot], ((item / Cfg::RAW_SLOTS) & 1) ^ 1, abort_flag, kSiteProducerEmpty)) {
            ok = false;
            break;
          }
          uint8_t* dst = smem + Cfg::OFF_RAW + slot * Cfg::RAW + lane * rows_box * D;
          const int taken = part >> 1 ? box_take >> 8 : box_take & 0xFF;
          const bool load = lane < boxes && box_block >= 0 && !taken;
          const uint32_t bytes = __popc(__ballot_sync(0xFFFFFFFFu, load)) * rows_box * D;
          if (cur.odd) {
            if (lane < boxes && taken) kv_fill_box(dst, rows_box * D, kv_four_taken(taken));
            __syncwarp();
          }
          ++issued;
          if (lane == 0) mbar_arrive_expect_tx(&raw_full[slot], bytes);
          __syncwarp();
          if (load)
            tma_load_2d(dst, part >> 1 ? &tmV : &tmK, &raw_full[slot], 0, row_of(box_block, cur.h) + (my & (P - 1)));
          if (part == 0) {
            const uint32_t st = tiles_done % Cfg::SCALES;
            if (lane < 8) sSC[st * 8 + lane] = make_float2(slice_k, log2f(slice_v));
            if (lane == 0) sNan[st] = 0;
            __syncwarp();
            if (lane == 0) mbar_arrive(&sc_full[st]);
          }
        }
        if (i == 0 && ok) fetch(next);
      }
      cur = next;
    }
    // every copy has landed before the CTA's shared memory goes
    for (uint32_t i = 0; i < Cfg::RAW_SLOTS; ++i)
      if (issued > i) mbar_drain(&raw_full[i], kv_ring_last_parity(issued, i, Cfg::RAW_SLOTS), kWaitBudgetNs);
  } else if (warp == 13) {
    // ------------------------------------------------------------------ products (the whole warp keeps step, one thread issues)
    constexpr uint32_t kHi = smem_desc_hi(1024, kSwizzle128B);
    constexpr uint32_t kLoK = smem_desc_lo_lbo(16), kLoN = smem_desc_lo_lbo(kKvManyTile * 128);
    constexpr uint32_t kIdS1 = kv_idesc_f16(128, 128, false), kIdS2 = kv_idesc_f16(128, 64, false), kIdO = kv_idesc_f16(128, D, true);
    const uint32_t q_lo = (smem_u32(smem) >> 4) | kLoK, f_lo = smem_u32(smem + Cfg::OFF_F16) >> 4;
    uint32_t tiles_done = 0, done = 0, segments[2] = {0, 0};  // done: pieces of each half in the segments before
    bool ok = true, single = false;
    int pieces = 0;
    KvSegment v;
    // S of piece j: of half h, or of both where a unit has one row half
    auto scores = [&](int h, int j) {
      if (j >= pieces) return;
      const uint32_t item = 2 * (tiles_done + (single ? j : j >> 1)), slot = item % Cfg::F16_SLOTS;
      ok = kv_wait(&f_full[slot], (item / Cfg::F16_SLOTS) & 1, abort_flag, kSiteMmaFull);
      if (ok && j == 0) ok = kv_wait(&q_full[h], segments[h]++ & 1, abort_flag, kSiteMmaFull);
      if (!ok) return;
      tc_fence_after();
      const int piece = single ? 0 : j & 1;
      const uint32_t k_lo = __shfl_sync(0xFFFFFFFFu, ((f_lo + slot * (Cfg::WIDE / 16)) | kLoK) + piece * (64 * 128 / 16), 0);
      const uint32_t qh_lo = q_lo + h * (Cfg::WIDE / 16), to = tmem + kv_tree_scores(single, h, done + j);
      const uint32_t id = single ? kIdS1 : kIdS2;
      if (kv_elect()) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t at = (k / 4) * (kKvManyTile * 128 / 16) + (k % 4) * 2;
          umma_f16_ss(to, desc_from_words(qh_lo + at, kHi), desc_from_words(k_lo + at, kHi), id, k > 0);
        }
        umma_commit(&s_full[2 * h + ((done + j) & 1)]);
        if (single) umma_commit(&s_full[2 + ((done + j) & 1)]);
        if (single || (h == 1 && piece == 1)) umma_commit(&f_empty[slot]);
      }
      __syncwarp();
    };
    auto output = [&](int h, int j) {  // O_h += P_h V of piece j
      const uint32_t g = done + j, item = 2 * (tiles_done + (single ? j : j >> 1)) + 1, slot = item % Cfg::F16_SLOTS;
      ok = kv_wait(&f_full[slot], (item / Cfg::F16_SLOTS) & 1, abort_flag, kSiteMmaFull) &&
           kv_wait(&p_full[2 * h + (g & 1)], (g >> 1) & 1, abort_flag, kSiteMmaTmemEmpty);
      if (!ok) return;
      tc_fence_after();
      const int piece = single ? h : j & 1;
      const uint32_t v_lo = __shfl_sync(0xFFFFFFFFu, ((f_lo + slot * (Cfg::WIDE / 16)) | kLoN) + piece * (64 * 128 / 16), 0);
      const uint32_t from = tmem + kv_tree_scores(single, h, g);
      if (kv_elect()) {
#pragma unroll
        for (int k = 0; k < 4; ++k)  // 16 tokens at a time
          umma_f16_ts(tmem + 256 + h * 128, from + k * 8, desc_from_words(v_lo + k * (16 * 128 / 16), kHi), kIdO, j > 0 || k > 0);
        umma_commit(&pv_done[2 * h + (g & 1)]);
        if (h == 1 && (single || piece == 1)) umma_commit(&f_empty[slot]);
      }
      __syncwarp();
    };
    while (ok && next_segment(v)) {
      const int count = __shfl_sync(0xFFFFFFFFu, v.count, 0);
      single = v.rows <= 128;
      pieces = single ? count : 2 * count;
      for (int j = 0; j < 2 && ok; ++j) {
        scores(0, j);
        if (!single && ok) scores(1, j);
      }
      for (int j = 0; j < pieces && ok; ++j) {
        output(0, j);
        if (!single && ok) scores(0, j + 2);
        if (ok) output(1, j);
        if (ok) scores(single ? 0 : 1, j + 2);
      }
      tiles_done += count;
      done += pieces;
    }
    // every product has ended before the tensor memory goes
    if (kv_elect()) {
      umma_commit(drain_bar);
      mbar_drain(drain_bar, 0, kWaitBudgetNs);
    }
    __syncwarp();
  } else if (warp >= 8 && warp < 12) {
    // ------------------------------------------------------------------ codes -> FP16
    constexpr int CH = D / 16;      // 16-code words of a token
    constexpr int WORDS = CH / 2;   // words of half a tile that a lane takes
    const int wq = warp - 8, tl = lane & 7;
    uint32_t tiles_done = 0;
    bool ok = true;
    KvSegment v;
    while (ok && next_segment(v)) {
      const uint32_t parts = 4 * (tiles_done + v.count);
#pragma unroll 1
      for (uint32_t part = 4 * tiles_done; part < parts; ++part) {
        const uint32_t slot = part % Cfg::RAW_SLOTS, item = part >> 1, fs = item % Cfg::F16_SLOTS;
        ok = kv_wait(&raw_full[slot], (part / Cfg::RAW_SLOTS) & 1, abort_flag, kSiteMmaFull) &&
             ((part & 1) || kv_wait(&f_empty[fs], ((item / Cfg::F16_SLOTS) & 1) ^ 1, abort_flag, kSiteProducerEmpty));
        if (!ok) break;
        uint8_t* src = smem + Cfg::OFF_RAW + slot * Cfg::RAW;
        uint8_t* dst = smem + Cfg::OFF_F16 + fs * Cfg::WIDE + (part & 1) * (64 * 128);
        // lane: row tl of 8, word lane / 8 of 4; D = 128 has two groups of 4 words
        auto raw_at = [&](int n, int& row, int& word) {
          row = 16 * wq + 8 * (n / (CH / 4)) + tl;
          word = (n % (CH / 4)) * 4 + (lane >> 3);
          return reinterpret_cast<uint4*>(src + (D == 128 ? row * 128 + ((word ^ (row & 7)) << 4)
                                                          : row * 64 + ((word ^ ((row >> 1) & 3)) << 4)));
        };
        const int token = v.token + static_cast<int>(item / 2 - tiles_done) * kKvManyTile;
        if ((item & 1) && (token < v.all_lo || token + kKvManyTile > v.all_hi)) {
          // V of a tile that some row does not see whole: clear what no row sees; take NaN codes out and note them
          uint32_t any = 0;
          const int row0 = 64 * static_cast<int>(part & 1);
#pragma unroll 1
          for (int n = 0; n < WORDS; ++n) {
            int row, word;
            uint4* at = raw_at(n, row, word);
            const uint4 x = *at;
            const bool out = token + row0 + row < v.any_lo || token + row0 + row >= v.len;
            uint32_t c[4] = {x.x, x.y, x.z, x.w}, bits = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (out) c[j] = 0;
              const uint32_t y = kv_nan_bytes<FMT>(c[j]);
              c[j] &= ~((y >> 7) * 0xFFu);
              bits |= ((y >> 7 & 1) | (y >> 14 & 2) | (y >> 21 & 4) | (y >> 28 & 8)) << (4 * j);
            }
            *at = make_uint4(c[0], c[1], c[2], c[3]);
            reinterpret_cast<uint16_t*>(nan_notes)[((item / 2 & 3) * kKvManyTile + row0 + row) * CH + word] = static_cast<uint16_t>(bits);
            any |= bits;
          }
          if (any) sNan[item / 2 % Cfg::SCALES] = 1;
          __threadfence_block();
        }
        uint4 x[WORDS];
        int row[WORDS], word[WORDS];
#pragma unroll
        for (int n = 0; n < WORDS; ++n) x[n] = *raw_at(n, row[n], word[n]);
#pragma unroll
        for (int n = 0; n < WORDS; ++n) {
          const uint32_t c[4] = {x[n].x, x[n].y, x[n].z, x[n].w};
          uint32_t f[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) kv_codes4_to_f16<FMT>(c[j], f[2 * j], f[2 * j + 1]);
          uint8_t* to = dst + (word[n] >> 2) * (kKvManyTile * 128) + row[n] * 128;
          const int ch = (word[n] & 3) * 2;
          *reinterpret_cast<uint4*>(to + ((ch ^ (row[n] & 7)) << 4)) = make_uint4(f[0], f[1], f[2], f[3]);
          *reinterpret_cast<uint4*>(to + (((ch + 1) ^ (row[n] & 7)) << 4)) = make_uint4(f[4], f[5], f[6], f[7]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&raw_empty[slot]);
          if (part & 1) mbar_arrive(&f_full[fs]);
        }
      }
      tiles_done += v.count;
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------------ softmax, a row a thread
    const int half = warp >> 2, row = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tO = tmem + 256 + half * 128 + lanes;
    uint8_t* sQ = smem + half * Cfg::WIDE;
    float2* join_ml = reinterpret_cast<float2*>(smem + Cfg::WIDE);          // one row half: half 1's (m, l) and NaN notes
    uint32_t* join_nan = reinterpret_cast<uint32_t*>(smem + Cfg::WIDE + 1024);  // (where its queries would be)
    uint32_t tiles_done = 0, g = 0, joins = 0;  // g: pieces that this half has done
    bool ok = true;
    // A segment's queries as FP16; returns what this thread's row of scores is to be multiplied with.  The rows
    // are copied to their places as they are, D / 8 lanes a row, and converted there, a row a thread.  (Short
    // loops: code that runs once a segment is not in the instruction cache, and costs by its length.)
    auto bring = [&](const KvSegment& v) {
      constexpr int LANES = D / 8, AT_ONCE = 32 / LANES;
      const bool single = v.rows <= 128;
      if (single && half == 1) {  // half 0 brings the rows of both
        ok = kv_wait(&q_full[0], (seg - 1) & 1, abort_flag, kSiteEpiTmemFull);
        return sMul[row];
      }
      const int word = lane % LANES, sub = lane / LANES, row0 = 32 * (warp & 3);
      int r = row0 + sub, qi = (v.row0 + half * 128 + r) / group, hg = v.row0 + half * 128 + r - qi * group;
      const int qi_step = AT_ONCE / group, hg_step = AT_ONCE % group;
      const uint32_t to = smem_u32(sQ) + (word >> 3) * (128 * 128);
#pragma unroll 1
      for (; r < row0 + 32; r += AT_ONCE) {
        const uint16_t* src = a.q + (v.q0 + qi) * a.stride_t + (v.head * group + hg) * a.stride_h + 8 * word;
        const uint32_t bytes = half * 128 + r < v.rows ? 16 : 0;  // (the rest of the 16 is zeros)
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
      if (lane == 0) mbar_arrive(&q_full[half]);
      return row_mul;
    };
    KvSegment v;
    bool more = next_segment(v);
    float row_mul = more ? bring(v) : 0.f;
    while (ok && more) {
      const bool single = v.rows <= 128;  // both halves work on the same rows, on a piece each of every tile
      const int my_row = single ? row : 128 * half + row;
      const bool live = my_row < v.rows;
      const int qi = (v.row0 + my_row) / group, hg = v.row0 + my_row - qi * group;
      const int context = v.len - v.rows_q;
      const uint64_t* nodes = live ? a.tree_mask + static_cast<int64_t>(v.q0 + qi) * a.tree_words : nullptr;
      const int lo = live ? kv_tree_first(a, v.q0 + qi, context, v.rows_q) : 0;
      const int pieces = single ? v.count : 2 * v.count;
      float m = -INFINITY, l = 0.f;
      uint32_t nan_d[D / 32];
#pragma unroll
      for (int i = 0; i < D / 32; ++i) nan_d[i] = 0;
#pragma unroll 1
      for (int i = 0; i < pieces; ++i, ++g) {
        const int piece = single ? half : i & 1, nth = single ? i : i >> 1;
        const int tile_token = v.token + nth * kKvManyTile, token = tile_token + 64 * piece;
        const uint32_t tile = tiles_done + nth, st = tile % Cfg::SCALES;
        const uint32_t tS = tmem + lanes + kv_tree_scores(single, half, g);
        ok = kv_wait(&sc_full[st], (tile / Cfg::SCALES) & 1, abort_flag, kSiteEpiTmemFull) &&
             kv_wait(&s_full[2 * half + (g & 1)], (g >> 1) & 1, abort_flag, kSiteEpiTmemFull);
        if (!ok) break;
        tc_fence_after();
        uint32_t x[2][32];
        tmem_ld_32x32b_x32(tS, x[0]);
        tmem_ld_32x32b_x32(tS + 32, x[1]);
        const float2* scales = sSC + st * 8 + 4 * piece;
        const bool edge = tile_token < v.all_lo || tile_token + kKvManyTile > v.all_hi;
        tmem_ld_wait();
        tmem_regs_ready(x[0]);
        tmem_regs_ready(x[1]);
        if (edge) {  // what the row does not see becomes -inf
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t seen = kv_tree_sees16(nodes, a.tree_words, v.rows_q, context, lo, token + 16 * k);
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (!(seen >> j & 1)) x[k >> 1][16 * (k & 1) + j] = 0xFF800000u;
          }
        }
        // the row's largest z + log2 sV
        float most = -INFINITY;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t* y = &x[k >> 1][16 * (k & 1)];
          float y0 = __uint_as_float(y[0]), y1 = __uint_as_float(y[1]);
#pragma unroll
          for (int j = 2; j < 16; j += 4) {
            y0 = fmaxf(fmaxf(y0, __uint_as_float(y[j])), __uint_as_float(y[(j + 1) % 16]));
            if (j + 2 < 16) y1 = fmaxf(fmaxf(y1, __uint_as_float(y[j + 2])), __uint_as_float(y[j + 3]));
          }
          const float2 sc = scales[k];
          most = fmaxf(most, fmaf(fmaxf(y0, y1), row_mul * sc.x, sc.y));
        }
        const bool past = most > m + 8.f;
        if (__any_sync(0xFFFFFFFFu, past)) {
          const float keep = past && m > -INFINITY ? kv_exp2(m - most) : 1.f;  // (at m = -inf O and l are 0, or NaN)
          l *= keep;
          m = past ? most : m;
          if (i > 0) {  // (behind the product that is under way)
            ok = kv_wait(&pv_done[2 * half + ((g - 1) & 1)], ((g - 1) >> 1) & 1, abort_flag, kSiteEpiTmemFull);
            if (!ok) break;
            tc_fence_after();
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
        // the weights, over the scores
#pragma unroll
        for (int k2 = 0; k2 < 2; ++k2) {
          uint32_t packed[16];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float2 sc = scales[2 * k2 + k];
            const float mul = row_mul * sc.x, add = sc.y - ref;
            const uint64_t mul2 = pack_f32x2(mul, mul), add2 = pack_f32x2(add, add);
            uint64_t sum2[2] = {0, 0};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const uint32_t* y = &x[k2][16 * k + 2 * j];
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
          tmem_st_32x32b_x16(tS + 16 * k2, packed);
        }
        tmem_st_wait();
        tc_fence_before();
        if (edge) {  // NaN codes of V in tokens that this row sees
          const uint32_t v_item = 2 * tile + 1;
          ok = kv_wait(&f_full[v_item % Cfg::F16_SLOTS], (v_item / Cfg::F16_SLOTS) & 1, abort_flag, kSiteEpiTmemFull);
          if (!ok) break;
          if (sNan[st]) {
            for (int j = max(lo - token, 0); j < min(v.len - token, 64); ++j) {
              if (!(kv_tree_sees16(nodes, a.tree_words, v.rows_q, context, lo, token + j) & 1)) continue;
              const volatile uint32_t* note =
                  reinterpret_cast<const volatile uint32_t*>(nan_notes + ((tile & 3) * kKvManyTile + 64 * piece + j) * (D / 8));
#pragma unroll
              for (int k = 0; k < D / 32; ++k) nan_d[k] |= note[k];
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[2 * half + (g & 1)]);
      }
      if (!ok) break;
      tiles_done += v.count;
      KvSegment next;
      more = next_segment(next);
      float f0 = 1.f, f1 = 0.f;  // O = f0 O_half + f1 O_1
      ok = kv_wait(&pv_done[2 * half + ((g - 1) & 1)], ((g - 1) >> 1) & 1, abort_flag, kSiteEpiTmemFull);
      if (!ok) break;
      tc_fence_after();
      if (single && half == 1) {
        join_ml[row] = make_float2(m, l);
#pragma unroll
        for (int j = 0; j < D / 32; ++j) join_nan[row * (D / 32) + j] = nan_d[j];
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(join_full);
        ok = kv_wait(join_empty, joins++ & 1, abort_flag, kSiteEpiTmemFull);
      } else if (single) {
        ok = kv_wait(join_full, joins++ & 1, abort_flag, kSiteEpiTmemFull) &&
             kv_wait(&pv_done[2 + ((g - 1) & 1)], ((g - 1) >> 1) & 1, abort_flag, kSiteEpiTmemFull);
        tc_fence_after();
        const float2 other = join_ml[row];
        const float most = fmaxf(m, other.x), ref = most == -INFINITY ? 0.f : most;
        f0 = kv_exp2(m - ref);
        f1 = kv_exp2(other.x - ref);
        l = l * f0 + other.y * f1;
        m = most;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) nan_d[j] |= join_nan[row * (D / 32) + j];
      }
      if (!ok) break;
      // The queries of the next segment, so that its first products run under this one's output.  (The products with the
      // present ones have ended: their last scores have come.  Half 1's place has held what it tells half 0, of one row
      // half; and half 0 brings no further queries before half 1 has come to the end of this segment too.)
      if (more) row_mul = bring(next);
      if (!single || half == 0) {
        const bool whole = v.part == 0;
        const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
        f0 *= inv;
        f1 *= inv;
        const int64_t at_row = static_cast<int64_t>(v.q0 + qi) * a.heads + v.head * group + hg;
        float* part = reinterpret_cast<float*>(workspace + kv_many_slots_at(a.requests, D) + (2 * blockIdx.x + max(v.part - 1, 0)) * Cfg::SLOT);
#pragma unroll 1
        for (int j = 0; j < D / 16; ++j) {
          uint32_t o[16];
          float f[16];
          tmem_ld_32x32b_x16(tO + 16 * j, o);
          tmem_ld_wait();
          tmem_regs_ready16(o);
#pragma unroll
          for (int k = 0; k < 16; ++k) f[k] = __uint_as_float(o[k]) * f0;
          if (single) {
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
      v = next;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 13) tmem_dealloc(tmem, 512);
}

}  // namespace mxgb
