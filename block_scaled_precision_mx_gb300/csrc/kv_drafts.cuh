// kv_drafts.cuh -- trees of drafted tokens beside the 8-bit key/value cache: which nodes a node sees and where it
// stands, which drafts the target model keeps, and the kept ones' codes moved together in the cache.
#pragma once

#include "kv_cache.cuh"

namespace mxgb {

constexpr int kKvMostNodes = 1024;            // nodes of a request's tree
constexpr int kKvMostContext = 1 << 30;       // cached tokens of a request

// A request's rows [q0, q0 + n) of the step's tokens; n = -1 where its starts break their contract.
struct KvRows {
  int q0, n;
};
__device__ __forceinline__ KvRows kv_rows(const int32_t* q_start, int r, int tokens, int most) {
  const int q0 = q_start[r], end = q_start[r + 1];
  // (compared before they are subtracted: differences of any two 32-bit numbers do not fit)
  const bool ok = q0 >= 0 && q0 <= end && end <= tokens && end - q0 <= most;
  return {ok ? q0 : 0, ok ? end - q0 : -1};
}
// the first row that no request has (or `tokens`, where that is not to be had)
__device__ __forceinline__ int kv_rows_end(const int32_t* q_start, int requests, int tokens) {
  const int end = q_start[requests];
  return end >= 0 && end <= tokens ? end : tokens;
}

// ================================================================== trees
struct KvTreesArgs {
  const int32_t* parents;  // [tokens], within a request's rows; -1: none
  const int32_t* lengths;  // [requests], the rows among them
  const int32_t* q_start;  // [requests + 1]
  uint64_t* mask;          // [tokens][words]
  int32_t* positions;      // [tokens]
  int requests, tokens, most, words, window;
};

constexpr int kKvTreesThreads = 128;

// A request a CTA.  Its parents come into shared memory; a node a thread then walks up to its root, sets the
// bits of what it passes and counts its depth.  Parents are smaller than their children, so the words of a node's
// mask are finished one after the other on the way.  Latency is the bound: a launch, two dependent loads, as many
// steps in shared memory as the tree is deep.  64 trees of 32 nodes 2.2 us, 2000 of 100 to 200 8.4 us (12 MB: 1.8 us; words
// of 8 bytes that a thread writes one by one, 32 apart).
__global__ void __launch_bounds__(kKvTreesThreads) kv_draft_trees_kernel(const KvTreesArgs a) {
  pdl_prologue();
  __shared__ int16_t up[kKvMostNodes];
  const int tid = threadIdx.x;
  for (int64_t i = kv_rows_end(a.q_start, a.requests, a.tokens) + static_cast<int64_t>(blockIdx.x) * kKvTreesThreads + tid;
       i < a.tokens; i += static_cast<int64_t>(gridDim.x) * kKvTreesThreads) {
    for (int w = 0; w < a.words; ++w) a.mask[i * a.words + w] = 0;
    a.positions[i] = -1;
  }
  const KvRows rows = kv_rows(a.q_start, blockIdx.x, a.tokens, a.most);
  const int len = a.lengths[blockIdx.x];
  if (rows.n < 0 || len < rows.n || len > kKvMostContext) {
    if (tid == 0) atomicOr(&g_mx_error_word, kSiteBadCache);
    return;
  }
  bool bad = false;
  for (int i = tid; i < rows.n; i += kKvTreesThreads) {
    const int p = a.parents[rows.q0 + i];
    bad = bad || p < -1 || p >= i;
    up[i] = static_cast<int16_t>(p);
  }
  bad = __syncthreads_or(bad);
  if (bad && tid == 0) atomicOr(&g_mx_error_word, kSiteBadCache);
  for (int i = tid; i < rows.n; i += kKvTreesThreads) {
    uint64_t* row = a.mask + static_cast<int64_t>(rows.q0 + i) * a.words;
    int w = a.words - 1, depth = 0;
    uint64_t bits = 0;
    for (int at = bad ? -1 : i; at >= 0; at = up[at], ++depth) {
      for (; w > at >> 6; --w) {
        row[w] = bits;
        bits = 0;
      }
      if (a.window == 0 || depth < a.window) bits |= 1ull << (at & 63);
    }
    for (; w >= 0; --w) {
      row[w] = bits;
      bits = 0;
    }
    a.positions[rows.q0 + i] = bad ? -1 : len - rows.n + depth - 1;
  }
}

// ================================================================== verification
struct KvVerifyArgs {
  const float* target;  // [tokens] rows of probabilities over the vocabulary
  const float* draft;   // [tokens] rows that the children of a node were drawn from; null: drafts are certain
  int64_t target_stride, draft_stride;
  const int32_t* drafts;
  const int32_t* parents;
  const int32_t* q_start;
  const float* accept;  // [tokens]
  const float* sample;  // [requests]
  int32_t* path;        // [tokens]
  int32_t* next;        // [tokens]: the tokens that the step gives
  int32_t* counts;      // [requests]
  int requests, tokens, most, vocab;
};

constexpr int kKvVerifyThreads = 256;
constexpr int kKvVerifySegment = 512;               // vocabulary entries that a warp sums at a time
constexpr int kKvVerifyMostVocab = 1 << 20;
constexpr int kKvVerifyMostCluster = 8;

// A row's sums are of whole multiples of 2^-44, to which each P is rounded: they come out the same in any order and on any
// number of CTAs, and are off by 2^-45 an entry and a little, all of them the same way where the entries are alike (128256:
// 4e-9 at worst; 1e-11 where the roundings are independent).  Sums in 64-bit floating point would be nearer, but their unit
// runs at 2 a cycle and SM (a row of 128256 would take it 100 us).  Single numbers are kept in units of 2^-60, cut off there:
// of 1 in sums, of the larger of p and q in a test.
constexpr uint64_t kKvOne = 1ull << 60, kKvTakenOne = 1ull << 53;  // 1 so; 1 in W's units
// A sum of P is below 2, or the row is no distribution, which is told.  Z stays below 2 then, so that no product of it passes
// 64 bits, and so does what a number in [0, 2) is times a probability; a warp's part of a sum (below 2^63) stays below
// kKvMostPart, so that no sum of all 64 parts does, and from kKvMostSum on there is no next token.
constexpr uint64_t kKvSumTwo = 1ull << 45, kKvMostSum = 1ull << 56, kKvMostPart = 1ull << 57;

// [0, 2), or -0
__device__ __forceinline__ bool kv_is_probability(float p) {
  const uint32_t u = __float_as_uint(p);
  return u < 0x40000000u || u == 0x80000000u;
}
// anything else counts as 0, and is told
__device__ __forceinline__ float kv_probability(float p, bool& bad) {
  if (kv_is_probability(p)) return p;
  bad = true;
  return 0.f;
}
__device__ __forceinline__ uint64_t kv_fixed(float p) {
  const uint32_t u = __float_as_uint(p), e = (u >> 23) & 0xFFu, m = e ? (u << 8) | 0x80000000u : 0u;
  uint64_t r;
  asm("shr.u64 %0, %1, %2;" : "=l"(r) : "l"(static_cast<uint64_t>(m) << 32), "r"(130u - e));  // (64 and more: 0)
  return r;
}
// the power of two that brings the larger of two into [1, 2) (of two below 2^-126, near to it)
__device__ __forceinline__ float kv_near_one(float p, float q) {
  const uint32_t e = __float_as_uint(fmaxf(fabsf(p), fabsf(q))) >> 23;
  return __uint_as_float((e ? 254 - e : 253) << 23);
}
// max(p - W q, 0) of numbers so kept, W in units of 2^-53.  W grows with every rejected sibling, so W q may be far
// past what 64 bits hold of it: it is compared before it is shifted.
__device__ __forceinline__ uint64_t kv_residual(uint64_t p, uint64_t q, uint64_t taken) {
  if (taken == kKvTakenOne) return p > q ? p - q : 0;
  const uint64_t high = __umul64hi(taken, q << 3);  // W q in units of 2^-52
  return p >> 8 >= high ? p - (high << 8) : 0;
}

// Sums of P, in two limbs: units of 2^-22, and of 2^-44 (signed).  A number plus 2 has the first in its last bits, and what
// is left of it, plus 1.5 * 2^-21, the second; both are added up as they stand, bits and all, and what is too much is
// taken off at the end.  p - q is taken as the nearest FP32 and its error, which together are exact (Knuth's sum of two).
struct KvAmount {
  uint32_t hi = 0, lo = 0;
  int n = 0;
  __device__ __forceinline__ void add(float p, float q) {
    float d = p - q;
    const float b = d - p, e = d > 0.f ? (p - (d - b)) - (q + b) : 0.f;
    d = fmaxf(d, 0.f);
    const float h = d + 2.f;
    hi += __float_as_uint(h);
    lo += __float_as_uint(((d - (h - 2.f)) + e) + 1.5f / (1 << 21));
    ++n;
  }
  __device__ __forceinline__ uint64_t sum() const {
    const uint32_t h = hi - n * 0x40000000u;
    const int32_t l = static_cast<int32_t>(lo - n * __float_as_uint(1.5f / (1 << 21)));
    return (static_cast<uint64_t>(h) << 22) + static_cast<int64_t>(l);
  }
};

// P of an entry, in units of 2^-44.  (q is 0 where W is.)
__device__ __forceinline__ uint64_t kv_amount(float p, float q, uint64_t taken) {
  if (taken > kKvTakenOne) return (kv_residual(kv_fixed(p), kv_fixed(q), taken) + (1u << 15)) >> 16;
  KvAmount a;
  a.add(p, q);
  return a.sum();
}

__device__ __forceinline__ uint64_t kv_warp_sum(uint64_t x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
  return x;
}

__device__ __forceinline__ void kv_cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint64_t kv_cluster_read(const uint64_t* at, uint32_t rank) {
  uint32_t to;
  uint64_t x;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(smem_u32(at)), "r"(rank));
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(x) : "r"(to) : "memory");
  return x;
}

struct KvVerifySmem {
  int16_t up[kKvMostNodes];
  int16_t way[kKvMostNodes];
  int32_t token[kKvMostNodes];
  float p[kKvMostNodes], q[kKvMostNodes], random[kKvMostNodes];  // of a node's token, at its parent
  uint64_t segment[kKvVerifyMostVocab / kKvVerifySegment + 1];  // (one more: rows begin between 16-byte boundaries)
  uint64_t total;
  uint64_t warp_total[kKvVerifyThreads / 32];
};

// four entries from v0 on, of which those in [0, vocab) count.  v0 may be negative: rows are taken from 16-byte
// boundaries on, wherever they begin.
__device__ __forceinline__ float4 kv_row4(const float* row, int v0, int vocab, bool wide) {
  if (wide && v0 >= 0 && v0 + 4 <= vocab) return __ldg(reinterpret_cast<const float4*>(row + v0));
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  if (v0 >= 0 && v0 < vocab) x.x = row[v0];
  if (v0 + 1 >= 0 && v0 + 1 < vocab) x.y = row[v0 + 1];
  if (v0 + 2 >= 0 && v0 + 2 < vocab) x.z = row[v0 + 2];
  if (v0 + 3 >= 0 && v0 + 3 < vocab) x.w = row[v0 + 3];
  return x;
}

// A request's walk from its root (node 0): the children of the last accepted node u are tried in order.  With
// P = p(u), Z = 1, W = 0 at first, child x drawn from q(u) is accepted if r q(x) Z < P(x), else W += Z,
// P = max(p - W q, 0), Z = sum P.  (That is the usual chain of residuals, not divided by their sums: each is
// max(previous / Z - q, 0).)  A certain draft has q = 1 at x alone: P(x) becomes 0 and Z -= p(x), and no sum is needed.  At
// the end the next token is the first one whose running sum of P passes s times all of it.
//
// A cluster of CTAs has a request.  What the tests compare is fetched for all nodes at once, before the walk, so that
// it waits for memory once.  A row's sum is taken in segments of 512, a warp each, 16 bytes a lane and load; the CTAs'
// sums meet in distributed shared memory, and the last sum's segments say where the next token is, which one warp
// then finds.  64 requests with chains of 5 over 128256 tokens: 20.6 us, 3.2 TB/s, 0.47 of the measured copy rate; one with
// 26 nodes over 32000: 8.3 us; 16 with 60 nodes, most of them rejected, 25.1 us.  What bounds it is the chain starts
// - nodes - two probabilities - rows - meeting - segment, about 8 us, in front of and behind the 10 us that the rows
// take.  (Two CTAs of 256 threads a SM, whose loads all fit their registers: three or four CTAs 24 us, two of 512
// threads 23; the sums in three places of the code, 32.)
template <bool CERTAIN>
__global__ void __launch_bounds__(kKvVerifyThreads, 2) kv_verify_kernel(const KvVerifyArgs a) {
  pdl_prologue();
  __shared__ KvVerifySmem sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t rank, ranks;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
  const int request = blockIdx.x / ranks;
  for (int64_t i = kv_rows_end(a.q_start, a.requests, a.tokens) + static_cast<int64_t>(blockIdx.x) * kKvVerifyThreads + tid;
       i < a.tokens; i += static_cast<int64_t>(gridDim.x) * kKvVerifyThreads)
    a.path[i] = a.next[i] = -1;
  const KvRows rows = kv_rows(a.q_start, request, a.tokens, a.most);
  const int n = rows.n;
  // (a cluster's CTAs take the same ways out, so that none waits for another)
  if (n <= 0) {
    if (rank == 0 && tid == 0) {
      if (n < 0) atomicOr(&g_mx_error_word, kSiteBadCache);
      a.counts[request] = 0;
    }
    return;
  }
  bool broken = false, bad = false;
  for (int i = tid; i < n; i += kKvVerifyThreads) {
    const int up = a.parents[rows.q0 + i], token = a.drafts[rows.q0 + i];
    const bool ok = up >= -1 && up < i && (i == 0 || up < 0 || (token >= 0 && token < a.vocab));
    broken = broken || !ok;
    sm.up[i] = static_cast<int16_t>(up);
    sm.token[i] = token;
    sm.random[i] = kv_probability(a.accept[rows.q0 + i], bad);
    float p = 0.f, q = 0.f;
    if (ok && up >= 0) {
      p = a.target[(rows.q0 + up) * a.target_stride + token];
      if (!CERTAIN) q = a.draft[(rows.q0 + up) * a.draft_stride + token];
      p = kv_probability(p, bad);
      q = kv_probability(q, bad);
    }
    sm.p[i] = p;
    sm.q[i] = q;
  }
  if (__syncthreads_or(broken)) {
    for (int i = tid; rank == 0 && i < n; i += kKvVerifyThreads) a.path[rows.q0 + i] = a.next[rows.q0 + i] = -1;
    if (rank == 0 && tid == 0) {
      atomicOr(&g_mx_error_word, kSiteBadCache);
      a.counts[request] = 0;
    }
    return;
  }

  int node = 0, count = 1;
  uint64_t left = kKvOne, taken = 0;  // Z, W
  uint64_t sum = 0;                   // of P, as last taken
  bool own = false;                   // nothing is left of P: the target's own probabilities are drawn from
  const int phase_all = (a.vocab + 3 + kKvVerifySegment - 1) / kKvVerifySegment;  // segments of a row, wherever it begins
  const int per = (phase_all + ranks - 1) / ranks, seg0 = min(static_cast<int>(rank) * per, phase_all);
  const int segs = min(per, phase_all - seg0);
  auto entry_at = [&](const float* row) { return -static_cast<int>((reinterpret_cast<uintptr_t>(row) >> 2) & 3); };
  const float* target = nullptr;
  const float* draft = nullptr;
  bool wide = false;
  auto set_rows = [&]() {
    target = a.target + (rows.q0 + node) * a.target_stride;
    draft = CERTAIN ? target : a.draft + (rows.q0 + node) * a.draft_stride;
    wide = entry_at(target) == entry_at(draft);  // (else the draft's row is read by single words)
  };
  auto clean = [&](float4 (&x)[4], float4 (&y)[4]) {  // (rare)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[k] = make_float4(kv_probability(x[k].x, bad), kv_probability(x[k].y, bad), kv_probability(x[k].z, bad), kv_probability(x[k].w, bad));
      y[k] = make_float4(kv_probability(y[k].x, bad), kv_probability(y[k].y, bad), kv_probability(y[k].z, bad), kv_probability(y[k].w, bad));
    }
  };
  // sums of P by segments into shared memory; returns the sum over all CTAs
  uint64_t before = 0;
  auto sum_rows = [&]() {
    set_rows();
    const int v00 = entry_at(target);
    uint64_t mine = 0;
    for (int s = warp; s < segs; s += kKvVerifyThreads / 32) {
      const int begin = v00 + (seg0 + s) * kKvVerifySegment, v0 = begin + 4 * lane;
      const bool minus = !CERTAIN && taken;
      float4 x[4], y[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) y[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (wide && begin >= 0 && begin + kKvVerifySegment <= a.vocab) {  // (no choice between the loads, which then run together)
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = __ldg(reinterpret_cast<const float4*>(target + v0 + 128 * k));
        if (minus)
#pragma unroll
          for (int k = 0; k < 4; ++k) y[k] = __ldg(reinterpret_cast<const float4*>(draft + v0 + 128 * k));
      } else {
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
          const float4 u = kv_row4(target, v0 + 128 * k, a.vocab, true);
          const float4 t = minus ? kv_row4(draft, v0 + 128 * k, a.vocab, wide) : make_float4(0.f, 0.f, 0.f, 0.f);
          // (straight choices: an index would put x and y into local memory)
          if (k == 0) x[0] = u, y[0] = t;
          if (k == 1) x[1] = u, y[1] = t;
          if (k == 2) x[2] = u, y[2] = t;
          if (k == 3) x[3] = u, y[3] = t;
        }
      }
      uint32_t most = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        most = max(max(most, max(__float_as_uint(x[k].x), __float_as_uint(x[k].y))), max(__float_as_uint(x[k].z), __float_as_uint(x[k].w)));
        most = max(max(most, max(__float_as_uint(y[k].x), __float_as_uint(y[k].y))), max(__float_as_uint(y[k].z), __float_as_uint(y[k].w)));
      }
      if (most >= 0x40000000u) clean(x, y);
      uint64_t sum = 0;
      if (CERTAIN || taken <= kKvTakenOne) {
        KvAmount p;
#pragma unroll
        for (int k = 0; k < 4; ++k) p.add(x[k].x, y[k].x), p.add(x[k].y, y[k].y), p.add(x[k].z, y[k].z), p.add(x[k].w, y[k].w);
        sum = p.sum();
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          sum += kv_amount(x[k].x, y[k].x, taken) + kv_amount(x[k].y, y[k].y, taken) + kv_amount(x[k].z, y[k].z, taken) +
                 kv_amount(x[k].w, y[k].w, taken);
      }
      sum = kv_warp_sum(sum);
      mine += sum;
      if (lane == 0) sm.segment[s] = sum;
    }
    if (lane == 0) sm.warp_total[warp] = min(mine, kKvMostPart);
    __syncthreads();
    if (CERTAIN && warp == 0) {
      // the rejected children's tokens do not count: taken off their segments, and each once
      uint64_t off = 0;
      for (int i = node + 1 + lane; !own && i < n; i += 32) {
        if (sm.up[i] != node) continue;
        bool again = false;
        for (int j = node + 1; j < i; ++j) again = again || (sm.up[j] == node && sm.token[j] == sm.token[i]);
        const int s = (sm.token[i] - v00) / kKvVerifySegment - seg0;
        if (again || s < 0 || s >= segs) continue;
        const uint64_t x = kv_amount(sm.p[i], 0.f, 0);
        off += x;
        atomicAdd(reinterpret_cast<unsigned long long*>(&sm.segment[s]), ~static_cast<unsigned long long>(x) + 1);
      }
      off = kv_warp_sum(off);
      if (lane == 0) sm.total = ~off + 1;
    }
    if (warp == 0) {
      const uint64_t t = kv_warp_sum(lane < kKvVerifyThreads / 32 ? sm.warp_total[lane] : 0);
      if (lane == 0) sm.total = t + (CERTAIN ? sm.total : 0);
    }
    __syncwarp();
    kv_cluster_sync();
    uint64_t sum = 0;
    before = 0;
    for (uint32_t c = 0; c < ranks; ++c) {
      const uint64_t t = kv_cluster_read(&sm.total, c);
      if (c < rank) before += t;
      sum += t;
    }
    __syncwarp();
    kv_cluster_sync();  // (before any of it is written again, or its CTA has gone)
    bad = bad || sum >= kKvSumTwo;
    return sum;
  };

  // the walk, by every warp for itself
  if (tid == 0) sm.way[0] = 0;
  bool summed = false;  // sum is of the present P
  for (int i0 = 1;;) {
    bool rejected = false;
    while (i0 < n) {
      const uint32_t children = __ballot_sync(0xFFFFFFFFu, i0 + lane < n && sm.up[i0 + lane] == node);
      if (!children) {
        i0 += 32;
        continue;
      }
      const int i = i0 + __ffs(children) - 1;
      i0 = i + 1;
      // r q Z < max(p - W q, 0) holds as well for p and q times a power of two (r and p, of a certain draft): so large that
      // 2^-60 of the larger one is what is cut off, for tokens that are next to impossible too
      const float r = sm.random[i], by = CERTAIN ? r : sm.q[i], up = kv_near_one(sm.p[i], by);
      uint64_t p = kv_fixed(sm.p[i] * up), mark = kv_fixed(by * up);
      if (CERTAIN) {
        bool again = false;
        for (int j = node + 1 + lane; j < i; j += 32) again = again || (sm.up[j] == node && sm.token[j] == sm.token[i]);
        if (__any_sync(0xFFFFFFFFu, again)) p = 0;
      } else {
        if (taken) p = kv_residual(p, mark, taken);
        else if (sm.p[i] > 0.f) p = max(p, static_cast<uint64_t>(1));  // (more than r = 0)
        mark = min(static_cast<uint64_t>(__umul64hi(mark << 3, kv_fixed(r) << 3) >> 2), 2 * kKvOne - 1);
      }
      mark = __umul64hi(mark << 3, left << 3) >> 2;
      if (mark < p) {
        if (tid == 0) sm.way[count] = static_cast<int16_t>(i);
        node = i;
        ++count;
        left = kKvOne;
        taken = 0;
        summed = false;
      } else if (CERTAIN) {
        if (p) left -= min(kv_fixed(sm.p[i]), left);
      } else {
        taken += left >> 7;
        rejected = true;
        break;
      }
    }
    if (!rejected && summed) {
      if (sum || own) break;
      taken = 0;  // (the distributions are the same, or differ by rounding)
      own = true;
    }
    // (what stays where there is no next token: nothing is left of P, or it is far from a distribution; in front of the
    // CTAs' meeting, and so of the token)
    if (rank == 0 && tid == 0) a.next[rows.q0 + count - 1] = -1;
    sum = sum_rows();
    summed = true;
    if (rejected) left = min(sum, kKvSumTwo - 1) << 16;
  }
  set_rows();
  // the next token
  if (sum == 0 || sum >= kKvMostSum) {
    if (rank == 0 && tid == 0) atomicOr(&g_mx_error_word, kSiteBadCache);
  } else if (warp == 0) {
    const float s = a.sample[request];
    // what the running sum has to pass
    const uint64_t mark = __umul64hi(sum, min(kv_fixed(kv_probability(s, bad)), kKvOne - 1) << 4);
    bad = bad || !(s < 1.f);
    if (mark >= before && mark - before < sm.total) {
      uint64_t at = before;
      int found = 0;
      for (int s0 = 0; s0 < segs; s0 += 32) {
        uint64_t x = s0 + lane < segs ? sm.segment[s0 + lane] : 0, upto = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint64_t y = __shfl_up_sync(0xFFFFFFFFu, upto, o);
          if (lane >= o) upto += y;
        }
        const uint32_t past = __ballot_sync(0xFFFFFFFFu, at + upto > mark);
        if (past) {
          const int l = __ffs(past) - 1;
          found = s0 + l;
          at += __shfl_sync(0xFFFFFFFFu, upto - x, l);
          break;
        }
        at += __shfl_sync(0xFFFFFFFFu, upto, 31);
      }
      const int v00 = entry_at(target) + (seg0 + found) * kKvVerifySegment;
      int token = -1;
      for (int k = 0; k < 4 && token < 0; ++k) {
        const int v0 = v00 + 128 * k + 4 * lane;
        float4 x[4] = {kv_row4(target, v0, a.vocab, true)}, y[4] = {};
        if (!CERTAIN && taken) y[0] = kv_row4(draft, v0, a.vocab, wide);
        clean(x, y);
        uint64_t v[4] = {kv_amount(x[0].x, y[0].x, taken), kv_amount(x[0].y, y[0].y, taken), kv_amount(x[0].z, y[0].z, taken),
                         kv_amount(x[0].w, y[0].w, taken)};
        if (CERTAIN && !own)
          for (int i = node + 1; i < n; ++i)
            if (sm.up[i] == node)
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (sm.token[i] == v0 + j) v[j] = 0;
        const uint64_t mine = v[0] + v[1] + v[2] + v[3];
        uint64_t upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint64_t z = __shfl_up_sync(0xFFFFFFFFu, upto, o);
          if (lane >= o) upto += z;
        }
        const uint32_t past = __ballot_sync(0xFFFFFFFFu, at + upto > mark);
        if (past) {
          const int l = __ffs(past) - 1;
          uint64_t run = at + upto - mine;
          int j = 0;
          while (j < 3 && run + v[j] <= mark) run += v[j++];
          token = __shfl_sync(0xFFFFFFFFu, v0 + j, l);
        }
        at += __shfl_sync(0xFFFFFFFFu, upto, 31);
      }
      if (lane == 0) a.next[rows.q0 + count - 1] = token;
    }
  }
  if (bad) atomicOr(&g_mx_error_word, kSiteBadCache);
  if (rank == 0) {
    __syncthreads();  // (the way, written by the first thread)
    for (int i = tid; i < n; i += kKvVerifyThreads) {
      a.path[rows.q0 + i] = i < count ? sm.way[i] : -1;
      if (i != count - 1) a.next[rows.q0 + i] = i < count - 1 ? sm.token[sm.way[i + 1]] : -1;
    }
    if (tid == 0) a.counts[request] = count;
  }
}

// ================================================================== compaction
struct KvCompactArgs {
  const int32_t* path;     // [tokens]
  const int32_t* counts;   // [requests]
  const int32_t* lengths;  // [requests]
  const int32_t* q_start;  // [requests + 1]
  const int32_t* tables;   // [requests][max_blocks]
  uint8_t* codes[2];
  float* scale[2];
  int32_t* kept;           // [requests]
  int64_t num_blocks;
  int requests, tokens, max_blocks, kv_heads, shift;
};

constexpr int kKvCompactThreads = 128;

// the largest finite code's magnitude, as FP32, among 16
template <int FMT>
__device__ __forceinline__ float kv_codes_amax(uint4 c) {
  constexpr uint32_t kNan = FMT == 0 ? 0x7F : 0x7C;
  uint32_t m = __vmaxu4(__vmaxu4(c.x & 0x7F7F7F7Fu, c.y & 0x7F7F7F7Fu), __vmaxu4(c.z & 0x7F7F7F7Fu, c.w & 0x7F7F7F7Fu));
  m = __vmaxu4(m, m >> 16);
  m = max(m & 0xFFu, (m >> 8) & 0xFFu);
  if (m >= kNan) {  // (rare) only the finite ones count
    m = 0;
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t x = (w[i / 4] >> (8 * (i % 4))) & 0x7Fu;
      if (x < kNan) m = max(m, x);
    }
  }
  return kv_f16x2_to_float2(kv_codes_to_f16x2<FMT>(m)).x;
}
// codes times ratio, rounded again
template <int FMT>
__device__ __forceinline__ uint4 kv_codes_times(uint4 c, float ratio) {
  uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 lo = kv_f16x2_to_float2(kv_codes_to_f16x2<FMT>(w[i] & 0xFFFFu));
    const float2 hi = kv_f16x2_to_float2(kv_codes_to_f16x2<FMT>(w[i] >> 16));
    w[i] = kv_codes_from_floats<FMT>(lo.x * ratio, lo.y * ratio) | (kv_codes_from_floats<FMT>(hi.x * ratio, hi.y * ratio) << 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Node path[i] of a request moves to place i behind its context.  Paths rise, so path[i] >= i: nodes from the first
// one on that is not in its place move towards the front, and going through them in order never writes what is
// still to be read.  What moves into one block is a run, as in kv_cache_append: the block keeps its scale or, where the
// run's values need a larger one, raises it, and its codes in front are rounded again.  A warp has a request's
// keys, or values, of one kv head: it looks over the path and the blocks, then takes run by run, reading the
// codes for their largest value only where a scale differs.  Latency is the bound: starts, path, tables, scales, codes, one
// after the other: 64 requests of 32 nodes 3.1 us, 500 of 100 nodes with blocks of 16 and 16 heads 10 us (16000 warps, each
// of which goes through that chain for about six tokens).
template <int FMT, int D>
__global__ void __launch_bounds__(kKvCompactThreads) kv_compact_kernel(const KvCompactArgs a) {
  pdl_prologue();
  constexpr int LANES = D / 16, ROWS = 32 / LANES;  // 16 codes a lane
  constexpr float kMax = FMT == 0 ? 448.f : 57344.f;
  const int lane = threadIdx.x & 31, item = blockIdx.x * (kKvCompactThreads / 32) + (threadIdx.x >> 5);
  if (item >= 2 * a.kv_heads) return;  // (whole warps, which have nothing to do with each other)
  const int r = blockIdx.y, which = item / a.kv_heads, h = item - which * a.kv_heads;
  const KvRows rows = kv_rows(a.q_start, r, a.tokens, kKvMostNodes);
  const int len = a.lengths[r], count = a.counts[r], n = rows.n;
  const int32_t* path = a.path + rows.q0;
  const int32_t* table = a.tables + static_cast<int64_t>(r) * a.max_blocks;
  uint8_t* codes = which ? a.codes[1] : a.codes[0];
  float* scales = which ? a.scale[1] : a.scale[0];
  const int P = 1 << a.shift, context = len - n;
  bool ok = n >= 0 && len >= n && len <= a.max_blocks << a.shift && count >= 0 && count <= n;
  int first = count;  // the first node that moves
  if (ok) {
    for (int i0 = 0; i0 < count; i0 += 32) {
      const int i = i0 + lane;
      bool broken = false, moves = false;
      if (i < count) {
        const int node = path[i];
        moves = node != i;
        broken = node < i || node >= n || (i && node <= path[i - 1]);
        if (!broken && moves) {
          const int from = table[(context + node) >> a.shift], to = table[(context + i) >> a.shift];
          broken = from < 0 || from >= a.num_blocks || to < 0 || to >= a.num_blocks;
        }
      }
      if (__any_sync(0xFFFFFFFFu, broken)) ok = false;
      const uint32_t m = __ballot_sync(0xFFFFFFFFu, moves);
      if (m) first = min(first, i0 + __ffs(m) - 1);
    }
  }
  if (item == 0 && lane == 0) {
    a.kept[r] = ok ? context + count : len;
    if (!ok) atomicOr(&g_mx_error_word, kSiteBadCache);
  }
  if (!ok) return;
  const int sub = lane / LANES, word = lane % LANES;
  for (int j0 = first; j0 < count;) {
    const int off = (context + j0) & (P - 1), end = min(count, j0 + P - off);  // the run
    const int64_t to = static_cast<int64_t>(table[(context + j0) >> a.shift]) * a.kv_heads + h;
    const float old = scales[to];
    uint8_t* dst = codes + to * (static_cast<int64_t>(P) * D) + 16 * word;
    auto source = [&](int j, float& s) {
      const int at = context + path[j];
      const int64_t from = static_cast<int64_t>(table[at >> a.shift]) * a.kv_heads + h;
      s = scales[from];
      return codes + (from * P + (at & (P - 1))) * D + 16 * word;
    };
    auto in_range = [](float s) { return s == 0.f || (s >= kKvLeastScale && s <= kKvMostScale); };
    bool odd = !in_range(old);
    float amax = 0.f;
    for (int j = j0 + sub; j < end; j += ROWS) {
      float s;
      const uint8_t* at = source(j, s);
      odd = odd || !in_range(s);
      // (what becomes NaN says nothing of the scale: it would wipe out what is in front and beside it)
      if (s != old && in_range(s)) amax = fmaxf(amax, kv_codes_amax<FMT>(*reinterpret_cast<const uint4*>(at)) * s);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
    if (odd) atomicOr(&g_mx_error_word, kSiteBadCache);
    if (in_range(old)) {  // (a block of any other scale is NaN to who sees it, and stays so)
      float now = old;
      if (old == 0.f) now = amax > 0.f ? kv_scale_for<FMT>(amax) : 1.f;  // (the block is zeros: it takes the run's own)
      else if (amax > kMax * old) now = fmaxf(old, kv_scale_for<FMT>(amax));
      if (now != old) {
        const float ratio = old / now;
        for (int row = sub; row < off; row += ROWS) {
          uint4* at = reinterpret_cast<uint4*>(dst + row * D);
          *at = old == 0.f ? make_uint4(0, 0, 0, 0) : kv_codes_times<FMT>(*at, ratio);
        }
      }
      for (int j1 = j0; j1 < end; j1 += ROWS) {
        const int j = j1 + sub;
        uint4 c = make_uint4(0, 0, 0, 0);
        if (j < end) {
          float s;
          const uint8_t* at = source(j, s);
          c = *reinterpret_cast<const uint4*>(at);
          if (!in_range(s)) c = make_uint4(0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu);
          else if (s != now) c = s == 0.f ? make_uint4(0, 0, 0, 0) : kv_codes_times<FMT>(c, s / now);
        }
        __syncwarp();  // all of these have been read before one is written
        if (j < end) *reinterpret_cast<uint4*>(dst + (off + j - j0) * D) = c;
      }
      __syncwarp();
      if (lane == 0 && now != old) scales[to] = now;
    }
    __syncwarp();
    j0 = end;
  }
}

}  // namespace mxgb
