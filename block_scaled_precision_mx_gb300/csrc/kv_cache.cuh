// kv_cache.cuh -- the 8-bit key/value cache: block tables and slot maps from request lengths, and
// the quantizing write of new keys and values.
//
// A cache holds codes [blocks][kv heads][P tokens][D] (E4M3 or E5M2) and one FP32 scale for each
// block of P tokens and kv head, [blocks][kv heads]; a token's value is code * scale.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

#include "mx_device.cuh"

namespace mxgb {

// ================================================================== block tables
struct KvTablesArgs {
  int32_t* tables;         // [requests][max_blocks]
  const int32_t* before;   // [requests] tokens each request's blocks hold now
  const int32_t* after;    // [requests] tokens they are to hold
  int32_t* free_list;      // [capacity], a stack of unused blocks
  const int32_t* free_count;
  int32_t* q_start;        // [requests + 1]
  int64_t* slots;          // [num_tokens]
  int32_t* positions;      // [num_tokens]
  int32_t* info;           // {free blocks left, blocks missing}
  int requests, max_blocks, capacity, num_tokens, shift;  // P = 1 << shift
  int wide;                // slots and positions are 16-byte aligned
};

constexpr int kKvTablesThreads = 512;
constexpr int kKvMaxRequests = 16384;  // three prefix arrays of 4 bytes each in shared memory

// largest r with prefix[r] <= i, for prefix[0] = 0 <= i < prefix[n]
__device__ __forceinline__ int kv_prefix_find(const int* prefix, int n, int i) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

// With held = ceil(before / P) and want = ceil(after / P): a request that shrinks pushes its table
// entries want..held-1 on the free stack, one that grows pops entries held..want-1 off its top, in
// request order, pushes first.  Tokens before..after-1 of the growing requests are the step's new
// tokens, numbered request by request.
//
// All of it follows from three exclusive prefix sums over the requests (new tokens, popped blocks,
// pushed blocks), which every CTA computes for itself: no CTA waits for another and one launch does
// all.  Nothing that is read is written: pops read stack entries below free_count and table entries
// of shrinking requests, pushes write entries from free_count on, and only growing requests' tables
// are written.  Latency is the bound: 64 requests 4.6 us, 2000 requests with 206669 new tokens 17 us (4 MB).
__global__ void __launch_bounds__(kKvTablesThreads) kv_block_tables_kernel(const KvTablesArgs a) {
  pdl_prologue();
  extern __shared__ int kv_prefix_smem[];
  const int R = a.requests, P = 1 << a.shift;
  int* new_at = kv_prefix_smem;       // [R + 1]
  int* need_at = new_at + R + 1;      // [R + 1]
  int* gone_at = need_at + R + 1;     // [R + 1]
  __shared__ long long warp_sums[3][kKvTablesThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  bool bad = false;
  const long long longest = static_cast<long long>(a.max_blocks) << a.shift;
  // each thread takes a stretch of the requests; the stretches' sums are scanned
  const int per = (R + kKvTablesThreads - 1) / kKvTablesThreads;
  const int first_r = min(tid * per, R), end_r = min(first_r + per, R);
  auto moves = [&](int r, int (&v)[3]) {
    const int before = a.before[r], after = a.after[r];
    v[0] = v[1] = v[2] = 0;
    if (before < 0 || after < 0 || before > longest || after > longest) return false;
    const int held = (before + P - 1) >> a.shift, want = (after + P - 1) >> a.shift;
    v[0] = max(after - before, 0);
    v[1] = max(want - held, 0);
    v[2] = max(held - want, 0);
    return true;
  };
  long long sum[3] = {0, 0, 0}, carry[3];
  for (int r = first_r; r < end_r; ++r) {
    int v[3];
    if (!moves(r, v)) bad = true;
#pragma unroll
    for (int k = 0; k < 3; ++k) sum[k] += v[k];
  }
  long long at[3];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    long long incl = sum[k];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += u;
    }
    if (lane == 31) warp_sums[k][warp] = incl;
    at[k] = incl - sum[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    long long s = lane < kKvTablesThreads / 32 ? warp_sums[k][lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xFFFFFFFFu, s, o);
      if (lane >= o) s += u;
    }
    carry[k] = __shfl_sync(0xFFFFFFFFu, s, 31);
    at[k] += warp ? __shfl_sync(0xFFFFFFFFu, s, warp - 1) : 0;
  }
  for (int r = first_r; r < end_r; ++r) {  // (sums past 2^31 are only ever those of a call that is refused below)
    int v[3];
    moves(r, v);
    new_at[r] = static_cast<int>(at[0]);
    need_at[r] = static_cast<int>(at[1]);
    gone_at[r] = static_cast<int>(at[2]);
#pragma unroll
    for (int k = 0; k < 3; ++k) at[k] += v[k];
  }
  const long long count = *a.free_count, avail = count + carry[2], left = avail - carry[1];
  if (count < 0 || avail > a.capacity || carry[0] > a.num_tokens) bad = true;
  bad = __syncthreads_or(bad);
  const bool fits = !bad && left >= 0;
  if (tid == 0) {
    new_at[R] = static_cast<int>(carry[0]);
    need_at[R] = static_cast<int>(carry[1]);
    gone_at[R] = static_cast<int>(carry[2]);
    if (blockIdx.x == 0) {
      if (bad) atomicOr(&g_mx_error_word, kSiteBadCache);
      a.info[0] = static_cast<int>(fits ? left : count);
      a.info[1] = static_cast<int>(!bad && left < 0 ? -left : 0);
    }
  }
  __syncthreads();
  const int first = blockIdx.x * kKvTablesThreads + tid, step = gridDim.x * kKvTablesThreads;
  for (int r = first; r <= R; r += step) a.q_start[r] = bad ? 0 : new_at[r];

  const int icount = static_cast<int>(count), iavail = static_cast<int>(avail);
  auto pushed = [&](int i) {  // the i-th block that this call puts on the stack
    const int r = kv_prefix_find(gone_at, R, i);
    const int want = (a.after[r] + P - 1) >> a.shift;
    return a.tables[static_cast<int64_t>(r) * a.max_blocks + want + (i - gone_at[r])];
  };
  auto popped = [&](int j) {  // the j-th block that it takes off
    const int at = iavail - 1 - j;
    return at < icount ? a.free_list[at] : pushed(at - icount);
  };
  bool negative = false;  // a block number below 0 among the held, the free or the given-back ones
  if (fits) {
    const int pops = need_at[R], pushes = max(gone_at[R] - pops, 0);
    for (int j = first; j < pops; j += step) {
      const int r = kv_prefix_find(need_at, R, j);
      const int held = (a.before[r] + P - 1) >> a.shift;
      const int block = popped(j);
      negative = negative || block < 0;
      a.tables[static_cast<int64_t>(r) * a.max_blocks + held + (j - need_at[r])] = block;
    }
    for (int i = first; i < pushes; i += step) {
      const int block = pushed(i);
      negative = negative || block < 0;
      a.free_list[icount + i] = block;
    }
  }
  // four tokens a thread: one search, then along the prefix
  const int tokens = fits ? new_at[R] : 0;
  for (int64_t t0 = 4ll * first; t0 < a.num_tokens; t0 += 4ll * step) {
    int64_t slot[4];
    int pos[4];
    int r = -1, next_at = 0, before = 0, held = 0, last_b = -1, block = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = static_cast<int>(t0) + i;
      slot[i] = -1;
      pos[i] = -1;
      if (t < tokens) {
        if (r < 0 || t >= next_at) {
          if (r < 0) r = kv_prefix_find(new_at, R, t);
          else
            while (new_at[r + 1] <= t) ++r;
          next_at = new_at[r + 1];
          before = a.before[r];
          held = (before + P - 1) >> a.shift;
          last_b = -1;
        }
        pos[i] = before + (t - new_at[r]);
        const int b = pos[i] >> a.shift;
        if (b != last_b) {
          block = b < held ? a.tables[static_cast<int64_t>(r) * a.max_blocks + b] : popped(need_at[r] + b - held);
          last_b = b;
        }
        negative = negative || block < 0;  // (such a token has no slot: -1, not one that may happen to be -1)
        slot[i] = block < 0 ? -1 : (static_cast<int64_t>(block) << a.shift) + (pos[i] & (P - 1));
      }
    }
    if (a.wide && t0 + 4 <= a.num_tokens) {
      longlong2* s = reinterpret_cast<longlong2*>(a.slots + t0);
      s[0] = make_longlong2(slot[0], slot[1]);
      s[1] = make_longlong2(slot[2], slot[3]);
      *reinterpret_cast<int4*>(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (t0 + i < a.num_tokens) {
          a.slots[t0 + i] = slot[i];
          a.positions[t0 + i] = pos[i];
        }
    }
  }
  if (negative) atomicOr(&g_mx_error_word, kSiteBadCache);
}

// ================================================================== 8-bit codes
// FMT 0 = E4M3, 1 = E5M2.  Both hold every code exactly in FP16, which the matrix products use.
template <int FMT>
__device__ __forceinline__ uint32_t kv_codes_to_f16x2(uint32_t two_codes) {
  uint32_t r;
  if (FMT == 0)
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(two_codes));
  else
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e5m2x2 %0, lo;\n\t}" : "=r"(r) : "r"(two_codes));
  return r;
}
// four codes, low pair and high pair
template <int FMT>
__device__ __forceinline__ void kv_codes4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (FMT == 0)
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  else
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e5m2x2 %0, l;\n\tcvt.rn.f16x2.e5m2x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}
template <int FMT>
__device__ __forceinline__ uint32_t kv_codes_from_floats(float lo, float hi) {
  return FMT == 0 ? cvt_e4m3x2(lo, hi) : cvt_e5m2x2(lo, hi);
}
__device__ __forceinline__ float2 kv_f16x2_to_float2(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// ================================================================== append
struct KvAppendArgs {
  const uint16_t* x[2];         // keys, values: [tokens][kv heads][D], bf16 or fp16
  int64_t stride_t[2], stride_h[2];
  uint8_t* codes[2];            // [blocks][kv heads][P][D]
  float* scale[2];              // [blocks][kv heads]
  const int64_t* slots;         // [tokens]; -1: no place
  int64_t num_slots;            // blocks * P
  int tokens, kv_heads, shift, chunk;
};

constexpr int kKvAppendThreads = 256;
constexpr int kKvMaxExp = 48;  // scales are 2^-48 .. 2^48
constexpr float kKvLeastScale = 1.f / (1ull << kKvMaxExp), kKvMostScale = static_cast<float>(1ull << kKvMaxExp);

// Scale 2^k: k the smallest with MAX * 2^k >= amax, in [-48, 48].  MAX is 1.75 * 2^8 (E4M3) or
// 1.75 * 2^15 (E5M2), so k follows from amax's exponent and whether its significand is above 1.75.
template <int FMT>
__device__ __forceinline__ float kv_scale_for(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  int k = static_cast<int>(bits >> 23) - 127 - (FMT == 0 ? 8 : 15) + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  k = min(max(k, -kKvMaxExp), kKvMaxExp);
  return __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
}

template <bool F16>
__device__ __forceinline__ float2 kv_unpack2(uint32_t w) {
  if (F16) return kv_f16x2_to_float2(w);
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// A run is a stretch of new tokens with consecutive slots of one block.  A group of W warps takes one
// (run, head, keys or values) at a time: the run's rows come into registers in one go (16 bytes a
// thread and load, D / 8 lanes a row, PASSES loads a thread for a whole block), the group finds the
// largest finite |x|, settles the block's scale and writes the codes.  A run that starts a block sets its
// scale; one that goes on in a block keeps the block's scale or grows it, and then the tokens in front are
// re-rounded to the new scale (scales are powers of two, so that is exact but for codes that become
// subnormal).  One read of the input, one write of the codes; the block's old codes move only when its
// scale grows.  The bound is memory; what keeps it busy is many small groups a SM (W and PASSES follow the
// block's size so that a thread holds 4 or 8 words), hence few registers.
template <int FMT, bool F16, int D, int W, int PASSES>
__global__ void __launch_bounds__(kKvAppendThreads, 5) kv_append_kernel(const KvAppendArgs a) {
  pdl_prologue();
  constexpr int kLanesPerRow = D / 8, kGroupThreads = 32 * W, kRowsPerPass = kGroupThreads / kLanesPerRow;
  constexpr int kGroups = kKvAppendThreads / kGroupThreads;
  __shared__ int64_t slot_of[2 * 128 + 1];  // slots of tokens t0 - 1 .. t0 + chunk + P - 1
  __shared__ int starts[128];
  __shared__ int num_starts;
  __shared__ uint32_t group_max[kGroups][W];
  const int tid = threadIdx.x, lane = tid & 31;
  const int P = 1 << a.shift, t0 = blockIdx.x * a.chunk;
  if (tid == 0) num_starts = 0;
  for (int i = tid; i <= a.chunk + P; i += kKvAppendThreads) {
    const int t = t0 - 1 + i;
    slot_of[i] = t >= 0 && t < a.tokens ? a.slots[t] : -1;
  }
  __syncthreads();
  if (tid < a.chunk) {
    const int64_t slot = slot_of[tid + 1];
    if (slot >= 0 && slot < a.num_slots) {
      if ((slot & (P - 1)) == 0 || slot_of[tid] != slot - 1) starts[atomicAdd(&num_starts, 1)] = tid;
    } else if (slot != -1) {
      atomicOr(&g_mx_error_word, kSiteBadCache);
    }
  }
  __syncthreads();
  const int group = tid / kGroupThreads, gt = tid % kGroupThreads;
  const int item = blockIdx.y * kGroups + group;
  if (item >= 2 * a.kv_heads) return;  // (whole groups leave; the barriers below are a group's own)
  const int which = item / a.kv_heads, h = item - which * a.kv_heads;
  const int row0 = gt / kLanesPerRow, lr = gt % kLanesPerRow;
  // (chosen, not indexed: an index would copy the arguments to local memory)
  const uint16_t* x_at = which ? a.x[1] : a.x[0];
  const int64_t stride_t = which ? a.stride_t[1] : a.stride_t[0], stride_h = which ? a.stride_h[1] : a.stride_h[0];
  uint8_t* codes = which ? a.codes[1] : a.codes[0];
  float* scales = which ? a.scale[1] : a.scale[0];
  for (int s = 0; s < num_starts; ++s) {
    const int at_t = starts[s];
    const int64_t slot = slot_of[at_t + 1];
    const int off = static_cast<int>(slot & (P - 1));
    const int64_t block = slot >> a.shift;
    float* scale_at = scales + block * a.kv_heads + h;
    const float old_scale = off ? *scale_at : 0.f;
    int n = 0;  // the run's length
    for (int i0 = 0; i0 < P; i0 += 32) {
      const int i = i0 + lane;
      const uint32_t m = __ballot_sync(0xFFFFFFFFu, off + i < P && slot_of[at_t + 1 + i] == slot + i);
      n += m == 0xFFFFFFFFu ? 32 : __ffs(~m) - 1;
      if (m != 0xFFFFFFFFu) break;
    }
    const uint16_t* src = x_at + (t0 + at_t) * stride_t + h * stride_h + lr * 8;
    uint8_t* dst = codes + (block * a.kv_heads + h) * (static_cast<int64_t>(P) * D) + lr * 8;
    uint4 v[PASSES];
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int row = row0 + p * kRowsPerPass;
      v[p] = row < n ? *reinterpret_cast<const uint4*>(src + row * stride_t) : make_uint4(0, 0, 0, 0);
    }
    // largest |x| as 16-bit patterns, two at a time: finite values order like their patterns
    uint32_t m2 = 0;
#pragma unroll
    for (int p = 0; p < PASSES; ++p)
      m2 = __vmaxu2(m2, __vmaxu2(__vmaxu2(v[p].x & 0x7FFF7FFFu, v[p].y & 0x7FFF7FFFu),
                                 __vmaxu2(v[p].z & 0x7FFF7FFFu, v[p].w & 0x7FFF7FFFu)));
    constexpr uint32_t kInf = F16 ? 0x7C00u : 0x7F80u;
    uint32_t m1 = max(m2 & 0xFFFFu, m2 >> 16);
    if (m1 >= kInf) {  // an Inf or NaN among this thread's values: only the finite ones count
      m1 = 0;
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        const uint32_t w[4] = {v[p].x, v[p].y, v[p].z, v[p].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t lo = w[j] & 0x7FFFu, hi = (w[j] >> 16) & 0x7FFFu;
          if (lo < kInf) m1 = max(m1, lo);
          if (hi < kInf) m1 = max(m1, hi);
        }
      }
    }
    m1 = __reduce_max_sync(0xFFFFFFFFu, m1);
    if (W > 1) {
      if (lane == 0) group_max[group][gt >> 5] = m1;
      asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(kGroupThreads) : "memory");
#pragma unroll
      for (int w = 0; w < W; ++w) m1 = max(m1, group_max[group][w]);
      // (the next round's write is behind the barrier at the end of this one)
    }
    // A block that goes on has a scale in range, or 0: it holds zeros.  Any other leaves the run out.  (Looked at behind
    // the meeting, so that the maximum does not wait for the scale: 64k tokens 76 us, 86 in front of it.)
    if (off && !(old_scale == 0.f || (old_scale >= kKvLeastScale && old_scale <= kKvMostScale))) {
      if (gt == 0) atomicOr(&g_mx_error_word, kSiteBadCache);
    } else {
      const float amax = F16 ? __half2float(__ushort_as_half(static_cast<unsigned short>(m1))) : __uint_as_float(m1 << 16);
      float scale = amax > 0.f ? kv_scale_for<FMT>(amax) : (off && old_scale > 0.f ? old_scale : 1.f);
      if (off) scale = fmaxf(scale, old_scale);
      if (gt == 0) *scale_at = scale;
      if (off && scale > old_scale) {
        const float ratio = old_scale / scale;
        for (int row = row0; row < off; row += kRowsPerPass) {
          uint2* at = reinterpret_cast<uint2*>(dst + row * D);
          uint2 c = *at;
          uint32_t w[2] = {c.x, c.y};
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float2 lo = kv_f16x2_to_float2(kv_codes_to_f16x2<FMT>(w[j] & 0xFFFFu));
            const float2 hi = kv_f16x2_to_float2(kv_codes_to_f16x2<FMT>(w[j] >> 16));
            w[j] = kv_codes_from_floats<FMT>(lo.x * ratio, lo.y * ratio) |
                   (kv_codes_from_floats<FMT>(hi.x * ratio, hi.y * ratio) << 16);
          }
          *at = old_scale == 0.f ? make_uint2(0, 0) : make_uint2(w[0], w[1]);
        }
      }
      const float inv = 1.f / scale;
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        const int row = row0 + p * kRowsPerPass;
        if (row < n) {
          const float2 x0 = kv_unpack2<F16>(v[p].x), x1 = kv_unpack2<F16>(v[p].y), x2 = kv_unpack2<F16>(v[p].z),
                       x3 = kv_unpack2<F16>(v[p].w);
          const uint32_t lo = kv_codes_from_floats<FMT>(x0.x * inv, x0.y * inv) |
                              (kv_codes_from_floats<FMT>(x1.x * inv, x1.y * inv) << 16);
          const uint32_t hi = kv_codes_from_floats<FMT>(x2.x * inv, x2.y * inv) |
                              (kv_codes_from_floats<FMT>(x3.x * inv, x3.y * inv) << 16);
          *reinterpret_cast<uint2*>(dst + static_cast<int64_t>(off + row) * D) = make_uint2(lo, hi);
        }
      }
    }
    if (W > 1) asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(kGroupThreads) : "memory");
  }
}

}  // namespace mxgb
