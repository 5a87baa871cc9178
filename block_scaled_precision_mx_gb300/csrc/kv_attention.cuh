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
};

constexpr float kLn2 = 0.69314718055994531f;

// One CTA per query row: keys in chunks of 128, one key a thread; then one or more output elements a
// thread.  Right for every call and nothing more.
template <int FMT, bool F16, int D>
__global__ void __launch_bounds__(128) kv_attention_rows_kernel(const KvAttnArgs a) {
  pdl_prologue();
  const int t = blockIdx.x, head = blockIdx.y, h = head / (a.heads / a.kv_heads), tid = threadIdx.x;
  __shared__ float qs[D], ps[128], red[4];
  __shared__ int64_t where[128];
  int lo = 0, hi = a.requests;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.q_start[mid] <= t) lo = mid;
    else hi = mid;
  }
  const int r = lo, P = 1 << a.shift;
  int len = a.lengths[r];
  const int pos = len - (a.q_start[r + 1] - t);
  if (t >= a.q_start[a.requests]) len = 0;
  const int begin = a.window ? max(0, pos - a.window + 1) : 0;
  const int end = a.causal ? min(len, pos + 1) : len;
  if (tid < D) {
    const uint16_t* src = a.q + t * a.stride_t + head * a.stride_h + tid;
    qs[tid] = F16 ? __half2float(__ushort_as_half(*src)) : bf16_bits_to_float(*src);
  }
  float m = -INFINITY, l = 0.f, o = 0.f;
  __syncthreads();
  for (int j0 = begin; j0 < end; j0 += 128) {
    const int j = j0 + tid;
    float z = -INFINITY, sv = 0.f;
    if (j < end) {
      const int block = a.tables[static_cast<int64_t>(r) * a.max_blocks + (j >> a.shift)];
      const bool there = block >= 0 && block < a.num_blocks;
      const int64_t bh = static_cast<int64_t>(there ? block : 0) * a.kv_heads + h;
      const int64_t at = (bh * P + (j & (P - 1))) * D;
      float acc = 0.f;
      for (int d = 0; d < D; d += 4) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(a.k_codes + at + d);
        const float2 x = kv_f16x2_to_float2(kv_codes_to_f16x2<FMT>(w & 0xFFFFu));
        const float2 y = kv_f16x2_to_float2(kv_codes_to_f16x2<FMT>(w >> 16));
        acc += qs[d] * x.x + qs[d + 1] * x.y + qs[d + 2] * y.x + qs[d + 3] * y.y;
      }
      z = acc * a.scale_log2 * a.k_scale[bh];
      sv = a.v_scale[bh];
      where[tid] = at;
      if (!there) atomicOr(&g_mx_error_word, kSiteBadCache);
    }
    float zm = z;
    for (int s = 16; s; s >>= 1) zm = fmaxf(zm, __shfl_xor_sync(0xFFFFFFFFu, zm, s));
    if ((tid & 31) == 0) red[tid >> 5] = zm;
    __syncthreads();
    const float m_new = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    const float m_use = m_new == -INFINITY ? 0.f : m_new;
    const float p = exp2f(z - m_use), keep = exp2f(m - m_use);
    ps[tid] = p * sv;
    float sum = p;
    for (int s = 16; s; s >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, s);
    __syncthreads();
    if ((tid & 31) == 0) red[tid >> 5] = sum;
    __syncthreads();
    l = l * keep + (red[0] + red[1]) + (red[2] + red[3]);
    m = m_new;
    o *= keep;
    if (tid < D)
      for (int i = 0; i < min(128, end - j0); ++i)
        o += ps[i] * kv_f16x2_to_float2(kv_codes_to_f16x2<FMT>(a.v_codes[where[i] + tid])).x;
    __syncthreads();
  }
  if (tid < D) {
    const float x = end > begin ? o / l : 0.f;
    const int64_t at = (static_cast<int64_t>(t) * a.heads + head) * D + tid;
    a.out[at] = F16 ? __half_as_ushort(__float2half_rn(x)) : __bfloat16_as_ushort(__float2bfloat16_rn(x));
  }
  if (tid == 0) a.lse[static_cast<int64_t>(t) * a.heads + head] = end > begin ? m * kLn2 + logf(l) : -INFINITY;
}

}  // namespace mxgb
