// qk_norm.cuh -- RMS norm of each head of queries and keys and their rotation to positions, in one pass; and its
// backward pass.
//
//   y = R(p) (w * x r),  r = (mean x^2 + eps)^(-1/2)
//   g = R(p)^T dy,  xh = x r:   dx = r (w g - xh mean(w g xh)),   dw = sum over tokens and heads of g xh
//
// R turns pairs (i, rot / 2 + i), or neighbours (2i, 2i + 1), of a head's first `rot` values by the angle whose cosine
// and sine the table has at the token's position.
#pragma once

#include "kv_cache.cuh"

namespace mxgb {

struct QkNormArgs {
  const uint16_t* x[2];     // queries, keys: [tokens][heads][D], bf16 or fp16
  int64_t xst[2], xsh[2];
  const uint16_t* dy[2];    // (backward)
  int64_t dst[2], dsh[2];
  uint16_t* out[2];         // y, or dx
  int64_t ost[2], osh[2];
  const void* weight[2];    // [D], x's type or FP32
  const float* table;       // [positions][rot]: cosines, then sines; null: no rotation
  const int32_t* positions; // [tokens]; -1 leaves a token out; may be null without a table
  float* partial;           // (backward) [CTAs][2][D]
  float eps;
  int tokens, heads[2], dim, rot, most_pos, interleaved, weight_f32;
};

constexpr int kQkThreads = 256;

// eight values of a head's row, as FP32
template <bool F16>
__device__ __forceinline__ void qk_load8(float (&f)[8], const uint16_t* at, bool on) {
  const uint4 v = on ? *reinterpret_cast<const uint4*>(at) : make_uint4(0, 0, 0, 0);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = kv_unpack2<F16>(w[i]);
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}
template <bool F16>
__device__ __forceinline__ uint32_t qk_pack2(float lo, float hi) {
  if (F16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <bool F16>
__device__ __forceinline__ void qk_store8(uint16_t* at, const float (&f)[8]) {
  *reinterpret_cast<uint4*>(at) = make_uint4(qk_pack2<F16>(f[0], f[1]), qk_pack2<F16>(f[2], f[3]),
                                             qk_pack2<F16>(f[4], f[5]), qk_pack2<F16>(f[6], f[7]));
}
template <int LANES>
__device__ __forceinline__ float qk_sum(float x) {
#pragma unroll
  for (int o = LANES / 2; o; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
  return x;
}

// A lane's part of a token's cosines and sines, and of a weight: eight values each.  `turns` and `partner` say where
// the lane's values lie in the rotation.
template <int LANES>
struct QkLane {
  float c[8], s[8];
  int col, partner;  // the first of its values; the lane (of the warp) that has what they are turned with
  bool on, turns;

  __device__ __forceinline__ QkLane(const QkNormArgs& a) {
    const int lane = threadIdx.x & 31, l = lane % LANES, half = a.rot / 16;
    col = 8 * l;
    on = col < a.dim;
    turns = col < a.rot;
    partner = a.interleaved || !turns ? lane : l < half ? lane + half : lane - half;
  }
  // the angles of a position.  Interleaved: a pair's values have the same; else the two halves have.
  __device__ __forceinline__ void angles(const QkNormArgs& a, int p) {
    if (!turns) return;
    const float* row = a.table + static_cast<int64_t>(p) * a.rot;
    const int half = a.rot / 2;
    if (a.interleaved) {
      const float4 cc = *reinterpret_cast<const float4*>(row + col / 2), ss = *reinterpret_cast<const float4*>(row + half + col / 2);
      c[0] = c[1] = cc.x, c[2] = c[3] = cc.y, c[4] = c[5] = cc.z, c[6] = c[7] = cc.w;
      s[1] = ss.x, s[3] = ss.y, s[5] = ss.z, s[7] = ss.w;
      s[0] = -ss.x, s[2] = -ss.y, s[4] = -ss.z, s[6] = -ss.w;
    } else {
      const int at = col < half ? col : col - half;
      const float sign = col < half ? -1.f : 1.f;
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        const float4 cc = *reinterpret_cast<const float4*>(row + at + i), ss = *reinterpret_cast<const float4*>(row + half + at + i);
        c[i] = cc.x, c[i + 1] = cc.y, c[i + 2] = cc.z, c[i + 3] = cc.w;
        s[i] = sign * ss.x, s[i + 1] = sign * ss.y, s[i + 2] = sign * ss.z, s[i + 3] = sign * ss.w;
      }
    }
  }
  // f turned (BACK: turned back).  By all lanes of a warp.
  template <bool BACK>
  __device__ __forceinline__ void turn(const QkNormArgs& a, float (&f)[8]) const {
    if (a.rot == 0) return;
    float o[8];
    if (a.interleaved) {
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = f[i ^ 1];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = __shfl_sync(0xFFFFFFFFu, f[i], partner);
    }
    if (!turns) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = fmaf(BACK ? -s[i] : s[i], o[i], f[i] * c[i]);
  }
};

__device__ __forceinline__ void qk_weights(float (&w)[8], const QkNormArgs& a, int which, int col, bool on, bool f16) {
  const void* from = which ? a.weight[1] : a.weight[0];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    w[i] = 0.f;
    if (!on) continue;
    if (a.weight_f32) w[i] = static_cast<const float*>(from)[col + i];
    else if (f16) w[i] = __half2float(static_cast<const __half*>(from)[col + i]);
    else w[i] = __bfloat162float(static_cast<const __nv_bfloat16*>(from)[col + i]);
  }
}

// The token's position; -1: it is left out.  Others out of range are told.
__device__ __forceinline__ int qk_position(const QkNormArgs& a, int token) {
  if (!a.positions) return 0;
  const int p = a.positions[token];
  if (p >= 0 && (!a.table || p < a.most_pos)) return p;
  if (p != -1) atomicOr(&g_mx_error_word, kSiteBadCache);
  return -1;
}

// LANES lanes have a head's row, eight values each; a warp takes HEADS * 32 / LANES heads of a token's queries or of
// its keys at a time, all loads first.  Memory is the bound.
template <int LANES, bool F16, int HEADS>
__global__ void __launch_bounds__(kQkThreads) qk_norm_rope_kernel(const QkNormArgs a) {
  pdl_prologue();
  constexpr int ROWS = 32 / LANES, AT_ONCE = ROWS * HEADS;
  const int sub = (threadIdx.x & 31) / LANES;
  const int parts0 = (a.heads[0] + AT_ONCE - 1) / AT_ONCE, parts = parts0 + (a.heads[1] + AT_ONCE - 1) / AT_ONCE;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * (kQkThreads / 32) + (threadIdx.x >> 5);
  if (item >= static_cast<int64_t>(a.tokens) * parts) return;
  const int token = static_cast<int>(item / parts), part = static_cast<int>(item - static_cast<int64_t>(token) * parts);
  const int which = part >= parts0, h0 = (which ? part - parts0 : part) * AT_ONCE + sub;
  const int heads = which ? a.heads[1] : a.heads[0];
  QkLane<LANES> lane(a);
  const int p = qk_position(a, token);
  if (p < 0) return;
  const uint16_t* x = (which ? a.x[1] : a.x[0]) + token * (which ? a.xst[1] : a.xst[0]) + lane.col;
  uint16_t* y = (which ? a.out[1] : a.out[0]) + token * (which ? a.ost[1] : a.ost[0]) + lane.col;
  const int64_t xsh = which ? a.xsh[1] : a.xsh[0], osh = which ? a.osh[1] : a.osh[0];
  float f[HEADS][8], w[8];
#pragma unroll
  for (int i = 0; i < HEADS; ++i) qk_load8<F16>(f[i], x + (h0 + i * ROWS) * xsh, lane.on && h0 + i * ROWS < heads);
  qk_weights(w, a, which, lane.col, lane.on, F16);
  lane.angles(a, p);
  const float inv_dim = 1.f / a.dim;
#pragma unroll
  for (int i = 0; i < HEADS; ++i) {
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = fmaf(f[i][j], f[i][j], sum);
    const float r = rsqrtf(fmaf(qk_sum<LANES>(sum), inv_dim, a.eps));
#pragma unroll
    for (int j = 0; j < 8; ++j) f[i][j] *= r * w[j];
    lane.template turn<false>(a, f[i]);
    if (lane.on && h0 + i * ROWS < heads) qk_store8<F16>(y + (h0 + i * ROWS) * osh, f[i]);
  }
}

// The same items, warp after warp of a grid of a fixed size; the weights' gradients are summed by each lane over all its
// items, then over the CTA's warps, and the CTAs' sums by the next kernel, in the same order each time.
template <int LANES, bool F16, int HEADS>
__global__ void __launch_bounds__(kQkThreads) qk_norm_rope_backward_kernel(const QkNormArgs a) {
  pdl_prologue();
  constexpr int ROWS = 32 / LANES, AT_ONCE = ROWS * HEADS, WARPS = kQkThreads / 32;
  const int warp = threadIdx.x >> 5, sub = (threadIdx.x & 31) / LANES;
  const int parts0 = (a.heads[0] + AT_ONCE - 1) / AT_ONCE, parts = parts0 + (a.heads[1] + AT_ONCE - 1) / AT_ONCE;
  const int64_t items = static_cast<int64_t>(a.tokens) * parts;
  QkLane<LANES> lane(a);
  const float inv_dim = 1.f / a.dim;
  float dw[2][8] = {};
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * WARPS + warp; item < items; item += static_cast<int64_t>(gridDim.x) * WARPS) {
    const int token = static_cast<int>(item / parts), part = static_cast<int>(item - static_cast<int64_t>(token) * parts);
    const int which = part >= parts0, h0 = (which ? part - parts0 : part) * AT_ONCE + sub;
    const int heads = which ? a.heads[1] : a.heads[0];
    const int p = qk_position(a, token);
    const uint16_t* x = (which ? a.x[1] : a.x[0]) + token * (which ? a.xst[1] : a.xst[0]) + lane.col;
    const uint16_t* dy = (which ? a.dy[1] : a.dy[0]) + token * (which ? a.dst[1] : a.dst[0]) + lane.col;
    uint16_t* dx = (which ? a.out[1] : a.out[0]) + token * (which ? a.ost[1] : a.ost[0]) + lane.col;
    const int64_t xsh = which ? a.xsh[1] : a.xsh[0], dsh = which ? a.dsh[1] : a.dsh[0], osh = which ? a.osh[1] : a.osh[0];
    float f[HEADS][8], g[HEADS][8], w[8];
#pragma unroll
    for (int i = 0; i < HEADS; ++i) {
      const bool on = p >= 0 && lane.on && h0 + i * ROWS < heads;
      qk_load8<F16>(f[i], x + (h0 + i * ROWS) * xsh, on);
      qk_load8<F16>(g[i], dy + (h0 + i * ROWS) * dsh, on);
    }
    qk_weights(w, a, which, lane.col, lane.on, F16);
    lane.angles(a, max(p, 0));
#pragma unroll
    for (int i = 0; i < HEADS; ++i) {
      lane.template turn<true>(a, g[i]);
      float sum = 0.f, dot = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        sum = fmaf(f[i][j], f[i][j], sum);
        dot = fmaf(g[i][j] * w[j], f[i][j], dot);
      }
      const float r = rsqrtf(fmaf(qk_sum<LANES>(sum), inv_dim, a.eps));
      const float mean = qk_sum<LANES>(dot) * r * inv_dim;
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float xh = f[i][j] * r, gx = g[i][j] * xh;
        o[j] = r * fmaf(g[i][j], w[j], -xh * mean);
        dw[0][j] += which ? 0.f : gx;
        dw[1][j] += which ? gx : 0.f;
      }
      if (lane.on && h0 + i * ROWS < heads) qk_store8<F16>(dx + (h0 + i * ROWS) * osh, o);
    }
  }
  // the warp's rows, then the CTA's warps
  __shared__ float sums[WARPS][2][8 * LANES];
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
#pragma unroll
      for (int o = LANES; o < 32; o <<= 1) dw[k][j] += __shfl_xor_sync(0xFFFFFFFFu, dw[k][j], o);
      if (sub == 0) sums[warp][k][lane.col + j] = dw[k][j];
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * a.dim; i += kQkThreads) {
    const int k = i >= a.dim, d = k ? i - a.dim : i;
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < WARPS; ++j) sum += sums[j][k][d];
    a.partial[static_cast<int64_t>(blockIdx.x) * 2 * a.dim + i] = sum;
  }
}

// Sums of the CTAs' partial sums: 32 columns a CTA, a stretch of the CTAs a warp.
__global__ void __launch_bounds__(1024) qk_weight_grad_kernel(const float* partial, int ctas, int dim, float* dqw, float* dkw) {
  pdl_prologue();
  __shared__ float sums[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  float sum = 0.f;
  if (col < 2 * dim)
    for (int c = warp; c < ctas; c += 32) sum += partial[static_cast<int64_t>(c) * 2 * dim + col];
  sums[warp][lane] = sum;
  __syncthreads();
  if (warp == 0 && col < 2 * dim) {
    float all = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) all += sums[i][lane];
    (col < dim ? dqw : dkw)[col < dim ? col : col - dim] = all;
  }
}

}  // namespace mxgb
