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

template <bool F16>
__device__ __forceinline__ uint32_t kv_pack2(float lo, float hi) {
  if (F16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

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

// A lane has eight values of a head's row, four at `at[0]` and four at `at[1]`, so chosen that what a rotation turns
// together is in one lane: with pairs (i, rot / 2 + i) four from each half, else eight in a row.  (Eight in a row for both,
// with a shuffle for each value: 16384 tokens of 40 heads 120 us.)
template <int LANES, bool INTER>
struct QkLane {
  int at[2];
  float c[4], s[4];  // cosines and sines: of (i, 4 + i) of its values, or of (2i, 2i + 1)
  int turn_at;
  bool on, turns;

  __device__ __forceinline__ QkLane(const QkNormArgs& a) {
    const int l = threadIdx.x % LANES;
    on = 8 * l < a.dim;
    turns = 8 * l < a.rot;
    turn_at = 4 * l;
    at[0] = !INTER && turns ? 4 * l : 8 * l;
    at[1] = !INTER && turns ? a.rot / 2 + 4 * l : 8 * l + 4;
  }
  __device__ __forceinline__ void load(uint2 (&v)[2], const uint16_t* row, bool live) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) v[i] = on && live ? *reinterpret_cast<const uint2*>(row + at[i]) : make_uint2(0, 0);
  }
  template <bool F16>
  __device__ __forceinline__ void store(uint16_t* row, const float (&f)[8], bool live) const {
    if (!on || !live) return;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      *reinterpret_cast<uint2*>(row + at[i]) =
          make_uint2(kv_pack2<F16>(f[4 * i], f[4 * i + 1]), kv_pack2<F16>(f[4 * i + 2], f[4 * i + 3]));
  }
  template <bool F16>
  __device__ __forceinline__ void weights(float (&w)[8], const QkNormArgs& a, int which) const {
    const void* from = which ? a.weight[1] : a.weight[0];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (on && a.weight_f32) {
        v = *reinterpret_cast<const float4*>(static_cast<const float*>(from) + at[i]);
      } else if (on) {
        const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(from) + at[i]);
        const float2 lo = kv_unpack2<F16>(u.x), hi = kv_unpack2<F16>(u.y);
        v = make_float4(lo.x, lo.y, hi.x, hi.y);
      }
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
  }
  __device__ __forceinline__ void angles(const QkNormArgs& a, int p) {
    float4 cc = make_float4(1.f, 1.f, 1.f, 1.f), ss = make_float4(0.f, 0.f, 0.f, 0.f);
    if (turns) {
      const float* row = a.table + static_cast<int64_t>(p) * a.rot + turn_at;
      cc = *reinterpret_cast<const float4*>(row);
      ss = *reinterpret_cast<const float4*>(row + a.rot / 2);
    }
    c[0] = cc.x, c[1] = cc.y, c[2] = cc.z, c[3] = cc.w;
    s[0] = ss.x, s[1] = ss.y, s[2] = ss.z, s[3] = ss.w;
  }
  // f turned (BACK: turned back)
  template <bool BACK>
  __device__ __forceinline__ void turn(float (&f)[8]) const {
    if (!turns) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float& x = f[INTER ? 2 * i : i];
      float& y = f[INTER ? 2 * i + 1 : 4 + i];
      const float sn = BACK ? -s[i] : s[i], u = x;
      x = fmaf(-sn, y, u * c[i]);
      y = fmaf(sn, u, y * c[i]);
    }
  }
};
template <bool F16>
__device__ __forceinline__ void qk_unpack8(float (&f)[8], const uint2 (&v)[2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 lo = kv_unpack2<F16>(v[i].x), hi = kv_unpack2<F16>(v[i].y);
    f[4 * i] = lo.x, f[4 * i + 1] = lo.y, f[4 * i + 2] = hi.x, f[4 * i + 3] = hi.y;
  }
}
template <int LANES>
__device__ __forceinline__ float qk_sum(float x) {
#pragma unroll
  for (int o = LANES / 2; o; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
  return x;
}

// The token's position; -1: it is left out.  Others out of range are told.
__device__ __forceinline__ int qk_position(const QkNormArgs& a, int token) {
  if (!a.positions) return 0;
  const int p = a.positions[token];
  if (p >= 0 && (!a.table || p < a.most_pos)) return p;
  if (p != -1) atomicOr(&g_mx_error_word, kSiteBadCache);
  return -1;
}

// LANES lanes have a head's row; a warp takes HEADS * 32 / LANES heads of a token's queries or of its keys at a time, and
// the next ones' rows are on their way while it works on these.  Memory is the bound: 16384 tokens of 40 heads of 128
// 63.7 us, 5.4 TB/s, 0.80 of the measured copy rate.  (Three CTAs a SM, 85 registers: two 71 us, four 73; without the rows
// ahead, a warp an item, 76; two heads at a time 74 to 89, eight 70 to 83.)
template <int LANES, bool F16, bool INTER, int HEADS>
__global__ void __launch_bounds__(kQkThreads, 3) qk_norm_rope_kernel(const QkNormArgs a) {
  pdl_prologue();
  constexpr int ROWS = 32 / LANES, AT_ONCE = ROWS * HEADS;
  const int sub = (threadIdx.x & 31) / LANES;
  const int parts0 = (a.heads[0] + AT_ONCE - 1) / AT_ONCE, parts = parts0 + (a.heads[1] + AT_ONCE - 1) / AT_ONCE;
  QkLane<LANES, INTER> lane(a);
  const float inv_dim = 1.f / a.dim;
  const uint32_t items = static_cast<uint32_t>(a.tokens) * parts, step = gridDim.x * (kQkThreads / 32);
  uint2 v[HEADS][2];
  int p = -1, token = 0, which = 0, h0 = 0;
  auto fetch = [&](uint32_t item) {
    if (item >= items) return;
    token = item / static_cast<uint32_t>(parts);
    const int part = item - static_cast<uint32_t>(token) * parts;
    which = part >= parts0;
    h0 = (which ? part - parts0 : part) * AT_ONCE + sub;
    const uint16_t* x = (which ? a.x[1] : a.x[0]) + token * (which ? a.xst[1] : a.xst[0]);
    const int64_t xsh = which ? a.xsh[1] : a.xsh[0];
    const int heads = which ? a.heads[1] : a.heads[0];
#pragma unroll
    for (int i = 0; i < HEADS; ++i) lane.load(v[i], x + (h0 + i * ROWS) * xsh, h0 + i * ROWS < heads);
    p = qk_position(a, token);
  };
  uint32_t item = blockIdx.x * (kQkThreads / 32) + (threadIdx.x >> 5);
  fetch(item);
  for (; item < items; item += step) {
    uint2 u[HEADS][2];
#pragma unroll
    for (int i = 0; i < HEADS; ++i) u[i][0] = v[i][0], u[i][1] = v[i][1];
    const int at = p, heads = which ? a.heads[1] : a.heads[0], first = h0, w_of = which;
    uint16_t* y = (which ? a.out[1] : a.out[0]) + token * (which ? a.ost[1] : a.ost[0]);
    const int64_t osh = which ? a.osh[1] : a.osh[0];
    if (at >= 0) lane.angles(a, at);
    fetch(item + step);
    if (at < 0) continue;
    float w[8];
    lane.template weights<F16>(w, a, w_of);
#pragma unroll
    for (int i = 0; i < HEADS; ++i) {
      float f[8], sum = 0.f;
      qk_unpack8<F16>(f, u[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fmaf(f[j], f[j], sum);
      const float r = rsqrtf(fmaf(qk_sum<LANES>(sum), inv_dim, a.eps));
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] *= r * w[j];
      lane.template turn<false>(f);
      lane.template store<F16>(y + (first + i * ROWS) * osh, f, first + i * ROWS < heads);
    }
  }
}

// For few heads, whose items above would be half empty: HEADS * 32 / LANES rows in a row, of whatever tokens.  The angles
// are each row's own then.
template <int LANES, bool F16, bool INTER, int HEADS>
__global__ void __launch_bounds__(kQkThreads, 3) qk_norm_rope_rows_kernel(const QkNormArgs a) {
  pdl_prologue();
  constexpr int ROWS = 32 / LANES, AT_ONCE = ROWS * HEADS;
  const int sub = (threadIdx.x & 31) / LANES;
  QkLane<LANES, INTER> lane(a);
  const float inv_dim = 1.f / a.dim;
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    const uint32_t heads = which ? a.heads[1] : a.heads[0], rows = a.tokens * heads;
    const uint16_t* x = which ? a.x[1] : a.x[0];
    uint16_t* y = which ? a.out[1] : a.out[0];
    const int64_t xst = which ? a.xst[1] : a.xst[0], xsh = which ? a.xsh[1] : a.xsh[0];
    const int64_t ost = which ? a.ost[1] : a.ost[0], osh = which ? a.osh[1] : a.osh[0];
    float w[8];
    if (rows) lane.template weights<F16>(w, a, which);
    for (uint32_t row0 = (blockIdx.x * (kQkThreads / 32) + (threadIdx.x >> 5)) * AT_ONCE; row0 < rows;
         row0 += gridDim.x * (kQkThreads / 32) * AT_ONCE) {
      uint2 v[HEADS][2];
      int p[HEADS];
#pragma unroll
      for (int i = 0; i < HEADS; ++i) {
        const uint32_t row = row0 + sub + i * ROWS, token = row / heads, h = row - token * heads;
        lane.load(v[i], x + token * xst + h * xsh, row < rows);
        p[i] = row < rows ? qk_position(a, token) : -1;
      }
#pragma unroll
      for (int i = 0; i < HEADS; ++i) {
        const uint32_t row = row0 + sub + i * ROWS, token = row / heads, h = row - token * heads;
        lane.angles(a, max(p[i], 0));
        float f[8], sum = 0.f;
        qk_unpack8<F16>(f, v[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = fmaf(f[j], f[j], sum);
        const float r = rsqrtf(fmaf(qk_sum<LANES>(sum), inv_dim, a.eps));
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] *= r * w[j];
        lane.template turn<false>(f);
        lane.template store<F16>(y + token * ost + h * osh, f, p[i] >= 0);
      }
    }
  }
}

// The queries' items, then the keys', warp after warp of a grid of a fixed size; the weights' gradients are summed by
// each lane over its items, then over the CTA's warps, and the CTAs' sums by the next kernel, in the same order each time.
// 8191 tokens of 48 heads of 64: 37 us with that kernel, 4.1 TB/s; a lane's two loads a head, the turn and two sums over
// the lanes, one behind the other, keep it from more.  (Two CTAs a SM, four heads at a time; one head 45, two 45; with the
// next rows ahead, which then cost registers that the heads had, 41 to 49.)
// FLAT: items are rows in a row, as for few heads above.
template <int LANES, bool F16, bool INTER, int HEADS, bool FLAT>
__global__ void __launch_bounds__(kQkThreads, 2) qk_norm_rope_backward_kernel(const QkNormArgs a) {
  pdl_prologue();
  constexpr int ROWS = 32 / LANES, AT_ONCE = ROWS * HEADS, WARPS = kQkThreads / 32;
  __shared__ float sums[WARPS][2][8 * LANES];
  const int warp = threadIdx.x >> 5, sub = (threadIdx.x & 31) / LANES;
  QkLane<LANES, INTER> lane(a);
  const float inv_dim = 1.f / a.dim;
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    const uint32_t heads = which ? a.heads[1] : a.heads[0], parts = (heads + AT_ONCE - 1) / AT_ONCE, rows = a.tokens * heads;
    const uint32_t items = FLAT ? (rows + AT_ONCE - 1) / AT_ONCE : a.tokens * parts;
    const int64_t xst = which ? a.xst[1] : a.xst[0], dst = which ? a.dst[1] : a.dst[0], ost = which ? a.ost[1] : a.ost[0];
    const int64_t xsh = which ? a.xsh[1] : a.xsh[0], dsh = which ? a.dsh[1] : a.dsh[0], osh = which ? a.osh[1] : a.osh[0];
    const uint16_t* x = which ? a.x[1] : a.x[0];
    const uint16_t* dy = which ? a.dy[1] : a.dy[0];
    uint16_t* dx = which ? a.out[1] : a.out[0];
    float w[8], dw[8] = {};
    if (items) lane.template weights<F16>(w, a, which);
    for (uint32_t item = blockIdx.x * WARPS + warp; item < items; item += gridDim.x * WARPS) {
      const uint32_t whole = FLAT ? 0 : item / parts, h0 = FLAT ? 0 : (item - whole * parts) * AT_ONCE + sub;
      uint2 v[HEADS][2], u[HEADS][2];
      int p[FLAT ? HEADS : 1];
      auto place = [&](int i, uint32_t& token, uint32_t& h) {  // row i of the item; whether there is one
        const uint32_t row = item * AT_ONCE + sub + i * ROWS;
        token = FLAT ? row / heads : whole;
        h = FLAT ? row - token * heads : h0 + i * ROWS;
        return FLAT ? row < rows : h < heads;
      };
      if (!FLAT) p[0] = qk_position(a, whole);
#pragma unroll
      for (int i = 0; i < HEADS; ++i) {
        uint32_t token, h;
        const bool live = place(i, token, h);
        lane.load(v[i], x + token * xst + h * xsh, live);
        lane.load(u[i], dy + token * dst + h * dsh, live);
        if (FLAT) p[FLAT ? i : 0] = live ? qk_position(a, token) : -1;
      }
      if (!FLAT) lane.angles(a, max(p[0], 0));
#pragma unroll
      for (int i = 0; i < HEADS; ++i) {
        uint32_t token, h;
        const bool live = place(i, token, h);
        const int at = p[FLAT ? i : 0];
        if (FLAT) lane.angles(a, max(at, 0));
        float f[8], g[8], sum = 0.f, dot = 0.f;
        qk_unpack8<F16>(f, v[i]);
        qk_unpack8<F16>(g, u[i]);
        lane.template turn<true>(g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          sum = fmaf(f[j], f[j], sum);
          dot = fmaf(g[j] * w[j], f[j], dot);
        }
        const float r = rsqrtf(fmaf(qk_sum<LANES>(sum), inv_dim, a.eps));
        const float mean = qk_sum<LANES>(dot) * r * inv_dim;
        float o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float xh = f[j] * r;
          o[j] = at < 0 ? 0.f : r * fmaf(g[j], w[j], -xh * mean);
          if (at >= 0 && live) dw[j] = fmaf(g[j], xh, dw[j]);
        }
        lane.template store<F16>(dx + token * ost + h * osh, o, live);
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
#pragma unroll
      for (int o = LANES; o < 32; o <<= 1) dw[j] += __shfl_xor_sync(0xFFFFFFFFu, dw[j], o);
      if (sub == 0 && lane.on) sums[warp][which][lane.at[j / 4] + j % 4] = dw[j];
    }
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
