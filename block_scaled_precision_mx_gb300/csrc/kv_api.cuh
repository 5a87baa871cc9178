// kv_api.cuh -- C ABI entry points of the 8-bit key/value cache (include/mx.h): host-side validation
// and launches.  Included by mx_api.cu.
#pragma once

namespace {

// tokens of a call, of a request and of a window: sums and differences of two stay within 32 bits
constexpr int64_t kKvMostTokens = 1 << 30;

// 2^shift tokens a block, for 16, 32, 64 or 128; -1 otherwise
int kv_block_shift(int block_tokens) {
  return block_tokens == 16 ? 4 : block_tokens == 32 ? 5 : block_tokens == 64 ? 6 : block_tokens == 128 ? 7 : -1;
}

// shared checks of a cache's shape: code offsets within 63 bits, rows of codes within a tensor map's 31
bool kv_cache_shape_ok(int64_t num_blocks, int64_t kv_heads, int block_tokens, int head_dim) {
  if (num_blocks < 1 || kv_heads < 1 || kv_heads > 1024 || kv_block_shift(block_tokens) < 0) return false;
  if (head_dim != 64 && head_dim != 128) return false;
  return num_blocks <= 0x7FFFFFFFll / (kv_heads * block_tokens);
}

// 8-row tiles of the kernel for few rows: 1 or 2; 0 where a kv head has more than 16 rows and the kernel for
// many takes them.  (24 requests, 2048-token windows: 8 rows 30 us, 16 rows 38 us here; 24 to 64 rows 54 to 56 us
// there.  Four row tiles here would hold 32 rows of O in 128 registers a thread: 63 us at best.)
int kv_row_tiles(int64_t max_q_len, int64_t group) {
  if (max_q_len > 16 || group > 16) return max_q_len ? 0 : 1;
  const int64_t rows = max_q_len * group;
  return rows <= 8 ? 1 : rows <= 16 ? 2 : 0;
}

// codes as rows of head_dim bytes; a box is up to 64 tokens of one block and head
bool kv_codes_tmap(CUtensorMap* map, const void* codes, int64_t num_blocks, int64_t kv_heads, int block_tokens,
                   int head_dim) {
  return encode_2d(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, codes, static_cast<uint64_t>(head_dim),
                   static_cast<uint64_t>(num_blocks * kv_heads * block_tokens), static_cast<uint64_t>(head_dim),
                   static_cast<uint32_t>(head_dim), static_cast<uint32_t>(block_tokens < kKvTile ? block_tokens : kKvTile),
                   head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

template <int FMT, int D, int NT, bool TREE>
mx_status kv_few_launch(const KvAttnArgs& a, int block_tokens, int64_t max_q_len, void* workspace, cudaStream_t st) {
  using Cfg = KvFewCfg<D, NT>;
  auto kern = kv_attention_few_kernel<FMT, D, NT, TREE>;
  static std::atomic<int> ctas[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MX_ERR_CUDA;
  int n = ctas[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM) != cudaSuccess)
      return MX_ERR_CUDA;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, kKvFewThreads, Cfg::SMEM) != cudaSuccess || n <= 0)
      return MX_ERR_CUDA;
    const int sms = device_sms();
    if (sms <= 0) return MX_ERR_CUDA;
    n = n * sms < kKvMaxCtas ? n * sms : kKvMaxCtas;
    ctas[dev].store(n, std::memory_order_relaxed);
  }
  CUtensorMap tk, tv;
  if (!kv_codes_tmap(&tk, a.k_codes, a.num_blocks, a.kv_heads, block_tokens, D) ||
      !kv_codes_tmap(&tv, a.v_codes, a.num_blocks, a.kv_heads, block_tokens, D))
    return MX_ERR_CUDA;
  const int most_q = static_cast<int>(max_q_len);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  if (pdl_launch(kern, n, kKvFewThreads, Cfg::SMEM, st, tk, tv, a, most_q, ws) != cudaSuccess) return MX_ERR_CUDA;
  return launch_status();
}

template <int FMT, int D, bool F16, bool TREE, bool ONE>
mx_status kv_many_launch(const KvAttnArgs& a, int block_tokens, int64_t max_q_len, void* workspace, cudaStream_t st) {
  using Cfg = KvManyCfg<D, TREE, ONE>;
  auto kern = kv_attention_many_kernel<FMT, D, F16, TREE, ONE>;
  static std::atomic<bool> attr_set[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MX_ERR_CUDA;
  if (!attr_set[dev].load(std::memory_order_relaxed)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM) != cudaSuccess)
      return MX_ERR_CUDA;
    attr_set[dev].store(true, std::memory_order_relaxed);
  }
  const int sms = device_sms();
  if (sms <= 0) return MX_ERR_CUDA;
  const int n = sms < kKvManyMaxCtas ? sms : kKvManyMaxCtas;
  CUtensorMap tk, tv;
  if (!kv_codes_tmap(&tk, a.k_codes, a.num_blocks, a.kv_heads, block_tokens, D) ||
      !kv_codes_tmap(&tv, a.v_codes, a.num_blocks, a.kv_heads, block_tokens, D))
    return MX_ERR_CUDA;
  const int most_q = static_cast<int>(max_q_len);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  // up to a request a thread, of up to 32 units, the kernel plans for itself
  const int planned = a.requests > kKvManyThreads || max_q_len * (a.heads / a.kv_heads) > 32 * kKvManyRows;
  if (planned && pdl_launch(kv_plan_kernel<TREE>, 1, kKvPlanThreads, 0, st, a, most_q, n, ws) != cudaSuccess) return MX_ERR_CUDA;
  if (pdl_launch(kern, n, kKvManyThreads, Cfg::SMEM, st, tk, tv, a, most_q, planned, ws) != cudaSuccess)
    return MX_ERR_CUDA;
  if (n > 1 && pdl_launch(kv_join_kernel<D>, dim3(n - 1, 16), 128, 0, st, a, static_cast<const uint8_t*>(ws),
                          kv_many_slots_at(a.requests, D)) != cudaSuccess)
    return MX_ERR_CUDA;
  return launch_status();
}

template <int FMT, int D, bool TREE>
mx_status kv_attention_launch(const KvAttnArgs& a, int block_tokens, int64_t max_q_len, void* workspace, cudaStream_t st) {
  switch (kv_row_tiles(max_q_len, a.heads / a.kv_heads)) {
    case 1: return kv_few_launch<FMT, D, 1, TREE>(a, block_tokens, max_q_len, workspace, st);
    case 2: return kv_few_launch<FMT, D, 2, TREE>(a, block_tokens, max_q_len, workspace, st);
  }
  if constexpr (TREE && D == 128)  // (D = 64 has room for its buffers in either case)
    if (max_q_len * (a.heads / a.kv_heads) <= 128)
      return a.f16 ? kv_many_launch<FMT, D, true, TREE, true>(a, block_tokens, max_q_len, workspace, st)
                   : kv_many_launch<FMT, D, false, TREE, true>(a, block_tokens, max_q_len, workspace, st);
  return a.f16 ? kv_many_launch<FMT, D, true, TREE, false>(a, block_tokens, max_q_len, workspace, st)
               : kv_many_launch<FMT, D, false, TREE, false>(a, block_tokens, max_q_len, workspace, st);
}

// A group of W warps holds a block's values of one head, 4 words of 8 a thread, or 8 where 8 warps would
// not do otherwise.
template <int FMT, bool F16>
cudaError_t kv_append_launch(const KvAppendArgs& a, int head_dim, dim3 grid, cudaStream_t st) {
#define KV_APPEND(D, W, PASSES) pdl_launch(kv_append_kernel<FMT, F16, D, W, PASSES>, grid, kKvAppendThreads, 0, st, a)
  if (head_dim == 64)
    return a.shift == 4 ? KV_APPEND(64, 1, 4) : a.shift == 5 ? KV_APPEND(64, 2, 4) : a.shift == 6 ? KV_APPEND(64, 4, 4)
                                                                                                  : KV_APPEND(64, 8, 4);
  return a.shift == 4 ? KV_APPEND(128, 2, 4) : a.shift == 5 ? KV_APPEND(128, 4, 4) : a.shift == 6 ? KV_APPEND(128, 8, 4)
                                                                                                  : KV_APPEND(128, 8, 8);
#undef KV_APPEND
}

std::mutex kv_turn;

// kv_attention and, with a mask, kv_tree_attention
template <bool TREE>
mx_status kv_attention_call(const void* q, mx_half type, int64_t num_tokens, int64_t heads, int64_t q_stride_token,
                       int64_t q_stride_head, const void* k_codes, const void* v_codes, const float* k_scale,
                       const float* v_scale, mx_elem elem, int64_t num_blocks, int64_t kv_heads, int block_tokens,
                       int head_dim, const int32_t* block_tables, int64_t max_blocks, const int32_t* lengths,
                       const int32_t* q_start, int64_t requests, int64_t max_q_len, const int64_t* tree_mask,
                       int64_t mask_words, const int32_t* positions, float softmax_scale, int causal, int64_t window,
                       void* out, float* lse, void* workspace, void* stream) {
  if (num_tokens < 0 || num_tokens > kKvMostTokens || requests < 1 || requests > kKvMaxRequests)
    return MX_ERR_INVALID_ARG;
  if (!k_codes || !v_codes || !k_scale || !v_scale || !block_tables || !lengths || !q_start || !workspace ||
      (num_tokens && (!q || !out || !lse)))
    return MX_ERR_INVALID_ARG;
  if (type != MX_HALF_BF16 && type != MX_HALF_F16) return MX_ERR_INVALID_ARG;
  if (elem != MX_E4M3 && elem != MX_E5M2) return elem == MX_E2M1 ? MX_ERR_UNSUPPORTED : MX_ERR_INVALID_ARG;
  if (!kv_cache_shape_ok(num_blocks, kv_heads, block_tokens, head_dim)) return MX_ERR_INVALID_ARG;
  if (heads < 1 || heads > 65535 || heads % kv_heads) return MX_ERR_INVALID_ARG;
  if (max_blocks < 1 || max_blocks > kKvMostTokens / block_tokens) return MX_ERR_INVALID_ARG;
  if (num_tokens > kKvMostTokens / (heads / kv_heads)) return MX_ERR_INVALID_ARG;  // (rows of a kv head)
  if (max_q_len < 0 || max_q_len > num_tokens || window < 0 || window > 0x7FFFFFFF) return MX_ERR_INVALID_ARG;
  if (causal != 0 && causal != 1) return MX_ERR_INVALID_ARG;
  if (!(softmax_scale > 0.f) || softmax_scale > 1e30f) return MX_ERR_INVALID_ARG;
  if (q_stride_token % 8 || q_stride_head % 8) return MX_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_codes, 16) || !aligned(v_codes, 16) || !aligned(k_scale, 4) ||
      !aligned(v_scale, 4) || !aligned(block_tables, 4) || !aligned(lengths, 4) || !aligned(q_start, 4) ||
      !aligned(out, 32) || !aligned(lse, 4) || !aligned(workspace, 32))
    return MX_ERR_INVALID_ARG;
  if (TREE) {
    if (max_q_len > kKvMostNodes || mask_words < 1 || mask_words > kKvMostNodes / 64 || mask_words * 64 < max_q_len ||
        !aligned(tree_mask, 8) || !aligned(positions, 4) || (num_tokens && (!tree_mask || (window && !positions))))
      return MX_ERR_INVALID_ARG;
  }
  if (num_tokens == 0) return MX_OK;
  KvAttnArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.stride_t = q_stride_token;
  a.stride_h = q_stride_head;
  a.k_codes = static_cast<const uint8_t*>(k_codes);
  a.v_codes = static_cast<const uint8_t*>(v_codes);
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.tables = block_tables;
  a.lengths = lengths;
  a.q_start = q_start;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.scale_log2 = static_cast<float>(static_cast<double>(softmax_scale) * 1.4426950408889634);
  a.num_blocks = num_blocks;
  a.tokens = static_cast<int>(num_tokens);
  a.heads = static_cast<int>(heads);
  a.kv_heads = static_cast<int>(kv_heads);
  a.requests = static_cast<int>(requests);
  a.max_blocks = static_cast<int>(max_blocks);
  a.shift = kv_block_shift(block_tokens);
  a.causal = causal;
  a.f16 = type == MX_HALF_F16;
  a.window = static_cast<int>(window < kKvMostTokens ? window : kKvMostTokens);
  a.tree_mask = reinterpret_cast<const uint64_t*>(tree_mask);
  a.positions = positions;
  a.tree_words = static_cast<int>(mask_words);
  cudaStream_t st = as_stream(stream);
  // A call's launches speak to each other through the workspace.  Host threads that share a stream, and with it a
  // workspace, take turns, so that no other call's launch comes between them.
  const std::lock_guard<std::mutex> hold(kv_turn);
  if (elem == MX_E5M2)
    return head_dim == 64 ? kv_attention_launch<1, 64, TREE>(a, block_tokens, max_q_len, workspace, st)
                          : kv_attention_launch<1, 128, TREE>(a, block_tokens, max_q_len, workspace, st);
  return head_dim == 64 ? kv_attention_launch<0, 64, TREE>(a, block_tokens, max_q_len, workspace, st)
                        : kv_attention_launch<0, 128, TREE>(a, block_tokens, max_q_len, workspace, st);
}

}  // namespace

extern "C" {

mx_status kv_block_tables(int32_t* block_tables, int64_t requests, int64_t max_blocks, const int32_t* len_before,
                          const int32_t* len_after, int32_t* free_list, int64_t free_capacity,
                          const int32_t* free_count, int block_tokens, int64_t num_tokens, int32_t* q_start,
                          int64_t* slot_map, int32_t* positions, int32_t* info, void* stream) {
  const int shift = kv_block_shift(block_tokens);
  if (!block_tables || !len_before || !len_after || !free_list || !free_count || !q_start || !info || shift < 0)
    return MX_ERR_INVALID_ARG;
  if (num_tokens < 0 || num_tokens > kKvMostTokens || (num_tokens && (!slot_map || !positions)))
    return MX_ERR_INVALID_ARG;
  if (requests < 1 || requests > kKvMaxRequests || max_blocks < 1 || max_blocks > (kKvMostTokens >> shift) ||
      free_capacity < 1 || free_capacity > 0x7FFFFFFF)
    return MX_ERR_INVALID_ARG;
  if (!aligned(block_tables, 4) || !aligned(len_before, 4) || !aligned(len_after, 4) || !aligned(free_list, 4) ||
      !aligned(free_count, 4) || !aligned(q_start, 4) || !aligned(slot_map, 8) || !aligned(positions, 4) ||
      !aligned(info, 4))
    return MX_ERR_INVALID_ARG;
  static std::atomic<bool> attr_set[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MX_ERR_CUDA;
  if (!attr_set[dev].load(std::memory_order_relaxed)) {
    if (cudaFuncSetAttribute(kv_block_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             3 * 4 * (kKvMaxRequests + 1)) != cudaSuccess)
      return MX_ERR_CUDA;
    attr_set[dev].store(true, std::memory_order_relaxed);
  }
  KvTablesArgs a{};
  a.tables = block_tables;
  a.before = len_before;
  a.after = len_after;
  a.free_list = free_list;
  a.free_count = free_count;
  a.q_start = q_start;
  a.slots = slot_map;
  a.positions = positions;
  a.info = info;
  a.requests = static_cast<int>(requests);
  a.max_blocks = static_cast<int>(max_blocks);
  a.capacity = static_cast<int>(free_capacity);
  a.num_tokens = static_cast<int>(num_tokens);
  a.shift = shift;
  a.wide = aligned(slot_map, 16) && aligned(positions, 16);
  // four tokens a thread, up to about two CTAs a SM; every CTA scans the requests for itself
  const int64_t want = (num_tokens + 4 * kKvTablesThreads - 1) / (4 * kKvTablesThreads);
  const unsigned grid = static_cast<unsigned>(want < 1 ? 1 : want > 304 ? 304 : want);
  if (pdl_launch(kv_block_tables_kernel, grid, kKvTablesThreads, 3 * 4 * (static_cast<size_t>(requests) + 1),
                 as_stream(stream), a) != cudaSuccess)
    return MX_ERR_CUDA;
  return launch_status();
}

mx_status kv_cache_append(const void* k, const void* v, mx_half type, int64_t num_tokens, int64_t k_stride_token,
                          int64_t k_stride_head, int64_t v_stride_token, int64_t v_stride_head,
                          const int64_t* slot_map, void* k_codes, void* v_codes, float* k_scale, float* v_scale,
                          mx_elem elem, int64_t num_blocks, int64_t kv_heads, int block_tokens, int head_dim,
                          void* stream) {
  if (num_tokens < 0 || num_tokens > kKvMostTokens) return MX_ERR_INVALID_ARG;
  if (!k_codes || !v_codes || !k_scale || !v_scale || (num_tokens && (!k || !v || !slot_map))) return MX_ERR_INVALID_ARG;
  if (type != MX_HALF_BF16 && type != MX_HALF_F16) return MX_ERR_INVALID_ARG;
  if (elem != MX_E4M3 && elem != MX_E5M2) return elem == MX_E2M1 ? MX_ERR_UNSUPPORTED : MX_ERR_INVALID_ARG;
  if (!kv_cache_shape_ok(num_blocks, kv_heads, block_tokens, head_dim)) return MX_ERR_INVALID_ARG;
  if (k_stride_token % 8 || k_stride_head % 8 || v_stride_token % 8 || v_stride_head % 8) return MX_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slot_map, 8) || !aligned(k_codes, 16) || !aligned(v_codes, 16) ||
      !aligned(k_scale, 4) || !aligned(v_scale, 4))
    return MX_ERR_INVALID_ARG;
  if (num_tokens == 0) return MX_OK;
  KvAppendArgs a{};
  a.x[0] = static_cast<const uint16_t*>(k);
  a.x[1] = static_cast<const uint16_t*>(v);
  a.stride_t[0] = k_stride_token;
  a.stride_t[1] = v_stride_token;
  a.stride_h[0] = k_stride_head;
  a.stride_h[1] = v_stride_head;
  a.codes[0] = static_cast<uint8_t*>(k_codes);
  a.codes[1] = static_cast<uint8_t*>(v_codes);
  a.scale[0] = k_scale;
  a.scale[1] = v_scale;
  a.slots = slot_map;
  a.num_slots = num_blocks * block_tokens;
  a.tokens = static_cast<int>(num_tokens);
  a.kv_heads = static_cast<int>(kv_heads);
  a.shift = kv_block_shift(block_tokens);
  const int64_t warps = static_cast<int64_t>(block_tokens) * head_dim / 1024;
  const int groups = warps >= 8 ? 1 : static_cast<int>(8 / warps);
  const int64_t gy = (2 * kv_heads + groups - 1) / groups;
  // Tokens looked over by a CTA: a power of two that leaves about 2048 CTAs, at most a block's tokens.
  int chunk = 1;
  while (chunk < block_tokens && num_tokens * gy > 2048ll * chunk) chunk *= 2;
  a.chunk = chunk;
  const dim3 grid(static_cast<unsigned>((num_tokens + chunk - 1) / chunk), static_cast<unsigned>(gy));
  cudaStream_t st = as_stream(stream);
  const bool f16 = type == MX_HALF_F16;
  const cudaError_t e = elem == MX_E4M3
                            ? (f16 ? kv_append_launch<0, true>(a, head_dim, grid, st) : kv_append_launch<0, false>(a, head_dim, grid, st))
                            : (f16 ? kv_append_launch<1, true>(a, head_dim, grid, st) : kv_append_launch<1, false>(a, head_dim, grid, st));
  if (e != cudaSuccess) return MX_ERR_CUDA;
  return launch_status();
}

size_t kv_attention_workspace_bytes(int64_t num_tokens, int64_t requests, int64_t max_q_len, int64_t heads,
                                    int64_t kv_heads, int head_dim) {
  if (num_tokens < 0 || requests < 1 || max_q_len < 0 || heads < 1 || kv_heads < 1 || heads % kv_heads) return 0;
  if (head_dim != 64 && head_dim != 128) return 0;
  const int nt = kv_row_tiles(max_q_len, heads / kv_heads);
  if (!nt)
    return kv_many_slots_at(requests, head_dim) + 2ull * kKvManyMaxCtas * kKvManyRows * (head_dim + 2) * 4;
  return kKvSlotsAt + 2ull * kKvMaxCtas * (8 * nt) * (head_dim + 2) * 4;
}

mx_status kv_attention(const void* q, mx_half type, int64_t num_tokens, int64_t heads, int64_t q_stride_token,
                       int64_t q_stride_head, const void* k_codes, const void* v_codes, const float* k_scale,
                       const float* v_scale, mx_elem elem, int64_t num_blocks, int64_t kv_heads, int block_tokens,
                       int head_dim, const int32_t* block_tables, int64_t max_blocks, const int32_t* lengths,
                       const int32_t* q_start, int64_t requests, int64_t max_q_len, float softmax_scale, int causal,
                       int64_t window, void* out, float* lse, void* workspace, void* stream) {
  return kv_attention_call<false>(q, type, num_tokens, heads, q_stride_token, q_stride_head, k_codes, v_codes, k_scale, v_scale,
                                  elem, num_blocks, kv_heads, block_tokens, head_dim, block_tables, max_blocks, lengths, q_start,
                                  requests, max_q_len, nullptr, 0, nullptr, softmax_scale, causal, window, out, lse, workspace,
                                  stream);
}

mx_status kv_tree_attention(const void* q, mx_half type, int64_t num_tokens, int64_t heads, int64_t q_stride_token,
                            int64_t q_stride_head, const void* k_codes, const void* v_codes, const float* k_scale,
                            const float* v_scale, mx_elem elem, int64_t num_blocks, int64_t kv_heads, int block_tokens,
                            int head_dim, const int32_t* block_tables, int64_t max_blocks, const int32_t* lengths,
                            const int32_t* q_start, int64_t requests, int64_t max_q_len, const int64_t* tree_mask,
                            int64_t mask_words, const int32_t* positions, float softmax_scale, int64_t window, void* out,
                            float* lse, void* workspace, void* stream) {
  return kv_attention_call<true>(q, type, num_tokens, heads, q_stride_token, q_stride_head, k_codes, v_codes, k_scale, v_scale,
                                 elem, num_blocks, kv_heads, block_tokens, head_dim, block_tables, max_blocks, lengths, q_start,
                                 requests, max_q_len, tree_mask, mask_words, positions, softmax_scale, 0, window, out, lse,
                                 workspace, stream);
}

}  // extern "C"
