// kv_drafts_api.cuh -- C ABI entry points for drafted tokens beside the 8-bit key/value cache, and for the norm and
// rotation in front of it (include/mx.h): host-side validation and launches.  Included by mx_api.cu.
#pragma once

namespace {

// whether an output shares bytes with an input or with another output: some CTA may still read what another writes
bool kv_overlap(std::initializer_list<Span> outputs, std::initializer_list<Span> inputs) {
  for (const Span* a = outputs.begin(); a != outputs.end(); ++a) {
    for (const Span& b : inputs)
      if (spans_meet(*a, b)) return true;
    for (const Span* b = outputs.begin(); b != a; ++b)
      if (spans_meet(*a, *b)) return true;
  }
  return false;
}

// starts of up to kKvMaxRequests requests of up to kKvMostNodes rows each
bool kv_drafts_ok(const int32_t* q_start, int64_t requests, int64_t num_tokens, int64_t max_q_len) {
  return q_start && aligned(q_start, 4) && requests >= 1 && requests <= kKvMaxRequests && num_tokens >= 0 &&
         num_tokens <= kKvMostTokens && max_q_len >= 0 && max_q_len <= kKvMostNodes && max_q_len <= num_tokens;
}

// ------------------------------------------------------------------ norm and rotation
constexpr int kQkCtas = 456, kQkBackCtas = 304;  // three and two a SM

// What the two passes share: shapes, types, table, positions.  Rows' addresses and strides by qk_rows_ok.
bool qk_norm_ok(mx_half type, int64_t num_tokens, int64_t heads, int64_t kv_heads, int head_dim, const void* q_weight,
                const void* k_weight, int weight_f32, const float* cos_sin, int64_t max_positions, int rot_dim,
                const int32_t* positions, float eps, int interleaved) {
  if (type != MX_HALF_BF16 && type != MX_HALF_F16) return false;
  if (num_tokens < 0 || num_tokens > kKvMostTokens || heads < 1 || heads > 65535 || kv_heads < 0 || kv_heads > 65535)
    return false;
  if (num_tokens * (heads + kv_heads) > 0x7FFFFFFF) return false;
  if (head_dim < 8 || head_dim > 256 || head_dim % 8) return false;
  if (!q_weight || (kv_heads && !k_weight) || (weight_f32 != 0 && weight_f32 != 1)) return false;
  if (!aligned(q_weight, 16) || !aligned(k_weight, 16)) return false;
  if (rot_dim < 0 || rot_dim > head_dim || rot_dim % 16 || (interleaved != 0 && interleaved != 1)) return false;
  if (rot_dim && (!cos_sin || !aligned(cos_sin, 16) || !positions || max_positions < 1 || max_positions > kKvMostTokens))
    return false;
  if (!aligned(positions, 4)) return false;
  return eps >= 0.f && eps <= 1.f;  // (and no NaN)
}
bool qk_rows_ok(const void* x, int64_t tokens, int64_t heads, int64_t st, int64_t sh) {
  return tokens == 0 || heads == 0 || (x && aligned(x, 16) && st % 8 == 0 && sh % 8 == 0);
}
// Rows of 16-bit values: queries, keys, their results or gradients.
struct QkRows {
  const void* at;
  int64_t heads, st, sh;
};
// Outputs i = 0, 1 (queries, keys) may be their own inputs, which the same lanes read in front of that; else no output
// shares bytes with an input or another output, nor its rows with each other.
bool qk_apart(int64_t tokens, int head_dim, const QkRows (&out)[2], std::initializer_list<QkRows> in0, std::initializer_list<QkRows> in1,
              std::initializer_list<Span> more_out, std::initializer_list<Span> more_in) {
  auto rows = [&](const QkRows& r) { return span(r.at, 2 * head_dim, tokens, 2 * r.st, r.heads, 2 * r.sh); };
  auto same = [&](const QkRows& a, const QkRows& b) {
    return a.at == b.at && (tokens == 1 || a.st == b.st) && (a.heads == 1 || a.sh == b.sh);
  };
  const Span spans[2] = {rows(out[0]), rows(out[1])};
  for (int i = 0; i < 2; ++i) {
    if (spans[i].n[0] == 0) continue;
    if (!rows_apart(2 * head_dim, tokens, 2 * out[i].st, out[i].heads, 2 * out[i].sh)) return false;
    for (const QkRows& r : in0)
      if ((i || !same(out[i], r)) && spans_meet(spans[i], rows(r))) return false;
    for (const QkRows& r : in1)
      if ((!i || !same(out[i], r)) && spans_meet(spans[i], rows(r))) return false;
    for (const Span& x : more_in)
      if (spans_meet(spans[i], x)) return false;
    for (const Span& x : more_out)
      if (spans_meet(spans[i], x)) return false;
  }
  for (const Span& o : more_out) {
    for (const QkRows& r : in0)
      if (spans_meet(o, rows(r))) return false;
    for (const QkRows& r : in1)
      if (spans_meet(o, rows(r))) return false;
  }
  return !spans_meet(spans[0], spans[1]) && !kv_overlap(more_out, more_in);
}
template <bool BACK, int LANES, bool F16, bool INTER, int HEADS>
mx_status qk_norm_launch_as(const QkNormArgs& a, cudaStream_t st, int64_t* ctas) {
  constexpr int kAtOnce = 32 / LANES * HEADS;
  const int64_t parts = (a.heads[0] + kAtOnce - 1) / kAtOnce + (a.heads[1] + kAtOnce - 1) / kAtOnce, heads = a.heads[0] + a.heads[1];
  // Items of one token's heads, or of rows in a row where the former would leave a third of their places empty or more.
  // (100 MB of rows, forward and backward, us: 3 + 1 heads of 80, 4 of 16 places, 205 and 368 by tokens, 84 and 139 by
  // rows; 16 + 2 of 64, 18 of 32, 63 and 110, 54 and 83; 12 + 12 of 96, 24 of 32, 65 and 115, 66 and 107; 32 + 8 of 128, all
  // places, 40 and 71, 51 and 80.)
  const bool flat = 2 * kAtOnce * parts >= 3 * heads;
  const int64_t items = flat ? (a.tokens * heads + kAtOnce - 1) / kAtOnce : a.tokens * parts;
  int64_t grid = (items + kQkThreads / 32 - 1) / (kQkThreads / 32);
  constexpr int64_t kMost = BACK ? kQkBackCtas : kQkCtas;
  if (grid > kMost) grid = kMost;
  if (ctas) *ctas = grid;
  auto kern = flat ? qk_norm_rope_rows_kernel<LANES, F16, INTER, HEADS> : qk_norm_rope_kernel<LANES, F16, INTER, HEADS>;
  if (BACK) kern = flat ? qk_norm_rope_backward_kernel<LANES, F16, INTER, HEADS, true> : qk_norm_rope_backward_kernel<LANES, F16, INTER, HEADS, false>;
  return pdl_launch(kern, static_cast<unsigned>(grid), kQkThreads, 0, st, a) == cudaSuccess ? launch_status() : MX_ERR_CUDA;
}
template <bool BACK, bool F16, bool INTER>
mx_status qk_norm_launch_with(const QkNormArgs& a, cudaStream_t st, int64_t* ctas) {
  return a.dim <= 64    ? qk_norm_launch_as<BACK, 8, F16, INTER, 4>(a, st, ctas)
         : a.dim <= 128 ? qk_norm_launch_as<BACK, 16, F16, INTER, 4>(a, st, ctas)
                        : qk_norm_launch_as<BACK, 32, F16, INTER, 4>(a, st, ctas);
}
template <bool BACK>
mx_status qk_norm_launch(const QkNormArgs& a, bool f16, cudaStream_t st, int64_t* ctas) {
  if (f16) return a.interleaved ? qk_norm_launch_with<BACK, true, true>(a, st, ctas) : qk_norm_launch_with<BACK, true, false>(a, st, ctas);
  return a.interleaved ? qk_norm_launch_with<BACK, false, true>(a, st, ctas) : qk_norm_launch_with<BACK, false, false>(a, st, ctas);
}

}  // namespace

extern "C" {

mx_status qk_norm_rope(const void* q, const void* k, mx_half type, int64_t num_tokens, int64_t heads, int64_t kv_heads,
                       int head_dim, int64_t q_stride_token, int64_t q_stride_head, int64_t k_stride_token,
                       int64_t k_stride_head, const void* q_weight, const void* k_weight, int weight_f32,
                       const float* cos_sin, int64_t max_positions, int rot_dim, const int32_t* positions, float eps,
                       int interleaved, void* q_out, void* k_out, int64_t q_out_stride_token, int64_t q_out_stride_head,
                       int64_t k_out_stride_token, int64_t k_out_stride_head, void* stream) {
  if (!qk_norm_ok(type, num_tokens, heads, kv_heads, head_dim, q_weight, k_weight, weight_f32, cos_sin, max_positions, rot_dim,
                  positions, eps, interleaved) ||
      !qk_rows_ok(q, num_tokens, heads, q_stride_token, q_stride_head) ||
      !qk_rows_ok(k, num_tokens, kv_heads, k_stride_token, k_stride_head) ||
      !qk_rows_ok(q_out, num_tokens, heads, q_out_stride_token, q_out_stride_head) ||
      !qk_rows_ok(k_out, num_tokens, kv_heads, k_out_stride_token, k_out_stride_head))
    return MX_ERR_INVALID_ARG;
  if (num_tokens == 0) return MX_OK;
  const int64_t weight_bytes = (weight_f32 ? 4 : 2) * static_cast<int64_t>(head_dim);
  if (!qk_apart(num_tokens, head_dim,
                {{q_out, heads, q_out_stride_token, q_out_stride_head}, {k_out, kv_heads, k_out_stride_token, k_out_stride_head}},
                {{q, heads, q_stride_token, q_stride_head}}, {{k, kv_heads, k_stride_token, k_stride_head}}, {},
                {span(q_weight, weight_bytes), span(kv_heads ? k_weight : nullptr, weight_bytes),
                 span(rot_dim ? cos_sin : nullptr, 4 * max_positions * rot_dim), span(positions, 4 * num_tokens)}))
    return MX_ERR_INVALID_ARG;
  QkNormArgs a{};
  a.x[0] = static_cast<const uint16_t*>(q);
  a.x[1] = static_cast<const uint16_t*>(k);
  a.xst[0] = q_stride_token, a.xst[1] = k_stride_token, a.xsh[0] = q_stride_head, a.xsh[1] = k_stride_head;
  a.out[0] = static_cast<uint16_t*>(q_out);
  a.out[1] = static_cast<uint16_t*>(k_out);
  a.ost[0] = q_out_stride_token, a.ost[1] = k_out_stride_token, a.osh[0] = q_out_stride_head, a.osh[1] = k_out_stride_head;
  a.weight[0] = q_weight, a.weight[1] = k_weight;
  a.table = rot_dim ? cos_sin : nullptr;
  a.positions = positions;
  a.eps = eps;
  a.tokens = static_cast<int>(num_tokens);
  a.heads[0] = static_cast<int>(heads), a.heads[1] = static_cast<int>(kv_heads);
  a.dim = head_dim, a.rot = rot_dim, a.most_pos = static_cast<int>(max_positions);
  a.interleaved = interleaved, a.weight_f32 = weight_f32;
  return qk_norm_launch<false>(a, type == MX_HALF_F16, as_stream(stream), nullptr);
}

size_t qk_norm_rope_workspace_bytes(int head_dim) {
  return head_dim < 8 || head_dim > 256 || head_dim % 8 ? 0 : static_cast<size_t>(kQkBackCtas) * 2 * head_dim * 4;
}

mx_status qk_norm_rope_backward(const void* dq_out, const void* dk_out, const void* q, const void* k, mx_half type,
                                int64_t num_tokens, int64_t heads, int64_t kv_heads, int head_dim,
                                int64_t dq_out_stride_token, int64_t dq_out_stride_head, int64_t dk_out_stride_token,
                                int64_t dk_out_stride_head, int64_t q_stride_token, int64_t q_stride_head,
                                int64_t k_stride_token, int64_t k_stride_head, const void* q_weight, const void* k_weight,
                                int weight_f32, const float* cos_sin, int64_t max_positions, int rot_dim,
                                const int32_t* positions, float eps, int interleaved, void* dq, void* dk,
                                int64_t dq_stride_token, int64_t dq_stride_head, int64_t dk_stride_token,
                                int64_t dk_stride_head, float* dq_weight, float* dk_weight, void* workspace, void* stream) {
  if (!qk_norm_ok(type, num_tokens, heads, kv_heads, head_dim, q_weight, k_weight, weight_f32, cos_sin, max_positions, rot_dim,
                  positions, eps, interleaved) ||
      !qk_rows_ok(q, num_tokens, heads, q_stride_token, q_stride_head) ||
      !qk_rows_ok(k, num_tokens, kv_heads, k_stride_token, k_stride_head) ||
      !qk_rows_ok(dq_out, num_tokens, heads, dq_out_stride_token, dq_out_stride_head) ||
      !qk_rows_ok(dk_out, num_tokens, kv_heads, dk_out_stride_token, dk_out_stride_head) ||
      !qk_rows_ok(dq, num_tokens, heads, dq_stride_token, dq_stride_head) ||
      !qk_rows_ok(dk, num_tokens, kv_heads, dk_stride_token, dk_stride_head))
    return MX_ERR_INVALID_ARG;
  if (!dq_weight || !dk_weight || !workspace || !aligned(dq_weight, 4) || !aligned(dk_weight, 4) || !aligned(workspace, 16))
    return MX_ERR_INVALID_ARG;
  const int64_t weight_bytes = (weight_f32 ? 4 : 2) * static_cast<int64_t>(head_dim);
  if (!qk_apart(num_tokens, head_dim, {{dq, heads, dq_stride_token, dq_stride_head}, {dk, kv_heads, dk_stride_token, dk_stride_head}},
                {{dq_out, heads, dq_out_stride_token, dq_out_stride_head}, {q, heads, q_stride_token, q_stride_head}},
                {{dk_out, kv_heads, dk_out_stride_token, dk_out_stride_head}, {k, kv_heads, k_stride_token, k_stride_head}},
                {span(dq_weight, 4 * static_cast<int64_t>(head_dim)), span(dk_weight, 4 * static_cast<int64_t>(head_dim)),
                 span(workspace, static_cast<int64_t>(qk_norm_rope_workspace_bytes(head_dim)))},
                {span(q_weight, weight_bytes), span(kv_heads ? k_weight : nullptr, weight_bytes),
                 span(rot_dim ? cos_sin : nullptr, 4 * max_positions * rot_dim), span(positions, 4 * num_tokens)}))
    return MX_ERR_INVALID_ARG;
  QkNormArgs a{};
  a.x[0] = static_cast<const uint16_t*>(q);
  a.x[1] = static_cast<const uint16_t*>(k);
  a.xst[0] = q_stride_token, a.xst[1] = k_stride_token, a.xsh[0] = q_stride_head, a.xsh[1] = k_stride_head;
  a.dy[0] = static_cast<const uint16_t*>(dq_out);
  a.dy[1] = static_cast<const uint16_t*>(dk_out);
  a.dst[0] = dq_out_stride_token, a.dst[1] = dk_out_stride_token, a.dsh[0] = dq_out_stride_head, a.dsh[1] = dk_out_stride_head;
  a.out[0] = static_cast<uint16_t*>(dq);
  a.out[1] = static_cast<uint16_t*>(dk);
  a.ost[0] = dq_stride_token, a.ost[1] = dk_stride_token, a.osh[0] = dq_stride_head, a.osh[1] = dk_stride_head;
  a.weight[0] = q_weight, a.weight[1] = k_weight;
  a.table = rot_dim ? cos_sin : nullptr;
  a.positions = positions;
  a.partial = static_cast<float*>(workspace);
  a.eps = eps;
  a.tokens = static_cast<int>(num_tokens);
  a.heads[0] = static_cast<int>(heads), a.heads[1] = static_cast<int>(kv_heads);
  a.dim = head_dim, a.rot = rot_dim, a.most_pos = static_cast<int>(max_positions);
  a.interleaved = interleaved, a.weight_f32 = weight_f32;
  cudaStream_t st = as_stream(stream);
  const std::lock_guard<std::mutex> hold(kv_turn);  // (the two launches speak to each other through the workspace)
  int64_t ctas = 0;
  if (num_tokens) {
    const mx_status s = qk_norm_launch<true>(a, type == MX_HALF_F16, st, &ctas);
    if (s != MX_OK) return s;
  }
  if (pdl_launch(qk_weight_grad_kernel, static_cast<unsigned>((2 * head_dim + 31) / 32), 1024, 0, st,
                 static_cast<const float*>(a.partial), static_cast<int>(ctas), head_dim, dq_weight, dk_weight) != cudaSuccess)
    return MX_ERR_CUDA;
  return launch_status();
}

mx_status kv_draft_trees(const int32_t* parents, int64_t num_tokens, const int32_t* lengths, const int32_t* q_start,
                         int64_t requests, int64_t max_q_len, int64_t window, int64_t* tree_mask, int64_t mask_words,
                         int32_t* positions, void* stream) {
  if (!kv_drafts_ok(q_start, requests, num_tokens, max_q_len) || !lengths || !aligned(lengths, 4)) return MX_ERR_INVALID_ARG;
  if (mask_words < 1 || mask_words > kKvMostNodes / 64 || mask_words * 64 < max_q_len || window < 0 || window > 0x7FFFFFFF)
    return MX_ERR_INVALID_ARG;
  if (num_tokens && (!parents || !tree_mask || !positions)) return MX_ERR_INVALID_ARG;
  if (!aligned(parents, 4) || !aligned(tree_mask, 8) || !aligned(positions, 4)) return MX_ERR_INVALID_ARG;
  if (num_tokens == 0) return MX_OK;
  const int64_t r4 = 4 * requests, t4 = 4 * num_tokens;
  if (kv_overlap({span(tree_mask, 2 * t4 * mask_words), span(positions, t4)},
                 {span(parents, t4), span(lengths, r4), span(q_start, r4 + 4)}))
    return MX_ERR_INVALID_ARG;
  KvTreesArgs a{};
  a.parents = parents;
  a.lengths = lengths;
  a.q_start = q_start;
  a.mask = reinterpret_cast<uint64_t*>(tree_mask);
  a.positions = positions;
  a.requests = static_cast<int>(requests);
  a.tokens = static_cast<int>(num_tokens);
  a.most = static_cast<int>(max_q_len);
  a.words = static_cast<int>(mask_words);
  a.window = static_cast<int>(window);
  if (pdl_launch(kv_draft_trees_kernel, static_cast<unsigned>(requests), kKvTreesThreads, 0, as_stream(stream), a) != cudaSuccess)
    return MX_ERR_CUDA;
  return launch_status();
}

mx_status kv_verify_drafts(const float* target_probs, int64_t target_stride, const float* draft_probs, int64_t draft_stride,
                           int64_t vocab, const int32_t* drafts, const int32_t* parents, int64_t num_tokens,
                           const int32_t* q_start, int64_t requests, int64_t max_q_len, const float* accept_random,
                           const float* sample_random, int32_t* path, int32_t* tokens, int32_t* counts, void* stream) {
  if (!kv_drafts_ok(q_start, requests, num_tokens, max_q_len)) return MX_ERR_INVALID_ARG;
  if (vocab < 1 || vocab > kKvVerifyMostVocab || target_stride < vocab || (draft_probs && draft_stride < vocab))
    return MX_ERR_INVALID_ARG;
  if (!sample_random || !counts ||
      (num_tokens && (!target_probs || !drafts || !parents || !accept_random || !path || !tokens)))
    return MX_ERR_INVALID_ARG;
  if (!aligned(target_probs, 4) || !aligned(draft_probs, 4) || !aligned(drafts, 4) || !aligned(parents, 4) ||
      !aligned(accept_random, 4) || !aligned(sample_random, 4) || !aligned(path, 4) || !aligned(tokens, 4) || !aligned(counts, 4))
    return MX_ERR_INVALID_ARG;
  const int64_t r4 = 4 * requests, t4 = 4 * num_tokens;
  if (kv_overlap({span(path, t4), span(tokens, t4), span(counts, r4)},
                 {span(drafts, t4), span(parents, t4), span(q_start, r4 + 4), span(accept_random, t4), span(sample_random, r4),
                  span(target_probs, 4 * vocab, num_tokens, 4 * target_stride),
                  span(draft_probs, 4 * vocab, num_tokens, 4 * draft_stride)}))
    return MX_ERR_INVALID_ARG;
  KvVerifyArgs a{};
  a.target = target_probs;
  a.draft = draft_probs;
  a.target_stride = target_stride;
  a.draft_stride = draft_stride;
  a.drafts = drafts;
  a.parents = parents;
  a.q_start = q_start;
  a.accept = accept_random;
  a.sample = sample_random;
  a.path = path;
  a.next = tokens;
  a.counts = counts;
  a.requests = static_cast<int>(requests);
  a.tokens = static_cast<int>(num_tokens);
  a.most = static_cast<int>(max_q_len);
  a.vocab = static_cast<int>(vocab);
  // CTAs a request: as many as keep two a SM, and no more than have a segment for each of their warps
  const int64_t segments = (vocab + kKvVerifySegment - 1) / kKvVerifySegment;
  unsigned ranks = kKvVerifyMostCluster;
  while (ranks > 1 && (requests * ranks > 304 || segments * 2 < ranks * (kKvVerifyThreads / 32))) ranks /= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(requests) * ranks);
  cfg.blockDim = dim3(kKvVerifyThreads);
  cfg.stream = as_stream(stream);
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = ranks;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, draft_probs ? kv_verify_kernel<false> : kv_verify_kernel<true>, a) != cudaSuccess)
    return MX_ERR_CUDA;
  return launch_status();
}

mx_status kv_cache_compact(const int32_t* path, const int32_t* counts, int64_t num_tokens, const int32_t* lengths,
                           const int32_t* q_start, int64_t requests, const int32_t* block_tables, int64_t max_blocks,
                           void* k_codes, void* v_codes, float* k_scale, float* v_scale, mx_elem elem, int64_t num_blocks,
                           int64_t kv_heads, int block_tokens, int head_dim, int32_t* kept_lengths, void* stream) {
  if (!kv_drafts_ok(q_start, requests, num_tokens, 0) || !counts || !lengths || !block_tables || !kept_lengths ||
      (num_tokens && !path))
    return MX_ERR_INVALID_ARG;
  if (!k_codes || !v_codes || !k_scale || !v_scale) return MX_ERR_INVALID_ARG;
  if (elem != MX_E4M3 && elem != MX_E5M2) return elem == MX_E2M1 ? MX_ERR_UNSUPPORTED : MX_ERR_INVALID_ARG;
  if (!kv_cache_shape_ok(num_blocks, kv_heads, block_tokens, head_dim)) return MX_ERR_INVALID_ARG;
  if (max_blocks < 1 || max_blocks > kKvMostTokens / block_tokens) return MX_ERR_INVALID_ARG;
  if (!aligned(path, 4) || !aligned(counts, 4) || !aligned(lengths, 4) || !aligned(block_tables, 4) || !aligned(k_codes, 16) ||
      !aligned(v_codes, 16) || !aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(kept_lengths, 4))
    return MX_ERR_INVALID_ARG;
  // (every CTA of a request reads its length and count, and one writes what it keeps)
  const int64_t r4 = 4 * requests, t4 = 4 * num_tokens;
  // (and keys' and values' warps move without looking at each other)
  const int64_t heads_of_blocks = num_blocks * kv_heads, code_bytes = heads_of_blocks * block_tokens * head_dim;
  if (kv_overlap({span(kept_lengths, r4), span(k_codes, code_bytes), span(v_codes, code_bytes), span(k_scale, 4 * heads_of_blocks),
                  span(v_scale, 4 * heads_of_blocks)},
                 {span(lengths, r4), span(counts, r4), span(q_start, r4 + 4), span(path, t4), span(block_tables, r4 * max_blocks)}))
    return MX_ERR_INVALID_ARG;
  KvCompactArgs a{};
  a.path = path;
  a.counts = counts;
  a.lengths = lengths;
  a.q_start = q_start;
  a.tables = block_tables;
  a.codes[0] = static_cast<uint8_t*>(k_codes);
  a.codes[1] = static_cast<uint8_t*>(v_codes);
  a.scale[0] = k_scale;
  a.scale[1] = v_scale;
  a.kept = kept_lengths;
  a.num_blocks = num_blocks;
  a.requests = static_cast<int>(requests);
  a.tokens = static_cast<int>(num_tokens);
  a.max_blocks = static_cast<int>(max_blocks);
  a.kv_heads = static_cast<int>(kv_heads);
  a.shift = kv_block_shift(block_tokens);
  constexpr int kWarps = kKvCompactThreads / 32;
  const dim3 grid(static_cast<unsigned>((2 * kv_heads + kWarps - 1) / kWarps), static_cast<unsigned>(requests));
  const auto kern = elem == MX_E5M2 ? (head_dim == 64 ? kv_compact_kernel<1, 64> : kv_compact_kernel<1, 128>)
                                    : (head_dim == 64 ? kv_compact_kernel<0, 64> : kv_compact_kernel<0, 128>);
  if (pdl_launch(kern, grid, kKvCompactThreads, 0, as_stream(stream), a) != cudaSuccess) return MX_ERR_CUDA;
  return launch_status();
}

}  // extern "C"
