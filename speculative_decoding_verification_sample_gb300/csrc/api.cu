// C-ABI entry points: host-side argument validation, then asynchronous launch
// on the caller's stream. No allocation, no synchronisation.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/specverify.h"
#include "launch.h"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int elem_bytes(int dtype) { return dtype == SPEC_BF16 ? 2 : (dtype == SPEC_F32 ? 4 : 0); }

}  // namespace

extern "C" {

int spec_version(void) { return 100; }

const char* spec_status_string(int status) {
  switch (status) {
    case SPEC_OK:
      return "ok";
    case SPEC_EINVAL:
      return "invalid argument";
    case SPEC_ECUDA:
      return "CUDA launch failed";
    case SPEC_ENOTSUP:
      return "unsupported configuration";
    default:
      return "unknown status";
  }
}

size_t spec_verify_workspace_bytes(int B, int K, int V, int dtype) {
  const int eb = elem_bytes(dtype);
  if (eb == 0 || B < 1 || K < 1 || K > 31 || V < 1 || (int64_t(V) * eb) % 16 != 0) return 0;
  const size_t a = sv::sample_workspace_bytes(B, K, V, dtype);
  const size_t g = sv::greedy_workspace_bytes(B, K, V, dtype);
  return a > g ? a : g;
}

static int check_workspace(void* ws, size_t bytes, int B, int K, int V, int dtype) {
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return SPEC_EINVAL;
  if (bytes < spec_verify_workspace_bytes(B, K, V, dtype)) return SPEC_EINVAL;
  return SPEC_OK;
}

int spec_verify_greedy(const void* target_logits, const int32_t* draft_tokens, int B, int K,
                       int V, int32_t* out_tokens, int32_t* out_num_accepted, void* stream,
                       int dtype, int32_t* err_flag, void* workspace, size_t workspace_bytes,
                       uint64_t* accept_counters) {
  const int eb = elem_bytes(dtype);
  if (!target_logits || !draft_tokens || !out_tokens || !out_num_accepted) return SPEC_EINVAL;
  if (eb == 0 || B < 1 || K < 1 || K > 31 || V < 1) return SPEC_EINVAL;
  if (!aligned16(target_logits)) return SPEC_EINVAL;
  if ((int64_t(V) * eb) % 16 != 0) return SPEC_ENOTSUP;
  if (int64_t(B) * (V / (16 / eb)) > INT32_MAX) return SPEC_EINVAL;
  if (check_workspace(workspace, workspace_bytes, B, K, V, dtype) != SPEC_OK) return SPEC_EINVAL;
  sv::GreedyLaunch g{target_logits, draft_tokens, B, K, V, dtype, out_tokens, out_num_accepted,
                     err_flag, stream, workspace,
                     reinterpret_cast<unsigned long long*>(accept_counters), nullptr, nullptr};
  return sv::launch_verify_greedy(g);
}

int spec_verify_tree_greedy(const void* target_logits, const int32_t* tree_parents,
                            const int32_t* tree_tokens, int B, int N, int V, int32_t* out_tokens,
                            int32_t* out_num_accepted, int32_t* out_slots, void* stream,
                            int dtype, int32_t* err_flag, void* workspace,
                            size_t workspace_bytes) {
  const int eb = elem_bytes(dtype);
  if (!target_logits || !tree_parents || !tree_tokens || !out_tokens || !out_num_accepted)
    return SPEC_EINVAL;
  if (eb == 0 || B < 1 || N < 1 || N > 31 || V < 1) return SPEC_EINVAL;
  if (!aligned16(target_logits)) return SPEC_EINVAL;
  if ((int64_t(V) * eb) % 16 != 0) return SPEC_ENOTSUP;
  if (int64_t(B) * (V / (16 / eb)) > INT32_MAX) return SPEC_EINVAL;
  if (check_workspace(workspace, workspace_bytes, B, N, V, dtype) != SPEC_OK) return SPEC_EINVAL;
  sv::GreedyLaunch g{target_logits, tree_tokens, B, N, V, dtype, out_tokens, out_num_accepted,
                     err_flag, stream, workspace, nullptr, tree_parents, out_slots};
  return sv::launch_verify_greedy(g);
}

int spec_verify_sample(const void* target_logits, const void* draft_logits,
                       const int32_t* draft_tokens, const float* uniforms, float temperature,
                       int B, int K, int V, int32_t* out_tokens, int32_t* out_num_accepted,
                       void* stream, int dtype, int32_t* err_flag, int32_t* row_info,
                       float* q_at_d, float* p_at_d, void* workspace, size_t workspace_bytes,
                       uint64_t* accept_counters, const float* target_threshold,
                       const float* draft_threshold) {
  if (std::isnan(temperature) || temperature < 0.0f || std::isinf(temperature)) return SPEC_EINVAL;
  if (temperature == 0.0f) {
    const int st = spec_verify_greedy(target_logits, draft_tokens, B, K, V, out_tokens,
                                      out_num_accepted, stream, dtype, err_flag, workspace,
                                      workspace_bytes, accept_counters);
    if (st == SPEC_OK && row_info)
      if (cudaMemsetAsync(row_info, 0, size_t(B) * sizeof(int32_t),
                          static_cast<cudaStream_t>(stream)) != cudaSuccess)
        return SPEC_ECUDA;
    return st;
  }
  const int eb = elem_bytes(dtype);
  if (!target_logits || !draft_logits || !draft_tokens || !uniforms || !out_tokens ||
      !out_num_accepted)
    return SPEC_EINVAL;
  if ((q_at_d == nullptr) != (p_at_d == nullptr)) return SPEC_EINVAL;
  if (eb == 0 || B < 1 || K < 1 || K > 31 || V < 1) return SPEC_EINVAL;
  if (!aligned16(target_logits) || !aligned16(draft_logits)) return SPEC_EINVAL;
  if ((int64_t(V) * eb) % 16 != 0) return SPEC_ENOTSUP;
  if (int64_t(B) * (V / (16 / eb)) > INT32_MAX) return SPEC_EINVAL;
  if (check_workspace(workspace, workspace_bytes, B, K, V, dtype) != SPEC_OK) return SPEC_EINVAL;
  sv::SampleLaunch s{target_logits, draft_logits, draft_tokens, uniforms, temperature, B, K, V,
                     dtype, out_tokens, out_num_accepted, err_flag, row_info, q_at_d, p_at_d,
                     stream, workspace, reinterpret_cast<unsigned long long*>(accept_counters),
                     target_threshold, draft_threshold};
  return sv::launch_verify_sample(s);
}

int spec_filter_thresholds(const void* logits, int R, int V, int dtype, float temperature,
                           int top_k, float top_p, float* out_threshold, void* stream,
                           int32_t* err_flag) {
  const int eb = elem_bytes(dtype);
  if (!logits || !out_threshold) return SPEC_EINVAL;
  if (eb == 0 || R < 1 || V < 1 || top_k < 0) return SPEC_EINVAL;
  if (!(top_p > 0.0f) || top_p > 1.0f) return SPEC_EINVAL;
  if (std::isnan(temperature) || !(temperature > 0.0f) || std::isinf(temperature)) return SPEC_EINVAL;
  if (!aligned16(logits)) return SPEC_EINVAL;
  if ((int64_t(V) * eb) % 16 != 0) return SPEC_ENOTSUP;
  if (V > (1 << 24)) return SPEC_ENOTSUP;
  sv::FilterLaunch f{logits, R, V, dtype, top_k, temperature, top_p, out_threshold, err_flag,
                     stream};
  return sv::launch_filter(f);
}

int kv_commit_rollback(int32_t* block_table, int32_t* seq_lens, const int32_t* num_accepted,
                       int32_t* prov_blocks, void* kv_pool, int num_blocks, int num_layers,
                       int num_kv_heads, int head_dim, int kv_elem_bytes, int block_size, int B,
                       int K, int max_blocks, int P, int32_t* free_stack, int32_t* free_top,
                       int32_t* status, void* stream, const int32_t* slot_map) {
  if (!block_table || !seq_lens || !num_accepted || !prov_blocks || !kv_pool || !free_stack ||
      !free_top || !status)
    return SPEC_EINVAL;
  if (num_blocks < 1 || num_layers < 1 || num_kv_heads < 1 || head_dim < 1 || kv_elem_bytes < 1 ||
      block_size < 1 || B < 1 || K < 0 || K > 31 || max_blocks < 1 || P < 1 || P > 512)
    return SPEC_EINVAL;
  const int64_t slot = int64_t(num_kv_heads) * head_dim * kv_elem_bytes;
  if (slot % 16 != 0 || !aligned16(kv_pool)) return SPEC_ENOTSUP;
  sv::KvLaunch k{block_table, seq_lens, num_accepted, prov_blocks, kv_pool, num_blocks,
                 num_layers,  num_kv_heads, head_dim, kv_elem_bytes, block_size, B, K,
                 max_blocks,  P, free_stack, free_top, status, stream, slot_map};
  return sv::launch_kv_commit(k);
}

static int kv_truncate(int32_t* block_table, int32_t* seq_lens, const int32_t* num_accepted,
                       int num_blocks, int block_size, int B, int K, int max_blocks,
                       int32_t* free_stack, int32_t* free_top, int32_t* status, void* stream) {
  if (!block_table || !seq_lens || !free_stack || !free_top || !status) return SPEC_EINVAL;
  if (num_blocks < 1 || block_size < 1 || B < 1 || K < 0 || K > 31 || max_blocks < 1)
    return SPEC_EINVAL;
  sv::KvTruncLaunch k{block_table, seq_lens, num_accepted, num_blocks, block_size, B, K,
                      max_blocks, free_stack, free_top, status, stream};
  return sv::launch_kv_truncate(k);
}

int kv_commit_inplace(int32_t* block_table, int32_t* seq_lens, const int32_t* num_accepted,
                      int num_blocks, int block_size, int B, int K, int max_blocks,
                      int32_t* free_stack, int32_t* free_top, int32_t* status, void* stream) {
  if (!num_accepted) return SPEC_EINVAL;
  return kv_truncate(block_table, seq_lens, num_accepted, num_blocks, block_size, B, K,
                     max_blocks, free_stack, free_top, status, stream);
}

int kv_evict_provisional(int32_t* block_table, int32_t* seq_lens, int num_blocks,
                         int block_size, int B, int K, int max_blocks, int32_t* free_stack,
                         int32_t* free_top, int32_t* status, void* stream) {
  return kv_truncate(block_table, seq_lens, nullptr, num_blocks, block_size, B, K, max_blocks,
                     free_stack, free_top, status, stream);
}

// Positions of a row fit 2^30, so that sums of a few of them fit an int.
static bool bad_table(int num_blocks, int block_size, int B, int max_blocks) {
  return num_blocks < 1 || block_size < 1 || B < 1 || max_blocks < 1 ||
         int64_t(max_blocks) * block_size > (int64_t(1) << 30) ||
         int64_t(B) * max_blocks > INT32_MAX / 2;
}

constexpr int kMaxPageRows = 8192;  // rows or pairs of one call of the block operators

int kv_reserve(int32_t* block_table, const int32_t* seq_lens, const int32_t* num_new, int n,
               int num_blocks, int block_size, int B, int max_blocks, const int32_t* free_stack,
               int32_t* free_top, int32_t* status, void* stream) {
  if (!block_table || !seq_lens || !free_stack || !free_top || !status) return SPEC_EINVAL;
  if (bad_table(num_blocks, block_size, B, max_blocks) || (!num_new && n < 0)) return SPEC_EINVAL;
  if (B > kMaxPageRows) return SPEC_ENOTSUP;
  sv::KvReserveLaunch k{block_table, seq_lens, num_new, n, num_blocks, block_size, B, max_blocks,
                        free_stack, free_top, status, stream};
  return sv::launch_kv_reserve(k);
}

int kv_fork(int32_t* block_table, int32_t* seq_lens, int32_t* extra_refs, const int32_t* src_rows,
            const int32_t* dst_rows, int n, void* kv_pool, int planes, int token_bytes,
            float* kv_scales, int num_blocks, int block_size, int B, int max_blocks,
            int32_t* free_stack, int32_t* free_top, int32_t* status, void* stream) {
  if (!block_table || !seq_lens || !extra_refs || !src_rows || !dst_rows || !kv_pool ||
      !free_stack || !free_top || !status)
    return SPEC_EINVAL;
  if (bad_table(num_blocks, block_size, B, max_blocks) || n < 1 || planes < 1 || token_bytes < 1)
    return SPEC_EINVAL;
  if (n > kMaxPageRows || int64_t(n) * max_blocks > INT32_MAX / 2) return SPEC_ENOTSUP;
  // a CTA addresses its planes' words with 32 bits
  if (token_bytes % 16 != 0 || !aligned16(kv_pool) || int64_t(block_size) * token_bytes > (1 << 27))
    return SPEC_ENOTSUP;
  sv::KvForkLaunch k{block_table, seq_lens, extra_refs, src_rows, dst_rows, kv_pool, kv_scales,
                     planes, token_bytes, num_blocks, block_size, B, max_blocks, n, free_stack,
                     free_top, status, stream};
  return sv::launch_kv_fork(k);
}

int kv_free(int32_t* block_table, int32_t* seq_lens, int32_t* extra_refs, const int32_t* rows,
            int n, int num_blocks, int B, int max_blocks, int32_t* free_stack, int32_t* free_top,
            int32_t* status, void* stream) {
  if (!block_table || !seq_lens || !extra_refs || !rows || !free_stack || !free_top || !status)
    return SPEC_EINVAL;
  if (bad_table(num_blocks, 1, B, max_blocks) || n < 1) return SPEC_EINVAL;
  if (n > kMaxPageRows || int64_t(n) * max_blocks > INT32_MAX / 2) return SPEC_ENOTSUP;
  sv::KvFreeLaunch k{block_table, seq_lens, extra_refs, rows, num_blocks, B, max_blocks, n,
                     free_stack, free_top, status, stream};
  return sv::launch_kv_free(k);
}

static int check_q8_pool(const void* pool, const float* scales, int num_blocks, int num_layers,
                         int layer, int num_kv_heads, int head_dim, int block_size, int B,
                         int max_blocks) {
  if (!pool || !scales) return SPEC_EINVAL;
  if (bad_table(num_blocks, block_size, B, max_blocks) || num_layers < 1 || layer < 0 ||
      layer >= num_layers || num_kv_heads < 1 || head_dim < 1)
    return SPEC_EINVAL;
  if (head_dim % 16 != 0 || !aligned16(pool)) return SPEC_ENOTSUP;
  if (int64_t(num_layers) * 2 * num_kv_heads > INT32_MAX ||
      int64_t(block_size) * head_dim > INT32_MAX / 4)
    return SPEC_ENOTSUP;
  return SPEC_OK;
}

int kv_q8_append(const void* k, const void* v, int dtype, void* kv_pool, float* kv_scales,
                 const int32_t* block_table, const int32_t* seq_lens, const int32_t* num_new,
                 int num_blocks, int num_layers, int layer, int num_kv_heads, int head_dim,
                 int block_size, int B, int T, int max_blocks, void* stream, int32_t* err_flag) {
  if (!k || !v || !block_table || !seq_lens || elem_bytes(dtype) == 0 || T < 1)
    return SPEC_EINVAL;
  const int st = check_q8_pool(kv_pool, kv_scales, num_blocks, num_layers, layer, num_kv_heads,
                               head_dim, block_size, B, max_blocks);
  if (st != SPEC_OK) return st;
  if (T > (1 << 30) - 2 * block_size) return SPEC_EINVAL;
  if (!aligned16(k) || !aligned16(v)) return SPEC_ENOTSUP;
  sv::Q8AppendLaunch a{k, v, dtype, kv_pool, kv_scales, block_table, seq_lens, num_new,
                       num_blocks, num_layers, layer, num_kv_heads, head_dim, block_size, B, T,
                       max_blocks, stream, err_flag};
  return sv::launch_kv_q8_append(a);
}

// What the two calls that norm and turn heads have in common. `tokens`: of one CTA at most.
static int check_norm_rope(const sv::NormRopeLaunch& r, int tokens) {
  const int eb = elem_bytes(r.dtype);
  if (!r.q || !r.q_out || eb == 0 || r.B < 1 || r.T < 1 || r.Hq < 1 || r.H < 0) return SPEC_EINVAL;
  if (r.D < 2 || r.D % 2 != 0 || r.half < 0 || r.half > r.D / 2 ||
      (r.half > 0) != (r.inv_freq != nullptr))
    return SPEC_EINVAL;
  if (!(r.eps >= 0.0f) || std::isinf(r.eps) || !std::isfinite(r.factor)) return SPEC_EINVAL;
  if (!r.seq_lens && (!r.positions || r.pool)) return SPEC_EINVAL;
  if (r.D > 256 || int64_t(r.B) * r.T > INT32_MAX || r.T > (1 << 30) ||
      int64_t(tokens) * (int64_t(r.Hq) + r.H) > INT32_MAX)
    return SPEC_ENOTSUP;
  const int64_t q_min = int64_t(r.Hq) * r.D, k_min = int64_t(r.H) * r.D;
  if (r.q_stride < q_min || r.q_out_stride < q_min || r.k_stride < k_min ||
      (r.v && r.v_stride < k_min) || (r.k_out && r.k_out_stride < k_min))
    return SPEC_EINVAL;
  for (const int64_t s : {r.q_stride, r.k_stride, r.v_stride, r.q_out_stride, r.k_out_stride})
    if (s > (int64_t(1) << 31)) return SPEC_ENOTSUP;
  for (const void* p : {r.q, r.k, r.v, (const void*)r.q_out, (const void*)r.k_out, r.q_weight,
                        r.k_weight})
    if (reinterpret_cast<uintptr_t>(p) % eb != 0) return SPEC_ENOTSUP;
  return SPEC_OK;
}

int qk_norm_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride, int dtype,
                 void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride,
                 const void* q_weight, const void* k_weight, float eps, const float* inv_freq,
                 int num_pairs, int interleaved, float rope_factor, const int32_t* seq_lens,
                 const int32_t* positions, const int32_t* num_new, int num_q_heads,
                 int num_kv_heads, int head_dim, int B, int T, void* stream, int32_t* err_flag) {
  if ((k != nullptr) != (k_out != nullptr) || (k != nullptr) != (num_kv_heads > 0))
    return SPEC_EINVAL;
  sv::NormRopeLaunch r = {};
  r.q = q;
  r.q_stride = q_stride;
  r.k = k;
  r.k_stride = k ? k_stride : 0;
  r.dtype = dtype;
  r.q_out = q_out;
  r.q_out_stride = q_out_stride;
  r.k_out = k_out;
  r.k_out_stride = k ? k_out_stride : 0;
  r.q_weight = q_weight;
  r.k_weight = k ? k_weight : nullptr;
  r.eps = eps;
  r.inv_freq = inv_freq;
  r.half = num_pairs;
  r.interleaved = interleaved != 0;
  r.factor = rope_factor;
  r.seq_lens = seq_lens;
  r.positions = positions;
  r.num_new = num_new;
  r.Hq = num_q_heads;
  r.H = num_kv_heads;
  r.D = head_dim;
  r.B = B;
  r.T = T;
  r.stream = stream;
  r.err = err_flag;
  const int st = check_norm_rope(r, 16);
  return st != SPEC_OK ? st : sv::launch_norm_rope(r);
}

int kv_q8_norm_rope_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                           const void* v, int64_t v_stride, int dtype, void* q_out,
                           int64_t q_out_stride, const void* q_weight, const void* k_weight,
                           float eps, const float* inv_freq, int num_pairs, int interleaved,
                           float rope_factor, void* kv_pool, float* kv_scales,
                           const int32_t* block_table, const int32_t* seq_lens,
                           const int32_t* positions, const int32_t* num_new, int num_blocks,
                           int num_layers, int layer, int num_q_heads, int num_kv_heads,
                           int head_dim, int block_size, int B, int T, int max_blocks,
                           void* stream, int32_t* err_flag) {
  if (!k || !v || !block_table || !seq_lens) return SPEC_EINVAL;
  const int pool = check_q8_pool(kv_pool, kv_scales, num_blocks, num_layers, layer, num_kv_heads,
                                 head_dim, block_size, B, max_blocks);
  if (pool != SPEC_OK) return pool;
  if (T > (1 << 30) - 2 * block_size) return SPEC_EINVAL;
  sv::NormRopeLaunch r = {};
  r.q = q;
  r.q_stride = q_stride;
  r.k = k;
  r.k_stride = k_stride;
  r.v = v;
  r.v_stride = v_stride;
  r.dtype = dtype;
  r.q_out = q_out;
  r.q_out_stride = q_out_stride;
  r.q_weight = q_weight;
  r.k_weight = k_weight;
  r.eps = eps;
  r.inv_freq = inv_freq;
  r.half = num_pairs;
  r.interleaved = interleaved != 0;
  r.factor = rope_factor;
  r.seq_lens = seq_lens;
  r.positions = positions;
  r.num_new = num_new;
  r.Hq = num_q_heads;
  r.H = num_kv_heads;
  r.D = head_dim;
  r.B = B;
  r.T = T;
  r.pool = kv_pool;
  r.scales = kv_scales;
  r.block_table = block_table;
  r.num_blocks = num_blocks;
  r.num_layers = num_layers;
  r.layer = layer;
  r.bs = block_size;
  r.max_blocks = max_blocks;
  r.stream = stream;
  r.err = err_flag;
  const int st = check_norm_rope(r, T < block_size ? T : block_size);
  return st != SPEC_OK ? st : sv::launch_norm_rope(r);
}

size_t kv_q8_attention_workspace_bytes(int T, int num_q_heads, int num_kv_heads, int head_dim) {
  if (T < 1 || T > 32 || num_kv_heads < 1 || num_q_heads < num_kv_heads ||
      num_q_heads % num_kv_heads != 0 || head_dim < 16 || head_dim > 256 || head_dim % 16 != 0)
    return 0;
  return sv::kv_q8_attention_workspace(T, num_q_heads / num_kv_heads, head_dim);
}

int kv_q8_attention(const void* q, int dtype, const void* kv_pool, const float* kv_scales,
                    const int32_t* block_table, const int32_t* seq_lens, const int32_t* num_new,
                    const uint32_t* tree_mask, void* out, float softmax_scale, int window,
                    int sinks, int num_blocks, int num_layers, int layer, int num_q_heads,
                    int num_kv_heads, int head_dim, int block_size, int B, int T, int max_blocks,
                    void* workspace, size_t workspace_bytes, void* stream, int32_t* err_flag) {
  if (!q || !out || !block_table || !seq_lens || elem_bytes(dtype) == 0) return SPEC_EINVAL;
  if (!(softmax_scale > 0.0f) || std::isinf(softmax_scale) || window < 0 || sinks < 0 ||
      (sinks > 0 && window == 0))
    return SPEC_EINVAL;
  const int st = check_q8_pool(kv_pool, kv_scales, num_blocks, num_layers, layer, num_kv_heads,
                               head_dim, block_size, B, max_blocks);
  if (st != SPEC_OK) return st;
  if (T < 1 || num_q_heads < num_kv_heads || num_q_heads % num_kv_heads != 0) return SPEC_EINVAL;
  if (tree_mask && window > 0) return SPEC_ENOTSUP;
  const size_t need = kv_q8_attention_workspace_bytes(T, num_q_heads, num_kv_heads, head_dim);
  if (need == 0 || int64_t(T) * num_q_heads > (1 << 20)) return SPEC_ENOTSUP;
  if (!aligned16(q) || !aligned16(out)) return SPEC_ENOTSUP;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || workspace_bytes < need)
    return SPEC_EINVAL;
  sv::Q8AttnLaunch a{q, dtype, kv_pool, kv_scales, block_table, seq_lens, num_new, tree_mask, out,
                     softmax_scale, window, sinks, num_blocks, num_layers, layer, num_kv_heads,
                     num_q_heads / num_kv_heads, head_dim, block_size, B, T, max_blocks, workspace,
                     stream, err_flag};
  return sv::launch_kv_q8_attention(a);
}

size_t kv_prefix_plan_bytes(int B, int num_groups, int num_members) {
  if (B < 1 || B > kMaxPageRows || num_groups < 0 || num_groups > kMaxPageRows ||
      num_members < 0 || num_members > kMaxPageRows)
    return 0;
  return sv::kv_prefix_plan_size(B, num_groups, num_members);
}

int kv_prefix_plan(const int32_t* block_table, const int32_t* seq_lens, const int32_t* num_new,
                   const int32_t* group_starts, const int32_t* group_rows, int num_groups,
                   int num_members, int T, int num_q_heads, int num_kv_heads, int num_blocks,
                   int block_size, int B, int max_blocks, void* plan, size_t plan_bytes,
                   void* stream, int32_t* err_flag) {
  if (!block_table || !seq_lens || !group_starts || (!group_rows && num_members > 0) || !plan)
    return SPEC_EINVAL;
  if (bad_table(num_blocks, block_size, B, max_blocks) || num_groups < 0 || num_members < 0 ||
      T < 1 || num_kv_heads < 1 || num_q_heads < num_kv_heads || num_q_heads % num_kv_heads != 0)
    return SPEC_EINVAL;
  const size_t need = kv_prefix_plan_bytes(B, num_groups, num_members);
  if (need == 0 || T > 32 || int64_t(T) * num_q_heads > (1 << 20) ||
      int64_t(B > num_members ? B : num_members) * T * num_q_heads > INT32_MAX)
    return SPEC_ENOTSUP;
  if ((reinterpret_cast<uintptr_t>(plan) & 255u) != 0 || plan_bytes < need) return SPEC_EINVAL;
  sv::KvPrefixPlanLaunch k{block_table, seq_lens, num_new, group_starts, group_rows, num_groups,
                           num_members, T, num_q_heads / num_kv_heads, num_kv_heads, num_blocks,
                           block_size, B, max_blocks, plan, stream, err_flag};
  return sv::launch_kv_prefix_plan(k);
}

size_t kv_q8_prefix_attention_workspace_bytes(int B, int T, int num_q_heads, int num_kv_heads,
                                              int head_dim) {
  const size_t each = kv_q8_attention_workspace_bytes(T, num_q_heads, num_kv_heads, head_dim);
  if (B < 1 || B > kMaxPageRows || each == 0) return 0;
  return sv::kv_prefix_workspace(B, T, num_kv_heads, num_q_heads / num_kv_heads, head_dim);
}

int kv_q8_prefix_attention(const void* q, int dtype, const void* kv_pool, const float* kv_scales,
                           const int32_t* block_table, const int32_t* seq_lens,
                           const int32_t* num_new, const uint32_t* tree_mask, const void* plan,
                           size_t plan_bytes, void* out, float softmax_scale, int num_blocks,
                           int num_layers, int layer, int num_q_heads, int num_kv_heads,
                           int head_dim, int block_size, int B, int T, int max_blocks,
                           void* workspace, size_t workspace_bytes, void* stream,
                           int32_t* err_flag) {
  if (!plan || (reinterpret_cast<uintptr_t>(plan) & 255u) != 0) return SPEC_EINVAL;
  const size_t need =
      kv_q8_prefix_attention_workspace_bytes(B, T, num_q_heads, num_kv_heads, head_dim);
  if (!sv::kv_prefix_takes(dtype, head_dim, block_size,
                           int64_t(num_blocks) * num_layers * 2 * num_kv_heads) ||
      need == 0)
    // each row by itself (and the refusals that the calls have in common)
    return B > kMaxPageRows
               ? SPEC_ENOTSUP
               : kv_q8_attention(q, dtype, kv_pool, kv_scales, block_table, seq_lens, num_new,
                                 tree_mask, out, softmax_scale, 0, 0, num_blocks, num_layers,
                                 layer, num_q_heads, num_kv_heads, head_dim, block_size, B, T,
                                 max_blocks, workspace, workspace_bytes, stream, err_flag);
  if (!q || !out || !block_table || !seq_lens) return SPEC_EINVAL;
  if (plan_bytes < kv_prefix_plan_bytes(B, 0, 0)) return SPEC_EINVAL;
  if (!(softmax_scale > 0.0f) || std::isinf(softmax_scale)) return SPEC_EINVAL;
  const int st = check_q8_pool(kv_pool, kv_scales, num_blocks, num_layers, layer, num_kv_heads,
                               head_dim, block_size, B, max_blocks);
  if (st != SPEC_OK) return st;
  if (int64_t(T) * num_q_heads > (1 << 20) || int64_t(B) * T * num_q_heads > INT32_MAX)
    return SPEC_ENOTSUP;
  if (!aligned16(q) || !aligned16(out)) return SPEC_ENOTSUP;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || workspace_bytes < need)
    return SPEC_EINVAL;
  sv::Q8AttnLaunch a{q, dtype, kv_pool, kv_scales, block_table, seq_lens, num_new, tree_mask, out,
                     softmax_scale, 0, 0, num_blocks, num_layers, layer, num_kv_heads,
                     num_q_heads / num_kv_heads, head_dim, block_size, B, T, max_blocks, workspace,
                     stream, err_flag};
  return sv::launch_kv_prefix_attention(a, plan, plan_bytes);
}

}  // extern "C"
