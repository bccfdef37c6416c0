// prefill_attention.cu -- attention of many query tokens per sequence over the paged cache, with
// score rules, for sm_103a.  Declared in pkv_step.h.
//
// out[r, h] = sum_t p_t V_t, p = softmax over the keys t that row r sees, of
//   x_t = cap(scale q . K_t) - slope_h |i - t|,
// i the row's position, visible keys [lo, i] and the prefix [0, pre).
#include <algorithm>
#include <cmath>

#include "kernels.h"
#include "ptx.cuh"
#include "pkv_step.h"

namespace pkv {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

// What sequence b's rows need; n = 0 for one that is refused.
struct PrefillSeq {
  int q0, n, L, pre, err;
};

__device__ __forceinline__ PrefillSeq prefill_seq(const PrefillAttnArgs& a, int b) {
  PrefillSeq s{0, 0, 0, 0, 0};
  const int q0 = a.query_starts[b], q1 = a.query_starts[b + 1], L = a.context_lens[b];
  if (q0 < 0 || q1 < q0 || q1 > a.T) {
    s.err = PKV_DEV_BAD_QUERY_RANGE;
  } else if (L < 0 || L > a.MB * 16 || q1 - q0 > L) {
    s.err = PKV_DEV_BAD_CONTEXT_LEN;
  } else {
    s.q0 = q0;
    s.n = q1 - q0;
    s.L = L;
    s.pre = a.prefix_lens != nullptr ? min(max(a.prefix_lens[b], 0), L) : 0;
  }
  return s;
}

// First key of the interval that packed row r at position i sees (i + 1: none).
__device__ __forceinline__ int interval_start(const PrefillAttnArgs& a, int r, int i) {
  int lo = a.window > 0 && i >= a.window ? i - a.window + 1 : 0;
  if (a.doc_starts != nullptr) lo = min(max(lo, a.doc_starts[r]), i + 1);
  return lo;
}

// One row, one warp: each lane holds D / 32 elements, keys one at a time, online softmax.
template <int D>
__global__ void __launch_bounds__(256) prefill_rows_kernel(const PrefillAttnArgs a) {
  constexpr int E = D / 32;
  const long long item = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  grid_dependency_wait();
  grid_launch_dependents();
  if (item < a.B && lane == 0) {
    const PrefillSeq s = prefill_seq(a, (int)item);
    if (s.err != 0) record_error(a.err, s.err);
  }
  if (item >= (long long)a.T * a.Hq) return;
  const int r = (int)(item / a.Hq), h = (int)(item - (long long)r * a.Hq);
  int lo_b = 0, hi_b = a.B;
  while (hi_b - lo_b > 1) {
    const int mid = (lo_b + hi_b) >> 1;
    if (a.query_starts[mid] <= r) lo_b = mid; else hi_b = mid;
  }
  const int b = lo_b;
  const PrefillSeq s = prefill_seq(a, b);
  if (r < s.q0 || r >= s.q0 + s.n) return;
  const int i = s.L - s.n + (r - s.q0), g = h / a.G;
  int lo = interval_start(a, r, i);
  const int pre = s.pre;
  float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __bfloat162float(a.q[((size_t)r * a.Hq + h) * D + lane * E + e]);
    o[e] = 0.f;
  }
  const float slope = a.slopes != nullptr ? a.slopes[h] * kLog2e : 0.f;
  for (int t = 0; t < max(pre, i + 1); ++t) {
    if (t >= pre && t < lo) {
      t = lo;
      if (t > i) break;
    }
    const int phys = a.block_tables[(size_t)b * a.MB + (t >> 4)];
    if (phys < 0 || phys >= a.NB) {
      if (lane == 0) record_error(a.err, PKV_DEV_BAD_BLOCK_ID);
      continue;
    }
    const size_t row = (((size_t)phys * a.Hkv + g) * 16 + (t & 15)) * D + lane * E;
    float x = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) x = fmaf(q[e], __bfloat162float(a.k_cache[row + e]), x);
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) x += __shfl_xor_sync(kFullMask, x, w);
    x *= a.scale_log2;
    if (a.cap_log2 > 0.f) x = cap_logit(x, a.cap_log2, a.cap_in);
    x -= slope * fabsf((float)(i - t));
    const float top = fmaxf(m, x);
    const float ref = top == -INFINITY ? 0.f : top;
    const float keep = exp2f(m - ref), p = exp2f(x - ref);
    m = top;
    l = l * keep + p;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * keep + p * __bfloat162float(a.v_cache[row + e]);
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) a.out[((size_t)r * a.Hq + h) * D + lane * E + e] = __float2bfloat16_rn(o[e] * inv);
}

}  // namespace

size_t prefill_attention_workspace(int B, int T, int G, int D) {
  (void)B; (void)T; (void)G; (void)D;
  return 256;
}

cudaError_t launch_prefill_attention(const PrefillAttnArgs& a, int head_dim, cudaStream_t stream) {
  PrefillAttnArgs args = a;
  void* params[] = {&args};
  const long long warps = std::max((long long)a.T * a.Hq, (long long)a.B);
  const void* f = head_dim == 128 ? (const void*)prefill_rows_kernel<128> : (const void*)prefill_rows_kernel<64>;
  return launch_pdl(f, dim3((unsigned)((warps + 7) / 8)), dim3(256), 0, stream, params);
}

}  // namespace pkv

using namespace pkv;

namespace {

int check_prefill(const pkv_dims* dims, int32_t total_tokens) {
  const int st = check_dims(dims, true);
  if (st != PKV_OK) return st;
  if (dims->batch > kMaxStepBatch || total_tokens < 0) return PKV_ERR_DIMS;
  if (dims->num_q_heads / dims->num_kv_heads > kMaxGroup) return PKV_ERR_GQA;
  if ((long long)dims->num_blocks * dims->num_kv_heads * PKV_BLOCK_SIZE >= (1ll << 31) ||
      (long long)dims->max_blocks_per_seq * PKV_BLOCK_SIZE >= (1ll << 30) ||
      (long long)total_tokens * dims->num_q_heads >= (1ll << 31))
    return PKV_ERR_DIMS;
  return PKV_OK;
}

}  // namespace

extern "C" {

size_t pkv_prefill_workspace_bytes(const pkv_dims* dims, int32_t total_tokens) {
  if (check_prefill(dims, total_tokens) != PKV_OK) return 0;
  return prefill_attention_workspace(dims->batch, total_tokens, dims->num_q_heads / dims->num_kv_heads, dims->head_dim);
}

int pkv_paged_prefill_attention(void* out, const void* q, const void* k_cache, const void* v_cache,
                                const int32_t* block_tables, const int32_t* context_lens,
                                const int32_t* query_starts, int32_t total_tokens, float scale,
                                const pkv_score_rules* rules, void* workspace, size_t workspace_bytes,
                                const pkv_dims* dims, int32_t* error_word, void* stream) {
  int st = check_prefill(dims, total_tokens);
  if (st != PKV_OK) return st;
  if (rules != nullptr) {
    st = check_rules(rules);
    if (st != PKV_OK) return st;
  }
  if (dims->batch == 0 || total_tokens == 0) return PKV_OK;
  if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens || !query_starts) return PKV_ERR_NULL_POINTER;
  if (!workspace || workspace_bytes < pkv_prefill_workspace_bytes(dims, total_tokens)) return PKV_ERR_WORKSPACE;
  if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(workspace))
    return PKV_ERR_ALIGNMENT;
  st = device_ready();
  if (st != PKV_OK) return st;
  PrefillAttnArgs a{};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k_cache = static_cast<const __nv_bfloat16*>(k_cache);
  a.v_cache = static_cast<const __nv_bfloat16*>(v_cache);
  a.out = static_cast<__nv_bfloat16*>(out);
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.query_starts = query_starts;
  a.err = error_word;
  a.B = dims->batch;
  a.T = total_tokens;
  a.Hq = dims->num_q_heads;
  a.Hkv = dims->num_kv_heads;
  a.NB = dims->num_blocks;
  a.MB = dims->max_blocks_per_seq;
  a.G = dims->num_q_heads / dims->num_kv_heads;
  a.scale_log2 = scale * kLog2e;
  if (rules != nullptr) {
    a.window = rules->window;
    a.slopes = rules->alibi_slopes;
    a.doc_starts = rules->doc_starts;
    a.prefix_lens = rules->prefix_lens;
    a.cap_log2 = rules->softcap * kLog2e;
    a.cap_in = rules->softcap > 0.f ? 2.f / rules->softcap : 0.f;
  }
  return cuda_status(launch_prefill_attention(a, dims->head_dim, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
