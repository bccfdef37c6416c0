// step.cu -- the step's block tables and slots on the GPU, and the append into FP8 pools with one
// scale per (block, kv head), for sm_103a.  Declared in pkv_step.h.
#include <cooperative_groups.h>

#include <algorithm>
#include <cmath>

#include "kernels.h"
#include "ptx.cuh"
#include "pkv_step.h"

namespace pkv {
namespace {

// ------------------------------------------------------------------------------- step tables
//
// Three exclusive sums over the sequences (new tokens, blocks to take, blocks given back) decide
// everything: the place of each token in the packed batch, of each taken block on the free stack
// and of each pushed block.  The kernel reads a few bytes per sequence and writes 12 per token, so
// its floor is the launch and a chain of dependent loads; one CTA runs it, and the checks of all
// inputs come before the first write.
constexpr int kStepThreads = 1024;

// The largest i < n with start[i] <= x (start ascending, start[0] = 0, x below the total, so that
// entry owns x: of equal starts the last one has the items).
__device__ __forceinline__ int owner_of(const int* start, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kStepThreads) step_tables_kernel(const StepArgs a) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gtid = rank * blockDim.x + tid, gsize = (int)cluster.num_blocks() * blockDim.x;
  const int warps = blockDim.x >> 5;
  extern __shared__ int s_dyn[];
  int* s_tok = s_dyn;             // [B + 1] exclusive sum of the new tokens
  int* s_take = s_tok + a.B + 1;  // [B] exclusive sum of the blocks taken
  int* s_push = s_take + a.B;     // [B] exclusive sum of the blocks given back
  int* s_len = s_push + a.B;      // [B] context lengths at the call
  __shared__ int s_warp[3][32];
  __shared__ int s_carry[3];
  __shared__ int s_err;           // rank 0's copy collects the cluster's errors
  if (tid == 0) s_err = PKV_DEV_OK;
  if (tid < 3) s_carry[tid] = 0;
  grid_dependency_wait();
  grid_launch_dependents();
  cluster.sync();
  int* err0 = cluster.map_shared_rank(&s_err, 0);
  auto fail = [&](int code) { atomicCAS(err0, PKV_DEV_OK, code); };

  for (int base = 0; base < a.B; base += blockDim.x) {
    const int b = base + tid;
    int v[3] = {0, 0, 0};
    int c = 0;
    if (b < a.B) {
      c = a.context_lens[b];
      const int n = a.new_tokens[b];
      const long long cap = (long long)a.MB * 16;
      if (c < 0 || c > cap || (n > 0 && (long long)c + n > cap)) fail(PKV_DEV_BAD_CONTEXT_LEN);
      else if (n < -1) fail(PKV_DEV_BAD_QUERY_RANGE);
      else {
        // more tokens than the step holds are an error below; the cut keeps the sums in 32 bits
        const int m = min(n, a.max_tokens + 1);
        v[0] = max(m, 0);
        v[1] = m > 0 ? ((c + m + 15) >> 4) - ((c + 15) >> 4) : 0;
        v[2] = n < 0 ? (c + 15) >> 4 : 0;
      }
    }
    int incl[3];
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      int x = v[q];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(kFullMask, x, o);
        if (lane >= o) x += t;
      }
      incl[q] = x;
      if (lane == 31) s_warp[q][warp] = x;
    }
    __syncthreads();
    if (warp < 3) {
      const int own = lane < warps ? s_warp[warp][lane] : 0;
      int x = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(kFullMask, x, o);
        if (lane >= o) x += t;
      }
      const int carry = s_carry[warp];
      s_warp[warp][lane] = carry + x - own;
      __syncwarp();
      if (lane == 31) s_carry[warp] = carry + x;
    }
    __syncthreads();
    if (b < a.B) {
      s_tok[b] = s_warp[0][warp] + incl[0] - v[0];
      s_take[b] = s_warp[1][warp] + incl[1] - v[1];
      s_push[b] = s_warp[2][warp] + incl[2] - v[2];
      s_len[b] = c;
    }
    __syncthreads();
  }
  const int T = s_carry[0], A = s_carry[1], R = s_carry[2];
  const int count = a.free_count[0];
  if (tid == 0) {
    s_tok[a.B] = T;
    if (T > a.max_tokens) fail(PKV_DEV_BAD_QUERY_RANGE);
    else if (count < 0 || count > a.NB || R > a.NB - count || A > count + R) fail(PKV_DEV_NO_BLOCKS);
  }
  cluster.sync();
  const int top = count + R;
  bool ok = *err0 == PKV_DEV_OK;
  if (ok) {
    // push the ended sequences' blocks past the live entries (not live until the count says so)
    for (int r = gtid; r < R; r += gsize) {
      const int b = owner_of(s_push, a.B, r);
      const int id = a.block_tables[(size_t)b * a.MB + (r - s_push[b])];
      if (id < 0 || id >= a.NB) fail(PKV_DEV_BAD_BLOCK_ID);
      a.free_blocks[count + r] = id;
    }
    // the blocks that this step writes into: a sequence's part-filled last block, and those taken
    for (int b = gtid; b < a.B; b += gsize) {
      const int c = s_len[b];
      if ((c & 15) != 0 && s_tok[b + 1] > s_tok[b]) {
        const int id = a.block_tables[(size_t)b * a.MB + (c >> 4)];
        if (id < 0 || id >= a.NB) fail(PKV_DEV_BAD_BLOCK_ID);
      }
    }
  }
  __threadfence();
  cluster.sync();
  if (ok) {
    for (int p = gtid; p < A; p += gsize) {
      const int id = __ldcg(a.free_blocks + top - 1 - p);
      if (id < 0 || id >= a.NB) fail(PKV_DEV_BAD_BLOCK_ID);
    }
  }
  cluster.sync();
  const int code = *err0;
  ok = code == PKV_DEV_OK;
  for (int b = gtid; b <= a.B; b += gsize) {
    a.query_starts[b] = ok ? s_tok[b] : 0;
    if (b == a.B) continue;
    const int n = s_tok[b + 1] - s_tok[b];
    // ended: this one pushes blocks, or is an empty sequence that ends (0 either way)
    const bool ended = (b + 1 < a.B ? s_push[b + 1] : R) > s_push[b];
    a.context_lens_out[b] = ok ? (ended ? 0 : s_len[b] + n) : s_len[b];
  }
  for (int i = gtid; i < a.max_tokens; i += gsize) {
    long long slot = -1;
    int pos = -1;
    if (ok && i < T) {
      const int b = owner_of(s_tok, a.B, i);
      const int c = s_len[b], held = (c + 15) >> 4;
      pos = c + i - s_tok[b];
      const int j = pos >> 4;
      const int id = j < held ? a.block_tables[(size_t)b * a.MB + j]
                              : __ldcg(a.free_blocks + top - 1 - (s_take[b] + j - held));
      slot = (long long)id * 16 + (pos & 15);
    }
    a.slot_mapping[i] = slot;
    a.positions[i] = pos;
  }
  if (ok) {
    for (int p = gtid; p < A; p += gsize) {
      const int b = owner_of(s_take, a.B, p);
      a.block_tables[(size_t)b * a.MB + ((s_len[b] + 15) >> 4) + (p - s_take[b])] =
          __ldcg(a.free_blocks + top - 1 - p);
    }
  }
  if (gtid == 0) {
    a.free_count_out[0] = ok ? top - A : count;
    if (!ok) record_error(a.err, code);
  }
  cluster.sync();  // rank 0's error word is read by all until here
}

// --------------------------------------------------------------------------------- FP8 append

// E4M3 codes of two fp32 values (round to nearest even, saturating), `lo` in the low byte.
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t w) {
  const uint32_t h = e4m3x2_to_f16x2(w);
  return make_float2(f16_lo_to_f32(h), f16_hi_to_f32(h));
}

// The smallest power of two s with amax / s <= 448, its exponent kept in [-120, 119]: 448 is
// 1.75 * 2^8, so with amax = f 2^E, f in [1, 2), the exponent is E - 8, or E - 7 above f = 1.75.
__device__ __forceinline__ float needed_scale(float amax) {
  const int bits = __float_as_int(amax);
  int e = (bits >> 23) - 127 - 8 + ((bits & 0x7fffff) > 0x600000 ? 1 : 0);
  e = max(-120, min(119, e));  // zero and subnormal rows have the lowest exponent field
  return __int_as_float((e + 127) << 23);
}

// One warp per (token, kv head); the first token of a block in the call leads the block's run of
// adjacent tokens and the warps of the others end at once, so a block's scale has one writer.
// Lanes 0-15 hold the K rows, lanes 16-31 the V rows, D / 16 elements each.
template <int D>
__global__ void __launch_bounds__(256) kv_append_f8_kernel(uint8_t* __restrict__ kq, uint8_t* __restrict__ vq,
                                                           float* __restrict__ ks, float* __restrict__ vs,
                                                           const __nv_bfloat16* __restrict__ k,
                                                           const __nv_bfloat16* __restrict__ v,
                                                           const int64_t* __restrict__ slots, int64_t T,
                                                           int Hkv, int NB, int32_t* err) {
  constexpr int E = D / 16;   // elements per lane
  constexpr int W = E / 2;    // words of two bf16
  const int64_t item = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  grid_dependency_wait();
  grid_launch_dependents();
  if (item >= T * Hkv) return;
  const int64_t tok = item / Hkv;
  const int g = (int)(item - tok * Hkv);
  const int64_t slot = __ldg(slots + tok);
  if (slot < 0) return;
  if (slot >= (int64_t)NB * 16) {
    if (lane == 0) record_error(err, PKV_DEV_BAD_SLOT);
    return;
  }
  const int64_t blk = slot >> 4;
  if (tok > 0) {
    const int64_t before = __ldg(slots + tok - 1);
    if (before >= 0 && (before >> 4) == blk) {
      if (before >= slot && lane == 0) record_error(err, PKV_DEV_BAD_SLOT);
      return;
    }
  }
  // the run: lane l looks at token tok + l, which belongs while every one up to it is in the block
  // and above the one before
  int off = -1;
  {
    int64_t s = -1;
    if (lane < 16 && tok + lane < T) s = __ldg(slots + tok + lane);
    if (s >= 0 && (s >> 4) == blk) off = (int)(s & 15);
  }
  const int prev = __shfl_up_sync(kFullMask, off, 1);
  const uint32_t in_run = __ballot_sync(kFullMask, off >= 0 && (lane == 0 || off > prev));
  const int run = __ffs(~in_run) - 1;
  const size_t row0 = ((size_t)blk * Hkv + g) * 16;

  const int h = lane & 15;
  const __nv_bfloat16* src = (lane < 16 ? k : v) + ((size_t)tok * Hkv + g) * D + h * E;
  uint32_t x[16][W];
  uint32_t good = 0;  // tokens of the run whose K and V rows are finite
  float amax = 0.f;
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    if (r >= run) break;
    const __nv_bfloat16* p = src + (size_t)r * Hkv * D;
    if constexpr (W == 4) {
      const uint4 w = __ldg(reinterpret_cast<const uint4*>(p));
      x[r][0] = w.x; x[r][1] = w.y; x[r][2] = w.z; x[r][3] = w.w;
    } else {
      const uint2 w = __ldg(reinterpret_cast<const uint2*>(p));
      x[r][0] = w.x; x[r][1] = w.y;
    }
  }
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    if (r >= run) break;
    float m = 0.f;
    bool finite = true;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const float lo = bf16_lo_to_f32(x[r][i]), hi = bf16_hi_to_f32(x[r][i]);
      finite &= isfinite(lo) && isfinite(hi);
      m = fmaxf(m, fmaxf(fabsf(lo), fabsf(hi)));
    }
    if (__all_sync(kFullMask, finite)) {
      good |= 1u << r;
      amax = fmaxf(amax, m);
    } else if (lane == 0) {
      record_error(err, PKV_DEV_BAD_VALUE);
    }
  }
  if (good == 0) return;
#pragma unroll
  for (int m = 1; m < 16; m <<= 1) amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, m));  // the half-warp
  float* scale_at = (lane < 16 ? ks : vs) + (size_t)blk * Hkv + g;
  uint8_t* codes = (lane < 16 ? kq : vq) + row0 * D + h * E;
  const bool anew = (slot & 15) == 0;
  const float old = anew ? 0.f : *scale_at;
  if (!__all_sync(kFullMask, old >= 0.f && old <= 3.4028234e38f)) {
    if (lane == 0) record_error(err, PKV_DEV_BAD_VALUE);
    return;
  }
  const float now = fmaxf(needed_scale(amax), old);
  uint32_t written = (lane < run && ((good >> lane) & 1u)) ? 1u << off : 0u;
  written = __reduce_or_sync(kFullMask, written);
  if (!anew && now != old) {  // the block's other rows move to the larger scale
    const float ratio = __fdiv_rn(old, now);
#pragma unroll 4
    for (int o = 0; o < 16; ++o) {
      if ((written >> o) & 1u) continue;
      uint32_t* at = reinterpret_cast<uint32_t*>(codes + o * D);
#pragma unroll
      for (int i = 0; i < E / 4; ++i) {
        const uint32_t w = at[i];
        const float2 c01 = e4m3x2_to_f32(w & 0xffffu), c23 = e4m3x2_to_f32(w >> 16);
        at[i] = pack_e4m3x2(c01.x * ratio, c01.y * ratio) | (pack_e4m3x2(c23.x * ratio, c23.y * ratio) << 16);
      }
    }
  }
  // x / scale: by the exact reciprocal where the scale is a power of two (every scale that the append
  // makes), by a division where the caller's own scale is not
  const bool pow2 = (__float_as_int(now) & 0x7fffff) == 0 && now >= 1.1754944e-38f;
  const float inv = pow2 ? __frcp_rn(now) : 0.f;
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    if (r >= run) break;
    const int o = __shfl_sync(kFullMask, off, r);
    if (!((good >> r) & 1u)) continue;
    uint32_t out[E / 4];
#pragma unroll
    for (int i = 0; i < E / 4; ++i) {
      float f[4] = {bf16_lo_to_f32(x[r][2 * i]), bf16_hi_to_f32(x[r][2 * i]), bf16_lo_to_f32(x[r][2 * i + 1]),
                    bf16_hi_to_f32(x[r][2 * i + 1])};
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] = pow2 ? f[e] * inv : __fdiv_rn(f[e], now);
      out[i] = pack_e4m3x2(f[0], f[1]) | (pack_e4m3x2(f[2], f[3]) << 16);
    }
    if constexpr (E == 8)
      *reinterpret_cast<uint2*>(codes + o * D) = make_uint2(out[0], out[1]);
    else
      *reinterpret_cast<uint32_t*>(codes + o * D) = out[0];
  }
  if (h == 0 && now != old) *scale_at = now;
}

}  // namespace

size_t step_smem_bytes(int batch) { return sizeof(int) * (4 * (size_t)batch + 1); }

cudaError_t step_device_setup() {
  return cudaFuncSetAttribute((const void*)step_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)step_smem_bytes(kMaxStepBatch));
}

cudaError_t launch_step_tables(const StepArgs& a, cudaStream_t stream) {
  StepArgs args = a;
  void* params[] = {&args};
  return launch_pdl((const void*)step_tables_kernel, dim3(1), dim3(kStepThreads), step_smem_bytes(a.B), stream, params);
}

cudaError_t launch_kv_append_f8(void* kq, void* vq, float* ks, float* vs, const void* k, const void* v,
                                const int64_t* slots, int64_t T, int Hkv, int D, int NB, int32_t* err,
                                cudaStream_t stream) {
  const int64_t blocks = (T * Hkv + 7) / 8;
  void* params[] = {&kq, &vq, &ks, &vs, &k, &v, &slots, &T, &Hkv, &NB, &err};
  const void* f = D == 128 ? (const void*)kv_append_f8_kernel<128> : (const void*)kv_append_f8_kernel<64>;
  return launch_pdl(f, dim3((unsigned)blocks), dim3(256), 0, stream, params);
}

}  // namespace pkv

using namespace pkv;

extern "C" {

int pkv_kv_step_tables(int32_t* block_tables, int32_t* context_lens_out, int32_t* query_starts, int64_t* slot_mapping,
                       int32_t* positions, int32_t* free_count_out, int32_t* free_blocks, const int32_t* free_count,
                       const int32_t* context_lens, const int32_t* new_tokens, int32_t max_new_tokens,
                       const pkv_dims* dims, int32_t* error_word, void* stream) {
  if (dims == nullptr) return PKV_ERR_NULL_POINTER;
  if (dims->block_size != PKV_BLOCK_SIZE) return PKV_ERR_BLOCK_SIZE;
  if (dims->batch < 0 || dims->batch > kMaxStepBatch || dims->num_blocks < 0 || dims->max_blocks_per_seq < 0)
    return PKV_ERR_DIMS;
  // table entries, slots of one sequence and pushed blocks are counted in 32 bits
  if ((long long)dims->batch * dims->max_blocks_per_seq >= (1ll << 30) ||
      (long long)dims->max_blocks_per_seq * PKV_BLOCK_SIZE >= (1ll << 30))
    return PKV_ERR_DIMS;
  if (max_new_tokens < 0 || max_new_tokens > PKV_MAX_STEP_TOKENS) return PKV_ERR_ARGUMENT;
  if (!query_starts || !free_count || !free_count_out) return PKV_ERR_NULL_POINTER;
  if (dims->batch > 0 && (!context_lens_out || !context_lens || !new_tokens)) return PKV_ERR_NULL_POINTER;
  if (dims->batch > 0 && dims->max_blocks_per_seq > 0 && !block_tables) return PKV_ERR_NULL_POINTER;
  if (max_new_tokens > 0 && (!slot_mapping || !positions)) return PKV_ERR_NULL_POINTER;
  if (dims->num_blocks > 0 && !free_blocks) return PKV_ERR_NULL_POINTER;
  const int st = device_ready();
  if (st != PKV_OK) return st;
  StepArgs a{};
  a.block_tables = block_tables;
  a.context_lens_out = context_lens_out;
  a.query_starts = query_starts;
  a.slot_mapping = reinterpret_cast<long long*>(slot_mapping);
  a.positions = positions;
  a.free_count_out = free_count_out;
  a.free_blocks = free_blocks;
  a.free_count = free_count;
  a.context_lens = context_lens;
  a.new_tokens = new_tokens;
  a.err = error_word;
  a.B = dims->batch;
  a.MB = dims->max_blocks_per_seq;
  a.NB = dims->num_blocks;
  a.max_tokens = max_new_tokens;
  return cuda_status(launch_step_tables(a, static_cast<cudaStream_t>(stream)));
}

int pkv_kv_append_f8(void* k_codes, void* v_codes, float* k_scales, float* v_scales, const void* k, const void* v,
                     const int64_t* slot_mapping, int64_t num_tokens, const pkv_dims* dims, int32_t* error_word,
                     void* stream) {
  int st = check_dims(dims, false);
  if (st != PKV_OK) return st;
  if (num_tokens < 0 || num_tokens * dims->num_kv_heads >= (1ll << 33)) return PKV_ERR_DIMS;
  if (num_tokens == 0) return PKV_OK;
  if (!k_codes || !v_codes || !k_scales || !v_scales || !k || !v || !slot_mapping) return PKV_ERR_NULL_POINTER;
  if (!aligned16(k_codes) || !aligned16(v_codes) || !aligned16(k) || !aligned16(v) ||
      ((reinterpret_cast<uintptr_t>(k_scales) | reinterpret_cast<uintptr_t>(v_scales)) & 3u))
    return PKV_ERR_ALIGNMENT;
  st = device_ready();
  if (st != PKV_OK) return st;
  return cuda_status(launch_kv_append_f8(k_codes, v_codes, k_scales, v_scales, k, v, slot_mapping, num_tokens,
                                         dims->num_kv_heads, dims->head_dim, dims->num_blocks, error_word,
                                         static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
