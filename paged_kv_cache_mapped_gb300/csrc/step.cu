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
// its floor is the launch and a chain of dependent loads (64 decoding sequences 4.4 us, 4096 with prompts among
// them 17 us on the GPU).  One cluster runs it, of one CTA or (large steps) of eight: every CTA has all the
// sums, the tokens and blocks are dealt out, and the cluster's barriers put the checks of all inputs before the
// first write without a word of workspace.
constexpr int kStepThreads = 1024;
constexpr int kStepRunMost = kMaxStepBatch / kStepThreads;
constexpr int kStepCluster = 8;
// More tokens or sequences than this are for eight CTAs (us with one and with eight: 64 tokens 4.4, 5.8; 2048 of
// as many sequences 8.2, 8.6; 4096 of 16 sequences 6.4, 6.3; 4096 of as many 12.4, 10.3; 64000 61.7, 8.5).
constexpr int kStepLarge = 2048;

// kStepRun: sequences of a thread.  CLUSTER: eight CTAs, or one (whose barriers are the block's).
template <int kStepRun, bool CLUSTER>
__global__ void __launch_bounds__(kStepThreads) step_tables_kernel(const StepArgs a) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = CLUSTER ? (int)cluster.block_rank() : 0;
  auto sync_all = [&] {
    if constexpr (CLUSTER) cluster.sync();
    else __syncthreads();
  };
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gtid = rank * blockDim.x + tid, gsize = (CLUSTER ? kStepCluster : 1) * (int)blockDim.x;
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
  grid_dependency_wait();
  grid_launch_dependents();
  sync_all();
  int* err0 = CLUSTER ? cluster.map_shared_rank(&s_err, 0) : &s_err;
  auto fail = [&](int code) { atomicCAS(err0, PKV_DEV_OK, code); };

  // a thread's run of up to kStepRun sequences, summed here, then across the block
  int v[3][kStepRun], sum[3] = {0, 0, 0};
  const int run0 = tid * kStepRun;
#pragma unroll
  for (int k = 0; k < kStepRun; ++k) {
    const int b = run0 + k;
#pragma unroll
    for (int q = 0; q < 3; ++q) v[q][k] = 0;
    if (b < a.B) {
      const int c = a.context_lens[b], n = a.new_tokens[b];
      const long long cap = (long long)a.MB * 16;
      if (c < 0 || c > cap || (n > 0 && (long long)c + n > cap)) fail(PKV_DEV_BAD_CONTEXT_LEN);
      else if (n < -1) fail(PKV_DEV_BAD_QUERY_RANGE);
      else {
        // more tokens than the step holds are an error below; the cut keeps the sums in 32 bits
        const int m = min(n, a.max_tokens + 1);
        v[0][k] = max(m, 0);
        v[1][k] = m > 0 ? ((c + m + 15) >> 4) - ((c + 15) >> 4) : 0;
        v[2][k] = n < 0 ? (c + 15) >> 4 : 0;
      }
      s_len[b] = c;
    }
#pragma unroll
    for (int q = 0; q < 3; ++q) sum[q] += v[q][k];
  }
  int incl[3];
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    int x = sum[q];
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
    s_warp[warp][lane] = x - own;
    if (lane == 31) s_carry[warp] = x;
  }
  __syncthreads();
  {
    int at[3];
#pragma unroll
    for (int q = 0; q < 3; ++q) at[q] = s_warp[q][warp] + incl[q] - sum[q];
#pragma unroll
    for (int k = 0; k < kStepRun; ++k) {
      if (run0 + k < a.B) {
        s_tok[run0 + k] = at[0];
        s_take[run0 + k] = at[1];
        s_push[run0 + k] = at[2];
      }
#pragma unroll
      for (int q = 0; q < 3; ++q) at[q] += v[q][k];
    }
  }
  const int T = s_carry[0], A = s_carry[1], R = s_carry[2];
  const int count = a.free_count[0];
  if (tid == 0) {
    s_tok[a.B] = T;
    if (T > a.max_tokens) fail(PKV_DEV_BAD_QUERY_RANGE);
    else if (count < 0 || count > a.NB || R > a.NB - count || A > count + R) fail(PKV_DEV_NO_BLOCKS);
  }
  sync_all();
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
  sync_all();
  if (ok) {
    for (int p = gtid; p < A; p += gsize) {
      const int id = __ldcg(a.free_blocks + top - 1 - p);
      if (id < 0 || id >= a.NB) fail(PKV_DEV_BAD_BLOCK_ID);
    }
  }
  sync_all();
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
  // four tokens a thread: one search, then along; 16-byte stores
  for (int i0 = 4 * gtid; i0 < a.max_tokens; i0 += 4 * gsize) {
    long long slot[4];
    int pos[4];
    int b = 0, block_j = -1, id = 0;
    if (ok && i0 < T) b = owner_of(s_tok, a.B, i0);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      slot[k] = -1;
      pos[k] = -1;
      if (ok && i0 + k < T) {
        while (s_tok[b + 1] <= i0 + k) {
          ++b;
          block_j = -1;
        }
        const int c = s_len[b], held = (c + 15) >> 4;
        pos[k] = c + i0 + k - s_tok[b];
        const int j = pos[k] >> 4;
        if (j != block_j) {
          id = j < held ? a.block_tables[(size_t)b * a.MB + j]
                        : __ldcg(a.free_blocks + top - 1 - (s_take[b] + j - held));
          block_j = j;
        }
        slot[k] = (long long)id * 16 + (pos[k] & 15);
      }
    }
    if (a.wide && i0 + 4 <= a.max_tokens) {
      *reinterpret_cast<longlong2*>(a.slot_mapping + i0) = make_longlong2(slot[0], slot[1]);
      *reinterpret_cast<longlong2*>(a.slot_mapping + i0 + 2) = make_longlong2(slot[2], slot[3]);
      *reinterpret_cast<int4*>(a.positions + i0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (i0 + k >= a.max_tokens) break;
        a.slot_mapping[i0 + k] = slot[k];
        a.positions[i0 + k] = pos[k];
      }
    }
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
  sync_all();  // rank 0's error word is read by all until here
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

// One run for one kv head: `tok` leads it; lane l has the slot of token tok + l (l < 16; -1 past the last).
template <int D>
__device__ __forceinline__ void append_run(uint8_t* kq, uint8_t* vq, float* ks, float* vs, const __nv_bfloat16* k,
                                           const __nv_bfloat16* v, int64_t lane_slot, int Hkv, int64_t tok, int g,
                                           int32_t* err) {
  constexpr int E = D / 16;   // elements per lane
  constexpr int W = E / 2;    // words of two bf16
  constexpr int kRows = 8;    // in registers at a time
  const int lane = threadIdx.x & 31;
  const int64_t slot = __shfl_sync(kFullMask, lane_slot, 0);
  const int64_t blk = slot >> 4;
  // the run: token tok + l belongs while every one up to it is in the block and above the one before
  const int off = lane < 16 && lane_slot >= 0 && (lane_slot >> 4) == blk ? (int)(lane_slot & 15) : -1;
  const int prev = __shfl_up_sync(kFullMask, off, 1);
  const uint32_t in_run = __ballot_sync(kFullMask, off >= 0 && (lane == 0 || off > prev));
  const int run = __ffs(~in_run) - 1;
  const size_t row0 = ((size_t)blk * Hkv + g) * 16;

  const int h = lane & 15;
  const __nv_bfloat16* src = (lane < 16 ? k : v) + ((size_t)tok * Hkv + g) * D + h * E;
  uint32_t bad = 0;
  uint32_t most = 0;  // largest |x| so far as bf16 bits, a pair of 16-bit numbers (sign cleared they order like the values)
  uint32_t x[kRows][W];
  auto load = [&](int r0) {
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (r0 + r >= run) break;
      const __nv_bfloat16* p = src + (size_t)(r0 + r) * Hkv * D;
      if constexpr (W == 4) {
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(p));
        x[r][0] = w.x; x[r][1] = w.y; x[r][2] = w.z; x[r][3] = w.w;
      } else {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(p));
        x[r][0] = w.x; x[r][1] = w.y;
      }
    }
  };
  for (int r0 = 0; r0 < run; r0 += kRows) {
    load(r0);
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (r0 + r >= run) break;
      uint32_t m = x[r][0] & 0x7fff7fffu;
#pragma unroll
      for (int i = 1; i < W; ++i) m = __vmaxu2(m, x[r][i] & 0x7fff7fffu);
      if ((m & 0xffffu) >= 0x7f80u || (m >> 16) >= 0x7f80u) bad |= 1u << (r0 + r);
      most = __vmaxu2(most, m);
    }
  }
  bad = __reduce_or_sync(kFullMask, bad);  // tokens of the run with a non-finite element in their K or V row
  const uint32_t good = ((1u << run) - 1u) & ~bad;
  if (bad != 0) {  // the other rows' largest, once more
    if (lane == 0) record_error(err, PKV_DEV_BAD_VALUE);
    most = 0;
    for (int r0 = 0; r0 < run; r0 += kRows) {
      load(r0);
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        if (!((good >> (r0 + r)) & 1u)) continue;
#pragma unroll
        for (int i = 0; i < W; ++i) most = __vmaxu2(most, x[r][i] & 0x7fff7fffu);
      }
    }
  }
  if (good == 0) return;
#pragma unroll
  for (int m = 1; m < 16; m <<= 1) most = __vmaxu2(most, __shfl_xor_sync(kFullMask, most, m));  // the half-warp
  const float amax = __uint_as_float(max(most & 0xffffu, most >> 16) << 16);
  float* scale_at = (lane < 16 ? ks : vs) + (size_t)blk * Hkv + g;
  uint8_t* codes = (lane < 16 ? kq : vq) + row0 * D + h * E;
  const bool anew = (slot & 15) == 0 && (good & 1u) != 0;  // offset 0 is written, not only asked for
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
  // the run's offsets, four bits each
  const uint32_t own = lane < run ? (uint32_t)off << (4 * (lane & 7)) : 0u;
  const uint32_t offs0 = __reduce_or_sync(kFullMask, lane < 8 ? own : 0u), offs1 = __reduce_or_sync(kFullMask, lane < 8 ? 0u : own);
  // x / scale: by the exact reciprocal where the scale is a power of two (every scale that the append
  // makes), by a division where the caller's own scale is not
  const bool pow2 = (__float_as_int(now) & 0x7fffff) == 0 && now >= 1.1754944e-38f;
  const float inv = pow2 ? __frcp_rn(now) : 0.f;
  for (int r0 = 0; r0 < run; r0 += kRows) {
    load(r0);
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (!((good >> (r0 + r)) & 1u)) continue;
      const int o = (int)(((r0 + r < 8 ? offs0 : offs1) >> (4 * ((r0 + r) & 7))) & 15u);
      uint32_t out[E / 4];
      if (pow2) {
        const uint64_t inv2 = pack2(inv, inv);
#pragma unroll
        for (int i = 0; i < E / 4; ++i) {
          const float2 a = unpack2(fmul2(bf16x2_to_f32x2(x[r][2 * i]), inv2));
          const float2 b = unpack2(fmul2(bf16x2_to_f32x2(x[r][2 * i + 1]), inv2));
          out[i] = pack_e4m3x2(a.x, a.y) | (pack_e4m3x2(b.x, b.y) << 16);
        }
      } else {
#pragma unroll
        for (int i = 0; i < E / 4; ++i)
          out[i] = pack_e4m3x2(__fdiv_rn(bf16_lo_to_f32(x[r][2 * i]), now), __fdiv_rn(bf16_hi_to_f32(x[r][2 * i]), now)) |
                   (pack_e4m3x2(__fdiv_rn(bf16_lo_to_f32(x[r][2 * i + 1]), now),
                                __fdiv_rn(bf16_hi_to_f32(x[r][2 * i + 1]), now)) << 16);
      }
      if constexpr (E == 8)
        *reinterpret_cast<uint2*>(codes + o * D) = make_uint2(out[0], out[1]);
      else
        *reinterpret_cast<uint32_t*>(codes + o * D) = out[0];
    }
  }
  if (h == 0 && now != old) *scale_at = now;
}

// The first token of a block in the call leads the block's run of adjacent tokens, and one warp takes the run
// for one kv head, so a block's scale has one writer.  Lanes 0-15 have the K rows, lanes 16-31 the V rows,
// D / 16 elements each, eight rows at a time: once for the maxima, and again (from L1) for the codes, which leaves
// registers for four CTAs an SM (all 16 rows kept: two, 69.0 against 59.6 us for 64000 tokens).  A CTA has a
// window of tokens, whose leaders times kv heads its warps share, and brings the window's rows into L2 while its
// slots are read (80.1 -> 73.2 us then).  The window is one token where there are few (64 decoding sequences, 8
// heads, 2.5 us; in windows of 16 one CTA would have 128 runs, 18.9 us), 16 where there are many (64000 tokens; a CTA
// a token, of which 15 of 16 end at once, 225 us), between them what lets all CTAs run at once (4096 tokens of
// prompts 8.6 us and of as many sequences 15.1; with half as many CTAs 7.5 and 19.9).  The bytes bound it: 64000
// tokens, 8 heads, d 128, 393 MB, 6.6 TB/s.
constexpr int kAppendWarps = 8;

template <int D>
__global__ void __launch_bounds__(kAppendWarps * 32, 4)
kv_append_f8_kernel(uint8_t* __restrict__ kq, uint8_t* __restrict__ vq, float* __restrict__ ks, float* __restrict__ vs,
                    const __nv_bfloat16* __restrict__ k, const __nv_bfloat16* __restrict__ v,
                    const int64_t* __restrict__ slots, int64_t T, int Hkv, int NB, int window, int32_t* err) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t tok0 = (int64_t)blockIdx.x * window;
  if (window > 1 && threadIdx.x == 0) {  // the window's rows on their way while its slots are read
    const uint32_t bytes = (uint32_t)(min((int64_t)window, T - tok0) * Hkv * D * 2);
    prefetch_l2(k + tok0 * Hkv * D, bytes);
    prefetch_l2(v + tok0 * Hkv * D, bytes);
  }
  uint32_t leaders;
  int64_t slot = -1;  // of token tok0 + lane: the window's, and 15 more for the run of its last
  {
    int code = 0;
    bool leads = false;
    const int64_t t = tok0 + lane;
    if (t < T) slot = __ldg(slots + t);
    if (lane < window && t < T) {
      const int64_t before = t > 0 ? __ldg(slots + t - 1) : -1;
      if (slot >= (int64_t)NB * 16) code = PKV_DEV_BAD_SLOT;
      else if (slot >= 0) {
        leads = before < 0 || (before >> 4) != (slot >> 4);
        if (!leads && before >= slot) code = PKV_DEV_BAD_SLOT;  // not above the one before
      }
    }
    if (warp == 0 && code != 0) record_error(err, code);
    leaders = __ballot_sync(kFullMask, leads);
  }
  const int runs = __popc(leaders);
  for (int item = warp; item < runs * Hkv; item += kAppendWarps) {
    const int nth = item / Hkv, g = item - nth * Hkv;
    const int at = (int)__fns(leaders, 0, nth + 1);
    const int64_t lane_slot = __shfl_sync(kFullMask, slot, (at + lane) & 31);
    append_run<D>(kq, vq, ks, vs, k, v, lane_slot, Hkv, tok0 + at, g, err);
  }
}

}  // namespace

size_t step_smem_bytes(int batch) { return sizeof(int) * (4 * (size_t)batch + 1); }

cudaError_t step_device_setup() {
  return cudaFuncSetAttribute((const void*)step_tables_kernel<kStepRunMost, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)step_smem_bytes(kMaxStepBatch));
}

cudaError_t launch_step_tables(const StepArgs& a, cudaStream_t stream) {
  StepArgs args = a;
  args.wide = ((reinterpret_cast<uintptr_t>(a.slot_mapping) | reinterpret_cast<uintptr_t>(a.positions)) & 15u) == 0;
  void* params[] = {&args};
  const bool large = a.max_tokens > kStepLarge || a.B > kStepLarge;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(large ? kStepCluster : 1);
  cfg.blockDim = dim3(a.B <= 512 && !large ? 256 : kStepThreads);
  cfg.dynamicSmemBytes = step_smem_bytes(a.B);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = large ? kStepCluster : 1;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = large ? 2 : 1;
  const void* f = !large              ? (const void*)step_tables_kernel<2, false>
                  : a.B <= kStepThreads ? (const void*)step_tables_kernel<1, true>
                                        : (const void*)step_tables_kernel<kStepRunMost, true>;
  return cudaLaunchKernelExC(&cfg, f, params);
}

cudaError_t launch_kv_append_f8(void* kq, void* vq, float* ks, float* vs, const void* k, const void* v,
                                const int64_t* slots, int64_t T, int Hkv, int D, int NB, int32_t* err, int sms,
                                cudaStream_t stream) {
  // the window: as many tokens as let all CTAs run at once (four on each SM)
  int window = (int)std::min<int64_t>(16, (T + 4 * sms - 1) / (4 * sms));
  const int64_t blocks = (T + window - 1) / window;
  void* params[] = {&kq, &vq, &ks, &vs, &k, &v, &slots, &T, &Hkv, &NB, &window, &err};
  const void* f = D == 128 ? (const void*)kv_append_f8_kernel<128> : (const void*)kv_append_f8_kernel<64>;
  return launch_pdl(f, dim3((unsigned)blocks), dim3(kAppendWarps * 32), 0, stream, params);
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
  uintptr_t words = reinterpret_cast<uintptr_t>(slot_mapping) & 4u;
  for (const void* p : {(const void*)block_tables, (const void*)context_lens_out, (const void*)query_starts,
                        (const void*)slot_mapping, (const void*)positions, (const void*)free_count_out,
                        (const void*)free_blocks, (const void*)free_count, (const void*)context_lens,
                        (const void*)new_tokens, (const void*)error_word})
    words |= reinterpret_cast<uintptr_t>(p) & 3u;
  if (words != 0) return PKV_ERR_ALIGNMENT;
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
  if (num_tokens < 0 || num_tokens >= (1ll << 33) / dims->num_kv_heads) return PKV_ERR_DIMS;
  if (num_tokens == 0) return PKV_OK;
  if (!k_codes || !v_codes || !k_scales || !v_scales || !k || !v || !slot_mapping) return PKV_ERR_NULL_POINTER;
  if (!aligned16(k_codes) || !aligned16(v_codes) || !aligned16(k) || !aligned16(v) ||
      ((reinterpret_cast<uintptr_t>(k_scales) | reinterpret_cast<uintptr_t>(v_scales) |
        reinterpret_cast<uintptr_t>(error_word)) & 3u) || (reinterpret_cast<uintptr_t>(slot_mapping) & 7u))
    return PKV_ERR_ALIGNMENT;
  int sms = 0;
  st = device_ready(&sms);
  if (st != PKV_OK) return st;
  return cuda_status(launch_kv_append_f8(k_codes, v_codes, k_scales, v_scales, k, v, slot_mapping, num_tokens,
                                         dims->num_kv_heads, dims->head_dim, dims->num_blocks, error_word, sms,
                                         static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
