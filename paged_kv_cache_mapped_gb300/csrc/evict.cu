// evict.cu -- eviction from the paged cache by accumulated attention weight, in place, for sm_103a.
// Declared in pkv_evict.h.
//
// Of the L tokens of a (sequence, kv head) the `budget` greatest stay, by the order (protected, score, lower slot).
// The kept rows need not be in order, so only those behind the budget move, into the places of evicted ones:
// sources lie at or past the budget and destinations below it, so the moves are disjoint and need no
// order among them.  (Shifting the kept rows down instead would move nearly all of them, and each
// only after the row before it: 1536 rows a head instead of 256 where a sequence is cut from 1796 to 1540.)
//
// Two kernels:
//  * evict_select_kernel, a CTA for each (sequence, kv head): the threshold key, the lists of places and of
//    rows to go there, scores and positions.
//  * evict_move_kernel: the rows, many CTAs for each (sequence, kv head); one more CTA does the lengths and the
//    free stack.
#include <algorithm>

#include "kernels.h"
#include "pkv_evict.h"
#include "ptx.cuh"

namespace pkv {
namespace {

struct EvictArgs {
  unsigned char* k;
  unsigned char* v;
  float* k_scales;               // INT8 pools
  float* v_scales;
  const int32_t* block_tables;   // [B, MB]
  const int32_t* context_lens;   // [B]
  int32_t* context_lens_out;
  pkv_evict_state st;
  int32_t* free_blocks;          // or nullptr
  const int32_t* free_count;
  int32_t* free_count_out;
  int32_t* err;
  int32_t* count;                // [B * Hkv] moves of each (sequence, kv head)
  int2* moves;                   // [B * Hkv, budget] (slot from, slot to)
  int B, Hkv, NB, MB;
  int n_sink, n_recent, budget, trigger;
  int cached;                    // keys of a row that shared memory holds
  int splits;                    // CTAs that share the moves of one (sequence, kv head)
};

constexpr int kMaxEvictBatch = 4096;

// A sequence's length, its positions' offset, and whether it shrinks; err != 0: left alone without copies.
struct EvictSeq {
  int L, dropped, err;
  bool cut;
};

__device__ __forceinline__ EvictSeq evict_seq(const EvictArgs& a, int b) {
  EvictSeq s;
  s.L = a.context_lens[b];
  s.dropped = a.st.dropped[b];
  const bool bad = s.L < 0 || s.L > a.MB * 16 || s.L > a.st.stride || s.dropped < 0 || s.dropped > 0x7fffffff - s.L;
  s.err = bad ? PKV_DEV_BAD_CONTEXT_LEN : 0;
  s.cut = !bad && s.L > a.trigger;
  return s;
}

// Exclusive sum over the block; the total in *total.  `sums` holds 33 ints; two barriers.
__device__ __forceinline__ int block_sum_before(int v, int* sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(kFullMask, x, o);
    if (lane >= o) x += t;
  }
  __syncthreads();  // the sums of the call before have been read
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  int mine = lane < warps ? sums[lane] : 0, before = lane < warp ? mine : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    mine += __shfl_xor_sync(kFullMask, mine, o);
    before += __shfl_xor_sync(kFullMask, before, o);
  }
  *total = mine;
  return before + x - v;
}

// ------------------------------------------------------------------------------------ selection
//
// Keys are the scores mapped to uint32 in their order (a protected token has the largest, a NaN the
// smallest).  The key of the last place is found in rounds: a histogram of 2048 equal bins over the range of
// keys that are left (their own least to greatest in the first round, so that the few exponents of real
// scores fill many bins), then the bin that holds it, until at most a thread's worth of keys each
// is left, which are ranked against one another.  Three rounds at most end in a range of one key.

constexpr int kEvictBins = 2048;
constexpr int kEvictMaxThreads = 1024;
constexpr uint32_t kProtectedKey = 0xffffffffu;

__device__ __forceinline__ uint32_t order_key(float s) {
  if (s != s) return 0u;
  uint32_t u = __float_as_uint(s);
  if (u == 0x80000000u) u = 0u;  // -0.0 ranks as 0.0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(kEvictMaxThreads, 1) evict_select_kernel(const EvictArgs a) {
  extern __shared__ uint32_t s_keys[];  // [cached]
  __shared__ int s_hist[kEvictBins];
  __shared__ uint32_t s_list[kEvictMaxThreads];
  __shared__ int s_sums[33];
  __shared__ uint32_t s_min, s_max;
  __shared__ int s_protected, s_n, s_bin, s_above, s_in;
  __shared__ uint32_t s_key;
  __shared__ int s_ties;
  const int tid = threadIdx.x, lane = tid & 31, T = blockDim.x;
  const int bg = blockIdx.x, b = bg / a.Hkv;
  if (tid == 0) {
    s_min = 0xffffffffu;
    s_max = 0u;
    s_protected = 0;
  }
  grid_dependency_wait();
  grid_launch_dependents();
  const EvictSeq s = evict_seq(a, b);
  const float* scores = a.st.scores + (size_t)bg * a.st.stride;
  const int32_t* slot_pos = a.st.slot_pos + (size_t)bg * a.st.stride;
  float* scores_out = a.st.scores_out + (size_t)bg * a.st.stride;
  int32_t* pos_out = a.st.slot_pos_out + (size_t)bg * a.st.stride;
  if (!s.cut) {
    if (tid == 0) {
      a.count[bg] = 0;
      if (s.err != 0) record_error(a.err, s.err);
    }
    if (s.err == 0) {
      for (int i = tid; i < s.L; i += T) {
        if (scores_out != scores) scores_out[i] = scores[i];
        if (pos_out != slot_pos) pos_out[i] = slot_pos[i];
      }
    }
    return;
  }
  __syncthreads();
  const int L = s.L, recent0 = L + s.dropped - a.n_recent;  // (n_recent <= budget < L)
  auto position = [&](int i) {
    const int p = slot_pos[i];
    return p >= 0 ? p : i + s.dropped;
  };
  auto key_of = [&](int i) {
    const int p = position(i);
    return p < a.n_sink || p >= recent0 ? kProtectedKey : order_key(scores[i]);
  };
  auto key_at = [&](int i) { return i < a.cached ? s_keys[i] : key_of(i); };

  // ---- keys into shared memory; their range
  uint32_t least = 0xffffffffu, most = 0u;
  int prot = 0;
  bool nan = false;
  for (int i = tid; i < L; i += T) {
    const uint32_t k = key_of(i);
    if (i < a.cached) s_keys[i] = k;
    nan |= k == 0u;
    if (k == kProtectedKey) {
      ++prot;
    } else {
      least = min(least, k);
      most = max(most, k);
    }
  }
  least = __reduce_min_sync(kFullMask, least);
  most = __reduce_max_sync(kFullMask, most);
  prot = __reduce_add_sync(kFullMask, prot);
  if (lane == 0) {
    atomicMin(&s_min, least);
    atomicMax(&s_max, most);
    atomicAdd(&s_protected, prot);
  }
  if (nan) record_error(a.err, PKV_DEV_BAD_SCORE);
  __syncthreads();

  // ---- the last place: keys above s_key stay, and the first s_ties of those equal to it
  int need = a.budget - s_protected;  // among the unprotected, fewer than they are
  if (need <= 0) {
    if (tid == 0) {
      s_key = kProtectedKey;
      s_ties = a.budget;
    }
  } else {
    uint32_t lo = s_min, hi = s_max;
    for (;;) {
      const uint32_t range = hi - lo;
      if (range == 0u) {
        if (tid == 0) {
          s_key = lo;
          s_ties = need;
        }
        break;
      }
      const int shift = max(0, 32 - __clz(range) - 11);
      for (int i = tid; i < kEvictBins; i += T) s_hist[i] = 0;
      if (tid == 0) s_n = 0;
      __syncthreads();
      int at_lo = 0;  // the least key is often that of many (tokens without any weight)
      for (int i = tid; i < L; i += T) {
        const uint32_t k = key_at(i);
        if (k == lo) ++at_lo;
        else if (k > lo && k <= hi) atomicAdd(&s_hist[(k - lo) >> shift], 1);
      }
      at_lo = __reduce_add_sync(kFullMask, at_lo);
      if (lane == 0 && at_lo > 0) atomicAdd(&s_hist[0], at_lo);
      __syncthreads();
      const int per = kEvictBins / T;  // (T divides it)
      int sum = 0;
      for (int q = 0; q < per; ++q) sum += s_hist[tid * per + q];
      int total;
      int above = block_sum_before(sum, s_sums, &total);
      above = total - above - sum;  // keys in bins past this thread's
      for (int q = per - 1; q >= 0; --q) {
        const int h = s_hist[tid * per + q];
        if (above < need && need <= above + h) {
          s_bin = tid * per + q;
          s_above = above;
          s_in = h;
        }
        above += h;
      }
      __syncthreads();
      lo += (uint32_t)s_bin << shift;
      hi = min(hi, lo + ((1u << shift) - 1u));
      need -= s_above;
      const int in = s_in;
      if (in <= T && lo != hi) {
        for (int i = tid; i < L; i += T) {
          const uint32_t k = key_at(i);
          if (k >= lo && k <= hi) s_list[atomicAdd(&s_n, 1)] = k;
        }
        __syncthreads();
        if (tid < in) {
          const uint32_t k = s_list[tid];
          int more = 0, same = 0;
          for (int i = 0; i < in; ++i) {
            more += s_list[i] > k ? 1 : 0;
            same += s_list[i] == k ? 1 : 0;
          }
          if (more < need && need <= more + same) {  // (every thread that has this key writes the same)
            s_key = k;
            s_ties = need - more;
          }
        }
        break;
      }
    }
  }
  __syncthreads();
  const uint32_t last = s_key;
  const int ties = s_ties;

  // ---- the moves: a thread has a run of slots (of an odd length, which spreads the banks)
  const int run = ((L + T - 1) / T) | 1;
  const int i0 = min(tid * run, L), i1 = min(i0 + run, L);
  int equal = 0;
  for (int i = i0; i < i1; ++i) equal += key_at(i) == last ? 1 : 0;
  int total;
  const int equal0 = block_sum_before(equal, s_sums, &total);
  int2* moves = a.moves + (size_t)bg * a.budget;
  int seen = equal0, to = 0, from = 0;
  for (int i = i0; i < i1; ++i) {
    const uint32_t k = key_at(i);
    const bool keep = k > last || (k == last && seen < ties);
    seen += k == last ? 1 : 0;
    to += !keep && i < a.budget ? 1 : 0;
    from += keep && i >= a.budget ? 1 : 0;
  }
  int n;
  to = block_sum_before(to, s_sums, &total);
  from = block_sum_before(from, s_sums, &n);
  seen = equal0;
  for (int i = i0; i < i1; ++i) {
    const uint32_t k = key_at(i);
    const bool keep = k > last || (k == last && seen < ties);
    seen += k == last ? 1 : 0;
    if (!keep && i < a.budget) moves[to++].y = i;
    if (keep && i >= a.budget) moves[from++].x = i;
  }
  if (tid == 0) a.count[bg] = n;

  // ---- scores and positions: those that stay, those that move, then the slots behind
  for (int i = tid; i < a.budget; i += T) {
    if (scores_out != scores) scores_out[i] = scores[i];
    pos_out[i] = position(i);
  }
  __syncthreads();
  for (int j = tid; j < n; j += T) {
    const int2 m = moves[j];
    scores_out[m.y] = scores[m.x];
    pos_out[m.y] = position(m.x);
  }
  __syncthreads();
  for (int i = a.budget + tid; i < L; i += T) {
    scores_out[i] = 0.f;
    pos_out[i] = -1;
  }
}

// ------------------------------------------------------------------------------------ the rows

constexpr int kMoveThreads = 256;
constexpr int kPushEach = 8;  // blocks that a thread of the last CTA takes at a time

// Lengths and the free stack, by one CTA: the sequences in groups of a CTA's threads, and the blocks of a
// group's sequences as one list.
__device__ __forceinline__ void evict_tables(const EvictArgs& a) {
  __shared__ int s_start[kMoveThreads + 1];
  __shared__ int s_sums[33];
  const int tid = threadIdx.x;
  const int kept = (a.budget + 15) >> 4;
  int top = a.free_blocks != nullptr ? a.free_count[0] : 0;
  const bool push = a.free_blocks != nullptr && top >= 0 && top <= a.NB;
  if (a.free_blocks != nullptr && !push && tid == 0) record_error(a.err, PKV_DEV_NO_BLOCKS);
  for (int b0 = 0; b0 < a.B; b0 += kMoveThreads) {
    const int b = b0 + tid;
    int back = 0;
    if (b < a.B) {
      const EvictSeq s = evict_seq(a, b);
      a.context_lens_out[b] = s.cut ? a.budget : s.L;
      a.st.dropped_out[b] = s.cut ? s.dropped + s.L - a.budget : s.dropped;
      back = s.cut ? ((s.L + 15) >> 4) - kept : 0;
    }
    if (!push) continue;
    int all;
    const int at = block_sum_before(back, s_sums, &all);
    s_start[tid] = at;
    __syncthreads();
    for (int r0 = 0; r0 < all; r0 += kMoveThreads * kPushEach) {
      int id[kPushEach], good = 0;
#pragma unroll
      for (int q = 0; q < kPushEach; ++q) {
        const int r = r0 + tid * kPushEach + q;
        id[q] = -1;
        if (r < all) {
          const int w = owner_of(s_start, kMoveThreads, r);
          id[q] = a.block_tables[(size_t)(b0 + w) * a.MB + kept + (r - s_start[w])];
          if (id[q] < 0 || id[q] >= a.NB) {
            id[q] = -1;
            record_error(a.err, PKV_DEV_BAD_BLOCK_ID);
          }
        }
        good += id[q] >= 0 ? 1 : 0;
      }
      int n;
      int to = top + block_sum_before(good, s_sums, &n);
#pragma unroll
      for (int q = 0; q < kPushEach; ++q) {
        if (id[q] < 0) continue;
        if (to < a.NB) a.free_blocks[to] = id[q];
        else record_error(a.err, PKV_DEV_NO_BLOCKS);
        ++to;
      }
      top = min(top + n, a.NB);
    }
    __syncthreads();  // the starts have been read
  }
  if (a.free_blocks != nullptr && tid == 0) a.free_count_out[0] = top;
}

// RB: bytes of a row; SCALES: INT8 pools.  A warp takes 2 KB of K rows and as much of V at a time: lanes find the rows,
// then every lane has eight 16-byte loads in flight before it stores.
template <int RB, bool SCALES>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs a) {
  constexpr int CPR = RB / 16, NR = 128 / CPR;  // 16-byte pieces of a row; rows of a warp at a time
  static_assert(NR <= 32 && NR * CPR == 4 * 32, "four pieces of K and of V a lane");
  grid_dependency_wait();
  grid_launch_dependents();
  if (blockIdx.x == 0) {
    evict_tables(a);
    return;
  }
  const int item = (int)blockIdx.x - 1;
  const int bg = item / a.splits, part = item - bg * a.splits;
  const int b = bg / a.Hkv, g = bg - b * a.Hkv;
  const int n = a.count[bg], lane = threadIdx.x & 31;
  const int2* moves = a.moves + (size_t)bg * a.budget;
  constexpr int kWarps = kMoveThreads / 32;
  for (int j0 = (part * kWarps + (int)(threadIdx.x >> 5)) * NR; j0 < n; j0 += a.splits * kWarps * NR) {
    long long src = -1, dst = -1;  // pool rows of this lane's move
    if (lane < NR && j0 + lane < n) {
      const int2 m = moves[j0 + lane];
      const int32_t* bt = a.block_tables + (size_t)b * a.MB;
      const int from = bt[m.x >> 4], to = bt[m.y >> 4];
      if (from < 0 || from >= a.NB || to < 0 || to >= a.NB) {
        record_error(a.err, PKV_DEV_BAD_BLOCK_ID);
      } else {
        src = ((long long)from * a.Hkv + g) * 16 + (m.x & 15);
        dst = ((long long)to * a.Hkv + g) * 16 + (m.y & 15);
      }
    }
    uint4 kb[4], vb[4];
    long long at[4];
    float ks = 0.f, vs = 0.f;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int c = q * 32 + lane;
      const long long from = __shfl_sync(kFullMask, src, c / CPR);
      at[q] = __shfl_sync(kFullMask, dst, c / CPR);
      if (at[q] >= 0) {
        kb[q] = reinterpret_cast<const uint4*>(a.k + from * RB)[c % CPR];
        vb[q] = reinterpret_cast<const uint4*>(a.v + from * RB)[c % CPR];
      }
    }
    if (SCALES && src >= 0) {
      ks = a.k_scales[src];
      vs = a.v_scales[src];
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int c = q * 32 + lane;
      if (at[q] >= 0) {
        reinterpret_cast<uint4*>(a.k + at[q] * RB)[c % CPR] = kb[q];
        reinterpret_cast<uint4*>(a.v + at[q] * RB)[c % CPR] = vb[q];
      }
    }
    if (SCALES && src >= 0) {
      a.k_scales[dst] = ks;
      a.v_scales[dst] = vs;
    }
  }
}

// Keys that shared memory holds; a longer row's others are worked out again from memory at each pass.
constexpr int kEvictCachedKeys = 49152;

size_t align256e(size_t x) { return (x + 255) & ~size_t(255); }

// int32 counts | int2 moves
size_t evict_moves_offset(const pkv_dims* d) {
  return align256e(sizeof(int32_t) * (size_t)d->batch * d->num_kv_heads);
}

int check_evict(const pkv_dims* d, const pkv_evict_rules* r) {
  const int st = check_dims(d, false);
  if (st != PKV_OK) return st;
  if (r == nullptr) return PKV_ERR_NULL_POINTER;
  if (d->batch > kMaxEvictBatch) return PKV_ERR_DIMS;
  if (r->n_sink < 0 || r->k_top < 0 || r->n_recent < 0) return PKV_ERR_ARGUMENT;
  const long long budget = (long long)r->n_sink + r->k_top + r->n_recent;
  if (budget >= (1ll << 30)) return PKV_ERR_ARGUMENT;
  // table entries, slots of one sequence, and (sequence, kv head) pairs are counted in 32 bits
  if ((long long)d->batch * d->max_blocks_per_seq >= (1ll << 30) ||
      (long long)d->max_blocks_per_seq * PKV_BLOCK_SIZE >= (1ll << 30) ||
      (long long)d->batch * d->num_kv_heads >= (1ll << 24))
    return PKV_ERR_DIMS;
  return PKV_OK;
}

int evict_common(void* k, void* v, float* ks, float* vs, const int32_t* block_tables, const int32_t* context_lens,
                 int32_t* context_lens_out, const pkv_evict_state* state, const pkv_evict_rules* rules,
                 int32_t* free_blocks, const int32_t* free_count, int32_t* free_count_out, void* workspace,
                 size_t workspace_bytes, const pkv_dims* dims, int32_t* err, void* stream, bool q8) {
  int st = check_evict(dims, rules);
  if (st != PKV_OK) return st;
  if (state == nullptr) return PKV_ERR_NULL_POINTER;
  if (state->stride < 0) return PKV_ERR_DIMS;
  if (free_blocks != nullptr && (!free_count || !free_count_out)) return PKV_ERR_NULL_POINTER;
  if (dims->batch == 0 && free_blocks == nullptr) return PKV_OK;
  if (dims->batch > 0) {
    if (!block_tables || !context_lens || !context_lens_out || !state->dropped || !state->dropped_out)
      return PKV_ERR_NULL_POINTER;
    if (state->stride > 0 && (!state->scores || !state->scores_out || !state->slot_pos || !state->slot_pos_out))
      return PKV_ERR_NULL_POINTER;
    if (dims->num_blocks > 0 && (!k || !v || (q8 && (!ks || !vs)))) return PKV_ERR_NULL_POINTER;
    if (!workspace || workspace_bytes < pkv_evict_workspace_bytes(dims, rules)) return PKV_ERR_WORKSPACE;
  }
  uintptr_t words = 0;
  for (const void* p : {(const void*)block_tables, (const void*)context_lens, (const void*)context_lens_out,
                        (const void*)state->scores, (const void*)state->scores_out, (const void*)state->slot_pos,
                        (const void*)state->slot_pos_out, (const void*)state->dropped, (const void*)state->dropped_out,
                        (const void*)free_blocks, (const void*)free_count, (const void*)free_count_out, (const void*)err})
    words |= reinterpret_cast<uintptr_t>(p) & 3u;
  if (words != 0 || !aligned16(k) || !aligned16(v) || !aligned16(ks) || !aligned16(vs) || !aligned16(workspace))
    return PKV_ERR_ALIGNMENT;
  int sms = 0;
  st = device_ready(&sms);
  if (st != PKV_OK) return st;
  EvictArgs a{};
  a.k = static_cast<unsigned char*>(k);
  a.v = static_cast<unsigned char*>(v);
  a.k_scales = ks;
  a.v_scales = vs;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.context_lens_out = context_lens_out;
  a.st = *state;
  a.free_blocks = free_blocks;
  a.free_count = free_count;
  a.free_count_out = free_count_out;
  a.err = err;
  a.B = dims->batch;
  a.Hkv = dims->num_kv_heads;
  a.NB = dims->num_blocks;
  a.MB = dims->max_blocks_per_seq;
  a.n_sink = rules->n_sink;
  a.n_recent = rules->n_recent;
  a.budget = rules->n_sink + rules->k_top + rules->n_recent;
  a.trigger = std::max(rules->trigger, a.budget);
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  a.count = reinterpret_cast<int32_t*>(ws);
  a.moves = reinterpret_cast<int2*>(ws + evict_moves_offset(dims));
  const int longest = std::min(state->stride, a.MB * PKV_BLOCK_SIZE);  // cached tokens at most
  const int pairs = a.B * a.Hkv;
  cudaStream_t cu = static_cast<cudaStream_t>(stream);
  const int RB = q8 ? dims->head_dim : 2 * dims->head_dim;
  if (pairs > 0) {
    a.cached = std::min(longest, kEvictCachedKeys);
    const int threads = longest > 4096 ? 1024 : longest > 1024 ? 512 : 256;
    void* params[] = {&a};
    const cudaError_t e = launch_pdl((const void*)evict_select_kernel, dim3((unsigned)pairs), dim3(threads),
                                     sizeof(uint32_t) * (size_t)a.cached, cu, params);
    if (e != cudaSuccess) return cuda_status(e);
  }
  // CTAs for the rows of a pair: a warp's share each where that is not too many in all
  const int per_cta = kMoveThreads / 32 * (128 * 16 / RB);
  const int most = std::max(0, std::min(a.budget, longest - a.budget));  // moves of a pair at most
  const long long fill = pairs > 0 ? (64ll * sms + pairs - 1) / pairs : 1;
  a.splits = (int)std::max(1ll, std::min<long long>((most + per_cta - 1) / per_cta, fill));
  const void* f = q8 ? (dims->head_dim == 128 ? (const void*)evict_move_kernel<128, true> : (const void*)evict_move_kernel<64, true>)
                     : (dims->head_dim == 128 ? (const void*)evict_move_kernel<256, false> : (const void*)evict_move_kernel<128, false>);
  void* params[] = {&a};
  return cuda_status(launch_pdl(f, dim3(1 + (unsigned)pairs * (unsigned)a.splits), dim3(kMoveThreads), 0, cu, params));
}

}  // namespace

cudaError_t evict_device_setup() {
  return cudaFuncSetAttribute((const void*)evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)(sizeof(uint32_t) * kEvictCachedKeys));
}

}  // namespace pkv

using namespace pkv;

extern "C" {

size_t pkv_evict_workspace_bytes(const pkv_dims* dims, const pkv_evict_rules* rules) {
  if (check_evict(dims, rules) != PKV_OK) return 0;
  const size_t budget = (size_t)rules->n_sink + rules->k_top + rules->n_recent;
  return align256e(evict_moves_offset(dims) + sizeof(int2) * budget * dims->batch * dims->num_kv_heads + 1);
}

int pkv_kv_evict(void* k_cache, void* v_cache, const int32_t* block_tables, const int32_t* context_lens,
                 int32_t* context_lens_out, const pkv_evict_state* state, const pkv_evict_rules* rules,
                 int32_t* free_blocks, const int32_t* free_count, int32_t* free_count_out, void* workspace,
                 size_t workspace_bytes, const pkv_dims* dims, int32_t* error_word, void* stream) {
  return evict_common(k_cache, v_cache, nullptr, nullptr, block_tables, context_lens, context_lens_out, state, rules,
                      free_blocks, free_count, free_count_out, workspace, workspace_bytes, dims, error_word, stream, false);
}

int pkv_kv_evict_q8(void* k_codes, void* v_codes, float* k_scales, float* v_scales, const int32_t* block_tables,
                    const int32_t* context_lens, int32_t* context_lens_out, const pkv_evict_state* state,
                    const pkv_evict_rules* rules, int32_t* free_blocks, const int32_t* free_count,
                    int32_t* free_count_out, void* workspace, size_t workspace_bytes, const pkv_dims* dims,
                    int32_t* error_word, void* stream) {
  return evict_common(k_codes, v_codes, k_scales, v_scales, block_tables, context_lens, context_lens_out, state, rules,
                      free_blocks, free_count, free_count_out, workspace, workspace_bytes, dims, error_word, stream, true);
}

}  // extern "C"
