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
//
// What has to move: 8 bytes a slot and kv head of scores and positions, as many written, and each moved row of K and
// of V read and written.  What bounds it (calls in a graph):
//  * 32 sequences of ~4000 bf16 tokens cut to 1540, 8 heads of 128: 65 us.  Profiled alone 16 for the selection and 51 for
//    the rows, at 71 % of peak DRAM (whole 256-byte rows, reads and writes mixed).
//  * 4 of 65536 cut to 8191: 74-77 us.  The kept rows behind the budget lie one or two in a block, and such single rows reach
//    some 50 % of peak DRAM (CTAs for twice or three times the rows in flight change nothing).  The selection's 45000 cycles
//    in a cluster of four are 9500 of loads and ten steps of 2500 to 4500 between barriers.  One sequence of 32768: 27 us, of
//    200000: 61.
//  * 64 of 1800 INT8 tokens, 270 moved a head: 18 us; 2 of 300: 11 us.  Two launches and a chain of latencies:
//    lengths, slots, histogram, scan, list, rank, words, lists, moves, then count, moves, rows.
#include <cooperative_groups.h>

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
  int4* moves;                   // [B * Hkv, budget] (from, to: block * 16 + offset, or -1; score bits, position)
  int32_t* to_slot;              // [B * Hkv, budget] the slot that each goes to
  int B, Hkv, NB, MB;
  int n_sink, n_recent, budget, trigger;
  int wide;                      // 1: rows of scores and slot_pos may be read and written four slots at a time
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
  const bool bad = s.L < 0 || s.L > a.MB * 16 || s.L > a.st.stride || s.L > PKV_MAX_EVICT_TOKENS || s.dropped < 0 || s.dropped > 0x7fffffff - s.L;
  s.err = bad ? PKV_DEV_BAD_CONTEXT_LEN : 0;
  s.cut = !bad && s.L > a.trigger;
  return s;
}

// Exclusive sum over the block; the total in *total.  `sums` holds 33 ints; two barriers.  T: int or uint32_t.
template <typename T>
__device__ __forceinline__ T block_sum_before(T v, int* sums, T* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  T x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T t = __shfl_up_sync(kFullMask, x, o);
    if (lane >= o) x += t;
  }
  __syncthreads();  // the sums of the call before have been read
  if (lane == 31) sums[warp] = (int)x;
  __syncthreads();
  T mine = lane < warps ? (T)sums[lane] : T(0), before = lane < warp ? mine : T(0);
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
// keys that are left (in the first round those of positive scores, from their own least to their greatest, so that
// the few exponents of real scores fill many bins; the others only if the positive ones do not suffice), then the bin that
// holds it, until at most a key a thread is left, which are ranked against one another.  32 bits are three rounds at most, and
// one more where the positive ones did not suffice.
// A row of few (sequence, kv head) pairs is shared by a cluster of CTAs, each with its part of the slots and
// all with the sums of the others' histograms.

constexpr int kEvictBins = 2048;
constexpr int kEvictMinThreads = 256, kEvictMaxThreads = 1024;
constexpr int kEvictBatch = 8, kEvictWide = 4;  // loads of slots, and of four of them, that a thread has in flight
constexpr int kEvictRanks = 8;  // CTAs of a cluster at most
constexpr int kMoveBatch = 4;   // likewise, moves
constexpr int kEvictSlots = 32768;  // of a CTA at most: 32 words of 32 for each of 32 warps
static_assert(PKV_MAX_EVICT_TOKENS == kEvictRanks * kEvictSlots, "the longest row");
constexpr uint32_t kProtectedKey = 0xffffffffu;
constexpr uint32_t kZeroKey = 0x80000000u;  // of a score of 0

__device__ __forceinline__ uint32_t order_key(float s) {
  if (s != s) return 0u;
  uint32_t u = __float_as_uint(s);
  if (u == 0x80000000u) u = 0u;  // -0.0 ranks as 0.0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

static_assert(kEvictBins >= 2 * kEvictMaxThreads, "two bins a thread");

template <bool CLUSTER>
struct EvictShared {
  alignas(8) int hist[kEvictBins];
  alignas(8) int all[CLUSTER ? kEvictBins : 2];  // the histogram of the row
  uint32_t list[kEvictMaxThreads];
  int sums[33];
  uint32_t least, most, key;  // least key of a positive score (less the key of zero), greatest unprotected one (plus 1)
  int guarded, n, bin, above, in, total, ties, cut;
  // what each CTA of the cluster found, written there by itself: as above, equal keys, places to fill and rows to go there
  uint32_t leasts[kEvictRanks], mosts[kEvictRanks];
  int guards[kEvictRanks], equals[kEvictRanks], tos[kEvictRanks], froms[kEvictRanks];
};

// One row, bg, by a CTA or a cluster, unless it shrinks from more than `upto` slots.  s_keys: keys of this CTA's slots, a
// multiple of four.
template <bool CLUSTER>
__device__ __forceinline__ void select_row(const EvictArgs& a, int bg, int upto, EvictShared<CLUSTER>& sh, uint32_t* s_keys) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = CLUSTER ? (int)cluster.num_blocks() : 1, rank = CLUSTER ? (int)cluster.block_rank() : 0;
  auto sync_all = [&] {
    if constexpr (CLUSTER) cluster.sync();
    else __syncthreads();
  };
  auto of_rank = [&](int r) { return CLUSTER ? cluster.map_shared_rank(&sh, r) : &sh; };
  const int tid = threadIdx.x, lane = tid & 31, T = blockDim.x, b = bg / a.Hkv;
  const EvictSeq s = evict_seq(a, b);
  const float* scores = a.st.scores + (size_t)bg * a.st.stride;
  const int32_t* slot_pos = a.st.slot_pos + (size_t)bg * a.st.stride;
  float* scores_out = a.st.scores_out + (size_t)bg * a.st.stride;
  int32_t* pos_out = a.st.slot_pos_out + (size_t)bg * a.st.stride;
  if (!s.cut) {
    if (tid == 0 && rank == 0) {
      a.count[bg] = 0;
      if (s.err != 0) record_error(a.err, s.err);
    }
    if (s.err == 0) {
      if (scores_out != scores)
        for (int i = rank * T + tid; i < s.L; i += ranks * T) scores_out[i] = scores[i];
      if (pos_out != slot_pos)
        for (int i = rank * T + tid; i < s.L; i += ranks * T) pos_out[i] = slot_pos[i];
    }
    return;
  }
  if (s.L > upto) return;
  if constexpr (CLUSTER) cluster_arrive();  // (what is written to another CTA comes after it has begun)
  if (tid == 0) {
    sh.least = 0xffffffffu;
    sh.most = 0u;
    sh.guarded = 0;
    sh.n = 0;
  }
  for (int i = tid; i < kEvictBins; i += T) sh.hist[i] = 0;
  __syncthreads();
  const int recent0 = s.L + s.dropped - a.n_recent;  // (n_recent <= budget < L)
  // this CTA's slots
  const int chunk = ((s.L + ranks - 1) / ranks + 3) & ~3, first = min(rank * chunk, s.L), end = min(first + chunk, s.L), own = end - first;
  auto place = [&](int p, int i) { return p >= 0 ? p : i + s.dropped; };
  auto make_key = [&](int p, int i, float score) {
    p = place(p, i);
    return p < a.n_sink || p >= recent0 ? kProtectedKey : order_key(score);
  };

  // ---- keys into shared memory; their range.  Scores and positions of the slots below the budget go out at once (those
  // that are filled get theirs with the rows); the ones past it are read again when what moves is known.
  {
    const bool same_scores = scores_out == scores, same_pos = pos_out == slot_pos;
    const int mid = min(end, a.budget) - first;
    uint32_t least = 0xffffffffu, most = 0u;
    int guarded = 0;
    bool nan = false;
    const float* sc = scores + first;
    const int32_t* sp = slot_pos + first;
    auto keep = [&](int j, float x, int p) {
      if (!same_scores) scores_out[first + j] = x;
      if (!same_pos || p < 0) pos_out[first + j] = place(p, first + j);
    };
    auto take = [&](int j, float x, int p) {
      const uint32_t k = make_key(p, first + j, x);
      nan |= k == 0u;
      guarded += k == kProtectedKey ? 1 : 0;
      least = min(least, k - (kZeroKey + 1u));  // (keys up to that of zero wrap to the end)
      most = max(most, k + 1u);                 // (the protected one wraps to 0)
      return k;
    };
    if (a.wide) {  // four slots a load (those past the end lie within the row)
      for (int v0 = tid; v0 < (own + 3) >> 2; v0 += kEvictWide * T) {
        float4 x[kEvictWide];
        int4 p[kEvictWide];
#pragma unroll
        for (int q = 0; q < kEvictWide; ++q) {
          const int v = v0 + q * T;
          if (4 * v < own) {
            x[q] = reinterpret_cast<const float4*>(sc)[v];
            p[q] = reinterpret_cast<const int4*>(sp)[v];
          }
        }
#pragma unroll
        for (int q = 0; q < kEvictWide; ++q) {
          const int j = 4 * (v0 + q * T);
          if (j >= own) continue;
          if (j + 3 < mid) {
            if (!same_scores) reinterpret_cast<float4*>(scores_out + first)[j >> 2] = x[q];
            const int i = first + j;
            const int4 y = make_int4(place(p[q].x, i), place(p[q].y, i + 1), place(p[q].z, i + 2), place(p[q].w, i + 3));
            if (!same_pos || (p[q].x | p[q].y | p[q].z | p[q].w) < 0) reinterpret_cast<int4*>(pos_out + first)[j >> 2] = y;
          } else if (j < mid) {  // one to three of the four
            keep(j, x[q].x, p[q].x);
            if (j + 1 < mid) keep(j + 1, x[q].y, p[q].y);
            if (j + 2 < mid) keep(j + 2, x[q].z, p[q].z);
          }
          uint4 k;
          k.x = take(j, x[q].x, p[q].x);
          k.y = j + 1 < own ? take(j + 1, x[q].y, p[q].y) : kProtectedKey;
          k.z = j + 2 < own ? take(j + 2, x[q].z, p[q].z) : kProtectedKey;
          k.w = j + 3 < own ? take(j + 3, x[q].w, p[q].w) : kProtectedKey;
          reinterpret_cast<uint4*>(s_keys)[j >> 2] = k;
        }
      }
    } else {
      for (int j0 = tid; j0 < own; j0 += kEvictBatch * T) {
        float x[kEvictBatch];
        int p[kEvictBatch];
#pragma unroll
        for (int q = 0; q < kEvictBatch; ++q) {
          if (j0 + q * T < own) {
            x[q] = sc[j0 + q * T];
            p[q] = sp[j0 + q * T];
          }
        }
#pragma unroll
        for (int q = 0; q < kEvictBatch; ++q) {
          const int j = j0 + q * T;
          if (j < own) s_keys[j] = take(j, x[q], p[q]);
          if (j < mid) keep(j, x[q], p[q]);
        }
      }
      // (the passes below read four keys at a time; a protected one is not counted there)
      if (tid < (-own & 3)) s_keys[own + tid] = kProtectedKey;
    }
    least = __reduce_min_sync(kFullMask, least);
    most = __reduce_max_sync(kFullMask, most);
    guarded = __reduce_add_sync(kFullMask, guarded);
    if (lane == 0) {
      atomicMin(&sh.least, least);
      atomicMax(&sh.most, most);
      atomicAdd(&sh.guarded, guarded);
    }
    if (nan) record_error(a.err, PKV_DEV_BAD_SCORE);
  }
  __syncthreads();
  uint32_t lo = sh.least, hi = sh.most;
  int need = a.budget - sh.guarded;  // among the unprotected, fewer than they are
  if constexpr (CLUSTER) {
    cluster_wait();
    if (tid < ranks) {
      auto* o = of_rank(tid);
      o->leasts[rank] = lo;
      o->mosts[rank] = hi;
      o->guards[rank] = a.budget - need;
    }
    cluster.sync();
    need = a.budget;
    for (int r = 0; r < ranks; ++r) {
      lo = min(lo, sh.leasts[r]);
      hi = max(hi, sh.mosts[r]);
      need -= sh.guards[r];
    }
  }
  hi -= 1u;
  lo += kZeroKey + 1u;

  // ---- the last place: keys above sh.key stay, and the first sh.ties of those equal to it, all of them unless sh.cut
  if (need <= 0) {
    if (tid == 0) {
      sh.key = kProtectedKey;
      sh.ties = a.budget;
      sh.cut = need < 0 ? 1 : 0;
    }
  } else {
    bool above_zero = true, clean = true;
    if (lo > hi || hi <= kZeroKey) {  // no score is positive
      lo = 0u;
      hi = kZeroKey;
      above_zero = false;
    }
    for (;;) {
      const uint32_t range = hi - lo;
      if (range == 0u && !above_zero) {
        if (tid == 0) {
          sh.key = lo;
          sh.ties = need;
          sh.cut = 1;
        }
        break;
      }
      const int shift = max(0, 32 - __clz(range) - 11);
      if (!clean) {
        for (int i = tid; i < kEvictBins; i += T) sh.hist[i] = 0;
        __syncthreads();
      }
      clean = false;
      const uint4* keys4 = reinterpret_cast<const uint4*>(s_keys);
#pragma unroll 2
      for (int v = tid; v < (own + 3) >> 2; v += T) {
        const uint4 k = keys4[v];
        if (k.x - lo <= range) atomicAdd(&sh.hist[(k.x - lo) >> shift], 1);
        if (k.y - lo <= range) atomicAdd(&sh.hist[(k.y - lo) >> shift], 1);
        if (k.z - lo <= range) atomicAdd(&sh.hist[(k.z - lo) >> shift], 1);
        if (k.w - lo <= range) atomicAdd(&sh.hist[(k.w - lo) >> shift], 1);
      }
      sync_all();
      if constexpr (CLUSTER) {  // each CTA adds up its share of the bins, for all
        const int share = kEvictBins / ranks;
        for (int i = rank * share + tid; i < (rank + 1) * share; i += T) {
          int n = 0;
#pragma unroll
          for (int r = 0; r < kEvictRanks; ++r)
            if (r < ranks) n += of_rank(r)->hist[i];
#pragma unroll
          for (int r = 0; r < kEvictRanks; ++r)
            if (r < ranks) of_rank(r)->all[i] = n;
        }
        cluster.sync();
      }
      // a thread's bins of the whole row, and the keys in the bins past them
      const int per = kEvictBins / T;  // two at least (T divides it)
      int h[kEvictBins / kEvictMinThreads], sum = 0;
      const int2* bins = reinterpret_cast<const int2*>((CLUSTER ? sh.all : sh.hist) + tid * per);
#pragma unroll
      for (int q = 0; q < kEvictBins / kEvictMinThreads; q += 2) {
        const int2 x = q < per ? bins[q >> 1] : make_int2(0, 0);
        h[q] = x.x;
        h[q + 1] = x.y;
      }
#pragma unroll
      for (int q = 0; q < kEvictBins / kEvictMinThreads; ++q) sum += h[q];
      int total;
      int above = block_sum_before(sum, sh.sums, &total);
      above = total - above - sum;
      if (tid == 0) sh.total = total;
#pragma unroll
      for (int q = kEvictBins / kEvictMinThreads - 1; q >= 0; --q) {
        if (q >= per) continue;
        if (above < need && need <= above + h[q]) {
          sh.bin = tid * per + q;
          sh.above = above;
          sh.in = h[q];
        }
        above += h[q];
      }
      __syncthreads();  // (and the histogram has been read)
      if (above_zero && sh.total < need) {  // all positive scores stay, and some of the others
        need -= sh.total;
        lo = 0u;
        hi = kZeroKey;
        above_zero = false;
        continue;
      }
      above_zero = false;
      lo += (uint32_t)sh.bin << shift;
      hi = min(hi, lo + ((1u << shift) - 1u));
      need -= sh.above;
      const int in = sh.in;
      if (in <= T && lo != hi) {
        auto* o = of_rank(0);
        const uint32_t width = hi - lo;
        auto list = [&](uint32_t k) {
          if (k - lo <= width) o->list[atomicAdd(&o->n, 1)] = k;
        };
#pragma unroll 2
        for (int v = tid; v < (own + 3) >> 2; v += T) {
          const uint4 k = keys4[v];
          list(k.x);
          list(k.y);
          list(k.z);
          list(k.w);
        }
        sync_all();
        if (rank == 0) {  // a warp a key
          for (int c = tid >> 5; c < in; c += T >> 5) {
            const uint32_t k = sh.list[c];
            int more = 0, same = 0;
            for (int i = lane; i < in; i += 32) {
              more += sh.list[i] > k ? 1 : 0;
              same += sh.list[i] == k ? 1 : 0;
            }
            more = __reduce_add_sync(kFullMask, more);
            same = __reduce_add_sync(kFullMask, same);
            if (lane < ranks && more < need && need <= more + same) {  // (every warp that has this key writes the same)
              auto* to = of_rank(lane);
              to->key = k;
              to->ties = need - more;
              to->cut = need < more + same ? 1 : 0;
            }
          }
        }
        break;
      }
    }
  }
  sync_all();
  const uint32_t last = sh.key;
  const int ties = sh.ties;

  // ---- the moves: a warp has a run of up to 32 words of 32 slots, a word a lane
  const int warp = tid >> 5, warps = T >> 5;
  const int run = ((own + warps - 1) / warps + 31) & ~31;  // (at most 1024: kEvictSlots)
  const int j0 = min(warp * run, own), j1 = min(j0 + run, own), n_words = (j1 - j0 + 31) >> 5;
  const uint32_t below = (1u << lane) - 1u;
  const bool cut = sh.cut != 0;
  int before = 0;  // equal keys before this warp's slots, where only some of them stay
  if (cut) {
    int equal = 0, total;
#pragma unroll 4
    for (int j = j0 + lane; j < j1; j += 32) equal += s_keys[j] == last ? 1 : 0;
    equal = __reduce_add_sync(kFullMask, equal);
    before = block_sum_before(lane == 0 ? equal : 0, sh.sums, &total);
    before = __shfl_sync(kFullMask, before, 0);
    if constexpr (CLUSTER) {
      if (tid < ranks) of_rank(tid)->equals[rank] = total;
      cluster.sync();
      for (int r = 0; r < rank; ++r) before += sh.equals[r];
    }
  }
  auto sum_to_lane = [&](int v) {  // over the lanes up to this one
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(kFullMask, v, o);
      if (lane >= o) v += t;
    }
    return v;
  };
  uint32_t stay = 0u;  // the lane's word: slots that stay
  if (!cut) {
#pragma unroll 4
    for (int t = 0; t < n_words; ++t) {
      const int j = j0 + 32 * t + lane;
      const uint32_t m = __ballot_sync(kFullMask, j < j1 && s_keys[min(j, own - 1)] >= last);
      stay = lane == t ? m : stay;
    }
  } else {
    uint32_t same = 0u;
#pragma unroll 4
    for (int t = 0; t < n_words; ++t) {
      const int j = j0 + 32 * t + lane;
      const uint32_t k = s_keys[min(j, own - 1)];
      const uint32_t m = __ballot_sync(kFullMask, j < j1 && k > last), e = __ballot_sync(kFullMask, j < j1 && k == last);
      stay = lane == t ? m : stay;
      same = lane == t ? e : same;
    }
    int take = ties - (before + sum_to_lane(__popc(same)) - __popc(same));  // of this word's equal keys, the lowest
    if (take <= 0) {
      same = 0u;
    } else if (take < __popc(same)) {
      uint32_t rest = same;
      for (; take > 0; --take) rest &= rest - 1u;
      same &= ~rest;
    }
    stay |= same;
  }
  const int w0 = j0 + 32 * lane;  // the word's first slot
  const int low = max(0, min(min(32, j1 - w0), a.budget - first - w0));
  const uint32_t front = low == 32 ? kFullMask : (1u << low) - 1u;
  const uint32_t gone = front & ~stay, late = stay & ~front;  // slots that are filled, slots that go there
  // both counts in a word (together at most kEvictSlots)
  const uint32_t upto_lane = (uint32_t)sum_to_lane(__popc(gone) | __popc(late) << 16);
  uint32_t all;
  const uint32_t of_warp = __shfl_sync(kFullMask, upto_lane, 31);
  const uint32_t start = __shfl_sync(kFullMask, block_sum_before(lane == 0 ? of_warp : 0u, sh.sums, &all), 0);
  const int to = (int)(start & 0xffffu), from = (int)(start >> 16), n_to = (int)(all & 0xffffu), n_from = (int)(all >> 16);
  int to0 = 0, from0 = 0, n = n_from;  // places of this CTA's first ones, and all moves
  if constexpr (CLUSTER) {
    if (tid < ranks) {
      auto* o = of_rank(tid);
      o->tos[rank] = n_to;
      o->froms[rank] = n_from;
    }
    cluster.sync();  // the last: nothing of another CTA is read or written past it
    n = 0;
    for (int r = 0; r < ranks; ++r) {
      if (r < rank) {
        to0 += sh.tos[r];
        from0 += sh.froms[r];
      }
      n += sh.froms[r];
    }
  }
  if (tid == 0 && rank == 0) a.count[bg] = n;
  // The CTA's slots as lists, in place of the keys; then all that the rows' kernel needs of them.  (That kernel joins
  // the two lists: a CTA writes its own part of each and reads no other's.)
  int* s_to = reinterpret_cast<int*>(s_keys);
  int* s_from = s_to + n_to;  // (n_to + n_from <= own)
  __syncthreads();            // the keys have been read
#pragma unroll 2
  for (int t = 0; t < n_words; ++t) {
    const uint32_t g = __shfl_sync(kFullMask, gone, t), l = __shfl_sync(kFullMask, late, t);
    const uint32_t upto_word = __shfl_sync(kFullMask, upto_lane, t);
    const int g1 = (int)(upto_word & 0xffffu), l1 = (int)(upto_word >> 16);
    const int i = first + j0 + 32 * t + lane;
    if ((g >> lane) & 1u) s_to[to + g1 - __popc(g & ~below)] = i;
    if ((l >> lane) & 1u) s_from[from + l1 - __popc(l & ~below)] = i;
  }
  __syncthreads();
  const int32_t* bt = a.block_tables + (size_t)b * a.MB;
  auto pool_slot = [&](int i, int blk) {
    if (blk >= 0 && blk < a.NB) return blk * 16 + (i & 15);
    record_error(a.err, PKV_DEV_BAD_BLOCK_ID);
    return -1;
  };
  int4* moves = a.moves + (size_t)bg * a.budget;
  int32_t* to_slot = a.to_slot + (size_t)bg * a.budget;
  for (int m0 = tid; m0 < max(n_to, n_from); m0 += kMoveBatch * T) {
    int i[kMoveBatch], j[kMoveBatch], blk_i[kMoveBatch], blk_j[kMoveBatch], p[kMoveBatch];
    float x[kMoveBatch];
#pragma unroll
    for (int q = 0; q < kMoveBatch; ++q) {
      const int m = m0 + q * T;
      if (m < n_from) {
        i[q] = s_from[m];
        x[q] = scores[i[q]];
        p[q] = slot_pos[i[q]];
        blk_i[q] = bt[i[q] >> 4];
      }
      if (m < n_to) {
        j[q] = s_to[m];
        blk_j[q] = bt[j[q] >> 4];
      }
    }
#pragma unroll
    for (int q = 0; q < kMoveBatch; ++q) {
      const int m = m0 + q * T;
      if (m < n_from) {
        int4* at = moves + from0 + m;
        at->x = pool_slot(i[q], blk_i[q]);
        at->z = __float_as_int(x[q]);
        at->w = place(p[q], i[q]);
      }
      if (m < n_to) {
        moves[to0 + m].y = pool_slot(j[q], blk_j[q]);
        to_slot[to0 + m] = j[q];
      }
    }
  }
  __syncthreads();  // the moved slots' values have been read
  const int z0 = max(first, a.budget), z1 = a.wide ? min((z0 + 3) & ~3, end) : end, z2 = a.wide ? max(z1, end & ~3) : end;
  for (int i = z0 + tid; i < z1; i += T) {
    scores_out[i] = 0.f;
    pos_out[i] = -1;
  }
  for (int i = z1 + 4 * tid; i < z2; i += 4 * T) {
    *reinterpret_cast<float4*>(scores_out + i) = make_float4(0.f, 0.f, 0.f, 0.f);
    *reinterpret_cast<int4*>(pos_out + i) = make_int4(-1, -1, -1, -1);
  }
  for (int i = z2 + tid; i < end; i += T) {
    scores_out[i] = 0.f;
    pos_out[i] = -1;
  }
}

// A CTA or cluster a row; or, MANY, few clusters that take the rows of more than `above` slots in turn.  (Apart: in the loop
// the compiler keeps the arguments in registers, which the CTA a row has no room for: 32 x 4000 tokens 72 us against 66.
// Held to 64 registers, 1024 threads a CTA, MANY spills 172 bytes a thread, the clusters without it 12, the CTA a row none.)
template <bool CLUSTER, bool MANY>
__global__ void __launch_bounds__(kEvictMaxThreads, 1) evict_select_kernel(const __grid_constant__ EvictArgs a, int above, int upto) {
  extern __shared__ __align__(16) uint32_t s_keys[];
  __shared__ EvictShared<CLUSTER> sh;
  const int ranks = CLUSTER ? (int)cooperative_groups::this_cluster().num_blocks() : 1;
  const int first = (int)blockIdx.x / ranks;
  grid_dependency_wait();
  grid_launch_dependents();
  if constexpr (!MANY) {
    select_row<CLUSTER>(a, first, upto, sh, s_keys);
  } else {
    const int pairs = a.B * a.Hkv, step = (int)gridDim.x / ranks, lane = threadIdx.x & 31;
    for (int base = first; base < pairs; base += 32 * step) {  // (every warp looks at the same 32)
      const int bg = base + lane * step;
      bool mine = false;
      if (bg < pairs) {
        const EvictSeq s = evict_seq(a, bg / a.Hkv);
        mine = s.cut && s.L > above;
      }
      for (uint32_t todo = __ballot_sync(kFullMask, mine); todo != 0u; todo &= todo - 1u)
        select_row<CLUSTER>(a, base + (__ffs(todo) - 1) * step, upto, sh, s_keys);
    }
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
// then every lane has eight 16-byte loads in flight before it stores.  CTAS: resident an SM (a few spilled words with five).
template <int RB, bool SCALES, int CTAS>
__global__ void __launch_bounds__(kMoveThreads, CTAS) evict_move_kernel(const __grid_constant__ EvictArgs a) {
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
  const int g = bg % a.Hkv;
  const int n = a.count[bg], lane = threadIdx.x & 31;
  const int4* moves = a.moves + (size_t)bg * a.budget;
  const int32_t* to_slot = a.to_slot + (size_t)bg * a.budget;
  constexpr int kWarps = kMoveThreads / 32;
  const int step = a.splits * kWarps * NR;
  int j0 = (part * kWarps + (int)(threadIdx.x >> 5)) * NR;
  // the lane's move of the NR at j (none: slots of -1), on its way while the rows before it are copied
  int4 m;
  int slot;
  auto fetch = [&](int j) {
    m = make_int4(-1, -1, 0, 0);
    slot = -1;
    if (lane < NR && j + lane < n) {
      m = moves[j + lane];
      slot = to_slot[j + lane];
    }
  };
  // 16-byte piece c % CPR of the row of a slot
  auto piece = [&](int s, int c) { return (((size_t)(s >> 4) * a.Hkv + g) * 16 + (s & 15)) * RB + (c % CPR) * 16; };
  fetch(j0);
  for (; j0 < n; j0 += step) {
    const bool live = m.x >= 0 && m.y >= 0;
    const int src = live ? m.x : -1, dst = m.y;
    if (slot >= 0) {
      a.st.scores_out[(size_t)bg * a.st.stride + slot] = __int_as_float(m.z);
      a.st.slot_pos_out[(size_t)bg * a.st.stride + slot] = m.w;
    }
    uint4 kb[4], vb[4];
    float ks = 0.f, vs = 0.f;
    uint32_t have = 0u;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int c = q * 32 + lane, from = __shfl_sync(kFullMask, src, c / CPR);
      if (from >= 0) {
        have |= 1u << q;
        kb[q] = __ldcs(reinterpret_cast<const uint4*>(a.k + piece(from, c)));
        vb[q] = __ldcs(reinterpret_cast<const uint4*>(a.v + piece(from, c)));
      }
    }
    if (SCALES && src >= 0) {
      ks = a.k_scales[piece(src, 0) / RB];
      vs = a.v_scales[piece(src, 0) / RB];
    }
    fetch(j0 + step);
    // (stores that do not stay in L2: 32 rows of 4000 tokens 80.9 -> 76.9 us)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int c = q * 32 + lane, to = __shfl_sync(kFullMask, dst, c / CPR);
      if ((have >> q) & 1u) {
        __stcs(reinterpret_cast<uint4*>(a.k + piece(to, c)), kb[q]);
        __stcs(reinterpret_cast<uint4*>(a.v + piece(to, c)), vb[q]);
      }
    }
    if (SCALES && src >= 0) {
      a.k_scales[piece(dst, 0) / RB] = ks;
      a.v_scales[piece(dst, 0) / RB] = vs;
    }
  }
}

constexpr int kShortSlots = 16384;  // of a row that a CTA takes where there are many: three CTAs' keys an SM

// `longest`: slots of a row at most, which the tables' width gives, not the sequences' lengths.  With few pairs a
// launch has clusters of as many CTAs a row as the SMs hold at once, of 4096 slots at least (a call for 4 x 8 rows of 32768, the
// longest that one CTA takes, cut to 4096: 51 us with a CTA a row, 45 with two, 40 with the four of this rule).  With many and wide tables one launch has a CTA for each row of up to
// kShortSlots, and another few clusters that take the longer ones in turn (256 sequences of 1800 INT8 tokens, 8 heads: 89 us in tables
// of 1920 slots, 114 in ones of 131072).
// Threads: as many as leave all CTAs on the SMs at once (64 registers each), of eight slots at least.
cudaError_t launch_select(const EvictArgs& a, int pairs, int longest, int sms, cudaStream_t stream) {
  EvictArgs args = a;
  args.wide = (a.st.stride & 3) == 0 && aligned16(a.st.scores) && aligned16(a.st.slot_pos) && aligned16(a.st.scores_out) &&
              aligned16(a.st.slot_pos_out);
  auto launch = [&](const void* kernel, int ctas, int ranks, int slots, int above) {
    const int most = ((slots + ranks - 1) / ranks + 3) & ~3;
    int threads = kEvictMinThreads;
    while (threads < kEvictMaxThreads && most > 8 * threads &&
           (ctas <= sms * (kEvictMaxThreads / (2 * threads)) || most > 32 * threads))
      threads *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = sizeof(uint32_t) * (size_t)most;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ranks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ranks > 1 ? 2 : 1;
    void* params[] = {&args, &above, &slots};
    return cudaLaunchKernelExC(&cfg, kernel, params);
  };
  const void* one = (const void*)evict_select_kernel<false, false>;
  int ranks = 1;
  while (ranks < 8 && pairs * 2 * ranks <= sms && longest / (2 * ranks) >= 4096) ranks *= 2;
  if (longest <= kShortSlots || (pairs * ranks <= sms && longest <= ranks * kEvictSlots))
    return launch(ranks > 1 ? (const void*)evict_select_kernel<true, false> : one, pairs * ranks, ranks, longest, 0);
  const cudaError_t e = launch(one, pairs, 1, kShortSlots, 0);
  if (e != cudaSuccess) return e;
  ranks = longest > 4 * kShortSlots ? 8 : longest > 2 * kShortSlots ? 4 : 2;
  return launch((const void*)evict_select_kernel<true, true>, std::max(1, sms / ranks) * ranks, ranks, longest, kShortSlots);
}

// bf16: five CTAs an SM where the kept rows behind the budget lie far apart, fewer than four of a block (4 sequences of 65536 cut
// to 8191: 74-77 us, 78-81 with four), and four where they lie close (32 of ~4000 cut to 1540: 64.8 us, 66.4 with
// five).  The border lies somewhere between these two points, and the tables' width stands for the lengths, which the host
// does not know: short sequences in wide tables get five, which costs the 2 % above.  INT8: four (256 of 1800 in tables of 131072 slots, which say
// far apart: 114 us, 118 with five).
const void* move_kernel(bool q8, int head_dim, bool apart) {
  if (q8) return head_dim == 128 ? (const void*)evict_move_kernel<128, true, 4> : (const void*)evict_move_kernel<64, true, 4>;
  if (apart) return head_dim == 128 ? (const void*)evict_move_kernel<256, false, 5> : (const void*)evict_move_kernel<128, false, 5>;
  return head_dim == 128 ? (const void*)evict_move_kernel<256, false, 4> : (const void*)evict_move_kernel<128, false, 4>;
}

size_t align256e(size_t x) { return (x + 255) & ~size_t(255); }

// int32 counts | int4 moves | int32 slots
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
  // table entries, slots of one sequence and of the pool, and (sequence, kv head) pairs are counted in 32 bits
  if ((long long)d->batch * d->max_blocks_per_seq >= (1ll << 30) ||
      (long long)d->max_blocks_per_seq * PKV_BLOCK_SIZE >= (1ll << 30) ||
      (long long)d->batch * d->num_kv_heads >= (1ll << 24) || d->num_blocks >= (1 << 27))
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
  a.moves = reinterpret_cast<int4*>(ws + evict_moves_offset(dims));
  const int pairs = a.B * a.Hkv;
  a.to_slot = reinterpret_cast<int32_t*>(a.moves + (size_t)a.budget * pairs);
  const int longest = std::min({state->stride, a.MB * PKV_BLOCK_SIZE, PKV_MAX_EVICT_TOKENS});  // cached tokens at most
  cudaStream_t cu = static_cast<cudaStream_t>(stream);
  const int RB = q8 ? dims->head_dim : 2 * dims->head_dim;
  if (pairs > 0) {
    const cudaError_t e = launch_select(a, pairs, longest, sms, cu);
    if (e != cudaSuccess) return cuda_status(e);
  }
  // CTAs for the rows of a pair: a warp's share each where that is not too many in all
  const int per_cta = kMoveThreads / 32 * (128 * 16 / RB);
  const int most = std::max(0, std::min(a.budget, longest - a.budget));  // moves of a pair at most
  const long long fill = pairs > 0 ? (16ll * sms + pairs - 1) / pairs : 1;
  a.splits = (int)std::max(1ll, std::min<long long>((most + per_cta - 1) / per_cta, fill));
  const void* f = move_kernel(q8, dims->head_dim, longest > 4ll * a.budget);
  void* params[] = {&a};
  return cuda_status(launch_pdl(f, dim3(1 + (unsigned)pairs * (unsigned)a.splits), dim3(kMoveThreads), 0, cu, params));
}

}  // namespace

cudaError_t evict_device_setup() {
  const int bytes = (int)(sizeof(uint32_t) * kEvictSlots);
  for (const void* f : {(const void*)evict_select_kernel<false, false>, (const void*)evict_select_kernel<true, false>,
                        (const void*)evict_select_kernel<true, true>}) {
    const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace pkv

using namespace pkv;

extern "C" {

size_t pkv_evict_workspace_bytes(const pkv_dims* dims, const pkv_evict_rules* rules) {
  if (check_evict(dims, rules) != PKV_OK) return 0;
  const size_t budget = (size_t)rules->n_sink + rules->k_top + rules->n_recent;
  return align256e(evict_moves_offset(dims) + (sizeof(int4) + sizeof(int32_t)) * budget * dims->batch * dims->num_kv_heads + 1);
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
