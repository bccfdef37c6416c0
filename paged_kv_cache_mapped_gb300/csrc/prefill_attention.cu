// prefill_attention.cu -- attention of many query tokens per sequence over the paged cache, with
// score rules, on the 5th-generation tensor cores (sm_103a).  Declared in pkv_step.h.
//
// out[r, h] = sum_t p_t V_t, p = softmax over the keys t that row r sees, of
//   x_t = cap(scale q . K_t) - slope_h |i - t|,
// i the row's position, visible keys [lo, i] and the prefix [0, pre).
//
// Three kernels:
//  * prefill_plan_kernel (one CTA) checks every sequence and cuts the batch into work items: one or two row
//    tiles of 128 rows (tokens x the G heads of a kv head) of one sequence, and, where there are fewer of
//    those than the GPU holds, a share of their keys.
//  * prefill_attention_kernel runs the items, each for one kv head, taken by ticket by one CTA (two row tiles
//    an item) or two CTAs (one) per SM.  Q tiles and a ring of 128-key K and V tiles (8 cache blocks each) come by TMA.
//    S = Q K^T goes into tensor memory, 64 keys a step, and O += P V takes P from where S was and V as it
//    lies (MN-major).  Each row tile has 4 softmax warps, a row a thread: they read S, apply the
//    rules, keep the running maximum (moved only when exceeded by 2^8, and O rescaled then) and sum,
//    and write P.  The softmax of one step runs under the products of the next, and of the other row tile.
//  * prefill_merge_kernel joins the shares of split items by their maxima and sums.
// What bounds it: long chunks the chain of a step (products, load, maximum, exponentials, store) at two softmax warps a
// scheduler, no unit being full (4096 tokens on 16384 keys, 32 / 8 heads, d 128: 720-750 us, 1290-1340 TFLOP/s, 67-70 % of
// the measured bf16 rate; tensor pipe 56 %, issue 47 %, exponentials 28 %; with a distance bias 810 us; capped 836-871 where the
// scores stay below a fifth of the cap, 1020-1045 below 0.8 of it, 1490-1520 beyond); d 64 the same chain, its
// products halved (4 prompts of 3000, 8 heads, bias and a window of 1000: 57-59 us, tensor pipe 16 %, issue 36 %); many single
// tokens the loads in flight, a K and a V tile a CTA (64 on 2000 keys each 110 us, 4.8 TB/s, DRAM at 62 % of its peak; 4
// on 131072 336-338 us, 6.4 TB/s); small batches the chain of plan, first loads and merge (one token on 200 keys 19 us).
// A CTA holds two row tiles because every K and V tile that comes into shared memory then serves 256 rows.
// P is rounded to bf16 for the product (the sum takes it in fp32).  Rows over more than kTwoTermTiles key
// tiles take that one term: its error, at most 2^-8 of each weight, is of the size of a bf16 output's own rounding
// where a few keys or equal weights carry a row, and averages out where many unequal ones do.  Shorter rows, where few weights may carry the result, add the
// remainder as a second term, which costs half as many MMAs again (all rows in two terms: chunk of 4096 on 16384
// 937 us against 730; none: 24 mixed sequences 26.3 against 28.5).
// Non-finite V: a masked key's weight is 0, and 0 * NaN is NaN, so V rows past the sequence are cleared,
// and an output row that owes a NaN to a masked key is computed again over what it sees.
// Every wait is bounded; bad block ids are cleared tiles, recorded.
#include <algorithm>
#include <cmath>
#include <cstddef>
#include <type_traits>

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

constexpr int kKeys = 128;           // keys per K/V tile in shared memory
constexpr int kTileBlocks = kKeys / 16;
constexpr int kStep = 64;            // keys of a softmax step: half a tile
constexpr int kStepBlocks = kStep / 16;
constexpr int kHalf = kKeys * 128;   // bytes of one 64-element half of a tile
constexpr float kSlack = 8.0f;       // the running maximum moves only when exceeded by this (base 2)
constexpr int kTwoTermTiles = 4;     // rows over at most this many key tiles take P as two bf16 terms (above)
constexpr int kMinChunk = 4;         // key tiles of a share at least where items outnumber the CTAs

template <int D, int NT>
struct Geo {
  static constexpr int kHalves = D / 64;
  static constexpr int kTile = kHalves * kHalf;  // bytes of a Q, K or V tile
  static constexpr int kSlots = NT == 2 ? (D == 128 ? 4 : 8) : (D == 128 ? 2 : 5);
  static constexpr int kSoftmaxWarps = NT * 4;  // a row a thread
  // and a producer, two issuers (one for each row tile, or for each product of the one), the ticket taker
  static constexpr int kThreads = NT * 128 + 128;
  static constexpr int kProducer = kSoftmaxWarps, kIssuer = kProducer + 1, kTicket = kIssuer + 2;
  static constexpr int kCtas = NT == 1 ? 2 : 1;  // per SM (shared and tensor memory allow no more)
  // Registers a thread: a launch gives every warp the same, which the softmax warps (their logits are in
  // registers) then take from the others.  NT = 2: 384 x 168 = 256 x 216 + 128 x 72; NT = 1 (two CTAs):
  // 256 x 128 = 128 x 184 + 128 x 72.
  static constexpr int kLaunchRegs = NT == 2 ? 168 : 128;
  static constexpr int kSoftmaxRegs = NT == 2 ? 216 : 184, kOtherRegs = 72;
  static_assert(kSoftmaxWarps * 32 * kSoftmaxRegs + 128 * kOtherRegs <= kThreads * kLaunchRegs, "register split");
  static constexpr uint32_t kTmemCols = NT * (2 * kStep + D) <= 256 ? 256 : 512;
  static constexpr size_t kSmem = 1024 + (size_t)(NT + kSlots) * kTile;
};

// ------------------------------------------------------------------------------------ the plan
//
// Sequence b has ceil(n_b / (NT R)) row tile groups ("entries") of R = 128 / G tokens a tile; entry e has kt_e key
// tiles (an upper bound where documents hide some), and Hkv items of it make P = entries * Hkv.  `slots` CTAs
// run at a time.
//  * P < slots: every entry is cut into shares of at most c key tiles, c chosen among ktmax / s for a few s for
//    the least estimate of the end, an item costing a tile beside its own: c + 1 where all shares run at once,
//    else the smaller of the mean + c (any list schedule) and the rounds times c + 1; and a tile's time plus one
//    for 4000 rows where rows have to be merged (2 x 300 tokens of 1000, 19200 rows: 30 us whole, 43 us in
//    shares; 2 x 114 tokens of ~1550, 12768 rows: 35.9 us in shares, 38.5 whole; 4 single tokens of 131072 keys: 342 us in 19 shares each, 359 in 16; 3 sequences of ~500 keys, 12 tokens:
//    18.4 us in shares of a tile, 24.8 whole).
//  * P >= slots: entries above one and a half times the fair share W / slots are cut to that.  If there are
//    none, the last P mod slots items, which would leave most CTAs idle for a whole item, are cut in s shares each (chunk of 4096 on 16384,
//    512 items on 152 CTAs: 56 items in two shares, capped 0.99 -> 0.87 ms).
// The shares of split entries number at most 2 slots, which bounds the partial rows.  The list has the entries
// with more than half of ktmax first, a sequence's last rows first within either part.
struct Entry {
  int b, tile, ntile, tokens, kt;
};

// seq: (queries, keys, prefix) of each sequence.
__device__ __forceinline__ Entry plan_entry(const PrefillAttnArgs& a, const int* base, const int* seq, int e, int per_item) {
  Entry x;
  x.b = owner_of(base, a.B, e);
  const struct { int n, L, pre; } s = {seq[3 * x.b], seq[3 * x.b + 1], seq[3 * x.b + 2]};
  x.ntile = base[x.b + 1] - base[x.b];
  x.tile = x.ntile - 1 - (e - base[x.b]);
  x.tokens = min(s.n - x.tile * per_item, per_item);
  const int i0 = s.L - s.n + x.tile * per_item, i1 = i0 + x.tokens - 1;
  const int lo = a.window > 0 && i0 >= a.window ? i0 - a.window + 1 : 0;
  const int pre_units = (s.pre + 15) >> 4;
  const int nblk = pre_units + max((i1 >> 4) - max(lo >> 4, pre_units) + 1, 0);
  x.kt = (nblk + kTileBlocks - 1) / kTileBlocks;
  return x;
}

constexpr int kMaxShares = 64;     // of an entry
constexpr int kPlanEntries = 512;  // entries kept in shared memory: the most that the first rule meets

__global__ void __launch_bounds__(1024) prefill_plan_kernel(const PrefillAttnArgs a, int per_item) {
  extern __shared__ int s_base[];  // [B + 1] first entry of each sequence, then [B] (queries, keys, prefix)
  int* s_seq = s_base + a.B + 1;
  __shared__ int s_split;
  __shared__ long long s_sum[34];
  __shared__ int s_kt[kPlanEntries];
  __shared__ short s_tokens[kPlanEntries];
  __shared__ int s_max;
  __shared__ unsigned long long s_best;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  if (tid == 0) {
    s_max = 0;
    s_split = 0;
    s_best = ~0ull;
    s_base[0] = 0;
  }
  grid_dependency_wait();
  grid_launch_dependents();
  // exclusive block sum of v; the total in s_sum[32]
  auto scan = [&](long long v) -> long long {
    long long x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long t = __shfl_up_sync(kFullMask, x, o);
      if (lane >= o) x += t;
    }
    __syncthreads();  // the sums of the scan before have been read
    if (lane == 31) s_sum[warp] = x;
    __syncthreads();
    if (warp == 0) {
      const long long own = lane < warps ? s_sum[lane] : 0;
      long long y = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long t = __shfl_up_sync(kFullMask, y, o);
        if (lane >= o) y += t;
      }
      __syncwarp();
      s_sum[lane] = y - own;
      if (lane == 31) s_sum[32] = y;
    }
    __syncthreads();
    return s_sum[warp] + x - v;
  };
  int carry = 0;
  bool unordered = false;
  for (int base = 0; base < a.B; base += blockDim.x) {
    int ntile = 0;
    PrefillSeq s{0, 0, 0, 0, 0};
    if (base + tid < a.B) s = prefill_seq(a, base + tid);
    // Ascending starts make the sequences' rows disjoint, which bounds the entries (and gives each row one
    // writer).  Where some are not, a sequence is refused that starts below any start before its own.
    unordered = __syncthreads_or(s.err == PKV_DEV_BAD_QUERY_RANGE) != 0 || unordered;
    if (unordered && base + tid < a.B && s.err == 0) {
      int most = 0;
      for (int k = 0; k < base + tid; ++k) most = max(most, a.query_starts[k]);
      if (s.q0 < most) s = PrefillSeq{0, 0, 0, 0, PKV_DEV_BAD_QUERY_RANGE};
    }
    if (base + tid < a.B) {
      if (s.err != 0) record_error(a.err, s.err);
      ntile = (s.n + per_item - 1) / per_item;
      s_seq[3 * (base + tid)] = s.n;
      s_seq[3 * (base + tid) + 1] = s.L;
      s_seq[3 * (base + tid) + 2] = s.pre;
    }
    const int at = carry + (int)scan(ntile);
    if (base + tid < a.B) s_base[base + tid + 1] = at + ntile;
    carry += (int)s_sum[32];
  }
  __syncthreads();
  const int entries = carry;
  if (entries == 0) {  // every sequence idle or refused: nothing to share out
    if (tid < 3) a.plan_head[tid] = 0;
    return;
  }
  long long work = 0;
  int most = 0;
  for (int e = tid; e < entries; e += blockDim.x) {
    const Entry x = plan_entry(a, s_base, s_seq, e, per_item);
    if (e < kPlanEntries) {
      s_kt[e] = x.kt;
      s_tokens[e] = (short)x.tokens;
    }
    work += x.kt;
    most = max(most, x.kt);
  }
  most = __reduce_max_sync(kFullMask, most);
  if (lane == 0) atomicMax(&s_max, most);
  (void)scan(work);
  const long long W = s_sum[32] * a.Hkv, P = (long long)entries * a.Hkv;
  const int ktmax = max(s_max, 1);
  int chunk, tail = entries, tail_split = 1;
  if (P < a.slots && entries <= kPlanEntries) {
    for (int q = warp; q < 16; q += warps) {
      // 1 .. 6, 8, 10, 16, .., 64, and what fills the CTAs once and twice if all entries are alike
      const int once = (int)(a.slots / P);
      const int sp = q < 6    ? q + 1
                     : q < 13 ? (q & 1) ? 5 << ((q >> 1) - 2) : 4 << ((q >> 1) - 2)
                              : min(kMaxShares, q == 13 ? once : q == 14 ? 2 * once : (int)(2 * a.slots / P));
      const int c = (ktmax + sp - 1) / sp;
      int shares = 0, rows = 0;
      for (int e = lane; e < entries; e += 32) {
        const int n = min(kMaxShares, max(1, (s_kt[e] + c - 1) / c));
        shares += n;
        rows += n > 1 ? s_tokens[e] : 0;
      }
      shares = __reduce_add_sync(kFullMask, shares);
      rows = __reduce_add_sync(kFullMask, rows);
      const long long items = (long long)shares * a.Hkv;
      if (sp > 1 && items > 2 * a.slots) continue;
      long long end = c + 1;
      if (items > a.slots) end = min((W + items) / a.slots + c, (items + a.slots - 1) / a.slots * end);
      if (rows > 0) end += 1 + (long long)rows * a.Hq / 4000;
      if (lane == 0) atomicMin(&s_best, (unsigned long long)end << 32 | (0xffffffffu - (unsigned)c));
    }
    __syncthreads();
    chunk = (int)(0xffffffffu - (unsigned)(s_best & 0xffffffffull));  // of equal ends the fewest shares
  } else {
    chunk = (int)max((long long)kMinChunk, (W + W / 2) / a.slots);
    if (ktmax <= chunk) {
      const int t = (int)(P % a.slots) / a.Hkv * a.Hkv;  // whole entries
      float best = 2.f;
      for (int sp = 1; sp <= 8 && t > 0 && (long long)t * sp <= 2 * a.slots; ++sp) {
        const float end = (float)((t * sp + a.slots - 1) / a.slots) / (float)sp + 0.03f * (float)sp;
        if (end < best) {
          best = end;
          tail_split = sp;
        }
      }
      if (tail_split > 1) tail = entries - t / a.Hkv;
    }
  }
  auto shares_of = [&](int e, int kt) {
    if (e >= tail) return min(tail_split, max(1, kt / kMinChunk));
    return min(kMaxShares, max(1, (kt + chunk - 1) / chunk));
  };
  // places in the list: the long entries' shares, then the others'; partial rows of the split ones
  long long first = 0;
  for (int e = tid; e < entries; e += blockDim.x) {
    const int kt = e < kPlanEntries ? s_kt[e] : plan_entry(a, s_base, s_seq, e, per_item).kt;
    if (2 * kt > ktmax) first += shares_of(e, kt);
  }
  (void)scan(first);
  long long at[2] = {0, s_sum[32]};
  long long row = 0;
  for (int base = 0; base < entries; base += blockDim.x) {
    const int e = base + tid;
    Entry x{};
    int shares = 0, part = 1;
    if (e < entries) {
      x = plan_entry(a, s_base, s_seq, e, per_item);
      shares = shares_of(e, x.kt);
      part = 2 * x.kt > ktmax ? 0 : 1;
    }
    const long long both = scan(part == 0 ? (long long)shares << 32 : shares);
    const long long both_all = s_sum[32];
    const long long row0 = row + scan(shares > 1 ? (long long)x.tokens * a.Hq * shares : 0);
    row += s_sum[32];
    if (e < entries) {
      const long long item0 = at[part] + (part == 0 ? both >> 32 : both & 0xffffffffll);
      const int q0 = a.query_starts[x.b] + x.tile * per_item, L = s_seq[3 * x.b + 1];
      if (shares > 1) a.plan_split[atomicAdd(&s_split, 1)] = make_int4(q0, x.tokens, shares, (int)row0);
      const int4 where = make_int4(x.b, q0, x.tokens, L - s_seq[3 * x.b] + x.tile * per_item);
      for (int k = 0; k < shares; ++k) {
        a.plan_items[2 * (item0 + k)] = where;
        a.plan_items[2 * (item0 + k) + 1] = make_int4(L, s_seq[3 * x.b + 2], k | shares << 16, (int)row0);
      }
    }
    at[0] += both_all >> 32;
    at[1] += both_all & 0xffffffffll;
  }
  __syncthreads();
  if (tid == 0) {
    a.plan_head[0] = (int)at[1];  // items
    a.plan_head[1] = 0;           // the ticket counter
    a.plan_head[2] = s_split;     // split entries
  }
}

// --------------------------------------------------------------------------------- rows again
//
// A row that is not finite comes from a V that it sees, from a masked key, whose weight is 0, and 0 times a V of NaN or
// infinity is NaN, or (V of 2^119 and more) from weights of up to 2^8 where those of at most 1 would do.  Only the
// first is its own.  non_finite_v looks for the others; a row that has a masked key that is not finite, or whose keys
// all are, is computed again, 5 us for 32 keys with the row's warp alone.  A V of NaN that every row of its row tile
// sees costs the search, from the last step back (chunk of 4096 on 16384: 761 us with one that the last 64 rows see, 2.65 ms
// with one at 8192, 4.66 with one at 0, against 746 us; all such rows computed again, 911 ms); rows before it in its
// own tile are computed again (a NaN at 16382: 90 ms), as are rows of up to 512 keys (2.4 ms in all).

// A row: sequence, kv head, packed row, query head; position, interval start, prefix; entries [e0, e1) of the key
// list, of which entry e is block e, or e + shift from pre_units on.
struct Row {
  int b, g, r, h;
  int i, lo, pre;
  int e0, e1;
  int pre_units, shift;
};

// The keys of block `blk` that the row sees, a bit each.
__device__ __forceinline__ uint32_t seen_keys(int i, int lo, int pre, int blk) {
  const int hi_c = i - blk * 16, lo_c = lo - blk * 16, pre_c = pre - blk * 16;
  uint32_t see = hi_c >= 15 ? 0xffffu : hi_c < 0 ? 0u : (2u << hi_c) - 1u;
  see &= lo_c <= 0 ? 0xffffu : lo_c > 15 ? 0u : 0xffffu << lo_c;
  return see | (pre_c >= 16 ? 0xffffu : pre_c <= 0 ? 0u : (1u << pre_c) - 1u);
}

// Whether a key in list entries [e0, e1) has a non-finite V (1), and (2) whether there is one that this lane's row
// (i, lo, pre; the other fields are the warp's) does not see, by one warp.  L: the sequence's keys (V rows past it
// were cleared).
template <int D>
__device__ __noinline__ int non_finite_v(const PrefillAttnArgs& a, const Row& w, int L) {
  const int lane = threadIdx.x & 31;
  int found = 0;
  for (int en = w.e0; en < w.e1; ++en) {
    const int blk = en < w.pre_units ? en : en + w.shift;
    const int phys = a.block_tables[(size_t)w.b * a.MB + blk];
    if (phys < 0 || phys >= a.NB) continue;
    // lanes 2c and 2c + 1 have the halves of row c
    const uint4* v = reinterpret_cast<const uint4*>(a.v_cache + (((size_t)phys * a.Hkv + w.g) * 16 + (lane >> 1)) * D) +
                     (lane & 1) * (D / 16);
    bool bad = false;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      const uint4 x = v[k];
      for (const uint32_t p : {x.x, x.y, x.z, x.w}) bad |= (p & 0x7f80u) == 0x7f80u || (p & 0x7f800000u) == 0x7f800000u;
    }
    uint32_t rows = __ballot_sync(kFullMask, bad);
    if (rows == 0u) continue;
    rows = (rows | rows >> 1) & 0x55555555u;  // a bit in two, brought together
    rows = (rows | rows >> 1) & 0x33333333u;
    rows = (rows | rows >> 2) & 0x0f0f0f0fu;
    rows = (rows | rows >> 4) & 0x00ff00ffu;
    rows = (rows | rows >> 8) & 0xffffu;
    if (L - blk * 16 < 16) rows &= (1u << (L - blk * 16)) - 1u;
    found |= ((rows & ~seen_keys(w.i, w.lo, w.pre, blk)) != 0u ? 2 : 0) | (rows != 0u ? 1 : 0);
  }
  return found;
}

// What the tensor cores compute for the row, without the masked keys, by one warp, 32 keys at a time: eight lanes
// a K row for the products, then a key a lane, then D / 32 elements of the output a lane.  Writes the output row, or
// partial row `part` if that is not negative.  A sum that is no number stays so, and ends it.
template <int D>
__device__ __noinline__ void exact_row(const PrefillAttnArgs& a, const Row& w, long long part) {
  constexpr int E = D / 32, H = D / 64;
  const int lane = threadIdx.x & 31, sub = lane & 7;
  const int key = (lane >> 3) + 4 * sub;  // of the 32: lanes 8 g .. 8 g + 7 read the rows of keys g + 4 n
  float o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  uint32_t q[H][4];
#pragma unroll
  for (int h = 0; h < H; ++h) {
    const uint4 u = *reinterpret_cast<const uint4*>(a.q + ((size_t)w.r * a.Hq + w.h) * D + h * 64 + sub * 8);
    q[h][0] = u.x; q[h][1] = u.y; q[h][2] = u.z; q[h][3] = u.w;
  }
  const float slope = a.slopes != nullptr ? a.slopes[w.h] * kLog2e : 0.f;
  auto block_of = [&](int e) { return e < w.pre_units ? e : e + w.shift; };
  auto id_of = [&](int en) {  // the pool block of the lane's key, of entries en and en + 1; -1: none
    const int e = en + (key >> 4);
    const int id = e < w.e1 ? a.block_tables[(size_t)w.b * a.MB + block_of(e)] : -1;
    return id < a.NB ? id : -1;
  };
  int next = id_of(w.e0);
  for (int en = w.e0; en < w.e1; en += 2) {
    const int phys = next, blk = block_of(en + (key >> 4)), c = key & 15;
    next = id_of(en + 2);
    const bool see = phys >= 0 && ((seen_keys(w.i, w.lo, w.pre, blk) >> c) & 1u);
    const uint32_t seen = __ballot_sync(kFullMask, see);
    const long long row = ((long long)phys * a.Hkv + w.g) * 16 + c;
    uint32_t v[16][E / 2];  // V of half of the keys, the first half's on their way while the logits are worked out
    auto load_v = [&](int s0) {
#pragma unroll
      for (int s = 0; s < 16; ++s) {
        const long long at = __shfl_sync(kFullMask, row, s0 + s);
        const uint32_t* src = reinterpret_cast<const uint32_t*>(a.v_cache + at * D + lane * E);
#pragma unroll
        for (int k = 0; k < E / 2; ++k) v[s][k] = ((seen >> (s0 + s)) & 1u) ? src[k] : 0u;
      }
    };
    load_v(0);
    float x = 0.f;
#pragma unroll 1
    for (int n0 = 0; n0 < 8; n0 += 4) {
      uint4 t[4][H];
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const int from = (lane & 24) | (n0 + n);
        const long long at = __shfl_sync(kFullMask, row, from);
#pragma unroll
        for (int h = 0; h < H; ++h)
          t[n][h] = ((seen >> from) & 1u) ? *reinterpret_cast<const uint4*>(a.k_cache + at * D + h * 64 + sub * 8)
                                          : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        float y = 0.f;
#pragma unroll
        for (int h = 0; h < H; ++h) {
          const uint32_t ts[4] = {t[n][h].x, t[n][h].y, t[n][h].z, t[n][h].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            y = fmaf(bf16_lo_to_f32(q[h][k]), bf16_lo_to_f32(ts[k]), y);
            y = fmaf(bf16_hi_to_f32(q[h][k]), bf16_hi_to_f32(ts[k]), y);
          }
        }
#pragma unroll
        for (int s = 4; s > 0; s >>= 1) y += __shfl_xor_sync(kFullMask, y, s);
        if (n0 + n == sub) x = y;
      }
    }
    x *= a.scale_log2;
    if (a.cap_log2 > 0.f) x = cap_logit(x, a.cap_log2, a.cap_in);
    x -= slope * fabsf((float)(w.i - (blk * 16 + c)));
    if (!see) x = -INFINITY;
    float top = x;
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, s));
    top = fmaxf(m, top);
    const float ref = top == -INFINITY ? 0.f : top;
    const float keep = exp2f(m - ref), p = exp2f(x - ref);
    m = top;
    l = l * keep + p;
    if (__any_sync(kFullMask, l != l)) {
      l = __int_as_float(0x7fffffff);
      break;
    }
#pragma unroll
    for (int k = 0; k < E; ++k) o[k] *= keep;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      if (half == 1) load_v(16);
#pragma unroll
      for (int s = 0; s < 16; ++s) {
        const float ps = __shfl_sync(kFullMask, p, 16 * half + s);
#pragma unroll
        for (int k = 0; k < E; ++k)
          o[k] = fmaf(ps, (k & 1) ? bf16_hi_to_f32(v[s][k >> 1]) : bf16_lo_to_f32(v[s][k >> 1]), o[k]);
      }
    }
  }
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) l += __shfl_xor_sync(kFullMask, l, s);
  const float f = part >= 0 ? 1.f : l > 0.f ? 1.f / l : (l == l ? 0.f : l);
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int c = lane * E + e;
    if (part >= 0) a.part_o[part * D + c] = o[e];
    else a.out[((size_t)w.r * a.Hq + w.h) * D + c] = __float2bfloat16_rn(o[e] * f);
  }
  if (part >= 0 && lane == 0) a.part_ml[part] = make_float2(m, l);
}

// ------------------------------------------------------------------------------- the attention

// One work item for one kv head, and the key list of its rows: the blocks of the prefix, then those of
// the union of the rows' intervals, in tiles of 8.
struct Item {
  int b, g, split, nsplit, part;  // part: first partial row of the entry
  int L, pre;                     // of the sequence
  int row0, tokens, nx;           // first packed row, tokens, row tiles
  int pos0;                       // position of the first token
  int pre_units, nblk, shift, nt_all, ts, nt;  // list entries, key tiles of the rows, this share's
  int ns;                                      // steps of this share

  __device__ __forceinline__ int block_of(int e) const { return e < pre_units ? e : e + shift; }
};

// Steps run from the last one back, so that with a distance bias the nearest keys set the maximum.  Row tile x
// runs those from hi down to lo: later ones lie past its last row, earlier ones before its first interval.
// Step j is half j & 1 of the share's tile j >> 1, which is the (nt - 1 - (j >> 1))-th to be loaded.
struct Steps {
  int hi, lo;
};

// p, q: the record of item it.
__device__ __forceinline__ Item item_of(const PrefillAttnArgs& a, int it, int4 p, int4 q, int NT) {
  Item w;
  w.b = p.x;
  w.g = it % a.Hkv;
  w.row0 = p.y;
  w.tokens = p.z;
  w.pos0 = p.w;
  w.L = q.x;
  w.pre = q.y;
  w.split = q.z & 0xffff;
  w.nsplit = q.z >> 16;
  w.part = q.w;
  w.nx = NT == 2 && w.tokens > a.R ? 2 : 1;
  return w;
}

// lo_min: the least interval start of the item's rows.
__device__ __forceinline__ void set_keys(Item& w, int lo_min) {
  const int i_max = w.pos0 + w.tokens - 1;
  w.pre_units = (w.pre + 15) >> 4;
  const int first = max(lo_min >> 4, w.pre_units);
  w.nblk = w.pre_units + (lo_min <= i_max ? max((i_max >> 4) - first + 1, 0) : 0);
  w.shift = first - w.pre_units;
  w.nt_all = (w.nblk + kTileBlocks - 1) / kTileBlocks;
  const int per = (w.nt_all + w.nsplit - 1) / w.nsplit;
  w.ts = min(w.split * per, w.nt_all);
  w.nt = min(w.ts + per, w.nt_all) - w.ts;
  w.ns = (min(w.nblk, (w.ts + w.nt) * kTileBlocks) - w.ts * kTileBlocks + kStepBlocks - 1) / kStepBlocks;
}

// lo_least: the least interval start of row tile x.
__device__ __forceinline__ Steps steps_of(const PrefillAttnArgs& a, const Item& w, int x, int lo_least) {
  const int e_base = w.ts * kTileBlocks;
  const int i_last = w.pos0 + min(w.tokens, (x + 1) * a.R) - 1;
  const int e_last = max((i_last >> 4) - w.shift, w.pre_units - 1), e_first = w.pre_units > 0 ? 0 : (lo_least >> 4) - w.shift;
  return Steps{min(w.ns - 1, (e_last - e_base) >> 2), max(0, (e_first - e_base) >> 2)};
}

template <int D, int NT>
struct Shared {
  uint64_t q_full, kv_full[Geo<D, NT>::kSlots], kv_empty[Geo<D, NT>::kSlots];
  uint64_t s_full[NT][2], p_full[NT][2], pv_done[NT][2];  // by buffer: S ready, P ready, P V added
  uint64_t drained[2];  // after a timeout: an issuer's MMAs have ended
  uint32_t tmem;
  int4 record[2];                       // of the next item
  int lo_least[NT], lo_most[NT], abort, next;  // interval starts of the row tiles' rows
};

// Loads the item's Q tiles and its K and V tiles through the ring (one warp).  n_kv counts K and V tiles
// since the kernel's start, n_q loaded items.
template <int D, int NT>
__device__ __forceinline__ void produce(const PrefillAttnArgs& a, Shared<D, NT>& sh, const Item& w, unsigned char* sq,
                                        uint32_t& n_kv, uint32_t n_q) {
  using GE = Geo<D, NT>;
  constexpr int NS = GE::kSlots, H = GE::kHalves;
  const int lane = threadIdx.x & 31;
  unsigned char* skv = sq + NT * GE::kTile;
  const uint64_t pol = l2_policy_evict_last();  // K and V tiles are read by every row tile of the sequence
  if (lane == 0) {
    const uint64_t pol_q = l2_policy_evict_first();
    mbar_arrive_expect_tx(&sh.q_full, (uint32_t)(w.nx * H * 128 * a.G * a.R));
    for (int y = 0; y < w.nx; ++y)
#pragma unroll
      for (int h = 0; h < H; ++h)
        tma_load_3d(sq + y * GE::kTile + h * kHalf, &a.tmap_q, h * 64, w.g * a.G, w.row0 + y * a.R, &sh.q_full, pol_q);
  }
  auto id_of = [&](int j) -> int {  // lane p < 8: the pool block of entry p of the j-th key tile, -1: none
    const int e = (w.ts + w.nt - 1 - j) * kTileBlocks + lane;
    int id = -1;
    if (lane < kTileBlocks && j < w.nt && e < w.nblk) {
      id = __ldg(a.block_tables + (size_t)w.b * a.MB + w.block_of(e));
      if (id < 0 || id >= a.NB) {
        record_error(a.err, PKV_DEV_BAD_BLOCK_ID);
        id = -1;
      }
    }
    return id;
  };
  int id = id_of(0);
  bool ok = true;
  for (int j = 0; j < w.nt && ok; ++j) {
    const int next = id_of(j + 1);
    const uint32_t have = __ballot_sync(kFullMask, id >= 0);
    for (int kv = 0; kv < 2; ++kv, ++n_kv) {
      const uint32_t slot = n_kv % NS;
      if (n_kv >= NS) ok = mbar_wait_spin(&sh.kv_empty[slot], ((n_kv / NS) - 1) & 1u, a.timeout_ns);
      ok = __all_sync(kFullMask, ok);
      if (!ok) break;
      unsigned char* dst = skv + slot * GE::kTile;
      if (have != 0xffu) {  // blocks past the list (or refused): zeros
        for (int p = 0; p < kTileBlocks; ++p) {
          if ((have >> p) & 1u) continue;
          for (int h = 0; h < H; ++h)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              *reinterpret_cast<uint4*>(dst + h * kHalf + p * 2048 + (c * 32 + lane) * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        __syncwarp();
      }
      if (lane == 0) mbar_arrive_expect_tx(&sh.kv_full[slot], (uint32_t)(__popc(have) * H * 2048));
      __syncwarp();
      if (id >= 0) {
        const int y = (id * a.Hkv + w.g) * 16;
#pragma unroll
        for (int h = 0; h < H; ++h)
          tma_load_2d(dst + h * kHalf + lane * 2048, kv == 0 ? &a.tmap_k : &a.tmap_v, h * 64, y, &sh.kv_full[slot], pol);
      }
    }
    id = next;
  }
  if (!ok) {
    if (lane == 0) {
      record_error(a.err, PKV_DEV_WAIT_TIMEOUT);
      sh.abort = 1;
      // what is in flight lands before the CTA goes
      (void)mbar_wait_spin(&sh.q_full, n_q & 1u, a.timeout_ns);
      for (uint32_t c = n_kv > NS ? n_kv - NS : 0; c < n_kv; ++c)
        (void)mbar_wait_spin(&sh.kv_full[c % NS], (c / NS) & 1u, a.timeout_ns);
    }
    __syncwarp();
  }
}

// Issues MMAs of the item's row tile y: QK the products S = Q K^T, PV the products O += P V (a warp's elected
// lane; what the MMAs take is the same in every lane and kept in uniform registers).  S has two buffers of 64
// keys in tensor memory, and P takes the place of its S: while the softmax works on a step, S of the next one
// is there, and that of the step after follows the product that reads P from its columns (the tensor core runs
// one thread's MMAs in the order of issue).  One product for a whole 128-key tile, a third fewer MMAs and a
// quarter less tensor time, leaves no room for the second buffer and is slower (chunk of 4096 on 16384: 863
// against 720 us): the softmax then waits out every product.
// Beside the softmax warps a thread needs 60 to 120 cycles an MMA and a hundred or more for each barrier: one
// issuer for two row tiles leaves the tensor core idle (chunk of 4096 on 16384, plain, 1.07 ms; one for each
// 0.92; one for each product of each 0.75 against 0.72, its warps taking issue slots from the softmax).  With
// one row tile and two CTAs an SM the products have an issuer each (64 tokens on 2000 keys each: 129 -> 112 us).
// A ring tile is free once both row tiles have read it; a row tile that does not read it only says so.
template <int D, int NT, bool QK, bool PV>
__device__ __forceinline__ void issue_mmas(const PrefillAttnArgs& a, Shared<D, NT>& sh, const Item& w, unsigned char* sq,
                                           uint32_t tmem_any, uint32_t leader, int y, uint32_t& n_kv, uint32_t n_q,
                                           uint32_t& n_step) {
  using GE = Geo<D, NT>;
  using SH = Shared<D, NT>;
  constexpr int NS = GE::kSlots;
  constexpr uint32_t id_qk = umma_idesc_bf16(128, kStep), id_pv = umma_idesc_bf16_bmn(128, D);
  auto uniform = [](uint32_t v) { return __shfl_sync(kFullMask, v, 0); };
  const uint32_t base = uniform(smem_u32(sq)), bars = uniform(smem_u32(&sh));
  const uint32_t kv_base = uniform(n_kv);  // K of the i-th tile loaded is tile kv_base + 2 i of the ring, V the next
  auto free_tile = [&](uint32_t c) { umma_commit_by(leader, bars + (uint32_t)offsetof(SH, kv_empty) + (c % NS) * 8); };
  auto wait = [&](uint64_t* bar, uint32_t phase) {
    if (__all_sync(kFullMask, mbar_wait_spin(bar, phase & 1u, a.timeout_ns))) return true;
    if (leader) {
      record_error(a.err, PKV_DEV_WAIT_TIMEOUT);
      sh.abort = 1;
    }
    return false;
  };
  auto wait_kv = [&](uint32_t c) { return wait(&sh.kv_full[c % NS], c / NS); };
  n_kv = kv_base + 2 * w.nt;
  bool ok = true;
  const int nt = (int)uniform((uint32_t)w.nt);
  const Steps range = y < w.nx ? steps_of(a, w, y, sh.lo_least[y]) : Steps{-1, 0};
  const int hi = (int)uniform((uint32_t)range.hi), lo = (int)uniform((uint32_t)range.lo);
  auto pass = [&](int from, int to) {  // the loads [from, to) that this row tile does not read
    for (int i = from; i < to && ok; ++i)
      for (int v = QK ? 0 : 1; v < (PV ? 2 : 1) && ok; ++v) {
        ok = wait_kv(kv_base + 2 * i + v);
        if (ok) free_tile(kv_base + 2 * i + v);
      }
  };
  if (hi < lo) {
    pass(0, nt);
    return;
  }
  const bool two = uniform((uint32_t)w.nt_all) <= (uint32_t)kTwoTermTiles;
  const uint32_t step0 = uniform(n_step);
  const uint32_t s0 = uniform(tmem_any) + y * 2 * kStep, o = uniform(tmem_any) + NT * 2 * kStep + y * D;
  constexpr uint32_t kTile16 = GE::kTile / 16, kStep16 = kStep * 128 / 16;  // descriptors count 16 bytes
  const uint32_t qa = umma_lo_k(base) + y * kTile16, k0 = umma_lo_k(base + NT * GE::kTile);
  const uint32_t v0 = umma_lo_mn(base + NT * GE::kTile, kHalf);
  auto k_tile = [&](int j) { return kv_base + 2u * (uint32_t)(nt - 1 - (j >> 1)); };
  // S of step j; its tile's K is awaited before the tile's first step and freed after the last
  auto wait_k = [&](int j) { return (j != hi && !(j & 1)) || wait_kv(k_tile(j)); };
  auto qk = [&](int j) {
    const uint32_t buf = (step0 + (uint32_t)(hi - j)) & 1u, kb = k0 + (k_tile(j) % NS) * kTile16 + (j & 1) * kStep16;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      const uint32_t off = (uint32_t)((k >> 2) * kHalf + (k & 3) * 32) / 16;
      umma_bf16_lo(leader, s0 + buf * kStep, qa + off, kb + off, id_qk, k > 0);
    }
    umma_commit_by(leader, bars + (uint32_t)offsetof(SH, s_full) + (y * 2 + buf) * 8);
    if (!(j & 1) || j == lo) free_tile(k_tile(j));
  };
  auto pv = [&](int j) {
    const uint32_t buf = (step0 + (uint32_t)(hi - j)) & 1u, tile = k_tile(j) + 1u;
    const uint32_t vb = v0 + (tile % NS) * kTile16 + (j & 1) * kStep16;
    const uint32_t p = s0 + buf * kStep;
#pragma unroll
    for (int k = 0; k < kStep / 16; ++k)  // 32 keys' first terms, then their remainders, 16 columns each
      umma_bf16_ts_lo(leader, o, p + 32 * (k >> 1) + 8 * (k & 1), vb + k * 128, id_pv, k > 0 || j < hi);
    if (two) {
#pragma unroll
      for (int k = 0; k < kStep / 16; ++k)
        umma_bf16_ts_lo(leader, o, p + 32 * (k >> 1) + 16 + 8 * (k & 1), vb + k * 128, id_pv, true);
    }
    umma_commit_by(leader, bars + (uint32_t)offsetof(SH, pv_done) + (y * 2 + buf) * 8);
    if (!(j & 1) || j == lo) free_tile(tile);
  };
  if constexpr (QK) ok = wait(&sh.q_full, n_q);
  pass(0, nt - 1 - (hi >> 1));
  if constexpr (QK) {
    for (int j = hi; j >= max(lo, hi - 1) && ok; --j) {  // (the second tile may need the first one's place)
      ok = wait_k(j);
      if (!ok) break;
      tc_fence_after();
      qk(j);
    }
  }
  for (int j = hi; j >= lo && ok; --j) {
    const uint32_t c = step0 + (uint32_t)(hi - j);
    if constexpr (PV) {
      if (j == hi || (j & 1)) ok = wait_kv(k_tile(j) + 1u);  // V of the tile's first step
      ok = ok && wait(&sh.p_full[y][c & 1u], c >> 1);
      if (!ok) break;
      tc_fence_after();
      pv(j);
    }
    if (QK && j - 2 >= lo) {
      ok = wait_k(j - 2);
      if constexpr (!PV) {  // the product has read P from the columns
        ok = ok && wait(&sh.pv_done[y][c & 1u], c >> 1);
        tc_fence_after();
      }
      if (!ok) break;
      qk(j - 2);
    }
  }
  pass(nt - (lo >> 1), nt);
  if (!ok) {  // the MMAs in flight end before tensor memory goes
    const uint32_t at = NT == 2 ? (uint32_t)y : (PV ? 1u : 0u);
    umma_commit_by(leader, bars + (uint32_t)offsetof(SH, drained) + at * 8);
    (void)mbar_wait_spin(&sh.drained[at], 0, a.timeout_ns);
  }
  n_step = step0 + (uint32_t)(hi - lo + 1);
}

// Largest of N values (of their sizes when ABS), in four chains of three-operand maxima.
template <bool ABS, int N>
__device__ __forceinline__ float row_max(const float (&v)[N]) {
  static_assert(N % 8 == 4 || N % 8 == 0, "pairs for four chains");
  float t[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) t[c] = fmax3(ABS ? fabsf(v[2 * c]) : v[2 * c], ABS ? fabsf(v[2 * c + 1]) : v[2 * c + 1], -INFINITY);
#pragma unroll
  for (int c = 8; c < N; c += 2)
    t[(c >> 1) & 3] = fmax3(t[(c >> 1) & 3], ABS ? fabsf(v[c]) : v[c], ABS ? fabsf(v[c + 1]) : v[c + 1]);
  return fmaxf(fmax3(t[0], t[1], t[2]), t[3]);
}

// tanh(u) / u as a polynomial of u^2, of the least largest relative error on |u| <= kCapNear (degree 2, 1.1e-7)
// and on |u| <= kCapFar (degree 5, 5.8e-8), found by Remez' exchange in 40 digits; as stored 1.2e-7 and 6.8e-8, in
// fp32 steps 1.5e-7 and 1.1e-7.
constexpr float kCapNear = 0.2f, kCapFar = 0.8f;
constexpr float kCapWide = 256.f;  // caps (base 2) whose last bits are more than 2^-14, a 64th of a bf16 output's half step
__device__ constexpr float kCap2[3] = {0.99999988f, -0.3332859f, 0.13015407f};
__device__ constexpr float kCap5[6] = {0.99999994f, -0.33332676f, 0.13321048f, -0.053114317f, 0.019093301f, -0.0043552998f};

// v = v P(v^2 k^2) with P = tanh(u) / u, for |v k| <= kCapFar.
template <int N>
__device__ __forceinline__ void cap_poly(float (&v)[N], float k) {
  uint64_t p[6];
  float w = 1.f;
#pragma unroll
  for (int n = 0; n < 6; ++n, w *= k * k) p[n] = pack2(kCap5[n] * w, kCap5[n] * w);
#pragma unroll
  for (int c = 0; c < N; c += 2) {
    const uint64_t x = pack2(v[c], v[c + 1]);
    const uint64_t q = fmul2(x, x);
    uint64_t f = p[5];
#pragma unroll
    for (int n = 4; n >= 0; --n) f = ffma2(f, q, p[n]);
    const float2 y = unpack2(fmul2(x, f));
    v[c] = y.x;
    v[c + 1] = y.y;
  }
}

// v = cap2 tanh(v ku), each key by the polynomial or the exponential form as its own u = v ku asks (an infinite u
// gives +-cap2, NaN stays).  Both forms a key, in place of one: for caps above 177 whose scores, or a masked key beside
// them, come near the cap (chunk of 4096 on 16384, 2.84 against 1.51 ms).
template <int N>
__device__ __forceinline__ void cap_each(float (&v)[N], float ku, float cap2) {
#pragma unroll
  for (int c = 0; c < N; ++c) {
    const float u = v[c] * ku, w = u * u;
    float f = kCap5[5];
#pragma unroll
    for (int n = 4; n >= 0; --n) f = fmaf(f, w, kCap5[n]);
    const float big = 1.f - 2.f * rcp_approx(ex2_approx(u * (2.f * kLog2e)) + 1.f);
    v[c] = cap2 * (fabsf(u) < kCapFar ? u * f : big);
  }
}

// A thread's base-2 logits are v[c] mul + base + step (c / 8), mul > 0.
struct Logits {
  float mul, base, step;
};

// For the rules that need each key's own value: the products S of a thread's N keys, in place, brought into
// that form of x = cap(S sl2) - slope |i - t|.  (Without such rules v = S and mul = sl2.)  e0: the list entry of
// its first key.
template <int N>
__device__ __forceinline__ Logits apply_rules(const PrefillAttnArgs& a, bool cap, bool bias, float (&v)[N], float slope2, int i, const Item& w,
                                              int e0) {
  Logits x{a.scale_log2, 0.f, 0.f};
  if (cap) {
    // u = S ku is the logit over the cap.  Up to kCapFar for every key of the warp's rows the polynomial serves.
    // Else 1 - 2 / (e^2u + 1), an exponential and a reciprocal a key, whose error for a small u is that of the
    // cap's last bits, about 2^-22 cap_log2.  The large u beside it may be a masked key's or another row's, so a
    // cap above kCapWide takes the form of each key's own u
    const float ku = a.scale_log2 * a.cap_in * 0.34657359f;
    const float far = row_max<true>(v) * fabsf(ku);
    x.mul = a.cap_log2 * ku;
    if (x.mul > 0.f && __all_sync(kFullMask, far < kCapFar && fabsf(ku) < 1e3f)) {
      cap_poly(v, ku);
    } else if (a.cap_log2 > kCapWide) {
      cap_each(v, ku, a.cap_log2);
      x.mul = 1.f;
    } else {
      const float k = ku * (2.f * kLog2e), twice = -2.f * a.cap_log2;
      const uint64_t k2 = pack2(k, k), one = pack2(1.f, 1.f), top = pack2(a.cap_log2, a.cap_log2), m2 = pack2(twice, twice);
#pragma unroll
      for (int c = 0; c < N; c += 2) {
        const float2 z = unpack2(fmul2(pack2(v[c], v[c + 1]), k2));
        const float2 e = unpack2(fadd2(pack2(ex2_approx(z.x), ex2_approx(z.y)), one));
        const float2 y = unpack2(ffma2(pack2(rcp_approx(e.x), rcp_approx(e.y)), m2, top));
        v[c] = y.x;
        v[c + 1] = y.y;
      }
      x.mul = 1.f;
    }
  }
  if (bias && a.slopes != nullptr) {
    const uint64_t m2 = pack2(x.mul, x.mul);
    if (e0 >= w.pre_units) {
      // the interval's part of the list is one run of positions, and keys past i are masked: the distance
      // is i - t, linear along the tile; within eight keys it is added here, the rest goes into the exponent
      x.base = -slope2 * (float)(i - w.block_of(e0) * 16);
      x.step = 8.f * slope2;
      uint64_t near[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) near[c] = pack2(slope2 * (float)(2 * c), slope2 * (float)(2 * c + 1));
#pragma unroll
      for (int c = 0; c < N; c += 2) {
        const float2 y = unpack2(ffma2(pack2(v[c], v[c + 1]), m2, near[(c >> 1) & 3]));
        v[c] = y.x;
        v[c + 1] = y.y;
      }
    } else {
#pragma unroll
      for (int p = 0; p < N / 16; ++p) {
        const float d0 = (float)(i - w.block_of(e0 + p) * 16);
#pragma unroll
        for (int c = 0; c < 16; ++c) v[16 * p + c] = fmaf(-slope2, fabsf(d0 - (float)c), v[16 * p + c] * x.mul);
      }
    }
    x.mul = 1.f;
  } else if (!(x.mul > 0.f)) {
#pragma unroll
    for (int c = 0; c < N; ++c) v[c] *= x.mul;
    x.mul = 1.f;
  }
  return x;
}

// One step's weights for a thread's 64 unmasked keys in one pass: p = 2^(logit - ref), written as bf16 pairs
// over S, and their sum.  The logit is S c0, or with CAP S c0 P(S^2 ku^2), P of that degree with the scales folded
// into its coefficients (here at each step: kept over the steps they cost the registers of the logits, capped
// 0.89 -> 0.93 ms).  BIAS: plus base + slope2 c for key c of the step.
template <int CAP, bool BIAS>
__device__ __forceinline__ float step_weights(const float (&v)[kStep], uint32_t ts_addr, float c0, float ku, float base,
                                              float slope2) {
  uint64_t kc[CAP + 1];
  if constexpr (CAP == 0) {
    kc[0] = pack2(c0, c0);
  } else {
    asm volatile("" : "+f"(ku));
    const float w = ku * ku;
#pragma unroll
    for (int n = 0; n <= CAP; ++n, c0 *= w) {
      const float k = c0 * (CAP == 2 ? kCap2[n] : kCap5[n]);
      kc[n] = pack2(k, k);
    }
  }
  uint64_t near[4], sum[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    near[k] = BIAS ? pack2(fmaf(slope2, (float)(2 * k), base), fmaf(slope2, (float)(2 * k + 1), base)) : pack2(base, base);
    sum[k] = pack2(0.f, 0.f);
  }
#pragma unroll
  for (int c = 0; c < kStep / 32; ++c) {
    uint32_t hi[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const uint64_t x = pack2(v[32 * c + 2 * k], v[32 * c + 2 * k + 1]);
      uint64_t b = near[k & 3];
      if constexpr (BIAS) {
        const float far = slope2 * (float)(32 * c + 8 * (k >> 2));
        if (c > 0 || k >= 4) b = fadd2(b, pack2(far, far));
      }
      uint64_t f = kc[CAP];
      if constexpr (CAP > 0) {
        const uint64_t q = fmul2(x, x);
#pragma unroll
        for (int n = CAP - 1; n >= 0; --n) f = ffma2(f, q, kc[n]);
      }
      const float2 z = unpack2(ffma2(x, f, b));
      const float p0 = ex2_approx(z.x), p1 = ex2_approx(z.y);
      hi[k] = pack_bf16x2(p0, p1);
      sum[k & 3] = fadd2(sum[k & 3], pack2(p0, p1));
    }
    tmem_st_x16(ts_addr + 32 * c, hi);
  }
  const float2 t = unpack2(fadd2(fadd2(sum[0], sum[1]), fadd2(sum[2], sum[3])));
  return t.x + t.y;
}

// The item's softmax and output for this thread's row r of row tile x: position i (-1: none), interval start
// lo; prow and h name the output row.
// MODE: the rules that need each key's own logit, 1 a cap and 2 a distance bias (or a scale that is not positive),
// 4: asked of the arguments at each step.
template <int D, int NT, int MODE>
__device__ __forceinline__ void softmax_rows(const PrefillAttnArgs& a, Shared<D, NT>& sh, const Item& w,
                                             unsigned char* sq, uint32_t tmem, int x, int r, bool valid, int i,
                                             int lo, int prow, int h, uint32_t n_kv, uint32_t& n_step) {
  using GE = Geo<D, NT>;
  constexpr int NS = GE::kSlots, H = GE::kHalves, N = kStep;
  const int lane = threadIdx.x & 31;
  unsigned char* skv = sq + NT * GE::kTile;
  const bool cap = MODE == 4 ? a.cap_log2 > 0.f : (MODE & 1) != 0;
  const bool bias = MODE == 4 ? a.slopes != nullptr || !(a.scale_log2 > 0.f) : (MODE & 2) != 0;
  const float slope2 = bias && valid && a.slopes != nullptr ? __ldg(a.slopes + h) * kLog2e : 0.f;
  const int pre = valid ? w.pre : 0;
  const bool two = w.nt_all <= kTwoTermTiles;
  // the cap as a polynomial of S: u = S ku, the logit cap_log2 u P(u^2)
  const float ku = a.scale_log2 * a.cap_in * 0.34657359f, ku_size = fabsf(ku) < 1e3f ? fabsf(ku) : INFINITY;
  const Steps range = steps_of(a, w, x, sh.lo_least[x]);
  // steps whose keys all rows of the row tile see: a range of the interval's part of the list, and one of the
  // prefix's.  The list's position of entry e is 16 (e + shift) there.
  const int e_base = w.ts * kTileBlocks;
  int full0 = (max(w.pre_units, ((sh.lo_most[x] + 15) >> 4) - w.shift) - e_base + kStepBlocks - 1) >> 2;
  const int full1 = (((w.pos0 + x * a.R + 1) >> 4) - w.shift - e_base) >> 2;  // whole blocks up to the first row's position
  full0 = max(full0, 0);
  const int full_pre = ((w.pre >> 4) - e_base) >> 2;
  static_assert(kStepBlocks == 4, "steps of four blocks");
  // the block that ends past the sequence: its V rows there are cleared, by the warps of each row tile before
  // they hand over the step's P (both write the same zeros)
  const int last_blk = (w.L - 1) >> 4;
  const int e_last = last_blk < w.pre_units ? last_blk : last_blk - w.shift;
  const int tail_step = (w.L & 15) != 0 && e_last >= 0 && e_last < w.nblk && w.block_of(e_last) == last_blk
                            ? (e_last - e_base) >> 2 : -1;
  const uint32_t t_lane = tmem + ((uint32_t)(r & ~31) << 16);
  const uint32_t to_addr = t_lane + NT * 2 * kStep + x * D;
  bool ok = true;
  float m = -INFINITY, l = 0.f;
  float reach = kCapNear;  // of the polynomial tried for the cap
  for (int j = range.hi; j >= range.lo; --j) {
    const uint32_t buf = n_step & 1u;
    const uint32_t ts_addr = t_lane + x * 2 * kStep + buf * kStep;
    ok = __all_sync(kFullMask, mbar_wait_spin(&sh.s_full[x][buf], (n_step >> 1) & 1u, a.timeout_ns));
    if (!ok) break;
    tc_fence_after();
    float v[N];
#pragma unroll
    for (int c = 0; c < N / 32; ++c) tmem_ld_x32(ts_addr + 32 * c, *reinterpret_cast<float(*)[32]>(v + 32 * c));
    tmem_wait_ld();
    const int e0 = e_base + j * kStepBlocks;
    const bool full = (j >= full0 && j < full1) || j < full_pre;
    // Steps without a mask take one pass over the row.  With a cap or a bias, the products' largest size bounds
    // the logits: the step's nearest key lies within twice that below the bound, so where that is 2^80 or less
    // the bound serves as the maximum (the weights stay within fp32 and bf16 range), and the cap and the bias
    // are part of the exponent's FMAs
    bool fast = full && !two;
    float mx = -INFINITY, base = 0.f;
    Logits y{a.scale_log2, 0.f, 0.f};
    if (fast && !cap && !bias) {
      mx = row_max<false>(v) * a.scale_log2;
    } else if (fast) {
      const float far = row_max<true>(v);
      const float size = far * fabsf(a.scale_log2);
      mx = size;
      if (bias && slope2 != 0.f) {
        base = -slope2 * (float)(i - w.block_of(e0) * 16);
        mx += fmaxf(base, fmaf(slope2, (float)(kStep - 1), base));
      }
      const bool in = 2.f * size <= 80.f && (!bias || slope2 == 0.f || j >= full_pre);
      const float u = cap ? far * ku_size : 0.f;
      fast = __all_sync(kFullMask, in && u < reach);
      if (cap && (!fast || reach != kCapNear)) {  // the other polynomial, here and from here on
        const bool near = fast && __all_sync(kFullMask, u < kCapNear);
        reach = near ? kCapNear : kCapFar;
        fast = fast || __all_sync(kFullMask, in && u < reach);
      }
    }
    if (!fast) {
      if (cap || bias) y = apply_rules(a, cap, bias, v, slope2, i, w, e0);
      if (!full) {
#pragma unroll
        for (int p = 0; p < N / 16; ++p) {
          const uint32_t see = seen_keys(i, lo, pre, w.block_of(e0 + p));
#pragma unroll
          for (int c = 0; c < 16; ++c) v[16 * p + c] = ((see >> c) & 1u) ? v[16 * p + c] : -INFINITY;
        }
      }
      if (y.step == 0.f) {
        mx = fmaf(row_max<false>(v), y.mul, y.base);
      } else {
        mx = -INFINITY;
#pragma unroll
        for (int g = 0; g < N / 8; ++g) {
          const float* t = v + 8 * g;
          const float top = fmax3(fmax3(t[0], t[1], t[2]), fmax3(t[3], t[4], t[5]), fmaxf(t[6], t[7]));
          mx = fmaxf(mx, top + fmaf(y.step, (float)g, y.base));
        }
      }
    }
    const bool move = mx > m + kSlack;
    if (__any_sync(kFullMask, move)) {
      const float scale = move ? ex2_approx(m - mx) : 1.f;
      if (move) m = mx;
      l *= scale;
      if (j < range.hi) {  // O moves to the new reference once the last product has ended
        ok = __all_sync(kFullMask, mbar_wait_spin(&sh.pv_done[x][(n_step - 1) & 1u], ((n_step - 1) >> 1) & 1u, a.timeout_ns));
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          float o[16];
          tmem_ld_x16(to_addr + 16 * c, o);
          tmem_wait_ld();
          uint32_t u[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) u[k] = __float_as_uint(o[k] * scale);
          tmem_st_x16(to_addr + 16 * c, u);
        }
      }
    }
    const float ref = m == -INFINITY ? 0.f : m;
    if (fast) {
      base -= ref;
      const float c0 = cap ? a.cap_log2 * ku : a.scale_log2;
      if (!bias) {
        if (!cap) l += step_weights<0, false>(v, ts_addr, c0, 0.f, base, 0.f);
        else if (reach == kCapNear) l += step_weights<2, false>(v, ts_addr, c0, ku, base, 0.f);
        else l += step_weights<5, false>(v, ts_addr, c0, ku, base, 0.f);
      } else {
        if (!cap) l += step_weights<0, true>(v, ts_addr, c0, 0.f, base, slope2);
        else if (reach == kCapNear) l += step_weights<2, true>(v, ts_addr, c0, ku, base, slope2);
        else l += step_weights<5, true>(v, ts_addr, c0, ku, base, slope2);
      }
    } else {
      y.base -= ref;
      const uint64_t mul2 = pack2(y.mul, y.mul);
      uint64_t sum2[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) sum2[k] = pack2(0.f, 0.f);
      if (!two) {
#pragma unroll
        for (int c = 0; c < N / 32; ++c) {
          uint32_t hi[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float off = fmaf(y.step, (float)(4 * c + k / 4), y.base);
            const float2 z = unpack2(ffma2(pack2(v[32 * c + 2 * k], v[32 * c + 2 * k + 1]), mul2, pack2(off, off)));
            const float p0 = ex2_approx(z.x), p1 = ex2_approx(z.y);
            hi[k] = pack_bf16x2(p0, p1);
            sum2[k & 3] = fadd2(sum2[k & 3], pack2(p0, p1));
          }
          tmem_st_x16(ts_addr + 32 * c, hi);
        }
      } else {
#pragma unroll
        for (int c = 0; c < N / 32; ++c) {
          uint32_t hi[16], rest[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float off = fmaf(y.step, (float)(4 * c + k / 4), y.base);
            const float2 z = unpack2(ffma2(pack2(v[32 * c + 2 * k], v[32 * c + 2 * k + 1]), mul2, pack2(off, off)));
            const float p0 = ex2_approx(z.x), p1 = ex2_approx(z.y);
            hi[k] = pack_bf16x2(p0, p1);
            rest[k] = pack_bf16x2(p0 - bf16_lo_to_f32(hi[k]), p1 - bf16_hi_to_f32(hi[k]));
            sum2[k & 3] = fadd2(sum2[k & 3], pack2(p0, p1));
          }
          tmem_st_x16(ts_addr + 32 * c, hi);
          tmem_st_x16(ts_addr + 32 * c + 16, rest);
        }
      }
      const float2 sum = unpack2(fadd2(fadd2(sum2[0], sum2[1]), fadd2(sum2[2], sum2[3])));
      l += sum.x + sum.y;
    }
    if (j == tail_step) {
      const uint32_t vtile = n_kv + 2 * (w.nt - 1 - (j >> 1)) + 1;  // this tile's V in the count of K and V tiles
      ok = __all_sync(kFullMask, mbar_wait_spin(&sh.kv_full[vtile % NS], (vtile / NS) & 1u, a.timeout_ns));
      if (!ok) break;
      unsigned char* rows = skv + (vtile % NS) * GE::kTile + (e_last % kTileBlocks) * 2048;
      const int gone = 16 - (w.L & 15);
      for (int c = r; c < gone * 8 * H; c += 128)
        *reinterpret_cast<uint4*>(rows + (c / (gone * 8)) * kHalf + (w.L & 15) * 128 + (c % (gone * 8)) * 16) =
            make_uint4(0u, 0u, 0u, 0u);
      fence_proxy_async_smem();
    }
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.p_full[x][buf]);
    ++n_step;
  }
  const bool some = range.hi >= range.lo;
  if (ok && some) {
    ok = __all_sync(kFullMask, mbar_wait_spin(&sh.pv_done[x][(n_step - 1) & 1u], ((n_step - 1) >> 1) & 1u, a.timeout_ns));
    tc_fence_after();
  }
  if (!ok) {
    if (lane == 0) {
      record_error(a.err, PKV_DEV_WAIT_TIMEOUT);
      sh.abort = 1;
    }
    return;
  }
  // ---- the rows out: bf16, or this share's unnormalised row with its maximum and sum
  const bool split = w.nsplit > 1;
  const long long part =
      split ? (long long)w.part + ((long long)w.split * w.tokens + (prow - w.row0)) * a.Hq + h : 0;
  const float f = split ? 1.f : (l > 0.f ? 1.f / l : 0.f);
  bool bad = !(l <= 3.4028234e38f);
#pragma unroll
  for (int c = 0; c < D / 16; ++c) {
    float o[16];
    __syncwarp();
    if (some) {
      tmem_ld_x16(to_addr + 16 * c, o);
      tmem_wait_ld();
    }
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      o[k] = some ? o[k] * f : 0.f;
      bad |= !(fabsf(o[k]) <= 3.4028234e38f);
    }
    if (valid && split) {
      float4* dst = reinterpret_cast<float4*>(a.part_o + part * D + 16 * c);
#pragma unroll
      for (int k = 0; k < 4; ++k) dst[k] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
    } else if (valid) {
      uint4* dst = reinterpret_cast<uint4*>(a.out + ((size_t)prow * a.Hq + h) * D + 16 * c);
#pragma unroll
      for (int k = 0; k < 2; ++k)
        dst[k] = make_uint4(pack_bf16x2(o[8 * k], o[8 * k + 1]), pack_bf16x2(o[8 * k + 2], o[8 * k + 3]),
                            pack_bf16x2(o[8 * k + 4], o[8 * k + 5]), pack_bf16x2(o[8 * k + 6], o[8 * k + 7]));
    }
  }
  if (split && valid) a.part_ml[part] = make_float2(m, l);
  // Rows that are not finite and may owe it to other than a V that they see.  (Rows of two terms, at most 512 keys
  // long, are all taken: an infinite V times the terms may be NaN.)
  uint32_t again = __ballot_sync(kFullMask, valid && bad);
  if (again != 0u) {
    Row row;
    row.b = w.b;
    row.g = w.g;
    row.pre_units = w.pre_units;
    row.shift = w.shift;
    row.i = i;
    row.lo = lo;
    row.pre = pre;
    int found = 0;
    for (int full = 0; full < 2; ++full) {  // (a masked key is in a step with a mask; in the others one key is enough)
      for (int j = range.hi; j >= range.lo && !two && !(full && (found & 1)); --j) {
        if (((j >= full0 && j < full1) || j < full_pre) != (full != 0)) continue;
        row.e0 = e_base + j * kStepBlocks;
        row.e1 = min(row.e0 + kStepBlocks, w.nblk);
        found |= non_finite_v<D>(a, row, w.L);
      }
    }
    const bool owes = two || !(l <= 3.4028234e38f) || found != 1;
    again = __ballot_sync(kFullMask, valid && bad && owes);
    __syncwarp();  // the rows are stored by other lanes after this one's stores
    while (again != 0u) {
      const int src = __ffs(again) - 1;
      again &= again - 1;
      row.r = __shfl_sync(kFullMask, prow, src);
      row.h = __shfl_sync(kFullMask, h, src);
      row.i = __shfl_sync(kFullMask, i, src);
      row.lo = __shfl_sync(kFullMask, lo, src);
      row.pre = __shfl_sync(kFullMask, pre, src);
      row.e0 = w.ts * kTileBlocks;
      row.e1 = min((w.ts + w.nt) * kTileBlocks, w.nblk);
      exact_row<D>(a, row, split ? __shfl_sync(kFullMask, part, src) : -1);
    }
  }
}

template <int D, int NT>
__global__ void __launch_bounds__(Geo<D, NT>::kThreads, Geo<D, NT>::kCtas)
prefill_attention_kernel(const __grid_constant__ PrefillAttnArgs a) {
  using GE = Geo<D, NT>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* sq = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ Shared<D, NT> sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 32) {
    prefetch_tensor_map(&a.tmap_q);
    prefetch_tensor_map(&a.tmap_k);
    prefetch_tensor_map(&a.tmap_v);
  }
  if (threadIdx.x == 0) {
    mbar_init(&sh.q_full, 1);
    for (int s = 0; s < GE::kSlots; ++s) {
      mbar_init(&sh.kv_full[s], 1);
      mbar_init(&sh.kv_empty[s], NT);
    }
    for (int x = 0; x < NT; ++x) {
      for (int q = 0; q < 2; ++q) {
        mbar_init(&sh.s_full[x][q], 1);
        mbar_init(&sh.p_full[x][q], 4);
        mbar_init(&sh.pv_done[x][q], 1);
      }
    }
    mbar_init(&sh.drained[0], 1);
    mbar_init(&sh.drained[1], 1);
    sh.abort = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(&sh.tmem, GE::kTmemCols);
    tmem_relinquish();
  }
  grid_dependency_wait();  // the plan
  grid_launch_dependents();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  // (a CTA without an item reads past the list's end, inside the workspace)
  const int4* first = a.plan_items + 2 * ((int)blockIdx.x / a.Hkv);
  int4 rec0 = first[0], rec1 = first[1];
  const int total = a.plan_head[0] * a.Hkv;
  // Each role has the whole item loop, so that its registers are its own.  Three block barriers an item:
  // the shared minimum is reset, it is complete, every role has left the item.
  uint32_t n_kv = 0, n_q = 0;  // K and V tiles, and items with tiles, since the kernel's start (barrier phases)
  if (warp < GE::kSoftmaxWarps) {
    setmaxnreg_inc<GE::kSoftmaxRegs>();
    // a warp reaches the tensor memory lanes of its number mod 4
    const int x = warp >> 2, r = 32 * (warp & 3) + lane;
    const int tok = r / a.G, head = r - tok * a.G;
    uint32_t n_step = 0;
    const int mode = (a.cap_log2 > 0.f ? 1 : 0) | (a.slopes != nullptr || !(a.scale_log2 > 0.f) ? 2 : 0);
    for (int it = blockIdx.x; it < total; it = sh.next, rec0 = sh.record[0], rec1 = sh.record[1]) {
      Item w = item_of(a, it, rec0, rec1, NT);
      if (threadIdx.x == 0) {
        for (int y = 0; y < NT; ++y) {
          sh.lo_least[y] = 0x7fffffff;
          sh.lo_most[y] = 0;
        }
      }
      __syncthreads();
      const bool valid = tok < a.R && x * a.R + tok < w.tokens;
      const int prow = w.row0 + x * a.R + tok;
      const int i = valid ? w.pos0 + x * a.R + tok : -1;
      const int lo = valid ? interval_start(a, prow, i) : 0;
      const int least = __reduce_min_sync(kFullMask, valid ? lo : 0x7fffffff);
      const int most = __reduce_max_sync(kFullMask, lo);
      if (lane == 0) {
        atomicMin(&sh.lo_least[x], least);
        atomicMax(&sh.lo_most[x], most);
      }
      __syncthreads();
      set_keys(w, min(sh.lo_least[0], sh.lo_least[NT - 1]));
      if (x < w.nx) {
        const int h = w.g * a.G + head;
        auto rows = [&](auto m) {
          softmax_rows<D, NT, decltype(m)::value>(a, sh, w, sq, tmem, x, r, valid, i, lo, prow, h, n_kv, n_step);
        };
        // a loop for each set of rules: one for all is 3 to 5 % slower with a cap (0.88 against 0.84 ms, a chunk
        // of 4096 on 16384 keys).  One row tile has the registers of half the threads: there the loop for all
        // serves (64 tokens on 2000 keys 109 us, 114 with four loops, which spill)
        if constexpr (NT == 1) {
          rows(std::integral_constant<int, 4>{});
        } else {
          if (mode == 0) rows(std::integral_constant<int, 0>{});
          else if (mode == 1) rows(std::integral_constant<int, 1>{});
          else if (mode == 2) rows(std::integral_constant<int, 2>{});
          else rows(std::integral_constant<int, 3>{});
        }
      }
      n_kv += 2 * w.nt;
      tc_fence_before();
      __syncthreads();
      if (sh.abort != 0) break;
    }
  } else {
    setmaxnreg_dec<GE::kOtherRegs>();
    uint32_t n_step = 0;
    const uint32_t leader = elect_one();
    for (int it = blockIdx.x; it < total; it = sh.next, rec0 = sh.record[0], rec1 = sh.record[1]) {
      Item w = item_of(a, it, rec0, rec1, NT);
      __syncthreads();
      __syncthreads();
      set_keys(w, min(sh.lo_least[0], sh.lo_least[NT - 1]));
      if (w.nt > 0) {
        if (warp == GE::kProducer) {
          produce<D, NT>(a, sh, w, sq, n_kv, n_q);
        } else if (warp < GE::kTicket) {
          tc_fence_after();
          const int k = warp - GE::kIssuer;
          if constexpr (NT == 2) {
            issue_mmas<D, NT, true, true>(a, sh, w, sq, tmem, leader, k, n_kv, n_q, n_step);
          } else {
            if (k == 0) issue_mmas<D, NT, true, false>(a, sh, w, sq, tmem, leader, 0, n_kv, n_q, n_step);
            else issue_mmas<D, NT, false, true>(a, sh, w, sq, tmem, leader, 0, n_kv, n_q, n_step);
          }
        }
        ++n_q;
      }
      // meanwhile the next item's ticket is taken, its record read
      if (warp == GE::kTicket && lane == 0) {
        const int next = (int)gridDim.x + atomicAdd(a.plan_head + 1, 1);
        sh.next = next;
        if (next < total) {
          sh.record[0] = a.plan_items[2 * (next / a.Hkv)];
          sh.record[1] = a.plan_items[2 * (next / a.Hkv) + 1];
        }
      }
      __syncwarp();
      __syncthreads();
      if (sh.abort != 0) break;
    }
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, GE::kTmemCols);
}

// ------------------------------------------------------------------------------------ the merge

// A warp a row of a split entry: lane k has the (maximum, sum) of shares k and k + 32, then the rows of all
// shares are added, four loads in flight.
template <int D>
__global__ void __launch_bounds__(256) prefill_merge_kernel(const PrefillAttnArgs a, int per_item) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  grid_dependency_wait();
  grid_launch_dependents();
  const int per_entry = min(per_item, a.T) * a.Hq;  // rows at most
  const long long rows = (long long)a.plan_head[2] * per_entry;
  for (long long row = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5; row < rows;
       row += ((long long)gridDim.x * blockDim.x) >> 5) {
    const int k = (int)(row / per_entry), in = (int)(row - (long long)k * per_entry);
    const int4 split = a.plan_split[k];  // (first packed row, tokens, shares, first partial row)
    const int per = split.y * a.Hq;
    if (in >= per) continue;
    const long long p0 = (long long)split.w + in;
    float2 ml[2];
    float m = -INFINITY;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int sh = lane + 32 * q;
      ml[q] = sh < split.z ? __ldcg(a.part_ml + p0 + (long long)sh * per) : make_float2(-INFINITY, 0.f);
      m = fmaxf(m, ml[q].x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFullMask, m, o));
    const float ref = m == -INFINITY ? 0.f : m;
    float w[2], l = 0.f;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      w[q] = exp2f(ml[q].x - ref);  // 0 for a share that saw nothing
      l += w[q] * ml[q].y;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(kFullMask, l, o);
    float o[E] = {};
#pragma unroll 4
    for (int sh = 0; sh < split.z; ++sh) {
      const float f = __shfl_sync(kFullMask, sh < 32 ? w[0] : w[1], sh & 31);
      const float* src = a.part_o + (p0 + (long long)sh * per) * D + lane * E;
      float x[E];
      if constexpr (E == 4) {
        const float4 t = __ldcg(reinterpret_cast<const float4*>(src));
        x[0] = t.x; x[1] = t.y; x[2] = t.z; x[3] = t.w;
      } else {
        const float2 t = __ldcg(reinterpret_cast<const float2*>(src));
        x[0] = t.x; x[1] = t.y;
      }
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = f == 0.f ? o[e] : fmaf(f, x[e], o[e]);
    }
    const float inv = l > 0.f ? 1.f / l : (l == l ? 0.f : l);
    __nv_bfloat16* dst = a.out + ((long long)split.x * a.Hq + in) * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2)
      *reinterpret_cast<uint32_t*>(dst + e) = pack_bf16x2(o[e] * inv, o[e + 1] * inv);
  }
}

}  // namespace

namespace {
constexpr int kMaxSms = 160;                             // CTAs a plan counts on: at most kCtas on each of these
constexpr long long kMaxPartRows = 2ll * kMaxSms * 256;  // rows of 2 slots shares (43 MB of partial rows at d = 128)
size_t align256p(size_t x) { return (x + 255) & ~size_t(255); }

struct PrefillWorkspace {
  size_t items, split, ml, o, total;
};

// head | int4[2] items | int4 split entries | float2 (m, l) | float o.  Entries: at most one per 128 rows, and one
// more per sequence; items: those and the shares of split ones.
PrefillWorkspace plan_prefill(long long B, long long T, int Hq, int G, int D) {
  PrefillWorkspace w{};
  const long long entries = T / (128 / G) + B;
  const long long rows = std::min(kMaxPartRows, T * Hq * kMaxShares);
  w.items = 256;
  w.split = align256p(w.items + 2 * sizeof(int4) * (size_t)(entries + 4 * kMaxSms));
  w.ml = align256p(w.split + sizeof(int4) * (size_t)std::min<long long>(entries, 4 * kMaxSms));
  w.o = align256p(w.ml + sizeof(float2) * (size_t)rows);
  w.total = align256p(w.o + sizeof(float) * (size_t)rows * D);
  return w;
}

size_t plan_smem_bytes(int B) { return sizeof(int) * (4 * (size_t)B + 1); }

template <int D, int NT>
cudaError_t launch_attention(const PrefillAttnArgs& a, cudaStream_t stream) {
  using GE = Geo<D, NT>;
  PrefillAttnArgs args = a;
  args.slots = std::min(a.sms, kMaxSms) * GE::kCtas;
  int per_item = NT * a.R;
  void* plan_params[] = {&args, &per_item};
  // a whole call with a plan of 512 and of 1024 threads, us: one token 19.1, 20.0; 24 mixed sequences 28.1, 28.9; 300
  // sequences 39.1, 40.3; 1000 37.6, 36.5; 4000 114, 106 (256 threads: 19.3, 28.5, 41.2, 42.4, 140)
  cudaError_t e = launch_pdl((const void*)prefill_plan_kernel, dim3(1), dim3(a.B > 512 ? 1024 : 512), plan_smem_bytes(a.B),
                             stream, plan_params);
  if (e != cudaSuccess) return e;
  void* params[] = {&args};
  // a CTA for every slot: even one token's keys are cut into shares for all of them
  e = launch_pdl((const void*)prefill_attention_kernel<D, NT>, dim3((unsigned)args.slots), dim3(GE::kThreads), GE::kSmem, stream, params);
  if (e != cudaSuccess) return e;
  const long long entries = (long long)a.T / per_item + a.B;  // at most
  const long long warps = std::min(entries * std::min(per_item, a.T) * a.Hq, 8ll * 8 * a.sms);
  return launch_pdl((const void*)prefill_merge_kernel<D>, dim3((unsigned)((warps + 7) / 8)), dim3(256), 0, stream, plan_params);
}

template <int D, int NT>
cudaError_t setup_attention() {
  return cudaFuncSetAttribute((const void*)prefill_attention_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)Geo<D, NT>::kSmem);
}
}  // namespace

size_t prefill_attention_workspace(int B, int T, int Hq, int G, int D) { return plan_prefill(B, T, Hq, G, D).total; }

cudaError_t prefill_attention_device_setup() {
  cudaError_t e = cudaFuncSetAttribute((const void*)prefill_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)plan_smem_bytes(kMaxStepBatch));
  if (e == cudaSuccess) e = setup_attention<128, 1>();
  if (e == cudaSuccess) e = setup_attention<128, 2>();
  if (e == cudaSuccess) e = setup_attention<64, 1>();
  if (e == cudaSuccess) e = setup_attention<64, 2>();
  return e;
}

cudaError_t launch_prefill_attention(const PrefillAttnArgs& a, void* workspace, int head_dim, cudaStream_t stream) {
  PrefillAttnArgs args = a;
  const PrefillWorkspace w = plan_prefill(a.B, a.T, a.Hq, a.G, head_dim);
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  args.plan_head = reinterpret_cast<int*>(ws);
  args.plan_items = reinterpret_cast<int4*>(ws + w.items);
  args.plan_split = reinterpret_cast<int4*>(ws + w.split);
  args.part_ml = reinterpret_cast<float2*>(ws + w.ml);
  args.part_o = reinterpret_cast<float*>(ws + w.o);
  // two row tiles an item when the sequences fill more than one on average (64 single tokens on 2000 keys, d 128:
  // 110 us with one, 149 with two; 8 x 16 on 5000 52 and 64; 4 x 2048 prompts 205 and 163; 4 x 512 on 4096 with
  // one head a kv head 62 and 56)
  const bool two = (long long)a.T > (long long)a.B * a.R;
  if (head_dim == 128) return two ? launch_attention<128, 2>(args, stream) : launch_attention<128, 1>(args, stream);
  return two ? launch_attention<64, 2>(args, stream) : launch_attention<64, 1>(args, stream);
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
  return prefill_attention_workspace(dims->batch, total_tokens, dims->num_q_heads,
                                     dims->num_q_heads / dims->num_kv_heads, dims->head_dim);
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
  if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(workspace) ||
      ((reinterpret_cast<uintptr_t>(block_tables) | reinterpret_cast<uintptr_t>(context_lens) |
        reinterpret_cast<uintptr_t>(query_starts) | reinterpret_cast<uintptr_t>(error_word)) & 3u))
    return PKV_ERR_ALIGNMENT;
  int sms = 0;
  st = device_ready(&sms);
  if (st != PKV_OK) return st;
  PrefillAttnArgs a{};
  const long long pool_rows = (long long)dims->num_blocks * dims->num_kv_heads * PKV_BLOCK_SIZE;
  const int group = dims->num_q_heads / dims->num_kv_heads;
  st = encode_pool_map(&a.tmap_k, k_cache, pool_rows, dims->head_dim);
  if (st == PKV_OK) st = encode_pool_map(&a.tmap_v, v_cache, pool_rows, dims->head_dim);
  if (st == PKV_OK)
    st = encode_window_map(&a.tmap_q, q, total_tokens, dims->num_q_heads, dims->head_dim, group, 128 / group);
  if (st != PKV_OK) return st;
  a.sms = sms;
  a.R = 128 / group;
  a.timeout_ns = kWaitTimeoutNs;
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
  a.G = group;
  a.scale_log2 = scale * kLog2e;
  if (rules != nullptr) {
    a.window = rules->window;
    a.slopes = rules->alibi_slopes;
    a.doc_starts = rules->doc_starts;
    a.prefix_lens = rules->prefix_lens;
    a.cap_log2 = rules->softcap * kLog2e;
    a.cap_in = rules->softcap > 0.f ? 2.f / rules->softcap : 0.f;
  }
  return cuda_status(launch_prefill_attention(a, workspace, dims->head_dim, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
