// Attention for a batch whose sequences share long beginnings, over the paged 8-bit cache:
//
//   out = (sum_{t < c} w_t v_t + sum_{c <= t <= p} w_t v_t) / (the same sums of w_t),
//   w_t = exp(scale q.k_t),
//
// c the tokens that a row's group of sequences shares. The first sums are worked out for all the
// group's rows at once, so that a shared key is read once a call instead of once a sequence: rows
// of many sequences fill the tensor cores' tiles. The second are each sequence's own. Both leave
// a running maximum m, l = sum exp(x - m) and O = sum exp(x - m) v in fp32, joined by
// O exp(m - M), l exp(m - M).
//
// Launches: a plan (the batch's entries read and checked once, units of the shared part and where
// their results go), the shared part, the own parts (and those of sequences with many rows, where
// there may be any, on tcgen05), and the joining. The shared part is cut along its tokens too, as
// far as SMs are left without work. The own parts do not wait for it: the shared part's kernel
// takes as many SMs as the plan gives it and lets the other start on the rest (64 answers to a
// prompt of 8192 tokens, 32 query and 8 kv heads of 128: 49 us, and 58 one after the other). The
// joining is a kernel of its own: taking the shared parts in at the end of every own unit cost
// that kernel 9 of 34 us there and 40 of 100 with 200 sequences.
//
// The shared part goes to the tcgen05 kernel (256 rows x 64 keys a step; its units here have no
// masks) where the groups have rows enough, to the kernel of few rows otherwise.
//
// Bound: for long shared parts the tcgen05 kernel's step (1.3 us for 256 rows x 64 keys of 128
// elements, 6.5 of 12.4 TFLOP/s an SM; 64 x 1 token over 65536 shared: 106 us, 1060 with every
// sequence reading them), for short ones the launches (17 us for 2 sequences over 1024 tokens) and
// the own units' beginnings and ends.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>
#include <string>
#include <type_traits>

#include "cache_rows.cuh"
#include "cache_shared.cuh"
#include "csa_internal.h"

namespace csa {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanGroups = 64, kPlanSequences = 256;

// From this many rows a group on average (tokens x query heads of a kv head) the shared part is
// the tcgen05 kernel's: over 65536 tokens (8 kv heads) 16 and 32 rows take 65 and 89 us there and
// 65 and 87 here, 64 rows 89 there and 150 here; over 4 groups of 8192 32 rows take 66 there, 60 here.
constexpr int kPrefixFrom = 33;
// Below so many bytes of codes that it would keep from being read again (by all SMs), the shared
// part is not worth its launches and sequences read it for themselves. us with a shared part,
// without one in this call, and with cache_attention_forward (8 kv heads of 128 but for the last;
// 100 own tokens each):
//   64 x 1 token over 1024 (132 MB)  29 / -  / 34      16 x 1 over 1024 (31 MB)   21 / 27 / 17
//   64 x 1 over 512 (66 MB)          28 / -  / 25      8 x 1 over 2048 (29 MB)    22 / 21 / 16
//   64 x 1 over 256 (33 MB)          28 / 32 / 21      4 x 1 over 4096 (25 MB)    22 / 22 / 16
//   64 x 1 over 192 (25 MB)          28 / 31 / 20      128 x 1 over 128 (33 MB)   33 / 35 / 26
//   64 x 1 over 128 (17 MB)          28 / 25 / 18      20 x 1 over 5008 (30 MB)   27 / 25 / 20
// Without one the kernel of the shared part is launched for nothing (5 us of those of 25 to 33 MB),
// unless the host sees that the tables have no room for so much (the 25 us over 128): a bound that
// fits both, and what the plan itself and the joining take (6 us where nothing is shared), is left.
constexpr long long kWorthBytes = 32LL << 20;
// Room for parts beyond one for each row and head: what cutting along the tokens may take.
constexpr long long kSpareParts = 2LL * kMaxSms * kPrefixRows;

struct PlanArgs {
  KvView v;
  const int* groups;  // [group_count + 1]
  const int* shared;  // [group_count]
  SharedPlan plan;
  long long rows_heads;  // rows of own_there
  int group_heads;
  int unit_rows, tile;  // of the shared part's kernel
  int sms, per_sm;      // and what works on a unit at a time, of an SM
  float tile_us, start, first;  // a tile's time there, what a unit takes beyond its tiles (in
                                // tiles), the kernel beyond its units
  float part_us;        // what one part takes, written and read again
  int own_rows, own_tile, own_start;  // of the own parts' kernel, the same
  float own_us, own_first;            // (own_us: a tile of all kv heads on one SM)
  bool drop;            // whether a sequence or two may be left out of a group
  long long worth;      // keys, over all kv heads, whose reading the shared part has to save
  long long prompt_blocks;  // as in AttendArgs
};

// CTA 0 plans, the others clear the marks of the rows.
__global__ void __launch_bounds__(kPlanThreads, 1) shared_plan_sm103a_kernel(const PlanArgs a) {
  __shared__ int s_bad, s_most, s_chunk, s_sms;
  __shared__ unsigned long long s_saved, s_blocks, s_tiles, s_own, s_long, s_key[kPlanThreads / 32];
  // (what fits is kept here until the end)
  __shared__ SharedGroup s_groups[kPlanGroups];
  __shared__ SharedSequence s_sequences[kPlanSequences];
  const KvView& v = a.v;
  const SharedPlan& plan = a.plan;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, G = plan.group_count,
            S = v.sequences;
  SharedGroup* const groups = G <= kPlanGroups ? s_groups : plan.groups;
  SharedSequence* const sequences = S <= kPlanSequences ? s_sequences : plan.sequences;
  grid_dependency_wait();
  if (blockIdx.x > 0) {
    const long long n = (a.rows_heads + 3) / 4;
    for (long long i = (blockIdx.x - 1) * static_cast<long long>(kPlanThreads) + tid; i < n;
         i += static_cast<long long>(gridDim.x - 1) * kPlanThreads)
      reinterpret_cast<int4*>(plan.own_there)[i] = make_int4(0, 0, 0, 0);
    return;
  }
  if (tid == 0) s_bad = s_most = 0, s_saved = s_blocks = s_tiles = s_own = s_long = 0;
  __syncthreads();

  // The groups: bounds in order, whole pages.
  for (int g = tid; g < G; g += kPlanThreads) {
    const int from = a.groups[g], to = a.groups[g + 1], tokens = a.shared[g];
    if (from < 0 || to < from || to > S) s_bad = 1;
    const bool ok = tokens >= 0 && (tokens & (v.page_tokens - 1)) == 0 &&
                    tokens <= static_cast<long long>(v.table_width) * v.page_tokens;
    SharedGroup p{};
    p.sequence = from;
    p.rows = to;  // (for now: where the group ends)
    p.tokens = ok ? tokens : -1;
    groups[g] = p;
  }
  __syncthreads();
  const bool bad = s_bad != 0;  // then nothing is computed
  if (bad && tid == 0) report_index(v.status, kIndexSequence);

  // The sequences, each with its group (found by its bounds); and what their own parts take, those
  // of more rows than kRowLimit apart: another kernel's, if there are blocks enough of them.
  long long own = 0, own_long = 0;
  for (int s = tid; s < S; s += kPlanThreads) {
    SharedSequence r{};
    r.q = kv_sequence(v, s);
    r.group = -1;
    if (bad) r.q.n = 0;
    int lo = -1, hi = G;  // the last group that begins at s or before
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (groups[mid].sequence <= s) lo = mid;
      else hi = mid;
    }
    if (lo >= 0 && r.q.n > 0) {
      const SharedGroup p = groups[lo];
      if (s < p.rows) {
        if (p.tokens < 0 || (p.tokens > 0 && r.q.first < p.tokens)) {
          report_index(v.status, p.tokens < 0 ? kIndexLength : kIndexRows);
          r.q.n = 0;
        } else if (p.tokens > 0) {
          r.group = lo;
          r.lead = p.tokens;
          r.leader = p.sequence;
        }
      }
    }
    const long long rows = static_cast<long long>(r.q.n) * a.group_heads;
    if (rows > 0) {
      const long long work = (rows + a.own_rows - 1) / a.own_rows *
                             (max((r.q.length - r.lead + a.own_tile - 1) / a.own_tile, 1) + a.own_start);
      if (a.prompt_blocks > 0 && rows > kRowLimit) {
        atomicAdd(&s_blocks, static_cast<unsigned long long>((rows + 15) / 16 * v.heads));
        own_long += work;
      } else {
        own += work;
      }
    }
    sequences[s] = r;
  }
#pragma unroll
  for (int d = 16; d > 0; d /= 2) {
    own += __shfl_xor_sync(0xFFFFFFFFu, own, d);
    own_long += __shfl_xor_sync(0xFFFFFFFFu, own_long, d);
  }
  if (lane == 0 && own > 0) atomicAdd(&s_own, static_cast<unsigned long long>(own));
  if (lane == 0 && own_long > 0) atomicAdd(&s_long, static_cast<unsigned long long>(own_long));
  __syncthreads();

  // The groups' rows: from the first to the last of their sequences that have any; and what a
  // shared part saves: all of their sequences but one would read its tokens again.
  for (int g = warp; g < G; g += kPlanThreads / 32) {
    SharedGroup p = groups[g];
    // (bounds out of order may be any numbers)
    const int from = bad ? 0 : p.sequence, to = bad ? 0 : p.rows;
    int row0 = INT_MAX, end = 0, members = 0;
    for (int s = from + lane; s < to; s += 32) {
      const SharedSequence q = sequences[s];
      if (q.group == g) {
        row0 = min(row0, q.q.row0);
        end = max(end, q.q.row0 + q.q.n);
        ++members;
      }
    }
    __syncwarp();
    row0 = __reduce_min_sync(0xFFFFFFFFu, row0);
    end = __reduce_max_sync(0xFFFFFFFFu, end);
    members = __reduce_add_sync(0xFFFFFFFFu, members);
    // A last block of few rows costs as much as a whole one: where one or two sequences are all of
    // it, they read the shared tokens for themselves.
    const int rest = row0 < end ? (end - row0) * a.group_heads % a.unit_rows : 0;
    if (a.drop && rest > 0 && rest <= kRowLimit && (end - row0) * a.group_heads > a.unit_rows) {
      const int s = to - 1 - lane;
      const SharedSequence q = sequences[max(s, 0)];
      const bool in = s >= from && q.group == g;
      const int first = in ? q.q.row0 : INT_MAX;
      const uint32_t there = __ballot_sync(0xFFFFFFFFu, in);
      int cut = end, dropped = 0;
      for (uint32_t left = there; left != 0 && dropped < 2 && (end - cut) * a.group_heads < rest;
           left &= left - 1, ++dropped)
        cut = min(cut, __shfl_sync(0xFFFFFFFFu, first, __ffs(left) - 1));
      if ((end - cut) * a.group_heads >= rest && (end - cut) * a.group_heads <= kRowLimit &&
          cut > row0) {
        if (in && first >= cut) {
          sequences[s].group = -1;
          const long long rows = static_cast<long long>(q.q.n) * a.group_heads;
          atomicAdd(&s_own, static_cast<unsigned long long>((rows + a.own_rows - 1) / a.own_rows *
                                                            (q.lead / a.own_tile)));
        }
        end = cut;
        members -= dropped;
      }
    }
    __syncwarp();
    p.row0 = p.rows = p.tiles = p.blocks = p.pieces = 0;
    if (row0 < end) {
      p.row0 = row0;
      p.rows = end - row0;
      p.tiles = (p.tokens + a.tile - 1) / a.tile;
      p.blocks = (p.rows * a.group_heads + a.unit_rows - 1) / a.unit_rows;
      if (lane == 0) {
        atomicMax(&s_most, p.tiles);
        atomicAdd(&s_tiles, static_cast<unsigned long long>(p.tiles) * p.blocks * v.heads);
        atomicAdd(&s_saved, static_cast<unsigned long long>(members - 1) * p.tokens);
      }
    }
    if (lane == 0) groups[g] = p;
    __syncwarp();
  }
  __syncthreads();
  const bool worth = static_cast<long long>(s_saved) * v.heads >= a.worth;
  const bool prompts = static_cast<long long>(s_blocks) > a.prompt_blocks;
  // How many SMs take the shared part, and the longest run of tiles of a unit there (the longest
  // group's cut into 1, 2, ... pieces): what takes the least time, the shared part as rounds of
  // equal units and in parts, the own ones beside it, and has room. Numbers of SMs around those
  // that the two parts' work is in proportion to.
  {
    // (12 x 9 tokens of 4 heads over 8192 shared and 3000 own, too few blocks for the kernel of prompts:
    // 124 us; 1620 when their own parts were not counted and got one SM)
    const float own_us = static_cast<float>(s_own + (prompts ? 0 : s_long)) * a.own_us;
    const float shared_us = static_cast<float>(s_tiles) * a.tile_us / static_cast<float>(a.per_sm);
    const float middle = static_cast<float>(a.sms) * (shared_us / (shared_us + own_us + 1e-6f));
    const int sms = min(max(static_cast<int>(middle + static_cast<float>(a.sms * ((tid & 15) - 7)) / 32.0f + 0.5f), 1),
                        max(a.sms - 1, 1));
    float best = INFINITY;
    int best_chunk = 1;
    const int most_pieces = min(s_most, G <= 16 ? 512 : 64);
    for (int cut = (tid >> 4) + 1; cut <= most_pieces && worth; cut += kPlanThreads / 16) {
      const int chunk = (s_most + cut - 1) / cut;
      long long units = 0, parts = 0, tiles = 0;
      for (int g = 0; g < G; ++g) {
        const SharedGroup p = groups[g];
        const long long pieces = (p.tiles + chunk - 1) / chunk;
        units += pieces * p.blocks * v.heads;
        tiles += static_cast<long long>(p.tiles) * p.blocks * v.heads;
        parts += pieces * p.rows * a.group_heads * v.heads;
      }
      // (half as rounds of units of the longest run, half as if work could be dealt out evenly)
      const float takers = static_cast<float>(sms * a.per_sm);
      const float rounds = ceilf(static_cast<float>(units) / takers);
      float us = 0.5f * a.tile_us *
                 (rounds * (static_cast<float>(chunk) + a.start) +
                  fmaxf((static_cast<float>(tiles) + a.start * static_cast<float>(units)) / takers,
                        static_cast<float>(chunk) + a.start));
      const float other = own_us / static_cast<float>(max(a.sms - sms, 1)) + a.own_first;
      us = a.sms == 1 ? us + other : fmaxf(us + a.first, other);
      us += static_cast<float>(parts) * a.part_us;
      if (parts <= plan.parts && us < best) best = us, best_chunk = chunk;
    }
    __syncwarp();
    // (of equal ones the lowest thread's)
    unsigned long long key =
        static_cast<unsigned long long>(__float_as_uint(best)) << 32 | static_cast<unsigned>(tid);
#pragma unroll
    for (int d = 16; d > 0; d /= 2) key = min(key, __shfl_xor_sync(0xFFFFFFFFu, key, d));
    if (lane == 0) s_key[warp] = key;
    __syncthreads();
    key = s_key[lane];
#pragma unroll
    for (int d = 16; d > 0; d /= 2) key = min(key, __shfl_xor_sync(0xFFFFFFFFu, key, d));
    if (tid == static_cast<int>(key & 0xFFFFFFFFu)) s_chunk = best_chunk, s_sms = worth ? sms : 0;
    __syncthreads();
  }
  if (warp == 0) {
    const int chunk = s_chunk;
    long long units_before = 0, parts_before = 0;
    for (int g0 = 0; g0 < G; g0 += 32) {
      const int g = g0 + lane;
      SharedGroup p{};
      if (g < G) p = groups[g];
      p.pieces = worth ? (p.tiles + chunk - 1) / chunk : 0;
      long long units = static_cast<long long>(p.pieces) * p.blocks * v.heads;
      long long parts = static_cast<long long>(p.pieces) * p.rows * a.group_heads * v.heads;
      const long long my_units = units, my_parts = parts;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const long long u = __shfl_up_sync(0xFFFFFFFFu, units, d);
        const long long q = __shfl_up_sync(0xFFFFFFFFu, parts, d);
        if (lane >= d) units += u, parts += q;
      }
      p.unit0 = static_cast<int>(min(units_before + units - my_units, 0x7FFFFFFFll));
      p.part0 = parts_before + parts - my_parts;
      if (g < G) groups[g] = p;
      units_before += __shfl_sync(0xFFFFFFFFu, units, 31);
      parts_before += __shfl_sync(0xFFFFFFFFu, parts, 31);
    }
    if (lane == 0) {
      // (more than there is room for only where rows are in several sequences: nothing is computed)
      const bool room = parts_before <= plan.parts && units_before <= INT_MAX;
      plan.head->units = room ? static_cast<int>(units_before) : 0;
      plan.head->shared_sms = s_sms;
      plan.head->own_sms = max(a.sms - s_sms, 1);
      plan.head->shared = PromptList{0u, 0};
      plan.head->own = PromptList{0u, prompts ? kRowLimit : kNoRowLimit};
      if (!room) report_index(v.status, kIndexRows);
      s_bad = room ? 0 : 1;
    }
    __syncwarp();
  }
  __syncthreads();
  for (int s = tid; s < S; s += kPlanThreads) {
    SharedSequence r = sequences[s];
    if (r.group >= 0) {
      // (its rows are the group's, whatever the offsets are)
      const SharedGroup p = groups[r.group];
      if (p.pieces > 0 && r.q.row0 >= p.row0 && r.q.row0 + r.q.n <= p.row0 + p.rows) {
        r.start = r.lead;
        r.part0 = p.part0;
        r.group_rows = p.rows * a.group_heads;
        r.pieces = p.pieces;
        r.row = (r.q.row0 - p.row0) * a.group_heads;
      } else {
        r.group = -1;
      }
    }
    if (s_bad) r.q.n = 0;
    plan.sequences[s] = r;
  }
  if (G <= kPlanGroups)
    for (int g = tid; g < G; g += kPlanThreads) plan.groups[g] = groups[g];
}

// kWarps warps a row and head: its own part, whole or in pieces, and its shared ones, in a fixed
// order.
template <int HSP, int kWarps>
__global__ void __launch_bounds__(128) shared_join_sm103a_kernel(const AttendArgs a, int q_heads) {
  grid_dependency_wait();
  constexpr int V = HSP / 32, kRowsAtOnce = 4 / kWarps;
  using Vec = typename std::conditional<V == 4, float4, float2>::type;
  __shared__ Vec s_acc[4][32];
  __shared__ float s_sum[4], s_top[4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, w0 = warp % kWarps;
  const unsigned all = static_cast<unsigned>(a.v.rows) * static_cast<unsigned>(q_heads);
  const unsigned step = gridDim.x * kRowsAtOnce;
  unsigned i = blockIdx.x * kRowsAtOnce + warp / kWarps;
  int there = i < all ? a.plan.own_there[i] : 0;
  OwnRow w = i < all ? a.plan.own[i] : OwnRow{};
  for (; i < all; i += step) {
    const int this_there = there;
    const OwnRow r = w;
    if (i + step < all) {  // (asked for before this row is done)
      there = a.plan.own_there[i + step];
      w = a.plan.own[i + step];
    }
    if (this_there == 0) continue;  // (the warps of a row alike)
    const int first = max(r.pieces, 1), n = first + r.shared;
    // (two sequences that claim a row write this over each other)
    const bool whole_record = r.pieces >= 0 && r.shared >= 0 && r.at >= 0 &&
                              r.at + r.shared <= a.plan.parts && r.row >= 0 &&
                              r.row < kMaxRows && r.worker >= 0 &&
                              r.worker + r.pieces <= kMaxWorkers;
    if (!whole_record) continue;
    // Piece p's maximum, sum and output.
    auto piece = [&](int p, float& m, float& l) -> const float* {
      if (p < first && r.pieces > 0) {
        const int slot = p == 0 ? 2 * r.worker + 1 : 2 * (r.worker + p);
        const float* part = a.parts + static_cast<long long>(slot) * a.part_floats;
        m = part[r.row];
        l = part[kMaxRows + r.row];
        return part + 2 * kMaxRows + r.row * HSP;
      }
      const long long at = p < first ? static_cast<long long>(i) : r.at + p - first;
      const float2 x = p < first ? a.plan.own_ml[at] : a.plan.ml[at];
      m = x.x;
      l = x.y;
      return (p < first ? a.plan.own_o : a.plan.o) + at * HSP;
    };
    // Warp w0 takes pieces w0, w0 + kWarps, ..., relative to the largest maximum among its own.
    float top = kNothing, sum = 0.0f, acc[V] = {};
    for (int p0 = w0; p0 < n; p0 += 32 * kWarps) {
      const int p = p0 + lane * kWarps;
      float m = kNothing, l = 0.0f;
      const float* o = nullptr;
      if (p < n) o = piece(p, m, l);
      __syncwarp();
      float most = fmaxf(top, m);
#pragma unroll
      for (int d = 16; d > 0; d /= 2) most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, d));
      // (in two factors, neither of which comes out as 0, for the sums)
      const float back = ex2_approx(0.5f * (top - most));
      sum = sum * back * back;
#pragma unroll
      for (int k = 0; k < V; ++k) acc[k] *= back * back;
      top = most;
      const float half = ex2_approx(0.5f * (m - top)), c = half * half;
      sum = fmaf(l * half, half, sum);
      const int here = min((n - p0 + kWarps - 1) / kWarps, 32);
#pragma unroll 8
      for (int q = 0; q < here; ++q) {
        const float cq = __shfl_sync(0xFFFFFFFFu, c, q);
        const float* from = reinterpret_cast<const float*>(
            __shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(o), q));
        const Vec x = reinterpret_cast<const Vec*>(from)[lane];
        const float* v = reinterpret_cast<const float*>(&x);
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] = fmaf(v[k], cq, acc[k]);
      }
    }
#pragma unroll
    for (int d = 16; d > 0; d /= 2) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
    if constexpr (kWarps > 1) {
      s_acc[warp][lane] = *reinterpret_cast<const Vec*>(acc);
      if (lane == 0) s_sum[warp] = sum, s_top[warp] = top;
      __syncthreads();
      top = fmaxf(fmaxf(s_top[0], s_top[1]), fmaxf(s_top[2], s_top[3]));
      sum = 0.0f;
#pragma unroll
      for (int k = 0; k < V; ++k) acc[k] = 0.0f;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float half = ex2_approx(0.5f * (s_top[q] - top)), c = half * half;
        sum = fmaf(s_sum[q] * half, half, sum);
        const Vec x = s_acc[q][lane];
        const float* v = reinterpret_cast<const float*>(&x);
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] = fmaf(v[k], c, acc[k]);
      }
      __syncthreads();
      if (warp > 0) continue;
    }
    const int row = static_cast<int>(i / static_cast<unsigned>(q_heads));
    const int head = static_cast<int>(i - static_cast<unsigned>(row) * static_cast<unsigned>(q_heads));
    uint32_t y[V / 2];
#pragma unroll
    for (int k = 0; k < V; k += 2) {
      const float v0 = sum == 0.0f ? 0.0f : acc[k] / sum;
      const float v1 = sum == 0.0f ? 0.0f : acc[k + 1] / sum;
      if (a.half) {
        y[k / 2] = half2_of(v0, v1);
      } else {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v0, v1);
        y[k / 2] = *reinterpret_cast<const uint32_t*>(&b);
      }
    }
    if (lane * V < a.v.head_size) {
      uint16_t* to = static_cast<uint16_t*>(a.out) + row * a.out_token + head * a.out_head + lane * V;
      if constexpr (V == 4) *reinterpret_cast<uint2*>(to) = make_uint2(y[0], y[1]);
      else *reinterpret_cast<uint32_t*>(to) = y[0];
    }
  }
}

template <int HSP>
cudaError_t launch_join(const AttendArgs& a, int q_heads, long long rows_heads, int sms,
                        cudaStream_t stream) {
  // Four warps a row while there are places for all of them at once (64 rows of 57 pieces take 8 us
  // with four warps each, 21 with one).
  const long long most = 16LL * sms;
  return rows_heads <= most
             ? launch_programmatic(shared_join_sm103a_kernel<HSP, 4>,
                                   dim3(static_cast<unsigned>(rows_heads)), 128, 0, stream, a, q_heads)
             : launch_programmatic(shared_join_sm103a_kernel<HSP, 1>,
                                   dim3(static_cast<unsigned>(std::min((rows_heads + 3) / 4, most))),
                                   128, 0, stream, a, q_heads);
}

size_t up16(size_t n) { return (n + 15) / 16 * 16; }

// The workspace: the rows kernel's, the plan, the parts.
size_t lay_out(int head_size, long long rows_heads, int sequences, int groups, char* base,
               SharedPlan& plan) {
  size_t at = up16(rows_workspace_bytes(head_size));
  auto take = [&](size_t bytes) {
    char* const got = base + at;
    at += up16(bytes);
    return got;
  };
  plan.group_count = groups;
  plan.parts = rows_heads + kSpareParts;
  plan.head = reinterpret_cast<SharedHead*>(take(sizeof(SharedHead)));
  plan.groups = reinterpret_cast<SharedGroup*>(take(static_cast<size_t>(groups) * sizeof(SharedGroup)));
  plan.sequences =
      reinterpret_cast<SharedSequence*>(take(static_cast<size_t>(sequences) * sizeof(SharedSequence)));
  plan.ml = reinterpret_cast<float2*>(take(static_cast<size_t>(plan.parts) * sizeof(float2)));
  const size_t row = static_cast<size_t>(padded_head(head_size)) * sizeof(float);
  plan.o = reinterpret_cast<float*>(take(static_cast<size_t>(plan.parts) * row));
  plan.own_there = reinterpret_cast<int*>(take(static_cast<size_t>(rows_heads) * sizeof(int)));
  plan.own = reinterpret_cast<OwnRow*>(take(static_cast<size_t>(rows_heads) * sizeof(OwnRow)));
  plan.own_ml = reinterpret_cast<float2*>(take(static_cast<size_t>(rows_heads) * sizeof(float2)));
  plan.own_o = reinterpret_cast<float*>(take(static_cast<size_t>(rows_heads) * row));
  return at;
}

}  // namespace

size_t cache_attention_shared_workspace_bytes(int head_size, long long rows_heads, int sequences,
                                              int groups) {
  SharedPlan plan;
  return lay_out(head_size, rows_heads, sequences, groups, nullptr, plan);
}

int cache_attention_shared_launch(const csa_kv_cache& cache, const csa_kv_batch& batch,
                                  const AttendCall& call, const int* groups, const int* shared,
                                  int group_count, cudaStream_t stream, const DeviceInfo& dev,
                                  std::string& err) {
  AttendArgs a = rows_args(cache, batch, call, call.workspace, dev);
  const long long rows_heads = static_cast<long long>(batch.rows) * call.q_heads;
  lay_out(cache.head_size, rows_heads, batch.sequences, group_count,
          static_cast<char*>(call.workspace), a.plan);
  const int sms = std::min(dev.sm_count, kMaxSms);
  const long long batch_rows = static_cast<long long>(batch.rows) * a.group;
  const bool prefix_tc = batch_rows >= static_cast<long long>(kPrefixFrom) * group_count;
  const bool prefix_eight = batch_rows <= 8LL * group_count;
  const int hsp = padded_head(cache.head_size), sub = cache.page_tokens < 32 ? 1 : 2;
  // (rows a block of the own parts, and whether some may be prompts': see cache_attention_launch)
  const long long most_rows = static_cast<long long>(batch.max_new) * a.group;
  a.prompt_blocks = static_cast<long long>(kBlocksPerSm) * sms;
  const long long sequences = std::min<long long>(batch.sequences, batch_rows / (kRowLimit + 1));
  const bool prompts = most_rows > kRowLimit &&
                       (batch_rows / 16 + sequences) * cache.heads > a.prompt_blocks;
  if (!prompts) a.prompt_blocks = 0;
  const bool eight =
      most_rows <= 8 || (a.group <= 8 && (prompts || batch_rows <= 8LL * batch.sequences));

  // The times that the plan weighs the two parts by (measured as the best of 9 divisions of the SMs
  // for 12 batches; what it chooses is within 5 % of those).
  // What the kernel of few rows needs for a tile: an SM's groups take its codes at 38 GB/s between
  // them (5.8 TB/s over all), or twice as long with 16 rows.
  auto groups_of = [&](bool of_eight) {
    return hsp == 64 ? (of_eight ? kGroups<64, 1> : kGroups<64, 2>)
                     : (of_eight ? kGroups<128, 1> : kGroups<128, 2>);
  };
  auto rows_tile_us = [&](bool of_eight) {
    return (of_eight ? 1.0f : 2.0f) * 64.0f * sub * 2.0f * cache.head_size / 38e3f *
           groups_of(of_eight);
  };

  PlanArgs p;
  p.v = a.v;
  p.sms = sms;
  p.own_rows = eight ? 8 : 16;
  p.own_tile = 64 * sub;
  p.own_start = (eight ? 2 : 3) * (2 / sub);
  p.own_us = cache.heads * rows_tile_us(eight) / groups_of(eight);
  p.groups = groups;
  p.shared = shared;
  p.plan = a.plan;
  p.rows_heads = rows_heads;
  p.group_heads = a.group;
  p.worth = shared_part_mode() == CSA_SHARED_ALWAYS
                ? 0
                : kWorthBytes * sms / kMaxSms / (2 * cache.head_size);
  p.prompt_blocks = a.prompt_blocks;
  p.part_us = 8.0f * static_cast<float>(hsp) / 5e6f;  // (8 HSP bytes at 5 TB/s)
  p.own_first = 8.0f;
  if (prefix_tc) {
    p.unit_rows = kPrefixRows;
    p.tile = kPrefixTile;
    p.per_sm = 1;
    p.tile_us = hsp == 64 ? 1.0f : 1.2f;
    p.first = 8.0f;
    p.start = 5.0f;  // (9000 cycles from a unit's end to the next one's first scores, 1900 a tile)
    p.drop = true;
  } else {
    p.unit_rows = prefix_eight ? 8 : 16;
    p.tile = 64 * sub;
    p.per_sm = groups_of(prefix_eight);
    p.tile_us = rows_tile_us(prefix_eight);
    p.start = static_cast<float>((prefix_eight ? 2 : 3) * (2 / sub));
    p.first = 4.0f;
    p.drop = false;
  }
  const unsigned clear =
      static_cast<unsigned>(std::min<long long>((rows_heads / 4 + kPlanThreads) / kPlanThreads, sms));
  cudaError_t e = launch_programmatic(shared_plan_sm103a_kernel, dim3(1 + clear), kPlanThreads, 0,
                                      stream, p);
  int rc = CSA_OK;
  // (not even were all tables full and shared)
  const bool never = static_cast<double>(batch.sequences - 1) * batch.table_width *
                         cache.page_tokens * cache.heads <
                     static_cast<double>(p.worth);
  if (e == cudaSuccess && !never) {
    if (prefix_tc) {
      rc = cache_prefix_launch(cache, batch, call, a.plan, false, stream, dev, err);
    } else {
      a.prefix = 1;
      e = launch_rows<true>(a, prefix_eight, cache.format, sms, dev, stream, rc, err);
      a.prefix = 0;
    }
    a.beside = sms > 1 ? 1 : 0;
  }
  if (e == cudaSuccess && rc == CSA_OK)
    e = launch_rows<true>(a, eight, cache.format, sms, dev, stream, rc, err);
  if (e == cudaSuccess && rc == CSA_OK && prompts)
    rc = cache_prefix_launch(cache, batch, call, a.plan, true, stream, dev, err);
  if (e == cudaSuccess && rc == CSA_OK) {
    e = hsp == 64 ? launch_join<64>(a, call.q_heads, rows_heads, sms, stream)
                  : launch_join<128>(a, call.q_heads, rows_heads, sms, stream);
  }
  if (rc != CSA_OK) {
    err = "cache_attention_shared_forward: " + err;
    return rc;
  }
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) {
    err = std::string("cache_attention_shared_forward: launch: ") + cudaGetErrorString(e);
    return CSA_ERR_LAUNCH;
  }
  return CSA_OK;
}

}  // namespace csa
