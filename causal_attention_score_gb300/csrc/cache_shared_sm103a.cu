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
// Four launches: a plan (one CTA: the batch's entries read and checked once, units of the shared
// part and where their results go), the shared part, the own parts, and the joining of own parts
// that were split. The shared part is cut along its tokens too, as far as SMs are left without
// work; a row of an own part that no split touches takes its shared parts in as it is finished.
//
// The shared part goes to the tcgen05 kernel (256 rows x 64 keys a step; its units here have no
// masks) where the groups have rows enough, to the kernel of few rows otherwise.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>
#include <string>

#include "cache_rows.cuh"
#include "cache_shared.cuh"
#include "csa_internal.h"

namespace csa {
namespace {

constexpr int kPlanThreads = 1024;
// From this many rows a group on average (tokens x query heads of a kv head) the shared part is
// the tcgen05 kernel's.
constexpr int kPrefixFrom = 33;
// Room for parts beyond one for each row and head: what cutting along the tokens may take.
constexpr long long kSpareParts = 2LL * kMaxSms * kPrefixRows;

struct PlanArgs {
  KvView v;
  const int* groups;  // [group_count + 1]
  const int* shared;  // [group_count]
  SharedPlan plan;
  int group_heads;
  int unit_rows, tile;  // of the shared part's kernel
  int workers;          // what works on a unit at a time
  int start;            // what a unit costs beyond its tiles, in tiles
};

// Sum over the CTA and each thread's share of it before it, for a run of values a thread each.
struct Sums {
  long long warp[kPlanThreads / 32];
  __device__ long long before(long long mine, long long& total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    long long up = mine;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const long long x = __shfl_up_sync(0xFFFFFFFFu, up, d);
      if (lane >= d) up += x;
    }
    __syncthreads();
    if (lane == 31) warp[w] = up;
    __syncthreads();
    long long at = up - mine;
    total = 0;
    for (int i = 0; i < kPlanThreads / 32; ++i) {
      if (i < w) at += warp[i];
      total += warp[i];
    }
    return at;
  }
};

__global__ void __launch_bounds__(kPlanThreads, 1) shared_plan_sm103a_kernel(const PlanArgs a) {
  __shared__ Sums sums;
  __shared__ int s_bad, s_most;
  __shared__ unsigned long long s_best;
  __shared__ int s_chunk;
  const KvView& v = a.v;
  const SharedPlan& plan = a.plan;
  const int tid = threadIdx.x, G = plan.group_count, S = v.sequences;
  grid_dependency_wait();
  if (tid == 0) s_bad = s_most = 0, s_best = ~0ull;
  __syncthreads();

  // The groups: bounds in order, whole pages.
  for (int g = tid; g < G; g += kPlanThreads) {
    const int from = a.groups[g], to = a.groups[g + 1], tokens = a.shared[g];
    if (from < 0 || to < from || to > S) s_bad = 1;
    const bool ok = tokens >= 0 && tokens % v.page_tokens == 0 &&
                    tokens <= static_cast<long long>(v.table_width) * v.page_tokens;
    SharedGroup p{};
    p.sequence = from;
    p.rows = to;  // (for now: where the group ends)
    p.tokens = ok ? tokens : -1;
    plan.groups[g] = p;
  }
  __syncthreads();
  const bool bad = s_bad != 0;  // then nothing is computed
  if (bad && tid == 0) report_index(v.status, kIndexSequence);

  // The sequences, each with its group (found by its bounds).
  for (int s = tid; s < S; s += kPlanThreads) {
    SharedSequence r{};
    r.q = kv_sequence(v, s);
    r.group = -1;
    if (bad) r.q.n = 0;
    int lo = -1, hi = G;  // the last group that begins at s or before
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (plan.groups[mid].sequence <= s) lo = mid;
      else hi = mid;
    }
    if (lo >= 0 && s < plan.groups[lo].rows && r.q.n > 0) {
      const int tokens = plan.groups[lo].tokens;
      if (tokens < 0 || (tokens > 0 && r.q.first < tokens)) {
        report_index(v.status, tokens < 0 ? kIndexLength : kIndexRows);
        r.q.n = 0;
      } else if (tokens > 0) {
        r.group = lo;
        r.start = tokens;
      }
    }
    plan.sequences[s] = r;
  }
  __syncthreads();

  // The groups' rows: from the first to the last of their sequences that have any.
  for (int g = tid >> 5; g < G; g += kPlanThreads / 32) {
    SharedGroup p = plan.groups[g];
    // (bounds out of order may be any numbers)
    const int from = bad ? 0 : p.sequence, to = bad ? 0 : p.rows;
    int row0 = INT_MAX, end = 0;
    for (int s = from + (tid & 31); s < to; s += 32) {
      const SharedSequence q = plan.sequences[s];
      if (q.group == g) {
        row0 = min(row0, q.q.row0);
        end = max(end, q.q.row0 + q.q.n);
      }
    }
    __syncwarp();
    row0 = __reduce_min_sync(0xFFFFFFFFu, row0);
    end = __reduce_max_sync(0xFFFFFFFFu, end);
    p.row0 = p.rows = p.tiles = p.blocks = p.pieces = 0;
    if (row0 < end) {
      p.row0 = row0;
      p.rows = end - row0;
      p.tiles = (p.tokens + a.tile - 1) / a.tile;
      p.blocks = (p.rows * a.group_heads + a.unit_rows - 1) / a.unit_rows;
      if ((tid & 31) == 0) atomicMax(&s_most, p.tiles);
    }
    if ((tid & 31) == 0) plan.groups[g] = p;
    __syncwarp();
  }
  __syncthreads();

  // The longest run of tiles of a unit: the longest group's cut into 1, 2, ... 1024 pieces, that
  // which takes the least time as rounds of equal units, and room.
  {
    const int chunk = max((s_most + tid) / (tid + 1), 1);
    long long units = 0, parts = 0;
    for (int g = 0; g < G; ++g) {
      const SharedGroup p = plan.groups[g];
      const long long pieces = (p.tiles + chunk - 1) / chunk;
      units += pieces * p.blocks * v.heads;
      parts += pieces * p.rows * a.group_heads * v.heads;
    }
    const unsigned long long rounds = (units + a.workers - 1) / a.workers;
    const unsigned long long cost =
        parts <= plan.parts ? min(rounds * (chunk + a.start), 1ull << 50) : 1ull << 51;
    // (of equal ones the fewest pieces)
    atomicMin(&s_best, cost << 11 | static_cast<unsigned long long>(tid));
    __syncthreads();
    if (tid == static_cast<int>(s_best & 2047)) s_chunk = chunk;
    __syncthreads();
  }
  const int chunk = s_chunk;
  long long units_before = 0, parts_before = 0;
  for (int g0 = 0; g0 < G; g0 += kPlanThreads) {
    const int g = g0 + tid;
    SharedGroup p{};
    if (g < G) {
      p = plan.groups[g];
      p.pieces = (p.tiles + chunk - 1) / chunk;
    }
    long long units = 0, parts = 0;
    const long long mine = static_cast<long long>(p.pieces) * p.blocks * v.heads;
    const long long room = static_cast<long long>(p.pieces) * p.rows * a.group_heads * v.heads;
    p.unit0 = static_cast<int>(units_before + sums.before(mine, units));
    p.part0 = parts_before + sums.before(room, parts);
    units_before += units;
    parts_before += parts;
    if (g < G) plan.groups[g] = p;
  }
  if (tid == 0) {
    // (more than there is room for only where rows are in several sequences: nothing is computed)
    const bool room = parts_before <= plan.parts && units_before <= INT_MAX;
    plan.head->units = room ? static_cast<int>(units_before) : 0;
    plan.head->list = PromptList{0u, 0};
    if (!room) report_index(v.status, kIndexRows);
    s_bad = room ? 0 : 1;
  }
  __syncthreads();
  if (s_bad)
    for (int s = tid; s < S; s += kPlanThreads) plan.sequences[s].q.n = 0;
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
  plan.o = reinterpret_cast<float*>(
      take(static_cast<size_t>(plan.parts) * padded_head(head_size) * sizeof(float)));
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
  lay_out(cache.head_size, static_cast<long long>(batch.rows) * call.q_heads, batch.sequences,
          group_count, static_cast<char*>(call.workspace), a.plan);
  const int sms = std::min(dev.sm_count, kMaxSms);
  const long long batch_rows = static_cast<long long>(batch.rows) * a.group;
  const bool prefix_tc = batch_rows >= static_cast<long long>(kPrefixFrom) * group_count;
  const bool prefix_eight = batch_rows <= 8LL * group_count;
  const int hsp = padded_head(cache.head_size), sub = cache.page_tokens < 32 ? 1 : 2;

  PlanArgs p;
  p.v = a.v;
  p.groups = groups;
  p.shared = shared;
  p.plan = a.plan;
  p.group_heads = a.group;
  if (prefix_tc) {
    p.unit_rows = kPrefixRows;
    p.tile = kPrefixTile;
    p.workers = dev.sm_count;
    p.start = 5;  // (9000 cycles from a unit's end to the next one's first scores, 1900 a tile)
  } else {
    p.unit_rows = prefix_eight ? 8 : 16;
    p.tile = 64 * sub;
    p.workers = sms * (hsp == 64 ? (prefix_eight ? kGroups<64, 1> : kGroups<64, 2>)
                                 : (prefix_eight ? kGroups<128, 1> : kGroups<128, 2>));
    p.start = (prefix_eight ? 2 : 3) * (2 / sub);
  }
  cudaError_t e = launch_programmatic(shared_plan_sm103a_kernel, dim3(1), kPlanThreads, 0, stream, p);
  int rc = CSA_OK;
  if (e == cudaSuccess) {
    if (prefix_tc) {
      rc = cache_prefix_launch(cache, batch, call, a.plan, stream, dev, err);
    } else {
      a.prefix = 1;
      e = launch_rows<true>(a, prefix_eight, cache.format, sms, dev, stream, rc, err);
      a.prefix = 0;
    }
  }
  // (rows a block: see cache_attention_launch)
  const long long most_rows = static_cast<long long>(batch.max_new) * a.group;
  const bool eight = most_rows <= 8 || (a.group <= 8 && batch_rows <= 8LL * batch.sequences);
  if (e == cudaSuccess && rc == CSA_OK)
    e = launch_rows<true>(a, eight, cache.format, sms, dev, stream, rc, err);
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
