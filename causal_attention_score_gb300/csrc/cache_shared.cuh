// Attention for a batch whose sequences share long beginnings: what the plan, the kernels of the
// shared part and those of the sequences' own parts hand to one another.
#pragma once

#include <cstdint>

#include "csa_internal.h"
#include "kv_cache.cuh"

namespace csa {

// A unit of the tcgen05 form: rows and tokens of a tile.
constexpr int kPrefixRows = 256, kPrefixTile = 64;

// A group of sequences, next to each other in the batch, and its shared tokens. Its query rows
// (rows x query heads of a kv head), cut into blocks, times the kv heads, times `pieces` runs of
// its tiles of tokens are the units of work of the shared part.
struct SharedGroup {
  int sequence;       // whose table names the shared pages
  int row0, rows;     // of the batch
  int tokens, tiles;  // shared
  int blocks, pieces;
  int unit0;          // units of the groups before
  long long part0;    // parts of the groups before
};

// A sequence as the plan read and checked it.
struct SharedSequence {
  KvSequence q;
  int start;  // its first token that is not shared
  int group;  // -1: none, or none with shared tokens
};

struct SharedHead {
  int units;
  PromptList list;  // of the tcgen05 form
};

// What a unit leaves for each of its rows: the running maximum, the sum and the output. Row rr
// of a group and kv head has `pieces` of them, one after another.
struct SharedPlan {
  SharedHead* head;
  SharedGroup* groups;
  SharedSequence* sequences;
  float2* ml;   // [parts]
  float* o;     // [parts][padded head size]
  int group_count;
  long long parts;  // that there is room for
};

__device__ __forceinline__ long long shared_part(const SharedGroup& g, int group_heads, int head,
                                                 int rr) {
  return g.part0 +
         (static_cast<long long>(head) * g.rows * group_heads + rr) * g.pieces;
}

// The group of unit u.
__device__ __forceinline__ int shared_group_of(const SharedPlan& plan, int u) {
  int lo = 0, hi = plan.group_count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (plan.groups[mid].unit0 <= u) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Unit u of its group: blocks of rows next to each other, which read the same keys, then heads,
// then pieces.
struct SharedUnit {
  int head, block, piece, tile0, tiles;
};
__device__ __forceinline__ SharedUnit shared_unit(const SharedGroup& g, int heads, int u) {
  SharedUnit r;
  const int i = u - g.unit0;
  const int rest = i / g.blocks;
  r.block = i - rest * g.blocks;
  r.piece = rest / heads;
  r.head = rest - r.piece * heads;
  r.tile0 = static_cast<int>(static_cast<long long>(r.piece) * g.tiles / g.pieces);
  r.tiles = static_cast<int>(static_cast<long long>(r.piece + 1) * g.tiles / g.pieces) - r.tile0;
  return r;
}

// Joins the n parts from `at` on to (m, l, acc), four elements from d on of a row.
template <int HSP>
__device__ __forceinline__ void join_parts(const SharedPlan& plan, long long at, int n, int d,
                                           float m, float& l, float4& acc) {
  float top = m;
#pragma unroll 8
  for (int i = 0; i < n; ++i) top = fmaxf(top, plan.ml[at + i].x);
  // (in two factors, neither of which comes out as 0, for the sum)
  float half = ex2_approx(0.5f * (m - top)), c = half * half;
  l = l * half * half;
  acc.x *= c;
  acc.y *= c;
  acc.z *= c;
  acc.w *= c;
#pragma unroll 8
  for (int i = 0; i < n; ++i) {
    const float2 x = plan.ml[at + i];
    const float4 o = *reinterpret_cast<const float4*>(plan.o + (at + i) * HSP + d);
    half = ex2_approx(0.5f * (x.x - top));
    c = half * half;
    l = fmaf(x.y * half, half, l);
    acc.x = fmaf(o.x, c, acc.x);
    acc.y = fmaf(o.y, c, acc.y);
    acc.z = fmaf(o.z, c, acc.z);
    acc.w = fmaf(o.w, c, acc.w);
  }
}

// The tcgen05 kernel over the shared tokens (cache_prefix_sm103a.cu).
int cache_prefix_launch(const csa_kv_cache& cache, const csa_kv_batch& batch,
                        const AttendCall& call, const SharedPlan& plan, cudaStream_t stream,
                        const DeviceInfo& dev, std::string& err);

}  // namespace csa
