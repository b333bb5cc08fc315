// Attention for a batch whose sequences share long beginnings: what the plan, the kernels of the
// shared part and those of the sequences' own parts hand to one another.
#pragma once

#include <cstdint>

#include "csa_internal.h"
#include "kv_cache.cuh"

namespace csa {

// Lets the kernel behind this one in the stream start; it waits for this one's end itself.
__device__ __forceinline__ void grid_dependents_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

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

// A sequence as the plan read and checked it. Its tokens below `lead` are looked up in sequence
// `leader`'s table row; those below `start` are the shared part's (start is 0 or lead).
struct alignas(16) SharedSequence {
  KvSequence q;
  int start, lead, leader;
  int group;  // -1: none, or one whose shared part is not worth a unit of its own
  // Where its shared parts are (see shared_part): the group's first one, its query rows of a kv
  // head and pieces, and this sequence's first query row there.
  long long part0;
  int group_rows, pieces, row;
};

// What the kernels of the own parts leave for one row and head, beside its maximum, sum and output:
// where the rest of it is.
struct OwnRow {
  long long at;        // of its shared parts, the first
  int shared;          // how many
  int pieces, worker;  // an own part in pieces, the first by this worker (0: whole, below)
  int row;             // of that piece's rows
};

struct SharedHead {
  int units;          // of the shared part
  int shared_sms;     // that work on it, while
  int own_sms;        // these work on the own parts
  PromptList shared;  // those taken
  PromptList own;     // of the own parts: sequences of more than row_limit rows are its kernel's
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
  // by row and query head:
  int* own_there;   // 0: no row of a sequence
  OwnRow* own;
  float2* own_ml;
  float* own_o;     // [..][padded head size]
};

__device__ __forceinline__ long long shared_part(long long part0, int group_rows, int pieces,
                                                 int head, int rr) {
  return part0 + (static_cast<long long>(head) * group_rows + rr) * pieces;
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

// The tcgen05 kernel over the shared tokens, and over the own parts of sequences with many rows
// (cache_prefix_sm103a.cu).
int cache_prefix_launch(const csa_kv_cache& cache, const csa_kv_batch& batch,
                        const AttendCall& call, const SharedPlan& plan, bool own,
                        cudaStream_t stream, const DeviceInfo& dev, std::string& err);

}  // namespace csa
