// The kernel of cache_prompt_sm103a.cu and, with another kMode, of cache_prefix_sm103a.cu.
//
// Attention of many new tokens per sequence (prompts and their chunks) over the
// paged 8-bit cache: the same function as the rows kernel of
// cache_attention_sm103a.cu, on tcgen05.
//
// A unit of work is 256 rows (tokens x query heads of one kv head) of a
// sequence: two groups A and B of 128, each a TMEM accumulator's lanes, which
// share every tile of 64 keys. One CTA per SM takes units from a counter
// (longest first within a sequence), with 16 warps:
//  - warps 0..7: softmax, warps 0..3 group A, 4..7 group B, a thread a row. Per
//    tile: scores from TMEM, x - m, their maximum, and the weights exp2(x - m) as
//    fp16 over S (P, the second product's A operand in TMEM), all 64 of a row in
//    registers at once. m is raised, to 7 below the maximum, only when a value passes
//    m + 15; then the thread's O row and its l are rescaled. They copy a unit's Q
//    to shared memory before they write the last one's O / l.
//  - warps 8..11: conversion, from raw codes in shared memory to the
//    128-byte-swizzle K-major layout, K as [token][element] in Q's type, V
//    transposed in registers to [element][token] in fp16 (both exact). A slot of
//    the ring holds V of tile j and K of tile j + 1, what one step of the products
//    reads.
//  - warps 12 and 13: one thread each issues a group's products, S = Q K^T of a tile
//    or O += P V of one before it, whichever has its operands first (in a fixed order
//    V waited for the next K: 207 us instead of 197 for the chunks below). S has two
//    buffers of 64 columns, so the softmax finds the next scores ready when it is done with the
//    last. A thread's MMAs run in issue order, so S may overwrite the weights that
//    the product issued before it reads. (With both groups on one warp the issue
//    itself, 48 to 96 cycles an MMA, was the longest path.)
//  - warp 14: takes a unit from the list's counter (workspace, cleared by the rows
//    kernel ahead in the stream) when the copies ask for it, some tiles before they are
//    through with the last one: early enough to hide the way to the first scores, late
//    enough that a CTA holds no unit that another could have begun.
//  - warp 15: copies. A page's part of a tile is contiguous, so one thread moves it
//    with bulk copies (two slots ahead of the conversion); the warp also turns the
//    scales into the softmax's factors.
// Every role's loop is kept short: with the codes fetched to registers by the
// conversion warps themselves, straight-line code that one warp in four executes once
// per tile missed the instruction cache and the conversion was the longest path.
//
// Scales (see cache_attention_sm103a.cu): with c ks and log2(vs) per 16 tokens in
// shared memory, x = s (c ks) + log2(vs) and the weight has V's scale in it; the
// denominator sums w / vs, and what that loses beside far larger scales apart.
//
// Bound: 4 HSP flops and one exp2 per row and key; per 256 rows x 64 keys 1024 cycles
// of MMA at the dense rate (HSP = 128), 1280 at the rates that these shapes run at alone
// (48 cycles for 128 x 64 x 16 with both operands in shared memory, whose reads bound it;
// 64 for 128 x 128 x 16 with A in TMEM). Measured: 2 prompts of 4096 tokens, 16 heads of
// 128: 144 us (955 TFLOP/s); 5 chunks of 200 to 777 tokens after up to 9000, 32 query and
// 4 kv heads of 64: 174 us. A step takes 1900 cycles (1650 with heads of 64): a softmax
// warp 1450 (1230) and the rest of waiting, a conversion warp 1700 (1160); a unit's end
// and the next one's first scores 9000. No unit is saturated (tensor pipe 44 %, issue
// slots 53 %, MUFU 22 %): what counts is the latency of each role's chain. What moved it:
// waits in which every lane looks at the barrier (one lane looking for its warp: 176 us
// instead of 147), all of the conversion's loads ahead of its stores (192 / 176), ring
// places counted instead of divided (147 / 144). Without gain: one pass over the scores
// with the maximum checked afterwards (155), a fourth ring slot (147), Q as fp16 for
// bf16 rows, which shortens K's conversion (154), the next unit's Q asked for under the last
// tile (146).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <string>

#include "cache_shared.cuh"
#include "csa_internal.h"
#include "kv_cache.cuh"
#include "sm103a_ptx.cuh"

namespace csa {
namespace {

constexpr int kSoftmaxWarps = 8;
constexpr int kConvertWarps = 4;
constexpr int kMmaWarp = kSoftmaxWarps + kConvertWarps;
constexpr int kListWarp = kMmaWarp + 2;
constexpr int kCopyWarp = kListWarp + 1;
constexpr int kThreads = 32 * (kCopyWarp + 1);
constexpr int kRows = 128;          // per group
constexpr int kUnitRows = 2 * kRows;
constexpr int kTile = 64;           // keys per step
constexpr int kSlots = 3;           // of the ring of converted keys and values
constexpr int kFactorSlots = 16;    // tiles whose factors are kept (more than are in the rings)
constexpr int kUnitSlots = 2;
constexpr int kAskAhead = 12;       // tiles before a unit's end when the next is asked for
constexpr int kTmemCols = 512;      // S_A (two buffers), S_B, O_A, O_B
constexpr float kRaise = 15.0f;     // an exponent past this raises m,
constexpr float kHeadroom = 7.0f;   // to this far below it
constexpr float kFar = 8.673617379884035e-19f;  // 2^-60: scales of V this far apart
constexpr float kNothing = -1e30f;  // the running maximum of a row that has seen nothing

static_assert(kUnitRows == kPrefixRows && kTile == kPrefixTile, "as the plan divides them");

struct PromptArgs {
  KvView v;
  const void* q;
  void* out;
  long long q_token, q_head, out_token, out_head;
  int half;
  int group;
  int window, sinks;
  float scale_log2;
  PromptList* list;
  int* status;
  unsigned long long wait_limit_ns;
  int inject;
  SharedPlan plan;  // kSharedPart, kOwnPart
};

// What 16 keys' scores are multiplied with (to the base-2 exponent), log2 of their V's
// scale, its inverse.
struct Factor {
  float k, log2v, inv;
  uint32_t far;  // of a tile's first: not 0 where V of 16 of its keys lies far below others'
};

// kSharedPart: the units are the plan's, 256 rows of a group over a run of its tokens; kOwnPart:
// as in kWhole those of sequences, but from their first own token on. What they leave is joined
// later.
enum Mode { kWhole, kSharedPart, kOwnPart };

// Where the unit's rows' parts are (kOwnPart: what the joining needs to find the shared ones); its
// first token; whose table row names which tokens.
template <int kMode>
struct UnitParts {};
template <>
struct UnitParts<kSharedPart> {
  long long first;
  int pieces, base;
};
template <>
struct UnitParts<kOwnPart> {
  long long first;
  int pieces, base, lead, leader;
};

template <int kMode>
struct Unit : UnitParts<kMode> {
  KvSequence q;
  int s, head, row0, rows;  // rows [row0, row0 + rows) of the sequence
  int sink_tiles, window_tile;
  int hidden_to;            // keys below this, from a.sinks on, are no row's to see
  int n[2];                 // tiles of each group; n[0] < 0: the list has ended
};

template <int HSP, int kMode>
struct Layout {
  static constexpr int kQBytes = kRows * HSP * 2;  // per group: [HSP / 64][128 rows][128 B]
  static constexpr int kKBytes = kTile * HSP * 2;  // per slot: [HSP / 64][64 rows][128 B]
  static constexpr int kVBytes = HSP * kTile * 2;  // per slot: [HSP rows][128 B]
  static constexpr int kRawBytes = kTile * HSP;    // K's or V's codes: [64 tokens][head_size]
  static constexpr int kRawSlots = HSP == 64 ? 4 : 3;  // of the ring of codes: what fits
  static constexpr int kQ = 0, kK = 2 * kQBytes, kV = kK + kSlots * kKBytes,
                       kRaw = kV + kSlots * kVBytes,
                       kFactors = kRaw + kRawSlots * 2 * kRawBytes,
                       kBars = kFactors + kFactorSlots * 4 * static_cast<int>(sizeof(Factor)),
                       kMisc = kBars + 8 * 40, kUnits = kMisc + 32,
                       kTotal = kUnits + kUnitSlots * static_cast<int>(sizeof(Unit<kMode>));
};

// The list's u-th unit: sequences by their longest unit, the longest first (up to
// kThreads of them; more keep their order), within a sequence the last rows, which see
// the most keys, first.
__device__ __forceinline__ long long units_of(const PromptArgs& a, int row_limit,
                                              const KvSequence& q) {
  const long long rows = static_cast<long long>(q.n) * a.group;
  return rows <= row_limit ? 0 : (rows + kUnitRows - 1) / kUnitRows * a.v.heads;
}

template <int kMode>
__device__ KvSequence sequence_of(const PromptArgs& a, int s) {
  if constexpr (kMode == kOwnPart) return a.plan.sequences[s].q;
  return kv_sequence(a.v, s);
}

template <int kMode>
__device__ Unit<kMode> decode_unit(const PromptArgs& a, int row_limit, const long long* prefix,
                            const int* order, int per, long long u) {
  int lo = 0, hi = kThreads;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (prefix[mid] <= u) lo = mid;
    else hi = mid;
  }
  Unit<kMode> r{};
  long long base = prefix[lo];
  for (r.s = per == 1 ? order[lo] : lo * per;; ++r.s) {
    r.q = sequence_of<kMode>(a, r.s);
    const long long n = units_of(a, row_limit, r.q);
    if (u < base + n) break;
    base += n;
    if (per == 1 || r.s + 1 >= a.v.sequences) return r;  // lengths changed under the call: no rows
  }
  const int all_rows = static_cast<int>(static_cast<long long>(r.q.n) * a.group);
  const int blocks = (all_rows + kUnitRows - 1) / kUnitRows;
  const int i = static_cast<int>(u - base);
  const int back = i / a.v.heads;
  r.head = i - back * a.v.heads;
  r.row0 = (blocks - 1 - back) * kUnitRows;
  r.rows = min(all_rows - r.row0, kUnitRows);
  r.sink_tiles = r.window_tile = r.hidden_to = 0;
  if (a.window > 0) {
    const int from = max(max(r.q.first + r.row0 / a.group, 0) - a.window + 1, 0);
    r.hidden_to = from;
    r.window_tile = from / kTile;
    r.sink_tiles = min((min(a.sinks, from) + kTile - 1) / kTile, r.window_tile);
  }
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const int rows = min(r.rows - g * kRows, kRows);
    r.n[g] = 0;
    if (rows <= 0) continue;
    const int last = r.q.first + (r.row0 + g * kRows + rows - 1) / a.group;  // position
    if constexpr (kMode == kOwnPart) {
      const SharedSequence p = a.plan.sequences[r.s];
      r.base = p.start;
      r.lead = p.lead;
      r.leader = p.leader;
      r.first = shared_part(p.part0, p.group_rows, p.pieces, r.head, p.row + r.row0);
      r.pieces = p.pieces;
      if (last >= p.start) r.n[g] = (last - p.start) / kTile + 1;
      continue;
    }
    if (last >= 0) r.n[g] = r.sink_tiles + max(last / kTile + 1 - r.window_tile, 0);
  }
  return r;
}

// Unit u of the plan: 256 rows of a group over a run of its tokens, all of which they see.
__device__ inline Unit<kSharedPart> decode_shared(const PromptArgs& a, int u) {
  const SharedGroup g = a.plan.groups[shared_group_of(a.plan, u)];
  const SharedUnit unit = shared_unit(g, a.v.heads, u);
  Unit<kSharedPart> r{};
  r.q = {g.row0, g.rows, g.tokens, 1 << 30};  // (behind every key)
  r.s = g.sequence;
  r.head = unit.head;
  r.row0 = unit.block * kUnitRows;
  r.rows = min(g.rows * a.group - r.row0, kUnitRows);
  r.sink_tiles = r.window_tile = r.hidden_to = 0;
  r.base = unit.tile0 * kTile;
  r.n[0] = unit.tiles;
  r.n[1] = r.rows > kRows ? unit.tiles : 0;
  r.first = shared_part(g.part0, g.rows * a.group, g.pieces, r.head, r.row0) + unit.piece;
  r.pieces = g.pieces;
  return r;
}

// (checking build) whether a unit's rows and tiles are its sequence's.
template <int kMode>
__device__ __forceinline__ bool unit_ok(const PromptArgs& a, const Unit<kMode>& u) {
  if constexpr (kMode != kWhole) {
    if (u.first < 0 || u.first + static_cast<long long>(u.rows - 1) * u.pieces >= a.plan.parts)
      return false;
  }
  const int tiles = (u.q.length + kTile - 1) / kTile;
  return u.s >= 0 && u.s < a.v.sequences && u.head >= 0 && u.head < a.v.heads && u.row0 >= 0 &&
         u.rows > 0 && u.rows <= kUnitRows &&
         u.row0 + u.rows <= static_cast<long long>(u.q.n) * a.group && u.q.row0 >= 0 &&
         u.q.row0 + u.q.n <= a.v.rows && u.n[0] <= tiles && u.n[1] >= 0 && u.n[1] <= tiles;
}

template <int kMode>
__device__ __forceinline__ int tile_token(const Unit<kMode>& u, int j) {
  if constexpr (kMode != kWhole) return u.base + j * kTile;
  return (j < u.sink_tiles ? j : j - u.sink_tiles + u.window_tile) * kTile;
}

__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// A place in a ring of kSize barriers and the parity of its phase.
template <uint32_t kSize>
struct Ring {
  uint32_t slot = 0, phase = 0;
  __device__ __forceinline__ void next() {
    if (++slot == kSize) slot = 0, phase ^= 1u;
  }
  __device__ __forceinline__ void skip(uint32_t n) {
    const uint32_t at = slot + n;
    slot = at % kSize;
    phase ^= at / kSize & 1u;
  }
};

// One lane of a converged warp: its MMAs' operands may stay in uniform registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// Instruction descriptor, kind::f16: A = B = fp16, D = f32, both K-major.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// D[tmem] (+)= A * B[smem]^T for 16-bit operands, A in shared memory (ss) or in TMEM
// (ts: 128 rows are lanes, two K-elements to a 32-bit column). Shared-memory
// descriptors as their low words and the high word that all of them share.
__device__ __forceinline__ void umma_f16_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo,
                                            uint32_t hi, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo,
                                            uint32_t hi, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 32 lanes x 8 or 16 consecutive 32-bit columns and a thread's registers, with their waits.
__device__ __forceinline__ void tmem_st_8cols(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n\t"
      "tcgen05.wait::st.sync.aligned;" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}
__device__ __forceinline__ void tmem_ld_16cols(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_8cols(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr)
      : "memory");
}
// Bulk copy global -> shared (16-byte multiples), completing on an mbarrier.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// mbar_wait_warp_inline with every lane looking for itself: nothing to hand round when the
// phase is complete.
__device__ __forceinline__ bool mbar_wait_lanes(uint32_t bar, uint32_t parity, const Watchdog& wd,
                                                int site) {
  bool ok = true;
  if (!mbar_test(bar, parity)) {
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t it = 1;; ++it) {
      if (mbar_test(bar, parity)) break;
      if ((it & 127u) == 0u) {
        if (*wd.abort_flag) {
          ok = false;
          break;
        }
        if (globaltimer_ns() - t0 > wd.limit_ns) {
          *wd.abort_flag = 1;
          if (atomicCAS(wd.status, 0, CSA_ERR_TIMEOUT) == 0) atomicExch(wd.status + 1, site);
          ok = false;
          break;
        }
      }
    }
  }
  return __all_sync(0xFFFFFFFFu, ok);
}

// Whether a phase has completed, for a whole warp, without waiting.
__device__ __forceinline__ bool mbar_poll_warp(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return __all_sync(0xFFFFFFFFu, done != 0);
}

// For a warp that polls: whether it may go on, `since` being when it began. False (recorded)
// when the CTA has given up or the time has run out.
__device__ __forceinline__ bool mbar_time_left(uint64_t since, const Watchdog& wd, int site) {
  int ok = 1;
  if (lane_id() == 0) {
    if (*wd.abort_flag) {
      ok = 0;
    } else if (globaltimer_ns() - since > wd.limit_ns) {
      *wd.abort_flag = 1;
      if (atomicCAS(wd.status, 0, CSA_ERR_TIMEOUT) == 0) atomicExch(wd.status + 1, site);
      ok = 0;
    }
  }
  return __shfl_sync(0xFFFFFFFFu, ok, 0) != 0;
}

// 16-byte global -> shared copy past L1; zeros where bytes is 0.
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}

__device__ __forceinline__ void st_shared16(uint32_t addr, const uint32_t* w) {
  st_shared_v4(addr, w[0], w[1], w[2], w[3]);
}

template <int HSP, int kFormat, bool kBf16, int kMode>
__global__ void __launch_bounds__(kThreads, 1)
    attend_prompt_sm103a_kernel(const PromptArgs a) {
  using L = Layout<HSP, kMode>;
  using Unit = Unit<kMode>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ long long s_prefix[kThreads + 1];
  __shared__ long long s_warp[kThreads / 32];
  __shared__ int s_order[kThreads], s_keys[kThreads];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t bars = base + L::kBars;
  auto k_full = [&](uint32_t s) { return bars + 8u * s; };
  auto v_full = [&](uint32_t s) { return bars + 8u * (36 + s); };
  auto empty = [&](uint32_t s) { return bars + 8u * (4 + s); };
  constexpr int kRawSlots = L::kRawSlots;
  auto raw_full = [&](uint32_t s) { return bars + 8u * (28 + s); };
  auto raw_empty = [&](uint32_t s) { return bars + 8u * (32 + s); };
  auto q_ready = [&](uint32_t g) { return bars + 8u * (8 + g); };
  auto s_full = [&](uint32_t g, uint32_t b) { return bars + 8u * (10 + 2 * g + b); };
  auto p_ready = [&](uint32_t g, uint32_t b) { return bars + 8u * (14 + 2 * g + b); };
  // (of a group's even and odd products: a parity tells only neighbouring phases apart,
  // and a waiter may be up to two products behind)
  auto pv_done = [&](uint32_t g, uint32_t b) { return bars + 8u * (18 + 2 * g + b); };
  auto u_full = [&](uint32_t s) { return bars + 8u * (22 + s); };
  auto u_empty = [&](uint32_t s) { return bars + 8u * (24 + s); };
  const uint32_t u_want = bars + 8u * 26;
  const uint32_t drain = bars + 8u * 27;
  const uint32_t tmem_slot = base + L::kMisc;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + L::kMisc + 4);
  Factor* factors = reinterpret_cast<Factor*>(gbase + L::kFactors);
  // Bit i: the 16 tokens i of a raw slot's K (bits 4..7: V) have codes there.
  volatile uint32_t* raw_pages = reinterpret_cast<volatile uint32_t*>(gbase + L::kMisc + 16);
  const Watchdog wd{a.wait_limit_ns, a.status, abort_flag};
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(k_full(s), kConvertWarps);
      mbar_init(v_full(s), kConvertWarps);
      mbar_init(empty(s), 2);  // one commit of each group's issuer
    }
    for (int s = 0; s < kRawSlots; ++s) {
      mbar_init(raw_full(s), 1);
      mbar_init(raw_empty(s), kConvertWarps);
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(q_ready(g), 4);
      for (int b = 0; b < 2; ++b) {
        mbar_init(pv_done(g, b), 1);
        mbar_init(s_full(g, b), 1);
        mbar_init(p_ready(g, b), 4);
      }
    }
    mbar_init(drain, 2);
    mbar_init(u_want, 1);
    for (int s = 0; s < kUnitSlots; ++s) {
      mbar_init(u_full(s), 1);
      mbar_init(u_empty(s), kThreads / 32 - 1);  // every warp but the list's
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
    tc_fence_before_sync();
  }
  grid_dependency_wait();
  if constexpr (kMode == kSharedPart) grid_dependents_launch();  // (the own parts, beside this)

  // The work list: thread i counts the units of sequences [i per, (i + 1) per).
  const int S = a.v.sequences, row_limit = kMode == kSharedPart ? 0 : a.list->row_limit;
  const int per = (S + kThreads - 1) / kThreads;
  if constexpr (kMode != kSharedPart) {
    long long mine = 0;
    if (per == 1) {
      const int i = threadIdx.x;
      int key = -1;
      if (i < S) {
        const KvSequence q = sequence_of<kMode>(a, i);
        if (units_of(a, row_limit, q) > 0)
          key = a.window > 0 && a.window < q.length - q.n ? a.window + q.n : q.length;
      }
      s_keys[i] = key;
      __syncthreads();
      if (i < S) {
        int rank = 0;
        for (int o = 0; o < S; ++o) rank += s_keys[o] > key || (s_keys[o] == key && o < i);
        s_order[rank] = i;
      }
      __syncthreads();
      if (i < S) mine = units_of(a, row_limit, sequence_of<kMode>(a, s_order[i]));
    } else {
      const long long from = static_cast<long long>(threadIdx.x) * per;
      for (long long s = from; s < min(static_cast<long long>(S), from + per); ++s)
        mine += units_of(a, row_limit, sequence_of<kMode>(a, static_cast<int>(s)));
    }
    long long sum = mine;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const long long up = __shfl_up_sync(0xFFFFFFFFu, sum, d);
      if (lane >= d) sum += up;
    }
    if (lane == 31) s_warp[warp] = sum;
    __syncthreads();
    long long before = 0;
    for (int w = 0; w < warp; ++w) before += s_warp[w];
    s_prefix[threadIdx.x + 1] = before + sum;
    if (threadIdx.x == 0) s_prefix[0] = 0;
  }
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, ld_shared_b32(tmem_slot), 0);
  const long long total =
      kMode != kSharedPart ? s_prefix[kThreads]
      : static_cast<int>(blockIdx.x) < a.plan.head->shared_sms ? a.plan.head->units : 0;
  // The k-th unit that this CTA works on, for a whole warp; false: a wait ran out.
  auto take_unit = [&](uint32_t k, Unit& u) {
    const uint32_t slot = k % kUnitSlots;
    if (!mbar_wait_lanes(u_full(slot), (k / kUnitSlots) & 1u, wd, kSiteSched)) return false;
    u = reinterpret_cast<const Unit*>(gbase + L::kUnits)[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(u_empty(slot));
    return CSA_CHECK(u.n[0] < 0 || unit_ok(a, u), wd, kCheckTile);
  };
  const int D = a.v.head_size;

  if (warp < kSoftmaxWarps) {
    // ------------------------------------------------------------ softmax --
    const uint32_t g = warp >> 2;
    const int r = threadIdx.x & 127;                       // row of the group
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // TMEM lane field
    const uint32_t o_tmem = tmem + lanes + 2 * kRows + g * HSP;
    const uint32_t q_smem = base + L::kQ + g * L::kQBytes;
    // Rows go between HBM and shared memory a warp's 32 at a time: kLanes lanes of 16
    // bytes to a row.
    constexpr int kLanes = HSP / 8, kRowsAtOnce = 32 / kLanes;
    const int piece = lane % kLanes;  // this lane's 8 elements of such a row
    uint32_t products = 0;            // of the group, before this unit
    uint32_t tiles = 0;               // of the CTA, before this unit (the factors' slots)
    bool ok = true;
    // A unit as this thread's row sees it.
    struct Row {
      int token, head, pos;  // row of q and out, head; -1: no such row
      bool live;
    };
    Unit u;
    Row row;
    // Takes the k-th unit and copies its Q to shared memory; false: no more units.
    auto next_unit = [&](uint32_t k) {
      if (!take_unit(k, u) || u.n[0] < 0) return false;
      const int rr = u.row0 + static_cast<int>(g) * kRows + r;
      const int j_tok = rr / a.group;
      row.live = static_cast<int>(g) * kRows + r < u.rows;
      row.token = u.q.row0 + j_tok;
      row.head = u.head * a.group + (rr - j_tok * a.group);
      row.pos = row.live ? u.q.first + j_tok : -1;
      if ((g == 0 ? u.n[0] : u.n[1]) > 0) {
#pragma unroll 4
        for (int i = 0; i < kLanes; ++i) {
          const int from = i * kRowsAtOnce + lane / kLanes;  // row of the warp
          const int token = __shfl_sync(0xFFFFFFFFu, row.live ? row.token : -1, from);
          const int head = __shfl_sync(0xFFFFFFFFu, row.head, from);
          const bool in = token >= 0 && piece * 8 < D;
          const uint32_t sr = static_cast<uint32_t>((warp & 3) * 32 + from);
          cp_async_16(q_smem + (piece >> 3) * (kRows * 128) + sr * 128 +
                          (((piece & 7) ^ (sr & 7)) << 4),
                      static_cast<const uint16_t*>(a.q) +
                          (in ? token * a.q_token + head * a.q_head + piece * 8 : 0),
                      in ? 16u : 0u);
        }
        cp_async_commit();
        cp_async_wait<0>();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_ready(g));
      }
      return true;
    };
    bool more = next_unit(0);
    for (uint32_t k = 1; more; ++k) {
      const int n = g == 0 ? u.n[0] : u.n[1];
      const bool live = row.live;
      const int pos = row.pos;
      float l = 0.0f, m = kNothing;
      const int pos_low = __reduce_min_sync(0xFFFFFFFFu, live ? pos : 0x7FFFFFFF);
      const int pos_high = __reduce_max_sync(0xFFFFFFFFu, pos);
      for (int step = 0; ok && step < n; ++step) {
        const uint32_t product = products + step, buffer = product & 1u;
        const uint32_t s_tmem = tmem + lanes + g * kRows + buffer * kTile;
        const int tb = tile_token(u, step);
        if (!mbar_wait_lanes(s_full(g, buffer), (product >> 1) & 1u, wd,
                                   kSiteEpilogueFull)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const Factor* fac = factors + ((tiles + step) % kFactorSlots) * 4;
        const bool edge = kMode != kSharedPart &&
                          !(tb + kTile - 1 <= pos_low &&
                            (a.window == 0 || pos_high - tb < a.window || tb + kTile - 1 < a.sinks));
        // columns 0 .. last are at or before this row; from first_window on, or below
        // sink_cols, they are in its window or sinks
        const int last = pos - tb;
        const int first_window = a.window ? last - a.window + 1 : -kTile;
        const int sink_cols = a.window ? a.sinks - tb : 0;
        const bool fresh = m == kNothing;  // nothing seen yet: the first value sets m
        const float less = fresh ? 0.0f : m;
        uint32_t x[kTile];
        tmem_ld_64cols(s_tmem, x);
#pragma unroll
        for (int i = 0; i < kTile / 16; ++i) {
          const Factor c = fac[i];
          const float add = c.log2v - less;
          const uint64_t fk2 = pack_f32x2(c.k, c.k), add2 = pack_f32x2(add, add);
#pragma unroll
          for (int e = 16 * i; e < 16 * i + 16; e += 2) {
            float y0, y1;
            fma_f32x2(y0, y1, __uint_as_float(x[e]), __uint_as_float(x[e + 1]), fk2, add2);
            x[e] = __float_as_uint(y0);
            x[e + 1] = __float_as_uint(y1);
          }
        }
        if (__builtin_expect(edge, 0)) {
#pragma unroll
          for (int i = 0; i < kTile; ++i)
            if (i > last || (i < first_window && i >= sink_cols))
              x[i] = __float_as_uint(-INFINITY);
        }
        float tops[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) tops[i] = fmaxf(__uint_as_float(x[i]), __uint_as_float(x[i + 4]));
#pragma unroll
        for (int i = 8; i < kTile; i += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            tops[e] = fmaxf(fmaxf(tops[e], __uint_as_float(x[i + e])), __uint_as_float(x[i + 4 + e]));
        const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
        const bool far = fac[0].far != 0;  // (the CTA's)
        const bool raise = top > (fresh ? -INFINITY : kRaise);
        if (__builtin_expect(__any_sync(0xFFFFFFFFu, raise || far), 0)) {
          if (__any_sync(0xFFFFFFFFu, raise)) {
            // (rare) a new maximum: what was computed with the old one, O and l, is rescaled
            const float up = fmaxf(top - kHeadroom, fresh ? kNothing : 0.0f);
            const float half = fresh ? 1.0f : ex2_approx(-0.5f * up), corr = half * half;
            m = less + up;
            l = l * half * half;
            const float off = fresh && top == -INFINITY ? 0.0f : up;
#pragma unroll
            for (int i = 0; i < kTile; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) - off);
            if (step > 0) {
              // O is the product issued last's until that is complete (the one before it
              // is: this tile's scores were issued later)
              const uint32_t before = product - 1;
              if (!mbar_wait_lanes(pv_done(g, before & 1u), (before >> 1) & 1u, wd,
                                   kSiteEpilogueFull))
                ok = false;
              tc_fence_after_sync();
#pragma unroll 1
              for (int d = 0; d < HSP; d += 8) {
                uint32_t y[8];
                tmem_ld_8cols(o_tmem + d, y);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  y[i] = __float_as_uint(__uint_as_float(y[i]) * corr);
                tmem_st_8cols(o_tmem + d, y);
              }
            }
          }
          if (far) {
            // V far below that of others: weights that come out as 0 are added to the sum
            // without V's scale, from the scores again
#pragma unroll 1
            for (int e = 0; e < kTile; e += 8) {
              uint32_t y[8];
              tmem_ld_8cols(s_tmem + e, y);
              const Factor c = fac[e / 16];
              const float add = c.log2v - m;
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float z = fmaf(__uint_as_float(y[i]), c.k, add);
                if (z < -126.0f && z != -INFINITY && e + i <= last &&
                    (e + i >= first_window || e + i < sink_cols))
                  l += ex2_approx(z - c.log2v);
              }
            }
          }
        }
        // Weights, as fp16 over S (whose scores have all been read)
#pragma unroll
        for (int i = 0; i < kTile / 16; ++i) {
          uint64_t sum = 0;
#pragma unroll
          for (int e = 16 * i; e < 16 * i + 16; e += 2) {
            const float y0 = ex2_approx(__uint_as_float(x[e]));
            const float y1 = ex2_approx(__uint_as_float(x[e + 1]));
            sum = add_f32x2(sum, pack_f32x2(y0, y1));
            x[e / 2] = half2_of(y0, y1);
          }
          float s0, s1;
          unpack_f32x2(sum, s0, s1);
          l = fmaf(s0 + s1, fac[i].inv, l);
        }
        uint32_t p[kTile / 2];
#pragma unroll
        for (int i = 0; i < kTile / 2; ++i) p[i] = x[i];
        tmem_st_32cols(s_tmem, p);
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_ready(g, buffer));
      }
      if (!ok) break;
      products += n;
      tiles += max(u.n[0], u.n[1]);
      // The next unit's Q takes the place of this one's, whose last scores have been
      // seen, so that its first scores are computed while O is written.
      uint16_t* to = static_cast<uint16_t*>(a.out) +
                     (live ? row.token * a.out_token + row.head * a.out_head : 0);
      [[maybe_unused]] long long part = 0, own = 0;
      [[maybe_unused]] int shared = 0;
      if constexpr (kMode != kWhole) {
        part = u.first + (static_cast<long long>(g) * kRows + r) * u.pieces;
        own = static_cast<long long>(row.token) * (a.v.heads * a.group) + row.head;
        shared = u.pieces;
      }
      more = next_unit(k);
      if (n > 0) {
        const uint32_t final = products - 1;
        if (!mbar_wait_lanes(pv_done(g, final & 1u), (final >> 1) & 1u, wd,
                                   kSiteEpilogueFull))
          break;
        tc_fence_after_sync();
      }
      if constexpr (kMode != kWhole) {
        constexpr bool kOwn = kMode == kOwnPart;
        if (live && (kOwn || n > 0)) {
          if (kOwn) {
            a.plan.own_ml[own] = make_float2(m, l);
            a.plan.own[own] = OwnRow{part, shared, 0, 0, 0};
            a.plan.own_there[own] = 1;
          } else {
            a.plan.ml[part] = make_float2(m, l);
          }
        }
        __syncwarp();
        float* to_o = kOwn ? a.plan.own_o + own * HSP : a.plan.o + part * HSP;
#pragma unroll 1
        for (int d0 = 0; (kOwn || n > 0) && d0 < HSP; d0 += 64) {
          uint32_t x[64];
          if (n > 0) {
            tmem_ld_64cols(o_tmem + d0, x);
          } else {
#pragma unroll
            for (int i = 0; i < 64; ++i) x[i] = 0u;
          }
          if (live) {
#pragma unroll
            for (int d = 0; d < 64; d += 4)
              *reinterpret_cast<uint4*>(to_o + d0 + d) =
                  make_uint4(x[d], x[d + 1], x[d + 2], x[d + 3]);
          }
          __syncwarp();
        }
        tc_fence_before_sync();
        continue;
      }
      const float inv_l = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll 1
      for (int d0 = 0; d0 < D; d0 += 64) {
        uint32_t x[64];
        if (n > 0) {
          tmem_ld_64cols(o_tmem + d0, x);
        } else {
#pragma unroll
          for (int i = 0; i < 64; ++i) x[i] = 0u;
        }
#pragma unroll
        for (int d = 0; d < 64; d += 8) {
          uint32_t y[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float v0 = __uint_as_float(x[d + 2 * i]) * inv_l;
            float v1 = __uint_as_float(x[d + 2 * i + 1]) * inv_l;
            if (l == 0.0f) v0 = v1 = 0.0f;
            if (kBf16) {
              const __nv_bfloat162 b = __floats2bfloat162_rn(v0, v1);
              y[i] = *reinterpret_cast<const uint32_t*>(&b);
            } else {
              y[i] = half2_of(v0, v1);
            }
          }
          if (live && d0 + d < D)
            *reinterpret_cast<uint4*>(to + d0 + d) = make_uint4(y[0], y[1], y[2], y[3]);
        }
      }
      tc_fence_before_sync();  // O may be overwritten after the next unit's p_ready
    }
  } else if (warp < kMmaWarp) {
    // --------------------------------------------------------- conversion --
    const int w = warp - kSoftmaxWarps;
    constexpr int kLaneVBytes = HSP / 16;  // V elements a lane transposes, for 8 tokens
    constexpr int kChunks = HSP / 16, kKRows = 32 / kChunks;  // 16-byte chunks of a row
    // K: a warp's 16 tokens, kKRows rows at once. V: tokens 8 oct .., elements vd ..;
    // four octets and eight runs of elements a warp, so that neither the loads' nor the
    // stores' bank conflicts are more than four- and twofold.
    const int chunk = lane % kChunks, k_row = 16 * w + lane / kChunks;
    const int oct = 4 * (w & 1) + (lane & 3), vt = 8 * oct;
    const int vd = (w >> 1) * (HSP / 2) + (lane >> 2) * kLaneVBytes;
    Ring<kSlots> to_slot;
    Ring<kRawSlots> from_slot;
    bool ok = true;
    for (uint32_t k = 0; ok; ++k) {
      Unit u;
      if (!take_unit(k, u) || u.n[0] < 0) break;
      const int n = max(u.n[0], u.n[1]);
      // slot j: K of tile j + 1, V of tile j
      if (n > 0)
        for (int j = -1; j < n; ++j, to_slot.next(), from_slot.next()) {
          const uint32_t slot = to_slot.slot, rs = from_slot.slot;
          if (!CSA_CHECK(slot < kSlots && rs < kRawSlots, wd, kCheckRing)) {
            ok = false;
            break;
          }
          if (!mbar_wait_lanes(raw_full(rs), from_slot.phase, wd, kSiteLoaderEmpty) ||
              !mbar_wait_lanes(empty(slot), to_slot.phase ^ 1u, wd, kSiteLoaderEmpty)) {
            ok = false;
            break;
          }
          const uint8_t* codes = gbase + L::kRaw + rs * 2 * L::kRawBytes;
          const uint32_t here = raw_pages[rs];
          uint32_t vx[8][kLaneVBytes / 4];
          if (j >= 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint8_t* from = codes + L::kRawBytes + (vt + i) * D + vd;
              if constexpr (kLaneVBytes == 8) {
                const uint2 x = *reinterpret_cast<const uint2*>(from);
                vx[i][0] = x.x;
                vx[i][1] = x.y;
              } else {
                vx[i][0] = *reinterpret_cast<const uint32_t*>(from);
              }
            }
          }
          if (j + 1 < n) {
            const uint32_t ks = base + L::kK + slot * L::kKBytes;
            const bool in = (here >> w & 1u) != 0 && chunk * 16 < D;
            uint4 xs[16 / kKRows];  // all of a lane's loads before the first store
#pragma unroll
            for (int i = 0; i < 16 / kKRows; ++i) {
              xs[i] = make_uint4(0, 0, 0, 0);
              if (in)
                xs[i] = *reinterpret_cast<const uint4*>(codes + (k_row + i * kKRows) * D +
                                                        chunk * 16);
            }
#pragma unroll
            for (int i = 0; i < 16 / kKRows; ++i) {
              const uint32_t row = k_row + i * kKRows;
              const uint32_t c[4] = {xs[i].x, xs[i].y, xs[i].z, xs[i].w};
              uint32_t y[8];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if constexpr (kBf16) codes4_to_bf162x2<kFormat>(c[e], y[2 * e], y[2 * e + 1]);
                else codes4_to_half2x2<kFormat>(c[e], y[2 * e], y[2 * e + 1]);
              }
              const uint32_t at = ks + (chunk >> 2) * (kTile * 128) + row * 128;
              const uint32_t unit = 2 * (chunk & 3);
              st_shared16(at + ((unit ^ (row & 7)) << 4), y);
              st_shared16(at + (((unit + 1) ^ (row & 7)) << 4), y + 4);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(k_full(slot));
          if (j >= 0) {
            // (what is loaded past the sequence's end, where no row's window reaches, or past
            // head_size, is whatever the slot held, and zeroed)
            const int from = tile_token(u, j) + vt;  // the octet's first token
            const int have =
                (here >> (4 + (oct >> 1)) & 1u) != 0 && vd < D ? u.q.length - from : 0;
            if (__builtin_expect(have < 8 || from < u.hidden_to, 0)) {
#pragma unroll
              for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int c = 0; c < kLaneVBytes / 4; ++c)
                  if (i >= have || (from + i < u.hidden_to && from + i >= a.sinks)) vx[i][c] = 0;
            }
            const uint32_t vs = base + L::kV + slot * L::kVBytes;
#pragma unroll
            for (int c = 0; c < kLaneVBytes / 4; ++c) {
              // eight tokens of four elements: pairs of tokens, then rows of V^T
              uint32_t y[4][4];
#pragma unroll
              for (int p = 0; p < 4; ++p) {
                uint32_t x0 = vx[2 * p][c], x1 = vx[2 * p + 1][c];
                if (kFormat == CSA_KV_INT8) {
                  x0 ^= 0x80808080u;
                  x1 ^= 0x80808080u;
                }
                const uint32_t lo = byte_perm(x0, x1, 0x5140), hi = byte_perm(x0, x1, 0x7362);
                if (kFormat == CSA_KV_INT8) {
                  y[0][p] = flipped_pair_to_half2<0x4140>(lo);
                  y[1][p] = flipped_pair_to_half2<0x4342>(lo);
                  y[2][p] = flipped_pair_to_half2<0x4140>(hi);
                  y[3][p] = flipped_pair_to_half2<0x4342>(hi);
                } else {
                  y[0][p] = e4m3x2_to_half2(lo & 0xFFFFu);
                  y[1][p] = e4m3x2_to_half2(lo >> 16);
                  y[2][p] = e4m3x2_to_half2(hi & 0xFFFFu);
                  y[3][p] = e4m3x2_to_half2(hi >> 16);
                }
              }
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t row = vd + 4 * c + e;
                st_shared16(vs + row * 128 + ((oct ^ (row & 7)) << 4), y[e]);
              }
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(v_full(slot));
            mbar_arrive(raw_empty(rs));
          }
        }
    }
  } else if (warp == kCopyWarp) {
    // ------------------------------------------------------------- copies --
    uint32_t it = 0, tiles = 0;
    bool ok = true, injected = false;
    const int P = a.v.page_tokens, page_mask = P - 1;
    const long long page_bytes = static_cast<long long>(P) * D;
    // Lanes that copy: the first of each page's groups in the tile.
    const int groups = min(P, kTile) / 16;  // of a page in a tile
    const bool copies = lane < 4 && lane % groups == 0;
    const uint32_t copy_mask = __ballot_sync(0xFFFFFFFFu, copies);
    const uint32_t copy_bytes = static_cast<uint32_t>(groups) * 16u * D;
    // The table's entries for a tile's four groups of 16 tokens, in lanes 0..3; read a
    // step before they are checked, so that nothing waits for them. (None past the length,
    // nor where no row sees any of a page's tokens in the tile.)
    struct Entry {
      int page;
      bool there;
    };
    const int before = lane % groups * 16, after = groups * 16 - before;
    auto row_of = [&](const Unit& u, int tok) {
      if constexpr (kMode == kOwnPart) return tok < u.lead ? u.leader : u.s;
      return u.s;
    };
    auto entries_of = [&](const Unit& u, int j) {
      const int tok = tile_token(u, j) + 16 * lane;
      Entry e{-1, lane < 4 && tok < u.q.length &&
                      (tok + after > u.hidden_to || tok - before < a.sinks)};
      if (e.there)
        e.page = __ldg(a.v.table + (static_cast<long long>(row_of(u, tok)) * a.v.table_width +
                                    (tok >> a.v.page_shift)));
      return e;
    };
    auto pages_of = [&](const Entry& e) {  // -1: none there
      if (e.there && (e.page < 0 || e.page >= a.v.pages)) {
        report_index(a.v.status, kIndexPage);
        return -1;
      }
      return e.page;
    };
    auto part_of = [&](const Unit& u, int j, int page, int which) {  // of a page: this lane's
      return a.v.codes[which] + (static_cast<long long>(page) * a.v.heads + u.head) * page_bytes +
             ((tile_token(u, j) + 16 * lane) & page_mask) * D;
    };
    for (uint32_t k = 0; ok; ++k) {
      Unit u;
      if (k == 0 && lane == 0) mbar_arrive(u_want);
      if (!take_unit(k, u) || u.n[0] < 0) break;
      const int n = max(u.n[0], u.n[1]);
      const int ask = max(n - kAskAhead, -1);
      if (n == 0) {
        if (lane == 0) mbar_arrive(u_want);
        continue;
      }
      // A pipeline over the tiles, as each stage waits for the one before: the table's
      // entry (read), the page (checked), its scales (read), the copy.
      int page_v = -1;                              // of tile j
      const Entry none{-1, false};
      int page = pages_of(entries_of(u, 0));        // of tile j + 1
      int page2 = n > 1 ? pages_of(entries_of(u, 1)) : -1;
      Entry entry = n > 2 ? entries_of(u, 2) : none;  // of tile j + 3
      struct Scales {
        float k, v;
      };
      auto scales_of = [&](int pg) {
        Scales f{1.0f, 1.0f};
        if (pg >= 0) {
          const long long unit = static_cast<long long>(pg) * a.v.heads + u.head;
          f.k = __ldg(a.v.scale[0] + unit);
          f.v = __ldg(a.v.scale[1] + unit);
        }
        return f;
      };
      Scales f = scales_of(page), f2 = scales_of(page2);
      float vmost = 0.0f;  // the largest scale of V so far
      for (int j = -1; j < n; ++j, ++it) {
        const uint32_t rs = it % kRawSlots;
        // Everything is worked out before the slot is free.
        const bool k_here = j + 1 < n && page >= 0, v_here = page_v >= 0;
        if (!__all_sync(0xFFFFFFFFu,
                        CSA_CHECK(rs < kRawSlots && page < a.v.pages && page_v < a.v.pages &&
                                      (!copies || (tile_token(u, j + 1) + 16 * lane) % P +
                                                          16 * groups <= P),
                                  wd, kCheckRing))) {
          ok = false;
          break;
        }
        const uint32_t here = __ballot_sync(0xFFFFFFFFu, k_here && lane < 4) |
                              __ballot_sync(0xFFFFFFFFu, v_here && lane < 4) << 4;
        const uint32_t bytes = copy_bytes * (__popc(here & copy_mask) + __popc(here >> 4 & copy_mask));
        const uint8_t* k_from = part_of(u, j + 1, page, 0);
        const uint8_t* v_from = part_of(u, j, page_v, 1);
        const uint32_t to = base + L::kRaw + rs * 2 * L::kRawBytes + 16 * lane * D;
        // -inf masks 16 tokens of no page. A block of scale 0 holds zeros, at any scale (and
        // its V is not copied).
        const float scale_v = fmaxf(f.v, kScaleFloor);
        vmost = fmaxf(vmost, __uint_as_float(__reduce_max_sync(
                                 0xFFFFFFFFu, page >= 0 ? __float_as_uint(scale_v) : 0u)));
        const uint32_t fars = __ballot_sync(0xFFFFFFFFu, page >= 0 && scale_v < vmost * kFar);
        if (j + 1 < n && lane < 4)
          factors[((tiles + j + 1) % kFactorSlots) * 4 + lane] =
              Factor{a.scale_log2 * f.k, page >= 0 ? __log2f(scale_v) : -INFINITY,
                     __fdividef(1.0f, scale_v), fars};
        if (j == ask && lane == 0) mbar_arrive(u_want);
        if (!mbar_wait_lanes(raw_empty(rs), ((it / kRawSlots) & 1u) ^ 1u, wd,
                                   kSiteProducerEmpty)) {
          ok = false;
          break;
        }
        if (a.inject && !injected) {
          injected = true;  // withhold the CTA's first slot: the conversion's wait runs out
        } else {
          if (lane == 0) {
            raw_pages[rs] = here;
            mbar_arrive_expect_tx(raw_full(rs), bytes);
          }
          __syncwarp();
          if (k_here && copies) bulk_load(to, k_from, copy_bytes, raw_full(rs));
          if (v_here && copies) bulk_load(to + L::kRawBytes, v_from, copy_bytes, raw_full(rs));
        }
        page_v = j + 1 < n && f.v != 0.0f ? page : -1;
        page = page2;
        f = f2;
        page2 = j + 3 < n ? pages_of(entry) : -1;
        f2 = scales_of(page2);
        entry = j + 4 < n ? entries_of(u, j + 4) : none;
      }
      tiles += n;
    }
    // Copies in flight (after a wait that ran out: otherwise the conversion has seen
    // them all) land before shared memory goes away.
    if (lane == 0 && *abort_flag) {
      for (uint32_t i = it > kRawSlots ? it - kRawSlots : (injected ? 1u : 0u); i < it; ++i) {
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_test(raw_full(i % kRawSlots), (i / kRawSlots) & 1u) &&
               globaltimer_ns() - t0 < a.wait_limit_ns) {
        }
      }
    }
    __syncwarp();
  } else if (warp == kListWarp) {
    // --------------------------------------------------------------- list --
    if (lane == 0) {
      for (uint32_t k = 0;; ++k) {
        const uint32_t slot = k % kUnitSlots;
        if (!mbar_wait(u_want, k & 1u, wd, kSiteSched)) break;
        const long long at =
            kMode == kSharedPart && total == 0 ? 0 : atomicAdd(&a.list->taken, 1u);
        Unit u;
        if (at >= total) u.n[0] = -1;
        else if constexpr (kMode == kSharedPart) u = decode_shared(a, static_cast<int>(at));
        else u = decode_unit<kMode>(a, row_limit, s_prefix, s_order, per, at);
        if (!mbar_wait(u_empty(slot), ((k / kUnitSlots) & 1u) ^ 1u, wd, kSiteSched)) break;
        reinterpret_cast<Unit*>(gbase + L::kUnits)[slot] = u;
        mbar_arrive(u_full(slot));
        if (at >= total) break;
      }
    }
    __syncwarp();
  } else {
    // -------------------------------------------------------- MMA issuers --
    const uint32_t g = warp - kMmaWarp;
    constexpr uint32_t kIdescS = kBf16 ? idesc_bf16_f32(kRows, kTile) : idesc_f16_f32(kRows, kTile);
    constexpr uint32_t kIdescO = idesc_f16_f32(kRows, HSP);
    // Descriptors' low words (the start address in units of 16 bytes); moving along a
    // tile adds to them.
    const uint64_t desc = umma_desc_k_sw128(base);
    const uint32_t desc_hi = static_cast<uint32_t>(desc >> 32), lo = static_cast<uint32_t>(desc);
    const uint32_t s_tmem = tmem + g * kRows, o_tmem = tmem + 2 * kRows + g * HSP;
    const uint32_t qd = lo + ((L::kQ + g * L::kQBytes) >> 4);
    uint32_t products = 0, q_phase = 0;
    Ring<kSlots> unit_slot;
    bool ok = true;
    for (uint32_t k = 0; ok; ++k) {
      Unit u;
      if (!take_unit(k, u) || u.n[0] < 0) break;
      // (shuffled so that the compiler knows them to be the warp's: what is computed
      // from them then stays in uniform registers, which the MMAs' operands are)
      const int n = __shfl_sync(0xFFFFFFFFu, g == 0 ? u.n[0] : u.n[1], 0);
      const int n_all = __shfl_sync(0xFFFFFFFFu, max(u.n[0], u.n[1]), 0);
      if (n_all == 0) continue;
      if (n > 0) {
        if (!mbar_wait_lanes(q_ready(g), q_phase, wd, kSiteMmaFull)) break;
        q_phase ^= 1u;
      }
      // Scores of tile `next_s` and output of tile `next_o`, whichever has its operands
      // first; S(i) takes the buffer that O(i - 2) has read. Slot e of the unit (K of tile e,
      // V of tile e - 1) goes back when both are issued.
      int next_s = 0, next_o = 0, given = 0;
      Ring<kSlots> at_s = unit_slot, at_o = unit_slot, at_given = unit_slot;
      at_o.next();
      uint64_t since = 0;
      uint32_t spins = 0;
      while (next_o < n) {
        bool did = false;
        if (next_o < next_s) {
          const uint32_t p = products + next_o, slot = at_o.slot;
          if (!CSA_CHECK(slot < kSlots && o_tmem - tmem + HSP <= kTmemCols, wd, kCheckTmem)) {
            ok = false;
            break;
          }
          if (mbar_poll_warp(p_ready(g, p & 1u), (p >> 1) & 1u) &&
              mbar_poll_warp(v_full(slot), at_o.phase)) {
            tc_fence_after_sync();
            const uint32_t vd = lo + ((L::kV + slot * L::kVBytes) >> 4);
            if (elect_one()) {
#pragma unroll
              for (int s = 0; s < kTile / 16; ++s)
                umma_f16_ts(o_tmem, s_tmem + (p & 1u) * kTile + 8 * s, vd + 2 * s, desc_hi, kIdescO,
                            next_o > 0 || s > 0);
              umma_commit(pv_done(g, p & 1u));
            }
            __syncwarp();
            ++next_o;
            at_o.next();
            did = true;
          }
        }
        if (next_s < n && next_s <= next_o + 1) {
          const uint32_t slot = at_s.slot;
          if (!CSA_CHECK(slot < kSlots && s_tmem - tmem + 2 * kTile <= kTmemCols, wd,
                         kCheckTmem)) {
            ok = false;
            break;
          }
          if (mbar_poll_warp(k_full(slot), at_s.phase)) {
            tc_fence_after_sync();
            const uint32_t buffer = (products + next_s) & 1u;
            const uint32_t kd = lo + ((L::kK + slot * L::kKBytes) >> 4);
            if (elect_one()) {
#pragma unroll
              for (int s = 0; s < HSP / 16; ++s)
                umma_f16_ss(s_tmem + buffer * kTile,
                            qd + (((s >> 2) * (kRows * 128) + (s & 3) * 32) >> 4),
                            kd + (((s >> 2) * (kTile * 128) + (s & 3) * 32) >> 4), desc_hi,
                            kIdescS, s > 0);
              umma_commit(s_full(g, buffer));
            }
            __syncwarp();
            ++next_s;
            at_s.next();
            did = true;
          }
        }
        if (did) {
          while (given <= next_o && next_s >= min(given + 1, n)) {
            if (elect_one()) umma_commit(empty(at_given.slot));
            __syncwarp();
            ++given;
            at_given.next();
          }
          spins = 0;
        } else if ((++spins & 127u) == 0) {
          if (spins == 128) since = globaltimer_ns();
          if (!mbar_time_left(since, wd, kSiteMmaFull)) {
            ok = false;
            break;
          }
        }
      }
      // slots of tiles past this group's own are only given back
      for (; ok && given <= n_all; ++given, at_given.next()) {
        ok = mbar_wait_lanes(k_full(at_given.slot), at_given.phase, wd, kSiteMmaFull) &&
             mbar_wait_lanes(v_full(at_given.slot), at_given.phase, wd, kSiteMmaFull);
        if (!ok) break;
        if (elect_one()) umma_commit(empty(at_given.slot));
        __syncwarp();
      }
      unit_slot.skip(static_cast<uint32_t>(n_all) + 1u);
      products += n;
    }
    // Every MMA must be complete before TMEM and shared memory go away.
    if (elect_one()) {
      umma_commit(drain);
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_test(drain, 0) && globaltimer_ns() - t0 < a.wait_limit_ns) {
      }
    }
    __syncwarp();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

template <int HSP, int kFormat, bool kBf16, int kMode>
cudaError_t launch_prompt(const PromptArgs& a, const DeviceInfo& dev, cudaStream_t stream, int& rc,
                          std::string& err) {
  const auto kernel = attend_prompt_sm103a_kernel<HSP, kFormat, kBf16, kMode>;
  const int smem = Layout<HSP, kMode>::kTotal + 1024;
  rc = set_max_dynamic_smem(reinterpret_cast<const void*>(kernel), smem, dev.device, err);
  if (rc != CSA_OK) return cudaSuccess;
  return launch_programmatic(kernel, static_cast<unsigned>(dev.sm_count), kThreads, smem, stream, a);
}

template <int HSP, int kMode>
cudaError_t launch_prompt(const PromptArgs& a, int format, const DeviceInfo& dev,
                          cudaStream_t stream, int& rc, std::string& err) {
  if (format == CSA_KV_INT8)
    return a.half ? launch_prompt<HSP, CSA_KV_INT8, false, kMode>(a, dev, stream, rc, err)
                  : launch_prompt<HSP, CSA_KV_INT8, true, kMode>(a, dev, stream, rc, err);
  return a.half ? launch_prompt<HSP, CSA_KV_E4M3, false, kMode>(a, dev, stream, rc, err)
                : launch_prompt<HSP, CSA_KV_E4M3, true, kMode>(a, dev, stream, rc, err);
}

// What both callers' arguments have in common, and the launch.
PromptArgs prompt_args(const csa_kv_cache& cache, const csa_kv_batch& batch,
                       const AttendCall& call, PromptList* list, const DeviceInfo& dev) {
  PromptArgs a{};
  a.v = kv_view(cache, batch, dev);
  a.q = call.q;
  a.out = call.out;
  a.q_token = call.q_token;
  a.q_head = call.q_head;
  a.out_token = call.out_token;
  a.out_head = call.out_head;
  a.half = call.dtype == CSA_F16;
  a.group = call.q_heads / cache.heads;
  a.window = call.window;
  a.sinks = call.window > 0 ? call.sinks : 0;
  a.scale_log2 = static_cast<float>(static_cast<double>(call.scale) * 1.4426950408889634);
  a.status = dev.status_word;
  a.wait_limit_ns = wait_limit_ns();
  a.inject = take_inject() ? 1 : 0;
  a.list = list;
  return a;
}

template <int kMode>
int launch_prompt(const PromptArgs& a, const csa_kv_cache& cache, cudaStream_t stream,
                  const DeviceInfo& dev, std::string& err) {
  int rc = CSA_OK;
  cudaError_t e;
  e = cache.head_size <= 64 ? launch_prompt<64, kMode>(a, cache.format, dev, stream, rc, err)
                            : launch_prompt<128, kMode>(a, cache.format, dev, stream, rc, err);
  if (rc != CSA_OK) return rc;
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) {
    err = std::string("launch: ") + cudaGetErrorString(e);
    return CSA_ERR_LAUNCH;
  }
  return CSA_OK;
}

}  // namespace
}  // namespace csa
