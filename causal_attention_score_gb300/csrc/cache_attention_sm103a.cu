// Attention of new tokens over the paged 8-bit cache, for few rows per
// sequence and kv head (decoding): row r of a sequence sits at position p and
//
//   out = sum_t w_t v_t / sum_t w_t,  w_t = exp(c q.k_t),  over the visible t:
//   t <= p, and p - t < window or t < sinks where there is a window.
//
// G = q_heads / heads query heads share a kv head, so a unit of work is a block
// of 8 (or 16) rows (tokens x G) of one sequence and kv head. The step is bound
// by reading the codes of K and V once from HBM; the tensor cores are far from
// busy (8 useful flops a byte at G = 1), so mma.sync, whose operands are
// registers, is the right instruction here: codes go from HBM to registers to
// the tensor core with no trip through shared memory.
//
// Measured: 64 sequences of 300 to 8191 tokens, 16 heads of 128: 139 us, 6.4 TB/s of
// codes (0.94 of the copy rate); 48 of 100 to 15000 with a window of 4096, 8 kv heads:
// 62 us (0.71). One sequence of 777 tokens, 12 heads of 64: 10 us, all latency (the work
// list 1.3 us, the way to the first codes 2.5 us, the join 3 us). With 16 rows a block
// the instructions of a step bound it (4 TB/s at 64 x 4K tokens), not HBM.
//
// Roles: mma.m16n8k16 with the cache as its A operand: scores are S^T = K Q^T
// (16 tokens x 8 rows) and the output O^T = V^T P^T (16 elements x 8 rows), so
// that 8 rows fill the instruction (with Q as A, 16 would be needed) and the
// accumulator of a 128-element head takes 32 registers. P^T comes out of the
// first product as an accumulator and goes into the second as a B operand: one
// movmatrix (an 8 x 8 transposition) per 8 tokens in between.
//
// Codes and scales. Codes become fp16 exactly (|int8| <= 127; e4m3 has 4
// significant bits). Q becomes fp16 after a power-of-two scale per row that
// puts its largest element near 2^14, so a bf16 row keeps all 8 bits down to
// 2^-29 of that. Scores accumulate in fp32; K's scale (constant over a block),
// 1/sqrt and log2(e) multiply the score. V's scale s goes into the exponent:
// with x = c q.k log2(e) + log2(s) the weight w = exp2(x - m) has V's scale in
// it, so one accumulator in units of codes serves blocks of different scales,
// and the denominator sums w / s. Beside a block whose scale is more than 2^60
// times its own a block's weights may come out as 0 (below 2^-126) although their
// keys count: those are added to the denominator as exp2(c q.k log2(e) - m), and
// the denominator is rescaled in two factors, neither of which comes out as 0.
// m is set to 7 below the running maximum of x and raised when a value passes
// m + 15, so that most blocks rescale nothing: the largest w is from 2^7 to 2^15,
// at the upper end of fp16, to which w is rounded for the tensor core (to 11 bits,
// and to 2^-32 of the largest where fp16 is subnormal); sums stay in fp32.
//
// Layout trick: a dot product may run over the elements in any order, so lane
// (g, t) of a warp loads 16 contiguous bytes of token g's K row and uses its
// four words as four k-steps (Q's fragments are loaded to match), and the 16
// contiguous bytes of a V row that a lane loads are 16 rows of V^T.
//
// Work split: all (sequence, head, row block) units in a row, each of as many
// tiles of tokens as its rows see and some for its start (kUnitTiles); every group of
// four warps takes an equal run of that, wherever it begins and ends, so ragged batches
// and few sequences alike use every SM. A group that covers a unit writes its rows; the
// others leave (m, l, O) in the workspace, and a second kernel joins them in a fixed
// order. The work list is computed on the device from the lengths.
//
// Loads: a step's codes are asked for in registers while the step before is computed,
// and in L2 a step before that; across units too (the next piece of the run is worked
// out while the one at hand begins). Without the L2 requests the first case takes 2 % more,
// without those across units another 4 %.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <limits>
#include <string>

#include "csa_internal.h"
#include "kv_cache.cuh"
#include "sm103a_ptx.cuh"

namespace csa {
namespace {

// Groups of four warps per CTA (one CTA per SM), as many as registers allow: heads of up
// to 128 elements need 168 a thread with one 8-row block, 255 with two; of up to 64, 128
// and 168 (64 sequences of 4K tokens, 16 kv heads of 64: 78 us with four groups, 87 with
// three; 4 kv heads with 16 rows each: 41 with three, 50 with two).
template <int HSP, int NB>
constexpr int kGroups = (HSP == 64 ? 4 : 3) - (NB - 1);
// A warp takes kSub blocks of 16 tokens per step, all in one page: two where pages hold 32
// tokens or more. A tile is what a group's four warps take.
template <int kSub>
constexpr int kTileTokens = 64 * kSub;
// A unit counts in the division of work as kUnitTiles tiles more than it has: about what
// finishing a unit and starting the next takes a group. Without it the groups that short
// sequences fall to come last: 64 sequences of 300 to 8191 tokens take 171 us instead
// of 139, 32 of 60 to 2000 tokens 44 instead of 29, 16-row units of 4K tokens 90 instead of 69.
// (One tile: 153, 32, 80; four: 141, 31, 67.)
template <int NB, int kSub>
constexpr int kUnitTiles = (NB == 1 ? 2 : 3) * (2 / kSub);
constexpr int kMaxSms = 152;
constexpr int kMaxWorkers = kMaxSms * 4;
constexpr int kMaxRows = 16;
// Which kernel a sequence's rows go to: those of more than kRowLimit to the one for prompts
// where the batch holds more than kBlocksPerSm blocks of 16 of them for each SM. These are
// counted on the device: single tokens beside a short prompt must not make it one of a
// batch of prompts (63 of 300 to 7300 tokens and one of 40 new over 64K, 8 heads: 176 us, and
// 1022 us with that one in the prompt kernel; the count takes the others' calls 1 us).
// Here each block of 16 rows reads the keys again; the prompt kernel reads them once for 256
// rows, but nothing splits its units along the keys. With 8K keys a block of 16 rows of one
// kv head takes 0.41 us of the whole GPU, 32 rows as much as a unit there (0.82 us) where
// units fill it; where they do not, its 120 us for the first unit buy this kernel 2 blocks an
// SM: 1 sequence of 64 new tokens (8 rows each, 8 heads) takes 113 us here and 130 us there
// (64K keys: 790 and 960 us; none: 15 and 16 us), one of 96 tokens 164 and 131 us.
constexpr int kRowLimit = 32;
constexpr int kBlocksPerSm = 2;
constexpr int kNoRowLimit = std::numeric_limits<int>::max();
constexpr float kRaise = 15.0f;             // an exponent past this raises m,
constexpr float kHeadroom = 7.0f;           // to this far below it
constexpr float kFar = 8.673617379884035e-19f;  // 2^-60: scales of V this far apart
// The running maximum of a row that has seen nothing: finite, so that
// differences of two of them are 0.
constexpr float kNothing = -1e30f;

struct AttendArgs {
  KvView v;
  const void* q;
  void* out;
  long long q_token, q_head, out_token, out_head;
  int half;        // rows are fp16 (else bf16)
  int group;       // query heads per kv head
  int window, sinks;
  float scale_log2;
  int workers;
  int most_rows;   // of a block
  // Sequences of more than kRowLimit rows (tokens x group) are left to the prompt kernel
  // where their blocks of 16 rows, times heads, are more than this.
  long long prompt_blocks;
  int* headers;  // [workers][8]
  PromptList* list;  // the prompt kernel's, written here
  float* parts;    // [2 * workers][part_floats]
  int part_floats;
};

// A piece that begins a unit but does not end it: what the join needs.
enum HeaderWord { kHeadPieces = 0, kHeadRow0, kHeadFirst, kHeadHead, kHeadRows };

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The transposed 8 x 8 matrix of 16-bit elements (lane (g, t): row g, columns
// 2t and 2t + 1).
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ void group_sync(int group) {
  asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory");
}

__device__ __forceinline__ void store_out(const AttendArgs& a, long long at, float v) {
  if (a.half)
    static_cast<__half*>(a.out)[at] = __float2half_rn(v);
  else
    static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(v);
}

// What a sequence asks for: rows (tokens x group), their tiles of tokens (the
// first `sink_tiles`, then those from `window_tile` on).
struct SeqWork {
  KvSequence q;
  int rows, blocks, tiles, sink_tiles, window_tile;
};

template <int NB, int kSub>
__device__ __forceinline__ SeqWork seq_work(const AttendArgs& a, int row_limit, int s) {
  SeqWork w;
  w.q = kv_sequence(a.v, s);
  const long long rows = static_cast<long long>(w.q.n) * a.group;
  if (rows == 0 || rows > row_limit) {
    w.rows = w.blocks = w.tiles = w.sink_tiles = w.window_tile = 0;
    return w;
  }
  w.rows = static_cast<int>(rows);
  w.blocks = (w.rows + 8 * NB - 1) / (8 * NB);
  w.sink_tiles = w.window_tile = 0;
  constexpr int T = kTileTokens<kSub>;
  const int all = (w.q.length + T - 1) / T;
  if (a.window > 0) {
    const int from = max(max(w.q.first, 0) - a.window + 1, 0);  // first key any row's window has
    w.window_tile = from / T;
    const int sinks = min(a.sinks, from);
    w.sink_tiles = min((sinks + T - 1) / T, w.window_tile);
  }
  w.tiles = max(1, w.sink_tiles + all - w.window_tile);  // rows that see nothing: one, for their zeros
  return w;
}

// What a unit of a sequence counts.
template <int NB, int kSub>
__device__ __forceinline__ long long unit_weight(const SeqWork& w) {
  return w.tiles + kUnitTiles<NB, kSub>;
}

// A group's place in the work list and the piece of a unit that it is at. Kept
// in shared memory: the main loop needs the registers.
struct Piece {
  long long at, end;  // the group's run still to do
  long long base;     // where sequence s begins in the list
  SeqWork w;
  int s;
  int head, row_first, rows;  // the unit
  int hidden_to;              // keys below this, from a.sinks on, are no row's to see
  int tile0, count;           // its tiles [tile0, tile0 + count); count 0: no more pieces
  long long after;            // what the unit counts past this piece
};

template <int NB, int kSub>
__device__ __forceinline__ void next_piece(const AttendArgs& a, int row_limit, Piece& p) {
  constexpr int E = kUnitTiles<NB, kSub>;
  p.count = 0;
  while (p.at < p.end) {
    long long weight;
    for (;;) {
      weight = unit_weight<NB, kSub>(p.w);
      const long long all = static_cast<long long>(p.w.blocks) * a.v.heads * weight;
      if (p.at < p.base + all) break;
      p.base += all;
      if (++p.s >= a.v.sequences) {  // lengths changed under the call: nothing more
        p.at = p.end;
        return;
      }
      p.w = seq_work<NB, kSub>(a, row_limit, p.s);
    }
    const long long off = p.at - p.base;
    const int unit = static_cast<int>(
        (off >> 32) == 0 ? static_cast<unsigned>(off) / static_cast<unsigned>(weight)
                         : off / weight);
    const int from = static_cast<int>(off - static_cast<long long>(unit) * weight);
    const int to = static_cast<int>(min(weight, static_cast<long long>(from) + (p.end - p.at)));
    p.at += to - from;
    if (to <= E) continue;  // the run ends before the unit's first tile
    p.tile0 = max(from - E, 0);
    p.count = to - E - p.tile0;
    p.after = weight - to;
    p.head = unit / p.w.blocks;
    p.row_first = (unit - p.head * p.w.blocks) * (8 * NB);
    p.rows = min(p.w.rows - p.row_first, 8 * NB);
    p.hidden_to = a.window > 0 ? p.w.q.first + p.row_first / a.group - a.window + 1 : 0;
    return;
  }
}

// (checking build) whether a piece's rows and tiles are its sequence's.
[[maybe_unused]] __device__ __forceinline__ bool piece_ok(const AttendArgs& a,
                                                          const volatile Piece& p) {
  return p.s >= 0 && p.s < a.v.sequences && p.head >= 0 && p.head < a.v.heads &&
         p.row_first >= 0 && p.rows > 0 && p.rows <= kMaxRows &&
         p.row_first + p.rows <= p.w.rows && p.w.q.row0 >= 0 &&
         p.w.q.row0 + p.w.q.n <= a.v.rows && p.tile0 >= 0 && p.count > 0 &&
         p.tile0 + p.count <= p.w.tiles;
}

template <int HSP, int NB>
struct GroupSmem {
  // Floats per lane column and row, padded so that the float4 accesses of eight
  // lanes (two g, four t) fall into different banks.
  static constexpr int kColStride = HSP / 8 + 4;
  static constexpr int kRowStride = 8 * kColStride + 4;
  // Q's fragments stay in registers with one row block; two take this.
  static constexpr bool kSharedQ = NB == 2 && HSP == 128;
  float o[4][8 * NB][kRowStride];
  uint4 q[kSharedQ ? NB * HSP / 32 : 1][32];
  float m[4][8 * NB], l[4][8 * NB];
  Piece piece[2];  // the one at hand and the next
};

// HSP: head size padded to 64 or 128; kFull: head_size == HSP (no bounds on the
// element loads).
template <int HSP, int NB, int kSub, int kFormat, bool kFull>
__global__ void __launch_bounds__(128 * kGroups<HSP, NB>, 1)
    attend_rows_sm103a_kernel(const AttendArgs a) {
  constexpr int kThreads = 128 * kGroups<HSP, NB>;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  __shared__ long long s_prefix[kThreads + 1];
  __shared__ long long s_warp[kThreads / 32];
  __shared__ unsigned long long s_blocks;
  [[maybe_unused]] __shared__ int s_abort;
  [[maybe_unused]] const Watchdog wd{0, a.v.status, &s_abort};
  using Smem = GroupSmem<HSP, NB>;
  Smem* groups = reinterpret_cast<Smem*>(smem_raw);
  constexpr int kChunks = HSP / 64;       // 16-byte chunks of a K row per lane
  constexpr int kVBytes = HSP / 8;        // bytes of a V row per lane
  constexpr int kVWords = kVBytes / 4;
  constexpr int kTilesM = HSP / 16;       // m-tiles of the output

  grid_dependency_wait();

  // -------------------------------------------------------- the work list --
  // Thread i sums the work of sequences [i c, (i + 1) c); a scan over the CTA
  // gives where each run begins.
  const int S = a.v.sequences;
  const int c = (S + kThreads - 1) / kThreads;
  const int lane = threadIdx.x & 31, warp_id = threadIdx.x >> 5;
  const long long from = static_cast<long long>(threadIdx.x) * c;
  const long long until = min(static_cast<long long>(S), from + c);
  if (threadIdx.x == 0) s_blocks = 0;
  __syncthreads();
  if (a.prompt_blocks > 0) {
    unsigned long long mine = 0;
    for (long long s = from; s < until; ++s) {
      const long long rows =
          static_cast<long long>(kv_sequence(a.v, static_cast<int>(s)).n) * a.group;
      if (rows > kRowLimit) mine += (rows + 15) / 16 * a.v.heads;
    }
    if (mine > 0) atomicAdd(&s_blocks, mine);
    __syncthreads();
  }
  // (read again wherever it is needed: the main loop needs the registers)
  auto row_limit = [&] {
    return static_cast<long long>(s_blocks) > a.prompt_blocks ? kRowLimit : kNoRowLimit;
  };
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.list = PromptList{0u, row_limit()};
  {
    long long mine = 0;
    for (long long s = from; s < until; ++s) {
      const SeqWork w = seq_work<NB, kSub>(a, row_limit(), static_cast<int>(s));
      mine += static_cast<long long>(w.blocks) * a.v.heads * unit_weight<NB, kSub>(w);
    }
    long long sum = mine;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const long long up = __shfl_up_sync(0xFFFFFFFFu, sum, d);
      if (lane >= d) sum += up;
    }
    if (lane == 31) s_warp[warp_id] = sum;
    __syncthreads();
    long long before = 0;
    for (int w = 0; w < warp_id; ++w) before += s_warp[w];
    s_prefix[threadIdx.x + 1] = before + sum;
    if (threadIdx.x == 0) s_prefix[0] = 0;
    __syncthreads();
  }
  const long long total = s_prefix[kThreads];
  const int gi = warp_id >> 2;       // group in the CTA
  const int warp = warp_id & 3;      // warp in the group
  const int gtid = threadIdx.x & 127;
  const int worker = blockIdx.x * kGroups<HSP, NB> + gi;
  const long long share = (total + a.workers - 1) / a.workers;
  Smem& sm = groups[gi];
  const int g = lane >> 2, t = lane & 3;
  const int D = kFull ? HSP : a.v.head_size;
  int* header = a.headers + worker * 8;
  bool left_open = false;

  if (gtid == 0) {
    Piece& p = sm.piece[0];
    p.at = min(share * worker, total);
    p.end = min(p.at + share, total);
    if (p.at < p.end) {
      int lo = 0, hi = kThreads;  // s_prefix[lo] <= at < s_prefix[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (s_prefix[mid] <= p.at) lo = mid;
        else hi = mid;
      }
      p.s = lo * c;
      p.base = s_prefix[lo];
      p.w = seq_work<NB, kSub>(a, row_limit(), p.s);
    }
    next_piece<NB, kSub>(a, row_limit(), p);
  }
  group_sync(gi);

  // K's chunks and V's of a step's blocks as they come from HBM, their page's scales.
  uint4 kr[kSub][2][kChunks];
  uint32_t vr[kSub][4][kVWords];
  float ks = 1.0f, vs = 1.0f;
  // Where this warp's tokens of the step at hand and of the next are: page * heads + head
  // (below 2^31 for any cache that fits in memory), -1 where there is nothing to read; the
  // first of the tokens.
  int unit = -1, unit_next = -1, tb = 0, tb_next = 0;
  bool begin = true;
  for (int cur = 0;; cur ^= 1) {
    const volatile Piece& piece = sm.piece[cur];
    const int count = piece.count;
    if (count == 0) break;
    if (!CSA_CHECK(piece_ok(a, piece), wd, kCheckTile)) break;
    const int head = piece.head;
    const int length = piece.w.q.length;

    // The same of step i; past the piece's end, of the next piece's.
    auto look = [&](int i, int& first) {
      const bool past = i >= count;
      const volatile Piece& p = sm.piece[past ? cur ^ 1 : cur];
      if (past) {
        i -= count;
        if (i >= p.count) return -1;
      }
      const int tile = p.tile0 + i;
      first = (tile < p.w.sink_tiles ? tile : tile + p.w.window_tile - p.w.sink_tiles) *
                  kTileTokens<kSub> +
              warp * (16 * kSub);
      if (first >= p.w.q.length) return -1;
      if (a.window != 0 && first >= a.sinks && first + 16 * kSub <= p.hidden_to) return -1;
      if (!CSA_CHECK(first >= 0 && (first & (a.v.page_tokens - 1)) + 16 * kSub <= a.v.page_tokens,
                     wd, kCheckTile))
        return -1;
      const int page = kv_page(a.v, p.s, first >> a.v.page_shift);
      return page < 0 ? -1 : page * a.v.heads + p.head;
    };
    // Lane (g, t): tokens g and g + 8, chunks t and t + 4 of their K rows; tokens
    // 2t, 2t + 1, 2t + 8, 2t + 9, chunk g of their V rows.
    const uint8_t* k_lane = a.v.codes[0] + (g * D + t * 16);
    const uint8_t* v_lane = a.v.codes[1] + (2 * t * D + g * kVBytes);
    const int page_bytes = a.v.page_tokens * D;
    auto load_k = [&](int first, int u0) {
      const uint8_t* from = k_lane + (static_cast<long long>(u0) * page_bytes +
                                      (first & (a.v.page_tokens - 1)) * D);
#pragma unroll
      for (int u = 0; u < kSub; ++u)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int h = 0; h < kChunks; ++h)
            kr[u][n][h] = kFull || (4 * h + t) * 16 < D
                              ? __ldg(reinterpret_cast<const uint4*>(from + (16 * u + 8 * n) * D +
                                                                     64 * h))
                              : make_uint4(0, 0, 0, 0);
      ks = __ldg(a.v.scale[0] + u0);
    };
    auto load_v = [&](int first, int u0) {
      const uint8_t* from = v_lane + (static_cast<long long>(u0) * page_bytes +
                                      (first & (a.v.page_tokens - 1)) * D);
      const bool in = kFull || g * kVBytes < D;
#pragma unroll
      for (int u = 0; u < kSub; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint8_t* row = from + (16 * u + (i & 1) + 8 * (i >> 1)) * D;
          if constexpr (kVWords == 4) {
            const uint4 x = in ? __ldg(reinterpret_cast<const uint4*>(row)) : make_uint4(0, 0, 0, 0);
            vr[u][i][0] = x.x;
            vr[u][i][1] = x.y;
            vr[u][i][2] = x.z;
            vr[u][i][3] = x.w;
          } else {
            const uint2 x = in ? __ldg(reinterpret_cast<const uint2*>(row)) : make_uint2(0, 0);
            vr[u][i][0] = x.x;
            vr[u][i][1] = x.y;
          }
        }
      vs = __ldg(a.v.scale[1] + u0);
    };
    // Asks for a step's codes in L2 (they are one run of memory in K and in V).
    auto prefetch = [&](int first, int u0) {
      if (lane < 2)
        bulk_prefetch_l2(a.v.codes[lane] + static_cast<long long>(u0) * page_bytes +
                             (first & (a.v.page_tokens - 1)) * D,
                         16 * kSub * D);
    };
    if (begin) {
      begin = false;
      unit = look(0, tb);
      if (count > 1) unit_next = look(1, tb_next);
      if (unit >= 0) {
        load_k(tb, unit);
        load_v(tb, unit);
      }
    }

    // ------------------------------------------------------ Q's fragments --
    // Lane (g, t): row g (and g + 8), the 16 elements of chunks t and t + 4.
    uint32_t qf[NB][kChunks][8];
    float fr[NB][2];  // of rows 2t, 2t + 1 (this lane's columns of S^T)
    int pr[NB][2];
    int pos_low, pos_high;
    {
      const int row_first = piece.row_first, rows = piece.rows;
      const int first = piece.w.q.first, row0 = piece.w.q.row0;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int rr = row_first + 8 * b + g;
        const int j = rr / a.group;
        const bool live = 8 * b + g < rows;
        float back = 1.0f, most = 0.0f;
#pragma unroll
        for (int h = 0; h < kChunks; ++h) {
          const int d = (4 * h + t) * 16;
          uint4 raw[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
          if (live && (kFull || d < D)) {
            const uint4* from = reinterpret_cast<const uint4*>(
                static_cast<const uint16_t*>(a.q) + (row0 + j) * a.q_token +
                (head * a.group + (rr - j * a.group)) * a.q_head + d);
            raw[0] = from[0];
            raw[1] = from[1];
          }
          const uint32_t* word = reinterpret_cast<const uint32_t*>(raw);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            qf[b][h][i] = word[i];
            most = fmaxf(most, fmaxf(fabsf(__uint_as_float(word[i] << 16)),
                                     fabsf(__uint_as_float(word[i] & 0xFFFF0000u))));
          }
        }
        if (!a.half) {  // bf16 rows: to fp16, scaled
          most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
          most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
          const uint32_t e = max(__float_as_uint(most) >> 23, 15u);
          const float up = __uint_as_float((268u - e) << 23);  // 2^(14 - exponent)
          back = __uint_as_float((e - 14u) << 23);
#pragma unroll
          for (int h = 0; h < kChunks; ++h)
#pragma unroll
            for (int i = 0; i < 8; ++i)
              qf[b][h][i] = half2_of(__uint_as_float(qf[b][h][i] << 16) * up,
                                     __uint_as_float(qf[b][h][i] & 0xFFFF0000u) * up);
        }
        if constexpr (Smem::kSharedQ) {
          if (warp == 0)
#pragma unroll
            for (int h = 0; h < kChunks; ++h)
#pragma unroll
              for (int k = 0; k < 2; ++k)
                sm.q[(b * kChunks + h) * 2 + k][lane] =
                    make_uint4(qf[b][h][4 * k], qf[b][h][4 * k + 1], qf[b][h][4 * k + 2],
                               qf[b][h][4 * k + 3]);
        }
        const float f = a.scale_log2 * back;
        const int pos = live ? first + j : -1;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          fr[b][e] = __shfl_sync(0xFFFFFFFFu, f, (2 * t + e) * 4);
          pr[b][e] = __shfl_sync(0xFFFFFFFFu, pos, (2 * t + e) * 4);
        }
      }
      pos_low = first + row_first / a.group;
      pos_high = first + (row_first + rows - 1) / a.group;
    }
    // The next piece, so that its first steps' codes are asked for before this one ends.
    if (gtid == 0) {
      Piece& next = sm.piece[cur ^ 1];
      next = sm.piece[cur];
      next_piece<NB, kSub>(a, row_limit(), next);
    }
    group_sync(gi);
    if (count == 1) unit_next = look(1, tb_next);
    if (unit_next >= 0) prefetch(tb_next, unit_next);

    float o[NB][kTilesM][4];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < kTilesM; ++i) o[b][i][0] = o[b][i][1] = o[b][i][2] = o[b][i][3] = 0.0f;
    float m[NB][2], l[NB][2];
    float far = 0.0f;  // 2^-60 of the largest scale of V so far
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      m[b][0] = m[b][1] = kNothing;
      l[b][0] = l[b][1] = 0.0f;
    }

    for (int i = 0; i < count; ++i) {
      int tb_after = 0;
      const int unit_after = look(i + 2, tb_after);
      if (unit >= 0) {
        float sc[kSub][NB][4];
#pragma unroll
        for (int u = 0; u < kSub; ++u)
#pragma unroll
          for (int b = 0; b < NB; ++b) sc[u][b][0] = sc[u][b][1] = sc[u][b][2] = sc[u][b][3] = 0.0f;
#pragma unroll
        for (int h = 0; h < kChunks; ++h)
#pragma unroll
          for (int k2 = 0; k2 < 2; ++k2) {
            uint32_t q4[NB][4];
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              if constexpr (Smem::kSharedQ) {
                const uint4 x = sm.q[(b * kChunks + h) * 2 + k2][lane];
                q4[b][0] = x.x;
                q4[b][1] = x.y;
                q4[b][2] = x.z;
                q4[b][3] = x.w;
              } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) q4[b][e] = qf[b][h][4 * k2 + e];
              }
            }
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int u = 0; u < kSub; ++u) {
                const uint32_t* k0 = reinterpret_cast<const uint32_t*>(&kr[u][0][h]);
                const uint32_t* k1 = reinterpret_cast<const uint32_t*>(&kr[u][1][h]);
                uint32_t a0, a1, a2, a3;
                codes4_to_half2x2<kFormat>(k0[2 * k2 + k], a0, a2);
                codes4_to_half2x2<kFormat>(k1[2 * k2 + k], a1, a3);
#pragma unroll
                for (int b = 0; b < NB; ++b)
                  mma_f16(sc[u][b], a0, a1, a2, a3, q4[b][2 * k], q4[b][2 * k + 1]);
              }
          }
        // A block of scale 0 holds zeros, at any scale.
        const bool zeros = vs == 0.0f;
        vs = fmaxf(vs, kScaleFloor);
        const float lv = __log2f(vs), inv = __fdividef(1.0f, vs);
        float fk[NB][2];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          fk[b][0] = fr[b][0] * ks;
          fk[b][1] = fr[b][1] * ks;
        }
        if (unit_next >= 0) load_k(tb_next, unit_next);
        // sc element e: token g + 8 (e / 2), row 2t + e % 2. A masked score is -inf, and
        // stays so whatever the scales.
        const int last = tb + 16 * kSub - 1;
        const bool open = last <= pos_low &&
                          (a.window == 0 || pos_high - tb < a.window || last < a.sinks);
        float x[kSub][NB][4];
        bool raise = false;
#pragma unroll
        for (int u = 0; u < kSub; ++u)
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              x[u][b][e] = fmaf(sc[u][b][e], fk[b][e & 1], lv - m[b][e & 1]);
              if (!open) {
                const int tok = tb + 16 * u + g + 8 * (e >> 1), p = pr[b][e & 1];
                if (tok > p || (a.window != 0 && p - tok >= a.window && tok >= a.sinks)) {
                  sc[u][b][e] = -INFINITY;
                  x[u][b][e] = -INFINITY;
                }
              }
              raise |= x[u][b][e] > kRaise;
            }
        raise |= vs < far;  // (rare, and the warp's)
        far = fmaxf(far, vs * kFar);
        if (__any_sync(0xFFFFFFFFu, raise)) {
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              float y[kSub][2], most = -INFINITY;
#pragma unroll
              for (int u = 0; u < kSub; ++u)
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                  y[u][n] = sc[u][b][2 * n + r] == -INFINITY
                                ? -INFINITY
                                : fmaf(sc[u][b][2 * n + r], fk[b][r], lv);
                  most = fmaxf(most, y[u][n]);
                }
              most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 4));
              most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 8));
              most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 16));
              const float top = fmaxf(m[b][r], most - kHeadroom);
              const float half = ex2_approx(0.5f * (m[b][r] - top)), corr = half * half;
              m[b][r] = top;
              l[b][r] = l[b][r] * half * half;
#pragma unroll
              for (int j = 0; j < kTilesM; ++j) {
                o[b][j][r] *= corr;
                o[b][j][2 + r] *= corr;
              }
#pragma unroll
              for (int u = 0; u < kSub; ++u)
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                  x[u][b][2 * n + r] = y[u][n] - top;
                  // (V far below that of others: what comes out as 0 is added without its scale)
                  if (x[u][b][2 * n + r] < -126.0f) l[b][r] += ex2_approx(x[u][b][2 * n + r] - lv);
                }
            }
        }
        uint32_t pb[kSub][NB][2];
#pragma unroll
        for (int u = 0; u < kSub; ++u)
#pragma unroll
          for (int b = 0; b < NB; ++b) {
#pragma unroll
            for (int e = 0; e < 4; ++e) x[u][b][e] = ex2_approx(x[u][b][e]);
            l[b][0] = fmaf(x[u][b][0] + x[u][b][2], inv, l[b][0]);
            l[b][1] = fmaf(x[u][b][1] + x[u][b][3], inv, l[b][1]);
            pb[u][b][0] = transpose_8x8(half2_of(x[u][b][0], x[u][b][1]));
            pb[u][b][1] = transpose_8x8(half2_of(x[u][b][2], x[u][b][3]));
          }
        // Slots past the sequence's end, and those that no row's window reaches, may hold the
        // codes of no number (int8 has none: there a weight of 0 is enough).
        if (last >= length || zeros ||
            (kFormat == CSA_KV_E4M3 && a.window != 0 && pos_low - tb >= a.window)) {
          const int hidden_to = a.window != 0 ? pos_low - a.window + 1 : 0;
          const int end = zeros ? 0 : length;
#pragma unroll
          for (int u = 0; u < kSub; ++u)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int tok = tb + 16 * u + 2 * t + (k & 1) + 8 * (k >> 1);
              if (tok >= end ||
                  (kFormat == CSA_KV_E4M3 && tok < hidden_to && tok >= a.sinks)) {
#pragma unroll
                for (int j = 0; j < kVWords; ++j) vr[u][k][j] = 0;
              }
            }
        }
#pragma unroll
        for (int u = 0; u < kSub; ++u)
#pragma unroll
          for (int j = 0; j < kVWords; ++j) {
            // four elements of two token pairs: bytes to (token, token + 1) pairs
            uint32_t f[4][2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              uint32_t v0 = vr[u][2 * k][j], v1 = vr[u][2 * k + 1][j];
              if (kFormat == CSA_KV_INT8) {
                v0 ^= 0x80808080u;
                v1 ^= 0x80808080u;
              }
              const uint32_t lo = byte_perm(v0, v1, 0x5140), hi = byte_perm(v0, v1, 0x7362);
              if (kFormat == CSA_KV_INT8) {
                f[0][k] = flipped_pair_to_half2<0x4140>(lo);
                f[1][k] = flipped_pair_to_half2<0x4342>(lo);
                f[2][k] = flipped_pair_to_half2<0x4140>(hi);
                f[3][k] = flipped_pair_to_half2<0x4342>(hi);
              } else {
                f[0][k] = e4m3x2_to_half2(lo & 0xFFFFu);
                f[1][k] = e4m3x2_to_half2(lo >> 16);
                f[2][k] = e4m3x2_to_half2(hi & 0xFFFFu);
                f[3][k] = e4m3x2_to_half2(hi >> 16);
              }
            }
            // m-tile 2j: elements 4j (rows g) and 4j + 1 (rows g + 8) of the chunk
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              mma_f16(o[b][2 * j], f[0][0], f[1][0], f[0][1], f[1][1], pb[u][b][0], pb[u][b][1]);
              mma_f16(o[b][2 * j + 1], f[2][0], f[3][0], f[2][1], f[3][1], pb[u][b][0],
                      pb[u][b][1]);
            }
          }
      } else if (unit_next >= 0) {
        load_k(tb_next, unit_next);
      }
      if (unit_next >= 0) load_v(tb_next, unit_next);
      if (unit_after >= 0) prefetch(tb_after, unit_after);
      unit = unit_next;
      tb = tb_next;
      unit_next = unit_after;
      tb_next = tb_after;
    }

    // ------------------------------------------- the four warps' results --
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
#pragma unroll
        for (int d = 4; d < 32; d *= 2) l[b][r] += __shfl_xor_sync(0xFFFFFFFFu, l[b][r], d);
        if (g == 0) {
          sm.m[warp][8 * b + 2 * t + r] = m[b][r];
          sm.l[warp][8 * b + 2 * t + r] = l[b][r];
        }
      }
    group_sync(gi);
    const int rows = piece.rows;
    auto row_max = [&](int r) {
      return fmaxf(fmaxf(sm.m[0][r], sm.m[1][r]), fmaxf(sm.m[2][r], sm.m[3][r]));
    };
    // lane (g, t) holds elements g * kVBytes .. of rows 2t and 2t + 1: element 2j of
    // a chunk in o[j][0..1], 2j + 1 in o[j][2..3]
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * b + 2 * t + e;
        if (r >= rows) continue;
        const float corr = ex2_approx(m[b][e] - row_max(r));
        float* to = &sm.o[warp][r][g * Smem::kColStride];
#pragma unroll
        for (int j = 0; j < kTilesM; j += 2)
          *reinterpret_cast<float4*>(to + 2 * j) =
              make_float4(o[b][j][e] * corr, o[b][j][2 + e] * corr, o[b][j + 1][e] * corr,
                          o[b][j + 1][2 + e] * corr);
      }
    group_sync(gi);
    const bool begins = piece.tile0 == 0, whole = begins && piece.count == piece.w.tiles;
    const int row_first = piece.row_first, row0 = piece.w.q.row0, out_head = piece.head * a.group;
    const int slot = 2 * worker + (begins ? 1 : 0);
    if (!CSA_CHECK(slot < 2 * kMaxWorkers, wd, kCheckRing)) break;
    float* part = a.parts + static_cast<long long>(slot) * a.part_floats;
    for (int e = gtid; e < rows * HSP; e += 128) {
      const int r = e / HSP, d = e % HSP;
      const int idx = (d / kVBytes) * Smem::kColStride + d % kVBytes;
      const float mm = row_max(r);
      const float acc = (sm.o[0][r][idx] + sm.o[1][r][idx]) + (sm.o[2][r][idx] + sm.o[3][r][idx]);
      float lt = 0.0f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float half = ex2_approx(0.5f * (sm.m[k][r] - mm));
        lt += sm.l[k][r] * half * half;
      }
      if (whole) {
        const int rr = row_first + r;
        const int j = rr / a.group;
        if (kFull || d < D)
          store_out(a,
                    (row0 + j) * a.out_token + (out_head + (rr - j * a.group)) * a.out_head + d,
                    lt == 0.0f ? 0.0f : acc / lt);
      } else {
        part[2 * kMaxRows + r * HSP + d] = acc;
        if (d == 0) {
          part[r] = mm;
          part[kMaxRows + r] = lt;
        }
      }
    }
    if (!whole && begins) {
      left_open = true;
      if (gtid == 0) {
        // (at most those there are: lengths may have changed under the call)
        header[kHeadPieces] = static_cast<int>(
            min(1 + (piece.after + share - 1) / share, static_cast<long long>(a.workers - worker)));
        header[kHeadRow0] = row0;
        header[kHeadFirst] = row_first;
        header[kHeadHead] = piece.head;
        header[kHeadRows] = rows;
      }
    }
    group_sync(gi);  // sm is reused
  }
  if (!left_open && gtid == 0) header[kHeadPieces] = 0;
}

// Joins the pieces of each unit that was split: row blockIdx.y of the unit that the
// last piece of worker blockIdx.x begins. Piece 0 is that worker's second slot, piece
// i the first slot of worker + i. Warp w takes pieces w, w + 4, ...; the four sums are
// added in order.
template <int HSP>
__global__ void __launch_bounds__(128) attend_join_sm103a_kernel(const AttendArgs a) {
  __shared__ float s_o[4][HSP];
  __shared__ float s_l[4], s_m[4];
  grid_dependency_wait();
  const int worker = blockIdx.x, r = blockIdx.y;
  const int* header = a.headers + worker * 8;
  const int pieces = header[kHeadPieces];
  if (pieces == 0 || r >= header[kHeadRows]) return;
  [[maybe_unused]] __shared__ int s_abort;
  [[maybe_unused]] const Watchdog wd{0, a.v.status, &s_abort};
  if (!CSA_CHECK(pieces > 0 && worker + pieces <= static_cast<int>(gridDim.x) &&
                     2 * (worker + pieces) <= 2 * kMaxWorkers,
                 wd, kCheckRing))
    return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int E = HSP / 32;
  auto part_of = [&](int i) {
    const int slot = i == 0 ? 2 * worker + 1 : 2 * (worker + i);
    return a.parts + static_cast<long long>(slot) * a.part_floats;
  };
  float m = kNothing;
  for (int i = threadIdx.x; i < pieces; i += 128) m = fmaxf(m, part_of(i)[r]);
#pragma unroll
  for (int d = 1; d < 32; d *= 2) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
  if (lane == 0) s_m[warp] = m;
  __syncthreads();
  m = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
  float acc[E] = {}, l = 0.0f;
#pragma unroll 4
  for (int i = warp; i < pieces; i += 4) {
    const float* p = part_of(i);
    const float half = ex2_approx(0.5f * (p[r] - m)), c = half * half;
    l = fmaf(p[kMaxRows + r] * half, half, l);
#pragma unroll
    for (int k = 0; k < E; ++k)
      acc[k] = fmaf(p[2 * kMaxRows + r * HSP + lane * E + k], c, acc[k]);
  }
#pragma unroll
  for (int k = 0; k < E; ++k) s_o[warp][lane * E + k] = acc[k];
  if (lane == 0) s_l[warp] = l;
  __syncthreads();
  const float lt = (s_l[0] + s_l[1]) + (s_l[2] + s_l[3]);
  const int rr = header[kHeadFirst] + r;
  const int j = rr / a.group;
  const int d = threadIdx.x;
  if (d < a.v.head_size)
    store_out(a,
              (header[kHeadRow0] + j) * a.out_token +
                  (header[kHeadHead] * a.group + (rr - j * a.group)) * a.out_head + d,
              lt == 0.0f ? 0.0f : ((s_o[0][d] + s_o[1][d]) + (s_o[2][d] + s_o[3][d])) / lt);
}

template <int HSP, int NB, int kSub, int kFormat, bool kFull>
cudaError_t launch_rows(AttendArgs a, int sms, const DeviceInfo& dev, cudaStream_t stream, int& rc,
                        std::string& err) {
  const auto kernel = attend_rows_sm103a_kernel<HSP, NB, kSub, kFormat, kFull>;
  const int smem = static_cast<int>(sizeof(GroupSmem<HSP, NB>)) * kGroups<HSP, NB>;
  a.workers = sms * kGroups<HSP, NB>;
  rc = set_max_dynamic_smem(reinterpret_cast<const void*>(kernel), smem, dev.device, err);
  if (rc != CSA_OK) return cudaSuccess;
  cudaError_t e = launch_programmatic(kernel, static_cast<unsigned>(sms), 128 * kGroups<HSP, NB>, smem,
                                      stream, a);
  if (e != cudaSuccess) return e;
  return launch_programmatic(attend_join_sm103a_kernel<HSP>,
                             dim3(static_cast<unsigned>(a.workers),
                                  static_cast<unsigned>(std::min(a.most_rows, 8 * NB))),
                             128, 0, stream, a);
}

template <int HSP, int NB, int kSub>
cudaError_t launch_rows(const AttendArgs& a, int format, int sms, const DeviceInfo& dev,
                        cudaStream_t stream, int& rc, std::string& err) {
  const bool full = a.v.head_size == HSP;
  if (format == CSA_KV_INT8)
    return full ? launch_rows<HSP, NB, kSub, CSA_KV_INT8, true>(a, sms, dev, stream, rc, err)
                : launch_rows<HSP, NB, kSub, CSA_KV_INT8, false>(a, sms, dev, stream, rc, err);
  return full ? launch_rows<HSP, NB, kSub, CSA_KV_E4M3, true>(a, sms, dev, stream, rc, err)
              : launch_rows<HSP, NB, kSub, CSA_KV_E4M3, false>(a, sms, dev, stream, rc, err);
}

template <int HSP, int NB>
cudaError_t launch_rows(const AttendArgs& a, int format, int sms, const DeviceInfo& dev,
                        cudaStream_t stream, int& rc, std::string& err) {
  return a.v.page_tokens < 32 ? launch_rows<HSP, NB, 1>(a, format, sms, dev, stream, rc, err)
                              : launch_rows<HSP, NB, 2>(a, format, sms, dev, stream, rc, err);
}

int padded_head(int head_size) { return head_size <= 64 ? 64 : 128; }

}  // namespace

size_t cache_attention_workspace_bytes(int head_size) {
  return static_cast<size_t>(kMaxWorkers + 1) * 8 * sizeof(int) +
         static_cast<size_t>(2 * kMaxWorkers) *
             (2 * kMaxRows + kMaxRows * static_cast<size_t>(padded_head(head_size))) *
             sizeof(float);
}

int cache_attention_launch(const csa_kv_cache& cache, const csa_kv_batch& batch,
                           const AttendCall& call, cudaStream_t stream, const DeviceInfo& dev,
                           std::string& err) {
  AttendArgs a;
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
  const int sms = std::min(dev.sm_count, kMaxSms);
  a.workers = 0;
  const long long most_rows = static_cast<long long>(batch.max_new) * a.group;
  const long long batch_rows = static_cast<long long>(batch.rows) * a.group;
  // Whether the batch's rows could be prompts enough, however they are shared out.
  a.prompt_blocks = static_cast<long long>(kBlocksPerSm) * sms;
  const long long sequences = std::min<long long>(batch.sequences, batch_rows / (kRowLimit + 1));
  const bool prompts = most_rows > kRowLimit &&
                       (batch_rows / 16 + sequences) * cache.heads > a.prompt_blocks;
  if (!prompts) a.prompt_blocks = 0;
  const int hsp = padded_head(cache.head_size);
  a.headers = static_cast<int*>(call.workspace);
  a.list = reinterpret_cast<PromptList*>(a.headers + kMaxWorkers * 8);
  a.parts = reinterpret_cast<float*>(a.headers + (kMaxWorkers + 1) * 8);
  a.part_floats = 2 * kMaxRows + kMaxRows * hsp;
  a.most_rows = static_cast<int>(std::min<long long>(most_rows, kMaxRows));
  // Rows a block. 16 read the codes of 9 to 16 rows once instead of twice, but cost 8 and
  // fewer a second product for nothing and a third group of warps: 64 sequences of 16 rows
  // over 4K tokens take 69 us with 16, 81 us with 8; a batch of 4, 8 and 12 rows takes
  // 81 us with 16, 62 us with 8. So: 16 where a token alone has more than 8, or where
  // the batch's average does (prompts, which are another kernel's, left out of it).
  const bool one = most_rows <= 8 ||
                   (a.group <= 8 && (prompts || batch_rows <= 8LL * batch.sequences));
  int rc = CSA_OK;
  cudaError_t e;
  if (hsp == 64)
    e = one ? launch_rows<64, 1>(a, cache.format, sms, dev, stream, rc, err)
            : launch_rows<64, 2>(a, cache.format, sms, dev, stream, rc, err);
  else
    e = one ? launch_rows<128, 1>(a, cache.format, sms, dev, stream, rc, err)
            : launch_rows<128, 2>(a, cache.format, sms, dev, stream, rc, err);
  if (rc != CSA_OK) {
    err = "cache_attention_forward: " + err;
    return rc;
  }
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) {
    err = std::string("cache_attention_forward: launch: ") + cudaGetErrorString(e);
    return CSA_ERR_LAUNCH;
  }
  if (prompts) {
    rc = cache_prompt_launch(cache, batch, call, a.list, stream, dev, err);
    if (rc != CSA_OK) {
      err = "cache_attention_forward: " + err;
      return rc;
    }
  }
  return CSA_OK;
}

}  // namespace csa
