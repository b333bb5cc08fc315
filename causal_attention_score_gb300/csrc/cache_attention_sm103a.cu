// Attention of new tokens over the paged 8-bit cache, for few rows per
// sequence and kv head (decoding): row r of a sequence sits at position p and
//
//   out = sum_t w_t v_t / sum_t w_t,  w_t = exp(c q.k_t),  over the visible t:
//   t <= p, and p - t < window or t < sinks where there is a window.
//
// G = q_heads / heads query heads share a kv head, so a unit of work is up to
// 16 rows (tokens x G) of one sequence and kv head: the M of one
// mma.m16n8k16, whatever G is. The step is bound by reading the codes of K and
// V once from HBM; the tensor cores are far from busy (8 useful flops a byte
// at G = 1), so mma.sync, whose operands are registers, is the right
// instruction here: codes go from HBM to registers to the tensor core with no
// trip through shared memory.
//
// Codes and scales. Codes become fp16 exactly (|int8| <= 127; e4m3 has 4
// significant bits). Q becomes fp16 after a power-of-two scale per row that
// puts its largest element near 2^14, so a bf16 row keeps all 8 bits down to
// 2^-29 of that. Scores accumulate in fp32; K's scale (constant over a block),
// 1/sqrt and log2(e) multiply the score. V's scale s goes into the exponent:
// with x = c q.k log2(e) + log2(s) the weight w = exp2(x - m) has V's scale in
// it, so one accumulator in units of codes serves blocks of different scales,
// and the denominator sums w / s. m is within 8 of the running maximum of x
// (it is raised when a value passes m + 8, so that most blocks rescale
// nothing): w <= 256, and w is rounded to fp16 (11 bits) for the tensor core;
// sums stay in fp32.
//
// Layout trick: a dot product may run over the elements in any order, so lane
// (g, t) of a warp loads 16 contiguous bytes of token g's K row and uses its
// four words as four k-steps (Q's fragments are laid out to match), and the 16
// contiguous bytes of a V row that a lane loads are 16 of its n-tiles.
//
// Work split: all (sequence, head, row block) units in a row, each of as many
// 64-token tiles as its rows see; every group of four warps takes an equal run
// of tiles, wherever it begins and ends, so ragged batches and few sequences
// alike use every SM. A group that covers a unit writes its rows; the others
// leave (m, l, O) in the workspace, and a second kernel joins them in a fixed
// order. The work list is computed on the device from the lengths.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <string>

#include "csa_internal.h"
#include "kv_cache.cuh"
#include "sm103a_ptx.cuh"

namespace csa {
namespace {

constexpr int kGroups = 3;                  // groups of four warps per CTA
constexpr int kThreads = kGroups * 128;
constexpr int kRows = 16;
constexpr int kTileTokens = 64;             // per group and step: 16 a warp
constexpr int kMaxSms = 152;
constexpr int kMaxWorkers = kMaxSms * kGroups;
constexpr float kRaise = 8.0f;              // the running maximum is raised past this
constexpr float kNegInf = -INFINITY;

struct AttendArgs {
  KvView v;
  const void* q;
  void* out;
  long long q_token, q_head, out_token, out_head;
  int group;       // query heads per kv head
  int window, sinks;
  float scale_log2;
  int workers;
  int row_limit;   // sequences of more rows (tokens x group) are left to another kernel
  int* headers;    // [workers][8]
  float* parts;    // [2 * workers][part_floats]
  int part_floats;
};

// A piece that begins a unit but does not end it: what the join needs.
enum HeaderWord { kHeadPieces = 0, kHeadRow0, kHeadFirst, kHeadHead, kHeadRows };

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint4& a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ void group_sync(int group) {
  asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory");
}

// What a sequence asks for: rows (tokens x group), their 64-token tiles (the
// first `sink_tiles`, then those from `window_tile` on).
struct SeqWork {
  KvSequence q;
  int rows, blocks, tiles, sink_tiles, window_tile;
};

__device__ __forceinline__ SeqWork seq_work(const AttendArgs& a, int s) {
  SeqWork w;
  w.q = kv_sequence(a.v, s);
  const long long rows = static_cast<long long>(w.q.n) * a.group;
  if (rows == 0 || rows > a.row_limit) {
    w.rows = w.blocks = w.tiles = w.sink_tiles = w.window_tile = 0;
    return w;
  }
  w.rows = static_cast<int>(rows);
  w.blocks = (w.rows + kRows - 1) / kRows;
  w.sink_tiles = w.window_tile = 0;
  const int all = (w.q.length + kTileTokens - 1) / kTileTokens;
  if (a.window > 0) {
    const int from = max(max(w.q.first, 0) - a.window + 1, 0);  // first key any row's window has
    w.window_tile = from / kTileTokens;
    const int sinks = min(a.sinks, from);
    w.sink_tiles = min((sinks + kTileTokens - 1) / kTileTokens, w.window_tile);
  }
  w.tiles = max(1, w.sink_tiles + all - w.window_tile);  // rows that see nothing: one, for their zeros
  return w;
}

template <int HSP>
struct GroupSmem {
  static constexpr int kColStride = HSP / 8 + 4;             // floats per n column, padded
  static constexpr int kRowStride = 8 * kColStride + 4;
  uint4 q[HSP / 16][32];
  float o[4][kRows][kRowStride];
  float factor[kRows];
  int pos[kRows];
  float m[4][kRows], l[4][kRows];
};

template <typename T>
__device__ __forceinline__ T to_out(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 to_out<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half to_out<__half>(float v) {
  return __float2half_rn(v);
}

template <int HSP, int kFormat, typename T>
__global__ void __launch_bounds__(kThreads, 1) attend_rows_sm103a_kernel(const AttendArgs a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  __shared__ long long s_prefix[kThreads + 1];
  __shared__ long long s_warp[kThreads / 32];
  GroupSmem<HSP>* groups = reinterpret_cast<GroupSmem<HSP>*>(smem_raw);
  constexpr int kChunks = HSP / 64;       // 16-byte chunks of a K row per lane
  constexpr int kVWords = HSP / 32;       // words of a V row per lane
  constexpr int kTilesN = HSP / 8;        // n-tiles of the output

  grid_dependency_wait();

  // -------------------------------------------------------- the work list --
  // Thread i sums the work of sequences [i c, (i + 1) c); a scan over the CTA
  // gives where each run begins.
  const int S = a.v.sequences;
  const int c = (S + kThreads - 1) / kThreads;
  const int lane = threadIdx.x & 31, warp_id = threadIdx.x >> 5;
  {
    long long mine = 0;
    for (int s = threadIdx.x * c; s < min(S, (static_cast<int>(threadIdx.x) + 1) * c); ++s) {
      const SeqWork w = seq_work(a, s);
      mine += static_cast<long long>(w.blocks) * w.tiles * a.v.heads;
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
  const int worker = blockIdx.x * kGroups + gi;
  const long long share = (total + a.workers - 1) / a.workers;
  long long at = share * worker;
  const long long end = min(at + share, total);
  GroupSmem<HSP>& sm = groups[gi];
  const int g = lane >> 2, t = lane & 3;
  const int D = a.v.head_size;
  int* header = a.headers + worker * 8;
  bool left_open = false;

  int s = 0;
  long long base = 0;
  SeqWork w{};
  if (at < end) {
    int lo = 0, hi = kThreads;  // s_prefix[lo] <= at < s_prefix[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (s_prefix[mid] <= at) lo = mid;
      else hi = mid;
    }
    s = lo * c;
    base = s_prefix[lo];
    w = seq_work(a, s);
  }
  while (at < end) {
    const long long units = static_cast<long long>(w.blocks) * a.v.heads;
    if (at >= base + units * w.tiles) {
      base += units * w.tiles;
      w = seq_work(a, ++s);
      continue;
    }
    const long long off = at - base;
    const int unit = static_cast<int>(off / w.tiles);
    const int tile0 = static_cast<int>(off - static_cast<long long>(unit) * w.tiles);
    const int head = unit / w.blocks;
    const int row_first = (unit - head * w.blocks) * kRows;
    const int rows = min(w.rows - row_first, kRows);
    const int count = static_cast<int>(min(static_cast<long long>(w.tiles - tile0), end - at));
    at += count;

    // ------------------------------------------------------ Q's fragments --
    {
      const int r = gtid >> 3, part = gtid & 7;  // 16 elements of a row
      const int rr = row_first + r;
      const int j = rr / a.group;
      const bool live = r < rows;
      uint4 raw[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
      if (live && part * 16 < D) {
        const uint4* from = reinterpret_cast<const uint4*>(
            static_cast<const T*>(a.q) + (w.q.row0 + j) * a.q_token +
            (head * a.group + (rr - j * a.group)) * a.q_head + part * 16);
        raw[0] = from[0];
        raw[1] = from[1];
      }
      const uint32_t* word = reinterpret_cast<const uint32_t*>(raw);
      uint32_t h[8];
      float back = 1.0f;
      if constexpr (std::is_same<T, __half>::value) {
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = word[i];
      } else {
        float x[16], most = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[2 * i] = __uint_as_float(word[i] << 16);
          x[2 * i + 1] = __uint_as_float(word[i] & 0xFFFF0000u);
          most = fmaxf(most, fmaxf(fabsf(x[2 * i]), fabsf(x[2 * i + 1])));
        }
#pragma unroll
        for (int d = 1; d < 8; d *= 2) most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, d));
        const uint32_t e = max(__float_as_uint(most) >> 23, 15u);
        const float up = __uint_as_float((268u - e) << 23);  // 2^(14 - exponent)
        back = __uint_as_float((e - 14u) << 23);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = half2_of(x[2 * i] * up, x[2 * i + 1] * up);
      }
      if (part * 16 < HSP) {
        // chunk `part` is lane (r % 8, part % 4)'s, in k-steps 4 (part / 4) + 0..3
        const int to = (r & 7) * 4 + (part & 3);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t* f = reinterpret_cast<uint32_t*>(&sm.q[(part >> 2) * 4 + i][to]);
          f[r >> 3] = h[2 * i];
          f[2 + (r >> 3)] = h[2 * i + 1];
        }
      }
      if (part == 0) {
        sm.factor[r] = a.scale_log2 * back;
        sm.pos[r] = live ? w.q.first + j : -1;
      }
    }
    group_sync(gi);
    const float f0 = sm.factor[g], f1 = sm.factor[g + 8];
    const int pos0 = sm.pos[g], pos1 = sm.pos[g + 8];
    const int pos_low = sm.pos[0], pos_high = sm.pos[rows - 1];

    float o[kTilesN][4];
#pragma unroll
    for (int i = 0; i < kTilesN; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
    float m0 = kNegInf, m1 = kNegInf, l0 = 0.0f, l1 = 0.0f;

    uint4 kr[2][kChunks];
    uint32_t vr[4][kVWords];
    float ks = 0.0f, vs = 1.0f;
    // First token of this warp's 16 in step i, and its page (-1: nothing there).
    auto token_of = [&](int i) {
      const int tile = tile0 + i;
      return (tile < w.sink_tiles ? tile : tile - w.sink_tiles + w.window_tile) * kTileTokens +
             warp * 16;
    };
    auto page_of = [&](int i) {
      if (i >= count) return -1;
      const int tb = token_of(i);
      return tb < w.q.length ? kv_page(a.v, s, tb >> a.v.page_shift) : -1;
    };
    auto load_k = [&](int tb, int page) {
      const uint8_t* from = a.v.codes[0] + kv_page_offset(a.v, page, head) +
                            (tb & (a.v.page_tokens - 1)) * D;
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int h = 0; h < kChunks; ++h) {
          const int d = (h * 4 + t) * 16;
          kr[n][h] = d < D ? *reinterpret_cast<const uint4*>(from + (8 * n + g) * D + d)
                           : make_uint4(0, 0, 0, 0);
        }
      ks = a.v.scale[0][static_cast<long long>(page) * a.v.heads + head];
    };
    auto load_v = [&](int tb, int page) {
      const uint8_t* from = a.v.codes[1] + kv_page_offset(a.v, page, head) +
                            (tb & (a.v.page_tokens - 1)) * D + g * (HSP / 8);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint8_t* row = from + (2 * t + (i & 1) + 8 * (i >> 1)) * D;
        const bool in = g * (HSP / 8) < D;
        if constexpr (kVWords == 4) {
          const uint4 x = in ? *reinterpret_cast<const uint4*>(row) : make_uint4(0, 0, 0, 0);
          vr[i][0] = x.x;
          vr[i][1] = x.y;
          vr[i][2] = x.z;
          vr[i][3] = x.w;
        } else {
          const uint2 x = in ? *reinterpret_cast<const uint2*>(row) : make_uint2(0, 0);
          vr[i][0] = x.x;
          vr[i][1] = x.y;
        }
      }
      vs = a.v.scale[1][static_cast<long long>(page) * a.v.heads + head];
    };

    int page = page_of(0), page_next = page_of(1);
    if (page >= 0) {
      load_k(token_of(0), page);
      load_v(token_of(0), page);
    }
    for (int i = 0; i < count; ++i) {
      const int tb = token_of(i);
      const int page_after = page_of(i + 2);
      const bool here = page >= 0;
      uint4 pa = make_uint4(0, 0, 0, 0);
      if (here) {
        float sc[2][4] = {};
#pragma unroll
        for (int h = 0; h < kChunks; ++h)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint4 qa = sm.q[h * 4 + k][lane];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              const uint32_t word = k == 0   ? kr[n][h].x
                                    : k == 1 ? kr[n][h].y
                                    : k == 2 ? kr[n][h].z
                                             : kr[n][h].w;
              uint32_t b0, b1;
              codes4_to_half2x2<kFormat>(word, b0, b1);
              mma_f16(sc[n], qa, b0, b1);
            }
          }
        const float fk0 = f0 * ks, fk1 = f1 * ks;
        const float lv = __log2f(vs), inv = __fdividef(1.0f, vs);
        if (page_next >= 0) load_k(token_of(i + 1), page_next);
        float x[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[n][e] = fmaf(sc[n][e], e < 2 ? fk0 : fk1, lv);
        const bool open = tb + 15 <= pos_low &&
                          (a.window == 0 || pos_high - tb < a.window || tb + 15 < a.sinks);
        if (!open) {
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int tok = tb + 8 * n + 2 * t + (e & 1);
              const int p = e < 2 ? pos0 : pos1;
              if (tok > p || (a.window != 0 && p - tok >= a.window && tok >= a.sinks))
                x[n][e] = kNegInf;
            }
        }
        float mx0 = fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[1][0], x[1][1]));
        float mx1 = fmaxf(fmaxf(x[0][2], x[0][3]), fmaxf(x[1][2], x[1][3]));
        if (__any_sync(0xFFFFFFFFu, mx0 > m0 + kRaise || mx1 > m1 + kRaise)) {
#pragma unroll
          for (int d = 1; d < 4; d *= 2) {
            mx0 = fmaxf(mx0, __shfl_xor_sync(0xFFFFFFFFu, mx0, d));
            mx1 = fmaxf(mx1, __shfl_xor_sync(0xFFFFFFFFu, mx1, d));
          }
          const float n0 = fmaxf(m0, mx0), n1 = fmaxf(m1, mx1);
          const float c0 = n0 == kNegInf ? 1.0f : ex2_approx(m0 - n0);
          const float c1 = n1 == kNegInf ? 1.0f : ex2_approx(m1 - n1);
          m0 = n0;
          m1 = n1;
          l0 *= c0;
          l1 *= c1;
#pragma unroll
          for (int j = 0; j < kTilesN; ++j) {
            o[j][0] *= c0;
            o[j][1] *= c0;
            o[j][2] *= c1;
            o[j][3] *= c1;
          }
        }
        const float z0 = m0 == kNegInf ? 0.0f : m0, z1 = m1 == kNegInf ? 0.0f : m1;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[n][e] = ex2_approx(x[n][e] - (e < 2 ? z0 : z1));
        l0 = fmaf((x[0][0] + x[0][1]) + (x[1][0] + x[1][1]), inv, l0);
        l1 = fmaf((x[0][2] + x[0][3]) + (x[1][2] + x[1][3]), inv, l1);
        pa.x = half2_of(x[0][0], x[0][1]);
        pa.y = half2_of(x[0][2], x[0][3]);
        pa.z = half2_of(x[1][0], x[1][1]);
        pa.w = half2_of(x[1][2], x[1][3]);
        if (tb + 16 > w.q.length) {
          // slots past the sequence's end may hold the codes of no number
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (tb + 2 * t + (k & 1) + 8 * (k >> 1) >= w.q.length) {
#pragma unroll
              for (int j = 0; j < kVWords; ++j) vr[k][j] = 0;
            }
        }
#pragma unroll
        for (int j = 0; j < kVWords; ++j) {
          // four elements of two token pairs: bytes to (token, token + 1) pairs
          uint32_t lo[2], hi[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t u = vr[2 * k][j], v = vr[2 * k + 1][j];
            if (kFormat == CSA_KV_INT8) {
              u ^= 0x80808080u;
              v ^= 0x80808080u;
            }
            lo[k] = byte_perm(u, v, 0x5140);
            hi[k] = byte_perm(u, v, 0x7362);
          }
          uint32_t b[4][2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            if (kFormat == CSA_KV_INT8) {
              b[0][k] = flipped_pair_to_half2<0x4140>(lo[k]);
              b[1][k] = flipped_pair_to_half2<0x4342>(lo[k]);
              b[2][k] = flipped_pair_to_half2<0x4140>(hi[k]);
              b[3][k] = flipped_pair_to_half2<0x4342>(hi[k]);
            } else {
              b[0][k] = e4m3x2_to_half2(lo[k] & 0xFFFFu);
              b[1][k] = e4m3x2_to_half2(lo[k] >> 16);
              b[2][k] = e4m3x2_to_half2(hi[k] & 0xFFFFu);
              b[3][k] = e4m3x2_to_half2(hi[k] >> 16);
            }
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) mma_f16(o[4 * j + k], pa, b[k][0], b[k][1]);
        }
      } else if (page_next >= 0) {
        load_k(token_of(i + 1), page_next);
      }
      if (page_next >= 0) load_v(token_of(i + 1), page_next);
      page = page_next;
      page_next = page_after;
    }

    // ------------------------------------------- the four warps' results --
#pragma unroll
    for (int d = 1; d < 4; d *= 2) {
      l0 += __shfl_xor_sync(0xFFFFFFFFu, l0, d);
      l1 += __shfl_xor_sync(0xFFFFFFFFu, l1, d);
    }
    if (t == 0) {
      sm.m[warp][g] = m0;
      sm.m[warp][g + 8] = m1;
      sm.l[warp][g] = l0;
      sm.l[warp][g + 8] = l1;
    }
    group_sync(gi);
    {
      const float n0 = fmaxf(fmaxf(sm.m[0][g], sm.m[1][g]), fmaxf(sm.m[2][g], sm.m[3][g]));
      const float n1 =
          fmaxf(fmaxf(sm.m[0][g + 8], sm.m[1][g + 8]), fmaxf(sm.m[2][g + 8], sm.m[3][g + 8]));
      const float c0 = n0 == kNegInf ? 1.0f : ex2_approx(m0 - n0);
      const float c1 = n1 == kNegInf ? 1.0f : ex2_approx(m1 - n1);
      // element (n-tile j, column n) is dimension n * HSP / 8 + j
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = g + (e >> 1) * 8;
        if (r >= rows) continue;
        float* to = &sm.o[warp][r][(2 * t + (e & 1)) * GroupSmem<HSP>::kColStride];
        const float cc = e < 2 ? c0 : c1;
#pragma unroll
        for (int j = 0; j < kTilesN; j += 4)
          *reinterpret_cast<float4*>(to + j) = make_float4(o[j][e] * cc, o[j + 1][e] * cc,
                                                           o[j + 2][e] * cc, o[j + 3][e] * cc);
      }
    }
    group_sync(gi);
    const bool whole = tile0 == 0 && count == w.tiles;
    const int slot = 2 * worker + (tile0 == 0 ? 1 : 0);
    float* part = a.parts + static_cast<long long>(slot) * a.part_floats;
    // 128 threads over rows x HSP
    for (int e = gtid; e < rows * HSP; e += 128) {
      const int r = e / HSP, d = e % HSP;
      const int idx = (d / (HSP / 8)) * GroupSmem<HSP>::kColStride + d % (HSP / 8);
      const float mm = fmaxf(fmaxf(sm.m[0][r], sm.m[1][r]), fmaxf(sm.m[2][r], sm.m[3][r]));
      const float acc = (sm.o[0][r][idx] + sm.o[1][r][idx]) + (sm.o[2][r][idx] + sm.o[3][r][idx]);
      float l = 0.0f;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        l += sm.l[k][r] * (mm == kNegInf ? 1.0f : ex2_approx(sm.m[k][r] - mm));
      if (whole) {
        const int rr = row_first + r;
        const int j = rr / a.group;
        if (d < D)
          static_cast<T*>(a.out)[(w.q.row0 + j) * a.out_token +
                                 (head * a.group + (rr - j * a.group)) * a.out_head + d] =
              to_out<T>(l == 0.0f ? 0.0f : acc / l);
      } else {
        part[2 * kRows + r * HSP + d] = acc;
        if (d == 0) {
          part[r] = mm;
          part[kRows + r] = l;
        }
      }
    }
    if (!whole && tile0 == 0) {
      left_open = true;
      if (gtid == 0) {
        header[kHeadPieces] =
            1 + static_cast<int>((w.tiles - count + share - 1) / share);
        header[kHeadRow0] = w.q.row0;
        header[kHeadFirst] = row_first;
        header[kHeadHead] = head;
        header[kHeadRows] = rows;
      }
    }
    group_sync(gi);  // sm is reused
  }
  if (!left_open && gtid == 0) header[kHeadPieces] = 0;
}

// Joins the pieces of each unit that was split: the CTA of the worker whose
// last piece begins the unit. Piece 0 is that worker's second slot, piece i the
// first slot of worker + i. Warp w takes pieces w, w + 4, ...; the four sums
// are added in order.
template <int HSP, typename T>
__global__ void __launch_bounds__(128) attend_join_sm103a_kernel(const AttendArgs a) {
  __shared__ float s_o[4][HSP];
  __shared__ float s_l[4], s_m[4];
  grid_dependency_wait();
  const int worker = blockIdx.x;
  const int* header = a.headers + worker * 8;
  const int pieces = header[kHeadPieces];
  if (pieces == 0) return;
  const int row0 = header[kHeadRow0], first = header[kHeadFirst], head = header[kHeadHead];
  const int rows = header[kHeadRows];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int E = HSP / 32;
  auto part_of = [&](int i) {
    const int slot = i == 0 ? 2 * worker + 1 : 2 * (worker + i);
    return a.parts + static_cast<long long>(slot) * a.part_floats;
  };
  for (int r = 0; r < rows; ++r) {
    float m = kNegInf;
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
      const float c = m == kNegInf ? 1.0f : ex2_approx(p[r] - m);
      l = fmaf(p[kRows + r], c, l);
#pragma unroll
      for (int k = 0; k < E; ++k)
        acc[k] = fmaf(p[2 * kRows + r * HSP + lane * E + k], c, acc[k]);
    }
#pragma unroll
    for (int k = 0; k < E; ++k) s_o[warp][lane * E + k] = acc[k];
    if (lane == 0) s_l[warp] = l;
    __syncthreads();
    const float lt = (s_l[0] + s_l[1]) + (s_l[2] + s_l[3]);
    const int rr = first + r;
    const int j = rr / a.group;
    const int d = threadIdx.x;
    if (d < a.v.head_size)
      static_cast<T*>(a.out)[(row0 + j) * a.out_token +
                             (head * a.group + (rr - j * a.group)) * a.out_head + d] =
          to_out<T>(lt == 0.0f
                        ? 0.0f
                        : ((s_o[0][d] + s_o[1][d]) + (s_o[2][d] + s_o[3][d])) / lt);
    __syncthreads();
  }
}

template <int HSP, int kFormat, typename T>
cudaError_t launch_rows(const AttendArgs& a, int sms, const DeviceInfo& dev, cudaStream_t stream,
                        int& rc, std::string& err) {
  const int smem = static_cast<int>(sizeof(GroupSmem<HSP>)) * kGroups;
  rc = set_max_dynamic_smem(
      reinterpret_cast<const void*>(attend_rows_sm103a_kernel<HSP, kFormat, T>), smem, dev.device,
      err);
  if (rc != CSA_OK) return cudaSuccess;
  cudaError_t e = launch_programmatic(attend_rows_sm103a_kernel<HSP, kFormat, T>,
                                      static_cast<unsigned>(sms), kThreads, smem, stream, a);
  if (e != cudaSuccess) return e;
  return launch_programmatic(attend_join_sm103a_kernel<HSP, T>, static_cast<unsigned>(a.workers),
                             128, 0, stream, a);
}

template <int HSP, int kFormat>
cudaError_t launch_rows_t(int dtype, const AttendArgs& a, int sms, const DeviceInfo& dev,
                          cudaStream_t stream, int& rc, std::string& err) {
  return dtype == CSA_F16 ? launch_rows<HSP, kFormat, __half>(a, sms, dev, stream, rc, err)
                          : launch_rows<HSP, kFormat, __nv_bfloat16>(a, sms, dev, stream, rc, err);
}

int padded_head(int head_size) { return head_size <= 64 ? 64 : 128; }

}  // namespace

size_t cache_attention_workspace_bytes(int head_size) {
  return static_cast<size_t>(kMaxWorkers) * 8 * sizeof(int) +
         static_cast<size_t>(2 * kMaxWorkers) *
             (2 * kRows + kRows * static_cast<size_t>(padded_head(head_size))) * sizeof(float);
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
  a.group = call.q_heads / cache.heads;
  a.window = call.window;
  a.sinks = call.window > 0 ? call.sinks : 0;
  a.scale_log2 = static_cast<float>(static_cast<double>(call.scale) * 1.4426950408889634);
  const int sms = std::min(dev.sm_count, kMaxSms);
  a.workers = sms * kGroups;
  a.row_limit = 0x7FFFFFFF;
  const int hsp = padded_head(cache.head_size);
  a.headers = static_cast<int*>(call.workspace);
  a.parts = reinterpret_cast<float*>(a.headers + kMaxWorkers * 8);
  a.part_floats = 2 * kRows + kRows * hsp;
  int rc = CSA_OK;
  cudaError_t e;
  if (hsp == 64)
    e = cache.format == CSA_KV_INT8
            ? launch_rows_t<64, CSA_KV_INT8>(call.dtype, a, sms, dev, stream, rc, err)
            : launch_rows_t<64, CSA_KV_E4M3>(call.dtype, a, sms, dev, stream, rc, err);
  else
    e = cache.format == CSA_KV_INT8
            ? launch_rows_t<128, CSA_KV_INT8>(call.dtype, a, sms, dev, stream, rc, err)
            : launch_rows_t<128, CSA_KV_E4M3>(call.dtype, a, sms, dev, stream, rc, err);
  if (rc != CSA_OK) {
    err = "cache_attention_forward: " + err;
    return rc;
  }
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) {
    err = std::string("cache_attention_forward: launch: ") + cudaGetErrorString(e);
    return CSA_ERR_LAUNCH;
  }
  return CSA_OK;
}

}  // namespace csa
