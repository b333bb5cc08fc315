// Log probabilities of given tokens, with entropy and the top alternatives, from rows of
// logits x [rows][vocab], and the gradient of what is made of them. With p = softmax(s x):
//
//   logprob = s x[tok] - lse,   lse = s m + log S,   m = max x,  S = sum exp(s (x - m))
//   entropy = -sum p log p = log S - T / S,          T = sum exp(d) d,  d = s (x - m)
//   top: the k largest logits (of equal ones the lowest index), and their log probabilities
//   dx_j = s [ g (1{j = tok} - p_j) - h p_j (log p_j + H) + sum_i g_i (1{j = top_i} - p_j) ]
//
// One pass over the logits: a thread keeps the maximum of what it has seen and S and T
// relative to it, rescaled when the maximum grows (T' = r (T - D S), S' = r S, r = exp(-D)).
// Exponents are worked out as (x - m) c with c = s log2(e), the difference first, which is
// exact near the maximum. All sums are fp32: a thread adds up its chunks' sums (of 4 or 8 weights)
// one after the other, at most 512 of them (a row of 524288 words in fp32; 49 at 50257), which then
// go to a sum of such runs, and the threads' sums make a
// tree. A forbidden word's -inf has weight 0 and adds 0 to T (its d is clamped for the
// product); a NaN or +inf makes its row's results NaN.
//
// Top alternatives without a second pass: the k-th largest of the maxima that four threads have
// between them is a lower bound of the k-th largest logit, and only threads whose own maximum
// reaches it (about k of 256) hold larger ones. Their elements alone are read again, what
// reaches the bound is ranked by counting. Where many threads' maxima tie at the bound, the
// index of their first such element tells them apart.
//
// Bound: HBM, one read of the logits (and one write of the gradient). Short rows have a warp each,
// without barriers (figures below). Else a CTA of 256 threads takes
// a row and four 16-byte loads a thread at once; six such CTAs an SM, so that some load while
// others rank. 8192 x 50257 in fp32 with two alternatives: 244 us (6.6 TB/s, 0.97 of the copy rate; five
// CTAs 253, four 270); in bf16 with the gradient behind it, of five CTAs an SM, 351 us (four 360,
// six 350; a read of the logits beside the gradient's write goes at 6.6 TB/s). Few rows are split
// over a cluster of up to eight CTAs, whose results meet in the first one's shared memory: 48 x
// 50257 in fp32 with five alternatives 8.8 us, a chain of loads, bound, second look and barriers.
//
// A token nearly certain has log p = -log S with S next to 1: right to fp32's half step of 1,
// which is what the sum is held to, not to a part of itself. Leaving the largest element out of
// the sum and log1p of the rest would give that, and cost 8 % of the time with the gradient and
// 15 % of a few rows'.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <string>
#include <type_traits>

#include "csa_internal.h"
#include "kv_cache.cuh"
#include "sm103a_ptx.cuh"

namespace csa {
namespace {

constexpr int kThreads = 256;
constexpr int kForwardPerSm = 6, kBackwardPerSm = 5;  // CTAs an SM
// Each row, or part of one, has a CTA, given to an SM when a place is free there: rows left out
// then keep no place (8192 x 50257 in bf16, a tenth left out: forward 117 us, 134 with rows taken in
// turn by as many CTAs as there are places; backward 232 and 253).
constexpr long long kMostCtas = 1LL << 30;
// A row of so few bytes has a warp: always, or where there are more than kManyRounds rows for every
// place of a CTA. us with a warp / a CTA a row, forward; forward with four alternatives; backward:
//   524288 x 64 bf16     126 / 936     416 / 3666    207 / 1401
//   65536 x 2000 fp32    74 / 172      108 / 330     152 / 248
//   16384 x 8000 bf16    44 / 63       67 / 100      81 / 93
//   16384 x 8000 fp32    73 / 77       110 / 109     154 / 152
//   2000 x 2000 bf16     3.6 / 6.1     7.6 / 14.0    4.7 / 7.6
//   2000 x 8000 bf16     8.0 / 8.9     14.7 / 15.2   10.8 / 10.6
//   100 x 500 fp32       2.1 / 2.3     4.2 / 4.6     2.9 / 2.5
//   1 x 2000 fp32        3.1 / 2.3     6.0 / 4.2     4.4 / 2.5
// Five CTAs of them an SM (524288 x 64 and 16384 x 8000 in bf16, forward: four 137 and 47, six 130
// and 46).
constexpr long long kShortAlways = 2048;  // forward
constexpr long long kShortOfMany = 16384;
constexpr int kManyRounds = 2, kShortPerSm = 5;
constexpr long long kShortRounds = 8;  // CTAs in turn, that rows left out keep few places
constexpr int kWarps = kThreads / 32;
constexpr int kMaxTop = 32;
constexpr int kMaxCluster = 8;
static_assert(kWarps >= kMaxCluster, "a warp for each CTA's list");
constexpr int kLoads = 4;         // 16-byte loads that a thread has in flight
// Chunks of a run: what a thread adds up of them, kRunLoads loads' sums one after the other, goes to a
// sum of runs then.
constexpr int kRunLoads = 512;
constexpr int kRunChunks = kRunLoads * kThreads;
constexpr int kCandidates = 1024; // elements that reach the bound
constexpr int kColumns = 4 * kMaxTop;  // threads whose elements are looked at again
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLeast = -1000.0f;  // exponents below have weight 0; finite, for products with it

template <typename T>
struct Logit;
template <>
struct Logit<float> {
  static constexpr int kVec = 4;
  static __device__ __forceinline__ float get(float v) { return v; }
  static __device__ __forceinline__ float put(float v) { return v; }
  static __device__ __forceinline__ void unpack(const uint4& w, float (&x)[4]) {
    x[0] = __uint_as_float(w.x);
    x[1] = __uint_as_float(w.y);
    x[2] = __uint_as_float(w.z);
    x[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                      __float_as_uint(x[3]));
  }
};
template <>
struct Logit<__nv_bfloat16> {
  static constexpr int kVec = 8;
  static __device__ __forceinline__ float get(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
  static __device__ __forceinline__ void unpack(const uint4& q, float (&x)[8]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Logit<__half> {
  static constexpr int kVec = 8;
  static __device__ __forceinline__ float get(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half put(float v) { return __float2half_rn(v); }
  static __device__ __forceinline__ void unpack(const uint4& q, float (&x)[8]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

struct ForwardArgs {
  const void* logits;
  long long stride;
  long long rows;
  int vocab, top;
  const int* tokens;
  float scale;
  float* logprob;
  float* entropy;
  float2* stats;
  float* top_logprob;
  int* top_token;
  int* status;
  int cluster;  // CTAs of a row
};

// A float as an integer of the same order, zeros alike; NaN counts as -inf. Above 0.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) x = -INFINITY;
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

// What a thread has seen: S and T relative to m, in units of log2.
struct Partial {
  float top = -INFINITY;  // the largest; m = max(top, -FLT_MAX), so that differences from it are numbers
  float m = -FLT_MAX, s = 0.0f, t = 0.0f;

  // S and T relative to a larger maximum.
  __device__ __forceinline__ void raise(float to, float c) {
    const float d = fminf((to - m) * c, 1e30f);  // (finite, so that it times 0 is 0)
    const float r = ex2_approx(-d);
    t = r * fmaf(-d, s, t);
    s *= r;
    m = to;
  }
  template <int N>
  __device__ __forceinline__ void add(const float (&x)[N], float c) {
    float most = x[0];
#pragma unroll
    for (int i = 1; i < N; ++i) most = fmaxf(most, x[i]);
    if (most > m) raise(most, c);
    top = fmaxf(top, most);
    const uint64_t less = pack_f32x2(-m, -m), c2 = pack_f32x2(c, c);
    uint64_t s2 = 0, t2 = 0;
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const uint64_t y = mul_f32x2(add_f32x2(pack_f32x2(x[i], x[i + 1]), less), c2);
      float y0, y1;
      unpack_f32x2(y, y0, y1);
      const uint64_t e = pack_f32x2(ex2_approx(y0), ex2_approx(y1));
      s2 = add_f32x2(s2, e);
      t2 = fma_f32x2(e, pack_f32x2(fmaxf(y0, kLeast), fmaxf(y1, kLeast)), t2);
    }
    float a, b;
    unpack_f32x2(s2, a, b);
    s += a + b;
    unpack_f32x2(t2, a, b);
    t += a + b;
  }
  // This and another's S and T.
  __device__ __forceinline__ void join(Partial q, float c) {
    if (q.m > m) raise(q.m, c);
    else if (m > q.m) q.raise(m, c);
    s += q.s;
    t += q.t;
  }
  __device__ __forceinline__ void add_one(float x, float c) {
    if (x > m) raise(x, c);
    top = fmaxf(top, x);
    const float y = (x - m) * c, e = ex2_approx(y);
    s += e;
    t = fmaf(e, fmaxf(y, kLeast), t);
  }
};

// A run [begin, end) of a row's elements as 16-byte chunks with the elements before the first
// and behind the last.
template <typename T>
struct Run {
  const T* row;
  int begin, end;
  int head, tail;  // elements at begin, and at the end, that belong to no chunk
  int chunks;
  const uint4* body;
  __device__ Run(const T* r, int from, int to) : row(r), begin(from), end(to) {
    constexpr int V = Logit<T>::kVec;
    const int n = to - from;
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(r + from) % 16) / static_cast<int>(sizeof(T));
    head = min(n, off == 0 ? 0 : V - off);
    chunks = (n - head) / V;
    tail = n - head - chunks * V;
    body = reinterpret_cast<const uint4*>(r + from + head);
  }
  // Element index of the i-th that belongs to no chunk.
  __device__ __forceinline__ int loose(int i) const {
    return i < head ? begin + i : begin + head + chunks * Logit<T>::kVec + (i - head);
  }
};

struct alignas(16) Shared {
  float m[kWarps], s[kWarps], t[kWarps];
  float row_m, row_s, row_t;   // of this CTA's part of the row
  uint32_t key[kMaxTop];       // its top alternatives, in order
  int index[kMaxTop];
  int columns[kColumns];       // threads that may hold them
  int count, found;
  uint32_t quads[64];          // the largest of four threads each
  uint32_t bound;
  float3 all[kMaxCluster];     // of every CTA of the row, at its first one
  uint32_t all_key[kMaxCluster][kMaxTop];
  int all_index[kMaxCluster][kMaxTop];
  uint32_t best_key[kWarps];
  int best_index[kWarps];
  union {
    float3 runs[kThreads];  // long rows: what a thread's runs before this one came to
    uint32_t cand_key[kCandidates];  // (once all sums are done)
  };
  int cand_index[kCandidates];
};

// Whether (key, index) comes before (k2, i2).
__device__ __forceinline__ bool before(uint32_t key, int index, uint32_t k2, int i2) {
  return key > k2 || (key == k2 && index < i2);
}

// The k-th largest (or, found sooner, a number that exactly k reach) of the 64 largest `mine` of
// four threads next to each other, by one warp. Between two barriers.
__device__ __forceinline__ uint32_t kth_largest(uint32_t mine, int k, Shared& sh) {
  static_assert(kThreads == 256 && kMaxTop <= 32, "two of them a lane");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t quad = max(mine, __shfl_xor_sync(0xFFFFFFFFu, mine, 1));
  quad = max(quad, __shfl_xor_sync(0xFFFFFFFFu, quad, 2));
  if (lane % 4 == 0) sh.quads[warp * 8 + lane / 4] = quad;
  __syncwarp();
  __syncthreads();
  if (warp == 0) {
    const uint32_t x = sh.quads[lane], y = sh.quads[lane + 32];
    // 32 of them reach the least of the lanes' larger ones
    uint32_t v = __reduce_min_sync(0xFFFFFFFFu, max(x, y));
    uint32_t top = __reduce_max_sync(0xFFFFFFFFu, max(x, y));
    while (v < top) {
      const uint32_t mid = top - (top - v) / 2;
      const int n = __popc(__ballot_sync(0xFFFFFFFFu, x >= mid)) +
                    __popc(__ballot_sync(0xFFFFFFFFu, y >= mid));
      if (n >= k) v = mid;
      else top = mid - 1;
      if (n == k) break;
    }
    if (lane == 0) sh.bound = v;
    __syncwarp();
  }
  __syncthreads();
  return sh.bound;
}

// The k first of the candidates, of which those from `bound` on matter, into sh.key / sh.index.
// Ends in a barrier.
__device__ __forceinline__ void rank_candidates(int k, uint32_t bound, Shared& sh) {
  const int found = sh.found;
  for (int i = threadIdx.x; i < found; i += kThreads) {
    const uint32_t key = sh.cand_key[i];
    const int index = sh.cand_index[i];
    if (key < bound) continue;
    int rank = 0;
    for (int j = 0; j < found; ++j) rank += before(sh.cand_key[j], sh.cand_index[j], key, index);
    if (rank < k) {
      sh.key[rank] = key;
      sh.index[rank] = index;
    }
  }
  __syncwarp();
  __syncthreads();
}

// The k first elements of the CTA's run into sh.key / sh.index (fewer where the run is
// shorter: key 0). `top` is the thread's largest; all threads take part.
template <typename T>
__device__ void select_top(const Run<T>& run, float top, int k, Shared& sh) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int V = Logit<T>::kVec;
  const bool any = tid < run.chunks || tid < run.head + run.tail;
  const uint32_t mine = any ? order_key(top) : 0u;
  if (tid < k) sh.key[tid] = 0, sh.index[tid] = -1;
  if (tid == 0) sh.count = sh.found = 0;
  // (0: fewer than k of them hold elements; then all there are)
  const uint32_t bound = max(kth_largest(mine, k, sh), 1u);
  auto take = [&](bool holds) {
    if (holds) {
      const int at = atomicAdd(&sh.count, 1);
      if (at < kColumns) sh.columns[at] = tid;
    }
    __syncwarp();
    __syncthreads();
  };
  take(mine >= bound);
  // Where many threads tie at the bound: those whose first such element comes first.
  int last = 0x7FFFFFFF;
  if (sh.count > kColumns) {
    int first = run.end;
    if (mine == bound) {
      if (tid < run.head + run.tail) {
        const int i = run.loose(tid);
        if (order_key(Logit<T>::get(run.row[i])) == bound) first = i;
      }
      for (int c = tid, at = run.begin + run.head + tid * V; c < run.chunks && at < first;
           c += kThreads, at += kThreads * V) {
        float x[V];
        Logit<T>::unpack(__ldg(run.body + c), x);
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (order_key(x[i]) == bound) first = min(first, at + i);
      }
    }
    __syncwarp();
    // (threads above the bound count as if theirs were before all)
    const uint32_t left = mine > bound ? run.end - run.begin + 1 : mine == bound ? run.end - first : 0;
    const uint32_t least = max(kth_largest(left, k, sh), 1u);
    last = run.end - static_cast<int>(least);
    if (tid == 0) sh.count = 0;
    __syncwarp();
    __syncthreads();
    take(left >= least);
  }
  // Their elements: an item is a 16-byte chunk of one, or its loose element.
  const int columns = min(sh.count, kColumns);
  const int per = (run.chunks + kThreads - 1) / kThreads + 1, items = columns * per;
  auto for_items = [&](auto f) {
#pragma unroll 2
    for (int i = tid; i < items; i += kThreads) {
      const int column = sh.columns[i / per], n = i % per - 1;
      if (n < 0) {
        if (column < run.head + run.tail) {
          const int e = run.loose(column);
          f(Logit<T>::get(run.row[e]), e);
        }
      } else if (column + n * kThreads < run.chunks) {
        float x[V];
        Logit<T>::unpack(__ldg(run.body + column + n * kThreads), x);
#pragma unroll
        for (int e = 0; e < V; ++e)
          f(x[e], run.begin + run.head + (column + n * kThreads) * V + e);
      }
    }
    __syncwarp();
  };
  for_items([&](float x, int index) {
    const uint32_t key = order_key(x);
    if (key > bound || (key == bound && index <= last)) {
      const int at = atomicAdd(&sh.found, 1);
      if (at < kCandidates) {
        sh.cand_key[at] = key;
        sh.cand_index[at] = index;
      }
    }
  });
  __syncthreads();
  const int found = sh.found;
  if (found <= kCandidates) {
    uint32_t least = 0;
    if (found > 2 * kColumns) {  // (short rows: a bound from all of them is closer)
      uint32_t most = 0;
      for (int i = tid; i < found; i += kThreads) most = max(most, sh.cand_key[i]);
      least = kth_largest(most, k, sh);
    }
    rank_candidates(k, least, sh);
    return;
  }
  // (rare: a few threads hold very many of the largest) one after another
  uint32_t last_key = 0xFFFFFFFFu;
  int last_index = -1;
  for (int n = 0; n < k; ++n) {
    uint32_t key = 0;
    int index = 0x7FFFFFFF;
    for_items([&](float x, int at) {
      const uint32_t q = order_key(x);
      if (before(last_key, last_index, q, at) && before(q, at, key, index)) key = q, index = at;
    });
#pragma unroll
    for (int d = 16; d > 0; d /= 2) {
      const uint32_t q = __shfl_xor_sync(0xFFFFFFFFu, key, d);
      const int at = __shfl_xor_sync(0xFFFFFFFFu, index, d);
      if (before(q, at, key, index)) key = q, index = at;
    }
    if (lane == 0) sh.best_key[warp] = key, sh.best_index[warp] = index;
    __syncthreads();
    key = 0, index = 0x7FFFFFFF;
    for (int w = 0; w < kWarps; ++w)
      if (before(sh.best_key[w], sh.best_index[w], key, index))
        key = sh.best_key[w], index = sh.best_index[w];
    if (tid == 0) sh.key[n] = key, sh.index[n] = key == 0 ? -1 : index;
    last_key = key;
    last_index = index;
    __syncthreads();
  }
}

// kCluster: a row's CTAs are a cluster of a.cluster (else 1). kLong: a CTA's part of a row may be
// more than a run (of 2 MB; apart, as the loop costs others 0.5 %).
template <typename T, bool kTop, bool kCluster, bool kLong>
__global__ void __launch_bounds__(kThreads, kCluster ? 2 : kForwardPerSm)
    logprobs_forward_sm103a_kernel(const ForwardArgs a) {
  __shared__ Shared sh;
  constexpr int V = Logit<T>::kVec;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cluster = kCluster ? a.cluster : 1;
  const int rank = static_cast<int>(blockIdx.x) % cluster;
  const float c = a.scale * kLog2e;
  // This CTA's part of every row: 16-byte multiples but for the last one's end.
  const int each = ((a.vocab + cluster - 1) / cluster + 15) / 16 * 16;
  const int from = min(rank * each, a.vocab), to = min(from + each, a.vocab);
  grid_dependency_wait();
  if constexpr (kCluster) cluster_sync();  // (all have begun before one writes to another)
  for (long long r = blockIdx.x / cluster; r < a.rows; r += gridDim.x / cluster) {
    const int token = a.tokens[r];
    const T* row = static_cast<const T*>(a.logits) + r * a.stride;
    // A row left out takes part as one of no elements: no barrier depends on what is read.
    const bool out = token < 0 || token >= a.vocab;
    // (few rows: the first loads are asked for before the token is there)
    Run<T> run(row, from, !kCluster && out ? from : to);
    uint4 early[kCluster ? kLoads : 1];
    if constexpr (kCluster) {
#pragma unroll
      for (int k = 0; k < kLoads; ++k)
        if (tid + k * kThreads < run.chunks) early[k] = __ldg(run.body + tid + k * kThreads);
      if (out) run.chunks = run.head = run.tail = 0;
    }
    const float given = out ? 0.0f : Logit<T>::get(row[token]);
    Partial p;
    int i = tid;
    for (int end = kLong ? min(run.chunks, kRunChunks) : run.chunks;;
         end = min(run.chunks, end + kRunChunks)) {
      for (; i < end; i += kLoads * kThreads) {
        uint4 w[kLoads];
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
          if (k > 0 && i + k * kThreads >= end) continue;
          if (kCluster && i == tid) w[k] = early[kCluster ? k : 0];
          else w[k] = __ldg(run.body + i + k * kThreads);
        }
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
          if (k > 0 && i + k * kThreads >= end) break;
          float x[V];
          Logit<T>::unpack(w[k], x);
          p.add(x, c);
        }
      }
      if (!kLong || run.chunks <= kRunChunks) break;
      if (end > kRunChunks) {  // with the runs before
        const float3 q = sh.runs[tid];
        Partial before;
        before.m = q.x, before.s = q.y, before.t = q.z;
        p.join(before, c);
      }
      if (end == run.chunks) break;
      sh.runs[tid] = make_float3(p.m, p.s, p.t);
      p.s = p.t = 0.0f;
    }
    if (tid < run.head + run.tail) p.add_one(Logit<T>::get(row[run.loose(tid)]), c);
    __syncwarp();

    // The CTA's maximum, then S and T relative to it.
    float m = p.m;
#pragma unroll
    for (int d = 16; d > 0; d /= 2) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
    if (lane == 0) sh.m[warp] = m;
    __syncthreads();
    m = sh.m[lane % kWarps];
#pragma unroll
    for (int d = kWarps / 2; d > 0; d /= 2) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
    if (m > p.m) p.raise(m, c);
#pragma unroll
    for (int d = 16; d > 0; d /= 2) {
      p.s += __shfl_xor_sync(0xFFFFFFFFu, p.s, d);
      p.t += __shfl_xor_sync(0xFFFFFFFFu, p.t, d);
    }
    if (lane == 0) sh.s[warp] = p.s, sh.t[warp] = p.t;
    __syncthreads();
    if (warp == 0) {
      float s = sh.s[lane % kWarps], t = sh.t[lane % kWarps];
#pragma unroll
      for (int d = kWarps / 2; d > 0; d /= 2) {
        s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
        t += __shfl_xor_sync(0xFFFFFFFFu, t, d);
      }
      if (lane == 0) sh.row_m = m, sh.row_s = s, sh.row_t = t;
    }
    __syncwarp();
    if constexpr (kTop) select_top(run, p.top, a.top, sh);
    else __syncthreads();
    if constexpr (kCluster) {  // to the first CTA of the row
      Shared* first = reinterpret_cast<Shared*>(__cluster_map_shared_rank(&sh, 0));
      if (tid == 0) first->all[rank] = {sh.row_m, sh.row_s, sh.row_t};
      if (kTop && tid < a.top) {
        first->all_key[rank][tid] = sh.key[tid];
        first->all_index[rank][tid] = sh.index[tid];
      }
      __syncwarp();
      cluster_sync();
    }
    if (rank == 0 && ((kCluster && kTop) || warp == 0)) {
      // The row's S and T, from its CTAs' (each warp for itself).
      Partial all;
      if (lane < cluster) {
        const float3 part = kCluster ? sh.all[lane] : make_float3(sh.row_m, sh.row_s, sh.row_t);
        all.m = part.x, all.s = part.y, all.t = part.z;
      }
      __syncwarp();
      float most = all.m;
#pragma unroll
      for (int d = kMaxCluster / 2; d > 0; d /= 2)
        most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, d));
      if (most > all.m) all.raise(most, c);
#pragma unroll
      for (int d = kMaxCluster / 2; d > 0; d /= 2) {
        all.s += __shfl_xor_sync(0xFFFFFFFFu, all.s, d);
        all.t += __shfl_xor_sync(0xFFFFFFFFu, all.t, d);
      }
      const float s = __shfl_sync(0xFFFFFFFFu, all.s, 0), t = __shfl_sync(0xFFFFFFFFu, all.t, 0);
      most = __shfl_sync(0xFFFFFFFFu, most, 0);
      const bool none = s == 0.0f;  // every logit is -inf
      const float log_s = none ? 0.0f : logf(s);
      if (tid == 0) {
        if (token >= a.vocab) report_index(a.status, kIndexToken);
        a.stats[r] = out ? make_float2(0.0f, 0.0f) : make_float2(none ? -INFINITY : most, log_s);
        a.logprob[r] = out ? 0.0f : none ? -INFINITY : fmaf(given - most, a.scale, -log_s);
        a.entropy[r] = none ? 0.0f : log_s - kLn2 * (t / s);
      }
      __syncwarp();
      if constexpr (kTop) {
        const int k = a.top;
        if constexpr (kCluster) {  // the first of the CTAs' alternatives, one a thread
          const bool in = warp < cluster && lane < k;
          const uint32_t key = in ? sh.all_key[warp][lane] : 0u;
          if (tid == 0) sh.found = 0;
          const uint32_t bound = max(kth_largest(key, k, sh), 1u);
          if (key >= bound) {
            const int at = atomicAdd(&sh.found, 1);
            sh.cand_key[at] = key;
            sh.cand_index[at] = sh.all_index[warp][lane];
          }
          __syncwarp();
          __syncthreads();
          rank_candidates(k, 0, sh);
        }
        if (tid < k) {
          const uint32_t key = sh.key[tid];
          if (out || key != 0) {
            a.top_logprob[r * k + tid] = out    ? 0.0f
                                         : none ? -INFINITY
                                                : fmaf(key_value(key) - most, a.scale, -log_s);
            a.top_token[r * k + tid] = out ? -1 : sh.index[tid];
          }
        }
      }
    }
    __syncwarp();
    if constexpr (kCluster) cluster_sync();  // the next row's part overwrites what was read
    else __syncthreads();
  }
}

// (as many as a row has whose chunks leave a lane without: 31 of 8 words and 14 loose ones are 262)
constexpr int kShortCandidates = 288;

struct alignas(16) ShortShared {
  uint32_t key[kShortCandidates];
  int index[kShortCandidates];
  int columns[32];  // lanes whose elements are looked at again
  int found;
};

// The k first elements of a short row, by one warp: lane i has the i-th's key and index (key 0: the
// row has fewer). `top` is the lane's largest.
template <typename T>
__device__ void select_short(const Run<T>& run, float top, int k, ShortShared& sh, uint32_t& my_key,
                             int& my_index) {
  constexpr int V = Logit<T>::kVec;
  const int lane = threadIdx.x & 31;
  const bool any = lane < run.chunks || lane < run.head + run.tail;
  const uint32_t mine = any ? order_key(top) : 0u;
  // k lanes reach the k-th largest of the lanes' maxima (0: fewer than k hold elements)
  uint32_t bound = __reduce_min_sync(0xFFFFFFFFu, mine), most = __reduce_max_sync(0xFFFFFFFFu, mine);
  while (bound < most) {
    const uint32_t mid = most - (most - bound) / 2;
    const int n = __popc(__ballot_sync(0xFFFFFFFFu, mine >= mid));
    if (n >= k) bound = mid;
    else most = mid - 1;
    if (n == k) break;
  }
  bound = max(bound, 1u);
  // Their elements, dealt out to all lanes: an item is a 16-byte chunk of one, or its loose element.
  const uint32_t holds = __ballot_sync(0xFFFFFFFFu, mine >= bound);
  if (holds >> lane & 1u) sh.columns[__popc(holds & ((1u << lane) - 1))] = lane;
  const int per = (run.chunks + 31) / 32 + 1, items = __popc(holds) * per;
  auto for_elements = [&](auto f) {
    if (run.chunks <= 32) {  // (no lane has two: each its own, 416 us of 524288 x 64 bf16; dealt 457)
      if (mine >= bound) {
        if (lane < run.head + run.tail) {
          const int e = run.loose(lane);
          f(Logit<T>::get(run.row[e]), e);
        }
        if (lane < run.chunks) {
          float x[V];
          Logit<T>::unpack(__ldg(run.body + lane), x);
#pragma unroll
          for (int e = 0; e < V; ++e) f(x[e], run.begin + run.head + lane * V + e);
        }
      }
      __syncwarp();
      return;
    }
#pragma unroll 2
    for (int i = lane; i < items; i += 32) {
      const int column = sh.columns[i / per], n = i % per - 1;
      if (n < 0) {
        if (column < run.head + run.tail) {
          const int e = run.loose(column);
          f(Logit<T>::get(run.row[e]), e);
        }
      } else if (column + n * 32 < run.chunks) {
        float x[V];
        Logit<T>::unpack(__ldg(run.body + column + n * 32), x);
#pragma unroll
        for (int e = 0; e < V; ++e) f(x[e], run.begin + run.head + (column + n * 32) * V + e);
      }
    }
    __syncwarp();
  };
  if (lane == 0) sh.found = 0;
  __syncwarp();
  for_elements([&](float x, int index) {
    const uint32_t key = order_key(x);
    if (key >= bound) {
      const int at = atomicAdd(&sh.found, 1);
      if (at < kShortCandidates) sh.key[at] = key, sh.index[at] = index;
    }
  });
  const int found = sh.found;
  my_key = 0;
  my_index = -1;
  uint32_t key = 0;  // the lane's first that is left
  int index = 0x7FFFFFFF;
  uint32_t last_key = 0xFFFFFFFFu;
  int last_index = -1;
  auto look = [&](uint32_t q, int at) {
    if (before(last_key, last_index, q, at) && before(q, at, key, index)) key = q, index = at;
  };
  for (int n = 0; n < k; ++n) {
    if (n == 0 || (key == last_key && index == last_index)) {
      key = 0, index = 0x7FFFFFFF;
      if (found <= kShortCandidates)
        for (int i = lane; i < found; i += 32) look(sh.key[i], sh.index[i]);
    }
    __syncwarp();
    // (rare: ties at the bound, or few lanes hold very many of the largest) the row once more
    if (found > kShortCandidates) {
      key = 0, index = 0x7FFFFFFF;
      for_elements([&](float x, int at) { look(order_key(x), at); });
    }
    last_key = __reduce_max_sync(0xFFFFFFFFu, key);
    last_index = static_cast<int>(__reduce_min_sync(
        0xFFFFFFFFu, key == last_key ? static_cast<unsigned>(index) : 0x7FFFFFFFu));
    if (lane == n) my_key = last_key, my_index = last_key == 0 ? -1 : last_index;
  }
}

// A warp a row.
template <typename T, bool kTop>
__global__ void __launch_bounds__(kThreads, kShortPerSm)
    logprobs_forward_short_sm103a_kernel(const ForwardArgs a) {
  __shared__ ShortShared sh[kTop ? kWarps : 1];
  constexpr int V = Logit<T>::kVec;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float c = a.scale * kLog2e;
  grid_dependency_wait();
  for (long long r = static_cast<long long>(blockIdx.x) * kWarps + warp; r < a.rows;
       r += static_cast<long long>(gridDim.x) * kWarps) {
    const int token = __shfl_sync(0xFFFFFFFFu, a.tokens[r], 0);  // (one for all lanes)
    const T* row = static_cast<const T*>(a.logits) + r * a.stride;
    const bool out = token < 0 || token >= a.vocab;
    const Run<T> run(row, 0, out ? 0 : a.vocab);
    const float given = out ? 0.0f : Logit<T>::get(row[token]);
    Partial p;
    for (int i = lane; i < run.chunks; i += kLoads * 32) {
      uint4 w[kLoads];
#pragma unroll
      for (int k = 0; k < kLoads; ++k)
        if (k == 0 || i + k * 32 < run.chunks) w[k] = __ldg(run.body + i + k * 32);
#pragma unroll
      for (int k = 0; k < kLoads; ++k) {
        if (k > 0 && i + k * 32 >= run.chunks) break;
        float x[V];
        Logit<T>::unpack(w[k], x);
        p.add(x, c);
      }
    }
    if (lane < run.head + run.tail) p.add_one(Logit<T>::get(row[run.loose(lane)]), c);
    __syncwarp();
    float m = p.m;
#pragma unroll
    for (int d = 16; d > 0; d /= 2) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
    if (m > p.m) p.raise(m, c);
#pragma unroll
    for (int d = 16; d > 0; d /= 2) {
      p.s += __shfl_xor_sync(0xFFFFFFFFu, p.s, d);
      p.t += __shfl_xor_sync(0xFFFFFFFFu, p.t, d);
    }
    const bool none = p.s == 0.0f;  // every logit is -inf
    const float log_s = none ? 0.0f : logf(p.s);
    if (lane == 0) {
      if (token >= a.vocab) report_index(a.status, kIndexToken);
      a.stats[r] = out ? make_float2(0.0f, 0.0f) : make_float2(none ? -INFINITY : m, log_s);
      a.logprob[r] = out ? 0.0f : none ? -INFINITY : fmaf(given - m, a.scale, -log_s);
      a.entropy[r] = none ? 0.0f : log_s - kLn2 * (p.t / p.s);
    }
    __syncwarp();
    if constexpr (kTop) {
      uint32_t key = 0;
      int index = -1;
      if (!out) select_short(run, p.top, a.top, sh[warp], key, index);
      if (lane < a.top && (out || key != 0)) {
        a.top_logprob[r * a.top + lane] = out    ? 0.0f
                                          : none ? -INFINITY
                                                 : fmaf(key_value(key) - m, a.scale, -log_s);
        a.top_token[r * a.top + lane] = index;
      }
      __syncwarp();
    }
  }
}

struct BackwardArgs {
  const void* logits;
  void* dlogits;
  long long stride, d_stride;
  long long rows;
  int vocab, top;
  const int* tokens;
  float scale;
  const float2* stats;
  const float* entropy;
  const float* d_logprob;  // or nullptr, as the next two
  const float* d_entropy;
  const float* d_top;
  const int* top_token;
  int* status;
  int parts;  // CTAs of a row
};

// -s p (g + h (log p + H)) of a logit, with z = log2 p: p (A + B z).
struct Slope {
  float m, c, log2_s, A, B;
  __device__ __forceinline__ float operator()(float x) const {
    const float z = (x - m) * c - log2_s;
    return ex2_approx(z) * fmaf(B, fmaxf(z, kLeast), A);
  }
};

// kVector: rows of logits and gradient begin at the same place of a 16-byte chunk.
template <typename T, bool kVector>
__global__ void __launch_bounds__(kThreads, kBackwardPerSm)
    logprobs_backward_sm103a_kernel(const BackwardArgs a) {
  __shared__ int s_at[kMaxTop + 1];    // the token and the alternatives
  __shared__ float s_g[kMaxTop + 1];
  constexpr int V = Logit<T>::kVec;
  const int tid = threadIdx.x;
  const int each = ((a.vocab + a.parts - 1) / a.parts + 15) / 16 * 16;
  grid_dependency_wait();
  for (long long job = blockIdx.x; job < a.rows * a.parts; job += gridDim.x) {
    const long long r = job / a.parts;
    const int from = min(static_cast<int>(job - r * a.parts) * each, a.vocab);
    const int to = min(from + each, a.vocab);
    const T* row = static_cast<const T*>(a.logits) + r * a.stride;
    T* drow = static_cast<T*>(a.dlogits) + r * a.d_stride;
    const Run<T> run(row, from, to);
    const int token = a.tokens[r];
    const float2 st = a.stats[r];
    const int k = a.d_top ? a.top : 0;
    const bool out = token < 0 || token >= a.vocab;
    if (out && token >= 0 && tid == 0 && from == 0) report_index(a.status, kIndexToken);
    const bool zero = out || st.x == -INFINITY;  // left out, or no logit above -inf
    __syncwarp();
    if (tid == 0) {
      s_at[0] = token;
      s_g[0] = a.d_logprob ? a.d_logprob[r] : 0.0f;
    } else if (tid <= k) {
      const int t = a.top_token[r * a.top + tid - 1];
      s_at[tid] = t;
      s_g[tid] = a.d_top[r * a.top + tid - 1];
      if (!out && (t < 0 || t >= a.vocab)) {
        report_index(a.status, kIndexToken);
        s_g[tid] = 0.0f;
      }
    }
    __syncwarp();
    __syncthreads();
    float g = 0.0f;
    for (int i = 0; i <= k; ++i) g += s_g[i];
    const float h = a.d_entropy ? a.d_entropy[r] : 0.0f;
    Slope f;
    f.m = st.x;
    f.c = a.scale * kLog2e;
    f.log2_s = st.y * kLog2e;
    f.A = -a.scale * fmaf(h, h != 0.0f ? a.entropy[r] : 0.0f, g);
    f.B = -a.scale * h * kLn2;
    // The elements with a weight of their own: thread i the i-th, unless an earlier one is the same.
    bool special = false;
    float d_special = 0.0f;
    int at = -1;
    if (tid <= k && !zero) {
      at = s_at[tid];
      special = at >= from && at < to;
      float own = 0.0f;
      for (int i = 0; i <= k; ++i)
        if (s_at[i] == at) {
          if (i < tid) special = false;
          own += s_g[i];
        }
      if (special) d_special = fmaf(a.scale, own, f(Logit<T>::get(row[at])));
    }
    __syncwarp();
    __syncthreads();  // (before the gradient takes the logits' place)
    if constexpr (kVector) {
      uint4* to_body = reinterpret_cast<uint4*>(drow + (reinterpret_cast<const T*>(run.body) - row));
      int i = tid;
      for (; i < run.chunks; i += kLoads * kThreads) {
        uint4 w[kLoads];
#pragma unroll
        for (int n = 0; n < kLoads; ++n)
          if (!zero && i + n * kThreads < run.chunks) w[n] = run.body[i + n * kThreads];
#pragma unroll
        for (int n = 0; n < kLoads; ++n) {
          if (i + n * kThreads >= run.chunks) break;
          float x[V];
          if (zero) {
            to_body[i + n * kThreads] = make_uint4(0, 0, 0, 0);
          } else {
            Logit<T>::unpack(w[n], x);
#pragma unroll
            for (int e = 0; e < V; ++e) x[e] = f(x[e]);
            to_body[i + n * kThreads] = Logit<T>::pack(x);
          }
        }
      }
      if (tid < run.head + run.tail) {
        const int e = run.loose(tid);
        drow[e] = Logit<T>::put(zero ? 0.0f : f(Logit<T>::get(row[e])));
      }
    } else {
      for (int e = from + tid; e < to; e += kThreads)
        drow[e] = Logit<T>::put(zero ? 0.0f : f(Logit<T>::get(row[e])));
    }
    __syncwarp();
    __syncthreads();
    if (special) drow[at] = Logit<T>::put(d_special);
  }
}

// A warp a row.
template <typename T, bool kVector>
__global__ void __launch_bounds__(kThreads, kShortPerSm)
    logprobs_backward_short_sm103a_kernel(const BackwardArgs a) {
  __shared__ int s_at[kWarps][kMaxTop + 1];  // the token and the alternatives
  __shared__ float s_g[kWarps][kMaxTop + 1];
  constexpr int V = Logit<T>::kVec;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int k = a.d_top ? a.top : 0;
  int* const at = s_at[warp];
  float* const own = s_g[warp];
  grid_dependency_wait();
  for (long long r = static_cast<long long>(blockIdx.x) * kWarps + warp; r < a.rows;
       r += static_cast<long long>(gridDim.x) * kWarps) {
    const T* row = static_cast<const T*>(a.logits) + r * a.stride;
    T* drow = static_cast<T*>(a.dlogits) + r * a.d_stride;
    const Run<T> run(row, 0, a.vocab);
    const int token = __shfl_sync(0xFFFFFFFFu, a.tokens[r], 0);
    const float2 st = a.stats[r];
    const bool out = token < 0 || token >= a.vocab;
    const bool zero = out || st.x == -INFINITY;  // left out, or no logit above -inf
    if (out && token >= 0 && lane == 0) report_index(a.status, kIndexToken);
    for (int i = lane; i <= k; i += 32) {
      int t = token;
      float g = 0.0f;
      if (i == 0) {
        if (a.d_logprob) g = a.d_logprob[r];
      } else {
        t = a.top_token[r * a.top + i - 1];
        g = a.d_top[r * a.top + i - 1];
        if (!out && (t < 0 || t >= a.vocab)) {
          report_index(a.status, kIndexToken);
          g = 0.0f;
        }
      }
      at[i] = t;
      own[i] = g;
    }
    __syncwarp();
    float g = 0.0f;
    for (int i = 0; i <= k; ++i) g += own[i];
    const float h = a.d_entropy ? a.d_entropy[r] : 0.0f;
    Slope f;
    f.m = st.x;
    f.c = a.scale * kLog2e;
    f.log2_s = st.y * kLog2e;
    f.A = -a.scale * fmaf(h, h != 0.0f ? a.entropy[r] : 0.0f, g);
    f.B = -a.scale * h * kLn2;
    // The elements with a weight of their own, as above: lane i the i-th, lane 0 the last of 33 too.
    int where[2] = {-1, -1};
    float special[2] = {0.0f, 0.0f};
    if (!zero) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int n = lane + 32 * j;
        if (n > k) continue;
        const int e = at[n];
        bool first = e >= 0 && e < a.vocab;
        float sum = 0.0f;
        for (int i = 0; i <= k; ++i)
          if (at[i] == e) {
            if (i < n) first = false;
            sum += own[i];
          }
        if (first) {
          where[j] = e;
          special[j] = fmaf(a.scale, sum, f(Logit<T>::get(row[e])));
        }
      }
    }
    __syncwarp();  // (before the gradient takes the logits' place)
    if constexpr (kVector) {
      uint4* to_body = reinterpret_cast<uint4*>(drow + (reinterpret_cast<const T*>(run.body) - row));
      for (int i = lane; i < run.chunks; i += kLoads * 32) {
        uint4 w[kLoads];
#pragma unroll
        for (int n = 0; n < kLoads; ++n)
          if (!zero && i + n * 32 < run.chunks) w[n] = run.body[i + n * 32];
#pragma unroll
        for (int n = 0; n < kLoads; ++n) {
          if (i + n * 32 >= run.chunks) break;
          if (zero) {
            to_body[i + n * 32] = make_uint4(0, 0, 0, 0);
          } else {
            float x[V];
            Logit<T>::unpack(w[n], x);
#pragma unroll
            for (int e = 0; e < V; ++e) x[e] = f(x[e]);
            to_body[i + n * 32] = Logit<T>::pack(x);
          }
        }
      }
      if (lane < run.head + run.tail) {
        const int e = run.loose(lane);
        drow[e] = Logit<T>::put(zero ? 0.0f : f(Logit<T>::get(row[e])));
      }
    } else {
      for (int e = lane; e < a.vocab; e += 32)
        drow[e] = Logit<T>::put(zero ? 0.0f : f(Logit<T>::get(row[e])));
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (where[j] >= 0) drow[where[j]] = Logit<T>::put(special[j]);
    __syncwarp();
  }
}

bool many_rows(long long rows, const DeviceInfo& dev) {
  return rows > static_cast<long long>(kManyRounds) * kForwardPerSm * dev.sm_count;
}
unsigned short_grid(long long rows, const DeviceInfo& dev) {
  const long long most = static_cast<long long>(kShortPerSm) * dev.sm_count;
  return static_cast<unsigned>(
      std::min((rows + kWarps - 1) / kWarps, dev.limited ? most : kShortRounds * most));
}

template <typename T>
cudaError_t launch_forward(ForwardArgs a, const DeviceInfo& dev, cudaStream_t stream) {
  const long long bytes = static_cast<long long>(a.vocab) * static_cast<long long>(sizeof(T));
  if (bytes <= kShortAlways || (bytes <= kShortOfMany && many_rows(a.rows, dev)))
    return launch_programmatic(a.top > 0 ? logprobs_forward_short_sm103a_kernel<T, true>
                                         : logprobs_forward_short_sm103a_kernel<T, false>,
                               dim3(short_grid(a.rows, dev)), kThreads, 0, stream, a);
  // CTAs of a row: as many as leave each 16 KB of it, while there are SMs without work.
  a.cluster = 1;
  while (a.cluster < kMaxCluster && a.rows * a.cluster < dev.sm_count &&
         bytes / (2 * a.cluster) >= 8192)
    a.cluster *= 2;
  const int per_sm = a.cluster > 1 ? 2 : kForwardPerSm;
  const long long most = a.cluster == 1 && !dev.limited
                             ? kMostCtas
                             : std::max(per_sm * dev.sm_count / a.cluster, 1);
  const unsigned grid = static_cast<unsigned>(std::min(a.rows, most) * a.cluster);
  const bool is_long = bytes / a.cluster >= 16LL * kRunChunks;
  auto launch = [&](auto top, auto l) {
    constexpr bool kTop = decltype(top)::value, kLong = decltype(l)::value;
    return a.cluster > 1
               ? launch_programmatic_cluster(logprobs_forward_sm103a_kernel<T, kTop, true, kLong>, grid,
                                             kThreads, 0, stream, static_cast<unsigned>(a.cluster), a)
               : launch_programmatic(logprobs_forward_sm103a_kernel<T, kTop, false, kLong>, dim3(grid),
                                     kThreads, 0, stream, a);
  };
  using Yes = std::true_type;
  using No = std::false_type;
  return a.top > 0 ? is_long ? launch(Yes{}, Yes{}) : launch(Yes{}, No{})
                   : is_long ? launch(No{}, Yes{}) : launch(No{}, No{});
}

template <typename T>
cudaError_t launch_backward(BackwardArgs a, const DeviceInfo& dev, cudaStream_t stream) {
  const long long bytes = static_cast<long long>(a.vocab) * static_cast<long long>(sizeof(T));
  const bool vector =
      reinterpret_cast<uintptr_t>(a.logits) % 16 == reinterpret_cast<uintptr_t>(a.dlogits) % 16 &&
      (a.rows == 1 || (a.stride - a.d_stride) * static_cast<long long>(sizeof(T)) % 16 == 0);
  if (bytes <= kShortOfMany && many_rows(a.rows, dev))
    return launch_programmatic(vector ? logprobs_backward_short_sm103a_kernel<T, true>
                                      : logprobs_backward_short_sm103a_kernel<T, false>,
                               dim3(short_grid(a.rows, dev)), kThreads, 0, stream, a);
  a.parts = 1;
  const long long most = static_cast<long long>(kBackwardPerSm) * dev.sm_count;
  while (a.rows * a.parts < most && bytes / (2 * a.parts) >= 8192) a.parts *= 2;
  const unsigned grid =
      static_cast<unsigned>(std::min(a.rows * a.parts, dev.limited ? most : kMostCtas));
  const auto kernel = vector ? logprobs_backward_sm103a_kernel<T, true>
                             : logprobs_backward_sm103a_kernel<T, false>;
  return launch_programmatic(kernel, dim3(grid), kThreads, 0, stream, a);
}

int launched(const char* who, cudaError_t e, std::string& err) {
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e == cudaSuccess) return CSA_OK;
  err = std::string(who) + ": launch: " + cudaGetErrorString(e);
  return CSA_ERR_LAUNCH;
}

}  // namespace

int logprobs_forward_launch(const LogprobsCall& c, cudaStream_t stream, const DeviceInfo& dev,
                            std::string& err) {
  ForwardArgs a;
  a.logits = c.logits;
  a.stride = c.stride;
  a.rows = c.rows;
  a.vocab = c.vocab;
  a.top = c.top;
  a.tokens = c.tokens;
  a.scale = c.scale;
  a.logprob = c.logprob;
  a.entropy = c.entropy;
  a.stats = reinterpret_cast<float2*>(c.stats);
  a.top_logprob = c.top_logprob;
  a.top_token = c.top_token;
  a.status = dev.status_word;
  const cudaError_t e = c.dtype == CSA_F32   ? launch_forward<float>(a, dev, stream)
                        : c.dtype == CSA_F16 ? launch_forward<__half>(a, dev, stream)
                                             : launch_forward<__nv_bfloat16>(a, dev, stream);
  return launched("token_logprobs_forward", e, err);
}

int logprobs_backward_launch(const LogprobsGrad& c, cudaStream_t stream, const DeviceInfo& dev,
                             std::string& err) {
  BackwardArgs a;
  a.logits = c.logits;
  a.dlogits = c.dlogits;
  a.stride = c.stride;
  a.d_stride = c.d_stride;
  a.rows = c.rows;
  a.vocab = c.vocab;
  a.top = c.top;
  a.tokens = c.tokens;
  a.scale = c.scale;
  a.stats = reinterpret_cast<const float2*>(c.stats);
  a.entropy = c.entropy;
  a.d_logprob = c.d_logprob;
  a.d_entropy = c.d_entropy;
  a.d_top = c.d_top;
  a.top_token = c.top_token;
  a.status = dev.status_word;
  const cudaError_t e = c.dtype == CSA_F32   ? launch_backward<float>(a, dev, stream)
                        : c.dtype == CSA_F16 ? launch_backward<__half>(a, dev, stream)
                                             : launch_backward<__nv_bfloat16>(a, dev, stream);
  return launched("token_logprobs_backward", e, err);
}

}  // namespace csa
