// The books of a paged cache: which pages each sequence has, and how many name each page.
// A page is free when its count is 0; free ones are given out lowest first, in the order of a
// call's entries, so a call's result does not depend on how it is scheduled.
//
//   extend   rank of an entry = pages that the entries before it want; its pages are the free
//            ones of ranks [rank, rank + want)
//   fork     whole pages are shared (their counts grow), the written part of a last one is
//            copied to a page of its own, so that no shared page is ever written again
//   compact  with n pages in use, the m free pages below n and the m used ones from n on, both
//            in ascending order, are paired, and the latter move into the former
//
// Two or three launches. The first turns the counts into a bit a page (set: free) and counts
// them by chunks, at most 1024 of them, while one CTA works out the entries' ranks. In the
// second every CTA sums the chunks for itself and finds the page of a rank by bisection over
// the chunks and a walk over one chunk's words: nothing waits for another CTA. Compacting lists
// its moves in the second launch and makes them in the third.
//
// Bound: the copies by HBM (a job is 16 KB of one page, four 16-byte loads a thread, eight CTAs
// an SM, given out one by one; 280 MB that compacting moves take 90 us, 6.2 TB/s), the rest by
// launches and dependent loads: 24 sequences' end, 256 forks of 32 prompts and room for 352 more
// are five launches and 21 us. One launch of one CTA for calls of few entries, and a second launch
// begun before the first one's end, took no less.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>
#include <string>

#include "csa_internal.h"
#include "kv_cache.cuh"
#include "sm103a_ptx.cuh"

namespace csa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPlanThreads = 1024;
constexpr int kMaxChunks = 1024;
constexpr int kChunkPages = 1024;    // a chunk's pages, doubled until there are few enough chunks
constexpr int kJobBytes = 16384;     // of a page, copied by a CTA at once
constexpr int kCopyPerSm = 8;        // CTAs an SM
constexpr int kForkPieceBytes = 32768;

// The device's view of csa_kv_pages.
struct Books {
  int* refs;     // [pages]
  int* lengths;  // [sequences]
  int* table;    // [sequences][width]
  int pages, sequences, width, page_tokens, shift;
  int* status;
};

// What an entry of a call asks for, worked out once.
struct Entry {
  int sequence;    // -1: left out
  int parent;      // fork
  int old_tokens;  // extend: before
  int tokens;      // after
  int rank, want;
};

struct Scan {
  uint32_t* bits;  // [words]: a set bit is a free page
  int* free_in;    // [chunks]
  int* wanted;     // compact: the number of moves
  unsigned long long* taken;  // compact: jobs that CTAs have taken beside their first ones
  int* claims;     // [sequences]
  Entry* entries;
  int* movers;     // [pages] compact: the pages that move, in order
  int chunks, chunk_pages;
};

struct EntryArgs {
  Books b;
  Scan s;
  const int* sequences;  // extend: sequences; fork: children
  const int* parents;    // fork
  const int* tokens;     // extend: more; fork: how many, or nullptr: all
  int n;
  bool fork;
};

__device__ __forceinline__ int blocks_of(const Books& b, int tokens) {
  return static_cast<int>((static_cast<long long>(tokens) + b.page_tokens - 1) >> b.shift);
}
__device__ __forceinline__ bool length_ok(const Books& b, int tokens) {
  return tokens >= 0 && tokens <= static_cast<long long>(b.width) * b.page_tokens;
}

// CTA 0: the entries' ranks. An entry that breaks the rules, or whose sequence an earlier one has
// taken, wants nothing.
__device__ void plan_entries(const EntryArgs& a) {
  __shared__ long long s_warp[kPlanThreads / 32];
  const Books& b = a.b;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto in = [&](int s) { return s >= 0 && s < b.sequences; };
  for (int i = tid; i < a.n; i += kPlanThreads) {
    const int s = a.sequences[i];
    if (in(s)) a.s.claims[s] = INT_MAX;
  }
  __syncthreads();
  for (int i = tid; i < a.n; i += kPlanThreads) {
    const int s = a.sequences[i];
    if (in(s)) atomicMin(a.s.claims + s, i);
  }
  __syncthreads();
  long long base = 0;
  for (int i0 = 0; i0 < a.n; i0 += kPlanThreads) {
    const int i = i0 + tid;
    Entry e{-1, -1, 0, 0, 0, 0};
    if (i < a.n) {
      const int s = a.sequences[i];
      bool ok = in(s) && *const_cast<volatile int*>(a.s.claims + s) == i;
      bool length = true;
      if (ok) {
        const int have = b.lengths[s];
        if (a.fork) {
          const int p = a.parents[i];
          ok = in(p) && p != s;
          if (ok) {
            const int all = b.lengths[p];
            e.tokens = a.tokens ? a.tokens[i] : all;
            length = length_ok(b, all) && e.tokens >= 0 && e.tokens <= all && have == 0;
            e.parent = p;
            e.want = (e.tokens & (b.page_tokens - 1)) != 0;
          }
        } else {
          const int more = a.tokens[i];
          length = length_ok(b, have) && more >= 0 && more <= INT_MAX - max(have, 0) &&
                   more <= static_cast<long long>(b.width) * b.page_tokens - have;
          if (length) {
            e.old_tokens = have;
            e.tokens = have + more;
            e.want = blocks_of(b, e.tokens) - blocks_of(b, have);
          }
        }
      }
      if (ok && length) {
        e.sequence = s;
      } else {
        e.want = 0;
        report_index(b.status, ok ? kIndexLength : kIndexSequence);
      }
    }
    __syncwarp();
    long long sum = e.want;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const long long up = __shfl_up_sync(0xFFFFFFFFu, sum, d);
      if (lane >= d) sum += up;
    }
    if (lane == 31) s_warp[warp] = sum;
    __syncthreads();
    long long before = base;
    for (int w = 0; w < warp; ++w) before += s_warp[w];
    for (int w = 0; w < kPlanThreads / 32; ++w) base += s_warp[w];
    e.rank = static_cast<int>(min(before + sum - e.want, static_cast<long long>(INT_MAX)));
    if (i < a.n) a.s.entries[i] = e;
    __syncthreads();
  }
}

// CTAs from 1 on: a warp a chunk, its free pages as bits and their number.
__global__ void __launch_bounds__(kPlanThreads, 1) pages_scan_sm103a_kernel(const EntryArgs a) {
  grid_dependency_wait();
  if (blockIdx.x == 0) {
    if (a.n > 0) plan_entries(a);
    return;
  }
  const int lane = threadIdx.x & 31;
  const int warps = static_cast<int>(gridDim.x - 1) * (kPlanThreads / 32);
  for (int c = (blockIdx.x - 1) * (kPlanThreads / 32) + (threadIdx.x >> 5); c < a.s.chunks; c += warps) {
    int count = 0;
    const long long first = static_cast<long long>(c) * a.s.chunk_pages;
    for (int w = 0; w < a.s.chunk_pages / 32; w += 8) {
      int r[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const long long p = first + (w + i) * 32 + lane;
        r[i] = p < a.b.pages ? a.b.refs[p] : 1;
      }
      uint32_t mine = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t word = __ballot_sync(0xFFFFFFFFu, r[i] == 0);
        count += __popc(word);
        if (lane == i) mine = word;
      }
      if (lane < 8) a.s.bits[first / 32 + w + lane] = mine;
    }
    if (lane == 0) a.s.free_in[c] = count;
  }
}

// Free pages before each chunk, summed by every CTA for itself.
struct FreeList {
  int before[kMaxChunks + 1];
  int warp[kWarps];

  __device__ void sum(const Scan& s) {
    const int tid = threadIdx.x, lane = tid & 31;
    constexpr int kEach = kMaxChunks / kThreads;
    int mine[kEach], total = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int c = tid * kEach + i;
      mine[i] = c < s.chunks ? s.free_in[c] : 0;
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) total += mine[i];
    int up = total;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int x = __shfl_up_sync(0xFFFFFFFFu, up, d);
      if (lane >= d) up += x;
    }
    if (lane == 31) warp[tid >> 5] = up;
    __syncthreads();
    int at = up - total;
    for (int w = 0; w < (tid >> 5); ++w) at += warp[w];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      before[tid * kEach + i] = at;
      at += mine[i];
    }
    if (tid == kThreads - 1) before[kMaxChunks] = at;
    __syncthreads();
  }
  __device__ __forceinline__ int total() const { return before[kMaxChunks]; }
  // Free pages below page p <= pages.
  __device__ int below(const Scan& s, int p) const {
    const int c = p / s.chunk_pages;
    int n = before[min(c, kMaxChunks)];
    if (c >= s.chunks) return n;
    const int first = c * (s.chunk_pages / 32);
    for (int w = first; w < p / 32; ++w) n += __popc(s.bits[w]);
    if (p % 32) n += __popc(s.bits[p / 32] & ((1u << p % 32) - 1));
    return n;
  }
  // The free page of rank r < total().
  __device__ int page(const Scan& s, int r) const {
    int lo = 0, hi = kMaxChunks;  // before[lo] <= r < before[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (before[mid] <= r) lo = mid;
      else hi = mid;
    }
    int left = r - before[lo];
    const int words = s.chunk_pages / 32;
    for (int w = 0; w < words; w += 8) {
      const uint4* from = reinterpret_cast<const uint4*>(s.bits + lo * words + w);
      const uint4 a = from[0], b = from[1];
      const uint32_t word[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint32_t bits = word[i];
        const int n = __popc(bits);
        if (left >= n) {
          left -= n;
          continue;
        }
        int at = 0;  // the left-th set bit
#pragma unroll
        for (int half = 16; half > 0; half /= 2) {
          const int low = __popc(bits & ((1u << half) - 1));
          if (left >= low) {
            left -= low;
            bits >>= half;
            at += half;
          }
        }
        return (lo * words + w + i) * 32 + at;
      }
    }
    return -1;  // (the arrays changed under the call)
  }
};

// A CTA an entry.
__global__ void __launch_bounds__(kThreads) pages_extend_sm103a_kernel(const EntryArgs a) {
  __shared__ FreeList list;
  grid_dependency_wait();
  const Entry e = a.s.entries[blockIdx.x];
  if (e.sequence < 0) return;
  const Books& b = a.b;
  if (e.want > 0) {
    list.sum(a.s);
    if (e.want > list.total() - min(e.rank, list.total())) {
      if (threadIdx.x == 0) report_pages(b.status);
      return;
    }
    int* row = b.table + static_cast<long long>(e.sequence) * b.width + blocks_of(b, e.old_tokens);
    for (int i = threadIdx.x; i < e.want; i += kThreads) {
      const int page = list.page(a.s, e.rank + i);
      if (page < 0 || page >= b.pages) continue;
      row[i] = page;
      b.refs[page] = 1;
    }
  }
  if (threadIdx.x == 0) b.lengths[e.sequence] = e.tokens;
}

// A cache's codes and scales, K and V.
struct Pool {
  uint8_t* codes[2];
  float* scale[2];
};

struct ForkArgs {
  EntryArgs e;
  Pool pool;
  int heads, head_size;
};

// CTA (entry, piece): the first piece writes the books, all of them copy.
__global__ void __launch_bounds__(kThreads) cache_fork_sm103a_kernel(const ForkArgs a) {
  __shared__ FreeList list;
  __shared__ int s_page;
  grid_dependency_wait();
  const Entry e = a.e.s.entries[blockIdx.x];
  if (e.sequence < 0) return;
  const Books& b = a.e.b;
  const int tid = threadIdx.x, whole = e.tokens >> b.shift;
  if (e.want == 0 && blockIdx.y > 0) return;
  int page = -1;
  if (e.want > 0) {
    list.sum(a.e.s);
    if (e.rank >= list.total()) {
      if (tid == 0 && blockIdx.y == 0) report_pages(b.status);
      return;
    }
    if (tid == 0) s_page = list.page(a.e.s, e.rank);
    __syncthreads();
    page = s_page;
    if (page < 0 || page >= b.pages) return;
  }
  const int* from = b.table + static_cast<long long>(e.parent) * b.width;
  if (blockIdx.y == 0) {
    int* to = b.table + static_cast<long long>(e.sequence) * b.width;
    for (int i = tid; i < whole; i += kThreads) {
      const int p = from[i];
      to[i] = p;
      if (p >= 0 && p < b.pages) atomicAdd(b.refs + p, 1);
      else report_index(b.status, kIndexPage);
    }
    if (tid == 0) {
      if (page >= 0) {
        to[whole] = page;
        b.refs[page] = 1;
      }
      b.lengths[e.sequence] = e.tokens;
    }
  }
  if (page < 0) return;
  const int source = from[whole];
  if (source < 0 || source >= b.pages) {
    if (tid == 0 && blockIdx.y == 0) report_index(b.status, kIndexPage);
    return;
  }
  if (blockIdx.y == 0)
    for (int i = tid; i < 2 * a.heads; i += kThreads) {
      const int h = i >> 1;
      float* scale = a.pool.scale[i & 1];
      scale[static_cast<long long>(page) * a.heads + h] =
          scale[static_cast<long long>(source) * a.heads + h];
    }
  // The written slots of every head, 16 bytes at a time.
  const int run = (e.tokens - (whole << b.shift)) * a.head_size / 16;  // of a head
  const int block = b.page_tokens * a.head_size / 16, all = 2 * a.heads * run;
  for (int i = blockIdx.y * kThreads + tid; i < all; i += gridDim.y * kThreads) {
    const int unit = i / run, at = i - unit * run;
    uint4* codes = reinterpret_cast<uint4*>(a.pool.codes[unit & 1]);
    const int h = unit >> 1;
    codes[(static_cast<long long>(page) * a.heads + h) * block + at] =
        codes[(static_cast<long long>(source) * a.heads + h) * block + at];
  }
}

// A CTA an entry: its pages' counts go down.
__global__ void __launch_bounds__(128) pages_free_sm103a_kernel(const Books b, const int* which) {
  __shared__ int s_sequence, s_tokens;
  grid_dependency_wait();
  if (threadIdx.x == 0) {
    const int at = which[blockIdx.x];
    s_sequence = at;
    s_tokens = 0;
    if (at < 0 || at >= b.sequences) {
      report_index(b.status, kIndexSequence);
    } else if (!length_ok(b, b.lengths[at])) {
      report_index(b.status, kIndexLength);
    } else {
      const int tokens = atomicExch(b.lengths + at, 0);  // (named twice, the second finds nothing)
      if (length_ok(b, tokens)) s_tokens = tokens;
    }
  }
  __syncthreads();
  const int s = s_sequence;
  const int blocks = blocks_of(b, s_tokens);
  for (int i = threadIdx.x; i < blocks; i += 128) {
    const int p = b.table[static_cast<long long>(s) * b.width + i];
    if (p < 0 || p >= b.pages) {
      report_index(b.status, kIndexPage);
    } else if (atomicAdd(b.refs + p, -1) <= 0) {
      atomicAdd(b.refs + p, 1);  // it was free
      report_index(b.status, kIndexPage);
    }
  }
}

struct CopyArgs {
  Pool from, to;
  const int* sources;  // [count]
  const int* targets;  // [count], or by source where `moves`
  const int* moves;    // compact: a page's new number
  const int* counted;  // compact: the number of moves, on the device
  unsigned long long* taken;  // compact: the next job's number, or nullptr: jobs in turn
  int count;
  int from_pages, to_pages;
  int heads, block_bytes;  // of a page's K
  int jobs;                // 16 KB parts of them
  Books b;                 // compact
  int* in_use;
  int table_ctas;
};

// Compact's list: a warp 32 pages.
__global__ void __launch_bounds__(kThreads)
    pages_rank_sm103a_kernel(const Books b, const Scan s, int* moves, int* in_use) {
  __shared__ FreeList list;
  __shared__ int s_holes;
  grid_dependency_wait();
  list.sum(s);
  const int lane = threadIdx.x & 31;
  const int used = b.pages - list.total();
  if (threadIdx.x == 0) s_holes = list.below(s, used);
  __syncthreads();
  const int first_mover = used - s_holes;  // used pages below `used`
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *in_use = used;
    *s.wanted = s_holes;
    *s.taken = 0;
  }
  const int warps = static_cast<int>(gridDim.x) * kWarps, words = s.chunk_pages / 32;
  const int last = (b.pages + 31) / 32;
  for (int word = blockIdx.x * kWarps + (threadIdx.x >> 5); word < last; word += warps) {
    const int c = word / words;
    int n = 0;  // free pages of the chunk before this word
    for (int w = c * words + lane; w < word; w += 32) n += __popc(s.bits[w]);
    n = list.before[c] + __reduce_add_sync(0xFFFFFFFFu, n);
    const uint32_t bits = s.bits[word];
    const int p = word * 32 + lane;
    if (p < b.pages) {
      int to = -1;
      if (!(bits >> lane & 1u)) {
        to = p;
        if (p >= used) {
          const int j = p - (n + __popc(bits & ((1u << lane) - 1))) - first_mover;
          if (j >= 0 && j < s_holes) {
            to = list.page(s, j);
            s.movers[j] = p;
          }
        }
      }
      moves[p] = to;
    }
    __syncwarp();
  }
}

// A job: 16 KB of a page's K or V.
template <bool kCompact>
__device__ __forceinline__ void copy_job(const CopyArgs& a, long long job) {
  const int tid = threadIdx.x;
  const int i = static_cast<int>(job / a.jobs), part = static_cast<int>(job - static_cast<long long>(i) * a.jobs);
  const int source = a.sources[i];
  if (source < 0 || source >= a.from_pages) {
    if (tid == 0 && part == 0) report_index(a.b.status, kIndexPage);
    return;
  }
  const int target = kCompact ? a.moves[source] : a.targets[i];
  if (target < 0 || target >= a.to_pages) {
    if (tid == 0 && part == 0) report_index(a.b.status, kIndexPage);
    return;
  }
  const int half = a.jobs / 2, which = part >= half, at = (part - which * half) * kJobBytes;
  const uint4* from = reinterpret_cast<const uint4*>(
      a.from.codes[which] + static_cast<long long>(source) * a.block_bytes + at);
  uint4* to = reinterpret_cast<uint4*>(a.to.codes[which] +
                                       static_cast<long long>(target) * a.block_bytes + at);
  const int units = min(kJobBytes, a.block_bytes - at) / 16;
  constexpr int kLoads = kJobBytes / 16 / kThreads;
  uint4 x[kLoads];
#pragma unroll
  for (int k = 0; k < kLoads; ++k)
    if (tid + k * kThreads < units) x[k] = from[tid + k * kThreads];
#pragma unroll
  for (int k = 0; k < kLoads; ++k)
    if (tid + k * kThreads < units) to[tid + k * kThreads] = x[k];
  if (at == 0) {
    for (int h = tid; h < a.heads; h += kThreads)
      a.to.scale[which][static_cast<long long>(target) * a.heads + h] =
          a.from.scale[which][static_cast<long long>(source) * a.heads + h];
    if (kCompact && tid == 0 && which == 0) {
      a.b.refs[target] = a.b.refs[source];
      a.b.refs[source] = 0;
    }
  }
}

// Copies pages; compact: and renames the table's entries.
template <bool kCompact>
__global__ void __launch_bounds__(kThreads, kCopyPerSm) cache_copy_sm103a_kernel(const CopyArgs a) {
  __shared__ long long s_next[2];
  grid_dependency_wait();
  const int tid = threadIdx.x;
  if (kCompact && static_cast<int>(blockIdx.x) < a.table_ctas) {
    const Books& b = a.b;
    const int lane = tid & 31;
    for (int s = blockIdx.x * kWarps + (tid >> 5); s < b.sequences; s += a.table_ctas * kWarps) {
      const int tokens = b.lengths[s];
      if (!length_ok(b, tokens)) {
        if (lane == 0) report_index(b.status, kIndexLength);
        continue;
      }
      int* row = b.table + static_cast<long long>(s) * b.width;
      const int blocks = blocks_of(b, tokens);
      for (int i = lane; i < blocks; i += 32) {
        const int p = row[i], to = p >= 0 && p < b.pages ? a.moves[p] : -1;
        if (to < 0) report_index(b.status, kIndexPage);
        else if (to != p) row[i] = to;
      }
    }
    return;
  }
  const int skip = kCompact ? a.table_ctas : 0;
  const int count = kCompact ? min(*a.counted, a.b.pages) : a.count;
  const long long jobs = static_cast<long long>(count) * a.jobs;
  const int step = static_cast<int>(gridDim.x) - skip;
  long long job = static_cast<int>(blockIdx.x) - skip;
  for (int turn = 0; job < jobs; turn ^= 1) {
    // (asked for while the job is under way; two places, so one barrier a job is enough)
    if (kCompact && a.taken && tid == 0) s_next[turn] = static_cast<long long>(atomicAdd(a.taken, 1ull));
    copy_job<kCompact>(a, job);
    if (kCompact && a.taken) {
      __syncwarp();
      __syncthreads();
      job = step + s_next[turn];
    } else {
      job += step;
    }
  }
}

Books books_of(const csa_kv_pages& p, const DeviceInfo& dev) {
  Books b;
  b.refs = p.refs;
  b.lengths = p.lengths;
  b.table = p.table;
  b.pages = p.pages;
  b.sequences = p.sequences;
  b.width = p.table_width;
  b.page_tokens = p.page_tokens;
  b.shift = 0;
  while (1 << b.shift < p.page_tokens) ++b.shift;
  b.status = dev.status_word;
  return b;
}

Pool pool_of(const csa_kv_cache& c) {
  return {{static_cast<uint8_t*>(c.k), static_cast<uint8_t*>(c.v)}, {c.k_scale, c.v_scale}};
}

size_t up16(size_t n) { return (n + 15) / 16 * 16; }

// The workspace's parts, and its size.
size_t lay_out(const csa_kv_pages& p, int entries, void* workspace, Scan& s) {
  s.chunk_pages = kChunkPages;
  while (static_cast<long long>(s.chunk_pages) * kMaxChunks < p.pages) s.chunk_pages *= 2;
  s.chunks = static_cast<int>((static_cast<long long>(p.pages) + s.chunk_pages - 1) / s.chunk_pages);
  char* base = static_cast<char*>(workspace);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* const got = base + at;
    at += up16(bytes);
    return got;
  };
  s.free_in = reinterpret_cast<int*>(take(kMaxChunks * sizeof(int)));
  s.wanted = reinterpret_cast<int*>(take(sizeof(int)));
  s.taken = reinterpret_cast<unsigned long long*>(take(sizeof(unsigned long long)));
  s.bits = reinterpret_cast<uint32_t*>(
      take(static_cast<size_t>(s.chunks) * (s.chunk_pages / 32) * sizeof(uint32_t)));
  s.movers = reinterpret_cast<int*>(take(static_cast<size_t>(p.pages) * sizeof(int)));
  s.claims = reinterpret_cast<int*>(take(static_cast<size_t>(p.sequences) * sizeof(int)));
  s.entries = reinterpret_cast<Entry*>(take(static_cast<size_t>(entries) * sizeof(Entry)));
  return at;
}

cudaError_t launch_scan(const EntryArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  const int ctas = std::min((a.s.chunks + kPlanThreads / 32 - 1) / (kPlanThreads / 32), dev.sm_count);
  return launch_programmatic(pages_scan_sm103a_kernel, dim3(1 + static_cast<unsigned>(ctas)),
                             kPlanThreads, 0, stream, a);
}

int launched(const char* who, cudaError_t e, std::string& err) {
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e == cudaSuccess) return CSA_OK;
  err = std::string(who) + ": launch: " + cudaGetErrorString(e);
  return CSA_ERR_LAUNCH;
}

}  // namespace

size_t kv_pages_workspace_bytes(const csa_kv_pages& pages, int entries) {
  Scan s;
  return lay_out(pages, entries, nullptr, s);
}

int kv_pages_extend_launch(const csa_kv_pages& pages, const int* sequences, const int* tokens,
                           int n, void* workspace, cudaStream_t stream, const DeviceInfo& dev,
                           std::string& err) {
  EntryArgs a{};
  a.b = books_of(pages, dev);
  lay_out(pages, n, workspace, a.s);
  a.sequences = sequences;
  a.tokens = tokens;
  a.n = n;
  cudaError_t e = launch_scan(a, dev, stream);
  if (e == cudaSuccess)
    e = launch_programmatic(pages_extend_sm103a_kernel, dim3(static_cast<unsigned>(n)), kThreads, 0,
                            stream, a);
  return launched("kv_pages_extend", e, err);
}

int kv_cache_fork_launch(const csa_kv_cache& cache, const csa_kv_pages& pages, const int* parents,
                         const int* children, const int* tokens, int n, void* workspace,
                         cudaStream_t stream, const DeviceInfo& dev, std::string& err) {
  ForkArgs a{};
  a.e.b = books_of(pages, dev);
  lay_out(pages, n, workspace, a.e.s);
  a.e.sequences = children;
  a.e.parents = parents;
  a.e.tokens = tokens;
  a.e.n = n;
  a.e.fork = true;
  a.pool = pool_of(cache);
  a.heads = cache.heads;
  a.head_size = cache.head_size;
  const long long bytes = 2LL * cache.heads * cache.page_tokens * cache.head_size;
  const unsigned pieces = static_cast<unsigned>(
      std::min<long long>((bytes + kForkPieceBytes - 1) / kForkPieceBytes, 16));
  cudaError_t e = launch_scan(a.e, dev, stream);
  if (e == cudaSuccess)
    e = launch_programmatic(cache_fork_sm103a_kernel, dim3(static_cast<unsigned>(n), pieces),
                            kThreads, 0, stream, a);
  return launched("kv_cache_fork", e, err);
}

int kv_pages_free_launch(const csa_kv_pages& pages, const int* sequences, int n,
                         cudaStream_t stream, const DeviceInfo& dev, std::string& err) {
  return launched("kv_pages_free",
                  launch_programmatic(pages_free_sm103a_kernel, dim3(static_cast<unsigned>(n)), 128,
                                      0, stream, books_of(pages, dev), sequences),
                  err);
}

namespace {

CopyArgs copy_args(const csa_kv_cache& to, const csa_kv_cache& from) {
  CopyArgs a{};
  a.from = pool_of(from);
  a.to = pool_of(to);
  a.from_pages = from.pages;
  a.to_pages = to.pages;
  a.heads = from.heads;
  a.block_bytes = from.heads * from.page_tokens * from.head_size;
  a.jobs = 2 * ((a.block_bytes + kJobBytes - 1) / kJobBytes);
  return a;
}

// Whether jobs are large enough to be given out one by one, which evens out how long SMs take:
// 4095 pages of 2 x 64 KB 158 us (6.8 TB/s) and 179 in turn, but 16383 of 2 x 8 KB 92 and 83;
// compacting a cache of 1 GB, with sequences copied out of it before, 119 us and 135 in turn.
bool whole_jobs(const CopyArgs& a) { return a.block_bytes >= kJobBytes; }

}  // namespace

int kv_cache_copy_launch(const csa_kv_cache& to, const csa_kv_cache& from, const int* to_pages,
                         const int* from_pages, int n, cudaStream_t stream, const DeviceInfo& dev,
                         std::string& err) {
  CopyArgs a = copy_args(to, from);
  a.sources = from_pages;
  a.targets = to_pages;
  a.count = n;
  a.b.status = dev.status_word;
  // A CTA a job, as places are free; jobs in turn where they are smaller ones.
  const long long most = whole_jobs(a) && !dev.limited ? 1LL << 30 : kCopyPerSm * dev.sm_count;
  const unsigned grid =
      static_cast<unsigned>(std::min<long long>(static_cast<long long>(n) * a.jobs, most));
  return launched("kv_cache_copy",
                  launch_programmatic(cache_copy_sm103a_kernel<false>, dim3(grid), kThreads, 0,
                                      stream, a),
                  err);
}

int kv_cache_compact_launch(const csa_kv_cache& cache, const csa_kv_pages& pages, int* moves,
                            int* in_use, void* workspace, cudaStream_t stream,
                            const DeviceInfo& dev, std::string& err) {
  EntryArgs scan{};
  scan.b = books_of(pages, dev);
  lay_out(pages, 0, workspace, scan.s);
  CopyArgs a = copy_args(cache, cache);
  a.sources = scan.s.movers;
  a.moves = moves;
  a.counted = scan.s.wanted;
  a.taken = whole_jobs(a) ? scan.s.taken : nullptr;
  a.b = scan.b;
  a.in_use = in_use;
  const int most = kCopyPerSm * dev.sm_count;
  a.table_ctas = std::max(1, std::min((pages.sequences + kWarps - 1) / kWarps, most / 8));
  const long long jobs = static_cast<long long>(pages.pages) * a.jobs;
  const unsigned grid = static_cast<unsigned>(
      a.table_ctas + std::max<long long>(1, std::min<long long>(jobs, most - a.table_ctas)));
  cudaError_t e = launch_scan(scan, dev, stream);
  if (e == cudaSuccess)
    e = launch_programmatic(pages_rank_sm103a_kernel,
                            dim3(static_cast<unsigned>(
                                std::min((pages.pages + 32 * kWarps - 1) / (32 * kWarps),
                                         4 * dev.sm_count))),
                            kThreads, 0, stream, scan.b, scan.s, moves, in_use);
  if (e == cudaSuccess)
    e = launch_programmatic(cache_copy_sm103a_kernel<true>, dim3(grid), kThreads, 0, stream, a);
  return launched("kv_cache_compact", e, err);
}

}  // namespace csa
