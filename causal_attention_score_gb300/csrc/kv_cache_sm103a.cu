// Writing keys and values into the paged 8-bit cache, and reading them back.
//
// A block is the page_tokens tokens of one page and head; it has one scale.
//   int8:  s = the smallest value of 8 significant bits with 127 s >= m,
//          code = x / s to the nearest whole number (ties to even);
//   e4m3:  s = the smallest power of two with 448 s >= m, code = e4m3(x / s);
// m is the block's largest finite magnitude and s >= 2^-100. NaN becomes 0 and
// infinities the largest code, so a written cache holds finite values only.
// When a block grows, s = max(s_old, s of the new tokens), and if that is more
// than s_old the block's older codes become code * s_old / s, rounded again.
//
// Why such scales: with x of at most 11 significant bits and s of 8, x / s is
// either half-way between two codes or at least 2^-13 away from half-way, and
// code * s_old / s = q is at least 2^-18 max(1, q) away. An fp32 quotient, off by at most
// q * 2^-24, therefore rounds to the code of the exact one, and a tie is
// computed exactly: the codes are those of the definition in real numbers. The
// 8 bits cost at most 2^-7 of the step. A power of two does the same for e4m3
// for free, where the step is relative to begin with.
//
// Bound: HBM, with the issue slots close behind (a bf16 element is 3 bytes moved: at
// the copy rate an SM has 16 instructions' worth of lanes for it), so quotients are
// computed two at a time (packed fp32) and positions with a multiplication. A write
// reads the new rows once (two passes over registers: the magnitude, then the codes)
// and writes one byte an element; older codes of a block are read and written only when
// its scale grew (a token of 256 sequences, 8 heads of 128: 5.5 us, and 16 us where
// every block of up to 32 tokens grows, 48 us with 128: one warp a block). A unit of
// work is one (sequence, page, K or V, head); units of one page's heads are neighbours,
// so that CTAs running side by side read neighbouring memory of a row. A unit's place
// (sequence, page) is looked up while the rows of the one before are on their way.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <string>
#include <type_traits>

#include "csa_internal.h"
#include "kv_cache.cuh"
#include "sm103a_ptx.cuh"

namespace csa {
namespace {

constexpr int kBlockThreads = 256;
// A unit that is written has one worker, which holds its new rows in registers: a warp
// (4 vectors of 8 elements a lane) where no sequence has more than 8 new tokens, else as
// many warps as hold a whole block in 8 vectors a lane, one (16 x 128) to eight
// (128 x 128). (With 256 threads for every block the lanes without elements took
// the issue slots: 96 us instead of 53 for 28K tokens of 16 heads of 128.)
constexpr int kStepTokens = 8;
constexpr int kStepVecs = 4;
constexpr int kBlockVecs = 8;
constexpr int kWritePerSm = 4;  // CTAs by registers; the grid has kWriteGrid an SM
constexpr int kWriteGrid = 8;

struct CacheArgs {
  KvView v;
  void* x[2];                           // rows of K, V
  long long token[2], head_stride[2];   // their strides in elements
  int touched;                          // most pages a sequence's new tokens lie in
  unsigned by_chunks;                   // 2^31 / (8-element chunks of a row), rounded up
  unsigned step_s;                      // gridDim.x * workers of a CTA, in units:
  int step_j, step_which, step_h;       //   sequences, pages, K or V, heads
};

// e / chunks: exact while e * chunks < 2^31 (both stay below 2^13).
__device__ __forceinline__ int row_of(const CacheArgs& a, int e) {
  return static_cast<int>(__umulhi(2u * static_cast<unsigned>(e), a.by_chunks));
}

struct Unit {
  unsigned s;
  int j, which, h;
};

__device__ __forceinline__ Unit first_unit(const CacheArgs& a, unsigned u) {
  Unit r;
  const unsigned q = u / a.v.heads;
  r.h = static_cast<int>(u - q * a.v.heads);
  r.which = static_cast<int>(q & 1);
  r.s = (q >> 1) / a.touched;
  r.j = static_cast<int>((q >> 1) - r.s * a.touched);
  return r;
}
__device__ __forceinline__ void next_unit(const CacheArgs& a, Unit& u) {
  u.h += a.step_h;
  u.which += a.step_which;
  u.j += a.step_j;
  u.s += a.step_s;
  if (u.h >= a.v.heads) u.h -= a.v.heads, ++u.which;
  if (u.which >= 2) u.which -= 2, ++u.j;
  if (u.j >= a.touched) u.j -= a.touched, ++u.s;
}

// The part of a sequence's rows that lies in its j-th page from the first that
// they touch: tokens [t0, t1) of block `block`, from row `row`. False: none.
struct Part {
  int block, t0, t1, row;
};
__device__ __forceinline__ bool part_of(const KvView& v, const KvSequence& q, int j, Part& p) {
  const int from = max(q.first, 0);
  if (q.n <= 0 || from >= q.length) return false;
  p.block = (from >> v.page_shift) + j;
  const long long base = static_cast<long long>(p.block) << v.page_shift;
  if (base >= q.length) return false;
  p.t0 = max(from - static_cast<int>(base), 0);
  p.t1 = min(q.length - static_cast<int>(base), v.page_tokens);
  p.row = q.row0 + static_cast<int>(base) + p.t0 - q.first;
  return true;
}

template <typename T>
__device__ __forceinline__ float to_float(uint32_t bits16);
template <>
__device__ __forceinline__ float to_float<__nv_bfloat16>(uint32_t b) {
  return __uint_as_float(b << 16);
}
template <>
__device__ __forceinline__ float to_float<__half>(uint32_t b) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(b)));
}
// Both values of a word.
template <typename T>
__device__ __forceinline__ void to_float2(uint32_t w, float& lo, float& hi);
template <>
__device__ __forceinline__ void to_float2<__nv_bfloat16>(uint32_t w, float& lo, float& hi) {
  lo = __uint_as_float(w << 16);
  hi = __uint_as_float(w & 0xFFFF0000u);
}
template <>
__device__ __forceinline__ void to_float2<__half>(uint32_t w, float& lo, float& hi) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  lo = f.x;
  hi = f.y;
}
template <typename T>
constexpr uint32_t kInfBits = 0x7F80u;
template <>
constexpr uint32_t kInfBits<__half> = 0x7C00u;

template <int kFormat>
__device__ __forceinline__ float scale_of(float m) {
  if (kFormat == CSA_KV_INT8) {
    float s = __uint_as_float(__float_as_uint(__fdiv_rn(m, 127.0f)) & 0xFFFF0000u);
    if (s * 127.0f < m) s = __uint_as_float(__float_as_uint(s) + 0x10000u);
    return fmaxf(s, kScaleFloor);
  }
  // m = 1.f * 2^(E - 127); 448 = 1.75 * 2^8
  const uint32_t b = __float_as_uint(m);
  const int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return e < -100 ? kScaleFloor : __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// x / s correctly rounded, two at a time: r is 1 / s to nearest, and one Newton
// correction of the quotient x * r gives the rounded quotient (Markstein, 1990).
// Four values (finite, within 127 s or 448 s) as codes.
template <int kFormat>
__device__ __forceinline__ uint32_t codes4(const float (&x)[4], float s, float r) {
  if (kFormat == CSA_KV_INT8) {
    const uint64_t r2 = pack_f32x2(r, r), s2 = pack_f32x2(-s, -s);
    // 1.5 * 2^23 + code: the code is the low byte
    const uint64_t magic = pack_f32x2(12582912.0f, 12582912.0f);
    uint32_t b[4];
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const uint64_t v = pack_f32x2(x[i], x[i + 1]);
      const uint64_t y = mul_f32x2(v, r2);
      const uint64_t q = fma_f32x2(fma_f32x2(y, s2, v), r2, y);
      float lo, hi;
      unpack_f32x2(add_f32x2(q, magic), lo, hi);
      b[i] = __float_as_uint(lo);
      b[i + 1] = __float_as_uint(hi);
    }
    return byte_perm(byte_perm(b[0], b[1], 0x0040), byte_perm(b[2], b[3], 0x0040), 0x5410);
  }
  return e4m3x2_from_float2(x[0] * r, x[1] * r) | (e4m3x2_from_float2(x[2] * r, x[3] * r) << 16);
}

// The same for values that may be infinite or NaN.
template <int kFormat>
__device__ __forceinline__ uint32_t codes4_any(float (&x)[4], float s, float r) {
  const float top = (kFormat == CSA_KV_INT8 ? 127.0f : 448.0f) * s;
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = isnan(x[i]) ? 0.0f : fminf(fmaxf(x[i], -top), top);
  return codes4<kFormat>(x, s, r);
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Where a unit's rows and codes are; page < 0: it has nothing to do.
struct Place {
  Part p;
  int page;
};
__device__ __forceinline__ Place place_of(const CacheArgs& a, const Unit& u) {
  Place r;
  r.page = -1;
  if (u.s >= static_cast<unsigned>(a.v.sequences)) return r;
  const KvSequence q = kv_sequence(a.v, u.s);
  if (part_of(a.v, q, u.j, r.p)) r.page = kv_page(a.v, u.s, r.p.block);
  return r;
}

// (checking build) whether a place is inside the cache and the rows.
[[maybe_unused]] __device__ __forceinline__ bool place_ok(const CacheArgs& a, const Unit& u,
                                                          const Place& at) {
  const Part& p = at.p;
  return u.h >= 0 && u.h < a.v.heads && (u.which == 0 || u.which == 1) && at.page < a.v.pages &&
         p.t0 >= 0 && p.t0 < p.t1 && p.t1 <= a.v.page_tokens && p.row >= 0 &&
         p.row + p.t1 - p.t0 <= a.v.rows;
}

template <int kThreads>
__device__ __forceinline__ void worker_sync(int worker) {
  asm volatile("bar.sync %0, %1;" ::"r"(1 + worker), "n"(kThreads) : "memory");
}

// kThreads are a worker, NV the vectors that each holds.
template <typename T, int kFormat, int kThreads, int NV>
__global__ void __launch_bounds__(kBlockThreads, kWritePerSm)
    cache_write_sm103a_kernel(const CacheArgs a) {
  grid_dependency_wait();
  constexpr int kWorkers = kBlockThreads / kThreads;
  __shared__ uint32_t s_max[kBlockThreads / 32];
  [[maybe_unused]] __shared__ int s_abort;
  [[maybe_unused]] const Watchdog wd{0, a.v.status, &s_abort};
  const int tid = threadIdx.x % kThreads;
  const int worker = threadIdx.x / kThreads;
  const int D8 = a.v.head_size / 8;
  Unit u = first_unit(a, blockIdx.x * kWorkers + worker);
  Place next = place_of(a, u);
  while (u.s < static_cast<unsigned>(a.v.sequences)) {
    const Place at = next;
    const Unit w = u;
    next_unit(a, u);
    if (at.page < 0) {
      next = place_of(a, u);
      continue;
    }
    const Part& p = at.p;
    if (!CSA_CHECK(place_ok(a, w, at) && (p.t1 - p.t0) * D8 <= kThreads * NV, wd, kCheckTile)) {
      next = place_of(a, u);
      continue;
    }
    const long long token = a.token[w.which];
    const T* x = static_cast<const T*>(a.x[w.which]) + static_cast<long long>(p.row) * token +
                 w.h * a.head_stride[w.which];
    uint8_t* codes = a.v.codes[w.which] + kv_page_offset(a.v, at.page, w.h);
    float* scale = a.v.scale[w.which] + static_cast<long long>(at.page) * a.v.heads + w.h;
    const float s_old = p.t0 > 0 ? *scale : 0.0f;

    const int nvec = (p.t1 - p.t0) * D8;
    uint4 in[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = tid + i * kThreads;
      in[i] = make_uint4(0, 0, 0, 0);
      if (e < nvec) {
        const int t = row_of(a, e);
        in[i] = __ldg(reinterpret_cast<const uint4*>(x + t * token + (e - t * D8) * 8));
      }
    }
    next = place_of(a, u);
    uint32_t all = 0, finite = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint32_t m = max_u16x2(
          max_u16x2(in[i].x & 0x7FFF7FFFu, in[i].y & 0x7FFF7FFFu),
          max_u16x2(in[i].z & 0x7FFF7FFFu, in[i].w & 0x7FFF7FFFu));
      all = max_u16x2(all, m);
    }
    all = max(all & 0xFFFFu, all >> 16);
    // Largest magnitude over the worker, as the type's bits (ordered like the values).
    auto reduce = [&](uint32_t m) {
      m = __reduce_max_sync(0xFFFFFFFFu, m);
      if constexpr (kThreads > 32) {
        worker_sync<kThreads>(worker);
        if ((threadIdx.x & 31) == 0) s_max[threadIdx.x / 32] = m;
        worker_sync<kThreads>(worker);
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) m = max(m, s_max[worker * (kThreads / 32) + i]);
      }
      return m;
    };
    all = reduce(all);
    finite = all;
    const bool odd = all >= kInfBits<T>;  // an infinity or a NaN among them
    if (odd) {
      finite = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const uint32_t part[4] = {in[i].x, in[i].y, in[i].z, in[i].w};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t b = (part[k / 2] >> (16 * (k & 1))) & 0x7FFFu;
          if (b < kInfBits<T>) finite = max(finite, b);
        }
      }
      finite = reduce(finite);
    }
    const float s_new = scale_of<kFormat>(to_float<T>(finite));
    const float s = fmaxf(s_old, s_new);
    const float r = __frcp_rn(s);

    if (p.t0 > 0 && s > s_old) {
      // older codes of the block, to the new scale
      const int n8 = p.t0 * D8;
      for (int e = tid; e < n8; e += kThreads) {
        uint2* to = reinterpret_cast<uint2*>(codes) + e;
        uint2 c = *to;
        uint32_t* half = reinterpret_cast<uint32_t*>(&c);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float f[4];
          codes4_to_float<kFormat>(half[k], f);
#pragma unroll
          for (int i = 0; i < 4; ++i) f[i] *= s_old;
          half[k] = codes4_any<kFormat>(f, s, r);
        }
        *to = c;
      }
    }
    uint2* to = reinterpret_cast<uint2*>(codes) + p.t0 * D8;
    auto put = [&](auto any) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int e = tid + i * kThreads;
        if (e >= nvec) break;
        const uint32_t part[4] = {in[i].x, in[i].y, in[i].z, in[i].w};
        uint32_t c[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float f[4];
          to_float2<T>(part[2 * k], f[0], f[1]);
          to_float2<T>(part[2 * k + 1], f[2], f[3]);
          if constexpr (decltype(any)::value) c[k] = codes4_any<kFormat>(f, s, r);
          else c[k] = codes4<kFormat>(f, s, r);
        }
        to[e] = make_uint2(c[0], c[1]);
      }
    };
    if (odd) put(std::true_type{});
    else put(std::false_type{});
    if (tid == 0) *scale = s;
  }
}

template <typename T>
__device__ __forceinline__ void store8(T* to, const float (&f)[8]);
template <>
__device__ __forceinline__ void store8<float>(float* to, const float (&f)[8]) {
  reinterpret_cast<float4*>(to)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(to)[1] = make_float4(f[4], f[5], f[6], f[7]);
}
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* to, const float (&f)[8]) {
  uint4 r;
  uint32_t* w = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(to) = r;
}
template <>
__device__ __forceinline__ void store8<__half>(__half* to, const float (&f)[8]) {
  uint4 r;
  uint32_t* w = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(to) = r;
}

// code * s in fp32 is exact for int8 (7 and 8 bits) and e4m3 (a power of two)
// where this library wrote it; it is rounded once, to T. A warp a unit, a lane 8 codes a
// load and kReadVecs loads in flight; a warp's store of 16-bit values is one run of
// memory. (A CTA a unit with one load in flight: 86 us instead of 49; 16 codes a load,
// whose values leave gaps between a store's lanes: 66 us.)
constexpr int kReadVecs = 8;
constexpr int kReadPerSm = 3;  // CTAs by registers; 32 an SM in the grid: 49 us, 3: 57
constexpr int kReadGrid = 32;
template <typename T, int kFormat>
__global__ void __launch_bounds__(kBlockThreads, kReadPerSm)
    cache_read_sm103a_kernel(const CacheArgs a) {
  grid_dependency_wait();
  constexpr int kWorkers = kBlockThreads / 32;
  [[maybe_unused]] __shared__ int s_abort;
  [[maybe_unused]] const Watchdog wd{0, a.v.status, &s_abort};
  const int lane = threadIdx.x % 32;
  const int D8 = a.v.head_size / 8;
  Unit u = first_unit(a, blockIdx.x * kWorkers + threadIdx.x / 32);
  Place next = place_of(a, u);
  while (u.s < static_cast<unsigned>(a.v.sequences)) {
    const Place at = next;
    const Unit w = u;
    next_unit(a, u);
    if (at.page < 0) {
      next = place_of(a, u);
      continue;
    }
    const Part& p = at.p;
    if (!CSA_CHECK(place_ok(a, w, at), wd, kCheckTile)) {
      next = place_of(a, u);
      continue;
    }
    const long long token = a.token[w.which];
    T* y = static_cast<T*>(a.x[w.which]) + static_cast<long long>(p.row) * token +
           w.h * a.head_stride[w.which];
    const uint2* codes = reinterpret_cast<const uint2*>(a.v.codes[w.which] +
                                                        kv_page_offset(a.v, at.page, w.h)) +
                         p.t0 * D8;
    const float s = a.v.scale[w.which][static_cast<long long>(at.page) * a.v.heads + w.h];
    const int nvec = (p.t1 - p.t0) * D8;
    for (int e0 = 0; e0 < nvec; e0 += 32 * kReadVecs) {
      uint2 c[kReadVecs];
#pragma unroll
      for (int i = 0; i < kReadVecs; ++i) {
        const int e = e0 + lane + 32 * i;
        c[i] = make_uint2(0, 0);
        if (e < nvec) c[i] = codes[e];
      }
      if (e0 == 0) next = place_of(a, u);
#pragma unroll
      for (int i = 0; i < kReadVecs; ++i) {
        const int e = e0 + lane + 32 * i;
        if (e >= nvec) break;
        const int t = row_of(a, e);
        float f[4], g[4];
        codes4_to_float<kFormat>(c[i].x, f);
        codes4_to_float<kFormat>(c[i].y, g);
        const float o[8] = {f[0] * s, f[1] * s, f[2] * s, f[3] * s,
                            g[0] * s, g[1] * s, g[2] * s, g[3] * s};
        store8<T>(y + t * token + (e - t * D8) * 8, o);
      }
    }
  }
}

template <typename Kernel>
cudaError_t launch_workers(Kernel kernel, int workers, int per_sm, CacheArgs a, int sms,
                           cudaStream_t stream) {
  const long long units =
      static_cast<long long>(a.v.sequences) * a.touched * 2 * a.v.heads;
  const unsigned grid = static_cast<unsigned>(
      std::min<long long>((units + workers - 1) / workers,
                          static_cast<long long>(sms) * per_sm));
  unsigned step = grid * workers;
  a.step_h = static_cast<int>(step % a.v.heads);
  step /= a.v.heads;
  a.step_which = static_cast<int>(step % 2);
  step /= 2;
  a.step_j = static_cast<int>(step % a.touched);
  a.step_s = step / a.touched;
  const unsigned chunks = a.v.head_size / 8;
  a.by_chunks = ((1u << 31) + chunks - 1) / chunks;
  return launch_programmatic(kernel, grid, kBlockThreads, 0, stream, a);
}

template <typename T, int kFormat, bool kWrite>
cudaError_t launch_cache(const CacheArgs& a, int sms, cudaStream_t stream) {
  if constexpr (kWrite) {
    const int vectors = a.v.page_tokens * a.v.head_size / 8;
    if (a.v.max_new <= kStepTokens)
      return launch_workers(cache_write_sm103a_kernel<T, kFormat, 32, kStepVecs>, 8, kWriteGrid, a, sms,
                            stream);
    if (vectors <= 32 * kBlockVecs)
      return launch_workers(cache_write_sm103a_kernel<T, kFormat, 32, kBlockVecs>, 8, kWriteGrid, a, sms,
                            stream);
    if (vectors <= 64 * kBlockVecs)
      return launch_workers(cache_write_sm103a_kernel<T, kFormat, 64, kBlockVecs>, 4, kWriteGrid, a, sms,
                            stream);
    if (vectors <= 128 * kBlockVecs)
      return launch_workers(cache_write_sm103a_kernel<T, kFormat, 128, kBlockVecs>, 2, kWriteGrid, a, sms,
                            stream);
    return launch_workers(cache_write_sm103a_kernel<T, kFormat, 256, kBlockVecs>, 1, kWriteGrid, a, sms,
                          stream);
  } else {
    return launch_workers(cache_read_sm103a_kernel<T, kFormat>, 8, kReadGrid, a, sms, stream);
  }
}

template <typename T, bool kWrite>
cudaError_t launch_cache(const CacheArgs& a, int format, int sms, cudaStream_t stream) {
  return format == CSA_KV_INT8 ? launch_cache<T, CSA_KV_INT8, kWrite>(a, sms, stream)
                               : launch_cache<T, CSA_KV_E4M3, kWrite>(a, sms, stream);
}

}  // namespace

KvView kv_view(const csa_kv_cache& c, const csa_kv_batch& b, const DeviceInfo& dev) {
  KvView v;
  v.codes[0] = static_cast<uint8_t*>(c.k);
  v.codes[1] = static_cast<uint8_t*>(c.v);
  v.scale[0] = c.k_scale;
  v.scale[1] = c.v_scale;
  v.offsets = b.offsets;
  v.lengths = b.lengths;
  v.table = b.table;
  v.pages = c.pages;
  v.heads = c.heads;
  v.page_tokens = c.page_tokens;
  v.page_shift = 0;
  while ((1 << v.page_shift) < c.page_tokens) ++v.page_shift;
  v.head_size = c.head_size;
  v.sequences = b.sequences;
  v.table_width = b.table_width;
  v.rows = b.rows;
  v.max_new = b.max_new;
  v.status = dev.status_word;
  return v;
}

int kv_cache_launch(const csa_kv_cache& cache, const csa_kv_batch& batch, const KvRows& rows,
                    bool write, cudaStream_t stream, const DeviceInfo& dev, std::string& err) {
  CacheArgs a;
  a.v = kv_view(cache, batch, dev);
  for (int i = 0; i < 2; ++i) {
    a.x[i] = rows.x[i];
    a.token[i] = rows.token[i];
    a.head_stride[i] = rows.head[i];
  }
  // n tokens lie in at most (n + P - 2) / P + 1 pages
  a.touched = static_cast<int>(std::min<long long>(
      (static_cast<long long>(batch.max_new) + cache.page_tokens - 2) / cache.page_tokens + 1,
      batch.table_width));
  cudaError_t e;
  if (write)
    e = rows.dtype == CSA_F16
            ? launch_cache<__half, true>(a, cache.format, dev.sm_count, stream)
            : launch_cache<__nv_bfloat16, true>(a, cache.format, dev.sm_count, stream);
  else
    e = rows.dtype == CSA_F32   ? launch_cache<float, false>(a, cache.format, dev.sm_count, stream)
        : rows.dtype == CSA_F16 ? launch_cache<__half, false>(a, cache.format, dev.sm_count, stream)
                                : launch_cache<__nv_bfloat16, false>(a, cache.format, dev.sm_count,
                                                                     stream);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) {
    err = std::string(write ? "kv_cache_write" : "kv_cache_read") + ": launch: " +
          cudaGetErrorString(e);
    return CSA_ERR_LAUNCH;
  }
  return CSA_OK;
}

}  // namespace csa
