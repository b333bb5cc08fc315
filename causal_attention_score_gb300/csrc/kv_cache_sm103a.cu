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
// Bound: HBM. A write reads the new rows once (two passes over registers: the
// magnitude, then the codes) and writes one byte an element; older codes of a
// block are read and written only when its scale grew. A unit of work is one
// (sequence, page, K or V, head); units of one page's heads are neighbours, so
// that CTAs running side by side read neighbouring memory of a row.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <string>

#include "csa_internal.h"
#include "kv_cache.cuh"
#include "sm103a_ptx.cuh"

namespace csa {
namespace {

constexpr int kBlockThreads = 256;
constexpr int kBlockVecs = 8;  // 8-element vectors a thread holds: 128 tokens x 128 / 256 / 8
// Sequences of at most this many new tokens take a warp per unit (and up to 4
// vectors a lane); longer ones a CTA of 256 threads.
constexpr int kStepTokens = 8;
constexpr int kStepVecs = 4;
constexpr float kScaleFloor = 7.888609052210118e-31f;  // 2^-100

struct CacheArgs {
  KvView v;
  void* x[2];                           // rows of K, V
  long long token[2], head_stride[2];   // their strides in elements
  int touched;                          // most pages a sequence's new tokens lie in
  long long units;
};

struct Unit {
  int s, j, which, h;
};

__device__ __forceinline__ Unit decode_unit(const CacheArgs& a, long long u) {
  Unit r;
  const int H = a.v.heads;
  const long long q = u / H;
  r.h = static_cast<int>(u - q * H);
  r.which = static_cast<int>(q & 1);
  const long long p = q >> 1;
  r.s = static_cast<int>(p / a.touched);
  r.j = static_cast<int>(p - static_cast<long long>(r.s) * a.touched);
  return r;
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

// x / s correctly rounded: r is 1 / s to nearest, and one Newton correction of
// the quotient x * r gives the rounded quotient (Markstein, 1990).
__device__ __forceinline__ float quotient(float x, float s, float r) {
  const float y = x * r;
  return fmaf(fmaf(-y, s, x), r, y);
}

// Four values (finite, within 127 s or 448 s) as codes.
template <int kFormat>
__device__ __forceinline__ uint32_t codes4(const float (&x)[4], float s, float r) {
  if (kFormat == CSA_KV_INT8) {
    uint32_t b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)  // 1.5 * 2^23 + code: the code is the low byte
      b[i] = __float_as_uint(quotient(x[i], s, r) + 12582912.0f);
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

// kThreads = 32: a warp is the worker (kStepVecs vectors a lane); else the CTA.
template <typename T, int kFormat, int kThreads>
__global__ void __launch_bounds__(kBlockThreads) cache_write_sm103a_kernel(const CacheArgs a) {
  grid_dependency_wait();
  constexpr int NV = kThreads == 32 ? kStepVecs : kBlockVecs;
  __shared__ uint32_t s_max[kBlockThreads / 32];
  const int tid = threadIdx.x % kThreads;
  const int worker = threadIdx.x / kThreads;
  constexpr int kWorkers = kBlockThreads / kThreads;
  const int D8 = a.v.head_size / 8;
  for (long long u = static_cast<long long>(blockIdx.x) * kWorkers + worker; u < a.units;
       u += static_cast<long long>(gridDim.x) * kWorkers) {
    const Unit w = decode_unit(a, u);
    const KvSequence q = kv_sequence(a.v, w.s);
    Part p;
    if (!part_of(a.v, q, w.j, p)) continue;
    const int page = kv_page(a.v, w.s, p.block);
    if (page < 0) continue;
    const T* x = static_cast<const T*>(a.x[w.which]) +
                 static_cast<long long>(p.row) * a.token[w.which] + w.h * a.head_stride[w.which];
    uint8_t* codes = a.v.codes[w.which] + kv_page_offset(a.v, page, w.h);
    float* scale = a.v.scale[w.which] + static_cast<long long>(page) * a.v.heads + w.h;
    const float s_old = p.t0 > 0 ? *scale : 0.0f;

    const int nvec = (p.t1 - p.t0) * D8;
    uint4 in[NV];
    uint32_t all = 0, finite = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = tid + i * kThreads;
      in[i] = make_uint4(0, 0, 0, 0);
      if (e < nvec) {
        const int t = e / D8;
        in[i] = *reinterpret_cast<const uint4*>(x + t * a.token[w.which] + (e - t * D8) * 8);
      }
    }
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
      if (kThreads > 32) {
        __syncthreads();
        if ((threadIdx.x & 31) == 0) s_max[threadIdx.x / 32] = m;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kBlockThreads / 32; ++i) m = max(m, s_max[i]);
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
        uint2* at = reinterpret_cast<uint2*>(codes) + e;
        uint2 c = *at;
        uint32_t* half = reinterpret_cast<uint32_t*>(&c);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float f[4];
          codes4_to_float<kFormat>(half[k], f);
#pragma unroll
          for (int i = 0; i < 4; ++i) f[i] *= s_old;
          half[k] = codes4_any<kFormat>(f, s, r);
        }
        *at = c;
      }
    }
    uint2* to = reinterpret_cast<uint2*>(codes) + p.t0 * D8;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = tid + i * kThreads;
      if (e >= nvec) break;
      const uint32_t part[4] = {in[i].x, in[i].y, in[i].z, in[i].w};
      uint32_t c[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float f[4] = {to_float<T>(part[2 * k] & 0xFFFFu), to_float<T>(part[2 * k] >> 16),
                      to_float<T>(part[2 * k + 1] & 0xFFFFu), to_float<T>(part[2 * k + 1] >> 16)};
        c[k] = odd ? codes4_any<kFormat>(f, s, r) : codes4<kFormat>(f, s, r);
      }
      to[e] = make_uint2(c[0], c[1]);
    }
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
// where this library wrote it; it is rounded once, to T.
template <typename T, int kFormat, int kThreads>
__global__ void __launch_bounds__(kBlockThreads) cache_read_sm103a_kernel(const CacheArgs a) {
  grid_dependency_wait();
  const int tid = threadIdx.x % kThreads;
  const int worker = threadIdx.x / kThreads;
  constexpr int kWorkers = kBlockThreads / kThreads;
  const int D8 = a.v.head_size / 8;
  for (long long u = static_cast<long long>(blockIdx.x) * kWorkers + worker; u < a.units;
       u += static_cast<long long>(gridDim.x) * kWorkers) {
    const Unit w = decode_unit(a, u);
    const KvSequence q = kv_sequence(a.v, w.s);
    Part p;
    if (!part_of(a.v, q, w.j, p)) continue;
    const int page = kv_page(a.v, w.s, p.block);
    if (page < 0) continue;
    T* y = static_cast<T*>(a.x[w.which]) + static_cast<long long>(p.row) * a.token[w.which] +
           w.h * a.head_stride[w.which];
    const uint2* codes = reinterpret_cast<const uint2*>(a.v.codes[w.which] +
                                                        kv_page_offset(a.v, page, w.h)) +
                         p.t0 * D8;
    const float s = a.v.scale[w.which][static_cast<long long>(page) * a.v.heads + w.h];
    const int nvec = (p.t1 - p.t0) * D8;
#pragma unroll 4
    for (int e = tid; e < nvec; e += kThreads) {
      const int t = e / D8;
      const uint2 c = codes[e];
      float f[4], g[4];
      codes4_to_float<kFormat>(c.x, f);
      codes4_to_float<kFormat>(c.y, g);
      const float o[8] = {f[0] * s, f[1] * s, f[2] * s, f[3] * s,
                          g[0] * s, g[1] * s, g[2] * s, g[3] * s};
      store8<T>(y + t * a.token[w.which] + (e - t * D8) * 8, o);
    }
  }
}

template <typename T, int kFormat, bool kWrite>
cudaError_t launch_cache(CacheArgs a, int sms, cudaStream_t stream) {
  const bool step = a.v.max_new <= kStepTokens;
  const int workers = step ? kBlockThreads / 32 : 1;
  const long long blocks = (a.units + workers - 1) / workers;
  const unsigned grid = static_cast<unsigned>(
      std::min<long long>(blocks, static_cast<long long>(sms) * (2048 / kBlockThreads)));
  if constexpr (kWrite)
    return step ? launch_programmatic(cache_write_sm103a_kernel<T, kFormat, 32>, grid,
                                      kBlockThreads, 0, stream, a)
                : launch_programmatic(cache_write_sm103a_kernel<T, kFormat, kBlockThreads>, grid,
                                      kBlockThreads, 0, stream, a);
  else
    return step ? launch_programmatic(cache_read_sm103a_kernel<T, kFormat, 32>, grid,
                                      kBlockThreads, 0, stream, a)
                : launch_programmatic(cache_read_sm103a_kernel<T, kFormat, kBlockThreads>, grid,
                                      kBlockThreads, 0, stream, a);
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
  a.units = static_cast<long long>(batch.sequences) * a.touched * 2 * cache.heads;
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
