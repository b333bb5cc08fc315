// The paged 8-bit cache as its kernels see it: addressing with bounds checks,
// and the conversions between codes and values.
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

#include "csa.h"
#include "sm103a_ptx.cuh"

namespace csa {

// Asks for `bytes` (a multiple of 16, at a 16-byte boundary) in L2.
__device__ __forceinline__ void bulk_prefetch_l2(const void* from, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                   reinterpret_cast<uint64_t>(from)),
               "r"(bytes)
               : "memory");
}

// Two fp32 products and multiply-adds at once, each rounded to nearest.
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

constexpr float kScaleFloor = 7.888609052210118e-31f;  // 2^-100, the smallest scale written

// Device view of csa_kv_cache + csa_kv_batch.
struct KvView {
  uint8_t* codes[2];  // K, V: [pages][heads][page_tokens][head_size]
  float* scale[2];    // [pages][heads]
  const int* offsets;  // [sequences + 1]
  const int* lengths;  // [sequences]
  const int* table;    // [sequences][table_width]
  int pages, heads, page_tokens, page_shift, head_size;
  int sequences, table_width, rows, max_new;
  int* status;
};

// Identifiers of refused indices, recorded beside CSA_ERR_INDEX.
enum IndexSite : int {
  kIndexPage = 201,     // a table entry outside [0, pages)
  kIndexRows = 202,     // offsets outside [0, rows], decreasing, or more than max_new apart
  kIndexLength = 203,   // a length outside [0, table_width * page_tokens]
};

__device__ __forceinline__ void report_index(int* status, int site) {
  if (atomicCAS(status, 0, CSA_ERR_INDEX) == 0) atomicExch(status + 1, site);
}

// One sequence of a batch: its rows [row0, row0 + n) are its last n tokens, at
// positions first .. first + n - 1 = length - 1 (negative ones have no place).
struct KvSequence {
  int row0, n, length, first;
};

// Reads and checks a sequence's entry. A bad one is recorded and has no rows.
__device__ __forceinline__ KvSequence kv_sequence(const KvView& v, int s) {
  KvSequence q;
  q.row0 = v.offsets[s];
  const int end = v.offsets[s + 1];
  q.length = v.lengths[s];
  const bool rows_ok =
      q.row0 >= 0 && end >= q.row0 && end <= v.rows && end - q.row0 <= v.max_new;
  const bool length_ok =
      q.length >= 0 && q.length <= static_cast<long long>(v.table_width) * v.page_tokens;
  if (!rows_ok || !length_ok) {
    report_index(v.status, rows_ok ? kIndexLength : kIndexRows);
    q.row0 = q.n = q.length = q.first = 0;
    return q;
  }
  q.n = end - q.row0;
  q.first = q.length - q.n;
  return q;
}

// Page of block `block` of sequence s, or -1 (recorded) when the entry names none.
__device__ __forceinline__ int kv_page(const KvView& v, int s, int block) {
  const int p = v.table[static_cast<long long>(s) * v.table_width + block];
  if (p < 0 || p >= v.pages) {
    report_index(v.status, kIndexPage);
    return -1;
  }
  return p;
}

__device__ __forceinline__ long long kv_page_offset(const KvView& v, int page, int head) {
  return (static_cast<long long>(page) * v.heads + head) * v.page_tokens * v.head_size;
}

// Two e4m3 codes (low byte first) as fp16 values: exact.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t codes16) {
  uint32_t h;
  asm("{\n\t.reg .b16 c;\n\tcvt.u16.u32 c, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}"
      : "=r"(h)
      : "r"(codes16));
  return h;
}

// Two fp32 values as e4m3 codes, rounded to nearest even, past 448 saturated.
__device__ __forceinline__ uint32_t e4m3x2_from_float2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b16 c;\n\tcvt.rn.satfinite.e4m3x2.f32 c, %2, %1;\n\tcvt.u32.u16 %0, c;\n\t}"
      : "=r"(r)
      : "f"(lo), "f"(hi));
  return r;
}

__device__ __forceinline__ uint32_t byte_perm(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}

__device__ __forceinline__ uint32_t half2_sub(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Byte pairs of int8 codes as fp16 values, exactly: a code with its sign bit
// flipped is code + 128; as the low byte of 0x64xx it is the fp16 number
// 1024 + (code + 128), from which 1152 is subtracted. `u` holds flipped codes;
// kSel picks the two bytes (0x4140: bytes 0 and 1, 0x4342: bytes 2 and 3).
template <uint32_t kSel>
__device__ __forceinline__ uint32_t flipped_pair_to_half2(uint32_t u) {
  return half2_sub(byte_perm(u, 0x64646464u, kSel), 0x64806480u);
}

// Four codes of one word (bytes 0..3) as two fp16 pairs.
template <int kFormat>
__device__ __forceinline__ void codes4_to_half2x2(uint32_t w, uint32_t& p01, uint32_t& p23) {
  if (kFormat == CSA_KV_INT8) {
    const uint32_t u = w ^ 0x80808080u;
    p01 = flipped_pair_to_half2<0x4140>(u);
    p23 = flipped_pair_to_half2<0x4342>(u);
  } else {
    p01 = e4m3x2_to_half2(w & 0xFFFFu);
    p23 = e4m3x2_to_half2(w >> 16);
  }
}

// Four codes of one word as two bf16 pairs, exactly. int8: 0x43xx with the code's
// byte as xx is, without bit 7, 128 + (its low 7 bits), and with bit 7 alone, which
// is the exponent's last, 128 or 256: their difference is the code.
__device__ __forceinline__ uint32_t bf162_sub(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <int kFormat>
__device__ __forceinline__ void codes4_to_bf162x2(uint32_t w, uint32_t& p01, uint32_t& p23) {
  if (kFormat == CSA_KV_INT8) {
    const uint32_t t = byte_perm(w, 0x43434343u, 0x4140), u = byte_perm(w, 0x43434343u, 0x4342);
    p01 = bf162_sub(t & 0xFF7FFF7Fu, t & 0xFF80FF80u);
    p23 = bf162_sub(u & 0xFF7FFF7Fu, u & 0xFF80FF80u);
  } else {
    uint32_t h[2] = {e4m3x2_to_half2(w & 0xFFFFu), e4m3x2_to_half2(w >> 16)};
    uint32_t* to[2] = {&p01, &p23};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<__half2*>(&h[i]));
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(*to[i]) : "f"(f.y), "f"(f.x));
    }
  }
}

// The same four codes as fp32 values.
template <int kFormat>
__device__ __forceinline__ void codes4_to_float(uint32_t w, float (&f)[4]) {
  uint32_t a, b;
  codes4_to_half2x2<kFormat>(w, a, b);
  const float2 x = __half22float2(*reinterpret_cast<__half2*>(&a));
  const float2 y = __half22float2(*reinterpret_cast<__half2*>(&b));
  f[0] = x.x;
  f[1] = x.y;
  f[2] = y.x;
  f[3] = y.y;
}

}  // namespace csa
