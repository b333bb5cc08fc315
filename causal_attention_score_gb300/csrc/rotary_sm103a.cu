// Rotary positions on sm_103a: each pair (x0, x1) of a head's first rot_dim
// elements is turned by the angle p * f_i of its token's position p,
//
//   y0 = a (x0 cos - x1 sin),  y1 = a (x1 cos + x0 sin),
//
// with pairs (i, i + rot_dim/2) or (2i, 2i + 1); elements past rot_dim are
// copied. The gradient is the turn by the opposite angle.
//
// Angles. A position times a frequency in fp32 loses the angle of far
// positions (2^20 turns of the fastest pair leave 4 bits after the point), and
// fp64 arithmetic is slow on this GPU. The frequencies come as turns per
// position in 64-bit fixed point, F = round(f / 2pi * 2^64): the product p * F
// modulo 2^64, one integer multiplication, is the fraction of a turn itself,
// reduced exactly, off by at most |p| * 2^-65 turns. Its upper 32 bits become
// an angle in half turns for sincospif.
//
// Bound: HBM (one read and one write of x); sin and cos are computed once per
// (token, pair) and thread and shared by the heads that thread turns. A thread
// takes one slot (16 bytes of each half of the rotated part, or 16 bytes of
// interleaved pairs) of one token and kHeads heads.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <string>
#include <type_traits>

#include "csa_internal.h"
#include "sm103a_ptx.cuh"

namespace csa {
namespace {

constexpr int kRotThreads = 256;
constexpr int kHeads = 4;  // heads a thread turns with one set of sines

struct RotaryArgs {
  const void* x;
  void* out;
  long long x_token, x_head, out_token, out_head;  // strides in elements
  const unsigned long long* turns;                 // [rot_dim / 2], 2^-64 turns per position
  const int* positions;                            // nullptr: start + token % period
  long long tokens;
  long long items;
  int heads, rot_dim, head_size;
  int slots, rot_slots;  // per head: rotated slots, then copied ones
  int groups;            // head groups per token (kHeads heads each, groups apart)
  int start, period;
  float amplitude;
  int backward;
};

template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static __device__ __forceinline__ float get(float v) { return v; }
  static __device__ __forceinline__ float put(float v) { return v; }
};
template <>
struct Elem<__half> {
  static __device__ __forceinline__ float get(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half put(float v) { return __float2half_rn(v); }
};
template <>
struct Elem<__nv_bfloat16> {
  static __device__ __forceinline__ float get(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
};

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T e[V];
};

// One item: slot `slot` of token t in the heads h0, h0 + groups, ... The vector
// form (V elements of 16 bytes) needs 16-byte rows; V = 1 takes any layout.
template <typename T, int V, bool kInterleaved>
__global__ void __launch_bounds__(kRotThreads) rotary_sm103a_kernel(const RotaryArgs a) {
  grid_dependency_wait();
  // Interleaved pairs lie in one run of 2 elements or more; halves in two runs.
  constexpr int kRun = kInterleaved && V == 1 ? 2 : V;
  constexpr int kRuns = kInterleaved ? 1 : 2;
  constexpr int kPairs = kInterleaved ? kRun / 2 : V;
  using R = typename std::conditional<V == 1, T, Vec<T, V>>::type;
  constexpr int kLoads = V == 1 ? kRun : 1;  // loads per run

  const T* x = static_cast<const T*>(a.x);  // may be out itself
  T* out = static_cast<T*>(a.out);
  const long long step = static_cast<long long>(gridDim.x) * kRotThreads;
  for (long long it = static_cast<long long>(blockIdx.x) * kRotThreads + threadIdx.x; it < a.items;
       it += step) {
    const long long rest = it / a.slots;
    const int slot = static_cast<int>(it - rest * a.slots);
    const long long t = rest / a.groups;
    const int h0 = static_cast<int>(rest - t * a.groups);
    int pos;
    if (a.positions) {
      pos = a.positions[t];
      if (pos < 0) continue;  // padding
    } else {
      pos = a.start + static_cast<int>(a.period > 0 ? t % a.period : t);
    }
    const long long xt = t * a.x_token, ot = t * a.out_token;

    if (slot >= a.rot_slots) {  // elements past rot_dim
      const int d = a.rot_dim + (slot - a.rot_slots) * V;
#pragma unroll
      for (int k = 0; k < kHeads; ++k) {
        const int h = h0 + k * a.groups;
        if (h < a.heads)
          *reinterpret_cast<R*>(out + ot + h * a.out_head + d) =
              *reinterpret_cast<const R*>(x + xt + h * a.x_head + d);
      }
      continue;
    }

    const int d0 = slot * kRun;          // first element of the first run
    const int d1 = d0 + a.rot_dim / 2;   // of the second (halves)
    const int pair0 = kInterleaved ? d0 / 2 : d0;
    alignas(16) T in[kHeads][kRuns][kRun];
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
      const int h = h0 + k * a.groups;
      if (h >= a.heads) break;
#pragma unroll
      for (int r = 0; r < kRuns; ++r)
#pragma unroll
        for (int l = 0; l < kLoads; ++l)
          reinterpret_cast<R*>(in[k][r])[l] =
              *reinterpret_cast<const R*>(x + xt + h * a.x_head + (r ? d1 : d0) + l);
    }
    float c[kPairs], s[kPairs];
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const unsigned long long turn =
          static_cast<unsigned long long>(static_cast<long long>(pos)) * a.turns[pair0 + i];
      // the upper 32 bits as a signed fraction, in [-1, 1) half turns
      const float half = static_cast<float>(static_cast<int>(turn >> 32)) * 4.656612873077393e-10f;
      sincospif(half, &s[i], &c[i]);
      s[i] *= a.backward ? -a.amplitude : a.amplitude;
      c[i] *= a.amplitude;
    }
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
      const int h = h0 + k * a.groups;
      if (h >= a.heads) break;
      alignas(16) T y[kRuns][kRun];
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        const float x0 = Elem<T>::get(kInterleaved ? in[k][0][2 * i] : in[k][0][i]);
        const float x1 = Elem<T>::get(kInterleaved ? in[k][0][2 * i + 1] : in[k][kRuns - 1][i]);
        const T y0 = Elem<T>::put(x0 * c[i] - x1 * s[i]);
        const T y1 = Elem<T>::put(x1 * c[i] + x0 * s[i]);
        if (kInterleaved) {
          y[0][2 * i] = y0;
          y[0][2 * i + 1] = y1;
        } else {
          y[0][i] = y0;
          y[kRuns - 1][i] = y1;
        }
      }
#pragma unroll
      for (int r = 0; r < kRuns; ++r)
#pragma unroll
        for (int l = 0; l < kLoads; ++l)
          *reinterpret_cast<R*>(out + ot + h * a.out_head + (r ? d1 : d0) + l) =
              reinterpret_cast<const R*>(y[r])[l];
    }
  }
}

template <typename T, bool kInterleaved>
cudaError_t launch_rotary(const RotaryArgs& a, bool vector, unsigned grid, cudaStream_t stream) {
  constexpr int V = 16 / sizeof(T);
  return vector ? launch_programmatic(rotary_sm103a_kernel<T, V, kInterleaved>, grid, kRotThreads,
                                      0, stream, a)
                : launch_programmatic(rotary_sm103a_kernel<T, 1, kInterleaved>, grid, kRotThreads,
                                      0, stream, a);
}

}  // namespace

int rotary_launch(const RotaryCall& call, cudaStream_t stream, const DeviceInfo& dev,
                  std::string& err) {
  RotaryArgs a;
  a.x = call.x;
  a.out = call.out;
  a.x_token = call.x_token;
  a.x_head = call.x_head;
  a.out_token = call.out_token;
  a.out_head = call.out_head;
  a.turns = reinterpret_cast<const unsigned long long*>(call.turns);
  a.positions = call.positions;
  a.tokens = call.tokens;
  a.heads = call.heads;
  a.rot_dim = call.rot_dim;
  a.head_size = call.head_size;
  a.start = call.start;
  a.period = call.period;
  a.amplitude = call.amplitude;
  a.backward = call.backward;
  const int esize = call.dtype == CSA_F32 ? 4 : 2;
  const int V = 16 / esize;
  auto rows16 = [&](const void* p, long long token, long long head) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && token % V == 0 && head % V == 0;
  };
  const bool in_place = call.out == call.x;
  const bool vector = rows16(call.x, call.x_token, call.x_head) &&
                      rows16(call.out, call.out_token, call.out_head) &&
                      (in_place || call.head_size % V == 0) &&
                      (call.interleaved ? call.rot_dim : call.rot_dim / 2) % V == 0;
  const int w = vector ? V : 1;
  a.rot_slots = call.interleaved ? call.rot_dim / std::max(w, 2) : call.rot_dim / 2 / w;
  a.slots = a.rot_slots + (in_place ? 0 : (call.head_size - call.rot_dim) / w);
  a.groups = (call.heads + kHeads - 1) / kHeads;
  a.items = call.tokens * a.groups * a.slots;
  const long long blocks = (a.items + kRotThreads - 1) / kRotThreads;
  const unsigned grid = static_cast<unsigned>(
      std::min<long long>(blocks, static_cast<long long>(dev.sm_count) * (2048 / kRotThreads)));
  cudaError_t e;
  if (call.dtype == CSA_F32)
    e = call.interleaved ? launch_rotary<float, true>(a, vector, grid, stream)
                         : launch_rotary<float, false>(a, vector, grid, stream);
  else if (call.dtype == CSA_F16)
    e = call.interleaved ? launch_rotary<__half, true>(a, vector, grid, stream)
                         : launch_rotary<__half, false>(a, vector, grid, stream);
  else
    e = call.interleaved ? launch_rotary<__nv_bfloat16, true>(a, vector, grid, stream)
                         : launch_rotary<__nv_bfloat16, false>(a, vector, grid, stream);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) {
    err = std::string("rotary: launch: ") + cudaGetErrorString(e);
    return CSA_ERR_LAUNCH;
  }
  return CSA_OK;
}

}  // namespace csa
