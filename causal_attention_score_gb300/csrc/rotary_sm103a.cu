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
// reduced exactly. It is off by |p| times what F is: 2^-65 turns by its own
// rounding, f 2^-51 / 2pi by f's, which is a double after a few operations (p f 2^-51
// radians: 2^-20 at f = 1 and p = 2^31, below the rounding to fp32 up to p f = 2^27).
// Its upper 32 bits become an angle in half turns for sincospif.
//
// Bound: HBM (one read and one write of x). A thread takes one slot (16 bytes of
// each half of the rotated part, or 16 bytes of interleaved pairs) of one token in
// several heads, 64 bytes that it asks for at once, and computes the sines of that slot
// once for all of them. Where that leaves SMs without work, a thread takes one head.
// 8192 x 24 heads of 64 in bf16: 10.3 us (4.9 TB/s); 8192 x 32 of 128 in fp32: 46 us
// (5.8 TB/s). With 128 bytes a thread and 80 registers: 11.5 and 51 us; with the sines
// before the loads and divisions for every item: 14.2 and 59 us.
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

constexpr int kRotThreads = 128;
// Heads that a thread turns with one set of sines: 64 bytes in flight.
template <int V, bool kInterleaved>
constexpr int kHeads = V == 1 ? 4 : kInterleaved ? 4 : 2;

struct RotaryArgs {
  const void* x;
  void* out;
  long long x_token, x_head, out_token, out_head;  // strides in elements
  const unsigned long long* turns;                 // [rot_dim / 2], 2^-64 turns per position
  const int* positions;                            // nullptr: start + token % period
  long long tokens;
  int heads, rot_dim, head_size;
  int slots, rot_slots;  // per head: rotated slots, then copied ones
  int groups;            // head groups per token (heads `groups` apart)
  long long step_t;      // threads of the grid, in items: tokens, groups, slots
  int step_g, step_slot;
  int start, period;
  float amplitude;
  int backward;
  int* status;
};

// Elements of type T in 32-bit words: one (fp32) or two.
template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static constexpr int kPerWord = 1;
  static __device__ __forceinline__ float get(float v) { return v; }
  static __device__ __forceinline__ float put(float v) { return v; }
};
template <>
struct Elem<__half> {
  static constexpr int kPerWord = 2;
  static __device__ __forceinline__ float get(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half put(float v) { return __float2half_rn(v); }
  static __device__ __forceinline__ void unpack(uint32_t w, float& lo, float& hi) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    lo = f.x;
    hi = f.y;
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};
template <>
struct Elem<__nv_bfloat16> {
  static constexpr int kPerWord = 2;
  static __device__ __forceinline__ float get(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
  static __device__ __forceinline__ void unpack(uint32_t w, float& lo, float& hi) {
    lo = __uint_as_float(w << 16);
    hi = __uint_as_float(w & 0xFFFF0000u);
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};

struct Sines {
  float s, c;
};
__device__ __forceinline__ void turn(float& x0, float& x1, const Sines& t) {
  const float y0 = x0 * t.c - x1 * t.s;
  x1 = x1 * t.c + x0 * t.s;
  x0 = y0;
}
// 16 bytes of each half: pairs (a's element, b's element).
template <typename T>
__device__ __forceinline__ void turn_halves(uint4& a, uint4& b, const Sines* t) {
  uint32_t* wa = reinterpret_cast<uint32_t*>(&a);
  uint32_t* wb = reinterpret_cast<uint32_t*>(&b);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (Elem<T>::kPerWord == 1) {
      float x0 = __uint_as_float(wa[i]), x1 = __uint_as_float(wb[i]);
      turn(x0, x1, t[i]);
      wa[i] = __float_as_uint(x0);
      wb[i] = __float_as_uint(x1);
    } else {
      float x0[2], x1[2];
      Elem<T>::unpack(wa[i], x0[0], x0[1]);
      Elem<T>::unpack(wb[i], x1[0], x1[1]);
      turn(x0[0], x1[0], t[2 * i]);
      turn(x0[1], x1[1], t[2 * i + 1]);
      wa[i] = Elem<T>::pack(x0[0], x0[1]);
      wb[i] = Elem<T>::pack(x1[0], x1[1]);
    }
  }
}
// 16 bytes of interleaved pairs.
template <typename T>
__device__ __forceinline__ void turn_neighbours(uint4& a, const Sines* t) {
  uint32_t* w = reinterpret_cast<uint32_t*>(&a);
  if constexpr (Elem<T>::kPerWord == 1) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float x0 = __uint_as_float(w[2 * i]), x1 = __uint_as_float(w[2 * i + 1]);
      turn(x0, x1, t[i]);
      w[2 * i] = __float_as_uint(x0);
      w[2 * i + 1] = __float_as_uint(x1);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float x0, x1;
      Elem<T>::unpack(w[i], x0, x1);
      turn(x0, x1, t[i]);
      w[i] = Elem<T>::pack(x0, x1);
    }
  }
}

// One item: slot `slot` of token t in the heads h0, h0 + groups, ... The vector
// form (V elements of 16 bytes) needs 16-byte rows; V = 1 takes any layout.
template <typename T, int V, bool kInterleaved>
__global__ void __launch_bounds__(kRotThreads, 8) rotary_sm103a_kernel(const RotaryArgs a) {
  grid_dependency_wait();
  constexpr int kRuns = kInterleaved ? 1 : 2;
  constexpr int kRun = V > 1 ? V : kInterleaved ? 2 : 1;  // elements of a run
  constexpr int kPairs = kRun * kRuns / 2;
  using R = typename std::conditional<V == 1, T, uint4>::type;
  constexpr int kLoads = V == 1 ? kRun : 1;  // loads a run
  const T* x = static_cast<const T*>(a.x);  // may be out itself
  T* out = static_cast<T*>(a.out);
  constexpr int kMost = kHeads<V, kInterleaved>;
  [[maybe_unused]] __shared__ int s_abort;
  [[maybe_unused]] const Watchdog wd{0, a.status, &s_abort};
  const unsigned first = blockIdx.x * kRotThreads + threadIdx.x;
  const unsigned rest = first / a.slots;
  int slot = static_cast<int>(first - rest * a.slots);
  long long t = rest / a.groups;
  int h0 = static_cast<int>(rest % a.groups);
  auto advance = [&] {
    slot += a.step_slot;
    h0 += a.step_g;
    t += a.step_t;
    if (slot >= a.slots) slot -= a.slots, ++h0;
    if (h0 >= a.groups) h0 -= a.groups, ++t;
  };
  for (; t < a.tokens; advance()) {
    if (!CSA_CHECK(t >= 0 && slot >= 0 && slot < a.slots && h0 >= 0 && h0 < a.groups &&
                       h0 < a.heads &&
                       (slot < a.rot_slots
                            ? (slot + 1) * kRun * kRuns <= a.rot_dim
                            : a.rot_dim + (slot - a.rot_slots + 1) * V <= a.head_size),
                   wd, kCheckTile))
      break;
    int pos;
    if (a.positions)
      pos = a.positions[t];
    else if (a.period <= 0)
      pos = a.start + static_cast<int>(t);
    else
      pos = a.start + static_cast<int>((t >> 32) == 0 ? static_cast<unsigned>(t) % a.period
                                                      : t % a.period);
    const long long xt = t * a.x_token, ot = t * a.out_token;

    if (slot >= a.rot_slots) {  // elements past rot_dim
      const int d = a.rot_dim + (slot - a.rot_slots) * V;
      R v[kMost];
#pragma unroll
      for (int k = 0; k < kMost; ++k) {
        const int h = h0 + k * a.groups;
        if (h < a.heads) v[k] = *reinterpret_cast<const R*>(x + xt + h * a.x_head + d);
      }
      if (pos < 0) continue;  // padding
#pragma unroll
      for (int k = 0; k < kMost; ++k) {
        const int h = h0 + k * a.groups;
        if (h < a.heads) *reinterpret_cast<R*>(out + ot + h * a.out_head + d) = v[k];
      }
      continue;
    }

    const int d0 = slot * kRun;         // first element of the first run
    const int d1 = d0 + a.rot_dim / 2;  // of the second (halves)
    const int pair0 = kInterleaved ? d0 / 2 : d0;
    R in[kMost][kRuns][kLoads];
#pragma unroll
    for (int k = 0; k < kMost; ++k) {
      const int h = h0 + k * a.groups;
      if (h >= a.heads) break;
#pragma unroll
      for (int r = 0; r < kRuns; ++r)
#pragma unroll
        for (int l = 0; l < kLoads; ++l)
          in[k][r][l] = reinterpret_cast<const R*>(x + xt + h * a.x_head + (r ? d1 : d0))[l];
    }
    if (pos < 0) continue;
    Sines sc[kPairs];
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const unsigned long long angle =
          static_cast<unsigned long long>(static_cast<long long>(pos)) * a.turns[pair0 + i];
      // the upper 32 bits as a signed fraction, in [-1, 1) half turns
      const float half = static_cast<float>(static_cast<int>(angle >> 32)) * 4.656612873077393e-10f;
      sincospif(half, &sc[i].s, &sc[i].c);
      sc[i].s *= a.backward ? -a.amplitude : a.amplitude;
      sc[i].c *= a.amplitude;
    }
#pragma unroll
    for (int k = 0; k < kMost; ++k) {
      const int h = h0 + k * a.groups;
      if (h >= a.heads) break;
      if constexpr (V == 1) {
        T& a0 = in[k][0][0];
        T& a1 = kInterleaved ? in[k][0][kLoads - 1] : in[k][kRuns - 1][0];
        float x0 = Elem<T>::get(a0), x1 = Elem<T>::get(a1);
        turn(x0, x1, sc[0]);
        a0 = Elem<T>::put(x0);
        a1 = Elem<T>::put(x1);
      } else if constexpr (kInterleaved) {
        turn_neighbours<T>(in[k][0][0], sc);
      } else {
        turn_halves<T>(in[k][0][0], in[k][kRuns - 1][0], sc);
      }
#pragma unroll
      for (int r = 0; r < kRuns; ++r)
#pragma unroll
        for (int l = 0; l < kLoads; ++l)
          reinterpret_cast<R*>(out + ot + h * a.out_head + (r ? d1 : d0))[l] = in[k][r][l];
    }
  }
}

template <typename T, int V, bool kInterleaved>
cudaError_t launch_rotary(RotaryArgs a, int sms, cudaStream_t stream) {
  constexpr int kMost = kHeads<V, kInterleaved>;
  constexpr int kPerSm = 8;  // resident: 64 registers a thread
  a.groups = (a.heads + kMost - 1) / kMost;
  if (a.tokens * a.groups * a.slots < static_cast<long long>(sms) * kRotThreads * 2)
    a.groups = a.heads;
  const long long blocks = (a.tokens * a.groups * a.slots + kRotThreads - 1) / kRotThreads;
  const unsigned grid = static_cast<unsigned>(
      std::min<long long>(blocks, static_cast<long long>(sms) * kPerSm));
  unsigned step = grid * kRotThreads;
  a.step_slot = static_cast<int>(step % a.slots);
  step /= a.slots;
  a.step_g = static_cast<int>(step % a.groups);
  a.step_t = step / a.groups;
  return launch_programmatic(rotary_sm103a_kernel<T, V, kInterleaved>, grid, kRotThreads, 0,
                             stream, a);
}

template <typename T>
cudaError_t launch_rotary(const RotaryArgs& a, bool vector, bool interleaved, int sms,
                          cudaStream_t stream) {
  constexpr int V = 16 / sizeof(T);
  if (interleaved)
    return vector ? launch_rotary<T, V, true>(a, sms, stream)
                  : launch_rotary<T, 1, true>(a, sms, stream);
  return vector ? launch_rotary<T, V, false>(a, sms, stream)
                : launch_rotary<T, 1, false>(a, sms, stream);
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
  a.status = dev.status_word;
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
  cudaError_t e =
      call.dtype == CSA_F32
          ? launch_rotary<float>(a, vector, call.interleaved, dev.sm_count, stream)
      : call.dtype == CSA_F16
          ? launch_rotary<__half>(a, vector, call.interleaved, dev.sm_count, stream)
          : launch_rotary<__nv_bfloat16>(a, vector, call.interleaved, dev.sm_count, stream);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) {
    err = std::string("rotary: launch: ") + cudaGetErrorString(e);
    return CSA_ERR_LAUNCH;
  }
  return CSA_OK;
}

}  // namespace csa
