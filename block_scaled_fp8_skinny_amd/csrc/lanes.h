// Exchanges between the lanes of a wave in the vector unit, and the hand-over between workgroups. Not part of the public
// ABI.
#pragma once

#include "device.h"

namespace bsfp8 {
namespace {

// Lane exchanges in the vector unit (DPP inside a row of 16, then the row swaps): a tenth of the latency of
// an LDS permute, and these kernels' second launch is one long chain of them.
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
}
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ double dpp(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, (uint64_t)dpp<CTRL, ROWS>((uint32_t)(b >> 32)) << 32 | dpp<CTRL, ROWS>((uint32_t)b));
}
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ uint64_t dpp(uint64_t v) {
  return (uint64_t)dpp<CTRL, ROWS>((uint32_t)(v >> 32)) << 32 | dpp<CTRL, ROWS>((uint32_t)v);
}
constexpr int XOR1 = 0xB1, XOR2 = 0x4E, HALF_MIRROR = 0x141, MIRROR = 0x140, SHR = 0x110, BCAST15 = 0x142, BCAST31 = 0x143;

// f over all lanes of the wave, or of each LANES neighbours; f is associative and commutative
template <int LANES = 64, typename F>
__device__ __forceinline__ float wave_reduce(float v, F f) {
  auto step = [&](uint32_t o) { v = f(v, __uint_as_float(o)); };
  step(dpp<XOR1>(__float_as_uint(v)));
  step(dpp<XOR2>(__float_as_uint(v)));
  if constexpr (LANES >= 8) step(dpp<HALF_MIRROR>(__float_as_uint(v)));
  if constexpr (LANES >= 16) step(dpp<MIRROR>(__float_as_uint(v)));
  if constexpr (LANES >= 32) {
    auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = f(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  if constexpr (LANES >= 64) {
    auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = f(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  return v;
}
// the same of integers (whole wave)
template <typename F>
__device__ __forceinline__ uint32_t wave_reduce(uint32_t v, F f) {
  v = f(v, dpp<XOR1>(v));
  v = f(v, dpp<XOR2>(v));
  v = f(v, dpp<HALF_MIRROR>(v));
  v = f(v, dpp<MIRROR>(v));
  auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = f((uint32_t)r[0], (uint32_t)r[1]);
  r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return f((uint32_t)r[0], (uint32_t)r[1]);
}
__device__ __forceinline__ float wave_max(float v) {
  return wave_reduce(v, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ double from_lane(double v, int lane) {        // uniform lane
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)b, lane), hi = __builtin_amdgcn_readlane((uint32_t)(b >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ uint64_t from_lane(uint64_t v, int lane) {
  const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)v, lane), hi = __builtin_amdgcn_readlane((uint32_t)(v >> 32), lane);
  return (uint64_t)hi << 32 | lo;
}
template <typename T>
__device__ __forceinline__ T wave_scan(T v) {                           // inclusive; T: double, uint32_t or uint64_t
  v += dpp<SHR + 1>(v);
  v += dpp<SHR + 2>(v);
  v += dpp<SHR + 4>(v);
  v += dpp<SHR + 8>(v);
  v += dpp<BCAST15, 0xA>(v);
  v += dpp<BCAST31, 0xC>(v);
  return v;
}
__device__ __forceinline__ double wave_sum(double v) { return from_lane(wave_scan(v), 63); }
__device__ __forceinline__ uint64_t wave_sum(uint64_t v) { return from_lane(wave_scan(v), 63); }

// The arrival of a workgroup at a sequence's counter: true for the last of `n`, which sees what the others
// stored before theirs (whole workgroup). What is handed over is stored and
// loaded by relaxed device-scope atomics only, which pass the XCDs' L2s by, so it is enough that each wave
// waits for its stores' completion before the count: a release fence would also write back the whole L2 of
// the XCD, once per workgroup (32 sequences' chains over 131072 columns took 57 us with it).
__device__ __forceinline__ bool last_to_arrive(int* counter, int n, int* shared) {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (threadIdx.x == 0)
    *shared = __hip_atomic_fetch_add(counter, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == n - 1;
  __syncthreads();
  return *shared != 0;
}

}  // namespace
}  // namespace bsfp8
