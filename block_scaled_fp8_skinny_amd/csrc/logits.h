// Rows of logits and their 64-bit weights, shared by the verification of drafts and the sampling (verify.hip, sample.hip).
// Not part of the public ABI.
#pragma once

#include "lanes.h"

namespace bsfp8 {
namespace {

constexpr int PIECE = 1024;                         // elements a wave holds: 16 per lane

// The element type's 16-byte vectors, and how many a piece has per lane.
template <typename T> struct Vec;
template <> struct Vec<float> {
  static constexpr int E = 4, N = PIECE / 256;
  static __device__ __forceinline__ void get(const u32x4_t& r, float (&x)[E]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(r[i]);
  }
};
template <> struct Vec<uint16_t> {
  static constexpr int E = 8, N = PIECE / 512;
  static __device__ __forceinline__ void get(const u32x4_t& r, float (&x)[E]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(r[i] << 16);
      x[2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
    }
  }
};

constexpr float NEG_INF = -__builtin_inff();

// What a lane loads of a vector: its 16 bytes and, in a bf16 row that starts in the middle of a 4-byte word, the word
// after them.
struct Words {
  u32x4_t w;
  uint32_t next;
};

// A wave's view of one row of V elements: word w, element i is row element w * E + i wherever the row starts in memory, so
// that rows of equal logits are summed in the same order and their probabilities cancel. Buffer loads need 4-byte
// addresses; a bf16 row of an odd start is read from the element before it and shifted by half a word. Elements
// past the row's end (the neighbouring row's) read as -inf. The descriptor ends with the row's last whole 4-byte word, so
// nothing past the row is read; a bf16 row's last element in half a word is read by itself.
template <typename T>
struct Row {
  static constexpr int E = Vec<T>::E, N = Vec<T>::N;
  __amdgpu_buffer_rsrc_t r;
  int V;
  bool odd, half;
  float last;
  // the V_ elements from element `first` of base (16-byte aligned)
  __device__ __forceinline__ Row(const void* base, int64_t first, int V_) : V(V_), odd(false), half(false), last(0.f) {
    const T* const at = reinterpret_cast<const T*>(base) + first;
    if constexpr (sizeof(T) == 2) {
      odd = first & 1;
      half = (odd + V_) & 1;
      if (half) last = __uint_as_float((uint32_t)at[V_ - 1] << 16);
    }
    r = __builtin_amdgcn_make_buffer_rsrc((void*)(at - odd), 0, (odd + V_) * (int)sizeof(T) & ~3, RSRC_WORD3);
  }
  __device__ __forceinline__ Words load(int piece, int lane, int v) const {
    const int at = index(piece, lane, v, 0) * (int)sizeof(T);
    Words w;
    w.w = __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0);
    w.next = 0;
    if constexpr (sizeof(T) == 2)
      if (odd) w.next = __builtin_amdgcn_raw_buffer_load_b32(r, at + 16, 0, 0);   // uniform
    return w;
  }
  __device__ __forceinline__ void load(int piece, int lane, Words (&w)[N]) const {
#pragma unroll
    for (int v = 0; v < N; ++v) w[v] = load(piece, lane, v);
  }
  __device__ __forceinline__ int index(int piece, int lane, int v, int i) const {
    return (piece * (PIECE / E) + v * 64 + lane) * E + i;
  }
  // A vector's elements; outside the row: -inf. NaN stays (it loses every maximum, and weighs nothing).
  __device__ __forceinline__ void get(const Words& from, int piece, int lane, int v, float (&x)[E]) const {
    u32x4_t w = from.w;
    if constexpr (sizeof(T) == 2) {
      if (odd) {                                    // uniform
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __builtin_amdgcn_alignbit(i < 3 ? from.w[i + 1] : from.next, from.w[i], 16);
      }
    }
    Vec<T>::get(w, x);
    if ((piece + 1) * PIECE > V) {                  // the row's end (uniform)
      const int at = index(piece, lane, v, 0);
#pragma unroll
      for (int i = 0; i < E; ++i) x[i] = half && at + i == V - 1 ? last : at + i < V ? x[i] : NEG_INF;
    }
  }
  __device__ __forceinline__ void get(const Words (&w)[N], int piece, int lane, float (&x)[N][E]) const {
#pragma unroll
    for (int v = 0; v < N; ++v) get(w[v], piece, lane, v, x[v]);
  }
};

template <typename T>
__device__ __forceinline__ float element(const void* base, int64_t at) {
  if constexpr (sizeof(T) == 4) return reinterpret_cast<const float*>(base)[at];
  else return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(base)[at] << 16);
}

// exp(y) = 2^n 2^(j/64) e^r with y = (64 n + j) ln2 / 64 + r: the table's 64 powers (in LDS) and the Taylor
// polynomial of degree 5 (|r| <= ln2 / 128, next term below 2^-54). Some 20 instructions, where the
// library's exp takes three times as many.
__device__ const double POWERS[64] = {
    0x1.0000000000000p+0, 0x1.02c9a3e778061p+0, 0x1.059b0d3158574p+0, 0x1.0874518759bc8p+0,
    0x1.0b5586cf9890fp+0, 0x1.0e3ec32d3d1a2p+0, 0x1.11301d0125b51p+0, 0x1.1429aaea92de0p+0,
    0x1.172b83c7d517bp+0, 0x1.1a35beb6fcb75p+0, 0x1.1d4873168b9aap+0, 0x1.2063b88628cd6p+0,
    0x1.2387a6e756238p+0, 0x1.26b4565e27cddp+0, 0x1.29e9df51fdee1p+0, 0x1.2d285a6e4030bp+0,
    0x1.306fe0a31b715p+0, 0x1.33c08b26416ffp+0, 0x1.371a7373aa9cbp+0, 0x1.3a7db34e59ff7p+0,
    0x1.3dea64c123422p+0, 0x1.4160a21f72e2ap+0, 0x1.44e086061892dp+0, 0x1.486a2b5c13cd0p+0,
    0x1.4bfdad5362a27p+0, 0x1.4f9b2769d2ca7p+0, 0x1.5342b569d4f82p+0, 0x1.56f4736b527dap+0,
    0x1.5ab07dd485429p+0, 0x1.5e76f15ad2148p+0, 0x1.6247eb03a5585p+0, 0x1.6623882552225p+0,
    0x1.6a09e667f3bcdp+0, 0x1.6dfb23c651a2fp+0, 0x1.71f75e8ec5f74p+0, 0x1.75feb564267c9p+0,
    0x1.7a11473eb0187p+0, 0x1.7e2f336cf4e62p+0, 0x1.82589994cce13p+0, 0x1.868d99b4492edp+0,
    0x1.8ace5422aa0dbp+0, 0x1.8f1ae99157736p+0, 0x1.93737b0cdc5e5p+0, 0x1.97d829fde4e50p+0,
    0x1.9c49182a3f090p+0, 0x1.a0c667b5de565p+0, 0x1.a5503b23e255dp+0, 0x1.a9e6b5579fdbfp+0,
    0x1.ae89f995ad3adp+0, 0x1.b33a2b84f15fbp+0, 0x1.b7f76f2fb5e47p+0, 0x1.bcc1e904bc1d2p+0,
    0x1.c199bdd85529cp+0, 0x1.c67f12e57d14bp+0, 0x1.cb720dcef9069p+0, 0x1.d072d4a07897cp+0,
    0x1.d5818dcfba487p+0, 0x1.da9e603db3285p+0, 0x1.dfc97337b9b5fp+0, 0x1.e502ee78b3ff6p+0,
    0x1.ea4afa2a490dap+0, 0x1.efa1bee615a27p+0, 0x1.f50765b6e4540p+0, 0x1.fa7c1819e90d8p+0,
};
__device__ __forceinline__ void load_powers(double* lds) {
  if (threadIdx.x < 64) lds[threadIdx.x] = POWERS[threadIdx.x];
}

// Weights exp((x - M) / t) of one row, for x <= M. it = 1 / t.
struct Weights {
  double c;                                         // 64 it / ln2
  float M;
  const double* powers;
  __device__ __forceinline__ Weights(float M_, double it, const double* powers_) : M(M_), powers(powers_) {
    c = it * 0x1.71547652b82fep+6;                  // 64 / ln 2
  }
  // never 0: what is too small (also -inf and NaN) gives 2^-1022, which no sum with a maximum of 1 notices
  __device__ __forceinline__ double some(float x) const {
    const double z = fmax(((double)x - (double)M) * c, -1022.0 * 64);
    const double t = z + 0x1.8p52, r = z - (t - 0x1.8p52);
    const int n = (int)(uint32_t)__builtin_bit_cast(uint64_t, t);
    double q = fma(r, 0x1.5d87fe78a6731p-40, 0x1.3b2ab6fba4e77p-31);
    q = fma(r, q, 0x1.c6b08d704a0c0p-23);
    q = fma(r, q, 0x1.ebfbdff82c58fp-15);
    q = fma(r, q, 0x1.62e42fefa39efp-7);
    const double w = powers[n & 63];
    const uint64_t b = __builtin_bit_cast(uint64_t, fma(w, r * q, w));
    return __builtin_bit_cast(double, b + ((uint64_t)(uint32_t)(n >> 6) << 52));
  }
  // 0 for -inf, NaN and what falls below 2^-1000; 1 for the maximum itself (also an infinite one)
  __device__ __forceinline__ double operator()(float x) const {
    const double w = some(x);
    return x == M ? 1.0 : w > 0x1p-1000 ? w : 0.0;
  }
};

// 1 / t (0 for an infinite one: equal weights), or -1 for a greedy row (t = 0, negative or NaN).
__device__ __forceinline__ double inv_temperature(float t) { return t > 0.f ? 1.0 / (double)t : -1.0; }
__device__ __forceinline__ bool is_greedy(double it) { return it < 0; }

}  // namespace
}  // namespace bsfp8
