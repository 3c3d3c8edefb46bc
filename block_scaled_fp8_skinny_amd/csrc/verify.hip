// Verification of drafted tokens for gfx950 (MI355X): acceptance of a chain by the ratio of target to
// draft probability, with the residual distribution at the first refusal, and the walk down a tree by
// the tokens that its nodes sample.
//
// Every probability is exp((x - M) / t) / S with the row's maximum M and sum S. A row of logits is cut
// into pieces of PIECE elements, one per wave, that stay in registers: the wave finds the piece's own
// maximum m and sum s = sum exp((x - m) / t) and stores the pair, so the logits are read once; a
// row's M and S follow from its pieces' pairs (S = sum of s * exp((m - M) / t)). A sampled token is then
// found in two steps, the piece from the pairs' running sums, the element by one more look at that
// piece alone. Which element a running sum passes is decided between neighbouring sums of up to 2^17
// terms, so exponentials and sums are fp64.
//
// Two launches, the second starting from the pairs:
//   chain   every workgroup of a sequence repeats the few acceptance tests; after a refusal each wave
//           sums max(p - q, 0) over its piece, and the workgroup that arrives last (a counter per
//           sequence, zeroed by the first launch) picks the token. Otherwise the sequence's first workgroup picks.
//   tree    one wave per node samples its token; the sequence's last workgroup walks down.
// Times: 32 chains of 6 over 131072 columns, 36 us for the pairs (184 MB at 5.1 TB/s, the vector ALUs 84% busy with the
// exponentials: bf16 logits take as long) and 18 for the rest, of which 8 are its chain of dependent loads (a single chain's
// 8.3) and the others the second look at the refused rows; 16 trees of 32 nodes over 32768 columns 15 and 6.5 us.
#include "device.h"

namespace bsfp8 {
namespace {

constexpr int PIECE = 1024;                         // elements a wave holds: 16 per lane
constexpr int MAX_T = 64;

struct Pair {                                       // one piece of a row: 16 bytes
  double s;
  float m;
  float pad;
};

struct VerifyParams {
  const void *logits, *draft;
  const int32_t *tokens, *parents;
  const float *temperature, *u, *u_sample;
  int* counters;                                    // [B]: workgroups of the second launch that have arrived
  Pair* pairs;                                      // [rows][pieces]: the target's rows, then the draft's
  double* rest;                                     // [B][pieces][vectors]: sums of a refused row; a tree's tokens [B][T]
  int32_t *out_tokens, *path, *n_accepted;
  int B, T, V, pieces;
  int share;                                        // vectors of a refused row that a wave sums: 1, or a whole piece's
};

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
  __device__ __forceinline__ Row(const void* base, int64_t row, int V_) : V(V_), odd(false), half(false), last(0.f) {
    const int64_t first = row * V_;
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
constexpr int XOR1 = 0xB1, XOR2 = 0x4E, HALF_MIRROR = 0x141, MIRROR = 0x140, SHR = 0x110, BCAST15 = 0x142, BCAST31 = 0x143;

// f over all lanes of the wave; f is associative and commutative
template <typename F>
__device__ __forceinline__ float wave_reduce(float v, F f) {
  auto step = [&](uint32_t o) { v = f(v, __uint_as_float(o)); };
  step(dpp<XOR1>(__float_as_uint(v)));
  step(dpp<XOR2>(__float_as_uint(v)));
  step(dpp<HALF_MIRROR>(__float_as_uint(v)));
  step(dpp<MIRROR>(__float_as_uint(v)));
  auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = f(__uint_as_float(r[0]), __uint_as_float(r[1]));
  r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return f(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float wave_max(float v) {
  return wave_reduce(v, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ double from_lane(double v, int lane) {        // uniform lane
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)b, lane), hi = __builtin_amdgcn_readlane((uint32_t)(b >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_scan(double v) {                 // inclusive
  v += dpp<SHR + 1>(v);
  v += dpp<SHR + 2>(v);
  v += dpp<SHR + 4>(v);
  v += dpp<SHR + 8>(v);
  v += dpp<BCAST15, 0xA>(v);
  v += dpp<BCAST31, 0xC>(v);
  return v;
}
__device__ __forceinline__ double wave_sum(double v) { return from_lane(wave_scan(v), 63); }

// 1 / t (0 for an infinite one: equal weights), or -1 for a greedy row (t = 0, negative or NaN).
__device__ __forceinline__ double inv_temperature(float t) { return t > 0.f ? 1.0 / (double)t : -1.0; }
__device__ __forceinline__ bool is_greedy(double it) { return it < 0; }

// The pairs of every piece of every row (blockIdx.x; rows of sequence b: the target's b * T + i, then the
// draft's B * T + b * (T - 1) + i).
template <typename T>
__global__ void __launch_bounds__(256) verify_pairs_kernel(VerifyParams p) {
  constexpr int E = Row<T>::E, N = Row<T>::N;
  __shared__ double powers[64];
  const int lane = threadIdx.x & 63;
  const int piece = blockIdx.y * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row = blockIdx.x, targets = p.B * p.T;
  // (not left at zero by the last call instead: where they lie depends on its sizes)
  if (row < p.B && blockIdx.y == 0 && threadIdx.x == 0) p.counters[row] = 0;
  const bool is_draft = row >= targets;
  const int local = is_draft ? row - targets : row;
  const Row<T> r(is_draft ? p.draft : p.logits, local, p.V);
  Words w[N];
  r.load(piece, lane, w);                           // (past the row's end: nothing is read)
  load_powers(powers);
  const int b = is_draft ? local / (p.T - 1) : local / p.T;
  const double it = inv_temperature(p.temperature[b]);
  __syncthreads();
  if (piece >= p.pieces) return;
  float x[N][E];
  r.get(w, piece, lane, x);
  float m = NEG_INF;
#pragma unroll
  for (int v = 0; v < N; ++v)
#pragma unroll
    for (int i = 0; i < E; ++i) m = fmaxf(m, x[v][i]);
  m = wave_max(m);
  double s = 0;
  if (!is_greedy(it) && m > NEG_INF) {
    if (m < -NEG_INF) {
      const Weights f(m, it, powers);
#pragma unroll
      for (int v = 0; v < N; ++v)
#pragma unroll
        for (int i = 0; i < E; ++i) s += f.some(x[v][i]);
    } else {
#pragma unroll
      for (int v = 0; v < N; ++v)
#pragma unroll
        for (int i = 0; i < E; ++i) s += x[v][i] == m ? 1.0 : 0.0;
    }
    s = wave_sum(s);
  }
  if (lane == 0) p.pairs[(int64_t)row * p.pieces + piece] = Pair{s, m, 0.f};
}

// Maximum and sum of a row from its pairs (whole wave). `first` holds pairs `lane` and `lane` + 64, asked for by the
// caller ahead: the only ones of up to 2^17 elements.
struct Total {
  float M;
  double S;
};
struct Pairs {
  Pair a, b;
};
__device__ __forceinline__ Pairs first_pairs(const Pair* pr, int pieces, int lane) {
  const Pair none{0, NEG_INF, 0.f};
  return Pairs{lane < pieces ? pr[lane] : none, lane + 64 < pieces ? pr[lane + 64] : none};
}
__device__ __forceinline__ Total row_total(const Pair* pr, const Pairs& first, int pieces, int lane, double it,
                                           const double* powers) {
  float M = fmaxf(first.a.m, first.b.m);
  for (int i = lane + 128; i < pieces; i += 64) M = fmaxf(M, pr[i].m);
  M = wave_max(M);
  double S = 0;
  if (!is_greedy(it) && M > NEG_INF) {
    const Weights f(M, it, powers);
    S = first.a.s * f(first.a.m) + first.b.s * f(first.b.m);
    for (int i = lane + 128; i < pieces; i += 64) S += pr[i].s * f(pr[i].m);
    S = wave_sum(S);
  }
  return Total{M, S};
}

// The first piece whose running sum passes `target` (whole wave; f(i) = the sum of piece i), the
// last piece with a positive sum if rounding leaves none; `before` = the running sum before it.
template <typename F>
__device__ __forceinline__ int pick_piece(int pieces, int lane, double target, double& before, F f) {
  double base = 0, last_before = 0;
  int last = 0;
  for (int i0 = 0; i0 < pieces; i0 += 64) {
    const double v = i0 + lane < pieces ? f(i0 + lane) : 0.0;
    const double run = wave_scan(v);
    const uint64_t past = __ballot(v > 0 && base + run > target);
    const uint64_t some = __ballot(v > 0);
    const int at = past ? __builtin_ctzll(past) : some ? 63 - __builtin_clzll(some) : -1;
    if (at >= 0) {
      last = i0 + at;
      last_before = base + from_lane(run - v, at);
    }
    if (past) break;
    base += from_lane(run, 63);
  }
  before = last_before;
  return last;
}

// The first element of a piece whose running sum passes `target`, the last one of positive weight if
// rounding leaves none (whole wave; w = the lane's weights, in element order per vector).
template <int E, int N>
__device__ __forceinline__ int pick_element(const double (&w)[N][E], int lane, double target) {
  double base = 0;
  int found = -1, last = -1;
#pragma unroll
  for (int v = 0; v < N; ++v) {
    double own = 0;
#pragma unroll
    for (int i = 0; i < E; ++i) own += w[v][i];
    const double run = wave_scan(own);
    double c = base + (run - own);
    int hit = -1, pos = -1;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      c += w[v][i];
      pos = w[v][i] > 0 ? i : pos;
      hit = hit < 0 && w[v][i] > 0 && c > target ? i : hit;
    }
    const uint64_t hits = __ballot(hit >= 0), some = __ballot(pos >= 0);
    if (found < 0 && hits) {
      const int l = __builtin_ctzll(hits);
      found = (v * 64 + l) * E + __builtin_amdgcn_readlane(hit, l);
    }
    if (some) {
      const int l = 63 - __builtin_clzll(some);
      last = (v * 64 + l) * E + __builtin_amdgcn_readlane(pos, l);
    }
    base += from_lane(run, 63);
  }
  return found >= 0 ? found : last;
}

// The lowest index of the row's largest logit (whole wave).
template <typename T>
__device__ __forceinline__ int pick_greedy(const Row<T>& r, const Pair* pr, int pieces, int lane, float M) {
  constexpr int E = Row<T>::E, N = Row<T>::N;
  if (!(M > NEG_INF)) return 0;
  int piece = 0;
  for (int i0 = 0; i0 < pieces; i0 += 64) {
    const uint64_t is = __ballot(i0 + lane < pieces && pr[min(i0 + lane, pieces - 1)].m == M);
    if (is) {
      piece = i0 + __builtin_ctzll(is);
      break;
    }
  }
  Words w[N];
  r.load(piece, lane, w);
  float x[N][E];
  r.get(w, piece, lane, x);
  for (int v = 0; v < N; ++v) {
    int at = E;
#pragma unroll
    for (int i = E - 1; i >= 0; --i) at = x[v][i] == M ? i : at;
    const uint64_t is = __ballot(at < E);
    if (is) {
      const int l = __builtin_ctzll(is);
      return r.index(piece, l, v, 0) + __builtin_amdgcn_readlane(at, l);
    }
  }
  return 0;
}

// A token from the row's own distribution (whole wave).
template <typename T>
__device__ __forceinline__ int pick_row(const Row<T>& r, const Pair* pr, int pieces, int lane, const Total& t, double it,
                                        float u, const double* powers) {
  constexpr int E = Row<T>::E, N = Row<T>::N;
  if (is_greedy(it)) return pick_greedy(r, pr, pieces, lane, t.M);
  if (!(t.M > NEG_INF)) return 0;
  const Weights f(t.M, it, powers);
  const double target = (double)u * t.S;
  double before;
  const int piece = pick_piece(pieces, lane, target, before, [&](int i) { return pr[i].s * f(pr[i].m); });
  Words raw[N];
  r.load(piece, lane, raw);
  float x[N][E];
  r.get(raw, piece, lane, x);
  double w[N][E];
#pragma unroll
  for (int v = 0; v < N; ++v)
#pragma unroll
    for (int i = 0; i < E; ++i) w[v][i] = f(x[v][i]);
  const int at = pick_element<E, N>(w, lane, target - before);
  return at < 0 ? 0 : r.index(piece, 0, 0, 0) + at;
}

// max(p - q, 0) of the lane's elements of a piece.
template <typename T>
struct Residual {
  static constexpr int E = Vec<T>::E, N = Vec<T>::N;
  Row<T> rp, rq;
  Weights fp, fq;
  double ip, iq;                                    // 1 / S
  __device__ __forceinline__ Residual(const VerifyParams& p, int64_t prow, int64_t qrow, const Total& tp, const Total& tq,
                                      double it, const double* powers)
      : rp(p.logits, prow, p.V), rq(p.draft, qrow, p.V), fp(tp.M, it, powers), fq(tq.M, it, powers) {
    ip = 1.0 / tp.S;
    iq = tq.S > 0 ? 1.0 / tq.S : 0.0;
  }
  // vector v of a piece: (a, b) = its words of both rows
  __device__ __forceinline__ void load(int piece, int lane, int v, Words& a, Words& b) const {
    a = rp.load(piece, lane, v);
    b = rq.load(piece, lane, v);
  }
  __device__ __forceinline__ void get(const Words& a, const Words& b, int piece, int lane, int v, double (&w)[E]) const {
    float x[E], y[E];
    rq.get(b, piece, lane, v, y);
    rp.get(a, piece, lane, v, x);
#pragma unroll
    for (int i = 0; i < E; ++i) {
#pragma clang fp contract(off)                       // equal rows must cancel: both products rounded alike
      w[i] = fmax(fp(x[i]) * ip - fq(y[i]) * iq, 0.0);
    }
  }
};

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

template <typename T>
__global__ void __launch_bounds__(256, 4) verify_chain_kernel(VerifyParams p) {
  __shared__ double powers[64];
  __shared__ Total totals[2 * MAX_T];
  __shared__ int shared_n, shared_last;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int b = blockIdx.x, D = p.T - 1;
  const double it = inv_temperature(p.temperature[b]);
  const bool greedy = is_greedy(it);
  const Pair* target_pairs = p.pairs + (int64_t)b * p.T * p.pieces;
  const Pair* draft_pairs = p.pairs + ((int64_t)p.B * p.T + (int64_t)b * D) * p.pieces;
  // draft i on lane i of wave 0: its logits in both rows, asked for before the totals
  int x = -1;
  float lp = NEG_INF, lq = NEG_INF, ui = 0.f;
  if (wave == 0 && lane < D) {
    x = p.tokens[(int64_t)b * D + lane];
    ui = p.u[(int64_t)b * D + lane];
    if (x >= 0 && x < p.V) {
      lp = element<T>(p.logits, ((int64_t)b * p.T + lane) * p.V + x);
      lq = element<T>(p.draft, ((int64_t)b * D + lane) * p.V + x);
    }
  }
  load_powers(powers);
  auto pairs_of = [&](int i) {
    return i < p.T ? target_pairs + (int64_t)i * p.pieces : draft_pairs + (int64_t)(i - p.T) * p.pieces;
  };
  constexpr int ROWS = 3;                           // rows of a wave whose pairs are asked for together
  const int rows = p.T + D;
  Pairs first[ROWS];
  auto ask = [&](int i0) {
#pragma unroll
    for (int j = 0; j < ROWS; ++j) first[j] = first_pairs(pairs_of(min(i0 + 4 * j, rows - 1)), p.pieces, lane);
  };
  ask(wave);
  __syncthreads();
  for (int i0 = wave; i0 < rows; i0 += 4 * ROWS) {
    if (i0 != wave) ask(i0);
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      const int i = i0 + 4 * j;
      if (i >= rows) break;
      const Total t = row_total(pairs_of(i), first[j], p.pieces, lane, it, powers);
      if (lane == 0) totals[i] = t;
    }
  }
  __syncthreads();
  if (wave == 0) {
    bool ok = false;
    if (lane < D && x >= 0 && x < p.V) {
      const Total tp = totals[lane], tq = totals[p.T + lane];
      if (greedy) {
        ok = lp == tp.M && tp.M > NEG_INF;          // a candidate: whether it is the lowest index is tested below
      } else if (tp.M > NEG_INF) {
        const double pp = Weights(tp.M, it, powers)(lp) / tp.S;
        const double pq = tq.M > NEG_INF ? Weights(tq.M, it, powers)(lq) / tq.S : 0.0;
        ok = (double)ui * pq < pp;
      }
    }
    const uint64_t oks = __ballot(ok);
    int n = 0;
    for (; n < D && (oks >> n & 1); ++n) {
      if (greedy) {
        const Row<T> r(p.logits, (int64_t)b * p.T + n, p.V);
        if (pick_greedy(r, target_pairs + (int64_t)n * p.pieces, p.pieces, lane, totals[n].M) !=
            __builtin_amdgcn_readlane(x, n))
          break;
      }
    }
    if (lane == 0) shared_n = n;
  }
  __syncthreads();
  const int n = __builtin_amdgcn_readfirstlane(shared_n);
  const int64_t prow = (int64_t)b * p.T + n;
  const Total tp = totals[n];
  int next = -1;
  if (n < D && !greedy && tp.M > NEG_INF) {         // a refusal
    const Residual<T> res(p, prow, (int64_t)b * D + n, tp, totals[p.T + n], it, powers);
    constexpr int E = Vec<T>::E, N = Vec<T>::N;
    double* rest = p.rest + (int64_t)b * p.pieces * N;   // a sum for every vector
    const int at0 = (blockIdx.y * 4 + wave) * p.share, piece = at0 / N, v0 = at0 % N;
    if (piece < p.pieces) {
      Words a[N], c[N];
#pragma unroll
      for (int v = 0; v < N; ++v)
        if (v < p.share) res.load(piece, lane, v0 + v, a[v], c[v]);
#pragma unroll
      for (int v = 0; v < N; ++v) {
        if (v >= p.share) break;
        double w[E], s = 0;
        res.get(a[v], c[v], piece, lane, v0 + v, w);
#pragma unroll
        for (int i = 0; i < E; ++i) s += w[i];
        s = wave_sum(s);
        if (lane == 0) __hip_atomic_store(rest + at0 + v, s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
    }
    if (!last_to_arrive(p.counters + b, gridDim.y, &shared_last) || wave != 0) return;
    const float us = p.u_sample[b];
    // lane l: the sums of pieces l and l + 64 (all there are of up to 2^17 elements), in registers for both looks
    double own[2][N];
    auto sum_of = [&](int i) {
      double t = 0;
#pragma unroll
      for (int v = 0; v < N; ++v) t += __hip_atomic_load(rest + i * N + v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      return t;
    };
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int v = 0; v < N; ++v)
        own[k][v] = lane + 64 * k < p.pieces ? __hip_atomic_load(rest + (lane + 64 * k) * N + v, __ATOMIC_RELAXED,
                                                                 __HIP_MEMORY_SCOPE_AGENT)
                                             : 0.0;
    double both[2] = {0, 0};
#pragma unroll
    for (int v = 0; v < N; ++v) {
      both[0] += own[0][v];
      both[1] += own[1][v];
    }
    double total = both[0] + both[1];
    for (int i = lane + 128; i < p.pieces; i += 64) total += sum_of(i);
    total = wave_sum(total);
    if (total > 0) {
      const double target = (double)us * total;
      double before;
      const int at = pick_piece(p.pieces, lane, target, before,
                                [&](int i) { return i < 64 ? both[0] : i < 128 ? both[1] : sum_of(i); });
      double left = target - before, start = left;  // the vector: the first that passes, or the last with a weight
      int v = 0;
      bool found = false;
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const double s = at < 64 ? from_lane(own[0][k], at) : at < 128 ? from_lane(own[1][k], at - 64)
                         : __hip_atomic_load(rest + at * N + k, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (s > 0 && !found) {
          v = k;
          start = left;
          found = s > left;
          left -= s;
        }
      }
      Words a, c;
      double w[1][E];
      res.load(at, lane, v, a, c);
      res.get(a, c, at, lane, v, w[0]);
      const int e = pick_element<E, 1>(w, lane, start);
      next = e < 0 ? 0 : res.rp.index(at, 0, v, 0) + e;
    }
  } else if (blockIdx.y != 0 || wave != 0) {
    return;
  }
  if (next < 0)
    next = pick_row(Row<T>(p.logits, prow, p.V), target_pairs + (int64_t)n * p.pieces, p.pieces, lane, tp, it, p.u_sample[b],
                    powers);
  if (lane < p.T) p.out_tokens[(int64_t)b * p.T + lane] = lane < n ? x : lane == n ? next : -1;
  if (lane == 0) p.n_accepted[b] = n;
}

// One node per wave; the sequence's last workgroup walks down.
template <typename T>
__global__ void __launch_bounds__(256) verify_tree_kernel(VerifyParams p) {
  __shared__ double powers[64];
  __shared__ int shared_last;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), b = blockIdx.x;
  const double it = inv_temperature(p.temperature[b]);
  int* sampled = reinterpret_cast<int*>(p.rest) + (int64_t)b * p.T;
  load_powers(powers);
  __syncthreads();
  const int i = blockIdx.y * 4 + wave;
  if (i < p.T) {
    const int64_t row = (int64_t)b * p.T + i;
    const Pair* pr = p.pairs + row * p.pieces;
    const float u = p.u[row];
    const Total t = row_total(pr, first_pairs(pr, p.pieces, lane), p.pieces, lane, it, powers);
    const int x = pick_row(Row<T>(p.logits, row, p.V), pr, p.pieces, lane, t, it, u, powers);
    if (lane == 0) __hip_atomic_store(sampled + i, x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  if (!last_to_arrive(p.counters + b, gridDim.y, &shared_last) || wave != 0) return;
  int parent = -1, token = -1, mine = -1;           // node `lane`'s
  if (lane < p.T) {
    mine = __hip_atomic_load(sampled + lane, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (lane > 0) {
      parent = p.parents[(int64_t)b * p.T + lane];
      token = p.tokens[(int64_t)b * p.T + lane];
      if (parent >= lane) parent = -1;
    }
  }
  int cur = 0, n = 0, out = -1, step = -1;          // lane n keeps the path's n-th node
  for (;;) {
    const int x = __builtin_amdgcn_readlane(mine, cur);
    if (lane == n) {
      out = x;
      step = cur;
    }
    const uint64_t child = __ballot(parent == cur && token == x);
    if (!child) break;
    cur = __builtin_ctzll(child);                   // above its parent: the walk ends
    ++n;
  }
  if (lane < p.T) {
    p.out_tokens[(int64_t)b * p.T + lane] = out;
    p.path[(int64_t)b * p.T + lane] = step;
  }
  if (lane == 0) p.n_accepted[b] = n;
}

inline int pieces_of(int64_t V) { return (int)((V + PIECE - 1) / PIECE); }
inline size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace

size_t verify_ws_bytes(int64_t B, int64_t T, int64_t V) {
  const size_t pieces = (size_t)pieces_of(V);
  return align256((size_t)B * 4) + align256((size_t)B * (2 * T - 1) * pieces * sizeof(Pair)) +
         (size_t)B * (pieces * 4 > 32 ? pieces * 4 : 32) * 8;   // at least T sampled tokens of a tree
}

int launch_verify(const VerifyArgs& a, bool tree, hipStream_t stream) {
  VerifyParams p{};
  p.logits = a.logits;
  p.draft = a.draft;
  p.tokens = a.tokens;
  p.parents = a.parents;
  p.temperature = a.temperature;
  p.u = a.u;
  p.u_sample = a.u_sample;
  p.B = (int)a.B;
  p.T = (int)a.T;
  p.V = (int)a.V;
  p.pieces = pieces_of(a.V);
  p.out_tokens = a.out_tokens;
  p.path = a.path;
  p.n_accepted = a.n_accepted;
  char* ws = reinterpret_cast<char*>(a.ws);
  p.counters = reinterpret_cast<int*>(ws);
  ws += align256((size_t)a.B * 4);
  p.pairs = reinterpret_cast<Pair*>(ws);
  ws += align256((size_t)a.B * (2 * a.T - 1) * p.pieces * sizeof(Pair));
  p.rest = reinterpret_cast<double*>(ws);
  // A refused row's second look by a wave for each vector while that keeps every workgroup in one round of the GPU (four
  // per CU): one chain over 32768 columns 11.7 us, by a wave for each piece 13.4; else a piece, since every workgroup
  // repeats the acceptance tests.
  const int vectors = a.f32 ? Vec<float>::N : Vec<uint16_t>::N;
  p.share = (int64_t)a.B * ((p.pieces * vectors + 3) / 4) <= 1024 ? 1 : vectors;
  const unsigned shares = (unsigned)((p.pieces * (vectors / p.share) + 3) / 4);
  const unsigned blocks = (unsigned)((p.pieces + 3) / 4);
  const unsigned rows = (unsigned)(tree ? a.B * a.T : a.B * (2 * a.T - 1));
  if (a.f32)
    hipLaunchKernelGGL(verify_pairs_kernel<float>, dim3(rows, blocks), dim3(256), 0, stream, p);
  else
    hipLaunchKernelGGL(verify_pairs_kernel<uint16_t>, dim3(rows, blocks), dim3(256), 0, stream, p);
  if (hipGetLastError() != hipSuccess) return BSFP8_EHIP;
  if (tree && a.f32)
    hipLaunchKernelGGL(verify_tree_kernel<float>, dim3((unsigned)a.B, (unsigned)((a.T + 3) / 4)), dim3(256), 0, stream, p);
  else if (tree)
    hipLaunchKernelGGL(verify_tree_kernel<uint16_t>, dim3((unsigned)a.B, (unsigned)((a.T + 3) / 4)), dim3(256), 0, stream, p);
  else if (a.f32)
    hipLaunchKernelGGL(verify_chain_kernel<float>, dim3((unsigned)a.B, shares), dim3(256), 0, stream, p);
  else
    hipLaunchKernelGGL(verify_chain_kernel<uint16_t>, dim3((unsigned)a.B, shares), dim3(256), 0, stream, p);
  return hip_status(hipGetLastError());
}

}  // namespace bsfp8
