// Attention of drafted tokens over the paged MXFP8 cache for gfx950 (MI355X).
//
// Decoding (one token a sequence), chains and trees alike. The rows of one key/value head
// are its (node, query head) pairs, g * T of them (g query heads share it). With s = q . k * scale in
// base 2 (scale * log2 e), a running reference m per row, and weights w = 2^(s - m):
//   l = sum w,  O = sum w V,  out = O / l,
// one pass over the positions; m only moves (to the largest score so far; O and l are rescaled) when a score
// passes it by more than HEADROOM, which bounds the weights.
//
// Products on bf16 MFMA (16x16x32), transposed so that nothing crosses lanes between them:
//   S^T = K Q^T: a lane ends with four tokens of one row, which in pairs of 16-token groups are just
//   the eight k-values that it has to supply of P^T in O^T += V^T P^T (the order of tokens inside a
//   product is free as long as both operands agree).
// K and V are rebuilt from codes and scale bytes to exact bf16 by the scaled conversions on their way
// from LDS into the operand registers; V's transposition is done there too: a lane reads, of each of
// its eight tokens, the codes of D/16 neighbouring values, and interleaves the converted pairs of two
// tokens (byte permutes).
//
// Two kernels, chosen by the rows g * T of a key/value head (attention_plan):
//   ring  up to 96 rows (64 above dim 128): a workgroup's waves share 16 to 48 rows and split their tokens in tiles of 32,
//         each wave with a ring of NS tiles in LDS that the LDS mode of global loads fills (codes are contiguous per 16
//         tokens of a page and head); waves only wait for their own loads, and are joined through LDS at an item's end.
//         Bound by HBM: the loop of a chain of 6 over 131072 positions (64 heads over 8 of dim 128) streams 6.2 TB/s by the
//         clock read in the kernel (a plain read of as much 6.2 to 6.6); 71 us in all (62 in a graph), of which 5 go before the
//         first tile is asked for, 10 to the waves' skew and join, 6 to the joining kernel.
//   wide  more rows: the waves split the rows and share the tokens, which are rebuilt once per workgroup (see there).
// Work is cut evenly over the grid: the units (the tokens that a workgroup's waves take in one step, of one head and row
// block) of all sequences, in order, are divided into equal runs, one per workgroup, so that ragged lengths leave nobody
// idle; a head that falls into several runs leaves partial (m, l, O) in the workspace for a joining kernel. Short contexts
// are not cut: a workgroup for each head and row block, one launch. A launch is as short as its code: the instruction
// cache starts cold, and 5 KB of straight code took 3 us (masks by single comparisons, sums unrolled per row block).
#include <initializer_list>

#include "device.h"

namespace bsfp8 {
namespace {

constexpr int TILE = 32;                            // tokens of a wave's tile
// Waves of the ring kernel's workgroup. A CU's LDS has rings for eight waves (dim <= 128) or four. Eight in one
// workgroup leave half as many partial results as two workgroups of four (a chain over 131072 positions, 48 rows: 75
// against 89 us); two workgroups hide each other's beginnings and ends, which counts for more where results are small
// (16 sequences' single tokens, dim 64: 25 against 29 us).
constexpr int ring_waves(int dim, int mt) { return dim == 128 && mt >= 2 ? 8 : 4; }
constexpr int ring_grid(int dim, int mt) { return dim <= 128 && ring_waves(dim, mt) == 4 ? 512 : 256; }
constexpr float HEADROOM = 8.f;                     // weights are at most 2^8
constexpr float M_NONE = -3.4028234664e38f;         // reference of a row that has seen nothing: no finite score is below it

struct AttnParams {
  const uint16_t* q;
  const uint8_t *kq, *ks, *vq, *vs;
  const int32_t *pages, *lens, *nodes;
  const int64_t* mask;
  uint16_t* out;
  float* part;                                      // [nwg][2][rows of a block][D]
  float2* stat;                                     // [nwg][2][rows of a block]: m, l
  int2* owners;                                     // [items]: the workgroups of an item's first and last unit
  int64_t ldq, ld_pages, n_pages;
  float scale2;                                     // |scale| * log2 e (1 for a scale of 0)
  uint32_t q_keep, q_flip;                          // the scale's sign, or a scale of 0, on the queries
  int B, T, hq, hkv, g, rows, mblocks, page, max_len, nwg;
  int br, unit, unit_shift, start_cost;             // rows of a block; tokens of a unit and their logarithm
  int direct;                                       // a workgroup for each item
  FastDiv dpage, dg;
};

__device__ __forceinline__ int seq_len(const AttnParams& p, int b) { return max(0, min(p.lens[b], p.max_len)); }
// Units of an item, and its length in the order that is cut into runs: `start_cost` more, what it costs a
// workgroup to begin another item in units (drain, join, queries, table, first tiles), so that runs that
// hold the beginnings of items get fewer of them.
__device__ __forceinline__ int seq_units(const AttnParams& p, int b) { return (seq_len(p, b) + p.unit - 1) >> p.unit_shift; }

__device__ __forceinline__ int seq_span(const AttnParams& p, int b) {
  const int n = seq_units(p, b);
  return n > 0 ? n + p.start_cost : 0;
}

// The run of units of workgroup w out of `total`: the first `rem` runs hold per + 1.
struct Runs {
  int per, rem;
  __device__ __forceinline__ Runs(int total, int nwg) : per(total / nwg), rem(total - (total / nwg) * nwg) {}
  __device__ __forceinline__ int start(int w) const { return w * per + min(w, rem); }
};

// Units before each sequence, per head and row block, by a scan over the batch (whole wave; lane l
// covers sequences l * c .. l * c + c - 1).
struct Batch {
  int c, incl, own, total;
  __device__ __forceinline__ Batch(const AttnParams& p, int lane) {
    c = (p.B + 63) >> 6;
    own = 0;
    for (int i = lane * c; i < min(lane * c + c, p.B); ++i) own += seq_span(p, i);
    incl = own;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(incl, o);
      if (lane >= o) incl += v;
    }
    total = __builtin_amdgcn_readfirstlane(__shfl(incl, 63));
  }
  // the sequence that holds unit v (< total); `before` = the units before it
  __device__ __forceinline__ int find(const AttnParams& p, int v, int& before) const {
    const int l = __builtin_ctzll(__ballot(v < incl));
    before = __builtin_amdgcn_readfirstlane(__shfl(incl, l) - __shfl(own, l));
    int b = l * c;
    for (;; ++b) {
      const int n = seq_span(p, b);
      if (v < before + n) return b;
      before += n;
    }
  }
};

// A workgroup's run [u, u_end), its first sequence b and the first unit of that (base); false for an empty run. Without
// splitting (direct) the run is an item; an item of an empty sequence has its outputs zeroed here.
template <int D>
__device__ __forceinline__ bool first_run(const AttnParams& p, int lane, int br, int& u, int& u_end, int& b, int& base) {
  const int ipb = p.hkv * p.mblocks;                // heads and row blocks of a sequence
  if (p.direct) {
    b = blockIdx.x / ipb;
    base = 0;
    const int item = blockIdx.x - b * ipb, span = seq_span(p, b);
    if (span == 0) {
      const int h = item / p.mblocks, m0 = (item - h * p.mblocks) * br, rows = min(br, p.rows - m0);
      for (int x = threadIdx.x; x < rows * (D / 8); x += blockDim.x) {
        const int m = m0 + x / (D / 8), nd = fdiv(m, p.dg);
        *reinterpret_cast<uint4*>(p.out + (((int64_t)b * p.T + nd) * p.hq + (int64_t)h * p.g + (m - nd * p.g)) * D +
                                  x % (D / 8) * 8) = make_uint4(0, 0, 0, 0);
      }
      return false;
    }
    u = item * span;
    u_end = u + span;
    return true;
  }
  const Batch batch(p, lane);
  const Runs runs(batch.total * ipb, p.nwg);
  u = runs.start(blockIdx.x);
  u_end = runs.start(blockIdx.x + 1);
  if (u >= u_end) return false;
  int before;
  b = batch.find(p, u / ipb, before);
  base = before * ipb;
  return true;
}

// Global loads in LDS mode (see lds_load16 of device.h): 64-bit addresses, as a cache passes 4 GiB. The
// base may come from a lane exchange or readfirstlane, so the five wait states that a vector-written
// scalar needs before a memory instruction reads it are spent here (s_nop 4).
__device__ __forceinline__ const uint8_t* uniform(const uint8_t* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return reinterpret_cast<const uint8_t*>((uint64_t)hi << 32 | lo);
}
// N loads of 1 KB from one base to N consecutive kilobytes of LDS
template <int N>
__device__ __forceinline__ void gload_lds16(const uint8_t* base, const uint32_t* off, lds_addr_t lds) {
  static_assert(N >= 1 && N <= 4, "up to four kilobytes");
  uint32_t saved;
  const uint32_t to = __builtin_amdgcn_readfirstlane(lds);
  base = uniform(base);
  if constexpr (N == 1)
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %3, %2\n\ts_mov_b32 m0, %0"
                 : "=&s"(saved) : "s"(to), "s"(base), "v"(off[0]) : "memory");
  else if constexpr (N == 2)
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %3, %2\n\t"
                 "s_add_i32 m0, m0, 0x400\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %4, %2\n\ts_mov_b32 m0, %0"
                 : "=&s"(saved) : "s"(to), "s"(base), "v"(off[0]), "v"(off[1]) : "memory", "scc");
  else if constexpr (N == 3)
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %3, %2\n\t"
                 "s_add_i32 m0, m0, 0x400\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %4, %2\n\t"
                 "s_add_i32 m0, m0, 0x400\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %5, %2\n\ts_mov_b32 m0, %0"
                 : "=&s"(saved) : "s"(to), "s"(base), "v"(off[0]), "v"(off[1]), "v"(off[2]) : "memory", "scc");
  else
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %3, %2\n\t"
                 "s_add_i32 m0, m0, 0x400\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %4, %2\n\t"
                 "s_add_i32 m0, m0, 0x400\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %5, %2\n\t"
                 "s_add_i32 m0, m0, 0x400\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %6, %2\n\ts_mov_b32 m0, %0"
                 : "=&s"(saved) : "s"(to), "s"(base), "v"(off[0]), "v"(off[1]), "v"(off[2]), "v"(off[3]) : "memory", "scc");
}
__device__ __forceinline__ void gload_lds4(const uint8_t* addr, lds_addr_t lds) {
  uint32_t saved;
  asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %2, off\n\ts_mov_b32 m0, %0"
               : "=&s"(saved) : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(addr) : "memory");
}

// Where the 16-token groups of a stretch of a sequence lie, in LDS: entry i = the group of tokens t0 + 16 i .., as its
// index among the cache's groups of all heads ((page, head) major, so its codes start at 16 D times that), or -1
// past the sequence's end and in a page that does not exist. Filled by the whole workgroup, with a barrier of the
// caller's before and after; table_absent, after it, says whether a group below the end is absent.
constexpr int TABLE = 512;                          // the last eight hold the waves' findings
constexpr int STRETCH = (TABLE - 8) * 16;
__device__ __forceinline__ bool fill_table(const AttnParams& p, int b, int h, int t0, int len, int32_t* table) {
  bool absent = false;
  for (int i = threadIdx.x; i < TABLE - 8; i += blockDim.x) {
    const int t = t0 + i * 16;
    int entry = -1;
    if (t < len) {
      const int at = fdiv(t, p.dpage), pg = p.pages[(int64_t)b * p.ld_pages + at];
      if (pg >= 0 && pg < p.n_pages) entry = (int)((((int64_t)pg * p.hkv + h) * p.page + (t - at * p.page)) >> 4);
      else absent = true;
    }
    table[i] = entry;
  }
  absent = __any(absent);
  if ((threadIdx.x & 63) == 0) table[TABLE - 8 + (threadIdx.x >> 6)] = absent;
  return absent;
}
__device__ __forceinline__ bool table_absent(bool mine, const int32_t* table) {
  int any = mine;
  for (int w = 0; w < (int)blockDim.x / 64; ++w) any |= table[TABLE - 8 + w];
  return __builtin_amdgcn_readfirstlane(any) != 0;
}

// Geometry of one 16-token group in LDS.
template <int D>
struct Geo {
  static constexpr int CODES = 16 * D;              // bytes of one group's codes
  static constexpr int SCALES = D / 2;              // bytes of one group's scales
  static constexpr int STAGE = 4 * CODES + 4 * SCALES;   // K0 K1 V0 V1, then their scales
  static constexpr int LOADS = D / 64;              // 1 KB loads per group
  static constexpr int SLOADS = (D + 127) / 128;    // 4-byte loads of a tile's scales
  static constexpr int PER_TILE = 4 * LOADS + SLOADS;
  // K row r keeps granule (16 bytes) x at place x ^ swizzle(r), so that the sixteen rows' granules that
  // one read fetches lie in different banks: eight rows span all 128-byte phases
  static __device__ __forceinline__ int swizzle(int r) { return D % 128 == 0 ? r & 7 : (r >> 1) & 3; }
};

// Offset in a group's codes of the 16 bytes that lane `lane` of load n fetches. K: row-major with the
// swizzle. V: the row of token t stands at (t % 4) * 4 + t / 4, so that the four tokens that the lane
// quarters read together are neighbours.
template <int D>
__device__ __forceinline__ uint32_t k_source(int n, int lane) {
  const int at = n * 1024 + lane * 16, row = at / D, slot = (at % D) / 16;
  return (uint32_t)(row * D + (slot ^ Geo<D>::swizzle(row)) * 16);
}
template <int D>
__device__ __forceinline__ uint32_t v_source(int n, int lane) {
  const int at = n * 1024 + lane * 16, row = at / D;
  return (uint32_t)(((row & 3) * 4 + (row >> 2)) * D + at % D);
}

// One dword of V's codes of each of the lane's eight tokens -> the A operands of four 16-row tiles
// (values d + 0..3 of the lane): pairs of tokens side by side.
__device__ __forceinline__ void v_operands(const uint32_t (&raw)[8], const float (&sc)[8], bf16x8_t (&a)[4]) {
  u32x4_t t[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t x0 = bits_of(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(raw[2 * j], sc[2 * j], false));
    const uint32_t x1 = bits_of(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(raw[2 * j], sc[2 * j], true));
    const uint32_t y0 = bits_of(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(raw[2 * j + 1], sc[2 * j + 1], false));
    const uint32_t y1 = bits_of(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(raw[2 * j + 1], sc[2 * j + 1], true));
    t[0][j] = __builtin_amdgcn_perm(y0, x0, 0x05040100u);
    t[1][j] = __builtin_amdgcn_perm(y0, x0, 0x07060302u);
    t[2][j] = __builtin_amdgcn_perm(y1, x1, 0x05040100u);
    t[3][j] = __builtin_amdgcn_perm(y1, x1, 0x07060302u);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = __builtin_bit_cast(bf16x8_t, t[i]);
}

// Value of the head that lane column x (0..15) of 16-row tile i stands for: a lane's tiles are D/16
// neighbouring values (for D = 192: eight of the first 128, then four of the last 64).
template <int D>
__device__ __forceinline__ int v_value(int x, int i) {
  if constexpr (D == 192) return i < 8 ? x * 8 + i : 128 + x * 4 + (i - 8);
  else return x * (D / 16) + i;
}

// NaN and infinite values of V (a, four operand tiles) must not reach rows that do not see their token,
// though 0 * NaN is NaN in the product: they are replaced by zeros here, and the rows that do see one
// (the product of the flags of such values with the flags of seen tokens is positive) get it added.
__device__ __forceinline__ uint32_t nonfinite(uint32_t v) {   // ones in the halves of a bf16 pair that are NaN or infinite
  return ((v & 0x7F80u) == 0x7F80u ? 0xFFFFu : 0u) | ((v & 0x7F800000u) == 0x7F800000u ? 0xFFFF0000u : 0u);
}
template <int MT>
__device__ __forceinline__ void flag_rows(bf16x8_t (&a)[4], const uint32_t (&sees)[MT], f32x4_t* o, int stride) {
#pragma unroll 1
  for (int kind = 0; kind < 3; ++kind) {            // infinity, its negative, NaN
    const float what = __uint_as_float(kind == 0 ? 0x7F800000u : kind == 1 ? 0xFF800000u : 0x7FC00000u);
    auto flag_of = [&](uint32_t h) {                // h: a bf16 value
      return (kind == 2 ? (h & 0x7FFFu) > 0x7F80u : h == (kind == 0 ? 0x7F80u : 0xFF80u)) ? 0x3F80u : 0u;
    };
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const u32x4_t v = __builtin_bit_cast(u32x4_t, a[k]);
      u32x4_t flag;
#pragma unroll
      for (int j = 0; j < 4; ++j) flag[j] = flag_of(v[j] & 0xFFFFu) | flag_of(v[j] >> 16) << 16;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        u32x4_t w;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          w[j] = ((sees[mt] >> (2 * j)) & 1 ? 0x3F80u : 0u) | ((sees[mt] >> (2 * j + 1)) & 1 ? 0x3F800000u : 0u);
        const f32x4_t n = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            __builtin_bit_cast(bf16x8_t, flag), __builtin_bit_cast(bf16x8_t, w), f32x4_t{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (n[r] > 0.f) o[mt * stride + k][r] += what;
      }
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    u32x4_t v = __builtin_bit_cast(u32x4_t, a[k]);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] &= ~nonfinite(v[j]);
    a[k] = __builtin_bit_cast(bf16x8_t, v);
  }
}
// Whether codes (of one 32-bit word a token) or their scales can give such values: a NaN code (all ones but the
// sign), a scale byte of 255, or one from 247, where 448 times the scale passes the largest bf16. (May say so of
// values that are finite, not the reverse.)
__device__ __forceinline__ bool maybe_nonfinite(const uint32_t (&raw)[8], const float (&sc)[8]) {
  uint32_t nan = 0, top = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    nan |= (raw[e] & 0x7F7F7F7Fu) + 0x01010101u;
    top = max(top, __float_as_uint(sc[e]) & 0x7F800000u);
  }
  return (nan & 0x80808080u) != 0 || top >= 247u << 23;
}

// Four bits, of tokens first .. first + 3 (counted from the sequence's first node): bit i is set where node `nd` sees
// the token. `word`: the node's mask; without masks (a chain) every token up to its own.
__device__ __forceinline__ uint32_t seen4(bool masks, uint64_t word, int nd, int first) {
  if (!masks) return first > nd ? 0u : 15u >> max(first + 3 - nd, 0);   // (28 at most when first <= nd)
  const uint32_t before = first >= 0 ? 0u : 15u >> max(first + 4, 0);   // the prefix: seen
  const int at = max(first, 0);
  return before | ((at < 64 ? (uint32_t)(word >> at) : 0u) << min(at - first, 31) & 15u);
}

// Scores of tokens that a row does not see: -inf, and its bit of `sees` cleared. s: two 16-token groups of MT
// row blocks, m = the lane's row of the first block, tok0 = its first token of the first group; exist: bit e is
// set where the lane's token e is below the sequence's end, in a page that exists.
template <int MT>
__device__ __forceinline__ void mask_scores(const AttnParams& p, int b, int m, int here, int prefix, int tok0, uint32_t exist,
                                            f32x4_t (&s)[2][MT], uint32_t (&sees)[MT]) {
  asm volatile("" : "+v"(m), "+v"(tok0));           // nothing of this is worth a register across the loop
#pragma unroll
  for (int mt = 0; mt < MT; ++mt, m += 16) {
    const int nd = m < p.rows ? fdiv(m, p.dg) : here;
    uint64_t word = 0;
    if (p.mask && nd < here) word = (uint64_t)p.mask[(int64_t)b * p.T + nd];
    const int first = tok0 - prefix;
    uint32_t see = seen4(p.mask != nullptr, word, nd, first) | seen4(p.mask != nullptr, word, nd, first + 16) << 4;
    see = nd < here ? see & exist : 0u;
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e >> 2][mt][e & 3] = see & (1u << e) ? s[e >> 2][mt][e & 3] : -__builtin_inff();
    sees[mt] = see;
  }
  // The compiler would else wait, after the branch that this stands in, for the loads above to land, on
  // the way without them too: and with them for the loads of the ring, which it does not know of.
  __builtin_amdgcn_s_waitcnt(0x0F70);               // vmcnt(0)
}

// The lane's eight tokens tok0 + 0..3 and + 16..19 that are there (see mask_scores).
__device__ __forceinline__ uint32_t existing(int tok0, int len, int pg0, int pg1) {
  const int left = len - tok0;
  const uint32_t low = pg0 < 0 || left <= 0 ? 0u : 15u >> max(4 - left, 0);
  const uint32_t high = pg1 < 0 || left <= 16 ? 0u : 15u >> max(20 - left, 0);
  return low | high << 4;
}

// The weights 2^(s - m) of MT row blocks' eight scores a lane (q . k, times scale2 for the base-2 score) as B operands, and
// their sums. The references move to the rows' largest scores when one of the wave's scores is more than 2^HEADROOM times
// its row's: rarely, so the exchange between lanes and the rescaling (rescale(mt, f): everything so far times f) are off
// the common path, and all exponentials come after the one branch (taking them first and testing their sums left 11
// register moves a row block, a sixth of the wide kernel's vector instructions).
// The weights are rounded to bf16 for the matrix product (at most half a step, 2^-8, each); the sum takes them
// unrounded.
template <int MT, typename R>
__device__ __forceinline__ void weights(const f32x4_t (&s)[2][MT], float scale2, float (&mref)[MT], float (&l)[MT],
                                        bf16x8_t (&pf)[MT], R rescale) {
  float x[MT][8];
  bool far = false;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[mt][e] = fmaf(s[e >> 2][mt][e & 3], scale2, -mref[mt]);
    float top = x[mt][0];
#pragma unroll
    for (int e = 1; e < 8; ++e) top = fmaxf(top, x[mt][e]);
    far = far || top > HEADROOM;
  }
  if (__builtin_expect(__any(far), 0)) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      float t = s[0][mt][0];
#pragma unroll
      for (int e = 1; e < 8; ++e) t = fmaxf(t, s[e >> 2][mt][e & 3]);
      t *= scale2;
      t = fmaxf(t, __shfl_xor(t, 16));
      t = fmaxf(t, __shfl_xor(t, 32));
      const float m = fmaxf(mref[mt], t), f = __builtin_amdgcn_exp2f(mref[mt] - m);
      mref[mt] = m;
      l[mt] *= f;
      rescale(mt, f);
      // the product rounded as the reference's was: fused, half a unit in the last place of a score of 2^32 is
      // left over, and 2 to that power may be infinite or leave nothing of the row
#pragma unroll
      for (int e = 0; e < 8; ++e) {
#pragma clang fp contract(off)
        x[mt][e] = s[e >> 2][mt][e & 3] * scale2 - m;
      }
    }
  }
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[mt][e] = __builtin_amdgcn_exp2f(x[mt][e]);
    l[mt] += ((x[mt][0] + x[mt][1]) + (x[mt][2] + x[mt][3])) + ((x[mt][4] + x[mt][5]) + (x[mt][6] + x[mt][7]));
    const u32x4_t w = {pack_bf16x2(x[mt][0], x[mt][1]), pack_bf16x2(x[mt][2], x[mt][3]), pack_bf16x2(x[mt][4], x[mt][5]),
                       pack_bf16x2(x[mt][6], x[mt][7])};
    pf[mt] = __builtin_bit_cast(bf16x8_t, w);
  }
}

// Scale factors (2^(byte - 127), in the exponent field; the conversions read nothing else of the operand,
// so the byte only has to be rotated there) of one 16-token group.
template <int D>
struct Scales {
  static constexpr int TB = D / 32;                 // bytes per token
  static __device__ __forceinline__ float rotated(uint32_t w, int byte) {
    return __uint_as_float(__builtin_amdgcn_alignbit(w, w, 8 * byte + 9));
  }
  // K: token r16, blocks 2j + half (j = 0 .. D/64 - 1)
  static __device__ __forceinline__ void k(const uint8_t* s, int r16, int half, float (&f)[D / 64]) {
    if constexpr (D == 256) {
      const uint2 w = *reinterpret_cast<const uint2*>(s + r16 * 8);
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = rotated(j < 2 ? w.x : w.y, 2 * (j & 1) + half);
    } else if constexpr (D == 128) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(s + r16 * 4);
#pragma unroll
      for (int j = 0; j < 2; ++j) f[j] = rotated(w, 2 * j + half);
    } else {
#pragma unroll
      for (int j = 0; j < D / 64; ++j) f[j] = rotated(*reinterpret_cast<const uint16_t*>(s + r16 * TB + 2 * j), half);
    }
  }
  // V: tokens q4 * 4 + 0..3, the block of the lane's values of operand tiles 4c .. 4c + 3
  static __device__ __forceinline__ void v(const uint8_t* s, int r16, int q4, int c, float* f) {
    if constexpr (D == 128) {
      const uint4 w = *reinterpret_cast<const uint4*>(s + q4 * 16);
      const uint32_t t[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = rotated(t[j], r16 >> 2);
    } else if constexpr (D == 64) {
      const uint2 w = *reinterpret_cast<const uint2*>(s + q4 * 8);
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = rotated(j < 2 ? w.x : w.y, 2 * (j & 1) + (r16 >> 3));
    } else if constexpr (D == 256) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        f[j] = rotated(*reinterpret_cast<const uint32_t*>(s + (q4 * 4 + j) * 8 + (r16 >> 3) * 4), (r16 >> 1) & 3);
    } else {
      const int block = c < 2 ? r16 >> 2 : 4 + (r16 >> 3);
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = block_scale(s[(q4 * 4 + j) * TB + block]);
    }
  }
};

template <int D, int MT, int NS>
__global__ void __launch_bounds__(64 * ring_waves(D, MT), D <= 128 ? 2 : 1) attention_kernel(AttnParams p) {
  using G = Geo<D>;
  constexpr int NW = ring_waves(D, MT), UNIT = NW * TILE;
  constexpr int ND = D / 16, NK = D / 32, BR = MT * 16;
  constexpr int RING = NW * NS * G::STAGE, RESULT = MT * ND * 1024;
  // waves that put their result into LDS for the join: all, or half of them after adding the other half's
  constexpr int HELD = NW * RESULT <= RING ? NW : NW / 2;
  static_assert(HELD * RESULT <= RING, "the results take the ring's place");
  static_assert((NS - 1) * G::PER_TILE <= 63, "vector memory counter range");
  static_assert(NW * 8 <= NK * 64, "the statistics take the queries' place");
  __shared__ __align__(16) uint8_t ring[RING];
  __shared__ __align__(16) uint4 queries[MT * NK * 64];   // B operands: row mt*16 + r16, values of K's operand order
  __shared__ __align__(16) int32_t table[TABLE];
  float2* const stats = reinterpret_cast<float2*>(queries);

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, q4 = lane >> 4;
  int u, u_end, b, base;
  if (!first_run<D>(p, lane, BR, u, u_end, b, base)) return;
  const int ipb = p.hkv * p.mblocks;                // heads and row blocks of a sequence
  const int first_u = u;

  uint32_t ksrc[G::LOADS], vsrc[G::LOADS];
#pragma unroll
  for (int n = 0; n < G::LOADS; ++n) {
    ksrc[n] = k_source<D>(n, lane);
    vsrc[n] = v_source<D>(n, lane);
  }
  uint8_t* const my_ring = ring + wave * NS * G::STAGE;

  while (u < u_end) {
    const int len = seq_len(p, b), units = (len + UNIT - 1) / UNIT, span = units + p.start_cost;
    const int item = (u - base) / span;             // head and row block
    const int va = (u - base) - item * span, vb = min(span, va + (u_end - u));
    const int ua = max(va - p.start_cost, 0), ub = vb - p.start_cost;
    const int h = item / p.mblocks, mb = item - h * p.mblocks;
    const int here = p.nodes ? max(0, min(p.nodes[b], p.T)) : p.T;
    const int prefix = len - here;

    if (ub <= ua) break;                            // the run ends in the item's cost
    // the queries and the first stretch of the table, asked for together
    __syncthreads();                                // the last item's ring, queries and statistics are done with
    int qw = wave;                                  // what follows from it is not worth keeping from item to item
    asm volatile("" : "+s"(qw));
    uint4 qv[(MT * NK + NW - 1) / NW];
#pragma unroll
    for (int k = 0; k < (MT * NK + NW - 1) / NW; ++k) {
      const int f = qw + k * NW, j = f % NK, m = mb * BR + f / NK * 16 + r16;   // fragment f: rows, values
      const int nd = fdiv(min(m, p.rows - 1), p.dg), hd = m - nd * p.g;
      qv[k] = make_uint4(0, 0, 0, 0);
      if (f < MT * NK && m < p.rows && nd < here)
        qv[k] = *reinterpret_cast<const uint4*>(p.q + ((int64_t)b * p.T + nd) * p.ldq + ((int64_t)h * p.g + hd) * D +
                                                (j >> 1) * 64 + q4 * 16 + (j & 1) * 8);
    }
    bool absent = fill_table(p, b, h, ua * UNIT, len, table);
    __syncthreads();
    absent = table_absent(absent, table);
    f32x4_t o[MT][ND];
    float mref[MT], l[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      mref[mt] = M_NONE;
      l[mt] = 0.f;
#pragma unroll
      for (int i = 0; i < ND; ++i) o[mt][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }

    for (int uc = ua; uc < ub;) {                   // as many units as the table covers
      const int uz = min(ub, uc + STRETCH / UNIT), tbase = uc * UNIT;
      if (uc != ua) {
        __syncthreads();                            // the table is free
        absent = fill_table(p, b, h, tbase, len, table);
        __syncthreads();
        absent = table_absent(absent, table);
      }
      const int t0 = tbase + wave * TILE;           // this wave's first token; then every UNIT
      const int nt = t0 < len ? min(uz - uc, (len - t0 + UNIT - 1) / UNIT) : 0;

      auto issue = [&](int i) {
        uint8_t* st = my_ring + (i % NS) * G::STAGE;
        const int2 en = *reinterpret_cast<const int2*>(table + ((t0 - tbase + i * UNIT) >> 4));
        // absent tokens: some group, not used
        const int64_t at[2] = {max(__builtin_amdgcn_readfirstlane(en.x), 0), max(__builtin_amdgcn_readfirstlane(en.y), 0)};
#pragma unroll
        for (int gr = 0; gr < 2; ++gr) {
          gload_lds16<G::LOADS>(p.kq + at[gr] * (16 * D), ksrc, lds_addr(st + gr * G::CODES));
          gload_lds16<G::LOADS>(p.vq + at[gr] * (16 * D), vsrc, lds_addr(st + (2 + gr) * G::CODES));
        }
        constexpr int Q = D / 8;                    // dwords of one group's scales
#pragma unroll
        for (int n = 0; n < G::SLOADS; ++n) {
          const int e = n * 64 + lane, quarter = e / Q;
          const uint8_t* a = (quarter & 2 ? p.vs : p.ks) + (quarter & 1 ? at[1] : at[0]) * (D / 2);
          if (e < 4 * Q) gload_lds4(a + (e - quarter * Q) * 4, lds_addr(st + 4 * G::CODES + n * 256));
        }
      };
      auto compute = [&](int i) {
        const uint8_t* st = my_ring + (i % NS) * G::STAGE;
        const uint8_t* scales = st + 4 * G::CODES;
        const int t = t0 + i * UNIT;
        // a tile that some row may not see whole: nodes, the sequence's end, absent pages (uniform)
        const bool special = t + TILE > min(prefix, len) || absent;
        const int* pg = table + ((t - tbase) >> 4);   // the groups' entries: below 0, no tokens (special tiles)
        f32x4_t s[2][MT];
        float kf[2][D / 64];
#pragma unroll
        for (int gr = 0; gr < 2; ++gr) {
          Scales<D>::k(scales + gr * G::SCALES, r16, q4 >> 1, kf[gr]);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) s[gr][mt] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        }
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
          bf16x8_t a[2][2];
#pragma unroll
          for (int gr = 0; gr < 2; ++gr) {
            const uint4 w = *reinterpret_cast<const uint4*>(st + gr * G::CODES + r16 * D +
                                                            (((4 * j + q4) ^ G::swizzle(r16)) * 16));
            a[gr][0] = dequant8(w.x, w.y, kf[gr][j]);
            a[gr][1] = dequant8(w.z, w.w, kf[gr][j]);
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const bf16x8_t qf = __builtin_bit_cast(bf16x8_t, queries[(mt * NK + 2 * j + e) * 64 + lane]);
#pragma unroll
              for (int gr = 0; gr < 2; ++gr)
                s[gr][mt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[gr][e], qf, s[gr][mt], 0, 0, 0);
            }
        }
        // tokens of the lane: t + (e / 4) * 16 + q4 * 4 + e % 4, e = 0..7
        bf16x8_t pf[MT];
        uint32_t sees[MT];                          // bit e: the row sees token e
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) sees[mt] = 0xFF;
        uint32_t exist = 0xFF;
        if (special) {
          exist = existing(t + q4 * 4, len, pg[0], pg[1]);
          mask_scores<MT>(p, b, mb * BR + r16, here, prefix, t + q4 * 4, exist, s, sees);
        }
        weights<MT>(s, p.scale2, mref, l, pf, [&](int mt, float f) {
#pragma unroll
          for (int k = 0; k < ND; ++k) o[mt][k] *= f;
        });
        // V: dword c of the lane's values of each token; their block is the same for all four
#pragma unroll
        for (int c = 0; c < ND / 4; ++c) {
          // the scheduler would hoist every chunk's reads, and spill; spilled registers are reloaded through
          // the counter that the ring's loads use, so a wait for one would drain the ring
          __builtin_amdgcn_sched_barrier(0);
          uint32_t raw[8];
          float f[8];
          const int d = v_value<D>(r16, 4 * c);
#pragma unroll
          for (int gr = 0; gr < 2; ++gr) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              raw[gr * 4 + j] = *reinterpret_cast<const uint32_t*>(st + (2 + gr) * G::CODES + (j * 4 + q4) * D + d);
            Scales<D>::v(scales + (2 + gr) * G::SCALES, r16, q4, c, f + gr * 4);
          }
          bool flagged = false;
          if (special) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              raw[e] = exist & (1u << e) ? raw[e] : 0u;
              f[e] = exist & (1u << e) ? f[e] : 1.f;
            }
            flagged = __any(maybe_nonfinite(raw, f));
          }
          bf16x8_t a[4];
          v_operands(raw, f, a);
          if (__builtin_expect(flagged, 0)) flag_rows<MT>(a, sees, &o[0][0] + 4 * c, ND);
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
              o[mt][4 * c + k] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[k], pf[mt], o[mt][4 * c + k], 0, 0, 0);
        }
      };

#pragma unroll 1
      for (int i = 0; i < NS && i < nt; ++i) issue(i);
      if (uc == ua) {                               // while the first tiles are on their way
#pragma unroll
        for (int k = 0; k < (MT * NK + NW - 1) / NW; ++k) {
          const int f = qw + k * NW;
          if (f >= MT * NK) break;
          queries[f * 64 + lane] = make_uint4((qv[k].x & p.q_keep) ^ p.q_flip, (qv[k].y & p.q_keep) ^ p.q_flip,
                                              (qv[k].z & p.q_keep) ^ p.q_flip, (qv[k].w & p.q_keep) ^ p.q_flip);
        }
        __syncthreads();
      }
#pragma unroll 1
      for (int i = 0; i < nt; ++i) {
        const int ahead = min(NS - 1, nt - 1 - i);  // tiles in flight beyond this one
        if (ahead >= 3) wait_vmcnt_le<(NS > 3 ? 3 * G::PER_TILE : 0)>();
        else if (ahead == 2) wait_vmcnt_le<(NS > 2 ? 2 * G::PER_TILE : 0)>();
        else if (ahead == 1) wait_vmcnt_le<G::PER_TILE>();
        else wait_vmcnt_le<0>();
        compute(i);
        if (i + NS < nt) {
          asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // this tile's reads, before it is refilled
          issue(i + NS);
        }
      }
      uc = uz;
    }

    // join the waves: a common reference, then the sums in a fixed order, a part of them by each wave
    __syncthreads();                                // the rings and queries are done with
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      l[mt] += __shfl_xor(l[mt], 16);
      l[mt] += __shfl_xor(l[mt], 32);
      if (q4 == 0) stats[wave * BR + mt * 16 + r16] = make_float2(mref[mt], l[mt]);
    }
    __syncthreads();
    f32x4_t* const join = reinterpret_cast<f32x4_t*>(ring);
    constexpr int SPAN = RESULT / 16;
    auto total = [&](int row, float& m) {           // a row's reference and sum
      m = M_NONE;
#pragma unroll
      for (int w = 0; w < NW; ++w) m = fmaxf(m, stats[w * BR + row].x);
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) sum += stats[w * BR + row].y * __builtin_amdgcn_exp2f(stats[w * BR + row].x - m);
      return sum;
    };
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      float m = M_NONE;
#pragma unroll
      for (int w = 0; w < NW; ++w) m = fmaxf(m, stats[w * BR + mt * 16 + r16].x);
      const float f = __builtin_amdgcn_exp2f(mref[mt] - m);
#pragma unroll
      for (int i = 0; i < ND; ++i) o[mt][i] *= f;
    }
    auto put = [&](f32x4_t* d) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < ND; ++i) d[(mt * ND + i) * 64 + lane] = o[mt][i];
    };
    if (HELD == NW || wave >= HELD) put(join + wave % HELD * SPAN);
    if constexpr (HELD < NW) {
      __syncthreads();
      if (wave < HELD) {
        f32x4_t* d = join + wave * SPAN;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int i = 0; i < ND; ++i) d[(mt * ND + i) * 64 + lane] += o[mt][i];
      }
    }
    __syncthreads();
    const bool whole = ua == 0 && ub == units;
    const int64_t slot = (int64_t)blockIdx.x * 2 + (u == first_u ? 0 : 1);
    if (threadIdx.x == 0 && !p.direct) {
      int2* own = p.owners + ((int64_t)b * p.hkv + h) * p.mblocks + mb;
      if (ua == 0) own->x = (int)slot;
      if (ub == units) own->y = blockIdx.x;
    }
#pragma unroll 1
    for (int part = wave; part < MT * (ND / 4); part += NW) {   // a row block's values of four operand tiles
      const int mt = part / (ND / 4), c = part % (ND / 4);
      const f32x4_t* d = join + (mt * ND + 4 * c) * 64 + lane;
      f32x4_t v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[k] = d[k * 64];
#pragma unroll
        for (int w = 1; w < HELD; ++w) v[k] += d[w * SPAN + k * 64];
      }
      const int row = mt * 16 + r16, m = mb * BR + row;
      if (m >= p.rows) continue;
      float top;
      const float sum = total(row, top);
      if (whole) {
        const int nd = fdiv(m, p.dg);
        const bool live = nd < here && sum != 0.f;   // NaN passes
        const float f = 1.f / sum;
        uint16_t* dst = p.out + (((int64_t)b * p.T + nd) * p.hq + (int64_t)h * p.g + (m - nd * p.g)) * D;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          *reinterpret_cast<uint2*>(dst + v_value<D>(q4 * 4 + e, 4 * c)) =
              live ? make_uint2(pack_bf16x2(v[0][e] * f, v[1][e] * f), pack_bf16x2(v[2][e] * f, v[3][e] * f))
                   : make_uint2(0, 0);
      } else {
        float* dst = p.part + (slot * BR + row) * D;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          *reinterpret_cast<f32x4_t*>(dst + v_value<D>(q4 * 4 + e, 4 * c)) = f32x4_t{v[0][e], v[1][e], v[2][e], v[3][e]};
        if (c == 0 && q4 == 0) p.stat[slot * BR + row] = make_float2(top, sum);
      }
    }
    u += vb - va;
    while (u < u_end && u >= base + seq_span(p, b) * ipb) {
      base += seq_span(p, b) * ipb;
      ++b;
    }
  }
}

// Join the partial results of the heads that several workgroups shared, and zero the rows that nobody
// wrote (empty sequences). Who holds an item's partial results stands in `owners`. A workgroup takes `jr` rows of a
// head and row block, so that there are about JOIN_BLOCKS of them. D/4 lanes hold four values of a row each; the
// workgroup's 256 / (D/4) slices take rows side by side, or, when a row's partial results are many, all take one
// row and every so-many-th result of it.
constexpr int JOIN_BLOCKS = 1024;
template <int D>
__global__ void __launch_bounds__(256) attention_join_kernel(AttnParams p, int jr, int jblocks) {
  constexpr int LD = D / 4, SL = 256 / LD;
  __shared__ f32x4_t sums[SL][LD];
  const int BR = p.br, lane = threadIdx.x & 63;
  const int part = blockIdx.x % (unsigned)jblocks, item = blockIdx.x / (unsigned)jblocks;
  int r = item;
  const int mb = r % p.mblocks;
  r /= p.mblocks;
  const int h = r % p.hkv, b = r / p.hkv;
  const int2 own = p.owners[item];                  // (of an empty sequence: whatever, not used)
  const int len = seq_len(p, b), here = p.nodes ? p.nodes[b] : p.T;
  const int row0 = part * jr, row1 = min(min(row0 + jr, BR), p.rows - mb * BR);
  const int c = threadIdx.x % LD, sl = threadIdx.x / LD;
  auto out_at = [&](int row) {
    const int m = mb * BR + row, node = fdiv(m, p.dg);
    return p.out + (((int64_t)b * p.T + node) * p.hq + (int64_t)h * p.g + (m - node * p.g)) * D + c * 4;
  };
  if (len == 0) {
    for (int row = row0 + sl; sl < SL && row < row1; row += SL) *reinterpret_cast<uint2*>(out_at(row)) = make_uint2(0, 0);
    return;
  }
  const int w0 = own.x >> 1, w1 = own.y, n = w1 - w0 + 1;
  if (n == 1) return;
  // the first workgroup's result stands in its slot own.x & 1, the others' in their first
  auto slot_of = [&](int w) { return (int64_t)(w == w0 ? own.x : w * 2) * BR; };
  auto store = [&](int row, const f32x4_t& acc, float l) {
    const float f = 1.f / l;
    const bool live = l != 0.f && fdiv(mb * BR + row, p.dg) < here;
    *reinterpret_cast<uint2*>(out_at(row)) =
        live ? make_uint2(pack_bf16x2(acc[0] * f, acc[1] * f), pack_bf16x2(acc[2] * f, acc[3] * f)) : make_uint2(0, 0);
  };
  if (n <= 8) {                                     // all results of a row at once, one row per slice
    for (int row = row0 + sl; sl < SL && row < row1; row += SL) {
      float2 st[8];
      f32x4_t v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (k % 4 == 0 && k >= n) break;
        const int64_t at = slot_of(min(w0 + k, w1)) + row;
        st[k] = p.stat[at];
        v[k] = *reinterpret_cast<const f32x4_t*>(p.part + at * D + c * 4);
      }
      float top = fmaxf(fmaxf(st[0].x, st[1].x), fmaxf(st[2].x, st[3].x));
      if (n > 4) top = fmaxf(top, fmaxf(fmaxf(st[4].x, st[5].x), fmaxf(st[6].x, st[7].x)));
      f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
      float l = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (k >= n) break;
        const float f = __builtin_amdgcn_exp2f(st[k].x - top);
        l += st[k].y * f;
        acc += v[k] * f;
      }
      store(row, acc, l);
    }
    return;
  }
  for (int row = row0; row < row1; ++row) {
    // references and sums by the lanes of every wave, the values by the slices
    float top = M_NONE, l = 0.f;
    for (int w = w0 + lane; w <= w1; w += 64) top = fmaxf(top, p.stat[slot_of(w) + row].x);
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) top = fmaxf(top, __shfl_xor(top, o));
    for (int w = w0 + lane; w <= w1; w += 64) {
      const float2 s = p.stat[slot_of(w) + row];
      l += s.y * __builtin_amdgcn_exp2f(s.x - top);
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) l += __shfl_xor(l, o);
    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int w = w0 + sl; sl < SL && w <= w1; w += SL) {
      const int64_t at = slot_of(w) + row;
      acc += *reinterpret_cast<const f32x4_t*>(p.part + at * D + c * 4) * __builtin_amdgcn_exp2f(p.stat[at].x - top);
    }
    if (sl < SL) sums[sl][c] = acc;
    __syncthreads();
    if (sl == 0) {
#pragma unroll
      for (int i = 1; i < SL; ++i) acc += sums[i][c];
      store(row, acc, l);
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------------------------------------
// Many rows (trees, or many heads that share a key/value head): the waves of a workgroup take different
// rows, MT blocks of 16 each, and share the tokens. Codes and scales of a tile travel through a ring of
// STAGES tiles in LDS (the LDS mode of global loads); from there K and V are rebuilt once per workgroup
// into operand order, also in LDS (a fragment of one MFMA is 64 lanes x 16 bytes, read back without bank
// conflicts), two buffers deep: while a tile is computed, the next one is rebuilt, a unit of K and one of V
// by each wave. The operand order of V is value c * 64 + x * 4 + k for column x of 16-row tile 4c + k.
// Trees of 64 nodes over 16384 positions of 4 sequences, 64 heads over 8 of dim 128 (137 GFLOP): 176 us, 0.78 PFLOP/s.
// Counters: matrix cores busy 35% of the time, vector ALUs 47%, LDS 29%; two waves a SIMD overlap them little (all the
// registers are taken at 32 rows a wave). The instances of 32 rows of dim 128 and of dim 256 keep two and four vector registers
// in scratch, read once an item; every instance of both kernels keeps 110 to 290 scalars in lanes of vector registers. Taking turns by halves, products against softmax with a barrier after each
// phase, was slower (217 us), as was rebuilding V in half the waves and K in the others (180).
// ------------------------------------------------------------------------------------------------
constexpr int WW = 8;                               // waves per workgroup

template <int D>
struct Wide {
  static constexpr int TOKENS = D == 64 ? 128 : D == 128 ? 64 : 32;   // of a tile
  static constexpr int SHIFT = D == 64 ? 7 : D == 128 ? 6 : 5;
  static constexpr int SETS = TOKENS / 32, GROUPS = TOKENS / 16;
  // K's fragments of the next tile are read after the products with V, where both do not fit the registers (reading
  // them before spilled 43 registers, and a reload waits for the ring)
  static constexpr bool LATE_K = D == 256;
  static_assert(!LATE_K || SETS == 1, "the next tile's");
  static constexpr int KU = GROUPS * (D / 64), VU = SETS * (D / 64) * 2;   // rebuilding units: 16 codes, 8 x 2 codes a lane
  static constexpr int KF = GROUPS * (D / 32) * 64, VF = SETS * (D / 16) * 64;   // 16-byte words of a buffer
  static constexpr int CODES = TOKENS * D;                            // bytes of K's codes of a tile, and of V's
  static constexpr int SCALES = CODES / 32;
  static constexpr int STAGE = 2 * CODES + 2 * SCALES, STAGES = 4;    // K, V, K's scales, V's scales
  static constexpr int CL = 2 * GROUPS * (D / 64), LOADS = CL + 2 * GROUPS;   // loads of a tile: 1 KB of codes; a group's scales
  static constexpr int KW = (KU + WW - 1) / WW, VW = (VU + WW - 1) / WW;   // units per wave
  static_assert(CODES * 4 + STAGES * STAGE + TABLE * 4 <= 160 * 1024 && 2 * (KF + VF) * 16 == CODES * 8, "LDS");
};

template <int D, int MT>
__global__ void __launch_bounds__(64 * WW, 2) attention_wide_kernel(AttnParams p) {
  using W = Wide<D>;
  constexpr int ND = D / 16, NK = D / 32, NC = D / 64, BR = WW * MT * 16, STAGES = W::STAGES;
  __shared__ __align__(16) uint4 frags[2][W::KF + W::VF];
  __shared__ __align__(16) uint8_t ring[STAGES * W::STAGE];
  __shared__ int32_t table[TABLE];
  __shared__ int spoiled[3][W::SETS];               // of tile i in slot i % 3: a set has NaN or infinite values of V

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, q4 = lane >> 4;
  int u, u_end, b, base;
  if (!first_run<D>(p, lane, BR, u, u_end, b, base)) return;
  const int ipb = p.hkv * p.mblocks;
  const int first_u = u;

  // this wave's loads of a tile: 1 KB of a group's codes of K or V, or the scales of a group
  constexpr int MY = (W::LOADS + WW - 1) / WW;
  struct {
    const uint8_t* base;
    uint32_t off;
    int group, lds;
  } my[MY];
#pragma unroll
  for (int k = 0; k < MY; ++k) {
    const int n = wave + k * WW;
    const bool codes = n < W::CL;
    const int per = codes ? 2 * NC : 2, at = codes ? n : n - W::CL;
    const int gr = at / per, x = at % per, c = x % NC;
    const bool is_v = x >= per / 2;                 // the first half of a group's loads are K's
    my[k].group = gr;
    my[k].base = codes ? (is_v ? p.vq : p.kq) : (is_v ? p.vs : p.ks);
    my[k].off = is_v ? v_source<D>(c, lane) : k_source<D>(c, lane);
    my[k].lds = codes ? (is_v ? W::CODES : 0) + gr * 16 * D + c * 1024 : 2 * W::CODES + (is_v ? W::SCALES : 0) + gr * (D / 2);
  }

  while (u < u_end) {
    const int len = seq_len(p, b), units = (len + W::TOKENS - 1) / W::TOKENS, span = units + p.start_cost;
    const int item = (u - base) / span;
    const int va = (u - base) - item * span, vb = min(span, va + (u_end - u));
    const int ua = max(va - p.start_cost, 0), ub = vb - p.start_cost;
    if (ub <= ua) break;                            // the run ends in the item's cost
    const int h = item / p.mblocks, mb = item - h * p.mblocks;
    const int here = p.nodes ? max(0, min(p.nodes[b], p.T)) : p.T;
    const int prefix = len - here;
    const int m0 = mb * BR + wave * MT * 16;        // this wave's first row

    bf16x8_t qf[MT][NK];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int m = m0 + mt * 16 + r16, nd = fdiv(min(m, p.rows - 1), p.dg), hd = m - nd * p.g;
      const bool on = m < p.rows && nd < here;
      const uint16_t* src = p.q + ((int64_t)b * p.T + nd) * p.ldq + ((int64_t)h * p.g + hd) * D;
#pragma unroll
      for (int j = 0; j < NK; ++j) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (on) v = *reinterpret_cast<const uint4*>(src + (j >> 1) * 64 + q4 * 16 + (j & 1) * 8);
        const u32x4_t w = {(v.x & p.q_keep) ^ p.q_flip, (v.y & p.q_keep) ^ p.q_flip, (v.z & p.q_keep) ^ p.q_flip,
                           (v.w & p.q_keep) ^ p.q_flip};
        qf[mt][j] = __builtin_bit_cast(bf16x8_t, w);
      }
    }
    f32x4_t o[MT][ND];
    float mref[MT], l[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      mref[mt] = M_NONE;
      l[mt] = 0.f;
#pragma unroll
      for (int i = 0; i < ND; ++i) o[mt][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }

    for (int uc = ua; uc < ub;) {                   // as many tiles as the table covers
      const int uz = min(ub, uc + STRETCH / W::TOKENS), tbase = uc * W::TOKENS;
      __syncthreads();                              // the table, ring and buffers are free; nothing is in flight
      bool absent = fill_table(p, b, h, tbase, len, table);
      __syncthreads();
      absent = table_absent(absent, table);
      auto issue = [&](int i) {
        uint8_t* st = ring + (i % STAGES) * W::STAGE;
        const int* en = table + (i - uc) * W::GROUPS;
        int entry[MY];                              // read together, before the loads that each needs one
#pragma unroll
        for (int k = 0; k < MY; ++k) entry[k] = en[my[k].group < W::GROUPS ? my[k].group : 0];
#pragma unroll
        for (int k = 0; k < MY; ++k) {
          if (wave + k * WW >= W::LOADS) break;
          const int64_t at = max(__builtin_amdgcn_readfirstlane(entry[k]), 0);   // absent: some group, not used
          if (k < W::CL / WW || wave + k * WW < W::CL)
            gload_lds16<1>(my[k].base + at * (16 * D), &my[k].off, lds_addr(st + my[k].lds));
          else if (lane < D / 8)
            gload_lds4(uniform(my[k].base + at * (D / 2)) + lane * 4, lds_addr(st + my[k].lds));
        }
      };
      // wait for this wave's loads but those of the newest `tiles` tiles
      auto landed = [&](int tiles) {
        constexpr int FEW = W::LOADS / WW, MANY = (W::LOADS + WW - 1) / WW;
        if (wave < W::LOADS % WW) {
          if (tiles >= 2) wait_vmcnt_le<2 * MANY>();
          else if (tiles == 1) wait_vmcnt_le<MANY>();
          else wait_vmcnt_le<0>();
        } else {
          if (tiles >= 2) wait_vmcnt_le<2 * FEW>();
          else if (tiles == 1) wait_vmcnt_le<FEW>();
          else wait_vmcnt_le<0>();
        }
      };
      // Rebuilding tile i: a unit of K (two fragments of 16 tokens) and one of V (two fragments of 32 tokens) per
      // wave; the codes and scales are read a phase before they are converted.
      struct Raw {
        uint4 k[W::KW];
        uint32_t v[W::VW][8], ks[W::KW], vs[W::VW][8];
      };
      auto read_raw = [&](int i, Raw& r) {
        const uint8_t* st = ring + (i % STAGES) * W::STAGE;
        const uint8_t* sc = st + 2 * W::CODES;
#pragma unroll
        for (int n = 0; n < W::KW; ++n) {
          const int unit = wave + n * WW, gr = unit / NC, j = unit % NC;
          if (W::KU % WW && unit >= W::KU) break;
          r.k[n] = *reinterpret_cast<const uint4*>(st + gr * 16 * D + r16 * D + (((4 * j + q4) ^ Geo<D>::swizzle(r16)) * 16));
          r.ks[n] = sc[gr * (D / 2) + r16 * (D / 32) + 2 * j + (q4 >> 1)];
        }
#pragma unroll
        for (int n = 0; n < W::VW; ++n) {
          const int unit = wave + n * WW, half = unit & 1, set = (unit >> 1) / NC, c = (unit >> 1) % NC;
          if (W::VU % WW && unit >= W::VU) break;
#pragma unroll
          for (int gr = 0; gr < 2; ++gr) {
            const uint8_t* codes = st + W::CODES + (set * 2 + gr) * 16 * D + q4 * D + c * 64 + r16 * 4 + half * 2;
#pragma unroll
            for (int j = 0; j < 4; ++j) r.v[n][gr * 4 + j] = *reinterpret_cast<const uint16_t*>(codes + j * 4 * D);
            const uint8_t* g = sc + W::SCALES + (set * 2 + gr) * (D / 2);
            uint32_t* w = r.vs[n] + gr * 4;         // words that hold the tokens' scales (see v_scale)
            if constexpr (D == 128) {
              const uint4 x = *reinterpret_cast<const uint4*>(g + q4 * 16);
              w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
            } else if constexpr (D == 64) {
              const uint2 x = *reinterpret_cast<const uint2*>(g + q4 * 8);
              w[0] = w[1] = x.x, w[2] = w[3] = x.y;
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j) w[j] = *reinterpret_cast<const uint16_t*>(g + (q4 * 4 + j) * (D / 32) + 2 * c);
            }
          }
        }
      };
      // (kept out of read_raw: nothing there may wait for LDS)
      auto v_scale = [&](uint32_t word, int j, int c) {
        return Scales<D>::rotated(word, (D == 128 ? 2 * c : D == 64 ? 2 * (j & 1) : 0) + (r16 >> 3));
      };
      auto rebuild = [&](int i, Raw& r, uint4* buf) {
#pragma unroll
        for (int n = 0; n < W::KW; ++n) {
          const int unit = wave + n * WW, gr = unit / NC, j = unit % NC;
          if (W::KU % WW && unit >= W::KU) break;
          uint4* dst = buf + (gr * NK + 2 * j) * 64 + lane;
          const float f = block_scale(r.ks[n]);
          dst[0] = __builtin_bit_cast(uint4, dequant8(r.k[n].x, r.k[n].y, f));
          dst[64] = __builtin_bit_cast(uint4, dequant8(r.k[n].z, r.k[n].w, f));
        }
#pragma unroll
        for (int n = 0; n < W::VW; ++n) {
          const int unit = wave + n * WW, half = unit & 1, set = (unit >> 1) / NC, c = (unit >> 1) % NC;
          if (W::VU % WW && unit >= W::VU) break;
          const int t = i * W::TOKENS + set * 32;
          float f[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = v_scale(r.vs[n][e], e & 3, c);
          if (t + 32 > len || absent) {             // tokens that are not there: zeros
            const int* pg = table + ((t - tbase) >> 4);
            const uint32_t exist = existing(t + q4 * 4, len, pg[0], pg[1]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              r.v[n][e] = exist & (1u << e) ? r.v[n][e] : 0u;
              f[e] = exist & (1u << e) ? f[e] : 1.f;
            }
          }
          u32x4_t a0, a1;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t x = bits_of(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(r.v[n][2 * j], f[2 * j], false));
            const uint32_t y = bits_of(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(r.v[n][2 * j + 1], f[2 * j + 1], false));
            a0[j] = __builtin_amdgcn_perm(y, x, 0x05040100u);
            a1[j] = __builtin_amdgcn_perm(y, x, 0x07060302u);
          }
          // a row may not see its token: NaN and infinite values leave the product (see poison)
          if (t + 32 > prefix) {
            uint32_t any = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t x = nonfinite(a0[j]), y = nonfinite(a1[j]);
              a0[j] &= ~x;
              a1[j] &= ~y;
              any |= x | y;
            }
            if (__any(any != 0) && lane == 0) spoiled[i % 3][set] = 1;
          }
          uint4* dst = buf + W::KF + (set * ND + 4 * c + 2 * half) * 64 + lane;
          dst[0] = __builtin_bit_cast(uint4, a0);
          dst[64] = __builtin_bit_cast(uint4, a1);
        }
      };
      auto ask_k = [&](const uint4* buf, int set, uint4 (&fr)[2 * NK]) {
#pragma unroll
        for (int j = 0; j < 2 * NK; ++j) fr[j] = buf[(set * 2 * NK + j) * 64 + lane];
      };
      // Rows that see a NaN or infinite value of V get it added there (the rebuilt fragments hold zeros in its place),
      // from the raw codes (flag_rows).
      auto poison = [&](int i, int set, const uint32_t (&sees)[MT]) {
        const uint8_t* st = ring + (i % STAGES) * W::STAGE;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          uint32_t raw[8];
          float f[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int gr = set * 2 + (e >> 2), j = e & 3;
            raw[e] = *reinterpret_cast<const uint32_t*>(st + W::CODES + gr * 16 * D + (j * 4 + q4) * D + c * 64 + r16 * 4);
            f[e] = block_scale(st[2 * W::CODES + W::SCALES + gr * (D / 2) + (q4 * 4 + j) * (D / 32) + 2 * c + (r16 >> 3)]);
          }
          bf16x8_t a[4];
          v_operands(raw, f, a);
          flag_rows<MT>(a, sees, &o[0][0] + 4 * c, ND);
          __builtin_amdgcn_sched_barrier(0);
        }
      };
      // Tile i is loaded in iteration i - 3, rebuilt in iteration i - 1 and computed in iteration i. One barrier an
      // iteration, before its last products with V: by then everyone has rebuilt its share of the next tile, has
      // this tile's last fragments in registers (so its buffer is free), and its loads of the tile after the
      // next have landed. Every read of LDS is asked for a phase ahead: V's fragments before the softmax, the next
      // K's before the products with V, the codes to rebuild at the top.
#pragma unroll 1
      for (int i = uc; i < min(uc + 3, uz); ++i) issue(i);
      if (threadIdx.x < 3 * W::SETS) spoiled[threadIdx.x / W::SETS][threadIdx.x % W::SETS] = 0;
      landed(min(uz - uc, 3) - 1);
      __syncthreads();
      Raw raw;
      read_raw(uc, raw);
      rebuild(uc, raw, frags[uc & 1]);
      landed(max(min(uz - uc, 3) - 2, 0));
      __syncthreads();
      uint4 kf[2 * NK];
      ask_k(frags[uc & 1], 0, kf);
#pragma unroll 1
      for (int i = uc; i < uz; ++i) {
        const uint4* buf = frags[i & 1];
        if (threadIdx.x < W::SETS) spoiled[(i + 2) % 3][threadIdx.x] = 0;   // read an iteration ago, set in the next
        if (i + 3 < uz) issue(i + 3);
        if (i + 1 < uz) read_raw(i + 1, raw);
#pragma unroll
        for (int set = 0; set < W::SETS; ++set) {
          const int t = i * W::TOKENS + set * 32;
          // some row may not see all of it: nodes, the sequence's end, absent pages (uniform)
          const bool special = t + 32 > min(prefix, len) || absent;
          f32x4_t s[2][MT];
#pragma unroll
          for (int gr = 0; gr < 2; ++gr)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) s[gr][mt] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < NK; ++j)
#pragma unroll
            for (int gr = 0; gr < 2; ++gr)
#pragma unroll
              for (int mt = 0; mt < MT; ++mt)
                s[gr][mt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, kf[gr * NK + j]), qf[mt][j],
                                                                    s[gr][mt], 0, 0, 0);
          const uint4* vf = buf + W::KF + set * ND * 64 + lane;
          uint4 fr[ND];
#pragma unroll
          for (int k = 0; k < ND; ++k) fr[k] = vf[k * 64];
          __builtin_amdgcn_sched_barrier(0);
          uint32_t sees[MT] = {};
          if (__builtin_expect(special, 0)) {
            const int* pg = table + ((t - tbase) >> 4);
            mask_scores<MT>(p, b, m0 + r16, here, prefix, t + q4 * 4, existing(t + q4 * 4, len, pg[0], pg[1]), s, sees);
          }
          if (set == 0 && i + 1 < uz) rebuild(i + 1, raw, frags[(i + 1) & 1]);
          bf16x8_t pf[MT];
          weights<MT>(s, p.scale2, mref, l, pf, [&](int mt, float f) {
#pragma unroll
            for (int k = 0; k < ND; ++k) o[mt][k] *= f;
          });
          // (after the rescaling, which would make a NaN of an infinity)
          if (__builtin_expect(special, 0) && __builtin_amdgcn_readfirstlane(spoiled[i % 3][set])) poison(i, set, sees);
          if (set + 1 < W::SETS) {
            ask_k(buf, set + 1, kf);
          } else {
            landed(i + 3 < uz ? 1 : 0);             // all but tile i + 3's: tile i + 2 is there
            __syncthreads();
            if (!W::LATE_K) ask_k(frags[(i + 1) & 1], 0, kf);   // (after the last tile: not used)
          }
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int k = 0; k < ND; ++k)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
              o[mt][k] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, fr[k]), pf[mt], o[mt][k], 0, 0, 0);
          if (W::LATE_K) {
            __builtin_amdgcn_sched_barrier(0);
            ask_k(frags[(i + 1) & 1], 0, kf);
          }
        }
      }
      uc = uz;
    }

    const bool whole = ua == 0 && ub == units;
    const int64_t slot = (int64_t)blockIdx.x * 2 + (u == first_u ? 0 : 1);
    if (threadIdx.x == 0 && !p.direct) {
      int2* own = p.owners + ((int64_t)b * p.hkv + h) * p.mblocks + mb;
      if (ua == 0) own->x = (int)slot;
      if (ub == units) own->y = blockIdx.x;
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      l[mt] += __shfl_xor(l[mt], 16);
      l[mt] += __shfl_xor(l[mt], 32);
      const int m = m0 + mt * 16 + r16, row = m - mb * BR;
      if (m >= p.rows) continue;
      if (whole) {
        const int nd = fdiv(m, p.dg);
        const bool live = nd < here && l[mt] != 0.f;   // NaN passes
        const float f = 1.f / l[mt];
        uint16_t* dst = p.out + (((int64_t)b * p.T + nd) * p.hq + (int64_t)h * p.g + (m - nd * p.g)) * D + q4 * 16;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            u32x4_t w;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int k = 4 * c + (x & 1) * 2, r = e + (x >> 1);
              w[x] = live ? pack_bf16x2(o[mt][k][r] * f, o[mt][k + 1][r] * f) : 0u;
            }
            *reinterpret_cast<u32x4_t*>(dst + c * 64 + e * 4) = w;
          }
      } else {
        float* dst = p.part + (slot * BR + row) * D + q4 * 16;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            *reinterpret_cast<f32x4_t*>(dst + c * 64 + e * 4) =
                f32x4_t{o[mt][4 * c][e], o[mt][4 * c + 1][e], o[mt][4 * c + 2][e], o[mt][4 * c + 3][e]};
        if (q4 == 0) p.stat[slot * BR + row] = make_float2(mref[mt], l[mt]);
      }
    }
    u += vb - va;
    while (u < u_end && u >= base + seq_span(p, b) * ipb) {
      base += seq_span(p, b) * ipb;
      ++b;
    }
  }
}

// The two kernels' row blocks (mt steps of rows, at most `most`), units and grids.
struct AttnKernel {
  bool wide;
  int dim;
  int64_t step() const { return wide ? WW * 16 : 16; }
  int64_t most() const { return wide ? (dim == 64 ? 3 : dim == 128 ? 2 : 1) : dim <= 128 ? 3 : 2; }
  int64_t blocks(int64_t rows) const { return (rows + step() * most() - 1) / (step() * most()); }
  int unit_shift(int mt) const { return !wide ? (ring_waves(dim, mt) == 8 ? 8 : 7) : dim == 64 ? 7 : dim == 128 ? 6 : 5; }
  int64_t grid(int mt) const { return wide ? 256 : ring_grid(dim, mt); }
  int64_t unsplit() const { return wide ? (dim == 64 ? 256 : 128) : dim <= 128 ? 512 : 256; }   // (see attention_plan)
};
// The ring kernel takes up to two of its blocks of rows, though it reads keys and values twice then: 16 sequences of
// 4096 positions, 4 heads, 64 rows: 26 against 33 us at dim 64, 38 against 45 at 128, 58 against 62 at 192, 71 against
// 77 at 256 (three blocks, 96 rows at dim 256: 99 against 79; 144 rows at dim 64: 38 against 45)
inline int64_t ring_rows(int dim) { return AttnKernel{false, dim}.most() * 16 * 2; }

struct AttnPlan {
  int wide, mt, br, unit_shift, start_cost, mblocks, nwg, direct;
};
// Rows of a block and the grid: every unit its own workgroup up to one workgroup per CU.
AttnPlan attention_plan(const AttentionArgs& a) {
  const int64_t rows = a.T * (a.hq / a.cache.heads);
  AttnPlan p;
  p.wide = rows > ring_rows((int)a.cache.dim);
  const AttnKernel k{p.wide != 0, (int)a.cache.dim};
  const int64_t step = k.step(), blocks = k.blocks(rows);
  p.mt = (int)((rows + step * blocks - 1) / (step * blocks));
  p.br = (int)(p.mt * step);
  p.mblocks = (int)((rows + p.br - 1) / p.br);
  p.unit_shift = k.unit_shift(p.mt);
  const int64_t units = a.B * a.cache.heads * p.mblocks * ((a.max_len + (1 << p.unit_shift) - 1) >> p.unit_shift);
  const int64_t grid = k.grid(p.mt);
  const int64_t items = a.B * a.cache.heads * p.mblocks;
  // Units of a run: with n workgroups it costs about t units / n (t = 1 us, wide 2) to compute them, and to write and
  // read back n partial results at 4 TB/s and 35 ns for each of an item's in the join; the least sum. (One token over
  // 131072 positions, 8 heads over 1: 25 us, with runs of one unit 40; 59 nodes over 1024, 14 heads over 2: 24 against 30.)
  const double values = (double)((rows < p.br ? rows : p.br) * a.cache.dim);
  const double joined = (double)units * (values * 2e-6 + 0.035 / (double)(items > 0 ? items : 1));
  const double least = __builtin_sqrt(joined / (p.wide ? 2. : 1.));
  const int64_t run = least < 1.5 ? 1 : (int64_t)(least + 0.5), runs = (units + run - 1) / run;
  p.nwg = (int)(runs < 1 ? 1 : runs > grid ? grid : runs);
  // short contexts: a workgroup for each item, nothing to join (one sequence, 16 heads over 2 of dim 64: at 128 positions
  // 6.8 against 9.2 us, at 1024 11.5 against 10.2; 40 nodes, 16 heads over 4 of dim 128: at 128 positions 14.9 against
  // 17.6, at 256 19.3 against 17.8); longer ones where runs are longer than a unit, up to four (28 sequences of 275
  // positions, 53 nodes, 56 heads over 8 of dim 64: 27 against 52 us)
  p.direct = a.max_len <= k.unsplit() + ((run < 4 ? run : 4) - 1) * ((int64_t)1 << p.unit_shift);
  if (p.direct) {
    p.nwg = (int)items;
    p.start_cost = 0;
    return p;
  }
  // beginning an item costs about as long as four units (32 chains of 6, ragged, 64 heads over 8 of dim 128: 77 us, with 0
  // 96, with 8 81; 16 single tokens of dim 64: 26, 28 and 27; 24 x 3 nodes of dim 192: 56, 68 and - with 2 - 60); with few
  // units a workgroup has no second item
  p.start_cost = units > 4 * grid ? 4 : 0;
  return p;
}

template <int D>
int join(const AttnParams& p, hipStream_t stream) {
  const int64_t items = (int64_t)p.B * p.hkv * p.mblocks, rows = p.rows < p.br ? p.rows : p.br;
  int64_t jr = items * rows / JOIN_BLOCKS;
  jr = jr < 1 ? 1 : jr > rows ? rows : jr;
  const int64_t jblocks = (rows + jr - 1) / jr;
  hipLaunchKernelGGL((attention_join_kernel<D>), dim3((unsigned)(items * jblocks)), dim3(256), 0, stream, p, (int)jr,
                     (int)jblocks);
  return hip_status(hipGetLastError());
}

template <int D, int MT, int NS>
int ring(const AttnParams& p, hipStream_t stream) {
  hipLaunchKernelGGL((attention_kernel<D, MT, NS>), dim3((unsigned)p.nwg), dim3(64 * ring_waves(D, MT)), 0, stream, p);
  if (p.direct) return hip_status(hipGetLastError());
  return hipGetLastError() == hipSuccess ? join<D>(p, stream) : BSFP8_EHIP;
}
template <int D, int MT>
int wide(const AttnParams& p, hipStream_t stream) {
  hipLaunchKernelGGL((attention_wide_kernel<D, MT>), dim3((unsigned)p.nwg), dim3(64 * WW), 0, stream, p);
  if (p.direct) return hip_status(hipGetLastError());
  return hipGetLastError() == hipSuccess ? join<D>(p, stream) : BSFP8_EHIP;
}

inline size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace

// The most that a plan of these sizes or of a smaller batch, fewer nodes or a smaller max_len uses (a plan itself may use
// less for larger ones: short contexts of many sequences are not cut), so that one workspace serves a program's calls.
size_t attention_ws_bytes(const AttentionArgs& a) {
  const int dim = (int)a.cache.dim;
  const int64_t most_rows = a.T * (a.hq / a.cache.heads);
  int64_t part_rows = 0, mblocks = 1;
  bool split = false;
  for (const bool wide : {false, true}) {
    if (wide && most_rows <= ring_rows(dim)) break;
    const AttnKernel k{wide, dim};
    const int64_t rows = wide || most_rows < ring_rows(dim) ? most_rows : ring_rows(dim), blocks = k.blocks(rows);
    if (blocks > mblocks) mblocks = blocks;
    if (a.max_len > k.unsplit()) split = true;
    for (int mt = 1; mt <= k.most() && (mt - 1) * k.step() < rows; ++mt) {
      const int64_t tokens = (int64_t)1 << k.unit_shift(mt);
      const int64_t units = a.B * a.cache.heads * blocks * ((a.max_len + tokens - 1) / tokens);
      const int64_t held = k.step() * mt * (units < k.grid(mt) ? units : k.grid(mt));
      if (held > part_rows) part_rows = held;
    }
  }
  if (!split) return 256;                           // (not read)
  const size_t rows = (size_t)part_rows * 2;
  return align256((size_t)(a.B * a.cache.heads * mblocks) * sizeof(int2)) + align256(rows * sizeof(float2)) +
         rows * (size_t)dim * 4;
}

int launch_tree_attention(const AttentionArgs& a, hipStream_t stream) {
  const AttnPlan pl = attention_plan(a);
  AttnParams p{};
  p.q = a.q;
  p.kq = a.cache.kq;
  p.ks = a.cache.ks;
  p.vq = a.cache.vq;
  p.vs = a.cache.vs;
  p.pages = a.pages;
  p.lens = a.lens;
  p.nodes = a.nodes;
  p.mask = a.mask;
  p.out = a.out;
  char* ws = reinterpret_cast<char*>(a.ws);
  p.owners = reinterpret_cast<int2*>(ws);
  ws += align256((size_t)a.B * a.cache.heads * pl.mblocks * sizeof(int2));
  p.stat = reinterpret_cast<float2*>(ws);
  p.part = reinterpret_cast<float*>(ws + align256((size_t)pl.nwg * 2 * pl.br * sizeof(float2)));
  p.ldq = a.ldq;
  p.ld_pages = a.ld_pages;
  p.n_pages = a.cache.pages;
  p.scale2 = a.scale == 0.f ? 1.f : (a.scale < 0.f ? -a.scale : a.scale) * 1.4426950408889634f;
  p.q_keep = a.scale == 0.f ? 0u : ~0u;
  p.q_flip = a.scale < 0.f ? 0x80008000u : 0u;
  p.B = (int)a.B;
  p.T = (int)a.T;
  p.hq = (int)a.hq;
  p.hkv = (int)a.cache.heads;
  p.g = p.hq / p.hkv;
  p.rows = p.g * p.T;
  p.mblocks = pl.mblocks;
  p.page = (int)a.cache.page;
  const int64_t held = a.cache.pages == 0 ? 0 : a.ld_pages * a.cache.page;
  p.max_len = (int)(a.max_len < held ? a.max_len : held);
  p.nwg = pl.nwg;
  p.br = pl.br;
  p.unit_shift = pl.unit_shift;
  p.unit = 1 << pl.unit_shift;
  p.start_cost = pl.start_cost;
  p.direct = pl.direct;
  p.dpage = make_fastdiv((uint32_t)a.cache.page);
  p.dg = make_fastdiv((uint32_t)p.g);
  const int D = (int)a.cache.dim, mt = pl.mt;
  if (pl.wide) {
    if (D == 64)
      return mt == 1 ? wide<64, 1>(p, stream) : mt == 2 ? wide<64, 2>(p, stream) : wide<64, 3>(p, stream);
    if (D == 128) return mt == 1 ? wide<128, 1>(p, stream) : wide<128, 2>(p, stream);
    return D == 192 ? wide<192, 1>(p, stream) : wide<256, 1>(p, stream);
  }
  if (D == 64) return mt == 1 ? ring<64, 1, 4>(p, stream) : mt == 2 ? ring<64, 2, 4>(p, stream) : ring<64, 3, 4>(p, stream);
  if (D == 128) return mt == 1 ? ring<128, 1, 2>(p, stream) : mt == 2 ? ring<128, 2, 2>(p, stream) : ring<128, 3, 2>(p, stream);
  if (D == 192) return mt == 1 ? ring<192, 1, 2>(p, stream) : ring<192, 2, 2>(p, stream);
  return mt == 1 ? ring<256, 1, 2>(p, stream) : ring<256, 2, 2>(p, stream);
}

}  // namespace bsfp8
