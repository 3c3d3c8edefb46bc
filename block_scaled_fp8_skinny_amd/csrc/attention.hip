// Attention of drafted tokens over the paged MXFP8 cache for gfx950 (MI355X).
//
// One kernel for decoding (one token a sequence), chains and trees. The rows of one key/value head
// are its (node, query head) pairs, g * T of them (g query heads share it). With s = q . k * scale in
// base 2 (scale * log2 e), a running reference m per row, and weights w = 2^(s - m):
//   l = sum w,  O = sum w V,  out = O / l,
// one pass over the positions; m only moves (and O and l are rescaled) when a tile's maximum passes
// it by more than MOVE, so that 2^MOVE bounds the weights.
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
// A workgroup is NW waves that share a head's rows and split its tokens in tiles of 32, each wave
// with a ring of NS tiles in LDS that the LDS mode of global loads fills (codes are contiguous per
// 16 tokens of a page and head); waves only wait for their own loads. The waves' results are joined
// through LDS. Work is cut evenly over the grid: the units (128 tokens of one head and row block) of
// all sequences, in order, are divided into equal runs, one per workgroup, so that ragged lengths
// leave nobody idle; a head that falls into several runs leaves partial (m, l, O) in the workspace
// for a second kernel to join.
#include "device.h"

namespace bsfp8 {
namespace {

constexpr int NW = 4;                               // waves per workgroup
constexpr int TILE = 32;                            // tokens of a wave's tile
constexpr int UNIT = NW * TILE;
constexpr int TABLE = 512;                          // page numbers held in LDS at a time
constexpr float MOVE = 8.f;
constexpr float M_NONE = -1e30f;                    // reference of a row that has seen nothing

struct AttnParams {
  const uint16_t* q;
  const uint8_t *kq, *ks, *vq, *vs;
  const int32_t *pages, *lens, *nodes;
  const int64_t* mask;
  uint16_t* out;
  float* part;                                      // [nwg][2][rows of a block][D]
  float2* stat;                                     // [nwg][2][rows of a block]: m, l
  int64_t ldq, ld_pages, n_pages;
  float scale2;                                     // |scale| * log2 e (1 for a scale of 0)
  uint32_t q_keep, q_flip;                          // the scale's sign, or a scale of 0, on the queries
  int B, T, hq, hkv, g, rows, mblocks, page, max_len, nwg;
  FastDiv dpage, dg;
};

__device__ __forceinline__ int seq_len(const AttnParams& p, int b) { return max(0, min(p.lens[b], p.max_len)); }
__device__ __forceinline__ int seq_units(const AttnParams& p, int b) { return (seq_len(p, b) + UNIT - 1) / UNIT; }

// The run of units of workgroup w out of `total`: the first `rem` runs hold per + 1.
struct Runs {
  int per, rem;
  __device__ __forceinline__ Runs(int total, int nwg) : per(total / nwg), rem(total - (total / nwg) * nwg) {}
  __device__ __forceinline__ int start(int w) const { return w * per + min(w, rem); }
  __device__ __forceinline__ int owner(int u) const {
    const int wide = rem * (per + 1);
    return u < wide ? u / (per + 1) : rem + (u - wide) / per;
  }
};

// Units before each sequence, per head and row block, by a scan over the batch (whole wave; lane l
// covers sequences l * c .. l * c + c - 1).
struct Batch {
  int c, incl, own, total;
  __device__ __forceinline__ Batch(const AttnParams& p, int lane) {
    c = (p.B + 63) >> 6;
    own = 0;
    for (int i = lane * c; i < min(lane * c + c, p.B); ++i) own += seq_units(p, i);
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
      const int n = seq_units(p, b);
      if (v < before + n) return b;
      before += n;
    }
  }
  // the units before sequence b
  __device__ __forceinline__ int before(const AttnParams& p, int b) const {
    const int l = b / c;
    int v = __shfl(incl, l) - __shfl(own, l);
    for (int i = l * c; i < b; ++i) v += seq_units(p, i);
    return v;
  }
};

// Global loads in LDS mode (see lds_load16 of device.h): 64-bit addresses, as a cache passes 4 GiB. The
// base may come from a lane exchange or readfirstlane, so the five wait states that a vector-written
// scalar needs before a memory instruction reads it are spent here (s_nop 4).
__device__ __forceinline__ const uint8_t* uniform(const uint8_t* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return reinterpret_cast<const uint8_t*>((uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ void gload_lds16(const uint8_t* base, uint32_t off, lds_addr_t lds) {
  uint32_t saved;
  asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %2, %3\n\ts_mov_b32 m0, %0"
               : "=&s"(saved) : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(off), "s"(uniform(base)) : "memory");
}
__device__ __forceinline__ void gload_lds4(const uint8_t* addr, lds_addr_t lds) {
  uint32_t saved;
  asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %2, off\n\ts_mov_b32 m0, %0"
               : "=&s"(saved) : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(addr) : "memory");
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
// (the product of the flags of such values with the flags of seen tokens is positive) get NaN.
template <int MT>
__device__ __forceinline__ void unseen_nonfinite(bf16x8_t (&a)[4], const uint32_t (&sees)[MT], f32x4_t* o, int stride) {
  auto bad = [](uint32_t v) {                       // ones where a half is NaN or infinite
    return ((v & 0x7F80u) == 0x7F80u ? 0xFFFFu : 0u) | ((v & 0x7F800000u) == 0x7F800000u ? 0xFFFF0000u : 0u);
  };
  uint32_t any = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int j = 0; j < 4; ++j) any |= bad(__builtin_bit_cast(u32x4_t, a[k])[j]);
  if (!__any(any != 0)) return;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    u32x4_t v = __builtin_bit_cast(u32x4_t, a[k]), flag;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t x = bad(v[j]);
      flag[j] = 0x3F803F80u & x;
      v[j] &= ~x;
    }
    a[k] = __builtin_bit_cast(bf16x8_t, v);
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
        if (n[r] > 0.f) o[mt * stride + k][r] = __uint_as_float(0x7FC00000u);
    }
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
__global__ void __launch_bounds__(64 * NW, D <= 128 ? 2 : 1) attention_kernel(AttnParams p) {
  using G = Geo<D>;
  constexpr int ND = D / 16, NK = D / 32, BR = MT * 16;
  constexpr int RING = NW * NS * G::STAGE, JOIN = 2 * MT * ND * 1024;
  constexpr int BYTES = RING > JOIN ? RING : JOIN;
  static_assert((NS - 1) * G::PER_TILE <= 63, "vector memory counter range");
  static_assert(NW * BR * 8 <= TABLE * 4, "the statistics take the table's place");
  __shared__ __align__(16) uint8_t ring[BYTES];
  __shared__ __align__(16) uint4 queries[MT * NK * 64];   // B operands: row mt*16 + r16, values of K's operand order
  __shared__ __align__(16) int32_t table[TABLE];
  float2* const stats = reinterpret_cast<float2*>(table);

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, q4 = lane >> 4;
  const Batch batch(p, lane);
  const int ipb = p.hkv * p.mblocks;                // heads and row blocks of a sequence
  const int total = batch.total * ipb;
  const Runs runs(total, p.nwg);
  int u = runs.start(blockIdx.x);
  const int u_end = runs.start(blockIdx.x + 1);
  if (u >= u_end) return;
  int before;
  int b = batch.find(p, u / ipb, before);
  int base = before * ipb;                          // first unit of sequence b
  const int first_u = u;

  uint32_t ksrc[G::LOADS], vsrc[G::LOADS];
#pragma unroll
  for (int n = 0; n < G::LOADS; ++n) {
    ksrc[n] = k_source<D>(n, lane);
    vsrc[n] = v_source<D>(n, lane);
  }
  uint8_t* const my_ring = ring + wave * NS * G::STAGE;

  while (u < u_end) {
    const int len = seq_len(p, b), units = (len + UNIT - 1) / UNIT;
    const int item = (u - base) / units;            // head and row block
    const int ua = (u - base) - item * units, ub = min(units, ua + (u_end - u));
    const int h = item / p.mblocks, mb = item - h * p.mblocks;
    const int here = p.nodes ? max(0, min(p.nodes[b], p.T)) : p.T;
    const int prefix = len - here;

    __syncthreads();                                // the last run's ring, queries and statistics are done with
    for (int i = threadIdx.x; i < MT * NK * 64; i += 64 * NW) {
      const int l = i & 63, j = (i >> 6) % NK, m = mb * BR + (i >> 6) / NK * 16 + (l & 15);
      const int nd = fdiv(min(m, p.rows - 1), p.dg), hd = m - nd * p.g;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (m < p.rows && nd < here) {
        v = *reinterpret_cast<const uint4*>(p.q + ((int64_t)b * p.T + nd) * p.ldq + ((int64_t)h * p.g + hd) * D +
                                            (j >> 1) * 64 + (l >> 4) * 16 + (j & 1) * 8);
        v.x = (v.x & p.q_keep) ^ p.q_flip;
        v.y = (v.y & p.q_keep) ^ p.q_flip;
        v.z = (v.z & p.q_keep) ^ p.q_flip;
        v.w = (v.w & p.q_keep) ^ p.q_flip;
      }
      queries[i] = v;
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

    for (int uc = ua; uc < ub;) {                   // as many units as the table's page numbers cover
      const int p0 = fdiv(uc * UNIT, p.dpage);
      const int uz = (int)min((int64_t)ub, ((int64_t)p0 + TABLE) * p.page / UNIT);
      const int np = fdiv(min(uz * UNIT, len) - 1, p.dpage) + 1 - p0;
      if (uc != ua) __syncthreads();                // the table is free
      for (int i = threadIdx.x; i < np; i += 64 * NW) {
        const int pg = p.pages[(int64_t)b * p.ld_pages + p0 + i];
        table[i] = pg >= 0 && pg < p.n_pages ? pg : -1;
      }
      __syncthreads();
      const int t0 = uc * UNIT + wave * TILE;       // this wave's first token; then every UNIT
      const int nt = t0 < len ? min(uz - uc, (len - t0 + UNIT - 1) / UNIT) : 0;

      auto page_of = [&](int t) {                   // page number of the group at t; -1: no tokens there
        return t < len ? __builtin_amdgcn_readfirstlane(table[fdiv(t, p.dpage) - p0]) : -1;
      };
      auto issue = [&](int i) {
        uint8_t* st = my_ring + (i % NS) * G::STAGE;
        int64_t at[2];                              // the groups' first rows; absent tokens: some page, not used
#pragma unroll
        for (int gr = 0; gr < 2; ++gr) {
          const int t = t0 + i * UNIT + gr * 16;
          const int pg = max(page_of(t), 0);
          const int off = t < len ? t - fdiv(t, p.dpage) * p.page : 0;
          at[gr] = ((int64_t)pg * p.hkv + h) * p.page + off;
#pragma unroll
          for (int n = 0; n < G::LOADS; ++n) {
            gload_lds16(p.kq + at[gr] * D, ksrc[n], lds_addr(st + gr * G::CODES + n * 1024));
            gload_lds16(p.vq + at[gr] * D, vsrc[n], lds_addr(st + (2 + gr) * G::CODES + n * 1024));
          }
        }
        constexpr int Q = D / 8;                    // dwords of one group's scales
#pragma unroll
        for (int n = 0; n < G::SLOADS; ++n) {
          const int e = n * 64 + lane, quarter = e / Q;
          const uint8_t* a = (quarter & 2 ? p.vs : p.ks) + (quarter & 1 ? at[1] : at[0]) * (D / 32);
          if (e < 4 * Q) gload_lds4(a + (e - quarter * Q) * 4, lds_addr(st + 4 * G::CODES + n * 256));
        }
      };
      auto compute = [&](int i) {
        const uint8_t* st = my_ring + (i % NS) * G::STAGE;
        const uint8_t* scales = st + 4 * G::CODES;
        const int t = t0 + i * UNIT, pg0 = page_of(t), pg1 = page_of(t + 16);
        // a tile that some row does not see whole: nodes, the sequence's end, an absent page (uniform)
        const bool special = t + TILE > prefix || t + TILE > len || pg0 < 0 || pg1 < 0;
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
        uint32_t sees[MT];                          // bit e: the row sees token e (special tiles)
        if (special) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const int m = mb * BR + mt * 16 + r16, nd = m < p.rows ? fdiv(m, p.dg) : here;
            uint64_t bits = 0;
            if (p.mask && nd < here) bits = (uint64_t)p.mask[(int64_t)b * p.T + nd];
            uint32_t see = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int tok = t + (e >> 2) * 16 + q4 * 4 + (e & 3), rel = tok - prefix;
              bool seen = tok < len && (e < 4 ? pg0 : pg1) >= 0 && nd < here;
              if (rel >= 0) seen = seen && (p.mask ? (bits >> (rel & 63) & 1) != 0 : rel <= nd);
              s[e >> 2][mt][e & 3] = seen ? s[e >> 2][mt][e & 3] : -__builtin_inff();
              see |= seen ? 1u << e : 0u;
            }
            sees[mt] = see;
          }
        } else {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) sees[mt] = 0xFF;
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          float x[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = s[e >> 2][mt][e & 3];
          float top = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7]))) * p.scale2;
          if (__any(top > mref[mt] + MOVE)) {
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            const float m = fmaxf(mref[mt], top), f = __builtin_amdgcn_exp2f(mref[mt] - m);
            mref[mt] = m;
            l[mt] *= f;
#pragma unroll
            for (int k = 0; k < ND; ++k) o[mt][k] *= f;
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            x[e] = __builtin_amdgcn_exp2f(fmaf(x[e], p.scale2, -mref[mt]));
            l[mt] += x[e];
          }
          const u32x4_t w = {pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                             pack_bf16x2(x[6], x[7])};
          pf[mt] = __builtin_bit_cast(bf16x8_t, w);
        }
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
          if (special) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (t + (e >> 2) * 16 + q4 * 4 + (e & 3) >= len || (e < 4 ? pg0 : pg1) < 0) {
                raw[e] = 0;
                f[e] = 1.f;
              }
          }
          bf16x8_t a[4];
          v_operands(raw, f, a);
          if (special) unseen_nonfinite<MT>(a, sees, &o[0][0] + 4 * c, ND);
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
              o[mt][4 * c + k] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[k], pf[mt], o[mt][4 * c + k], 0, 0, 0);
        }
      };

#pragma unroll 1
      for (int i = 0; i < NS && i < nt; ++i) issue(i);
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

    // join the waves: common reference, then the sums by a fixed tree (2, 3 into 0, 1; 1 into 0)
    __syncthreads();                                // the table's page numbers are done with
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      l[mt] += __shfl_xor(l[mt], 16);
      l[mt] += __shfl_xor(l[mt], 32);
      if (q4 == 0) stats[wave * BR + mt * 16 + r16] = make_float2(mref[mt], l[mt]);
    }
    __syncthreads();
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      float2 st[NW];
      float m = M_NONE;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        st[w] = stats[w * BR + mt * 16 + r16];
        m = fmaxf(m, st[w].x);
      }
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) sum += st[w].y * __builtin_amdgcn_exp2f(st[w].x - m);
      const float f = __builtin_amdgcn_exp2f(mref[mt] - m);
#pragma unroll
      for (int i = 0; i < ND; ++i) o[mt][i] *= f;
      mref[mt] = m;
      l[mt] = sum;
    }
    f32x4_t* join = reinterpret_cast<f32x4_t*>(ring);
    constexpr int SPAN = MT * ND * 64;
    auto put = [&](f32x4_t* d) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < ND; ++i) d[(mt * ND + i) * 64 + lane] = o[mt][i];
    };
    auto add = [&](const f32x4_t* d) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < ND; ++i) o[mt][i] += d[(mt * ND + i) * 64 + lane];
    };
    if (wave >= 2) put(join + (wave - 2) * SPAN);
    __syncthreads();
    if (wave < 2) add(join + wave * SPAN);
    if (wave == 1) put(join + SPAN);
    __syncthreads();
    if (wave == 0) {
      add(join + SPAN);
      const bool whole = ua == 0 && ub == units;
      const int64_t slot = (int64_t)blockIdx.x * 2 + (u == first_u ? 0 : 1);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const int row = mt * 16 + r16, m = mb * BR + row;
        if (m >= p.rows) continue;
        if (whole) {
          const int nd = fdiv(m, p.dg);
          const bool live = nd < here && l[mt] != 0.f;   // NaN passes
          const float f = 1.f / l[mt];
          uint16_t* dst = p.out + (((int64_t)b * p.T + nd) * p.hq + (int64_t)h * p.g + (m - nd * p.g)) * D;
#pragma unroll
          for (int c = 0; c < ND / 4; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              *reinterpret_cast<uint2*>(dst + v_value<D>(q4 * 4 + e, 4 * c)) =
                  live ? make_uint2(pack_bf16x2(o[mt][4 * c][e] * f, o[mt][4 * c + 1][e] * f),
                                    pack_bf16x2(o[mt][4 * c + 2][e] * f, o[mt][4 * c + 3][e] * f))
                       : make_uint2(0, 0);
        } else {
          float* dst = p.part + (slot * BR + row) * D;
#pragma unroll
          for (int c = 0; c < ND / 4; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              *reinterpret_cast<f32x4_t*>(dst + v_value<D>(q4 * 4 + e, 4 * c)) =
                  f32x4_t{o[mt][4 * c][e], o[mt][4 * c + 1][e], o[mt][4 * c + 2][e], o[mt][4 * c + 3][e]};
          if (q4 == 0) p.stat[slot * BR + row] = make_float2(mref[mt], l[mt]);
        }
      }
    }
    u += ub - ua;
    while (u < u_end && u >= base + seq_units(p, b) * ipb) {
      base += seq_units(p, b) * ipb;
      ++b;
    }
  }
}

// Join the partial results of the heads that several workgroups shared, and zero the rows that nobody
// wrote (empty sequences). A workgroup takes `jr` rows of a head and row block, so that there are about
// JOIN_BLOCKS of them: the search for the runs' owners comes before the first row. D/4 lanes hold
// four values of a row each; the workgroup's 256 / (D/4) slices take rows side by side, or, when a
// row's partial results are many, all take one row and every so-many-th result of it.
constexpr int JOIN_BLOCKS = 1024;
template <int D, int MT>
__global__ void __launch_bounds__(256) attention_join_kernel(AttnParams p, int jr, int jblocks) {
  constexpr int LD = D / 4, SL = 256 / LD, BR = MT * 16;
  __shared__ f32x4_t sums[SL][LD];
  const int lane = threadIdx.x & 63;
  const int part = blockIdx.x % (unsigned)jblocks;
  int r = blockIdx.x / (unsigned)jblocks;
  const int mb = r % p.mblocks;
  r /= p.mblocks;
  const int h = r % p.hkv, b = r / p.hkv;
  const int units = seq_units(p, b);
  const int row0 = part * jr, row1 = min(min(row0 + jr, BR), p.rows - mb * BR);
  const int here = p.nodes ? p.nodes[b] : p.T;
  const int c = threadIdx.x % LD, sl = threadIdx.x / LD;
  auto out_at = [&](int row) {
    const int m = mb * BR + row, node = fdiv(m, p.dg);
    return p.out + (((int64_t)b * p.T + node) * p.hq + (int64_t)h * p.g + (m - node * p.g)) * D + c * 4;
  };
  if (units == 0) {
    for (int row = row0 + sl; sl < SL && row < row1; row += SL) *reinterpret_cast<uint2*>(out_at(row)) = make_uint2(0, 0);
    return;
  }
  const Batch batch(p, lane);
  const int ipb = p.hkv * p.mblocks;
  const Runs runs(batch.total * ipb, p.nwg);
  const int u0 = batch.before(p, b) * ipb + (h * p.mblocks + mb) * units;
  const int w0 = runs.owner(u0), w1 = runs.owner(u0 + units - 1), n = w1 - w0 + 1;
  if (n == 1) return;
  const int64_t head = (int64_t)w0 * 2 + (runs.start(w0) < u0 ? 1 : 0);
  auto slot_of = [&](int w) { return (w == w0 ? head : (int64_t)w * 2) * BR; };
  auto store = [&](int row, const f32x4_t& acc, float l) {
    const float f = 1.f / l;
    const bool live = l != 0.f && fdiv(mb * BR + row, p.dg) < here;
    *reinterpret_cast<uint2*>(out_at(row)) =
        live ? make_uint2(pack_bf16x2(acc[0] * f, acc[1] * f), pack_bf16x2(acc[2] * f, acc[3] * f)) : make_uint2(0, 0);
  };
  // sum of the results w0 + first, + step, ... of one row, relative to its largest reference
  auto gather = [&](int row, int first, int step, float& top, float& l) {
    top = M_NONE;
    for (int w = w0; w <= w1; ++w) top = fmaxf(top, p.stat[slot_of(w) + row].x);
    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
    l = 0.f;
#pragma unroll 4
    for (int w = w0 + first; w <= w1; w += step) {
      const int64_t at = slot_of(w) + row;
      const float2 s = p.stat[at];
      const float f = __builtin_amdgcn_exp2f(s.x - top);
      l += s.y * f;
      acc += *reinterpret_cast<const f32x4_t*>(p.part + at * D + c * 4) * f;
    }
    return acc;
  };
  float top, l;
  if (n <= SL && row1 - row0 > 1) {
    for (int row = row0 + sl; sl < SL && row < row1; row += SL) {
      const f32x4_t acc = gather(row, 0, 1, top, l);
      store(row, acc, l);
    }
    return;
  }
  for (int row = row0; row < row1; ++row) {
    // references and sums by the lanes of every wave, the values by the slices
    top = M_NONE;
    for (int w = w0 + lane; w <= w1; w += 64) top = fmaxf(top, p.stat[slot_of(w) + row].x);
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) top = fmaxf(top, __shfl_xor(top, o));
    l = 0.f;
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

struct AttnPlan {
  int mt, mblocks, nwg;
};
// Row blocks of 16 * mt rows, and the grid: every unit its own workgroup up to two per CU.
AttnPlan attention_plan(const AttentionArgs& a) {
  const int64_t rows = a.T * (a.hq / a.cache.heads);
  const int most = a.cache.dim <= 128 ? 3 : 2;
  AttnPlan p;
  p.mt = (int)((rows + 15) / 16);
  if (p.mt > most) p.mt = most;
  p.mblocks = (int)((rows + p.mt * 16 - 1) / (p.mt * 16));
  const int64_t units = a.B * a.cache.heads * p.mblocks * ((a.max_len + UNIT - 1) / UNIT);
  p.nwg = (int)(units < 1 ? 1 : units > 512 ? 512 : units);
  return p;
}

template <int D, int MT, int NS>
int run(const AttnParams& p, hipStream_t stream) {
  hipLaunchKernelGGL((attention_kernel<D, MT, NS>), dim3((unsigned)p.nwg), dim3(64 * NW), 0, stream, p);
  if (hipGetLastError() != hipSuccess) return BSFP8_EHIP;
  const int64_t items = (int64_t)p.B * p.hkv * p.mblocks, rows = p.rows < MT * 16 ? p.rows : MT * 16;
  int64_t jr = items * rows / JOIN_BLOCKS;
  jr = jr < 1 ? 1 : jr > rows ? rows : jr;
  const int64_t jblocks = (rows + jr - 1) / jr;
  hipLaunchKernelGGL((attention_join_kernel<D, MT>), dim3((unsigned)(items * jblocks)), dim3(256), 0, stream, p, (int)jr,
                     (int)jblocks);
  return hip_status(hipGetLastError());
}

inline size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace

size_t attention_ws_bytes(const AttentionArgs& a) {
  const AttnPlan pl = attention_plan(a);
  const size_t rows = (size_t)pl.nwg * 2 * pl.mt * 16;
  return align256(rows * sizeof(float2)) + rows * (size_t)a.cache.dim * 4;
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
  p.stat = reinterpret_cast<float2*>(a.ws);
  p.part = reinterpret_cast<float*>(reinterpret_cast<char*>(a.ws) +
                                    align256((size_t)pl.nwg * 2 * pl.mt * 16 * sizeof(float2)));
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
  p.dpage = make_fastdiv((uint32_t)a.cache.page);
  p.dg = make_fastdiv((uint32_t)p.g);
  const int D = (int)a.cache.dim, mt = pl.mt;
  if (D == 64) return mt == 1 ? run<64, 1, 4>(p, stream) : mt == 2 ? run<64, 2, 4>(p, stream) : run<64, 3, 4>(p, stream);
  if (D == 128) return mt == 1 ? run<128, 1, 2>(p, stream) : mt == 2 ? run<128, 2, 2>(p, stream) : run<128, 3, 2>(p, stream);
  if (D == 192) return mt == 1 ? run<192, 1, 2>(p, stream) : run<192, 2, 2>(p, stream);
  return mt == 1 ? run<256, 1, 2>(p, stream) : run<256, 2, 2>(p, stream);
}

}  // namespace bsfp8
