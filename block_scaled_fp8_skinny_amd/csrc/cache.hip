// The paged MXFP8 key/value cache for gfx950 (MI355X): writing it (head norms, rotation and
// quantisation in one pass over the projection's output) and reading rows of it back.
//
// Both kernels move each byte once: HBM bounds them for many rows, the latency of one
// load-compute-store chain for few. Writing 8191 tokens (64 + 2 x 8 heads of 128, half of each rotated) takes 68 us,
// 4.7 TB/s (a copy here: 5.0), with the vector ALUs 82% busy, mostly unpacking, norms and codes; reading 65536 tokens of
// 8 heads of 128 takes 77 us, 5.3 TB/s; six tokens 3.9 us, 517 of 2 heads 2.6 us.

#include "device.h"

namespace bsfp8 {
namespace {

typedef __attribute__((ext_vector_type(2))) uint32_t u32x2_t;

constexpr int CW_THREADS = 256;

struct CacheWriteParams {
  const uint16_t *q, *k, *v, *qw, *kw;
  const float* cs;
  const int64_t *slots, *positions;
  uint16_t* q_out;
  uint8_t *kq, *ks, *vq, *vs;
  int64_t ldq, ldk, ldv, n_positions, n_slots;
  float eps;
  int64_t rows;
  int hq, hkv, page, rot, interleaved, parts, tokens;
  FastDiv dpage, dheads;
};

__device__ __forceinline__ void unpack8(const uint4& r, float (&x)[8]) {
  const uint32_t d[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(d[i] << 16);
    x[2 * i + 1] = __uint_as_float(d[i] & 0xFFFF0000u);
  }
}

// One head of one token is held by LPH neighbouring lanes, eight values each (one 16-byte load):
//   norm      sum of squares by lane exchanges inside the LPH lanes;
//   rotation  value i pairs with i + rot/2, rot/16 lanes away (the halves are whole lanes since
//             rot % 16 == 0), or with its neighbour inside the lane when interleaved: every lane
//             keeps its eight cosines and signed sines in registers for all heads of its token;
//   MXFP8     a 32-value block is four neighbouring lanes: its maximum by two exchanges.
// A workgroup holds one token (blockIdx.x) and, for few tokens, a part of its heads (blockIdx.y),
// CW_THREADS / LPH heads at a time; the next head's load is issued before this one is computed. Tokens of few heads
// share a workgroup (p.tokens of them), all heads at once.
// (an instance of its own: with a token for each lane its addresses are vectors, which cost 10% of a prompt's time)
template <int D, bool SHARED>
__global__ void __launch_bounds__(CW_THREADS) cache_write_kernel(CacheWriteParams p) {
  constexpr int LPH = D == 64 ? 8 : D == 128 ? 16 : 32;   // lanes per head (24 of 32 used for 192)
  constexpr int GROUPS = CW_THREADS / LPH;
  const int sub = threadIdx.x % LPH, grp = threadIdx.x / LPH;
  const int heads = p.hq + 2 * p.hkv;
  const int mine = SHARED ? fdiv(grp, p.dheads) : 0;   // of the workgroup's tokens
  const int64_t r = SHARED ? (int64_t)blockIdx.x * p.tokens + mine : blockIdx.x;
  if (SHARED && (mine >= p.tokens || r >= p.rows)) return;   // whole heads leave together
  const bool on = sub * 8 < D;
  const int d0 = sub * 8;
  const int base = (threadIdx.x & 63) - sub;        // the head's first lane in its wave
  const int step = SHARED ? heads : p.parts * GROUPS;

  const int64_t slot = p.slots[r];
  const bool stored = slot >= 0 && slot < p.n_slots;
  const int pg = stored ? fdiv((int)slot, p.dpage) : 0;
  const int off = stored ? (int)slot - pg * p.page : 0;

  auto load = [&](int h) {
    const uint16_t* src = h < p.hq ? p.q + r * p.ldq + (int64_t)h * D
                          : h < p.hq + p.hkv ? p.k + r * p.ldk + (int64_t)(h - p.hq) * D
                                             : p.v + r * p.ldv + (int64_t)(h - p.hq - p.hkv) * D;
    return on ? *reinterpret_cast<const uint4*>(src + d0) : make_uint4(0, 0, 0, 0);
  };
  int h = SHARED ? grp - mine * heads : blockIdx.y * GROUPS + grp;
  if (h >= heads) return;
  uint4 next = load(h);

  // cosines and sines of the lane's values; sines carry the sign of the partner's term
  float cs[8], sn[8];
  const int half = p.rot >> 1;
  const bool turns = d0 < p.rot && on;
  int partner = threadIdx.x & 63;
  if (turns) {
    const int64_t pos = p.positions[r];
    const bool known = pos >= 0 && pos < p.n_positions;
    const float* row = p.cs + (known ? pos : 0) * p.rot;
    if (p.interleaved) {
      const f32x4_t c = *reinterpret_cast<const f32x4_t*>(row + d0 / 2);
      const f32x4_t s = *reinterpret_cast<const f32x4_t*>(row + half + d0 / 2);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        cs[i] = c[i / 2];
        sn[i] = (i & 1) ? s[i / 2] : -s[i / 2];
      }
    } else {
      const bool first = d0 < half;
      const int j = first ? d0 : d0 - half;
      partner = base + (first ? sub + half / 8 : sub - half / 8);
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        const f32x4_t c = *reinterpret_cast<const f32x4_t*>(row + j + i);
        const f32x4_t s = *reinterpret_cast<const f32x4_t*>(row + half + j + i);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          cs[i + e] = c[e];
          sn[i + e] = first ? -s[e] : s[e];
        }
      }
    }
    if (!known) {
#pragma unroll
      for (int i = 0; i < 8; ++i) cs[i] = sn[i] = __uint_as_float(0x7FC00000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      cs[i] = 1.f;
      sn[i] = 0.f;
    }
  }

  for (; h < heads; h += step) {
    float x[8];
    unpack8(next, x);
    if (h + step < heads) next = load(h + step);
    const bool is_q = h < p.hq, is_v = h >= p.hq + p.hkv;
    const uint16_t* w = is_q ? p.qw : p.kw;
    if (!is_v && w) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) s += x[i] * x[i];
#pragma unroll
      for (int o = 1; o < LPH; o <<= 1) s += __shfl_xor(s, o);
      const float inv = rsqrtf(s * (1.f / D) + p.eps);
      float wf[8];
      unpack8(on ? *reinterpret_cast<const uint4*>(w + d0) : make_uint4(0, 0, 0, 0), wf);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * wf[i];
    }
    if (!is_v && p.rot) {
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = p.interleaved ? x[i ^ 1] : __shfl(x[i], partner);
      if (turns) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x[i] * cs[i] + y[i] * sn[i];
      }
    }
    if (is_q) {
      if (on)
        *reinterpret_cast<uint4*>(p.q_out + (r * p.hq + h) * D + d0) = make_uint4(
            pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
      continue;
    }
    // the rule of quantize_mx_kernel on the fp32 values (inf and NaN patterns exceed every finite one)
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(x[i]) & 0x7FFFFFFFu);
    amax = max(amax, (uint32_t)__shfl_xor((int)amax, 1));
    amax = max(amax, (uint32_t)__shfl_xor((int)amax, 2));
    const int E = (int)(amax >> 23);
    const int s = max(E == 0 ? -127 : E - 135, -127);
    const bool finite = E != 255;
    uint32_t c[2];
    if (finite) {
      float sv[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) sv[i] = fminf(fmaxf(ldexpf(x[i], -s), -448.f), 448.f);
      c[0] = e4m3x4(sv[0], sv[1], sv[2], sv[3]);
      c[1] = e4m3x4(sv[4], sv[5], sv[6], sv[7]);
    } else {
      c[0] = c[1] = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i >> 2] |= ((__float_as_uint(x[i]) >> 31) ? 0xFFu : 0x7Fu) << (8 * (i & 3));
    }
    if (stored && on) {
      const int hk = is_v ? h - p.hq - p.hkv : h - p.hq;
      const int64_t row = ((int64_t)pg * p.hkv + hk) * p.page + off;
      uint8_t* codes = is_v ? p.vq : p.kq;
      uint8_t* scales = is_v ? p.vs : p.ks;
      *reinterpret_cast<u32x2_t*>(codes + row * D + d0) = u32x2_t{c[0], c[1]};
      if ((sub & 3) == 0) scales[row * (D / 32) + sub / 4] = finite ? (uint8_t)(s + 127) : (uint8_t)255;
    }
  }
}

struct CacheReadParams {
  const uint8_t *kq, *ks, *vq, *vs;
  const int64_t* slots;
  uint16_t *k_out, *v_out;
  int64_t n_slots, rows;                            // rows = tokens * heads
  int heads, page;
  FastDiv dpage, dheads;
};

// Sixteen codes per lane: one 16-byte load, eight conversions, two 16-byte stores; blockIdx.y is 0 for
// keys, 1 for values.
template <int D>
__global__ void __launch_bounds__(256) cache_read_kernel(CacheReadParams p) {
  constexpr int LPR = D / 16;                       // lanes per row
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = t / LPR;
  const int c = (int)(t % LPR);
  if (row >= p.rows) return;
  const int r = fdiv((int)row, p.dheads);
  const int h = (int)row - r * p.heads;
  const int64_t slot = p.slots[r];
  const uint8_t* codes = blockIdx.y ? p.vq : p.kq;
  const uint8_t* scales = blockIdx.y ? p.vs : p.ks;
  u32x4_t o[2] = {};
  if (slot >= 0 && slot < p.n_slots) {
    const int pg = fdiv((int)slot, p.dpage);
    const int64_t at = ((int64_t)pg * p.heads + h) * p.page + ((int)slot - pg * p.page);
    const uint4 q = *reinterpret_cast<const uint4*>(codes + at * D + c * 16);
    const float s = block_scale(scales[at * (D / 32) + c / 2]);
    o[0] = __builtin_bit_cast(u32x4_t, dequant8(q.x, q.y, s));
    o[1] = __builtin_bit_cast(u32x4_t, dequant8(q.z, q.w, s));
  }
  u32x4_t* dst = reinterpret_cast<u32x4_t*>((blockIdx.y ? p.v_out : p.k_out) + row * D + c * 16);
  dst[0] = o[0];
  dst[1] = o[1];
}

template <int D>
void write_rows(const CacheWriteParams& p, dim3 grid, hipStream_t stream) {
  if (p.tokens > 1) hipLaunchKernelGGL((cache_write_kernel<D, true>), grid, dim3(CW_THREADS), 0, stream, p);
  else hipLaunchKernelGGL((cache_write_kernel<D, false>), grid, dim3(CW_THREADS), 0, stream, p);
}

}  // namespace

int launch_cache_write(const CacheWriteArgs& a, hipStream_t stream) {
  CacheWriteParams p{};
  p.q = a.q;
  p.k = a.k;
  p.v = a.v;
  p.qw = a.q_weight;
  p.kw = a.k_weight;
  p.cs = a.cos_sin;
  p.slots = a.slots;
  p.positions = a.positions;
  p.q_out = a.q_out;
  p.kq = a.cache.kq;
  p.ks = a.cache.ks;
  p.vq = a.cache.vq;
  p.vs = a.cache.vs;
  p.ldq = a.ldq;
  p.ldk = a.ldk;
  p.ldv = a.ldv;
  p.n_positions = a.n_positions;
  p.n_slots = a.cache.pages * a.cache.page;
  p.eps = a.eps;
  p.hq = (int)a.hq;
  p.hkv = (int)a.cache.heads;
  p.page = (int)a.cache.page;
  p.rot = (int)a.rot;
  p.interleaved = a.interleaved;
  p.dpage = make_fastdiv((uint32_t)a.cache.page);
  const int D = (int)a.cache.dim;
  const int groups = CW_THREADS / (D == 64 ? 8 : D == 128 ? 16 : 32);
  const int rounds = (p.hq + 2 * p.hkv + groups - 1) / groups;
  // a token's heads over several workgroups while the tokens alone do not fill the GPU (256 CUs of
  // eight such workgroups)
  p.parts = a.R >= 2048 ? 1 : (int)((2048 + a.R - 1) / a.R);
  if (p.parts > rounds) p.parts = rounds;
  // tokens whose heads leave half of a workgroup or more idle share one, once there are enough for that (27210 tokens of
  // 8 + 2 heads of 64: 23.5 against 28.8 us)
  const int heads = p.hq + 2 * p.hkv;
  p.tokens = a.R >= 2048 && heads * 2 <= groups ? groups / heads : 1;
  p.rows = a.R;
  p.dheads = make_fastdiv((uint32_t)heads);
  const dim3 grid((unsigned)((a.R + p.tokens - 1) / p.tokens), (unsigned)p.parts);
  if (D == 64) write_rows<64>(p, grid, stream);
  else if (D == 128) write_rows<128>(p, grid, stream);
  else if (D == 192) write_rows<192>(p, grid, stream);
  else write_rows<256>(p, grid, stream);
  return hip_status(hipGetLastError());
}

int launch_cache_read(const bsfp8_kv_cache& c, const int64_t* slots, int64_t R, uint16_t* k_out, uint16_t* v_out,
                      hipStream_t stream) {
  CacheReadParams p{};
  p.kq = c.kq;
  p.ks = c.ks;
  p.vq = c.vq;
  p.vs = c.vs;
  p.slots = slots;
  p.k_out = k_out;
  p.v_out = v_out;
  p.n_slots = c.pages * c.page;
  p.rows = R * c.heads;
  p.heads = (int)c.heads;
  p.page = (int)c.page;
  p.dpage = make_fastdiv((uint32_t)c.page);
  p.dheads = make_fastdiv((uint32_t)c.heads);
  const int D = (int)c.dim;
  const dim3 grid((unsigned)((p.rows * (D / 16) + 255) / 256), 2);
  if (D == 64) hipLaunchKernelGGL(cache_read_kernel<64>, grid, dim3(256), 0, stream, p);
  else if (D == 128) hipLaunchKernelGGL(cache_read_kernel<128>, grid, dim3(256), 0, stream, p);
  else if (D == 192) hipLaunchKernelGGL(cache_read_kernel<192>, grid, dim3(256), 0, stream, p);
  else hipLaunchKernelGGL(cache_read_kernel<256>, grid, dim3(256), 0, stream, p);
  return hip_status(hipGetLastError());
}

}  // namespace bsfp8
