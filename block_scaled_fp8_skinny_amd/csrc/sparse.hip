// Which pages of the paged MXFP8 cache a query attends to, for gfx950 (MI355X): bounds of each page's keys, and the pages
// with the largest bound of a query's scores.
//
// With kmin, kmax the least and largest value of each key dimension over a page's tokens,
//   u = sum_d max(q_d kmin_d, q_d kmax_d)
// is at least q . k for every key of the page; a page's score for one token and key/value head is the largest u of the
// query heads that share the head. Bounds are the cache's own values (e4m3 codes times scales, exact in bf16), so they are
// exact and do not depend on an order. Scores are sums of products of bf16 values in fp64, where they are exact but for
// queries and keys of extreme range: which page is the last to be taken is a decision between neighbours.

#include "lanes.h"

namespace bsfp8 {
namespace {

// ---------------------------------------------------------------------------------------------
// bounds
// ---------------------------------------------------------------------------------------------
struct BoundsParams {
  const uint8_t *kq, *ks;
  const int32_t *pages, *lens, *first;
  uint16_t* bounds;
  int64_t ld_pages, n_pages, items;                 // items: B * heads * per
  int heads, page, max_new, per, max_len;           // per: pages of a sequence that a call may touch
  FastDiv dpage, dheads, dper;
};

// A wave for each page and head. A token's codes lie on D/16 lanes (16 each; 12 of 16 lanes used for 192), the wave takes
// 64 / LPT tokens at a time, BATCH such loads in flight; a token past the sequence's end repeats the last one, which
// changes neither bound. Bound by HBM for a prompt.
template <int D>
__global__ void __launch_bounds__(256) cache_bounds_kernel(BoundsParams p) {
  constexpr int LPT = D == 64 ? 4 : D == 128 ? 8 : 16, TOKENS = 64 / LPT, BATCH = 8;
  const int lane = threadIdx.x & 63;
  const int64_t item = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (item >= p.items) return;
  // item = (sequence, page of those touched, head)
  const int bp = fdiv((int)item, p.dheads), h = (int)item - bp * p.heads;
  const int b = fdiv(bp, p.dper), k = bp - b * p.per;
  const int len = max(0, min(p.lens[b], p.max_len));
  int from = p.first ? max(0, min(p.first[b], len)) : 0;
  from = max(from, len - p.max_new);
  const int j = fdiv(from, p.dpage) + k;
  const int64_t t0 = (int64_t)j * p.page;
  if (from >= len || t0 >= len) return;
  const int id = p.pages[(int64_t)b * p.ld_pages + j];
  if (id < 0 || id >= p.n_pages) return;
  const int tokens = min(p.page, (int)(len - t0));  // of the page that are there
  const int sub = lane % LPT, tok = lane / LPT;
  const bool on = sub * 16 < D;
  const int64_t row0 = ((int64_t)id * p.heads + h) * p.page;
  const uint8_t* codes = p.kq + row0 * D + (on ? sub * 16 : 0);
  const uint8_t* scales = p.ks + row0 * (D / 32) + (on ? sub / 2 : 0);
  float lo[16], hi[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    lo[i] = __builtin_inff();
    hi[i] = -__builtin_inff();
  }
  uint32_t nan = 0;                                 // bit i: a NaN among value i
  for (int s0 = 0; s0 < tokens; s0 += TOKENS * BATCH) {
    u32x4_t w[BATCH];
    uint32_t e[BATCH];
#pragma unroll
    for (int n = 0; n < BATCH; ++n) {
      const int at = min(s0 + n * TOKENS + tok, tokens - 1);
      w[n] = *reinterpret_cast<const u32x4_t*>(codes + (int64_t)at * D);
      e[n] = scales[(int64_t)at * (D / 32)];
    }
#pragma unroll
    for (int n = 0; n < BATCH; ++n) {
      if (s0 + n * TOKENS >= tokens) break;         // uniform
      const float f = block_scale(e[n]);
      const bf16x8_t a = dequant8(w[n][0], w[n][1], f), c = dequant8(w[n][2], w[n][3], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float x = (float)a[i], y = (float)c[i];
        lo[i] = fminf(lo[i], x);
        hi[i] = fmaxf(hi[i], x);
        lo[8 + i] = fminf(lo[8 + i], y);
        hi[8 + i] = fmaxf(hi[8 + i], y);
      }
      uint32_t code = 0;                            // a NaN code is all ones but its sign
#pragma unroll
      for (int i = 0; i < 4; ++i) code |= ((w[n][i] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
      if (__any(code != 0 || e[n] == 255)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) nan |= ((float)a[i] != (float)a[i] ? 1u : 0u) << i | ((float)c[i] != (float)c[i] ? 1u : 0u) << (8 + i);
      }
    }
  }
#pragma unroll
  for (int o = LPT; o < 64; o <<= 1) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      lo[i] = fminf(lo[i], __shfl_xor(lo[i], o));
      hi[i] = fmaxf(hi[i], __shfl_xor(hi[i], o));
    }
    nan |= (uint32_t)__shfl_xor((int)nan, o);
  }
  if (nan) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (nan >> i & 1) lo[i] = hi[i] = __uint_as_float(0x7FC00000u);
  }
  if (tok < 2 && on) {                              // lane group 0 stores the least values, 1 the largest
    uint16_t* dst = p.bounds + (((int64_t)id * p.heads + h) * 2 + tok) * D + sub * 16;
    u32x4_t o[2];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      o[i >> 2][i & 3] = tok ? pack_bf16x2(hi[2 * i], hi[2 * i + 1]) : pack_bf16x2(lo[2 * i], lo[2 * i + 1]);
    reinterpret_cast<u32x4_t*>(dst)[0] = o[0];
    reinterpret_cast<u32x4_t*>(dst)[1] = o[1];
  }
}

// ---------------------------------------------------------------------------------------------
// scores
// ---------------------------------------------------------------------------------------------
struct SelectParams {
  const uint16_t *q, *bounds;
  const int32_t *pages, *lens, *nodes;
  uint64_t* keys;                                   // [B * T][heads][width]
  int32_t *selected, *held;
  int64_t ldq, ld_pages, n_pages;
  int B, T, hq, heads, g, page, max_len, width, count, sinks, recent;
  int gp, tokens, blocks;                           // see select_score_kernel
  FastDiv dpage;
};

// Positions that node t of sequence b sees: its own and those before it.
__device__ __forceinline__ int positions_seen(const SelectParams& p, int b, int t) {
  const int len = max(0, min(p.lens[b], p.max_len)), here = p.nodes ? max(0, min(p.nodes[b], p.T)) : p.T;
  return t < here ? max(0, len - here + t + 1) : 0;
}
__device__ __forceinline__ int pages_for(const SelectParams& p, int n) { return n > 0 ? fdiv(n - 1, p.dpage) + 1 : 0; }

// Scores ordered as integers: a page that does not exist 0, else above it; infinite for bounds or queries that are not finite.
__device__ __forceinline__ uint64_t score_key(double u) {
  u += 0.0;                                         // -0 is 0
  const uint64_t b = __builtin_bit_cast(uint64_t, u);
  return b >> 63 ? ~b : b | 0x8000000000000000ull;
}

typedef double f64x4_t __attribute__((ext_vector_type(4)));

// One wave scores 16 pages of a sequence and head for all of its tokens, by fp64 matrix products of 16 rows x 16 pages x 4
// values: the row's positive part times the largest values plus its negative part times the least. A lane loads eight
// neighbouring values of its page (lane % 16) and row at a time; which of them meet in one product is free as long as
// both sides agree. Rows: the g query heads of a token are filled up to gp = 1, 2, 4, 8 or 16 by repeating the last one
// (or take several blocks of 16), so that a token's maximum is taken over whole registers and lane groups; `tokens` of
// them in a block of rows. Element r of a lane's result is row 4 r + lane / 16 of its page.
template <int D>
__global__ void __launch_bounds__(256) select_score_kernel(SelectParams p) {
  constexpr int STEPS = D / 32;
  const int lane = threadIdx.x & 63, r16 = lane & 15, q4 = lane >> 4;
  const int b = blockIdx.x / p.heads, h = blockIdx.x - b * p.heads;
  const int j0 = (blockIdx.y * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * 16;
  const int most = pages_for(p, max(0, min(p.lens[b], p.max_len)));
  if (j0 >= most) return;
  const int j = j0 + r16;
  const int id = j < most ? p.pages[(int64_t)b * p.ld_pages + j] : -1;
  const bool there = id >= 0 && id < p.n_pages;
  const uint16_t* at = p.bounds + ((int64_t)(there ? id : 0) * p.heads + h) * 2 * D + q4 * 8;
  u32x4_t lo[STEPS], hi[STEPS];
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    lo[s] = *reinterpret_cast<const u32x4_t*>(at + s * 32);
    hi[s] = *reinterpret_cast<const u32x4_t*>(at + D + s * 32);
  }
  for (int rb = 0; rb * p.tokens < p.T; ++rb) {
    double best[4];                                 // largest so far: by register, over a token's blocks of heads
#pragma unroll
    for (int r = 0; r < 4; ++r) best[r] = -__builtin_inf();
    const int t = rb * p.tokens + (p.blocks > 1 ? 0 : r16 / p.gp);
    for (int blk = 0; blk < p.blocks; ++blk) {
      const int head = min(blk * 16 + (p.blocks > 1 ? r16 : r16 % p.gp), p.g - 1);
      const uint16_t* qr = p.q + ((int64_t)b * p.T + min(t, p.T - 1)) * p.ldq + ((int64_t)h * p.g + head) * D + q4 * 8;
      f64x4_t acc = {0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        const u32x4_t w = *reinterpret_cast<const u32x4_t*>(qr + s * 32);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t shift = i & 1 ? 0 : 16;
          const float x = __uint_as_float((w[i / 2] << shift) & 0xFFFF0000u);
          const float l = __uint_as_float((lo[s][i / 2] << shift) & 0xFFFF0000u);
          const float m = __uint_as_float((hi[s][i / 2] << shift) & 0xFFFF0000u);
          // (NaN passes to both)
          acc = __builtin_amdgcn_mfma_f64_16x16x4f64((double)(x <= 0.f ? 0.f : x), (double)m, acc, 0, 0, 0);
          acc = __builtin_amdgcn_mfma_f64_16x16x4f64((double)(x >= 0.f ? 0.f : x), (double)l, acc, 0, 0, 0);
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const double u = __builtin_fabs(acc[r]) < __builtin_inf() ? acc[r] : __builtin_inf();
        best[r] = fmax(best[r], u);
      }
    }
    // over the rows of a token: 16 / gp tokens in the block
    const int gp = p.blocks > 1 ? 16 : p.gp;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (gp >= 2) best[r] = fmax(best[r], __shfl_xor(best[r], 16));
      if (gp >= 4) best[r] = fmax(best[r], __shfl_xor(best[r], 32));
    }
    if (gp >= 8) {
      best[0] = fmax(best[0], best[1]);
      best[2] = fmax(best[2], best[3]);
    }
    if (gp >= 16) best[0] = fmax(best[0], best[2]);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 4 * r + q4, tt = rb * p.tokens + row / gp;
      if (row % gp == 0 && tt < p.T && j < most)
        p.keys[(((int64_t)b * p.T + tt) * p.heads + h) * p.width + j] = there ? score_key(best[r]) : 0ull;
    }
  }
}

// ---------------------------------------------------------------------------------------------
// the pages with the largest scores
// ---------------------------------------------------------------------------------------------
constexpr int PICK_LIST = 64;                       // keys that one wave ranks against each other
constexpr int PICK_HELD = 8;                        // keys of a thread, where they are held

// The list of one token and head (a workgroup): the first `sinks` and the last `recent` of its N pages and, of the others,
// those with the largest keys, the lower index first among equals. The least key that is taken is found by histograms of
// the keys still in question, over the range that they span: each splits it into up to 4 * THREADS parts, keeps the one that
// holds the border, and usually leaves a handful after the first, which one wave ranks against each other. What is in the
// list is then counted off in the order of the pages. HELD: the keys stay in registers, PICK_HELD a thread (else they
// are read again in each round).
template <int THREADS, bool HELD>
__global__ void __launch_bounds__(THREADS) select_pick_kernel(SelectParams p) {
  constexpr int WAVES = THREADS / 64, BINS = THREADS * 4, BIN_BITS = THREADS == 256 ? 10 : 12;
  static_assert(BINS == 1 << BIN_BITS, "bins");
  __shared__ __align__(16) int bins[BINS];
  __shared__ uint64_t list[PICK_LIST];
  __shared__ int list_at[PICK_LIST];
  __shared__ uint32_t lows[WAVES], highs[WAVES];
  __shared__ int sums[HELD ? PICK_HELD * WAVES : WAVES], found[3], n_list, last_at;
  __shared__ uint64_t last_key;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = blockIdx.x / p.heads, h = blockIdx.x - r * p.heads, b = r / p.T;
  const int n = positions_seen(p, b, r - b * p.T), N = pages_for(p, n);
  int32_t* out = p.selected + ((int64_t)r * p.heads + h) * p.count;
  const int m = min(N, p.count);
  if (h == 0 && tid == 0) p.held[r] = N > 0 ? (m - 1) * p.page + (n - (N - 1) * p.page) : 0;
  for (int i = m + tid; i < p.count; i += THREADS) out[i] = -1;
  const int32_t* table = p.pages + (int64_t)b * p.ld_pages;
  auto entry = [&](int j) {
    const int id = table[j];
    return id >= 0 && id < p.n_pages ? id : -1;
  };
  if (N <= p.count) {
    for (int i = tid; i < N; i += THREADS) out[i] = entry(i);
    return;
  }
  // in question: pages sinks .. N - recent - 1 (more than are needed, so N - recent > sinks)
  const uint64_t* keys = p.keys + ((int64_t)r * p.heads + h) * p.width;
  const int j0 = p.sinks, j1 = N - p.recent;
  uint64_t held[HELD ? PICK_HELD : 1];
  if constexpr (HELD) {
#pragma unroll
    for (int k = 0; k < PICK_HELD; ++k) {
      const int j = k * THREADS + tid;
      held[k] = j < N ? keys[j] : 0;
    }
  }
  // f(page, key) of the thread's pages in question
  auto each = [&](auto f) {
    if constexpr (HELD) {
#pragma unroll
      for (int k = 0; k < PICK_HELD; ++k) {
        const int j = k * THREADS + tid;
        if (k * THREADS >= N) break;                // uniform
        if (j >= j0 && j < j1) f(j, held[k]);
      }
    } else {
      for (int j = j0 + tid; j < j1; j += THREADS) f(j, keys[j]);
    }
  };
  auto clear = [&] { *reinterpret_cast<int4*>(bins + tid * 4) = make_int4(0, 0, 0, 0); };
  int need = p.count - p.sinks - p.recent;
  // taken: keys above `edge`, and of those equal to it the ones up to page `last`
  uint64_t edge = ~0ull;
  int last = -1;
  if (need > 0) {
    uint32_t low = ~0u, high = 0;                   // of the keys' upper halves
    each([&](int, uint64_t k) {
      low = min(low, (uint32_t)(k >> 32));
      high = max(high, (uint32_t)(k >> 32));
    });
    low = wave_reduce(low, [](uint32_t x, uint32_t y) { return min(x, y); });
    high = wave_reduce(high, [](uint32_t x, uint32_t y) { return max(x, y); });
    if (lane == 0) {
      lows[wave] = low;
      highs[wave] = high;
    }
    if (tid == 0) n_list = 0;
    clear();
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      low = min(low, lows[w]);
      high = max(high, highs[w]);
    }
    uint64_t lo = (uint64_t)low << 32, hi = (uint64_t)high << 32 | 0xFFFFFFFFull;
    int left = j1 - j0;                             // keys in [lo, hi]
    // each round leaves a shorter range: at most seven for 64 bits
    while (left > PICK_LIST && lo < hi) {
      const int shift = max(64 - __builtin_clzll(hi - lo) - BIN_BITS, 0);
      each([&](int, uint64_t k) {
        if (k >= lo && k <= hi) atomicAdd(&bins[(int)((hi - k) >> shift)], 1);
      });
      __syncthreads();
      const int4 own4 = *reinterpret_cast<const int4*>(bins + tid * 4);
      const int own[4] = {own4.x, own4.y, own4.z, own4.w}, sum = own[0] + own[1] + own[2] + own[3];
      const int run = (int)wave_scan((uint32_t)sum);
      if (lane == 63) sums[wave] = run;
      clear();
      __syncthreads();
      int before = run - sum;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) before += w < wave ? sums[w] : 0;
      if (before < need && before + sum >= need) {  // one thread's: left >= need
        int bin = tid * 4;
#pragma unroll
        for (int k = 0; k < 3; ++k)
          if (bin == tid * 4 + k && before + own[k] < need) {
            before += own[k];
            ++bin;
          }
        found[0] = bin;
        found[1] = before;
        found[2] = own[bin - tid * 4 == 0 ? 0 : bin - tid * 4 == 1 ? 1 : bin - tid * 4 == 2 ? 2 : 3];
      }
      __syncthreads();
      need -= found[1];
      left = found[2];
      const uint64_t top = hi - ((uint64_t)found[0] << shift), part = (1ull << shift) - 1;
      lo = top - lo > part ? top - part : lo;
      hi = top;
    }
    edge = lo;
    if (left == need) {                             // all of them: keys from lo on
      last = N;
    } else if (left <= PICK_LIST) {
      each([&](int j, uint64_t k) {
        if (k >= lo && k <= hi) {
          const int i = atomicAdd(&n_list, 1);
          list[i] = k;
          list_at[i] = j;
        }
      });
      __syncthreads();
      if (wave == 0) {
        const uint64_t k = lane < left ? list[lane] : 0;
        const int j = lane < left ? list_at[lane] : 0;
        int rank = 0;
        for (int i = 0; i < left; ++i) {            // (uniform)
          const uint64_t o = from_lane(k, i);
          rank += o > k || (o == k && __builtin_amdgcn_readlane(j, i) < j) ? 1 : 0;
        }
        if (lane < left && rank == need - 1) {
          last_key = k;
          last_at = j;
        }
      }
      __syncthreads();
      edge = last_key;
      last = last_at;
    } else {                                        // equal keys: the first `need` of them
      int seen = 0;
      for (int i0 = j0; i0 < j1; i0 += THREADS) {
        const int j = i0 + tid;
        const bool is = j < j1 && keys[j] == lo;
        const uint64_t mask = __ballot(is);
        __syncthreads();
        if (lane == 0) sums[wave] = __builtin_popcountll(mask);
        __syncthreads();
        int at = seen + __builtin_popcountll(mask & ((1ull << lane) - 1));
        for (int w = 0; w < WAVES; ++w) {
          if (w < wave) at += sums[w];
          seen += sums[w];
        }
        if (is && at == need - 1) last_at = j;
        if (seen >= need) break;                    // uniform
      }
      __syncthreads();
      last = last_at;
    }
  }
  // in the order of the pages
  auto in = [&](int j, uint64_t k) { return j < N && (j < j0 || j >= j1 || k > edge || (k == edge && j <= last)); };
  const uint64_t below = (1ull << lane) - 1;
  if constexpr (HELD) {
    uint64_t mask[PICK_HELD];
    __syncthreads();                                // `sums` is free
#pragma unroll
    for (int k = 0; k < PICK_HELD; ++k) {
      mask[k] = __ballot(in(k * THREADS + tid, held[k]));
      if (lane == 0) sums[k * WAVES + wave] = __builtin_popcountll(mask[k]);
    }
    __syncthreads();
    int base = 0;
#pragma unroll
    for (int k = 0; k < PICK_HELD; ++k) {
      if (k * THREADS >= N) break;                  // uniform
      int at = base;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) {
        at += w < wave ? sums[k * WAVES + w] : 0;
        base += sums[k * WAVES + w];
      }
      if (mask[k] >> lane & 1) out[at + __builtin_popcountll(mask[k] & below)] = entry(k * THREADS + tid);
    }
  } else {
    int base = 0;
    for (int i0 = 0; i0 < N; i0 += THREADS) {
      const int j = i0 + tid;
      const bool is = j < N && in(j, keys[j]);
      const uint64_t mask = __ballot(is);
      __syncthreads();
      if (lane == 0) sums[wave] = __builtin_popcountll(mask);
      __syncthreads();
      int at = base + __builtin_popcountll(mask & below);
      for (int w = 0; w < WAVES; ++w) {
        if (w < wave) at += sums[w];
        base += sums[w];
      }
      if (is) out[at] = entry(j);
    }
  }
}

}  // namespace

int launch_cache_bounds(const CacheBoundsArgs& a, hipStream_t stream) {
  BoundsParams p{};
  p.kq = a.cache.kq;
  p.ks = a.cache.ks;
  p.pages = a.pages;
  p.lens = a.lens;
  p.first = a.first;
  p.bounds = a.bounds;
  p.ld_pages = a.ld_pages;
  p.n_pages = a.cache.pages;
  p.heads = (int)a.cache.heads;
  p.page = (int)a.cache.page;
  const int64_t held = a.ld_pages * a.cache.page;
  p.max_len = (int)(held < INT32_MAX ? held : INT32_MAX);
  p.max_new = (int)a.max_new;
  p.per = (int)bounds_pages(a);
  p.items = a.B * a.cache.heads * p.per;
  p.dpage = make_fastdiv((uint32_t)a.cache.page);
  p.dheads = make_fastdiv((uint32_t)a.cache.heads);
  p.dper = make_fastdiv((uint32_t)p.per);
  const dim3 grid((unsigned)((p.items + 3) / 4));
  const int D = (int)a.cache.dim;
  if (D == 64) hipLaunchKernelGGL(cache_bounds_kernel<64>, grid, dim3(256), 0, stream, p);
  else if (D == 128) hipLaunchKernelGGL(cache_bounds_kernel<128>, grid, dim3(256), 0, stream, p);
  else if (D == 192) hipLaunchKernelGGL(cache_bounds_kernel<192>, grid, dim3(256), 0, stream, p);
  else hipLaunchKernelGGL(cache_bounds_kernel<256>, grid, dim3(256), 0, stream, p);
  return hip_status(hipGetLastError());
}

// Pages of a sequence that max_new positions can touch.
int64_t bounds_pages(const CacheBoundsArgs& a) {
  const int64_t n = (a.max_new - 1 + a.cache.page - 1) / a.cache.page + 1;
  return n < a.ld_pages ? n : a.ld_pages;
}

size_t select_ws_bytes(int64_t B, int64_t T, int64_t hkv, int64_t width) { return (size_t)B * T * hkv * width * 8; }

int launch_select_pages(const SelectPagesArgs& a, hipStream_t stream) {
  SelectParams p{};
  p.q = a.q;
  p.bounds = a.bounds;
  p.pages = a.pages;
  p.lens = a.lens;
  p.nodes = a.nodes;
  p.keys = reinterpret_cast<uint64_t*>(a.ws);
  p.selected = a.selected;
  p.held = a.held;
  p.ldq = a.ldq;
  p.ld_pages = a.ld_pages;
  p.n_pages = a.n_pages;
  p.B = (int)a.B;
  p.T = (int)a.T;
  p.hq = (int)a.hq;
  p.heads = (int)a.heads;
  p.g = (int)(a.hq / a.heads);
  p.page = (int)a.page;
  const int64_t held = a.ld_pages * a.page;
  p.max_len = (int)(a.n_pages == 0 ? 0 : a.max_len < held ? a.max_len : held);
  p.width = (int)((p.max_len + a.page - 1) / a.page);
  p.count = (int)a.count;
  p.sinks = (int)a.sinks;
  p.recent = (int)a.recent;
  p.blocks = (p.g + 15) / 16;
  p.gp = 16;
  while (p.blocks == 1 && p.gp / 2 >= p.g) p.gp /= 2;
  p.tokens = p.blocks > 1 ? 1 : 16 / p.gp;
  p.dpage = make_fastdiv((uint32_t)a.page);
  const int D = (int)a.dim;
  if (p.width > p.count) {                          // (else every page is taken)
    const dim3 grid((unsigned)(a.B * a.heads), (unsigned)((p.width + 63) / 64));
    if (D == 64) hipLaunchKernelGGL(select_score_kernel<64>, grid, dim3(256), 0, stream, p);
    else if (D == 128) hipLaunchKernelGGL(select_score_kernel<128>, grid, dim3(256), 0, stream, p);
    else if (D == 192) hipLaunchKernelGGL(select_score_kernel<192>, grid, dim3(256), 0, stream, p);
    else hipLaunchKernelGGL(select_score_kernel<256>, grid, dim3(256), 0, stream, p);
    if (hipGetLastError() != hipSuccess) return BSFP8_EHIP;
  }
  const dim3 grid((unsigned)(a.B * a.T * a.heads));
  if (p.width <= 256 * PICK_HELD) hipLaunchKernelGGL((select_pick_kernel<256, true>), grid, dim3(256), 0, stream, p);
  else if (p.width <= 1024 * PICK_HELD) hipLaunchKernelGGL((select_pick_kernel<1024, true>), grid, dim3(1024), 0, stream, p);
  else hipLaunchKernelGGL((select_pick_kernel<1024, false>), grid, dim3(1024), 0, stream, p);
  return hip_status(hipGetLastError());
}

}  // namespace bsfp8
