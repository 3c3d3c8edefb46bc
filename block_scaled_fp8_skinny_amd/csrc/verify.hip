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
//           sequence, left at zero) picks the token. Otherwise the sequence's first workgroup picks.
//   tree    one workgroup per sequence: its waves sample the nodes, one each at a time, then the first
//           walks down.
#include "device.h"

namespace bsfp8 {
namespace {

constexpr int PIECE = 2048;                         // elements a wave holds: 32 per lane
constexpr int TREE_WAVES = 16;
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
  int* counters;                                    // [B], zero between calls
  Pair* pairs;                                      // [rows][pieces]: the target's rows, then the draft's
  double* rest;                                     // [B][pieces]: residual sums of a refused row
  int32_t *out_tokens, *path, *n_accepted;
  int B, T, V, pieces;
};

// The element type's 16-byte vectors, and how many a piece has per lane.
template <typename T> struct Vec;
template <> struct Vec<float> {
  static constexpr int E = 4, N = 8;
  static __device__ __forceinline__ void get(const u32x4_t& r, float (&x)[E]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(r[i]);
  }
};
template <> struct Vec<uint16_t> {
  static constexpr int E = 8, N = 4;
  static __device__ __forceinline__ void get(const u32x4_t& r, float (&x)[E]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(r[i] << 16);
      x[2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
    }
  }
};

constexpr float NEG_INF = -__builtin_inff();

// A wave's view of one row of V elements. Rows start anywhere, so the row is addressed in 16-byte
// words from the word that holds its first element: word w, element i is row element w * E + i - lead,
// and elements outside [0, V) (the neighbouring rows') read as -inf. The descriptor ends with the
// row's last 4-byte word, so nothing past it is read.
template <typename T>
struct Row {
  static constexpr int E = Vec<T>::E, N = Vec<T>::N;
  __amdgpu_buffer_rsrc_t r;
  int lead, V;
  __device__ __forceinline__ Row(const void* base, int64_t row, int V_) : V(V_) {
    const int64_t first = row * V_;
    lead = (int)(first & (E - 1));
    const int64_t bytes = ((int64_t)(lead + V_) * (int64_t)sizeof(T) + 3) & ~(int64_t)3;
    r = __builtin_amdgcn_make_buffer_rsrc((void*)(reinterpret_cast<const T*>(base) + (first - lead)), 0, (int)bytes,
                                          RSRC_WORD3);
  }
  __device__ __forceinline__ void load(int piece, int lane, u32x4_t (&w)[N]) const {
#pragma unroll
    for (int v = 0; v < N; ++v)
      w[v] = __builtin_amdgcn_raw_buffer_load_b128(r, (piece * (PIECE / E) + v * 64 + lane) * 16, 0, 0);
  }
  __device__ __forceinline__ int index(int piece, int lane, int v, int i) const {
    return (piece * (PIECE / E) + v * 64 + lane) * E + i - lead;
  }
  // elements of vector v; outside the row, and NaN: -inf
  __device__ __forceinline__ void get(const u32x4_t& w, int piece, int lane, int v, float (&x)[E]) const {
    Vec<T>::get(w, x);
    const int at = index(piece, lane, v, 0);
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] = (unsigned)(at + i) < (unsigned)V && x[i] == x[i] ? x[i] : NEG_INF;
  }
};

template <typename T>
__device__ __forceinline__ float element(const void* base, int64_t at) {
  if constexpr (sizeof(T) == 4) return reinterpret_cast<const float*>(base)[at];
  else return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(base)[at] << 16);
}

// exp((x - M) * it) for x <= M; 1 where x is the maximum itself (also for an infinite one).
__device__ __forceinline__ double weight(float x, float M, double it) {
  return x == M ? 1.0 : exp(((double)x - (double)M) * it);
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o);
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}
__device__ __forceinline__ double wave_scan(double v, int lane) {       // inclusive
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const double w = __shfl_up(v, o);
    if (lane >= o) v += w;
  }
  return v;
}

// 1 / t, or 0 for a greedy row (t = 0, negative or NaN).
__device__ __forceinline__ double inv_temperature(float t) { return t > 0.f ? 1.0 / (double)t : 0.0; }

// The pairs of every piece of every row (blockIdx.x; rows of sequence b: the target's b * T + i, then the
// draft's B * T + b * (T - 1) + i).
template <typename T>
__global__ void __launch_bounds__(256) verify_pairs_kernel(VerifyParams p) {
  const int lane = threadIdx.x & 63;
  const int piece = blockIdx.y * 4 + (threadIdx.x >> 6);
  if (piece >= p.pieces) return;
  const int row = blockIdx.x, targets = p.B * p.T;
  const bool is_draft = row >= targets;
  const int local = is_draft ? row - targets : row;
  const int b = is_draft ? local / (p.T - 1) : local / p.T;
  const Row<T> r(is_draft ? p.draft : p.logits, local, p.V);
  u32x4_t w[Row<T>::N];
  r.load(piece, lane, w);
  const double it = inv_temperature(p.temperature[b]);
  float m = NEG_INF;
#pragma unroll
  for (int v = 0; v < Row<T>::N; ++v) {
    float x[Row<T>::E];
    r.get(w[v], piece, lane, v, x);
#pragma unroll
    for (int i = 0; i < Row<T>::E; ++i) m = fmaxf(m, x[i]);
  }
  m = wave_max(m);
  double s = 0;
  if (it > 0 && m > NEG_INF) {
#pragma unroll
    for (int v = 0; v < Row<T>::N; ++v) {
      float x[Row<T>::E];
      r.get(w[v], piece, lane, v, x);
#pragma unroll
      for (int i = 0; i < Row<T>::E; ++i) s += weight(x[i], m, it);
    }
    s = wave_sum(s);
  }
  if (lane == 0) p.pairs[(int64_t)row * p.pieces + piece] = Pair{s, m, 0.f};
}

// Maximum and sum of a row from its pairs (whole wave).
struct Total {
  float M;
  double S;
};
__device__ __forceinline__ Total row_total(const Pair* pr, int pieces, int lane, double it) {
  float M = NEG_INF;
  for (int i = lane; i < pieces; i += 64) M = fmaxf(M, pr[i].m);
  M = wave_max(M);
  double S = 0;
  if (it > 0 && M > NEG_INF)
    for (int i = lane; i < pieces; i += 64) S += pr[i].m > NEG_INF ? pr[i].s * weight(pr[i].m, M, it) : 0.0;
  return Total{M, wave_sum(S)};
}

// The first piece whose running sum passes `target` (whole wave; f(i) = the sum of piece i), the
// last piece with a positive sum if rounding leaves none; `before` = the running sum before it.
template <typename F>
__device__ __forceinline__ int pick_piece(int pieces, int lane, double target, double& before, F f) {
  double base = 0, last_before = 0;
  int last = 0;
  for (int i0 = 0; i0 < pieces; i0 += 64) {
    const double v = i0 + lane < pieces ? f(i0 + lane) : 0.0;
    const double run = wave_scan(v, lane);
    const uint64_t past = __ballot(v > 0 && base + run > target);
    const uint64_t some = __ballot(v > 0);
    const int at = past ? __builtin_ctzll(past) : some ? 63 - __builtin_clzll(some) : -1;
    if (at >= 0) {
      last = i0 + at;
      last_before = base + __shfl(run, at) - __shfl(v, at);
    }
    if (past) break;
    base += __shfl(run, 63);
  }
  before = last_before;
  return last;
}

// The first element of a piece whose running sum passes `target`, the last one of positive weight if
// rounding leaves none (whole wave; w = the lane's weights in element order per vector).
template <int E, int N>
__device__ __forceinline__ int pick_element(const double (&w)[N][E], int lane, double target) {
  double base = 0;
  int found = -1, last = -1;
#pragma unroll
  for (int v = 0; v < N; ++v) {
    double own = 0;
#pragma unroll
    for (int i = 0; i < E; ++i) own += w[v][i];
    const double run = wave_scan(own, lane), start = base + (run - own);
    double c = start;
    int hit = -1, pos = -1;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      c += w[v][i];
      if (w[v][i] > 0) {
        pos = i;
        if (hit < 0 && c > target) hit = i;
      }
    }
    const uint64_t hits = __ballot(hit >= 0), some = __ballot(pos >= 0);
    if (found < 0 && hits) {
      const int l = __builtin_ctzll(hits);
      found = (v * 64 + l) * E + __shfl(hit, l);
    }
    if (some) {
      const int l = 63 - __builtin_clzll(some);
      last = (v * 64 + l) * E + __shfl(pos, l);
    }
    base += __shfl(run, 63);
  }
  return found >= 0 ? found : last;
}

// The lowest index of the row's largest logit (whole wave).
template <typename T>
__device__ __forceinline__ int pick_greedy(const Row<T>& r, const Pair* pr, int pieces, int lane, float M) {
  if (!(M > NEG_INF)) return 0;
  int piece = 0;
  for (int i0 = 0; i0 < pieces; i0 += 64) {
    const uint64_t is = __ballot(i0 + lane < pieces && pr[i0 + lane < pieces ? i0 + lane : 0].m == M);
    if (is) {
      piece = i0 + __builtin_ctzll(is);
      break;
    }
  }
  u32x4_t w[Row<T>::N];
  r.load(piece, lane, w);
  int best = 0x7fffffff;
#pragma unroll
  for (int v = Row<T>::N - 1; v >= 0; --v) {
    float x[Row<T>::E];
    r.get(w[v], piece, lane, v, x);
#pragma unroll
    for (int i = Row<T>::E - 1; i >= 0; --i)
      if (x[i] == M) best = r.index(piece, lane, v, i);
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) best = min(best, __shfl_xor(best, o));
  return best == 0x7fffffff ? 0 : best;
}

// A token from the row's own distribution (whole wave).
template <typename T>
__device__ __forceinline__ int pick_row(const Row<T>& r, const Pair* pr, int pieces, int lane, const Total& t,
                                        double it, float u) {
  if (!(it > 0)) return pick_greedy(r, pr, pieces, lane, t.M);
  if (!(t.M > NEG_INF)) return 0;
  const double target = (double)u * t.S;
  double before;
  const int piece = pick_piece(pieces, lane, target, before,
                               [&](int i) { return pr[i].m > NEG_INF ? pr[i].s * weight(pr[i].m, t.M, it) : 0.0; });
  u32x4_t raw[Row<T>::N];
  r.load(piece, lane, raw);
  double w[Row<T>::N][Row<T>::E];
#pragma unroll
  for (int v = 0; v < Row<T>::N; ++v) {
    float x[Row<T>::E];
    r.get(raw[v], piece, lane, v, x);
#pragma unroll
    for (int i = 0; i < Row<T>::E; ++i) w[v][i] = weight(x[i], t.M, it);
  }
  const int at = pick_element<Row<T>::E, Row<T>::N>(w, lane, target - before);
  return at < 0 ? 0 : r.index(piece, 0, 0, 0) + at;
}

// max(p - q, 0) of the lane's elements of a piece, in the target row's layout. The draft's row may
// start at another place in its 16-byte words (an odd V): its elements are then read one by one.
template <typename T>
struct Residual {
  static constexpr int E = Vec<T>::E, N = Vec<T>::N;
  Row<T> rp, rq;
  __amdgpu_buffer_rsrc_t q_row;                     // the draft's row from its first element
  Total tp, tq;
  double it;
  __device__ __forceinline__ Residual(const VerifyParams& p, int64_t prow, int64_t qrow, const Total& tp_, const Total& tq_,
                                      double it_)
      : rp(p.logits, prow, p.V), rq(p.draft, qrow, p.V), tp(tp_), tq(tq_), it(it_) {
    q_row = __builtin_amdgcn_make_buffer_rsrc((void*)(reinterpret_cast<const T*>(p.draft) + qrow * p.V), 0,
                                              (int)(p.V * (int)sizeof(T)), RSRC_WORD3);
  }
  __device__ __forceinline__ void get(int piece, int lane, double (&w)[N][E]) const {
    u32x4_t a[N], b[N];
    const bool same = rp.lead == rq.lead;           // uniform
    rp.load(piece, lane, a);
    if (same) rq.load(piece, lane, b);
    const double ip = 1.0 / tp.S, iq = tq.S > 0 ? 1.0 / tq.S : 0.0;
#pragma unroll
    for (int v = 0; v < N; ++v) {
      float x[E], y[E];
      rp.get(a[v], piece, lane, v, x);
      if (same) {
        rq.get(b[v], piece, lane, v, y);
      } else {
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const int j = rp.index(piece, lane, v, i);
          if constexpr (sizeof(T) == 4)
            y[i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(q_row, j * 4, 0, 0));
          else
            y[i] = __uint_as_float((uint32_t)__builtin_amdgcn_raw_buffer_load_b16(q_row, j * 2, 0, 0) << 16);
          if ((unsigned)j >= (unsigned)rp.V || y[i] != y[i]) y[i] = NEG_INF;
        }
      }
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const double pw = x[i] > NEG_INF ? weight(x[i], tp.M, it) * ip : 0.0;
        const double qw = y[i] > NEG_INF ? weight(y[i], tq.M, it) * iq : 0.0;
        w[v][i] = fmax(pw - qw, 0.0);
      }
    }
  }
};

template <typename T>
__global__ void __launch_bounds__(256) verify_chain_kernel(VerifyParams p) {
  __shared__ Total totals[2 * MAX_T];
  __shared__ int shared_n, shared_last;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, b = blockIdx.x, D = p.T - 1;
  const double it = inv_temperature(p.temperature[b]);
  const bool greedy = !(it > 0);
  const Pair* target_pairs = p.pairs + (int64_t)b * p.T * p.pieces;
  const Pair* draft_pairs = p.pairs + ((int64_t)p.B * p.T + (int64_t)b * D) * p.pieces;
  for (int i = wave; i < p.T + D; i += 4) {
    const Pair* pr = i < p.T ? target_pairs + (int64_t)i * p.pieces : draft_pairs + (int64_t)(i - p.T) * p.pieces;
    const Total t = row_total(pr, p.pieces, lane, it);
    if (lane == 0) totals[i] = t;
  }
  __syncthreads();
  if (wave == 0) {                                  // draft i on lane i
    bool ok = false;
    if (lane < D) {
      const int x = p.tokens[(int64_t)b * D + lane];
      if (x >= 0 && x < p.V) {
        const Total tp = totals[lane], tq = totals[p.T + lane];
        const float lp = element<T>(p.logits, ((int64_t)b * p.T + lane) * p.V + x);
        const float lq = element<T>(p.draft, ((int64_t)b * D + lane) * p.V + x);
        if (greedy) {
          ok = lp == tp.M && tp.M > NEG_INF;        // a candidate: the lowest index is tested below
        } else {
          const double pp = lp > NEG_INF ? weight(lp, tp.M, it) / tp.S : 0.0;
          const double pq = lq > NEG_INF && tq.S > 0 ? weight(lq, tq.M, it) / tq.S : 0.0;
          ok = (double)p.u[(int64_t)b * D + lane] * pq < pp;
        }
      }
    }
    uint64_t oks = __ballot(ok);
    int n = 0;
    for (; n < D && (oks >> n & 1); ++n) {
      if (greedy) {
        const Row<T> r(p.logits, (int64_t)b * p.T + n, p.V);
        if (pick_greedy(r, target_pairs + (int64_t)n * p.pieces, p.pieces, lane, totals[n].M) !=
            p.tokens[(int64_t)b * D + n])
          break;
      }
    }
    if (lane == 0) shared_n = n;
  }
  __syncthreads();
  const int n = shared_n;
  const int64_t prow = (int64_t)b * p.T + n;
  const Total tp = totals[n];
  const bool refused = n < D && !greedy && tp.M > NEG_INF;
  int next = -1;
  if (refused) {
    const Residual<T> res(p, prow, (int64_t)b * D + n, tp, totals[p.T + n], it);
    double* rest = p.rest + (int64_t)b * p.pieces;
    const int piece = blockIdx.y * 4 + wave;
    if (piece < p.pieces) {
      double w[Vec<T>::N][Vec<T>::E], s = 0;
      res.get(piece, lane, w);
#pragma unroll
      for (int v = 0; v < Vec<T>::N; ++v)
#pragma unroll
        for (int i = 0; i < Vec<T>::E; ++i) s += w[v][i];
      s = wave_sum(s);
      if (lane == 0) __hip_atomic_store(rest + piece, s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      __threadfence();
      const int old = atomicAdd(p.counters + b, 1);
      shared_last = old == (int)gridDim.y - 1;
      if (shared_last) __hip_atomic_store(p.counters + b, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      __threadfence();
    }
    __syncthreads();
    if (!shared_last || wave != 0) return;
    auto sum_of = [&](int i) { return __hip_atomic_load(rest + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); };
    double total = 0;
    for (int i = lane; i < p.pieces; i += 64) total += sum_of(i);
    total = wave_sum(total);
    if (total > 0) {
      const double target = (double)p.u_sample[b] * total;
      double before;
      const int at = pick_piece(p.pieces, lane, target, before, sum_of);
      double w[Vec<T>::N][Vec<T>::E];
      res.get(at, lane, w);
      const int e = pick_element<Vec<T>::E, Vec<T>::N>(w, lane, target - before);
      next = e < 0 ? 0 : res.rp.index(at, 0, 0, 0) + e;
    }
  } else if (blockIdx.y != 0 || wave != 0) {
    return;
  }
  if (next < 0)
    next = pick_row(Row<T>(p.logits, prow, p.V), target_pairs + (int64_t)n * p.pieces, p.pieces, lane, tp, it, p.u_sample[b]);
  if (lane < p.T) p.out_tokens[(int64_t)b * p.T + lane] = lane < n ? p.tokens[(int64_t)b * D + lane] : lane == n ? next : -1;
  if (lane == 0) p.n_accepted[b] = n;
}

template <typename T>
__global__ void __launch_bounds__(64 * TREE_WAVES) verify_tree_kernel(VerifyParams p) {
  __shared__ int sampled[MAX_T];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, b = blockIdx.x;
  const double it = inv_temperature(p.temperature[b]);
  for (int i = wave; i < p.T; i += TREE_WAVES) {
    const int64_t row = (int64_t)b * p.T + i;
    const Pair* pr = p.pairs + row * p.pieces;
    const Total t = row_total(pr, p.pieces, lane, it);
    const int x = pick_row(Row<T>(p.logits, row, p.V), pr, p.pieces, lane, t, it, p.u[row]);
    if (lane == 0) sampled[i] = x;
  }
  __syncthreads();
  if (wave != 0) return;
  int parent = -1, token = -1;                      // node `lane`'s
  if (lane > 0 && lane < p.T) {
    parent = p.parents[(int64_t)b * p.T + lane];
    token = p.tokens[(int64_t)b * p.T + lane];
    if (parent >= lane) parent = -1;
  }
  int cur = 0, n = 0, out = -1, step = -1;          // lane n keeps the path's n-th node
  for (;;) {
    const int x = sampled[cur];
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

inline int pieces_of(int64_t V) { return (int)((V + 7 + PIECE - 1) / PIECE); }
inline size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace

size_t verify_ws_bytes(int64_t B, int64_t T, int64_t V) {
  const size_t pieces = (size_t)pieces_of(V);
  return align256((size_t)B * 4) + align256((size_t)B * (2 * T - 1) * pieces * sizeof(Pair)) + (size_t)B * pieces * 8;
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
  const unsigned blocks = (unsigned)((p.pieces + 3) / 4);
  const unsigned rows = (unsigned)(tree ? a.B * a.T : a.B * (2 * a.T - 1));
  if (a.f32)
    hipLaunchKernelGGL(verify_pairs_kernel<float>, dim3(rows, blocks), dim3(256), 0, stream, p);
  else
    hipLaunchKernelGGL(verify_pairs_kernel<uint16_t>, dim3(rows, blocks), dim3(256), 0, stream, p);
  if (hipGetLastError() != hipSuccess) return BSFP8_EHIP;
  if (tree && a.f32)
    hipLaunchKernelGGL(verify_tree_kernel<float>, dim3((unsigned)a.B), dim3(64 * TREE_WAVES), 0, stream, p);
  else if (tree)
    hipLaunchKernelGGL(verify_tree_kernel<uint16_t>, dim3((unsigned)a.B), dim3(64 * TREE_WAVES), 0, stream, p);
  else if (a.f32)
    hipLaunchKernelGGL(verify_chain_kernel<float>, dim3((unsigned)a.B, blocks), dim3(256), 0, stream, p);
  else
    hipLaunchKernelGGL(verify_chain_kernel<uint16_t>, dim3((unsigned)a.B, blocks), dim3(256), 0, stream, p);
  return hip_status(hipGetLastError());
}

}  // namespace bsfp8
