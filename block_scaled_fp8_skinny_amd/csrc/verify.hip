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
#include "logits.h"

namespace bsfp8 {
namespace {

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
  const Row<T> r(is_draft ? p.draft : p.logits, (int64_t)local * p.V, p.V);
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
      : rp(p.logits, prow * p.V, p.V), rq(p.draft, qrow * p.V, p.V), fp(tp.M, it, powers), fq(tq.M, it, powers) {
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
        const Row<T> r(p.logits, ((int64_t)b * p.T + n) * p.V, p.V);
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
    next = pick_row(Row<T>(p.logits, prow * p.V, p.V), target_pairs + (int64_t)n * p.pieces, p.pieces, lane, tp, it, p.u_sample[b],
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
    const int x = pick_row(Row<T>(p.logits, row * p.V, p.V), pr, p.pieces, lane, t, it, u, powers);
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
