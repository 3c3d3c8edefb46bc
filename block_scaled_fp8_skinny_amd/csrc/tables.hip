// Page tables and slots of a step's tokens from the requests' lengths, for gfx950 (MI355X).
//
// Request b holds lens[b] tokens and will hold new_lens[b]. With had = ceil(lens / page), want = ceil(new_lens / page), three
// exclusive prefix sums over the requests place everything: of the tokens added, of the pages taken (want - had, if
// positive) and of the pages given back (had - want). The pages given back go on top of the stack of free pages, and the
// pages taken come from its top. Since what is taken may have been given back in the same call, such a page is looked up
// in the giver's row of the table, not in the stack: nothing that a workgroup reads is written by another.
//
// Every workgroup repeats the sums over all requests (8 bytes each, from L2), so that one launch does; then the rows, the
// pages taken and the pages given are shared out. Bound by latency (loads, two barriers, a search of log2(requests) steps
// in LDS) for a decode step, by the 20 bytes written for each row otherwise.

#include "device.h"

namespace bsfp8 {
namespace {

constexpr int TT = 512;                             // threads
constexpr int ROWS = 4;                             // neighbouring rows of a thread

struct TablesParams {
  const int32_t *lens, *new_lens;
  int32_t *pages, *free_pages;
  const int32_t* n_free;
  int32_t* n_free_out;                              // null: left to n_free_kernel
  int64_t *slots, *positions;
  int32_t *seqs, *starts, *held, *counts;
  int64_t ld_pages, capacity, R;
  int B, width, page, per_seq, chunk;               // chunk: requests of a thread
  FastDiv dpage, dseq;
};

struct Request {
  int64_t old_len, added, new_len;
  int had, takes, gives;                            // pages; takes and gives within the table's width
  int64_t wants;                                    // pages that it lacks, those past the table's width too
};
__device__ __forceinline__ int64_t pages_of(const TablesParams& p, int len) { return ((int64_t)fdiv(max(len - 1, 0), p.dpage)) + (len > 0); }
__device__ __forceinline__ Request request(const TablesParams& p, int b) {
  const int o = max(p.lens[b], 0), n = max(p.new_lens[b], 0);
  Request r;
  r.old_len = o;
  r.new_len = n;
  r.added = max(n - o, 0);
  const int64_t had = pages_of(p, o), want = pages_of(p, n);
  r.had = (int)min(had, (int64_t)p.width);
  const int to = (int)min(want, (int64_t)p.width);
  r.takes = max(to - r.had, 0);
  r.gives = max(r.had - to, 0);
  r.wants = max(want - had, (int64_t)0);
  return r;
}

struct Sums {
  int64_t tokens, takes, gives, wants;
  __device__ __forceinline__ void operator+=(const Sums& o) {
    tokens += o.tokens;
    takes += o.takes;
    gives += o.gives;
    wants += o.wants;
  }
  __device__ __forceinline__ void add(const Request& r) {
    tokens += r.added;
    takes += r.takes;
    gives += r.gives;
    wants += r.wants;
  }
};
__device__ __forceinline__ Sums from_up(const Sums& s, int o) {
  return Sums{__shfl_up(s.tokens, o), __shfl_up(s.takes, o), __shfl_up(s.gives, o), __shfl_up(s.wants, o)};
}

__global__ void __launch_bounds__(TT) step_tables_kernel(TablesParams p) {
  // before[i] = the sums before the first request of thread i; [TT] = all
  __shared__ int64_t tokens[TT + 1], takes[TT + 1], gives[TT + 1], wants[TT + 1];
  __shared__ Sums waves[TT / 64];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int64_t n_free = max((int64_t)0, min((int64_t)p.n_free[0], p.capacity));
  const int b0 = min((int64_t)t * p.chunk, (int64_t)p.B), b1 = min((int64_t)b0 + p.chunk, (int64_t)p.B);
  Sums own{0, 0, 0, 0};
  for (int b = b0; b < b1; ++b) own.add(request(p, b));
  Sums run = own;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const Sums up = from_up(run, o);
    if (lane >= o) run += up;
  }
  if (lane == 63) waves[wave] = run;
  __syncthreads();
  Sums base{0, 0, 0, 0}, all{0, 0, 0, 0};
  for (int w = 0; w < TT / 64; ++w) {
    if (w < wave) base += waves[w];
    all += waves[w];
  }
  run += base;
  tokens[t + 1] = run.tokens;
  takes[t + 1] = run.takes;
  gives[t + 1] = run.gives;
  wants[t + 1] = run.wants;
  if (t == 0) tokens[0] = takes[0] = gives[0] = wants[0] = 0;
  __syncthreads();
  const int64_t stack = n_free + all.gives, granted = min(all.takes, stack);

  if (blockIdx.x == 0) {
    Sums at{tokens[t], takes[t], gives[t], wants[t]};
    for (int b = b0; b < b1; ++b) {
      const Request r = request(p, b);
      p.starts[b] = (int32_t)min(at.tokens, (int64_t)INT32_MAX);
      const int64_t got = max((int64_t)0, min((int64_t)r.takes, granted - at.takes));
      p.held[b] = (int32_t)(r.added > 0 ? min(r.new_len, (r.had + got) * p.page) : r.new_len);
      at.add(r);
    }
    if (t == 0) {
      p.starts[p.B] = (int32_t)min(all.tokens, (int64_t)INT32_MAX);
      p.counts[0] = (int32_t)min(all.tokens, (int64_t)INT32_MAX);
      p.counts[1] = (int32_t)granted;
      p.counts[2] = (int32_t)all.gives;
      p.counts[3] = (int32_t)min(all.wants - granted, (int64_t)INT32_MAX);
      if (p.n_free_out) *p.n_free_out = (int32_t)min(stack - granted, p.capacity);
    }
  }

  // The request that holds item i of a sum (i < the sum's total), with what precedes it.
  auto find = [&](const int64_t* sum, int64_t i, auto of, int64_t& before) {
    int lo = 0, hi = TT - 1;                        // the thread whose requests hold it
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (sum[mid + 1] > i) hi = mid;
      else lo = mid + 1;
    }
    int b = lo * p.chunk;
    before = sum[lo];
    for (;; ++b) {
      const int64_t n = of(request(p, b));
      if (i < before + n) return b;
      before += n;
    }
  };
  // page i of those taken (0 first, from the stack's top); -1 where there is none left
  auto taken_page = [&](int64_t i) -> int {
    const int64_t at = stack - 1 - i;
    if (at < 0) return -1;
    if (at < n_free) return p.free_pages[at];
    int64_t before;
    const int b = find(gives, at - n_free, [](const Request& r) { return r.gives; }, before);
    const Request r = request(p, b);
    return p.pages[(int64_t)b * p.ld_pages + r.had - r.gives + (at - n_free - before)];
  };
  const int64_t first = (int64_t)blockIdx.x * TT + t, all_threads = (int64_t)gridDim.x * TT;

  // pages given back, onto the stack
  for (int64_t i = first; i < all.gives; i += all_threads) {
    if (n_free + i >= p.capacity) break;
    int64_t before;
    const int b = find(gives, i, [](const Request& r) { return r.gives; }, before);
    const Request r = request(p, b);
    p.free_pages[n_free + i] = p.pages[(int64_t)b * p.ld_pages + r.had - r.gives + (i - before)];
  }
  // pages taken, into the table
  for (int64_t i = first; i < all.takes; i += all_threads) {
    int64_t before;
    const int b = find(takes, i, [](const Request& r) { return r.takes; }, before);
    p.pages[(int64_t)b * p.ld_pages + request(p, b).had + (i - before)] = taken_page(i);
  }
  // rows: ROWS neighbours a thread
  for (int64_t r0 = first * ROWS; r0 < p.R; r0 += all_threads * ROWS) {
    int b = -1;
    int64_t before = 0, end = 0;                    // the rows of request b's tokens: [before, end)
    Request q{};
    int64_t take0 = 0;                              // the pages taken before it
    auto enter = [&](int to) {
      b = to;
      q = request(p, b);
      const int c = b / p.chunk;
      take0 = takes[c];
      for (int i = c * p.chunk; i < b; ++i) take0 += request(p, i).takes;
    };
    int64_t slot[ROWS], position[ROWS];
    int seq[ROWS];
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      const int64_t r = r0 + k;
      slot[k] = -1;
      position[k] = 0;
      seq[k] = -1;
      int64_t i = -1;                               // the token's number among its request's new ones
      if (p.per_seq) {
        const int to = fdiv((int)min(r, p.R - 1), p.dseq);
        if (r < p.R && to < p.B) {
          if (b != to) enter(to);
          i = r - (int64_t)to * p.per_seq;
          if (i >= q.added) i = -1;
        }
      } else if (r < p.R && r < all.tokens) {
        if (b < 0 || r >= end) {
          enter(find(tokens, r, [](const Request& x) { return x.added; }, before));
          end = before + q.added;
        }
        i = r - before;
      }
      if (i >= 0) {
        const int64_t pos = q.old_len + i;
        const int j = fdiv((int)pos, p.dpage);
        int entry = -1;
        if (j < q.had) entry = p.pages[(int64_t)b * p.ld_pages + j];
        else if (j < q.had + q.takes) entry = taken_page(take0 + (j - q.had));
        position[k] = pos;
        seq[k] = b;
        if (entry >= 0) slot[k] = (int64_t)entry * p.page + (pos - (int64_t)j * p.page);
      }
    }
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      if (r0 + k >= p.R) break;
      p.slots[r0 + k] = slot[k];
      p.positions[r0 + k] = position[k];
      p.seqs[r0 + k] = seq[k];
    }
  }
}

// The stack's new height in place of the old, when every workgroup has read that.
__global__ void n_free_kernel(const int32_t* counts, int32_t* n_free, int64_t capacity) {
  const int64_t n = max((int64_t)0, min((int64_t)n_free[0], capacity));
  n_free[0] = (int32_t)min(n + counts[2] - counts[1], capacity);
}

}  // namespace

int launch_step_tables(const StepTablesArgs& a, hipStream_t stream) {
  TablesParams p{};
  p.lens = a.lens;
  p.new_lens = a.new_lens;
  p.pages = a.pages;
  p.free_pages = a.free_pages;
  p.n_free = a.n_free;
  p.n_free_out = a.n_free_out;
  p.slots = a.slots;
  p.positions = a.positions;
  p.seqs = a.seqs;
  p.starts = a.starts;
  p.held = a.held;
  p.counts = a.counts;
  p.ld_pages = a.ld_pages;
  p.capacity = a.capacity;
  p.R = a.R;
  p.B = (int)a.B;
  p.width = (int)a.ld_pages;
  p.page = (int)a.page;
  p.per_seq = (int)a.per_seq;
  p.chunk = (int)((a.B + TT - 1) / TT);
  if (p.chunk < 1) p.chunk = 1;
  p.dpage = make_fastdiv((uint32_t)a.page);
  p.dseq = make_fastdiv((uint32_t)(a.per_seq > 0 ? a.per_seq : 1));
  const int64_t want = (a.R + TT * ROWS - 1) / (TT * ROWS);
  const unsigned grid = (unsigned)(want < 1 ? 1 : want > 256 ? 256 : want);
  hipLaunchKernelGGL(step_tables_kernel, dim3(grid), dim3(TT), 0, stream, p);
  if (hipGetLastError() != hipSuccess) return BSFP8_EHIP;
  if (!a.n_free_out) hipLaunchKernelGGL(n_free_kernel, dim3(1), dim3(1), 0, stream, a.counts, a.n_free, a.capacity);
  return hip_status(hipGetLastError());
}

}  // namespace bsfp8
