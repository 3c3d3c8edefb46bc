// Page tables and slots of a step's tokens from the requests' lengths, for gfx950 (MI355X).
//
// Request b holds lens[b] tokens and will hold new_lens[b]. With had = ceil(lens / page), want = ceil(new_lens / page), three
// exclusive prefix sums over the requests place everything: of the tokens added, of the pages taken (want - had, if
// positive) and of the pages given back (had - want). The pages given back go on top of the stack of free pages, and the
// pages taken come from its top. Since what is taken may have been given back in the same call, such a page is looked up
// in the giver's row of the table, not in the stack: nothing that a workgroup reads is written by another.
//
// Every workgroup repeats the sums over all requests (8 bytes each, from L2), so that one launch does; then the rows, the
// pages taken and the pages given are shared out, one a thread. Bound by latency (lengths, two barriers, a search of 9 steps in
// LDS, the table): 4.7 us for 256 requests of a token each; 96 requests with 393792 rows take 8.2 us, of which 1.6 are the
// 7.9 MB written. (Four rows a thread, one after another: 9.0 and 13.7 us.)

#include "lanes.h"

namespace bsfp8 {
namespace {

constexpr int TT = 512;                             // threads

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
__device__ __forceinline__ int64_t pages_of(const TablesParams& p, int len) { return (int64_t)fdiv(max(len - 1, 0), p.dpage) + (len > 0); }
__device__ __forceinline__ Request request_of(const TablesParams& p, int o, int n) {
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

// Sums over requests. Pages within the tables are below 2^31 in all: takes in the low half, gives in the high.
struct Sums {
  uint64_t tokens, pages, wants;
  __device__ __forceinline__ void operator+=(const Sums& o) {
    tokens += o.tokens;
    pages += o.pages;
    wants += o.wants;
  }
  __device__ __forceinline__ void add(const Request& r) {
    tokens += (uint64_t)r.added;
    pages += (uint64_t)r.gives << 32 | (uint32_t)r.takes;
    wants += (uint64_t)r.wants;
  }
  __device__ __forceinline__ int takes() const { return (int)(uint32_t)pages; }
  __device__ __forceinline__ int gives() const { return (int)(pages >> 32); }
};
__device__ __forceinline__ int at_most(uint64_t n) { return (int)min(n, (uint64_t)INT32_MAX); }

__global__ void __launch_bounds__(TT) step_tables_kernel(TablesParams p) {
  // sums before the first request of thread i (tokens cut at 2^31 - 1, past every row); [TT] = all
  __shared__ int tokens[TT + 1], takes[TT + 1], gives[TT + 1];
  __shared__ int2 lens[TT];                         // a thread's request, where it has one
  __shared__ Sums waves[TT / 64];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int b0 = (int)min((int64_t)t * p.chunk, (int64_t)p.B), b1 = (int)min((int64_t)b0 + p.chunk, (int64_t)p.B);
  auto load = [&](int b) { return make_int2(max(p.lens[b], 0), max(p.new_lens[b], 0)); };
  auto request = [&](int b) {
    const int2 l = p.chunk == 1 ? lens[b] : load(b);
    return request_of(p, l.x, l.y);
  };
  const int n_free = max(0, min(p.n_free[0], (int)p.capacity));
  Sums own{0, 0, 0};
  for (int b = b0; b < b1; ++b) {
    const int2 l = load(b);
    lens[t] = l;
    own.add(request_of(p, l.x, l.y));
  }
  Sums run{wave_scan(own.tokens), wave_scan(own.pages), wave_scan(own.wants)};
  if (lane == 63) waves[wave] = run;
  __syncthreads();
  Sums base{0, 0, 0}, all{0, 0, 0};
#pragma unroll
  for (int w = 0; w < TT / 64; ++w) {
    if (w < wave) base += waves[w];
    all += waves[w];
  }
  run += base;
  tokens[t + 1] = at_most(run.tokens);
  takes[t + 1] = run.takes();
  gives[t + 1] = run.gives();
  if (t == 0) tokens[0] = takes[0] = gives[0] = 0;
  __syncthreads();
  const int n_tokens = at_most(all.tokens), n_takes = all.takes(), n_gives = all.gives();
  const int64_t stack = (int64_t)n_free + n_gives, granted = min((int64_t)n_takes, stack);

  if (blockIdx.x == 0) {
    uint64_t at = run.tokens - own.tokens;
    int before = takes[t];
    for (int b = b0; b < b1; ++b) {
      const Request r = request(b);
      p.starts[b] = at_most(at);
      const int64_t got = max((int64_t)0, min((int64_t)r.takes, granted - before));
      p.held[b] = (int32_t)(r.added > 0 ? min(r.new_len, (r.had + got) * p.page) : r.new_len);
      at += (uint64_t)r.added;
      before += r.takes;
    }
    if (t == 0) {
      p.starts[p.B] = n_tokens;
      p.counts[0] = n_tokens;
      p.counts[1] = (int32_t)granted;
      p.counts[2] = n_gives;
      p.counts[3] = at_most(all.wants - (uint64_t)granted);
      if (p.n_free_out) *p.n_free_out = (int32_t)min(stack - granted, p.capacity);
    }
  }

  // The request that holds item i of a sum (i < the sum's total), with what precedes it.
  enum Kind { TOKENS, TAKES, GIVES };
  auto find = [&](Kind kind, int i, int64_t& before) {
    const int* sum = kind == TOKENS ? tokens : kind == TAKES ? takes : gives;
    int lo = 0, hi = TT - 1;                        // the thread whose requests hold it
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (sum[mid + 1] > i) hi = mid;
      else lo = mid + 1;
    }
    int b = lo * p.chunk;
    before = sum[lo];
    if (p.chunk == 1) return b;
    for (;; ++b) {
      const Request r = request(b);
      const int64_t n = kind == TOKENS ? r.added : kind == TAKES ? r.takes : r.gives;
      if (i < before + n) return b;
      before += n;
    }
  };
  // page i of those given back
  auto given_page = [&](int i) -> int {
    int64_t before;
    const int b = find(GIVES, i, before);
    const Request r = request(b);
    return p.pages[(int64_t)b * p.ld_pages + r.had - r.gives + (i - before)];
  };
  // page i of those taken (0 first, from the stack's top); -1 where there is none left
  auto taken_page = [&](int i) -> int {
    const int64_t at = stack - 1 - i;
    return at < 0 ? -1 : at < n_free ? p.free_pages[at] : given_page((int)(at - n_free));
  };
  const int64_t first = (int64_t)blockIdx.x * TT + t, all_threads = (int64_t)gridDim.x * TT;

  // pages given back, onto the stack, and pages taken, into the table
  for (int64_t k = first; k < (int64_t)n_gives + n_takes; k += all_threads) {
    if (k < n_gives) {
      if (n_free + k < p.capacity) p.free_pages[n_free + k] = given_page((int)k);
    } else {
      const int i = (int)(k - n_gives);
      int64_t before;
      const int b = find(TAKES, i, before);
      p.pages[(int64_t)b * p.ld_pages + request(b).had + (i - before)] = taken_page(i);
    }
  }
  for (int64_t r = first; r < p.R; r += all_threads) {
    int64_t slot = -1, pos = 0, before = 0;
    int b = 0;
    bool live;
    if (p.per_seq) {
      b = fdiv((int)r, p.dseq);
      before = (int64_t)b * p.per_seq;
      live = b < p.B && r - before < request(b).added;
    } else {
      live = r < n_tokens;
      if (live) b = find(TOKENS, (int)r, before);
    }
    if (live) {
      const Request q = request(b);
      pos = q.old_len + (r - before);
      const int j = fdiv((int)pos, p.dpage);
      int entry = -1;
      if (j < q.had) {
        entry = p.pages[(int64_t)b * p.ld_pages + j];
      } else if (j < q.had + q.takes) {
        const int c = b / p.chunk;
        int i = takes[c] + (j - q.had);             // among the pages taken
        for (int o = c * p.chunk; o < b; ++o) i += request(o).takes;
        entry = taken_page(i);
      }
      if (entry >= 0) slot = (int64_t)entry * p.page + (pos - (int64_t)j * p.page);
    }
    p.slots[r] = slot;
    p.positions[r] = pos;
    p.seqs[r] = live ? b : -1;
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
  const int64_t want = (a.R + TT - 1) / TT;
  const int64_t most = p.chunk > 1 ? 256 : 1024;     // (each repeats the sums)
  const unsigned grid = (unsigned)(want < 1 ? 1 : want > most ? most : want);
  hipLaunchKernelGGL(step_tables_kernel, dim3(grid), dim3(TT), 0, stream, p);
  if (hipGetLastError() != hipSuccess) return BSFP8_EHIP;
  if (!a.n_free_out) hipLaunchKernelGGL(n_free_kernel, dim3(1), dim3(1), 0, stream, a.counts, a.n_free, a.capacity);
  return hip_status(hipGetLastError());
}

}  // namespace bsfp8
