// Page tables and slot maps of a step (bd_paged_plan).
//
// Every place is a function of four prefix sums over the requests: of new rows, of pages given back, of
// pages promised, and whether a request's promise is within the stack.  Page x that a request takes is the
// stack's entry (top - 1 - its place among the promises); where that entry is one that was given
// back in this call, the same sums say whose it was, so that no thread waits for another's store.  So every
// block works the sums out for itself (1024 requests are two loads and two scans) and takes an equal part of the
// rows and of the moved pages, which it finds by binary search in shared memory; of its threads some write the requests'
// places and move pages, the others the rows.  Nothing that the rows' and pages' threads read is written in the launch.
// Bound by its latency: the launch, one round trip for the counts, the scans, one more for tables and stack (8 requests of 16
// rows 3.9 us; 512 requests, 66 000 rows, counts in place: 6.0 us, on one block alone 18.6 us).
#include "bd_checks.h"
#include "bd_paged_device.cuh"

namespace bd {

BD_DEFINE_ERROR_TAKER(take_error_word_paged_plan)

namespace {

constexpr int kPlanThreads = 512;
constexpr int kPlanEach = BD_PAGED_MAX_REQUESTS / kPlanThreads;  // requests of a thread
constexpr int kPlanMovers = 128;  // threads that write the requests' places and move pages, beside the others' rows

struct PlanArgs {
  bd_paged_pages p;
  const int32_t *len, *n_new;
  int give_back, n_rows;
  int32_t *seq_len, *row_start, *row_request, *row_pos;
  int64_t *slot_map;
  int32_t *n_short;
  int counts, rest;  // whether held_out and free_count_out are written, and all else
};

// Sum of the threads before this one, and of all (two uses need a barrier between them).
template <int N> __device__ __forceinline__ void scan(long long (&x)[N], long long (&all)[N], long long (*warp_sum_s)[N]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long mine[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    mine[i] = x[i];
    all[i] = 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x[i], o);
      if (lane >= o) x[i] += y;
    }
    if (lane == 31) warp_sum_s[warp][i] = x[i];
    x[i] -= mine[i];
  }
  __syncthreads();
  for (int w = 0; w < kPlanThreads / 32; ++w)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (w == warp) x[i] += all[i];
      all[i] += warp_sum_s[w][i];
    }
}

// The last request of those with before[b] <= x (before[0] = 0 <= x < before[n]).
__device__ __forceinline__ int owner(const int *before, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (before[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(const __grid_constant__ PlanArgs A) {
  constexpr int N = BD_PAGED_MAX_REQUESTS;
  // before each request: rows (at most n_rows), pages given back, pages promised (at most what the stack has)
  __shared__ int rows_before[N + 1], gives_before[N + 1], takes_before[N + 1];
  __shared__ int keep_s[N], held_s[N], need_s[N];  // slots kept (below 0: the request is short), pages held and needed
  __shared__ long long row_sums[kPlanThreads / 32][1], page_sums[kPlanThreads / 32][2];
  __shared__ int short_s, taken_s;
  const bd_paged_pages &p = A.p;
  const int tid = threadIdx.x, B = p.n_requests, ps = p.page_size;
  if (tid == 0) short_s = taken_s = 0;
  pdl_wait();
  pdl_trigger();
  int free = *p.free_count;
  if (free < 0 || free > p.n_free) {
    atomicOr(&g_error_word, DEVERR_BAD_INDEX);
    free = 0;
  }
  int keep[kPlanEach], fresh[kPlanEach], held[kPlanEach], need[kPlanEach], gives[kPlanEach], takes[kPlanEach];
  bool fine[kPlanEach];
  long long rows[1] = {0}, all_rows[1], pages[2] = {0, 0}, all_pages[2];  // pages: given back, promised
#pragma unroll
  for (int u = 0; u < kPlanEach; ++u) {
    const int b = tid * kPlanEach + u;
    keep[u] = fresh[u] = held[u] = 0;
    if (b < B) {
      keep[u] = A.len[b];
      fresh[u] = A.n_new[b];
      held[u] = p.held[b];
    }
    rows[0] += max(0, fresh[u]);
  }
  scan(rows, all_rows, row_sums);
  long long row = rows[0];
#pragma unroll
  for (int u = 0; u < kPlanEach; ++u) {
    const long long n = static_cast<long long>(keep[u]) + fresh[u];
    row += max(0, fresh[u]);
    fine[u] = keep[u] >= 0 && fresh[u] >= 0 && held[u] >= 0 && held[u] <= p.table_width &&
              n <= static_cast<long long>(p.table_width) * ps && n < (1ll << 31) - ps &&
              keep[u] <= static_cast<long long>(held[u]) * ps && row <= A.n_rows;
    need[u] = fine[u] ? (static_cast<int>(n) + ps - 1) / ps : 0;
    gives[u] = fine[u] && A.give_back ? max(0, held[u] - need[u]) : 0;
    takes[u] = fine[u] ? max(0, need[u] - held[u]) : 0;
    pages[0] += gives[u];
    pages[1] += takes[u];
  }
  scan(pages, all_pages, page_sums);
  // the stack when everything has been given back; what does not fit on it is lost (a stack too small for its pool)
  long long top = free + all_pages[0];
  if (top > p.n_free) {
    atomicOr(&g_error_word, DEVERR_BAD_INDEX);
    top = p.n_free;
  }
#pragma unroll
  for (int u = 0; u < kPlanEach; ++u) {
    const int b = tid * kPlanEach + u;
    const long long row_end = rows[0] + max(0, fresh[u]), gives_end = pages[0] + gives[u], takes_end = pages[1] + takes[u];
    const bool served = fine[u] && (takes[u] == 0 || takes_end <= top);
    if (b < B) {
      rows_before[b] = static_cast<int>(min(rows[0], static_cast<long long>(A.n_rows)));
      gives_before[b] = static_cast<int>(min(pages[0], top - free));
      takes_before[b] = static_cast<int>(min(pages[1], top));
      keep_s[b] = served ? keep[u] : -1;
      held_s[b] = held[u];
      need_s[b] = need[u];
      if (!fine[u]) atomicOr(&g_error_word, DEVERR_BAD_INDEX);
      if (!served) atomicAdd(&short_s, 1);
      else if (takes[u] > 0) atomicMax(&taken_s, static_cast<int>(takes_end));  // the served promises are the first ones
    }
    if (b == B - 1) {
      rows_before[B] = static_cast<int>(min(row_end, static_cast<long long>(A.n_rows)));
      gives_before[B] = static_cast<int>(min(gives_end, top - free));
      takes_before[B] = static_cast<int>(min(takes_end, top));
    }
    rows[0] = row_end;
    pages[0] = gives_end;
    pages[1] = takes_end;
  }
  __syncthreads();
  // page x of the promises, from 0 on: the stack from its top down
  auto page_at = [&](int x) {
    const int i = static_cast<int>(top) - 1 - x;
    if (i < free) return p.free_pages[i];
    const int b = owner(gives_before, B, i - free);
    return p.page_table[static_cast<int64_t>(b) * p.table_width + need_s[b] + i - free - gives_before[b]];
  };
  if (tid < kPlanMovers) {
    const int at = blockIdx.x * kPlanMovers + tid, step = gridDim.x * kPlanMovers;
    for (int b = at; b < B; b += step) {
      const bool served = keep_s[b] >= 0;
      const int fresh_b = rows_before[b + 1] - rows_before[b], h = held_s[b], n = need_s[b];
      if (A.rest) {
        A.seq_len[b] = served ? keep_s[b] + fresh_b : 0;
        A.row_start[b] = rows_before[b];
      }
      if (A.counts) p.held_out[b] = !served ? h : n > h || A.give_back ? n : h;
    }
    if (at == 0) {
      if (A.counts) *p.free_count_out = static_cast<int>(top) - taken_s;
      A.row_start[B] = rows_before[B];
      if (A.n_short) *A.n_short = short_s;
    }
    if (!A.rest) return;
    for (int g = at; g < gives_before[B]; g += step) {
      const int b = owner(gives_before, B, g);
      p.free_pages[free + g] = p.page_table[static_cast<int64_t>(b) * p.table_width + need_s[b] + g - gives_before[b]];
    }
    for (int t = at; t < takes_before[B]; t += step) {
      const int b = owner(takes_before, B, t);
      if (keep_s[b] >= 0) p.page_table[static_cast<int64_t>(b) * p.table_width + held_s[b] + t - takes_before[b]] = page_at(t);
    }
    return;
  }
  if (!A.rest) return;
  const int at = blockIdx.x * (kPlanThreads - kPlanMovers) + tid - kPlanMovers, step = gridDim.x * (kPlanThreads - kPlanMovers);
  for (int r = at; r < A.n_rows; r += step) {
    int b = -1, pos = -1;
    int64_t slot = -1;
    if (r < rows_before[B]) {
      b = owner(rows_before, B, r);
      if (keep_s[b] >= 0) {
        pos = keep_s[b] + r - rows_before[b];
        const int k = pos / static_cast<uint32_t>(ps), h = held_s[b];
        const int page = k < h ? p.page_table[static_cast<int64_t>(b) * p.table_width + k] : page_at(takes_before[b] + k - h);
        slot = static_cast<int64_t>(page) * ps + pos - k * ps;
      }
    }
    if (A.row_request) A.row_request[r] = b;
    A.row_pos[r] = pos;
    A.slot_map[r] = slot;
  }
}

// A thread a row, up to two blocks an SM.  Several blocks do not write what others of them read: held counts and the stack's
// count in place are a second launch's, which works the sums out again (512 requests, 66 000 rows: 2 us of it).
std::string launch_plan(PlanArgs A, cudaStream_t s) {
  constexpr int kRows = kPlanThreads - kPlanMovers;
  int blocks = A.n_rows <= kRows ? 1 : (A.n_rows + kRows - 1) / kRows;
  if (blocks > 2 * num_sms()) blocks = 2 * num_sms();
  const bool in_place = A.p.held_out == A.p.held || A.p.free_count_out == A.p.free_count, twice = blocks > 1 && in_place;
  A.counts = !twice;
  A.rest = 1;
  cudaError_t e = launch_pdl(paged_plan_kernel, dim3(blocks), dim3(kPlanThreads), 0, s, A);
  if (e == cudaSuccess && twice) {
    A.counts = 1;
    A.rest = 0;
    e = launch_pdl(paged_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, A);
  }
  return e == cudaSuccess ? std::string() : std::string("paged plan: ") + cudaGetErrorString(e);
}

}  // namespace
}  // namespace bd

using namespace bd;

extern "C" bd_status bd_paged_plan(const bd_paged_pages *pages, const int32_t *len, const int32_t *n_new, int give_back,
                                   int n_rows, int32_t *seq_len, int32_t *row_start, int32_t *row_request, int32_t *row_pos,
                                   int64_t *slot_map, int32_t *n_short, void *stream) {
  if (!pages) return refuse(BD_ERR_INVALID_ARG, "paged plan: pages is NULL");
  const bd_paged_pages &p = *pages;
  if (p.n_requests < 1 || p.n_requests > BD_PAGED_MAX_REQUESTS)
    return refuse(BD_ERR_INVALID_ARG, "paged plan: n_requests must be in 1..1024");
  if (p.table_width < 1 || p.table_width > (1 << 30) || p.page_size < 1 || p.page_size > (1 << 30) || p.n_free < 1 || p.n_free > (1 << 30))
    return refuse(BD_ERR_INVALID_ARG, "paged plan: table_width, page_size and n_free must be in 1..2^30");
  if (n_rows < 0 || n_rows > (1 << 28)) return refuse(BD_ERR_INVALID_ARG, "paged plan: n_rows must be in 0..2^28");
  const int64_t ints = 4ll * p.n_requests, rows = 4ll * n_rows;
  struct Array {
    const void *p;
    int64_t bytes;
    const char *name;
    int in_out;  // 1: read, 2: written
  } arrays[] = {{len, ints, "len", 1}, {n_new, ints, "n_new", 1}, {p.held, ints, "held", 1}, {p.free_count, 4, "free_count", 1},
                {p.page_table, ints * p.table_width, "page_table", 3}, {p.free_pages, 4ll * p.n_free, "free_pages", 3},
                {p.held_out, ints, "held_out", 2}, {p.free_count_out, 4, "free_count_out", 2}, {seq_len, ints, "seq_len", 2},
                {row_start, ints + 4, "row_start", 2}, {row_pos, rows, "row_pos", 2}, {slot_map, 2 * rows, "slot_map", 2},
                {row_request, row_request ? rows : 0, "row_request", 2}, {n_short, n_short ? 4 : 0, "n_short", 2}};
  for (const Array &x : arrays) {
    if ((!x.p && x.bytes > 0) || misaligned(x.p, x.p == slot_map ? 8 : 4))
      return refuse(BD_ERR_INVALID_ARG, std::string("paged plan: ") + x.name + " must be given, aligned to its entries");
    for (const Array &y : arrays) {
      // held_out may be held, free_count_out free_count
      const bool same = x.p == y.p && ((&x == arrays + 2 && &y == arrays + 6) || (&x == arrays + 3 && &y == arrays + 7));
      if (&x != &y && (y.in_out & 2) && !same && overlap(x.p, x.bytes, y.p, y.bytes))
        return refuse(BD_ERR_INVALID_ARG, std::string("paged plan: ") + x.name + " and " + y.name + " overlap");
    }
  }
  PlanArgs A = {p, len, n_new, give_back != 0, n_rows, seq_len, row_start, row_request, row_pos, slot_map, n_short, 1, 1};
  use_target_kernels();
  return ran(launch_plan(A, static_cast<cudaStream_t>(stream)));
}
