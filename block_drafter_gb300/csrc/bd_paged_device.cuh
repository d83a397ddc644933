// Device helpers of the paged-cache kernels: a request's checked sizes, a slot's place in the
// pool, what a row sees.
#pragma once
#include "bd_device.cuh"
#include "bd_paged.h"

namespace bd {

// Sizes of one request as the device arrays give them, checked against the call's bounds: rows
// outside them take no part, a length outside them counts as zero.  A thread that finds a bad one
// flags the error word.
struct Request {
  int n;       // slots held
  int row0;    // first row
  int rows;    // rows; row i is slot n - rows + i
};

__device__ __forceinline__ int request_len(const PagedArgs &a, int b) {
  const int n = a.seq_len[b];
  if (n < 0 || n > a.max_len || n > static_cast<int64_t>(a.table_width) * a.page_size) {
    atomicOr(&g_error_word, DEVERR_BAD_INDEX);
    return 0;
  }
  return n;
}
__device__ __forceinline__ Request request_of(const PagedArgs &a, int b) {
  Request r;
  r.n = request_len(a, b);
  r.row0 = a.row_start[b];
  const int end = a.row_start[b + 1];
  r.rows = end - r.row0;
  if (r.row0 < 0 || end < r.row0 || end > a.n_rows || r.rows > a.max_rows) {
    atomicOr(&g_error_word, DEVERR_BAD_INDEX);
    r.row0 = r.rows = 0;
  }
  return r;
}

// Element offset of slot j (KV head 0) in the pools where it lies in `page`, or -1 (flagged) where
// that is no page of the pool.
__device__ __forceinline__ int64_t page_offset(const PagedArgs &a, int page, int j) {
  if (static_cast<unsigned>(page) >= static_cast<unsigned>(a.n_pages)) {
    atomicOr(&g_error_word, DEVERR_BAD_INDEX);
    return -1;
  }
  return page * a.page_stride + (j % a.page_size) * a.slot_stride;
}
// The same by the request's row of the page table.  0 <= j < the request's checked length.
__device__ __forceinline__ int64_t slot_offset(const PagedArgs &a, const int32_t *table_row, int j) {
  return page_offset(a, __ldg(table_row + j / a.page_size), j);
}

// Whether some of slots j .. j + n - 1 are seen by rows whose first slot beside the sinks is f_low and whose last is
// p_high.  The page of slots that no row sees is not looked at: behind a window it may be given back, its
// entry no page of the pool.
__device__ __forceinline__ bool any_seen(const PagedArgs &a, int j, int n, int f_low, int p_high) {
  return j <= p_high && (j + n > f_low || j < a.n_sink);
}

// First slot beside the sinks that the row at slot p sees (p >= 0).
__host__ __device__ __forceinline__ int window_first(const PagedArgs &a, int p) {
  return a.window > 0 && p >= a.window ? p - a.window + 1 : 0;
}

// 2^x (ex2.approx.ftz: relative error about 2^-22; 2^-inf = 0)
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <typename T> struct Pair;  // two 16-bit values in a word <-> fp32
template <> struct Pair<__nv_bfloat16> {
  static __device__ __forceinline__ float2 unpack(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&h);
  }
};
template <> struct Pair<__half> {
  static __device__ __forceinline__ float2 unpack(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&h);
  }
};

constexpr float kLn2 = 0.693147180559945309f;

}  // namespace bd
