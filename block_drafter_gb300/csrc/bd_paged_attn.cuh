// What both attention kernels of the paged cache share: results, the joining of parts, and the
// exact row.
#pragma once
#include "bd_paged_device.cuh"

#include <type_traits>

namespace bd {

// First unit of block g's share among `ctas` <= 1024 blocks of `units` units (a 64-bit division takes
// some hundred cycles: the usual sizes do without).
__device__ __forceinline__ int64_t share_begin(int64_t units, int ctas, int g) {
  if (units < (1 << 22)) return static_cast<uint32_t>(units) * static_cast<uint32_t>(g) / static_cast<uint32_t>(ctas);
  return units * g / ctas;
}
// Block whose share holds unit u.
__device__ __forceinline__ int share_owner(int64_t units, int ctas, int64_t u) {
  int g = units < (1 << 22) ? static_cast<int>(static_cast<uint32_t>(u) * static_cast<uint32_t>(ctas) / static_cast<uint32_t>(units))
                            : static_cast<int>(u * ctas / units);
  while (share_begin(units, ctas, g + 1) <= u) ++g;
  while (share_begin(units, ctas, g) > u) --g;
  return g;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Whether one of slots [from, to) holds a value that is not finite (KV head at V); one warp.  The slots are hidden from
// the row: a page that is none of the pool holds nothing, and is reported only by rows that see it.
template <typename T, int D>
__device__ __noinline__ bool holds_garbage(const PagedArgs &a, const T *V, const int32_t *table, int from, int to, int lane) {
  constexpr uint32_t kExp = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;  // all ones: infinity or NaN
  bool bad = false;
  for (int j = from + lane; j < to; j += 32) {
    const int page = __ldg(table + j / a.page_size);
    if (static_cast<unsigned>(page) >= static_cast<unsigned>(a.n_pages)) continue;
    const int64_t off = page_offset(a, page, j);
#pragma unroll 4
    for (int c = 0; c < D / 8; ++c) {
      const uint4 w = __ldg(reinterpret_cast<const uint4 *>(V + off) + c);
      const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int x = 0; x < 4; ++x) bad |= (v[x] & kExp) == kExp || (v[x] >> 16 & kExp) == kExp;
    }
  }
  return __any_sync(0xffffffffu, bad);
}

// One row of one query head by one warp, over exactly the slots it sees: each lane forms one
// slot's score, then adds the 32 weighted values of its own D/32 columns.  The tiled kernels
// multiply hidden slots by a zero weight, which an infinity or NaN among the hidden values turns
// into NaN; they send a row whose result is not finite through here (its lse is
// right already: a hidden slot's score is dropped, not multiplied).  Where the slots that its tiles
// can hold beside those that it sees are finite, the result stands: a visible value brought it about, and
// every later row may share it, too many to be done again one by one.
template <typename T, int D>
__device__ __noinline__ void attend_row(const PagedAttnArgs &A, const Request &rq, int b, int i, int head, int lane) {
  const PagedArgs &a = A.p;
  __syncwarp();  // other lanes of the warp have stored this row: their values before these
  const int row = rq.row0 + i, p = rq.n - rq.rows + i;
  const T *q = static_cast<const T *>(a.q) + row * a.q_stride + head * D;
  constexpr int C = D / 32;  // columns of a lane
  const int first = p >= 0 ? window_first(a, p) : 0;
  const int n_sinks = min(a.n_sink, first);
  const int count = p >= 0 ? n_sinks + p + 1 - first : 0;
  const int64_t head_off = static_cast<int64_t>(head / a.group) * a.head_stride;
  const T *K = static_cast<const T *>(a.k) + head_off, *V = static_cast<const T *>(a.v) + head_off;
  const int32_t *table = a.page_table + static_cast<int64_t>(b) * a.table_width;
  // hidden slots of the same tiles: of the window's beginning and of later rows (at most 256 rows and a tile
  // of 128 slots away), and behind the sinks
  if (p >= 0 && !(holds_garbage<T, D>(a, V, table, max(n_sinks, first - 384), first, lane) ||
                 holds_garbage<T, D>(a, V, table, n_sinks, min(first, n_sinks + 128), lane) ||
                 holds_garbage<T, D>(a, V, table, p + 1, min(rq.n, p + 385), lane)))
    return;
  float m = -INFINITY, l = 0.f, o[C];
#pragma unroll
  for (int c = 0; c < C; ++c) o[c] = 0.f;
  for (int t0 = 0; t0 < count; t0 += 32) {
    const int t = t0 + lane;
    int64_t off = -1;
    float s = -INFINITY;
    if (t < count) {
      off = slot_offset(a, table, t < n_sinks ? t : first + t - n_sinks);
      if (off >= 0) {
        s = 0.f;
        const uint4 *kr = reinterpret_cast<const uint4 *>(K + off);
#pragma unroll 4
        for (int c = 0; c < D / 8; ++c) {
          const uint4 w = __ldg(kr + c);
          const float2 x0 = Pair<T>::unpack(w.x), x1 = Pair<T>::unpack(w.y), x2 = Pair<T>::unpack(w.z),
                       x3 = Pair<T>::unpack(w.w);
          const uint4 z = __ldg(reinterpret_cast<const uint4 *>(q) + c);
          const float2 y0 = Pair<T>::unpack(z.x), y1 = Pair<T>::unpack(z.y), y2 = Pair<T>::unpack(z.z),
                       y3 = Pair<T>::unpack(z.w);
          s += x0.x * y0.x + x0.y * y0.y + x1.x * y1.x + x1.y * y1.y + x2.x * y2.x + x2.y * y2.y + x3.x * y3.x +
               x3.y * y3.y;
        }
        s *= a.scale_log2;
      }
    }
    const float mn = fmaxf(m, warp_max(s));
    const float ref = mn == -INFINITY ? 0.f : mn;
    const float w = exp2f(s - ref), scale = exp2f(m - ref);
    m = mn;
    l = l * scale + warp_sum(w);
#pragma unroll
    for (int c = 0; c < C; ++c) o[c] *= scale;
    for (int u = 0; u < 32; ++u) {
      const int64_t ou = __shfl_sync(0xffffffffu, off, u);
      const float wu = __shfl_sync(0xffffffffu, w, u);
      if (ou < 0) continue;
#pragma unroll
      for (int c = 0; c < C; ++c) o[c] += wu * to_f(V[ou + c * 32 + lane]);
    }
  }
  T *out = static_cast<T *>(A.out) + row * A.out_stride + head * D;
#pragma unroll
  for (int c = 0; c < C; ++c) out[c * 32 + lane] = from_f<T>(l == 0.f ? 0.f : o[c] / l);
}

// Writes rows r0.. of an item: output row r = token r / group, head r % group of KV head h.
template <typename T>
__device__ __forceinline__ void store4(const PagedAttnArgs &A, const Request &rq, int h, int r, int d, float4 o, float inv) {
  const int g = A.p.group, i = r / g, head = h * g + r - i * g;
  T *out = static_cast<T *>(A.out) + (rq.row0 + i) * A.out_stride + head * A.p.head_dim + d;
  *reinterpret_cast<uint2 *>(out) = make_uint2(Pair<T>::pack(o.x * inv, o.y * inv), Pair<T>::pack(o.z * inv, o.w * inv));
}
__device__ __forceinline__ void store_lse(const PagedAttnArgs &A, const Request &rq, int h, int r, float m, float l) {
  if (!A.lse) return;
  const int g = A.p.group, i = r / g, head = h * g + r - i * g;
  A.lse[static_cast<int64_t>(rq.row0 + i) * A.p.n_kv_heads * g + head] = l == 0.f ? -INFINITY : kLn2 * (m + log2f(l));
}

// One finished piece of a row (4 columns from d on): sums o against the reference m, row sum l.
// Returns whether it is not finite.
template <typename T>
__device__ __forceinline__ bool finish4(const PagedAttnArgs &A, const Request &rq, int h, int r, int d, float4 o, float m, float l) {
  const float inv = l == 0.f ? 0.f : 1.f / l;
  store4<T>(A, rq, h, r, d, o, inv);
  if (d == 0) store_lse(A, rq, h, r, m, l);
  return !(fabsf((o.x + o.y + o.z + o.w) * inv) <= 3.4e38f);
}
// Does the rows of bad_rows (from row `from` on) again, a warp each; all threads of the block.
template <typename T, int D, int NT>
__device__ __noinline__ void redo_rows(const PagedAttnArgs &A, const Request &rq, int b, int h, int from, int n,
                                       const unsigned &bad_rows) {
  for (int r = threadIdx.x >> 5; r < n; r += NT / 32)
    if (bad_rows >> r & 1)
      attend_row<T, D>(A, rq, b, (from + r) / A.p.group, h * A.p.group + (from + r) % A.p.group, threadIdx.x & 31);
  __syncthreads();
}

constexpr int kJoinParts = 320;  // parts of an item at most: the blocks of a kernel, and one more

// Rows of request rq that have no slot of their own or before them: zeros.  `step` threads, this one
// the tid-th.
template <typename T, int D>
__device__ void empty_rows(const PagedAttnArgs &A, const Request &rq, int rows, int tid, int step) {
  const int64_t per = static_cast<int64_t>(A.p.n_kv_heads) * A.p.group;
  for (int64_t x = tid; x < rows * per * (D / 8); x += step) {
    const int64_t hr = x / (D / 8), i = hr / per, head = hr - i * per;
    T *out = static_cast<T *>(A.out) + (rq.row0 + i) * A.out_stride + head * D + (x - hr * (D / 8)) * 8;
    *reinterpret_cast<uint4 *>(out) = make_uint4(0, 0, 0, 0);
    if (A.lse && x == hr * (D / 8)) A.lse[(rq.row0 + i) * per + head] = -INFINITY;
  }
}

}  // namespace bd
