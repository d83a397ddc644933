// Attention of a call's rows over their requests' paged slots (bd_paged_attention).
//
// One pass over the keys and values with the running maximum m and sum l of a softmax:
//   m' = max(m, max s),  l' = l 2^(m-m') + sum 2^(s-m'),  o' = o 2^(m-m') + sum 2^(s-m') v
// (scores s in log2 units), and parts over different slots joined by the same rule.
//
// attention_few: calls whose rows of one KV head (rows x group) are at most kFewRows = 16 --
// decoding and short blocks.  Bound by the bytes of K and V, so it is built to keep loads in
// flight (16 ragged requests of up to 32 768 slots: 184 us, 6.5 TB/s).  Long calls are a list of units
// of 16 slots, ordered by request, KV head and
// slot; the blocks (two an SM) take equal shares of it whatever the lengths are, so that one long
// request spreads over all SMs and short ones share a block.  Shorter ones, bound by their start and the
// joining launch, give each head to a cluster instead (kClusterSlots).  Inside a block every warp works alone:
// it takes every fourth unit of the block's part, copies the unit's K and V rows page by page into
// its own shared memory with cp.async (kStages units deep, no barrier between warps), and feeds
// mma.sync m16n8k16 from there (the tensor work is small: tcgen05's 128-row tiles would be 7/8
// padding).  The warps join at the end of each (request, KV head); heads that several blocks worked
// on are joined by attention_join from fp32 parts in the workspace.
//
// The weights enter the second product as a 16-bit high part and a 16-bit rest: the rounding to
// 16 bits (2^-8 relative in bf16, as large as the output's own) then disappears from the result.  With at
// most 8 rows the rest takes the idle upper 8 rows of the product and costs nothing.
#include "bd_paged_attn.cuh"

namespace bd {

BD_DEFINE_ERROR_TAKER(take_error_word_paged_attn)

// ------------------------------------------------------------------ few rows: layout
constexpr int kUnit = 16;  // slots of a unit
constexpr int kFewWarps = 4;
constexpr int kFewThreads = 32 * kFewWarps;
template <int D> struct Few {
  static constexpr int kRowBytes = 2 * D;
  static constexpr int kTile = kUnit * kRowBytes;       // K (or V) of a unit
  static constexpr int kStages = D == 128 ? 3 : 5;
  static constexpr int kWarpBytes = kStages * 2 * kTile;  // 24 KB / 20 KB
  static constexpr int kSmem = kFewWarps * kWarpBytes;
};
// Weights are formed against 2^-kHead of the maximum: fp16 keeps small ones above its subnormals.
template <typename T> struct Head { static constexpr float k = 0.f; };
template <> struct Head<__half> { static constexpr float k = 12.f; };

// The slots some row of a request sees, as tiles of kUnit: the sinks' tiles, then those from the
// earliest row's window on.
struct Tiles {
  int sinks, first, count;  // tiles of sinks, first tile behind them, tiles in all
  __device__ int at(int t) const { return t < sinks ? t : first + t - sinks; }
};
__device__ __forceinline__ Tiles tiles_of(const PagedArgs &a, const Request &rq) {
  Tiles t = {0, 0, 0};
  if (rq.rows == 0 || rq.n == 0) return t;
  const int first = window_first(a, max(0, rq.n - rq.rows));
  t.first = first / kUnit;
  t.sinks = min((min(a.n_sink, first) + kUnit - 1) / kUnit, t.first);
  t.count = t.sinks + (rq.n + kUnit - 1) / kUnit - t.first;
  return t;
}

// Blocks that work: a unit for each of their four warps, but as many as there are heads (a block takes
// its heads one after the other, about 2.5 us each).
__device__ __forceinline__ int ctas_used(int64_t units, int heads, int most) {
  const int64_t quarter = (units + kFewWarps - 1) >> 2, c = quarter > heads ? quarter : units < heads ? units : heads;
  return c < 1 ? 1 : static_cast<int>(c < most ? c : most);
}
__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__half>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The part of one (request, KV head) over tiles [t0, t1) by one warp (every kFewWarps-th tile):
// o, m, l of its rows.  HALF: at most 8 rows; rows 8..15 of the second product carry the rest of
// the weights.  Row r of the fragment (lane / 4, and + 8) is token r / group.
template <typename T, int D, bool HALF>
struct FewWarp {
  static constexpr int NK = D / 16, NV = D / 8;
  float o[NV][4];
  float m[2], l[2];

  __device__ __forceinline__ void run(const PagedAttnArgs &A, const Request &rq, const Tiles &tl, int b, int h, int t0, int t1,
                                      uint32_t sm, int warp, int lane) {
    const PagedArgs &a = A.p;
    using F = Few<D>;
    constexpr int CPR = D / 8;       // 16-byte pieces of a row
    constexpr int RPI = 32 / CPR;    // rows one copy instruction of the warp covers
    const int quad = lane >> 2, col = (lane & 3) * 2;
    const int R = rq.rows * a.group;
    // query fragments
    uint32_t q[NK][4];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r = quad + 8 * half;
      const bool ok = (half == 0 || !HALF) && r < R;
      const int i = ok ? r / a.group : 0;
      const T *src = static_cast<const T *>(a.q) + (rq.row0 + i) * a.q_stride + (h * a.group + (ok ? r - i * a.group : 0)) * D + col;
#pragma unroll
      for (int kk = 0; kk < NK; ++kk) {
        q[kk][half] = ok ? *reinterpret_cast<const uint32_t *>(src + kk * 16) : 0u;
        q[kk][half + 2] = ok ? *reinterpret_cast<const uint32_t *>(src + kk * 16 + 8) : 0u;
      }
    }
    // what this thread's rows see: slots <= p, from f on or among the sinks
    int p[2], f[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r = quad + 8 * half;
      p[half] = r < R ? rq.n - rq.rows + r / a.group : -1;
      f[half] = p[half] >= 0 ? window_first(a, p[half]) : 0;
    }
    const int p_low = rq.n - rq.rows, f_high = window_first(a, rq.n - 1);
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;

    const int32_t *table = a.page_table + static_cast<int64_t>(b) * a.table_width;
    const int64_t head_off = static_cast<int64_t>(h) * a.head_stride;
    const T *K = static_cast<const T *>(a.k) + head_off, *V = static_cast<const T *>(a.v) + head_off;
    // page of slot lane % 16 of tile t (the load alone: several go out side by side), then the
    // slot's offset, -1 for a slot no row sees
    const int f_low = window_first(a, max(0, p_low));
    auto page_of = [&](int t) { return __ldg(table + min(tl.at(max(min(t, t1 - 1), 0)) * kUnit + (lane & 15), rq.n - 1) / a.page_size); };
    auto offset = [&](int t, int page) -> int64_t {
      const int j = tl.at(t) * kUnit + (lane & 15);
      if (t >= t1 || j >= rq.n || (j >= a.n_sink && j < f_low)) return -1;
      return page_offset(a, page, j);
    };
    auto issue = [&](int t, int stage, int64_t off) {
      if (t < t1) {
        const uint32_t dst = sm + stage * 2 * F::kTile;
        const int c = lane % CPR;
#pragma unroll
        for (int u = 0; u < kUnit / RPI; ++u) {
          const int r = u * RPI + lane / CPR;
          const int64_t ro = __shfl_sync(0xffffffffu, off, r);
          const uint32_t d = dst + r * F::kRowBytes + ((c ^ (r & 7)) << 4);
          const int64_t so = ro < 0 ? 0 : ro + c * 8;
          cp_async16(d, K + so, ro >= 0);
          cp_async16(d + F::kTile, V + so, ro >= 0);
        }
      }
      cp_async_commit();
    };
    int t = t0 + warp;
    int pages[F::kStages];
#pragma unroll
    for (int s = 0; s < F::kStages; ++s) pages[s] = page_of(t + s * kFewWarps);
#pragma unroll
    for (int s = 0; s < F::kStages - 1; ++s) issue(t + s * kFewWarps, s, offset(t + s * kFewWarps, pages[s]));
    int next = pages[F::kStages - 1];
    int stage = 0;
    for (; t < t1; t += kFewWarps) {
      cp_async_wait<F::kStages - 2>();
      __syncwarp();
      {  // the stage freed by the previous tile takes the tile kStages - 1 ahead
        const int ahead = t + (F::kStages - 1) * kFewWarps;
        issue(ahead, stage == 0 ? F::kStages - 1 : stage - 1, offset(ahead, next));
        next = page_of(ahead + kFewWarps);
      }
      const uint32_t kb = sm + stage * 2 * F::kTile, vb = kb + F::kTile;
      // scores: 16 rows x 16 slots
      float c[2][4] = {};
      {
        const int r = (lane & 7) + ((lane >> 4) << 3), cc = (lane >> 3) & 1;
#pragma unroll
        for (int kk = 0; kk < NK; ++kk) {
          uint32_t kf[4];
          ldmatrix4(kb + r * F::kRowBytes + (((kk * 2 + cc) ^ (r & 7)) << 4), kf);
          mma16816<T>(c[0], q[kk], kf[0], kf[1]);
          mma16816<T>(c[1], q[kk], kf[2], kf[3]);
        }
      }
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) c[n][e] *= a.scale_log2;
      const int j0 = tl.at(t) * kUnit;
      if (!(j0 + kUnit - 1 <= p_low && (j0 >= f_high || j0 + kUnit <= a.n_sink))) {  // some row does not see all of it
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = j0 + n * 8 + col + (e & 1), half = e >> 1;
            if (!(j <= p[half] && (j >= f[half] || j < a.n_sink))) c[n][e] = -INFINITY;
          }
      }
      // running maximum; the sums are rescaled only when a row's moves
      uint32_t hi[4], lo[4];
      float mx[2];
#pragma unroll
      for (int half = 0; half < (HALF ? 1 : 2); ++half) {
        float x = fmaxf(fmaxf(c[0][2 * half], c[0][2 * half + 1]), fmaxf(c[1][2 * half], c[1][2 * half + 1]));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
        mx[half] = fmaxf(m[half], x);
      }
      const bool moved = mx[0] > m[0] || (!HALF && mx[1] > m[1]);
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int half = 0; half < (HALF ? 1 : 2); ++half) {
          const float w = m[half] == mx[half] ? 1.f : exp2_fast(m[half] - mx[half]);
          m[half] = mx[half];
          l[half] *= w;
#pragma unroll
          for (int n = 0; n < NV; ++n) {
            o[n][2 * half] *= w;
            o[n][2 * half + 1] *= w;
            if (HALF) {
              o[n][2] *= w;
              o[n][3] *= w;
            }
          }
        }
      }
#pragma unroll
      for (int half = 0; half < (HALF ? 1 : 2); ++half) {
        const float ref = m[half] == -INFINITY ? 0.f : m[half] - Head<T>::k;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const float x = exp2_fast(c[n][2 * half] - ref), y = exp2_fast(c[n][2 * half + 1] - ref);
          l[half] += x + y;
          const uint32_t hv = Pair<T>::pack(x, y);
          const float2 back = Pair<T>::unpack(hv);
          hi[2 * n + half] = hv;
          lo[2 * n + half] = Pair<T>::pack(x - back.x, y - back.y);
        }
      }
      if (HALF) {
        hi[1] = lo[0];
        hi[3] = lo[2];
      }
      {
        const int r = (lane & 7) + (((lane >> 3) & 1) << 3), cc = lane >> 4;
#pragma unroll
        for (int n = 0; n < NV / 2; ++n) {
          uint32_t vf[4];
          ldmatrix4t(vb + r * F::kRowBytes + (((n * 2 + cc) ^ (r & 7)) << 4), vf);
          mma16816<T>(o[2 * n], hi, vf[0], vf[1]);
          mma16816<T>(o[2 * n + 1], hi, vf[2], vf[3]);
          if (!HALF) {
            mma16816<T>(o[2 * n], lo, vf[0], vf[1]);
            mma16816<T>(o[2 * n + 1], lo, vf[2], vf[3]);
          }
        }
      }
      __syncwarp();
      stage = stage + 1 == F::kStages ? 0 : stage + 1;
    }
    cp_async_wait<0>();
    __syncwarp();
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      l[half] += __shfl_xor_sync(0xffffffffu, l[half], 1);
      l[half] += __shfl_xor_sync(0xffffffffu, l[half], 2);
      if (m[half] != -INFINITY) m[half] -= Head<T>::k;  // the reference the sums are against
    }
  }
};

// start[b] = units of the requests before b; all threads of the block.
// The first NT requests' sizes are kept in `first`.
template <int NT>
__device__ void scan_requests(const PagedArgs &a, int64_t *start, int64_t *warp_sum_s, Request *first) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int64_t base = 0;
  for (int b0 = 0; b0 < a.n_requests; b0 += NT) {
    const int b = b0 + tid;
    int64_t v = 0;
    if (b < a.n_requests) {
      const Request rq = request_of(a, b);
      if (b0 == 0) first[tid] = rq;
      v = static_cast<int64_t>(tiles_of(a, rq).count) * a.n_kv_heads;
    }
    int64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) warp_sum_s[warp] = x;
    __syncthreads();
    for (int w = 0; w < NT / 32; ++w) {
      if (w < warp) x += warp_sum_s[w];
    }
    if (b < a.n_requests) start[b + 1] = base + x;
    for (int w = 0; w < NT / 32; ++w) base += warp_sum_s[w];
    __syncthreads();
  }
  if (tid == 0) start[0] = 0;
  __syncthreads();
}
// Request of unit u (the last one that starts at or before it and has units).
__device__ __forceinline__ int request_at(const int64_t *start, int n, int64_t u) {
  int lo = 0, hi = n;  // start[lo] <= u < start[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= u) lo = mid; else hi = mid;
  }
  return lo;
}

template <typename T, int D, bool HALF>
__global__ void __launch_bounds__(kFewThreads, 2) attention_few(const __grid_constant__ PagedAttnArgs A) {
  extern __shared__ __align__(1024) uint8_t sm_raw[];
  __shared__ int64_t start[BD_PAGED_MAX_REQUESTS + 1];
  __shared__ int64_t warp_sum_s[kFewWarps];
  __shared__ Request first[kFewThreads];
  __shared__ float2 ml[kFewWarps][kFewRows];
  __shared__ __align__(8) float2 block_ml[kFewRows];  // of a cluster's block, its sums in place of its first warp's
  __shared__ unsigned bad_rows;
  const PagedArgs &a = A.p;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_trigger();
  const int g = blockIdx.x;
  int64_t units = 0, u = 0, u1 = 1;
  int ctas = 1;
  if (!A.whole) {
    scan_requests<kFewThreads>(a, start, warp_sum_s, first);
    units = start[a.n_requests];
    ctas = ctas_used(units, a.n_requests * a.n_kv_heads, A.n_ctas);
    for (int b = g; b < a.n_requests; b += gridDim.x)
      if (start[b + 1] == start[b]) {  // rows without a slot
        const Request rq = request_of(a, b);
        empty_rows<T, D>(A, rq, rq.rows, tid, kFewThreads);
      }
    if (tid == 0) A.join[g].np = 0;
    if (units == 0 || g >= ctas) return;
    u = share_begin(units, ctas, g);
    u1 = share_begin(units, ctas, g + 1);
  }
  uint8_t *mine = sm_raw + warp * Few<D>::kWarpBytes;
  do {
    int b, h, t0, t1;
    Request rq;
    Tiles tl;
    if (A.whole) {  // one head, or a cluster's block's part of one
      const int item = g / static_cast<uint32_t>(A.cluster), rank = g - item * A.cluster;
      b = item / a.n_kv_heads;
      h = item - b * a.n_kv_heads;
      rq = request_of(a, b);
      tl = tiles_of(a, rq);
      t0 = tl.count * rank / A.cluster;
      t1 = tl.count * (rank + 1) / A.cluster;
      u = t0;
      u1 = t1;
      if (tl.count == 0) {
        if (h == 0 && rank == 0) empty_rows<T, D>(A, rq, rq.rows, tid, kFewThreads);
        return;
      }
    } else {
      b = request_at(start, a.n_requests, u);
      rq = b < kFewThreads ? first[b] : request_of(a, b);
      tl = tiles_of(a, rq);
      const uint32_t in = static_cast<uint32_t>(u - start[b]);  // below 2^31: checked by the host
      h = in / static_cast<uint32_t>(tl.count);
      t0 = in - h * tl.count;
      t1 = static_cast<int>(u1 - u < tl.count - t0 ? t0 + (u1 - u) : tl.count);
    }
    const int R = rq.rows * a.group;
    {
      FewWarp<T, D, HALF> w;
      w.run(A, rq, tl, b, h, t0, t1, smem_u32(mine), warp, lane);
      float *so = reinterpret_cast<float *>(mine);
      const int quad = lane >> 2, col = (lane & 3) * 2;
#pragma unroll
      for (int n = 0; n < D / 8; ++n) {
        if (HALF) {
          *reinterpret_cast<float2 *>(so + quad * D + n * 8 + col) = make_float2(w.o[n][0] + w.o[n][2], w.o[n][1] + w.o[n][3]);
        } else {
          *reinterpret_cast<float2 *>(so + quad * D + n * 8 + col) = make_float2(w.o[n][0], w.o[n][1]);
          *reinterpret_cast<float2 *>(so + (quad + 8) * D + n * 8 + col) = make_float2(w.o[n][2], w.o[n][3]);
        }
      }
      if ((lane & 3) == 0) {
        ml[warp][quad] = make_float2(w.m[0], w.l[0]);
        ml[warp][quad + 8] = make_float2(w.m[1], w.l[1]);
      }
    }
    const bool whole = t0 == 0 && t1 == tl.count;
    const int64_t slot = (2 * g + (t0 > 0 ? 0 : 1)) * kFewRows;
    if (tid == 0 && !A.whole && t0 > 0 && share_begin(units, ctas, g - 1) <= u - t0)  // the first block to begin inside this head
      A.join[g] = {b, h, 0, R, share_owner(units, ctas, u - t0 + tl.count - 1) - g + 2, rq.row0, rq.n, rq.rows};
    bool bad = false;
    if (tid == 0) bad_rows = 0u;
    __syncthreads();
    for (int c = tid; c < R * (D / 4); c += kFewThreads) {  // join the warps
      const int r = c / (D / 4), d = (c - r * (D / 4)) * 4;
      float2 x[kFewWarps];
      float M = -INFINITY, L = 0.f;
#pragma unroll
      for (int i = 0; i < kFewWarps; ++i) {
        x[i] = ml[i][r];
        if (x[i].y != 0.f) M = fmaxf(M, x[i].x);
      }
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < kFewWarps; ++i) {
        const float4 v = *reinterpret_cast<const float4 *>(sm_raw + i * Few<D>::kWarpBytes + (r * D + d) * 4);
        if (x[i].y != 0.f) {  // a weight of zero counts: it keeps a visible infinity or NaN
          const float w = exp2f(x[i].x - M);
          L += w * x[i].y;
          o.x += w * v.x;
          o.y += w * v.y;
          o.z += w * v.z;
          o.w += w * v.w;
        }
      }
      if (A.cluster > 1) {
        *reinterpret_cast<float4 *>(sm_raw + (r * D + d) * 4) = o;
        if (d == 0) block_ml[r] = make_float2(M, L);
      } else if (whole) {
        if (finish4<T>(A, rq, h, r, d, o, M, L)) {
          atomicOr(&bad_rows, 1u << r);
          bad = true;
        }
      } else {
        *reinterpret_cast<float4 *>(A.part_o + (slot + r) * D + d) = o;
        if (d == 0) A.part_ml[slot + r] = make_float2(M, L);
      }
    }
    if (A.cluster > 1) {  // the blocks' parts: a warp takes every kth row
      __syncwarp();
      cluster_sync();
      const int rank = g % static_cast<uint32_t>(A.cluster), d = lane * 4;
      for (int r = rank + A.cluster * warp; r < R; r += A.cluster * kFewWarps) {
        float4 v[kMostCluster];
        const uint32_t at = smem_u32(sm_raw) + (r * D + d % D) * 4;
#pragma unroll
        for (int i = 0; i < kMostCluster; ++i)
          if (i < A.cluster) v[i] = ld_cluster_f4(cluster_map(at, i));
        float2 x = make_float2(-INFINITY, 0.f);
        if (lane < A.cluster) {
          const uint32_t y = cluster_map(smem_u32(block_ml + r), lane);
          x = make_float2(ld_cluster_f32(y), ld_cluster_f32(y + 4));
        }
        const float M = warp_max(x.y == 0.f ? -INFINITY : x.x), w = x.y == 0.f ? 0.f : exp2f(x.x - M), L = warp_sum(w * x.y);
        const unsigned seen = __ballot_sync(0xffffffffu, x.y != 0.f);  // blocks that saw a slot
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kMostCluster; ++i) {
          const float wi = __shfl_sync(0xffffffffu, w, i);
          if (seen >> i & 1) {
            o.x += wi * v[i].x;
            o.y += wi * v[i].y;
            o.z += wi * v[i].z;
            o.w += wi * v[i].w;
          }
        }
        const bool off = d < D && finish4<T>(A, rq, h, r, d, o, M, L);
        if (__any_sync(0xffffffffu, off)) attend_row<T, D>(A, rq, b, r / a.group, h * a.group + r % a.group, lane);
      }
      __syncwarp();
      cluster_sync();  // every block's sums are read
      return;
    }
    if (__syncthreads_or(bad)) redo_rows<T, D, kFewThreads>(A, rq, b, h, 0, R, bad_rows);
    u += t1 - t0;
  } while (u < u1);
}

// ------------------------------------------------------------------ join
// Block (g, y): rows 4y .. 4y+3 of the join that block g of the few-rows kernel left, a head of which
// blocks g-1, g, ... each worked on a part (one context of 4096 slots and 8 heads: 39 parts).  All that bounds it
// is round trips to L2, so nothing waits for one part at a time: a warp takes the references and sums of
// a row's parts side by side and leaves their weights in shared memory; then the threads, as many groups
// of them as fit, each add every kth part.
constexpr int kJoinThreads = 512;
constexpr int kJoinHeld = 10;  // parts of a thread in registers
constexpr int kJoinRows = 4;
template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads) attention_join(const __grid_constant__ PagedAttnArgs A) {
  __shared__ unsigned bad_rows;
  __shared__ float weight[kJoinRows][kJoinParts];
  __shared__ float2 row_ml[kJoinRows];
  __shared__ float4 sums[kJoinThreads];
  const int g = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_trigger();
  const PagedJoin j = A.join[g];
  const int r0 = blockIdx.y * kJoinRows, n = min(j.n - r0, kJoinRows);
  if (j.np == 0 || n <= 0) return;
  const Request rq = {j.len, j.row0, j.rows};
  auto slot = [&](int i) { return static_cast<int64_t>(2 * (g - 1 + i) + (i == 0 ? 1 : 0)) * kFewRows + r0; };
  const int pieces = n * (D / 4);  // at most kJoinThreads
  const int groups = kJoinThreads / pieces, k = tid / pieces, c = tid - k * pieces;
  const int r = c / (D / 4), d = (c - r * (D / 4)) * 4;
  // this thread's first parts are on their way while the weights are worked out
  float4 held[kJoinHeld];
#pragma unroll
  for (int x = 0; x < kJoinHeld; ++x) {
    const int i = k + x * groups;
    if (k < groups && i < j.np) held[x] = __ldcg(reinterpret_cast<const float4 *>(A.part_o + (slot(i) + r) * D + d));
  }
  if (tid == 0) bad_rows = 0u;
  if (warp < n) {
    float m = -INFINITY, l = 0.f;
    for (int i = lane; i < j.np; i += 32) {
      const float2 x = __ldcg(A.part_ml + slot(i) + warp);
      const float mn = x.y == 0.f ? m : fmaxf(m, x.x);
      l = (l == 0.f ? 0.f : l * exp2f(m - mn)) + (x.y == 0.f ? 0.f : x.y * exp2f(x.x - mn));
      m = mn;
      weight[warp][i] = x.y == 0.f ? INFINITY : x.x;  // infinity: a part that saw no slot
    }
    const float M = warp_max(m);
    const float L = warp_sum(l == 0.f ? 0.f : l * exp2f(m - M));
    for (int i = lane; i < j.np; i += 32) {
      const float x = weight[warp][i];
      weight[warp][i] = x == INFINITY ? -1.f : exp2f(x - M);
    }
    if (lane == 0) row_ml[warp] = make_float2(M, L);
  }
  __syncthreads();
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](int i, const float4 &v) {
    const float w = weight[r][i];
    if (!(w < 0.f)) {  // a weight of zero counts: it keeps a visible infinity or NaN
      o.x += w * v.x;
      o.y += w * v.y;
      o.z += w * v.z;
      o.w += w * v.w;
    }
  };
  if (k < groups) {
#pragma unroll
    for (int x = 0; x < kJoinHeld; ++x)
      if (k + x * groups < j.np) add(k + x * groups, held[x]);
#pragma unroll 4
    for (int i = k + kJoinHeld * groups; i < j.np; i += groups)
      add(i, __ldcg(reinterpret_cast<const float4 *>(A.part_o + (slot(i) + r) * D + d)));
  }
  if (groups > 1) {
    sums[tid] = o;
    __syncthreads();
    if (k == 0)
      for (int i = 1; i < groups; ++i) {
        const float4 v = sums[tid + i * pieces];
        o.x += v.x;
        o.y += v.y;
        o.z += v.z;
        o.w += v.w;
      }
  }
  const bool bad = k == 0 && finish4<T>(A, rq, j.h, j.from + r0 + r, d, o, row_ml[r].x, row_ml[r].y);
  if (bad) atomicOr(&bad_rows, 1u << r);
  if (__syncthreads_or(bad)) redo_rows<T, D, kJoinThreads>(A, rq, j.b, j.h, j.from + r0, n, bad_rows);
}
static_assert(kJoinRows * 128 / 4 <= kJoinThreads, "a block's pieces");

// ------------------------------------------------------------------ host
// A head of few slots is not split but one block's, whose warps take eight units of it at most: that saves
// summing up the lengths and the joining launch (8 requests x 8 heads of 512 slots: 9.3 us, shared out 13.1 us).
constexpr int kWholeSlots = 512;
// Where there are fewer heads than blocks, a head is a cluster's, whose blocks join their parts through distributed
// shared memory: as many blocks as are left and kBlockSlots slots for each (8 heads of 512 slots: eight
// blocks 5.8 us, four 6.5 us, one 9.1 us; of 128 slots: one 4.9 us, two 5.8 us).
// More heads than the device holds clusters at once would go in turns (2 requests of 4096 slots, 16 heads, of which
// it holds 14 clusters of sixteen: eight blocks each 12.7 us, sixteen 17.6 us).
constexpr int kBlockSlots = 64;
// What a block of a cluster goes through alone is weighed against an even share of the call, the joining launch and its
// parts (a head is at most n_ctas / heads parts), all in slots of a block (us of a cluster of sixteen / shared out; one
// request, group 4, D = 128):
//   KV heads     4096       16 384      20 480      24 576      28 672      32 768
//   1         7.5/10.9   16.8/21.3   19.8/24.5   22.6/24.7   25.5/25.0   28.3/25.5
//   2         7.8/12.7   16.8/19.0   19.8/20.0   22.6/20.3   25.6/20.9   28.4/21.9
//   4         8.3/14.0   17.1/19.2   20.1/20.7   22.9/21.7   25.8/22.8   28.8/23.9
//   8         9.8/14.5   20.3/21.9   23.9/24.7   27.3/27.3   30.9/29.4   34.2/32.0
// The rule shares out from 23 777, 19 729, 19 281 and 24 193 slots on; both take as long at about 27 500, 20 300, 20 900 and
// 24 600 (group 1: 20 900, 16 400 and 24 600 of 1, 2 and 8 heads; group 16: 22 000, 16 800 and 18 000; D = 64 within a
// tenth of group 4).  It goes by the bound max_len: a shorter request under a larger bound takes the second figure.
// Where clusters give every SM a block, shares have no more of the device: up to kClusterFilled slots a block (windows, 8
// heads: 5 requests, 8192 slots, 4 blocks a head 34.9/37.9; 10 requests, 4096 slots, 2 blocks 34.8/38.5; 19
// requests 51.0/57.7).
// All of this holds for heads that are alike, as a window or a call of one request makes them.  Else a cluster is as slow as
// its longest head, and max_len only bounds it: up to kClusterSlots slots a block (8 requests of 16 384 slots and one head
// 20.4/22.5, 2 requests of 8 heads 34.1/31.3; 16 ragged requests, a block up to 16 384 slots: 236/184).
constexpr int kClusterSlots = 1088, kClusterFilled = 2176;
constexpr int kJoinSlots = 800, kPartSlots = 2;

static int few_blocks() { return few_ctas() < kJoinParts ? few_ctas() : kJoinParts - 1; }

size_t few_bytes(int head_dim) {
  const size_t parts = 2 * static_cast<size_t>(few_blocks()) * kFewRows;
  return align256(few_blocks() * sizeof(PagedJoin)) + align256(parts * head_dim * 4) + align256(parts * 8);
}

template <typename T, int D, bool HALF> static cudaError_t launch(PagedAttnArgs &A, cudaStream_t s) {
  const PagedArgs &a = A.p;
  auto kernel = attention_few<T, D, HALF>;
  static const ClustersAtOnce fit(kernel, kFewThreads, Few<D>::kSmem);
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Few<D>::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t seen = visible_slots(a), heads = static_cast<int64_t>(a.n_requests) * a.n_kv_heads;
  int blocks = 1;
  while (blocks < kMostCluster && seen > (blocks > 1 ? blocks : 2) * kBlockSlots && heads <= fit.of(2 * blocks)) blocks *= 2;
  const bool alike = seen < a.max_len || a.n_requests == 1;
  const int64_t each = (seen + blocks - 1) / blocks, share = heads * seen / A.n_ctas;  // a block's slots, either way
  if (blocks == 1)
    A.whole = seen <= kWholeSlots;
  else if (alike)
    A.whole = each <= share + kJoinSlots + kPartSlots * A.n_ctas / heads || (heads * blocks >= num_sms() && each <= kClusterFilled);
  else
    A.whole = each <= kClusterSlots;
  A.cluster = A.whole ? blocks : 1;
  if (A.whole) {
    const cudaError_t c = allow_cluster(kernel, blocks);
    if (c != cudaSuccess) return c;
    return launch_pdl_cluster(kernel, dim3(static_cast<unsigned>(heads * blocks)), dim3(kFewThreads), Few<D>::kSmem, s, blocks, A);
  }
  const cudaError_t f = launch_pdl(kernel, dim3(A.n_ctas), dim3(kFewThreads), Few<D>::kSmem, s, A);
  if (f != cudaSuccess) return f;
  const int rows = a.max_rows * a.group;
  return launch_pdl(attention_join<T, D>, dim3(A.n_ctas, (rows + kJoinRows - 1) / kJoinRows), dim3(kJoinThreads), 0, s, A);
}
template <typename T, int D> static cudaError_t launch(PagedAttnArgs &A, cudaStream_t s) {
  return A.p.max_rows * A.p.group <= 8 ? launch<T, D, true>(A, s) : launch<T, D, false>(A, s);
}

std::string launch_attention_few(PagedAttnArgs A, void *workspace, int dtype, cudaStream_t s) {
  uint8_t *p = static_cast<uint8_t *>(workspace);
  A.n_ctas = few_blocks();
  const size_t parts = 2 * static_cast<size_t>(A.n_ctas) * kFewRows;
  A.join = reinterpret_cast<PagedJoin *>(p);
  p += align256(A.n_ctas * sizeof(PagedJoin));
  A.part_o = reinterpret_cast<float *>(p);
  p += align256(parts * A.p.head_dim * 4);
  A.part_ml = reinterpret_cast<float2 *>(p);
  cudaError_t e;
  if (dtype == BD_BF16)
    e = A.p.head_dim == 128 ? launch<__nv_bfloat16, 128>(A, s) : launch<__nv_bfloat16, 64>(A, s);
  else
    e = A.p.head_dim == 128 ? launch<__half, 128>(A, s) : launch<__half, 64>(A, s);
  return e == cudaSuccess ? std::string() : std::string("paged attention: ") + cudaGetErrorString(e);
}

}  // namespace bd
