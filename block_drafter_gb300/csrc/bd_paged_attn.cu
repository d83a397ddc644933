// Attention of a call's rows over their requests' paged slots (bd_paged_attention).
//
// One warp per (row, query head): it walks the slots the row sees 32 at a time -- each lane
// forms one slot's score, the warp keeps the running maximum m and sum l of exp2(s - m), and each
// lane adds the 32 weighted values of its own D/32 columns:
//   m' = max(m, max s),  l' = l 2^(m-m') + sum 2^(s-m'),  o' = o 2^(m-m') + sum 2^(s-m') v
#include "bd_paged_device.cuh"

namespace bd {

BD_DEFINE_ERROR_TAKER(take_error_word_paged_attn)

template <typename T, int D>
__device__ void attend_row(const PagedAttnArgs &A, const Request &rq, int b, int i, int head, float *qs, int lane) {
  const PagedArgs &a = A.p;
  const int hq = a.n_kv_heads * a.group, row = rq.row0 + i, p = rq.n - rq.rows + i;
  const T *q = static_cast<const T *>(a.q) + row * a.q_stride + head * D;
  constexpr int C = D / 32;  // columns of a lane
#pragma unroll
  for (int c = 0; c < C; ++c) qs[c * 32 + lane] = to_f(q[c * 32 + lane]);
  __syncwarp();
  const int first = p >= 0 ? window_first(a, p) : 0;
  const int n_sinks = min(a.n_sink, first);
  const int count = p >= 0 ? n_sinks + p + 1 - first : 0;
  const int64_t head_off = static_cast<int64_t>(head / a.group) * a.head_stride;
  const T *K = static_cast<const T *>(a.k) + head_off, *V = static_cast<const T *>(a.v) + head_off;
  const int32_t *table = a.page_table + static_cast<int64_t>(b) * a.table_width;
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
          const float *y = qs + c * 8;
          s += x0.x * y[0] + x0.y * y[1] + x1.x * y[2] + x1.y * y[3] + x2.x * y[4] + x2.y * y[5] + x3.x * y[6] +
               x3.y * y[7];
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
  if (A.lse && lane == 0)
    A.lse[static_cast<int64_t>(row) * hq + head] = l == 0.f ? -INFINITY : kLn2 * (m + log2f(l));
  __syncwarp();
}

template <typename T, int D>
__global__ void __launch_bounds__(128) paged_attention_rows(const __grid_constant__ PagedAttnArgs A) {
  __shared__ float qs[4][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, b = blockIdx.y;
  pdl_wait();
  pdl_trigger();
  const Request rq = request_of(A.p, b);
  const int hq = A.p.n_kv_heads * A.p.group;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * 4 + warp; u < static_cast<int64_t>(rq.rows) * hq; u += gridDim.x * 4)
    attend_row<T, D>(A, rq, b, static_cast<int>(u / hq), static_cast<int>(u % hq), qs[warp], lane);
}

std::string launch_paged_attention(const PagedAttnArgs &A, int dtype, cudaStream_t s) {
  const PagedArgs &a = A.p;
  const int64_t units = static_cast<int64_t>(a.max_rows) * a.n_kv_heads * a.group;
  const int64_t blocks = (units + 3) / 4;
  const dim3 grid(static_cast<unsigned>(blocks < 65535 ? blocks : 65535), a.n_requests);
  auto go = [&](auto kernel) { return launch_pdl(kernel, grid, dim3(128), 0, s, A); };
  cudaError_t e;
  if (dtype == BD_BF16)
    e = a.head_dim == 128 ? go(paged_attention_rows<__nv_bfloat16, 128>) : go(paged_attention_rows<__nv_bfloat16, 64>);
  else
    e = a.head_dim == 128 ? go(paged_attention_rows<__half, 128>) : go(paged_attention_rows<__half, 64>);
  return e == cudaSuccess ? std::string() : std::string("paged attention: ") + cudaGetErrorString(e);
}

}  // namespace bd
