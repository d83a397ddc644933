// Head norms with the position rotation (bd_head_norm_rope).
//
// A lane holds 8 consecutive values of a head, so a head of D values is D / 8 lanes: its sum of squares is a
// shuffle tree over them, and a half-split pair's other value lies rotary / 16 lanes away and comes by shuffle as it was
// read (two 16-bit values a word); interleaved pairs lie in one lane.  A warp takes heads of one row, kHeadsEach loads
// of them in flight.  The angles depend on the row and the pair only: a block works them out once for its rows, before
// its warps need them and while their first heads are on their way, and keeps cosines and sines in shared memory.
// Angles are reduced without error: pos * turns is the angle in 2^-64 turns modulo one turn (integer), its upper
// 32 bits as a signed fraction of a half turn are what sincospif gets: off by 2^-24 relative, at any position.
// Bound by the bytes, each value read and written once; of few rows by the launch.
#include "bd_checks.h"
#include "bd_paged_device.cuh"

namespace bd {

static std::atomic<bool> target_used{false};  // some call of these files has launched, or been captured
void use_target_kernels() { target_used.store(true, std::memory_order_release); }
unsigned take_error_words_target() {
  if (!target_used.load(std::memory_order_acquire)) return 0;
  return take_error_word_paged_plan() | take_error_word_paged4() | take_error_word_paged4_attn() | take_error_word_logprobs();
}

namespace {

constexpr int kHeadThreads = 256;
constexpr int kHeadsEach = 4;     // loads of a warp in flight
constexpr int kHeadRowsMost = 8;  // rows of a block

struct HeadArgs {
  bd_head_rope c;
  int n_rows, rows_per_cta;
  const int32_t *pos;
  const uint16_t *q, *k;
  uint16_t *q_out, *k_out;
  int64_t q_stride, k_stride, q_out_stride, k_out_stride;
};

template <typename T> __device__ __forceinline__ void unpack8(const uint4 &w, float (&x)[8]) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = Pair<T>::unpack(v[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

template <typename T, int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kHeadThreads) head_norm_rope_kernel(const __grid_constant__ HeadArgs A) {
  constexpr int L = D / 8, H = 32 / L;  // lanes of a head, heads of a warp's load
  __shared__ __align__(16) float cs[kHeadRowsMost][2][D / 2];  // cosines and sines of the block's rows
  __shared__ int pos_s[kHeadRowsMost];
  const bd_head_rope &c = A.c;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int piece = lane % L, sub = lane / L, half = c.rotary_dim / 2;
  const int r0 = blockIdx.x * A.rows_per_cta, n = min(A.rows_per_cta, A.n_rows - r0);
  const int heads = c.n_q_heads + c.n_kv_heads, units = (heads + H * kHeadsEach - 1) / (H * kHeadsEach);
  pdl_wait();
  pdl_trigger();
  uint4 raw[kHeadsEach];
  auto load = [&](int u) {  // unit u: heads of row u / units
    const int r = u / units, h0 = (u - r * units) * H * kHeadsEach + sub;
#pragma unroll
    for (int i = 0; i < kHeadsEach; ++i) {
      const int h = h0 + i * H;
      raw[i] = make_uint4(0, 0, 0, 0);
      if (r >= n || h >= heads) continue;
      const int64_t row = r0 + r;
      const uint16_t *src = h < c.n_q_heads ? A.q + row * A.q_stride + h * D : A.k + row * A.k_stride + (h - c.n_q_heads) * D;
      raw[i] = *reinterpret_cast<const uint4 *>(src + piece * 8);
    }
  };
  load(warp);
  const uint4 none = make_uint4(0, 0, 0, 0);
  // this lane's gains, and those of its half-split partners
  const bool first = piece * 8 < half, turned = piece * 8 < c.rotary_dim;
  const int partner = !turned ? piece : first ? piece + half / 8 : piece - half / 8;
  const uint4 *qg = static_cast<const uint4 *>(c.q_gain), *kg = static_cast<const uint4 *>(c.k_gain);
  const uint4 qg0 = qg ? __ldg(qg + piece) : none, qg1 = qg ? __ldg(qg + partner) : none;
  const uint4 kg0 = kg ? __ldg(kg + piece) : none, kg1 = kg ? __ldg(kg + partner) : none;
  if (tid < n) pos_s[tid] = A.pos[r0 + tid];
  for (int x = tid; x < n * half; x += kHeadThreads) {
    const int r = x / half, j = x - r * half;
    const uint64_t turn = static_cast<uint64_t>(static_cast<int64_t>(A.pos[r0 + r])) * __ldg(c.turns + j);
    float s, co;
    sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f, &s, &co);
    cs[r][0][j] = co;
    cs[r][1][j] = s;
  }
  __syncthreads();
  for (int u = warp; u < n * units; u += kHeadThreads / 32) {
    if (u != warp) load(u);
    const int r = u / units, h0 = (u - r * units) * H * kHeadsEach + sub;
    const int64_t row = r0 + r;
    const bool skip = pos_s[r] < 0;
    float co[8], si[8];
    if (INTERLEAVED) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = piece * 4 + e;
        co[e] = turned ? cs[r][0][j] : 1.f;
        si[e] = turned ? cs[r][1][j] : 0.f;
      }
    } else {
      const int j0 = first ? piece * 8 : piece * 8 - half;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        co[e] = turned ? cs[r][0][j0 + e] : 1.f;
        si[e] = !turned ? 0.f : first ? -cs[r][1][j0 + e] : cs[r][1][j0 + e];
      }
    }
#pragma unroll
    for (int i = 0; i < kHeadsEach; ++i) {
      const int h = h0 + i * H;
      float x[8], y[8], g[8];
      unpack8<T>(raw[i], x);
      auto mean_square = [&](float f) {  // of x f
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += x[e] * f * (x[e] * f);
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        return sum * (1.f / D);
      };
      const float mean = mean_square(1.f);
      float inv = rsqrtf(mean + c.eps);
      if (__any_sync(0xffffffffu, mean == INFINITY)) {  // squares beyond fp32: of values 2^-70 as large
        const float small = mean_square(0x1p-70f);
        if (mean == INFINITY) inv = rsqrtf(small) * 0x1p-70f;
      }
      const bool is_q = h < c.n_q_heads, plain = is_q ? qg == nullptr : kg == nullptr;
      unpack8<T>(is_q ? qg0 : kg0, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= plain ? inv : inv * g[e];
      if (INTERLEAVED) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          y[2 * e] = x[2 * e] * co[e] - x[2 * e + 1] * si[e];
          y[2 * e + 1] = x[2 * e] * si[e] + x[2 * e + 1] * co[e];
        }
      } else {
        uint4 other;
        const int from = sub * L + partner;
        other.x = __shfl_sync(0xffffffffu, raw[i].x, from);
        other.y = __shfl_sync(0xffffffffu, raw[i].y, from);
        other.z = __shfl_sync(0xffffffffu, raw[i].z, from);
        other.w = __shfl_sync(0xffffffffu, raw[i].w, from);
        unpack8<T>(other, y);
        unpack8<T>(is_q ? qg1 : kg1, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = x[e] * co[e] + y[e] * (plain ? inv : inv * g[e]) * si[e];
      }
      if (h < heads && !skip) {
        uint16_t *dst = is_q ? A.q_out + row * A.q_out_stride + h * D : A.k_out + row * A.k_out_stride + (h - c.n_q_heads) * D;
        *reinterpret_cast<uint4 *>(dst + piece * 8) =
            make_uint4(Pair<T>::pack(y[0], y[1]), Pair<T>::pack(y[2], y[3]), Pair<T>::pack(y[4], y[5]), Pair<T>::pack(y[6], y[7]));
      }
    }
  }
}

template <typename T, int D> cudaError_t launch(const HeadArgs &A, cudaStream_t s) {
  const dim3 grid((A.n_rows + A.rows_per_cta - 1) / A.rows_per_cta);
  return launch_pdl(A.c.interleaved ? head_norm_rope_kernel<T, D, true> : head_norm_rope_kernel<T, D, false>, grid, dim3(kHeadThreads), 0, s, A);
}
template <typename T> cudaError_t launch(const HeadArgs &A, cudaStream_t s) {
  return A.c.head_dim == 64 ? launch<T, 64>(A, s) : A.c.head_dim == 128 ? launch<T, 128>(A, s) : launch<T, 256>(A, s);
}

}  // namespace
}  // namespace bd

using namespace bd;

extern "C" bd_status bd_head_norm_rope(const bd_head_rope *c, int n_rows, const int32_t *pos, const void *q, int64_t q_stride,
                                       const void *k, int64_t k_stride, void *q_out, int64_t q_out_stride, void *k_out,
                                       int64_t k_out_stride, void *stream) {
  constexpr const char *kWho = "head norm";
  if (!c) return refuse(BD_ERR_INVALID_ARG, "head norm: the configuration is NULL");
  if (c->dtype != BD_BF16 && c->dtype != BD_F16) return refuse(BD_ERR_UNSUPPORTED, "head norm: dtype must be BD_BF16 or BD_F16");
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
    return refuse(BD_ERR_UNSUPPORTED, "head norm: head_dim must be 64, 128 or 256");
  if (c->rotary_dim < 0 || c->rotary_dim > c->head_dim || c->rotary_dim % 16)
    return refuse(BD_ERR_UNSUPPORTED, "head norm: rotary_dim must be a multiple of 16 up to head_dim");
  if (c->n_q_heads < 0 || c->n_kv_heads < 0 || c->n_q_heads > (1 << 17) || c->n_kv_heads > (1 << 17))
    return refuse(BD_ERR_INVALID_ARG, "head norm: head counts must be in 0..2^17");
  if (!(c->eps > 0.f) || !std::isfinite(c->eps)) return refuse(BD_ERR_INVALID_ARG, "head norm: eps must be > 0 and finite");
  if (misaligned(c->q_gain, 16) || misaligned(c->k_gain, 16) || misaligned(c->turns, 8) || (c->rotary_dim > 0 && !c->turns))
    return refuse(BD_ERR_INVALID_ARG, "head norm: gains must be 16-byte aligned, and turns given, 8-byte aligned");
  if (n_rows < 0 || n_rows > (1 << 28)) return refuse(BD_ERR_INVALID_ARG, "head norm: n_rows must be in 0..2^28");
  if (n_rows == 0 || c->n_q_heads + c->n_kv_heads == 0) return BD_OK;
  if (!pos || misaligned(pos, 4)) return refuse(BD_ERR_INVALID_ARG, "head norm: pos must be given");
  struct Side {
    const void *in, *out;
    int64_t stride, out_stride, width;
    const char *name, *out_name;
  } sides[] = {{q, q_out, q_stride, q_out_stride, static_cast<int64_t>(c->n_q_heads) * c->head_dim, "q", "q_out"},
               {k, k_out, k_stride, k_out_stride, static_cast<int64_t>(c->n_kv_heads) * c->head_dim, "k", "k_out"}};
  for (const Side &x : sides) {
    if (x.width == 0) continue;
    if (bd_status st = check_rows(x.in, x.stride, x.width, n_rows, x.name, kWho)) return st;
    if (bd_status st = check_rows(x.out, x.out_stride, x.width, n_rows, x.out_name, kWho)) return st;
  }
  // Rows side by side in one projection's rows interleave without sharing an element: two arrays of one stride
  // whose rows lie apart within it do not overlap.
  auto clash = [&](const void *a, int64_t sa, int64_t wa, const void *b, int64_t sb, int64_t wb) {
    if (wa == 0 || wb == 0 || !overlap(a, row_bytes(sa, wa, n_rows), b, row_bytes(sb, wb, n_rows))) return false;
    if (sa != sb || sa < wa || sa < wb) return true;
    const int64_t d = (static_cast<const char *>(b) - static_cast<const char *>(a)) / 2, m = ((d % sa) + sa) % sa;
    return !(m >= wa && m + wb <= sa);
  };
  for (const Side &x : sides) {
    for (const Side &y : sides) {
      const bool own = &x == &y && x.in == x.out && x.stride == x.out_stride;
      if (!own && clash(x.out, x.out_stride, x.width, y.in, y.stride, y.width))
        return refuse(BD_ERR_INVALID_ARG, std::string("head norm: ") + x.out_name + " and " + y.name + " overlap");
    }
    for (const void *g : {c->q_gain, c->k_gain})
      if (x.width && g && overlap(x.out, row_bytes(x.out_stride, x.width, n_rows), g, 2 * c->head_dim))
        return refuse(BD_ERR_INVALID_ARG, std::string("head norm: ") + x.out_name + " overlaps a gain");
    if (x.width && (overlap(x.out, row_bytes(x.out_stride, x.width, n_rows), pos, 4ll * n_rows) ||
                    overlap(x.out, row_bytes(x.out_stride, x.width, n_rows), c->turns, 4ll * c->rotary_dim)))
      return refuse(BD_ERR_INVALID_ARG, std::string("head norm: ") + x.out_name + " overlaps pos or turns");
  }
  if (clash(q_out, q_out_stride, sides[0].width, k_out, k_out_stride, sides[1].width))
    return refuse(BD_ERR_INVALID_ARG, "head norm: q_out and k_out overlap");
  HeadArgs A = {};
  A.c = *c;
  A.n_rows = n_rows;
  A.pos = pos;
  A.q = static_cast<const uint16_t *>(q);
  A.k = static_cast<const uint16_t *>(k);
  A.q_out = static_cast<uint16_t *>(q_out);
  A.k_out = static_cast<uint16_t *>(k_out);
  A.q_stride = q_stride;
  A.k_stride = k_stride;
  A.q_out_stride = q_out_stride;
  A.k_out_stride = k_out_stride;
  // a row a block while the SMs are not filled; then as many as keep four blocks an SM
  A.rows_per_cta = 1;
  while (2 * A.rows_per_cta <= kHeadRowsMost && n_rows >= 8 * A.rows_per_cta * num_sms()) A.rows_per_cta *= 2;
  const cudaError_t e = c->dtype == BD_BF16 ? launch<__nv_bfloat16>(A, static_cast<cudaStream_t>(stream)) : launch<__half>(A, static_cast<cudaStream_t>(stream));
  return ran(e == cudaSuccess ? std::string() : std::string("head norm: ") + cudaGetErrorString(e));
}
