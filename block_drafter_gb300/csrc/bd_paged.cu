// Paged K/V cache: the entry points' checks, and the kernels of the append, the accumulated
// attention weights and the eviction.
#include "bd_paged_device.cuh"

#include <cmath>

namespace bd {

BD_DEFINE_ERROR_TAKER(take_error_word_paged)

// ------------------------------------------------------------------ append
// Copies each row's keys and values into its slot, 16 bytes a thread.  A block takes rows_per_cta
// consecutive rows and first finds the request of each: every thread tests some of the requests'
// row ranges against the block's.
constexpr int kAppendThreads = 256;
constexpr int kAppendRows = 8;

struct PagedAppendArgs {
  PagedArgs p;
  const void *k_new, *v_new;
  int64_t k_stride, v_stride;
  int rows_per_cta;
};

__global__ void __launch_bounds__(kAppendThreads) paged_append_kernel(const __grid_constant__ PagedAppendArgs A) {
  const PagedArgs &a = A.p;
  __shared__ int64_t off[kAppendRows];  // element offset of the row's slot, -1: not stored
  const int r0 = blockIdx.x * A.rows_per_cta, r1 = min(a.n_rows, r0 + A.rows_per_cta);
  if (threadIdx.x < kAppendRows) off[threadIdx.x] = -1;
  pdl_wait();
  pdl_trigger();
  __syncthreads();
  for (int b = threadIdx.x; b < a.n_requests; b += kAppendThreads) {
    const int s = a.row_start[b], e = a.row_start[b + 1];
    if (s < 0 || e < s || e > a.n_rows || e - s > a.max_rows) {
      atomicOr(&g_error_word, DEVERR_BAD_INDEX);
      continue;
    }
    if (s >= r1 || e <= r0) continue;
    const int n = request_len(a, b);
    for (int r = max(s, r0); r < min(e, r1); ++r) {
      const int p = n - (e - r);
      off[r - r0] = p < 0 ? -1 : slot_offset(a, a.page_table + static_cast<int64_t>(b) * a.table_width, p);
    }
  }
  __syncthreads();
  const int per_head = a.head_dim / 8, per_side = a.n_kv_heads * per_head, per_row = 2 * per_side;
  for (int c = threadIdx.x; c < (r1 - r0) * per_row; c += kAppendThreads) {
    const int r = c / per_row, u = c - r * per_row;
    if (off[r] < 0) continue;
    const bool v = u >= per_side;
    const int w = v ? u - per_side : u, h = w / per_head, x = (w - h * per_head) * 8;
    const uint16_t *src = static_cast<const uint16_t *>(v ? A.v_new : A.k_new) +
                          (r0 + r) * (v ? A.v_stride : A.k_stride) + w * 8;
    uint16_t *dst = static_cast<uint16_t *>(const_cast<void *>(v ? a.v : a.k)) + off[r] + h * a.head_stride + x;
    *reinterpret_cast<uint4 *>(dst) = *reinterpret_cast<const uint4 *>(src);
  }
}

static std::string launch_append(PagedAppendArgs &A, cudaStream_t s) {
  A.rows_per_cta = A.p.n_rows > 8 * num_sms() ? kAppendRows : 1;
  const int grid = (A.p.n_rows + A.rows_per_cta - 1) / A.rows_per_cta;
  const cudaError_t e = launch_pdl(paged_append_kernel, dim3(grid), dim3(kAppendThreads), 0, s, A);
  return e == cudaSuccess ? std::string() : std::string("paged append: ") + cudaGetErrorString(e);
}

// ------------------------------------------------------------------ accumulated weights
// out[j] = decay in[j] + sum over rows i and heads of 2^(scale log2(e) k_j.q_i - log2(e) lse_i).
// Bound by K's bytes for a token or a block, by the tensor cores for many rows.  A warp owns 16 slots of
// a request: their keys are the A operand of mma.sync m16n8k16 and stay in registers while the rows of
// the KV head pass by, 8 at a time, as B; so a slot's weights are summed in the registers of four lanes,
// without atomics, over all rows and heads of the warp.  Few slots give a block's eight warps fewer tiles
// and split the KV heads among them (summed through shared memory in a fixed order).
// The order of the D products of a score is free, so both operands take it as 16-byte pieces from
// global memory: lane l holds pieces l%4, l%4 + 4, ... of its rows, two MMA steps each.
constexpr int kWeightWarps = 8;

template <typename T> __device__ __forceinline__ void mma_kq(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma_kq<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma_kq<__half>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// P pieces of 16 bytes (every fourth from this lane's on) of a row, zeros where p is null.
template <int P> __device__ __forceinline__ void load_pieces(uint4 (&v)[P], const void *p) {
#pragma unroll
  for (int c = 0; c < P; ++c) v[c] = p ? __ldg(static_cast<const uint4 *>(p) + 4 * c) : make_uint4(0, 0, 0, 0);
}

template <typename T, int D>
__global__ void __launch_bounds__(32 * kWeightWarps, 2) paged_weights_kernel(const __grid_constant__ PagedWeightsArgs A, int head_split) {
  constexpr int P = D / 32;  // pieces of a row per lane
  __shared__ float part[kWeightWarps][16];
  const PagedArgs &a = A.p;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, b = blockIdx.y, quad = lane >> 2, kq = lane & 3;
  const int tiles = kWeightWarps / head_split;           // slot tiles of the block
  const int hs = warp / tiles;                           // this warp's KV heads: hs, hs + head_split, ...
  const int j0 = (blockIdx.x * tiles + warp % tiles) * 16;
  pdl_wait();
  pdl_trigger();
  const Request rq = request_of(a, b);
  if (blockIdx.x * tiles * 16 >= rq.n) return;
  const int used = A.rows_used ? max(0, min(A.rows_used[b], rq.rows)) : rq.rows;
  const int base = rq.n - rq.rows, G = a.group, hq = a.n_kv_heads * G;
  // tokens i (slots base + i) that see some slot of the tile, and those that see all of it
  const int j1 = min(j0 + 15, rq.n - 1);
  const bool sinks = j0 < a.n_sink, all_sinks = j1 < a.n_sink;
  int i_lo = max(0, j0 - base), i_hi = used;  // [i_lo, i_hi)
  int f_lo = max(0, j1 - base), f_hi = used;
  if (a.window > 0) {
    auto behind = [&](int j) {  // the first token that does not see slot j any more, 0 .. used
      const int64_t i = static_cast<int64_t>(j) + a.window - base;
      return static_cast<int>(i < 0 ? 0 : i < used ? i : used);
    };
    if (!sinks) i_hi = behind(j1);
    if (!all_sinks) f_hi = behind(j0);
  }
  float acc[2] = {0.f, 0.f};  // slots j0 + quad, + 8
  if (j0 < rq.n && i_lo < i_hi) {
    const int32_t *table = a.page_table + static_cast<int64_t>(b) * a.table_width;
    const T *K[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int j = j0 + quad + 8 * x;
      const int64_t off = j < rq.n ? slot_offset(a, table, j) : -1;
      K[x] = off < 0 ? nullptr : static_cast<const T *>(a.k) + off + kq * 8;
    }
    const int t0 = i_lo * G / 8, t1 = (i_hi * G + 7) / 8;  // row tiles
    const int full0 = f_lo * G, full1 = f_hi * G;          // rows that see all of the tile's slots
    const int R = i_hi * G;
    uint4 k[2][P];
    if (hs < a.n_kv_heads)
#pragma unroll
      for (int x = 0; x < 2; ++x) load_pieces(k[x], K[x] ? K[x] + hs * a.head_stride : nullptr);
    for (int h = hs; h < a.n_kv_heads; h += head_split) {
      uint32_t kf[2 * P][4];
#pragma unroll
      for (int c = 0; c < P; ++c) {
        const uint4 u = k[0][c], v = k[1][c];
        kf[2 * c][0] = u.x, kf[2 * c][1] = v.x, kf[2 * c][2] = u.y, kf[2 * c][3] = v.y;
        kf[2 * c + 1][0] = u.z, kf[2 * c + 1][1] = v.z, kf[2 * c + 1][2] = u.w, kf[2 * c + 1][3] = v.w;
      }
      if (h + head_split < a.n_kv_heads)
#pragma unroll
        for (int x = 0; x < 2; ++x) load_pieces(k[x], K[x] ? K[x] + (h + head_split) * a.head_stride : nullptr);
      // this lane's row of a tile: token i, head e of the group
      const uint32_t r0 = t0 * 8 + quad;
      int i = r0 / static_cast<uint32_t>(G), e = r0 - i * G;
      const int di = 8 / G, de = 8 - di * G;
      const T *q = static_cast<const T *>(a.q) + rq.row0 * a.q_stride + h * G * D + kq * 8;
      const float *lse = A.lse + static_cast<int64_t>(rq.row0) * hq + h * G;
      uint4 qn[P];
      load_pieces(qn, i < i_hi ? q + i * a.q_stride + e * D : nullptr);
      float ln = i < i_hi ? lse[static_cast<int64_t>(i) * hq + e] : INFINITY;  // no weight behind the last row
      for (int t = t0; t < t1; ++t) {
        uint4 qf[P];
#pragma unroll
        for (int c = 0; c < P; ++c) qf[c] = qn[c];
        const float l = ln * (1.f / kLn2);
        const int token = i;
        i += di;
        e += de;
        if (e >= G) e -= G, ++i;
        if (t + 1 < t1) {
          load_pieces(qn, i < i_hi ? q + i * a.q_stride + e * D : nullptr);
          ln = i < i_hi ? lse[static_cast<int64_t>(i) * hq + e] : INFINITY;
        }
        float c0[4] = {}, c1[4] = {};
#pragma unroll
        for (int c = 0; c < P; ++c) {
          mma_kq<T>(c0, kf[2 * c], qf[c].x, qf[c].y);
          mma_kq<T>(c1, kf[2 * c + 1], qf[c].z, qf[c].w);
        }
        // columns of this lane: rows 2 kq and 2 kq + 1 of the tile
        const float l0 = __shfl_sync(0xffffffffu, l, 8 * kq), l1 = __shfl_sync(0xffffffffu, l, 8 * kq + 4);
        float w[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) w[x] = exp2_fast(fmaf(c0[x] + c1[x], a.scale_log2, -(x & 1 ? l1 : l0)));
        if (t * 8 < full0 || t * 8 + 8 > full1) {
          const int p0 = base + __shfl_sync(0xffffffffu, token, 8 * kq), p1 = base + __shfl_sync(0xffffffffu, token, 8 * kq + 4);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int p = x & 1 ? p1 : p0, j = j0 + quad + (x & 2 ? 8 : 0);
            if (!(p >= 0 && j <= p && (j >= window_first(a, p) || j < a.n_sink)) || t * 8 + 2 * kq + (x & 1) >= R) w[x] = 0.f;
          }
        }
        acc[0] += w[0] + w[1];
        acc[1] += w[2] + w[3];
      }
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      acc[x] += __shfl_xor_sync(0xffffffffu, acc[x], 1);
      acc[x] += __shfl_xor_sync(0xffffffffu, acc[x], 2);
    }
  }
  if (kq == 0) {
    part[warp][quad] = acc[0];
    part[warp][quad + 8] = acc[1];
  }
  if (head_split > 1) __syncthreads(); else __syncwarp();
  const int j = j0 + lane;
  if (warp < tiles && lane < 16 && j < rq.n) {
    float sum = 0.f;
    for (int x = 0; x < head_split; ++x) sum += part[warp + x * tiles][lane];
    const int64_t at = b * A.score_stride + j;
    A.score_out[at] = (A.score_in ? A.decay * A.score_in[at] : 0.f) + sum;
  }
}

static std::string launch_weights(const PagedWeightsArgs &A, int dtype, cudaStream_t s) {
  const PagedArgs &a = A.p;
  // Warps of their own for slot tiles first; while these are fewer than two blocks an SM hold, the KV
  // heads are split (a token at 16 384 slots of one request: 8 heads in one warp 31 us, in eight 13 us).
  int split = 1;
  const int64_t tiles = static_cast<int64_t>(a.n_requests) * ((a.max_len + 15) / 16), want = 2ll * kWeightWarps * num_sms();
  while (split < kWeightWarps && 2 * split <= a.n_kv_heads && tiles * split < want) split *= 2;
  const int per = 16 * kWeightWarps / split;
  const dim3 grid((a.max_len + per - 1) / per, a.n_requests);
  auto go = [&](auto kernel) { return launch_pdl(kernel, grid, dim3(32 * kWeightWarps), 0, s, A, split); };
  cudaError_t e;
  if (dtype == BD_BF16)
    e = a.head_dim == 128 ? go(paged_weights_kernel<__nv_bfloat16, 128>) : go(paged_weights_kernel<__nv_bfloat16, 64>);
  else
    e = a.head_dim == 128 ? go(paged_weights_kernel<__half, 128>) : go(paged_weights_kernel<__half, 64>);
  return e == cudaSuccess ? std::string() : std::string("paged weights: ") + cudaGetErrorString(e);
}

// ------------------------------------------------------------------ eviction
// Order-preserving integer image of a score: NaN as -inf, -0 as +0.
__device__ __forceinline__ uint32_t score_key(float x) {
  if (x != x) x = -INFINITY;
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

constexpr int kSelThreads = 1024;

// One block per request.  The key of the last slot that stays is found by radix selection, eleven,
// eleven and ten bits a pass: a histogram of the slots that match the bits found so far, then the digit
// that holds the wanted rank.  Scores of one magnitude share their leading bits, so lanes with the same
// digit count it together.  Then each warp, over a run of slots of its own, counts what stays -- what is
// larger, and of what is equal the first ones -- and, knowing what stays before its run, places it.
// Bound by the passes over the scores (L2) and the barriers between them.
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;

__global__ void __launch_bounds__(kSelThreads) paged_select_kernel(const __grid_constant__ PagedEvictArgs A) {
  __shared__ int hist[kBins];
  __shared__ int2 warp_cnt[kSelWarps];  // a run's larger and equal slots; those before it
  __shared__ int warp_sum_s[kSelWarps];
  __shared__ uint32_t s_digit;
  __shared__ int s_need;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b = blockIdx.x;
  pdl_wait();
  pdl_trigger();
  const int n = request_len(A.p, b);
  const float *score = A.score + b * A.score_stride;
  float *score_out = A.score_out ? A.score_out + b * A.score_out_stride : nullptr;
  int32_t *kept = A.kept + static_cast<int64_t>(b) * A.budget;
  if (n <= A.budget) {
    for (int j = tid; j < n; j += kSelThreads) {
      kept[j] = j;
      if (score_out && score_out != score) score_out[j] = score[j];
    }
    if (tid == 0) A.len_out[b] = n;
    return;
  }
  // slots [lo, hi) compete for `need` places; those outside stay
  const int lo = A.n_sink, hi = n - A.n_recent;
  int need = A.budget - A.n_sink - A.n_recent;
  const bool none = need == 0;
  uint32_t key = 0xffffffffu;  // key of the last one that stays (none: no score has this one)
  if (!none) {
    uint32_t mask = 0;
    key = 0;
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : 2048;
      for (int d = tid; d < kBins; d += kSelThreads) hist[d] = 0;
      __syncthreads();
#pragma unroll 4
      for (int j0 = lo; j0 < hi; j0 += kSelThreads) {
        const int j = j0 + tid;
        const uint32_t u = j < hi ? score_key(score[j]) : 0u;
        const bool in = j < hi && (u & mask) == key;
        const uint32_t digit = in ? (u >> shift) & (bins - 1) : kBins;
        const unsigned same = __match_any_sync(0xffffffffu, digit);
        if (in && lane == __ffs(same) - 1) atomicAdd(&hist[digit], __popc(same));
      }
      __syncthreads();
      // thread t holds digits bins-1-2t and bins-2-2t, the larger first
      int c[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) c[x] = bins - 1 - 2 * tid - x >= 0 ? hist[bins - 1 - 2 * tid - x] : 0;
      int sum = c[0] + c[1];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += x;
      }
      if (lane == 31) warp_sum_s[warp] = sum;
      __syncthreads();
      int before = lane < warp ? warp_sum_s[lane] : 0;  // 32 warps: a lane each
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
      before += sum - c[0] - c[1];
      if (before < need && before + c[0] + c[1] >= need) {
        const int x = before + c[0] < need;
        s_digit = bins - 1 - 2 * tid - x;
        s_need = need - before - (x ? c[0] : 0);
      }
      __syncthreads();
      key |= s_digit << shift;
      need = s_need;
      mask |= (bins - 1u) << shift;
    }
  }
  // need: how many of the slots whose key is `key` stay (the first ones)
  const int run = (n + kSelThreads - 1) / kSelThreads * 32, j_lo = min(n, warp * run), j_hi = min(n, j_lo + run);
  int2 cnt = make_int2(0, 0);
#pragma unroll 4
  for (int j0 = j_lo; j0 < j_hi; j0 += 32) {
    const int j = j0 + lane;
    const bool in = j < j_hi && j >= lo && j < hi;
    const uint32_t u = in ? score_key(score[j]) : 0u;
    cnt.x += __popc(__ballot_sync(0xffffffffu, j < j_hi && (!in || u > key)));
    cnt.y += __popc(__ballot_sync(0xffffffffu, in && u == key));
  }
  if (lane == 0) warp_cnt[warp] = cnt;
  __syncthreads();
  int2 at = lane < warp ? warp_cnt[lane] : make_int2(0, 0);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    at.x += __shfl_xor_sync(0xffffffffu, at.x, o);
    at.y += __shfl_xor_sync(0xffffffffu, at.y, o);
  }
  int larger = at.x, equal = at.y;  // before this run
  if (none) need = 0;
  const bool in_place = score_out == score;
#pragma unroll 1
  for (int x = 0; x < run; x += 32) {
    const int j = j_lo + x + lane;
    const bool here = j < j_hi, in = here && j >= lo && j < hi;
    const float v = here ? score[j] : 0.f;
    const uint32_t u = in ? score_key(v) : 0u;
    const unsigned below = (1u << lane) - 1;
    const unsigned gt = __ballot_sync(0xffffffffu, here && (!in || u > key)), eq = __ballot_sync(0xffffffffu, in && u == key);
    const int e = equal + __popc(eq & below), place = larger + __popc(gt & below) + min(e, need);
    const bool keep = here && (!in || u > key || (u == key && e < need));
    larger += __popc(gt);
    equal += __popc(eq);
    if (keep) {
      kept[place] = j;
      if (score_out && !in_place) score_out[place] = v;
    }
  }
  if (in_place) {
    // score i comes from kept[i] >= i: a block of them is written when all of it has been read, and the
    // blocks behind it read behind what it wrote
    __syncthreads();
    for (int i0 = 0; i0 < n; i0 += kSelThreads) {
      const int i = i0 + tid;
      const float v = i < A.budget ? score[kept[i]] : 0.f;
      __syncthreads();
      if (i < n) score_out[i] = v;  // behind the kept ones zero: slots filled later start from there
    }
  }
  if (tid == 0) A.len_out[b] = A.budget;
}

// Moves the kept slots.  Slot i's row of one pool and KV head is D contiguous values; a thread
// moves 16 bytes of it.  To other pages every block takes kMoveRows slots of its own, each thread its
// pieces side by side: slot, page and piece are three round trips, whatever their number.
constexpr int kMoveThreads = 256;
constexpr int kMoveEach = 8;  // 16-byte pieces of a thread

__device__ __forceinline__ int64_t dst_offset(const PagedEvictArgs &A, int b, int i) {
  if (!A.dst_table) return slot_offset(A.p, A.p.page_table + static_cast<int64_t>(b) * A.p.table_width, i);
  return slot_offset(A.p, A.dst_table + static_cast<int64_t>(b) * A.dst_width, i);
}

template <int CPR>  // pieces of a row
__global__ void __launch_bounds__(kMoveThreads) paged_move_kernel(const __grid_constant__ PagedEvictArgs A) {
  const PagedArgs &a = A.p;
  const int b = blockIdx.z, h = blockIdx.y >> 1;
  uint16_t *pool = static_cast<uint16_t *>(const_cast<void *>(blockIdx.y & 1 ? a.v : a.k)) + h * a.head_stride;
  pdl_wait();
  pdl_trigger();
  const int n = min(A.len_out[b], A.budget);
  const int32_t *kept = A.kept + static_cast<int64_t>(b) * A.budget;
  const int32_t *table = a.page_table + static_cast<int64_t>(b) * a.table_width;
  constexpr int STEP = kMoveThreads / CPR;
  const int i0 = blockIdx.x * STEP * kMoveEach + threadIdx.x / CPR, x = (threadIdx.x % CPR) * 8;
  if (blockIdx.x * STEP * kMoveEach >= n) return;
  int j[kMoveEach];
#pragma unroll
  for (int u = 0; u < kMoveEach; ++u) j[u] = kept[min(i0 + u * STEP, n - 1)];
  int64_t src[kMoveEach], dst[kMoveEach];
#pragma unroll
  for (int u = 0; u < kMoveEach; ++u) {
    src[u] = slot_offset(a, table, j[u]);
    dst[u] = i0 + u * STEP < n ? dst_offset(A, b, i0 + u * STEP) : -1;
  }
  uint4 v[kMoveEach];
#pragma unroll
  for (int u = 0; u < kMoveEach; ++u)
    if (src[u] >= 0 && dst[u] >= 0) v[u] = *reinterpret_cast<const uint4 *>(pool + src[u] + x);
#pragma unroll
  for (int u = 0; u < kMoveEach; ++u)
    if (src[u] >= 0 && dst[u] >= 0) *reinterpret_cast<uint4 *>(pool + dst[u] + x) = v[u];
}

// In place, one block per (request, KV head, pool) goes up through the slots in chunks of
// kChunkRows.  Slot i comes from old slot kept[i] >= i, so a chunk's writes can only hit rows that
// this chunk or an earlier one reads: a chunk is written after all of it has been read, and the
// next chunk's reads may go ahead of it.
constexpr int kInThreads = 512;
constexpr int kInRegs = 8;  // 16-byte pieces of a chunk per thread

__global__ void __launch_bounds__(kInThreads) paged_move_in_place_kernel(const __grid_constant__ PagedEvictArgs A) {
  const PagedArgs &a = A.p;
  const int b = blockIdx.y, h = blockIdx.x >> 1;
  uint16_t *pool = static_cast<uint16_t *>(const_cast<void *>(blockIdx.x & 1 ? a.v : a.k)) + h * a.head_stride;
  const int cpr = a.head_dim / 8;
  const int chunk = kInThreads * kInRegs / cpr;  // rows
  pdl_wait();
  pdl_trigger();
  const int n = min(A.len_out[b], A.budget);
  const int32_t *kept = A.kept + static_cast<int64_t>(b) * A.budget;
  const int32_t *table = a.page_table + static_cast<int64_t>(b) * a.table_width;
  for (int i0 = 0; i0 < n; i0 += chunk) {
    uint4 v[kInRegs];
    int64_t dst[kInRegs];
#pragma unroll
    for (int u = 0; u < kInRegs; ++u) {
      const int c = u * kInThreads + threadIdx.x, i = i0 + c / cpr, x = (c % cpr) * 8;
      dst[u] = -1;
      if (i < n) {
        const int j = kept[i];
        if (j != i) {
          const int64_t src = slot_offset(a, table, j), d = slot_offset(a, table, i);
          if (src >= 0 && d >= 0) {
            dst[u] = d + x;
            v[u] = *reinterpret_cast<const uint4 *>(pool + src + x);
          }
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kInRegs; ++u)
      if (dst[u] >= 0) *reinterpret_cast<uint4 *>(pool + dst[u]) = v[u];
  }
}

static std::string launch_evict(const PagedEvictArgs &A, cudaStream_t s) {
  const PagedArgs &a = A.p;
  cudaError_t e = launch_pdl(paged_select_kernel, dim3(a.n_requests), dim3(kSelThreads), 0, s, A);
  if (e == cudaSuccess) {
    const int most = A.budget < a.max_len ? A.budget : a.max_len;
    if (A.dst_table) {
      const int rows = kMoveThreads * kMoveEach / (a.head_dim / 8);  // of a block
      const dim3 grid((most + rows - 1) / rows, 2 * a.n_kv_heads, a.n_requests);
      if (most > 0) e = launch_pdl(a.head_dim == 128 ? paged_move_kernel<16> : paged_move_kernel<8>, grid, dim3(kMoveThreads), 0, s, A);
    } else if (A.budget < a.max_len) {  // else nothing can leave
      e = launch_pdl(paged_move_in_place_kernel, dim3(2 * a.n_kv_heads, a.n_requests), dim3(kInThreads), 0, s, A);
    }
  }
  return e == cudaSuccess ? std::string() : std::string("paged eviction: ") + cudaGetErrorString(e);
}

// ------------------------------------------------------------------ host checks
namespace {

bd_status refuse(bd_status st, const std::string &msg) {
  set_last_error(msg);
  return st;
}
bool misaligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

// Whether [p, p + np) and [q, q + nq) (bytes) share any.
bool overlap(const void *p, int64_t np, const void *q, int64_t nq) {
  const char *a = static_cast<const char *>(p), *b = static_cast<const char *>(q);
  return np > 0 && nq > 0 && a < b + nq && b < a + np;
}

bd_status check_kv(const bd_paged_kv *c) {
  if (!c) return refuse(BD_ERR_INVALID_ARG, "paged kv is NULL");
  if (c->dtype != BD_BF16 && c->dtype != BD_F16)
    return refuse(BD_ERR_UNSUPPORTED, "paged kv: dtype must be BD_BF16 or BD_F16");
  if (c->head_dim != 64 && c->head_dim != 128) return refuse(BD_ERR_UNSUPPORTED, "paged kv: head_dim must be 64 or 128");
  if (c->n_kv_heads <= 0 || c->n_q_heads <= 0 || c->n_q_heads % c->n_kv_heads != 0)
    return refuse(BD_ERR_INVALID_ARG, "paged kv: n_q_heads must be a positive multiple of n_kv_heads");
  if (c->n_q_heads / c->n_kv_heads > BD_PAGED_MAX_GROUP || c->n_kv_heads > 1024)
    return refuse(BD_ERR_UNSUPPORTED, "paged kv: at most 128 query heads per KV head and 1024 KV heads");
  if (c->page_size < 1 || c->n_pages < 1) return refuse(BD_ERR_INVALID_ARG, "paged kv: page_size and n_pages must be >= 1");
  if (!c->k || !c->v || misaligned(c->k, 16) || misaligned(c->v, 16))
    return refuse(BD_ERR_INVALID_ARG, "paged kv: k and v must be 16-byte aligned pools");
  for (int64_t s : {c->page_stride, c->head_stride, c->slot_stride})
    if (s < 0 || s % 8) return refuse(BD_ERR_INVALID_ARG, "paged kv: strides must be multiples of 8 elements, >= 0");
  if ((c->page_size > 1 && c->slot_stride < c->head_dim) || (c->n_kv_heads > 1 && c->head_stride < c->head_dim) ||
      (c->n_pages > 1 && c->page_stride < c->head_dim))
    return refuse(BD_ERR_INVALID_ARG, "paged kv: strides must be at least head_dim elements");
  return BD_OK;
}

bd_status check_batch(const bd_paged_kv *c, const bd_paged_batch *t, bool rows) {
  if (bd_status st = check_kv(c)) return st;
  if (!t) return refuse(BD_ERR_INVALID_ARG, "paged batch is NULL");
  if (t->n_requests < 1 || t->n_requests > BD_PAGED_MAX_REQUESTS)
    return refuse(BD_ERR_INVALID_ARG, "paged batch: n_requests must be in 1..1024");
  if (t->table_width < 1 || t->max_len < 0 ||
      t->max_len > static_cast<int64_t>(t->table_width) * c->page_size || t->max_len > (1 << 30))
    return refuse(BD_ERR_INVALID_ARG, "paged batch: max_len must be within table_width * page_size (and 2^30)");
  if (!t->page_table || !t->seq_len || misaligned(t->page_table, 4) || misaligned(t->seq_len, 4))
    return refuse(BD_ERR_INVALID_ARG, "paged batch: page_table and seq_len must be given");
  if (rows) {
    if (!t->row_start || misaligned(t->row_start, 4)) return refuse(BD_ERR_INVALID_ARG, "paged batch: row_start must be given");
    if (t->n_rows < 0 || t->max_rows < 0 || t->max_rows > t->n_rows || t->n_rows > (1 << 28))
      return refuse(BD_ERR_INVALID_ARG, "paged batch: 0 <= max_rows <= n_rows <= 2^28");
  }
  return BD_OK;
}

bd_status check_rows(const void *p, int64_t stride, int64_t width, int n_rows, const char *name) {
  if (!p || misaligned(p, 16) || stride % 8 || (n_rows > 1 && stride < width))
    return refuse(BD_ERR_INVALID_ARG, std::string("paged cache: ") + name +
                                          " must be 16-byte aligned rows with a stride that is a multiple of 8 and holds a row");
  return BD_OK;
}
int64_t row_bytes(int64_t stride, int64_t width, int n_rows) {
  return n_rows < 1 ? 0 : ((n_rows - 1) * stride + width) * 2;
}

bd_status check_mask(int window, int n_sink, float scale) {
  if (window < 0 || n_sink < 0) return refuse(BD_ERR_INVALID_ARG, "paged attention: window and n_sink must be >= 0");
  if (!(scale > 0.f) || !std::isfinite(scale)) return refuse(BD_ERR_INVALID_ARG, "paged attention: scale must be > 0 and finite");
  return BD_OK;
}

PagedArgs args_of(const bd_paged_kv *c, const bd_paged_batch *t) {
  PagedArgs a = {};
  a.k = c->k;
  a.v = c->v;
  a.page_stride = c->page_stride;
  a.head_stride = c->head_stride;
  a.slot_stride = c->slot_stride;
  a.n_kv_heads = c->n_kv_heads;
  a.group = c->n_q_heads / c->n_kv_heads;
  a.head_dim = c->head_dim;
  a.page_size = c->page_size;
  a.n_pages = c->n_pages;
  a.n_requests = t->n_requests;
  a.table_width = t->table_width;
  a.n_rows = t->n_rows;
  a.max_rows = t->max_rows;
  a.max_len = t->max_len;
  a.page_table = t->page_table;
  a.seq_len = t->seq_len;
  a.row_start = t->row_start;
  return a;
}
bd_status ran(const std::string &e) { return e.empty() ? BD_OK : refuse(BD_ERR_CUDA, e); }

}  // namespace
}  // namespace bd

using namespace bd;

extern "C" {

size_t bd_paged_workspace_bytes(const bd_paged_kv *kv, int n_requests, int max_rows) {
  if (check_kv(kv)) return 0;
  if (n_requests < 1 || n_requests > BD_PAGED_MAX_REQUESTS || max_rows < 0) {
    refuse(BD_ERR_INVALID_ARG, "paged workspace: n_requests must be in 1..1024 and max_rows >= 0");
    return 0;
  }
  // a batch made for many rows may hold few (and the other way round): the larger of the two
  const size_t few = few_bytes(kv->head_dim);
  const size_t many = many_bytes(n_requests, max_rows, kv->n_q_heads / kv->n_kv_heads, kv->head_dim);
  return few > many ? few : many;
}

bd_status bd_paged_append(const bd_paged_kv *kv, const bd_paged_batch *batch, const void *k_new, int64_t k_stride,
                          const void *v_new, int64_t v_stride, void *stream) {
  if (bd_status st = check_batch(kv, batch, true)) return st;
  if (batch->n_rows == 0) return BD_OK;
  const int64_t width = static_cast<int64_t>(kv->n_kv_heads) * kv->head_dim;
  if (bd_status st = check_rows(k_new, k_stride, width, batch->n_rows, "k_new")) return st;
  if (bd_status st = check_rows(v_new, v_stride, width, batch->n_rows, "v_new")) return st;
  PagedAppendArgs A = {};
  A.p = args_of(kv, batch);
  A.k_new = k_new;
  A.v_new = v_new;
  A.k_stride = k_stride;
  A.v_stride = v_stride;
  return ran(launch_append(A, static_cast<cudaStream_t>(stream)));
}

bd_status bd_paged_attention(const bd_paged_kv *kv, const bd_paged_batch *batch, const void *q, int64_t q_stride, void *out,
                             int64_t out_stride, float *lse, int window, int n_sink, float scale, void *workspace,
                             size_t workspace_bytes, void *stream) {
  if (bd_status st = check_batch(kv, batch, true)) return st;
  if (bd_status st = check_mask(window, n_sink, scale)) return st;
  if (batch->max_rows == 0) return BD_OK;
  const int64_t width = static_cast<int64_t>(kv->n_q_heads) * kv->head_dim;
  if (bd_status st = check_rows(q, q_stride, width, batch->n_rows, "q")) return st;
  if (bd_status st = check_rows(out, out_stride, width, batch->n_rows, "out")) return st;
  if (overlap(q, row_bytes(q_stride, width, batch->n_rows), out, row_bytes(out_stride, width, batch->n_rows)))
    return refuse(BD_ERR_INVALID_ARG, "paged attention: q and out overlap");
  if (misaligned(lse, 4)) return refuse(BD_ERR_INVALID_ARG, "paged attention: lse misaligned");
  if ((static_cast<int64_t>(batch->max_len) / 16 + 8) * kv->n_kv_heads >= (1ll << 31) ||
      static_cast<int64_t>(batch->max_rows) * kv->n_q_heads > (1 << 30))
    return refuse(BD_ERR_UNSUPPORTED, "paged attention: max_len * n_kv_heads or max_rows * n_q_heads too large");
  if (!workspace || misaligned(workspace, 256) ||
      workspace_bytes < bd_paged_workspace_bytes(kv, batch->n_requests, batch->max_rows))
    return refuse(BD_ERR_WORKSPACE, "paged attention: workspace NULL, not 256-byte aligned or too small");
  PagedAttnArgs A = {};
  A.p = args_of(kv, batch);
  A.p.q = q;
  A.p.q_stride = q_stride;
  A.p.window = window;
  A.p.n_sink = n_sink;
  A.p.scale_log2 = static_cast<float>(scale * 1.4426950408889634);
  A.out = out;
  A.out_stride = out_stride;
  A.lse = lse;
  const bool few = static_cast<int64_t>(batch->max_rows) * A.p.group <= kFewRows;
  return ran((few ? launch_attention_few : launch_attention_many)(A, workspace, kv->dtype, static_cast<cudaStream_t>(stream)));
}

bd_status bd_paged_weights(const bd_paged_kv *kv, const bd_paged_batch *batch, const void *q, int64_t q_stride,
                           const float *lse, const int32_t *rows_used, int window, int n_sink, float scale, float decay,
                           const float *score_in, float *score_out, int64_t score_stride, void *stream) {
  if (bd_status st = check_batch(kv, batch, true)) return st;
  if (bd_status st = check_mask(window, n_sink, scale)) return st;
  if (batch->max_len == 0) return BD_OK;
  const int64_t width = static_cast<int64_t>(kv->n_q_heads) * kv->head_dim;
  if (batch->max_rows > 0) {
    if (bd_status st = check_rows(q, q_stride, width, batch->n_rows, "q")) return st;
    if (!lse || misaligned(lse, 4)) return refuse(BD_ERR_INVALID_ARG, "paged weights: lse must be given");
  }
  if (misaligned(rows_used, 4)) return refuse(BD_ERR_INVALID_ARG, "paged weights: rows_used misaligned");
  if (static_cast<int64_t>(batch->max_rows) * kv->n_q_heads > (1 << 30))
    return refuse(BD_ERR_UNSUPPORTED, "paged weights: max_rows * n_q_heads too large");
  if (!std::isfinite(decay)) return refuse(BD_ERR_INVALID_ARG, "paged weights: decay must be finite");
  if (!score_out || misaligned(score_out, 4) || misaligned(score_in, 4) || score_stride < batch->max_len)
    return refuse(BD_ERR_INVALID_ARG, "paged weights: score_out must be given, with rows of at least max_len entries");
  const int64_t bytes = ((batch->n_requests - 1) * score_stride + batch->max_len) * 4;
  if (score_in && score_in != score_out && overlap(score_in, bytes, score_out, bytes))
    return refuse(BD_ERR_INVALID_ARG, "paged weights: score_in must be score_out or not overlap it");
  PagedWeightsArgs A = {};
  A.p = args_of(kv, batch);
  A.p.q = q;
  A.p.q_stride = q_stride;
  A.p.window = window;
  A.p.n_sink = n_sink;
  A.p.scale_log2 = static_cast<float>(scale * 1.4426950408889634);
  A.lse = lse;
  A.rows_used = rows_used;
  A.decay = decay;
  A.score_in = score_in;
  A.score_out = score_out;
  A.score_stride = score_stride;
  return ran(launch_weights(A, kv->dtype, static_cast<cudaStream_t>(stream)));
}

bd_status bd_paged_evict(const bd_paged_kv *kv, const bd_paged_batch *batch, const float *score, int64_t score_stride,
                         int budget, int n_sink, int n_recent, const int32_t *dst_table, int dst_width, int32_t *kept_out,
                         int32_t *len_out, float *score_out, int64_t score_out_stride, void *stream) {
  if (bd_status st = check_batch(kv, batch, false)) return st;
  if (budget < 1 || n_sink < 0 || n_recent < 0 || static_cast<int64_t>(n_sink) + n_recent > budget)
    return refuse(BD_ERR_INVALID_ARG, "paged eviction: budget must be >= 1 and hold n_sink + n_recent");
  const int most = budget < batch->max_len ? budget : batch->max_len;
  if (!score || misaligned(score, 4) || score_stride < batch->max_len)
    return refuse(BD_ERR_INVALID_ARG, "paged eviction: score must be given, with rows of at least max_len entries");
  if (!kept_out || !len_out || misaligned(kept_out, 4) || misaligned(len_out, 4))
    return refuse(BD_ERR_INVALID_ARG, "paged eviction: kept_out and len_out must be given");
  if (dst_table && (misaligned(dst_table, 4) || dst_width < 1 || static_cast<int64_t>(dst_width) * kv->page_size < most))
    return refuse(BD_ERR_INVALID_ARG, "paged eviction: dst_table's rows must hold min(budget, max_len) slots");
  if (dst_table == batch->page_table && dst_table)
    return refuse(BD_ERR_INVALID_ARG, "paged eviction: dst_table is page_table (NULL moves in place)");
  if (score_out) {
    if (misaligned(score_out, 4) || score_out_stride < most)
      return refuse(BD_ERR_INVALID_ARG, "paged eviction: score_out's rows must hold min(budget, max_len) entries");
    const int64_t in = ((batch->n_requests - 1) * score_stride + batch->max_len) * 4;
    const int64_t out = ((batch->n_requests - 1) * score_out_stride + most) * 4;
    if (score_out == score ? score_out_stride != score_stride : overlap(score, in, score_out, out))
      return refuse(BD_ERR_INVALID_ARG, "paged eviction: score_out must be score (same stride) or not overlap it");
  }
  PagedEvictArgs A = {};
  A.p = args_of(kv, batch);
  A.score = score;
  A.score_stride = score_stride;
  A.budget = budget;
  A.n_sink = n_sink;
  A.n_recent = n_recent;
  A.dst_table = dst_table;
  A.dst_width = dst_width;
  A.kept = kept_out;
  A.len_out = len_out;
  A.score_out = score_out;
  A.score_out_stride = score_out_stride;
  return ran(launch_evict(A, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
