// Attention of many rows (bd_paged_attention with more than kFewRows rows of a KV head: longer
// blocks, wide head groups, prompt chunks) on the tensor cores.
//
// An item is kItemRows = 256 rows of one KV head (row = token * group + head in the group), as two
// MMA tiles of 128; its keys come in tiles of 128 slots.  Per tile and 128 rows
//   S = Q K^T  (fp32, 128 TMEM columns),  P = 2^(scale log2(e) S - ref)  (16 bits, TMEM),  O += P V
// with the softmax's running reference and sum in the row's own thread.  Bound by the tensor cores
// for long chunks (4 * 128 * 128 * D flops a tile and stream), by the K/V bytes for blocks.
//   warps 0-3, 4-7  softmax of stream 0 and 1, one row a thread: S from TMEM, P back to TMEM (the
//                   second product takes it from there as its A operand), results at the end
//   warp 8          one thread issues the MMAs
//   warps 10, 11    copy K and V rows with cp.async into a ring of shared-memory tiles; slots lie in
//                   pages of any size, so every row has its own address, and a row that nobody sees
//                   becomes zero
// While one stream's softmax works, the tensor cores run the other stream's products.  An item of
// more than 128 rows gives each stream 128 of them; a smaller one gives the streams every other key
// tile of the same rows, joined at the end through TMEM.
//
// A call's units (key tiles of all items) are split evenly over one block an SM whatever lengths and
// masks are: attention_plan counts them, attention_many works, attention_join_many joins the items
// that were split.  The reference of a row moves only when a score exceeds it by more than 2^8, so
// sums are rarely rescaled; weights round to 16 bits (2^-9 relative), as the result does.
#include "bd_paged_attn.cuh"

#include <atomic>
#include <type_traits>

namespace bd {

BD_DEFINE_ERROR_TAKER(take_error_word_paged_tc)

namespace {

constexpr int kItemRows = 256;
constexpr int kTileSlots = 128;
constexpr int kTcThreads = 384;
constexpr int kLoaderThreads = 64;
// Registers a thread: the softmax warpgroups take what the third one gives up.  The sum may not
// exceed what the block starts with (checked at the first launch).
constexpr int kRegsSoftmax = 208, kRegsOther = 88;
constexpr uint32_t kAtom = 16384;  // 128 rows x 128 bytes, 128-byte swizzled
constexpr int kLag = 2;            // copy groups in flight behind the one just issued

template <int D> struct Tc {
  static constexpr uint32_t kTile = (D / 64) * kAtom;      // 128 rows of D values
  static constexpr int kSlots = D == 128 ? 5 : 8;          // ring tiles
  static constexpr uint32_t kOffRing = 2 * kTile;          // behind the two query tiles
  static constexpr uint32_t kOffBar = kOffRing + kSlots * kTile;
  static constexpr size_t kSmem = 1024 + kOffBar + 256;
  // TMEM columns of stream s.  With D = 128 the weights take the place of their scores: the products
  // have one shape, so the next scores are written after the weights have been read.
  static constexpr uint32_t kS = 0, kO = 256, kP = D == 128 ? 0 : 384;
  static constexpr uint32_t kStepS = 128, kStepO = D, kStepP = D == 128 ? 128 : 64;
};
// Weights are formed against 2^-kHead of the reference: fp16 keeps small ones above its subnormals
// and, with the reference at most 2^8 behind, the largest below 2^15.
template <typename T> struct Head { static constexpr float k = 0.f; };
template <> struct Head<__half> { static constexpr float k = 6.f; };
constexpr float kMove = 8.f;

template <typename T> constexpr uint32_t ab_format() { return std::is_same<T, __half>::value ? 0u : 1u; }

// A from TMEM, B from shared memory.
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Key tiles of one item: those of the sinks, then those from its first row's window on.
struct ItemTiles {
  int sinks, first, count;
  __device__ int at(int t) const { return t < sinks ? t : first + t - sinks; }
};
__device__ __forceinline__ ItemTiles item_tiles(const PagedArgs &a, const Request &rq, int qt) {
  ItemTiles t = {0, 0, 0};
  const int64_t r0 = static_cast<int64_t>(qt) * kItemRows, R = static_cast<int64_t>(rq.rows) * a.group;
  if (r0 >= R) return t;
  const int base = rq.n - rq.rows;
  const int p_high = base + static_cast<int>(((r0 + kItemRows < R ? r0 + kItemRows : R) - 1) / a.group);
  if (p_high < 0) return t;
  const int first = window_first(a, max(0, base + static_cast<int>(r0 / a.group)));
  t.first = first / kTileSlots;
  t.sinks = min((min(a.n_sink, first) + kTileSlots - 1) / kTileSlots, t.first);
  t.count = t.sinks + p_high / kTileSlots + 1 - t.first;
  return t;
}
__device__ __forceinline__ int many_ctas_used(int64_t units, int most) {
  return static_cast<int>(units < 1 ? 1 : units < most ? units : most);
}

// ------------------------------------------------------------------ plan
// unit_start[i] = units before item list entry i = b * nqt + qt (every KV head of it), and the entry
// each block's share begins in.  One block.
constexpr int kPlanThreads = 1024;
__global__ void __launch_bounds__(kPlanThreads) attention_plan(const __grid_constant__ PagedAttnArgs A, int nqt) {
  __shared__ int64_t warp_total[kPlanThreads / 32];
  const PagedArgs &a = A.p;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int N = a.n_requests * nqt;
  pdl_wait();
  pdl_trigger();
  int64_t base = 0;
  for (int i0 = 0; i0 < N; i0 += kPlanThreads) {
    const int i = i0 + tid;
    int64_t x = 0;
    if (i < N) {
      const int b = i / nqt;
      x = static_cast<int64_t>(item_tiles(a, request_of(a, b), i - b * nqt).count) * a.n_kv_heads;
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) warp_total[warp] = x;
    __syncthreads();
    int64_t t = warp_total[lane];  // 32 warps
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += y;
    }
    const int64_t before = __shfl_sync(0xffffffffu, t, warp > 0 ? warp - 1 : 0);
    if (i < N) A.unit_start[i + 1] = base + x + (warp > 0 ? before : 0);
    base += __shfl_sync(0xffffffffu, t, 31);
    __syncthreads();
  }
  if (tid == 0) A.unit_start[0] = 0;
  __syncthreads();
  const int64_t units = base;
  const int ctas = many_ctas_used(units, A.n_ctas);
  for (int i = tid; i < N; i += kPlanThreads) {
    const int64_t s = A.unit_start[i], e = A.unit_start[i + 1];
    if (s == e) continue;
    int g = static_cast<int>(s * ctas / units);
    while (share_begin(units, ctas, g) < s) ++g;
    for (; g < ctas && share_begin(units, ctas, g) < e; ++g) A.cta_item[g] = i;
  }
}

// ------------------------------------------------------------------ the block's segments
// A segment: tiles [t0, t1) of one item and KV head.
struct Segment {
  Request rq;
  ItemTiles tl;
  int b, h, qt, t0, t1;
  bool whole, split;  // split: at most 128 rows, the streams share them
  int64_t u;          // first unit
};
struct Walk {
  int64_t u, end;
  int i;
  __device__ Walk(const PagedAttnArgs &A, int64_t units, int ctas) {
    u = share_begin(units, ctas, blockIdx.x);
    end = share_begin(units, ctas, blockIdx.x + 1);
    i = A.cta_item[blockIdx.x];
  }
  __device__ bool next(const PagedAttnArgs &A, int nqt, Segment &s) {
    if (u >= end) return false;
    while (A.unit_start[i + 1] <= u) ++i;
    const PagedArgs &a = A.p;
    s.b = i / nqt;
    s.qt = i - s.b * nqt;
    s.rq = request_of(a, s.b);
    s.tl = item_tiles(a, s.rq, s.qt);
    const int64_t in = u - A.unit_start[i];
    s.h = static_cast<int>(in / s.tl.count);
    s.t0 = static_cast<int>(in - static_cast<int64_t>(s.h) * s.tl.count);
    s.t1 = static_cast<int>(end - u < s.tl.count - s.t0 ? s.t0 + (end - u) : s.tl.count);
    s.whole = s.t0 == 0 && s.t1 == s.tl.count;
    s.split = static_cast<int64_t>(s.rq.rows) * a.group - static_cast<int64_t>(s.qt) * kItemRows <= 128;
    s.u = u;
    u += s.t1 - s.t0;
    return true;
  }
};

struct Bars {
  uint64_t *full, *empty;                    // ring tiles
  uint64_t *s_full, *p_full, *o_full, *q_full;  // of each stream
  volatile int *stop;                        // a wait gave up: every role ends
};

__device__ __forceinline__ bool wait_or_stop(const Bars &B, uint64_t *bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  if (!*B.stop && mbar_wait(bar, parity)) return true;
  *B.stop = 1;
  return false;
}
__device__ __forceinline__ bool wait_warp(const Bars &B, uint64_t *bar, uint32_t parity) {
  return __all_sync(0xffffffffu, wait_or_stop(B, bar, parity));
}

// ------------------------------------------------------------------ copies
// Warp w of the two copies rows 64w .. 64w+63 of every tile; lane l holds the places of rows 64w + l
// and 64w + 32 + l.  Copies are announced kLag groups later, when they have landed: the writing threads
// order them before the tensor cores' reads (async proxy) and arrive.
template <typename T, int D>
__device__ void load_role(const PagedAttnArgs &A, int nqt, int64_t units, int ctas, uint32_t ring, const Bars &B, int warp, int lane) {
  constexpr uint32_t NS = Tc<D>::kSlots;
  constexpr int CPR = D / 8, RPI = 32 / CPR;
  const PagedArgs &a = A.p;
  Walk walk(A, units, ctas);
  Segment s;
  uint32_t q = 0;  // copy groups issued
  auto announce = [&](uint32_t g) {
    fence_proxy_async_shared();
    mbar_arrive(&B.full[g % NS]);
  };
  while (walk.next(A, nqt, s)) {
    const int32_t *table = a.page_table + static_cast<int64_t>(s.b) * a.table_width;
    const int64_t head_off = static_cast<int64_t>(s.h) * a.head_stride;
    const T *K = static_cast<const T *>(a.k) + head_off, *V = static_cast<const T *>(a.v) + head_off;
    const int64_t r0 = static_cast<int64_t>(s.qt) * kItemRows, R = static_cast<int64_t>(s.rq.rows) * a.group;
    const int base = s.rq.n - s.rq.rows;
    const int f_low = window_first(a, max(0, base + static_cast<int>(r0 / a.group)));
    const int p_high = base + static_cast<int>(((r0 + kItemRows < R ? r0 + kItemRows : R) - 1) / a.group);
    auto slot_of = [&](int t, int k) { return s.tl.at(min(t, s.t1 - 1)) * kTileSlots + warp * 64 + k * 32 + lane; };
    auto page_at = [&](int t, int k) { return __ldg(table + min(slot_of(t, k), p_high) / a.page_size); };
    int page[2] = {page_at(s.t0, 0), page_at(s.t0, 1)};
    for (int t = s.t0; t < s.t1; ++t) {
      int64_t off[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int j = slot_of(t, k);
        off[k] = j <= p_high && (j >= f_low || j < a.n_sink) ? page_offset(a, page[k], j) : -1;
      }
      page[0] = page_at(t + 1, 0);
      page[1] = page_at(t + 1, 1);
#pragma unroll 1
      for (int v = 0; v < 2; ++v) {
        const uint32_t slot = q % NS;
        if (q >= NS && !wait_warp(B, &B.empty[slot], ((q / NS) - 1) & 1)) {
          cp_async_wait<0>();
          return;
        }
        const T *src = v ? V : K;
        const int c = lane % CPR;
        const uint32_t dst = ring + slot * Tc<D>::kTile + (c >> 3) * kAtom;
#pragma unroll
        for (int u = 0; u < 64 / RPI; ++u) {
          const int rl = u * RPI + lane / CPR, r = warp * 64 + rl;
          const int64_t ro = __shfl_sync(0xffffffffu, off[u * RPI / 32], rl & 31);
          cp_async16(dst + r * 128 + (((c & 7) ^ (r & 7)) << 4), src + (ro < 0 ? 0 : ro + c * 8), ro >= 0);
        }
        cp_async_commit();
        ++q;
        if (q > kLag) {
          cp_async_wait<kLag>();
          announce(q - 1 - kLag);
        }
      }
    }
  }
  cp_async_wait<0>();
  for (uint32_t g = q > kLag ? q - kLag : 0; g < q; ++g) announce(g);
}

// ------------------------------------------------------------------ products (one thread)
template <typename T, int D>
__device__ void mma_role(const PagedAttnArgs &A, int nqt, int64_t units, int ctas, uint32_t sm, const Bars &B, uint32_t tmem) {
  using C = Tc<D>;
  constexpr uint32_t NS = C::kSlots;
  const uint32_t idesc_s = umma_idesc(ab_format<T>(), 128, kTileSlots);
  const uint32_t idesc_o = umma_idesc(ab_format<T>(), 128, D) | (1u << 16);  // V: N-major
  const uint32_t ring = sm + C::kOffRing;
  uint32_t base = 0;           // ring group of the segment's first key tile
  uint32_t n_p[2] = {0, 0}, n_q[2] = {0, 0};
  auto ready = [&](uint32_t g) {
    const bool ok = wait_or_stop(B, &B.full[g % NS], (g / NS) & 1);
    tc_fence_after();
    return ok;
  };
  auto scores = [&](int s, int qtile, uint32_t g) {
    const uint32_t qb = sm + qtile * C::kTile, kb = ring + (g % NS) * C::kTile;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      const uint32_t off = (kk >> 2) * kAtom + (kk & 3) * 32;
      umma_bf16(tmem + C::kS + s * C::kStepS, umma_desc_sw128(qb + off), umma_desc_sw128(kb + off), idesc_s, kk > 0);
    }
    umma_commit(&B.s_full[s]);
  };
  auto values = [&](int s, uint32_t g, bool add) {
    const uint32_t vb = ring + (g % NS) * C::kTile;
#pragma unroll
    for (int kk = 0; kk < kTileSlots / 16; ++kk)
      umma_ts(tmem + C::kO + s * C::kStepO, tmem + C::kP + s * C::kStepP + kk * 8,
              umma_desc_sw128_mn(vb + kk * 2048, kAtom, 1024), idesc_o, add || kk > 0);
  };
  auto weights = [&](int s) {
    const bool ok = wait_or_stop(B, &B.p_full[s], n_p[s]++ & 1);
    tc_fence_after();
    return ok;
  };
  Walk walk(A, units, ctas);
  Segment g;
  while (walk.next(A, nqt, g)) {
    const int nt = g.t1 - g.t0;
    if (!wait_or_stop(B, &B.q_full[0], n_q[0]++ & 1)) return;
    if (!g.split && !wait_or_stop(B, &B.q_full[1], n_q[1]++ & 1)) return;
    tc_fence_after();
    if (!g.split) {  // both streams take every tile
      if (!ready(base)) return;
      scores(0, 0, base);
      scores(1, 1, base);
      umma_commit(&B.empty[base % NS]);
      for (int t = 0; t < nt; ++t) {
        const uint32_t gv = base + 2 * t + 1, gk = gv + 1;
        if (!ready(gv) || !weights(0)) return;
        values(0, gv, t > 0);
        if (t + 1 < nt) {
          if (!ready(gk)) return;
          scores(0, 0, gk);
        } else {
          umma_commit(&B.o_full[0]);
        }
        if (!weights(1)) return;
        values(1, gv, t > 0);
        umma_commit(&B.empty[gv % NS]);
        if (t + 1 < nt) {
          scores(1, 1, gk);
          umma_commit(&B.empty[gk % NS]);
        } else {
          umma_commit(&B.o_full[1]);
        }
      }
    } else {  // stream t % 2 takes tile t
      for (int t = 0; t < 2 && t < nt; ++t) {
        if (!ready(base + 2 * t)) return;
        scores(t, 0, base + 2 * t);
        umma_commit(&B.empty[(base + 2 * t) % NS]);
      }
      for (int t = 0; t < nt; ++t) {
        const uint32_t gv = base + 2 * t + 1, gk = base + 2 * t + 4;
        const int s = t & 1;
        if (!ready(gv) || !weights(s)) return;
        values(s, gv, t > 1);
        umma_commit(&B.empty[gv % NS]);
        if (t + 2 < nt) {
          if (!ready(gk)) return;
          scores(s, 0, gk);
          umma_commit(&B.empty[gk % NS]);
        } else {
          umma_commit(&B.o_full[s]);
        }
      }
    }
    base += 2 * nt;
  }
}

// ------------------------------------------------------------------ softmax and results
constexpr int kBarBoth = 1;  // named barrier of the two softmax warpgroups

template <typename T, int D>
__device__ void softmax_role(const PagedAttnArgs &A, int nqt, int64_t units, int ctas, uint8_t *smp, const Bars &B, uint32_t tmem,
                             int wg, int wt) {
  using C = Tc<D>;
  const PagedArgs &a = A.p;
  const uint32_t lanes = static_cast<uint32_t>(wt & ~31) << 16;  // TMEM lane of the warp's first row
  const uint32_t ts = tmem + lanes + C::kS + wg * C::kStepS, tp = tmem + lanes + C::kP + wg * C::kStepP;
  const uint32_t to[2] = {tmem + lanes + C::kO, tmem + lanes + C::kO + C::kStepO};
  uint32_t n_s = 0, n_o = 0;
  Walk walk(A, units, ctas);
  Segment g;
  bool ok = true;  // false once a wait gave up: what follows only keeps the warpgroups' barriers
  while (walk.next(A, nqt, g)) {
    ok = __all_sync(0xffffffffu, ok && !*B.stop);
    const int64_t R = static_cast<int64_t>(g.rq.rows) * a.group;
    const int64_t tile0 = static_cast<int64_t>(g.qt) * kItemRows + (g.split ? 0 : wg * 128);
    const int base = g.rq.n - g.rq.rows;
    // query tile: 16 bytes a thread and step, consecutive threads along a row
    if (ok && (wg == 0 || !g.split)) {
      constexpr int CPR = D / 8;
      uint8_t *qt = smp + wg * C::kTile;
#pragma unroll 4
      for (int u = 0; u < CPR; ++u) {
        const int x = u * 128 + wt, r = x / CPR, c = x % CPR;
        const int64_t row = tile0 + r;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (row < R) {
          const int i = static_cast<int>(row / a.group), e = static_cast<int>(row - static_cast<int64_t>(i) * a.group);
          v = __ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(a.q) + (g.rq.row0 + i) * a.q_stride +
                                                    (g.h * a.group + e) * D + c * 8));
        }
        *reinterpret_cast<uint4 *>(qt + (c >> 3) * kAtom + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = v;
      }
      fence_proxy_async_shared();
      mbar_arrive(&B.q_full[wg]);
    }
    // what this thread's row sees: slots <= p, from f on or among the sinks; and the whole tile's rows
    const int64_t row = tile0 + wt;
    const bool valid = row < R;
    const int p = valid ? base + static_cast<int>(row / a.group) : -1;
    const int f = p >= 0 ? window_first(a, p) : 0;
    const int p_low = base + static_cast<int>(tile0 / a.group);
    const int f_high = window_first(a, max(0, base + static_cast<int>(((tile0 + 128 < R ? tile0 + 128 : R) - 1) / a.group)));
    float ref = -INFINITY, l = 0.f;
    const int step = g.split ? 2 : 1;
    bool any = false;
    for (int t = g.t0 + (g.split ? wg : 0); t < g.t1 && ok; t += step) {
      ok = wait_warp(B, &B.s_full[wg], n_s++ & 1);
      if (!ok) break;
      tc_fence_after();
      uint32_t w[4][32];
#pragma unroll
      for (int k = 0; k < 4; ++k) tmem_ld32_nowait(ts + 32 * k, w[k]);
      tmem_ld_wait();
      const int j0 = g.tl.at(t) * kTileSlots;
      if (!(j0 + kTileSlots - 1 <= p_low && (j0 >= f_high || j0 + kTileSlots <= a.n_sink))) {
        const int lim = p - j0, from = f - j0, sink = a.n_sink - j0;  // visible: x <= lim and (x >= from or x < sink)
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int x = 0; x < 32; ++x)
            if (!(k * 32 + x <= lim && (k * 32 + x >= from || k * 32 + x < sink))) w[k][x] = 0xff800000u;
      }
      float mx[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        mx[k] = __uint_as_float(w[k][0]);
#pragma unroll
        for (int x = 1; x < 32; ++x) mx[k] = fmaxf(mx[k], __uint_as_float(w[k][x]));
      }
      const float m = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale_log2 - Head<T>::k;
      const bool move = m > ref + kMove || (ref == -INFINITY && m > -INFINITY);
      if (__any_sync(0xffffffffu, move)) {
        const float to_ref = move ? m : ref;
        const float scale = move ? exp2_fast(ref - to_ref) : 1.f;
        ref = to_ref;
        l *= scale;
        if (any) {  // the sums of the tiles before (complete: the scores of this tile came after them)
          const uint32_t o = to[wg];
#pragma unroll 1
          for (int k = 0; k < D / 32; ++k) {
            uint32_t x[32];
            tmem_ld32_nowait(o + 32 * k, x);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * scale);
            tmem_st32(o + 32 * k, x);
          }
        }
      }
      any = true;
      const float sub = ref == -INFINITY ? 0.f : ref;
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < 4; k += 2) {
        uint32_t pk[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float x = exp2_fast(fmaf(__uint_as_float(w[k + (e >> 4)][2 * (e & 15)]), a.scale_log2, -sub));
          const float y = exp2_fast(fmaf(__uint_as_float(w[k + (e >> 4)][2 * (e & 15) + 1]), a.scale_log2, -sub));
          sum[e & 3] += x + y;
          pk[e] = Pair<T>::pack(x, y);
        }
        tmem_st32(tp + 16 * k, pk);
      }
      l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&B.p_full[wg]);
    }
    if (ok && any) ok = wait_warp(B, &B.o_full[wg], n_o++ & 1);
    tc_fence_after();
    float w0 = 1.f, w1 = 0.f;
    if (g.split) {  // stream 1 hands its reference and sum over; stream 0 joins both and writes
      float2 *xch = reinterpret_cast<float2 *>(smp + C::kTile);  // the second query tile is not used
      if (wg == 1) xch[wt] = make_float2(ref, any ? l : 0.f);
      tc_fence_before();
      named_bar(kBarBoth, 256);
      tc_fence_after();
      if (wg == 0) {
        const float2 x = xch[wt];
        const float M = fmaxf(l == 0.f ? -INFINITY : ref, x.y == 0.f ? -INFINITY : x.x);
        w0 = l == 0.f ? 0.f : exp2f(ref - M);
        w1 = x.y == 0.f ? 0.f : exp2f(x.x - M);
        l = (l == 0.f ? 0.f : w0 * l) + (x.y == 0.f ? 0.f : w1 * x.y);
        ref = M;
      }
    }
    if (ok && (wg == 0 || !g.split)) {
      const int slot = 2 * blockIdx.x + (g.u == share_begin(units, ctas, blockIdx.x) ? 0 : 1);
      const int64_t part = static_cast<int64_t>(slot) * kItemRows + (g.split ? 0 : wg * 128) + wt;
      const float inv = g.whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
      const int i = valid ? static_cast<int>(row / a.group) : 0;
      const int head = g.h * a.group + (valid ? static_cast<int>(row - static_cast<int64_t>(i) * a.group) : 0);
      T *out = static_cast<T *>(A.out) + (g.rq.row0 + i) * A.out_stride + head * D;
      bool bad = false;
      const bool two = __any_sync(0xffffffffu, w1 != 0.f);
#pragma unroll 1
      for (int k = 0; k < D / 32; ++k) {
        uint32_t x[32];
        tmem_ld32_nowait(to[g.split ? 0 : wg] + 32 * k, x);
        tmem_ld_wait();
        float o[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = w0 == 0.f ? 0.f : __uint_as_float(x[e]) * w0;
        if (two) {
          tmem_ld32_nowait(to[1] + 32 * k, x);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (w1 != 0.f) o[e] += __uint_as_float(x[e]) * w1;
        }
        if (!valid) continue;
        if (g.whole) {
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            o[e] = l == 0.f ? 0.f : o[e] * inv;
            bad |= !(fabsf(o[e]) <= 3.4e38f);
          }
#pragma unroll
          for (int e = 0; e < 32; e += 8)
            *reinterpret_cast<uint4 *>(out + 32 * k + e) =
                make_uint4(Pair<T>::pack(o[e], o[e + 1]), Pair<T>::pack(o[e + 2], o[e + 3]),
                           Pair<T>::pack(o[e + 4], o[e + 5]), Pair<T>::pack(o[e + 6], o[e + 7]));
        } else {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<float4 *>(A.part_o + part * D + 32 * k + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        }
      }
      if (valid) {
        if (g.whole)
          store_lse(A, g.rq, g.h, static_cast<int>(row), ref, l);
        else
          A.part_ml[part] = make_float2(ref, l);
      }
      unsigned redo = __ballot_sync(0xffffffffu, bad);
      while (redo) {
        const int e = __ffs(redo) - 1;
        redo &= redo - 1;
        const int64_t r = tile0 + (wt & ~31) + e;
        attend_row<T, D>(A, g.rq, g.b, static_cast<int>(r / a.group), g.h * a.group + static_cast<int>(r % a.group), wt & 31);
      }
    }
    tc_fence_before();
    if (g.split) named_bar(kBarBoth, 256);  // stream 1's sums and the exchange are read
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kTcThreads, 1) attention_many(const __grid_constant__ PagedAttnArgs A, int nqt) {
  using C = Tc<D>;
  extern __shared__ uint8_t sm_raw[];
  uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(sm_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(sm + C::kOffBar);
  Bars B;
  B.full = bars;
  B.empty = bars + C::kSlots;
  B.s_full = bars + 2 * C::kSlots;
  B.p_full = B.s_full + 2;
  B.o_full = B.s_full + 4;
  B.q_full = B.s_full + 6;
  uint64_t *drain = B.s_full + 8;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(B.s_full + 9);
  int *stop = reinterpret_cast<int *>(tmem_slot + 1);
  B.stop = stop;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(&B.full[i], kLoaderThreads);
      mbar_init(&B.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&B.s_full[i], 1);
      mbar_init(&B.p_full[i], 128);
      mbar_init(&B.o_full[i], 1);
      mbar_init(&B.q_full[i], 128);
    }
    mbar_init(drain, 1);
    *stop = 0;
    fence_barrier_init();
  }
  if (warp == 8) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();
  const int64_t units = A.unit_start[A.p.n_requests * nqt];
  const int ctas = many_ctas_used(units, A.n_ctas);
  if (units > 0 && blockIdx.x < ctas) {
    if (warp < 8) {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
      softmax_role<T, D>(A, nqt, units, ctas, sm, B, tmem, warp >> 2, tid & 127);
    } else {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
      if (warp >= 10) {
        load_role<T, D>(A, nqt, units, ctas, smem_u32(sm + C::kOffRing), B, warp - 10, lane);
      } else if (warp == 8 && lane == 0) {
        mma_role<T, D>(A, nqt, units, ctas, smem_u32(sm), B, tmem);
        umma_commit(drain);  // nothing of this block is in flight when its TMEM is freed
        mbar_wait(drain, 0);
      }
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ join
// Block (x, y): rows 16y .. 16y+15 of the item that block x of the kernel before is the first to
// begin inside; and the rows before their requests' first slot.
constexpr int kJoinManyThreads = 256;
constexpr int kJoinManyRows = 16;
template <typename T, int D>
__global__ void __launch_bounds__(kJoinManyThreads) attention_join_many(const __grid_constant__ PagedAttnArgs A, int nqt) {
  const PagedArgs &a = A.p;
  const int g = blockIdx.x, tid = threadIdx.x;
  pdl_wait();
  pdl_trigger();
  if (blockIdx.y == 0)
    for (int b = g; b < a.n_requests; b += gridDim.x) {
      const Request rq = request_of(a, b);
      const int64_t per = static_cast<int64_t>(a.n_kv_heads) * a.group, none = max(0, rq.rows - rq.n) * per;
      for (int64_t x = tid; x < none * (D / 8); x += kJoinManyThreads) {
        const int64_t hr = x / (D / 8), i = hr / per, head = hr - i * per;
        T *out = static_cast<T *>(A.out) + (rq.row0 + i) * A.out_stride + head * D + (x - hr * (D / 8)) * 8;
        *reinterpret_cast<uint4 *>(out) = make_uint4(0, 0, 0, 0);
        if (A.lse && x == hr * (D / 8)) A.lse[(rq.row0 + i) * per + head] = -INFINITY;
      }
    }
  const int64_t units = A.unit_start[a.n_requests * nqt];
  const int ctas = many_ctas_used(units, A.n_ctas);
  if (units == 0 || g == 0 || g >= ctas) return;
  const int64_t here = share_begin(units, ctas, g), prev = share_begin(units, ctas, g - 1);
  const int i = A.cta_item[g], b = i / nqt, qt = i - b * nqt;
  const int64_t start = A.unit_start[i], count = (A.unit_start[i + 1] - start) / a.n_kv_heads;
  const int h = static_cast<int>((here - start) / count);
  const int64_t begin = start + h * count;
  if (here == begin || prev > begin) return;
  int last = g;  // blocks g-1 .. last worked on it
  while (last + 1 < ctas && share_begin(units, ctas, last + 1) < begin + count) ++last;
  const int first = prev == begin ? 0 : 1;
  const Request rq = request_of(a, b);
  const int64_t left = static_cast<int64_t>(rq.rows) * a.group - static_cast<int64_t>(qt) * kItemRows;
  const int r0 = blockIdx.y * kJoinManyRows;
  const int n = static_cast<int>(left - r0 < kJoinManyRows ? left - r0 : kJoinManyRows);
  if (n <= 0) return;
  join_rows<T, D, kJoinManyThreads, kJoinManyRows>(A, rq, b, h, qt * kItemRows + r0, n, last - g + 2, [&](int k) {
    return static_cast<int64_t>(2 * (g - 1 + k) + (k == 0 ? first : 0)) * kItemRows + r0;
  });
}

// ------------------------------------------------------------------ host
int many_blocks() { return num_sms() < kJoinParts ? num_sms() : kJoinParts; }
int64_t item_count(int max_rows, int group) {
  return (static_cast<int64_t>(max_rows) * group + kItemRows - 1) / kItemRows;
}

template <typename T, int D> cudaError_t launch(const PagedAttnArgs &A, int nqt, cudaStream_t s) {
  static std::atomic<bool> checked{false};  // the register split fits what the compiler gave the block
  if (!checked.load(std::memory_order_relaxed)) {
    cudaFuncAttributes at;
    const cudaError_t e = cudaFuncGetAttributes(&at, attention_many<T, D>);
    if (e != cudaSuccess) return e;
    if (at.numRegs * kTcThreads < 256 * kRegsSoftmax + 128 * kRegsOther) return cudaErrorInvalidConfiguration;
    checked.store(true, std::memory_order_relaxed);
  }
  cudaError_t e = cudaFuncSetAttribute(attention_many<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Tc<D>::kSmem);
  if (e == cudaSuccess) e = launch_pdl(attention_plan, dim3(1), dim3(kPlanThreads), 0, s, A, nqt);
  if (e == cudaSuccess) e = launch_pdl(attention_many<T, D>, dim3(A.n_ctas), dim3(kTcThreads), Tc<D>::kSmem, s, A, nqt);
  if (e == cudaSuccess)
    e = launch_pdl(attention_join_many<T, D>, dim3(A.n_ctas, kItemRows / kJoinManyRows), dim3(kJoinManyThreads), 0, s, A, nqt);
  return e;
}

}  // namespace

size_t many_bytes(int n_requests, int max_rows, int group, int head_dim) {
  if (static_cast<int64_t>(max_rows) * group <= kFewRows) return 0;
  const size_t parts = 2 * static_cast<size_t>(many_blocks()) * kItemRows;
  return align256((static_cast<size_t>(n_requests) * item_count(max_rows, group) + 1) * 8) + align256(many_blocks() * 4) +
         align256(parts * head_dim * 4) + align256(parts * 8);
}

std::string launch_attention_many(PagedAttnArgs A, void *workspace, int dtype, cudaStream_t s) {
  const PagedArgs &a = A.p;
  const int64_t nqt = item_count(a.max_rows, a.group);
  if (nqt * a.n_requests > (1 << 30) || static_cast<int64_t>(a.max_rows) * a.group > (1 << 30))
    return "too many rows for one call";
  uint8_t *p = static_cast<uint8_t *>(workspace);
  A.n_ctas = many_blocks();
  const size_t parts = 2 * static_cast<size_t>(A.n_ctas) * kItemRows;
  A.unit_start = reinterpret_cast<int64_t *>(p);
  p += align256((static_cast<size_t>(a.n_requests) * nqt + 1) * 8);
  A.cta_item = reinterpret_cast<int32_t *>(p);
  p += align256(A.n_ctas * 4);
  A.part_o = reinterpret_cast<float *>(p);
  p += align256(parts * a.head_dim * 4);
  A.part_ml = reinterpret_cast<float2 *>(p);
  cudaError_t e;
  if (dtype == BD_BF16)
    e = a.head_dim == 128 ? launch<__nv_bfloat16, 128>(A, static_cast<int>(nqt), s)
                          : launch<__nv_bfloat16, 64>(A, static_cast<int>(nqt), s);
  else
    e = a.head_dim == 128 ? launch<__half, 128>(A, static_cast<int>(nqt), s) : launch<__half, 64>(A, static_cast<int>(nqt), s);
  return e == cudaSuccess ? std::string() : std::string("paged attention: ") + cudaGetErrorString(e);
}

}  // namespace bd
