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
//   warp 8          issues the MMAs
//   warp 9          works out the block's segments ahead of the others
//   warps 10, 11    bring K and V into a ring of shared-memory tiles: TMA boxes of as many slots as
//                   lie together in a page (a power of two, 8 to 128); the values around the request's
//                   end, and everything for page sizes that are not a multiple of 8, row by row with
//                   cp.async, rows that nobody sees as zeros
// While one stream's softmax works, the tensor cores run the other stream's products.  An item of
// more than 128 rows gives each stream 128 of them; a smaller one gives the streams every other key
// tile of the same rows, joined at the end through TMEM.
//
// Ragged calls: the units (key tiles of all items, and kItemCost for beginning and ending each) are split
// evenly over one block an SM whatever lengths and masks are; attention_join_many joins the items that were
// split.  Calls of few or of like items need no joining launch: each item is one block's or a cluster's
// (plan_whole).
//
// The reference of a row moves only when a score exceeds it by more than 2^8, so sums are rarely rescaled;
// weights round to 16 bits (half a step: 2^-8 relative in bf16), as the result does.  A second operand with the rest
// would be half as many products again.  Root-mean-square error against 64 bits, of a form with 32-bit weights, of one
// whose weights are rounded against the row's maximum, and here, where the largest weight is no power of two and
// rounds, too: a block of 16 rows 0.00166, 0.00202, 0.00227; a prompt 0.00166, 0.00194, 0.00219.
//
// Measured: 8192 rows of one request, 32 heads over 8 KV heads, D = 128, bf16: 372 us, 1480 TFLOP/s.  A tile of
// both streams takes the tensor cores 2048 cycles and the softmax's exponentials, 32 a cycle, 1024; what is left
// of its about 2900 are the softmax's other instructions and the waits between the two.  8 requests
// of 16 rows over up to 16 384 slots: 77 us, 4.8 TB/s.
#include "bd_paged_tc.cuh"

#include <atomic>
#include <type_traits>

namespace bd {

BD_DEFINE_ERROR_TAKER(take_error_word_paged_tc)

namespace {

constexpr int kItemRows = 256;
constexpr int kTcThreads = 384;
constexpr int kLoaderThreads = 64;
// Registers a thread: the softmax warpgroups take what the third one gives up.  The sum may not
// exceed what the block starts with (checked at the first launch).
constexpr int kRegsSoftmax = 208, kRegsOther = 88;
constexpr int kSegments = 4;         // segments worked out ahead
constexpr int kSegmentReaders = 11;  // warps that read them
// What an item costs besides its tiles, in tiles (measured: queries in, pipeline filled and drained,
// results out take about 16000 cycles, a tile about 2900).
constexpr int kItemCost = 5;
constexpr int kLag = 2;            // copy groups in flight behind the one just issued

template <int D> struct Tc {
  static constexpr uint32_t kTile = (D / 64) * kAtom;      // 128 rows of D values
  static constexpr int kSlots = D == 128 ? 5 : 8;          // ring tiles
  static constexpr uint32_t kOffRing = 2 * kTile;          // behind the two query tiles
  static constexpr uint32_t kOffBar = kOffRing + kSlots * kTile;
  static constexpr uint32_t kOffPart = kOffRing + kItemRows * D * 4;  // (reference, sum) of a cluster's block's part
  static_assert(kOffPart + kItemRows * 8 <= kOffBar, "a part lies in the ring");
  static constexpr uint32_t kOffSeg = kOffBar + 320;       // [kSegments] segments of 64 bytes
  static constexpr size_t kSmem = 1024 + kOffSeg + kSegments * 64 + 128;  // and the walk
  static_assert(32 + 8 * kTcThreads / 32 <= 128, "the walk and the warps' totals");
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

// Key tiles of one item: those of the sinks, then those from its first row's window on.
struct ItemTiles {
  int sinks, first, count;
};
// Rows of the item list entry qt, and the slots of its first and last row (rows * group < 2^30).
struct ItemRows {
  int r0, n, p_low, p_high;  // n <= 0: none
};
__host__ __device__ __forceinline__ ItemRows item_rows(const PagedArgs &a, const Request &rq, int qt, int rows) {
  ItemRows x;
  x.r0 = qt * rows;
  x.n = rq.rows * a.group - x.r0;
  if (x.n > rows) x.n = rows;
  x.p_low = rq.n - rq.rows + x.r0 / static_cast<uint32_t>(a.group);
  x.p_high = rq.n - rq.rows + (x.r0 + (x.n > 1 ? x.n - 1 : 0)) / static_cast<uint32_t>(a.group);
  return x;
}
__host__ __device__ __forceinline__ ItemTiles item_tiles(const PagedArgs &a, const ItemRows &x) {
  ItemTiles t = {0, 0, 0};
  if (x.n <= 0 || x.p_high < 0) return t;
  const int first = window_first(a, x.p_low > 0 ? x.p_low : 0);
  t.first = first / kTileSlots;
  t.sinks = ((a.n_sink < first ? a.n_sink : first) + kTileSlots - 1) / kTileSlots;
  if (t.sinks > t.first) t.sinks = t.first;
  t.count = t.sinks + x.p_high / kTileSlots + 1 - t.first;
  return t;
}
// Units of one KV head of an item.
__host__ __device__ __forceinline__ int item_units(const ItemTiles &t) { return t.count > 0 ? t.count + kItemCost : 0; }
__device__ __forceinline__ int many_ctas_used(int64_t units, int most) {
  return static_cast<int>(units < 1 ? 1 : units < most ? units : most);
}

// ------------------------------------------------------------------ shares
// The item list: entry i = b * nqt + qt is rows 256 qt .. of request b, every KV head of it.
__device__ __forceinline__ int list_units(const PagedArgs &a, int nqt, int i) {
  const int b = i / nqt;
  return item_units(item_tiles(a, item_rows(a, request_of(a, b), i - b * nqt, kItemRows)));
}
// Inclusive sum over the block (NT threads; two uses need a barrier between them), and its total.
template <int NT> __device__ __forceinline__ int64_t block_sum(int64_t x, int64_t *warp_total, int64_t &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_total[warp] = x;
  __syncthreads();
  total = 0;
#pragma unroll 1
  for (int w = 0; w < NT / 32; ++w) {
    if (w == warp) x += total;
    total += warp_total[w];
  }
  return x;
}

// Lists of up to kListEach entries a thread are summed up by every block itself; longer ones by this
// kernel (one block).
constexpr int kListEach = 3;
constexpr int kPlanThreads = 1024;
__global__ void __launch_bounds__(kPlanThreads) attention_plan(const __grid_constant__ PagedAttnArgs A, int nqt) {
  __shared__ int64_t warp_total[kPlanThreads / 32];
  const PagedArgs &a = A.p;
  const int tid = threadIdx.x, N = a.n_requests * nqt;
  pdl_wait();
  pdl_trigger();
  int64_t base = 0;
  for (int i0 = 0; i0 < N; i0 += kPlanThreads) {
    const int i = i0 + tid;
    int64_t total;
    const int64_t mine = i < N ? static_cast<int64_t>(list_units(a, nqt, i)) * a.n_kv_heads : 0;
    const int64_t x = block_sum<kPlanThreads>(mine, warp_total, total);
    if (i < N) A.units[i + 1] = base + x;
    base += total;
    __syncthreads();
  }
  if (tid == 0) A.units[0] = 0;
  __syncthreads();
  const int ctas = many_ctas_used(base, A.n_ctas);
  for (int i = tid; i < N; i += kPlanThreads) {
    const int64_t s = A.units[i], e = A.units[i + 1];
    if (s == e) continue;
    int g = share_owner(base, ctas, s);
    if (share_begin(base, ctas, g) < s) ++g;
    for (; g < ctas && share_begin(base, ctas, g) < e; ++g) A.share[g] = {s, i, 0};
  }
}

// ------------------------------------------------------------------ the block's segments
struct Bars {
  uint64_t *full, *empty;                       // ring tiles
  uint64_t *s_full, *p_full, *o_full, *q_full;  // of each stream (p_full: of each half of a tile's slots)
  uint64_t *seg_full, *seg_empty;               // segments
  uint64_t *x_ready, *x_done;                   // stream 1's part of a segment they share
  volatile int *stop;                           // a wait gave up: every role ends
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

// Key tiles t0 .. t1-1 of one item and KV head.
struct __align__(16) Segment {
  int b, h, t0, t1;              // t0 == t1: no more
  int row0, base;                // request: first row of the call; slot of its row 0
  int r0, n;                     // the item's rows (of the request's rows * group)
  int p_low, p_high;             // slots of its first and last row
  int sinks, first;              // ItemTiles
  int whole, split;              // all of the item; at most 128 rows (the streams share them)
  int len;                       // slots of the request
  int pad;
  __device__ int tile(int t) const { return t < sinks ? t : first + t - sinks; }
};
static_assert(sizeof(Segment) == 64, "segment ring");

// Reads the segments in order: seg = next() until it is null; done() when it is not needed any more.
struct Segments {
  const Bars &B;
  const Segment *ring;
  uint32_t k = 0;
  __device__ Segments(const Bars &b, const Segment *r) : B(b), ring(r) {}
  __device__ const Segment *next() {
    if (!wait_warp(B, &B.seg_full[k % kSegments], (k / kSegments) & 1)) return nullptr;
    const Segment *s = ring + k % kSegments;
    return s->t0 == s->t1 ? nullptr : s;
  }
  __device__ void done(int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&B.seg_empty[k % kSegments]);
    ++k;
  }
};

// Where a block is in its share: unit u of u .. end, item i of the list, the units before it.  Without
// shares: round u of u .. end.
struct SegmentWalk {
  int64_t u, end, before;
  int i;
};
// Place `place` of the items of a call that is not shared out -- the requests' last rows first, which have the most
// tiles -- is of request b and KV head h; returns how many row tiles of 256 (128) rows lie behind its.
__device__ __forceinline__ int whole_entry(const PagedArgs &a, uint32_t place, int &b, int &h) {
  const uint32_t entry = place / a.n_kv_heads, back = entry / static_cast<uint32_t>(a.n_requests);
  h = place - entry * a.n_kv_heads;
  b = entry - back * a.n_requests;
  return static_cast<int>(back);
}
// That row tile's number; below 0: there is none.
__device__ __forceinline__ int whole_tile(const PagedAttnArgs &A, const Request &rq, int back) {
  return (rq.rows * A.p.group + A.item_rows - 1) / A.item_rows - 1 - back;
}
// The block's next segment; t0 == t1: none.
__device__ __forceinline__ void next_segment(const PagedAttnArgs &A, int nqt, int64_t units, int ctas, SegmentWalk &w, Segment &s) {
  const PagedArgs &a = A.p;
  s.t0 = s.t1 = 0;
  while (w.u < w.end && s.t0 == s.t1) {
    int qt;
    if (A.whole) {
      // the clusters are taken in turn there and back: who has one of a round's largest items has one of the
      // next round's smallest
      const uint32_t r = static_cast<uint32_t>(w.u++), n = gridDim.x / A.cluster, k = blockIdx.x / A.cluster;
      qt = whole_entry(a, r * n + (r & 1 ? n - 1 - k : k), s.b, s.h);
    } else {
      s.b = w.i / nqt;
      qt = w.i - s.b * nqt;
    }
    const Request rq = request_of(a, s.b);
    if (A.whole && (qt = whole_tile(A, rq, qt)) < 0) continue;
    const ItemRows ir = item_rows(a, rq, qt, A.item_rows);
    const ItemTiles tl = item_tiles(a, ir);
    int from = 0, to = tl.count;
    if (A.cluster > 1) {  // an even part
      const int rank = blockIdx.x % A.cluster;
      from = tl.count * rank / A.cluster;
      to = tl.count * (rank + 1) / A.cluster;
    } else if (!A.whole) {
      const int per = item_units(tl);
      const int64_t all = static_cast<int64_t>(per) * a.n_kv_heads;
      if (w.u >= w.before + all) {  // to the next item, past what the request does not fill
        w.i = ir.n > 0 ? w.i + 1 : (s.b + 1) * nqt;
        w.before += all;
        continue;
      }
      const uint32_t in = static_cast<uint32_t>(w.u - w.before);  // below 2^31: checked by the host
      s.h = in / static_cast<uint32_t>(per);
      from = in - s.h * per;
      to = w.end - w.u < per - from ? from + static_cast<int>(w.end - w.u) : per;
      if (from > 0 && from < tl.count && share_begin(units, ctas, blockIdx.x - 1) <= w.u - from)  // the first block to begin inside it
        A.join[blockIdx.x] = {s.b, s.h, ir.r0, ir.n, share_owner(units, ctas, w.u - from + tl.count - 1) - static_cast<int>(blockIdx.x) + 2,
                              rq.row0, rq.n, rq.rows};
      w.u += to - from;
    }
    s.t0 = min(from, tl.count);  // the units behind the tiles hold nothing
    s.t1 = min(to, tl.count);
    s.row0 = rq.row0;
    s.base = rq.n - rq.rows;
    s.r0 = ir.r0;
    s.n = ir.n;
    s.p_low = ir.p_low;
    s.p_high = ir.p_high;
    s.sinks = tl.sinks;
    s.first = tl.first;
    s.whole = s.t0 == 0 && s.t1 == tl.count && A.cluster == 1;
    s.split = ir.n <= 128;
    s.len = rq.n;
  }
}

// One thread works them out.
__device__ void segment_role(const PagedAttnArgs &A, int nqt, int64_t units, int ctas, SegmentWalk w, Segment *ring, const Bars &B) {
  for (uint32_t k = 0;; ++k) {
    Segment s = {};
    next_segment(A, nqt, units, ctas, w, s);
    if (k >= kSegments && !wait_or_stop(B, &B.seg_empty[k % kSegments], ((k / kSegments) - 1) & 1)) return;
    ring[k % kSegments] = s;
    mbar_arrive(&B.seg_full[k % kSegments]);
    if (s.t0 == s.t1) return;
  }
}

// ------------------------------------------------------------------ copies
// Both warps arrive on every tile with all their threads.  By TMA, lane l of the first warp brings
// box l / (D/64), columns 64 (l % (D/64)) .. of it.  Row by row, warp w copies rows 64w .. 64w+63, lane
// l holding the places of rows 64w + l and 64w + 32 + l; such copies are announced when they have
// landed, up to kLag groups later: the writing threads order them before the tensor cores' reads
// (async proxy) and arrive.
template <typename T, int D>
__device__ void load_role(const PagedAttnArgs &A, const PoolMaps &M, int box, const Segment *segs, uint32_t ring, const Bars &B,
                          int warp, int lane) {
  constexpr uint32_t NS = Tc<D>::kSlots;
  constexpr int CPR = D / 8, RPI = 32 / CPR;
  const PagedArgs &a = A.p;
  Segments walk(B, segs);
  uint32_t q = 0, late = 0;  // groups issued; of them, the last `late` are not announced
  auto announce = [&](uint32_t most) {
    for (; late > most; --late) {
      fence_proxy_async_shared();
      mbar_arrive(&B.full[(q - late) % NS]);
    }
  };
  auto leave = [&]() {  // nothing is in flight when the block ends, after a wait that gave up either
    cp_async_wait<0>();
    announce(0);
    bool ok = true;
    for (uint32_t g = q < NS ? 0 : q - NS; box && ok && g < q; ++g) ok = mbar_wait(&B.full[g % NS], (g / NS) & 1);
  };
  constexpr int ATOMS = D / 64;
  const int boxes = box ? kTileSlots / box : 0;
  const bool mine = warp == 0 && lane < boxes * ATOMS;  // this thread issues a TMA box
  const int bx = mine ? lane / ATOMS * box : 0;         // its first row in the tile
  while (const Segment *seg = walk.next()) {
    const Segment s = *seg;
    walk.done(lane);
    const int32_t *table = a.page_table + static_cast<int64_t>(s.b) * a.table_width;
    const int64_t head_off = static_cast<int64_t>(s.h) * a.head_stride;
    const T *K = static_cast<const T *>(a.k) + head_off, *V = static_cast<const T *>(a.v) + head_off;
    const int f_low = window_first(a, max(0, s.p_low)), p_high = s.p_high;
    auto slot_of = [&](int t, int k) { return s.tile(min(t, s.t1 - 1)) * kTileSlots + warp * 64 + k * 32 + lane; };
    auto page_at = [&](int t, int k) { return __ldg(table + min(slot_of(t, k), p_high) / a.page_size); };
    // page of this thread's box of tile t; beyond the pool (zeros) where no row of the item sees a slot of it
    auto box_seen = [&](int j) { return mine && any_seen(a, j, box, f_low, p_high); };
    auto box_page = [&](int t) {
      const int j = s.tile(min(t, s.t1 - 1)) * kTileSlots + bx;
      return box_seen(j) ? __ldg(table + j / a.page_size) : a.n_pages;
    };
    auto offset = [&](int t, int k, int page) {
      const int j = slot_of(t, k);
      return any_seen(a, j, 1, f_low, p_high) ? page_offset(a, page, j) : static_cast<int64_t>(-1);
    };
    auto free_slot = [&]() {  // the ring tile of group q
      return q < NS || wait_warp(B, &B.empty[q % NS], ((q / NS) - 1) & 1);
    };
    auto copy_rows = [&](const T *src, const int64_t (&off)[2]) {
      const int c = lane % CPR;
      const uint32_t dst = ring + q % NS * Tc<D>::kTile + (c >> 3) * kAtom;
#pragma unroll 4
      for (int u = 0; u < 64 / RPI; ++u) {
        const int rl = u * RPI + lane / CPR, r = warp * 64 + rl;
        const int64_t ro = __shfl_sync(0xffffffffu, u * RPI < 32 ? off[0] : off[1], rl & 31);
        cp_async16(dst + r * 128 + (((c & 7) ^ (r & 7)) << 4), src + (ro < 0 ? 0 : ro + c * 8), ro >= 0);
      }
      cp_async_commit();
      ++q;
      ++late;
    };
    if (box) {
      int next = box_page(s.t0);
      for (int t = s.t0; t < s.t1; ++t) {
        const int j0 = s.tile(t) * kTileSlots, in_page = (j0 + bx) % a.page_size;
        int pg = next;
        next = box_page(t + 1);
        if (static_cast<unsigned>(pg) >= static_cast<unsigned>(a.n_pages)) {
          if (box_seen(j0 + bx)) atomicOr(&g_error_word, DEVERR_BAD_INDEX);
          pg = a.n_pages;
        }
        if (late) {
          cp_async_wait<0>();
          announce(0);
        }
        // whatever a hidden key holds, its score is dropped; a hidden value meets a zero weight, so the
        // values of the tile that the request's end lies in come row by row, with zeros behind it
        const bool whole_v = j0 + kTileSlots <= s.len;
#pragma unroll 1
        for (int v = 0; v < (whole_v ? 2 : 1); ++v) {
          if (!free_slot()) return leave();
          const uint32_t slot = q % NS;
          if (mine) {
            mbar_arrive_expect_tx(&B.full[slot], static_cast<uint32_t>(box) * 128);
            tma_load_4d(ring + slot * Tc<D>::kTile + (lane % ATOMS) * kAtom + bx * 128, v ? &M.v : &M.k, &B.full[slot],
                        (lane % ATOMS) * 64, in_page, s.h, pg);
          } else {
            mbar_arrive(&B.full[slot]);
          }
          ++q;
        }
        if (!whole_v) {
          const int64_t off[2] = {offset(t, 0, page_at(t, 0)), offset(t, 1, page_at(t, 1))};
          if (!free_slot()) return leave();
          copy_rows(V, off);
        }
      }
    } else {
      int page[2] = {page_at(s.t0, 0), page_at(s.t0, 1)};
      for (int t = s.t0; t < s.t1; ++t) {
        const int64_t off[2] = {offset(t, 0, page[0]), offset(t, 1, page[1])};
        page[0] = page_at(t + 1, 0);
        page[1] = page_at(t + 1, 1);
#pragma unroll 1
        for (int v = 0; v < 2; ++v) {
          if (!free_slot()) return leave();
          copy_rows(v ? V : K, off);
          if (late > kLag) {
            cp_async_wait<kLag>();
            announce(kLag);
          }
        }
      }
    }
  }
  leave();
}

// ------------------------------------------------------------------ products (one warp)
template <typename T, int D>
__device__ void mma_role(const Segment *segs, uint32_t sm, const Bars &B, uint32_t tmem, int lane) {
  using C = Tc<D>;
  constexpr uint32_t NS = C::kSlots;
  const uint32_t lead = elect_lead();
  const uint32_t idesc_s = umma_idesc(ab_format<T>(), 128, kTileSlots);
  const uint32_t idesc_o = umma_idesc(ab_format<T>(), 128, D) | (1u << 16);  // V: N-major
  const uint32_t ring = sm + C::kOffRing;
  uint32_t base = 0;           // ring group of the segment's first key tile
  uint32_t n_p[2] = {0, 0}, n_q[2] = {0, 0};
  auto ready = [&](uint32_t g) {
    const bool ok = wait_warp(B, &B.full[g % NS], (g / NS) & 1);
    tc_fence_after();
    return ok;
  };
  // descriptors differ in their address field alone (16-byte units; the ring ends below 2^18 bytes)
  const uint64_t q0 = umma_desc_sw128(sm), k0 = umma_desc_sw128(ring), v0 = umma_desc_sw128_mn(ring, kAtom, 1024);
  auto scores = [&](int s, int qtile, uint32_t g) {
    const uint64_t qd = q0 + qtile * (C::kTile >> 4), kd = k0 + (g % NS) * (C::kTile >> 4);
    const uint32_t d = tmem + C::kS + s * C::kStepS;
    mma_ss<false>(lead, d, qd, kd, idesc_s);
#pragma unroll
    for (int kk = 1; kk < D / 16; ++kk) {
      const uint32_t off = ((kk >> 2) * kAtom + (kk & 3) * 32) >> 4;
      mma_ss<true>(lead, d, qd + off, kd + off, idesc_s);
    }
    commit(lead, &B.s_full[s]);
  };
  // the first half of the tile's slots as soon as its weights are there
  auto values = [&](int s, uint32_t g, bool add) {
    const uint64_t vd = v0 + (g % NS) * (C::kTile >> 4);
    const uint32_t d = tmem + C::kO + s * C::kStepO, p = tmem + C::kP + s * C::kStepP;
    const uint32_t parity = n_p[s]++ & 1;
    if (!wait_warp(B, &B.p_full[2 * s], parity)) return false;
    tc_fence_after();
    mma_ts(lead, d, p, vd, idesc_o, add);
#pragma unroll
    for (int kk = 1; kk < 4; ++kk) mma_ts(lead, d, p + kk * 8, vd + kk * 128, idesc_o, 1);
    if (!wait_warp(B, &B.p_full[2 * s + 1], parity)) return false;
    tc_fence_after();
#pragma unroll
    for (int kk = 4; kk < 8; ++kk) mma_ts(lead, d, p + kk * 8, vd + kk * 128, idesc_o, 1);
    return true;
  };
  Segments walk(B, segs);
  while (const Segment *g = walk.next()) {
    const int nt = __shfl_sync(0xffffffffu, g->t1 - g->t0, 0);
    const bool split = __shfl_sync(0xffffffffu, g->split, 0) != 0;
    walk.done(lane);
    if (!wait_warp(B, &B.q_full[0], n_q[0]++ & 1)) return;
    if (!split && !wait_warp(B, &B.q_full[1], n_q[1]++ & 1)) return;
    tc_fence_after();
    if (!split) {  // both streams take every tile
      if (!ready(base)) return;
      scores(0, 0, base);
      scores(1, 1, base);
      commit(lead, &B.empty[base % NS]);
      for (int t = 0; t < nt; ++t) {
        const uint32_t gv = base + 2 * t + 1, gk = gv + 1;
        if (!ready(gv) || !values(0, gv, t > 0)) return;
        if (t + 1 < nt) {
          if (!ready(gk)) return;
          scores(0, 0, gk);
        } else {
          commit(lead, &B.o_full[0]);
        }
        if (!values(1, gv, t > 0)) return;
        commit(lead, &B.empty[gv % NS]);
        if (t + 1 < nt) {
          scores(1, 1, gk);
          commit(lead, &B.empty[gk % NS]);
        } else {
          commit(lead, &B.o_full[1]);
        }
      }
    } else {  // stream t % 2 takes tile t
      for (int t = 0; t < 2 && t < nt; ++t) {
        if (!ready(base + 2 * t)) return;
        scores(t, 0, base + 2 * t);
        commit(lead, &B.empty[(base + 2 * t) % NS]);
      }
      for (int t = 0; t < nt; ++t) {
        const uint32_t gv = base + 2 * t + 1, gk = base + 2 * t + 4;
        const int s = t & 1;
        if (!ready(gv) || !values(s, gv, t > 1)) return;
        commit(lead, &B.empty[gv % NS]);
        if (t + 2 < nt) {
          if (!ready(gk)) return;
          scores(s, 0, gk);
          commit(lead, &B.empty[gk % NS]);
        } else {
          commit(lead, &B.o_full[s]);
        }
      }
    }
    base += 2 * nt;
  }
}

// ------------------------------------------------------------------ softmax and results
// Weights 2^(s scale - sub) of 32 columns of scores, rounded to T, to 16 TMEM columns (which lie among
// scores taken already); their sums before the rounding are added to sum.
template <typename T>
__device__ __forceinline__ void weights32(const uint32_t (&w)[32], uint32_t tp, uint64_t scale2, uint64_t sub2, uint64_t (&sum)[2]) {
  float pk[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const float2 y = unpair(fma2(pair_bits(w[2 * e], w[2 * e + 1]), scale2, sub2));
    const float y0 = exp2_fast(y.x), y1 = exp2_fast(y.y);
    sum[e & 1] = add2(sum[e & 1], pair(y0, y1));
    pk[e] = __uint_as_float(Pair<T>::pack(y0, y1));
  }
  tmem_st16(tp, pk);
}
// Half of a tile's weights are in TMEM: the products may take them.
__device__ __forceinline__ void half_ready(uint64_t *bar) {
  tmem_st_wait();
  tc_fence_before();
  mbar_arrive(bar);
}
// Columns 32k .. 32k+31 of a tile at the border of what the row sees (x <= last and (x >= from or
// x < sink)), -inf where it sees nothing.  Such tiles are few: their loops stay rolled, for less code.
__device__ __forceinline__ void edge32(uint32_t (&w)[32], uint32_t ts, int k, int last, int from, int sink) {
  tmem_ld32_nowait(ts + 32 * k, w);
  tmem_ld_wait();
  tmem_values(w);
  const uint32_t bits = seen_bits(last - 32 * k, from - 32 * k, sink - 32 * k);
#pragma unroll
  for (int x = 0; x < 32; ++x)
    if (!(bits & (1u << x))) w[x] = 0xff800000u;
}
__device__ __forceinline__ float max32(const uint32_t (&w)[32]) {
  float m[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    m[k] = max3(__uint_as_float(w[k]), __uint_as_float(w[k + 4]), __uint_as_float(w[k + 8]));
    m[k] = max3(m[k], __uint_as_float(w[k + 12]), __uint_as_float(w[k + 16]));
    m[k] = max3(m[k], __uint_as_float(w[k + 20]), __uint_as_float(w[k + 24]));
  }
  m[0] = max3(m[0], __uint_as_float(w[28]), __uint_as_float(w[29]));
  m[1] = max3(m[1], __uint_as_float(w[30]), __uint_as_float(w[31]));
  return max3(m[0], m[1], fmaxf(m[2], m[3]));
}

// Thread of row wt of stream st.
template <typename T, int D>
__device__ void softmax_role(const PagedAttnArgs &A, const Segment *segs, uint8_t *smp, const Bars &B, uint32_t tmem, int st, int wt) {
  using C = Tc<D>;
  const PagedArgs &a = A.p;
  const uint32_t lanes = static_cast<uint32_t>(wt & ~31) << 16;  // TMEM lane of the warp's first row
  const uint32_t ts = tmem + lanes + C::kS + st * C::kStepS, tp = tmem + lanes + C::kP + st * C::kStepP;
  const uint32_t to0 = tmem + lanes + C::kO;
  const uint32_t group = a.group;
  // A warp's 32 rows of its stream's query tile are its own: it fills them, and passes its results through
  // them on their way to whole rows in global memory.  Lane: piece c of rows r_first, r_first + RPI, ...
  constexpr int CPR = D / 8, RPI = 32 / CPR;
  const int lane = wt & 31, c = lane % CPR, r_first = (wt & ~31) + lane / CPR;
  const uint32_t qt = smem_u32(smp + st * C::kTile) + (c >> 3) * kAtom;
  const uint32_t step_e = RPI % group;
  const int64_t step_q = RPI / group * a.q_stride + step_e * D;
  uint32_t n_s = 0, n_o = 0, n_x = 0;
  Segments walk(B, segs);
  while (const Segment *g = walk.next()) {
    const bool split = g->split;
    const int R = g->r0 + g->n, tile0 = g->r0 + (split ? 0 : st * 128);  // the stream's rows: tile0 .. below R
    // query tile: every warp the rows of its own 32, consecutive lanes along a row
    if (st == 0 || !split) {
      const T *src = static_cast<const T *>(a.q) + g->row0 * a.q_stride + g->h * a.group * D + c * 8;
      uint32_t i = (tile0 + r_first) / group, e = tile0 + r_first - i * group;
      int64_t at = i * a.q_stride + e * D;
#pragma unroll 4
      for (int r = r_first; r < r_first + 32; r += RPI) {
        const bool in = tile0 + r < R;
        cp_async16(qt + r * 128 + (((c & 7) ^ (r & 7)) << 4), in ? src + at : a.q, in);
        e += step_e;
        at += step_q;
        if (e >= group) {
          e -= group;
          at += a.q_stride - a.group * D;
        }
      }
      cp_async_commit();
      cp_async_wait<0>();
      fence_proxy_async_shared();
      mbar_arrive(&B.q_full[st]);
    }
    // what this thread's row sees: slots <= p, from f on or among the sinks; and the whole tile's rows
    const int row = tile0 + wt;
    const int p = row < R ? g->base + static_cast<int>(row / group) : -1;
    const int f = p >= 0 ? window_first(a, p) : 0;
    const int p_low = g->base + static_cast<int>(tile0 / group);
    const int f_high = window_first(a, max(0, g->base + static_cast<int>((min(tile0 + 128, R) - 1) / group)));
    const int step = split ? 2 : 1, t1 = g->t1;
    float ref = -INFINITY, l = 0.f;
    bool any = false;
#pragma unroll 1
    for (int t = g->t0 + (split ? st : 0); t < t1; t += step) {
      const int j0 = g->tile(t) * kTileSlots;
      if (!wait_warp(B, &B.s_full[st], n_s++ & 1)) return;
      tc_fence_after();
      const bool edge = !(j0 + kTileSlots - 1 <= p_low && (j0 >= f_high || j0 + kTileSlots <= a.n_sink));
      uint32_t w[4][32];
      float m;
      if (edge) {
        m = -INFINITY;
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
          edge32(w[0], ts, k, p - j0, f - j0, a.n_sink - j0);
          m = fmaxf(m, max32(w[0]));
        }
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) tmem_ld32_nowait(ts + 32 * k, w[k]);
        tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 4; ++k) tmem_values(w[k]);
        m = fmaxf(fmaxf(max32(w[0]), max32(w[1])), fmaxf(max32(w[2]), max32(w[3])));
      }
      m = m * a.scale_log2 - Head<T>::k;
      const bool move = m > ref + kMove || (ref == -INFINITY && m > -INFINITY);
      if (__any_sync(0xffffffffu, move)) {
        const float to_ref = move ? m : ref;
        const float scale = move ? exp2_fast(ref - to_ref) : 1.f;
        ref = to_ref;
        l *= scale;
        if (any) {  // the sums of the tiles before (complete: the scores of this tile came after them)
          const uint32_t o = to0 + st * C::kStepO;
#pragma unroll 1
          for (int k = 0; k < D / 16; ++k) {
            float x[16];
            tmem_ld16(o + 16 * k, x);
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] *= scale;
            tmem_st16(o + 16 * k, x);
          }
        }
      }
      any = true;
      const float sub = ref == -INFINITY ? 0.f : ref;
      const uint64_t scale2 = pair(a.scale_log2, a.scale_log2), sub2 = pair(-sub, -sub);
      uint64_t sum[2] = {0, 0};
      if (edge) {
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
          edge32(w[0], ts, k, p - j0, f - j0, a.n_sink - j0);
          weights32<T>(w[0], tp + 16 * k, scale2, sub2, sum);
          if (k & 1) half_ready(&B.p_full[2 * st + (k >> 1)]);
        }
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          weights32<T>(w[k], tp + 16 * k, scale2, sub2, sum);
          if (k & 1) half_ready(&B.p_full[2 * st + (k >> 1)]);
        }
      }
      const float2 sums = unpair(add2(sum[0], sum[1]));
      l += sums.x + sums.y;
    }
    if (any && !wait_warp(B, &B.o_full[st], n_o++ & 1)) return;
    // a cluster's block leaves its part in the ring, which the other stream's products must have read too
    if (A.cluster > 1 && !split && !wait_warp(B, &B.o_full[st ^ 1], 0)) return;
    tc_fence_after();
    float w0 = 1.f, w1 = 0.f;
    bool has0 = l != 0.f, has1 = false;  // the streams that saw a slot; a weight of zero keeps a visible infinity or NaN
    if (split) {  // stream 0 joins both streams' sums and writes; the second query tile carries (ref, l)
      float2 *xch = reinterpret_cast<float2 *>(smp + C::kTile) + wt;
      if (st == 1) {
        *xch = make_float2(ref, l);
        tc_fence_before();
        mbar_arrive(B.x_ready);
        if (!wait_warp(B, B.x_done, n_x++ & 1)) return;
        tc_fence_after();
        walk.done(wt & 31);
        continue;
      }
      if (!wait_warp(B, B.x_ready, n_x++ & 1)) return;
      tc_fence_after();
      const float2 x = *xch;
      has1 = x.y != 0.f;
      const float M = fmaxf(has0 ? ref : -INFINITY, has1 ? x.x : -INFINITY);
      w0 = has0 ? exp2f(ref - M) : 0.f;
      w1 = has1 ? exp2f(x.x - M) : 0.f;
      l = (has0 ? w0 * l : 0.f) + (has1 ? w1 * x.y : 0.f);
      ref = M;
    }
    const bool valid = row < R, whole = g->whole;
    const bool two = __any_sync(0xffffffffu, has1);
    {
      const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
      w0 *= inv;
      w1 *= inv;
    }
    bool bad = false;
    const uint32_t own = smem_u32(smp + st * C::kTile) + wt * 128;  // this row in the tile
    T *out = static_cast<T *>(A.out) + g->row0 * A.out_stride + g->h * a.group * D + c * 8;
    // a block's parts: of the item that its share begins inside, and of the one that it ends inside
    const int64_t slot = static_cast<int64_t>(2 * blockIdx.x + (g->t0 > 0 ? 0 : 1)) * kItemRows;
    float *part = (A.cluster > 1 ? reinterpret_cast<float *>(smp + C::kOffRing) : A.part_o + slot * D) + (tile0 - g->r0) * D;
    float2 *part_ml = A.cluster > 1 ? reinterpret_cast<float2 *>(smp + C::kOffPart) : A.part_ml + slot;
    // 16-bit results fill the rows once, 32-bit parts take the two halves of D in turn
#pragma unroll 1
    for (int turn = 0; turn < (whole ? 1 : 2); ++turn) {
#pragma unroll 1
      for (int k = 0; k < (whole ? D : D / 2); k += 16) {  // 16 columns
        float o[16];
        tmem_ld16(to0 + (split ? 0 : st * C::kStepO) + turn * (D / 2) + k, o);
#pragma unroll
        for (int x = 0; x < 16; ++x) o[x] = has0 ? o[x] * w0 : 0.f;
        if (two) {
          float y[16];
          tmem_ld16(to0 + C::kStepO + turn * (D / 2) + k, y);
#pragma unroll
          for (int x = 0; x < 16; ++x)
            if (has1) o[x] += y[x] * w1;
        }
        const uint32_t word = whole ? k / 2 : k;  // 4-byte words before these columns
        uint32_t v[16];
        if (whole) {
#pragma unroll
          for (int x = 0; x < 16; ++x) bad |= !(fabsf(o[x]) <= 3.4e38f);
#pragma unroll
          for (int x = 0; x < 8; ++x) v[x] = Pair<T>::pack(o[2 * x], o[2 * x + 1]);
        } else {
#pragma unroll
          for (int x = 0; x < 16; ++x) v[x] = __float_as_uint(o[x]);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (x < 2 || !whole) {
            const uint32_t piece = word / 4 + x;
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(own + (piece >> 3) * kAtom + (((piece & 7) ^ (wt & 7)) << 4)),
                         "r"(v[4 * x]), "r"(v[4 * x + 1]), "r"(v[4 * x + 2]), "r"(v[4 * x + 3])
                         : "memory");
          }
      }
      __syncwarp();
      uint32_t i = (tile0 + r_first) / group, e = tile0 + r_first - i * group;
      int64_t at = i * A.out_stride + e * D;
#pragma unroll 4
      for (int r = r_first; r < r_first + 32; r += RPI) {
        uint4 v;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(qt + r * 128 + (((c & 7) ^ (r & 7)) << 4)) : "memory");
        if (tile0 + r < R) {
          if (whole)
            *reinterpret_cast<uint4 *>(out + at) = v;
          else
            *reinterpret_cast<uint4 *>(part + r * D + turn * (D / 2) + 4 * c) = v;
        }
        e += step_e;
        at += RPI / group * A.out_stride + step_e * D;
        if (e >= group) {
          e -= group;
          at += A.out_stride - a.group * D;
        }
      }
      __syncwarp();
    }
    bad = bad && valid;
    tc_fence_before();
    if (split) mbar_arrive(B.x_done);  // stream 1's sums and its exchange are read
    const Request rq = {g->len, g->row0, g->len - g->base};
    if (valid) {
      if (whole)
        store_lse(A, rq, g->h, row, ref, l);
      else
        part_ml[row - g->r0] = make_float2(ref, l);
    }
    const int b = g->b, h = g->h;
    walk.done(wt & 31);
    for (unsigned redo = __ballot_sync(0xffffffffu, bad); redo; redo &= redo - 1) {  // rows that are not finite
      const uint32_t r = tile0 + (wt & ~31) + __ffs(redo) - 1;
      attend_row<T, D>(A, rq, b, r / group, h * a.group + r % group, wt & 31);
    }
  }
}

// The parts of a cluster's blocks, which each block left in its ring, joined: a warp takes every kth row.  The
// softmax warps of all blocks; the others only pass the two barriers.
template <typename T, int D>
__device__ __noinline__ void cluster_join(const PagedAttnArgs &A, uint8_t *smp, int warp, int lane) {
  using C = Tc<D>;
  const int rank = blockIdx.x % A.cluster;
  int b, h;
  const int back = whole_entry(A.p, blockIdx.x / A.cluster, b, h);
  const Request rq = request_of(A.p, b);
  const ItemRows ir = item_rows(A.p, rq, max(0, whole_tile(A, rq, back)), A.item_rows);
  const ItemTiles tl = item_tiles(A.p, ir);
  if (tl.count * rank / A.cluster == tl.count * (rank + 1) / A.cluster)  // this block had no tile
    for (int r = threadIdx.x; r < kItemRows; r += 256)
      reinterpret_cast<float2 *>(smp + C::kOffPart)[r] = make_float2(-INFINITY, 0.f);
  __syncwarp();
  cluster_sync();
  if (whole_tile(A, rq, back) >= 0 && tl.count > 0) {
    const int d = lane * 4;
    const uint32_t part = smem_u32(smp + C::kOffRing), ml = smem_u32(smp + C::kOffPart);
    constexpr int kRows = 4, kBlocks = 4;  // rows and blocks whose parts are on their way together
    const int step = A.cluster * 8;        // between a warp's rows
    for (int r0 = rank + A.cluster * warp; r0 < ir.n; r0 += kRows * step) {
      float2 x[kRows];
      float M[kRows], w[kRows], L[kRows];
      unsigned seen[kRows];  // blocks that saw a slot; a weight of zero keeps a visible infinity or NaN
      float4 o[kRows];
#pragma unroll
      for (int q = 0; q < kRows; ++q) {
        const int r = r0 + q * step;
        x[q] = make_float2(-INFINITY, 0.f);
        o[q] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (lane < A.cluster && r < ir.n) {
          const uint32_t y = cluster_map(ml + r * 8, lane);
          x[q] = make_float2(ld_cluster_f32(y), ld_cluster_f32(y + 4));
        }
      }
#pragma unroll 1
      for (int i0 = 0; i0 < A.cluster; i0 += kBlocks) {
        float4 v[kBlocks][kRows];
#pragma unroll
        for (int i = 0; i < kBlocks; ++i)
          if (i0 + i < A.cluster) {
            const uint32_t at = cluster_map(part + d % D * 4, i0 + i);
#pragma unroll
            for (int q = 0; q < kRows; ++q)
              if (r0 + q * step < ir.n) v[i][q] = ld_cluster_f4(at + (r0 + q * step) * D * 4);
          }
        if (i0 == 0) {
#pragma unroll
          for (int q = 0; q < kRows; ++q) {
            seen[q] = __ballot_sync(0xffffffffu, x[q].y != 0.f);
            M[q] = warp_max(x[q].y == 0.f ? -INFINITY : x[q].x);
            w[q] = x[q].y == 0.f ? 0.f : exp2f(x[q].x - M[q]);
            L[q] = warp_sum(w[q] * x[q].y);
          }
        }
#pragma unroll
        for (int i = 0; i < kBlocks; ++i)
#pragma unroll
          for (int q = 0; q < kRows; ++q) {
            const float wi = __shfl_sync(0xffffffffu, w[q], i0 + i);
            if (seen[q] >> (i0 + i) & 1) {
              o[q].x += wi * v[i][q].x;
              o[q].y += wi * v[i][q].y;
              o[q].z += wi * v[i][q].z;
              o[q].w += wi * v[i][q].w;
            }
          }
      }
#pragma unroll
      for (int q = 0; q < kRows; ++q) {
        const int r = r0 + q * step;
        if (r >= ir.n) break;
        const bool off = d < D && finish4<T>(A, rq, h, ir.r0 + r, d, o[q], M[q], L[q]);
        if (__any_sync(0xffffffffu, off)) attend_row<T, D>(A, rq, b, (ir.r0 + r) / A.p.group, h * A.p.group + (ir.r0 + r) % A.p.group, lane);
      }
    }
  }
  __syncwarp();
  cluster_sync();  // every block's part is read
}

template <typename T, int D>
__global__ void __launch_bounds__(kTcThreads, 1) attention_many(const __grid_constant__ PagedAttnArgs A,
                                                                const __grid_constant__ PoolMaps M, int box, int nqt) {
  using C = Tc<D>;
  extern __shared__ uint8_t sm_raw[];
  uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(sm_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(sm + C::kOffBar);
  Bars B;
  B.full = bars;
  B.empty = bars + C::kSlots;
  B.s_full = bars + 2 * C::kSlots;
  B.p_full = B.s_full + 2;
  B.o_full = B.s_full + 6;
  B.q_full = B.s_full + 8;
  B.seg_full = B.s_full + 10;
  B.seg_empty = B.seg_full + kSegments;
  B.x_ready = B.seg_empty + kSegments;
  B.x_done = B.x_ready + 1;
  uint64_t *drain = B.x_ready + 2;
  static_assert((2 * C::kSlots + 10 + 2 * kSegments + 3) * 8 + 8 <= 320, "barriers");
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
  int *stop = reinterpret_cast<int *>(tmem_slot + 1);
  Segment *segs = reinterpret_cast<Segment *>(sm + C::kOffSeg);
  SegmentWalk *walk = reinterpret_cast<SegmentWalk *>(segs + kSegments);
  int64_t *warp_total = reinterpret_cast<int64_t *>(walk + 1);  // [warps]
  B.stop = stop;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(&B.full[i], kLoaderThreads);
      mbar_init(&B.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&B.s_full[i], 1);
      mbar_init(&B.p_full[2 * i], 128);
      mbar_init(&B.p_full[2 * i + 1], 128);
      mbar_init(&B.o_full[i], 1);
      mbar_init(&B.q_full[i], 128);
    }
    for (int i = 0; i < kSegments; ++i) {
      mbar_init(&B.seg_full[i], 1);
      mbar_init(&B.seg_empty[i], kSegmentReaders);
    }
    mbar_init(B.x_ready, 128);
    mbar_init(B.x_done, 128);
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
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  pdl_wait();
  pdl_trigger();
  // the block's work: an item of its own, or a share, whose beginning is summed up here or by
  // attention_plan
  const int N = A.p.n_requests * nqt;
  int64_t units = 1;
  if (A.whole) {
    if (tid == 0) *walk = {0, A.whole, 0, 0};
  } else {
    if (tid == 0) A.join[blockIdx.x].np = 0;
    int64_t u = 0;
    int ctas = 1;
    if (N <= kListEach * kTcThreads) {
      int64_t x[kListEach], mine = 0;
#pragma unroll
      for (int k = 0; k < kListEach; ++k) {
        const int i = tid * kListEach + k;
        x[k] = i < N ? static_cast<int64_t>(list_units(A.p, nqt, i)) * A.p.n_kv_heads : 0;
        mine += x[k];
      }
      int64_t before = block_sum<kTcThreads>(mine, warp_total, units) - mine;
      ctas = many_ctas_used(units, A.n_ctas);
      u = share_begin(units, ctas, blockIdx.x);
#pragma unroll
      for (int k = 0; k < kListEach; ++k) {
        if (u >= before && u < before + x[k]) {
          *walk = {u, share_begin(units, ctas, blockIdx.x + 1), before, tid * kListEach + k};
        }
        before += x[k];
      }
    } else {
      units = A.units[N];
      ctas = many_ctas_used(units, A.n_ctas);
      if (tid == 0 && blockIdx.x < ctas) {
        const PagedShare sh = A.share[blockIdx.x];
        *walk = {share_begin(units, ctas, blockIdx.x), share_begin(units, ctas, blockIdx.x + 1), sh.before, sh.item};
      }
    }
  }
  __syncthreads();
  const int ctas = A.whole ? static_cast<int>(gridDim.x) : many_ctas_used(units, A.n_ctas);
  if (units > 0 && blockIdx.x < ctas) {
    if (warp < 8) {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
      softmax_role<T, D>(A, segs, sm, B, tmem, warp >> 2, tid & 127);
      if (A.cluster > 1) cluster_join<T, D>(A, sm, warp, lane);
    } else {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
      if (warp >= 10) {
        load_role<T, D>(A, M, box, segs, smem_u32(sm + C::kOffRing), B, warp - 10, lane);
      } else if (warp == 8) {
        mma_role<T, D>(segs, smem_u32(sm), B, tmem, lane);
        __syncwarp();
        commit(elect_lead(), drain);  // nothing of this block is in flight when its TMEM is freed
        mbar_wait(drain, 0);
      } else if (lane == 0) {
        segment_role(A, nqt, units, ctas, *walk, segs, B);
      }
      if (A.cluster > 1) {  // cluster_join's barriers
        __syncwarp();
        cluster_sync();
        cluster_sync();
      }
    }
    __syncwarp();
  }
  if (warp >= 10)
    for (int b = blockIdx.x; b < A.p.n_requests; b += gridDim.x) {  // rows before their requests' first slot
      const Request rq = request_of(A.p, b);
      empty_rows<T, D>(A, rq, max(0, rq.rows - rq.n), tid - 320, 64);
    }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ join
// Warp y of list place g: row y of the join that block g left.  The lanes hold the weights of up to 32
// parts side by side (more are rare: they go round again), then add the parts, four columns (two with
// D = 64) a lane.
constexpr int kJoinWarps = 8;
constexpr int kJoinHeld = 4;
template <typename T, int D>
__global__ void __launch_bounds__(32 * kJoinWarps) attention_join_many(const __grid_constant__ PagedAttnArgs A) {
  constexpr int C = D / 32;
  const int g = blockIdx.x, lane = threadIdx.x & 31, r = blockIdx.y * kJoinWarps + (threadIdx.x >> 5);
  pdl_wait();
  pdl_trigger();
  const PagedJoin j = A.join[g];
  if (j.np == 0 || r >= j.n) return;
  auto slot = [&](int i) { return static_cast<int64_t>(2 * (g - 1 + i) + (i == 0 ? 1 : 0)) * kItemRows + r; };
  float M = -INFINITY, L = 0.f, o[C];
#pragma unroll
  for (int c = 0; c < C; ++c) o[c] = 0.f;
  for (int i0 = 0; i0 < j.np; i0 += 32) {
    const int n = min(32, j.np - i0);
    auto part = [&](int i, float (&y)[C]) {
      const float *v = A.part_o + slot(i0 + i) * D + C * lane;
      if constexpr (C == 4)
        *reinterpret_cast<float4 *>(y) = __ldcg(reinterpret_cast<const float4 *>(v));
      else
        *reinterpret_cast<float2 *>(y) = __ldcg(reinterpret_cast<const float2 *>(v));
    };
    float held[kJoinHeld][C];  // the first parts are on their way while the weights are worked out
#pragma unroll
    for (int i = 0; i < kJoinHeld; ++i)
      if (i < n) part(i, held[i]);
    float2 x = make_float2(-INFINITY, 0.f);
    if (i0 + lane < j.np) x = __ldcg(A.part_ml + slot(i0 + lane));
    if (x.y == 0.f) x.x = -INFINITY;
    const float m = fmaxf(M, warp_max(x.x));
    const unsigned seen = __ballot_sync(0xffffffffu, x.y != 0.f);  // parts that saw a slot; a weight of zero keeps a visible infinity or NaN
    const float back = M == -INFINITY ? 0.f : exp2f(M - m), w = x.y == 0.f ? 0.f : exp2f(x.x - m);
    L = L * back + warp_sum(w * x.y);
    M = m;
#pragma unroll
    for (int c = 0; c < C; ++c) o[c] *= back;
    auto add = [&](int i, const float (&y)[C]) {
      const float wi = __shfl_sync(0xffffffffu, w, i);
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (seen >> i & 1) o[c] += wi * y[c];
    };
#pragma unroll
    for (int i = 0; i < kJoinHeld; ++i)
      if (i < n) add(i, held[i]);
#pragma unroll 4
    for (int i = kJoinHeld; i < n; ++i) {
      float y[C];
      part(i, y);
      add(i, y);
    }
  }
  const Request rq = {j.len, j.row0, j.rows};
  const uint32_t row = j.from + r, group = A.p.group, t = row / group;
  const int head = j.h * A.p.group + row - t * group;
  const float inv = L == 0.f ? 0.f : 1.f / L;
  uint32_t *out = reinterpret_cast<uint32_t *>(static_cast<T *>(A.out) + (rq.row0 + static_cast<int>(t)) * A.out_stride + head * D + C * lane);
  bool bad = false;
#pragma unroll
  for (int c = 0; c < C; c += 2) {
    const float y0 = o[c] * inv, y1 = o[c + 1] * inv;
    bad |= !(fabsf(y0) <= 3.4e38f) || !(fabsf(y1) <= 3.4e38f);
    out[c / 2] = Pair<T>::pack(y0, y1);
  }
  if (lane == 0) store_lse(A, rq, j.h, row, M, L);
  if (__any_sync(0xffffffffu, bad)) attend_row<T, D>(A, rq, j.b, t, head, lane);
}

// ------------------------------------------------------------------ host
int many_blocks() { return num_sms() < kJoinParts - 1 ? num_sms() : kJoinParts - 1; }
// A call is not shared out, but every item and KV head is one block's, where that leaves the busiest block
// less than what sharing costs: its even part of the tiles, an item that it shares and, about
// kJoinCost tiles, the joins (8 heads, group 4: 512 rows 12.4 us in items of 128 rows, 14.6 us of 256, shared out
// 25.3 us; 8192 rows 376 us, shared out 410 us).  Items of 128 rows, whose tiles the two streams share, where there
// are blocks for them.
// Bounds stand for the lengths here; of several requests, ones of equal rows, as n_rows tells.
constexpr int kJoinCost = 8;
// An item may also be a cluster's, whose blocks join their parts through distributed shared memory, for about
// kClusterCost tiles more than a whole item, up to kClusterTiles tiles a block (16 rows, 8 heads, group 4: 2048
// slots, eight blocks an item 16.8 us, one 25.0 us; 8 requests of 4096 slots, two blocks 38.2 us, shared out 43.6 us,
// of 1024 slots, two blocks 21.2 us, one 17.8 us; 16 384 slots, eight blocks 33.1 us, shared out 29.4 us).
constexpr int kClusterCost = 5, kClusterTiles = 8;
constexpr int kMostWhole = 4096;  // items that are weighed on the host: more take milliseconds, joins or not
int64_t item_count(int max_rows, int group, int rows) {
  return (static_cast<int64_t>(max_rows) * group + rows - 1) / rows;
}
struct WholeLoad {
  int most, even;  // the busiest block's units; an even part of them
};
WholeLoad whole_load(const PagedArgs &a, int rows, int blocks) {
  const Request rq = {a.max_len, 0, a.max_rows < a.max_len ? a.max_rows : a.max_len};
  const bool shared = rows < kItemRows || a.max_rows * a.group <= kItemRows / 2;  // by the two streams
  const int per = a.n_requests * a.n_kv_heads;
  int load[kJoinParts] = {}, most = 0, at = 0;
  int64_t all = 0;
  bool back = false;
  for (int64_t qt = item_count(a.max_rows, a.group, rows) - 1; qt >= 0; --qt) {
    const ItemTiles t = item_tiles(a, item_rows(a, rq, static_cast<int>(qt), rows));
    const int units = shared ? (t.count + 1) / 2 + kItemCost : item_units(t);
    for (int x = 0; x < per; ++x) {
      int &l = load[back ? blocks - 1 - at : at];
      l += units;
      most = l > most ? l : most;
      if (++at == blocks) at = 0, back = !back;
    }
    all += static_cast<int64_t>(units) * per;
  }
  return {most, static_cast<int>(all / blocks)};
}
// Sets A.whole, A.cluster and A.item_rows.
template <typename Fit> void plan_whole(PagedAttnArgs &A, const Fit &fit) {
  const PagedArgs &a = A.p;
  const int blocks = A.n_ctas;
  const int64_t items = item_count(a.max_rows, a.group, kItemRows) * a.n_requests * a.n_kv_heads;
  A.whole = 0;
  A.cluster = 1;
  A.item_rows = kItemRows;
  const bool alike = static_cast<int64_t>(a.n_rows) * 20 >= static_cast<int64_t>(a.n_requests) * a.max_rows * 19;
  if (items > kMostWhole || (items > blocks && !alike)) return;
  const WholeLoad w = whole_load(a, kItemRows, blocks);
  int best = w.even + kItemCost + kJoinCost;
  auto take = [&](int most, int rows, int cluster) {
    if (most > best) return;
    best = most;
    A.item_rows = rows;
    A.cluster = cluster;
    A.whole = static_cast<int>((item_count(a.max_rows, a.group, rows) * a.n_requests * a.n_kv_heads + blocks - 1) / blocks);
  };
  // items of a cluster each: the most blocks of which the device holds a cluster for each
  auto spread = [&](int rows) {
    const int64_t n = item_count(a.max_rows, a.group, rows) * a.n_requests * a.n_kv_heads;
    int size = kMostCluster;
    while (size > 1 && n > fit.of(size)) size /= 2;
    if (size == 1) return;
    const Request rq = {a.max_len, 0, a.max_rows < a.max_len ? a.max_rows : a.max_len};
    const int last = static_cast<int>(item_count(a.max_rows, a.group, rows)) - 1;
    const int tiles = (item_tiles(a, item_rows(a, rq, last, rows)).count + size - 1) / size;
    const int units = rows == kItemRows && a.max_rows * a.group > kItemRows / 2 ? tiles : (tiles + 1) / 2;
    if (units <= kClusterTiles) take(units + kItemCost + kClusterCost, rows, size);
  };
  take(w.most, kItemRows, 1);
  if (items <= blocks) {
    take(whole_load(a, kItemRows / 2, blocks).most, kItemRows / 2, 1);
    spread(kItemRows);
    if (a.max_rows * a.group > kItemRows / 2) spread(kItemRows / 2);
  }
}

template <typename T, int D> cudaError_t launch(PagedAttnArgs &A, cudaStream_t s) {
  static const ClustersAtOnce fit(attention_many<T, D>, kTcThreads, Tc<D>::kSmem);
  plan_whole(A, fit);
  const int nqt = static_cast<int>(item_count(A.p.max_rows, A.p.group, A.item_rows));
  static std::atomic<bool> checked{false};  // the register split fits what the compiler gave the block
  if (!checked.load(std::memory_order_relaxed)) {
    cudaFuncAttributes at;
    const cudaError_t e = cudaFuncGetAttributes(&at, attention_many<T, D>);
    if (e != cudaSuccess) return e;
    if (at.numRegs * kTcThreads < 256 * kRegsSoftmax + 128 * kRegsOther) return cudaErrorInvalidConfiguration;
    checked.store(true, std::memory_order_relaxed);
  }
  cudaError_t e = cudaFuncSetAttribute(attention_many<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Tc<D>::kSmem);
  if (e == cudaSuccess && !A.whole && A.p.n_requests * nqt > kListEach * kTcThreads)
    e = launch_pdl(attention_plan, dim3(1), dim3(kPlanThreads), 0, s, A, nqt);
  PoolMaps M = {};
  int box = box_rows(A.p.page_size);
  const bool bf16 = std::is_same<T, __nv_bfloat16>::value;
  if (box && !(pool_map(&M.k, A.p, A.p.k, bf16, box) && pool_map(&M.v, A.p, A.p.v, bf16, box))) box = 0;
  const int items = A.p.n_requests * nqt * A.p.n_kv_heads;
  const int blocks = A.whole && items * A.cluster < A.n_ctas ? items * A.cluster : A.n_ctas;
  if (e == cudaSuccess) e = allow_cluster(attention_many<T, D>, A.cluster);
  if (e == cudaSuccess)
    e = launch_pdl_cluster(attention_many<T, D>, dim3(blocks), dim3(kTcThreads), Tc<D>::kSmem, s, A.cluster, A, M, box, nqt);
  if (e == cudaSuccess && !A.whole) {
    const int rows = A.p.max_rows * A.p.group, most = rows < kItemRows ? rows : kItemRows;
    e = launch_pdl(attention_join_many<T, D>, dim3(A.n_ctas, (most + kJoinWarps - 1) / kJoinWarps), dim3(32 * kJoinWarps), 0, s, A);
  }
  return e;
}

}  // namespace

size_t many_bytes(int n_requests, int max_rows, int group, int head_dim) {
  if (static_cast<int64_t>(max_rows) * group <= kFewRows) return 0;
  const size_t parts = 2 * static_cast<size_t>(many_blocks()) * kItemRows;
  return align256((static_cast<size_t>(n_requests) * item_count(max_rows, group, kItemRows) + 1) * 8) +
         align256(many_blocks() * sizeof(PagedShare)) + align256(many_blocks() * sizeof(PagedJoin)) + align256(parts * head_dim * 4) + align256(parts * 8);
}

std::string launch_attention_many(PagedAttnArgs A, void *workspace, int dtype, cudaStream_t s) {
  const PagedArgs &a = A.p;
  uint8_t *p = static_cast<uint8_t *>(workspace);
  A.n_ctas = many_blocks();
  const size_t parts = 2 * static_cast<size_t>(A.n_ctas) * kItemRows;
  A.units = reinterpret_cast<int64_t *>(p);
  p += align256((static_cast<size_t>(a.n_requests) * item_count(a.max_rows, a.group, kItemRows) + 1) * 8);
  A.share = reinterpret_cast<PagedShare *>(p);
  p += align256(A.n_ctas * sizeof(PagedShare));
  A.join = reinterpret_cast<PagedJoin *>(p);
  p += align256(A.n_ctas * sizeof(PagedJoin));
  A.part_o = reinterpret_cast<float *>(p);
  p += align256(parts * a.head_dim * 4);
  A.part_ml = reinterpret_cast<float2 *>(p);
  cudaError_t e;
  if (dtype == BD_BF16)
    e = a.head_dim == 128 ? launch<__nv_bfloat16, 128>(A, s) : launch<__nv_bfloat16, 64>(A, s);
  else
    e = a.head_dim == 128 ? launch<__half, 128>(A, s) : launch<__half, 64>(A, s);
  return e == cudaSuccess ? std::string() : std::string("paged attention: ") + cudaGetErrorString(e);
}

}  // namespace bd
