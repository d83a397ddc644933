// Log probabilities of given tokens, entropy and top alternatives (bd_token_logprobs).
//
// One pass over a row's logits x with the running maximum m of a softmax, c = log2(e) / temperature:
//   s = sum 2^d,  t = sum 2^d d,  d = (x - m) c;   m -> m':  w = 2^((m-m') c),  t' = w (t + s (m-m') c),  s' = w s
//   lse = m c ln2 + ln s,  entropy = ln2 (log2 s - t / s),  logprob = (x_token - m) c ln2 - ln s.
// The entropy is formed from d <= 0 and not as lse minus a mean: nothing large cancels.
//
// The largest logits come out of the same pass: a block keeps those that reach its threshold in a buffer, as keys
// that order by value, then by the lower id; now and then it thins the buffer to the top_k largest, the last of which is
// the next threshold.  The first threshold is the top_k-th largest of the threads' maxima over the row's first
// logits, which the threads still hold then; so of 152 000 logits a few hundred reach the buffer.  Where more reach it than
// it holds (values in ascending order, many equal ones), the round is done again with the threshold that the buffer
// gives, which is larger each time.
//
// Few rows are a cluster's of up to 16 blocks, each with an equal part of the row; the first one joins their sums and
// candidates through distributed shared memory.  Bound by the bytes of the logits.
#include <cfloat>

#include "bd_checks.h"
#include "bd_paged_device.cuh"

namespace bd {

BD_DEFINE_ERROR_TAKER(take_error_word_logprobs)

namespace {

constexpr int kLpThreads = 512;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpCluster = 16;
constexpr int kLpEach = 4;  // vectors of a thread in flight
constexpr int kTop = BD_LOGPROB_TOP_MAX;
constexpr int kKeys = 512;             // candidates that a block thins at once, a thread each
constexpr int kBuffer = kKeys - kTop;  // those of a round, beside the ones kept before
static_assert(kLpCluster * kTop <= kKeys && kKeys <= kLpThreads, "the joining block thins every block's candidates");

struct LogprobArgs {
  const void *logits;
  int64_t row_stride;
  int rows, vocab, cluster;
  float scale, inv_t;  // log2(e) / temperature, 1 / temperature
  const int32_t *tokens;
  int n_given, top_k;
  float *logprob, *entropy, *lse;
  int32_t *top_ids;
  float *top_logprob;
};

// 16 bytes of logits as fp32.
template <typename T> struct Vec {
  static constexpr int N = 16 / sizeof(T);
  static __device__ __forceinline__ void unpack(const uint4 &w, float (&x)[N]) {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = Pair<T>::unpack(v[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
};
template <> struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(const uint4 &w, float (&x)[4]) {
    x[0] = __uint_as_float(w.x);
    x[1] = __uint_as_float(w.y);
    x[2] = __uint_as_float(w.z);
    x[3] = __uint_as_float(w.w);
  }
};

// Larger for larger values, among equal ones for lower ids (-0 is 0, NaN counts as -inf).
__device__ __forceinline__ uint64_t key_of(float x, int id) {
  const uint32_t b = x != x ? 0xff800000u : __float_as_uint(x + 0.f);
  return static_cast<uint64_t>(b & 0x80000000u ? ~b : b | 0x80000000u) << 32 | static_cast<uint32_t>(~id);
}
__device__ __forceinline__ float key_value(uint64_t k) {
  const uint32_t b = static_cast<uint32_t>(k >> 32);
  return __uint_as_float(b & 0x80000000u ? b & 0x7fffffffu : ~b);
}
__device__ __forceinline__ int key_id(uint64_t k) { return static_cast<int>(~static_cast<uint32_t>(k)); }

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN where one is
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

__device__ __forceinline__ uint64_t ld_cluster_u64(uint32_t addr) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}

struct Sums {
  float m, s, t;
};
__device__ __forceinline__ void rescale(Sums &a, float m, float c) {  // m >= a.m
  if (m == a.m) return;
  const float d = fmaxf((a.m - m) * c, -150.f), w = exp2_fast(d);
  a.t = w * (a.t + a.s * d);
  a.s *= w;
  a.m = m;
}
__device__ __forceinline__ Sums join(Sums a, Sums b, float c) {
  const float m = fmaxf(a.m, b.m);
  rescale(a, m, c);
  rescale(b, m, c);
  return {m, a.s + b.s, a.t + b.t};
}

// The k largest of keys[0 .. n), n <= kKeys, to keys[0 .. k) in descending order; all threads.
__device__ __forceinline__ void thin(uint64_t *keys, int n, int k) {
  __syncthreads();
  const int i = threadIdx.x;
  uint64_t mine = 0;
  int rank = k;
  if (i < n) {
    mine = keys[i];
    rank = 0;
    for (int j = 0; j < n; ++j) rank += keys[j] > mine;
  }
  __syncthreads();
  if (rank < k) keys[rank] = mine;
  __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(kLpThreads, 2) logprobs_kernel(const __grid_constant__ LogprobArgs A) {
  using V = Vec<T>;
  constexpr int N = V::N;
  __shared__ __align__(16) uint64_t keys[kKeys], best[kTop];  // this round's candidates; those kept before
  __shared__ __align__(16) float top_of[kLpThreads];  // the threads' maxima
  __shared__ Sums warp_sums[kLpWarps];
  __shared__ Sums block_sums;
  __shared__ int count;
  __shared__ uint64_t first_threshold;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x / static_cast<uint32_t>(A.cluster), rank = blockIdx.x - row * A.cluster, k = A.top_k;
  const float c = A.scale;
  const T *x = static_cast<const T *>(A.logits) + static_cast<int64_t>(row) * A.row_stride;
  // whole 16-byte vectors lie from `head` on; what is before and behind them is the first block's, an element a thread
  const int head = min(A.vocab, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(x) & 15)) % 16 / sizeof(T)));
  const int vecs = (A.vocab - head) / N, tail = head + vecs * N;
  const uint4 *xv = reinterpret_cast<const uint4 *>(x + head);
  const int v0 = static_cast<int>(static_cast<int64_t>(vecs) * rank / A.cluster);
  const int v1 = static_cast<int>(static_cast<int64_t>(vecs) * (rank + 1) / A.cluster);
  if (tid == 0) count = 0;
  pdl_wait();
  pdl_trigger();
  Sums a = {-FLT_MAX, 0.f, 0.f};
  uint64_t threshold = 0;  // of the keys that are kept
  float reach = -INFINITY; // its value

  auto add = [&](const auto &v) {
    constexpr int n = sizeof(v) / sizeof(v[0]);
    float m = a.m;
#pragma unroll
    for (int e = 0; e < n; ++e) m = fmaxf(m, v[e]);
    rescale(a, m, c);
#pragma unroll
    for (int e = 0; e < n; ++e) {
      const float d = max_nan((v[e] - a.m) * c, -150.f), w = exp2_fast(d);
      a.s += w;
      a.t = fmaf(w, d, a.t);
    }
  };
  auto offer = [&](float v, int id) {
    if (!(v >= reach) && v == v) return;
    const uint64_t key = key_of(v, id);
    if (key < threshold) return;
    const int at = atomicAdd(&count, 1);
    if (at < kBuffer) keys[at] = key;
  };
  // the loose elements
  float one[1], &loose = one[0];
  int loose_id = -1;
  if (rank == 0) {
    if (tid < head) loose_id = tid;
    else if (tid - head < A.vocab - tail) loose_id = tail + tid - head;
    if (loose_id >= 0) {
      loose = to_f<T>(x[loose_id]);
      add(one);
    }
  }
  // the first vector of every thread, which gives the first threshold
  float v[N];
  int at = v0 + tid;
  const bool has = at < v1;
  if (has) {
    V::unpack(__ldg(xv + at), v);
    add(v);
  }
  __syncthreads();
  if (k > 0) {
    if (tid == 0) first_threshold = 0;
    float m = -INFINITY;
    if (has)
#pragma unroll
      for (int e = 0; e < N; ++e) m = fmaxf(m, v[e]);
    top_of[tid] = m;
    __syncthreads();
    int larger = 0;
    for (int j = 0; j < kLpThreads; j += 4) {
      const float4 o = *reinterpret_cast<const float4 *>(top_of + j);
      larger += (o.x > m || (o.x == m && j < tid)) + (o.y > m || (o.y == m && j + 1 < tid)) + (o.z > m || (o.z == m && j + 2 < tid)) +
                (o.w > m || (o.w == m && j + 3 < tid));
    }
    // k maxima are at least this: no smaller value is among the k largest
    if (larger == k - 1) first_threshold = key_of(m, 0x7fffffff);
    __syncthreads();
    threshold = first_threshold;
    reach = key_value(threshold);
  }
  // rounds: the first vectors and loose elements, an eighth of the rest, the rest
  const int from = v0 + kLpThreads, rest = max(0, v1 - from), cut = from + rest / 8;
  int kept = 0;  // candidates of the rounds before
  for (int round = 0; round < 3; ++round) {
    const int r0 = round == 2 ? cut : from, r1 = round == 0 ? from : round == 1 ? cut : from + rest;
    for (bool again = false;;) {
      if (round == 0) {
        if (k > 0) {
          if (loose_id >= 0) offer(loose, loose_id);
          if (has)
#pragma unroll
            for (int e = 0; e < N; ++e) offer(v[e], head + at * N + e);
        }
      } else {
        for (int i = r0 + tid; i < r1; i += kLpEach * kLpThreads) {
          uint4 w[kLpEach];
#pragma unroll
          for (int u = 0; u < kLpEach; ++u)
            if (i + u * kLpThreads < r1) w[u] = __ldg(xv + i + u * kLpThreads);
#pragma unroll
          for (int u = 0; u < kLpEach; ++u) {
            if (i + u * kLpThreads >= r1) continue;
            float y[N];
            V::unpack(w[u], y);
            if (!again) add(y);
            if (k > 0) {
              float m = y[0];
#pragma unroll
              for (int e = 1; e < N; ++e) m = fmaxf(m, y[e]);
              if (!(m < reach)) {
#pragma unroll 1
                for (int e = 0; e < N; ++e) offer(y[e], head + (i + u * kLpThreads) * N + e);
              }
            }
          }
        }
      }
      if (k == 0) break;
      __syncthreads();
      const int n = count;
      again = n > kBuffer;
      if (again) {  // k of those in the buffer are at least the next threshold
        thin(keys, kBuffer, k);
      } else {
        if (tid < kept) keys[n + tid] = best[tid];
        thin(keys, n + kept, k);
        kept = min(n + kept, k);
        if (tid < kept) best[tid] = keys[tid];
      }
      if (again || kept == k) {
        threshold = max(threshold, keys[k - 1]);
        reach = key_value(threshold);
      }
      if (tid == 0) count = 0;
      __syncthreads();
      if (!again) break;
    }
  }
  // the block's sums
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Sums b = {__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.s, o), __shfl_xor_sync(0xffffffffu, a.t, o)};
    a = join(a, b, c);
  }
  if (lane == 0) warp_sums[warp] = a;
  if (tid < k && tid >= kept) best[tid] = 0;  // below every key
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kLpWarps; ++w) a = join(a, warp_sums[w], c);
    block_sums = a;
  }
  __syncthreads();
  if (A.cluster > 1) {
    cluster_sync();
    if (rank == 0) {
      const int from_block = k > 0 ? tid / k : A.cluster, which = tid - from_block * k;
      uint64_t key = 0;
      if (from_block < A.cluster) key = ld_cluster_u64(cluster_map(smem_u32(best + which), from_block));
      if (tid == 0)
        for (int b = 1; b < A.cluster; ++b) {
          const uint32_t p = cluster_map(smem_u32(&block_sums), b);
          a = join(a, {ld_cluster_f32(p), ld_cluster_f32(p + 4), ld_cluster_f32(p + 8)}, c);
        }
      if (k > 0) {
        if (from_block < A.cluster) keys[tid] = key;
        thin(keys, A.cluster * k, k);
        if (tid < k) best[tid] = keys[tid];
      }
      if (tid == 0) block_sums = a;
    }
    __syncthreads();
    cluster_sync();  // every block's sums and candidates are read
    if (rank != 0) return;
  }
  const Sums r = block_sums;
  const float ln_s = logf(r.s);
  if (tid == 0) {
    if (A.lse) A.lse[row] = r.m * A.inv_t + ln_s;
    if (A.entropy) A.entropy[row] = ln_s - kLn2 * (r.t / r.s);
  }
  auto logprob = [&](float z) { return r.s == 0.f ? NAN : (z - r.m) * A.inv_t - ln_s; };
  if (tid < k) {
    const uint64_t key = best[tid];
    A.top_ids[static_cast<int64_t>(row) * k + tid] = key_id(key);
    if (A.top_logprob) A.top_logprob[static_cast<int64_t>(row) * k + tid] = logprob(key_value(key));
  }
  for (int g = tid; g < A.n_given; g += kLpThreads) {
    const int id = A.tokens[static_cast<int64_t>(row) * A.n_given + g];
    float p = 0.f;
    if (id >= 0 && id < A.vocab) {
      p = logprob(to_f<T>(x[id]));
    } else if (id != -1) {
      atomicOr(&g_error_word, DEVERR_BAD_INDEX);
      p = NAN;
    }
    A.logprob[static_cast<int64_t>(row) * A.n_given + g] = p;
  }
}

template <typename T> cudaError_t launch(const LogprobArgs &A, cudaStream_t s) {
  auto kernel = logprobs_kernel<T>;
  const cudaError_t e = allow_cluster(kernel, A.cluster);
  if (e != cudaSuccess) return e;
  return launch_pdl_cluster(kernel, dim3(static_cast<unsigned>(A.rows) * A.cluster), dim3(kLpThreads), 0, s, A.cluster, A);
}

}  // namespace
}  // namespace bd

using namespace bd;

extern "C" bd_status bd_token_logprobs(const void *logits, int64_t row_stride, int dtype, int rows, int vocab, float temperature,
                                       const int32_t *tokens, int n_given, float *logprob, float *entropy, float *lse, int top_k,
                                       int32_t *top_ids, float *top_logprob, void *stream) {
  if (dtype != BD_BF16 && dtype != BD_F16 && dtype != BD_F32)
    return refuse(BD_ERR_UNSUPPORTED, "log probabilities: dtype must be BD_BF16, BD_F16 or BD_F32");
  if (rows < 0 || rows > (1 << 24) || vocab < 1 || vocab > (1 << 24))
    return refuse(BD_ERR_INVALID_ARG, "log probabilities: rows must be in 0..2^24 and vocab in 1..2^24");
  if (n_given < 0 || n_given > BD_LOGPROB_GIVEN_MAX || top_k < 0 || top_k > kTop || top_k > vocab)
    return refuse(BD_ERR_INVALID_ARG, "log probabilities: n_given must be in 0..64, top_k in 0..32 and at most vocab");
  const float scale = static_cast<float>(1.4426950408889634 / temperature), inv_t = static_cast<float>(1.0 / temperature);
  if (!(temperature > 0.f) || !std::isnormal(scale) || !std::isnormal(inv_t))
    return refuse(BD_ERR_INVALID_ARG, "log probabilities: temperature and its reciprocal must be > 0 and finite");
  if (rows == 0) return BD_OK;
  const int64_t size = dtype == BD_F32 ? 4 : 2;
  if (!logits || misaligned(logits, size) || (rows > 1 && row_stride < vocab))
    return refuse(BD_ERR_INVALID_ARG, "log probabilities: logits must be given, rows of at least vocab elements");
  const int64_t given = 4ll * rows * n_given, tops = 4ll * rows * top_k;
  struct Out {
    const void *p;
    int64_t bytes;
    const char *name;
  } outs[] = {{logprob, given, "logprob"}, {entropy, entropy ? 4ll * rows : 0, "entropy"}, {lse, lse ? 4ll * rows : 0, "lse"},
              {top_ids, tops, "top_ids"}, {top_logprob, top_logprob ? tops : 0, "top_logprob"}};
  if ((given > 0 && !tokens) || misaligned(tokens, 4)) return refuse(BD_ERR_INVALID_ARG, "log probabilities: tokens must be given");
  for (const Out &o : outs) {
    if ((o.bytes > 0 && !o.p) || misaligned(o.p, 4))
      return refuse(BD_ERR_INVALID_ARG, std::string("log probabilities: ") + o.name + " must be given, 4-byte aligned");
    if (overlap(o.p, o.bytes, logits, ((rows - 1) * row_stride + vocab) * size) || overlap(o.p, o.bytes, tokens, given))
      return refuse(BD_ERR_INVALID_ARG, std::string("log probabilities: ") + o.name + " and an input overlap");
    for (const Out &q : outs)
      if (&q != &o && overlap(o.p, o.bytes, q.p, q.bytes))
        return refuse(BD_ERR_INVALID_ARG, std::string("log probabilities: ") + o.name + " and " + q.name + " overlap");
  }
  LogprobArgs A = {};
  A.logits = logits;
  A.row_stride = rows > 1 ? row_stride : 0;
  A.rows = rows;
  A.vocab = vocab;
  A.scale = scale;
  A.inv_t = inv_t;
  A.tokens = tokens;
  A.n_given = n_given;
  A.top_k = top_k;
  A.logprob = logprob;
  A.entropy = entropy;
  A.lse = lse;
  A.top_ids = top_ids;
  A.top_logprob = top_logprob;
  // blocks of a row while there are SMs left for them and 16 KB of logits for each
  A.cluster = 1;
  while (A.cluster < kLpCluster && static_cast<int64_t>(rows) * A.cluster * 2 <= num_sms() && vocab * size > A.cluster * 16384) A.cluster *= 2;
  use_target_kernels();
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == BD_F32 ? launch<float>(A, s) : dtype == BD_BF16 ? launch<__nv_bfloat16>(A, s) : launch<__half>(A, s);
  return ran(e == cudaSuccess ? std::string() : std::string("log probabilities: ") + cudaGetErrorString(e));
}
