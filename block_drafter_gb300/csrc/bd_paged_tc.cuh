// Tensor-core helpers of the paged-cache kernels: TMA boxes out of the pools, MMAs issued by a warp,
// TMEM values, packed arithmetic.
#pragma once
#include "bd_paged_attn.cuh"

#include <atomic>
#include <type_traits>

namespace bd {
namespace {

constexpr int kTileSlots = 128;
constexpr uint32_t kAtom = 16384;  // 128 rows x 128 bytes, 128-byte swizzled

template <typename T> constexpr uint32_t ab_format() { return std::is_same<T, __half>::value ? 0u : 1u; }

struct PoolMaps {  // [page][KV head][slot][D], boxes of `rows` slots x 64 values, 128-byte swizzled
  CUtensorMap k, v;
};
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, uint64_t *bar, int x, int slot, int head, int page) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst), "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(slot), "r"(head), "r"(page)
      : "memory");
}
// 32 lanes x 16 consecutive columns stored from registers.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7]), "f"(r[8]), "f"(r[9]),
      "f"(r[10]), "f"(r[11]), "f"(r[12]), "f"(r[13]), "f"(r[14]), "f"(r[15])
      : "memory");
}
// The values of a TMEM load are there (after its wait): nothing that uses them moves before this.
__device__ __forceinline__ void tmem_values(uint32_t (&r)[32]) {
  asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
               "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
  asm volatile("" : "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
               "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]));
}
// Bit x: whether column 32k + x lies at or before `last` and, from `from` on or before `sink`, in view.
__device__ __forceinline__ uint32_t seen_bits(int last, int from, int sink) {
  const uint32_t a = last < 0 ? 0u : last >= 31 ? ~0u : (2u << last) - 1u;
  const uint32_t b = from <= 0 ? ~0u : from > 31 ? 0u : ~0u << from;
  const uint32_t c = sink <= 0 ? 0u : sink > 31 ? ~0u : (1u << sink) - 1u;
  return a & (b | c);
}

// Products issued by one thread (`lead`) of a warp that runs the issuing code as a whole: in uniform
// control flow the operands stay in uniform registers (issued from a one-thread branch the same code
// took about twice as long per product, more than the product itself).
__device__ __forceinline__ uint32_t elect_lead() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}
template <bool ADD> __device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 q, %4, 0;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(lead), "n"(ADD ? 1 : 0)
      : "memory");
}
// A from TMEM.
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 q, %4, 0;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(lead), "r"(add)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t lead, uint64_t *bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(lead)
      : "memory");
}

// Slots of a TMA box: as many as always lie together in one page and one tile; 0: too few.
inline int box_rows(int page_size) {
  int b = kTileSlots;
  while (page_size % b) b >>= 1;
  return b >= 8 ? b : 0;
}

// Tiled map, boxes of boxes[0] x boxes[1] x ...; strides in bytes.
inline bool tiled_map(CUtensorMap *m, CUtensorMapDataType type, const void *p, int rank, const cuuint64_t *dims, const int64_t *stride,
                      const cuuint32_t *boxes, CUtensorMapSwizzle swizzle) {
  using Encode = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                              const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static const Encode encode = [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<Encode>(f);
  }();
  if (!encode) return false;
  cuuint64_t strides[3];
  for (int i = 0; i + 1 < rank; ++i) strides[i] = dims[i + 1] > 1 ? static_cast<cuuint64_t>(stride[i]) : 16;
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return encode(m, type, rank, const_cast<void *>(p), dims, strides, boxes, one, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// The same of 16-bit values, 128-byte swizzled, boxes of 64 x box[1] x ...; strides in elements.
inline bool tiled_map(CUtensorMap *m, const void *p, bool bf16, int rank, const cuuint64_t *dims, const int64_t *stride, const cuuint32_t *boxes) {
  int64_t bytes[3];
  for (int i = 0; i + 1 < rank; ++i) bytes[i] = stride[i] * 2;
  return tiled_map(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, p, rank, dims, bytes, boxes,
                   CU_TENSOR_MAP_SWIZZLE_128B);
}

inline bool pool_map(CUtensorMap *m, const PagedArgs &a, const void *pool, bool bf16, int box) {
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(a.head_dim), static_cast<cuuint64_t>(a.page_size),
                              static_cast<cuuint64_t>(a.n_kv_heads), static_cast<cuuint64_t>(a.n_pages)};
  const int64_t stride[3] = {a.slot_stride, a.head_stride, a.page_stride};
  const cuuint32_t boxes[4] = {64, static_cast<cuuint32_t>(box), 1, 1};
  return tiled_map(m, pool, bf16, 4, dims, stride, boxes);
}

}  // namespace
}  // namespace bd
