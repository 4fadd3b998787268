// q4_tiles.cuh — what the tensor-core attention kernels (prompts, paged cache)
// share: tile sizes, references of the softmax, small helpers of its threads,
// tensor maps of packed rows.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <type_traits>

#include "q4_ptx.cuh"

namespace q4 {

constexpr int BM = 128;                 // packed rows per tile
constexpr int BN = 128;                 // keys per block
constexpr float NEG_INF = -INFINITY;
constexpr float GROW = 8.0f;            // log2 of how far a score may pass the reference before the sums are rescaled

// log2 of what the weights, rounded to T for the second product, are taken by.  bfloat16 has
// exponents enough.  binary16 ends at 2^-24 and the sum does not: lifted to just below its
// largest numbers, a weight of 2^-b of the reference's keeps all its bits for b <= 21 and is off by
// 2^-32 at most below that.  Four binades more, with GROW = 4, would cost 5 to 9% where scores
// are sharp (four times the spread), as sums are rescaled more often; the lift itself costs nothing.
template <typename T>
constexpr float LIFT = std::is_same<T, __nv_bfloat16>::value ? 0.0f : 7.0f;

// References of this size (in units of log2) and above have steps that a weight would show:
// a score's product with the scale less its own rounding is not 0 (past 2^24 it may be 2 to
// any power).  Such a row is "far": its reference is a score, which is taken off the others, in
// tensor memory, before the product.  All of a far row's blocks call for another
// reference, so that this is done where sums are rescaled and costs the others nothing; a
// subtraction or a choice in the weights' own loop would cost every block 2 to 3%.
constexpr float FAR = 0x1p12f;

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Barrier of a tile's 256 softmax threads; with a vote: whether any says yes.
__device__ __forceinline__ void tile_sync(int t) { asm volatile("bar.sync %0, 256;" ::"r"(1 + t) : "memory"); }
__device__ __forceinline__ bool tile_vote(int t, bool yes) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %2, 0;\n\t"
      "bar.red.or.pred q, %1, 256, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(1 + t), "r"((uint32_t)yes)
      : "memory");
  return any != 0;
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// Whether eight 16-bit values hold an infinity or a NaN: an exponent of all
// ones carries into the sign's place when one is added.
template <typename T>
__device__ __forceinline__ bool nonfinite8(const uint4& v) {
  constexpr uint32_t E = std::is_same<T, __half>::value ? 0x7C007C00u : 0x7F807F80u;
  constexpr uint32_t ONE = std::is_same<T, __half>::value ? 0x04000400u : 0x00800080u;
  return ((((v.x & E) + ONE) | ((v.y & E) + ONE) | ((v.z & E) + ONE) | ((v.w & E) + ONE)) & 0x80008000u) != 0;
}

// Sixteen 16-bit values.  A thread's rows are not its neighbours', so a store
// costs as many cycles as it has lanes; 32 bytes at once halve their number.
__device__ __forceinline__ void store16(void* p, const uint32_t (&v)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  } else {
    static_cast<uint4*>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    static_cast<uint4*>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

// A pair with infinities and NaN replaced by 0.
template <typename T>
__device__ __forceinline__ uint32_t finite2(uint32_t w) {
  constexpr uint32_t E = std::is_same<T, __half>::value ? 0x7C00u : 0x7F80u;
  if ((w & E) == E) w &= 0xFFFF0000u;
  if (((w >> 16) & E) == E) w &= 0x0000FFFFu;
  return w;
}

// ---- host ----
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeFn encode_fn() {
  static std::atomic<void*> fn{nullptr};
  void* p = fn.load();
  if (!p) {
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) !=
            cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      return nullptr;
    fn.store(p);
  }
  return reinterpret_cast<EncodeFn>(p);
}

// Map of rows x heads x D values; a box is `positions` rows of `group` heads of 64 values.
inline bool make_rows_map(CUtensorMap* map, bool bf16, const void* p, int64_t rows, int64_t heads, int D, const int64_t* st,
              int group, int positions) {
  const EncodeFn encode = encode_fn();
  if (!encode) return false;
  // a stride is not used where there is one row or one head
  const cuuint64_t head_st = heads == 1 ? (cuuint64_t)D * 2 : (cuuint64_t)st[1] * 2;
  const cuuint64_t row_st = rows == 1 ? (cuuint64_t)D * 2 * heads : (cuuint64_t)st[0] * 2;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {head_st, row_st};
  const cuuint32_t box[3] = {64, (cuuint32_t)group, (cuuint32_t)positions};
  const cuuint32_t elem[3] = {1, 1, 1};
  return encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                const_cast<void*>(p), dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace q4
