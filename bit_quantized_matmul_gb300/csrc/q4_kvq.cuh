// q4_kvq.cuh — device layout of the 4-bit KV cache and the small helpers its
// kernels share (not part of the public ABI).
//
// Layout.  A (slot, head) plane is a run of tiles of 32 positions (4,608 bytes
// at D = 128, 2,304 at D = 64); a tile holds, one after another,
//   K codes   32 rows of D/2 bytes      K scales  32 x D/32 binary16
//   V codes   32 rows of D/2 bytes      V scales  32 x D/32 binary16
// so a warp fetches one tile with one bulk copy, and the K half alone is one
// copy too.  Codes are the nibbles q = 0..15 of the Q4_0 rule; block b of a
// row (32 values) is four words, word j holding values 8j .. 8j+7 from the low
// nibble up.
//
// K row: word j of block b sits at byte j*4*NB + 4b (NB = D/32).  In an
// m16n8k16 product with keys along n, lane 4g + tq feeds key g with the words
// j = tq, which are then contiguous; the lanes of a warp read the rows of
// eight keys in address order.  Which value sits at which k index does not
// matter as long as the query fragment agrees.
// V: half-word g (values 4g .. 4g+3 of a block) of block b of two neighbouring
// positions is one word, the even position in its low half, and the words of
// eight positions are stored as [g][pair][b]: lane (g, tq) of the P V product,
// with values along m and keys along k, reads the two keys 2 tq, 2 tq + 1 of
// each register ready made, and the warp again reads in address order.
// Scales are stored by pairs of positions too: [r / 2][block][r % 2].
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "q4mm_internal.h"

namespace q4 {

template <int D>
struct Kvq {
  static constexpr int NB = D / 32;                       // blocks (scales) per row
  static constexpr int POS = KVQ_POS;                     // positions per tile
  static constexpr int ROW = D / 2;                       // code bytes per row
  static constexpr int SCL = 2 * NB;                      // scale bytes per row
  static constexpr int KS_OFF = POS * ROW;                // K scales
  static constexpr int V_OFF = KS_OFF + POS * SCL;        // V codes (= bytes of the K half)
  static constexpr int VS_OFF = V_OFF + POS * ROW;        // V scales
  static constexpr int BYTES = VS_OFF + POS * SCL;        // one tile
};

// Byte offset in a tile of word j (values 8j .. 8j+7) of block b of position r's K.
template <int D>
__device__ __forceinline__ int kvq_k_word(int r, int b, int j) {
  return r * Kvq<D>::ROW + (j * Kvq<D>::NB + b) * 4;
}

// Byte offset in a tile of the words of group g of positions r and r ^ 1.
template <int D>
__device__ __forceinline__ int kvq_v_group(int r, int g) {
  return Kvq<D>::V_OFF + (r >> 3) * 8 * Kvq<D>::ROW + (4 * g + ((r >> 1) & 3)) * Kvq<D>::NB * 4;
}

// Byte offset in a tile of half-word g (values 4g .. 4g+3) of block b of position r's V.
template <int D>
__device__ __forceinline__ int kvq_v_half(int r, int b, int g) {
  return kvq_v_group<D>(r, g) + b * 4 + (r & 1) * 2;
}

// Byte offset in a tile of the scale of block b of position r.
template <int D>
__device__ __forceinline__ int kvq_scale(int kv, int r, int b) {
  return (kv ? Kvq<D>::VS_OFF : Kvq<D>::KS_OFF) + (((r >> 1) * Kvq<D>::NB + b) * 2 + (r & 1)) * 2;
}

// Loads of what a call is given.  EARLY: the kernel is launched early, so an earlier
// launch may be writing the address while the kernel lives.  It waits before it reads, and
// the wait makes those writes visible to ordinary loads, but not to the read-only path:
// so the step's description, which every warp reads again, comes by a load that
// the compiler cannot turn into one of those (from the L2 each time, eight positions
// a warp read for 32 requests would take 25 us longer), rows that are read once from the L2.
template <bool EARLY>
__device__ __forceinline__ int32_t kvq_ld(const int32_t* p) {
  if constexpr (EARLY) {
    int32_t v;
    asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
  } else {
    return __ldg(p);
  }
}
template <bool EARLY, typename V>
__device__ __forceinline__ V kvq_ld_row(const V* p) {
  if constexpr (EARLY) return __ldcg(p);
  else return __ldg(p);
}

// The request whose packed rows contain row t, found by a whole warp: the last s
// with offsets[s] <= t (offsets are expected to be non-decreasing; callers check
// the result).  32 offsets a round: a search by halves would wait for memory
// log2(S) times.
template <bool EARLY>
__device__ __forceinline__ int kvq_find_request(const int32_t* offsets, int S, int64_t t, int lane) {
  int lo = 0, n = S;  // the answer lies in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32, at = lo + lane * step;
    const bool below = lane * step < n && (int64_t)kvq_ld<EARLY>(offsets + at) <= t;
    const unsigned hit = __ballot_sync(0xFFFFFFFFu, below) | 1u;
    const int k = 31 - __clz(hit);
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

// Request s of a step: its packed rows [b, e), slot and first position.
struct KvqRequest {
  int64_t b, e, slot, pos;
  // rows that fit the packed step, the cache and a slot of it
  __device__ __forceinline__ bool ok(int64_t total, int64_t slots, int64_t capacity) const {
    return b >= 0 && e >= b && e <= total && slot >= 0 && slot < slots && pos >= 0 && pos + (e - b) <= capacity;
  }
};

template <bool EARLY>
__device__ __forceinline__ KvqRequest kvq_request(const int32_t* offsets, const int32_t* slot, const int32_t* pos,
                                                  int s) {
  return {kvq_ld<EARLY>(offsets + s), kvq_ld<EARLY>(offsets + s + 1), kvq_ld<EARLY>(slot + s), kvq_ld<EARLY>(pos + s)};
}

// The operand registers of a word of codes: exact binary16 pairs q - 8 of
// nibbles (0, 4), (1, 5), (2, 6) and (3, 7), as 1024 + q less 1032, or
// (1024 + 16 q) / 16 less 72.
__device__ __forceinline__ void kvq_unpack_centred(uint32_t w, uint32_t (&r)[4]) {
  const __half2 k1032 = __float2half2_rn(-1032.0f), k72 = __float2half2_rn(-72.0f), k16 = __float2half2_rn(0.0625f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t v = i < 2 ? w : w >> 8;
    const uint32_t x = (v & ((i & 1) ? 0x00F000F0u : 0x000F000Fu)) | 0x64006400u;
    const __half2 h = *reinterpret_cast<const __half2*>(&x);
    const __half2 y = (i & 1) ? __hfma2(h, k16, k72) : __hadd2(h, k1032);
    r[i] = *reinterpret_cast<const uint32_t*>(&y);
  }
}

// Eight consecutive elements as fp32 (16-byte aligned).
template <bool EARLY>
__device__ __forceinline__ void kvq_load8(const float* p, float (&v)[8]) {
  const float4 a = kvq_ld_row<EARLY>(reinterpret_cast<const float4*>(p));
  const float4 b = kvq_ld_row<EARLY>(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
template <bool EARLY>
__device__ __forceinline__ void kvq_load8(const __half* p, float (&v)[8]) {
  const uint4 a = kvq_ld_row<EARLY>(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
template <bool EARLY>
__device__ __forceinline__ void kvq_load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 a = kvq_ld_row<EARLY>(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// Eight consecutive elements from fp32, rounded once (16-byte aligned).
__device__ __forceinline__ void kvq_store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void kvq_store8(__half* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void kvq_store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Four consecutive elements from fp32, rounded once (8-byte aligned, 16 for fp32).
template <typename T>
__device__ __forceinline__ void kvq_store4(T* p, const float (&v)[4]) {
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
    const T h[4] = {(T)v[0], (T)v[1], (T)v[2], (T)v[3]};
    *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(h);
  }
}

}  // namespace q4
