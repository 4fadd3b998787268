// q4_prompt.cu — attention over packed prompts on the tensor cores.
//
//   o[i] = sum_{j <= lim(i)} softmax_j(scale q_i . k_j) v_j,
//   lim(i) = i + klen - qlen (causal) or klen - 1, per sequence and head.
//
// Bound by the tensor cores: 4 D flops per visible pair and query head, in
// 16-bit operands with fp32 accumulators.  The G query heads that share a
// key/value head are packed with the positions into the 128 rows of a tile
// (row r = position r / G, head r % G of the group): a tile has 128 useful
// rows (126 for G = 7) even when a sequence has only a few positions, K and V
// are fetched once for the whole group, and the causal edge is only 128 / G
// positions wide.
//
// A CTA takes two such tiles, one after another in a sequence, against key
// blocks of 128.  Roles (384 threads, three warpgroups):
//   warps 0-3, 4-7  softmax of tile 0 / tile 1: a thread owns one row, so its
//                   maximum and sum need no exchange.  S comes from tensor
//                   memory, the weights go back over it as 16-bit values (the A
//                   operand of the second product), and the accumulator O
//                   stays in tensor memory.  O is rescaled only when a row's
//                   maximum has grown by more than 2^8 since the last time:
//                   the factor is kept in the sum as well, so the result is
//                   the same softmax.
//   warp 8          copies Q, and K and V through a ring of blocks, by TMA
//                   tensor maps with the 128-byte swizzle
//   warp 9          issues the products: S of one tile while the other tile's
//                   softmax runs
// The launch gives each thread 168 registers; the softmax warpgroups take 224
// and leave the third 56 (2 * 224 + 56 = 3 * 168), so a row of scores stays in
// registers.  Weights are handed over in two halves, so the second product
// starts while the second half is computed.
// The products of a CTA run in order, so when S of block i + 1 is there, the
// accumulation of block i is done and O may be rescaled without a wait.
//
// Masked places.  Scores past a row's limit are replaced, not added to.  A
// weight of 0 times a NaN of V would still be NaN, so in blocks where some row
// has such a limit warp 8 clears what V holds past the sequence, and sets
// aside infinities and NaN of rows that only some of the tile's rows see (they
// are added back at the end to the rows that do see them).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <type_traits>

#include "q4_ptx.cuh"
#include "q4mm_internal.h"

namespace q4 {
namespace {

constexpr int BM = 128;                 // packed rows per tile
constexpr int BN = 128;                 // keys per block
constexpr int TMA_WARP = 8, MMA_WARP = 9;
constexpr int THREADS = 384;
constexpr int TMEM_COLS = 512;
constexpr float NEG_INF = -INFINITY;
constexpr float RESCALE = 8.0f;         // log2 of the growth that triggers a rescale

template <int D>
struct Cfg {
  static constexpr int CHUNKS = D / 64;                 // 128-byte column chunks of a row
  static constexpr int CHUNK = BN * 128;                // bytes of one chunk of a tile (16 KB)
  static constexpr int TILE = CHUNKS * CHUNK;           // one Q tile, K block or V block
  static constexpr int STAGES = D == 128 ? 4 : 8;       // K, V blocks in the ring (even: K and V alternate)
  static constexpr int BAR_OFF = (2 + STAGES) * TILE;
  static constexpr int SMEM = BAR_OFF + 512 + 1024;     // + alignment slack
  static constexpr int O_COL = 2 * BN;                  // S0, S1, then O0, O1
};

struct Args {
  const void *v;
  void* out;
  int64_t v_row, v_head;  // strides of v in elements
  int64_t q_total, k_total;
  int q_heads, kv_heads, group, positions;  // positions per tile
  int S, causal, ctas;
  float scale_log2;
  const int32_t *q_offsets, *k_offsets;
  unsigned* status;
  unsigned long long wait_ns;
};

struct Seq {
  int qb, qlen, kb, klen;
};

__device__ __forceinline__ bool load_seq(const Args& a, int s, Seq* q) {
  const int qb = __ldg(a.q_offsets + s), qe = __ldg(a.q_offsets + s + 1);
  const int kb = __ldg(a.k_offsets + s), ke = __ldg(a.k_offsets + s + 1);
  *q = Seq{qb, qe - qb, kb, ke - kb};
  return qb >= 0 && qe >= qb && qe <= a.q_total && kb >= 0 && ke >= kb && ke <= a.k_total;
}

// What a CTA works on.
struct Work {
  int ok;       // 0: nothing
  int pos0;     // first position of tile 0 in the sequence
  Seq q;
};

// The CTA's pair of tiles: pair `index` of all sequences' pairs, counted from
// the last one back (the longest causal rows first).
__device__ void find_work(const Args& a, int index, Work* out) {
  __shared__ int warp_sum[THREADS / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int step = 2 * a.positions;
  const int chunk = (a.S + THREADS - 1) / THREADS;
  const int s0 = min(a.S, tid * chunk), s1 = min(a.S, s0 + chunk);
  int mine = 0;
  bool bad = false;
  for (int s = s0; s < s1; ++s) {
    Seq q;
    if (load_seq(a, s, &q)) mine += (q.qlen + step - 1) / step;
    else bad = true;
  }
  if (bad && blockIdx.x == 0 && blockIdx.y == 0) atomicOr(a.status, STATUS_KV_RANGE);
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_sum[warp] = incl;
  if (tid == 0) out->ok = 0;
  __syncthreads();
  int base = 0, all = 0;
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) base += warp_sum[w];
    all += warp_sum[w];
  }
  const int want = all - 1 - index;
  int start = base + incl - mine;
  if (want >= start && want < start + mine) {
    for (int s = s0; s < s1; ++s) {
      Seq q;
      if (!load_seq(a, s, &q)) continue;
      const int n = (q.qlen + step - 1) / step;
      if (want < start + n) {
        *out = Work{1, (want - start) * step, q};
        break;
      }
      start += n;
    }
  }
  __syncthreads();
}

// Rows that belong to no sequence, or to one that is out of range, are zero.
template <int D, typename T>
__device__ void clear_rows(const Args& a) {
  const int64_t row = (int64_t)a.q_heads * D * sizeof(T) / 16;  // 16-byte vectors of a packed row
  auto clear = [&](int64_t r0, int64_t r1) {
    uint4* p = static_cast<uint4*>(a.out);
    r0 = r0 < 0 ? 0 : r0;
    r1 = r1 > a.q_total ? a.q_total : r1;
    for (int64_t i = r0 * row + threadIdx.x; i < r1 * row; i += blockDim.x) p[i] = make_uint4(0u, 0u, 0u, 0u);
  };
  clear(0, a.q_offsets[0]);
  clear(a.q_offsets[a.S], a.q_total);
  for (int s = 0; s < a.S; ++s) {
    Seq q;
    if (!load_seq(a, s, &q)) clear(q.qb, (int64_t)q.qb + q.qlen);
  }
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
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

// Whether a pair of 16-bit values holds an infinity or a NaN.
template <typename T>
__device__ __forceinline__ bool nonfinite2(uint32_t w) {
  constexpr uint32_t E = std::is_same<T, __half>::value ? 0x7C00u : 0x7F80u;
  return (w & E) == E || ((w >> 16) & E) == E;
}

// A pair with infinities and NaN replaced by 0.
template <typename T>
__device__ __forceinline__ uint32_t finite2(uint32_t w) {
  constexpr uint32_t E = std::is_same<T, __half>::value ? 0x7C00u : 0x7F80u;
  if ((w & E) == E) w &= 0xFFFF0000u;
  if (((w >> 16) & E) == E) w &= 0x0000FFFFu;
  return w;
}

template <int D, typename T>
__global__ void __launch_bounds__(THREADS, 1)
    prompt_kernel(const Args a, const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v) {
  using C = Cfg<D>;
  constexpr bool BF16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr int NST = C::STAGES, NV = NST / 2;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Work work;
  __shared__ int s_err, s_nonfinite;
  __shared__ uint32_t s_tmem;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  if ((int)blockIdx.x == a.ctas) {
    if (blockIdx.y == 0) clear_rows<D, T>(a);
    return;
  }
  find_work(a, blockIdx.x, &work);
  if (!work.ok) return;
  const Seq sq = work.q;
  const int head = blockIdx.y;
  const int G = a.group, P = a.positions;
  // the last key that a position sees, and the key blocks of each tile
  const int shift = a.causal ? sq.klen - sq.qlen : 0;
  auto limit = [&](int pos) { return a.causal ? pos + shift : sq.klen - 1; };
  int blocks[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int p0 = work.pos0 + t * P;
    const int last = limit(min(p0 + P, sq.qlen) - 1);
    blocks[t] = p0 < sq.qlen && last >= 0 ? last / BN + 1 : 0;
  }
  const int nblocks = max(blocks[0], blocks[1]);
  // blocks from here on hold keys that some row of the CTA does not see
  const int first_hidden = max(0, min(limit(work.pos0) + 1, sq.klen));
  const int zone = first_hidden / BN;  // beyond the last block when nothing is hidden

  const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem_p = smem_raw + (smem - smem_u32(smem_raw));
  const uint32_t q_smem = smem, ring = smem + 2 * C::TILE, bars = smem + C::BAR_OFF;
  const uint32_t q_full = bars, full = bars + 8, empty = full + 8 * NST, fixed = empty + 8 * NST;
  const uint32_t s_full = fixed + 8 * NST, p_full = s_full + 16, o_full = p_full + 32, drain = o_full + 16;
  volatile int* err = &s_err;
  if (tid == 0) {
    mbar_init(q_full, 1);
    mbar_init(drain, 1);
    for (int i = 0; i < NST; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 1);
      mbar_init(fixed + 8 * i, 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(s_full + 8 * t, 1);
      mbar_init(p_full + 16 * t, 4);
      mbar_init(p_full + 16 * t + 8, 4);
      mbar_init(o_full + 8 * t, 1);
    }
    s_err = 0;
    s_nonfinite = 0;
    mbar_init_fence();
  }
  if (warp == MMA_WARP) tmem_alloc(smem_u32(&s_tmem), TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;

  if (warp >= TMA_WARP) {
  fewer_registers<56>();
  if (warp == TMA_WARP) {
    // ---------------- copies ----------------
    int issued = 0;
    if (lane == 0 && nblocks > 0) {
      uint32_t bytes = 0;
      for (int t = 0; t < 2; ++t)
        if (blocks[t]) bytes += (uint32_t)(C::CHUNKS * P * G * 128);
      mbar_expect_tx(q_full, bytes);
      for (int t = 0; t < 2; ++t)
        if (blocks[t])
          for (int c = 0; c < C::CHUNKS; ++c)
            tensor_load(q_smem + t * C::TILE + c * C::CHUNK, &map_q, 64 * c, head * G, sq.qb + work.pos0 + t * P,
                        q_full);
    }
    bool ok = true;
    for (int i = 0; i < nblocks && ok; ++i) {
      for (int kv = 0; kv < 2 && ok; ++kv) {
        const int n = 2 * i + kv, st = n % NST;
        if (lane == 0) {
          if (n >= NST) ok = mbar_wait(empty + 8 * st, ((n / NST) - 1) & 1, err, a.wait_ns);
          if (ok) {
            mbar_expect_tx(full + 8 * st, C::TILE);
            for (int c = 0; c < C::CHUNKS; ++c)
              tensor_load(ring + st * C::TILE + c * C::CHUNK, kv ? (const void*)&map_v : (const void*)&map_k, 64 * c,
                          head, sq.kb + i * BN, full + 8 * st);
          }
        }
        ok = __shfl_sync(0xFFFFFFFFu, (int)ok, 0) != 0;
        if (ok) issued = n + 1;
      }
      if (ok && i >= zone) {  // make V safe to multiply with weights of 0
        const int n = 2 * i + 1, st = n % NST;
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(full + 8 * st, (n / NST) & 1, err, a.wait_ns));
        if (!ok) break;
        const int r0 = max(0, first_hidden - i * BN), end = min(BN, sq.klen - i * BN);
        uint8_t* vb = smem_p + (ring - smem) + st * C::TILE;
        bool found = false;
        for (int it = lane; it < (BN - r0) * C::CHUNKS * 8; it += 32) {
          const int row = r0 + it / (C::CHUNKS * 8), e = it % (C::CHUNKS * 8);
          uint4* p = reinterpret_cast<uint4*>(vb + (e >> 3) * C::CHUNK + row * 128 + ((e & 7) ^ (row & 7)) * 16);
          if (row >= end) {
            *p = make_uint4(0u, 0u, 0u, 0u);
          } else {
            const uint4 v = *p;
            if (nonfinite2<T>(v.x) || nonfinite2<T>(v.y) || nonfinite2<T>(v.z) || nonfinite2<T>(v.w)) {
              found = true;
              *p = make_uint4(finite2<T>(v.x), finite2<T>(v.y), finite2<T>(v.z), finite2<T>(v.w));
            }
          }
        }
        if (found) atomicExch(&s_nonfinite, 1);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(fixed + 8 * st);
      }
    }
    // the copies in flight land before the CTA ends, also when another role has given up
    if (nblocks > 0) mbar_wait_warp(q_full, 0, a.wait_ns);
    for (int n = max(0, issued - NST); n < issued; ++n)
      mbar_wait_warp(full + 8 * (n % NST), (n / NST) & 1, a.wait_ns);
  } else if (warp == MMA_WARP) {
    // ---------------- products ----------------
    if (lane == 0 && nblocks > 0) {
      constexpr uint32_t ID_S = idesc_f16(BF16, BN, false), ID_O = idesc_f16(BF16, D, true);
      auto qk = [&](int t, int st) {  // S_t = Q_t K^T
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = (uint32_t)((k >> 2) * C::CHUNK + (k & 3) * 32);
          mma_ss(tmem + t * BN, desc_sw128(q_smem + t * C::TILE + off, 16, 1024),
                 desc_sw128(ring + st * C::TILE + off, 16, 1024), ID_S, k > 0);
        }
        mma_commit(s_full + 8 * t);
      };
      bool ok = mbar_wait(q_full, 0, err, a.wait_ns) && mbar_wait(full, 0, err, a.wait_ns);
      tc_fence_after();
      if (ok) {
        for (int t = 0; t < 2; ++t)
          if (blocks[t]) qk(t, 0);
        mma_commit(empty);
      }
      for (int i = 0; i < nblocks && ok; ++i) {
        const int nv = 2 * i + 1, sv = nv % NST, nk = nv + 1, sk = nk % NST;
        ok = mbar_wait(full + 8 * sv, (nv / NST) & 1, err, a.wait_ns);
        if (ok && i >= zone) ok = mbar_wait(fixed + 8 * sv, ((i - zone) / NV) & 1, err, a.wait_ns);
        if (ok && i + 1 < nblocks) ok = mbar_wait(full + 8 * sk, (nk / NST) & 1, err, a.wait_ns);
        for (int t = 0; t < 2 && ok; ++t) {
          if (i >= blocks[t]) continue;
#pragma unroll
          for (int h = 0; h < 2 && ok; ++h) {  // O_t += P_t V, a half of the keys at a time
            ok = mbar_wait(p_full + 16 * t + 8 * h, i & 1, err, a.wait_ns);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int k = h * BN / 32; k < (h + 1) * BN / 32; ++k)
              mma_ts(tmem + C::O_COL + t * D, tmem + t * BN + k * 8,
                     desc_sw128(ring + sv * C::TILE + k * 2048, C::CHUNK, 1024), ID_O, i > 0 || k > 0);
          }
          if (!ok) break;
          if (i + 1 < blocks[t]) qk(t, sk);
          else mma_commit(o_full + 8 * t);
        }
        if (ok) {
          mma_commit(empty + 8 * sv);
          if (i + 1 < nblocks) mma_commit(empty + 8 * sk);
        }
      }
      if (!ok) {  // every product issued is done before tensor memory is freed
        mma_commit(drain);
        const unsigned long long t0 = globaltimer();
        while (!mbar_try(drain, 0) && globaltimer() - t0 < a.wait_ns) {}
      }
    }
    __syncwarp();
  }
  } else {
    more_registers<224>();
    // ---------------- softmax ----------------
    const int t = warp >> 2;
    const int r = tid & 127;
    const int pos = work.pos0 + t * P + r / G;
    const bool live = r < P * G && pos < sq.qlen;
    const int lim = live ? limit(pos) : -1;
    // keys up to here are seen by every live row of the warp (rows are in position order)
    const int first_row = (warp & 3) * 32;
    const int clear = limit(min(work.pos0 + t * P + first_row / G, sq.qlen - 1));
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_addr = tmem + lanes + t * BN, o_addr = tmem + lanes + C::O_COL + t * D;
    float m = NEG_INF, l = 0.0f;  // in units of log2, scaled
    bool ok = true;
    for (int i = 0; i < blocks[t]; ++i) {
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(s_full + 8 * t, i & 1, err, a.wait_ns));
      if (!ok) break;
      tc_fence_after();
      uint32_t s[128];
      tmem_ld32<0>(s_addr, s);
      tmem_ld32<32>(s_addr + 32, s);
      tmem_ld32<64>(s_addr + 64, s);
      tmem_ld32<96>(s_addr + 96, s);
      tmem_wait_ld();
      if ((i + 1) * BN - 1 > clear) {
        const int seen = lim - i * BN;  // columns up to here
#pragma unroll
        for (int c = 0; c < BN; ++c) s[c] = c <= seen ? s[c] : __float_as_uint(NEG_INF);
      }
      float top[4] = {NEG_INF, NEG_INF, NEG_INF, NEG_INF};
#pragma unroll
      for (int c = 0; c < BN; c += 2)
        top[(c >> 1) & 3] = max3(top[(c >> 1) & 3], __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
      float mn = max3(fmaxf(top[0], top[1]), top[2], top[3]);
      mn *= a.scale_log2;  // positive: checked on the host
      if (i == 0) {
        m = mn;
      } else if (__any_sync(0xFFFFFFFFu, mn > m + RESCALE)) {
        const float nm = fmaxf(m, mn);
        const float f = m == NEG_INF ? 0.0f : ex2(m - nm);
        m = nm;
        l *= f;
#pragma unroll
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          tmem_ld32<0>(o_addr + c, o);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
          tmem_st32<0>(o_addr + c, o);
        }
      }
      const float mm = m == NEG_INF ? 0.0f : m;
      const F2 sc2 = f2(a.scale_log2, a.scale_log2), mm2 = f2(-mm, -mm);
      F2 sum[2] = {f2(0.0f, 0.0f), f2(0.0f, 0.0f)};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int c = h * BN / 2; c < (h + 1) * BN / 2; c += 2) {
          const float2 x = unf2(fma2(f2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), sc2, mm2));
          const float p0 = ex2(x.x), p1 = ex2(x.y);
          sum[(c >> 1) & 1] = add2(sum[(c >> 1) & 1], f2(p0, p1));
          s[c / 2] = pack2<T>(p0, p1);
        }
        if (h == 0) tmem_st32<0>(s_addr, s);
        else tmem_st32<32>(s_addr + 32, s);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + 16 * t + 8 * h);
      }
      const float2 l2 = unf2(add2(sum[0], sum[1]));
      l += l2.x + l2.y;
    }
    // ---- O / l to memory ----
    const int hq = head * G + r % G;
    T* dst = static_cast<T*>(a.out) + ((int64_t)(sq.qb + pos) * a.q_heads + hq) * D;
    if (blocks[t] == 0) {
      if (live)
        for (int c = 0; c < D; c += 8) *reinterpret_cast<uint4*>(dst + c) = make_uint4(0u, 0u, 0u, 0u);
    } else if (ok) {
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(o_full + 8 * t, 0, err, a.wait_ns));
      if (ok) {
        tc_fence_after();
        const float inv = lim < 0 ? 0.0f : 1.0f / l;
        const bool extra = s_nonfinite != 0;
#pragma unroll
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          tmem_ld32<0>(o_addr + c, o);
          tmem_wait_ld();
          float x[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) x[e] = lim < 0 ? 0.0f : __uint_as_float(o[e]) * inv;
          if (live) {
            if (extra) {  // what was set aside: keys that this row sees
              const T* v = static_cast<const T*>(a.v) + (int64_t)head * a.v_head + c;
              for (int j = first_hidden; j <= lim; ++j)
                for (int e = 0; e < 32; ++e) {
                  const float f = (float)v[(int64_t)(sq.kb + j) * a.v_row + e];
                  if (!isfinite(f)) x[e] += f;
                }
            }
#pragma unroll
            for (int e = 0; e < 32; e += 8)
              *reinterpret_cast<uint4*>(dst + c + e) =
                  make_uint4(pack2<T>(x[e], x[e + 1]), pack2<T>(x[e + 2], x[e + 3]), pack2<T>(x[e + 4], x[e + 5]),
                             pack2<T>(x[e + 6], x[e + 7]));
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == MMA_WARP) tmem_dealloc(tmem, TMEM_COLS);
  if (tid == 0 && s_err) atomicOr(a.status, STATUS_TIMEOUT);
}

// ---------------------------------------------------------------- host
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
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
bool make_map(CUtensorMap* map, bool bf16, const void* p, int64_t rows, int64_t heads, int D, const int64_t* st,
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

template <int D, typename T>
int launch_as(const PromptAttn& c, cudaStream_t s) {
  constexpr bool BF16 = std::is_same<T, __nv_bfloat16>::value;
  Args a;
  a.v = c.v;
  a.out = c.out;
  a.v_row = c.v_strides[0];
  a.v_head = c.v_strides[1];
  a.q_total = c.q_total;
  a.k_total = c.k_total;
  a.q_heads = c.q_heads;
  a.kv_heads = c.kv_heads;
  a.group = c.q_heads / c.kv_heads;
  a.positions = BM / a.group;
  a.S = c.S;
  a.causal = c.causal;
  a.scale_log2 = c.scale * 1.44269504088896340736f;
  a.q_offsets = c.q_offsets;
  a.k_offsets = c.k_offsets;
  a.status = c.status;
  a.wait_ns = wait_limit_ns();
  // pairs of tiles: whole ones and at most one ragged per sequence
  const int64_t ctas = c.q_total / (2 * a.positions) + (c.S < c.q_total ? c.S : c.q_total);
  if (ctas >= INT32_MAX) return Q4_ERR_SHAPE;
  a.ctas = (int)ctas;
  CUtensorMap mq, mk, mv;
  // without keys nothing is read from k and v: any valid map will do
  const bool keys = c.k_total > 0;
  if (!make_map(&mq, BF16, c.q, c.q_total, c.q_heads, D, c.q_strides, a.group, a.positions) ||
      !make_map(&mk, BF16, keys ? c.k : c.q, keys ? c.k_total : 1, keys ? c.kv_heads : 1, D, c.k_strides, 1, BN) ||
      !make_map(&mv, BF16, keys ? c.v : c.q, keys ? c.k_total : 1, keys ? c.kv_heads : 1, D, c.v_strides, 1, BN))
    return Q4_ERR_INVALID_ARG;
  static std::atomic<bool> sized[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return Q4_ERR_CUDA;
  if (!sized[dev].load()) {
    if (cudaFuncSetAttribute(prompt_kernel<D, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::SMEM) !=
        cudaSuccess)
      return Q4_ERR_CUDA;
    sized[dev].store(true);
  }
  prompt_kernel<D, T><<<dim3((unsigned)ctas + 1, c.kv_heads), THREADS, Cfg<D>::SMEM, s>>>(a, mq, mk, mv);
  return cudaGetLastError() == cudaSuccess ? Q4_OK : Q4_ERR_CUDA;
}

}  // namespace

int launch_prompt_attention(const PromptAttn& c, cudaStream_t s) {
  if (c.dtype == Q4_DTYPE_F16)
    return c.head_dim == 128 ? launch_as<128, __half>(c, s) : launch_as<64, __half>(c, s);
  return c.head_dim == 128 ? launch_as<128, __nv_bfloat16>(c, s) : launch_as<64, __nv_bfloat16>(c, s);
}

}  // namespace q4
