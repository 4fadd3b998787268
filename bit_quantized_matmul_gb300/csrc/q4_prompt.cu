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
// blocks of 128; when it is done with them it takes over a pair of tiles that
// another CTA of the launch was to do and has not begun (the longest come
// first), so that the copies and first products of one pair run under the end
// of the last one.  Roles (640 threads, five warpgroups):
//   warps 0-15  softmax: warpgroups 0 and 1 have the two halves of tile 0's key
//               columns, 2 and 3 those of tile 1; a thread owns half a row.  S
//               comes from tensor memory, the weights go back over it as 16-bit
//               values (the A operand of the second product), and the
//               accumulator O stays in tensor memory.  The scores are taken
//               relative to a reference, the row's maximum of some earlier
//               block; only when a score passes it by more than 2^8 do the
//               halves exchange their maxima and rescale O (the sum keeps the
//               factor, so the result is the same softmax).  One barrier with a
//               vote per block tells both halves.
//   warp 16     finds the work and copies Q, and K and V through a ring of
//               blocks, by TMA tensor maps with the 128-byte swizzle
//   warps 17,18 issue the products of tile 0 / tile 1, S of one tile while the
//               other tile's softmax runs; the second product of a half of the
//               keys starts when its weights are there
//   warp 19     looks after masked places in V (below)
// The launch gives each thread 96 registers; the softmax warpgroups take 104
// and leave the fifth 64 (4 * 104 + 64 = 5 * 96).
// The products of a tile run in order, so when S of block i + 1 is there, the
// accumulation of block i is done and O may be rescaled without a wait.
//
// Measured (28/4 heads of 128, in a graph): a bf16 prompt of 16,384 rows takes 1.19 ms,
// 1,617 TFLOP/s, over the same inputs again, 1.21 to 1.29 ms over others in turn and
// 1.29 when it is called without a pause (1,490: the clock gives way); one of 4,096
// rows 102 us, 1,180 TFLOP/s (tensor pipe 59% busy, issue slots 43%, exponentials 30%);
// nine fp16 prompts of 15,374 rows 197 us, 1,042 TFLOP/s.  Scores of four times the
// spread, whose sums are rescaled more often, cost 5 to 9% more.
// What is lost there is the ends: a pair's first scores and its last output
// have no other product beside them, about 1.5 us a pair.  Issuing a product
// from one lane's registers instead of the warp's uniform ones cost a fifth
// (1.46 ms), clearing rows by looking through them 3%, 16-byte output stores 5% of
// the packed prompts.
//
// Masked places.  Scores past a row's limit are replaced, not added to.  A
// weight of 0 times a NaN of V would still be NaN, so in blocks where some row
// has such a limit warp 19 clears the rows of V that no row sees, and sets
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
constexpr int SOFTMAX_WARPS = 16;
constexpr int TMA_WARP = 16, MMA_WARP = 17, FIX_WARP = 19;  // and MMA_WARP + 1
constexpr int WORKS = 2;                // the pair that is copied and the one before
constexpr int THREADS = 640;
constexpr int TMEM_COLS = 512;
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
  int S, causal;
  int wide;  // out is 32-byte aligned
  float scale_log2;
  const int32_t *q_offsets, *k_offsets;
  unsigned* status;
  unsigned long long wait_ns;
  int stall;  // test setting: no copy is issued, so every wait for one runs out
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

// A pair of tiles.
struct Work {
  int ok;       // 0: there is no more
  int head;
  int pos0;     // first position of tile 0 in the sequence
  Seq q;
};

// Finds pairs for the CTA, run by one warp.  Pairs are counted from the last
// one back (the longest causal rows of a sequence first).
struct Finder {
  Seq q;        // with at most 32 sequences: the lane's own
  int n, upto;  // its pairs, and all up to and with it
  int all;
  bool gaps;    // some rows belong to no sequence, or to one that is out of range
  __device__ __forceinline__ static int pairs(const Args& a, int s, Seq* q, bool* bad) {
    const int step = 2 * a.positions;
    *q = Seq{0, 0, 0, 0};
    if (s >= a.S) return 0;
    if (load_seq(a, s, q)) return (q->qlen + step - 1) / step;
    *bad = true;
    return 0;
  }
  __device__ __forceinline__ static int scan(int v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xFFFFFFFFu, v, o);
      if (lane >= o) v += x;
    }
    return v;
  }
  __device__ __forceinline__ void begin(const Args& a, int lane) {
    bool bad = false;
    all = 0;
    for (int s = 0; s < a.S; s += 32) {
      n = pairs(a, s + lane, &q, &bad);
      upto = scan(n, lane);
      all += __shfl_sync(0xFFFFFFFFu, upto, 31);
    }
    bad = __any_sync(0xFFFFFFFFu, bad);
    if (bad && lane == 0) atomicOr(a.status, STATUS_KV_RANGE);
    gaps = bad || (a.S > 0 && (__ldg(a.q_offsets) > 0 || __ldg(a.q_offsets + a.S) < a.q_total));
  }
  // pair `index` of one head; false when there is none.  Every lane gets it.
  __device__ __forceinline__ bool find(const Args& a, int index, int lane, Work* w) {
    const int want = all - 1 - index;
    if (want < 0) return false;
    int base = 0;
    for (int s = 0;; s += 32) {
      if (a.S > 32) {
        bool bad = false;
        n = pairs(a, s + lane, &q, &bad);
        upto = scan(n, lane);
      }
      const unsigned hit = __ballot_sync(0xFFFFFFFFu, want < base + upto);
      if (hit) {
        const int l = __ffs(hit) - 1;
        const int first = base + __shfl_sync(0xFFFFFFFFu, upto - n, l);
        w->q.qb = __shfl_sync(0xFFFFFFFFu, q.qb, l);
        w->q.qlen = __shfl_sync(0xFFFFFFFFu, q.qlen, l);
        w->q.kb = __shfl_sync(0xFFFFFFFFu, q.kb, l);
        w->q.klen = __shfl_sync(0xFFFFFFFFu, q.klen, l);
        w->pos0 = (want - first) * 2 * a.positions;
        w->ok = 1;
        return true;
      }
      base += __shfl_sync(0xFFFFFFFFu, upto, 31);
    }
  }
};

// What the roles derive from a pair.
struct Plan {
  int blocks[2];     // key blocks of each tile
  int nblocks;       // of the pair
  int first_hidden;  // the first key that some row does not see, klen when all are seen
  int seen_end;      // keys from here on are seen by no row
  int zone;          // blocks from here on hold such keys, or end past the sequence
  int shift;
  __device__ __forceinline__ int limit(const Args& a, const Work& w, int pos) const {
    return a.causal ? pos + shift : w.q.klen - 1;
  }
  __device__ __forceinline__ Plan(const Args& a, const Work& w) {
    shift = w.q.klen - w.q.qlen;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int p0 = w.pos0 + t * a.positions;
      const int last = limit(a, w, min(p0 + a.positions, w.q.qlen) - 1);
      blocks[t] = p0 < w.q.qlen && last >= 0 ? last / BN + 1 : 0;
    }
    nblocks = max(blocks[0], blocks[1]);
    seen_end = min(limit(a, w, min(w.pos0 + 2 * a.positions, w.q.qlen) - 1) + 1, w.q.klen);
    first_hidden = max(0, min(limit(a, w, w.pos0) + 1, w.q.klen));
    zone = first_hidden / BN;  // past the last block when nothing is hidden
  }
};

// Rows that belong to no sequence, or to one that is out of range, are zero:
// the share of one of `threads` threads.
template <int D, typename T>
__device__ void clear_rows(const Args& a, int64_t thread, int64_t threads) {
  const int64_t row = (int64_t)a.q_heads * D * sizeof(T) / 16;  // 16-byte vectors of a packed row
  auto clear = [&](int64_t r0, int64_t r1) {
    uint4* p = static_cast<uint4*>(a.out);
    r0 = r0 < 0 ? 0 : r0;
    r1 = r1 > a.q_total ? a.q_total : r1;
    for (int64_t i = r0 * row + thread; i < r1 * row; i += threads) p[i] = make_uint4(0u, 0u, 0u, 0u);
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

template <int D, typename T>
__global__ void __launch_bounds__(THREADS, 1)
    prompt_kernel(const Args a, const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v) {
  using C = Cfg<D>;
  constexpr bool BF16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr int NST = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Work work[WORKS];
  __shared__ __align__(16) uint4 taken;
  __shared__ int s_err, s_nonfinite[WORKS];
  __shared__ float s_max[2][2][BM], s_sum[2][2][BM];  // [tile][half][row]: what the halves exchange
  __shared__ uint32_t s_tmem;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);  // one value for the warp, as far as the compiler can see
  const int G = a.group, P = a.positions;

  const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem_p = smem_raw + (smem - smem_u32(smem_raw));
  const uint32_t q_smem = smem, ring = smem + 2 * C::TILE, bars = smem + C::BAR_OFF;
  const uint32_t q_full = bars, q_empty = q_full + 8, drain = q_empty + 8, answer = drain + 8;
  const uint32_t full = answer + 8, empty = full + 8 * NST, hidden = empty + 8 * NST, fixed = hidden + 8 * NST;
  const uint32_t s_full = fixed + 8 * NST, p_full = s_full + 16, o_full = p_full + 32, o_empty = o_full + 16;
  const uint32_t turn = o_empty + 16, work_full = turn + 16, work_empty = work_full + 8 * WORKS;
  volatile int* err = &s_err;
  if (tid == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 2);
    mbar_init(drain, 2);
    mbar_init(answer, 1);
    for (int i = 0; i < NST; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 2);
      mbar_init(hidden + 8 * i, 1);
      mbar_init(fixed + 8 * i, 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(s_full + 8 * t, 1);
      mbar_init(p_full + 16 * t, 4);
      mbar_init(p_full + 16 * t + 8, 4);
      mbar_init(o_full + 8 * t, 1);
      mbar_init(o_empty + 8 * t, 8);
      mbar_init(turn + 8 * t, 1);
    }
    for (int i = 0; i < WORKS; ++i) {
      mbar_init(work_full + 8 * i, 1);
      mbar_init(work_empty + 8 * i, SOFTMAX_WARPS + 3);  // and the products' and V's warps
      s_nonfinite[i] = 0;
    }
    mbar_arrive(turn);  // tile 0 begins
    s_err = 0;
    mbar_init_fence();
  }
  if (warp == MMA_WARP) tmem_alloc(smem_u32(&s_tmem), TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  // The roles go through the same pairs in the same order, each with its own
  // count of what it has waited for.  The next pair, false when there is none.
  auto next_work = [&](int nth, Work* w) {
    const bool ok = mbar_wait(work_full + 8 * (nth % WORKS), (nth / WORKS) & 1, err, a.wait_ns);
    if (!ok) return false;
    *w = work[nth % WORKS];
    return w->ok != 0;
  };

  // One pair's copies, by one warp: n blocks and nq Q pairs so far.
  auto copy_pair = [&](const Work& w, int& n, int& nq, bool& ok) {
    const Plan p(a, w);
    const Seq sq = w.q;
    if (p.nblocks > 0) {
      if (lane == 0) {
        if (nq > 0) ok = mbar_wait(q_empty, (nq - 1) & 1, err, a.wait_ns);
        if (ok && !a.stall) {
          uint32_t bytes = 0;
          for (int t = 0; t < 2; ++t)
            if (p.blocks[t]) bytes += (uint32_t)(C::CHUNKS * P * G * 128);
          mbar_expect_tx(q_full, bytes);
          for (int t = 0; t < 2; ++t)
            if (p.blocks[t])
              for (int c = 0; c < C::CHUNKS; ++c)
                tensor_load(q_smem + t * C::TILE + c * C::CHUNK, &map_q, 64 * c, w.head * G,
                            sq.qb + w.pos0 + t * P, q_full);
        }
      }
      ok = __shfl_sync(0xFFFFFFFFu, (int)ok, 0) != 0;
      if (ok) ++nq;
    }
    for (int i = 0; i < p.nblocks && ok; ++i) {
      for (int kv = 0; kv < 2 && ok; ++kv) {
        const int st = n % NST;
        if (lane == 0) {
          if (n >= NST) ok = mbar_wait(empty + 8 * st, ((n / NST) - 1) & 1, err, a.wait_ns);
          if (ok && !a.stall) {
            mbar_expect_tx(full + 8 * st, C::TILE);
            for (int c = 0; c < C::CHUNKS; ++c)
              tensor_load(ring + st * C::TILE + c * C::CHUNK, kv ? (const void*)&map_v : (const void*)&map_k,
                          64 * c, w.head, sq.kb + i * BN, full + 8 * st);
            if (kv && i >= p.zone) mbar_arrive(hidden + 8 * st);  // tells V's warp, which only waits for these
          }
        }
        ok = __shfl_sync(0xFFFFFFFFu, (int)ok, 0) != 0;
        if (ok) ++n;
      }
    }
  };

  if (warp >= TMA_WARP) {
    fewer_registers<64>();
    if (warp == TMA_WARP) {
      // ---------------- work and copies ----------------
      Finder f;
      f.begin(a, lane);
      int n = 0, nq = 0;  // blocks and Q pairs so far
      int nth = 0;        // pairs so far
      bool ok = true, more = true;
      uint32_t index = blockIdx.x;
      for (int asked = 0; ok && more; ++asked) {
        if (lane == 0) {  // the answer is wanted when this pair's copies are under way
          mbar_expect_tx(answer, 16);
          take_cta(smem_u32(&taken), answer);
        }
        __syncwarp();
        Work w;
        const bool found = f.find(a, (int)(index / a.kv_heads), lane, &w);
        w.head = (int)(index % a.kv_heads);
        if (f.gaps) clear_rows<D, T>(a, (int64_t)index * 32 + lane, (int64_t)gridDim.x * 32);
        if (found) {
          if (nth >= WORKS) {  // every role is done with the pair that had the slot
            const int v = nth - WORKS;
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(work_empty + 8 * (v % WORKS), (v / WORKS) & 1, err, a.wait_ns));
          }
          if (ok && lane == 0) {
            work[nth % WORKS] = w;
            s_nonfinite[nth % WORKS] = 0;
            mbar_arrive(work_full + 8 * (nth % WORKS));
          }
          __syncwarp();
          if (ok) copy_pair(w, n, nq, ok);
          ++nth;
        }
        if (!mbar_wait_warp(answer, asked & 1, a.wait_ns)) {
          *err = 1;
          break;
        }
        more = taken_cta(smem_u32(&taken), &index);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
      }
      if (ok && !more) {
        if (nth >= WORKS) {
          const int v = nth - WORKS;
          ok = __all_sync(0xFFFFFFFFu, mbar_wait(work_empty + 8 * (v % WORKS), (v / WORKS) & 1, err, a.wait_ns));
        }
        if (ok && lane == 0) {
          work[nth % WORKS].ok = 0;
          mbar_arrive(work_full + 8 * (nth % WORKS));
        }
      }
      // the copies in flight land before the CTA ends, also when another role has given up
      if (nq > 0) mbar_wait_warp(q_full, (nq - 1) & 1, a.wait_ns);
      for (int v = max(0, n - NST); v < n; ++v) mbar_wait_warp(full + 8 * (v % NST), (v / NST) & 1, a.wait_ns);
    } else if (warp == FIX_WARP) {
      // ---------------- V in masked places: safe to multiply with weights of 0 ----------------
      int n = 0;
      uint32_t seen_once = 0;  // parity of each stage's `hidden`
      bool ok = true;
      Work w;
      for (int nth = 0; ok; ++nth) {
        if (!__all_sync(0xFFFFFFFFu, next_work(nth, &w))) break;
        const Plan p(a, w);
        for (int i = p.zone; i < p.nblocks; ++i) {
          const int v = n + 2 * i + 1, st = v % NST;
          ok = __all_sync(0xFFFFFFFFu, mbar_wait(hidden + 8 * st, (seen_once >> st) & 1, err, a.wait_ns) &&
                                           mbar_wait(full + 8 * st, (v / NST) & 1, err, a.wait_ns));
          seen_once ^= 1u << st;
          if (!ok) break;
          // rows [r0, end) some rows see, those after it none
          const int r0 = max(0, p.first_hidden - i * BN), end = min(BN, p.seen_end - i * BN);
          uint8_t* vb = smem_p + (ring - smem) + st * C::TILE;
          constexpr int VPR = C::CHUNKS * 8;  // 16-byte vectors per row
          auto at = [&](int row, int e) {
            return reinterpret_cast<uint4*>(vb + (e >> 3) * C::CHUNK + row * 128 + ((e & 7) ^ (row & 7)) * 16);
          };
          const int e = lane % VPR;
          bool found = false;
          for (int row = r0 + lane / VPR; row < end; row += 4 * (32 / VPR)) {
            uint4 x[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int ru = row + u * (32 / VPR);
              x[u] = ru < end ? *at(ru, e) : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              if (nonfinite8<T>(x[u])) {
                found = true;
                *at(row + u * (32 / VPR), e) =
                    make_uint4(finite2<T>(x[u].x), finite2<T>(x[u].y), finite2<T>(x[u].z), finite2<T>(x[u].w));
              }
            }
          }
          for (int row = max(r0, end) + lane / VPR; row < BN; row += 32 / VPR) *at(row, e) = make_uint4(0u, 0u, 0u, 0u);
          if (found) atomicExch(&s_nonfinite[nth % WORKS], 1);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(fixed + 8 * st);
        }
        n += 2 * p.nblocks;
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(work_empty + 8 * (nth % WORKS));
      }
    } else {
      // ---------------- products of a tile ----------------
      // The whole warp runs the loop and one lane issues: what a product is told is
      // then the same for the warp, and the compiler makes it in uniform registers.
      // Descriptors are bases plus constants (the address field counts 16 bytes, and
      // no address carries out of it).  A product takes 64 cycles; put together anew
      // for each, in one lane's registers, its operands took up to 110.
      const int t = warp - MMA_WARP;
      constexpr uint32_t ID_S = idesc_f16(BF16, BN, false), ID_O = idesc_f16(BF16, D, true);
      constexpr uint32_t TILE16 = C::TILE / 16, CHUNK16 = C::CHUNK / 16;
      const uint64_t q_desc = desc_sw128(q_smem, 16, 1024) + t * TILE16;
      const uint64_t k_desc = desc_sw128(ring, 16, 1024), v_desc = desc_sw128(ring, C::CHUNK, 1024);
      const uint32_t s_col = tmem + t * BN, o_col = tmem + C::O_COL + t * D;
      const bool one = lane == 0;
      int n = 0, nq = 0, np = 0, no = 0, nt = 0;  // blocks, Q pairs, weights taken, outputs begun and turns so far
      uint32_t fixed_once = 0;                    // parity of each stage's `fixed`
      auto wait = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, err, a.wait_ns)) != 0;
      };
      auto loaded = [&](int v) { return wait(full + 8 * (v % NST), (v / NST) & 1); };
      auto give = [&](uint32_t bar) {
        if (one) mbar_arrive(bar);
      };
      // the tiles take turns: left alone they fall into step, and both wait for
      // products and then both for weights
      auto my_turn = [&]() { return wait(turn + 8 * t, nt++ & 1); };
      auto qk = [&](int st) {  // S_t = Q_t K^T
        const uint64_t kd = k_desc + st * TILE16;
        if (one) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            mma_ss(s_col, q_desc + ((k >> 2) * CHUNK16 + (k & 3) * 2), kd + ((k >> 2) * CHUNK16 + (k & 3) * 2), ID_S,
                   k > 0);
          mma_commit(s_full + 8 * t);
          mma_commit(empty + 8 * st);
        }
      };
      auto pv = [&](int st, int h, bool first) {  // O_t += P_t V, a half of the keys
        const uint64_t v = v_desc + (st * TILE16 + h * (BN / 2) * 8);
        const uint32_t p = s_col + h * (BN / 2), more = first ? 0 : 1;
        if (one) {
          mma_ts(o_col, p, v, ID_O, more);
#pragma unroll
          for (int k = 1; k < BN / 32; ++k) mma_ts(o_col, p + k * 8, v + k * 128, ID_O, 1);
        }
      };
      bool ok = true;
      Work w;
      for (int nth = 0;; ++nth) {
        if (!__all_sync(0xFFFFFFFFu, ok && next_work(nth, &w))) break;
        w.pos0 = __shfl_sync(0xFFFFFFFFu, w.pos0, 0);
        w.q.qlen = __shfl_sync(0xFFFFFFFFu, w.q.qlen, 0);
        w.q.klen = __shfl_sync(0xFFFFFFFFu, w.q.klen, 0);
        const Plan p(a, w);
        const int blocks = t ? p.blocks[1] : p.blocks[0];
        if (p.nblocks > 0) {
          ok = wait(q_full, nq & 1) && loaded(n);
          if (!ok) break;
          ++nq;
          tc_fence_after();
          if (blocks > 0) qk(n % NST);
          else give(empty + 8 * (n % NST));
          if (blocks <= 1 && one) mma_commit(q_empty);
        }
        // blocks that only the other tile has are waited for and given back
        for (int i = 0; i < p.nblocks; ++i, n += 2) {
          const int sv = (n + 1) % NST, sk = (n + 2) % NST;
          ok = loaded(n + 1) && (i + 1 >= p.nblocks || loaded(n + 2));
          if (ok && i >= p.zone) {
            ok = wait(fixed + 8 * sv, (fixed_once >> sv) & 1);
            fixed_once ^= 1u << sv;
          }
          if (!ok) break;
          if (i >= blocks) {
            ok = my_turn();
            if (!ok) break;
            give(turn + 8 * (1 - t));
            give(empty + 8 * sv);
            if (i + 1 < p.nblocks) give(empty + 8 * sk);
            continue;
          }
          if (i == 0) {  // the last output of this tile has been read
            if (no > 0) ok = wait(o_empty + 8 * t, (no - 1) & 1);
            ++no;
          }
          ok = ok && wait(p_full + 16 * t, np & 1) && my_turn();
          if (!ok) break;
          tc_fence_after();
          pv(sv, 0, i == 0);
          ok = wait(p_full + 16 * t + 8, np & 1);
          if (!ok) break;
          tc_fence_after();
          pv(sv, 1, false);
          ++np;
          if (i + 1 < blocks) {
            qk(sk);
            if (i + 2 == blocks && one) mma_commit(q_empty);  // the tile's last scores
          } else {
            if (one) mma_commit(o_full + 8 * t);
            if (i + 1 < p.nblocks) give(empty + 8 * sk);
          }
          if (one) {
            mbar_arrive(turn + 8 * (1 - t));
            mma_commit(empty + 8 * sv);
          }
        }
        if (!ok) break;
        give(work_empty + 8 * (nth % WORKS));
      }
      // every product issued is done before tensor memory is freed
      if (one) {
        mma_commit(drain);
        const unsigned long long t0 = globaltimer();
        while (!mbar_try(drain, 0) && globaltimer() - t0 < a.wait_ns) {}
      }
      __syncwarp();
    }
  } else {
    more_registers<104>();
    // ---------------- softmax ----------------
    // A thread that gives up stays in the loops and takes part in the tile's
    // barriers; the vote at the next pair's beginning ends both halves together.
    constexpr int HN = BN / 2, HD = D / 2;  // columns of S and of O that a thread has
    const int t = warp >> 3, h = (warp >> 2) & 1;
    const int r = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_addr = tmem + lanes + t * BN + h * HN;
    const uint32_t o_addr = tmem + lanes + C::O_COL + t * D + h * HD;
    const int row_pos = r / G, row_head = r - row_pos * G;
    const int first_pos = ((warp & 3) * 32) / G;  // of the warp's rows, which are in position order
    int ns = 0, no = 0;                           // scores and outputs so far
    bool ok = true;
    Work w;
    for (int nth = 0;; ++nth) {
      ok = ok && next_work(nth, &w);
      if (tile_vote(t, !ok)) break;
      const Plan p(a, w);
      const int blocks = t ? p.blocks[1] : p.blocks[0];
      const int pos = w.pos0 + t * P + row_pos;
      const bool live = r < P * G && pos < w.q.qlen;
      const int lim = live ? p.limit(a, w, pos) : -1;
      // keys up to here are seen by every live row of the warp
      const int clear = p.limit(a, w, min(w.pos0 + t * P + first_pos, w.q.qlen - 1));
      // The reference, in units of log2, scaled and less LIFT (-LIFT in far rows, 0 before the first score); the
      // scaled score that calls for another (-inf: any does); a far row's reference.
      float m = 0.0f, most = NEG_INF, l = 0.0f, far_ref = NEG_INF;
      for (int i = 0; i < blocks; ++i, ++ns) {
        ok = __all_sync(0xFFFFFFFFu, ok && mbar_wait(s_full + 8 * t, ns & 1, err, a.wait_ns));
        const int c0 = i * BN + h * HN, seen = lim - c0;  // columns up to `seen` count
        const bool masked = c0 + HN - 1 > clear;
        // 32 scores, again from tensor memory for the weights: registers for all 64 would spill
        auto scores = [&](int c, uint32_t (&s)[32]) {
          tmem_ld32<0>(s_addr + c, s);
          tmem_wait_ld();
          if (masked) {
#pragma unroll
            for (int e = 0; e < 32; ++e) s[e] = c + e <= seen ? s[e] : __float_as_uint(NEG_INF);
          }
        };
        float mn = NEG_INF;
        if (ok) {
          tc_fence_after();
          float top[4] = {NEG_INF, NEG_INF, NEG_INF, NEG_INF};
#pragma unroll
          for (int c = 0; c < HN; c += 32) {
            uint32_t s[32];
            scores(c, s);
#pragma unroll
            for (int e = 0; e < 32; e += 2)
              top[(e >> 1) & 3] = max3(top[(e >> 1) & 3], __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
          }
          mn = live ? max3(fmaxf(top[0], top[1]), top[2], top[3]) : NEG_INF;  // Q's rows past the tile hold anything
        }
        if (tile_vote(t, i == 0 || mn * a.scale_log2 > most)) {  // a positive scale: checked on the host
          s_max[t][h][r] = mn;
          tile_sync(t);
          const float score = fmaxf(mn, s_max[t][1 - h][r]), top = score * a.scale_log2;
          const bool was_far = far_ref != NEG_INF, none = most == NEG_INF && !was_far;
          const bool far =
              was_far || (fabsf(top) >= FAR && score != NEG_INF && (none || top - LIFT<T> > m));
          float f;
          if (far) {
            const float ref = fmaxf(far_ref, score);
            f = was_far ? ex2((far_ref - ref) * a.scale_log2) : none ? 0.0f : ex2(m + LIFT<T> - top);
            far_ref = ref;
            m = -LIFT<T>;
            most = NEG_INF;
          } else {
            const float nm = none ? top - LIFT<T> : fmaxf(m, top - LIFT<T>);
            f = none ? 0.0f : ex2(m - nm);
            m = nm == NEG_INF ? 0.0f : nm;
            most = nm + (LIFT<T> + GROW);
          }
          if (i > 0) {
            l *= f;
            if (ok) {
#pragma unroll
              for (int c = 0; c < HD; c += 16) {
                uint32_t o[16];
                tmem_ld16(o_addr + c, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st16(o_addr + c, o);
              }
              tmem_wait_st();
              tc_fence_before();
            }
            tile_sync(t);  // a half's weights go to all of O: both halves of it are rescaled before
          }
          if (__any_sync(0xFFFFFFFFu, far) && ok) {
            const float off = far ? far_ref : 0.0f;
#pragma unroll 1
            for (int c = 0; c < HN; c += 16) {
              uint32_t s[16];
              tmem_ld16(s_addr + c, s);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) s[e] = __float_as_uint(__uint_as_float(s[e]) - off);
              tmem_st16(s_addr + c, s);
            }
            tmem_wait_st();
          }
        }
        if (ok) {
          const F2 sc2 = f2(a.scale_log2, a.scale_log2), mm2 = f2(-m, -m);
          F2 sum[2] = {f2(0.0f, 0.0f), f2(0.0f, 0.0f)};
#pragma unroll
          for (int c = 0; c < HN; c += 32) {
            uint32_t s[32], q[16];
            scores(c, s);
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float2 x = unf2(fma2(f2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), sc2, mm2));
              const float p0 = ex2(x.x), p1 = ex2(x.y);
              sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], f2(p0, p1));
              q[e / 2] = pack2<T>(p0, p1);
            }
            tmem_st16(s_addr + c / 2, q);  // over scores that this thread has read
          }
          const float2 l2 = unf2(add2(sum[0], sum[1]));
          l += l2.x + l2.y;
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_full + 16 * t + 8 * h);
        }
      }
      // ---- O / l to memory ----
      T* dst = static_cast<T*>(a.out) + ((int64_t)(w.q.qb + pos) * a.q_heads + w.head * G + row_head) * D + h * HD;
      if (blocks == 0) {
        if (live)
          for (int c = 0; c < HD; c += 8) *reinterpret_cast<uint4*>(dst + c) = make_uint4(0u, 0u, 0u, 0u);
      } else {
        s_sum[t][h][r] = l;
        tile_sync(t);
        l += s_sum[t][1 - h][r];
        ok = __all_sync(0xFFFFFFFFu, ok && mbar_wait(o_full + 8 * t, no & 1, err, a.wait_ns));
        ++no;
        if (ok) {
          tc_fence_after();
          uint32_t o[HD];
          tmem_ld32<0>(o_addr, o);
          if constexpr (D == 128) tmem_ld32<32>(o_addr + 32, o);
          tmem_wait_ld();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(o_empty + 8 * t);
          const float inv = 1.0f / l;
          const bool extra = s_nonfinite[nth % WORKS] != 0;
          if (live) {
#pragma unroll
            for (int c = 0; c < HD; c += 16) {
              float x[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) x[e] = lim < 0 ? 0.0f : __uint_as_float(o[c + e]) * inv;
              if (extra) {  // what was set aside: keys that this row sees
                const T* v = static_cast<const T*>(a.v) + (int64_t)w.head * a.v_head + h * HD + c;
                for (int j = p.first_hidden; j <= lim; ++j)
                  for (int e = 0; e < 16; ++e) {
                    const float f = (float)v[(int64_t)(w.q.kb + j) * a.v_row + e];
                    if (!isfinite(f)) x[e] += f;
                  }
              }
              uint32_t y[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) y[e] = pack2<T>(x[2 * e], x[2 * e + 1]);
              store16(dst + c, y, a.wide);
            }
          }
        }
      }
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(work_empty + 8 * (nth % WORKS));
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
  a.wide = (reinterpret_cast<uintptr_t>(c.out) & 31u) == 0;
  a.scale_log2 = c.scale * 1.44269504088896340736f;
  a.q_offsets = c.q_offsets;
  a.k_offsets = c.k_offsets;
  a.status = c.status;
  a.wait_ns = wait_limit_ns();
  a.stall = stall_for_test();
  // pairs of tiles: whole ones and at most one ragged per sequence
  const int64_t ctas = c.q_total / (2 * a.positions) + (c.S < c.q_total ? c.S : c.q_total);
  if (ctas >= INT32_MAX / c.kv_heads) return Q4_ERR_SHAPE;
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
  prompt_kernel<D, T><<<(unsigned)(ctas * c.kv_heads), THREADS, Cfg<D>::SMEM, s>>>(a, mq, mk, mv);
  return cudaGetLastError() == cudaSuccess ? Q4_OK : Q4_ERR_CUDA;
}

}  // namespace

int launch_prompt_attention(const PromptAttn& c, cudaStream_t s) {
  if (c.dtype == Q4_DTYPE_F16)
    return c.head_dim == 128 ? launch_as<128, __half>(c, s) : launch_as<64, __half>(c, s);
  return c.head_dim == 128 ? launch_as<128, __nv_bfloat16>(c, s) : launch_as<64, __nv_bfloat16>(c, s);
}

}  // namespace q4
