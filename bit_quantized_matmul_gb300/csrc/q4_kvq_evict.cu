// q4_kvq_evict.cu — a 4-bit cache thinned out to the positions that collected
// most attention weight.
//
// Of a head's n positions the last `recent` stay, and of the others the
// keep - recent of largest weight (the lowest position among equals); their
// order is kept.  Select: a radix select over the weights' order-preserving
// 32-bit keys (four passes of 8 bits) gives the smallest weight that stays and
// how many positions of exactly that weight do; then each warp counts what
// stays in a run of positions, and with the runs before it known numbers them.
// The weights are read once, into shared memory (caches of up to 48,000
// positions; longer ones are read again by each pass): the passes are then
// bound by their barriers, not by six trips to memory.
// Move: row i of the result is row kept[i] >= i, so a copy within one slot runs
// step by step, each step read whole before it is written: a cluster of eight
// CTAs does that with its barrier between the two.  A copy to another slot has
// no order, and more clusters share it.  A pair of V rows shares its sectors, so
// rows that stay alone bring their neighbours along: of 5,000 positions of
// which 2,048 stay the copy reads nearly all of V.  128 heads of that take
// 26 us cold (75 MB of kept rows read and written: 2.9 TB/s), bound by those
// sectors and by the latency of one gathered step after another.  Four pieces
// per thread and step instead of two leave that as it is, and a short eviction
// (2 x 1,500 positions to 513, in place) goes from 15 to 16.5 us; eight take
// 14 us more.
#include <atomic>

#include "q4_kvq.cuh"

namespace q4 {
namespace {

constexpr int SEL_THREADS = 1024;
constexpr int SEL_WARPS = SEL_THREADS / 32;
constexpr int64_t SEL_SHARED_MOST = 48000;  // positions whose weights fit shared memory
constexpr int MOVE_THREADS = 256;
constexpr int MOVE_VEC = 2;      // pieces per thread and step
constexpr int MOVE_CLUSTER = 8;

// A request whose slots, length and neighbours allow it.
__device__ bool evict_ok(const KvqEvict& a, int s) {
  const int64_t src = a.src[s], dst = a.dst[s], n = a.len[s];
  return src >= 0 && src < a.slots && dst >= 0 && dst < a.slots && n >= 0 && n <= a.capacity;
}

// No other request of the call writes this one's slots or reads its target.
__device__ bool evict_apart(const KvqEvict& a, int s) {
  const int src = a.src[s], dst = a.dst[s];
  bool clash = false;
  for (int i = threadIdx.x; i < a.S; i += blockDim.x)
    if (i != s) clash |= a.dst[i] == dst || a.dst[i] == src || a.src[i] == dst;
  return !__syncthreads_or(clash);
}

// Weights in ascending order as unsigned keys; NaN below everything.
__device__ __forceinline__ uint32_t order_key(float f) {
  if (isnan(f)) return 0u;
  f += 0.0f;  // -0 and 0 are equal
  const uint32_t u = __float_as_uint(f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// SHARED: the weights are kept in shared memory.
template <bool SHARED>
__global__ void __launch_bounds__(SEL_THREADS) evict_select_kernel(const KvqEvict a) {
  extern __shared__ float s_mass[];
  __shared__ unsigned hist[256];
  __shared__ int2 runs[SEL_WARPS];  // per warp's run: positions that stay for sure, and of exactly the smallest weight
  __shared__ uint32_t s_prefix;
  __shared__ unsigned s_want;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int s = blockIdx.x / (int)a.heads, h = blockIdx.x % (int)a.heads;
  const bool ok = evict_ok(a, s);
  const bool apart = evict_apart(a, s);
  int32_t* kept = a.kept + (int64_t)blockIdx.x * a.keep;
  if (!ok || !apart) {
    if (tid == 0) {
      atomicOr(a.status, STATUS_KV_RANGE);
      if (h == 0) a.new_len[s] = -1;
    }
    for (int i = tid; i < a.keep; i += SEL_THREADS) kept[i] = -1;
    return;
  }
  const int n = a.len[s];
  const int out_n = min(n, a.keep);
  const int first = n - min(n, min(a.recent, a.keep));  // positions below compete
  const int want = out_n - (n - first);                 // of which so many stay
  const float* mass = a.mass + ((int64_t)a.src[s] * a.heads + h) * a.capacity;
  float* mass_out = a.mass + ((int64_t)a.dst[s] * a.heads + h) * a.capacity;
  if (tid == 0 && h == 0) a.new_len[s] = out_n;
  for (int i = out_n + tid; i < a.keep; i += SEL_THREADS) kept[i] = -1;
  if (SHARED) {
#pragma unroll 4
    for (int p = tid; p < n; p += SEL_THREADS) s_mass[p] = mass[p];
  }
  auto weight = [&](int p) { return SHARED ? s_mass[p] : mass[p]; };

  // the key of rank `want` from the top, 8 bits at a time
  uint32_t prefix = 0;
  unsigned left = (unsigned)want;  // of the positions that match the prefix, so many stay
  if (want > 0 && want < first) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
#pragma unroll 4
      for (int p = tid; p < first; p += SEL_THREADS) {
        const uint32_t k = order_key(weight(p));
        if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(k >> shift) & 255u], 1u);
      }
      __syncthreads();
      if (warp == 0) {  // lane i sums the bins 8i .. 8i+7; the first lane from the top that reaches `left` looks closer
        unsigned mine = 0;
        for (int b = 0; b < 8; ++b) mine += hist[lane * 8 + b];
        unsigned above = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned v = __shfl_down_sync(0xFFFFFFFFu, above, o);
          if (lane + o < 32) above += v;
        }
        above -= mine;  // in the bins above this lane's
        if (above < left && above + mine >= left) {
          unsigned c = above;
          for (int b = 7; b >= 0; --b) {
            const unsigned v = hist[lane * 8 + b];
            if (c + v >= left) {
              s_prefix = prefix | (uint32_t)(lane * 8 + b) << shift;
              s_want = left - c;
              break;
            }
            c += v;
          }
        }
      }
      __syncthreads();
      prefix = s_prefix;
      left = s_want;
    }
  } else {
    __syncthreads();
  }
  const bool all_stay = want >= first, none_stays = want <= 0;

  // each warp has a run of positions, 32 at a time
  const int run = (n + SEL_THREADS - 1) / SEL_THREADS * 32, p0 = warp * run, p1 = min(n, p0 + run);
  auto look = [&](int p, unsigned* sure, unsigned* tie) {
    const bool in = p < p1;
    const uint32_t k = in && p < first ? order_key(weight(p)) : 0u;
    *sure = __ballot_sync(0xFFFFFFFFu, in && (p >= first || all_stay || (!none_stays && k > prefix)));
    *tie = __ballot_sync(0xFFFFFFFFu, in && p < first && !all_stay && !none_stays && k == prefix);
  };
  int2 mine = make_int2(0, 0);
  for (int p = p0; p < p1; p += 32) {
    unsigned sure, tie;
    look(p + lane, &sure, &tie);
    mine.x += __popc(sure);
    mine.y += __popc(tie);
  }
  if (lane == 0) runs[warp] = mine;
  __syncthreads();
  int2 before = make_int2(0, 0);
  for (int w = 0; w < warp; ++w) {
    before.x += runs[w].x;
    before.y += runs[w].y;
  }
  // of the first x positions, the sure ones stay and min(ties, left) of the others
  for (int p = p0; p < p1; p += 32) {
    unsigned sure, tie;
    look(p + lane, &sure, &tie);
    const unsigned below = (1u << lane) - 1u;
    const unsigned ties = before.y + __popc(tie & below);
    if ((sure >> lane & 1u) || ((tie >> lane & 1u) && ties < left))
      kept[before.x + __popc(sure & below) + min(ties, left)] = p + lane;
    before.x += __popc(sure);
    before.y += __popc(tie);
  }
  __syncthreads();
  // the weights: kept[i] >= i, so a step's are read before the places of any later one's are written
  for (int i0 = 0; i0 < out_n; i0 += SEL_THREADS) {
    const int i = i0 + tid;
    const float w = i < out_n ? weight(kept[i]) : 0.0f;
    if (!SHARED) __syncthreads();
    if (i < out_n) mass_out[i] = w;
  }
}

// A pair of result rows as pieces: 16-byte vectors of K codes (of either row),
// the V word groups (both rows interleaved) and the scale words of K and V
// (likewise).
template <int D>
struct PairPieces {
  using L = Kvq<D>;
  static constexpr int NB = L::NB;
  static constexpr int CV = D / 32;          // K code vectors per row
  static constexpr int PIECES = 2 * CV + 8 + 2;
  struct Piece {
    uint32_t w[4];
  };
  __device__ static uint8_t* tile(uint8_t* plane, int64_t p) { return plane + p / L::POS * L::BYTES; }
  __device__ static uint4* k_vec(uint8_t* plane, int64_t p, int e) {
    return reinterpret_cast<uint4*>(tile(plane, p) + (int)(p % L::POS) * L::ROW + e * 16);
  }
  // NB words of positions p and p ^ 1: V's group e, or the scales of K (8) or V (9)
  __device__ static uint32_t* words(uint8_t* plane, int64_t p, int e) {
    const int r = (int)(p % L::POS);
    return reinterpret_cast<uint32_t*>(tile(plane, p) +
                                       (e < 8 ? kvq_v_group<D>(r, e) : kvq_scale<D>(e - 8, r & ~1, 0)));
  }
  __device__ static Piece load(const uint32_t* p) {
    Piece v;
    if constexpr (NB == 4) *reinterpret_cast<uint4*>(v.w) = *reinterpret_cast<const uint4*>(p);
    else *reinterpret_cast<uint2*>(v.w) = *reinterpret_cast<const uint2*>(p);
    return v;
  }
  // piece e of the pair whose rows are positions p0 and p1 of `src`
  __device__ static Piece read(uint8_t* src, int64_t p0, int64_t p1, int e) {
    Piece v;
    if (e < 2 * CV) {
      *reinterpret_cast<uint4*>(v.w) = *k_vec(src, e < CV ? p0 : p1, e % CV);
      return v;
    }
    v = load(words(src, p0, e - 2 * CV));
    const Piece b = load(words(src, p1, e - 2 * CV));
    // the half of each word that the position owns
    const unsigned sel = ((p0 & 1) ? 0x32u : 0x10u) | ((p1 & 1) ? 0x7600u : 0x5400u);
#pragma unroll
    for (int i = 0; i < NB; ++i) v.w[i] = __byte_perm(v.w[i], b.w[i], sel);
    return v;
  }
  __device__ static void write(uint8_t* dst, int64_t p, int e, const Piece& v) {  // p even
    if (e < 2 * CV) {
      *k_vec(dst, p + (e < CV ? 0 : 1), e % CV) = *reinterpret_cast<const uint4*>(v.w);
      return;
    }
    uint32_t* q = words(dst, p, e - 2 * CV);
    if constexpr (NB == 4) *reinterpret_cast<uint4*>(q) = *reinterpret_cast<const uint4*>(v.w);
    else *reinterpret_cast<uint2*>(q) = *reinterpret_cast<const uint2*>(v.w);
  }
};

template <int D>
__global__ void __cluster_dims__(MOVE_CLUSTER, 1, 1) __launch_bounds__(MOVE_THREADS)
    evict_move_kernel(const KvqEvict a, int64_t plane_bytes) {
  using R = PairPieces<D>;
  const int s = blockIdx.y / (int)a.heads, h = blockIdx.y % (int)a.heads;
  const int n = a.new_len[s];
  if (n <= 0) return;
  const int64_t src_slot = a.src[s], dst_slot = a.dst[s];
  const bool in_place = src_slot == dst_slot;
  // (whole clusters leave)
  if (in_place && (blockIdx.x >= MOVE_CLUSTER || n == a.len[s])) return;
  uint8_t* src = a.cache + (src_slot * a.heads + h) * plane_bytes;
  uint8_t* dst = a.cache + (dst_slot * a.heads + h) * plane_bytes;
  const int32_t* kept = a.kept + (int64_t)blockIdx.y * a.keep;
  const int items = (n + 1) / 2 * R::PIECES;  // below 2^31: checked on the host
  constexpr int STEP = MOVE_THREADS * MOVE_VEC;
  const int stride = (in_place ? MOVE_CLUSTER : gridDim.x) * STEP;
  for (int step = 0; step < items; step += stride) {
    const int i0 = step + blockIdx.x * STEP;
    typename R::Piece v[MOVE_VEC];
#pragma unroll
    for (int u = 0; u < MOVE_VEC; ++u) {
      const int it = i0 + u * MOVE_THREADS + threadIdx.x;
      if (it < items) {
        const int pair = it / R::PIECES, e = it - pair * R::PIECES;
        const int p0 = kept[2 * pair];
        const int p1 = 2 * pair + 1 < n ? kept[2 * pair + 1] : p0;  // a last odd row: its neighbour is never used
        v[u] = R::read(src, p0, p1, e);
      }
    }
    if (in_place)  // the step is read before it is written; later steps read from further on
      asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
#pragma unroll
    for (int u = 0; u < MOVE_VEC; ++u) {
      const int it = i0 + u * MOVE_THREADS + threadIdx.x;
      if (it < items) {
        const int pair = it / R::PIECES;
        R::write(dst, 2 * (int64_t)pair, it - pair * R::PIECES, v[u]);
      }
    }
  }
}

}  // namespace

int launch_kvq_evict(const KvqEvict& c, cudaStream_t s) {
  const int64_t planes = (int64_t)c.S * c.heads;
  if (c.capacity <= SEL_SHARED_MOST) {
    static std::atomic<bool> sized[64];  // per device: the kernel's shared memory limit is set
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return Q4_ERR_CUDA;
    if (!sized[dev].load()) {
      if (cudaFuncSetAttribute(evict_select_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)(SEL_SHARED_MOST * sizeof(float))) != cudaSuccess)
        return Q4_ERR_CUDA;
      sized[dev].store(true);
    }
    evict_select_kernel<true><<<(unsigned)planes, SEL_THREADS, (size_t)c.capacity * sizeof(float), s>>>(c);
  } else {
    evict_select_kernel<false><<<(unsigned)planes, SEL_THREADS, 0, s>>>(c);
  }
  if (cudaGetLastError() != cudaSuccess) return Q4_ERR_CUDA;
  const int64_t items = (int64_t)((c.keep + 1) / 2) * (2 * (c.head_dim / 32) + 10);
  const int64_t steps = (items + MOVE_THREADS * MOVE_VEC - 1) / (MOVE_THREADS * MOVE_VEC);
  int64_t gx = ((int64_t)c.num_sms * 32 + planes - 1) / planes;
  if (gx > steps) gx = steps;
  gx = (gx + MOVE_CLUSTER - 1) / MOVE_CLUSTER * MOVE_CLUSTER;
  const dim3 grid((unsigned)gx, (unsigned)planes);
  const int64_t pb = kvq_plane_bytes(c.head_dim, c.capacity);
  if (c.head_dim == 128) evict_move_kernel<128><<<grid, MOVE_THREADS, 0, s>>>(c, pb);
  else evict_move_kernel<64><<<grid, MOVE_THREADS, 0, s>>>(c, pb);
  return cudaGetLastError() == cudaSuccess ? Q4_OK : Q4_ERR_CUDA;
}

}  // namespace q4
