// q4_kvq_evict.cu — a 4-bit cache thinned out to the positions that collected
// most attention weight.
//
// Of a head's n positions the last `recent` stay, and of the others the
// keep - recent of largest weight (the lowest position among equals); their
// order is kept.  Select: a radix select over the weights' order-preserving
// 32-bit keys (four passes of 8 bits) gives the smallest weight that stays and
// how many positions of exactly that weight do; then each warp counts what
// stays in a run of positions, and with the runs before it known numbers them.
// The weights are read once, as keys into shared memory (caches of up to 48,000
// positions; longer ones are read again by each pass): the passes are then
// bound by their barriers, not by six trips to memory.
// Move: row i of the result is row kept[i] >= i, so a copy within one slot runs
// step by step, each step read whole before it is written: a cluster of eight
// CTAs does that with its barrier between the two.  A copy to another slot has
// no order, and more clusters share it.  V's rows lie four to a sector, so rows
// that stay bring others along: of 5,000 positions of which 2,048 stay the copy
// reads nearly all of V.  128 heads of that take 22 us cold, 91 MB read and 38 MB
// written (5.9 TB/s).  A thread takes one piece a step: two or four at once
// were slower (71 and 76 us for copy, eviction and read together, against 68).
#include <atomic>
#include <type_traits>

#include "q4_kvq.cuh"

namespace q4 {
namespace {

constexpr int SEL_THREADS = 1024;
constexpr int SEL_WARPS = SEL_THREADS / 32;
constexpr int64_t SEL_SHARED_MOST = 48000;  // positions whose weights fit shared memory
constexpr int MOVE_THREADS = 256;
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

__device__ __forceinline__ float key_weight(uint32_t k) {
  return k == 0u ? NAN : __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}

// SHARED: the weights' keys are kept in shared memory.
template <bool SHARED>
__global__ void __launch_bounds__(SEL_THREADS) evict_select_kernel(const KvqEvict a) {
  extern __shared__ uint32_t s_key[];
  __shared__ unsigned hist[256];
  __shared__ int2 runs[SEL_WARPS];  // per warp's run: positions that stay for sure, and of exactly the smallest weight
  __shared__ uint32_t s_prefix;
  __shared__ unsigned s_want;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int s = blockIdx.x / (int)a.heads, h = blockIdx.x % (int)a.heads;
  asm volatile("griddepcontrol.launch_dependents;");
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
    for (int p = tid; p < n; p += SEL_THREADS) s_key[p] = order_key(mass[p]);
  }
  auto key = [&](int p) { return SHARED ? s_key[p] : order_key(mass[p]); };

  // the key of rank `want` from the top, 8 bits at a time
  uint32_t prefix = 0;
  unsigned left = (unsigned)want;  // of the positions that match the prefix, so many stay
  if (want > 0 && want < first) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
#pragma unroll 4
      for (int p = tid; p < first; p += SEL_THREADS) {
        const uint32_t k = key(p);
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
    const uint32_t k = in && p < first ? key(p) : 0u;
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
  const int2 other = lane < warp ? runs[lane] : make_int2(0, 0);
  int2 before = make_int2((int)__reduce_add_sync(0xFFFFFFFFu, (unsigned)other.x),
                          (int)__reduce_add_sync(0xFFFFFFFFu, (unsigned)other.y));
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
    const float w = i >= out_n ? 0.0f : SHARED ? key_weight(s_key[kept[i]]) : mass[kept[i]];
    if (!SHARED) __syncthreads();
    if (i < out_n) mass_out[i] = w;
  }
}

// A pair of result rows as pieces of a lane's load: four of K codes (of each of
// the two rows), eight V word groups (both rows interleaved) and the scale words of K
// and V (likewise).  Two loads make any piece; K's are two stores.
template <int D>
struct PairPieces {
  using L = Kvq<D>;
  static constexpr unsigned W = 4 * L::NB, K = 4, PIECES = K + 8 + 2;
  using Vec = std::conditional_t<D == 128, uint4, uint2>;
  static_assert(K * W == L::ROW && sizeof(Vec) == W, "a K row is four pieces");
  // byte of piece e of position p in a plane
  __device__ static int64_t at(unsigned p, unsigned e) {
    const unsigned r = p % L::POS;
    const int in = e < K ? r * L::ROW + e * W : e < K + 8 ? kvq_v_group<D>(r, e - K) : kvq_scale<D>(e - K - 8, r & ~1u, 0);
    return (int64_t)(p / L::POS) * L::BYTES + in;
  }
  // a and b with the half of each word that positions p0 and p1 own
  __device__ static Vec merge(Vec a, Vec b, unsigned p0, unsigned p1) {
    const unsigned sel = ((p0 & 1) ? 0x32u : 0x10u) | ((p1 & 1) ? 0x7600u : 0x5400u);
    a.x = __byte_perm(a.x, b.x, sel);
    a.y = __byte_perm(a.y, b.y, sel);
    if constexpr (D == 128) {
      a.z = __byte_perm(a.z, b.z, sel);
      a.w = __byte_perm(a.w, b.w, sel);
    }
    return a;
  }
};

template <int D>
__global__ void __cluster_dims__(MOVE_CLUSTER, 1, 1) __launch_bounds__(MOVE_THREADS)
    evict_move_kernel(const KvqEvict a, int64_t plane_bytes) {
  using R = PairPieces<D>;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the select launch has ended
  asm volatile("griddepcontrol.launch_dependents;");  // not before: a later launch waits for this one only
  const int s = blockIdx.y / (int)a.heads, h = blockIdx.y % (int)a.heads;
  const int n_out = kvq_ld<true>(a.new_len + s);
  if (n_out <= 0) return;
  const unsigned n = n_out;
  const int64_t src_slot = kvq_ld<true>(a.src + s), dst_slot = kvq_ld<true>(a.dst + s);
  const bool in_place = src_slot == dst_slot;
  // (whole clusters leave)
  if (in_place && (blockIdx.x >= MOVE_CLUSTER || n_out == kvq_ld<true>(a.len + s))) return;
  uint8_t* src = a.cache + (src_slot * a.heads + h) * plane_bytes;
  uint8_t* dst = a.cache + (dst_slot * a.heads + h) * plane_bytes;
  const int32_t* kept = a.kept + (int64_t)blockIdx.y * a.keep;
  const unsigned items = (n + 1) / 2 * R::PIECES;  // below 2^31: checked on the host
  const unsigned stride = (in_place ? MOVE_CLUSTER : gridDim.x) * MOVE_THREADS;
  // (the barrier is for all threads of the cluster: the loop runs by whole steps)
  for (unsigned step = 0; step < items; step += stride) {
    const unsigned it = step + blockIdx.x * MOVE_THREADS + threadIdx.x;
    const unsigned pair = it / R::PIECES, e = it % R::PIECES;
    typename R::Vec v0, v1;
    unsigned p0, p1;
    if (it < items) {
      p0 = kvq_ld<true>(kept + 2 * pair);
      p1 = 2 * pair + 1 < n ? kvq_ld<true>(kept + 2 * pair + 1) : p0;  // a last odd row: its neighbour is never used
      v0 = *reinterpret_cast<const typename R::Vec*>(src + R::at(p0, e));
      v1 = *reinterpret_cast<const typename R::Vec*>(src + R::at(p1, e));
    }
    if (in_place)  // the step is read before it is written; later steps read from further on
      asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
    if (it < items) {
      auto* out = reinterpret_cast<typename R::Vec*>(dst + R::at(2 * pair, e));
      *out = e < R::K ? v0 : R::merge(v0, v1, p0, p1);
      if (e < R::K) out[R::K] = v1;  // the next row's
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
  const int64_t items = (int64_t)((c.keep + 1) / 2) * PairPieces<128>::PIECES;
  const int64_t steps = (items + MOVE_THREADS - 1) / MOVE_THREADS;
  int64_t gx = ((int64_t)c.num_sms * 32 + planes - 1) / planes;
  if (gx > steps) gx = steps;
  gx = (gx + MOVE_CLUSTER - 1) / MOVE_CLUSTER * MOVE_CLUSTER;
  const dim3 grid((unsigned)gx, (unsigned)planes);
  const int64_t pb = kvq_plane_bytes(c.head_dim, c.capacity);
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(MOVE_THREADS);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return (c.head_dim == 128 ? cudaLaunchKernelEx(&cfg, evict_move_kernel<128>, c, pb)
                            : cudaLaunchKernelEx(&cfg, evict_move_kernel<64>, c, pb)) == cudaSuccess
             ? Q4_OK
             : Q4_ERR_CUDA;
}

}  // namespace q4
