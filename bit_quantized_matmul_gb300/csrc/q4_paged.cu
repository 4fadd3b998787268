// q4_paged.cu — pages of a 16-bit KV cache: block tables and slot maps from the
// requests' lengths, and the append of a step's rows.
//
// Reserve.  Request s of a step has h pages and wants n = ceil((pos + rows) / P).
// With back(s) = max(0, h - n) and more(s) = max(0, n - h), and both summed over
// the requests before s, page i of those that go back is cell
//     count + sum back + i                      of the free list, and the i-th that s is given is cell
//     count + all back - 1 - (sum more + i),
// so every page has its place without any order between the threads, and the
// same step on the same state always gives the same tables.  A packed row finds its page
// the same way, so the slot map does not wait for the tables; the row that begins a page enters it.
// Bound by latency: a few dependent loads and nine barriers of 1,024 threads, four more for every further
// 1,024 requests (two a sum).  One CTA for a decode step (64 requests: 4 us in a graph); from 4,096 rows and requests on a cluster of eight, each of
// which makes the sums for itself (they are cheap) and takes a share of the rows (512 requests with
// 47,886 rows: 12 us; with one row or page of a thread on its way at a time 14).
//
// Append.  Each 16-byte piece of a cached row is one thread's: the row and its
// place in the slot map are loaded side by side, then stored.  Bound by memory
// bandwidth for prompts and by one chain of latency for decode steps: 64 rows 1.5 us, 6,072
// of 2 x 4 x 128 fp16 values 5.8 us (4.3 TB/s; with K and V by threads of their own 6.3).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <type_traits>

#include "q4mm_internal.h"

namespace q4 {
namespace {

constexpr int THREADS = 1024;
constexpr int WARPS = THREADS / 32;
constexpr int CLUSTER = 8;
constexpr int64_t ONE_CTA = 4096;  // rows and requests up to which one CTA is enough
constexpr int FEW = 4;             // loads of a thread on their way at once

__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The sum over the threads before this one (by thread number), and over all of
// them in *all; for the whole CTA, scratch of one value a warp.
template <typename V>
__device__ __forceinline__ V scan_block(V x, V* warps, V* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  V upto = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const V y = __shfl_up_sync(0xFFFFFFFFu, upto, o);
    if (lane >= o) upto += y;
  }
  if (lane == 31) warps[warp] = upto;
  __syncthreads();
  V w = warps[lane];  // as many warps as lanes
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const V y = __shfl_up_sync(0xFFFFFFFFu, w, o);
    if (lane >= o) w += y;
  }
  *all = __shfl_sync(0xFFFFFFFFu, w, 31);
  const V before = __shfl_sync(0xFFFFFFFFu, w, warp ? warp - 1 : 0);
  __syncthreads();  // the scratch may be written again
  return (warp ? before : 0) + upto - x;
}
static_assert(WARPS == 32, "one lane of the second scan for each warp");

struct Reserve {
  int32_t *table, *held, *free_list, *free_count;
  int slots, width, pages, shift, S;  // a page is 1 << shift positions
  int64_t total;
  const int32_t *offsets, *slot, *pos;
  int32_t *slot_map, *new_len;
  unsigned* status;
};

// Shared memory of a call: the requests' numbers, and two bits for each slot.
struct ReserveSmem {
  int32_t *off, *slot, *pos, *have, *back, *more;  // back, more: sums before the request
  uint32_t *seen, *twice;
  __host__ __device__ static int words(int slots) { return (slots + 31) / 32; }
  __host__ static size_t bytes(int S, int slots) { return 4 * ((size_t)6 * S + 1 + 2 * (size_t)words(slots)); }
  __device__ ReserveSmem(int32_t* base, int S, int slots) {
    off = base;
    slot = off + S + 1;
    pos = slot + S;
    have = pos + S;
    back = have + S;
    more = back + S;
    seen = reinterpret_cast<uint32_t*>(more + S);
    twice = seen + words(slots);
  }
};

__global__ void __launch_bounds__(THREADS) reserve_kernel(const Reserve a) {
  extern __shared__ int32_t smem[];
  __shared__ int64_t s_scan[WARPS];
  __shared__ int s_bad, s_given;
  const ReserveSmem m(smem, a.S, a.slots);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const unsigned rank = cluster_rank(), ctas = gridDim.x;
  const int page = 1 << a.shift;

  for (int i = tid; i < 2 * ReserveSmem::words(a.slots); i += THREADS) m.seen[i] = 0;  // `twice` follows
  if (tid == 0) {
    s_bad = 0;
    s_given = 0;
  }
  const int count = *a.free_count;
  __syncthreads();
  for (int s = tid; s < a.S; s += THREADS) {
    const int slot = a.slot[s], b = a.offsets[s], e = a.offsets[s + 1];
    m.off[s] = b;
    if (s == a.S - 1) m.off[a.S] = e;
    m.slot[s] = slot;
    m.pos[s] = a.pos[s];
    if (b < 0 || e < b || e > a.total) s_bad = 1;  // no row can be told whose it is
    if (slot >= 0 && slot < a.slots) {
      const uint32_t bit = 1u << (slot & 31);
      if (atomicOr(&m.seen[slot >> 5], bit) & bit) atomicOr(&m.twice[slot >> 5], bit);
    }
  }
  __syncthreads();
  bool refused = false;  // some request of this thread's
  int64_t all_back = 0, all_more = 0;
  for (int s0 = 0; s0 < a.S; s0 += THREADS) {
    const int s = s0 + tid;
    int64_t back = 0, more = 0;
    int have = -1;
    if (s < a.S) {
      const int slot = m.slot[s], pos = m.pos[s];
      const int64_t len = (int64_t)pos + m.off[s + 1] - m.off[s];
      if (slot >= 0 && slot < a.slots && !(m.twice[slot >> 5] >> (slot & 31) & 1) && pos >= 0 &&
          len <= (int64_t)a.width * page) {
        have = a.held[slot];
        // a slot's pages cover the positions before the step's
        if (have < 0 || have > a.width || (int64_t)have * page < pos) have = -1;
      }
      if (have >= 0) {
        const int need = (int)((len + page - 1) >> a.shift);
        back = max(0, have - need);
        more = max(0, need - have);
      } else {
        refused = true;
      }
    }
    int64_t sum;
    const int64_t back0 = all_back + scan_block(back, s_scan, &sum);
    all_back += sum;
    const int64_t more0 = all_more + scan_block(more, s_scan, &sum);
    all_more += sum;
    if (s < a.S) {
      m.have[s] = have;
      m.back[s] = (int)back0;  // beyond the pages there are, the call is refused
      m.more[s] = (int)more0;  // at most one page for each row
    }
  }
  // a pool that holds more pages than there are is not touched
  const bool none = s_bad || count < 0 || count > a.pages || count + all_back > a.pages;
  if (rank == 0 && (refused || none)) atomicOr(a.status, STATUS_KV_RANGE);
  const int top = none ? 0 : count + (int)all_back;
  __syncthreads();

  // ---- pages that go back, by a warp a request ----
  if (!none) {
    for (int s = rank * WARPS + warp; s < a.S; s += ctas * WARPS) {
      const int have = m.have[s];
      if (have < 0) continue;
      const int need = (int)(((int64_t)m.pos[s] + m.off[s + 1] - m.off[s] + page - 1) >> a.shift);
      int32_t* row = a.table + (int64_t)m.slot[s] * a.width;
      for (int i0 = need + lane; i0 < have; i0 += 32 * FEW) {
        int id[FEW];
#pragma unroll
        for (int u = 0; u < FEW; ++u)
          if (i0 + 32 * u < have) id[u] = row[i0 + 32 * u];
#pragma unroll
        for (int u = 0; u < FEW; ++u) {
          const int i = i0 + 32 * u;
          if (i >= have) break;
          a.free_list[count + m.back[s] + i - need] = id[u];
          row[i] = -1;
        }
      }
    }
  }
  cluster_barrier();  // the free list is whole, and every CTA has read what the step began with

  // ---- the requests' ends ----
  // -1: refused; else the pages it wants, which it has or is given
  auto wants = [&](int s) {
    const int have = m.have[s];
    if (none || have < 0) return -1;
    const int need = (int)(((int64_t)m.pos[s] + m.off[s + 1] - m.off[s] + page - 1) >> a.shift);
    return need > have && m.more[s] + need - have > top ? -1 : need;
  };
  if (rank == 0) {
    int given = 0;  // pages, up to the thread's last request that got some
    bool out = false;
    for (int s = tid; s < a.S; s += THREADS) {
      const int need = wants(s);
      a.new_len[s] = need < 0 ? -1 : m.pos[s] + m.off[s + 1] - m.off[s];
      if (need >= 0) {
        a.held[m.slot[s]] = need;
        if (need > m.have[s]) given = max(given, m.more[s] + need - m.have[s]);
      } else if (!none && m.have[s] >= 0) {
        out = true;
      }
    }
    if (out) atomicOr(a.status, STATUS_PAGES);
    if (given) atomicMax(&s_given, given);
    __syncthreads();
    if (tid == 0 && !none) *a.free_count = top - s_given;
  }

  // ---- rows ----
  bool wild = false;
  const int64_t stride = (int64_t)ctas * THREADS;
  for (int64_t t0 = (int64_t)rank * THREADS + tid; t0 < a.total; t0 += FEW * stride) {
    int32_t* entry[FEW];  // where the row's page stands or is entered; null where the row has none
    int id[FEW], at[FEW];
    bool enters[FEW];
#pragma unroll
    for (int u = 0; u < FEW; ++u) {
      const int64_t t = t0 + u * stride;
      entry[u] = nullptr;
      if (t >= a.total) continue;
      int lo = 0, n = a.S;  // the last request that begins at t or before it
      while (n > 1) {
        const int half = n >> 1;
        if (m.off[lo + half] <= t) {
          lo += half;
          n -= half;
        } else {
          n = half;
        }
      }
      if (t < m.off[lo] || t >= m.off[lo + 1] || wants(lo) < 0) continue;
      const int have = m.have[lo], p = m.pos[lo] + (int)(t - m.off[lo]), i = p >> a.shift;
      at[u] = p & (page - 1);
      entry[u] = a.table + (int64_t)m.slot[lo] * a.width + i;
      enters[u] = i >= have && at[u] == 0;
      id[u] = i < have ? *entry[u] : __ldcg(a.free_list + (top - 1 - (m.more[lo] + i - have)));
    }
#pragma unroll
    for (int u = 0; u < FEW; ++u) {
      const int64_t t = t0 + u * stride;
      if (t >= a.total) break;
      int to = -1;
      if (entry[u]) {
        if (enters[u]) *entry[u] = id[u];
        if (id[u] >= 0 && id[u] < a.pages) to = (id[u] << a.shift) + at[u];
        else wild = true;
      }
      a.slot_map[t] = to;
    }
  }
  if (wild) atomicOr(a.status, STATUS_KV_RANGE);
}

// ---------------------------------------------------------------- append

struct Append {
  const void* src[2];
  void* pages[2];
  int64_t row[2], head[2];  // strides of the source in elements
  const int32_t* slot_map;
  int total, heads, shift;
  int64_t places;  // pages * positions of one
  unsigned* status;
};

template <typename T>
__device__ __forceinline__ uint32_t pair_of(float a, float b) {
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// Cached type T; F32: rows come in fp32 and are rounded.  A thread's piece is one of K
// and the same one of V, so that two rows and the place are on their way at once.
template <int D, typename T, bool F32>
__global__ void __launch_bounds__(256) paged_append_kernel(const Append a) {
  constexpr int VPR = D / 8;  // 16-byte pieces of a cached row
  const uint32_t per_row = (uint32_t)a.heads * VPR, items = (uint32_t)a.total * per_row;
  auto take = [&](const void* src, int64_t from) {
    if constexpr (F32) {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(src) + from);
      const float4 f = __ldg(p), g = __ldg(p + 1);
      return make_uint4(pair_of<T>(f.x, f.y), pair_of<T>(f.z, f.w), pair_of<T>(g.x, g.y), pair_of<T>(g.z, g.w));
    } else {
      return __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(src) + from));
    }
  };
  for (uint32_t it = blockIdx.x * 256u + threadIdx.x; it < items; it += gridDim.x * 256u) {
    const uint32_t t = it / per_row, hv = it - t * per_row, h = hv / VPR, v = hv % VPR;
    const int to = __ldg(a.slot_map + t);
    const uint4 k = take(a.src[0], t * a.row[0] + h * a.head[0] + v * 8);
    const uint4 x = take(a.src[1], t * a.row[1] + h * a.head[1] + v * 8);
    if (to >= 0 && to < a.places) {
      const int64_t page = to >> a.shift, at = to & ((1 << a.shift) - 1);
      const int64_t place = ((((page * a.heads + h) << a.shift) + at) * D) / 8 + v;
      static_cast<uint4*>(a.pages[0])[place] = k;
      static_cast<uint4*>(a.pages[1])[place] = x;
    } else if (to != -1 && hv == 0) {
      atomicOr(a.status, STATUS_KV_RANGE);
    }
  }
}

template <int D, typename T>
int append_as(const PagedAppend& c, const Append& a, cudaStream_t s) {
  const int64_t blocks = ((int64_t)a.total * a.heads * (D / 8) + 255) / 256;
  const int64_t most = (int64_t)c.num_sms * 8;
  const unsigned grid = (unsigned)(blocks < most ? blocks : most);
  if (c.dtype == Q4_DTYPE_F32) paged_append_kernel<D, T, true><<<grid, 256, 0, s>>>(a);
  else paged_append_kernel<D, T, false><<<grid, 256, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? Q4_OK : Q4_ERR_CUDA;
}

}  // namespace

int launch_paged_reserve(const PagedReserve& c, cudaStream_t s) {
  Reserve a{c.table, c.held, c.free_list, c.free_count, (int)c.slots, (int)c.width, (int)c.pages, c.shift,
            (int)c.S, c.total, c.offsets, c.slot, c.pos, c.slot_map, c.new_len, c.status};
  const size_t smem = ReserveSmem::bytes(a.S, a.slots);
  static std::atomic<bool> sized[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return Q4_ERR_CUDA;
  if (!sized[dev].load()) {
    if (cudaFuncSetAttribute(reserve_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)ReserveSmem::bytes(PAGED_REQUESTS, PAGED_SLOTS)) != cudaSuccess)
      return Q4_ERR_CUDA;
    sized[dev].store(true);
  }
  const int ctas = c.total + c.S <= ONE_CTA ? 1 : CLUSTER;
  if (ctas == 1) {  // a cluster of one by itself
    reserve_kernel<<<1, THREADS, smem, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? Q4_OK : Q4_ERR_CUDA;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = ctas;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, reserve_kernel, a) == cudaSuccess ? Q4_OK : Q4_ERR_CUDA;
}

int launch_paged_append(const PagedAppend& c, cudaStream_t s) {
  Append a{{c.k_new, c.v_new}, {c.k_pages, c.v_pages}, {c.k_strides[0], c.v_strides[0]},
           {c.k_strides[1], c.v_strides[1]}, c.slot_map, (int)c.total, (int)c.heads, c.shift, c.pages << c.shift,
           c.status};
  if (c.cache_dtype == Q4_DTYPE_F16)
    return c.head_dim == 128 ? append_as<128, __half>(c, a, s) : append_as<64, __half>(c, a, s);
  return c.head_dim == 128 ? append_as<128, __nv_bfloat16>(c, a, s) : append_as<64, __nv_bfloat16>(c, a, s);
}

}  // namespace q4
