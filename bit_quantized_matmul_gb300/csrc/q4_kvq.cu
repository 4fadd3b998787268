// q4_kvq.cu — rows into and out of the 4-bit KV cache.
//
// Append: each 32-value block of a new K or V row becomes a scale d = m / -8
// (m the first value of largest magnitude) and codes q = clamp(round(x / d) +
// 8, 0, 15) with IEEE fp32 division and round-half-away, the rule of
// q4_quantize, so the cache costs 4.5 bits a value where the 16-bit cache of
// q4_kv_append costs 16.  Read: the rows back as (q - 8) * d.
//
// Both are bound by memory: a thread owns one 32-bit word of codes (eight
// values), so a row is D/8 neighbouring lanes, its loads are 16 or 32 bytes a
// lane and its codes one 32- or 64-byte run; a block's largest magnitude is
// found with two shuffles among the four lanes that hold it.
#include "q4_kvq.cuh"

namespace q4 {
namespace {

template <typename T>
struct AppendArgs {
  uint8_t* cache;
  const T* src[2];                  // K, V new rows
  int64_t s_token[2], s_head[2];    // their strides in elements
  int64_t slots, heads, capacity, total, plane_bytes;
  const int32_t *offsets, *slot, *pos;
  int S;
  unsigned* status;
};

template <int D, typename T>
__global__ void __launch_bounds__(256) kvq_append_kernel(const AppendArgs<T> a) {
  using L = Kvq<D>;
  constexpr int LPR = D / 8;  // lanes per row
  const int64_t rows = a.total * a.heads;
  const int kv = blockIdx.y;
  const int w = threadIdx.x % LPR;  // word of the row: block w / 4, word w % 4 of the block
  const int b = w >> 2, j = w & 3;
  // whole rows per step, so the four lanes of a block always run together
  for (int64_t r = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / LPR; r < rows;
       r += (int64_t)gridDim.x * blockDim.x / LPR) {
    const int64_t t = r / a.heads, h = r - t * a.heads;
    const int s = kvq_find_request(a.offsets, a.S, t);
    const KvqRequest q = kvq_request(a.offsets, a.slot, a.pos, s);
    if (t < q.b || t >= q.e) continue;  // a packed row that belongs to no request
    if (!q.ok(a.total, a.slots, a.capacity)) {
      if (kv == 0 && w == 0 && h == 0) atomicOr(a.status, STATUS_KV_RANGE);
      continue;  // the whole request is left unwritten
    }
    float v[8];
    kvq_load8(a.src[kv] + t * a.s_token[kv] + h * a.s_head[kv] + w * 8, v);
    // the first value of largest magnitude (lowest index among equals), and
    // whether all are finite: NaN and infinity have the largest exponent
    float m = v[0];
    bool finite = isfinite(v[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) {
      finite = finite && isfinite(v[i]);
      if (fabsf(v[i]) > fabsf(m)) m = v[i];
    }
    const unsigned quad = 0xFu << (threadIdx.x & 28);  // the block's four lanes
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      const float om = __shfl_xor_sync(quad, m, o);
      const bool take = (j & o) ? fabsf(om) >= fabsf(m) : fabsf(om) > fabsf(m);  // the lower lane's on equality
      m = take ? om : m;
    }
    finite = __all_sync(quad, finite);
    const float d = __fdiv_rn(m, -8.0f);
    uint16_t d16 = __half_as_ushort(__float2half_rn(d));
    uint32_t codes = 0;
    if (!finite || (d16 & 0x7C00u) == 0x7C00u) {
      // a block that binary16 cannot scale reads back as NaN, as the values themselves would
      if (j == 0) atomicOr(a.status, finite ? STATUS_KV_SCALE : STATUS_KV_NONFINITE);
      d16 = 0x7FFFu;
      codes = 0x99999999u;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        int qi = 8;
        if (d != 0.0f) {
          qi = (int)roundf(__fdiv_rn(v[i], d)) + 8;  // roundf: half away from zero
          qi = qi < 0 ? 0 : (qi > 15 ? 15 : qi);
        }
        codes |= (uint32_t)qi << (4 * i);
      }
    }
    const int64_t p = q.pos + (t - q.b);
    const int row = (int)(p % L::POS);
    uint8_t* tile = a.cache + (q.slot * a.heads + h) * a.plane_bytes + p / L::POS * L::BYTES;
    if (kv == 0) {
      *reinterpret_cast<uint32_t*>(tile + kvq_k_word<D>(row, b, j)) = codes;
    } else {
      *reinterpret_cast<uint16_t*>(tile + kvq_v_half<D>(row, b, 2 * j)) = (uint16_t)codes;
      *reinterpret_cast<uint16_t*>(tile + kvq_v_half<D>(row, b, 2 * j + 1)) = (uint16_t)(codes >> 16);
    }
    if (j == 0) *reinterpret_cast<uint16_t*>(tile + kvq_scale<D>(kv, row, b)) = d16;
  }
}

template <typename T>
struct ReadArgs {
  const uint8_t* cache;
  T* dst[2];  // [total, heads, D] contiguous
  int64_t slots, heads, capacity, total, plane_bytes;
  const int32_t *offsets, *slot, *pos;
  int S;
  unsigned* status;
};

template <int D, typename T>
__global__ void __launch_bounds__(256) kvq_read_kernel(const ReadArgs<T> a) {
  using L = Kvq<D>;
  constexpr int LPR = D / 8;
  const int64_t rows = a.total * a.heads;
  const int kv = blockIdx.y;
  const int w = threadIdx.x % LPR;
  const int b = w >> 2, j = w & 3;
  for (int64_t r = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / LPR; r < rows;
       r += (int64_t)gridDim.x * blockDim.x / LPR) {
    const int64_t t = r / a.heads, h = r - t * a.heads;
    const int s = kvq_find_request(a.offsets, a.S, t);
    const KvqRequest q = kvq_request(a.offsets, a.slot, a.pos, s);
    float v[8] = {};
    if (t >= q.b && t < q.e) {
      if (!q.ok(a.total, a.slots, a.capacity)) {
        if (kv == 0 && w == 0 && h == 0) atomicOr(a.status, STATUS_KV_RANGE);
      } else {
        const int64_t p = q.pos + (t - q.b);
        const int row = (int)(p % L::POS);
        const uint8_t* tile = a.cache + (q.slot * a.heads + h) * a.plane_bytes + p / L::POS * L::BYTES;
        uint32_t codes;
        if (kv == 0) {
          codes = *reinterpret_cast<const uint32_t*>(tile + kvq_k_word<D>(row, b, j));
        } else {
          codes = *reinterpret_cast<const uint16_t*>(tile + kvq_v_half<D>(row, b, 2 * j)) |
                  (uint32_t)*reinterpret_cast<const uint16_t*>(tile + kvq_v_half<D>(row, b, 2 * j + 1)) << 16;
        }
        const float d =
            __half2float(__ushort_as_half(*reinterpret_cast<const uint16_t*>(tile + kvq_scale<D>(kv, row, b))));
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (float)((int)((codes >> (4 * i)) & 15u) - 8) * d;
      }
    }
    kvq_store8(a.dst[kv] + r * D + w * 8, v);
  }
}

// Blocks along x for `rows` rows of D values in each of the two planes.
unsigned row_blocks(int64_t rows, int D, int num_sms) {
  const int64_t per = 256 / (D / 8);
  const int64_t need = (rows + per - 1) / per, most = (int64_t)num_sms * 8;
  return (unsigned)(need < most ? need : most);
}

template <typename T>
int append_as(const KvqStep& c, const void* k_new, const void* v_new, const int64_t* ks, const int64_t* vs,
              uint8_t* cache, cudaStream_t s) {
  AppendArgs<T> a;
  a.cache = cache;
  a.src[0] = static_cast<const T*>(k_new);
  a.src[1] = static_cast<const T*>(v_new);
  a.s_token[0] = ks[0];
  a.s_head[0] = ks[1];
  a.s_token[1] = vs[0];
  a.s_head[1] = vs[1];
  a.slots = c.slots;
  a.heads = c.heads;
  a.capacity = c.capacity;
  a.total = c.total;
  a.plane_bytes = kvq_plane_bytes(c.head_dim, c.capacity);
  a.offsets = c.offsets;
  a.slot = c.slot;
  a.pos = c.pos;
  a.S = c.S;
  a.status = c.status;
  const dim3 grid(row_blocks(c.total * c.heads, c.head_dim, c.num_sms), 2);
  if (c.head_dim == 128) kvq_append_kernel<128, T><<<grid, 256, 0, s>>>(a);
  else kvq_append_kernel<64, T><<<grid, 256, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? Q4_OK : Q4_ERR_CUDA;
}

template <typename T>
int read_as(const KvqStep& c, const uint8_t* cache, void* k_out, void* v_out, cudaStream_t s) {
  ReadArgs<T> a;
  a.cache = cache;
  a.dst[0] = static_cast<T*>(k_out);
  a.dst[1] = static_cast<T*>(v_out);
  a.slots = c.slots;
  a.heads = c.heads;
  a.capacity = c.capacity;
  a.total = c.total;
  a.plane_bytes = kvq_plane_bytes(c.head_dim, c.capacity);
  a.offsets = c.offsets;
  a.slot = c.slot;
  a.pos = c.pos;
  a.S = c.S;
  a.status = c.status;
  const dim3 grid(row_blocks(c.total * c.heads, c.head_dim, c.num_sms), 2);
  if (c.head_dim == 128) kvq_read_kernel<128, T><<<grid, 256, 0, s>>>(a);
  else kvq_read_kernel<64, T><<<grid, 256, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? Q4_OK : Q4_ERR_CUDA;
}

}  // namespace

int launch_kvq_append(const KvqStep& c, uint8_t* cache, const void* k_new, const void* v_new, const int64_t* ks,
                      const int64_t* vs, int dtype, cudaStream_t s) {
  if (dtype == Q4_DTYPE_F32) return append_as<float>(c, k_new, v_new, ks, vs, cache, s);
  if (dtype == Q4_DTYPE_F16) return append_as<__half>(c, k_new, v_new, ks, vs, cache, s);
  return append_as<__nv_bfloat16>(c, k_new, v_new, ks, vs, cache, s);
}

int launch_kvq_read(const KvqStep& c, const uint8_t* cache, void* k_out, void* v_out, int dtype, cudaStream_t s) {
  if (dtype == Q4_DTYPE_F32) return read_as<float>(c, cache, k_out, v_out, s);
  if (dtype == Q4_DTYPE_F16) return read_as<__half>(c, cache, k_out, v_out, s);
  return read_as<__nv_bfloat16>(c, cache, k_out, v_out, s);
}

}  // namespace q4
