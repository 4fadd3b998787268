// q4_kvq.cu — rows into and out of the 4-bit KV cache.
//
// Append: each 32-value block of a new K or V row becomes a scale d = m / -8
// (m the first value of largest magnitude) and codes q = clamp(round(x / d) +
// 8, 0, 15) with IEEE fp32 division and round-half-away, the rule of
// q4_quantize, so the cache costs 4.5 bits a value where the 16-bit cache of
// q4_kv_append costs 16.  Read: the rows back as (q - 8) * d.
//
// A decode step is bound by the latency of a few loads one after another: 64 rows
// of 4 x 128 fp32 values appended and read back take 5.6 us together (two
// launches).  Long appends are bound by instruction issue (about 250 per warp
// and 256 values, the request's lookup included): 4,569 rows of bf16, 9.4 MB in
// and 2.6 MB out, 13.2 us with the read back, of which the append is 10.5;
// dividing every value cost it 12.1.  A warp takes K or V of one packed row, all
// heads: it finds the row's request once (32 offsets a load) while the row's first
// values are on their way; a lane owns one 32-bit word of codes (eight values) at
// a time, so its loads or stores of values are 16 or 32 bytes, and a block's
// largest magnitude is found with two shuffles among the four lanes that hold it.
#include "q4_kvq.cuh"

namespace q4 {
namespace {

constexpr int ROW_THREADS = 128;

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

// Quantizes the eight values of word j of a block (the quad of lanes has the
// block): its codes, and the block's scale.  status: what was wrong with it.
// WIDE: the values have more than 16 bits.
template <bool WIDE>
__device__ __forceinline__ uint32_t quantize_word(const float (&v)[8], int j, int lane, uint16_t* scale,
                                                  unsigned* status) {
  // the first value of largest magnitude (lowest index among equals), and
  // whether all are finite
  float m = v[0];
  bool finite = isfinite(v[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    finite = finite && isfinite(v[i]);
    if (fabsf(v[i]) > fabsf(m)) m = v[i];
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    const float om = __shfl_xor_sync(0xFFFFFFFFu, m, o);
    const bool take = (j & o) ? fabsf(om) >= fabsf(m) : fabsf(om) > fabsf(m);  // the lower lane's on equality
    m = take ? om : m;
  }
  const unsigned odd = __ballot_sync(0xFFFFFFFFu, !finite) >> (lane & 28) & 0xFu;
  const float d = m * -0.125f;
  const uint16_t d16 = __half_as_ushort(__float2half_rn(d));
  if (odd || (d16 & 0x7C00u) == 0x7C00u) {
    // a block that binary16 cannot scale reads back as NaN, as the values themselves would
    *status = odd ? STATUS_KV_NONFINITE : STATUS_KV_SCALE;
    *scale = 0x7FFFu;
    return 0x99999999u;
  }
  if ((d16 & 0x7FFFu) == 0) {  // a scale of 0 (or -0) makes every value 0 whatever its code
    *scale = 0;
    return 0x88888888u;
  }
  // x / d to the nearest integer, halves away from zero.  |x / d| is about 8 at
  // most, and y = x * (1 / d) has a relative error below 2^-22.
  // Values of 16 bits: x / d is a half exactly, or off it by 2^-15.1 of itself or more
  // (x - h d is a whole number of units of d's last place, of which h d has
  // 17 * 2^11 at most).  So y a little larger, by 2^-18, is never near a half.
  // Values of 32 bits: the few y near a half, 2^-17, divide.
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));  // within 2^-23; |d| is 2^-25 or more
  if (!WIDE) r *= 1.0f + 0x1p-18f;
  constexpr float BASE = 0x1.8p23f;  // BASE + y holds y's integer in its low bits
  float t[8];
  bool clear = true;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float y = v[i] * r;
    t[i] = y + BASE;
    if (WIDE) clear = clear && fabsf(y - (t[i] - BASE)) < 0.5f - 0x1p-17f;
  }
  if (WIDE && !clear) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!(fabsf(v[i] * r - (t[i] - BASE)) < 0.5f - 0x1p-17f))
        t[i] = roundf(__fdiv_rn(v[i], d)) + BASE;  // roundf: half away from zero
  }
  uint32_t codes = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    codes |= (uint32_t)min(max(__float_as_int(t[i]) - (0x4B400000 - 8), 0), 15) << (4 * i);
  *scale = d16;
  return codes;
}

template <int D, typename T>
__global__ void __launch_bounds__(ROW_THREADS) kvq_append_kernel(const AppendArgs<T> a) {
  using L = Kvq<D>;
  constexpr int LPR = D / 8, ROWS = 32 / LPR;  // lanes per row, heads that a warp takes at once
  const int lane = threadIdx.x & 31;
  const int w = lane % LPR, b = w >> 2, j = w & 3;
  asm volatile("griddepcontrol.launch_dependents;");
  const int units = 2 * (int)a.total;  // (row, K or V); below 2^31: checked on the host
  for (int u = blockIdx.x * (ROW_THREADS / 32) + (threadIdx.x >> 5); u < units; u += gridDim.x * (ROW_THREADS / 32)) {
    const int kv = u & 1, t = u >> 1;
    const int64_t s_head = kv ? a.s_head[1] : a.s_head[0];
    const T* src = kv ? a.src[1] + t * a.s_token[1] : a.src[0] + t * a.s_token[0];
    src += w * 8;
    int h = lane / LPR;
    float v[8] = {};
    if (h < a.heads) kvq_load8<false>(src + h * s_head, v);
    const int s = kvq_find_request<false>(a.offsets, a.S, t, lane);
    const KvqRequest q = kvq_request<false>(a.offsets, a.slot, a.pos, s);
    if (t < q.b || t >= q.e) continue;  // a packed row that belongs to no request
    if (!q.ok(a.total, a.slots, a.capacity)) {
      if (lane == 0) atomicOr(a.status, STATUS_KV_RANGE);
      continue;  // the whole request is left unwritten
    }
    const int p = (int)(q.pos + (t - q.b)), row = p % L::POS;
    uint8_t* tile = a.cache + q.slot * a.heads * a.plane_bytes + (int64_t)(p / L::POS) * L::BYTES;
    for (int h0 = 0; h0 < a.heads; h0 += ROWS) {
      float next[8] = {};
      if (h + ROWS < a.heads) kvq_load8<false>(src + (h + ROWS) * s_head, next);
      uint16_t d16;
      unsigned bad = 0;
      const uint32_t codes = quantize_word<sizeof(T) == 4>(v, j, lane, &d16, &bad);
      if (h < a.heads) {
        if (bad && j == 0) atomicOr(a.status, bad);
        uint8_t* dst = tile + h * a.plane_bytes;
        if (kv == 0) {
          *reinterpret_cast<uint32_t*>(dst + kvq_k_word<D>(row, b, j)) = codes;
        } else {
          *reinterpret_cast<uint16_t*>(dst + kvq_v_half<D>(row, b, 2 * j)) = (uint16_t)codes;
          *reinterpret_cast<uint16_t*>(dst + kvq_v_half<D>(row, b, 2 * j + 1)) = (uint16_t)(codes >> 16);
        }
        if (j == 0) *reinterpret_cast<uint16_t*>(dst + kvq_scale<D>(kv, row, b)) = d16;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = next[i];
      h += ROWS;
    }
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

// The reads' launch begins under the end of the one before, whose kernel may have
// had the cache's older lines in the L1: codes and scales are loaded past it.
__device__ __forceinline__ void load2(const uint32_t* p, uint32_t* w) {
  const uint2 v = __ldcg(reinterpret_cast<const uint2*>(p));
  w[0] = v.x;
  w[1] = v.y;
}

template <int D, typename T>
__global__ void __launch_bounds__(ROW_THREADS) kvq_read_kernel(const ReadArgs<T> a) {
  using L = Kvq<D>;
  constexpr int LPR = D / 8, ROWS = 32 / LPR;
  const int lane = threadIdx.x & 31;
  const int w = lane % LPR, b = w >> 2, j = w & 3;
  const int units = 2 * (int)a.total;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // K and V of neighbouring rows go to the warps of a CTA: V's rows share their memory sectors
  for (int u = blockIdx.x * (ROW_THREADS / 32) + (threadIdx.x >> 5); u < units; u += gridDim.x * (ROW_THREADS / 32)) {
    const int kv = u & 1, t = u >> 1;
    const int s = kvq_find_request<true>(a.offsets, a.S, t, lane);
    const KvqRequest q = kvq_request<true>(a.offsets, a.slot, a.pos, s);
    T* dst = (kv ? a.dst[1] : a.dst[0]) + (int64_t)t * a.heads * D + w * 8;
    bool held = t >= q.b && t < q.e;
    if (held && !q.ok(a.total, a.slots, a.capacity)) {
      if (lane == 0) atomicOr(a.status, STATUS_KV_RANGE);
      held = false;
    }
    const int p = held ? (int)(q.pos + (t - q.b)) : 0, row = p % L::POS;
    const uint8_t* tile = a.cache + (held ? q.slot * a.heads * a.plane_bytes + (int64_t)(p / L::POS) * L::BYTES : 0);
#pragma unroll 2
    for (int h = lane / LPR; h < a.heads; h += ROWS) {
      float v[8] = {};
      if (held) {
        const uint8_t* src = tile + h * a.plane_bytes;
        uint32_t codes;
        if (kv == 0) {
          codes = __ldcg(reinterpret_cast<const uint32_t*>(src + kvq_k_word<D>(row, b, j)));
        } else {
          codes = __ldcg(reinterpret_cast<const uint16_t*>(src + kvq_v_half<D>(row, b, 2 * j))) |
                  (uint32_t)__ldcg(reinterpret_cast<const uint16_t*>(src + kvq_v_half<D>(row, b, 2 * j + 1))) << 16;
        }
        const float d = __half2float(
            __ushort_as_half(__ldcg(reinterpret_cast<const uint16_t*>(src + kvq_scale<D>(kv, row, b)))));
        uint32_t r[4];
        kvq_unpack_centred(codes, r);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r[i]));
          v[i] = f.x * d;
          v[i + 4] = f.y * d;
        }
      }
      kvq_store8(dst + h * D, v);
    }
  }
}

// The same for steps of long runs of rows: a warp takes the rows of one head
// that lie in eight neighbouring positions (aligned), so it reads K's and V's
// codes of all of them as 512 consecutive bytes each (D = 128) and finds the
// request once.  Rows 8c .. 8c + 7 of the step are one CTA warp's; they lie in
// two such groups at most unless a request ends among them.  65,536 rows of
// 4 heads (32 requests, bf16) take 27.5 us, 38 MB of cache in and 134 MB of values
// out: 6.2 TB/s, bound by memory.
template <int D, typename T>
__global__ void __launch_bounds__(ROW_THREADS) kvq_read_groups_kernel(const ReadArgs<T> a) {
  using L = Kvq<D>;
  constexpr int NB = L::NB;
  const int lane = threadIdx.x & 31;
  const int g = lane >> 2, tq = lane & 3;
  const int chunks = (int)((a.total + 7) / 8), units = chunks * (int)a.heads;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int u = blockIdx.x * (ROW_THREADS / 32) + (threadIdx.x >> 5); u < units; u += gridDim.x * (ROW_THREADS / 32)) {
    const int h = u % (int)a.heads, c = u / (int)a.heads;
    const int t_end = (int)min(a.total, (int64_t)8 * c + 8);
    for (int t = 8 * c; t < t_end;) {
      const int s = kvq_find_request<true>(a.offsets, a.S, t, lane);
      const KvqRequest q = kvq_request<true>(a.offsets, a.slot, a.pos, s);
      bool held = t >= q.b && t < q.e;
      // rows up to the request's end, or (outside of one) up to the next one's beginning
      int stop = t_end;
      if (held) stop = (int)min((int64_t)stop, q.e);
      else if (t < q.b) stop = (int)min((int64_t)stop, q.b);
      else if (s + 1 < a.S) stop = (int)min((int64_t)stop, max((int64_t)kvq_ld<true>(a.offsets + s + 1), (int64_t)t + 1));
      if (held && !q.ok(a.total, a.slots, a.capacity)) {
        if (lane == 0) atomicOr(a.status, STATUS_KV_RANGE);
        held = false;
      }
      const int p = held ? (int)(q.pos + (t - q.b)) : 0;
      const int first = p & 7;  // the group's rows are positions p - first ..
      if (held) stop = min(stop, t + 8 - first);
      const int count = stop - t;
      // lane (g, tq): K words j = tq of row g; V words of group g of the pair 2 tq, 2 tq + 1
      uint32_t kw[NB], vw[NB], ks[NB], vs[NB];
      if (held) {
        const uint8_t* tile = a.cache + (q.slot * a.heads + h) * a.plane_bytes + (int64_t)(p / L::POS) * L::BYTES;
        const int r0 = (p % L::POS) & ~7;
        const uint32_t* k = reinterpret_cast<const uint32_t*>(tile + r0 * L::ROW) + lane * NB;
        const uint32_t* v = reinterpret_cast<const uint32_t*>(tile + L::V_OFF + r0 * L::ROW) + lane * NB;
        const uint32_t* kd = reinterpret_cast<const uint32_t*>(tile + kvq_scale<D>(0, r0 + (g & 6), 0));
        const uint32_t* vd = reinterpret_cast<const uint32_t*>(tile + kvq_scale<D>(1, r0 + 2 * tq, 0));
#pragma unroll
        for (int b = 0; b < NB; b += 2) {
          load2(k + b, kw + b);
          load2(v + b, vw + b);
          load2(kd + b, ks + b);
          load2(vd + b, vs + b);
        }
      } else {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          kw[b] = vw[b] = 0x88888888u;
          ks[b] = vs[b] = 0;
        }
      }
      // row r of the group is packed row t + r - first
      auto in = [&](int r) { return r >= first && r < first + count; };
      const int64_t width = a.heads * D;
      T* kd = a.dst[0] + (int64_t)(t + g - first) * width + h * D + 8 * tq;
      T* vd = a.dst[1] + (int64_t)(t + 2 * tq - first) * width + h * D + 4 * g;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const float2 dk = __half22float2(*reinterpret_cast<const __half2*>(&ks[b]));
        const float2 dv = __half22float2(*reinterpret_cast<const __half2*>(&vs[b]));
        const float d = (g & 1) ? dk.y : dk.x;
        uint32_t r[4];
        float x[8], even[4], odd[4];
        kvq_unpack_centred(kw[b], r);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r[i]));
          x[i] = f.x * d;
          x[i + 4] = f.y * d;
        }
        if (in(g)) kvq_store8(kd + 32 * b, x);
        kvq_unpack_centred(vw[b], r);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r[i]));
          even[i] = f.x * dv.x;
          odd[i] = f.y * dv.y;
        }
        if (in(2 * tq)) kvq_store4(vd + 32 * b, even);
        if (in(2 * tq + 1)) kvq_store4(vd + width + 32 * b, odd);
      }
      t = stop;
    }
  }
}

// CTAs for so many warps' work.
unsigned row_blocks(int64_t warps, int num_sms) {
  constexpr int PER = ROW_THREADS / 32;
  const int64_t need = (warps + PER - 1) / PER, most = (int64_t)num_sms * (2048 / ROW_THREADS);
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
  const unsigned grid = row_blocks(2 * c.total, c.num_sms);
  if (c.head_dim == 128) kvq_append_kernel<128, T><<<grid, ROW_THREADS, 0, s>>>(a);
  else kvq_append_kernel<64, T><<<grid, ROW_THREADS, 0, s>>>(a);
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
  // Groups pay where most rows have neighbours in their request (28 us against 51
  // for 32 x 2,048 rows); a decode step's single rows would wait for eight requests
  // one after another (9 us against 3 for 64).
  const bool groups = c.total >= 8 * (int64_t)c.S;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(row_blocks(groups ? (c.total + 7) / 8 * c.heads : 2 * c.total, c.num_sms));
  cfg.blockDim = dim3(ROW_THREADS);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const auto kernel = c.head_dim == 128 ? (groups ? kvq_read_groups_kernel<128, T> : kvq_read_kernel<128, T>)
                                        : (groups ? kvq_read_groups_kernel<64, T> : kvq_read_kernel<64, T>);
  return cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess ? Q4_OK : Q4_ERR_CUDA;
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
