// q4_attn_api.cu — C ABI of the 4-bit KV cache and of prompt attention:
// argument checks on the host, then one call into the launchers.
#include <cuda_runtime.h>

#include <cstdint>

#include "q4_checks.h"

using namespace q4;

namespace {

int check_cache(int64_t slots, int64_t heads, int64_t head_dim, int64_t capacity) {
  if (slots < 1 || heads < 1 || capacity < 1 || slots >= LIM || heads >= LIM || capacity > MOST)
    return Q4_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return Q4_ERR_SHAPE;
  // bytes and plane indexes stay far below 2^63
  if (slots > (LIM << 20) / heads) return Q4_ERR_INVALID_ARG;
  return slots * heads > ((int64_t)1 << 60) / kvq_plane_bytes(head_dim, capacity) ? Q4_ERR_INVALID_ARG : Q4_OK;
}

int check_step(const int32_t* offsets, const int32_t* slot, const int32_t* pos, int64_t S, int64_t total,
               int64_t heads) {
  if (S < 0 || S > MOST || total < 0 || total > MOST / 2 || total > MOST / heads)
    return Q4_ERR_INVALID_ARG;
  if (total > 0 && S > 0 && (!offsets || !slot || !pos)) return Q4_ERR_INVALID_ARG;
  return Q4_OK;
}

KvqStep make_step(int64_t slots, int64_t heads, int64_t head_dim, int64_t capacity, const int32_t* offsets,
                  const int32_t* slot, const int32_t* pos, int64_t S, int64_t total, const ScratchLock& l) {
  return KvqStep{slots, heads, capacity, total, (int)head_dim, (int)S, offsets, slot, pos, l.ws.status, l.num_sms};
}

}  // namespace

extern "C" {

int q4_kvq_cache_bytes(int64_t slots, int64_t heads, int64_t head_dim, int64_t capacity, size_t* bytes) {
  if (!bytes) return Q4_ERR_INVALID_ARG;
  const int st = check_cache(slots, heads, head_dim, capacity);
  if (st) return st;
  *bytes = (size_t)(slots * heads) * (size_t)kvq_plane_bytes(head_dim, capacity);
  return Q4_OK;
}

int q4_kvq_append(void* cache, const void* k_new, const void* v_new, int dtype, int64_t slots, int64_t heads,
                  int64_t head_dim, int64_t capacity, const int64_t* k_strides, const int64_t* v_strides,
                  const int32_t* offsets, const int32_t* slot, const int32_t* pos, int64_t S, int64_t total,
                  cudaStream_t stream) {
  int st = check_cache(slots, heads, head_dim, capacity);
  if (!st) st = check_step(offsets, slot, pos, S, total, heads);
  if (st) return st;
  const int eb = elem_bytes(dtype);
  if (!eb || !strides_ok(k_strides) || !strides_ok(v_strides)) return Q4_ERR_INVALID_ARG;
  if (S == 0 || total == 0) return Q4_OK;
  if (!cache || !k_new || !v_new) return Q4_ERR_INVALID_ARG;
  if (!aligned16(cache) || !aligned16(k_new) || !aligned16(v_new) || !strides_aligned(k_strides, eb, total, heads) ||
      !strides_aligned(v_strides, eb, total, heads))
    return Q4_ERR_ALIGN;
  ScratchLock l;
  st = scratch_acquire(0, &l);
  if (st) return st;
  return launch_kvq_append(make_step(slots, heads, head_dim, capacity, offsets, slot, pos, S, total, l),
                           static_cast<uint8_t*>(cache), k_new, v_new, k_strides, v_strides, dtype, stream);
}

int q4_kvq_read(const void* cache, void* k_out, void* v_out, int dtype, int64_t slots, int64_t heads,
                int64_t head_dim, int64_t capacity, const int32_t* offsets, const int32_t* slot,
                const int32_t* pos, int64_t S, int64_t total, cudaStream_t stream) {
  int st = check_cache(slots, heads, head_dim, capacity);
  if (!st) st = check_step(offsets, slot, pos, S, total, heads);
  if (st) return st;
  if (!elem_bytes(dtype)) return Q4_ERR_INVALID_ARG;
  if (total == 0) return Q4_OK;
  if (!cache || !k_out || !v_out || S == 0) return Q4_ERR_INVALID_ARG;
  if (!aligned16(cache) || !aligned16(k_out) || !aligned16(v_out)) return Q4_ERR_ALIGN;
  const int64_t bytes = total * heads * head_dim * elem_bytes(dtype);
  if (meet(k_out, bytes, v_out, bytes)) return Q4_ERR_INVALID_ARG;
  ScratchLock l;
  st = scratch_acquire(0, &l);
  if (st) return st;
  return launch_kvq_read(make_step(slots, heads, head_dim, capacity, offsets, slot, pos, S, total, l),
                         static_cast<const uint8_t*>(cache), k_out, v_out, dtype, stream);
}

int q4_kvq_attention(const void* cache, const void* q, void* out, float* mass, int dtype, int64_t slots,
                     int64_t heads, int64_t q_heads, int64_t head_dim, int64_t capacity, const int64_t* q_strides,
                     float scale, const int32_t* offsets, const int32_t* slot, const int32_t* pos, int64_t S,
                     int64_t total, cudaStream_t stream) {
  int st = check_cache(slots, heads, head_dim, capacity);
  if (!st) st = check_step(offsets, slot, pos, S, total, heads);
  if (st) return st;
  const int eb = elem_bytes(dtype);
  if (!eb || !strides_ok(q_strides) || q_heads < 1 || q_heads % heads || !scale_ok(scale))
    return Q4_ERR_INVALID_ARG;
  if (q_heads > 65535 || total > MOST / q_heads) return Q4_ERR_SHAPE;  // a grid dimension; 32-bit row counts
  if (total == 0) return Q4_OK;
  if (!cache || !q || !out || S == 0) return Q4_ERR_INVALID_ARG;
  if (!aligned16(cache) || !aligned16(q) || !aligned16(out) || !strides_aligned(q_strides, eb, total, q_heads)) return Q4_ERR_ALIGN;
  // a row's queries are read before it is written, but the weights read them again
  const Rows queries(q, q_strides, total, q_heads, head_dim, eb);
  const int64_t out_bytes = total * q_heads * head_dim * eb;
  if (queries.meets(out, out_bytes) && (mass || !queries.same(out, q_heads, head_dim, eb))) return Q4_ERR_INVALID_ARG;
  if (mass && meet(mass, slots * heads * capacity * 4, out, out_bytes)) return Q4_ERR_INVALID_ARG;
  ScratchLock l;
  st = scratch_acquire(0, &l);
  if (st) return st;
  const size_t need = kvq_attn_scratch_bytes(S, total, (int)q_heads, mass != nullptr, l.num_sms, nullptr, nullptr);
  if (need > l.ws.attn_bytes) {
    l.lock.unlock();
    st = scratch_acquire(need, &l);
    if (st) return st;
  }
  KvqAttnScratch ws;
  kvq_attn_scratch_bytes(S, total, (int)q_heads, mass != nullptr, l.num_sms, &ws, l.ws.attn);
  return launch_kvq_attention(make_step(slots, heads, head_dim, capacity, offsets, slot, pos, S, total, l),
                              static_cast<const uint8_t*>(cache), q, q_strides, (int)q_heads, scale, out, mass, dtype,
                              ws, stream);
}

int q4_kvq_evict(void* cache, float* mass, int64_t slots, int64_t heads, int64_t head_dim, int64_t capacity,
                 const int32_t* src, const int32_t* dst, const int32_t* len, int64_t S, int64_t keep, int64_t recent,
                 int32_t* new_len, int32_t* kept, cudaStream_t stream) {
  int st = check_cache(slots, heads, head_dim, capacity);
  if (st) return st;
  if (S < 0 || S > MOST || keep < 1 || keep > capacity || recent < 0 || recent > keep)
    return Q4_ERR_INVALID_ARG;
  if (S == 0) return Q4_OK;
  if (!cache || !mass || !src || !dst || !len || !new_len || !kept) return Q4_ERR_INVALID_ARG;
  // a grid dimension, and the 32-bit item index of one plane's copy
  if (S * heads > 65535 || keep > INT32_MAX / 16) return Q4_ERR_SHAPE;
  if (!aligned16(cache)) return Q4_ERR_ALIGN;
  for (const int32_t* in : {src, dst, len})  // read by every CTA, whichever writes first
    if (meet(in, S * 4, new_len, S * 4) || meet(in, S * 4, kept, S * heads * keep * 4)) return Q4_ERR_INVALID_ARG;
  if (meet(new_len, S * 4, kept, S * heads * keep * 4)) return Q4_ERR_INVALID_ARG;
  ScratchLock l;
  st = scratch_acquire(0, &l);
  if (st) return st;
  const KvqEvict c{static_cast<uint8_t*>(cache), mass, slots, heads, capacity, (int)head_dim, (int)S, (int)keep,
                   (int)recent, src, dst, len, new_len, kept, l.ws.status, l.num_sms};
  return launch_kvq_evict(c, stream);
}

int q4_prompt_attention(const void* q, const void* k, const void* v, void* out, int dtype, int64_t q_heads,
                        int64_t kv_heads, int64_t head_dim, const int64_t* q_strides, const int64_t* k_strides,
                        const int64_t* v_strides, float scale, int causal, const int32_t* q_offsets,
                        const int32_t* k_offsets, int64_t S, int64_t q_total, int64_t k_total, cudaStream_t stream) {
  if (dtype != Q4_DTYPE_F16 && dtype != Q4_DTYPE_BF16) return Q4_ERR_INVALID_ARG;
  if (!strides_ok(q_strides) || !strides_ok(k_strides) || !strides_ok(v_strides) || !scale_ok(scale) ||
      q_heads < 1 || kv_heads < 1 || q_heads % kv_heads || S < 0 || S > MOST || q_total < 0 || q_total > MOST ||
      k_total < 0 || k_total > MOST)
    return Q4_ERR_INVALID_ARG;
  // one tile of 128 rows takes all query heads of a key/value head; 32-bit output row index
  if ((head_dim != 64 && head_dim != 128) || q_heads / kv_heads > 128 || q_heads >= 65536 ||
      q_total > MOST / q_heads)
    return Q4_ERR_SHAPE;
  if (q_total == 0) return Q4_OK;
  if (!q || !out || S == 0 || !q_offsets || !k_offsets || (k_total > 0 && (!k || !v))) return Q4_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || !strides_aligned(q_strides, 2, q_total, q_heads) ||
      !strides_aligned(k_strides, 2, k_total, kv_heads) || !strides_aligned(v_strides, 2, k_total, kv_heads))
    return Q4_ERR_ALIGN;
  // a tile's queries are read before its rows are written, keys and values by other tiles too
  const Rows queries(q, q_strides, q_total, q_heads, head_dim, 2);
  const int64_t out_bytes = q_total * q_heads * head_dim * 2;
  if ((queries.meets(out, out_bytes) && !queries.same(out, q_heads, head_dim, 2)) ||
      Rows(k, k_strides, k_total, kv_heads, head_dim, 2).meets(out, out_bytes) ||
      Rows(v, v_strides, k_total, kv_heads, head_dim, 2).meets(out, out_bytes))
    return Q4_ERR_INVALID_ARG;
  ScratchLock l;
  const int st = scratch_acquire(0, &l);
  if (st) return st;
  if (!l.sm103) return Q4_ERR_UNSUPPORTED;
  PromptAttn c{q, k, v, out, {q_strides[0], q_strides[1]}, {k_strides[0], k_strides[1]},
               {v_strides[0], v_strides[1]}, q_total, k_total, dtype, (int)q_heads, (int)kv_heads, (int)head_dim,
               (int)S, causal ? 1 : 0, scale, q_offsets, k_offsets, l.ws.status, l.num_sms};
  return launch_prompt_attention(c, stream);
}

}  // extern "C"
