// q4_paged_api.cu — C ABI of the paged 16-bit KV cache: argument checks on the
// host, then one call into the launchers.
#include <cuda_runtime.h>

#include <cstdint>

#include "q4_checks.h"

using namespace q4;

namespace {

// log2 of a page's positions, -1 where there is none
int page_shift(int64_t page_size) {
  return page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : page_size == 128 ? 7 : -1;
}

bool is16(int dtype) { return dtype == Q4_DTYPE_F16 || dtype == Q4_DTYPE_BF16; }

// Pages of a cache: places and the copies' coordinates stay in 32 bits.
int check_pages(int64_t pages, int64_t heads, int64_t head_dim, int64_t page_size) {
  if (pages < 1 || heads < 1 || pages >= LIM || heads >= LIM) return Q4_ERR_INVALID_ARG;
  if ((head_dim != 64 && head_dim != 128) || page_shift(page_size) < 0) return Q4_ERR_SHAPE;
  return pages > MOST / page_size || pages + 1 > MOST / heads / (page_size / 8) ? Q4_ERR_INVALID_ARG : Q4_OK;
}

int64_t pages_bytes(int64_t pages, int64_t heads, int64_t head_dim, int64_t page_size) {
  return pages * heads * page_size * head_dim * 2;  // at most 2^31 rows of eight: below 2^42
}

// A block table: positions of a slot stay in 32 bits.
int check_table(int64_t slots, int64_t width, int64_t page_size) {
  if (slots < 1 || width < 1 || slots >= LIM || width > MOST / page_size) return Q4_ERR_INVALID_ARG;
  return Q4_OK;
}

}  // namespace

extern "C" {

int q4_paged_reserve(int32_t* table, int32_t* held, int32_t* free_list, int32_t* free_count, int64_t slots,
                     int64_t width, int64_t pages, int64_t page_size, const int32_t* offsets, const int32_t* slot,
                     const int32_t* pos, int64_t S, int64_t total, int32_t* slot_map, int32_t* new_len,
                     cudaStream_t stream) {
  const int shift = page_shift(page_size);
  if (shift < 0) return Q4_ERR_SHAPE;
  int st = check_table(slots, width, page_size);
  if (st) return st;
  if (pages < 1 || pages > MOST / page_size || S < 0 || total < 0 || total > MOST / 2) return Q4_ERR_INVALID_ARG;
  if (S > PAGED_REQUESTS || slots > PAGED_SLOTS) return Q4_ERR_SHAPE;  // both lie in shared memory
  if (S == 0 && total == 0) return Q4_OK;
  if (S == 0 || !table || !held || !free_list || !free_count || !offsets || !slot || !pos || !new_len ||
      (total > 0 && !slot_map))
    return Q4_ERR_INVALID_ARG;
  // what the call writes overlaps nothing else
  const struct {
    const void* p;
    int64_t n;
  } out[] = {{table, slots * width * 4}, {held, slots * 4}, {free_list, pages * 4}, {free_count, 4},
             {new_len, S * 4}, {slot_map, total * 4}},
    in[] = {{offsets, (S + 1) * 4}, {slot, S * 4}, {pos, S * 4}};
  for (int i = 0; i < 6; ++i) {
    for (int j = i + 1; j < 6; ++j)
      if (meet(out[i].p, out[i].n, out[j].p, out[j].n)) return Q4_ERR_INVALID_ARG;
    for (const auto& x : in)
      if (meet(out[i].p, out[i].n, x.p, x.n)) return Q4_ERR_INVALID_ARG;
  }
  ScratchLock l;
  st = scratch_acquire(0, &l);
  if (st) return st;
  return launch_paged_reserve(PagedReserve{table, held, free_list, free_count, slots, width, pages, total, shift,
                                           (int)S, offsets, slot, pos, slot_map, new_len, l.ws.status},
                              stream);
}

int q4_paged_append(void* k_pages, void* v_pages, int cache_dtype, const void* k_new, const void* v_new, int dtype,
                    int64_t pages, int64_t heads, int64_t head_dim, int64_t page_size, const int64_t* k_strides,
                    const int64_t* v_strides, const int32_t* slot_map, int64_t total, cudaStream_t stream) {
  int st = check_pages(pages, heads, head_dim, page_size);
  if (st) return st;
  const int eb = elem_bytes(dtype);
  if (!is16(cache_dtype) || (dtype != cache_dtype && dtype != Q4_DTYPE_F32) || !strides_ok(k_strides) ||
      !strides_ok(v_strides) || total < 0 || total > MOST / heads / (head_dim / 8))
    return Q4_ERR_INVALID_ARG;
  if (total == 0) return Q4_OK;
  if (!k_pages || !v_pages || !k_new || !v_new || !slot_map) return Q4_ERR_INVALID_ARG;
  if (!aligned16(k_pages) || !aligned16(v_pages) || !aligned16(k_new) || !aligned16(v_new) ||
      !strides_aligned(k_strides, eb, total, heads) || !strides_aligned(v_strides, eb, total, heads))
    return Q4_ERR_ALIGN;
  const int64_t bytes = pages_bytes(pages, heads, head_dim, page_size);
  if (meet(k_pages, bytes, v_pages, bytes)) return Q4_ERR_INVALID_ARG;
  const Rows k(k_new, k_strides, total, heads, head_dim, eb), v(v_new, v_strides, total, heads, head_dim, eb);
  for (const void* p : {k_pages, v_pages})
    if (k.meets(p, bytes) || v.meets(p, bytes) || meet(p, bytes, slot_map, total * 4)) return Q4_ERR_INVALID_ARG;
  ScratchLock l;
  st = scratch_acquire(0, &l);
  if (st) return st;
  return launch_paged_append(PagedAppend{k_pages, v_pages, k_new, v_new, cache_dtype, dtype, pages, heads, total,
                                         (int)head_dim, page_shift(page_size), {k_strides[0], k_strides[1]},
                                         {v_strides[0], v_strides[1]}, slot_map, l.ws.status, l.num_sms},
                             stream);
}

int q4_paged_attention(const void* k_pages, const void* v_pages, const void* q, void* out, int dtype, int64_t pages,
                       int64_t heads, int64_t q_heads, int64_t head_dim, int64_t page_size, const int64_t* q_strides,
                       float scale, const int32_t* table, int64_t slots, int64_t width, const int32_t* offsets,
                       const int32_t* slot, const int32_t* pos, int64_t S, int64_t total, cudaStream_t stream) {
  int st = check_pages(pages, heads, head_dim, page_size);
  if (!st) st = check_table(slots, width, page_size);
  if (st) return st;
  if (!is16(dtype) || !strides_ok(q_strides) || q_heads < 1 || q_heads % heads || !scale_ok(scale) || S < 0 ||
      S > MOST || total < 0 || total > MOST / 2)
    return Q4_ERR_INVALID_ARG;
  // one tile of 128 rows takes all query heads of a key/value head; 32-bit output row index
  if (q_heads / heads > 128 || q_heads >= 65536 || total > MOST / q_heads) return Q4_ERR_SHAPE;
  if (total == 0) return Q4_OK;
  if (S == 0 || !k_pages || !v_pages || !q || !out || !table || !offsets || !slot || !pos) return Q4_ERR_INVALID_ARG;
  if (!aligned16(k_pages) || !aligned16(v_pages) || !aligned16(q) || !aligned16(out) ||
      !strides_aligned(q_strides, 2, total, q_heads))
    return Q4_ERR_ALIGN;
  // the tensor map of q takes strides below 2^40 bytes
  if ((total > 1 && q_strides[0] >= (LIM << 8)) || (q_heads > 1 && q_strides[1] >= (LIM << 8))) return Q4_ERR_INVALID_ARG;
  // a tile's queries are read before its rows are written
  const Rows queries(q, q_strides, total, q_heads, head_dim, 2);
  const int64_t out_bytes = total * q_heads * head_dim * 2, bytes = pages_bytes(pages, heads, head_dim, page_size);
  if ((queries.meets(out, out_bytes) && !queries.same(out, q_heads, head_dim, 2)) ||
      meet(out, out_bytes, k_pages, bytes) || meet(out, out_bytes, v_pages, bytes) ||
      meet(out, out_bytes, table, slots * width * 4) || meet(out, out_bytes, offsets, (S + 1) * 4) ||
      meet(out, out_bytes, slot, S * 4) || meet(out, out_bytes, pos, S * 4))
    return Q4_ERR_INVALID_ARG;
  ScratchLock l;
  st = scratch_acquire(0, &l);
  if (st) return st;
  if (!l.sm103) return Q4_ERR_UNSUPPORTED;
  const size_t need = paged_attn_scratch_bytes(head_dim, l.num_sms, nullptr, nullptr);
  if (need > l.ws.attn_bytes) {
    l.lock.unlock();
    st = scratch_acquire(need, &l);
    if (st) return st;
  }
  PagedAttn c{k_pages, v_pages, q, out, dtype, pages, slots, width, total, (int)heads, (int)q_heads, (int)head_dim,
              page_shift(page_size), (int)S, {q_strides[0], q_strides[1]}, scale, table, offsets, slot, pos, {},
              l.ws.status, l.num_sms};
  paged_attn_scratch_bytes(head_dim, l.num_sms, &c.ws, l.ws.attn);
  return launch_paged_attention(c, stream);
}

}  // extern "C"
