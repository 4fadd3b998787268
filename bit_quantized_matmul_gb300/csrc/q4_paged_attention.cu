// q4_paged_attention.cu — attention of a step's rows over a paged 16-bit cache,
// on the tensor cores.
//
//   o[j] = sum_{p <= pos + j} softmax_p(scale q_j . k_p) v_p,
//   position p in row p % P of page table[slot][p / P], per request and head.
//
// One launch takes single rows, drafts and chunks of prompts.  An item is a head
// of a request and a pair of tiles of its rows, as in prompt attention: the G query
// heads that share a key/value head are packed with the positions into the 128
// rows of a tile, and blocks of 128 keys are fetched once for both tiles.  A request of at most
// eight rows (positions times G) has one item a head and no tiles: see below.
//
// Shares.  The items' blocks stand in one line, request by request, and each of the launch's CTAs, one
// an SM, takes an equal piece of it, weighed by what blocks and ends of items cost, so
// that 64 decode rows and a chunk of 4,096 keep all SMs busy alike.  Each CTA finds
// its share from the step's description by itself.  An item that is cut leaves unnormalised sums
// and references in scratch (two pieces a CTA at most), and a second launch
// joins them.
//
// Roles (640 threads, registers split as in prompt attention):
//   warps 0-15  softmax of two tiles, two threads a row; warps 0-7 the light rows
//   warp 16     walks the share, and copies Q, and K and V through a ring of blocks: a page of a
//               head is one tensor-map copy (four dimensions: 64 values, eight rows, the chunks of 64
//               values, the groups of eight rows), issued by a lane each, so that a block in pages of
//               16 takes one instruction; the next piece's page numbers are on their way meanwhile
//   warps 17,18 issue the products of tile 0 / tile 1
//   warp 19     clears places of V that no row sees, sets aside infinities and NaN that
//               some rows do not see, gives back what the light rows' warps have read
// In shared memory a block of K or V is groups of eight keys, each chunk by chunk
// under the 128-byte swizzle: what one copy leaves is what products and ldmatrix read.
//
// Light rows.  With eight rows at most the tiles' products would be padding, and their
// chain of products and softmax, 1.4 us a block, as long as the copy.  So eight warps take 16 keys
// of a block each: S = K Q^T and O = V^T P^T as 16 x 8 mma.sync products with
// keys and then values along m, a running reference and sums of their own, joined in
// shared memory at the end.  Their work hides behind the copies: without it the calls below take 1.5 us less.
//
// Weights are rounded to the cache's type for the product with V: tcgen05 takes both operands in one 16-bit type, and light
// rows keep to it.  Sums of weights keep the unrounded ones.  A weight is off by 2^-8 (bf16) or 2^-11 of itself at most,
// and the error of the whole result against 64 bits is 2.1e-3 instead of the 1.7e-3 that rounding the output alone
// makes (64 rows, bf16; chunks 2.3e-3; fp16 2.9e-4 instead of 2.1e-4).  A second term for light rows' weights, of what
// the rounding took, brings them to 1.7e-3 and takes 90 us instead of 84 (64 rows), 180 instead of 160 (four chunks
// beside 60 rows).
//
// Bounds, measured in a graph (7B: 28/4 heads of 128): 8 requests of 30,001 to 32,768 positions, 91 us,
// 5.7 TB/s; 64 of 33 to 6,000, 83 us, 5.2 TB/s (HBM; without start and join about 6.2); 2,048
// rows over 14,001, 326 us, 1,353 TFLOP/s, 4,096 over 28,672, 1,170 us, 1,542 TFLOP/s (tensor cores: 1.56 us a block
// of two tiles, 1,637 TFLOP/s; the join of items that were cut, 15 us; starts and ends of pairs, 15 us).  The compiler still
// spills 24 bytes a thread at heads of 128, 32 at 64.
// One row over 2,049 positions, 0.5B, takes 11.5 us: the start 5 (three dependent loads, code that is
// not in the instruction cache), a block and its join in the CTA 3, the second launch 3.
// Joining the pieces at the end of the first launch, by the CTA that is last, was slower (its code costs the
// loops registers: 366 us instead of 326), as was one tile for light rows with its blocks in
// turn on both tiles' warps (98 us instead of 91).  What a product is told has to be made in uniform
// registers: with a place in the ring that the warp counted itself, in a loop with branches, the chunks
// took 1,300 us; it now comes with the piece.
//
// Barriers of the ring.  A warp that waits for a phase by its parity must never be two
// phases away from it.  So who does not take part in a piece's blocks (products in light ones, light rows' warps
// in others) waits, before it does again, until every role is done with the piece before.
#include "q4_tiles.cuh"
#include "q4mm_internal.h"

namespace q4 {
namespace {

constexpr int SOFTMAX_WARPS = 16;
constexpr int COPY_WARP = 16, MMA_WARP = 17, FIX_WARP = 19;  // and MMA_WARP + 1
constexpr int LIGHT_WARPS = 8;                               // warps 0-7
constexpr int WORKS = 4;                                     // pieces that the roles may be at
constexpr int THREADS = 640;
constexpr int TMEM_COLS = 512;
constexpr int LIGHT = 8;            // rows (positions times heads of a group) of a request that needs no tiles
constexpr int WARP_REQUESTS = 128;  // requests up to which one warp finds a CTA's share

// What a block of keys costs, and an item beside its blocks: of light rows, of one tile (a chain of products
// and softmax) and of two.  Only their ratios count; they were chosen by trying them on calls of each kind and mixed
// ones.  Clocks in the kernel have a block at 1.1 to 1.45 us (light rows; the more SMs copy at once, the longer), 1.3
// and 1.6 us, an end at 1.7, 2.3 and about 8 us.  Where both kinds meet (four chunks beside 60 rows) CTAs with light
// rows are done 13 us after those with tiles, of 150.
constexpr int BLOCK_LIGHT = 4, BLOCK_ONE = 5, BLOCK_TWO = 6;
constexpr int END_LIGHT = 4, END_ONE = 8, END_TWO = 16;
constexpr int SHARE_MIN = 6;  // at least a block's units, so that a share inside an item has a piece of it

template <int D>
struct Cfg {
  static constexpr int CHUNKS = D / 64;              // 128-byte column chunks of a row
  static constexpr int TILE = BM * D * 2;            // one Q tile, K block or V block
  static constexpr int Q_CHUNK = BM * 128;           // Q: chunk by chunk
  static constexpr int GROUP = CHUNKS * 1024;        // K, V: eight keys, chunk by chunk
  static constexpr int STAGES = D == 128 ? 4 : 8;    // K, V blocks in the ring (even: K and V alternate)
  static constexpr int BAR_OFF = (2 + STAGES) * TILE;
  static constexpr int SMEM = BAR_OFF + 768 + 1024;  // + alignment slack
  static constexpr int O_COL = 2 * BN;               // S0, S1, then O0, O1
};

struct Args {
  const void* v_pages;
  void* out;
  int64_t total, slots, width;
  int pages, heads, q_heads, group, positions, shift;  // positions per tile; a page is 1 << shift positions
  int S;
  int wide;  // out is 32-byte aligned
  float scale_log2;
  const int32_t *table, *offsets, *slot, *pos;
  PagedAttnScratch ws;
  unsigned* status;
  unsigned long long wait_ns;
  int stall;  // test setting: no copy is issued, so every wait for one runs out
};

struct Request {
  int qb, rows, past, slot;
};

// The launch begins under the end of the one before, which may have written what the
// call describes: after the wait by a load that the compiler cannot take for a read-only one.
__device__ __forceinline__ int32_t ld_int(const int32_t* p) {
  int32_t v;
  asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

__device__ __forceinline__ bool load_request(const Args& a, int s, Request* r) {
  const int b = ld_int(a.offsets + s), e = ld_int(a.offsets + s + 1);
  *r = Request{b, (int)((unsigned)e - (unsigned)b), ld_int(a.pos + s), ld_int(a.slot + s)};
  return b >= 0 && e >= b && e <= a.total && r->slot >= 0 && r->slot < a.slots && r->past >= 0 &&
         (int64_t)r->past + r->rows <= a.width << a.shift;
}

// The key blocks of full pairs 0 .. n - 1 of a request: pair i sees up to position
// past + (i + 1) 2 P - 1, which repeats with the period of 64 pairs (P blocks).
__host__ __device__ __forceinline__ int64_t full_blocks(int past, int positions, int n) {
  const int step = 2 * positions, q = n / 64, r = n % 64;
  int part = 0, period = 0, last = past - 1;
  const int upto = q ? 64 : r;
#pragma unroll 4
  for (int i = 0; i < upto; ++i) {
    last += step;
    period += last / BN + 1;
    if (i + 1 == r) part = period;
  }
  if (!q) return part;
  return part + (int64_t)q * period + (int64_t)positions * 64 * ((int64_t)q * (q - 1) / 2) + (int64_t)r * q * positions;
}
// Units of a block of a request, and of an item beside its blocks.
__host__ __device__ __forceinline__ int block_units(int rows, int positions, int group) {
  return rows * group <= LIGHT ? BLOCK_LIGHT : rows <= positions ? BLOCK_ONE : BLOCK_TWO;
}
__host__ __device__ __forceinline__ int end_units(int rows, int positions, int group) {
  return rows * group <= LIGHT ? END_LIGHT : rows <= positions ? END_ONE : END_TWO;
}
// Units of one head of a request.
__host__ __device__ __forceinline__ int64_t head_units(int past, int rows, int positions, int group) {
  const int step = 2 * positions, n = rows / step;
  int64_t blocks = n ? full_blocks(past, positions, n) : 0;
  if (rows % step) blocks += (past + rows - 1) / BN + 1;
  return blocks * block_units(rows, positions, group) +
         (int64_t)((rows + step - 1) / step) * end_units(rows, positions, group);
}

// All units in n equal shares.
struct Shares {
  int64_t all, each;
  int n, rest;
  __host__ __device__ __forceinline__ Shares(int64_t all, int ctas) : all(all) {
    n = all / SHARE_MIN < ctas ? (int)(all / SHARE_MIN) : ctas;
    if (n < 1) n = 1;
    if (all < (int64_t)1 << 31) {
      each = (unsigned)all / (unsigned)n;
      rest = (int)((unsigned)all % (unsigned)n);
    } else {
      each = all / n;
      rest = (int)(all % n);
    }
  }
  // the first unit of share c
  __host__ __device__ __forceinline__ int64_t begin(int c) const { return each * c + (unsigned)(rest * c) / (unsigned)n; }
  // the share that has a unit
  __host__ __device__ __forceinline__ int of(int64_t unit) const {
    int c = (int)((float)unit / (float)all * (float)n);
    c = c < 0 ? 0 : c > n - 1 ? n - 1 : c;
    while (c > 0 && begin(c) > unit) --c;
    while (c < n - 1 && begin(c + 1) <= unit) ++c;
    return c;
  }
};

// Beside a join's pieces: some piece of the share had a page number out of range.
constexpr int JOIN_WILD = 1 << 30;

// Where the table has the page of a request's last position.  It is -1 where reserve refused the request for want of
// pages: tables begin as -1, and entries past what a slot holds stay so.  The copies take -1 as any number out
// of range; such requests are looked for after them, since telling them apart any earlier costs the loops
// registers (8 requests of 32k 93 us instead of 91, four chunks 167 instead of 160).
__device__ __forceinline__ int64_t last_entry(const Args& a, const Request& r) {
  return (int64_t)r.slot * a.width + ((r.past + r.rows - 1) >> a.shift);
}

// A share's piece of an item: blocks [b0, b1) of a pair of tiles of one head.
struct Piece {
  int ok;          // 0: there is no more
  int head, pos0;  // first row of tile 0 in the request
  Request r;
  int b0, b1;
  int n;           // blocks (K and V) of the pieces before it
  int part;        // where its sums go: -1: the whole item, straight to the output
  bool last;       // the item's last
  int64_t first;   // the unit of the item's block 0
};

// What the roles derive from a piece.
struct Plan {
  bool light;        // few rows: no tiles
  int mine[2];       // the piece's blocks that each tile sees
  int nblocks;       // of the piece
  int first_hidden;  // the first position that some row of the pair does not see
  int seen_end;      // positions from here on are seen by no row of it
  int zone;          // blocks from here on hold such positions
  __device__ __forceinline__ Plan(const Args& a, const Piece& w) {
    nblocks = w.b1 - w.b0;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int p0 = w.pos0 + t * a.positions;
      const int blocks = p0 < w.r.rows ? (w.r.past + min(p0 + a.positions, w.r.rows) - 1) / BN + 1 : 0;
      mine[t] = max(0, min(blocks, w.b1) - w.b0);
    }
    light = w.r.rows * a.group <= LIGHT;
    if (light) mine[0] = mine[1] = 0;
    seen_end = w.r.past + min(w.pos0 + 2 * a.positions, w.r.rows);
    first_hidden = w.r.past + w.pos0 + 1;
    zone = first_hidden / BN;
  }
};

__device__ __forceinline__ int64_t scan64(int64_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += x;
  }
  return v;
}

// Rows that belong to no request, or to one that is out of range, are zero: the
// share of one of `threads` threads.
template <int D>
__device__ void clear_rows(const Args& a, bool bad, int64_t thread, int64_t threads) {
  const int64_t row = (int64_t)a.q_heads * D / 8;  // 16-byte vectors of a packed row
  auto clear = [&](int64_t r0, int64_t r1) {
    uint4* p = static_cast<uint4*>(a.out);
    r0 = r0 < 0 ? 0 : r0;
    r1 = r1 > a.total ? a.total : r1;
    for (int64_t i = r0 * row + thread; i < r1 * row; i += threads) p[i] = make_uint4(0u, 0u, 0u, 0u);
  };
  clear(0, ld_int(a.offsets));
  clear(ld_int(a.offsets + a.S), a.total);
  for (int s = 0; bad && s < a.S; ++s) {
    Request r;
    if (!load_request(a, s, &r)) clear(r.qb, ld_int(a.offsets + s + 1));  // its count of rows may pass 32 bits
  }
}

// Goes through the pieces of a CTA's share, run by one warp.
struct Walk {
  Request r;          // lane l: request base + l
  int base;
  int s, head, pair;  // the item it stands at
  int64_t skip;       // units of it that belong to shares before
  int64_t left, at;   // units of the share that are left; the unit it stands at
  __device__ __forceinline__ void load(const Args& a, int lane) {
    r = Request{0, 0, 0, 0};
    if (base + lane < a.S && !load_request(a, base + lane, &r)) r.rows = 0;
  }
  // at unit `rem` of request s0, which is unit u0 of all
  __device__ __forceinline__ void begin(const Args& a, int s0, int64_t rem, int64_t u0, int64_t u1, int lane) {
    base = s = s0;
    at = u0;
    left = u1 - u0;
    load(a, lane);
    const int past = __shfl_sync(0xFFFFFFFFu, r.past, 0), rows = __shfl_sync(0xFFFFFFFFu, r.rows, 0);
    const int64_t each = head_units(past, rows, a.positions, a.group);
    head = rem < (int64_t)1 << 31 && each < (int64_t)1 << 31 ? (int)((unsigned)rem / (unsigned)max((int)each, 1))
                                                             : (int)(rem / each);
    rem -= head * each;
    const int step = 2 * a.positions, pairs = (rows + step - 1) / step;
    const int block = block_units(rows, a.positions, a.group), end = end_units(rows, a.positions, a.group);
    // 32 pairs at a time
    pair = 0;
    for (int i = 0; pairs > 1 && i < pairs; i += 32) {
      const int p = i + lane;
      const int64_t u =
          p < pairs ? (int64_t)((past + (int)min((p + 1) * (int64_t)step, (int64_t)rows) - 1) / BN + 1) * block + end : 0;
      const int64_t upto = scan64(u, lane);
      const unsigned hit = __ballot_sync(0xFFFFFFFFu, rem < upto);
      if (hit) {
        const int l = __ffs(hit) - 1;
        pair = i + l;
        rem -= __shfl_sync(0xFFFFFFFFu, upto - u, l);
        break;
      }
      rem -= __shfl_sync(0xFFFFFFFFu, upto, 31);
    }
    skip = rem;
  }
  // The next piece, the same for every lane; false when there is none.
  __device__ __forceinline__ bool next(const Args& a, int cta, int lane, Piece* w) {
    const int step = 2 * a.positions;
    while (left > 0) {
      if (s - base >= 32) {
        base = s;
        load(a, lane);
      }
      if (base >= a.S) break;
      if (head == 0 && pair == 0) {  // the next request that has rows
        const unsigned rest = __ballot_sync(0xFFFFFFFFu, r.rows > 0) >> (s - base);
        if (!rest) {
          s = base + 32;
          continue;
        }
        s += __ffs(rest) - 1;
      }
      const int l = s - base;
      w->r.qb = __shfl_sync(0xFFFFFFFFu, r.qb, l);
      w->r.rows = __shfl_sync(0xFFFFFFFFu, r.rows, l);
      w->r.past = __shfl_sync(0xFFFFFFFFu, r.past, l);
      w->r.slot = __shfl_sync(0xFFFFFFFFu, r.slot, l);
      w->ok = 1;
      w->head = head;
      w->pos0 = pair * step;
      const int nb = (w->r.past + (int)min((int64_t)w->pos0 + step, (int64_t)w->r.rows) - 1) / BN + 1;
      const int block = block_units(w->r.rows, a.positions, a.group), end = end_units(w->r.rows, a.positions, a.group);
      const int64_t upto = min((int64_t)nb * block + end, skip + left);
      // a block is the share's that has its first unit
      auto blocks_before = [&](int64_t unit) {
        return unit <= end ? 0 : (int)(((unsigned)min(unit - end, (int64_t)nb * block) + block - 1) / (unsigned)block);
      };
      w->b0 = blocks_before(skip);
      w->b1 = blocks_before(upto);
      w->part = w->b0 == 0 && w->b1 == nb ? -1 : 2 * cta + (w->b0 > 0 ? 0 : 1);
      w->first = at - skip + end;
      w->last = w->b1 == nb;
      at += upto - skip;
      left -= upto - skip;
      skip = 0;
      if ((int64_t)w->pos0 + step < w->r.rows) {
        ++pair;
      } else {
        pair = 0;
        if (++head == a.heads) {
          head = 0;
          ++s;
        }
      }
      if (w->b1 > w->b0) return true;
    }
    return false;
  }
};

// The largest reference (log2) of sums that are joined, a sum being (l, reference, a
// far row's score); sums of nothing have l = 0.  Far rows have scores, whose differences keep
// their bits.  A factor is never 0, so that infinities and NaN stay.
struct Reference {
  float ref = NEG_INF, far = NEG_INF;
  __device__ __forceinline__ void take(float l, float r, float f) {
    if (l != 0.0f) {
      ref = fmaxf(ref, r);
      far = fmaxf(far, f);
    }
  }
  __device__ __forceinline__ bool is_far(float scale_log2) const { return far * scale_log2 == ref; }
  __device__ __forceinline__ float factor(float l, float r, float f, float scale_log2) const {
    if (l == 0.0f) return 0.0f;
    return fmaxf(ex2(f != NEG_INF && is_far(scale_log2) ? (f - far) * scale_log2 : r - ref), 0x1p-126f);
  }
};

// ---- small products, for light rows ----
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
template <typename T>
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                 "{%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                 "{%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D, typename T>
__global__ void __launch_bounds__(THREADS, 1)
    paged_kernel(const Args a, const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                 const __grid_constant__ CUtensorMap map_v) {
  using C = Cfg<D>;
  constexpr bool BF16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr int NST = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Piece work[WORKS];
  __shared__ PagedJoin s_join;  // the item whose last piece this share has
  __shared__ int64_t s_join_first, s_join_last;
  __shared__ int s_err, s_bad, s_first, s_nonfinite[WORKS];
  __shared__ int64_t s_rem, s_scan[THREADS / 32];
  __shared__ float s_max[2][2][BM], s_sum[2][2][BM];  // [tile][half][row]: what the halves exchange
  __shared__ uint32_t s_tmem;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);  // one value for the warp, as far as the compiler can see
  const int G = a.group, P = a.positions;

  const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem_p = smem_raw + (smem - smem_u32(smem_raw));
  const uint32_t q_smem = smem, ring = smem + 2 * C::TILE, bars = smem + C::BAR_OFF;
  const uint32_t q_full = bars, q_empty = q_full + 8, drain = q_empty + 8;
  const uint32_t full = drain + 8, empty = full + 8 * NST, hidden = empty + 8 * NST, fixed = hidden + 8 * NST;
  const uint32_t s_full = fixed + 8 * NST, p_full = s_full + 16, o_full = p_full + 32, o_empty = o_full + 16;
  const uint32_t turn = o_empty + 16, work_full = turn + 16, work_empty = work_full + 8 * WORKS;
  const uint32_t used = work_empty + 8 * WORKS, q_used = used + 8 * NST;
  volatile int* err = &s_err;
  if (tid == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 2);
    mbar_init(drain, 2);
    for (int i = 0; i < NST; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 2);
      mbar_init(hidden + 8 * i, 1);
      mbar_init(fixed + 8 * i, 1);
      mbar_init(used + 8 * i, LIGHT_WARPS);
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
    mbar_init(q_used, LIGHT_WARPS);
    mbar_arrive(turn);  // tile 0 begins
    s_err = 0;
    s_bad = 0;
    s_join = PagedJoin{0, 0, 0, 0};
    mbar_init_fence();
  }
  if (warp == MMA_WARP) tmem_alloc(smem_u32(&s_tmem), TMEM_COLS);
  if (warp == COPY_WARP && lane < 3) prefetch_map(lane == 0 ? &map_q : lane == 1 ? &map_k : &map_v);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  // ---- the CTA's share of the units: each of `threads` threads has a run of requests ----
  // Few requests are looked through by the warp that copies; the others need not wait for it.
  const bool by_warp = a.S <= WARP_REQUESTS;
  int first_s = 0;
  int64_t rem = 0, all = 0;
  if (!by_warp || warp == COPY_WARP) {
    const int threads = by_warp ? 32 : THREADS, thread = by_warp ? lane : tid;
    const int per = (a.S + threads - 1) / threads, s_begin = min(a.S, thread * per), s_end = min(a.S, s_begin + per);
    auto units_of = [&](int s, bool* bad) -> int64_t {
      Request r;
      if (load_request(a, s, &r)) return a.heads * head_units(r.past, r.rows, P, G);
      *bad = true;
      return 0;
    };
    int64_t units = 0;
    bool bad = false;
    for (int s = s_begin; s < s_end; ++s) units += units_of(s, &bad);
    const int64_t upto = scan64(units, lane);
    int64_t before = upto - units;
    if (by_warp) {
      all = __shfl_sync(0xFFFFFFFFu, upto, 31);
    } else {
      if (lane == 31) s_scan[warp] = upto;
      if (bad) s_bad = 1;
      __syncthreads();
      for (int i = 0; i < THREADS / 32; ++i) {
        if (i < warp) before += s_scan[i];
        all += s_scan[i];
      }
    }
    const Shares shares(all, (int)gridDim.x);
    const int64_t u0 = shares.begin(min((int)blockIdx.x, shares.n));
    const bool mine = u0 >= before && u0 < before + units;
    if (mine) {
      rem = u0 - before;
      first_s = s_begin;
      for (int s = s_begin; s < s_end - 1; ++s) {
        const int64_t u = units_of(s, &bad);
        if (rem < u) break;
        rem -= u;
        ++first_s;
      }
    }
    if (by_warp) {
      const int l = __ffs(__ballot_sync(0xFFFFFFFFu, mine)) - 1;
      first_s = __shfl_sync(0xFFFFFFFFu, first_s, l);
      rem = __shfl_sync(0xFFFFFFFFu, rem, l);
    } else {
      if (mine) {
        s_first = first_s;
        s_rem = rem;
      }
      __syncthreads();
      if (s_bad || ld_int(a.offsets) > 0 || ld_int(a.offsets + a.S) < a.total)
        clear_rows<D>(a, s_bad != 0, (int64_t)blockIdx.x * THREADS + tid, (int64_t)gridDim.x * THREADS);
      if (tid == 0 && s_bad && blockIdx.x == 0) atomicOr(a.status, STATUS_KV_RANGE);
      first_s = s_first;
      rem = s_rem;
    }
  }

  const uint32_t tmem = s_tmem;
  // The roles go through the same pieces in the same order, each with its own
  // count of what it has waited for.  The next piece, false when there is none.
  auto next_work = [&](int nth, Piece* w) {
    const bool ok = mbar_wait(work_full + 8 * (nth % WORKS), (nth / WORKS) & 1, err, a.wait_ns);
    if (!ok) return false;
    *w = work[nth % WORKS];
    return w->ok != 0;
  };

  if (warp >= COPY_WARP) {
    fewer_registers<64>();
    if (warp == COPY_WARP) {
      // ---------------- work and copies ----------------
      const Shares shares(all, (int)gridDim.x);
      Walk walk;
      walk.left = 0;
      if ((int)blockIdx.x < shares.n && all > 0)
        walk.begin(a, first_s, rem, shares.begin(blockIdx.x), shares.begin(blockIdx.x + 1), lane);
      int n = 0, nq = 0;  // blocks and Q pairs so far
      int nth = 0;        // pieces so far
      bool ok = true, wild = false;
      // the numbers of a piece's pages: lane l has page first + l, and the one 32 later
      struct Numbers {
        int first, id, next;
      };
      const int per_block = BN >> a.shift;
      auto number = [&](const Piece& w, int page) {
        const int last_page = (w.r.past + min(w.pos0 + 2 * P, w.r.rows) - 1) >> a.shift;
        return page <= last_page ? ld_int(a.table + (int64_t)w.r.slot * a.width + page) : 0;
      };
      auto numbers = [&](const Piece& w) {
        const int first = (w.b0 * per_block) & ~31;
        return Numbers{first, number(w, first + lane), number(w, first + 32 + lane)};
      };
      Piece w, then;
      Numbers ids{0, 0, 0}, ids_then{0, 0, 0};
      bool light_before = false, have = walk.next(a, blockIdx.x, lane, &w);
      if (have) ids = numbers(w);
      for (bool more = false; ok && have; have = more, w = then, ids = ids_then) {
        if (nth >= WORKS) {  // every role is done with the piece that had the slot
          const int v = nth - WORKS;
          ok = __all_sync(0xFFFFFFFFu, mbar_wait(work_empty + 8 * (v % WORKS), (v / WORKS) & 1, err, a.wait_ns));
        }
        if (!ok) break;
        const Plan p(a, w);
        w.n = n;
        if (lane == 0) {
          work[nth % WORKS] = w;
          s_nonfinite[nth % WORKS] = 0;
          mbar_arrive(work_full + 8 * (nth % WORKS));
        }
        if (light_before && !p.light)  // the light rows' sums lie where tile 1's rows go
          ok = __all_sync(0xFFFFFFFFu, mbar_wait(work_empty + 8 * ((nth - 1) % WORKS), ((nth - 1) / WORKS) & 1, err,
                                                 a.wait_ns));
        light_before = p.light;
        ++nth;
        if (!ok) break;
        const int last_page = (p.seen_end - 1) >> a.shift;
        if (lane == 0) {
          if (nq > 0) ok = mbar_wait(q_empty, (nq - 1) & 1, err, a.wait_ns);
          if (ok && !a.stall) {
            uint32_t bytes = 0;
            for (int t = 0; t < 2; ++t)
              if (p.mine[t] || (p.light && t == 0)) bytes += (uint32_t)(C::CHUNKS * P * G * 128);
            mbar_expect_tx(q_full, bytes);
            for (int t = 0; t < 2; ++t)
              if (p.mine[t] || (p.light && t == 0))
                for (int c = 0; c < C::CHUNKS; ++c)
                  tensor_load(q_smem + t * C::TILE + c * C::Q_CHUNK, &map_q, 64 * c, w.head * G,
                              w.r.qb + w.pos0 + t * P, q_full);
          }
        }
        ok = __shfl_sync(0xFFFFFFFFu, (int)ok, 0) != 0;
        if (ok) ++nq;
        const uint32_t page_bytes = (uint32_t)(D * 2) << a.shift;
        const int page_groups = 1 << (a.shift - 3);
        if (w.part >= 0 && w.last && lane == 0) {
          s_join = PagedJoin{0, w.r.qb + w.pos0, min(2 * P, w.r.rows - w.pos0), w.head};
          s_join_first = w.first;
          s_join_last = last_entry(a, w.r);
        }
        for (int i = w.b0; i < w.b1 && ok; ++i) {
          if (i == min(w.b0 + NST / 2, w.b1 - 1)) {  // the ring is full: the next piece, whose numbers are then on their way
            more = walk.next(a, blockIdx.x, lane, &then);
            if (more) ids_then = numbers(then);
          }
          const int pg = i * per_block, here = min(per_block, last_page - pg + 1);
          if (pg >= ids.first + 32) {
            ids.first += 32;
            ids.id = ids.next;
            ids.next = number(w, ids.first + 32 + lane);
          }
          const int page = D == 64 ? lane & 7 : lane;  // of the block
          int mine = __shfl_sync(0xFFFFFFFFu, ids.id, (pg - ids.first + page) & 31);
          if (page < here && (mine < 0 || mine >= a.pages)) {
            wild = true;
            mine = a.pages;  // past the end: the copy fills in zeros
          }
          const int at = (mine * a.heads + w.head) * page_groups;
          // K and V by one instruction, lanes 0-7 and 8-15: half this warp's time a block, which bounds D = 64 (8/8
          // heads, 8 requests of 32k in pages of 16: 124 us instead of 144; copies alone take 117).  At D = 128 the ring
          // has two blocks, and K must not wait for V's place (2,048 rows over 14,001: 467 us instead of 326).
          if constexpr (D == 64) {
            const int st = n % NST, sv = st + 1;  // n is even
            if (lane == 0) {
              if (n >= NST)
                ok = mbar_wait(empty + 8 * st, ((n / NST) - 1) & 1, err, a.wait_ns) &&
                     mbar_wait(empty + 8 * sv, ((n / NST) - 1) & 1, err, a.wait_ns);
              if (ok && !a.stall) {
                mbar_expect_tx(full + 8 * st, (uint32_t)here * page_bytes);
                mbar_expect_tx(full + 8 * sv, (uint32_t)here * page_bytes);
                if (i >= p.zone) mbar_arrive(hidden + 8 * sv);  // tells V's warp, which only waits for these
              }
            }
            ok = __shfl_sync(0xFFFFFFFFu, (int)ok, 0) != 0;
            const int kv = lane >> 3;
            if (ok && !a.stall && kv < 2 && page < here)
              tensor_load4(ring + (st + kv) * C::TILE + page * page_bytes,
                           kv ? (const void*)&map_v : (const void*)&map_k, 0, 0, 0, at, full + 8 * (st + kv));
            __syncwarp();
            if (ok) n += 2;
          } else {
            for (int kv = 0; kv < 2 && ok; ++kv) {
              const int st = n % NST;
              if (lane == 0) {
                if (n >= NST) ok = mbar_wait(empty + 8 * st, ((n / NST) - 1) & 1, err, a.wait_ns);
                if (ok && !a.stall) {
                  mbar_expect_tx(full + 8 * st, (uint32_t)here * page_bytes);
                  if (kv && i >= p.zone) mbar_arrive(hidden + 8 * st);  // tells V's warp, which only waits for these
                }
              }
              ok = __shfl_sync(0xFFFFFFFFu, (int)ok, 0) != 0;
              if (ok && !a.stall && lane < here)
                tensor_load4(ring + st * C::TILE + lane * page_bytes, kv ? (const void*)&map_v : (const void*)&map_k, 0,
                             0, 0, at, full + 8 * st);
              __syncwarp();
              if (ok) ++n;
            }
          }
        }
      }
      if (ok) {
        if (nth >= WORKS) {
          const int v = nth - WORKS;
          ok = __all_sync(0xFFFFFFFFu, mbar_wait(work_empty + 8 * (v % WORKS), (v / WORKS) & 1, err, a.wait_ns));
        }
        if (ok && lane == 0) {
          work[nth % WORKS].ok = 0;
          mbar_arrive(work_full + 8 * (nth % WORKS));
        }
      }
      wild = __any_sync(0xFFFFFFFFu, wild);  // of what kind the second launch finds out
      if (lane == 0) {
        PagedJoin join = s_join;
        if (join.rows && ld_int(a.table + s_join_last) != -1)  // a refused request's rows are cleared
          join.pieces = (int)blockIdx.x - shares.of(s_join_first) + 1;
        if (wild) join.pieces |= JOIN_WILD;
        a.ws.joins[blockIdx.x] = join;
      }
      // the copies in flight land before the CTA ends, also when another role has given up
      if (nq > 0) mbar_wait_warp(q_full, (nq - 1) & 1, a.wait_ns);
      for (int v = max(0, n - NST); v < n; ++v) mbar_wait_warp(full + 8 * (v % NST), (v / NST) & 1, a.wait_ns);
    } else if (warp == FIX_WARP) {
      // ---------------- V in masked places: safe to multiply with weights of 0 ----------------
      uint32_t seen_once = 0, used_once = 0;  // parities of each stage's `hidden` and `used`
      int nl = 0;                             // light pieces so far
      bool ok = true, tiles_before = false;
      if (by_warp) {  // rows of no request
        bool bad = false;
        for (int s = lane; s < a.S; s += 32) {
          Request r;
          bad |= !load_request(a, s, &r);
        }
        bad = __any_sync(0xFFFFFFFFu, bad);
        if (bad || ld_int(a.offsets) > 0 || ld_int(a.offsets + a.S) < a.total)
          clear_rows<D>(a, bad, (int64_t)blockIdx.x * 32 + lane, (int64_t)gridDim.x * 32);
        if (bad && lane == 0 && blockIdx.x == 0) atomicOr(a.status, STATUS_KV_RANGE);
      }
      Piece w;
      for (int nth = 0; ok; ++nth) {
        if (!__all_sync(0xFFFFFFFFu, next_work(nth, &w))) break;
        const Plan p(a, w);
        const int n = w.n;
        if (p.light && tiles_before)  // as for the light rows' warps
          ok = __all_sync(0xFFFFFFFFu, mbar_wait(work_empty + 8 * ((nth - 1) % WORKS), ((nth - 1) / WORKS) & 1, err,
                                                 a.wait_ns));
        tiles_before = !p.light;
        if (ok && p.light) {
          ok = __all_sync(0xFFFFFFFFu, mbar_wait(q_used, nl++ & 1, err, a.wait_ns));
          if (ok && lane == 0) mbar_arrive_n(q_empty, 2);
        }
        // of light rows, gives back what their warps have read
        auto give_back = [&](int v) {
          const int st = v % NST;
          ok = __all_sync(0xFFFFFFFFu, ok && mbar_wait(full + 8 * st, (v / NST) & 1, err, a.wait_ns) &&
                                           mbar_wait(used + 8 * st, (used_once >> st) & 1, err, a.wait_ns));
          used_once ^= 1u << st;
          if (ok && lane == 0) mbar_arrive_n(empty + 8 * st, 2);
        };
        for (int i = p.light ? w.b0 : max(p.zone, w.b0); ok && i < w.b1; ++i) {
          const int v = n + 2 * (i - w.b0) + 1, st = v % NST;
          if (p.light) {
            give_back(v - 1);
            if (i < p.zone) {
              give_back(v);
              continue;
            }
          }
          if (!ok) break;
          ok = __all_sync(0xFFFFFFFFu, mbar_wait(hidden + 8 * st, (seen_once >> st) & 1, err, a.wait_ns) &&
                                           mbar_wait(full + 8 * st, (v / NST) & 1, err, a.wait_ns));
          seen_once ^= 1u << st;
          if (!ok) break;
          // rows [r0, end) some rows see, those after it none
          const int r0 = max(0, p.first_hidden - i * BN), end = min(BN, p.seen_end - i * BN);
          uint8_t* vb = smem_p + (ring - smem) + st * C::TILE;
          constexpr int VPR = C::CHUNKS * 8;  // 16-byte vectors per row
          auto at = [&](int row, int e) {
            return reinterpret_cast<uint4*>(vb + (row >> 3) * C::GROUP + (e >> 3) * 1024 + (row & 7) * 128 +
                                            ((e & 7) ^ (row & 7)) * 16);
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
          // (light rows' warps take keys by 16, products whole blocks)
          const int stop = p.light ? (end + 15) & ~15 : BN;
          for (int row = max(r0, end) + lane / VPR; row < stop; row += 32 / VPR) *at(row, e) = make_uint4(0u, 0u, 0u, 0u);
          if (found) atomicExch(&s_nonfinite[nth % WORKS], 1);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(fixed + 8 * st);
          if (p.light) give_back(v);
        }
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(work_empty + 8 * (nth % WORKS));
      }
    } else {
      // ---------------- products of a tile ----------------
      // The whole warp runs the loop and one lane issues, so that what a product is
      // told is made in uniform registers.
      const int t = warp - MMA_WARP;
      constexpr uint32_t ID_S = idesc_f16(BF16, BN, false), ID_O = idesc_f16(BF16, D, true);
      constexpr uint32_t TILE16 = C::TILE / 16, Q_CHUNK16 = C::Q_CHUNK / 16, GROUP16 = C::GROUP / 16;
      const uint64_t q_desc = desc_sw128(q_smem, 16, 1024) + t * TILE16;
      const uint64_t k_desc = desc_sw128(ring, 16, C::GROUP), v_desc = desc_sw128(ring, 1024, C::GROUP);
      const uint32_t s_col = tmem + t * BN, o_col = tmem + C::O_COL + t * D;
      const bool one = lane == 0;
      int np = 0, no = 0, nt = 0;                 // weights taken, outputs begun and turns so far
      uint32_t fixed_once = 0;                    // parity of each stage's `fixed`
      bool light_before = false;                  // the piece before had no tiles
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
            mma_ss(s_col, q_desc + ((k >> 2) * Q_CHUNK16 + (k & 3) * 2), kd + ((k >> 2) * 64 + (k & 3) * 2), ID_S,
                   k > 0);
          mma_commit(s_full + 8 * t);
          mma_commit(empty + 8 * st);
        }
      };
      auto pv = [&](int st, int h, bool first) {  // O_t += P_t V, a half of the keys
        const uint64_t v = v_desc + (st * TILE16 + h * (BN / 2 / 8) * GROUP16);
        const uint32_t p = s_col + h * (BN / 2), more = first ? 0 : 1;
        if (one) {
          mma_ts(o_col, p, v, ID_O, more);
#pragma unroll
          for (int k = 1; k < BN / 32; ++k) mma_ts(o_col, p + k * 8, v + k * 2 * GROUP16, ID_O, 1);
        }
      };
      bool ok = true;
      Piece w;
      for (int nth = 0;; ++nth) {
        if (!__all_sync(0xFFFFFFFFu, ok && next_work(nth, &w))) break;
        w.pos0 = __shfl_sync(0xFFFFFFFFu, w.pos0, 0);
        w.r.rows = __shfl_sync(0xFFFFFFFFu, w.r.rows, 0);
        w.r.past = __shfl_sync(0xFFFFFFFFu, w.r.past, 0);
        w.b0 = __shfl_sync(0xFFFFFFFFu, w.b0, 0);
        w.b1 = __shfl_sync(0xFFFFFFFFu, w.b1, 0);
        int n = __shfl_sync(0xFFFFFFFFu, w.n, 0);  // blocks so far
        const Plan p(a, w);
        const int blocks = t ? p.mine[1] : p.mine[0];
        if (p.light) {
          for (int i = max(p.zone, w.b0); i < w.b1; ++i) fixed_once ^= 1u << ((n + 2 * (i - w.b0) + 1) % NST);
          give(work_empty + 8 * (nth % WORKS));
          light_before = true;
          continue;
        }
        if (light_before) {  // its copies have all been taken up: no barrier is two phases from where this warp believes it
          ok = wait(work_empty + 8 * ((nth - 1) % WORKS), ((nth - 1) / WORKS) & 1);
          light_before = false;
        }
        ok = ok && wait(q_full, nth & 1) && loaded(n);
        if (!ok) break;
        tc_fence_after();
        if (blocks > 0) qk(n % NST);
        else give(empty + 8 * (n % NST));
        if (blocks <= 1 && one) mma_commit(q_empty);
        // blocks that only the other tile has are waited for and given back
        for (int i = 0; i < p.nblocks; ++i, n += 2) {
          const int sv = (n + 1) % NST, sk = (n + 2) % NST;
          ok = loaded(n + 1) && (i + 1 >= p.nblocks || loaded(n + 2));
          if (ok && w.b0 + i >= p.zone) {
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
    // barriers; the vote at the next piece's beginning ends both halves together.
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
    // What the loop over a piece's blocks needs of it, and no more: registers for the whole of it spill by more still.
    struct View {
      int blocks;        // that the tile sees
      int seen, clear;   // the last column of its first block that the row sees; that all of the warp's live rows see
      bool live, any_live;
    };
    auto view = [&](const Piece& w) {
      const Plan p(a, w);
      const int tile_pos = w.pos0 + t * P, c0 = w.b0 * BN + h * HN;
      View v;
      v.blocks = t ? p.mine[1] : p.mine[0];
      v.live = r < P * G && tile_pos + row_pos < w.r.rows;
      v.any_live = __any_sync(0xFFFFFFFFu, v.live);  // the other warps' rows are padding
      v.seen = (v.live ? w.r.past + tile_pos + row_pos : -1) - c0;
      v.clear = w.r.past + min(tile_pos + first_pos, w.r.rows - 1) - c0;
      return v;
    };
    // What was set aside of V: positions of a piece that the row sees, N columns from col.
    auto set_aside = [&](const Piece& w, int first_hidden, int lim, int col, float* x, int N) {
      const int j1 = min(lim, w.b1 * BN - 1);
      for (int j = max(first_hidden, w.b0 * BN); j <= j1; ++j) {
        const int id = ld_int(a.table + (int64_t)w.r.slot * a.width + (j >> a.shift));
        if (id < 0 || id >= a.pages) continue;
        const T* v = static_cast<const T*>(a.v_pages) +
                     ((((int64_t)id * a.heads + w.head) << a.shift) + (j & ((1 << a.shift) - 1))) * D + col;
        for (int e = 0; e < N; ++e) {
          const float f = (float)v[e];
          if (!isfinite(f)) x[e] += f;
        }
      }
    };
    // Light rows (at most eight), on warps 0-7.  Each has 16 keys of every block, and sums of its own over
    // them: S = K Q^T and O = V^T P^T in 16 x 8 products, keys and then values along their 16 rows.
    uint32_t fixed_once = 0;  // parity of each stage's `fixed`
    auto light_piece = [&](const Piece& w, const Plan& p, int nth) {
      const int g = lane >> 2, tq = lane & 3;
      ok = __all_sync(0xFFFFFFFFu, ok && mbar_wait(q_full, nth & 1, err, a.wait_ns));
      uint32_t q[D / 32][4];  // fragments of Q, 32 values each
#pragma unroll
      for (int k = 0; k < D / 32; ++k) {
        const int vec = 4 * k + (lane >> 3);
        ldsm4(q_smem + (vec >> 3) * C::Q_CHUNK + (lane & 7) * 128 + (((vec & 7) ^ (lane & 7)) << 4), q[k]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(q_used);
      // rows 2 tq and 2 tq + 1: last position seen, reference (a score), the lane's share of the sum
      const int live_rows = w.r.rows * G;
      const int lim0 = 2 * tq < live_rows ? w.r.past + 2 * tq / G : -1;
      const int lim1 = 2 * tq + 1 < live_rows ? w.r.past + (2 * tq + 1) / G : -1;
      float ref0 = NEG_INF, ref1 = NEG_INF, l0 = 0.0f, l1 = 0.0f, o[D / 16][4] = {};
      const uint32_t k_at = (2 * warp + ((lane >> 3) & 1)) * C::GROUP + (lane & 7) * 128;
      const uint32_t v_at = (2 * warp + (lane >> 4)) * C::GROUP + (lane & 7) * 128;
      int n = w.n;
      for (int i = w.b0; i < w.b1; ++i, n += 2) {
        const int sk = n % NST, sv = (n + 1) % NST, key = i * BN + warp * 16 + g;
        const bool some = i * BN + warp * 16 < p.seen_end;  // of the warp's keys
        ok = __all_sync(0xFFFFFFFFu, ok && mbar_wait(full + 8 * sk, (n / NST) & 1, err, a.wait_ns));
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (ok && some) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const int vec = 2 * k + (lane >> 4);
            uint32_t x[4];
            ldsm4(ring + sk * C::TILE + k_at + (vec >> 3) * 1024 + (((vec & 7) ^ (lane & 7)) << 4), x);
            mma16<T>(s, x, q[k / 2][(k & 1) * 2], q[k / 2][(k & 1) * 2 + 1]);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(used + 8 * sk);
        uint32_t p0 = 0, p1 = 0;
        if (ok && some) {
          if (key > lim0) s[0] = NEG_INF;
          if (key > lim1) s[1] = NEG_INF;
          if (key + 8 > lim0) s[2] = NEG_INF;
          if (key + 8 > lim1) s[3] = NEG_INF;
          float m0 = fmaxf(s[0], s[2]), m1 = fmaxf(s[1], s[3]);
#pragma unroll
          for (int d = 4; d < 32; d *= 2) {
            m0 = fmaxf(m0, __shfl_xor_sync(0xFFFFFFFFu, m0, d));
            m1 = fmaxf(m1, __shfl_xor_sync(0xFFFFFFFFu, m1, d));
          }
          // a first score, or one that passes the reference by more than 2^GROW
          const bool more0 = m0 > ref0 && !((m0 - ref0) * a.scale_log2 <= GROW);
          const bool more1 = m1 > ref1 && !((m1 - ref1) * a.scale_log2 <= GROW);
          if (__any_sync(0xFFFFFFFFu, more0 || more1)) {
            const float f0 = more0 ? ex2((ref0 - m0) * a.scale_log2) : 1.0f;
            const float f1 = more1 ? ex2((ref1 - m1) * a.scale_log2) : 1.0f;
            ref0 = more0 ? m0 : ref0;
            ref1 = more1 ? m1 : ref1;
            l0 *= f0;
            l1 *= f1;
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
              o[d][0] *= f0;
              o[d][1] *= f1;
              o[d][2] *= f0;
              o[d][3] *= f1;
            }
          }
          // differences of scores keep their bits, however far from zero the scores are
          const float r0 = ref0 == NEG_INF ? 0.0f : ref0, r1 = ref1 == NEG_INF ? 0.0f : ref1;
          const float w0 = ex2(fmaf(s[0] - r0, a.scale_log2, LIFT<T>)), w1 = ex2(fmaf(s[1] - r1, a.scale_log2, LIFT<T>));
          const float w2 = ex2(fmaf(s[2] - r0, a.scale_log2, LIFT<T>)), w3 = ex2(fmaf(s[3] - r1, a.scale_log2, LIFT<T>));
          l0 += w0 + w2;
          l1 += w1 + w3;
          p0 = transpose8(pack2<T>(w0, w1));
          p1 = transpose8(pack2<T>(w2, w3));
        }
        ok = __all_sync(0xFFFFFFFFu, ok && mbar_wait(full + 8 * sv, ((n + 1) / NST) & 1, err, a.wait_ns));
        if (i >= p.zone) {
          ok = __all_sync(0xFFFFFFFFu, ok && mbar_wait(fixed + 8 * sv, (fixed_once >> sv) & 1, err, a.wait_ns));
          fixed_once ^= 1u << sv;
        }
        if (ok && some) {
#pragma unroll
          for (int d = 0; d < D / 16; ++d) {
            const int vec = 2 * d + ((lane >> 3) & 1);
            uint32_t x[4];
            ldsm4_t(ring + sv * C::TILE + v_at + (vec >> 3) * 1024 + (((vec & 7) ^ (lane & 7)) << 4), x);
            mma16<T>(o[d], x, p0, p1);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(used + 8 * sv);
      }
      // the warps' sums, joined through the place of tile 1's rows
#pragma unroll
      for (int d = 4; d < 32; d *= 2) {
        l0 += __shfl_xor_sync(0xFFFFFFFFu, l0, d);
        l1 += __shfl_xor_sync(0xFFFFFFFFu, l1, d);
      }
      tile_sync(0);
      // [warp][8 rows][D], columns turned so that banks differ
      float* const sums = reinterpret_cast<float*>(smem_p + C::TILE);
#pragma unroll
      for (int d = 0; d < D / 16; ++d) {
        float* row = sums + (warp * 8 + 2 * tq) * D;
        row[(d * 16 + g) ^ (tq * 8)] = o[d][0];
        row[D + ((d * 16 + g) ^ (tq * 8))] = o[d][1];
        row[(d * 16 + g + 8) ^ (tq * 8)] = o[d][2];
        row[D + ((d * 16 + g + 8) ^ (tq * 8))] = o[d][3];
      }
      if (g == 0) {
        s_max[0][0][warp * 8 + 2 * tq] = ref0;
        s_max[0][0][warp * 8 + 2 * tq + 1] = ref1;
        s_sum[0][0][warp * 8 + 2 * tq] = l0;
        s_sum[0][0][warp * 8 + 2 * tq + 1] = l1;
      }
      tile_sync(0);
      const int row = tid / (D / 4), col = tid % (D / 4) * 4;
      if (ok && row < live_rows) {
        Reference top;
#pragma unroll
        for (int i = 0; i < LIGHT_WARPS; ++i) {
          const float ref = s_max[0][0][i * 8 + row];
          top.take(s_sum[0][0][i * 8 + row], ref * a.scale_log2, ref);
        }
        float l = 0.0f, x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < LIGHT_WARPS; ++i) {
          const float ref = s_max[0][0][i * 8 + row], li = s_sum[0][0][i * 8 + row];
          const float f = top.factor(li, ref * a.scale_log2, ref, a.scale_log2);
          if (f == 0.0f) continue;
          l += f * li;
          const float4 y = *reinterpret_cast<const float4*>(sums + (i * 8 + row) * D + (col ^ (((row >> 1) & 3) * 8)));
          x[0] += f * y.x;
          x[1] += f * y.y;
          x[2] += f * y.z;
          x[3] += f * y.w;
        }
        const bool whole = w.part < 0;
        const float inv = whole ? 1.0f / l : 1.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] *= inv;
        const int pos = row / G;
        if (s_nonfinite[nth % WORKS]) set_aside(w, p.first_hidden, w.r.past + pos, col, x, 4);
        if (whole) {
          T* dst = static_cast<T*>(a.out) + ((int64_t)(w.r.qb + pos) * a.q_heads + w.head * G + row % G) * D + col;
          *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]));
        } else {
          const int64_t place = (int64_t)w.part * 2 * BM + row;
          *reinterpret_cast<float4*>(a.ws.partial + place * D + col) = make_float4(x[0], x[1], x[2], x[3]);
          if (col == 0) a.ws.ml[place] = make_float4(l, top.ref, top.far, 0.0f);
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // copies come there again
    };
    bool tiles_before = false;  // the piece before had tiles
    for (int nth = 0;; ++nth) {
      View u;
      {
        Piece w;
        ok = ok && next_work(nth, &w);
        if (tile_vote(t, !ok)) break;
        const Plan p(a, w);
        if (p.light) {
          if (t == 0) {
            // Its copies have all been taken up: no barrier is two phases from where these warps believe it to be.
            if (tiles_before)
              ok = __all_sync(0xFFFFFFFFu, ok && mbar_wait(work_empty + 8 * ((nth - 1) % WORKS), ((nth - 1) / WORKS) & 1,
                                                           err, a.wait_ns));
            light_piece(w, p, nth);
          }
          tiles_before = false;
          __syncwarp();
          if (ok && lane == 0) mbar_arrive(work_empty + 8 * (nth % WORKS));
          continue;
        }
        tiles_before = true;
        for (int i = max(p.zone, w.b0); i < w.b1; ++i) fixed_once ^= 1u << ((w.n + 2 * (i - w.b0) + 1) % NST);
        u = view(w);
      }
      const bool live = u.live;
      // The reference, in units of log2, scaled and less LIFT (-LIFT in far rows, 0 before the first score); the
      // scaled score that calls for another (-inf: any does); a far row's reference.
      float m = 0.0f, most = NEG_INF, l = 0.0f, far_ref = NEG_INF;
      for (int i = 0; i < u.blocks; ++i, ++ns, u.seen -= BN, u.clear -= BN) {
        ok = __all_sync(0xFFFFFFFFu, ok && mbar_wait(s_full + 8 * t, ns & 1, err, a.wait_ns));
        const bool masked = HN - 1 > u.clear, use = ok && u.any_live;
        // 32 scores, again from tensor memory for the weights: there are no registers for all 64
        auto scores = [&](int c, uint32_t (&s)[32]) {
          tmem_ld32<0>(s_addr + c, s);
          tmem_wait_ld();
          if (masked) {
#pragma unroll
            for (int e = 0; e < 32; ++e) s[e] = c + e <= u.seen ? s[e] : __float_as_uint(NEG_INF);
          }
        };
        float mn = NEG_INF;
        if (use) {
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
            if (use) {
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
          if (__any_sync(0xFFFFFFFFu, far) && use) {
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
        if (use) {
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
        }
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(p_full + 16 * t + 8 * h);
      }
      // ---- O / l to memory, or O, l and their reference to scratch ----
      const Piece w = work[nth % WORKS];
      const Plan p(a, w);
      const int blocks = t ? p.mine[1] : p.mine[0];
      const int pos = w.pos0 + t * P + row_pos, lim = w.r.past + pos;
      const bool whole = w.part < 0;
      const int64_t place = ((int64_t)(whole ? 0 : w.part) * 2 + t) * BM + r;
      T* const dst = static_cast<T*>(a.out) + ((int64_t)(w.r.qb + pos) * a.q_heads + w.head * G + row_head) * D;
      float* const part = a.ws.partial + place * D;
      auto put = [&](int col, float (&x)[16], bool extra) {  // 16 columns of the row
        if (extra) set_aside(w, p.first_hidden, lim, col, x, 16);
        if (whole) {
          uint32_t y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = pack2<T>(x[2 * e], x[2 * e + 1]);
          store16(dst + col, y, a.wide);
        } else {
#pragma unroll
          for (int e = 0; e < 16; e += 8) {
            uint32_t y[8];
#pragma unroll
            for (int f = 0; f < 8; ++f) y[f] = __float_as_uint(x[e + f]);
            store16(part + col + e, y, true);
          }
        }
      };
      const float ref =
          far_ref != NEG_INF ? far_ref * a.scale_log2 : most == NEG_INF ? NEG_INF : m + LIFT<T>;
      if (blocks == 0) {
        if (!whole && live && h == 0) a.ws.ml[place] = make_float4(0.0f, NEG_INF, NEG_INF, 0.0f);
      } else {
        s_sum[t][h][r] = l;
        tile_sync(t);
        l += s_sum[t][1 - h][r];
        ok = __all_sync(0xFFFFFFFFu, ok && mbar_wait(o_full + 8 * t, no & 1, err, a.wait_ns));
        ++no;
        if (ok) {
          tc_fence_after();
          const float inv = whole ? 1.0f / l : 1.0f;
          const bool extra = s_nonfinite[nth % WORKS] != 0;
          if (live && !whole && h == 0) a.ws.ml[place] = make_float4(l, ref, far_ref, 0.0f);
#pragma unroll 1
          for (int c = 0; c < HD; c += 32) {
            uint32_t o[32];
            tmem_ld32<0>(o_addr + c, o);
            tmem_wait_ld();
            if (c + 32 == HD) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(o_empty + 8 * t);
            }
            if (live) {
#pragma unroll
              for (int d = 0; d < 32; d += 16) {
                float x[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) x[e] = __uint_as_float(o[d + e]) * inv;
                put(h * HD + c + d, x, extra);
              }
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

// ---- the pieces of items that were cut, joined ----
//   out = sum_k f_k O_k / sum_k f_k l_k,  f_k = 2^(reference_k - largest reference)
// A warp a row, whose references lie in its lanes, 32 pieces at a time.  Bound by latency: the
// first pieces' sums are loaded beside the references.  One row of 17 pieces takes 3 us, 76 items of
// two tiles 15 (39 MB of sums; two or four rows a warp at once took 1 to 10 us more, as did
// factors that every lane makes for itself, all for fewer warps on an SM).
constexpr int JOIN_WARPS = 8, JOIN_CTAS = 8;  // CTAs for each share

// For a share that met a page number out of range: the rows of requests that reserve refused become zeros, whatever the
// first launch made of the pages that they have (the share that has a request's last position meets its -1),
// and the status says what there was.  A warp a request; shares that come here together write the same.
template <int D>
__device__ __noinline__ void find_wild(const Args& a, int warp, int lane) {
  const int64_t row = (int64_t)a.q_heads * D / 8;  // 16-byte vectors of a packed row
  for (int s = warp; s < a.S; s += JOIN_CTAS * JOIN_WARPS) {
    Request r;
    if (!load_request(a, s, &r) || r.rows == 0) continue;
    if (ld_int(a.table + last_entry(a, r)) == -1) {
      uint4* p = static_cast<uint4*>(a.out) + r.qb * row;
      for (int64_t i = lane; i < r.rows * row; i += 32) p[i] = make_uint4(0u, 0u, 0u, 0u);
      if (lane == 0) atomicOr(a.status, STATUS_PAGES);
      continue;
    }
    bool wild = false;
    for (int64_t i = (int64_t)r.slot * a.width + lane; i <= last_entry(a, r); i += 32) {
      const int id = ld_int(a.table + i);
      wild |= id < 0 || id >= a.pages;
    }
    if (__any_sync(0xFFFFFFFFu, wild) && lane == 0) atomicOr(a.status, STATUS_KV_RANGE);
  }
}

template <int D, typename T>
__global__ void __launch_bounds__(32 * JOIN_WARPS) paged_join_kernel(const Args a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int4 d = __ldcg(reinterpret_cast<const int4*>(a.ws.joins + blockIdx.x));
  const PagedJoin j{d.x & ~JOIN_WILD, d.y, d.z, d.w};
  const int lane = threadIdx.x & 31, G = a.group, P = a.positions;
  if (d.x & JOIN_WILD) find_wild<D>(a, blockIdx.y * JOIN_WARPS + (threadIdx.x >> 5), lane);
  const int rows = j.pieces ? j.rows * G : 0, c0 = (int)blockIdx.x - j.pieces + 1;
  constexpr int V = D / 32, EARLY = 4;  // values of a lane; pieces loaded early
  for (int i = blockIdx.y * JOIN_WARPS + (threadIdx.x >> 5); i < rows; i += JOIN_CTAS * JOIN_WARPS) {
    // row i of the item: position i / G, in tile 0 or 1
    const int pos = i / G, head = i - pos * G, t = pos >= P ? 1 : 0;
    const int64_t base = (int64_t)(4 * c0 + t) * BM + (pos - t * P) * G + head;
    auto place = [&](int k) { return base + (4 * k + (k == 0 ? 2 : 0)) * BM; };  // piece k: the first is its share's last
    auto load = [&](float (&x)[V], int k) {
      const float* p = a.ws.partial + place(k) * D + lane * V;
      if constexpr (V == 4) {
        const float4 y = __ldcg(reinterpret_cast<const float4*>(p));
        x[0] = y.x, x[1] = y.y, x[2] = y.z, x[3] = y.w;
      } else {
        const float2 y = __ldcg(reinterpret_cast<const float2*>(p));
        x[0] = y.x, x[1] = y.y;
      }
    };
    float l = 0.0f, o[V] = {};
    auto add = [&](float f, float lk, const float (&x)[V]) {
      l += f * lk;
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] += f == 0.0f ? 0.0f : f * x[e];  // pieces of nothing have not been written
    };
    auto references = [&](int k) { return k < j.pieces ? __ldcg(a.ws.ml + place(k)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f); };
    float4 ml = references(lane);
    float early[EARLY][V];
#pragma unroll
    for (int k = 0; k < EARLY; ++k)
      if (k < j.pieces) load(early[k], k);
    Reference top;
    top.take(ml.x, ml.y, ml.z);
    for (int k = lane + 32; k < j.pieces; k += 32) {
      const float4 x = references(k);
      top.take(x.x, x.y, x.z);
    }
#pragma unroll
    for (int n = 16; n; n >>= 1) {
      top.ref = fmaxf(top.ref, __shfl_xor_sync(0xFFFFFFFFu, top.ref, n));
      top.far = fmaxf(top.far, __shfl_xor_sync(0xFFFFFFFFu, top.far, n));
    }
    for (int k0 = 0; k0 < j.pieces; k0 += 32) {
      if (k0 > 0) ml = references(k0 + lane);
      const float lk = ml.x, f = top.factor(lk, ml.y, ml.z, a.scale_log2);
      const int n = min(32, j.pieces - k0);
      int k = 0;
      if (k0 == 0) {
#pragma unroll
        for (int e = 0; e < EARLY; ++e) {
          const float fk = __shfl_sync(0xFFFFFFFFu, f, e), lkk = __shfl_sync(0xFFFFFFFFu, lk, e);
          if (e < n) add(fk, lkk, early[e]);
        }
        k = EARLY;
      }
#pragma unroll 4
      for (; k < n; ++k) {
        float x[V];
        load(x, k0 + k);
        add(__shfl_sync(0xFFFFFFFFu, f, k), __shfl_sync(0xFFFFFFFFu, lk, k), x);
      }
    }
    const float inv = 1.0f / l;
    T* dst = static_cast<T*>(a.out) + ((int64_t)(j.row + pos) * a.q_heads + j.head * G + head) * D + lane * V;
    if constexpr (V == 4)
      *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<T>(o[0] * inv, o[1] * inv), pack2<T>(o[2] * inv, o[3] * inv));
    else
      *reinterpret_cast<uint32_t*>(dst) = pack2<T>(o[0] * inv, o[1] * inv);
  }
}

// ---------------------------------------------------------------- host

// Map of the pages of K or V: eight rows, chunks of a row, groups of eight rows; a box is a page of one head.
bool make_pages_map(CUtensorMap* map, bool bf16, const void* p, int64_t groups, int D, int page) {
  const EncodeFn encode = encode_fn();
  if (!encode) return false;
  const cuuint64_t dims[4] = {64, 8, (cuuint64_t)(D / 64), (cuuint64_t)groups};
  const cuuint64_t strides[3] = {(cuuint64_t)D * 2, 128, (cuuint64_t)D * 16};
  const cuuint32_t box[4] = {64, 8, (cuuint32_t)(D / 64), (cuuint32_t)(page / 8)};
  const cuuint32_t elem[4] = {1, 1, 1, 1};
  return encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                const_cast<void*>(p), dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, typename T>
int launch_as(const PagedAttn& c, cudaStream_t s) {
  constexpr bool BF16 = std::is_same<T, __nv_bfloat16>::value;
  Args a;
  a.v_pages = c.v_pages;
  a.out = c.out;
  a.total = c.total;
  a.slots = c.slots;
  a.width = c.width;
  a.pages = (int)c.pages;
  a.heads = c.heads;
  a.q_heads = c.q_heads;
  a.group = c.q_heads / c.heads;
  a.positions = BM / a.group;
  a.shift = c.shift;
  a.S = c.S;
  a.wide = (reinterpret_cast<uintptr_t>(c.out) & 31u) == 0;
  a.scale_log2 = c.scale * 1.44269504088896340736f;
  a.table = c.table;
  a.offsets = c.offsets;
  a.slot = c.slot;
  a.pos = c.pos;
  a.ws = c.ws;
  a.status = c.status;
  a.wait_ns = wait_limit_ns();
  a.stall = stall_for_test();
  CUtensorMap mq, mk, mv;
  const int64_t groups = (c.pages * c.heads) << (c.shift - 3);
  if (!make_rows_map(&mq, BF16, c.q, c.total, c.q_heads, D, c.q_strides, a.group, a.positions) ||
      !make_pages_map(&mk, BF16, c.k_pages, groups, D, 1 << c.shift) ||
      !make_pages_map(&mv, BF16, c.v_pages, groups, D, 1 << c.shift))
    return Q4_ERR_INVALID_ARG;
  static std::atomic<bool> sized[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return Q4_ERR_CUDA;
  if (!sized[dev].load()) {
    if (cudaFuncSetAttribute(paged_kernel<D, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::SMEM) !=
        cudaSuccess)
      return Q4_ERR_CUDA;
    sized[dev].store(true);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)c.num_sms);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = Cfg<D>::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, paged_kernel<D, T>, a, mq, mk, mv) != cudaSuccess) return Q4_ERR_CUDA;
  cfg.gridDim = dim3((unsigned)c.num_sms, JOIN_CTAS);
  cfg.blockDim = dim3(32 * JOIN_WARPS);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, paged_join_kernel<D, T>, a) == cudaSuccess ? Q4_OK : Q4_ERR_CUDA;
}

}  // namespace

size_t paged_attn_scratch_bytes(int64_t head_dim, int num_sms, PagedAttnScratch* out, uint8_t* base) {
  const size_t rows = (size_t)num_sms * 2 * 2 * BM;  // two pieces a share, two tiles each
  const size_t partial = rows * head_dim * sizeof(float), ml = rows * sizeof(float4);
  if (out) {
    out->partial = reinterpret_cast<float*>(base);
    out->ml = reinterpret_cast<float4*>(base + partial);
    out->joins = reinterpret_cast<PagedJoin*>(base + partial + ml);
  }
  return partial + ml + (size_t)num_sms * sizeof(PagedJoin);
}

int launch_paged_attention(const PagedAttn& c, cudaStream_t s) {
  if (c.dtype == Q4_DTYPE_F16)
    return c.head_dim == 128 ? launch_as<128, __half>(c, s) : launch_as<64, __half>(c, s);
  return c.head_dim == 128 ? launch_as<128, __nv_bfloat16>(c, s) : launch_as<64, __nv_bfloat16>(c, s);
}

}  // namespace q4
