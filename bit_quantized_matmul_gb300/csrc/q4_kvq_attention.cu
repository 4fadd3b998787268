// q4_kvq_attention.cu — attention of a step's query rows over the 4-bit cache.
//
//   o[r] = sum_p w[r,p] v[p],  w[r,p] = exp(s[r,p]) / sum_p' exp(s[r,p']),
//   s[r,p] = scale * q[r] . k[p],  p = 0 .. pos + j for row j of a request,
//
// for every (row, query head) r; the G query heads of a key/value head share
// its cache rows.  One pass over the cache with a running maximum and sum per
// row; the cache is read once per eight virtual rows (row j, head h of the
// group: j*G + h), which is once for a decode row of up to eight heads a group.
//
// Accuracy.  Codes are exact in binary16 and the other operand x is a pair of
// binary16 terms, x = hi + lo, so products carry the accuracy of fp32.
//
// Scores.  A nibble masked in place is the binary16 number q * 2^-24 (low
// nibble of a byte) or 16 q * 2^-24 (high nibble), a subnormal that the tensor
// core takes as it is: five integer instructions give four operand registers.
// The factor 16 is taken out of the query fragment, and the offset -8 enters
// as -8 sum(x), added to each block's sum.  The tensor core aligns
// products by their operands' exponents, of which a subnormal has the
// largest that it can have, and drops what lies below: the query's hi terms
// are therefore integers (the row scaled to |x| <= 2048), of whose sums
// nothing is dropped, and lo is the rest.  One m16n8k16 product takes the hi
// terms of eight virtual rows in its rows 0-7 and their lo terms in rows 8-15,
// and a thread holds both.  K's scales multiply each block's partial score.
//
// Output.  Weights differ by many binades within a row, so here hi is x
// rounded to binary16 and the codes are made q - 8 exactly (one more
// instruction a register, none for the offset).  V's scales are folded into the
// weights of their block, x = w d: with w = wh + wl split once for all blocks,
// hi = wh d rounded, and lo = (wh d - hi) + wl d, whose first part a fused
// multiply-add gives exactly: three instructions for two weights.  Weights and V's
// scales are taken times powers of two (the weights 2^9, the scales so that the
// largest so far is about 1), so that they and x fit binary16 and lo keeps its
// bits.  A scale's costs one more instruction for two: 64 ragged requests called in
// turn take 38.0 us with it, 37.0 without, 8 at 32k 43.3 and 43.1.  Lo ends at 2^-24
// all the same: next to a key of weight 1 the others are held to 2^-29 of V's largest
// scale each, so of a weight 2^-b about 33 - b bits count.  Values lie along m and
// virtual rows along n, and hi and lo go into one accumulator.  Rows of 16 bits get
// the lo terms too: without them sums that nearly cancel keep errors of 2^-12 of their
// terms, more than their own rounding (8 bf16 requests at 32k would take 38.1 us
// instead of 42.4, in one graph over the same inputs).
//
// Work.  A unit is one cache tile (32 positions) of one item (request, head,
// eight virtual rows).  The launch's warps take equal, contiguous ranges of
// units whatever the lengths are (each CTA sums the lengths itself, so the
// host needs none of them), each through its own ring of bulk copies; after
// the plan no warp waits for another.  Items cut between warps leave
// (reference score, sum, o) in scratch and a second launch joins them.
//
// Launches.  Each begins under the end of the one before and waits for it on the device.
// One that let others begin before its own wait was done would let them begin while
// a kernel two places back still ran, and their waits are for the launch before them
// only: so the first launch lets the join begin after its wait, and what the join and the
// weights' launch read before theirs is older than the call.  Nothing comes by the
// read-only path, which is for memory that no kernel writes meanwhile.  The early
// beginning of the first launch is worth 0.8 us of a call that follows another
// (64 ragged requests called in turn 38.9 us without, 38.1 with; 32 with weights,
// behind the copy of theirs, 53.2 and 50.2).
//
// Measured (28/4 heads of 128; both launches in a graph, inputs past the L2): 64
// fp32 rows over 176,432 positions 37.4 us (103 MB: 2.8 TB/s), 8 bf16 rows over
// 254,706 44.2 us (147 MB: 3.3 TB/s).  The copies alone take 23 and 31 us.  What is
// left is the arithmetic of 4-bit operands on warp-wide products: 395 warp
// instructions for 16 positions (fp32 rows), with which issue slots are 52% busy, the
// ALU 41%, the products 33%; three CTAs per SM (168 registers) hide no more of
// their latency, and four (128 registers) were slower.  44 draft rows of 16
// requests (five row groups a head, each unpacks the cache for itself) take 23.6 us,
// one row over 2,049 positions of 2 heads of 64 7.9 us, all of it launches and the
// latency of one short chain.
#include <atomic>

#include "q4_kvq.cuh"
#include "q4_ptx.cuh"

namespace q4 {
namespace {

constexpr int WARPS = 4;
constexpr int THREADS = 32 * WARPS;
constexpr int ROWS = 8;               // virtual rows of an item
constexpr int CTAS_PER_SM = 3;
constexpr int STAGES = 3;             // tiles in flight per warp
constexpr int JOIN_WARPS = 8;
constexpr int MASS_STAGES = 4;        // K halves in flight per warp of the weights' launch
constexpr int MASS_CTAS_PER_SM = 4;
constexpr int ITEM_UNITS = 2;         // what beginning an item costs, in tiles: its queries, its sums' end
constexpr float NEG_INF = -INFINITY;
constexpr float SLACK = 5.0f;         // log2 of how far a weight may pass 1 before the sums are rescaled
// References of this size (in units of log2) and above have steps that a power of two added to them
// would be lost in: their rows' weights are taken as they are, and the reference has no slack.
constexpr float FAR = 0x1p16f;

template <typename T>
struct Args {
  const uint8_t* cache;
  const T* q;
  int64_t q_token, q_head;  // strides in elements
  T* out;                   // [total, q_heads, D]
  float scale_log2;         // scale * log2(e)
  int64_t slots, capacity, plane_bytes, total;
  int heads, group, S;
  const int32_t *offsets, *slot, *pos;
  unsigned* status;
  unsigned long long wait_ns;
  int stall;                // test setting: no copy is issued, so every wait runs out
  float* partial;           // [2 * workers][ROWS][D]
  float2* partial_ml;       // [2 * workers][ROWS] (reference score, sum)
  int64_t* unit_start;      // [S + 1]
  int workers;              // warps of the main launch
  float2* lse;              // [total, q_heads] a row's reference and the log2 of its sum of exponentials, or null
  float* mass;              // [slots, heads, capacity], or null
};

// D = A B + C, m16n8k16, binary16 operands, fp32 sums
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1,
                                    const float (&c)[4]) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

__device__ __forceinline__ F2 half2_f2(uint32_t w) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  return f2(f.x, f.y);
}

__device__ __forceinline__ uint32_t pack(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// hi and lo terms of two values
__device__ __forceinline__ void split(F2 x, __half2& hi, __half2& lo) {
  const float2 v = unf2(x);
  hi = __floats2half2_rn(v.x, v.y);
  const float2 h = __half22float2(hi);
  const float2 l = unf2(fma2(f2(h.x, h.y), f2(-1.0f, -1.0f), x));
  lo = __floats2half2_rn(l.x, l.y);
}
__device__ __forceinline__ uint32_t bits(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }
__device__ __forceinline__ __half2 half2_of(uint32_t w) { return *reinterpret_cast<const __half2*>(&w); }

// The operand registers of a word of codes: nibbles (0, 4), 16 * (1, 5),
// (2, 6) and 16 * (3, 7) as binary16 pairs scaled by 2^-24.
__device__ __forceinline__ void unpack(uint32_t w, uint32_t (&r)[4]) {
  r[0] = w & 0x000F000Fu;
  r[1] = w & 0x00F000F0u;
  r[2] = (w >> 8) & 0x000F000Fu;
  r[3] = (w >> 8) & 0x00F000F0u;
}

// ---------------------------------------------------------------- work ranges
struct Request {
  int b, pos, slot;
  int n, tiles, items;  // rows, cache tiles, items (heads x row groups); 0 tiles: nothing to do
  // an item counts as some units more than its tiles: the first ones stand for its beginning
  __device__ __forceinline__ int span() const { return tiles ? tiles + ITEM_UNITS : 0; }
  __device__ __forceinline__ int64_t units() const { return (int64_t)span() * items; }
};

template <typename T>
__device__ __forceinline__ Request load_request(const Args<T>& a, int s, bool by_rows, bool* bad = nullptr) {
  const KvqRequest q = kvq_request<true>(a.offsets, a.slot, a.pos, s);
  Request r{(int)q.b, (int)q.pos, (int)q.slot, 0, 0, 0};
  if (!q.ok(a.total, a.slots, a.capacity)) {
    if (bad) *bad = q.e > q.b;
    return r;
  }
  r.n = (int)(q.e - q.b);
  if (r.n == 0) return r;
  r.tiles = (r.pos + r.n + KVQ_POS - 1) / KVQ_POS;
  r.items = a.heads * (by_rows ? (r.n * a.group + ROWS - 1) / ROWS : 1);
  return r;
}

// How `all` units are shared out: the first `more` of `workers` get size + 1,
// the others size.  A worker is a warp; worker w is warp w / CTAs of CTA
// w % CTAs, so that few units spread over all SMs.
struct Shares {
  int64_t size;
  int more, workers;
  __device__ __forceinline__ Shares(int64_t all, int most) {
    workers = (int)min(all, (int64_t)most);
    if (all < (int64_t)1 << 31) {
      size = workers ? (int)all / workers : 0;
    } else {
      size = all / workers;
    }
    more = (int)(all - size * workers);
  }
  __device__ __forceinline__ int64_t start(int w) const { return w * size + min(w, more); }
  // the worker that has unit u
  __device__ __forceinline__ int of(int64_t u) const {
    const int64_t big = more * (size + 1);
    if (u < big) return big < (int64_t)1 << 31 ? (int)u / ((int)size + 1) : (int)(u / (size + 1));
    u -= big;
    return more + (u < (int64_t)1 << 31 && size < (int64_t)1 << 31 ? (int)u / (int)size : (int)(u / size));
  }
};

// A worker's range of units.
struct Range {
  int64_t left;       // units to do
  int s, item, unit;  // from this unit of the item on
  Request r;
};

// Sums every request's units and finds where this warp's share starts.
// by_rows: an item per eight virtual rows (else one per head).  CTA 0 writes
// down the requests' first units.
template <typename T>
__device__ __forceinline__ Range plan_range(const Args<T>& a, bool by_rows, int64_t* unit_start) {
  __shared__ int64_t warp_sum[WARPS];
  __shared__ Range found[WARPS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int chunk = (a.S + THREADS - 1) / THREADS;
  const int s0 = min(a.S, tid * chunk), s1 = min(a.S, s0 + chunk);
  int64_t mine = 0;
  bool any_bad = false;
  Request r{};
  for (int s = s0; s < s1; ++s) {
    bool bad = false;
    r = load_request(a, s, by_rows, &bad);
    any_bad |= bad;
    mine += r.units();
  }
  if (any_bad && blockIdx.x == 0) atomicOr(a.status, STATUS_KV_RANGE);
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_sum[warp] = incl;
  if (tid < WARPS) found[tid].left = 0;
  __syncthreads();
  int64_t base = 0, all = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) base += warp_sum[w];
    all += warp_sum[w];
  }
  int64_t start = base + incl - mine;
  const Shares share(all, gridDim.x * WARPS);
  const bool note = unit_start && blockIdx.x == 0;
#pragma unroll 1
  for (int s = s0; s < s1; ++s) {
    if (chunk > 1) r = load_request(a, s, by_rows);
    const int64_t units = r.units();
    if (note) unit_start[s] = start;
#pragma unroll 1
    for (int w = 0; w < WARPS; ++w) {
      const int worker = w * gridDim.x + blockIdx.x;
      if (worker >= share.workers) break;
      const int64_t u0 = share.start(worker);
      if (u0 < start || u0 >= start + units) continue;
      const int64_t in = u0 - start;
      const int item = in < (int64_t)1 << 31 ? (int)in / r.span() : (int)(in / r.span());
      found[w] = Range{share.start(worker + 1) - u0, s, item, (int)(in - (int64_t)item * r.span()), r};
    }
    start += units;
  }
  if (note && tid == THREADS - 1) unit_start[a.S] = all;
  __syncthreads();
  return found[warp];
}

// Walks a range segment by segment: a run of tiles of one item.
template <typename T>
struct Walk {
  int64_t left;
  int s, item, t0, t1;  // the segment: tiles [t0, t1) of the item; t0 == t1 when none is left
  Request r;
  __device__ __forceinline__ void begin(const Args<T>& a, const Range& g, bool by_rows) {
    left = g.left;
    s = g.s;
    item = g.item;
    r = g.r;
    t0 = t1 = 0;
    if (left > 0 && !cut(g.unit)) next(a, by_rows);
  }
  // the segment from unit u of the item on; false when no tile is in it
  __device__ __forceinline__ bool cut(int u) {
    const int end = (int)min(u + left, (int64_t)r.span());
    left -= end - u;
    t0 = max(u - ITEM_UNITS, 0);
    t1 = max(end - ITEM_UNITS, 0);
    return t0 < t1;
  }
  __device__ __forceinline__ void next(const Args<T>& a, bool by_rows) {
    do {
      t0 = t1 = 0;
      if (left <= 0) return;
      if (++item >= r.items) {
        item = 0;
        do {
          if (++s >= a.S) {
            left = 0;
            return;
          }
          r = load_request(a, s, by_rows);
        } while (r.tiles == 0);
      }
    } while (!cut(0));
  }
};

// ---------------------------------------------------------------- queries
// The query of eight virtual rows.  Its fragments (A registers of each block and
// k-step, rows 0-7 hi and rows 8-15 lo) are kept in shared memory, a 16-byte
// vector per lane: they serve four products each time they are loaded, and the
// registers that they would hold keep three CTAs per SM free of spills.
template <int D>
struct Query {
  const uint4* frag;        // [block][k-step][lane]
  float bias[Kvq<D>::NB];   // row g: what a block's partial score has too much, negative
  float factor;             // row g: from partial scores to scores
};
template <int D>
constexpr int QUERY_BYTES = Kvq<D>::NB * 2 * 32 * 16;

// 2^e for -126 <= e <= 127
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

template <int D, typename T>
__device__ __forceinline__ void load_query(Query<D>& f, uint4* frag, const Args<T>& a, const Request& r, int head,
                                           int row0, int lane) {
  constexpr int NB = Kvq<D>::NB;
  const int g = lane >> 2, tq = lane & 3;
  const int vr = row0 + g;
  float x[NB][8];
  float top = 0.0f;
  if (vr < r.n * a.group) {
    const int j = vr / a.group, hg = vr - j * a.group;
    const T* p = a.q + (int64_t)(r.b + j) * a.q_token + (int64_t)(head * a.group + hg) * a.q_head + 8 * tq;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      kvq_load8<true>(p + 32 * b, x[b]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[b][i] *= a.scale_log2;
        top = fmaxf(top, fabsf(x[b][i]));
      }
    }
  } else {
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < 8; ++i) x[b][i] = 0.0f;
  }
  top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
  top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
  // the row's largest value goes to [1024, 2048); two factors, as 2^-e may not be a normal number
  int e = 0;
  if (top > 0.0f && top < INFINITY) e = max(((__float_as_int(top) >> 23) & 255) - 127, -126) - 10;
  const float up1 = pow2((-e) / 2), up2 = pow2(-e - (-e) / 2);
  f.factor = scalbnf(1.0f, 24 + e);
  f.frag = frag + lane;
  __syncwarp();  // the last query's fragments have been read
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    float sum = 0.0f;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 2; ++k) {  // values (2s + k) and (2s + k) + 4; the second pair meets codes of factor 16
        const float x0 = x[b][2 * s + k] * up1 * up2, x1 = x[b][2 * s + k + 4] * up1 * up2;
        const float h0 = rintf(x0), h1 = rintf(x1);
        const float down = k ? 0.0625f : 1.0f, back = k ? 16.0f : 1.0f;
        w[2 * k] = pack(h0 * down, h1 * down);
        w[2 * k + 1] = pack((x0 - h0) * down, (x1 - h1) * down);
        const float2 fl = __half22float2(*reinterpret_cast<const __half2*>(&w[2 * k + 1]));
        sum += (h0 + fl.x * back) + (h1 + fl.y * back);
      }
      frag[(2 * b + s) * 32 + lane] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
    f.bias[b] = sum * (-8.0f * 0x1p-24f);
  }
  __syncwarp();
}

template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x;
    w[1] = v.y;
    w[2] = v.z;
    w[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x;
    w[1] = v.y;
  }
}

// The scale pairs of a lane's two columns, positions 8t + 2 tq and the next.
template <int D>
__device__ __forceinline__ void load_scales(const uint8_t* scl, int t, int tq, uint32_t (&w)[Kvq<D>::NB]) {
  load_words<Kvq<D>::NB>(scl + (4 * t + tq) * 4 * Kvq<D>::NB, w);
}

// Scores (log2 units) of a tile: sc[u] for this lane's row g and the positions
// 8u + 2 tq, + 1.
template <int D>
__device__ __forceinline__ void scores(const uint8_t* tile, const Query<D>& q, int g, int tq,
                                       float (&sc)[KVQ_POS / 8][2]) {
  constexpr int NB = Kvq<D>::NB, N = KVQ_POS / 8;
  uint32_t w[N][NB], d[N][NB];
  F2 s[N];
#pragma unroll
  for (int u = 0; u < N; ++u) {
    load_words<NB>(tile + 8 * u * Kvq<D>::ROW + (4 * g + tq) * 4 * NB, w[u]);
    load_scales<D>(tile + Kvq<D>::KS_OFF, u, tq, d[u]);
    s[u] = f2(0.0f, 0.0f);
  }
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const uint4 x = q.frag[2 * b * 32], y = q.frag[(2 * b + 1) * 32];
    const uint32_t a0[4] = {x.x, x.y, x.z, x.w}, a1[4] = {y.x, y.y, y.z, y.w};
    const float zero[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int u = 0; u < N; ++u) {
      float c[4];
      uint32_t r[4];
      unpack(w[u][b], r);
      mma(c, a0, r[0], r[1], zero);
      mma(c, a1, r[2], r[3], c);
      const F2 t = add2(add2(f2(c[0], c[1]), f2(q.bias[b], q.bias[b])), f2(c[2], c[3]));
      s[u] = fma2(half2_f2(d[u][b]), t, s[u]);
    }
  }
#pragma unroll
  for (int u = 0; u < N; ++u) {
    const float2 x = unf2(mul2(s[u], f2(q.factor, q.factor)));
    sc[u][0] = x.x;
    sc[u][1] = x.y;
  }
}

// ---------------------------------------------------------------- sums
constexpr uint32_t HALF_ONE = 0x3C00u;   // 1 in binary16
constexpr uint32_t HALF_TOP = 0x7800u;   // 2^15
constexpr uint32_t HALF_LOW = 0x0400u;   // 2^-14, its smallest normal number

// A warp's running sums over the positions it has taken.  Weights are
// w = 2^(score - m + up), where m is at most SLACK below the largest score, and meet V's
// scales times a power of two: with T the largest scale so far as a power of two,
// kept within 2^-14 .. 2^15, up is 9 and the scales are taken by 1 / T where T <= 1,
// else up is 9 - log2 T and they are taken as they are.  A weight times a scale is then
// at most 2^14 (2^15 for scales above 2^15), and o holds 2^9 / T times its sum either way.
template <int D>
struct Sums {
  float o[Kvq<D>::NB][2][4];  // [block][values 4g + 2i, + 1][rows 2 tq, 2 tq + 1, twice]
  F2 l;                       // row g
  float m, off;               // row g: the reference score, and m - up (m in far rows, 0 while m is -inf)
  float most;                 // row g: the score that calls for another reference
  uint32_t dtop;              // T in both halves
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int b = 0; b < Kvq<D>::NB; ++b)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[b][i][k] = 0.0f;
    l = f2(0.0f, 0.0f);
    m = most = NEG_INF;
    off = 0.0f;
    dtop = HALF_LOW << 16 | HALF_LOW;
  }
  __device__ __forceinline__ int top_exponent() const { return (int)(dtop >> 26) - 15; }  // log2 T
  __device__ __forceinline__ int up() const { return 9 - max(top_exponent(), 0); }
  // row g's own
  __device__ __forceinline__ bool far() const { return fabsf(m) >= FAR; }
  __device__ __forceinline__ int row_up() const { return far() ? 0 : up(); }
  // what the scales are multiplied with, in both halves: 1 / T, at least 1
  __device__ __forceinline__ __half2 lift() const {
    return __hmax2(half2_of((HALF_TOP << 16 | HALF_TOP) - dtop), half2_of(HALF_ONE << 16 | HALF_ONE));
  }
};

// Takes the positions p0 .. p0 + 31 of a tile.  MASKED: some row does not see
// them all; row g sees those up to `last`, and what lies at `end` and after
// may be anything.
template <int D, bool MASKED>
__device__ __forceinline__ void take_tile(const uint8_t* tile, int p0, const Query<D>& q, Sums<D>& a, int g, int tq,
                                          int last, int end) {
  using L = Kvq<D>;
  constexpr int NB = L::NB, N = L::POS / 8;
  // V scale pairs of eight positions; those of positions past the end are zero
  auto v_scales = [&](int u, uint32_t (&vd)[NB]) {
    load_scales<D>(tile + L::VS_OFF, u, tq, vd);
    if constexpr (MASKED) {
      const int p = p0 + 8 * u + 2 * tq;
      const uint32_t keep = (p < end ? 0x0000FFFFu : 0u) | (p + 1 < end ? 0xFFFF0000u : 0u);
#pragma unroll
      for (int b = 0; b < NB; ++b) vd[b] &= keep;
    }
  };
  float sc[N][2];
  scores<D>(tile, q, g, tq, sc);
  float top = NEG_INF;
  __half2 dm = *reinterpret_cast<const __half2*>(&a.dtop);
#pragma unroll
  for (int u = 0; u < N; ++u) {
    if constexpr (MASKED) {
      const int p = p0 + 8 * u + 2 * tq;
      if (p > last) sc[u][0] = NEG_INF;
      if (p + 1 > last) sc[u][1] = NEG_INF;
    }
    top = fmaxf(top, fmaxf(sc[u][0], sc[u][1]));
    uint32_t vd[NB];
    v_scales(u, vd);
#pragma unroll
    for (int b = 0; b < NB; ++b) dm = __hmax2(dm, __habs2(*reinterpret_cast<const __half2*>(&vd[b])));
  }
  const uint32_t dmw = *reinterpret_cast<const uint32_t*>(&dm);
  if (__any_sync(0xFFFFFFFFu, top > a.most || dmw != a.dtop)) {
    float mn = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    mn = fmaxf(a.m, fmaxf(mn, __shfl_xor_sync(0xFFFFFFFFu, mn, 2)));
    uint32_t h = max(dmw & 0xFFFFu, dmw >> 16);  // magnitudes order as integers
    h = max(h, __shfl_xor_sync(0xFFFFFFFFu, h, 1));
    h = max(h, __shfl_xor_sync(0xFFFFFFFFu, h, 2));
    h = max(min((h + 0x3FFu) & 0x7C00u, HALF_TOP), HALF_LOW);  // up to a power of two
    const int up = a.up(), top_e = a.top_exponent();
    a.dtop = h | h << 16;
    const bool none = a.m == NEG_INF;
    a.m = mn;
    const float no = mn == NEG_INF ? 0.0f : a.far() ? mn : mn - (float)a.up();
    const float f = none ? 1.0f : ex2(a.off - no);  // nothing summed yet while m is -inf
    a.off = no;
    a.most = a.far() ? mn : mn + SLACK;
    a.l = mul2(a.l, f2(f, f));
    // o's own factor has the change of the scales' lift
    const float fo = f * pow2((top_e + up) - (a.top_exponent() + a.up()));
    const float f0 = __shfl_sync(0xFFFFFFFFu, fo, 8 * tq), f1 = __shfl_sync(0xFFFFFFFFu, fo, 8 * tq + 4);
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        a.o[b][i][0] *= f0;
        a.o[b][i][1] *= f1;
        a.o[b][i][2] *= f0;
        a.o[b][i][3] *= f1;
      }
  }
  const __half2 lift = a.lift();
#pragma unroll
  for (int k = 0; k < N / 2; ++k) {  // sixteen keys a product: eight positions 2k, eight positions 2k + 1
    __half2 wh[2], wl[2];
    uint32_t vd[2][NB], vw[2][NB], keep[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int e = 2 * k + u;
      const float w0 = ex2(sc[e][0] - a.off), w1 = ex2(sc[e][1] - a.off);
      const F2 w = f2(w0, w1);
      a.l = add2(a.l, w);
      split(w, wh[u], wl[u]);
      // a weight of 0 keeps a NaN scale out
      if constexpr (MASKED) keep[u] = (sc[e][0] == NEG_INF ? 0u : 0x0000FFFFu) | (sc[e][1] == NEG_INF ? 0u : 0xFFFF0000u);
      v_scales(e, vd[u]);
      load_words<NB>(tile + L::V_OFF + 8 * e * L::ROW + (4 * g + tq) * 4 * NB, vw[u]);
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      // weights times the block's V scales, as hi and lo terms: B operand with keys along k
      uint32_t hi[2], lo[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const __half2 d = __hmul2(half2_of(vd[u][b]), lift);  // exact
        const __half2 h = __hmul2(wh[u], d);
        hi[u] = bits(h);
        lo[u] = bits(__hfma2(wl[u], d, __hfma2(wh[u], d, __hneg2(h))));
        if constexpr (MASKED) {
          hi[u] &= keep[u];
          lo[u] &= keep[u];
        }
      }
      uint32_t r0[4], r1[4];
      kvq_unpack_centred(vw[0][b], r0);
      kvq_unpack_centred(vw[1][b], r1);
#pragma unroll
      for (int i = 0; i < 2; ++i) {  // values 4g + 2i and 4g + 2i + 1 of the block as rows g and g + 8
        const uint32_t av[4] = {r0[2 * i], r0[2 * i + 1], r1[2 * i], r1[2 * i + 1]};
        mma(a.o[b][i], av, hi[0], hi[1], a.o[b][i]);
        mma(a.o[b][i], av, lo[0], lo[1], a.o[b][i]);
      }
    }
  }
}

// ---------------------------------------------------------------- main kernel
template <int D, typename T>
__global__ void __launch_bounds__(THREADS, CTAS_PER_SM) kvq_attention_kernel(const Args<T> a) {
  using L = Kvq<D>;
  constexpr int NB = L::NB;
  extern __shared__ __align__(128) uint8_t smem[];  // a ring per warp, then a query per warp
  __shared__ uint64_t bars[WARPS][STAGES];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, tq = lane & 3;
  const uint8_t* ring = smem + warp * STAGES * L::BYTES;
  const uint32_t ring_u32 = smem_u32(ring), bar_u32 = smem_u32(bars[warp]);
  if (lane < STAGES) mbar_init(bar_u32 + 8 * lane, 1);
  mbar_init_fence();
  __syncwarp();
  asm volatile("griddepcontrol.wait;" ::: "memory");  // this launch begins under the end of the one before
  // Only now may the join begin, and behind it the weights' launch: what they read
  // before their own waits (the step's description, queries, the cache) was written by
  // launches that ended before this line.
  asm volatile("griddepcontrol.launch_dependents;");
  const int worker = warp * gridDim.x + blockIdx.x;

  // the issue cursor runs ahead of the consuming one by up to STAGES tiles
  Walk<T> in, out;
  {
    const Range range = plan_range(a, true, a.unit_start);
    in.begin(a, range, true);
    out.begin(a, range, true);
  }
  const uint8_t* in_ptr = nullptr;  // the next tile of the issue cursor's segment
  int in_left = 0;                  // and how many are left of it
  auto enter = [&]() {
    const int head = in.item / (in.r.items / a.heads);
    in_ptr = a.cache + ((int64_t)in.r.slot * a.heads + head) * a.plane_bytes + (int64_t)in.t0 * L::BYTES;
    in_left = in.t1 - in.t0;
  };
  if (in.t0 < in.t1) enter();
  unsigned issued = 0, taken = 0;
  auto issue = [&]() {  // the next tile, if any, into the ring
    if (in_left == 0) {
      if (in.t0 >= in.t1) return;
      in.next(a, true);
      if (in.t0 >= in.t1) return;
      enter();
    }
    if (lane == 0 && !a.stall) {
      const unsigned st = issued % STAGES;
      mbar_expect_tx(bar_u32 + 8 * st, L::BYTES);
      bulk_load(ring_u32 + st * L::BYTES, in_ptr, L::BYTES, bar_u32 + 8 * st);
    }
    ++issued;
    --in_left;
    in_ptr += L::BYTES;
  };
  // One tile each before the rest: asked for all at once, the first tiles come
  // in among the others', and every warp begins late.
  issue();
  int primed = 1;

  while (out.t0 < out.t1) {
    const Request& r = out.r;
    const int groups = r.items / a.heads;  // row groups of a head
    const int head = out.item / groups, row0 = (out.item - head * groups) * ROWS;
    Query<D> q;
    load_query<D, T>(q, reinterpret_cast<uint4*>(smem + WARPS * STAGES * L::BYTES + warp * QUERY_BYTES<D>), a, r, head,
                     row0, lane);
    for (; primed < STAGES; ++primed) issue();
    Sums<D> sums;
    sums.clear();
    const int last = r.pos + (row0 + g) / a.group;  // the row's last visible position
    const int clear = r.pos + row0 / a.group + 1;   // positions below are visible to every row
    const int end = r.pos + r.n;                    // positions from here on hold anything

    for (int t = out.t0; t < out.t1; ++t) {
      const unsigned st = taken % STAGES;
      if (!mbar_wait_warp(bar_u32 + 8 * st, (taken / STAGES) & 1, a.wait_ns)) {
        // a copy never landed: wait (again with a limit) for the others in flight and give up
        if (lane == 0) atomicOr(a.status, STATUS_TIMEOUT);
        for (; taken < issued; ++taken)
          mbar_wait_warp(bar_u32 + 8 * (taken % STAGES), (taken / STAGES) & 1, a.wait_ns);
        return;
      }
      ++taken;
      const uint8_t* tile = ring + st * L::BYTES;
      if ((t + 1) * L::POS <= clear) take_tile<D, false>(tile, t * L::POS, q, sums, g, tq, last, end);
      else take_tile<D, true>(tile, t * L::POS, q, sums, g, tq, last, end);
      __syncwarp();  // every lane has read the stage before it is written again
      issue();
    }

    // ---- the segment's sums: the result, or a part for the join ----
    const float2 lp = unf2(sums.l);
    float l = lp.x + lp.y;
    l += __shfl_xor_sync(0xFFFFFFFFu, l, 1);
    l += __shfl_xor_sync(0xFFFFFFFFu, l, 2);
    const float down = pow2(-sums.row_up());                             // l's factor, and that of the scales in o
    const float down_scales = pow2(sums.top_exponent() + sums.up() - 9);
    const bool whole = out.t0 == 0 && out.t1 == r.tiles;
    const int rows = r.n * a.group;
    // the row of this lane's l is g, those of its values 2 tq and 2 tq + 1
    const int64_t slot = ((int64_t)2 * worker + (out.t0 == 0 ? 1 : 0)) * ROWS;
    const float f = whole ? down_scales / l : down * down_scales;
    if (whole) {
      if (a.lse && tq == 0 && row0 + g < rows) {
        const int j = (row0 + g) / a.group;
        a.lse[(int64_t)(r.b + j) * (a.heads * a.group) + head * a.group + row0 + g - j * a.group] =
            make_float2(sums.off, log2f(l));
      }
    } else if (tq == 0) {
      a.partial_ml[slot + g] = make_float2(sums.m, l * down);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int row = 2 * tq + k;
      const float fr = __shfl_sync(0xFFFFFFFFu, f, 4 * row);
      const int j = (row0 + row) / a.group;
      const int64_t at = (int64_t)(r.b + j) * (a.heads * a.group) + head * a.group + row0 + row - j * a.group;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const float v[4] = {sums.o[b][0][k] * fr, sums.o[b][0][2 + k] * fr, sums.o[b][1][k] * fr,
                            sums.o[b][1][2 + k] * fr};
        if (!whole) kvq_store4(a.partial + (slot + row) * D + 32 * b + 4 * g, v);
        else if (row0 + row < rows) kvq_store4(a.out + at * D + 32 * b + 4 * g, v);
      }
    }
    out.next(a, true);
  }
}

// ---------------------------------------------------------------- join
// Joins the partial sums of items cut between workers; rows of no request, or of
// one that is out of range, get zeros.  PER_ROW warps take a (packed row, query
// head): one where an item has few parts, the whole CTA where it has many.  Bound by
// the latency of a few dependent loads, most of it under the main launch's end: 64
// rows of 28 heads take 8.5 us cold and alone, and add 3 us to the main launch.
template <int D, typename T, int PER_ROW>
__global__ void __launch_bounds__(32 * JOIN_WARPS) kvq_join_kernel(const Args<T> a) {
  constexpr int PER = D / 32, AT_ONCE = 8;
  __shared__ float2 s_ml[JOIN_WARPS];
  __shared__ float s_acc[JOIN_WARPS][D];
  const int lane = threadIdx.x & 31;
  const int warp = PER_ROW == 1 ? 0 : threadIdx.x >> 5, tid = warp * 32 + lane;  // within the row's warps
  const int q_heads = a.heads * a.group;
  const int at = PER_ROW == 1 ? blockIdx.x * JOIN_WARPS + (threadIdx.x >> 5) : blockIdx.x;
  const int t = at / q_heads, hq = at - t * q_heads;
  // the weights' launch may begin: what it reads before its wait, the main launch does not write
  asm volatile("griddepcontrol.launch_dependents;");
  const int s = kvq_find_request<true>(a.offsets, a.S, t, lane);
  const Request r = load_request(a, s, true);
  T* out = a.out + (int64_t)at * D;
  if (r.tiles == 0 || t < r.b || t >= r.b + r.n) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (t < a.total) {
      for (int d = tid; d < D; d += 32 * PER_ROW) out[d] = (T)0.0f;
      if (a.lse && tid == 0) a.lse[at] = make_float2(NEG_INF, 0.0f);
    }
    return;
  }
  const int head = hq / a.group;
  const int vr = (t - r.b) * a.group + (hq - head * a.group);
  const int item = head * (r.items / a.heads) + vr / ROWS, row = vr % ROWS;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t all = __ldcg(a.unit_start + a.S), u_item = __ldcg(a.unit_start + s);
  const Shares share(all, a.workers);
  const int64_t u0 = u_item + (int64_t)item * r.span() + ITEM_UNITS;  // the first tile
  const int wa = share.of(u0), wb = share.of(u0 + r.tiles - 1);
  if (wa == wb) return;  // written by the main launch
  // eight parts on their way at once per warp
  float top = NEG_INF, sum = 0.0f, acc[PER] = {};
  auto scale_of = [](float m, float top) { return m == NEG_INF ? 0.0f : ex2(m - top); };
  for (int w0 = wa + warp; w0 <= wb; w0 += PER_ROW * AT_ONCE) {
    float2 ml[AT_ONCE];
    float v[AT_ONCE][PER];
    float nt = top;
#pragma unroll
    for (int k = 0; k < AT_ONCE; ++k) {
      const int w = w0 + k * PER_ROW;
      ml[k] = make_float2(NEG_INF, 0.0f);
#pragma unroll
      for (int i = 0; i < PER; ++i) v[k][i] = 0.0f;
      if (w <= wb) {
        const int64_t p = (int64_t)(2 * w + (w == wa)) * ROWS + row;
        ml[k] = __ldcg(a.partial_ml + p);
        if constexpr (PER == 4) *reinterpret_cast<float4*>(v[k]) = __ldcg(reinterpret_cast<const float4*>(a.partial + p * D + lane * 4));
        else *reinterpret_cast<float2*>(v[k]) = __ldcg(reinterpret_cast<const float2*>(a.partial + p * D + lane * 2));
      }
    }
#pragma unroll
    for (int k = 0; k < AT_ONCE; ++k) nt = fmaxf(nt, ml[k].x);
    const float f0 = scale_of(top, nt);
    top = nt;
    sum *= f0;
#pragma unroll
    for (int i = 0; i < PER; ++i) acc[i] *= f0;
#pragma unroll
    for (int k = 0; k < AT_ONCE; ++k) {
      const float f = scale_of(ml[k].x, nt);
      sum = fmaf(ml[k].y, f, sum);
#pragma unroll
      for (int i = 0; i < PER; ++i) acc[i] = fmaf(v[k][i], f, acc[i]);
    }
  }
  if (PER_ROW == 1) {
    const float inv = 1.0f / sum;
#pragma unroll
    for (int i = 0; i < PER; ++i) out[lane * PER + i] = (T)(acc[i] * inv);
    if (a.lse && lane == 0) a.lse[at] = make_float2(top, log2f(sum));
    return;
  }
  if (lane == 0) s_ml[warp] = make_float2(top, sum);
#pragma unroll
  for (int i = 0; i < PER; ++i) s_acc[warp][lane * PER + i] = acc[i];
  __syncthreads();
  if (tid >= D) return;
  top = NEG_INF;
#pragma unroll
  for (int w = 0; w < JOIN_WARPS; ++w) top = fmaxf(top, s_ml[w].x);
  sum = 0.0f;
  float x = 0.0f;
#pragma unroll
  for (int w = 0; w < JOIN_WARPS; ++w) {
    const float f = scale_of(s_ml[w].x, top);
    sum = fmaf(s_ml[w].y, f, sum);
    x = fmaf(s_acc[w][tid], f, x);
  }
  out[tid] = (T)(x / sum);
  if (a.lse && tid == 0) a.lse[at] = make_float2(top, log2f(sum));
}

// ---------------------------------------------------------------- weights
// mass[slot, head, p] += sum over the request's rows and the group's heads of
// exp2(s - m - log2 l), m a row's reference and l its sum; a position that this step appended starts from 0.  Reads the
// K half of the cache again: keeping the scores instead would write and read
// as many bytes for a group of seven heads.  The eight rows' weights of a tile
// are summed over lanes and dealt out in seven shuffles, a position to each
// lane; every position belongs to one lane, so the sums have a fixed order.
// 32 requests of 103,047 positions (4 heads of 128): 17 us cold, 30 MB of K;
// it starts when the join is done and is bound as the main launch is.
template <int D, typename T>
__global__ void __launch_bounds__(THREADS) kvq_mass_kernel(const Args<T> a) {
  using L = Kvq<D>;
  constexpr int HALF = L::V_OFF;  // bytes of a tile's K half
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint4 frags[WARPS][QUERY_BYTES<D> / 16];
  __shared__ uint64_t bars[WARPS][MASS_STAGES];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, tq = lane & 3;
  const uint8_t* ring = smem + warp * MASS_STAGES * HALF;
  const uint32_t ring_u32 = smem_u32(ring), bar_u32 = smem_u32(bars[warp]);
  if (lane < MASS_STAGES) mbar_init(bar_u32 + 8 * lane, 1);
  mbar_init_fence();
  __syncwarp();
  const Range range = plan_range(a, false, nullptr);
  // the lane's position of a tile after the sums are dealt out: 8u + 2 tq + c
  const int mine = ((g >> 1) & 3) * 8 + 2 * tq + (g & 1);
  unsigned issued = 0, taken = 0;
  bool waited = false;
  Walk<T> it;
  for (it.begin(a, range, false); it.t0 < it.t1; it.next(a, false)) {
    const Request& r = it.r;
    const int head = it.item;
    const uint8_t* plane = a.cache + ((int64_t)r.slot * a.heads + head) * a.plane_bytes;
    float* mass = a.mass + ((int64_t)r.slot * a.heads + head) * a.capacity;
    const int rows = r.n * a.group, end = r.pos + r.n;
    for (int row0 = 0; row0 < rows; row0 += ROWS) {
      int next = it.t0;
      auto issue = [&]() {
        if (next >= it.t1) return;
        if (lane == 0 && !a.stall) {
          const unsigned st = issued % MASS_STAGES;
          mbar_expect_tx(bar_u32 + 8 * st, HALF);
          bulk_load(ring_u32 + st * HALF, plane + (int64_t)next * L::BYTES, HALF, bar_u32 + 8 * st);
        }
        ++issued;
        ++next;
      };
      for (int i = 0; i < MASS_STAGES; ++i) issue();
      Query<D> q;
      load_query<D, T>(q, frags[warp], a, r, head, row0, lane);
      if (!waited) {  // what follows needs the rows' sums
        asm volatile("griddepcontrol.wait;" ::: "memory");
        waited = true;
      }
      const int vr = row0 + g;
      const bool live = vr < rows;
      const int j = live ? vr / a.group : 0;
      const int64_t row = (int64_t)(r.b + j) * (a.heads * a.group) + head * a.group + vr - j * a.group;
      const float2 lse = live ? __ldcg(a.lse + row) : make_float2(0.0f, 0.0f);
      const int last = live ? r.pos + j : -1;
      for (int t = it.t0; t < it.t1; ++t) {
        const int pm = t * L::POS + mine;
        const float old = pm < end && (row0 > 0 || pm < r.pos) ? __ldcg(mass + pm) : 0.0f;
        const unsigned st = taken % MASS_STAGES;
        if (!mbar_wait_warp(bar_u32 + 8 * st, (taken / MASS_STAGES) & 1, a.wait_ns)) {
          if (lane == 0) atomicOr(a.status, STATUS_TIMEOUT);
          for (; taken < issued; ++taken)
            mbar_wait_warp(bar_u32 + 8 * (taken % MASS_STAGES), (taken / MASS_STAGES) & 1, a.wait_ns);
          return;
        }
        ++taken;
        float sc[L::POS / 8][2];
        scores<D>(ring + st * HALF, q, g, tq, sc);
        __syncwarp();
        issue();
        float w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int p = t * L::POS + 8 * (e >> 1) + 2 * tq + (e & 1);
          w[e] = p <= last ? ex2(sc[e >> 1][e & 1] - lse.x - lse.y) : 0.0f;
        }
        // bits 2, 1, 0 of a value's index go to bits 2, 1, 0 of the lane's g
#pragma unroll
        for (int k = 4; k > 0; k >>= 1) {
          const bool high = g & k;
#pragma unroll
          for (int e = 0; e < k; ++e) {
            const float give = high ? w[e] : w[e + k];
            const float got = __shfl_xor_sync(0xFFFFFFFFu, give, 4 * k);
            w[e] = (high ? w[e + k] : w[e]) + got;
          }
        }
        if (pm < end) mass[pm] = old + w[0];
      }
    }
  }
  if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");  // the launch ends after the ones before
}

template <int D, typename T>
int launch_as(const KvqStep& c, const uint8_t* cache, const void* q, const int64_t* qs, int q_heads, float scale,
              void* out, float* mass, const KvqAttnScratch& ws, cudaStream_t s) {
  Args<T> a;
  a.cache = cache;
  a.q = static_cast<const T*>(q);
  a.q_token = qs[0];
  a.q_head = qs[1];
  a.out = static_cast<T*>(out);
  a.scale_log2 = scale * 1.44269504088896340736f;
  a.slots = c.slots;
  a.capacity = c.capacity;
  a.plane_bytes = kvq_plane_bytes(D, c.capacity);
  a.total = c.total;
  a.heads = (int)c.heads;
  a.group = q_heads / (int)c.heads;
  a.S = c.S;
  a.offsets = c.offsets;
  a.slot = c.slot;
  a.pos = c.pos;
  a.status = c.status;
  a.wait_ns = wait_limit_ns();
  a.stall = stall_for_test();
  a.workers = c.num_sms * CTAS_PER_SM * WARPS;
  a.partial = ws.partial;
  a.partial_ml = ws.partial_ml;
  a.unit_start = ws.unit_start;
  a.lse = mass ? ws.lse : nullptr;
  a.mass = mass;
  constexpr int SMEM = WARPS * (STAGES * Kvq<D>::BYTES + QUERY_BYTES<D>);
  constexpr int MASS_SMEM = WARPS * MASS_STAGES * Kvq<D>::V_OFF;
  static std::atomic<bool> sized[64];  // per device: the kernels' shared memory limits are set
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return Q4_ERR_CUDA;
  if (!sized[dev].load()) {
    if (cudaFuncSetAttribute(kvq_attention_kernel<D, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM) !=
            cudaSuccess ||
        cudaFuncSetAttribute(kvq_mass_kernel<D, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, MASS_SMEM) !=
            cudaSuccess)
      return Q4_ERR_CUDA;
    sized[dev].store(true);
  }
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(c.num_sms * CTAS_PER_SM);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kvq_attention_kernel<D, T>, a) != cudaSuccess) return Q4_ERR_CUDA;
  // Parts an item has on average: a warp joins up to 16 in two rounds of loads.
  // 64 ragged requests (7 parts) take 41.4 us in all with a CTA a row, 35.2 with a
  // warp; 8 requests at 32k (57 parts) 8 us less with a CTA than with a warp; one
  // of 2,049 12.0 and 8.1.
  const int64_t rows = c.total * q_heads;
  const int64_t items = c.total * c.heads * ((a.group + ROWS - 1) / ROWS);
  const bool few = items * 16 >= a.workers;
  cfg.gridDim = dim3((unsigned)(few ? (rows + JOIN_WARPS - 1) / JOIN_WARPS : rows));
  cfg.blockDim = dim3(32 * JOIN_WARPS);
  cfg.dynamicSmemBytes = 0;
  if ((few ? cudaLaunchKernelEx(&cfg, kvq_join_kernel<D, T, 1>, a)
           : cudaLaunchKernelEx(&cfg, kvq_join_kernel<D, T, JOIN_WARPS>, a)) != cudaSuccess)
    return Q4_ERR_CUDA;
  if (mass) {
    cfg.gridDim = dim3(c.num_sms * MASS_CTAS_PER_SM);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = MASS_SMEM;
    if (cudaLaunchKernelEx(&cfg, kvq_mass_kernel<D, T>, a) != cudaSuccess) return Q4_ERR_CUDA;
  }
  return Q4_OK;
}

template <typename T>
int launch_d(const KvqStep& c, const uint8_t* cache, const void* q, const int64_t* qs, int q_heads, float scale,
             void* out, float* mass, const KvqAttnScratch& ws, cudaStream_t s) {
  return c.head_dim == 128 ? launch_as<128, T>(c, cache, q, qs, q_heads, scale, out, mass, ws, s)
                           : launch_as<64, T>(c, cache, q, qs, q_heads, scale, out, mass, ws, s);
}

}  // namespace

size_t kvq_attn_scratch_bytes(int64_t S, int64_t total, int q_heads, bool mass, int num_sms, KvqAttnScratch* out,
                              uint8_t* base) {
  // sized for D = 128, so one area serves both head sizes
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += (bytes + 255) / 256 * 256;
    return o;
  };
  const size_t segs = (size_t)2 * num_sms * CTAS_PER_SM * WARPS * ROWS;
  const size_t p = take(segs * 128 * sizeof(float)), ml = take(segs * sizeof(float2));
  const size_t us = take((size_t)(S + 1) * sizeof(int64_t)), ls = take(mass ? (size_t)total * q_heads * sizeof(float2) : 0);
  if (out) {
    out->partial = reinterpret_cast<float*>(base + p);
    out->partial_ml = reinterpret_cast<float2*>(base + ml);
    out->unit_start = reinterpret_cast<int64_t*>(base + us);
    out->lse = reinterpret_cast<float2*>(base + ls);
  }
  return at;
}

int launch_kvq_attention(const KvqStep& c, const uint8_t* cache, const void* q, const int64_t* qs, int q_heads,
                         float scale, void* out, float* mass, int dtype, const KvqAttnScratch& ws, cudaStream_t s) {
  if (dtype == Q4_DTYPE_F32) return launch_d<float>(c, cache, q, qs, q_heads, scale, out, mass, ws, s);
  if (dtype == Q4_DTYPE_F16) return launch_d<__half>(c, cache, q, qs, q_heads, scale, out, mass, ws, s);
  return launch_d<__nv_bfloat16>(c, cache, q, qs, q_heads, scale, out, mass, ws, s);
}

}  // namespace q4
