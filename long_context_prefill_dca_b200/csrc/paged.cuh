// paged.cuh — the paged fp16 cache of DCA keys and values: what its kernels share, the append
// of a ragged batch of tokens, and the decode attention of a batch (one query token per
// sequence), all keys or a sliding window with sinks.
//
// Cache: k_pages, v_pages [n_pages][Hkv][page_size][D] fp16; position j of sequence b lives in
// page page_table[b][j / page_size], row j % page_size, its key rotated at j mod L (the same
// remap as the contiguous cache: rope_dca.cuh). Lengths, token offsets and page tables are
// device arrays, so one captured graph serves every step of a generation.
#pragma once

#include "q1m_device.cuh"
#include "rope_dca.cuh"
#include "decode.cuh"

namespace q1m {

constexpr int PG_MAX_CTAS = 160;     // persistent CTAs at most (scratch is sized for it)
constexpr int PG_MAX_BATCH = Q1M_MAX_PAGED_BATCH;
constexpr int32_t PG_MAX_LEN = 1 << 30;   // positions of a sequence

// What every paged kernel knows of the cache.
struct PagedCacheArgs {
  const int32_t* page_table;   // [batch] rows
  int64_t table_stride;        // entries between rows
  int32_t n_pages;
  int32_t page_log2;           // page_size = 1 << page_log2, 16 .. 128
  int32_t hkv;
  int32_t max_len;             // positions that a table row's own entries hold, PG_MAX_LEN at most
};

// dca_query_pos in 32 bits (a 64-bit remainder takes over 100 cycles more).
__device__ __forceinline__ int32_t dca_query_pos32(int32_t i, int view, int32_t L, int32_t c) {
  const int32_t t = i % L;
  if (view == VIEW_INTRA) return t;
  if (view == VIEW_SUCC) return t < c - 1 - L ? t + L : c - 1;
  return c - 1;
}

// Programmatic dependent launch: a kernel launched with that attribute may start before its
// predecessor in the stream has ended; grid_wait() returns once the predecessor's writes are
// visible, grid_release() lets the successor start.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Bounded wait of a whole warp. It gives up when its budget runs out (Q1M_ERR_TIMEOUT is then
// latched) or when another warp of the CTA gave up; a range or page fault that some other call
// latched does not stop it.
__device__ __forceinline__ bool pg_wait(uint64_t* bar, uint32_t parity, volatile int* gave_up) {
  bool ok = mbar_try_wait(bar, parity);
  if (!ok) {
    const unsigned long long budget = g_wait_cycles;
    const long long t0 = clock64();
    while (true) {
      if (mbar_try_wait(bar, parity)) { ok = true; break; }
      if (*gave_up) break;
      if ((unsigned long long)(clock64() - t0) > budget) {
        latch_timeout();
        *gave_up = 1;
        break;
      }
    }
  }
  return __all_sync(0xFFFFFFFFu, ok);
}

// Wait of one thread for what the hardware has under way (a copy, an MMA) and ends by itself. Its
// limit is its own: neither a short wait budget nor another warp's giving up may let a CTA end, or
// free its tensor memory, before.
__device__ __forceinline__ void pg_land(uint64_t* bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (clock64() - t0 > 2000000000ll) {
      latch_timeout();
      break;
    }
  }
}

// Page of entry `i` of a table row, -1 when the row has no such entry or the entry is not a page of
// the cache.
__device__ __forceinline__ int32_t pg_entry(const PagedCacheArgs& c, const int32_t* row, int64_t i) {
  if (i >= c.max_len >> c.page_log2) return -1;
  const int32_t page = __ldg(row + i);
  return page < c.n_pages ? page : -1;
}

// The same of a needed page: Q1M_ERR_PAGE is latched when there is none.
__device__ __forceinline__ int32_t pg_page(const PagedCacheArgs& c, const int32_t* row, int64_t i) {
  const int32_t page = pg_entry(c, row, i);
  if (page < 0) latch(Q1M_ERR_PAGE);
  return page;
}

// Length of a sequence. One that its table row cannot hold is cut (Q1M_ERR_PAGE is latched):
// lists and counters are sized by what tables hold.
__device__ __forceinline__ int32_t pg_len(const PagedCacheArgs& c, const int32_t* seq_len, int b) {
  const int32_t len = __ldg(seq_len + b);
  if (len > c.max_len) {
    latch(Q1M_ERR_PAGE);
    return c.max_len;
  }
  return len < 0 ? 0 : len;
}

// ---------------------------------------------------------------------------------------
// Append. Sequence b's new tokens are rows cu[b] .. cu[b+1] of k and v (row b when cu is null)
// and sit at the end of its seq_len[b] positions. Each (token, 16 elements of a head: 8 pairs)
// is one item; a thread loads an item with 16-byte loads of k, v and the table while it rotates
// and stores the one before. The step moves each element once, so it is bound by HBM (large
// batches) or by the chain token -> sequence -> page -> store (small ones): a warp finds the
// sequences of its tokens 32 candidates at a time, then its lanes look up all their pages at
// once, while the block's first loads are in flight. Measured: 32,768 tokens of 8 KV heads, D =
// 128, bf16 (268 MB) 54 us, 0.75 of the copy rate (84 us with one item a thread and no load
// ahead); one token each of 16 sequences 3.3 us.
// ---------------------------------------------------------------------------------------
struct PagedAppendArgs {
  PagedCacheArgs c;
  const void *k, *v;
  int64_t k_stride, v_stride;    // elements between tokens
  int64_t n_tokens;
  const int32_t* cu;             // [batch + 1] or null
  const int32_t* seq_len;        // [batch]
  int32_t batch;
  int32_t d, L;
  const float2* table;
  uint16_t *k_pages, *v_pages;
};

// Sequence of token `row` (cu[b] <= row < cu[b + 1]), found by a whole warp; batch when none.
__device__ __forceinline__ int pg_sequence(const int32_t* cu, int batch, int64_t row) {
  int lo = 0, n = batch;                       // the answer is lo + (entries <= row among cu[lo+1 ..])
  while (n > 0) {
    const int step = (n + 31) / 32;
    const int i = lo + (int)lane_id() * step + step;   // lane's probe: the end of its share
    const bool below = i <= lo + n && (int64_t)__ldg(cu + i) <= row;
    const int k = __popc(__ballot_sync(0xFFFFFFFFu, below));
    const int rest = lo + n - (lo + k * step);
    lo += k * step;
    if (step == 1) break;
    n = rest < step ? rest : step;
  }
  return lo;
}

constexpr int PG_APPEND_THREADS = 256;
constexpr int PG_APPEND_TOKENS = 256;        // of a block at most

// One item's inputs, as loaded.
template <typename T>
struct PgItem {
  static constexpr int W = sizeof(T) / 2;    // 16-byte loads of 8 elements
  uint4 k[2][W], v[2][W];
  float4 cs[4];                              // (cos, sin) of pairs 2q, 2q + 1
  __device__ __forceinline__ void load_kv(const PagedAppendArgs& a, int64_t row, int at) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4* ks = reinterpret_cast<const uint4*>(static_cast<const T*>(a.k) + row * a.k_stride + at + h * (a.d >> 1));
      const uint4* vs = reinterpret_cast<const uint4*>(static_cast<const T*>(a.v) + row * a.v_stride + at + h * (a.d >> 1));
#pragma unroll
      for (int x = 0; x < W; ++x) { k[h][x] = __ldg(ks + x); v[h][x] = __ldg(vs + x); }
    }
  }
  __device__ __forceinline__ void load_table(const PagedAppendArgs& a, int32_t pos, int f0) {
    const float4* t = reinterpret_cast<const float4*>(a.table + (int64_t)pos * (a.d >> 1) + f0);
#pragma unroll
    for (int q = 0; q < 4; ++q) cs[q] = __ldg(t + q);
  }
  static __device__ __forceinline__ void unpack(const uint4* u, float* x) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(u);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      x[i] = W == 2 ? __uint_as_float(w[i]) : __uint_as_float((i & 1) ? (w[i >> 1] & 0xFFFF0000u) : (w[i >> 1] << 16));
  }
};

// Eight values as fp16; `bad` collects what is out of its range, or NaN.
__device__ __forceinline__ uint4 pack8_f16(const float* x, bool& bad) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    bad |= !(fabsf(x[2 * i]) <= 65504.f) || !(fabsf(x[2 * i + 1]) <= 65504.f);
    w[i] = pack_f16x2(x[2 * i], x[2 * i + 1]);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T>
__global__ void __launch_bounds__(PG_APPEND_THREADS)
paged_append_kernel(const PagedAppendArgs a, int units, int tokens) {
  __shared__ int64_t dst_row[PG_APPEND_TOKENS];    // row of KV head 0 in the pages, -1: skipped
  __shared__ int32_t pos_of[PG_APPEND_TOKENS];
  const int64_t t0 = (int64_t)blockIdx.x * tokens;
  const int hd = a.d >> 1, n8 = hd >> 3;
  if (a.n_tokens - t0 < tokens) tokens = (int)(a.n_tokens - t0);
  const int items = tokens * units;
  PgItem<T> ahead;
  if ((int)threadIdx.x < items) {
    const int tl = threadIdx.x / units, u = threadIdx.x - tl * units, g = u / n8;
    ahead.load_kv(a, t0 + tl, g * a.d + (u - g * n8) * 8);
  }
  // cu may be anything: every block looks all of it over before the first store
  bool malformed = false, missing = false;
  if (a.cu != nullptr) {
    malformed = threadIdx.x == 0 && (__ldg(a.cu) != 0 || __ldg(a.cu + a.batch) > a.n_tokens);
    for (int b = threadIdx.x; b < a.batch; b += PG_APPEND_THREADS) malformed |= __ldg(a.cu + b + 1) < __ldg(a.cu + b);
  }
  // the block's tokens, up to 32 a warp
  const int per_warp = (tokens + PG_APPEND_THREADS / 32 - 1) / (PG_APPEND_THREADS / 32);
  {
    const int i0 = warp_id() * per_warp, i1 = min(tokens, i0 + per_warp);
    int b = a.batch;
    if (a.cu == nullptr) {
      b = (int)t0 + i0 + lane_id();
    } else {
      for (int i = i0; i < i1; ++i) {
        const int at = t0 + i < (int64_t)__ldg(a.cu) ? a.batch : pg_sequence(a.cu, a.batch, t0 + i);
        if ((int)lane_id() == i - i0) b = at;
      }
    }
    const int i = i0 + lane_id();
    if (i < i1) {
      int64_t p = -1, dst = -1;
      int32_t pos = 0;
      if (a.cu == nullptr) p = (int64_t)__ldg(a.seq_len + b) - 1;
      else if (b < a.batch) p = (int64_t)__ldg(a.seq_len + b) - ((int64_t)__ldg(a.cu + b + 1) - (t0 + i));
      if (p >= 0) {
        const int32_t page = pg_entry(a.c, a.c.page_table + b * a.c.table_stride, p >> a.c.page_log2);
        const int64_t in_page = p & ((1 << a.c.page_log2) - 1);
        missing = page < 0;
        if (page >= 0) dst = (((int64_t)page * a.c.hkv) << a.c.page_log2) + in_page;
        pos = (int32_t)(p % a.L);
      }
      dst_row[i] = dst;
      pos_of[i] = pos;
    }
  }
  if (__syncthreads_or(malformed)) {
    if (threadIdx.x == 0) latch(Q1M_ERR_INVALID);
    return;
  }
  if (missing) latch(Q1M_ERR_PAGE);
  bool bad = false;
  int it = threadIdx.x;
  if (it < items) {
    const int tl = it / units, u = it - tl * units;
    ahead.load_table(a, pos_of[tl], u % n8 * 8);
  }
  while (it < items) {
    const PgItem<T> x = ahead;
    const int tl = it / units, u = it - tl * units, g = u / n8, f0 = (u - g * n8) * 8;
    it += PG_APPEND_THREADS;
    if (it < items) {
      const int tn = it / units, un = it - tn * units, gn = un / n8, fn = (un - gn * n8) * 8;
      ahead.load_kv(a, t0 + tn, gn * a.d + fn);
      ahead.load_table(a, pos_of[tn], fn);
    }
    if (dst_row[tl] < 0) continue;
    const int64_t dst = (dst_row[tl] + ((int64_t)g << a.c.page_log2)) * a.d + f0;
    float x1[8], x2[8], lo[8], hi[8];
    x.unpack(x.k[0], x1);
    x.unpack(x.k[1], x2);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float2 ca = make_float2(x.cs[q].x, x.cs[q].y), cb = make_float2(x.cs[q].z, x.cs[q].w);
      lo[2 * q] = rot_lo(x1[2 * q], x2[2 * q], ca);
      lo[2 * q + 1] = rot_lo(x1[2 * q + 1], x2[2 * q + 1], cb);
      hi[2 * q] = rot_hi(x1[2 * q], x2[2 * q], ca);
      hi[2 * q + 1] = rot_hi(x1[2 * q + 1], x2[2 * q + 1], cb);
    }
    *reinterpret_cast<uint4*>(a.k_pages + dst) = pack8_f16(lo, bad);
    *reinterpret_cast<uint4*>(a.k_pages + dst + hd) = pack8_f16(hi, bad);
    x.unpack(x.v[0], x1);
    x.unpack(x.v[1], x2);
    *reinterpret_cast<uint4*>(a.v_pages + dst) = pack8_f16(x1, bad);
    *reinterpret_cast<uint4*>(a.v_pages + dst + hd) = pack8_f16(x2, bad);
  }
  if (bad) latch(Q1M_ERR_RANGE);
}

// ---------------------------------------------------------------------------------------
// Decode of a batch. The step reads every visible K/V row once (4 D Hkv bytes a key) for
// about G FLOP per byte, so it is HBM-bound; the contraction runs on mma.sync with the G <= 8
// heads of a KV group as rows 0..7 of the 16-row tile. Rows 8..15 carry what fp16 loses: the
// query views enter as q = hi + lo (rows r and r + 8), the weights as p = hi + lo, and the two
// halves of the accumulators are added, so the products see q and p to about 22 bits at the
// cost of instructions that the padding rows pay for anyway.
//
//  * Work is one flat list of 32-key tiles over (sequence, KV head, visible tile), cut into
//    runs of equal cost, one per persistent CTA: a tile costs one unit and a pair (sequence, KV
//    head) PD_PAIR_COST more, in front of its tiles, for its queries and results. A CTA's run
//    covers at most two cut pairs, at its ends; their partials go to the CTA's two scratch
//    slots and paged_merge_kernel joins them in a fixed order. Pairs inside a run are finished
//    and written by the CTA.
//  * One producer warp keeps PD_STAGES tiles in flight (TMA, 128-byte swizzle), also across
//    pairs: each lane decodes one of the next 32 tiles and looks up its page(s) ahead of use.
//    A stage's turns use two barriers alternately: its consumers change, so a warp may ask for
//    a turn when the one before has not landed, which one barrier's parity could not tell from
//    a completed turn; with two, the turn before on the same barrier has been consumed.
//  * Eight consumer warps take the tiles in turn, each with its own online softmax: HBM brings an
//    SM a tile every 680 cycles, and a warp's chain of dependent steps is longer than that.
//    Nothing holds them together: the last warp to finish its part of a pair joins the parts
//    (in tile order, whoever is last) while the others are at the next pairs, so many short
//    sequences keep all warps busy.
//  * Two warps prepare the query views (rotation, scale, split into hi and lo, laid out as
//    fragments) a few ahead, so that the fetch of a pair's queries delays nobody.
//  * Each tile's product P V is a fresh sum that is added to the warp's total with rounding: the
//    tensor core cuts what it adds to an accumulator towards zero, so a total kept in its
//    accumulator lost 1.0e-4 of the result at 131,000 keys a pair and 1.2e-5 at 16,000 (values of
//    one sign); this way 9e-8, and no slower (128 windowed sequences 119 us, 123 before: half the
//    accumulators, as hi and lo rows are added tile by tile, and no spills).
//  * Rows of a tile that the token does not see (past its end, between sinks and window) are
//    masked in S and zeroed in the V tile: whatever an unwritten page holds meets no product.
//    Pages that hold no visible key are not looked up; TMA fills their rows with zeros.
//
// Measured with the merge, from a captured graph: 131,071 keys of 4 KV heads, D = 128 (268 MB) 54
// us; 1,048,575 keys (2.1 GB) 314 us in pages of 128 (6.9 TB/s) and 341 us in pages of 16 (6.3);
// 128 sequences with 4,096-key windows (670 MB) 120 us, 5.6 TB/s; 48 of 1 .. 32,768 keys (590 MB,
// pages of 16) 116 to 119 us on different boxes. About 3 us pass until a CTA knows its run, 2 more until its first tile
// has landed, and 5 go to the merge.
// ---------------------------------------------------------------------------------------
constexpr int PD_WARPS = 8;                 // consumer warps
constexpr int PD_QUERY_WARPS = 2;
constexpr int PD_THREADS = 32 * (PD_WARPS + PD_QUERY_WARPS + 1);
constexpr int PD_TILE = 32;                 // keys per tile
constexpr int PD_STAGES = 10;
constexpr int PD_QUERIES = 4;               // query views in flight
constexpr int PD_JOINS = 32;                // pairs in flight at most: warps are within 18 tiles of
                                            // one another (each takes every eighth, 10 stages)
// of a (sequence, KV head) pair, in tiles: short pairs that many warps take at once cost about 4,
// ones of a dozen tiles about 9; one value for both, so that mixed batches of many short sequences
// pay for the others (128 windowed sequences: 134, 124, 119 and 119 us at 4, 6, 8 and 9; 48
// sequences of 1 .. 32,768 keys: 110, 113, 118 and 116)
constexpr int PD_PAIR_COST = 8;
constexpr int PD_MIN_UNITS = PD_PAIR_COST + 4;   // of a CTA's run at least
// weights are kept as 2^PD_BIAS p in fp16 (p <= 1), so that its subnormals start at 2^-26
constexpr float PD_BIAS = 12.f;

struct PagedDecodeArgs {
  PagedCacheArgs c;
  const void* q;                // [batch] rows of Hq x D, q_stride elements apart
  int64_t q_stride;
  const int32_t* seq_len;       // [batch]
  int32_t batch, hq, G;
  int32_t window, sinks;        // window 0: every key
  int32_t first_key;            // keys below it are someone else's (the shared prefix)
  int32_t L, chunk;
  float scale;
  const float2* table;
  void* out;                    // [batch][Hq][D]
  float* lse;                   // [Hq][batch] or null
  float* o_part;                // [2 x CTAs][8][D], normalised
  float* lse_part;              // [2 x CTAs][8], log2-sum-exp2
  int4* cut;                    // [CTAs]: the pair whose first cut is the CTA's begin: sequence (-1:
                                // none), KV head, first CTA, CTAs
  // when a prefix part is to be joined to every pair (null otherwise):
  int2* pairs;                  // [batch][Hkv]: first CTA, CTAs (0: no keys here)
  float* o_whole;               // [batch][Hq][D] and [batch][Hq]: results of uncut pairs
  float* lse_whole;
};

// Visible keys of one sequence behind first_key, as 32-key tiles: n_a tiles from first_tile
// (sinks), then tiles lo_tile .. end_tile - 1 (window, or everything).
struct PagedSpan {
  int32_t len, lo, sinks;       // key j is visible iff j < len and (j >= lo or j < sinks)
  int32_t n_a, first_tile, lo_tile, n;
};

__device__ __forceinline__ PagedSpan pd_span(const PagedDecodeArgs& a, int b) {
  PagedSpan s;
  s.len = pg_len(a.c, a.seq_len, b);
  s.lo = a.window > 0 && s.len > a.window ? s.len - a.window : 0;
  s.sinks = a.window > 0 ? (a.sinks < s.lo ? a.sinks : s.lo) : 0;
  const int32_t from = s.lo > a.first_key ? s.lo : a.first_key;
  s.first_tile = a.first_key / PD_TILE;
  s.lo_tile = from / PD_TILE;
  const int32_t end = (s.len + PD_TILE - 1) / PD_TILE;
  const int32_t n_b = end > s.lo_tile ? end - s.lo_tile : 0;
  int32_t a_end = (s.sinks + PD_TILE - 1) / PD_TILE;
  if (a_end > s.lo_tile) a_end = s.lo_tile;
  s.n_a = n_b > 0 && a_end > s.first_tile ? a_end - s.first_tile : 0;
  s.n = s.n_a + n_b;
  return s;
}

__device__ __forceinline__ int32_t pd_tile(const PagedSpan& s, int32_t i) {
  return i < s.n_a ? s.first_tile + i : s.lo_tile + (i - s.n_a);
}

// The run of CTA `c`: units [c T / n, (c + 1) T / n) of the flat list.
struct PagedRuns {
  int64_t total;
  int32_t ctas;
  // a / b, in 32 bits where they fit (a 64-bit division takes over 100 cycles more)
  static __device__ __forceinline__ int64_t div(int64_t a, int64_t b) {
    return ((uint64_t)(a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
  }
  __device__ __forceinline__ int64_t begin(int64_t c) const { return div(c * total, ctas); }
  // the CTA whose run holds unit u
  __device__ __forceinline__ int32_t owner(int64_t u) const {
    return (int32_t)(div((u + 1) * ctas + total - 1, total) - 1);
  }
};

__device__ __forceinline__ PagedRuns pg_runs(int64_t total, int32_t ctas, int32_t min_units) {
  PagedRuns r;
  const int64_t most = PagedRuns::div(total, min_units);
  r.total = total;
  r.ctas = most < 1 ? 1 : (most < ctas ? (int32_t)most : ctas);
  return r;
}

template <int D>
struct PdSmem {
  static constexpr int TILE = PD_TILE * D * 2;
  alignas(1024) uint8_t k[PD_STAGES][TILE];
  alignas(1024) uint8_t v[PD_STAGES][TILE];
  uint4 q[PD_QUERIES][D / 16][32];          // A fragments of each lane
  float o[PD_WARPS][8][D];                  // the warps' parts of a pair
  float m[PD_WARPS][8], l[PD_WARPS][8];
  int32_t before[PG_MAX_BATCH + 1];         // tiles of the sequences before b, per KV head
  int32_t cost[PG_MAX_BATCH + 1];           // and their units
  uint64_t full[PD_STAGES][2], empty[PD_STAGES], q_full[PD_QUERIES], q_empty[PD_QUERIES], o_free[PD_WARPS];
  int32_t warp_sum[PD_THREADS / 32][2];
  int32_t joined[PD_JOINS];                 // parts of a pair that are in place
  int gave_up;
};

static_assert(sizeof(PdSmem<128>) + 1024 <= 227 * 1024, "fits a CTA's shared memory");

// A CTA's share of one pair: tiles o .. o + take - 1 of its run, i0 .. of the pair.
struct PdPiece {
  int b, g, i0, o, take, k;                 // k: number of the piece
  PagedSpan s;
  int32_t intra, succ;                      // first keys of the token's DCA chunk and of the one before
  uint32_t views;                           // bit v: some tile has view v
  __device__ __forceinline__ int32_t key0(int i) const { return pd_tile(s, i0 + i) * PD_TILE; }
  __device__ __forceinline__ int view(int i) const {
    const int32_t j = key0(i);
    return j >= intra ? VIEW_INTRA : (j >= succ ? VIEW_SUCC : VIEW_INTER);
  }
  __device__ __forceinline__ void set(const PagedDecodeArgs& a, int n_mine) {
    take = min(s.n - i0, n_mine - o);
    intra = (s.len - 1) / a.L * a.L;
    succ = intra - a.L;
    // views change towards the token, one by one over neighbouring keys
    const int na = min(max(s.n_a - i0, 0), take);
    views = (na > 0 ? (2u << view(0)) - (1u << view(na - 1)) : 0u) |
            (na < take ? (2u << view(na)) - (1u << view(take - 1)) : 0u);
  }
  __device__ __forceinline__ void next(const PagedDecodeArgs& a, int n_mine) {
    o += take;
    ++k;
    i0 = 0;
    if (o >= n_mine) return;
    if (++g == a.c.hkv) {
      g = 0;
      do { s = pd_span(a, ++b); } while (s.n == 0);
    }
    set(a, n_mine);
  }
};

__device__ __forceinline__ void store4(float* p, const float* y) {
  *reinterpret_cast<float4*>(p) = make_float4(y[0], y[1], y[2], y[3]);
}
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float* y) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
}

__device__ __forceinline__ float2 load2_f32(const __nv_bfloat16* p) {
  const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ float2 load2_f32(const float* p) { return *reinterpret_cast<const float2*>(p); }

// (a, b) = hi + lo in fp16 pairs; `bad` collects what is out of fp16's range, or NaN.
__device__ __forceinline__ void split_f16x2(float a, float b, uint32_t& hi, uint32_t& lo, bool& bad) {
  bad |= !(fabsf(a) <= 65504.f) || !(fabsf(b) <= 65504.f);
  hi = pack_f16x2(a, b);
  const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  lo = pack_f16x2(a - back.x, b - back.y);
}

// A query's heads of one KV group in one view, as a warp loads them and as A fragments
// (row gid = hi, row gid + 8 = lo).
template <typename T, int D>
struct PdQuery {
  static constexpr int KS = D / 16;
  float2 x1[KS], x2[KS];                              // pairs 8 j + 2 tig, + 1
  float4 cs[KS];
  __device__ __forceinline__ void load(const PagedDecodeArgs& a, int b, int g, int32_t pos, int view) {
    const int gid = lane_id() >> 2, tig = lane_id() & 3;
    if (gid >= a.G) return;
    const T* q = static_cast<const T*>(a.q) + (int64_t)b * a.q_stride + (int64_t)(g * a.G + gid) * D + 2 * tig;
    const float2* trow = a.table + (int64_t)dca_query_pos32(pos, view, a.L, a.chunk) * (D / 2) + 2 * tig;
#pragma unroll
    for (int j = 0; j < KS; ++j) {
      x1[j] = load2_f32(q + 8 * j);
      x2[j] = load2_f32(q + 8 * j + D / 2);
      cs[j] = __ldg(reinterpret_cast<const float4*>(trow + 8 * j));
    }
  }
  __device__ __forceinline__ void store(const PagedDecodeArgs& a, uint4 (*dst)[32]) const {
    const bool live = (int)(lane_id() >> 2) < a.G;
    bool bad = false;
#pragma unroll
    for (int kk = 0; kk < KS / 2; ++kk) {
      uint32_t lo[4] = {0u, 0u, 0u, 0u}, hi[4] = {0u, 0u, 0u, 0u};   // dims 16 kk .. and D/2 + 16 kk ..
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int j = 2 * kk + hf;
        const float2 ca = make_float2(cs[j].x, cs[j].y), cb = make_float2(cs[j].z, cs[j].w);
        const float a1 = x1[j].x * a.scale, a2 = x2[j].x * a.scale, b1 = x1[j].y * a.scale, b2 = x2[j].y * a.scale;
        if (live) {
          split_f16x2(rot_lo(a1, a2, ca), rot_lo(b1, b2, cb), lo[2 * hf], lo[2 * hf + 1], bad);
          split_f16x2(rot_hi(a1, a2, ca), rot_hi(b1, b2, cb), hi[2 * hf], hi[2 * hf + 1], bad);
        }
      }
      dst[kk][lane_id()] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      dst[kk + KS / 2][lane_id()] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    }
    if (bad) latch(Q1M_ERR_RANGE);
  }
};

// Joins the parts of a piece that its n warps (from warp o mod PD_WARPS on) left in shared
// memory and writes the result: to the output, or to scratch when the pair is cut or a prefix
// part is still to come.
template <typename TO, int D>
__device__ __forceinline__ void pd_join(PdSmem<D>& sm, const PagedDecodeArgs& a, const PdPiece& p, int n) {
  const int lane = lane_id();
  const bool whole = p.take == p.s.n;
  const int64_t slot = 2 * (int64_t)blockIdx.x + (p.i0 == 0 ? 1 : 0);   // its end or its beginning is cut off
  // the parts' weights, over their maxima: lane 8 r + j has part j of heads r and r + 4
  const int pj = (p.o + (lane & 7)) & (PD_WARPS - 1);
  const bool has = (lane & 7) < n;
#pragma unroll
  for (int r = lane >> 3; r < 8; r += 4) {
    const float m = has ? sm.m[pj][r] : -INFINITY, l = has ? sm.l[pj][r] : 0.f;
    float M = m;
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
    const float f = l == 0.f ? 0.f : (M == -INFINITY ? 1.f : ex2(m - M));   // no maximum: NaN logits
    float L = f * l;
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) L += __shfl_xor_sync(0xFFFFFFFFu, L, o);
    if (has) sm.m[pj][r] = L > 0.f ? f / L : (L == 0.f ? 0.f : L);          // a NaN sum stays one
    if ((lane & 7) == 0 && r < a.G) {
      const float lse2 = L > 0.f ? M + __log2f(L) : (L == 0.f ? -INFINITY : L);
      const int h = p.g * a.G + r;
      if (!whole) a.lse_part[slot * 8 + r] = lse2;
      else if (a.pairs) a.lse_whole[(int64_t)p.b * a.hq + h] = lse2;
      else if (a.lse) a.lse[(int64_t)h * a.batch + p.b] = lse2 * 0.69314718055994531f;
    }
  }
  __syncwarp();
  constexpr int ROWS = 128 / D;                       // heads at a time
  const int d0 = 4 * (lane % (D / 4));
#pragma unroll
  for (int r0 = 0; r0 < 8; r0 += ROWS) {
    const int r = r0 + lane / (D / 4);
    if (r >= a.G) continue;
    float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < PD_WARPS; ++j) {
      if (j >= n) break;
      const int pw = (p.o + j) & (PD_WARPS - 1);
      const float f = sm.m[pw][r];
      const float4 x = *reinterpret_cast<const float4*>(&sm.o[pw][r][d0]);
      y[0] += f * x.x; y[1] += f * x.y; y[2] += f * x.z; y[3] += f * x.w;
    }
    const int64_t at = (int64_t)p.b * a.hq + p.g * a.G + r;
    if (!whole) store4(a.o_part + (slot * 8 + r) * D + d0, y);
    else if (a.pairs) store4(a.o_whole + at * D + d0, y);
    else store4(static_cast<TO*>(a.out) + at * D + d0, y);
  }
}

template <typename T, typename TO, int D>
__global__ void __launch_bounds__(PD_THREADS, 1)
paged_decode_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                    const PagedDecodeArgs a) {
  extern __shared__ uint8_t pd_raw[];
  PdSmem<D>& sm = *reinterpret_cast<PdSmem<D>*>((reinterpret_cast<uintptr_t>(pd_raw) + 1023) & ~uintptr_t(1023));
  constexpr int KS = D / 16, DN = D / 8;
  const int w = warp_id(), lane = lane_id();
  grid_release();                               // what follows may take its place, and waits for this grid
  if (threadIdx.x == 0) {
    sm.gave_up = 0;
    sm.before[0] = sm.cost[0] = 0;
  }
  if (w == 1) {
    if (lane < PD_STAGES) { mbar_init(&sm.full[lane][0], 1); mbar_init(&sm.full[lane][1], 1); mbar_init(&sm.empty[lane], 1); }
    if (lane < PD_QUERIES) { mbar_init(&sm.q_full[lane], 1); mbar_init(&sm.q_empty[lane], PD_WARPS); }
    if (lane < PD_WARPS) mbar_init(&sm.o_free[lane], 1);
    sm.joined[lane] = 0;
    fence_mbar_init();
  }
  // tiles and units before each sequence: every thread takes a contiguous share of the batch
  {
    const int per = (a.batch + PD_THREADS - 1) / PD_THREADS;
    const int b0 = threadIdx.x * per, b1 = min(a.batch, b0 + per);
    int32_t sum = 0, nz = 0;
    for (int b = b0; b < b1; ++b) {
      const int32_t n = pd_span(a, b).n;
      sum += n;
      nz += n > 0;
    }
    int32_t inc = sum, inc_nz = nz;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t y = __shfl_up_sync(0xFFFFFFFFu, inc, o), z = __shfl_up_sync(0xFFFFFFFFu, inc_nz, o);
      if (lane >= o) { inc += y; inc_nz += z; }
    }
    if (lane == 31) { sm.warp_sum[w][0] = inc; sm.warp_sum[w][1] = inc_nz; }
    __syncthreads();
    int32_t run = inc - sum, run_nz = inc_nz - nz;
    for (int i = 0; i < w; ++i) { run += sm.warp_sum[i][0]; run_nz += sm.warp_sum[i][1]; }
    for (int b = b0; b < b1; ++b) {
      const int32_t n = pd_span(a, b).n;
      run += n;
      run_nz += n > 0;
      sm.before[b + 1] = run;
      sm.cost[b + 1] = run + PD_PAIR_COST * run_nz;
    }
    __syncthreads();
  }
  // sequences that see nothing
  for (int b = blockIdx.x; b < a.batch; b += gridDim.x) {
    if (sm.before[b + 1] != sm.before[b]) continue;
    if (a.pairs) {
      for (int g = threadIdx.x; g < a.c.hkv; g += PD_THREADS) a.pairs[(int64_t)b * a.c.hkv + g] = make_int2(0, 0);
    } else {
      const float zero[4] = {0.f, 0.f, 0.f, 0.f};
      for (int i = threadIdx.x; i < a.hq * (D / 4); i += PD_THREADS)
        store4(static_cast<TO*>(a.out) + (int64_t)b * a.hq * D + 4 * i, zero);
      if (a.lse)
        for (int h = threadIdx.x; h < a.hq; h += PD_THREADS) a.lse[(int64_t)h * a.batch + b] = -INFINITY;
    }
  }
  const int64_t hkv = a.c.hkv, total = sm.cost[a.batch] * hkv;
  const PagedRuns R = pg_runs(total, gridDim.x, PD_MIN_UNITS);
  if (total == 0 || (int)blockIdx.x >= R.ctas) {
    if (threadIdx.x == 0) a.cut[blockIdx.x] = make_int4(-1, 0, 0, 0);
    return;
  }
  // the sequence whose part [before[b] hkv, before[b + 1] hkv) of the list holds u
  auto find = [&](const int32_t* before, int64_t u) {
    int lo = 0, hi = a.batch - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (before[mid] * hkv <= u) lo = mid; else hi = mid - 1;
    }
    return lo;
  };
  // the first tile at or behind unit u
  auto tile_at = [&](int64_t u) {
    if (u >= total) return sm.before[a.batch] * hkv;
    const int b = find(sm.cost, u);
    const int32_t n = sm.before[b + 1] - sm.before[b];
    const int64_t rel = u - sm.cost[b] * hkv, g = PagedRuns::div(rel, n + PD_PAIR_COST);
    const int64_t i = rel - g * (n + PD_PAIR_COST) - PD_PAIR_COST;
    return sm.before[b] * hkv + g * n + (i > 0 ? i : 0);
  };
  const int64_t u0 = tile_at(R.begin(blockIdx.x)), u1 = tile_at(R.begin(blockIdx.x + 1));
  const int n_mine = (int)(u1 - u0);            // may be 0: a run of nothing but a pair's cost
  volatile int* gave_up = &sm.gave_up;
  PdPiece p{};
  if (n_mine > 0) {
    p.b = find(sm.before, u0);
    p.s = pd_span(a, p.b);
    const int64_t rel = u0 - sm.before[p.b] * hkv;
    p.g = (int)PagedRuns::div(rel, p.s.n);
    p.i0 = (int)(rel - (int64_t)p.g * p.s.n);
    p.set(a, n_mine);
  }
  // first unit of the piece's pair that is a tile
  auto first_unit = [&](const PdPiece& x) { return sm.cost[x.b] * hkv + (int64_t)x.g * (x.s.n + PD_PAIR_COST) + PD_PAIR_COST; };

  if (w == PD_WARPS) {
    // ---- producer: lane i looks up the pages of tile o + i -------------------------------
    const int lp = a.c.page_log2;
    const int none = (int)(((int64_t)a.c.n_pages * a.c.hkv) << lp);   // a row past the pages: zeros
    auto lookup = [&](int o, int* y) {
      y[0] = y[1] = none;
      if (o >= n_mine) return;
      const int b = find(sm.before, u0 + o);
      const PagedSpan s = pd_span(a, b);
      const int64_t rel = u0 + o - sm.before[b] * hkv;
      const int g = (int)PagedRuns::div(rel, s.n);
      const int32_t key0 = pd_tile(s, (int32_t)(rel - (int64_t)g * s.n)) * PD_TILE;
      const int32_t* row = a.c.page_table + (int64_t)b * a.c.table_stride;
      const int rows = lp == 4 ? 16 : PD_TILE;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int32_t k0 = key0 + h * rows;
        if (h * rows >= PD_TILE || k0 >= s.len || (k0 + rows <= s.lo && k0 >= s.sinks)) continue;
        const int32_t page = pg_page(a.c, row, k0 >> lp);
        if (page >= 0) y[h] = (int)((((int64_t)page * a.c.hkv + g) << lp) + (k0 & ((1 << lp) - 1)));
      }
    };
    int cur[2], nxt[2];
    lookup(lane, nxt);
    bool ok = true;
    int issued = 0;
    for (int o0 = 0; o0 < n_mine && ok; o0 += 32) {
      cur[0] = nxt[0]; cur[1] = nxt[1];
      const int n = min(32, n_mine - o0);
      for (int i = 0; i < n; ++i) {
        const int o = o0 + i, st = o % PD_STAGES;
        if (i == min(n, PD_STAGES) - 1) lookup(o0 + 32 + lane, nxt);   // behind a full ring
        ok = pg_wait(&sm.empty[st], ((o / PD_STAGES) & 1) ^ 1, gave_up);
        if (!ok) break;
        if (lane == i) {
          uint64_t* full = &sm.full[st][(o / PD_STAGES) & 1];
          mbar_expect_tx(full, 2 * PdSmem<D>::TILE);
          tma_load_3d(sm.k[st], &mk, full, 0, cur[0], 0);
          if (lp == 4) tma_load_3d(sm.k[st] + PdSmem<D>::TILE / 2, &mk, full, 0, cur[1], 0);
          tma_load_3d(sm.v[st], &mv, full, 0, cur[0], 0);
          if (lp == 4) tma_load_3d(sm.v[st] + PdSmem<D>::TILE / 2, &mv, full, 0, cur[1], 0);
        }
        __syncwarp();
        issued = o + 1;
      }
    }
    // whoever gave up, the last copies land before the CTA's memory goes
    if (lane < min(issued, PD_STAGES)) {
      const uint32_t o = issued - 1 - lane, turn = o / PD_STAGES;
      pg_land(&sm.full[o % PD_STAGES][turn & 1], (turn >> 1) & 1);
    }
  } else if (w > PD_WARPS) {
    // ---- query views: every PD_QUERY_WARPS-th of the run's (piece, view) list, the loads of
    // the next one issued before this one's turn comes --------------------------------------
    uint32_t e = 0;                               // entries of the list seen so far
    int v = VIEW_INTER + 1;
    auto advance = [&]() {                        // to this warp's next entry
      while (p.o < n_mine) {
        while (--v >= 0) {
          if (!((p.views >> v) & 1u)) continue;
          if (e++ % PD_QUERY_WARPS == (uint32_t)(w - PD_WARPS - 1)) return true;
        }
        p.next(a, n_mine);
        v = VIEW_INTER + 1;
      }
      return false;
    };
    PdQuery<T, D> ahead;
    bool ok = advance();
    if (ok) ahead.load(a, p.b, p.g, p.s.len - 1, v);
    while (ok) {
      const PdQuery<T, D> now = ahead;
      const uint32_t at = e - 1, st = at % PD_QUERIES;
      const bool more = advance();
      if (more) ahead.load(a, p.b, p.g, p.s.len - 1, v);
      if (!pg_wait(&sm.q_empty[st], ((at / PD_QUERIES) & 1) ^ 1, gave_up)) break;
      now.store(a, sm.q[st]);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.q_full[st]);
      ok = more;
    }
  } else {
    // ---- consumers ----------------------------------------------------------------------
    const int gid = lane >> 2, tig = lane & 3;
    // A copy brings the 64-dim halves of a box one after the other, 128 bytes a row, and a tile is
    // one box of 32 rows or two of 16: byte offsets of rows 16 .. 31 and of dims 64 .. 127.
    const uint32_t part = a.c.page_log2 == 4 ? PdSmem<D>::TILE / 2 : 2048, half = a.c.page_log2 == 4 ? 2048 : 4096;
    auto chunk = [&](int r, int c) { return (uint32_t)(c >> 3) * half + sw128_offset((uint32_t)r, (uint32_t)(c & 7)); };
    if (threadIdx.x == 0) {
      int4 cut = make_int4(-1, 0, 0, 0);
      if (n_mine > 0 && p.i0 > 0) {
        const int64_t first = first_unit(p);
        const int c0 = R.owner(first);
        if (c0 + 1 == (int)blockIdx.x) cut = make_int4(p.b, p.g, c0, R.owner(first + p.s.n - 1) - c0 + 1);
      }
      a.cut[blockIdx.x] = cut;
    }
    bool ok = true;
    uint32_t e = 0, joins = 0;
    for (; p.o < n_mine; p.next(a, n_mine)) {
      // which CTAs have parts of the pair: before any wait, so that the merge finds it in any case
      if (a.pairs && threadIdx.x == 0 && p.i0 == 0) {
        const int n_own = p.take == p.s.n ? 1 : R.owner(first_unit(p) + p.s.n - 1) - (int)blockIdx.x + 1;
        a.pairs[(int64_t)p.b * hkv + p.g] = make_int2((int)blockIdx.x, n_own);
      }
      float m_run = -INFINITY, l_run = 0.f;
      float oacc[DN][2];
#pragma unroll
      for (int n = 0; n < DN; ++n) oacc[n][0] = oacc[n][1] = 0.f;
      // tiles o .. o + take - 1 of the run; this warp's are those with index = w modulo PD_WARPS
      int i = (w - p.o) & (PD_WARPS - 1);
      const bool mine = i < p.take;
      for (int v = VIEW_INTER; v >= 0; --v) {
        if (!((p.views >> v) & 1u)) continue;
        uint32_t qa[KS][4];
        const uint32_t qs = e % PD_QUERIES;
        ok = ok && pg_wait(&sm.q_full[qs], (e / PD_QUERIES) & 1, gave_up);
        if (i < p.take) {
#pragma unroll
          for (int kk = 0; kk < KS; ++kk) {
            const uint4 f = sm.q[qs][kk][lane];
            qa[kk][0] = f.x; qa[kk][1] = f.y; qa[kk][2] = f.z; qa[kk][3] = f.w;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.q_empty[qs]);
        ++e;
        for (; ok && i < p.take && p.view(i) == v; i += PD_WARPS) {
          const int st = (p.o + i) % PD_STAGES;
          const int32_t key0 = p.key0(i);
          const uint32_t turn = (uint32_t)(p.o + i) / PD_STAGES;
          ok = pg_wait(&sm.full[st][turn & 1], (turn >> 1) & 1, gave_up);
          if (!ok) break;
          const uint32_t kb = smem_u32(sm.k[st]), vb = smem_u32(sm.v[st]);
          const int j4 = lane >> 3, r8 = lane & 7;
          float sc[4][4];
#pragma unroll
          for (int nt = 0; nt < 4; ++nt) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
#pragma unroll
          for (int kk = 0; kk < KS; ++kk) {
#pragma unroll
            for (int np = 0; np < 2; ++np) {
              uint32_t bf[4];
              ldsm_x4(kb + np * part + chunk(8 * (j4 >> 1) + r8, 2 * kk + (j4 & 1)), bf);
              mma_16816(sc[2 * np], qa[kk], bf[0], bf[1]);
              mma_16816(sc[2 * np + 1], qa[kk], bf[2], bf[3]);
            }
          }
          float x[4][2];
#pragma unroll
          for (int nt = 0; nt < 4; ++nt) { x[nt][0] = sc[nt][0] + sc[nt][2]; x[nt][1] = sc[nt][1] + sc[nt][3]; }
          if (key0 + PD_TILE > p.s.len || (key0 < p.s.lo && key0 + PD_TILE > p.s.sinks)) {
            auto seen = [&](int32_t j) { return j < p.s.len && (j >= p.s.lo || j < p.s.sinks); };
#pragma unroll
            for (int nt = 0; nt < 4; ++nt)
#pragma unroll
              for (int c = 0; c < 2; ++c)
                if (!seen(key0 + 8 * nt + 2 * tig + c)) x[nt][c] = -INFINITY;
            if (!seen(key0 + lane)) {
#pragma unroll
              for (int c = 0; c < D / 8; ++c)
                *reinterpret_cast<uint4*>(sm.v[st] + (lane >> 4) * part + chunk(lane & 15, c)) =
                    make_uint4(0u, 0u, 0u, 0u);
              fence_async_smem();                    // before the stage's next copy
            }
            __syncwarp();
          }
          float mx = fmaxf(fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[1][0], x[1][1])),
                           fmaxf(fmaxf(x[2][0], x[2][1]), fmaxf(x[3][0], x[3][1])));
          mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
          const float m_new = fmaxf(m_run, mx - PD_BIAS);
          const float alpha = m_run == -INFINITY ? 0.f : ex2(m_run - m_new);
          m_run = m_new;
          const float mu = m_new == -INFINITY ? 0.f : m_new;
          float pw[4][2];
          float ps = 0.f;
#pragma unroll
          for (int nt = 0; nt < 4; ++nt) {
            pw[nt][0] = ex2(x[nt][0] - mu);
            pw[nt][1] = ex2(x[nt][1] - mu);
            ps += pw[nt][0] + pw[nt][1];
          }
          l_run = l_run * alpha + ps;               // this thread's columns; summed per row at the end
          uint32_t pa[2][4];
#pragma unroll
          for (int ks = 0; ks < 2; ++ks)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const float p0 = pw[2 * ks + hf][0], p1 = pw[2 * ks + hf][1];
              const uint32_t hi = pack_f16x2(p0, p1);
              const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&hi));
              pa[ks][2 * hf] = hi;
              pa[ks][2 * hf + 1] = pack_f16x2(p0 - back.x, p1 - back.y);
            }
          // a fresh product of the tile, added to the sum of the earlier ones with rounding
#pragma unroll
          for (int dp = 0; dp < DN / 2; ++dp) {
            float t[2][4];
#pragma unroll
            for (int c = 0; c < 4; ++c) t[0][c] = t[1][c] = 0.f;
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
              uint32_t bf[4];
              ldsm_x4_t(vb + ks * part + chunk(8 * (j4 & 1) + r8, 2 * dp + (j4 >> 1)), bf);
              mma_16816(t[0], pa[ks], bf[0], bf[1]);
              mma_16816(t[1], pa[ks], bf[2], bf[3]);
            }
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int c = 0; c < 2; ++c)
                oacc[2 * dp + n][c] = fmaf(oacc[2 * dp + n][c], alpha, t[n][c] + t[n][c + 2]);
          }
          // every lane's reads (and zeroes) of the stage are done: hand it back to the copies
          __syncwarp();
          if (lane == 0) { fence_async_smem(); mbar_arrive(&sm.empty[st]); }
        }
      }
      if (!mine) continue;
      // leave this warp's part; the last of the piece's warps joins them
      float lt = l_run;
      lt += __shfl_xor_sync(0xFFFFFFFFu, lt, 1);
      lt += __shfl_xor_sync(0xFFFFFFFFu, lt, 2);
      if (joins > 0) ok = pg_wait(&sm.o_free[w], (joins - 1) & 1, gave_up) && ok;
      ++joins;
#pragma unroll
      for (int n = 0; n < DN; ++n)
        *reinterpret_cast<float2*>(&sm.o[w][gid][8 * n + 2 * tig]) =
            make_float2(oacc[n][0], oacc[n][1]);
      if (tig == 0) { sm.m[w][gid] = m_run; sm.l[w][gid] = lt; }
      const int n_parts = min(p.take, PD_WARPS);
      __threadfence_block();
      __syncwarp();
      int arrived = 0;
      if (lane == 0) arrived = atomicAdd(&sm.joined[p.k % PD_JOINS], 1);
      arrived = __shfl_sync(0xFFFFFFFFu, arrived, 0);
      if (arrived == n_parts - 1) {
        __threadfence_block();
        if (lane == 0) sm.joined[p.k % PD_JOINS] = 0;
        if (ok) pd_join<TO, D>(sm, a, p, n_parts);
        __syncwarp();
        if (lane < n_parts) mbar_arrive(&sm.o_free[(p.o + lane) & (PD_WARPS - 1)]);
      }
    }
  }
}

// ---------------------------------------------------------------------------------------
// Joins the parts of a decode row: out = sum 2^(lse_x - lse) o_x, in a fixed order. The parts
// are the cut pieces of the pair (in CTA order) and, with a shared prefix, that many prefix
// parts. One block per row; without a prefix only the rows of cut pairs, at most one pair per
// CTA boundary. Its four warps take the parts in turn, 8 loads in flight each.
// ---------------------------------------------------------------------------------------
struct PagedMergeArgs {
  PagedDecodeArgs d;
  int32_t n_prefix, n_last;      // prefix parts of a row, of a row of the last row tile (0: none)
  int32_t n_rt;                  // row tiles of the prefix
  const float* o_prefix;         // [row tiles][Hkv][n_prefix][rows][D]; row of (b, h): b G + h % G
  const float* lse_prefix;
  int32_t prefix_rows;           // rows of a prefix row tile
};

template <typename TO, int D>
__global__ void __launch_bounds__(128)
paged_merge_kernel(const PagedMergeArgs a) {
  constexpr int PER = D / 32;
  __shared__ float so[4][D], sm_[4], sl[4];
  const int w = warp_id(), lane = lane_id();
  int b, g, r, c0, n_own;
  grid_wait();
  if (a.d.pairs) {
    b = blockIdx.x / a.d.hq;
    g = blockIdx.x % a.d.hq / a.d.G;
    r = blockIdx.x % a.d.G;
    const int2 at = a.d.pairs[(int64_t)b * a.d.c.hkv + g];
    c0 = at.x;
    n_own = at.y;
  } else {
    const int4 cut = a.d.cut[blockIdx.x / a.d.G + 1];
    if (cut.x < 0) return;
    b = cut.x;
    g = cut.y;
    r = blockIdx.x % a.d.G;
    c0 = cut.z;
    n_own = cut.w;
  }
  const int h = g * a.d.G + r;
  const int64_t prow = (int64_t)b * a.d.G + r;
  const int64_t pm = a.prefix_rows > 0 ? prow / a.prefix_rows : 0;
  const int n_parts = n_own + (pm + 1 == a.n_rt ? a.n_last : a.n_prefix);
  auto part = [&](int i, const float** o) -> float {
    if (i < n_own) {
      if (n_own == 1) {
        *o = a.d.o_whole + ((int64_t)b * a.d.hq + h) * D;
        return a.d.lse_whole[(int64_t)b * a.d.hq + h];
      }
      const int64_t slot = 2 * (int64_t)(c0 + i) + (i == 0 ? 1 : 0);
      *o = a.d.o_part + (slot * 8 + r) * D;
      return a.d.lse_part[slot * 8 + r];
    }
    const int64_t at = ((pm * a.d.c.hkv + g) * a.n_prefix + (i - n_own)) * a.prefix_rows + prow % a.prefix_rows;
    *o = a.o_prefix + at * D;
    return a.lse_prefix[at];
  };
  float M = -INFINITY, wsum = 0.f, acc[PER];
#pragma unroll
  for (int c = 0; c < PER; ++c) acc[c] = 0.f;
  for (int i0 = w; i0 < n_parts; i0 += 32) {       // 8 parts of this warp at a time
    float ls[8], y[8][PER];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = i0 + 4 * k;
      ls[k] = -INFINITY;
      if (i < n_parts) {
        const float* o;
        ls[k] = part(i, &o);
#pragma unroll
        for (int c = 0; c < PER; ++c) y[k][c] = o[lane + 32 * c];
      }
    }
    float mx = M;
#pragma unroll
    for (int k = 0; k < 8; ++k) mx = fmaxf(mx, ls[k]);
    if (mx == -INFINITY) {
#pragma unroll
      for (int k = 0; k < 8; ++k) if (ls[k] != ls[k]) wsum = ls[k];   // NaN parts stay visible
      continue;
    }
    const float f = M == -INFINITY ? 0.f : ex2(M - mx);
    wsum *= f;
#pragma unroll
    for (int c = 0; c < PER; ++c) acc[c] *= f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (ls[k] == -INFINITY) continue;
      const float wgt = ex2(ls[k] - mx);
      wsum += wgt;
#pragma unroll
      for (int c = 0; c < PER; ++c) acc[c] += wgt * y[k][c];
    }
    M = mx;
  }
#pragma unroll
  for (int c = 0; c < PER; ++c) so[w][lane + 32 * c] = acc[c];
  if (lane == 0) { sm_[w] = M; sl[w] = wsum; }
  __syncthreads();
  M = fmaxf(fmaxf(sm_[0], sm_[1]), fmaxf(sm_[2], sm_[3]));
  for (int d = threadIdx.x; d < D; d += 128) {
    float O = 0.f, Ls = 0.f;
#pragma unroll
    for (int ww = 0; ww < 4; ++ww) {
      const float f = sm_[ww] == -INFINITY ? (sl[ww] == 0.f ? 0.f : sl[ww]) : ex2(sm_[ww] - M);
      Ls += f * sl[ww];
      O += f * so[ww][d];
    }
    const float y = Ls > 0.f ? O / Ls : (Ls == 0.f ? 0.f : Ls);
    TO* out = static_cast<TO*>(a.d.out) + ((int64_t)b * a.d.hq + h) * D + d;
    if constexpr (sizeof(TO) == 2) *out = __float2bfloat16_rn(y);
    else *out = y;
    if (d == 0 && a.d.lse)
      a.d.lse[(int64_t)h * a.d.batch + b] =
          (Ls > 0.f ? M + __log2f(Ls) : (Ls == 0.f ? -INFINITY : Ls)) * 0.69314718055994531f;
  }
}

}  // namespace q1m
