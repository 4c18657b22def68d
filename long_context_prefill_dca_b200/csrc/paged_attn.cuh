// paged_attn.cuh — DCA attention of many query rows over the paged cache on the 5th-generation
// tensor cores: the prompts of a ragged batch (causal, all keys or a sliding window with
// sinks), and the query tokens of a whole batch over a prefix that they share.
//
// Rows are packed: row R of a KV head is query token R / G and head R % G of the group, so a
// key tile serves the G heads of a token at once and short prompts still fill the 128 lanes of
// an accumulator. A row tile holds up to 256 rows (two 128-row "slots"); every slot streams
// the row tile's key tiles of 128 positions:
//
//  * Work is a flat list of (KV head, row tile, key tile), cut into runs of equal cost, one per
//    persistent CTA, so ragged batches, few long rows and many short ones all fill the GPU. A
//    row tile costs PA_ROW_COST units in front of its key tiles, for its queries and results.
//    A row tile that a run boundary cuts leaves partials that paged_attn_merge_kernel joins in
//    a fixed order; uncut ones are written directly. For a shared prefix every row tile is cut
//    into as many equal key ranges, a last one of at most 128 rows into half as many, and the
//    decode's merge joins them; the ranges of all row tiles run at the same time, so K/V come
//    from HBM about once.
//  * A row tile of at most 128 rows would leave slot 1 idle; its key tiles then alternate
//    between the slots, which hold the same rows, and the two results are joined through
//    shared memory.
//  * Each row has its own position: its DCA view (same chunk, chunk before, older) of a key
//    tile follows from the two chunk numbers, and its mask (causal, window, sinks) is two
//    bounds and a count. The softmax warps rotate their rows into shared memory in the view
//    of the current key chunk, again when the stream enters another chunk; no rotated query
//    goes through HBM.
//  * Warp roles, tensor memory and the issue order are those of block_sparse_attn_kernel:
//    warps 0-3 / 4-7 softmax of slot 0 / 1 (one row per thread), warp 8 loads K, warp 9
//    issues tcgen05.mma, warp 10 loads V; P is written as fp16 over S. What bounds it is the
//    same chain too (QK^T, softmax, PV of a slot): about 4,400 cycles a key tile of two slots at
//    D = 128, of which the tensor pipe and the multi-function unit are busy 2,050 each.
//  * 32-bit outputs (PREC): q and P enter the products as hi + lo fp16 pairs (slot 1's query
//    buffer holds the low parts, P's low parts follow the high ones in S's columns), twice the
//    MMAs on one slot, whose products are summed tile by tile: 3e-7 to 6e-7 off 64 bits.
//
// Measured (captured graph, G = 7, D = 128, bf16): 1,000 tokens over 32,700 keys 443 us, 1.04
// PFLOP/s; 16,384 tokens with a 4,096-key window 1,084 us, 0.90; with 32-bit outputs 1,113 and 2,752
// us. Behind 262,144 shared keys (537 MB) 8 sequences take this kernel 100 us, 5.4 TB/s, and the
// call, with their own keys (22 us) and the merge (6 us) around it, 120 to 126; with 32-bit outputs
// the call takes 200.
#pragma once

#include "paged.cuh"

namespace q1m {

constexpr int PA_NK = 2, PA_NV = 2;
constexpr int PA_THREADS = 384;
constexpr int PA_REGS_SOFTMAX = 192, PA_REGS_OTHER = 120;   // 384 x 168 = 256 x 192 + 128 x 120
constexpr float PA_RESCALE_THRESHOLD = 8.0f;
// weights are held as 2^PA_BIAS p in fp16: with the lazy rescale at most 2^15 < 65504, and
// subnormals start 2^-21 below the running maximum
constexpr float PA_BIAS = 7.0f;
// units of a key tile, of one whose row tile uses both slots in turn, and of a row tile
constexpr int PA_TILE_COST = 5, PA_LIGHT_COST = 3, PA_ROW_COST = 18;
constexpr int PA_MIN_UNITS = 25;

// Rows of a row tile: with PREC one slot's.
__host__ __device__ constexpr int pa_rows(bool prec) { return prec ? 128 : 256; }

// A prompt's row tile and the key tiles that some of its rows sees.
struct PagedRowTile {
  int32_t b, row0, nrows, tok0;   // sequence, first packed row, rows, first query token
  int32_t pos0, len;              // position of query token tok0 (may be negative), keys
  int32_t n, n_a, lo_tile;        // key tiles: n_a sink tiles, then lo_tile ..
  int32_t w;                      // units of a key tile
};

// A row tile that the begin of a CTA's run is the first to cut (nrows 0: none): its parts are
// those of CTAs c0 .. c1.
struct PagedRowCut {
  int32_t row0, nrows, tok0, g, c0, c1;
};

struct PagedAttnArgs {
  PagedCacheArgs c;
  const void* q;
  int64_t q_stride, n_tokens;
  int32_t q_f32;
  const int32_t* cu;             // prompts: [batch + 1]; null: shared prefix
  const int32_t* seq_len;        // [batch]
  int32_t batch, hq, G;
  int32_t window, sinks, L, chunk;
  float scale;
  const float2* table;
  const uint16_t* v_pages;
  void* out;                     // [n_tokens][Hq][D]
  float* lse;                    // [Hq][n_tokens] or null
  float* o_part;                 // [parts][rows of a row tile][D], normalised
  float* lse_part;               // [parts][rows of a row tile], log2
  PagedRowCut* cut;              // [CTAs]: prompts
  int32_t n_split, last_split, n_rt, prefix_tiles;   // shared prefix: key ranges of a row tile, of the last
};

// ---------------------------------------------------------------------------------------
// Plan of a ragged batch: every CTA counts the row tiles, their key tiles and units, and finds
// its run. (n_rt / 384 row tiles a thread: microseconds next to their attention, and cheaper
// than a kernel of its own in front.)
// ---------------------------------------------------------------------------------------
struct PaPlan {
  int32_t first_rt[PG_MAX_BATCH + 1];   // row tiles of the sequences before b
  int64_t sums[PA_THREADS / 32][2];
  int64_t at[2], before;                // tiles of the list before the run's ends; units before its first row tile
  int32_t n_rt, g, rt, i0, n;           // the run: its first KV head, row tile and tile, its tiles
};

// Row tile rt, of sequence b.
__device__ __forceinline__ PagedRowTile pa_row_tile(const PagedAttnArgs& a, const int32_t* first_rt, int b, int rt, int rows) {
  PagedRowTile t;
  t.b = b;
  t.tok0 = __ldg(a.cu + b);
  const int nq = __ldg(a.cu + b + 1) - t.tok0;
  t.len = pg_len(a.c, a.seq_len, b);
  t.row0 = (rt - first_rt[b]) * rows;
  const int64_t left = (int64_t)nq * a.G - t.row0;
  t.nrows = left < rows ? (int)left : rows;
  t.pos0 = t.len - nq;
  const int p0 = t.pos0 + t.row0 / a.G, p1 = t.pos0 + (t.row0 + t.nrows - 1) / a.G;
  const int from = a.window > 0 && p0 >= a.window ? p0 - a.window + 1 : 0;
  t.lo_tile = from / 128;
  const int end = p1 < 0 ? 0 : p1 / 128;
  const int sink = a.window > 0 ? (min(a.sinks, from) + 127) / 128 : 0;
  t.n_a = sink < t.lo_tile ? sink : t.lo_tile;
  t.n = t.n_a + (end - t.lo_tile + 1);        // a row tile without visible keys keeps one tile
  t.w = rows > 128 && t.nrows <= 128 ? PA_LIGHT_COST : PA_TILE_COST;
  return t;
}

// Sums of x and y over the threads before this one, and over all.
__device__ __forceinline__ void pa_scan(int64_t (*sums)[2], int64_t& x, int64_t& y, int64_t& all_x, int64_t& all_y) {
  const int64_t x0 = x, y0 = y;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xFFFFFFFFu, x, o), v = __shfl_up_sync(0xFFFFFFFFu, y, o);
    if ((int)lane_id() >= o) { x += u; y += v; }
  }
  if (lane_id() == 31) { sums[warp_id()][0] = x; sums[warp_id()][1] = y; }
  x -= x0;
  y -= y0;
  __syncthreads();
  all_x = all_y = 0;
#pragma unroll
  for (int i = 0; i < PA_THREADS / 32; ++i) {
    if (i < (int)warp_id()) { x += sums[i][0]; y += sums[i][1]; }
    all_x += sums[i][0];
    all_y += sums[i][1];
  }
  __syncthreads();
}

__device__ __forceinline__ void pa_plan(PaPlan& P, const PagedAttnArgs& a, int rows) {
  const int tid = threadIdx.x, c = blockIdx.x;
  // cu may be anything: nothing else is read through it before it is known to be sound
  const int per_b = (a.batch + PA_THREADS - 1) / PA_THREADS, b0 = tid * per_b, b1 = min(a.batch, b0 + per_b);
  auto count = [&](int b) { return ((int64_t)(__ldg(a.cu + b + 1) - (int64_t)__ldg(a.cu + b)) * a.G + rows - 1) / rows; };
  bool bad = tid == 0 && (__ldg(a.cu) != 0 || __ldg(a.cu + a.batch) > a.n_tokens);
  int64_t mine = 0, none = 0, n_rt, x;
  for (int b = b0; b < b1; ++b) {
    bad |= __ldg(a.cu + b + 1) < __ldg(a.cu + b);
    mine += count(b);
  }
  if (__syncthreads_or(bad)) {
    if (tid == 0) {
      latch(Q1M_ERR_INVALID);
      P.n = 0;
      a.cut[c].nrows = 0;
    }
    __syncthreads();
    return;
  }
  pa_scan(P.sums, mine, none, n_rt, x);
  for (int b = b0; b < b1; ++b) { P.first_rt[b] = (int)mine; mine += count(b); }
  if (tid == 0) { P.first_rt[a.batch] = P.n_rt = (int)n_rt; P.n = 0; P.i0 = 0; }
  __syncthreads();
  const int per = (int)((n_rt + PA_THREADS - 1) / PA_THREADS), r0 = min((int)n_rt, tid * per), r1 = min((int)n_rt, r0 + per);
  int first_b = 0;
  if (r0 < r1) {
    int hi = a.batch - 1;
    while (first_b < hi) {
      const int mid = (first_b + hi + 1) >> 1;
      if (P.first_rt[mid] <= r0) first_b = mid; else hi = mid - 1;
    }
  }
  int64_t units = 0, tiles = 0, total, all_tiles;
  for (int rt = r0, b = first_b; rt < r1; ++rt) {
    while (rt >= P.first_rt[b + 1]) ++b;
    const PagedRowTile t = pa_row_tile(a, P.first_rt, b, rt, rows);
    tiles += t.n;
    units += PA_ROW_COST + (int64_t)t.n * t.w;
  }
  const int64_t own = units;
  pa_scan(P.sums, units, tiles, total, all_tiles);
  const PagedRuns R = pg_runs(total * a.c.hkv, gridDim.x, PA_MIN_UNITS);
  if (total == 0 || c >= R.ctas) {
    if (tid == 0) a.cut[c].nrows = 0;
    __syncthreads();
    return;
  }
  // the first tile at or behind each end of the run, found by the thread whose share holds it
#pragma unroll 1
  for (int k = 0; k < 2; ++k) {
    const int64_t u = R.begin(c + k);
    int g = (int)PagedRuns::div(u, total);
    const int64_t rel = u - g * total;
    if (g >= a.c.hkv) {
      if (tid == 0) P.at[k] = all_tiles * a.c.hkv;
    } else if (rel >= units && rel < units + own) {
      int64_t before = units, seen = tiles;
      for (int rt = r0, b = first_b; rt < r1; ++rt) {
        while (rt >= P.first_rt[b + 1]) ++b;
        const PagedRowTile t = pa_row_tile(a, P.first_rt, b, rt, rows);
        const int64_t cost = PA_ROW_COST + (int64_t)t.n * t.w;
        if (rel < before + cost) {
          const int64_t in = rel - before - PA_ROW_COST;
          int i0 = in > 0 ? (int)((in + t.w - 1) / t.w) : 0;
          P.at[k] = all_tiles * g + seen + i0;
          if (k == 0) {
            if (i0 == t.n) {                         // behind its last tile
              i0 = 0;
              if (++rt == n_rt) { rt = 0; ++g; }
            }
            P.g = g; P.rt = rt; P.i0 = i0; P.before = before;
          }
          break;
        }
        before += cost;
        seen += t.n;
      }
    }
  }
  __syncthreads();
  if (tid == 0) {
    P.n = (int)(P.at[1] - P.at[0]);
    PagedRowCut cut{};
    if (P.n > 0 && P.i0 > 0) {
      int b = 0, hi = a.batch - 1;
      while (b < hi) {
        const int mid = (b + hi + 1) >> 1;
        if (P.first_rt[mid] <= P.rt) b = mid; else hi = mid - 1;
      }
      const PagedRowTile t = pa_row_tile(a, P.first_rt, b, P.rt, rows);
      const int64_t first = P.g * total + P.before + PA_ROW_COST;
      const int c0 = R.owner(first);
      if (c0 == c - 1) cut = {t.row0, t.nrows, t.tok0, P.g, c0, R.owner(first + (int64_t)(t.n - 1) * t.w)};
    }
    a.cut[c] = cut;
  }
  __syncthreads();
}

// ---------------------------------------------------------------------------------------
// A CTA's pieces, in the order that every warp role walks them.
// ---------------------------------------------------------------------------------------
struct PaItem {
  int b, g, row0, nrows, tok0, pos0, len;
  int n_a, lo_tile, i0, take;
  int p_first, p_last;    // positions of the first and last row (prompts)
  int64_t part;           // partial slot, -1: written directly
  __device__ __forceinline__ int tile(int i) const {
    i += i0;
    return i < n_a ? i : lo_tile + (i - n_a);
  }
};

struct PaWalk {
  int g, rt, i0, left, b, done;   // done: items of a shared prefix
  __device__ __forceinline__ void init(const PagedAttnArgs& a, const PaPlan& P) {
    done = 0;
    if (a.cu) {
      g = P.g; rt = P.rt; i0 = P.i0; left = P.n;
      int lo = 0, hi = a.batch - 1;
      while (left > 0 && lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (P.first_rt[mid] <= rt) lo = mid; else hi = mid - 1;
      }
      b = lo;
    } else {
      g = rt = i0 = b = 0;
      left = a.c.hkv * (a.n_split * (a.n_rt - 1) + a.last_split);
    }
  }
  __device__ __forceinline__ bool next(const PagedAttnArgs& a, const PaPlan& P, int rows, PaItem& it) {
    if (a.cu) {
      if (left <= 0) return false;
      while (rt >= P.first_rt[b + 1]) ++b;
      const PagedRowTile t = pa_row_tile(a, P.first_rt, b, rt, rows);
      it.b = t.b; it.g = g; it.row0 = t.row0; it.nrows = t.nrows; it.tok0 = t.tok0; it.pos0 = t.pos0;
      it.len = t.len;
      it.n_a = t.n_a; it.lo_tile = t.lo_tile; it.i0 = i0;
      it.take = min(left, t.n - i0);
      it.p_first = t.pos0 + t.row0 / a.G;
      it.p_last = t.pos0 + (t.row0 + t.nrows - 1) / a.G;
      it.part = it.take == t.n ? -1 : 2 * (int64_t)blockIdx.x + (i0 == 0 ? 1 : 0);   // its end or its beginning is cut off
      left -= it.take;
      i0 = 0;
      if (++rt == P.n_rt) { rt = b = 0; ++g; }
      return true;
    }
    const int idx = blockIdx.x + done * gridDim.x;
    if (idx >= left) return false;
    ++done;
    const int full = a.n_split * (a.n_rt - 1), per = full + a.last_split;
    const int rel = idx % per, m = rel < full ? rel / a.n_split : a.n_rt - 1;
    const int s = rel - m * a.n_split, n = rel < full ? a.n_split : a.last_split;
    it.g = idx / per;
    it.b = 0; it.tok0 = 0; it.pos0 = 0;
    it.len = a.prefix_tiles * 128;
    it.row0 = m * rows;
    it.nrows = min(rows, a.batch * a.G - it.row0);
    it.n_a = 0; it.lo_tile = 0;
    it.i0 = (int)((int64_t)s * a.prefix_tiles / n);
    it.take = (int)((int64_t)(s + 1) * a.prefix_tiles / n) - it.i0;
    it.p_first = 0; it.p_last = it.len - 1;
    it.part = ((int64_t)m * a.c.hkv + it.g) * a.n_split + s;
    return true;
  }
};

// A warp's next piece, into shared memory; false when there is none.
__device__ __forceinline__ bool pa_advance(const PagedAttnArgs& a, const PaPlan& P, int rows, PaWalk* walk, PaItem* it) {
  __syncwarp();
  int more = 0;
  if (lane_id() == 0) {
    PaWalk w = *walk;
    PaItem n;
    more = w.next(a, P, rows, n);
    *walk = w;
    if (more) *it = n;
  }
  __syncwarp();
  return __shfl_sync(0xFFFFFFFFu, more, 0) != 0;
}

// First tile behind `tile` whose DCA chunk gives a row another view of its query. Chunks older
// than every row's predecessor chunk all take the last view (prompts; for a shared prefix the
// rows' chunks are not known here and each chunk counts).
__device__ __forceinline__ int pa_view_end(const PagedAttnArgs& a, const PaItem& it, int tile) {
  const int lt = a.L / 128, ck = tile / lt;
  const int oldest = a.cu ? (it.p_first > 0 ? it.p_first / a.L : 0) - 2 : -2;
  return ((ck > oldest ? ck : oldest) + 1) * lt;
}

template <int D>
struct PaSmem {
  static constexpr int TILE = 128 * D * 2;
  alignas(1024) uint8_t q[2][TILE];         // slots' queries; the exchange of joined slots
  alignas(1024) uint8_t k[PA_NK][TILE];
  alignas(1024) uint8_t v[PA_NV][TILE];
  uint64_t k_full[PA_NK], k_empty[PA_NK], v_full[PA_NV], v_empty[PA_NV];
  uint64_t q_full[2], s_full[2], p_full[2], o_done[2], pv_done[2];
  uint64_t drain;
  float slot_lse[128];
  PaItem piece[10][2];                      // of each softmax warp and the MMA warp: the piece at hand
  PaWalk walk[10];                          // and the one before or behind it
  PaPlan plan;
  uint32_t tmem_base;
  int gave_up;
};

// ---------------------------------------------------------------------------------------
// Loaders: ROLE 0 streams K tiles, ROLE 1 V tiles. One lane per (page of the tile, 64-dim
// half) issues its TMA copy; pages without a visible key are not looked up and come as zeros.
// The V rows past the sequence's end, where a page may hold anything, are zeroed: that tile is
// copied row by row.
// ---------------------------------------------------------------------------------------
__device__ __forceinline__ void cp_async16_or_zero(void* dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}

template <int D, int ROLE>
__device__ void pa_loader(PaSmem<D>& sm, const PagedAttnArgs& a, const CUtensorMap* map, int rows) {
  constexpr int NS = ROLE == 0 ? PA_NK : PA_NV;
  uint64_t* full = ROLE == 0 ? sm.k_full : sm.v_full;
  uint64_t* empty = ROLE == 0 ? sm.k_empty : sm.v_empty;
  volatile int* gave_up = &sm.gave_up;
  const int lp = a.c.page_log2, ps = 1 << lp, npg = 128 >> lp;
  const int lane = lane_id();
  const int pg = lane & (npg - 1), hf = lane >> (7 - lp);
  const bool issuer = hf < D / 64;
  const int none = (int)(((int64_t)a.c.n_pages * a.c.hkv) << lp);
  PaWalk walk;
  walk.init(a, sm.plan);
  PaItem it;
  uint32_t kt = 0;
  bool ok = true;
  while (ok && walk.next(a, sm.plan, rows, it)) {
    const int32_t* row = a.c.page_table + (int64_t)it.b * a.c.table_stride;
    const int lo = a.window > 0 && it.p_first >= a.window ? it.p_first - a.window + 1 : 0;
    const int sinks = a.window > 0 ? a.sinks : 0;
    // this lane's page of a tile: its table entry is fetched one tile ahead and looked at when
    // the tile's turn comes, so that the fetch overlaps the wait for a free stage
    auto needed = [&](int key0) {
      const int k0 = key0 + (pg << lp);
      return issuer && k0 <= it.p_last && (k0 + ps > lo || k0 < sinks);
    };
    auto entry = [&](int key0) {
      const int i = (key0 >> lp) + pg;
      return needed(key0) ? __ldg(row + i) : -1;       // a visible key lies within the table (pg_len)
    };
    int32_t page = entry(it.tile(0) * 128);
    for (int i = 0; i < it.take; ++i, ++kt) {
      const int key0 = it.tile(i) * 128;
      const int32_t page_next = i + 1 < it.take ? entry(it.tile(i + 1) * 128) : -1;
      const int st = kt % NS;
      ok = pg_wait(&empty[st], ((kt / NS) & 1) ^ 1, gave_up);
      if (!ok) break;
      uint8_t* dst = ROLE == 0 ? sm.k[st] : sm.v[st];
      if (ROLE == 1 && key0 + 128 > it.len && (it.len & (ps - 1)) != 0) {
        for (int r = lane; r < 128; r += 32) {
          const int j = key0 + r;
          const uint16_t* src = a.v_pages;
          bool valid = j < it.len && !(j > it.p_last) && (j >= lo || j < sinks);
          if (valid) {
            const int32_t page = pg_page(a.c, row, j >> lp);
            valid = page >= 0;
            if (valid) src += ((((int64_t)page * a.c.hkv + it.g) << lp) + (j & (ps - 1))) * D;
          }
#pragma unroll
          for (int c = 0; c < D / 8; ++c)
            cp_async16_or_zero(dst + (c >> 3) * 16384 + sw128_offset((uint32_t)r, (uint32_t)(c & 7)),
                               valid ? src + c * 8 : src, valid);
        }
        cp_async_wait_all();
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[st]);
      } else {
        if (lane == 0) mbar_expect_tx(&full[st], PaSmem<D>::TILE);
        __syncwarp();
        int y = none;
        if (needed(key0)) {
          if (page >= 0 && page < a.c.n_pages) y = (int)(((int64_t)page * a.c.hkv + it.g) << lp);
          else latch(Q1M_ERR_PAGE);
        }
        if (issuer) tma_load_2d(dst + hf * 16384 + (pg << lp) * 128, map, &full[st], 64 * hf, y);
      }
      page = page_next;
    }
  }
  // whoever gave up, the last copies land before the CTA's memory goes (kt: tiles issued)
  if (lane < min((int)kt, NS)) pg_land(&full[(kt - 1 - lane) % NS], ((kt - 1 - lane) / NS) & 1);
}

// ---------------------------------------------------------------------------------------
// MMA warp.
// ---------------------------------------------------------------------------------------
struct PaSlot {
  int pend_v = -1;            // V stage of the slot's pending PV (-1: none)
  uint32_t pend_kt = 0;
  bool pend_last = false;     // it is the slot's last tile of the piece
  bool o_started = false;
  uint32_t qn = 0, pn = 0, pvd_issued = 0, pvd_waited = 0;
  int view_end = INT32_MIN;   // first tile that needs other queries than the staged ones
};

struct PaDesc {
  uint64_t q[2], k[PA_NK], v[PA_NV];
  __device__ __forceinline__ uint64_t kd(int st) const { return st ? k[1] : k[0]; }
  __device__ __forceinline__ uint64_t vd(int st) const { return st ? v[1] : v[0]; }
};
static_assert(PA_NK == 2 && PA_NV == 2, "two stages of each");

// Column of the accumulator of PV number n (PREC).
__device__ __forceinline__ uint32_t pa_turn(uint32_t n) { return n & 1 ? 384u : 128u; }

template <int D, bool PREC, int S>
__device__ __forceinline__ bool pa_pv(PaSmem<D>& sm, const PaDesc& dsc, PaSlot& sl, uint32_t tb, uint32_t& v_users) {
  constexpr uint32_t IDESC_PV = idesc_f16(128, D, 1);
  volatile int* gave_up = &sm.gave_up;
  if (!pg_wait(&sm.p_full[S], sl.pn & 1, gave_up)) return false;
  ++sl.pn;
  const int vst = sl.pend_v;
  if (!pg_wait(&sm.v_full[vst], (sl.pend_kt / PA_NV) & 1, gave_up)) return false;
  tc_fence_after();
  // with PREC every PV is a fresh sum, in two accumulators by turns
  const uint32_t p_t = tb + 256u * S, o_t = PREC ? tb + pa_turn(sl.pn - 1) : p_t + 128u;
  const uint64_t vd = dsc.vd(vst);
  const uint32_t sh = 4u * (uint32_t)vst;
  const uint32_t u = ((v_users >> sh) & 0xFu) - 1u;
  if (elect_one()) {
    if (PREC) {   // the low halves first, while the accumulator is small
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) mma_ts(o_t, p_t + 64u + kk * 8u, vd + (uint64_t)(kk * 128), IDESC_PV, kk > 0 ? 1u : 0u);
    }
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)
      mma_ts(o_t, p_t + kk * 8u, vd + (uint64_t)(kk * 128), IDESC_PV, (PREC || sl.o_started || kk > 0) ? 1u : 0u);
    mma_commit(&sm.pv_done[S]);      // P lives in S: the slot's next QK^T waits for this
    if (sl.pend_last) mma_commit(&sm.o_done[S]);
    if (u == 0) mma_commit(&sm.v_empty[vst]);
  }
  __syncwarp();
  sl.o_started = !sl.pend_last;
  ++sl.pvd_issued;
  v_users = (v_users & ~(0xFu << sh)) | (u << sh);
  sl.pend_v = -1;
  return true;
}

template <int D, bool PREC, int S>
__device__ __forceinline__ bool pa_qk(PaSmem<D>& sm, const PagedAttnArgs& a, const PaItem& it, const PaDesc& dsc,
                                      PaSlot& sl, int tile, bool last, int kst, int vst, uint32_t kt, uint32_t tb) {
  constexpr uint32_t IDESC_QK = idesc_f16(128, 128, 0);
  volatile int* gave_up = &sm.gave_up;
  if (tile >= sl.view_end) {
    if (!pg_wait(&sm.q_full[S], sl.qn & 1, gave_up)) return false;
    ++sl.qn;
    sl.view_end = pa_view_end(a, it, tile);
    tc_fence_after();
  }
  if (sl.pvd_waited < sl.pvd_issued) {
    if (!pg_wait(&sm.pv_done[S], sl.pvd_waited & 1, gave_up)) return false;
    ++sl.pvd_waited;
    tc_fence_after();
  }
  const uint32_t s_t = tb + 256u * S;
  const uint64_t qd = dsc.q[S], kd = dsc.kd(kst);
  if (elect_one()) {
    if (PREC) {   // the low halves first, while the accumulator is small
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint64_t off = (uint64_t)((kk >> 2) * 1024 + (kk & 3) * 2);
        mma_ss(s_t, dsc.q[1] + off, kd + off, IDESC_QK, kk > 0 ? 1u : 0u);
      }
    }
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      const uint64_t off = (uint64_t)((kk >> 2) * 1024 + (kk & 3) * 2);
      mma_ss(s_t, qd + off, kd + off, IDESC_QK, PREC || kk > 0 ? 1u : 0u);
    }
    mma_commit(&sm.s_full[S]);
  }
  __syncwarp();
  sl.pend_v = vst;
  sl.pend_kt = kt;
  sl.pend_last = last;
  return true;
}

template <int D, bool PREC>
__device__ void pa_mma(PaSmem<D>& sm, const PagedAttnArgs& a) {
  const uint32_t tb = sm.tmem_base;
  volatile int* gave_up = &sm.gave_up;
  PaDesc dsc;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    dsc.q[i] = sdesc_sw128(smem_u32(sm.q[i]), 16u, 1024u);
    dsc.k[i] = sdesc_sw128(smem_u32(sm.k[i]), 16u, 1024u);
    dsc.v[i] = sdesc_sw128(smem_u32(sm.v[i]), 16384u, 1024u);
  }
  PaItem* const piece = sm.piece[warp_id()];
  PaWalk* const walk = &sm.walk[warp_id()];
  if (lane_id() == 0) walk->init(a, sm.plan);
  PaSlot s0, s1;
  uint32_t v_users = 0, kt = 0;
  bool ok = true;
  int cur = 0;
  bool have = pa_advance(a, sm.plan, pa_rows(PREC), walk, &piece[0]);
  while (have && ok) {
    const PaItem& it = piece[cur];
    const int take = it.take;
    const bool alt = !PREC && it.nrows <= 128;
    s0.view_end = s1.view_end = INT32_MIN;
    for (int i = 0; i < take && ok; ++i, ++kt) {
      const int kst = kt % PA_NK, vst = kt % PA_NV;
      const bool u0 = !alt || !(i & 1), u1 = alt ? (i & 1) : !PREC;
      const bool last = i + (alt ? 2 : 1) >= take;
      const int tile = it.tile(i);
      if (u0 && s0.pend_v >= 0) ok = pa_pv<D, PREC, 0>(sm, dsc, s0, tb, v_users);
      if (!ok) break;
      if (alt && u1 && s1.pend_v >= 0) ok = pa_pv<D, PREC, 1>(sm, dsc, s1, tb, v_users);
      if (!ok) break;
      ok = pg_wait(&sm.k_full[kst], (kt / PA_NK) & 1, gave_up);
      if (!ok) break;
      tc_fence_after();
      const uint32_t sh = 4u * (uint32_t)vst;
      v_users = (v_users & ~(0xFu << sh)) | ((uint32_t)(u0 + u1) << sh);
      if (u0) ok = pa_qk<D, PREC, 0>(sm, a, it, dsc, s0, tile, last, kst, vst, kt, tb);
      if (ok && !alt && u1 && s1.pend_v >= 0) ok = pa_pv<D, PREC, 1>(sm, dsc, s1, tb, v_users);
      if (ok && u1) ok = pa_qk<D, PREC, 1>(sm, a, it, dsc, s1, tile, last, kst, vst, kt, tb);
      if (!ok) break;
      if (elect_one()) mma_commit(&sm.k_empty[kst]);
      __syncwarp();
    }
    cur ^= 1;
    have = pa_advance(a, sm.plan, pa_rows(PREC), walk, &piece[cur]);
    // the last PVs ride behind the next piece's first QK^T unless the slots are joined or the
    // next piece uses them in turn
    if (ok && (alt || !have || (!PREC && piece[cur].nrows <= 128))) {
      if (s0.pend_v >= 0) ok = pa_pv<D, PREC, 0>(sm, dsc, s0, tb, v_users);
      if (ok && s1.pend_v >= 0) ok = pa_pv<D, PREC, 1>(sm, dsc, s1, tb, v_users);
    }
  }
  // whatever else went wrong, the MMAs already issued end before tensor memory is freed
  if (elect_one()) mma_commit(&sm.drain);
  __syncwarp();
  pg_land(&sm.drain, 0);
}

// ---------------------------------------------------------------------------------------
// Softmax warpgroup of slot S (one code for both slots: the loop has to stay in the instruction
// cache): thread t owns row t of the slot. The pieces live in shared memory, a copy per warp, so
// that the loop's registers are the row of S and a handful more.
// ---------------------------------------------------------------------------------------
struct PaRow {
  bool valid;
  int token, head, p;      // query token (of the call), head, position (-1: sees nothing)
};

__device__ __forceinline__ PaRow pa_row(const PagedAttnArgs& a, const PaItem& it, int i) {
  PaRow r;
  r.valid = i < it.nrows;
  const int R = it.row0 + (r.valid ? i : 0);
  const int ti = R / a.G;
  r.token = it.tok0 + ti;
  r.head = it.g * a.G + (R - ti * a.G);
  r.p = !r.valid ? -1 : (a.cu ? it.pos0 + ti : min(max(__ldg(a.seq_len + ti), 0), a.c.max_len) - 1);   // as pg_len
  return r;
}

// load8_f32 through the read-only path: the compiler may move it over stores to shared memory.
__device__ __forceinline__ void load8_ro(const float* p, float* x) { load8_f32(p, x); }
__device__ __forceinline__ void load8_ro(const __nv_bfloat16* p, float* x) {
  const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x[2 * k] = __uint_as_float(w[k] << 16);
    x[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
  }
}

// Rotates a warp's 32 rows (lane i has row i) into its slot's query buffer (128-byte swizzle),
// each in its view of key chunk `ck`. D / 16 lanes share a row, each with 8 of its pairs, so that
// the loads are of whole lines, and several rows' loads are under way at once.
template <typename T, int D, bool PREC>
__device__ __forceinline__ void pa_stage_rows(PaSmem<D>& sm, const PagedAttnArgs& a, const PaRow& r, int ck, int S) {
  constexpr int HD = D / 2, LANES = D / 16, ROWS = 32 / LANES;
  const bool live = r.valid && r.p >= 0;
  const int back = live ? r.p / a.L - ck : 0;
  const int view = back <= 0 ? VIEW_INTRA : (back == 1 ? VIEW_SUCC : VIEW_INTER);
  const int pos = live ? (int)dca_query_pos32(r.p, view, a.L, a.chunk) : -1;
  const int64_t q_of = (int64_t)r.token * a.q_stride + (int64_t)r.head * D;
  const int c = lane_id() % LANES;
  bool bad = false;
#pragma unroll(sizeof(T) == 2 ? 4 : 1)
  for (int s = 0; s < 32 / ROWS; ++s) {
    const int at = s * ROWS + lane_id() / LANES, t = 32 * (warp_id() & 3) + at;
    const int p = __shfl_sync(0xFFFFFFFFu, pos, at);
    const int64_t q = __shfl_sync(0xFFFFFFFFu, q_of, at) + 8 * c;
    uint32_t hi[2][4], lo[2][4];
    // rows that see nothing load what their clamped indices point to (no branch: the loads of
    // several rows have to be under way together) and become zeros, whatever that is
    const float4* cs4 = reinterpret_cast<const float4*>(a.table + (int64_t)max(p, 0) * HD + 8 * c);
    bool out_of_range = false;
    float x1[8], x2[8];
    load8_ro(static_cast<const T*>(a.q) + q, x1);
    load8_ro(static_cast<const T*>(a.q) + q + HD, x2);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float4 t4 = __ldg(cs4 + k);
      const float2 ca = make_float2(t4.x, t4.y), cb = make_float2(t4.z, t4.w);
      const float a1 = x1[2 * k] * a.scale, a2 = x2[2 * k] * a.scale;
      const float b1 = x1[2 * k + 1] * a.scale, b2 = x2[2 * k + 1] * a.scale;
      // fp16 views: the products see 11 bits of q, as the contiguous prefill's do; PREC adds
      // what the rounding left
      split_f16x2(rot_lo(a1, a2, ca), rot_lo(b1, b2, cb), hi[0][k], lo[0][k], out_of_range);
      split_f16x2(rot_hi(a1, a2, ca), rot_hi(b1, b2, cb), hi[1][k], lo[1][k], out_of_range);
    }
    bad |= out_of_range && p >= 0;
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int h = 0; h < 2; ++h) { hi[h][k] = p >= 0 ? hi[h][k] : 0u; lo[h][k] = p >= 0 ? lo[h][k] : 0u; }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int ch = c + h * LANES;                  // 16-byte chunk of the row
      const uint32_t off = (uint32_t)(ch >> 3) * 16384u + sw128_offset((uint32_t)t, (uint32_t)(ch & 7));
      *reinterpret_cast<uint4*>(sm.q[S] + off) = make_uint4(hi[h][0], hi[h][1], hi[h][2], hi[h][3]);
      if (PREC) *reinterpret_cast<uint4*>(sm.q[1] + off) = make_uint4(lo[h][0], lo[h][1], lo[h][2], lo[h][3]);
    }
  }
  if (bad) latch(Q1M_ERR_RANGE);
}

template <int D, bool PREC>
__device__ __forceinline__ void pa_stage(PaSmem<D>& sm, const PagedAttnArgs& a, const PaRow& r, int tile, int S) {
  const int ck = tile / (a.L / 128);
  if (a.q_f32) pa_stage_rows<float, D, PREC>(sm, a, r, ck, S);
  else pa_stage_rows<__nv_bfloat16, D, PREC>(sm, a, r, ck, S);
  fence_async_smem();
  __syncwarp();
  if (lane_id() == 0) mbar_arrive(&sm.q_full[S]);
}

// Writes 32 columns (from column 32 c) of a row: directly in the output's type, or a partial.
template <int D, bool PREC>
__device__ __forceinline__ void pa_store32(const PagedAttnArgs& a, const PaItem& it, const PaRow& r, int i,
                                           int c, const float* y) {
  if (PREC || it.part >= 0) {
    float* dst = it.part >= 0 ? a.o_part + (it.part * pa_rows(PREC) + i) * D + 32 * c
                              : static_cast<float*>(a.out) + ((int64_t)r.token * a.hq + r.head) * D + 32 * c;
#pragma unroll
    for (int j = 0; j < 32; j += 4)
      *reinterpret_cast<float4*>(dst + j) = make_float4(y[j], y[j + 1], y[j + 2], y[j + 3]);
  } else {
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) + ((int64_t)r.token * a.hq + r.head) * D + 32 * c;
#pragma unroll
    for (int j = 0; j < 32; j += 8)
      *reinterpret_cast<uint4*>(dst + j) = make_uint4(pack_bf16x2(y[j], y[j + 1]), pack_bf16x2(y[j + 2], y[j + 3]),
                                                      pack_bf16x2(y[j + 4], y[j + 5]), pack_bf16x2(y[j + 6], y[j + 7]));
  }
}

template <int D, bool PREC>
__device__ __forceinline__ void pa_store_lse(const PagedAttnArgs& a, const PaItem& it, const PaRow& r, int i, float lse2) {
  if (it.part >= 0) a.lse_part[it.part * pa_rows(PREC) + i] = lse2;
  else if (a.lse) a.lse[(int64_t)r.head * a.n_tokens + r.token] = lse2 * 0.69314718055994531f;
}

// Bits 0 .. n - 1.
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : (n >= 32 ? ~0u : (1u << n) - 1u); }

template <int D, bool PREC>
__device__ void pa_softmax(PaSmem<D>& sm, const PagedAttnArgs& a, const int S) {
  if (PREC && S == 1) return;                        // one slot; its low halves use q[1]
  const int t = threadIdx.x & 127;
  const uint32_t tb = sm.tmem_base + ((32u * (warp_id() & 3u)) << 16) + 256u * S;
  volatile int* gave_up = &sm.gave_up;
  PaItem* const piece = sm.piece[warp_id()];
  PaWalk* const walk = &sm.walk[warp_id()];
  if (lane_id() == 0) walk->init(a, sm.plan);
  auto advance = [&](PaItem* it) { return pa_advance(a, sm.plan, pa_rows(PREC), walk, it); };
  uint32_t sn = 0, on = 0;
  bool ok = true, have = advance(&piece[0]), written = true;
  int cur = 0;
  bool alt = false;
  int i = 0, end = 0, view_end = 0, hi = 0, lo = 0;   // tiles i .. end - 1; key j visible iff j <= hi
  const int sk = a.window > 0 ? a.sinks : 0;          // and (j >= lo or j < sk)
  float m = -INFINITY, l = 0.f, m_total = -INFINITY;  // m_total: what PREC's total is relative to
  auto enter = [&]() {
    const PaItem& it = piece[cur];
    alt = !PREC && it.nrows <= 128;
    i = alt ? S : 0;
    end = it.take;
    view_end = INT32_MIN;
  };
  if (have) enter();
  while (true) {
    // the next tile's queries, where its view is new: the slot's last S has been read, so its
    // QK^T is done with the buffer; for a new piece its first QK^T runs while the results of the
    // one before come out
    if (have && i < end && ok) {
      const PaItem& it = piece[cur];
      const int tile = it.tile(i);
      if (tile >= view_end) {
        const int row = alt ? t : 128 * S + t;
        const PaRow r = pa_row(a, it, row);
        if (view_end == INT32_MIN) {                  // rows behind the last see all: nothing to mask
          hi = !r.valid ? INT32_MAX : (a.cu ? r.p : min(r.p, it.len - 1));
          lo = a.window > 0 && r.p >= a.window ? r.p - a.window + 1 : 0;
        }
        pa_stage<D, PREC>(sm, a, r, tile, S);
        view_end = pa_view_end(a, it, tile);
      }
    }
    if (!written) {                                    // the finished piece, one slot's own rows
      const PaItem& it = piece[cur ^ 1];
      const int row = 128 * S + t;
      const PaRow r = pa_row(a, it, row);
      if (ok) ok = pg_wait(&sm.o_done[S], on & 1, gave_up);
      ++on;
      tc_fence_after();
      const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);      // a NaN sum stays one
      const float f = PREC ? (m_total == m ? 1.f : ex2(m_total - m)) : 0.f;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t rr[32];
        tmem_ld32(tb + (PREC ? pa_turn(sn - 1) : 128u) + 32u * c, rr);
        float y[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) y[j] = __uint_as_float(rr[j]);
        if (PREC && it.take > 1) {
          tmem_ld32(tb + 256u + 32u * c, rr);
#pragma unroll
          for (int j = 0; j < 32; ++j) y[j] = fmaf(__uint_as_float(rr[j]), f, y[j]);
        }
#pragma unroll
        for (int j = 0; j < 32; ++j) y[j] = l == 0.f ? 0.f : y[j] * inv;
        if (ok && r.valid) pa_store32<D, PREC>(a, it, r, row, c, y);
      }
      if (ok && r.valid)
        pa_store_lse<D, PREC>(a, it, r, row, l > 0.f ? m - PA_BIAS + __log2f(l) : (l == 0.f ? -INFINITY : l));
      tc_fence_before();
      m = -INFINITY;
      l = 0.f;
      written = true;
    }
    if (!have) break;
    if (i < end && ok) {
      const int key0 = piece[cur].tile(i) * 128;
      const bool first = i == (alt ? S : 0);           // O holds nothing yet
      ok = pg_wait(&sm.s_full[S], sn & 1, gave_up);
      ++sn;
      tc_fence_after();
      uint32_t xr[128];
      tmem_ld128(tb, xr);
      float* x = reinterpret_cast<float*>(xr);
      if (__any_sync(0xFFFFFFFFu, key0 + 127 > hi || (key0 < lo && key0 + 127 >= sk))) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int k0 = key0 + 32 * q;
          // hi - k0 may be far above 32: clamp before the + 1
          const uint32_t seen = low_bits(min(hi - k0, 31) + 1) & (~low_bits(lo - k0) | low_bits(sk - k0));
#pragma unroll
          for (int c = 0; c < 32; ++c) x[32 * q + c] = (seen >> c) & 1u ? x[32 * q + c] : -INFINITY;
        }
      }
      float a8[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) a8[k] = x[k];
#pragma unroll
      for (int c = 8; c < 128; c += 8)
#pragma unroll
        for (int k = 0; k < 8; ++k) a8[k] = fmaxf(a8[k], x[c + k]);
#pragma unroll
      for (int wdt = 4; wdt >= 1; wdt /= 2)
#pragma unroll
        for (int k = 0; k < wdt; ++k) a8[k] = fmaxf(a8[k], a8[k + wdt]);
      const float mx = a8[0], m_before = m;
      const bool need = mx > m + PA_RESCALE_THRESHOLD;
      if (__any_sync(0xFFFFFFFFu, need)) {
        const float m_new = need ? mx : m;
        const float alpha = need ? ex2(m - m_new) : 1.f;
        l *= alpha;
        if (!PREC && !first) {
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t rr[32];
            tmem_ld32(tb + 128u + 32u * c, rr);
#pragma unroll
            for (int j = 0; j < 32; ++j) rr[j] = __float_as_uint(__uint_as_float(rr[j]) * alpha);
            tmem_st32(tb + 128u + 32u * c, rr);
          }
        }
        m = m_new;
      }
      const float mu = m == -INFINITY ? 0.f : m - PA_BIAS;
      const uint64_t nmu = f2_pack(-mu, -mu);
      uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
      for (int ch = 0; ch < 4; ++ch) {
        uint32_t pk[16], pl[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const int j = 32 * ch + 2 * c;
          float d0, d1;
          f2_unpack(f2_add(f2_pack(x[j], x[j + 1]), nmu), d0, d1);
          const float p0 = ex2(d0), p1 = ex2(d1);
          acc[c & 3] = f2_add(acc[c & 3], f2_pack(p0, p1));
          pk[c] = pack_f16x2(p0, p1);
          if (PREC) {
            const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&pk[c]));
            pl[c] = pack_f16x2(p0 - back.x, p1 - back.y);
          }
        }
        tmem_st16(tb + 16u * ch, pk);
        if (PREC) tmem_st16(tb + 64u + 16u * ch, pl);
      }
      float s0, s1, s2, s3;
      f2_unpack(f2_add(acc[0], acc[1]), s0, s1);
      f2_unpack(f2_add(acc[2], acc[3]), s2, s3);
      l += (s0 + s1) + (s2 + s3);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane_id() == 0) mbar_arrive(&sm.p_full[S]);
      if (PREC && !first) {
        // The tensor core cuts what it adds to an accumulator towards zero, a bias that grows
        // with every step (6e-6 of the result at 16,384 keys in one accumulator); so each tile's
        // product (done: this tile's S came after it) is added to the total here, rounded.
        const float f = m_total == m_before ? 1.f : ex2(m_total - m_before);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t rr[32], tt[32];
          tmem_ld32(tb + pa_turn(sn) + 32u * c, rr);
          if (i > 1) {
            tmem_ld32(tb + 256u + 32u * c, tt);
#pragma unroll
            for (int j = 0; j < 32; ++j) rr[j] = __float_as_uint(fmaf(__uint_as_float(tt[j]), f, __uint_as_float(rr[j])));
          }
          tmem_st32(tb + 256u + 32u * c, rr);
        }
        tmem_wait_st();
        tc_fence_before();
      }
      if (PREC) m_total = first ? -INFINITY : m_before;
      i += alt ? 2 : 1;
    }
    if (i < end && ok) continue;
    // the piece is finished
    if (alt) {
      // two slots with every second tile of the same rows: slot 1 hands its result over
      const PaItem& it = piece[cur];
      const PaRow r = pa_row(a, it, t);
      const bool some = S < it.take;                   // the slot had a tile
      if (ok && some) {
        ok = pg_wait(&sm.o_done[S], on & 1, gave_up);
        tc_fence_after();
      }
      if (some) ++on;
      const bool held = ok && some;
      const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
      const float lse2 = l > 0.f ? m - PA_BIAS + __log2f(l) : (l == 0.f ? -INFINITY : l);
      float* box = reinterpret_cast<float*>(&sm.q[0][0]) + t * D;
      named_bar_sync(1, 256);                          // both slots are done with their queries
      float f0 = inv, f1 = 0.f, row_lse = 0.f;
      if (S == 1) sm.slot_lse[t] = held ? lse2 : -INFINITY;
      if (S == 0) named_bar_sync(2, 256);
      if (S == 0) {
        const float other = sm.slot_lse[t];
        const float M = fmaxf(lse2, other);
        const float w0 = lse2 == -INFINITY ? 0.f : ex2(lse2 - M), w1 = other == -INFINITY ? 0.f : ex2(other - M);
        const float ws = w0 + w1;
        f0 = ws == 0.f ? 0.f : w0 / ws * inv;
        f1 = ws == 0.f ? 0.f : w1 / ws;
        row_lse = ws == 0.f ? -INFINITY : M + __log2f(ws);
      }
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t rr[32];
        tmem_ld32(tb + 128u + 32u * c, rr);
        float y[32];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float4* b4 = reinterpret_cast<float4*>(box + 4 * ((8 * c + j) ^ (t & 15)));
          float4 v4 = make_float4(0.f, 0.f, 0.f, 0.f);
          if (S == 0) v4 = *b4;
          const float o4[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            y[4 * j + k] = (!held || f0 == 0.f ? 0.f : f0 * __uint_as_float(rr[4 * j + k])) + f1 * o4[k];
          if (S == 1) *b4 = make_float4(y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]);
        }
        if (S == 0 && held && r.valid) pa_store32<D, PREC>(a, it, r, t, c, y);
      }
      if (S == 0 && held && r.valid) pa_store_lse<D, PREC>(a, it, r, t, row_lse);
      tc_fence_before();
      if (S == 1) named_bar_sync(2, 256);
      named_bar_sync(3, 256);                          // the exchange buffer is free again
      m = -INFINITY;
      l = 0.f;
    }
    written = alt;
    cur ^= 1;
    have = advance(&piece[cur]);
    if (have) enter();
    else i = end;
  }
}

template <int D, bool PREC>
__global__ void __launch_bounds__(PA_THREADS, 1)
paged_attn_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                  const PagedAttnArgs a) {
  extern __shared__ uint8_t pa_raw[];
  PaSmem<D>& sm = *reinterpret_cast<PaSmem<D>*>((reinterpret_cast<uintptr_t>(pa_raw) + 1023) & ~uintptr_t(1023));
  const int w = warp_id();
  grid_release();
  if (threadIdx.x == 0) {
    for (int i = 0; i < PA_NK; ++i) { mbar_init(&sm.k_full[i], 1); mbar_init(&sm.k_empty[i], 1); }
    for (int i = 0; i < PA_NV; ++i) { mbar_init(&sm.v_full[i], 1); mbar_init(&sm.v_empty[i], 1); }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm.q_full[s], 4); mbar_init(&sm.s_full[s], 1); mbar_init(&sm.p_full[s], 4);
      mbar_init(&sm.o_done[s], 1); mbar_init(&sm.pv_done[s], 1);
    }
    mbar_init(&sm.drain, 1);
    fence_mbar_init();
    sm.gave_up = 0;
  }
  if (w == 9) { tmem_alloc(&sm.tmem_base, 512); tmem_relinquish(); }
  if (w == 8 && lane_id() == 0) { tma_prefetch(&mk); tma_prefetch(&mv); }
  if (a.cu) pa_plan(sm.plan, a, pa_rows(PREC));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (w < 8) {
    regs_increase<PA_REGS_SOFTMAX>();
    pa_softmax<D, PREC>(sm, a, w >> 2);
  } else {
    regs_decrease<PA_REGS_OTHER>();
    if (w == 8) pa_loader<D, 0>(sm, a, &mk, pa_rows(PREC));
    else if (w == 9) pa_mma<D, PREC>(sm, a);
    else if (w == 10) pa_loader<D, 1>(sm, a, &mv, pa_rows(PREC));
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (w == 9) { __syncwarp(); tmem_dealloc(sm.tmem_base, 512); }
  grid_wait();   // behind a decode kernel this grid ends after it, so that the merge's wait covers both
}

// Joins the partials of the row tiles that run boundaries cut, in CTA order: blocks (c, .) take
// the row tile that the begin of CTA c + 1's run is the first to cut, one warp a row.
template <int D, bool PREC>
__global__ void __launch_bounds__(256)
paged_attn_merge_kernel(const PagedAttnArgs a) {
  constexpr int ROWS = pa_rows(PREC);
  grid_wait();
  const PagedRowCut cut = a.cut[blockIdx.x + 1];
  const int i = blockIdx.y * 8 + warp_id(), lane = lane_id();
  if (i >= cut.nrows) return;
  const int n = cut.c1 - cut.c0 + 1;
  auto slot = [&](int k) { return (2 * (int64_t)(cut.c0 + k) + (k == 0 ? 1 : 0)) * ROWS + i; };
  const float mine = lane < n ? a.lse_part[slot(lane)] : -INFINITY;
  float M = mine;
  for (int k = lane + 32; k < n; k += 32) M = fmaxf(M, a.lse_part[slot(k)]);
#pragma unroll
  for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
  float sum = 0.f, y[4] = {0.f, 0.f, 0.f, 0.f};
  const int d0 = 4 * lane;
  for (int k0 = 0; k0 < n; k0 += 4) {
    float4 x[4];
    float ls[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      ls[k] = -INFINITY;
      if (k0 + k < n) {
        if (d0 < D) x[k] = *reinterpret_cast<const float4*>(a.o_part + slot(k0 + k) * D + d0);
        ls[k] = k0 + k < 32 ? __shfl_sync(0xFFFFFFFFu, mine, k0 + k) : a.lse_part[slot(k0 + k)];
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      // a part without keys weighs nothing; a NaN part stays one (M may not see it)
      const float f = ls[k] == -INFINITY ? 0.f : (M == -INFINITY ? ls[k] : ex2(ls[k] - M));
      sum += f;
      y[0] += f * x[k].x; y[1] += f * x[k].y; y[2] += f * x[k].z; y[3] += f * x[k].w;
    }
  }
  const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
#pragma unroll
  for (int c = 0; c < 4; ++c) y[c] *= inv;
  const int R = cut.row0 + i, ti = R / a.G, h = cut.g * a.G + (R - ti * a.G);
  const int64_t token = cut.tok0 + ti, at = (token * a.hq + h) * D + d0;
  if (d0 < D) {
    if (PREC) store4(static_cast<float*>(a.out) + at, y);
    else store4(static_cast<__nv_bfloat16*>(a.out) + at, y);
  }
  if (a.lse && lane == 0)
    a.lse[(int64_t)h * a.n_tokens + token] =
        (sum > 0.f ? M + __log2f(sum) : (sum == 0.f ? -INFINITY : sum)) * 0.69314718055994531f;
}

}  // namespace q1m
