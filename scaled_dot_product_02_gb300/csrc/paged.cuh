// paged.cuh -- the paged-cache attention's view of its work, shared by its two
// kernels: sequences, the keys that a block of tokens sees, and the cutting of
// all key tiles into equal shares (paged.cu describes it).
#pragma once
#include "common.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace sdpa {

constexpr int kTile = 128;            // keys of a tile
constexpr int kStage = 32768;         // bytes of a ring stage
constexpr int kSmemMax = 232448;      // 227 KB
constexpr float kLn2 = 0.6931471805599453f;

// What a CTA records of the item its share starts in, for the join.
struct PagedCut {
  long long at;      // first tile of that item
  int n, b, i0, unit;
};

__device__ __forceinline__ long long share_at(long long total, int w, int workers) { return total * w / workers; }

// One sequence of the batch: its rows and its cached keys.
struct PagedSeq {
  int row0, q_len, kv_len;
};
__device__ __forceinline__ PagedSeq paged_seq(const PagedParams& p, int b) {
  PagedSeq s;
  s.row0 = s.q_len = s.kv_len = 0;
  if (SDPA_ADDR_OK(p.chk, p.cu_q + b, 8) && SDPA_ADDR_OK(p.chk, p.kv_lens + b, 4)) {
    s.row0 = __ldg(p.cu_q + b);
    s.q_len = __ldg(p.cu_q + b + 1) - s.row0;
    s.kv_len = __ldg(p.kv_lens + b);
  }
  return s;
}
// Whether it fits what the host was told (every other index follows from it).
__device__ __forceinline__ bool paged_seq_ok(const PagedParams& p, const PagedSeq& s) {
  return s.row0 >= 0 && s.q_len >= 0 && s.q_len <= p.max_q && s.kv_len >= 0 && s.kv_len <= p.max_kv &&
         s.row0 <= p.total_q - s.q_len;
}

// A sequence as this launch sees it: without rows when the other kernel serves
// it (the rows kernel takes those of at most small_q new tokens).
__device__ __forceinline__ PagedSeq paged_mine(const PagedParams& p, PagedSeq s) {
  if ((s.q_len <= p.small_q) != (p.small != 0)) s.q_len = 0;
  return s;
}

// Keys that the tokens [i0, i1] of a sequence see between them: [lo, hi).
struct PagedSpan {
  int lo, hi, tile0, tiles;  // tiles: 128-key tiles that hold them (0: none)
};
__device__ __forceinline__ PagedSpan paged_span(const PagedParams& p, const PagedSeq& s, int i0, int i1) {
  PagedSpan r;
  const int off = s.kv_len - s.q_len;
  r.hi = p.causal ? max(0, i1 + off + 1) : s.kv_len;  // i1 < q_len: never past kv_len
  r.lo = p.window >= 0 ? max(0, i0 + off - p.window) : 0;
  r.tile0 = r.lo / kTile;
  r.tiles = r.hi > r.lo ? (r.hi + kTile - 1) / kTile - r.tile0 : 0;
  return r;
}

// An item's place among those of its block of tokens: the kv head, the block of
// its group's query heads (the first, and how many there are), and which part
// of the value columns.
struct PagedUnit {
  int kvh, head0, heads, split;
};
__device__ __forceinline__ PagedUnit paged_unit(const PagedParams& p, int unit) {
  PagedUnit u;
  u.split = unit % p.dv_splits;
  unit /= p.dv_splits;
  u.kvh = unit / p.head_blocks;
  const int first = (unit - u.kvh * p.head_blocks) * p.block_heads;
  u.head0 = u.kvh * p.group + first;
  u.heads = min(p.block_heads, p.group - first);
  return u;
}

__device__ __forceinline__ int paged_weight(const PagedParams& p, const PagedSpan& s) {
  return p.split ? max(1, s.tiles) : 1;
}

// Items of one sequence: blocks of `tokens` tokens, and within a block the kv
// heads (times the head blocks of a wide group). An item without keys counts
// as one tile, so that someone writes its zeros. Unless items are split
// (p.split), each weighs one, whatever its keys: shares are whole items.
__device__ __forceinline__ long long paged_units(const PagedParams& p, const PagedSeq& s) {
  if (!p.split) return (long long)((s.q_len + p.tokens - 1) / p.tokens) * p.units_per_block;
  long long n = 0;
  for (int i0 = 0; i0 < s.q_len; i0 += p.tokens)
    n += paged_weight(p, paged_span(p, s, i0, min(i0 + p.tokens, s.q_len) - 1));
  return n * p.units_per_block;
}

// A CTA's share of the tiles, walked item by item. Every role walks its own copy.
struct PagedWalk {
  long long u, u_end;     // tiles of all items, end to end
  long long block_at;     // first tile of block (b, i0)
  int b, i0;
  PagedSeq s;
  PagedSpan span;
  // the current item
  int unit;               // kv head and head block
  long long at;           // its first tile
  int weight;             // its length in the row of all items
  int j0, j1;             // its tiles in this share

  __device__ __forceinline__ int i1(const PagedParams& p) const { return min(i0 + p.tokens, s.q_len) - 1; }
  __device__ __forceinline__ bool whole() const { return j0 == 0 && j1 == span.tiles; }
  __device__ __forceinline__ void locate(const PagedParams& p) {
    weight = paged_weight(p, span);
    unit = (int)((u - block_at) / weight);
    at = block_at + (long long)unit * weight;
    j0 = (int)(u - at);
    j1 = p.split ? min(span.tiles, (int)min((long long)weight, u_end - at)) : span.tiles;
  }
  __device__ __forceinline__ void start(const PagedParams& p, int b_, int i0_, long long block_at_, long long u_,
                                        long long u_end_) {
    u = u_;
    u_end = u_end_;
    block_at = block_at_;
    b = b_;
    i0 = i0_;
    s = paged_mine(p, paged_seq(p, b));
    span = paged_span(p, s, i0, i1(p));
    locate(p);
  }
  // The next item of the share; false when it is done.
  __device__ __forceinline__ bool next(const PagedParams& p) {
    u = at + weight;
    if (u >= u_end) return false;
    if (unit + 1 == p.units_per_block) {
      block_at += (long long)p.units_per_block * weight;
      i0 += p.tokens;
      while (i0 >= s.q_len) {  // u < u_end: a later sequence has rows
        s = paged_mine(p, paged_seq(p, ++b));
        i0 = 0;
      }
      span = paged_span(p, s, i0, i1(p));
    }
    locate(p);
    return true;
  }
};

// One lane's part of a key tile's copy: box_rows slots of one page.
struct PagedBox {
  int page, slot;
  uint32_t live;  // lanes with slots to copy
  bool mine;
};
// Lane's box of the tile that starts at key0, of a span; every lane of the warp calls it.
__device__ __forceinline__ PagedBox paged_box(const PagedParams& p, const PagedSpan& span, int b, int key0, int lane) {
  PagedBox x;
  const int key = key0 + lane * p.box_rows;
  x.mine = lane * p.box_rows < kTile && key < span.hi && key + p.box_rows > span.lo;
  x.page = p.num_pages;  // outside the map: reads as zeros
  x.slot = 0;
  if (x.mine) {
    const int col = key / p.page_size;
    x.slot = key - col * p.page_size;
    const int32_t* at = p.block_table + b * p.table_stride + col;
    const int id = SDPA_ADDR_OK(p.chk, at, 4) ? __ldg(at) : -1;
    if (id >= 0 && id < p.num_pages)
      x.page = id;
    else
      record_error(p.err, SDPA_ERR_BAD_INDEX);
  }
  x.live = __popc(__ballot_sync(0xffffffffu, x.mine));
  return x;
}

// Where the shares of a launch lie. Every CTA adds up the batch itself.
struct PagedShares {
  bool fit;           // every sequence fits what the host was told
  long long total;    // length of all items end to end (0 unless they fit)
};
struct PagedScan {    // shared memory of the scan
  long long warp_sum[16], block_at[2];
  int b[2], i0[2];
};
// Adds up all sequences and finds the blocks of tokens in which the shares of
// workers w0, w0 + step, ... (n_w of them, at most two) start. All THREADS
// threads call it.
template <int THREADS>
__device__ __forceinline__ PagedShares paged_scan(const PagedParams& p, PagedScan* sc, int w0, int step, int n_w,
                                                  int most_workers) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int per = (p.batch + THREADS - 1) / THREADS;  // thread t takes sequences [t per, (t + 1) per)
  const int b_lo = min(p.batch, (int)threadIdx.x * per), b_hi = min(p.batch, b_lo + per);
  long long own = 0;
  bool fits = true;
  for (int b = b_lo; b < b_hi; ++b) {
    const PagedSeq s = paged_seq(p, b);
    if (paged_seq_ok(p, s) && (b > 0 || s.row0 == 0))
      own += paged_units(p, paged_mine(p, s));
    else
      fits = false;
  }
  long long upto = own;  // inclusive sum over the warp
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  if (lane == 31) sc->warp_sum[warp] = upto;
  PagedShares r;
  r.fit = __syncthreads_and(fits);
  long long before = upto - own;
  r.total = 0;
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) before += sc->warp_sum[w];
    r.total += sc->warp_sum[w];
  }
  if (!r.fit) r.total = 0;
  const int workers = (int)min((long long)most_workers, r.total);
  for (int x = 0; x < n_w; ++x) {
    const int w = w0 + x * step;
    if (w >= workers) break;
    const long long u = share_at(r.total, w, workers);
    if (u < before || u >= before + own) continue;  // one thread: the share starts in its sequences
    int b = b_lo;
    long long at = before;
    PagedSeq s = paged_mine(p, paged_seq(p, b));
    for (long long n = paged_units(p, s); u >= at + n; n = paged_units(p, s)) {
      at += n;
      s = paged_mine(p, paged_seq(p, ++b));
    }
    int i0 = 0;
    while (true) {
      const long long n = (long long)p.units_per_block *
                          paged_weight(p, paged_span(p, s, i0, min(i0 + p.tokens, s.q_len) - 1));
      if (u < at + n) break;
      at += n;
      i0 += p.tokens;
    }
    sc->b[x] = b;
    sc->i0[x] = i0;
    sc->block_at[x] = at;
  }
  __syncthreads();
  return r;
}

// A piece of work as the scheduler of a pipeline publishes it.
struct PagedPiece {
  int row0, q_len, kv_len, i0, unit;  // row0 < 0: no more
  int j0, j1;                         // its key tiles, counted from the span's first
  int slot;                           // its partial result, or -1: the whole item
};

// Where a pipeline's pieces come from: its share of the tiles (p.split), or
// the tickets, last block of tokens first and the items of a block together.
// A whole warp walks it.
struct PagedFeed {
  PagedWalk w;
  bool more;
  long long u0;
  int blocks, tickets;

  __device__ __forceinline__ void take(const PagedParams& p, int lane) {
    while (true) {
      int t = tickets;  // a counter the address check rejects hands out none
      if (lane == 0 && SDPA_ADDR_OK(p.chk, p.tickets, 4)) t = atomicAdd(p.tickets, 1);
      t = __shfl_sync(0xffffffffu, t, 0);
      more = t < tickets;
      if (!more) return;
      w.unit = t % p.units_per_block;
      t /= p.units_per_block;
      w.b = t % p.batch;
      w.i0 = (blocks - 1 - t / p.batch) * p.tokens;
      w.s = paged_mine(p, paged_seq(p, w.b));
      if (w.i0 >= w.s.q_len) continue;
      w.span = paged_span(p, w.s, w.i0, w.i1(p));
      w.at = 0;
      w.j0 = 0;
      w.j1 = w.span.tiles;
      return;
    }
  }
  // Worker `me` of `workers`; x: its place in the scan.
  __device__ __forceinline__ void start(const PagedParams& p, const PagedScan* sc, int x, long long total, int me,
                                        int workers, int lane) {
    u0 = 0;
    tickets = blocks = 0;
    more = me < workers;
    if (!more) return;
    if (p.split) {
      u0 = share_at(total, me, workers);
      w.start(p, sc->b[x], sc->i0[x], sc->block_at[x], u0, share_at(total, me + 1, workers));
      PagedCut* cut = p.cuts + me;
      if (lane == 0 && SDPA_ADDR_OK(p.chk, cut, sizeof(PagedCut))) *cut = PagedCut{w.at, w.weight, w.b, w.i0, w.unit};
    } else {
      blocks = (p.max_q + p.tokens - 1) / p.tokens;
      tickets = blocks * p.batch * p.units_per_block;
      take(p, lane);
    }
  }
  __device__ __forceinline__ void next(const PagedParams& p, int lane) {
    if (p.split)
      more = w.next(p);
    else
      take(p, lane);
  }
  __device__ __forceinline__ PagedPiece piece() const {
    return PagedPiece{more ? w.s.row0 : -1, w.s.q_len, w.s.kv_len, w.i0, w.unit, w.j0, w.j1,
                      w.whole() ? -1 : (w.at < u0 ? 0 : 1)};
  }
};

}  // namespace sdpa
