// paged.cuh -- the paged-cache attention's view of its work, shared by its two
// kernels: sequences, the keys that a block of tokens sees, and the cutting of
// all key tiles into equal shares (paged.cu describes it).
#pragma once
#include <climits>

#include "common.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace sdpa {

constexpr int kTile = 128;            // keys of a tile
constexpr int kStage = 32768;         // bytes of a ring stage
constexpr int kSmemMax = 232448;      // 227 KB
constexpr float kLn2 = 0.6931471805599453f;

// What a worker records of the item its share starts in, for the join.
struct PagedCut {
  long long at;          // where that item starts
  int n, row0, tokens, unit;  // its length, first row, tokens, and place in its block
};

// Equal shares of the row of all items: where share w starts.
struct PagedShare {
  long long base;
  int rest, workers;
  __device__ __forceinline__ PagedShare(long long total, int most_workers) {
    workers = (int)min((long long)most_workers, total);
    base = 0;
    rest = 0;
    if (workers > 0) {
      if (total < (1ll << 32)) {  // a 64-bit division costs several times as much
        base = (unsigned)total / (unsigned)workers;
      } else {
        base = total / workers;
      }
      rest = (int)(total - base * workers);
    }
  }
  __device__ __forceinline__ long long at(int w) const { return base * w + min(w, rest); }
  // The share that holds position u.
  __device__ __forceinline__ int of(long long u) const {
    const long long longer = (base + 1) * rest;  // the first `rest` shares hold one more
    const long long past = u < longer ? u : u - longer, n = u < longer ? base + 1 : base;
    return (u < longer ? 0 : rest) + (int)(past < (1ll << 32) && n < (1ll << 32) ? (unsigned)past / (unsigned)n : past / n);
  }
};

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

// An item's length in the row of all items: its tiles, behind p.lead places that stand for what an item costs by itself.
__device__ __forceinline__ int paged_weight(const PagedParams& p, const PagedSpan& s) {
  return p.split && s.tiles > 0 ? s.tiles + p.lead : 1;
}

// Items of one sequence: blocks of `tokens` tokens, and within a block the kv
// heads (times the head blocks of a wide group). An item without keys counts
// as one place, so that someone writes its zeros. Unless items are split
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
  // Whether the share holds all of the item's places (with p.lead it may hold all tiles, but not those in front).
  __device__ __forceinline__ bool covers() const { return u <= at && at + weight <= u_end; }
  __device__ __forceinline__ void locate(const PagedParams& p) {
    weight = paged_weight(p, span);
    unit = (int)((unsigned)(u - block_at) / (unsigned)weight);  // the host bounds a block's length
    at = block_at + (long long)unit * weight;
    j0 = max(0, (int)(u - at) - p.lead);
    j1 = p.split ? min(span.tiles, max(0, (int)min((long long)weight, u_end - at) - p.lead)) : span.tiles;
  }
  __device__ __forceinline__ PagedCut cut(const PagedParams& p) const {
    return PagedCut{at, weight, s.row0 + i0, i1(p) - i0 + 1, unit};
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

// One copy of a key tile: box_rows slots of one page.
struct PagedBox {
  int page, slot;
  bool mine;  // its keys are seen
};
// Box `box` of the tile that starts at key0, of a span.
__device__ __forceinline__ PagedBox paged_box(const PagedParams& p, const PagedSpan& span, int b, int key0, int box) {
  PagedBox x;
  const int key = key0 + box * p.box_rows;
  x.mine = box * p.box_rows < kTile && key < span.hi && key + p.box_rows > span.lo;
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
  return x;
}
// How many boxes of the tile's keys [k_lo, k_hi) (multiples of box_rows) are copied.
__device__ __forceinline__ int paged_boxes(const PagedParams& p, const PagedSpan& span, int key0, int k_lo, int k_hi) {
  const int lo = max(span.lo - key0, k_lo), hi = min(span.hi - key0, k_hi);
  return hi > lo ? (hi + p.box_rows - 1) / p.box_rows - lo / p.box_rows : 0;
}

// Where the shares of a launch lie. Every CTA adds up the batch itself.
struct PagedShares {
  bool fit;           // every sequence fits what the host was told
  long long total;    // length of all items end to end (0 unless they fit)
};
struct PagedScan {    // shared memory of the scan: sums, and the walk as the share starts
  long long warp_sum[16];
  PagedWalk start;
};
// Adds up all sequences and, with LOCATE, finds the block of tokens in which the
// share of worker w of at most most_workers starts. All THREADS threads call it.
template <int THREADS, bool LOCATE>
__device__ __forceinline__ PagedShares paged_scan(const PagedParams& p, PagedScan* sc, int w = 0, int most_workers = 1) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int per = (p.batch + THREADS - 1) / THREADS;  // thread t takes sequences [t per, (t + 1) per)
  const int b_lo = min(p.batch, (int)threadIdx.x * per), b_hi = min(p.batch, b_lo + per);
  long long own = 0;
  bool fits = true;
  PagedSeq first{0, 0, 0};
  for (int b = b_lo; b < b_hi; ++b) {
    const PagedSeq s = paged_seq(p, b), mine = paged_mine(p, s);
    if (b == b_lo) first = mine;
    if (paged_seq_ok(p, s) && (b > 0 || s.row0 == 0))
      own += paged_units(p, mine);
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
  const PagedShare share(r.total, most_workers);
  const long long u = LOCATE && w < share.workers ? share.at(w) : -1;
  if (LOCATE && u >= before && u < before + own) {  // one thread: the share starts in its sequences
    PagedWalk& k = sc->start;
    k.u = u;
    k.u_end = share.at(w + 1);
    k.b = b_lo;
    k.block_at = before;
    k.s = b_hi - b_lo == 1 ? first : paged_mine(p, paged_seq(p, b_lo));
    if (b_hi - b_lo > 1)
      for (long long n = paged_units(p, k.s); u >= k.block_at + n; n = paged_units(p, k.s)) {
        k.block_at += n;
        k.s = paged_mine(p, paged_seq(p, ++k.b));
      }
    k.i0 = 0;
    while (true) {
      k.span = paged_span(p, k.s, k.i0, k.i1(p));
      const long long n = (long long)p.units_per_block * paged_weight(p, k.span);
      if (u < k.block_at + n) break;
      k.block_at += n;
      k.i0 += p.tokens;
    }
    k.locate(p);
  }
  __syncthreads();
  return r;
}

// A piece of work as the scheduler of a pipeline publishes it.
struct PagedPiece {
  int row0, q_len, kv_len, b, i0, unit;  // row0 < 0: no more
  int j0, j1;                         // its key tiles, counted from the span's first
  int slot;                           // where its partial result goes, or -1: the whole item
};

// A place in the order that the tickets follow: the sequences with the most
// keys first (up to kSorted of them; a larger batch in its own order), the last
// blocks of tokens first, and the items of a block together. So the longest
// items start first, and the CTAs at work share the same few sequences' keys.
// Each step through a sorted batch goes over all of it. Sorted against in their
// order, 30 to 250 tokens each over 300 to 4000 keys: 16 sequences at head_dim 128
// 94 / 121 us, at 512 207 / 265; 32 at 128 168 / 193; 64 at 128 301 / 330, at 192
// 454 / 463; 80 at 128 333 / 354, at 192 486 / 491. Another 80 at 512: 272 / 251.
constexpr int kSorted = 32;

struct PagedOrder {
  long long key;      // of the sequence: its keys, then its place
  PagedSeq s;
  int b, blocks, blk;  // the sequence, its blocks of tokens, the current one counted from the last

  __device__ __forceinline__ void before_all() {
    key = LLONG_MAX;
    b = -1;
    blocks = blk = 0;
  }
  __device__ __forceinline__ int first_token(const PagedParams& p, int k) const { return (blocks - 1 - k) * p.tokens; }
  __device__ __forceinline__ PagedSpan span_of(const PagedParams& p, int k) const {
    const int i0 = first_token(p, k);
    return paged_span(p, s, i0, min(i0 + p.tokens, s.q_len) - 1);
  }
  // The first block of the next sequence with rows; false when there is none. A whole warp calls it.
  __device__ __forceinline__ bool next_sequence(const PagedParams& p, int lane) {
    long long best = -1;  // the largest key below the current one
    if (p.batch <= kSorted) {
      for (int i = lane; i < p.batch; i += 32) {
        const PagedSeq x = paged_mine(p, paged_seq(p, i));
        const long long k = (long long)x.kv_len << 32 | (unsigned)(p.batch - i);
        if (x.q_len > 0 && k < key && k > best) best = k;
      }
#pragma unroll
      for (int o = 16; o > 0; o /= 2) {
        const long long other = __shfl_xor_sync(0xffffffffu, best, o);
        best = other > best ? other : best;
      }
      if (best >= 0) b = p.batch - (int)(best & 0xffffffff);
    } else {
      for (int b0 = b + 1; b0 < p.batch && best < 0; b0 += 32) {
        const uint32_t live =
            __ballot_sync(0xffffffffu, b0 + lane < p.batch && paged_mine(p, paged_seq(p, b0 + lane)).q_len > 0);
        if (live) {
          b = b0 + __ffs(live) - 1;
          best = 0;
        }
      }
    }
    if (best < 0) return false;
    key = best;
    s = paged_mine(p, paged_seq(p, b));
    blocks = (s.q_len + p.tokens - 1) / p.tokens;
    blk = 0;
    return true;
  }
};

// Where a pipeline's pieces come from. The tickets hand out whole items, as
// many as go round all pipelines evenly (all items when p.tail is 0: the items
// are many, or too short for more); the key tiles of the rest, laid end to end
// in the same order, are cut into p.tail equal shares and handed out by further
// tickets, and the items that cross a cut are joined afterwards. A whole warp
// walks it.
struct PagedFeed {
  PagedWalk w;          // the current piece; u .. u_end: of its share
  bool more;
  PagedOrder at;        // the block of the last whole item's ticket, or of the current piece of a share
  int done;             // blocks of the sequences before at's
  int whole, share;     // whole items handed out; the current share, or -1
  PagedOrder rest;      // where the rest begins
  long long rest_at;    // its block's start, counted from the rest's first item
  long long total;      // length of the rest, -1: not yet added up
  int asked;            // lane 0: the next ticket, when it has been asked for
  bool has_asked;

  // Ask for the next ticket, so that it is there when the current item's last copies are out (but no earlier: a
  // ticket kept behind a long item is work that waits).
  __device__ __forceinline__ void ask(const PagedParams& p, int lane) {
    if (has_asked) return;
    has_asked = true;
    asked = 0x7fffffff;  // a counter the address check rejects hands out none
    if (lane == 0 && SDPA_ADDR_OK(p.chk, p.tickets, 4)) asked = atomicAdd(p.tickets, 1);
  }
  __device__ __forceinline__ void set_piece(const PagedParams& p) {
    w.b = at.b;
    w.s = at.s;
    w.i0 = at.first_token(p, at.blk);
    w.span = at.span_of(p, at.blk);
    w.weight = max(1, w.span.tiles);
  }
  // Moves `o`, whose block starts at `start`, to the block that holds position u; false behind the last one, with
  // start the length of all.
  __device__ __forceinline__ bool seek(const PagedParams& p, PagedOrder& o, long long& start, long long u, int lane) {
    while (true) {
      while (o.blk < o.blocks) {
        const int k = o.blk + lane;
        const long long own = k < o.blocks ? (long long)p.units_per_block * max(1, o.span_of(p, k).tiles) : 0;
        long long upto = own;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const long long y = __shfl_up_sync(0xffffffffu, upto, d);
          if (lane >= d) upto += y;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, u < start + upto);
        if (past) {
          const int l = __ffs(past) - 1;
          start += __shfl_sync(0xffffffffu, upto - own, l);
          o.blk += l;
          return true;
        }
        start += __shfl_sync(0xffffffffu, upto, 31);
        o.blk += 32;
      }
      if (!o.next_sequence(p, lane)) return false;
    }
  }
  __device__ __forceinline__ void take(const PagedParams& p, int lane) {
    ask(p, lane);
    has_asked = false;
    const int t = __shfl_sync(0xffffffffu, asked, 0);
    more = false;
    share = -1;
    if (t < whole || total < 0) {
      const int goal = min(t, whole), block = goal / p.units_per_block;  // the rest's first item, once it has begun
      while (block >= done + at.blocks) {
        done += at.blocks;
        at.blocks = 0;
        if (!at.next_sequence(p, lane)) return;
      }
      at.blk = block - done;
      w.unit = goal - block * p.units_per_block;
      if (t < whole) {
        set_piece(p);
        w.at = 0;
        w.j0 = 0;
        w.j1 = w.span.tiles;
        more = true;
        return;
      }
      if (p.tail == 0) return;
      rest = at;
      rest_at = -(long long)w.unit * max(1, at.span_of(p, at.blk).tiles);
      PagedOrder end = rest;
      total = rest_at;
      seek(p, end, total, LLONG_MAX, lane);
    }
    const PagedShare cut(total, p.tail);
    if (t - whole >= cut.workers) return;
    share = t - whole;
    w.u = cut.at(share);
    w.u_end = cut.at(share + 1);
    at = rest;
    w.block_at = rest_at;
    more = seek(p, at, w.block_at, w.u, lane);
    set_piece(p);
    locate(p);
    PagedCut* to = p.cuts + share;
    if (lane == 0 && SDPA_ADDR_OK(p.chk, to, sizeof(PagedCut))) *to = w.cut(p);
    if (lane == 0 && SDPA_ADDR_OK(p.chk, p.total_tiles, 8)) *p.total_tiles = total;
  }
  // The piece of the share that starts at w.u, in the block at w.block_at.
  __device__ __forceinline__ void locate(const PagedParams& p) {
    w.unit = (int)((unsigned)(w.u - w.block_at) / (unsigned)w.weight);
    w.at = w.block_at + (long long)w.unit * w.weight;
    w.j0 = (int)(w.u - w.at);
    w.j1 = min(w.span.tiles, (int)min((long long)w.weight, w.u_end - w.at));
  }
  // items: all items of the launch; pipes: the pipelines that share them.
  __device__ __forceinline__ void start(const PagedParams& p, long long items, int pipes, bool mine, int lane) {
    at.before_all();
    done = 0;
    share = total = -1;
    whole = p.tail ? (int)(items - items % pipes) : 0x7fffffff;
    more = has_asked = false;
    if (mine) take(p, lane);
  }
  // Whether the current piece is the last before the next ticket.
  __device__ __forceinline__ bool last() const { return share < 0 || w.at + w.weight >= w.u_end; }
  __device__ __forceinline__ void next(const PagedParams& p, int lane) {
    if (!last()) {
      w.u = w.at + w.weight;
      if (w.unit + 1 == p.units_per_block) {
        w.block_at += (long long)p.units_per_block * w.weight;
        if (++at.blk >= at.blocks) at.next_sequence(p, lane);  // w.u < w.u_end: there is one
        set_piece(p);
      }
      locate(p);
    } else {
      take(p, lane);
    }
  }
  __device__ __forceinline__ PagedPiece piece(const PagedParams& p) const {
    // at most one item continues from the share before, and one into the next
    const int slot = share < 0 || w.whole() ? -1 : share * 2 + (w.at < PagedShare(total, p.tail).at(share) ? 0 : 1);
    return PagedPiece{more ? w.s.row0 : -1, w.s.q_len, w.s.kv_len, w.b, w.i0, w.unit, w.j0, w.j1, slot};
  }
};

// Producer `pw` of three copies its boxes (3 e + pw, one a lane) of the K and V
// tiles [j0, j1) of an item through the ring (V of a tile behind its K, or behind
// the next tile's, as C says); c counts the stages. Every producer arrives on each stage, with copies in
// it or not, or the ring could go on without one and leave it a phase behind.
// Producer 0 sets the byte count; the others' copies may complete before it. feed:
// asked for the next ticket with the last tile.
template <class C>
__device__ __forceinline__ bool load_tiles(const PagedParams& p, const CUtensorMap& tmK, const CUtensorMap& tmV,
                                           const PagedSpan& span, int b, const PagedUnit& un, int j0, int j1, uint64_t* full,
                                           uint64_t* empty, uint8_t* sStage, int& c, int pw, int lane,
                                           volatile int* abort_flag, PagedFeed* feed = nullptr) {
  const int box = lane * 3 + pw, first = box * p.box_rows;  // this lane's box of a tile, its first key
  const uint32_t box_bytes = p.box_rows * 128;
  auto next_slot = [&](uint32_t bytes) -> int {
    const int slot = c % C::NST;
    if (!__all_sync(0xffffffffu, mbar_wait(&empty[slot], ((c / C::NST) & 1) ^ 1, abort_flag))) return -1;
    if (lane == 0) {
      if (pw == 0)
        mbar_arrive_expect_tx(&full[slot], bytes);
      else
        mbar_arrive(&full[slot]);
    }
    ++c;
    return slot;
  };
  auto copy = [&](const CUtensorMap* m, int slot, uint8_t* dst, int col, const PagedBox& x) {
    tma_load_4d(m, &full[slot], dst, col, p.slot_first ? x.slot : un.kvh, p.slot_first ? un.kvh : x.slot, x.page);
  };
  auto load_k = [&](const PagedBox& x, int key0) -> bool {
    const int boxes = paged_boxes(p, span, key0, 0, kTile);
    for (int kb = 0; kb < C::KST; ++kb) {
      const int atoms = C::k_atoms(kb), slot = next_slot(boxes * atoms * box_bytes);
      if (slot < 0) return false;
      uint8_t* dst = sStage + slot * kStage + first * 128;
      if (x.mine)
        for (int a = 0; a < atoms; ++a) copy(&tmK, slot, dst + a * 16384, kb * 128 + a * 64, x);
      __syncwarp();
    }
    return true;
  };
  auto load_v = [&](const PagedBox& x, int key0) -> bool {
    for (int vs = 0; vs < C::VST; ++vs) {
      const int slot = next_slot(paged_boxes(p, span, key0, vs * C::VROWS, (vs + 1) * C::VROWS) * (C::DV_ITEM / 64) * box_bytes);
      if (slot < 0) return false;
      uint8_t* dst = sStage + slot * kStage + (first - vs * C::VROWS) * 128;
      if (x.mine && first / C::VROWS == vs)
        for (int a = 0; a < C::DV_ITEM / 64; ++a) copy(&tmV, slot, dst + a * C::V_ATOM, un.split * C::DV_ITEM + a * 64, x);
      __syncwarp();
    }
    return true;
  };
  auto box_of = [&](int j) { return paged_box(p, span, b, (span.tile0 + j) * kTile, box); };
  PagedBox cur = box_of(j0), prev = cur;
#pragma unroll 1
  for (int j = j0; j < j1; ++j) {
    const PagedBox ahead = j + 1 < j1 ? box_of(j + 1) : cur;  // its table entry arrives while this tile's copies go out
    const int key0 = (span.tile0 + j) * kTile;
    if (feed && j + 1 == j1) feed->ask(p, lane);
    if (!load_k(cur, key0)) return false;
    if (!C::V_BEHIND) {
      if (!load_v(cur, key0)) return false;
    } else if (j > j0 && !load_v(prev, key0 - kTile)) {
      return false;
    }
    prev = cur;
    cur = ahead;
  }
  return !C::V_BEHIND || load_v(prev, (span.tile0 + j1 - 1) * kTile);
}

}  // namespace sdpa
