// paged_pair.cu -- attention over a paged cache for chunks of many tokens at
// head_dim 128: as paged_chunk.cu, with two items in flight per CTA. One item's
// softmax runs while the tensor pipe works on the other's MMAs, which at this
// width (as many exponentials per MMA flop as it gets) one item cannot overlap
// by itself.
//
// 384 threads: warps 0-3 / 4-7 softmax and output of pipeline 0 / 1 (one thread
// per query row), warps 8 / 9 their schedulers and TMA producers, warp 10 TMEM
// allocator and MMA issuer for both, warp 11 completes its warpgroup. Pipeline
// x has O at TMEM columns [256 x, 256 x + 128) and S / P behind it; within a
// pipeline S_j, softmax_j and P V_j follow one another, and the issuer serves
// the two strictly in turn, which keeps them half a period apart.
#include <algorithm>
#include <cuda.h>
#include <cuda_runtime.h>

#include "paged.cuh"
#include "row_pass.cuh"

namespace sdpa {

namespace {

struct PairCfg {
  static constexpr int THREADS = 384;
  static constexpr int Q_BYTES = 32768;
  static constexpr int NST = 2;
  static constexpr int PIPE_BYTES = Q_BYTES + NST * kStage;
  static constexpr int PIPE_BARS = 16;                             // mbarriers of a pipeline
  static constexpr int STG_BYTES = 8 * 2048;                       // per softmax warp: 32 rows x 64 bytes of output
  static constexpr int SMEM = 1024 + 2 * PIPE_BYTES + 2 * PIPE_BARS * 8 + STG_BYTES + 1024;
  static constexpr uint32_t TM_S = 128, TM_PIPE = 256;
  // two softmax warpgroups and the third out of 3 x 168, the registers the block is launched with
  static constexpr int REGS_SOFTMAX = 192, REGS_OTHER = 120;
  static_assert(2 * REGS_SOFTMAX + REGS_OTHER <= 3 * 168 && SMEM <= kSmemMax, "register split and tile plan");
};

// Shared-memory objects of one pipeline.
struct Pipe {
  uint8_t *sQ, *sStage;
  uint64_t* full;         // [NST]
  uint64_t* empty;        // [NST]
  uint64_t* bar_q;        // Q landed
  uint64_t* bar_s;        // S_j in TMEM
  uint64_t* bar_p;        // P_j in TMEM (and O rescaled)
  uint64_t* bar_o;        // an item's last P V is done
  uint64_t* q_free;       // an item's last S is done: Q may be replaced
  uint64_t* o_free;       // the output has read O
  uint64_t* sched_full;   // [2] a piece published
  uint64_t* sched_empty;  // [2] read by the issuer and the softmax warps
  PagedPiece* pieces;     // [2]
};
__device__ __forceinline__ Pipe pipe_of(uint8_t* smem, PagedPiece* pieces, int x) {
  using C = PairCfg;
  Pipe P;
  P.sQ = smem + x * C::PIPE_BYTES;
  P.sStage = P.sQ + C::Q_BYTES;
  uint64_t* b = reinterpret_cast<uint64_t*>(smem + 2 * C::PIPE_BYTES) + x * C::PIPE_BARS;
  P.full = b;
  P.empty = b + C::NST;
  P.bar_q = b + 2 * C::NST;
  P.bar_s = P.bar_q + 1;
  P.bar_p = P.bar_q + 2;
  P.bar_o = P.bar_q + 3;
  P.q_free = P.bar_q + 4;
  P.o_free = P.bar_q + 5;
  P.sched_full = P.bar_q + 6;
  P.sched_empty = P.bar_q + 8;
  P.pieces = pieces + 2 * x;
  return P;
}

template <bool BF16>
__global__ void __launch_bounds__(PairCfg::THREADS, 1)
    paged_pair_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const __grid_constant__ PagedParams p,
                      const int pipes) {
  using C = PairCfg;
  using E = Elem<BF16>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* stg = smem + 2 * C::PIPE_BYTES + 2 * C::PIPE_BARS * 8;
  PagedScan* scan = reinterpret_cast<PagedScan*>(stg + C::STG_BYTES);
  PagedPiece* pieces = reinterpret_cast<PagedPiece*>(scan + 1);  // [2][2]
  uint64_t* bar_drain = reinterpret_cast<uint64_t*>(pieces + 4);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bar_drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (threadIdx.x == 0) {
    for (int x = 0; x < 2; ++x) {
      const Pipe P = pipe_of(smem, pieces, x);
      for (int i = 0; i < C::NST; ++i) {
        mbar_init(&P.full[i], 1);
        mbar_init(&P.empty[i], 1);
      }
      mbar_init(P.bar_q, 1);
      mbar_init(P.bar_s, 1);
      mbar_init(P.bar_p, 128);
      mbar_init(P.bar_o, 1);
      mbar_init(P.q_free, 1);
      mbar_init(P.o_free, 128);
      for (int i = 0; i < 2; ++i) {
        mbar_init(&P.sched_full[i], 1);
        mbar_init(&P.sched_empty[i], 129);
      }
    }
    mbar_init(bar_drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 10) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  const PagedShares all = paged_scan<C::THREADS>(p, scan, 0, 0, 0, 1);
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  if (threadIdx.x == 0 && blockIdx.x == 0 && !all.fit) record_error(p.err, SDPA_ERR_BAD_SEQLENS);

  if (all.total == 0) {
    // no work: fall through to the end
  } else if (warp >= 8) {
    regs_dec<C::REGS_OTHER>();
    if (warp == 8 || warp == 9) {
      // ---------------------------------------------------------- scheduler + producer of pipeline warp - 8
      const Pipe P = pipe_of(smem, pieces, warp - 8);
      if (lane == 0) {
        prefetch_tmap(&tmQ);
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
      }
      const uint32_t box_bytes = p.box_rows * 128;
      int c = 0, nq = 0, np = 0;
      bool ok = true;
      PagedFeed feed;
      // pipeline x of CTA c is pipeline x * gridDim.x + c
      feed.start(p, all.total, pipes, (warp - 8) * (int)gridDim.x + (int)blockIdx.x < pipes, lane);
      const PagedWalk& w = feed.w;
      while (true) {
        const int e = np & 1;
        if (!__all_sync(0xffffffffu, mbar_wait(&P.sched_empty[e], ((np >> 1) & 1) ^ 1, abort_flag))) {
          ok = false;
          break;
        }
        if (lane == 0) {
          P.pieces[e] = feed.piece(p);
          mbar_arrive(&P.sched_full[e]);
        }
        ++np;
        if (!feed.more) break;
        if (w.span.tiles > 0) {
          const PagedUnit un = paged_unit(p, w.unit);
          if (nq > 0 && !__all_sync(0xffffffffu, mbar_wait(P.q_free, (nq - 1) & 1, abort_flag))) {
            ok = false;
            break;
          }
          if (lane == 0) {
            mbar_arrive_expect_tx(P.bar_q, (uint32_t)p.q_box_rows * 256);
            tma_load_3d(&tmQ, P.bar_q, P.sQ, 0, un.head0, w.s.row0 + w.i0);
            tma_load_3d(&tmQ, P.bar_q, P.sQ + 16384, 64, un.head0, w.s.row0 + w.i0);
          }
          ++nq;
          auto box_of = [&](int j) { return paged_box(p, w.span, w.b, (w.span.tile0 + j) * kTile, lane); };
          PagedIds cur = paged_ids(box_of(w.j0));
          for (int j = w.j0; j < w.j1 && ok; ++j) {
            PagedBox ahead;  // its table entry arrives while this tile's copies go out
            if (j + 1 < w.j1)
              ahead = box_of(j + 1);
            else if (feed.last())
              feed.ask(p, lane);
            const uint32_t bytes = paged_boxes(p, w.span, (w.span.tile0 + j) * kTile, 0, kTile) * 2 * box_bytes;
            for (int kv = 0; kv < 2; ++kv, ++c) {
              const int slot = c % C::NST;
              if (!__all_sync(0xffffffffu, mbar_wait(&P.empty[slot], ((c / C::NST) & 1) ^ 1, abort_flag))) {
                ok = false;
                break;
              }
              // one thread issues: with two stages a pipeline, the time that the copies take to go out is on
              // the way of the next S (issued by the lanes that hold the boxes they are serialised at some
              // 100 cycles each)
              if (elect_one()) {
                mbar_arrive_expect_tx(&P.full[slot], bytes);
                paged_copy128(p, kv ? &tmV : &tmK, &P.full[slot], P.sStage + slot * kStage, un.kvh, cur);
              }
              __syncwarp();
            }
            if (j + 1 < w.j1) cur = paged_ids(ahead);
          }
          if (!ok) break;
        }
        feed.next(p, lane);
      }
      if (lane == 0) {
        if (!ok) {
          *abort_flag = 1;
          record_error(p.err, SDPA_ERR_TIMEOUT);
        }
        // every copy lands before the CTA ends
        for (int k = max(0, c - C::NST); k < c; ++k) mbar_wait_drain(&P.full[k % C::NST], (k / C::NST) & 1);
        if (nq > 0) mbar_wait_drain(P.bar_q, (nq - 1) & 1);
      }
    } else if (warp == 10) {
      // ---------------------------------------------------------- MMA issuer for both pipelines
      if (elect_one()) {
        constexpr uint32_t ID_S = idesc_f16(128, 128, BF16, false, false);
        constexpr uint32_t ID_O = idesc_f16(128, 128, BF16, false, true);
        struct State {
          int np, c, nq, tiles, no, n, j;  // pieces, ring stages, Q loads, P V MMAs, items done; this item's tiles, tile
          bool done;
        };
        State st[2];
        for (int x = 0; x < 2; ++x) st[x] = State{0, 0, 0, 0, 0, 0, 0, false};
        bool ok = true;
        // next piece with keys of pipeline x (false: its work is out, or a wait failed)
        auto next_item = [&](int x) -> bool {
          const Pipe P = pipe_of(smem, pieces, x);
          State& m = st[x];
          while (true) {
            const int e = m.np & 1;
            if (!mbar_wait(&P.sched_full[e], (m.np >> 1) & 1, abort_flag)) {
              ok = false;
              return false;
            }
            const bool end = P.pieces[e].row0 < 0;
            const int n = P.pieces[e].j1 - P.pieces[e].j0;
            mbar_arrive(&P.sched_empty[e]);
            ++m.np;
            if (end) {
              m.done = true;
              return false;
            }
            if (n == 0) continue;
            if (!mbar_wait(P.bar_q, m.nq & 1, abort_flag)) {
              ok = false;
              return false;
            }
            ++m.nq;
            tc_fence_after();
            m.n = n;
            m.j = 0;
            return true;
          }
        };
        // S_j = Q K_j^T of pipeline x (its previous P V has been issued, so P_{j-1} is consumed first)
        auto issue_s = [&](int x) -> bool {
          const Pipe P = pipe_of(smem, pieces, x);
          State& m = st[x];
          const int slot = m.c % C::NST;
          if (!mbar_wait(&P.full[slot], (m.c / C::NST) & 1, abort_flag)) return false;
          tc_fence_after();
          const uint32_t q_base = smem_u32(P.sQ), base = smem_u32(P.sStage + slot * kStage);
#pragma unroll
          for (int ks = 0; ks < 8; ++ks) {
            const uint32_t off = (ks >> 2) * 16384 + (ks & 3) * 32;
            mma_ss(tmem + x * C::TM_PIPE + C::TM_S, smem_desc_sw128(q_base + off, 16, 1024),
                   smem_desc_sw128(base + off, 16, 1024), ID_S, ks != 0);
          }
          mma_commit(&P.empty[slot]);
          if (m.j == m.n - 1) mma_commit(P.q_free);
          mma_commit(P.bar_s);
          ++m.c;
          return true;
        };
        // O += P_j V_j of pipeline x; an item's first one overwrites O, which the output before must have read
        auto issue_pv = [&](int x) -> bool {
          const Pipe P = pipe_of(smem, pieces, x);
          State& m = st[x];
          if (m.j == 0 && m.no > 0 && !mbar_wait(P.o_free, (m.no - 1) & 1, abort_flag)) return false;
          if (!mbar_wait(P.bar_p, m.tiles & 1, abort_flag)) return false;
          ++m.tiles;
          const int slot = m.c % C::NST;
          if (!mbar_wait(&P.full[slot], (m.c / C::NST) & 1, abort_flag)) return false;
          tc_fence_after();
          const uint32_t base = smem_u32(P.sStage + slot * kStage);
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            mma_ts(tmem + x * C::TM_PIPE, tmem + x * C::TM_PIPE + C::TM_S + ks * 8,
                   smem_desc_sw128(base + ks * 2048, 16384, 1024), ID_O, (m.j | ks) != 0);
          mma_commit(&P.empty[slot]);
          ++m.c;
          return true;
        };
        for (int x = 0; x < 2 && ok; ++x)
          if (next_item(x) && !issue_s(x)) ok = false;
        while (ok && !(st[0].done && st[1].done)) {
          for (int x = 0; x < 2 && ok; ++x) {
            State& m = st[x];
            if (m.done) continue;
            if (!issue_pv(x)) {
              ok = false;
              break;
            }
            if (m.j == m.n - 1) {
              mma_commit(pipe_of(smem, pieces, x).bar_o);
              ++m.no;
              if (!next_item(x)) continue;  // out of work (or ok cleared)
            } else {
              ++m.j;
            }
            if (!issue_s(x)) ok = false;
          }
        }
        if (!ok) {
          *abort_flag = 1;
          record_error(p.err, SDPA_ERR_TIMEOUT);
          mma_commit(bar_drain);  // every MMA issued so far ends before TMEM is released
          mbar_wait_drain(bar_drain, 0);
        }
      }
    }
  } else {
    regs_inc<C::REGS_SOFTMAX>();
    // ------------------------------------------------------------ softmax + output of pipeline warp / 4
    const int x = warp >> 2;
    const Pipe P = pipe_of(smem, pieces, x);
    const int r = (warp & 3) * 32 + lane;  // row of the item, and key of a tile
    const uint32_t lanes = tmem + x * C::TM_PIPE + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t scol = lanes + C::TM_S;
    const float sl2 = p.scale_log2;
    int np = 0, tiles = 0, no = 0;
    bool ok = true;
    while (ok) {
      const int e = np & 1;
      if (!__all_sync(0xffffffffu, mbar_wait(&P.sched_full[e], (np >> 1) & 1, abort_flag))) {
        ok = false;
        break;
      }
      int lo, hi, lo_last, hi_first, kb0, n, span_lo, span_hi;
      bool valid;
      long long out_row;  // row x head of the output
      float* part;        // this row's partial result, or nullptr: the whole item
      {
        const PagedPiece w = P.pieces[e];
        __syncwarp();
        mbar_arrive(&P.sched_empty[e]);
        ++np;
        if (w.row0 < 0) break;
        const int i1 = min(w.i0 + p.tokens, w.q_len) - 1;
        const PagedSpan span = paged_span(p, PagedSeq{w.row0, w.q_len, w.kv_len}, w.i0, i1);
        const PagedUnit un = paged_unit(p, w.unit);
        const int ti = r / p.block_heads, h = r - ti * p.block_heads;
        const int off = w.kv_len - w.q_len, i = w.i0 + ti;
        valid = i <= i1 && h < un.heads;
        // keys of this row's token, and of the block's last and first
        lo = p.window >= 0 ? max(0, i + off - p.window) : 0;
        hi = p.causal ? min(w.kv_len, max(0, i + off + 1)) : w.kv_len;
        lo_last = p.window >= 0 ? max(0, i1 + off - p.window) : 0;
        hi_first = p.causal ? max(0, w.i0 + off + 1) : w.kv_len;
        span_lo = span.lo;
        span_hi = span.hi;
        kb0 = (span.tile0 + w.j0) * kTile;
        n = w.j1 - w.j0;
        out_row = (long long)(w.row0 + i) * p.hq + un.head0 + h;
        part = w.slot < 0 ? nullptr
                          : p.parts + (long long)w.slot * (128 * 130);
      }
      float mbs = -INFINITY, l = 0.f;  // running maximum of S * scale * log2 e, and the sum
      for (int j = 0; j < n; ++j) {
        if (!__all_sync(0xffffffffu, mbar_wait(P.bar_s, tiles & 1, abort_flag))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const int kb = kb0 + j * kTile;
        const bool interior = lo_last <= kb && hi_first >= kb + kTile;
        // One pass against the running maximum; while no P exceeds 2^8 the maximum stays. A row whose scores jumped
        // higher, or that sees its first key, is recomputed against its new one (S is intact until P is written).
        const float mb = mbs == -INFINITY ? 0.f : mbs;
        float rs = 0.f, tmax = -INFINITY;
        uint32_t pk[64];
        if (interior)
          p_pass<false, E>(scol, sl2, mb, kb, lo, hi, pk, rs, tmax);
        else
          p_pass<true, E>(scol, sl2, mb, kb, lo, hi, pk, rs, tmax);
        const bool redo = tmax > 8.f || (mbs == -INFINITY && tmax > -INFINITY);
        float f = 1.f;
        if (__any_sync(0xffffffffu, redo)) {
          const float mb2 = redo ? mb + tmax : mb;
          float t2 = -INFINITY;
          if (interior)
            p_pass<false, E>(scol, sl2, mb2, kb, lo, hi, pk, rs, t2);
          else
            p_pass<true, E>(scol, sl2, mb2, kb, lo, hi, pk, rs, t2);
        }
        if (redo) {
          f = mbs == -INFINITY ? 0.f : ex2(-tmax);
          mbs = mb + tmax;
        }
        l = l * f + rs;
#pragma unroll
        for (int cc = 0; cc < 4; ++cc) {
          uint32_t q16[16];
#pragma unroll
          for (int k2 = 0; k2 < 16; ++k2) q16[k2] = pk[cc * 16 + k2];
          tmem_st16(scol + cc * 16, q16);
        }
        // P V of the tile before completed before this S was computed: O can be rescaled
        if (__any_sync(0xffffffffu, f != 1.f) && j > 0) {
#pragma unroll 1
          for (int cc = 0; cc < 4; ++cc) {
            uint32_t u[32];
            tmem_ld32(lanes + cc * 32, u);
            tmem_wait_ld();
            reg_fence(u);
#pragma unroll
            for (int k2 = 0; k2 < 32; ++k2) u[k2] = __float_as_uint(__uint_as_float(u[k2]) * f);
            tmem_st32(lanes + cc * 32, u);
          }
        }
        // keys that no row of the item sees have P = 0, but their values may be anything
        // (unused slots): zeros in their place keep 0 x NaN out. V is in the slot behind
        // K's, whose use before was the V that the P V before consumed.
        if (kb < span_lo || kb + kTile > span_hi) {
          const int cv = 2 * tiles + 1, slot = cv % C::NST;
          if (!__all_sync(0xffffffffu, mbar_wait(&P.full[slot], (cv / C::NST) & 1, abort_flag))) {
            ok = false;
            break;
          }
          if (kb + r < span_lo || kb + r >= span_hi) {
            uint8_t* v = P.sStage + slot * kStage + r * 128;
#pragma unroll
            for (int y = 0; y < 16; ++y)
              *reinterpret_cast<uint4*>(v + (y >> 3) * 16384 + (((y + r) & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        ++tiles;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(P.bar_p);
      }
      if (!ok) break;
      const float inv = part ? 1.f : (l == 0.f ? 0.f : 1.f / l);
      if (n > 0) {
        if (!__all_sync(0xffffffffu, mbar_wait(P.bar_o, no & 1, abort_flag))) {
          ok = false;
          break;
        }
        ++no;
        tc_fence_after();
      }
      // 32 columns (64 bytes of a row) at a time, staged in shared memory so
      // that each store writes eight rows' 64 contiguous bytes
      uint8_t* wst = stg + warp * 2048;
#pragma unroll 1
      for (int cc = 0; cc < 4; ++cc) {
        uint32_t u[32];
        if (n > 0) {
          tmem_ld32(lanes + cc * 32, u);
          tmem_wait_ld();
          reg_fence(u);
          if (cc == 3) {
            tc_fence_before();
            mbar_arrive(P.o_free);
          }
        } else {
#pragma unroll
          for (int k2 = 0; k2 < 32; ++k2) u[k2] = 0u;
        }
        if (part) {  // the same for the whole CTA's pipeline
          float* at = part + r * 128 + cc * 32;
          if (valid && SDPA_ADDR_OK(p.chk, at, 128)) {
#pragma unroll
            for (int k2 = 0; k2 < 8; ++k2)
              reinterpret_cast<uint4*>(at)[k2] = make_uint4(u[4 * k2], u[4 * k2 + 1], u[4 * k2 + 2], u[4 * k2 + 3]);
          }
          continue;
        }
        // segment k2 of row `lane` at position k2 ^ (lane % 4): four wavefronts a store
#pragma unroll
        for (int k2 = 0; k2 < 4; ++k2) {
          uint32_t v[4];
#pragma unroll
          for (int y = 0; y < 4; ++y)
            v[y] = E::pack(__uint_as_float(u[8 * k2 + 2 * y]) * inv, __uint_as_float(u[8 * k2 + 2 * y + 1]) * inv);
          *reinterpret_cast<uint4*>(wst + lane * 64 + ((k2 ^ (lane & 3)) << 4)) = make_uint4(v[0], v[1], v[2], v[3]);
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int rr = k * 8 + (lane >> 2), seg = lane & 3;  // row of the warp, 16-byte segment
          const uint4 v4 = *reinterpret_cast<const uint4*>(wst + rr * 64 + ((seg ^ (rr & 3)) << 4));
          const long long row = __shfl_sync(0xffffffffu, out_row, rr);
          const bool vr = __shfl_sync(0xffffffffu, valid ? 1 : 0, rr) != 0;
          typename E::T* dst = static_cast<typename E::T*>(p.o) + row * 128 + cc * 32 + seg * 8;
          if (vr && SDPA_ADDR_OK(p.chk, dst, 16)) *reinterpret_cast<uint4*>(dst) = v4;
        }
        __syncwarp();
      }
      if (valid) {
        if (!part) {
          float* at = p.lse + out_row;
          if (SDPA_ADDR_OK(p.chk, at, 4)) *at = l == 0.f ? -INFINITY : mbs * kLn2 + logf(l);
        } else if (SDPA_ADDR_OK(p.chk, part + 128 * 128 + r, 4) && SDPA_ADDR_OK(p.chk, part + 128 * 129 + r, 4)) {
          part[128 * 128 + r] = mbs;
          part[128 * 129 + r] = l;
        }
      }
    }
    if (!ok) {
      *abort_flag = 1;
      record_error(p.err, SDPA_ERR_TIMEOUT);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 10) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (p.behind && blockIdx.x == 0 && threadIdx.x == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <bool BF16>
int launch_pair_t(const PagedLaunch& L, int sms, int* launches) {
  auto kern = paged_pair_kernel<BF16>;
  if (const int rc = set_kernel_smem(reinterpret_cast<const void*>(kern), PairCfg::SMEM, 100)) return rc;
  const int grid = std::min(L.workers, sms);
  if (const int rc = launch_early(kern, dim3((unsigned)grid), PairCfg::THREADS, PairCfg::SMEM, L.stream, L.p.behind != 0,
                                  L.tmQ, L.tmK, L.tmV, L.p, L.workers))
    return rc;
  ++*launches;
  if (!L.p.tail) return SDPA_OK;  // no item crosses a cut
  ++*launches;
  return launch_paged_join(L, 128, 128, L.p.tail, BF16);
}

}  // namespace

int launch_paged_pair(const PagedLaunch& L, int sms, bool bf16, int* launches) {
  return bf16 ? launch_pair_t<true>(L, sms, launches) : launch_pair_t<false>(L, sms, launches);
}

}  // namespace sdpa
