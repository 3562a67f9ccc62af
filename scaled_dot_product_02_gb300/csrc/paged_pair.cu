// paged_pair.cu -- attention over a paged cache for chunks of many tokens at
// head_dim 128: as paged_chunk.cu, with items of 256 rows, two 128-row tiles of Q
// against one stream of key tiles. While one tile's softmax runs the tensor pipe
// works on the other's MMAs, which at this width (as many exponentials per MMA
// flop as it gets) one tile cannot overlap by itself; and each K and V tile that
// comes from the L2 serves 256 rows. (Two pipelines with an item and a ring of
// two stages each read 11.6 TB/s from the L2 at 1.25 PFLOP/s, which bound them.)
//
// 384 threads: warps 0-3 / 4-7 softmax and output of rows 0-127 / 128-255 (one
// thread per query row), warp 8 scheduler and TMA producer, warps 9 and 11 further
// producers, warp 10 TMEM allocator and MMA issuer. Half x has O at TMEM columns
// [256 x, 256 x + 128) and S / P behind it; within a half S_j, softmax_j and P V_j
// follow one another, and the issuer serves the two in turn, which keeps them
// half a period apart. A block of fewer tokens than one tile holds leaves the
// second half out.
//
// Measured, 32 query heads on 8 kv heads: 2048 tokens over 16384 keys 371 us, 1.39
// PFLOP/s (256 items on 152 SMs, two rounds); 8 x 1024 over 32768 2.6 ms, 1.68
// PFLOP/s; 2048 over 131072 2.72 ms, 1.60 PFLOP/s.
#include <algorithm>
#include <cuda.h>
#include <cuda_runtime.h>

#include "paged.cuh"
#include "row_pass.cuh"

namespace sdpa {

namespace {

struct PairCfg {
  static constexpr int THREADS = 384;
  static constexpr int Q_BYTES = 32768;                            // of one half
  static constexpr int KST = 1, VST = 1, DV_ITEM = 128, VROWS = 128, V_ATOM = 16384;
  static constexpr bool V_BEHIND = false;
  static constexpr int NST = 4;
  static constexpr int STG_BYTES = 8 * 2048;                       // per softmax warp: 32 rows x 64 bytes of output
  static constexpr int MISC = 1024;
  static constexpr int SMEM = 1024 + 2 * Q_BYTES + NST * kStage + STG_BYTES + MISC;
  static constexpr uint32_t TM_S = 128, TM_HALF = 256;
  static __device__ __forceinline__ constexpr int k_atoms(int) { return 2; }
  // two softmax warpgroups and the third out of 3 x 168, the registers the block is launched with
  static constexpr int REGS_SOFTMAX = 192, REGS_OTHER = 120;
  static_assert(2 * REGS_SOFTMAX + REGS_OTHER <= 3 * 168 && SMEM <= kSmemMax, "register split and tile plan");
};

template <bool BF16>
__global__ void __launch_bounds__(PairCfg::THREADS, 1)
    paged_pair_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const __grid_constant__ PagedParams p) {
  using C = PairCfg;
  using E = Elem<BF16>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sQ = smem;
  uint8_t* sStage = smem + 2 * C::Q_BYTES;
  uint8_t* stg = sStage + C::NST * kStage;
  uint64_t* full = reinterpret_cast<uint64_t*>(stg + C::STG_BYTES);
  uint64_t* empty = full + C::NST;
  uint64_t* bar_q = empty + C::NST;   // both halves' Q landed
  uint64_t* q_free = bar_q + 1;       // an item's last S is done: Q may be replaced
  uint64_t* bar_s = q_free + 1;       // [2] S_j of a half in TMEM
  uint64_t* bar_p = bar_s + 2;        // [2] its P_j in TMEM (and O rescaled)
  uint64_t* bar_o = bar_p + 2;        // [2] its last P V is done
  uint64_t* o_free = bar_o + 2;       // [2] its output has read O
  uint64_t* sched_full = o_free + 2;  // [2] a piece published
  uint64_t* sched_empty = sched_full + 2;
  uint64_t* bar_drain = sched_empty + 2;
  PagedScan* scan = reinterpret_cast<PagedScan*>(bar_drain + 1);
  PagedPiece* pieces = reinterpret_cast<PagedPiece*>(scan + 1);  // [2]
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(pieces + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int half_tokens = p.tokens / 2;  // tokens of one half
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NST; ++i) {
      mbar_init(&full[i], 3);  // every producer, so that none falls a phase behind
      mbar_init(&empty[i], 1);
    }
    mbar_init(bar_q, 1);
    mbar_init(q_free, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar_s[i], 1);
      mbar_init(&bar_p[i], 128);
      mbar_init(&bar_o[i], 1);
      mbar_init(&o_free[i], 128);
      mbar_init(&sched_full[i], 1);
      mbar_init(&sched_empty[i], 259);  // issuer, two producers, 256 softmax threads
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
  const PagedShares all = paged_scan<C::THREADS, false>(p, scan);
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  if (threadIdx.x == 0 && blockIdx.x == 0 && !all.fit) record_error(p.err, SDPA_ERR_BAD_SEQLENS);

  if (all.total == 0) {
    // no work: fall through to the end
  } else if (warp >= 8) {
    regs_dec<C::REGS_OTHER>();
    if (warp == 8) {
      // ---------------------------------------------------------- scheduler + producer
      if (lane == 0) {
        prefetch_tmap(&tmQ);
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
      }
      int c = 0, nq = 0, np = 0;
      bool ok = true;
      PagedFeed feed;
      feed.start(p, all.total, gridDim.x, true, lane);
      const PagedWalk& w = feed.w;
      while (true) {
        const int e = np & 1;
        if (!__all_sync(0xffffffffu, mbar_wait(&sched_empty[e], ((np >> 1) & 1) ^ 1, abort_flag))) {
          ok = false;
          break;
        }
        if (lane == 0) {
          pieces[e] = feed.piece(p);
          mbar_arrive(&sched_full[e]);
        }
        ++np;
        if (!feed.more) break;
        if (w.span.tiles > 0) {
          const PagedUnit un = paged_unit(p, w.unit);
          if (nq > 0 && !__all_sync(0xffffffffu, mbar_wait(q_free, (nq - 1) & 1, abort_flag))) {
            ok = false;
            break;
          }
          if (lane == 0) {
            const int halves = w.i1(p) - w.i0 >= half_tokens ? 2 : 1;
            mbar_arrive_expect_tx(bar_q, (uint32_t)(halves * p.q_box_rows * 256));
            for (int x = 0; x < halves; ++x)
              for (int a = 0; a < 2; ++a)
                tma_load_3d(&tmQ, bar_q, sQ + x * C::Q_BYTES + a * 16384, a * 64, un.head0,
                            w.s.row0 + w.i0 + x * half_tokens);
          }
          ++nq;
          ok = load_tiles<C>(p, tmK, tmV, w.span, w.b, un, w.j0, w.j1, full, empty, sStage, c, 0, lane, abort_flag,
                             feed.last() ? &feed : nullptr);
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
        for (int k = max(0, c - C::NST); k < c; ++k) mbar_wait_drain(&full[k % C::NST], (k / C::NST) & 1);
        if (nq > 0) mbar_wait_drain(bar_q, (nq - 1) & 1);
      }
    } else if (warp == 9 || warp == 11) {
      // ---------------------------------------------------------- further producers
      int c = 0, np = 0;
      bool ok = true;
      while (true) {
        const int e = np & 1;
        if (!__all_sync(0xffffffffu, mbar_wait(&sched_full[e], (np >> 1) & 1, abort_flag))) {
          ok = false;
          break;
        }
        const PagedPiece w = pieces[e];
        __syncwarp();
        if (lane == 0) mbar_arrive(&sched_empty[e]);
        ++np;
        if (w.row0 < 0) break;
        if (w.j1 == w.j0) continue;
        const PagedSpan span =
            paged_span(p, PagedSeq{w.row0, w.q_len, w.kv_len}, w.i0, min(w.i0 + p.tokens, w.q_len) - 1);
        ok = load_tiles<C>(p, tmK, tmV, span, w.b, paged_unit(p, w.unit), w.j0, w.j1, full, empty, sStage, c,
                           warp == 9 ? 1 : 2, lane, abort_flag);
        if (!ok) break;
      }
      if (lane == 0) {
        if (!ok) {
          *abort_flag = 1;
          record_error(p.err, SDPA_ERR_TIMEOUT);
        }
        for (int k = max(0, c - C::NST); k < c; ++k) mbar_wait_drain(&full[k % C::NST], (k / C::NST) & 1);
      }
    } else {
      // ---------------------------------------------------------- MMA issuer
      if (elect_one()) {
        constexpr uint32_t ID_S = idesc_f16(128, 128, BF16, false, false);
        constexpr uint32_t ID_O = idesc_f16(128, 128, BF16, false, true);
        const uint32_t q_base = smem_u32(sQ);
        int np = 0, c = 0, nq = 0;            // pieces, ring stages, Q loads
        int pv[2] = {0, 0}, no[2] = {0, 0};   // of a half: P V MMAs, items done
        bool ok = true;
        while (ok) {
          const int e = np & 1;
          if (!mbar_wait(&sched_full[e], (np >> 1) & 1, abort_flag)) {
            ok = false;
            break;
          }
          const PagedPiece w = pieces[e];
          mbar_arrive(&sched_empty[e]);
          ++np;
          if (w.row0 < 0) break;
          const int n = w.j1 - w.j0;
          if (n == 0) continue;
          const int halves = min(w.q_len - w.i0, p.tokens) > half_tokens ? 2 : 1;
          if (!mbar_wait(bar_q, nq & 1, abort_flag)) {
            ok = false;
            break;
          }
          ++nq;
          tc_fence_after();
          // tile j is at ring stages c + 2 j (K) and c + 2 j + 1 (V)
          auto landed = [&](int stage) {
            if (!mbar_wait(&full[stage % C::NST], (stage / C::NST) & 1, abort_flag)) return false;
            tc_fence_after();
            return true;
          };
          auto issue_s = [&](int x, int j) {  // S = Q_x K_j^T
            const uint32_t base = smem_u32(sStage + ((c + 2 * j) % C::NST) * kStage), qa = q_base + x * C::Q_BYTES;
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
              const uint32_t off = (ks >> 2) * 16384 + (ks & 3) * 32;
              mma_ss(tmem + x * C::TM_HALF + C::TM_S, smem_desc_sw128(qa + off, 16, 1024),
                     smem_desc_sw128(base + off, 16, 1024), ID_S, ks != 0);
            }
            mma_commit(&bar_s[x]);
            if (x == halves - 1) {  // both halves have used K_j
              mma_commit(&empty[(c + 2 * j) % C::NST]);
              if (j == n - 1) mma_commit(q_free);
            }
          };
          auto issue_pv = [&](int x, int j) {  // O_x += P V_j
            const uint32_t base = smem_u32(sStage + ((c + 2 * j + 1) % C::NST) * kStage);
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              mma_ts(tmem + x * C::TM_HALF, tmem + x * C::TM_HALF + C::TM_S + ks * 8,
                     smem_desc_sw128(base + ks * 2048, 16384, 1024), ID_O, (j | ks) != 0);
            if (x == halves - 1) mma_commit(&empty[(c + 2 * j + 1) % C::NST]);
            if (j == n - 1) mma_commit(&bar_o[x]);
          };
          ok = landed(c);
#pragma unroll
          for (int x = 0; x < 2; ++x)
            if (ok && x < halves) issue_s(x, 0);
          for (int j = 0; ok && j < n; ++j) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              if (!ok || x >= halves) continue;
              // an item's first P V overwrites O, which the output before must have read
              if (j == 0 && no[x] > 0 && !mbar_wait(&o_free[x], (no[x] - 1) & 1, abort_flag)) ok = false;
              if (ok && !mbar_wait(&bar_p[x], pv[x] & 1, abort_flag)) ok = false;
              ++pv[x];
              if (!ok || !landed(c + 2 * j + 1)) {
                ok = false;
                continue;
              }
              issue_pv(x, j);
              // the next S of this half: its P has been issued, so the columns are free behind it
              if (j + 1 < n) {
                ok = landed(c + 2 * j + 2);
                if (ok) issue_s(x, j + 1);
              } else {
                ++no[x];
              }
            }
          }
          c += 2 * n;
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
    // ------------------------------------------------------------ softmax + output of half warp / 4
    const int x = warp >> 2;
    const int r = (warp & 3) * 32 + lane;  // row of the half, and key of a tile
    const uint32_t lanes = tmem + x * C::TM_HALF + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t scol = lanes + C::TM_S;
    const float sl2 = p.scale_log2;
    int np = 0, tiles = 0, no = 0, c = 0;  // pieces, tiles and items of this half, ring stages
    bool ok = true;
    while (ok) {
      const int e = np & 1;
      if (!__all_sync(0xffffffffu, mbar_wait(&sched_full[e], (np >> 1) & 1, abort_flag))) {
        ok = false;
        break;
      }
      int lo, hi, lo_last, hi_first, kb0, n, span_lo, span_hi;
      bool valid;
      long long out_row;  // row x head of the output
      float* part;        // the item's partial result, or nullptr: the whole item
      int part_row;
      {
        const PagedPiece w = pieces[e];
        __syncwarp();
        mbar_arrive(&sched_empty[e]);
        ++np;
        if (w.row0 < 0) break;
        const int i1 = min(w.i0 + p.tokens, w.q_len) - 1;
        const PagedSpan span = paged_span(p, PagedSeq{w.row0, w.q_len, w.kv_len}, w.i0, i1);
        const PagedUnit un = paged_unit(p, w.unit);
        const int ti = r / p.block_heads, h = r - ti * p.block_heads;
        const int h0 = w.i0 + x * half_tokens, h1 = min(i1, h0 + half_tokens - 1);  // tokens of this half
        const int off = w.kv_len - w.q_len, i = h0 + ti;
        n = w.j1 - w.j0;
        if (h0 > i1) {  // none in this half
          c += 2 * n;
          continue;
        }
        valid = i <= h1 && h < un.heads;
        // keys of this row's token, and of the half's last and first
        lo = p.window >= 0 ? max(0, i + off - p.window) : 0;
        hi = p.causal ? min(w.kv_len, max(0, i + off + 1)) : w.kv_len;
        lo_last = p.window >= 0 ? max(0, h1 + off - p.window) : 0;
        hi_first = p.causal ? max(0, h0 + off + 1) : w.kv_len;
        span_lo = span.lo;
        span_hi = span.hi;
        kb0 = (span.tile0 + w.j0) * kTile;
        out_row = (long long)(w.row0 + i) * p.hq + un.head0 + h;
        part = w.slot < 0 ? nullptr : p.parts + (long long)w.slot * (256 * 130);
        part_row = x * half_tokens * p.block_heads + r;
      }
      float mbs = -INFINITY, l = 0.f;  // running maximum of S * scale * log2 e, and the sum
      for (int j = 0; j < n; ++j) {
        if (!__all_sync(0xffffffffu, mbar_wait(&bar_s[x], tiles & 1, abort_flag))) {
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
        // (unused slots): zeros in their place keep 0 x NaN out. The first half's warps
        // write them, ahead of its P V and so of the second's. (The slot's use before was
        // V of an earlier tile, which both halves were done with when this S was formed.)
        if (x == 0 && (kb < span_lo || kb + kTile > span_hi)) {
          const int cv = c + 2 * j + 1;
          if (!__all_sync(0xffffffffu, mbar_wait(&full[cv % C::NST], (cv / C::NST) & 1, abort_flag))) {
            ok = false;
            break;
          }
          if (kb + r < span_lo || kb + r >= span_hi) {
            uint8_t* v = sStage + (cv % C::NST) * kStage + r * 128;
#pragma unroll
            for (int y = 0; y < 16; ++y)
              *reinterpret_cast<uint4*>(v + (y >> 3) * 16384 + (((y + r) & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        ++tiles;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&bar_p[x]);
      }
      if (!ok) break;
      c += 2 * n;
      const float inv = part ? 1.f : (l == 0.f ? 0.f : 1.f / l);
      if (n > 0) {
        if (!__all_sync(0xffffffffu, mbar_wait(&bar_o[x], no & 1, abort_flag))) {
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
            mbar_arrive(&o_free[x]);
          }
        } else {
#pragma unroll
          for (int k2 = 0; k2 < 32; ++k2) u[k2] = 0u;
        }
        if (part) {  // the same for the whole half
          float* at = part + part_row * 128 + cc * 32;
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
        } else if (SDPA_ADDR_OK(p.chk, part + 256 * 128 + part_row, 4) &&
                   SDPA_ADDR_OK(p.chk, part + 256 * 129 + part_row, 4)) {
          part[256 * 128 + part_row] = mbs;
          part[256 * 129 + part_row] = l;
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
int launch_pair_t(const PagedLaunch& L, int* launches) {
  auto kern = paged_pair_kernel<BF16>;
  if (const int rc = set_kernel_smem(reinterpret_cast<const void*>(kern), PairCfg::SMEM, 100)) return rc;
  if (const int rc = launch_early(kern, dim3((unsigned)L.workers), PairCfg::THREADS, PairCfg::SMEM, L.stream,
                                  L.p.behind != 0, L.tmQ, L.tmK, L.tmV, L.p))
    return rc;
  ++*launches;
  if (!L.p.tail) return SDPA_OK;  // no item crosses a cut
  ++*launches;
  return launch_paged_join(L, 256, 128, L.p.tail, BF16);
}

}  // namespace

int launch_paged_pair(const PagedLaunch& L, bool bf16, int* launches) {
  return bf16 ? launch_pair_t<true>(L, launches) : launch_pair_t<false>(L, launches);
}

}  // namespace sdpa
