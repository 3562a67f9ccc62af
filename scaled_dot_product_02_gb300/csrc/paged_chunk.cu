// paged_chunk.cu -- attention over a paged cache for sequences with many new
// tokens (chunks of a prompt) at head dims 192 to 512 (paged_pair.cu serves 128):
// the work is bound by the tensor pipe and by K and V on their way from the L2 (at
// 512 a tile of 192 KB for 128 rows). Measured, pages of 64: 4 x 1024 tokens over
// 32768 keys at head_dim 256 1.60 ms, 1.36 PFLOP/s, at 512 4.52 ms, 0.96 PFLOP/s; 2048
// over 16384 at 192/128 0.58 ms, 1.12 PFLOP/s (0.63 ms with pages of 32).
//
// An item is 128 query rows that share one kv head (tokens times the heads of
// its GQA group, so a tile of keys serves the whole group) and, for head_dim
// 512, one half of the value columns, which keeps O within 256 TMEM columns:
//   S = Q K^T (M = 128 rows, N = 128 keys),  O += P V (P from TMEM).
// CTAs take items from a ticket counter, the longest first; where items are few
// and long, the last ones are cut into equal shares of their key tiles and
// joined afterwards (PagedFeed in paged.cuh).
//
// Roles (256 threads): warp 0 scheduler and TMA producer, warps 2 and 3 further
// producers (each lane fetches one page's rows; a warp issues its lanes' copies
// one after another), warp 1 TMEM allocator and MMA issuer, warps 4-7 softmax
// and output, one thread per query row. The scheduler hands each piece of work
// to the others through a two-entry queue in shared memory.
#include <algorithm>
#include <cuda.h>
#include <cuda_runtime.h>

#include "paged.cuh"

namespace sdpa {

namespace {

template <int DQK, int DV>
struct ChunkCfg {
  static constexpr int THREADS = 256;
  static constexpr int KST = (DQK + 127) / 128;  // K stages of a tile (128 keys x up to 128 columns)
  static __device__ __forceinline__ constexpr int k_atoms(int kb) { return DQK / 64 - 2 * kb >= 2 ? 2 : 1; }
  static constexpr int DV_ITEM = DV;
  static constexpr bool V_BEHIND = true;           // V of a tile follows K of the next one in the ring
  static constexpr int VROWS = kStage / (DV * 2);  // keys of a V stage
  static constexpr int VST = kTile / VROWS;
  static constexpr int V_ATOM = VROWS * 128;       // bytes of 64 columns of a V stage
  static constexpr int Q_BYTES = DQK * 256;
  static constexpr int MISC = 1024;
  static constexpr int NST_FIT = (kSmemMax - 1024 - Q_BYTES - MISC) / kStage;
  static constexpr int NST = NST_FIT > 5 ? 5 : NST_FIT;
  static constexpr int SMEM = 1024 + Q_BYTES + NST * kStage + MISC;
  static constexpr int TM_S = DV;                  // TMEM columns: O, then two S / P buffers
  static_assert(SMEM <= kSmemMax && NST >= VST && DV + 256 <= 512, "the tile plan fits one SM");
};

template <int DQK, int DV, bool BF16>
__global__ void __launch_bounds__(256, 1)
    paged_chunk_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const __grid_constant__ PagedParams p) {
  using C = ChunkCfg<DQK, DV>;
  using E = Elem<BF16>;
  using T = typename E::T;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sQ = smem;
  uint8_t* sStage = smem + C::Q_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(sStage + C::NST * kStage);
  uint64_t* empty = full + C::NST;
  uint64_t* bar_q = empty + C::NST;
  uint64_t* bar_s = bar_q + 1;        // [2]
  uint64_t* bar_p = bar_s + 2;        // [2]
  uint64_t* bar_o = bar_p + 2;
  uint64_t* q_free = bar_o + 1;       // an item's last S is done: Q may be replaced
  uint64_t* o_free = q_free + 1;      // the output has read O
  uint64_t* sched_full = o_free + 1;  // [2]
  uint64_t* sched_empty = sched_full + 2;
  uint64_t* bar_drain = sched_empty + 2;
  PagedScan* scan = reinterpret_cast<PagedScan*>(bar_drain + 1);
  PagedPiece* pieces = reinterpret_cast<PagedPiece*>(scan + 1);  // [2]
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(pieces + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NST; ++i) {
      mbar_init(&full[i], 3);  // every producer, so that none falls a phase behind
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar_s[i], 1);
      mbar_init(&bar_p[i], 128);
      mbar_init(&sched_full[i], 1);
      mbar_init(&sched_empty[i], 131);  // issuer, two producers, 128 softmax threads
    }
    for (uint64_t* b : {bar_q, bar_o, q_free, bar_drain}) mbar_init(b, 1);
    mbar_init(o_free, 128);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  const int me = blockIdx.x;
  const PagedShares all = paged_scan<C::THREADS, false>(p, scan);
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  if (threadIdx.x == 0 && me == 0 && !all.fit) record_error(p.err, SDPA_ERR_BAD_SEQLENS);

  if (all.total > 0) {
    if (warp == 0) {
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
            mbar_arrive_expect_tx(bar_q, (uint32_t)p.q_box_rows * DQK * 2);
            for (int a = 0; a < DQK / 64; ++a)
              tma_load_3d(&tmQ, bar_q, sQ + a * 16384, a * 64, un.head0, w.s.row0 + w.i0);
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
    } else if (warp == 2 || warp == 3) {
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
        ok = load_tiles<C>(p, tmK, tmV, span, w.b, paged_unit(p, w.unit), w.j0, w.j1, full, empty, sStage, c, warp - 1, lane,
                           abort_flag);
        if (!ok) break;
      }
      if (lane == 0) {
        if (!ok) {
          *abort_flag = 1;
          record_error(p.err, SDPA_ERR_TIMEOUT);
        }
        for (int k = max(0, c - C::NST); k < c; ++k) mbar_wait_drain(&full[k % C::NST], (k / C::NST) & 1);
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------- MMA issuer
      if (elect_one()) {
        constexpr uint32_t ID_S = idesc_f16(128, 128, BF16, false, false);
        constexpr uint32_t ID_O = idesc_f16(128, DV, BF16, false, true);
        const uint32_t q_base = smem_u32(sQ);
        int c = 0, nq = 0, gs = 0, np = 0;  // ring stages, items with keys, tiles of earlier pieces, pieces
        bool ok = true;
        while (ok) {
          const int e = np & 1;
          if (!mbar_wait(&sched_full[e], (np >> 1) & 1, abort_flag)) {
            ok = false;
            break;
          }
          const bool end = pieces[e].row0 < 0;
          const int n = pieces[e].j1 - pieces[e].j0;
          mbar_arrive(&sched_empty[e]);
          ++np;
          if (end) break;
          if (n == 0) continue;
          if (!mbar_wait(bar_q, nq & 1, abort_flag)) {
            ok = false;
            break;
          }
          ++nq;
          tc_fence_after();
          auto mma_s = [&](int j) -> bool {
            const int sj = gs + j;
            const uint32_t d = tmem + C::TM_S + (sj & 1) * 128;
            for (int kb = 0; kb < C::KST; ++kb, ++c) {
              const int slot = c % C::NST;
              if (!mbar_wait(&full[slot], (c / C::NST) & 1, abort_flag)) return false;
              tc_fence_after();
              const uint32_t k_base = smem_u32(sStage + slot * kStage), qa = q_base + kb * 2 * 16384;
              const int steps = 4 * C::k_atoms(kb);
#pragma unroll
              for (int ks = 0; ks < 8; ++ks) {
                if (ks >= steps) break;
                const uint32_t off = (ks >> 2) * 16384 + (ks & 3) * 32;
                mma_ss(d, smem_desc_sw128(qa + off, 16, 1024), smem_desc_sw128(k_base + off, 16, 1024), ID_S,
                       (kb | ks) != 0);
              }
              mma_commit(&empty[slot]);
            }
            mma_commit(&bar_s[sj & 1]);
            if (j == n - 1) mma_commit(q_free);
            return true;
          };
          auto mma_o = [&](int j) -> bool {
            const int sj = gs + j;
            if (j == 0 && nq > 1 && !mbar_wait(o_free, (nq - 2) & 1, abort_flag)) return false;
            if (!mbar_wait(&bar_p[sj & 1], (sj >> 1) & 1, abort_flag)) return false;
            tc_fence_after();
            const uint32_t pcol = tmem + C::TM_S + (sj & 1) * 128;
            for (int vs = 0; vs < C::VST; ++vs, ++c) {
              const int slot = c % C::NST;
              if (!mbar_wait(&full[slot], (c / C::NST) & 1, abort_flag)) return false;
              tc_fence_after();
              const uint32_t v_base = smem_u32(sStage + slot * kStage);
#pragma unroll
              for (int ks = 0; ks < C::VROWS / 16; ++ks)
                mma_ts(tmem, pcol + (vs * C::VROWS + ks * 16) / 2,
                       smem_desc_sw128(v_base + ks * 2048, C::V_ATOM, 1024), ID_O, (j | vs | ks) != 0);
              mma_commit(&empty[slot]);
            }
            mma_commit(bar_o);
            return true;
          };
          for (int j = 0; j < n && ok; ++j) {
            ok = mma_s(j);
            if (ok && j >= 1) ok = mma_o(j - 1);
          }
          if (ok) ok = mma_o(n - 1);
          gs += n;
        }
        if (!ok) {
          *abort_flag = 1;
          record_error(p.err, SDPA_ERR_TIMEOUT);
          mma_commit(bar_drain);  // every MMA issued so far ends before TMEM is released
          mbar_wait_drain(bar_drain, 0);
        }
      }
    } else if (warp >= 4) {
      // ---------------------------------------------------------- softmax and output
      const int r = (warp - 4) * 32 + lane;  // row of the item, and key of a tile
      const uint32_t lanes = tmem + ((uint32_t)((warp - 4) * 32) << 16);
      const float sl2 = p.scale_log2;
      int gs = 0, c0 = 0, np = 0;  // tiles and ring stages of earlier pieces, pieces
      bool ok = true;
      while (ok) {
        const int e = np & 1;
        if (!__all_sync(0xffffffffu, mbar_wait(&sched_full[e], (np >> 1) & 1, abort_flag))) {
          ok = false;
          break;
        }
        const PagedPiece w = pieces[e];
        __syncwarp();
        mbar_arrive(&sched_empty[e]);
        ++np;
        if (w.row0 < 0) break;
        const PagedSeq seq{w.row0, w.q_len, w.kv_len};
        const int i1 = min(w.i0 + p.tokens, w.q_len) - 1;
        const PagedSpan span = paged_span(p, seq, w.i0, i1);
        const PagedUnit un = paged_unit(p, w.unit);
        const int ti = r / p.block_heads, h = r - ti * p.block_heads;
        const bool valid = w.i0 + ti <= i1 && h < un.heads;
        // keys of this row's token, and of the block's first and last
        const int off = w.kv_len - w.q_len, i = w.i0 + ti;
        const int lo = p.window >= 0 ? max(0, i + off - p.window) : 0;
        const int hi = p.causal ? min(w.kv_len, max(0, i + off + 1)) : w.kv_len;
        const int lo_last = p.window >= 0 ? max(0, i1 + off - p.window) : 0;
        const int hi_first = p.causal ? max(0, w.i0 + off + 1) : w.kv_len;
        const int n = w.j1 - w.j0;
        float m_used = -INFINITY, l = 0.f;
        for (int j = 0; j < n; ++j) {
          const int sj = gs + j;
          if (!__all_sync(0xffffffffu, mbar_wait(&bar_s[sj & 1], (sj >> 1) & 1, abort_flag))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t scol = lanes + C::TM_S + (sj & 1) * 128;
          float s[128];
          float mt;  // the tile's row maximum (the loads return it for an unmasked tile)
          {
            uint32_t u0[32], u1[32], u2[32], u3[32];
            float x0, x1, x2, x3;
            tmem_ld32_max(scol, u0, x0);
            tmem_ld32_max(scol + 32, u1, x1);
            tmem_ld32_max(scol + 64, u2, x2);
            tmem_ld32_max(scol + 96, u3, x3);
            tmem_wait_ld();
            reg_fence(u0);
            reg_fence(u1);
            reg_fence(u2);
            reg_fence(u3);
            asm volatile("" : "+f"(x0), "+f"(x1), "+f"(x2), "+f"(x3));
            mt = fmaxf(fmaxf(x0, x1), fmaxf(x2, x3));
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              s[k] = __uint_as_float(u0[k]);
              s[32 + k] = __uint_as_float(u1[k]);
              s[64 + k] = __uint_as_float(u2[k]);
              s[96 + k] = __uint_as_float(u3[k]);
            }
          }
          const int kb = (span.tile0 + w.j0 + j) * kTile;
          if (!(lo_last <= kb && hi_first >= kb + kTile)) {  // edge tile (uniform branch)
#pragma unroll
            for (int k = 0; k < 128; ++k) s[k] = in_range(kb + k, lo, hi) ? s[k] : -INFINITY;
            float mc[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
            for (int k = 4; k < 128; ++k) mc[k & 3] = fmaxf(mc[k & 3], s[k]);
            mt = fmaxf(fmaxf(mc[0], mc[1]), fmaxf(mc[2], mc[3]));
          }
          // O and the sum are rescaled only when the maximum grows by more than 2^8 (P stays <= 256)
          const float m_new = fmaxf(m_used, mt);
          bool need = false;
          float f = 1.f;
          if (m_used == -INFINITY) {
            m_used = m_new;
          } else if ((m_new - m_used) * sl2 > 8.f) {
            need = true;
            f = ex2((m_used - m_new) * sl2);
            m_used = m_new;
          }
          const float mb = m_used == -INFINITY ? 0.f : m_used * sl2;
          float rs = 0.f;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t pk[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const float p0 = ex2(fmaf(s[half * 64 + 2 * k], sl2, -mb));
              const float p1 = ex2(fmaf(s[half * 64 + 2 * k + 1], sl2, -mb));
              rs += p0 + p1;
              pk[k] = E::pack(p0, p1);
            }
            tmem_st32(scol + half * 32, pk);
          }
          l = l * f + rs;
          if (j >= 1) {
            // P V of the tile before is done before O is touched (and V's slots are looked at)
            if (!__all_sync(0xffffffffu, mbar_wait(bar_o, (sj - 1) & 1, abort_flag))) {
              ok = false;
              break;
            }
            tc_fence_after();
            if (__any_sync(0xffffffffu, need)) {
#pragma unroll 1
              for (int k = 0; k < DV / 32; ++k) {
                uint32_t u[32];
                tmem_ld32(lanes + k * 32, u);
                tmem_wait_ld();
                reg_fence(u);
#pragma unroll
                for (int x = 0; x < 32; ++x) u[x] = __float_as_uint(__uint_as_float(u[x]) * f);
                tmem_st32(lanes + k * 32, u);
              }
            }
          }
          // keys that no row of the item sees have P = 0, but their values may be
          // anything (unused slots): zeros in their place keep 0 x NaN out. A stage
          // barrier tells a phase from its neighbour only, so the K of the next tile,
          // which was copied ahead of this tile's V, must have been used.
          if (kb < span.lo || kb + kTile > span.hi) {
            if (j + 1 < n && !__all_sync(0xffffffffu, mbar_wait(&bar_s[(sj + 1) & 1], ((sj + 1) >> 1) & 1, abort_flag))) {
              ok = false;
              break;
            }
            const int cv = c0 + (j == n - 1 ? n * C::KST + (n - 1) * C::VST : (j + 2) * C::KST + j * C::VST);
            for (int vs = 0; vs < C::VST && ok; ++vs) {
              const int slot = (cv + vs) % C::NST;
              ok = __all_sync(0xffffffffu, mbar_wait(&full[slot], ((cv + vs) / C::NST) & 1, abort_flag));
              if (ok && r / C::VROWS == vs && (kb + r < span.lo || kb + r >= span.hi)) {
                uint8_t* v = sStage + slot * kStage + (r % C::VROWS) * 128;
                for (int a = 0; a < DV / 64; ++a)
#pragma unroll
                  for (int x = 0; x < 8; ++x)
                    *reinterpret_cast<uint4*>(v + a * C::V_ATOM + (((x + r) & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
              }
            }
            if (!ok) break;
            fence_proxy_async_smem();
          }
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(&bar_p[sj & 1]);
        }
        if (!ok) break;
        if (n > 0) {
          if (!__all_sync(0xffffffffu, mbar_wait(bar_o, (gs + n - 1) & 1, abort_flag))) {
            ok = false;
            break;
          }
          tc_fence_after();
        }
        const bool whole = w.slot < 0;
        const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
        const long long row = w.row0 + i;
        T* orow = static_cast<T*>(p.o) + (row * p.hq + un.head0 + h) * p.dv + un.split * DV;
        float* part = p.parts + (long long)(whole ? 0 : w.slot) * (128 * (DV + 2));
#pragma unroll 1
        for (int k = 0; k < DV / 32; ++k) {
          uint32_t u[32];
          if (n > 0) {
            tmem_ld32(lanes + k * 32, u);
            tmem_wait_ld();
            reg_fence(u);
            if (k == DV / 32 - 1) {  // all of O is read: the next item may overwrite it
              tc_fence_before();
              mbar_arrive(o_free);
            }
          } else {
#pragma unroll
            for (int x = 0; x < 32; ++x) u[x] = 0u;
          }
          if (!valid) continue;
          if (whole) {
            if (SDPA_ADDR_OK(p.chk, orow + k * 32, 64)) {
              uint4* dst = reinterpret_cast<uint4*>(orow + k * 32);
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                uint32_t v[4];
#pragma unroll
                for (int y = 0; y < 4; ++y)
                  v[y] = E::pack(__uint_as_float(u[8 * x + 2 * y]) * inv, __uint_as_float(u[8 * x + 2 * y + 1]) * inv);
                dst[x] = make_uint4(v[0], v[1], v[2], v[3]);
              }
            }
          } else if (SDPA_ADDR_OK(p.chk, part + r * DV + k * 32, 128)) {
            uint4* dst = reinterpret_cast<uint4*>(part + r * DV + k * 32);
#pragma unroll
            for (int x = 0; x < 8; ++x) dst[x] = make_uint4(u[4 * x], u[4 * x + 1], u[4 * x + 2], u[4 * x + 3]);
          }
        }
        if (valid) {
          const float m = m_used == -INFINITY ? -INFINITY : m_used * sl2;
          if (whole) {
            float* at = p.lse + row * p.hq + un.head0 + h;
            if (un.split == 0 && SDPA_ADDR_OK(p.chk, at, 4)) *at = l == 0.f ? -INFINITY : m * kLn2 + logf(l);
          } else if (SDPA_ADDR_OK(p.chk, part + 128 * DV + r, 4) && SDPA_ADDR_OK(p.chk, part + 128 * DV + 128 + r, 4)) {
            part[128 * DV + r] = m;
            part[128 * DV + 128 + r] = l;
          }
        }
        gs += n;
        c0 += n * (C::KST + C::VST);
      }
      if (!ok) {
        *abort_flag = 1;
        record_error(p.err, SDPA_ERR_TIMEOUT);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (p.behind && blockIdx.x == 0 && threadIdx.x == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <int DQK, int DV, bool BF16>
int launch_chunk_t(const PagedLaunch& L, int* launches) {
  using C = ChunkCfg<DQK, DV>;
  auto kern = paged_chunk_kernel<DQK, DV, BF16>;
  if (const int rc = set_kernel_smem(reinterpret_cast<const void*>(kern), C::SMEM, -1)) return rc;
  if (const int rc = launch_early(kern, dim3((unsigned)L.workers), C::THREADS, C::SMEM, L.stream, L.p.behind != 0, L.tmQ,
                                  L.tmK, L.tmV, L.p))
    return rc;
  ++*launches;
  if (!L.p.tail) return SDPA_OK;  // no item crosses a cut
  ++*launches;
  return launch_paged_join(L, 128, DV, L.p.tail, BF16);
}

}  // namespace

int launch_paged_chunk(const PagedLaunch& L, int head_dim, bool bf16, int* launches) {
#define CHUNK(A, B) return bf16 ? launch_chunk_t<A, B, true>(L, launches) : launch_chunk_t<A, B, false>(L, launches)
  if (head_dim == 192) CHUNK(192, 128);
  if (head_dim == 256) CHUNK(256, 256);
  if (head_dim == 512) CHUNK(512, 256);
#undef CHUNK
  return SDPA_ERR_UNSUPPORTED;
}

}  // namespace sdpa
