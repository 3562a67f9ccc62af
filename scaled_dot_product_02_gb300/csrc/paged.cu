// paged.cu -- attention of new tokens over a paged key/value cache.
//
// paged_rows_kernel serves few query rows per sequence (decoding, speculative
// tokens): the work is reading the cache, so it is bound by HBM. An item is
// the query rows that share one kv head -- up to N = 16, 32 or 64 rows, tokens
// times the heads of a GQA group -- against the keys they see, 128 at a time:
//   S^T = K Q^T     (M = 128 keys, N rows; K tile and Q in shared memory)
//   O^T += V^T P^T  (M = 128 value columns, N rows; V tile and P in shared memory)
// Keys on the M side keep the tensor work proportional to the rows there are
// (a 128-row query tile would be mostly padding), let all 128 softmax threads
// work on 16 to 64 scores each whatever the number of rows, and put O^T of a
// 512-wide head into 4 N TMEM columns.
//
// The key tiles of all items, laid end to end, are cut into one equal share
// per CTA (the lengths live on the device; every CTA adds them up itself), so
// ragged batches and a single long sequence both fill the machine. An item
// that crosses a cut leaves unnormalised fp32 partial results, at most two
// per CTA, which paged_join_kernel combines in a fixed order: results are
// bitwise reproducible.
//
// Roles (192 threads): warps 0-3 softmax and output, one thread per key of a
// tile (and per value column of the output); warp 4 TMA producer, its lanes
// each fetching one page's rows of a tile; warp 5 TMEM allocator and MMA
// issuer. K and V tiles go through a ring of 32 KB stages (128 keys x 128
// columns); S^T and P are double-buffered, so S^T of the next tile is formed
// while the softmax works on this one.
#include <algorithm>
#include <cuda.h>
#include <cuda_runtime.h>

#include "paged.cuh"

namespace sdpa {

namespace {

// ---------------------------------------------------------------- the kernel

template <int DQK, int DV, int N>
struct RowsCfg {
  static constexpr int THREADS = 192;
  static constexpr int KST = (DQK + 127) / 128;  // K stages of a tile
  static constexpr int VST = DV / 128;           // V stages of a tile
  static __device__ __forceinline__ constexpr int k_atoms(int kb) { return DQK / 64 - 2 * kb >= 2 ? 2 : 1; }
  static constexpr int Q_BYTES = N * DQK * 2;
  static constexpr int NQ = Q_BYTES <= 16384 ? 2 : 1;
  static constexpr int P_BYTES = kTile * N * 2;
  static constexpr int MISC = 1024 + 13 * N * 4 + 512;  // barriers and row statistics
  static constexpr int NST_FIT = (kSmemMax - 1024 - NQ * Q_BYTES - 2 * P_BYTES - MISC) / kStage;
  static constexpr int NST = NST_FIT > 6 ? 6 : NST_FIT;
  static constexpr int SMEM = 1024 + NQ * Q_BYTES + 2 * P_BYTES + NST * kStage + MISC;
  static constexpr int TM_S = VST * N;           // TMEM columns: O^T, then two S^T buffers
  static constexpr int TM_NEED = (VST + 2) * N;
  static constexpr int TM_COLS = TM_NEED <= 64 ? 64 : TM_NEED <= 128 ? 128 : TM_NEED <= 256 ? 256 : 512;
  static_assert(SMEM <= kSmemMax && TM_NEED <= 512, "the tile plan fits one SM");
  // the softmax waits for a whole tile of V (to clear unseen keys) before P V takes its first stage
  static_assert(NST >= VST, "the ring holds a tile of V");
  static_assert(N == 16 || N == 32 || N == 64, "one swizzle span of 2N bytes");
};

// Descriptor of P (B operand, rows contiguous): 2N bytes a key, swizzled over
// exactly that span, eight keys a group.
template <int N>
__device__ __forceinline__ uint64_t p_desc(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFF);
  d |= (uint64_t)((kTile * N * 2) >> 4) << 16;
  d |= (uint64_t)((16 * N) >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)(N == 64 ? 2 : N == 32 ? 4 : 6) << 61;
  return d;
}
// Byte offset of 16-byte chunk c of key r in P.
template <int N>
__device__ __forceinline__ uint32_t p_offset(int r, int c) {
  const uint32_t a = r * (2 * N) + c * 16;
  return a ^ ((a >> 3) & (2 * N - 16));
}

__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// Sum v[n] over the 32 lanes, leaving N/32 sums (or one, twice) a lane: rows
// N <= 32: lane / (32 / N), N = 64: 2 * lane + i.
template <int N>
__device__ __forceinline__ void scatter_sum(float (&v)[N], int lane) {
  int o = 16;
#pragma unroll
  for (int cnt = N; cnt > 1 && o >= 1; cnt /= 2, o /= 2) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < cnt / 2; ++i) {
      const float send = up ? v[i] : v[i + cnt / 2];
      const float keep = up ? v[i + cnt / 2] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
    }
  }
  if (N == 16) v[0] += __shfl_xor_sync(0xffffffffu, v[0], 1);
}

template <int N>
__device__ __forceinline__ void tmem_cols(uint32_t taddr, float (&s)[N]) {
  if constexpr (N == 16) {
    uint32_t u[16];
    tmem_ld16(taddr, u);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      asm volatile("" : "+r"(u[i]));
      s[i] = __uint_as_float(u[i]);
    }
  } else {
#pragma unroll
    for (int h = 0; h < N / 32; ++h) {
      uint32_t u[32];
      tmem_ld32(taddr + h * 32, u);
      tmem_wait_ld();
      reg_fence(u);
#pragma unroll
      for (int i = 0; i < 32; ++i) s[h * 32 + i] = __uint_as_float(u[i]);
    }
  }
}

template <int DQK, int DV, int N, bool BF16>
__global__ void __launch_bounds__(192, 1)
    paged_rows_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const __grid_constant__ PagedParams p) {
  using C = RowsCfg<DQK, DV, N>;
  using E = Elem<BF16>;
  using T = typename E::T;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sQ = smem;
  uint8_t* sP = sQ + C::NQ * C::Q_BYTES;
  uint8_t* sStage = sP + 2 * C::P_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(sStage + C::NST * kStage);
  uint64_t* empty = full + C::NST;
  uint64_t* bar_q = empty + C::NST;    // [NQ] Q is in shared memory
  uint64_t* q_free = bar_q + C::NQ;    // [NQ] the item's last S^T is done
  uint64_t* bar_s = q_free + C::NQ;    // [2] S^T is in TMEM
  uint64_t* bar_p = bar_s + 2;         // [2] P is in shared memory
  uint64_t* bar_o = bar_p + 2;         // [2] O^T has this tile (and P may be replaced)
  uint64_t* o_free = bar_o + 2;        // the item's O^T has been read
  uint64_t* bar_drain = o_free + 1;
  PagedScan* scan = reinterpret_cast<PagedScan*>(bar_drain + 1);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(scan + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  float* s_m = reinterpret_cast<float*>(sStage + C::NST * kStage + 1024);  // [N] running maxima (log2 units)
  float* s_f = s_m + N;        // [N] factors of a rescale
  float* s_w = s_f + N;        // [4][N] warps' maxima, then their sums
  float* s_l = s_w + 4 * N;    // [N] sums of an item

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NST; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < C::NQ; ++i) {
      mbar_init(&bar_q[i], 1);
      mbar_init(&q_free[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar_s[i], 1);
      mbar_init(&bar_p[i], 128);
      mbar_init(&bar_o[i], 1);
    }
    mbar_init(o_free, 128);
    mbar_init(bar_drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 5) {
    tmem_alloc(tmem_holder, C::TM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  const int me = blockIdx.x;
  const PagedShares all = paged_scan<C::THREADS>(p, scan, me, 1, 1, gridDim.x);
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const int workers = (int)min((long long)gridDim.x, all.total);
  const bool work = me < workers;
  const long long u0 = work ? share_at(all.total, me, workers) : 0;
  if (threadIdx.x == 0 && me == 0) {
    if (SDPA_ADDR_OK(p.chk, p.total_tiles, 8)) *p.total_tiles = all.total;
    if (!all.fit) record_error(p.err, SDPA_ERR_BAD_SEQLENS);
  }

  if (work) {
    PagedWalk w;
    w.start(p, scan->b[0], scan->i0[0], scan->block_at[0], u0, share_at(all.total, me + 1, workers));
    if (threadIdx.x == 0) {
      PagedCut* cut = p.cuts + me;
      if (SDPA_ADDR_OK(p.chk, cut, sizeof(PagedCut))) *cut = PagedCut{w.at, w.weight, w.b, w.i0, w.unit};
    }
    if (warp == 4) {
      // ---------------------------------------------------------- producer
      if (lane == 0) {
        prefetch_tmap(&tmQ);
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
      }
      const uint32_t box_bytes = p.box_rows * 128;
      int c = 0, nq = 0;
      bool ok = true;
      do {
        if (w.span.tiles == 0) continue;
        const PagedUnit un = paged_unit(p, w.unit);
        const int qb = nq % C::NQ;
        if (nq >= C::NQ && !__all_sync(0xffffffffu, mbar_wait(&q_free[qb], (nq / C::NQ - 1) & 1, abort_flag))) {
          ok = false;
          break;
        }
        if (lane == 0) {
          mbar_arrive_expect_tx(&bar_q[qb], (uint32_t)p.q_box_rows * DQK * 2);
          for (int a = 0; a < DQK / 64; ++a)
            tma_load_3d(&tmQ, &bar_q[qb], sQ + qb * C::Q_BYTES + a * (N * 128), a * 64, un.head0, w.s.row0 + w.i0);
        }
        ++nq;
        auto box_of = [&](int j) { return paged_box(p, w.span, w.b, (w.span.tile0 + j) * kTile, lane); };
        auto fetch = [&](const CUtensorMap* m, const PagedBox& x, int col, int atoms) -> bool {
          const int slot = c % C::NST;
          if (!__all_sync(0xffffffffu, mbar_wait(&empty[slot], ((c / C::NST) & 1) ^ 1, abort_flag))) return false;
          if (lane == 0) mbar_arrive_expect_tx(&full[slot], x.live * atoms * box_bytes);
          __syncwarp();
          if (x.mine) {
            uint8_t* dst = sStage + slot * kStage + lane * box_bytes;
            for (int a = 0; a < atoms; ++a)
              tma_load_4d(m, &full[slot], dst + a * 16384, col + a * 64, p.slot_first ? x.slot : un.kvh,
                          p.slot_first ? un.kvh : x.slot, x.page);
          }
          ++c;
          return true;
        };
        PagedBox cur = box_of(w.j0), prev = cur;
        for (int j = w.j0; j < w.j1 && ok; ++j) {
          const PagedBox ahead = j + 1 < w.j1 ? box_of(j + 1) : cur;  // its table entry arrives while this tile's copies go out
          for (int kb = 0; kb < C::KST && ok; ++kb) ok = fetch(&tmK, cur, kb * 128, C::k_atoms(kb));
          if (j > w.j0)
            for (int vb = 0; vb < C::VST && ok; ++vb) ok = fetch(&tmV, prev, vb * 128, 2);
          prev = cur;
          cur = ahead;
        }
        for (int vb = 0; vb < C::VST && ok; ++vb) ok = fetch(&tmV, prev, vb * 128, 2);
      } while (ok && w.next(p));
      if (lane == 0) {
        if (!ok) {
          *abort_flag = 1;
          record_error(p.err, SDPA_ERR_TIMEOUT);
        }
        // every copy lands before the CTA ends
        for (int k = max(0, c - C::NST); k < c; ++k) mbar_wait_drain(&full[k % C::NST], (k / C::NST) & 1);
        for (int k = max(0, nq - C::NQ); k < nq; ++k) mbar_wait_drain(&bar_q[k % C::NQ], (k / C::NQ) & 1);
      }
    } else if (warp == 5) {
      // ---------------------------------------------------------- MMA issuer
      if (elect_one()) {
        constexpr uint32_t ID_S = idesc_f16(128, N, BF16, false, false);
        constexpr uint32_t ID_O = idesc_f16(128, N, BF16, true, true);
        int c = 0, nq = 0, gs = 0;  // ring stages, items with keys, tiles of earlier items
        bool ok = true;
        do {
          if (w.span.tiles == 0) continue;
          const int n = w.j1 - w.j0;
          const uint32_t q_base = smem_u32(sQ + (nq % C::NQ) * C::Q_BYTES);
          uint64_t* my_q_free = &q_free[nq % C::NQ];
          if (!mbar_wait(&bar_q[nq % C::NQ], (nq / C::NQ) & 1, abort_flag)) {
            ok = false;
            break;
          }
          ++nq;
          tc_fence_after();
          auto mma_s = [&](int j) -> bool {
            const int sj = gs + j;
            const uint32_t d = tmem + C::TM_S + (sj & 1) * N;
            for (int kb = 0; kb < C::KST; ++kb, ++c) {
              const int slot = c % C::NST;
              if (!mbar_wait(&full[slot], (c / C::NST) & 1, abort_flag)) return false;
              tc_fence_after();
              const uint32_t k_base = smem_u32(sStage + slot * kStage);
              const int steps = 4 * C::k_atoms(kb);
#pragma unroll
              for (int ks = 0; ks < 8; ++ks) {
                if (ks >= steps) break;
                mma_ss(d, smem_desc_sw128(k_base + (ks >> 2) * 16384 + (ks & 3) * 32, 16, 1024),
                       smem_desc_sw128(q_base + (kb * 2 + (ks >> 2)) * (N * 128) + (ks & 3) * 32, 16, 1024), ID_S,
                       (kb | ks) != 0);
              }
              mma_commit(&empty[slot]);
            }
            mma_commit(&bar_s[sj & 1]);
            if (j == n - 1) mma_commit(my_q_free);
            return true;
          };
          auto mma_o = [&](int j) -> bool {
            const int sj = gs + j;
            if (j == 0 && nq > 1 && !mbar_wait(o_free, (nq - 2) & 1, abort_flag)) return false;
            if (!mbar_wait(&bar_p[sj & 1], (sj >> 1) & 1, abort_flag)) return false;
            tc_fence_after();
            const uint32_t p_base = smem_u32(sP + (sj & 1) * C::P_BYTES);
            for (int vb = 0; vb < C::VST; ++vb, ++c) {
              const int slot = c % C::NST;
              if (!mbar_wait(&full[slot], (c / C::NST) & 1, abort_flag)) return false;
              tc_fence_after();
              const uint32_t v_base = smem_u32(sStage + slot * kStage);
#pragma unroll
              for (int ks = 0; ks < 8; ++ks)
                mma_ss(tmem + vb * N, smem_desc_sw128(v_base + ks * 2048, 16384, 1024),
                       p_desc<N>(p_base + ks * (32 * N)), ID_O, (j | ks) != 0);
              mma_commit(&empty[slot]);
            }
            mma_commit(&bar_o[sj & 1]);
            return true;
          };
          for (int j = 0; j < n && ok; ++j) {
            ok = mma_s(j);
            if (ok && j >= 1) ok = mma_o(j - 1);
          }
          if (ok) ok = mma_o(n - 1);
          gs += n;
        } while (ok && w.next(p));
        if (!ok) {
          *abort_flag = 1;
          record_error(p.err, SDPA_ERR_TIMEOUT);
          mma_commit(bar_drain);  // every MMA issued so far ends before TMEM is released
          mbar_wait_drain(bar_drain, 0);
        }
      }
    } else {
      // ---------------------------------------------------------- softmax and output
      const int tid = threadIdx.x;  // key of a tile, and value column
      const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
      const float sl2 = p.scale_log2;
      int gs = 0, c0 = 0;  // tiles and ring stages of earlier items
      bool ok = true;
      do {
        const int n = w.j1 - w.j0;
        const bool keys = w.span.tiles > 0;
        const PagedUnit un = paged_unit(p, w.unit);
        const int tok = w.i1(p) - w.i0 + 1, rows = tok * p.block_heads;
        const int off = w.s.kv_len - w.s.q_len;
        if (tid < N) s_m[tid] = -INFINITY;
        named_bar_sync(1, 128);
        float l[N];
#pragma unroll
        for (int i = 0; i < N; ++i) l[i] = 0.f;
        for (int j = 0; keys && j < n; ++j) {
          const int sj = gs + j;
          if (!__all_sync(0xffffffffu, mbar_wait(&bar_s[sj & 1], (sj >> 1) & 1, abort_flag))) ok = false;
          tc_fence_after();
          float s[N];
          tmem_cols<N>(lanes + C::TM_S + (sj & 1) * N, s);
          // the rows that see this thread's key: [r_lo, r_hi). Row r is head r % block_heads of token r / block_heads
          const int kb = (w.span.tile0 + w.j0 + j) * kTile, key = kb + tid;
          int r_lo = 0, r_hi = key < w.span.hi ? rows : 0;
          if (p.causal) {
            r_lo = min(rows, max(0, key - off - w.i0) * p.block_heads);
            if (p.window >= 0) r_hi = min(r_hi, max(0, key - off + p.window - w.i0 + 1) * p.block_heads);
          }
          const unsigned span = max(0, r_hi - r_lo);
#pragma unroll
          for (int i = 0; i < N; ++i) s[i] = (unsigned)(i - r_lo) < span ? s[i] * sl2 : -INFINITY;
          float top = -INFINITY;
          float t[N];
#pragma unroll
          for (int i = 0; i < N; ++i) {
            t[i] = s[i] - s_m[i];  // +inf where a row has no maximum yet
            t[i] = s[i] == -INFINITY ? -INFINITY : t[i];
            top = fmaxf(top, t[i]);
          }
          // P <= 2^8 against the running maximum: only a row that jumps higher
          // (or sees its first key) has its maximum moved and O^T and the sums rescaled
          if (!named_bar_and(1, 128, ok && !(top > 8.f))) {
            if (!named_bar_and(1, 128, ok)) {
              ok = false;
              break;
            }
#pragma unroll
            for (int i = 0; i < N; ++i) {
              const float m = warp_max(s[i]);
              if (lane == 0) s_w[warp * N + i] = m;
            }
            named_bar_sync(1, 128);
            if (tid < N) {
              const float m = fmaxf(fmaxf(s_w[tid], s_w[N + tid]), fmaxf(s_w[2 * N + tid], s_w[3 * N + tid]));
              const float old = s_m[tid];
              const bool move = m > old + 8.f || (old == -INFINITY && m > -INFINITY);
              s_f[tid] = !move ? 1.f : old == -INFINITY ? 0.f : ex2(old - m);
              if (move) s_m[tid] = m;
            }
            named_bar_sync(1, 128);
#pragma unroll
            for (int i = 0; i < N; ++i) {
              l[i] *= s_f[i];
              t[i] = s[i] == -INFINITY ? -INFINITY : s[i] - s_m[i];
            }
            if (j > 0) {
              if (!__all_sync(0xffffffffu, mbar_wait(&bar_o[(sj - 1) & 1], ((sj - 1) >> 1) & 1, abort_flag))) ok = false;
              tc_fence_after();
#pragma unroll 1
              for (int x = 0; x < C::VST * N / 16; ++x) {
                uint32_t u[16];
                tmem_ld16(lanes + x * 16, u);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  asm volatile("" : "+r"(u[i]));
                  u[i] = __float_as_uint(__uint_as_float(u[i]) * s_f[(x * 16 + i) % N]);
                }
                tmem_st16(lanes + x * 16, u);
              }
              tmem_wait_st();
            }
          }
          // P of two tiles ago has been read
          if (sj >= 2 && !__all_sync(0xffffffffu, mbar_wait(&bar_o[sj & 1], ((sj - 2) >> 1) & 1, abort_flag))) ok = false;
          uint8_t* pb = sP + (sj & 1) * C::P_BYTES;
#pragma unroll
          for (int ch = 0; ch < N / 8; ++ch) {
            uint32_t u[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float p0 = ex2(t[ch * 8 + 2 * e]), p1 = ex2(t[ch * 8 + 2 * e + 1]);
              l[ch * 8 + 2 * e] += p0;
              l[ch * 8 + 2 * e + 1] += p1;
              u[e] = E::pack(p0, p1);
            }
            *reinterpret_cast<uint4*>(pb + p_offset<N>(tid, ch)) = make_uint4(u[0], u[1], u[2], u[3]);
          }
          // keys that none of the item's rows sees have P = 0, but their values
          // may be anything (unused slots): zeros in their place keep 0 x NaN out
          if (kb < w.span.lo || kb + kTile > w.span.hi) {
            // a stage barrier tells a phase from its neighbour only: what used V's slots before must be done, which
            // is P V of the tile before (its V) and S^T of the next tile (its K, copied ahead of this tile's V)
            if (j > 0 && !__all_sync(0xffffffffu, mbar_wait(&bar_o[(sj - 1) & 1], ((sj - 1) >> 1) & 1, abort_flag)))
              ok = false;
            if (j + 1 < n && !__all_sync(0xffffffffu, mbar_wait(&bar_s[(sj + 1) & 1], ((sj + 1) >> 1) & 1, abort_flag)))
              ok = false;
            const int cv = c0 + (j == n - 1 ? n * C::KST + (n - 1) * C::VST : (j + 2) * C::KST + j * C::VST);
            for (int vb = 0; vb < C::VST; ++vb) {
              const int slot = (cv + vb) % C::NST;
              if (!__all_sync(0xffffffffu, mbar_wait(&full[slot], ((cv + vb) / C::NST) & 1, abort_flag))) ok = false;
              if (ok && (key < w.span.lo || key >= w.span.hi)) {
                uint8_t* v = sStage + slot * kStage + tid * 128;
#pragma unroll
                for (int e = 0; e < 16; ++e)
                  *reinterpret_cast<uint4*>(v + (e >> 3) * 16384 + (((e + tid) & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
              }
            }
          }
          fence_proxy_async_smem();
          tc_fence_before();
          mbar_arrive(&bar_p[sj & 1]);
        }
        // the item's sums: lanes, then warps
        scatter_sum<N>(l, lane);
        if constexpr (N == 64) {
          s_w[warp * N + 2 * lane] = l[0];
          s_w[warp * N + 2 * lane + 1] = l[1];
        } else {
          s_w[warp * N + lane / (32 / N)] = l[0];
        }
        if (!named_bar_and(1, 128, ok)) {
          ok = false;
          break;
        }
        if (tid < N) s_l[tid] = (s_w[tid] + s_w[N + tid]) + (s_w[2 * N + tid] + s_w[3 * N + tid]);
        named_bar_sync(1, 128);
        const long long row0 = w.s.row0 + w.i0;
        const bool whole = w.whole();
        // at most one item continues from the CTA before, and one into the next
        float* part = p.parts + ((long long)me * 2 + (w.at < u0 ? 0 : 1)) * (N * (DV + 2));
        if (tid < rows && tid % p.block_heads < un.heads) {
          const float m = s_m[tid], sum = s_l[tid];
          if (whole) {
            float* at = p.lse + (row0 + tid / p.block_heads) * p.hq + un.head0 + tid % p.block_heads;
            if (SDPA_ADDR_OK(p.chk, at, 4)) *at = sum == 0.f ? -INFINITY : m * kLn2 + logf(sum);
          } else if (SDPA_ADDR_OK(p.chk, part + N * DV + tid, 4) && SDPA_ADDR_OK(p.chk, part + N * DV + N + tid, 4)) {
            part[N * DV + tid] = m;
            part[N * DV + N + tid] = sum;
          }
        }
        if (keys) {
          const int last = gs + n - 1;
          if (!__all_sync(0xffffffffu, mbar_wait(&bar_o[last & 1], (last >> 1) & 1, abort_flag))) ok = false;
          tc_fence_after();
        }
        if (!named_bar_and(1, 128, ok)) {
          ok = false;
          break;
        }
#pragma unroll 1
        for (int vb = 0; vb < C::VST; ++vb) {
          float o[N];
          if (keys) {
            tmem_cols<N>(lanes + vb * N, o);
          } else {
#pragma unroll
            for (int i = 0; i < N; ++i) o[i] = 0.f;
          }
          if (keys && vb == C::VST - 1) {
            tc_fence_before();
            mbar_arrive(o_free);
          }
          int ti = 0, h = 0;
#pragma unroll
          for (int i = 0; i < N; ++i) {
            if (i < rows && h < un.heads) {
              if (whole) {
                const float sum = s_l[i];
                T* at = static_cast<T*>(p.o) + ((row0 + ti) * p.hq + un.head0 + h) * DV + vb * 128 + tid;
                const float v = o[i] * (sum == 0.f ? 0.f : 1.f / sum);
                const uint32_t packed = E::pack(v, 0.f);
                if (SDPA_ADDR_OK(p.chk, at, 2)) *reinterpret_cast<uint16_t*>(at) = (uint16_t)packed;
              } else {
                float* at = part + i * DV + vb * 128 + tid;
                if (SDPA_ADDR_OK(p.chk, at, 4)) *at = o[i];
              }
            }
            if (++h == p.block_heads) {
              h = 0;
              ++ti;
            }
          }
        }
        if (keys) {
          gs += n;
          c0 += n * (C::KST + C::VST);
        }
      } while (ok && w.next(p));
      if (!ok) {
        *abort_flag = 1;
        record_error(p.err, SDPA_ERR_TIMEOUT);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TM_COLS);
  }
}

// Items that cross cuts: CTA w joins the item that cut w (the start of worker
// w's share) falls into, if w is the first cut inside it. Its parts come from
// worker w - 1 (which began it) and the workers whose shares start in it:
//   m = max m_k,  l = sum l_k 2^(m_k - m),  O = sum O_k 2^(m_k - m) / l.
// A part holds N rows of DV values, then N maxima and N sums. CTA (w, y) joins
// rows 16 y to 16 y + 15: with all rows of an item in one CTA the join of a
// chunk's 128-row items took 29 us (128 columns) to 49 us (256), one round of
// loads after another.
template <int DV, int N, bool BF16>
__global__ void __launch_bounds__(256) paged_join_kernel(const __grid_constant__ PagedParams p, int grid) {
  using E = Elem<BF16>;
  using T = typename E::T;
  __shared__ float s_m[16], s_inv[16];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!SDPA_ADDR_OK(p.chk, p.total_tiles, 8)) return;
  const long long total = *reinterpret_cast<volatile long long*>(p.total_tiles);
  const int workers = (int)min((long long)grid, total);
  const int w = blockIdx.x + 1;
  if (w >= workers || !SDPA_ADDR_OK(p.chk, p.cuts + w, sizeof(PagedCut))) return;
  const PagedCut cut = p.cuts[w];
  if (share_at(total, w, workers) == cut.at || share_at(total, w - 1, workers) > cut.at) return;
  const PagedSeq s = paged_seq(p, cut.b);
  const int tok = min(cut.i0 + p.tokens, s.q_len) - cut.i0, r0 = blockIdx.y * 16;
  const int rows = min(16, tok * p.block_heads - r0);
  if (rows <= 0) return;
  int parts = 1;  // worker w - 1, then w, w + 1, ...
  while (w - 1 + parts < workers && share_at(total, w - 1 + parts, workers) < cut.at + cut.n) ++parts;
  constexpr int SLOT = N * (DV + 2);
  auto part = [&](int k) { return p.parts + ((long long)(w - 1 + k) * 2 + (k == 0 ? 1 : 0)) * SLOT; };
  const PagedUnit un = paged_unit(p, cut.unit);
  const long long row0 = s.row0 + cut.i0;
  auto stat = [&](int k, int i) {
    const float* at = part(k) + N * DV + i;
    return SDPA_ADDR_OK(p.chk, at, 4) ? *at : -INFINITY;
  };
  {
    const int i = threadIdx.x / 16, q = threadIdx.x % 16, r = r0 + i;  // 16 threads a row
    float m = -INFINITY, l = 0.f;
    const bool live = i < rows && r % p.block_heads < un.heads;
    if (live)
      for (int k = q; k < parts; k += 16) m = fmaxf(m, stat(k, r));
#pragma unroll
    for (int o = 8; o > 0; o /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (live && m != -INFINITY)
      for (int k = q; k < parts; k += 16) l += stat(k, N + r) * ex2(stat(k, r) - m);
#pragma unroll
    for (int o = 8; o > 0; o /= 2) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (live && q == 0) {
      s_m[i] = m;
      s_inv[i] = l == 0.f ? 0.f : 1.f / l;
      float* at = p.lse + (row0 + r / p.block_heads) * p.hq + un.head0 + r % p.block_heads;
      if (un.split == 0 && SDPA_ADDR_OK(p.chk, at, 4)) *at = l == 0.f ? -INFINITY : m * kLn2 + logf(l);
    }
  }
  __syncthreads();
  constexpr int V4 = DV / 4;
#pragma unroll 2
  for (int x = threadIdx.x; x < rows * V4; x += 256) {
    const int i = x / V4, r = r0 + i, d = (x % V4) * 4;
    if (r % p.block_heads >= un.heads) continue;
    const float mr = s_m[i];
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    if (mr != -INFINITY) {
#pragma unroll 4
      for (int k = 0; k < parts; ++k) {
        const float mk = stat(k, r), f = mk == -INFINITY ? 0.f : ex2(mk - mr);
        const float* at = part(k) + r * DV + d;
        const float4 v = SDPA_ADDR_OK(p.chk, at, 16) ? *reinterpret_cast<const float4*>(at) : make_float4(0.f, 0.f, 0.f, 0.f);
        a.x = fmaf(f, v.x, a.x);
        a.y = fmaf(f, v.y, a.y);
        a.z = fmaf(f, v.z, a.z);
        a.w = fmaf(f, v.w, a.w);
      }
    }
    const float inv = s_inv[i];
    T* dst = static_cast<T*>(p.o) + ((row0 + r / p.block_heads) * p.hq + un.head0 + r % p.block_heads) * p.dv +
             un.split * DV + d;
    if (SDPA_ADDR_OK(p.chk, dst, 8))
      *reinterpret_cast<uint2*>(dst) = make_uint2(E::pack(a.x * inv, a.y * inv), E::pack(a.z * inv, a.w * inv));
  }
}

// Launched while the attention kernel runs; it waits for it before reading.
template <int DV, int N, bool BF16>
int launch_join_t(const PagedLaunch& L) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)L.workers - 1, N / 16);
  cfg.blockDim = dim3(256);
  cfg.stream = L.stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_join_kernel<DV, N, BF16>, L.p, L.workers) == cudaSuccess ? SDPA_OK : SDPA_ERR_CUDA;
}

template <int DQK, int DV, int N, bool BF16>
int launch_rows_t(const PagedLaunch& L, int* launches) {
  using C = RowsCfg<DQK, DV, N>;
  auto kern = paged_rows_kernel<DQK, DV, N, BF16>;
  if (const int rc = set_kernel_smem(reinterpret_cast<const void*>(kern), C::SMEM, -1)) return rc;
  kern<<<(unsigned)L.workers, C::THREADS, C::SMEM, L.stream>>>(L.tmQ, L.tmK, L.tmV, L.p);
  if (cudaGetLastError() != cudaSuccess) return SDPA_ERR_CUDA;
  ++*launches;
  if (L.workers == 1 || !L.p.split) return SDPA_OK;  // no item crosses a cut
  ++*launches;
  return launch_join_t<DV, N, BF16>(L);
}

template <int DQK, int DV, bool BF16>
int launch_rows_n(const PagedLaunch& L, int n, int* launches) {
  if (n == 16) return launch_rows_t<DQK, DV, 16, BF16>(L, launches);
  if (n == 32 || DV == 512) return launch_rows_t<DQK, DV, 32, BF16>(L, launches);
  if constexpr (DV != 512) return launch_rows_t<DQK, DV, 64, BF16>(L, launches);
  return SDPA_ERR_UNSUPPORTED;
}

}  // namespace

int launch_paged_join(const PagedLaunch& L, int n, int dv, bool bf16) {
#define JOIN(A, B) return bf16 ? launch_join_t<A, B, true>(L) : launch_join_t<A, B, false>(L)
  if (n == 128 && dv == 128) JOIN(128, 128);
  if (n == 128 && dv == 256) JOIN(256, 128);
#undef JOIN
  return SDPA_ERR_UNSUPPORTED;
}

size_t paged_cut_bytes() { return sizeof(PagedCut); }

int launch_paged_rows(const PagedLaunch& L, int n, int head_dim, bool bf16, int* launches) {
#define ROWS(A, B) return bf16 ? launch_rows_n<A, B, true>(L, n, launches) : launch_rows_n<A, B, false>(L, n, launches)
  if (head_dim == 128) ROWS(128, 128);
  if (head_dim == 192) ROWS(192, 128);
  if (head_dim == 256) ROWS(256, 256);
  if (head_dim == 512) ROWS(512, 512);
#undef ROWS
  return SDPA_ERR_UNSUPPORTED;
}

}  // namespace sdpa
