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
// Roles (256 threads): warps 0-3 softmax and output, one thread per key of a
// tile (and per value column of the output); warps 4-6 TMA producers, each
// lane fetching one page's rows of a tile (a warp issues its lanes' copies one
// after another, about 100 cycles each: with pages of 16 one producer warp was
// the bound: 64 sequences of 500 to 16384 keys took 397 us, with three 350);
// warp 7 TMEM allocator and MMA issuer. K and V tiles go through a ring of 32 KB
// stages (128 keys x 128 columns); S^T and P are double-buffered, so S^T of the
// next tile is formed while the softmax works on this one.
//
// Measured with the join: that batch 338 to 356 us, 6.2 to 6.5 TB/s; 48 sequences at
// head_dim 256 with a window of 1024 70 to 73 us, 5.2 TB/s; one token over 999 keys
// 9.1 to 9.6 us in a captured graph.
#include <algorithm>
#include <cuda.h>
#include <cuda_runtime.h>

#include "paged.cuh"
#include "row_sums.cuh"

namespace sdpa {

namespace {

// ---------------------------------------------------------------- the kernel

template <int DQK, int DV, int N>
struct RowsCfg {
  static constexpr int THREADS = 256;
  static constexpr int PRODUCERS = 3;
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
__global__ void __launch_bounds__(256, 1)
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

  if (threadIdx.x == 128) {  // not one of the threads that read a small batch
    for (int i = 0; i < C::NST; ++i) {
      mbar_init(&full[i], C::PRODUCERS);  // every producer, so that none falls a phase behind
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
  if (warp == 7) {
    tmem_alloc(tmem_holder, C::TM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  const int me = blockIdx.x;
  const PagedShares all = paged_scan<C::THREADS, true>(p, scan, me, gridDim.x);
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  if (threadIdx.x == 0 && me == 0) {
    if (SDPA_ADDR_OK(p.chk, p.total_tiles, 8)) *p.total_tiles = all.total;
    if (!all.fit) record_error(p.err, SDPA_ERR_BAD_SEQLENS);
  }

  if (me < min((long long)gridDim.x, all.total)) {
    PagedWalk w = scan->start;
    const long long u0 = w.u;
    if (threadIdx.x == 0 && p.split) {  // whole items need no join, and the workspace holds no records for one
      PagedCut* cut = p.cuts + me;
      if (SDPA_ADDR_OK(p.chk, cut, sizeof(PagedCut))) *cut = w.cut(p);
    }
    if (warp >= 4 && warp < 7) {
      // ---------------------------------------------------------- producers
      const int pw = warp - 4, box = lane * C::PRODUCERS + pw;  // this lane's box of a tile
      if (lane == 0 && pw == 0) {
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
        if (pw == 0 && nq >= C::NQ &&
            !__all_sync(0xffffffffu, mbar_wait(&q_free[qb], (nq / C::NQ - 1) & 1, abort_flag))) {
          ok = false;
          break;
        }
        if (lane == 0 && pw == 0) {
          mbar_arrive_expect_tx(&bar_q[qb], (uint32_t)p.q_box_rows * DQK * 2);
          for (int a = 0; a < DQK / 64; ++a)
            tma_load_3d(&tmQ, &bar_q[qb], sQ + qb * C::Q_BYTES + a * (N * 128), a * 64, un.head0, w.s.row0 + w.i0);
        }
        ++nq;
        auto box_of = [&](int j) { return paged_box(p, w.span, w.b, (w.span.tile0 + j) * kTile, box); };
        auto fetch = [&](const CUtensorMap* m, const PagedBox& x, int boxes, int col, int atoms) -> bool {
          const int slot = c % C::NST;
          if (!__all_sync(0xffffffffu, mbar_wait(&empty[slot], ((c / C::NST) & 1) ^ 1, abort_flag))) return false;
          // every producer arrives, with copies in this stage or not (the ring could go on without one otherwise and
          // leave it a phase behind); the others' copies may complete before producer 0 sets the byte count
          if (lane == 0) {
            if (pw == 0)
              mbar_arrive_expect_tx(&full[slot], boxes * atoms * box_bytes);
            else
              mbar_arrive(&full[slot]);
          }
          if (x.mine) {
            uint8_t* dst = sStage + slot * kStage + box * box_bytes;
            for (int a = 0; a < atoms; ++a)
              tma_load_4d(m, &full[slot], dst + a * 16384, col + a * 64, p.slot_first ? x.slot : un.kvh,
                          p.slot_first ? un.kvh : x.slot, x.page);
          }
          __syncwarp();
          ++c;
          return true;
        };
        auto boxes_of = [&](int j) { return paged_boxes(p, w.span, (w.span.tile0 + j) * kTile, 0, kTile); };
        PagedBox cur = box_of(w.j0), prev = cur;
        for (int j = w.j0; j < w.j1 && ok; ++j) {
          const PagedBox ahead = j + 1 < w.j1 ? box_of(j + 1) : cur;  // its table entry arrives while this tile's copies go out
          const int boxes = boxes_of(j);
          for (int kb = 0; kb < C::KST && ok; ++kb) ok = fetch(&tmK, cur, boxes, kb * 128, C::k_atoms(kb));
          if (j > w.j0) {
            const int before = boxes_of(j - 1);
            for (int vb = 0; vb < C::VST && ok; ++vb) ok = fetch(&tmV, prev, before, vb * 128, 2);
          }
          prev = cur;
          cur = ahead;
        }
        const int last = boxes_of(w.j1 - 1);
        for (int vb = 0; vb < C::VST && ok; ++vb) ok = fetch(&tmV, prev, last, vb * 128, 2);
      } while (ok && w.next(p));
      if (lane == 0) {
        if (!ok) {
          *abort_flag = 1;
          record_error(p.err, SDPA_ERR_TIMEOUT);
        }
        // every copy lands before the CTA ends
        for (int k = max(0, c - C::NST); k < c; ++k) mbar_wait_drain(&full[k % C::NST], (k / C::NST) & 1);
        for (int k = max(0, nq - C::NQ); pw == 0 && k < nq; ++k) mbar_wait_drain(&bar_q[k % C::NQ], (k / C::NQ) & 1);
      }
    } else if (warp == 7) {
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
          int t_lo = 0, t_hi = key < w.span.hi ? tok : 0;
          if (p.causal) {
            t_lo = min(tok, max(0, key - off - w.i0));
            if (p.window >= 0) t_hi = min(t_hi, max(0, key - off + p.window - w.i0 + 1));
          }
          const int r_lo = t_lo * p.block_heads, r_hi = t_hi * p.block_heads;
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
        const long long row0 = w.s.row0 + w.i0;
        const bool whole = w.whole();
        // at most one item continues from the CTA before, and one into the next
        float* part = p.parts + ((long long)me * 2 + (w.at < u0 ? 0 : 1)) * (N * (DV + 2));
        if (tid < N) {
          const float m = s_m[tid], sum = (s_w[tid] + s_w[N + tid]) + (s_w[2 * N + tid] + s_w[3 * N + tid]);
          s_l[tid] = whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
          if (tid < rows && tid % p.block_heads < un.heads) {
            if (whole) {
              float* at = p.lse + (row0 + tid / p.block_heads) * p.hq + un.head0 + tid % p.block_heads;
              if (SDPA_ADDR_OK(p.chk, at, 4)) *at = sum == 0.f ? -INFINITY : m * kLn2 + logf(sum);
            } else if (SDPA_ADDR_OK(p.chk, part + N * DV + tid, 4) && SDPA_ADDR_OK(p.chk, part + N * DV + N + tid, 4)) {
              part[N * DV + tid] = m;
              part[N * DV + N + tid] = sum;
            }
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
        // four rows at a time: unrolled over all N, the code took longer to fetch than to run
#pragma unroll 1
        for (int vb = 0; vb < C::VST; ++vb) {
          int ti = 0, h = 0;
#pragma unroll 1
          for (int i0 = 0; i0 < rows; i0 += 4) {
            uint32_t o[4] = {0u, 0u, 0u, 0u};
            if (keys) {
              tmem_ld4(lanes + vb * N + i0, o);
              tmem_wait_ld();
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              asm volatile("" : "+r"(o[e]));
              const int i = i0 + e;
              const float v = __uint_as_float(o[e]) * s_l[i];
              if (i < rows && h < un.heads) {
                if (whole) {
                  T* at = static_cast<T*>(p.o) + ((row0 + ti) * p.hq + un.head0 + h) * DV + vb * 128 + tid;
                  if (SDPA_ADDR_OK(p.chk, at, 2)) *reinterpret_cast<uint16_t*>(at) = (uint16_t)E::pack(v, 0.f);
                } else {
                  float* at = part + i * DV + vb * 128 + tid;
                  if (SDPA_ADDR_OK(p.chk, at, 4)) *at = v;
                }
              }
              if (++h == p.block_heads) {
                h = 0;
                ++ti;
              }
            }
          }
        }
        if (keys) {
          tc_fence_before();
          mbar_arrive(o_free);
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
  if (warp == 7) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TM_COLS);
  }
}

// Items that cross cuts. Their parts come from the worker that began the item
// and from those whose shares start in it:
//   m = max m_k,  l = sum l_k 2^(m_k - m),  O = sum O_k 2^(m_k - m) / l.
// A part holds N rows of DV values, then N maxima and N sums. Every cut inside an
// item (the start of worker w's share, CTAs (w, y)) takes an equal portion of its
// elements, four columns of a row each with its own copy of the row's
// statistics: after the wait there are two rounds of loads, the cut and the
// parts. Of an item of more than eight parts four lanes share an element, so
// that no thread walks many of them in turn. (With the item's first cut alone
// at work, 4 sequences of 4 tokens over 10786 keys at head_dim 512, 38 parts an
// item, took 58 us; one item of 64 parts of 128 rows 96 us.)
constexpr int join_rows(int n) { return n >= 128 ? 32 : 8; }

template <int DV, int N, bool BF16>
__global__ void __launch_bounds__(256) paged_join_kernel(const __grid_constant__ PagedParams p, int grid) {
  using E = Elem<BF16>;
  using T = typename E::T;
  const int w = blockIdx.x + 1, lane = threadIdx.x % 32;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // a chunk kernel behind needs nothing of this
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!SDPA_ADDR_OK(p.chk, p.total_tiles, 8) || !SDPA_ADDR_OK(p.chk, p.cuts + w, sizeof(PagedCut))) return;
  const long long total = *reinterpret_cast<volatile long long*>(p.total_tiles);
  const PagedCut cut = p.cuts[w];  // read with the total; a worker without a share leaves it unset
  const PagedShare share(total, grid);
  if (w >= share.workers || share.at(w) == cut.at) return;
  const int first = share.of(cut.at), parts = share.of(cut.at + cut.n - 1) - first + 1;
  const int helper = (w - first - 1) * gridDim.y + blockIdx.y, helpers = (parts - 1) * gridDim.y;
  constexpr int SLOT = N * (DV + 2), V4 = DV / 4;
  static_assert(V4 % 32 == 0, "a warp's elements lie in one row");
  const PagedUnit un = paged_unit(p, cut.unit);
  const int lanes = parts > 8 ? 4 : 1, width = 32 / lanes;  // lanes that share an element, elements of a warp
  const int elements = cut.tokens * p.block_heads * V4, mine = lane / width;
  for (int x = (helper * 8 + threadIdx.x / 32) * width; x < elements; x += helpers * 8 * width) {
    const int r = x / V4, d = (x % V4 + lane % width) * 4;
    const int ti = r / p.block_heads, h = r - ti * p.block_heads;
    if (h >= un.heads) continue;
    float m = -INFINITY, l = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float mk, float lk, const float4& v) {
      if (mk == -INFINITY) return;  // a part without keys for this row
      const float top = fmaxf(m, mk), f = m == -INFINITY ? 0.f : ex2(m - top), g = ex2(mk - top);
      m = top;
      l = l * f + lk * g;
      a.x = a.x * f + v.x * g;
      a.y = a.y * f + v.y * g;
      a.z = a.z * f + v.z * g;
      a.w = a.w * f + v.w * g;
    };
    for (int k0 = mine; k0 < parts; k0 += 4 * lanes) {
      float mk[4], lk[4];
      float4 v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int k = k0 + e * lanes;
        const float* part = p.parts + ((long long)(first + k) * 2 + (k == 0 ? 1 : 0)) * SLOT;
        const bool in = k < parts && SDPA_ADDR_OK(p.chk, part + N * DV + r, 4) &&
                        SDPA_ADDR_OK(p.chk, part + N * DV + N + r, 4) && SDPA_ADDR_OK(p.chk, part + r * DV + d, 16);
        mk[e] = in ? part[N * DV + r] : -INFINITY;
        lk[e] = in ? part[N * DV + N + r] : 0.f;
        v[e] = in ? *reinterpret_cast<const float4*>(part + r * DV + d) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) add(mk[e], lk[e], v[e]);
    }
    if (lanes > 1) {
#pragma unroll
      for (int o = 8; o <= 16; o *= 2) {
        const float mk = __shfl_xor_sync(0xffffffffu, m, o), lk = __shfl_xor_sync(0xffffffffu, l, o);
        const float4 v = make_float4(__shfl_xor_sync(0xffffffffu, a.x, o), __shfl_xor_sync(0xffffffffu, a.y, o),
                                     __shfl_xor_sync(0xffffffffu, a.z, o), __shfl_xor_sync(0xffffffffu, a.w, o));
        add(mk, lk, v);
      }
      if (mine > 0) continue;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const long long at = (long long)(cut.row0 + ti) * p.hq + un.head0 + h;
    T* dst = static_cast<T*>(p.o) + at * p.dv + un.split * DV + d;
    if (SDPA_ADDR_OK(p.chk, dst, 8))
      *reinterpret_cast<uint2*>(dst) = make_uint2(E::pack(a.x * inv, a.y * inv), E::pack(a.z * inv, a.w * inv));
    if (d == 0 && un.split == 0 && SDPA_ADDR_OK(p.chk, p.lse + at, 4))
      p.lse[at] = l == 0.f ? -INFINITY : m * kLn2 + logf(l);
  }
}

// Launched while the attention kernel runs; it waits for it before reading.
template <int DV, int N, bool BF16>
int launch_join_t(const PagedLaunch& L, int shares) {
  auto kern = paged_join_kernel<DV, N, BF16>;
  // the attention kernels' division of an SM between L1 and shared memory
  if (const int rc = set_kernel_smem(reinterpret_cast<const void*>(kern), 0, 100)) return rc;
  return launch_early(kern, dim3((unsigned)shares - 1, N / join_rows(N)), 256, 0, L.stream, true, L.p, shares);
}

template <int DQK, int DV, int N, bool BF16>
int launch_rows_t(const PagedLaunch& L, int* launches) {
  using C = RowsCfg<DQK, DV, N>;
  auto kern = paged_rows_kernel<DQK, DV, N, BF16>;
  if (const int rc = set_kernel_smem(reinterpret_cast<const void*>(kern), C::SMEM, -1)) return rc;
  if (const int rc = launch_early(kern, dim3((unsigned)L.workers), C::THREADS, C::SMEM, L.stream, false, L.tmQ, L.tmK, L.tmV, L.p))
    return rc;
  ++*launches;
  if (L.workers == 1 || !L.p.split) return SDPA_OK;  // no item crosses a cut
  ++*launches;
  return launch_join_t<DV, N, BF16>(L, L.workers);
}

template <int DQK, int DV, bool BF16>
int launch_rows_n(const PagedLaunch& L, int n, int* launches) {
  if (n == 16) return launch_rows_t<DQK, DV, 16, BF16>(L, launches);
  if (n == 32 || DV == 512) return launch_rows_t<DQK, DV, 32, BF16>(L, launches);
  if constexpr (DV != 512) return launch_rows_t<DQK, DV, 64, BF16>(L, launches);
  return SDPA_ERR_UNSUPPORTED;
}

}  // namespace

int launch_paged_join(const PagedLaunch& L, int n, int dv, int shares, bool bf16) {
  if (shares < 2) return SDPA_OK;
#define JOIN(A, B) return bf16 ? launch_join_t<A, B, true>(L, shares) : launch_join_t<A, B, false>(L, shares)
  if (n == 8 && dv == 128) JOIN(128, 8);
  if (n == 8 && dv == 256) JOIN(256, 8);
  if (n == 8 && dv == 512) JOIN(512, 8);
  if (n == 16 && dv == 128) JOIN(128, 16);
  if (n == 32 && dv == 128) JOIN(128, 32);
  if (n == 16 && dv == 256) JOIN(256, 16);
  if (n == 128 && dv == 128) JOIN(128, 128);
  if (n == 256 && dv == 128) JOIN(128, 256);
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
