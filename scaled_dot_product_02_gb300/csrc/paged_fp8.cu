// paged_fp8.cu -- attention of new tokens over a paged cache in 8 bits: E4M3 codes
// with a power of two a row (fp8_row.cuh).
//   S_ij = scale q_i . k_j 2^ek_j,  O_i = sum_j softmax(S)_ij v_j 2^ev_j
// with k_j, v_j the codes' values and q in 16 bits. The work is reading the
// cache, so it is bound by HBM; codes go to the tensor cores as they are.
//
// The split into items, shares and partial results is the rows kernel's
// (paged.cu): an item is up to N = 16 or 32 query rows that share a kv head,
// against 128 keys at a time, keys on the M side:
//   S^T = K Q^T   (A: 128 keys x D codes),   O^T += V^T P^T   (A: 128 value columns x 128 keys).
// An 8-bit MMA wants both operands in 8 bits, and Q and P have more. Each is
// written as a sum of three E5M2 terms, every one the rest of those before it
// rounded to nearest: three significant bits and a sign each, 2^-11 of the
// value left over and the range of fp16 (E5M2 is fp16's upper byte). For Q,
// scaled by a power of two a row, the sum is exact: 11 bits at most are there.
// The terms lie side by side on the N side -- 3 N rows of Q, 4 N columns of
// P with the last N unused -- so a tile of codes is read once for all three,
// and the threads that read the products from tensor memory add them up.
// (Converting the codes to 16 bits in shared memory instead moves 96 KB more
// per 32 KB of codes through it, as much as it passes in the time HBM takes to
// deliver them.)
//
// The scales: a thread of the softmax has one key, so 2^ek is one factor for its
// scores; and as 2^ev belongs to its weight, the running maximum is taken over
// score + ev (log2 units) and P = 2^(score + ev - m). The denominator adds up P 2^-ev.
// With P at most 2^4 past the maximum in use, times 2^11, the largest weight
// of a row is at least 2^11 and what E5M2's last step (2^-16) cannot hold is below
// 2^-28 of it.
//
// Roles (384 threads): warps 0-3 softmax and output, one thread per key of a
// tile (and per value column of the output); 4-6 TMA producers; 7 TMEM allocator
// and MMA issuer; 8 takes the items' rows of Q apart, an item ahead; 9-11 fetch
// the scale bytes, in turn a tile each, up to SST tiles ahead (table entry, then
// byte: two trips to memory). K and V tiles go through a ring of 16 KB stages
// (128 keys x 128 codes).
#include <algorithm>
#include <cuda.h>
#include <cuda_runtime.h>

#include "fp8_row.cuh"
#include "paged.cuh"
#include "row_sums.cuh"

namespace sdpa {

namespace {

constexpr int kCodes = 16384;      // bytes of a ring stage
constexpr float kLift = 11.f;      // log2 of what P is multiplied by
constexpr float kSlack = 4.f;      // how far (log2) a weight may pass the maximum in use
constexpr int kScaleLo = 47, kScaleHi = 207;  // the scale bytes that rows are given

template <int DQK, int DV, int N>
struct Fp8Cfg {
  static constexpr int THREADS = 384;
  static constexpr int PRODUCERS = 3, LOADERS = 3;
  static constexpr int KST = (DQK + 127) / 128;  // K stages of a tile
  static constexpr int VST = DV / 128;           // V stages of a tile
  static __device__ __forceinline__ constexpr int k_steps(int kb) { return DQK / 32 - 4 * kb >= 4 ? 4 : DQK / 32 - 4 * kb; }
  static constexpr int NS = 3 * N;               // columns of S^T: Q's terms
  static constexpr int NO = 4 * N;               // columns of O^T: P's terms, and a fourth of no use
  static constexpr int NQ = 2;                   // buffers of Q's terms
  static constexpr int Q_ATOM = NS * 128;        // bytes of 128 columns of Q's terms
  static constexpr int Q_BYTES = KST * Q_ATOM;
  static constexpr int P_BYTES = kTile * NO;
  static constexpr int SST = 8;                  // tiles of scales
  static constexpr int SCALE_BYTES = SST * kTile * 8;
  static constexpr int MISC = 1536 + (7 + NQ) * N * 4;
  static constexpr int NST_FIT = (kSmemMax - 1024 - NQ * Q_BYTES - 2 * P_BYTES - SCALE_BYTES - MISC) / kCodes;
  static constexpr int NST = NST_FIT > 12 ? 12 : NST_FIT;
  static constexpr int SMEM = 1024 + NQ * Q_BYTES + 2 * P_BYTES + NST * kCodes + SCALE_BYTES + MISC;
  static constexpr int TM_S = VST * NO;          // TMEM columns: O^T, then two S^T buffers
  static constexpr int TM_NEED = TM_S + 2 * NS;
  static constexpr int TM_COLS = TM_NEED <= 256 ? 256 : 512;
  static_assert(SMEM <= kSmemMax && TM_NEED <= 512, "the tile plan fits one SM");
  // the softmax waits for a whole tile of V (to clear unseen keys) before P V takes its first stage
  static_assert(NST >= VST && NST >= KST, "the ring holds a tile of V");
  static_assert(N == 16 || N == 32, "one swizzle span of 4 N bytes");
  static_assert((2 * NST + 2 * NQ + 8 + 2 * SST) * 8 + sizeof(PagedScan) + 16 <= 1536, "barriers and the scan");
};

// A: E4M3, B: E5M2, fp32 sums.
constexpr uint32_t idesc_f8(int n, bool a_mn, bool b_mn) {
  return (1u << 4) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(128 >> 4) << 24);
}

// Descriptor of P (B operand, rows contiguous): 4 N bytes a key, swizzled over exactly that span, eight keys a group.
template <int N>
__device__ __forceinline__ uint64_t p_desc(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFF);
  d |= (uint64_t)((kTile * 4 * N) >> 4) << 16;
  d |= (uint64_t)((32 * N) >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)(N == 32 ? 2 : 4) << 61;
  return d;
}
// Byte offset of 16-byte chunk c of key r in P.
template <int N>
__device__ __forceinline__ uint32_t p_offset(int r, int c) {
  const uint32_t a = r * (4 * N) + c * 16;
  return a ^ ((a >> 3) & (4 * N - 16));
}

// Two fp16 -> two E5M2 codes (nearest, saturating), and back.
__device__ __forceinline__ uint16_t to_e5m2x2(uint32_t h) {
  uint16_t c;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(c) : "r"(h));
  return c;
}
__device__ __forceinline__ uint32_t from_e5m2x2(uint16_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h) : "h"(c));
  return h;
}
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// Four values as three words of four E5M2 terms.
__device__ __forceinline__ void split4(float x0, float x1, float x2, float x3, uint32_t (&term)[3]) {
  uint32_t lo = Elem<false>::pack(x0, x1), hi = Elem<false>::pack(x2, x3);
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    const uint16_t a = to_e5m2x2(lo), b = to_e5m2x2(hi);
    term[k] = (uint32_t)a | (uint32_t)b << 16;
    if (k < 2) {
      lo = hsub2(lo, from_e5m2x2(a));
      hi = hsub2(hi, from_e5m2x2(b));
    }
  }
}

// S^T of a tile: this thread's key against the item's rows, Q's terms added up.
template <int N>
__device__ __forceinline__ void scores(uint32_t taddr, float (&s)[N]) {
  if constexpr (N == 16) {
    uint32_t a[16], b[16], c[16];
    tmem_ld16(taddr, a);
    tmem_ld16(taddr + 16, b);
    tmem_ld16(taddr + 32, c);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      asm volatile("" : "+r"(a[i]), "+r"(b[i]), "+r"(c[i]));
      s[i] = (__uint_as_float(c[i]) + __uint_as_float(b[i])) + __uint_as_float(a[i]);
    }
  } else {
    uint32_t a[32], b[32];
    tmem_ld32(taddr + 64, a);
    tmem_ld32(taddr + 32, b);
    tmem_wait_ld();
    reg_fence(a);
    reg_fence(b);
#pragma unroll
    for (int i = 0; i < 32; ++i) s[i] = __uint_as_float(a[i]) + __uint_as_float(b[i]);
    tmem_ld32(taddr, a);
    tmem_wait_ld();
    reg_fence(a);
#pragma unroll
    for (int i = 0; i < 32; ++i) s[i] += __uint_as_float(a[i]);
  }
}

// One item's rows of Q as their terms in shared memory ([128 columns][term][row], K-major, 128-byte swizzle), and what
// undoes the power of two that a row was multiplied by. A warp calls it. Rows that the item does not have are zeros.
template <int DQK, int N, bool BF16>
__device__ __forceinline__ void split_q(const PagedFp8Params& f, const PagedWalk& w, const PagedUnit& un, uint8_t* sQ,
                                        float* s_fq, int lane) {
  using E = Elem<BF16>;
  constexpr int VECS = DQK / 8, LPR = VECS >= 32 ? 32 : VECS == 24 ? 32 : VECS, RP = 32 / LPR, VPL = (VECS + 31) / 32;
  constexpr int U = 4;  // passes whose loads are in flight together
  static_assert(N % (RP * U) == 0, "whole passes");
  const PagedParams& p = f.a;
  const int tok = w.i1(p) - w.i0 + 1, sub = lane % LPR;
#pragma unroll 1
  for (int r0 = lane / LPR; r0 < N; r0 += RP * U) {
    uint4 x[U][VPL];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * RP, ti = r / p.block_heads, h = r - ti * p.block_heads;
      const uint8_t* row = static_cast<const uint8_t*>(f.q) +
                           ((long long)(w.s.row0 + w.i0 + ti) * f.q_stride + (long long)(un.head0 + h) * DQK) * 2;
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        const int vec = v * 32 + sub;
        x[u][v] = make_uint4(0u, 0u, 0u, 0u);
        if (ti < tok && h < un.heads && vec < VECS && SDPA_ADDR_OK(p.chk, row + vec * 16, 16))
          x[u][v] = __ldg(reinterpret_cast<const uint4*>(row + vec * 16));
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * RP;
      float2 y[VPL][4];
      float top = 0.f;
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        y[v][0] = E::unpack(x[u][v].x);
        y[v][1] = E::unpack(x[u][v].y);
        y[v][2] = E::unpack(x[u][v].z);
        y[v][3] = E::unpack(x[u][v].w);
#pragma unroll
        for (int e = 0; e < 4; ++e) top = fmaxf(top, fmaxf(fabsf(y[v][e].x), fabsf(y[v][e].y)));
      }
#pragma unroll
      for (int o = LPR / 2; o > 0; o /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      // the row's largest magnitude to 2^14 .. 2^15
      const int up = top > 0.f ? min(14 + 127 - (__float_as_int(top) >> 23), 126) : 0;
      const float by = exp2_int(up);
      if (sub == 0) s_fq[r] = exp2_int(-up);
      auto term_of = [&](float a) { return fabsf(a) == INFINITY ? NAN : a * by; };  // the terms have no infinity
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        const int vec = v * 32 + sub;
        uint32_t lo[3], hi[3];
        split4(term_of(y[v][0].x), term_of(y[v][0].y), term_of(y[v][1].x), term_of(y[v][1].y), lo);
        split4(term_of(y[v][2].x), term_of(y[v][2].y), term_of(y[v][3].x), term_of(y[v][3].y), hi);
        if (vec >= VECS) continue;
        uint8_t* to = sQ + (vec / 16) * (3 * N * 128) + r * 128 + ((((vec % 16) / 2) ^ (r & 7)) << 4) + (vec & 1) * 8;
#pragma unroll
        for (int k = 0; k < 3; ++k) *reinterpret_cast<uint2*>(to + k * N * 128) = make_uint2(lo[k], hi[k]);
      }
    }
  }
}

template <int DQK, int DV, int N, bool BF16>
__global__ void __launch_bounds__(384, 1)
    paged_fp8_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ PagedFp8Params f) {
  using C = Fp8Cfg<DQK, DV, N>;
  using E = Elem<BF16>;
  using T = typename E::T;
  const PagedParams& p = f.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sStage = smem;
  uint8_t* sQ = sStage + C::NST * kCodes;
  uint8_t* sP = sQ + C::NQ * C::Q_BYTES;
  float2* sScale = reinterpret_cast<float2*>(sP + 2 * C::P_BYTES);  // [SST][128] 2^ek and ev
  uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(sScale) + C::SCALE_BYTES);
  uint64_t* empty = full + C::NST;
  uint64_t* bar_q = empty + C::NST;      // [NQ] Q's terms are in shared memory
  uint64_t* q_free = bar_q + C::NQ;      // [NQ] the item's last S^T is done and its rows' factors are read
  uint64_t* sc_full = q_free + C::NQ;    // [SST] a tile's scales
  uint64_t* sc_free = sc_full + C::SST;  // [SST] read by the softmax
  uint64_t* bar_s = sc_free + C::SST;    // [2] S^T is in TMEM
  uint64_t* bar_p = bar_s + 2;           // [2] P is in shared memory
  uint64_t* bar_o = bar_p + 2;           // [2] O^T has this tile (and P may be replaced)
  uint64_t* o_free = bar_o + 2;          // the item's O^T has been read
  uint64_t* bar_drain = o_free + 1;
  PagedScan* scan = reinterpret_cast<PagedScan*>(bar_drain + 1);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(scan + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  float* s_m = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(full) + 1536);  // [N] running maxima (log2 units)
  float* s_f = s_m + N;        // [N] factors of a rescale
  float* s_w = s_f + N;        // [4][N] warps' maxima, then their sums
  float* s_l = s_w + 4 * N;    // [N] sums of an item
  float* s_fq = s_l + N;       // [NQ][N] what undoes the rows' scaling

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (threadIdx.x == 128) {  // not one of the threads that read a small batch
    for (int i = 0; i < C::NST; ++i) {
      mbar_init(&full[i], C::PRODUCERS);  // every producer, so that none falls a phase behind
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < C::NQ; ++i) {
      mbar_init(&bar_q[i], 32);
      mbar_init(&q_free[i], 1 + 128);
    }
    for (int i = 0; i < C::SST; ++i) {
      mbar_init(&sc_full[i], 32);
      mbar_init(&sc_free[i], 128);
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
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
      }
      const uint32_t box_bytes = p.box_rows * 128;
      int c = 0;
      bool ok = true;
      do {
        if (w.span.tiles == 0) continue;
        const PagedUnit un = paged_unit(p, w.unit);
        auto box_of = [&](int j) { return paged_box(p, w.span, w.b, (w.span.tile0 + j) * kTile, box); };
        auto fetch = [&](const CUtensorMap* m, const PagedBox& x, int boxes, int col) -> bool {
          const int slot = c % C::NST;
          if (!__all_sync(0xffffffffu, mbar_wait(&empty[slot], ((c / C::NST) & 1) ^ 1, abort_flag))) return false;
          // every producer arrives, with copies in this stage or not (the ring could go on without one otherwise and
          // leave it a phase behind); the others' copies may complete before producer 0 sets the byte count
          if (lane == 0) {
            if (pw == 0)
              mbar_arrive_expect_tx(&full[slot], boxes * box_bytes);
            else
              mbar_arrive(&full[slot]);
          }
          if (x.mine)
            tma_load_4d(m, &full[slot], sStage + slot * kCodes + box * box_bytes, col, p.slot_first ? x.slot : un.kvh,
                        p.slot_first ? un.kvh : x.slot, x.page);
          __syncwarp();
          ++c;
          return true;
        };
        auto boxes_of = [&](int j) { return paged_boxes(p, w.span, (w.span.tile0 + j) * kTile, 0, kTile); };
        PagedBox cur = box_of(w.j0), prev = cur;
        for (int j = w.j0; j < w.j1 && ok; ++j) {
          const PagedBox ahead = j + 1 < w.j1 ? box_of(j + 1) : cur;  // its table entry arrives while this tile's copies go out
          const int boxes = boxes_of(j);
          for (int kb = 0; kb < C::KST && ok; ++kb) ok = fetch(&tmK, cur, boxes, kb * 128);
          if (j > w.j0) {
            const int before = boxes_of(j - 1);
            for (int vb = 0; vb < C::VST && ok; ++vb) ok = fetch(&tmV, prev, before, vb * 128);
          }
          prev = cur;
          cur = ahead;
        }
        const int last = boxes_of(w.j1 - 1);
        for (int vb = 0; vb < C::VST && ok; ++vb) ok = fetch(&tmV, prev, last, vb * 128);
      } while (ok && w.next(p));
      if (lane == 0) {
        if (!ok) {
          *abort_flag = 1;
          record_error(p.err, SDPA_ERR_TIMEOUT);
        }
        // every copy lands before the CTA ends
        for (int k = max(0, c - C::NST); k < c; ++k) mbar_wait_drain(&full[k % C::NST], (k / C::NST) & 1);
      }
    } else if (warp == 8) {
      // ---------------------------------------------------------- Q's terms
      int nq = 0;
      bool ok = true;
      do {
        if (w.span.tiles == 0) continue;
        const int qb = nq % C::NQ;
        if (nq >= C::NQ && !__all_sync(0xffffffffu, mbar_wait(&q_free[qb], (nq / C::NQ - 1) & 1, abort_flag))) {
          ok = false;
          break;
        }
        split_q<DQK, N, BF16>(f, w, paged_unit(p, w.unit), sQ + qb * C::Q_BYTES, s_fq + qb * N, lane);
        fence_proxy_async_smem();
        mbar_arrive(&bar_q[qb]);
        ++nq;
      } while (ok && w.next(p));
      if (!ok && lane == 0) {
        *abort_flag = 1;
        record_error(p.err, SDPA_ERR_TIMEOUT);
      }
    } else if (warp > 8) {
      // ---------------------------------------------------------- scales
      int g = 0;  // tiles so far
      bool ok = true;
      do {
        const PagedUnit un = paged_unit(p, w.unit);
        for (int j = w.j0; j < w.j1 && ok; ++j, ++g) {
          if (g % C::LOADERS != warp - 9) continue;
          // four keys a lane, which lie in one page
          const int key = (w.span.tile0 + j) * kTile + 4 * lane;
          int ek[4] = {127, 127, 127, 127}, ev[4] = {127, 127, 127, 127};
          if (key < w.span.hi && key + 4 > w.span.lo) {
            const int col = key / p.page_size, slot = key - col * p.page_size;
            const int32_t* at = p.block_table + w.b * p.table_stride + col;
            const int id = SDPA_ADDR_OK(p.chk, at, 4) ? __ldg(at) : -1;
            if (id >= 0 && id < p.num_pages) {
              const uint8_t* ks = f.k_scale + id * f.ks_page + slot * f.ks_slot + un.kvh * f.ks_head;
              const uint8_t* vs = f.v_scale + id * f.vs_page + slot * f.vs_slot + un.kvh * f.vs_head;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if (key + e < w.span.lo || key + e >= w.span.hi) continue;
                if (SDPA_ADDR_OK(p.chk, ks + e * f.ks_slot, 1)) ek[e] = __ldg(ks + e * f.ks_slot);
                if (SDPA_ADDR_OK(p.chk, vs + e * f.vs_slot, 1)) ev[e] = __ldg(vs + e * f.vs_slot);
              }
            }
          }
          const int slot = g % C::SST;
          if (!__all_sync(0xffffffffu, mbar_wait(&sc_free[slot], ((g / C::SST) & 1) ^ 1, abort_flag))) {
            ok = false;
            break;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e)
            sScale[slot * kTile + 4 * lane + e] = make_float2(exp2_byte(min(max(ek[e], kScaleLo), kScaleHi)),
                                                              (float)(min(max(ev[e], kScaleLo), kScaleHi) - 127));
          mbar_arrive(&sc_full[slot]);
        }
      } while (ok && w.next(p));
      if (!ok && lane == 0) {
        *abort_flag = 1;
        record_error(p.err, SDPA_ERR_TIMEOUT);
      }
    } else if (warp == 7) {
      // ---------------------------------------------------------- MMA issuer
      if (elect_one()) {
        constexpr uint32_t ID_S = idesc_f8(C::NS, false, false);
        constexpr uint32_t ID_O = idesc_f8(C::NO, true, true);
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
            const uint32_t d = tmem + C::TM_S + (sj & 1) * C::NS;
            for (int kb = 0; kb < C::KST; ++kb, ++c) {
              const int slot = c % C::NST;
              if (!mbar_wait(&full[slot], (c / C::NST) & 1, abort_flag)) return false;
              tc_fence_after();
              const uint32_t k_base = smem_u32(sStage + slot * kCodes);
              const int steps = C::k_steps(kb);
#pragma unroll
              for (int ks = 0; ks < 4; ++ks) {
                if (ks >= steps) break;
                mma_f8_ss(d, smem_desc_sw128(k_base + ks * 32, 16, 1024),
                          smem_desc_sw128(q_base + kb * C::Q_ATOM + ks * 32, 16, 1024), ID_S, (kb | ks) != 0);
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
              const uint32_t v_base = smem_u32(sStage + slot * kCodes);
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)  // 32 keys each
                mma_f8_ss(tmem + vb * C::NO, smem_desc_sw128(v_base + ks * 4096, kCodes, 1024),
                          p_desc<N>(p_base + ks * (128 * N)), ID_O, (j | ks) != 0);
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
      int gs = 0, c0 = 0, nq = 0;  // tiles and ring stages of earlier items, items with keys
      bool ok = true;
      do {
        const int n = w.j1 - w.j0;
        const bool keys = w.span.tiles > 0;
        const PagedUnit un = paged_unit(p, w.unit);
        const int tok = w.i1(p) - w.i0 + 1, rows = tok * p.block_heads;
        const int off = w.s.kv_len - w.s.q_len;
        const float* fq = s_fq + (nq % C::NQ) * N;
        if (tid < N) s_m[tid] = -INFINITY;
        named_bar_sync(1, 128);
        if (keys && !__all_sync(0xffffffffu, mbar_wait(&bar_q[nq % C::NQ], (nq / C::NQ) & 1, abort_flag))) ok = false;
        float l[N];
#pragma unroll
        for (int i = 0; i < N; ++i) l[i] = 0.f;
        for (int j = 0; keys && j < n; ++j) {
          const int sj = gs + j, slot = sj % C::SST;
          if (!__all_sync(0xffffffffu, mbar_wait(&sc_full[slot], (sj / C::SST) & 1, abort_flag))) ok = false;
          const float2 sc = sScale[slot * kTile + tid];
          mbar_arrive(&sc_free[slot]);
          if (!__all_sync(0xffffffffu, mbar_wait(&bar_s[sj & 1], (sj >> 1) & 1, abort_flag))) ok = false;
          tc_fence_after();
          float s[N];
          scores<N>(lanes + C::TM_S + (sj & 1) * C::NS, s);
          // the rows that see this thread's key: [r_lo, r_hi). Row r is head r % block_heads of token r / block_heads
          const int kb = (w.span.tile0 + w.j0 + j) * kTile, key = kb + tid;
          int t_lo = 0, t_hi = key < w.span.hi ? tok : 0;
          if (p.causal) {
            t_lo = min(tok, max(0, key - off - w.i0));
            if (p.window >= 0) t_hi = min(t_hi, max(0, key - off + p.window - w.i0 + 1));
          }
          const int r_lo = t_lo * p.block_heads, r_hi = t_hi * p.block_heads;
          const unsigned span = max(0, r_hi - r_lo);
          const float sk = sl2 * sc.x;
#pragma unroll
          for (int i = 0; i < N; ++i) s[i] = (unsigned)(i - r_lo) < span ? fmaf(s[i] * fq[i], sk, sc.y) : -INFINITY;
          float top = -INFINITY;
          float t[N];
#pragma unroll
          for (int i = 0; i < N; ++i) {
            t[i] = s[i] - s_m[i];  // +inf where a row has no maximum yet
            t[i] = s[i] == -INFINITY ? -INFINITY : t[i];
            top = fmaxf(top, t[i]);
          }
          // only a row that jumps past the maximum in use (or sees its first key) has it moved and O^T and the sums rescaled
          if (!named_bar_and(1, 128, ok && !(top > kSlack))) {
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
              const bool move = m > old + kSlack || (old == -INFINITY && m > -INFINITY);
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
              for (int vb = 0; vb < C::VST; ++vb)
#pragma unroll 1
                for (int x = 0; x < C::NS / 16; ++x) {
                  uint32_t u[16];
                  tmem_ld16(lanes + vb * C::NO + x * 16, u);
                  tmem_wait_ld();
#pragma unroll
                  for (int i = 0; i < 16; ++i) {
                    asm volatile("" : "+r"(u[i]));
                    u[i] = __float_as_uint(__uint_as_float(u[i]) * s_f[(x * 16 + i) % N]);
                  }
                  tmem_st16(lanes + vb * C::NO + x * 16, u);
                }
              tmem_wait_st();
            }
          }
          // P of two tiles ago has been read
          if (sj >= 2 && !__all_sync(0xffffffffu, mbar_wait(&bar_o[sj & 1], ((sj - 2) >> 1) & 1, abort_flag))) ok = false;
          uint8_t* pb = sP + (sj & 1) * C::P_BYTES;
          const float un_v = ex2(-sc.y);
#pragma unroll
          for (int ch = 0; ch < N / 16; ++ch) {
            uint32_t u[3][4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float x[4];
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const int i = ch * 16 + e * 4 + y;
                x[y] = ex2(t[i] + kLift);
                l[i] = fmaf(x[y], un_v, l[i]);
              }
              uint32_t term[3];
              split4(x[0], x[1], x[2], x[3], term);
              u[0][e] = term[0];
              u[1][e] = term[1];
              u[2][e] = term[2];
            }
#pragma unroll
            for (int k = 0; k < 3; ++k)
              *reinterpret_cast<uint4*>(pb + p_offset<N>(tid, k * (N / 16) + ch)) = make_uint4(u[k][0], u[k][1], u[k][2], u[k][3]);
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
                uint8_t* v = sStage + slot * kCodes + tid * 128;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  *reinterpret_cast<uint4*>(v + (((e + tid) & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
              }
            }
          }
          fence_proxy_async_smem();
          tc_fence_before();
          mbar_arrive(&bar_p[sj & 1]);
        }
        if (keys) {
          mbar_arrive(&q_free[nq % C::NQ]);
          ++nq;
        }
        // the item's sums: lanes, then warps
        scatter_sum<N>(l, lane);
        s_w[warp * N + lane / (32 / N)] = l[0];
        if (!named_bar_and(1, 128, ok)) {
          ok = false;
          break;
        }
        const long long row0 = w.s.row0 + w.i0;
        const bool whole = w.whole();
        // at most one item continues from the CTA before, and one into the next
        float* part = p.parts + ((long long)me * 2 + (w.at < u0 ? 0 : 1)) * (N * (DV + 2));
        if (tid < N) {
          // l and O^T carry 2^kLift alike: it counts into the maximum. A sum that is NaN makes the part's maximum so, or the
          // join would take a part without one for a part without keys
          const float sum = (s_w[tid] + s_w[N + tid]) + (s_w[2 * N + tid] + s_w[3 * N + tid]);
          const float m = isnan(sum) ? sum : s_m[tid] - kLift;
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
#pragma unroll 1
        for (int vb = 0; vb < C::VST; ++vb) {
          int ti = 0, h = 0;
#pragma unroll 1
          for (int i0 = 0; i0 < rows; i0 += 4) {
            uint32_t o[3][4] = {};
            if (keys) {
#pragma unroll
              for (int k = 0; k < 3; ++k) tmem_ld4(lanes + vb * C::NO + k * N + i0, o[k]);
              tmem_wait_ld();
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              asm volatile("" : "+r"(o[0][e]), "+r"(o[1][e]), "+r"(o[2][e]));
              const int i = i0 + e;
              const float v = ((__uint_as_float(o[2][e]) + __uint_as_float(o[1][e])) + __uint_as_float(o[0][e])) * s_l[i];
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

template <int DQK, int DV, int N, bool BF16>
int launch_t(const PagedFp8Launch& L, int* launches) {
  using C = Fp8Cfg<DQK, DV, N>;
  auto kern = paged_fp8_kernel<DQK, DV, N, BF16>;
  if (const int rc = set_kernel_smem(reinterpret_cast<const void*>(kern), C::SMEM, -1)) return rc;
  if (const int rc = launch_early(kern, dim3((unsigned)L.workers), C::THREADS, C::SMEM, L.stream, false, L.tmK, L.tmV, L.p))
    return rc;
  ++*launches;
  if (L.workers == 1 || !L.p.a.split) return SDPA_OK;  // no item crosses a cut
  ++*launches;
  PagedLaunch join;
  join.p = L.p.a;
  join.workers = L.workers;
  join.stream = L.stream;
  return launch_paged_join(join, N, DV, L.workers, BF16);
}

}  // namespace

int launch_paged_fp8(const PagedFp8Launch& L, int n, int head_dim, bool bf16, int* launches) {
#define ROWS(A, B, NN) return bf16 ? launch_t<A, B, NN, true>(L, launches) : launch_t<A, B, NN, false>(L, launches)
  if (head_dim == 128 && n == 16) ROWS(128, 128, 16);
  if (head_dim == 128 && n == 32) ROWS(128, 128, 32);
  if (head_dim == 192 && n == 16) ROWS(192, 128, 16);
  if (head_dim == 192 && n == 32) ROWS(192, 128, 32);
  if (head_dim == 256 && n == 16) ROWS(256, 256, 16);
  if (head_dim == 256 && n == 32) ROWS(256, 256, 32);
  if (head_dim == 512 && n == 16) ROWS(512, 512, 16);
#undef ROWS
  return SDPA_ERR_UNSUPPORTED;
}

}  // namespace sdpa
