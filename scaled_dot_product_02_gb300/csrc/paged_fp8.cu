// paged_fp8.cu -- attention of new tokens over a paged cache in 8 bits: E4M3 codes
// with a power of two a row (fp8_row.cuh).
//   S_ij = scale q_i . k_j 2^ek_j,  O_i = sum_j softmax(S)_ij v_j 2^ev_j
// with k_j, v_j the codes' values and q in 16 bits. The work is reading the
// cache, so it is bound by HBM; codes go to the tensor cores as they are.
//
// The split into items, shares and partial results is the rows kernel's
// (paged.cu): an item is up to N = 8, 16 or 32 query rows that share a kv head,
// against 128 keys at a time, keys on the M side:
//   S^T = K Q^T   (A: 128 keys x D codes),   O^T += V^T P^T   (A: 128 value columns x 128 keys).
// An 8-bit MMA wants both operands in 8 bits, and Q and P have more. Each is
// written as a sum of three E5M2 terms, every one the rest of those before it
// rounded to nearest: three significant bits and a sign each, 2^-11 of the
// value left over and the range of fp16 (E5M2 is fp16's upper byte). A row of Q is
// scaled by a power of two that brings its largest magnitude to 2^14 .. 2^15; then
// the sum is exact for values down to 2^-23 of the largest (bf16; fp16, of 11 bits,
// 2^-20), and below that off by at most half of the last term's least step (2^-16):
// 2^-31 of the row's largest, in every value.
// The terms lie side by side on the N side, so a tile of codes is read once for
// all three, and the threads that read the products from tensor memory add them
// up: every 4 rows take 16 columns, their first terms, second, third, and 4 of
// no use. So 4 rows are one 16-column load and one 16-byte store, and the code
// for rows that an item does not have is passed over (a decoding step of a GQA
// group of 4 has 4 of them; fetching straight-line code for more, at the start
// of a kernel, costs more than running it).
// (Converting the codes to 16 bits in shared memory instead moves 96 KB more
// per 32 KB of codes through it, as much as it passes in the time HBM takes to
// deliver them.)
//
// The scales: a thread of the softmax has one key, so 2^ek is one factor for its
// scores, applied before the row's (products of at most 2^33 times 2^ek stay within
// fp32, times a row's power of two alone they need not); and as 2^ev belongs to its
// weight, the running maximum m is taken over score + ev (log2 units): d = 2^(score - m)
// goes into the denominator and P = d 2^ev to the product. With P at most 2^4 past the
// maximum in use, times 2^11, the largest weight of a row is at least 2^11 and what
// E5M2's last step (2^-16) cannot hold is below 2^-28 of it.
// Denominators know nothing of ev: beside value rows of 2^80, a row of zeros (ev = -80)
// with the same score has the same share of them. With one maximum for both, they lie
// between 2^(11 - 80) (all of their weight on the largest values) and 2^(15 + 80) a key,
// within fp32's range for 2^30 keys, and what is too small for a d is below 2^-57 of the
// row's. Where two of them meet (a new maximum, the two warpgroups, parts of an item)
// the factor between their maxima can be 2^-160: a new maximum takes half of it twice,
// the two warpgroups compare denominators instead of maxima, and so do parts whose
// denominator l is beyond 2^-48 .. 2^48: there m takes the power of two (elsewhere it
// stays what it is, as large scores leave a sum no room for it).
//
// Roles (512 threads): warps 0-3 and 4-7 softmax, a tile each in turn, one thread
// per key (and per value column of the output). Each of the two warpgroups has its
// own S^T, P, maximum, sums and O^T, which meet at an item's end: a tile's way
// through barriers, tensor memory and exponentials takes longer than its codes
// from HBM. Warps 8-11 TMA producers (a warp issues its lanes' copies one after
// another, some 100 cycles each, and pages of 16 make 8 of a stage); 12 TMEM
// allocator and MMA issuer; 13-15 take an item's rows of Q apart and then fetch its
// scale bytes, a tile each in turn, up to SST tiles ahead. K and V tiles go through
// a ring of 16 KB stages (128 keys x 128 codes).
//
// In the equal shares an item counts for a few tiles more than it has, about what
// its start and end cost (PagedParams::lead); a share may so get none of the tiles of
// an item that it touches, and leaves an empty part.
//
// Measured with the join, twelve passes in a captured graph (the 16-bit cache, so
// measured, in brackets): 64 sequences of 500 to 16384 keys, 32 heads on 8 of 128,
// 206 to 212 us, 5.3 to 5.4 TB/s (348 to 356), with [page][head][slot] pages 173; 32 of
// them at head_dim 256 180, 16 at 512 173 us (6.2, 6.4 TB/s); 48 sequences with a window
// of 1024 at head_dim 256 43 (69.5); one token over 999 keys 9.9 (9.4). Items of many
// rows are bound by the softmax: over the first batch's keys 4 tokens of 4 heads 234 us
// (347), 8 tokens 363 (353); 32 sequences with 32 heads on one kv head of 128 41 (37).
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
constexpr float kNone = -3.402823466e38f;  // in place of a maximum: no key yet (the least number: finite, so that no inf - inf arises)
constexpr int kStay = 48;           // the largest power of two that stays with a part's sum
constexpr int kScaleLo = 47, kScaleHi = 207;  // the scale bytes that rows are given

template <int DQK, int DV, int N>
struct Fp8Cfg {
  static constexpr int THREADS = 512;
  static constexpr int PRODUCERS = 4, AUX = 3;
  static constexpr int W_MMA = 8 + PRODUCERS, W_AUX = W_MMA + 1;  // behind the softmax warps and the producers
  static constexpr int LOADS = N == 32 ? 1 : 2;  // 16-column loads in flight (two spill at N = 32)
  static constexpr int KST = (DQK + 127) / 128;  // K stages of a tile
  static constexpr int VST = DV / 128;           // V stages of a tile
  static __device__ __forceinline__ constexpr int k_steps(int kb) { return DQK / 32 - 4 * kb >= 4 ? 4 : DQK / 32 - 4 * kb; }
  static constexpr int QUADS = N / 4;
  static constexpr int NT = 4 * N;               // columns of S^T and of 128 value columns' O^T: the rows' terms
  static constexpr int NQ = 2;                   // buffers of Q's terms
  static constexpr int Q_ATOM = NT * 128;        // bytes of 128 columns of Q's terms
  static constexpr int Q_BYTES = KST * Q_ATOM;
  static constexpr int P_BYTES = kTile * NT;
  static constexpr int SST = 8;                  // tiles of scales
  static constexpr int SCALE_BYTES = SST * kTile * 8;
  static constexpr int MISC = 1536 + (14 + NQ) * N * 4;
  static constexpr int NST_FIT = (kSmemMax - 1024 - NQ * Q_BYTES - 2 * P_BYTES - SCALE_BYTES - MISC) / kCodes;
  static constexpr int NST = NST_FIT > 12 ? 12 : NST_FIT;
  static constexpr int SMEM = 1024 + NQ * Q_BYTES + 2 * P_BYTES + NST * kCodes + SCALE_BYTES + MISC;
  static constexpr int TM_O = VST * NT;          // TMEM columns: each warpgroup's O^T, then its S^T
  static constexpr int TM_S = 2 * TM_O;
  static constexpr int TM_NEED = TM_S + 2 * NT;
  static constexpr int TM_COLS = TM_NEED <= 128 ? 128 : TM_NEED <= 256 ? 256 : 512;
  static_assert(SMEM <= kSmemMax && TM_NEED <= 512, "the tile plan fits one SM");
  // the softmax waits for a whole tile of V (to clear unseen keys) before P V takes its first stage
  static_assert(NST >= VST && NST >= KST, "the ring holds a tile of V");
  static_assert(N == 8 || N == 16 || N == 32, "one swizzle span of 4 N bytes");
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
  d |= (uint64_t)(N == 32 ? 2 : N == 16 ? 4 : 6) << 61;
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

// The exponent of a positive number; of 0, infinity and NaN one whose power of two leaves them what they are.
__device__ __forceinline__ int exponent_of(float x) { return min((__float_as_int(x) >> 23) - 127, 126); }

// The sum of a value's three terms, of 16 columns of 4 rows.
__device__ __forceinline__ float terms_sum(const uint32_t (&u)[16], int r) {
  return (__uint_as_float(u[8 + r]) + __uint_as_float(u[4 + r])) + __uint_as_float(u[r]);
}
__device__ __forceinline__ void fence16(uint32_t (&u)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) asm volatile("" : "+r"(u[i]));
}

// One item's rows of Q as their terms in shared memory (K-major, 128-byte swizzle), and what makes scores of their
// products, the softmax scale (log2 units) over the power of two that a row was multiplied by: the share of warp `part` of
// PARTS. Rows past the item's stay as they are: nothing of theirs is looked at.
template <int DQK, int N, bool BF16, int PARTS>
__device__ __forceinline__ void split_q(const PagedFp8Params& f, const PagedWalk& w, const PagedUnit& un, uint8_t* sQ,
                                        float* s_fq, int part, int lane) {
  using E = Elem<BF16>;
  constexpr int VECS = DQK / 8, LPR = VECS >= 32 ? 32 : VECS == 24 ? 32 : VECS, RP = 32 / LPR, VPL = (VECS + 31) / 32;
  constexpr int U = VPL > 1 ? 1 : N == 32 ? 4 : 2;  // rows of a lane whose loads are in flight together
  const PagedParams& p = f.a;
  const int rows = (w.i1(p) - w.i0 + 1) * p.block_heads, sub = lane % LPR;
#pragma unroll 1
  for (int r0 = part * RP * U + lane / LPR; r0 - lane / LPR < rows; r0 += PARTS * RP * U) {
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
        if (r < rows && h < un.heads && vec < VECS && SDPA_ADDR_OK(p.chk, row + vec * 16, 16))
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
      if (r >= rows) continue;
      if (sub == 0) s_fq[r] = exp2_int(-up) * p.scale_log2;
      auto term_of = [&](float a) { return fabsf(a) == INFINITY ? NAN : a * by; };  // the terms have no infinity
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        const int vec = v * 32 + sub;
        uint32_t lo[3], hi[3];
        split4(term_of(y[v][0].x), term_of(y[v][0].y), term_of(y[v][1].x), term_of(y[v][1].y), lo);
        split4(term_of(y[v][2].x), term_of(y[v][2].y), term_of(y[v][3].x), term_of(y[v][3].y), hi);
        if (vec >= VECS) continue;
        uint8_t* to = sQ + (vec / 16) * (4 * N * 128) + (vec & 1) * 8;
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          const int at = (r / 4) * 16 + k * 4 + r % 4;
          *reinterpret_cast<uint2*>(to + at * 128 + ((((vec % 16) / 2) ^ (at & 7)) << 4)) = make_uint2(lo[k], hi[k]);
        }
      }
    }
  }
}

template <int DQK, int DV, int N, bool BF16>
__global__ void __launch_bounds__(512, 1)
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
  float* s_m = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(full) + 1536);  // [N] running maxima (log2 units) less kLift
  float* s_f = s_m + 2 * N;    // [N] factors of a rescale
  float* s_w = s_f + 2 * N;    // [4][N] warps' maxima, then their sums
  float* s_l = s_w + 8 * N;    // [N] factors of an item's output (these four for each softmax warpgroup)
  float* s_fq = s_l + 2 * N;   // [NQ][N] the rows' factors of split_q

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (threadIdx.x == 256) {  // not one of the threads that read a small batch
    for (int i = 0; i < C::NST; ++i) {
      mbar_init(&full[i], C::PRODUCERS);  // every producer, so that none falls a phase behind
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < C::NQ; ++i) {
      mbar_init(&bar_q[i], 32 * C::AUX);
      mbar_init(&q_free[i], 1 + 256);
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
    mbar_init(o_free, 256);
    mbar_init(bar_drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == C::W_MMA) {
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
    if (warp >= 8 && warp < C::W_MMA) {
      // ---------------------------------------------------------- producers
      const int pw = warp - 8, box = lane * C::PRODUCERS + pw;  // this lane's box of a tile
      if (lane == 0 && pw == 0) {
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
      }
      const uint32_t box_bytes = p.box_rows * 128;
      const int shift = __ffs(p.box_rows) - 1;  // a power of two
      const int step_col = kTile / p.page_size, step_slot = kTile - step_col * p.page_size;  // from a tile to the next
      int c = 0;
      bool ok = true;
      do {
        if (w.j1 == w.j0) continue;  // no keys, or none of its tiles
        const PagedUnit un = paged_unit(p, w.unit);
        // The page numbers come 32 at a time, one a lane, the next 32 behind them: a load for every tile made every tile
        // wait for it.
        const int first = (w.span.tile0 + w.j0) * kTile, last_col = (w.span.hi - 1) / p.page_size;
        int tile_col = first / p.page_size, tile_slot = first - tile_col * p.page_size;  // where the tile starts
        int col = (first + box * p.box_rows) / p.page_size;                              // where this lane's box does
        int slot_in = first + box * p.box_rows - col * p.page_size;
        const int32_t* row = p.block_table + w.b * p.table_stride;
        auto entry = [&](int x) {
          return x >= w.span.lo / p.page_size && x <= last_col && SDPA_ADDR_OK(p.chk, row + x, 4) ? __ldg(row + x) : -1;
        };
        int base = tile_col, ids = entry(base + lane), ids_next = entry(base + 32 + lane);
        auto box_here = [&](int j) {
          const int key0 = (w.span.tile0 + j) * kTile, key = key0 + box * p.box_rows;
          if (tile_col - base >= 32) {
            base += 32;
            ids = ids_next;
            ids_next = entry(base + 32 + lane);
          }
          const int at = col - base;  // below 64: a tile starts within the first 32 and lies on at most 9 pages
          const int a = __shfl_sync(0xffffffffu, ids, at & 31), b = __shfl_sync(0xffffffffu, ids_next, at & 31);
          PagedBox x;
          x.mine = box < kTile >> shift && key < w.span.hi && key + p.box_rows > w.span.lo;
          x.page = at < 32 ? a : b;
          x.slot = slot_in;
          if (x.mine && (unsigned)x.page >= (unsigned)p.num_pages) {
            x.page = p.num_pages;  // outside the map: reads as zeros
            record_error(p.err, SDPA_ERR_BAD_INDEX);
          }
          auto advance = [&](int& at_col, int& at_slot) {
            at_col += step_col;
            at_slot += step_slot;
            if (at_slot >= p.page_size) {
              at_slot -= p.page_size;
              ++at_col;
            }
          };
          advance(tile_col, tile_slot);
          advance(col, slot_in);
          return x;
        };
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
        auto boxes_of = [&](int j) {
          const int key0 = (w.span.tile0 + j) * kTile, lo = max(w.span.lo - key0, 0), hi = min(w.span.hi - key0, kTile);
          return ((hi + p.box_rows - 1) >> shift) - (lo >> shift);
        };
        PagedBox prev;
        int before = 0;
#pragma unroll 1
        for (int j = w.j0; j <= w.j1 && ok; ++j) {
          PagedBox cur;
          int boxes = 0;
          if (j < w.j1) {
            cur = box_here(j);
            boxes = boxes_of(j);
#pragma unroll 1
            for (int kb = 0; kb < C::KST && ok; ++kb) ok = fetch(&tmK, cur, boxes, kb * 128);
          }
          if (j > w.j0)
#pragma unroll 1
            for (int vb = 0; vb < C::VST && ok; ++vb) ok = fetch(&tmV, prev, before, vb * 128);
          prev = cur;
          before = boxes;
        }
      } while (ok && w.next(p));
      if (lane == 0) {
        if (!ok) {
          *abort_flag = 1;
          record_error(p.err, SDPA_ERR_TIMEOUT);
        }
        // every copy lands before the CTA ends
        for (int k = max(0, c - C::NST); k < c; ++k) mbar_wait_drain(&full[k % C::NST], (k / C::NST) & 1);
      }
    } else if (warp >= C::W_AUX) {
      // ---------------------------------------------------------- Q's terms, and scales
      const int aux = warp - C::W_AUX;
      int nq = 0, gs = 0;  // items with keys, tiles of earlier items
      bool ok = true;
      do {
        if (w.j1 == w.j0) continue;  // no keys, or none of its tiles
        const PagedUnit un = paged_unit(p, w.unit);
        const int n = w.j1 - w.j0;
        // four keys a lane, which lie in one page; not looked at before they are stored, a tile later
        int ek[4], ev[4];
        auto load = [&](int j) {
#pragma unroll
          for (int e = 0; e < 4; ++e) ek[e] = ev[e] = 127;
          const int key = (w.span.tile0 + w.j0 + j) * kTile + 4 * lane;
          if (j < n && key < w.span.hi && key + 4 > w.span.lo) {
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
        };
        int j = (aux + C::AUX - gs % C::AUX) % C::AUX;  // tiles in turn, whatever item they belong to
        load(j);
        const int qb = nq % C::NQ;
        if (nq >= C::NQ && !__all_sync(0xffffffffu, mbar_wait(&q_free[qb], (nq / C::NQ - 1) & 1, abort_flag))) {
          ok = false;
          break;
        }
        split_q<DQK, N, BF16, C::AUX>(f, w, un, sQ + qb * C::Q_BYTES, s_fq + qb * N, aux, lane);
        fence_proxy_async_smem();
        mbar_arrive(&bar_q[qb]);
        ++nq;
        for (; j < n; j += C::AUX) {
          const int slot = (gs + j) % C::SST;
          if (!__all_sync(0xffffffffu, mbar_wait(&sc_free[slot], (((gs + j) / C::SST) & 1) ^ 1, abort_flag))) {
            ok = false;
            break;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e)
            sScale[slot * kTile + 4 * lane + e] = make_float2(exp2_byte(min(max(ek[e], kScaleLo), kScaleHi)),
                                                              (float)(min(max(ev[e], kScaleLo), kScaleHi) - 127));
          mbar_arrive(&sc_full[slot]);
          load(j + C::AUX);
        }
        gs += n;
      } while (ok && w.next(p));
      if (!ok && lane == 0) {
        *abort_flag = 1;
        record_error(p.err, SDPA_ERR_TIMEOUT);
      }
    } else if (warp == C::W_MMA) {
      // ---------------------------------------------------------- MMA issuer
      if (elect_one()) {
        constexpr uint32_t ID_S = idesc_f8(C::NT, false, false);
        constexpr uint32_t ID_O = idesc_f8(C::NT, true, true);
        int c = 0, nq = 0, gs = 0;  // ring stages, items with keys, tiles of earlier items
        bool ok = true;
        do {
          if (w.j1 == w.j0) continue;  // no keys, or none of its tiles
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
            const uint32_t d = tmem + C::TM_S + (sj & 1) * C::NT;
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
                mma_f8_ss(tmem + (sj & 1) * C::TM_O + vb * C::NT, smem_desc_sw128(v_base + ks * 4096, kCodes, 1024),
                          p_desc<N>(p_base + ks * (128 * N)), ID_O, j >= 2 || ks > 0);
              mma_commit(&empty[slot]);
            }
            mma_commit(&bar_o[sj & 1]);
            return true;
          };
#pragma unroll 1
          for (int j = 0; j <= n && ok; ++j) {
            if (j < n) ok = mma_s(j);
            if (ok && j >= 1) ok = mma_o(j - 1);
          }
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
      const int me_g = warp / 4, tid = threadIdx.x % 128;  // warpgroup; key of a tile, and value column
      const uint32_t lanes = tmem + ((uint32_t)((warp % 4) * 32) << 16);
      const uint32_t my_o = lanes + me_g * C::TM_O, my_s = lanes + C::TM_S + me_g * C::NT;
      const int bar_id = 1 + me_g;  // named barriers: a warpgroup's, and 3 for both
      float *const m_g = s_m + me_g * N, *const f_g = s_f + me_g * N, *const w_g = s_w + me_g * 4 * N;
      uint8_t* const pb = sP + me_g * C::P_BYTES;
      int gs = 0, c0 = 0, nq = 0;  // tiles and ring stages of earlier items, items with keys
      bool ok = true;
      do {
        const int n = w.j1 - w.j0;
        const bool keys = n > 0;
        const PagedUnit un = paged_unit(p, w.unit);
        const int tok = w.i1(p) - w.i0 + 1, rows = tok * p.block_heads, quads = (rows + 3) / 4;
        const int off = w.s.kv_len - w.s.q_len;
        const float* fq = s_fq + (nq % C::NQ) * N;
        if (tid < N) m_g[tid] = kNone;
        named_bar_sync(bar_id, 128);
        if (keys && !__all_sync(0xffffffffu, mbar_wait(&bar_q[nq % C::NQ], (nq / C::NQ) & 1, abort_flag))) ok = false;
        float l[N];
#pragma unroll
        for (int i = 0; i < N; ++i) l[i] = 0.f;
        const int j_first = (gs ^ me_g) & 1;  // tiles in turn, whatever item they belong to
        for (int j = j_first; keys && j < n; j += 2) {
          const int sj = gs + j, slot = sj % C::SST;
          // the rows that see this thread's key: [r_lo, r_hi). Row r is head r % block_heads of token r / block_heads
          const int kb = (w.span.tile0 + w.j0 + j) * kTile, key = kb + tid;
          int t_lo = 0, t_hi = key < w.span.hi ? tok : 0;
          if (p.causal) {
            t_lo = min(tok, max(0, key - off - w.i0));
            if (p.window >= 0) t_hi = min(t_hi, max(0, key - off + p.window - w.i0 + 1));
          }
          const int r_lo = t_lo * p.block_heads, r_hi = t_hi * p.block_heads;
          const unsigned span = max(0, r_hi - r_lo);
          // S^T of this tile; with it P V of two tiles ago is done, and its P may be replaced (they were issued in that order)
          if (!__all_sync(0xffffffffu, mbar_wait_both(&sc_full[slot], (sj / C::SST) & 1, &bar_s[me_g], (sj >> 1) & 1, abort_flag)))
            ok = false;
          tc_fence_after();
          const float2 sc = sScale[slot * kTile + tid];
          float s[N], top = -INFINITY;
#pragma unroll
          for (int c = 0; c < C::QUADS; c += C::LOADS) {
            if (c >= quads) break;
            uint32_t u[C::LOADS][16];
#pragma unroll
            for (int x = 0; x < C::LOADS; ++x)
              if (c + x < quads) tmem_ld16(my_s + (c + x) * 16, u[x]);
            tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < C::LOADS; ++x) fence16(u[x]);
#pragma unroll
            for (int x = 0; x < C::LOADS; ++x) {
              if (c + x >= quads) break;
              const float4 f4 = *reinterpret_cast<const float4*>(fq + (c + x) * 4);
              const float4 m4 = *reinterpret_cast<const float4*>(m_g + (c + x) * 4);
              const float fr[4] = {f4.x, f4.y, f4.z, f4.w}, mr[4] = {m4.x, m4.y, m4.z, m4.w};
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                const int i = (c + x) * 4 + r;
                s[i] = (unsigned)(i - r_lo) < span ? terms_sum(u[x], r) * sc.x * fr[r] : -INFINITY;
                top = fmaxf(top, s[i] - mr[r]);
              }
            }
          }
          mbar_arrive(&sc_free[slot]);
          // only a row that jumps past the maximum in use (or sees its first key) has it moved and O^T and the sums rescaled
          if (!named_bar_and(bar_id, 128, ok && !(top + sc.y > kLift + kSlack))) {
            if (!named_bar_and(bar_id, 128, ok)) {
              ok = false;
              break;
            }
#pragma unroll
            for (int c = 0; c < C::QUADS; ++c) {
              if (c >= quads) break;
              const float4 m4 = make_float4(warp_max(s[c * 4] + sc.y), warp_max(s[c * 4 + 1] + sc.y),
                                            warp_max(s[c * 4 + 2] + sc.y), warp_max(s[c * 4 + 3] + sc.y));
              if (lane == 0) *reinterpret_cast<float4*>(w_g + (warp % 4) * N + c * 4) = m4;
            }
            named_bar_sync(bar_id, 128);
            if (tid < quads * 4) {
              const float m = fmaxf(fmaxf(w_g[tid], w_g[N + tid]), fmaxf(w_g[2 * N + tid], w_g[3 * N + tid])) - kLift;
              const float old = m_g[tid];
              const bool move = m > old + kSlack;
              f_g[tid] = move ? ex2(0.5f * (old - m)) : 1.f;  // the root of the factor
              if (move) m_g[tid] = m;
            }
            named_bar_sync(bar_id, 128);
#pragma unroll
            for (int c = 0; c < C::QUADS; ++c) {
              if (c >= quads) break;
              const float4 f4 = *reinterpret_cast<const float4*>(f_g + c * 4);
              l[c * 4] = l[c * 4] * f4.x * f4.x;
              l[c * 4 + 1] = l[c * 4 + 1] * f4.y * f4.y;
              l[c * 4 + 2] = l[c * 4 + 2] * f4.z * f4.z;
              l[c * 4 + 3] = l[c * 4 + 3] * f4.w * f4.w;
            }
            if (j >= 2) {  // this warpgroup's last P V is done: see above
#pragma unroll 1
              for (int vb = 0; vb < C::VST; ++vb)
#pragma unroll 1
                for (int c = 0; c < quads; ++c) {
                  uint32_t u[16];
                  tmem_ld16(my_o + vb * C::NT + c * 16, u);
                  tmem_wait_ld();
                  fence16(u);
                  const float4 f4 = *reinterpret_cast<const float4*>(f_g + c * 4);
                  const float fr[4] = {f4.x * f4.x, f4.y * f4.y, f4.z * f4.z, f4.w * f4.w};
#pragma unroll
                  for (int i = 0; i < 12; ++i) u[i] = __float_as_uint(__uint_as_float(u[i]) * fr[i % 4]);
                  tmem_st16(my_o + vb * C::NT + c * 16, u);
                }
              tmem_wait_st();
            }
          }
          const float by_v = exp2_int((int)sc.y);
#pragma unroll
          for (int c = 0; c < C::QUADS; ++c) {
            if (c >= quads) break;
            const float4 m4 = *reinterpret_cast<const float4*>(m_g + c * 4);
            const float mr[4] = {m4.x, m4.y, m4.z, m4.w};
            float x[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float d = ex2(s[c * 4 + r] - mr[r]);
              l[c * 4 + r] += d;
              x[r] = d * by_v;
            }
            uint32_t term[3];
            split4(x[0], x[1], x[2], x[3], term);
            *reinterpret_cast<uint4*>(pb + p_offset<N>(tid, c)) = make_uint4(term[0], term[1], term[2], 0u);
          }
          // keys that none of the item's rows sees have P = 0, but their values
          // may be anything (unused slots): zeros in their place keep 0 x NaN out
          if (kb < w.span.lo || kb + kTile > w.span.hi) {
            // A stage barrier tells a phase from its neighbour only: what used V's slots before must be done. This tile's
            // S^T says so of all stages before its K; in a short ring the slots may also have been those of the V before
            // and the K after, which P V of the tile before and S^T of the next one have used.
            if (C::NST <= 2 * (C::KST + C::VST)) {
              if (j > 0 && !__all_sync(0xffffffffu, mbar_wait(&bar_o[(sj - 1) & 1], ((sj - 1) >> 1) & 1, abort_flag)))
                ok = false;
              if (j + 1 < n && !__all_sync(0xffffffffu, mbar_wait(&bar_s[(sj + 1) & 1], ((sj + 1) >> 1) & 1, abort_flag)))
                ok = false;
            }
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
          mbar_arrive(&bar_p[me_g]);
        }
        // the item's sums: lanes, then warps, then warpgroups
        scatter_sum<N>(l, lane);
        w_g[(warp % 4) * N + lane / (32 / N)] = l[0];
        if (keys) {
          mbar_arrive(&q_free[nq % C::NQ]);
          ++nq;
        }
        if (!named_bar_and(3, 256, ok)) {
          ok = false;
          break;
        }
        const long long row0 = w.s.row0 + w.i0;
        const bool whole = w.covers();
        // at most one item continues from the CTA before, and one into the next
        float* part = p.parts + ((long long)me * 2 + (w.at < u0 ? 0 : 1)) * (N * (DV + 2));
        if (threadIdx.x < N) {
          const float* a = s_w + tid;
          const float* b = a + 4 * N;
          const float la = (a[0] + a[N]) + (a[2 * N] + a[3 * N]), lb = (b[0] + b[N]) + (b[2 * N] + b[3 * N]);
          const int ea = exponent_of(la), eb = exponent_of(lb);
          const float ua = exp2_int(-ea), ub = exp2_int(-eb);
          const float apart = (s_m[tid] - s_m[N + tid]) + (float)(ea - eb);
          const float fa = ex2(fminf(apart, 0.f)), fb = ex2(fminf(-apart, 0.f));  // 0 without a key
          const float base = apart >= 0.f ? s_m[tid] : s_m[N + tid];
          const int up = apart >= 0.f ? ea : eb, stay = whole || abs(up) > kStay ? 0 : up;
          float sum = fa * (la * ua) + fb * (lb * ub);  // times 2^(base + up)
          // a sum that is NaN makes the part's maximum so, or the join would take a part without one for one without keys
          const float m = isnan(sum) ? sum : sum == 0.f ? -INFINITY : base + (float)(up - stay);
          const float f = whole ? (sum == 0.f ? 0.f : 1.f / sum) : exp2_int(stay);
          if (!whole) sum *= f;
          s_l[tid] = fa * f * ua;
          s_l[N + tid] = fb * f * ub;
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
        if (keys) {  // the last P V, and with it all before
          const int last = gs + n - 1;
          if (!__all_sync(0xffffffffu, mbar_wait(&bar_o[last & 1], (last >> 1) & 1, abort_flag))) ok = false;
          tc_fence_after();
        }
        if (!named_bar_and(3, 256, ok)) {
          ok = false;
          break;
        }
        const bool has[2] = {keys && (n > 1 || !(gs & 1)), keys && (n > 1 || (gs & 1))};  // warpgroups that had a tile
#pragma unroll 1
        for (int x = me_g; x < C::VST * quads; x += 2) {
          const int vb = x / quads, c = x - vb * quads;
          float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            if (!has[g]) continue;
            uint32_t u[16];
            tmem_ld16(lanes + g * C::TM_O + vb * C::NT + c * 16, u);
            tmem_wait_ld();
            fence16(u);
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] = fmaf(terms_sum(u, r), s_l[g * N + c * 4 + r], v[r]);
          }
          int ti = c * 4 / p.block_heads, h = c * 4 - ti * p.block_heads;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int i = c * 4 + r;
            if (i < rows && h < un.heads) {
              if (whole) {
                T* at = static_cast<T*>(p.o) + ((row0 + ti) * p.hq + un.head0 + h) * DV + vb * 128 + tid;
                if (SDPA_ADDR_OK(p.chk, at, 2)) *reinterpret_cast<uint16_t*>(at) = (uint16_t)E::pack(v[r], 0.f);
              } else {
                float* at = part + i * DV + vb * 128 + tid;
                if (SDPA_ADDR_OK(p.chk, at, 4)) *at = v[r];
              }
            }
            if (++h == p.block_heads) {
              h = 0;
              ++ti;
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
  if (warp == C::W_MMA) {
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
  if (head_dim == 128 && n == 8) ROWS(128, 128, 8);
  if (head_dim == 192 && n == 8) ROWS(192, 128, 8);
  if (head_dim == 256 && n == 8) ROWS(256, 256, 8);
  if (head_dim == 512 && n == 8) ROWS(512, 512, 8);
  if (head_dim == 128 && n == 16) ROWS(128, 128, 16);
  if (head_dim == 128 && n == 32) ROWS(128, 128, 32);
  if (head_dim == 192 && n == 16) ROWS(192, 128, 16);
  if (head_dim == 192 && n == 32) ROWS(192, 128, 32);
  if (head_dim == 256 && n == 16) ROWS(256, 256, 16);
#undef ROWS
  return SDPA_ERR_UNSUPPORTED;
}

}  // namespace sdpa
