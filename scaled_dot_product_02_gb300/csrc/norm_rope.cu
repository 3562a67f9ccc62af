// norm_rope.cu -- per-head norm of queries and keys with the position rotation
// in the same pass, its gradient, and the append of new rows to a paged cache
// (which is the same pass with other destinations).
//
// One row x is head_dim values of one head of one token:
//   r = 1 / sqrt(mean(x^2) + eps),  y = x r w,  and the first `rot` values of y
//   turn in pairs (a, b) by the token's angle: (a c - b s, b c + a s).
// Backward, with g the output's gradient turned back and h = g w:
//   dx = r h - x r^3 mean(h x),   dw = sum over rows of g x r.
// All of it is in fp32 from the 16-bit inputs and rounds once at the store.
//
// Memory-bound: every row is read once and written once. A row is shared by
// LPH lanes of a warp, each holding VPL 16-byte vectors of it, so a warp reads
// SUB = 32 / LPH rows of one token side by side and the statistics are one
// butterfly over LPH lanes. What keeps it from the memory's rate is the number
// of instructions per value, so a token's cosines and sines and the weights
// are folded into two coefficients a value, shared by all heads of a warp:
//   y' = r (x A + z B),   A = w cos,  B = +-(partner's w) sin,  z = x's partner,
// in packed pairs. A pair (i, i + rot/2) lies in two vectors: the partner's
// vector is loaded a second time (an L1 hit, issued with the first load), which
// serves every rot with one code path and no exchange of lanes.
//
// Measured (bf16, 18000 tokens, 32 + 8 heads of 128): forward 67 us, 5.6 TB/s;
// gradient 94 us, 6.0 TB/s. The append copies 14035 rows of width 256 in 39 us,
// 5.9 TB/s.
#include <algorithm>
#include <cuda_runtime.h>

#include "common.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace sdpa {

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

template <int D>
struct Row {
  static constexpr int VECS = D / 8;  // 16-byte vectors of a row
  static constexpr int LPH = D == 128 ? 16 : 32;           // D = 192: the last eight lanes of a row idle
  static constexpr int VPL = (VECS + LPH - 1) / LPH;
  static constexpr int SUB = 32 / LPH;
  static constexpr int UNROLL = 4 / VPL > 1 ? 4 / VPL : 1;  // rows a lane has in flight
  static constexpr int STEP = SUB * UNROLL;                 // heads of one step of a warp
  // heads of one tensor that a warp takes: a step, or several where a step is so
  // few rows that loading the angles for it would cost as much as the rows
  static constexpr int HEADS = STEP > 4 ? STEP : 4;
  static constexpr int DV = D == 192 ? 128 : D;  // width of a value row
  // whether vector idx lies in a row of `width` values (always, but for the idle lanes)
  static __device__ __forceinline__ bool in(int idx, int width) { return VPL * LPH == DV / 8 || idx * 8 < width; }
};

__device__ __forceinline__ uint4 load16(AddrTable* chk, const void* p) {
  return SDPA_ADDR_OK(chk, p, 16) ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0u, 0u, 0u, 0u);
}
__device__ __forceinline__ void store16(AddrTable* chk, void* p, uint4 v) {
  if (SDPA_ADDR_OK(chk, p, 16)) *reinterpret_cast<uint4*>(p) = v;
}
__device__ __forceinline__ int load_i32(AddrTable* chk, const int32_t* p, int otherwise) {
  return SDPA_ADDR_OK(chk, p, 4) ? __ldg(p) : otherwise;
}

template <class E>
__device__ __forceinline__ void unpack8(const uint4& x, float2 (&f)[4]) {
  f[0] = E::unpack(x.x);
  f[1] = E::unpack(x.y);
  f[2] = E::unpack(x.z);
  f[3] = E::unpack(x.w);
}
template <class E>
__device__ __forceinline__ uint4 pack8(const float2 (&f)[4]) {
  return make_uint4(E::pack(f[0].x, f[0].y), E::pack(f[1].x, f[1].y), E::pack(f[2].x, f[2].y), E::pack(f[3].x, f[3].y));
}

template <int LPH>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LPH / 2; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// Both sums over the LPH lanes of a row, with one exchange more than one sum's:
// half of the lanes reduce a, the other half b.
template <int LPH>
__device__ __forceinline__ void row_sums(float& a, float& b, int lane) {
  constexpr int H = LPH / 2;
  const bool up = lane & H;
  float v = (up ? b : a) + __shfl_xor_sync(0xffffffffu, up ? a : b, H);
#pragma unroll
  for (int o = H / 2; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
  const float w = __shfl_xor_sync(0xffffffffu, v, H);
  a = up ? w : v;
  b = up ? v : w;
}

// Which of a lane's vectors turns, and the vector that holds its pairs' other
// halves (itself for adjacent pairs).
struct Place {
  bool on, second;
  int partner;
};
__device__ __forceinline__ Place place_of(int idx, int rot, bool interleaved) {
  Place t;
  const int half = rot / 2;  // a multiple of 8: a vector lies in one half
  t.on = idx * 8 < rot;
  t.second = !interleaved && idx * 8 >= half;
  t.partner = !t.on || interleaved ? idx : t.second ? idx - half / 8 : idx + half / 8;
  return t;
}
// The cosines of vector idx and its sines, signed for turning forwards: value e
// becomes y_e c_e + partner_e s_e.
template <bool SHARED = false>
__device__ __forceinline__ void angles_of(const Place& t, int idx, const float* row, int rot, bool interleaved,
                                          float2 (&c)[4], float2 (&s)[4], AddrTable* chk) {
  const int half = rot / 2;
  auto get = [&](const float* from) { return SHARED ? *reinterpret_cast<const uint4*>(from) : load16(chk, from); };
  if (!t.on) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      c[e] = make_float2(1.f, 1.f);
      s[e] = make_float2(0.f, 0.f);
    }
  } else if (interleaved) {
    const uint4 a = get(row + idx * 4), b = get(row + half + idx * 4);
    const float cs[4] = {__uint_as_float(a.x), __uint_as_float(a.y), __uint_as_float(a.z), __uint_as_float(a.w)};
    const float sn[4] = {__uint_as_float(b.x), __uint_as_float(b.y), __uint_as_float(b.z), __uint_as_float(b.w)};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      c[e] = make_float2(cs[e], cs[e]);
      s[e] = make_float2(-sn[e], sn[e]);
    }
  } else {
    const int i0 = idx * 8 - (t.second ? half : 0);
    const float sg = t.second ? 1.f : -1.f;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint4 a = get(row + i0 + q * 4), b = get(row + half + i0 + q * 4);
      c[2 * q] = make_float2(__uint_as_float(a.x), __uint_as_float(a.y));
      c[2 * q + 1] = make_float2(__uint_as_float(a.z), __uint_as_float(a.w));
      s[2 * q] = make_float2(sg * __uint_as_float(b.x), sg * __uint_as_float(b.y));
      s[2 * q + 1] = make_float2(sg * __uint_as_float(b.z), sg * __uint_as_float(b.w));
    }
  }
}

// Where a token of the packed batch goes in the cache.
struct Slot {
  bool live;     // its rows are written
  int position;  // in its sequence
  long long k_at, v_at;  // element offsets of head 0
};

// The sequence of a token is the number of sequences that end at or before it
// (32 ends per step of the warp, so a batch of 32 takes one step).
__device__ __forceinline__ Slot find_slot(const NormRopeParams& p, long long row, int lane) {
  Slot s;
  s.live = false;
  s.position = 0;
  s.k_at = s.v_at = 0;
  int b = 0;
  for (int base = 0; base < p.batch; base += 32) {
    const int i = base + lane;
    const bool behind = i < p.batch && load_i32(p.chk, p.cu_q + i + 1, 0) <= row;
    b += __popc(__ballot_sync(0xffffffffu, behind));
  }
  if (b >= p.batch) return s;  // behind the last sequence
  const int first = load_i32(p.chk, p.cu_q + b, 0), end = load_i32(p.chk, p.cu_q + b + 1, 0);
  const long long pos = (long long)load_i32(p.chk, p.kv_lens + b, 0) - (end - row);
  const long long col = pos / p.page_size;
  if (first > row || end <= row || end > p.rows || pos < 0 || col >= p.max_pages) {
    if (lane == 0) record_error(p.err, SDPA_ERR_BAD_SEQLENS);
    return s;
  }
  const int page = load_i32(p.chk, p.table_ids + b * p.table_stride + col, -1);
  if (page < 0 || page >= p.num_pages) {
    if (lane == 0) record_error(p.err, SDPA_ERR_BAD_INDEX);
    return s;
  }
  const int slot = (int)(pos - col * p.page_size);
  s.live = true;
  s.position = (int)pos;
  s.k_at = page * p.kc_page + slot * p.kc_slot;
  s.v_at = page * p.vc_page + slot * p.vc_slot;
  return s;
}

// A warp takes Row::HEADS heads of one tensor (q, k or, appending, v) of one token.
template <bool BF16, int D, bool APPEND, bool NORM>
__global__ void __launch_bounds__(kThreads, Row<D>::VPL == 1 ? 6 : 4)
    norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  using E = Elem<BF16>;
  using T = typename E::T;
  using R = Row<D>;
  const int lane = threadIdx.x % 32, sub = lane % R::LPH, grp = lane / R::LPH;
  const long long w = (long long)blockIdx.x * kWarps + threadIdx.x / 32;
  const long long row = w / p.parts;
  if (row >= p.rows) return;
  int part = (int)(w - row * p.parts);
  const bool is_q = part < p.parts_q;
  if (!is_q) part -= p.parts_q;
  const bool is_v = APPEND && !is_q && part >= p.parts_k;
  if (is_v) part -= p.parts_k;
  const int heads = is_q ? p.hq : p.hkv;
  const int h_end = min(heads, (part + 1) * R::HEADS);
  const int width = is_v ? R::DV : D;
  const T* src = is_q   ? static_cast<const T*>(p.q) + row * p.qs
                 : is_v ? static_cast<const T*>(p.v) + row * p.vs
                        : static_cast<const T*>(p.k) + row * p.ks;
  const bool inter = p.interleaved != 0;
  Place at[R::VPL];
#pragma unroll
  for (int v = 0; v < R::VPL; ++v) at[v] = place_of(v * R::LPH + sub, NORM ? p.rot : 0, inter);

  uint4 x[R::UNROLL][R::VPL], z[R::UNROLL][R::VPL];
  auto fetch = [&](int h0) {
#pragma unroll
    for (int u = 0; u < R::UNROLL; ++u) {
      const int h = h0 + grp + u * R::SUB;
#pragma unroll
      for (int v = 0; v < R::VPL; ++v) {
        const bool in = h < h_end && R::in(v * R::LPH + sub, width);
        x[u][v] = z[u][v] = make_uint4(0u, 0u, 0u, 0u);
        if (in) x[u][v] = load16(p.chk, src + h * width + (v * R::LPH + sub) * 8);
        if (NORM && in && !is_v && at[v].on && !inter) z[u][v] = load16(p.chk, src + h * width + at[v].partner * 8);
      }
    }
  };
  int h0 = part * R::HEADS;
  fetch(h0);

  Slot slot;
  if (APPEND) {
    slot = find_slot(p, row, lane);
    if (!slot.live) return;
  }
  // where head h of this tensor goes
  T* dst = is_q ? static_cast<T*>(p.q_out) + row * p.hq * D : static_cast<T*>(p.k_out) + row * p.hkv * D;
  long long step = D;
  if (APPEND && !is_q) {
    dst = is_v ? static_cast<T*>(p.vc) + slot.v_at : static_cast<T*>(p.kc) + slot.k_at;
    step = is_v ? p.vc_head : p.kc_head;
  }
  float2 ca[R::VPL][4], cb[R::VPL][4];
  if (NORM && !is_v) {
    const float* angles = nullptr;
    if (p.rot > 0) {
      const int pos = APPEND && !p.pos ? slot.position : load_i32(p.chk, p.pos + row, -1);
      if (pos < 0 || pos >= p.max_pos) {
        if (lane == 0) record_error(p.err, SDPA_ERR_BAD_INDEX);
        return;
      }
      angles = p.table + (long long)pos * p.rot;
    }
    const T* weight = static_cast<const T*>(is_q ? p.wq : p.wk);
#pragma unroll
    for (int v = 0; v < R::VPL; ++v) {
      const int idx = v * R::LPH + sub;
      float2 c[4], s[4], wt[4], wp[4];
      const bool in = R::in(idx, D);
      unpack8<E>(in ? load16(p.chk, weight + idx * 8) : make_uint4(0u, 0u, 0u, 0u), wt);
      unpack8<E>(in ? load16(p.chk, weight + at[v].partner * 8) : make_uint4(0u, 0u, 0u, 0u), wp);
      angles_of(at[v], idx, angles, p.rot, inter, c, s, p.chk);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        ca[v][e] = fmul2(wt[e], c[e]);
        cb[v][e] = fmul2(inter ? make_float2(wp[e].y, wp[e].x) : wp[e], s[e]);
      }
    }
  } else if (NORM && APPEND && p.rot > 0) {
    const int pos = p.pos ? load_i32(p.chk, p.pos + row, -1) : slot.position;  // a token with a bad one is skipped whole
    if (pos < 0 || pos >= p.max_pos) return;
  }

  while (true) {
#pragma unroll
    for (int u = 0; u < R::UNROLL; ++u) {
      const int h = h0 + grp + u * R::SUB;
      if (NORM && !is_v) {
        float2 f[R::VPL][4], ss = make_float2(0.f, 0.f);
#pragma unroll
        for (int v = 0; v < R::VPL; ++v) {
          unpack8<E>(x[u][v], f[v]);
#pragma unroll
          for (int e = 0; e < 4; ++e) ss = ffma2(f[v][e], f[v][e], ss);
        }
        const float r1 = rsqrtf(row_sum<R::LPH>(ss.x + ss.y) * (1.f / D) + p.eps);
        const float2 r = make_float2(r1, r1);
#pragma unroll
        for (int v = 0; v < R::VPL; ++v) {
          float2 g[4];
          unpack8<E>(z[u][v], g);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 other = inter ? make_float2(f[v][e].y, f[v][e].x) : g[e];
            const float2 t = fmul2(f[v][e], ca[v][e]);
            g[e] = fmul2(at[v].on ? ffma2(other, cb[v][e], t) : t, r);
          }
          x[u][v] = pack8<E>(g);
        }
      }
      if (h >= h_end) continue;
#pragma unroll
      for (int v = 0; v < R::VPL; ++v)
        if (R::in(v * R::LPH + sub, width)) store16(p.chk, dst + h * step + (v * R::LPH + sub) * 8, x[u][v]);
    }
    h0 += R::STEP;
    if (h0 >= h_end) break;
    fetch(h0);
  }
}

// ---------------------------------------------------------------- many tokens
// With many tokens the rows come through shared memory: every warp owns a ring
// of stages and walks its own units -- a share of one tensor's heads of one
// token, with the token's angles -- so the next units' bulk copies are in flight
// while it works on one, without costing registers. (Loads to registers, one
// unit a warp, reached 3.8 TB/s with 24 warps an SM: too few bytes in flight for
// a chain of position, angles, rows and stores.) The warps meet nowhere.
constexpr int kFwdWarps = 24;  // 24 x 32 threads of at most 85 registers; the gradient needs 128
constexpr int kBwdWarps = 16;
constexpr int kRingSmem = 232448 - 2048;  // of the 227 KB, less the barriers

// Shared memory of a warp's stage: bytes of rows, then the angles.
template <int D>
struct RingRows {
  static constexpr int FWD_HEADS = 4096 / (2 * D);  // heads of a unit: 4 KB of rows
  static constexpr int BWD_HEADS = 2048 / (2 * D);  // of each of x and dy
};

// A warp's units lie `stride` apart in the order (row, part): a cursor steps
// through them without dividing.
struct RingCursor {
  long long row, step_row;
  int part, step_part, parts;
  __device__ __forceinline__ void start(long long unit, long long stride, int parts_) {
    parts = parts_;
    row = unit / parts;
    part = (int)(unit - row * parts);
    step_row = stride / parts;
    step_part = (int)(stride - step_row * parts);
  }
  __device__ __forceinline__ void next() {
    row += step_row;
    part += step_part;
    if (part >= parts) {
      part -= parts;
      ++row;
    }
  }
};

// The stages of one warp. Filled by its lane 0; `pos` of the units in flight
// are in the callers' registers.
struct Ring {
  uint8_t* base;
  uint64_t* bar;
  int stage_bytes, stages;
  volatile int* abort_flag;
  __device__ __forceinline__ uint8_t* at(int i) const { return base + (i % stages) * stage_bytes; }
  __device__ __forceinline__ uint64_t* bar_of(int i) const { return &bar[i % stages]; }
  __device__ __forceinline__ bool wait(int i) const {
    return __all_sync(0xffffffffu, mbar_wait(bar_of(i), (i / stages) & 1, abort_flag));
  }
};
__device__ __forceinline__ void ring_copy(AddrTable* chk, void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  if (SDPA_ADDR_OK(chk, src, bytes))
    bulk_load(dst, src, bytes, bar);
  else
    mbar_complete_tx(bar, bytes);
}

template <bool BF16, int D, bool INTER>
__global__ void __launch_bounds__(kFwdWarps * 32, 1) norm_rope_ring_kernel(const __grid_constant__ NormRopeParams p) {
  using E = Elem<BF16>;
  using T = typename E::T;
  using R = Row<D>;
  constexpr int HEADS = RingRows<D>::FWD_HEADS;
  constexpr int UN = R::VPL == 1 ? 4 : 1;  // rows a lane works on at a time
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t bars[kFwdWarps][4];
  __shared__ int s_abort;
  const int lane = threadIdx.x % 32, sub = lane % R::LPH, grp = lane / R::LPH, warp = threadIdx.x / 32;
  Ring ring{smem + warp * p.stages * p.stage_bytes, bars[warp], p.stage_bytes, p.stages, &s_abort};
  if (threadIdx.x == 0) s_abort = 0;
  if (lane == 0) {
    for (int i = 0; i < p.stages; ++i) mbar_init(&ring.bar[i], 1);
    fence_mbar_init();
  }
  __syncthreads();
  Place at[R::VPL];
#pragma unroll
  for (int v = 0; v < R::VPL; ++v) at[v] = place_of(v * R::LPH + sub, p.rot, INTER);
  const long long units = p.rows * p.parts, stride = (long long)gridDim.x * kFwdWarps;
  const long long first = (long long)blockIdx.x * kFwdWarps + warp;
  const int mine = first < units ? (int)((units - first + stride - 1) / stride) : 0;
  RingCursor cur, fil, ahead;  // the unit at work, the next to copy, the next whose position is read
  cur.start(first, stride, p.parts);
  fil = ahead = cur;
  int n_ahead = 0;
  auto position = [&]() {
    const int x = p.rot > 0 && n_ahead < mine ? load_i32(p.chk, p.pos + ahead.row, -1) : 0;
    ++n_ahead;
    ahead.next();
    return x;
  };
  auto bad = [&](int pos) { return p.rot > 0 && (pos < 0 || pos >= p.max_pos); };
  // heads of a unit and where they start
  auto heads_of = [&](int part, bool& is_q, int& h0) {
    is_q = part < p.parts_q;
    h0 = (is_q ? part : part - p.parts_q) * HEADS;
    return min(HEADS, (is_q ? p.hq : p.hkv) - h0);
  };
  int filled = 0;
  auto fill = [&](int pos) {
    if (filled < mine && lane == 0) {
      uint64_t* bar = ring.bar_of(filled);
      if (bad(pos)) {  // not copied: an empty arrival passes the stage's phase
        mbar_arrive(bar);
      } else {
        bool is_q;
        int h0;
        const int n = heads_of(fil.part, is_q, h0);
        const T* src = (is_q ? static_cast<const T*>(p.q) + fil.row * p.qs : static_cast<const T*>(p.k) + fil.row * p.ks) + h0 * D;
        mbar_arrive_expect_tx(bar, n * D * 2 + p.rot * 4);
        ring_copy(p.chk, ring.at(filled), src, n * D * 2, bar);
        if (p.rot > 0)
          ring_copy(p.chk, ring.at(filled) + HEADS * D * 2, p.table + (long long)pos * p.rot, p.rot * 4, bar);
      }
    }
    if (filled < mine) ++filled;
    fil.next();
  };
  int pos[4];  // positions of the units in flight, oldest first, and of the next one
#pragma unroll
  for (int i = 0; i < 4; ++i) pos[i] = position();
#pragma unroll
  for (int i = 0; i < 3; ++i)
    if (i < p.stages) fill(pos[i]);
  for (int i = 0; i < mine; ++i) {
    const int later = position();
    if (!ring.wait(i)) {
      if (lane == 0) {
        *ring.abort_flag = 1;
        record_error(p.err, SDPA_ERR_TIMEOUT);
      }
      break;
    }
    if (bad(pos[0])) {
      if (lane == 0) record_error(p.err, SDPA_ERR_BAD_INDEX);
    } else {
      bool is_q;
      int h0;
      const int n = heads_of(cur.part, is_q, h0);
      const uint8_t* st = ring.at(i);
      const T* weight = static_cast<const T*>(is_q ? p.wq : p.wk);
      float2 ca[R::VPL][4], cb[R::VPL][4];
#pragma unroll
      for (int v = 0; v < R::VPL; ++v) {
        const int idx = v * R::LPH + sub;
        float2 c[4], s[4], wt[4], wp[4];
        const bool in = R::in(idx, D);
        unpack8<E>(in ? load16(p.chk, weight + idx * 8) : make_uint4(0u, 0u, 0u, 0u), wt);
        unpack8<E>(in ? load16(p.chk, weight + at[v].partner * 8) : make_uint4(0u, 0u, 0u, 0u), wp);
        angles_of<true>(at[v], idx, reinterpret_cast<const float*>(st + HEADS * D * 2), p.rot, INTER, c, s, p.chk);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          ca[v][e] = fmul2(wt[e], c[e]);
          // where nothing turns the sine is zero; a weight that is not finite must not meet it
          cb[v][e] = at[v].on ? fmul2(INTER ? make_float2(wp[e].y, wp[e].x) : wp[e], s[e]) : make_float2(0.f, 0.f);
        }
      }
      T* dst = (is_q ? static_cast<T*>(p.q_out) + cur.row * p.hq * D : static_cast<T*>(p.k_out) + cur.row * p.hkv * D) + h0 * D;
#pragma unroll 1
      for (int hh = 0; hh < n; hh += R::SUB * UN) {
#pragma unroll
        for (int x = 0; x < UN; ++x) {
          const int h = min(hh + grp + x * R::SUB, n - 1);  // rows past the end repeat the last one, unstored
          const T* row = reinterpret_cast<const T*>(st) + h * D;
          float2 f[R::VPL][4], g[R::VPL][4], ss = make_float2(0.f, 0.f);
#pragma unroll
          for (int v = 0; v < R::VPL; ++v) {
            const int idx = v * R::LPH + sub;
            const bool in = R::in(idx, D);
            unpack8<E>(in ? *reinterpret_cast<const uint4*>(row + idx * 8) : make_uint4(0u, 0u, 0u, 0u), f[v]);
            unpack8<E>(!INTER && in && at[v].on ? *reinterpret_cast<const uint4*>(row + at[v].partner * 8)
                                                : make_uint4(0u, 0u, 0u, 0u),
                       g[v]);
#pragma unroll
            for (int e = 0; e < 4; ++e) ss = ffma2(f[v][e], f[v][e], ss);
          }
          const float r1 = rsqrtf(row_sum<R::LPH>(ss.x + ss.y) * (1.f / D) + p.eps);
          const float2 r = make_float2(r1, r1);
#pragma unroll
          for (int v = 0; v < R::VPL; ++v) {
            const int idx = v * R::LPH + sub;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              // where nothing turns, g or cb are zeros; a neighbour that is not finite must not meet them
              const float2 other = !INTER ? g[v][e] : at[v].on ? make_float2(f[v][e].y, f[v][e].x) : make_float2(0.f, 0.f);
              g[v][e] = fmul2(ffma2(other, cb[v][e], fmul2(f[v][e], ca[v][e])), r);
            }
            if (hh + grp + x * R::SUB < n && R::in(idx, D)) store16(p.chk, dst + h * D + idx * 8, pack8<E>(g[v]));
          }
        }
      }
    }
    __syncwarp();  // every lane has read the stage
    fill(p.stages == 3 ? pos[3] : p.stages == 2 ? pos[2] : pos[1]);
    cur.next();
#pragma unroll
    for (int x = 0; x < 3; ++x) pos[x] = pos[x + 1];
    pos[3] = later;
  }
  // every copy lands before the CTA ends (all have, unless a wait gave up)
  if (lane == 0)
    for (int i = max(0, filled - p.stages); i < filled; ++i) mbar_wait_drain(ring.bar_of(i), (i / p.stages) & 1);
}

// Gradient, through the same rings. Warps [0, warps_q) of the grid serve q, the
// others k, in proportion to their work; a warp keeps its sums of dw in
// registers. Block b writes the sum of its q warps to slot b and that of its k
// warps to slot b + 1 (only one block can have both); dw_kernel adds the slots
// in order.
template <bool BF16, int D, bool INTER>
__global__ void __launch_bounds__(kBwdWarps * 32, 1) norm_rope_bwd_kernel(const __grid_constant__ NormRopeBwdParams p) {
  using E = Elem<BF16>;
  using T = typename E::T;
  using R = Row<D>;
  constexpr int HEADS = RingRows<D>::BWD_HEADS;
  constexpr int UN = D == 128 ? 2 : 1;  // rows a lane works on at a time (two at 192 to 512 spill)
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t bars[kBwdWarps][4];
  __shared__ int s_abort;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x % 32, sub = lane % R::LPH, grp = lane / R::LPH, warp = threadIdx.x / 32;
  Ring ring{smem + warp * p.stages * p.stage_bytes, bars[warp], p.stage_bytes, p.stages, &s_abort};
  if (threadIdx.x == 0) s_abort = 0;
  if (lane == 0) {
    for (int i = 0; i < p.stages; ++i) mbar_init(&ring.bar[i], 1);
    fence_mbar_init();
  }
  __syncthreads();
  const int gw = blockIdx.x * kBwdWarps + warp;
  const bool is_q = gw < p.warps_q;
  const int heads = is_q ? p.hq : p.hkv, parts = (heads + HEADS - 1) / HEADS;
  const long long xs = is_q ? p.qs : p.ks, ds = is_q ? p.dqs : p.dks;
  const T* const x0 = static_cast<const T*>(is_q ? p.q : p.k);
  const T* const g0 = static_cast<const T*>(is_q ? p.gq : p.gk);
  T* const d0 = static_cast<T*>(is_q ? p.dq : p.dk);
  Place at[R::VPL];
  float2 wt[R::VPL][4], acc[R::VPL][4];
#pragma unroll
  for (int v = 0; v < R::VPL; ++v) {
    at[v] = place_of(v * R::LPH + sub, p.rot, INTER);
    unpack8<E>(R::in(v * R::LPH + sub, D) ? load16(p.chk, static_cast<const T*>(is_q ? p.wq : p.wk) + (v * R::LPH + sub) * 8)
                                          : make_uint4(0u, 0u, 0u, 0u),
               wt[v]);
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[v][e] = make_float2(0.f, 0.f);
  }
  const long long units = p.rows * parts, stride = is_q ? p.warps_q : gridDim.x * kBwdWarps - p.warps_q;
  const long long first = is_q ? gw : gw - p.warps_q;
  const int mine = first < units ? (int)((units - first + stride - 1) / stride) : 0;
  RingCursor cur, fil, ahead;  // the unit at work, the next to copy, the next whose position is read
  cur.start(first, stride, parts);
  fil = ahead = cur;
  int n_ahead = 0;
  auto position = [&]() {
    const int x = p.rot > 0 && n_ahead < mine ? load_i32(p.chk, p.pos + ahead.row, -1) : 0;
    ++n_ahead;
    ahead.next();
    return x;
  };
  auto bad = [&](int pos) { return p.rot > 0 && (pos < 0 || pos >= p.max_pos); };
  constexpr int SIDE = HEADS * D * 2;  // x, then dy, then the angles
  int filled = 0;
  auto fill = [&](int pos) {
    if (filled < mine && lane == 0) {
      uint64_t* bar = ring.bar_of(filled);
      if (bad(pos)) {  // not copied: an empty arrival passes the stage's phase
        mbar_arrive(bar);
      } else {
        const int h0 = fil.part * HEADS, n = min(HEADS, heads - h0);
        uint8_t* st = ring.at(filled);
        mbar_arrive_expect_tx(bar, 2 * n * D * 2 + p.rot * 4);
        ring_copy(p.chk, st, x0 + fil.row * xs + h0 * D, n * D * 2, bar);
        ring_copy(p.chk, st + SIDE, g0 + (fil.row * heads + h0) * D, n * D * 2, bar);
        if (p.rot > 0) ring_copy(p.chk, st + 2 * SIDE, p.table + (long long)pos * p.rot, p.rot * 4, bar);
      }
    }
    if (filled < mine) ++filled;
    fil.next();
  };
  int pos[4];  // positions of the units in flight, oldest first, and of the next one
#pragma unroll
  for (int i = 0; i < 4; ++i) pos[i] = position();
#pragma unroll
  for (int i = 0; i < 3; ++i)
    if (i < p.stages) fill(pos[i]);
  for (int i = 0; i < mine; ++i) {
    const int later = position();
    if (!ring.wait(i)) {
      if (lane == 0) {
        *ring.abort_flag = 1;
        record_error(p.err, SDPA_ERR_TIMEOUT);
      }
      break;
    }
    const int h0 = cur.part * HEADS, n = min(HEADS, heads - h0);
    const uint8_t* st = ring.at(i);
    T* dst = d0 + cur.row * ds + h0 * D;
    if (bad(pos[0])) {  // a position outside the table: zeros
      if (lane == 0) record_error(p.err, SDPA_ERR_BAD_INDEX);
      for (int x = lane; x < n * D / 8; x += 32) store16(p.chk, dst + x * 8, make_uint4(0u, 0u, 0u, 0u));
    } else {
      float2 c[R::VPL][4], s[R::VPL][4];
#pragma unroll
      for (int v = 0; v < R::VPL; ++v) {
        angles_of<true>(at[v], v * R::LPH + sub, reinterpret_cast<const float*>(st + 2 * SIDE), p.rot, INTER, c[v], s[v],
                        p.chk);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[v][e] = make_float2(-s[v][e].x, -s[v][e].y);  // turned back
      }
#pragma unroll 1
      for (int hh = 0; hh < n; hh += R::SUB * UN) {
#pragma unroll
        for (int x = 0; x < UN; ++x) {
          const int h = min(hh + grp + x * R::SUB, n - 1);  // rows past the end repeat the last one, unused
          const T* xr = reinterpret_cast<const T*>(st) + h * D;
          const T* gr = reinterpret_cast<const T*>(st + SIDE) + h * D;
          float2 f[R::VPL][4], g[R::VPL][4];
          float2 ss = make_float2(0.f, 0.f), dot = make_float2(0.f, 0.f);
#pragma unroll
          for (int v = 0; v < R::VPL; ++v) {
            const int idx = v * R::LPH + sub;
            const bool in = R::in(idx, D);
            const uint4 none = make_uint4(0u, 0u, 0u, 0u);
            float2 o[4];
            unpack8<E>(in ? *reinterpret_cast<const uint4*>(xr + idx * 8) : none, f[v]);
            unpack8<E>(in ? *reinterpret_cast<const uint4*>(gr + idx * 8) : none, g[v]);
            unpack8<E>(!INTER && in && at[v].on ? *reinterpret_cast<const uint4*>(gr + at[v].partner * 8) : none, o);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              // where nothing turns, o or s are zeros; a neighbour that is not finite must not meet them
              const float2 other = !INTER ? o[e] : at[v].on ? make_float2(g[v][e].y, g[v][e].x) : make_float2(0.f, 0.f);
              g[v][e] = ffma2(other, s[v][e], fmul2(g[v][e], c[v][e]));
              ss = ffma2(f[v][e], f[v][e], ss);
              dot = ffma2(fmul2(g[v][e], wt[v][e]), f[v][e], dot);
            }
          }
          float a = ss.x + ss.y, b = dot.x + dot.y;
          row_sums<R::LPH>(a, b, lane);
          if (hh + grp + x * R::SUB >= n) continue;
          // r^3 by itself would leave fp32's range for rows of 1e15 (or, with eps 0, 1e-13): the mean, some 1 / r, first
          const float r1 = rsqrtf(a * (1.f / D) + p.eps), k1 = -(r1 * (b * (1.f / D))) * r1 * r1;
          const float2 r = make_float2(r1, r1), k3 = make_float2(k1, k1);
#pragma unroll
          for (int v = 0; v < R::VPL; ++v) {
            const int idx = v * R::LPH + sub;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 t = fmul2(g[v][e], r);
              acc[v][e] = ffma2(t, f[v][e], acc[v][e]);
              f[v][e] = ffma2(k3, f[v][e], fmul2(t, wt[v][e]));
            }
            if (R::in(idx, D)) store16(p.chk, dst + h * D + idx * 8, pack8<E>(f[v]));
          }
        }
      }
    }
    __syncwarp();  // every lane has read the stage
    fill(p.stages == 3 ? pos[3] : p.stages == 2 ? pos[2] : pos[1]);
    cur.next();
#pragma unroll
    for (int x = 0; x < 3; ++x) pos[x] = pos[x + 1];
    pos[3] = later;
  }
  // every copy lands before the CTA ends (all have, unless a wait gave up)
  if (lane == 0)
    for (int i = max(0, filled - p.stages); i < filled; ++i) mbar_wait_drain(ring.bar_of(i), (i / p.stages) & 1);
  // the block's sums of dw, in the rings' memory: row groups of a warp by shuffles, warps in order
  __syncthreads();
  float* sum = reinterpret_cast<float*>(smem);  // [kBwdWarps][D]
#pragma unroll
  for (int v = 0; v < R::VPL; ++v)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
#pragma unroll
      for (int o = R::LPH; o < 32; o *= 2) {
        acc[v][e].x += __shfl_xor_sync(0xffffffffu, acc[v][e].x, o);
        acc[v][e].y += __shfl_xor_sync(0xffffffffu, acc[v][e].y, o);
      }
      if (grp == 0 && R::in(v * R::LPH + sub, D))
        *reinterpret_cast<float2*>(sum + warp * D + (v * R::LPH + sub) * 8 + 2 * e) = acc[v][e];
    }
  __syncthreads();
  const int q_warps = min(max(p.warps_q - (int)blockIdx.x * kBwdWarps, 0), kBwdWarps);
  for (int i = threadIdx.x; i < 2 * D; i += kBwdWarps * 32) {
    const bool q_side = i < D;
    if (q_side ? q_warps == 0 : q_warps == kBwdWarps) continue;
    float t = 0.f;
    for (int k = q_side ? 0 : q_warps; k < (q_side ? q_warps : kBwdWarps); ++k) t += sum[k * D + i % D];
    float* to = p.part + (long long)(blockIdx.x + (q_side ? 0 : 1)) * D + i % D;
    if (SDPA_ADDR_OK(p.chk, to, 4)) *to = t;
  }
}

// dw = the blocks' partial sums, added in a fixed order: 16 columns of q's or
// k's weights per CTA, 32 threads a column, each over every 32nd slot.
// Slots [0, end_q) are q's, [first_k, slots) k's.
__global__ void __launch_bounds__(512) dw_kernel(const float* part, int end_q, int first_k, int slots, int d, float* dwq,
                                                 float* dwk, AddrTable* chk) {
  __shared__ float sum[32][17];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int x = threadIdx.x % 16, k = threadIdx.x / 16, at = blockIdx.x * 16 + x;
  const bool is_q = at < d;
  const int col = is_q ? at : at - d, end = is_q ? end_q : slots;
  float t = 0.f;
#pragma unroll 8
  for (int b = (is_q ? 0 : first_k) + k; b < end; b += 32) {
    const float* from = part + (long long)b * d + col;
    t += SDPA_ADDR_OK(chk, from, 4) ? *from : 0.f;
  }
  sum[k][x] = t;
  __syncthreads();
  if (k == 0) {
#pragma unroll
    for (int i = 1; i < 32; ++i) t += sum[i][x];
    float* to = is_q ? dwq + col : dwk + col;
    if (SDPA_ADDR_OK(chk, to, 4)) *to = t;
  }
}

// Stages of a warp's ring, each `bytes`: at most three, as many as fit.
int ring_stages(int bytes, int warps) { return std::min(3, kRingSmem / (warps * bytes)); }

template <bool BF16, int D>
int launch_t(NormRopeParams p, bool append, cudaStream_t s) {
  using R = Row<D>;
  if (!append) {
    constexpr int HEADS = RingRows<D>::FWD_HEADS;
    const int parts_q = (p.hq + HEADS - 1) / HEADS, parts_k = (p.hkv + HEADS - 1) / HEADS;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return SDPA_ERR_CUDA;
    // the rings pay from a few units a warp on; below, registers are quicker to start
    if (p.rows * (parts_q + parts_k) >= (long long)sms * kFwdWarps * 2) {
      auto kern = p.interleaved ? norm_rope_ring_kernel<BF16, D, true> : norm_rope_ring_kernel<BF16, D, false>;
      p.parts_q = parts_q;
      p.parts = parts_q + parts_k;
      p.stage_bytes = HEADS * D * 2 + p.rot * 4;
      p.stages = ring_stages(p.stage_bytes, kFwdWarps);
      if (const int rc = set_kernel_smem(reinterpret_cast<const void*>(kern), kRingSmem, 100)) return rc;
      kern<<<(unsigned)sms, kFwdWarps * 32, kFwdWarps * p.stages * p.stage_bytes, s>>>(p);
      return cudaGetLastError() == cudaSuccess ? SDPA_OK : SDPA_ERR_CUDA;
    }
  }
  p.parts_q = (p.hq + R::HEADS - 1) / R::HEADS;
  p.parts_k = (p.hkv + R::HEADS - 1) / R::HEADS;
  p.parts = p.parts_q + (append ? 2 : 1) * p.parts_k;
  const long long blocks = (p.rows * p.parts + kWarps - 1) / kWarps;
  if (blocks > 0x7fffffffLL) return SDPA_ERR_UNSUPPORTED;
  const unsigned grid = (unsigned)blocks;
  if (!append)
    norm_rope_kernel<BF16, D, false, true><<<grid, kThreads, 0, s>>>(p);
  else if (p.wk)
    norm_rope_kernel<BF16, D, true, true><<<grid, kThreads, 0, s>>>(p);
  else
    norm_rope_kernel<BF16, D, true, false><<<grid, kThreads, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? SDPA_OK : SDPA_ERR_CUDA;
}

template <bool BF16, int D>
int launch_bwd_t(NormRopeBwdParams p, cudaStream_t s) {
  auto kern = p.interleaved ? norm_rope_bwd_kernel<BF16, D, true> : norm_rope_bwd_kernel<BF16, D, false>;
  p.stage_bytes = 2 * RingRows<D>::BWD_HEADS * D * 2 + p.rot * 4;
  p.stages = ring_stages(p.stage_bytes, kBwdWarps);
  if (const int rc = set_kernel_smem(reinterpret_cast<const void*>(kern), kRingSmem, 100)) return rc;
  const int bytes = std::max(kBwdWarps * p.stages * p.stage_bytes, kBwdWarps * D * 4);
  kern<<<(unsigned)p.blocks, kBwdWarps * 32, bytes, s>>>(p);
  if (cudaGetLastError() != cudaSuccess) return SDPA_ERR_CUDA;
  // started while the kernel above runs (with its split of an SM between L1 and shared memory); it waits for it
  // before reading
  if (const int rc = set_kernel_smem(reinterpret_cast<const void*>(&dw_kernel), 0, 100)) return rc;
  return launch_early(dw_kernel, dim3(2 * D / 16), 512, 0, s, true, (const float*)p.part, (p.warps_q + kBwdWarps - 1) / kBwdWarps,
                      p.warps_q / kBwdWarps + 1, p.blocks + 1, D, p.dwq, p.dwk, p.chk);
}

}  // namespace

NormRopeBwdPlan norm_rope_bwd_plan(long long rows, int hq, int hkv, int head_dim) {
  // one block on each of the 152 SMs of the device this is written for: the
  // plan must not depend on the device in use, since the workspace size is
  // asked for without one, and the order of the sums follows from it
  constexpr long long kBlocks = 152;
  const int per = 2048 / (2 * head_dim);  // heads of a unit
  const long long units = rows * ((hq + per - 1) / per + (hkv + per - 1) / per);
  // A unit's work: its rounds over its rows (norm_rope_bwd_kernel's SUB * UN rows each) and about one more of copies
  // and waits. Divided by heads alone, few kv heads starve: 32 + 1 heads of 128, 3000 tokens, 58 us against 20.
  const int round = head_dim == 128 ? 4 : 1;
  auto work = [&](int heads) {
    const long long rest = heads % per;
    return heads / per * (1LL + (per + round - 1) / round) + (rest ? 1 + (rest + round - 1) / round : 0);
  };
  const long long wq = work(hq), all = wq + work(hkv);
  NormRopeBwdPlan pl;
  pl.blocks = (int)std::max<long long>(1, std::min<long long>(kBlocks, (units + kBwdWarps - 1) / kBwdWarps));
  const long long warps = (long long)pl.blocks * kBwdWarps;
  pl.warps_q = (int)std::max<long long>(1, std::min(warps - 1, (warps * wq + all / 2) / all));
  return pl;
}

int launch_norm_rope(NormRopeParams p, int head_dim, bool bf16, bool append, cudaStream_t s) {
#define NR(DD) return bf16 ? launch_t<true, DD>(p, append, s) : launch_t<false, DD>(p, append, s)
  if (head_dim == 128) NR(128);
  if (head_dim == 192) NR(192);
  if (head_dim == 256) NR(256);
  if (head_dim == 512) NR(512);
#undef NR
  return SDPA_ERR_UNSUPPORTED;
}

int launch_norm_rope_bwd(const NormRopeBwdParams& p, int head_dim, bool bf16, int* launches, cudaStream_t s) {
  *launches = 2;
#define NR(DD) return bf16 ? launch_bwd_t<true, DD>(p, s) : launch_bwd_t<false, DD>(p, s)
  if (head_dim == 128) NR(128);
  if (head_dim == 192) NR(192);
  if (head_dim == 256) NR(256);
  if (head_dim == 512) NR(512);
#undef NR
  return SDPA_ERR_UNSUPPORTED;
}

}  // namespace sdpa
