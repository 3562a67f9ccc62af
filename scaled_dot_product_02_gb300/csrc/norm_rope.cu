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
// butterfly over LPH lanes. A warp walks the heads of its share of a token
// with UNROLL rows per lane in flight, and keeps the token's cosines and sines
// and the weights in registers. A pair (i, i + rot/2) lies in two vectors: the
// partner's vector is loaded a second time (an L1 hit, issued with the first
// load), which serves every rot with one code path and no exchange of lanes.
#include <algorithm>
#include <cuda_runtime.h>

#include "common.cuh"
#include "kernels.h"

namespace sdpa {

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

template <int D>
struct Row {
  static constexpr int VECS = D / 8;  // 16-byte vectors of a row
  static constexpr int LPH = D == 128 ? 16 : (D == 192 ? 8 : 32);
  static constexpr int VPL = VECS / LPH;
  static constexpr int SUB = 32 / LPH;
  static constexpr int UNROLL = 4 / VPL > 1 ? 4 / VPL : 1;
  static constexpr int DV = D == 192 ? 128 : D;  // width of a value row
  static constexpr int VPL_V = DV / 8 / LPH;
  static_assert(VPL * LPH == VECS && VPL_V * LPH == DV / 8, "rows are whole vectors of their lanes");
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
__device__ __forceinline__ void unpack8(const uint4& x, float (&f)[8]) {
  const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 t = E::unpack(u[e]);
    f[2 * e] = t.x;
    f[2 * e + 1] = t.y;
  }
}
template <class E>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(E::pack(f[0], f[1]), E::pack(f[2], f[3]), E::pack(f[4], f[5]), E::pack(f[6], f[7]));
}

template <int LPH>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LPH / 2; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A lane's share of one token's rotation: for each of its vectors whether it
// turns, the vector its pairs' other halves lie in (itself for adjacent pairs),
// and the eight cosines and sines; the sine carries the sign of the half.
template <int VPL>
struct Turn {
  bool on[VPL];
  int partner[VPL];
  float c[VPL][8], s[VPL][8];
};

template <int D>
__device__ __forceinline__ void load_turn(Turn<Row<D>::VPL>& t, const float* row, int rot, bool interleaved, int sub,
                                          AddrTable* chk) {
  using R = Row<D>;
  const int half = rot / 2;
#pragma unroll
  for (int v = 0; v < R::VPL; ++v) {
    const int idx = v * R::LPH + sub;
    t.on[v] = idx * 8 < rot;
    t.partner[v] = idx;
    if (!t.on[v]) continue;
    if (interleaved) {
      const uint4 c = load16(chk, row + idx * 4), s = load16(chk, row + half + idx * 4);
      const uint32_t cu[4] = {c.x, c.y, c.z, c.w}, su[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        t.c[v][2 * e] = t.c[v][2 * e + 1] = __uint_as_float(cu[e]);
        t.s[v][2 * e] = -__uint_as_float(su[e]);
        t.s[v][2 * e + 1] = __uint_as_float(su[e]);
      }
    } else {
      const bool second = idx * 8 >= half;  // half is a multiple of 8: a vector lies in one half
      t.partner[v] = second ? idx - half / 8 : idx + half / 8;
      const int i0 = idx * 8 - (second ? half : 0);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint4 c = load16(chk, row + i0 + q * 4), s = load16(chk, row + half + i0 + q * 4);
        const uint32_t cu[4] = {c.x, c.y, c.z, c.w}, su[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          t.c[v][q * 4 + e] = __uint_as_float(cu[e]);
          t.s[v][q * 4 + e] = second ? __uint_as_float(su[e]) : -__uint_as_float(su[e]);
        }
      }
    }
  }
}

// One vector turned: y the values, z their partners' values (the other halves'
// vector, or for adjacent pairs y itself with neighbours exchanged).
// sign = -1 turns back.
__device__ __forceinline__ void turn8(float (&y)[8], const float (&z)[8], const float (&c)[8], const float (&s)[8],
                                      bool interleaved, float sign) {
  float o[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float other = interleaved ? y[e ^ 1] : z[e];
    o[e] = fmaf(other, sign * s[e], y[e] * c[e]);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = o[e];
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

// Heads of a token in order: q, k and (append) v; p.parts warps share a token.
template <bool BF16, int D, bool APPEND, bool NORM>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  using E = Elem<BF16>;
  using T = typename E::T;
  using R = Row<D>;
  const int lane = threadIdx.x % 32, sub = lane % R::LPH, grp = lane / R::LPH;
  const long long w = (long long)blockIdx.x * kWarps + threadIdx.x / 32;
  const long long row = w / p.parts;
  if (row >= p.rows) return;
  const int part = (int)(w - row * p.parts);
  const int heads = p.hq + (APPEND ? 2 : 1) * p.hkv;
  const int per = (heads + p.parts - 1) / p.parts;
  const int h_end = min(heads, (part + 1) * per);

  Slot slot;
  if (APPEND) {
    slot = find_slot(p, row, lane);
    if (!slot.live) return;
  }
  Turn<R::VPL> turn;
  const bool inter = p.interleaved != 0;
  uint4 wq[R::VPL], wk[R::VPL], wqp[R::VPL], wkp[R::VPL];
  if (NORM) {
    if (p.rot > 0) {
      const int pos = APPEND && !p.pos ? slot.position : load_i32(p.chk, p.pos + row, -1);
      if (pos < 0 || pos >= p.max_pos) {
        if (lane == 0) record_error(p.err, SDPA_ERR_BAD_INDEX);
        return;
      }
      load_turn<D>(turn, p.table + (long long)pos * p.rot, p.rot, inter, sub, p.chk);
    } else {
#pragma unroll
      for (int v = 0; v < R::VPL; ++v) {
        turn.on[v] = false;
        turn.partner[v] = v * R::LPH + sub;
      }
    }
#pragma unroll
    for (int v = 0; v < R::VPL; ++v) {
      const int own = (v * R::LPH + sub) * 8, other = turn.partner[v] * 8;
      wk[v] = load16(p.chk, static_cast<const T*>(p.wk) + own);
      wkp[v] = load16(p.chk, static_cast<const T*>(p.wk) + other);
      if (p.hq > 0) {
        wq[v] = load16(p.chk, static_cast<const T*>(p.wq) + own);
        wqp[v] = load16(p.chk, static_cast<const T*>(p.wq) + other);
      }
    }
  }

  for (int h0 = part * per + grp; __any_sync(0xffffffffu, h0 < h_end); h0 += R::SUB * R::UNROLL) {
    uint4 x[R::UNROLL][R::VPL], z[R::UNROLL][R::VPL];
#pragma unroll
    for (int u = 0; u < R::UNROLL; ++u) {
      const int h = h0 + u * R::SUB;
      const bool is_v = APPEND && h >= p.hq + p.hkv;
      const T* src = h < p.hq ? static_cast<const T*>(p.q) + row * p.qs + (long long)h * D
                     : !is_v  ? static_cast<const T*>(p.k) + row * p.ks + (long long)(h - p.hq) * D
                              : static_cast<const T*>(p.v) + row * p.vs + (long long)(h - p.hq - p.hkv) * R::DV;
#pragma unroll
      for (int v = 0; v < R::VPL; ++v) {
        const bool in = h < h_end && (!is_v || v < R::VPL_V);
        x[u][v] = z[u][v] = make_uint4(0u, 0u, 0u, 0u);
        if (in) x[u][v] = load16(p.chk, src + (v * R::LPH + sub) * 8);
        if (NORM && !inter && in && !is_v && turn.on[v]) z[u][v] = load16(p.chk, src + turn.partner[v] * 8);
      }
    }
#pragma unroll
    for (int u = 0; u < R::UNROLL; ++u) {
      const int h = h0 + u * R::SUB;
      const bool is_q = h < p.hq, is_v = APPEND && h >= p.hq + p.hkv;
      if (NORM) {
        float ss = 0.f;
#pragma unroll
        for (int v = 0; v < R::VPL; ++v) {
          float f[8];
          unpack8<E>(x[u][v], f);
#pragma unroll
          for (int e = 0; e < 8; ++e) ss = fmaf(f[e], f[e], ss);
        }
        const float r = rsqrtf(row_sum<R::LPH>(ss) * (1.f / D) + p.eps);
        if (!is_v) {
#pragma unroll
          for (int v = 0; v < R::VPL; ++v) {
            float f[8], wt[8];
            unpack8<E>(x[u][v], f);
            unpack8<E>(is_q ? wq[v] : wk[v], wt);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = f[e] * r * wt[e];
            if (turn.on[v]) {
              float g[8];
              unpack8<E>(z[u][v], g);
              unpack8<E>(is_q ? wqp[v] : wkp[v], wt);
#pragma unroll
              for (int e = 0; e < 8; ++e) g[e] = g[e] * r * wt[e];
              turn8(f, g, turn.c[v], turn.s[v], inter, 1.f);
            }
            x[u][v] = pack8<E>(f);
          }
        }
      }
      if (h >= h_end) continue;
      T* dst;
      if (is_q)
        dst = static_cast<T*>(p.q_out) + (row * p.hq + h) * D;
      else if (!APPEND)
        dst = static_cast<T*>(p.k_out) + (row * p.hkv + (h - p.hq)) * D;
      else if (!is_v)
        dst = static_cast<T*>(p.kc) + slot.k_at + (h - p.hq) * p.kc_head;
      else
        dst = static_cast<T*>(p.vc) + slot.v_at + (h - p.hq - p.hkv) * p.vc_head;
#pragma unroll
      for (int v = 0; v < R::VPL; ++v)
        if (!is_v || v < R::VPL_V) store16(p.chk, dst + (v * R::LPH + sub) * 8, x[u][v]);
    }
  }
}

// Gradient. Each block walks (token, share of its heads) in strides of the
// grid, keeps the sums of dw in registers (one set for q, one for k), and
// writes one partial sum per block; dw_kernel adds the blocks' in order.
template <bool BF16, int D>
__global__ void __launch_bounds__(kThreads) norm_rope_bwd_kernel(const __grid_constant__ NormRopeBwdParams p) {
  using E = Elem<BF16>;
  using T = typename E::T;
  using R = Row<D>;
  constexpr int UN = R::VPL == 1 ? 2 : 1;
  const int lane = threadIdx.x % 32, sub = lane % R::LPH, grp = lane / R::LPH, warp = threadIdx.x / 32;
  const int heads = p.hq + p.hkv, per = (heads + p.parts - 1) / p.parts;
  const long long units = p.rows * p.parts;
  const bool inter = p.interleaved != 0;
  uint4 wq[R::VPL], wk[R::VPL];
  float aq[R::VPL][8], ak[R::VPL][8];
#pragma unroll
  for (int v = 0; v < R::VPL; ++v) {
    wq[v] = load16(p.chk, static_cast<const T*>(p.wq) + (v * R::LPH + sub) * 8);
    wk[v] = load16(p.chk, static_cast<const T*>(p.wk) + (v * R::LPH + sub) * 8);
#pragma unroll
    for (int e = 0; e < 8; ++e) aq[v][e] = ak[v][e] = 0.f;
  }
  for (long long w = (long long)blockIdx.x * kWarps + warp; w < units; w += (long long)gridDim.x * kWarps) {
    const long long row = w / p.parts;
    const int part = (int)(w - row * p.parts), h_end = min(heads, (part + 1) * per);
    Turn<R::VPL> turn;
    bool skip = false;  // a position outside the table: zeros
    if (p.rot > 0) {
      const int pos = load_i32(p.chk, p.pos + row, -1);
      skip = pos < 0 || pos >= p.max_pos;
      if (skip && lane == 0) record_error(p.err, SDPA_ERR_BAD_INDEX);
      load_turn<D>(turn, p.table + (skip ? 0ll : (long long)pos * p.rot), p.rot, inter, sub, p.chk);
    } else {
#pragma unroll
      for (int v = 0; v < R::VPL; ++v) {
        turn.on[v] = false;
        turn.partner[v] = v * R::LPH + sub;
      }
    }
    for (int h0 = part * per + grp; __any_sync(0xffffffffu, h0 < h_end); h0 += R::SUB * UN) {
      uint4 x[UN][R::VPL], y[UN][R::VPL], z[UN][R::VPL];
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        const int h = h0 + u * R::SUB;
        const bool is_q = h < p.hq;
        const T* xs = is_q ? static_cast<const T*>(p.q) + row * p.qs + (long long)h * D
                           : static_cast<const T*>(p.k) + row * p.ks + (long long)(h - p.hq) * D;
        const T* gs = is_q ? static_cast<const T*>(p.gq) + (row * p.hq + h) * D
                           : static_cast<const T*>(p.gk) + (row * p.hkv + (h - p.hq)) * D;
        const bool in = h < h_end && !skip;
#pragma unroll
        for (int v = 0; v < R::VPL; ++v) {
          x[u][v] = y[u][v] = z[u][v] = make_uint4(0u, 0u, 0u, 0u);
          if (in) x[u][v] = load16(p.chk, xs + (v * R::LPH + sub) * 8);
          if (in) y[u][v] = load16(p.chk, gs + (v * R::LPH + sub) * 8);
          if (in && !inter && turn.on[v]) z[u][v] = load16(p.chk, gs + turn.partner[v] * 8);
        }
      }
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        const int h = h0 + u * R::SUB;
        const bool is_q = h < p.hq;
        float ss = 0.f, dot = 0.f;
        float g[R::VPL][8];
#pragma unroll
        for (int v = 0; v < R::VPL; ++v) {
          float f[8], o[8], wt[8];
          unpack8<E>(x[u][v], f);
          unpack8<E>(y[u][v], g[v]);
          if (turn.on[v]) {
            unpack8<E>(z[u][v], o);
            turn8(g[v], o, turn.c[v], turn.s[v], inter, -1.f);
          }
          unpack8<E>(is_q ? wq[v] : wk[v], wt);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            ss = fmaf(f[e], f[e], ss);
            dot = fmaf(g[v][e] * wt[e], f[e], dot);
          }
        }
#pragma unroll
        for (int o = R::LPH / 2; o > 0; o /= 2) {
          ss += __shfl_xor_sync(0xffffffffu, ss, o);
          dot += __shfl_xor_sync(0xffffffffu, dot, o);
        }
        if (h >= h_end) continue;
        const float r = skip ? 0.f : rsqrtf(ss * (1.f / D) + p.eps), k3 = r * r * r * (dot * (1.f / D));
        T* dst = is_q ? static_cast<T*>(p.dq) + row * p.dqs + (long long)h * D
                      : static_cast<T*>(p.dk) + row * p.dks + (long long)(h - p.hq) * D;
#pragma unroll
        for (int v = 0; v < R::VPL; ++v) {
          float f[8], wt[8];
          unpack8<E>(x[u][v], f);
          unpack8<E>(is_q ? wq[v] : wk[v], wt);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float t = g[v][e] * f[e] * r;
            aq[v][e] += is_q ? t : 0.f;
            ak[v][e] += is_q ? 0.f : t;
            f[e] = fmaf(-k3, f[e], r * g[v][e] * wt[e]);
          }
          store16(p.chk, dst + (v * R::LPH + sub) * 8, pack8<E>(f));
        }
      }
    }
  }
  // the block's sum of dw: row groups of a warp by shuffles, warps in order
  __shared__ float sum[kWarps][2][D];
#pragma unroll
  for (int v = 0; v < R::VPL; ++v)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
#pragma unroll
      for (int o = R::LPH; o < 32; o *= 2) {
        aq[v][e] += __shfl_xor_sync(0xffffffffu, aq[v][e], o);
        ak[v][e] += __shfl_xor_sync(0xffffffffu, ak[v][e], o);
      }
      if (grp == 0) {
        sum[warp][0][(v * R::LPH + sub) * 8 + e] = aq[v][e];
        sum[warp][1][(v * R::LPH + sub) * 8 + e] = ak[v][e];
      }
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) t += sum[k][i / D][i % D];
    float* at = p.part + (long long)blockIdx.x * 2 * D + i;
    if (SDPA_ADDR_OK(p.chk, at, 4)) *at = t;
  }
}

// dw = the blocks' partial sums, added in a fixed order: 32 columns per CTA,
// eight threads a column, each over every eighth block.
__global__ void __launch_bounds__(256) dw_kernel(const float* part, int blocks, int d, float* dwq, float* dwk,
                                                 AddrTable* chk) {
  __shared__ float sum[8][32];
  const int col = blockIdx.x * 32 + threadIdx.x % 32, k = threadIdx.x / 32;
  float t = 0.f;
#pragma unroll 8
  for (int b = k; b < blocks; b += 8) {
    const float* at = part + (long long)b * 2 * d + col;
    t += SDPA_ADDR_OK(chk, at, 4) ? *at : 0.f;
  }
  sum[k][threadIdx.x % 32] = t;
  __syncthreads();
  if (k == 0) {
#pragma unroll
    for (int i = 1; i < 8; ++i) t += sum[i][threadIdx.x % 32];
    float* at = col < d ? dwq + col : dwk + (col - d);
    if (SDPA_ADDR_OK(chk, at, 4)) *at = t;
  }
}

// Warps that share a token's heads: one when there are tokens enough for
// `want` warps (the token's angles and the weights are then loaded once), else
// more, down to one unrolled step of heads per warp.
int share(long long rows, int heads, int step, long long want) {
  const long long most = (heads + step - 1) / step;
  return (int)std::max<long long>(1, std::min(most, (want + rows - 1) / std::max<long long>(rows, 1)));
}

int sm_count(int* sms) {
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess &&
                 cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess
             ? SDPA_OK
             : SDPA_ERR_CUDA;
}

template <bool BF16, int D>
int launch_t(NormRopeParams p, bool append, cudaStream_t s) {
  using R = Row<D>;
  int sms = 0;
  if (const int rc = sm_count(&sms)) return rc;
  const int heads = p.hq + (append ? 2 : 1) * p.hkv;
  p.parts = share(p.rows, heads, R::SUB * R::UNROLL, (long long)sms * 32);
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
int launch_bwd_t(const NormRopeBwdParams& p, cudaStream_t s) {
  norm_rope_bwd_kernel<BF16, D><<<(unsigned)p.blocks, kThreads, 0, s>>>(p);
  if (cudaGetLastError() != cudaSuccess) return SDPA_ERR_CUDA;
  dw_kernel<<<2 * D / 32, 256, 0, s>>>(p.part, p.blocks, D, p.dwq, p.dwk, p.chk);
  return cudaGetLastError() == cudaSuccess ? SDPA_OK : SDPA_ERR_CUDA;
}

}  // namespace

int norm_rope_bwd_blocks(long long rows, int hq, int hkv, int head_dim, int* parts) {
  // written for 152 SMs: the count must not depend on the device in use, since
  // the workspace size is asked for without one
  constexpr long long kBlocks = 152 * 6;
  const int step = head_dim == 128 ? 4 : head_dim == 192 ? 4 : 1;
  *parts = share(rows, hq + hkv, step, kBlocks * kWarps);
  return (int)std::max<long long>(1, std::min<long long>(kBlocks, (rows * *parts + kWarps - 1) / kWarps));
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
