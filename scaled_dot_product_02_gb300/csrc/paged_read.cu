// paged_read.cu -- the last keys and values of every sequence of an 8-bit paged
// cache as packed 16-bit rows: y = code 2^e (fp8_row.cuh), rounded once (not at
// all when the type is the one the row was quantised from).
//
// Bound by memory: a byte read and two written a value. A warp takes 1, 4
// or 8 tokens, all heads: their places in the cache are found by a lane each (a
// binary search among the sequences' ends), then all lanes walk the tokens'
// values, eight a lane and step, with several steps' loads in flight.
//
// Measured (twelve passes in a captured graph): 73536 tokens of 8 heads of 128 74.5 us,
// 6.1 TB/s; 6669 of 8 heads of 256 23.4 us, 3.5 TB/s (a chain of search, table, codes and
// stores once).
#include <algorithm>
#include <cuda_runtime.h>

#include "common.cuh"
#include "fp8_row.cuh"
#include "kernels.h"

namespace sdpa {

namespace {

constexpr int kThreads = 128;
constexpr int kSteps = 8;   // loads a lane has in flight
// A warp takes one token, or four from kFew rows on where a token's vectors are one round of its loads or less. Captured
// us with one / four: 8 kv heads of 128 (256 vectors), 1000 rows 4.1 / 7.7, 10000 14.6 / 15.4, 39000 43.9 / 44.4, 60000 64.9
// / 63.5; 2 of 512 (256), 39000 43.8 / 44.2, 60000 64.5 / 63.4; of more vectors one is quicker throughout: 16 of 128 or 8 of
// 256 (512), 20000 41.6 / 50.5, 60000 112 / 122; 8 of 512 (1024), 20000 80 / 93, 39000 146 / 164. (The K or the V of one
// token a warp: 8 of 128, 16000 rows 31.2 against 23.5.)
constexpr int kFew = 40000;
// A token of up to kNarrow 16-byte vectors leaves lanes and steps idle: from kFewNarrow tokens a vector up a warp's lanes walk
// kFlat tokens at once (heads of 128; us so / as above, both a pass a graph, 2 to 3 us more): 1 kv head, 2000 rows 6.3 / 6.3,
// 16000 8.3 / 15.8, 64000 18.5 / 41.1; 2 heads, 16000 rows 10.9 / 16.5; 4 heads, 8000 rows 14.4 / 11.2, 16000 18.6 / 18.5, 64000
// 42.3 / 48.3; 6 heads, 16000 rows 25.6 / 20.7, 64000 61.4 / 56.9.
constexpr int kNarrow = 128, kFewNarrow = 100, kFlat = 8;

struct Place {
  long long k_at, v_at;    // head 0's codes
  long long ks_at, vs_at;  // and scale bytes
  bool live;
};

__device__ __forceinline__ Place place_of(const PagedReadParams& p, long long row) {
  Place x;
  x.live = false;
  x.k_at = x.v_at = x.ks_at = x.vs_at = 0;
  // the first sequence that ends behind the row
  int lo = 0, hi = p.batch;
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    const int32_t* end = p.cu + mid + 1;
    if ((SDPA_ADDR_OK(p.chk, end, 4) ? __ldg(end) : 0) <= row)
      lo = mid + 1;
    else
      hi = mid;
  }
  if (lo >= p.batch) return x;  // behind the last sequence
  const bool in = SDPA_ADDR_OK(p.chk, p.cu + lo, 8) && SDPA_ADDR_OK(p.chk, p.kv_lens + lo, 4);
  const int first = in ? __ldg(p.cu + lo) : 0, end = in ? __ldg(p.cu + lo + 1) : 0;
  const long long pos = (long long)(in ? __ldg(p.kv_lens + lo) : 0) - (end - row);
  const long long col = pos / p.page_size;
  if (first > row || end <= row || end > p.rows || pos < 0 || col >= p.max_pages) {
    record_error(p.err, SDPA_ERR_BAD_SEQLENS);
    return x;
  }
  const int32_t* id = p.block_table + lo * p.table_stride + col;
  const int page = SDPA_ADDR_OK(p.chk, id, 4) ? __ldg(id) : -1;
  if (page < 0 || page >= p.num_pages) {
    record_error(p.err, SDPA_ERR_BAD_INDEX);
    return x;
  }
  const long long slot = pos - col * p.page_size;
  x.live = true;
  x.k_at = page * p.k_page + slot * p.k_slot;
  x.v_at = page * p.v_page + slot * p.v_slot;
  x.ks_at = page * p.ks_page + slot * p.ks_slot;
  x.vs_at = page * p.vs_page + slot * p.vs_slot;
  return x;
}

__device__ __forceinline__ long long from_lane(long long x, int lane) { return __shfl_sync(0xffffffffu, x, lane); }

// Eight codes as 16-bit values, written.
template <bool BF16>
__device__ __forceinline__ void write_vec(const PagedReadParams& p, uint16_t* to, uint2 c, int e) {
  const float s = exp2_byte(e);
  uint32_t y[4];
#pragma unroll
  for (int z = 0; z < 4; ++z) {
    const float2 f = Elem<false>::unpack(unpack_e4m3x2((uint16_t)((z < 2 ? c.x : c.y) >> (16 * (z & 1)))));
    y[z] = Elem<BF16>::pack(f.x * s, f.y * s);
  }
  if (SDPA_ADDR_OK(p.chk, to, 16)) *reinterpret_cast<uint4*>(to) = make_uint4(y[0], y[1], y[2], y[3]);
}

// TOKENS: of a warp. FLAT: the lanes walk all of them at once, else one after the other.
template <bool BF16, int D, int DV, int TOKENS, bool FLAT>
__global__ void __launch_bounds__(kThreads) paged_read_kernel(const __grid_constant__ PagedReadParams p) {
  const int lane = threadIdx.x % 32;
  const long long row0 = ((long long)blockIdx.x * (kThreads / 32) + threadIdx.x / 32) * TOKENS;
  if (row0 >= p.rows) return;
  Place mine;
  mine.live = false;
  mine.k_at = mine.v_at = mine.ks_at = mine.vs_at = 0;
  if (lane < TOKENS && row0 + lane < p.rows) mine = place_of(p, row0 + lane);
  const uint32_t live = __ballot_sync(0xffffffffu, mine.live);
  const int vecs_k = p.hkv * (D / 8), vecs = vecs_k + p.hkv * (DV / 8);  // of a token: K's, then V's
  auto load = [&](const uint8_t* k, const uint8_t* v, const uint8_t* ks, const uint8_t* vs, int i, bool here, uint2& c, int& e) {
    const bool is_v = i >= vecs_k;
    const int w = is_v ? DV / 8 : D / 8, j = is_v ? i - vecs_k : i, h = j / w;
    const uint8_t* from = (is_v ? v + h * p.v_head : k + h * p.k_head) + (j - h * w) * 8;
    const uint8_t* se = is_v ? vs + h * p.vs_head : ks + h * p.ks_head;
    const bool in = here && SDPA_ADDR_OK(p.chk, from, 8) && SDPA_ADDR_OK(p.chk, se, 1);
    c = in ? __ldg(reinterpret_cast<const uint2*>(from)) : make_uint2(0u, 0u);
    e = in ? __ldg(se) : 127;
  };
  uint16_t* ko = static_cast<uint16_t*>(p.k_out) + row0 * p.k_row;
  uint16_t* vo = static_cast<uint16_t*>(p.v_out) + row0 * p.v_row;
  if constexpr (FLAT) {
#pragma unroll 1
    for (int i0 = 0; i0 < vecs * TOKENS; i0 += 32 * kSteps) {
      uint2 c[kSteps];
      int e[kSteps];
#pragma unroll
      for (int x = 0; x < kSteps; ++x) {
        const int n = i0 + x * 32 + lane, t = min(n / vecs, TOKENS - 1);
        load(p.k_cache + from_lane(mine.k_at, t), p.v_cache + from_lane(mine.v_at, t), p.k_scale + from_lane(mine.ks_at, t),
             p.v_scale + from_lane(mine.vs_at, t), n - t * vecs, n < vecs * TOKENS && (live >> t & 1), c[x], e[x]);
      }
#pragma unroll
      for (int x = 0; x < kSteps; ++x) {
        const int n = i0 + x * 32 + lane, t = n / vecs, i = n - t * vecs;
        if (t >= TOKENS || !(live >> t & 1)) continue;
        write_vec<BF16>(p, i >= vecs_k ? vo + t * p.v_row + (i - vecs_k) * 8 : ko + t * p.k_row + i * 8, c[x], e[x]);
      }
    }
  } else {
#pragma unroll 1
    for (int t = 0; t < TOKENS; ++t, ko += p.k_row, vo += p.v_row) {
      if (!(live >> t & 1)) continue;
      const uint8_t *k = p.k_cache + from_lane(mine.k_at, t), *v = p.v_cache + from_lane(mine.v_at, t);
      const uint8_t *ks = p.k_scale + from_lane(mine.ks_at, t), *vs = p.v_scale + from_lane(mine.vs_at, t);
#pragma unroll 1
      for (int i0 = lane; i0 < vecs; i0 += 32 * kSteps) {
        uint2 c[kSteps];
        int e[kSteps];
#pragma unroll
        for (int x = 0; x < kSteps; ++x) load(k, v, ks, vs, i0 + x * 32, i0 + x * 32 < vecs, c[x], e[x]);
#pragma unroll
        for (int x = 0; x < kSteps; ++x) {
          const int i = i0 + x * 32;
          if (i >= vecs) break;
          write_vec<BF16>(p, i >= vecs_k ? vo + (i - vecs_k) * 8 : ko + i * 8, c[x], e[x]);
        }
      }
    }
  }
}

template <bool BF16, int D, int DV>
int launch_t(const PagedReadParams& p, cudaStream_t s) {
  const int vecs = p.hkv * (D + DV) / 8;
  const bool flat = vecs <= kNarrow && p.rows > kFewNarrow * (long long)vecs;
  const int tokens = flat ? kFlat : vecs > 32 * kSteps || p.rows <= kFew ? 1 : 4;
  const int per = kThreads / 32 * tokens;  // rows of a block
  const unsigned grid = (unsigned)((p.rows + per - 1) / per);
  auto kern = flat          ? paged_read_kernel<BF16, D, DV, kFlat, true>
              : tokens == 1 ? paged_read_kernel<BF16, D, DV, 1, false>
                            : paged_read_kernel<BF16, D, DV, 4, false>;
  kern<<<grid, kThreads, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? SDPA_OK : SDPA_ERR_CUDA;
}

}  // namespace

int launch_paged_read(const PagedReadParams& p, int head_dim, bool bf16, cudaStream_t s) {
#define READ(A, B) return bf16 ? launch_t<true, A, B>(p, s) : launch_t<false, A, B>(p, s)
  if (head_dim == 128) READ(128, 128);
  if (head_dim == 192) READ(192, 128);
  if (head_dim == 256) READ(256, 256);
  if (head_dim == 512) READ(512, 512);
#undef READ
  return SDPA_ERR_UNSUPPORTED;
}

}  // namespace sdpa
