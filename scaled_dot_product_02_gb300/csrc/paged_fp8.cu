// paged_fp8.cu -- attention of new tokens over a paged cache in 8 bits: E4M3 codes
// with a power of two a row (fp8_row.cuh).
//   S_ij = scale q_i . k_j 2^ek_j,  O_i = sum_j softmax(S)_ij v_j 2^ev_j
//
// The plainest form: a CTA takes one query row of one head, each of its warps
// every fourth key with a running maximum and sum, and the warps' results are
// put together at the end.
#include <cuda_runtime.h>

#include "fp8_row.cuh"
#include "paged.cuh"

namespace sdpa {

namespace {

template <int D, int DV, bool BF16>
__global__ void __launch_bounds__(128) paged_fp8_kernel(const __grid_constant__ PagedFp8Params f) {
  using E = Elem<BF16>;
  using T = typename E::T;
  const PagedParams& p = f.a;
  __shared__ PagedScan scan;
  __shared__ float s_m[4], s_l[4], s_o[4][DV];
  const PagedShares all = paged_scan<128, false>(p, &scan);
  if (!all.fit) {
    if (blockIdx.x == 0 && threadIdx.x == 0) record_error(p.err, SDPA_ERR_BAD_SEQLENS);
    return;
  }
  const int row = blockIdx.x / p.hq, head = blockIdx.x % p.hq, kvh = head / p.group;
  int b = 0;
  PagedSeq seq = paged_seq(p, 0);
  while (row >= seq.row0 + seq.q_len) {
    if (++b >= p.batch) return;
    seq = paged_seq(p, b);
  }
  const int i = row - seq.row0, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const PagedSpan span = paged_span(p, seq, i, i);
  float q[D / 32], o[DV / 32], m = -INFINITY, l = 0.f;
  const T* qr = static_cast<const T*>(f.q) + row * f.q_stride + head * D + lane * (D / 32);
  for (int x = 0; x < D / 32; ++x) q[x] = SDPA_ADDR_OK(p.chk, qr + x, 2) ? (float)qr[x] : 0.f;
  for (int x = 0; x < DV / 32; ++x) o[x] = 0.f;
  for (int key = span.lo + warp; key < span.hi; key += 4) {
    const int col = key / p.page_size, slot = key - col * p.page_size;
    const int32_t* id = p.block_table + b * p.table_stride + col;
    const int page = SDPA_ADDR_OK(p.chk, id, 4) ? __ldg(id) : -1;
    const bool in = page >= 0 && page < p.num_pages;
    if (!in) record_error(p.err, SDPA_ERR_BAD_INDEX);
    const uint8_t* kr = f.k_cache + page * f.k_page + slot * f.k_slot + kvh * f.k_head + lane * (D / 32);
    const uint8_t* vr = f.v_cache + page * f.v_page + slot * f.v_slot + kvh * f.v_head + lane * (DV / 32);
    const uint8_t* ks = f.k_scale + page * f.ks_page + slot * f.ks_slot + kvh * f.ks_head;
    const uint8_t* vs = f.v_scale + page * f.vs_page + slot * f.vs_slot + kvh * f.vs_head;
    const bool ok = in && SDPA_ADDR_OK(p.chk, kr, D / 32) && SDPA_ADDR_OK(p.chk, vr, DV / 32) &&
                    SDPA_ADDR_OK(p.chk, ks, 1) && SDPA_ADDR_OK(p.chk, vs, 1);
    auto value = [](uint8_t code) { return Elem<false>::unpack(unpack_e4m3x2(code)).x; };
    float s = 0.f;
    for (int x = 0; x < D / 32; ++x) s += q[x] * (ok ? value(kr[x]) : 0.f);
    for (int x = 16; x > 0; x /= 2) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= p.scale_log2 * (ok ? exp2_byte(*ks) : 0.f);
    const float top = fmaxf(m, s), g = m == -INFINITY ? 0.f : ex2(m - top), e = ex2(s - top);
    m = top;
    l = l * g + e;
    const float w = e * (ok ? exp2_byte(*vs) : 0.f);
    for (int x = 0; x < DV / 32; ++x) o[x] = o[x] * g + w * (ok ? value(vr[x]) : 0.f);
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
  for (int x = 0; x < DV / 32; ++x) s_o[warp][lane * (DV / 32) + x] = o[x];
  __syncthreads();
  const float top = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
  float g[4], sum = 0.f;
  for (int w = 0; w < 4; ++w) {
    g[w] = s_m[w] == -INFINITY ? 0.f : ex2(s_m[w] - top);
    sum += g[w] * s_l[w];
  }
  for (int x = threadIdx.x; x < DV; x += 128) {
    const float v = g[0] * s_o[0][x] + g[1] * s_o[1][x] + g[2] * s_o[2][x] + g[3] * s_o[3][x];
    T* to = static_cast<T*>(p.o) + ((long long)row * p.hq + head) * DV + x;
    if (SDPA_ADDR_OK(p.chk, to, 2)) *to = (T)(sum == 0.f ? 0.f : v / sum);
  }
  float* to = p.lse + (long long)row * p.hq + head;
  if (threadIdx.x == 0 && SDPA_ADDR_OK(p.chk, to, 4)) *to = sum == 0.f ? -INFINITY : top * kLn2 + logf(sum);
}

}  // namespace

int launch_paged_fp8(const PagedFp8Launch& L, int, int head_dim, bool bf16, int* launches) {
  auto kern = head_dim == 128   ? (bf16 ? paged_fp8_kernel<128, 128, true> : paged_fp8_kernel<128, 128, false>)
              : head_dim == 192 ? (bf16 ? paged_fp8_kernel<192, 128, true> : paged_fp8_kernel<192, 128, false>)
              : head_dim == 256 ? (bf16 ? paged_fp8_kernel<256, 256, true> : paged_fp8_kernel<256, 256, false>)
                                : (bf16 ? paged_fp8_kernel<512, 512, true> : paged_fp8_kernel<512, 512, false>);
  const long long grid = (long long)L.p.a.total_q * L.p.a.hq;
  if (grid > 0x7fffffffLL) return SDPA_ERR_UNSUPPORTED;
  kern<<<(unsigned)grid, 128, 0, L.stream>>>(L.p);
  if (cudaGetLastError() != cudaSuccess) return SDPA_ERR_CUDA;
  ++*launches;
  return SDPA_OK;
}

}  // namespace sdpa
