// api.cu -- the C ABI declared in include/sdpa.h: host-side validation,
// TMA descriptor encoding, workspace carving and kernel launches. No call
// here allocates device memory or synchronises, except
// sdpa_get_device_error, which is documented to synchronise.
#include <cudaTypedefs.h>
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstddef>
#include <cstdint>
#include <algorithm>
#include <array>
#include <atomic>
#include <cstring>
#include <limits>
#include <mutex>
#include <numeric>
#include <set>
#include <utility>
#include <vector>

#include "../../include/sdpa.h"
#include "kernels.h"

// The per-device error word. Kernels receive its device address.
static __device__ int g_sdpa_error_word;

namespace sdpa {
namespace {

thread_local int t_last_launches = 0;

// Event pairs recorded around launches while profiling is on (this thread).
struct Profiler {
  bool on = false;
  struct Mark {
    cudaEvent_t a, b;
    int kind;
  };
  std::vector<Mark> marks;
  size_t used = 0;
  Mark* next(int kind) {
    if (!on || used >= 65536) return nullptr;
    if (used == marks.size()) {
      Mark m{nullptr, nullptr, kind};
      if (cudaEventCreate(&m.a) != cudaSuccess || cudaEventCreate(&m.b) != cudaSuccess) return nullptr;
      marks.push_back(m);
    }
    Mark* m = &marks[used++];
    m->kind = kind;
    return m;
  }
};
thread_local Profiler t_prof;

// Launch `fn` (returning an sdpa_status) between two profiling events.
template <class F>
int timed(int kind, cudaStream_t s, F&& fn) {
  Profiler::Mark* m = t_prof.next(kind);
  if (m) cudaEventRecord(m->a, s);
  const int rc = fn();
  if (m) cudaEventRecord(m->b, s);
  return rc;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

int* error_word() { return static_cast<int*>(device_symbol_address(&g_sdpa_error_word)); }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Extent {
  uintptr_t lo, hi;
};
Extent extent(const void* p, size_t bytes) {
  return {reinterpret_cast<uintptr_t>(p), reinterpret_cast<uintptr_t>(p) + bytes};
}
bool overlaps(Extent a, Extent b) { return a.lo < b.hi && b.lo < a.hi && a.hi > a.lo && b.hi > b.lo; }

// ---- address-checked build (SDPA_ADDR_CHECK): each entry point registers the
// extents of the buffers it was given; its kernels test every computed access
// against them (addr_ok in common.cuh).
#ifdef SDPA_ADDR_CHECK
constexpr bool kAddrCheck = true;
static __device__ AddrTable g_sdpa_addr_table;
std::atomic<long long> g_addr_shrink{0};

AddrTable* addr_table() { return static_cast<AddrTable*>(device_symbol_address(&g_sdpa_addr_table)); }

// Writes the call's extents (less the debug shrink) ahead of its kernels on
// stream s; the violation counters are left as they are.
AddrTable* bind_extents(std::initializer_list<Extent> ex, int* err, cudaStream_t s) {
  AddrTable* t = addr_table();
  if (!t) return nullptr;
  AddrTable h;
  std::memset(&h, 0, sizeof(h));
  const long long shrink = g_addr_shrink.load(std::memory_order_relaxed);
  for (const Extent& e : ex) {
    if (e.hi <= e.lo || h.n >= (unsigned long long)kAddrExtents) continue;
    const uintptr_t cut = shrink > 0 ? std::min<uintptr_t>((uintptr_t)shrink, e.hi - e.lo) : 0;
    h.lo[h.n] = e.lo;
    h.hi[h.n] = e.hi - cut;
    ++h.n;
  }
  h.err = err;
  // pageable source: the call returns once the bytes are staged, in stream order
  if (cudaMemcpyAsync(t, &h, offsetof(AddrTable, violations), cudaMemcpyHostToDevice, s) != cudaSuccess)
    return nullptr;
  return t;
}
#else
constexpr bool kAddrCheck = false;
AddrTable* bind_extents(std::initializer_list<Extent>, int*, cudaStream_t) { return nullptr; }
#endif

// Rows/heads of the generic row x head x D view (see common.cuh).
void view(const sdpa_problem* p, int& rows_q, int& rows_kv, int& nh_q, int& nh_kv) {
  if (p->layout == SDPA_THD) {
    rows_q = p->total_q;
    rows_kv = p->total_kv;
    nh_q = p->num_heads_q;
    nh_kv = p->num_heads_kv;
  } else if (p->layout == SDPA_BSHD) {
    rows_q = p->batch * p->seqlen_q;
    rows_kv = p->batch * p->seqlen_kv;
    nh_q = p->num_heads_q;
    nh_kv = p->num_heads_kv;
  } else {
    rows_q = p->seqlen_q;
    rows_kv = p->seqlen_kv;
    nh_q = p->batch * p->num_heads_q;
    nh_kv = p->batch * p->num_heads_kv;
  }
}

bool causal(const sdpa_problem* p) { return p->mask_type != SDPA_MASK_NONE; }

// Width of V and O rows (head_dim_v 0 means the symmetric head_dim).
int dv_of(const sdpa_problem* p) { return p->head_dim_v ? p->head_dim_v : p->head_dim; }

// (head_dim, head_dim_v) pairs with a forward kernel: the symmetric 128, 256,
// 512, and (192, 128) (the asymmetric pair the pages' forward engine lists).
bool head_dims_supported(int d, int dv) {
  if (d == dv) return d == 128 || d == 256 || d == 512;
  return d == 192 && dv == 128;
}

int check(const sdpa_problem* p) {
  if (!p) return SDPA_ERR_INVALID_ARG;
  if (p->layout < SDPA_BSHD || p->layout > SDPA_THD) return SDPA_ERR_INVALID_ARG;
  if (p->dtype != SDPA_BF16 && p->dtype != SDPA_FP16) return SDPA_ERR_UNSUPPORTED;
  if (p->mask_type < SDPA_MASK_NONE || p->mask_type > SDPA_MASK_CAUSAL_BOTTOM_RIGHT) return SDPA_ERR_INVALID_ARG;
  if (p->batch < 0 || p->seqlen_q < 0 || p->seqlen_kv < 0) return SDPA_ERR_INVALID_ARG;
  if (p->num_heads_q <= 0 || p->num_heads_kv <= 0) return SDPA_ERR_INVALID_ARG;
  if (p->num_heads_q % p->num_heads_kv) return SDPA_ERR_INVALID_ARG;
  if (p->head_dim_v < 0) return SDPA_ERR_INVALID_ARG;
  if (!head_dims_supported(p->head_dim, dv_of(p))) return SDPA_ERR_UNSUPPORTED;
  if (p->window_left < -1 || p->window_right < -1) return SDPA_ERR_INVALID_ARG;
  if (causal(p) && p->window_right > 0) return SDPA_ERR_INVALID_ARG;
  if (!causal(p) && (p->window_left >= 0 || p->window_right >= 0) && p->seqlen_q != p->seqlen_kv)
    return SDPA_ERR_UNSUPPORTED;
  if (!std::isfinite(p->softmax_scale)) return SDPA_ERR_INVALID_ARG;
  if (p->deterministic != 0 && p->deterministic != 1) return SDPA_ERR_INVALID_ARG;
  if (p->kv_chunk < 0 || p->kv_chunk % 128) return SDPA_ERR_INVALID_ARG;
  if (p->layout == SDPA_THD) {
    if (p->total_q < 0 || p->total_kv < 0) return SDPA_ERR_INVALID_ARG;
  } else if (p->seqlen_q > 0 && p->seqlen_kv == 0 && p->batch > 0) {
    return SDPA_ERR_INVALID_ARG;  // every query would attend an empty key set
  }
  int rq, rk, hq, hk;
  view(p, rq, rk, hq, hk);
  const long long q_elems = (long long)rq * hq * p->head_dim;
  const long long k_elems = (long long)rk * hk * std::max(p->head_dim, dv_of(p));
  if (q_elems >= (1LL << 40) || k_elems >= (1LL << 40)) return SDPA_ERR_UNSUPPORTED;
  if ((long long)p->batch * p->seqlen_q >= (1LL << 31) || (long long)p->batch * p->seqlen_kv >= (1LL << 31))
    return SDPA_ERR_UNSUPPORTED;
  return SDPA_OK;
}

Geom make_geom(const sdpa_problem* p, const int32_t* cu_q, const int32_t* cu_kv) {
  Geom g;
  g.layout = p->layout;
  g.mask = p->mask_type;
  g.batch = p->batch;
  g.sq = p->seqlen_q;
  g.sk = p->seqlen_kv;
  g.hq = p->num_heads_q;
  g.hkv = p->num_heads_kv;
  g.d = p->head_dim;
  g.dv = dv_of(p);
  g.wl = p->window_left;
  g.wr = causal(p) ? 0 : p->window_right;
  g.scale = p->softmax_scale;
  g.scale_log2 = p->softmax_scale * 1.4426950408889634f;
  view(p, g.rows_q, g.rows_kv, g.nh_q, g.nh_kv);
  g.cu_q = cu_q;
  g.cu_kv = cu_kv;
  g.chk = nullptr;
  return g;
}

// 3-D map {D, heads, rows} over a contiguous [rows][heads][D] 16-bit tensor;
// boxes are 64 columns (128 bytes, 128-byte swizzle) x 1 head x box_rows.
int encode(CUtensorMap* m, const void* base, int d, int nh, int rows, int box_rows, bool bf16) {
  auto fn = encode_fn();
  if (!fn) return SDPA_ERR_CUDA;
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)nh, (cuuint64_t)(rows > 0 ? rows : 1)};
  cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)nh * d * 2};
  cuuint32_t box[3] = {64, 1, (cuuint32_t)box_rows};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                  const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? SDPA_OK : SDPA_ERR_CUDA;
}

// 3-D map over a contiguous one-byte (E4M3) tensor with 128-byte-swizzled boxes:
// dims[0] is the innermost (contiguous) extent, strides[i] the byte stride of dims[i+1].
int encode_u8(CUtensorMap* m, const void* base, const cuuint64_t (&dims)[3], const cuuint64_t (&strides)[2],
              const cuuint32_t (&box)[3]) {
  auto fn = encode_fn();
  if (!fn) return SDPA_ERR_CUDA;
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? SDPA_OK : SDPA_ERR_CUDA;
}

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Keys of the FP8 forward's transposed V per (kv head, d): every sequence's
// keys start on a multiple of 16 (see vt_row0 in fwd_fp8.cu).
size_t fp8_vt_rows(const sdpa_problem* p) {
  if (p->layout == SDPA_THD) return round_up((size_t)p->total_kv + 16 * (size_t)p->batch, 16);
  if (p->layout == SDPA_BSHD) return (size_t)p->batch * round_up((size_t)p->seqlen_kv, 16);
  return round_up((size_t)p->seqlen_kv, 16);
}

// FP8 forward: head_dim 128 or 256, equal for Q/K and V (PR #3527 "Scope"
// serves FP8 at head dims up to 256).
int check_fp8(const sdpa_problem* p) {
  const int rc = check(p);
  if (rc) return rc;
  return ((p->head_dim == 128 || p->head_dim == 256) && dv_of(p) == p->head_dim) ? SDPA_OK : SDPA_ERR_UNSUPPORTED;
}

// Key tiles one 128-row query tile can touch (the slot count of the head_dim
// 256/512 tile arrays): the whole key range, or the window's span.
int kv_slots(const sdpa_problem* p) {
  const int nkt = (p->seqlen_kv + 127) / 128;
  const int wr = causal(p) ? 0 : p->window_right;
  if (p->window_left >= 0 && wr >= 0) {
    const long long span = 128LL + p->window_left + wr;  // keys one query tile can see
    return (int)std::min<long long>(nkt, span / 128 + 2);
  }
  return nkt;
}

// Key-tile chunking of the head_dim 256/512 backward (bwd_big.cu): the P / dS
// tile arrays hold one chunk of key tiles at a time, so their size does not
// grow with the key length (TransformerEngine PR #3527, "Known limitations":
// the prior art's workspace grows to 74 GiB at 64k tokens and caps the
// context). A bounded (left, right) window already bounds the key tiles one
// query tile sees; otherwise the chunk is as many key tiles as fit the
// budget below (at least one).
constexpr size_t kBwdTileBudget = size_t(512) << 20;

struct BigPlan {
  int chunk;   // key tiles per chunk
  int slots;   // tile slots per (batch, q head, q tile)
  int chunks;  // number of chunks
};
BigPlan big_plan(const sdpa_problem* p) {
  const int nkt = (p->seqlen_kv + 127) / 128;
  const int kvs = kv_slots(p);
  const size_t tile_bytes = 2 * 32768;  // the P and dS images of one (query tile, key tile) pair
  const size_t per_slot = (size_t)p->batch * p->num_heads_q * ((p->seqlen_q + 127) / 128) * tile_bytes;
  const int wr = causal(p) ? 0 : p->window_right;
  BigPlan pl;
  if (p->kv_chunk > 0) {  // the caller's chunk
    pl.chunk = std::max(1, std::min(nkt, p->kv_chunk / 128));
    pl.slots = std::min(pl.chunk, kvs);
  } else if ((p->window_left >= 0 && wr >= 0) || (size_t)kvs * per_slot <= kBwdTileBudget || nkt <= 1) {
    pl.chunk = std::max(nkt, 1);
    pl.slots = kvs;
  } else {
    pl.chunk = (int)std::max<size_t>(1, std::min<size_t>(kBwdTileBudget / std::max<size_t>(per_slot, 1), nkt));
    pl.slots = std::min(pl.chunk, kvs);
  }
  pl.chunks = (nkt + pl.chunk - 1) / pl.chunk;
  return pl;
}

// Backward workspace carve-up. head_dim 128: per-row statistics and the fp32
// dQ accumulator. head_dim 256/512: statistics, the fp32 dQ accumulator when
// the key tiles are split into chunks, and the 16-bit P / dS tile arrays of
// one chunk.
struct BwdWs {
  size_t guard_off, order_off, lse2_off, delta_off, acc_off, ptile_off, dstile_off, total;
  int stat_rows;
  bool has_acc;
};
BwdWs bwd_ws(const sdpa_problem* p) {
  int rq, rk, hq, hk;
  view(p, rq, rk, hq, hk);
  BwdWs w;
  // rows of the per-head statistics arrays (see SeqInfo::srow0), plus 128 rows of
  // padding for query tiles that overhang the last sequence
  size_t srows;
  if (p->layout == SDPA_THD)
    srows = round_up((size_t)p->total_q + 4 * (size_t)p->batch + 3, 4);
  else if (p->layout == SDPA_BSHD)
    srows = (size_t)p->batch * round_up((size_t)p->seqlen_q, 4);
  else
    srows = round_up((size_t)p->seqlen_q, 4);
  w.stat_rows = (int)(srows + 128);
  w.guard_off = 0;
  // THD, head_dim 128: the sequence order the guard writes (longest first)
  const bool ordered = p->layout == SDPA_THD && p->head_dim == 128;
  w.order_off = ordered ? 256 : 0;
  w.lse2_off = ordered ? 256 + round_up((size_t)p->batch * 4, 256) : 256;
  w.delta_off = round_up(w.lse2_off + (size_t)hq * w.stat_rows * 4, 256);
  const size_t after_stats = round_up(w.delta_off + (size_t)hq * w.stat_rows * 4, 256);
  const size_t acc_bytes = (size_t)hq * rq * p->head_dim * 4;
  if (p->head_dim == 128) {
    // the deterministic backward writes dQ directly and needs no accumulator
    w.acc_off = after_stats;
    w.has_acc = !p->deterministic;
    w.ptile_off = w.dstile_off = 0;
    w.total = p->deterministic ? after_stats : round_up(w.acc_off + acc_bytes, 256);
  } else {
    const BigPlan pl = big_plan(p);
    const size_t tiles = (size_t)p->batch * p->num_heads_q * ((p->seqlen_q + 127) / 128) * pl.slots;
    w.has_acc = pl.chunks > 1;
    w.acc_off = after_stats;
    const size_t after_acc = w.has_acc ? w.acc_off + acc_bytes : after_stats;
    w.ptile_off = round_up(after_acc, 1024);
    w.dstile_off = w.ptile_off + tiles * 32768;
    w.total = w.dstile_off + tiles * 32768;
  }
  return w;
}

// kv heads whose key tiles interleave in the D128 backward grid: the largest
// divisor of num_heads_kv whose query-side rows (Q and dO, plus the fp32 dQ
// accumulator unless deterministic) fit in 128 MiB, about the L2. Interleaving
// heads lets the heavy first key tiles of every head start early; keeping their
// rows within the L2 keeps the CTAs that walk the same rows from re-reading
// them from HBM.
int bwd_head_block(const sdpa_problem* p) {
  const int group = p->num_heads_q / p->num_heads_kv;
  const size_t per_head = (size_t)p->seqlen_q * group * p->head_dim * (p->deterministic ? 4 : 8);
  int hb = 1;
  for (int d = 1; d <= p->num_heads_kv; ++d)
    if (p->num_heads_kv % d == 0 && (size_t)d * per_head <= (size_t)128 << 20) hb = d;
  return hb;
}

// ---- norms, rotation and the paged cache

int check_norm_rope(const sdpa_norm_rope_problem* p) {
  if (!p) return SDPA_ERR_INVALID_ARG;
  if (p->dtype != SDPA_BF16 && p->dtype != SDPA_FP16) return SDPA_ERR_UNSUPPORTED;
  if (p->head_dim != 128 && p->head_dim != 192 && p->head_dim != 256 && p->head_dim != 512)
    return SDPA_ERR_UNSUPPORTED;
  if (p->num_heads_q <= 0 || p->num_heads_kv <= 0 || p->rows < 0) return SDPA_ERR_INVALID_ARG;
  if (p->num_heads_q > 65536 || p->num_heads_kv > 65536 || p->rows > 0x7fffffffLL) return SDPA_ERR_UNSUPPORTED;
  if (p->rotary_dim < 0 || p->rotary_dim > p->head_dim || p->rotary_dim % 16) return SDPA_ERR_INVALID_ARG;
  if (p->rotary_dim > 0 && p->max_positions < 1) return SDPA_ERR_INVALID_ARG;
  if (p->interleaved != 0 && p->interleaved != 1) return SDPA_ERR_INVALID_ARG;
  if (!std::isfinite(p->eps) || p->eps < 0.f) return SDPA_ERR_INVALID_ARG;
  const long long qw = (long long)p->num_heads_q * p->head_dim, kw = (long long)p->num_heads_kv * p->head_dim;
  for (const auto& [st, wd] : {std::pair<long long, long long>{p->q_stride, qw}, {p->k_stride, kw},
                               {p->dq_stride, qw}, {p->dk_stride, kw}})
    if (st != 0 && (st < wd || st % 8 || st >= (1LL << 32))) return SDPA_ERR_INVALID_ARG;
  return SDPA_OK;
}

// Whether rows of `aw` and of `bw` 16-bit values, `as` and `bs` elements apart, lie apart: two outputs apart as a whole,
// or slices of one tensor's rows, which interleave.
bool rows_apart(Extent a, long long as, long long aw, Extent b, long long bs, long long bw) {
  if (!overlaps(a, b)) return true;
  if (as != bs || a.lo == b.lo) return false;
  return b.lo > a.lo ? b.lo - a.lo >= (uintptr_t)aw * 2 && b.lo - a.lo + bw * 2 <= (uintptr_t)as * 2
                     : a.lo - b.lo >= (uintptr_t)bw * 2 && a.lo - b.lo + aw * 2 <= (uintptr_t)as * 2;
}

// The axes of a rotation of `rot` values for the kernels; a: may be NULL (one position a token).
int make_axes(const sdpa_rope_axes* a, int rot, long long rows, RopeAxes* out) {
  std::memset(out, 0, sizeof(*out));
  if (!a) return SDPA_OK;
  if (a->num_axes < 1 || a->num_axes > SDPA_ROPE_AXES_MAX) return SDPA_ERR_INVALID_ARG;
  if (a->position_stride != 0 && (a->position_stride < rows || a->position_stride >= (1LL << 36))) return SDPA_ERR_INVALID_ARG;
  out->n = a->num_axes;
  out->pos_stride = a->position_stride ? a->position_stride : rows;
  int at = 0;
  for (int x = 0; x < SDPA_ROPE_AXES_MAX; ++x) {
    out->end[x] = std::numeric_limits<int>::max();
    if (x >= a->num_axes) continue;
    if (a->pairs[x] < 1 || a->pairs[x] > rot / 2 - at) return SDPA_ERR_INVALID_ARG;
    const int end = at + a->pairs[x];
    if (x + 1 < a->num_axes) out->end[x] = end;
    // whole blocks of 4 pairs (16 bytes, what a bulk copy moves); rot / 2 is a multiple of 8
    out->lo[x] = at & ~3;
    out->len[x] = ((end + 3) & ~3) - out->lo[x];
    out->cos_at[x] = out->floats - out->lo[x];
    out->sin_at[x] = out->cos_at[x] + out->len[x];
    out->floats += 2 * out->len[x];
    at = end;
  }
  return at == rot / 2 ? SDPA_OK : SDPA_ERR_INVALID_ARG;
}

// Bytes of the positions of `rows` tokens.
size_t positions_bytes(const RopeAxes& a, long long rows) {
  return 4 * (size_t)((a.n ? (a.n - 1) * a.pos_stride : 0) + rows);
}

// Bytes spanned by `rows` rows of `width` 16-bit values, `stride` elements apart.
size_t span(long long rows, long long stride, long long width) {
  return rows > 0 ? (size_t)((rows - 1) * stride + width) * 2 : 0;
}

// Width of V rows of a paged problem (192 pairs with 128).
int paged_dv(const sdpa_paged_problem* p) {
  if (p->head_dim_v) return p->head_dim_v;
  return p->head_dim == 192 ? 128 : p->head_dim;
}

int check_paged(const sdpa_paged_problem* p) {
  if (!p) return SDPA_ERR_INVALID_ARG;
  if (p->dtype != SDPA_BF16 && p->dtype != SDPA_FP16) return SDPA_ERR_UNSUPPORTED;
  if (p->head_dim_v < 0) return SDPA_ERR_INVALID_ARG;
  if (!head_dims_supported(p->head_dim, paged_dv(p))) return SDPA_ERR_UNSUPPORTED;
  if (p->batch < 0 || p->total_q < 0 || p->seqlen_q < 0 || p->seqlen_kv < 0) return SDPA_ERR_INVALID_ARG;
  if (p->num_heads_q <= 0 || p->num_heads_kv <= 0 || p->num_heads_q % p->num_heads_kv) return SDPA_ERR_INVALID_ARG;
  if (p->num_heads_q > 65536 || p->batch > (1 << 20) || p->seqlen_kv > (1 << 30) || p->seqlen_q > (1 << 30))
    return SDPA_ERR_UNSUPPORTED;
  if (p->page_size <= 0 || p->num_pages <= 0 || p->max_pages <= 0) return SDPA_ERR_INVALID_ARG;
  if (p->page_size % 16 || p->page_size > (1 << 20)) return SDPA_ERR_UNSUPPORTED;
  if ((long long)p->max_pages * p->page_size < p->seqlen_kv) return SDPA_ERR_INVALID_ARG;
  if (p->table_stride != 0 && p->table_stride < p->max_pages) return SDPA_ERR_INVALID_ARG;
  if (p->mask_type < SDPA_MASK_NONE || p->mask_type > SDPA_MASK_CAUSAL_BOTTOM_RIGHT) return SDPA_ERR_INVALID_ARG;
  if (p->mask_type == SDPA_MASK_CAUSAL_TOP_LEFT) return SDPA_ERR_UNSUPPORTED;  // cached keys precede the new ones
  if (p->window_left < -1) return SDPA_ERR_INVALID_ARG;
  if (p->window_left >= 0 && p->mask_type == SDPA_MASK_NONE) return SDPA_ERR_UNSUPPORTED;
  if (!std::isfinite(p->softmax_scale) || p->softmax_scale < 0.f) return SDPA_ERR_INVALID_ARG;
  const int d = p->head_dim, dv = paged_dv(p);
  for (const auto& [st, wd] : {std::pair<long long, long long>{p->k_page_stride, d}, {p->k_slot_stride, d},
                               {p->k_head_stride, d}, {p->v_page_stride, dv}, {p->v_slot_stride, dv},
                               {p->v_head_stride, dv}})
    if (st < wd || st % 8 || st >= (1LL << 36)) return SDPA_ERR_INVALID_ARG;
  // the order of head and slot is the strides', K's and V's the same, and each stride a multiple of the smaller one
  // (a dimension of one head has no order)
  const bool one = p->num_heads_kv == 1;
  for (const auto& [page, slot, head] :
       {std::array<long long, 3>{p->k_page_stride, p->k_slot_stride, p->k_head_stride},
        std::array<long long, 3>{p->v_page_stride, p->v_slot_stride, p->v_head_stride}}) {
    const long long lo = one ? slot : std::min(slot, head), hi = one ? slot : std::max(slot, head);
    if ((!one && lo == hi) || hi % lo || (p->num_pages > 1 && page % hi)) return SDPA_ERR_UNSUPPORTED;
  }
  if (!one && (p->k_slot_stride < p->k_head_stride) != (p->v_slot_stride < p->v_head_stride)) return SDPA_ERR_UNSUPPORTED;
  for (const auto& [st, wd] : {std::pair<long long, long long>{p->q_stride, (long long)p->num_heads_q * d},
                               {p->k_stride, (long long)p->num_heads_kv * d},
                               {p->v_stride, (long long)p->num_heads_kv * dv}})
    if (st != 0 && (st < wd || st % 8 || st >= (1LL << 32))) return SDPA_ERR_INVALID_ARG;
  return SDPA_OK;
}

// One launch of the paged attention: how it cuts a sequence's rows into items.
struct PagedCutting {
  bool used, fits;
  int n;                         // rows of an item
  int block_heads, head_blocks;  // heads of a group in an item, items a group takes
  int q_tokens, tokens;          // tokens of one Q copy, and in an item
  int dv_item, dv_splits;        // value columns an item accumulates, items that share a row
  bool split;                    // rows kernel: items may be split over workers
  int tail;                      // chunk kernels: shares that the last items are cut into
  int workers;                   // CTAs, at most one per SM
};
struct PagedPlan {
  int small_q;         // sequences of at most this many new tokens go to the rows kernel, longer ones to the chunk kernel
  PagedCutting rows, chunk;
  size_t cuts_off[2], parts_off[2], total;  // workspace of the rows and of the chunk kernel
};
// The SMs of the device the library is written for: the plan, and with it the
// workspace size, must not depend on the device in use.
constexpr int kPagedWorkers = 152;

// n: rows of an item, in copies of q_rows.
PagedCutting paged_cutting(const sdpa_paged_problem* p, int n, int q_rows, int max_q, int dv_item) {
  PagedCutting c;
  constexpr int most = kPagedWorkers;
  const int group = p->num_heads_q / p->num_heads_kv, dv = paged_dv(p);
  c.used = true;
  c.n = n;
  c.block_heads = std::min(group, q_rows);
  c.head_blocks = (group + c.block_heads - 1) / c.block_heads;
  c.q_tokens = std::max(1, std::min(q_rows / c.block_heads, max_q));
  c.tokens = c.q_tokens * (n / q_rows);
  c.dv_item = dv_item;
  c.dv_splits = dv / dv_item;
  // the most items the batch can have, and the most key tiles one of them sees
  const long long blocks = std::min((long long)p->batch * ((max_q + c.tokens - 1) / c.tokens),
                                    (long long)p->total_q / c.tokens + p->batch);
  const long long items = blocks * p->num_heads_kv * c.head_blocks * c.dv_splits;
  long long tiles = (p->seqlen_kv + 127) / 128;
  if (p->window_left >= 0) tiles = std::min<long long>(tiles, ((long long)p->window_left + c.tokens) / 128 + 2);
  if (n <= 64) {
    // short items are not worth the join (and its launch)
    c.split = tiles > 4;
    c.tail = 0;
  } else {
    // Whole items by ticket keep the CTAs on the same keys (with all items cut into equal shares, 2048 tokens over
    // 131072 keys took 14 % longer, 8 x 1024 over 32768 41 %). The last, uneven round is cut into shares where it leaves
    // enough SMs idle, for long enough to pay for the join. Whole -> cut in us, by items of the batch and key tiles:
    //   up to half of the SMs   192/128: 56 items of 16 tiles 32 -> 35, of 32 54 -> 41; 256: 72 of 20 46 -> 57, of 48 93 ->
    //                           83; 128 (256-row items): 24 of 16 36 -> 41, of 32 58 -> 44; 72 of 32 58 -> 62, of 48 79 -> 71
    //   up to two thirds        192/128: 88 of 48 74 -> 64; 256: 93 -> 96; 512: 126 -> 116
    //   at most 3/4 full, long  192/128: 104 of 96 136 -> 116, 248 of 64 173 -> 174, of 96 257 -> 241; 256: 104 of 64 122 ->
    //                           126, of 96 175 -> 166; but 512: 136 of 96 259 -> 316, 288 of 96 492 -> 537
    //   at most half full       192/128: 224 of 32 99 -> 104, of 48 140 -> 136; 512: 512 of 48 482 -> 460; but 256: 576 of 64
    //                           451 -> 509 (79 % full), 896 of 48 525 -> 549 (89 %)
    //   128, up to two rounds   200 of 64 176 -> 178, of 256 715 -> 557; 256 of 256 727 -> 700; but 136 of 256 375 -> 404,
    //                           296 of 256 768 -> 798
    // A share for every CTA where all items are cut: 17 sequences at head_dim 256, 163 -> 143 us against two.
    c.split = false;
    const long long rest = items % most, start = std::max(16LL, items * 2 / 5 + (n == 256 ? 8 : 0));
    bool cut = false;
    if (items * 2 <= most)
      cut = tiles >= start;
    else if (items < most * 2 && rest * 4 <= most * 3 && tiles >= (n == 256 ? 256 : 96))
      cut = true;
    else if (n == 128)
      cut = tiles >= 48 && (items < most ? items * 3 <= most * 2 : items < most * 6 && rest * 2 <= most);
    c.tail = !cut ? 0 : items < most ? most : 2 * most;
  }
  // the length of a block and the ticket counter are 32-bit numbers
  c.fits = (long long)p->num_heads_kv * c.head_blocks * c.dv_splits * std::max(tiles, 1LL) < (1LL << 31) &&
           items < 0x7fff0000LL;
  const long long pieces = (c.split || c.tail) && items < most ? items * std::max(tiles, 1LL) : items;
  c.workers = (int)std::max(1LL, std::min<long long>(most, pieces));
  return c;
}

// Where the two launches' records lie in the workspace.
void paged_workspace(PagedPlan& pl) {
  size_t at = 256;  // totals and tickets
  for (int x = 0; x < 2; ++x) {
    const PagedCutting& c = x ? pl.chunk : pl.rows;
    pl.cuts_off[x] = at;
    const size_t shares = !c.used ? 0 : c.tail ? c.tail : c.split ? c.workers : 0;
    at = round_up(at + shares * paged_cut_bytes(), 256);
    pl.parts_off[x] = at;
    at = round_up(at + shares * 2 * c.n * (c.dv_item + 2) * 4, 256);
  }
  pl.total = at;
}

PagedPlan paged_plan(const sdpa_paged_problem* p) {
  PagedPlan pl;
  const int group = p->num_heads_q / p->num_heads_kv, dv = paged_dv(p);
  const int most = dv == 512 ? 32 : 64;  // rows of the rows kernel: a 64-row Q of 512 columns leaves the ring too few stages
  const int few = std::max(1, most / group);
  pl.rows.used = pl.chunk.used = false;
  // where the rows add up to seqlen_q for every sequence there is none for the rows kernel, whose launch and join cost
  // some 10 us even so; the chunk kernel serves a shorter sequence as well, only less well
  const bool uniform = p->total_q >= (long long)p->batch * p->seqlen_q;
  pl.small_q = p->seqlen_q <= few ? p->seqlen_q : uniform ? -1 : few;
  if (pl.small_q >= 0) {
    const int max_q = std::min(p->seqlen_q, pl.small_q);
    const long long rows = (long long)group * std::max(max_q, 1);
    const int n = rows <= 16 ? 16 : (rows <= 32 || most == 32) ? 32 : 64;
    pl.rows = paged_cutting(p, n, n, max_q, dv);
  }
  if (p->seqlen_q > pl.small_q) pl.chunk = paged_cutting(p, p->head_dim == 128 ? 256 : 128, 128, p->seqlen_q, std::min(dv, 256));
  paged_workspace(pl);
  return pl;
}

// The attention over an 8-bit cache: one kernel for any number of tokens, in items of 8, 16 or 32 rows, at most as many as
// the tensor memory holds O of with its three terms, twice: 32 of 128 columns, 16 of 256, 8 of 512.
PagedPlan paged_fp8_plan(const sdpa_paged_problem* p) {
  PagedPlan pl;
  const int group = p->num_heads_q / p->num_heads_kv, dv = paged_dv(p);
  pl.rows.used = pl.chunk.used = false;
  pl.small_q = p->seqlen_q;
  const long long rows = (long long)group * std::max(p->seqlen_q, 1);
  const int n = rows <= 8 || dv == 512 ? 8 : rows <= 16 || dv == 256 ? 16 : 32;
  pl.rows = paged_cutting(p, n, n, p->seqlen_q, dv);
  pl.rows.fits = pl.rows.fits && (long long)p->num_heads_kv * pl.rows.head_blocks * ((p->seqlen_kv + 127) / 128 + 8LL) < (1LL << 31);
  paged_workspace(pl);
  return pl;
}

// What a launch of the paged attention is told, apart from its copies.
PagedParams paged_params(const sdpa_paged_problem* p, const PagedPlan& pl, bool small, const int32_t* cu_seqlens_q,
                         const int32_t* kv_lens, const int32_t* block_table, void* o, float* lse, uint8_t* ws, int* err,
                         AddrTable* chk) {
  const PagedCutting* c = small ? &pl.rows : &pl.chunk;
  PagedParams P;
  std::memset(&P, 0, sizeof(P));
  P.batch = p->batch;
  P.total_q = p->total_q;
  P.max_q = p->seqlen_q;
  P.max_kv = p->seqlen_kv;
  P.hq = p->num_heads_q;
  P.group = p->num_heads_q / p->num_heads_kv;
  P.block_heads = c->block_heads;
  P.head_blocks = c->head_blocks;
  P.tokens = c->tokens;
  P.dv = paged_dv(p);
  P.dv_splits = c->dv_splits;
  P.units_per_block = p->num_heads_kv * c->head_blocks * c->dv_splits;
  P.small_q = pl.small_q;
  P.small = small;
  P.split = c->split;
  P.tail = c->tail;
  P.q_box_rows = c->q_tokens * c->block_heads;
  P.causal = p->mask_type != SDPA_MASK_NONE;
  P.window = p->window_left < p->seqlen_kv ? p->window_left : -1;  // as wide as every length: no window
  // Never 0: the chunk kernel masks a score by -inf before the scale, and -inf x 0 is NaN. By the smallest number
  // above 0 every finite score is below 2^-20 instead, whose 2^x is 1 to an fp32 rounding or two. (Zeroing the
  // scores in the kernel: 4 x 1024 tokens over 32768 keys at head_dim 256 1.59 -> 1.72 ms, whatever the scale.)
  P.scale_log2 = p->softmax_scale * 1.4426950408889634f;
  if (!(P.scale_log2 > 0.f)) P.scale_log2 = std::numeric_limits<float>::denorm_min();
  P.page_size = p->page_size;
  P.num_pages = p->num_pages;
  P.cu_q = cu_seqlens_q;
  P.kv_lens = kv_lens;
  P.block_table = block_table;
  P.table_stride = p->table_stride ? p->table_stride : p->max_pages;
  P.o = o;
  P.lse = lse;
  P.behind = !small && pl.rows.used;
  P.total_tiles = reinterpret_cast<long long*>(ws + (small ? 0 : 64));
  P.tickets = reinterpret_cast<int*>(ws + 128);
  P.cuts = reinterpret_cast<PagedCut*>(ws + pl.cuts_off[small ? 0 : 1]);
  P.parts = reinterpret_cast<float*>(ws + pl.parts_off[small ? 0 : 1]);
  P.err = err;
  P.chk = chk;
  return P;
}

// Whether a slot's heads lie apart by more than its pages' slots ([page][head][slot]);
// a single head counts as [page][slot][head].
bool slot_first(const sdpa_paged_problem* p) { return p->num_heads_kv > 1 && p->k_slot_stride < p->k_head_stride; }

// 4-D map of a paged cache {width, then head and slot by increasing stride, page}: boxes are 128 bytes of a row (64
// 16-bit values or 128 codes, 128-byte swizzle) x box_rows slots of one head of one page.
int encode_cache(CUtensorMap* m, const void* base, const sdpa_paged_problem* p, int width, long long page, long long slot,
                 long long head, int box_rows, CUtensorMapDataType type, int bytes) {
  auto fn = encode_fn();
  if (!fn) return SDPA_ERR_CUDA;
  const bool first = slot_first(p);
  if (p->num_heads_kv == 1) head = slot;  // strides of single entries are never taken: keep the map's order
  const long long lo = std::min(slot, head), hi = std::max(slot, head);
  if (p->num_pages == 1) page = hi;
  const cuuint64_t dims[4] = {(cuuint64_t)width, (cuuint64_t)(first ? p->page_size : p->num_heads_kv),
                              (cuuint64_t)(first ? p->num_heads_kv : p->page_size), (cuuint64_t)p->num_pages};
  const cuuint64_t strides[3] = {(cuuint64_t)lo * bytes, (cuuint64_t)hi * bytes, (cuuint64_t)page * bytes};
  const cuuint32_t box[4] = {(cuuint32_t)(128 / bytes), (cuuint32_t)(first ? box_rows : 1), (cuuint32_t)(first ? 1 : box_rows), 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  // 256 bytes from memory at a time only where they belong to one row: a 128-byte row, or the last 128 bytes of one of 384,
  // would bring the next head's along, for nobody (64 sequences of 500 to 16384 keys, 256 bytes at a time everywhere / as
  // here: codes of head_dim 128 297 / 253 us; 16-bit rows of 192 446 / 420, 16 sequences of 1 to 16 tokens 71 to 78 / 68 to
  // 76; with [head][slot] pages, whose next row is wanted too, and in the chunk kernels within 0.4 %)
  const auto promotion = (long long)width * bytes % 256 == 0 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B;
  CUresult r = fn(m, type, 4, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, promotion, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? SDPA_OK : SDPA_ERR_CUDA;
}
int encode_cache(CUtensorMap* m, const void* base, const sdpa_paged_problem* p, int width, long long page, long long slot,
                 long long head, int box_rows, bool bf16) {
  return encode_cache(m, base, p, width, page, slot, head, box_rows,
                      bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2);
}
int encode_codes(CUtensorMap* m, const void* base, const sdpa_paged_problem* p, int width, long long page, long long slot,
                 long long head, int box_rows) {
  return encode_cache(m, base, p, width, page, slot, head, box_rows, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1);
}

// One of a paged cache's tensors: rows of `width` values of `bytes` each, one for every page, slot and head.
struct CacheView {
  const void* base;
  long long page, slot, head;  // elements between pages, slots and heads
  int width, bytes;
};
CacheView k_view(const sdpa_paged_problem* p, const void* base, int bytes = 2) {
  return {base, p->k_page_stride, p->k_slot_stride, p->k_head_stride, p->head_dim, bytes};
}
CacheView v_view(const sdpa_paged_problem* p, const void* base, int bytes = 2) {
  return {base, p->v_page_stride, p->v_slot_stride, p->v_head_stride, paged_dv(p), bytes};
}

// The bytes from its first element to its last.
Extent cache_extent(const sdpa_paged_problem* p, const CacheView& c) {
  return extent(c.base, (size_t)((p->num_pages - 1) * c.page + (p->page_size - 1) * c.slot + (p->num_heads_kv - 1) * c.head +
                                 c.width) * c.bytes);
}

// Whether every row of the two tensors lies apart from all others. Where their spans interleave (pages that hold K and V
// together), addresses are compared modulo a step that both tensors' strides from some level on are multiples of, all of
// them (scale bytes' strides need not be multiples of one another): the stretch of a step that one fills and the one that
// the other fills must not meet.
bool caches_apart(const sdpa_paged_problem* p, const CacheView& kc, const CacheView& vc) {
  struct Level {
    long long stride, fill;  // in bytes; fill: from the first to the last within one step of the stride
  };
  const bool one = p->num_heads_kv == 1;  // a single head's stride is never taken
  auto levels = [&](const CacheView& c) {
    const bool first = one || c.slot < c.head;  // slots vary before heads
    const long long lo = first ? c.slot : c.head, hi = one || !first ? c.slot : c.head;
    const long long inner = one ? c.width : ((first ? p->page_size : p->num_heads_kv) - 1) * lo + c.width;
    const long long whole = ((first && !one ? p->num_heads_kv : p->page_size) - 1) * hi + inner;
    const long long b = c.bytes;
    return std::array<Level, 3>{Level{lo * b, c.width * b}, Level{hi * b, inner * b}, Level{c.page * b, whole * b}};
  };
  const auto k = levels(kc), v = levels(vc);
  const int used = p->num_pages > 1 ? 3 : 2;
  for (int i = 0; i < used; ++i)
    if (k[i].fill > k[i].stride || v[i].fill > v[i].stride) return false;
  if (!overlaps(cache_extent(p, kc), cache_extent(p, vc))) return true;
  const long long off = (long long)(reinterpret_cast<uintptr_t>(vc.base) - reinterpret_cast<uintptr_t>(kc.base));
  for (int i = 0; i < used; ++i) {
    long long step = 0;
    for (int j = i; j < used; ++j) step = std::gcd(step, std::gcd(k[j].stride, v[j].stride));
    const long long at = (off % step + step) % step;
    if (at >= k[i].fill && at + v[i].fill <= step) return true;
  }
  return false;
}

// The scale bytes beside an 8-bit cache of a checked problem: whether they and the codes' strides can be served.
int check_fp8_cache(const sdpa_paged_problem* p, const sdpa_paged_scales* c) {
  if (!c || !c->k || !c->v) return SDPA_ERR_INVALID_ARG;
  // codes are moved 16 bytes at a time
  for (long long st : {p->k_page_stride, p->k_slot_stride, p->k_head_stride, p->v_page_stride, p->v_slot_stride,
                       p->v_head_stride})
    if (st % 16) return SDPA_ERR_INVALID_ARG;
  for (long long st : {c->k_page_stride, c->k_slot_stride, c->k_head_stride, c->v_page_stride, c->v_slot_stride,
                       c->v_head_stride})
    if (st < 1 || st >= (1LL << 36)) return SDPA_ERR_INVALID_ARG;
  return SDPA_OK;
}
CacheView k_scale_view(const sdpa_paged_scales* c) {
  return {c->k, c->k_page_stride, c->k_slot_stride, c->k_head_stride, 1, 1};
}
CacheView v_scale_view(const sdpa_paged_scales* c) {
  return {c->v, c->v_page_stride, c->v_slot_stride, c->v_head_stride, 1, 1};
}

}  // namespace

static std::atomic<int> g_max_ctas{0};
int debug_max_ctas() { return g_max_ctas.load(std::memory_order_relaxed); }

// Unique ID of the calling thread's current context (cuCtxGetId; IDs are not
// reused within a process), 0 when there is none or the driver lacks the call.
static unsigned long long current_context_id() {
  using GetCurrent = CUresult (*)(CUcontext*);
  using GetId = CUresult (*)(CUcontext, unsigned long long*);
  static GetCurrent get_current = nullptr;
  static GetId get_id = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &ptr, 4000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      get_current = reinterpret_cast<GetCurrent>(ptr);
    ptr = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuCtxGetId", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      get_id = reinterpret_cast<GetId>(ptr);
  });
  if (!get_current || !get_id) return 0;
  CUcontext ctx = nullptr;
  unsigned long long id = 0;
  if (get_current(&ctx) != CUDA_SUCCESS || !ctx || get_id(ctx, &id) != CUDA_SUCCESS) return 0;
  return id;
}

void* device_symbol_address(const void* symbol) {
  struct Entry {
    const void* symbol;
    int dev;
    unsigned long long ctx;
    void* addr;
  };
  static std::mutex mu;
  static Entry cache[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return nullptr;
  std::lock_guard<std::mutex> lock(mu);
  const unsigned long long ctx = current_context_id();
  Entry* slot = nullptr;
  for (Entry& e : cache) {
    if (e.symbol == symbol && e.dev == dev) {
      slot = &e;
      break;
    }
    if (!slot && !e.symbol) slot = &e;  // first free entry, unless a match follows
  }
  if (slot && slot->symbol == symbol && slot->dev == dev && ctx != 0 && slot->ctx == ctx) return slot->addr;
  void* addr = nullptr;
  if (cudaGetSymbolAddress(&addr, symbol) != cudaSuccess || !addr) return nullptr;
  const unsigned long long now = current_context_id();  // the lookup may have made the context current
  if (slot && now != 0) *slot = Entry{symbol, dev, now, addr};
  return addr;
}

int set_kernel_smem(const void* kernel, int bytes, int carveout) {
  static std::mutex mu;
  static std::set<std::pair<const void*, int>> done;  // (kernel, device) already configured
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return SDPA_ERR_CUDA;
  std::lock_guard<std::mutex> lock(mu);
  if (done.count({kernel, dev})) return SDPA_OK;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
    return SDPA_ERR_CUDA;
  if (carveout >= 0 && cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, carveout) !=
                           cudaSuccess)
    return SDPA_ERR_CUDA;
  done.insert({kernel, dev});
  return SDPA_OK;
}

}  // namespace sdpa

using namespace sdpa;

extern "C" {

int sdpa_check_problem(const sdpa_problem* p) { return check(p); }

size_t sdpa_fwd_workspace_size(const sdpa_problem* p) {
  if (check(p) != SDPA_OK) return 0;
  // THD: the metadata guard word at offset 0; head_dim 128: the tile ticket
  // counter of the persistent kernel at offset 128
  return (p->layout == SDPA_THD || p->head_dim == 128) ? 256 : 0;
}

size_t sdpa_bwd_workspace_size(const sdpa_problem* p) {
  if (check(p) != SDPA_OK || dv_of(p) != p->head_dim) return 0;
  return bwd_ws(p).total;
}

int sdpa_fwd(const sdpa_problem* p, const void* q, const void* k, const void* v, void* o, float* lse,
             const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_kv, void* workspace, size_t ws_bytes,
             void* stream) {
  t_last_launches = 0;
  int rc = check(p);
  if (rc) return rc;
  int rq, rk, hq, hk;
  view(p, rq, rk, hq, hk);
  const bool thd = p->layout == SDPA_THD;
  if (p->batch == 0 || rq == 0) return SDPA_OK;
  if (!q || !k || !v || !o || !lse) return SDPA_ERR_INVALID_ARG;
  if (thd && (!cu_seqlens_q || !cu_seqlens_kv)) return SDPA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
    return SDPA_ERR_ALIGNMENT;
  const size_t need = sdpa_fwd_workspace_size(p);
  if (ws_bytes < need || (need && !workspace)) return SDPA_ERR_WORKSPACE_TOO_SMALL;
  if (need && !aligned16(workspace)) return SDPA_ERR_ALIGNMENT;
  const size_t qb = (size_t)rq * hq * p->head_dim * 2, kb = (size_t)rk * hk * p->head_dim * 2;
  const size_t vb = (size_t)rk * hk * dv_of(p) * 2, ob = (size_t)rq * hq * dv_of(p) * 2;
  const Extent eo = extent(o, ob), el = extent(lse, (size_t)rq * hq * 4);
  for (Extent in : {extent(q, qb), extent(k, kb), extent(v, vb)})
    if (overlaps(eo, in) || overlaps(el, in)) return SDPA_ERR_OVERLAP;
  if (overlaps(eo, el)) return SDPA_ERR_OVERLAP;
  if (need && (overlaps(extent(workspace, need), eo) || overlaps(extent(workspace, need), el)))
    return SDPA_ERR_OVERLAP;

  int* err = error_word();
  if (!err) return SDPA_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool bf16 = p->dtype == SDPA_BF16;
  FwdLaunch L;
  std::memset(&L, 0, sizeof(L));
  L.p.g = make_geom(p, cu_seqlens_q, cu_seqlens_kv);
  const size_t cub = thd ? 4 * ((size_t)p->batch + 1) : 0;
  L.p.g.chk = bind_extents({extent(q, qb), extent(k, kb), extent(v, vb), eo, el, extent(cu_seqlens_q, cub),
                            extent(cu_seqlens_kv, cub), extent(workspace, need)},
                           err, s);
  if (kAddrCheck && !L.p.g.chk) return SDPA_ERR_CUDA;
  L.p.o = o;
  L.p.lse = lse;
  L.p.err = err;
  L.p.guard = thd ? static_cast<const int*>(workspace) : nullptr;
  L.p.n_q_tiles = (p->seqlen_q + 127) / 128;
  L.p.dv_splits = p->head_dim == 512 ? 2 : 1;
  L.p.tile_counter = p->head_dim == 128 ? reinterpret_cast<int*>(static_cast<uint8_t*>(workspace) + 128) : nullptr;
  L.stream = s;
  const int dv_cta = dv_of(p) == 512 ? 256 : dv_of(p);  // value columns one CTA accumulates
  if ((rc = encode(&L.tmQ, q, p->head_dim, hq, rq, 128, bf16))) return rc;
  if ((rc = encode(&L.tmK, k, p->head_dim, hk, rk, 128, bf16))) return rc;
  if ((rc = encode(&L.tmV, v, dv_of(p), hk, rk, 32768 / (dv_cta * 2), bf16))) return rc;
  int launches = 0;
  if (thd) {
    rc = timed(SDPA_KERNEL_GUARD, s,
               [&] { return launch_guard(L.p.g, p->total_q, p->total_kv, static_cast<int*>(workspace), err, s); });
    if (rc) return rc;
    ++launches;
  }
  if ((rc = timed(SDPA_KERNEL_FWD, s, [&] { return launch_fwd(L, p->head_dim, dv_of(p), bf16); }))) return rc;
  ++launches;
  t_last_launches = launches;
  return SDPA_OK;
}

int sdpa_bwd(const sdpa_problem* p, const void* q, const void* k, const void* v, const void* o, const float* lse,
             const void* dout, void* dq, void* dk, void* dv, const int32_t* cu_seqlens_q,
             const int32_t* cu_seqlens_kv, void* workspace, size_t ws_bytes, void* stream) {
  t_last_launches = 0;
  int rc = check(p);
  if (rc) return rc;
  if (dv_of(p) != p->head_dim) return SDPA_ERR_UNSUPPORTED;  // the backward is symmetric only
  int rq, rk, hq, hk;
  view(p, rq, rk, hq, hk);
  const bool thd = p->layout == SDPA_THD;
  if (p->batch == 0 || (rq == 0 && rk == 0)) return SDPA_OK;
  if (!q || !k || !v || !o || !lse || !dout || !dq || !dk || !dv) return SDPA_ERR_INVALID_ARG;
  if (thd && (!cu_seqlens_q || !cu_seqlens_kv)) return SDPA_ERR_INVALID_ARG;
  for (const void* ptr : {q, k, v, o, (const void*)lse, dout, (const void*)dq, (const void*)dk, (const void*)dv})
    if (!aligned16(ptr)) return SDPA_ERR_ALIGNMENT;
  const BwdWs w = bwd_ws(p);
  if (ws_bytes < w.total || !workspace) return SDPA_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned16(workspace) || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return SDPA_ERR_ALIGNMENT;
  const size_t qb = (size_t)rq * hq * p->head_dim * 2, kb = (size_t)rk * hk * p->head_dim * 2;
  const Extent outs[4] = {extent(dq, qb), extent(dk, kb), extent(dv, kb), extent(workspace, w.total)};
  const Extent ins[6] = {extent(q, qb), extent(k, kb), extent(v, kb), extent(o, qb), extent(lse, (size_t)rq * hq * 4),
                         extent(dout, qb)};
  for (int a = 0; a < 4; ++a) {
    for (int b = 0; b < 6; ++b)
      if (overlaps(outs[a], ins[b])) return SDPA_ERR_OVERLAP;
    for (int b = a + 1; b < 4; ++b)
      if (overlaps(outs[a], outs[b])) return SDPA_ERR_OVERLAP;
  }

  int* err = error_word();
  if (!err) return SDPA_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool bf16 = p->dtype == SDPA_BF16;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  int* guard = thd ? reinterpret_cast<int*>(ws + w.guard_off) : nullptr;
  int* order = w.order_off ? reinterpret_cast<int*>(ws + w.order_off) : nullptr;
  float* lse2 = reinterpret_cast<float*>(ws + w.lse2_off);
  float* delta = reinterpret_cast<float*>(ws + w.delta_off);
  float* acc = reinterpret_cast<float*>(ws + w.acc_off);
  Geom g = make_geom(p, cu_seqlens_q, cu_seqlens_kv);
  const size_t cub = thd ? 4 * ((size_t)p->batch + 1) : 0;
  g.chk = bind_extents({outs[0], outs[1], outs[2], outs[3], ins[0], ins[1], ins[2], ins[3], ins[4], ins[5],
                        extent(cu_seqlens_q, cub), extent(cu_seqlens_kv, cub)},
                       err, s);
  if (kAddrCheck && !g.chk) return SDPA_ERR_CUDA;
  int launches = 0;
  if (thd) {
    if ((rc = timed(SDPA_KERNEL_GUARD, s, [&] { return launch_guard(g, p->total_q, p->total_kv, guard, err, s, order); })))
      return rc;
    ++launches;
  }
  PrepParams pp;
  pp.g = g;
  pp.o = o;
  pp.dout = dout;
  pp.lse = lse;
  pp.lse2 = lse2;
  pp.delta = delta;
  pp.stat_rows = w.stat_rows;
  pp.dq_acc = w.has_acc ? acc : nullptr;
  pp.guard = guard;
  if ((rc = timed(SDPA_KERNEL_PREPROCESS, s, [&] { return launch_preprocess(pp, bf16, s); }))) return rc;
  ++launches;

  if (p->head_dim != 128) {
    BigBwdLaunch B;
    std::memset(&B, 0, sizeof(B));
    B.p.g = g;
    B.p.p_tiles = ws + w.ptile_off;
    B.p.ds_tiles = ws + w.dstile_off;
    B.p.nlse2 = lse2;
    B.p.delta = delta;
    B.p.stat_rows = w.stat_rows;
    B.p.dq = dq;
    B.p.dk = dk;
    B.p.dv = dv;
    B.p.err = err;
    B.p.guard = guard;
    B.p.n_q_tiles = (p->seqlen_q + 127) / 128;
    B.p.n_kv_tiles = (p->seqlen_kv + 127) / 128;
    const BigPlan pl = big_plan(p);
    B.p.slots = pl.slots;
    B.p.chunk = pl.chunk;
    B.p.chunk_lo = 0;
    B.p.chunk_hi = B.p.n_kv_tiles;
    B.p.dq_acc = w.has_acc ? acc : nullptr;
    B.stream = s;
    if ((rc = encode(&B.tmQ, q, p->head_dim, hq, rq, 128, bf16))) return rc;
    if ((rc = encode(&B.tmDO, dout, p->head_dim, hq, rq, 128, bf16))) return rc;
    if ((rc = encode(&B.tmK, k, p->head_dim, hk, rk, 128, bf16))) return rc;
    if ((rc = encode(&B.tmV, v, p->head_dim, hk, rk, 128, bf16))) return rc;
    if ((rc = encode(&B.tmQ64, q, p->head_dim, hq, rq, 64, bf16))) return rc;
    if ((rc = encode(&B.tmDO64, dout, p->head_dim, hq, rq, 64, bf16))) return rc;
    if ((rc = encode(&B.tmK64, k, p->head_dim, hk, rk, 64, bf16))) return rc;
    int n = 0;
    if ((rc = timed(SDPA_KERNEL_BWD, s, [&] { return launch_bwd_big(B, p->head_dim, bf16, &n); }))) return rc;
    launches += n;
    if (w.has_acc) {  // dQ summed over the key-tile chunks: scale and convert once
      if ((rc = timed(SDPA_KERNEL_DQ_FINALIZE, s, [&] { return launch_dq_finalize(g, acc, dq, guard, bf16, s); })))
        return rc;
      ++launches;
    }
    t_last_launches = launches;
    return SDPA_OK;
  }

  BwdLaunch L;
  std::memset(&L, 0, sizeof(L));
  L.p.g = g;
  L.p.dq_acc = acc;
  L.p.lse2 = lse2;
  L.p.delta = delta;
  L.p.stat_rows = w.stat_rows;
  L.p.dk = dk;
  L.p.dv = dv;
  L.p.err = err;
  L.p.guard = guard;
  L.p.order = order;
  L.p.head_block = bwd_head_block(p);
  L.p.n_kv_tiles = (p->seqlen_kv + 127) / 128;
  L.stream = s;
  if ((rc = encode(&L.tmQ, q, p->head_dim, hq, rq, 64, bf16))) return rc;
  if ((rc = encode(&L.tmDO, dout, p->head_dim, hq, rq, 64, bf16))) return rc;
  if ((rc = encode(&L.tmK, k, p->head_dim, hk, rk, 128, bf16))) return rc;
  if ((rc = encode(&L.tmV, v, p->head_dim, hk, rk, 128, bf16))) return rc;
  const bool det = p->deterministic != 0;
  L.p.dq_acc = det ? nullptr : acc;
  int n = 0;
  if ((rc = timed(SDPA_KERNEL_BWD, s, [&] { return launch_bwd_dkdv(L, p->head_dim, bf16, !det, &n); }))) return rc;
  launches += n;
  if (det) {
    // dQ per query tile, key tiles in a fixed order, written once
    DqLaunch Dq;
    std::memset(&Dq, 0, sizeof(Dq));
    Dq.p.g = g;
    Dq.p.dq = dq;
    Dq.p.nlse2 = lse2;
    Dq.p.delta = delta;
    Dq.p.stat_rows = w.stat_rows;
    Dq.p.err = err;
    Dq.p.guard = guard;
    Dq.p.n_q_tiles = (p->seqlen_q + 127) / 128;
    Dq.stream = s;
    if ((rc = encode(&Dq.tmQ, q, p->head_dim, hq, rq, 128, bf16))) return rc;
    if ((rc = encode(&Dq.tmDO, dout, p->head_dim, hq, rq, 128, bf16))) return rc;
    if ((rc = encode(&Dq.tmK, k, p->head_dim, hk, rk, 128, bf16))) return rc;
    if ((rc = encode(&Dq.tmV, v, p->head_dim, hk, rk, 128, bf16))) return rc;
    if ((rc = timed(SDPA_KERNEL_BWD_DQ, s, [&] { return launch_dq128(Dq, bf16); }))) return rc;
    ++launches;
  } else {
    if ((rc = timed(SDPA_KERNEL_DQ_FINALIZE, s, [&] { return launch_dq_finalize(g, acc, dq, guard, bf16, s); })))
      return rc;
    ++launches;
  }
  t_last_launches = launches;
  return SDPA_OK;
}

size_t sdpa_fwd_fp8_workspace_size(const sdpa_problem* p) {
  if (check_fp8(p) != SDPA_OK) return 0;
  int rq, rk, hq, hk;
  view(p, rq, rk, hq, hk);
  return 256 + (size_t)hk * p->head_dim * fp8_vt_rows(p);
}

int sdpa_fwd_fp8(const sdpa_problem* p, const void* q8, const void* k8, const void* v8, float descale_q,
                 float descale_k, float descale_v, void* o, float* lse, const int32_t* cu_seqlens_q,
                 const int32_t* cu_seqlens_kv, void* workspace, size_t ws_bytes, void* stream) {
  t_last_launches = 0;
  int rc = check_fp8(p);
  if (rc) return rc;
  if (!std::isfinite(descale_q) || !std::isfinite(descale_k) || !std::isfinite(descale_v) || !(descale_q > 0.f) ||
      !(descale_k > 0.f) || !(descale_v > 0.f))
    return SDPA_ERR_INVALID_ARG;
  int rq, rk, hq, hk;
  view(p, rq, rk, hq, hk);
  const bool thd = p->layout == SDPA_THD;
  if (p->batch == 0 || rq == 0) return SDPA_OK;
  if (!q8 || !k8 || !v8 || !o || !lse) return SDPA_ERR_INVALID_ARG;
  if (thd && (!cu_seqlens_q || !cu_seqlens_kv)) return SDPA_ERR_INVALID_ARG;
  if (!aligned16(q8) || !aligned16(k8) || !aligned16(v8) || !aligned16(o) || !aligned16(lse))
    return SDPA_ERR_ALIGNMENT;
  const size_t need = sdpa_fwd_fp8_workspace_size(p);
  if (ws_bytes < need || !workspace) return SDPA_ERR_WORKSPACE_TOO_SMALL;
  if (reinterpret_cast<uintptr_t>(workspace) & 255u) return SDPA_ERR_ALIGNMENT;
  const size_t D = (size_t)p->head_dim;
  const size_t qb = (size_t)rq * hq * D, kb = (size_t)rk * hk * D, ob = (size_t)rq * hq * D * 2;
  const Extent outs[3] = {extent(o, ob), extent(lse, (size_t)rq * hq * 4), extent(workspace, need)};
  const Extent ins[3] = {extent(q8, qb), extent(k8, kb), extent(v8, kb)};
  for (int x = 0; x < 3; ++x) {
    for (int y = 0; y < 3; ++y)
      if (overlaps(outs[x], ins[y])) return SDPA_ERR_OVERLAP;
    for (int y = x + 1; y < 3; ++y)
      if (overlaps(outs[x], outs[y])) return SDPA_ERR_OVERLAP;
  }
  int* err = error_word();
  if (!err) return SDPA_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  Fp8Launch L;
  std::memset(&L, 0, sizeof(L));
  L.p.g = make_geom(p, cu_seqlens_q, cu_seqlens_kv);
  const size_t cub = thd ? 4 * ((size_t)p->batch + 1) : 0;
  L.p.g.chk = bind_extents({outs[0], outs[1], outs[2], ins[0], ins[1], ins[2], extent(cu_seqlens_q, cub),
                            extent(cu_seqlens_kv, cub)},
                           err, s);
  if (kAddrCheck && !L.p.g.chk) return SDPA_ERR_CUDA;
  L.p.g.scale = p->softmax_scale * descale_q * descale_k;  // scores of the decoded codes
  L.p.g.scale_log2 = L.p.g.scale * 1.4426950408889634f;
  L.p.v = static_cast<const uint8_t*>(v8);
  L.p.vt = ws + 256;
  L.p.tile_counter = reinterpret_cast<int*>(ws + 128);
  L.p.vt_rows = (int)fp8_vt_rows(p);
  L.p.o = o;
  L.p.lse = lse;
  L.p.err = err;
  L.p.guard = thd ? reinterpret_cast<const int*>(ws) : nullptr;
  L.p.n_q_tiles = (p->seqlen_q + 127) / 128;
  L.p.o_scale = descale_v / 448.f;
  L.stream = s;
  if ((size_t)L.p.vt_rows * hk * D >= (1ull << 40)) return SDPA_ERR_UNSUPPORTED;
  {
    // Q, K: boxes of 128 one-byte columns (a head_dim 256 tile is two); Vt: one box of D rows
    const cuuint64_t dq[3] = {D, (cuuint64_t)hq, (cuuint64_t)(rq > 0 ? rq : 1)};
    const cuuint64_t sq[2] = {D, (cuuint64_t)hq * D};
    const cuuint64_t dk[3] = {D, (cuuint64_t)hk, (cuuint64_t)(rk > 0 ? rk : 1)};
    const cuuint64_t sk[2] = {D, (cuuint64_t)hk * D};
    const cuuint64_t dvt[3] = {(cuuint64_t)L.p.vt_rows, D, (cuuint64_t)hk};
    const cuuint64_t svt[2] = {(cuuint64_t)L.p.vt_rows, (cuuint64_t)L.p.vt_rows * D};
    const cuuint32_t box_rows[3] = {128, 1, 128}, box_vt[3] = {128, (cuuint32_t)D, 1};
    if ((rc = encode_u8(&L.tmQ, q8, dq, sq, box_rows))) return rc;
    if ((rc = encode_u8(&L.tmK, k8, dk, sk, box_rows))) return rc;
    if ((rc = encode_u8(&L.tmVt, L.p.vt, dvt, svt, box_vt))) return rc;
  }
  int launches = 0;
  if (thd) {
    if ((rc = timed(SDPA_KERNEL_GUARD, s,
                    [&] { return launch_guard(L.p.g, p->total_q, p->total_kv, reinterpret_cast<int*>(ws), err, s); })))
      return rc;
    ++launches;
  }
  if ((rc = timed(SDPA_KERNEL_V_TRANSPOSE, s, [&] { return launch_vt(L.p, s); }))) return rc;
  ++launches;
  if ((rc = timed(SDPA_KERNEL_FWD, s, [&] { return launch_fwd_fp8(L, p->dtype == SDPA_BF16); }))) return rc;
  ++launches;
  t_last_launches = launches;
  return SDPA_OK;
}

int sdpa_merge(const sdpa_merge_problem* p, const void* o_parts, const float* lse_parts, void* o, float* lse,
               void* stream) {
  t_last_launches = 0;
  if (!p) return SDPA_ERR_INVALID_ARG;
  if (p->n_parts < 1 || p->n_parts > 64 || p->items < 0) return SDPA_ERR_INVALID_ARG;
  if (p->dtype != SDPA_BF16 && p->dtype != SDPA_FP16) return SDPA_ERR_UNSUPPORTED;
  if (p->head_dim != 128 && p->head_dim != 256 && p->head_dim != 512) return SDPA_ERR_UNSUPPORTED;
  if (p->items == 0) return SDPA_OK;
  if (!o_parts || !lse_parts || !o || !lse) return SDPA_ERR_INVALID_ARG;
  if (!aligned16(o_parts) || !aligned16(lse_parts) || !aligned16(o) || !aligned16(lse)) return SDPA_ERR_ALIGNMENT;
  const size_t ob = (size_t)p->items * p->head_dim * 2, lb = (size_t)p->items * 4;
  const Extent eo = extent(o, ob), el = extent(lse, lb);
  for (Extent in : {extent(o_parts, ob * p->n_parts), extent(lse_parts, lb * p->n_parts)})
    if (overlaps(eo, in) || overlaps(el, in)) return SDPA_ERR_OVERLAP;
  if (overlaps(eo, el)) return SDPA_ERR_OVERLAP;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  AddrTable* chk = bind_extents({eo, el, extent(o_parts, ob * p->n_parts), extent(lse_parts, lb * p->n_parts)},
                                error_word(), s);
  if (kAddrCheck && !chk) return SDPA_ERR_CUDA;
  const int rc = timed(SDPA_KERNEL_MERGE, s, [&] {
    return launch_merge(o_parts, lse_parts, o, lse, p->items, p->head_dim, p->n_parts, p->dtype == SDPA_BF16, chk,
                        s);
  });
  if (rc) return rc;
  t_last_launches = 1;
  return SDPA_OK;
}

static int norm_rope_call(const sdpa_norm_rope_problem* p, const sdpa_rope_axes* axes, const void* q, const void* k,
                          const void* q_weight, const void* k_weight, const float* cos_sin, const int32_t* positions,
                          void* q_out, void* k_out, void* stream) {
  t_last_launches = 0;
  int rc = check_norm_rope(p);
  if (rc) return rc;
  RopeAxes ax;
  if ((rc = make_axes(axes, p->rotary_dim, p->rows, &ax))) return rc;
  if (p->rows == 0) return SDPA_OK;
  if (!q || !k || !q_weight || !k_weight || !q_out || !k_out) return SDPA_ERR_INVALID_ARG;
  if (p->rotary_dim > 0 && (!cos_sin || !positions)) return SDPA_ERR_INVALID_ARG;
  for (const void* ptr : {q, k, q_weight, k_weight, (const void*)cos_sin, (const void*)q_out, (const void*)k_out})
    if (!aligned16(ptr)) return SDPA_ERR_ALIGNMENT;
  const long long qw = (long long)p->num_heads_q * p->head_dim, kw = (long long)p->num_heads_kv * p->head_dim;
  NormRopeParams L;
  std::memset(&L, 0, sizeof(L));
  L.rows = p->rows;
  L.hq = p->num_heads_q;
  L.hkv = p->num_heads_kv;
  L.rot = p->rotary_dim;
  L.interleaved = p->interleaved;
  L.eps = p->eps;
  L.q = q;
  L.k = k;
  L.qs = p->q_stride ? p->q_stride : qw;
  L.ks = p->k_stride ? p->k_stride : kw;
  L.wq = q_weight;
  L.wk = k_weight;
  L.table = cos_sin;
  L.max_pos = p->max_positions;
  L.pos = positions;
  L.axes = ax;
  L.q_out = q_out;
  L.k_out = k_out;
  const size_t wb = (size_t)p->head_dim * 2;
  const Extent eq = extent(q_out, (size_t)p->rows * qw * 2), ek = extent(k_out, (size_t)p->rows * kw * 2);
  const Extent ins[6] = {extent(q, span(p->rows, L.qs, qw)), extent(k, span(p->rows, L.ks, kw)),
                         extent(q_weight, wb), extent(k_weight, wb),
                         extent(cos_sin, p->rotary_dim ? (size_t)p->max_positions * p->rotary_dim * 4 : 0),
                         extent(positions, p->rotary_dim ? positions_bytes(ax, p->rows) : 0)};
  for (const Extent& in : ins)
    if (overlaps(eq, in) || overlaps(ek, in)) return SDPA_ERR_OVERLAP;
  if (overlaps(eq, ek)) return SDPA_ERR_OVERLAP;
  L.err = error_word();
  if (!L.err) return SDPA_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  L.chk = bind_extents({eq, ek, ins[0], ins[1], ins[2], ins[3], ins[4], ins[5]}, L.err, s);
  if (kAddrCheck && !L.chk) return SDPA_ERR_CUDA;
  rc = timed(SDPA_KERNEL_NORM_ROPE, s,
             [&] { return launch_norm_rope(L, p->head_dim, p->dtype == SDPA_BF16, false, s); });
  if (rc) return rc;
  t_last_launches = 1;
  return SDPA_OK;
}

int sdpa_qk_norm_rope(const sdpa_norm_rope_problem* p, const void* q, const void* k, const void* q_weight,
                      const void* k_weight, const float* cos_sin, const int32_t* positions, void* q_out, void* k_out,
                      void* stream) {
  return norm_rope_call(p, nullptr, q, k, q_weight, k_weight, cos_sin, positions, q_out, k_out, stream);
}

int sdpa_qk_norm_rope_axes(const sdpa_norm_rope_problem* p, const sdpa_rope_axes* axes, const void* q, const void* k,
                           const void* q_weight, const void* k_weight, const float* cos_sin, const int32_t* positions,
                           void* q_out, void* k_out, void* stream) {
  if (!axes) return SDPA_ERR_INVALID_ARG;
  return norm_rope_call(p, axes, q, k, q_weight, k_weight, cos_sin, positions, q_out, k_out, stream);
}

size_t sdpa_qk_norm_rope_bwd_workspace_size(const sdpa_norm_rope_problem* p) {
  if (check_norm_rope(p) != SDPA_OK || p->rows == 0) return 0;
  return (size_t)(norm_rope_bwd_plan(p->rows, p->num_heads_q, p->num_heads_kv, p->head_dim).blocks + 1) * p->head_dim * 4;
}

static int norm_rope_bwd_call(const sdpa_norm_rope_problem* p, const sdpa_rope_axes* axes, const void* dq_out,
                              const void* dk_out, const void* q, const void* k, const void* q_weight,
                              const void* k_weight, const float* cos_sin, const int32_t* positions, void* dq, void* dk,
                              float* dq_weight, float* dk_weight, void* workspace, size_t ws_bytes, void* stream) {
  t_last_launches = 0;
  int rc = check_norm_rope(p);
  if (rc) return rc;
  RopeAxes ax;
  if ((rc = make_axes(axes, p->rotary_dim, p->rows, &ax))) return rc;
  if (!dq_weight || !dk_weight) return SDPA_ERR_INVALID_ARG;
  if (!aligned16(dq_weight) || !aligned16(dk_weight)) return SDPA_ERR_ALIGNMENT;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const size_t gw = (size_t)p->head_dim * 4;
  if (p->rows == 0) {  // the weights' gradients of no rows are zeros
    if (overlaps(extent(dq_weight, gw), extent(dk_weight, gw))) return SDPA_ERR_OVERLAP;
    if (cudaMemsetAsync(dq_weight, 0, gw, s) != cudaSuccess || cudaMemsetAsync(dk_weight, 0, gw, s) != cudaSuccess)
      return SDPA_ERR_CUDA;
    return SDPA_OK;
  }
  if (!dq_out || !dk_out || !q || !k || !q_weight || !k_weight || !dq || !dk) return SDPA_ERR_INVALID_ARG;
  if (p->rotary_dim > 0 && (!cos_sin || !positions)) return SDPA_ERR_INVALID_ARG;
  for (const void* ptr : {dq_out, dk_out, q, k, q_weight, k_weight, (const void*)cos_sin, (const void*)dq,
                          (const void*)dk})
    if (!aligned16(ptr)) return SDPA_ERR_ALIGNMENT;
  const size_t need = sdpa_qk_norm_rope_bwd_workspace_size(p);
  if (!workspace || ws_bytes < need) return SDPA_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned16(workspace)) return SDPA_ERR_ALIGNMENT;
  const long long qw = (long long)p->num_heads_q * p->head_dim, kw = (long long)p->num_heads_kv * p->head_dim;
  NormRopeBwdParams L;
  std::memset(&L, 0, sizeof(L));
  L.rows = p->rows;
  L.hq = p->num_heads_q;
  L.hkv = p->num_heads_kv;
  L.rot = p->rotary_dim;
  L.interleaved = p->interleaved;
  L.eps = p->eps;
  L.gq = dq_out;
  L.gk = dk_out;
  L.q = q;
  L.k = k;
  L.qs = p->q_stride ? p->q_stride : qw;
  L.ks = p->k_stride ? p->k_stride : kw;
  L.wq = q_weight;
  L.wk = k_weight;
  L.table = cos_sin;
  L.max_pos = p->max_positions;
  L.pos = positions;
  L.axes = ax;
  L.dq = dq;
  L.dk = dk;
  L.dqs = p->dq_stride ? p->dq_stride : qw;
  L.dks = p->dk_stride ? p->dk_stride : kw;
  L.part = static_cast<float*>(workspace);
  L.dwq = dq_weight;
  L.dwk = dk_weight;
  const NormRopeBwdPlan pl = norm_rope_bwd_plan(p->rows, p->num_heads_q, p->num_heads_kv, p->head_dim);
  L.warps_q = pl.warps_q;
  L.blocks = pl.blocks;
  const size_t wb = (size_t)p->head_dim * 2;
  const Extent outs[5] = {extent(dq, span(p->rows, L.dqs, qw)), extent(dk, span(p->rows, L.dks, kw)),
                          extent(dq_weight, gw), extent(dk_weight, gw), extent(workspace, need)};
  const Extent ins[8] = {extent(dq_out, (size_t)p->rows * qw * 2), extent(dk_out, (size_t)p->rows * kw * 2),
                         extent(q, span(p->rows, L.qs, qw)), extent(k, span(p->rows, L.ks, kw)),
                         extent(q_weight, wb), extent(k_weight, wb),
                         extent(cos_sin, p->rotary_dim ? (size_t)p->max_positions * p->rotary_dim * 4 : 0),
                         extent(positions, p->rotary_dim ? positions_bytes(ax, p->rows) : 0)};
  for (int a = 0; a < 5; ++a) {
    for (const Extent& in : ins)
      if (overlaps(outs[a], in)) return SDPA_ERR_OVERLAP;
    for (int b = a + 1; b < 5; ++b) {
      const bool slices = a == 0 && b == 1 && rows_apart(outs[0], L.dqs, qw, outs[1], L.dks, kw);
      if (!slices && overlaps(outs[a], outs[b])) return SDPA_ERR_OVERLAP;
    }
  }
  L.err = error_word();
  if (!L.err) return SDPA_ERR_CUDA;
  L.chk = bind_extents({outs[0], outs[1], outs[2], outs[3], outs[4], ins[0], ins[1], ins[2], ins[3], ins[4], ins[5],
                        ins[6], ins[7]},
                       L.err, s);
  if (kAddrCheck && !L.chk) return SDPA_ERR_CUDA;
  int n = 0;
  rc = timed(SDPA_KERNEL_NORM_ROPE, s,
             [&] { return launch_norm_rope_bwd(L, p->head_dim, p->dtype == SDPA_BF16, &n, s); });
  if (rc) return rc;
  t_last_launches = n;
  return SDPA_OK;
}

int sdpa_qk_norm_rope_bwd(const sdpa_norm_rope_problem* p, const void* dq_out, const void* dk_out, const void* q,
                          const void* k, const void* q_weight, const void* k_weight, const float* cos_sin,
                          const int32_t* positions, void* dq, void* dk, float* dq_weight, float* dk_weight,
                          void* workspace, size_t ws_bytes, void* stream) {
  return norm_rope_bwd_call(p, nullptr, dq_out, dk_out, q, k, q_weight, k_weight, cos_sin, positions, dq, dk, dq_weight,
                            dk_weight, workspace, ws_bytes, stream);
}

int sdpa_qk_norm_rope_axes_bwd(const sdpa_norm_rope_problem* p, const sdpa_rope_axes* axes, const void* dq_out,
                               const void* dk_out, const void* q, const void* k, const void* q_weight,
                               const void* k_weight, const float* cos_sin, const int32_t* positions, void* dq, void* dk,
                               float* dq_weight, float* dk_weight, void* workspace, size_t ws_bytes, void* stream) {
  if (!axes) return SDPA_ERR_INVALID_ARG;
  return norm_rope_bwd_call(p, axes, dq_out, dk_out, q, k, q_weight, k_weight, cos_sin, positions, dq, dk, dq_weight,
                            dk_weight, workspace, ws_bytes, stream);
}

int sdpa_check_paged(const sdpa_paged_problem* p) { return check_paged(p); }

// scales: of a cache of E4M3 codes, or NULL (a 16-bit cache).
static int append_call(const sdpa_paged_problem* p, const sdpa_norm_rope_problem* n, const sdpa_rope_axes* axes,
                       const sdpa_paged_scales* scales, const void* q, const void* k, const void* v, const void* q_weight,
                       const void* k_weight, const float* cos_sin, const int32_t* positions, void* q_out, void* k_cache,
                       void* v_cache, const int32_t* cu_seqlens_q, const int32_t* kv_lens, const int32_t* block_table,
                       void* stream) {
  t_last_launches = 0;
  int rc = check_paged(p);
  if (rc) return rc;
  if (n) {
    sdpa_norm_rope_problem full = *n;  // its sizes are the paged problem's
    full.dtype = p->dtype;
    full.num_heads_q = p->num_heads_q;
    full.num_heads_kv = p->num_heads_kv;
    full.head_dim = p->head_dim;
    full.rows = p->total_q;
    full.q_stride = full.k_stride = full.dq_stride = full.dk_stride = 0;
    if ((rc = check_norm_rope(&full))) return rc;
  }
  RopeAxes ax;
  if (axes && !n) return SDPA_ERR_INVALID_ARG;
  if ((rc = make_axes(axes, n ? n->rotary_dim : 0, p->total_q, &ax))) return rc;
  if (scales && (rc = check_fp8_cache(p, scales))) return rc;
  if (p->batch == 0 || p->total_q == 0) return SDPA_OK;
  if (!k || !v || !k_cache || !v_cache || !cu_seqlens_q || !kv_lens || !block_table) return SDPA_ERR_INVALID_ARG;
  const bool rot = n && n->rotary_dim > 0;
  if (n && (!q || !q_out || !q_weight || !k_weight)) return SDPA_ERR_INVALID_ARG;
  if (rot && !cos_sin) return SDPA_ERR_INVALID_ARG;
  if (axes && !positions) return SDPA_ERR_INVALID_ARG;  // a cache position has no axes
  for (const void* ptr : {k, v, (const void*)k_cache, (const void*)v_cache})
    if (!aligned16(ptr)) return SDPA_ERR_ALIGNMENT;
  if (n)
    for (const void* ptr : {q, (const void*)q_out, q_weight, k_weight, (const void*)cos_sin})
      if (!aligned16(ptr)) return SDPA_ERR_ALIGNMENT;
  const int d = p->head_dim, dv = paged_dv(p);
  const long long qw = (long long)p->num_heads_q * d, kw = (long long)p->num_heads_kv * d,
                  vw = (long long)p->num_heads_kv * dv;
  NormRopeParams L;
  std::memset(&L, 0, sizeof(L));
  L.rows = p->total_q;
  L.hq = n ? p->num_heads_q : 0;
  L.hkv = p->num_heads_kv;
  L.k = k;
  L.v = v;
  L.ks = p->k_stride ? p->k_stride : kw;
  L.vs = p->v_stride ? p->v_stride : vw;
  if (n) {
    L.rot = n->rotary_dim;
    L.interleaved = n->interleaved;
    L.eps = n->eps;
    L.q = q;
    L.qs = p->q_stride ? p->q_stride : qw;
    L.wq = q_weight;
    L.wk = k_weight;
    L.table = cos_sin;
    L.max_pos = n->max_positions;
    L.pos = rot ? positions : nullptr;
    L.axes = ax;
    L.q_out = q_out;
  }
  L.batch = p->batch;
  L.max_pages = p->max_pages;
  L.num_pages = p->num_pages;
  L.page_size = p->page_size;
  L.cu_q = cu_seqlens_q;
  L.kv_lens = kv_lens;
  L.table_ids = block_table;
  L.table_stride = p->table_stride ? p->table_stride : p->max_pages;
  L.kc = k_cache;
  L.vc = v_cache;
  L.kc_page = p->k_page_stride;
  L.kc_slot = p->k_slot_stride;
  L.kc_head = p->k_head_stride;
  L.vc_page = p->v_page_stride;
  L.vc_slot = p->v_slot_stride;
  L.vc_head = p->v_head_stride;
  if (scales) {
    L.k_scale = scales->k;
    L.v_scale = scales->v;
    L.ks_page = scales->k_page_stride;
    L.ks_slot = scales->k_slot_stride;
    L.ks_head = scales->k_head_stride;
    L.vs_page = scales->v_page_stride;
    L.vs_slot = scales->v_slot_stride;
    L.vs_head = scales->v_head_stride;
  }
  const size_t wb = (size_t)d * 2;
  CacheView views[4] = {k_view(p, k_cache, scales ? 1 : 2), v_view(p, v_cache, scales ? 1 : 2)};
  const int n_views = scales ? 4 : 2;
  Extent outs[5] = {cache_extent(p, views[0]), cache_extent(p, views[1]),
                    extent(q_out, n ? (size_t)p->total_q * qw * 2 : 0), extent(nullptr, 0), extent(nullptr, 0)};
  if (scales) {
    views[2] = k_scale_view(scales);
    views[3] = v_scale_view(scales);
    outs[3] = cache_extent(p, views[2]);
    outs[4] = cache_extent(p, views[3]);
  }
  const Extent ins[10] = {extent(k, span(p->total_q, L.ks, kw)), extent(v, span(p->total_q, L.vs, vw)),
                          extent(q, n ? span(p->total_q, L.qs, qw) : 0), extent(q_weight, n ? wb : 0),
                          extent(k_weight, n ? wb : 0),
                          extent(cos_sin, rot ? (size_t)n->max_positions * n->rotary_dim * 4 : 0),
                          extent(positions, L.pos ? positions_bytes(ax, p->total_q) : 0),
                          extent(cu_seqlens_q, 4 * ((size_t)p->batch + 1)), extent(kv_lens, 4 * (size_t)p->batch),
                          extent(block_table, 4 * (size_t)((p->batch - 1) * L.table_stride + p->max_pages))};
  for (const Extent& out : outs)
    for (const Extent& in : ins)
      if (overlaps(out, in)) return SDPA_ERR_OVERLAP;
  for (int a = 0; a < n_views; ++a)
    for (int b = a + 1; b < n_views; ++b)
      if (!caches_apart(p, views[a], views[b])) return SDPA_ERR_OVERLAP;
  for (int a : {0, 1, 3, 4})
    if (overlaps(outs[2], outs[a])) return SDPA_ERR_OVERLAP;
  L.err = error_word();
  if (!L.err) return SDPA_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  L.chk = bind_extents({outs[0], outs[1], outs[2], outs[3], outs[4], ins[0], ins[1], ins[2], ins[3], ins[4], ins[5], ins[6], ins[7],
                        ins[8], ins[9]},
                       L.err, s);
  if (kAddrCheck && !L.chk) return SDPA_ERR_CUDA;
  rc = timed(SDPA_KERNEL_APPEND, s, [&] { return launch_norm_rope(L, d, p->dtype == SDPA_BF16, true, s); });
  if (rc) return rc;
  t_last_launches = 1;
  return SDPA_OK;
}

int sdpa_paged_append(const sdpa_paged_problem* p, const sdpa_norm_rope_problem* n, const void* q, const void* k,
                      const void* v, const void* q_weight, const void* k_weight, const float* cos_sin,
                      const int32_t* positions, void* q_out, void* k_cache, void* v_cache,
                      const int32_t* cu_seqlens_q, const int32_t* kv_lens, const int32_t* block_table, void* stream) {
  return append_call(p, n, nullptr, nullptr, q, k, v, q_weight, k_weight, cos_sin, positions, q_out, k_cache, v_cache,
                     cu_seqlens_q, kv_lens, block_table, stream);
}

int sdpa_paged_append_axes(const sdpa_paged_problem* p, const sdpa_norm_rope_problem* n, const sdpa_rope_axes* axes,
                           const void* q, const void* k, const void* v, const void* q_weight, const void* k_weight,
                           const float* cos_sin, const int32_t* positions, void* q_out, void* k_cache, void* v_cache,
                           const int32_t* cu_seqlens_q, const int32_t* kv_lens, const int32_t* block_table, void* stream) {
  if (!axes) return SDPA_ERR_INVALID_ARG;
  return append_call(p, n, axes, nullptr, q, k, v, q_weight, k_weight, cos_sin, positions, q_out, k_cache, v_cache,
                     cu_seqlens_q, kv_lens, block_table, stream);
}

int sdpa_paged_append_fp8(const sdpa_paged_problem* p, const sdpa_norm_rope_problem* n, const sdpa_rope_axes* axes,
                          const sdpa_paged_scales* scales, const void* q, const void* k, const void* v,
                          const void* q_weight, const void* k_weight, const float* cos_sin, const int32_t* positions,
                          void* q_out, void* k_cache, void* v_cache, const int32_t* cu_seqlens_q, const int32_t* kv_lens,
                          const int32_t* block_table, void* stream) {
  if (!scales) return SDPA_ERR_INVALID_ARG;
  return append_call(p, n, axes, scales, q, k, v, q_weight, k_weight, cos_sin, positions, q_out, k_cache, v_cache,
                     cu_seqlens_q, kv_lens, block_table, stream);
}

int sdpa_paged_read_fp8(const sdpa_paged_problem* p, const sdpa_paged_scales* scales, const void* k_cache,
                        const void* v_cache, void* k_out, void* v_out, const int32_t* cu_seqlens, const int32_t* kv_lens,
                        const int32_t* block_table, void* stream) {
  t_last_launches = 0;
  int rc = check_paged(p);
  if (rc) return rc;
  if ((rc = check_fp8_cache(p, scales))) return rc;
  if (p->batch == 0 || p->total_q == 0) return SDPA_OK;
  if (!k_cache || !v_cache || !k_out || !v_out || !cu_seqlens || !kv_lens || !block_table) return SDPA_ERR_INVALID_ARG;
  for (const void* ptr : {k_cache, v_cache, (const void*)k_out, (const void*)v_out})
    if (!aligned16(ptr)) return SDPA_ERR_ALIGNMENT;
  PagedReadParams L;
  std::memset(&L, 0, sizeof(L));
  L.rows = p->total_q;
  L.batch = p->batch;
  L.hkv = p->num_heads_kv;
  L.page_size = p->page_size;
  L.num_pages = p->num_pages;
  L.max_pages = p->max_pages;
  L.k_cache = static_cast<const uint8_t*>(k_cache);
  L.v_cache = static_cast<const uint8_t*>(v_cache);
  L.k_scale = scales->k;
  L.v_scale = scales->v;
  L.k_page = p->k_page_stride;
  L.k_slot = p->k_slot_stride;
  L.k_head = p->k_head_stride;
  L.v_page = p->v_page_stride;
  L.v_slot = p->v_slot_stride;
  L.v_head = p->v_head_stride;
  L.ks_page = scales->k_page_stride;
  L.ks_slot = scales->k_slot_stride;
  L.ks_head = scales->k_head_stride;
  L.vs_page = scales->v_page_stride;
  L.vs_slot = scales->v_slot_stride;
  L.vs_head = scales->v_head_stride;
  const long long kw = (long long)p->num_heads_kv * p->head_dim, vw = (long long)p->num_heads_kv * paged_dv(p);
  L.k_out = k_out;
  L.v_out = v_out;
  L.k_row = p->k_stride ? p->k_stride : kw;
  L.v_row = p->v_stride ? p->v_stride : vw;
  L.cu = cu_seqlens;
  L.kv_lens = kv_lens;
  L.block_table = block_table;
  L.table_stride = p->table_stride ? p->table_stride : p->max_pages;
  const Extent outs[2] = {extent(k_out, span(p->total_q, L.k_row, kw)), extent(v_out, span(p->total_q, L.v_row, vw))};
  const Extent ins[7] = {cache_extent(p, k_view(p, k_cache, 1)), cache_extent(p, v_view(p, v_cache, 1)),
                         cache_extent(p, k_scale_view(scales)), cache_extent(p, v_scale_view(scales)),
                         extent(cu_seqlens, 4 * ((size_t)p->batch + 1)), extent(kv_lens, 4 * (size_t)p->batch),
                         extent(block_table, 4 * (size_t)((p->batch - 1) * L.table_stride + p->max_pages))};
  for (const Extent& out : outs)
    for (const Extent& in : ins)
      if (overlaps(out, in)) return SDPA_ERR_OVERLAP;
  if (!rows_apart(outs[0], L.k_row, kw, outs[1], L.v_row, vw)) return SDPA_ERR_OVERLAP;
  L.err = error_word();
  if (!L.err) return SDPA_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  L.chk = bind_extents({outs[0], outs[1], ins[0], ins[1], ins[2], ins[3], ins[4], ins[5], ins[6]}, L.err, s);
  if (kAddrCheck && !L.chk) return SDPA_ERR_CUDA;
  rc = timed(SDPA_KERNEL_READ, s, [&] { return launch_paged_read(L, p->head_dim, p->dtype == SDPA_BF16, s); });
  if (rc) return rc;
  t_last_launches = 1;
  return SDPA_OK;
}

size_t sdpa_paged_fwd_workspace_size(const sdpa_paged_problem* p) {
  if (check_paged(p) != SDPA_OK || p->batch == 0 || p->total_q == 0) return 0;
  return paged_plan(p).total;
}

int sdpa_paged_fwd(const sdpa_paged_problem* p, const void* q, const void* k_cache, const void* v_cache, void* o,
                   float* lse, const int32_t* cu_seqlens_q, const int32_t* kv_lens, const int32_t* block_table,
                   void* workspace, size_t ws_bytes, void* stream) {
  t_last_launches = 0;
  int rc = check_paged(p);
  if (rc) return rc;
  if (p->batch == 0 || p->total_q == 0) return SDPA_OK;
  if (!q || !k_cache || !v_cache || !o || !lse || !cu_seqlens_q || !kv_lens || !block_table) return SDPA_ERR_INVALID_ARG;
  for (const void* ptr : {q, k_cache, v_cache, (const void*)o, (const void*)lse})
    if (!aligned16(ptr)) return SDPA_ERR_ALIGNMENT;
  const int d = p->head_dim, dv = paged_dv(p);
  const long long qw = (long long)p->num_heads_q * d, qs = p->q_stride ? p->q_stride : qw;
  if (qs % d) return SDPA_ERR_UNSUPPORTED;  // a copy's strides are multiples of one another
  const PagedPlan pl = paged_plan(p);
  if ((pl.rows.used && !pl.rows.fits) || (pl.chunk.used && !pl.chunk.fits)) return SDPA_ERR_UNSUPPORTED;
  if (!workspace || ws_bytes < pl.total) return SDPA_ERR_WORKSPACE_TOO_SMALL;
  if (reinterpret_cast<uintptr_t>(workspace) & 255u) return SDPA_ERR_ALIGNMENT;
  const long long ts = p->table_stride ? p->table_stride : p->max_pages;
  const Extent outs[3] = {extent(o, (size_t)p->total_q * p->num_heads_q * dv * 2),
                          extent(lse, (size_t)p->total_q * p->num_heads_q * 4), extent(workspace, pl.total)};
  const Extent ins[6] = {extent(q, span(p->total_q, qs, qw)),
                         cache_extent(p, k_view(p, k_cache)), cache_extent(p, v_view(p, v_cache)),
                         extent(cu_seqlens_q, 4 * ((size_t)p->batch + 1)), extent(kv_lens, 4 * (size_t)p->batch),
                         extent(block_table, 4 * (size_t)((p->batch - 1) * ts + p->max_pages))};
  for (int a = 0; a < 3; ++a) {
    for (const Extent& in : ins)
      if (overlaps(outs[a], in)) return SDPA_ERR_OVERLAP;
    for (int b = a + 1; b < 3; ++b)
      if (overlaps(outs[a], outs[b])) return SDPA_ERR_OVERLAP;
  }
  int* err = error_word();
  if (!err) return SDPA_ERR_CUDA;
  auto encode_map = encode_fn();
  if (!encode_map) return SDPA_ERR_CUDA;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return SDPA_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool bf16 = p->dtype == SDPA_BF16;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  AddrTable* chk = bind_extents({outs[0], outs[1], outs[2], ins[0], ins[1], ins[2], ins[3], ins[4], ins[5]}, err, s);
  if (kAddrCheck && !chk) return SDPA_ERR_CUDA;
  int launches = 0;
  // the chunk kernel's length of the rest (at 64) and ticket counter (at 128)
  if (pl.chunk.used && cudaMemsetAsync(ws + 64, 0, 68, s) != cudaSuccess) return SDPA_ERR_CUDA;
  // the chunk kernel starts while the rows kernel and its join still run: each SM turns to it as it gets free
  for (const PagedCutting* c : {&pl.rows, &pl.chunk}) {
    if (!c->used) continue;
    const bool small = c == &pl.rows;
    PagedLaunch L;
    std::memset(&L, 0, sizeof(L));
    PagedParams& P = L.p;
    P = paged_params(p, pl, small, cu_seqlens_q, kv_lens, block_table, o, lse, ws, err, chk);
    // slots one copy brings: within a page and, for the chunk kernel, within a V stage
    P.box_rows = std::min(p->page_size & -p->page_size, small || c->dv_item == 128 ? 128 : 64);
    P.slot_first = slot_first(p);
    const bool pair = !small && d == 128;
    L.workers = std::min(c->workers, sms);
    if (debug_max_ctas() > 0) L.workers = std::min(L.workers, debug_max_ctas());
    L.stream = s;
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)p->num_heads_q, (cuuint64_t)p->total_q};
    const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)qs * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)c->block_heads, (cuuint32_t)c->q_tokens}, estr[3] = {1, 1, 1};
    if (encode_map(&L.tmQ, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                   const_cast<void*>(q), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return SDPA_ERR_CUDA;
    if ((rc = encode_cache(&L.tmK, k_cache, p, d, p->k_page_stride, p->k_slot_stride, p->k_head_stride, P.box_rows, bf16)))
      return rc;
    if ((rc = encode_cache(&L.tmV, v_cache, p, dv, p->v_page_stride, p->v_slot_stride, p->v_head_stride, P.box_rows, bf16)))
      return rc;
    rc = timed(SDPA_KERNEL_PAGED, s, [&] {
      return small  ? launch_paged_rows(L, c->n, d, bf16, &launches)
             : pair ? launch_paged_pair(L, bf16, &launches)
                    : launch_paged_chunk(L, d, bf16, &launches);
    });
    if (rc) return rc;
  }
  t_last_launches = launches;
  return SDPA_OK;
}

size_t sdpa_paged_fwd_fp8_workspace_size(const sdpa_paged_problem* p) {
  if (check_paged(p) != SDPA_OK || p->batch == 0 || p->total_q == 0) return 0;
  return paged_fp8_plan(p).total;
}

int sdpa_paged_fwd_fp8(const sdpa_paged_problem* p, const sdpa_paged_scales* scales, const void* q, const void* k_cache,
                       const void* v_cache, void* o, float* lse, const int32_t* cu_seqlens_q, const int32_t* kv_lens,
                       const int32_t* block_table, void* workspace, size_t ws_bytes, void* stream) {
  t_last_launches = 0;
  int rc = check_paged(p);
  if (rc) return rc;
  if ((rc = check_fp8_cache(p, scales))) return rc;
  if (p->batch == 0 || p->total_q == 0) return SDPA_OK;
  if (!q || !k_cache || !v_cache || !o || !lse || !cu_seqlens_q || !kv_lens || !block_table) return SDPA_ERR_INVALID_ARG;
  for (const void* ptr : {q, k_cache, v_cache, (const void*)o, (const void*)lse})
    if (!aligned16(ptr)) return SDPA_ERR_ALIGNMENT;
  const int d = p->head_dim, dv = paged_dv(p);
  const long long qw = (long long)p->num_heads_q * d, qs = p->q_stride ? p->q_stride : qw;
  const PagedPlan pl = paged_fp8_plan(p);
  if (!pl.rows.fits) return SDPA_ERR_UNSUPPORTED;
  if (!workspace || ws_bytes < pl.total) return SDPA_ERR_WORKSPACE_TOO_SMALL;
  if (reinterpret_cast<uintptr_t>(workspace) & 255u) return SDPA_ERR_ALIGNMENT;
  const Extent outs[3] = {extent(o, (size_t)p->total_q * p->num_heads_q * dv * 2),
                          extent(lse, (size_t)p->total_q * p->num_heads_q * 4), extent(workspace, pl.total)};
  const long long ts = p->table_stride ? p->table_stride : p->max_pages;
  const Extent ins[8] = {extent(q, span(p->total_q, qs, qw)),
                         cache_extent(p, k_view(p, k_cache, 1)), cache_extent(p, v_view(p, v_cache, 1)),
                         cache_extent(p, k_scale_view(scales)), cache_extent(p, v_scale_view(scales)),
                         extent(cu_seqlens_q, 4 * ((size_t)p->batch + 1)), extent(kv_lens, 4 * (size_t)p->batch),
                         extent(block_table, 4 * (size_t)((p->batch - 1) * ts + p->max_pages))};
  for (int a = 0; a < 3; ++a) {
    for (const Extent& in : ins)
      if (overlaps(outs[a], in)) return SDPA_ERR_OVERLAP;
    for (int b = a + 1; b < 3; ++b)
      if (overlaps(outs[a], outs[b])) return SDPA_ERR_OVERLAP;
  }
  int* err = error_word();
  if (!err) return SDPA_ERR_CUDA;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return SDPA_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  AddrTable* chk = bind_extents({outs[0], outs[1], outs[2], ins[0], ins[1], ins[2], ins[3], ins[4], ins[5], ins[6], ins[7]},
                                err, s);
  if (kAddrCheck && !chk) return SDPA_ERR_CUDA;
  PagedFp8Launch L;
  std::memset(&L, 0, sizeof(L));
  L.p.a = paged_params(p, pl, true, cu_seqlens_q, kv_lens, block_table, o, lse, static_cast<uint8_t*>(workspace), err, chk);
  L.p.a.scale_log2 = p->softmax_scale * 1.4426950408889634f;  // 0 may be 0: masked scores never meet it
  L.p.a.box_rows = std::min(p->page_size & -p->page_size, 128);
  L.p.a.slot_first = slot_first(p);
  // An item's own cost, in key tiles: some 2.5 us for its first scores, its end and its output, against 0.8 us for the 32 KB
  // of a tile at head_dim 128 and 3 for the 128 KB at 512. Counted as nothing, the CTAs with many short items ended last. us (a
  // pass a graph) by 0 / 2, 1, 1 / 3, 2, 1 / 4, 3, 2 / 6, 4, 2 tiles at 128, 192 and 256, 512: 64 sequences of 100 to 1000 keys at
  // 128 49.2, 39.5, 37.7, 37.7, 37.5, at 512 45.3, 42.1, 42.1, 42.6, 42.6; 48 sequences, window of 1024, at 256 57.4, 50.4, 47.2,
  // 46.2, 46.7; 9 of up to 5 tokens at 192 34.5, 31.4, 30.3, 29.1, 29.0; 64 of 500 to 16384 keys at 128 all 210 to 211.
  L.p.a.lead = pl.rows.split ? (d == 128 ? 4 : d == 512 ? 1 : 3) : 0;
  L.p.q = q;
  L.p.q_stride = qs;
  L.p.k_scale = scales->k;
  L.p.v_scale = scales->v;
  L.p.ks_page = scales->k_page_stride;
  L.p.ks_slot = scales->k_slot_stride;
  L.p.ks_head = scales->k_head_stride;
  L.p.vs_page = scales->v_page_stride;
  L.p.vs_slot = scales->v_slot_stride;
  L.p.vs_head = scales->v_head_stride;
  if ((rc = encode_codes(&L.tmK, k_cache, p, d, p->k_page_stride, p->k_slot_stride, p->k_head_stride, L.p.a.box_rows)))
    return rc;
  if ((rc = encode_codes(&L.tmV, v_cache, p, dv, p->v_page_stride, p->v_slot_stride, p->v_head_stride, L.p.a.box_rows)))
    return rc;
  L.workers = std::min(pl.rows.workers, sms);
  if (debug_max_ctas() > 0) L.workers = std::min(L.workers, debug_max_ctas());
  L.stream = s;
  int launches = 0;
  rc = timed(SDPA_KERNEL_PAGED, s, [&] { return launch_paged_fp8(L, pl.rows.n, d, p->dtype == SDPA_BF16, &launches); });
  if (rc) return rc;
  t_last_launches = launches;
  return SDPA_OK;
}

int sdpa_get_device_error(void* stream) {
  int* err = error_word();
  if (!err) return SDPA_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cudaStreamSynchronize(s) != cudaSuccess) return SDPA_ERR_CUDA;
  int host = 0;
  if (cudaMemcpyFromSymbol(&host, g_sdpa_error_word, sizeof(int)) != cudaSuccess) return SDPA_ERR_CUDA;
  const int zero = 0;
  if (cudaMemcpyToSymbol(g_sdpa_error_word, &zero, sizeof(int)) != cudaSuccess) return SDPA_ERR_CUDA;
  return host;
}

const char* sdpa_error_string(int status) {
  switch (status) {
    case SDPA_OK: return "ok";
    case SDPA_ERR_INVALID_ARG: return "invalid argument";
    case SDPA_ERR_UNSUPPORTED: return "unsupported problem (dtype, head_dim, layout or mask/window combination)";
    case SDPA_ERR_ALIGNMENT: return "a device pointer is not 16-byte aligned";
    case SDPA_ERR_OVERLAP: return "an output buffer overlaps another buffer";
    case SDPA_ERR_WORKSPACE_TOO_SMALL: return "workspace missing or smaller than the required size";
    case SDPA_ERR_BAD_SEQLENS: return "cu_seqlens rejected by the device-side guard";
    case SDPA_ERR_TIMEOUT: return "a bounded wait inside a kernel gave up";
    case SDPA_ERR_CUDA: return "a CUDA runtime or driver call failed";
    case SDPA_ERR_ADDRESS: return "a kernel access fell outside the call's buffers (address-checked library)";
    case SDPA_ERR_BAD_INDEX: return "a page number or a position lies outside its table";
    default: return "unknown status";
  }
}

int sdpa_last_launch_count(void) { return t_last_launches; }

int sdpa_debug_set_max_ctas(int max_ctas) {
  if (max_ctas < 0) return SDPA_ERR_INVALID_ARG;
  g_max_ctas.store(max_ctas, std::memory_order_relaxed);
  return SDPA_OK;
}

int sdpa_debug_address_report(unsigned long long* violations, unsigned long long* first_addr,
                              unsigned long long* first_bytes) {
#ifdef SDPA_ADDR_CHECK
  AddrTable* t = addr_table();
  if (!t || cudaDeviceSynchronize() != cudaSuccess) return SDPA_ERR_CUDA;
  unsigned long long v[3] = {0, 0, 0};
  uint8_t* counters = reinterpret_cast<uint8_t*>(t) + offsetof(AddrTable, violations);
  if (cudaMemcpy(v, counters, sizeof(v), cudaMemcpyDeviceToHost) != cudaSuccess) return SDPA_ERR_CUDA;
  const unsigned long long zero[3] = {0, 0, 0};
  if (cudaMemcpy(counters, zero, sizeof(zero), cudaMemcpyHostToDevice) != cudaSuccess) return SDPA_ERR_CUDA;
  if (violations) *violations = v[0];
  if (first_addr) *first_addr = v[1];
  if (first_bytes) *first_bytes = v[2];
  return SDPA_OK;
#else
  (void)violations;
  (void)first_addr;
  (void)first_bytes;
  return SDPA_ERR_UNSUPPORTED;
#endif
}

int sdpa_debug_address_shrink(long long bytes) {
#ifdef SDPA_ADDR_CHECK
  if (bytes < 0) return SDPA_ERR_INVALID_ARG;
  g_addr_shrink.store(bytes, std::memory_order_relaxed);
  return SDPA_OK;
#else
  (void)bytes;
  return SDPA_ERR_UNSUPPORTED;
#endif
}

int sdpa_selftest_bounded_wait(unsigned limit_us, void* stream) {
  int* err = error_word();
  if (!err) return SDPA_ERR_CUDA;
  if (limit_us == 0 || limit_us > 1000000u) return SDPA_ERR_INVALID_ARG;
  return launch_wait_selftest((uint64_t)limit_us * 1000ull, err, static_cast<cudaStream_t>(stream));
}

int sdpa_profile_begin(void) {
  t_prof.on = true;
  t_prof.used = 0;
  return SDPA_OK;
}

int sdpa_profile_end(double* ms_by_kind, int* launches_by_kind, int n_kinds) {
  if (n_kinds < 0 || (n_kinds > 0 && (!ms_by_kind || !launches_by_kind))) return SDPA_ERR_INVALID_ARG;
  for (int k = 0; k < n_kinds; ++k) {
    ms_by_kind[k] = 0.0;
    launches_by_kind[k] = 0;
  }
  int rc = SDPA_OK;
  for (size_t i = 0; i < t_prof.used; ++i) {
    const Profiler::Mark& m = t_prof.marks[i];
    float ms = 0.f;
    if (cudaEventSynchronize(m.b) != cudaSuccess || cudaEventElapsedTime(&ms, m.a, m.b) != cudaSuccess) {
      rc = SDPA_ERR_CUDA;
      continue;
    }
    if (m.kind < n_kinds) {
      ms_by_kind[m.kind] += ms;
      launches_by_kind[m.kind] += 1;
    }
  }
  t_prof.on = false;
  t_prof.used = 0;
  return rc;
}

}  // extern "C"
