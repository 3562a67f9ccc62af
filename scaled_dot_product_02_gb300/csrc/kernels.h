// kernels.h -- parameter blocks and launchers shared between the C-ABI layer
// (api.cu) and the kernel translation units.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include "common.cuh"

namespace sdpa {

// Testing aid (sdpa_debug_set_max_ctas): the most CTAs a kernel may have in
// one launch, 0 = no cap.
int debug_max_ctas();

// Launch `total` CTAs as one grid, or, under a CTA cap, as successive grids of
// at most that many CTAs: fn(offset, count) launches CTAs [offset,
// offset + count) of the index space (kernels add their params' item_offset
// to blockIdx.x). Returns the first failing status.
template <class F>
int launch_in_grids(long long total, F&& fn) {
  const long long cap = debug_max_ctas();
  if (cap <= 0 || total <= cap) return total > 0 ? fn(0LL, total) : 0;
  for (long long off = 0; off < total; off += cap) {
    const int rc = fn(off, total - off < cap ? total - off : cap);
    if (rc) return rc;
  }
  return 0;
}

// Launch a kernel; early = true lets it start while the kernel before it in the
// stream still runs (once all of that one's CTAs have allowed it or ended). It
// may not touch what that kernel writes before griddepcontrol.wait, and must
// execute that wait before it ends, so that its own end implies the other's.
template <class... P, class... A>
int launch_early(void (*kern)(P...), dim3 grid, int threads, int smem, cudaStream_t s, bool early, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = early ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, P(args)...) == cudaSuccess ? SDPA_OK : SDPA_ERR_CUDA;
}

// Raise a kernel's dynamic shared-memory limit to `bytes` and, when
// carveout >= 0, set its preferred shared-memory carveout (percent), once per
// (kernel, current device): function attributes belong to each device's
// instance of the module, and several host threads may make their first call
// at the same time. Returns an sdpa_status.
int set_kernel_smem(const void* kernel, int bytes, int carveout);
// Device address of a __device__ variable (its host-side stand-in `symbol`)
// on the current device, cached per device for the context it was taken in: a
// context created later (after cudaDeviceReset) looks the address up again.
// nullptr on failure.
void* device_symbol_address(const void* symbol);

struct FwdParams {
  Geom g;
  void* o;
  float* lse;
  int* err;          // sticky per-device error word
  const int* guard;  // per-call metadata-guard result (THD) or nullptr
  int n_q_tiles;     // ceil(seqlen_q / 128)
  int dv_splits;     // 1, or 2 when each CTA owns half of the value columns
  int* tile_counter;  // head_dim 128: ticket counter in the workspace (zeroed per call)
  int total_tiles;    // head_dim 128: tickets (query tiles x heads x batch)
  int item_offset;       // added to blockIdx.x (launches split under a CTA cap)
};

struct FwdLaunch {
  CUtensorMap tmQ, tmK, tmV;
  FwdParams p;
  cudaStream_t stream;
};

int launch_fwd(const FwdLaunch& L, int head_dim, int head_dim_v, bool bf16);

struct BwdParams {
  Geom g;
  float* dq_acc;         // [nh_q][rows_q][D] fp32, zeroed by the preprocess kernel
  const float* lse2;     // [nh_q][stat_rows] -LSE * log2(e) (-inf for rows without keys)
  const float* delta;    // [nh_q][stat_rows] rowsum(dO * O)
  int stat_rows;         // padded row count of lse2/delta (>= rows_q + 64, multiple of 4)
  void* dk;
  void* dv;
  int* err;
  const int* guard;
  int n_kv_tiles;        // ceil(seqlen_kv / 128)
  int d_lo, d_hi;        // dK/dV columns this launch owns (all of D for head_dim 128)
  int item_offset;       // added to blockIdx.x (launches split under a CTA cap)
  const int* order;      // THD: sequence indices, longest first (written by the guard); else null
  int head_block;        // kv heads whose key tiles interleave in the grid (divides hkv)
};

struct BwdLaunch {
  CUtensorMap tmQ, tmK, tmV, tmDO;
  BwdParams p;
  cudaStream_t stream;
};

// with_dq = false: dK and dV only (the deterministic backward forms dQ with
// launch_dq128 instead of fp32 reductions).
int launch_bwd_dkdv(const BwdLaunch& L, int head_dim, bool bf16, bool with_dq, int* launches);

// Deterministic head_dim 128 dQ (bwd_dq.cu): per query tile, key tiles in a
// fixed order, dQ accumulated in TMEM and written once.
struct DqParams {
  Geom g;
  void* dq;             // written (dtype, scaled)
  const float* nlse2;   // [nh_q][stat_rows] -LSE * log2(e)
  const float* delta;   // [nh_q][stat_rows]
  int stat_rows;
  int* err;
  const int* guard;
  int n_q_tiles;
  int item_offset;       // added to blockIdx.x (launches split under a CTA cap)
};
struct DqLaunch {
  CUtensorMap tmQ, tmDO, tmK, tmV;  // 128-row boxes
  DqParams p;
  cudaStream_t stream;
};
int launch_dq128(const DqLaunch& L, bool bf16);

// head_dim 256/512 backward (bwd_big.cu): score kernels write 16-bit P and
// dS tiles, GEMM kernels form dQ, dV, dK from them.
struct BigBwdParams {
  Geom g;
  uint8_t* p_tiles;      // [B][Hq][n_q_tiles][slots] 32 KB tile images of one key-tile chunk
  uint8_t* ds_tiles;     // same shape
  const float* nlse2;    // [nh_q][stat_rows] -LSE * log2(e)
  const float* delta;    // [nh_q][stat_rows]
  int stat_rows;
  void* dq;
  void* dk;
  void* dv;
  int* err;
  const int* guard;
  int n_q_tiles, n_kv_tiles, slots;
  int chunk_lo, chunk_hi;  // key tiles [chunk_lo, chunk_hi) of this launch set
  int chunk;               // key tiles per chunk (the last chunk may be shorter)
  float* dq_acc;           // [nh_q][rows_q][D] fp32 dQ sum over chunks, zeroed by the
                           // preprocess; nullptr when one chunk covers every key tile
  int item_offset;       // added to blockIdx.x (launches split under a CTA cap)
  int block_major;       // phase-2 grid by (batch, kv head) block (bounded window) or by mode
};

struct BigBwdLaunch {
  CUtensorMap tmQ, tmK, tmV, tmDO;    // 128-row boxes
  CUtensorMap tmQ64, tmK64, tmDO64;    // 64-row boxes
  BigBwdParams p;
  cudaStream_t stream;
};

int launch_bwd_big(const BigBwdLaunch& L, int head_dim, bool bf16, int* launches);

// FP8 E4M3 forward, head_dim 128 (fwd_fp8.cu): vt_kernel writes V transposed
// into the workspace, fwd_fp8_kernel computes O and LSE.
struct Fp8Params {
  Geom g;               // scale / scale_log2 include the Q and K descales
  const uint8_t* v;     // E4M3 V [rows_kv][nh_kv][128]
  uint8_t* vt;          // transposed V [nh_kv][128][vt_rows] (workspace)
  int vt_rows;          // keys of Vt per (head, d): every sequence 16-aligned, gaps zero
  void* o;              // [rows_q][nh_q][128], bf16 or fp16
  float* lse;
  int* err;
  const int* guard;
  int n_q_tiles;
  float o_scale;        // d_v / 448 (the epilogue divides by the row sum as well)
  int total_tiles;      // query tiles of the order (tickets of the persistent forward)
  int* tile_counter;    // ticket counter in the workspace (zeroed per call)
};
struct Fp8Launch {
  CUtensorMap tmQ, tmK, tmVt;  // E4M3 128-byte rows, 128-row boxes; Vt 128 keys x 128 d boxes
  Fp8Params p;
  cudaStream_t stream;
};
int launch_vt(const Fp8Params& p, cudaStream_t stream);
int launch_fwd_fp8(const Fp8Launch& L, bool bf16);

// Memory-bound helpers (aux.cu).
struct PrepParams {
  Geom g;
  const void* o;
  const void* dout;
  const float* lse;
  float* lse2;
  float* delta;
  int stat_rows;
  float* dq_acc;  // zeroed here when non-null
  const int* guard;
};
// order (THD backward, else null): receives the sequence indices, longest first
int launch_guard(const Geom& g, int total_q, int total_kv, int* guard, int* err, cudaStream_t s,
                 int* order = nullptr);
int launch_preprocess(const PrepParams& pp, bool bf16, cudaStream_t s);
int launch_wait_selftest(uint64_t limit_ns, int* err, cudaStream_t s);
int launch_dq_finalize(const Geom& g, const float* dq_acc, void* dq, const int* guard, bool bf16, cudaStream_t s);

// Rotation with several positions a token: pair i turns by the angle of axis a's
// position, for the a with end[a - 1] <= i < end[a].
struct RopeAxes {
  int n;                       // axes; 0: one position a token
  int end[4];                  // behind the last pair of each axis (INT_MAX for the last and what follows)
  long long pos_stride;        // elements between the axes' positions
  // A token's angles as staged in shared memory: of each axis the pairs [lo, lo + len), whole blocks of 4, cosines
  // then sines; pair i's at cos_at + i and sin_at + i of floats in all.
  int lo[4], len[4], cos_at[4], sin_at[4], floats;
};

// Per-head norm + rotation, and the append to a paged cache (norm_rope.cu).
struct NormRopeParams {
  long long rows;              // tokens
  int hq, hkv;                 // heads of q (0: none given) and of k (and v)
  int rot;                     // leading values rotated (0: none)
  int interleaved;
  float eps;
  const void *q, *k, *v;       // v: append only
  long long qs, ks, vs;        // elements between tokens
  const void *wq, *wk;         // nullptr: rows are copied as they are (append)
  const float* table;          // [max_pos][rot]
  int max_pos;
  const int32_t* pos;          // [rows] of each axis; nullptr: cache positions (append)
  RopeAxes axes;
  void *q_out, *k_out;         // contiguous (k_out: not for the append)
  int parts, parts_q, parts_k;  // warps that share one token, its q heads, its k (and v) heads
  int stage_bytes, stages;     // a warp's ring in shared memory (many tokens)
  // append: the batch and the cache
  int batch, max_pages, num_pages, page_size;
  const int32_t *cu_q, *kv_lens, *table_ids;
  long long table_stride;
  void *kc, *vc;
  long long kc_page, kc_slot, kc_head, vc_page, vc_slot, vc_head;
  uint8_t *k_scale, *v_scale;  // scale bytes of a cache of E4M3 codes; nullptr: a 16-bit cache
  long long ks_page, ks_slot, ks_head, vs_page, vs_slot, vs_head;
  int* err;
  AddrTable* chk;
};
int launch_norm_rope(NormRopeParams p, int head_dim, bool bf16, bool append, cudaStream_t s);

struct NormRopeBwdParams {
  long long rows;
  int hq, hkv, rot, interleaved;
  float eps;
  const void *gq, *gk;         // gradients of the outputs, contiguous
  const void *q, *k;
  long long qs, ks;
  const void *wq, *wk;
  const float* table;
  int max_pos;
  const int32_t* pos;
  RopeAxes axes;
  void *dq, *dk;
  long long dqs, dks;
  float* part;                 // [blocks + 1][D] partial sums of dw
  float *dwq, *dwk;
  int warps_q, blocks;         // warps that serve q (the others k), all blocks
  int stage_bytes, stages;     // a warp's ring in shared memory
  int* err;
  AddrTable* chk;
};
// How the backward is cut: a function of the problem alone, so the order of the
// sums of dw is fixed.
struct NormRopeBwdPlan {
  int warps_q, blocks;
};
NormRopeBwdPlan norm_rope_bwd_plan(long long rows, int hq, int hkv, int head_dim);
int launch_norm_rope_bwd(const NormRopeBwdParams& p, int head_dim, bool bf16, int* launches, cudaStream_t s);

// The last keys and values of every sequence of an 8-bit paged cache as packed 16-bit rows (paged_read.cu).
struct PagedReadParams {
  long long rows;              // of k_out and v_out
  int batch, hkv, page_size, num_pages, max_pages;
  const uint8_t *k_cache, *v_cache, *k_scale, *v_scale;
  long long k_page, k_slot, k_head, v_page, v_slot, v_head;
  long long ks_page, ks_slot, ks_head, vs_page, vs_slot, vs_head;
  void *k_out, *v_out;
  long long k_row, v_row;      // elements between their rows
  const int32_t *cu, *kv_lens, *block_table;
  long long table_stride;
  int* err;
  AddrTable* chk;
};
int launch_paged_read(const PagedReadParams& p, int head_dim, bool bf16, cudaStream_t s);

// Attention over a paged cache: paged.cu serves sequences with few query rows,
// paged_pair.cu (head_dim 128) and paged_chunk.cu the others.
struct PagedCut;  // a worker's record for the join, in the workspace
struct PagedParams {
  int batch, total_q, max_q, max_kv;
  int hq, group;               // heads of q, and of q per kv head
  int block_heads, head_blocks;  // heads of a group in one item, items a group takes
  int tokens;                  // tokens in one item
  int dv, dv_splits;           // width of O rows; parts of it that separate items accumulate
  int units_per_block;         // items of one block of tokens: kv heads x head_blocks x dv_splits
  int small_q, small;          // this launch serves the sequences of at most small_q tokens (small), or the others
  int split;                   // rows kernel: items may be split over workers
  int lead;                    // and an item counts for that many key tiles more than it has
  int tail;                    // chunk kernels: shares that the last items are cut into (0: none)
  int behind;                  // started while the rows kernel of the same call (and its join) still run
  int q_box_rows;              // rows one Q copy brings (half of an item's at head_dim 128 chunks)
  int causal, window;          // window < 0: none
  float scale_log2;
  int page_size, num_pages, box_rows;  // box_rows: slots one copy brings (divides page_size and 128)
  int slot_first;              // cache order [page][head][slot]: slots vary before heads
  const int32_t *cu_q, *kv_lens, *block_table;
  long long table_stride;
  void* o;
  float* lse;
  long long* total_tiles;      // workspace: length of what the shares cut (0: refused, or nothing)
  int* tickets;                // workspace: the next item or share (chunk kernels)
  PagedCut* cuts;              // [shares]
  float* parts;                // [shares][2] partial results
  int* err;
  AddrTable* chk;
};
struct PagedLaunch {
  CUtensorMap tmQ, tmK, tmV;
  PagedParams p;
  int workers;                 // CTAs
  cudaStream_t stream;
};
size_t paged_cut_bytes();
// n: rows of an item, 16, 32 or 64 (64 not with head_dim 512)
int launch_paged_rows(const PagedLaunch& L, int n, int head_dim, bool bf16, int* launches);
// Items of 128 rows, head dims 192 to 512.
int launch_paged_chunk(const PagedLaunch& L, int head_dim, bool bf16, int* launches);
// Items of 256 rows, head_dim 128.
int launch_paged_pair(const PagedLaunch& L, bool bf16, int* launches);
// Joins the items that cross a cut between `shares` shares: n rows of dv values an item.
int launch_paged_join(const PagedLaunch& L, int n, int dv, int shares, bool bf16);

// Attention over a paged cache of E4M3 codes with a scale byte a row (paged_fp8.cu).
struct PagedFp8Params {
  PagedParams a;
  const void* q;
  long long q_stride;          // elements between tokens
  const uint8_t *k_scale, *v_scale;
  long long ks_page, ks_slot, ks_head, vs_page, vs_slot, vs_head;
};
struct PagedFp8Launch {
  CUtensorMap tmK, tmV;        // codes: 128 columns x box_rows slots
  PagedFp8Params p;
  int workers;                 // CTAs
  cudaStream_t stream;
};
int launch_paged_fp8(const PagedFp8Launch& L, int n, int head_dim, bool bf16, int* launches);

// Log-sum-exp merge of partial results over a split of the keys (merge.cu).
int launch_merge(const void* o_parts, const float* lse_parts, void* o, float* lse, long long items, int head_dim,
                 int n_parts, bool bf16, AddrTable* chk, cudaStream_t s);

}  // namespace sdpa
