// C-ABI entry points (include/pa.h): argument validation, workspace layout,
// TMA descriptor encoding and kernel launches. Host code only; every step of
// the computation runs in the kernels of the other translation units.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <cmath>
#include <cstring>
#include <mutex>

#include "pa.h"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kAbiVersion = 1;
constexpr size_t kAlign = 256;
// Positions, keys and rows of one call that the operators around attention
// count in 32 bits, with room for a step past the end.
constexpr int kMaxKeys = 1 << 30;

inline size_t align_up(size_t x, size_t a = kAlign) { return (x + a - 1) / a * a; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline int cdiv(long long a, long long b) { return static_cast<int>((a + b - 1) / b); }

// Split targets (work items per KV head) per kernel class, from the SM count:
// the split-KV kernel runs 2 CTAs per SM and aims at ~2 waves; the prefill
// kernel runs 1 CTA per SM.
inline int target_split(int sms, int H_kv) { return cdiv(4LL * sms, H_kv); }
inline int target_tc(int sms, int H_kv) { return cdiv(1LL * sms, H_kv); }

// Segments with more than kRowsSplit packed query rows go to the tcgen05
// prefill kernel; the rest to the split-KV kernel.
constexpr bool kTcAvailable = true;

struct PassDims {
  int num_segs;   // segments planned
  int total_q;
  int max_q;      // host bound of a segment's query length
  bool single;    // one segment of total_q queries (cascade prefix pass)
  int G, H, H_kv, D;
  int sms;
  bool all_partial = false;   // every item keeps a partial-state slot (cascade prefix pass)
  bool kv_fp8 = false;        // FP8 pools (head size 128; the prefill kernel widens them)
  // The prefill kernel takes the row maximum of the raw scores and scales it
  // afterwards, which needs softmax_scale > 0; a zero or negative scale runs
  // every segment on the split-KV kernel (which scales before the maximum).
  bool tc_allowed = true;
  int max_kv = 0x7fffffff;    // host bound of a segment's key count
};

// Which kernels a pass can need, from host-known bounds only.
// Packed rows above which a segment takes the prefill kernel: every segment
// at head sizes the split-KV kernel does not take.
int tc_min_rows(int D) { return D > kMaxHeadSplit ? 0 : kTcMinRows; }
bool pass_has_tc(const PassDims& d) {
  const long long rows = static_cast<long long>(d.single ? d.total_q : d.max_q) * d.G;
  return kTcAvailable && d.tc_allowed && tc_tile_rows(d.G) > 0 && rows > tc_min_rows(d.D);
}
bool pass_has_split(const PassDims& d) {
  return d.D <= kMaxHeadSplit && (!d.single || !pass_has_tc(d));
}

// Workspace layout of one pass starting at byte offset `base`.
PassLayout layout_pass(const PassDims& d, size_t base) {
  PassLayout L{};
  const bool tc = pass_has_tc(d), sp = pass_has_split(d);
  L.target[0] = sp ? target_split(d.sms, d.H_kv) : 0;
  L.target[1] = tc ? target_tc(d.sms, d.H_kv) : 0;
  const long long rows = static_cast<long long>(d.total_q) * d.G;
  L.items_bound[0] = sp ? L.target[0] + d.num_segs + cdiv(rows, kRowsSplit) + 1 : 0;
  L.items_bound[1] = tc ? L.target[1] + d.num_segs + cdiv(rows, tc_item_rows(d.G, d.D)) + 1 : 0;
  // A second bound from the key lengths: a segment splits into at most
  // ceil(max_kv / smallest chunk) items per row tile. Where the keys are
  // short (decode suffixes of a cascade, a prefix of a few thousand keys) it
  // is far below the first, so the launches carry fewer blocks that find no
  // item and return (blocks are dispatched in index order, and a dependent
  // launch starts only once every block of its predecessor has started).
  auto by_keys = [&](int rpi, int min_chunk) {
    const long long seg_rows = static_cast<long long>(d.single ? d.total_q : d.max_q) * d.G;
    long long nrt = static_cast<long long>(d.num_segs) * cdiv(seg_rows, rpi);
    const long long nrt2 = d.num_segs + static_cast<long long>(cdiv(rows, rpi));
    if (nrt2 < nrt) nrt = nrt2;
    const long long nsp = d.max_kv > 0 ? cdiv(d.max_kv, min_chunk) : 1;
    const long long b = nrt * nsp;
    return static_cast<int>(b < 1 ? 1 : (b > 0x7fffffffLL ? 0x7fffffffLL : b));
  };
  if (sp && by_keys(kRowsSplit, kMinChunkSplit) < L.items_bound[0])
    L.items_bound[0] = by_keys(kRowsSplit, kMinChunkSplit);
  if (tc && by_keys(tc_item_rows(d.G, d.D), kMinChunkTc) < L.items_bound[1])
    L.items_bound[1] = by_keys(tc_item_rows(d.G, d.D), kMinChunkTc);
  L.slots_bound[0] = sp ? 2 * L.target[0] + 2 : 0;
  L.slots_bound[1] = tc ? 2 * L.target[1] + 2 : 0;
  if (d.all_partial) {
    L.slots_bound[0] = L.items_bound[0];
    L.slots_bound[1] = L.items_bound[1];
  }
  // A work item holds at most min(rows per item of its kernel, q_len * G) rows.
  const long long rows_bound = static_cast<long long>(d.single ? d.total_q : d.max_q) * d.G;
  auto clamp_rows = [&](int item_rows) {
    return static_cast<int>(rows_bound < item_rows ? (rows_bound > 0 ? rows_bound : 1)
                                                   : item_rows);
  };
  L.slot_rows[0] = clamp_rows(kRowsSplit);
  L.slot_rows[1] = clamp_rows(tc ? tc_item_rows(d.G, d.D) : 1);
  size_t off = align_up(base);
  L.header = off;                 off = align_up(off + 64 * sizeof(int));
  L.seg = off;                    off = align_up(off + static_cast<size_t>(d.num_segs) * 16);
  L.segsplit = off;               off = align_up(off + static_cast<size_t>(d.num_segs) * 16);
  L.items[0] = off;               off = align_up(off + static_cast<size_t>(L.items_bound[0]) * 16);
  L.items[1] = off;               off = align_up(off + static_cast<size_t>(L.items_bound[1]) * 16);
  L.groups[0] = off;              off = align_up(off + static_cast<size_t>(d.all_partial ? L.items_bound[0] : 0) * 16);
  L.groups[1] = off;              off = align_up(off + static_cast<size_t>(d.all_partial ? L.items_bound[1] : 0) * 16);
  for (int c = 0; c < 2; ++c) {
    const size_t slot_rows = static_cast<size_t>(L.slots_bound[c]) * d.H_kv * L.slot_rows[c];
    L.counters[c] = off;          off = align_up(off + static_cast<size_t>(L.slots_bound[c]) * d.H_kv * 4);
    L.part_lse[c] = off;          off = align_up(off + slot_rows * 4);
    L.part_o[c] = off;            off = align_up(off + slot_rows * d.D * 4);
  }
  L.end = off;
  return L;
}

struct CascadeLayout {
  PassLayout prefix, suffix;
  size_t end;
};

// prefix_len < 0 (the size queries, which do not take it): the bound of
// either pass's keys is max_k, which covers every prefix length.
CascadeLayout layout_cascade(int num_seqs, int total_q, int max_q, int max_k, int prefix_len,
                             int G, int H, int H_kv, int D, int sms, bool kv_fp8,
                             bool tc_allowed) {
  CascadeLayout C{};
  PassDims pd{1, total_q, total_q, true, G, H, H_kv, D, sms, true, kv_fp8, tc_allowed};
  pd.max_kv = prefix_len < 0 ? max_k : prefix_len;
  C.prefix = layout_pass(pd, 0);
  PassDims sd{num_seqs, total_q, max_q, false, G, H, H_kv, D, sms, true, kv_fp8, tc_allowed};
  sd.max_kv = prefix_len < 0 ? max_k : (max_k > prefix_len ? max_k - prefix_len : 0);
  C.suffix = layout_pass(sd, C.prefix.end);
  C.end = C.suffix.end;
  return C;
}

// Workspace bytes reported by the size queries: enough for either kernel
// choice (the choice also depends on the sign of softmax_scale, which the
// queries do not take).
size_t varlen_bytes(PassDims d) {
  d.tc_allowed = true;
  const size_t a = layout_pass(d, 0).end;
  d.tc_allowed = false;
  const size_t b = layout_pass(d, 0).end;
  return a > b ? a : b;
}
size_t cascade_bytes(int num_seqs, int total_q, int max_q, int max_k, int G, int H, int H_kv,
                     int D, int sms, bool kv_fp8) {
  const size_t a =
      layout_cascade(num_seqs, total_q, max_q, max_k, -1, G, H, H_kv, D, sms, kv_fp8, true).end;
  const size_t b =
      layout_cascade(num_seqs, total_q, max_q, max_k, -1, G, H, H_kv, D, sms, kv_fp8, false).end;
  return a > b ? a : b;
}

// The count of a device does not change: asked once per device.
int query_sms(int sm_count) {
  static std::atomic<int> known[kMaxDevices];
  if (sm_count > 0) return sm_count;
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  const bool cached = dev >= 0 && dev < kMaxDevices;
  if (cached && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (cached) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

// Checks shared by the attention entry points that need no device pointer.
pa_status check_shape(int num_seqs, int total_q, int max_seqlen_q, int max_seqlen_k, int H,
                      int H_kv, int D, int bs, int dtype) {
  if (num_seqs < 0 || total_q < 0 || max_seqlen_q < 0 || max_seqlen_k < 0) return PA_ERR_INVALID_ARG;
  if (H <= 0 || H_kv <= 0 || H % H_kv != 0) return PA_ERR_INVALID_ARG;
  if (dtype != PA_BF16 && dtype != PA_F16) return PA_ERR_UNSUPPORTED;
  if (D != 64 && D != 128 && D != 256) return PA_ERR_UNSUPPORTED;
  if (bs <= 0 || bs % 16 != 0 || bs > 1024) return PA_ERR_BLOCK_SIZE;
  return PA_OK;
}

// Element type of the K/V pools: bf16, e4m3 codes with per-KV-head scales, or
// 4-bit codes with a scale and a minimum per row.
struct KvFormat {
  bool fp8;
  const float* k_scale;
  const float* v_scale;
  bool int4 = false;
  uint32_t* k_params = nullptr;
  uint32_t* v_params = nullptr;
  int64_t params_stride = 0;
};
constexpr KvFormat kKvBf16{false, nullptr, nullptr};

KvFormat int4_format(const pa_kv_int4* p) {
  KvFormat f{false, nullptr, nullptr, true};
  if (p) {
    f.k_params = static_cast<uint32_t*>(p->k_params);
    f.v_params = static_cast<uint32_t*>(p->v_params);
    f.params_stride = p->params_block_stride;
  }
  return f;
}

// Checks of a 4-bit cache.
pa_status check_int4(const KvFormat& kv, const void* kc, const void* vc, int64_t block_stride,
                     int H_kv, int D, int bs) {
  if (D != 64 && D != 128) return PA_ERR_UNSUPPORTED;
  if (!kc || !vc || !aligned16(kc) || !aligned16(vc) || !kv.k_params || !kv.v_params)
    return PA_ERR_INVALID_ARG;
  if (!aligned16(kv.k_params) || !aligned16(kv.v_params)) return PA_ERR_INVALID_ARG;
  if (block_stride < static_cast<int64_t>(bs) * H_kv * (D / 2) || block_stride % 16 != 0 ||
      kv.params_stride < static_cast<int64_t>(bs) * H_kv || kv.params_stride % 4 != 0)
    return PA_ERR_INVALID_ARG;
  return PA_OK;
}

pa_status check_attn_ptrs(const void* q, int64_t q_stride, const void* kc, const void* vc,
                          int64_t block_stride, const int32_t* cu, const int32_t* lens,
                          const int32_t* bt, int bt_stride, int num_seqs, int total_q,
                          int num_blocks, int H, int H_kv, int D, int bs, float scale, int causal,
                          const void* out, const float* lse, const KvFormat& kv) {
  if (num_seqs > 0 && (!cu || !lens || !bt)) return PA_ERR_INVALID_ARG;
  if (total_q > 0 && (!q || !out)) return PA_ERR_INVALID_ARG;
  if (!kc || !vc) return PA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(kc) || !aligned16(vc) || !aligned16(out)) return PA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(lse) & 3u) != 0) return PA_ERR_INVALID_ARG;
  if (q_stride < static_cast<int64_t>(H) * D || q_stride % 8 != 0) return PA_ERR_INVALID_ARG;
  if (kv.int4) {
    const pa_status st = check_int4(kv, kc, vc, block_stride, H_kv, D, bs);
    if (st != PA_OK) return st;
  } else
  // Page strides are whole 16-byte units (a TMA rule): 8 bf16 or 16 e4m3 elements.
  if (block_stride < static_cast<int64_t>(bs) * H_kv * D || block_stride % (kv.fp8 ? 16 : 8) != 0)
    return PA_ERR_INVALID_ARG;
  if (kv.fp8) {
    if (D != 128) return PA_ERR_UNSUPPORTED;
    if (!kv.k_scale || !kv.v_scale) return PA_ERR_INVALID_ARG;
    if (((reinterpret_cast<uintptr_t>(kv.k_scale) | reinterpret_cast<uintptr_t>(kv.v_scale)) & 3u) != 0)
      return PA_ERR_INVALID_ARG;
  }
  if (bt_stride < 0 || num_blocks < 0) return PA_ERR_INVALID_ARG;
  if (!std::isfinite(scale)) return PA_ERR_INVALID_ARG;
  // Head size 256 runs on the prefill kernel only, which needs a positive
  // scale and groups of at most 128 heads.
  if (D > kMaxHeadSplit && (!(scale > 0.f) || tc_tile_rows(H / H_kv) == 0))
    return PA_ERR_UNSUPPORTED;
  if (causal != 0 && causal != 1) return PA_ERR_INVALID_ARG;
  return PA_OK;
}

// cuTensorMapEncodeTiled through the runtime's driver entry point (no link
// dependency on libcuda).
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// 4-D view of a page pool: (dim, kv head, row in page, page), 128-byte
// swizzled boxes of 128 bytes of dims (64 bf16 or 128 e4m3) x 1 head x
// box_rows rows x 1 page. Coordinates past the pool (a page id == num_blocks)
// read as zeros.
bool encode_pool_map(CUtensorMap* map, const void* base, int D, int H_kv, int bs, int num_blocks,
                     int64_t block_stride, int box_rows, bool fp8, bool f16) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t esz = fp8 ? 1 : 2;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(H_kv),
                        static_cast<cuuint64_t>(bs),
                        static_cast<cuuint64_t>(num_blocks > 0 ? num_blocks : 1)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(D) * esz,
                           static_cast<cuuint64_t>(H_kv) * D * esz,
                           static_cast<cuuint64_t>(block_stride) * esz};
  cuuint32_t box[4] = {static_cast<cuuint32_t>(128 / esz), 1, static_cast<cuuint32_t>(box_rows),
                       1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUtensorMapDataType ty = fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                : f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                      : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  CUresult r = fn(map, ty, 4,
                  const_cast<void*>(base), dims, strides,
                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

int log2_or_none(int n) {
  for (int b = 0; b < 31; ++b)
    if (n == 1 << b) return b;
  return -1;
}

int gcd_int(int a, int b) {
  while (b) {
    int t = a % b;
    a = b;
    b = t;
  }
  return a;
}

struct CommonAttn {
  const void* q;
  int64_t q_stride;
  const void* kc;
  const void* vc;
  int64_t block_stride;
  const int32_t* cu;
  const int32_t* lens;
  const int32_t* bt;
  int bt_stride, num_seqs, total_q, max_q, max_k, H, H_kv, D, bs, num_blocks;
  float scale;
  int32_t* status;
  cudaStream_t st;
  KvFormat kv;
  const float* sinks;   // [H] or NULL
  int dtype;            // PA_BF16 or PA_F16: q, out and the 2-byte pools
};

PlanArgs make_plan(const CommonAttn& c, uint8_t* ws, const PassLayout& L, int single, int single_kv,
                   int kv_off, int kv_cap, int causal, int check_cascade, int partials_only = 0) {
  PlanArgs p{};
  p.cu_seqlens_q = c.cu;
  p.seqused_k = c.lens;
  p.num_segs = c.num_seqs;
  p.single_segment = single;
  p.total_q = c.total_q;
  p.single_kv_len = single_kv;
  p.kv_len_offset = kv_off;
  p.kv_len_cap = kv_cap;
  p.max_q = c.max_q;
  p.max_k = c.max_k;
  p.G = c.H / c.H_kv;
  p.H_kv = c.H_kv;
  p.D = c.D;
  p.tc_enabled = L.items_bound[1] > 0 ? 1 : 0;
  p.tc_min_rows = tc_min_rows(c.D);
  p.min_chunk_tc = kMinChunkTc;
  p.causal = causal;
  p.target0 = L.target[0];
  p.target1 = L.target[1];
  p.items_bound0 = L.items_bound[0];
  p.items_bound1 = L.items_bound[1];
  p.slots_bound0 = L.slots_bound[0];
  p.slots_bound1 = L.slots_bound[1];
  p.ws = ws;
  p.L = L;
  p.status = c.status;
  p.check_cascade = check_cascade;
  p.partials_only = partials_only;
  return p;
}

AttnArgs make_attn(const CommonAttn& c, uint8_t* ws, const PassLayout& L, int bt_row_stride,
                   int bt_col_offset, int causal, void* out, float* lse) {
  AttnArgs a{};
  a.q = static_cast<const uint16_t*>(c.q);
  a.q_stride = c.q_stride;
  a.bt = c.bt;
  a.bt_row_stride = bt_row_stride;
  a.bt_col_offset = bt_col_offset;
  a.H = c.H;
  a.H_kv = c.H_kv;
  a.G = c.H / c.H_kv;
  a.D = c.D;
  a.bs = c.bs;
  // (The coordinate of pages outside the pool, too; a map has one page at least, so a
  // pool of none takes one in front of it.)
  a.num_blocks = c.num_blocks > 0 ? c.num_blocks : -1;
  a.scale_log2 = c.scale * 1.4426950408889634f;
  a.causal = causal;
  a.out = static_cast<uint16_t*>(out);
  a.f16 = c.dtype == PA_F16 ? 1 : 0;
  a.lse = lse;
  a.lse_stride = c.total_q;
  a.header = reinterpret_cast<const int*>(ws + L.header);
  a.abort_all = reinterpret_cast<int*>(ws + L.header) + 2;
  a.seg = reinterpret_cast<const int4*>(ws + L.seg);
  a.segsplit = reinterpret_cast<const int4*>(ws + L.segsplit);
  a.items = reinterpret_cast<const int4*>(ws + L.items[0]);
  a.status = c.status;
  a.box_rows = gcd_int(c.bs, kKeyTile);
  a.sinks = c.sinks;
  a.kv_fp8 = c.kv.fp8 ? 1 : 0;
  a.k_scale = c.kv.k_scale;
  a.v_scale = c.kv.v_scale;
  return a;
}

// Q viewed as (dim, head, token), boxes of 64 dims x G heads x floor(128/G)
// tokens: exactly the tc_tile_rows(G) packed rows of one prefill Q tile,
// 128-byte swizzled.
bool encode_q_map(CUtensorMap* map, const void* q, int D, int H, int total_q, int64_t q_stride,
                  int G, bool f16) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(H),
                        static_cast<cuuint64_t>(total_q > 0 ? total_q : 1)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(q_stride) * 2};
  // G <= 128 here (wider groups never use the prefill kernel).
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(kTcTileRows / G)};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                  const_cast<void*>(q), dims, strides,
                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// The maps of a 4-bit cache's decode kernel (see Int4Maps).
bool encode_int4_maps(Int4Maps* maps, const KvFormat& kv, const void* kc, const void* vc,
                      int64_t block_stride, int H_kv, int D, int bs, int num_blocks) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t pages = num_blocks > 0 ? num_blocks : 1, row = D / 2;
  const cuuint32_t heads = int4_decode_heads(H_kv), one[4] = {1, 1, 1, 1};
  const cuuint64_t dims[4] = {row, static_cast<cuuint64_t>(bs), static_cast<cuuint64_t>(H_kv),
                              pages};
  const cuuint64_t strides[3] = {H_kv * row, row, static_cast<cuuint64_t>(block_stride)};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(row), 16, heads, 1};
  const cuuint64_t pdims[3] = {static_cast<cuuint64_t>(bs), static_cast<cuuint64_t>(H_kv), pages};
  const cuuint64_t pstrides[2] = {static_cast<cuuint64_t>(bs) * 4,
                                  static_cast<cuuint64_t>(kv.params_stride) * 4};
  const cuuint32_t pbox[3] = {16, heads, 1};
  const void* codes[2] = {kc, vc};
  void* params[2] = {kv.k_params, kv.v_params};
  for (int x = 0; x < 2; ++x) {
    if (fn(&maps->m[x], CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(codes[x]), dims,
           strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
           D == 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return false;
    if (fn(&maps->m[2 + x], CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, params[x], pdims, pstrides, pbox,
           one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return false;
  }
  return true;
}

// Point a kernel's arguments at its class's work list and partial-slot pool.
void set_class(AttnArgs& a, uint8_t* ws, const PassLayout& L, int c) {
  a.items = reinterpret_cast<const int4*>(ws + L.items[c]);
  a.groups = reinterpret_cast<const int4*>(ws + L.groups[c]);
  a.counters = reinterpret_cast<int*>(ws + L.counters[c]);
  a.part_lse = reinterpret_cast<float*>(ws + L.part_lse[c]);
  a.part_o = reinterpret_cast<float*>(ws + L.part_o[c]);
  a.slot_rows = L.slot_rows[c];
}

// Launch the kernels of one pass. *first is set while no attention kernel of
// the call has been launched since the planner; that kernel waits for the
// plan in every block (see AttnArgs::pdl_first).
pa_status launch_pass(const CommonAttn& c, const CUtensorMap& tmK, const CUtensorMap& tmV,
                      const CUtensorMap& tmQ, const AttnArgs& a, uint8_t* ws,
                      const PassLayout& L, bool* first) {
  if (L.items_bound[1] > 0) {
    AttnArgs a1 = a;
    set_class(a1, ws, L, 1);
    a1.pdl_first = *first ? 1 : 0;
    *first = false;
    if (launch_attn_tc(tmK, tmV, tmQ, a1, L.items_bound[1], c.st) != cudaSuccess)
      return PA_ERR_CUDA;
  }
  if (L.items_bound[0] > 0) {
    AttnArgs a0 = a;
    set_class(a0, ws, L, 0);
    a0.pdl_first = *first ? 1 : 0;
    *first = false;
    if (launch_attn_split(tmK, tmV, a0, L.items_bound[0], c.st) != cudaSuccess)
      return PA_ERR_CUDA;
  }
  return PA_OK;
}

// Checks of pa_reshape_and_cache's arguments (nothing launched).
pa_status check_update(const void* key, const void* value, int64_t key_token_stride,
                       int64_t value_token_stride, const void* key_cache, const void* value_cache,
                       int64_t cache_block_stride, const int64_t* slot_mapping, int num_tokens,
                       int num_kv_heads, int head_size, int block_size, int num_blocks,
                       int dtype, const KvFormat& kv = kKvBf16) {
  if (num_tokens < 0 || num_kv_heads <= 0 || num_blocks < 0) return PA_ERR_INVALID_ARG;
  if (dtype != PA_BF16 && dtype != PA_F16) return PA_ERR_UNSUPPORTED;
  if (head_size != 64 && head_size != 128 && head_size != 256) return PA_ERR_UNSUPPORTED;
  if (kv.fp8 && head_size != 128) return PA_ERR_UNSUPPORTED;
  if (kv.int4 && head_size != 64 && head_size != 128) return PA_ERR_UNSUPPORTED;
  if (block_size <= 0 || block_size % 16 != 0 || block_size > 1024) return PA_ERR_BLOCK_SIZE;
  if (num_tokens == 0) return PA_OK;
  if (kv.fp8 && (!kv.k_scale || !kv.v_scale ||
                 ((reinterpret_cast<uintptr_t>(kv.k_scale) |
                   reinterpret_cast<uintptr_t>(kv.v_scale)) & 3u) != 0))
    return PA_ERR_INVALID_ARG;
  if (!key || !value || !key_cache || !value_cache || !slot_mapping) return PA_ERR_INVALID_ARG;
  if (!aligned16(key) || !aligned16(value) || !aligned16(key_cache) || !aligned16(value_cache))
    return PA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(slot_mapping) & 7u) != 0) return PA_ERR_INVALID_ARG;
  const int64_t row = static_cast<int64_t>(num_kv_heads) * head_size;
  if (key_token_stride < row || value_token_stride < row || key_token_stride % 8 ||
      value_token_stride % 8)
    return PA_ERR_INVALID_ARG;
  if (kv.int4 && row > (1 << 28)) return PA_ERR_INVALID_ARG;   // 32-bit offsets in a token's row
  if (kv.int4)
    return check_int4(kv, key_cache, value_cache, cache_block_stride, num_kv_heads, head_size,
                      block_size);
  if (cache_block_stride < row * block_size || cache_block_stride % (kv.fp8 ? 16 : 8))
    return PA_ERR_INVALID_ARG;
  return PA_OK;
}

// The scatter of pa_reshape_and_cache(_fp8, _int4) for the cache format kv.
cudaError_t launch_scatter(const void* key, const void* value, int64_t kstride, int64_t vstride,
                           void* kc, void* vc, int64_t block_stride, const int64_t* slots,
                           int num_tokens, int H_kv, int D, int bs, int num_blocks,
                           const KvFormat& kv, int32_t* status, cudaStream_t st, int sms,
                           bool pdl, int dtype) {
  if (kv.int4) {   // the rotation's pass, without queries and positions
    RopeArgs a{};
    a.k = static_cast<const uint16_t*>(key);
    a.v = static_cast<const uint16_t*>(value);
    a.k_stride = kstride;
    a.v_stride = vstride;
    a.kc = static_cast<uint8_t*>(kc);
    a.vc = static_cast<uint8_t*>(vc);
    a.block_stride_bytes = block_stride;
    a.slots = slots;
    a.k_params = kv.k_params;
    a.v_params = kv.v_params;
    a.params_stride = kv.params_stride;
    a.num_tokens = num_tokens;
    a.H_kv = H_kv;
    a.bs = bs;
    a.num_slots = static_cast<int64_t>(num_blocks) * bs;
    a.status = status;
    return launch_rope_and_cache(a, D, dtype == PA_F16, CachePool::int4, st, sms);
  }
  if (kv.fp8)
    return launch_reshape_and_cache_fp8(key, value, kstride, vstride, kc, vc, block_stride, slots,
                                        num_tokens, H_kv, D, bs, num_blocks, kv.k_scale,
                                        kv.v_scale, status, st, sms, pdl, dtype == PA_F16);
  return launch_reshape_and_cache(key, value, kstride, vstride, kc, vc, block_stride, slots,
                                  num_tokens, H_kv, D, bs, num_blocks, status, st, sms, pdl);
}

// Validate an optional K/V update of an update-and-attend call.
pa_status check_kv_update(const pa_kv_update* u, const CommonAttn& c, void* key_cache,
                          void* value_cache, int dtype) {
  if (!u || u->num_tokens == 0) return u && u->num_tokens < 0 ? PA_ERR_INVALID_ARG : PA_OK;
  return check_update(u->key, u->value, u->key_token_stride, u->value_token_stride, key_cache,
                      value_cache, c.block_stride, u->slot_mapping, u->num_tokens, c.H_kv, c.D,
                      c.bs, c.num_blocks, dtype, c.kv);
}

// Launch the update's scatter right after the planner, as a programmatic
// dependent: it overlaps the planner (its inputs predate the call), and the
// first attention kernel waits for it before reading the cache.
pa_status launch_kv_update(const pa_kv_update* u, const CommonAttn& c, void* key_cache,
                           void* value_cache, int sms) {
  if (!u || u->num_tokens == 0) return PA_OK;
  return launch_scatter(u->key, u->value, u->key_token_stride, u->value_token_stride, key_cache,
                        value_cache, c.block_stride, u->slot_mapping, u->num_tokens, c.H_kv, c.D,
                        c.bs, c.num_blocks, c.kv, c.status, c.st, sms, true, c.dtype) == cudaSuccess
             ? PA_OK
             : PA_ERR_CUDA;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" {

const char* pa_status_string(pa_status s) {
  switch (s) {
    case PA_OK: return "PA_OK";
    case PA_ERR_INVALID_ARG: return "PA_ERR_INVALID_ARG: invalid argument";
    case PA_ERR_BLOCK_SIZE: return "PA_ERR_BLOCK_SIZE: block size must be a multiple of 16 (<= 1024)";
    case PA_ERR_UNSUPPORTED: return "PA_ERR_UNSUPPORTED: head size or dtype not supported";
    case PA_ERR_WORKSPACE: return "PA_ERR_WORKSPACE: workspace missing, misaligned or too small";
    case PA_ERR_CUDA: return "PA_ERR_CUDA: CUDA launch or query failed";
    case PA_ERR_NOALLOC_LIMIT:
      return "PA_ERR_NOALLOC_LIMIT: the problem needs more scratch than the fixed no-allocation "
             "buffer (PA_NOALLOC_SCRATCH_BYTES) holds; use pa_varlen_fwd with a workspace";
    default: return "PA_ERR_UNKNOWN";
  }
}

int pa_abi_version(void) { return kAbiVersion; }

pa_status pa_reshape_and_cache(const void* key, const void* value, int64_t key_token_stride,
                               int64_t value_token_stride, void* key_cache, void* value_cache,
                               int64_t cache_block_stride, const int64_t* slot_mapping,
                               int num_tokens, int num_kv_heads, int head_size, int block_size,
                               int num_blocks, int dtype, int32_t* dev_status, void* stream) {
  const pa_status st = check_update(key, value, key_token_stride, value_token_stride, key_cache,
                                    value_cache, cache_block_stride, slot_mapping, num_tokens,
                                    num_kv_heads, head_size, block_size, num_blocks, dtype);
  if (st != PA_OK || num_tokens == 0) return st;
  const int sms = query_sms(0);
  if (sms <= 0) return PA_ERR_CUDA;
  cudaError_t e = launch_reshape_and_cache(key, value, key_token_stride, value_token_stride,
                                           key_cache, value_cache, cache_block_stride,
                                           slot_mapping, num_tokens, num_kv_heads, head_size,
                                           block_size, num_blocks, dev_status,
                                           static_cast<cudaStream_t>(stream), sms, false);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

size_t pa_varlen_fwd_workspace_size(int num_seqs, int total_q, int max_seqlen_q, int max_seqlen_k,
                                    int num_heads, int num_kv_heads, int head_size, int block_size,
                                    int sm_count) {
  if (check_shape(num_seqs, total_q, max_seqlen_q, max_seqlen_k, num_heads, num_kv_heads,
                  head_size, block_size, PA_BF16) != PA_OK)
    return 0;
  const int sms = query_sms(sm_count);
  if (sms <= 0) return 0;
  PassDims d{num_seqs, total_q, max_seqlen_q, false, num_heads / num_kv_heads, num_heads,
             num_kv_heads, head_size, sms};
  d.max_kv = max_seqlen_k;
  return varlen_bytes(d);
}

size_t pa_cascade_fwd_workspace_size(int num_seqs, int total_q, int max_seqlen_q,
                                     int max_seqlen_k, int num_heads, int num_kv_heads,
                                     int head_size, int block_size, int sm_count) {
  if (check_shape(num_seqs, total_q, max_seqlen_q, max_seqlen_k, num_heads, num_kv_heads,
                  head_size, block_size, PA_BF16) != PA_OK)
    return 0;
  const int sms = query_sms(sm_count);
  if (sms <= 0) return 0;
  return cascade_bytes(num_seqs, total_q, max_seqlen_q, max_seqlen_k, num_heads / num_kv_heads,
                       num_heads, num_kv_heads, head_size, sms, false);
}

// The factor of a product in the exponential of a capped score.
constexpr double kLog2e64 = 1.4426950408889634;
static float score_cap_in(float scale, float cap) {
  return static_cast<float>(2.0 * kLog2e64 * scale / cap);
}

// The polynomial of tanh for |u| <= 1/2 in terms of the product x, u = cap_u x. The
// seventh power of cap_u has to stay a normal number.
static void set_cap(AttnArgs& a, float scale, float cap) {
  a.cap = static_cast<float>(cap * kLog2e64);
  a.cap_in = score_cap_in(scale, cap);
  const double u = static_cast<double>(scale) / cap;
  a.cap_u = static_cast<float>(u);
  a.cap_x4 = -1.f;
  if (!(std::fabs(u) >= 6e-6 && std::fabs(u) <= 1e4)) return;
  constexpr double c4[4] = {kTanhHalf0, kTanhHalf1, kTanhHalf2, kTanhHalf3};
  double p = u;
  for (int k = 0; k < 4; ++k, p *= u * u) a.cap_c4[k] = static_cast<float>(c4[k] * p);
  a.cap_x4 = static_cast<float>(0.5 / std::fabs(u));
}

// pa_varlen_fwd, optionally preceded by a K/V update of the same cache.
static pa_status varlen_impl(const pa_kv_update* upd, const void* q, int64_t q_token_stride,
                             void* key_cache, void* value_cache, int64_t cache_block_stride,
                             const int32_t* cu_seqlens_q, const int32_t* seqused_k,
                             const int32_t* block_table, int bt_stride, int num_seqs, int total_q,
                             int max_seqlen_q, int max_seqlen_k, int num_heads, int num_kv_heads,
                             int head_size, int block_size, int num_blocks, float softmax_scale,
                             int causal, void* out, float* lse, void* workspace,
                             size_t workspace_bytes, int dtype, int32_t* dev_status,
                             void* stream, const KvFormat& kv, const float* sinks = nullptr,
                             int window = 0, int num_first = 0,
                             const pa_score* score = nullptr) {
  pa_status st = check_shape(num_seqs, total_q, max_seqlen_q, max_seqlen_k, num_heads,
                             num_kv_heads, head_size, block_size, dtype);
  if (st != PA_OK) return st;
  st = check_attn_ptrs(q, q_token_stride, key_cache, value_cache, cache_block_stride, cu_seqlens_q,
                       seqused_k, block_table, bt_stride, num_seqs, total_q, num_blocks, num_heads,
                       num_kv_heads, head_size, block_size, softmax_scale, causal, out, lse, kv);
  if (st != PA_OK) return st;
  if ((reinterpret_cast<uintptr_t>(sinks) & 3u) != 0) return PA_ERR_INVALID_ARG;
  CommonAttn c{q, q_token_stride, key_cache, value_cache, cache_block_stride, cu_seqlens_q,
               seqused_k, block_table, bt_stride, num_seqs, total_q, max_seqlen_q, max_seqlen_k,
               num_heads, num_kv_heads, head_size, block_size, num_blocks, softmax_scale,
               dev_status, static_cast<cudaStream_t>(stream), kv, sinks, dtype};
  st = check_kv_update(upd, c, key_cache, value_cache, dtype);
  if (st != PA_OK) return st;
  if (num_seqs == 0 || total_q == 0) {   // nothing to attend: the update alone
    if (!upd || upd->num_tokens == 0) return PA_OK;
    const int sms = query_sms(0);
    if (sms <= 0) return PA_ERR_CUDA;
    return launch_scatter(upd->key, upd->value, upd->key_token_stride, upd->value_token_stride,
                          key_cache, value_cache, cache_block_stride, upd->slot_mapping,
                          upd->num_tokens, num_kv_heads, head_size, block_size, num_blocks, kv,
                          dev_status, c.st, sms, false, dtype) == cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
  }
  const int sms = query_sms(0);
  if (sms <= 0) return PA_ERR_CUDA;
  PassDims d{num_seqs, total_q, max_seqlen_q, false, num_heads / num_kv_heads, num_heads,
             num_kv_heads, head_size, sms};
  d.max_kv = max_seqlen_k;
  d.kv_fp8 = kv.fp8;
  // (With changed scores the prefill kernel takes negative scales too.)
  d.tc_allowed = softmax_scale > 0.f || (score && softmax_scale < 0.f);
  if (window > 0) {
    // A window of at least every sequence is no window; else a row tile reads
    // at most the first tokens, the window and its own tokens, in whole TMA
    // boxes (of at most 64 keys).
    if (window >= max_seqlen_k) window = num_first = 0;
    if (num_first > max_seqlen_k) num_first = max_seqlen_k;
    const long long reach = static_cast<long long>(cdiv(num_first, kKeyTile)) * kKeyTile + window +
                            2 * kTcTileRows + 2 + kKeyTile;
    if (window > 0 && reach < d.max_kv) d.max_kv = static_cast<int>(reach);
  }
  const PassLayout L = layout_pass(d, 0);
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) % kAlign) != 0 ||
      workspace_bytes < L.end)
    return PA_ERR_WORKSPACE;
  if (window > 0 && static_cast<long long>(max_seqlen_q) * d.G <= kWinRows) {
    // Slices of 16 keys that a sequence's queries see: the first tokens, and
    // window + max_seqlen_q - 1 keys at any offset.
    const long long slices = cdiv(num_first, 16) +
                             (static_cast<long long>(window) + max_seqlen_q - 1) / 16 + 2;
    // A long window of a few (sequence, KV head) pairs is read faster by the
    // planned kernel's finer splits: one sequence of 8 KV heads of 128 takes
    // 24.2 us (25.3 planned) at window 12000, 30.1 (26.8) at 16000; two take
    // 36.7 (50.0).
    const long long units = static_cast<long long>(num_seqs) * num_kv_heads;
    if (slices <= (units * kWinMaxParts < sms ? 3 : 4) * (kWinMaxParts * kWinPartSlices / 4) &&
        units * kWinMaxParts <= 0x7fffffffLL) {
      if (upd && upd->num_tokens > 0 &&
          launch_scatter(upd->key, upd->value, upd->key_token_stride, upd->value_token_stride,
                         key_cache, value_cache, cache_block_stride, upd->slot_mapping,
                         upd->num_tokens, num_kv_heads, head_size, block_size, num_blocks, kv,
                         dev_status, c.st, sms, false, dtype) != cudaSuccess)
        return PA_ERR_CUDA;
      WinDecodeArgs w{};
      w.q = static_cast<const uint16_t*>(q);
      w.q_stride = q_token_stride;
      w.kc = static_cast<const uint8_t*>(key_cache);
      w.vc = static_cast<const uint8_t*>(value_cache);
      w.block_stride_bytes = cache_block_stride * (kv.fp8 ? 1 : 2);
      w.cu = cu_seqlens_q;
      w.seqused_k = seqused_k;
      w.bt = block_table;
      w.bt_stride = bt_stride;
      w.H = num_heads;
      w.H_kv = num_kv_heads;
      w.G = d.G;
      w.bs = block_size;
      w.bs_shift = log2_or_none(block_size);
      w.num_blocks = num_blocks;
      w.total_q = total_q;
      w.max_q = max_seqlen_q;
      w.max_k = max_seqlen_k;
      const long long cap = static_cast<long long>(bt_stride) * block_size;
      w.kv_len_cap = cap > 0x7fffff00 ? 0x7fffff00 : static_cast<int>(cap);
      w.window = window;
      w.first = num_first;
      w.scale_log2 = softmax_scale * 1.4426950408889634f;
      w.k_scale = kv.k_scale;
      w.v_scale = kv.v_scale;
      w.sinks = sinks;
      w.out = static_cast<uint16_t*>(out);
      w.lse = lse;
      w.status = dev_status;
      return launch_window_decode(w, num_seqs, static_cast<int>(slices), head_size,
                                  dtype == PA_F16, c.st, sms) == cudaSuccess
                 ? PA_OK
                 : PA_ERR_CUDA;
    }
  }
  const int box_rows = gcd_int(block_size, kKeyTile);
  CUtensorMap tmK, tmV;
  if (!encode_pool_map(&tmK, key_cache, head_size, num_kv_heads, block_size, num_blocks,
                       cache_block_stride, box_rows, kv.fp8, dtype == PA_F16) ||
      !encode_pool_map(&tmV, value_cache, head_size, num_kv_heads, block_size, num_blocks,
                       cache_block_stride, box_rows, kv.fp8, dtype == PA_F16))
    return PA_ERR_CUDA;
  CUtensorMap tmQ{};
  if (L.items_bound[1] > 0 &&
      !encode_q_map(&tmQ, q, head_size, num_heads, total_q, q_token_stride,
                    num_heads / num_kv_heads, dtype == PA_F16))
    return PA_ERR_CUDA;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const long long cap = static_cast<long long>(bt_stride) * block_size;
  PlanPasses pp{};
  pp.p[0] = make_plan(c, ws, L, 0, 0, 0, cap > 0x7fffffff ? 0x7fffffff : static_cast<int>(cap),
                      causal, 0);
  pp.p[0].window = window;
  pp.p[0].first = num_first;
  pp.p[0].box_rows = box_rows;
  if (launch_plan(pp, 1, c.st) != cudaSuccess) return PA_ERR_CUDA;
  st = launch_kv_update(upd, c, key_cache, value_cache, sms);
  if (st != PA_OK) return st;
  AttnArgs a = make_attn(c, ws, L, bt_stride, 0, causal, out, lse);
  a.window = window;
  a.first = num_first;
  if (score) {
    a.scored = 1;
    if (score->softcap > 0.f) set_cap(a, softmax_scale, score->softcap);
    a.slopes = score->alibi_slopes;
    a.prefix = score->prefix_lens;
    a.first_key = score->first_key;
  }
  bool first = true;
  return launch_pass(c, tmK, tmV, tmQ, a, ws, L, &first);
}

pa_status pa_use_cascade_attention(int common_prefix_len, int num_seqs, int num_kv_heads,
                                   int head_size, int split_kv, int* use_cascade) {
  if (!use_cascade || common_prefix_len < 0 || num_seqs < 0 || num_kv_heads <= 0 ||
      head_size <= 0)
    return PA_ERR_INVALID_ARG;
  *use_cascade = 0;
  if (common_prefix_len < 256 || num_seqs < 8) return PA_OK;   // the pages' two thresholds
  if (!split_kv) {
    *use_cascade = 1;
    return PA_OK;
  }
  // Bytes of the shared prefix that flat attention re-reads (K and V, bf16)
  // against the bytes the cascade's fixed cost could have moved.
  const double reread = static_cast<double>(num_seqs - 1) * common_prefix_len * num_kv_heads *
                        head_size * 4.0;
  const double fixed = PA_CASCADE_FIXED_US * 1e-6 * PA_CASCADE_HBM_GBS * 1e9;
  *use_cascade = reread > fixed ? 1 : 0;
  return PA_OK;
}

pa_status pa_varlen_fwd(const void* q, int64_t q_token_stride, const void* key_cache,
                        const void* value_cache, int64_t cache_block_stride,
                        const int32_t* cu_seqlens_q, const int32_t* seqused_k,
                        const int32_t* block_table, int bt_stride, int num_seqs, int total_q,
                        int max_seqlen_q, int max_seqlen_k, int num_heads, int num_kv_heads,
                        int head_size, int block_size, int num_blocks, float softmax_scale,
                        int causal, void* out, float* lse, void* workspace,
                        size_t workspace_bytes, int dtype, int32_t* dev_status, void* stream) {
  return varlen_impl(nullptr, q, q_token_stride, const_cast<void*>(key_cache),
                     const_cast<void*>(value_cache), cache_block_stride, cu_seqlens_q, seqused_k,
                     block_table, bt_stride, num_seqs, total_q, max_seqlen_q, max_seqlen_k,
                     num_heads, num_kv_heads, head_size, block_size, num_blocks, softmax_scale,
                     causal, out, lse, workspace, workspace_bytes, dtype, dev_status, stream,
                     kKvBf16);
}

pa_status pa_varlen_fwd_with_update(const pa_kv_update* update, const void* q,
                                    int64_t q_token_stride, void* key_cache, void* value_cache,
                                    int64_t cache_block_stride, const int32_t* cu_seqlens_q,
                                    const int32_t* seqused_k, const int32_t* block_table,
                                    int bt_stride, int num_seqs, int total_q, int max_seqlen_q,
                                    int max_seqlen_k, int num_heads, int num_kv_heads,
                                    int head_size, int block_size, int num_blocks,
                                    float softmax_scale, int causal, void* out, float* lse,
                                    void* workspace, size_t workspace_bytes, int dtype,
                                    int32_t* dev_status, void* stream) {
  return varlen_impl(update, q, q_token_stride, key_cache, value_cache, cache_block_stride,
                     cu_seqlens_q, seqused_k, block_table, bt_stride, num_seqs, total_q,
                     max_seqlen_q, max_seqlen_k, num_heads, num_kv_heads, head_size, block_size,
                     num_blocks, softmax_scale, causal, out, lse, workspace, workspace_bytes,
                     dtype, dev_status, stream, kKvBf16);
}

pa_status pa_merge_attn_states(void* out, float* out_lse, const void* prefix_out,
                               const float* prefix_lse, const void* suffix_out,
                               const float* suffix_lse, int num_tokens, int num_heads,
                               int head_size, int dtype, void* stream) {
  if (num_tokens < 0 || num_heads <= 0) return PA_ERR_INVALID_ARG;
  if (dtype != PA_BF16 && dtype != PA_F16) return PA_ERR_UNSUPPORTED;
  if (head_size <= 0 || head_size % 8 != 0 || head_size > 256) return PA_ERR_UNSUPPORTED;
  if (num_tokens == 0) return PA_OK;
  if (!out || !prefix_out || !suffix_out || !prefix_lse || !suffix_lse) return PA_ERR_INVALID_ARG;
  if (!aligned16(out) || !aligned16(prefix_out) || !aligned16(suffix_out)) return PA_ERR_INVALID_ARG;
  if (((reinterpret_cast<uintptr_t>(prefix_lse) | reinterpret_cast<uintptr_t>(suffix_lse) |
        reinterpret_cast<uintptr_t>(out_lse)) & 3u) != 0)
    return PA_ERR_INVALID_ARG;
  if (out_lse && (out_lse == prefix_lse || out_lse == suffix_lse)) return PA_ERR_INVALID_ARG;
  const int sms = query_sms(0);
  if (sms <= 0) return PA_ERR_CUDA;
  cudaError_t e = launch_merge(out, out_lse, prefix_out, prefix_lse, suffix_out, suffix_lse,
                               num_tokens, num_heads, head_size,
                               static_cast<cudaStream_t>(stream), sms, dtype == PA_F16);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status pa_merge_attn_states_n(void* out, float* out_lse, const void* parts_out,
                                 int64_t part_stride_out, const float* parts_lse,
                                 int64_t part_stride_lse, int num_parts, int num_tokens,
                                 int num_heads, int head_size, int dtype, void* stream) {
  if (num_parts < 1 || num_parts > PA_MERGE_N_MAX || num_tokens < 0 || num_heads <= 0)
    return PA_ERR_INVALID_ARG;
  if (dtype != PA_BF16 && dtype != PA_F16) return PA_ERR_UNSUPPORTED;
  if (head_size <= 0 || head_size % 8 != 0 || head_size > 256) return PA_ERR_UNSUPPORTED;
  if (num_tokens == 0) return PA_OK;
  if (!out || !parts_out || !parts_lse) return PA_ERR_INVALID_ARG;
  if (!aligned16(out) || !aligned16(parts_out)) return PA_ERR_INVALID_ARG;
  if (((reinterpret_cast<uintptr_t>(parts_lse) | reinterpret_cast<uintptr_t>(out_lse)) & 3u) != 0)
    return PA_ERR_INVALID_ARG;
  const int64_t row_elems = static_cast<int64_t>(num_tokens) * num_heads * head_size;
  const int64_t lse_elems = static_cast<int64_t>(num_heads) * num_tokens;
  if (num_parts > 1 && (part_stride_out < row_elems || part_stride_out % 8 != 0 ||
                        part_stride_lse < lse_elems))
    return PA_ERR_INVALID_ARG;
  if (out_lse) {   // out_lse must not overlap any part's LSE (other threads still read them)
    const float* lo = parts_lse;
    const float* hi = parts_lse + (num_parts - 1) * part_stride_lse + lse_elems;
    if (out_lse + lse_elems > lo && out_lse < hi) return PA_ERR_INVALID_ARG;
  }
  const int sms = query_sms(0);
  if (sms <= 0) return PA_ERR_CUDA;
  cudaError_t e = launch_merge_n(out, out_lse, parts_out, part_stride_out, parts_lse,
                                 part_stride_lse, num_parts, num_tokens, num_heads, head_size,
                                 static_cast<cudaStream_t>(stream), sms, dtype == PA_F16);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

// pa_cascade_fwd, optionally preceded by a K/V update of the same cache.
static pa_status cascade_impl(const pa_kv_update* upd, const void* q, int64_t q_token_stride,
                              void* key_cache, void* value_cache, int64_t cache_block_stride,
                              const int32_t* cu_seqlens_q, const int32_t* seqused_k,
                              const int32_t* block_table, int bt_stride, int num_seqs,
                              int total_q, int max_seqlen_q, int max_seqlen_k, int num_heads,
                              int num_kv_heads, int head_size, int block_size, int num_blocks,
                              float softmax_scale, int common_prefix_len, void* out, float* lse,
                              void* workspace, size_t workspace_bytes, int dtype,
                              int32_t* dev_status, void* stream, const KvFormat& kv,
                              const float* sinks = nullptr) {
  pa_status st = check_shape(num_seqs, total_q, max_seqlen_q, max_seqlen_k, num_heads,
                             num_kv_heads, head_size, block_size, dtype);
  if (st != PA_OK) return st;
  st = check_attn_ptrs(q, q_token_stride, key_cache, value_cache, cache_block_stride, cu_seqlens_q,
                       seqused_k, block_table, bt_stride, num_seqs, total_q, num_blocks, num_heads,
                       num_kv_heads, head_size, block_size, softmax_scale, 1, out, lse, kv);
  if (st != PA_OK) return st;
  if ((reinterpret_cast<uintptr_t>(sinks) & 3u) != 0) return PA_ERR_INVALID_ARG;
  if (st != PA_OK) return st;
  if (common_prefix_len < 0 || common_prefix_len % block_size != 0) return PA_ERR_INVALID_ARG;
  if (static_cast<long long>(common_prefix_len) > static_cast<long long>(bt_stride) * block_size)
    return PA_ERR_INVALID_ARG;
  {
    const CommonAttn cu{q, q_token_stride, key_cache, value_cache, cache_block_stride,
                        cu_seqlens_q, seqused_k, block_table, bt_stride, num_seqs, total_q,
                        max_seqlen_q, max_seqlen_k, num_heads, num_kv_heads, head_size,
                        block_size, num_blocks, softmax_scale, dev_status,
                        static_cast<cudaStream_t>(stream), kv, sinks, dtype};
    st = check_kv_update(upd, cu, key_cache, value_cache, dtype);
    if (st != PA_OK) return st;
  }
  if (num_seqs == 0 || total_q == 0) {   // nothing to attend: the update alone
    if (!upd || upd->num_tokens == 0) return PA_OK;
    const int sms = query_sms(0);
    if (sms <= 0) return PA_ERR_CUDA;
    return launch_scatter(upd->key, upd->value, upd->key_token_stride, upd->value_token_stride,
                          key_cache, value_cache, cache_block_stride, upd->slot_mapping,
                          upd->num_tokens, num_kv_heads, head_size, block_size, num_blocks, kv,
                          dev_status, static_cast<cudaStream_t>(stream), sms, false, dtype) == cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
  }
  const int sms = query_sms(0);
  if (sms <= 0) return PA_ERR_CUDA;
  const int G = num_heads / num_kv_heads;
  const CascadeLayout CL = layout_cascade(num_seqs, total_q, max_seqlen_q, max_seqlen_k,
                                          common_prefix_len, G, num_heads, num_kv_heads,
                                          head_size, sms, kv.fp8, softmax_scale > 0.f);
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) % kAlign) != 0 ||
      workspace_bytes < CL.end)
    return PA_ERR_WORKSPACE;
  CommonAttn c{q, q_token_stride, key_cache, value_cache, cache_block_stride, cu_seqlens_q,
               seqused_k, block_table, bt_stride, num_seqs, total_q, max_seqlen_q, max_seqlen_k,
               num_heads, num_kv_heads, head_size, block_size, num_blocks, softmax_scale,
               dev_status, static_cast<cudaStream_t>(stream), kv, sinks, dtype};
  const int box_rows = gcd_int(block_size, kKeyTile);
  CUtensorMap tmK, tmV;
  if (!encode_pool_map(&tmK, key_cache, head_size, num_kv_heads, block_size, num_blocks,
                       cache_block_stride, box_rows, kv.fp8, dtype == PA_F16) ||
      !encode_pool_map(&tmV, value_cache, head_size, num_kv_heads, block_size, num_blocks,
                       cache_block_stride, box_rows, kv.fp8, dtype == PA_F16))
    return PA_ERR_CUDA;
  CUtensorMap tmQ{};
  if ((CL.prefix.items_bound[1] > 0 || CL.suffix.items_bound[1] > 0) &&
      !encode_q_map(&tmQ, q, head_size, num_heads, total_q, q_token_stride, G, dtype == PA_F16))
    return PA_ERR_CUDA;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const int P = common_prefix_len;
  const int pages = P / block_size;
  const long long cap = (static_cast<long long>(bt_stride) - pages) * block_size;
  PlanPasses pp{};
  // Pass A: all queries, one non-causal segment, row 0's first P keys; every
  // work item leaves its partial state in its slot.
  pp.p[0] = make_plan(c, ws, CL.prefix, 1, P, 0, P, 0, 0, 1);
  // The prefix pass's items hold every query row of a KV head, and the two
  // passes run side by side. Over 2-byte pools the suffix pass is the longer
  // and finer prefix chunks only take SMs from it; over e4m3 pools the suffix
  // streams half the bytes and the prefix pass is the longer one. Measured on
  // 64 decode requests sharing 2048 tokens (graph step): 2-byte pools 48.2 us
  // with 512-key chunks, 52.4 with 256; e4m3 pools 50.3 with 512, 46.2 with
  // 256.
  pp.p[0].min_chunk_tc = kv.fp8 ? kMinChunkTc : 2 * kMinChunkTc;
  // Pass B: each sequence, causal, its own keys from position P on; each final
  // row is merged with pass A's partial states of the same row.
  pp.p[1] = make_plan(c, ws, CL.suffix, 0, 0, P,
                      cap > 0x7fffffff ? 0x7fffffff : static_cast<int>(cap), 1, 1, 1);
  pp.p[1].make_groups = 1;
  if (launch_plan(pp, 2, c.st) != cudaSuccess) return PA_ERR_CUDA;
  st = launch_kv_update(upd, c, key_cache, value_cache, sms);
  if (st != PA_OK) return st;
  AttnArgs pa_ = make_attn(c, ws, CL.prefix, 0, 0, 0, nullptr, nullptr);
  pa_.partials_only = 1;
  bool first = true;
  st = launch_pass(c, tmK, tmV, tmQ, pa_, ws, CL.prefix, &first);
  if (st != PA_OK) return st;
  // Pass B: each sequence, causal, its own keys from position P on; every
  // work item leaves its partial state too, so no block of either pass waits
  // for the other.
  AttnArgs pb = make_attn(c, ws, CL.suffix, bt_stride, pages, 1, out, lse);
  pb.partials_only = 1;
  st = launch_pass(c, tmK, tmV, tmQ, pb, ws, CL.suffix, &first);
  if (st != PA_OK) return st;
  // Combine: each row of pass B merges its own partial states with pass A's.
  AttnArgs cb = pb;
  cb.partials_only = 0;
  cb.merge_parts = 1;
  cb.mp_seg = reinterpret_cast<const int4*>(ws + CL.prefix.seg);
  cb.mp_segsplit = reinterpret_cast<const int4*>(ws + CL.prefix.segsplit);
  for (int k = 0; k < 2; ++k) {
    cb.mp_part_lse[k] = reinterpret_cast<const float*>(ws + CL.prefix.part_lse[k]);
    cb.mp_part_o[k] = reinterpret_cast<const float*>(ws + CL.prefix.part_o[k]);
    cb.mp_slot_rows[k] = CL.prefix.slot_rows[k];
  }
  AttnArgs c0 = cb, c1 = cb;
  set_class(c0, ws, CL.suffix, 0);
  set_class(c1, ws, CL.suffix, 1);
  if (launch_cascade_combine(c0, c1, CL.suffix.items_bound[0], CL.suffix.items_bound[1], c.st) !=
      cudaSuccess)
    return PA_ERR_CUDA;
  return PA_OK;
}

pa_status pa_cascade_fwd(const void* q, int64_t q_token_stride, const void* key_cache,
                         const void* value_cache, int64_t cache_block_stride,
                         const int32_t* cu_seqlens_q, const int32_t* seqused_k,
                         const int32_t* block_table, int bt_stride, int num_seqs, int total_q,
                         int max_seqlen_q, int max_seqlen_k, int num_heads, int num_kv_heads,
                         int head_size, int block_size, int num_blocks, float softmax_scale,
                         int common_prefix_len, void* out, float* lse, void* workspace,
                         size_t workspace_bytes, int dtype, int32_t* dev_status, void* stream) {
  return cascade_impl(nullptr, q, q_token_stride, const_cast<void*>(key_cache),
                      const_cast<void*>(value_cache), cache_block_stride, cu_seqlens_q, seqused_k,
                      block_table, bt_stride, num_seqs, total_q, max_seqlen_q, max_seqlen_k,
                      num_heads, num_kv_heads, head_size, block_size, num_blocks, softmax_scale,
                      common_prefix_len, out, lse, workspace, workspace_bytes, dtype, dev_status,
                      stream, kKvBf16);
}

pa_status pa_cascade_fwd_with_update(const pa_kv_update* update, const void* q,
                                     int64_t q_token_stride, void* key_cache, void* value_cache,
                                     int64_t cache_block_stride, const int32_t* cu_seqlens_q,
                                     const int32_t* seqused_k, const int32_t* block_table,
                                     int bt_stride, int num_seqs, int total_q, int max_seqlen_q,
                                     int max_seqlen_k, int num_heads, int num_kv_heads,
                                     int head_size, int block_size, int num_blocks,
                                     float softmax_scale, int common_prefix_len, void* out,
                                     float* lse, void* workspace, size_t workspace_bytes,
                                     int dtype, int32_t* dev_status, void* stream) {
  return cascade_impl(update, q, q_token_stride, key_cache, value_cache, cache_block_stride,
                      cu_seqlens_q, seqused_k, block_table, bt_stride, num_seqs, total_q,
                      max_seqlen_q, max_seqlen_k, num_heads, num_kv_heads, head_size, block_size,
                      num_blocks, softmax_scale, common_prefix_len, out, lse, workspace,
                      workspace_bytes, dtype, dev_status, stream, kKvBf16);
}

// ---------------------------------------------------------------- FP8 cache
static KvFormat fp8_format(const pa_kv_fp8* f) {
  return KvFormat{true, f ? f->k_scale : nullptr, f ? f->v_scale : nullptr};
}

pa_status pa_reshape_and_cache_fp8(const void* key, const void* value, int64_t key_token_stride,
                                   int64_t value_token_stride, void* key_cache, void* value_cache,
                                   int64_t cache_block_stride, const int64_t* slot_mapping,
                                   int num_tokens, int num_kv_heads, int head_size,
                                   int block_size, int num_blocks, const pa_kv_fp8* scales,
                                   int dtype, int32_t* dev_status, void* stream) {
  const KvFormat kv = fp8_format(scales);
  const pa_status st =
      check_update(key, value, key_token_stride, value_token_stride, key_cache, value_cache,
                   cache_block_stride, slot_mapping, num_tokens, num_kv_heads, head_size,
                   block_size, num_blocks, dtype, kv);
  if (st != PA_OK || num_tokens == 0) return st;
  const int sms = query_sms(0);
  if (sms <= 0) return PA_ERR_CUDA;
  return launch_scatter(key, value, key_token_stride, value_token_stride, key_cache, value_cache,
                        cache_block_stride, slot_mapping, num_tokens, num_kv_heads, head_size,
                        block_size, num_blocks, kv, dev_status, static_cast<cudaStream_t>(stream),
                        sms, false, dtype) == cudaSuccess
             ? PA_OK
             : PA_ERR_CUDA;
}

size_t pa_varlen_fwd_fp8kv_workspace_size(int num_seqs, int total_q, int max_seqlen_q,
                                          int max_seqlen_k, int num_heads, int num_kv_heads,
                                          int head_size, int block_size, int sm_count) {
  if (check_shape(num_seqs, total_q, max_seqlen_q, max_seqlen_k, num_heads, num_kv_heads,
                  head_size, block_size, PA_BF16) != PA_OK || head_size != 128)
    return 0;
  const int sms = query_sms(sm_count);
  if (sms <= 0) return 0;
  PassDims d{num_seqs, total_q, max_seqlen_q, false, num_heads / num_kv_heads, num_heads,
             num_kv_heads, head_size, sms};
  d.max_kv = max_seqlen_k;
  d.kv_fp8 = true;
  return varlen_bytes(d);
}

size_t pa_cascade_fwd_fp8kv_workspace_size(int num_seqs, int total_q, int max_seqlen_q,
                                           int max_seqlen_k, int num_heads, int num_kv_heads,
                                           int head_size, int block_size, int sm_count) {
  if (check_shape(num_seqs, total_q, max_seqlen_q, max_seqlen_k, num_heads, num_kv_heads,
                  head_size, block_size, PA_BF16) != PA_OK || head_size != 128)
    return 0;
  const int sms = query_sms(sm_count);
  if (sms <= 0) return 0;
  return cascade_bytes(num_seqs, total_q, max_seqlen_q, max_seqlen_k, num_heads / num_kv_heads,
                       num_heads, num_kv_heads, head_size, sms, true);
}

pa_status pa_varlen_fwd_fp8kv(const pa_kv_update* update, const void* q, int64_t q_token_stride,
                              void* key_cache, void* value_cache, int64_t cache_block_stride,
                              const int32_t* cu_seqlens_q, const int32_t* seqused_k,
                              const int32_t* block_table, int bt_stride, int num_seqs,
                              int total_q, int max_seqlen_q, int max_seqlen_k, int num_heads,
                              int num_kv_heads, int head_size, int block_size, int num_blocks,
                              float softmax_scale, int causal, const pa_kv_fp8* scales, void* out,
                              float* lse, void* workspace, size_t workspace_bytes, int dtype,
                              int32_t* dev_status, void* stream) {
  return varlen_impl(update, q, q_token_stride, key_cache, value_cache, cache_block_stride,
                     cu_seqlens_q, seqused_k, block_table, bt_stride, num_seqs, total_q,
                     max_seqlen_q, max_seqlen_k, num_heads, num_kv_heads, head_size, block_size,
                     num_blocks, softmax_scale, causal, out, lse, workspace, workspace_bytes,
                     dtype, dev_status, stream, fp8_format(scales));
}

pa_status pa_cascade_fwd_fp8kv(const pa_kv_update* update, const void* q,
                               int64_t q_token_stride, void* key_cache, void* value_cache,
                               int64_t cache_block_stride, const int32_t* cu_seqlens_q,
                               const int32_t* seqused_k, const int32_t* block_table,
                               int bt_stride, int num_seqs, int total_q, int max_seqlen_q,
                               int max_seqlen_k, int num_heads, int num_kv_heads, int head_size,
                               int block_size, int num_blocks, float softmax_scale,
                               int common_prefix_len, const pa_kv_fp8* scales, void* out,
                               float* lse, void* workspace, size_t workspace_bytes, int dtype,
                               int32_t* dev_status, void* stream) {
  return cascade_impl(update, q, q_token_stride, key_cache, value_cache, cache_block_stride,
                      cu_seqlens_q, seqused_k, block_table, bt_stride, num_seqs, total_q,
                      max_seqlen_q, max_seqlen_k, num_heads, num_kv_heads, head_size, block_size,
                      num_blocks, softmax_scale, common_prefix_len, out, lse, workspace,
                      workspace_bytes, dtype, dev_status, stream, fp8_format(scales));
}

// ---------------------------------------------------------------- options
pa_status pa_varlen_fwd_ex(const pa_kv_update* update, const void* q, int64_t q_token_stride,
                           void* key_cache, void* value_cache, int64_t cache_block_stride,
                           const int32_t* cu_seqlens_q, const int32_t* seqused_k,
                           const int32_t* block_table, int bt_stride, int num_seqs, int total_q,
                           int max_seqlen_q, int max_seqlen_k, int num_heads, int num_kv_heads,
                           int head_size, int block_size, int num_blocks, float softmax_scale,
                           int causal, const pa_attn_opts* opts, void* out, float* lse,
                           void* workspace, size_t workspace_bytes, int dtype,
                           int32_t* dev_status, void* stream) {
  const KvFormat kv = opts && opts->fp8 ? fp8_format(opts->fp8) : kKvBf16;
  return varlen_impl(update, q, q_token_stride, key_cache, value_cache, cache_block_stride,
                     cu_seqlens_q, seqused_k, block_table, bt_stride, num_seqs, total_q,
                     max_seqlen_q, max_seqlen_k, num_heads, num_kv_heads, head_size, block_size,
                     num_blocks, softmax_scale, causal, out, lse, workspace, workspace_bytes,
                     dtype, dev_status, stream, kv, opts ? opts->sinks : nullptr);
}

pa_status pa_cascade_fwd_ex(const pa_kv_update* update, const void* q, int64_t q_token_stride,
                            void* key_cache, void* value_cache, int64_t cache_block_stride,
                            const int32_t* cu_seqlens_q, const int32_t* seqused_k,
                            const int32_t* block_table, int bt_stride, int num_seqs,
                            int total_q, int max_seqlen_q, int max_seqlen_k, int num_heads,
                            int num_kv_heads, int head_size, int block_size, int num_blocks,
                            float softmax_scale, int common_prefix_len, const pa_attn_opts* opts,
                            void* out, float* lse, void* workspace, size_t workspace_bytes,
                            int dtype, int32_t* dev_status, void* stream) {
  const KvFormat kv = opts && opts->fp8 ? fp8_format(opts->fp8) : kKvBf16;
  return cascade_impl(update, q, q_token_stride, key_cache, value_cache, cache_block_stride,
                      cu_seqlens_q, seqused_k, block_table, bt_stride, num_seqs, total_q,
                      max_seqlen_q, max_seqlen_k, num_heads, num_kv_heads, head_size, block_size,
                      num_blocks, softmax_scale, common_prefix_len, out, lse, workspace,
                      workspace_bytes, dtype, dev_status, stream, kv,
                      opts ? opts->sinks : nullptr);
}

// ---------------------------------------------------------------- sliding window
pa_status pa_window_fwd(const pa_kv_update* update, const void* q, int64_t q_token_stride,
                        void* key_cache, void* value_cache, int64_t cache_block_stride,
                        const int32_t* cu_seqlens_q, const int32_t* seqused_k,
                        const int32_t* block_table, int bt_stride, int num_seqs, int total_q,
                        int max_seqlen_q, int max_seqlen_k, int num_heads, int num_kv_heads,
                        int head_size, int block_size, int num_blocks, float softmax_scale,
                        int window, int num_first, const pa_attn_opts* opts, void* out,
                        float* lse, void* workspace, size_t workspace_bytes, int dtype,
                        int32_t* dev_status, void* stream) {
  if (window < 1 || num_first < 0) return PA_ERR_INVALID_ARG;
  const KvFormat kv = opts && opts->fp8 ? fp8_format(opts->fp8) : kKvBf16;
  return varlen_impl(update, q, q_token_stride, key_cache, value_cache, cache_block_stride,
                     cu_seqlens_q, seqused_k, block_table, bt_stride, num_seqs, total_q,
                     max_seqlen_q, max_seqlen_k, num_heads, num_kv_heads, head_size, block_size,
                     num_blocks, softmax_scale, 1, out, lse, workspace, workspace_bytes, dtype,
                     dev_status, stream, kv, opts ? opts->sinks : nullptr, window, num_first);
}

// ---------------------------------------------------------------- changed scores
pa_status pa_score_fwd(const pa_kv_update* update, const void* q, int64_t q_token_stride,
                       void* key_cache, void* value_cache, int64_t cache_block_stride,
                       const int32_t* cu_seqlens_q, const int32_t* seqused_k,
                       const int32_t* block_table, int bt_stride, int num_seqs, int total_q,
                       int max_seqlen_q, int max_seqlen_k, int num_heads, int num_kv_heads,
                       int head_size, int block_size, int num_blocks, float softmax_scale,
                       const pa_score* score, const pa_attn_opts* opts, void* out, float* lse,
                       void* workspace, size_t workspace_bytes, int dtype, int32_t* dev_status,
                       void* stream) {
  if (opts && opts->fp8) return PA_ERR_UNSUPPORTED;
  if (score) {
    if (!std::isfinite(score->softcap) || score->softcap < 0.f ||
        !std::isfinite(static_cast<float>(score->softcap * kLog2e64)))
      return PA_ERR_INVALID_ARG;
    if (score->softcap > 0.f && !std::isfinite(score_cap_in(softmax_scale, score->softcap)))
      return PA_ERR_INVALID_ARG;
    if (((reinterpret_cast<uintptr_t>(score->alibi_slopes) |
          reinterpret_cast<uintptr_t>(score->prefix_lens) |
          reinterpret_cast<uintptr_t>(score->first_key)) & 3u) != 0)
      return PA_ERR_INVALID_ARG;
    if (score->softcap == 0.f && !score->alibi_slopes && !score->prefix_lens && !score->first_key)
      score = nullptr;
  }
  return varlen_impl(update, q, q_token_stride, key_cache, value_cache, cache_block_stride,
                     cu_seqlens_q, seqused_k, block_table, bt_stride, num_seqs, total_q,
                     max_seqlen_q, max_seqlen_k, num_heads, num_kv_heads, head_size, block_size,
                     num_blocks, softmax_scale, 1, out, lse, workspace, workspace_bytes, dtype,
                     dev_status, stream, kKvBf16, opts ? opts->sinks : nullptr, 0, 0, score);
}

// ---------------------------------------------------------------- rotary positions
pa_status pa_rope_table(float* cos_sin, int table_len, int rot_dim, double base,
                        const pa_rope_scaling* scaling, void* stream) {
  constexpr double kTwoPi = 6.283185307179586;
  if (table_len < 0 || table_len > kMaxKeys || rot_dim < 2 || rot_dim > 256 || rot_dim % 2 != 0)
    return PA_ERR_INVALID_ARG;
  if (!std::isfinite(base) || !(base > 0.0)) return PA_ERR_INVALID_ARG;
  const pa_rope_scaling none{PA_ROPE_NONE, 1.0, 1.0, 1.0, 2.0, 1.0};
  const pa_rope_scaling& s = scaling ? *scaling : none;
  if (s.kind < PA_ROPE_NONE || s.kind > PA_ROPE_YARN || !std::isfinite(s.mscale))
    return PA_ERR_INVALID_ARG;
  if (s.kind != PA_ROPE_NONE && (!std::isfinite(s.factor) || !(s.factor > 0.0)))
    return PA_ERR_INVALID_ARG;
  if (s.kind == PA_ROPE_WAVELENGTH || s.kind == PA_ROPE_YARN) {
    if (!std::isfinite(s.orig_len) || !(s.orig_len > 0.0) || !std::isfinite(s.high) ||
        !(s.low > 0.0) || !(s.high > s.low))
      return PA_ERR_INVALID_ARG;
  }
  double ramp_lo = 0.0, ramp_len = 1.0;
  if (s.kind == PA_ROPE_NTK) {
    if (rot_dim == 2) return PA_ERR_INVALID_ARG;
    base *= std::pow(s.factor, rot_dim / (rot_dim - 2.0));
    if (!std::isfinite(base) || !(base > 0.0)) return PA_ERR_INVALID_ARG;
  }
  if (s.kind == PA_ROPE_YARN) {
    if (!(base > 1.0)) return PA_ERR_INVALID_ARG;
    auto pair_of = [&](double turns) {
      return rot_dim * std::log(s.orig_len / (turns * kTwoPi)) / (2.0 * std::log(base));
    };
    ramp_lo = std::fmax(std::floor(pair_of(s.high)), 0.0);
    ramp_len = std::fmax(std::fmin(std::ceil(pair_of(s.low)), rot_dim - 1.0) - ramp_lo, 0.001);
  }
  auto unit = [](double x) { return std::fmin(1.0, std::fmax(0.0, x)); };
  RopeTableArgs a{};
  a.table_len = table_len;
  a.rot = rot_dim;
  a.mscale = static_cast<float>(s.mscale);
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot_dim), keep = 1.0;   // share of the unscaled rate
    if (s.kind == PA_ROPE_LINEAR) keep = 0.0;
    if (s.kind == PA_ROPE_WAVELENGTH)
      keep = unit((s.orig_len * f / kTwoPi - s.low) / (s.high - s.low));
    if (s.kind == PA_ROPE_YARN) keep = 1.0 - unit((i - ramp_lo) / ramp_len);
    f = keep == 1.0 ? f : f / s.factor * (1.0 - keep) + f * keep;
    const double turns = f / kTwoPi;
    if (!(turns < 9007199254740992.0)) return PA_ERR_INVALID_ARG;   // 2^53: no fraction left
    const double frac = (turns - std::floor(turns)) * 0x1p32, hi = std::floor(frac);
    a.rate[i] = (static_cast<unsigned long long>(hi) << 32) +
                static_cast<unsigned long long>(std::nearbyint((frac - hi) * 0x1p32));
  }
  if (table_len == 0) return PA_OK;
  if (!cos_sin || !aligned16(cos_sin)) return PA_ERR_INVALID_ARG;
  const int sms = query_sms(0);
  if (sms <= 0) return PA_ERR_CUDA;
  return launch_rope_table(cos_sin, a, static_cast<cudaStream_t>(stream), sms) == cudaSuccess
             ? PA_OK
             : PA_ERR_CUDA;
}

static pa_status rope_impl(const pa_rope* rope, const int64_t* positions, const void* q,
                           int64_t q_token_stride, void* q_out, int64_t q_out_token_stride,
                           const pa_kv_update* update, void* key_cache, void* value_cache,
                           int64_t cache_block_stride, int num_heads, int num_kv_heads,
                           int head_size, int block_size, int num_blocks, const KvFormat& kv,
                           int dtype, int32_t* dev_status, void* stream) {
  if (!rope || !update || num_heads <= 0) return PA_ERR_INVALID_ARG;
  // Offsets within a token's row are 32-bit.
  if (static_cast<int64_t>(num_heads) * head_size > (1 << 28) ||
      static_cast<int64_t>(num_kv_heads) * head_size > (1 << 28))
    return PA_ERR_INVALID_ARG;
  pa_status st = check_update(update->key, update->value, update->key_token_stride,
                              update->value_token_stride, key_cache, value_cache,
                              cache_block_stride, update->slot_mapping, update->num_tokens,
                              num_kv_heads, head_size, block_size, num_blocks, dtype, kv);
  if (st != PA_OK) return st;
  if (rope->table_len < 0 || rope->rot_dim < 16 || rope->rot_dim % 16 != 0 ||
      rope->rot_dim > head_size || (rope->interleaved != 0 && rope->interleaved != 1))
    return PA_ERR_INVALID_ARG;
  if (!std::isfinite(rope->norm_eps) || rope->norm_eps < 0.f) return PA_ERR_INVALID_ARG;
  const int T = update->num_tokens;
  if (T == 0) return PA_OK;
  if (!positions || (reinterpret_cast<uintptr_t>(positions) & 7u) != 0) return PA_ERR_INVALID_ARG;
  if (!rope->cos_sin || !aligned16(rope->cos_sin) || !aligned16(rope->q_norm) ||
      !aligned16(rope->k_norm))
    return PA_ERR_INVALID_ARG;
  if (!q || !q_out || !aligned16(q) || !aligned16(q_out)) return PA_ERR_INVALID_ARG;
  const int64_t row = static_cast<int64_t>(num_heads) * head_size;
  if (q_token_stride < row || q_out_token_stride < row || q_token_stride % 8 != 0 ||
      q_out_token_stride % 8 != 0)
    return PA_ERR_INVALID_ARG;
  if (q_out != q || q_out_token_stride != q_token_stride) {
    // Rows are read and written by different warps: in place or apart, or, with
    // one stride, q_out's rows between those of q.
    const char* lo = static_cast<const char*>(q);
    const char* out = static_cast<const char*>(q_out);
    if (out < lo + 2 * ((T - 1) * q_token_stride + row) &&
        lo < out + 2 * ((T - 1) * q_out_token_stride + row)) {
      const int64_t step = 2 * q_token_stride;
      const int64_t at = ((out - lo) % step + step) % step;   // in the rows of q
      if (q_out_token_stride != q_token_stride || at < 2 * row || step - at < 2 * row)
        return PA_ERR_INVALID_ARG;
    }
  }
  const int sms = query_sms(0);
  if (sms <= 0) return PA_ERR_CUDA;
  RopeArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(update->key);
  a.v = static_cast<const uint16_t*>(update->value);
  a.q_out = static_cast<uint16_t*>(q_out);
  a.q_stride = q_token_stride;
  a.k_stride = update->key_token_stride;
  a.v_stride = update->value_token_stride;
  a.q_out_stride = q_out_token_stride;
  a.kc = static_cast<uint8_t*>(key_cache);
  a.vc = static_cast<uint8_t*>(value_cache);
  a.block_stride_bytes = cache_block_stride * (kv.fp8 || kv.int4 ? 1 : 2);
  a.slots = update->slot_mapping;
  a.positions = positions;
  a.cos_sin = rope->cos_sin;
  a.table_len = rope->table_len;
  a.rot = rope->rot_dim;
  a.interleaved = rope->interleaved;
  a.q_norm = rope->q_norm;
  a.k_norm = rope->k_norm;
  a.eps = rope->norm_eps;
  a.k_scale = kv.k_scale;
  a.v_scale = kv.v_scale;
  a.k_params = kv.k_params;
  a.v_params = kv.v_params;
  a.params_stride = kv.params_stride;
  a.num_tokens = T;
  a.H = num_heads;
  a.H_kv = num_kv_heads;
  a.bs = block_size;
  a.num_slots = static_cast<int64_t>(num_blocks) * block_size;
  a.status = dev_status;
  return launch_rope_and_cache(a, head_size, dtype == PA_F16,
                               kv.fp8    ? CachePool::e4m3
                               : kv.int4 ? CachePool::int4
                                         : CachePool::same,
                               static_cast<cudaStream_t>(stream), sms) == cudaSuccess
             ? PA_OK
             : PA_ERR_CUDA;
}

pa_status pa_rope_and_cache(const pa_rope* rope, const int64_t* positions, const void* q,
                            int64_t q_token_stride, void* q_out, int64_t q_out_token_stride,
                            const pa_kv_update* update, void* key_cache, void* value_cache,
                            int64_t cache_block_stride, int num_heads, int num_kv_heads,
                            int head_size, int block_size, int num_blocks, const pa_kv_fp8* fp8,
                            int dtype, int32_t* dev_status, void* stream) {
  return rope_impl(rope, positions, q, q_token_stride, q_out, q_out_token_stride, update,
                   key_cache, value_cache, cache_block_stride, num_heads, num_kv_heads, head_size,
                   block_size, num_blocks, fp8 ? fp8_format(fp8) : kKvBf16, dtype, dev_status,
                   stream);
}

// ---------------------------------------------------------------- 4-bit cache
pa_status pa_rope_and_cache_int4(const pa_rope* rope, const int64_t* positions, const void* q,
                                 int64_t q_token_stride, void* q_out, int64_t q_out_token_stride,
                                 const pa_kv_update* update, void* key_cache, void* value_cache,
                                 int64_t cache_block_stride, const pa_kv_int4* int4, int num_heads,
                                 int num_kv_heads, int head_size, int block_size, int num_blocks,
                                 int dtype, int32_t* dev_status, void* stream) {
  if (!int4) return PA_ERR_INVALID_ARG;
  return rope_impl(rope, positions, q, q_token_stride, q_out, q_out_token_stride, update,
                   key_cache, value_cache, cache_block_stride, num_heads, num_kv_heads, head_size,
                   block_size, num_blocks, int4_format(int4), dtype, dev_status, stream);
}

pa_status pa_reshape_and_cache_int4(const void* key, const void* value, int64_t key_token_stride,
                                    int64_t value_token_stride, void* key_cache, void* value_cache,
                                    int64_t cache_block_stride, const pa_kv_int4* int4,
                                    const int64_t* slot_mapping, int num_tokens, int num_kv_heads,
                                    int head_size, int block_size, int num_blocks, int dtype,
                                    int32_t* dev_status, void* stream) {
  if (!int4) return PA_ERR_INVALID_ARG;
  const KvFormat kv = int4_format(int4);
  const pa_status st =
      check_update(key, value, key_token_stride, value_token_stride, key_cache, value_cache,
                   cache_block_stride, slot_mapping, num_tokens, num_kv_heads, head_size,
                   block_size, num_blocks, dtype, kv);
  if (st != PA_OK || num_tokens == 0) return st;
  const int sms = query_sms(0);
  if (sms <= 0) return PA_ERR_CUDA;
  return launch_scatter(key, value, key_token_stride, value_token_stride, key_cache, value_cache,
                        cache_block_stride, slot_mapping, num_tokens, num_kv_heads, head_size,
                        block_size, num_blocks, kv, dev_status, static_cast<cudaStream_t>(stream),
                        sms, false, dtype) == cudaSuccess
             ? PA_OK
             : PA_ERR_CUDA;
}

pa_status pa_gather_cache_int4(const void* key_cache, const void* value_cache,
                               int64_t cache_block_stride, const pa_kv_int4* int4,
                               const int64_t* slot_mapping, int num_tokens, int num_kv_heads,
                               int head_size, int block_size, int num_blocks, void* key,
                               void* value, int dtype, int32_t* dev_status, void* stream) {
  if (!int4 || num_tokens < 0 || num_kv_heads <= 0 || num_blocks < 0) return PA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(num_kv_heads) * head_size > (1 << 28)) return PA_ERR_INVALID_ARG;
  if (dtype != PA_BF16 && dtype != PA_F16) return PA_ERR_UNSUPPORTED;
  if (head_size != 64 && head_size != 128) return PA_ERR_UNSUPPORTED;
  if (block_size <= 0 || block_size % 16 != 0 || block_size > 1024) return PA_ERR_BLOCK_SIZE;
  if (num_tokens == 0) return PA_OK;
  const KvFormat kv = int4_format(int4);
  const pa_status st = check_int4(kv, key_cache, value_cache, cache_block_stride, num_kv_heads,
                                  head_size, block_size);
  if (st != PA_OK) return st;
  if (!slot_mapping || (reinterpret_cast<uintptr_t>(slot_mapping) & 7u) != 0 || !key || !value ||
      !aligned16(key) || !aligned16(value))
    return PA_ERR_INVALID_ARG;
  const int sms = query_sms(0);
  if (sms <= 0) return PA_ERR_CUDA;
  Int4RowsArgs a{};
  a.kc = static_cast<const uint8_t*>(key_cache);
  a.vc = static_cast<const uint8_t*>(value_cache);
  a.block_stride_bytes = cache_block_stride;
  a.k_params = kv.k_params;
  a.v_params = kv.v_params;
  a.params_stride = kv.params_stride;
  a.slots = slot_mapping;
  a.key = static_cast<uint16_t*>(key);
  a.value = static_cast<uint16_t*>(value);
  a.num_tokens = num_tokens;
  a.H_kv = num_kv_heads;
  a.bs = block_size;
  a.num_slots = static_cast<int64_t>(num_blocks) * block_size;
  a.status = dev_status;
  return launch_int4_rows(a, head_size, dtype == PA_F16, static_cast<cudaStream_t>(stream), sms) ==
                 cudaSuccess
             ? PA_OK
             : PA_ERR_CUDA;
}

// The kernels of a call over 4-bit pools, from host-known bounds only: decode of
// at most 8 packed rows (nr = 1), short queries of more (nr = 2 to 4), prompts.
struct Int4Plan {
  bool few, some, many;
  int nr;                // of `some`: groups of 8 rows
  PassLayout tc;         // of `many`
  size_t table, parts, end;   // partial states of the decode kernels; all bytes
  size_t part_rows;
};

static Int4Plan plan_int4(const PassDims& d) {
  Int4Plan p{};
  const long long rows = static_cast<long long>(d.max_q) * d.G;
  p.few = d.G <= 8;
  // Its most rows: whole tokens within the bound and the class.
  const long long most = rows < kI4MaxRows ? rows : static_cast<long long>(kI4MaxRows / d.G) * d.G;
  p.nr = most <= 16 ? 2 : most <= 24 ? 3 : 4;
  p.some = d.max_q > 8 / d.G && kI4MaxRows / d.G > 8 / d.G;
  p.many = rows > kI4MaxRows;
  size_t off = 0;
  if (p.many) {
    p.tc = layout_pass(d, 0);
    off = p.tc.end;
  }
  p.table = align_up(off);
  p.parts = align_up(p.table + (static_cast<size_t>(d.num_segs) + 1) * 8);
  if (p.few) p.part_rows = int4_decode_part_rows(d.sms, d.H_kv, 1, d.num_segs);
  if (p.some) {
    const size_t n = int4_decode_part_rows(d.sms, d.H_kv, p.nr, d.num_segs);
    if (n > p.part_rows) p.part_rows = n;
  }
  p.end = align_up(p.parts + p.part_rows * 4) + p.part_rows * d.D * 4;
  return p;
}

static PassDims int4_dims(int num_seqs, int total_q, int max_q, int max_k, int H, int H_kv, int D,
                          int sms) {
  PassDims d{num_seqs, total_q, max_q, false, H / H_kv, H, H_kv, D, sms};
  d.max_kv = max_k;
  return d;
}

size_t pa_varlen_fwd_int4kv_workspace_size(int num_seqs, int total_q, int max_seqlen_q,
                                           int max_seqlen_k, int num_heads, int num_kv_heads,
                                           int head_size, int block_size, int sm_count) {
  if (check_shape(num_seqs, total_q, max_seqlen_q, max_seqlen_k, num_heads, num_kv_heads,
                  head_size, block_size, PA_BF16) != PA_OK ||
      (head_size != 64 && head_size != 128) || num_heads / num_kv_heads > kTcTileRows)
    return 0;
  const int sms = query_sms(sm_count);
  if (sms <= 0) return 0;
  return plan_int4(int4_dims(num_seqs, total_q, max_seqlen_q, max_seqlen_k, num_heads,
                             num_kv_heads, head_size, sms)).end;
}

pa_status pa_varlen_fwd_int4kv(const pa_kv_update* update, const void* q, int64_t q_token_stride,
                               void* key_cache, void* value_cache, int64_t cache_block_stride,
                               const int32_t* cu_seqlens_q, const int32_t* seqused_k,
                               const int32_t* block_table, int bt_stride, int num_seqs,
                               int total_q, int max_seqlen_q, int max_seqlen_k, int num_heads,
                               int num_kv_heads, int head_size, int block_size, int num_blocks,
                               float softmax_scale, int causal, const pa_kv_int4* int4,
                               const float* sinks, void* out, float* lse, void* workspace,
                               size_t workspace_bytes, int dtype, int32_t* dev_status,
                               void* stream) {
  if (!int4) return PA_ERR_INVALID_ARG;
  const KvFormat kv = int4_format(int4);
  pa_status st = check_shape(num_seqs, total_q, max_seqlen_q, max_seqlen_k, num_heads,
                             num_kv_heads, head_size, block_size, dtype);
  if (st != PA_OK) return st;
  if (head_size > 128 || num_heads / num_kv_heads > kTcTileRows) return PA_ERR_UNSUPPORTED;
  st = check_attn_ptrs(q, q_token_stride, key_cache, value_cache, cache_block_stride, cu_seqlens_q,
                       seqused_k, block_table, bt_stride, num_seqs, total_q, num_blocks, num_heads,
                       num_kv_heads, head_size, block_size, softmax_scale, causal, out, lse, kv);
  if (st != PA_OK) return st;
  if ((reinterpret_cast<uintptr_t>(sinks) & 3u) != 0) return PA_ERR_INVALID_ARG;
  if (max_seqlen_k > kMaxKeys || static_cast<int64_t>(num_kv_heads) * head_size > (1 << 28) ||
      static_cast<int64_t>(num_seqs) * num_kv_heads > 0x7fffffff)
    return PA_ERR_INVALID_ARG;
  CommonAttn c{q, q_token_stride, key_cache, value_cache, cache_block_stride, cu_seqlens_q,
               seqused_k, block_table, bt_stride, num_seqs, total_q, max_seqlen_q, max_seqlen_k,
               num_heads, num_kv_heads, head_size, block_size, num_blocks, softmax_scale,
               dev_status, static_cast<cudaStream_t>(stream), kv, sinks, dtype};
  st = check_kv_update(update, c, key_cache, value_cache, dtype);
  if (st != PA_OK) return st;
  const bool attends = num_seqs > 0 && total_q > 0;
  const bool writes = update && update->num_tokens > 0;
  if (!attends && !writes) return PA_OK;
  const int sms = query_sms(0);
  if (sms <= 0) return PA_ERR_CUDA;
  const PassDims d = int4_dims(num_seqs, total_q, max_seqlen_q, max_seqlen_k, num_heads,
                               num_kv_heads, head_size, sms);
  const Int4Plan p = plan_int4(d);
  if (attends && (!workspace || (reinterpret_cast<uintptr_t>(workspace) % kAlign) != 0 ||
                  workspace_bytes < p.end))
    return PA_ERR_WORKSPACE;
  if (writes &&
      launch_scatter(update->key, update->value, update->key_token_stride,
                     update->value_token_stride, key_cache, value_cache, cache_block_stride,
                     update->slot_mapping, update->num_tokens, num_kv_heads, head_size, block_size,
                     num_blocks, kv, dev_status, c.st, sms, false, dtype) != cudaSuccess)
    return PA_ERR_CUDA;
  if (!attends) return PA_OK;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const long long cap = static_cast<long long>(bt_stride) * block_size;
  const int kv_cap = cap > kMaxKeys ? kMaxKeys : static_cast<int>(cap);
  if (p.many) {
    CUtensorMap tmQ;
    if (!encode_q_map(&tmQ, q, head_size, num_heads, total_q, q_token_stride, d.G,
                      dtype == PA_F16))
      return PA_ERR_CUDA;
    PlanPasses pp{};
    pp.p[0] = make_plan(c, ws, p.tc, 0, 0, 0, kv_cap, causal, 0);
    if (launch_plan(pp, 1, c.st) != cudaSuccess) return PA_ERR_CUDA;
    AttnArgs t = make_attn(c, ws, p.tc, bt_stride, 0, causal, out, lse);
    set_class(t, ws, p.tc, 1);
    t.pdl_first = 1;
    const Int4Pools pools{static_cast<const uint8_t*>(key_cache),
                          static_cast<const uint8_t*>(value_cache),
                          cache_block_stride,
                          kv.k_params,
                          kv.v_params,
                          kv.params_stride};
    if (launch_int4_prompt(tmQ, t, pools, p.tc.items_bound[1], c.st) != cudaSuccess)
      return PA_ERR_CUDA;
  }
  Int4DecodeArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.q_stride = q_token_stride;
  a.cu = cu_seqlens_q;
  a.seqused_k = seqused_k;
  a.bt = block_table;
  a.bt_stride = bt_stride;
  a.num_seqs = num_seqs;
  a.H = num_heads;
  a.H_kv = num_kv_heads;
  a.G = d.G;
  a.bs = block_size;
  a.bs_shift = log2_or_none(block_size);
  a.num_blocks = num_blocks;
  a.no_page = num_blocks > 0 ? num_blocks : 1;
  a.total_q = total_q;
  a.max_q = max_seqlen_q;
  a.max_k = max_seqlen_k;
  a.kv_len_cap = kv_cap;
  a.causal = causal;
  a.scale_log2 = softmax_scale * 1.4426950408889634f;
  a.sinks = sinks;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.table = reinterpret_cast<long long*>(ws + p.table);
  a.part_lse = reinterpret_cast<float*>(ws + p.parts);
  a.part_o = reinterpret_cast<float*>(ws + align_up(p.parts + p.part_rows * 4));
  a.status = dev_status;
  Int4Maps maps;
  if ((p.few || p.some) &&
      !encode_int4_maps(&maps, kv, key_cache, value_cache, cache_block_stride, num_kv_heads,
                        head_size, block_size, num_blocks))
    return PA_ERR_CUDA;
  if (p.few) {
    a.tokens_min = 0;
    a.tokens_max = 8 / d.G;
    if (launch_int4_decode(maps, a, head_size, dtype == PA_F16, 1, sms, c.st) != cudaSuccess)
      return PA_ERR_CUDA;
  }
  if (p.some) {
    a.tokens_min = 8 / d.G;
    a.tokens_max = kI4MaxRows / d.G;
    if (launch_int4_decode(maps, a, head_size, dtype == PA_F16, p.nr, sms, c.st) != cudaSuccess)
      return PA_ERR_CUDA;
  }
  return PA_OK;
}

// ---------------------------------------------------------------- weights, eviction
pa_status pa_attn_weights(const void* q, int64_t q_token_stride, const void* key_cache,
                          int64_t cache_block_stride, const float* lse,
                          const int32_t* cu_seqlens_q, const int32_t* seqused_k,
                          const int32_t* block_table, int bt_stride, int num_seqs, int total_q,
                          int max_seqlen_q, int max_seqlen_k, int num_heads, int num_kv_heads,
                          int head_size, int block_size, int num_blocks, float softmax_scale,
                          int causal, float* weights, int64_t weights_block_stride,
                          const pa_kv_fp8* fp8, int dtype, int32_t* dev_status, void* stream) {
  pa_status st = check_shape(num_seqs, total_q, max_seqlen_q, max_seqlen_k, num_heads,
                             num_kv_heads, head_size, block_size, dtype);
  if (st != PA_OK) return st;
  if (fp8 && head_size != 128) return PA_ERR_UNSUPPORTED;
  if (fp8 && (!fp8->k_scale || (reinterpret_cast<uintptr_t>(fp8->k_scale) & 3u) != 0))
    return PA_ERR_INVALID_ARG;
  if (num_seqs > 0 && (!cu_seqlens_q || !seqused_k || !block_table)) return PA_ERR_INVALID_ARG;
  if (total_q > 0 && (!q || !lse)) return PA_ERR_INVALID_ARG;
  if (!key_cache || !weights) return PA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(key_cache) || !aligned16(weights)) return PA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(lse) & 3u) != 0) return PA_ERR_INVALID_ARG;
  if (q_token_stride < static_cast<int64_t>(num_heads) * head_size || q_token_stride % 8 != 0)
    return PA_ERR_INVALID_ARG;
  if (cache_block_stride < static_cast<int64_t>(block_size) * num_kv_heads * head_size ||
      cache_block_stride % (fp8 ? 16 : 8) != 0)
    return PA_ERR_INVALID_ARG;
  if (weights_block_stride < static_cast<int64_t>(block_size) * num_kv_heads ||
      weights_block_stride % 4 != 0)
    return PA_ERR_INVALID_ARG;
  if (bt_stride < 0 || num_blocks < 0 || !std::isfinite(softmax_scale) ||
      (causal != 0 && causal != 1))
    return PA_ERR_INVALID_ARG;
  // The larger of the two launches: a block per kWeightKeys keys of a sequence
  // and KV head, and one more. (Divided, since the product may pass 64 bits.)
  if (max_seqlen_k > kMaxKeys ||
      static_cast<long long>(total_q) * (num_heads / num_kv_heads) > kMaxKeys ||
      static_cast<long long>(num_seqs) * (max_seqlen_k > 0 ? cdiv(max_seqlen_k, kWeightKeys) : 1) >
          0x7ffffffeLL / num_kv_heads)
    return PA_ERR_INVALID_ARG;
  if (num_seqs == 0 || total_q == 0) return PA_OK;
  const int sms = query_sms(0);
  if (sms <= 0) return PA_ERR_CUDA;
  WeightArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.q_stride = q_token_stride;
  a.kc = static_cast<const uint8_t*>(key_cache);
  a.block_stride_bytes = cache_block_stride * (fp8 ? 1 : 2);
  a.lse = lse;
  a.weights = weights;
  a.weights_stride = weights_block_stride;
  a.cu = cu_seqlens_q;
  a.seqused_k = seqused_k;
  a.bt = block_table;
  a.bt_stride = bt_stride;
  a.H = num_heads;
  a.H_kv = num_kv_heads;
  a.G = num_heads / num_kv_heads;
  a.bs = block_size;
  a.bs_shift = log2_or_none(block_size);
  a.num_blocks = num_blocks;
  a.total_q = total_q;
  a.max_q = max_seqlen_q;
  a.max_k = max_seqlen_k;
  const long long cap = static_cast<long long>(bt_stride) * block_size;
  a.kv_len_cap = cap > kMaxKeys ? kMaxKeys : static_cast<int>(cap);
  a.scale_log2 = softmax_scale * 1.4426950408889634f;
  a.causal = causal;
  a.k_scale = fp8 ? fp8->k_scale : nullptr;
  a.status = dev_status;
  a.tc_min_rows = 0x7fffffff;
  CUtensorMap tmQ{};
  if (tc_tile_rows(a.G) > 0 && static_cast<long long>(max_seqlen_q) * a.G > kWeightsTcMinRows) {
    if (!encode_q_map(&tmQ, q, head_size, num_heads, total_q, q_token_stride, a.G,
                      dtype == PA_F16))
      return PA_ERR_CUDA;
    a.tc_min_rows = kWeightsTcMinRows;
  }
  return launch_attn_weights(tmQ, a, num_seqs, head_size, dtype == PA_F16, fp8 != nullptr,
                             static_cast<cudaStream_t>(stream), sms) == cudaSuccess
             ? PA_OK
             : PA_ERR_CUDA;
}

pa_status pa_evict(void* key_cache, void* value_cache, int64_t cache_block_stride, float* weights,
                   int64_t weights_block_stride, const int32_t* seqused_k,
                   const int32_t* block_table, int bt_stride, int num_seqs, int max_seqlen_k,
                   int num_kv_heads, int head_size, int block_size, int num_blocks, int elem_size,
                   int budget, int num_first, int num_recent, int32_t* kept, int32_t* new_lens,
                   int32_t* dev_status, void* stream) {
  if (num_seqs < 0 || max_seqlen_k < 0 || num_kv_heads <= 0 || num_kv_heads > 65535 ||
      num_blocks < 0 || bt_stride < 0)
    return PA_ERR_INVALID_ARG;
  if (budget < 1 || budget > kMaxKeys || num_first < 0 || num_recent < 0 || num_first > budget ||
      num_recent > budget - num_first)
    return PA_ERR_INVALID_ARG;
  if (elem_size != 1 && elem_size != 2) return PA_ERR_UNSUPPORTED;
  if (head_size != 64 && head_size != 128 && head_size != 256) return PA_ERR_UNSUPPORTED;
  if (elem_size == 1 && head_size != 128) return PA_ERR_UNSUPPORTED;
  if (block_size <= 0 || block_size % 16 != 0 || block_size > 1024) return PA_ERR_BLOCK_SIZE;
  if (num_seqs == 0) return PA_OK;
  if (num_seqs > 0x7fffffff / 64) return PA_ERR_INVALID_ARG;   // blocks of one launch
  if (!key_cache || !value_cache || !weights || !seqused_k || !block_table || !kept || !new_lens)
    return PA_ERR_INVALID_ARG;
  if (!aligned16(key_cache) || !aligned16(value_cache) || !aligned16(weights))
    return PA_ERR_INVALID_ARG;
  if (((reinterpret_cast<uintptr_t>(kept) | reinterpret_cast<uintptr_t>(new_lens)) & 3u) != 0)
    return PA_ERR_INVALID_ARG;
  if (cache_block_stride < static_cast<int64_t>(block_size) * num_kv_heads * head_size ||
      cache_block_stride % (elem_size == 1 ? 16 : 8) != 0)
    return PA_ERR_INVALID_ARG;
  if (weights_block_stride < static_cast<int64_t>(block_size) * num_kv_heads ||
      weights_block_stride % 4 != 0)
    return PA_ERR_INVALID_ARG;
  const int sms = query_sms(0);
  if (sms <= 0) return PA_ERR_CUDA;
  EvictArgs a{};
  a.kc = static_cast<uint8_t*>(key_cache);
  a.vc = static_cast<uint8_t*>(value_cache);
  a.block_stride_bytes = cache_block_stride * elem_size;
  a.weights = weights;
  a.weights_stride = weights_block_stride;
  a.seqused_k = seqused_k;
  a.bt = block_table;
  a.bt_stride = bt_stride;
  a.H_kv = num_kv_heads;
  a.bs = block_size;
  a.num_blocks = num_blocks;
  a.row_bytes = head_size * elem_size;
  a.bs_shift = log2_or_none(block_size);
  a.max_k = max_seqlen_k;
  const long long cap = static_cast<long long>(bt_stride) * block_size;
  a.kv_len_cap = cap > kMaxKeys ? kMaxKeys : static_cast<int>(cap);
  a.budget = budget;
  a.first = num_first;
  a.recent = num_recent;
  a.kept = kept;
  a.new_lens = new_lens;
  a.status = dev_status;
  return launch_evict(a, num_seqs, static_cast<cudaStream_t>(stream), sms) == cudaSuccess
             ? PA_OK
             : PA_ERR_CUDA;
}

}  // extern "C"
