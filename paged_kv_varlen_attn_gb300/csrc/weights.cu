// Accumulated attention weight of every cached key: the column sums of the
// attention matrix, w_j += sum_i exp(scale q_i.k_j - lse_i), recomputed from
// K and the LSE that the attention call returned (the matrix itself never
// exists in memory). Each key has one owner, so there are no atomics and the
// sums are the same bits on every run.
#include <cuda_runtime.h>

#include <type_traits>

#include "device_common.cuh"

namespace pa {

// ---------------------------------------------------------------------------
// Decode and short queries (at most tc_min_rows packed query rows).
// A block, one warp, takes kSlices slices of 16 keys of a sequence and KV head.
// A slice's keys are the M dimension of the warp MMA and 8 packed query rows
// (token, head of the group) its N, so a key's sum is a sum along the
// accumulator's columns: no reduction until the end, where the four lanes of a
// row add up.
// The head dimension is permuted alike in the K (A) and Q (B) fragments so
// that a lane's elements are 16-byte runs and four lanes read 64 consecutive
// bytes; Q goes straight to registers, K through a ring of slots
// filled by asynchronous copies, where every lane reads back its own bytes
// (the ring holds what registers could not: no barrier but the warp's own).
// Decode is bound by the read of K; the ring keeps one to three slices of every
// warp on their way, and a block's place is taken by the next one as soon as it
// is done. On the 64-sequence decode batch (483 MB): 77.3 us, 6.2 TB/s, 92%
// of the measured copy rate (blocks of four warps 77.9); with K read straight
// into registers 92 us (two slices in flight, 16 warps per SM) and 121 us (one
// slice per warp, the chain of dependent reads in front of it exposed). Two
// slots of 256-byte rows a warp beat four by 1.4 us (more warps per SM), and 8
// slices per warp beat 4 and 16 by 2.3.
// 16 keys never cross a page (pages are multiples of 16 keys).
// ---------------------------------------------------------------------------
constexpr int kSlices = kWeightKeys / 16;

template <int D, bool FP8>
struct WwCfg {
  static constexpr int ROW = D * (FP8 ? 1 : 2);            // bytes of a key
  static constexpr int SLOT = 16 * ROW + 64;               // a slice and its old sums
  static constexpr int SLOTS = ROW >= 256 ? 2 : 4;
  static constexpr int SMEM_BYTES = SLOTS * SLOT;
};

// Lengths of sequence s for both kernels: false if the call has nothing to add
// for it. Blocks with `reports` set flag metadata outside the stated bounds.
__device__ __forceinline__ bool weight_lengths(const WeightArgs& a, int s, bool reports, int& q0,
                                               int& q_len, int& kv) {
  q0 = __ldg(a.cu + s);
  const int q1 = __ldg(a.cu + s + 1);
  kv = __ldg(a.seqused_k + s);
  if (q0 < 0 || q1 > a.total_q || q1 < q0 || q1 - q0 > a.max_q) {
    if (reports) flag_status(a.status, PA_DEV_BAD_SEQLEN);
    return false;
  }
  q_len = q1 - q0;
  if (reports && (kv < 0 || kv > a.max_k || kv > a.kv_len_cap))
    flag_status(a.status, PA_DEV_BAD_SEQLEN);
  kv = min(kv, a.kv_len_cap);
  return q_len > 0;
}

template <int D, bool F16, bool FP8>
__global__ void __launch_bounds__(32)
weights_kernel(const __grid_constant__ WeightArgs a, int tiles) {
  using E = Elem<F16>;
  using C = WwCfg<D, FP8>;
  constexpr int NQ = D / 32;                    // 16-byte pieces of a query row per lane
  constexpr int NV = C::ROW / 64;               // of a key row
  static_assert(kSlices <= 32 && kSlices % C::SLOTS == 0, "a lane holds a slice's page id");
  // Beside the tensor-core kernel (see launch_weights_d) one more block, which
  // has no keys, holds this grid's end back until that kernel's.
  if (blockIdx.x == gridDim.x - 1) {
    pdl_wait();
    return;
  }
  extern __shared__ __align__(16) uint8_t ring[];
  // KV head fastest: a page's heads are read at about the same time (13% on
  // the decode batch over all of one head's blocks before the next head's).
  const int unit = blockIdx.x / a.H_kv;
  const int hk = blockIdx.x - unit * a.H_kv;
  const int s = unit / tiles;
  const int lane = threadIdx.x;
  const int g = lane >> 2, c = lane & 3;
  const int base = (unit - s * tiles) * kWeightKeys;
  int q0, q_len, kv;
  if (!weight_lengths(a, s, base == 0 && hk == 0 && lane == 0, q0, q_len, kv)) return;
  if (base >= kv || q_len * a.G > a.tc_min_rows) return;
  const int past = kv - q_len;          // query i is at position past + i
  const int rows = q_len * a.G;
  const int nslices = min(kSlices, (kv - base + 15) >> 4);

  // Lane i: page of slice i (-1: none, or outside the pool), its first row.
  int page_l = -1, row_l = 0;
  if (lane < nslices) {
    const int key0 = base + 16 * lane;
    const int lp = a.bs_shift >= 0 ? key0 >> a.bs_shift : key0 / a.bs;
    row_l = key0 - lp * a.bs;
    page_l = __ldg(a.bt + static_cast<int64_t>(s) * a.bt_stride + lp);
    if (page_l < 0 || page_l >= a.num_blocks) {
      page_l = -1;
      flag_status(a.status, PA_DEV_BAD_PAGE);
    }
  }
  // One group of copies per slice, empty or not: keys g and g + 8, pieces
  // 4 v + c, each to this lane's own places; the old sums (zero for the call's
  // own keys) behind them. Rows past kv are in the page and feed only their
  // own, unwritten sums.
  auto fetch = [&](int i) {
    const int page = __shfl_sync(0xffffffffu, page_l, i & 31);
    const int prow = __shfl_sync(0xffffffffu, row_l, i & 31);
    if (i < nslices && page >= 0) {
      const uint32_t dst = smem_u32(ring + (i % C::SLOTS) * C::SLOT);
      const int64_t rstep = static_cast<int64_t>(a.H_kv) * C::ROW;
      const uint8_t* p = a.kc + page * a.block_stride_bytes + hk * C::ROW + (prow + g) * rstep;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        cp_async16(dst + (2 * v) * 512 + lane * 16, p + (4 * v + c) * 16);
        cp_async16(dst + (2 * v + 1) * 512 + lane * 16, p + 8 * rstep + (4 * v + c) * 16);
      }
      if (lane < 16)
        cp_async4(dst + 16 * C::ROW + lane * 4,
                  a.weights + page * a.weights_stride + static_cast<int64_t>(hk) * a.bs + prow + lane,
                  base + 16 * i + lane < past);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < C::SLOTS - 1; ++i) fetch(i);

  const float sl2 = FP8 ? a.scale_log2 * __ldg(a.k_scale + hk) : a.scale_log2;
  // Queries r .. r + 7 of the packed rows: B fragments (row r + g), and LSE and
  // last visible key of columns r + 2c, r + 2c + 1.
  uint4 qv[NQ];
  float nl[2];
  int lim[2];
  auto load_queries = [&](int r) {
    const int rq = min(r + g, rows - 1);
    const int iq = rq / a.G;
    const uint4* qrow = reinterpret_cast<const uint4*>(
        a.q + static_cast<int64_t>(q0 + iq) * a.q_stride +
        static_cast<int64_t>(hk * a.G + rq - iq * a.G) * D);
#pragma unroll
    for (int v = 0; v < NQ; ++v)
      qv[v] = __ldg(qrow + (FP8 ? 8 * (v >> 1) + 2 * c + (v & 1) : 4 * v + c));
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int re = r + 2 * c + e;
      const int rr = min(re, rows - 1);
      const int i = rr / a.G;
      const float lse =
          __ldg(a.lse + static_cast<int64_t>(hk * a.G + rr - i * a.G) * a.total_q + q0 + i);
      nl[e] = -lse * kLog2e;
      // A row that saw nothing (lse = -inf) or does not exist sees no key here.
      lim[e] = re < rows && lse != -INFINITY ? (a.causal ? past + i : kv - 1) : -1;
    }
  };
  if (rows <= 8) load_queries(0);

#pragma unroll 1
  for (int i = 0; i < nslices; ++i) {
    fetch(i + C::SLOTS - 1);
    cp_async_wait<C::SLOTS - 1>();
    __syncwarp();
    const int page = __shfl_sync(0xffffffffu, page_l, i);
    const int prow = __shfl_sync(0xffffffffu, row_l, i);
    if (page < 0) continue;             // warp-uniform
    const uint8_t* slot = ring + (i % C::SLOTS) * C::SLOT;
    uint4 x0[NV], x1[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      x0[v] = *reinterpret_cast<const uint4*>(slot + (2 * v) * 512 + lane * 16);
      x1[v] = *reinterpret_cast<const uint4*>(slot + (2 * v + 1) * 512 + lane * 16);
    }
    const float* old = reinterpret_cast<const float*>(slot + 16 * C::ROW);
    const float old0 = old[g], old1 = old[g + 8];
    __syncwarp();                       // the slot may be filled again
    const int key0 = base + 16 * i;
    // The first query that sees a key of the slice.
    const int i0 = a.causal ? max(0, key0 - past) : 0;
    float sum[2] = {0.f, 0.f};
    for (int r = rows > 8 ? i0 * a.G : 0; r < rows; r += 8) {
      if (rows > 8) load_queries(r);
      float st[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const uint32_t w0[4] = {x0[v].x, x0[v].y, x0[v].z, x0[v].w};
        const uint32_t w1[4] = {x1[v].x, x1[v].y, x1[v].z, x1[v].w};
        if constexpr (FP8) {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const uint4& q = qv[2 * v + (x >> 1)];
            E::mma(st, widen_e4m3x2<F16>(w0[x]), widen_e4m3x2<F16>(w1[x]),
                   widen_e4m3x2<F16>(w0[x] >> 16), widen_e4m3x2<F16>(w1[x] >> 16),
                   (x & 1) ? q.z : q.x, (x & 1) ? q.w : q.y);
          }
        } else {
          E::mma(st, w0[0], w1[0], w0[1], w1[1], qv[v].x, qv[v].y);
          E::mma(st, w0[2], w1[2], w0[3], w1[3], qv[v].z, qv[v].w);
        }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int j = key0 + g + 8 * x;
        float p = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (j <= lim[e]) p += fast_exp2(fmaf(st[2 * x + e], sl2, nl[e]));
        sum[x] += p;
      }
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      sum[x] += __shfl_xor_sync(0xffffffffu, sum[x], 1);
      sum[x] += __shfl_xor_sync(0xffffffffu, sum[x], 2);
    }
    if (c < 2 && key0 + g + 8 * c < kv)
      a.weights[page * a.weights_stride + static_cast<int64_t>(hk) * a.bs + prow + g + 8 * c] =
          c == 0 ? old0 + sum[0] : old1 + sum[1];
  }
  cp_async_wait<0>();
}

// ---------------------------------------------------------------------------
// Prompts and prompt chunks: the product on the tensor cores (tcgen05), S^T =
// K Q^T. A block owns XT * 128 keys of a sequence and KV head -- XT MMA tiles
// whose M dimension, the TMEM lanes, are keys -- and walks the packed query
// rows that see them in tiles of N = 128 (whole tokens, as in the prefill
// kernel). The sum over queries is then a sum along a lane's columns: a thread
// adds up its own key, without shuffles or shared memory, and K is read once.
//   warp 0       TMA producer: Q tiles into a ring of stages
//   warp 1       MMA issuer: the products (query tile t, key tile X) in order,
//                product n into TMEM buffer n % 3
//   warps 4-15   three warpgroups; the first XT bring a key tile each from its
//                pages into TMEM (e4m3 widened to the MMA's type), then group g
//                takes products g, g + 3, ...: p = exp2(S scale log2(e) - lse
//                log2(e)), summed per thread and key tile.
// K is the MMA's A operand and stays in TMEM: from shared memory it would be
// read again for every query tile, 4 KB beside the 4 KB of Q per 128x128x16
// MMA, which is all that shared memory gives in the MMA's 64 clocks, and the
// copies of Q come on top. XT = 2 halves the read of Q (32 KB per tile at head
// size 128) from L2; at head size 256 K takes the TMEM of both.
// Under a causal mask the first keys of a sequence are seen by all of its
// queries and the last by few: a cluster of `parts` blocks shares a key tile
// (block r takes query tiles r, r + parts, ...) and the first of them adds up
// the parts' sums in order, read from its own shared memory.
// Bound by a block's start -- the key rows, one thread each, into registers and
// TMEM before the first product, about 25 us of 80 for two prompts of
// 2,500-4,096 tokens (32/8 heads of 128) -- and then by the exponentials and
// sums, one FMA, one exponential and one add per score and thread (tensor pipe
// 32%, issue slots 42%).
// Every wait on a barrier in shared memory is bounded; on a timeout the block
// records PA_DEV_TIMEOUT, waits for its copies in flight, frees its TMEM and
// returns, and its keys are not written. (Cluster barriers are reached by every
// thread of the cluster on every path.)
// ---------------------------------------------------------------------------
template <int D>
struct WtCfg {
  static constexpr int XT = D > 128 ? 1 : 2;           // key tiles of a block
  static constexpr int KEYS = XT * 128, COLS = 128;
  static constexpr int HALVES = D / 64;
  static constexpr int HALF = 128 * 128;               // 128 rows of 128 bytes
  static constexpr int TILE = HALVES * HALF;           // a Q tile
  static constexpr int STAGES = D > 128 ? 3 : 4;
  static constexpr int GROUPS = 3;                     // warpgroups that add up, S buffers
  static constexpr int PARTS = 2;                      // largest cluster
  static constexpr int OFF_NL = STAGES * TILE;         // float[GROUPS][2][COLS]
  static constexpr int OFF_SUM = OFF_NL + GROUPS * 2 * COLS * 4;   // float[GROUPS][KEYS]
  static constexpr int OFF_PART = OFF_SUM + GROUPS * KEYS * 4;     // float[PARTS - 1][KEYS]
  static constexpr int OFF_BAR = OFF_PART + (PARTS - 1) * KEYS * 4;
  // At least 120 KB: one block per SM, which owns the SM's tensor memory.
  static constexpr int USED = OFF_BAR + 256 + 1024;
  static constexpr int SMEM_BYTES = USED > 120 * 1024 ? USED : 120 * 1024;
  static constexpr int THREADS = 128 + GROUPS * 128;
  // TMEM columns: K of key tile X at X * D / 2 (two elements a column), S of
  // buffer b at 128 + 128 b.
  static constexpr int S_COL = 128, TMEM_COLS = 512;
  static_assert(XT * D / 2 <= S_COL && S_COL + GROUPS * COLS <= TMEM_COLS, "fits tensor memory");
  static_assert(SMEM_BYTES <= 227 * 1024, "fits shared memory");
};

struct WtBars {
  uint64_t k_full;        // K tiles in TMEM (KEYS arrivals)
  uint64_t q_full[4], q_empty[4];
  uint64_t s_full[3], s_empty[3];   // per S buffer
  uint64_t drain;
  uint32_t tmem_base;
  volatile int abort;
  volatile int issued, consumed;   // Q tiles
  int part_failed[1];              // of the cluster's other block (written by it)
};
static_assert(sizeof(WtBars) <= 256, "the barriers fit their space");

// Barrier `id` of 128 threads: does any of them bring p?
__device__ __forceinline__ bool group_any(int id, bool p) {
  uint32_t any;
  asm volatile("{\n.reg .pred a, b;\nsetp.ne.u32 a, %2, 0;\nbar.red.or.pred b, %1, 128, a;\n"
               "selp.u32 %0, 1, 0, b;\n}"
               : "=r"(any)
               : "r"(id), "r"(static_cast<uint32_t>(p))
               : "memory");
  return any != 0;
}

template <int D, bool F16, bool FP8>
__global__ void __launch_bounds__(WtCfg<D>::THREADS, 1)
weights_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ WeightArgs a,
                  int num_seqs, int parts) {
  using C = WtCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  WtBars* bars = reinterpret_cast<WtBars*>(smem + C::OFF_BAR);
  pdl_trigger();   // the other kernel may start: it takes the other sequences
  // Part fastest, then KV head, sequence, keys: under a causal mask the first
  // keys are seen by the most queries, so blocks start longest first.
  const int unit = blockIdx.x / parts;
  const int part = parts > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int hk = unit % a.H_kv;
  const int ts = unit / a.H_kv;
  const int s = ts % num_seqs;
  const int key0 = ts / num_seqs * C::KEYS;
  int q0, q_len, kv;
  if (!weight_lengths(a, s, false, q0, q_len, kv)) return;   // reported by the other kernel
  if (key0 >= kv || q_len * a.G <= a.tc_min_rows) return;
  const int G = a.G, TR = tc_tile_rows(G), TPT = TR / G;   // rows, tokens of a Q tile
  const int past = kv - q_len;
  const int i0 = a.causal ? max(0, key0 - past) : 0;       // first query that sees a key
  // This block's query tiles: tile t starts at query first + t step.
  const int all_tiles = (q_len - i0 + TPT - 1) / TPT;
  const int ntiles = (all_tiles - part + parts - 1) / parts;
  const int step = parts * TPT, first = i0 + part * TPT;
  // Key tiles of the block that hold keys, and the query tiles that the second
  // one leaves out (none of their queries is at its first key yet).
  const int xt = C::XT == 2 && key0 + 128 < kv ? 2 : 1;
  int skip1 = 0;
  if (C::XT == 2 && a.causal) {
    const int d = key0 + 128 - past - first - TPT;
    skip1 = d >= 0 ? min(ntiles, d / step + 1) : 0;
  }
  // Products in order: query tile after query tile, both key tiles of each
  // (the first skip1 with key tile 0 alone).
  const int alone = xt == 1 ? ntiles : skip1;
  const int nprod = alone + 2 * (ntiles - alone);
  auto tile_of = [&](int n) { return n < alone ? n : alone + ((n - alone) >> 1); };
  auto key_tile_of = [&](int n) { return n < alone ? 0 : (n - alone) & 1; };
  if (parts > 1) cluster_arrive();   // this block has started (see the end)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // The key rows are asked for first: thread `tid` of warpgroup X brings key
  // X * 128 + tid (zeros past the sequence and for pages outside the pool).
  const int wg = (warp - 4) >> 2, tid = threadIdx.x & 127;
  constexpr int EB = FP8 ? 1 : 2;
  constexpr int KV16 = D * EB / 16;                    // 16-byte pieces of a key
  constexpr int KB = KV16 < 16 ? KV16 : 16;            // held at a time
  const uint4* krow = nullptr;
  uint4 kx[KB];
  if (warp >= 4 && wg < C::XT) {
    const int j = key0 + wg * 128 + tid;
    if (j < kv) {
      const int lp = j / a.bs;
      const int page = __ldg(a.bt + static_cast<int64_t>(s) * a.bt_stride + lp);
      if (page >= 0 && page < a.num_blocks)
        krow = reinterpret_cast<const uint4*>(
            a.kc + page * a.block_stride_bytes +
            (static_cast<int64_t>(j - lp * a.bs) * a.H_kv + hk) * (D * EB));
    }
#pragma unroll
    for (int u = 0; u < KB; ++u) kx[u] = krow ? __ldg(krow + u) : make_uint4(0, 0, 0, 0);
  }

  if (threadIdx.x == 0) {
    mbar_init(&bars->k_full, C::KEYS);
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&bars->q_full[i], 1);
      mbar_init(&bars->q_empty[i], 1);
    }
    for (int i = 0; i < C::GROUPS; ++i) {
      mbar_init(&bars->s_full[i], 1);
      mbar_init(&bars->s_empty[i], 128);
    }
    mbar_init(&bars->drain, 1);
    bars->abort = 0;
    bars->issued = bars->consumed = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&bars->tmem_base, C::TMEM_COLS);
    tmem_relinquish();
  }
  // Rows of a Q stage that no copy fills (groups that do not divide 128):
  // zeros, so that their columns are finite.
  if (TR < C::COLS) {
    for (int st = 0; st < C::STAGES; ++st)
      for (int idx = threadIdx.x; idx < (C::COLS - TR) * C::HALVES * 8; idx += C::THREADS) {
        const int r = TR + idx / (C::HALVES * 8), rem = idx % (C::HALVES * 8);
        *reinterpret_cast<uint4*>(smem + st * C::TILE + (rem >> 3) * C::HALF + r * 128 +
                                  (rem & 7) * 16) = make_uint4(0, 0, 0, 0);
      }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  float sum[2] = {0.f, 0.f};   // per key tile

  if (warp == 0) {
    // -------------------------------------------------------------- producer
    if (lane == 0) {
      tma_prefetch_desc(&tmQ);
      for (int t = 0; t < ntiles; ++t) {
        const int st = t % C::STAGES;
        if (t >= C::STAGES && !mbar_wait(&bars->q_empty[st], ((t / C::STAGES) - 1) & 1)) {
          bars->abort = 1;
          break;
        }
        if (bars->abort) break;
        mbar_arrive_expect_tx(&bars->q_full[st], C::HALVES * TR * 128);
        for (int h = 0; h < C::HALVES; ++h)
          tma_load_3d(smem + st * C::TILE + h * C::HALF, &tmQ, &bars->q_full[st], h * 64,
                      hk * G, q0 + first + t * step);
        bars->issued = t + 1;
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp walks the loop and one elected lane issues: with the
    // control flow uniform, descriptors live in uniform registers.
    constexpr uint32_t idesc = mma_idesc(128, C::COLS, false, Elem<F16>::kTcFormat);
    const uint32_t lead = elect_one();
    const uint64_t qdesc = smem_desc_sw128(smem_u32(smem), 16, 1024);
    bool ok = __all_sync(0xffffffffu, mbar_wait(&bars->k_full, 0));
    tc_fence_after();
    for (int n = 0, b = 0, use = 0; ok && n < nprod; ++n) {
      const int t = tile_of(n), x = key_tile_of(n);
      const int st = t % C::STAGES;
      if (x == 0) {
        ok = __all_sync(0xffffffffu,
                        !bars->abort && mbar_wait(&bars->q_full[st], (t / C::STAGES) & 1));
        if (!ok) break;
        if (lane == 0) bars->consumed = t + 1;
      }
      ok = __all_sync(0xffffffffu, use == 0 || mbar_wait(&bars->s_empty[b], (use - 1) & 1));
      if (!ok) break;
      tc_fence_after();
      const uint64_t qd = qdesc + static_cast<uint32_t>(st * (C::TILE >> 4));
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = ((kk >> 2) * C::HALF + (kk & 3) * 32) >> 4;
        tc_mma_ts_if(lead, tmem + C::S_COL + b * C::COLS, tmem + x * (D / 2) + kk * 8, qd + off,
                     idesc, kk > 0);
      }
      tc_commit_if(lead, &bars->s_full[b]);
      if (x == 1 || n < alone) tc_commit_if(lead, &bars->q_empty[st]);   // the tile's last product
      if (++b == C::GROUPS) b = 0, ++use;
    }
    if (!ok) {
      bars->abort = 1;
      tc_commit_if(lead, &bars->drain);   // arrives once every MMA issued above has completed
      mbar_wait(&bars->drain, 0);
    }
  } else if (warp >= 4) {
    // -------------------------------------------------------- K tiles, sums
    const uint32_t tm_row = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    if (wg < C::XT) {
      // Row tid of key tile wg: element pairs 2c, 2c + 1 in column c.
#pragma unroll
      for (int u0 = 0; u0 < KV16; u0 += KB) {
        if (u0 > 0) {
#pragma unroll
          for (int u = 0; u < KB; ++u)
            kx[u] = krow ? __ldg(krow + u0 + u) : make_uint4(0, 0, 0, 0);
        }
        constexpr int W = FP8 ? 8 : 4;                 // columns of 16 bytes
#pragma unroll
        for (int c0 = 0; c0 < KB * W; c0 += 32) {
          uint32_t v[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const uint4& x = kx[(c0 + c) / W];
            const uint32_t word[4] = {x.x, x.y, x.z, x.w};
            if constexpr (FP8) {
              const uint32_t two = word[((c0 + c) % W) / 2];
              v[c] = widen_e4m3x2<F16>((c & 1) ? two >> 16 : two);
            } else {
              v[c] = word[(c0 + c) % W];
            }
          }
          tmem_st32(tm_row + wg * (D / 2) + u0 * W + c0, v);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&bars->k_full);
    }
    const uint32_t tm = tm_row + C::S_COL + wg * C::COLS;
    float* nl = reinterpret_cast<float*>(smem + C::OFF_NL) + wg * 2 * C::COLS;
    const float sl2 = FP8 ? a.scale_log2 * __ldg(a.k_scale + hk) : a.scale_log2;
    // This thread also fetches the LSE of column tid: token tid / G of a tile.
    const int ctok = tid / G;
    const float* lse_row = a.lse + static_cast<int64_t>(hk * G + tid - ctok * G) * a.total_q + q0;
    auto fetch = [&](int t) -> float {
      const int i = first + t * step + ctok;
      if (tid >= TR || i >= q_len) return -INFINITY;
      const float v = __ldg(lse_row + i);
      return v == -INFINITY ? -INFINITY : -v * kLog2e;   // a row that saw nothing adds nothing
    };
    float next = wg < nprod ? fetch(tile_of(wg)) : 0.f;
    float acc[4];
    auto sum_tile = [&](const float* nlb, int c0, int c1, auto mask) {
#pragma unroll
      for (int c = 0; c < C::COLS / 32; ++c) {
        uint32_t v[32];
        tmem_ld32(tm + c * 32, v);
        tmem_wait_ld();
        if (c == C::COLS / 32 - 1) {
          tc_fence_before();
          mbar_arrive(&bars->s_empty[wg]);
        }
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 n4 = *reinterpret_cast<const float4*>(nlb + c * 32 + e);
          float y[4];
          ffma2(y[0], y[1], __uint_as_float(v[e]), __uint_as_float(v[e + 1]), sl2, sl2, n4.x, n4.y);
          ffma2(y[2], y[3], __uint_as_float(v[e + 2]), __uint_as_float(v[e + 3]), sl2, sl2, n4.z,
                n4.w);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            y[k] = fast_exp2(y[k]);
            if constexpr (decltype(mask)::value > 0) {
              const int col = c * 32 + e + k;
              y[k] = col >= c0 && col < c1 ? y[k] : 0.f;
            }
            if constexpr (decltype(mask)::value > 1) {
              const float nk = k == 0 ? n4.x : k == 1 ? n4.y : k == 2 ? n4.z : n4.w;
              y[k] = nk != -INFINITY ? y[k] : 0.f;
            }
          }
          fadd2(acc[0], acc[1], acc[0], acc[1], y[0], y[1]);
          fadd2(acc[2], acc[3], acc[2], acc[3], y[2], y[3]);
        }
      }
    };
    bool ok = true;
    for (int n = wg, it = 0; n < nprod; n += C::GROUPS, ++it) {
      const int t = tile_of(n), x = key_tile_of(n);
      float* nlb = nl + (it & 1) * C::COLS;
      nlb[tid] = next;
      // (A query that saw nothing may hold anything: its products are dropped
      // by a select, not by the exponential.)
      const bool blind = group_any(1 + wg, tid < TR && next == -INFINITY);
      if (n + C::GROUPS < nprod) next = fetch(tile_of(n + C::GROUPS));
      // Columns [c0, c1) of the tile see this key: queries from its own
      // position on, rows of the sequence.
      const int tok0 = first + t * step;
      // (A key far in front of the queries: clamped in tokens, since keys x heads
      // of the group may pass 32 bits. The other side is at most 255 tokens.)
      const int c0 = a.causal ? max(0, key0 + x * 128 + tid - past - tok0) * G : 0;
      const int c1 = min(TR, (q_len - tok0) * G);
      const bool edge =
          tok0 + TPT > q_len || (a.causal && tok0 < key0 + x * 128 + 127 - past);
      // A warp whose wait gave up goes on through the group's barriers without
      // work, so that no other warp waits for it.
      if (ok) ok = !bars->abort && mbar_wait(&bars->s_full[wg], it & 1);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) {
        bars->abort = 1;
        continue;
      }
      tc_fence_after();
      acc[0] = acc[1] = acc[2] = acc[3] = 0.f;
      // Three bodies, so that a tile that every key sees whole pays no select
      // (one for all: 4 us of 84 on two prompts of 2,500-4,096 tokens).
      if (blind)
        sum_tile(nlb, c0, c1, std::integral_constant<int, 2>{});
      else if (edge)
        sum_tile(nlb, c0, c1, std::integral_constant<int, 1>{});
      else
        sum_tile(nlb, c0, c1, std::integral_constant<int, 0>{});
      const float got = (acc[0] + acc[1]) + (acc[2] + acc[3]);
      sum[0] += x == 0 ? got : 0.f;
      sum[1] += x == 0 ? 0.f : got;
    }
    float* mine = reinterpret_cast<float*>(smem + C::OFF_SUM) + wg * C::KEYS + tid;
    mine[0] = sum[0];
    if (C::XT == 2) mine[128] = sum[1];
  }

  // ---------------------------------------------------------------- teardown
  tc_fence_before();
  __syncthreads();
  bool failed = bars->abort != 0;
  if (threadIdx.x == 0 && failed) {
    flag_status(a.status, PA_DEV_TIMEOUT);
    for (int t = bars->consumed; t < bars->issued; ++t)
      if (!mbar_wait(&bars->q_full[t % C::STAGES], (t / C::STAGES) & 1)) break;
  }
  // One thread per key goes on.
  const int key = static_cast<int>(threadIdx.x) - 128;
  const bool adds = key >= 0 && key < C::KEYS;
  float total = 0.f;
  if (adds)
    for (int g = 0; g < C::GROUPS; ++g)
      total += reinterpret_cast<const float*>(smem + C::OFF_SUM)[g * C::KEYS + key];
  float* others = reinterpret_cast<float*>(smem + C::OFF_PART);
  if (parts > 1) {
    // Every block of the cluster has started (its shared memory is there);
    // the sums go to block 0; block 0 sees them, and nobody leaves before.
    cluster_wait();
    if (part > 0) {
      if (adds) store_remote(others + (part - 1) * C::KEYS + key, 0, __float_as_uint(total));
      if (threadIdx.x == 0) store_remote(&bars->part_failed[part - 1], 0, failed);
    }
    cluster_arrive();
    cluster_wait();
    if (part == 0)
      for (int r = 1; r < parts; ++r) failed |= bars->part_failed[r - 1] != 0;
  }
  if (!failed && adds && part == 0) {
    const int j = key0 + key;
    if (j < kv) {
      const int lp = j / a.bs;
      const int page = __ldg(a.bt + static_cast<int64_t>(s) * a.bt_stride + lp);
      if (page >= 0 && page < a.num_blocks) {
        for (int r = 1; r < parts; ++r) total += others[(r - 1) * C::KEYS + key];
        float* w = a.weights + page * a.weights_stride + static_cast<int64_t>(hk) * a.bs +
                   (j - lp * a.bs);
        *w = (j >= past ? 0.f : *w) + total;
      } else {
        flag_status(a.status, PA_DEV_BAD_PAGE);
      }
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

template <int D, bool F16, bool FP8>
static cudaError_t launch_weights_d(const CUtensorMap& tmQ, const WeightArgs& a, int num_seqs,
                                    int keys, cudaStream_t st, int sms) {
  const int tiles = keys > 0 ? (keys + kWeightKeys - 1) / kWeightKeys : 1;
  bool tc = false;   // the tensor-core kernel was launched
  if (a.tc_min_rows < 0x7fffffff) {
    using C = WtCfg<D>;
    static std::atomic<bool> configured_tc[kMaxDevices];
    cudaError_t e =
        opt_in_smem(weights_tc_kernel<D, F16, FP8>, C::SMEM_BYTES, configured_tc);
    if (e != cudaSuccess) return e;
    const long long units =
        static_cast<long long>((keys + C::KEYS - 1) / C::KEYS) * num_seqs * a.H_kv;
    if (units > 0) {
      // Fewer than two key tiles per SM: two blocks share each, which halves
      // the longest block. 8 KV heads, prompts of 2,500-4,096 tokens: one
      // prompt of 4,096 (128 tiles of 256 keys) 74.0 us in pairs against 123.8;
      // two (184) 85.3 against 96.5; four (about 400) 163 against 147; sixteen
      // 755 against 647.
      const int parts = units < 2LL * sms ? 2 : 1;
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(static_cast<unsigned>(units * parts));
      cfg.blockDim = dim3(C::THREADS);
      cfg.dynamicSmemBytes = C::SMEM_BYTES;
      cfg.stream = st;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = parts;
      attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = parts > 1 ? 1 : 0;
      e = cudaLaunchKernelEx(&cfg, weights_tc_kernel<D, F16, FP8>, tmQ, a, num_seqs, parts);
      if (e != cudaSuccess) return e;
      e = cudaGetLastError();
      if (e != cudaSuccess) return e;
      tc = true;
    }
  }
  using W = WwCfg<D, FP8>;
  static std::atomic<bool> configured[kMaxDevices];
  cudaError_t e = opt_in_smem(weights_kernel<D, F16, FP8>, W::SMEM_BYTES, configured);
  if (e != cudaSuccess) return e;
  // Behind the tensor-core kernel as its programmatic dependent: the two add
  // to different sequences' keys, so the blocks of one fill in beside the
  // other's, or find nothing to do while it runs.
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(num_seqs) * tiles * a.H_kv + 1u);
  cfg.blockDim = dim3(32);
  cfg.dynamicSmemBytes = W::SMEM_BYTES;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = tc ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, weights_kernel<D, F16, FP8>, a, tiles);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

cudaError_t launch_attn_weights(const CUtensorMap& tmQ, const WeightArgs& a, int num_seqs, int D,
                                bool f16, bool fp8, cudaStream_t st, int sms) {
  const int keys = a.max_k < a.kv_len_cap ? a.max_k : a.kv_len_cap;
  if (fp8) return f16 ? launch_weights_d<128, true, true>(tmQ, a, num_seqs, keys, st, sms)
                      : launch_weights_d<128, false, true>(tmQ, a, num_seqs, keys, st, sms);
  if (f16) {
    if (D == 256) return launch_weights_d<256, true, false>(tmQ, a, num_seqs, keys, st, sms);
    if (D == 128) return launch_weights_d<128, true, false>(tmQ, a, num_seqs, keys, st, sms);
    return launch_weights_d<64, true, false>(tmQ, a, num_seqs, keys, st, sms);
  }
  if (D == 256) return launch_weights_d<256, false, false>(tmQ, a, num_seqs, keys, st, sms);
  if (D == 128) return launch_weights_d<128, false, false>(tmQ, a, num_seqs, keys, st, sms);
  return launch_weights_d<64, false, false>(tmQ, a, num_seqs, keys, st, sms);
}

}  // namespace pa
