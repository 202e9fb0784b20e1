// Accumulated attention weight of every cached key: the column sums of the
// attention matrix, w_j += sum_i exp(scale q_i.k_j - lse_i), recomputed from
// K and the LSE that the attention call returned (the matrix itself never
// exists in memory). Each key has one owner, so there are no atomics and the
// sums are the same bits on every run.
#include <cuda_runtime.h>

#include <atomic>

#include "device_common.cuh"

namespace pa {

// ---------------------------------------------------------------------------
// Decode and short queries (at most tc_min_rows packed query rows).
// One warp per 16 keys of a sequence and KV head. The keys are the M
// dimension of the warp MMA and 8 packed query rows (token, head of the
// group) its N, so a key's sum is a sum along the accumulator's columns: no
// reduction until the end, where the four lanes of a row add up. K goes from
// global memory straight to the A fragments (held for all query rows) and Q
// straight to the B fragments: the head dimension is permuted alike in both
// so that a lane's elements are 16-byte runs and four lanes read 64
// consecutive bytes. No shared memory, no barriers: at 4 warps a block and 8
// loads in flight per lane, decode is bound by the read of K.
// 16 keys never cross a page (pages are multiples of 16 keys).
// ---------------------------------------------------------------------------
constexpr int kWeightWarps = 4;

// Two e4m3 bytes as a pair of the MMA's element type (exact in both).
template <bool F16>
__device__ __forceinline__ uint32_t widen_e4m3x2(uint32_t two) {
  const uint32_t h = e4m3x2_to_f16x2(two);
  if constexpr (F16) {
    return h;
  } else {
    const float2 f = Elem<true>::unpack(h);
    return Elem<false>::pack(f.x, f.y);
  }
}

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
__global__ void __launch_bounds__(kWeightWarps * 32)
weights_kernel(const __grid_constant__ WeightArgs a, int tiles) {
  using E = Elem<F16>;
  constexpr int DK = D / 16;        // k-steps
  const int s = blockIdx.x / tiles;
  const int hk = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const int key0 = ((blockIdx.x - s * tiles) * kWeightWarps + warp) * 16;
  int q0, q_len, kv;
  if (!weight_lengths(a, s, key0 == 0 && hk == 0 && lane == 0, q0, q_len, kv)) return;
  if (key0 >= kv || q_len * a.G > a.tc_min_rows) return;
  const int lp = key0 / a.bs;
  const int page = __ldg(a.bt + static_cast<int64_t>(s) * a.bt_stride + lp);
  if (page < 0 || page >= a.num_blocks) {
    if (lane == 0) flag_status(a.status, PA_DEV_BAD_PAGE);
    return;
  }
  const int prow = key0 - lp * a.bs;   // the slice's first row of the page

  // A fragments: keys key0 + g and key0 + g + 8 (rows past kv are in the page
  // and feed only their own, unwritten sums).
  uint32_t kf[DK][4];
  {
    constexpr int E16 = FP8 ? 16 : 8;   // elements of 16 bytes
    constexpr int row_bytes = D * (FP8 ? 1 : 2);
    const uint8_t* base = a.kc + page * a.block_stride_bytes +
                          (static_cast<int64_t>(prow) * a.H_kv + hk) * row_bytes;
    const int64_t rstep = static_cast<int64_t>(a.H_kv) * row_bytes;
    const uint4* p0 = reinterpret_cast<const uint4*>(base + g * rstep);
    const uint4* p1 = reinterpret_cast<const uint4*>(base + (g + 8) * rstep);
    constexpr int NV = D / (4 * E16);
    uint4 x0[NV], x1[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      x0[v] = __ldg(p0 + 4 * v + c);
      x1[v] = __ldg(p1 + 4 * v + c);
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const uint32_t w0[4] = {x0[v].x, x0[v].y, x0[v].z, x0[v].w};
      const uint32_t w1[4] = {x1[v].x, x1[v].y, x1[v].z, x1[v].w};
      if constexpr (FP8) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          kf[4 * v + k][0] = widen_e4m3x2<F16>(w0[k]);
          kf[4 * v + k][1] = widen_e4m3x2<F16>(w1[k]);
          kf[4 * v + k][2] = widen_e4m3x2<F16>(w0[k] >> 16);
          kf[4 * v + k][3] = widen_e4m3x2<F16>(w1[k] >> 16);
        }
      } else {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          kf[2 * v + k][0] = w0[2 * k];
          kf[2 * v + k][1] = w1[2 * k];
          kf[2 * v + k][2] = w0[2 * k + 1];
          kf[2 * v + k][3] = w1[2 * k + 1];
        }
      }
    }
  }
  const float sl2 = FP8 ? a.scale_log2 * __ldg(a.k_scale + hk) : a.scale_log2;
  const int past = kv - q_len;          // query i is at position past + i
  const int rows = q_len * a.G;
  // The first query that sees a key of the slice.
  const int i0 = a.causal ? max(0, key0 - past) : 0;
  float sum[2] = {0.f, 0.f};
  for (int r = i0 * a.G; r < rows; r += 8) {
    // B fragments: packed row r + g.
    const int rq = min(r + g, rows - 1);
    const int iq = rq / a.G;
    const uint4* qrow = reinterpret_cast<const uint4*>(
        a.q + static_cast<int64_t>(q0 + iq) * a.q_stride +
        static_cast<int64_t>(hk * a.G + rq - iq * a.G) * D);
    uint4 qv[D / 32];
#pragma unroll
    for (int v = 0; v < D / 32; ++v)
      qv[v] = __ldg(qrow + (FP8 ? 8 * (v >> 1) + 2 * c + (v & 1) : 4 * v + c));
    // Columns r + 2c and r + 2c + 1: their LSE and last visible key.
    float nl[2];
    int lim[2];
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
    float st[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int v = 0; v < D / 32; ++v) {
      E::mma(st, kf[2 * v][0], kf[2 * v][1], kf[2 * v][2], kf[2 * v][3], qv[v].x, qv[v].y);
      E::mma(st, kf[2 * v + 1][0], kf[2 * v + 1][1], kf[2 * v + 1][2], kf[2 * v + 1][3], qv[v].z,
             qv[v].w);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int j = key0 + g + 8 * k;
      float p = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (j <= lim[e]) p += fast_exp2(fmaf(st[2 * k + e], sl2, nl[e]));
      sum[k] += p;
    }
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], 1);
    sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], 2);
    const int j = key0 + g + 8 * k;
    if (c == 0 && j < kv) {
      float* w = a.weights + page * a.weights_stride + static_cast<int64_t>(hk) * a.bs + prow + g +
                 8 * k;
      *w = (j >= past ? 0.f : *w) + sum[k];
    }
  }
}

// ---------------------------------------------------------------------------
// Prompts and prompt chunks: the product on the tensor cores (tcgen05), S^T =
// K Q^T. A block owns 128 keys of a sequence and KV head -- the M dimension,
// one TMEM lane each -- and walks the packed query rows that see them in tiles
// of N = 128 (whole tokens, as in the prefill kernel). The sum over queries is
// then a sum along a lane's columns: a thread adds up its own key, without
// shuffles or shared memory, and K is read once.
//   warp 0        TMA producer: Q tiles into a ring of stages
//   warp 1        MMA issuer (one lane): S^T of tile t into TMEM buffer t % 2
//   warps 4-11    two warpgroups; they first bring the K tile into shared
//                 memory (plain loads through the block table, e4m3 widened to
//                 the MMA's type), then group g takes tiles g, g + 2, ...:
//                 p = exp2(S scale log2(e) - lse log2(e)), summed per thread.
// Bound by the exponentials (16 per clock and SM: 1024 clocks per tile against
// 620 for its MMAs); two blocks per SM cover each other's start and end. Every
// wait is bounded; on a timeout the block records PA_DEV_TIMEOUT, waits for its
// copies in flight, frees its TMEM and returns without writing.
// ---------------------------------------------------------------------------
template <int D>
struct WtCfg {
  static constexpr int KEYS = 128, COLS = 128;
  static constexpr int HALVES = D / 64;
  static constexpr int HALF = 128 * 128;               // 128 rows of 128 bytes
  static constexpr int TILE = HALVES * HALF;
  static constexpr int STAGES = D == 64 ? 4 : 2;
  static constexpr int OFF_Q = TILE;                   // K tile first
  static constexpr int OFF_NL = OFF_Q + STAGES * TILE; // float[2 groups][2][COLS]
  static constexpr int OFF_SUM = OFF_NL + 4 * COLS * 4;
  static constexpr int OFF_BAR = OFF_SUM + KEYS * 4;
  static constexpr int SMEM_BYTES = OFF_BAR + 256 + 1024;
  static constexpr int THREADS = 384;
  static constexpr int BLOCKS = D > 128 ? 1 : 2;       // per SM (shared memory, TMEM)
  static constexpr int TMEM_COLS = 2 * COLS;
};
static_assert(2 * WtCfg<128>::SMEM_BYTES <= 226 * 1024, "two blocks fit an SM");
static_assert(2 * WtCfg<64>::SMEM_BYTES <= 226 * 1024 && 3 * WtCfg<64>::SMEM_BYTES > 228 * 1024,
              "two blocks (512 TMEM columns), not three, fit an SM");
static_assert(WtCfg<256>::SMEM_BYTES <= 227 * 1024, "head size 256 fits shared memory");

struct WtBars {
  uint64_t k_full;        // K tile in shared memory (256 arrivals)
  uint64_t q_full[4], q_empty[4];
  uint64_t s_full[2], s_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  volatile int abort;
  volatile int issued, consumed;   // Q tiles
};

template <int D, bool F16, bool FP8>
__global__ void __launch_bounds__(WtCfg<D>::THREADS, WtCfg<D>::BLOCKS)
weights_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ WeightArgs a,
                  int num_seqs) {
  using C = WtCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  WtBars* bars = reinterpret_cast<WtBars*>(smem + C::OFF_BAR);
  // KV head fastest, then sequence, then key tile: under a causal mask the
  // first keys are seen by the most queries, so blocks start longest first.
  const int hk = blockIdx.x % a.H_kv;
  const int ts = blockIdx.x / a.H_kv;
  const int s = ts % num_seqs;
  const int key0 = ts / num_seqs * C::KEYS;
  int q0, q_len, kv;
  if (!weight_lengths(a, s, false, q0, q_len, kv)) return;   // reported by the other kernel
  if (key0 >= kv || q_len * a.G <= a.tc_min_rows) return;
  const int G = a.G, TR = tc_tile_rows(G), TPT = TR / G;   // rows, tokens of a Q tile
  const int past = kv - q_len;
  const int i0 = a.causal ? max(0, key0 - past) : 0;       // first query that sees a key
  const int ntiles = (q_len - i0 + TPT - 1) / TPT;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(&bars->k_full, 256);
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&bars->q_full[i], 1);
      mbar_init(&bars->q_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
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
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  float sum = 0.f;
  bool ok = true;

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
          tma_load_3d(smem + C::OFF_Q + st * C::TILE + h * C::HALF, &tmQ, &bars->q_full[st], h * 64,
                      hk * G, q0 + i0 + t * TPT);
        bars->issued = t + 1;
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc = mma_idesc(C::KEYS, C::COLS, false, Elem<F16>::kTcFormat);
      const uint64_t kdesc = smem_desc_sw128(smem_u32(smem), 16, 1024);
      const uint64_t qdesc = smem_desc_sw128(smem_u32(smem + C::OFF_Q), 16, 1024);
      ok = mbar_wait(&bars->k_full, 0);
      for (int t = 0; ok && t < ntiles; ++t) {
        const int st = t % C::STAGES, b = t & 1;
        if (bars->abort) { ok = false; break; }
        if (!(ok = mbar_wait(&bars->q_full[st], (t / C::STAGES) & 1))) break;
        bars->consumed = t + 1;
        if (t >= 2 && !(ok = mbar_wait(&bars->s_empty[b], ((t >> 1) - 1) & 1))) break;
        tc_fence_after();
        const uint64_t qd = qdesc + static_cast<uint32_t>(st * (C::TILE >> 4));
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * C::HALF + (kk & 3) * 32) >> 4;
          tc_mma(tmem + b * C::COLS, kdesc + off, qd + off, idesc, kk > 0);
        }
        tc_commit(&bars->s_full[b]);
        tc_commit(&bars->q_empty[st]);
      }
      if (!ok) {
        bars->abort = 1;
        tc_commit(&bars->drain);   // arrives once every MMA issued above has completed
        mbar_wait(&bars->drain, 0);
      }
    }
  } else if (warp >= 4) {
    // -------------------------------------------------------- K tile, sums
    const int et = threadIdx.x - 128;      // 0 .. 255
    const int32_t* bt = a.bt + static_cast<int64_t>(s) * a.bt_stride;
    {
      constexpr int EB = FP8 ? 1 : 2;
      constexpr int CPR = D * EB / 16;     // 16-byte chunks of a key
      for (int idx = et; idx < C::KEYS * CPR; idx += 256) {
        const int r = idx / CPR, c = idx % CPR;
        const int j = key0 + r;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (j < kv) {
          const int lp = j / a.bs;
          const int page = __ldg(bt + lp);
          if (page >= 0 && page < a.num_blocks)
            x = __ldg(reinterpret_cast<const uint4*>(
                          a.kc + page * a.block_stride_bytes +
                          (static_cast<int64_t>(j - lp * a.bs) * a.H_kv + hk) * (D * EB)) +
                      c);
        }
        auto store = [&](int chunk, const uint4& y) {
          *reinterpret_cast<uint4*>(smem + (chunk >> 3) * C::HALF + r * 128 +
                                    (((chunk & 7) ^ (r & 7)) << 4)) = y;
        };
        if constexpr (FP8) {
          store(2 * c, make_uint4(widen_e4m3x2<F16>(x.x), widen_e4m3x2<F16>(x.x >> 16),
                                  widen_e4m3x2<F16>(x.y), widen_e4m3x2<F16>(x.y >> 16)));
          store(2 * c + 1, make_uint4(widen_e4m3x2<F16>(x.z), widen_e4m3x2<F16>(x.z >> 16),
                                      widen_e4m3x2<F16>(x.w), widen_e4m3x2<F16>(x.w >> 16)));
        } else {
          store(c, x);
        }
      }
      // Rows of a Q stage that no copy fills (groups that do not divide 128):
      // zeros, so that their columns are finite.
      for (int st = 0; st < C::STAGES; ++st)
        for (int idx = et; idx < (C::COLS - TR) * C::HALVES * 8; idx += 256) {
          const int r = TR + idx / (C::HALVES * 8), rem = idx % (C::HALVES * 8);
          *reinterpret_cast<uint4*>(smem + C::OFF_Q + st * C::TILE + (rem >> 3) * C::HALF +
                                    r * 128 + (rem & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(&bars->k_full);
    }
    const int grp = (warp - 4) >> 2;       // warpgroup: tiles grp, grp + 2, ...
    const int tid = et & 127;              // TMEM lane: key key0 + tid
    const uint32_t tm = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + grp * C::COLS;
    float* nl = reinterpret_cast<float*>(smem + C::OFF_NL) + grp * 2 * C::COLS;
    const float sl2 = FP8 ? a.scale_log2 * __ldg(a.k_scale + hk) : a.scale_log2;
    // This thread also fetches the LSE of column tid: token tid / G of a tile.
    const int ctok = tid / G;
    const float* lse_row = a.lse + static_cast<int64_t>(hk * G + tid - ctok * G) * a.total_q + q0;
    auto fetch = [&](int t) -> float {
      const int i = i0 + t * TPT + ctok;
      if (tid >= TR || i >= q_len) return -INFINITY;
      const float v = __ldg(lse_row + i);
      return v == -INFINITY ? -INFINITY : -v * kLog2e;   // a row that saw nothing adds nothing
    };
    float next = grp < ntiles ? fetch(grp) : 0.f;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int t = grp, it = 0; t < ntiles; t += 2, ++it) {
      float* nlb = nl + (it & 1) * C::COLS;
      nlb[tid] = next;
      asm volatile("bar.sync %0, 128;" ::"r"(1 + grp) : "memory");
      if (t + 2 < ntiles) next = fetch(t + 2);
      // Columns [c0, c1) of the tile see this key: queries from its own
      // position on, rows of the sequence.
      const int tok0 = i0 + t * TPT;
      const int c0 = a.causal ? max(0, (key0 + tid - past - tok0) * G) : 0;
      const int c1 = min(TR, (q_len - tok0) * G);
      const bool edge = tok0 + TPT > q_len || (a.causal && tok0 < key0 + C::KEYS - 1 - past);
      // A warp whose wait gave up goes on through the group's barriers without
      // work, so that no other warp waits for it.
      if (ok) ok = !bars->abort && mbar_wait(&bars->s_full[grp], it & 1);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) {
        bars->abort = 1;
        continue;
      }
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < C::COLS / 32; ++c) {
        uint32_t v[32];
        tmem_ld32(tm + c * 32, v);
        tmem_wait_ld();
        if (c == C::COLS / 32 - 1) {
          tc_fence_before();
          mbar_arrive(&bars->s_empty[grp]);
        }
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 n4 = *reinterpret_cast<const float4*>(nlb + c * 32 + e);
          float y0, y1, y2, y3;
          ffma2(y0, y1, __uint_as_float(v[e]), __uint_as_float(v[e + 1]), sl2, sl2, n4.x, n4.y);
          ffma2(y2, y3, __uint_as_float(v[e + 2]), __uint_as_float(v[e + 3]), sl2, sl2, n4.z, n4.w);
          float p0 = fast_exp2(y0), p1 = fast_exp2(y1), p2 = fast_exp2(y2), p3 = fast_exp2(y3);
          if (edge) {
            const int col = c * 32 + e;
            p0 = col >= c0 && col < c1 ? p0 : 0.f;
            p1 = col + 1 >= c0 && col + 1 < c1 ? p1 : 0.f;
            p2 = col + 2 >= c0 && col + 2 < c1 ? p2 : 0.f;
            p3 = col + 3 >= c0 && col + 3 < c1 ? p3 : 0.f;
          }
          fadd2(acc[0], acc[1], acc[0], acc[1], p0, p1);
          fadd2(acc[2], acc[3], acc[2], acc[3], p2, p3);
        }
      }
      sum += (acc[0] + acc[1]) + (acc[2] + acc[3]);
      acc[0] = acc[1] = acc[2] = acc[3] = 0.f;
    }
    if (grp == 1) reinterpret_cast<float*>(smem + C::OFF_SUM)[tid] = sum;
  }

  // ---------------------------------------------------------------- teardown
  tc_fence_before();
  __syncthreads();
  const bool failed = bars->abort != 0;
  if (threadIdx.x == 0 && failed) {
    flag_status(a.status, PA_DEV_TIMEOUT);
    for (int t = bars->consumed; t < bars->issued; ++t)
      if (!mbar_wait(&bars->q_full[t % C::STAGES], (t / C::STAGES) & 1)) break;
  }
  if (!failed && warp >= 4 && warp < 8) {
    const int j = key0 + threadIdx.x - 128;
    if (j < kv) {
      const int lp = j / a.bs;
      const int page = __ldg(a.bt + static_cast<int64_t>(s) * a.bt_stride + lp);
      if (page >= 0 && page < a.num_blocks) {
        float* w = a.weights + page * a.weights_stride + static_cast<int64_t>(hk) * a.bs +
                   (j - lp * a.bs);
        *w = (j >= past ? 0.f : *w) +
             (sum + reinterpret_cast<const float*>(smem + C::OFF_SUM)[threadIdx.x - 128]);
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
                                    int keys, cudaStream_t st) {
  constexpr int kTileKeys = kWeightWarps * 16;
  const int tiles = keys > 0 ? (keys + kTileKeys - 1) / kTileKeys : 1;
  if (a.tc_min_rows < 0x7fffffff) {
    using C = WtCfg<D>;
    // A per-device function attribute: set on the first launch on each device
    // (before any stream capture), not again.
    static std::atomic<bool> configured[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool known = dev >= 0 && dev < kMaxDevices;
    if (!known || !configured[dev].load(std::memory_order_acquire)) {
      e = cudaFuncSetAttribute(weights_tc_kernel<D, F16, FP8>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
      if (e != cudaSuccess) return e;
      if (known) configured[dev].store(true, std::memory_order_release);
    }
    const long long blocks =
        static_cast<long long>((keys + C::KEYS - 1) / C::KEYS) * num_seqs * a.H_kv;
    if (blocks > 0) {
      weights_tc_kernel<D, F16, FP8>
          <<<static_cast<unsigned>(blocks), C::THREADS, C::SMEM_BYTES, st>>>(tmQ, a, num_seqs);
      e = cudaGetLastError();
      if (e != cudaSuccess) return e;
    }
  }
  weights_kernel<D, F16, FP8>
      <<<dim3(static_cast<unsigned>(num_seqs) * tiles, a.H_kv), kWeightWarps * 32, 0, st>>>(a,
                                                                                            tiles);
  return cudaGetLastError();
}

cudaError_t launch_attn_weights(const CUtensorMap& tmQ, const WeightArgs& a, int num_seqs, int D,
                                bool f16, bool fp8, cudaStream_t st) {
  const int keys = a.max_k < a.kv_len_cap ? a.max_k : a.kv_len_cap;
  if (fp8) return f16 ? launch_weights_d<128, true, true>(tmQ, a, num_seqs, keys, st)
                      : launch_weights_d<128, false, true>(tmQ, a, num_seqs, keys, st);
  if (f16) {
    if (D == 256) return launch_weights_d<256, true, false>(tmQ, a, num_seqs, keys, st);
    if (D == 128) return launch_weights_d<128, true, false>(tmQ, a, num_seqs, keys, st);
    return launch_weights_d<64, true, false>(tmQ, a, num_seqs, keys, st);
  }
  if (D == 256) return launch_weights_d<256, false, false>(tmQ, a, num_seqs, keys, st);
  if (D == 128) return launch_weights_d<128, false, false>(tmQ, a, num_seqs, keys, st);
  return launch_weights_d<64, false, false>(tmQ, a, num_seqs, keys, st);
}

}  // namespace pa
