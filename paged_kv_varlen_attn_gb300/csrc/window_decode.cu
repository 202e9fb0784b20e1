// Decode under a sliding window with first tokens: out = softmax(scale q.k) v
// over the keys j <= p with j > p - window or j < first, for sequences of at
// most kWinRows packed query rows (tokens x heads of the group).
#include <cuda_runtime.h>

#include "device_common.cuh"

namespace pa {

// ---------------------------------------------------------------------------
// A window leaves every sequence about the same few hundred to few thousand
// keys, known to the host up to their offset, so nothing is planned on the
// device: a cluster of `parts` blocks takes a (sequence, KV head), its warps
// take equal runs of the visible keys in slices of 16 (a slice never crosses a
// page), and nothing but the plain launch stands before the first read.
// A warp streams K and V slices through a ring of its own, filled by
// asynchronous copies and drained with no barrier but the warp's:
//   S^T[16 keys x 8 rows] = K Q^T      keys on the MMA's M side; K and Q with
//     the head dimension permuted alike, so that every lane reads back the 16
//     bytes it copied itself
//   P^T by exponentials against a running maximum that is raised only when a
//     score passes it by more than 2^8 (the sums stay far inside float32, the
//     weights inside the element type). The weights are rounded to that type (f16
//     over e4m3 pools) for the second product, as in every attention kernel here:
//     at most 2^-8 (f16 2^-11) of each, the size of the output's own rounding;
//     their sum is taken in float32 before that. An f16 weight below 2^-25 of the
//     running maximum's is lost.
//   O^T[D x 8 rows] += V^T P^T         V by transposed matrix loads from a
//     swizzled slice; P^T as the B operand by two 8x8 register transposes
// e4m3 pools: both products on f16 MMAs, which hold every e4m3 value and the
// query (see below) exactly; the K scale joins the scores', the V scale the
// final division.
// Rows of a slice that no query sees (before the window, past the sequence)
// are filled with zeros in V and masked in S: what their memory holds does not
// matter. The states (maximum, sum, O) of the warps meet in shared memory,
// those of the blocks of a cluster through distributed shared memory, always
// in the same order: no workspace, no atomics, the same bits on every run.
// Bound by the read of K and V: 64 sequences, 32/8 heads of 128, 46.0 us at
// window 1024 (276 MB, 6.0 TB/s), where the planned split kernel takes 73.5,
// and 169 us at window 4096 (6.35 TB/s; 203). e4m3 pools 36.7 us (54.0), by
// the conversions of K and V; head size 256 (16/8 heads) 89 us (149). Three
// slots per warp: with two, two sequences at window 16000 take 43.5 us instead
// of 36.7; with four, three blocks fit an SM (64 sequences in pages that are
// not cached 57.6 us instead of 51.7).
// ---------------------------------------------------------------------------
constexpr int kWdWarps = 4;

template <int D, bool FP8>
struct WdCfg {
  static constexpr int SLOTS = 3;
  static constexpr int BLOCKS = D > 128 ? 2 : 4;       // per SM
  static constexpr int ROW = D * (FP8 ? 1 : 2);        // bytes of a key
  static constexpr int TILE = 16 * ROW;                // a slice of K or of V
  static constexpr int RING = SLOTS * TILE;            // of a warp
  // A warp's state, in its ring: O[row][PITCH] (pitch of 4 banks mod 32: the
  // eight lanes and four row pairs of a store take different banks).
  static constexpr int PITCH = D + 4;
  static constexpr int OFF_ML = kWdWarps * RING;       // float[WARPS + 1][2][8]
  static constexpr int SMEM_BYTES = OFF_ML + (kWdWarps + 1) * 16 * 4;
  static_assert(kWinRows * PITCH * 4 <= RING, "the state fits the ring");
};

template <int D, bool F16, bool FP8>
__global__ void __launch_bounds__(kWdWarps * 32, WdCfg<D, FP8>::BLOCKS)
window_decode_kernel(const __grid_constant__ WinDecodeArgs a) {
  using E = Elem<F16>;
  using C = WdCfg<D, FP8>;
  constexpr int NV = C::ROW / 64;                      // 16-byte pieces of a key row per lane
  constexpr int NQ = D / 32;                           // of a query row
  constexpr int PIECES = C::ROW / 16;                  // of a row
  extern __shared__ __align__(128) uint8_t smem[];
  // Parts fastest, then KV head: a page's heads are read at about the same time.
  const int parts = a.parts;
  const int unit = blockIdx.x / parts;
  const int part = parts > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int s = unit / a.H_kv;
  const int hk = unit - s * a.H_kv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;

  const int q0 = __ldg(a.cu + s), q1 = __ldg(a.cu + s + 1);
  int kv = __ldg(a.seqused_k + s);
  int q_len = q1 - q0, bad = 0;
  if (q0 < 0 || q1 > a.total_q || q1 < q0 || q_len > a.max_q) {
    bad = PA_DEV_BAD_SEQLEN;
    q_len = 0;
  }
  if (kv < 0 || kv > a.max_k || kv > a.kv_len_cap) bad = PA_DEV_BAD_SEQLEN;
  kv = min(max(kv, 0), a.kv_len_cap);
  if (bad && hk == 0 && part == 0 && threadIdx.x == 0) flag_status(a.status, bad);
  if (q_len == 0) return;                              // the whole cluster
  const int rows = q_len * a.G;
  const int past = kv - q_len;                         // position of query 0
  const int lo = max(0, past - a.window + 1);          // first key of the windows
  const int first = min(a.first, kv);
  // Slices: those of the first tokens, then those of the windows.
  const int nb0 = lo >> 4, na = min((first + 15) >> 4, nb0);
  const int n = na + ((kv + 15) >> 4) - nb0;
  const int w = part * kWdWarps + warp, nw = parts * kWdWarps;
  const int v0 = w * n / nw, count = (w + 1) * n / nw - v0;   // <= 32
  auto slice_key = [&](int i) { return 16 * (v0 + i < na ? v0 + i : v0 + i - na + nb0); };

  // Lane i: page of slice i (-1: outside the pool), its first row.
  int page_l = -1, row_l = 0;
  if (lane < count) {
    const int key0 = slice_key(lane);
    const int lp = a.bs_shift >= 0 ? key0 >> a.bs_shift : key0 / a.bs;
    row_l = key0 - lp * a.bs;
    page_l = __ldg(a.bt + static_cast<int64_t>(s) * a.bt_stride + lp);
    if (page_l < 0 || page_l >= a.num_blocks) {
      page_l = -1;                                     // reads as zeros
      flag_status(a.status, PA_DEV_BAD_PAGE);
    }
  }
  uint8_t* ring = smem + warp * C::RING;
  const uint32_t ring_at = smem_u32(ring);
  const int64_t rstep = static_cast<int64_t>(a.H_kv) * C::ROW;
  // Copies of slice i of K or V into slot `to`, one group, empty or not.
  auto fetch = [&](int i, bool is_v, int to) {
    const int page = __shfl_sync(0xffffffffu, page_l, i & 31);
    const int prow = __shfl_sync(0xffffffffu, row_l, i & 31);
    if (i < count) {
      const bool in = page >= 0;
      const uint32_t dst = ring_at + to * C::TILE;
      const int64_t at = max(page, 0) * a.block_stride_bytes + hk * C::ROW + prow * rstep;
      if (!is_v) {
        // Keys g and g + 8, pieces 4 v + c, each to this lane's own places.
        const uint8_t* p = a.kc + at + g * rstep + c * 16;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          cp_async16(dst + (2 * v) * 512 + lane * 16, p + v * 64, in);
          cp_async16(dst + (2 * v + 1) * 512 + lane * 16, p + 8 * rstep + v * 64, in);
        }
      } else {
        const int key0 = slice_key(i);
        const uint8_t* p = a.vc + at;
#pragma unroll
        for (int it = 0; it < PIECES / 2; ++it) {
          const int idx = it * 32 + lane, r = idx / PIECES, x = idx % PIECES;
          const int j = key0 + r;
          cp_async16(dst + r * C::ROW + ((x ^ (r & 7)) << 4), p + r * rstep + x * 16,
                     in && j < kv && (j >= lo || j < first));
        }
      }
    }
    cp_async_commit();
  };
  int to = 0;                                          // slot of the next copies
  auto fetch_next = [&](int i, bool is_v) {
    fetch(i, is_v, to);
    if (++to == C::SLOTS) to = 0;
  };
#pragma unroll
  for (int u = 0; u < C::SLOTS - 1; ++u) fetch_next(u >> 1, u & 1);

  // Q as B fragments: packed row g (rows past the last repeat it, unwritten).
  uint4 qv[NQ];
  {
    const int r = min(g, rows - 1), i = r / a.G;
    const uint4* qrow = reinterpret_cast<const uint4*>(
        a.q + static_cast<int64_t>(q0 + i) * a.q_stride +
        static_cast<int64_t>(hk * a.G + r - i * a.G) * D);
#pragma unroll
    for (int v = 0; v < NQ; ++v)
      qv[v] = __ldg(qrow + (FP8 ? 8 * (v >> 1) + 2 * c + (v & 1) : 4 * v + c));
  }
  // This lane's rows 2c, 2c + 1: their positions.
  int pos[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) pos[e] = past + min(2 * c + e, rows - 1) / a.G;

  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  float acc[D / 16][4];
#pragma unroll
  for (int t = 0; t < D / 16; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[t][e] = 0.f;
  // Row and piece of this lane in the transposed loads of V, two pieces at a
  // time: matrices keys 0-7 | 8-15 of a piece (e4m3), or pieces of keys 0-7,
  // then of keys 8-15.
  const int vr = (lane & 7) + ((lane >> (FP8 ? 3 : 4)) & 1) * 8;
  const int vx = (lane >> (FP8 ? 4 : 3)) & 1;
  // Scale of the scores of rows 2c, 2c + 1.
  float sl2[2] = {a.scale_log2, a.scale_log2};
  using P = Elem<F16 || FP8>;                          // the MMA's type (e4m3 is exact in f16)
  if constexpr (FP8) {
    float qs = __ldg(a.k_scale + hk);
    if constexpr (!F16) {
      // A bf16 query as f16, its row brought to a maximum of 2^14 to 2^15 by a
      // power of two: exact but for elements of less than 2^-32 of the row's
      // largest, which are off by 2^-40 of it at most.
      float q[NQ][8], top = 0.f;
#pragma unroll
      for (int v = 0; v < NQ; ++v) {
        const uint32_t x[4] = {qv[v].x, qv[v].y, qv[v].z, qv[v].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 f = E::unpack(x[k]);
          q[v][2 * k] = f.x;
          q[v][2 * k + 1] = f.y;
          top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // By the exponent field of top: a finite row goes down by 2^113 at most and
      // up by 2^126 (so that 2^up and 2^-up are normal numbers; a smaller row's
      // maximum then stays below 2^14, zeros stay zeros). Infinities, too.
      const int ex = static_cast<int>(__float_as_uint(top) >> 23);
      const int up = ex == 255 ? 0 : min(126, 141 - ex);
      const float by = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
#pragma unroll
      for (int v = 0; v < NQ; ++v)
        qv[v] = make_uint4(pack_f16(q[v][0] * by, q[v][1] * by), pack_f16(q[v][2] * by, q[v][3] * by),
                           pack_f16(q[v][4] * by, q[v][5] * by), pack_f16(q[v][6] * by, q[v][7] * by));
      qs *= __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e)
      sl2[e] = a.scale_log2 * __shfl_sync(0xffffffffu, qs, (2 * c + e) * 4);
  }

  int from = 0;                                        // slot of the slice in use
#pragma unroll 1
  for (int i = 0; i < count; ++i) {
    const int key0 = slice_key(i);
    // ------------------------------------------------------------- S^T = K Q^T
    fetch_next((2 * i + C::SLOTS - 1) >> 1, (C::SLOTS - 1) & 1);
    cp_async_wait<C::SLOTS - 1>();
    __syncwarp();
    float st[4] = {0.f, 0.f, 0.f, 0.f};
    {
      const uint8_t* slot = ring + from * C::TILE + lane * 16;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const uint4 x0 = *reinterpret_cast<const uint4*>(slot + (2 * v) * 512);
        const uint4 x1 = *reinterpret_cast<const uint4*>(slot + (2 * v + 1) * 512);
        if constexpr (FP8) {
          const uint32_t w0[4] = {x0.x, x0.y, x0.z, x0.w}, w1[4] = {x1.x, x1.y, x1.z, x1.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint4& q = qv[2 * v + (k >> 1)];
            P::mma(st, e4m3x2_to_f16x2(w0[k]), e4m3x2_to_f16x2(w1[k]),
                   e4m3x2_to_f16x2(w0[k] >> 16), e4m3x2_to_f16x2(w1[k] >> 16),
                   (k & 1) ? q.z : q.x, (k & 1) ? q.w : q.y);
          }
        } else {
          P::mma(st, x0.x, x1.x, x0.y, x1.y, qv[v].x, qv[v].y);
          P::mma(st, x0.z, x1.z, x0.w, x1.w, qv[v].z, qv[v].w);
        }
      }
    }
    if (++from == C::SLOTS) from = 0;
    __syncwarp();                                      // the slot may be filled again
    fetch_next((2 * i + C::SLOTS) >> 1, C::SLOTS & 1);
    // ------------------------------------------------------------- softmax
    float x[4];                                        // (key g, rows) (key g + 8, rows)
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = st[e] * sl2[e & 1];
    const bool whole = key0 + 15 <= past &&
                       (key0 > past + q_len - 1 - a.window || key0 + 15 < first);
    if (!whole) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = key0 + g + 8 * (e >> 1), p = pos[e & 1];
        if (!(j <= p && (j > p - a.window || j < first))) x[e] = -INFINITY;
      }
    }
    const float mx0 = fmaxf(x[0], x[2]), mx1 = fmaxf(x[1], x[3]);
    if (__any_sync(0xffffffffu, mx0 > m[0] + 8.f || mx1 > m[1] + 8.f)) {
      float mx[2] = {mx0, mx1};
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], o));
        const float nm = fmaxf(m[e], mx[e]);
        const float f = m[e] == -INFINITY ? 0.f : fast_exp2(m[e] - nm);
        l[e] *= f;
        m[e] = nm;
#pragma unroll
        for (int t = 0; t < D / 16; ++t) {
          acc[t][e] *= f;
          acc[t][2 + e] *= f;
        }
      }
    }
    float p[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      p[e] = fast_exp2(x[e] - (m[e & 1] == -INFINITY ? 0.f : m[e & 1]));
    l[0] += p[0] + p[2];
    l[1] += p[1] + p[3];
    const uint32_t pb0 = movmatrix_trans(P::pack(p[0], p[1]));
    const uint32_t pb1 = movmatrix_trans(P::pack(p[2], p[3]));
    // ------------------------------------------------------------- O^T += V^T P^T
    cp_async_wait<C::SLOTS - 1>();
    __syncwarp();
    const uint32_t vrow = ring_at + from * C::TILE + vr * C::ROW;
#pragma unroll
    for (int t = 0; t < C::ROW / 32; ++t) {
      uint32_t r[4];
      ldsm_x4_t(vrow + (((2 * t + vx) ^ (vr & 7)) << 4), r[0], r[1], r[2], r[3]);
      if constexpr (FP8) {
        // A lane holds bytes (keys 2c, 2c + 1) x (dims 2g, 2g + 1) of a piece:
        // even dims become rows 0-7 of the MMA, odd ones rows 8-15.
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t lo8 = r[2 * k], hi8 = r[2 * k + 1];
          P::mma(acc[2 * t + k], e4m3x2_to_f16x2(prmt(lo8, 0, 0x4420)),
                 e4m3x2_to_f16x2(prmt(lo8, 0, 0x4431)), e4m3x2_to_f16x2(prmt(hi8, 0, 0x4420)),
                 e4m3x2_to_f16x2(prmt(hi8, 0, 0x4431)), pb0, pb1);
        }
      } else {
        P::mma(acc[t], r[0], r[1], r[2], r[3], pb0, pb1);
      }
    }
    if (++from == C::SLOTS) from = 0;
    __syncwarp();
  }
  cp_async_wait<0>();
  __syncwarp();

  // ---------------------------------------------------------------- the warps' states
  float* ml = reinterpret_cast<float*>(smem + C::OFF_ML);   // [warp][m, l][row]; then the block's
#pragma unroll
  for (int e = 0; e < 2; ++e)
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], o);
  float* mine = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    if (g == 0) {
      ml[warp * 16 + 2 * c + e] = m[e];
      ml[warp * 16 + 8 + 2 * c + e] = l[e];
    }
#pragma unroll
    for (int t = 0; t < D / 16; ++t) {
      const int d = 16 * t + (FP8 ? 2 * g : g);
      mine[(2 * c + e) * C::PITCH + d] = acc[t][e];
      mine[(2 * c + e) * C::PITCH + d + (FP8 ? 1 : 8)] = acc[t][2 + e];
    }
  }
  __syncthreads();

  // Four dims of a row, finished: the sink joins, the sum divides.
  const float vs = FP8 ? __ldg(a.v_scale + hk) : 1.f;
  auto finish = [&](int row, int d, float M, float L, float4 o) {
    const int i = row / a.G, head = hk * a.G + row - i * a.G;
    if (a.sinks) {
      const float f = add_sink(M, L, __ldg(a.sinks + head) * kLog2e);
      o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
    }
    const float inv = L == 0.f ? 0.f : vs / L;
    *reinterpret_cast<uint2*>(a.out + (static_cast<int64_t>(q0 + i) * a.H + head) * D + d) =
        make_uint2(E::pack(o.x * inv, o.y * inv), E::pack(o.z * inv, o.w * inv));
    if (d == 0 && a.lse)
      a.lse[static_cast<int64_t>(head) * a.total_q + q0 + i] =
          L == 0.f ? -INFINITY : (M + fast_log2(L)) * kLn2;
  };
  constexpr int UNITS = kWinRows * D / 4;              // (row, four dims)
  for (int u = threadIdx.x; u < UNITS; u += kWdWarps * 32) {
    const int row = u / (D / 4), d = u % (D / 4) * 4;
    if (row >= rows) break;
    float M = -INFINITY, L = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kWdWarps; ++k) M = fmaxf(M, ml[k * 16 + row]);
#pragma unroll
    for (int k = 0; k < kWdWarps; ++k) {
      const float mk = ml[k * 16 + row];
      const float f = mk == -INFINITY ? 0.f : fast_exp2(mk - M);
      const float4 x = *reinterpret_cast<const float4*>(smem + k * C::RING + (row * C::PITCH + d) * 4);
      L += f * ml[k * 16 + 8 + row];
      o = make_float4(o.x + f * x.x, o.y + f * x.y, o.z + f * x.z, o.w + f * x.w);
    }
    if (parts == 1) {
      finish(row, d, M, L, o);
    } else {
      // The block's state, in place of warp 0's (read by this thread alone).
      *reinterpret_cast<float4*>(smem + (row * C::PITCH + d) * 4) = o;
      if (d == 0) {
        ml[kWdWarps * 16 + row] = M;
        ml[kWdWarps * 16 + 8 + row] = L;
      }
    }
  }
  if (parts == 1) return;
  // ---------------------------------------------------------------- the cluster's states
  cluster_arrive();
  cluster_wait();
  const float* bml = ml + kWdWarps * 16;
  for (int u = part * (UNITS / parts) + threadIdx.x; u < (part + 1) * (UNITS / parts);
       u += kWdWarps * 32) {
    const int row = u / (D / 4), d = u % (D / 4) * 4;
    if (row >= rows) break;
    float M = -INFINITY, L = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < parts; ++k) M = fmaxf(M, load_remote(bml + row, k));
    for (int k = 0; k < parts; ++k) {
      const float mk = load_remote(bml + row, k);
      const float f = mk == -INFINITY ? 0.f : fast_exp2(mk - M);
      const float4 x =
          load_remote4(reinterpret_cast<const float*>(smem) + row * C::PITCH + d, k);
      L += f * load_remote(bml + 8 + row, k);
      o = make_float4(o.x + f * x.x, o.y + f * x.y, o.z + f * x.z, o.w + f * x.w);
    }
    finish(row, d, M, L, o);
  }
  cluster_arrive();                                    // nobody leaves while its state is read
  cluster_wait();
}

template <int D, bool F16, bool FP8>
static cudaError_t launch_window_decode_d(const WinDecodeArgs& a, unsigned grid, cudaStream_t st) {
  using C = WdCfg<D, FP8>;
  static std::atomic<bool> configured[kMaxDevices];
  cudaError_t e = opt_in_smem(window_decode_kernel<D, F16, FP8>, C::SMEM_BYTES, configured);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kWdWarps * 32);
  cfg.dynamicSmemBytes = C::SMEM_BYTES;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = a.parts;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.parts > 1 ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, window_decode_kernel<D, F16, FP8>, a);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

cudaError_t launch_window_decode(WinDecodeArgs a, int num_seqs, int slices, int D, bool f16,
                                 cudaStream_t st, int sms) {
  const long long units = static_cast<long long>(num_seqs) * a.H_kv;
  // Blocks per (sequence, KV head): what the page ids of a warp's lanes ask
  // for, and then two waves of one block per SM as long as a warp keeps two
  // slices. 16 sequences of 8 KV heads, window 1024: 15.0 us with 4 parts, 16.3
  // with 2, 19.8 with 8; 32 sequences 29.8, 27.9 (one) and 32.6; one sequence
  // 8.0 with 8 parts.
  int parts = 1;
  while (parts < kWinMaxParts && (slices > parts * kWinPartSlices ||
                                  (units * parts < 2LL * sms && slices > 2 * kWdWarps * parts)))
    parts *= 2;
  a.parts = parts;
  const unsigned grid = static_cast<unsigned>(units * parts);
  if (a.k_scale) return f16 ? launch_window_decode_d<128, true, true>(a, grid, st)
                            : launch_window_decode_d<128, false, true>(a, grid, st);
  if (f16) {
    if (D == 256) return launch_window_decode_d<256, true, false>(a, grid, st);
    if (D == 128) return launch_window_decode_d<128, true, false>(a, grid, st);
    return launch_window_decode_d<64, true, false>(a, grid, st);
  }
  if (D == 256) return launch_window_decode_d<256, false, false>(a, grid, st);
  if (D == 128) return launch_window_decode_d<128, false, false>(a, grid, st);
  return launch_window_decode_d<64, false, false>(a, grid, st);
}

}  // namespace pa
