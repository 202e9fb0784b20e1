// Accumulated attention weight of every cached key: the column sums of the
// attention matrix, w_j += sum_i exp(scale q_i.k_j - lse_i), recomputed from
// K and the LSE that the attention call returned (the matrix itself never
// exists in memory). Each key has one owner, so there are no atomics and the
// sums are the same bits on every run.
#include <cuda_runtime.h>

#include "device_common.cuh"

namespace pa {

// ---------------------------------------------------------------------------
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
  const int q0 = __ldg(a.cu + s), q1 = __ldg(a.cu + s + 1);
  int kv = __ldg(a.seqused_k + s);
  const bool reports = key0 == 0 && hk == 0 && lane == 0;
  if (q0 < 0 || q1 > a.total_q || q1 < q0 || q1 - q0 > a.max_q) {
    if (reports) flag_status(a.status, PA_DEV_BAD_SEQLEN);
    return;
  }
  const int q_len = q1 - q0;
  if (reports && (kv < 0 || kv > a.max_k || kv > a.kv_len_cap))
    flag_status(a.status, PA_DEV_BAD_SEQLEN);
  kv = min(kv, a.kv_len_cap);
  if (key0 >= kv || q_len == 0) return;
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

cudaError_t launch_attn_weights(const WeightArgs& a, int num_seqs, int D, bool f16, bool fp8,
                                cudaStream_t st) {
  const int keys = a.max_k < a.kv_len_cap ? a.max_k : a.kv_len_cap;
  const int tiles = keys > 0 ? (keys + kWeightWarps * 16 - 1) / (kWeightWarps * 16) : 1;
  auto run = [&](auto kernel) {
    kernel<<<dim3(static_cast<unsigned>(num_seqs) * tiles, a.H_kv), kWeightWarps * 32, 0, st>>>(
        a, tiles);
    return cudaGetLastError();
  };
  if (fp8) return f16 ? run(weights_kernel<128, true, true>) : run(weights_kernel<128, false, true>);
  if (f16) {
    if (D == 256) return run(weights_kernel<256, true, false>);
    if (D == 128) return run(weights_kernel<128, true, false>);
    return run(weights_kernel<64, true, false>);
  }
  if (D == 256) return run(weights_kernel<256, false, false>);
  if (D == 128) return run(weights_kernel<128, false, false>);
  return run(weights_kernel<64, false, false>);
}

}  // namespace pa
