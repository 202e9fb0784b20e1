// Rows of a 4-bit cache back as values.
#include <cuda_runtime.h>

#include "device_common.cuh"
#include "quantize.cuh"

namespace pa {

// ---------------------------------------------------------------------------
// A word of 8 codes per lane; a token's words of K, then of V, are taken 32 at
// a time by one warp, kRowsAhead of them in flight. code * scale + minimum is
// one float32 product and sum (the product of a 4-bit and an 11-bit number is
// exact), rounded once to the output type.
// ---------------------------------------------------------------------------
constexpr int kRowsAhead = 4;

template <int D, bool F16>
__global__ void __launch_bounds__(128) int4_rows_kernel(const __grid_constant__ Int4RowsArgs a) {
  constexpr int WPH = D / 8;                 // words of a head
  const int lane = threadIdx.x & 31;
  const int words = a.H_kv * WPH;            // of a token's K row
  const int64_t stride = static_cast<int64_t>(gridDim.x) * 4;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5); t < a.num_tokens;
       t += stride) {
    const int64_t slot = __ldg(a.slots + t);
    const bool in = slot >= 0 && slot < a.num_slots;
    if (slot >= a.num_slots && lane == 0) flag_status(a.status, PA_DEV_BAD_SLOT);
    const int64_t page = in ? slot / a.bs : 0, row = in ? slot - page * a.bs : 0;
    const int64_t crow = page * a.block_stride_bytes + row * words * 4;
    const int64_t prow = page * a.params_stride + row;
    for (int w0 = lane; w0 < 2 * words; w0 += 32 * kRowsAhead) {
      uint32_t code[kRowsAhead], par[kRowsAhead];
#pragma unroll
      for (int u = 0; u < kRowsAhead; ++u) {
        const int w = w0 + 32 * u;
        code[u] = par[u] = 0;
        if (w < 2 * words && in) {
          const int x = w < words ? w : w - words;
          code[u] = __ldg(reinterpret_cast<const uint32_t*>((w < words ? a.kc : a.vc) + crow) + x);
          par[u] = __ldg((w < words ? a.k_params : a.v_params) + prow +
                         static_cast<int64_t>(x / WPH) * a.bs);
        }
      }
#pragma unroll
      for (int u = 0; u < kRowsAhead; ++u) {
        const int w = w0 + 32 * u;
        if (w >= 2 * words) break;
        const float2 sm = Elem<true>::unpack(par[u]);
        uint32_t y[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float n0 = static_cast<float>((code[u] >> (4 * k)) & 15u);
          const float n1 = static_cast<float>((code[u] >> (16 + 4 * k)) & 15u);
          y[k] = Elem<F16>::pack(fmaf(n0, sm.x, sm.y), fmaf(n1, sm.x, sm.y));
        }
        const int x = w < words ? w : w - words;
        *reinterpret_cast<uint4*>((w < words ? a.key : a.value) + t * words * 8 + x * 8) =
            make_uint4(y[0], y[1], y[2], y[3]);
      }
    }
  }
}

cudaError_t launch_int4_rows(const Int4RowsArgs& a, int D, bool f16, cudaStream_t st, int sms) {
  if (a.num_tokens == 0) return cudaSuccess;
  const long long want = (static_cast<long long>(a.num_tokens) + 3) / 4, most = 16LL * sms;
  const unsigned grid = static_cast<unsigned>(want < most ? want : most);
  if (D == 128) {
    if (f16) int4_rows_kernel<128, true><<<grid, 128, 0, st>>>(a);
    else int4_rows_kernel<128, false><<<grid, 128, 0, st>>>(a);
  } else {
    if (f16) int4_rows_kernel<64, true><<<grid, 128, 0, st>>>(a);
    else int4_rows_kernel<64, false><<<grid, 128, 0, st>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace pa
