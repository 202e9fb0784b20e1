// Rotary positions: the cos/sin table of a model's positions, and the pass
// that turns a step's new queries and keys -- with the per-head RMS norms, if
// the model has them -- and writes K and V into their pages (the cache write
// of "FlashAttention 在 vLLM 中的实现分析" §4.2, with the arithmetic that
// precedes it in a decoder layer).
#include <cuda_runtime.h>

#include "device_common.cuh"
#include "quantize.cuh"

namespace pa {

// ---------------------------------------------------------------------------
// Table. Pair i turns f_i / 2 pi times per position. The turn count of
// position p is only needed modulo 1, so each thread keeps its pair's rate as
// a 64-bit fraction F = round(2^64 * frac(f_i / 2 pi)) and multiplies it by
// p in 64-bit integers, which drop whole turns by themselves: the phase is
// off by p * 2^-65 turns from F's rounding and p * 2^-53 * f_i / 2 pi from
// the double behind it (under 1e-9 radian at a million positions), where a
// float32 angle would be off by p * f_i * 2^-24. The phase is split into the
// nearest quarter turn and a signed remainder of at most an eighth, so the
// float32 sinpi / cospi that follow see a remainder with full relative
// precision.
// Double precision is slow on this part (2 operations per clock and SM): it
// is used once per thread, for the rate, and never per entry.
// ---------------------------------------------------------------------------
constexpr int kTableThreads = 256;

__device__ __forceinline__ double rope_rate(const RopeTableArgs& a, int i) {
  double f = pow(a.base, -2.0 * i / a.rot);
  switch (a.kind) {
    case PA_ROPE_LINEAR:
      f /= a.factor;
      break;
    case PA_ROPE_WAVELENGTH: {
      // Turns within the original length: at most `low` are interpolated, at
      // least `high` kept, a linear mix of the two in between.
      const double mix = fmin(1.0, fmax(0.0, (a.orig_len * f * 0.15915494309189535 - a.low) /
                                                 (a.high - a.low)));
      f = f / a.factor * (1.0 - mix) + f * mix;
      break;
    }
    case PA_ROPE_YARN: {
      const double ramp = fmin(1.0, fmax(0.0, (i - a.ramp_lo) / a.ramp_len));
      f = f / a.factor * ramp + f * (1.0 - ramp);
      break;
    }
    default:
      break;   // PA_ROPE_NTK: the host has changed the base
  }
  return f * 0.15915494309189535;   // turns per position
}

__global__ void __launch_bounds__(kTableThreads)
rope_table_kernel(float* __restrict__ table, const __grid_constant__ RopeTableArgs a) {
  const int half = a.rot >> 1;
  const int step = kTableThreads / half;   // positions a block writes per step
  const int i = threadIdx.x % half, r = threadIdx.x / half;
  if (r >= step) return;
  const double turns = rope_rate(a, i);
  const double frac = turns - floor(turns);
  // 2^64 frac, rounded: two halves, as frac may carry 53 bits below 2^-11.
  const double hi = floor(frac * 0x1p32);
  const unsigned long long rate =
      (static_cast<unsigned long long>(hi) << 32) +
      static_cast<unsigned long long>(rint((frac * 0x1p32 - hi) * 0x1p32));
  const int p0 = blockIdx.x * a.per_block;
  const int p1 = min(a.table_len, p0 + a.per_block);
  for (int p = p0 + r; p < p1; p += step) {
    const unsigned long long ph = rate * static_cast<unsigned>(p);
    const unsigned q = static_cast<unsigned>((ph + (1ull << 61)) >> 62);   // nearest quarter
    const long long rem = static_cast<long long>(ph - (static_cast<unsigned long long>(q) << 62));
    float sn, cs;
    sincospif(static_cast<float>(rem) * 0x1p-63f, &sn, &cs);   // rem 2^-64 turns, in half turns
    const float c = (q & 1) ? sn : cs, s = (q & 1) ? cs : sn;
    const float cm = ((q + 1) & 2) ? -a.mscale : a.mscale, sm = (q & 2) ? -a.mscale : a.mscale;
    float* row = table + static_cast<int64_t>(p) * a.rot;
    row[i] = c * cm;
    row[half + i] = s * sm;
  }
}

cudaError_t launch_rope_table(float* table, RopeTableArgs a, cudaStream_t st, int sms) {
  if (a.table_len == 0) return cudaSuccess;
  const int step = kTableThreads / (a.rot / 2);
  // Eight blocks per SM (every thread resident) share the positions, in
  // whole steps.
  const long long blocks = 8LL * sms;
  const long long per = (a.table_len + blocks * step - 1) / (blocks * step) * step;
  a.per_block = static_cast<int>(per);
  const int grid = static_cast<int>((a.table_len + per - 1) / per);
  rope_table_kernel<<<grid, kTableThreads, 0, st>>>(table, a);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// Norm, rotation and cache write in one pass over the new tokens: every q, k
// and v element is read once and written once. A warp takes one token (or
// part of its heads); D / 8 lanes hold a head, 16 bytes each, so an item --
// 32 * 8 / D heads of q, k or v -- is one coalesced 512-byte access, and
// kUnroll items are in flight. The token's cos and sin stay in registers for
// all of its heads. The partner of an element under rotation is in the same
// lane (interleaved pairs) or rot / 16 lanes away (half layout: one shuffle
// per element). Everything between the load and the store is float32; the
// store is the only rounding.
// ---------------------------------------------------------------------------
constexpr int kRopeThreads = 256;
constexpr int kRopeWarps = kRopeThreads / 32;
constexpr int kRopeUnroll = 4;

template <bool F16>
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t h[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 a = Elem<F16>::unpack(h[k]);
    f[2 * k] = a.x;
    f[2 * k + 1] = a.y;
  }
}

template <bool F16>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(Elem<F16>::pack(f[0], f[1]), Elem<F16>::pack(f[2], f[3]),
                    Elem<F16>::pack(f[4], f[5]), Elem<F16>::pack(f[6], f[7]));
}

__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

template <int D, bool F16, bool FP8>
__global__ void __launch_bounds__(kRopeThreads)
rope_and_cache_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int LPH = D / 8;        // lanes per head
  constexpr int HPI = 32 / LPH;     // heads per item
  const int lane = threadIdx.x & 31;
  const int sub = lane / LPH, l = lane % LPH;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * kRopeWarps + (threadIdx.x >> 5);
  const int64_t t = w / a.chunks;
  const int part = static_cast<int>(w - t * a.chunks);
  if (t >= a.num_tokens) return;
  const int64_t pos = __ldg(a.positions + t), slot = __ldg(a.slots + t);
  if (pos < 0) return;                       // padding token
  if (pos >= a.table_len) {
    if (part == 0 && lane == 0) flag_status(a.status, PA_DEV_BAD_POSITION);
    return;
  }
  const bool cached = slot >= 0 && slot < a.num_slots;
  if (slot >= a.num_slots && part == 0 && lane == 0) flag_status(a.status, PA_DEV_BAD_SLOT);
  const int nq = (a.H + HPI - 1) / HPI, nkv = (a.H_kv + HPI - 1) / HPI;
  const int first = part * a.items_per_warp;
  const int last = min(first + a.items_per_warp, cached ? nq + 2 * nkv : nq);

  // This lane's cos and sin, the latter with the sign of its element's term.
  const bool turns = 8 * l < a.rot;
  const int half = a.rot >> 1;
  float c[8], s[8];
  int partner = lane;
  if (turns) {
    const float* row = a.cos_sin + pos * a.rot;
    if (a.interleaved) {
      const float4 cc = __ldg(reinterpret_cast<const float4*>(row + 4 * l));
      const float4 ss = __ldg(reinterpret_cast<const float4*>(row + half + 4 * l));
      const float cv[4] = {cc.x, cc.y, cc.z, cc.w}, sv[4] = {ss.x, ss.y, ss.z, ss.w};
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        c[k] = cv[k >> 1];
        s[k] = (k & 1) ? sv[k >> 1] : -sv[k >> 1];
      }
    } else {
      const bool lower = 8 * l < half;
      const int i0 = lower ? 8 * l : 8 * l - half;
      partner = lower ? lane + (a.rot >> 4) : lane - (a.rot >> 4);
      load8(row + i0, c);
      load8(row + half + i0, s);
#pragma unroll
      for (int k = 0; k < 8; ++k) s[k] = lower ? -s[k] : s[k];
    }
  }
  const int64_t page = cached ? slot / a.bs : 0;
  // Byte offset of the token's row in a pool (rows hold [H_kv, D]).
  const int64_t crow = page * a.block_stride_bytes +
                       (cached ? slot - page * a.bs : 0) * a.H_kv * D * (FP8 ? 1 : 2);

  for (int it = first; it < last; it += kRopeUnroll) {
    uint4 x[kRopeUnroll];
#pragma unroll
    for (int u = 0; u < kRopeUnroll; ++u) {
      const int item = it + u;
      x[u] = make_uint4(0, 0, 0, 0);
      if (item >= last) continue;
      const int kind = item < nq ? 0 : (item < nq + nkv ? 1 : 2);
      const int h = (item - (kind == 0 ? 0 : (kind == 1 ? nq : nq + nkv))) * HPI + sub;
      if (h >= (kind == 0 ? a.H : a.H_kv)) continue;
      const uint16_t* src = kind == 0 ? a.q + t * a.q_stride
                                      : (kind == 1 ? a.k + t * a.k_stride : a.v + t * a.v_stride);
      x[u] = __ldcs(reinterpret_cast<const uint4*>(src + h * D) + l);
    }
#pragma unroll
    for (int u = 0; u < kRopeUnroll; ++u) {
      const int item = it + u;
      if (item >= last) break;               // warp-uniform, like kind below
      const int kind = item < nq ? 0 : (item < nq + nkv ? 1 : 2);
      const int h = (item - (kind == 0 ? 0 : (kind == 1 ? nq : nq + nkv))) * HPI + sub;
      const bool live = h < (kind == 0 ? a.H : a.H_kv);
      float f[8];
      if (FP8 || kind < 2) unpack8<F16>(x[u], f);
      if (kind < 2) {
        const float* wt = kind == 0 ? a.q_norm : a.k_norm;
        if (wt) {
          float ss = 0.f;
#pragma unroll
          for (int k = 0; k < 8; ++k) ss = fmaf(f[k], f[k], ss);
#pragma unroll
          for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          const float r = rsqrtf(ss * (1.f / D) + a.eps);
          float wv[8];
          load8(wt + 8 * l, wv);
#pragma unroll
          for (int k = 0; k < 8; ++k) f[k] = f[k] * r * wv[k];
        }
        float g[8];
        if (a.interleaved) {
#pragma unroll
          for (int k = 0; k < 8; ++k) g[k] = f[k ^ 1];
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) g[k] = __shfl_sync(0xffffffffu, f[k], partner);
        }
        if (turns) {
#pragma unroll
          for (int k = 0; k < 8; ++k) f[k] = fmaf(g[k], s[k], f[k] * c[k]);
        }
      }
      if (!live) continue;
      // What neither the norm nor the rotation touches keeps its bits.
      const bool as_is = kind == 2 || (!turns && !(kind == 0 ? a.q_norm : a.k_norm));
      if (kind == 0) {
        *(reinterpret_cast<uint4*>(a.q_out + t * a.q_out_stride + h * D) + l) =
            as_is ? x[u] : pack8<F16>(f);
      } else {
        uint8_t* row = (kind == 1 ? a.kc : a.vc) + crow;
        if constexpr (FP8) {
          const ScaleDiv d = scale_div(__ldg((kind == 1 ? a.k_scale : a.v_scale) + h));
          *(reinterpret_cast<uint2*>(row + h * D) + l) = quantize8(f, d);
        } else {
          *(reinterpret_cast<uint4*>(row + h * D * 2) + l) = as_is ? x[u] : pack8<F16>(f);
        }
      }
    }
  }
}

cudaError_t launch_rope_and_cache(RopeArgs a, int D, bool f16, bool fp8, cudaStream_t st,
                                  int sms) {
  if (a.num_tokens == 0) return cudaSuccess;
  const int hpi = 256 / D;
  const int items = (a.H + hpi - 1) / hpi + 2 * ((a.H_kv + hpi - 1) / hpi);
  // Few tokens: their heads are shared among more warps, down to one item
  // each, until about 32 warps per SM have work.
  const long long want = static_cast<long long>(a.num_tokens) * items / (32LL * sms);
  const int per = static_cast<int>(want < 1 ? 1 : (want > items ? items : want));
  a.chunks = (items + per - 1) / per;
  a.items_per_warp = (items + a.chunks - 1) / a.chunks;
  const long long warps = static_cast<long long>(a.num_tokens) * a.chunks;
  const unsigned grid = static_cast<unsigned>((warps + kRopeWarps - 1) / kRopeWarps);
  auto run = [&](auto kernel) {
    kernel<<<grid, kRopeThreads, 0, st>>>(a);
    return cudaGetLastError();
  };
  if (fp8) return f16 ? run(rope_and_cache_kernel<128, true, true>)
                      : run(rope_and_cache_kernel<128, false, true>);
  if (f16) {
    if (D == 256) return run(rope_and_cache_kernel<256, true, false>);
    if (D == 128) return run(rope_and_cache_kernel<128, true, false>);
    return run(rope_and_cache_kernel<64, true, false>);
  }
  if (D == 256) return run(rope_and_cache_kernel<256, false, false>);
  if (D == 128) return run(rope_and_cache_kernel<128, false, false>);
  return run(rope_and_cache_kernel<64, false, false>);
}

}  // namespace pa
