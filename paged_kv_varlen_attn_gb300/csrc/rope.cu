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
// position p is only needed modulo 1, so the host hands over each pair's rate
// as a 64-bit fraction of a turn, round(2^64 * frac(f_i / 2 pi)), and a thread
// multiplies it by p in 64-bit integers, which drop whole turns by themselves:
// the phase is off by p * 2^-65 turns from that rounding and p * 2^-53 * f_i /
// 2 pi from the double behind it (under 1e-9 radian at a million positions),
// where a float32 angle would be off by p * f_i * 2^-24. The phase is split
// into the nearest quarter turn and a signed remainder of at most an eighth,
// u = remainder / (1/8 turn) in [-1, 1], for which sin(pi/4 u) = u S(u^2) and
// cos(pi/4 u) = C(u^2) with S and C the minimax polynomials of degree 3 and 4
// (from a linear program over 3001 points: absolute error 1.2e-9 and 4.3e-11,
// with the coefficients rounded to float32 2.5e-8 and 7.3e-9, evaluated in
// float32 at most 2.2 and 1.8 units of 2^-24). No double arithmetic on
// the device (2 operations per clock and SM; the rates alone took 60 us for a
// table of any size) and no general argument reduction: 67 MB of table are
// bound by their write (11.6 us, 85% of the measured copy rate; sincospif
// instead: 20.8 us).
// ---------------------------------------------------------------------------
constexpr int kTableThreads = 256;

__global__ void __launch_bounds__(kTableThreads)
rope_table_kernel(float* __restrict__ table, const __grid_constant__ RopeTableArgs a) {
  const int half = a.rot >> 1;
  const int step = kTableThreads / half;   // positions a block writes per step
  const int i = threadIdx.x % half, r = threadIdx.x / half;
  if (r >= step) return;
  const unsigned long long rate = a.rate[i];
  const int p0 = blockIdx.x * a.per_block;
  const int p1 = min(a.table_len, p0 + a.per_block);
  // Phase of position p plus an eighth of a turn: its top two bits are the
  // nearest quarter turn, the bits below it the remainder plus an eighth.
  unsigned long long ph = rate * static_cast<unsigned>(p0 + r) + (1ull << 61);
  const unsigned long long dph = rate * static_cast<unsigned>(step);
  float* row = table + static_cast<int64_t>(p0 + r) * a.rot + i;
  const int64_t drow = static_cast<int64_t>(step) * a.rot;
  for (int p = p0 + r; p < p1; p += step, ph += dph, row += drow) {
    const unsigned hi = static_cast<unsigned>(ph >> 32);
    const unsigned q = hi >> 30;
    const int rem = static_cast<int>(__funnelshift_l(static_cast<unsigned>(ph), hi, 2) ^ 0x80000000u);
    const float u = static_cast<float>(rem) * 0x1p-31f, w = u * u;
    float sn = fmaf(fmaf(fmaf(-0x1.2cf016p-15f, w, 0x1.465a12p-9f), w, -0x1.4abba6p-4f), w,
                    0x1.921fb4p-1f) * u;
    float cs = fmaf(fmaf(fmaf(fmaf(0x1.d9ae2cp-19f, w, -0x1.55c52ap-12f), w, 0x1.03c1dcp-6f), w,
                         -0x1.3bd3ccp-2f), w, 1.f);
    const float c = (q & 1) ? sn : cs, s = (q & 1) ? cs : sn;
    row[0] = c * (((q + 1) & 2) ? -a.mscale : a.mscale);
    row[half] = s * ((q & 2) ? -a.mscale : a.mscale);
  }
}

cudaError_t launch_rope_table(float* table, RopeTableArgs& a, cudaStream_t st, int sms) {
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
// and v element is read once and written once. D / 8 lanes hold a head, 16
// bytes each, so an item -- 32 * 8 / D heads of q, k or v -- is one coalesced
// 512-byte access, and item i of a token's q (k, v) starts 512 i bytes into
// the token's row, whatever D is. A warp takes up to kRopeItems items of one
// token (of q, or of k then v), all of whose loads are in flight before the
// first is used; none of them waits for the token's position.
// With w the norm weights (1 without a norm) and r = 1 / rms, an element x_j
// with partner x_p becomes r (x_j w_j cos -+ x_p w_p sin): the coefficients
// w_j cos and -+w_p sin of the lane's 8 elements are set up once per warp. The
// partner is in the same register (interleaved pairs: swapped halves) or rot /
// 16 lanes away (half layout: one shuffle per pair of elements). Everything
// between the load and the store is float32; the store is the only rounding.
// A block is one warp: its place on the SM is taken by the next one as soon as
// it is done, so loads are always on their way. Bound by HBM without norms:
// 16,384 tokens of 32/8 heads of 128 (405 MB) take 62.2 us, 96% of the measured
// copy rate (blocks of two warps 67.5, of four 70.8; 28 blocks per SM 66.6).
// 4,109 tokens of 64/8 heads with norms into e4m3 pools (162 MB) take 33.2 us,
// 72% (two warps 41, four 42.2; 24 blocks per SM 33.8); there nothing is full
// (profiler: DRAM 36%, issue slots 63%, resident warps 38%): a warp waits for the
// shuffles of its items one after another, four of the norm's sum and four of
// the partners each. A decode step's 64 tokens take 3.0 us.
// ---------------------------------------------------------------------------
constexpr int kRopeItems = 8;

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

// INTER: interleaved pairs. NORM: q or k (or both) are normed.
template <int D, bool F16, bool FP8, bool INTER, bool NORM>
__global__ void __launch_bounds__(32, NORM ? 28 : 32)
rope_and_cache_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int LPH = D / 8;        // lanes per head
  constexpr int HPI = 32 / LPH;     // heads per item
  const int lane = threadIdx.x;
  const int l = lane % LPH;
  const int t = static_cast<int>(blockIdx.x / static_cast<unsigned>(a.chunks));
  const int part = static_cast<int>(blockIdx.x - static_cast<unsigned>(t) * a.chunks);
  const int64_t pos = __ldg(a.positions + t), slot = __ldg(a.slots + t);
  // This warp's items: q items, or the k items followed by the v items.
  const bool is_q = part < a.q_chunks;
  const int nkv = (a.H_kv + HPI - 1) / HPI;
  const int n_all = is_q ? (a.H + HPI - 1) / HPI : 2 * nkv;
  const int first = (is_q ? part : part - a.q_chunks) * a.items_per_warp;
  const int n = min(a.items_per_warp, n_all - first);
  const int row_bytes = (is_q ? a.H : a.H_kv) * D * 2;
  const uint8_t* src = reinterpret_cast<const uint8_t*>(is_q ? a.q + t * a.q_stride
                                                             : a.k + t * a.k_stride) +
                       lane * 16;
  const uint8_t* src_v = reinterpret_cast<const uint8_t*>(a.v + t * a.v_stride) + lane * 16;

  uint4 x[kRopeItems];
#pragma unroll
  for (int u = 0; u < kRopeItems; ++u) {
    x[u] = make_uint4(0, 0, 0, 0);
    if (u >= n) continue;
    const int item = first + u;
    const bool v = !is_q && item >= nkv;
    const int off = (v ? item - nkv : item) * 512;
    if (off + lane * 16 < row_bytes)
      x[u] = __ldcs(reinterpret_cast<const uint4*>((v ? src_v : src) + off));
  }
  if (pos < 0) return;                       // padding token
  if (pos >= a.table_len) {
    if (part == 0 && lane == 0) flag_status(a.status, PA_DEV_BAD_POSITION);
    return;
  }
  if (slot >= a.num_slots && part == 0 && lane == 0) flag_status(a.status, PA_DEV_BAD_SLOT);
  if (!is_q && (slot < 0 || slot >= a.num_slots)) return;

  const bool turns = 8 * l < a.rot;
  const int half = a.rot >> 1;
  const bool lower = 8 * l < half;           // half layout: first elements of their pairs
  const int away = INTER || !turns ? 0 : (lower ? a.rot >> 4 : -(a.rot >> 4));
  const float* wt = NORM ? (is_q ? a.q_norm : a.k_norm) : nullptr;
  float ca[8], cb[8];                        // coefficients of x_j and of its partner
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    ca[k] = 1.f;
    cb[k] = 0.f;
  }
  if (turns && first < (is_q ? n_all : nkv)) {   // (not for v items alone)
    const float* row = a.cos_sin + pos * a.rot;
    if constexpr (INTER) {
      const float4 cc = __ldg(reinterpret_cast<const float4*>(row + 4 * l));
      const float4 ss = __ldg(reinterpret_cast<const float4*>(row + half + 4 * l));
      const float cv[4] = {cc.x, cc.y, cc.z, cc.w}, sv[4] = {ss.x, ss.y, ss.z, ss.w};
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        ca[k] = cv[k >> 1];
        cb[k] = (k & 1) ? sv[k >> 1] : -sv[k >> 1];
      }
    } else {
      const int i0 = lower ? 8 * l : 8 * l - half;
      load8(row + i0, ca);
      load8(row + half + i0, cb);
#pragma unroll
      for (int k = 0; k < 8; ++k) cb[k] = lower ? -cb[k] : cb[k];
    }
  }
  if (NORM && wt) {
    float wv[8];
    load8(wt + 8 * l, wv);
#pragma unroll
    for (int k = 0; k < 8; ++k) ca[k] *= wv[k];
    if constexpr (INTER) {
#pragma unroll
      for (int k = 0; k < 8; ++k) cb[k] *= wv[k ^ 1];
    } else {
      load8(wt + 8 * (l + away), wv);
#pragma unroll
      for (int k = 0; k < 8; ++k) cb[k] *= wv[k];
    }
  }
  // Where item 0's 16 (8 for e4m3) bytes of this lane go: the query row, or
  // the token's row in the pools (rows hold [H_kv, D]).
  constexpr int OUT = FP8 ? 256 : 512;       // bytes of a k or v item in the pools
  uint8_t* dst;
  int64_t crow = 0;
  if (is_q) {
    dst = reinterpret_cast<uint8_t*>(a.q_out + t * a.q_out_stride) + lane * 16;
  } else {
    const int64_t page = slot / a.bs;
    crow = page * a.block_stride_bytes +
           (slot - page * a.bs) * static_cast<int64_t>(a.H_kv * D * (FP8 ? 1 : 2)) +
           lane * (FP8 ? 8 : 16);
    dst = a.kc + crow;
  }

#pragma unroll
  for (int u = 0; u < kRopeItems; ++u) {
    if (u >= n) break;
    const int item = first + u;
    const bool v = !is_q && item >= nkv;
    const int at = v ? item - nkv : item;
    const bool live = at * 512 + lane * 16 < row_bytes;
    float f[8];
    if (FP8 || !v) unpack8<F16>(x[u], f);
    if (!v) {
      uint4 px;
      if constexpr (INTER) {
        px = make_uint4(prmt(x[u].x, 0, 0x1032), prmt(x[u].y, 0, 0x1032),
                        prmt(x[u].z, 0, 0x1032), prmt(x[u].w, 0, 0x1032));
      } else {
        px.x = __shfl_sync(0xffffffffu, x[u].x, lane + away);
        px.y = __shfl_sync(0xffffffffu, x[u].y, lane + away);
        px.z = __shfl_sync(0xffffffffu, x[u].z, lane + away);
        px.w = __shfl_sync(0xffffffffu, x[u].w, lane + away);
      }
      if (!turns) px = make_uint4(0, 0, 0, 0);
      float g[8];
      unpack8<F16>(px, g);
      float r = 1.f;
      if (NORM && wt) {
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int k = 0; k < 8; k += 2) ffma2(s0, s1, f[k], f[k + 1], f[k], f[k + 1], s0, s1);
        float ss = s0 + s1;
#pragma unroll
        for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        r = rsqrtf(ss * (1.f / D) + a.eps);
      }
#pragma unroll
      for (int k = 0; k < 8; k += 2) {
        fmul2(f[k], f[k + 1], f[k], f[k + 1], ca[k], ca[k + 1]);
        ffma2(f[k], f[k + 1], g[k], g[k + 1], cb[k], cb[k + 1], f[k], f[k + 1]);
        if (NORM) fmul2(f[k], f[k + 1], f[k], f[k + 1], r, r);
      }
    }
    if (!live) continue;
    // What neither the norm nor the rotation touches keeps its bits.
    const bool as_is = v || (!turns && !wt);
    if (!FP8 || is_q) {
      const uint4 y = as_is ? x[u] : pack8<F16>(f);
      *reinterpret_cast<uint4*>((v ? a.vc + crow : dst) + at * 512) = y;
    } else if constexpr (FP8) {
      const int h = at * HPI + lane / LPH;
      const ScaleDiv d = scale_div(__ldg((v ? a.v_scale : a.k_scale) + h));
      *reinterpret_cast<uint2*>((v ? a.vc + crow : dst) + at * OUT) = quantize8(f, d);
    }
  }
}

template <int D, bool F16, bool FP8>
static cudaError_t launch_rope_d(const RopeArgs& a, unsigned grid, cudaStream_t st) {
  auto run = [&](auto kernel) {
    kernel<<<grid, 32, 0, st>>>(a);
    return cudaGetLastError();
  };
  const bool norm = a.q_norm || a.k_norm;
  if (a.interleaved) return norm ? run(rope_and_cache_kernel<D, F16, FP8, true, true>)
                                 : run(rope_and_cache_kernel<D, F16, FP8, true, false>);
  return norm ? run(rope_and_cache_kernel<D, F16, FP8, false, true>)
              : run(rope_and_cache_kernel<D, F16, FP8, false, false>);
}

cudaError_t launch_rope_and_cache(RopeArgs a, int D, bool f16, bool fp8, cudaStream_t st,
                                  int sms) {
  if (a.num_tokens == 0) return cudaSuccess;
  const int hpi = 256 / D;
  const int q_items = (a.H + hpi - 1) / hpi, kv_items = 2 * ((a.H_kv + hpi - 1) / hpi);
  // Few tokens: their heads are shared among more warps, down to one item
  // each, until about 24 warps per SM have work.
  const long long want =
      static_cast<long long>(a.num_tokens) * (q_items + kv_items) / (24LL * sms);
  const int per = static_cast<int>(want < 1 ? 1 : (want > kRopeItems ? kRopeItems : want));
  a.items_per_warp = per;
  a.q_chunks = (q_items + per - 1) / per;
  a.chunks = a.q_chunks + (kv_items + per - 1) / per;
  const long long warps = static_cast<long long>(a.num_tokens) * a.chunks;
  if (warps > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const unsigned grid = static_cast<unsigned>(warps);
  if (fp8) return f16 ? launch_rope_d<128, true, true>(a, grid, st)
                      : launch_rope_d<128, false, true>(a, grid, st);
  if (f16) {
    if (D == 256) return launch_rope_d<256, true, false>(a, grid, st);
    if (D == 128) return launch_rope_d<128, true, false>(a, grid, st);
    return launch_rope_d<64, true, false>(a, grid, st);
  }
  if (D == 256) return launch_rope_d<256, false, false>(a, grid, st);
  if (D == 128) return launch_rope_d<128, false, false>(a, grid, st);
  return launch_rope_d<64, false, false>(a, grid, st);
}

}  // namespace pa
