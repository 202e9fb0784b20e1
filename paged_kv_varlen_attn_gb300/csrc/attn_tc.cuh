// What the tensor-core (tcgen05) prefill kernels share: tile configuration,
// barriers, and the softmax warpgroup with its epilogue. attn_tc.cu describes
// the design; int4_prompt.cu is its form over 4-bit pools.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "device_common.cuh"
#include "epilogue.cuh"

namespace pa {

// Head sizes 64 and 128: two Q tiles per CTA and 128-key K/V tiles. Head
// size 256: one Q tile (its O takes 256 TMEM columns) and 64-key K/V tiles,
// so that two ring stages fit beside the 64 KB Q tile.
template <int D>
struct TcCfg {
  static constexpr int BM = 128;         // rows per Q tile (TMEM lanes)
  static constexpr int TILES = tc_tiles(D);   // Q tiles per CTA
  static constexpr int BN = D > 128 ? 64 : 128;   // keys per K/V tile
  static constexpr int HALVES = D / 64;
  static constexpr int Q_HALF = BM * 128;
  static constexpr int Q_TILE = HALVES * Q_HALF;
  static constexpr int KV_HALF = BN * 128;
  static constexpr int KV_TILE = HALVES * KV_HALF;
  static constexpr int STAGE = 2 * KV_TILE;
  static constexpr int STAGES = D == 64 ? 4 : 2;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_KV = TILES * Q_TILE;
  static constexpr int OFF_BAR = OFF_KV + STAGES * STAGE;
  static constexpr int SMEM_BYTES = OFF_BAR + 512 + 1024;
  static constexpr int THREADS = 384;   // 3 warpgroups: control, softmax A, softmax B
  static constexpr int TMEM_COLS = 512;
  // TMEM columns: S of tile X at X*128 (P of tile X as bf16 or f16 pairs in
  // its first BN / 2 columns); O of tile X at 256 + X*D.
  static constexpr int O_COL = 256;
  static constexpr float RESCALE_LOG2 = 8.0f;
};
// FP8 (e4m3) pools, head size 128. S = Q K^T runs on the e4m3 tensor MMA
// (kind::f8f6f4) straight from the TMA-staged key bytes, with Q taken as two
// e4m3 terms Qh + Ql after a power-of-two row scale (split in place, in the Q
// tiles' own shared memory, by two converter warps); P V stays on kind::f16:
// the converter warps widen each e4m3 V tile (exactly) into f16 tiles laid
// out as the 2-byte kernel's TMA tiles. Shared memory: Q 64 KB (Qh and Ql of
// tile X in its two 16 KB halves after the split), two widened V buffers
// (64 KB: V(t + 1) is widened while the P V products of tile t still read
// V(t)), two e4m3 stages of 32 KB, 1 KB of row scales. Measured on the 70B
// prefill with the keys widened too (one K buffer): 831 TFLOP/s; without
// widening the keys the converters' work halves.
struct TcFp8 {
  using C = TcCfg<128>;
  static constexpr int VBUF = 2;                          // widened V buffers
  static constexpr int OFF_VW = C::TILES * C::Q_TILE;     // widened V tiles
  static constexpr int OFF_R8 = OFF_VW + VBUF * C::KV_TILE;   // e4m3 ring
  static constexpr int TILE8 = C::BN * 128;               // 128 keys x 128 bytes
  static constexpr int STAGE8 = 2 * TILE8;
  static constexpr int STAGES8 = 2;                       // e4m3 ring stages
  static constexpr int OFF_RS = OFF_R8 + STAGES8 * STAGE8;   // float[TILES * BM]: 2^-k per row
  static constexpr int OFF_BAR = OFF_RS + C::TILES * C::BM * 4;
  static constexpr int SMEM_BYTES = OFF_BAR + 512 + 1024;
  static constexpr int CONV_THREADS = 64;                 // warps 2 and 3
};
static_assert(TcFp8::SMEM_BYTES <= 227 * 1024, "the FP8 layout fits shared memory");
static_assert(kTcTileRows == TcCfg<128>::BM, "a Q tile spans the 128 TMEM lanes");
static_assert(TcCfg<256>::SMEM_BYTES <= 227 * 1024, "head size 256 fits shared memory");
static_assert(TcCfg<256>::O_COL + 256 <= TcCfg<256>::TMEM_COLS, "head size 256 fits TMEM");

// Over 4-bit pools (head sizes 64 and 128): K is widened to codes in Q's type and V
// to f16 values, in tiles laid out as the 2-byte kernel's, two buffers of each, by
// warps 0 (K), 2 and 3 (V), which read the codes through rings of asynchronous
// copies of their own. A unit is 16 keys of K or of V: its codes and its 16 (scale,
// minimum) pairs.
template <int D>
struct TcI4 {
  using C = TcCfg<D>;
  static constexpr int BUFS = 2;                          // widened K and V tiles
  static constexpr int OFF_KW = C::TILES * C::Q_TILE;
  static constexpr int OFF_VW = OFF_KW + BUFS * C::KV_TILE;
  static constexpr int OFF_RING = OFF_VW + BUFS * C::KV_TILE;
  static constexpr int UNITS = C::BN / 16;                // of a K or V tile
  static constexpr int WARPS = 3;
  static constexpr int SLOTS = 8;                         // units in a warp's ring
  static constexpr int SLOT = 16 * D / 2 + 64;
  // Per key tile: scale (x 2^24 where the codes are 2^-24 of theirs) and minimum of
  // its keys as float32, (s, s, m, m) of two keys at a time. Those of tile t are
  // written when S(t - 2) is complete, so a ring of four leaves the softmax of t -
  // 1 its own.
  static constexpr int PARS = 4;
  static constexpr int OFF_PAR = OFF_RING + WARPS * SLOTS * SLOT;
  static constexpr int OFF_BAR = OFF_PAR + PARS * C::BN * 8;
  static constexpr int SMEM_BYTES = OFF_BAR + 512 + 1024;
};
static_assert(TcI4<128>::SMEM_BYTES <= 227 * 1024, "the 4-bit layout fits shared memory");

struct TcBars {
  uint64_t q_full;
  uint64_t kv_full[8];     // [s]: K of stage s, [STAGES + s]: V of stage s
  uint64_t kv_empty[8];
  uint64_t s_full[2];      // [tile]: S = Q K^T of the current key tile is in TMEM
  uint64_t p_full[2][2];   // [half][tile]: P of keys [64 half, +64) of the tile is in TMEM
  uint64_t pv_done[2];     // [tile]: O += P V of the current key tile completed
  uint64_t drain;
  // FP8 pools: Q split into e4m3 terms (64 converter arrivals); [buffer]:
  // widened V tile ready (64 arrivals), widened V buffer free again (MMA
  // commit). Buffer b holds tiles b, b + VBUF, ... (phase t / VBUF).
  uint64_t q_conv, vw_full[2], vw_free[2];
  // 4-bit pools: likewise widened K tiles (vw for V), one arrival per widening warp,
  // and the keys' scales and minima.
  uint64_t kw_full[2], kw_free[2], par_full[4];
  uint32_t tmem_base;
  volatile int abort;
  volatile int last;
  volatile int issued[2];    // K / V tiles issued by the producer
  volatile int consumed[2];  // K / V tiles whose arrival the MMA issuer observed
  int first_key;             // SC: first key that some row of the item sees
};

// V rows past the sequence end hold arbitrary bytes: zero them so the P V
// product (P = 0 there) cannot pick up NaN. Tile A's warps do it for key
// tile t before they publish the first half of its P; the MMA thread issues
// every product on V(t) -- tile A's and tile B's -- after observing that, so
// they all see the zeros. V(t) has its own barrier and may land after S(t):
// wait for it first, so the copy cannot overwrite the zeros. False on
// timeout.
// Sliding window (WIN), and changed masks: likewise the rows of keys [first, lo),
// which no query of the item sees.
template <int D, bool WIN>
__device__ __forceinline__ bool zero_v_tail(TcBars* bars, uint8_t* smem, int t, int key0,
                                            int kv_len, int tid, int first_key, int lo) {
  using C = TcCfg<D>;
  if (!mbar_wait(&bars->kv_full[C::STAGES + t % C::STAGES], (t / C::STAGES) & 1)) return false;
  const int first = max(0, kv_len - key0);
  uint8_t* vt = smem + C::OFF_KV + (t % C::STAGES) * C::STAGE + C::KV_TILE;
  const int n16 = (C::BN - first) * C::HALVES * 8;
  for (int idx = tid; idx < n16; idx += 128) {
    const int rr = first + idx / (C::HALVES * 8);
    const int rem = idx % (C::HALVES * 8);
    *reinterpret_cast<uint4*>(vt + (rem >> 3) * C::KV_HALF + rr * 128 + (rem & 7) * 16) =
        make_uint4(0, 0, 0, 0);
  }
  if constexpr (WIN) {
    const int from = max(0, first_key - key0), to = min(C::BN, lo - key0);
    for (int idx = tid; idx < (to - from) * C::HALVES * 8; idx += 128) {
      const int rr = from + idx / (C::HALVES * 8);
      const int rem = idx % (C::HALVES * 8);
      *reinterpret_cast<uint4*>(vt + (rem >> 3) * C::KV_HALF + rr * 128 + (rem & 7) * 16) =
          make_uint4(0, 0, 0, 0);
    }
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  return true;
}

// The kinds of the prefill kernels. FP8, I4: what the pools hold (else elements of
// the activations' type). WIN: sliding window. SC: changed scores and masks. WCAP: the
// cap is above kWideCap (a kernel of its own, since the code for it, unused, cost chunks
// with a bias at head size 64 132 -> 135 us).
template <int D_, bool F16_, bool FP8_, bool WIN_, bool SC_ = false, bool I4_ = false,
          bool WCAP_ = false>
struct TcKind {
  static constexpr int D = D_;
  static constexpr bool F16 = F16_, FP8 = FP8_, WIN = WIN_, SC = SC_, I4 = I4_, WCAP = WCAP_;
  // V reaches the MMA widened, P in f16.
  static constexpr bool WIDE = FP8 || I4;
};
static_assert(sizeof(TcBars) <= 512, "the barriers' place");

// Bits 0 .. n - 1 (none for n <= 0, all from n = 32 on).
__device__ __forceinline__ uint32_t below_mask(int n) {
  return n >= 32 ? ~0u : (n <= 0 ? 0u : (1u << n) - 1u);
}

// A load from shared memory that stays in its place among others.
__device__ __forceinline__ float4 lds_in_order(uint32_t at) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(at));
  return v;
}

// Sum of row r of a Q tile (128-byte swizzled rows of 64 elements).
template <int D, bool F16>
__device__ __forceinline__ float q_row_sum(const uint8_t* q, int r) {
  using C = TcCfg<D>;
  float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1   // (few registers: the caller has none to spare)
  for (int c = 0; c < D / 8; ++c) {
    const uint4 x = *reinterpret_cast<const uint4*>(q + (c >> 3) * C::Q_HALF + r * 128 +
                                                    (((c & 7) ^ (r & 7)) << 4));
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = Elem<F16>::unpack(w[k]);
      s[k] += f.x + f.y;
    }
  }
  return (s[0] + s[1]) + (s[2] + s[3]);
}

// x P(x^2) of two values, P's N coefficients the given ones.
template <int N>
__device__ __forceinline__ void odd_poly2(float& x0, float& x1, const float (&c)[N]) {
  float t0, t1, y0 = c[N - 1], y1 = c[N - 1];
  fmul2(t0, t1, x0, x1, x0, x1);
#pragma unroll
  for (int k = N - 2; k >= 0; --k) ffma2(y0, y1, y0, y1, t0, t1, c[k], c[k]);
  fmul2(x0, x1, x0, x1, y0, y1);
}

// SC: what a tile's values become scores with (in base 2): value x factor + bias of
// its group of eight keys, base + step x group.
struct TileScore {
  float factor, base, step;
};
// A tile's raw products, capped and biased (see pa.h), as values of a TileScore. The
// cap's tanh(u) = 1 - 2 / (1 + e^2u) takes two exponential-unit operations an element
// where the softmax itself takes one, so tiles whose |u| all stay below 1/2 (scores up
// to half the cap), or below 1, take a polynomial on the FMA pipe: four prompts of 2500
// to 4096 tokens, 32 heads of 128, 421 us where the exponential takes 487 and no cap
// 330. (A shorter polynomial for |u| below 1/4 gave nothing back: the code grew.) A
// tile with keys that a row does not see takes the exponentials, so that what those
// keys hold does not choose the form, and rows outside the item have no say; for a cap
// above kWideCap (WCAP) its elements choose by themselves.
// The bias is slope (key - row): each value takes its distance to the group's last key
// with its factor, in one two-lane FMA, and the group's own is left to the maximum and
// the exponent, once a group. (Last, so that the nearest key's score is not rounded at
// the size of the slope.) A tile across the diagonal of a row takes the distance's
// magnitude, an element at a time; the warp decides together, or both forms run. Six
// chunks of 701 tokens, 16 heads of 64: 131 us, 156 with a bias an element, 116 with
// none.
template <int BN, bool WCAP>
__device__ __forceinline__ TileScore score_tile(const AttnArgs& a, float* xs, float sl2, float slope,
                                                int pos, int key0, bool rvalid, bool hides) {
  float factor = sl2;
  if (a.cap > 0.f) {
    factor = a.cap;
    float m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int e = 0; e < BN; e += 8)
#pragma unroll
      for (int j = 0; j < 4; ++j) m[j] = fmax3(m[j], fabsf(xs[e + 2 * j]), fabsf(xs[e + 2 * j + 1]));
    float x = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
    if (!rvalid) x = 0.f;
    else if (hides) x = INFINITY;
    if (__builtin_expect(__all_sync(0xffffffffu, x <= a.cap_x4), 1)) {
#pragma unroll
      for (int e = 0; e < BN; e += 2) odd_poly2(xs[e], xs[e + 1], a.cap_c4);
    } else if (__all_sync(0xffffffffu, x * fabsf(a.cap_u) <= 1.f)) {
      // (As kTanhHalf0 .. 3, of seven terms for |u| <= 1: off by 7e-8 relative in float32.)
      constexpr float c7[7] = {0.99999994f,   -0.333328396f,  0.13325204f,  -0.0534570292f,
                               0.0202899817f, -0.00620337948f, 0.0010410226f};
#pragma unroll
      for (int e = 0; e < BN; e += 2) {
        fmul2(xs[e], xs[e + 1], xs[e], xs[e + 1], a.cap_u, a.cap_u);
        odd_poly2(xs[e], xs[e + 1], c7);
      }
    } else {
#pragma unroll
      for (int e = 0; e < BN; ++e)
        xs[e] = WCAP ? wide_capped_score(xs[e], a.cap_in, a.cap_u, 1.f)
                     : capped_score(xs[e], a.cap_in, 1.f);
    }
  } else if (sl2 < 0.f) {   // (the maximum comes before the factor)
    factor = -sl2;
#pragma unroll
    for (int e = 0; e < BN; ++e) xs[e] = -xs[e];
  }
  TileScore ts = {factor, 0.f, 0.f};
  if (a.slopes) {
    if (__all_sync(0xffffffffu, key0 + BN - 1 <= pos)) {
      ts.base = slope * static_cast<float>(key0 + 7 - pos);
      ts.step = slope * 8.f;
      float se[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) se[k] = slope * static_cast<float>(k - 7);
#pragma unroll
      for (int e = 0; e < BN; e += 2)
        ffma2(xs[e], xs[e + 1], xs[e], xs[e + 1], factor, factor, se[e & 7], se[(e + 1) & 7]);
    } else {
      const float d = static_cast<float>(key0 - pos);
#pragma unroll
      for (int e = 0; e < BN; ++e)
        xs[e] = fmaf(-slope, fabsf(d + static_cast<float>(e)), xs[e] * factor);
    }
    ts.factor = 1.f;
  }
  return ts;
}

// prefix (SC): keys that every row sees, causal or not.
template <class Kind>
__device__ __forceinline__ void tc_softmax_tile(const AttnArgs& a, TcBars* bars, uint8_t* smem,
                                                uint32_t tmem, int X, int q_start, int q_len,
                                                int kv_len, int kb, int ke, int ntiles, int row0,
                                                int R, int hk, int nsplit, int slot_base, int rt,
                                                int j, int win_lo, int prefix = 0) {
  constexpr int D = Kind::D;
  constexpr bool F16 = Kind::F16, FP8 = Kind::FP8, WIN = Kind::WIN, SC = Kind::SC, I4 = Kind::I4;
  using C = TcCfg<D>;
  using E = Elem<F16>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3;
  const int r = quarter * 32 + lane;              // TMEM lane
  const int TR = tc_tile_rows(a.G);               // rows of a Q tile (whole tokens)
  const int rl = X * TR + r;                      // row within the work item
  const uint32_t tm_row = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
  const uint32_t s_col = X * 128, o_col = C::O_COL + X * D;   // S / P and O columns
  const int G = a.G;
  const bool rvalid = r < TR && rl < R;
  const int pr = row0 + (rvalid ? rl : 0);
  const int ti = pr / G;
  const int tok = q_start + ti;
  const int head = hk * G + (pr - ti * G);
  // Last key this row may see (bottom-right causal), or the last key.
  int lim = !rvalid ? -1 : (a.causal ? kv_len - q_len + ti : kv_len - 1);
  // SC: this row's position, first key, and bias per key of distance (base 2).
  const int pos = rvalid ? lim : 1 << 30;
  int low = 0;
  float slope = 0.f;
  if constexpr (SC) {
    if (rvalid) {
      lim = max(lim, prefix - 1);
      if (a.first_key) low = max(__ldg(a.first_key + tok), 0);
      if (a.slopes) slope = __ldg(a.slopes + head) * kLog2e;
    }
  }
  // FP8 pools: scores use the stored codes, so k_scale joins the softmax
  // scale and v_scale the final normalisation.
  // 4-bit pools: the scale's sign has joined the keys' scales and minima (zeros
  // for a scale of zero).
  float sl2 = FP8  ? a.scale_log2 * __ldg(a.k_scale + hk)
              : I4 ? (a.scale_log2 == 0.f ? 1.f : fabsf(a.scale_log2))
                   : a.scale_log2;
  const int tid = threadIdx.x - 128 - X * 128;     // 0..127 within the warpgroup
  float m_use = -INFINITY, l = 0.f;
  bool ok = true;
  if constexpr (FP8) {
    // S holds q 2^k . k for the row's power of two 2^k (Q entered the e4m3
    // products as two e4m3 terms): 2^-k joins the softmax scale.
    if (ntiles > 0) {
      ok = mbar_wait(&bars->q_conv, 0);
      sl2 *= reinterpret_cast<const float*>(smem + TcFp8::OFF_RS)[X * C::BM + r];
    }
  }
  float tau = 0.f;   // I4: sum of the row's q
  if constexpr (I4) {
    if (ntiles > 0 && (ok = mbar_wait(&bars->q_full, 0)))
      tau = q_row_sum<D, F16>(smem + C::OFF_Q + X * C::Q_TILE, r);
  }
  for (int t = 0; ok && t < ntiles; ++t) {
    if (!mbar_wait(&bars->s_full[X], t & 1)) { ok = false; break; }
    tc_fence_after();
    const int key0 = kb + t * C::BN;
    const int vis_end = min(ke, lim + 1);   // keys [key0, vis_end) are visible
    const bool edge = key0 + C::BN > vis_end;
    uint32_t xs_u[C::BN];
#pragma unroll
    for (int c = 0; c < C::BN / 32; ++c)
      tmem_ld32(tm_row + s_col + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&xs_u[c * 32]));
    tmem_wait_ld();
    float* xs = reinterpret_cast<float*>(xs_u);
    if constexpr (I4) {
      // The products are with the keys' codes: q.k = scale (q.n) + minimum (sum of
      // q), in float32.
      using I = TcI4<D>;
      if (!mbar_wait(&bars->par_full[t % I::PARS], (t / I::PARS) & 1)) { ok = false; break; }
      const uint32_t par = smem_u32(smem + I::OFF_PAR + t % I::PARS * C::BN * 8);
      constexpr int AHEAD = 4;   // loads in flight (more of them, and registers spill)
#pragma unroll
      for (int e0 = 0; e0 < C::BN; e0 += 2 * AHEAD) {
        float4 p[AHEAD];
#pragma unroll
        for (int x = 0; x < AHEAD; ++x) p[x] = lds_in_order(par + (e0 + 2 * x) * 8);
#pragma unroll
        for (int x = 0; x < AHEAD; ++x) {
          const int e = e0 + 2 * x;
          float u0, u1;
          fmul2(u0, u1, p[x].z, p[x].w, tau, tau);
          ffma2(xs[e], xs[e + 1], p[x].x, p[x].y, xs[e], xs[e + 1], u0, u1);
        }
      }
    }
    TileScore ts = {sl2, 0.f, 0.f};
    if constexpr (SC) {
      ts = score_tile<C::BN, Kind::WCAP>(a, xs, sl2, slope, pos, key0, rvalid, edge || key0 < low);
      if (edge || key0 < low) {
#pragma unroll
        for (int c = 0; c < C::BN / 32; ++c) {
          const int base = key0 + c * 32;
          const uint32_t seen = below_mask(vis_end - base) & ~below_mask(low - base);
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (!(seen & (1u << e))) xs[c * 32 + e] = -INFINITY;
        }
      }
    } else if constexpr (WIN) {
      // Visible: keys below vis_end that are first tokens or past lim - window,
      // as one bit per key, so that the tests of an edge tile cost an element
      // two instructions.
      const int win_from = max(lim - a.window + 1, 0);
      if (edge || (key0 < win_from && key0 + C::BN > a.first)) {
#pragma unroll
        for (int c = 0; c < C::BN / 32; ++c) {
          const int base = key0 + c * 32;
          const uint32_t seen = below_mask(vis_end - base) &
                                (below_mask(a.first - base) | ~below_mask(win_from - base));
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (!(seen & (1u << e))) xs[c * 32 + e] = -INFINITY;
        }
      }
    } else if (edge) {
#pragma unroll
      for (int e = 0; e < C::BN; ++e)
        if (key0 + e >= vis_end) xs[e] = -INFINITY;
    }
    // Row max: eight independent chains of three-input maxima over the
    // values j, j+8, j+16, ... of the tile; with a bias per group of eight, the
    // groups' maxima in two chains.
    static_assert(C::BN % 16 == 0, "max chains take two values per step");
    float tmax;
    if constexpr (SC) {
      float mg[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int g = 0; g < C::BN / 8; ++g) {
        const float* x = xs + g * 8;
        const float m = fmaxf(fmax3(fmax3(x[0], x[1], x[2]), x[3], x[4]), fmax3(x[5], x[6], x[7]));
        mg[g & 1] = fmaxf(mg[g & 1], fmaf(m, ts.factor, fmaf(ts.step, static_cast<float>(g), ts.base)));
      }
      tmax = fmaxf(mg[0], mg[1]);
    } else {
      float mx8[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) mx8[j] = fmaxf(xs[j], xs[8 + j]);
#pragma unroll
      for (int e = 16; e < C::BN; e += 16)
#pragma unroll
        for (int j = 0; j < 8; ++j) mx8[j] = fmax3(mx8[j], xs[e + j], xs[e + 8 + j]);
      tmax = fmaxf(fmax3(mx8[0], mx8[1], mx8[2]),
                   fmax3(fmax3(mx8[3], mx8[4], mx8[5]), mx8[6], mx8[7])) *
             ts.factor;
    }
    float m_new = m_use;
    bool need = false;
    if (tmax > m_use) {
      if (m_use == -INFINITY) m_new = tmax;                 // O holds only zeros so far
      else if (tmax - m_use > C::RESCALE_LOG2) { need = true; m_new = tmax; }
    }
    // O_X is final here: this tile's S was issued after the previous P V
    // completed, and its commit covers that product.
    if (__any_sync(0xffffffffu, need)) {
      const float alpha = need ? fast_exp2(m_use - m_new) : 1.f;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t v[32];
        tmem_ld32(tm_row + o_col + c * 32, v);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * alpha);
        tmem_st32(tm_row + o_col + c * 32, v);
      }
      l *= alpha;
    }
    m_use = m_new;
    const float mu = m_use == -INFINITY ? 0.f : m_use;
    // Scores whose unit in the last place is no longer small (past 2^20): the
    // product below, unrounded, would differ from the rounded maximum by more
    // than an exponent can be, so it is rounded first.
    if constexpr (I4 || SC) {
      if (__any_sync(0xffffffffu, fabsf(mu) > 0x1p20f)) {
#pragma unroll
        for (int e = 0; e < C::BN; ++e) xs[e] *= ts.factor;
        ts.factor = 1.f;
      }
    }
    // Pass 2: P = exp2(S * scale * log2(e) - m) as bf16 pairs into the first
    // 64 columns of this tile's S region (key k -> column k / 2). Chunk c
    // reads S columns [32c, 32c+32) and writes P columns [16c, 16c+16), which
    // only the already-read chunks occupy.
    // P is published in two halves (keys 0-63, then 64-127), so the tensor
    // core multiplies the first half by V while the second is computed.
    float ls[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < C::BN / 32; ++c) {
      uint32_t pk[16];
#pragma unroll
      for (int e = 0; e < 32; e += 2) {
        const float c0 = SC ? fmaf(ts.step, static_cast<float>(c * 4 + e / 8), ts.base - mu) : -mu;
        // Pairs in the two-lane FMA / add: half the arithmetic instructions,
        // the same roundings and summation order as the scalar forms. The
        // MMA-issuing thread shares issue slots with these warps, and dense
        // FMA streams beside it starve it (measured: a single issuing thread
        // next to eight warps of FMA/max arithmetic issued one 128x128x16 MMA
        // per ~220 clocks instead of 64; next to exp2-only warps, 64).
        float y0, y1;
        ffma2(y0, y1, xs[c * 32 + e], xs[c * 32 + e + 1], ts.factor, ts.factor, c0, c0);
        const float p0 = fast_exp2(y0), p1 = fast_exp2(y1);
        fadd2(ls[e & 7], ls[(e + 1) & 7], ls[e & 7], ls[(e + 1) & 7], p0, p1);
        pk[e >> 1] = Elem<F16 || Kind::WIDE>::pack(p0, p1);   // P has the MMA's operand type
      }
      tmem_st16(tm_row + s_col + c * 16, pk);
      if (c == C::BN / 64 - 1) {   // the first half of the tile's keys
        tmem_wait_st();
        // warp-uniform condition and result
        if (!Kind::WIDE && X == 0 &&
            (key0 + C::BN > kv_len || (WIN && key0 < win_lo && key0 + C::BN > a.first) ||
             (SC && key0 < win_lo)))
          ok = __all_sync(0xffffffffu, zero_v_tail<D, WIN || SC>(bars, smem, t, key0, kv_len, tid,
                                                                 SC ? 0 : a.first, win_lo));
        if (!ok) break;
        tc_fence_before();
        mbar_arrive(&bars->p_full[0][X]);
      }
    }
    if (!ok) break;
    l += ((ls[0] + ls[1]) + (ls[2] + ls[3])) + ((ls[4] + ls[5]) + (ls[6] + ls[7]));
    tmem_wait_st();
    tc_fence_before();
    mbar_arrive(&bars->p_full[1][X]);
  }
  if (!ok) {
    abort_call(a);
    bars->abort = 1;
  }
  // ---------------------------------------------------------- epilogue
  ok = __all_sync(0xffffffffu, ok);   // TMEM loads below are warp-collective
  if (ok && ntiles > 0) {
    if (!mbar_wait(&bars->pv_done[X], (ntiles - 1) & 1)) {
      abort_call(a);
      bars->abort = 1;
      ok = false;
    }
    ok = __all_sync(0xffffffffu, ok);
    tc_fence_after();
  }
  const bool partial = nsplit > 1 || a.partials_only;
  float mf = m_use, lf = ok ? l : 0.f, of = 1.f;
  if (a.sinks && !partial && rvalid) of = add_sink(mf, lf, __ldg(a.sinks + head) * kLog2e);
  const bool any = ok && lf > 0.f;
  const float inv_l = any ? (FP8 ? __ldg(a.v_scale + hk) : 1.f) * of / lf : 0.f;
  float lse_nat = any ? (mf + fast_log2(lf)) * kLn2 : -INFINITY;
  const int slot = slot_base + rt * nsplit + j;
  const int64_t srow = slot_row(a, slot, hk, rl);
  // The output leaves through shared memory: each warp stages 32 rows x 32
  // columns in its quarter of Q tile X (free once the last S_X product has
  // completed, which the pv_done wait above implies) and stores them so that
  // every instruction writes whole row segments (fp32 partial rows of 128 B,
  // bf16 output rows of 64 B) instead of one 8- or 16-byte piece per row.
  // 16-byte granules are XOR-swizzled by row to keep the shared-memory
  // accesses free of bank conflicts.
  uint8_t* stage = smem + C::OFF_Q + X * C::Q_TILE + quarter * (C::Q_TILE / 4);
  const int rl0 = X * TR + quarter * 32;             // first row of this warp in the item
  const int64_t srow0 = slot_row(a, slot, hk, rl0);  // rows of a slot are consecutive
  // Rows of this warp that exist: inside the tile and inside the item.
  const int wrows = max(0, min(TR - quarter * 32, R - rl0));
#pragma unroll 1
  for (int c = 0; c < D / 32; ++c) {
    uint32_t v[32];
    if (ntiles > 0 && ok) {
      tmem_ld32(tm_row + o_col + c * 32, v);
      tmem_wait_ld();
    } else {
#pragma unroll
      for (int e = 0; e < 32; ++e) v[e] = 0u;
    }
    if (partial) {
#pragma unroll
      for (int g = 0; g < 8; ++g)
        *reinterpret_cast<float4*>(stage + lane * 128 + ((g ^ (lane & 7)) << 4)) =
            make_float4(__uint_as_float(v[4 * g]) * inv_l, __uint_as_float(v[4 * g + 1]) * inv_l,
                        __uint_as_float(v[4 * g + 2]) * inv_l, __uint_as_float(v[4 * g + 3]) * inv_l);
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = i * 4 + (lane >> 3), g = lane & 7;
        if (r < wrows)
          __stcg(reinterpret_cast<float4*>(a.part_o + (srow0 + r) * D + c * 32 + g * 4),
                 *reinterpret_cast<const float4*>(stage + r * 128 + ((g ^ (r & 7)) << 4)));
      }
    } else {
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        uint4 pk;
        pk.x = E::pack(__uint_as_float(v[8 * g]) * inv_l, __uint_as_float(v[8 * g + 1]) * inv_l);
        pk.y = E::pack(__uint_as_float(v[8 * g + 2]) * inv_l, __uint_as_float(v[8 * g + 3]) * inv_l);
        pk.z = E::pack(__uint_as_float(v[8 * g + 4]) * inv_l, __uint_as_float(v[8 * g + 5]) * inv_l);
        pk.w = E::pack(__uint_as_float(v[8 * g + 6]) * inv_l, __uint_as_float(v[8 * g + 7]) * inv_l);
        *reinterpret_cast<uint4*>(stage + lane * 64 + ((g ^ ((lane >> 1) & 3)) << 4)) = pk;
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = i * 8 + (lane >> 2), g = lane & 3;
        if (r < wrows) {
          const int prr = row0 + rl0 + r;
          const int tr = prr / G;
          const int64_t ob = (static_cast<int64_t>(q_start + tr) * a.H + hk * G + (prr - tr * G)) * D;
          *reinterpret_cast<uint4*>(a.out + ob + c * 32 + g * 8) =
              *reinterpret_cast<const uint4*>(stage + r * 64 + ((g ^ ((r >> 1) & 3)) << 4));
        }
      }
    }
    __syncwarp();
  }
  if (rvalid) {
    if (nsplit > 1 || a.partials_only) {
      __stcg(a.part_lse + srow, lse_nat);
    } else if (a.lse) {
      a.lse[static_cast<int64_t>(head) * a.lse_stride + tok] = lse_nat;
    }
  }
}

}  // namespace pa
