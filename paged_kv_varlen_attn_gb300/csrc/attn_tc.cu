// Tensor-core (tcgen05) prefill / chunked-prefill attention kernel.
//
// Computes the paged varlen attention of "FlashAttention 在 vLLM 中的实现分析"
// §4 / §5 with the tiled online softmax of §1.1 for segments with more than
// 64 packed query rows (prefill, chunked prefill with prior context, the
// cascade prefix pass of §6.3).
//
// One CTA per work item: two Q tiles A and B of packed query rows, each
// floor(128/G) tokens x the G query heads of one KV head (128 rows when G
// divides 128; otherwise the 128 TMEM lanes hold the whole tokens that fit
// and the rest stay idle) -- against a key range, in 128-key tiles. Every K/V
// byte brought into shared memory serves every row of both Q tiles (all G
// heads). Three warpgroups:
//   control (warps 0-3; 0 and 1 work, 2 and 3 idle), registers cut to 104;
//   softmax A (warps 4-7) and softmax B (warps 8-11), registers raised to 200.
// Warp roles:
//   warp 0     TMA producer: both Q tiles once, then K and V page boxes
//              (128-byte swizzle) into a ring of stages (full/empty mbarriers),
//              block-table entries prefetched a group of boxes ahead;
//   warp 1     MMA issuer (one lane): for each key tile, S_X = Q_X K^T into
//              TMEM (128 fp32 columns per Q tile X), then O_X += P_X V with P_X
//              read straight from TMEM (the A operand of the MMA) and V from
//              shared memory; tcgen05.commit arrives on the barriers that free
//              each buffer;
//   warps 4-7  softmax of tile A, warps 8-11 softmax of tile B: thread r owns
//              row r of its tile (TMEM lane r). It reads its 128 scores from
//              TMEM with one wait, masks (bottom-right causal, key range), keeps
//              a running max,
//              writes P = exp2(S - m) as bf16 pairs back into the first 64
//              columns of its S region, and finally reads O from TMEM, divides
//              by the row sum and writes the output and LSE.
// Keeping P in TMEM leaves shared memory to the TMA ring and the Q/K/V
// operands: per 128-key tile the tensor core reads Q and K (S) and V (P V)
// from shared memory and nothing else. While one warpgroup computes its
// softmax the tensor core runs the other tile's MMAs.
// The MMA issuer orders each tile as P_A V, S_A(next), P_B V, S_B(next): S_X
// of the next tile overwrites P_X, and the tensor core executes one thread's
// MMAs in issue order, so it runs after P_X V has read P_X; tile A's softmax
// thus starts its next tile without waiting for tile B's. The commit after
// S_X(next) covers P_X V, so O_X is final for the softmax's lazy rescale: a
// row's reference max only moves when its max grows by more than 2^8, so
// most tiles need no TMEM round trip for O (exact, since O and the row sum
// always share the same reference). K and V of a ring stage have separate
// barriers, so K(t) is refilled as soon as both S(t) are done.
// Causal tile skipping: the key range of an item is clamped to the last key
// its last row may see, so tiles above the diagonal are never loaded.
// Sliding window (WIN): the item's keys are numbered without the ones that none
// of its rows sees (WinGeo), so the loops are the same. Items are short: four
// prompts of 3,500-4,500 tokens (32/8 heads of 128) at window 1024 take 340 us,
// 39% of the measured matrix rate for the visible pairs; of an item's 24 us,
// nine key tiles of 128 take 17 (8 hold what a row sees) and 7 go to the start
// before the first product and the output after the last, which nothing
// overlaps at one block per SM. One Q tile per item and two blocks per SM: 469
// us, by twice the TMA boxes per row.
// Every mbarrier wait is bounded; on a timeout the CTA records
// PA_DEV_TIMEOUT and the call's abort word, drains its MMAs and copies, frees
// TMEM and returns.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>

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
  uint32_t tmem_base;
  volatile int abort;
  volatile int last;
  volatile int issued[2];    // K / V tiles issued by the producer
  volatile int consumed[2];  // K / V tiles whose arrival the MMA issuer observed
};

// V rows past the sequence end hold arbitrary bytes: zero them so the P V
// product (P = 0 there) cannot pick up NaN. Tile A's warps do it for key
// tile t before they publish the first half of its P; the MMA thread issues
// every product on V(t) -- tile A's and tile B's -- after observing that, so
// they all see the zeros. V(t) has its own barrier and may land after S(t):
// wait for it first, so the copy cannot overwrite the zeros. False on
// timeout.
// Sliding window (WIN): likewise the rows of keys [first, lo), which no query
// of the item sees.
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

// Widen an e4m3 K or V tile (BN keys x 128 bytes, TMA 128-byte swizzle:
// 16-byte chunk j of row r at r*128 + ((j ^ r%8) << 4)) to f16 in the layout
// of a bf16 TMA tile (two halves of BN rows x 128 bytes; 8-element chunk c
// of row r at r*128 + ((c ^ r%8) << 4)). Every e4m3 value is exact in f16.
// Rows from zero_from on are written as zeros (keys past the sequence end:
// their bytes are arbitrary and P = 0 there must not meet a NaN).
// WIN: rows [hide_from, hide_to) -- keys that no query of the item sees -- too.
template <bool WIN>
__device__ __forceinline__ void widen_e4m3_tile(const uint8_t* src, uint8_t* dst, int ct,
                                                int zero_from, int hide_from, int hide_to) {
  using C = TcCfg<128>;
  static_assert(TcFp8::CONV_THREADS % 8 == 0, "a thread keeps one chunk column");
  // Thread ct takes chunk column jj = ct % 8 of rows ct / 8, ct / 8 + 8, ...;
  // rows 8 apart share their swizzle phase, so every address below is a
  // per-thread base plus a multiple of 8 rows.
  const int jj = ct & 7, r0 = ct >> 3;
  const int s_sw = (jj ^ (r0 & 7)) << 4;                     // e4m3 chunk jj
  const int c0 = 2 * (jj & 3);                               // f16 chunks c0, c0 + 1
  const int d_lo = ((c0 ^ (r0 & 7)) << 4), d_hi = (((c0 + 1) ^ (r0 & 7)) << 4);
  const uint8_t* sp = src + r0 * 128 + s_sw;
  uint8_t* dp = dst + (jj >> 2) * C::KV_HALF + r0 * 128;
  constexpr int kStep = TcFp8::CONV_THREADS / 8;             // rows between a thread's chunks
#pragma unroll 4
  for (int r = r0; r < C::BN; r += kStep, sp += kStep * 128, dp += kStep * 128) {
    uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
    if (r < zero_from && (!WIN || r < hide_from || r >= hide_to)) {
      const uint4 w = *reinterpret_cast<const uint4*>(sp);
      lo = make_uint4(e4m3x2_to_f16x2(w.x), e4m3x2_to_f16x2(w.x >> 16), e4m3x2_to_f16x2(w.y),
                      e4m3x2_to_f16x2(w.y >> 16));
      hi = make_uint4(e4m3x2_to_f16x2(w.z), e4m3x2_to_f16x2(w.z >> 16), e4m3x2_to_f16x2(w.w),
                      e4m3x2_to_f16x2(w.w >> 16));
    }
    *reinterpret_cast<uint4*>(dp + d_lo) = lo;
    *reinterpret_cast<uint4*>(dp + d_hi) = hi;
  }
}

// Split the Q tiles in place into e4m3 terms for the kind::f8f6f4 S product.
// Row r of tile X holds dims 0..63 in half 0 and 64..127 in half 1 (2-byte
// elements, 128-byte swizzled rows: 16-byte chunk c at r*128 + ((c ^ r%8) << 4)).
// With 2^k putting the row's largest |q| in [128, 256) (k = 126 for a zero
// or subnormal maximum), q 2^k = Qh + Ql with Qh = e4m3(q 2^k) and
// Ql = e4m3(q 2^k - Qh); Qh's 128 bytes (dims in order) replace half 0 and
// Ql's replace half 1, in the same swizzled layout, which is the K-major
// e4m3 operand layout; 2^-k goes to rs[X*128 + r]. Thread ct takes rows ct
// and ct + 64 of each tile. Half 1 is read whole before any write; chunk c
// of half 0 is overwritten only after dims 8c..8c+7 were read.
template <bool F16>
__device__ __forceinline__ void q_split_e4m3(uint8_t* q, float* rs, int tiles, int ct) {
  using C = TcCfg<128>;
  for (int x = 0; x < tiles; ++x) {
    for (int r = ct; r < C::BM; r += TcFp8::CONV_THREADS) {
      uint8_t* h0 = q + x * C::Q_TILE + r * 128;
      uint8_t* h1 = h0 + C::Q_HALF;
      const int sw = r & 7;
      uint4 hi[8];
      float part[8];   // eight independent maximum chains, then a tree
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        hi[c] = *reinterpret_cast<const uint4*>(h1 + ((c ^ sw) << 4));
        const uint4 lo = *reinterpret_cast<const uint4*>(h0 + ((c ^ sw) << 4));
        const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi[c].x, hi[c].y, hi[c].z, hi[c].w};
        float m = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float2 f = Elem<F16>::unpack(w[k]);
          m = fmaxf(m, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
        part[c] = m;
      }
      const float amax = fmaxf(fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3])),
                               fmaxf(fmaxf(part[4], part[5]), fmaxf(part[6], part[7])));
      const int ebits = (__float_as_int(amax) >> 23) & 0xFF;
      const int kexp = max(-126, min(126, ebits == 0 ? 126 : 134 - ebits));
      const float up = __int_as_float((127 + kexp) << 23);
      rs[x * C::BM + r] = __int_as_float((127 - kexp) << 23);
#pragma unroll
      for (int c = 0; c < 8; ++c) {   // dims 16c .. 16c + 15
        uint4 a, b;
        if (c < 4) {
          a = *reinterpret_cast<const uint4*>(h0 + (((2 * c) ^ sw) << 4));
          b = *reinterpret_cast<const uint4*>(h0 + (((2 * c + 1) ^ sw) << 4));
        } else {
          a = hi[2 * c - 8];
          b = hi[2 * c - 7];
        }
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        uint32_t qh[4], ql[4];
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
          uint32_t hh = 0, ll = 0;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float2 f = Elem<F16>::unpack(w[k + e]);
            const float y0 = f.x * up, y1 = f.y * up;
            const uint32_t hb = f32x2_to_e4m3x2(y0, y1);
            const float2 hv = Elem<true>::unpack(e4m3x2_to_f16x2(hb));
            hh |= hb << (16 * e);
            ll |= f32x2_to_e4m3x2(y0 - hv.x, y1 - hv.y) << (16 * e);
          }
          qh[k / 2] = hh;
          ql[k / 2] = ll;
        }
        *reinterpret_cast<uint4*>(h0 + ((c ^ sw) << 4)) = make_uint4(qh[0], qh[1], qh[2], qh[3]);
        *reinterpret_cast<uint4*>(h1 + ((c ^ sw) << 4)) = make_uint4(ql[0], ql[1], ql[2], ql[3]);
      }
    }
  }
}

// Bits 0 .. n - 1 (none for n <= 0, all from n = 32 on).
__device__ __forceinline__ uint32_t below_mask(int n) {
  return n >= 32 ? ~0u : (n <= 0 ? 0u : (1u << n) - 1u);
}

template <int D, bool F16, bool FP8, bool WIN>
__device__ __forceinline__ void tc_softmax_tile(const AttnArgs& a, TcBars* bars, uint8_t* smem,
                                                uint32_t tmem, int X, int q_start, int q_len,
                                                int kv_len, int kb, int ke, int ntiles, int row0,
                                                int R, int hk, int nsplit, int slot_base, int rt,
                                                int j, int win_lo) {
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
  const int lim = !rvalid ? -1 : (a.causal ? kv_len - q_len + ti : kv_len - 1);
  // FP8 pools: scores use the stored codes, so k_scale joins the softmax
  // scale and v_scale the final normalisation.
  float sl2 = FP8 ? a.scale_log2 * __ldg(a.k_scale + hk) : a.scale_log2;
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
    if constexpr (WIN) {
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
    // values j, j+8, j+16, ... of the tile.
    static_assert(C::BN % 16 == 0, "max chains take two values per step");
    float mx8[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) mx8[j] = fmaxf(xs[j], xs[8 + j]);
#pragma unroll
    for (int e = 16; e < C::BN; e += 16)
#pragma unroll
      for (int j = 0; j < 8; ++j) mx8[j] = fmax3(mx8[j], xs[e + j], xs[e + 8 + j]);
    const float tmax = fmaxf(fmax3(mx8[0], mx8[1], mx8[2]),
                             fmax3(fmax3(mx8[3], mx8[4], mx8[5]), mx8[6], mx8[7])) * sl2;
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
        // Pairs in the two-lane FMA / add: half the arithmetic instructions,
        // the same roundings and summation order as the scalar forms. The
        // MMA-issuing thread shares issue slots with these warps, and dense
        // FMA streams beside it starve it (measured: a single issuing thread
        // next to eight warps of FMA/max arithmetic issued one 128x128x16 MMA
        // per ~220 clocks instead of 64; next to exp2-only warps, 64).
        float y0, y1;
        ffma2(y0, y1, xs[c * 32 + e], xs[c * 32 + e + 1], sl2, sl2, -mu, -mu);
        const float p0 = fast_exp2(y0), p1 = fast_exp2(y1);
        fadd2(ls[e & 7], ls[(e + 1) & 7], ls[e & 7], ls[(e + 1) & 7], p0, p1);
        pk[e >> 1] = Elem<F16 || FP8>::pack(p0, p1);   // P has the MMA's operand type
      }
      tmem_st16(tm_row + s_col + c * 16, pk);
      if (c == C::BN / 64 - 1) {   // the first half of the tile's keys
        tmem_wait_st();
        // warp-uniform condition and result
        if (!FP8 && X == 0 &&
            (key0 + C::BN > kv_len || (WIN && key0 < win_lo && key0 + C::BN > a.first)))
          ok = __all_sync(0xffffffffu, zero_v_tail<D, WIN>(bars, smem, t, key0, kv_len, tid,
                                                           a.first, win_lo));
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

template <int D, bool F16, bool FP8, bool WIN>
__global__ void __launch_bounds__(TcCfg<D>::THREADS, 1)
attn_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
               const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ AttnArgs a) {
  using C = TcCfg<D>;
  static_assert(!FP8 || D == 128, "FP8 pools: head size 128");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  TcBars* bars = reinterpret_cast<TcBars*>(smem + (FP8 ? TcFp8::OFF_BAR : C::OFF_BAR));

  pdl_enter(a.pdl_first);
  if (static_cast<int>(blockIdx.x) >= a.header[1] || call_aborted(a)) return;
  const int hk = blockIdx.y;
  const int4 it = a.items[blockIdx.x];
  const int seg = it.x, rt = it.y, j = it.z;
  const int4 sg = a.seg[seg];
  const int4 sp = a.segsplit[seg];
  const int q_start = sg.x, q_len = sg.y, kv_len = sg.z;
  const int nsplit = sp.x, slot_base = sp.y, chunk = sp.z;
  const int G = a.G;
  const int TR = tc_tile_rows(G);   // rows of a Q tile: TR / G whole tokens
  const int row0 = rt * C::TILES * TR;
  const int R = min(C::TILES * TR, q_len * G - row0);
  const bool two = R > TR;   // tile B has rows
  const int kb = j * chunk;
  // Sliding window: the item works on virtual keys, the sequence is len long.
  WinGeo geo{};
  if constexpr (WIN)
    geo = win_geo(kv_len, q_len, row0 / G, (row0 + R - 1) / G, a.window, a.first, a.box_rows);
  const int len = WIN ? kv_len - geo.gap : kv_len;
  const int win_lo = geo.lo - geo.gap;
  int ke = min(len, kb + chunk);
  if (a.causal) ke = min(ke, len - q_len + (row0 + R - 1) / G + 1);
  const int ntiles = ke > kb ? (ke - kb + C::BN - 1) / C::BN : 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(&bars->q_full, 1);
    for (int s = 0; s < 2 * C::STAGES; ++s) {
      mbar_init(&bars->kv_full[s], 1);
      // FP8: an e4m3 K stage is freed by the commit after its S products, a
      // V stage by the converter warps once they widened it.
      mbar_init(&bars->kv_empty[s], FP8 && s >= C::STAGES ? TcFp8::CONV_THREADS : 1);
    }
    if constexpr (FP8) {
      static_assert(TcFp8::STAGES8 == C::STAGES, "the e4m3 ring has the 2-byte ring's stages");
      mbar_init(&bars->q_conv, TcFp8::CONV_THREADS);
      for (int b = 0; b < 2; ++b) {
        mbar_init(&bars->vw_full[b], TcFp8::CONV_THREADS);
        mbar_init(&bars->vw_free[b], 1);
      }
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&bars->s_full[x], 1);
      mbar_init(&bars->p_full[0][x], 128);
      mbar_init(&bars->p_full[1][x], 128);
      mbar_init(&bars->pv_done[x], 1);
    }
    mbar_init(&bars->drain, 1);
    bars->abort = 0;
    bars->last = 0;
    bars->issued[0] = bars->issued[1] = 0;
    bars->consumed[0] = bars->consumed[1] = 0;
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
  // Register split: the block is launched with 384 x 168 registers. The
  // control warpgroup (producer, MMA issuer, two idle warps) drops to 104 and
  // the two softmax warpgroups rise to 200: 128*104 + 256*200 = 384*168
  // (the sum must not exceed the launch's, or setmaxnreg.inc never
  // returns). The softmax's two-lane FMAs need aligned register pairs; with
  // 200 registers they fit (measured on the 70B prefill: 1376 TFLOP/s at
  // 104/200 against 1202 at 120/192 with the two-lane FMA and 1348 at
  // 120/192 without it; 88/208 spills in the issuer, 1277).

  if (warp < 4) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 104;" ::: "memory");
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (ntiles > 0) {
      if (lane == 0) {
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
        // A Q box is TR / G tokens x G heads x 64 dims: TR rows of 128 B in
        // packed-row order. Lanes TR..127 of a tile keep stale rows, which
        // only feed their own (never written) S and O rows.
        const int token0 = q_start + row0 / G;
        mbar_arrive_expect_tx(&bars->q_full, (two ? 2 : 1) * C::HALVES * TR * 128);
        for (int x = 0; x < (two ? 2 : 1); ++x)
          for (int h = 0; h < C::HALVES; ++h)
            tma_load_3d(smem + C::OFF_Q + x * C::Q_TILE + h * C::Q_HALF, &tmQ, &bars->q_full,
                        h * 64, hk * G, token0 + x * (TR / G));
      }
      const int32_t* bt_row =
          a.bt + static_cast<int64_t>(seg) * a.bt_row_stride + a.bt_col_offset;
      if constexpr (FP8) {
        static_assert(2 * TcFp8::STAGES8 <= 8, "the ring barrier arrays hold 8");
        produce_kv<C::BN, 1, TcFp8::STAGES8, true, WIN>(
            &tmK, &tmV, a, smem + TcFp8::OFF_R8, bars->kv_full, bars->kv_empty, &bars->abort,
            bars->issued, bt_row, hk, kb, kv_len, ntiles, lane, 0, geo);
      } else {
        produce_kv<C::BN, C::HALVES, C::STAGES, true, WIN>(
            &tmK, &tmV, a, smem + C::OFF_KV, bars->kv_full, bars->kv_empty, &bars->abort,
            bars->issued, bt_row, hk, kb, kv_len, ntiles, lane, 0, geo);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // One lane issues. The tensor core starves when this thread gets few
    // issue slots (the softmax warps' arithmetic competes for them), so the
    // work per MMA is kept small: descriptor bases are built once and each
    // MMA adds a constant (the descriptor of address + c is the descriptor of
    // address plus c / 16; shared addresses stay below 2^18, so the 14-bit
    // field cannot carry).
    if (lane == 0 && ntiles > 0) {
      bool ok;
      if constexpr (!FP8) {
        // Operand type: the activations' (bf16 or f16).
        constexpr uint32_t fmt = Elem<F16>::kTcFormat;
        constexpr uint32_t idesc_s = mma_idesc(C::BM, C::BN, false, fmt);
        constexpr uint32_t idesc_o = mma_idesc(C::BM, D, true, fmt);
        // K / V operands: ring stage t % STAGES.
        constexpr int kBufs = C::STAGES;
        constexpr int vBufs = C::STAGES;
        constexpr int kStep = C::STAGE >> 4;   // descriptor step per stage
        const uint32_t sK = smem_u32(smem + C::OFF_KV);
        const uint32_t sV = sK + C::KV_TILE;
        const uint64_t qdesc[2] = {smem_desc_sw128(smem_u32(smem + C::OFF_Q), 16, 1024),
                                   smem_desc_sw128(smem_u32(smem + C::OFF_Q + C::Q_TILE), 16, 1024)};
        const uint64_t kdesc0 = smem_desc_sw128(sK, 16, 1024);
        const uint64_t vdesc0 = smem_desc_sw128(sV, C::KV_HALF, 1024);
        // S_X(t) = Q_X K(t)^T into TMEM columns [128 X, 128 X + 128).
        auto issue_s = [&](int x, int t) {
          tc_fence_after();
          const uint64_t qd = qdesc[x];
          const uint64_t kd = kdesc0 + static_cast<uint32_t>((t % kBufs) * kStep);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = ((kk >> 2) * C::Q_HALF + (kk & 3) * 32) >> 4;
            const uint32_t offk = ((kk >> 2) * C::KV_HALF + (kk & 3) * 32) >> 4;
            tc_mma(tmem + x * 128, qd + off, kd + offk, idesc_s, kk > 0);
          }
          tc_commit(&bars->s_full[x]);
        };
        // O_X += P_X(t) V(t) over keys [64 h, 64 h + 64), P_X read from TMEM
        // (the first 64 columns of S_X); the second half commits pv_done.
        auto issue_pv = [&](int x, int t, int h) {
          tc_fence_after();
          const uint64_t vd = vdesc0 + static_cast<uint32_t>((t % vBufs) * kStep);
#pragma unroll
          for (int k4 = 0; k4 < C::BN / 32; ++k4) {
            const int kk = h * (C::BN / 32) + k4;
            tc_mma_ts(tmem + C::O_COL + x * D, tmem + x * 128 + kk * 8, vd + ((kk * 16 * 128) >> 4),
                      idesc_o, (t > 0 || kk > 0) ? 1 : 0);
          }
          if (h == 1) tc_commit(&bars->pv_done[x]);
        };
        // Issue order per tile t: P_A V (in two halves, each as soon as the
        // softmax publishes it), S_A(t+1), P_B V (two halves), S_B(t+1). The
        // tensor core executes one thread's MMAs in issue order, so S_X(t+1)
        // overwrites P_X(t) only after P_X(t) V has read it, and the softmax
        // of tile A moves on as soon as its own product is done instead of
        // waiting for tile B's softmax. The commit after S_X(t+1) also covers
        // P_X(t) V, so O_X is final when the softmax sees S_X(t+1). K and V
        // have their own barriers: K(t) is released once both S(t) are done,
        // so its buffer refills while V(t) is still in use.
        //
        // The 2-byte and FP8 paths are written out separately: the issuing
        // thread is the bottleneck, and a single loop with shared wait /
        // release helpers measured 14% slower on the 70B prefill (1185
        // against 1378 TFLOP/s).
        constexpr int S_ = C::STAGES;
        ok = mbar_wait(&bars->q_full, 0) && mbar_wait(&bars->kv_full[0], 0);
        if (ok) {
          bars->consumed[0] = 1;
          issue_s(0, 0);
          if (two) issue_s(1, 0);
          tc_commit(&bars->kv_empty[0]);
        }
        for (int t = 0; ok && t < ntiles; ++t) {
          if (bars->abort) { ok = false; break; }
          const bool more = t + 1 < ntiles;
          if (!(ok = mbar_wait(&bars->p_full[0][0], t & 1))) break;
          if (!(ok = mbar_wait(&bars->kv_full[S_ + t % S_], (t / S_) & 1))) break;
          bars->consumed[1] = t + 1;
          issue_pv(0, t, 0);
          if (!(ok = mbar_wait(&bars->p_full[1][0], t & 1))) break;
          issue_pv(0, t, 1);
          if (more) {
            if (!(ok = mbar_wait(&bars->kv_full[(t + 1) % S_], ((t + 1) / S_) & 1))) break;
            bars->consumed[0] = t + 2;
            issue_s(0, t + 1);
          }
          if (two) {
            if (!(ok = mbar_wait(&bars->p_full[0][1], t & 1))) break;
            issue_pv(1, t, 0);
            if (!(ok = mbar_wait(&bars->p_full[1][1], t & 1))) break;
            issue_pv(1, t, 1);
          }
          tc_commit(&bars->kv_empty[S_ + t % S_]);
          if (more) {
            if (two) issue_s(1, t + 1);
            tc_commit(&bars->kv_empty[(t + 1) % S_]);
          }
        }
      } else {
        // FP8 pools: S_X(t) = Qh_X K(t)^T + Ql_X K(t)^T on kind::f8f6f4, K
        // straight from the e4m3 ring stage (128-byte swizzled rows, 32 bytes
        // of K per MMA); Qh_X and Ql_X are the two halves of Q tile X after
        // the converter warps' split. P V on kind::f16 from the widened V
        // buffers. The ring's K stage is released by the commit after both
        // tiles' S products; V stages by the converter warps.
        constexpr uint32_t idesc_s8 = mma_idesc(C::BM, C::BN, false, 0);   // e4m3 x e4m3
        constexpr uint32_t idesc_o = mma_idesc(C::BM, D, true, Elem<true>::kTcFormat);
        constexpr int VB = TcFp8::VBUF, S8 = TcFp8::STAGES8;
        const uint64_t qhdesc[2] = {smem_desc_sw128(smem_u32(smem + C::OFF_Q), 16, 1024),
                                    smem_desc_sw128(smem_u32(smem + C::OFF_Q + C::Q_TILE), 16, 1024)};
        const uint64_t k8desc0 = smem_desc_sw128(smem_u32(smem + TcFp8::OFF_R8), 16, 1024);
        const uint64_t vdesc0 = smem_desc_sw128(smem_u32(smem + TcFp8::OFF_VW), C::KV_HALF, 1024);
        auto issue_s = [&](int x, int t) {
          tc_fence_after();
          const uint64_t qh = qhdesc[x], ql = qhdesc[x] + (C::Q_HALF >> 4);
          const uint64_t kd = k8desc0 + static_cast<uint32_t>((t % S8) * (TcFp8::STAGE8 >> 4));
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc_mma_f8(tmem + x * 128, qh + kk * 2, kd + kk * 2, idesc_s8, kk > 0);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc_mma_f8(tmem + x * 128, ql + kk * 2, kd + kk * 2, idesc_s8, 1);
          tc_commit(&bars->s_full[x]);
        };
        auto issue_pv = [&](int x, int t, int h) {
          tc_fence_after();
          const uint64_t vd = vdesc0 + static_cast<uint32_t>((t % VB) * (C::KV_TILE >> 4));
#pragma unroll
          for (int k4 = 0; k4 < C::BN / 32; ++k4) {
            const int kk = h * (C::BN / 32) + k4;
            tc_mma_ts(tmem + C::O_COL + x * D, tmem + x * 128 + kk * 8,
                      vd + ((kk * 16 * 128) >> 4), idesc_o, (t > 0 || kk > 0) ? 1 : 0);
          }
          if (h == 1) tc_commit(&bars->pv_done[x]);
        };
        ok = mbar_wait(&bars->q_conv, 0) && mbar_wait(&bars->kv_full[0], 0);
        if (ok) {
          bars->consumed[0] = 1;
          issue_s(0, 0);
          if (two) issue_s(1, 0);
          tc_commit(&bars->kv_empty[0]);
        }
        for (int t = 0; ok && t < ntiles; ++t) {
          if (bars->abort) { ok = false; break; }
          const bool more = t + 1 < ntiles;
          if (!(ok = mbar_wait(&bars->p_full[0][0], t & 1))) break;
          if (!(ok = mbar_wait(&bars->vw_full[t % VB], (t / VB) & 1))) break;
          issue_pv(0, t, 0);
          if (!(ok = mbar_wait(&bars->p_full[1][0], t & 1))) break;
          issue_pv(0, t, 1);
          if (more) {
            if (!(ok = mbar_wait(&bars->kv_full[(t + 1) % S8], ((t + 1) / S8) & 1))) break;
            bars->consumed[0] = t + 2;
            issue_s(0, t + 1);
          }
          if (two) {
            if (!(ok = mbar_wait(&bars->p_full[0][1], t & 1))) break;
            issue_pv(1, t, 0);
            if (!(ok = mbar_wait(&bars->p_full[1][1], t & 1))) break;
            issue_pv(1, t, 1);
          }
          tc_commit(&bars->vw_free[t % VB]);
          if (more) {
            if (two) issue_s(1, t + 1);
            tc_commit(&bars->kv_empty[(t + 1) % S8]);
          }
        }
      }
      if (!ok) {
        abort_call(a);
        bars->abort = 1;
      }
      // Drain: arrive once every MMA issued above has completed.
      tc_commit(&bars->drain);
      mbar_wait(&bars->drain, 0);
    }
  } else if (FP8 && ntiles > 0) {
    // ------------------------------------------------------------ converters
    // Warps 2 and 3 (FP8 pools): split the Q tiles into e4m3 terms once,
    // then per key tile t widen the e4m3 V(t) (rows past the sequence end as
    // zeros) into V buffer t % VBUF once the P V products of tile t - VBUF
    // have read it, and free the ring's V stage as soon as it is widened.
    const int ct = threadIdx.x - 64;   // 0 .. 63
    constexpr int S8 = TcFp8::STAGES8, VB = TcFp8::VBUF;
    bool ok = mbar_wait(&bars->q_full, 0);
    if (ok) {
      q_split_e4m3<F16>(smem + C::OFF_Q, reinterpret_cast<float*>(smem + TcFp8::OFF_RS),
                        two ? 2 : 1, ct);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(&bars->q_conv);
    }
    for (int t = 0; ok && t < ntiles; ++t) {
      if (bars->abort) { ok = false; break; }
      const uint8_t* v8 = smem + TcFp8::OFF_R8 + (t % S8) * TcFp8::STAGE8 + TcFp8::TILE8;
      if (!(ok = mbar_wait(&bars->kv_full[S8 + t % S8], (t / S8) & 1))) break;
      if (ct == 0) bars->consumed[1] = t + 1;
      if (t >= VB && !(ok = mbar_wait(&bars->vw_free[t % VB], ((t / VB) - 1) & 1))) break;
      const int key0 = kb + t * C::BN;
      widen_e4m3_tile<WIN>(v8, smem + TcFp8::OFF_VW + (t % VB) * C::KV_TILE, ct, len - key0,
                           a.first - key0, win_lo - key0);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(&bars->vw_full[t % VB]);
      mbar_arrive(&bars->kv_empty[S8 + t % S8]);
    }
    if (!ok) {
      abort_call(a);
      bars->abort = 1;
    }
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;" ::: "memory");
    // ------------------------------------------------------------ softmax
    const int X = (warp - 4) >> 2;   // warps 4-7: tile A, 8-11: tile B
    if (X == 0 || two)
      tc_softmax_tile<D, F16, FP8, WIN>(a, bars, smem, tmem, X, q_start, q_len, len, kb, ke, ntiles,
                                        row0, R, hk, nsplit, slot_base, rt, j, win_lo);
    if (nsplit > 1 && !a.partials_only) {
      // Both warpgroups (256 threads) take part, active tile or not.
      __threadfence();
      asm volatile("bar.sync 1, 256;" ::: "memory");
      const int grp = slot_base + rt * nsplit;
      int* counter = a.counters + static_cast<int64_t>(grp) * a.H_kv + hk;
      const int tid = threadIdx.x - 128;
      if (tid == 0) bars->last = (atomicAdd(counter, 1) == nsplit - 1) ? 1 : 0;
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (bars->last) {
        __threadfence();
        combine_splits<D, F16>(a, grp, nsplit, hk, R, row0, q_start, tid, 256);
        if (tid == 0) *counter = 0;
      }
    }
  }

  // ---------------------------------------------------------------- teardown
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && bars->abort) {
    // After an abort, wait (bounded) for the copies still in flight.
    if (ntiles > 0) mbar_wait(&bars->q_full, 0);
    for (int p = 0; p < 2; ++p)
      for (int t = bars->consumed[p]; t < bars->issued[p]; ++t) {
        constexpr int STG = FP8 ? TcFp8::STAGES8 : C::STAGES;   // ring stages
        if (!mbar_wait(&bars->kv_full[p * STG + t % STG], (t / STG) & 1)) break;
      }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

template <int D, bool F16, bool FP8, bool WIN>
static cudaError_t launch_tc_w(const CUtensorMap& tmK, const CUtensorMap& tmV,
                               const CUtensorMap& tmQ, const AttnArgs& a, int items_bound,
                               cudaStream_t st) {
  using C = TcCfg<D>;
  // The shared-memory opt-in is a per-device function attribute: set it on
  // the first launch on each device (before any stream capture), not again.
  // The flags are atomics, so first calls from several host threads are
  // race-free (two threads may both set the attribute, which is harmless).
  static std::atomic<bool> configured[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool known = dev >= 0 && dev < kMaxDevices;
  if (!known || !configured[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(attn_tc_kernel<D, F16, FP8, WIN>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             FP8 ? TcFp8::SMEM_BYTES : C::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    if (known) configured[dev].store(true, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  // One column of blocks past the last item: the last block, which waits for
  // the predecessor grid (see pdl_enter), then has no item to delay.
  cfg.gridDim = dim3(items_bound + 1, a.H_kv);
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = FP8 ? TcFp8::SMEM_BYTES : C::SMEM_BYTES;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, attn_tc_kernel<D, F16, FP8, WIN>, tmK, tmV, tmQ, a);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

template <int D, bool F16, bool FP8 = false>
static cudaError_t launch_tc_d(const CUtensorMap& tmK, const CUtensorMap& tmV,
                               const CUtensorMap& tmQ, const AttnArgs& a, int items_bound,
                               cudaStream_t st) {
  return a.window > 0 ? launch_tc_w<D, F16, FP8, true>(tmK, tmV, tmQ, a, items_bound, st)
                      : launch_tc_w<D, F16, FP8, false>(tmK, tmV, tmQ, a, items_bound, st);
}

cudaError_t launch_attn_tc(const CUtensorMap& tmK, const CUtensorMap& tmV, const CUtensorMap& tmQ,
                           const AttnArgs& a, int items_bound, cudaStream_t st) {
  if (items_bound <= 0) return cudaSuccess;
  if (a.kv_fp8) {   // head size 128 (checked on the host)
    if (a.f16) return launch_tc_d<128, true, true>(tmK, tmV, tmQ, a, items_bound, st);
    return launch_tc_d<128, false, true>(tmK, tmV, tmQ, a, items_bound, st);
  }
  if (a.f16) {
    if (a.D == 256) return launch_tc_d<256, true>(tmK, tmV, tmQ, a, items_bound, st);
    if (a.D == 128) return launch_tc_d<128, true>(tmK, tmV, tmQ, a, items_bound, st);
    return launch_tc_d<64, true>(tmK, tmV, tmQ, a, items_bound, st);
  }
  if (a.D == 256) return launch_tc_d<256, false>(tmK, tmV, tmQ, a, items_bound, st);
  if (a.D == 128) return launch_tc_d<128, false>(tmK, tmV, tmQ, a, items_bound, st);
  return launch_tc_d<64, false>(tmK, tmV, tmQ, a, items_bound, st);
}

}  // namespace pa
