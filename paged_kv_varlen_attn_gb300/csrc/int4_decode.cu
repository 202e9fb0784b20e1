// Attention over 4-bit pools for decode and short queries: sequences of at
// most 32 packed query rows (tokens x heads of the group).
#include <cuda_runtime.h>

#include "device_common.cuh"
#include "epilogue.cuh"

namespace pa {

// ---------------------------------------------------------------------------
// A 4-bit cache halves the bytes of an e4m3 one, so at the full read rate an SM
// has about 2.7 instructions for each element of K and V. What an element costs
// here is most of the design:
//   K  A word's four masks (w & 0x000F000F, w & 0x00F000F0, and the same of
//      w >> 8) are f16 pairs already: a code n in the low four bits of an f16 is
//      the subnormal n 2^-24, in the next four n 2^-20. Both are exact, and the
//      MMA takes subnormals; the query's operand carries the 16 between them. No
//      conversion: 5 instructions for 8 codes. The products are summed over
//      codes, S^T[16 keys x 8 rows] = N Q^T, and the row's scale and minimum
//      join after: q.k = scale (q.n) + minimum (sum of q).
//   V  The MMA wants pairs of keys, so two keys' words are put together by
//      halves (byte permutes) and masked the same way: 6 instructions for 8.
//      O^T[D x 8 rows] += N^T W^T with W = weight x V's scale / ref, ref a power
//      of two that is raised when a scale passes it (the weights stay below 2^8,
//      so W stays inside f16 and keeps its eleven bits down to 2^-22 of that).
//      The rest of the value enters by sums per row: of weights x (minimum + 8
//      scale), and of W as rounded, eightfold, which is taken off: so a weight's
//      rounding weighs with code - 8 and not with the code. That sum is one more
//      row of the product (ones for codes), and is taken off every 128 keys
//      already, before the sums of codes grow past what float32 keeps of the
//      difference (f16 outputs were off by 3.4e-4 of their size otherwise, by
//      6e-4 without the eightfold sum; the output's own rounding is 2.1e-4).
// The weights are 2^(score - m) against a running maximum m that is raised only
// when a score passes it by more than 8; their sum is float32.
//
// Nothing is planned on the device and nothing depends on the key bound: the
// slices (32 keys) of all sequences of the class, one after another, are cut
// into equal ranges, and warp (range, KV head) streams its range through a ring
// of its own, filled by asynchronous copies that run ahead across sequences.
// Every warp counts the ranges for itself from the lengths. A sequence's state
// that a range does not hold whole goes to the workspace (two slots per warp),
// and int4_combine_kernel merges those, in order: no atomics, the same bits on
// every run. The warps of neighbouring KV heads are neighbours, so a page's
// bytes are read at about the same time.
// ---------------------------------------------------------------------------
constexpr int kI4Warps = 4;        // of a block; they share nothing
constexpr int kI4Slots = 3;        // slices in a warp's ring
constexpr int kI4MinSlices = 2;    // of a range
constexpr int kI4Keys = 32;        // of a slice: two halves of 16, each in one page

template <int D, int NR>
struct I4Cfg {
  static constexpr int CODES = 16 * D / 2;             // bytes of a half's K or V
  static constexpr int PAR = 4 * CODES;                // K of both halves, V of both, params
  static constexpr int SLOT = PAR + 2 * kI4Keys * 4;
  static constexpr int SMEM_BYTES = kI4Warps * kI4Slots * SLOT;
  static constexpr int BLOCKS = NR == 1 ? 4 : 2;   // per SM
};

// One sequence, as the kernels of this file count it.
struct I4Seq {
  int q0, q_len, kv;
  int n;             // slices; 0: not of this class
};

__device__ __forceinline__ I4Seq i4_seq(const Int4DecodeArgs& a, int s, bool report) {
  I4Seq q;
  q.q0 = __ldg(a.cu + s);
  const int q1 = __ldg(a.cu + s + 1);
  q.kv = __ldg(a.seqused_k + s);
  q.q_len = q1 - q.q0;
  int bad = 0;
  if (q.q0 < 0 || q1 > a.total_q || q1 < q.q0 || q.q_len > a.max_q) {
    bad = PA_DEV_BAD_SEQLEN;
    q.q_len = 0;
  }
  if (q.kv < 0 || q.kv > a.max_k || q.kv > a.kv_len_cap) bad = PA_DEV_BAD_SEQLEN;
  if (bad && report) flag_status(a.status, bad);
  q.kv = min(max(q.kv, 0), a.kv_len_cap);
  const bool mine = q.q_len > a.tokens_min && q.q_len <= a.tokens_max;
  // A sequence without keys has one slice that nobody sees.
  q.n = mine ? max(1, (q.kv + kI4Keys - 1) / kI4Keys) : 0;
  return q;
}

// 1 / x of a power of two.
__device__ __forceinline__ float inverse_power(float x) {
  return __uint_as_float((254u << 23) - __float_as_uint(x));
}

// Slices of a range, given all of them.
__device__ __forceinline__ long long i4_per_range(const Int4DecodeArgs& a, long long total) {
  const long long per = (total + a.ranges - 1) / a.ranges;
  return per < kI4MinSlices ? kI4MinSlices : per;
}

template <int D, bool F16, int NR>
__global__ void __launch_bounds__(kI4Warps * 32, I4Cfg<D, NR>::BLOCKS)
int4_decode_kernel(const __grid_constant__ Int4DecodeArgs a) {
  using C = I4Cfg<D, NR>;
  using E = Elem<F16>;
  constexpr int KW = D / 32;       // words of a key per lane in S^T
  constexpr int VW = D / 64;       // words of a key per lane in O^T
  constexpr unsigned kAll = 0xffffffffu;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  pdl_trigger();                   // the combine kernel may be placed when these blocks have been
  const int wid = static_cast<int>(blockIdx.x) * kI4Warps + warp;
  const int range = wid / a.H_kv, hk = wid - range * a.H_kv;
  if (range >= a.ranges) return;

  // All slices, then this warp's range and the sequence in which it starts.
  long long total = 0;
  for (int s = lane; s < a.num_seqs; s += 32) total += i4_seq(a, s, wid == 0).n;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kAll, total, o);
  const long long per = i4_per_range(a, total);
  const long long begin = range * per;
  if (begin >= total) return;
  const int count = static_cast<int>(min(per, total - begin));
  int base = 0;                    // lane i holds sequence base + i
  long long before = 0;            // slices of the sequences in front of base
  I4Seq sq;
  int first = 0;                   // lane of the first sequence
  for (;; base += 32) {
    if (base >= a.num_seqs) return;                    // (lengths changed under the call)
    sq = I4Seq{0, 0, 0, 0};
    if (base + lane < a.num_seqs) sq = i4_seq(a, base + lane, false);
    long long incl = sq.n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(kAll, incl, o);
      if (lane >= o) incl += x;
    }
    const unsigned past = __ballot_sync(kAll, before + incl > begin);
    if (past) {
      first = __ffs(past) - 1;
      before += __shfl_sync(kAll, incl - sq.n, first);
      break;
    }
    before += __shfl_sync(kAll, incl, 31);
  }
  int i = static_cast<int>(begin - before);            // slice of the sequence

  // ---------------------------------------------------------------- copies
  // The next slice to copy: slice f_i of f_n of the sequence in lane f_at of the
  // 32 whose lengths the lanes hold from f_base on. Lane x holds the page and the
  // row of half f_half0 + x of that sequence.
  int f_base = base, f_at = first, f_kv_l = sq.kv, f_n_l = sq.n;
  int f_i = i, f_n = __shfl_sync(kAll, f_n_l, f_at), f_kv = __shfl_sync(kAll, f_kv_l, f_at);
  int f_half0 = 0, f_left = count;
  int page_l = -1, row_l = 0;
  auto load_pages = [&]() {
    f_half0 = 2 * f_i;
    const int key0 = (f_half0 + lane) * 16;
    page_l = -1;
    row_l = 0;
    if (key0 < f_kv) {
      const int lp = a.bs_shift >= 0 ? key0 >> a.bs_shift : key0 / a.bs;
      row_l = key0 - lp * a.bs;
      page_l = __ldg(a.bt + static_cast<int64_t>(f_base + f_at) * a.bt_stride + lp);
      if (page_l < 0 || page_l >= a.num_blocks) {
        page_l = -1;                                   // reads as zeros
        flag_status(a.status, PA_DEV_BAD_PAGE);
      }
    }
  };
  load_pages();
  uint8_t* ring = smem + warp * (kI4Slots * C::SLOT);
  const uint32_t ring_at = smem_u32(ring);
  const int rstep = a.H_kv * (D / 2);                  // (checked to fit by the host)
  // Row g of S^T is key (g >> 1) + 4 (g & 1) of the half's halves: so the four
  // keys of a lane in O^T, 2c and 2c + 1 of each, are rows c and c + 4 of shared
  // memory, and eight lanes that read them take different banks.
  const int kg = (g >> 1) + 4 * (g & 1);
  // What this lane copies of a half. D = 128: of K its own pieces (rows kg and kg
  // + 8), of V piece c of rows g and g + 8 to place c ^ (g & 2); D = 64: piece
  // lane & 1 of row lane / 2 of both. And one row's scale and minimum, of K in
  // lanes 0-15, of V in the others: those of keys x, x + 8, x + 16, x + 24 of the
  // slice side by side.
  const int k_row = D == 128 ? kg : lane >> 1, v_row = D == 128 ? g : lane >> 1;
  const int piece = D == 128 ? c : lane & 1;
  const uint8_t* k_src = a.kc + hk * (D / 2) + static_cast<int64_t>(k_row) * rstep + piece * 16;
  const uint8_t* v_src = a.vc + hk * (D / 2) + static_cast<int64_t>(v_row) * rstep + piece * 16;
  const int p_row = lane & 15;
  const uint32_t* p_src = (lane < 16 ? a.k_params : a.v_params) +
                          static_cast<int64_t>(hk) * a.bs + p_row;
  const uint32_t v_place = D == 128 ? g * 64 + ((c ^ (g & 2)) << 4) : lane * 16;
  const uint32_t p_place = C::PAR + (lane >> 4) * (kI4Keys * 4) + (p_row & 7) * 16 + (p_row >> 3) * 4;
  auto fetch = [&](int slot) {
    if (f_left > 0) {
      if (f_i == f_n) {                                // the next sequence that has slices
        for (;;) {
          const unsigned later = __ballot_sync(kAll, f_n_l > 0) & ~((2u << f_at) - 1u);
          if (later) {
            f_at = __ffs(later) - 1;
            break;
          }
          f_base += 32;
          if (f_base >= a.num_seqs) {                  // (lengths changed under the call)
            f_left = 0;
            break;
          }
          f_n_l = 0;
          if (f_base + lane < a.num_seqs) {
            const I4Seq x = i4_seq(a, f_base + lane, false);
            f_n_l = x.n;
            f_kv_l = x.kv;
          }
          const unsigned any = __ballot_sync(kAll, f_n_l > 0);
          if (any) {
            f_at = __ffs(any) - 1;
            break;
          }
          f_at = 31;
        }
        if (f_left == 0) {
          cp_async_commit();
          return;
        }
        f_n = __shfl_sync(kAll, f_n_l, f_at);
        f_kv = __shfl_sync(kAll, f_kv_l, f_at);
        f_i = 0;
        load_pages();
      } else if (2 * f_i - f_half0 == 32) {
        load_pages();
      }
      const uint32_t dst0 = ring_at + slot * C::SLOT;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int page = __shfl_sync(kAll, page_l, 2 * f_i - f_half0 + h);
        const uint32_t prow = __shfl_sync(kAll, row_l, 2 * f_i - f_half0 + h);
        const uint32_t dst = dst0 + h * C::CODES;
        if (page >= 0) {
          const uint64_t at = static_cast<uint64_t>(static_cast<uint32_t>(page)) * a.page_bytes +
                              static_cast<uint64_t>(prow) * static_cast<uint32_t>(rstep);
          const uint8_t* kp = k_src + at;
          const uint8_t* vp = v_src + at;
          cp_async16(dst + lane * 16, kp);
          cp_async16(dst + 2 * C::CODES + v_place, vp);
          if constexpr (D == 128) {
            cp_async16(dst + 512 + lane * 16, kp + 8 * rstep);
            cp_async16(dst + 2 * C::CODES + 512 + v_place, vp + 8 * rstep);
          }
          // Scales and minima; zeros past the sequence (what is there is nobody's).
          cp_async4(dst0 + p_place + h * 8,
                    p_src + static_cast<uint64_t>(static_cast<uint32_t>(page)) * a.page_params + prow,
                    32 * f_i + 16 * h + p_row < f_kv);
        } else {
          // No page: codes do not matter where scale and minimum are zero, but
          // they must be some.
          cp_async4(dst0 + p_place + h * 8, p_src, false);
        }
      }
      ++f_i;
      --f_left;
    }
    cp_async_commit();
  };
#pragma unroll
  for (int u = 0; u < kI4Slots - 1; ++u) fetch(u);

  // ---------------------------------------------------------------- sequences
  int at = first, left = count;
  int slot = 0, to = kI4Slots - 1;
  long long flat = begin;          // slice of all slices at which this part starts
#pragma unroll 1
  while (left > 0) {
    while (base < a.num_seqs && __shfl_sync(kAll, sq.n, at) == 0) {   // the next sequence
      if (++at == 32) {
        base += 32;
        sq = I4Seq{0, 0, 0, 0};
        if (base + lane < a.num_seqs) sq = i4_seq(a, base + lane, false);
        at = 0;
      }
    }
    if (base >= a.num_seqs) break;                     // (lengths changed under the call)
    const int n = __shfl_sync(kAll, sq.n, at), kv = __shfl_sync(kAll, sq.kv, at);
    const int q0 = __shfl_sync(kAll, sq.q0, at), q_len = __shfl_sync(kAll, sq.q_len, at);
    const int i0 = i, i1 = min(n, i + left);
    const int rows = q_len * a.G, past = kv - q_len;
    // Keys that every row sees.
    const int seen_by_all = min(kv, a.causal ? past + 1 : kv);

    // Q as B fragments, f16 after a power-of-two scale that brings the row's
    // largest element to 2^14 .. 2^15 (infinities and NaN stay what they are);
    // the operand of the codes in the upper four bits is a sixteenth.
    uint32_t qf[NR][2 * KW][2];
    float sa[NR][2], sb[NR][2];    // of rows 2c, 2c + 1: scale of q.n, and of sum(q)
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) {
      const int r = min(8 * nr + g, rows - 1), t = r / a.G;
      const uint4* qrow = reinterpret_cast<const uint4*>(
          a.q + static_cast<int64_t>(q0 + t) * a.q_stride +
          static_cast<int64_t>(hk * a.G + r - t * a.G) * D + c * (8 * KW));
      float q[KW][8], top = 0.f, sum = 0.f;
#pragma unroll
      for (int v = 0; v < KW; ++v) {
        const uint4 x = __ldg(qrow + v);
        const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 f = E::unpack(xw[k]);
          q[v][2 * k] = f.x;
          q[v][2 * k + 1] = f.y;
          top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
      }
      top = fmaxf(top, __shfl_xor_sync(kAll, top, 1));
      top = fmaxf(top, __shfl_xor_sync(kAll, top, 2));
      const int ex = static_cast<int>(__float_as_uint(top) >> 23);
      const int up = ex == 255 ? 0 : min(126, 141 - ex);
      const float by = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
      const float down = __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
#pragma unroll
      for (int v = 0; v < KW; ++v) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float y0 = q[v][4 * k] * by, y1 = q[v][4 * k + 1] * by;
          const float y2 = q[v][4 * k + 2] * by, y3 = q[v][4 * k + 3] * by;
          sum += (y0 + y1) + (y2 + y3);
          qf[nr][2 * v + k][0] = pack_f16(y0, y1);
          qf[nr][2 * v + k][1] = pack_f16(y2 * 0.0625f, y3 * 0.0625f);
        }
      }
      sum += __shfl_xor_sync(kAll, sum, 1);
      sum += __shfl_xor_sync(kAll, sum, 2);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int from = (2 * c + e) * 4;
        sa[nr][e] = a.scale_log2 * __shfl_sync(kAll, down, from);
        sb[nr][e] = a.scale_log2 * (__shfl_sync(kAll, sum, from) * __shfl_sync(kAll, down, from));
      }
    }
    float m[NR][2], l[NR][2], lv[NR][2];               // lv: sum of weights x middle of V's row
    float acc[NR][D / 16][4], accw[NR][4];             // accw: sum of W, every entry of a column
    float ref = 0.f;                                   // power of two, at least V's scales so far
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[nr][e] = -INFINITY;
        l[nr][e] = lv[nr][e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) accw[nr][e] = 0.f;
#pragma unroll
      for (int t = 0; t < D / 16; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[nr][t][e] = 0.f;
    }
    // Takes the eightfold sum of W off the sums of codes.
    auto centre = [&]() {
#pragma unroll
      for (int nr = 0; nr < NR; ++nr) {
#pragma unroll
        for (int t = 0; t < D / 16; ++t) {
          ffma2(acc[nr][t][0], acc[nr][t][1], accw[nr][0], accw[nr][1], -0x1p-21f, -0x1p-21f,
                acc[nr][t][0], acc[nr][t][1]);
          ffma2(acc[nr][t][2], acc[nr][t][3], accw[nr][0], accw[nr][1], -0x1p-17f, -0x1p-17f,
                acc[nr][t][2], acc[nr][t][3]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) accw[nr][e] = 0.f;
      }
    };

#pragma unroll 1
    for (; i < i1; ++i) {
      fetch(to);
      if (++to == kI4Slots) to = 0;
      cp_async_wait<kI4Slots - 1>();
      __syncwarp();
      const uint8_t* sl = ring + slot * C::SLOT;
      const int key0 = kI4Keys * i;
      // ----------------------------------------------------------- S^T = N Q^T
      float st[NR][2][4];
#pragma unroll
      for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int h = 0; h < 2; ++h) st[nr][h][0] = st[nr][h][1] = st[nr][h][2] = st[nr][h][3] = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t w0[KW], w1[KW];
        if constexpr (D == 128) {
          const uint4 x0 = *reinterpret_cast<const uint4*>(sl + h * C::CODES + lane * 16);
          const uint4 x1 = *reinterpret_cast<const uint4*>(sl + h * C::CODES + 512 + lane * 16);
          w0[0] = x0.x; w0[1] = x0.y; w0[2] = x0.z; w0[3] = x0.w;
          w1[0] = x1.x; w1[1] = x1.y; w1[2] = x1.z; w1[3] = x1.w;
        } else {
          const uint2 x0 = *reinterpret_cast<const uint2*>(sl + h * C::CODES + kg * 32 + c * 8);
          const uint2 x1 = *reinterpret_cast<const uint2*>(sl + h * C::CODES + (8 + kg) * 32 + c * 8);
          w0[0] = x0.x; w0[1] = x0.y;
          w1[0] = x1.x; w1[1] = x1.y;
        }
#pragma unroll
        for (int v = 0; v < KW; ++v) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t a0 = w0[v] >> (8 * k), a1 = w1[v] >> (8 * k);
#pragma unroll
            for (int nr = 0; nr < NR; ++nr)
              mma_16816_f16(st[nr][h], a0 & 0x000F000Fu, a1 & 0x000F000Fu, a0 & 0x00F000F0u,
                            a1 & 0x00F000F0u, qf[nr][2 * v + k][0], qf[nr][2 * v + k][1]);
          }
        }
      }
      // ----------------------------------------------------------- softmax
      // Keys kg + 8 h of the slice, h = 0 .. 3: entries 2 (h & 1) of st[h >> 1].
      const uint4 pk = *reinterpret_cast<const uint4*>(sl + C::PAR + kg * 16);
      const uint4 pv = *reinterpret_cast<const uint4*>(sl + C::PAR + kI4Keys * 4 + kg * 16);
      const uint32_t pkw[4] = {pk.x, pk.y, pk.z, pk.w}, pvw[4] = {pv.x, pv.y, pv.z, pv.w};
      float ks[4], km[4], vs[4], vm[4];
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const float2 k = Elem<true>::unpack(pkw[h]), v = Elem<true>::unpack(pvw[h]);
        ks[h] = k.x * 0x1p24f;
        km[h] = k.y;
        vs[h] = v.x;
        vm[h] = fmaf(8.f, v.x, v.y);
      }
      const bool whole = key0 + kI4Keys <= seen_by_all;
      const float vtop = fmaxf(fmax3(vs[0], vs[1], vs[2]), vs[3]);
      if (__any_sync(kAll, vtop > ref)) {              // raise the reference of V's scales
        float top = vtop;
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
        // The power of two above it, and 4: a larger one is then seldom met.
        const float nr_ref = __uint_as_float(((__float_as_uint(top) >> 23) + 3u) << 23);
        const float f = ref == 0.f ? 0.f : ref * inverse_power(nr_ref);
        ref = nr_ref;
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
#pragma unroll
          for (int e = 0; e < 4; ++e) accw[nr][e] *= f;
#pragma unroll
          for (int t = 0; t < D / 16; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[nr][t][e] *= f;
        }
      }
      // W = weight x scale / ref x 2^6: at most 2^8 x 1 x 2^6 = 2^14.
      const float wscale = ref == 0.f ? 0.f : 64.f * inverse_power(ref);
      uint32_t wb[NR][4];
#pragma unroll
      for (int nr = 0; nr < NR; ++nr) {
        float x[4][2];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          float t0, t1, u0, u1;
          fmul2(t0, t1, ks[h], ks[h], sa[nr][0], sa[nr][1]);
          fmul2(u0, u1, km[h], km[h], sb[nr][0], sb[nr][1]);
          ffma2(x[h][0], x[h][1], st[nr][h >> 1][2 * (h & 1)], st[nr][h >> 1][2 * (h & 1) + 1], t0,
                t1, u0, u1);
        }
        if (!whole) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int row = min(8 * nr + 2 * c + e, rows - 1);
            const int lim = a.causal ? past + row / a.G : kv - 1;   // last visible key
#pragma unroll
            for (int h = 0; h < 4; ++h)
              if (key0 + kg + 8 * h > lim) x[h][e] = -INFINITY;
          }
        }
        const float x0 = fmaxf(fmax3(x[0][0], x[1][0], x[2][0]), x[3][0]);
        const float x1 = fmaxf(fmax3(x[0][1], x[1][1], x[2][1]), x[3][1]);
        if (__any_sync(kAll, x0 > m[nr][0] + 8.f || x1 > m[nr][1] + 8.f)) {
          float xm[2] = {x0, x1};
#pragma unroll
          for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) xm[e] = fmaxf(xm[e], __shfl_xor_sync(kAll, xm[e], o));
            const float nm = fmaxf(m[nr][e], xm[e]);
            const float f = m[nr][e] == -INFINITY ? 0.f : fast_exp2(m[nr][e] - nm);
            l[nr][e] *= f;
            lv[nr][e] *= f;
            m[nr][e] = nm;
            accw[nr][e] *= f;
            accw[nr][2 + e] *= f;
#pragma unroll
            for (int t = 0; t < D / 16; ++t) {
              acc[nr][t][e] *= f;
              acc[nr][t][2 + e] *= f;
            }
          }
        }
        const float m0 = m[nr][0] == -INFINITY ? 0.f : m[nr][0];
        const float m1 = m[nr][1] == -INFINITY ? 0.f : m[nr][1];
        float w[4][2];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          float y0, y1;
          fadd2(y0, y1, x[h][0], x[h][1], -m0, -m1);
          const float p0 = fast_exp2(y0), p1 = fast_exp2(y1);
          fadd2(l[nr][0], l[nr][1], l[nr][0], l[nr][1], p0, p1);
          const float f = vs[h] * wscale;
          if (whole) {
            ffma2(lv[nr][0], lv[nr][1], p0, p1, vm[h], vm[h], lv[nr][0], lv[nr][1]);
            fmul2(w[h][0], w[h][1], p0, p1, f, f);
          } else {   // a key that a row does not see adds nothing, whatever it holds
            const bool s0 = x[h][0] != -INFINITY, s1 = x[h][1] != -INFINITY;
            lv[nr][0] = s0 ? fmaf(p0, vm[h], lv[nr][0]) : lv[nr][0];
            lv[nr][1] = s1 ? fmaf(p1, vm[h], lv[nr][1]) : lv[nr][1];
            w[h][0] = s0 ? p0 * f : 0.f;
            w[h][1] = s1 ? p1 * f : 0.f;
          }
        }
#pragma unroll
        for (int h = 0; h < 4; ++h) wb[nr][h] = movmatrix_trans(pack_f16(w[h][0], w[h][1]));
      }
      // ----------------------------------------------------------- O^T += N^T W^T
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t wv[4][VW];        // keys c, c + 4, c + 8, c + 12 of the half; 8 VW dims
        const uint8_t* vt = sl + (2 + h) * C::CODES;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int r = c + 4 * k;
          if constexpr (D == 128) {
            const uint2 x = *reinterpret_cast<const uint2*>(
                vt + r * 64 + (((g >> 1) ^ (r & 2)) << 4) + (g & 1) * 8);
            wv[k][0] = x.x;
            wv[k][1] = x.y;
          } else {
            wv[k][0] = *reinterpret_cast<const uint32_t*>(vt + r * 32 + g * 4);
          }
        }
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
          mma_16816_f16(accw[nr], 0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u,
                        wb[nr][2 * h], wb[nr][2 * h + 1]);
#pragma unroll
        for (int j = 0; j < VW; ++j) {
#pragma unroll
          for (int odd = 0; odd < 2; ++odd) {
            const uint32_t t0 = prmt(wv[0][j], wv[1][j], odd ? 0x7632 : 0x5410);
            const uint32_t t1 = prmt(wv[2][j], wv[3][j], odd ? 0x7632 : 0x5410);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t u0 = t0 >> (8 * k), u1 = t1 >> (8 * k);
#pragma unroll
              for (int nr = 0; nr < NR; ++nr)
                mma_16816_f16(acc[nr][4 * j + 2 * odd + k], u0 & 0x000F000Fu, u0 & 0x00F000F0u,
                              u1 & 0x000F000Fu, u1 & 0x00F000F0u, wb[nr][2 * h], wb[nr][2 * h + 1]);
            }
          }
        }
      }
      if ((i & 3) == 3) centre();
      if (++slot == kI4Slots) slot = 0;
      __syncwarp();                                    // the slot may be filled again
    }
    centre();

    // ---------------------------------------------------------------- the state
    // acc[4 j + 2 odd + k] holds, of this lane's 8 j .. 8 j + 7 dims, 4 k + odd
    // (entries 0, 1: rows 2c, 2c + 1) and 4 k + 2 + odd (2, 3; sixteenfold).
    const bool all = i0 == 0 && i1 == n;
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float L = l[nr][e], V = lv[nr][e];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          L += __shfl_xor_sync(kAll, L, o);
          V += __shfl_xor_sync(kAll, V, o);
        }
        const int row = 8 * nr + 2 * c + e;
        if (row >= rows) continue;
        const int t = row / a.G, head = hk * a.G + row - t * a.G;
        float M = m[nr][e], of = 1.f;
        const float fw = ref * (0x1p24f / 64.f);       // of the sums of codes
        if (all && a.sinks) of = add_sink(M, L, __ldg(a.sinks + head) * kLog2e);
        const float inv = L == 0.f ? 0.f : of / L;
        const float lse = L == 0.f ? -INFINITY : (M + fast_log2(L)) * kLn2;
        float o[VW][8];
#pragma unroll
        for (int j = 0; j < VW; ++j)
#pragma unroll
          for (int x = 0; x < 4; ++x) {                // x = 2 odd + k
            const int d = 4 * (x & 1) + (x >> 1);
            o[j][d] = fmaf(acc[nr][4 * j + x][e], fw, V) * inv;
            o[j][d + 2] = fmaf(acc[nr][4 * j + x][2 + e], fw * 0.0625f, V) * inv;
          }
        if (all) {
          uint4* dst = reinterpret_cast<uint4*>(
              a.out + (static_cast<int64_t>(q0 + t) * a.H + head) * D + g * (8 * VW));
#pragma unroll
          for (int j = 0; j < VW; ++j)
            dst[j] = make_uint4(E::pack(o[j][0], o[j][1]), E::pack(o[j][2], o[j][3]),
                                E::pack(o[j][4], o[j][5]), E::pack(o[j][6], o[j][7]));
          if (a.lse && g == 0) a.lse[static_cast<int64_t>(head) * a.total_q + q0 + t] = lse;
        } else {
          const int64_t at_row =
              (static_cast<int64_t>(wid) * 2 + (flat == begin ? 0 : 1)) * (8 * NR) + row;
          float4* dst = reinterpret_cast<float4*>(a.part_o + at_row * D + g * (8 * VW));
#pragma unroll
          for (int j = 0; j < VW; ++j) {
            __stcg(dst + 2 * j, make_float4(o[j][0], o[j][1], o[j][2], o[j][3]));
            __stcg(dst + 2 * j + 1, make_float4(o[j][4], o[j][5], o[j][6], o[j][7]));
          }
          if (g == 0) __stcg(a.part_lse + at_row, lse);
        }
      }
    }
    left -= i1 - i0;
    flat += i1 - i0;
    i = 0;
    ++at;
    if (at == 32 && left > 0) {
      base += 32;
      sq = I4Seq{0, 0, 0, 0};
      if (base + lane < a.num_seqs) sq = i4_seq(a, base + lane, false);
      at = 0;
    }
  }
  cp_async_wait<0>();
}

// ---------------------------------------------------------------------------
// The sequences whose slices lie in more than one range: their states, in the
// ranges' order. A block per (sequence, KV head).
// ---------------------------------------------------------------------------
constexpr int kI4CombineThreads = 128;

template <int D, bool F16, int NR>
__global__ void __launch_bounds__(kI4CombineThreads)
int4_combine_kernel(const __grid_constant__ Int4DecodeArgs a) {
  __shared__ long long sums[2][kI4CombineThreads / 32];
  const int s = static_cast<int>(blockIdx.x) / a.H_kv;
  const int hk = static_cast<int>(blockIdx.x) - s * a.H_kv;
  const I4Seq sq = i4_seq(a, s, false);
  if (sq.n == 0) {
    pdl_leave();                                       // (the grid ends after its predecessor)
    return;
  }
  long long total = 0, before = 0;
  for (int x = threadIdx.x; x < a.num_seqs; x += kI4CombineThreads) {
    const int n = i4_seq(a, x, false).n;
    total += n;
    if (x < s) before += n;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    total += __shfl_xor_sync(0xffffffffu, total, o);
    before += __shfl_xor_sync(0xffffffffu, before, o);
  }
  if ((threadIdx.x & 31) == 0) {
    sums[0][threadIdx.x >> 5] = total;
    sums[1][threadIdx.x >> 5] = before;
  }
  __syncthreads();
  total = before = 0;
#pragma unroll
  for (int w = 0; w < kI4CombineThreads / 32; ++w) {
    total += sums[0][w];
    before += sums[1][w];
  }
  const long long per = i4_per_range(a, total);
  const int r0 = static_cast<int>(before / per);
  const int r1 = static_cast<int>((before + sq.n - 1) / per);
  if (r0 == r1) {                                      // written by its warp
    pdl_leave();
    return;
  }
  pdl_wait();
  const int rows = sq.q_len * a.G;
  const int64_t step = static_cast<int64_t>(a.H_kv) * 2 * (8 * NR);
  // The first part starts inside its range (slot 1) unless at its border.
  const int64_t at0 = (static_cast<int64_t>(r0) * a.H_kv + hk) * 2 * (8 * NR);
  const int64_t first = at0 + (before == r0 * per ? 0 : 8 * NR);
  for (int u = threadIdx.x; u < rows * (D / 4); u += kI4CombineThreads) {
    const int row = u / (D / 4), col = u % (D / 4) * 4;
    float mx = -INFINITY, sw = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    merge_states(mx, sw, o, a.part_lse, a.part_o, first + row, 0, 1, D, col);
    merge_states(mx, sw, o, a.part_lse, a.part_o, at0 + step + row, step, r1 - r0, D, col);
    const int t = row / a.G, head = hk * a.G + row - t * a.G;
    if (a.sinks) {
      const float ls[kBatch] = {__ldg(a.sinks + head)};
      const float4 z[kBatch] = {make_float4(0.f, 0.f, 0.f, 0.f)};
      merge_batch(mx, sw, o, ls, z, 1);
    }
    const float inv = sw == 0.f ? 0.f : 1.f / sw;
    *reinterpret_cast<uint2*>(a.out + (static_cast<int64_t>(sq.q0 + t) * a.H + head) * D + col) =
        make_uint2(Elem<F16>::pack(o[0] * inv, o[1] * inv),
                   Elem<F16>::pack(o[2] * inv, o[3] * inv));
    if (a.lse && col == 0)
      a.lse[static_cast<int64_t>(head) * a.total_q + sq.q0 + t] =
          sw == 0.f ? -INFINITY : mx + fast_log2(sw) * kLn2;
  }
}

template <int D, bool F16, int NR>
static cudaError_t launch_int4_decode_nr(const Int4DecodeArgs& a, cudaStream_t st) {
  using C = I4Cfg<D, NR>;
  static std::atomic<bool> configured[kMaxDevices];
  cudaError_t e = opt_in_smem(int4_decode_kernel<D, F16, NR>, C::SMEM_BYTES, configured);
  if (e != cudaSuccess) return e;
  const long long warps = static_cast<long long>(a.ranges) * a.H_kv;
  int4_decode_kernel<D, F16, NR>
      <<<static_cast<unsigned>((warps + kI4Warps - 1) / kI4Warps), kI4Warps * 32, C::SMEM_BYTES,
         st>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.num_seqs) * static_cast<unsigned>(a.H_kv));
  cfg.blockDim = dim3(kI4CombineThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, int4_combine_kernel<D, F16, NR>, a);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

int int4_decode_ranges(int sms, int H_kv, int nr) {
  const int blocks = nr == 1   ? I4Cfg<128, 1>::BLOCKS
                     : nr == 2 ? I4Cfg<128, 2>::BLOCKS
                     : nr == 3 ? I4Cfg<128, 3>::BLOCKS
                               : I4Cfg<128, 4>::BLOCKS;
  const int n = sms * blocks * kI4Warps / H_kv;
  return n < 1 ? 1 : n;
}

size_t int4_decode_part_rows(int sms, int H_kv, int nr) {
  return static_cast<size_t>(int4_decode_ranges(sms, H_kv, nr)) * H_kv * 2 * 8 * nr;
}

cudaError_t launch_int4_decode(Int4DecodeArgs a, int D, bool f16, int nr, int sms,
                               cudaStream_t st) {
  a.ranges = int4_decode_ranges(sms, a.H_kv, nr);
  auto by_rows = [&](auto d, auto half) {
    constexpr int kD = decltype(d)::value;
    constexpr bool kF16 = decltype(half)::value;
    if (nr == 1) return launch_int4_decode_nr<kD, kF16, 1>(a, st);
    if (nr == 2) return launch_int4_decode_nr<kD, kF16, 2>(a, st);
    if (nr == 3) return launch_int4_decode_nr<kD, kF16, 3>(a, st);
    return launch_int4_decode_nr<kD, kF16, 4>(a, st);
  };
  using std::integral_constant;
  if (D == 128)
    return f16 ? by_rows(integral_constant<int, 128>{}, std::true_type{})
               : by_rows(integral_constant<int, 128>{}, std::false_type{});
  return f16 ? by_rows(integral_constant<int, 64>{}, std::true_type{})
             : by_rows(integral_constant<int, 64>{}, std::false_type{});
}

}  // namespace pa
