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
//      of two that is raised when a scale's magnitude passes it (the weights stay
//      below 2^8, so W stays inside f16 and keeps its eleven bits down to 2^-22 of that).
//      The rest of the value enters by sums per row: of weights x (minimum + 8
//      scale), and of W as rounded, eightfold, which is taken off: so a weight's
//      rounding weighs with code - 8 and not with the code. That sum is one more
//      row of the product (with the code 8, of either size, so that it loses what
//      the MMA loses of products of subnormals), and is taken off after every 32
//      keys, before the sums of codes grow past what float32 keeps of the
//      difference. (Off by, of their size, f16 outputs: 3.0e-4; 3.2e-4 with a row
//      of ones; 6e-4 without that sum; 2.5e-4 with W in two f16 terms and ones,
//      but five tokens of 16 sequences take 20 us more than 99. The output's own
//      rounding is 2.1e-4. bf16 outputs, whose rounding is 1.7e-3, go without.)
// The weights are 2^(score - m) against a running maximum m that is raised only
// when a score passes it by more than 8; their sum is float32.
//
// Nothing is planned on the device and nothing depends on the key bound. A
// block's warps are HB KV heads times KS runs of 32 keys; a slice is the 32 KS
// keys that they take at a time. The slices of all sequences of the class, one
// after another, are cut into equal ranges, one per block of a head group, and
// every warp counts them for itself from the lengths. The block's warps take
// turns at copying the slices into its ring, by TMA boxes of 16 keys x HB heads
// that a lane issues per 16 keys; the copies run ahead across sequences. Every warp
// waits for each slice and gives its slot back, one without a head of its own (3, 6, 9,
// ... KV heads: three heads a block) too: a warp that copies turn T has then seen turn T
// - STAGES, the slot's last, in its slot, so the uses before that one are over, and the
// parity that it waits for means the use in question. (Waiting at its own turns only, it
// would know no more than that turn T - WARPS - STAGES is over, which is not enough with
// three stages.) A ring per warp, filled by its own 16-byte copies, cost 158 of 604
// instructions per 32 keys, and 64 sequences 77.4 us.
// A sequence's state that a warp does not hold whole goes to the workspace (see
// i4_piece), and int4_combine_kernel merges those, in order: no atomics, the same
// bits on every run.
// ---------------------------------------------------------------------------
constexpr int kI4MinSlices = 1;    // of a range
constexpr int kI4Keys = 32;        // of a warp: two halves of 16, each in one page

template <int D, int NR>
struct I4Cfg {
  static constexpr int WARPS = 4;
  static constexpr int THREADS = WARPS * 32;
  // Per SM. (Beyond 16 rows 255 registers a thread do not do at head size 128: 24 rows
  // spill 0.2 kB, 32 rows 0.9.)
  static constexpr int BLOCKS = NR == 1 ? 4 : 2;
  static constexpr int STAGES = (NR == 1 ? 3 : 6) + (D == 64 ? 2 : 0);
  // Of a stage: 16 keys of K of each warp, twice, as many of V, their params (of a
  // half's heads at a TMA destination of its own, so on 128 bytes).
  static constexpr int HALF = 16 * D / 2;              // 16 keys of a head
  static constexpr int OFF_V = 2 * WARPS * HALF;
  static constexpr int OFF_KP = 2 * OFF_V;
  static constexpr int OFF_VP = OFF_KP + 2 * WARPS * 128;
  static constexpr int STAGE = OFF_VP + 2 * WARPS * 128;
  static constexpr int OFF_BAR = STAGES * STAGE;
  static constexpr int SMEM_BYTES = OFF_BAR + 2 * STAGES * 8 + 64 + 1024;
};
static_assert(I4Cfg<128, 1>::STAGE % 1024 == 0 && I4Cfg<64, 1>::STAGE % 256 == 0, "swizzled tiles");
static_assert(I4Cfg<64, 1>::BLOCKS * (I4Cfg<64, 1>::SMEM_BYTES + 1024) <= 228 * 1024, "blocks");
static_assert(I4Cfg<128, 2>::BLOCKS * (I4Cfg<128, 2>::SMEM_BYTES + 1024) <= 228 * 1024, "blocks");
static_assert(I4Cfg<128, 1>::BLOCKS * (I4Cfg<128, 1>::SMEM_BYTES + 1024) <= 228 * 1024, "blocks");

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
  q.n = mine ? max(1, static_cast<int>((q.kv + a.slice_keys - 1u) / a.slice_keys)) : 0;
  return q;
}

// D += A(16x16, row) * B(16x8, col), f16 operands: mma_16816_f16 left to the
// compiler's scheduling.
__device__ __forceinline__ void mma_codes(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
      " {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 1 / x of a power of two.
__device__ __forceinline__ float inverse_power(float x) {
  return __uint_as_float((254u << 23) - __float_as_uint(x));
}

// A quotient; numbers of this size hardly ever need 64 bits.
__device__ __forceinline__ long long i4_div(long long a, long long b) {
  return (a | b) >> 32 ? a / b : static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
}
// Slices of a range, given all of them.
__device__ __forceinline__ long long i4_per_range(const Int4DecodeArgs& a, long long total) {
  const long long per = i4_div(total + a.ranges - 1, a.ranges);
  return per < kI4MinSlices ? kI4MinSlices : per;
}
// Token of a packed row (below 32).
__device__ __forceinline__ int i4_token(const Int4DecodeArgs& a, int row) {
  return row * a.g_inv >> 16;
}

// Where the states of sequence s's slices in a range go, in units of a head group's
// warps. With one key run a warp holds a sequence whole that lies in one range, and
// writes its output itself: two places a range, for a sequence that began in front of
// it or with it (0) and for one that starts inside and goes on (1). With several runs
// every sequence of a range leaves its states, however many there are: range + s, which
// grows from each piece to the next, since that is of the next range or of a later
// sequence.
__device__ __forceinline__ int64_t i4_piece(const Int4DecodeArgs& a, int range, int s,
                                            bool inside) {
  return a.key_runs == 1 ? 2 * static_cast<int64_t>(range) + inside
                         : static_cast<int64_t>(range) + s;
}

// Where a range starts: the sequence base + at (base a multiple of 32), its slice
// i, slice `begin` of all; and the range's slices (0: none).
struct I4Start {
  int base, at, i, count;
  long long begin;
};

// By one warp; the last block's leaves each sequence's first slice and the
// slices of a range to the combine kernel, in a.table.
__device__ __forceinline__ I4Start i4_start(const Int4DecodeArgs& a, int range, bool report,
                                            bool table) {
  constexpr unsigned kAll = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  I4Start f{};
  long long total = 0;
  for (int s = lane; s < a.num_seqs; s += 32) total += i4_seq(a, s, report).n;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kAll, total, o);
  const long long per = i4_per_range(a, total);
  f.begin = range * per;
  f.count = static_cast<int>(max(0ll, min(per, total - f.begin)));
  if (f.count == 0 && !table) return f;
  if (table && lane == 0) a.table[0] = per;
  bool found = false;
  long long before = 0;            // slices of the sequences in front of base
  for (int base = 0; base < a.num_seqs; base += 32) {
    const int n = base + lane < a.num_seqs ? i4_seq(a, base + lane, false).n : 0;
    int incl = n;                  // (32 times 2^25 slices: 31 bits)
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(kAll, incl, o);
      if (lane >= o) incl += x;
    }
    if (table && base + lane < a.num_seqs) a.table[1 + base + lane] = before + incl - n;
    const unsigned past = __ballot_sync(kAll, before + incl > f.begin);
    if (past && !found) {
      found = true;
      f.base = base;
      f.at = __ffs(past) - 1;
      f.i = static_cast<int>(f.begin - (before + __shfl_sync(kAll, incl - n, f.at)));
      if (!table) break;
    }
    before += __shfl_sync(kAll, incl, 31);
  }
  if (!found) f.count = 0;         // (or the lengths changed under the call)
  return f;
}

// Bytes between the params of a stage's halves.
__device__ __forceinline__ int i4_par_pitch(const Int4DecodeArgs& a) {
  return (a.heads_per_block * 64 + 127) & ~127;
}

// A warp's turns at copying: every WARPS-th slice of the block's range.
template <int D, int NR>
struct I4Copier {
  using C = I4Cfg<D, NR>;
  int base, at, n_l, kv_l;       // lane x holds the lengths of sequence base + x
  int i, n, kv;                  // the next slice, of sequence base + at
  int turn;                      // its place in the range
  int slot, phase;               // its slot, and the parity of the slot's last use
  int page, row;                 // lane h: of its half h

  __device__ __forceinline__ void load_pages(const Int4DecodeArgs& a) {
    const int lane = threadIdx.x & 31, halves = 2 * a.key_runs;
    page = a.no_page;                                  // outside the pool: reads as zeros
    row = 0;
    const int key0 = (i * halves + lane) * 16;
    if (lane < halves && key0 < kv) {
      const int lp = a.bs_shift >= 0 ? key0 >> a.bs_shift : key0 / a.bs;
      row = key0 - lp * a.bs;
      page = __ldg(a.bt + static_cast<int64_t>(base + at) * a.bt_stride + lp);
      if (page < 0 || page >= a.num_blocks) {
        page = a.no_page;
        flag_status(a.status, PA_DEV_BAD_PAGE);
      }
    }
  }
  // On by so many slices, across sequences; there are as many.
  __device__ __forceinline__ void advance(const Int4DecodeArgs& a, int by) {
    i += by;
    if (i >= n) next_sequence(a);
    load_pages(a);
  }
  __device__ __forceinline__ void next_sequence(const Int4DecodeArgs& a) {
    constexpr unsigned kAll = 0xffffffffu;
    const int lane = threadIdx.x & 31;
    while (i >= n) {
      i -= n;
      do {
        if (++at == 32) {
          at = 0;
          base += 32;
          n_l = kv_l = 0;
          if (base + lane < a.num_seqs) {
            const I4Seq q = i4_seq(a, base + lane, false);
            n_l = q.n;
            kv_l = q.kv;
          }
        }
        n = __shfl_sync(kAll, n_l, at);
      } while (n == 0 && base < a.num_seqs);
      kv = __shfl_sync(kAll, kv_l, at);
      if (n == 0) {                                    // (lengths changed under the call)
        i = kv = 0;
        break;
      }
    }
  }
  // The slice into its slot, once the slot's last one is used; on to the next.
  __device__ __forceinline__ bool copy(const Int4DecodeArgs& a, const CUtensorMap* tm,
                                       uint8_t* smem, uint64_t* full, uint64_t* empty, int head0,
                                       int count) {
    const int lane = threadIdx.x & 31;
    bool ok = true;
    if (turn >= C::STAGES) ok = mbar_wait(&empty[slot], phase ^ 1);
    if (!__all_sync(0xffffffffu, ok)) return false;
    if (lane == 0)
      mbar_arrive_expect_tx(&full[slot],
                            2 * a.key_runs * a.heads_per_block * (2 * C::HALF + 128));
    __syncwarp();
    if (lane < 2 * a.key_runs) {
      uint8_t* st = smem + slot * C::STAGE;
      const int of = lane * a.heads_per_block, p_of = lane * i4_par_pitch(a);
      tma_load_4d(st + of * C::HALF, tm, &full[slot], 0, row, head0, page);
      tma_load_4d(st + C::OFF_V + of * C::HALF, tm + 1, &full[slot], 0, row, head0, page);
      tma_load_3d(st + C::OFF_KP + p_of, tm + 2, &full[slot], row, head0, page);
      tma_load_3d(st + C::OFF_VP + p_of, tm + 3, &full[slot], row, head0, page);
    }
    for (slot += C::WARPS; slot >= C::STAGES; slot -= C::STAGES) phase ^= 1;
    turn += C::WARPS;
    if (turn < count) advance(a, C::WARPS);
    return true;
  }
};

template <int D, bool F16, int NR>
__global__ void __launch_bounds__(I4Cfg<D, NR>::THREADS, I4Cfg<D, NR>::BLOCKS)
int4_decode_kernel(const __grid_constant__ Int4Maps maps, const __grid_constant__ Int4DecodeArgs a) {
  using C = I4Cfg<D, NR>;
  using E = Elem<F16>;
  constexpr int KW = D / 32;       // words of a key per lane in S^T
  constexpr int CH = D / 32;       // 16-byte pieces of a key
  constexpr unsigned kAll = 0xffffffffu;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* empty = full + C::STAGES;
  I4Start* start = reinterpret_cast<I4Start*>(empty + C::STAGES);
  volatile int* abort = reinterpret_cast<volatile int*>(start + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  pdl_trigger();                   // the combine kernel may be placed when these blocks have been
  const int groups = a.H_kv / a.heads_per_block;
  const int range = static_cast<int>(blockIdx.x) / groups;
  const int group = static_cast<int>(blockIdx.x) - range * groups;
  const int consumers = a.heads_per_block * a.key_runs;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], C::WARPS);
    }
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 1 && lane < 4) tma_prefetch_desc(maps.m + lane);
  pdl_wait();                      // what the stream did before is done (see the launcher)
  if (warp == 0) {
    const I4Start f = i4_start(a, range, blockIdx.x == 0, blockIdx.x == gridDim.x - 1);
    if (lane == 0) *start = f;
  }
  __syncthreads();
  I4Start from = *start;
  if (from.count == 0) return;
  I4Seq sq{0, 0, 0, 0};            // lane x holds sequence base + x
  if (from.base + lane < a.num_seqs) sq = i4_seq(a, from.base + lane, false);
  const int head0 = group * a.heads_per_block;
  I4Copier<D, NR> copier;
  copier.base = from.base;
  copier.at = from.at;
  copier.n_l = sq.n;
  copier.kv_l = sq.kv;
  copier.i = from.i;
  copier.n = __shfl_sync(kAll, sq.n, from.at);
  copier.kv = __shfl_sync(kAll, sq.kv, from.at);
  copier.turn = warp;
  copier.slot = warp % C::STAGES;
  copier.phase = (warp / C::STAGES) & 1;
  bool ok = true;
  if (warp < from.count) copier.advance(a, warp);
  // The first slices: turns 0 .. STAGES - 2.
  while (copier.turn < min(C::STAGES - 1, from.count))
    copier.copy(a, maps.m, smem, full, empty, head0, from.count);
  int base = from.base, at = from.at, i = from.i;
  const long long begin = from.begin;
  const int run = warp / a.heads_per_block, hl = warp - run * a.heads_per_block;
  const int hk = head0 + hl;
  const bool idle = warp >= consumers;                 // has no head

  // This warp's first half in a stage, and from there to the second.
  const int k_at = (2 * run * a.heads_per_block + hl) * C::HALF, k_next = a.heads_per_block * C::HALF;
  const int p_next = i4_par_pitch(a), p_at = C::OFF_KP + 2 * run * p_next + hl * 64;
  // Row g (g + 8) of S^T is key g (g + 8) of a half; the tiles are swizzled: 16-byte
  // piece x of row r lies at x ^ (r / 2 % 4) of four (D = 64: x ^ (r / 4 % 2) of two).
  const int k_piece = D == 128 ? (c ^ ((g >> 1) & 3)) * 16 : ((c >> 1) ^ ((g >> 2) & 1)) * 16 + (c & 1) * 8;
  // This lane's row address in the transposed loads: matrices keys 0-7 | 8-15 of a
  // piece, then of the next.
  const uint32_t smem_at = smem_u32(smem);
  const int v_row = (lane & 7) + ((lane >> 3) & 1) * 8, v_half = lane >> 4;
  const int v_swizzle = D == 128 ? (v_row >> 1) & 3 : (v_row >> 2) & 1;
  int left = from.count, t = 0, slot = 0;
  uint32_t phase = 0;
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
      const int r = min(8 * nr + g, rows - 1), t = i4_token(a, r);
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
    float acc[NR][D / 16][4], accw[NR][4];             // accw: of 8 W, in a column's units
    float ref = 0.f;                                   // power of two, at least |V's scales| so far
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
          fadd2(acc[nr][t][0], acc[nr][t][1], acc[nr][t][0], acc[nr][t][1], -accw[nr][0],
                -accw[nr][1]);
          fadd2(acc[nr][t][2], acc[nr][t][3], acc[nr][t][2], acc[nr][t][3], -accw[nr][2],
                -accw[nr][3]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) accw[nr][e] = 0.f;
      }
    };

#pragma unroll 1
    for (; i < i1; ++i, ++t, ++slot) {
      if (slot == C::STAGES) {
        slot = 0;
        phase ^= 1;
      }
      // In turn, the slice that goes where the last one was: the other warps have
      // had this one's time to be done with that.
      const bool mine = copier.turn == t + C::STAGES - 1 && copier.turn < from.count;
      ok = __all_sync(kAll, ok && mbar_wait(&full[slot], phase));
      if (!ok) break;
      const uint8_t* sl = smem + slot * C::STAGE;
      const uint32_t sl_at = smem_at + slot * C::STAGE;
      const int key0 = (i * a.key_runs + run) * kI4Keys;
      if (idle || key0 >= kv) {                        // none of this warp's
        if (mine) ok = copier.copy(a, maps.m, smem, full, empty, head0, from.count);
        if (lane == 0) mbar_arrive(&empty[slot]);
        continue;
      }
      // ----------------------------------------------------------- S^T = N Q^T
      float st[NR][2][4];
#pragma unroll
      for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int h = 0; h < 2; ++h) st[nr][h][0] = st[nr][h][1] = st[nr][h][2] = st[nr][h][3] = 0.f;
      uint32_t w0[2][KW], w1[2][KW];                   // keys g, g + 8 of each half
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint8_t* kt = sl + k_at + h * k_next + g * (D / 2) + k_piece;
        if constexpr (D == 128) {
          const uint4 x0 = *reinterpret_cast<const uint4*>(kt);
          const uint4 x1 = *reinterpret_cast<const uint4*>(kt + 8 * (D / 2));
          w0[h][0] = x0.x; w0[h][1] = x0.y; w0[h][2] = x0.z; w0[h][3] = x0.w;
          w1[h][0] = x1.x; w1[h][1] = x1.y; w1[h][2] = x1.z; w1[h][3] = x1.w;
        } else {
          const uint2 x0 = *reinterpret_cast<const uint2*>(kt);
          const uint2 x1 = *reinterpret_cast<const uint2*>(kt + 8 * (D / 2));
          w0[h][0] = x0.x; w0[h][1] = x0.y;
          w1[h][0] = x1.x; w1[h][1] = x1.y;
        }
      }
#pragma unroll
      for (int v = 0; v < KW; ++v) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t a0 = w0[h][v] >> (8 * k), a1 = w1[h][v] >> (8 * k);
#pragma unroll
            for (int nr = 0; nr < NR; ++nr)
              mma_codes(st[nr][h], a0 & 0x000F000Fu, a1 & 0x000F000Fu, a0 & 0x00F000F0u,
                        a1 & 0x00F000F0u, qf[nr][2 * v + k][0], qf[nr][2 * v + k][1]);
          }
        }
      }
      // ----------------------------------------------------------- softmax
      // Keys 8 h + g of the warp's, h = 0 .. 3: entries 2 (h & 1) of st[h >> 1].
      const uint8_t* par = sl + p_at + g * 4;
      uint32_t pkw[4], pvw[4];
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const uint8_t* p = par + (h >> 1) * p_next + (h & 1) * 32;
        pkw[h] = *reinterpret_cast<const uint32_t*>(p);
        pvw[h] = *reinterpret_cast<const uint32_t*>(p + (C::OFF_VP - C::OFF_KP));
      }
      float ks[4], km[4], vs[4], vm[4];
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const float2 k = Elem<true>::unpack(pkw[h]), v = Elem<true>::unpack(pvw[h]);
        ks[h] = k.x * 0x1p24f;
        km[h] = k.y;
        vs[h] = v.x;
        vm[h] = F16 ? fmaf(8.f, v.x, v.y) : v.y;
      }
      const bool whole = key0 + kI4Keys <= seen_by_all;
      if (!whole) {                                    // what lies past the sequence is nobody's
#pragma unroll
        for (int h = 0; h < 4; ++h)
          if (key0 + 8 * h + g >= kv) vs[h] = vm[h] = 0.f;
      }
      const float vtop = fmaxf(fmax3(fabsf(vs[0]), fabsf(vs[1]), fabsf(vs[2])), fabsf(vs[3]));
      if (__any_sync(kAll, vtop > ref)) {              // raise the reference of V's scales
        float top = vtop;
        if (top == INFINITY) {   // (without these: rows that do not see them have no part in it)
          top = 0.f;
#pragma unroll
          for (int h = 0; h < 4; ++h)
            top = fmaxf(top, fabsf(vs[h]) == INFINITY ? 0.f : fabsf(vs[h]));
        }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
        // The power of two above it, and 4: a larger one is then seldom met.
        const float nr_ref =
            top > ref ? __uint_as_float(((__float_as_uint(top) >> 23) + 3u) << 23) : ref;
        const float f = ref == 0.f ? 0.f : ref * inverse_power(nr_ref);
        ref = nr_ref;
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
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
            const int lim = a.causal ? past + i4_token(a, row) : kv - 1;   // last visible key
#pragma unroll
            for (int h = 0; h < 4; ++h)
              if (key0 + 8 * h + g > lim) x[h][e] = -INFINITY;
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
        for (int h = 0; h < 4; ++h) {
          wb[nr][h] = movmatrix_trans(pack_f16(w[h][0], w[h][1]));
        }
      }
      // ----------------------------------------------------------- O^T += N^T W^T
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // Transposed loads: 16 bits of a key (four elements of one parity) are an
        // element of an 8x8 matrix, so a register holds them of two keys.
        const uint32_t vt = sl_at + C::OFF_V + k_at + h * k_next + v_row * (D / 2);
        uint32_t wv[CH][2];        // piece x, keys 2c, 2c + 1 and 2c + 8, 2c + 9
#pragma unroll
        for (int x = 0; x < CH; x += 2)
          ldsm_x4_t(vt + (((x + v_half) ^ v_swizzle) << 4), wv[x][0], wv[x][1], wv[x + 1][0],
                    wv[x + 1][1]);
        if constexpr (F16) {
#pragma unroll
          for (int nr = 0; nr < NR; ++nr)
            mma_codes(accw[nr], 0x00080008u, 0x00800080u, 0x00080008u, 0x00800080u, wb[nr][2 * h],
                      wb[nr][2 * h + 1]);
        }
#pragma unroll
        for (int x = 0; x < CH; ++x) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t u0 = wv[x][0] >> (8 * k), u1 = wv[x][1] >> (8 * k);
#pragma unroll
            for (int nr = 0; nr < NR; ++nr)
              mma_codes(acc[nr][2 * x + k], u0 & 0x000F000Fu, u0 & 0x00F000F0u, u1 & 0x000F000Fu,
                        u1 & 0x00F000F0u, wb[nr][2 * h], wb[nr][2 * h + 1]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[slot]);        // the slot may be filled again
      if (mine) ok = copier.copy(a, maps.m, smem, full, empty, head0, from.count);
      if (F16) centre();
    }
    if (!ok) break;

    // ---------------------------------------------------------------- the state
    // acc[2 x + k] holds elements 32 x + 8 (g / 2) + g % 2 + 4 k (entries 0, 1: rows
    // 2c, 2c + 1) and 2 further (2, 3; sixteenfold): with lane ^ 4, eight of a row.
    const bool all = i0 == 0 && i1 == n && a.key_runs == 1;
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) {
      if (idle) break;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float L = l[nr][e], V = lv[nr][e];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          L += __shfl_xor_sync(kAll, L, o);
          V += __shfl_xor_sync(kAll, V, o);
        }
        const int row = 8 * nr + 2 * c + e;
        const int t = i4_token(a, min(row, rows - 1)), head = hk * a.G + min(row, rows - 1) - t * a.G;
        float M = m[nr][e], of = 1.f;
        const float fw = ref * (0x1p24f / 64.f);       // of the sums of codes
        if (all && a.sinks) of = add_sink(M, L, __ldg(a.sinks + head) * kLog2e);
        const float inv = L == 0.f ? 0.f : of / L;
        const float lse = L == 0.f ? -INFINITY : (M + fast_log2(L)) * kLn2;
        const int64_t at_row =
            ((i4_piece(a, range, base + at, flat != begin) * groups + group) * C::WARPS + warp) *
                (8 * NR) + row;
#pragma unroll
        for (int x = 0; x < CH; ++x) {
          float o[4];                                  // elements 2 j + g % 2 of eight
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            o[2 * k] = fmaf(acc[nr][2 * x + k][e], fw, V) * inv;
            o[2 * k + 1] = fmaf(acc[nr][2 * x + k][2 + e], fw * 0.0625f, V) * inv;
          }
          // An even row of lanes takes elements 0 .. 3, an odd one 4 .. 7.
          const bool odd = g & 1;
          const float t0 = __shfl_xor_sync(kAll, odd ? o[0] : o[2], 4);
          const float t1 = __shfl_xor_sync(kAll, odd ? o[1] : o[3], 4);
          const float y0 = odd ? t0 : o[0], y1 = odd ? o[2] : t0;
          const float y2 = odd ? t1 : o[1], y3 = odd ? o[3] : t1;
          const int col = 32 * x + 4 * g;
          if (row >= rows) continue;
          if (all)
            *reinterpret_cast<uint2*>(a.out + (static_cast<int64_t>(q0 + t) * a.H + head) * D +
                                      col) = make_uint2(E::pack(y0, y1), E::pack(y2, y3));
          else
            __stcg(reinterpret_cast<float4*>(a.part_o + at_row * D + col),
                   make_float4(y0, y1, y2, y3));
        }
        if (g == 0 && row < rows) {
          if (!all) __stcg(a.part_lse + at_row, lse);
          else if (a.lse) a.lse[static_cast<int64_t>(head) * a.total_q + q0 + t] = lse;
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
  if (!ok) flag_status(a.status, PA_DEV_TIMEOUT);
  if (!ok || left > 0) *abort = 1;
  __syncthreads();
  // After a wait that gave up, and where lengths shrank under the call: the copies in
  // flight end before the block does.
  if (*abort && warp == 0)
    for (int u = 0; u < from.count; ++u)
      if (!mbar_wait(&full[u % C::STAGES], (u / C::STAGES) & 1)) break;
}

// ---------------------------------------------------------------------------
// The sequences whose slices lie in more than one range or key run: their
// states, in the ranges' order. A block takes two rows of a (sequence, KV head); a
// thread takes four dims of a row and a quarter (head size 64: an eighth) of the
// states, joined through shared memory in order. With rows for at most two blocks an
// SM (WIDE) a block takes one row and sixteen parts: few sequences have many states
// each. Four sequences of 60000 to 131072 keys, 64 heads: 80.6 us where two rows a
// block take 89.0; 64 sequences 86.8 and 75.9.
// ---------------------------------------------------------------------------
template <int D, bool WIDE>
struct I4Combine {
  static constexpr int THREADS = WIDE ? 4 * D : 256, ROWS = WIDE ? 1 : 2;
};

template <int D, bool F16, int NR, bool WIDE>
__global__ void __launch_bounds__(I4Combine<D, WIDE>::THREADS, 1280 / I4Combine<D, WIDE>::THREADS)
int4_combine_kernel(const __grid_constant__ Int4DecodeArgs a) {
  constexpr int THREADS = I4Combine<D, WIDE>::THREADS, ROWS = I4Combine<D, WIDE>::ROWS;
  __shared__ float4 part_o[THREADS];
  __shared__ float2 part_ml[THREADS];
  const int s = static_cast<int>(blockIdx.x) / a.H_kv;
  const int hk = static_cast<int>(blockIdx.x) - s * a.H_kv;
  // The lengths too: the decode kernel lets this one start before its own wait, so what
  // the stream did in front of the call may still be under way.
  pdl_wait();
  const I4Seq sq = i4_seq(a, s, false);
  if (sq.n == 0) return;
  const int groups = a.H_kv / a.heads_per_block, group = hk / a.heads_per_block;
  const int hl = hk - group * a.heads_per_block;
  constexpr int WIDTH = ROWS * (D / 4), PARTS = THREADS / WIDTH;
  const int rows = sq.q_len * a.G, part = threadIdx.x / WIDTH;
  const int unit = threadIdx.x - part * WIDTH;
  const int row = blockIdx.y * ROWS + unit / (D / 4), col = unit % (D / 4) * 4;
  if (blockIdx.y * ROWS >= rows) return;
  const long long per = __ldcg(a.table), before = __ldcg(a.table + 1 + s);
  const int r0 = static_cast<int>(i4_div(before, per));
  const int r1 = static_cast<int>(i4_div(before + sq.n - 1, per));
  const int n = (r1 - r0 + 1) * a.key_runs;
  if (n == 1) return;                                  // written by its warp
  // State j: range r0 + j / key_runs, run j % key_runs.
  const bool inside = before > r0 * per;
  const int run_shift = 31 - __clz(a.key_runs);        // 1, 2 or 4
  const int j1 = n * (part + 1) / PARTS;
  float mx = -INFINITY, sw = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  if (row < rows) {
    for (int j = n * part / PARTS; j < j1; j += kBatch) {
      float l[kBatch];
      float4 v[kBatch];
#pragma unroll
      for (int x = 0; x < kBatch; ++x) {
        if (j + x >= j1) continue;
        const int q = (j + x) >> run_shift, run = j + x - (q << run_shift);
        const int64_t slot =
            (i4_piece(a, r0 + q, s, q == 0 && inside) * groups + group) * I4Cfg<D, NR>::WARPS +
            run * a.heads_per_block + hl;
        const int64_t at = slot * (8 * NR) + row;
        l[x] = __ldcg(a.part_lse + at);
        v[x] = __ldcg(reinterpret_cast<const float4*>(a.part_o + at * D + col));
      }
      merge_batch(mx, sw, o, l, v, min(kBatch, j1 - j));
    }
  }
  part_o[threadIdx.x] = make_float4(o[0], o[1], o[2], o[3]);
  part_ml[threadIdx.x] = make_float2(mx, sw);
  __syncthreads();
  if (part != 0 || row >= rows) return;
#pragma unroll
  for (int p = 1; p < PARTS; ++p) {
    const float2 ml = part_ml[threadIdx.x + p * WIDTH];
    const float4 x = part_o[threadIdx.x + p * WIDTH];
    const float nm = fmaxf(mx, ml.x);
    const float f0 = mx == -INFINITY ? 0.f : fast_exp2((mx - nm) * kLog2e);
    const float f1 = ml.x == -INFINITY ? 0.f : fast_exp2((ml.x - nm) * kLog2e);
    mx = nm;
    sw = sw * f0 + ml.y * f1;
    o[0] = o[0] * f0 + x.x * f1;
    o[1] = o[1] * f0 + x.y * f1;
    o[2] = o[2] * f0 + x.z * f1;
    o[3] = o[3] * f0 + x.w * f1;
  }
  const int t = i4_token(a, row), head = hk * a.G + row - t * a.G;
  if (a.sinks) {
    const float ls[kBatch] = {__ldg(a.sinks + head)};
    const float4 z[kBatch] = {make_float4(0.f, 0.f, 0.f, 0.f)};
    merge_batch(mx, sw, o, ls, z, 1);
  }
  const float inv = sw == 0.f ? 0.f : 1.f / sw;
  *reinterpret_cast<uint2*>(a.out + (static_cast<int64_t>(sq.q0 + t) * a.H + head) * D + col) =
      make_uint2(Elem<F16>::pack(o[0] * inv, o[1] * inv), Elem<F16>::pack(o[2] * inv, o[3] * inv));
  if (a.lse && col == 0)
    a.lse[static_cast<int64_t>(head) * a.total_q + sq.q0 + t] =
        sw == 0.f ? -INFINITY : mx + fast_log2(sw) * kLn2;
}

template <int D, bool F16, int NR>
static cudaError_t launch_int4_decode_nr(const Int4Maps& maps, const Int4DecodeArgs& a, int sms,
                                         cudaStream_t st) {
  using C = I4Cfg<D, NR>;
  static std::atomic<bool> configured[kMaxDevices];
  cudaError_t e = opt_in_smem(int4_decode_kernel<D, F16, NR>, C::SMEM_BYTES, configured);
  if (e != cudaSuccess) return e;
  const unsigned blocks = static_cast<unsigned>(a.ranges) * (a.H_kv / a.heads_per_block);
  // Both kernels are programmatic dependents of what is in front of them on the
  // stream, of whatever kind: their blocks may be placed while that ends, and wait
  // for it (griddepcontrol.wait) before they read anything.
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = st;
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM_BYTES;
  e = cudaLaunchKernelEx(&cfg, int4_decode_kernel<D, F16, NR>, maps, a);
  if (e != cudaSuccess || (e = cudaGetLastError()) != cudaSuccess) return e;
  const int most = min(a.tokens_max, a.max_q) * a.G;   // rows of a sequence
  const unsigned units = static_cast<unsigned>(a.num_seqs) * static_cast<unsigned>(a.H_kv);
  cfg.dynamicSmemBytes = 0;
  if (static_cast<int64_t>(units) * most <= 2 * sms) {
    cfg.gridDim = dim3(units, most);
    cfg.blockDim = dim3(I4Combine<D, true>::THREADS);
    e = cudaLaunchKernelEx(&cfg, int4_combine_kernel<D, F16, NR, true>, a);
  } else {
    cfg.gridDim = dim3(units, (most + 1) / 2);
    cfg.blockDim = dim3(I4Combine<D, false>::THREADS);
    e = cudaLaunchKernelEx(&cfg, int4_combine_kernel<D, F16, NR, false>, a);
  }
  return e == cudaSuccess ? cudaGetLastError() : e;
}

int int4_decode_heads(int H_kv) {
  for (int h = I4Cfg<128, 1>::WARPS; h > 1; --h)
    if (H_kv % h == 0) return h;
  return 1;
}
// Ranges: the blocks that are resident, shared among the head groups.
static int i4_ranges(int sms, int H_kv, int nr) {
  const int blocks = nr == 1 ? I4Cfg<128, 1>::BLOCKS : I4Cfg<128, 2>::BLOCKS;
  const int n = sms * blocks / (H_kv / int4_decode_heads(H_kv));
  return n < 1 ? 1 : n;
}

// (Pieces: see i4_piece.)
size_t int4_decode_part_rows(int sms, int H_kv, int nr, int num_seqs) {
  const int heads = int4_decode_heads(H_kv);
  const size_t ranges = i4_ranges(sms, H_kv, nr);
  const size_t pieces = I4Cfg<128, 1>::WARPS / heads == 1 ? 2 * ranges : ranges + num_seqs;
  return pieces * (H_kv / heads) * I4Cfg<128, 1>::WARPS * 8 * nr;
}

cudaError_t launch_int4_decode(const Int4Maps& maps, Int4DecodeArgs a, int D, bool f16, int nr,
                               int sms, cudaStream_t st) {
  a.ranges = i4_ranges(sms, a.H_kv, nr);
  a.heads_per_block = int4_decode_heads(a.H_kv);
  a.key_runs = I4Cfg<128, 1>::WARPS / a.heads_per_block;
  a.slice_keys = a.key_runs * kI4Keys;
  a.g_inv = (65536 + a.G - 1) / a.G;
  auto by_rows = [&](auto d, auto half) {
    constexpr int kD = decltype(d)::value;
    constexpr bool kF16 = decltype(half)::value;
    if (nr == 1) return launch_int4_decode_nr<kD, kF16, 1>(maps, a, sms, st);
    if (nr == 2) return launch_int4_decode_nr<kD, kF16, 2>(maps, a, sms, st);
    if (nr == 3) return launch_int4_decode_nr<kD, kF16, 3>(maps, a, sms, st);
    return launch_int4_decode_nr<kD, kF16, 4>(maps, a, sms, st);
  };
  using std::integral_constant;
  if (D == 128)
    return f16 ? by_rows(integral_constant<int, 128>{}, std::true_type{})
               : by_rows(integral_constant<int, 128>{}, std::false_type{});
  return f16 ? by_rows(integral_constant<int, 64>{}, std::true_type{})
             : by_rows(integral_constant<int, 64>{}, std::false_type{});
}

}  // namespace pa
