// Attention over 4-bit pools for prompts: the tensor-core prefill kernel of
// attn_tc.cu with K widened to codes and V to values on the way.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>

#include "attn_tc.cuh"

namespace pa {

// ---------------------------------------------------------------------------
// Work items, softmax, products and epilogue are the prefill kernel's. What
// differs is how K, V and Q reach the products:
//  * Warp 0 of the control warpgroup widens K, warps 2 and 3 widen V, half a tile
//    each, which costs the three about the same. A unit is 16 keys; a warp takes
//    them by pairs, whose codes, scales and minima it copies ahead of their use
//    into a ring of its own (a lane copies the codes that it reads back itself), so
//    no barrier stands between the pools and the registers.
//  * K reaches the product as codes, exact in Q's type, and Q as it is: for f16 a
//    mask makes two subnormals n 2^-24, for bf16 128 + n by a mask and 128 taken
//    off. The softmax applies scale and minimum to the sums, in float32 (one
//    multiply and one multiply-add per two scores; each row sums its Q once): with
//    K rounded to f16 values instead, the log-sum-exp lost ten of its bits. The
//    sign of a negative softmax scale joins scale and minimum, so the row maximum
//    of what the softmax sees serves every scale.
//  * V becomes values: n exactly as f16 (from 1024 + n or 1024 + 16 n), and n
//    scale + minimum by one multiply-add: one rounding, at most half a step of
//    the value. Rows past the sequence are zeros.
//  * The widened tiles have the 2-byte kernel's layout (128-byte swizzle), two
//    buffers each for K and V; the products that read a buffer free it.
//  * What bounds it: four prompts of 2500 to 4096 tokens, 32 heads of 128
//    over 8, take 700 us (0.5 of 1.9 PFLOP/s), 443 with neither the widening nor the
//    scales and minima in the softmax. Widening K and V costs 135 of the difference,
//    the softmax's loads of scales and minima and their arithmetic 70, the two
//    together the rest: shared memory and issue slots are shared. (Seven widening
//    warps in four more warps of 56 registers: 960 us, they spill. Loading scales
//    before the products are there: 1250, likewise.)
// ---------------------------------------------------------------------------

// A piece of K, 32 codes (16 bytes), as 64 bytes of bf16 numbers or f16 2^-24 of
// them, at to[0 .. 3].
template <bool F16>
__device__ __forceinline__ void spread_int4_piece(const uint4& x, uint8_t* dst, const int (&to)[4]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    uint32_t y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      y[k] = w[v] >> (4 * k) & 0x000F000Fu;
      if constexpr (!F16) {
        y[k] |= 0x43004300u;                             // 128 + n
        const __nv_bfloat162 n = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&y[k]),
                                         __float2bfloat162_rn(128.f));
        y[k] = *reinterpret_cast<const uint32_t*>(&n);
      }
    }
    *reinterpret_cast<uint4*>(dst + to[v]) = make_uint4(y[0], y[1], y[2], y[3]);
  }
}

// A piece of V as 64 bytes of f16 values.
__device__ __forceinline__ void widen_int4_piece(const uint4& x, uint32_t params, uint8_t* dst,
                                                 const int (&to)[4]) {
  const __half2 s = __half2half2(__ushort_as_half(static_cast<unsigned short>(params & 0xffffu)));
  const __half2 m = __half2half2(__ushort_as_half(static_cast<unsigned short>(params >> 16)));
  const __half2 k1024 = __half2half2(__ushort_as_half(0x6400));
  const __half2 k16th = __half2half2(__ushort_as_half(0x2C00));
  const __half2 k64 = __half2half2(__ushort_as_half(0xD400));   // -1024 / 16
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    uint32_t y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t t = w[v] >> (8 * (k >> 1));
      uint32_t h = (t & ((k & 1) ? 0x00F000F0u : 0x000F000Fu)) | 0x64006400u;
      __half2 n = *reinterpret_cast<__half2*>(&h);
      n = (k & 1) ? __hfma2(n, k16th, k64) : __hsub2(n, k1024);
      n = __hfma2(n, s, m);
      y[k] = *reinterpret_cast<uint32_t*>(&n);
    }
    *reinterpret_cast<uint4*>(dst + to[v]) = make_uint4(y[0], y[1], y[2], y[3]);
  }
}

// A widening warp: units u0 .. u0 + UPT - 1 of every K (or V) tile, by pairs,
// through a ring of RING pairs at `ring`.
template <int D, bool F16, bool IS_V, int UPT, int RING>
__device__ __forceinline__ bool widen_tiles(const AttnArgs& a, const Int4Pools& pool, TcBars* bars,
                                            uint8_t* smem, uint8_t* ring, const int32_t* bt_row,
                                            int hk, int kb, int kv_len, int ntiles, int u0) {
  using C = TcCfg<D>;
  using I = TcI4<D>;
  constexpr int PIECES = D / 32;                         // of a row, 16 bytes each
  constexpr int PER = 16 * PIECES / 32;                  // of a unit, per lane (2 or 1)
  constexpr int PAIR = 2 * I::SLOT, PPT = UPT / 2;       // bytes of a pair, pairs of a tile
  const int lane = threadIdx.x & 31;
  const int px = lane % PIECES, pr = lane / PIECES;      // piece, first row
  const int64_t rstep = static_cast<int64_t>(a.H_kv) * (D / 2);
  const uint8_t* src0 = (IS_V ? pool.vc : pool.kc) + hk * (D / 2) + pr * rstep + px * 16;
  const uint32_t* par0 = (IS_V ? pool.v_params : pool.k_params) +
                         static_cast<int64_t>(hk) * a.bs + (lane & 15);
  const uint32_t ring_at = smem_u32(ring);
  const int pairs = ntiles * PPT;
  // Lane i: page and row of unit 2 page0 + i of this warp's.
  int page0 = 0, page_l = -1, row_l = 0;
  auto load_pages = [&](int q) {
    page0 = q;
    page_l = -1;
    row_l = 0;
    const int n = 2 * q + lane, key0 = kb + n / UPT * C::BN + (u0 + n % UPT) * 16;
    if (n < 2 * pairs && key0 < kv_len) {
      const int lp = key0 / a.bs;
      row_l = key0 - lp * a.bs;
      page_l = __ldg(bt_row + lp);
      if (page_l < 0 || page_l >= a.num_blocks) {
        page_l = -1;                                     // reads as zeros
        flag_status(a.status, PA_DEV_BAD_PAGE);
      }
    }
  };
  int f_slot = 0;
  auto fetch = [&](int q) {
    if (q < pairs) {
      if (q - page0 == 16) load_pages(q);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int page = __shfl_sync(0xffffffffu, page_l, 2 * (q - page0) + x);
        const int prow = __shfl_sync(0xffffffffu, row_l, 2 * (q - page0) + x);
        const uint32_t dst = ring_at + f_slot * PAIR + x * I::SLOT;
        const uint8_t* src = src0 + max(page, 0) * pool.block_stride_bytes + prow * rstep;
#pragma unroll
        for (int y = 0; y < PER; ++y)
          cp_async16(dst + y * 512 + lane * 16, src + y * (32 / PIECES) * rstep, page >= 0);
        // Scales and minima; zeros past the sequence.
        const int n = 2 * q + x, key0 = kb + n / UPT * C::BN + (u0 + n % UPT) * 16;
        if (lane < 16)
          cp_async4(dst + 16 * D / 2 + lane * 4,
                    par0 + max(page, 0) * pool.params_stride + prow,
                    page >= 0 && key0 + lane < kv_len);
      }
      if (++f_slot == RING) f_slot = 0;
    }
    cp_async_commit();
  };
  load_pages(0);
#pragma unroll
  for (int q = 0; q < RING - 1; ++q) fetch(q);
  // Where a piece of row pr (mod 8) goes in a 128-byte swizzled tile.
  int to[4];
#pragma unroll
  for (int v = 0; v < 4; ++v)
    to[v] = (px >> 1) * C::KV_HALF + pr * 128 + ((((px & 1) * 4 + v) ^ (pr & 7)) << 4);
  const float sign = a.scale_log2 > 0.f ? 1.f : a.scale_log2 < 0.f ? -1.f : 0.f;
  int slot = 0, q = 0;
  for (int t = 0; t < ntiles; ++t) {
    const int buf = t & 1;
    // The buffer's last reader: the products of tile t - 2.
    bool ok = true;
    if (t >= I::BUFS)
      ok = mbar_wait(IS_V ? &bars->vw_free[buf] : &bars->kw_free[buf], ((t >> 1) - 1) & 1);
    if (!__all_sync(0xffffffffu, ok && !bars->abort)) return false;
    uint8_t* dst = smem + (IS_V ? I::OFF_VW : I::OFF_KW) + buf * C::KV_TILE + u0 * 16 * 128;
    float* par_to = reinterpret_cast<float*>(smem + I::OFF_PAR + t % I::PARS * C::BN * 8);
#pragma unroll 1
    for (int p = 0; p < PPT; ++p, ++q, dst += 32 * 128) {
      fetch(q + RING - 1);
      cp_async_wait<RING - 1>();
      __syncwarp();
      const uint8_t* sl = ring + slot * PAIR;
      uint4 w[2][PER];
      uint32_t par[2][PER];
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int y = 0; y < PER; ++y) {
          w[x][y] = *reinterpret_cast<const uint4*>(sl + x * I::SLOT + y * 512 + lane * 16);
          if (IS_V)
            par[x][y] = *reinterpret_cast<const uint32_t*>(sl + x * I::SLOT + 16 * D / 2 +
                                                           (pr + y * (32 / PIECES)) * 4);
        }
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int y = 0; y < PER; ++y) {
          uint8_t* at = dst + (x * 16 + y * (32 / PIECES)) * 128;
          if (IS_V) widen_int4_piece(w[x][y], par[x][y], at, to);
          else spread_int4_piece<F16>(w[x][y], at, to);
        }
      if (!IS_V) {   // lane: key `lane` of the pair's 32
        const float2 sm = Elem<true>::unpack(*reinterpret_cast<const uint32_t*>(
            sl + (lane >> 4) * I::SLOT + 16 * D / 2 + (lane & 15) * 4));
        float* at = par_to + ((u0 + 2 * p) * 16 + lane) / 2 * 4 + (lane & 1);
        at[0] = sm.x * (F16 ? sign * 0x1p24f : sign);
        at[2] = sm.y * sign;
      }
      __syncwarp();                                      // the slot may be filled again
      if (++slot == RING) slot = 0;
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(IS_V ? &bars->vw_full[buf] : &bars->kw_full[buf]);
      if (!IS_V) mbar_arrive(&bars->par_full[t % I::PARS]);
    }
  }
  return true;
}

template <int D, bool F16>
__global__ void __launch_bounds__(TcCfg<D>::THREADS, 1)
int4_prompt_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ AttnArgs a,
                   const __grid_constant__ Int4Pools pool) {
  using C = TcCfg<D>;
  using I = TcI4<D>;
  using Kind = TcKind<D, F16, false, false, false, true>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  TcBars* bars = reinterpret_cast<TcBars*>(smem + I::OFF_BAR);

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
  const int TR = tc_tile_rows(G);
  const int row0 = rt * C::TILES * TR;
  const int R = min(C::TILES * TR, q_len * G - row0);
  const bool two = R > TR;
  const int kb = j * chunk;
  int ke = min(kv_len, kb + chunk);
  if (a.causal) ke = min(ke, kv_len - q_len + (row0 + R - 1) / G + 1);
  const int ntiles = ke > kb ? (ke - kb + C::BN - 1) / C::BN : 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(&bars->q_full, 1);
    for (int b = 0; b < I::BUFS; ++b) {
      mbar_init(&bars->kw_full[b], 1);             // one warp widens K, two V
      mbar_init(&bars->vw_full[b], 2);
      mbar_init(&bars->kw_free[b], 1);
      mbar_init(&bars->vw_free[b], 1);
    }
    for (int b = 0; b < I::PARS; ++b) mbar_init(&bars->par_full[b], 1);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&bars->s_full[x], 1);
      mbar_init(&bars->p_full[0][x], 128);
      mbar_init(&bars->p_full[1][x], 128);
      mbar_init(&bars->pv_done[x], 1);
    }
    mbar_init(&bars->drain, 1);
    bars->abort = 0;
    bars->last = 0;
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
  // The register split: 384 x 168 = 128 x 88 + 256 x 208. (200 a softmax thread, the
  // prefill kernel's split, spills three times as much: 714 us where this takes 700;
  // 216 leaves the widening warps too few: 735.)
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;" ::: "memory");
    if (warp == 1) {
      // ---------------------------------------------------------- MMA issuer
      if (lane == 0 && ntiles > 0) {
        constexpr uint32_t idesc_s = mma_idesc(C::BM, C::BN, false, Elem<F16>::kTcFormat);
        constexpr uint32_t idesc_o = mma_idesc(C::BM, D, true, Elem<true>::kTcFormat);
        constexpr int kStep = C::KV_TILE >> 4;
        const uint64_t qdesc[2] = {smem_desc_sw128(smem_u32(smem + C::OFF_Q), 16, 1024),
                                   smem_desc_sw128(smem_u32(smem + C::OFF_Q + C::Q_TILE), 16, 1024)};
        const uint64_t kdesc0 = smem_desc_sw128(smem_u32(smem + I::OFF_KW), 16, 1024);
        const uint64_t vdesc0 = smem_desc_sw128(smem_u32(smem + I::OFF_VW), C::KV_HALF, 1024);
        auto issue_s = [&](int x, int t) {
          tc_fence_after();
          const uint64_t qd = qdesc[x];
          const uint64_t kd = kdesc0 + static_cast<uint32_t>((t & 1) * kStep);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = ((kk >> 2) * C::Q_HALF + (kk & 3) * 32) >> 4;
            const uint32_t offk = ((kk >> 2) * C::KV_HALF + (kk & 3) * 32) >> 4;
            tc_mma(tmem + x * 128, qd + off, kd + offk, idesc_s, kk > 0);
          }
          tc_commit(&bars->s_full[x]);
        };
        auto issue_pv = [&](int x, int t, int h) {
          tc_fence_after();
          const uint64_t vd = vdesc0 + static_cast<uint32_t>((t & 1) * kStep);
#pragma unroll
          for (int k4 = 0; k4 < C::BN / 32; ++k4) {
            const int kk = h * (C::BN / 32) + k4;
            tc_mma_ts(tmem + C::O_COL + x * D, tmem + x * 128 + kk * 8, vd + ((kk * 16 * 128) >> 4),
                      idesc_o, (t > 0 || kk > 0) ? 1 : 0);
          }
          if (h == 1) tc_commit(&bars->pv_done[x]);
        };
        static_assert(I::BUFS == 2, "buffer t & 1, phase t >> 1");
        bool ok = mbar_wait(&bars->q_full, 0) && mbar_wait(&bars->kw_full[0], 0);
        if (ok) {
          issue_s(0, 0);
          if (two) issue_s(1, 0);
          tc_commit(&bars->kw_free[0]);
        }
        // The order of the prefill kernel: P_A V, S_A(next), P_B V, S_B(next).
        for (int t = 0; ok && t < ntiles; ++t) {
          if (bars->abort) { ok = false; break; }
          const bool more = t + 1 < ntiles;
          if (!(ok = mbar_wait(&bars->p_full[0][0], t & 1))) break;
          if (!(ok = mbar_wait(&bars->vw_full[t & 1], (t >> 1) & 1))) break;
          issue_pv(0, t, 0);
          if (!(ok = mbar_wait(&bars->p_full[1][0], t & 1))) break;
          issue_pv(0, t, 1);
          if (more) {
            if (!(ok = mbar_wait(&bars->kw_full[(t + 1) & 1], ((t + 1) >> 1) & 1))) break;
            issue_s(0, t + 1);
          }
          if (two) {
            if (!(ok = mbar_wait(&bars->p_full[0][1], t & 1))) break;
            issue_pv(1, t, 0);
            if (!(ok = mbar_wait(&bars->p_full[1][1], t & 1))) break;
            issue_pv(1, t, 1);
          }
          tc_commit(&bars->vw_free[t & 1]);
          if (more) {
            if (two) issue_s(1, t + 1);
            tc_commit(&bars->kw_free[(t + 1) & 1]);
          }
        }
        if (!ok) {
          abort_call(a);
          bars->abort = 1;
        }
        tc_commit(&bars->drain);
        mbar_wait(&bars->drain, 0);
      }
    } else if (ntiles > 0) {
      // ---------------------------------------------------------- widening warps
      const int cw = warp == 0 ? 0 : warp - 1;           // 0 .. 2
      if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tmQ);
        const int token0 = q_start + row0 / G;
        mbar_arrive_expect_tx(&bars->q_full, (two ? 2 : 1) * C::HALVES * TR * 128);
        for (int x = 0; x < (two ? 2 : 1); ++x)
          for (int h = 0; h < C::HALVES; ++h)
            tma_load_3d(smem + C::OFF_Q + x * C::Q_TILE + h * C::Q_HALF, &tmQ, &bars->q_full,
                        h * 64, hk * G, token0 + x * (TR / G));
      }
      const int32_t* bt_row = a.bt + static_cast<int64_t>(seg) * a.bt_row_stride;
      uint8_t* ring = smem + I::OFF_RING;
      constexpr int KP = I::SLOTS / 4 * 3;               // pairs: K's ring, V's halves of it
      const bool ok =
          cw == 0 ? widen_tiles<D, F16, false, I::UNITS, KP>(a, pool, bars, smem, ring, bt_row, hk,
                                                              kb, kv_len, ntiles, 0)
                  : widen_tiles<D, F16, true, I::UNITS / 2, KP / 2>(
                        a, pool, bars, smem, ring + (cw + 1) * KP * I::SLOT, bt_row, hk, kb, kv_len,
                        ntiles, (cw - 1) * (I::UNITS / 2));
      cp_async_wait<0>();
      if (!ok) {
        abort_call(a);
        bars->abort = 1;
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;" ::: "memory");
    const int X = (warp - 4) >> 2;
    if (X == 0 || two)
      tc_softmax_tile<Kind>(a, bars, smem, tmem, X, q_start, q_len, kv_len, kb, ke, ntiles, row0, R,
                            hk, nsplit, slot_base, rt, j, 0);
    if (nsplit > 1) {
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
  // After an abort: Q's copy may still be in flight.
  if (threadIdx.x == 0 && bars->abort && ntiles > 0) mbar_wait(&bars->q_full, 0);
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

template <int D, bool F16>
static cudaError_t launch_int4_prompt_d(const CUtensorMap& tmQ, const AttnArgs& a,
                                        const Int4Pools& pool, int items_bound, cudaStream_t st) {
  static std::atomic<bool> configured[kMaxDevices];
  cudaError_t e = opt_in_smem(int4_prompt_kernel<D, F16>, TcI4<D>::SMEM_BYTES, configured);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(items_bound + 1, a.H_kv);   // (one column more: see pdl_enter)
  cfg.blockDim = dim3(TcCfg<D>::THREADS);
  cfg.dynamicSmemBytes = TcI4<D>::SMEM_BYTES;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, int4_prompt_kernel<D, F16>, tmQ, a, pool);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

cudaError_t launch_int4_prompt(const CUtensorMap& tmQ, const AttnArgs& a, const Int4Pools& pool,
                               int items_bound, cudaStream_t st) {
  if (a.D == 128)
    return a.f16 ? launch_int4_prompt_d<128, true>(tmQ, a, pool, items_bound, st)
                 : launch_int4_prompt_d<128, false>(tmQ, a, pool, items_bound, st);
  return a.f16 ? launch_int4_prompt_d<64, true>(tmQ, a, pool, items_bound, st)
               : launch_int4_prompt_d<64, false>(tmQ, a, pool, items_bound, st);
}

}  // namespace pa
