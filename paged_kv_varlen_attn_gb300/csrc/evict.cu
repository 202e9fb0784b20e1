// Eviction: for every sequence longer than its budget, each KV head keeps its
// first keys, its most recent keys and the heaviest of the rest by
// accumulated attention weight, and the kept rows of K, V and the weights are
// moved together at the front of the sequence's pages, in order.
//
// Two kernels: the selection writes the kept indices; the move carries them
// out. Neither waits for another block.
#include <cuda_runtime.h>

#include "device_common.cuh"

namespace pa {

// ---------------------------------------------------------------------------
// Selection. One block per (KV head, sequence), or a cluster whose blocks share
// its candidates, add up each other's histograms and write one after another's
// kept indices (all read from the others' shared memory). The weights of the candidate
// keys [first, kv - recent) become 32-bit keys whose unsigned order is the
// weights' order (NaN as -inf, -0 as +0) and stay in shared memory if they
// fit (else every pass reads them again). A radix selection from the top
// digit (kRadixBits at a time; the first digit is counted while the keys are
// read) finds the smallest key prefix whose candidates are kept, and how many
// of the candidates with that prefix: it stops at the digit where that is all
// of them, or after the last digit, where they are equal and the ones of
// lowest index are kept. A last pass writes the kept indices in ascending
// order: each warp owns a contiguous run of candidates, counts its kept ones
// by ballots, and one scan over the warps gives its first output position.
// ---------------------------------------------------------------------------
constexpr int kSelParts = 4;             // blocks of a cluster at most
constexpr int kSelUnroll = 4;            // groups of four weights on their way per thread

// Logical page of key j (a shift for the usual page sizes).
__device__ __forceinline__ int page_of(const EvictArgs& a, int j) {
  return a.bs_shift >= 0 ? j >> a.bs_shift : j / a.bs;
}

__device__ __forceinline__ uint32_t weight_key(float w) {
  if (!(w == w)) w = -INFINITY;
  const uint32_t b = __float_as_uint(w + 0.f);   // -0 + 0 = +0
  return (b >> 31) ? ~b : b | 0x80000000u;
}

template <int kSelThreads, int kRadixBits, bool CLUSTER>
__global__ void __launch_bounds__(kSelThreads, 1)
evict_select_kernel(const __grid_constant__ EvictArgs a, int staged_max, int parts) {
  constexpr int kSelWarps = kSelThreads / 32, kRadixBins = 1 << kRadixBits;
  static_assert(kRadixBins % kSelThreads == 0, "whole bins per thread");
  extern __shared__ __align__(16) uint32_t staged[];   // [staged_max]
  // One histogram, or one per pass where other blocks read them.
  constexpr int kHists = CLUSTER ? (32 + kRadixBits - 1) / kRadixBits : 1;
  __shared__ int hist[kHists][kRadixBins];
  __shared__ int warp_sum[kSelWarps][2], block_sum[2];
  __shared__ int found[3];               // digit of this pass, candidates above it, in it
  const int part = CLUSTER ? static_cast<int>(cluster_rank()) : 0;
  const int s = CLUSTER ? blockIdx.x / parts : blockIdx.x, h = blockIdx.y;
  // What this block has written to its shared memory is seen by its threads,
  // and by the cluster's.
  auto sync = [&]() {
    if constexpr (CLUSTER) {
      cluster_arrive();
      cluster_wait();
    } else {
      __syncthreads();
    }
  };
  auto remote = [&](const int* at, int rank) {
    return __float_as_int(load_remote(reinterpret_cast<const float*>(at), rank));
  };
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int kv = __ldg(a.seqused_k + s);
  int bad = 0;
  if (kv < 0 || kv > a.max_k) bad = PA_DEV_BAD_SEQLEN;
  if (kv < 0) kv = 0;
  if (kv > a.kv_len_cap) {
    bad = PA_DEV_BAD_SEQLEN;
    kv = a.kv_len_cap;
  }
  int32_t* kept = a.kept + (static_cast<int64_t>(s) * a.H_kv + h) * a.budget;
  if (kv <= a.budget) {   // nothing to evict
    if (part > 0) return;
    if (bad && h == 0 && tid == 0) flag_status(a.status, bad);
    for (int d = tid; d < a.budget; d += kSelThreads) kept[d] = d < kv ? d : -1;
    return;
  }
  const int32_t* bt = a.bt + static_cast<int64_t>(s) * a.bt_stride;
  const int n = kv - a.first - a.recent;                // candidates
  const int need = a.budget - a.first - a.recent;       // of them kept; 0 <= need < n
  // Key of candidate i. Its page and the row in it follow from its index; a
  // page outside the pool holds nothing worth keeping.
  auto load_key = [&](int i) -> uint32_t {
    const int j = a.first + i;
    const int lp = page_of(a, j);
    const int page = __ldg(bt + lp);
    if (page < 0 || page >= a.num_blocks) {
      bad |= PA_DEV_BAD_PAGE;
      return weight_key(-INFINITY);
    }
    return weight_key(__ldg(a.weights + page * a.weights_stride + h * a.bs + (j - lp * a.bs)));
  };
  // The keys are read in groups of four (rows of one page, 16 bytes), from the
  // group that holds the first candidate on.
  const int off = a.first & 3, all = (off + n + 3) >> 2;
  const int base = static_cast<int>(static_cast<long long>(all) * part / parts);
  const int groups = static_cast<int>(static_cast<long long>(all) * (part + 1) / parts);
  const int i_lo = max(0, 4 * base - off), i_hi = min(n, 4 * groups - off);   // this block's
  const bool in_smem = 4 * (groups - base) <= staged_max;
  for (int i = tid; i < kHists * kRadixBins; i += kSelThreads) hist[0][i] = 0;
  __syncthreads();
  for (int g0 = base + tid; g0 < groups; g0 += kSelThreads * kSelUnroll) {
    int page[kSelUnroll], row[kSelUnroll];
#pragma unroll
    for (int u = 0; u < kSelUnroll; ++u) {
      const int j = a.first - off + 4 * (g0 + u * kSelThreads);
      const int lp = page_of(a, j);
      row[u] = j - lp * a.bs;
      page[u] = g0 + u * kSelThreads < groups ? __ldg(bt + lp) : 0;
    }
    uint4 k[kSelUnroll];
#pragma unroll
    for (int u = 0; u < kSelUnroll; ++u) {
      k[u] = make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u);   // -inf
      if (g0 + u * kSelThreads >= groups) continue;
      if (page[u] < 0 || page[u] >= a.num_blocks)
        bad |= PA_DEV_BAD_PAGE;
      else
        k[u] = __ldg(reinterpret_cast<const uint4*>(a.weights + page[u] * a.weights_stride +
                                                    h * a.bs + row[u]));
    }
#pragma unroll
    for (int u = 0; u < kSelUnroll; ++u) {
      const int gi = g0 + u * kSelThreads;
      if (gi >= groups) break;
      uint32_t x[4] = {k[u].x, k[u].y, k[u].z, k[u].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = weight_key(__uint_as_float(x[e]));
        const int i = 4 * gi + e - off;
        if (i >= 0 && i < n) atomicAdd(&hist[0][x[e] >> (32 - kRadixBits)], 1);
      }
      if (in_smem) reinterpret_cast<uint4*>(staged)[gi - base] = make_uint4(x[0], x[1], x[2], x[3]);
    }
  }
  sync();
  auto key_of = [&](int i) -> uint32_t {
    return in_smem ? staged[off + i - 4 * base] : load_key(i);
  };

  // Radix selection of the need-th largest key (none for need = 0).
  uint32_t prefix = 0, matched = 0;   // the digits found so far, and their bits
  int left = need;                    // kept candidates that match the prefix
  if (need > 0) {
    int shift = 32 - kRadixBits, bins = kRadixBins, pass = 0;
    while (true) {
      // Bins from the top: thread t takes the bins of ranks [t*per, t*per+per).
      constexpr int per = kRadixBins / kSelThreads;
      int count[per], sum = 0;
#pragma unroll
      for (int k = 0; k < per; ++k) {
        const int b = bins - 1 - (tid * per + k);
        count[k] = 0;
        if (b >= 0) {
          if constexpr (CLUSTER) {
            int c[kSelParts];                              // all on their way at once
#pragma unroll
            for (int r = 0; r < kSelParts; ++r) c[r] = r < parts ? remote(&hist[pass][b], r) : 0;
#pragma unroll
            for (int r = 0; r < kSelParts; ++r) count[k] += c[r];
          } else {
            count[k] = hist[0][b];
          }
        }
        sum += count[k];
      }
      int incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      if (lane == 31) warp_sum[warp][0] = incl;
      __syncthreads();
      int above = incl - sum;
#pragma unroll
      for (int w = 0; w < kSelWarps; ++w) above += w < warp ? warp_sum[w][0] : 0;
      if (above < left && left <= above + sum) {   // exactly one thread
#pragma unroll
        for (int k = 0; k < per; ++k) {
          if (above < left && left <= above + count[k]) {
            found[0] = bins - 1 - (tid * per + k);
            found[1] = above;
            found[2] = count[k];
          }
          above += count[k];
        }
      }
      __syncthreads();
      prefix |= static_cast<uint32_t>(found[0]) << shift;
      matched |= static_cast<uint32_t>(bins - 1) << shift;
      left -= found[1];
      if (shift == 0 || left == found[2]) break;
      const int bits = min(kRadixBits, shift);
      shift -= bits;
      bins = 1 << bits;
      if constexpr (CLUSTER) {
        ++pass;
      } else {
        for (int i = tid; i < bins; i += kSelThreads) hist[0][i] = 0;
        __syncthreads();
      }
      for (int i = i_lo + tid; i < i_hi; i += kSelThreads) {
        const uint32_t k = key_of(i);
        if ((k & matched) == prefix) atomicAdd(&hist[pass][(k >> shift) & (bins - 1)], 1);
      }
      sync();
    }
  }
  // Kept: the candidates above the prefix, and the first `left` that match it.
  const int run = (i_hi - i_lo + kSelThreads - 1) / kSelThreads * 32;   // candidates per warp
  const int r0 = min(i_hi, i_lo + warp * run), r1 = min(i_hi, r0 + run);
  int gt = 0, eq = 0;
  if (need > 0) {
    for (int i = r0 + lane; i < r1; i += 32) {
      const uint32_t k = key_of(i) & matched;
      gt += k > prefix;
      eq += k == prefix;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      gt += __shfl_xor_sync(0xffffffffu, gt, o);
      eq += __shfl_xor_sync(0xffffffffu, eq, o);
    }
  }
  __syncthreads();   // warp_sum's last readers are done
  if (lane == 0) {
    warp_sum[warp][0] = gt;
    warp_sum[warp][1] = eq;
  }
  __syncthreads();
  int gt0 = 0, eq0 = 0;
  for (int w = 0; w < warp; ++w) {
    gt0 += warp_sum[w][0];
    eq0 += warp_sum[w][1];
  }
  if constexpr (CLUSTER) {
    // The blocks before this one come first.
    if (tid == kSelThreads - 1) {
      block_sum[0] = gt0 + warp_sum[warp][0];
      block_sum[1] = eq0 + warp_sum[warp][1];
    }
    sync();
#pragma unroll
    for (int r = 0; r < kSelParts - 1; ++r) {
      gt0 += r < part ? remote(&block_sum[0], r) : 0;
      eq0 += r < part ? remote(&block_sum[1], r) : 0;
    }
  }
  if (need > 0) {
    const uint32_t below = (1u << lane) - 1u;
    for (int i0 = r0; i0 < r1; i0 += 32) {
      const int i = i0 + lane;
      const uint32_t k = i < r1 ? key_of(i) & matched : 0u;
      const uint32_t mg = __ballot_sync(0xffffffffu, i < r1 && k > prefix);
      const uint32_t me = __ballot_sync(0xffffffffu, i < r1 && k == prefix);
      const int ge = gt0 + __popc(mg & below), ee = eq0 + __popc(me & below);
      const bool take = ((mg >> lane) & 1u) || (((me >> lane) & 1u) && ee < left);
      if (take) kept[a.first + ge + min(ee, left)] = a.first + i;
      gt0 += __popc(mg);
      eq0 += __popc(me);
    }
  }
  if (part == 0) {
    for (int d = tid; d < a.first; d += kSelThreads) kept[d] = d;
    for (int d = tid; d < a.recent; d += kSelThreads)
      kept[a.budget - a.recent + d] = kv - a.recent + d;
  }
  if (bad) flag_status(a.status, bad);
  if constexpr (CLUSTER) sync();   // nobody leaves while its sums are read
}

// ---------------------------------------------------------------------------
// Move, in place. Row d of (sequence, KV head) becomes row kept[d]; kept
// ascends, so kept[d] >= d and a row is never overwritten before a row
// further on has been read, as long as the rows are taken in order: a block
// reads one chunk of rows into registers, waits for all of its threads, then
// writes the chunk. (Rows of later chunks are at or past their own, unwritten
// destinations.) Columns are independent of each other, so the rows are cut
// into slices of 16 * LANES bytes and a block moves one slice of K and of V --
// the same page and row in both pools, one address computation -- of one
// head; the weights are one more slice, of 4 bytes. While a chunk's rows are
// on their way the next chunk's indices and pages are looked up. Rows that
// stay where they are (kept[d] = d, a prefix) are skipped.
// Bound by HBM where many sequences are cut (selection and move 61.5 us for 64
// sequences of 900-1400 keys and 8 heads of 128 to 1024: 380 MB, 91% of the
// measured copy rate), by the passes of the selection and the chain of
// dependent chunks where few are (4 sequences of 14,000 keys to 2048: 25.2 us,
// 40%).
// ---------------------------------------------------------------------------
constexpr int kMoveUnroll = 4;

// Page-relative place of key j: page id (or -1 for a page outside the pool)
// and row in it.
__device__ __forceinline__ int place_of(const EvictArgs& a, const int32_t* bt, int j, int& row,
                                        int& bad) {
  const int lp = page_of(a, j);
  const int page = __ldg(bt + lp);
  row = j - lp * a.bs;
  if (page < 0 || page >= a.num_blocks) {
    bad |= PA_DEV_BAD_PAGE;
    return -1;
  }
  return page;
}

// copy(dst page, dst row, src page, src row) in two steps around the barrier:
// `load(u, page, row)` before, `store(u, page, row)` after.
template <int ROWS, typename Load, typename Store>
__device__ __forceinline__ void move_rows(const EvictArgs& a, const int32_t* kept,
                                          const int32_t* bt, int r0, int& bad, Load load,
                                          Store store) {
  constexpr int U = kMoveUnroll, CHUNK = ROWS * U;
  int page[U], row[U];                                 // of the sources; page < 0: not moved
  auto look_up = [&](int d0) {
    int src[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int d = d0 + u * ROWS + r0;
      src[u] = d < a.budget ? __ldg(kept + d) : -1;    // -1: no such row
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      page[u] = -1;
      if (src[u] > d0 + u * ROWS + r0) page[u] = place_of(a, bt, src[u], row[u], bad);
    }
  };
  look_up(0);
  for (int d0 = 0; d0 < a.budget; d0 += CHUNK) {
    int dpage[U], drow[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (page[u] >= 0) load(u, page[u], row[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      dpage[u] = -1;
      if (page[u] >= 0) dpage[u] = place_of(a, bt, d0 + u * ROWS + r0, drow[u], bad);
    }
    if (d0 + CHUNK < a.budget) look_up(d0 + CHUNK);
    __syncthreads();   // every thread has read its rows of this chunk
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (dpage[u] >= 0) store(u, dpage[u], drow[u]);
  }
}

template <int LANES, int kMoveThreads>
__global__ void __launch_bounds__(kMoveThreads)
evict_move_kernel(const __grid_constant__ EvictArgs a) {
  // The slices of a sequence's rows are neighbouring blocks, so that the
  // parts of a 128-byte line are wanted at about the same time.
  const int slices = a.row_bytes / (16 * LANES);
  const int s = blockIdx.x / (slices + 1), b = blockIdx.x - s * (slices + 1);
  const int h = blockIdx.y;
  const int32_t* kept = a.kept + (static_cast<int64_t>(s) * a.H_kv + h) * a.budget;
  const int32_t* bt = a.bt + static_cast<int64_t>(s) * a.bt_stride;
  int bad = 0;
  if (b < slices) {
    const int64_t col = static_cast<int64_t>(h) * a.row_bytes + b * (16 * LANES) +
                        threadIdx.x % LANES * 16;
    const int64_t row_stride = static_cast<int64_t>(a.H_kv) * a.row_bytes;
    uint4 k[kMoveUnroll], v[kMoveUnroll];
    move_rows<kMoveThreads / LANES>(
        a, kept, bt, threadIdx.x / LANES, bad,
        [&](int u, int page, int row) {
          const int64_t at = page * a.block_stride_bytes + row * row_stride + col;
          k[u] = *reinterpret_cast<const uint4*>(a.kc + at);
          v[u] = *reinterpret_cast<const uint4*>(a.vc + at);
        },
        [&](int u, int page, int row) {
          const int64_t at = page * a.block_stride_bytes + row * row_stride + col;
          *reinterpret_cast<uint4*>(a.kc + at) = k[u];
          *reinterpret_cast<uint4*>(a.vc + at) = v[u];
        });
  } else {
    float w[kMoveUnroll];
    move_rows<kMoveThreads>(
        a, kept, bt, threadIdx.x, bad,
        [&](int u, int page, int row) { w[u] = a.weights[page * a.weights_stride + h * a.bs + row]; },
        [&](int u, int page, int row) { a.weights[page * a.weights_stride + h * a.bs + row] = w[u]; });
    // The new length: the indices are a prefix of kept (the same for every
    // head). Written here, not in the selection, so that it may replace the
    // lengths that the selection reads.
    if (h == 0) {
      int n = 0;
      for (int d = threadIdx.x; d < a.budget; d += kMoveThreads) n += __ldg(kept + d) >= 0;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
      __shared__ int total[kMoveThreads / 32];
      if ((threadIdx.x & 31) == 0) total[threadIdx.x >> 5] = n;
      __syncthreads();
      if (threadIdx.x == 0) {
        n = 0;
        for (int w = 0; w < kMoveThreads / 32; ++w) n += total[w];
        a.new_lens[s] = n;
      }
    }
  }
  if (bad) flag_status(a.status, bad);
}

constexpr int kLongKeys = 4096;

template <int LANES, int THREADS>
static cudaError_t launch_move(const EvictArgs& a, int num_seqs, cudaStream_t st) {
  const int slices = a.row_bytes / (16 * LANES);
  evict_move_kernel<LANES, THREADS>
      <<<dim3(num_seqs * (slices + 1), a.H_kv), THREADS, 0, st>>>(a);
  return cudaGetLastError();
}

// Candidates kept in shared memory: what the host bound asks for, up to 48k
// keys (192 KB, one block per SM).
constexpr int kStageCap = 48 * 1024;

template <int THREADS, int BITS, bool CLUSTER>
static cudaError_t launch_select(const EvictArgs& a, int num_seqs, int bound, int parts,
                                 cudaStream_t st) {
  auto kernel = evict_select_kernel<THREADS, BITS, CLUSTER>;
  static std::atomic<bool> configured[kMaxDevices];
  cudaError_t e = opt_in_smem(kernel, kStageCap * 4, configured);
  if (e != cudaSuccess) return e;
  // A block's share of the groups of four, one more at either end.
  const int share = (bound / parts + 11) & ~3;
  const int staged = share < kStageCap ? share : kStageCap;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(num_seqs * parts, a.H_kv);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = static_cast<size_t>(staged) * 4;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = parts;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CLUSTER ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, kernel, a, staged, parts);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

cudaError_t launch_evict(const EvictArgs& a, int num_seqs, cudaStream_t st, int sms) {
  if (num_seqs == 0) return cudaSuccess;
  const int bound = a.max_k < a.kv_len_cap ? a.max_k : a.kv_len_cap;
  // Short sequences: many small blocks, digits of as many bins as threads, so
  // that a pass costs little beside the candidates (512 threads and 11 bits:
  // 66.1 us instead of 64.5 in all for 512 pairs to 1024 keys). Long ones:
  // clusters of such blocks while there are fewer blocks than SMs (32 pairs
  // from 14,000 keys to 2048: 25.4 us, 24.9 with 8 blocks, whose first, uncached
  // call is slower; 27.9 with one block of 1024 threads and 11 bits; 28 with 9
  // bits, 94 with 11, by the remote reads), one large block each from there on
  // (half the threads: 30.7).
  const long long units = static_cast<long long>(num_seqs) * a.H_kv;
  int parts = 1;
  while (parts < kSelParts && units * parts < sms && bound > kLongKeys) parts *= 2;
  cudaError_t e = bound <= kLongKeys ? launch_select<256, 8, false>(a, num_seqs, bound, 1, st)
                  : parts == 1       ? launch_select<1024, 11, false>(a, num_seqs, bound, 1, st)
                                     : launch_select<256, 8, true>(a, num_seqs, bound, parts, st);
  if (e != cudaSuccess) return e;
  // Rows of one head move in order, chunk by chunk: where there are fewer
  // (sequence, head) pairs than SMs, narrower slices and larger blocks make longer chunks
  // and more blocks (32 pairs to 2048 keys: 25.2 us with 32-byte slices and 256
  // threads, 28.2 with 128; 64-byte slices 32.6, 16-byte ones 41). Where there
  // are many, smaller blocks leave less of an SM waiting at a chunk's end (512
  // pairs to 1024 keys: 61.5 us with 64-byte slices and 128 threads, 64.4 with
  // 256, 63.5 with 64; 32-byte slices 73). As a programmatic dependent of the
  // selection the move was no faster.
  return units >= sms ? launch_move<4, 128>(a, num_seqs, st)
                      : launch_move<2, 256>(a, num_seqs, st);
}

}  // namespace pa
