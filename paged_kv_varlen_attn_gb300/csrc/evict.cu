// Eviction: for every sequence longer than its budget, each KV head keeps its
// first keys, its most recent keys and the heaviest of the rest by
// accumulated attention weight, and the kept rows of K, V and the weights are
// moved together at the front of the sequence's pages, in order.
//
// Two kernels: the selection writes the kept indices; the move carries them
// out. Neither waits for another block.
#include <cuda_runtime.h>

#include <atomic>

#include "device_common.cuh"

namespace pa {

// ---------------------------------------------------------------------------
// Selection. One block per (KV head, sequence). The weights of the candidate
// keys [first, kv - recent) become 32-bit keys whose unsigned order is the
// weights' order (NaN as -inf, -0 as +0) and stay in shared memory if they
// fit (else every pass reads them again). A radix selection from the top
// digit (kRadixBits at a time) finds the key of the last kept candidate and
// how many candidates equal to it are kept; those are the ones of lowest
// index. A last pass writes the kept indices in ascending order: each warp
// owns a contiguous run of candidates, counts its kept ones by ballots, and
// one scan over the warps gives its first output position.
// ---------------------------------------------------------------------------
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kRadixBits = 11;
constexpr int kRadixBins = 1 << kRadixBits;

__device__ __forceinline__ uint32_t weight_key(float w) {
  if (!(w == w)) w = -INFINITY;
  const uint32_t b = __float_as_uint(w + 0.f);   // -0 + 0 = +0
  return (b >> 31) ? ~b : b | 0x80000000u;
}

__global__ void __launch_bounds__(kSelThreads)
evict_select_kernel(const __grid_constant__ EvictArgs a, int staged_max) {
  extern __shared__ uint32_t staged[];   // [staged_max]
  __shared__ int hist[kRadixBins];
  __shared__ int warp_sum[kSelWarps][2];
  __shared__ int found[2];               // digit of this pass, candidates above it
  const int s = blockIdx.x, h = blockIdx.y;
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
    const int lp = j / a.bs;
    const int page = __ldg(bt + lp);
    if (page < 0 || page >= a.num_blocks) {
      bad |= PA_DEV_BAD_PAGE;
      return weight_key(-INFINITY);
    }
    return weight_key(__ldg(a.weights + page * a.weights_stride + h * a.bs + (j - lp * a.bs)));
  };
  const bool in_smem = n <= staged_max;
  if (in_smem)
    for (int i = tid; i < n; i += kSelThreads) staged[i] = load_key(i);
  auto key_of = [&](int i) -> uint32_t { return in_smem ? staged[i] : load_key(i); };

  // Radix selection of the need-th largest key (none for need = 0).
  uint32_t prefix = 0;      // the digits found so far
  int left = need;          // kept candidates that match the prefix
  if (need > 0) {
    int shift = 32;
    while (shift > 0) {
      const int bits = min(kRadixBits, shift);
      const uint32_t matched = shift == 32 ? 0u : ~0u << shift;
      shift -= bits;
      const int bins = 1 << bits;
      for (int i = tid; i < bins; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (int i = tid; i < n; i += kSelThreads) {
        const uint32_t k = key_of(i);
        if ((k & matched) == prefix) atomicAdd(&hist[(k >> shift) & (bins - 1)], 1);
      }
      __syncthreads();
      // Bins from the top: thread t takes the bins of ranks [t*per, t*per+per).
      constexpr int per = kRadixBins / kSelThreads;
      int sum = 0;
#pragma unroll
      for (int k = 0; k < per; ++k) {
        const int b = bins - 1 - (tid * per + k);
        sum += b >= 0 ? hist[b] : 0;
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
      for (int w = 0; w < warp; ++w) above += warp_sum[w][0];
      if (above < left && left <= above + sum) {   // exactly one thread
#pragma unroll
        for (int k = 0; k < per; ++k) {
          const int b = bins - 1 - (tid * per + k);
          const int c = b >= 0 ? hist[b] : 0;
          if (above < left && left <= above + c) {
            found[0] = b;
            found[1] = above;
          }
          above += c;
        }
      }
      __syncthreads();
      prefix |= static_cast<uint32_t>(found[0]) << shift;
      left -= found[1];
    }
  }
  // prefix is now the key of the last kept candidate; `left` of its equals
  // are kept, the ones of lowest index.
  const int run = (n + kSelThreads - 1) / kSelThreads * 32;   // candidates per warp
  const int r0 = min(n, warp * run), r1 = min(n, r0 + run);
  int gt = 0, eq = 0;
  if (need > 0) {
    for (int i = r0 + lane; i < r1; i += 32) {
      const uint32_t k = key_of(i);
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
  if (need > 0) {
    const uint32_t below = (1u << lane) - 1u;
    for (int i0 = r0; i0 < r1; i0 += 32) {
      const int i = i0 + lane;
      const uint32_t k = i < r1 ? key_of(i) : 0u;
      const uint32_t mg = __ballot_sync(0xffffffffu, i < r1 && k > prefix);
      const uint32_t me = __ballot_sync(0xffffffffu, i < r1 && k == prefix);
      const int ge = gt0 + __popc(mg & below), ee = eq0 + __popc(me & below);
      const bool take = ((mg >> lane) & 1u) || (((me >> lane) & 1u) && ee < left);
      if (take) kept[a.first + ge + min(ee, left)] = a.first + i;
      gt0 += __popc(mg);
      eq0 += __popc(me);
    }
  }
  for (int d = tid; d < a.first; d += kSelThreads) kept[d] = d;
  for (int d = tid; d < a.recent; d += kSelThreads) kept[a.budget - a.recent + d] = kv - a.recent + d;
  if (bad) flag_status(a.status, bad);
}

// ---------------------------------------------------------------------------
// Move, in place. Row d of (sequence, KV head) becomes row kept[d]; kept
// ascends, so kept[d] >= d and a row is never overwritten before a row
// further on has been read, as long as the rows are taken in order: a block
// reads one chunk of rows into registers, waits for all of its threads, then
// writes the chunk. (Rows of later chunks are at or past their own, unwritten
// destinations.) Columns are independent of each other, so the rows are cut
// into slices of kSliceBytes -- two sectors -- of K and of V, and one block
// moves one slice of one head; the weights are one more slice, of 4 bytes.
// The rows that stay where they are (kept[d] = d, a prefix) are skipped.
// ---------------------------------------------------------------------------
constexpr int kMoveThreads = 256;
constexpr int kSliceBytes = 64;
constexpr int kMoveUnroll = 4;

template <typename T>
__device__ __forceinline__ void move_rows(const EvictArgs& a, const int32_t* kept,
                                          const int32_t* bt, uint8_t* base, int64_t page_stride,
                                          int row_stride, int lanes, int& bad) {
  // Thread's column and first row; `lanes` threads of T cover a row's slice.
  const int col = threadIdx.x % lanes, r0 = threadIdx.x / lanes;
  const int rows = kMoveThreads / lanes;               // rows per pass
  const int chunk = rows * kMoveUnroll;
  auto address = [&](int j) -> uint8_t* {
    const int lp = j / a.bs;
    const int page = __ldg(bt + lp);
    if (page < 0 || page >= a.num_blocks) {
      bad |= PA_DEV_BAD_PAGE;
      return nullptr;
    }
    return base + page * page_stride + static_cast<int64_t>(j - lp * a.bs) * row_stride +
           col * static_cast<int>(sizeof(T));
  };
  for (int d0 = 0; d0 < a.budget; d0 += chunk) {
    T v[kMoveUnroll];
    bool moved[kMoveUnroll];
    int src[kMoveUnroll];
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const int d = d0 + u * rows + r0;
      src[u] = d < a.budget ? __ldg(kept + d) : -1;
    }
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const int d = d0 + u * rows + r0;
      moved[u] = src[u] > d;                           // -1: no such row; d: in place
      if (moved[u]) {
        const uint8_t* p = address(src[u]);
        moved[u] = p != nullptr;
        if (p) v[u] = *reinterpret_cast<const T*>(p);
      }
    }
    __syncthreads();   // every thread has read its rows of this chunk
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const int d = d0 + u * rows + r0;
      if (moved[u]) {
        uint8_t* p = address(d);
        if (p) *reinterpret_cast<T*>(p) = v[u];
      }
    }
  }
}

__global__ void __launch_bounds__(kMoveThreads)
evict_move_kernel(const __grid_constant__ EvictArgs a) {
  // The slices of a sequence's rows are neighbouring blocks, so that the two
  // halves of a 128-byte line are wanted at about the same time.
  const int slices = a.row_bytes / kSliceBytes;
  const int s = blockIdx.x / (2 * slices + 1), b = blockIdx.x - s * (2 * slices + 1);
  const int h = blockIdx.y;
  const int32_t* kept = a.kept + (static_cast<int64_t>(s) * a.H_kv + h) * a.budget;
  const int32_t* bt = a.bt + static_cast<int64_t>(s) * a.bt_stride;
  int bad = 0;
  if (b < 2 * slices) {
    uint8_t* pool = b < slices ? a.kc : a.vc;
    const int sl = b < slices ? b : b - slices;
    move_rows<uint4>(a, kept, bt, pool + static_cast<int64_t>(h) * a.row_bytes + sl * kSliceBytes,
                     a.block_stride_bytes, a.H_kv * a.row_bytes, kSliceBytes / 16, bad);
  } else {
    move_rows<float>(a, kept, bt,
                     reinterpret_cast<uint8_t*>(a.weights + static_cast<int64_t>(h) * a.bs),
                     a.weights_stride * 4, 4, 1, bad);
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

cudaError_t launch_evict(const EvictArgs& a, int num_seqs, cudaStream_t st) {
  if (num_seqs == 0) return cudaSuccess;
  // Candidates kept in shared memory: what the host bound asks for, up to
  // 48k keys (192 KB, one block per SM).
  constexpr int kStageCap = 48 * 1024;
  static std::atomic<bool> configured[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool known = dev >= 0 && dev < kMaxDevices;
  if (!known || !configured[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kStageCap * 4);
    if (e != cudaSuccess) return e;
    if (known) configured[dev].store(true, std::memory_order_release);
  }
  const int bound = a.max_k < a.kv_len_cap ? a.max_k : a.kv_len_cap;
  const int staged = bound < kStageCap ? bound : kStageCap;
  evict_select_kernel<<<dim3(num_seqs, a.H_kv), kSelThreads, static_cast<size_t>(staged) * 4, st>>>(
      a, staged);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int slices = a.row_bytes / kSliceBytes;
  evict_move_kernel<<<dim3(num_seqs * (2 * slices + 1), a.H_kv), kMoveThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace pa
