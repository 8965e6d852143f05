// Stable order of n integer keys (token ids, expert ids) by value: slot s of
// `perm` holds the entry that comes s-th by (key, entry).  Keys outside
// [0, K) count as key K: their entries come last, in their order.
//
// The key K included, keys have nbits = bits(K) bits.  Up to kOneDigitBits
// they are one digit and one stable counting pass orders them; above that
// the low and the high half of the bits are two digits, one pass each.  A
// pass cuts the entries into tiles:
//   count    one CTA per tile: its entries per digit value;
//   scan     one CTA: per digit value the exclusive sum over the tiles, then
//            the first slot of every value (their exclusive sum); up to
//            kFusedTiles tiles each CTA of the scatter does it for itself, and
//            with one tile there is nothing to count before either;
//   scatter  one CTA per tile, each warp a contiguous part of it: entries of
//            equal digit in a warp are ranked by their lane, in the tile by
//            their warp, so equal digits keep their order without atomics
//            on slots.
#include "common.cuh"
#include "internal.h"

namespace lsh {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kScanThreads = 1024;
constexpr int kOneDigitBits = 10;
constexpr int kMaxBins = 1 << 11;
constexpr int kFusedTiles = 64;
constexpr int kSmallPer = 4, kLargePer = 8;  // entries per thread

struct Plan {
  int bits, lo, hi;  // hi == 0: one digit of `lo` = `bits` bits
  int per, tiles;    // entries per thread, tiles of kThreads * per entries
  int bins_lo, bins_hi;
};

Plan make_plan(long long n, int K) {
  Plan p;
  p.bits = 32 - __builtin_clz((unsigned)K);  // K >= 1
  if (p.bits <= kOneDigitBits) {
    p.lo = p.bits;
    p.hi = 0;
    p.bins_lo = K + 1;
    p.bins_hi = 0;
  } else {
    p.lo = (p.bits + 1) / 2;
    p.hi = p.bits - p.lo;
    p.bins_lo = 1 << p.lo;
    p.bins_hi = (K >> p.lo) + 1;
  }
  // one tile while one holds them all, small tiles while the scatter's CTAs can
  // add up their counts themselves (both passes and the runs of 12287 tokens
  // over 50021 words: 17.1 us in tiles of 1024, 21.5 of 2048; 65536 tokens over
  // 32768: 22.0 and 22.3)
  const int small = kThreads * kSmallPer, large = kThreads * kLargePer;
  p.per = n > large && n <= (long long)small * kFusedTiles ? kSmallPer : kLargePer;
  p.tiles = (int)((n + kThreads * p.per - 1) / (kThreads * p.per));
  return p;
}

// The digit of entry e: of the caller's keys in the first pass, of the
// already cleaned keys of the first pass's order in the second.
template <typename I>
struct RawKeys {
  const I* keys;
  int K;
  __device__ int key(int e) const {
    const I k = keys[e];
    return k >= 0 && k < (I)K ? (int)k : K;
  }
  __device__ int entry(int e) const { return e; }
};

// Key 0 where the entry's own key lies in [0, range), 1 outside.
template <typename I>
struct InRange {
  const I* keys;
  int range;
  __device__ int key(int e) const {
    const I k = keys[e];
    return k >= 0 && k < (I)range ? 0 : 1;
  }
  __device__ int entry(int e) const { return e; }
};

struct OrderedKeys {
  const int32_t* keys;
  const int32_t* entries;
  __device__ int key(int e) const { return keys[e]; }
  __device__ int entry(int e) const { return entries[e]; }
};

template <typename S, int kPer>
__global__ void __launch_bounds__(kThreads)
key_count_kernel(const S src, int32_t* __restrict__ cnt, int2* __restrict__ runs, int n_runs,
                 int n, int bins, int shift, int mask) {
  extern __shared__ int32_t hist[];
  for (int b = threadIdx.x; b < bins; b += kThreads) hist[b] = 0;
  wait_prior_grid();
  __syncthreads();
  const int beg = blockIdx.x * (kThreads * kPer);
  int dg[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = beg + i * kThreads + threadIdx.x;
    dg[i] = e < n ? (src.key(e) >> shift) & mask : -1;
  }
  // runs start empty; the kernel after the sort fills in those that exist
  for (int v = blockIdx.x * kThreads + threadIdx.x; v < n_runs; v += gridDim.x * kThreads)
    runs[v] = make_int2(0, 0);
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (dg[i] >= 0) atomicAdd(&hist[dg[i]], 1);
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += kThreads) cnt[(size_t)blockIdx.x * bins + b] = hist[b];
}

// Exclusive scan of a[0..n) (shared memory) by a block of kBlock threads.
template <int kBlock>
__device__ void block_scan(int32_t* a, int n) {
  constexpr int kBlockWarps = kBlock / 32;
  __shared__ int32_t warp_tot[kBlockWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (n + kBlock - 1) / kBlock;
  const int lo = min(n, tid * per), hi = min(n, lo + per);
  int32_t local = 0;
  for (int t = lo; t < hi; ++t) local += a[t];
  int32_t incl = local;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) warp_tot[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    const int32_t w = lane < kBlockWarps ? warp_tot[lane] : 0;
    int32_t wi = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t y = __shfl_up_sync(0xffffffffu, wi, o);
      if (lane >= o) wi += y;
    }
    if (lane < kBlockWarps) warp_tot[lane] = wi - w;
  }
  __syncthreads();
  int32_t run = warp_tot[warp] + incl - local;
  for (int t = lo; t < hi; ++t) {
    const int32_t x = a[t];
    a[t] = run;
    run += x;
  }
  __syncthreads();
}

// cnt[t][b] -> slots of digit b taken before tile t; base[b] -> first slot of
// digit b (also to `offsets` when the digit is the whole key).
__global__ void __launch_bounds__(kScanThreads)
key_scan_kernel(int32_t* __restrict__ cnt, int32_t* __restrict__ base_out,
                int32_t* __restrict__ offsets, int bins, int tiles) {
  extern __shared__ int32_t base[];
  constexpr int kAhead = 16;  // tiles loaded before any is used
  wait_prior_grid();
  for (int b = threadIdx.x; b < bins; b += kScanThreads) {
    int32_t run = 0;
    for (int t0 = 0; t0 < tiles; t0 += kAhead) {
      int32_t x[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        x[k] = t0 + k < tiles ? cnt[(size_t)(t0 + k) * bins + b] : 0;
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (t0 + k < tiles) cnt[(size_t)(t0 + k) * bins + b] = run;
        run += x[k];
      }
    }
    base[b] = run;
  }
  __syncthreads();
  block_scan<kScanThreads>(base, bins);
  for (int b = threadIdx.x; b < bins; b += kScanThreads) {
    base_out[b] = base[b];
    if (offsets) offsets[b] = base[b];
  }
}

// perm / undo / sorted: any may be NULL.  sorted[s] is the whole key in slot s.
// kScanned: cnt and base come from the scan kernel.  Otherwise cnt holds the
// tiles' plain counts (not read when there is one tile) and every CTA adds up
// for itself what stands before it.
template <typename S, int kPer, bool kScanned>
__global__ void __launch_bounds__(kThreads)
key_scatter_kernel(const S src, const int32_t* __restrict__ cnt, const int32_t* __restrict__ base,
                   int32_t* __restrict__ perm, int32_t* __restrict__ undo,
                   int32_t* __restrict__ sorted, int32_t* __restrict__ offsets,
                   int2* __restrict__ runs, int n_runs, int n, int tiles, int bins, int shift,
                   int mask) {
  extern __shared__ int32_t off[];  // [kWarps][bins], then without kScanned first[bins], before[bins]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int32_t* mine = off + (size_t)warp * bins;
  for (int b = lane; b < bins; b += 32) mine[b] = 0;
  wait_prior_grid();
  const int beg = (blockIdx.x * kWarps + warp) * (32 * kPer);
  int key[kPer], entry[kPer];
  unsigned peers[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = beg + 32 * i + lane;
    key[i] = e < n ? src.key(e) : -1;
    entry[i] = e < n ? src.entry(e) : 0;
  }
  // (with one tile there was no count kernel to empty the runs)
  for (int v = blockIdx.x * kThreads + threadIdx.x; v < n_runs; v += gridDim.x * kThreads)
    runs[v] = make_int2(0, 0);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const bool valid = key[i] >= 0;
    const int dg = (key[i] >> shift) & mask;
    const unsigned m = __match_any_sync(0xffffffffu, valid ? dg : -1);
    peers[i] = m;
    if (valid && lane == 31 - __clz(m)) mine[dg] += __popc(m);
    __syncwarp();
  }
  __syncthreads();
  int32_t* first = off + (size_t)kWarps * bins;
  int32_t* before = first + bins;
  if constexpr (!kScanned) {
    constexpr int kAhead = 16;  // tiles loaded before any is used
    for (int b = threadIdx.x; b < bins; b += kThreads) {
      int32_t pre = 0, all = 0;
      if (tiles == 1) {
#pragma unroll
        for (int w = 0; w < kWarps; ++w) all += off[(size_t)w * bins + b];
      } else {
        for (int t0 = 0; t0 < tiles; t0 += kAhead) {
          int32_t x[kAhead];
#pragma unroll
          for (int k = 0; k < kAhead; ++k)
            x[k] = t0 + k < tiles ? cnt[(size_t)(t0 + k) * bins + b] : 0;
#pragma unroll
          for (int k = 0; k < kAhead; ++k) {
            if (t0 + k < (int)blockIdx.x) pre += x[k];
            all += x[k];
          }
        }
      }
      first[b] = all;
      before[b] = pre;
    }
    __syncthreads();
    block_scan<kThreads>(first, bins);
    if (offsets && blockIdx.x == 0)
      for (int b = threadIdx.x; b < bins; b += kThreads) offsets[b] = first[b];
  }
  const int32_t* c = cnt + (size_t)blockIdx.x * bins;
  for (int b = threadIdx.x; b < bins; b += kThreads) {
    int32_t run = kScanned ? base[b] + c[b] : first[b] + before[b];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const int32_t x = off[(size_t)w * bins + b];
      off[(size_t)w * bins + b] = run;
      run += x;
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const bool valid = key[i] >= 0;
    const int dg = (key[i] >> shift) & mask;
    int slot = 0;
    if (valid) slot = mine[dg] + __popc(peers[i] & ((1u << lane) - 1u));
    __syncwarp();
    if (valid) {
      if (perm) perm[slot] = entry[i];
      if (undo) undo[entry[i]] = slot;
      if (sorted) sorted[slot] = key[i];
      if (lane == 31 - __clz(peers[i])) mine[dg] += __popc(peers[i]);
    }
    __syncwarp();
  }
}

// runs[v] = the slots [x, y) that hold key v, where there are any; zeros[0,
// n_zeros) = 0 for the kernel after (n_zeros <= n).
__global__ void __launch_bounds__(kThreads)
key_runs_kernel(const int32_t* __restrict__ sorted, int2* __restrict__ runs,
                int32_t* __restrict__ zeros, int n_zeros, int n, int K) {
  wait_prior_grid();
  const int s = blockIdx.x * kThreads + threadIdx.x;
  if (s >= n) return;
  if (s < n_zeros) zeros[s] = 0;
  const int k = sorted[s];
  if (k >= K) return;
  if (s == 0 || sorted[s - 1] != k) runs[k].x = s;
  if (s == n - 1 || sorted[s + 1] != k) runs[k].y = s + 1;
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// Counts per tile, first slots, and for two digits the first pass's order.
struct Scratch {
  size_t cnt, base, keys, entries, total;
};

Scratch scratch_layout(long long n, const Plan& p) {
  const int bins = p.bins_lo > p.bins_hi ? p.bins_lo : p.bins_hi;
  Scratch s;
  size_t off = 0;
  s.cnt = off;  off += p.tiles > 1 ? align256((size_t)p.tiles * bins * sizeof(int32_t)) : 0;
  s.base = off; off += p.tiles > kFusedTiles ? align256((size_t)bins * sizeof(int32_t)) : 0;
  s.keys = off; off += p.hi ? align256((size_t)n * sizeof(int32_t)) : 0;
  s.entries = off; off += p.hi ? align256((size_t)n * sizeof(int32_t)) : 0;
  s.total = off;
  return s;
}

template <typename S, int kPer>
cudaError_t one_pass_per(const S& src, int32_t* cnt, int32_t* base, int32_t* offsets, int32_t* perm,
                     int32_t* undo, int32_t* sorted, int2* runs, int n_runs, int n, int tiles,
                     int bins, int bits, int shift, cudaStream_t st) {
  const int mask = (1 << bits) - 1;
  const size_t row = (size_t)bins * sizeof(int32_t);
  const bool fused = tiles <= kFusedTiles;
  cudaError_t e;
  if (tiles > 1) {
    if ((e = launch_dependent(key_count_kernel<S, kPer>, dim3(tiles), dim3(kThreads), row, st, src, cnt,
                              runs, n_runs, n, bins, shift, mask)))
      return e;
    note_launch();
    n_runs = 0;
  }
  if (!fused) {
    if ((e = launch_dependent(key_scan_kernel, dim3(1), dim3(kScanThreads), row, st, cnt, base,
                              offsets, bins, tiles)))
      return e;
    note_launch();
  }
  auto kernel = fused ? key_scatter_kernel<S, kPer, false> : key_scatter_kernel<S, kPer, true>;
  const size_t smem = (kWarps + (fused ? 2 : 0)) * row;
  if (smem > 48 * 1024 &&
      (e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)))
    return e;
  if ((e = launch_dependent(kernel, dim3(tiles), dim3(kThreads), smem, st, src,
                            static_cast<const int32_t*>(cnt), static_cast<const int32_t*>(base),
                            perm, undo, sorted, offsets, runs, n_runs, n, tiles, bins, shift, mask)))
    return e;
  note_launch();
  return cudaSuccess;
}

template <typename S>
cudaError_t one_pass(const Plan& p, const S& src, int32_t* cnt, int32_t* base, int32_t* offsets,
                     int32_t* perm, int32_t* undo, int32_t* sorted, int2* runs, int n_runs, int n,
                     int bins, int bits, int shift, cudaStream_t st) {
  return p.per == kSmallPer
             ? one_pass_per<S, kSmallPer>(src, cnt, base, offsets, perm, undo, sorted, runs, n_runs,
                                          n, p.tiles, bins, bits, shift, st)
             : one_pass_per<S, kLargePer>(src, cnt, base, offsets, perm, undo, sorted, runs, n_runs,
                                          n, p.tiles, bins, bits, shift, st);
}

}  // namespace

size_t key_sort_scratch_bytes(long long n, int K) {
  return scratch_layout(n, make_plan(n, K)).total;
}

cudaError_t launch_key_sort(long long n_, int K, const void* keys, bool keys64, int32_t* perm,
                            int32_t* undo, int32_t* offsets, int32_t* sorted, int2* runs,
                            int32_t* zeros, int n_zeros, void* scratch, cudaStream_t st) {
  const Plan p = make_plan(n_, K);
  if (p.bins_lo > kMaxBins || p.bins_hi > kMaxBins || n_ < 1) return cudaErrorInvalidValue;
  if (offsets && p.hi) return cudaErrorInvalidValue;
  const int n = (int)n_;
  const Scratch s = scratch_layout(n_, p);
  char* base = static_cast<char*>(scratch);
  int32_t* cnt = reinterpret_cast<int32_t*>(base + s.cnt);
  int32_t* first = reinterpret_cast<int32_t*>(base + s.base);
  int32_t* k1 = reinterpret_cast<int32_t*>(base + s.keys);
  int32_t* e1 = reinterpret_cast<int32_t*>(base + s.entries);
  const int n_runs = runs ? K : 0;
  const RawKeys<int64_t> r64{static_cast<const int64_t*>(keys), K};
  const RawKeys<int32_t> r32{static_cast<const int32_t*>(keys), K};
  int32_t* to_perm = p.hi ? e1 : perm;
  int32_t* to_undo = p.hi ? nullptr : undo;
  int32_t* to_sorted = p.hi ? k1 : sorted;
  cudaError_t e = keys64 ? one_pass(p, r64, cnt, first, offsets, to_perm, to_undo, to_sorted,
                                    runs, n_runs, n, p.bins_lo, p.lo, 0, st)
                         : one_pass(p, r32, cnt, first, offsets, to_perm, to_undo, to_sorted,
                                    runs, n_runs, n, p.bins_lo, p.lo, 0, st);
  if (e) return e;
  if (p.hi) {
    const OrderedKeys ord{k1, e1};
    if ((e = one_pass(p, ord, cnt, first, nullptr, perm, undo, sorted, nullptr, 0, n, p.bins_hi, p.hi,
                      p.lo, st)))
      return e;
  }
  if (runs) {
    if ((e = launch_dependent(key_runs_kernel, dim3((n + kThreads - 1) / kThreads),
                              dim3(kThreads), 0, st, static_cast<const int32_t*>(sorted), runs,
                              zeros, n_zeros, n, K)))
      return e;
    note_launch();
  }
  return cudaSuccess;
}

cudaError_t launch_row_order(long long n, int range, const void* keys, bool keys64, int32_t* perm,
                             int32_t* undo, int32_t* offsets, void* scratch, cudaStream_t st) {
  const Plan p = make_plan(n, 1);
  const Scratch s = scratch_layout(n, p);
  char* base = static_cast<char*>(scratch);
  int32_t* cnt = reinterpret_cast<int32_t*>(base + s.cnt);
  int32_t* first = reinterpret_cast<int32_t*>(base + s.base);
  const InRange<int64_t> r64{static_cast<const int64_t*>(keys), range};
  const InRange<int32_t> r32{static_cast<const int32_t*>(keys), range};
  return keys64 ? one_pass(p, r64, cnt, first, offsets, perm, undo, nullptr, nullptr, 0, (int)n,
                           p.bins_lo, p.lo, 0, st)
                : one_pass(p, r32, cnt, first, offsets, perm, undo, nullptr, nullptr, 0, (int)n,
                           p.bins_lo, p.lo, 0, st);
}

}  // namespace lsh
