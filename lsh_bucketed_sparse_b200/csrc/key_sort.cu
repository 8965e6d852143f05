// Stable order of n integer keys (token ids, expert ids) by value: slot s of
// `perm` holds the entry that comes s-th by (key, entry).  Keys outside
// [0, K) count as key K: their entries come last, in their order.
//
// The key K included, keys have nbits = bits(K) bits.  Up to kOneDigitBits
// they are one digit and one stable counting pass orders them; above that
// the low and the high half of the bits are two digits, one pass each.  In a
// pass every warp takes a contiguous part of the entries; entries of equal
// digit are ranked by their lane in a warp's 32, by their warp's counts in the
// block and by the blocks' counts before it, so equal digits keep their order
// without atomics on slots.
//
// Up to kClusterEntries entries one kernel does all passes: a cluster of up
// to 8 CTAs, which exchange their counts through distributed shared memory,
// with a cluster barrier where the passes meet.  It is latency that counts
// there (the order and the runs of 12287 tokens over 50021 words: 15.6 us in one
// launch; in the six of below 21.5 us.  65536 tokens over 32768 words would take
// 46 us on eight SMs, below they take 22).  More entries take tiles of kTile and
// up to three kernels a pass:
//   count    one CTA per tile: its entries per digit value;
//   scan     one CTA: per digit value the exclusive sum over the tiles, then
//            the first slot of every value (their exclusive sum); up to
//            kFusedTiles tiles each CTA of the scatter does it for itself;
//   scatter  one CTA per tile.
#include "common.cuh"
#include "internal.h"
#include "sm100.cuh"

namespace lsh {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kPer = 8;                       // entries per thread
constexpr int kTile = kThreads * kPer;
constexpr int kScanThreads = 1024;
// Tiles whose counts every CTA of the scatter adds up for itself; above it one
// CTA does so for all, in a launch of its own.  Order by 8 / 256 / 1023 experts, us,
// for itself and in its own launch: 64 tiles 14 / 18 / 25 and 16 / 21 / 23, 128 tiles
// 18 / 20 / 31 and 18 / 23 / 29, 512 tiles 41 / 78 / 158 and 33 / 49 / 72.
constexpr int kFusedTiles = 64;
constexpr int kOneDigitBits = 10;
constexpr int kMaxBins = 1 << 11;

constexpr int kClusterWarps = 16;
constexpr int kClusterThreads = kClusterWarps * 32;
constexpr int kMaxCluster = 8;                // CTAs of a portable cluster
constexpr int kClusterPer = 4;                // entries per thread
constexpr int kClusterEntries = kMaxCluster * kClusterThreads * kClusterPer;

struct Plan {
  int bits, lo, hi;  // hi == 0: one digit of `lo` = `bits` bits
  int tiles;         // 0: one cluster
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
  p.tiles = n <= kClusterEntries ? 0 : (int)((n + kTile - 1) / kTile);
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

// The first pass's order.  (Read past L1: in the cluster kernel other CTAs
// have just written it.)
struct OrderedKeys {
  const int32_t* keys;
  const int32_t* entries;
  __device__ int key(int e) const { return __ldcg(keys + e); }
  __device__ int entry(int e) const { return __ldcg(entries + e); }
};

// Marks slot s of the finished order where a run of its key begins or ends.
__device__ __forceinline__ void mark_run(const int32_t* sorted, int s, int n, int K, int2* runs,
                                         uint32_t* present) {
  const int k = __ldcg(sorted + s);
  if (k >= K) return;
  if (s == 0 || __ldcg(sorted + s - 1) != k) {
    runs[k].x = s;
    atomicOr(&present[k >> 5], 1u << (k & 31));
  }
  if (s == n - 1 || __ldcg(sorted + s + 1) != k) runs[k].y = s + 1;
}

// Counts a warp's entries per digit in mine[] (in order); peers[i]: the lanes
// of row i that hold the same digit.
template <int N>
__device__ __forceinline__ void count_warp(const int* key, unsigned* peers, int32_t* mine,
                                           int shift, int mask, int lane) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const bool valid = key[i] >= 0;
    const int dg = (key[i] >> shift) & mask;
    peers[i] = __match_any_sync(0xffffffffu, valid ? dg : -1);
    if (valid && lane == 31 - __clz(peers[i])) mine[dg] += __popc(peers[i]);
    __syncwarp();
  }
}

// Puts a warp's entries into their slots; mine[]: the next slot per digit.
template <int N>
__device__ __forceinline__ void place_warp(const int* key, const int* entry, const unsigned* peers,
                                           int32_t* mine, int shift, int mask, int lane,
                                           int32_t* perm, int32_t* undo, int32_t* sorted) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
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

// ---- one cluster --------------------------------------------------------------------
// perm, undo, sorted: any may be NULL; offsets: NULL or [bins].
template <typename S>
__device__ void cluster_pass(const S& src, int32_t* mem, int n, int bins, int shift, int mask,
                             int32_t* perm, int32_t* undo, int32_t* sorted, int32_t* offsets) {
  int32_t* off = mem;                            // [kClusterWarps][bins]
  int32_t* total = off + kClusterWarps * bins;   // this CTA's counts
  int32_t* first = total + bins;
  int32_t* before = first + bins;
  constexpr int N = kClusterPer;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)sm100::cluster_ctarank(), ctas = gridDim.x;
  int32_t* mine = off + warp * bins;
  for (int b = lane; b < bins; b += 32) mine[b] = 0;
  const int beg = (rank * kClusterWarps + warp) * (32 * N);
  int key[N], entry[N];
  unsigned peers[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = beg + 32 * i + lane;
    key[i] = e < n ? src.key(e) : -1;
    entry[i] = e < n ? src.entry(e) : 0;
  }
  __syncwarp();
  count_warp<N>(key, peers, mine, shift, mask, lane);
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += kClusterThreads) {
    int32_t run = 0;
#pragma unroll
    for (int w = 0; w < kClusterWarps; ++w) {
      const int32_t x = off[w * bins + b];
      off[w * bins + b] = run;
      run += x;
    }
    total[b] = run;
  }
  sm100::cluster_sync();
  for (int b = threadIdx.x; b < bins; b += kClusterThreads) {
    int32_t pre = 0, all = 0, x[kMaxCluster];
#pragma unroll
    for (int q = 0; q < kMaxCluster; ++q)
      asm volatile("ld.shared::cluster.s32 %0, [%1];"
                   : "=r"(x[q])
                   : "r"(sm100::cluster_addr(total + b, q < ctas ? q : 0)));
#pragma unroll
    for (int q = 0; q < kMaxCluster; ++q) {
      if (q < rank) pre += x[q];
      if (q < ctas) all += x[q];
    }
    first[b] = all;
    before[b] = pre;
  }
  __syncthreads();
  block_scan<kClusterThreads>(first, bins);
  if (offsets && rank == 0)
    for (int b = threadIdx.x; b < bins; b += kClusterThreads) offsets[b] = first[b];
  for (int b = threadIdx.x; b < bins; b += kClusterThreads) {
    const int32_t at = first[b] + before[b];
#pragma unroll
    for (int w = 0; w < kClusterWarps; ++w) off[w * bins + b] += at;
  }
  __syncthreads();
  place_warp<N>(key, entry, peers, mine, shift, mask, lane, perm, undo, sorted);
  sm100::cluster_sync();  // what was written is there, the counts have been read
}

// All of an order whose entries one cluster holds.
template <typename S>
__global__ void __launch_bounds__(kClusterThreads)
key_cluster_kernel(const S src, const KeyOrder o, int32_t* k1, int32_t* e1, int n, int K, int lo,
                   int hi, int bins_lo, int bins_hi) {
  extern __shared__ int32_t mem[];
  wait_prior_grid();
  const int id = blockIdx.x * kClusterThreads + threadIdx.x, threads = gridDim.x * kClusterThreads;
  if (o.runs)
    for (int i = id; i < (K + 31) / 32; i += threads) o.present[i] = 0;
  for (int i = id; i < o.n_zeros; i += threads) o.zeros[i] = 0;
  if (hi == 0) {
    cluster_pass(src, mem, n, bins_lo, 0, (1 << lo) - 1, o.perm, o.undo, o.sorted, o.offsets);
  } else {
    cluster_pass(src, mem, n, bins_lo, 0, (1 << lo) - 1, e1, nullptr, k1, nullptr);
    cluster_pass(OrderedKeys{k1, e1}, mem, n, bins_hi, lo, (1 << hi) - 1, o.perm,
                                 o.undo, o.sorted, nullptr);
  }
  if (o.runs)
    for (int s = id; s < n; s += threads) mark_run(o.sorted, s, n, K, o.runs, o.present);
}

// ---- tiles -------------------------------------------------------------------------
template <typename S>
__global__ void __launch_bounds__(kThreads)
key_count_kernel(const S src, int32_t* __restrict__ cnt, uint32_t* __restrict__ present,
                 int n_present, int n, int bins, int shift, int mask) {
  extern __shared__ int32_t hist[];
  for (int b = threadIdx.x; b < bins; b += kThreads) hist[b] = 0;
  wait_prior_grid();
  __syncthreads();
  const int beg = blockIdx.x * kTile;
  int dg[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = beg + i * kThreads + threadIdx.x;
    dg[i] = e < n ? (src.key(e) >> shift) & mask : -1;
  }
  // (the kernel after the sort sets the bits)
  for (int i = blockIdx.x * kThreads + threadIdx.x; i < n_present; i += gridDim.x * kThreads)
    present[i] = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (dg[i] >= 0) atomicAdd(&hist[dg[i]], 1);
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += kThreads) cnt[(size_t)blockIdx.x * bins + b] = hist[b];
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
// tiles' plain counts and every CTA adds up for itself what stands before it.
template <typename S, bool kScanned>
__global__ void __launch_bounds__(kThreads)
key_scatter_kernel(const S src, const int32_t* __restrict__ cnt, const int32_t* __restrict__ base,
                   int32_t* __restrict__ perm, int32_t* __restrict__ undo,
                   int32_t* __restrict__ sorted, int32_t* __restrict__ offsets, int n, int tiles,
                   int bins, int shift, int mask) {
  // [kWarps][bins], then without kScanned first[bins], before[bins]
  extern __shared__ int32_t off[];
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
  __syncwarp();
  count_warp<kPer>(key, peers, mine, shift, mask, lane);
  __syncthreads();
  int32_t* first = off + (size_t)kWarps * bins;
  int32_t* before = first + bins;
  if constexpr (!kScanned) {
    constexpr int kAhead = 16;  // tiles loaded before any is used
    for (int b = threadIdx.x; b < bins; b += kThreads) {
      int32_t pre = 0, all = 0;
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
  place_warp<kPer>(key, entry, peers, mine, shift, mask, lane, perm, undo, sorted);
}

// Runs of the finished order; zeros[0, n_zeros) = 0 for the kernel after.
__global__ void __launch_bounds__(kThreads)
key_runs_kernel(const KeyOrder o, int n, int K) {
  wait_prior_grid();
  const int s = blockIdx.x * kThreads + threadIdx.x;
  for (int i = s; i < o.n_zeros; i += gridDim.x * kThreads) o.zeros[i] = 0;
  if (s < n) mark_run(o.sorted, s, n, K, o.runs, o.present);
}

// ---------------------------------------------------------------- host side
size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// Counts per tile, first slots, and for two digits the first pass's order.
struct Scratch {
  size_t cnt, base, keys, entries, total;
};

Scratch scratch_layout(long long n, const Plan& p) {
  const int bins = p.bins_lo > p.bins_hi ? p.bins_lo : p.bins_hi;
  Scratch s;
  size_t off = 0;
  s.cnt = off;  off += align256((size_t)p.tiles * bins * sizeof(int32_t));
  s.base = off; off += p.tiles > kFusedTiles ? align256((size_t)bins * sizeof(int32_t)) : 0;
  s.keys = off; off += p.hi ? align256((size_t)n * sizeof(int32_t)) : 0;
  s.entries = off; off += p.hi ? align256((size_t)n * sizeof(int32_t)) : 0;
  s.total = off;
  return s;
}

template <typename S>
cudaError_t launch_cluster(const Plan& p, const S& src, const KeyOrder& o, int32_t* k1, int32_t* e1,
                           int n, int K, cudaStream_t st) {
  auto kernel = key_cluster_kernel<S>;
  const int bins = p.bins_lo > p.bins_hi ? p.bins_lo : p.bins_hi;
  const size_t smem = (size_t)(kClusterWarps + 3) * bins * sizeof(int32_t);
  cudaError_t e;
  if (smem > 48 * 1024 &&
      (e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)))
    return e;
  int ctas = 1;
  while (ctas < kMaxCluster && ctas * kClusterThreads * kClusterPer < n) ctas *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kClusterThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, kernel, src, o, k1, e1, n, K, p.lo, p.hi, p.bins_lo, p.bins_hi);
  if (e == cudaSuccess) note_launch();
  return e;
}

template <typename S>
cudaError_t one_pass(const Plan& p, const S& src, int32_t* cnt, int32_t* base, int32_t* offsets,
                     int32_t* perm, int32_t* undo, int32_t* sorted, uint32_t* present,
                     int n_present, int n, int bins, int bits, int shift, cudaStream_t st) {
  const int mask = (1 << bits) - 1;
  const size_t row = (size_t)bins * sizeof(int32_t);
  const bool fused = p.tiles <= kFusedTiles;
  cudaError_t e;
  if ((e = launch_dependent(key_count_kernel<S>, dim3(p.tiles), dim3(kThreads), row, st, src, cnt,
                            present, n_present, n, bins, shift, mask)))
    return e;
  note_launch();
  if (!fused) {
    if ((e = launch_dependent(key_scan_kernel, dim3(1), dim3(kScanThreads), row, st, cnt, base,
                              offsets, bins, p.tiles)))
      return e;
    note_launch();
  }
  auto kernel = fused ? key_scatter_kernel<S, false> : key_scatter_kernel<S, true>;
  const size_t smem = (kWarps + (fused ? 2 : 0)) * row;
  if (smem > 48 * 1024 &&
      (e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)))
    return e;
  if ((e = launch_dependent(kernel, dim3(p.tiles), dim3(kThreads), smem, st, src,
                            static_cast<const int32_t*>(cnt), static_cast<const int32_t*>(base),
                            perm, undo, sorted, offsets, n, p.tiles, bins, shift, mask)))
    return e;
  note_launch();
  return cudaSuccess;
}

template <typename S>
cudaError_t order_keys(const S& src, long long n_, int K, const KeyOrder& o, void* scratch,
                       cudaStream_t st) {
  const Plan p = make_plan(n_, K);
  if (p.bins_lo > kMaxBins || p.bins_hi > kMaxBins || n_ < 1) return cudaErrorInvalidValue;
  if (o.offsets && p.hi) return cudaErrorInvalidValue;
  const int n = (int)n_;
  const Scratch s = scratch_layout(n_, p);
  char* base = static_cast<char*>(scratch);
  int32_t* cnt = reinterpret_cast<int32_t*>(base + s.cnt);
  int32_t* first = reinterpret_cast<int32_t*>(base + s.base);
  int32_t* k1 = reinterpret_cast<int32_t*>(base + s.keys);
  int32_t* e1 = reinterpret_cast<int32_t*>(base + s.entries);
  if (p.tiles == 0) return launch_cluster(p, src, o, k1, e1, n, K, st);
  const int n_present = o.runs ? (K + 31) / 32 : 0;
  cudaError_t e = one_pass(p, src, cnt, first, o.offsets, p.hi ? e1 : o.perm,
                           p.hi ? nullptr : o.undo, p.hi ? k1 : o.sorted, o.present, n_present, n,
                           p.bins_lo, p.lo, 0, st);
  if (e) return e;
  if (p.hi) {
    if ((e = one_pass(p, OrderedKeys{k1, e1}, cnt, first, static_cast<int32_t*>(nullptr), o.perm,
                      o.undo, o.sorted, static_cast<uint32_t*>(nullptr), 0, n, p.bins_hi, p.hi,
                      p.lo, st)))
      return e;
  }
  if (o.runs) {
    if ((e = launch_dependent(key_runs_kernel, dim3((n + kThreads - 1) / kThreads),
                              dim3(kThreads), 0, st, o, n, K)))
      return e;
    note_launch();
  }
  return cudaSuccess;
}

}  // namespace

size_t key_sort_scratch_bytes(long long n, int K) {
  return scratch_layout(n, make_plan(n, K)).total;
}

cudaError_t launch_key_sort(long long n, int K, const void* keys, bool keys64, const KeyOrder& o,
                            void* scratch, cudaStream_t st) {
  return keys64 ? order_keys(RawKeys<int64_t>{static_cast<const int64_t*>(keys), K}, n, K, o,
                             scratch, st)
                : order_keys(RawKeys<int32_t>{static_cast<const int32_t*>(keys), K}, n, K, o,
                             scratch, st);
}

cudaError_t launch_row_order(long long n, int range, const void* keys, bool keys64,
                             const KeyOrder& o, void* scratch, cudaStream_t st) {
  return keys64 ? order_keys(InRange<int64_t>{static_cast<const int64_t*>(keys), range}, n, 1, o,
                             scratch, st)
                : order_keys(InRange<int32_t>{static_cast<const int32_t*>(keys), range}, n, 1, o,
                             scratch, st);
}

}  // namespace lsh
