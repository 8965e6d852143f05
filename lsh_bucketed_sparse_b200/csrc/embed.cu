// The token table read in, and its gradient:
//   out_t = scale * W[tok_t]                       (zero row for a token
//                                                   outside [0, V))
//   dW_v  = init_v + scale * sum_{t: tok_t = v} dout_t
//
// Lookup: a copy of 16-byte pieces, bound by memory.
//
// Gradient: the tokens are ordered by id (key_sort.cu), so a table row's sum
// runs over consecutive slots and is written once: the sum's order is fixed
// by the input alone.  Sums are float32 and rounded once.  The work is cut
// over slots, not over table rows, so that frequent tokens cost no more than
// rare ones; runs that cross a cut are joined in their order.
#include "common.cuh"
#include "internal.h"
#include "vec16.cuh"

namespace lsh {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxWindow = 64;  // slots that a group of lanes adds up, 8 at least
constexpr int kMinLanes = 8;    // of a group

// A thread takes kPieces pieces, kThreads apart: its tokens, then its rows are
// under way together.
constexpr int kPieces = 4;
template <typename T, typename I>
__global__ void __launch_bounds__(kThreads)
embed_kernel(const I* __restrict__ tokens, const T* __restrict__ table, T* __restrict__ out,
             long long pieces, int vocab, int d, float scale) {
  using V = Vec16<T>;
  wait_prior_grid();
  const int per_row = d / V::N;
  const PieceBlock at(blockIdx.x, kThreads * kPieces, per_row);
  int col[kPieces];
  I tok[kPieces];
  uint4 v[kPieces];
#pragma unroll
  for (int u = 0; u < kPieces; ++u) {
    long long row;
    at.locate(u * kThreads + threadIdx.x, per_row, &row, &col[u]);
    tok[u] = at.first + u * kThreads + threadIdx.x < pieces ? tokens[row] : (I)-1;
  }
#pragma unroll
  for (int u = 0; u < kPieces; ++u) {
    v[u] = make_uint4(0, 0, 0, 0);
    if (tok[u] >= 0 && tok[u] < (I)vocab)
      v[u] = V::raw(table + (size_t)tok[u] * d + col[u] * V::N);
  }
#pragma unroll
  for (int u = 0; u < kPieces; ++u) {
    const long long p = at.first + u * kThreads + threadIdx.x;
    if (p >= pieces) continue;
    float f[V::N];
    V::unpack(v[u], f);
    if (tok[u] >= 0 && tok[u] < (I)vocab) {
#pragma unroll
      for (int t = 0; t < V::N; ++t) f[t] *= scale;
    }
    V::store(out + p * V::N, f);
  }
}

// out[.. V::N values] = a * scale (+ init).
template <typename T>
__device__ __forceinline__ void put_row(T* out, const float* a, float scale, bool add,
                                        const uint4& old) {
  using V = Vec16<T>;
  float f[V::N];
  V::unpack(old, f);
#pragma unroll
  for (int t = 0; t < V::N; ++t) f[t] = add ? fmaf(a[t], scale, f[t]) : a[t] * scale;
  V::store(out, f);
}

// Blocks [0, slot_blocks * col_blocks): a block takes kThreads / lanes windows
// of `window` consecutive slots and `lanes` 16-byte pieces of every row; a
// group of `lanes` lanes adds up the rows of one window, whose loads depend
// on nothing but the plan in shared memory.  A run inside a window is written
// at once.  Runs that cross windows are joined in shared memory, in order, by
// the block's first group; what crosses blocks goes to part[block][0] (the run
// of the block's first slot) or [1], and the block that completes a run
// (arrived[], counted at its first block) adds its partial sums in order.
// Later blocks: table rows without a token.
//
// Rows under way per thread and resident blocks, measured on 65536 x 1024 bf16
// tokens without and 12287 x 520 float32 tokens with init: 4 rows, 4 blocks
// 54.0 / -, 6 and 4 49.5 us / -, 8 and 3 54.5 us; with init 4 and 4 53.6 us,
// 2 and 5 48.2, 2 and 6 44.7 (bf16 has no registers for a sixth block).
template <typename T, bool kInit>
__global__ void __launch_bounds__(kThreads, !kInit ? 4 : sizeof(T) == 4 ? 6 : 5)
embed_grad_kernel(const int32_t* __restrict__ perm, const int32_t* __restrict__ sorted,
                  const int2* __restrict__ runs, const uint32_t* __restrict__ present,
                  const T* __restrict__ dout, const T* init, T* dtable, float* part,
                  int32_t* arrived, int n, int slot_blocks, int col_blocks, int vocab, int d,
                  int lanes, int window, float scale) {
  using V = Vec16<T>;
  constexpr int kAhead = kInit ? 2 : 6;
  constexpr int max_slots = kThreads / kMinLanes * kMaxWindow;
  __shared__ int32_t keys_mem[max_slots + 2], entry[max_slots];
  __shared__ float sums[2 * kThreads * V::N];
  __shared__ int32_t open_key[2 * (kThreads / kMinLanes)];
  wait_prior_grid();
  if ((int)blockIdx.x >= slot_blocks * col_blocks) {
    const int per_row = d / V::N;
    const PieceBlock at(blockIdx.x - slot_blocks * col_blocks, kThreads * kPieces, per_row);
    bool empty[kPieces];
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      long long v;
      int col;
      at.locate(u * kThreads + threadIdx.x, per_row, &v, &col);
      empty[u] = v < vocab && !(present[v >> 5] >> (v & 31) & 1);
    }
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const long long p = at.first + u * kThreads + threadIdx.x;
      if (!empty[u]) continue;
      uint4 old = make_uint4(0, 0, 0, 0);
      if (kInit) old = V::raw(init + p * V::N);
      *reinterpret_cast<uint4*>(dtable + p * V::N) = old;
    }
    return;
  }
  const int sb = blockIdx.x / col_blocks, cb = blockIdx.x - sb * col_blocks;
  const int groups = kThreads / lanes, grp = threadIdx.x / lanes, lane = threadIdx.x & (lanes - 1);
  const int per_block = groups * window;
  const int b0 = sb * per_block, b1 = min(n, b0 + per_block);
  const int32_t* keys = keys_mem + 1 - b0;  // keys[b0 - 1 .. b1], -1 outside [0, n)
  const int32_t* ent = entry - b0;
  for (int i = threadIdx.x; i < b1 - b0 + 2; i += kThreads) {
    const int s = b0 - 1 + i;
    keys_mem[i] = s >= 0 && s < n ? sorted[s] : -1;
  }
  for (int i = threadIdx.x; i < b1 - b0; i += kThreads) entry[i] = perm[b0 + i];
  if (threadIdx.x < 2 * groups) open_key[threadIdx.x] = -1;
  __syncthreads();
  const int col = (cb * lanes + lane) * V::N;
  const bool live = col < d;
  const int g0 = b0 + grp * window, g1 = min(b1, g0 + window);
  if (g0 < g1) {
    bool open_left = keys[g0 - 1] == keys[g0];
    float a[V::N];
#pragma unroll
    for (int t = 0; t < V::N; ++t) a[t] = 0.f;
    for (int s0 = g0; s0 < g1; s0 += kAhead) {
      uint4 x[kAhead], old[kInit ? kAhead : 1];
      old[0] = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int s = s0 + i;
        const bool on = live && s < g1 && keys[s] < vocab;
        x[i] = make_uint4(0, 0, 0, 0);
        if (on) x[i] = V::raw(dout + (size_t)ent[s] * d + col);
        if constexpr (kInit) {
          if (on && keys[s + 1] != keys[s]) old[i] = V::raw(init + (size_t)keys[s] * d + col);
        }
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int s = s0 + i;
        if (s >= g1) continue;
        const int k = keys[s];
        float f[V::N];
        V::unpack(x[i], f);
#pragma unroll
        for (int t = 0; t < V::N; ++t) a[t] += f[t];
        const bool ends = keys[s + 1] != k;
        if (!ends && s + 1 < g1) continue;
        if (k < vocab && live) {
          if (ends && !open_left) {
            put_row(dtable + (size_t)k * d + col, a, scale, kInit, old[kInit ? i : 0]);
          } else {
            const int slot = 2 * grp + (open_left ? 0 : 1);
            if (lane == 0) open_key[slot] = k;
#pragma unroll
            for (int t = 0; t < V::N; ++t) sums[(slot * V::N + t) * lanes + lane] = a[t];
          }
        }
        open_left = false;
#pragma unroll
        for (int t = 0; t < V::N; ++t) a[t] = 0.f;
      }
    }
  }
  __syncthreads();
  if (grp != 0) return;
  const unsigned mask = (lanes == 32 ? 0u : 1u << lanes) - 1u;  // lanes of the first group
  int cur = -1;
  float a[V::N];
#pragma unroll
  for (int t = 0; t < V::N; ++t) a[t] = 0.f;
  for (int q = 0; q <= 2 * groups; ++q) {
    const int k = q < 2 * groups ? open_key[q] : -1;
    if (q < 2 * groups && k < 0) continue;
    if (k != cur && cur >= 0) {
      // the run of cur is complete as far as this block goes
      const bool left = keys[b0] == cur && keys[b0 - 1] == cur;
      const bool right = keys[b1 - 1] == cur && keys[b1] == cur;
      const size_t row = (size_t)cur * d + col;
      bool write = !left && !right;
      if (!write) {
        float* to = part + ((size_t)sb * 2 + (keys[b0] == cur ? 0 : 1)) * d + col;
        if (live) {
#pragma unroll
          for (int t = 0; t < V::N; t += 4)
            *reinterpret_cast<float4*>(to + t) = make_float4(a[t], a[t + 1], a[t + 2], a[t + 3]);
        }
        const int2 r = runs[cur];
        const int first = r.x / per_block, count = (r.y - 1) / per_block - first + 1;
        __threadfence();
        __syncwarp(mask);
        int before = 0;
        if (lane == 0) before = atomicAdd(&arrived[first * col_blocks + cb], 1);
        before = __shfl_sync(mask, before, 0);
        if (before == count - 1) {
          __threadfence();
          write = true;
          const bool shared = r.x > first * per_block;  // its first block begins with another run
#pragma unroll
          for (int t = 0; t < V::N; ++t) a[t] = 0.f;
          if (live) {
#pragma unroll 4
            for (int c = 0; c < count; ++c) {
              const float* from = part + ((size_t)(first + c) * 2 + (c == 0 && shared)) * d + col;
#pragma unroll
              for (int t = 0; t < V::N; t += 4) {
                const float4 v = __ldcg(reinterpret_cast<const float4*>(from + t));
                a[t] += v.x; a[t + 1] += v.y; a[t + 2] += v.z; a[t + 3] += v.w;
              }
            }
          }
        }
      }
      if (write && live)
        put_row(dtable + row, a, scale, kInit,
                kInit ? V::raw(init + row) : make_uint4(0, 0, 0, 0));
#pragma unroll
      for (int t = 0; t < V::N; ++t) a[t] = 0.f;
    }
    cur = k;
    if (k >= 0) {
#pragma unroll
      for (int t = 0; t < V::N; ++t) a[t] += sums[(q * V::N + t) * lanes + lane];
    }
  }
}

// How the gradient's blocks cut slots and columns.  Long windows leave fewer
// runs to join, short ones more blocks: the longest that gives every SM two
// (65536 x 1024 bf16 tokens: windows of 64 41.9 us, 32 49.7, 16 60.3; 12287 x
// 520 float32 ones with init: 57.6, 44.2, 44.4).
struct Cut {
  int lanes, window, slot_blocks, col_blocks;
};

Cut cut_of(const TableProblem& p) {
  const int pieces = (int)(p.d * p.elem() / 16);
  Cut c;
  c.lanes = lanes_of_row(pieces);
  if (c.lanes < kMinLanes) c.lanes = kMinLanes;
  c.col_blocks = (pieces + c.lanes - 1) / c.lanes;
  for (c.window = kMaxWindow;; c.window /= 2) {
    const int slots = kThreads / c.lanes * c.window;
    c.slot_blocks = (int)((p.rows + slots - 1) / slots);
    if (c.window == 8 || (long long)c.slot_blocks * c.col_blocks >= 2 * sm_count()) return c;
  }
}

template <typename T>
cudaError_t grad_t(const TableProblem& p, const int32_t* perm, const int32_t* sorted,
                   const int2* runs, const uint32_t* present, const void* dout, const void* init,
                   void* dtable, float* part, int32_t* arrived, const Cut& c, cudaStream_t st) {
  // rows without a token: nothing to do where the gradient is added in place
  const long long pieces = init == dtable ? 0 : (long long)p.vocab * (p.d / Vec16<T>::N);
  const long long blocks = (long long)c.slot_blocks * c.col_blocks +
                           (pieces + kThreads * kPieces - 1) / (kThreads * kPieces);
  cudaError_t e = launch_dependent(init ? embed_grad_kernel<T, true> : embed_grad_kernel<T, false>,
                                   dim3((unsigned)blocks), dim3(kThreads), 0, st, perm, sorted,
                                   runs, present, static_cast<const T*>(dout),
                                   static_cast<const T*>(init), static_cast<T*>(dtable), part,
                                   arrived, (int)p.rows,
                                   c.slot_blocks, c.col_blocks, p.vocab, p.d, c.lanes, c.window,
                                   p.scale);
  if (e) return e;
  note_launch();
  return cudaSuccess;
}

// dtable = init, or zeros (no tokens at all).
template <typename T>
__global__ void __launch_bounds__(kThreads)
embed_grad_none_kernel(const T* init, T* dtable, long long pieces) {
  using V = Vec16<T>;
  wait_prior_grid();
  const long long p = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (p >= pieces) return;
  float f[V::N];
#pragma unroll
  for (int t = 0; t < V::N; ++t) f[t] = 0.f;
  if (init) V::load(init + p * V::N, f);
  V::store(dtable + p * V::N, f);
}

template <typename T>
cudaError_t none_t(const TableProblem& p, const void* init, void* dtable, cudaStream_t st) {
  const long long pieces = (long long)p.vocab * p.d / Vec16<T>::N;
  cudaError_t e = launch_dependent(
      embed_grad_none_kernel<T>, dim3((unsigned)((pieces + kThreads - 1) / kThreads)),
      dim3(kThreads), 0, st, static_cast<const T*>(init), static_cast<T*>(dtable), pieces);
  if (e) return e;
  note_launch();
  return cudaSuccess;
}

template <typename T, typename I>
cudaError_t embed_t(const TableProblem& p, const void* tokens, const void* table, void* out,
                    cudaStream_t st) {
  const long long pieces = p.rows * (p.d / Vec16<T>::N);
  const long long blocks = (pieces + kThreads * kPieces - 1) / (kThreads * kPieces);
  cudaError_t e = launch_dependent(
      embed_kernel<T, I>, dim3((unsigned)blocks), dim3(kThreads), 0, st,
      static_cast<const I*>(tokens), static_cast<const T*>(table), static_cast<T*>(out),
      pieces, p.vocab, p.d, p.scale);
  if (e) return e;
  note_launch();
  return cudaSuccess;
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

struct Scratch {
  size_t perm, sorted, runs, present, part, arrived, sort, total;
  int n_arrived;  // counters, none where one block takes all slots
};

Scratch scratch_layout(const TableProblem& p) {
  const size_t n = (size_t)p.rows;
  const Cut c = cut_of(p);
  const bool joins = c.slot_blocks > 1;
  Scratch s;
  size_t off = 0;
  s.n_arrived = joins ? c.slot_blocks * c.col_blocks : 0;
  s.perm = off;    off += align256(n * sizeof(int32_t));
  s.sorted = off;  off += align256(n * sizeof(int32_t));
  s.runs = off;    off += align256((size_t)p.vocab * sizeof(int2));
  s.present = off; off += align256((size_t)(p.vocab + 31) / 32 * sizeof(uint32_t));
  s.part = off;    off += joins ? align256((size_t)c.slot_blocks * 2 * p.d * sizeof(float)) : 0;
  s.arrived = off; off += align256((size_t)s.n_arrived * sizeof(int32_t));
  s.sort = off;    off += key_sort_scratch_bytes(p.rows, p.vocab);
  s.total = off;
  return s;
}

}  // namespace

cudaError_t launch_embed(const TableProblem& p, const void* tokens, const void* table, void* out,
                         cudaStream_t st) {
  if (p.rows == 0) return cudaSuccess;
  if (p.bf16)
    return p.idx64 ? embed_t<__nv_bfloat16, int64_t>(p, tokens, table, out, st)
                   : embed_t<__nv_bfloat16, int32_t>(p, tokens, table, out, st);
  return p.idx64 ? embed_t<float, int64_t>(p, tokens, table, out, st)
                 : embed_t<float, int32_t>(p, tokens, table, out, st);
}

size_t embed_backward_workspace_bytes(const TableProblem& p) {
  return p.rows ? scratch_layout(p).total : 0;
}

cudaError_t launch_embed_backward(const TableProblem& p, const void* tokens, const void* dout,
                                  const void* init, void* dtable, void* workspace,
                                  cudaStream_t st) {
  if (p.rows == 0) {
    if (init == dtable) return cudaSuccess;
    return p.bf16 ? none_t<__nv_bfloat16>(p, init, dtable, st) : none_t<float>(p, init, dtable, st);
  }
  const Scratch s = scratch_layout(p);
  char* base = static_cast<char*>(workspace);
  int32_t* perm = reinterpret_cast<int32_t*>(base + s.perm);
  int32_t* sorted = reinterpret_cast<int32_t*>(base + s.sorted);
  int2* runs = reinterpret_cast<int2*>(base + s.runs);
  uint32_t* present = reinterpret_cast<uint32_t*>(base + s.present);
  float* part = reinterpret_cast<float*>(base + s.part);
  int32_t* arrived = reinterpret_cast<int32_t*>(base + s.arrived);
  KeyOrder o = {};
  o.perm = perm;
  o.sorted = sorted;
  o.runs = runs;
  o.present = present;
  o.zeros = arrived;
  o.n_zeros = s.n_arrived;
  cudaError_t e = launch_key_sort(p.rows, p.vocab, tokens, p.idx64, o, base + s.sort, st);
  if (e) return e;
  const Cut c = cut_of(p);
  return p.bf16 ? grad_t<__nv_bfloat16>(p, perm, sorted, runs, present, dout, init, dtable, part,
                                        arrived, c, st)
                : grad_t<float>(p, perm, sorted, runs, present, dout, init, dtable, part,
                                arrived, c, st);
}

}  // namespace lsh
