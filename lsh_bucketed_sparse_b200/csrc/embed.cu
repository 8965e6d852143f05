// The token table read in, and its gradient:
//   out_t = scale * W[tok_t]                       (zero row for a token
//                                                   outside [0, V))
//   dW_v  = init_v + scale * sum_{t: tok_t = v} dout_t
//
// Lookup: a copy of 16-byte pieces, bound by memory.
//
// Gradient: the tokens are ordered by id (key_sort.cu), so a table row's sum
// runs over consecutive slots and is written once, without atomics: the sum's
// order is fixed by the input alone.  Sums are float32 and rounded once.  A
// run of up to kChunk slots is summed by the lanes that own the row.  Longer
// runs (frequent tokens) are cut at multiples of kChunk: one CTA per chunk
// leaves a float32 partial sum, and a second kernel adds a run's partial
// sums in order.
#include "common.cuh"
#include "internal.h"
#include "vec16.cuh"

namespace lsh {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 64;  // longest run summed in one go

template <typename T, typename I>
__global__ void __launch_bounds__(kThreads)
embed_kernel(const I* __restrict__ tokens, const T* __restrict__ table, T* __restrict__ out,
             long long pieces, int vocab, int d, float scale) {
  using V = Vec16<T>;
  wait_prior_grid();
  const int per_row = d / V::N;
  const long long p = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (p >= pieces) return;
  const long long row = p / per_row;
  const int col = (int)(p - row * per_row) * V::N;
  const I tok = tokens[row];
  float f[V::N];
#pragma unroll
  for (int t = 0; t < V::N; ++t) f[t] = 0.f;
  if (tok >= 0 && tok < (I)vocab) {
    V::load(table + (size_t)tok * d + col, f);
#pragma unroll
    for (int t = 0; t < V::N; ++t) f[t] *= scale;
  }
  V::store(out + (size_t)row * d + col, f);
}

__device__ __forceinline__ bool frequent(int2 run) { return run.y - run.x > kChunk; }

// Blocks [0, chunks): the chunk's partial sums of frequent tokens, at most
// two (the run of its first slot -> part[chunk][0], another run that reaches
// past its end -> part[chunk][1]).  Later blocks: one table row per group of
// lanes, for rows that are not frequent.
template <typename T>
__global__ void __launch_bounds__(kThreads)
embed_grad_kernel(const int32_t* __restrict__ perm, const int32_t* __restrict__ sorted,
                  const int2* __restrict__ runs, const T* __restrict__ dout, const T* init,
                  T* dtable, float* __restrict__ part, int n, int chunks, int vocab, int d,
                  int lanes, float scale) {
  using V = Vec16<T>;
  wait_prior_grid();
  if ((int)blockIdx.x < chunks) {
    __shared__ int32_t rows[kChunk];
    const int c0 = blockIdx.x * kChunk, c1 = min(n, c0 + kChunk);
    const int k0 = sorted[c0], k1 = sorted[c1 - 1];
    const int2 r0 = k0 < vocab ? runs[k0] : make_int2(0, 0);
    const int2 r1 = k1 < vocab && k1 != k0 ? runs[k1] : make_int2(0, 0);
    if (!frequent(r0) && !frequent(r1)) return;
    for (int s = c0 + threadIdx.x; s < c1; s += kThreads) rows[s - c0] = perm[s];
    __syncthreads();
    for (int which = 0; which < 2; ++which) {
      const int2 r = which ? r1 : r0;
      if (!frequent(r)) continue;
      const int b = max(r.x, c0) - c0, e = min(r.y, c1) - c0;
      float* to = part + ((size_t)blockIdx.x * 2 + which) * d;
      for (int col = threadIdx.x * 4; col < d; col += kThreads * 4) {
        float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
        for (int s = b; s < e; ++s) {
          const T* x = dout + (size_t)rows[s] * d + col;
#pragma unroll
          for (int t = 0; t < 4; ++t) a[t] += to_f32(x[t]);
        }
        *reinterpret_cast<float4*>(to + col) = make_float4(a[0], a[1], a[2], a[3]);
      }
    }
    return;
  }
  const int per_block = kThreads / lanes;
  const long long v =
      (long long)(blockIdx.x - chunks) * per_block + threadIdx.x / lanes;
  if (v >= vocab) return;
  const int2 r = runs[v];
  if (frequent(r)) return;
  for (int col = (threadIdx.x % lanes) * V::N; col < d; col += lanes * V::N) {
    float a[V::N];
#pragma unroll
    for (int t = 0; t < V::N; ++t) a[t] = 0.f;
#pragma unroll 4
    for (int s = r.x; s < r.y; ++s) {
      float f[V::N];
      V::load(dout + (size_t)perm[s] * d + col, f);
#pragma unroll
      for (int t = 0; t < V::N; ++t) a[t] += f[t];
    }
#pragma unroll
    for (int t = 0; t < V::N; ++t) a[t] *= scale;
    if (init) {
      float f[V::N];
      V::load(init + (size_t)v * d + col, f);
#pragma unroll
      for (int t = 0; t < V::N; ++t) a[t] += f[t];
    }
    V::store(dtable + (size_t)v * d + col, a);
  }
}

// Grid (chunks, columns / kColumns): the CTA of the chunk in which a frequent
// run begins (at most one does: it reaches past the chunk's end) adds the
// run's partial sums, each warp every kSumWarps-th, then the warps' sums in
// order.
constexpr int kColumns = 128, kSumWarps = 8;
template <typename T>
__global__ void __launch_bounds__(kSumWarps * 32)
embed_grad_long_kernel(const int32_t* __restrict__ sorted, const int2* __restrict__ runs,
                       const float* __restrict__ part, const T* init, T* dtable, int n, int vocab,
                       int d, float scale) {
  __shared__ float4 sums[kSumWarps][32];
  wait_prior_grid();
  const int c0 = blockIdx.x * kChunk, c1 = min(n, c0 + kChunk);
  const int v = sorted[c1 - 1];
  if (v >= vocab) return;
  const int2 r = runs[v];
  if (!frequent(r) || r.x < c0) return;
  const int last = (r.y - 1) / kChunk;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col = blockIdx.y * kColumns + lane * 4;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  if (col < d) {
#pragma unroll 4
    for (int c = (int)blockIdx.x + warp; c <= last; c += kSumWarps) {
      const int which = c == (int)blockIdx.x && r.x > c0;
      const float4 x = *reinterpret_cast<const float4*>(part + ((size_t)c * 2 + which) * d + col);
      a.x += x.x; a.y += x.y; a.z += x.z; a.w += x.w;
    }
  }
  sums[warp][lane] = a;
  __syncthreads();
  if (warp != 0 || col >= d) return;
#pragma unroll
  for (int w = 1; w < kSumWarps; ++w) {
    const float4 x = sums[w][lane];
    a.x += x.x; a.y += x.y; a.z += x.z; a.w += x.w;
  }
  const float f[4] = {a.x, a.y, a.z, a.w};
  const size_t at = (size_t)v * d + col;
#pragma unroll
  for (int t = 0; t < 4; ++t)
    dtable[at + t] = from_f32<T>(f[t] * scale + (init ? to_f32(init[at + t]) : 0.f));
}

template <typename T>
cudaError_t grad_t(const TableProblem& p, const int32_t* perm, const int32_t* sorted,
                   const int2* runs, const void* dout, const void* init, void* dtable, float* part,
                   cudaStream_t st) {
  const int chunks = (int)((p.rows + kChunk - 1) / kChunk);
  int lanes = 1;
  while (lanes < 32 && lanes * Vec16<T>::N < p.d) lanes *= 2;
  const long long blocks = chunks + ((long long)p.vocab * lanes + kThreads - 1) / kThreads;
  const T* g = static_cast<const T*>(dout);
  const T* in = static_cast<const T*>(init);
  T* out = static_cast<T*>(dtable);
  cudaError_t e = launch_dependent(embed_grad_kernel<T>, dim3((unsigned)blocks), dim3(kThreads), 0,
                                   st, perm, sorted, runs, g, in, out, part, (int)p.rows, chunks,
                                   p.vocab, p.d, lanes, p.scale);
  if (e) return e;
  note_launch();
  if (p.rows <= kChunk) return cudaSuccess;  // no run is that long
  e = launch_dependent(embed_grad_long_kernel<T>, dim3(chunks, (p.d + kColumns - 1) / kColumns),
                       dim3(kSumWarps * 32), 0, st, sorted, runs, static_cast<const float*>(part),
                       in, out, (int)p.rows, p.vocab, p.d, p.scale);
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
  cudaError_t e = launch_dependent(
      embed_kernel<T, I>, dim3((unsigned)((pieces + kThreads - 1) / kThreads)), dim3(kThreads), 0,
      st, static_cast<const I*>(tokens), static_cast<const T*>(table), static_cast<T*>(out),
      pieces, p.vocab, p.d, p.scale);
  if (e) return e;
  note_launch();
  return cudaSuccess;
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

struct Scratch {
  size_t perm, sorted, runs, part, sort, total;
};

Scratch scratch_layout(const TableProblem& p) {
  const size_t n = (size_t)p.rows;
  Scratch s;
  size_t off = 0;
  s.perm = off;   off += align256(n * sizeof(int32_t));
  s.sorted = off; off += align256(n * sizeof(int32_t));
  s.runs = off;   off += align256((size_t)p.vocab * sizeof(int2));
  s.part = off;
  if (p.rows > kChunk) off += align256((n + kChunk - 1) / kChunk * 2 * p.d * sizeof(float));
  s.sort = off;   off += key_sort_scratch_bytes(p.rows, p.vocab);
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
  float* part = reinterpret_cast<float*>(base + s.part);
  cudaError_t e = launch_key_sort(p.rows, p.vocab, tokens, p.idx64, perm, nullptr, nullptr, sorted,
                                  runs, base + s.sort, st);
  if (e) return e;
  return p.bf16 ? grad_t<__nv_bfloat16>(p, perm, sorted, runs, dout, init, dtable, part, st)
                : grad_t<float>(p, perm, sorted, runs, dout, init, dtable, part, st);
}

}  // namespace lsh
