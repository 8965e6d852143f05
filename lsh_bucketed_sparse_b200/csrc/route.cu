// Tokens moved to their experts and back.  The plan (key_sort.cu) orders the
// entries (t, j) of the router's choice by expert: undo[t, j] is the slot of
// token t's j-th copy, and the slots from offsets[E] on hold dropped entries.
//   gather            xs[undo[t,j]] = x_t          (zero rows for dropped)
//   combine           out_t = sum_j w[t,j] y[undo[t,j]]   (kept j only)
//   gather backward   dx_t = sum_j dxs[undo[t,j]]  (combine without weights)
//   combine backward  dy[undo[t,j]] = w[t,j] dout_t,  dw[t,j] = dout_t . y[undo[t,j]]
// All are bound by memory.  Each runs over tokens, so a token's own row is
// read or written once and whole rows of 16-byte pieces go to or come from
// the slots; sums over j run in the order of j in float32.
#include "common.cuh"
#include "internal.h"
#include "vec16.cuh"

namespace lsh {
namespace {

constexpr int kThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kThreads)
route_gather_kernel(const T* __restrict__ x, const int32_t* __restrict__ undo,
                    const int32_t* __restrict__ kept, T* __restrict__ xs, long long pieces,
                    int entries, int k, int d) {
  wait_prior_grid();
  const int per_row = d / Vec16<T>::N;
  const long long p = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (p >= pieces) return;
  const long long t = p / per_row;
  const int col = (int)(p - t * per_row) * Vec16<T>::N;
  const int n_kept = *kept;
  const uint4 v = Vec16<T>::raw(x + (size_t)t * d + col);
  const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll 4
  for (int j = 0; j < k; ++j) {
    const int s = undo[t * k + j];
    if ((unsigned)s < (unsigned)entries)
      *reinterpret_cast<uint4*>(xs + (size_t)s * d + col) = s < n_kept ? v : zero;
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
route_combine_kernel(const T* __restrict__ y, const float* __restrict__ weights,
                     const int32_t* __restrict__ undo, const int32_t* __restrict__ kept,
                     T* __restrict__ out, long long pieces, int entries, int k, int d) {
  using V = Vec16<T>;
  wait_prior_grid();
  const int per_row = d / V::N;
  const long long p = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (p >= pieces) return;
  const long long t = p / per_row;
  const int col = (int)(p - t * per_row) * V::N;
  const int n_kept = min(*kept, entries);
  float a[V::N];
#pragma unroll
  for (int i = 0; i < V::N; ++i) a[i] = 0.f;
#pragma unroll 4
  for (int j = 0; j < k; ++j) {
    const int s = undo[t * k + j];
    if (s < 0 || s >= n_kept) continue;
    const float w = weights ? weights[t * k + j] : 1.f;
    float f[V::N];
    V::load(y + (size_t)s * d + col, f);
#pragma unroll
    for (int i = 0; i < V::N; ++i) a[i] = fmaf(w, f[i], a[i]);
  }
  V::store(out + (size_t)t * d + col, a);
}

// One warp per token.
template <typename T>
__global__ void __launch_bounds__(kThreads)
route_combine_grad_kernel(const T* __restrict__ dout, const T* __restrict__ y,
                          const float* __restrict__ weights, const int32_t* __restrict__ undo,
                          const int32_t* __restrict__ kept, T* __restrict__ dy,
                          float* __restrict__ dw, long long tokens, int entries, int k, int d) {
  using V = Vec16<T>;
  wait_prior_grid();
  const int lane = threadIdx.x & 31;
  const long long t = ((long long)blockIdx.x * kThreads + threadIdx.x) >> 5;
  if (t >= tokens) return;
  const int n_kept = *kept;
  const T* g = dout + (size_t)t * d;
  for (int j = 0; j < k; ++j) {
    const int s = undo[t * k + j];
    float dot = 0.f;
    if ((unsigned)s < (unsigned)entries) {
      const bool on = s < n_kept;
      const float w = on ? weights[t * k + j] : 0.f;
      for (int col = lane * V::N; col < d; col += 32 * V::N) {
        float r[V::N], f[V::N];
#pragma unroll
        for (int i = 0; i < V::N; ++i) r[i] = 0.f;
        if (on) {
          V::load(g + col, r);
          V::load(y + (size_t)s * d + col, f);
#pragma unroll
          for (int i = 0; i < V::N; ++i) {
            dot = fmaf(r[i], f[i], dot);
            r[i] *= w;
          }
        }
        V::store(dy + (size_t)s * d + col, r);
      }
    }
    dot = warp_sum(dot);
    if (lane == 0) dw[t * k + j] = dot;
  }
}

unsigned blocks_of(long long threads) { return (unsigned)((threads + kThreads - 1) / kThreads); }

template <typename T>
cudaError_t gather_t(const RouteProblem& p, const void* x, const int32_t* undo,
                     const int32_t* kept, void* xs, cudaStream_t st) {
  const long long pieces = p.tokens * (p.d / Vec16<T>::N);
  return launch_dependent(route_gather_kernel<T>, dim3(blocks_of(pieces)), dim3(kThreads), 0, st,
                          static_cast<const T*>(x), undo, kept, static_cast<T*>(xs), pieces,
                          (int)p.entries(), p.k, p.d);
}

template <typename T>
cudaError_t combine_t(const RouteProblem& p, const void* y, const float* weights,
                      const int32_t* undo, const int32_t* kept, void* out, cudaStream_t st) {
  const long long pieces = p.tokens * (p.d / Vec16<T>::N);
  return launch_dependent(route_combine_kernel<T>, dim3(blocks_of(pieces)), dim3(kThreads), 0, st,
                          static_cast<const T*>(y), weights, undo, kept, static_cast<T*>(out),
                          pieces, (int)p.entries(), p.k, p.d);
}

template <typename T>
cudaError_t combine_grad_t(const RouteProblem& p, const void* dout, const void* y,
                           const float* weights, const int32_t* undo, const int32_t* kept,
                           void* dy, float* dw, cudaStream_t st) {
  return launch_dependent(route_combine_grad_kernel<T>, dim3(blocks_of(p.tokens * 32)),
                          dim3(kThreads), 0, st, static_cast<const T*>(dout),
                          static_cast<const T*>(y), weights, undo, kept, static_cast<T*>(dy), dw,
                          p.tokens, (int)p.entries(), p.k, p.d);
}

cudaError_t noted(cudaError_t e) {
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace

cudaError_t launch_route_gather(const RouteProblem& p, const void* x, const int32_t* undo,
                                const int32_t* offsets, void* xs, cudaStream_t st) {
  if (p.tokens == 0) return cudaSuccess;
  const int32_t* kept = offsets + p.experts;
  return noted(p.bf16 ? gather_t<__nv_bfloat16>(p, x, undo, kept, xs, st)
                      : gather_t<float>(p, x, undo, kept, xs, st));
}

cudaError_t launch_route_combine(const RouteProblem& p, const void* y, const float* weights,
                                 const int32_t* undo, const int32_t* offsets, void* out,
                                 cudaStream_t st) {
  if (p.tokens == 0) return cudaSuccess;
  const int32_t* kept = offsets + p.experts;
  return noted(p.bf16 ? combine_t<__nv_bfloat16>(p, y, weights, undo, kept, out, st)
                      : combine_t<float>(p, y, weights, undo, kept, out, st));
}

cudaError_t launch_route_combine_backward(const RouteProblem& p, const void* dout, const void* y,
                                          const float* weights, const int32_t* undo,
                                          const int32_t* offsets, void* dy, float* dweights,
                                          cudaStream_t st) {
  if (p.tokens == 0) return cudaSuccess;
  const int32_t* kept = offsets + p.experts;
  return noted(p.bf16 ? combine_grad_t<__nv_bfloat16>(p, dout, y, weights, undo, kept, dy,
                                                      dweights, st)
                      : combine_grad_t<float>(p, dout, y, weights, undo, kept, dy, dweights, st));
}

}  // namespace lsh
