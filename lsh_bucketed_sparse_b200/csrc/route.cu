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

// A thread takes U pieces, kThreads apart, and B entries of each at a time:
// all U * B loads of rows are under way before the first is used.
template <typename T, int U, int B>
__global__ void __launch_bounds__(kThreads)
route_combine_kernel(const T* __restrict__ y, const float* __restrict__ weights,
                     const int32_t* __restrict__ undo, const int32_t* __restrict__ kept,
                     T* __restrict__ out, long long pieces, int entries, int k, int d) {
  using V = Vec16<T>;
  wait_prior_grid();
  const int per_row = d / V::N;
  const PieceBlock at(blockIdx.x, kThreads * U, per_row);
  const int n_kept = min(*kept, entries);
  long long t[U];
  int col[U];
  float a[U][V::N];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    at.locate(u * kThreads + threadIdx.x, per_row, &t[u], &col[u]);
    if (at.first + u * kThreads + threadIdx.x >= pieces) t[u] = -1;
    col[u] *= V::N;
#pragma unroll
    for (int i = 0; i < V::N; ++i) a[u][i] = 0.f;
  }
  for (int j0 = 0; j0 < k; j0 += B) {
    int s[U][B];
    float w[U][B];
    uint4 v[U][B];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < B; ++j) {
        const bool in = t[u] >= 0 && j0 + j < k;
        s[u][j] = in ? undo[t[u] * k + j0 + j] : -1;
        w[u][j] = in && weights ? weights[t[u] * k + j0 + j] : 1.f;
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < B; ++j)
        if (s[u][j] >= 0 && s[u][j] < n_kept) v[u][j] = V::raw(y + (size_t)s[u][j] * d + col[u]);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < B; ++j)
        if (s[u][j] >= 0 && s[u][j] < n_kept) {
          float f[V::N];
          V::unpack(v[u][j], f);
#pragma unroll
          for (int i = 0; i < V::N; ++i) a[u][i] = fmaf(w[u][j], f[i], a[u][i]);
        }
  }
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (t[u] >= 0) V::store(out + (size_t)t[u] * d + col[u], a[u]);
}

// A group of `lanes` lanes (a power of two) per token, kBatch entries at a
// time: the token's row is read once for all of them.
constexpr int kBatch = 4;
template <typename T>
__global__ void __launch_bounds__(kThreads)
route_combine_grad_kernel(const T* __restrict__ dout, const T* __restrict__ y,
                          const float* __restrict__ weights, const int32_t* __restrict__ undo,
                          const int32_t* __restrict__ kept, T* __restrict__ dy,
                          float* __restrict__ dw, long long tokens, int entries, int k, int d,
                          int lanes) {
  using V = Vec16<T>;
  wait_prior_grid();
  const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
  const long long t = id / lanes;
  const int lane = (int)(id & (lanes - 1));
  const bool there = t < tokens;
  const int n_kept = *kept;
  const T* g = dout + (size_t)t * d;
  for (int j0 = 0; j0 < k; j0 += kBatch) {
    int s[kBatch];
    float w[kBatch], dot[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      s[j] = there && j0 + j < k ? undo[t * k + j0 + j] : -1;
      if (s[j] >= entries) s[j] = -1;
      w[j] = s[j] >= 0 && s[j] < n_kept ? weights[t * k + j0 + j] : 0.f;
      dot[j] = 0.f;
    }
    if (there) {
#pragma unroll 2
      for (int col = lane * V::N; col < d; col += lanes * V::N) {
        const uint4 gr = V::raw(g + col);
        uint4 yr[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
          if (s[j] >= 0 && s[j] < n_kept) yr[j] = V::raw(y + (size_t)s[j] * d + col);
        float gv[V::N];
        V::unpack(gr, gv);
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          if (s[j] < 0) continue;
          float r[V::N];
#pragma unroll
          for (int i = 0; i < V::N; ++i) r[i] = 0.f;
          if (s[j] < n_kept) {
            float f[V::N];
            V::unpack(yr[j], f);
#pragma unroll
            for (int i = 0; i < V::N; ++i) {
              dot[j] = fmaf(gv[i], f[i], dot[j]);
              r[i] = w[j] * gv[i];
            }
          }
          V::store(dy + (size_t)s[j] * d + col, r);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      for (int o = lanes >> 1; o; o >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
      if (there && lane == 0 && j0 + j < k) dw[t * k + j0 + j] = dot[j];
    }
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
  auto kernel = p.k <= 2 ? route_combine_kernel<T, 2, 2> : route_combine_kernel<T, 1, 4>;
  return launch_dependent(kernel, dim3(blocks_of(p.k <= 2 ? (pieces + 1) / 2 : pieces)),
                          dim3(kThreads), 0, st, static_cast<const T*>(y), weights, undo, kept,
                          static_cast<T*>(out), pieces, (int)p.entries(), p.k, p.d);
}

template <typename T>
cudaError_t combine_grad_t(const RouteProblem& p, const void* dout, const void* y,
                           const float* weights, const int32_t* undo, const int32_t* kept,
                           void* dy, float* dw, cudaStream_t st) {
  const int lanes = lanes_of_row(p.d / Vec16<T>::N);
  return launch_dependent(route_combine_grad_kernel<T>, dim3(blocks_of(p.tokens * lanes)),
                          dim3(kThreads), 0, st, static_cast<const T*>(dout),
                          static_cast<const T*>(y), weights, undo, kept, static_cast<T*>(dy), dw,
                          p.tokens, (int)p.entries(), p.k, p.d, lanes);
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
