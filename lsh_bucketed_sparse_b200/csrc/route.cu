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
constexpr int kLongRow = 64;  // pieces

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

// A group of `lanes` lanes (a power of two) per token: the U pieces of B
// entries each that are under way at a time take half of the registers, which
// is what keeps HBM busy (131 KB per SM; with the sums of all U pieces alive
// next to them it is half of that, and 79 instead of 61 us for 65536 tokens of
// 1024 bf16, two entries each).
template <typename T, int U, int B>
__global__ void __launch_bounds__(kThreads)
route_combine_kernel(const T* __restrict__ y, const float* __restrict__ weights,
                     const int32_t* __restrict__ undo, const int32_t* __restrict__ kept,
                     T* __restrict__ out, long long tokens, int entries, int k, int d, int lanes) {
  using V = Vec16<T>;
  static_assert(U == 1 || B <= 4, "one piece where entries come in batches");
  wait_prior_grid();
  const long long t = (long long)blockIdx.x * (kThreads / lanes) + threadIdx.x / lanes;
  if (t >= tokens) return;
  const int n_kept = min(*kept, entries);
  const int lane = threadIdx.x & (lanes - 1), step = lanes * V::N;
  T* to = out + (size_t)t * d;
  int s[B];
  float w[B];
  // slots (-1: dropped or no such entry) and weights of entries j0..
  auto plan = [&](int j0) {
#pragma unroll
    for (int j = 0; j < B; ++j) {
      const bool in = j0 + j < k;
      s[j] = in ? undo[t * k + j0 + j] : -1;
      w[j] = in && weights ? weights[t * k + j0 + j] : 1.f;
    }
#pragma unroll
    for (int j = 0; j < B; ++j)
      if (s[j] >= n_kept) s[j] = -1;
  };
  plan(0);
  for (int col = lane * V::N; col < d; col += U * step) {
    uint4 v[U][B];
    auto load = [&] {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < B; ++j)
          if (s[j] >= 0 && (u == 0 || col + u * step < d))
            v[u][j] = V::raw(y + (size_t)s[j] * d + col + u * step);
    };
    auto add = [&](int u, float* a) {
#pragma unroll
      for (int j = 0; j < B; ++j)
        if (s[j] >= 0) {
          float f[V::N];
          V::unpack(v[u][j], f);
#pragma unroll
          for (int i = 0; i < V::N; ++i) a[i] = fmaf(w[j], f[i], a[i]);
        }
    };
    if constexpr (B <= 4) {  // k <= B
      load();
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (u == 0 || col + u * step < d) {
          float a[V::N];
#pragma unroll
          for (int i = 0; i < V::N; ++i) a[i] = 0.f;
          add(u, a);
          V::store(to + col + u * step, a);
        }
    } else {
      float a[V::N];
#pragma unroll
      for (int i = 0; i < V::N; ++i) a[i] = 0.f;
      for (int j0 = 0; j0 < k; j0 += B) {
        if (k > B) plan(j0);
        load();
        add(0, a);
      }
      V::store(to + col, a);
    }
  }
}

// The same for short rows: a thread takes U pieces, kThreads apart, of any
// tokens, so that no lane is idle.  (131072 tokens of 256 bf16, one entry each,
// 31 us instead of 47, 16384 of 264, eight each, 31 instead of 36; but 65536 of
// 1024, two each, 77 instead of 61, 21845 of 512, six each, 55 instead of 50.)
template <typename T, int U, int B>
__global__ void __launch_bounds__(kThreads)
route_combine_short_kernel(const T* __restrict__ y, const float* __restrict__ weights,
                     const int32_t* __restrict__ undo, const int32_t* __restrict__ kept,
                     T* __restrict__ out, long long pieces, int entries, int k, int d) {
  using V = Vec16<T>;
  static_assert(U == 1 || B < 8, "one piece where entries come in batches");
  wait_prior_grid();
  const int n_kept = min(*kept, entries);
  const int per_row = d / V::N;
  const PieceBlock at(blockIdx.x, kThreads * U, per_row);
  // slots (-1: dropped or no such entry) and weights of entries j0.. of token t
  auto plan = [&](long long t, int j0, int* s, float* w) {
#pragma unroll
    for (int j = 0; j < B; ++j) {
      const bool in = t >= 0 && j0 + j < k;
      s[j] = in ? undo[t * k + j0 + j] : -1;
      w[j] = in && weights ? weights[t * k + j0 + j] : 1.f;
    }
#pragma unroll
    for (int j = 0; j < B; ++j)
      if (s[j] >= n_kept) s[j] = -1;
  };
  auto add = [&](const uint4* v, const int* s, const float* w, float* a) {
#pragma unroll
    for (int j = 0; j < B; ++j)
      if (s[j] >= 0) {
        float f[V::N];
        V::unpack(v[j], f);
#pragma unroll
        for (int i = 0; i < V::N; ++i) a[i] = fmaf(w[j], f[i], a[i]);
      }
  };
  int s[U][B];
  float w[U][B];
  uint4 v[U][B];
  if constexpr (B < 8) {  // k <= B
#pragma unroll
    for (int u = 0; u < U; ++u) {
      long long t;
      int piece;
      at.locate(u * kThreads + threadIdx.x, per_row, &t, &piece);
      if (at.first + u * kThreads + threadIdx.x >= pieces) t = -1;
      plan(t, 0, s[u], w[u]);
#pragma unroll
      for (int j = 0; j < B; ++j)
        if (s[u][j] >= 0) v[u][j] = V::raw(y + ((size_t)s[u][j] * per_row + piece) * V::N);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long p = at.first + u * kThreads + threadIdx.x;
      if (p >= pieces) continue;
      float a[V::N];
#pragma unroll
      for (int i = 0; i < V::N; ++i) a[i] = 0.f;
      add(v[u], s[u], w[u], a);
      V::store(out + p * V::N, a);
    }
  } else {
    const long long p = at.first + threadIdx.x;
    if (p >= pieces) return;
    long long t;
    int piece;
    at.locate(threadIdx.x, per_row, &t, &piece);
    float a[V::N];
#pragma unroll
    for (int i = 0; i < V::N; ++i) a[i] = 0.f;
    for (int j0 = 0; j0 < k; j0 += B) {
      plan(t, j0, s[0], w[0]);
#pragma unroll
      for (int j = 0; j < B; ++j)
        if (s[0][j] >= 0) v[0][j] = V::raw(y + ((size_t)s[0][j] * per_row + piece) * V::N);
      add(v[0], s[0], w[0], a);
    }
    V::store(out + p * V::N, a);
  }
}

// A group of `lanes` lanes (a power of two) per token, kBatch entries at a
// time: the token's row is read once for all of them.  Four resident blocks
// (64 registers) rather than the three of its own choice: 102 to 94 us for
// 32768 tokens of 1024 bf16, four entries each (HBM: 92 us).
template <typename T, int kBatch>
__global__ void __launch_bounds__(kThreads, 4)
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
#pragma unroll (kBatch == 4 ? 2 : 4)
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

// A row per group of lanes, or a row's pieces wherever they fall.
template <typename T, int U, int B>
cudaError_t combine_rows(const RouteProblem& p, const void* y, const float* weights,
                         const int32_t* undo, const int32_t* kept, void* out, cudaStream_t st) {
  const int lanes = lanes_of_row(p.d / Vec16<T>::N);
  return launch_dependent(route_combine_kernel<T, U, B>, dim3(blocks_of(p.tokens * lanes)),
                          dim3(kThreads), 0, st, static_cast<const T*>(y), weights, undo, kept,
                          static_cast<T*>(out), p.tokens, (int)p.entries(), p.k, p.d, lanes);
}

template <typename T, int U, int B>
cudaError_t combine_pieces(const RouteProblem& p, const void* y, const float* weights,
                           const int32_t* undo, const int32_t* kept, void* out, cudaStream_t st) {
  const long long pieces = p.tokens * (p.d / Vec16<T>::N);
  return launch_dependent(route_combine_short_kernel<T, U, B>,
                          dim3(blocks_of((pieces + U - 1) / U)), dim3(kThreads), 0, st,
                          static_cast<const T*>(y), weights, undo, kept, static_cast<T*>(out),
                          pieces, (int)p.entries(), p.k, p.d);
}

template <typename T>
cudaError_t combine_t(const RouteProblem& p, const void* y, const float* weights,
                      const int32_t* undo, const int32_t* kept, void* out, cudaStream_t st) {
  const int pieces = p.d / Vec16<T>::N;
  if (pieces < kLongRow) {
    auto run = p.k == 1   ? combine_pieces<T, 4, 1>
               : p.k == 2 ? combine_pieces<T, 4, 2>
               : p.k <= 4 ? combine_pieces<T, 2, 4>
                          : combine_pieces<T, 1, 8>;
    return run(p, y, weights, undo, kept, out, st);
  }
  auto run = p.k <= 2   ? (pieces >= 128 ? combine_rows<T, 4, 2> : combine_rows<T, 2, 2>)
             : p.k <= 4 ? combine_rows<T, 2, 4>
                        : combine_rows<T, 1, 8>;
  return run(p, y, weights, undo, kept, out, st);
}

template <typename T>
cudaError_t combine_grad_t(const RouteProblem& p, const void* dout, const void* y,
                           const float* weights, const int32_t* undo, const int32_t* kept,
                           void* dy, float* dw, cudaStream_t st) {
  const int lanes = lanes_of_row(p.d / Vec16<T>::N);
  auto kernel = p.k == 1   ? route_combine_grad_kernel<T, 1>
                : p.k == 2 ? route_combine_grad_kernel<T, 2>
                           : route_combine_grad_kernel<T, 4>;
  return launch_dependent(kernel, dim3(blocks_of(p.tokens * lanes)),
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
