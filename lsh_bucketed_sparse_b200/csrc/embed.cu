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
// run of up to kChunk slots is summed by the threads that own the row's
// pieces.  Longer runs (frequent tokens) are cut at multiples of kChunk: one
// CTA per chunk leaves a float32 partial sum, and the last of a run's CTAs to
// finish adds them in order.
#include "common.cuh"
#include "internal.h"
#include "vec16.cuh"

namespace lsh {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 64;  // longest run summed in one go

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

__device__ __forceinline__ bool frequent(int2 run) { return run.y - run.x > kChunk; }

// Threads that share a row of float32 partial sums, four columns each.
__device__ __forceinline__ int width4(int width, int d) {
  while (width < kThreads && width * 4 < d) width *= 2;
  return width;
}

// Sum of `count` rows of `d` values, row i at src(i), over the block:
// `width` threads (a power of two) share a row, the block's kThreads / width
// groups share the rows, and the groups' sums are added in order.  The block's
// first `width` threads get the values; emit(col, values) is called for their
// columns.
template <int N, typename Load, typename Emit>
__device__ void block_sum_rows(int count, int d, int width, float* sums, Load load, Emit emit) {
  const int groups = kThreads / width, grp = threadIdx.x / width, at = threadIdx.x & (width - 1);
  for (int col0 = 0; col0 < d; col0 += width * N) {
    const int col = col0 + at * N;
    float a[N];
#pragma unroll
    for (int t = 0; t < N; ++t) a[t] = 0.f;
    if (col < d) {
#pragma unroll 8
      for (int s = grp; s < count; s += groups) {
        float f[N];
        load(s, col, f);
#pragma unroll
        for (int t = 0; t < N; ++t) a[t] += f[t];
      }
    }
    if (groups > 1) {
#pragma unroll
      for (int t = 0; t < N; ++t) sums[t * kThreads + threadIdx.x] = a[t];
      __syncthreads();
      if (grp == 0)
        for (int o = 1; o < groups; ++o)
#pragma unroll
          for (int t = 0; t < N; ++t) a[t] += sums[t * kThreads + o * width + at];
      __syncthreads();
    }
    if (grp == 0 && col < d) emit(col, a);
  }
}

// Blocks [0, chunks): the chunk's partial sums of frequent tokens, at most
// two (the run of its first slot -> part[chunk][0], another run that reaches
// past its end -> part[chunk][1]).  The block that completes a run's partial
// sums (arrived[], counted at the run's first chunk) adds them in their order
// and writes the table's row.  Later blocks: kRows table rows per group of
// `lanes` lanes (a power of two), for rows that are not frequent: the runs and
// first entries of all of them are read at once; U pieces of a row are under
// way at a time where it has one entry at most, four entries of a piece where
// it has more.
constexpr int kRows = 4;
template <typename T, int U>
__global__ void __launch_bounds__(kThreads)
embed_grad_kernel(const int32_t* __restrict__ perm, const int32_t* __restrict__ sorted,
                  const int2* __restrict__ runs, const T* __restrict__ dout, const T* init,
                  T* dtable, float* part, int32_t* arrived, int n, int chunks, int vocab, int d,
                  int lanes, int width, float scale) {
  using V = Vec16<T>;
  wait_prior_grid();
  if ((int)blockIdx.x < chunks) {
    __shared__ int32_t rows[kChunk];
    __shared__ float sums[kThreads * V::N];
    __shared__ int last;
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
      block_sum_rows<V::N>(
          e - b, d, width, sums,
          [&](int s, int col, float* f) { V::load(dout + (size_t)rows[b + s] * d + col, f); },
          [&](int col, const float* a) {
#pragma unroll
            for (int t = 0; t < V::N; t += 4)
              *reinterpret_cast<float4*>(to + col + t) =
                  make_float4(a[t], a[t + 1], a[t + 2], a[t + 3]);
          });
      const int first = r.x / kChunk, count = (r.y - 1) / kChunk - first + 1;
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) last = atomicAdd(&arrived[first], 1) == count - 1;
      __syncthreads();
      if (!last) continue;
      __threadfence();
      const size_t row = (size_t)(which ? k1 : k0) * d;
      const bool shared = r.x > first * kChunk;  // the first chunk begins with another run
      block_sum_rows<4>(
          count, d, width4(width, d), sums,
          [&](int c, int col, float* f) {
            const size_t at = ((size_t)(first + c) * 2 + (c == 0 && shared)) * d + col;
            const float4 x = __ldcg(reinterpret_cast<const float4*>(part + at));
            f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w;
          },
          [&](int col, const float* a) {
#pragma unroll
            for (int t = 0; t < 4; ++t)
              dtable[row + col + t] =
                  from_f32<T>(a[t] * scale + (init ? to_f32(init[row + col + t]) : 0.f));
          });
    }
    return;
  }
  const int lane = threadIdx.x & (lanes - 1), step = lanes * V::N;
  const long long v0 =
      ((long long)(blockIdx.x - chunks) * (kThreads / lanes) + threadIdx.x / lanes) * kRows;
  int2 run[kRows];
  int entry[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) run[i] = v0 + i < vocab ? runs[v0 + i] : make_int2(0, 0);
#pragma unroll
  for (int i = 0; i < kRows; ++i) entry[i] = run[i].x < run[i].y ? perm[run[i].x] : -1;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if (v0 + i >= vocab || frequent(run[i])) continue;
    const size_t row = (size_t)(v0 + i) * d;
    const bool one = run[i].y - run[i].x <= 1;
    for (int col = lane * V::N; col < d; col += U * step) {
      uint4 old[U], q[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        old[u] = q[u] = make_uint4(0, 0, 0, 0);
        if (u == 0 || col + u * step < d) {
          if (init) old[u] = V::raw(init + row + col + u * step);
          if (one && entry[i] >= 0) q[u] = V::raw(dout + (size_t)entry[i] * d + col + u * step);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (u == 0 || col + u * step < d) {
          float a[V::N], f[V::N];
          V::unpack(q[u], a);
          if (!one) {
            const T* from = dout + col + u * step;
            for (int s = run[i].x; s < run[i].y; s += 4) {
              uint4 x[4];
#pragma unroll
              for (int b = 0; b < 4; ++b)
                x[b] = s + b < run[i].y ? V::raw(from + (size_t)perm[s + b] * d)
                                        : make_uint4(0, 0, 0, 0);
#pragma unroll
              for (int b = 0; b < 4; ++b) {
                V::unpack(x[b], f);
#pragma unroll
                for (int t = 0; t < V::N; ++t) a[t] += f[t];
              }
            }
          }
          V::unpack(old[u], f);
#pragma unroll
          for (int t = 0; t < V::N; ++t) a[t] = a[t] * scale + f[t];
          V::store(dtable + row + col + u * step, a);
        }
    }
  }
}

template <typename T>
cudaError_t grad_t(const TableProblem& p, const int32_t* perm, const int32_t* sorted,
                   const int2* runs, const void* dout, const void* init, void* dtable, float* part,
                   int32_t* arrived, int chunks, cudaStream_t st) {
  const int pieces = p.d / Vec16<T>::N, lanes = lanes_of_row(pieces);
  int width = lanes;
  while (width < kThreads && width < pieces) width *= 2;
  const int each = (pieces + lanes - 1) / lanes, per_block = kThreads / lanes * kRows;
  const long long blocks = chunks + (p.vocab + per_block - 1) / per_block;
  auto kernel = each >= 4   ? embed_grad_kernel<T, 4>
                : each >= 2 ? embed_grad_kernel<T, 2>
                            : embed_grad_kernel<T, 1>;
  cudaError_t e = launch_dependent(kernel, dim3((unsigned)blocks), dim3(kThreads), 0, st, perm, sorted,
                                   runs, static_cast<const T*>(dout), static_cast<const T*>(init),
                                   static_cast<T*>(dtable), part, arrived, (int)p.rows, chunks,
                                   p.vocab, p.d, lanes, width, p.scale);
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
      embed_kernel<T, I>,
      dim3((unsigned)((pieces + kThreads * kPieces - 1) / (kThreads * kPieces))), dim3(kThreads), 0, st,
      static_cast<const I*>(tokens), static_cast<const T*>(table), static_cast<T*>(out),
      pieces, p.vocab, p.d, p.scale);
  if (e) return e;
  note_launch();
  return cudaSuccess;
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

struct Scratch {
  int chunks;  // none where no run can be that long
  size_t perm, sorted, runs, part, arrived, sort, total;
};

Scratch scratch_layout(const TableProblem& p) {
  const size_t n = (size_t)p.rows;
  Scratch s;
  size_t off = 0;
  s.perm = off;   off += align256(n * sizeof(int32_t));
  s.sorted = off; off += align256(n * sizeof(int32_t));
  s.runs = off;   off += align256((size_t)p.vocab * sizeof(int2));
  s.chunks = p.rows > kChunk ? (int)((n + kChunk - 1) / kChunk) : 0;
  s.part = off;   off += align256((size_t)s.chunks * 2 * p.d * sizeof(float));
  s.arrived = off; off += align256((size_t)s.chunks * sizeof(int32_t));
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
  int32_t* arrived = reinterpret_cast<int32_t*>(base + s.arrived);
  cudaError_t e = launch_key_sort(p.rows, p.vocab, tokens, p.idx64, perm, nullptr, nullptr, sorted,
                                  runs, arrived, s.chunks, base + s.sort, st);
  if (e) return e;
  return p.bf16 ? grad_t<__nv_bfloat16>(p, perm, sorted, runs, dout, init, dtable, part, arrived,
                                        s.chunks, st)
                : grad_t<float>(p, perm, sorted, runs, dout, init, dtable, part, arrived, s.chunks,
                                st);
}

}  // namespace lsh
