// Softmax cross entropy over the table's rows on CUDA cores, in float32:
//   z_iv = scale x_i . W_v,  lse_i = log sum_v exp z_iv,
//   loss_i = lse_i - z_i,t_i                  (0 where t_i is outside [0, V))
//          = log1p(sum_{v != t_i} exp(z_iv - z_i,t_i)),
//   g_iv = scale dloss_i (exp(z_iv - lse_i) - [v = t_i]),
//   dx_i = sum_v g_iv W_v,  dW_v = sum_i g_iv x_i.
// The logits are never stored: the forward keeps each row's running maximum
// and sum over the vocabulary, the backward recomputes them from lse one
// piece of the vocabulary at a time.  All products run as 64 x 64 tiles with
// 4 x 4 values per thread.
#include "common.cuh"
#include "internal.h"
#include "xent.cuh"

namespace lsh {
namespace {

constexpr int kT = 64, kK = 16, kThreads = 256;

// One operand of a product: element (row, k) at p[row * s_row + k * s_k];
// zero outside [0, rows) x [0, ks).
template <typename T>
struct Operand {
  const T* p;
  size_t s_row, s_k;
  int rows, ks;
};

struct Tiles {
  float a[kK][kT + 4], b[kK][kT + 4];
};

template <typename T>
__device__ __forceinline__ void load_tile(const Operand<T>& o, float (*to)[kT + 4], int row0,
                                          int k0) {
#pragma unroll
  for (int i = 0; i < kT * kK / kThreads; ++i) {
    const int e = threadIdx.x + i * kThreads;
    // consecutive threads along the contiguous dimension
    const int k = o.s_k == 1 ? e % kK : e / kT, r = o.s_k == 1 ? e / kK : e % kT;
    const bool in = row0 + r < o.rows && k0 + k < o.ks;
    to[k][r] = in ? to_f32(o.p[(size_t)(row0 + r) * o.s_row + (size_t)(k0 + k) * o.s_k]) : 0.f;
  }
}

// acc[i][j] = sum_k A(m0 + 4 ty + i, k) B(n0 + 4 tx + j, k)
template <typename TA, typename TB>
__device__ __forceinline__ void tile_product(const Operand<TA>& A, const Operand<TB>& B, int m0,
                                             int n0, Tiles& s, float (*acc)[4]) {
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
  for (int k0 = 0; k0 < A.ks; k0 += kK) {
    __syncthreads();
    load_tile(A, s.a, m0, k0);
    load_tile(B, s.b, n0, k0);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      const float4 a = *reinterpret_cast<const float4*>(&s.a[k][4 * ty]);
      const float4 b = *reinterpret_cast<const float4*>(&s.b[k][4 * tx]);
      const float av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
    }
  }
}

// Grid (row tiles, slices): running maximum and sum of one tile of rows over
// one slice of the vocabulary.
template <typename T, typename I>
__global__ void __launch_bounds__(kThreads)
xent_fwd_kernel(const Operand<T> x, const Operand<T> w, const I* __restrict__ targets,
                float2* __restrict__ part, float* __restrict__ zt, int slice, float scale2) {
  __shared__ Tiles s;
  wait_prior_grid();
  const int m0 = blockIdx.x * kT, tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const int v0 = blockIdx.y * slice, v1 = min(w.rows, v0 + slice);
  float m[4], sum[4];
  int t[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = m0 + 4 * ty + i;
    m[i] = -INFINITY;
    sum[i] = 0.f;
    t[i] = row < x.rows ? target_of(targets, row, w.rows) : -1;
  }
  for (int n0 = v0; n0 < v1; n0 += kT) {
    float acc[4][4];
    tile_product(x, w, m0, n0, s, acc);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int v = n0 + 4 * tx + j;
        if (v >= v1) continue;
        if (v == t[i]) zt[m0 + 4 * ty + i] = acc[i][j];
        if (v != t[i] || scale2 == 0.f) lse_add(m[i], sum[i], acc[i][j] * scale2, 1.f);
      }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int o = 8; o; o >>= 1) {  // the 16 threads of the row
      const float om = __shfl_xor_sync(0xffffffffu, m[i], o);
      const float os = __shfl_xor_sync(0xffffffffu, sum[i], o);
      lse_add(m[i], sum[i], om, os);
    }
    const int row = m0 + 4 * ty + i;
    if (tx == 0 && row < x.rows)
      part[(size_t)blockIdx.y * x.rows + row] = make_float2(m[i], sum[i]);
  }
}

// Grid (row tiles, column tiles).  g of the piece's columns [v0, v0 + w.rows) into g[rows][ld].
template <typename T, typename I>
__global__ void __launch_bounds__(kThreads)
xent_g_kernel(const Operand<T> x, const Operand<T> w, const I* __restrict__ targets,
              const float* __restrict__ lse, const float* __restrict__ dloss,
              float* __restrict__ g, size_t ld, int v0, int vocab, float scale) {
  __shared__ Tiles s;
  wait_prior_grid();
  const int m0 = blockIdx.x * kT, n0 = blockIdx.y * kT;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  float acc[4][4];
  tile_product(x, w, m0, n0, s, acc);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = m0 + 4 * ty + i;
    if (row >= x.rows) continue;
    const int t = target_of(targets, row, vocab);
    const float l = lse[row], up = t >= 0 ? dloss[row] * scale : 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int v = n0 + 4 * tx + j;
      if (v >= w.rows) continue;
      // a row without a target takes no part, whatever its logits are
      g[(size_t)row * ld + v] =
          t >= 0 ? up * (expf(acc[i][j] * scale - l) - (v0 + v == t ? 1.f : 0.f)) : 0.f;
    }
  }
}

// Grid (row tiles, column tiles).  out = A B^T (+ sum, a float32 matrix of
// earlier pieces); to `out` when it is not NULL, else back to `sum`.  With
// `targets`, rows that have none are zero in `out`, whatever the table holds.
template <typename TA, typename TB, typename TO, typename I>
__global__ void __launch_bounds__(kThreads)
xent_product_kernel(const Operand<TA> A, const Operand<TB> B, float* sum, int first, TO* out,
                    size_t ld, const I* __restrict__ targets, int vocab) {
  __shared__ Tiles s;
  wait_prior_grid();
  const int m0 = blockIdx.x * kT, n0 = blockIdx.y * kT;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  float acc[4][4];
  tile_product(A, B, m0, n0, s, acc);
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = m0 + 4 * ty + i, c = n0 + 4 * tx + j;
      if (r >= A.rows || c >= B.rows) continue;
      const size_t at = (size_t)r * ld + c;
      const float v = first ? acc[i][j] : sum[at] + acc[i][j];
      if (!out) sum[at] = v;
      else out[at] = from_f32<TO>(targets && target_of(targets, r, vocab) < 0 ? 0.f : v);
    }
}

int tiles_of(long long n) { return (int)((n + kT - 1) / kT); }

// Vocabulary slices of the forward: enough CTAs for every SM several times.
int slice_of(const TableProblem& p) {
  const int vt = tiles_of(p.vocab);
  const int want = (4 * sm_count() + tiles_of(p.rows) - 1) / tiles_of(p.rows);
  const int slices = want < 1 ? 1 : want > vt ? vt : want;
  return (vt + slices - 1) / slices * kT;
}

// Columns of a backward piece: g within 64 MB.
int piece_of(const TableProblem& p) {
  long long c = (long long)xent_piece_bytes(64 << 20) / (p.rows * 4) / kT * kT;
  if (c < kT) c = kT;
  const long long all = (long long)tiles_of(p.vocab) * kT;
  return (int)(c < all ? c : all);
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

template <typename T, typename I>
cudaError_t fwd_t(const TableProblem& p, const void* x, const void* table, const void* targets,
                  float2* part, float* zt, int slice, int slices, cudaStream_t st) {
  const Operand<T> X{static_cast<const T*>(x), (size_t)p.d, 1, (int)p.rows, p.d};
  const Operand<T> W{static_cast<const T*>(table), (size_t)p.d, 1, p.vocab, p.d};
  cudaError_t e =
      launch_dependent(xent_fwd_kernel<T, I>, dim3(tiles_of(p.rows), slices), dim3(kThreads), 0,
                       st, X, W, static_cast<const I*>(targets), part, zt, slice, p.scale * kLog2e);
  if (e == cudaSuccess) note_launch();
  return e;
}

template <typename T, typename I>
cudaError_t bwd_t(const TableProblem& p, const void* x, const void* table, const void* targets,
                  const float* lse, const float* dloss, void* dx, void* dtable, float* g,
                  float* sum, void* clean, cudaStream_t st) {
  const int piece = piece_of(p), n = (int)p.rows;
  const size_t ld = piece;
  const T* w = static_cast<const T*>(table);
  const Operand<T> X{static_cast<const T*>(x), (size_t)p.d, 1, n, p.d};
  const Operand<T> Xt{static_cast<const T*>(clean), 1, (size_t)p.d, p.d, n};
  cudaError_t e = launch_xent_clean(p, x, targets, clean, st);
  if (e) return e;
  for (int v0 = 0; v0 < p.vocab; v0 += piece) {
    const int nv = p.vocab - v0 < piece ? p.vocab - v0 : piece;
    const T* wp = w + (size_t)v0 * p.d;
    const Operand<T> W{wp, (size_t)p.d, 1, nv, p.d};
    const Operand<T> Wt{wp, 1, (size_t)p.d, p.d, nv};
    const Operand<float> G{g, ld, 1, n, nv}, Gt{g, 1, ld, nv, n};
    e = launch_dependent(xent_g_kernel<T, I>, dim3(tiles_of(n), tiles_of(nv)), dim3(kThreads), 0,
                         st, X, W, static_cast<const I*>(targets), lse, dloss, g, ld, v0,
                         p.vocab, p.scale);
    if (e) return e;
    note_launch();
    const bool last = v0 + piece >= p.vocab;
    e = launch_dependent(xent_product_kernel<float, T, T, I>, dim3(tiles_of(n), tiles_of(p.d)),
                         dim3(kThreads), 0, st, G, Wt, sum, (int)(v0 == 0),
                         last ? static_cast<T*>(dx) : static_cast<T*>(nullptr), (size_t)p.d,
                         static_cast<const I*>(targets), p.vocab);
    if (e) return e;
    note_launch();
    e = launch_dependent(xent_product_kernel<float, T, T, I>, dim3(tiles_of(nv), tiles_of(p.d)),
                         dim3(kThreads), 0, st, Gt, Xt, static_cast<float*>(nullptr), 1,
                         static_cast<T*>(dtable) + (size_t)v0 * p.d, (size_t)p.d,
                         static_cast<const I*>(nullptr), p.vocab);
    if (e) return e;
    note_launch();
  }
  return cudaSuccess;
}

}  // namespace

int xent_portable_slices(const TableProblem& p) {
  const int s = slice_of(p);
  return (p.vocab + s - 1) / s;
}

cudaError_t launch_xent_portable(const TableProblem& p, const void* x, const void* table,
                                 const void* targets, float2* part, float* zt, cudaStream_t st) {
  const int slice = slice_of(p), slices = xent_portable_slices(p);
  if (p.bf16)
    return p.idx64
               ? fwd_t<__nv_bfloat16, int64_t>(p, x, table, targets, part, zt, slice, slices, st)
               : fwd_t<__nv_bfloat16, int32_t>(p, x, table, targets, part, zt, slice, slices, st);
  return p.idx64 ? fwd_t<float, int64_t>(p, x, table, targets, part, zt, slice, slices, st)
                 : fwd_t<float, int32_t>(p, x, table, targets, part, zt, slice, slices, st);
}

size_t xent_portable_backward_bytes(const TableProblem& p) {
  return align256((size_t)p.rows * piece_of(p) * sizeof(float)) +
         align256((size_t)p.rows * p.d * sizeof(float)) + (size_t)p.rows * p.d * p.elem();
}

cudaError_t launch_xent_portable_backward(const TableProblem& p, const void* x, const void* table,
                                          const void* targets, const float* lse,
                                          const float* dloss, void* dx, void* dtable,
                                          void* workspace, cudaStream_t st) {
  float* g = static_cast<float*>(workspace);
  float* sum = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                        align256((size_t)p.rows * piece_of(p) * sizeof(float)));
  void* clean = reinterpret_cast<char*>(sum) + align256((size_t)p.rows * p.d * sizeof(float));
  auto run = p.bf16 ? (p.idx64 ? bwd_t<__nv_bfloat16, int64_t> : bwd_t<__nv_bfloat16, int32_t>)
                    : (p.idx64 ? bwd_t<float, int64_t> : bwd_t<float, int32_t>);
  return run(p, x, table, targets, lse, dloss, dx, dtable, g, sum, clean, st);
}

}  // namespace lsh
