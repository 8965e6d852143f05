// Cross entropy over the vocabulary: kernel choice, workspaces, and the last
// step of the forward (each row's slices joined into lse and loss).
#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "internal.h"
#include "xent.cuh"

namespace lsh {
namespace {

constexpr int kThreads = 256;

// lse_i = log(R_i + exp z_i,t_i), loss_i = lse_i - z_i,t_i = log1p(R_i / exp
// z_i,t_i), where R_i = s 2^m is the slices' sum, which leaves the target out: the
// loss of a row that is sure of its target keeps its digits, where 1 + R_i and
// the difference of two logits would cut them off.  lse is what the gradient
// takes its probabilities from: for such a row z_i,t_i + loss_i in one rounding.
// A block joins 32 rows: each warp every kJoinWarps-th slice, then the warps in
// order.
constexpr int kJoinWarps = kThreads / 32;
template <typename I>
__global__ void __launch_bounds__(kThreads)
xent_join_kernel(const float2* __restrict__ part, const float* __restrict__ zt,
                 const I* __restrict__ targets, float* __restrict__ loss, float* __restrict__ lse,
                 int rows, int slices, int vocab, float scale) {
  __shared__ float2 sums[kJoinWarps][32];
  wait_prior_grid();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.x * 32 + lane;
  float m = -INFINITY, s = 0.f;
  if (row < rows) {
#pragma unroll 8
    for (int k = warp; k < slices; k += kJoinWarps) {
      const float2 p = part[(size_t)k * rows + row];
      lse_add(m, s, p.x, p.y);
    }
  }
  sums[warp][lane] = make_float2(m, s);
  __syncthreads();
  if (warp != 0 || row >= rows) return;
#pragma unroll
  for (int w = 1; w < kJoinWarps; ++w) lse_add(m, s, sums[w][lane].x, sums[w][lane].y);
  if (target_of(targets, row, vocab) < 0) {
    lse[row] = (m + log2f(s)) * kLn2;
    loss[row] = 0.f;
    return;
  }
  const float unit = scale * kLog2e;
  const float z = zt[row], d = fmaf(-z, unit, m);  // m against the target, in one rounding
  if (unit == 0.f) {  // all logits are 0, the target's among s
    lse[row] = loss[row] = (d + log2f(s)) * kLn2;
    return;
  }
  const float over = d > 0.f ? (d + log2f(s + exp2f(-d))) * kLn2 : log1pf(s * exp2f(d));
  lse_add(m, s, z * unit, 1.f);
  const float all = (m + log2f(s)) * kLn2;
  lse[row] = over <= 1.f && !isnan(all) ? fmaf(z, scale, over) : all;
  loss[row] = isnan(all) ? all : over;
}

__global__ void __launch_bounds__(kThreads) xent_zero_kernel(uint4* out, long long pieces) {
  wait_prior_grid();
  const long long p = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (p < pieces) out[p] = make_uint4(0, 0, 0, 0);
}

template <typename I>
__global__ void __launch_bounds__(kThreads)
xent_clean_kernel(const uint4* __restrict__ x, const I* __restrict__ targets,
                  uint4* __restrict__ clean, long long pieces, int per_row, int vocab) {
  wait_prior_grid();
  const long long p = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (p >= pieces) return;
  clean[p] = target_of(targets, p / per_row, vocab) >= 0 ? x[p] : make_uint4(0, 0, 0, 0);
}

// lsh_attn_test_xent_piece_bytes sets it, so that small cases have several pieces.
std::atomic<unsigned long long> g_piece_bytes{~0ull};

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

int slices_of(const TableProblem& p) {
  if (xent_few_supported(p)) return xent_few_slices(p);
  return xent_tc_supported(p) ? xent_tc_slices(p) : xent_portable_slices(p);
}

}  // namespace

size_t xent_piece_bytes(size_t most) {
  return std::min<unsigned long long>(most, g_piece_bytes.load(std::memory_order_relaxed));
}

unsigned long long set_xent_piece_bytes(unsigned long long bytes) {
  return g_piece_bytes.exchange(bytes);
}

cudaError_t launch_xent_clean(const TableProblem& p, const void* x, const void* targets,
                              void* clean, cudaStream_t st) {
  const int per_row = (int)(p.d * p.elem() / 16);
  const long long pieces = p.rows * per_row;
  const dim3 grid((unsigned)((pieces + kThreads - 1) / kThreads)), block(kThreads);
  const uint4* src = static_cast<const uint4*>(x);
  uint4* dst = static_cast<uint4*>(clean);
  cudaError_t e =
      p.idx64 ? launch_dependent(xent_clean_kernel<int64_t>, grid, block, 0, st, src,
                                 static_cast<const int64_t*>(targets), dst, pieces, per_row,
                                 p.vocab)
              : launch_dependent(xent_clean_kernel<int32_t>, grid, block, 0, st, src,
                                 static_cast<const int32_t*>(targets), dst, pieces, per_row,
                                 p.vocab);
  if (e == cudaSuccess) note_launch();
  return e;
}

size_t xent_workspace_bytes(const TableProblem& p) {
  if (p.rows == 0) return 0;
  return align256((size_t)p.rows * slices_of(p) * sizeof(float2)) +
         align256((size_t)p.rows * sizeof(float)) +
         (!xent_few_supported(p) && xent_tc_supported(p) ? xent_tc_bytes(p) : 0);
}

cudaError_t launch_xent(const TableProblem& p, const void* x, const void* table,
                        const void* targets, float* loss, float* lse, void* workspace,
                        cudaStream_t st) {
  if (p.rows == 0) return cudaSuccess;
  const int slices = slices_of(p), rows = (int)p.rows;
  float2* part = static_cast<float2*>(workspace);
  float* zt = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                       align256((size_t)p.rows * slices * sizeof(float2)));
  void* scratch = reinterpret_cast<char*>(zt) + align256((size_t)p.rows * sizeof(float));
  cudaError_t e = xent_few_supported(p) ? launch_xent_few(p, x, table, targets, part, zt, st)
                  : xent_tc_supported(p)
                      ? launch_xent_tc(p, x, table, targets, part, zt, scratch, st)
                      : launch_xent_portable(p, x, table, targets, part, zt, st);
  if (e) return e;
  const dim3 grid((rows + 31) / 32), block(kThreads);
  e = p.idx64 ? launch_dependent(xent_join_kernel<int64_t>, grid, block, 0, st,
                                 static_cast<const float2*>(part), static_cast<const float*>(zt),
                                 static_cast<const int64_t*>(targets), loss, lse, rows, slices,
                                 p.vocab, p.scale)
              : launch_dependent(xent_join_kernel<int32_t>, grid, block, 0, st,
                                 static_cast<const float2*>(part), static_cast<const float*>(zt),
                                 static_cast<const int32_t*>(targets), loss, lse, rows, slices,
                                 p.vocab, p.scale);
  if (e == cudaSuccess) note_launch();
  return e;
}

size_t xent_backward_workspace_bytes(const TableProblem& p) {
  if (p.rows == 0) return 0;
  if (xent_few_supported(p)) return xent_few_backward_bytes(p);
  return xent_tc_supported(p) ? xent_tc_backward_bytes(p) : xent_portable_backward_bytes(p);
}

cudaError_t launch_xent_backward(const TableProblem& p, const void* x, const void* table,
                                 const void* targets, const float* lse, const float* dloss,
                                 void* dx, void* dtable, void* workspace, cudaStream_t st) {
  if (p.rows == 0) {  // no tokens: the table's gradient is zero
    const long long pieces = (long long)p.vocab * p.d * (long long)p.elem() / 16;
    cudaError_t e = launch_dependent(xent_zero_kernel,
                                     dim3((unsigned)((pieces + kThreads - 1) / kThreads)),
                                     dim3(kThreads), 0, st, static_cast<uint4*>(dtable), pieces);
    if (e == cudaSuccess) note_launch();
    return e;
  }
  if (xent_few_supported(p))
    return launch_xent_few_backward(p, x, table, targets, lse, dloss, dx, dtable, workspace, st);
  return xent_tc_supported(p) ? launch_xent_tc_backward(p, x, table, targets, lse, dloss, dx,
                                                        dtable, workspace, st)
                              : launch_xent_portable_backward(p, x, table, targets, lse, dloss,
                                                              dx, dtable, workspace, st);
}

}  // namespace lsh
