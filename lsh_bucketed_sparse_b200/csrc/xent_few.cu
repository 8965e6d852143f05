// Cross entropy of few float32 rows (up to 32) on CUDA cores (xent_portable.cu
// has the formulas).  The table is what such a call moves: it is read as it
// stands, once for the logits, once more for both gradients, where the tensor
// cores would need its three planes written first (one row against 131072
// words of 1024: 114 us forward and 284 backward, 470 and 1040 through planes).
// Rows are padded to kRows, a power of two.
//
// Logits: a warp takes R words at a time, its lanes share their columns, the
// rows of x stand in shared memory; R kRows sums per lane are then added up
// over the lanes in a transposing tree, which leaves every lane with values of
// one row: the forward's running maximum and sum, or the backward's g.
// Gradients: a thread owns a few columns of x and of dx and walks over a part
// of the words; dW is written as it goes, the parts' dx are added up in order.
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "xent.cuh"

namespace lsh {
namespace {

constexpr size_t kMaxX = 200 * 1024;  // bytes of x in shared memory

// Words per warp.  Each float4 of a row of x, read from shared memory, serves
// them all: with 32 rows two words (64 sums per lane) are bound by those reads,
// four (128 sums, half the warps) by the arithmetic: 325 and 279 us for 131072
// words of 1024.
constexpr __host__ __device__ int words_of(int rows) { return rows >= 16 ? 4 : 8; }
constexpr __host__ __device__ int logit_threads(int rows) { return rows >= 32 ? 256 : 512; }

struct Rows {
  const float* x;
  const float* table;
  const void* targets;
  const float* lse;    // gradient
  const float* dloss;
  float scale;
  int n, vocab, d;
  float2* part;        // logits: [gridDim.x][n]
  float* zt;           // [n]
  float* g;            // gradient: [vocab][kRows]
};

template <int kRows, bool kGrad, typename I>
__global__ void __launch_bounds__(logit_threads(kRows), 1) xent_few_logits_kernel(const Rows p) {
  constexpr int kLogitThreads = logit_threads(kRows), kLogitWarps = kLogitThreads / 32;
  constexpr int R = words_of(kRows), kSums = kRows * R, kMine = kSums / 32;
  extern __shared__ float x_smem[];  // [kRows][d]
  __shared__ float2 joined[kLogitWarps][kRows];
  wait_prior_grid();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, d = p.d;
  const I* targets = static_cast<const I*>(p.targets);
  for (int i = threadIdx.x * 4; i < kRows * d; i += kLogitThreads * 4) {
    const int row = i / d;
    // (the backward takes nothing from rows without a target)
    const bool on = row < p.n && (!kGrad || target_of(targets, row, p.vocab) >= 0);
    *reinterpret_cast<float4*>(x_smem + i) =
        on ? *reinterpret_cast<const float4*>(p.x + i) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __syncthreads();
  // this lane's values: of row `row`, of words r0 .. r0 + kMine - 1 of the R
  const int row = lane * kMine / R, r0 = lane * kMine % R;
  const int target = row < p.n ? target_of(targets, row, p.vocab) : -1;
  const float c = p.scale * kLog2e;
  float run_m = -INFINITY, run_s = 0.f;
  const int stride = gridDim.x * kLogitWarps * R;
  for (int w0 = (blockIdx.x * kLogitWarps + warp) * R; w0 < p.vocab; w0 += stride) {
    float a[kSums];
#pragma unroll
    for (int i = 0; i < kSums; ++i) a[i] = 0.f;
    const float* from = p.table + (size_t)w0 * d;
    auto load = [&](int col, float4* w) {
#pragma unroll
      for (int r = 0; r < R; ++r)
        w[r] = col < d && w0 + r < p.vocab
                   ? __ldg(reinterpret_cast<const float4*>(from + (size_t)r * d + col))
                   : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    float4 w[R];
    load(lane * 4, w);
    for (int col = lane * 4; col < d; col += 128) {
      float4 next[R];
      load(col + 128, next);
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const float4 x = *reinterpret_cast<const float4*>(x_smem + i * d + col);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          float& s = a[i * R + r];
          s = fmaf(x.x, w[r].x, s);
          s = fmaf(x.y, w[r].y, s);
          s = fmaf(x.z, w[r].z, s);
          s = fmaf(x.w, w[r].w, s);
        }
      }
#pragma unroll
      for (int r = 0; r < R; ++r) w[r] = next[r];
    }
    __syncwarp();
    // every step sends half of the sums away and keeps the other half
#pragma unroll
    for (int step = 0; step < 5; ++step) {
      const int o = 16 >> step, half = (kSums / 2) >> step;
      const bool upper = lane & o;
#pragma unroll
      for (int i = 0; i < kSums / 2; ++i) {
        if (i >= half) break;
        const float keep = upper ? a[i + half] : a[i], send = upper ? a[i] : a[i + half];
        a[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
      }
    }
#pragma unroll
    for (int t = 0; t < kMine; ++t) {
      const int word = w0 + r0 + t;
      if (word >= p.vocab || row >= p.n) {
        if (kGrad && word < p.vocab) p.g[(size_t)word * kRows + row] = 0.f;
        continue;
      }
      if (kGrad) {
        float g = 0.f;
        if (target >= 0) {  // (read here: the sums leave no registers for them)
          const float e = exp2f(fmaf(a[t], p.scale, -p.lse[row]) * kLog2e);
          g = p.dloss[row] * p.scale * (e - (word == target ? 1.f : 0.f));
        }
        p.g[(size_t)word * kRows + row] = g;
      } else {
        if (word == target) p.zt[row] = a[t];
        if (word != target || c == 0.f) lse_add(run_m, run_s, a[t] * c, 1.f);
      }
    }
  }
  if (kGrad) return;
#pragma unroll
  for (int o = R / kMine / 2; o; o >>= 1) {  // the lanes of the row
    const float m = __shfl_xor_sync(0xffffffffu, run_m, o);
    const float s = __shfl_xor_sync(0xffffffffu, run_s, o);
    lse_add(run_m, run_s, m, s);
  }
  if (r0 == 0) joined[warp][row] = make_float2(run_m, run_s);
  __syncthreads();
  if (threadIdx.x < p.n) {
    float2 v = joined[0][threadIdx.x];
    for (int q = 1; q < kLogitWarps; ++q)
      lse_add(v.x, v.y, joined[q][threadIdx.x].x, joined[q][threadIdx.x].y);
    p.part[(size_t)blockIdx.x * p.n + threadIdx.x] = v;
  }
}

// Grid (parts of the words, column blocks): dx[part][n][d], dW.
constexpr int kGradThreads = 128, kGradWords = 32;
constexpr __host__ __device__ int columns_of(int rows) { return rows >= 32 ? 2 : 4; }

template <int kRows, typename I>
__global__ void __launch_bounds__(kGradThreads)
xent_few_grad_kernel(const Rows p, float* __restrict__ dx, float* __restrict__ dtable, int words) {
  constexpr int C = columns_of(kRows);
  using Vec = typename std::conditional<C == 2, float2, float4>::type;
  __shared__ __align__(16) float g[kGradWords][kRows];
  wait_prior_grid();
  const int col = (blockIdx.y * kGradThreads + threadIdx.x) * C, d = p.d;
  const bool live = col < d;
  const I* targets = static_cast<const I*>(p.targets);
  auto load = [](const float* from, float* to) {
    const Vec v = *reinterpret_cast<const Vec*>(from);
#pragma unroll
    for (int t = 0; t < C; ++t) to[t] = reinterpret_cast<const float*>(&v)[t];
  };
  auto store = [](float* to, const float* from) {
    Vec v;
#pragma unroll
    for (int t = 0; t < C; ++t) reinterpret_cast<float*>(&v)[t] = from[t];
    *reinterpret_cast<Vec*>(to) = v;
  };
  float x[kRows][C], a[kRows][C];
#pragma unroll
  for (int i = 0; i < kRows; ++i)
#pragma unroll
    for (int t = 0; t < C; ++t) x[i][t] = a[i][t] = 0.f;
#pragma unroll
  for (int i = 0; i < kRows; ++i)
    if (live && i < p.n && target_of(targets, i, p.vocab) >= 0) load(p.x + (size_t)i * d + col, x[i]);
  const int v0 = blockIdx.x * words, v1 = min(p.vocab, v0 + words);
  // The next words and the next tile of g are under way while these are used.
  constexpr int kAhead = 4, kMine = kGradWords * kRows / kGradThreads;
  float w[kAhead][C], next[kAhead][C], mine[kMine];
  auto load_words = [&](int v, float (&to)[kAhead][C]) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (live && v + k < v1) load(p.table + (size_t)(v + k) * d + col, to[k]);
  };
  auto load_g = [&](int v) {
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
      const int i = threadIdx.x + j * kGradThreads;
      mine[j] = v + i / kRows < v1 ? p.g[(size_t)v * kRows + i] : 0.f;
    }
  };
  load_g(v0);
  load_words(v0, w);
  for (int v = v0; v < v1; v += kGradWords) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kMine; ++j) g[0][threadIdx.x + j * kGradThreads] = mine[j];
    __syncthreads();
    load_g(v + kGradWords);
    for (int k0 = 0; k0 < kGradWords; k0 += kAhead) {
      load_words(v + k0 + kAhead, next);
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (!live || v + k0 + k >= v1) continue;
        float dw[C];
#pragma unroll
        for (int t = 0; t < C; ++t) dw[t] = 0.f;
#pragma unroll
        for (int i = 0; i < kRows; i += 4) {
          const float4 g4 = *reinterpret_cast<const float4*>(&g[k0 + k][i]);
          const float gi[4] = {g4.x, g4.y, g4.z, g4.w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int t = 0; t < C; ++t) {
              a[i + j][t] = fmaf(gi[j], w[k][t], a[i + j][t]);
              dw[t] = fmaf(gi[j], x[i + j][t], dw[t]);
            }
        }
        store(dtable + (size_t)(v + k0 + k) * d + col, dw);
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
#pragma unroll
        for (int t = 0; t < C; ++t) w[k][t] = next[k][t];
    }
  }
  if (!live) return;
#pragma unroll
  for (int i = 0; i < kRows; ++i)
    if (i < p.n) store(dx + ((size_t)blockIdx.x * p.n + i) * d + col, a[i]);
}

// dx = the parts' sums in order: a block adds 32 float4 pieces, each warp every
// kSumWarps-th part, then the warps' sums.  Rows without a target are zero,
// whatever the table holds (0 times an infinite word is NaN in the parts).
constexpr int kSumWarps = 8;
template <typename I>
__global__ void __launch_bounds__(kSumWarps * 32)
xent_few_sum_kernel(const float4* __restrict__ parts, const I* __restrict__ targets,
                    float4* __restrict__ dx, int pieces, int n_parts, int per_row, int vocab) {
  __shared__ float4 sums[kSumWarps][32];
  wait_prior_grid();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, piece = blockIdx.x * 32 + lane;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  if (piece < pieces) {
#pragma unroll 8
    for (int q = warp; q < n_parts; q += kSumWarps) {
      const float4 v = parts[(size_t)q * pieces + piece];
      a.x += v.x; a.y += v.y; a.z += v.z; a.w += v.w;
    }
  }
  sums[warp][lane] = a;
  __syncthreads();
  if (warp != 0 || piece >= pieces) return;
#pragma unroll
  for (int q = 1; q < kSumWarps; ++q) {
    const float4 v = sums[q][lane];
    a.x += v.x; a.y += v.y; a.z += v.z; a.w += v.w;
  }
  if (target_of(targets, piece / per_row, vocab) < 0) a = make_float4(0.f, 0.f, 0.f, 0.f);
  dx[piece] = a;
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

int padded_rows(const TableProblem& p) {
  int r = 4;
  while (r < p.rows) r *= 2;
  return r;
}

int logit_blocks(const TableProblem& p) {
  const int words = logit_threads(padded_rows(p)) / 32 * words_of(padded_rows(p));
  const int all = (p.vocab + words - 1) / words;
  return all < sm_count() ? all : sm_count();
}

// Words per part of the gradients: four blocks per SM.
int part_words(const TableProblem& p) {
  const int per_block = kGradThreads * columns_of(padded_rows(p));
  const int col_blocks = (p.d + per_block - 1) / per_block;
  const int parts = (4 * sm_count() + col_blocks - 1) / col_blocks;
  const int words = (p.vocab + parts - 1) / parts;
  return (words + kGradWords - 1) / kGradWords * kGradWords;
}
int grad_parts(const TableProblem& p) { return (p.vocab + part_words(p) - 1) / part_words(p); }

template <int kRows, bool kGrad, typename I>
cudaError_t logits_t(const TableProblem& p, const Rows& r, cudaStream_t st) {
  auto kernel = xent_few_logits_kernel<kRows, kGrad, I>;
  const size_t smem = (size_t)kRows * p.d * sizeof(float);
  cudaError_t e;
  if (smem > 40 * 1024 &&
      (e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)))
    return e;
  e = launch_dependent(kernel, dim3(logit_blocks(p)), dim3(logit_threads(kRows)), smem, st, r);
  if (e == cudaSuccess) note_launch();
  return e;
}

template <bool kGrad, typename I>
cudaError_t logits(const TableProblem& p, const Rows& r, cudaStream_t st) {
  switch (padded_rows(p)) {
    case 4: return logits_t<4, kGrad, I>(p, r, st);
    case 8: return logits_t<8, kGrad, I>(p, r, st);
    case 16: return logits_t<16, kGrad, I>(p, r, st);
    default: return logits_t<32, kGrad, I>(p, r, st);
  }
}

template <typename I>
cudaError_t grads(const TableProblem& p, const Rows& r, float* parts, float* dx, float* dtable,
                  cudaStream_t st) {
  const int rows = padded_rows(p), per_block = kGradThreads * columns_of(rows);
  const dim3 grid(grad_parts(p), (p.d + per_block - 1) / per_block);
  auto kernel = rows == 4    ? xent_few_grad_kernel<4, I>
                : rows == 8  ? xent_few_grad_kernel<8, I>
                : rows == 16 ? xent_few_grad_kernel<16, I>
                             : xent_few_grad_kernel<32, I>;
  cudaError_t e =
      launch_dependent(kernel, grid, dim3(kGradThreads), 0, st, r, parts, dtable, part_words(p));
  if (e) return e;
  note_launch();
  const int pieces = (int)(p.rows * p.d / 4);
  e = launch_dependent(xent_few_sum_kernel<I>, dim3((pieces + 31) / 32), dim3(kSumWarps * 32), 0,
                       st, reinterpret_cast<const float4*>(parts),
                       static_cast<const I*>(r.targets), reinterpret_cast<float4*>(dx), pieces,
                       grad_parts(p), p.d / 4, p.vocab);
  if (e == cudaSuccess) note_launch();
  return e;
}

Rows rows_of(const TableProblem& p, const void* x, const void* table, const void* targets) {
  Rows r = {};
  r.x = static_cast<const float*>(x);
  r.table = static_cast<const float*>(table);
  r.targets = targets;
  r.scale = p.scale;
  r.n = (int)p.rows;
  r.vocab = p.vocab;
  r.d = p.d;
  return r;
}

}  // namespace

bool xent_few_supported(const TableProblem& p) {
  return !p.portable && !p.bf16 && p.rows <= 32 &&
         (size_t)padded_rows(p) * p.d * sizeof(float) <= kMaxX;
}

int xent_few_slices(const TableProblem& p) { return logit_blocks(p); }

cudaError_t launch_xent_few(const TableProblem& p, const void* x, const void* table,
                            const void* targets, float2* part, float* zt, cudaStream_t st) {
  Rows r = rows_of(p, x, table, targets);
  r.part = part;
  r.zt = zt;
  return p.idx64 ? logits<false, int64_t>(p, r, st) : logits<false, int32_t>(p, r, st);
}

size_t xent_few_backward_bytes(const TableProblem& p) {
  return align256((size_t)p.vocab * padded_rows(p) * sizeof(float)) +
         align256((size_t)grad_parts(p) * p.rows * p.d * sizeof(float));
}

cudaError_t launch_xent_few_backward(const TableProblem& p, const void* x, const void* table,
                                     const void* targets, const float* lse, const float* dloss,
                                     void* dx, void* dtable, void* workspace, cudaStream_t st) {
  Rows r = rows_of(p, x, table, targets);
  r.lse = lse;
  r.dloss = dloss;
  r.g = static_cast<float*>(workspace);
  float* parts = reinterpret_cast<float*>(
      static_cast<char*>(workspace) +
      align256((size_t)p.vocab * padded_rows(p) * sizeof(float)));
  cudaError_t e = p.idx64 ? logits<true, int64_t>(p, r, st) : logits<true, int32_t>(p, r, st);
  if (e) return e;
  float *to = static_cast<float*>(dx), *dw = static_cast<float*>(dtable);
  return p.idx64 ? grads<int64_t>(p, r, parts, to, dw, st)
                 : grads<int32_t>(p, r, parts, to, dw, st);
}

}  // namespace lsh
