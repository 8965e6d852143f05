// The cross entropy's products on the 5th-generation tensor cores, and the
// parts of it that run in their epilogues (xent_portable.cu has the formulas):
//   logits   Z = x W^T       -> each row's maximum and sum of exponentials
//   gradient Z = x W^T       -> g = scale dloss (exp(Z - lse) - [v = t])
//   dx = g W,  dW = g^T x    -> stored, or added to the sum of earlier pieces
// One kernel does all of them: a persistent GEMM of CTA pairs (cta_group::2).
// A pair computes 256 x `width` (<= 256) tiles of D = A B^T; each CTA stages
// its 128 rows of A and its half of B's columns, 64 of K at a time, and holds
// its 128 rows of D in tensor memory, twice, so that the next tile's products
// run while the epilogue reads the last one.  Per CTA:
//   warp 0      TMA loads into a ring of kSlots slots;
//   warp 1      allocates tensor memory; in CTA 0 one thread issues the MMAs;
//   warps 2..9  epilogue, two warps per quadrant of TMEM lanes, which share a
//               tile's 64-column groups between them.
// Operands stand K-major (x and W for the logits, g for dx) or MN-major (W for
// dx; g and x for dW), so that no transposed copy is made.
//
// float32 operands are taken apart into three bfloat16 values each (24 bits
// of significand), and the six products of planes that matter are summed
// in the same float32 accumulator, small ones first: the three left out are
// below 2^-24 of the largest.
#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "internal.h"
#include "sm100.cuh"
#include "vec16.cuh"
#include "xent.cuh"

namespace lsh {
namespace {

using namespace sm100;

constexpr int kTileM = 256;   // rows of a pair's tile, 128 per CTA
constexpr int kTileN = 256;   // most columns of a tile
constexpr int kBlockK = 64;   // one 128-byte swizzled row of bf16
constexpr int kOperand = 128 * kBlockK * 2;  // bytes of one CTA's A or B of a K block
// The ring's slots hold A and B of a K block, with float32 operands one plane
// of them (each is used by two or three of the six products): 6 or 2 K blocks.
constexpr int kSlots = 6;
constexpr int kSlotBytes = 2 * kOperand;
constexpr int kEpiWarps = 8;
constexpr int kThreads = (2 + kEpiWarps) * 32;
constexpr int kStaging = 32 * 128;  // bytes per epilogue warp: 32 rows of 128 bytes
constexpr int kBars = 2 * kSlots + 5;
constexpr int kSmem = 1024 + kSlots * kSlotBytes + kEpiWarps * kStaging + kBars * 8 + 16;
static_assert(kSmem <= 227 * 1024, "shared memory");
constexpr float kBf16Max = 3.3895313892515355e38f;

enum class Epi { kLse, kGrad, kStore, kAdd };

struct Gemm {
  int rows, cols;         // of D
  int m_tiles, n_tiles, width, last_width;
  int run, slices;        // n tiles of one work item, items per m tile
  int splits, kb_split;   // K in `splits` parts of kb_split blocks
  int kb;                 // K blocks of 64
  int a_planes;           // bf16 A (g): one plane or two, block by block of K
  bool planes;            // float32 operands
  int chunk;              // K blocks summed in one accumulator
  int group;              // m tiles that are walked together
  int items;
};

struct Params {
  Gemm g;
  unsigned int* err;
  // logits and gradient
  const void* targets;
  float scale;
  float2* part;           // [slices * 2][rows]
  float* zt;              // [rows]
  const float* lse;
  const float* dloss;
  int v0, vocab;          // the piece's first word
  // rows that have a target, counted on the device (backward): slot s of the
  // first *count holds row order[s]
  const int32_t* count;
  const int32_t* order;
  bool count_k;           // the count bounds K, not D's rows
  unsigned long long first_wait_ns;  // limit of the MMA thread's first wait for operands
};

// A place in the ring of slots: the stage and the parity of its round.
template <int kDepth>
struct Ring {
  int stage = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++stage == kDepth) { stage = 0; phase ^= 1; }
  }
};

struct Item {
  int m, n0, n1, k0, k1, split;
};

__device__ __forceinline__ Item decode(const Gemm& g, int item) {
  Item it;
  const int per = g.m_tiles * g.slices;
  it.split = item / per;
  const int r = item - it.split * per;
  const int grp = r / (g.group * g.slices);
  const int size = min(g.group, g.m_tiles - grp * g.group);
  const int q = r - grp * g.group * g.slices;
  it.m = grp * g.group + q % size;
  it.n0 = q / size * g.run;
  it.n1 = min(g.n_tiles, it.n0 + g.run);
  it.k0 = it.split * g.kb_split;
  it.k1 = min(g.kb * g.a_planes, it.k0 + g.kb_split);
  return it;
}

// MN-major operand, 128-byte swizzle: rows of 64 elements of M or N (one row
// per k), groups of 8 k 1024 bytes apart, the next 64 elements 8192 bytes on.
__device__ __forceinline__ uint64_t sdesc_mn(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(8192 >> 4) << 16) |
         ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// Two float32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// Largest (or smallest) of 32 values, three operands to an instruction.
template <bool kMax>
__device__ __forceinline__ float extreme(const float (&z)[32]) {
  auto of3 = [](float a, float b, float c) {
    float r;
    if (kMax) asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    else asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
  };
  float a[11];
#pragma unroll
  for (int i = 0; i < 10; ++i) a[i] = of3(z[3 * i], z[3 * i + 1], z[3 * i + 2]);
  a[10] = of3(z[30], z[31], z[31]);
  const float b0 = of3(a[0], a[1], a[2]), b1 = of3(a[3], a[4], a[5]), b2 = of3(a[6], a[7], a[8]);
  return of3(of3(b0, b1, b2), a[9], a[10]);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// T: type of D in memory; kPlanes: float32 operands in three planes each;
// kFine: bfloat16 operands of few rows (kFineRows below); kAMn: A (dW's) is
// MN-major, as B is of both gradients.  (Descriptors are sums with constants:
// with the layouts taken from a parameter the logits of 4093 x 131071 x 512
// took 419 us instead of 402.)
template <Epi kEpi, typename T, typename I, bool kPlanes, bool kFine = false, bool kAMn = false>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
xent_tc_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap,
               const __grid_constant__ CUtensorMap omap, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  constexpr bool kBMn = kEpi == Epi::kStore || kEpi == Epi::kAdd;
  constexpr int kOps = kPlanes ? 3 : 1, kDepth = kSlots / kOps;  // slots per K block, K blocks
  uint8_t* staging = smem + kSlots * kSlotBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(staging + kEpiWarps * kStaging);  // CTA 0's
  uint64_t* empty = full + kSlots;
  uint64_t* t_full = empty + kSlots;   // [2]
  uint64_t* t_empty = t_full + 2;       // [2], CTA 0's
  uint64_t* done = t_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* loads = reinterpret_cast<int*>(tmem_slot + 2);  // that this CTA's loader has issued
  // A wait ran out: every role of both CTAs leaves its loop.
  auto give_up = [&](unsigned int code) {
    atomicOr(p.err, code);
    raise_flag_cluster(const_cast<int*>(abort_flag), 0);
    raise_flag_cluster(const_cast<int*>(abort_flag), 1);
  };
  Gemm g = p.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&t_full[b], 1);
      mbar_init(&t_empty[b], 2 * kEpiWarps);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc_pair(tmem_slot, 512);
  tc_fence_before_sync();
  cluster_sync();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  wait_prior_grid();
  if (p.count) {
    const int count = *p.count;
    if (p.count_k) {
      g.kb = (count + kBlockK - 1) / kBlockK;
      g.kb_split = (g.kb * g.a_planes + g.splits - 1) / g.splits;
    } else {
      g.rows = count;
      g.m_tiles = (count + kTileM - 1) / kTileM;
      g.items = g.m_tiles * g.slices * g.splits;
    }
  }

  const int b_boxes = kBMn ? (g.width / 2 + 63) / 64 : 1;
  const uint32_t slot_bytes = kOperand + (kBMn ? b_boxes * 8192 : g.width / 2 * 128);
  if (warp == 0) {
    // -------------------------------------------------------------- loads
    if (lane == 0) {
      tma_prefetch_desc(&amap);
      tma_prefetch_desc(&bmap);
      int issued = 0;  // slots filled, kOps to a K block
      Ring<kDepth> at;
      bool ok = true;
      for (int item = pair; ok && item < g.items; item += pairs) {
        const Item it = decode(g, item);
        const int m0 = it.m * kTileM + rank * 128;
        for (int n = it.n0; ok && n < it.n1; ++n) {
          const int nw = n == g.n_tiles - 1 ? g.last_width : g.width;
          const int c0 = n * g.width + rank * (nw / 2);
          for (int kb = it.k0; ok && kb < it.k1; ++kb, at.next()) {
            // two planes of A meet the same block of B one after the other
            const bool two = kBMn && !kPlanes && g.a_planes == 2;
            const int first = two ? kb & 1 : 0, k = (two ? kb >> 1 : kb) * kBlockK;
            // planes in the order in which their slots become free
#pragma unroll
            for (int z = kOps - 1; z >= 0; --z) {
              const int s = at.stage * kOps + z;
              if (!mbar_wait(&empty[s], at.phase ^ 1, abort_flag)) {
                ok = false;
                break;
              }
              if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * slot_bytes);  // both CTAs'
              const uint32_t bar = cluster_addr(&full[s], 0);
              uint8_t* a = smem + s * kSlotBytes;
              uint8_t* b = a + kOperand;
              if constexpr (kAMn) {
                tma_load_3d_pair(a, &amap, bar, m0, k, first + z);
                tma_load_3d_pair(a + 8192, &amap, bar, m0 + 64, k, first + z);
              } else {
                tma_load_3d_pair(a, &amap, bar, k, m0, first + z);
              }
              if constexpr (kBMn) {
                for (int j = 0; j < b_boxes; ++j)
                  tma_load_3d_pair(b + j * 8192, &bmap, bar, c0 + 64 * j, k, z);
              } else {
                tma_load_3d_pair(b, &bmap, bar, k, c0, z);
              }
              ++issued;
            }
          }
        }
      }
      if (!ok) give_up(kErrWaitProducer);
      *loads = issued;
    }
  } else if (warp == 1) {
    // -------------------------------------------------------------- MMAs
    if (rank == 0 && lane == 0) {
      constexpr uint32_t major = (kAMn ? 1u << 15 : 0u) | (kBMn ? 1u << 16 : 0u);
      // descriptors of slot 0; addresses in them count 16 bytes
      constexpr uint32_t a_step = (kAMn ? 2048 : 32) >> 4, b_step = (kBMn ? 2048 : 32) >> 4;
      const uint32_t a0 = smem_u32(smem), b0 = a0 + kOperand;
      const uint64_t a_desc = kAMn ? sdesc_mn(a0) : sdesc_kmajor_sw128(a0);
      const uint64_t b_desc = kBMn ? sdesc_mn(b0) : sdesc_kmajor_sw128(b0);
      int tile = 0;
      Ring<kDepth> at;
      bool ok = true, issued = false;
      for (int item = pair; ok && item < g.items; item += pairs) {
        const Item it = decode(g, item);
        for (int n = it.n0; ok && n < it.n1; ++n) {
          const int nw = n == g.n_tiles - 1 ? g.last_width : g.width;
          const uint32_t idesc = idesc_bf16_f32(kTileM, nw) | major;
          for (int kc = it.k0; ok && kc < it.k1; kc += g.chunk, ++tile) {
            const int blocks = min(it.k1, kc + g.chunk) - kc;
            const int buf = tile & 1;
            const uint32_t d = tmem + buf * kTileN;
            if (!mbar_wait(&t_empty[buf], ((tile >> 1) & 1) ^ 1, abort_flag)) {
              ok = false;
              break;
            }
            tc_fence_after_sync();
            for (int kb = 0; ok && kb < blocks; ++kb, at.next()) {
              const int s0 = at.stage * kOps;
              const uint32_t parity = at.phase;
              // product of plane za of A and zb of B into the accumulator
              auto product = [&](int za, int zb, uint32_t accumulate) {
                const uint64_t a = a_desc + (uint32_t)((s0 + za) * (kSlotBytes >> 4));
                const uint64_t b = b_desc + (uint32_t)((s0 + zb) * (kSlotBytes >> 4));
#pragma unroll
                for (int k = 0; k < kBlockK / 16; ++k)  // 16 of K
                  mma_bf16_ss_pair(d, a + k * a_step, b + k * b_step, idesc,
                                   accumulate | (uint32_t)(k > 0));
                issued = true;
              };
              ok = mbar_wait_for(&full[s0], parity, abort_flag,
                                 issued ? kWaitLimitNs : p.first_wait_ns);
              if constexpr (kPlanes) {
                ok = ok && mbar_wait(&full[s0 + 2], parity, abort_flag);
                if (!ok) break;
                tc_fence_after_sync();
                product(0, 2, kb > 0);
                product(2, 0, 1);
                mma_commit_pair(&empty[s0 + 2]);
                ok = mbar_wait(&full[s0 + 1], parity, abort_flag);
                if (!ok) break;
                tc_fence_after_sync();
                product(1, 1, 1);
                product(0, 1, 1);
                product(1, 0, 1);
                mma_commit_pair(&empty[s0 + 1]);
                product(0, 0, 1);
              } else {
                if (!ok) break;
                tc_fence_after_sync();
                product(0, 0, kb > 0);
              }
              mma_commit_pair(&empty[s0]);
            }
            if (ok) mma_commit_pair(&t_full[buf]);
          }
        }
      }
      if (!ok) give_up(kErrWaitMma);
      if (issued) {  // every MMA finishes before tensor memory is released
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                smem_u32(done))
            : "memory");
        const unsigned long long t0 = globaltimer();
        while (!mbar_try_wait(done, 0)) {
          if (globaltimer() - t0 > kWaitLimitNs) { atomicOr(p.err, kErrWaitDrain); break; }
        }
      }
    }
  } else {
    // -------------------------------------------------------------- epilogue
    const int ew = warp - 2, quad = warp & 3, half = ew >> 2;
    const uint32_t lane_addr = tmem + ((uint32_t)(quad * 32) << 16);
    uint8_t* mine = staging + ew * kStaging;
    const I* targets = static_cast<const I*>(p.targets);
    const float c = p.scale * kLog2e;
    int tile = 0;
    bool ok = true;
    auto stage_free = [&] {  // the last store has read the staging tile
      if (lane == 0) bulk_wait_read();
      __syncwarp();
    };
    // g is written up to the end of the K block that holds its last row
    const int row_end = kEpi == Epi::kGrad ? (g.rows + kBlockK - 1) / kBlockK * kBlockK : g.rows;
    auto send = [&](int x, int y, int plane, int planes = 1) {  // from `mine`, 2 KB each
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0 && x < g.cols && y < row_end && y < p.g.rows) {
        if constexpr (kEpi == Epi::kAdd) tma_add_3d(&omap, mine, x, y, plane);
        else
          for (int i = 0; i < planes; ++i) tma_store_3d(&omap, mine + i * 2048, x, y, plane + i);
        bulk_commit();
      }
    };
    // 8 values to 16 bytes of bf16; with `rest` what the rounding left stays in z.
    auto pack8 = [](float* z, bool rest) {
      uint4 w;
      __nv_bfloat162* b2 = reinterpret_cast<__nv_bfloat162*>(&w);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        b2[i] = __floats2bfloat162_rn(z[2 * i], z[2 * i + 1]);
        if (rest) {
          const float2 f = __bfloat1622float2(b2[i]);
          z[2 * i] -= f.x;
          z[2 * i + 1] -= f.y;
        }
      }
      return w;
    };
    // 16-byte piece j of this lane's row of 128 or 64 bytes in the staging
    // tile, swizzled as its tensor map says.
    auto put128 = [&](int j, uint4 w) {
      *reinterpret_cast<uint4*>(mine + lane * 128 + ((j ^ (lane & 7)) << 4)) = w;
    };
    auto put64 = [&](int j, uint4 w, int plane = 0) {
      uint8_t* row = mine + plane * 2048 + lane * 64;
      *reinterpret_cast<uint4*>(row + ((j ^ ((lane >> 1) & 3)) << 4)) = w;
    };
    // (a vote, so that a wait that runs out ends for the whole warp)
    auto wait_tile = [&](int buf, int tile) {
      return __all_sync(0xffffffffu, mbar_wait(&t_full[buf], (tile >> 1) & 1, abort_flag));
    };
    auto release = [&](int buf) {
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(cluster_addr(&t_empty[buf], 0));
    };
    for (int item = pair; ok && item < g.items; item += pairs) {
      const Item it = decode(g, item);
      const int row0 = it.m * kTileM + rank * 128 + quad * 32, row = row0 + lane;
      int target = -1;
      float run_m = -INFINITY, run_s = 0.f, up = 0.f, lse = 0.f;
      if constexpr (kEpi == Epi::kLse || kEpi == Epi::kGrad) {
        if (row < g.rows) {
          if constexpr (kEpi == Epi::kGrad) {
            const int at = p.order[row];
            target = target_of(targets, at, p.vocab);
            up = p.dloss[at] * p.scale;
            lse = p.lse[at];
          } else {
            target = target_of(targets, row, p.vocab);
          }
        }
      }
      const bool all_there = __all_sync(0xffffffffu, target >= 0);
      // Half h, 32 columns at cc of D, of a 64-column group.
      auto take = [&](float (&z)[32], int h, int cc) {
        if constexpr (kEpi == Epi::kLse) {
          const int there = g.cols - cc;  // columns that exist
          if (there <= 0) return;
          if ((unsigned)(target - cc) < 32u) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (target - cc == i) {
                p.zt[row] = z[i];
                if (c != 0.f) z[i] = c > 0.f ? -INFINITY : INFINITY;  // 2^(z c) = 0
              }
          }
          if (there >= 32) {
            const float top = fmaxf(run_m, (c >= 0.f ? extreme<true>(z) : extreme<false>(z)) * c);
            const float ref = top == -INFINITY ? 0.f : top;
            const float2 c2 = make_float2(c, c), ref2 = make_float2(-ref, -ref);
            float2 a[2] = {make_float2(run_s * ex2(run_m - ref), 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 e = fma2(make_float2(z[2 * i], z[2 * i + 1]), c2, ref2);
              a[i & 1] = add2(a[i & 1], make_float2(ex2(e.x), ex2(e.y)));
            }
            run_s = (a[0].x + a[0].y) + (a[1].x + a[1].y);
            run_m = top;
          } else {
            float top = run_m;
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (i < there) top = fmaxf(top, z[i] * c);
            const float ref = top == -INFINITY ? 0.f : top;
            run_s *= ex2(run_m - ref);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (i < there) run_s += ex2(fmaf(z[i], c, -ref));
            run_m = top;
          }
        } else if constexpr (kEpi == Epi::kGrad) {
          // (the difference before the units of log2: what rounding is left of a
          // sure row's target, next to 1, is that of lse)
          const float2 s2 = make_float2(p.scale, p.scale), l2 = make_float2(-lse, -lse);
          const float2 log2e = make_float2(kLog2e, kLog2e);
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float2 e = mul2(fma2(make_float2(z[i], z[i + 1]), s2, l2), log2e);
            z[i] = ex2(e.x);
            z[i + 1] = ex2(e.y);
          }
          const int at = target - p.v0 - cc;
          if ((unsigned)at < 32u) {
#pragma unroll
            for (int i = 0; i < 32; ++i) z[i] -= at == i ? 1.f : 0.f;
          }
          const float2 up2 = make_float2(up, up);
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float2 e = mul2(make_float2(z[i], z[i + 1]), up2);
            z[i] = e.x;
            z[i + 1] = e.y;
          }
          // slots past the last row hold zeros, whatever their logits are
          if (!all_there && target < 0) {
#pragma unroll
            for (int i = 0; i < 32; ++i) z[i] = 0.f;
          }
          if constexpr (!kPlanes) {
            stage_free();
#pragma unroll
            for (int j = 0; j < 8; ++j) put64(j & 3, pack8(z + 8 * (j & 3), j < 4), j >> 2);
            send(cc, row0, 0, 2);
          } else {
#pragma unroll
            for (int pl = 0; pl < 3; ++pl) {
              stage_free();
#pragma unroll
              for (int j = 0; j < 4; ++j) put64(j, pack8(z + 8 * j, true));
              send(cc, row0, pl);
            }
          }
        } else if constexpr (sizeof(T) == 4) {
          stage_free();
#pragma unroll
          for (int j = 0; j < 8; ++j)
            put128(j, make_uint4(__float_as_uint(z[4 * j]), __float_as_uint(z[4 * j + 1]),
                                 __float_as_uint(z[4 * j + 2]), __float_as_uint(z[4 * j + 3])));
          send(cc, row0, it.split);
        } else {
          if (h == 0) stage_free();
#pragma unroll
          for (int j = 0; j < 4; ++j) put128(4 * h + j, pack8(z + 8 * j, false));
          if (h == 1) send(cc - 32, row0, it.split);
        }
      };
      for (int n = it.n0; ok && n < it.n1; ++n) {
        const int nw = n == g.n_tiles - 1 ? g.last_width : g.width;
        const int groups = (nw + 63) / 64, col0 = n * g.width;
        // this warp's 32-column chunks: halves of the groups half, half + 2
        const int chunks = groups > half + 2 ? 4 : groups > half ? 2 : 0;
        auto chunk_col = [&](int i) { return (half + (i & 2)) * 64 + (i & 1) * 32; };
        if (it.k0 >= it.k1) {  // no rows in this part of K
          float z[32];
          for (int i = 0; i < chunks; ++i) {
#pragma unroll
            for (int j = 0; j < 32; ++j) z[j] = 0.f;
            take(z, i & 1, col0 + chunk_col(i));
          }
          continue;
        }
        if constexpr (!kPlanes && !kFine) {
          const int buf = tile & 1;
          ok = wait_tile(buf, tile);
          if (!ok) break;
          tc_fence_after_sync();
          const uint32_t from = lane_addr + (uint32_t)(buf * kTileN);
          uint32_t u[2][32];
          if (chunks) {
            tmem_ld_32x32b_x32(from + (uint32_t)chunk_col(0), u[0]);
            tmem_ld_wait(u[0]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (i >= chunks) break;
            // the next chunk comes while this one is taken
            if (i + 1 < chunks) {
              __syncwarp();
              tmem_ld_32x32b_x32(from + (uint32_t)chunk_col(i + 1), u[(i + 1) & 1]);
            }
            float z[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) z[j] = __uint_as_float(u[i & 1][j]);
            take(z, i & 1, col0 + chunk_col(i));
            if (i + 1 < chunks) {
              __syncwarp();
              tmem_ld_wait(u[(i + 1) & 1]);
              // (the last one is here: the accumulator is free)
              if (i + 2 == chunks) release(buf);
            }
          }
          if (chunks == 0) release(buf);
          ++tile;
        } else {
          // the accumulators of the chunks of K are added up in registers (round
          // to nearest, where the tensor core truncates)
          float sum[4][32];
          for (int kc = it.k0; ok && kc < it.k1; kc += g.chunk, ++tile) {
            const int buf = tile & 1;
            ok = wait_tile(buf, tile);
            if (!ok) break;
            tc_fence_after_sync();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (i >= chunks) break;
              uint32_t u[32];
              tmem_ld_32x32b_x32(lane_addr + (uint32_t)(buf * kTileN + chunk_col(i)), u);
              tmem_ld_wait(u);
#pragma unroll
              for (int j = 0; j < 32; ++j)
                sum[i][j] = __uint_as_float(u[j]) + (kc == it.k0 ? 0.f : sum[i][j]);
            }
            release(buf);
          }
          if (!ok) break;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (i >= chunks) break;
            take(sum[i], i & 1, col0 + chunk_col(i));
          }
        }
      }
      if constexpr (kEpi == Epi::kLse) {
        if (ok && row < g.rows)
          p.part[(size_t)(it.n0 / g.run * 2 + half) * g.rows + row] = make_float2(run_m, run_s);
      }
    }
    if constexpr (kEpi != Epi::kLse) {
      if (lane == 0) bulk_wait();
    }
    if (!ok) give_up(kErrWaitEpilogue);
  }
  __syncwarp();
  tc_fence_before_sync();
  cluster_sync();
  // Every load has met its product, unless a wait ran out (which both CTAs
  // know of by now): then neither CTA may exit before the last loads of both
  // have landed.  A slot that only one CTA has filled completes without the
  // other's bytes.
  if (*abort_flag) {
    if (rank == 0 && threadIdx.x == 0) {
      const int mine = *loads, other = load_cluster(loads, 1), last = max(mine, other);
      const unsigned long long t0 = globaltimer();
      bool landed = true;
      // (the slots of earlier ones have been filled again, so they were used)
      for (int j = max(0, last - kSlots); landed && j < last; ++j) {
        const int block = j / kOps;
        uint64_t* bar = &full[block % kDepth * kOps + kOps - 1 - j % kOps];
        if (j >= mine) mbar_arrive_expect_tx(bar, slot_bytes);
        if (j >= other) mbar_complete_tx(bar, slot_bytes);
        while (landed && !mbar_try_wait(bar, (block / kDepth) & 1))
          landed = globaltimer() - t0 <= kWaitLimitNs;
      }
      if (!landed) atomicOr(p.err, kErrWaitDrain);
    }
    __syncwarp();
    cluster_sync();
  }
  tc_fence_after_sync();
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

// ---------------------------------------------------------------- preparation
// Eight values to the three planes of piece i of `pieces`.  (The first plane
// stops at bfloat16's largest value: float32's largest would round to infinity
// there.  The rest goes to the second.)
__device__ __forceinline__ void put_planes(__nv_bfloat16* planes, long long pieces, long long i,
                                           float* f) {
#pragma unroll
  for (int pl = 0; pl < 3; ++pl) {
    float b[8];
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      b[t] = __bfloat162float(__float2bfloat16_rn(f[t]));
      if (isinf(b[t]) && !isinf(f[t])) b[t] = copysignf(kBf16Max, f[t]);
      f[t] -= b[t];
    }
    Vec16<__nv_bfloat16>::store(planes + ((size_t)pl * pieces + i) * 8, b);
  }
}

__device__ __forceinline__ void load8(const float* p, float* f) {
  Vec16<float>::load(p, f);
  Vec16<float>::load(p + 4, f + 4);
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* f) {
  Vec16<__nv_bfloat16>::load(p, f);
}

// planes[3][rows][d]: three bfloat16 values whose sum is the float32 value to
// 24 bits.
__global__ void __launch_bounds__(256)
xent_planes_kernel(const float* __restrict__ src, __nv_bfloat16* __restrict__ planes,
                   long long pieces) {
  wait_prior_grid();
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= pieces) return;
  float f[8];
  load8(src + i * 8, f);
  put_planes(planes, pieces, i, f);
}

// The rows of x that have a target, in their order (float32 ones as planes),
// and zeros up to the end of the last K block.
template <typename T>
__global__ void __launch_bounds__(256)
xent_rows_kernel(const T* __restrict__ x, const int32_t* __restrict__ order,
                 const int32_t* __restrict__ count, __nv_bfloat16* __restrict__ rows,
                 long long pieces, int per_row) {
  wait_prior_grid();
  const int n = *count, end = (n + kBlockK - 1) / kBlockK * kBlockK;
  const PieceBlock at(blockIdx.x, 256, per_row);
  long long slot;
  int piece;
  at.locate(threadIdx.x, per_row, &slot, &piece);
  const long long i = at.first + threadIdx.x;
  if (i >= pieces || slot >= end) return;
  const T* from = x + ((size_t)(slot < n ? order[slot] : 0) * per_row + piece) * 8;
  if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<uint4*>(rows + i * 8) =
        slot < n ? Vec16<T>::raw(from) : make_uint4(0, 0, 0, 0);
  } else {
    float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (slot < n) load8(from, f);
    put_planes(rows, pieces, i, f);
  }
}

// out = the sum of the planes, in their order; with `slots`, row r of out is
// row slots[r] of the planes, or zeros where that is not below *count.
template <typename TS, typename T>
__global__ void __launch_bounds__(256)
xent_sum_kernel(const TS* __restrict__ sums, T* __restrict__ out,
                const int32_t* __restrict__ slots, const int32_t* __restrict__ count,
                long long pieces, int per_row, int planes) {
  wait_prior_grid();
  const PieceBlock at(blockIdx.x, 256, per_row);
  long long row;
  int piece;
  at.locate(threadIdx.x, per_row, &row, &piece);
  const long long i = at.first + threadIdx.x;
  if (i >= pieces) return;
  float a[8];
#pragma unroll
  for (int t = 0; t < 8; ++t) a[t] = 0.f;
  const long long slot = slots ? slots[row] : row;
  if (!slots || slot < *count) {
    const long long from = slot * per_row + piece;
#pragma unroll 4
    for (int s = 0; s < planes; ++s) {
      float f[8];
      load8(sums + ((size_t)s * pieces + from) * 8, f);
#pragma unroll
      for (int t = 0; t < 8; ++t) a[t] += f[t];
    }
  }
#pragma unroll
  for (int t = 0; t < 8; t += Vec16<T>::N) Vec16<T>::store(out + i * 8 + t, a + t);
}

// ---------------------------------------------------------------- host side
// Limit of the MMA thread's first wait (normally the 2 s of every bounded
// wait); lsh_attn_test_xent_first_wait sets it to exercise the timeout path.
std::atomic<unsigned long long> g_first_wait_ns{kWaitLimitNs};

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }
int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }
int pairs_of_device() { return std::max(1, sm_count() / 2); }

// Clock cycles per K block of a tile of `width` columns: the pair's tensor
// cores take 2 per column and product, but what a CTA has to fetch for it
// (16 KB of A, half the columns of B, of each plane) takes longer where there
// is one product.  Fitted to tiles of 256 and 192 (K of 9472), with planes of
// 256, 192 and 128 columns (K of 520: 3840, 3415 and 2846 cycles a block).
double block_cycles(int width, bool planes) {
  return planes ? std::max(12.0 * width, 1520 + 7.8 * width)
                : std::max(2.0 * width, 341 + 1.33 * width);
}
constexpr double kTileCycles = 3000;  // to fill and empty the pipeline

// K blocks per accumulator.  The tensor core truncates when it adds to one, an
// error that grows with the number of additions to a sum of full size (1.1e-5
// of dx after 500 of them): float32 operands get a new accumulator after
// kPlaneChunk blocks, 28 such additions: 6.5e-7 of dx and of dW, which sums in
// float32 do not better.  (2047 x 8009 x 520, loss and gradients: 2 blocks 426
// us, 4 401, 16 390; with 4 dW is further off than that, 1.5e-6.)
constexpr int kPlaneChunk = 2;
void set_chunk(Gemm* g) { g->chunk = g->planes ? kPlaneChunk : g->kb_split; }

// g of bfloat16 rows has two bfloat16 planes, 16 bits of significand, so that what
// shows in dx and dW is their own rounding (0.0017 of their size; with g in one
// plane, half of the products' work, 0.002 to 0.004).  The second plane is another
// K block of each product.
// Up to kFineRows rows (given, those without a target among them), where the
// products wait for the table and half of a tile's 256 rows is empty, the second
// plane is more rows of the same tile for dx (131072 words of 1024, 16 rows: 223
// us backward, 270 with more of K), and the logits' accumulators are cut every
// kFineChunk blocks (the loss of a few rows was off by up to 6e-6 of its size, now
// 1.4e-6; 82 us forward, 76 without).
constexpr int kFineRows = 128, kFineChunk = 4;
bool is_fine(const TableProblem& p) { return p.bf16 && p.rows <= kFineRows; }
int g_planes_of(const TableProblem& p) { return p.bf16 ? 2 : 3; }

// Cuts D's columns into tiles (of a multiple of 64) and K into parts (with
// may_split) so that the estimated time is least: fewer columns or a part of K
// per tile where whole tiles would leave pairs idle.  A part of K costs
// another plane of partial sums, written and read back at HBM's rate (some
// 4000 bytes per cycle) one after another.
void set_tiles(Gemm* g, bool may_split) {
  static constexpr int kParts[] = {1, 2, 3, 4, 5, 6, 7, 8, 12, 16, 24, 32, 48, 64};
  constexpr double kPlaneCycles = 200;
  const int pairs = pairs_of_device();
  double best = -1;
  for (int width = kTileN; width >= 64; width -= 64) {
    const int n = ceil_div(g->cols, width), last = g->cols - (n - 1) * width;
    const int last_width = ceil_div(last, 32) * 32;  // N of a pair's MMA
    const double block = (block_cycles(width, g->planes) * (n - 1) +
                          block_cycles(last_width, g->planes)) / n;
    const int blocks = g->kb * g->a_planes;
    for (int parts : kParts) {
      if (parts > 1 && (!may_split || parts > blocks)) break;
      const int kb = ceil_div(blocks, parts), s = ceil_div(blocks, kb);
      const double waves = ceil_div((long long)g->m_tiles * n * s, pairs);
      const double cost =
          waves * (kb * block + kTileCycles) +
          (s > 1 ? s * (kPlaneCycles + 2.0 * g->rows * g->cols * 4 / 4000) : 0.0);
      if (best >= 0 && cost >= best) continue;
      best = cost;
      g->width = width;
      g->n_tiles = n;
      g->last_width = last_width;
      g->splits = s;
      g->kb_split = kb;
    }
  }
  g->run = 1;
  g->slices = g->n_tiles;
  g->items = g->m_tiles * g->n_tiles * g->splits;
  set_chunk(g);
}

Gemm make_gemm(long long rows, int cols, int k, bool f32, bool may_split, int a_planes = 1) {
  Gemm g = {};
  g.a_planes = a_planes;
  g.rows = (int)rows;
  g.cols = cols;
  g.m_tiles = ceil_div(rows, kTileM);
  g.kb = ceil_div(k, kBlockK);
  g.planes = f32;
  g.group = 16;
  set_tiles(&g, may_split);
  return g;
}

// Logits: a work item is a run of n tiles of one m tile, with one pair of
// partial results per row.  The longest run that costs at most 2% more time
// than the best one.
Gemm logits_gemm(const TableProblem& p) {
  Gemm g = make_gemm(p.rows, p.vocab, p.d, !p.bf16, false);
  const int pairs = pairs_of_device();
  auto span = [&](int run) {
    return (long long)ceil_div((long long)g.m_tiles * ceil_div(g.n_tiles, run), pairs) * run;
  };
  long long best = span(1);
  const int most = std::min(g.n_tiles, 256);
  for (int run = 2; run <= most; ++run) best = std::min(best, span(run));
  for (int run = 1; run <= most; ++run)
    if (span(run) * 50 <= best * 51) g.run = run;
  g.slices = ceil_div(g.n_tiles, g.run);
  g.items = g.m_tiles * g.slices;
  g.group = 64;
  if (is_fine(p)) g.chunk = kFineChunk;
  return g;
}

// The backward's pieces: g of `words` columns (a multiple of 256) within
// kGradBytes.  Among those, the count whose pieces take the fewest waves of
// dW tiles, then the largest.  (32768 x 32768 x 1024 bf16: 9.24 ms; with half of
// the bytes, twice the pieces, 10.03.)
constexpr size_t kGradBytes = 1280u << 20;
struct Backward {
  int words, pieces;
  size_t ld;             // columns of g
  bool f32_dx, sum_dw;   // dx's rows in float32; dW's sums outside the result
  int dx_planes;         // sums of dx's rows
  Gemm dx, dw;           // of a whole piece
  size_t order, slots, count, rows, w_planes, g, dx_rows, dw_sums, sort, total;
};

Backward plan_backward(const TableProblem& p) {
  Backward b;
  const int planes = p.bf16 ? 1 : 3, g_planes = g_planes_of(p), pairs = pairs_of_device();
  const bool fine = is_fine(p);
  const int all = ceil_div(p.vocab, kTileM), nt = ceil_div(p.d, kTileN);
  const size_t per_tile = (size_t)g_planes * p.rows * kTileM * 2;
  const int most = (int)std::min<size_t>(all, std::max<size_t>(1, xent_piece_bytes(kGradBytes) / per_tile));
  int tiles = most;
  if (most < all) {
    long long best = -1;
    for (int t = most; t >= 1 && t >= most / 2; --t) {
      const int rest = all % t;
      const long long waves = (long long)(all / t) * ceil_div((long long)t * nt, pairs) +
                              ceil_div((long long)rest * nt, pairs);
      if (best < 0 || waves < best) { best = waves; tiles = t; }
    }
  }
  b.words = tiles * kTileM;
  b.pieces = ceil_div(all, tiles);
  b.ld = (size_t)b.words;
  const int words = std::min(b.words, p.vocab);
  // two planes of g are twice K, or for dx of few rows twice the rows, in the same tile
  b.dx = make_gemm(p.rows * (fine ? 2 : 1), p.d, words, !p.bf16, true, p.bf16 && !fine ? 2 : 1);
  b.dw = make_gemm(words, p.d, (int)p.rows, !p.bf16, true, p.bf16 ? 2 : 1);
  b.dx_planes = b.dx.splits * (fine ? 2 : 1);
  b.f32_dx = !p.bf16 || fine || b.dx.splits > 1 || b.pieces > 1;
  b.sum_dw = b.dw.splits > 1;
  const size_t n = (size_t)p.rows, nd = n * p.d, vd = (size_t)b.words * p.d;
  size_t off = 0;
  b.order = off;    off += align256(n * 4);
  b.slots = off;    off += align256(n * 4);
  b.count = off;    off += 256;
  b.rows = off;     off += align256(nd * 2 * planes);
  b.w_planes = off; off += p.bf16 ? 0 : align256((size_t)p.vocab * p.d * 6);
  b.g = off;        off += align256((size_t)g_planes * n * b.ld * 2);
  b.dx_rows = off;  off += align256(nd * (b.f32_dx ? 4 : 2) * b.dx_planes);
  b.dw_sums = off;  off += b.sum_dw ? align256(vd * 4 * b.dw.splits) : 0;
  b.sort = off;     off += key_sort_scratch_bytes(p.rows, 1);
  b.total = off;
  return b;
}

// A tensor of `planes` matrices [rows][ld] of which `cols` columns count.
bool encode(CUtensorMap* map, const void* base, bool f32, long long cols, long long rows,
            long long planes, size_t ld, long long plane_rows, int box_x, int box_y,
            CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  const size_t elem = f32 ? 4 : 2;
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)planes};
  const cuuint64_t strides[2] = {(cuuint64_t)(ld * elem), (cuuint64_t)(ld * elem * plane_rows)};
  const cuuint32_t box[3] = {(cuuint32_t)box_x, (cuuint32_t)box_y, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return tensor_map_encoder()(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                       : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                              3, const_cast<void*>(base), dims, strides, box, estr,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <Epi kEpi, typename T, typename I, bool kPlanes, bool kFine = false, bool kAMn = false>
cudaError_t launch(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& o,
                   const Params& p, cudaStream_t st) {
  auto kernel = xent_tc_kernel<kEpi, T, I, kPlanes, kFine, kAMn>;
  static std::atomic<unsigned long long> set{0};  // devices that know the size already
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
  if (!(set.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e) return e;
    set.fetch_or(bit, std::memory_order_relaxed);
  }
  const int pairs = std::min(pairs_of_device(), p.g.items);
  Params q = p;
  q.first_wait_ns = g_first_wait_ns.load(std::memory_order_relaxed);
  e = launch_dependent(kernel, dim3(2 * pairs), dim3(kThreads), (size_t)kSmem, st, a, b, o, q);
  if (e == cudaSuccess) note_launch();
  return e;
}

// Logits or gradient of rows whose targets are int64 or int32.
template <Epi kEpi>
cudaError_t launch_logits(bool idx64, bool fine, const CUtensorMap& a, const CUtensorMap& b,
                          const CUtensorMap& o, const Params& p, cudaStream_t st) {
  if (fine)
    return idx64 ? launch<kEpi, __nv_bfloat16, int64_t, false, true>(a, b, o, p, st)
                 : launch<kEpi, __nv_bfloat16, int32_t, false, true>(a, b, o, p, st);
  if (!p.g.planes)
    return idx64 ? launch<kEpi, __nv_bfloat16, int64_t, false>(a, b, o, p, st)
                 : launch<kEpi, __nv_bfloat16, int32_t, false>(a, b, o, p, st);
  return idx64 ? launch<kEpi, float, int64_t, true>(a, b, o, p, st)
               : launch<kEpi, float, int32_t, true>(a, b, o, p, st);
}

cudaError_t launch_planes(const void* src, long long values, void* planes, cudaStream_t st) {
  const long long pieces = values / 8;
  cudaError_t e = launch_dependent(xent_planes_kernel, dim3((unsigned)((pieces + 255) / 256)),
                                   dim3(256), 0, st, static_cast<const float*>(src),
                                   static_cast<__nv_bfloat16*>(planes), pieces);
  if (e == cudaSuccess) note_launch();
  return e;
}

cudaError_t launch_rows(const TableProblem& p, const void* x, const int32_t* order,
                        const int32_t* count, void* rows, cudaStream_t st) {
  const int per_row = p.d / 8;
  const long long pieces = p.rows * per_row;
  const dim3 grid((unsigned)((pieces + 255) / 256)), block(256);
  __nv_bfloat16* to = static_cast<__nv_bfloat16*>(rows);
  cudaError_t e =
      p.bf16 ? launch_dependent(xent_rows_kernel<__nv_bfloat16>, grid, block, 0, st,
                                static_cast<const __nv_bfloat16*>(x), order, count, to, pieces,
                                per_row)
             : launch_dependent(xent_rows_kernel<float>, grid, block, 0, st,
                                static_cast<const float*>(x), order, count, to, pieces, per_row);
  if (e == cudaSuccess) note_launch();
  return e;
}

// slots and count: see xent_sum_kernel.
template <typename TS, typename T>
cudaError_t launch_sum(const void* sums, void* out, const int32_t* slots, const int32_t* count,
                       long long rows, int d, int planes, cudaStream_t st) {
  const int per_row = d / 8;
  const long long pieces = rows * per_row;
  cudaError_t e = launch_dependent(xent_sum_kernel<TS, T>, dim3((unsigned)((pieces + 255) / 256)),
                                   dim3(256), 0, st, static_cast<const TS*>(sums),
                                   static_cast<T*>(out), slots, count, pieces, per_row, planes);
  if (e == cudaSuccess) note_launch();
  return e;
}

// Product into rows [0, g.rows) of out: straight into the result (splits == 1)
// or into g.splits planes of float32 sums; `add` to what is there.  count_k: *count
// is the length of K (dW), otherwise the number of rows (dx).
cudaError_t launch_product(const Gemm& g, const CUtensorMap& a, const CUtensorMap& b, void* out,
                           bool f32, int d, long long plane_rows, bool add, const int32_t* count,
                           bool count_k, unsigned int* err, cudaStream_t st) {
  CUtensorMap o;
  if (!encode(&o, out, f32, d, g.rows, g.splits, d, plane_rows, f32 ? 32 : 64, 32))
    return cudaErrorInvalidValue;
  Params p = {};
  p.g = g;
  p.err = err;
  p.count = count;
  p.count_k = count_k;
  constexpr Epi kStore = Epi::kStore, kAdd = Epi::kAdd;
  using B = __nv_bfloat16;
  if (count_k) {  // dW
    if (!f32) return launch<kStore, B, int32_t, false, false, true>(a, b, o, p, st);
    return g.planes ? launch<kStore, float, int32_t, true, false, true>(a, b, o, p, st)
                    : launch<kStore, float, int32_t, false, false, true>(a, b, o, p, st);
  }
  if (!f32) return launch<kStore, B, int32_t, false>(a, b, o, p, st);
  if (!g.planes)
    return add ? launch<kAdd, float, int32_t, false>(a, b, o, p, st)
               : launch<kStore, float, int32_t, false>(a, b, o, p, st);
  return add ? launch<kAdd, float, int32_t, true>(a, b, o, p, st)
             : launch<kStore, float, int32_t, true>(a, b, o, p, st);
}

}  // namespace

unsigned long long set_xent_first_wait_ns(unsigned long long ns) {
  return g_first_wait_ns.exchange(ns);
}

bool xent_tc_supported(const TableProblem& p) {
  // (the limit keeps the count of tiles within 32 bits)
  return !p.portable && tensor_map_encoder() != nullptr && p.rows <= (1 << 24);
}

int xent_tc_slices(const TableProblem& p) { return 2 * logits_gemm(p).slices; }

size_t xent_tc_bytes(const TableProblem& p) {
  return p.bf16 ? 0 : align256((size_t)p.rows * p.d * 6) + align256((size_t)p.vocab * p.d * 6);
}

cudaError_t launch_xent_tc(const TableProblem& p, const void* x, const void* table,
                           const void* targets, float2* part, float* zt, void* scratch,
                           cudaStream_t st) {
  cudaError_t e;
  const int planes = p.bf16 ? 1 : 3;
  if (!p.bf16) {
    void* xp = scratch;
    void* wp = static_cast<char*>(scratch) + align256((size_t)p.rows * p.d * 6);
    if ((e = launch_planes(x, p.rows * p.d, xp, st))) return e;
    if ((e = launch_planes(table, (long long)p.vocab * p.d, wp, st))) return e;
    x = xp;
    table = wp;
  }
  Params k = {};
  k.g = logits_gemm(p);
  k.err = device_error_word();
  if (!k.err) return cudaErrorUnknown;
  k.targets = targets;
  k.scale = p.scale;
  k.part = part;
  k.zt = zt;
  k.vocab = p.vocab;
  CUtensorMap a, b;
  if (!encode(&a, x, false, p.d, p.rows, planes, p.d, p.rows, kBlockK, 128) ||
      !encode(&b, table, false, p.d, p.vocab, planes, p.d, p.vocab, kBlockK, k.g.width / 2))
    return cudaErrorInvalidValue;
  return launch_logits<Epi::kLse>(p.idx64, is_fine(p), a, b, a, k, st);
}

size_t xent_tc_backward_bytes(const TableProblem& p) { return plan_backward(p).total; }

cudaError_t launch_xent_tc_backward(const TableProblem& p, const void* x, const void* table,
                                    const void* targets, const float* lse, const float* dloss,
                                    void* dx, void* dtable, void* workspace, cudaStream_t st) {
  const Backward plan = plan_backward(p);
  char* ws = static_cast<char*>(workspace);
  const int planes = p.bf16 ? 1 : 3, g_planes = g_planes_of(p);
  const bool f32 = !p.bf16, fine = is_fine(p);
  unsigned int* err = device_error_word();
  if (!err) return cudaErrorUnknown;
  cudaError_t e;
  int32_t* order = reinterpret_cast<int32_t*>(ws + plan.order);
  int32_t* slots = reinterpret_cast<int32_t*>(ws + plan.slots);
  int32_t* offsets = reinterpret_cast<int32_t*>(ws + plan.count);
  const int32_t* count = offsets + 1;
  void* rows = ws + plan.rows;
  const void* w = table;
  // the rows that have a target, side by side
  KeyOrder o = {};
  o.perm = order;
  o.undo = slots;
  o.offsets = offsets;
  if ((e = launch_row_order(p.rows, p.vocab, targets, p.idx64, o, ws + plan.sort, st))) return e;
  if ((e = launch_rows(p, x, order, count, rows, st))) return e;
  if (f32) {
    if ((e = launch_planes(table, (long long)p.vocab * p.d, ws + plan.w_planes, st))) return e;
    w = ws + plan.w_planes;
  }
  void* gbuf = ws + plan.g;
  void* dx_rows = ws + plan.dx_rows;
  void* dw_sums = ws + plan.dw_sums;
  CUtensorMap x_k, x_mn, w_k, w_mn, g_k, g_mn, g_out;
  if (!encode(&x_k, rows, false, p.d, p.rows, planes, p.d, p.rows, kBlockK, 128) ||
      !encode(&x_mn, rows, false, p.d, p.rows, planes, p.d, p.rows, 64, kBlockK))
    return cudaErrorInvalidValue;
  for (int v0 = 0; v0 < p.vocab; v0 += plan.words) {
    const int nv = std::min(plan.words, p.vocab - v0);
    const char* wv = static_cast<const char*>(w) + (size_t)v0 * p.d * 2;
    // g of the piece
    Params k = {};
    k.g = make_gemm(p.rows, nv, p.d, f32, false);
    if (fine) k.g.chunk = kFineChunk;  // (the forward's logits, bit for bit)
    k.err = err;
    k.targets = targets;
    k.scale = p.scale;
    k.lse = lse;
    k.dloss = dloss;
    k.count = count;
    k.order = order;
    k.v0 = v0;
    k.vocab = p.vocab;
    // (a piece sees its own words only: rows past them read as zeros)
    if (!encode(&w_k, wv, false, p.d, nv, planes, p.d, p.vocab, kBlockK, k.g.width / 2) ||
        !encode(&w_mn, wv, false, p.d, nv, planes, p.d, p.vocab, 64, kBlockK) ||
        !encode(&g_k, gbuf, false, nv, fine ? 2 * p.rows : p.rows, fine ? 1 : g_planes, plan.ld,
                p.rows, kBlockK, 128) ||
        !encode(&g_mn, gbuf, false, nv, p.rows, g_planes, plan.ld, p.rows, 64, kBlockK) ||
        !encode(&g_out, gbuf, false, nv, p.rows, g_planes, plan.ld, p.rows, 32, 32,
                CU_TENSOR_MAP_SWIZZLE_64B))
      return cudaErrorInvalidValue;
    if ((e = launch_logits<Epi::kGrad>(p.idx64, fine, x_k, w_k, g_out, k, st))) return e;
    // dx += g W
    // (the first piece's cut; a last, shorter one may have blocks for fewer parts)
    Gemm gx = plan.dx;
    gx.kb = ceil_div(nv, kBlockK);
    gx.kb_split = ceil_div(gx.kb * gx.a_planes, plan.dx.splits);
    gx.splits = ceil_div(gx.kb * gx.a_planes, gx.kb_split);
    gx.items = gx.m_tiles * gx.n_tiles * gx.splits;
    set_chunk(&gx);
    // (rows past the last one that has a target are not looked at below)
    if ((e = launch_product(gx, g_k, w_mn, dx_rows, plan.f32_dx, p.d, fine ? 2 * p.rows : p.rows,
                            v0 > 0, fine ? nullptr : count, false, err, st)))
      return e;
    // dW = g^T x
    Gemm gw = plan.dw;
    gw.rows = nv;
    gw.m_tiles = ceil_div(nv, kTileM);
    gw.items = gw.m_tiles * gw.n_tiles * gw.splits;
    char* dw_at = static_cast<char*>(dtable) + (size_t)v0 * p.d * p.elem();
    void* dw_to = plan.sum_dw ? dw_sums : dw_at;
    if ((e = launch_product(gw, g_mn, x_mn, dw_to, f32 || plan.sum_dw, p.d, nv, false, count, true,
                            err, st)))
      return e;
    if (plan.sum_dw) {
      e = f32 ? launch_sum<float, float>(dw_sums, dw_at, nullptr, nullptr, nv, p.d, gw.splits, st)
              : launch_sum<float, __nv_bfloat16>(dw_sums, dw_at, nullptr, nullptr, nv, p.d,
                                                 gw.splits, st);
      if (e) return e;
    }
  }
  // dx's rows to their places
  if (f32)
    return launch_sum<float, float>(dx_rows, dx, slots, count, p.rows, p.d, plan.dx_planes, st);
  if (plan.f32_dx)
    return launch_sum<float, __nv_bfloat16>(dx_rows, dx, slots, count, p.rows, p.d, plan.dx_planes,
                                            st);
  return launch_sum<__nv_bfloat16, __nv_bfloat16>(dx_rows, dx, slots, count, p.rows, p.d, 1, st);
}

}  // namespace lsh
