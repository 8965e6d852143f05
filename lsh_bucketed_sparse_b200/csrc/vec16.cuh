// 16-byte pieces of a float32 or bfloat16 row, unpacked to float32 and packed
// back (round to nearest even).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace lsh {

template <typename T> struct Vec16;
template <> struct Vec16<float> {
  static constexpr int N = 4;
  __device__ static uint4 raw(const float* p) { return *reinterpret_cast<const uint4*>(p); }
  __device__ static void unpack(const uint4& u, float* f) {
    f[0] = __uint_as_float(u.x); f[1] = __uint_as_float(u.y);
    f[2] = __uint_as_float(u.z); f[3] = __uint_as_float(u.w);
  }
  __device__ static void load(const float* p, float* f) { unpack(raw(p), f); }
  __device__ static void store(float* p, const float* f) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  }
};
template <> struct Vec16<__nv_bfloat16> {
  static constexpr int N = 8;
  __device__ static uint4 raw(const __nv_bfloat16* p) {
    return *reinterpret_cast<const uint4*>(p);
  }
  __device__ static void unpack(const uint4& u, float* f) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const float2 x = __bfloat1622float2(h[t]);
      f[2 * t] = x.x; f[2 * t + 1] = x.y;
    }
  }
  __device__ static void load(const __nv_bfloat16* p, float* f) { unpack(raw(p), f); }
  __device__ static void store(__nv_bfloat16* p, const float* f) {
    uint4 u;
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
    for (int t = 0; t < 4; ++t) h[t] = __floats2bfloat162_rn(f[2 * t], f[2 * t + 1]);
    *reinterpret_cast<uint4*>(p) = u;
  }
};

// A block's share of the pieces of a matrix, in row-major order: one 64-bit
// division for the block, a 32-bit one per piece.
struct PieceBlock {
  long long first, row0;
  unsigned rem;
  __device__ PieceBlock(unsigned block, unsigned size, int per_row) {
    first = (long long)block * size;
    row0 = first / per_row;
    rem = (unsigned)(first - row0 * per_row);
  }
  // Row and piece in the row of the block's i-th piece.
  __device__ void locate(unsigned i, int per_row, long long* row, int* piece) const {
    const unsigned q = rem + i, r = q / (unsigned)per_row;
    *row = row0 + r;
    *piece = (int)(q - r * (unsigned)per_row);
  }
};

// Lanes that share a row of `pieces` pieces: a power of two, 32 at most.
// (Fewer lanes where 32 leave some idle in a row's last pass cost more than
// those: 4093 x 264 float32, 66 pieces, 21 us with 8 lanes, 11 with 32.)
inline int lanes_of_row(int pieces) {
  int lanes = 1;
  while (lanes < 32 && lanes < pieces) lanes *= 2;
  return lanes;
}

}  // namespace lsh
