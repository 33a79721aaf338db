// tdt_attn_tile.cuh -- tiles of the attention kernels on the CUDA cores: float32 rows in shared memory and
// products of them.
//
// 256 threads form a 16 x 16 grid; each holds an MT x MT patch of a score
// tile (rows ty*MT+i, columns tx+16*j, so that the 16-byte reads of 8
// neighbouring threads fall into different banks: rows are padded by 4
// words), and MT rows x DP/16 columns of an output tile.
#pragma once

#include "tdt_attn_common.cuh"

namespace tdt {
namespace {

constexpr int kThreads = 256;

template <int DP> struct Tile {
  static constexpr int BT = DP <= 128 ? 64 : 32;  // rows and frames of a tile
  static constexpr int MT = BT / 16;
  static constexpr int LD = DP + 4;               // words of a stored row
  static constexpr int LP = BT + 4;
  static constexpr int NC = DP / 64;              // groups of 4 output columns a thread
};

// Rows [0, BT) of a tile from global memory as float32; rows at or past `valid` and columns
// past D are 0, whatever memory holds there.
template <int DT, int DP>
__device__ void load_tile(float *dst, const void *src, long long off, long long stride, int valid,
                          int D) {
  typedef typename Elem<DT>::T E;
  const E *p = static_cast<const E *>(src) + off;
  for (int x = threadIdx.x; x < Tile<DP>::BT * DP; x += kThreads) {
    const int r = x / DP, c = x % DP;
    dst[r * Tile<DP>::LD + c] = (r < valid && c < D) ? Elem<DT>::load(p + r * stride + c) : 0.0f;
  }
}

// acc[i][j] = sum_d A[ty*MT+i][d] B[tx+16*j][d]
template <int DP>
__device__ __forceinline__ void dot_tile(float (&acc)[Tile<DP>::MT][Tile<DP>::MT], const float *A,
                                         const float *B) {
  constexpr int MT = Tile<DP>::MT, LD = Tile<DP>::LD;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = 0.0f;
#pragma unroll 4
  for (int d = 0; d < DP; d += 4) {
    float4 x[MT], y[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) x[i] = *reinterpret_cast<const float4 *>(A + (ty * MT + i) * LD + d);
#pragma unroll
    for (int j = 0; j < MT; ++j) y[j] = *reinterpret_cast<const float4 *>(B + (tx + 16 * j) * LD + d);
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < MT; ++j)
        acc[i][j] += x[i].x * y[j].x + x[i].y * y[j].y + x[i].z * y[j].z + x[i].w * y[j].w;
  }
}

// acc[i][c] += sum_r P[ty*MT+i][r] B[r][c's columns]
template <int DP>
__device__ __forceinline__ void mul_tile(float (&acc)[Tile<DP>::MT][Tile<DP>::NC * 4],
                                         const float *P, const float *B) {
  constexpr int MT = Tile<DP>::MT, LD = Tile<DP>::LD, LP = Tile<DP>::LP, NC = Tile<DP>::NC;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  for (int r = 0; r < Tile<DP>::BT; r += 4) {
    float4 p[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) p[i] = *reinterpret_cast<const float4 *>(P + (ty * MT + i) * LP + r);
#pragma unroll
    for (int rr = 0; rr < 4; ++rr)
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const float4 y = *reinterpret_cast<const float4 *>(B + (r + rr) * LD + c * 64 + tx * 4);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const float w = rr == 0 ? p[i].x : rr == 1 ? p[i].y : rr == 2 ? p[i].z : p[i].w;
          acc[i][c * 4 + 0] += w * y.x;
          acc[i][c * 4 + 1] += w * y.y;
          acc[i][c * 4 + 2] += w * y.z;
          acc[i][c * 4 + 3] += w * y.w;
        }
      }
  }
}

// acc[i][c] += sum_r P[r][ty*MT+i] B[r][c's columns]
template <int DP>
__device__ __forceinline__ void mul_tile_t(float (&acc)[Tile<DP>::MT][Tile<DP>::NC * 4],
                                           const float *P, const float *B) {
  constexpr int MT = Tile<DP>::MT, LD = Tile<DP>::LD, LP = Tile<DP>::LP, NC = Tile<DP>::NC;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll 2
  for (int r = 0; r < Tile<DP>::BT; ++r) {
    float p[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) p[i] = P[r * LP + ty * MT + i];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const float4 y = *reinterpret_cast<const float4 *>(B + r * LD + c * 64 + tx * 4);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        acc[i][c * 4 + 0] += p[i] * y.x;
        acc[i][c * 4 + 1] += p[i] * y.y;
        acc[i][c * 4 + 2] += p[i] * y.z;
        acc[i][c * 4 + 3] += p[i] * y.w;
      }
    }
  }
}

template <int DT, int DP>
__device__ void store_rows(const float (&acc)[Tile<DP>::MT][Tile<DP>::NC * 4], void *dst,
                           long long off, long long stride, int rows, int D,
                           const float (&f)[Tile<DP>::MT]) {
  typedef typename Elem<DT>::T E;
  E *p = static_cast<E *>(dst) + off;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
  for (int i = 0; i < Tile<DP>::MT; ++i) {
    const int r = ty * Tile<DP>::MT + i;
    if (r >= rows) continue;
#pragma unroll
    for (int c = 0; c < Tile<DP>::NC * 4; ++c) {
      const int d = (c / 4) * 64 + tx * 4 + (c & 3);
      if (d < D) p[(long long)r * stride + d] = Elem<DT>::from_float(acc[i][c] * f[i]);
    }
  }
}

}  // namespace
}  // namespace tdt
