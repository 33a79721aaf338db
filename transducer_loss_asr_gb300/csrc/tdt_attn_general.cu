// tdt_attn_general.cu -- cross attention on the CUDA cores, for every type,
// head width up to 256 and stride; float32 products throughout.
//
// Forward: one CTA per tile of BT query rows of one head walks the frames
// that its rows see in tiles of BT, holding scores and the output in
// registers, with the running maximum m and sum l of the softmax:
//   m' = max(m, max_j s_j),  l' = l 2^(m - m') + sum_j 2^(s_j - m'),
//   o' = o 2^(m - m') + sum_j 2^(s_j - m') v_j          (s in base 2)
// so the frames are read once and no score is stored.
// Backward: two kernels, so that every sum has one owner and a fixed order:
// a CTA per query tile forms dq, a CTA per frame tile forms dk and dv over
// all query heads of its group.  Each recomputes p_ij = 2^(s_ij - lse_i).
//
// 256 threads form a 16 x 16 grid; each holds an MT x MT patch of a score
// tile (rows ty*MT+i, columns tx+16*j, so that the 16-byte reads of 8
// neighbouring threads fall into different banks: rows are padded by 4
// words), and MT rows x DP/16 columns of an output tile.
//
// They take what the other kernels do not: heads over 128, widths and strides
// that 16-byte loads do not fit.  Bound by the arithmetic's latency, one CTA
// an SM (1201 x 2000, 8 heads of 64, float32, forward and backward: 996 us,
// 17 TFLOP/s).
#include <climits>

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

struct RowTile {
  long long b;
  int h, i0;
};
__device__ __forceinline__ RowTile row_tile(long long id, int tiles, int heads, int BT) {
  RowTile t;
  t.i0 = (int)(id % tiles) * BT;
  const long long bh = id / tiles;
  t.h = (int)(bh % heads);
  t.b = bh / heads;
  return t;
}

// Ranges of the tile's rows into lo/hi[BT] and their hull into *first, *last (shared).
template <int BT>
__device__ void tile_ranges(const AttnArgs &a, long long b, int i0, const Lens &n, int *lo, int *hi,
                            int *first, int *last) {
  if (threadIdx.x == 0) {
    *first = INT_MAX;
    *last = 0;
  }
  __syncthreads();
  if (threadIdx.x < BT) {
    const int2 r = row_range(a, b, i0 + (int)threadIdx.x, n);
    lo[threadIdx.x] = r.x;
    hi[threadIdx.x] = r.y;
    if (r.y > r.x) {
      atomicMin(first, r.x);
      atomicMax(last, r.y);
    }
  }
  __syncthreads();
}

template <int DT, int DP>
__global__ void __launch_bounds__(kThreads, 1) attn_fwd_kernel(AttnArgs a, int tiles) {
  constexpr int BT = Tile<DP>::BT, MT = Tile<DP>::MT, LD = Tile<DP>::LD, LP = Tile<DP>::LP;
  extern __shared__ __align__(16) float sm[];
  float *Qs = sm, *Ks = Qs + BT * LD, *Vs = Ks + BT * LD, *Ps = Vs + BT * LD;
  __shared__ int lo[BT], hi[BT], first, last;
  const RowTile t = row_tile(blockIdx.x, tiles, a.H, BT);
  const Lens n = utt_lens(a, t.b);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, hk = t.h / a.G;
  tile_ranges<BT>(a, t.b, t.i0, n, lo, hi, &first, &last);
  load_tile<DT, DP>(Qs, a.q, t.b * a.sq.b + t.i0 * a.sq.l + t.h * a.sq.h, a.sq.l, n.nq - t.i0, a.D);
  const float c = a.scale * kLog2e;
  float m[MT], l[MT], o[MT][Tile<DP>::NC * 4], s[MT][MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.0f;
#pragma unroll
    for (int x = 0; x < Tile<DP>::NC * 4; ++x) o[i][x] = 0.0f;
  }
  for (int j0 = first == INT_MAX ? 0 : first / BT * BT; j0 < last; j0 += BT) {
    __syncthreads();
    load_tile<DT, DP>(Ks, a.k, t.b * a.sk.b + j0 * a.sk.l + hk * a.sk.h, a.sk.l, n.nk - j0, a.D);
    load_tile<DT, DP>(Vs, a.v, t.b * a.sv.b + j0 * a.sv.l + hk * a.sv.h, a.sv.l, n.nk - j0, a.D);
    __syncthreads();
    dot_tile<DP>(s, Qs, Ks);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int r = ty * MT + i, l0 = lo[r], h0 = hi[r];
      float top = m[i];
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        const int col = j0 + tx + 16 * j;
        s[i][j] = (col >= l0 && col < h0) ? s[i][j] * c : -INFINITY;
        top = fmaxf(top, s[i][j]);
      }
#pragma unroll
      for (int x = 8; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
      const float ref = top == -INFINITY ? 0.0f : top;  // nothing seen yet: every weight is 0
      const float f = fast_exp2(m[i] - ref);
      m[i] = top;
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        const float p = fast_exp2(s[i][j] - ref);
        Ps[r * LP + tx + 16 * j] = p;
        sum += p;
      }
#pragma unroll
      for (int x = 8; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
      l[i] = l[i] * f + sum;
#pragma unroll
      for (int x = 0; x < Tile<DP>::NC * 4; ++x) o[i][x] *= f;
    }
    __syncthreads();
    mul_tile<DP>(o, Ps, Vs);
  }
  float f[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int row = t.i0 + ty * MT + i;
    f[i] = n.bad ? NAN : l[i] == 0.0f ? 0.0f : 1.0f / l[i];
    if (a.lse && tx == 0 && row < a.Lq)
      a.lse[(t.b * a.H + t.h) * a.Lq + row] =
          n.bad ? NAN : l[i] == 0.0f ? -INFINITY : (m[i] + log2f(l[i])) * kLn2;
  }
  store_rows<DT, DP>(o, const_cast<void *>(a.out), t.b * a.so.b + t.i0 * a.so.l + t.h * a.so.h,
                     a.so.l, a.Lq - t.i0, a.D, f);
}

// p and ds of a score tile, from s = q.k and dp = grad_out.v of the same patch.
__device__ __forceinline__ void p_and_ds(float s, float dp, bool seen, float c, float lse2,
                                         float delta, float *p, float *ds) {
  *p = seen ? fast_exp2(s * c - lse2) : 0.0f;
  *ds = seen ? *p * (dp - delta) : 0.0f;
}

template <int DT, int DP>
__global__ void __launch_bounds__(kThreads, 1) attn_dq_kernel(AttnArgs a, int tiles) {
  constexpr int BT = Tile<DP>::BT, MT = Tile<DP>::MT, LD = Tile<DP>::LD, LP = Tile<DP>::LP;
  typedef typename Elem<DT>::T E;
  extern __shared__ __align__(16) float sm[];
  float *Qs = sm, *Os = Qs + BT * LD, *Ks = Os + BT * LD, *Vs = Ks + BT * LD, *Ds = Vs + BT * LD;
  __shared__ int lo[BT], hi[BT], first, last;
  __shared__ float lse2[BT], del[BT];
  const RowTile t = row_tile(blockIdx.x, tiles, a.H, BT);
  const Lens n = utt_lens(a, t.b);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, hk = t.h / a.G;
  tile_ranges<BT>(a, t.b, t.i0, n, lo, hi, &first, &last);
  load_tile<DT, DP>(Qs, a.q, t.b * a.sq.b + t.i0 * a.sq.l + t.h * a.sq.h, a.sq.l, n.nq - t.i0, a.D);
  load_tile<DT, DP>(Os, a.go, t.b * a.sgo.b + t.i0 * a.sgo.l + t.h * a.sgo.h, a.sgo.l, n.nq - t.i0,
                    a.D);
  __syncthreads();
  // delta_i = grad_out_i . out_i, one warp a row; kept for the dk/dv kernel
  for (int r = threadIdx.x >> 5; r < BT; r += kThreads / 32) {
    const int row = t.i0 + r, lane = threadIdx.x & 31;
    float x = 0.0f;
    if (row < n.nq) {
      const E *po = static_cast<const E *>(a.out) + t.b * a.so.b + row * a.so.l + t.h * a.so.h;
      for (int d = lane; d < a.D; d += 32) x += Os[r * LD + d] * Elem<DT>::load(po + d);
    }
    x = warp_sum(x);
    if (lane == 0) {
      const long long at = (t.b * a.H + t.h) * a.Lq + row;
      del[r] = x;
      lse2[r] = row < n.nq ? a.lse[at] * kLog2e : 0.0f;
      if (row < a.Lq) a.delta[at] = x;
    }
  }
  const float c = a.scale * kLog2e;
  float acc[MT][Tile<DP>::NC * 4], s[MT][MT], dp[MT][MT], f[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    f[i] = a.scale;
#pragma unroll
    for (int x = 0; x < Tile<DP>::NC * 4; ++x) acc[i][x] = 0.0f;
  }
  for (int j0 = first == INT_MAX ? 0 : first / BT * BT; j0 < last; j0 += BT) {
    __syncthreads();
    load_tile<DT, DP>(Ks, a.k, t.b * a.sk.b + j0 * a.sk.l + hk * a.sk.h, a.sk.l, n.nk - j0, a.D);
    load_tile<DT, DP>(Vs, a.v, t.b * a.sv.b + j0 * a.sv.l + hk * a.sv.h, a.sv.l, n.nk - j0, a.D);
    __syncthreads();
    dot_tile<DP>(s, Qs, Ks);
    dot_tile<DP>(dp, Os, Vs);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int r = ty * MT + i;
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        const int col = j0 + tx + 16 * j;
        float p, ds;
        p_and_ds(s[i][j], dp[i][j], col >= lo[r] && col < hi[r], c, lse2[r], del[r], &p, &ds);
        Ds[r * LP + tx + 16 * j] = ds;
      }
    }
    __syncthreads();
    mul_tile<DP>(acc, Ds, Ks);
  }
  store_rows<DT, DP>(acc, a.dq, t.b * a.sdq.b + t.i0 * a.sdq.l + t.h * a.sdq.h, a.sdq.l,
                     a.Lq - t.i0, a.D, f);
}

template <int DT, int DP>
__global__ void __launch_bounds__(kThreads, 1) attn_dkv_kernel(AttnArgs a, int tiles) {
  constexpr int BT = Tile<DP>::BT, MT = Tile<DP>::MT, LD = Tile<DP>::LD, LP = Tile<DP>::LP;
  extern __shared__ __align__(16) float sm[];
  float *Qs = sm, *Os = Qs + BT * LD, *Ks = Os + BT * LD, *Vs = Ks + BT * LD, *Ps = Vs + BT * LD,
        *Ds = Ps + BT * LP;
  __shared__ int lo[BT], hi[BT], first, last;
  __shared__ float lse2[BT], del[BT];
  const RowTile t = row_tile(blockIdx.x, tiles, a.Hkv, BT);  // i0: the first frame of the tile
  const Lens n = utt_lens(a, t.b);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, j0 = t.i0;
  load_tile<DT, DP>(Ks, a.k, t.b * a.sk.b + j0 * a.sk.l + t.h * a.sk.h, a.sk.l, n.nk - j0, a.D);
  load_tile<DT, DP>(Vs, a.v, t.b * a.sv.b + j0 * a.sv.l + t.h * a.sv.h, a.sv.l, n.nk - j0, a.D);
  const float c = a.scale * kLog2e;
  float dk[MT][Tile<DP>::NC * 4], dv[MT][Tile<DP>::NC * 4], s[MT][MT], dp[MT][MT], f[MT], one[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    f[i] = a.scale;
    one[i] = 1.0f;
#pragma unroll
    for (int x = 0; x < Tile<DP>::NC * 4; ++x) dk[i][x] = dv[i][x] = 0.0f;
  }
  const int rows = j0 < n.nk ? n.nq : 0;
  for (int h = t.h * a.G; h < (t.h + 1) * a.G; ++h) {
    for (int i0 = 0; i0 < rows; i0 += BT) {
      __syncthreads();
      tile_ranges<BT>(a, t.b, i0, n, lo, hi, &first, &last);
      if (last <= j0 || first >= j0 + BT) continue;  // no row of the tile sees these frames
      load_tile<DT, DP>(Qs, a.q, t.b * a.sq.b + i0 * a.sq.l + h * a.sq.h, a.sq.l, n.nq - i0, a.D);
      load_tile<DT, DP>(Os, a.go, t.b * a.sgo.b + i0 * a.sgo.l + h * a.sgo.h, a.sgo.l, n.nq - i0,
                        a.D);
      if (threadIdx.x < BT) {
        const int row = i0 + threadIdx.x;
        const long long at = (t.b * a.H + h) * a.Lq + row;
        lse2[threadIdx.x] = row < n.nq ? a.lse[at] * kLog2e : 0.0f;
        del[threadIdx.x] = row < n.nq ? a.delta[at] : 0.0f;
      }
      __syncthreads();
      dot_tile<DP>(s, Qs, Ks);
      dot_tile<DP>(dp, Os, Vs);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const int r = ty * MT + i;
#pragma unroll
        for (int j = 0; j < MT; ++j) {
          const int x = tx + 16 * j, col = j0 + x;
          float p, ds;
          p_and_ds(s[i][j], dp[i][j], col >= lo[r] && col < hi[r], c, lse2[r], del[r], &p, &ds);
          Ps[r * LP + x] = p;
          Ds[r * LP + x] = ds;
        }
      }
      __syncthreads();
      mul_tile_t<DP>(dv, Ps, Os);
      mul_tile_t<DP>(dk, Ds, Qs);
    }
  }
  store_rows<DT, DP>(dk, a.dk, t.b * a.sdk.b + j0 * a.sdk.l + t.h * a.sdk.h, a.sdk.l, a.Lk - j0,
                     a.D, f);
  store_rows<DT, DP>(dv, a.dv, t.b * a.sdv.b + j0 * a.sdv.l + t.h * a.sdv.h, a.sdv.l, a.Lk - j0,
                     a.D, one);
}

template <int DP> constexpr size_t smem_bytes(int tiles, int scores) {
  return 4 * (size_t)(tiles * Tile<DP>::BT * Tile<DP>::LD + scores * Tile<DP>::BT * Tile<DP>::LP);
}

template <typename K>
cudaError_t run(K kernel, const AttnArgs &a, long long heads, int length, int BT, size_t smem,
                cudaStream_t stream) {
  const int tiles = (length + BT - 1) / BT;
  const long long blocks = a.B * heads * tiles;
  if (blocks == 0) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)smem);
  if (e != cudaSuccess) return e;
  kernel<<<(unsigned)blocks, kThreads, smem, stream>>>(a, tiles);
  return cudaGetLastError();
}

template <int DT, int DP> cudaError_t fwd(const AttnArgs &a, cudaStream_t s) {
  return run(attn_fwd_kernel<DT, DP>, a, a.H, a.Lq, Tile<DP>::BT, smem_bytes<DP>(3, 1), s);
}
template <int DT, int DP> cudaError_t bwd(const AttnArgs &a, cudaStream_t s) {
  const cudaError_t e =
      run(attn_dq_kernel<DT, DP>, a, a.H, a.Lq, Tile<DP>::BT, smem_bytes<DP>(4, 1), s);
  if (e != cudaSuccess) return e;
  return run(attn_dkv_kernel<DT, DP>, a, a.Hkv, a.Lk, Tile<DP>::BT, smem_bytes<DP>(4, 2), s);
}

template <int DT> cudaError_t by_width(const AttnArgs &a, bool back, cudaStream_t s) {
  if (a.D <= 64) return back ? bwd<DT, 64>(a, s) : fwd<DT, 64>(a, s);
  if (a.D <= 128) return back ? bwd<DT, 128>(a, s) : fwd<DT, 128>(a, s);
  return back ? bwd<DT, 256>(a, s) : fwd<DT, 256>(a, s);
}
cudaError_t by_type(const AttnArgs &a, int dtype, bool back, cudaStream_t s) {
  return dtype == kF32 ? by_width<kF32>(a, back, s)
                       : dtype == kF16 ? by_width<kF16>(a, back, s) : by_width<kBF16>(a, back, s);
}

}  // namespace

cudaError_t launch_attn_general_fwd(const AttnArgs &a, int dtype, cudaStream_t stream) {
  return by_type(a, dtype, false, stream);
}
cudaError_t launch_attn_general_bwd(const AttnArgs &a, int dtype, cudaStream_t stream) {
  return by_type(a, dtype, true, stream);
}

}  // namespace tdt
