// tdt_paged_general.cu -- causal attention over a paged cache on the CUDA cores: every type, head width up to
// 256, stride and page size; float32 products throughout.
//
// A CTA per tile of BT queries of one head walks the positions that they see in tiles of BT, each row found
// through the page table, with the running maximum and sum of the softmax (tdt_attn_general.cu).
// It takes what the other kernels do not.
#include "tdt_attn_tile.cuh"
#include "tdt_paged.cuh"

namespace tdt {
namespace {

// Positions [j0, j0 + BT) of head h as float32; those at or past `end` and columns past D are 0.  Returns
// whether a position lies in a page that is not there (its row is 0, too).
template <int PT, int DP>
__device__ bool load_pages(float *dst, const Pages &p, const PageTable &t, long long b, int h, int j0, int end, int D) {
  bool bad = false;
  for (int x = threadIdx.x; x < Tile<DP>::BT * DP; x += kThreads) {
    const int r = x / DP, c = x % DP, pos = j0 + r;
    float v = 0.0f;
    if (pos < end && c < D) {
      const int page = page_of(t, b, pos), place = pos & ((1 << t.page_bits) - 1);
      if (page < 0) {
        bad = true;
      } else if constexpr (PT == kE4M3) {
        const unsigned char *row = static_cast<const unsigned char *>(p.data) + row_at(p.s, page, place, h);
        v = e4m3_to_float(__ldg(row + c)) * scale_of(__ldg(p.scales + row_at(p.ss, page, place, h)));
      } else {
        typedef typename Elem<PT>::T E;
        v = Elem<PT>::load(static_cast<const E *>(p.data) + row_at(p.s, page, place, h) + c);
      }
    }
    dst[r * Tile<DP>::LD + c] = v;
  }
  return bad;
}

template <int DT, int PT, int DP>
__global__ void __launch_bounds__(kThreads, 1) paged_general_kernel(const __grid_constant__ PagedArgs a, int tiles) {
  constexpr int BT = Tile<DP>::BT, MT = Tile<DP>::MT, LD = Tile<DP>::LD, LP = Tile<DP>::LP;
  extern __shared__ __align__(16) float sm[];
  float *Qs = sm, *Ks = Qs + BT * LD, *Vs = Ks + BT * LD, *Ps = Vs + BT * LD;
  const int i0 = blockIdx.x % tiles * BT;
  const unsigned bh = blockIdx.x / tiles;
  const int h = bh % a.H, hk = h / a.G;
  const long long b = bh / a.H;
  const NewRows n = new_rows(a.t, b, a.Lq);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int end = i0 < n.n ? n.first + min(i0 + BT, n.n) : 0;  // positions that some row sees
  load_tile<DT, DP>(Qs, a.q, b * a.sq.b + i0 * a.sq.l + h * a.sq.h, a.sq.l, n.n - i0, a.D);
  const float c = a.scale * kLog2e;
  float m[MT], l[MT], o[MT][Tile<DP>::NC * 4], s[MT][MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.0f;
#pragma unroll
    for (int x = 0; x < Tile<DP>::NC * 4; ++x) o[i][x] = 0.0f;
  }
  bool bad = n.bad;
  for (int j0 = 0; j0 < end; j0 += BT) {
    __syncthreads();
    bool gone = load_pages<PT, DP>(Ks, a.k, a.t, b, hk, j0, end, a.D);
    gone |= load_pages<PT, DP>(Vs, a.v, a.t, b, hk, j0, end, a.D);
    bad |= __syncthreads_or(gone) != 0;
    dot_tile<DP>(s, Qs, Ks);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int row = i0 + ty * MT + i, last = row < n.n ? n.first + row : -1;
      float top = m[i];
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        s[i][j] = j0 + tx + 16 * j <= last ? s[i][j] * c : -INFINITY;
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
        Ps[(ty * MT + i) * LP + tx + 16 * j] = p;
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
    const int row = i0 + ty * MT + i;
    const bool real = row < n.n;
    f[i] = bad ? NAN : real ? 1.0f / l[i] : 0.0f;
    if (a.lse && tx == 0 && row < a.Lq)
      a.lse[(b * a.H + h) * a.Lq + row] = bad ? NAN : real ? (m[i] + log2f(l[i])) * kLn2 : -INFINITY;
    if (!real)
#pragma unroll
      for (int x = 0; x < Tile<DP>::NC * 4; ++x) o[i][x] = 0.0f;
  }
  store_rows<DT, DP>(o, a.out, b * a.so.b + i0 * a.so.l + h * a.so.h, a.so.l, a.Lq - i0, a.D, f);
}

template <int DT, int PT, int DP> cudaError_t launch(const PagedArgs &a, cudaStream_t stream) {
  typedef Tile<DP> T;
  const size_t smem = (size_t)(3 * T::BT * T::LD + T::BT * T::LP) * sizeof(float);
  const int tiles = (a.Lq + T::BT - 1) / T::BT;
  const cudaError_t e = cudaFuncSetAttribute(paged_general_kernel<DT, PT, DP>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  paged_general_kernel<DT, PT, DP><<<(unsigned)(a.B * a.H * tiles), kThreads, smem, stream>>>(a, tiles);
  return cudaGetLastError();
}
template <int DT, int PT> cudaError_t by_width(const PagedArgs &a, cudaStream_t s) {
  return a.D <= 64 ? launch<DT, PT, 64>(a, s) : a.D <= 128 ? launch<DT, PT, 128>(a, s) : launch<DT, PT, 256>(a, s);
}
template <int DT> cudaError_t by_pages(const PagedArgs &a, int cache_dtype, cudaStream_t s) {
  return cache_dtype == kE4M3 ? by_width<DT, kE4M3>(a, s) : by_width<DT, DT>(a, s);
}

}  // namespace

cudaError_t launch_paged_general(const PagedArgs &a, int dtype, int cache_dtype, cudaStream_t stream) {
  return dtype == kF32   ? by_pages<kF32>(a, cache_dtype, stream)
         : dtype == kF16 ? by_pages<kF16>(a, cache_dtype, stream)
                         : by_pages<kBF16>(a, cache_dtype, stream);
}

}  // namespace tdt
