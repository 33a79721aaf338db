// tdt_paged_step32.cu -- causal attention of few float32 query rows over a paged cache (float32 or e4m3 pages), on the CUDA
// cores: float32 products throughout.
//
// The arithmetic is that of tdt_attn_step.cu: in a warp a position belongs to L lanes of 8 elements each, a lane holds its 8 elements of
// each row of q and of the running output, and each group of L lanes its own running maximum and sum.  A row of pages is found
// through the page table, looked up a turn before its loads, which are in flight a turn before they are used.  e4m3 values
// are exact in float32; a key's power of two multiplies its scores, a value row's its weights.
// The groups, the warps and then the CTAs of a cluster (over distributed shared memory) are joined in a fixed order.
// Bound by memory for one or two rows (64 ragged x 750, 16 heads of 64, float32: 70 us, 4.3 TB/s; e4m3: 45 us, its instructions).
#include <cooperative_groups.h>

#include <algorithm>

#include "tdt_paged.cuh"

namespace tdt {
namespace {

namespace cg = cooperative_groups;

constexpr int kCtaRows = 8;  // rows of a key head that a CTA has
constexpr int kWarps = 4;

struct Step32Args {
  PagedArgs a;
  int splits;  // CTAs of a cluster
  int groups;  // clusters that share the rows of a key head
};

// 8 elements of a row of pages and, in e4m3, its power of two
template <int PT> struct Piece;
template <> struct Piece<kF32> {
  float4 x, y;
  __device__ __forceinline__ void load(const Pages &p, int page, int place, int h, int d0) {
    const float4 *at = reinterpret_cast<const float4 *>(static_cast<const float *>(p.data) + row_at(p.s, page, place, h) + d0);
    x = __ldg(at);
    y = __ldg(at + 1);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
  }
  __device__ __forceinline__ float scale() const { return 1.0f; }
};
template <> struct Piece<kE4M3> {
  uint2 x;
  unsigned byte;
  __device__ __forceinline__ void load(const Pages &p, int page, int place, int h, int d0) {
    x = __ldg(reinterpret_cast<const uint2 *>(static_cast<const unsigned char *>(p.data) + row_at(p.s, page, place, h) + d0));
    byte = __ldg(p.scales + row_at(p.ss, page, place, h));
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const unsigned w[2] = {x.x, x.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = e4m3x2_to_float2(w[i / 2] >> (i % 2 * 16) & 0xffffu);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
  __device__ __forceinline__ float scale() const { return scale_of(byte); }
};

// R rows at most, L lanes a position
template <int PT, int R, int L>
__global__ void __launch_bounds__(kWarps * 32) paged_step32_kernel(const __grid_constant__ Step32Args f) {
  constexpr int F = 32 / L;  // positions of a group load
  constexpr int U = 2;       // group loads of a turn
  constexpr int D = L * 8;
  const PagedArgs &a = f.a;
  __shared__ float part_m[kWarps][R], part_l[kWarps][R];
  __shared__ __align__(16) float part_o[kWarps][R][D];
  __shared__ float cta_m[R], cta_l[R];
  __shared__ __align__(16) float cta_o[R][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane / L, d0 = lane % L * 8;
  const unsigned cluster_id = blockIdx.x / f.splits, unit = cluster_id / f.groups;  // = b * Hkv + hk
  const int split = blockIdx.x % f.splits, hk = unit % a.Hkv;
  const long long b = unit / a.Hkv;
  const NewRows n = new_rows(a.t, b, a.Lq);
  const int row0 = cluster_id % f.groups * kCtaRows;
  const int rows = min(R, a.Lq * a.G - row0);  // row r: query (row0 + r) / G, head hk * G + (row0 + r) % G
  const int used = min(n.n, (row0 + rows - 1) / a.G + 1);
  const int end = used > row0 / a.G ? n.first + used : 0;  // positions that some row sees
  const bool wide = d0 < a.D;                               // D is a multiple of 8
  int seen[R];
  float q[R][8], o[R][8], m[R], l[R];
  const float c = a.scale * kLog2e;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int i = (row0 + r) / a.G;
    const bool live = r < rows && i < n.n;
    seen[r] = live ? n.first + i + 1 : 0;
    const float *src = static_cast<const float *>(a.q) + b * a.sq.b + i * a.sq.l + (hk * a.G + (row0 + r) % a.G) * a.sq.h + d0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      q[r][k] = live && wide ? __ldg(src + k) * c : 0.0f;  // scores in base 2
      o[r][k] = 0.0f;
    }
    m[r] = -INFINITY;
    l[r] = 0.0f;
  }
  bool bad = false;
  // turns of F * U positions, over the splits and their warps
  const int turn = F * U, turns = (end + turn - 1) / turn, step = f.splits * kWarps, place_mask = (1 << a.t.page_bits) - 1;
  auto lookup = [&](int x, int (&page)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = x * turn + sub + u * F;
      page[u] = j < end ? page_of(a.t, b, j) : -1;
      bad |= j < end && page[u] < 0;
    }
  };
  Piece<PT> kx[U], vx[U], kn[U], vn[U];
  auto load = [&](int x, const int (&page)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int place = (x * turn + sub + u * F) & place_mask;
      kn[u] = Piece<PT>{};
      vn[u] = Piece<PT>{};
      if (page[u] >= 0 && wide) {  // positions past `end` are not read
        kn[u].load(a.k, page[u], place, hk, d0);
        vn[u].load(a.v, page[u], place, hk, d0);
      }
    }
  };
  int page[U];
  int x = split * kWarps + warp;
  lookup(x, page);
  load(x, page);
  lookup(x + step, page);
  for (; x < turns; x += step) {
    const int j0 = x * turn + sub;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      kx[u] = kn[u];
      vx[u] = vn[u];
    }
    if (x + step < turns) load(x + step, page);
    lookup(x + 2 * step, page);
    float s[R][U], ks[U], vs[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float kf[8];
      kx[u].get(kf);
      ks[u] = kx[u].scale();
      vs[u] = vx[u].scale();
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float p = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) p = fmaf(q[r][k], kf[k], p);
        s[r][u] = p;
      }
    }
#pragma unroll
    for (int x2 = L / 2; x2 > 0; x2 >>= 1)
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int r = 0; r < R; ++r) s[r][u] += __shfl_xor_sync(0xffffffffu, s[r][u], x2);
    // lanes past D have no power of two of their own
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (PT == kE4M3) {
        ks[u] = __shfl_sync(0xffffffffu, ks[u], sub * L);
        vs[u] = __shfl_sync(0xffffffffu, vs[u], sub * L);
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float top = m[r];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (PT == kE4M3) s[r][u] *= ks[u];
        if (j0 + u * F >= seen[r]) s[r][u] = -INFINITY;
        top = fmaxf(top, s[r][u]);
      }
      const float ref = top == -INFINITY ? 0.0f : top;
      const float down = fast_exp2(m[r] - ref);
      m[r] = top;
      l[r] *= down;
#pragma unroll
      for (int k = 0; k < 8; ++k) o[r][k] *= down;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        s[r][u] = fast_exp2(s[r][u] - ref);
        l[r] += s[r][u];
        if (PT == kE4M3) s[r][u] *= vs[u];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float vf[8];
      vx[u].get(vf);
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int k = 0; k < 8; ++k) o[r][k] = fmaf(s[r][u], vf[k], o[r][k]);
    }
  }
  // the groups of a warp
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (bad) m[r] = NAN;
#pragma unroll
    for (int x2 = L; x2 < 32; x2 <<= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m[r], x2), top = m[r] != m[r] || m2 != m2 ? NAN : fmaxf(m[r], m2);
      const float ref = top == -INFINITY ? 0.0f : top;
      const float f1 = fast_exp2(m[r] - ref), f2 = fast_exp2(m2 - ref);
      l[r] = l[r] * f1 + __shfl_xor_sync(0xffffffffu, l[r], x2) * f2;
#pragma unroll
      for (int k = 0; k < 8; ++k) o[r][k] = o[r][k] * f1 + __shfl_xor_sync(0xffffffffu, o[r][k], x2) * f2;
      m[r] = top;
    }
    if (sub == 0) {
#pragma unroll
      for (int k = 0; k < 8; ++k) part_o[warp][r][d0 + k] = o[r][k];
      if (lane == 0) {
        part_m[warp][r] = m[r];
        part_l[warp][r] = l[r];
      }
    }
  }
  __syncthreads();
  // the warps of a CTA: a thread an element
  for (int x2 = threadIdx.x; x2 < R * D; x2 += kWarps * 32) {
    const int r = x2 / D, d = x2 % D;
    float top = -INFINITY, sum = 0.0f, out = 0.0f;
    bool lost = false;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      lost |= part_m[w][r] != part_m[w][r];
      top = fmaxf(top, part_m[w][r]);
    }
    const float ref = top == -INFINITY ? 0.0f : top;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float e = fast_exp2(part_m[w][r] - ref);
      sum += e * part_l[w][r];
      out += e * part_o[w][r][d];
    }
    cta_o[r][d] = out;
    if (d == 0) {
      cta_m[r] = lost ? NAN : top;
      cta_l[r] = sum;
    }
  }
  cg::cluster_group cluster = cg::this_cluster();
  if (f.splits > 1)
    cluster.sync();
  else
    __syncthreads();
  // the CTAs of the cluster: each writes its part of the elements
  for (int x2 = split * (kWarps * 32) + threadIdx.x; x2 < rows * D; x2 += f.splits * kWarps * 32) {
    const int r = x2 / D, d = x2 % D;
    float top = -INFINITY, sum = 0.0f, out = 0.0f;
    bool lost = n.bad;
    if (f.splits == 1) {
      top = cta_m[r];
      sum = cta_l[r];
      out = cta_o[r][d];
      lost |= top != top;
    } else {
      for (int i = 0; i < f.splits; ++i) {
        const float m2 = *cluster.map_shared_rank(&cta_m[r], i);
        lost |= m2 != m2;
        top = fmaxf(top, m2);
      }
      const float ref = top == -INFINITY ? 0.0f : top;
      for (int i = 0; i < f.splits; ++i) {
        const float e = fast_exp2(*cluster.map_shared_rank(&cta_m[r], i) - ref);
        sum += e * *cluster.map_shared_rank(&cta_l[r], i);
        out += e * *cluster.map_shared_rank(&cta_o[r][d], i);
      }
    }
    const int i = (row0 + r) / a.G, h = hk * a.G + (row0 + r) % a.G;
    const bool live = i < n.n;
    if (d < a.D)
      static_cast<float *>(a.out)[b * a.so.b + i * a.so.l + h * a.so.h + d] = lost ? NAN : live ? out / sum : 0.0f;
    if (d == 0 && a.lse)
      a.lse[(b * a.H + h) * a.Lq + i] = lost ? NAN : live ? (top + log2f(sum)) * kLn2 : -INFINITY;
  }
  if (f.splits > 1) cluster.sync();  // nobody leaves while its memory may be read
}

template <int PT, int R, int L> cudaError_t launch(const Step32Args &f, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(f.a.B * f.a.Hkv * f.groups * f.splits));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = f.splits;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = f.splits > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, paged_step32_kernel<PT, R, L>, f);
}
template <int PT, int R> cudaError_t by_width(const Step32Args &f, cudaStream_t s) {
  return f.a.D <= 64 ? launch<PT, R, 8>(f, s) : f.a.D <= 128 ? launch<PT, R, 16>(f, s) : launch<PT, R, 32>(f, s);
}
template <int PT> cudaError_t by_rows(const Step32Args &f, cudaStream_t s) {
  const long long rows = (long long)f.a.Lq * f.a.G;
  return rows <= 1   ? by_width<PT, 1>(f, s)
         : rows <= 2 ? by_width<PT, 2>(f, s)
         : rows <= 4 ? by_width<PT, 4>(f, s)
                     : by_width<PT, 8>(f, s);
}

}  // namespace

bool paged_step32_takes(const PagedArgs &a, int dtype, int cache_dtype) {
  const int unit = cache_dtype == kE4M3 ? 8 : 4;  // elements of an access
  const uintptr_t bytes = cache_dtype == kE4M3 ? 8 : 16;
  auto axis = [&](long long n, long long stride) { return n <= 1 || stride % unit == 0; };
  auto fits = [&](const Pages &p) {
    return (uintptr_t)p.data % bytes == 0 && axis(a.t.n_pages, p.s.b) && axis(1LL << a.t.page_bits, p.s.l) && axis(a.Hkv, p.s.h);
  };
  return dtype == kF32 && a.D % 8 == 0 && (long long)a.Lq * a.G <= kStepRows && fits(a.k) && fits(a.v);
}

cudaError_t launch_paged_step32(const PagedArgs &a, int cache_dtype, cudaStream_t stream) {
  Step32Args f = {};
  f.a = a;
  f.groups = (a.Lq * a.G + kCtaRows - 1) / kCtaRows;
  // a cluster's CTAs, while CTAs leave the GPU idle and each keeps 64 positions
  const long long units = a.B * a.Hkv * f.groups, most = (long long)a.t.max_pages << a.t.page_bits;
  const long long s = std::min<long long>({units > 0 ? 8 * kSMs / units : 1, (most + 63) / 64, 8});
  f.splits = 1;
  while (f.splits * 2 <= s) f.splits *= 2;
  return cache_dtype == kE4M3 ? by_rows<kE4M3>(f, stream) : by_rows<kF32>(f, stream);
}

}  // namespace tdt
