// tdt_attn_step.cu -- cross attention of few query rows (a decoding step, a small beam), every type.
//
// With R = Lq * G rows a key head (G query heads share it; 8 a CTA, more rows: more CTAs, which mostly find
// k and v in L2), the work is to read k and v once: 4 R flops an element read; bound by memory for one or two
// rows (6.3 TB/s in float32, 5.4 TB/s in bfloat16 at 64 x 16 heads of 64 and 750 frames, of 6.8 measured), by
// instructions above.  64 ragged x 750, 16 heads of 64, float16: 30 us, 4.9 TB/s.  1 x 200, 8 heads of 64: 4.3 us,
// latency.
// A cluster of S CTAs has one (utterance, key head); its CTAs take the frames in turns of equal parts, the
// warps of a CTA again.  In a warp a frame belongs to L lanes (8, 16 or 32, of 8 elements each), so a 16-byte
// load a lane (two for float32) reads 32 / L frames; U = 4 such groups of k and v are in flight (2 for
// float32 or more rows), and the next turn's are loaded while this one's are at work.  A lane holds its 8
// elements of each row of q and of the running output, and each group of L lanes its own running maximum and
// sum, so lanes exchange partial scores only:
//   s = q . k (log2 L shuffles), m' = max(m, s), l = l 2^(m - m') + 2^(s - m'), o = o 2^(m - m') + 2^(s - m') v
// The groups, the warps and then the CTAs of the cluster (over distributed shared memory) are joined in
// a fixed order.
#include <cooperative_groups.h>

#include <algorithm>

#include "tdt_attn_common.cuh"

namespace tdt {
namespace {

namespace cg = cooperative_groups;

constexpr int kCtaRows = 8;  // rows of a key head that a CTA has
constexpr int kWarps = 4;

struct StepArgs {
  AttnArgs a;
  int splits;  // CTAs of a cluster
  int groups;  // clusters that share the rows of a key head
};

// 8 elements as float32
template <int DT> struct Load8;
template <> struct Load8<kF32> {
  float4 x, y;
  __device__ __forceinline__ void load(const float *p) {
    x = __ldg(reinterpret_cast<const float4 *>(p));
    y = __ldg(reinterpret_cast<const float4 *>(p) + 1);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
  }
};
template <int DT> struct Load8 {
  typedef typename Elem<DT>::T E;
  uint4 x;
  __device__ __forceinline__ void load(const E *p) { x = __ldg(reinterpret_cast<const uint4 *>(p)); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const unsigned w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (DT == kBF16) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      }
    }
  }
};

// R rows at most, L lanes a frame
template <int DT, int R, int L>
__global__ void __launch_bounds__(kWarps * 32) attn_step_kernel(const __grid_constant__ StepArgs f) {
  typedef typename Elem<DT>::T E;
  constexpr int F = 32 / L;                    // frames of a group load
  constexpr int U = R <= 2 && DT != kF32 ? 4 : 2;  // group loads of a turn
  constexpr int D = L * 8;
  const AttnArgs &a = f.a;
  __shared__ float part_m[kWarps][R], part_l[kWarps][R];
  __shared__ __align__(16) float part_o[kWarps][R][D];
  __shared__ float cta_m[R], cta_l[R];
  __shared__ __align__(16) float cta_o[R][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane / L, d0 = lane % L * 8;
  const unsigned cluster_id = blockIdx.x / f.splits, unit = cluster_id / f.groups;  // = b * Hkv + hk
  const int split = blockIdx.x % f.splits, hk = unit % a.Hkv;
  const long long b = unit / a.Hkv;
  const Lens n = utt_lens(a, b);
  const int row0 = cluster_id % f.groups * R;
  const int rows = a.Lq * a.G - row0;          // row r: query (row0 + r) / G, head hk * G + (row0 + r) % G
  const bool wide = d0 < a.D;                  // D is a multiple of 8
  int2 range[R];
  float q[R][8], o[R][8], m[R], l[R];
  int first = 0x7fffffff, last = 0;
  const float c = a.scale * kLog2e;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int i = (row0 + r) / a.G;
    range[r] = r < rows ? row_range(a, b, i, n) : make_int2(0, 0);
    if (range[r].y > range[r].x) {
      first = min(first, range[r].x);
      last = max(last, range[r].y);
    }
    Load8<DT> x;
    if (wide && range[r].y > range[r].x) {
      x.load(static_cast<const E *>(a.q) + b * a.sq.b + i * a.sq.l + (hk * a.G + (row0 + r) % a.G) * a.sq.h + d0);
      x.get(q[r]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) q[r][k] = 0.0f;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      q[r][k] *= c;  // scores in base 2
      o[r][k] = 0.0f;
    }
    m[r] = -INFINITY;
    l[r] = 0.0f;
  }
  if (last > first) {
    // parts of whole turns of F * U frames, over the splits and then the warps
    const int turn = F * U, turns = (last - first + turn - 1) / turn;
    const int2 t = share_of(turns, split * kWarps + warp, f.splits * kWarps);
    const E *kp = static_cast<const E *>(a.k) + b * a.sk.b + hk * a.sk.h + d0;
    const E *vp = static_cast<const E *>(a.v) + b * a.sv.b + hk * a.sv.h + d0;
    Load8<DT> kx[U], vx[U], kn[U], vn[U];
    auto load = [&](int x, Load8<DT> (&ko)[U], Load8<DT> (&vo)[U]) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int j = first + x * turn + sub + u * F;
        ko[u] = Load8<DT>{};
        vo[u] = Load8<DT>{};
        if (j < last && wide) {  // frames past `last` are not read
          ko[u].load(kp + (long long)j * a.sk.l);
          vo[u].load(vp + (long long)j * a.sv.l);
        }
      }
    };
    if (t.x < t.y) load(t.x, kn, vn);
    for (int x = t.x; x < t.y; ++x) {
      const int j0 = first + x * turn + sub;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        kx[u] = kn[u];
        vx[u] = vn[u];
      }
      if (x + 1 < t.y) load(x + 1, kn, vn);
      float s[R][U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float kf[8];
        kx[u].get(kf);
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
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float top = m[r];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int j = j0 + u * F;
          if (j < range[r].x || j >= range[r].y) s[r][u] = -INFINITY;
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
  }
  // the groups of a warp
#pragma unroll
  for (int r = 0; r < R; ++r) {
#pragma unroll
    for (int x = L; x < 32; x <<= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m[r], x), top = fmaxf(m[r], m2);
      const float ref = top == -INFINITY ? 0.0f : top;
      const float f1 = fast_exp2(m[r] - ref), f2 = fast_exp2(m2 - ref);
      l[r] = l[r] * f1 + __shfl_xor_sync(0xffffffffu, l[r], x) * f2;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        o[r][k] = o[r][k] * f1 + __shfl_xor_sync(0xffffffffu, o[r][k], x) * f2;
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
  for (int x = threadIdx.x; x < R * D; x += kWarps * 32) {
    const int r = x / D, d = x % D;
    float top = -INFINITY, sum = 0.0f, out = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, part_m[w][r]);
    const float ref = top == -INFINITY ? 0.0f : top;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float g = fast_exp2(part_m[w][r] - ref);
      sum += g * part_l[w][r];
      out += g * part_o[w][r][d];
    }
    cta_o[r][d] = out;
    if (d == 0) {
      cta_m[r] = top;
      cta_l[r] = sum;
    }
  }
  cg::cluster_group cluster = cg::this_cluster();
  if (f.splits > 1)
    cluster.sync();
  else
    __syncthreads();
  // the CTAs of the cluster: each writes its part of the elements
  for (int x = split * (kWarps * 32) + threadIdx.x; x < R * D; x += f.splits * kWarps * 32) {
    const int r = x / D, d = x % D;
    if (r >= rows) continue;
    float top = -INFINITY, sum = 0.0f, out = 0.0f;
    if (f.splits == 1) {
      top = cta_m[r];
      sum = cta_l[r];
      out = cta_o[r][d];
    } else {
      for (int i = 0; i < f.splits; ++i) top = fmaxf(top, *cluster.map_shared_rank(&cta_m[r], i));
      const float ref = top == -INFINITY ? 0.0f : top;
      for (int i = 0; i < f.splits; ++i) {
        const float g = fast_exp2(*cluster.map_shared_rank(&cta_m[r], i) - ref);
        sum += g * *cluster.map_shared_rank(&cta_l[r], i);
        out += g * *cluster.map_shared_rank(&cta_o[r][d], i);
      }
    }
    const int i = (row0 + r) / a.G, h = hk * a.G + (row0 + r) % a.G;
    const float v = n.bad ? NAN : sum == 0.0f ? 0.0f : out / sum;
    if (d < a.D)
      static_cast<E *>(const_cast<void *>(a.out))[b * a.so.b + i * a.so.l + h * a.so.h + d] =
          Elem<DT>::from_float(v);
    if (d == 0 && a.lse)
      a.lse[(b * a.H + h) * a.Lq + i] =
          n.bad ? NAN : sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
  }
  if (f.splits > 1) cluster.sync();  // nobody leaves while its memory may be read
}

template <int DT, int R, int L> cudaError_t launch(const StepArgs &f, cudaStream_t stream) {
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
  return cudaLaunchKernelEx(&cfg, attn_step_kernel<DT, R, L>, f);
}
template <int DT, int R> cudaError_t by_width(const StepArgs &f, cudaStream_t s) {
  return f.a.D <= 64 ? launch<DT, R, 8>(f, s)
                     : f.a.D <= 128 ? launch<DT, R, 16>(f, s) : launch<DT, R, 32>(f, s);
}
template <int DT> cudaError_t by_rows(const StepArgs &f, cudaStream_t s) {
  const int rows = f.a.Lq * f.a.G;
  return rows <= 1 ? by_width<DT, 1>(f, s)
                   : rows <= 2 ? by_width<DT, 2>(f, s)
                               : rows <= 4 ? by_width<DT, 4>(f, s) : by_width<DT, 8>(f, s);
}

}  // namespace

bool attn_step_fits(const AttnArgs &a, int dtype, bool tc_fits) {
  const long long unit = dtype == kF32 ? 4 : 8;  // elements of 16 bytes
  auto fits = [&](const void *p, const Strides &s, int L, int H) {
    return (uintptr_t)p % 16 == 0 && (a.B == 1 || s.b % unit == 0) && (L == 1 || s.l % unit == 0) &&
           (H == 1 || s.h % unit == 0);
  };
  // The arithmetic of R rows is on the CUDA cores: where the tensor-core kernel can take the call, it
  // is as fast from 3 rows on (bfloat16, 64 x 16 heads of 64, 750 frames: 1 row 36 us against 50,
  // 2 rows 40 against 50, 4 rows 74 against 51; the step then is bound by its instructions).  In float32
  // the tensor cores take six products and planes of k and v made beforehand, and this kernel is ahead up
  // to about 32 rows (64 x 8 heads of 64, 750 frames: 16 rows 105 us against 175, 32 rows 194 against 177,
  // of three query heads a key head 193 against 339; 200 frames, one utterance: 8 against 14).
  const int most = tc_fits && dtype != kF32 ? 2 : kStepRows;
  return (long long)a.Lq * a.G <= most && a.D % 8 == 0 && fits(a.q, a.sq, a.Lq, a.H) &&
         fits(a.k, a.sk, a.Lk, a.Hkv) && fits(a.v, a.sv, a.Lk, a.Hkv);
}

cudaError_t launch_attn_step(const AttnArgs &a, int dtype, cudaStream_t stream) {
  StepArgs f = {};
  f.a = a;
  // a cluster's CTAs, while CTAs leave the GPU idle (8 of 4 warps an SM) and each keeps 64 frames
  f.groups = (a.Lq * a.G + kCtaRows - 1) / kCtaRows;
  const long long units = a.B * a.Hkv * f.groups;
  long long s = units > 0 ? 8 * kSMs / units : 1;
  s = std::min<long long>({s, (a.Lk + 63) / 64, 8});
  f.splits = 1;
  while (f.splits * 2 <= s) f.splits *= 2;
  return dtype == kF32   ? by_rows<kF32>(f, stream)
         : dtype == kF16 ? by_rows<kF16>(f, stream)
                         : by_rows<kBF16>(f, stream);
}

}  // namespace tdt
