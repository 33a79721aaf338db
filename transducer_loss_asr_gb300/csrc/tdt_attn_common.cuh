// tdt_attn_common.cuh -- what the cross-attention kernels share: the argument
// block, which frames a query sees, and the launchers.
#pragma once

#include "tdt_common.cuh"

namespace tdt {

constexpr int kMaxHeadDim = 256;
constexpr int kSMs = 152;  // of a GB300
constexpr float kLn2 = 0.69314718055994531f;

// Element strides of (batch, position, head); the head's elements are contiguous.
struct Strides {
  long long b, l, h;
};

// One call's arguments, passed to the kernels by value.
struct AttnArgs {
  const void *q, *k, *v, *out, *go;  // out: written by the forward kernels
  void *dq, *dk, *dv;
  float *lse;                        // [B, H, Lq] or NULL (forward only)
  float *delta;                      // workspace, [B, H, Lq]: grad_out . out of each query
  Strides sq, sk, sv, so, sgo, sdq, sdk, sdv;
  long long B;
  int Lq, Lk, H, Hkv, G, D;          // G = H / Hkv
  const long long *k_lens, *q_lens;  // NULL: all
  const int *windows;                // [B, Lq, 2] or NULL
  float scale;
};

// Lengths of utterance b.  Lengths outside the tensors see nothing (bad).
struct Lens {
  int nq, nk;
  bool bad;
};
__device__ __forceinline__ Lens utt_lens(const AttnArgs &a, long long b) {
  const long long nk = a.k_lens ? a.k_lens[b] : a.Lk;
  const long long nq = a.q_lens ? a.q_lens[b] : a.Lq;
  Lens n;
  n.bad = nk < 0 || nk > a.Lk || nq < 0 || nq > a.Lq;
  n.nk = n.bad ? 0 : (int)nk;
  n.nq = n.bad ? 0 : (int)nq;
  return n;
}

// Frames [x, y) that query i of utterance b sees; x = y = 0 if none.
__device__ __forceinline__ int2 row_range(const AttnArgs &a, long long b, int i, const Lens &n) {
  int lo = 0, hi = n.nk;
  if (i >= n.nq) return make_int2(0, 0);
  if (a.windows) {
    const int2 w = *reinterpret_cast<const int2 *>(a.windows + (b * a.Lq + i) * 2);
    lo = max(lo, w.x);
    hi = min(hi, w.y);
  }
  return hi > lo ? make_int2(lo, hi) : make_int2(0, 0);
}

// Steps [first, last) of `all` that part `i` of `parts` takes.
__device__ __forceinline__ int2 share_of(int all, int i, int parts) {
  if (parts == 1) return make_int2(0, all);
  const int q = all / parts, more = all % parts;
  const int first = q * i + min(i, more);
  return make_int2(first, first + q + (i < more ? 1 : 0));
}

// The hull of the frame ranges of a CTA's rows.  Warps with rows note theirs; after a barrier every
// thread reads the hull of all.  Without windows it is known beforehand.
struct Hull {
  int lo[8], hi[8];
};
__device__ __forceinline__ void hull_note(Hull &h, int warp, int2 range) {
  const int lo = __reduce_min_sync(0xffffffffu, range.y > range.x ? range.x : 0x7fffffff);
  const int hi = __reduce_max_sync(0xffffffffu, range.y);
  if ((threadIdx.x & 31) == 0) {
    h.lo[warp] = lo;
    h.hi[warp] = hi;
  }
}
template <int WARPS> __device__ __forceinline__ int2 hull_of(const Hull &h) {
  int lo = h.lo[0], hi = h.hi[0];
#pragma unroll
  for (int i = 1; i < WARPS; ++i) {
    lo = min(lo, h.lo[i]);
    hi = max(hi, h.hi[i]);
  }
  return hi > 0 ? make_int2(lo, hi) : make_int2(0, 0);
}

// dot of the first `n` of N elements of two rows, n a multiple of a 16-byte load's elements; every load is
// in flight at once.  `xx`, if given: the square of x's norm.
template <int DT, int N>
__device__ __forceinline__ float dot_rows(const void *x, const void *y, int n, float *xx = nullptr) {
  typedef typename Elem<DT>::T E;
  constexpr int W = 16 / (int)sizeof(E);
  uint4 xv[N / W], yv[N / W];
#pragma unroll
  for (int d = 0; d < N; d += W) {
    xv[d / W] = yv[d / W] = make_uint4(0, 0, 0, 0);
    if (d < n) {
      xv[d / W] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const E *>(x) + d));
      yv[d / W] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const E *>(y) + d));
    }
  }
  float s = 0.0f, s2 = 0.0f;
#pragma unroll
  for (int d = 0; d < N / W; ++d) {
    const E *xe = reinterpret_cast<const E *>(&xv[d]), *ye = reinterpret_cast<const E *>(&yv[d]);
#pragma unroll
    for (int k = 0; k < W; ++k) {
      const float f = Elem<DT>::to_float(xe[k]);
      s = fmaf(f, Elem<DT>::to_float(ye[k]), s);
      if (xx) s2 = fmaf(f, f, s2);
    }
  }
  if (xx) *xx = s2;
  return s;
}

// Tensor-core kernels: which calls they take, their workspace (of the sizes alone), and the launch.
bool attn_tc_takes(int dtype, long long Lq, long long Lk, int G, int D, bool backward);  // by type and sizes
bool attn_fwd_tc_fits(const AttnArgs &a, int dtype);                      // and by strides and alignment
size_t attn_fwd_tc_workspace(long long B, long long Lq, long long Lk, int H, int Hkv, int D, int dtype);
cudaError_t launch_attn_fwd_tc(const AttnArgs &a, int dtype, void *workspace, cudaStream_t stream);
// Few rows: a kernel that reads k and v at memory speed.
constexpr int kStepRows = 32;  // rows of a key head at most
bool attn_step_fits(const AttnArgs &a, int dtype, bool tc_fits);
cudaError_t launch_attn_step(const AttnArgs &a, int dtype, cudaStream_t stream);
bool attn_bwd_tc_fits(const AttnArgs &a, int dtype);
size_t attn_bwd_tc_workspace(long long B, long long Lq, long long Lk, int H, int Hkv, int D, int dtype);
cudaError_t launch_attn_bwd_tc(const AttnArgs &a, int dtype, void *workspace, cudaStream_t stream);
// Float32 heads of 65 to 128 elements, as bfloat16 planes.
bool attn_planes_takes(int dtype, long long Lq, long long Lk, int G, int D, bool backward);
bool attn_planes_fits(const AttnArgs &a, int dtype, bool backward);
size_t attn_planes_workspace(long long B, long long Lq, long long Lk, int H, int Hkv, bool backward);
cudaError_t launch_attn_planes(const AttnArgs &a, bool backward, void *workspace, cudaStream_t stream);
// Heads that share a row tile, of a group of G: the largest power of two that divides G, up to 16.
int attn_row_pack(int G);
// CUDA-core kernels: every other call.
cudaError_t launch_attn_general_fwd(const AttnArgs &a, int dtype, cudaStream_t stream);
cudaError_t launch_attn_general_bwd(const AttnArgs &a, int dtype, cudaStream_t stream);

}  // namespace tdt
