// tdt_attn_api.cu -- the C ABI of cross attention (include/tdt_decoder.h):
// argument checks, workspace and the choice of kernels.
#include <math.h>

#include <algorithm>

#include "../../include/tdt_decoder.h"
#include "tdt_attn_common.cuh"

namespace tdt {
namespace {

int check_sizes(const int64_t sizes[6], int dtype) {
  if (!sizes) return TDT_ERR_NULL_POINTER;
  if (dtype != TDT_DTYPE_F32 && dtype != TDT_DTYPE_F16 && dtype != TDT_DTYPE_BF16)
    return TDT_ERR_BAD_DTYPE;
  const int64_t B = sizes[0], Lq = sizes[1], Lk = sizes[2], H = sizes[3], Hkv = sizes[4],
                D = sizes[5];
  if (H < 1 || Hkv < 1 || H % Hkv != 0 || H > 65536 || D < 1 || D > kMaxHeadDim)
    return TDT_ERR_BAD_HEADS;
  const int64_t limit = (int64_t)1 << 30;
  if (B < 0 || Lq < 0 || Lk < 0 || B >= limit || Lq >= limit || Lk >= limit)
    return TDT_ERR_BAD_SIZES;
  // one block a tile of 32 rows at the least: the grid has fewer than 2^31
  if (B * H >= ((int64_t)1 << 31) / std::max<int64_t>(1, (std::max(Lq, Lk) + 31) / 32))
    return TDT_ERR_BAD_SIZES;
  return TDT_OK;
}

// No two elements of an output may share an address: sorted by stride, each axis of more
// than one element steps over the whole extent of those below it.
bool writable(const Strides &s, int64_t B, int64_t L, int64_t H, int64_t D) {
  struct Axis {
    int64_t n, stride;
  } x[3] = {{B, s.b}, {L, s.l}, {H, s.h}};
  std::sort(x, x + 3, [](const Axis &p, const Axis &q) { return p.stride < q.stride; });
  int64_t extent = D;
  for (const Axis &p : x)
    if (p.n > 1) {
      if (p.stride < extent) return false;
      extent = p.stride * (p.n - 1) + extent;
    }
  return true;
}

Strides strides_of(const int64_t *s) { return Strides{s[0], s[1], s[2]}; }

int fill(AttnArgs *a, const int64_t sizes[6], const int64_t *strides, int n_tensors, int dtype,
         const int64_t *k_lens, const int64_t *q_lens, const int32_t *windows, double scale,
         const void *workspace, size_t workspace_bytes, int backward) {
  if (!strides) return TDT_ERR_NULL_POINTER;
  const int rc = check_sizes(sizes, dtype);
  if (rc != TDT_OK) return rc;
  const float f = (float)scale;
  if (!(f > 0.0f) || !isfinite(f)) return TDT_ERR_BAD_SCALE;
  for (int i = 0; i < 3 * n_tensors; ++i)
    if (strides[i] < 0) return TDT_ERR_BAD_STRIDES;
  a->B = sizes[0];
  a->Lq = (int)sizes[1];
  a->Lk = (int)sizes[2];
  a->H = (int)sizes[3];
  a->Hkv = (int)sizes[4];
  a->D = (int)sizes[5];
  a->G = a->H / a->Hkv;
  a->sq = strides_of(strides);
  a->sk = strides_of(strides + 3);
  a->sv = strides_of(strides + 6);
  a->so = strides_of(strides + 9);
  a->k_lens = reinterpret_cast<const long long *>(k_lens);
  a->q_lens = reinterpret_cast<const long long *>(q_lens);
  a->windows = windows;
  a->scale = f;
  if (((uintptr_t)k_lens | (uintptr_t)q_lens | (uintptr_t)windows) % 8 != 0)
    return TDT_ERR_BAD_ALIGNMENT;
  const size_t need = tdt_cross_attn_workspace_size(sizes, dtype, backward);
  if (need > 0) {
    if (!workspace) return TDT_ERR_NULL_POINTER;
    if ((uintptr_t)workspace % 256 != 0) return TDT_ERR_BAD_ALIGNMENT;
    if (workspace_bytes < need) return TDT_ERR_WORKSPACE_TOO_SMALL;
  }
  return TDT_OK;
}

size_t delta_bytes(const int64_t sizes[6]) {
  return ((size_t)sizes[0] * (size_t)sizes[1] * (size_t)sizes[3] * 4 + 255) / 256 * 256;
}

bool aligned(int dtype, std::initializer_list<const void *> ptrs) {
  const uintptr_t es = dtype == TDT_DTYPE_F32 ? 4 : 2;
  for (const void *p : ptrs)
    if ((uintptr_t)p % es != 0) return false;
  return true;
}

}  // namespace
}  // namespace tdt

extern "C" {

size_t tdt_cross_attn_workspace_size(const int64_t sizes[6], int dtype, int backward) {
  using namespace tdt;
  if (check_sizes(sizes, dtype) != TDT_OK) return 0;
  const int G = (int)(sizes[3] / sizes[4]), D = (int)sizes[5];
  const bool tc = attn_tc_takes(dtype, sizes[1], sizes[2], G, D, backward != 0);
  if (attn_planes_takes(dtype, sizes[1], sizes[2], G, D, backward != 0))
    return (backward ? delta_bytes(sizes) : 0) +
           attn_planes_workspace(sizes[0], sizes[1], sizes[2], (int)sizes[3], (int)sizes[4], backward != 0);
  if (!backward)
    return tc ? attn_fwd_tc_workspace(sizes[0], sizes[1], sizes[2], (int)sizes[3], (int)sizes[4],
                                      (int)sizes[5], dtype)
              : 0;
  return delta_bytes(sizes) + (tc ? attn_bwd_tc_workspace(sizes[0], sizes[1], sizes[2],
                                                          (int)sizes[3], (int)sizes[4],
                                                          (int)sizes[5], dtype)
                                  : 0);
}

int tdt_cross_attn_fwd(const void *q, const void *k, const void *v, const int64_t sizes[6],
                       const int64_t strides[12], int dtype, const int64_t *k_lens,
                       const int64_t *q_lens, const int32_t *windows, double scale, void *out,
                       float *lse, void *workspace, size_t workspace_bytes, void *stream) {
  using namespace tdt;
  AttnArgs a = {};
  const int rc = fill(&a, sizes, strides, 4, dtype, k_lens, q_lens, windows, scale, workspace,
                      workspace_bytes, 0);
  if (rc != TDT_OK) return rc;
  if (a.B == 0 || a.Lq == 0) return TDT_OK;
  if (!q || !out || (a.Lk > 0 && (!k || !v))) return TDT_ERR_NULL_POINTER;
  if (!aligned(dtype, {q, k, v, out}) || (uintptr_t)lse % 4 != 0) return TDT_ERR_BAD_ALIGNMENT;
  if (!writable(a.so, a.B, a.Lq, a.H, a.D)) return TDT_ERR_BAD_STRIDES;
  a.q = q;
  a.k = k;
  a.v = v;
  a.out = out;
  a.lse = lse;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool tc = attn_fwd_tc_fits(a, dtype);
  const cudaError_t e = attn_step_fits(a, dtype, tc)        ? launch_attn_step(a, dtype, s)
                        : tc                                ? launch_attn_fwd_tc(a, dtype, workspace, s)
                        : attn_planes_fits(a, dtype, false) ? launch_attn_planes(a, false, workspace, s)
                                                            : launch_attn_general_fwd(a, dtype, s);
  return e == cudaSuccess ? TDT_OK : TDT_ERR_CUDA;
}

int tdt_cross_attn_bwd(const void *grad_out, const void *q, const void *k, const void *v,
                       const void *out, const float *lse, const int64_t sizes[6],
                       const int64_t strides[24], int dtype, const int64_t *k_lens,
                       const int64_t *q_lens, const int32_t *windows, double scale, void *dq,
                       void *dk, void *dv, void *workspace, size_t workspace_bytes,
                       void *stream) {
  using namespace tdt;
  AttnArgs a = {};
  const int rc = fill(&a, sizes, strides, 8, dtype, k_lens, q_lens, windows, scale, workspace,
                      workspace_bytes, 1);
  if (rc != TDT_OK) return rc;
  if (a.B == 0 || (a.Lq == 0 && a.Lk == 0)) return TDT_OK;
  if (a.Lq > 0 && (!grad_out || !q || !out || !lse || !dq)) return TDT_ERR_NULL_POINTER;
  if (a.Lk > 0 && (!k || !v || !dk || !dv)) return TDT_ERR_NULL_POINTER;
  if (!aligned(dtype, {grad_out, q, k, v, out, dq, dk, dv}) || (uintptr_t)lse % 4 != 0)
    return TDT_ERR_BAD_ALIGNMENT;
  a.sgo = strides_of(strides + 12);
  a.sdq = strides_of(strides + 15);
  a.sdk = strides_of(strides + 18);
  a.sdv = strides_of(strides + 21);
  if (!writable(a.sdq, a.B, a.Lq, a.H, a.D) || !writable(a.sdk, a.B, a.Lk, a.Hkv, a.D) ||
      !writable(a.sdv, a.B, a.Lk, a.Hkv, a.D))
    return TDT_ERR_BAD_STRIDES;
  a.q = q;
  a.k = k;
  a.v = v;
  a.out = out;
  a.go = grad_out;
  a.lse = const_cast<float *>(lse);
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.delta = static_cast<float *>(workspace);
  void *rest = static_cast<char *>(workspace) + delta_bytes(sizes);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = attn_bwd_tc_fits(a, dtype)         ? launch_attn_bwd_tc(a, dtype, rest, s)
                        : attn_planes_fits(a, dtype, true) ? launch_attn_planes(a, true, rest, s)
                                                           : launch_attn_general_bwd(a, dtype, s);
  return e == cudaSuccess ? TDT_OK : TDT_ERR_CUDA;
}

}  // extern "C"
