// tdt_paged_api.cu -- the C ABI of the paged cache (include/tdt_decoder.h): argument checks, workspace and the
// choice of kernels.
#include <math.h>

#include <algorithm>

#include "../../include/tdt_decoder.h"
#include "tdt_paged.cuh"

namespace tdt {
namespace {

bool known(int dtype) { return dtype == TDT_DTYPE_F32 || dtype == TDT_DTYPE_F16 || dtype == TDT_DTYPE_BF16; }
uintptr_t size_of(int dtype) { return dtype == TDT_DTYPE_F32 ? 4 : dtype == TDT_DTYPE_E4M3 ? 1 : 2; }
Strides strides_of(const int64_t *s) { return Strides{s[0], s[1], s[2]}; }

// No two elements of an output may share an address (as in the checks of cross attention).
bool apart(const Strides &s, int64_t B, int64_t L, int64_t H, int64_t D) {
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

int page_bits_of(int64_t page_size) {
  int bits = 0;
  while ((int64_t)1 << bits < page_size) ++bits;
  return bits;
}

int check_cache(const tdt_paged_cache *c, int dtype, bool any_type) {
  if (!c) return TDT_ERR_NULL_POINTER;
  if (!known(dtype)) return TDT_ERR_BAD_DTYPE;
  if (!known(c->dtype) && c->dtype != TDT_DTYPE_E4M3) return TDT_ERR_BAD_DTYPE;
  if (!any_type && c->dtype != TDT_DTYPE_E4M3 && c->dtype != dtype) return TDT_ERR_BAD_DTYPE;
  if (c->n_heads < 1 || c->n_heads > 65536 || c->head_dim < 1 || c->head_dim > kMaxHeadDim) return TDT_ERR_BAD_HEADS;
  if (c->n_pages < 1 || c->n_pages > 0x7fffffff || c->page_size < 1 || c->page_size > 65536 ||
      (c->page_size & (c->page_size - 1)))
    return TDT_ERR_BAD_PAGES;
  const bool quantised = c->dtype == TDT_DTYPE_E4M3;
  for (int i = 0; i < (quantised ? 12 : 6); ++i)
    if (c->strides[i] < 0) return TDT_ERR_BAD_STRIDES;
  return TDT_OK;
}
int check_cache_memory(const tdt_paged_cache *c, bool written) {
  const bool quantised = c->dtype == TDT_DTYPE_E4M3;
  if (!c->k_pages || !c->v_pages || (quantised && (!c->k_scales || !c->v_scales))) return TDT_ERR_NULL_POINTER;
  if (((uintptr_t)c->k_pages | (uintptr_t)c->v_pages) % size_of(c->dtype)) return TDT_ERR_BAD_ALIGNMENT;
  if (written)
    for (int i = 0; i < (quantised ? 4 : 2); ++i)
      if (!apart(strides_of(c->strides + 3 * i), c->n_pages, c->page_size, c->n_heads, i < 2 ? c->head_dim : 1))
        return TDT_ERR_BAD_STRIDES;
  return TDT_OK;
}

Pages pages_of(const tdt_paged_cache *c, bool values) {
  Pages p = {};
  p.data = values ? c->v_pages : c->k_pages;
  p.s = strides_of(c->strides + (values ? 3 : 0));
  if (c->dtype == TDT_DTYPE_E4M3) {
    p.scales = values ? c->v_scales : c->k_scales;
    p.ss = strides_of(c->strides + (values ? 9 : 6));
  }
  return p;
}

// The table and lengths; max_pages * page_size < 2^30 holds.
int fill_table(PageTable *t, const tdt_paged_cache *c, const int32_t *ids, int64_t stride, const int64_t *kv_lens,
               const int64_t *q_lens, int64_t max_pages) {
  if (stride < 0) return TDT_ERR_BAD_STRIDES;
  if (!kv_lens || (!ids && max_pages > 0)) return TDT_ERR_NULL_POINTER;
  if ((uintptr_t)ids % 4 || ((uintptr_t)kv_lens | (uintptr_t)q_lens) % 8) return TDT_ERR_BAD_ALIGNMENT;
  t->ids = ids;
  t->stride = stride;
  t->kv_lens = reinterpret_cast<const long long *>(kv_lens);
  t->q_lens = reinterpret_cast<const long long *>(q_lens);
  t->n_pages = (int)c->n_pages;
  t->page_bits = page_bits_of(c->page_size);
  t->max_pages = (int)max_pages;
  return TDT_OK;
}

int check_rows(const int64_t *sizes, const tdt_paged_cache *c, int64_t heads, int64_t max_pages) {
  const int64_t limit = (int64_t)1 << 30, B = sizes[0], L = sizes[1];
  if (B < 0 || L < 0 || B >= limit || L >= limit) return TDT_ERR_BAD_SIZES;
  if (max_pages < 0 || max_pages >= limit || max_pages * c->page_size >= limit) return TDT_ERR_BAD_PAGES;
  // one block a row and head at the most: grids have fewer than 2^31
  if (L > 0 && B * L >= ((int64_t)1 << 31) / heads) return TDT_ERR_BAD_SIZES;
  return TDT_OK;
}

int cache_call(CacheArgs *a, const int64_t sizes[3], const int64_t strides[6], int dtype, bool any_type,
               const tdt_paged_cache *c, const int32_t *table, int64_t table_stride, const int64_t *kv_lens,
               const int64_t *q_lens) {
  if (!sizes || !strides) return TDT_ERR_NULL_POINTER;
  int rc = check_cache(c, dtype, any_type);
  if (rc == TDT_OK) rc = check_rows(sizes, c, c->n_heads, sizes[2]);
  if (rc != TDT_OK) return rc;
  for (int i = 0; i < 6; ++i)
    if (strides[i] < 0) return TDT_ERR_BAD_STRIDES;
  a->sk = strides_of(strides);
  a->sv = strides_of(strides + 3);
  a->pk = pages_of(c, false);
  a->pv = pages_of(c, true);
  a->L = (int)sizes[1];
  a->Hkv = (int)c->n_heads;
  a->D = (int)c->head_dim;
  a->B = sizes[0];
  if (a->B == 0 || a->L == 0) return TDT_OK;
  return fill_table(&a->t, c, table, table_stride, kv_lens, q_lens, sizes[2]);
}

// What the choice of kernels goes by: sizes and the cache.
PagedArgs attn_args(const int64_t sizes[4], const tdt_paged_cache *c) {
  PagedArgs a = {};
  a.B = sizes[0];
  a.Lq = (int)sizes[1];
  a.H = (int)sizes[2];
  a.Hkv = (int)c->n_heads;
  a.G = a.H / a.Hkv;
  a.D = (int)c->head_dim;
  a.k = pages_of(c, false);
  a.v = pages_of(c, true);
  a.t.n_pages = (int)c->n_pages;
  a.t.page_bits = page_bits_of(c->page_size);
  a.t.max_pages = (int)sizes[3];
  return a;
}
enum Way { kStep, kStep32, kTensor, kGather };
// The few-rows kernel reads k and v once for each 16 rows of a key head, the tensor-core kernel once for each row tile of each
// group of P heads; e4m3 pages are laid out densely for the latter first.  Costs of a read in microseconds at 16 x 2,000
// positions of 4 heads of 128, bfloat16 and e4m3: 18 (12) of the first kernel, 29 of the second, 24 of the layout (20 rows of 4
// heads in a group 37 us against 30, 12 rows 19 against 29; e4m3 64 rows 49 against 53, 96 rows 88 against 55; float16, 24 rows of 3
// heads, which do not share a tile, 84 against 184 at 58 x 6,800).
Way way_of(const PagedArgs &a, int dtype, int cache_dtype) {
  const bool step = paged_step_takes(a, dtype, cache_dtype), e8 = cache_dtype == kE4M3;
  const int P = attn_row_pack(a.G);
  const long long few = ((long long)a.Lq * a.G + 15) / 16, many = a.G / P * (((long long)a.Lq * P + 127) / 128);
  if (step && (e8 ? 12 * few <= 24 + 29 * many : 18 * few <= 29 * many)) return kStep;
  if (paged_step32_takes(a, dtype, cache_dtype)) return kStep32;
  // the few-rows kernel stands in where q or out does not suit TMA
  return step && dtype == cache_dtype && paged_tc_takes(a, dtype) ? kTensor : kGather;
}

// Scratch of a call that gathers: dense k and v, windows, lengths, then cross attention's own.
struct GatherSpace {
  size_t k, v, windows, lens, rest, total;
  int64_t sizes[6];  // of cross attention
};
GatherSpace gather_space(const int64_t sizes[4], int dtype, const tdt_paged_cache *c) {
  GatherSpace s = {};
  const int64_t L = sizes[3] * c->page_size;
  const int64_t all[6] = {sizes[0], sizes[1], L, sizes[2], c->n_heads, c->head_dim};
  std::copy(all, all + 6, s.sizes);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  const size_t dense = (size_t)(sizes[0] * L) * (size_t)(c->n_heads * c->head_dim) * size_of(dtype);
  s.k = take(dense);
  s.v = take(dense);
  s.windows = take((size_t)(sizes[0] * sizes[1]) * 8);
  s.lens = take((size_t)sizes[0] * 8);
  s.rest = at;
  s.total = at + tdt_cross_attn_workspace_size(s.sizes, dtype, 0);
  return s;
}

int attend_gathered(const PagedArgs &a, const int64_t sizes[4], const int64_t strides[6], int dtype,
                    const tdt_paged_cache *c, void *workspace, size_t bytes, cudaStream_t stream) {
  const GatherSpace at = gather_space(sizes, dtype, c);
  char *ws = static_cast<char *>(workspace);
  GatherArgs f = {};
  const int64_t L = at.sizes[2], Hkv = c->n_heads, D = c->head_dim;
  f.c.k = ws + at.k;
  f.c.v = ws + at.v;
  f.c.sk = f.c.sv = Strides{L * Hkv * D, Hkv * D, D};
  f.c.pk = a.k;
  f.c.pv = a.v;
  f.c.t = a.t;
  f.c.L = (int)L;
  f.c.Hkv = (int)Hkv;
  f.c.D = (int)D;
  f.c.B = a.B;
  f.Lq = a.Lq;
  f.windows = reinterpret_cast<int2 *>(ws + at.windows);
  f.lens = reinterpret_cast<long long *>(ws + at.lens);
  if (launch_gather(f, dtype, c->dtype, stream) != cudaSuccess) return TDT_ERR_CUDA;
  const int64_t dense[3] = {L * Hkv * D, Hkv * D, D};
  int64_t all[12];
  std::copy(strides, strides + 3, all);
  std::copy(dense, dense + 3, all + 3);
  std::copy(dense, dense + 3, all + 6);
  std::copy(strides + 3, strides + 6, all + 9);
  return tdt_cross_attn_fwd(a.q, f.c.k, f.c.v, at.sizes, all, dtype, reinterpret_cast<const int64_t *>(f.lens),
                            reinterpret_cast<const int64_t *>(a.t.q_lens), reinterpret_cast<const int32_t *>(f.windows), a.scale, a.out, a.lse, ws + at.rest,
                            bytes - at.rest, stream);
}

int check_attn(const int64_t sizes[4], int dtype, const tdt_paged_cache *c) {
  if (!sizes) return TDT_ERR_NULL_POINTER;
  int rc = check_cache(c, dtype, false);
  if (rc != TDT_OK) return rc;
  if (sizes[2] < 1 || sizes[2] > 65536 || sizes[2] % c->n_heads) return TDT_ERR_BAD_HEADS;
  return check_rows(sizes, c, sizes[2], sizes[3]);
}

}  // namespace
}  // namespace tdt

extern "C" {

int tdt_cache_write(const void *k, const void *v, const int64_t sizes[3], const int64_t strides[6], int dtype,
                    const tdt_paged_cache *cache, const int32_t *page_table, int64_t table_stride,
                    const int64_t *kv_lens, const int64_t *q_lens, void *stream) {
  using namespace tdt;
  CacheArgs a = {};
  int rc = cache_call(&a, sizes, strides, dtype, false, cache, page_table, table_stride, kv_lens, q_lens);
  if (rc != TDT_OK || a.B == 0 || a.L == 0) return rc;
  if (!k || !v) return TDT_ERR_NULL_POINTER;
  if (((uintptr_t)k | (uintptr_t)v) % size_of(dtype)) return TDT_ERR_BAD_ALIGNMENT;
  rc = check_cache_memory(cache, true);
  if (rc != TDT_OK) return rc;
  a.k = const_cast<void *>(k);
  a.v = const_cast<void *>(v);
  const cudaError_t e = launch_cache_write(a, dtype, cache->dtype, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? TDT_OK : TDT_ERR_CUDA;
}

int tdt_cache_read(const tdt_paged_cache *cache, const int32_t *page_table, int64_t table_stride,
                   const int64_t *kv_lens, const int64_t *q_lens, const int64_t sizes[3], const int64_t strides[6],
                   int dtype, void *k, void *v, void *stream) {
  using namespace tdt;
  CacheArgs a = {};
  int rc = cache_call(&a, sizes, strides, dtype, true, cache, page_table, table_stride, kv_lens, q_lens);
  if (rc != TDT_OK || a.B == 0 || a.L == 0) return rc;
  if (!k || !v) return TDT_ERR_NULL_POINTER;
  if (((uintptr_t)k | (uintptr_t)v) % size_of(dtype)) return TDT_ERR_BAD_ALIGNMENT;
  if (!apart(a.sk, sizes[0], a.L, a.Hkv, a.D) || !apart(a.sv, sizes[0], a.L, a.Hkv, a.D)) return TDT_ERR_BAD_STRIDES;
  rc = check_cache_memory(cache, false);
  if (rc != TDT_OK) return rc;
  a.k = k;
  a.v = v;
  const cudaError_t e = launch_cache_read(a, dtype, cache->dtype, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? TDT_OK : TDT_ERR_CUDA;
}

size_t tdt_paged_attn_workspace_size(const int64_t sizes[4], int dtype, const tdt_paged_cache *cache) {
  using namespace tdt;
  if (check_attn(sizes, dtype, cache) != TDT_OK || sizes[0] == 0 || sizes[1] == 0) return 0;
  const PagedArgs a = attn_args(sizes, cache);
  const Way way = way_of(a, dtype, cache->dtype);
  if (way == kStep || way == kStep32) return 0;
  if (way == kTensor)
    return paged_tc_workspace(a.B, a.Lq, sizes[3] * cache->page_size, a.H, a.Hkv, a.D);
  return gather_space(sizes, dtype, cache).total;
}

int tdt_paged_attn(const void *q, const int64_t sizes[4], const int64_t strides[6], int dtype,
                   const tdt_paged_cache *cache, const int32_t *page_table, int64_t table_stride,
                   const int64_t *kv_lens, const int64_t *q_lens, double scale, void *out, float *lse,
                   void *workspace, size_t workspace_bytes, void *stream) {
  using namespace tdt;
  if (!strides) return TDT_ERR_NULL_POINTER;
  int rc = check_attn(sizes, dtype, cache);
  if (rc != TDT_OK) return rc;
  const float f = (float)scale;
  if (!(f > 0.0f) || !isfinite(f)) return TDT_ERR_BAD_SCALE;
  for (int i = 0; i < 6; ++i)
    if (strides[i] < 0) return TDT_ERR_BAD_STRIDES;
  PagedArgs a = attn_args(sizes, cache);
  a.sq = strides_of(strides);
  a.so = strides_of(strides + 3);
  a.scale = f;
  const Way way = way_of(a, dtype, cache->dtype);
  if (way == kGather) {  // as cross attention asks of its sizes
    const int64_t longest = std::max<int64_t>(a.Lq, sizes[3] * cache->page_size);
    if (a.B * a.H >= ((int64_t)1 << 31) / std::max<int64_t>(1, (longest + 31) / 32)) return TDT_ERR_BAD_SIZES;
  }
  const size_t need = tdt_paged_attn_workspace_size(sizes, dtype, cache);
  if (need > 0) {
    if (!workspace) return TDT_ERR_NULL_POINTER;
    if ((uintptr_t)workspace % 256 != 0) return TDT_ERR_BAD_ALIGNMENT;
    if (workspace_bytes < need) return TDT_ERR_WORKSPACE_TOO_SMALL;
  }
  if (a.B == 0 || a.Lq == 0) return TDT_OK;
  rc = fill_table(&a.t, cache, page_table, table_stride, kv_lens, q_lens, sizes[3]);
  if (rc != TDT_OK) return rc;
  if (!q || !out) return TDT_ERR_NULL_POINTER;
  if (((uintptr_t)q | (uintptr_t)out) % size_of(dtype) || (uintptr_t)lse % 4) return TDT_ERR_BAD_ALIGNMENT;
  rc = check_cache_memory(cache, false);
  if (rc != TDT_OK) return rc;
  if (!apart(a.so, a.B, a.Lq, a.H, a.D)) return TDT_ERR_BAD_STRIDES;
  a.q = q;
  a.out = out;
  a.lse = lse;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (way == kGather) return attend_gathered(a, sizes, strides, dtype, cache, workspace, workspace_bytes, s);
  const cudaError_t e = way == kStep32                              ? launch_paged_step32(a, cache->dtype, s)
                        : way == kTensor && paged_tc_fits(a, dtype) ? launch_paged_tc(a, dtype, workspace, s)
                                                                    : launch_paged_step(a, dtype, cache->dtype, s);
  return e == cudaSuccess ? TDT_OK : TDT_ERR_CUDA;
}

}  // extern "C"
