// tdt_paged.cuh -- what the kernels of the paged cache share: the argument blocks, where a position lies,
// 8-bit values, and the launchers.
#pragma once

#include <cuda_fp8.h>

#include "tdt_attn_common.cuh"

namespace tdt {

constexpr int kE4M3 = 3;  // a page's type; the others are DType
constexpr int kByteBias = 127, kByteNaN = 255;
constexpr int kLeastExponent = -117, kMostExponent = 120;

// Keys or values of a cache: rows of D elements at (page, place, head), each with a byte in 8-bit pages.
struct Pages {
  void *data;
  unsigned char *scales;
  Strides s, ss;  // strides b: page, l: place, h: head
};

// Which pages and positions a call is about.
struct PageTable {
  const int *ids;  // [B, max_pages], rows `stride` apart
  long long stride;
  const long long *kv_lens, *q_lens;
  int n_pages, page_bits, max_pages;
};

// Utterance b's new rows are the positions [first, first + n) (bad lengths: none).
struct NewRows {
  int first, n;
  bool bad;
};
__device__ __forceinline__ NewRows new_rows(const PageTable &t, long long b, int L) {
  const long long nk = t.kv_lens[b], nq = t.q_lens ? t.q_lens[b] : L;
  NewRows r;
  r.bad = nq < 0 || nq > L || nk < nq || nk > (long long)t.max_pages << t.page_bits;
  r.n = r.bad ? 0 : (int)nq;
  r.first = r.bad ? 0 : (int)(nk - nq);
  return r;
}
// The page of position p, or -1 if the table names none.
__device__ __forceinline__ int page_of(const PageTable &t, long long b, int p) {
  const int id = __ldg(t.ids + b * t.stride + (p >> t.page_bits));
  return (unsigned)id < (unsigned)t.n_pages ? id : -1;
}
__device__ __forceinline__ long long row_at(const Strides &s, int page, int place, int h) {
  return page * s.b + place * s.l + h * s.h;
}

// 2^(byte - 127); byte 0 is below the normal numbers, 255 stands for NaN.
__device__ __forceinline__ float scale_of(unsigned byte) {
  return byte == kByteNaN ? NAN : __uint_as_float(byte == 0 ? 0x00400000u : byte << 23);
}
// Two e4m3 as float16 pairs (exact), the first in the low half.
__device__ __forceinline__ unsigned e4m3x2_to_half2(unsigned two) {
  unsigned r;
  asm("{\n\t.reg .b16 x;\n\tcvt.u16.u32 x, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, x;\n\t}" : "=r"(r) : "r"(two));
  return r;
}
__device__ __forceinline__ float2 e4m3x2_to_float2(unsigned two) {
  const unsigned h = e4m3x2_to_half2(two);
  return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}
__device__ __forceinline__ unsigned float2_to_e4m3x2(float lo, float hi) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// One call of attention over pages, passed by value.
struct PagedArgs {
  const void *q;
  void *out;
  float *lse;  // [B, H, Lq] or NULL
  Strides sq, so;
  Pages k, v;
  PageTable t;
  long long B;
  int Lq, H, Hkv, G, D;  // G = H / Hkv
  float scale;
};

// One call that writes or reads rows of pages.
struct CacheArgs {
  void *k, *v;  // [B, L, Hkv, D]
  Strides sk, sv;
  Pages pk, pv;
  PageTable t;
  long long B;
  int L, Hkv, D;
};
cudaError_t launch_cache_write(const CacheArgs &a, int dtype, int cache_dtype, cudaStream_t stream);
cudaError_t launch_cache_read(const CacheArgs &a, int dtype, int cache_dtype, cudaStream_t stream);
// Few query rows: a kernel that reads k and v at memory speed.  (It takes any number of rows; *_takes go by sizes and pages.)
bool paged_step_takes(const PagedArgs &a, int dtype, int cache_dtype);
cudaError_t launch_paged_step(const PagedArgs &a, int dtype, int cache_dtype, cudaStream_t stream);
// The same of up to kStepRows float32 rows, on the CUDA cores.
bool paged_step32_takes(const PagedArgs &a, int dtype, int cache_dtype);
cudaError_t launch_paged_step32(const PagedArgs &a, int cache_dtype, cudaStream_t stream);
// Many query rows on the tensor cores: which calls (paged_tc_fits: by q and out, too), and the workspace for up to `most`
// positions an utterance.
bool paged_tc_takes(const PagedArgs &a, int dtype);
bool paged_tc_fits(const PagedArgs &a, int dtype);
size_t paged_tc_workspace(long long B, long long Lq, long long most, int H, int Hkv, int D);
cudaError_t launch_paged_tc(const PagedArgs &a, int dtype, void *workspace, cudaStream_t stream);

// Every other call: the rows of whole utterances become dense tensors, for cross attention to read.
struct GatherArgs {
  CacheArgs c;        // k, v: [B, L, Hkv, D], L: the table's positions
  int Lq;
  int2 *windows;      // [B, Lq]: the positions that each query sees
  long long *lens;    // [B]: positions of an utterance, -1 where lengths are out of range
};
cudaError_t launch_gather(const GatherArgs &f, int dtype, int cache_dtype, cudaStream_t stream);

}  // namespace tdt
