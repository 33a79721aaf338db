// tdt_cache.cu -- rows of keys and values into their pages and back, as they are or as e4m3 with a power of
// two a row.
//
// A row of D elements belongs to as many lanes as have 8 elements each (a power of two, up to 32), so a row's
// largest magnitude takes log2 of that shuffles and nothing is read twice.  With a = max |x| and
// a = m 2^x, 1 <= m < 2, the least e with a <= 448 2^e = 1.75 2^(e + 8) is x - 8, or x - 7 where m > 1.75:
// it comes from the bits of a, and x 2^-e is exact, so the only rounding is e4m3's own (half a step, 2^-4 of
// the value, or 2^-10 2^e below 2^-6 2^e).
// Bound by memory, or by latency for a decoding step.
//
// The rows of whole utterances can also be laid out densely, for attention that reads no pages (launch_gather).
#include "tdt_paged.cuh"
#include "tdt_rowio.cuh"

namespace tdt {
namespace {

constexpr int kThreads = 256;

// 8 elements from `p`, those from `n` on as 0.
template <int DT, bool VEC>
__device__ __forceinline__ void load8(const typename Elem<DT>::T *p, int n, float (&x)[8]) {
  if (VEC) {
    if (n <= 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = 0.0f;
      return;
    }
    unpack<DT>(ld_vec(p), x);
    if (DT == kF32) unpack<DT>(ld_vec(p + 4), x + 4);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = i < n ? Elem<DT>::load(p + i) : 0.0f;
}
template <int DT, bool VEC>
__device__ __forceinline__ void store8(typename Elem<DT>::T *p, int n, const float (&x)[8]) {
  if (VEC) {
    if (n <= 0) return;
    *reinterpret_cast<uint4 *>(p) = pack<DT>(x);
    if (DT == kF32) *reinterpret_cast<uint4 *>(p + 4) = pack<DT>(x + 4);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) p[i] = Elem<DT>::from_float(x[i]);
}

struct Row {
  long long b;
  int i, h;
};
__device__ __forceinline__ Row row_of(const CacheArgs &a, unsigned r) {
  Row x;
  const unsigned bi = r / a.Hkv;
  x.h = r % a.Hkv;
  x.i = bi % a.L;
  x.b = bi / a.L;
  return x;
}

// blockIdx.y: keys or values.  PT: the pages' type, DT or kE4M3.
template <int DT, int PT, bool VEC>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const __grid_constant__ CacheArgs a, int lane_bits) {
  typedef typename Elem<DT>::T E;
  const unsigned long long x = (unsigned long long)blockIdx.x * kThreads + threadIdx.x;
  const unsigned r = (unsigned)min(x >> lane_bits, (unsigned long long)a.rows);
  const int d0 = ((int)x & ((1 << lane_bits) - 1)) * 8;
  const Pages &p = blockIdx.y ? a.pv : a.pk;
  const Strides &s = blockIdx.y ? a.sv : a.sk;
  int page = -1, place = 0;
  Row at = {};
  if (r < a.rows) {
    at = row_of(a, r);
    const NewRows n = new_rows(a.t, at.b, a.L);
    if (at.i < n.n) {
      const int pos = n.first + at.i;
      page = page_of(a.t, at.b, pos);
      place = pos & ((1 << a.t.page_bits) - 1);
    }
  }
  float v[8];
  const E *src = static_cast<const E *>(blockIdx.y ? a.v : a.k) + at.b * s.b + at.i * s.l + at.h * s.h + d0;
  load8<DT, VEC>(src, page < 0 ? 0 : a.D - d0, v);
  if (PT != kE4M3) {
    if (page >= 0) store8<DT, VEC>(static_cast<E *>(p.data) + row_at(p.s, page, place, at.h) + d0, a.D - d0, v);
    return;
  }
  unsigned top = 0;  // bits of the largest magnitude: a NaN's are above infinity's
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
  for (int o = 1; o < 1 << lane_bits; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (page < 0) return;
  const bool finite = top < 0x7f800000u;
  int e = (int)(top >> 23) - 127 - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = min(max(e, kLeastExponent), kMostExponent);
  const float down = __uint_as_float((unsigned)(127 - e) << 23);
  unsigned w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i / 2] |= float2_to_e4m3x2(v[2 * i] * down, v[2 * i + 1] * down) << (i % 2 * 16);
  unsigned char *dst = static_cast<unsigned char *>(p.data) + row_at(p.s, page, place, at.h) + d0;
  if (VEC) {
    if (d0 < a.D) *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (d0 + i < a.D) dst[i] = (unsigned char)(w[i / 4] >> (i % 4 * 8));
  }
  if (d0 == 0)
    p.scales[row_at(p.ss, page, place, at.h)] = (unsigned char)(finite ? e + kByteBias : kByteNaN);
}

// Elements [d0, d0 + 8) of a row of pages as float32, NaN if there is no such page.
template <int PT, bool VEC>
__device__ __forceinline__ void read8(const Pages &p, int page, int place, int h, int d0, int D, float (&v)[8]) {
  if (page < 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = NAN;
    return;
  }
  if constexpr (PT == kE4M3) {
    const unsigned char *src = static_cast<const unsigned char *>(p.data) + row_at(p.s, page, place, h) + d0;
    const float up = scale_of(__ldg(p.scales + row_at(p.ss, page, place, h)));
    unsigned w[2] = {0, 0};
    if (VEC) {
      const uint2 two = __ldg(reinterpret_cast<const uint2 *>(src));
      w[0] = two.x;
      w[1] = two.y;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (d0 + i < D) w[i / 4] |= (unsigned)__ldg(src + i) << (i % 4 * 8);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = e4m3x2_to_float2(w[i / 2] >> (i % 2 * 16) & 0xffffu);
      v[2 * i] = f.x * up;
      v[2 * i + 1] = f.y * up;
    }
  } else {
    typedef typename Elem<PT>::T P;
    load8<PT, VEC>(static_cast<const P *>(p.data) + row_at(p.s, page, place, h) + d0, D - d0, v);
  }
}

template <int DT, int PT, bool VEC>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const __grid_constant__ CacheArgs a, int lane_bits) {
  typedef typename Elem<DT>::T E;
  const unsigned long long x = (unsigned long long)blockIdx.x * kThreads + threadIdx.x;
  const unsigned r = (unsigned)min(x >> lane_bits, (unsigned long long)a.rows);
  const int d0 = ((int)x & ((1 << lane_bits) - 1)) * 8;
  if (r >= a.rows || d0 >= a.D) return;
  const Pages &p = blockIdx.y ? a.pv : a.pk;
  const Strides &s = blockIdx.y ? a.sv : a.sk;
  const Row at = row_of(a, r);
  const NewRows n = new_rows(a.t, at.b, a.L);
  float v[8];
  int page = -1;
  if (at.i < n.n) {
    const int pos = n.first + at.i;
    page = page_of(a.t, at.b, pos);
    read8<PT, VEC>(p, page, pos & ((1 << a.t.page_bits) - 1), at.h, d0, a.D, v);
  } else {  // nothing to read: 0 past the new rows, NaN where the lengths are bad
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = n.bad ? NAN : 0.0f;
  }
  store8<DT, VEC>(static_cast<E *>(blockIdx.y ? a.v : a.k) + at.b * s.b + at.i * s.l + at.h * s.h + d0, a.D - d0, v);
}

// The rows of whole utterances as dense [B, L, Hkv, D] tensors k and v of type DT, those past an utterance's end left as they are;
// float16 ends at 65504.  The pages' rows of a chunk of positions go to a block; blocks take chunks in turn.  Beside them the
// positions that each query sees, and lengths that cross attention refuses where this call's are out of range.
constexpr int kChunk = 32;  // positions
template <int DT, int PT, bool VEC>
__global__ void __launch_bounds__(kThreads) gather_kernel(const __grid_constant__ GatherArgs f, int lane_bits) {
  typedef typename Elem<DT>::T E;
  const CacheArgs &a = f.c;
  for (long long x = (long long)blockIdx.x * kThreads + threadIdx.x; x < f.B * f.Lq && blockIdx.y == 0;
       x += (long long)gridDim.x * kThreads) {
    const long long b = x / f.Lq;
    const int i = (int)(x % f.Lq);
    const NewRows n = new_rows(a.t, b, f.Lq);
    f.windows[x] = make_int2(0, i < n.n ? n.first + i + 1 : 0);
    if (i == 0) f.lens[b] = n.bad ? -1 : n.first + n.n;
  }
  const Pages &p = blockIdx.y ? a.pv : a.pk;
  const Strides &s = blockIdx.y ? a.sv : a.sk;
  const int chunks = (a.L + kChunk - 1) / kChunk, units = kChunk * a.Hkv << lane_bits;
  for (long long c = blockIdx.x; c < f.B * chunks; c += gridDim.x) {
    const long long b = c / chunks;
    const int first = (int)(c % chunks) * kChunk;
    const NewRows n = new_rows(a.t, b, f.Lq);
    const int end = n.first + n.n;
    if (first >= end) continue;
    for (int x = threadIdx.x; x < units; x += kThreads) {
      const int d0 = (x & ((1 << lane_bits) - 1)) * 8, r = x >> lane_bits, pos = first + r / a.Hkv, h = r % a.Hkv;
      if (pos >= end || d0 >= a.D) continue;
      const int page = page_of(a.t, b, pos), place = pos & ((1 << a.t.page_bits) - 1);
      float v[8];
      read8<PT, VEC>(p, page, place, h, d0, a.D, v);
      if (DT == kF16 && PT == kE4M3)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] != v[i] ? v[i] : fminf(fmaxf(v[i], -65504.0f), 65504.0f);
      store8<DT, VEC>(static_cast<E *>(blockIdx.y ? a.v : a.k) + b * s.b + pos * s.l + h * s.h + d0, a.D - d0, v);
    }
  }
}

// Whether 8 elements a lane can go as whole vectors.
bool vectors(const CacheArgs &a, int dtype, int cache_dtype) {
  auto fits = [&](const void *p, const Strides &s, int type) {
    const long long unit = type == kF32 ? 4 : 8;                      // elements of an access
    const uintptr_t bytes = type == kE4M3 ? 8 : 16;
    return (uintptr_t)p % bytes == 0 && s.b % unit == 0 && s.l % unit == 0 && s.h % unit == 0;
  };
  return a.D % 8 == 0 && fits(a.k, a.sk, dtype) && fits(a.v, a.sv, dtype) && fits(a.pk.data, a.pk.s, cache_dtype) &&
         fits(a.pv.data, a.pv.s, cache_dtype);
}

template <int DT, int PT, bool READ> cudaError_t launch(const CacheArgs &a, cudaStream_t stream) {
  int lane_bits = 0;
  while (8 << lane_bits < a.D) ++lane_bits;
  const unsigned blocks = (unsigned)((((unsigned long long)a.rows << lane_bits) + kThreads - 1) / kThreads);
  const dim3 grid(blocks, 2);
  const bool vec = vectors(a, DT, PT);
  if constexpr (READ) {
    if (vec)
      cache_read_kernel<DT, PT, true><<<grid, kThreads, 0, stream>>>(a, lane_bits);
    else
      cache_read_kernel<DT, PT, false><<<grid, kThreads, 0, stream>>>(a, lane_bits);
  } else {
    if (vec)
      cache_write_kernel<DT, PT, true><<<grid, kThreads, 0, stream>>>(a, lane_bits);
    else
      cache_write_kernel<DT, PT, false><<<grid, kThreads, 0, stream>>>(a, lane_bits);
  }
  return cudaGetLastError();
}

template <int DT, int PT> cudaError_t gather(const GatherArgs &f, cudaStream_t stream) {
  int lane_bits = 0;
  while (8 << lane_bits < f.c.D) ++lane_bits;
  const long long chunks = f.B * ((f.c.L + kChunk - 1) / kChunk), rows = (f.B * f.Lq + kThreads - 1) / kThreads;
  const long long most = chunks > rows ? chunks : rows;
  const dim3 grid((unsigned)(most < 8 * kSMs ? most : 8 * kSMs), 2);
  if (vectors(f.c, DT, PT))
    gather_kernel<DT, PT, true><<<grid, kThreads, 0, stream>>>(f, lane_bits);
  else
    gather_kernel<DT, PT, false><<<grid, kThreads, 0, stream>>>(f, lane_bits);
  return cudaGetLastError();
}

template <int DT> cudaError_t read_from(const CacheArgs &a, int cache_dtype, cudaStream_t s) {
  return cache_dtype == kE4M3  ? launch<DT, kE4M3, true>(a, s)
         : cache_dtype == kF32 ? launch<DT, kF32, true>(a, s)
         : cache_dtype == kF16 ? launch<DT, kF16, true>(a, s)
                               : launch<DT, kBF16, true>(a, s);
}
template <int DT> cudaError_t write_to(const CacheArgs &a, int cache_dtype, cudaStream_t s) {
  return cache_dtype == kE4M3 ? launch<DT, kE4M3, false>(a, s) : launch<DT, DT, false>(a, s);
}

template <int DT> cudaError_t gather_from(const GatherArgs &f, int cache_dtype, cudaStream_t s) {
  return cache_dtype == kE4M3 ? gather<DT, kE4M3>(f, s) : gather<DT, DT>(f, s);
}

}  // namespace

cudaError_t launch_gather(const GatherArgs &f, int dtype, int cache_dtype, cudaStream_t stream) {
  return dtype == kF32   ? gather_from<kF32>(f, cache_dtype, stream)
         : dtype == kF16 ? gather_from<kF16>(f, cache_dtype, stream)
                         : gather_from<kBF16>(f, cache_dtype, stream);
}
cudaError_t launch_cache_write(const CacheArgs &a, int dtype, int cache_dtype, cudaStream_t stream) {
  return dtype == kF32   ? write_to<kF32>(a, cache_dtype, stream)
         : dtype == kF16 ? write_to<kF16>(a, cache_dtype, stream)
                         : write_to<kBF16>(a, cache_dtype, stream);
}
cudaError_t launch_cache_read(const CacheArgs &a, int dtype, int cache_dtype, cudaStream_t stream) {
  return dtype == kF32   ? read_from<kF32>(a, cache_dtype, stream)
         : dtype == kF16 ? read_from<kF16>(a, cache_dtype, stream)
                         : read_from<kBF16>(a, cache_dtype, stream);
}

}  // namespace tdt
