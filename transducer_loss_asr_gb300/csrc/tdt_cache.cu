// tdt_cache.cu -- rows of keys and values into their pages and back, as they are or as e4m3 with a power of
// two a row.
//
// A row of D elements belongs to as many lanes as have 16 elements each (a power of two, up to 16), so a row's
// largest magnitude takes log2 of that shuffles and nothing is read twice.  With a = max |x| and
// a = m 2^x, 1 <= m < 2, the least e with a <= 448 2^e = 1.75 2^(e + 8) is x - 8, or x - 7 where m > 1.75:
// it comes from the bits of a, and x 2^-e is exact, so the only rounding is e4m3's own (half a step, 2^-4 of
// the value, or 2^-10 2^e below 2^-6 2^e).
// A decoding step is bound by latency: lengths, page table, row, each a trip to memory after the other (64 x 16 heads: 4 us).
// Prompts are bound by that and by instructions (16 ragged x 1024 rows of 4 heads of 128, bfloat16 to e4m3: 12.7 us, 70 % of the issue
// slots, and back 14.8 us, 60 %, for 38 and 46 MB; 21 us where a thread found its own row by divisions and had 8 elements).  So a
// block has whole positions of one utterance, and a thread several pieces of 16 elements, whose page lookups, and then loads, are in
// flight together.
//
// The rows of whole utterances can also be laid out densely, for attention that reads no pages (launch_gather).
#include <algorithm>

#include "tdt_paged.cuh"

namespace tdt {
namespace {

constexpr int kThreads = 256;
constexpr int kPiece = 16;  // elements of a thread

// A call's pieces.  The launch fills it in.
struct Pieces {
  int lane_bits;       // of the lanes that share a row
  int unit;            // pieces of a position: Hkv << lane_bits
  int chunk;           // positions of a block's round
  unsigned rounds, chunks;  // of the call, of an utterance
  unsigned div_m, by_m;     // division by `unit`, by `chunks` (64-bit divisions took more instructions than all else)
  int div_s, by_s;
};

// 16 elements of a type as they lie in memory, and how many pieces a thread holds.
template <int T> struct Raw {
  static constexpr int ES = T == kE4M3 ? 1 : T == kF32 ? 4 : 2;
  static constexpr int W = kPiece * ES / 4;
  static constexpr int U = ES == 1 ? 4 : ES == 2 ? 2 : 1;  // pieces of a thread in flight
  unsigned w[W];
  float up;  // e4m3: the row's power of two
};
// The first `n` elements from `p`, the others as 0.  VEC: n is a multiple of 8, p suits accesses of 16 bytes (8 for e4m3).
template <int T, bool VEC> __device__ __forceinline__ void load_raw(const unsigned char *p, int n, Raw<T> &r) {
  constexpr int ES = Raw<T>::ES;
#pragma unroll
  for (int i = 0; i < Raw<T>::W; ++i) r.w[i] = 0;
  if constexpr (VEC) {
    constexpr int B = ES == 1 ? 8 : 16;  // bytes of an access
#pragma unroll
    for (int i = 0; i < kPiece * ES; i += B)
      if (i < n * ES) {
        if constexpr (B == 16) {
          const uint4 x = __ldg(reinterpret_cast<const uint4 *>(p + i));
          r.w[i / 4] = x.x;
          r.w[i / 4 + 1] = x.y;
          r.w[i / 4 + 2] = x.z;
          r.w[i / 4 + 3] = x.w;
        } else {
          const uint2 x = __ldg(reinterpret_cast<const uint2 *>(p + i));
          r.w[i / 4] = x.x;
          r.w[i / 4 + 1] = x.y;
        }
      }
  } else {
#pragma unroll
    for (int i = 0; i < kPiece; ++i)
      if (i < n) {
        if constexpr (ES == 1) r.w[i / 4] |= (unsigned)__ldg(p + i) << (i % 4 * 8);
        if constexpr (ES == 2) r.w[i / 2] |= (unsigned)__ldg(reinterpret_cast<const unsigned short *>(p) + i) << (i % 2 * 16);
        if constexpr (ES == 4) r.w[i] = __ldg(reinterpret_cast<const unsigned *>(p) + i);
      }
  }
}
template <int T, bool VEC> __device__ __forceinline__ void store_raw(unsigned char *p, int n, const Raw<T> &r) {
  constexpr int ES = Raw<T>::ES;
  if constexpr (VEC) {
    constexpr int B = ES == 1 ? 8 : 16;
#pragma unroll
    for (int i = 0; i < kPiece * ES; i += B)
      if (i < n * ES) {
        if constexpr (B == 16)
          *reinterpret_cast<uint4 *>(p + i) = make_uint4(r.w[i / 4], r.w[i / 4 + 1], r.w[i / 4 + 2], r.w[i / 4 + 3]);
        else
          *reinterpret_cast<uint2 *>(p + i) = make_uint2(r.w[i / 4], r.w[i / 4 + 1]);
      }
  } else {
#pragma unroll
    for (int i = 0; i < kPiece; ++i)
      if (i < n) {
        if constexpr (ES == 1) p[i] = (unsigned char)(r.w[i / 4] >> (i % 4 * 8));
        if constexpr (ES == 2) reinterpret_cast<unsigned short *>(p)[i] = (unsigned short)(r.w[i / 2] >> (i % 2 * 16));
        if constexpr (ES == 4) reinterpret_cast<unsigned *>(p)[i] = r.w[i];
      }
  }
}
// Elements 2i and 2i + 1 as float32.
template <int T> __device__ __forceinline__ float2 pair_of(const Raw<T> &r, int i) {
  if constexpr (T == kE4M3) {
    const float2 f = e4m3x2_to_float2(r.w[i / 2] >> (i % 2 * 16) & 0xffffu);
    return make_float2(f.x * r.up, f.y * r.up);
  }
  if constexpr (T == kF32) return make_float2(__uint_as_float(r.w[2 * i]), __uint_as_float(r.w[2 * i + 1]));
  if constexpr (T == kF16) return __half22float2(*reinterpret_cast<const __half2 *>(&r.w[i]));
  return make_float2(__uint_as_float(r.w[i] << 16), __uint_as_float(r.w[i] & 0xffff0000u));
}
template <int T> __device__ __forceinline__ void set_pair(Raw<T> &r, int i, float2 v) {
  if constexpr (T == kF32) {
    r.w[2 * i] = __float_as_uint(v.x);
    r.w[2 * i + 1] = __float_as_uint(v.y);
  } else if constexpr (T == kF16) {
    const __half2 h = __floats2half2_rn(v.x, v.y);
    r.w[i] = *reinterpret_cast<const unsigned *>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
    r.w[i] = *reinterpret_cast<const unsigned *>(&h);
  }
}
// A piece of a page as a piece of type DT.  SATURATE: float16 ends at 65504.
template <int DT, int PT, bool SATURATE> __device__ __forceinline__ void convert(const Raw<PT> &x, Raw<DT> &y) {
#pragma unroll
  for (int i = 0; i < kPiece / 2; ++i) {
    if constexpr (DT == PT && DT != kE4M3) {
#pragma unroll
      for (int k = 0; k < Raw<DT>::W / (kPiece / 2); ++k)
        y.w[i * (Raw<DT>::W / (kPiece / 2)) + k] = x.w[i * (Raw<DT>::W / (kPiece / 2)) + k];
    } else {
      float2 v = pair_of<PT>(x, i);
      if (SATURATE && DT == kF16) {  // NaN stays
        v.x = v.x != v.x ? v.x : fminf(fmaxf(v.x, -65504.0f), 65504.0f);
        v.y = v.y != v.y ? v.y : fminf(fmaxf(v.y, -65504.0f), 65504.0f);
      }
      set_pair<DT>(y, i, v);
    }
  }
}
template <int DT> __device__ __forceinline__ void fill(Raw<DT> &y, float v) {
#pragma unroll
  for (int i = 0; i < kPiece / 2; ++i) set_pair<DT>(y, i, make_float2(v, v));
}

// Elements [d0, d0 + 16) of a row of pages; nothing is read if there is no such page.
template <int PT, bool VEC>
__device__ __forceinline__ void load_page(const Pages &p, int page, int place, int h, int d0, int D, Raw<PT> &r) {
  const unsigned char *src = static_cast<const unsigned char *>(p.data) + (row_at(p.s, page, place, h) + d0) * Raw<PT>::ES;
  load_raw<PT, VEC>(src, page < 0 ? 0 : D - d0, r);
  if (PT == kE4M3) r.up = page < 0 ? 0.0f : scale_of(__ldg(p.scales + row_at(p.ss, page, place, h)));
}

// Piece x of a chunk: row i of it, head h, elements from d0.
struct At {
  int i, h, d0;
};
__device__ __forceinline__ At piece_at(const Pieces &q, int x) {
  At at;
  at.i = (int)fast_div((unsigned)x, q.div_m, q.div_s);
  const int in = x - at.i * q.unit;
  at.h = in >> q.lane_bits;
  at.d0 = (in & ((1 << q.lane_bits) - 1)) * kPiece;
  return at;
}

// blockIdx.y: keys or values.  PT: the pages' type, DT or kE4M3.
template <int DT, int PT, bool VEC>
__global__ void __launch_bounds__(kThreads, 5) cache_write_kernel(const __grid_constant__ CacheArgs a, const __grid_constant__ Pieces q) {
  constexpr int U = Raw<DT>::U, ES = Raw<DT>::ES;
  const Pages &p = blockIdx.y ? a.pv : a.pk;
  const Strides &s = blockIdx.y ? a.sv : a.sk;
  const int units = q.chunk * q.unit, place_mask = (1 << a.t.page_bits) - 1;
  for (unsigned c = blockIdx.x; c < q.rounds; c += gridDim.x) {
    const unsigned utt = fast_div(c, q.by_m, q.by_s);
    const long long b = utt;
    const int i0 = (int)(c - utt * q.chunks) * q.chunk;
    const NewRows n = new_rows(a.t, b, a.L);
    if (i0 >= n.n) continue;
    const unsigned char *src = static_cast<const unsigned char *>(blockIdx.y ? a.v : a.k);
    for (int x0 = 0; x0 < units; x0 += U * kThreads) {  // the whole block goes round: lanes share rows
      At at[U];
      int page[U];
      Raw<DT> v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int x = x0 + u * kThreads + threadIdx.x;
        at[u] = piece_at(q, x);
        at[u].i += i0;
        const bool in = x < units && at[u].i < n.n;
        page[u] = in ? page_of(a.t, b, n.first + at[u].i) : -1;
        load_raw<DT, VEC>(src + (b * s.b + at[u].i * s.l + at[u].h * s.h + at[u].d0) * ES, in ? a.D - at[u].d0 : 0, v[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int place = (n.first + at[u].i) & place_mask;
        unsigned char *dst = static_cast<unsigned char *>(p.data) + (row_at(p.s, page[u], place, at[u].h) + at[u].d0) * Raw<PT>::ES;
        if constexpr (PT != kE4M3) {
          if (page[u] >= 0) store_raw<PT, VEC>(dst, a.D - at[u].d0, v[u]);
        } else {
          unsigned top = 0;  // bits of the largest magnitude: a NaN's are above infinity's
#pragma unroll
          for (int i = 0; i < kPiece / 2; ++i) {
            const float2 x = pair_of<DT>(v[u], i);
            top = max(top, max(__float_as_uint(x.x) & 0x7fffffffu, __float_as_uint(x.y) & 0x7fffffffu));
          }
          for (int o = 1; o < 1 << q.lane_bits; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
          if (page[u] < 0) continue;
          int e = (int)(top >> 23) - 127 - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
          e = min(max(e, kLeastExponent), kMostExponent);
          const float down = __uint_as_float((unsigned)(127 - e) << 23);
          Raw<kE4M3> y;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 x0 = pair_of<DT>(v[u], 2 * i), x1 = pair_of<DT>(v[u], 2 * i + 1);
            y.w[i] = float2_to_e4m3x2(x0.x * down, x0.y * down) | float2_to_e4m3x2(x1.x * down, x1.y * down) << 16;
          }
          store_raw<kE4M3, VEC>(dst, a.D - at[u].d0, y);
          if (at[u].d0 == 0)
            p.scales[row_at(p.ss, page[u], place, at[u].h)] = (unsigned char)(top < 0x7f800000u ? e + kByteBias : kByteNaN);
        }
      }
    }
  }
}

template <int DT, int PT, bool VEC>
__global__ void __launch_bounds__(kThreads, 5) cache_read_kernel(const __grid_constant__ CacheArgs a, const __grid_constant__ Pieces q) {
  constexpr int U = Raw<PT>::U;
  const Pages &p = blockIdx.y ? a.pv : a.pk;
  const Strides &s = blockIdx.y ? a.sv : a.sk;
  const int units = q.chunk * q.unit, place_mask = (1 << a.t.page_bits) - 1;
  for (unsigned c = blockIdx.x; c < q.rounds; c += gridDim.x) {
    const unsigned utt = fast_div(c, q.by_m, q.by_s);
    const long long b = utt;
    const int i0 = (int)(c - utt * q.chunks) * q.chunk;
    const NewRows n = new_rows(a.t, b, a.L);
    unsigned char *dst = static_cast<unsigned char *>(blockIdx.y ? a.v : a.k);
    for (int x0 = threadIdx.x; x0 < units; x0 += U * kThreads) {
      At at[U];
      int page[U];
      Raw<PT> v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int x = x0 + u * kThreads;
        at[u] = piece_at(q, x);
        at[u].i += i0;
        if (x >= units || at[u].d0 >= a.D) at[u].i = a.L;
        page[u] = at[u].i < n.n ? page_of(a.t, b, n.first + at[u].i) : -1;
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        load_page<PT, VEC>(p, page[u], (n.first + at[u].i) & place_mask, at[u].h, at[u].d0, a.D, v[u]);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (at[u].i >= a.L) continue;
        Raw<DT> y;
        if (page[u] >= 0)
          convert<DT, PT, false>(v[u], y);
        else  // past the new rows 0; NaN where there is no page, or lengths are bad
          fill<DT>(y, n.bad || at[u].i < n.n ? NAN : 0.0f);
        store_raw<DT, VEC>(dst + (b * s.b + at[u].i * s.l + at[u].h * s.h + at[u].d0) * Raw<DT>::ES, a.D - at[u].d0, y);
      }
    }
  }
}

// The rows of whole utterances as dense [B, L, Hkv, D] tensors k and v of type DT, those past an utterance's end left as they
// are; float16 ends at 65504.  Beside them the positions that each query sees, and lengths that cross attention refuses where
// this call's are out of range.
template <int DT, int PT, bool VEC>
__global__ void __launch_bounds__(kThreads, 5) gather_kernel(const __grid_constant__ GatherArgs f, const __grid_constant__ Pieces q) {
  constexpr int U = Raw<PT>::U;
  const CacheArgs &a = f.c;
  for (long long x = (long long)blockIdx.x * kThreads + threadIdx.x; x < a.B * f.Lq && blockIdx.y == 0;
       x += (long long)gridDim.x * kThreads) {
    const long long b = x / f.Lq;
    const int i = (int)(x - b * f.Lq);
    const NewRows n = new_rows(a.t, b, f.Lq);
    f.windows[x] = make_int2(0, i < n.n ? n.first + i + 1 : 0);
    if (i == 0) f.lens[b] = n.bad ? -1 : n.first + n.n;
  }
  const Pages &p = blockIdx.y ? a.pv : a.pk;
  const Strides &s = blockIdx.y ? a.sv : a.sk;
  const int units = q.chunk * q.unit, place_mask = (1 << a.t.page_bits) - 1;
  for (unsigned c = blockIdx.x; c < q.rounds; c += gridDim.x) {
    const unsigned utt = fast_div(c, q.by_m, q.by_s);
    const long long b = utt;
    const int i0 = (int)(c - utt * q.chunks) * q.chunk;
    const NewRows n = new_rows(a.t, b, f.Lq);
    const int end = n.first + n.n;
    if (i0 >= end) continue;
    unsigned char *dst = static_cast<unsigned char *>(blockIdx.y ? a.v : a.k);
    for (int x0 = threadIdx.x; x0 < units; x0 += U * kThreads) {
      At at[U];
      int page[U];
      Raw<PT> v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int x = x0 + u * kThreads;
        at[u] = piece_at(q, x);
        at[u].i += i0;
        if (x >= units || at[u].d0 >= a.D) at[u].i = end;
        page[u] = at[u].i < end ? page_of(a.t, b, at[u].i) : -1;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) load_page<PT, VEC>(p, page[u], at[u].i & place_mask, at[u].h, at[u].d0, a.D, v[u]);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (at[u].i >= end) continue;
        Raw<DT> y;
        if (page[u] >= 0)
          convert<DT, PT, PT == kE4M3>(v[u], y);
        else
          fill<DT>(y, NAN);
        store_raw<DT, VEC>(dst + (b * s.b + at[u].i * s.l + at[u].h * s.h + at[u].d0) * Raw<DT>::ES, a.D - at[u].d0, y);
      }
    }
  }
}

// Whether 8 elements can go as whole vectors.
bool vectors(const CacheArgs &a, int dtype, int cache_dtype) {
  auto fits = [&](const void *p, const Strides &s, int type) {
    const long long unit = type == kF32 ? 4 : 8;                      // elements of an access
    const uintptr_t bytes = type == kE4M3 ? 8 : 16;
    return (uintptr_t)p % bytes == 0 && s.b % unit == 0 && s.l % unit == 0 && s.h % unit == 0;
  };
  return a.D % 8 == 0 && fits(a.k, a.sk, dtype) && fits(a.v, a.sv, dtype) && fits(a.pk.data, a.pk.s, cache_dtype) &&
         fits(a.pv.data, a.pv.s, cache_dtype);
}

Pieces pieces_of(const CacheArgs &a, int in_flight) {
  Pieces q = {};
  while (kPiece << q.lane_bits < a.D) ++q.lane_bits;
  q.unit = a.Hkv << q.lane_bits;
  q.chunk = std::max(1, in_flight * kThreads / q.unit);
  auto chunks = [&] { return (a.L + (long long)q.chunk - 1) / q.chunk; };
  while (a.B * chunks() > 0x7fffffffLL / 2 && q.chunk < a.L) q.chunk *= 2;  // rounds count in 32 bits; B < 2^30
  q.chunks = (unsigned)std::max<long long>(1, chunks());
  q.rounds = (unsigned)(a.B * chunks());
  fast_div_setup(q.unit, &q.div_m, &q.div_s);
  fast_div_setup(q.chunks, &q.by_m, &q.by_s);
  return q;
}
// Blocks for `rounds` rounds: all of them, up to two waves of eight blocks an SM (of keys, and of values).
dim3 grid_of(long long rounds) { return dim3((unsigned)std::max<long long>(1, std::min<long long>(rounds, 8 * kSMs)), 2); }

template <int DT, int PT> cudaError_t write(const CacheArgs &a, cudaStream_t stream) {
  const Pieces q = pieces_of(a, Raw<DT>::U);
  const dim3 grid = grid_of(q.rounds);
  if (vectors(a, DT, PT))
    cache_write_kernel<DT, PT, true><<<grid, kThreads, 0, stream>>>(a, q);
  else
    cache_write_kernel<DT, PT, false><<<grid, kThreads, 0, stream>>>(a, q);
  return cudaGetLastError();
}
template <int DT, int PT> cudaError_t read(const CacheArgs &a, cudaStream_t stream) {
  const Pieces q = pieces_of(a, Raw<PT>::U);
  const dim3 grid = grid_of(q.rounds);
  if (vectors(a, DT, PT))
    cache_read_kernel<DT, PT, true><<<grid, kThreads, 0, stream>>>(a, q);
  else
    cache_read_kernel<DT, PT, false><<<grid, kThreads, 0, stream>>>(a, q);
  return cudaGetLastError();
}
template <int DT, int PT> cudaError_t gather(const GatherArgs &f, cudaStream_t stream) {
  const Pieces q = pieces_of(f.c, Raw<PT>::U);
  const dim3 grid = grid_of(std::max<long long>(q.rounds, (f.c.B * f.Lq + kThreads - 1) / kThreads));
  if (vectors(f.c, DT, PT))
    gather_kernel<DT, PT, true><<<grid, kThreads, 0, stream>>>(f, q);
  else
    gather_kernel<DT, PT, false><<<grid, kThreads, 0, stream>>>(f, q);
  return cudaGetLastError();
}

template <int DT> cudaError_t write_to(const CacheArgs &a, int cache_dtype, cudaStream_t s) {
  return cache_dtype == kE4M3 ? write<DT, kE4M3>(a, s) : write<DT, DT>(a, s);
}
template <int DT> cudaError_t read_from(const CacheArgs &a, int cache_dtype, cudaStream_t s) {
  return cache_dtype == kE4M3  ? read<DT, kE4M3>(a, s)
         : cache_dtype == kF32 ? read<DT, kF32>(a, s)
         : cache_dtype == kF16 ? read<DT, kF16>(a, s)
                               : read<DT, kBF16>(a, s);
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
