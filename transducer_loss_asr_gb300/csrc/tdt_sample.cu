// tdt_sample.cu -- draws a token of each row of logits (include/tdt_decoder.h, tdt_sample): temperature,
// top-k, top-p, min-p, then the inverse of the running sum at a given uniform number.
//
// Mathematics.  Weights are whole numbers, w = rint(2^31 * 2^z) with z = (x - X) * (log2(e) / T) and X the
// row's maximum, so sums of weights are exact whatever their order, and every filter keeps a prefix of the
// order (x falling, index rising): the kept set is "order key above a cut, and the first c tokens equal to
// it".  The cut is found by radix selection: a histogram of counts and weights over 256 stretches of the
// keys in question tells the stretch at which the count reaches top_k, or the weight the share top_p of
// what top_k leaves; the tokens of that stretch are ranked by one warp (more than 32 of them: further
// histograms).  Both cuts use the same first histogram.
//
// One CTA a row.  Every warp owns a contiguous range of the row, so sums by warp are running sums of the
// vocabulary's order.
//   pass 1  the maximum X; rows of up to 16,384 tokens stay in shared memory, as float32;
//   pass 2  the sum of all weights, if the settings need it, and the places of vectors with a token of
//           z >= -12 (overflowing: -6, -3); their tokens then go into a list in shared memory, each warp
//           its own part, in index order.  Rows of up to 1,024 tokens need no list.
// The cut usually lies among the listed tokens -- top_k of them exist, or their weight reaches top_p's
// share of all, or min_p is above any unlisted weight -- and then selection and draw read the list only.
// Otherwise they read the row again (from L2, where it does not stay).
// Bound: few rows by the latency of the phases (1 x 8,193: 10 us); 656 x 8,193 float32 with each row's own
// settings by the latency and barriers of the selection, at two CTAs an SM (96 registers of 256 threads, 86 KB), 70 us
// for 21 MB; 2,048 x 131,072 bfloat16 by pass 2's instructions (71 % of the issue slots over the kernel; its read comes
// from L2), 241 to 321 us for 537 MB, by card.
// Wide rows are bound by pass 2's instructions.  Its weights are below 2^-9 of the largest, apart from the
// listed ones, and adding 1.5 * 2^-8 to such a weight leaves rint(2^31 w) in the low bits of the sum: no
// conversion, and whole-number sums of those bits; what the listed tokens contribute is taken out when
// they are listed.  Two tokens an instruction where the hardware has it.
#include "../../include/tdt_decoder.h"
#include "tdt_rowio.cuh"
#include "tdt_tc.cuh"

namespace tdt {
namespace {

typedef unsigned long long u64;

constexpr int kListTokens = 4096;      // entries of the list
constexpr int kResident = 16384;       // tokens of a row that stays in shared memory
constexpr int kOwnList = 1024;         // tokens of a row that needs no list
constexpr int kListZ = 12;             // z >= -kListZ goes into the list; if that overflows, half of it, ...
constexpr int kListTries = 3;
constexpr float kZeroZ = 33.0f;        // z < -32 weighs 0
constexpr float kMagic = 1.5f / 256.0f;  // bits 0x3bc00000: bits 26 and 0 to 21 are clear

struct SampleArgs {
  const void *logits;
  long long row_stride;
  int V;
  const float *u, *temperatures, *top_ps, *min_ps;
  const int *top_ks;
  float temperature, top_p, min_p;
  int top_k;
  int *tokens;
  float *logprobs;
};

// Order of the floats as unsigned numbers; -0 counts as 0, NaN sorts below everything.  Of the 16-bit
// types the float32 bits that are always zero are left out.
template <int DT> struct Key {
  static constexpr int SHIFT = DT == kF32 ? 0 : DT == kF16 ? 13 : 16;
  static __device__ __forceinline__ unsigned of(float x) {
    const unsigned b = __float_as_uint(x + 0.0f);
    if (x != x) return 0;
    return ((b & 0x80000000u) ? ~b : b | 0x80000000u) >> SHIFT;
  }
  static __device__ __forceinline__ float value(unsigned k) {  // of a key of the type
    k <<= SHIFT;
    return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~(k | ((1u << SHIFT) - 1)));
  }
};

struct Weigher {
  float X, per;   // row maximum, log2(e) / T
  bool infinite;  // X = +inf: only the +inf entries weigh anything
  // rint(2^31 2^z); the two roundings of z are part of the definition, so no fused multiply
  __device__ __forceinline__ unsigned operator()(float x) const {
    if (infinite) return x == X ? 0x80000000u : 0u;
    const float z = fmaxf(__fmul_rn(__fsub_rn(x, X), per), -64.0f);  // NaN, -inf: weight 0
    return __float2uint_rn(fast_exp2(z) * 2147483648.0f);
  }
  // what pass 2 adds for a token
  __device__ __forceinline__ unsigned bits(float x) const {
    const float z = __fmul_rn(__fsub_rn(x, X), per);
    return __float_as_uint(__fadd_rn(fast_exp2(z), kMagic)) - __float_as_uint(kMagic);
  }
};

// floor(total * part24 / 2^24) for part24 <= 2^24
__device__ __forceinline__ u64 share(u64 total, unsigned part24) {
  return (total >> 24) * part24 + (((total & 0xffffffu) * part24) >> 24);
}

__device__ __forceinline__ u64 warp_sum64(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ int warp_sum_int(int v) { return __reduce_add_sync(0xffffffffu, v); }
// Sum of v over the lanes below this one.
__device__ __forceinline__ u64 warp_before64(u64 v) {
  const int lane = threadIdx.x & 31;
  u64 s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 t = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += t;
  }
  return s - v;
}
__device__ __forceinline__ int warp_before_int(int v) {
  const int lane = threadIdx.x & 31;
  int s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += t;
  }
  return s - v;
}

// What a warp's range holds of the kept set: weight above the cut, tokens equal to it.
struct Held {
  u64 mass;
  unsigned ties;
};

template <int NW> struct Shared {
  // of a stretch of keys: tokens, and their weight in three parts (over 2^48 + hi 2^16 + lo)
  __align__(16) unsigned cnt[256], lo[256], hi[256], over[256];
  unsigned keys[32], weights[32];  // tokens to be ranked
  Held held[NW], low[NW];
  int listed[NW];
  float red[NW];
  // one thread's findings for all
  unsigned digit, found_key, found_ties;
  u64 above_cnt, above_mass, found_mass, target;
  int winner, token, ranked;
  unsigned ties_left;
};

// The prefix that stays: keys above `key`, and the first `ties` tokens with that key.
struct Cut {
  unsigned key;
  unsigned ties;
  u64 mass;  // its weight
};

template <int DT, int NW, bool RESIDENT> struct Sampler {
  typedef typename Elem<DT>::T E;
  typedef Key<DT> K;
  static constexpr int VEC = Vec<DT>::N;
  static constexpr int CAP = kListTokens / NW;  // list entries of a warp

  Shared<NW> &s;
  float *own;     // the resident row, from its first vector on
  float *xs;      // the list: tokens' values, their indices, and the vectors they come from
  int *ids, *vecs;
  const E *row;
  int V, warp, lane, head, v0, v1;  // vectors [v0, v1) of the row are the warp's
  Weigher w;
  bool listed;    // the tokens read below are the list's
  bool whole;     // a short resident row: no list is made

  __device__ Sampler(Shared<NW> &sh, unsigned char *mem, const E *r, int v)
      : s(sh), row(r), V(v), listed(false), whole(false) {
    warp = threadIdx.x >> 5;
    lane = threadIdx.x & 31;
    // Vectors start at multiples of VEC counted from the 16-byte boundary below the row
    head = (int)(((uintptr_t)row % 16) / sizeof(E));
    const int vectors = (V + head + VEC - 1) / VEC, each = (vectors + NW - 1) / NW;
    v0 = min(each * warp, vectors);
    v1 = min(v0 + each, vectors);
    own = reinterpret_cast<float *>(mem);
    xs = own + (RESIDENT ? (V + 16 + 3) / 4 * 4 : 0);
    ids = reinterpret_cast<int *>(xs + kListTokens);
    vecs = ids + kListTokens;
  }

  // Vector v as float32: tokens outside the row and NaN come as -inf.
  __device__ __forceinline__ uint4 fetch(int v) const {
    const int i = v * VEC - head;
    uint4 raw;
    if (i >= 0 && i + VEC <= V) {
      raw = __ldg(reinterpret_cast<const uint4 *>(row + i));
    } else {
      E *e = reinterpret_cast<E *>(&raw);
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        e[j] = i + j >= 0 && i + j < V ? row[i + j] : Elem<DT>::from_float(-INFINITY);
    }
    return raw;
  }
  static __device__ __forceinline__ void unpack(uint4 raw, float (&x)[VEC]) {
    unsigned v[4] = {raw.x, raw.y, raw.z, raw.w};
    if constexpr (DT == kF32) {
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = fmaxf(__uint_as_float(v[j]), -INFINITY);
    } else if constexpr (DT == kBF16) {
      const __nv_bfloat162 low = __floats2bfloat162_rn(-INFINITY, -INFINITY);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 c = __hmax2(*reinterpret_cast<__nv_bfloat162 *>(&v[j]), low);
        const unsigned b = *reinterpret_cast<const unsigned *>(&c);
        x[2 * j] = __uint_as_float(b << 16);
        x[2 * j + 1] = __uint_as_float(b & 0xffff0000u);
      }
    } else {
      const __half2 low = __floats2half2_rn(-INFINITY, -INFINITY);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 c = __half22float2(__hmax2(*reinterpret_cast<__half2 *>(&v[j]), low));
        x[2 * j] = c.x;
        x[2 * j + 1] = c.y;
      }
    }
  }
  // The largest token of a vector, NaN apart.
  static __device__ __forceinline__ float top_of(uint4 raw) {
    unsigned v[4] = {raw.x, raw.y, raw.z, raw.w};
    if constexpr (DT == kF32) {
      return fmaxf(max3(__uint_as_float(v[0]), __uint_as_float(v[1]), __uint_as_float(v[2])),
                   __uint_as_float(v[3]));
    } else if constexpr (DT == kBF16) {
      __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(v);
      const __nv_bfloat162 c = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
      const unsigned b = *reinterpret_cast<const unsigned *>(&c);
      return fmaxf(__uint_as_float(b << 16), __uint_as_float(b & 0xffff0000u));
    } else {
      __half2 *h = reinterpret_cast<__half2 *>(v);
      const float2 c = __half22float2(__hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3])));
      return fmaxf(c.x, c.y);
    }
  }
  // f(vector, raw) for the warp's vectors in memory, a vector a lane; every lane takes every step, and
  // those past the warp's end get vectors of -inf.
  template <typename F> __device__ __forceinline__ void each_raw(F f) const {
    constexpr int U = 4;  // loads of a turn; the next turn's are in flight while this one's are at work
    const int inner0 = head > 0 ? 1 : 0, inner1 = min(v1, (V + head) / VEC);
    const uint4 *base = reinterpret_cast<const uint4 *>(row - head);
    int v = v0;
    auto edge = [&]() {
      const bool mine = v + lane < v1;
      f(v + lane, fetch(mine ? v + lane : (V + head) / VEC + 1));
      v += 32;
    };
    if (v < inner0 && v < v1) edge();
    if (v + 32 * U <= inner1) {
      uint4 raw[U], next[U];
#pragma unroll
      for (int u = 0; u < U; ++u) next[u] = __ldg(base + v + u * 32 + lane);
      while (v + 32 * U <= inner1) {
#pragma unroll
        for (int u = 0; u < U; ++u) raw[u] = next[u];
        if (v + 64 * U <= inner1)
#pragma unroll
          for (int u = 0; u < U; ++u) next[u] = __ldg(base + v + (U + u) * 32 + lane);
#pragma unroll
        for (int u = 0; u < U; ++u) f(v + u * 32 + lane, raw[u]);
        v += 32 * U;
      }
    }
    while (v < v1) edge();
  }
  // f(x) for every token of this thread's share of the warp's: the list's or the row's.
  template <typename F> __device__ __forceinline__ void each(F f) const {
    if (listed) {
      const int n = s.listed[warp], at = warp * CAP;
      for (int i = lane; i < n; i += 32) f(xs[at + i]);
    } else if (RESIDENT) {
      for (int p = max(v0 * VEC, head) + lane; p < min(v1 * VEC, V + head); p += 32) f(own[p]);
    } else {
      each_raw([&](int, uint4 raw) {
        float x[VEC];
        unpack(raw, x);
#pragma unroll
        for (int j = 0; j < VEC; ++j) f(x[j]);
      });
    }
  }
  // Token i of the row, NaN as -inf.
  __device__ __forceinline__ float token(int i) const {
    return RESIDENT ? own[i + head] : fmaxf(Elem<DT>::load(row + i), -INFINITY);
  }

  __device__ float maximum() {
    float m = -INFINITY;
    each_raw([&](int v, uint4 raw) {
      m = fmaxf(m, top_of(raw));  // fmaxf passes over NaN
      if (RESIDENT && v < v1) {
        float x[VEC];
        unpack(raw, x);
#pragma unroll
        for (int j = 0; j < VEC; j += 4)
          *reinterpret_cast<float4 *>(own + v * VEC + j) = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
      }
    });
    m = warp_max(m);
    if (lane == 0) s.red[warp] = m;
    __syncthreads();
    return warp_max(lane < NW ? s.red[lane] : -INFINITY);
  }

  // Pass 2.  MASS: the weight of the tokens that are not listed, by warp into low[].mass.  LIST: the tokens
  // of at least `near` into the list, their weight by warp into held[].mass.  Returns the number of listed
  // tokens, -1 if they do not fit (then the sums are of all tokens, in low[]).
  template <bool MASS, bool LIST> __device__ int weigh(float near) {
    u64 mass = 0, mass_listed = 0;
    int n = 0, nv = 0;
    bool fits = true;
    // reading a weight off the sum is exact below 2^-9: see the head of the file
    const bool small = !w.infinite && (near - w.X) * w.per < -9.5f;
    const float2 x2 = make_float2(-w.X, -w.X), per2 = make_float2(w.per, w.per),
                 magic2 = make_float2(kMagic, kMagic);
    auto take = [&](int v, const float (&x)[VEC], float top) {
      bool here = top >= near;
      if (MASS && small) {
        unsigned sum = 0, any = 0;
#pragma unroll
        for (int j = 0; j < VEC; j += 2) {
          const float2 z = mul2(add2(make_float2(x[j], x[j + 1]), x2), per2);
          const float2 m = add2(make_float2(fast_exp2(z.x), fast_exp2(z.y)), magic2);
          sum += __float_as_uint(m.x) + __float_as_uint(m.y);
          any |= __float_as_uint(m.x) | __float_as_uint(m.y);
        }
        mass += sum - VEC * __float_as_uint(kMagic);  // modulo 2^32; the sum itself is at most VEC 2^26
        // A weight of 2^-12 and more sets one of the bits 19 to 21, or (from 2^-9 on) bit 26, which the
        // others do not: vectors with a token of z >= -12 are among these.
        here = any & 0x04380000u;
      } else if (MASS) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) mass += w(x[j]);
      }
      if (!LIST && !(MASS && small)) return;
      const unsigned hit = __ballot_sync(0xffffffffu, here);
      if (hit) {
        const int at = nv + __popc(hit & ((1u << lane) - 1));
        nv += __popc(hit);
        if (nv > CAP)
          fits = false;
        else if (hit >> lane & 1)
          vecs[warp * CAP + at] = v;
      }
    };
    if (RESIDENT) {
      for (int v = v0; v < v1; v += 32) {
        float x[VEC], top = -INFINITY;
#pragma unroll
        for (int j = 0; j < VEC; j += 4) {
          const float4 q = v + lane < v1 ? *reinterpret_cast<const float4 *>(own + (v + lane) * VEC + j)
                                         : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
          x[j] = q.x;
          x[j + 1] = q.y;
          x[j + 2] = q.z;
          x[j + 3] = q.w;
          top = fmaxf(max3(q.x, q.y, top), fmaxf(q.z, q.w));
        }
        take(v + lane, x, top);
      }
    } else {
      each_raw([&](int v, uint4 raw) {
        float x[VEC];
        if (MASS) unpack(raw, x);
        take(v, x, MASS && small ? 0.0f : top_of(raw));
      });
    }
    // the tokens of the noted vectors, in order
    __syncwarp();
    if (fits) {
      uint4 raw_next = make_uint4(0, 0, 0, 0);
      int v_next = lane < nv ? vecs[warp * CAP + lane] : v0;
      if (!RESIDENT && nv > 0) raw_next = fetch(v_next);
      for (int e = 0; e < nv; e += 32) {
        const bool mine = e + lane < nv;
        const int v = v_next;
        float x[VEC];
        if (RESIDENT) {
#pragma unroll
          for (int j = 0; j < VEC; ++j) x[j] = own[v * VEC + j];
        } else {
          unpack(raw_next, x);
        }
        if (e + 32 < nv) {  // the next ones on their way
          v_next = e + 32 + lane < nv ? vecs[warp * CAP + e + 32 + lane] : v0;
          if (!RESIDENT) raw_next = fetch(v_next);
        }
        unsigned in = 0;
#pragma unroll
        for (int j = 0; j < VEC; ++j) in |= (mine && x[j] >= near ? 1u : 0u) << j;
        const int here = __popc(in);
        int at = n + warp_before_int(here);
        n += warp_sum_int(here);
        if (LIST && n > CAP) {
          fits = false;
          break;
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          if (in >> j & 1) {
            const unsigned v31 = w(x[j]);
            mass_listed += v31;
            if (MASS) mass -= small ? w.bits(x[j]) : v31;
            if (LIST) {
              xs[warp * CAP + at] = x[j];
              ids[warp * CAP + at] = v * VEC - head + j;
              ++at;
            }
          }
      }
    }
    if (!fits && MASS) {  // too many to set right: the plain sum
      mass = mass_listed = 0;
      each([&](float x) { mass += w(x); });
    }
    mass = warp_sum64(mass);
    mass_listed = warp_sum64(mass_listed);
    if (lane == 0) {
      s.low[warp].mass = mass;
      s.held[warp].mass = mass_listed;
      s.held[warp].ties = 0;
      s.listed[warp] = n;
    }
    if (__syncthreads_or(!fits)) return -1;
    return warp_sum_int(lane < NW ? s.listed[lane] : 0);
  }

  __device__ u64 total_mass() const { return warp_sum64(lane < NW ? s.held[lane].mass : 0ull); }
  __device__ u64 total_low() const { return warp_sum64(lane < NW ? s.low[lane].mass : 0ull); }

  // Sum over all threads, known to all.
  __device__ u64 total_of(u64 v) {
    v = warp_sum64(v);
    __syncthreads();
    if (lane == 0) s.held[warp].mass = v;
    __syncthreads();
    return total_mass();
  }

  // Counts and weights of the keys in [lo, lo + 2^bits), in stretches of 2^shift.
  __device__ void histogram(unsigned lo, int bits, int shift) {
    const unsigned digits = 1u << (bits - shift);  // at most 256
    __syncthreads();
    for (int i = threadIdx.x; i < 256; i += NW * 32) s.cnt[i] = s.lo[i] = s.hi[i] = s.over[i] = 0;
    __syncthreads();
    each([&](float x) {
      const unsigned k = K::of(x);
      if (k >= lo && ((k - lo) >> shift) < digits) {
        // a weight goes in as two halves of 16 bits, with native 32-bit adds; what a part overflows is
        // carried into the next one
        const unsigned d = (k - lo) >> shift, v = w(x), half = v & 0xffffu;
        atomicAdd(&s.cnt[d], 1u);
        const unsigned old = atomicAdd(&s.lo[d], half);
        const unsigned up = (v >> 16) + (old + half < old ? 0x10000u : 0u);
        const unsigned old_hi = atomicAdd(&s.hi[d], up);
        if (old_hi + up < old_hi) atomicAdd(&s.over[d], 1u);
      }
    });
    __syncthreads();
  }

  // Selection over the keys in [from, top]: the token at which, in falling order, the count (by_count) or
  // the weight reaches `target` >= 1, which the caller knows to be reached.  `bits`, `shift` are those of
  // the histogram that stands (bits 0: only one key).
  __device__ Cut select(bool by_count, u64 target, unsigned from, int bits, int shift, bool *stands) {
    unsigned lo = from;
    u64 above_cnt = 0, above_mass = 0;  // of the keys above those in question
    while (bits > 0) {
      if (warp == 0) {
        // lane 0 has the 8 highest digits, 248 to 255, lane 1 the 8 below them
        const int d0 = 248 - lane * 8;
        unsigned cnt[8];
        u64 mass[8], m = 0;
        unsigned c = 0;
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
          const uint4 n4 = *reinterpret_cast<const uint4 *>(&s.cnt[d0 + i]),
                      l4 = *reinterpret_cast<const uint4 *>(&s.lo[d0 + i]),
                      h4 = *reinterpret_cast<const uint4 *>(&s.hi[d0 + i]),
                      o4 = *reinterpret_cast<const uint4 *>(&s.over[d0 + i]);
          cnt[i] = n4.x; cnt[i + 1] = n4.y; cnt[i + 2] = n4.z; cnt[i + 3] = n4.w;
          mass[i] = ((u64)o4.x << 48) + ((u64)h4.x << 16) + l4.x;
          mass[i + 1] = ((u64)o4.y << 48) + ((u64)h4.y << 16) + l4.y;
          mass[i + 2] = ((u64)o4.z << 48) + ((u64)h4.z << 16) + l4.z;
          mass[i + 3] = ((u64)o4.w << 48) + ((u64)h4.w << 16) + l4.w;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          c += cnt[i];
          m += mass[i];
        }
        u64 bc = above_cnt + (unsigned)warp_before_int((int)c), bm = above_mass + warp_before64(m);
        const u64 at = by_count ? bc : bm, step = by_count ? (u64)c : m;
        if (at < target && at + step >= target) {
          bool found = false;
#pragma unroll
          for (int i = 7; i >= 0; --i)
            if (!found) {
              if ((by_count ? bc + cnt[i] : bm + mass[i]) >= target) {
                found = true;
                s.digit = d0 + i;
              } else {
                bc += cnt[i];
                bm += mass[i];
              }
            }
          s.above_cnt = bc;
          s.above_mass = bm;
          s.ranked = 0;
        }
      }
      __syncthreads();
      lo += s.digit << shift;
      above_cnt = s.above_cnt;
      above_mass = s.above_mass;
      bits = shift;
      if (bits == 0) break;
      const unsigned count = s.cnt[s.digit];
      if (count <= 32) {  // rank them
        each([&](float x) {
          const unsigned k = K::of(x);
          if (k >= lo && ((k - lo) >> bits) == 0) {
            const int at = atomicAdd(&s.ranked, 1);
            s.keys[at] = k;
            s.weights[at] = w(x);
          }
        });
        __syncthreads();
        if (warp == 0) {
          const unsigned k = lane < (int)count ? s.keys[lane] : 0, v = lane < (int)count ? s.weights[lane] : 0;
          unsigned gt = 0, ge = 0;
          u64 mass_gt = 0, mass_ge = 0;
          for (int i = 0; i < (int)count; ++i) {
            const unsigned k2 = __shfl_sync(0xffffffffu, k, i), v2 = __shfl_sync(0xffffffffu, v, i);
            gt += k2 > k;
            ge += k2 >= k;
            mass_gt += k2 > k ? v2 : 0;
            mass_ge += k2 >= k ? v2 : 0;
          }
          const bool here = lane < (int)count &&
                            (by_count ? above_cnt + gt < target && above_cnt + ge >= target
                                      : above_mass + mass_gt < target && above_mass + mass_ge >= target);
          const unsigned who = __ballot_sync(0xffffffffu, here);
          if (lane == __ffs(who) - 1) {
            s.found_key = k;
            s.above_cnt = above_cnt + gt;
            s.above_mass = above_mass + mass_gt;
          }
        }
        __syncthreads();
        lo = s.found_key;
        above_cnt = s.above_cnt;
        above_mass = s.above_mass;
        break;
      }
      shift = max(0, bits - 8);
      histogram(lo, bits, shift);
      *stands = false;
    }
    Cut c;
    c.key = lo;
    const u64 weight = w(K::value(lo));
    if (by_count)
      c.ties = (unsigned)(target - above_cnt);
    else
      c.ties = (unsigned)((target - above_mass + weight - 1) / weight);  // weight > 0: it moved the sum
    c.mass = above_mass + c.ties * weight;
    __syncthreads();
    return c;
  }

  __device__ __forceinline__ bool above(float x, const Cut &c, unsigned m) const {
    return K::of(x) > c.key && w(x) >= m;
  }

  // Reduces each warp's Held over its lanes; all threads then know the warp that the running sum
  // passes `target` in, what is left of the target and of the ties before it.
  __device__ void pick_warp(u64 mass, int ties, unsigned tie_weight, u64 *target, unsigned *ties_left) {
    mass = warp_sum64(mass);
    ties = warp_sum_int(ties);
    if (lane == 0) {
      s.held[warp].mass = mass;
      s.held[warp].ties = ties;
    }
    __syncthreads();
    find_warp(tie_weight, target, ties_left);
  }
  __device__ void find_warp(unsigned tie_weight, u64 *target, unsigned *ties_left) {
    if (warp == 0) {  // a lane a warp
      const Held h = lane < NW ? s.held[lane] : Held{0, 0};
      const unsigned before_t = (unsigned)warp_before_int((int)h.ties);
      const unsigned left = *ties_left > before_t ? *ties_left - before_t : 0;
      const u64 here = h.mass + (u64)min(left, h.ties) * tie_weight;
      const u64 before = warp_before64(here);
      const unsigned hit = __ballot_sync(0xffffffffu, lane < NW && before + here > *target);
      const int who = hit ? __ffs(hit) - 1 : NW - 1;
      if (lane == who) {
        s.winner = who;
        s.target = *target - before;
        s.ties_left = left;
      }
    }
    __syncthreads();
    *target = s.target;
    *ties_left = s.ties_left;
  }

  // 32 tokens, one a lane, in order: the first at which the running sum passes the target.
  // Returns the lane, or 32 with the target and the ties moved on.
  __device__ int step(float x, bool valid, const Cut &c, unsigned m, unsigned tie_weight,
                      u64 *target, unsigned *ties_left) const {
    const bool tie = valid && K::of(x) == c.key;
    const unsigned ties = __ballot_sync(0xffffffffu, tie);
    const unsigned rank = __popc(ties & ((1u << lane) - 1));
    u64 v = 0;
    if (tie && rank < *ties_left) v = tie_weight;
    if (valid && above(x, c, m)) v = w(x);
    const u64 before = warp_before64(v);
    const unsigned hit = __ballot_sync(0xffffffffu, before + v > *target);
    if (hit) return __ffs(hit) - 1;
    *target -= __shfl_sync(0xffffffffu, before + v, 31);
    *ties_left -= min(*ties_left, (unsigned)__popc(ties));
    return 32;
  }

  // The drawn token, valid in every thread.  `target` < the kept weight.  `sums_ready`: held[] is the sums
  // by warp of the kept tokens above the cut, and of the ties.
  __device__ int draw(const Cut &c, unsigned m, u64 target, bool sums_ready) {
    const unsigned wc = w(K::value(c.key)), tie_weight = wc >= m ? wc : 0;
    unsigned left = c.ties;
    if (threadIdx.x == 0) s.token = -1;
    if (sums_ready) {
      __syncthreads();
      find_warp(tie_weight, &target, &left);
    } else {
      u64 mass = 0;
      int ties = 0;
      each([&](float x) {
        const unsigned k = K::of(x);
        if (k > c.key) {
          const unsigned v = w(x);
          if (v >= m) mass += v;
        }
        ties += k == c.key ? 1 : 0;
      });
      __syncthreads();
      pick_warp(mass, ties, tie_weight, &target, &left);
    }
    const int winner = s.winner;
    if (listed) {
      if (warp == winner) {
        const int n = s.listed[warp];
        for (int i0 = 0; i0 < n; i0 += 32) {
          const int i = i0 + lane;
          const bool valid = i < n;
          const float x = valid ? xs[warp * CAP + i] : -INFINITY;
          const int hit = step(x, valid, c, m, tie_weight, &target, &left);
          if (hit < 32) {
            if (lane == hit) s.token = ids[warp * CAP + i];
            break;
          }
        }
      }
      __syncthreads();
      return s.token;
    }
    // the row: the winner's range is split over the warps again, until it is short
    const int vectors = (V + head + VEC - 1) / VEC, each_warp = (vectors + NW - 1) / NW;
    int a = max(0, min(each_warp * winner, vectors) * VEC - head),
        b = min(min(each_warp * (winner + 1), vectors) * VEC - head, V);
    while (NW > 1 && b - a > 128) {
      __syncthreads();
      const int piece = (b - a + NW - 1) / NW, p0 = a + piece * warp, p1 = min(b, p0 + piece);
      u64 mass = 0;
      int ties = 0;
      for (int i = p0 + lane; i < p1; i += 32) {
        const float x = token(i);
        if (above(x, c, m)) mass += w(x);
        ties += K::of(x) == c.key ? 1 : 0;
      }
      pick_warp(mass, ties, tie_weight, &target, &left);
      a += piece * s.winner;
      b = min(b, a + piece);
    }
    if (warp == 0) {
      for (int i0 = a; i0 < b; i0 += 32) {
        const int i = i0 + lane;
        const bool valid = i < b;
        const float x = valid ? token(i) : -INFINITY;
        const int hit = step(x, valid, c, m, tie_weight, &target, &left);
        if (hit < 32) {
          if (lane == hit) s.token = i;
          break;
        }
      }
    }
    __syncthreads();
    return s.token;
  }
};

template <int DT, int NW, bool RESIDENT>
__global__ void __launch_bounds__(NW * 32, NW == 16 && !RESIDENT ? 2 : 1) sample_kernel(SampleArgs a) {
  typedef typename Elem<DT>::T E;
  typedef Key<DT> K;
  extern __shared__ __align__(16) unsigned char mem[];
  __shared__ Shared<NW> s;
  const long long n = blockIdx.x;
  const E *row = static_cast<const E *>(a.logits) + n * a.row_stride;
  const float T = a.temperatures ? a.temperatures[n] : a.temperature;
  const float p = a.top_ps ? a.top_ps[n] : a.top_p;
  const float mp = a.min_ps ? a.min_ps[n] : a.min_p;
  int k = a.top_ks ? a.top_ks[n] : a.top_k;
  Sampler<DT, NW, RESIDENT> r(s, mem, row, a.V);
  const float X = r.maximum();
  const bool usable = T >= 0.0f && T < INFINITY && p >= 0.0f && p <= 1.0f && mp >= 0.0f &&
                      mp <= 1.0f && k >= 0 && X > -INFINITY;
  if (!usable) {
    if (threadIdx.x == 0) {
      a.tokens[n] = -1;
      if (a.logprobs) a.logprobs[n] = NAN;
    }
    return;
  }
  if (T == 0.0f) k = 1;
  if (k >= a.V) k = 0;
  r.w.X = X;
  r.w.infinite = X == INFINITY;
  r.w.per = T == 0.0f ? 0.0f : fminf(__fdiv_rn(kLog2e, T), 3.4e38f);
  const unsigned p24 = (unsigned)__float2int_rn(p * 16777216.0f);
  const unsigned m = __float2uint_ru(mp * 2147483648.0f);
  const unsigned u24 = (unsigned)min(max(__float2int_rd(a.u[n] * 16777216.0f), 0), 16777215);
  const bool by_p = p24 < (1u << 24), filters = k > 0 || by_p || m > 0;
  const bool need_all = by_p && k == 0;  // top-p's share is of the weight of every token
  const unsigned top = K::of(X);
  auto below = [&](float z) {  // the value at -z below the maximum
    return T == 0.0f || r.w.infinite ? X : X - z / r.w.per;
  };
  r.whole = RESIDENT && a.V <= kOwnList;
  Cut cut;
  u64 kept;
  bool sums_ready = false;
  if (!filters && !r.whole) {
    r.template weigh<true, false>(below((float)kListZ));
    // the sums by warp of every token, whatever pass 2 made of them
    if (threadIdx.x < NW) s.held[threadIdx.x].mass += s.low[threadIdx.x].mass;
    __syncthreads();
    cut.key = 0;
    cut.ties = 0;
    kept = r.total_mass();
    sums_ready = true;
  } else {
    u64 all = 0, listed_mass = 0;
    float near = 0.0f;
    bool enough = false, have_all = need_all;
    if (r.whole) {
      u64 mass = 0;
      r.each([&](float x) { mass += r.w(x); });
      all = r.total_of(mass);
      have_all = true;
    } else {
      int listed = -1, z = kListZ;
      for (int i = 0; i < kListTries && listed < 0; ++i) {
        z = kListZ >> i;
        near = below((float)z - 0.002f);  // so that pass 2's bits are sure to show every token from here up
        if (need_all && i == 0) {
          // ... also where neighbouring floats are far apart for the temperature, and this one weighs less than 2^-12
          if (r.w.bits(near) < 1u << 19 && near < X) near = nextafterf(near, X);
          listed = r.template weigh<true, true>(near);
          all = r.total_low() + r.total_mass();  // also where the list did not fit
        } else {
          listed = r.template weigh<false, true>(near);
        }
        listed_mass = r.total_mass();
        if (listed < 0) __syncthreads();  // before the sums are written again
      }
      // does the cut lie among the listed tokens?
      const unsigned low = (0x80000000u >> z) + (0x80000000u >> (z + 8));  // above any unlisted weight
      enough = listed > 0 && (k > 0   ? listed >= k || (!by_p && m >= low)
                              : by_p ? listed_mass >= share(all, p24)
                                     : m >= low);
      r.listed = enough;
      if (enough && listed < k) k = 0;  // top-k keeps more than min-p does
    }
    const unsigned from = K::of(enough ? near : below(kZeroZ));
    // one histogram for both cuts
    const int bits = 32 - __clz(top - from), shift = max(0, bits - 8);
    bool stands = false;
    // top-k, unless fewer tokens than that weigh anything
    cut.key = from;  // everything from `from` up
    cut.ties = 0xffffffffu;
    cut.mass = listed_mass;
    if (k > 0 && !enough) {
      u64 c = 0;
      r.each([&](float x) { c += K::of(x) >= from ? 1u : 0u; });
      if (r.total_of(c) < (u64)k) k = 0;
    }
    if (k > 0) {
      if (bits > 0) r.histogram(from, bits, shift);
      stands = true;
      cut = r.select(true, (u64)k, from, bits, shift, &stands);
    } else if (!enough) {  // the weight of everything from `from` up
      if (have_all) {
        cut.mass = all;
      } else {
        u64 mass = 0;
        r.each([&](float x) { mass += r.w(x); });
        cut.mass = r.total_of(mass);
      }
    }
    if (by_p) {
      const u64 need = share(need_all ? all : cut.mass, p24);
      if (!stands && bits > 0) r.histogram(from, bits, shift);
      cut = r.select(false, need > 0 ? need : 1, from, bits, shift, &stands);
    }
    kept = cut.mass;
    if (m > 0) {  // the weight that min-p leaves
      u64 mass = 0;
      int ties = 0;
      r.each([&](float x) {
        const unsigned key = K::of(x);
        if (key > cut.key) {
          const unsigned v = r.w(x);
          if (v >= m) mass += v;
        }
        ties += key == cut.key ? 1 : 0;
      });
      mass = warp_sum64(mass);
      ties = warp_sum_int(ties);
      __syncthreads();
      if (r.lane == 0) {
        s.held[r.warp].mass = mass;
        s.held[r.warp].ties = ties;
      }
      __syncthreads();
      const unsigned wc = r.w(K::value(cut.key));
      const u64 n_ties = warp_sum64(r.lane < NW ? (u64)s.held[r.lane].ties : 0ull);
      kept = r.total_mass() + (wc >= m ? (n_ties < cut.ties ? n_ties : cut.ties) * wc : 0);
      sums_ready = true;
    }
  }
  const int token = r.draw(cut, m, share(kept, u24), sums_ready);
  if (threadIdx.x == 0) {
    a.tokens[n] = token;
    if (a.logprobs) {
      const float x = r.token(token < 0 ? 0 : token);
      const float z = r.w.infinite || T == 0.0f ? 0.0f : __fmul_rn(__fsub_rn(x, X), r.w.per);
      a.logprobs[n] = token < 0 ? NAN : (z - log2f((float)kept * (1.0f / 2147483648.0f))) * 0.69314718055994531f;
    }
  }
}

template <int DT, int NW, bool RESIDENT>
cudaError_t launch(const SampleArgs &a, long long N, cudaStream_t s) {
  // a resident row starts at its first vector's place and is filled up to whole vectors
  constexpr size_t list = 3 * kListTokens * 4;
  auto row = [](int V) { return RESIDENT ? (size_t)((V + 16 + 3) / 4 * 4) * 4 : 0; };
  const size_t smem = row(a.V) + (RESIDENT && a.V <= kOwnList ? 0 : list);
  // The limit is the kernel's, shared by all host threads: the most that any call wants, never this call's own.
  const cudaError_t e = cudaFuncSetAttribute(sample_kernel<DT, NW, RESIDENT>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)(row(kResident) + list));
  if (e != cudaSuccess) return e;
  sample_kernel<DT, NW, RESIDENT><<<(unsigned)N, NW * 32, smem, s>>>(a);
  return cudaGetLastError();
}
// Warps a row: few for many rows, which share the SMs; many for few rows, where only the time of one counts.
// Measured, bfloat16, top_k 50 and top_p 0.95, us:
//     rows x tokens    1 warp   4 warps   8 warps   16 warps   32 warps
//        656 x 250       20.1      11.8
//      2,048 x 250       23.7      31.6
//        100 x 1,000               17.7                 11.5
//        300 x 1,000               18.5                 22.3
//        656 x 8,193                         55.4       60.1
//          1 x 16,384                        11.3        9.7
//          1 x 131,072                                  26.5       24.4
// Wide rows are read twice, and two a SM at a time are what L2 holds (2,048 x 131,072, top_p 0.9, on one card: 262 us;
// three of 8 warps 286, one of 32 warps 314).
template <int DT> cudaError_t launch(const SampleArgs &a, long long N, cudaStream_t s) {
  constexpr int kSMs = 152;
  if (a.V <= 256) return N > 8 * kSMs ? launch<DT, 1, true>(a, N, s) : launch<DT, 4, true>(a, N, s);
  if (a.V <= kOwnList) return N > kSMs ? launch<DT, 4, true>(a, N, s) : launch<DT, 16, true>(a, N, s);
  if (a.V <= kResident)
    return N > 2 * kSMs ? launch<DT, 8, true>(a, N, s) : launch<DT, 16, true>(a, N, s);
  return N > 2 * kSMs ? launch<DT, 16, false>(a, N, s) : launch<DT, 32, false>(a, N, s);
}

}  // namespace
}  // namespace tdt

extern "C" int tdt_sample(const void *logits, const int64_t sizes[2], int64_t row_stride,
                          int dtype, const float *uniforms, const float *temperatures,
                          const int32_t *top_ks, const float *top_ps, const float *min_ps,
                          double temperature, int64_t top_k, double top_p, double min_p,
                          int32_t *tokens, float *logprobs, void *stream) {
  using namespace tdt;
  if (!sizes) return TDT_ERR_NULL_POINTER;
  if (dtype != TDT_DTYPE_F32 && dtype != TDT_DTYPE_F16 && dtype != TDT_DTYPE_BF16)
    return TDT_ERR_BAD_DTYPE;
  const int64_t N = sizes[0], V = sizes[1];
  if (N < 0 || N > 2147483647LL || V < 1 || V > (1 << 24)) return TDT_ERR_BAD_SIZES;
  if (row_stride < 0) return TDT_ERR_BAD_STRIDES;
  if (!(temperature >= 0.0) || !(temperature <= 3.0e38) || !(top_p >= 0.0 && top_p <= 1.0) ||
      !(min_p >= 0.0 && min_p <= 1.0) || top_k < 0)
    return TDT_ERR_BAD_SAMPLING;
  if (N == 0) return TDT_OK;
  if (!logits || !uniforms || !tokens) return TDT_ERR_NULL_POINTER;
  const uintptr_t es = dtype == TDT_DTYPE_F32 ? 4 : 2;
  if ((uintptr_t)logits % es != 0 ||
      ((uintptr_t)uniforms | (uintptr_t)temperatures | (uintptr_t)top_ks | (uintptr_t)top_ps |
       (uintptr_t)min_ps | (uintptr_t)tokens | (uintptr_t)logprobs) % 4 != 0)
    return TDT_ERR_BAD_ALIGNMENT;
  SampleArgs a;
  a.logits = logits;
  a.row_stride = row_stride;
  a.V = (int)V;
  a.u = uniforms;
  a.temperatures = temperatures;
  a.top_ks = top_ks;
  a.top_ps = top_ps;
  a.min_ps = min_ps;
  a.temperature = (float)temperature;
  a.top_k = top_k > V ? 0 : (int)top_k;
  a.top_p = (float)top_p;
  a.min_p = (float)min_p;
  a.tokens = tokens;
  a.logprobs = logprobs;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == TDT_DTYPE_F32   ? launch<kF32>(a, N, s)
                        : dtype == TDT_DTYPE_F16 ? launch<kF16>(a, N, s)
                                                 : launch<kBF16>(a, N, s);
  return e == cudaSuccess ? TDT_OK : TDT_ERR_CUDA;
}
