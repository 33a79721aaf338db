// tdt_logprobs.cu -- log-probabilities of given tokens, entropy, the most probable alternatives, and the gradient
// (include/tdt_decoder.h, tdt_token_logprobs_*).
//
// With m the maximum of a row x, z_i = x_i - m, s = sum e^z_i and t = sum e^z_i z_i:
//   logprob = z_t - ln s,   entropy = ln s - t / s,
//   dx_i = -p_i (a + sum c + b (ln p_i + entropy)) + the given token's and the alternatives' own a and c_j,
//   ln p_i = z_i - ln s.
// An entry of -inf has p = 0; its logarithm (in base 2) is held above -200, in bfloat16 above about -2^31, in products with p, which is
// 0 there.  A weight b whose product with that would leave float32's range is formed 2^-k times, and p 2^k times.
//
// Forward: one read of the row in 16-byte vectors (whatever the row's alignment: elements before the first and after the last
// whole vector go one by one).  Arithmetic is in base 2 against a whole number R near the maximum,
//   z_i = x_i L - R (one fma; L = log2 e in float32),   s = sum 2^z_i,   t = sum 2^z_i z_i,
// so z is rounded once, at its own size, and what L is off by stays in differences to the maximum: m L - R is the same
// product.  A thread holds its own R, s and t; R moves only where the maximum has grown by 8.  They are joined in a
// fixed order.  R starts at -2^24: what lies far below, masked tokens (-inf, the type's lowest number), has weight 0 wherever it
// stands, so a thread that sees nothing else has sums of 0.  Where m L is past 2^24 on either side, and whole numbers are more than
// float32 holds, x_i - m is formed instead.
// A row belongs to a warp (short rows), a CTA of 128 or 256 threads, or a cluster of CTAs (few or long rows), whose CTAs have a stretch of it each and
// exchange their results through distributed shared memory.
// Alternatives: at least n_top elements reach a threshold that comes from the threads' maxima (the ceil(n_top / warps)-th largest
// of each warp, the least of the warps); only threads whose maximum reaches it, hardly more than n_top, look again, at the
// batches of vectors whose maximum does.  What reaches it is listed in shared memory and ranked by (value, index): the order in which the list
// fills does not matter.  A list that overflows (many equal elements) is given up for n_top passes over the row.
// Backward: a read and a write of the row; in one call with the forward pass, the row comes in bulk copies that are all asked for
// at once, and waits in shared memory (put there by the threads, which loaded a batch ahead, it took 11 us more of 173).
//
// 4,096 x 50,257 bfloat16, a quarter of the rows padding: forward 68 us, backward 125 us (5.8 TB/s), both in one call 147 us
// (4.9 TB/s: reading and writing a row take turns, four CTAs an SM, 60 % of the issue slots).  Masked tokens cost no more than others,
// in stretches, too (1,024 x 131,072 bfloat16, a tenth or seven of the tokens allowed: 45 us, all: 46).  2,048 x 131,072 bfloat16: 96 us (5.6
// TB/s), with twenty alternatives 111 us: what follows the read, threshold, list, ranks, is latency that four CTAs an SM cover in
// part.  656 x 8,193 float32: 10 us and 11 us, latency.  A whole row a CTA beats clusters of smaller stretches (131,072 scored: two CTAs 104 us, four 143).
#include <cooperative_groups.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "../../include/tdt_decoder.h"
#include "tdt_rowio.cuh"
#include "tdt_tc.cuh"

namespace tdt {
namespace {

namespace cg = cooperative_groups;

constexpr int kBlock = 256;
constexpr int kNarrow = 128;   // threads of a CTA where rows are many and not long
constexpr int kMostTop = 64;
constexpr int kMostCtas = 8;   // of a cluster
constexpr int kMostBatches = 5;  // of a stretch that is kept: 64 KB and a vector in 16 KB each (kNarrow: 40 KB in 8 KB)
constexpr float kLn2f = 0.69314718055994531f;
constexpr float kLeastZ = -200.0f;  // 2^-200 is 0
// log2 of a bound of c1 that keeps its products with held logarithms in float32: of under 2^8, in bfloat16 of under 2^31
template <int DT> constexpr int kMostSlope = DT == kBF16 ? 96 : 119;
constexpr float kLazy = 8.0f;
constexpr float kMostR = 16777216.0f;  // whole numbers to +-2^24 are exact, and x L - R is held to half a unit where x is the maximum

struct RowArgs {
  const void *x;
  void *dx;
  long long sx, sdx;  // row strides
  const long long *tokens;
  float *logprobs, *entropy, *top_logprobs;
  float2 *stats;
  int *top_tokens;
  const float *in_entropy;
  const float2 *in_stats;
  const int *in_top;
  const float *ga, *gb, *gc;
  unsigned N;
  int V, K;
  int cta_bits;       // log2 of the CTAs of a row
  int keep;           // vectors of a stretch that stay in dynamic shared memory for the backward pass (0: none do)
};

// What a row's gradient is formed with, each twice: 2^l (c0 + c1 l), l = k + log2 p = y L + neg + sum.
struct Slopes {
  float2 neg, sum, c0, c1;
};

// max that keeps NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// A vector's elements as float32.  In bfloat16 what lies below -2^30 (or is -inf) becomes -2^30, two elements an instruction, so that
// products with its weight, which is 0, are 0 wherever the reference is not below -2^24.  (The other types' z is held above kLeastZ
// instead.)
template <int DT> __device__ __forceinline__ void unpack_held(uint4 raw, float *v) {
  if constexpr (DT == kBF16) {
    unsigned w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(w[i]) : "r"(0xce80ce80u));
    raw = make_uint4(w[0], w[1], w[2], w[3]);
  }
  unpack<DT>(raw, v);
}
template <int DT> __device__ __forceinline__ float2 held(float2 z) {
  return DT == kBF16 ? z : make_float2(max_nan(z.x, kLeastZ), max_nan(z.y, kLeastZ));
}
// A vector's gradient but for the tokens with a part of their own.  ENTROPY: c1 is not 0.
template <int DT, bool ENTROPY> __device__ __forceinline__ void slopes(float (&y)[Vec<DT>::N], const Slopes &c) {
#pragma unroll
  for (int i = 0; i < Vec<DT>::N; i += 2) {
    const float2 lp = add2(fma2(make_float2(y[i], y[i + 1]), make_float2(kLog2e, kLog2e), c.neg), c.sum);
    const float2 f = mul2(make_float2(fast_exp2(lp.x), fast_exp2(lp.y)), ENTROPY ? fma2(c.c1, held<DT>(lp), c.c0) : c.c0);
    y[i] = f.x;
    y[i + 1] = f.y;
  }
}
// A vector's maximum, NaN left out.
template <int DT> __device__ __forceinline__ float vector_max(uint4 raw) {
  if constexpr (DT == kF32) {
    return fmaxf(fmaxf(__uint_as_float(raw.x), __uint_as_float(raw.y)), fmaxf(__uint_as_float(raw.z), __uint_as_float(raw.w)));
  } else {
    unsigned a, b;
    if constexpr (DT == kBF16) {
      asm("max.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(raw.x), "r"(raw.y));
      asm("max.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(raw.z), "r"(raw.w));
      asm("max.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
      return fmaxf(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u));
    } else {
      asm("max.f16x2 %0, %1, %2;" : "=r"(a) : "r"(raw.x), "r"(raw.y));
      asm("max.f16x2 %0, %1, %2;" : "=r"(b) : "r"(raw.z), "r"(raw.w));
      asm("max.f16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&a));
      return fmaxf(f.x, f.y);
    }
  }
}

// A stretch's maximum m, reference R (a whole number, -2^24 at least), sum of 2^z and sum of 2^z z, z = x log2 e - R.  s = 0: nothing
// that counts, whatever R.
struct Sums {
  float m, R, s, t;
};
__device__ __forceinline__ Sums join(const Sums &a, const Sums &b) {
  Sums r;
  r.m = fmaxf(a.m, b.m);
  r.R = fmaxf(a.R, b.R);
  const float da = fmaxf(a.R - r.R, kLeastZ), db = fmaxf(b.R - r.R, kLeastZ);
  const float fa = fast_exp2(da), fb = fast_exp2(db);
  r.s = a.s * fa + b.s * fb;
  r.t = fmaf(da, a.s, a.t) * fa + fmaf(db, b.s, b.t) * fb;
  return r;
}

// An element in the order of alternatives, the first the largest: by value (-0 equals 0), then by falling index.
__device__ __forceinline__ unsigned long long key_of(float v, int i) {
  const unsigned b = __float_as_uint(v + 0.0f);
  return (unsigned long long)(b & 0x80000000u ? ~b : b | 0x80000000u) << 32 | (0xffffffffu - (unsigned)i);
}
__device__ __forceinline__ float value_of(unsigned long long key) {
  const unsigned b = (unsigned)(key >> 32);
  return __uint_as_float(b & 0x80000000u ? b & 0x7fffffffu : ~b);
}
__device__ __forceinline__ int index_of(unsigned long long key) { return (int)(0xffffffffu - (unsigned)key); }

// Dynamic shared memory of a group (a warp or a block) where there are alternatives.
template <int T> struct TopShared {
  static constexpr int LIST = T == 32 ? 288 : 1024;
  static constexpr int GROUPS = T == 32 ? 1 : 16;  // of a thread's batches of vectors
  static constexpr int PAIRS = T == 32 ? 32 : 1024;
  unsigned long long list[LIST];
  float group_max[GROUPS][T];
  int pairs[PAIRS];  // groups of batches that reach the threshold: group * T + thread
};

// A group's shared memory.
template <int T> struct GroupShared {
  Sums sums[T / 32];
  float least[T / 32];
  unsigned long long best[T / 32];  // of the passes that stand in for a list that overflows
  int count, pairs;
  unsigned long long top[kMostTop];  // the stretch's own alternatives, ranked
  int top_n;
  Sums row;                // of the stretch, for the cluster
  float own_x[kMostTop + 1], own_add[kMostTop + 1];
  int own_at[kMostTop + 1];
};

// `bytes` (a multiple of 16) to shared memory, both addresses on 16 bytes; they arrive at `bar`.
__device__ __forceinline__ void bulk_load(void *to, const void *from, unsigned bytes, unsigned long long *bar) {
  asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(to)), "l"(from),
               "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

template <int T> __device__ __forceinline__ void group_sync() {
  if (T == 32)
    __syncwarp();
  else
    __syncthreads();
}

// The vectors [first, last) of 16 bytes that CTA `i` of 2^bits has of a row at p, and the elements before the first vector.
// (Divisions here took as many instructions as the exponentials of 50 elements a thread.)
struct Stretch {
  int head, first, last, vectors;
};
template <int DT> __device__ __forceinline__ Stretch stretch_of(const void *p, int V, int i, int bits) {
  Stretch s;
  s.head = min(head_elems<DT>(p), V);
  s.vectors = (V - s.head) / Vec<DT>::N;
  s.first = s.vectors * i >> bits;  // vectors <= 2^22, i < 8
  s.last = s.vectors * (i + 1) >> bits;
  return s;
}

template <int DT, bool FWD, bool BWD, int T>
__global__ void __launch_bounds__(T == kNarrow ? kNarrow : kBlock, T == kNarrow ? 8 : 4) rows_kernel(const __grid_constant__ RowArgs a) {
  typedef typename Elem<DT>::T E;
  constexpr int N = Vec<DT>::N, U = 4, WARPS = T / 32;
  constexpr bool IN_PLACE = BWD;  // the logits may be written in this kernel
  __shared__ GroupShared<T> shared[T == 32 ? kBlock / 32 : 1];
  GroupShared<T> &sh = shared[threadIdx.x / T];
  const int tid = threadIdx.x % T, lane = tid & 31, warp = tid >> 5;
  const int bits = T == 32 ? 0 : a.cta_bits, ctas = 1 << bits, part = T == 32 ? 0 : blockIdx.x & (ctas - 1);
  const unsigned n = T == 32 ? blockIdx.x * (kBlock / 32) + threadIdx.x / 32 : blockIdx.x >> bits;
  if (n >= a.N) return;  // a whole warp (T = 32)
  const E *x = static_cast<const E *>(a.x) + n * a.sx;
  const long long token = a.tokens[n];
  const bool real = token >= 0 && token < a.V;
  auto at = [&](int i) { return ld_elem<DT, IN_PLACE>(x + i); };
  const int K = a.K;
  // of the whole row: log2 p_i = x_i L - R - log2_s; R infinite: (x_i - m) L - log2_s
  float R = 0.0f, m = 0.0f, log2_s = 0.0f, ent = 0.0f;
  auto z_of = [&](float v) { return R < INFINITY ? fmaf(v, kLog2e, -R) : (v - m) * kLog2e; };
  extern __shared__ __align__(16) uint4 kept_row[];
  __shared__ unsigned long long full[kMostBatches];
  __shared__ int gave_up;
  TopShared<T> &lists = reinterpret_cast<TopShared<T> *>(kept_row + a.keep)[threadIdx.x / T];
  if (FWD && !real && part == 0) {
    const float none = token < 0 ? 0.0f : NAN;
    if (tid == 0) {
      a.logprobs[n] = none;
      if (a.entropy) a.entropy[n] = none;
      if (a.stats) a.stats[n] = make_float2(none, none);
    }
    for (int k = tid; k < K; k += T) {
      a.top_tokens[n * (long long)K + k] = -1;
      a.top_logprobs[n * (long long)K + k] = token < 0 ? -INFINITY : NAN;
    }
  }
  if (FWD && real) {
    const Stretch w = stretch_of<DT>(x, a.V, part, bits);
    const E *body = x + w.head;
    Sums r = {-INFINITY, -kMostR, 0.0f, 0.0f};
    float2 s2 = make_float2(0.0f, 0.0f), t2 = s2;  // running sums of even and odd elements
    auto grow = [&](float top) {
      r.m = fmaxf(r.m, top);
      const float y = top * kLog2e;
      if (y > r.R + kLazy) {
        const float now = rintf(y), down = fmaxf(r.R - now, kLeastZ), f = fast_exp2(down);
        t2 = make_float2(fmaf(down, s2.x, t2.x) * f, fmaf(down, s2.y, t2.y) * f);
        s2 = make_float2(s2.x * f, s2.y * f);
        r.R = now;
      }
    };
    const float2 L2 = make_float2(kLog2e, kLog2e);
    auto add_vector = [&](const float (&v)[N]) {
      const float2 neg = make_float2(-r.R, -r.R);
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        const float2 z = held<DT>(fma2(make_float2(v[i], v[i + 1]), L2, neg));
        const float2 p = make_float2(fast_exp2(z.x), fast_exp2(z.y));
        s2 = add2(s2, p);
        t2 = fma2(p, z, t2);
      }
    };
    // the elements outside whole vectors belong to the first CTA, one a thread
    const int tail = w.head + w.vectors * N, loose = w.head + a.V - tail;
    const int loose_at = part == 0 && tid < loose ? (tid < w.head ? tid : tail + tid - w.head) : -1;
    const float loose_x = loose_at >= 0 ? at(loose_at) : -INFINITY;
    const bool keep = BWD && T > 32 && a.keep > 0;
    // U vectors at a time, the next ones in flight.  Of each group of these batches a thread notes its maximum.
    constexpr int GROUPS = TopShared<T>::GROUPS;
    const int batches = (w.last - w.first + U * T - 1) / (U * T), per = (batches + GROUPS - 1) / GROUPS;  // batches of a group
    float best = -INFINITY;
    int group = 0, left = per;
    auto load = [&](int v0, uint4 (&raw)[U]) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (v0 + u * T < w.last) raw[u] = ld_row16<IN_PLACE>(reinterpret_cast<const uint4 *>(body + (long long)(v0 + u * T) * N));
    };
    auto take = [&](int v0, const uint4 (&raw)[U]) {
      float most = vector_max<DT>(raw[0]);
#pragma unroll
      for (int u = 1; u < U; ++u)
        if (v0 + u * T < w.last) most = fmaxf(most, vector_max<DT>(raw[u]));
      grow(most);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (v0 + u * T < w.last) {
          float v[N];
          unpack_held<DT>(raw[u], v);
          add_vector(v);
        }
      if (K > 0) {
        best = fmaxf(best, most);
        if (--left == 0) {
          lists.group_max[group++][tid] = best;
          best = -INFINITY;
          left = per;
        }
      }
    };
    uint4 raw[U];
    if (keep) {  // asked for at once, and waited for a batch at a time
      if constexpr (BWD && T > 32) {
        const int first = w.first, vectors = w.last - w.first;
        if (tid == 0) {
          gave_up = 0;
          for (int i = 0; i < batches; ++i) mbar_init(&full[i], 1);
          fence_mbar_init_cluster();
          for (int i = 0; i < batches; ++i) {
            const int here = min(U * T, vectors - i * U * T);
            arrive_expect_tx(&full[i], here * 16);
            bulk_load(kept_row + i * U * T, body + (long long)(first + i * U * T) * N, here * 16, &full[i]);
          }
        }
        __syncthreads();
        const Waiter wait{&gave_up};
        bool ok = true;
        for (int i = 0; i < batches; ++i) {
          ok = ok && wait(&full[i], 0);
          const int v0 = first + tid + i * U * T;
          if (!ok || v0 >= w.last) break;
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (v0 + u * T < w.last) raw[u] = kept_row[v0 + u * T - first];
          take(v0, raw);
        }
        if (!ok) {
          r.m = INFINITY;  // outputs become NaN
          if (tid == 0)    // copies in flight land before the CTA ends
            for (int i = 0; i < batches; ++i) Waiter::drain(&full[i], 0);
        }
      }
    } else {
      uint4 next[U];
      load(w.first + tid, raw);
      for (int v0 = w.first + tid; v0 < w.last; v0 += U * T) {
        load(v0 + U * T, next);
        take(v0, raw);
#pragma unroll
        for (int u = 0; u < U; ++u) raw[u] = next[u];
      }
    }
    if (K > 0 && group < GROUPS) lists.group_max[group++][tid] = best;  // each thread reads its own
    if (loose_at >= 0) {
      grow(loose_x);
      const float z = max_nan(fmaf(loose_x, kLog2e, -r.R), kLeastZ), p = fast_exp2(z);
      s2.x += p;
      t2.x = fmaf(p, z, t2.x);
    }
    r.s = s2.x + s2.y;
    r.t = t2.x + t2.y;
    if (K > 0) {
      // At least K elements reach the threshold: each warp all of whose lanes have vectors has ceil(K / such warps) lanes that
      // do; in a stretch too short for one, the first warp's lanes that have some.  (Where these are fewer than K, everything
      // is listed.)
      const int held_vectors = w.last - w.first, full = max(1, min(WARPS, held_vectors / 32));
      const int want = (K + full - 1) / full <= min(32, held_vectors) ? (K + full - 1) / full : 33;
      if (tid == 0) sh.count = sh.pairs = 0;
      if (warp >= full || want > 32) {
        if (lane == 0) sh.least[warp] = want > 32 ? -INFINITY : INFINITY;
      } else if (want <= 8) {  // the largest, one lane after the other
        const int bits = __float_as_int(r.m);
        int key = bits ^ (bits >> 31 & 0x7fffffff), top = 0;
        for (int i = 0; i < want; ++i) {
          top = __reduce_max_sync(0xffffffffu, key);
          if (lane == __ffs(__ballot_sync(0xffffffffu, key == top)) - 1) key = (int)0x80000000;
        }
        if (lane == 0) sh.least[warp] = __int_as_float(top ^ (top >> 31 & 0x7fffffff));
      } else {
        int ahead = 0;  // lanes with a larger maximum (equal ones: in order)
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float other = __shfl_sync(0xffffffffu, r.m, i);
          ahead += other > r.m || (other == r.m && i < lane);
        }
        if (ahead == want - 1) sh.least[warp] = r.m;
      }
      group_sync<T>();
      float threshold = sh.least[0];
#pragma unroll
      for (int i = 1; i < WARPS; ++i) threshold = fminf(threshold, sh.least[i]);
      threshold = fmaxf(threshold, -3.402823466e38f);  // not -inf entries
      auto note = [&](float v, int i) {
        if (v >= threshold) {
          const int k = atomicAdd(&sh.count, 1);
          if (k < TopShared<T>::LIST) lists.list[k] = key_of(v, i);
        }
      };
      auto look = [&](int v) {  // at a vector
        const uint4 x4 = ld_row16<IN_PLACE>(reinterpret_cast<const uint4 *>(body + (long long)v * N));
        if (vector_max<DT>(x4) >= threshold) {
          float y[N];
          unpack<DT>(x4, y);
#pragma unroll
          for (int i = 0; i < N; ++i) note(y[i], w.head + v * N + i);
        }
      };
      // Groups of batches that reach it are shared out, a vector a thread (a thread that looked through its own would wait
      // for memory once for each, and its warp for all of its lanes': 141 us against 111 of 2,048 x 131,072, n_top 20).
      if (r.m >= threshold) {
        for (int i = 0; i < group; ++i)
          if (lists.group_max[i][tid] >= threshold) {
            const int k = atomicAdd(&sh.pairs, 1);
            if (k < TopShared<T>::PAIRS)
              lists.pairs[k] = i * T + tid;
            else  // many equal elements
              for (int v = w.first + tid + i * per * U * T; v < min(w.last, w.first + (i + 1) * per * U * T); v += T) look(v);
          }
        if (loose_at >= 0) note(loose_x, loose_at);
      }
      group_sync<T>();
      const int found = min(sh.pairs, TopShared<T>::PAIRS), each = per * U;  // vectors of a pair
      for (int k = tid; k < found * each; k += T) {
        const int p = lists.pairs[k / each], v = w.first + p % T + (p / T * each + k % each) * T;
        if (v < w.last) look(v);
      }
    }
    // threads, then warps, then CTAs
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      Sums other;
      other.m = __shfl_xor_sync(0xffffffffu, r.m, o);
      other.R = __shfl_xor_sync(0xffffffffu, r.R, o);
      other.s = __shfl_xor_sync(0xffffffffu, r.s, o);
      other.t = __shfl_xor_sync(0xffffffffu, r.t, o);
      r = lane & o ? join(other, r) : join(r, other);
    }
    if (WARPS > 1) {
      if (lane == 0) sh.sums[warp] = r;
      __syncthreads();
      r = sh.sums[0];
#pragma unroll
      for (int i = 1; i < WARPS; ++i) r = join(r, sh.sums[i]);
    } else {
      __syncwarp();
    }
    if (K > 0) {
      const int count = sh.count;
      if (count <= TopShared<T>::LIST) {
        for (int i = tid; i < count; i += T) {
          const unsigned long long mine = lists.list[i];
          int rank = 0;
#pragma unroll 4
          for (int j = 0; j < count; ++j) rank += lists.list[j] > mine;
          if (rank < K) sh.top[rank] = mine;
        }
        if (tid == 0) sh.top_n = min(count, K);
      } else {  // the stretch again, once an alternative
        unsigned long long last = ~0ull;
        int found = 0;
        for (; found < K; ++found) {
          unsigned long long most = 0;  // of what comes after the last one
          auto offer = [&](float v, int i) {
            const unsigned long long key = key_of(v, i);
            if (v > -INFINITY && key < last && key > most) most = key;
          };
          for (int q = w.first * N + tid; q < w.last * N; q += T) offer(at(w.head + q), w.head + q);
          if (loose_at >= 0) offer(loose_x, loose_at);
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) {
            const unsigned long long other = __shfl_xor_sync(0xffffffffu, most, o);
            most = other > most ? other : most;
          }
          if (WARPS > 1) {
            __syncthreads();
            if (lane == 0) sh.best[warp] = most;
            __syncthreads();
            for (int i = 0; i < WARPS; ++i) most = sh.best[i] > most ? sh.best[i] : most;
          }
          if (most == 0) break;  // the same for all threads
          if (tid == 0) sh.top[found] = most;
          last = most;
        }
        if (tid == 0) sh.top_n = found;
      }
    }
    if constexpr (T > 32) {
      if (ctas > 1) {
        if (tid == 0) sh.row = r;
        cg::cluster_group cluster = cg::this_cluster();
        cluster.sync();
        r = *cluster.map_shared_rank(&sh.row, 0);
        for (int i = 1; i < ctas; ++i) r = join(r, *cluster.map_shared_rank(&sh.row, i));
      }
    }
    group_sync<T>();
    if (!(r.s > 0.0f && r.s < INFINITY && fabsf(r.m) * kLog2e <= kMostR) && fabsf(r.m) < INFINITY) {
      // NaN in the row, or numbers so large that a product with L loses whole units: against the maximum itself, by every CTA
      r.s = r.t = 0.0f;
      for (int i = tid; i < a.V; i += T) {
        const float z = max_nan((at(i) - r.m) * kLog2e, kLeastZ), p = fast_exp2(z);
        r.s += p;
        r.t = fmaf(p, z, r.t);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        r.s += __shfl_xor_sync(0xffffffffu, r.s, o);
        r.t += __shfl_xor_sync(0xffffffffu, r.t, o);
      }
      if (WARPS > 1) {
        if (lane == 0) sh.sums[warp] = r;
        __syncthreads();
        r.s = r.t = 0.0f;
        for (int i = 0; i < WARPS; ++i) {
          r.s += sh.sums[i].s;
          r.t += sh.sums[i].t;
        }
      }
      r.R = INFINITY;  // what z_of knows it by
    }
    const bool lost = !(r.s > 0.0f && r.s < INFINITY) || !(fabsf(r.m) < INFINITY);  // NaN, +inf, or nothing but -inf
    log2_s = lost ? NAN : log2f(r.s);
    ent = lost ? NAN : fmaxf((log2_s - r.t / r.s) * kLn2f, 0.0f);
    R = r.R;
    m = r.m;
    const float ln_s = lost ? NAN : (log2_s - z_of(m)) * kLn2f;
    auto ln_of = [&](float v) { return v - m - ln_s; };  // finite wherever v is
    if (part == 0) {
      if (tid == 0) {
        a.logprobs[n] = ln_of(at((int)token));
        if (a.entropy) a.entropy[n] = ent;
        if (a.stats) a.stats[n] = make_float2(lost ? NAN : m, ln_s);
      }
      if (K > 0) {
        int *to = a.top_tokens + n * (long long)K;
        float *lp = a.top_logprobs + n * (long long)K;
        int total = 0;
        if (lost) {
          for (int k = tid; k < K; k += T) {
            to[k] = -1;
            lp[k] = NAN;
          }
          total = K;
        } else if (ctas == 1) {
          total = sh.top_n;
          for (int k = tid; k < total; k += T) {
            to[k] = index_of(sh.top[k]);
            lp[k] = ln_of(value_of(sh.top[k]));
          }
        } else if constexpr (T > 32) {
          // each CTA's list is ranked; they come over together, and an entry's rank is its own plus those of the
          // others' entries before it
          cg::cluster_group cluster = cg::this_cluster();
          __syncthreads();  // the list's memory is free
          for (int q = tid; q < ctas * K; q += T) {
            const int i = q / K, k = q % K;
            lists.list[q] = k < *cluster.map_shared_rank(&sh.top_n, i) ? *cluster.map_shared_rank(&sh.top[k], i) : 0;
          }
          __syncthreads();
          for (int base = 0; base < ctas * K; base += T) {
            const int q = base + tid;
            const unsigned long long mine = q < ctas * K ? lists.list[q] : 0;
            total += __syncthreads_count(mine != 0);
            int rank = q % K;
            for (int j = 0; j < ctas && mine != 0 && rank < K; ++j) {
              if (j == q / K) continue;
              int lo = 0, hi = K;
              while (lo < hi) {  // entries of j before this one
                const int mid = (lo + hi) / 2;
                const bool before = lists.list[j * K + mid] > mine;
                lo = before ? mid + 1 : lo;
                hi = before ? hi : mid;
              }
              rank += lo;
            }
            if (mine != 0 && rank < K) {
              to[rank] = index_of(mine);
              lp[rank] = ln_of(value_of(mine));
            }
          }
          total = min(total, K);
        }
        if (total < K && warp == 0) {  // tokens that are not allowed fill up, the lowest first
          int k = total;
          for (int base = 0; base < a.V && k < K; base += 32) {
            const int i = base + lane;
            const bool none = i < a.V && at(i) == -INFINITY;
            const unsigned all = __ballot_sync(0xffffffffu, none);
            const int mine = k + __popc(all & ((1u << lane) - 1));
            if (none && mine < K) {
              to[mine] = i;
              lp[mine] = -INFINITY;
            }
            k += __popc(all);
          }
        }
      }
    }
  }
  if (BWD) {
    E *dx = static_cast<E *>(a.dx) + n * a.sdx;
    const Stretch w = stretch_of<DT>(dx, a.V, part, bits);
    const int tail = w.head + w.vectors * N, loose = w.head + a.V - tail;
    const int loose_at = part == 0 && tid < loose ? (tid < w.head ? tid : tail + tid - w.head) : -1;
    if (!real) {
      for (int v = w.first + tid; v < w.last; v += T)
        *reinterpret_cast<uint4 *>(dx + w.head + (long long)v * N) = make_uint4(0, 0, 0, 0);
      if (loose_at >= 0) dx[loose_at] = Elem<DT>::from_float(0.0f);
    } else {
      const float ga = a.ga ? a.ga[n] : 0.0f, gb = a.gb ? a.gb[n] : 0.0f;
      const int kept = a.gc ? K : 0;
      if (!FWD) {
        const float2 st = a.in_stats[n];
        m = st.x;
        R = rintf(m * kLog2e);
        if (!(fabsf(R) <= kMostR)) R = INFINITY;
        log2_s = st.y * kLog2e + (R < INFINITY ? fmaf(m, kLog2e, -R) : 0.0f);
        ent = a.gb ? a.in_entropy[n] : 0.0f;
      }
      // tokens with a part of their own that this CTA writes
      auto mine = [&](int i) {
        return i < w.head || i >= tail ? part == 0 : i >= w.head + w.first * N && i < w.head + w.last * N;
      };
      for (int j = tid; j <= kept; j += T) {
        const int i = j == kept ? (int)token : a.in_top[n * (long long)K + j];
        const bool in = i >= 0 && i < a.V;
        sh.own_at[j] = in ? i : -1;
        sh.own_add[j] = j == kept ? ga : a.gc[n * (long long)K + j];
        sh.own_x[j] = in && mine(i) ? at(i) : 0.0f;
      }
      const float loose_x = loose_at >= 0 ? at(loose_at) : 0.0f;
      if constexpr (FWD && T > 32) {
        if (ctas > 1) cg::this_cluster().sync();  // every read of the row, and of other CTAs' results, is done
      }
      group_sync<T>();
      float all = 0.0f;
      for (int j = 0; j <= kept; ++j) all += sh.own_add[j];
      // -p (all + gb (ln p + ent)), from l = k + log2 p; k = 0 but for weights of 2^96 and more
      float c0 = -fmaf(gb, ent, all), c1 = -gb * kLn2f, sum = -log2_s;
      const int k = (int)(__float_as_uint(c1) >> 23 & 255) - 126 - kMostSlope<DT>;  // |c1| < 2^(k + kMostSlope)
      if (k > 0) {
        const float down = __uint_as_float((unsigned)(127 - k) << 23);
        c1 *= down;
        c0 = -fmaf(gb * down, ent, all * down) - c1 * k;
        sum += k;
      }
      auto slope = [&](float y) {
        const float l = z_of(y) + sum;
        return fast_exp2(l) * fmaf(c1, max_nan(l, kLeastZ), c0);
      };
      const int mis = (int)((uintptr_t)(x + w.head) & 15);
      const Slopes pairs = {make_float2(-R, -R), make_float2(sum, sum), make_float2(c0, c0), make_float2(c1, c1)};
      auto finish = [&](uint4 raw, int v) {
        float y[N];
        unpack_held<DT>(raw, y);
        if (R < INFINITY) {
          if (c1 != 0.0f)
            slopes<DT, true>(y, pairs);
          else
            slopes<DT, false>(y, pairs);
        } else {
          unpack<DT>(raw, y);
#pragma unroll
          for (int i = 0; i < N; ++i) y[i] = slope(y[i]);
        }
        *reinterpret_cast<uint4 *>(dx + w.head + (long long)v * N) = pack<DT>(y);
      };
      const E *body = x + w.head;
      if (FWD && T > 32 && a.keep > 0 && mis == 0) {  // the thread's own vectors: the stretches are the same
        // (the choices outside the loop: 150 us for 154 of 4,096 x 50,257)
        auto finish_kept = [&](auto with_entropy) {
          const uint4 *from = kept_row + tid;
          uint4 *to = reinterpret_cast<uint4 *>(dx + w.head) + w.first + tid;
#pragma unroll 2
          for (int left = w.last - w.first - tid; left > 0; left -= T, from += T, to += T) {
            float y[N];
            unpack_held<DT>(*from, y);
            slopes<DT, decltype(with_entropy)::value>(y, pairs);
            *to = pack<DT>(y);
          }
        };
        if (!(R < INFINITY))
          for (int v = w.first + tid; v < w.last; v += T) finish(kept_row[v - w.first], v);
        else if (c1 != 0.0f)
          finish_kept(std::true_type());
        else
          finish_kept(std::false_type());
      } else if (mis == 0) {
        for (int v0 = w.first + tid; v0 < w.last; v0 += U * T) {
          uint4 raw[U];
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (v0 + u * T < w.last) raw[u] = ld_row16<IN_PLACE>(reinterpret_cast<const uint4 *>(body + (long long)(v0 + u * T) * N));
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (v0 + u * T < w.last) finish(raw[u], v0 + u * T);
        }
      } else {
        // The rows of logits and gradient lie differently to 16 bytes: a vector comes from two loads, each of
        // which holds some of its bytes.
        const unsigned char *low = reinterpret_cast<const unsigned char *>(body) - mis;
        for (int v0 = w.first + tid; v0 < w.last; v0 += 2 * T) {
          uint4 lo[2], hi[2];
#pragma unroll
          for (int u = 0; u < 2; ++u)
            if (v0 + u * T < w.last) {
              lo[u] = ld_row16_l1<IN_PLACE>(low + (long long)(v0 + u * T) * 16);
              hi[u] = ld_row16_l1<IN_PLACE>(low + (long long)(v0 + u * T) * 16 + 16);
            }
#pragma unroll
          for (int u = 0; u < 2; ++u)
            if (v0 + u * T < w.last) finish(funnel16(lo[u], hi[u], mis >> 2, (mis & 3) * 8), v0 + u * T);
        }
      }
      if (loose_at >= 0) dx[loose_at] = Elem<DT>::from_float(slope(loose_x));
      group_sync<T>();
      // each token with a part of its own is written again by the first that names it
      for (int j = tid; j <= kept; j += T) {
        const int i = sh.own_at[j];
        bool first = i >= 0 && mine(i);
        float add = 0.0f;
        for (int q = 0; q <= kept && first; ++q)
          if (sh.own_at[q] == i) {
            if (q < j) first = false;
            add += sh.own_add[q];
          }
        if (first) dx[i] = Elem<DT>::from_float(slope(sh.own_x[j]) + add);
      }
    }
  } else if constexpr (FWD && T > 32) {
    if (real && ctas > 1) cg::this_cluster().sync();  // nobody leaves while its results may be read
  }
}

bool known(int dtype) { return dtype == TDT_DTYPE_F32 || dtype == TDT_DTYPE_F16 || dtype == TDT_DTYPE_BF16; }

int check(const void *logits, const int64_t sizes[3], const int64_t *strides, bool grad, int dtype,
          const int64_t *tokens, RowArgs *a) {
  if (!sizes || !strides) return TDT_ERR_NULL_POINTER;
  if (!known(dtype)) return TDT_ERR_BAD_DTYPE;
  const int64_t N = sizes[0], V = sizes[1], K = sizes[2];
  if (N < 0 || N >= (int64_t)1 << 27 || V < 1 || V > 1 << 24) return TDT_ERR_BAD_SIZES;
  if (K < 0 || K > V || K > kMostTop) return TDT_ERR_BAD_TOP;
  if (strides[0] < 0 || (grad && strides[1] < V && N > 1)) return TDT_ERR_BAD_STRIDES;
  if (N == 0) return TDT_OK;
  if (!logits || !tokens) return TDT_ERR_NULL_POINTER;
  if ((uintptr_t)logits % (dtype == TDT_DTYPE_F32 ? 4 : 2) || (uintptr_t)tokens % 8) return TDT_ERR_BAD_ALIGNMENT;
  a->x = logits;
  a->sx = strides[0];
  a->tokens = reinterpret_cast<const long long *>(tokens);
  a->N = (unsigned)N;
  a->V = (int)V;
  a->K = (int)K;
  return TDT_OK;
}

// grad_out: aligned, and the logits themselves or apart from them
int check_grad(const RowArgs &a, void *grad_out, int64_t stride, int dtype) {
  const uintptr_t es = dtype == TDT_DTYPE_F32 ? 4 : 2;
  if (!grad_out) return TDT_ERR_NULL_POINTER;
  if ((uintptr_t)grad_out % es) return TDT_ERR_BAD_ALIGNMENT;
  const uintptr_t x0 = (uintptr_t)a.x, g0 = (uintptr_t)grad_out;
  const uintptr_t xn = ((uintptr_t)a.sx * (a.N - 1) + a.V) * es, gn = ((uintptr_t)stride * (a.N - 1) + a.V) * es;
  const bool same = x0 == g0 && (a.N == 1 || a.sx == stride);
  if (!same && g0 < x0 + xn && x0 < g0 + gn) return TDT_ERR_BAD_ALIASING;
  return TDT_OK;
}

bool off4(std::initializer_list<const void *> ptrs) {
  for (const void *p : ptrs)
    if ((uintptr_t)p % 4) return true;
  return false;
}

template <int DT, bool FWD, bool BWD, int T> cudaError_t launch_ctas(const RowArgs &a, cudaStream_t s) {
  const size_t smem = (size_t)a.keep * 16 + (FWD && a.K > 0 ? sizeof(TopShared<T>) : 0);
  if (FWD && smem > 0) {
    const cudaError_t e = cudaFuncSetAttribute(rows_kernel<DT, FWD, BWD, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               65536 + 16 + (int)sizeof(TopShared<T>));
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.N << a.cta_bits);
  cfg.blockDim = dim3(T);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 1 << a.cta_bits;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = FWD && a.cta_bits > 0 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, rows_kernel<DT, FWD, BWD, T>, a);
}
template <int DT, bool FWD, bool BWD> cudaError_t launch_rows(RowArgs a, cudaStream_t s) {
  const long long bytes = (long long)a.V * (DT == kF32 ? 4 : 2);
  if ((bytes <= 2048 || (bytes <= 8192 && a.N >= 1024)) && a.K <= 16 && a.N >= 8) {  // a warp a row (more alternatives take a warp long: 2,500 x 664: 137 us of 32, a CTA 37)
    const size_t smem = FWD && a.K > 0 ? sizeof(TopShared<32>) * (kBlock / 32) : 0;
    rows_kernel<DT, FWD, BWD, 32><<<(a.N + 7) / 8, kBlock, smem, s>>>(a);
    return cudaGetLastError();
  }
  // CTAs of a row: while each has over 256 KB (64 KB that wait in shared memory) or CTAs are too few for the SMs, and
  // keeps 8 KB
  const long long most = FWD && BWD ? 65536 : 262144;
  a.cta_bits = 0;
  auto share = [&] { return bytes >> a.cta_bits; };
  while (1 << a.cta_bits < kMostCtas && share() > 16384 && (share() > most || ((long long)a.N << a.cta_bits) < 4 * 152)) ++a.cta_bits;
  const long long kept = share() / 16 + 1;
  a.keep = FWD && BWD && kept * 16 <= 65536 + 16 ? (int)kept : 0;
  // Rows to 40 KB (whose batches the barriers cover), more of them than CTAs of 256 threads fit: a row's chain of latencies wants
  // more rows an SM (4,041 x 4,695 float32 scores 27 us against 35, with ten alternatives 39 against 57; 2,000 x 8,192 bfloat16 in
  // one call 20 against 26; 8,000 x 8,193 float32 78 against 88; 656 x 8,193 scores 12.3 against 14.3, but the gradient
  // alone takes longer: both calls 26.6 against 24.6)
  if constexpr (FWD)
    if (a.cta_bits == 0 && bytes / 16 < kMostBatches * 4 * kNarrow && a.N > 4 * 152) return launch_ctas<DT, FWD, BWD, kNarrow>(a, s);
  return launch_ctas<DT, FWD, BWD, kBlock>(a, s);
}
template <bool FWD, bool BWD> int launch(const RowArgs &a, int dtype, void *stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == kF32   ? launch_rows<kF32, FWD, BWD>(a, s)
                        : dtype == kF16 ? launch_rows<kF16, FWD, BWD>(a, s)
                                        : launch_rows<kBF16, FWD, BWD>(a, s);
  return e == cudaSuccess ? TDT_OK : TDT_ERR_CUDA;
}

int fill_outputs(RowArgs *a, float *logprobs, float *entropy, float *stats, int32_t *top_tokens,
                 float *top_logprobs) {
  if (!logprobs || (a->K > 0 && (!top_tokens || !top_logprobs))) return TDT_ERR_NULL_POINTER;
  if (off4({logprobs, entropy, top_tokens, top_logprobs}) || (uintptr_t)stats % 8) return TDT_ERR_BAD_ALIGNMENT;
  a->logprobs = logprobs;
  a->entropy = entropy;
  a->stats = reinterpret_cast<float2 *>(stats);
  a->top_tokens = top_tokens;
  a->top_logprobs = top_logprobs;
  return TDT_OK;
}

}  // namespace
}  // namespace tdt

extern "C" {

int tdt_token_logprobs_fwd(const void *logits, const int64_t sizes[3], int64_t row_stride, int dtype,
                           const int64_t *tokens, float *logprobs, float *entropy, float *stats,
                           int32_t *top_tokens, float *top_logprobs, void *stream) {
  using namespace tdt;
  RowArgs a = {};
  int rc = check(logits, sizes, &row_stride, false, dtype, tokens, &a);
  if (rc != TDT_OK || a.N == 0) return rc;
  rc = fill_outputs(&a, logprobs, entropy, stats, top_tokens, top_logprobs);
  if (rc != TDT_OK) return rc;
  return launch<true, false>(a, dtype, stream);
}

int tdt_token_logprobs_bwd(const void *logits, const int64_t sizes[3], const int64_t strides[2], int dtype,
                           const int64_t *tokens, const float *entropy, const float *stats,
                           const int32_t *top_tokens, const float *grad_logprobs, const float *grad_entropy,
                           const float *grad_top, void *grad_out, void *stream) {
  using namespace tdt;
  RowArgs a = {};
  int rc = check(logits, sizes, strides, true, dtype, tokens, &a);
  if (rc != TDT_OK || a.N == 0) return rc;
  if (!stats || (grad_entropy && !entropy) || (grad_top && a.K > 0 && !top_tokens)) return TDT_ERR_NULL_POINTER;
  if (off4({entropy, top_tokens, grad_logprobs, grad_entropy, grad_top}) || (uintptr_t)stats % 8)
    return TDT_ERR_BAD_ALIGNMENT;
  rc = check_grad(a, grad_out, strides[1], dtype);
  if (rc != TDT_OK) return rc;
  a.in_entropy = entropy;
  a.in_stats = reinterpret_cast<const float2 *>(stats);
  a.in_top = top_tokens;
  a.ga = grad_logprobs;
  a.gb = grad_entropy;
  a.gc = grad_top;
  a.dx = grad_out;
  a.sdx = strides[1];
  return launch<false, true>(a, dtype, stream);
}

int tdt_token_logprobs_fwd_bwd(const void *logits, const int64_t sizes[3], const int64_t strides[2], int dtype,
                               const int64_t *tokens, const float *grad_logprobs, const float *grad_entropy,
                               float *logprobs, float *entropy, float *stats, int32_t *top_tokens,
                               float *top_logprobs, void *grad_out, void *stream) {
  using namespace tdt;
  RowArgs a = {};
  int rc = check(logits, sizes, strides, true, dtype, tokens, &a);
  if (rc != TDT_OK || a.N == 0) return rc;
  rc = fill_outputs(&a, logprobs, entropy, stats, top_tokens, top_logprobs);
  if (rc != TDT_OK) return rc;
  if (off4({grad_logprobs, grad_entropy})) return TDT_ERR_BAD_ALIGNMENT;
  rc = check_grad(a, grad_out, strides[1], dtype);
  if (rc != TDT_OK) return rc;
  a.ga = grad_logprobs;
  a.gb = grad_entropy;
  a.dx = grad_out;
  a.sdx = strides[1];
  return launch<true, true>(a, dtype, stream);
}

}  // extern "C"
