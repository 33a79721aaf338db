// tdt_sample.cu -- draws a token of each row of logits (include/tdt_decoder.h,
// tdt_sample): temperature, top-k, top-p, min-p, then the inverse of the
// running sum at a given uniform number.
//
// Mathematics.  Weights are whole numbers, w = rint(2^31 * 2^z) with
// z = (x - X) * (log2(e) / T) and X the row's maximum, so sums of weights are
// exact whatever their order, and every filter keeps a prefix of the order
// (x falling, index rising): the kept set is "order key above a cut, and the
// first c tokens equal to it".  The cut is found by radix selection: the keys
// in 8-bit digits from the top, each digit's histogram of counts and weights
// scanned by one warp for the digit at which the count reaches top_k, or the
// weight reaches the share top_p of what top_k leaves.
//
// One CTA a row.  Every warp owns a contiguous range of the row, so sums by warp are running sums of the
// vocabulary's order.
//   pass 1  the maximum X; rows of up to 16,384 tokens stay in shared memory, as float32;
//   pass 2  the sum of all weights, if the settings need it, and the tokens with z >= -12 (overflowing:
//           -6, -3) into a list in shared memory, each warp its own part, in index order.
// The cut usually lies among the listed tokens -- top_k of them exist, or their weight reaches top_p's
// share of all, or min_p is above any unlisted weight -- and then selection and draw read the list only.
// Otherwise they read the row again (from L2, where it does not stay).
// Pass 2 is what bounds wide rows: its weights are below 2^-9 of the largest, apart from the listed ones,
// and adding 1.5 * 2^-8 to such a weight leaves rint(2^31 w) in the low bits of the sum: no conversion, and
// 32-bit sums.  Two tokens an instruction where the hardware has it.
#include "../../include/tdt_decoder.h"
#include "tdt_rowio.cuh"
#include "tdt_tc.cuh"

namespace tdt {
namespace {

typedef unsigned long long u64;

constexpr int kListTokens = 4096;      // entries of the list, 8 bytes each
constexpr int kResident = 16384;       // tokens of a row that stays in shared memory
constexpr int kListZ = 12;             // z >= -kListZ goes into the list; if that overflows, half of it, ...
constexpr int kListTries = 3;
constexpr float kZeroZ = 33.0f;        // z < -32 weighs 0

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

// Order of the floats as unsigned numbers; -0 counts as 0, NaN sorts below everything.
__device__ __forceinline__ unsigned order_key(float x) {
  const unsigned b = __float_as_uint(x + 0.0f);
  if (x != x) return 0;
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(unsigned k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}

struct Weigher {
  float X, per;   // row maximum, log2(e) / T
  bool infinite;  // X = +inf: only the +inf entries weigh anything
  // rint(2^31 2^z); the two roundings of z are part of the definition, so no fused multiply
  __device__ __forceinline__ unsigned operator()(float x) const {
    if (infinite) return x == X ? 0x80000000u : 0u;
    const float z = fmaxf(__fmul_rn(__fsub_rn(x, X), per), -64.0f);  // NaN, -inf: weight 0
    return __float2uint_rn(fast_exp2(z) * 2147483648.0f);
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

// What a warp's range holds of the kept set: weight above the cut, tokens equal to it.
struct Held {
  u64 mass;
  unsigned ties;
};

template <int NW> struct Shared {
  float xs[kListTokens];
  int ids[kListTokens];
  // of a digit: tokens, and their weight in three parts (over 2^48 + hi 2^16 + lo)
  unsigned cnt[256], lo[256], hi[256], over[256];
  Held held[NW];
  int listed[NW];
  float red[NW];
  // one thread's findings for all
  unsigned digit;
  u64 above_cnt, above_mass, target;
  int winner, token;
  unsigned ties_left;
  __align__(16) float row[4];  // the row itself, if it is resident
};

// The prefix that stays: keys above `key`, and the first `ties` tokens with that key.
struct Cut {
  unsigned key;
  unsigned ties;
  u64 mass;  // its weight
};

template <int DT, int NW, bool RESIDENT> struct Sampler {
  typedef typename Elem<DT>::T E;
  static constexpr int VEC = Vec<DT>::N;
  static constexpr int CAP = kListTokens / NW;  // list entries of a warp

  Shared<NW> &s;
  const E *row;
  int V, warp, lane, chunk, head;
  Weigher w;
  bool listed;  // the tokens read below are the list's

  __device__ Sampler(Shared<NW> &sh, const E *r, int v) : s(sh), row(r), V(v), listed(false) {
    warp = threadIdx.x >> 5;
    lane = threadIdx.x & 31;
    // Vectors start at multiples of VEC counted from the 16-byte boundary below the row
    head = (int)(((uintptr_t)row % 16) / sizeof(E));
    const int vectors = (V + head + VEC - 1) / VEC;
    chunk = (vectors + NW - 1) / NW * VEC;
  }

  // f(index, x) for the warp's range, VEC consecutive tokens a lane; 32 * VEC consecutive ones a step.
  // Every lane takes every step; tokens outside the row and NaN come as -inf.  `from_memory`: not from
  // the resident copy.  Steps come in pairs, so that two loads are in flight.
  template <typename F> __device__ __forceinline__ void each_vector(F f, bool from_memory = false) const {
    const int end = min(chunk * (warp + 1), V + head);
    const int p0 = chunk * warp + lane * VEC, steps = (end - chunk * warp + 32 * VEC - 1) / (32 * VEC);
    if (RESIDENT && !from_memory) {
      for (int t = 0; t < steps; ++t) {
        const int p = p0 + t * 32 * VEC;
        float x[VEC];
#pragma unroll
        for (int j = 0; j < VEC; j += 4) {
          const float4 v = p < end ? *reinterpret_cast<const float4 *>(s.row + p + j)
                                   : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
          x[j] = v.x;
          x[j + 1] = v.y;
          x[j + 2] = v.z;
          x[j + 3] = v.w;
        }
        f(p - head, x);
      }
      return;
    }
    constexpr int U = 4;
    for (int t = 0; t < steps; t += U) {
      uint4 raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int p = p0 + (t + u) * 32 * VEC, i = p - head;
        if (i >= 0 && i + VEC <= V && p < end) {
          raw[u] = __ldg(reinterpret_cast<const uint4 *>(row + i));
        } else {
          E *e = reinterpret_cast<E *>(&raw[u]);
#pragma unroll
          for (int j = 0; j < VEC; ++j)
            e[j] = (i + j >= 0 && i + j < V && p < end) ? row[i + j] : Elem<DT>::from_float(-INFINITY);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (t + u >= steps) break;
        float x[VEC];
        unpack(raw[u], x);
        f(p0 + (t + u) * 32 * VEC - head, x);
      }
    }
  }
  // VEC tokens as float32, NaN as -inf
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
  // f(x) for every token of this thread's share of the warp's tokens: the list's or the row's.
  template <typename F> __device__ __forceinline__ void each(F f) const {
    if (listed) {
      for (int i = lane; i < s.listed[warp]; i += 32) f(s.xs[warp * CAP + i]);
    } else {
      each_vector([&](int, const float *x) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) f(x[j]);
      });
    }
  }
  // Token i of the row, NaN as -inf.
  __device__ __forceinline__ float token(int i) const {
    return RESIDENT ? s.row[i + head] : fmaxf(Elem<DT>::load(row + i), -INFINITY);
  }

  __device__ float maximum() {
    float m = -INFINITY;
    each_vector(
        [&](int i, const float *x) {
#pragma unroll
          for (int j = 0; j < VEC; ++j) m = fmaxf(m, x[j]);
          // the resident copy; a thread reads back what it wrote, others only after a barrier
          if (RESIDENT && i < V && i + head < chunk * (warp + 1))
#pragma unroll
            for (int j = 0; j < VEC; j += 4)
              *reinterpret_cast<float4 *>(s.row + i + head + j) = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
        },
        true);
    m = warp_max(m);
    if (lane == 0) s.red[warp] = m;
    __syncthreads();
    m = warp_max(lane < NW ? s.red[lane] : -INFINITY);
    __syncthreads();
    return m;
  }

  // Pass 2.  MASS: the sum of the weights, by warp into held[].mass: of all tokens, or with LIST of those
  // below `near`.  LIST: the tokens from `near` up into the list.  Returns the number of listed tokens, -1
  // if they do not fit.
  template <bool MASS, bool LIST> __device__ int weigh(float near) {
    u64 mass = 0;
    int n = 0;
    bool fits = true;
    const float2 x2 = make_float2(-w.X, -w.X), per2 = make_float2(w.per, w.per);
    // z < -9 for tokens below `near`: reading a weight off the sum is exact (see the head of the file)
    const bool small = !w.infinite && (near - w.X) * w.per < -9.5f;
    constexpr float kMagic = 1.5f / 256.0f;
    each_vector([&](int i, const float *x) {
      if (MASS && small) {
        unsigned sum = 0;
#pragma unroll
        for (int j = 0; j < VEC; j += 2) {
          const float2 z = mul2(add2(make_float2(x[j], x[j + 1]), x2), per2);
          const float2 m = add2(make_float2(fast_exp2(z.x), fast_exp2(z.y)), make_float2(kMagic, kMagic));
          if (!(x[j] >= near)) sum += __float_as_uint(m.x) - __float_as_uint(kMagic);
          if (!(x[j + 1] >= near)) sum += __float_as_uint(m.y) - __float_as_uint(kMagic);
        }
        mass += sum;
        if (!LIST) {
#pragma unroll
          for (int j = 0; j < VEC; ++j)
            if (x[j] >= near) mass += w(x[j]);
        }
      } else if (MASS) {
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          if (!LIST || !(x[j] >= near)) mass += w(x[j]);
      }
      if (LIST) {
        float top = x[0];
#pragma unroll
        for (int j = 1; j < VEC; ++j) top = fmaxf(top, x[j]);
        if (!__any_sync(0xffffffffu, top >= near)) return;
        unsigned in = 0;
#pragma unroll
        for (int j = 0; j < VEC; ++j) in |= (x[j] >= near ? 1u : 0u) << j;
        // place of this lane's first token: the tokens of lower lanes come before it
        int before = __popc(in);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int t = __shfl_up_sync(0xffffffffu, before, o);
          if (lane >= o) before += t;
        }
        const int all = __shfl_sync(0xffffffffu, before, 31);
        int at = n + before - __popc(in);
        if (n + all > CAP) fits = false;
        if (fits) {
#pragma unroll
          for (int j = 0; j < VEC; ++j)
            if (in >> j & 1) {
              s.xs[warp * CAP + at] = x[j];
              s.ids[warp * CAP + at] = i + j;
              ++at;
            }
          n += all;
        }
      }
    });
    if (MASS) mass = warp_sum64(mass);
    if (lane == 0) {
      if (MASS) {
        s.held[warp].mass = mass;
        s.held[warp].ties = 0;
      }
      s.listed[warp] = n;
    }
    const int bad = __syncthreads_or(!fits);
    if (bad) return -1;
    int total = lane < NW ? s.listed[lane] : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    return total;
  }

  // Sum over all threads, known to all; a barrier before and after its use of held[].
  __device__ u64 total_of(u64 v) {
    v = warp_sum64(v);
    __syncthreads();
    if (lane == 0) s.held[warp].mass = v;
    __syncthreads();
    return total_mass();
  }

  __device__ u64 total_mass() const {
    return warp_sum64(lane < NW ? s.held[lane].mass : 0ull);
  }

  __device__ __forceinline__ u64 mass_of(int digit) const {
    return ((u64)s.over[digit] << 48) + ((u64)s.hi[digit] << 16) + s.lo[digit];
  }

  // Radix selection over the keys in [from, top]: the token at which, in falling order, the
  // count (by_count) or the weight reaches `target` >= 1.  The caller knows that it is reached.
  __device__ Cut select(bool by_count, u64 target, unsigned from, unsigned top) {
    unsigned lo = from;                         // keys [lo, lo + 2^bits) are still in question
    int bits = 32 - __clz(top - from);          // 0: only one key
    u64 above_cnt = 0, above_mass = 0;          // of the keys above that range
    while (bits > 0) {
      const int shift = max(0, bits - 8);
      const unsigned digits = 1u << (bits - shift);  // at most 256
      for (int i = threadIdx.x; i < 256; i += NW * 32) {
        s.cnt[i] = 0;
        s.lo[i] = 0;
        s.hi[i] = 0;
        s.over[i] = 0;
      }
      __syncthreads();
      each([&](float x) {
        const unsigned k = order_key(x);
        if (k >= lo && ((k - lo) >> shift) < digits) {
          // a weight goes in as two halves of 16 bits, with native 32-bit adds; what a part overflows
          // is carried into the next one
          const unsigned d = (k - lo) >> shift, v = w(x), half = v & 0xffffu;
          atomicAdd(&s.cnt[d], 1u);
          const unsigned old = atomicAdd(&s.lo[d], half);
          const unsigned up = (v >> 16) + (old + half < old ? 0x10000u : 0u);
          const unsigned old_hi = atomicAdd(&s.hi[d], up);
          if (old_hi + up < old_hi) atomicAdd(&s.over[d], 1u);
        }
      });
      __syncthreads();
      if (warp == 0) {
        // lane 0 has the 8 highest digits
        u64 c = 0, m = 0;
        for (int i = 0; i < 8; ++i) {
          c += s.cnt[255 - lane * 8 - i];
          m += mass_of(255 - lane * 8 - i);
        }
        u64 bc = above_cnt + warp_before64(c), bm = above_mass + warp_before64(m);
        const u64 at = by_count ? bc : bm, step = by_count ? c : m;
        if (at < target && at + step >= target) {
          int d = 255 - lane * 8;
          for (; d > 255 - lane * 8 - 7; --d) {
            if ((by_count ? bc + s.cnt[d] : bm + mass_of(d)) >= target) break;
            bc += s.cnt[d];
            bm += mass_of(d);
          }
          s.digit = d;
          s.above_cnt = bc;
          s.above_mass = bm;
        }
      }
      __syncthreads();
      lo += s.digit << shift;
      above_cnt = s.above_cnt;
      above_mass = s.above_mass;
      bits = shift;
    }
    __syncthreads();
    Cut c;
    c.key = lo;
    const u64 weight = w(key_value(lo));
    if (by_count)
      c.ties = (unsigned)(target - above_cnt);
    else
      c.ties = (unsigned)((target - above_mass + weight - 1) / weight);  // weight > 0: it moved the sum
    c.mass = above_mass + c.ties * weight;
    return c;
  }

  __device__ __forceinline__ bool above(float x, const Cut &c, unsigned m) const {
    return order_key(x) > c.key && w(x) >= m;
  }

  // Reduces each warp's Held over its lanes; all threads then know the warp that the running sum
  // passes `target` in, what is left of the target and of the ties before it.
  __device__ void pick_warp(u64 mass, unsigned ties, unsigned tie_weight, u64 *target,
                            unsigned *ties_left) {
    mass = warp_sum64(mass);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ties += __shfl_xor_sync(0xffffffffu, ties, o);
    if (lane == 0) {
      s.held[warp].mass = mass;
      s.held[warp].ties = ties;
    }
    __syncthreads();
    find_warp(tie_weight, target, ties_left);
  }
  __device__ void find_warp(unsigned tie_weight, u64 *target, unsigned *ties_left) {
    if (threadIdx.x == 0) {
      u64 run = 0;
      unsigned left = *ties_left;
      int i = 0;
      for (; i < NW - 1; ++i) {
        const unsigned t = min(left, s.held[i].ties);
        const u64 here = s.held[i].mass + (u64)t * tie_weight;
        if (run + here > *target) break;
        run += here;
        left -= t;
      }
      s.winner = i;
      s.target = *target - run;
      s.ties_left = left;
    }
    __syncthreads();
    *target = s.target;
    *ties_left = s.ties_left;
  }

  // 32 tokens, one a lane, in order: the first at which the running sum passes the target.
  // Returns the lane, or 32 with the target and the ties moved on.
  __device__ int step(float x, bool valid, const Cut &c, unsigned m, unsigned tie_weight,
                      u64 *target, unsigned *ties_left) const {
    const bool tie = valid && order_key(x) == c.key;
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

  // The drawn token, valid in every thread.  `target` < the kept weight.
  __device__ int draw(const Cut &c, unsigned m, u64 target, bool sums_ready) {
    const unsigned wc = w(key_value(c.key)), tie_weight = wc >= m ? wc : 0;
    unsigned left = c.ties;
    if (threadIdx.x == 0) s.token = -1;
    if (sums_ready) {
      __syncthreads();
      find_warp(tie_weight, &target, &left);
    } else {
      u64 mass = 0;
      unsigned ties = 0;
      each([&](float x) {
        const unsigned k = order_key(x);
        if (k > c.key) {
          const unsigned v = w(x);
          if (v >= m) mass += v;
        }
        ties += k == c.key ? 1u : 0u;
      });
      pick_warp(mass, ties, tie_weight, &target, &left);
    }
    const int winner = s.winner;
    if (listed) {
      if (warp == winner) {
        const int n = s.listed[warp];
        for (int i0 = 0; i0 < n; i0 += 32) {
          const int i = i0 + lane;
          const bool valid = i < n;
          const float x = valid ? s.xs[warp * CAP + i] : -INFINITY;
          const int hit = step(x, valid, c, m, tie_weight, &target, &left);
          if (hit < 32) {
            if (lane == hit) s.token = s.ids[warp * CAP + i];
            break;
          }
        }
      }
      __syncthreads();
      return s.token;
    }
    // the row: the winner's range is split over the warps again, until it is short
    int a = max(0, chunk * winner - head), b = min(chunk * (winner + 1) - head, V);
    while (b - a > 128) {
      __syncthreads();
      const int piece = (b - a + NW - 1) / NW, p0 = a + piece * warp, p1 = min(b, p0 + piece);
      u64 mass = 0;
      unsigned ties = 0;
      for (int i = p0 + lane; i < p1; i += 32) {
        const float x = token(i);
        if (above(x, c, m)) mass += w(x);
        ties += order_key(x) == c.key ? 1u : 0u;
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
__global__ void __launch_bounds__(NW * 32) sample_kernel(SampleArgs a) {
  typedef typename Elem<DT>::T E;
  extern __shared__ __align__(16) unsigned char raw[];
  Shared<NW> &s = *reinterpret_cast<Shared<NW> *>(raw);
  const long long n = blockIdx.x;
  const E *row = static_cast<const E *>(a.logits) + n * a.row_stride;
  const float T = a.temperatures ? a.temperatures[n] : a.temperature;
  const float p = a.top_ps ? a.top_ps[n] : a.top_p;
  const float mp = a.min_ps ? a.min_ps[n] : a.min_p;
  int k = a.top_ks ? a.top_ks[n] : a.top_k;
  Sampler<DT, NW, RESIDENT> r(s, row, a.V);
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
  const unsigned top = order_key(X);
  // the value at -z below the maximum, as a key's value
  auto below = [&](float z) {
    return T == 0.0f || r.w.infinite ? X : key_value(order_key(X - z / r.w.per));
  };
  Cut cut;
  u64 kept;
  bool sums_ready = false;
  if (!filters) {
    r.template weigh<true, false>(below((float)kListZ));
    cut.key = 0;
    cut.ties = 0;
    kept = r.total_mass();
    sums_ready = true;  // held[] is the sums by warp of every token
  } else {
    int listed = -1, z = kListZ;
    u64 all = 0;
    float near = 0.0f;
    for (int i = 0; i < kListTries && listed < 0; ++i) {
      z = kListZ >> i;
      near = below((float)z);
      listed = need_all && i == 0 ? r.template weigh<true, true>(near) : r.template weigh<false, true>(near);
      if (need_all && i == 0) {
        all = r.total_mass();  // of the tokens below the first `near`
        if (listed < 0) {      // the rest was not kept: sum it from the row
          u64 mass = 0;
          r.each([&](float x) { mass += x >= near ? (u64)r.w(x) : 0ull; });
          all += r.total_of(mass);
        }
      }
    }
    u64 listed_mass = 0;
    if (listed >= 0) {
      u64 mass = 0;
      r.listed = true;
      r.each([&](float x) { mass += r.w(x); });
      listed_mass = r.total_of(mass);
      if (need_all && z == kListZ) all += listed_mass;
    }
    // does the cut lie among the listed tokens?
    const unsigned low = (0x80000000u >> z) + (0x80000000u >> (z + 8));  // above any unlisted weight
    const bool enough = listed > 0 && (k > 0   ? listed >= k || (!by_p && m >= low)
                                       : by_p ? listed_mass >= share(all, p24)
                                              : m >= low);
    r.listed = enough;
    const unsigned from = order_key(enough ? near : below(kZeroZ));
    // top-k, unless fewer tokens than that weigh anything
    cut.key = from;  // everything from `from` up
    cut.ties = 0xffffffffu;
    bool cut_by_k = false;
    if (k > 0) {
      u64 have = (u64)max(listed, 0);
      if (!enough) {
        u64 c = 0;
        r.each([&](float x) { c += order_key(x) >= from ? 1u : 0u; });
        have = r.total_of(c);
      }
      if (have >= (u64)k) {
        cut = r.select(true, (u64)k, from, top);
        cut_by_k = true;
      }
    }
    if (!cut_by_k) {  // the weight of everything from `from` up
      if (enough) {
        cut.mass = listed_mass;
      } else if (need_all) {
        cut.mass = all;
      } else {
        u64 mass = 0;
        r.each([&](float x) { mass += r.w(x); });
        cut.mass = r.total_of(mass);
      }
    }
    if (by_p) {
      const u64 need = share(need_all ? all : cut.mass, p24);
      cut = r.select(false, need > 0 ? need : 1, from, top);
    }
    kept = cut.mass;
    if (m > 0) {  // the weight that min-p leaves
      u64 mass = 0;
      unsigned ties = 0;
      r.each([&](float x) {
        const unsigned key = order_key(x);
        if (key > cut.key) {
          const unsigned v = r.w(x);
          if (v >= m) mass += v;
        }
        ties += key == cut.key ? 1u : 0u;
      });
      mass = warp_sum64(mass);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ties += __shfl_xor_sync(0xffffffffu, ties, o);
      __syncthreads();
      if (r.lane == 0) {
        s.held[r.warp].mass = mass;
        s.held[r.warp].ties = ties;
      }
      __syncthreads();
      const unsigned wc = r.w(key_value(cut.key));
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
  const size_t smem = sizeof(Shared<NW>) + (RESIDENT ? (size_t)(a.V + 16) * 4 : 0);
  const cudaError_t e = cudaFuncSetAttribute(sample_kernel<DT, NW, RESIDENT>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  sample_kernel<DT, NW, RESIDENT><<<(unsigned)N, NW * 32, smem, s>>>(a);
  return cudaGetLastError();
}
template <int DT> cudaError_t launch(const SampleArgs &a, long long N, cudaStream_t s) {
  if (a.V <= 2048) return launch<DT, 4, true>(a, N, s);
  if (a.V <= kResident)
    return N > 2 * 152 ? launch<DT, 8, true>(a, N, s) : launch<DT, 16, true>(a, N, s);
  return N > 2 * 152 ? launch<DT, 8, false>(a, N, s) : launch<DT, 32, false>(a, N, s);
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
