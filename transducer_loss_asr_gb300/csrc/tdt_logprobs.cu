// tdt_logprobs.cu -- log-probabilities of given tokens, entropy, the most probable alternatives, and the gradient
// (include/tdt_decoder.h, tdt_token_logprobs_*).
//
// With m the maximum of a row x, z_i = x_i - m, s = sum e^z_i and t = sum e^z_i z_i:
//   logprob = z_t - ln s,   entropy = ln s - t / s,
//   dx_i = -p_i (a + sum c + b (ln p_i + entropy)) + the given token's and the alternatives' own a and c_j,
//   ln p_i = z_i - ln s.
// An entry of -inf has p = 0; ln p is held above -1e4 in products with p, which is 0 there.
#include <math.h>

#include "../../include/tdt_decoder.h"
#include "tdt_common.cuh"

namespace tdt {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMostTop = 64;
constexpr float kLn2f = 0.69314718055994531f;

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
};

// max that keeps NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

template <typename F> __device__ float block_reduce(float v, float *part, F f) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = part[0];
#pragma unroll
  for (int i = 1; i < kWarps; ++i) v = f(v, part[i]);
  return v;
}

template <int DT, bool FWD, bool BWD>
__global__ void __launch_bounds__(kThreads) rows_kernel(const __grid_constant__ RowArgs a) {
  typedef typename Elem<DT>::T E;
  __shared__ float part[kWarps];
  __shared__ int best_at[kWarps];
  const unsigned n = blockIdx.x;
  const E *x = static_cast<const E *>(a.x) + n * a.sx;
  const long long token = a.tokens[n];
  const bool real = token >= 0 && token < a.V;
  auto at = [&](int i) { return Elem<DT>::to_float(x[i]); };
  const int K = a.K;
  float m = 0.0f, ln_s = 0.0f, ent = 0.0f;
  if (FWD) {
    if (!real) {
      const float none = token < 0 ? 0.0f : NAN;
      if (threadIdx.x == 0) {
        a.logprobs[n] = none;
        if (a.entropy) a.entropy[n] = none;
        if (a.stats) a.stats[n] = make_float2(none, none);
      }
      for (int k = threadIdx.x; k < K; k += kThreads) {
        a.top_tokens[n * (long long)K + k] = -1;
        a.top_logprobs[n * (long long)K + k] = token < 0 ? -INFINITY : NAN;
      }
    } else {
      m = -INFINITY;
      for (int i = threadIdx.x; i < a.V; i += kThreads) m = max_nan(m, at(i));
      m = block_reduce(m, part, max_nan);
      float s = 0.0f, t = 0.0f;
      for (int i = threadIdx.x; i < a.V; i += kThreads) {
        const float z = at(i) - m, w = fast_exp2(z * kLog2e);
        s += w;
        t += w * max_nan(z, -1e4f);
      }
      auto add = [](float p, float q) { return p + q; };
      s = block_reduce(s, part, add);
      t = block_reduce(t, part, add);
      ln_s = log2f(s) * kLn2f;
      ent = ln_s - t / s;
      if (threadIdx.x == 0) {
        a.logprobs[n] = at((int)token) - m - ln_s;
        if (a.entropy) a.entropy[n] = ent;
        if (a.stats) a.stats[n] = make_float2(m, ln_s);
      }
      float last = INFINITY;
      int last_at = -1;
      const bool lost = s != s;
      for (int k = 0; k < K; ++k) {
        float v = -INFINITY;
        int v_at = a.V;
        for (int i = threadIdx.x; i < a.V && !lost; i += kThreads) {
          const float y = at(i);
          const bool after = y < last || (y == last && i > last_at);
          if (after && (y > v || v_at == a.V)) {
            v = y;
            v_at = i;
          }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const float v2 = __shfl_xor_sync(0xffffffffu, v, o);
          const int at2 = __shfl_xor_sync(0xffffffffu, v_at, o);
          if (at2 < a.V && (v_at == a.V || v2 > v || (v2 == v && at2 < v_at))) {
            v = v2;
            v_at = at2;
          }
        }
        __syncthreads();
        if ((threadIdx.x & 31) == 0) {
          part[threadIdx.x >> 5] = v;
          best_at[threadIdx.x >> 5] = v_at;
        }
        __syncthreads();
        v_at = a.V;
        for (int w = 0; w < kWarps; ++w)
          if (best_at[w] < a.V && (v_at == a.V || part[w] > v || (part[w] == v && best_at[w] < v_at))) {
            v = part[w];
            v_at = best_at[w];
          }
        last = v;
        last_at = v_at;
        if (threadIdx.x == 0) {
          a.top_tokens[n * (long long)K + k] = lost ? -1 : v_at;
          a.top_logprobs[n * (long long)K + k] = lost ? NAN : v - m - ln_s;
        }
      }
    }
  }
  if (BWD) {
    E *dx = static_cast<E *>(a.dx) + n * a.sdx;
    if (!real) {
      for (int i = threadIdx.x; i < a.V; i += kThreads) dx[i] = Elem<DT>::from_float(0.0f);
      return;
    }
    __shared__ int own_at[kMostTop + 1];
    __shared__ float own_add[kMostTop + 1], own_x[kMostTop + 1];
    const float ga = a.ga ? a.ga[n] : 0.0f, gb = a.gb ? a.gb[n] : 0.0f;
    const int kept = a.gc ? K : 0;
    if (!FWD) {
      const float2 st = a.in_stats[n];
      m = st.x;
      ln_s = st.y;
      ent = a.gb ? a.in_entropy[n] : 0.0f;
    }
    for (int j = threadIdx.x; j <= kept; j += kThreads) {
      const int i = j == kept ? (int)token : a.in_top[n * (long long)K + j];
      const bool in = i >= 0 && i < a.V;
      own_at[j] = in ? i : -1;
      own_add[j] = j == kept ? ga : a.gc[n * (long long)K + j];
      own_x[j] = in ? at(i) : 0.0f;
    }
    __syncthreads();
    float all = 0.0f;
    for (int j = 0; j <= kept; ++j) all += own_add[j];
    auto slope = [&](float y) {
      const float z = y - m, lp = z - ln_s;
      const float p = fast_exp2(lp * kLog2e);
      return -p * fmaf(gb, max_nan(lp, -1e4f) + ent, all);
    };
    for (int i = threadIdx.x; i < a.V; i += kThreads) dx[i] = Elem<DT>::from_float(slope(at(i)));
    __syncthreads();
    // tokens with a part of their own: each is written again by the first that names it
    for (int j = threadIdx.x; j <= kept; j += kThreads) {
      const int i = own_at[j];
      bool first = i >= 0;
      float add = 0.0f;
      for (int q = 0; q <= kept; ++q)
        if (own_at[q] == i) {
          if (q < j) first = false;
          add += own_add[q];
        }
      if (first) dx[i] = Elem<DT>::from_float(slope(own_x[j]) + add);
    }
  }
}

bool known(int dtype) { return dtype == TDT_DTYPE_F32 || dtype == TDT_DTYPE_F16 || dtype == TDT_DTYPE_BF16; }

int check(const void *logits, const int64_t sizes[3], const int64_t *strides, bool grad, int dtype,
          const int64_t *tokens, RowArgs *a) {
  if (!sizes || !strides) return TDT_ERR_NULL_POINTER;
  if (!known(dtype)) return TDT_ERR_BAD_DTYPE;
  const int64_t N = sizes[0], V = sizes[1], K = sizes[2];
  if (N < 0 || N >= (int64_t)1 << 31 || V < 1 || V > 1 << 24) return TDT_ERR_BAD_SIZES;
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

template <bool FWD, bool BWD> int launch(const RowArgs &a, int dtype, void *stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == kF32)
    rows_kernel<kF32, FWD, BWD><<<a.N, kThreads, 0, s>>>(a);
  else if (dtype == kF16)
    rows_kernel<kF16, FWD, BWD><<<a.N, kThreads, 0, s>>>(a);
  else
    rows_kernel<kBF16, FWD, BWD><<<a.N, kThreads, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? TDT_OK : TDT_ERR_CUDA;
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
