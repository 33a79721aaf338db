// tdt_tc.cu -- tensor maps for TMA (cuTensorMapEncodeTiled, looked up in the driver at its
// first use, so the library does not link against it).
#include "tdt_tc.cuh"

#include <atomic>
#include <mutex>

namespace tdt {
namespace {

typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encoder() {
  static EncodeTiled fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &found) == cudaSuccess &&
        found == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiled>(p);
  });
  return fn;
}

// An axis of one element has no stride to speak of; one of stride 0 repeats its element.
bool axis_fits(long long n, long long stride, int size) {
  return n <= 1 || stride == 0 || (stride * size % 16 == 0 && stride * size < (1LL << 40));
}
int size_of(int dtype) { return dtype == kF32 ? 4 : 2; }

}  // namespace

cudaError_t prepare_tc_kernel(const void *kernel, size_t smem, int regs) {
  // the registers are the compiled code's: looked up once a kernel
  constexpr int kMost = 64;
  static std::atomic<const void *> checked[kMost];
  int i = 0;
  for (; i < kMost; ++i) {
    const void *c = checked[i].load(std::memory_order_acquire);
    if (c == kernel) break;
    if (c && i + 1 < kMost) continue;
    cudaFuncAttributes a;
    const cudaError_t e = cudaFuncGetAttributes(&a, kernel);
    if (e != cudaSuccess) return e;
    if (a.numRegs != regs) return cudaErrorInvalidConfiguration;
    const void *none = nullptr;
    checked[i].compare_exchange_strong(none, kernel);
    break;
  }
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
}

bool map_fits(int dtype, const void *ptr, long long B, long long L, long long H, int D, long long sb,
              long long sl, long long sh) {
  const int es = size_of(dtype);
  return (uintptr_t)ptr % 16 == 0 && D * es % 16 == 0 && axis_fits(B, sb, es) && axis_fits(H, sh, es) &&
         axis_fits(L, sl, es) && (L <= 1 || sl != 0);
}

bool encode_map(TensorMap *m, const void *ptr, int dtype, long long B, long long L, long long H,
                int D, long long sb, long long sl, long long sh, int box_heads, int box_rows) {
  EncodeTiled fn = encoder();
  if (!fn) return false;
  m->b_mul = sb == 0 || B <= 1 ? 0 : 1;
  m->h_mul = sh == 0 || H <= 1 ? 0 : 1;
  // a head axis of stride 0 cannot be boxed with others
  if (!m->h_mul && box_heads > 1) return false;
  const long long unit = (long long)((D + 7) / 8 * 8);
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)(m->h_mul ? H : 1), (cuuint64_t)L,
                              (cuuint64_t)(m->b_mul ? B : 1)};
  const int es = size_of(dtype);
  const cuuint64_t strides[3] = {(cuuint64_t)(m->h_mul ? sh : unit) * es,
                                 (cuuint64_t)(L > 1 ? sl : unit) * es,
                                 (cuuint64_t)(m->b_mul ? sb : unit) * es};
  const cuuint32_t box[4] = {(cuuint32_t)(128 / es), (cuuint32_t)box_heads, (cuuint32_t)box_rows, 1};
  const cuuint32_t steps[4] = {1, 1, 1, 1};
  return fn(&m->map,
            dtype == kF32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
            : dtype == kBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                             : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
            4,
            const_cast<void *>(ptr), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_planes(TensorMap *m, const unsigned short *planes, long long B, long long L, long long H,
                   int chunks, int box_heads, int box_rows) {
  const int n = chunks * 192;
  return encode_map(m, planes, kBF16, B, L, H, n, H * L * n, n, L * n, box_heads, box_rows);
}

namespace {

struct PlaneArgs {
  PlaneSource t[4];
  long long rows[4];  // B * H * L
  int D, chunks;
};

// A thread has 8 columns of a row: 32 bytes in, 16 bytes out of each plane.  Bound by memory (q, dO, k and v
// of 1201 x 2000, 8 heads of 64: 6 us).
__global__ void __launch_bounds__(256) planes_kernel(const __grid_constant__ PlaneArgs a) {
  const PlaneSource &t = a.t[blockIdx.y];
  const long long x = (long long)blockIdx.x * 256 + threadIdx.x, row = x / (8 * a.chunks);
  const int d0 = (int)(x % (8 * a.chunks)) * 8;
  if (row >= a.rows[blockIdx.y]) return;
  const unsigned l = (unsigned)(row % t.L);
  const long long bh = row / t.L, b = bh / t.H, h = bh % t.H;
  const bool real = !t.lens || l < t.lens[b];
  const float *src = t.src + b * t.sb + l * t.sl + h * t.sh + d0;
  float v[8];
  if (real && d0 + 8 <= a.D && (uintptr_t)src % 16 == 0) {
    const float4 p = __ldg(reinterpret_cast<const float4 *>(src)),
                 q = __ldg(reinterpret_cast<const float4 *>(src) + 1);
    v[0] = p.x; v[1] = p.y; v[2] = p.z; v[3] = p.w;
    v[4] = q.x; v[5] = q.y; v[6] = q.z; v[7] = q.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = real && d0 + i < a.D ? __ldg(src + i) : 0.0f;
  }
  unsigned w[3][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    unsigned p[3];
    split2<kF32>(make_float2(v[2 * i], v[2 * i + 1]), p);
    w[0][i] = p[0];
    w[1][i] = p[1];
    w[2][i] = p[2];
  }
#pragma unroll
  for (int p = 0; p < 3; ++p)
    *reinterpret_cast<uint4 *>(t.dst + ((row * a.chunks + d0 / 64) * 3 + p) * 64 + d0 % 64) =
        make_uint4(w[p][0], w[p][1], w[p][2], w[p][3]);
}

}  // namespace

cudaError_t launch_planes(const PlaneSource *src, int n, long long B, int D, cudaStream_t stream) {
  PlaneArgs a = {};
  long long most = 0;
  for (int i = 0; i < n; ++i) {
    a.t[i] = src[i];
    a.rows[i] = B * src[i].H * src[i].L;
    most = a.rows[i] > most ? a.rows[i] : most;
  }
  a.D = D;
  a.chunks = (D + 63) / 64;
  if (most == 0) return cudaSuccess;
  planes_kernel<<<dim3((unsigned)((most * 8 * a.chunks + 255) / 256), n), 256, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace tdt
