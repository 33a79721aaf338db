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
bool axis_fits(long long n, long long stride) {
  return n <= 1 || stride == 0 || (stride % 8 == 0 && stride * 2 < (1LL << 40));
}

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

bool map_fits(const void *ptr, long long B, long long L, long long H, int D, long long sb,
              long long sl, long long sh) {
  return (uintptr_t)ptr % 16 == 0 && D % 8 == 0 && axis_fits(B, sb) && axis_fits(H, sh) &&
         axis_fits(L, sl) && (L <= 1 || sl != 0);
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
  const cuuint64_t strides[3] = {(cuuint64_t)(m->h_mul ? sh : unit) * 2,
                                 (cuuint64_t)(L > 1 ? sl : unit) * 2,
                                 (cuuint64_t)(m->b_mul ? sb : unit) * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows, 1};
  const cuuint32_t steps[4] = {1, 1, 1, 1};
  return fn(&m->map,
            dtype == kBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
            const_cast<void *>(ptr), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace tdt
