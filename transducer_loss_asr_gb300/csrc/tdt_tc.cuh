// tdt_tc.cuh -- tensor-core building blocks of the attention kernels (PTX ISA:
// tcgen05, cp.async.bulk.tensor, mbarrier): tensor maps, bounded waits, matrix
// descriptors, TMEM allocation and access.
//
// Tiles in shared memory are [rows][64 elements of 16 bits], 128 bytes a row with the
// 128-byte swizzle that TMA writes; a tile wider than 64 is several such chunks one after
// another.  The same bytes serve as an operand whose contraction runs along the row (K-major:
// q and k of q.k) or across the rows (MN-major: v of p.v), by the descriptor.
#pragma once

#include <cuda.h>

#include "tdt_async.cuh"

namespace tdt {

// ---- waits -------------------------------------------------------------------
// Every wait gives up after kWaitLimitCycles, or at once when another one of the CTA has, and
// then the CTA's outputs are NaN.
struct Waiter {
  int *gave_up;  // shared
  __device__ __forceinline__ bool operator()(unsigned long long *bar, unsigned parity) const {
    if (try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    do {
      if (try_wait(bar, parity)) return true;
      if (*reinterpret_cast<volatile int *>(gave_up)) return false;
    } while (clock64() - t0 < kWaitLimitCycles);
    *reinterpret_cast<volatile int *>(gave_up) = 1;
    return false;
  }
  // After giving up: waits for work in flight, for a hundredth of the limit at most.
  static __device__ __forceinline__ void drain(unsigned long long *bar, unsigned parity) {
    const long long end = clock64() + kWaitLimitCycles / 100;
    while (!try_wait(bar, parity) && clock64() < end) {
    }
  }
  static __device__ __forceinline__ bool try_wait(unsigned long long *bar, unsigned parity) {
    unsigned ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
  }
};
__device__ __forceinline__ void mbar_arrive(unsigned long long *bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// Writes to shared memory by this thread become visible to TMA and the tensor cores.
__device__ __forceinline__ void fence_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Moves registers between the warpgroups of a CTA.  What is taken may not exceed what the launch
// gave the CTA (registers at launch x threads): prepare_tc_kernel checks the launch's count.
template <int N> __device__ __forceinline__ void warpgroup_take_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N> __device__ __forceinline__ void warpgroup_give_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// ---- float32 as planes -----------------------------------------------------------
// The tensor cores multiply 16-bit numbers.  A float32 operand becomes three bfloat16 planes, x = x0 + x1 +
// x2 to 24 bits and more (each rounds what the ones before leave), and a product the six products of planes
// whose orders add up to 2 at the most, small ones first; what is left out is below 2^-25 of |x||y|.
template <int DT> constexpr int kPlanes = DT == kF32 ? 3 : 1;
template <int DT> constexpr int kPlanePairs = DT == kF32 ? 6 : 1;
template <int DT> __device__ __forceinline__ constexpr int plane_a(int i) {
  return DT != kF32 ? 0 : i == 0 ? 2 : i == 2 || i == 3 ? 1 : 0;  // 2 0 1 1 0 0
}
template <int DT> __device__ __forceinline__ constexpr int plane_b(int i) {
  return DT != kF32 ? 0 : i == 1 ? 2 : i == 2 || i == 4 ? 1 : 0;  // 0 2 1 0 1 0
}

// ---- TMA ----------------------------------------------------------------------
__device__ __forceinline__ void tma_load_4d(const CUtensorMap *map, void *dst,
                                            unsigned long long *bar, int x, int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}
// Stores a tile; elements past the tensor's ends are not written.  The thread that issues commits and
// waits until the tile has been read before its memory is used again or the CTA ends.
__device__ __forceinline__ void tma_store_4d(const CUtensorMap *map, const void *src, int x, int y,
                                             int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(
          map),
      "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}
__device__ __forceinline__ void tma_store_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void tma_store_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}
template <int THREADS> __device__ __forceinline__ void named_barrier(int id) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(THREADS) : "memory");
}

// ---- TMEM ---------------------------------------------------------------------
template <int COLS> __device__ __forceinline__ void tmem_alloc(unsigned *base) {  // one warp
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_u32(base)),
               "n"(COLS)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
template <int COLS> __device__ __forceinline__ void tmem_free(unsigned base) {  // the same warp
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "n"(COLS));
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// 32 columns of this thread's lane (32 x 32-bit).  Registers are valid after tmem_wait_ld.
__device__ __forceinline__ void tmem_ld32(unsigned addr, unsigned (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(unsigned addr, const unsigned (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(
          r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31]), "r"(addr)
      : "memory");
}

// One lane of a converged warp, the same at every call.  The compiler knows that a single lane is
// active behind it, and keeps the operands of the products issued there in uniform registers: a
// plain lane == 0 test was measured to cost about 100 cycles a product to issue, more than the 64
// it takes to run.
__device__ __forceinline__ bool elect_one() {
  unsigned p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// 16 columns.
__device__ __forceinline__ void tmem_st16(unsigned addr, const unsigned *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
      : "memory");
}

// ---- matrix products ---------------------------------------------------------------
// Shared-memory operand descriptors: start address, leading and stride offsets in 16-byte
// units, version 1, 128-byte swizzle.
constexpr unsigned long long kDescBase = (1ull << 46) | (2ull << 61);
// Contraction along the row: groups of 8 rows are 1,024 bytes apart.
__device__ __forceinline__ unsigned long long desc_k_major(unsigned addr) {
  return kDescBase | (unsigned long long)((addr >> 4) & 0x3fff) | (1ull << 16) | (64ull << 32);
}
// Contraction across the rows: groups of 8 rows 1,024 bytes apart, chunks of 64 columns
// `chunk_bytes` apart.
__device__ __forceinline__ unsigned long long desc_mn_major(unsigned addr, unsigned chunk_bytes) {
  return kDescBase | (unsigned long long)((addr >> 4) & 0x3fff) |
         ((unsigned long long)(chunk_bytes >> 4) << 16) | (64ull << 32);
}
// Instruction descriptor of kind::f16 with float32 accumulators, M = 128.
template <int DT>
__device__ __forceinline__ constexpr unsigned mma_desc(int N, bool b_mn_major, bool a_mn_major = false) {
  return (1u << 4) | ((DT != kF16 ? 1u : 0u) << 7) | ((DT != kF16 ? 1u : 0u) << 10) |
         ((a_mn_major ? 1u : 0u) << 15) | ((b_mn_major ? 1u : 0u) << 16) | ((unsigned)(N >> 3) << 17) | ((128u >> 4) << 24);
}
// d (+)= a b, both operands in shared memory.  One thread issues; K = 16.
__device__ __forceinline__ void mma_ss(unsigned d, unsigned long long a, unsigned long long b,
                                       unsigned idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((unsigned)accumulate)
      : "memory");
}
// The same with a in TMEM (lane = row, two 16-bit elements a column).
__device__ __forceinline__ void mma_ts(unsigned d, unsigned a, unsigned long long b,
                                       unsigned idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((unsigned)accumulate)
      : "memory");
}
// Arrive on the barrier once every product issued so far by this thread is done.
__device__ __forceinline__ void mma_commit(unsigned long long *bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_u32(bar))
      : "memory");
}

// d (+)= A B^T over DP columns: A [128 rows], B [N rows], both K-major tiles of DP / 64 chunks.
template <int DP>
__device__ __forceinline__ void mma_rows(unsigned d, unsigned a, unsigned a_chunk, unsigned b,
                                         unsigned b_chunk, unsigned idesc, bool accumulate) {
#pragma unroll
  for (int c = 0; c < DP / 64; ++c)
#pragma unroll
    for (int k = 0; k < 4; ++k)
      mma_ss(d, desc_k_major(a + c * a_chunk + k * 32), desc_k_major(b + c * b_chunk + k * 32),
             idesc, accumulate || c + k > 0);
}
// d (+)= P B over KR rows of B: P in TMEM, B [KR rows] an MN-major tile.
template <int KR>
__device__ __forceinline__ void mma_across(unsigned d, unsigned p, unsigned b, unsigned b_chunk,
                                           unsigned idesc, bool accumulate) {
#pragma unroll
  for (int k = 0; k < KR / 16; ++k)
    mma_ts(d, p + k * 8, desc_mn_major(b + k * 2048, b_chunk), idesc, accumulate || k > 0);
}

// The same over the pairs of planes; planes of A and B lie *_plane bytes apart, those of P in the TMEM
// columns p0, p1, p2.
template <int DT, int DP>
__device__ __forceinline__ void mma_rows_planes(unsigned d, unsigned a, unsigned b, unsigned chunk,
                                                unsigned plane, unsigned idesc) {
#pragma unroll
  for (int i = 0; i < kPlanePairs<DT>; ++i)
    mma_rows<DP>(d, a + plane_a<DT>(i) * plane, chunk, b + plane_b<DT>(i) * plane, chunk, idesc, i > 0);
}
template <int DT, int KR>
__device__ __forceinline__ void mma_across_planes(unsigned d, unsigned p0, unsigned p1, unsigned p2, unsigned b,
                                                  unsigned chunk, unsigned plane, unsigned idesc,
                                                  bool accumulate) {
#pragma unroll
  for (int i = 0; i < kPlanePairs<DT>; ++i)
    mma_across<KR>(d, plane_a<DT>(i) == 0 ? p0 : plane_a<DT>(i) == 1 ? p1 : p2, b + plane_b<DT>(i) * plane,
                   chunk, idesc, accumulate || i > 0);
}

// Two floats as one 32-bit pair of the 16-bit type (of bfloat16 planes for float32), the first in the
// low half.
template <int DT> __device__ __forceinline__ unsigned pack2(float lo, float hi) {
  unsigned r;
  if (DT != kF16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two float32 operations an instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mov.b64 c, {%6, %7};\n\tfma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 pair(unsigned a, unsigned b) {
  return make_float2(__uint_as_float(a), __uint_as_float(b));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Two floats as pairs of their planes.
template <int DT> __device__ __forceinline__ void split2(float2 v, unsigned (&out)[kPlanes<DT>]) {
  out[0] = pack2<DT>(v.x, v.y);
#pragma unroll
  for (int i = 1; i < kPlanes<DT>; ++i) {
    const float2 got = make_float2(-__uint_as_float(out[i - 1] << 16),
                                   -__uint_as_float(out[i - 1] & 0xffff0000u));
    v = add2(v, got);  // exact
    out[i] = pack2<DT>(v.x, v.y);
  }
}

// Columns [d0, d0 + 32) of a row as 16-bit elements into a tile, placed as TMA places them.  (A thread
// that holds a row would otherwise store it straight to memory: 32 lines an instruction, which was
// measured to take the load/store path away from everybody else.)
// Float32 tiles have chunks of 32 columns.
template <int DT>
__device__ __forceinline__ void stage32(unsigned char *tile, int chunk_bytes, int row, int d0,
                                        const float (&v)[32]) {
  if (DT == kF32) {
    unsigned char *at = tile + (d0 / 32) * chunk_bytes + row * 128;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      *reinterpret_cast<float4 *>(at + (k ^ (row & 7)) * 16) =
          make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
    return;
  }
  unsigned char *at = tile + (d0 / 64) * chunk_bytes + row * 128;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    *reinterpret_cast<uint4 *>(at + (((d0 % 64) / 8 + k) ^ (row & 7)) * 16) =
        make_uint4(pack2<DT>(v[8 * k], v[8 * k + 1]), pack2<DT>(v[8 * k + 2], v[8 * k + 3]),
                   pack2<DT>(v[8 * k + 4], v[8 * k + 5]), pack2<DT>(v[8 * k + 6], v[8 * k + 7]));
}

// 32 columns of a row as float32 into a partial result that lies column by column: neighbouring threads
// hold neighbouring rows.
__device__ __forceinline__ void store_columns(float *part, long long rows, const float (&v)[32]) {
#pragma unroll
  for (int k = 0; k < 32; ++k) part[k * rows] = v[k];
}

// Zeroes rows [first, rows) of a tile in shared memory (a warp), for the tensor cores to read.
__device__ __forceinline__ void zero_tail(unsigned char *tile, int chunks, int chunk_bytes,
                                          int first, int rows) {
  const int lane = threadIdx.x & 31;
  for (int c = 0; c < chunks; ++c)
    for (int x = first * 8 + lane; x < rows * 8; x += 32)
      *reinterpret_cast<uint4 *>(tile + c * chunk_bytes + x * 16) = make_uint4(0, 0, 0, 0);
  fence_async_shared();
  __syncwarp();
}

// A kernel that follows another one of the same call is launched while that one still runs, and waits
// for it (all of it: no kernel here lets its successor go early) before it reads its results.
__device__ __forceinline__ void wait_for_predecessor() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
template <typename... P, typename... A>
cudaError_t launch_follower(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem,
                            cudaStream_t stream, const A &...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Shared memory of a kernel, and a check that it launches with `regs` registers a thread, which
// its register moves count on.
cudaError_t prepare_tc_kernel(const void *kernel, size_t smem, int regs);

// ---- host: tensor maps ----------------------------------------------------------------
// A [B, L, H, D] tensor as the map (D, H, L, B) with boxes of 128 bytes (64 16-bit elements) x heads x
// rows / heads.  A batch or head axis of stride 0 becomes one of size 1 (b_mul, h_mul = 0).
struct TensorMap {
  CUtensorMap map;
  int b_mul, h_mul;
};
bool encode_map(TensorMap *m, const void *ptr, int dtype, long long B, long long L, long long H,
                int D, long long sb, long long sl, long long sh, int box_heads, int box_rows);
// Whether encode_map can take the tensor (16-byte alignment of base and strides).
bool map_fits(int dtype, const void *ptr, long long B, long long L, long long H, int D, long long sb,
              long long sl, long long sh);

// Float32 tensors as bfloat16 planes [B, H, L, chunk of 64 columns, 3, 64], rows at or past the utterance's
// length and columns past D as zeros.
struct PlaneSource {
  const float *src;
  long long sb, sl, sh;
  const long long *lens;  // or NULL
  int L, H;
  unsigned short *dst;
};
// of one chunk
inline size_t plane_bytes(long long B, long long L, long long H) { return (size_t)(B * L * H) * 3 * 64 * 2; }
cudaError_t launch_planes(const PlaneSource *src, int n, long long B, int D, cudaStream_t stream);
// The map of such planes, as if of heads of 192 elements a chunk.
bool encode_planes(TensorMap *m, const unsigned short *planes, long long B, long long L, long long H,
                   int chunks, int box_heads, int box_rows);

}  // namespace tdt
