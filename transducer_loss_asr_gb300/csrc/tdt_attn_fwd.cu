// tdt_attn_fwd.cu -- the forward pass of cross attention on the 5th-generation tensor cores, for
// float16 and bfloat16 heads of up to 128 elements and float32 heads of up to 64.
//
// A tile is 128 rows, a row being a (query, head) pair: where the group of a key head holds a
// power of two P of query heads, P heads of 128 / P queries share a tile and so share the frames
// that are loaded for it.  A stream is a row tile's walk over the frames, with 128 threads (thread =
// row) for its softmax:
//   wide    (more than 128 rows): a CTA walks two row tiles over the same frames;
//   single  (at most 128 rows):   a CTA walks one, with half of the SM's TMEM, registers and shared
//                                 memory, so that two CTAs share an SM.
// One warp loads tiles with TMA, one issues the products.  Per frame tile and stream:
//   S = Q K^T            128 x 128, float32 in TMEM, operands in shared memory
//   P = 2^(S c - m)      rounded to 16 bits, written over S in TMEM
//   O += P V             P from TMEM, O in TMEM
// The products of one stream run while the threads of the SM's other one are at their softmax.  The
// reference m of a row moves only when the running maximum has grown by 8 (in base 2), so O is
// rescaled rarely; weights are then at most 2^8, exact in effect: the factor cancels in O / l.
// The sum l adds the unrounded float32 weights; P is rounded to the tensors' type, as the
// products need (error u per term, at most the rounding of the output itself).
//
// float32: q, k and v are split beforehand into three bfloat16 planes (8 + 8 + 8 bits), P in the threads,
// and six products of planes stand for one; what they leave out is below 2^-24 of a term.  TMEM sums
// are cut, not rounded, so each tile's sum is added to float32 registers (error 8e-7 of the output's norm,
// 1.2e-5 when the sum stayed in TMEM).  Row of sums and scores together spill 660 bytes a thread where a CTA has two row
// tiles.
//
// Few row tiles: the frames are split over several CTAs, whose results (O, and the logarithm of
// the sum) a second kernel joins in a fixed order.
//
// Bound by the tensor cores at large sizes: 16 x 1024 queries x 4096 frames, 16 heads on 4 of 128, bfloat16:
// 345 us, 1,590 TFLOP/s of 1,936 measured for a library product; what is lost are the walk's two ends and
// exponentials that the other stream's products do not cover.  8 x 1201 x 2000 ragged, float16, 8 heads on
// 2 of 96, windows of 300 frames: 25.6 us.  8 x 121 x 7501 ragged, bfloat16, 16 heads on 4 of 128: 57 us.
// By memory for steps of shared heads: 128 x 1 x 6000, 32 heads on 8 of 128: 485 us, 6.5 TB/s of 6.8 measured.
// By latency at small ones: 4 x 41 x 200, 8 heads of 64: 7 us.  float32, 1201 x 2000, 8 heads of 64: 39 us
// with the planes.
// Two row tiles a CTA halve the reads of k and v from L2 (16 x 1024 x 4096, 8 heads on 2 of 128: 197 us
// against 210); where there is no second tile, one a CTA and two CTAs an SM (16 x 121 x 750, 16 heads of
// 64: 15.5 us against 24.1).
#include "tdt_attn_common.cuh"
#include "tdt_tc.cuh"

namespace tdt {
namespace {

constexpr int kRows = 128;          // rows of a tile, frames of a tile
constexpr int kMostSplits = 64;
constexpr float kLazy = 8.0f;
// float16 weights start at 2^7 and so stay clear of the type's least numbers; at most 2^15
template <int DT> constexpr float kShift = DT == kF16 ? 7.0f : 0.0f;

struct FwdPlan {
  int P;          // heads of a tile
  int packs;      // H / P
  int wide;       // 1: two row tiles a CTA, else one
  int tiles;      // row tiles (CTAs) of a pack
  int splits;     // CTAs that share the frames of a row tile
};

struct FwdArgs {
  AttnArgs a;
  FwdPlan p;
  int q_b, q_h, k_b, k_h, v_b, v_h, o_b, o_h;  // 0 for repeated axes
  float *part_o, *part_l;            // splits > 1: [split][CTA row][DP], [split][CTA row]
};

template <int DT, int DP, bool WIDE> struct FwdShape {
  static constexpr int CHUNKS = DP / 64;
  static constexpr int CHUNK = kRows * 128;          // bytes
  static constexpr int PLANES = kPlanes<DT>;
  static constexpr int PLANE = CHUNKS * CHUNK;
  static constexpr int TILE = PLANES * PLANE;
  static constexpr int NS = WIDE ? 2 : 1;            // streams
  static constexpr int SLOTS = PLANES == 3 ? (WIDE ? 2 : 3) : WIDE ? (DP == 64 ? 8 : 4) : (DP == 64 ? 5 : 2);
  static constexpr int BYTES = (NS + SLOTS) * TILE;
  static constexpr int THREADS = NS * 128 + 128;     // softmax; TMA, MMA, tails, a spare warp
  static constexpr int CTAS = WIDE ? 1 : 2;          // of an SM
  static constexpr int TMEM = WIDE ? 512 : 256;      // columns: S and O of each stream, a third plane of P
  // registers of a thread: at launch, then of the softmax warpgroups and of the other one, which
  // adds up to the same: 3 x 168 = 2 x 208 + 88, 2 x 128 = 200 + 56
  static constexpr int REGS = WIDE ? 168 : 128;
  static constexpr int SOFTMAX_REGS = WIDE ? 208 : 200;
  static constexpr int OTHER_REGS = WIDE ? 88 : 56;
};

struct FwdShared {
  unsigned long long full[8], empty[8], q_full, s_full[2], p_ready[2], o_full[2], tail_full, drained;
  unsigned tmem;
  int gave_up;
  Hull hull;
};

// 32 scores of a row (float32 bits) to weights 2^(s c - ref), packed in pairs of each plane and added to
// sum.
template <int DT, int N>
__device__ __forceinline__ void exp_pack(const unsigned (&s)[32], float c, float neg,
                                         unsigned (&out)[kPlanes<DT>][N], int at, float2 &sum) {
  const float2 c2 = make_float2(c, c), n2 = make_float2(neg, neg);
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    const float2 z = fma2(pair(s[i], s[i + 1]), c2, n2);
    const float2 p = make_float2(fast_exp2(z.x), fast_exp2(z.y));
    sum = add2(sum, p);
    unsigned planes[kPlanes<DT>];
    split2<DT>(p, planes);
#pragma unroll
    for (int k = 0; k < kPlanes<DT>; ++k) out[k][at + i / 2] = planes[k];
  }
}

template <int DT, int DP, bool WIDE>
__global__ void __launch_bounds__(FwdShape<DT, DP, WIDE>::THREADS, FwdShape<DT, DP, WIDE>::CTAS)
    attn_fwd_tc_kernel(const __grid_constant__ CUtensorMap qm, const __grid_constant__ CUtensorMap km,
                       const __grid_constant__ CUtensorMap vm, const __grid_constant__ CUtensorMap om,
                       const __grid_constant__ FwdArgs f) {
  typedef FwdShape<DT, DP, WIDE> S;
  extern __shared__ unsigned char raw[];
  __shared__ FwdShared sh;
  unsigned char *tiles = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  unsigned char *q_tile = tiles, *slots = tiles + S::NS * S::TILE;
  const AttnArgs &a = f.a;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  // this CTA's rows and frames
  unsigned id = blockIdx.x;
  const int split = id % f.p.splits;
  id /= f.p.splits;
  const unsigned cta = id;
  const int tile = id % f.p.tiles;
  id /= f.p.tiles;
  const int pack = id % f.p.packs;
  const long long b = id / f.p.packs;
  const int P = f.p.P, per = kRows / P, i0 = tile * S::NS * per;
  const int h0 = pack * P, hk = h0 / a.G;
  const Lens n = utt_lens(a, b);
  const bool some = i0 < n.nq && n.nk > 0;  // else no row sees a frame
  // frames [hull.x, hull.y) in tiles of 128 from hull.x; this CTA takes T tiles from `begin`
  int begin = 0, T = 0;
  // Frames past the utterance's end may hold anything, and 0 times NaN is NaN.  In the last tile of
  // v, which is the last tile loaded, a warp of its own zeroes them (unless TMA did, past the
  // tensor's end): the load then arrives at tail_full, and that warp hands the tile on.
  bool cut = false;
  auto walk = [&](int2 hull) {
    const int2 steps = share_of((hull.y - hull.x + kRows - 1) / kRows, split, f.p.splits);
    begin = hull.x + steps.x * kRows;
    T = steps.y - steps.x;
    cut = S::PLANES == 1 && T > 0 && n.nk < a.Lk && begin + T * kRows > n.nk;  // planes end in zeros
  };
  if (!a.windows && some) walk(make_int2(0, n.nk));
  auto frame = [&](int s) { return begin + s * kRows; };
  auto load = [&](int at) {  // tiles count up: k of step 0, v of step 0, k of step 1, ...
    const int slot = at % S::SLOTS, s = at / 2;
    const bool values = at & 1;
    unsigned long long *bar = cut && at == 2 * T - 1 ? &sh.tail_full : &sh.full[slot];
    arrive_expect_tx(bar, S::TILE);
    for (int ch = 0; ch < S::PLANES * S::CHUNKS; ++ch)
      tma_load_4d(values ? &vm : &km, slots + slot * S::TILE + ch * S::CHUNK, bar, ch * 64,
                  hk * (values ? f.v_h : f.k_h), frame(s), (int)b * (values ? f.v_b : f.k_b));
  };

  constexpr int kAux = S::NS * 4;  // the first warp past the softmax's: TMA
  const int stream = warp >> 2, r = threadIdx.x & 127;
  int row = 0, head = 0;
  int2 range = make_int2(0, 0);
  if (warp < kAux) {
    row = i0 + stream * per + r / P;
    head = h0 + r % P;
    range = row_range(a, b, row, n);
    if (a.windows) hull_note(sh.hull, warp, range);
  } else if (warp == kAux && lane == 0) {
    for (int i = 0; i < S::SLOTS; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
    }
    mbar_init(&sh.q_full, 1);
    mbar_init(&sh.tail_full, 1);
    mbar_init(&sh.drained, 1);
    for (int w = 0; w < S::NS; ++w) {
      mbar_init(&sh.s_full[w], 1);
      mbar_init(&sh.p_ready[w], 128);
      mbar_init(&sh.o_full[w], 1);
    }
    fence_mbar_init_cluster();
    sh.gave_up = 0;
    if (some) {
      arrive_expect_tx(&sh.q_full, S::NS * S::TILE);
      for (int t = 0; t < S::NS; ++t)
        for (int ch = 0; ch < S::PLANES * S::CHUNKS; ++ch)
          tma_load_4d(&qm, q_tile + t * S::TILE + ch * S::CHUNK, &sh.q_full, ch * 64, h0 * f.q_h,
                      i0 + t * per, (int)b * f.q_b);
    }
    if (T > 0) {  // no windows: the walk is known
      load(0);
      load(1);
    }
  } else if (warp == kAux + 1) {
    tmem_alloc<S::TMEM>(&sh.tmem);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const unsigned tmem = __shfl_sync(0xffffffffu, sh.tmem, 0);
  const Waiter wait{&sh.gave_up};
  if (a.windows) walk(hull_of<kAux>(sh.hull));
  const float c = a.scale * kLog2e;

  if (warp >= kAux) {
    warpgroup_give_registers<S::OTHER_REGS>();  // to the softmax warps, which hold a row of scores
    if (warp == kAux && lane == 0 && some && T == 0) wait(&sh.q_full, 0);  // nobody else does
    if (warp == kAux && lane == 0 && T > 0) {
      bool ok = true;
      int at = a.windows ? 0 : 2;  // the first two were loaded above
      for (; at < 2 * T; ++at) {
        ok = wait(&sh.empty[at % S::SLOTS], ((unsigned)(at / S::SLOTS) & 1) ^ 1);
        if (!ok) break;
        load(at);
      }
      if (!ok)  // copies in flight land before the CTA ends
        for (int i = max(0, at - S::SLOTS); i < at; ++i)
          Waiter::drain(&sh.full[i % S::SLOTS], (unsigned)(i / S::SLOTS) & 1);
    }
    if (warp == kAux + 2 && cut) {
      const int slot = (2 * T - 1) % S::SLOTS;
      if (__all_sync(0xffffffffu, wait(&sh.tail_full, 0)))
        zero_tail(slots + slot * S::TILE, S::CHUNKS, S::CHUNK, n.nk - frame(T - 1), kRows);
      if (lane == 0) mbar_arrive(&sh.full[slot]);
    }
    if (warp == kAux + 1 && T > 0 && elect_one()) {
      constexpr unsigned i_s = mma_desc<DT>(kRows, false), i_o = mma_desc<DT>(DP, true);
      const unsigned q_addr = smem_u32(q_tile), s_addr = smem_u32(slots);
      bool ok = wait(&sh.q_full, 0);
      auto loaded = [&](int at) {  // slots count up in the loader's order
        ok = ok && wait(&sh.full[at % S::SLOTS], (unsigned)(at / S::SLOTS) & 1);
      };
      auto scores = [&](int w, int at) {  // S_w = Q_w K^T
        tc_fence_after();
        if (!ok) return;
        const int slot = at % S::SLOTS;
        mma_rows_planes<DT, DP>(tmem + w * kRows, q_addr + w * S::TILE, s_addr + slot * S::TILE, S::CHUNK,
                                S::PLANE, i_s);
        mma_commit(&sh.s_full[w]);
        if (w == S::NS - 1) mma_commit(&sh.empty[slot]);
      };
      auto values = [&](int w, int s, int at) {  // O_w += P_w V
        const int slot = at % S::SLOTS;
        ok = ok && wait(&sh.p_ready[w], s & 1);
        tc_fence_after();
        if (!ok) return;
        const unsigned o_at = tmem + S::NS * kRows + w * DP, p_at = tmem + w * kRows,
                       third = tmem + S::NS * (kRows + DP) + w * 64, v_at = s_addr + slot * S::TILE;
        if constexpr (S::PLANES == 1) {
          mma_across<kRows>(o_at, p_at, v_at, S::CHUNK, i_o, s > 0);
        } else {  // this tile's part of O: 32 frames' planes 0 and 1 lie where their scores were
#pragma unroll
          for (int i = 0; i < kPlanePairs<DT>; ++i)
#pragma unroll
            for (int k = 0; k < kRows / 16; ++k) {
              const unsigned in = k / 2 * 32 + k % 2 * 8;
              const unsigned pa = plane_a<DT>(i) == 0   ? p_at + in
                                  : plane_a<DT>(i) == 1 ? p_at + in + 16
                                                        : third + k * 8;
              mma_ts(o_at, pa, desc_mn_major(v_at + plane_b<DT>(i) * S::PLANE + k * 2048, S::CHUNK), i_o,
                     i + k > 0);
            }
        }
        if (w == S::NS - 1) mma_commit(&sh.empty[slot]);
        if (s + 1 == T) mma_commit(&sh.o_full[w]);
      };
      loaded(0);
      for (int w = 0; w < S::NS; ++w) scores(w, 0);
      for (int s = 0; ok && s < T; ++s) {
        const int at = 1 + 2 * s;
        loaded(at);
#pragma unroll
        for (int w = 0; w < S::NS; ++w) {
          values(w, s, at);
          if (s + 1 < T) {
            if (w == 0) loaded(at + 1);
            scores(w, at + 1);
          }
        }
      }
      if (!ok) {  // products in flight end before TMEM is freed
        mma_commit(&sh.drained);
        Waiter::drain(&sh.drained, 0);
      }
    }
  } else {
    warpgroup_take_registers<S::SOFTMAX_REGS>();
    const unsigned lanes = (unsigned)((warp & 3) * 32) << 16;
    const unsigned s_col = tmem + lanes + stream * kRows, o_col = tmem + lanes + S::NS * kRows + stream * DP;
    float ref = -INFINITY, l = 0.0f;  // reference maximum (base 2) and sum
    // a row that sees nothing holds whatever its tile does: its result is set at the end
    const bool alive = range.y > range.x;
    float o_row[S::PLANES == 3 ? DP : 1];  // float32: the row of O, to which each tile's part is added
#pragma unroll
    for (int k = 0; k < (S::PLANES == 3 ? DP : 1); ++k) o_row[k] = 0.0f;
    auto add_tile = [&]() {
      if constexpr (S::PLANES == 3) {
#pragma unroll
        for (int i = 0; i < DP / 32; ++i) {
          unsigned o[32];
          tmem_ld32(o_col + i * 32, o);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 32; ++k) o_row[i * 32 + k] += __uint_as_float(o[k]);
        }
      }
    };
    bool ok = true;
    for (int s = 0; s < T; ++s) {
      ok = wait(&sh.s_full[stream], s & 1);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      const int j0 = frame(s);
      const bool masked = __any_sync(0xffffffffu, alive && (range.x > j0 || range.y < j0 + kRows));
      const int lo = range.x - j0;
      const unsigned len = (unsigned)(range.y - range.x);
      if constexpr (S::PLANES == 3) {
        // the scores are read twice, 32 at a time: registers hold the row of O
        unsigned x[32];
        auto scores = [&](int i) {
          tmem_ld32(s_col + i * 32, x);
          tmem_wait_ld();
          if (masked)
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if ((unsigned)(i * 32 + k - lo) >= len) x[k] = 0xff800000u;  // -inf
        };
        if (s > 0) add_tile();
        float m0 = -INFINITY;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          scores(i);
#pragma unroll
          for (int k = 0; k < 32; k += 2) m0 = max3(m0, __uint_as_float(x[k]), __uint_as_float(x[k + 1]));
        }
        const float top = m0 * c;
        if (alive && top > ref) {
          const float scale = fast_exp2(ref - top);
#pragma unroll
          for (int k = 0; k < DP; ++k) o_row[k] *= scale;
          l *= scale;
          ref = top;
        }
        __syncwarp();
        const float neg = ref == -INFINITY ? 0.0f : -ref;
        const unsigned third = tmem + lanes + S::NS * (kRows + DP) + stream * 64;
        float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          unsigned p[S::PLANES][16];
          scores(i);
          exp_pack<DT>(x, c, neg, p, 0, sum);
          tmem_st16(s_col + i * 32, p[0]);
          tmem_st16(s_col + i * 32 + 16, p[1]);
          tmem_st16(third + i * 16, p[2]);
        }
        l += sum.x + sum.y;
      } else {
        unsigned x[4][32];
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld32(s_col + i * 32, x[i]);
        tmem_wait_ld();
        if (masked) {
#pragma unroll
          for (int i = 0; i < 128; ++i)
            if ((unsigned)(i - lo) >= len) x[i >> 5][i & 31] = 0xff800000u;  // -inf
        }
        float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          m0 = max3(m0, __uint_as_float(x[0][i]), __uint_as_float(x[0][i + 1]));
          m1 = max3(m1, __uint_as_float(x[1][i]), __uint_as_float(x[1][i + 1]));
          m0 = max3(m0, __uint_as_float(x[2][i]), __uint_as_float(x[2][i + 1]));
          m1 = max3(m1, __uint_as_float(x[3][i]), __uint_as_float(x[3][i + 1]));
        }
        const float top = fmaxf(m0, m1) * c;
        const bool grow = alive && top > ref + (kLazy + kShift<DT>);  // from -inf: any score
        if (__any_sync(0xffffffffu, grow)) {
          const float now = grow ? top - kShift<DT> : ref;
          const float scale = grow ? fast_exp2(ref - now) : 1.0f;
          if (s > 0) {  // the products up to tile s - 1 are done: S of tile s came after them
            unsigned o[32];
#pragma unroll
            for (int i = 0; i < DP / 32; ++i) {
              tmem_ld32(o_col + i * 32, o);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * scale);
              tmem_st32(o_col + i * 32, o);
            }
          }
          l *= scale;
          ref = now;
        }
        const float neg = ref == -INFINITY ? 0.0f : -ref;
        float2 sum0 = make_float2(0.0f, 0.0f), sum1 = sum0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          unsigned p[S::PLANES][32];
          exp_pack<DT>(x[2 * i], c, neg, p, 0, sum0);
          exp_pack<DT>(x[2 * i + 1], c, neg, p, 16, sum1);
          tmem_st32(s_col + i * 32, p[0]);
        }
        sum0 = add2(sum0, sum1);
        l += sum0.x + sum0.y;
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&sh.p_ready[stream]);
    }
    if (T > 0 && ok) ok = wait(&sh.o_full[stream], 0);
    if (T == 0 && some) ok = wait(&sh.q_full, 0);  // the tile's memory is used below
    __syncwarp();
    tc_fence_after();
    if (S::PLANES == 3 && T > 0) add_tile();
    if (!alive) l = 0.0f;
    const bool bad = n.bad || !ok || *reinterpret_cast<volatile int *>(&sh.gave_up);
    const long long tile_at = (long long)split * f.p.tiles * f.p.packs * a.B + cta;  // of a partial result
    if (row < a.Lq) {
      const float total = bad ? NAN : l == 0.0f ? -INFINITY : ref + log2f(l);
      if (f.p.splits > 1)
        f.part_l[tile_at * (S::NS * kRows) + threadIdx.x] = total;
      else if (a.lse)
        a.lse[(b * a.H + head) * a.Lq + row] = total * kLn2;
    }
    const float inv = bad ? NAN : l == 0.0f ? 0.0f : 1.0f / l;
    unsigned char *out_tile = q_tile + stream * S::TILE;  // every product with q is done
#pragma unroll
    for (int i = 0; i < DP / 32; ++i) {
      unsigned o[32];
      if (S::PLANES == 1 && T > 0) {
        tmem_ld32(o_col + i * 32, o);
        tmem_wait_ld();
      }
      float v[32];
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        const float x = S::PLANES == 3 ? o_row[S::PLANES == 3 ? i * 32 + k : 0] : __uint_as_float(o[k]);
        v[k] = bad ? NAN : l == 0.0f ? 0.0f : x * inv;
      }
      if (f.p.splits == 1) {
        stage32<DT>(out_tile, S::CHUNK, r, i * 32, v);
      } else if (row < a.Lq) {
        store_columns(f.part_o + (tile_at * DP + i * 32) * (S::NS * kRows) + threadIdx.x, S::NS * kRows, v);
      }
      __syncwarp();
    }
    if (f.p.splits == 1) {
      fence_async_shared();
      named_barrier<128>(1 + stream);
      if (r == 0 && row < a.Lq) {
        constexpr int kColumns = DT == kF32 ? 32 : 64;  // of a chunk
        for (int ch = 0; ch < DP / kColumns; ++ch)
          if (ch * kColumns < a.D)
            tma_store_4d(&om, out_tile + ch * S::CHUNK, ch * kColumns, h0 * f.o_h, row, (int)b * f.o_b);
        tma_store_commit();
        tma_store_wait_read();
      }
      __syncwarp();
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == kAux + 1) tmem_free<S::TMEM>(tmem);
}

// Joins the splits for 32 rows and 32 columns: o = sum_s 2^(l_s - l) o_s, l = log2 sum_s 2^(l_s), the
// splits in order.  The partial results lie column by column; they leave row by row through shared memory.
// Blocks are small and every split's loads go out together: the kernel's time is a few memory latencies.
template <int DT, int DP>
__global__ void __launch_bounds__(256) attn_join_kernel(const __grid_constant__ FwdArgs f, int rows) {
  const AttnArgs &a = f.a;
  __shared__ float out[32][33];
  __shared__ float weight[kMostSplits][32];
  const unsigned d0 = blockIdx.x % (DP / 32) * 32, block = blockIdx.x / (DP / 32);
  const int groups = rows / 32, r = threadIdx.x & 31, part = threadIdx.x >> 5;
  const unsigned cta = block / groups, r0 = block % groups * 32;
  const unsigned ctas = gridDim.x / (DP / 32) / groups;
  const int tile = cta % f.p.tiles, pack = cta / f.p.tiles % f.p.packs;
  const long long b = cta / f.p.tiles / f.p.packs;
  const int first = tile * (rows / f.p.P) + r0 / f.p.P;  // position of row r0; P divides 32 or 32 divides it
  auto row_of = [&](int x) { return first + (int)((r0 % f.p.P + x) / f.p.P); };
  auto head_of = [&](int x) { return pack * f.p.P + (int)((r0 + x) % f.p.P); };
  if (first >= a.Lq) return;
  const bool real = row_of(r) < a.Lq;
  const int splits = f.p.splits;
  wait_for_predecessor();
  for (int s = part; s < splits; s += 8)
    weight[s][r] = real ? f.part_l[((long long)s * ctas + cta) * rows + r0 + r] : -INFINITY;
  const float *po = f.part_o + ((long long)cta * DP + d0 + part) * rows + r0 + r;
  const long long next = (long long)ctas * DP * rows;
  constexpr int U = 8;  // splits whose loads are in flight
  float v[U][4];
  auto load = [&](int s0) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[u][i] = real && s0 + u < splits ? po[(s0 + u) * next + i * 8 * rows] : 0.0f;
  };
  load(0);
  __syncthreads();
  float top = -INFINITY, sum = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  bool bad = false;
  for (int s = 0; s < splits; ++s) {
    const float x = weight[s][r];
    bad |= x != x;
    top = fmaxf(top, x);
  }
  for (int s0 = 0; s0 < splits; s0 += U) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (s0 + u < splits && top > -INFINITY) {
        const float w = fast_exp2(weight[s0 + u][r] - top);
        sum += w;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = fmaf(w, v[u][i], o[i]);
      }
    if (s0 + U < splits) load(s0 + U);
  }
  const float inv = bad ? NAN : sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) out[r][part + i * 8] = bad ? NAN : o[i] * inv;
  if (part == 0 && d0 == 0 && real && a.lse)
    a.lse[(b * a.H + head_of(r)) * a.Lq + row_of(r)] =
        bad ? NAN : sum > 0.0f ? (top + log2f(sum)) * kLn2 : -INFINITY;
  __syncthreads();
  if (threadIdx.x < 128) {
    const int rr = threadIdx.x / 4, d = threadIdx.x % 4 * 8;
    const float *x = &out[rr][d];
    if (row_of(rr) >= a.Lq || d0 + d >= a.D) {
    } else if constexpr (DT == kF32) {
      float *dst = static_cast<float *>(const_cast<void *>(a.out)) + b * a.so.b + row_of(rr) * a.so.l +
                   head_of(rr) * a.so.h + d0 + d;
      *reinterpret_cast<float4 *>(dst) = make_float4(x[0], x[1], x[2], x[3]);
      if (d0 + d + 4 < a.D)
        *reinterpret_cast<float4 *>(dst + 4) = make_float4(x[4], x[5], x[6], x[7]);
    } else {
      unsigned short *dst = static_cast<unsigned short *>(const_cast<void *>(a.out)) + b * a.so.b +
                            row_of(rr) * a.so.l + head_of(rr) * a.so.h + d0 + d;
      *reinterpret_cast<uint4 *>(dst) = make_uint4(pack2<DT>(x[0], x[1]), pack2<DT>(x[2], x[3]),
                                                   pack2<DT>(x[4], x[5]), pack2<DT>(x[6], x[7]));
    }
  }
}

FwdPlan plan(long long B, long long Lq, long long Lk, int H, int G, int dtype) {
  FwdPlan p;
  p.P = attn_row_pack(G);
  p.packs = H / p.P;
  const long long rows = Lq * p.P;
  p.wide = rows > kRows;
  const int tile_rows = p.wide ? 2 * kRows : kRows;
  p.tiles = (int)((rows + tile_rows - 1) / tile_rows);
  // split the frames while the CTAs leave SMs idle, if that saves a CTA a dozen tiles' time: joining
  // costs about as much as eight take; a float32 tile has six times the products and takes three times as
  // long.  More splits than SMs, so that utterances of other lengths even out, lose: 8 ragged x 121 x 7501, 16
  // heads on 4 of 128, 62 us with twice as many against 61; all of full length 69 against 63.
  const long long ctas = B * p.packs * p.tiles, steps = (Lk + kRows - 1) / kRows;
  long long s = ctas > 0 ? (p.wide ? 1 : 2) * kSMs / ctas : 1;
  if (s > steps / 4) s = steps / 4;
  if (s > kMostSplits) s = kMostSplits;
  p.splits = s < 2 || (steps - steps / s) * (dtype == kF32 ? 3 : 1) < 12 ? 1 : (int)s;
  return p;
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

template <int DT, int DP, bool WIDE>
cudaError_t launch(const FwdArgs &f, const TensorMap &q, const TensorMap &k, const TensorMap &v, const TensorMap &o,
                   cudaStream_t stream) {
  typedef FwdShape<DT, DP, WIDE> S;
  const size_t smem = S::BYTES + 1024;
  cudaError_t e = prepare_tc_kernel(reinterpret_cast<const void *>(attn_fwd_tc_kernel<DT, DP, WIDE>),
                                    smem, S::REGS);
  if (e != cudaSuccess) return e;
  const long long ctas = f.a.B * f.p.packs * f.p.tiles;
  attn_fwd_tc_kernel<DT, DP, WIDE>
      <<<(unsigned)(ctas * f.p.splits), S::THREADS, smem, stream>>>(q.map, k.map, v.map, o.map, f);
  e = cudaGetLastError();
  if (e != cudaSuccess || f.p.splits == 1) return e;
  const int rows = S::NS * kRows;
  return launch_follower(attn_join_kernel<DT, DP>, dim3((unsigned)(ctas * (rows / 32) * (DP / 32))), 256, 0,
                         stream, f, rows);
}

template <int DT>
cudaError_t by_shape(const FwdArgs &f, const TensorMap &q, const TensorMap &k, const TensorMap &v,
                     const TensorMap &o, cudaStream_t s) {
  if constexpr (DT != kF32)
    if (f.a.D > 64)
      return f.p.wide ? launch<DT, 128, true>(f, q, k, v, o, s) : launch<DT, 128, false>(f, q, k, v, o, s);
  return f.p.wide ? launch<DT, 64, true>(f, q, k, v, o, s) : launch<DT, 64, false>(f, q, k, v, o, s);
}

// The workspace: planes of q, k, v (float32), then the partial results of splits.
struct FwdSpace {
  size_t q, k, v, part_o, part_l, total;
};
FwdSpace space(const FwdPlan &p, long long B, long long Lq, long long Lk, int H, int Hkv, int D, int dtype) {
  FwdSpace s = {};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align256(bytes);
    return here;
  };
  if (dtype == kF32) {
    s.q = take(plane_bytes(B, Lq, H));
    s.k = take(plane_bytes(B, Lk, Hkv));
    s.v = take(plane_bytes(B, Lk, Hkv));
  }
  const size_t rows = p.splits == 1 ? 0 : (size_t)B * p.packs * p.tiles * p.splits * (p.wide ? 2 : 1) * kRows;
  s.part_o = take(rows * (D <= 64 ? 64 : 128) * 4);
  s.part_l = take(rows * 4);
  s.total = at;
  return s;
}

}  // namespace

int attn_row_pack(int G) {
  int P = 1;
  while (P < 16 && G % (2 * P) == 0) P *= 2;
  return P;
}

bool attn_tc_takes(int dtype, long long Lq, long long Lk, int G, int D, bool backward) {
  if (Lq == 0 || Lk == 0) return false;
  // no workspace for float32 steps
  return dtype == kF32 ? D <= 64 && (backward || Lq * G > kStepRows || D % 8 != 0) : D <= 128;
}

size_t attn_fwd_tc_workspace(long long B, long long Lq, long long Lk, int H, int Hkv, int D, int dtype) {
  return space(plan(B, Lq, Lk, H, H / Hkv, dtype), B, Lq, Lk, H, Hkv, D, dtype).total;
}

bool attn_fwd_tc_fits(const AttnArgs &a, int dtype) {
  auto fits = [&](const void *p, const Strides &s, long long L, int H) {
    return map_fits(dtype, p, a.B, L, H, a.D, s.b, s.l, s.h);
  };
  if (!attn_tc_takes(dtype, a.Lq, a.Lk, a.G, a.D, false) || !fits(a.out, a.so, a.Lq, a.H)) return false;
  return dtype == kF32 || (fits(a.q, a.sq, a.Lq, a.H) && fits(a.k, a.sk, a.Lk, a.Hkv) &&
                           fits(a.v, a.sv, a.Lk, a.Hkv) && (attn_row_pack(a.G) == 1 || a.sq.h != 0));
}

cudaError_t launch_attn_fwd_tc(const AttnArgs &a, int dtype, void *workspace, cudaStream_t stream) {
  FwdArgs f = {};
  f.a = a;
  f.p = plan(a.B, a.Lq, a.Lk, a.H, a.G, dtype);
  const FwdSpace at = space(f.p, a.B, a.Lq, a.Lk, a.H, a.Hkv, a.D, dtype);
  char *ws = static_cast<char *>(workspace);
  f.part_o = reinterpret_cast<float *>(ws + at.part_o);
  f.part_l = reinterpret_cast<float *>(ws + at.part_l);
  TensorMap q, k, v, o;
  bool ok = encode_map(&o, a.out, dtype, a.B, a.Lq, a.H, a.D, a.so.b, a.so.l, a.so.h, f.p.P, kRows / f.p.P);
  if (dtype == kF32) {
    const PlaneSource t[3] = {
        {static_cast<const float *>(a.q), a.sq.b, a.sq.l, a.sq.h, a.q_lens, a.Lq, a.H,
         reinterpret_cast<unsigned short *>(ws + at.q)},
        {static_cast<const float *>(a.k), a.sk.b, a.sk.l, a.sk.h, a.k_lens, a.Lk, a.Hkv,
         reinterpret_cast<unsigned short *>(ws + at.k)},
        {static_cast<const float *>(a.v), a.sv.b, a.sv.l, a.sv.h, a.k_lens, a.Lk, a.Hkv,
         reinterpret_cast<unsigned short *>(ws + at.v)}};
    const cudaError_t e = launch_planes(t, 3, a.B, a.D, stream);
    if (e != cudaSuccess) return e;
    ok = ok && encode_planes(&q, t[0].dst, a.B, a.Lq, a.H, 1, f.p.P, kRows / f.p.P) &&
         encode_planes(&k, t[1].dst, a.B, a.Lk, a.Hkv, 1, 1, kRows) &&
         encode_planes(&v, t[2].dst, a.B, a.Lk, a.Hkv, 1, 1, kRows);
  } else {
    ok = ok &&
         encode_map(&q, a.q, dtype, a.B, a.Lq, a.H, a.D, a.sq.b, a.sq.l, a.sq.h, f.p.P, kRows / f.p.P) &&
         encode_map(&k, a.k, dtype, a.B, a.Lk, a.Hkv, a.D, a.sk.b, a.sk.l, a.sk.h, 1, kRows) &&
         encode_map(&v, a.v, dtype, a.B, a.Lk, a.Hkv, a.D, a.sv.b, a.sv.l, a.sv.h, 1, kRows);
  }
  if (!ok) return cudaErrorInvalidValue;
  f.o_b = o.b_mul;
  f.o_h = o.h_mul;
  f.q_b = q.b_mul;
  f.q_h = q.h_mul;
  f.k_b = k.b_mul;
  f.k_h = k.h_mul;
  f.v_b = v.b_mul;
  f.v_h = v.h_mul;
  return dtype == kF32   ? by_shape<kF32>(f, q, k, v, o, stream)
         : dtype == kF16 ? by_shape<kF16>(f, q, k, v, o, stream)
                         : by_shape<kBF16>(f, q, k, v, o, stream);
}

}  // namespace tdt
