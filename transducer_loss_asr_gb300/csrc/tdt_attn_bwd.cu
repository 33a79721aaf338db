// tdt_attn_bwd.cu -- the backward pass of cross attention on the 5th-generation tensor cores, for
// float16 and bfloat16 heads of up to 128 elements and float32 heads of up to 64 (three bfloat16 planes a
// tensor, six products for one, each tile's sums added to float32 registers; as in the forward pass).
//
// Every sum has one owner and a fixed order (no atomic sums).  Where the rows of a key head fill at most one
// tile of 128 and heads are at most 64 wide (label states of one utterance), one kernel walks the frames
// and forms all three gradients with five products a tile; P and dS go through shared memory, since
// they are contracted along both axes.  Otherwise two kernels:
//   dq    a CTA holds 128 rows ((query, head) pairs, packed as in the forward pass) and walks the
//         frames:  S = Q K^T, dP = dO V^T, dS = P (dP - delta), dQ += dS K      3 products a tile
//   dk/dv a CTA holds 128 frames and walks the rows of the heads of its group, with the scores
//         transposed:  S^T = K Q^T, dP^T = V dO^T, dV += P^T dO, dK += dS^T Q    4 products a tile
// P = 2^(S c - lse) is formed again from the forward pass's lse.  Seven products where five would
// do with one walk; over several row tiles that one would add its dQ tiles to memory in float32, each
// frame tile in its turn for a fixed order.  Which is faster was not measured.
// delta = dO . O of each row is formed by the dq kernel and kept for the other (short walks: see kDeltaFrames).
//
// Two warpgroups share a tile's elementwise work (thread = TMEM lane, each group half of the
// columns); a warp loads with TMA, a warp issues products, one zeroes tails, and in the dk/dv kernel one
// fetches the rows' lse and delta.  P and dS are rounded to the tensors' type and written over S and dP in
// TMEM, each group over columns that it alone has read, and go into the products from there.
// Scores of the next tile are formed while the threads are at this one's dS.
//
// Few CTAs: the walk is split over several, whose float32 sums a third kernel adds in order.
//
// P, dS: rounding them to 16 bits is what the products need.  With delta from the rounded O (long walks only, see
// kDeltaFrames) it is what dq's error consists of (bfloat16: 2.4e-3 to 2.5e-3 of its norm, 1.7e-3 where only the result is
// rounded).  A dS of two planes would take two products more.
//
// Bound by the tensor cores and the shared memory that feeds them: a product of two shared-memory operands
// of 128 x 128 x 16 takes the 64 clocks of its reads, and S, dP in both kernels are such.  Measured:
//   16 x 1024 x 4096, 16 heads on 4 of 128, bfloat16   1,307 us (dq 567): 1,050 TFLOP/s on the five products
//                                                      of the formula, 1,470 on the seven done
//   8 x 1201 x 2000 ragged, 8 heads on 2 of 96, float16, windows of 300   88 us (max |v| 3, dq 39, dk/dv 46)
//   16 x 121 x 750, 16 heads of 64                     36.5 us by one kernel, 82.5 by two (ragged: 33.7)
//   4 x 41 x 200, 8 heads of 64                        9.8 us by one kernel; latency
//   1201 x 2000, 8 heads of 64, float32                135 us with the planes
// The float32 walks spill: 504 bytes of stores a thread in dq, 244 in dk/dv (scores, dP and sums of a row at once).
#include <algorithm>

#include "tdt_attn_common.cuh"
#include "tdt_tc.cuh"

namespace tdt {
namespace {

constexpr int kRows = 128;
constexpr int kThreads = 384;
constexpr int kLaunchRegs = 168;  // 3 warpgroups x 168 = 2 x 208 + 88
constexpr int kWorkRegs = 208, kOtherRegs = 88;
// float16 weights are held as 2^15 p for the product with dO (p <= 1, so below the type's most): what a
// frame gets from rows that hardly weigh it stays clear of the type's least numbers.
template <int DT> constexpr float kShift = DT == kF16 ? 15.0f : 0.0f;
template <int DT> constexpr float kUnshift = DT == kF16 ? 1.0f / 32768.0f : 1.0f;
constexpr int kTileBits = 4096;   // row tiles whose windows the dk/dv kernel looks at beforehand

// float16 dS is held as 2^e dS, since dS is as small as dO / frames and as large as dO . v: in 16 bits one falls
// below the type's normal range and the other goes past it where the gradients themselves are far from either.
//   |dS_ij| = p_ij |dO_i . v_j - delta_i| <= |dO_i| |v_j| + |delta_i| =: bound,   2^e bound in [2^14, 2^15),
// with |v_j| <= sqrt(D) max |v| over the utterance's frames of the key head, from a kernel that reads v beforehand
// (attn_v_most_kernel).  dq: an e for each row, so a row's accuracy is its own.  dk, dv and the one-tile kernel: one
// for the CTA, from the largest |dO_i| and |delta_i| of the rows of the key head.  2^e goes in with factors that are
// there anyway and out with `scale`.  Error of dq, 2,000 frames, dO of size 1, 1e-3, 1e-4: 3.0e-4, 5.1e-4, 4.6e-3 of its
// norm, where rounding the result alone gives 2.1e-4, 4.6e-4, 4.6e-3.  (bfloat16 has float32's range, and float32's
// planes too.)
constexpr int kVParts = 32;  // stretches of the frames whose max |v| is noted apart: a lane each

// 0 where there is nothing to bound, or no finite bound
__device__ __forceinline__ int ds_shift(float bound) {
  if (!(bound > 0.0f) || !(bound < INFINITY)) return 0;
  return min(14 - ((int)(__float_as_uint(bound) >> 23) - 127), 64);
}
__device__ __forceinline__ float power_of_2(int e) { return __uint_as_float((unsigned)(127 + e) << 23); }

struct BwdPlan {
  int P, packs, tiles;          // heads of a row tile, H / P, row tiles of a pack
  int f_tiles;                  // frame tiles
  int dq_splits, dkv_splits;
  bool one;                     // one row tile a key head and D <= 64: attn_one_tc_kernel
  int v_parts;                  // float16: stretches of the frames in v_most, else 0
};

struct BwdArgs {
  AttnArgs a;
  BwdPlan p;
  // 0 for repeated axes
  int out_b, out_h, q_b, q_h, go_b, go_h, k_b, k_h, v_b, v_h, dq_b, dq_h, dk_b, dk_h, dv_b, dv_h;
  float *part;                  // splits > 1: [split][CTA][128][DP], dk's after dv's
  // float16: [B][Hkv][v_parts] largest |v|, [B][packs][tiles] largest |dO_i| and |delta_i| of a row tile
  float *v_most;
  float2 *row_most;
};

template <int DT, int DP> struct BwdShape {
  static constexpr int CHUNKS = DP / 64;
  static constexpr int CHUNK = kRows * 128;
  static constexpr int PLANES = kPlanes<DT>;
  static constexpr int PLANE = CHUNKS * CHUNK;
  static constexpr int TILE = PLANES * PLANE;
  static constexpr int KS = PLANES == 3 ? 1 : 3, VS = PLANES == 3 ? 1 : 2;   // dq: slots of k and v
  static constexpr int RS = PLANES == 3 ? 1 : DP == 64 ? 4 : 2;              // dk/dv: slots of q and of dO
  static constexpr int DQ_BYTES = (2 + KS + VS) * TILE;
  static constexpr int DKV_BYTES = (2 + 2 * RS) * TILE;
};

struct Pipe {  // a ring of tiles
  unsigned long long full[4], empty[4];
};

__device__ __forceinline__ void pipe_init(Pipe &p, int slots) {
  for (int i = 0; i < slots; ++i) {
    mbar_init(&p.full[i], 1);
    mbar_init(&p.empty[i], 1);
  }
}

template <int DT, int DP>
__device__ __forceinline__ void load_rows(const CUtensorMap *m, unsigned char *dst,
                                          unsigned long long *bar, int h, int l, int b) {
  for (int c = 0; c < kPlanes<DT> * DP / 64; ++c)
    tma_load_4d(m, dst + c * BwdShape<DT, DP>::CHUNK, bar, c * 64, h, l, b);
}

// 16-bit types: delta is dO . O of the rounded O where rows see more frames than this (or a walk is split), and sum_j p_ij
// dP_ij, from a walk of its own over the same frames, where none of a CTA's rows does.  Error of dq over that of rounding
// the result alone, 41 and 150 rows: at 20 frames 1.6 from the rounded O and 1.4 from the sum, at 60 1.55 and 1.44, at 200
// 1.52 and 1.44, at 1,000 1.5 from the rounded O.  Time of the backward pass: 4 x 41 x 200, 8 heads of 64, 8.2 and 9.8 us;
// 16 x 1024 x 250, 16 heads on 4 of 128, 218 and 230; 8 x 1201 x 2000, 8 heads on 2 of 96, windows of 200, 77 and 83.
constexpr int kDeltaFrames = 256;

// The most frames that a row sees, as Hull does.
__device__ __forceinline__ void seen_note(int *seen, int warp, int2 range) {
  const int most = __reduce_max_sync(0xffffffffu, range.y - range.x);
  if ((threadIdx.x & 31) == 0) seen[warp] = most;
}
template <int WARPS> __device__ __forceinline__ int seen_of(const int *seen) {
  int most = seen[0];
#pragma unroll
  for (int i = 1; i < WARPS; ++i) most = max(most, seen[i]);
  return most;
}
// sum += p dP over the 64 frames from j0, of a row that sees those of `range`; neg: of p, -lse in base 2.  What a row that
// sees nothing gets may be anything.
__device__ __forceinline__ float2 sum_p_dp(unsigned (&x)[2][32], unsigned (&y)[2][32], int2 range, int j0, float c,
                                           float neg, float2 sum) {
  const bool alive = range.y > range.x;
  if (__any_sync(0xffffffffu, alive && (range.x > j0 || range.y < j0 + 64))) {
    const int lo = range.x - j0;
    const unsigned len = (unsigned)(range.y - range.x);
#pragma unroll
    for (int i = 0; i < 64; ++i)
      if ((unsigned)(i - lo) >= len) {
        x[i >> 5][i & 31] = 0xff800000u;
        y[i >> 5][i & 31] = 0;
      }
  }
  const float2 c2 = make_float2(c, c), n2 = make_float2(neg, neg);
#pragma unroll
  for (int i = 0; i < 64; i += 2) {
    const unsigned *xs = &x[i >> 5][i & 31], *ys = &y[i >> 5][i & 31];
    const float2 z = fma2(pair(xs[0], xs[1]), c2, n2);
    sum = fma2(make_float2(fast_exp2(z.x), fast_exp2(z.y)), pair(ys[0], ys[1]), sum);
  }
  return sum;
}

// ---- float16: the largest |v| ---------------------------------------------------------
// A CTA has a stretch of the frames of one (utterance, key head); 8 or 16 lanes a frame.  Bound by memory.
template <int L> __global__ void __launch_bounds__(256) attn_v_most_kernel(const __grid_constant__ BwdArgs f) {
  const AttnArgs &a = f.a;
  __shared__ float red[8];
  const int part = blockIdx.x % f.p.v_parts, hk = blockIdx.x / f.p.v_parts % a.Hkv;
  const long long b = blockIdx.x / f.p.v_parts / a.Hkv;
  const int2 mine = share_of(utt_lens(a, b).nk, part, f.p.v_parts);
  const int d0 = threadIdx.x % L * 8;
  const __half *v = static_cast<const __half *>(a.v) + b * a.sv.b + hk * a.sv.h + d0;
  constexpr int U = 4, F = 256 / L;  // loads in flight, frames at a time
  __half2 most = __float2half2_rn(0.0f);
  if (d0 < a.D)  // D is a multiple of 8
    for (int j0 = mine.x + threadIdx.x / L; j0 < mine.y; j0 += U * F) {
      uint4 x[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        x[u] = j0 + u * F < mine.y ? __ldg(reinterpret_cast<const uint4 *>(v + (j0 + u * F) * a.sv.l))
                                   : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const __half2 *h = reinterpret_cast<const __half2 *>(&x[u]);
#pragma unroll
        for (int k = 0; k < 4; ++k) most = __hmax2(most, __habs2(h[k]));
      }
    }
  const float2 m = __half22float2(most);
  const float top = warp_max(fmaxf(m.x, m.y));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = top;
  __syncthreads();
  if (threadIdx.x == 0) {
    float all = red[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) all = fmaxf(all, red[i]);
    f.v_most[blockIdx.x] = all;
  }
}
// sqrt(D) max |v|, by a whole warp; after the kernel above.
__device__ __forceinline__ float v_bound(const BwdArgs &f, long long b, int hk) {
  const int lane = threadIdx.x & 31;
  const float m = lane < f.p.v_parts ? f.v_most[(b * f.a.Hkv + hk) * f.p.v_parts + lane] : 0.0f;
  return warp_max(m) * sqrtf((float)f.a.D);
}

// ---- dq ---------------------------------------------------------------------------
struct DqShared {
  Pipe k, v;
  unsigned long long rows_full, scores, dp_free, ds_ready, done, tail_full, drained;
  unsigned tmem;
  int gave_up;
  Hull hull;
  int seen[8];
  float half[kRows], norm2[kRows];
  unsigned most[2];  // float16: bits of the rows' largest |dO|^2 and |delta|
};

template <int DT, int DP>
__global__ void __launch_bounds__(kThreads, 1)
    attn_dq_tc_kernel(const __grid_constant__ CUtensorMap qm, const __grid_constant__ CUtensorMap gm,
                      const __grid_constant__ CUtensorMap km, const __grid_constant__ CUtensorMap vm,
                      const __grid_constant__ CUtensorMap dqm, const __grid_constant__ BwdArgs f) {
  typedef BwdShape<DT, DP> S;
  typedef typename Elem<DT>::T E;
  extern __shared__ unsigned char raw[];
  __shared__ DqShared sh;
  unsigned char *tiles = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  unsigned char *q_tile = tiles, *g_tile = q_tile + S::TILE, *k_slots = g_tile + S::TILE,
                *v_slots = k_slots + S::KS * S::TILE;
  const AttnArgs &a = f.a;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  unsigned id = blockIdx.x;
  const int split = id % f.p.dq_splits;
  id /= f.p.dq_splits;
  const unsigned cta = id;
  const int tile = id % f.p.tiles;
  id /= f.p.tiles;
  const int pack = id % f.p.packs;
  const long long b = id / f.p.packs;
  const int P = f.p.P, per = kRows / P, i0 = tile * per, h0 = pack * P, hk = h0 / a.G;
  const Lens n = utt_lens(a, b);
  const bool some = i0 < n.nq && n.nk > 0;  // else no row sees a frame
  // frames [hull.x, hull.y) in tiles of 128 from hull.x; this CTA takes T tiles from `begin`
  int begin = 0, T = 0;
  int pre = 0, N = 0;  // steps that form delta (kDeltaFrames) before those that form dq: the same tiles; all steps
  // Frames past the utterance's end may hold anything, and 0 times NaN is NaN.  In the last tile of
  // k a warp of its own zeroes them (unless TMA did, past the tensor's end): the load then arrives
  // at tail_full, and that warp hands the tile on.
  bool cut = false;
  auto walk = [&](int2 hull) {
    const int2 steps = share_of((hull.y - hull.x + kRows - 1) / kRows, split, f.p.dq_splits);
    begin = hull.x + steps.x * kRows;
    T = steps.y - steps.x;
    cut = S::PLANES == 1 && T > 0 && n.nk < a.Lk && begin + T * kRows > n.nk;  // planes end in zeros
  };
  auto count = [&](int seen) {  // `seen`: frames that a row sees at the most
    pre = S::PLANES == 1 && f.p.dq_splits == 1 && seen <= kDeltaFrames ? T : 0;
    N = pre + T;
  };
  if (!a.windows && some) {
    walk(make_int2(0, n.nk));
    count(n.nk);
  }
  auto frame = [&](int s) { return begin + (s < pre ? s : s - pre) * kRows; };
  auto load_k = [&](int s) {
    const int slot = s % S::KS;
    unsigned long long *bar = cut && s == N - 1 ? &sh.tail_full : &sh.k.full[slot];
    arrive_expect_tx(bar, S::TILE);
    load_rows<DT, DP>(&km, k_slots + slot * S::TILE, bar, hk * f.k_h, frame(s), (int)b * f.k_b);
  };
  auto load_v = [&](int s) {
    const int slot = s % S::VS;
    arrive_expect_tx(&sh.v.full[slot], S::TILE);
    load_rows<DT, DP>(&vm, v_slots + slot * S::TILE, &sh.v.full[slot], hk * f.v_h, frame(s), (int)b * f.v_b);
  };
  const int group = warp >> 2, r = threadIdx.x & 127;
  const int row = i0 + r / P, head = h0 + r % P;
  int2 range = make_int2(0, 0);
  if (warp < 8) {
    range = row_range(a, b, row, n);
    if (a.windows) {
      hull_note(sh.hull, warp, range);
      seen_note(sh.seen, warp, range);
    }
  } else if (warp == 8 && lane == 0) {
    pipe_init(sh.k, S::KS);
    pipe_init(sh.v, S::VS);
    mbar_init(&sh.rows_full, 1);
    mbar_init(&sh.scores, 1);
    mbar_init(&sh.dp_free, 256);
    mbar_init(&sh.ds_ready, 256);
    mbar_init(&sh.done, 1);
    mbar_init(&sh.tail_full, 1);
    mbar_init(&sh.drained, 1);
    fence_mbar_init_cluster();
    sh.gave_up = 0;
    sh.most[0] = sh.most[1] = 0;
    if (some) {
      arrive_expect_tx(&sh.rows_full, 2 * S::TILE);
      load_rows<DT, DP>(&qm, q_tile, &sh.rows_full, h0 * f.q_h, i0, (int)b * f.q_b);
      load_rows<DT, DP>(&gm, g_tile, &sh.rows_full, h0 * f.go_h, i0, (int)b * f.go_b);
    }
    if (T > 0) {  // no windows: the walk is known
      load_k(0);
      load_v(0);
    }
  } else if (warp == 9) {
    tmem_alloc<512>(&sh.tmem);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const unsigned tmem = __shfl_sync(0xffffffffu, sh.tmem, 0);
  const Waiter wait{&sh.gave_up};
  if (a.windows) {
    walk(hull_of<8>(sh.hull));
    count(seen_of<8>(sh.seen));
  }
  constexpr unsigned kDp = 2 * kRows, kAcc = 3 * kRows;  // TMEM columns: S twice, dP, dQ,
  constexpr unsigned kThird = kAcc + 64;                 // the third plane of dS (float32)

  if (warp >= 8) {
    warpgroup_give_registers<kOtherRegs>();
    if (warp == 8 && lane == 0 && some && T == 0) wait(&sh.rows_full, 0);  // nobody else does
    if (warp == 8 && lane == 0 && T > 0) {
      bool ok = true;
      int s = 0;
      for (; ok && s < N; ++s) {
        if (s == 0 && !a.windows) continue;  // loaded above
        for (int x = 0; ok && x < 2; ++x)  // in the order of the products
          if ((x == 0) == (S::KS > 1)) {
            ok = wait(&sh.k.empty[s % S::KS], ((unsigned)(s / S::KS) & 1) ^ 1);
            if (ok) load_k(s);
          } else {
            ok = wait(&sh.v.empty[s % S::VS], ((unsigned)(s / S::VS) & 1) ^ 1);
            if (ok) load_v(s);
          }
      }
      if (!ok) {  // copies in flight land before the CTA ends
        Waiter::drain(&sh.rows_full, 0);
        for (int i = max(0, s - S::KS); i < s; ++i) {
          Waiter::drain(&sh.k.full[i % S::KS], (unsigned)(i / S::KS) & 1);
          Waiter::drain(&sh.v.full[i % S::VS], (unsigned)(i / S::VS) & 1);
        }
      }
    }
    if (warp == 10 && cut) {
      const int slot = (N - 1) % S::KS;
      if (__all_sync(0xffffffffu, wait(&sh.tail_full, 0)))
        zero_tail(k_slots + slot * S::TILE, S::CHUNKS, S::CHUNK, n.nk - frame(N - 1), kRows);
      if (lane == 0) mbar_arrive(&sh.k.full[slot]);
    }
    if (warp == 9 && T > 0 && elect_one()) {
      constexpr unsigned i_s = mma_desc<DT>(kRows, false), i_o = mma_desc<DT>(DP, true);
      const unsigned qa = smem_u32(q_tile), ga = smem_u32(g_tile), ka = smem_u32(k_slots),
                     va = smem_u32(v_slots);
      bool ok = wait(&sh.rows_full, 0);
      auto scores = [&](int s) {
        const int slot = s % S::KS;
        ok = ok && wait(&sh.k.full[slot], (unsigned)(s / S::KS) & 1);
        tc_fence_after();
        if (ok)
          mma_rows_planes<DT, DP>(tmem + (s & 1) * kRows, qa, ka + slot * S::TILE, S::CHUNK, S::PLANE, i_s);
      };
      auto grads = [&](int s) {  // dP of tile s
        const int slot = s % S::VS;
        ok = ok && wait(&sh.v.full[slot], (unsigned)(s / S::VS) & 1);
        tc_fence_after();
        if (!ok) return;
        mma_rows_planes<DT, DP>(tmem + kDp, ga, va + slot * S::TILE, S::CHUNK, S::PLANE, i_s);
        mma_commit(&sh.v.empty[slot]);
      };
      scores(0);
      grads(0);
      if (ok) mma_commit(&sh.scores);
      for (int s = 0; ok && s < N; ++s) {
        const int slot = s % S::KS;
        if (s + 1 < N) {
          if (S::KS > 1) scores(s + 1);
          ok = ok && wait(&sh.dp_free, s & 1);
          grads(s + 1);
          if (S::KS > 1 && ok) mma_commit(&sh.scores);
        }
        if (s < pre) {
          if (ok) mma_commit(&sh.k.empty[slot]);
          continue;
        }
        ok = ok && wait(&sh.ds_ready, (s - pre) & 1);
        tc_fence_after();
        if (!ok) break;
        const unsigned ds = tmem + (s & 1) * kRows, at = ka + slot * S::TILE;
#pragma unroll
        for (int g = 0; g < 2; ++g)  // the columns of each group
          mma_across_planes<DT, 64>(tmem + kAcc, ds + g * 64, ds + g * 64 + 32, tmem + kThird + g * 32,
                                    at + g * 64 * 128, S::CHUNK, S::PLANE, i_o,
                                    (S::PLANES == 1 && s > pre) || g > 0);
        mma_commit(&sh.k.empty[slot]);
        if (s + 1 == N) mma_commit(&sh.done);
        if (S::KS == 1 && s + 1 < N) {  // k's slot is free after these products only
          scores(s + 1);
          if (ok) mma_commit(&sh.scores);
        }
      }
      if (!ok) {
        mma_commit(&sh.drained);
        Waiter::drain(&sh.drained, 0);
      }
    }
  } else {
    warpgroup_take_registers<kWorkRegs>();
    // delta = dO . O of the row, half of the columns in each group; or sum p dP, half of the frames
    const bool real = row < n.nq, alive = range.y > range.x;
    const long long stat = (b * a.H + head) * a.Lq + row;
    float delta = 0.0f, lse2 = INFINITY, out_scale = a.scale;
    if (alive) lse2 = a.lse[stat] * kLog2e;  // else +inf: every weight is 0
    const float c = a.scale * kLog2e;
    const unsigned lanes = (unsigned)((warp & 3) * 32) << 16;
    bool ok = true;
    {
      const int d0 = group * (DP / 2), len = min(DP / 2, a.D - d0);
      float x = 0.0f, x2 = 0.0f;
      if (real)
        x = dot_rows<DT, DP / 2>(
            static_cast<const E *>(a.go) + b * a.sgo.b + row * a.sgo.l + head * a.sgo.h + d0,
            static_cast<const E *>(a.out) + b * a.so.b + row * a.so.l + head * a.so.h + d0, len,
            DT == kF16 ? &x2 : nullptr);
      if constexpr (S::PLANES == 1)
        if (pre > 0) {
          float2 sum = make_float2(0.0f, 0.0f);
          for (int s = 0; s < pre; ++s) {
            ok = wait(&sh.scores, s & 1);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            unsigned x[2][32], y[2][32];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              tmem_ld32(tmem + lanes + (s & 1) * kRows + group * 64 + i * 32, x[i]);
              tmem_ld32(tmem + lanes + kDp + group * 64 + i * 32, y[i]);
            }
            tmem_wait_ld();
            tc_fence_before();
            mbar_arrive(&sh.dp_free);
            sum = sum_p_dp(x, y, range, frame(s) + group * 64, c, -lse2, sum);
          }
          __syncwarp();
          x = alive ? sum.x + sum.y : 0.0f;
        }
      if (group == 1) {
        sh.half[r] = x;
        if (DT == kF16) sh.norm2[r] = x2;
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");
      const float y = sh.half[r], y2 = DT == kF16 ? sh.norm2[r] : 0.0f;
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (group == 0) {
        delta = x + y;
        sh.half[r] = delta;
        if (row < a.Lq && split == 0) a.delta[stat] = delta;
        if (DT == kF16) {
          sh.norm2[r] = x2 + y2;
          const unsigned m0 = __reduce_max_sync(0xffffffffu, __float_as_uint(x2 + y2)),
                         m1 = __reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(delta)));
          if (lane == 0) {  // the order does not matter to a maximum
            atomicMax(&sh.most[0], m0);
            atomicMax(&sh.most[1], m1);
          }
        }
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");
      delta = sh.half[r];
      if constexpr (DT == kF16) {
        if (threadIdx.x == 0 && split == 0)
          f.row_most[cta] = make_float2(sqrtf(__uint_as_float(sh.most[0])), __uint_as_float(sh.most[1]));
        wait_for_predecessor();  // v's largest
        const int e = ds_shift(fmaf(sqrtf(sh.norm2[r]), v_bound(f, b, hk), fabsf(delta)));
        lse2 -= (float)e;  // 2^e p
        out_scale *= power_of_2(-e);
      }
    }
    // float32: this thread's 32 columns of dQ, to which each tile's part is added
    float acc[32];
#pragma unroll
    for (int k = 0; k < 32; ++k) acc[k] = 0.0f;
    auto add_tile = [&]() {
      if constexpr (S::PLANES == 3) {
        unsigned o[32];
        tmem_ld32(tmem + lanes + kAcc + group * 32, o);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 32; ++k) acc[k] += __uint_as_float(o[k]);
      }
    };
    for (int s = pre; s < N; ++s) {
      ok = ok && wait(&sh.scores, s & 1);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      if (s > 0) add_tile();  // dQ of the tile before was issued before these scores
      const unsigned s_col = tmem + lanes + (s & 1) * kRows + group * 64,
                     p_col = tmem + lanes + kDp + group * 64;
      constexpr int H = S::PLANES == 3 ? 2 : 1;  // float32: half of the columns at a time, for the registers' sake
      unsigned x[2][32], y[2 / H][32];
      tmem_ld32(s_col, x[0]);
      tmem_ld32(s_col + 32, x[1]);
      const int j0 = frame(s) + group * 64, lo = range.x - j0;
      const unsigned len = (unsigned)(range.y - range.x);
      const float2 c2 = make_float2(c, c), l2 = make_float2(-lse2, -lse2),
                   d2 = make_float2(-delta, -delta);
      const bool part = __any_sync(0xffffffffu, alive && (range.x > j0 || range.y < j0 + 64));
#pragma unroll
      for (int h = 0; h < H; ++h) {
        constexpr int N = 64 / H;
#pragma unroll
        for (int i = 0; i < N / 32; ++i) tmem_ld32(p_col + h * N + i * 32, y[i]);
        tmem_wait_ld();
        if (h == H - 1) {
          tc_fence_before();
          mbar_arrive(&sh.dp_free);
        }
        if (part) {
          // frames that the row does not see: s = -inf weighs 0, and dP may be anything
#pragma unroll
          for (int i = 0; i < N; ++i)
            if ((unsigned)(h * N + i - lo) >= len) {
              x[(h * N + i) >> 5][i & 31] = 0xff800000u;
              y[i >> 5][i & 31] = 0;
            }
        }
        unsigned out[S::PLANES][N / 2];
#pragma unroll
        for (int i = 0; i < N; i += 2) {
          const unsigned *xs = &x[(h * N + i) >> 5][i & 31], *ys = &y[i >> 5][i & 31];
          const float2 z = fma2(pair(xs[0], xs[1]), c2, l2);
          const float2 p = make_float2(fast_exp2(z.x), fast_exp2(z.y));
          const float2 ds = mul2(p, add2(pair(ys[0], ys[1]), d2));
          unsigned planes[S::PLANES];
          split2<DT>(ds, planes);
#pragma unroll
          for (int k = 0; k < S::PLANES; ++k) out[k][i / 2] = planes[k];
        }
        if constexpr (S::PLANES == 3) {
          tmem_st16(s_col + h * 16, out[0]);
          tmem_st16(s_col + 32 + h * 16, out[1]);
          tmem_st16(tmem + lanes + kThird + group * 32 + h * 16, out[2]);
        } else {
          tmem_st32(s_col, out[0]);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&sh.ds_ready);
    }
    if (T > 0 && ok) ok = wait(&sh.done, 0);
    if (T == 0 && some) ok = wait(&sh.rows_full, 0);  // the tile's memory is used below
    __syncwarp();
    tc_fence_after();
    const bool bad = !ok || *reinterpret_cast<volatile int *>(&sh.gave_up);
    if (T > 0) add_tile();
#pragma unroll
    for (int i = 0; i < DP / 64; ++i) {
      const int d0 = (group * (DP / 64) + i) * 32;
      unsigned o[32];
      if (S::PLANES == 1 && T > 0) {
        tmem_ld32(tmem + lanes + kAcc + d0, o);
        tmem_wait_ld();
      }
      float v[32];
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        const float x = S::PLANES == 3 ? acc[k] : __uint_as_float(o[k]);
        v[k] = bad ? NAN : T > 0 && alive ? x * out_scale : 0.0f;
      }
      if (f.p.dq_splits == 1)
        stage32<DT>(q_tile, S::CHUNK, r, d0, v);  // every product with q is done
      else if (row < a.Lq)
        store_columns(f.part + (((long long)split * f.p.tiles * f.p.packs * a.B + cta) * DP + d0) * kRows + r,
                      kRows, v);
      __syncwarp();
    }
    if (f.p.dq_splits == 1) {
      fence_async_shared();
      named_barrier<256>(1);
      if (threadIdx.x == 0) {
        constexpr int kColumns = DT == kF32 ? 32 : 64;  // of a chunk
        for (int ch = 0; ch < DP / kColumns; ++ch)
          if (ch * kColumns < a.D)
            tma_store_4d(&dqm, q_tile + ch * S::CHUNK, ch * kColumns, h0 * f.dq_h, i0, (int)b * f.dq_b);
        tma_store_commit();
        tma_store_wait_read();
      }
      __syncwarp();
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 9) tmem_free<512>(tmem);
}

// ---- dk and dv ----------------------------------------------------------------------
constexpr int kStats = 4;  // row tiles whose statistics are held

struct DkvShared {
  Pipe q, g;
  unsigned long long frames_full, s_full, p_ready, dp_full, ds_ready, stat_full[kStats], stat_empty[kStats],
      done, q_tail[4], g_tail[4], drained;
  unsigned tmem;
  int gave_up;
  unsigned char active[kTileBits];  // row tiles with a query that sees these frames
  int cut[kStats];                  // whether some row of the tile sees only part of them
  float ds_in, ds_out;              // float16: 2^(e - 15), 2^-e
  __align__(16) float lse2[kStats][kRows], delta[kStats][kRows];  // of the rows, both negated
  __align__(16) int lo[kStats][kRows], len[kStats][kRows];
};

template <int DT, int DP>
__global__ void __launch_bounds__(kThreads, 1)
    attn_dkv_tc_kernel(const __grid_constant__ CUtensorMap qm, const __grid_constant__ CUtensorMap gm,
                       const __grid_constant__ CUtensorMap km, const __grid_constant__ CUtensorMap vm,
                       const __grid_constant__ CUtensorMap dkm, const __grid_constant__ CUtensorMap dvm,
                       const __grid_constant__ BwdArgs f) {
  typedef BwdShape<DT, DP> S;
  extern __shared__ unsigned char raw[];
  __shared__ DkvShared sh;
  unsigned char *tiles = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  unsigned char *k_tile = tiles, *v_tile = k_tile + S::TILE, *q_slots = v_tile + S::TILE,
                *g_slots = q_slots + S::RS * S::TILE;
  const AttnArgs &a = f.a;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  unsigned id = blockIdx.x;
  const int split = id % f.p.dkv_splits;
  id /= f.p.dkv_splits;
  const unsigned cta = id;
  const int j0 = (int)(id % f.p.f_tiles) * kRows;
  id /= f.p.f_tiles;
  const int hk = id % a.Hkv;
  const long long b = id / a.Hkv;
  const int P = f.p.P, per = kRows / P;
  const Lens n = utt_lens(a, b);
  // the walk: packs of the group x row tiles with queries, skipping those that see none of these
  // frames; this CTA takes the steps [t0, t1) of it
  const int row_tiles = j0 < n.nk ? (n.nq + per - 1) / per : 0;
  const int2 steps = share_of((a.G / P) * row_tiles, split, f.p.dkv_splits);
  const int t0 = steps.x, t1 = steps.y;
  if (warp == 8) {
    if (lane == 0) {
      pipe_init(sh.q, S::RS);
      pipe_init(sh.g, S::RS);
      mbar_init(&sh.frames_full, 1);
      mbar_init(&sh.s_full, 1);
      mbar_init(&sh.p_ready, 256);
      mbar_init(&sh.dp_full, 1);
      mbar_init(&sh.ds_ready, 256);
      for (int i = 0; i < kStats; ++i) {
        mbar_init(&sh.stat_full[i], 32);
        mbar_init(&sh.stat_empty[i], 256);
      }
      for (int i = 0; i < S::RS; ++i) {
        mbar_init(&sh.q_tail[i], 1);
        mbar_init(&sh.g_tail[i], 1);
      }
      mbar_init(&sh.done, 1);
      mbar_init(&sh.drained, 1);
      fence_mbar_init_cluster();
      sh.gave_up = 0;
      if (t1 > t0) {
        arrive_expect_tx(&sh.frames_full, 2 * S::TILE);
        load_rows<DT, DP>(&km, k_tile, &sh.frames_full, hk * f.k_h, j0, (int)b * f.k_b);
        load_rows<DT, DP>(&vm, v_tile, &sh.frames_full, hk * f.v_h, j0, (int)b * f.v_b);
      }
    }
  } else if (warp == 9) {
    tmem_alloc<512>(&sh.tmem);
  } else if (a.windows) {  // ten warps
    for (int t = warp < 8 ? warp : warp - 2; t < min(row_tiles, kTileBits); t += 10) {
      bool sees = false;
      for (int i = t * per + lane; i < min((t + 1) * per, n.nq); i += 32) {
        const int2 w = row_range(a, b, i, n);
        sees |= w.x < j0 + kRows && w.y > j0;
      }
      sees = __any_sync(0xffffffffu, sees);
      if (lane == 0) sh.active[t] = sees;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const unsigned tmem = __shfl_sync(0xffffffffu, sh.tmem, 0);
  const Waiter wait{&sh.gave_up};
  auto skip = [&](int t) {
    const int rt = t % row_tiles;
    return a.windows && rt < kTileBits && !sh.active[rt];
  };
  auto next = [&](int t) {  // the first step at or after t
    while (t < t1 && skip(t)) ++t;
    return t;
  };
  const int start = next(t0);
  const bool any = start < t1;
  // Rows past the utterance's end may hold anything, and 0 times NaN is NaN.  In the last row tile of
  // each walk over the rows a warp of its own zeroes them (unless TMA did, past the tensor's end):
  // the loads then arrive at q_tail and g_tail, and that warp hands the tiles on.
  auto cut = [&](int t) {
    return S::PLANES == 1 && n.nq < a.Lq && (t % row_tiles + 1) * per > n.nq;  // planes end in zeros
  };
  constexpr unsigned kDp = kRows, kDv = 2 * kRows, kDk = 2 * kRows + DP;
  constexpr unsigned kThird = kDk + DP;  // the third planes of P and of dS (float32)

  if (warp >= 8) {
    warpgroup_give_registers<kOtherRegs>();
    if (warp == 8 && lane == 0 && t1 > t0 && !any) wait(&sh.frames_full, 0);  // nobody else does
    if (warp == 8 && lane == 0 && any) {
      bool ok = true;
      int s = 0;
      for (int t = start; ok && t < t1; t = next(t + 1), ++s) {
        const int slot = s % S::RS, l = t % row_tiles * per, h = hk * a.G + t / row_tiles * P;
        const unsigned turn = ((unsigned)(s / S::RS) & 1) ^ 1;
        for (int x = 0; ok && x < 2; ++x)  // in the order of the products
          if ((x == 0) == (S::RS > 1)) {
            ok = wait(&sh.q.empty[slot], turn);
            if (!ok) break;
            unsigned long long *bar = cut(t) ? &sh.q_tail[slot] : &sh.q.full[slot];
            arrive_expect_tx(bar, S::TILE);
            load_rows<DT, DP>(&qm, q_slots + slot * S::TILE, bar, h * f.q_h, l, (int)b * f.q_b);
          } else {
            ok = wait(&sh.g.empty[slot], turn);
            if (!ok) break;
            unsigned long long *bar = cut(t) ? &sh.g_tail[slot] : &sh.g.full[slot];
            arrive_expect_tx(bar, S::TILE);
            load_rows<DT, DP>(&gm, g_slots + slot * S::TILE, bar, h * f.go_h, l, (int)b * f.go_b);
          }
      }
      if (!ok) {
        Waiter::drain(&sh.frames_full, 0);
        for (int i = max(0, s - S::RS); i < s; ++i) {
          Waiter::drain(&sh.q.full[i % S::RS], (unsigned)(i / S::RS) & 1);
          Waiter::drain(&sh.g.full[i % S::RS], (unsigned)(i / S::RS) & 1);
        }
      }
    }
    if (warp == 11 && any) {
      int s = 0;
      unsigned turns = 0;  // bit: parity of the slot's next cut tile
      for (int t = start; t < t1; t = next(t + 1), ++s) {
        if (!cut(t)) continue;
        const int slot = s % S::RS, valid = (n.nq - t % row_tiles * per) * P;
        if (!__all_sync(0xffffffffu, wait(&sh.q_tail[slot], turns >> slot & 1))) break;
        zero_tail(q_slots + slot * S::TILE, S::CHUNKS, S::CHUNK, valid, kRows);
        if (lane == 0) mbar_arrive(&sh.q.full[slot]);
        if (!__all_sync(0xffffffffu, wait(&sh.g_tail[slot], turns >> slot & 1))) break;
        zero_tail(g_slots + slot * S::TILE, S::CHUNKS, S::CHUNK, valid, kRows);
        if (lane == 0) mbar_arrive(&sh.g.full[slot]);
        turns ^= 1u << slot;
      }
    }
    if (warp == 9 && any && elect_one()) {
      constexpr unsigned i_s = mma_desc<DT>(kRows, false), i_o = mma_desc<DT>(DP, true);
      const unsigned ka = smem_u32(k_tile), va = smem_u32(v_tile), qa = smem_u32(q_slots),
                     ga = smem_u32(g_slots);
      bool ok = wait(&sh.frames_full, 0);
      auto scores = [&](int s) {  // S^T
        const int slot = s % S::RS;
        ok = ok && wait(&sh.q.full[slot], (unsigned)(s / S::RS) & 1);
        tc_fence_after();
        if (!ok) return;
        mma_rows_planes<DT, DP>(tmem, ka, qa + slot * S::TILE, S::CHUNK, S::PLANE, i_s);
        mma_commit(&sh.s_full);
      };
      auto grads = [&](int s) {  // dP^T
        const int slot = s % S::RS;
        ok = ok && wait(&sh.g.full[slot], (unsigned)(s / S::RS) & 1);
        tc_fence_after();
        if (!ok) return;
        mma_rows_planes<DT, DP>(tmem + kDp, va, ga + slot * S::TILE, S::CHUNK, S::PLANE, i_s);
        mma_commit(&sh.dp_full);
      };
      int t = start;
      scores(0);
      grads(0);
      for (int s = 0; ok && t < t1; ++s) {
        const int after = next(t + 1), slot = s % S::RS;
        ok = wait(&sh.p_ready, s & 1);
        tc_fence_after();
        if (!ok) break;
        const unsigned g_at = ga + slot * S::TILE, q_at = qa + slot * S::TILE;
#pragma unroll
        for (int g = 0; g < 2; ++g)  // dV += P^T dO, the columns of each group
          mma_across_planes<DT, 64>(tmem + kDv, tmem + g * 64, tmem + g * 64 + 32, tmem + kThird + g * 32,
                                    g_at + g * 64 * 128, S::CHUNK, S::PLANE, i_o,
                                    (S::PLANES == 1 && s > 0) || g > 0);
        mma_commit(&sh.g.empty[slot]);
        if (S::RS > 1 && after < t1) scores(s + 1);
        ok = ok && wait(&sh.ds_ready, s & 1);
        tc_fence_after();
        if (!ok) break;
#pragma unroll
        for (int g = 0; g < 2; ++g)  // dK += dS^T Q
          mma_across_planes<DT, 64>(tmem + kDk, tmem + kDp + g * 64, tmem + kDp + g * 64 + 32,
                                    tmem + kThird + 64 + g * 32, q_at + g * 64 * 128, S::CHUNK, S::PLANE, i_o,
                                    (S::PLANES == 1 && s > 0) || g > 0);
        mma_commit(&sh.q.empty[slot]);
        if (after >= t1) mma_commit(&sh.done);
        if (after < t1) grads(s + 1);
        if (S::RS == 1 && after < t1) scores(s + 1);  // q's slot is free after dK's products only
        t = after;
      }
      if (!ok) {
        mma_commit(&sh.drained);
        Waiter::drain(&sh.drained, 0);
      }
    }
    if (warp == 10) wait_for_predecessor();  // delta is the dq kernel's; and nobody overtakes it
    if (warp == 10 && any) {  // the rows' statistics
      float ds_in = kUnshift<DT>;
      if constexpr (DT == kF16) {
        const int tiles = a.G / P * f.p.tiles;
        const float2 *most = f.row_most + (b * a.Hkv + hk) * tiles;
        float g = 0.0f, d = 0.0f;
        bool finite = true;  // a maximum passes over NaN
        for (int t = lane; t < tiles; t += 32) {
          const float2 m = most[t];
          g = fmaxf(g, m.x);
          d = fmaxf(d, m.y);
          finite = finite && m.x + m.y < INFINITY;
        }
        const int e = ds_shift(fmaf(warp_max(g), v_bound(f, b, hk), warp_max(d)));
        ds_in *= __all_sync(0xffffffffu, finite) ? power_of_2(e) : 1.0f;
        if (lane == 0) {
          sh.ds_in = ds_in;
          sh.ds_out = kUnshift<DT> / ds_in;
        }
      }
      int s = 0;
      for (int t = start; t < t1; t = next(t + 1), ++s) {
        const int buf = s % kStats, i0 = t % row_tiles * per, h0 = hk * a.G + t / row_tiles * P;
        const bool ok = wait(&sh.stat_empty[buf], ((unsigned)(s / kStats) & 1) ^ 1);
        if (!__all_sync(0xffffffffu, ok)) break;
        bool cut = false;
        constexpr int X = kRows / 32;
        int2 w[X];
        float l2[X], dl[X];
#pragma unroll
        for (int x = 0; x < X; ++x) w[x] = row_range(a, b, i0 + (x * 32 + lane) / P, n);
#pragma unroll
        for (int x = 0; x < X; ++x) {  // every load in flight at once
          const int r = x * 32 + lane, i = min(i0 + r / P, a.Lq - 1);
          const long long at = (b * a.H + h0 + r % P) * a.Lq + i;
          l2[x] = __ldg(a.lse + at);
          dl[x] = a.delta[at];  // not the read-only path: it was written since this kernel was launched
        }
#pragma unroll
        for (int x = 0; x < X; ++x) {
          const int r = x * 32 + lane;
          const bool sees = w[x].y > w[x].x;  // else every weight is 0
          cut |= sees && (w[x].x > j0 || w[x].y < min(j0 + kRows, n.nk));
          sh.lse2[buf][r] = sees ? kShift<DT> - l2[x] * kLog2e : -INFINITY;
          sh.delta[buf][r] = sees ? -dl[x] * ds_in : 0.0f;
          sh.lo[buf][r] = w[x].x;
          sh.len[buf][r] = w[x].y - w[x].x;
        }
        cut = __any_sync(0xffffffffu, cut);
        if (lane == 0) sh.cut[buf] = cut;
        __syncwarp();
        mbar_arrive(&sh.stat_full[buf]);
      }
    }
  } else {
    warpgroup_take_registers<kWorkRegs>();
    const int group = warp >> 2, j = j0 + (threadIdx.x & 127);
    const unsigned lanes = (unsigned)((warp & 3) * 32) << 16;
    const unsigned s_col = tmem + lanes + group * 64, d_col = s_col + kDp;
    const float c = a.scale * kLog2e;
    const bool past = __any_sync(0xffffffffu, j >= n.nk);
    // float32: this thread's 32 columns of dV and of dK, to which each tile's part is added
    float acc[2][32];
#pragma unroll
    for (int k = 0; k < 64; ++k) acc[k / 32][k % 32] = 0.0f;
    auto add_tile = [&]() {
      if constexpr (S::PLANES == 3) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          unsigned o[32];
          tmem_ld32(tmem + lanes + (i ? kDk : kDv) + group * 32, o);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 32; ++k) acc[i][k] += __uint_as_float(o[k]);
        }
      }
    };
    bool ok = true;
    int s = 0;
    if (any)
      for (int t = start; t < t1; t = next(t + 1), ++s) {
        const int buf = s % kStats;
        ok = wait(&sh.stat_full[buf], (unsigned)(s / kStats) & 1) && wait(&sh.s_full, s & 1);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
        if (s > 0) add_tile();  // the products of the tile before were issued before these scores
        constexpr int H = S::PLANES == 3 ? 2 : 1, N = 64 / H;  // float32: half of the columns at a time
        unsigned x[2][32];
        tmem_ld32(s_col, x[0]);
        tmem_ld32(s_col + 32, x[1]);
        tmem_wait_ld();
        const float *lse2 = sh.lse2[buf] + group * 64, *delta = sh.delta[buf] + group * 64;
        const float ds_in = DT == kF16 ? sh.ds_in : 1.0f;
        const float2 c2 = make_float2(c, c);
#pragma unroll
        for (int i = 0; i < 64; i += 4) {
          const float4 l = *reinterpret_cast<const float4 *>(lse2 + i);
          unsigned *v = &x[i >> 5][i & 31];
          const float2 z0 = fma2(pair(v[0], v[1]), c2, make_float2(l.x, l.y)),
                       z1 = fma2(pair(v[2], v[3]), c2, make_float2(l.z, l.w));
          v[0] = __float_as_uint(fast_exp2(z0.x));
          v[1] = __float_as_uint(fast_exp2(z0.y));
          v[2] = __float_as_uint(fast_exp2(z1.x));
          v[3] = __float_as_uint(fast_exp2(z1.y));
        }
        if (past) {
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if (j >= n.nk) x[i >> 5][i & 31] = 0;
        }
        if (sh.cut[buf]) {
          const int *lo = sh.lo[buf] + group * 64, *len = sh.len[buf] + group * 64;
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if ((unsigned)(j - lo[i]) >= (unsigned)len[i]) x[i >> 5][i & 31] = 0;
        }
#pragma unroll
        for (int h = 0; h < H; ++h) {
          unsigned out[S::PLANES][N / 2];
#pragma unroll
          for (int i = 0; i < N; i += 2) {
            const unsigned *xs = &x[(h * N + i) >> 5][i & 31];
            unsigned planes[S::PLANES];
            split2<DT>(pair(xs[0], xs[1]), planes);
#pragma unroll
            for (int k = 0; k < S::PLANES; ++k) out[k][i / 2] = planes[k];
          }
          if constexpr (S::PLANES == 3) {
            tmem_st16(s_col + h * 16, out[0]);
            tmem_st16(s_col + 32 + h * 16, out[1]);
            tmem_st16(tmem + lanes + kThird + group * 32 + h * 16, out[2]);
          } else {
            tmem_st32(s_col, out[0]);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&sh.p_ready);
        ok = wait(&sh.dp_full, s & 1);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
        unsigned y[2][32];
        tmem_ld32(d_col, y[0]);
        tmem_ld32(d_col + 32, y[1]);
        tmem_wait_ld();
#pragma unroll
        for (int h = 0; h < H; ++h) {
          unsigned out[S::PLANES][N / 2];
#pragma unroll
          for (int i = h * N; i < h * N + N; i += 4) {
            const float4 dl = *reinterpret_cast<const float4 *>(delta + i);
            const float2 un = make_float2(ds_in, ds_in);
            const unsigned *p = &x[i >> 5][i & 31], *g = &y[i >> 5][i & 31];
            const float2 d0 = make_float2(dl.x, dl.y), d1 = make_float2(dl.z, dl.w);
            const float2 g0 = pair(g[0], g[1]), g1 = pair(g[2], g[3]);
            const float2 v0 = mul2(pair(p[0], p[1]), DT == kF16 ? fma2(g0, un, d0) : add2(g0, d0)),
                         v1 = mul2(pair(p[2], p[3]), DT == kF16 ? fma2(g1, un, d1) : add2(g1, d1));
            unsigned p0[S::PLANES], p1[S::PLANES];
            split2<DT>(v0, p0);
            split2<DT>(v1, p1);
#pragma unroll
            for (int k = 0; k < S::PLANES; ++k) {
              out[k][(i - h * N) / 2] = p0[k];
              out[k][(i - h * N) / 2 + 1] = p1[k];
            }
          }
          if constexpr (S::PLANES == 3) {
            tmem_st16(d_col + h * 16, out[0]);
            tmem_st16(d_col + 32 + h * 16, out[1]);
            tmem_st16(tmem + lanes + kThird + 64 + group * 32 + h * 16, out[2]);
          } else {
            tmem_st32(d_col, out[0]);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&sh.ds_ready);
        mbar_arrive(&sh.stat_empty[buf]);
      }
    if (any && ok) ok = wait(&sh.done, 0);
    if (!any && t1 > t0) ok = wait(&sh.frames_full, 0);  // the tiles' memory is used below
    __syncwarp();
    tc_fence_after();
    const bool bad = !ok || *reinterpret_cast<volatile int *>(&sh.gave_up);
    const bool keep = j < n.nk;  // frames past the end: their lanes hold no sums
    const long long ctas = (long long)f.p.f_tiles * a.Hkv * a.B;
    // 32 columns of dv (which 0) or dk (1), through the tile that no product needs any more
    auto put = [&](int which, int d0, const float (&v)[32]) {
      if (f.p.dkv_splits == 1)
        stage32<DT>(which ? k_tile : v_tile, S::CHUNK, threadIdx.x & 127, d0, v);
      else if (j < a.Lk)
        store_columns(f.part + (((which ? ctas * f.p.dkv_splits : 0) + split * ctas + cta) * DP + d0) * kRows +
                          (threadIdx.x & 127), kRows, v);
      __syncwarp();
    };
    if constexpr (S::PLANES == 3) {  // each group has half of the columns of both
      if (any) add_tile();
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float v[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) v[k] = bad ? NAN : any && keep ? acc[i][k] * (i ? a.scale : 1.0f) : 0.0f;
        put(i, group * 32, v);
      }
    } else {  // group 0 has dv, group 1 dk
      const float scale = !group ? kUnshift<DT> : DT == kF16 && any ? a.scale * sh.ds_out : a.scale;
#pragma unroll
      for (int i = 0; i < DP / 32; ++i) {
        unsigned o[32];
        if (any) {
          tmem_ld32(tmem + lanes + (group ? kDk : kDv) + i * 32, o);
          tmem_wait_ld();
        }
        float v[32];
#pragma unroll
        for (int k = 0; k < 32; ++k)
          v[k] = bad ? NAN : any && keep ? __uint_as_float(o[k]) * scale : 0.0f;
        put(group, i * 32, v);
      }
    }
    if (f.p.dkv_splits == 1) {
      fence_async_shared();
      named_barrier<256>(1);
      if ((threadIdx.x & 127) == 0) {
        constexpr int kColumns = DT == kF32 ? 32 : 64;  // of a chunk
        for (int ch = 0; ch < DP / kColumns; ++ch)
          if (ch * kColumns < a.D)
            tma_store_4d(group ? &dkm : &dvm, (group ? k_tile : v_tile) + ch * S::CHUNK, ch * kColumns,
                         hk * (group ? f.dk_h : f.dv_h), j0, (int)b * (group ? f.dk_b : f.dv_b));
        tma_store_commit();
        tma_store_wait_read();
      }
      __syncwarp();
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 9) tmem_free<512>(tmem);
}

// ---- dq, dk and dv of one row tile -----------------------------------------------------
// Threads: two warpgroups of elementwise work (thread = row, each group half of the frames), one that
// stores dk and dv tiles (thread = frame), four warps: loads, products, tails, one idle.
constexpr int kOneThreads = 512;
constexpr int kOneLaunchRegs = 128;  // 4 x 128 = 2 x 160 + 112 + 80
constexpr int kOneWorkRegs = 160, kOneStoreRegs = 112, kOneOtherRegs = 80;

struct OneShape {
  static constexpr int TILE = kRows * 128;            // 64 columns
  static constexpr int KS = 3, VS = 2;                // slots of k and of v
  static constexpr int PDS = 2 * TILE;                // P or dS: 128 x 128; P once, dS twice
  static constexpr int BYTES = (2 + KS + VS) * TILE + 3 * PDS;
};

struct OneShared {
  Pipe k, v;
  unsigned long long rows_in, rows_full, out_full, sp_full, sp_free, pds_ready, p_free, ds_free[2], dkv_full,
      dkv_free, dq_done[2], done, tail_full, drained;
  unsigned tmem;
  int gave_up;
  Hull hull;
  int seen[8];
  float half[kRows], norm2[kRows];
  unsigned most[2];  // float16: bits of the rows' largest |dO|^2 and |delta|
  float ds_out;      // float16: 2^-e
};

template <int DT>
__global__ void __launch_bounds__(kOneThreads, 1)
    attn_one_tc_kernel(const __grid_constant__ CUtensorMap qm, const __grid_constant__ CUtensorMap gm,
                       const __grid_constant__ CUtensorMap km, const __grid_constant__ CUtensorMap vm,
                       const __grid_constant__ CUtensorMap om, const __grid_constant__ CUtensorMap dqm,
                       const __grid_constant__ BwdArgs f) {
  constexpr int DP = 64;
  typedef OneShape S;
  typedef typename Elem<DT>::T E;
  extern __shared__ unsigned char raw[];
  __shared__ OneShared sh;
  unsigned char *tiles = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  unsigned char *q_tile = tiles, *g_tile = q_tile + S::TILE, *k_slots = g_tile + S::TILE,
                *v_slots = k_slots + S::KS * S::TILE, *p_tile = v_slots + S::VS * S::TILE,
                *ds_tiles = p_tile + S::PDS;
  const AttnArgs &a = f.a;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int split = blockIdx.x % f.p.dq_splits;
  const unsigned cta = blockIdx.x / f.p.dq_splits;  // = b * Hkv + hk
  const int hk = cta % a.Hkv, h0 = hk * a.G;
  const long long b = cta / a.Hkv;
  const int P = f.p.P;
  const Lens n = utt_lens(a, b);
  const int group = warp >> 2, r = threadIdx.x & 127, row = r / P, head = h0 + r % P;
  int2 range = make_int2(0, 0);
  // Rows and frames past the utterance's ends may hold anything, and 0 times NaN is NaN: a warp of its own
  // zeroes them in the tiles of q and dO and in the last tile of k before handing these on (unless TMA
  // did, past the tensor's ends).
  const bool some = n.nq > 0 && n.nk > 0, cut_rows = n.nq < a.Lq;
  // this CTA's frame tiles [t0, t1); those that a row sees are [ta, tb)
  const int2 mine = share_of(f.p.f_tiles, split, f.p.dq_splits);
  const int t0 = mine.x, t1 = mine.y;
  int ta = t1, tb = t1, T = 0;
  int pre = 0, N = 0;  // steps that form delta (kDeltaFrames) before those that form the gradients: the same tiles; all steps
  bool cut = false;
  auto walk = [&](int2 hull) {
    ta = hull.y > hull.x ? max(t0, hull.x / kRows) : t1;
    tb = min(t1, (hull.y + kRows - 1) / kRows);
    T = max(0, tb - ta);
    cut = T > 0 && n.nk < a.Lk && (ta + T) * kRows > n.nk;
  };
  auto count = [&](int seen) {  // `seen`: frames that a row sees at the most
    pre = f.p.dq_splits == 1 && seen <= kDeltaFrames ? T : 0;
    N = pre + T;
  };
  if (!a.windows && some) {
    walk(make_int2(0, n.nk));
    count(n.nk);
  }
  auto frame = [&](int s) { return (ta + (s < pre ? s : s - pre)) * kRows; };
  auto load_k = [&](int s) {
    const int slot = s % S::KS;
    unsigned long long *bar = cut && s == N - 1 ? &sh.tail_full : &sh.k.full[slot];
    arrive_expect_tx(bar, S::TILE);
    tma_load_4d(&km, k_slots + slot * S::TILE, bar, 0, hk * f.k_h, frame(s), (int)b * f.k_b);
  };
  auto load_v = [&](int s) {
    const int slot = s % S::VS;
    arrive_expect_tx(&sh.v.full[slot], S::TILE);
    tma_load_4d(&vm, v_slots + slot * S::TILE, &sh.v.full[slot], 0, hk * f.v_h, frame(s), (int)b * f.v_b);
  };
  if (group < 2) {
    range = row_range(a, b, row, n);
    if (a.windows) {
      hull_note(sh.hull, warp, range);
      seen_note(sh.seen, warp, range);
    }
  } else if (warp == 12 && lane == 0) {
    pipe_init(sh.k, S::KS);
    pipe_init(sh.v, S::VS);
    mbar_init(&sh.rows_in, 1);
    mbar_init(&sh.rows_full, 1);
    mbar_init(&sh.out_full, 1);
    mbar_init(&sh.sp_full, 1);
    mbar_init(&sh.sp_free, 256);
    mbar_init(&sh.pds_ready, 256);
    mbar_init(&sh.p_free, 1);
    mbar_init(&sh.ds_free[0], 128);
    mbar_init(&sh.ds_free[1], 128);
    mbar_init(&sh.dkv_full, 1);
    mbar_init(&sh.dkv_free, 128);
    mbar_init(&sh.dq_done[0], 1);
    mbar_init(&sh.dq_done[1], 1);
    mbar_init(&sh.done, 1);
    mbar_init(&sh.tail_full, 1);
    mbar_init(&sh.drained, 1);
    fence_mbar_init_cluster();
    sh.gave_up = 0;
    sh.most[0] = sh.most[1] = 0;
    if (some) {
      unsigned long long *in = cut_rows ? &sh.rows_in : &sh.rows_full;
      arrive_expect_tx(in, 2 * S::TILE);
      arrive_expect_tx(&sh.out_full, S::TILE);
      tma_load_4d(&om, p_tile, &sh.out_full, 0, h0 * f.out_h, 0, (int)b * f.out_b);  // P comes later
      tma_load_4d(&qm, q_tile, in, 0, h0 * f.q_h, 0, (int)b * f.q_b);
      tma_load_4d(&gm, g_tile, in, 0, h0 * f.go_h, 0, (int)b * f.go_b);
    }
    if (T > 0) {  // no windows: the walk is known
      load_k(0);
      load_v(0);
    }
  } else if (warp == 13) {
    tmem_alloc<512>(&sh.tmem);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const unsigned tmem = __shfl_sync(0xffffffffu, sh.tmem, 0);
  const Waiter wait{&sh.gave_up};
  if (a.windows) {
    walk(hull_of<8>(sh.hull));
    count(seen_of<8>(sh.seen));
  }
  constexpr unsigned kDp = kRows, kDv = 2 * kRows, kDk = kDv + DP, kAcc = kDk + DP;
  unsigned long long *rows = cut_rows ? &sh.rows_in : &sh.rows_full;
  if (group == 3) {
    warpgroup_give_registers<kOneOtherRegs>();
    if (warp == 12 && lane == 0 && some && T == 0) wait(rows, 0);  // nobody else does
    if (warp == 12 && lane == 0 && T > 0) {
      bool ok = true;
      int s = 0;
      for (; ok && s < N; ++s) {
        if (s == 0 && !a.windows) continue;  // loaded above
        ok = wait(&sh.k.empty[s % S::KS], ((unsigned)(s / S::KS) & 1) ^ 1);
        if (!ok) break;
        load_k(s);
        ok = wait(&sh.v.empty[s % S::VS], ((unsigned)(s / S::VS) & 1) ^ 1);
        if (!ok) {
          ++s;
          break;
        }
        load_v(s);
      }
      if (!ok) {  // copies in flight land before the CTA ends
        Waiter::drain(rows, 0);
        for (int i = max(0, s - S::KS); i < s; ++i) {
          Waiter::drain(&sh.k.full[i % S::KS], (unsigned)(i / S::KS) & 1);
          Waiter::drain(&sh.v.full[i % S::VS], (unsigned)(i / S::VS) & 1);
        }
      }
    }
    if (warp == 14 && T > 0) {
      if (cut_rows) {
        if (__all_sync(0xffffffffu, wait(&sh.rows_in, 0))) {
          zero_tail(q_tile, 1, S::TILE, n.nq * P, kRows);
          zero_tail(g_tile, 1, S::TILE, n.nq * P, kRows);
        }
        if (lane == 0) mbar_arrive(&sh.rows_full);
      }
      if (cut) {
        const int slot = (N - 1) % S::KS;
        if (__all_sync(0xffffffffu, wait(&sh.tail_full, 0)))
          zero_tail(k_slots + slot * S::TILE, 1, S::TILE, n.nk - frame(N - 1), kRows);
        if (lane == 0) mbar_arrive(&sh.k.full[slot]);
      }
    }
    if (warp == 13 && T > 0 && elect_one()) {
      constexpr unsigned i_s = mma_desc<DT>(kRows, false), i_t = mma_desc<DT>(DP, true, true),
                         i_o = mma_desc<DT>(DP, true);
      const unsigned qa = smem_u32(q_tile), ga = smem_u32(g_tile), ka = smem_u32(k_slots),
                     va = smem_u32(v_slots), pa = smem_u32(p_tile);
      bool ok = wait(&sh.rows_full, 0);
      auto scores = [&](int s) {  // S and dP
        const int ks = s % S::KS, vs = s % S::VS;
        ok = ok && wait(&sh.k.full[ks], (unsigned)(s / S::KS) & 1) &&
             wait(&sh.v.full[vs], (unsigned)(s / S::VS) & 1);
        tc_fence_after();
        if (!ok) return;
        mma_rows<DP>(tmem, qa, S::TILE, ka + ks * S::TILE, S::TILE, i_s, false);
        mma_rows<DP>(tmem + kDp, ga, S::TILE, va + vs * S::TILE, S::TILE, i_s, false);
        mma_commit(&sh.sp_full);
        mma_commit(&sh.v.empty[vs]);
      };
      scores(0);
      for (int x = 0; ok && x < N; ++x) {
        const int slot = x % S::KS, s = x - pre;
        const unsigned da = smem_u32(ds_tiles) + (s & 1) * S::PDS;
        if (x + 1 < N) {
          ok = wait(&sh.sp_free, x & 1);
          scores(x + 1);
        }
        if (s < 0) {
          if (ok) mma_commit(&sh.k.empty[slot]);
          continue;
        }
        ok = ok && wait(&sh.pds_ready, s & 1);
        ok = ok && wait(&sh.dkv_free, (s & 1) ^ 1);
        tc_fence_after();
        if (!ok) break;
#pragma unroll
        for (int k = 0; k < kRows / 16; ++k)  // dV = P^T dO
          mma_ss(tmem + kDv, desc_mn_major(pa + k * 2048, S::TILE), desc_mn_major(ga + k * 2048, S::TILE),
                 i_t, k > 0);
        mma_commit(&sh.p_free);
#pragma unroll
        for (int k = 0; k < kRows / 16; ++k)  // dK = dS^T Q
          mma_ss(tmem + kDk, desc_mn_major(da + k * 2048, S::TILE), desc_mn_major(qa + k * 2048, S::TILE),
                 i_t, k > 0);
        mma_commit(&sh.dkv_full);
#pragma unroll
        for (int k = 0; k < kRows / 16; ++k)  // dQ += dS K
          mma_ss(tmem + kAcc, desc_k_major(da + (k / 4) * S::TILE + (k % 4) * 32),
                 desc_mn_major(ka + slot * S::TILE + k * 2048, S::TILE), i_o, s > 0 || k > 0);
        mma_commit(&sh.k.empty[slot]);
        mma_commit(&sh.dq_done[s & 1]);
        if (s + 1 == T) mma_commit(&sh.done);
      }
      if (!ok) {
        mma_commit(&sh.drained);
        Waiter::drain(&sh.drained, 0);
      }
    }
  } else if (group == 2) {
    warpgroup_give_registers<kOneStoreRegs>();
    const unsigned lanes = (unsigned)((warp & 3) * 32) << 16;
    for (int t = t0; t < t1; ++t) {
      const int j = t * kRows + r, s = t - ta;
      if (t < ta || t >= tb) {  // no row sees these frames
        for (int x = r; x < kRows * 8; x += 128) {
          const int jz = t * kRows + x / 8, d = x % 8 * 8;
          if (jz >= a.Lk || d >= a.D) continue;
          typedef unsigned short Raw;
          *reinterpret_cast<uint4 *>(static_cast<Raw *>(a.dv) + b * a.sdv.b + jz * a.sdv.l + hk * a.sdv.h + d) =
              make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4 *>(static_cast<Raw *>(a.dk) + b * a.sdk.b + jz * a.sdk.l + hk * a.sdk.h + d) =
              make_uint4(0, 0, 0, 0);
        }
        continue;
      }
      bool ok = wait(&sh.dkv_full, s & 1);
      ok = __all_sync(0xffffffffu, ok) && !*reinterpret_cast<volatile int *>(&sh.gave_up);
      __syncwarp();
      tc_fence_after();
      unsigned packed[2][32];  // dv and dk of the frame
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        unsigned o[32];
        tmem_ld32(tmem + lanes + kDv + i * 32, o);
        tmem_wait_ld();
        const float f_out = i < 2 ? kUnshift<DT> : DT == kF16 ? a.scale * sh.ds_out : a.scale;
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
          const float2 v = mul2(pair(o[k], o[k + 1]), make_float2(f_out, f_out));
          packed[i / 2][(i & 1) * 16 + k / 2] = pack2<DT>(v.x, v.y);
        }
      }
      if (!ok || j >= n.nk) {
        const unsigned fill = ok ? 0u : pack2<DT>(NAN, NAN);
#pragma unroll
        for (int k = 0; k < 64; ++k) packed[k / 32][k % 32] = fill;
      }
      __syncwarp();
      tc_fence_before();
      mbar_arrive(&sh.dkv_free);
      // the tiles go out through the memory of this step's dS, once the products have read it
      wait(&sh.dq_done[s & 1], (unsigned)(s >> 1) & 1);
      __syncwarp();
      unsigned char *out_tile = ds_tiles + (s & 1) * S::PDS;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k)
          *reinterpret_cast<uint4 *>(out_tile + i * S::TILE + r * 128 + (k ^ (r & 7)) * 16) =
              make_uint4(packed[i][4 * k], packed[i][4 * k + 1], packed[i][4 * k + 2], packed[i][4 * k + 3]);
      named_barrier<128>(2);
      // 8 threads a row: whole lines.  Plain stores free this memory once it is in registers; a TMA store
      // frees it once it has been read.
      uint4 piece[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int x = i * 128 + r, jr = x % 1024 / 8, k = x % 8;
        piece[i] = *reinterpret_cast<const uint4 *>(out_tile + (x / 1024) * S::TILE + jr * 128 +
                                                    (k ^ (jr & 7)) * 16);
      }
      mbar_arrive(&sh.ds_free[s & 1]);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int x = i * 128 + r, jr = t * kRows + x % 1024 / 8, d = x % 8 * 8;
        const bool is_k = x >= 1024;
        const Strides &st = is_k ? a.sdk : a.sdv;
        if (jr < a.Lk && d < a.D)
          *reinterpret_cast<uint4 *>(static_cast<unsigned short *>(is_k ? a.dk : a.dv) + b * st.b + jr * st.l +
                                     hk * st.h + d) = piece[i];
      }
    }
    tc_fence_before();
  } else {
    warpgroup_take_registers<kOneWorkRegs>();
    const bool real = row < n.nq, alive = range.y > range.x;
    const long long stat = (b * a.H + head) * a.Lq + row;
    const float c = a.scale * kLog2e;
    const unsigned lanes = (unsigned)((warp & 3) * 32) << 16;
    const unsigned s_col = tmem + lanes + group * 64, d_col = s_col + kDp;
    bool ok = true;
    float delta, lse2 = -INFINITY;  // both negated
    float ds_in = kUnshift<DT>, out_scale = a.scale;
    {
      // dO . O: this group's half of the columns, from the tiles of dO and out; or sum p dP, half of the frames
      float x = 0.0f, x2 = 0.0f;
      if (some && wait(&sh.out_full, 0) && wait(rows, 0) && real) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int at = r * 128 + ((group * 4 + k) ^ (r & 7)) * 16;
          const uint4 gv = *reinterpret_cast<const uint4 *>(g_tile + at),
                      ov = *reinterpret_cast<const uint4 *>(p_tile + at);
          const E *ge = reinterpret_cast<const E *>(&gv), *oe = reinterpret_cast<const E *>(&ov);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float g = Elem<DT>::to_float(ge[i]);
            x = fmaf(g, Elem<DT>::to_float(oe[i]), x);
            if (DT == kF16) x2 = fmaf(g, g, x2);
          }
        }
      }
      __syncwarp();
      if (alive) lse2 = kShift<DT> - a.lse[stat] * kLog2e;
      if (pre > 0) {
        float2 sum = make_float2(0.0f, 0.0f);
        for (int s = 0; s < pre; ++s) {
          ok = wait(&sh.sp_full, s & 1);
          if (!__all_sync(0xffffffffu, ok)) break;
          tc_fence_after();
          unsigned x[2][32], y[2][32];
          tmem_ld32(s_col, x[0]);
          tmem_ld32(s_col + 32, x[1]);
          tmem_ld32(d_col, y[0]);
          tmem_ld32(d_col + 32, y[1]);
          tmem_wait_ld();
          tc_fence_before();
          mbar_arrive(&sh.sp_free);
          sum = sum_p_dp(x, y, range, frame(s) + group * 64, c, lse2 - kShift<DT>, sum);
        }
        __syncwarp();
        x = alive ? sum.x + sum.y : 0.0f;
      }
      if (group == 1) {
        sh.half[r] = x;
        if (DT == kF16) sh.norm2[r] = x2;
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");
      const float y = sh.half[r], y2 = DT == kF16 ? sh.norm2[r] : 0.0f;
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (group == 0) {
        sh.half[r] = x + y;
        if (DT == kF16) {
          const unsigned m0 = __reduce_max_sync(0xffffffffu, __float_as_uint(x2 + y2)),
                         m1 = __reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(x + y)));
          if (lane == 0) {  // the order does not matter to a maximum
            atomicMax(&sh.most[0], m0);
            atomicMax(&sh.most[1], m1);
          }
        }
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if constexpr (DT == kF16) {
        wait_for_predecessor();  // v's largest
        const int e = ds_shift(fmaf(sqrtf(__uint_as_float(sh.most[0])), v_bound(f, b, hk),
                                    __uint_as_float(sh.most[1])));
        ds_in *= power_of_2(e);
        out_scale *= power_of_2(-e);
        if (threadIdx.x == 0) sh.ds_out = power_of_2(-e);  // read after the first tile's products
      }
      delta = -sh.half[r] * ds_in;
    }
    const float2 c2 = make_float2(c, c), l2 = make_float2(lse2, lse2), d2 = make_float2(delta, delta),
                 un = make_float2(ds_in, ds_in);
    for (int s = 0; s < T; ++s) {
      ok = ok && wait(&sh.sp_full, (pre + s) & 1);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      unsigned x[2][32], y[2][32];
      tmem_ld32(s_col, x[0]);
      tmem_ld32(s_col + 32, x[1]);
      tmem_ld32(d_col, y[0]);
      tmem_ld32(d_col + 32, y[1]);
      tmem_wait_ld();
      tc_fence_before();
      mbar_arrive(&sh.sp_free);
      const int j0 = frame(pre + s) + group * 64;
      if (__any_sync(0xffffffffu, alive && (range.x > j0 || range.y < j0 + 64))) {
        // frames that the row does not see: s = -inf weighs 0, and dP may be anything
        const int lo = range.x - j0;
        const unsigned len = (unsigned)(range.y - range.x);
#pragma unroll
        for (int i = 0; i < 64; ++i)
          if ((unsigned)(i - lo) >= len) {
            x[i >> 5][i & 31] = 0xff800000u;
            y[i >> 5][i & 31] = 0;
          }
      }
      // what was in this P and dS has been read
      ok = wait(&sh.p_free, (s & 1) ^ 1) && wait(&sh.ds_free[s & 1], ((unsigned)(s >> 1) & 1) ^ 1);
      unsigned char *p_row = p_tile + group * S::TILE + r * 128,
                    *ds_row = ds_tiles + (s & 1) * S::PDS + group * S::TILE + r * 128;
      if (!__all_sync(0xffffffffu, ok)) break;
#pragma unroll
      for (int q = 0; q < 8; ++q) {  // 8 frames: 16 bytes of P and of dS, swizzled as TMA would
        unsigned pw[4], dw[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int i = q * 8 + k * 2;
          const float2 z = fma2(pair(x[i >> 5][i & 31], x[i >> 5][(i + 1) & 31]), c2, l2);
          const float2 p = make_float2(fast_exp2(z.x), fast_exp2(z.y));
          const float2 g = pair(y[i >> 5][i & 31], y[i >> 5][(i + 1) & 31]);
          const float2 ds = mul2(p, DT == kF16 ? fma2(g, un, d2) : add2(g, d2));
          pw[k] = pack2<DT>(p.x, p.y);
          dw[k] = pack2<DT>(ds.x, ds.y);
        }
        const int at = (q ^ (r & 7)) * 16;
        *reinterpret_cast<uint4 *>(p_row + at) = make_uint4(pw[0], pw[1], pw[2], pw[3]);
        *reinterpret_cast<uint4 *>(ds_row + at) = make_uint4(dw[0], dw[1], dw[2], dw[3]);
      }
      fence_async_shared();
      tc_fence_before();
      mbar_arrive(&sh.pds_ready);
    }
    if (T > 0 && ok) ok = wait(&sh.done, 0);
    if (T == 0 && some) ok = wait(rows, 0);  // the tile's memory is used below
    __syncwarp();
    tc_fence_after();
    const bool bad = !ok || *reinterpret_cast<volatile int *>(&sh.gave_up);
    unsigned o[32];
    if (T > 0) {
      tmem_ld32(tmem + lanes + kAcc + group * 32, o);
      tmem_wait_ld();
    }
    float v[32];
    // A row that sees nothing weighs 0 everywhere, but its dP meets frames past the utterance's end, whose v may hold
    // anything, and 0 times that need not be 0.  Its dS then spoils its own dQ, set here, and the dK of those frames, which
    // the storing warps set.
#pragma unroll
    for (int k = 0; k < 32; ++k) v[k] = bad ? NAN : T > 0 && alive ? __uint_as_float(o[k]) * out_scale : 0.0f;
    if (f.p.dq_splits == 1) {
      stage32<DT>(q_tile, S::TILE, r, group * 32, v);  // every product with q is done
      fence_async_shared();
      named_barrier<256>(1);
      if (threadIdx.x == 0) {
        tma_store_4d(&dqm, q_tile, 0, h0 * f.dq_h, 0, (int)b * f.dq_b);
        tma_store_commit();
        tma_store_wait_read();
      }
    } else if (row < a.Lq) {
      store_columns(f.part + (((long long)split * a.Hkv * a.B + cta) * DP + group * 32) * kRows + r, kRows, v);
    }
    __syncwarp();
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 13) tmem_free<512>(tmem);
}

// Adds the splits of a sum for 32 rows and 32 columns, in order.  The partial sums lie column by column; the
// results leave row by row through shared memory.  `which0` + blockIdx.y: 0 dq, 1 dv, 2 dk.
template <int DT, int DP>
__global__ void __launch_bounds__(256) attn_add_kernel(const __grid_constant__ BwdArgs f, int which0) {
  const AttnArgs &a = f.a;
  __shared__ float out[32][33];
  const int which = which0 + blockIdx.y, r = threadIdx.x & 31, part = threadIdx.x >> 5;
  const unsigned d0 = blockIdx.x % (DP / 32) * 32, block = blockIdx.x / (DP / 32);
  const unsigned cta = block / (kRows / 32), r0 = block % (kRows / 32) * 32;
  const long long ctas = gridDim.x / (DP / 32) / (kRows / 32);
  const int splits = which == 0 ? f.p.dq_splits : f.p.dkv_splits;
  void *to;
  long long base;         // of the CTA's first head in the result
  int first, count, per;  // position of row r0, positions of the tensor, rows of a position
  long long sl, sh;
  if (which == 0) {
    const unsigned bp = cta / f.p.tiles;
    first = (int)(cta % f.p.tiles) * (kRows / f.p.P) + r0 / f.p.P;
    per = f.p.P;
    count = a.Lq;
    to = a.dq;
    base = bp / f.p.packs * a.sdq.b + bp % f.p.packs * f.p.P * a.sdq.h;
    sl = a.sdq.l;
    sh = a.sdq.h;
  } else {
    const Strides &s = which == 2 ? a.sdk : a.sdv;
    const unsigned bh = cta / f.p.f_tiles;
    first = (int)(cta % f.p.f_tiles) * kRows + r0;
    per = 1;
    count = a.Lk;
    to = which == 2 ? a.dk : a.dv;
    base = bh / a.Hkv * s.b + bh % a.Hkv * s.h;
    sl = s.l;
    sh = 0;
  }
  if (first >= count) return;
  const bool real = first + r / per < count;
  wait_for_predecessor();
  const float *p = f.part + (((which == 2 ? ctas * splits : 0) + cta) * DP + d0 + part) * kRows + r0 + r;
  const long long next = ctas * (kRows * DP);
  constexpr int U = 8;  // splits whose loads are in flight
  float o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int s0 = 0; s0 < splits; s0 += U) {
    float v[U][4];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[u][i] = real && s0 + u < splits ? p[(s0 + u) * next + i * 8 * kRows] : 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] += v[u][i];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) out[r][part + i * 8] = o[i];
  __syncthreads();
  if (threadIdx.x < 128) {
    const int rr = threadIdx.x / 4, d = threadIdx.x % 4 * 8, at = first + rr / per;
    const float *x = &out[rr][d];
    if (at >= count || d0 + d >= a.D) {
    } else if constexpr (DT == kF32) {
      float *dst = static_cast<float *>(to) + base + at * sl + rr % per * sh + d0 + d;
      *reinterpret_cast<float4 *>(dst) = make_float4(x[0], x[1], x[2], x[3]);
      if (d0 + d + 4 < a.D) *reinterpret_cast<float4 *>(dst + 4) = make_float4(x[4], x[5], x[6], x[7]);
    } else {
      unsigned short *dst = static_cast<unsigned short *>(to) + base + at * sl + rr % per * sh + d0 + d;
      *reinterpret_cast<uint4 *>(dst) = make_uint4(pack2<DT>(x[0], x[1]), pack2<DT>(x[2], x[3]),
                                                   pack2<DT>(x[4], x[5]), pack2<DT>(x[6], x[7]));
    }
  }
}

BwdPlan plan(long long B, long long Lq, long long Lk, int H, int Hkv, int D, int dtype) {
  BwdPlan p;
  const int G = H / Hkv;
  p.P = attn_row_pack(G);
  p.packs = H / p.P;
  p.tiles = (int)((Lq * p.P + kRows - 1) / kRows);
  p.f_tiles = (int)((Lk + kRows - 1) / kRows);
  // split a walk while CTAs leave SMs idle and each keeps three steps
  auto splits = [](long long ctas, long long steps) {
    long long s = ctas > 0 ? kSMs / ctas : 1;
    if (s > steps / 3) s = steps / 3;
    return (int)(s < 1 ? 1 : s > 64 ? 64 : s);
  };
  p.dq_splits = splits(B * p.packs * p.tiles, p.f_tiles);
  p.one = dtype != kF32 && D <= 64 && p.P == G && p.tiles == 1;
  p.dkv_splits = p.one ? 1 : splits(B * Hkv * p.f_tiles, (long long)(G / p.P) * p.tiles);
  // v's reader: eight CTAs an SM, 64 frames each at the least
  p.v_parts = 0;
  if (dtype == kF16) {
    const long long parts = B * Hkv > 0 ? std::min<long long>({8 * kSMs / (B * Hkv), (Lk + 63) / 64, kVParts}) : 1;
    p.v_parts = (int)std::max<long long>(parts, 1);
  }
  return p;
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

struct Maps {
  TensorMap q, go, k, v, out, dq, dk, dv;
};

// The first kernel of a call; float16: after the one that reads v.
template <int DT, typename... P, typename... A>
cudaError_t launch_after_v_most(void (*kernel)(P...), const BwdArgs &f, unsigned blocks, unsigned threads, size_t smem,
                                cudaStream_t stream, const A &...args) {
  if constexpr (DT == kF16) {
    const unsigned parts = (unsigned)(f.a.B * f.a.Hkv * f.p.v_parts);
    if (f.a.D <= 64)
      attn_v_most_kernel<8><<<parts, 256, 0, stream>>>(f);
    else
      attn_v_most_kernel<16><<<parts, 256, 0, stream>>>(f);
    const cudaError_t e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_follower(kernel, dim3(blocks), threads, smem, stream, args...);
  } else {
    kernel<<<blocks, threads, smem, stream>>>(args...);
    return cudaGetLastError();
  }
}

template <int DT> cudaError_t launch_one(const BwdArgs &f, const Maps &m, cudaStream_t stream) {
  const cudaError_t e = prepare_tc_kernel(reinterpret_cast<const void *>(attn_one_tc_kernel<DT>),
                                          OneShape::BYTES + 1024, kOneLaunchRegs);
  if (e != cudaSuccess) return e;
  const unsigned ctas = (unsigned)(f.a.B * f.a.Hkv);
  const cudaError_t e1 = launch_after_v_most<DT>(attn_one_tc_kernel<DT>, f, ctas * f.p.dq_splits, kOneThreads,
                                                 OneShape::BYTES + 1024, stream, m.q.map, m.go.map, m.k.map, m.v.map,
                                                 m.out.map, m.dq.map, f);
  if (e1 == cudaSuccess && f.p.dq_splits > 1)
    return launch_follower(attn_add_kernel<DT, 64>, dim3(ctas * (kRows / 32) * 2, 1), 256, 0, stream,
                           f, 0);
  return e1;
}

template <int DT, int DP>
cudaError_t launch(const BwdArgs &f, const Maps &m, cudaStream_t stream) {
  typedef BwdShape<DT, DP> S;
  const AttnArgs &a = f.a;
  const long long rows = a.B * f.p.packs * f.p.tiles, frames = a.B * a.Hkv * f.p.f_tiles;
  const unsigned per_tile = (kRows / 32) * (DP / 32);  // blocks of the adding kernel
  cudaError_t e = prepare_tc_kernel(reinterpret_cast<const void *>(attn_dq_tc_kernel<DT, DP>),
                                    S::DQ_BYTES + 1024, kLaunchRegs);
  if (e != cudaSuccess) return e;
  e = launch_after_v_most<DT>(attn_dq_tc_kernel<DT, DP>, f, (unsigned)(rows * f.p.dq_splits), kThreads,
                              S::DQ_BYTES + 1024, stream, m.q.map, m.go.map, m.k.map, m.v.map, m.dq.map, f);
  if (e == cudaSuccess && f.p.dq_splits > 1)
    e = launch_follower(attn_add_kernel<DT, DP>, dim3((unsigned)rows * per_tile, 1), 256, 0, stream, f, 0);
  if (e == cudaSuccess)
    e = prepare_tc_kernel(reinterpret_cast<const void *>(attn_dkv_tc_kernel<DT, DP>),
                          S::DKV_BYTES + 1024, kLaunchRegs);
  if (e == cudaSuccess)
    e = launch_follower(attn_dkv_tc_kernel<DT, DP>, dim3((unsigned)(frames * f.p.dkv_splits)), kThreads,
                        S::DKV_BYTES + 1024, stream, m.q.map, m.go.map, m.k.map, m.v.map, m.dk.map,
                        m.dv.map, f);
  if (e == cudaSuccess && f.p.dkv_splits > 1)
    e = launch_follower(attn_add_kernel<DT, DP>, dim3((unsigned)frames * per_tile, 2), 256, 0, stream, f, 1);
  return e;
}

// The workspace: planes of q, dO, k, v (float32), then the partial sums of splits, then the sizes that dS's shift is
// chosen by (float16).
struct BwdSpace {
  size_t q, go, k, v, part, v_most, row_most, total;
};
BwdSpace space(const BwdPlan &p, long long B, long long Lq, long long Lk, int H, int Hkv, int D, int dtype) {
  BwdSpace s = {};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align256(bytes);
    return here;
  };
  if (dtype == kF32) {
    s.q = take(plane_bytes(B, Lq, H));
    s.go = take(plane_bytes(B, Lq, H));
    s.k = take(plane_bytes(B, Lk, Hkv));
    s.v = take(plane_bytes(B, Lk, Hkv));
  }
  const size_t tile = (size_t)kRows * (D <= 64 ? 64 : 128) * 4;
  const size_t dq = p.dq_splits > 1 ? tile * B * p.packs * p.tiles * p.dq_splits : 0;
  const size_t dkv = p.dkv_splits > 1 ? 2 * tile * B * Hkv * p.f_tiles * p.dkv_splits : 0;
  s.part = take(dq > dkv ? dq : dkv);
  s.v_most = take((size_t)B * Hkv * p.v_parts * 4);
  s.row_most = take(dtype == kF16 ? (size_t)B * p.packs * p.tiles * 8 : 0);
  s.total = at;
  return s;
}

}  // namespace

size_t attn_bwd_tc_workspace(long long B, long long Lq, long long Lk, int H, int Hkv, int D, int dtype) {
  return space(plan(B, Lq, Lk, H, Hkv, D, dtype), B, Lq, Lk, H, Hkv, D, dtype).total;
}

bool attn_bwd_tc_fits(const AttnArgs &a, int dtype) {
  auto fits = [&](const void *p, const Strides &s, long long L, int H) {
    return map_fits(dtype, p, a.B, L, H, a.D, s.b, s.l, s.h);
  };
  if (!attn_tc_takes(dtype, a.Lq, a.Lk, a.G, a.D, true)) return false;
  // out and dO are read in vectors of 16 bytes, the results are stored by TMA
  if (!fits(a.out, a.so, a.Lq, a.H) || !fits(a.go, a.sgo, a.Lq, a.H) || !fits(a.dq, a.sdq, a.Lq, a.H) ||
      !fits(a.dk, a.sdk, a.Lk, a.Hkv) || !fits(a.dv, a.sdv, a.Lk, a.Hkv))
    return false;
  return dtype == kF32 || ((attn_row_pack(a.G) == 1 || (a.sq.h != 0 && a.sgo.h != 0)) &&
                           fits(a.q, a.sq, a.Lq, a.H) && fits(a.k, a.sk, a.Lk, a.Hkv) &&
                           fits(a.v, a.sv, a.Lk, a.Hkv));
}

cudaError_t launch_attn_bwd_tc(const AttnArgs &a, int dtype, void *workspace, cudaStream_t stream) {
  BwdArgs f = {};
  f.a = a;
  f.p = plan(a.B, a.Lq, a.Lk, a.H, a.Hkv, a.D, dtype);
  const BwdSpace at = space(f.p, a.B, a.Lq, a.Lk, a.H, a.Hkv, a.D, dtype);
  char *ws = static_cast<char *>(workspace);
  f.part = reinterpret_cast<float *>(ws + at.part);
  f.v_most = reinterpret_cast<float *>(ws + at.v_most);
  f.row_most = reinterpret_cast<float2 *>(ws + at.row_most);
  Maps m;
  const int per = kRows / f.p.P;
  bool ok = !f.p.one ||
            encode_map(&m.out, a.out, dtype, a.B, a.Lq, a.H, a.D, a.so.b, a.so.l, a.so.h, f.p.P, per);
  ok = ok && encode_map(&m.dq, a.dq, dtype, a.B, a.Lq, a.H, a.D, a.sdq.b, a.sdq.l, a.sdq.h, f.p.P, per) &&
            encode_map(&m.dk, a.dk, dtype, a.B, a.Lk, a.Hkv, a.D, a.sdk.b, a.sdk.l, a.sdk.h, 1, kRows) &&
            encode_map(&m.dv, a.dv, dtype, a.B, a.Lk, a.Hkv, a.D, a.sdv.b, a.sdv.l, a.sdv.h, 1, kRows);
  if (dtype == kF32) {
    auto source = [&](const void *p, const Strides &s, const long long *lens, int L, int H, size_t to) {
      return PlaneSource{static_cast<const float *>(p), s.b, s.l, s.h, lens, L, H,
                         reinterpret_cast<unsigned short *>(ws + to)};
    };
    const PlaneSource t[4] = {source(a.q, a.sq, a.q_lens, a.Lq, a.H, at.q),
                              source(a.go, a.sgo, a.q_lens, a.Lq, a.H, at.go),
                              source(a.k, a.sk, a.k_lens, a.Lk, a.Hkv, at.k),
                              source(a.v, a.sv, a.k_lens, a.Lk, a.Hkv, at.v)};
    const cudaError_t e = launch_planes(t, 4, a.B, a.D, stream);
    if (e != cudaSuccess) return e;
    ok = ok && encode_planes(&m.q, t[0].dst, a.B, a.Lq, a.H, 1, f.p.P, per) &&
         encode_planes(&m.go, t[1].dst, a.B, a.Lq, a.H, 1, f.p.P, per) &&
         encode_planes(&m.k, t[2].dst, a.B, a.Lk, a.Hkv, 1, 1, kRows) &&
         encode_planes(&m.v, t[3].dst, a.B, a.Lk, a.Hkv, 1, 1, kRows);
  } else {
    ok = ok && encode_map(&m.q, a.q, dtype, a.B, a.Lq, a.H, a.D, a.sq.b, a.sq.l, a.sq.h, f.p.P, per) &&
         encode_map(&m.go, a.go, dtype, a.B, a.Lq, a.H, a.D, a.sgo.b, a.sgo.l, a.sgo.h, f.p.P, per) &&
         encode_map(&m.k, a.k, dtype, a.B, a.Lk, a.Hkv, a.D, a.sk.b, a.sk.l, a.sk.h, 1, kRows) &&
         encode_map(&m.v, a.v, dtype, a.B, a.Lk, a.Hkv, a.D, a.sv.b, a.sv.l, a.sv.h, 1, kRows);
  }
  if (!ok) return cudaErrorInvalidValue;
  f.out_b = f.p.one ? m.out.b_mul : 0;
  f.out_h = f.p.one ? m.out.h_mul : 0;
  f.q_b = m.q.b_mul;
  f.q_h = m.q.h_mul;
  f.go_b = m.go.b_mul;
  f.go_h = m.go.h_mul;
  f.k_b = m.k.b_mul;
  f.k_h = m.k.h_mul;
  f.v_b = m.v.b_mul;
  f.v_h = m.v.h_mul;
  f.dq_b = m.dq.b_mul;
  f.dq_h = m.dq.h_mul;
  f.dk_b = m.dk.b_mul;
  f.dk_h = m.dk.h_mul;
  f.dv_b = m.dv.b_mul;
  f.dv_h = m.dv.h_mul;
  if (dtype == kF32) return launch<kF32, 64>(f, m, stream);
  if (f.p.one) return dtype == kF16 ? launch_one<kF16>(f, m, stream) : launch_one<kBF16>(f, m, stream);
  if (dtype == kF16)
    return a.D <= 64 ? launch<kF16, 64>(f, m, stream) : launch<kF16, 128>(f, m, stream);
  return a.D <= 64 ? launch<kBF16, 64>(f, m, stream) : launch<kBF16, 128>(f, m, stream);
}

}  // namespace tdt
