// tdt_attn_planes.cu -- cross attention of float32 heads of 65 to 128 elements on the tensor cores, forward and
// backward: operands as three bfloat16 planes, six products for one (tdt_tc.cuh).
//
// A tile of 128 rows in planes takes 96 KB, so nothing stays in shared memory: halves of tiles (64 columns,
// 48 KB) pass through a ring of four, in the order in which the products want them.  A CTA holds the sums of
// a tile of 128 "own" rows and walks over the tiles of the other side:
//   forward  own: queries    walks frames    S = Q K^T,                    O  += P V
//   dq       own: queries    walks frames    S = Q K^T,   dP = dO V^T,     dQ += dS K
//   dk       own: frames     walks queries   S^T = K Q^T, dP^T = V dO^T,   dK += dS^T Q
//   dv       own: frames     walks queries   S^T = K Q^T,                  dV += P^T dO
// (dk and dv in one launch).  Eight products where seven would do if dk and dv shared S^T: their sums
// together are more registers than a thread has.  Two warpgroups, thread = own row, each half of the
// walk's 128 columns and half of the sum's; tiles' sums are formed in TMEM and added to float32 registers,
// since TMEM sums are cut, not rounded.  The elementwise work and the products of a CTA take turns.
//
// Few CTAs: a cluster of up to 8 shares the walk; the sums are added over distributed shared memory, in order.
//
// Bound by the loads and the waits between products and elementwise work: a step of dq has 4.6 us of products at
// the tensor cores' rate and loads 480 KB.  4 x 1201 x 2000, 8 heads of 128: forward 343 us, backward
// 1,166 us (91 TFLOP/s of float32 products).  2 x 801 x 982 ragged, 8 heads of 128, forward: 62 us with the
// call, 251 on the CUDA cores.  1 x 300 x 2000, 4 heads on 1 of 96, windows of 300: 23 us and 60 us.
// Products go plane by plane, the small ones of both halves first: TMEM's cut sums are then small while there are
// many of them (error 4 to 7e-7 of the results; half by half 1 to 2e-6, and a tenth faster).
#include <cooperative_groups.h>

#include "tdt_attn_common.cuh"
#include "tdt_tc.cuh"

namespace tdt {
namespace {

namespace cg = cooperative_groups;

constexpr int kRows = 128;
constexpr int kThreads = 384;
constexpr int kLaunchRegs = 168;  // 3 warpgroups x 168 = 2 x 208 + 88
constexpr int kWorkRegs = 208, kOtherRegs = 88;
constexpr int kTileBits = 4096;  // row tiles whose windows are looked at beforehand
constexpr int kSlots = 4;
constexpr int kMostSplits = 8;  // shares of 16 rows at the least
constexpr int kPlane = kRows * 128, kHalf = 3 * kPlane;  // bytes: 64 columns of a plane, of all planes
constexpr int kOutLd = kRows + 1;                        // the sums in shared memory: [column][row]
constexpr int kBytes = kSlots * kHalf + 1024;
constexpr unsigned kDp = kRows, kSpare = 2 * kRows, kAcc = kSpare + 96;  // TMEM columns; S is at 0
enum Side { kForward, kDq, kDkv };

struct PlanesArgs {
  AttnArgs a;
  int P, packs, tiles, f_tiles;  // heads of a row tile, H / P, row tiles of a pack, frame tiles
  int splits;                    // CTAs of a cluster
};

struct Shared {
  unsigned long long full[kSlots], empty[kSlots], scores, ready, done, drained;
  unsigned tmem;
  int gave_up;
  Hull hull;
  unsigned char active[kTileBits];
  float half[2][kRows], top[kRows], sum[kRows], weight[kMostSplits][kRows];
  __align__(16) float lse2[2][kRows], delta[2][kRows];  // dk, dv: of the walk's rows, both negated
  __align__(16) int lo[2][kRows], len[2][kRows];
};

template <int SIDE>
__global__ void __launch_bounds__(kThreads, 1)
    attn_planes_kernel(const __grid_constant__ CUtensorMap qm, const __grid_constant__ CUtensorMap gm,
                       const __grid_constant__ CUtensorMap km, const __grid_constant__ CUtensorMap vm,
                       const __grid_constant__ PlanesArgs f) {
  extern __shared__ unsigned char raw[];
  __shared__ Shared sh;
  unsigned char *ring = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  float *sums = reinterpret_cast<float *>(ring);  // after the walk
  cg::cluster_group cluster = cg::this_cluster();
  const AttnArgs &a = f.a;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int group = warp >> 2, r = threadIdx.x & 127;
  const int P = f.P, per = kRows / P;
  unsigned id = blockIdx.x;
  const int split = id % f.splits;
  id /= f.splits;
  bool with_dp = SIDE == kDq, dk = false;
  if (SIDE == kDkv) {
    with_dp = dk = id & 1;
    id >>= 1;
  }
  // own rows: from position own_l of heads from own_h
  int own_l, own_h;
  if (SIDE == kDkv) {
    own_l = (int)(id % f.f_tiles) * kRows;
    id /= f.f_tiles;
    own_h = id % a.Hkv;
    id /= a.Hkv;
  } else {
    own_l = (int)(id % f.tiles) * per;
    id /= f.tiles;
    own_h = (int)(id % f.packs) * P;
    id /= f.packs;
  }
  const long long b = id;
  const Lens n = utt_lens(a, b);
  const int hk = SIDE == kDkv ? own_h : own_h / a.G;
  // the walk: steps [t0, t1); frames from `begin`, or packs of the group x row tiles
  const int row_tiles = SIDE == kDkv && own_l < n.nk ? (n.nq + per - 1) / per : 0;
  int begin = 0, t0 = 0, t1 = 0;
  auto walk = [&](int all) {
    const int2 steps = share_of(all, split, f.splits);
    t0 = steps.x;
    t1 = steps.y;
  };
  int2 range = make_int2(0, 0);
  const int row = own_l + r / P, head = own_h + r % P;  // unless SIDE is kDkv
  if (warp == 8 && lane == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
    }
    mbar_init(&sh.scores, 1);
    mbar_init(&sh.ready, 256);
    mbar_init(&sh.done, 1);
    mbar_init(&sh.drained, 1);
    fence_mbar_init_cluster();
    sh.gave_up = 0;
  }
  __syncwarp();
  if (warp == 9) tmem_alloc<512>(&sh.tmem);
  if (SIDE != kDkv) {
    if (warp < 8) {
      range = row_range(a, b, row, n);
      hull_note(sh.hull, warp, range);
    }
  } else if (a.windows) {
    for (int t = warp; t < min(row_tiles, kTileBits); t += kThreads / 32) {
      bool sees = false;
      for (int i = t * per + lane; i < min((t + 1) * per, n.nq); i += 32) {
        const int2 w = row_range(a, b, i, n);
        sees |= w.x < own_l + kRows && w.y > own_l;
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
  if (SIDE == kDkv) {
    walk((a.G / P) * row_tiles);
  } else {
    const int2 hull = hull_of<8>(sh.hull);
    begin = hull.x;
    walk((hull.y - hull.x + kRows - 1) / kRows);
  }
  auto next = [&](int t) {  // the first step at or after t
    if constexpr (SIDE == kDkv)
      if (a.windows)
        while (t < t1 && t % row_tiles < kTileBits && !sh.active[t % row_tiles]) ++t;
    return t;
  };
  const int start = next(t0);
  const bool any = start < t1;

  if (warp >= 8) {
    warpgroup_give_registers<kOtherRegs>();
    if (warp == 8 && lane == 0) {  // loads
      int item = 0;
      bool ok = true;
      auto load = [&](const CUtensorMap *m, int c, int h, int l) {
        const int slot = item % kSlots;
        ok = ok && wait(&sh.empty[slot], ((unsigned)(item / kSlots) & 1) ^ 1);
        if (!ok) return;
        arrive_expect_tx(&sh.full[slot], kHalf);
        for (int p = 0; p < 3; ++p)
          tma_load_4d(m, ring + slot * kHalf + p * kPlane, &sh.full[slot], (c * 3 + p) * 64, h, l, (int)b);
        ++item;
      };
      for (int t = start; ok && t < t1; t = next(t + 1)) {
        const int h = SIDE == kDkv ? hk * a.G + t / row_tiles * P : hk,
                  l = SIDE == kDkv ? t % row_tiles * per : begin + t * kRows;
        for (int c = 0; c < 2; ++c) {
          load(SIDE == kDkv ? &km : &qm, c, own_h, own_l);
          load(SIDE == kDkv ? &qm : &km, c, h, l);
        }
        for (int c = 0; with_dp && c < 2; ++c) {
          load(SIDE == kDkv ? &vm : &gm, c, own_h, own_l);
          load(SIDE == kDkv ? &gm : &vm, c, h, l);
        }
        const CUtensorMap *m = SIDE == kForward ? &vm : SIDE == kDq ? &km : dk ? &qm : &gm;
        for (int c = 0; c < 2; ++c) load(m, c, h, l);
      }
      if (!ok)  // copies in flight land before the CTA ends
        for (int i = max(0, item - kSlots); i < item; ++i)
          Waiter::drain(&sh.full[i % kSlots], (unsigned)(i / kSlots) & 1);
    }
    if (warp == 9 && any && elect_one()) {  // products
      constexpr unsigned i_s = mma_desc<kF32>(kRows, false), i_o = mma_desc<kF32>(64, true);
      const unsigned at = smem_u32(ring);
      int item = 0;
      bool ok = true;
      auto scores = [&](unsigned d) {  // one product over both halves, small planes first
        for (int x = item; x < item + 4; ++x) ok = ok && wait(&sh.full[x % kSlots], (unsigned)(x / kSlots) & 1);
        tc_fence_after();
        if (!ok) return;
        auto plane = [&](int c, int i) {
          const int x = (item + 2 * c) % kSlots, y = (item + 2 * c + 1) % kSlots;
          mma_rows<64>(tmem + d, at + x * kHalf + plane_a<kF32>(i) * kPlane, kPlane,
                       at + y * kHalf + plane_b<kF32>(i) * kPlane, kPlane, i_s, c + i > 0);
        };
#pragma unroll
        for (int i = 0; i < kPlanePairs<kF32>; ++i) {
          plane(0, i);
          if (i == kPlanePairs<kF32> - 1) {
            mma_commit(&sh.empty[item % kSlots]);
            mma_commit(&sh.empty[(item + 1) % kSlots]);
          }
          plane(1, i);
        }
        mma_commit(&sh.empty[(item + 2) % kSlots]);
        mma_commit(&sh.empty[(item + 3) % kSlots]);
        item += 4;
      };
      auto step = [&]() {
        scores(0);
        if (with_dp) scores(kDp);
        if (ok) mma_commit(&sh.scores);
      };
      step();
      int t = start;
      for (int s = 0; ok && t < t1; ++s) {
        const int after = next(t + 1);
        ok = wait(&sh.ready, s & 1);
        for (int c = 0; ok && c < 2; ++c, ++item) {
          const int z = item % kSlots;
          ok = wait(&sh.full[z], (unsigned)(item / kSlots) & 1);
          tc_fence_after();
          if (!ok) break;
#pragma unroll
          for (int i = 0; i < kPlanePairs<kF32>; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g) {  // 32 of the walk's rows each: the halves of the two groups
              const unsigned p = g & 1 ? tmem + (g >> 1) * 64 : tmem + kSpare + (g >> 1) * 48;
              mma_across<32>(tmem + kAcc + c * 64, p + plane_a<kF32>(i) * 16,
                             at + z * kHalf + plane_b<kF32>(i) * kPlane + g * 32 * 128, kPlane, i_o, i + g > 0);
            }
          mma_commit(&sh.empty[z]);
        }
        if (ok && after >= t1) mma_commit(&sh.done);
        if (ok && after < t1) step();
        t = after;
      }
      if (!ok) {
        mma_commit(&sh.drained);
        Waiter::drain(&sh.drained, 0);
      }
    }
    __syncwarp();
  } else {
    warpgroup_take_registers<kWorkRegs>();
    const unsigned lanes = (unsigned)((warp & 3) * 32) << 16;
    const unsigned s_col = tmem + lanes + group * 64, spare = tmem + lanes + kSpare + group * 48;
    const float c = a.scale * kLog2e;
    const float2 c2 = make_float2(c, c);
    const bool alive = range.y > range.x, keep = SIDE != kDkv || own_l + r < n.nk;
    const int j = own_l + r;  // kDkv: the thread's frame
    float delta = 0.0f, lse2 = INFINITY, top = -INFINITY, sum = 0.0f;
    if (SIDE == kDq) {
      const long long stat = (b * a.H + head) * a.Lq + row;
      float x = 0.0f;
      if (row < n.nq)
        x = dot_rows<kF32, 64>(
            static_cast<const float *>(a.go) + b * a.sgo.b + row * a.sgo.l + head * a.sgo.h + group * 64,
            static_cast<const float *>(a.out) + b * a.so.b + row * a.so.l + head * a.so.h + group * 64,
            min(64, a.D - group * 64));
      sh.half[group][r] = x;
      named_barrier<256>(1);
      delta = sh.half[0][r] + sh.half[1][r];
      if (group == 0 && split == 0 && row < a.Lq) a.delta[stat] = delta;
      if (alive) lse2 = a.lse[stat] * kLog2e;  // else +inf: every weight is 0
    }
    float acc[64];  // the row's sums of 64 columns
#pragma unroll
    for (int k = 0; k < 64; ++k) acc[k] = 0.0f;
    auto add_tile = [&]() {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        unsigned o[32];
        tmem_ld32(tmem + lanes + kAcc + group * 64 + i * 32, o);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 32; ++k) acc[i * 32 + k] += __uint_as_float(o[k]);
      }
    };
    // 32 weights (or dS) of half h as planes to TMEM: the first half's scores are needed no more when the
    // second's planes are written over them
    auto put = [&](int h, const float (&w)[32]) {
      unsigned out[3][16];
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        unsigned planes[3];
        split2<kF32>(make_float2(w[i], w[i + 1]), planes);
        out[0][i / 2] = planes[0];
        out[1][i / 2] = planes[1];
        out[2][i / 2] = planes[2];
      }
#pragma unroll
      for (int p = 0; p < 3; ++p) tmem_st16((h ? s_col : spare) + p * 16, out[p]);
    };
    bool ok = true;
    int s = 0;
    for (int t = start; t < t1; t = next(t + 1), ++s) {
      if constexpr (SIDE == kDkv) {  // the rows' statistics
        if (group == 0) {
          const int i = t % row_tiles * per + r / P, h = hk * a.G + t / row_tiles * P + r % P;
          const int2 w = row_range(a, b, i, n);
          const bool sees = w.y > w.x;  // else every weight is 0
          const long long stat = (b * a.H + h) * a.Lq + min(i, a.Lq - 1);
          sh.lse2[s & 1][r] = sees ? -a.lse[stat] * kLog2e : -INFINITY;
          sh.delta[s & 1][r] = sees && dk ? -a.delta[stat] : 0.0f;
          sh.lo[s & 1][r] = w.x;
          sh.len[s & 1][r] = w.y - w.x;
        }
        named_barrier<256>(1);
      }
      // after giving up the steps go on without waits: the barriers between the threads need everybody
      ok = __all_sync(0xffffffffu, ok && wait(&sh.scores, s & 1));
      tc_fence_after();
      if (s > 0) add_tile();  // the products of the tile before were issued before these scores
      const int j0 = begin + t * kRows + group * 64;
      if constexpr (SIDE == kForward) {
        unsigned x[2][32];
        tmem_ld32(s_col, x[0]);
        tmem_ld32(s_col + 32, x[1]);
        tmem_wait_ld();
        if (__any_sync(0xffffffffu, range.x > j0 || range.y < j0 + 64)) {
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if ((unsigned)(j0 + i - range.x) >= (unsigned)(range.y - range.x)) x[i >> 5][i & 31] = 0xff800000u;
        }
        float most = -INFINITY;
#pragma unroll
        for (int i = 0; i < 64; ++i) most = fmaxf(most, __uint_as_float(x[i >> 5][i & 31]));
        sh.half[group][r] = most;
        named_barrier<256>(1);
        const float now = fmaxf(top, fmaxf(sh.half[0][r], sh.half[1][r]) * c);
        named_barrier<256>(1);
        const float ref = now == -INFINITY ? 0.0f : now;  // nothing seen yet: every weight is 0
        const float fade = fast_exp2(top - ref);
        top = now;
        sum *= fade;
#pragma unroll
        for (int k = 0; k < 64; ++k) acc[k] *= fade;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float w[32];
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float2 z = fma2(pair(x[h][i], x[h][i + 1]), c2, make_float2(-ref, -ref));
            w[i] = fast_exp2(z.x);
            w[i + 1] = fast_exp2(z.y);
            sum += w[i] + w[i + 1];
          }
          put(h, w);
        }
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          unsigned x[32], y[32];
          tmem_ld32(s_col + h * 32, x);
          if (with_dp) tmem_ld32(s_col + kDp + h * 32, y);
          tmem_wait_ld();
          float w[32];
          const float *l2 = sh.lse2[s & 1] + group * 64 + h * 32, *dl = sh.delta[s & 1] + group * 64 + h * 32;
          const int *lo = sh.lo[s & 1] + group * 64 + h * 32, *len = sh.len[s & 1] + group * 64 + h * 32;
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            // frames that the row does not see weigh 0, whatever S and dP are
            const bool sees = SIDE == kDq ? (unsigned)(j0 + h * 32 + i - range.x) < (unsigned)(range.y - range.x)
                                          : (unsigned)(j - lo[i]) < (unsigned)len[i];
            const float p = fast_exp2(fmaf(__uint_as_float(x[i]), c, SIDE == kDq ? -lse2 : l2[i]));
            w[i] = !sees ? 0.0f : with_dp ? p * (__uint_as_float(y[i]) + (SIDE == kDq ? -delta : dl[i])) : p;
          }
          put(h, w);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&sh.ready);
    }
    if (any && ok) ok = wait(&sh.done, 0);
    __syncwarp();
    tc_fence_after();
    if (any) add_tile();
    const float by = SIDE == kDq || dk ? a.scale : 1.0f;
    named_barrier<256>(1);  // both groups have seen every product done: the ring is free
#pragma unroll
    for (int k = 0; k < 64; ++k)
      sums[(group * 64 + k) * kOutLd + r] = keep ? acc[k] * by : 0.0f;
    if (SIDE == kForward) {
      sh.half[group][r] = sum;
      named_barrier<256>(1);
      if (group == 0) {
        sh.top[r] = top;
        sh.sum[r] = sh.half[0][r] + sh.half[1][r];
      }
    }
    __syncwarp();
    tc_fence_before();
  }
  cluster.sync();
  if (warp < 8) {  // a share of the rows each CTA
    const int share = kRows / f.splits, r0 = split * share, d = threadIdx.x & 127;
    auto place = [&](int x, int *h) {  // position and head of own row x
      *h = SIDE == kDkv ? own_h : own_h + x % P;
      return SIDE == kDkv ? own_l + x : own_l + x / P;
    };
    if (threadIdx.x < share) {  // what each CTA's sum of the row is multiplied with
      const int x = r0 + threadIdx.x;
      bool bad = SIDE == kForward && n.bad;
      float top[kMostSplits], sum[kMostSplits], most = -INFINITY, l = 0.0f;
#pragma unroll
      for (int k = 0; k < kMostSplits; ++k) {
        if (k >= f.splits) break;
        bad |= *cluster.map_shared_rank(&sh.gave_up, k) != 0;
        if (SIDE == kForward) {
          top[k] = *cluster.map_shared_rank(&sh.top[x], k);
          sum[k] = *cluster.map_shared_rank(&sh.sum[x], k);
          most = fmaxf(most, top[k]);
        }
      }
      const float ref = most == -INFINITY ? 0.0f : most;
      float w[kMostSplits];
#pragma unroll
      for (int k = 0; k < kMostSplits; ++k) {
        if (k >= f.splits) break;
        w[k] = SIDE == kForward ? fast_exp2(top[k] - ref) : 1.0f;
        if (SIDE == kForward) l = fmaf(sum[k], w[k], l);
      }
      const float all = bad ? NAN : SIDE != kForward ? 1.0f : l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
      for (int k = 0; k < kMostSplits; ++k)
        if (k < f.splits) sh.weight[k][x] = w[k] * all;
      int h;
      const int at = place(x, &h);
      if (SIDE == kForward && a.lse && at < a.Lq)
        a.lse[(b * a.H + h) * a.Lq + at] = bad ? NAN : l == 0.0f ? -INFINITY : (most + log2f(l)) * kLn2;
    }
    named_barrier<256>(1);
    const Strides &st = SIDE == kForward ? a.so : SIDE == kDq ? a.sdq : dk ? a.sdk : a.sdv;
    float *to = static_cast<float *>(SIDE == kForward ? const_cast<void *>(a.out) : SIDE == kDq ? a.dq
                                     : dk            ? a.dk
                                                     : a.dv) + b * st.b + d;
    constexpr int U = 8;  // loads in flight
    const float *whole = sums;  // [column][row] of the share, scaled
    int ld = kOutLd, first = r0;
    if (f.splits > 1) {  // neighbouring threads read neighbouring rows of the others' memory
      float *own = sums + kRows * kOutLd;
      ld = share + 1;
      first = 0;
      for (int e0 = threadIdx.x; e0 < share * kRows; e0 += 256 * U) {
        float v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = 0.0f;
        for (int k = 0; k < f.splits; ++k) {
          const float *from = cluster.map_shared_rank(sums, k) + r0;
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int e = e0 + u * 256;
            v[u] = fmaf(from[e / share * kOutLd + e % share], sh.weight[k][r0 + e % share], v[u]);
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) own[(e0 + u * 256) / share * ld + (e0 + u * 256) % share] = v[u];
      }
      named_barrier<256>(1);
      whole = own;
    }
    for (int i0 = threadIdx.x >> 7; i0 < share; i0 += 2 * U) {  // a thread has every other row
      float v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        v[u] = whole[d * ld + first + i0 + 2 * u];
        if (f.splits == 1) v[u] *= sh.weight[0][i0 + 2 * u];
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        int h;
        const int at = place(r0 + i0 + 2 * u, &h);
        if (d < a.D && at < (SIDE == kDkv ? a.Lk : a.Lq)) to[at * st.l + h * st.h] = v[u];
      }
    }
  }
  cluster.sync();  // the others have read this CTA's sums
  if (warp == 9) tmem_free<512>(tmem);
}

// CTAs of a cluster: while CTAs leave SMs idle and each keeps two steps
int splits_of(long long units, long long steps) {
  int s = 1;
  while (s < kMostSplits && units * s * 2 <= kSMs && steps / (s * 2) >= 2) s *= 2;
  return s;
}

template <int SIDE>
cudaError_t launch(PlanesArgs f, long long units, long long steps, const TensorMap &q, const TensorMap &go,
                   const TensorMap &k, const TensorMap &v, cudaStream_t stream) {
  const cudaError_t e =
      prepare_tc_kernel(reinterpret_cast<const void *>(attn_planes_kernel<SIDE>), kBytes, kLaunchRegs);
  if (e != cudaSuccess || units == 0) return e;
  f.splits = splits_of(units, steps);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * f.splits));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kBytes;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = f.splits;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = f.splits > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, attn_planes_kernel<SIDE>, q.map, go.map, k.map, v.map, f);
}

size_t tensor_bytes(long long B, long long L, long long H) { return (2 * plane_bytes(B, L, H) + 255) / 256 * 256; }

}  // namespace

bool attn_planes_takes(int dtype, long long Lq, long long Lk, int G, int D, bool backward) {
  return dtype == kF32 && D > 64 && D <= 128 && Lq > 0 && Lk > 0 &&
         (backward || Lq * G > kStepRows || D % 8 != 0);
}

bool attn_planes_fits(const AttnArgs &a, int dtype, bool backward) {
  auto fits = [&](const void *p, const Strides &s, long long L, int H) {  // 16-byte vectors
    return map_fits(dtype, p, a.B, L, H, a.D, s.b, s.l, s.h);
  };
  return attn_planes_takes(dtype, a.Lq, a.Lk, a.G, a.D, backward) &&
         (!backward || (fits(a.out, a.so, a.Lq, a.H) && fits(a.go, a.sgo, a.Lq, a.H)));
}

size_t attn_planes_workspace(long long B, long long Lq, long long Lk, int H, int Hkv, bool backward) {
  return (backward ? 2 : 1) * tensor_bytes(B, Lq, H) + 2 * tensor_bytes(B, Lk, Hkv);
}

cudaError_t launch_attn_planes(const AttnArgs &a, bool backward, void *workspace, cudaStream_t stream) {
  PlanesArgs f = {};
  f.a = a;
  f.P = attn_row_pack(a.G);
  f.packs = a.H / f.P;
  f.tiles = (int)(((long long)a.Lq * f.P + kRows - 1) / kRows);
  f.f_tiles = (a.Lk + kRows - 1) / kRows;
  char *ws = static_cast<char *>(workspace);
  auto source = [&](const void *p, const Strides &s, const long long *lens, int L, int H) {
    const PlaneSource t = {static_cast<const float *>(p), s.b, s.l, s.h, lens, L, H,
                           reinterpret_cast<unsigned short *>(ws)};
    ws += tensor_bytes(a.B, L, H);
    return t;
  };
  PlaneSource t[4];
  t[0] = source(a.q, a.sq, a.q_lens, a.Lq, a.H);
  t[1] = source(a.k, a.sk, a.k_lens, a.Lk, a.Hkv);
  t[2] = source(a.v, a.sv, a.k_lens, a.Lk, a.Hkv);
  if (backward) t[3] = source(a.go, a.sgo, a.q_lens, a.Lq, a.H);
  cudaError_t e = launch_planes(t, backward ? 4 : 3, a.B, a.D, stream);
  if (e != cudaSuccess) return e;
  TensorMap q, go, k, v;
  const int per = kRows / f.P;
  if (!encode_planes(&q, t[0].dst, a.B, a.Lq, a.H, 2, f.P, per) ||
      !encode_planes(&go, t[backward ? 3 : 0].dst, a.B, a.Lq, a.H, 2, f.P, per) ||
      !encode_planes(&k, t[1].dst, a.B, a.Lk, a.Hkv, 2, 1, kRows) ||
      !encode_planes(&v, t[2].dst, a.B, a.Lk, a.Hkv, 2, 1, kRows))
    return cudaErrorInvalidValue;
  const long long rows = a.B * f.packs * f.tiles, frames = 2 * a.B * a.Hkv * f.f_tiles;
  if (!backward) return launch<kForward>(f, rows, f.f_tiles, q, go, k, v, stream);
  e = launch<kDq>(f, rows, f.f_tiles, q, go, k, v, stream);
  if (e != cudaSuccess) return e;
  return launch<kDkv>(f, frames, (long long)(a.G / f.P) * f.tiles, q, go, k, v, stream);
}

}  // namespace tdt
