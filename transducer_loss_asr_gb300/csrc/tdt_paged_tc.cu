// tdt_paged_tc.cu -- causal attention of many query rows over a paged cache on the 5th-generation tensor cores: float16 and
// bfloat16 queries over pages of their own type, heads up to 128.
//
// A tile is 128 rows, a row being a (query, head) pair: P heads (the largest power of two that divides the group of a key
// head, up to 16) of 128 / P queries share a tile and so share the keys that are loaded for it.  A stream is a walk over
// tiles of 128 keys, with 128 threads (thread = row) for its softmax:
//   S = Q K^T            128 x 128, float32 in TMEM, operands in shared memory
//   P = 2^(S c - m)      rounded to 16 bits, written over S in TMEM
//   O += P V             P from TMEM, O in TMEM
// and the products of one stream run while the threads of the SM's other one are at their softmax:
//   wide    (more than 128 rows): a CTA walks two row tiles over the same keys;
//   single  (at most 128 rows):   a CTA walks one, with half of the SM's TMEM, registers and shared memory, so that two
//                                 CTAs share an SM.
// The reference m of a row moves only when its maximum has grown by 8 (in base 2): the factor cancels in O / l.  l adds the
// unrounded float32 weights.  A row sees the positions up to its own: a tile's walk ends at its last row's.
//
// One warp loads tiles with TMA, a box a page (pages of at least 8 places); a page that a tile does not need becomes one
// past the tensor's end, which TMA fills with zeros, and places past the utterance's end are zeroed in the last value tile,
// as they may hold anything.
//
// Few row tiles: the keys are split over several CTAs, whose results a second kernel joins in a fixed order.
//
// Bound by the tensor cores at large sizes: 8 x 1024 queries behind 7,168 positions, 16 heads on 4 of 128, bfloat16: 351 us, 1,470
// TFLOP/s of 1,927 measured for a library product; by latency at small ones: 16 ragged x 121 behind 750, 16 heads of 64: 18.7 us.
// e4m3 pages converted to float16 tiles by four warps of this kernel took 890 us at the large size, against 400 with the
// pages laid out densely beforehand and read by cross attention: the conversion and its powers of two want more issue slots than
// the softmax leaves.
#include "tdt_paged.cuh"
#include "tdt_tc.cuh"

namespace tdt {
namespace {

constexpr int kRows = 128;          // rows of a tile, keys of a tile
constexpr int kMostSplits = 64;
constexpr float kLazy = 8.0f;
// float16 weights start at 2^7 and so stay clear of the type's least numbers; at most 2^15
template <int DT> constexpr float kShift = DT == kF16 ? 7.0f : 0.0f;

struct TcPlan {
  int P;          // heads of a tile
  int packs;      // H / P
  int wide;       // 1: two row tiles a CTA, else one
  int tiles;      // row tiles (CTAs) of a pack
  int splits;     // CTAs that share the keys of a row tile
};

struct TcArgs {
  PagedArgs a;
  TcPlan p;
  int q_b, q_h, o_b, o_h, k_p, k_h, v_p, v_h;  // 0 for repeated axes
  float *part_o, *part_l;                      // splits > 1: [split][CTA row][DP], [split][CTA row]
};

template <int DP, bool WIDE> struct TcShape {
  static constexpr int CHUNKS = DP / 64;
  static constexpr int CHUNK = kRows * 128;          // bytes
  static constexpr int TILE = CHUNKS * CHUNK;
  static constexpr int NS = WIDE ? 2 : 1;            // streams
  static constexpr int SLOTS = WIDE ? (DP == 64 ? 8 : 4) : (DP == 64 ? 5 : 2);
  static constexpr int BYTES = (NS + SLOTS) * TILE;
  static constexpr int THREADS = NS * 128 + 128;     // softmax; TMA, MMA, tails, a spare warp
  static constexpr int CTAS = WIDE ? 1 : 2;          // of an SM
  static constexpr int TMEM = WIDE ? 512 : 256;      // columns: S and O of each stream
  // registers of a thread: at launch, then of the softmax warpgroups and of the other one, which
  // adds up to the same: 3 x 168 = 2 x 208 + 88, 2 x 128 = 200 + 56
  static constexpr int REGS = WIDE ? 168 : 128;
  static constexpr int SOFTMAX_REGS = WIDE ? 208 : 200;
  static constexpr int OTHER_REGS = WIDE ? 88 : 56;
};

struct TcShared {
  unsigned long long full[8], empty[8], q_full, s_full[2], p_ready[2], o_full[2], tail_full, drained;
  unsigned tmem;
  int gave_up, bad_page;
};

// 32 scores of a row (float32 bits) to weights 2^(s c - ref), packed in pairs and added to sum.
template <int DT, int N>
__device__ __forceinline__ void exp_pack(const unsigned (&s)[32], float c, float neg, unsigned (&out)[N], int at, float2 &sum) {
  const float2 c2 = make_float2(c, c), n2 = make_float2(neg, neg);
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    const float2 z = fma2(pair(s[i], s[i + 1]), c2, n2);
    const float2 p = make_float2(fast_exp2(z.x), fast_exp2(z.y));
    sum = add2(sum, p);
    out[at + i / 2] = pack2<DT>(p.x, p.y);
  }
}
template <int QT, int DP, bool WIDE>
__global__ void __launch_bounds__(TcShape<DP, WIDE>::THREADS, TcShape<DP, WIDE>::CTAS)
    paged_tc_kernel(const __grid_constant__ CUtensorMap qm, const __grid_constant__ CUtensorMap km,
                    const __grid_constant__ CUtensorMap vm, const __grid_constant__ CUtensorMap om,
                    const __grid_constant__ TcArgs f) {
  typedef TcShape<DP, WIDE> S;
  extern __shared__ unsigned char raw[];
  __shared__ TcShared sh;
  unsigned char *tiles = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  unsigned char *q_tile = tiles, *slots = tiles + S::NS * S::TILE;
  const PagedArgs &a = f.a;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  // this CTA's rows and keys; row tiles with the longest walks come first
  unsigned id = blockIdx.x;
  const int split = id % f.p.splits;
  id /= f.p.splits;
  const int tile = f.p.tiles - 1 - (int)(id % f.p.tiles);
  const unsigned cta = id - id % f.p.tiles + tile;
  id /= f.p.tiles;
  const int pack = id % f.p.packs;
  const long long b = id / f.p.packs;
  const int P = f.p.P, per = kRows / P, i0 = tile * S::NS * per;
  const int h0 = pack * P, hk = h0 / a.G;
  const NewRows n = new_rows(a.t, b, a.Lq);
  const bool some = i0 < n.n;                                              // else no row takes part
  const int end = some ? n.first + min(n.n, i0 + S::NS * per) : 0;     // positions that some row sees
  const int kv_end = n.first + n.n;
  const int2 steps = share_of((end + kRows - 1) / kRows, split, f.p.splits);
  const int begin = steps.x * kRows, T = steps.y - steps.x;                // T tiles of keys from `begin`
  auto frame = [&](int s) { return begin + s * kRows; };
  // A warp zeroes what lies past the utterance's end in its last tile of v, which is the last tile
  // loaded: the load then arrives at tail_full, and that warp hands the tile on.
  const bool cut = T > 0 && begin + T * kRows > kv_end;

  constexpr int kAux = S::NS * 4;  // the first warp past the softmax's: TMA
  const int stream = warp >> 2, r = threadIdx.x & 127;
  int row = 0, head = 0;
  int seen = 0;                    // positions that this thread's row sees
  if (warp < kAux) {
    row = i0 + stream * per + r / P;
    head = h0 + r % P;
    seen = row < n.n ? n.first + row + 1 : 0;
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
    sh.bad_page = 0;
    if (some) {
      arrive_expect_tx(&sh.q_full, S::NS * S::TILE);
      for (int t = 0; t < S::NS; ++t)
        for (int ch = 0; ch < S::CHUNKS; ++ch)
          tma_load_4d(&qm, q_tile + t * S::TILE + ch * S::CHUNK, &sh.q_full, ch * 64, h0 * f.q_h, i0 + t * per,
                      (int)b * f.q_b);
    }
  } else if (warp == kAux + 1) {
    tmem_alloc<S::TMEM>(&sh.tmem);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const unsigned tmem = __shfl_sync(0xffffffffu, sh.tmem, 0);
  const Waiter wait{&sh.gave_up};

  if (warp >= kAux) {
    warpgroup_give_registers<S::OTHER_REGS>();  // to the softmax warps, which hold a row of scores
    if (warp == kAux && some && T == 0) wait(&sh.q_full, 0);  // nobody else does
    if (warp == kAux && T > 0) {
      // lane l has box l of a tile: a page, or a tile's part of one
      const int page_size = 1 << a.t.page_bits, boxes = page_size < kRows ? kRows / page_size : 1;
      const int box_rows = page_size < kRows ? page_size : kRows;
      auto lookup = [&](int s) {  // the page of this lane's box of step s; one past the end: zeros
        const int pos = frame(s) + lane * box_rows;
        if (s >= T || lane >= boxes || pos >= end) return a.t.n_pages;
        const int page = page_of(a.t, b, pos);
        if (page < 0) sh.bad_page = 1;
        return page < 0 ? a.t.n_pages : page;
      };
      int page = lookup(0), next = 0;
      bool ok = true;
      int at = 0;
      for (; at < 2 * T; ++at) {  // tiles count up: k of step 0, v of step 0, k of step 1, ...
        const int slot = at % S::SLOTS, s = at / 2;
        const bool values = at & 1;
        if (!values) next = lookup(s + 1);
        ok = __all_sync(0xffffffffu, wait(&sh.empty[slot], ((unsigned)(at / S::SLOTS) & 1) ^ 1));
        if (!ok) break;
        unsigned long long *bar = cut && at == 2 * T - 1 ? &sh.tail_full : &sh.full[slot];
        if (lane == 0) arrive_expect_tx(bar, S::TILE);
        __syncwarp();
        if (lane < boxes) {
          const int place = page_size < kRows ? 0 : frame(s) & (page_size - 1);
          const int p = page == a.t.n_pages ? page : page * (values ? f.v_p : f.k_p);
#pragma unroll
          for (int ch = 0; ch < S::CHUNKS; ++ch)
            tma_load_4d(values ? &vm : &km, slots + slot * S::TILE + ch * S::CHUNK + lane * box_rows * 128, bar,
                        ch * 64, hk * (values ? f.v_h : f.k_h), place, p);
        }
        __syncwarp();
        if (values) page = next;
      }
      if (!ok && lane == 0)  // copies in flight land before the CTA ends
        for (int i = max(0, at - S::SLOTS); i < at; ++i)
          Waiter::drain(&sh.full[i % S::SLOTS], (unsigned)(i / S::SLOTS) & 1);
    }
    if (warp == kAux + 2 && cut) {
      const int slot = (2 * T - 1) % S::SLOTS;
      if (__all_sync(0xffffffffu, wait(&sh.tail_full, 0)))
        zero_tail(slots + slot * S::TILE, S::CHUNKS, S::CHUNK, kv_end - frame(T - 1), kRows);
      if (lane == 0) mbar_arrive(&sh.full[slot]);
    }
    if (warp == kAux + 1 && T > 0 && elect_one()) {
      constexpr unsigned i_s = mma_desc<QT>(kRows, false), i_o = mma_desc<QT>(DP, true);
      const unsigned q_addr = smem_u32(q_tile), s_addr = smem_u32(slots);
      bool ok = wait(&sh.q_full, 0);
      auto loaded = [&](int at) {
        ok = ok && wait(&sh.full[at % S::SLOTS], (unsigned)(at / S::SLOTS) & 1);
      };
      auto scores = [&](int w, int at) {  // S_w = Q_w K^T
        tc_fence_after();
        if (!ok) return;
        const int slot = at % S::SLOTS;
        mma_rows<DP>(tmem + w * kRows, q_addr + w * S::TILE, S::CHUNK, s_addr + slot * S::TILE, S::CHUNK,
                     i_s, false);
        mma_commit(&sh.s_full[w]);
        if (w == S::NS - 1) mma_commit(&sh.empty[slot]);
      };
      auto values = [&](int w, int k, int at, bool last) {  // O_w += P_w V, the stream's k-th
        const int slot = at % S::SLOTS;
        ok = ok && wait(&sh.p_ready[w], k & 1);
        tc_fence_after();
        if (!ok) return;
        mma_across<kRows>(tmem + S::NS * kRows + w * DP, tmem + w * kRows, s_addr + slot * S::TILE, S::CHUNK, i_o, k > 0);
        if (w == S::NS - 1) mma_commit(&sh.empty[slot]);
        if (last) mma_commit(&sh.o_full[w]);
      };
      loaded(0);
      for (int w = 0; w < S::NS; ++w) scores(w, 0);
      for (int s = 0; ok && s < T; ++s) {
        const int at = 1 + 2 * s;
        loaded(at);
#pragma unroll
        for (int w = 0; w < S::NS; ++w) {
          values(w, s, at, s + 1 == T);
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
    const bool alive = seen > 0;
    const bool used = __any_sync(0xffffffffu, alive);  // warps without a row that takes part only pass the tiles on
    bool ok = true;
    const float c = a.scale * kLog2e;
    for (int s = 0; s < T; ++s) {
      ok = wait(&sh.s_full[stream], s & 1);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      if (!used) {
        tc_fence_before();
        mbar_arrive(&sh.p_ready[stream]);
        continue;
      }
      const int j0 = frame(s);
      const bool masked = __any_sync(0xffffffffu, alive && seen < j0 + kRows);
      unsigned x[4][32];
#pragma unroll
      for (int i = 0; i < 4; ++i) tmem_ld32(s_col + i * 32, x[i]);
      tmem_wait_ld();
      if (masked) {
        const int from = seen - j0;
#pragma unroll
        for (int i = 0; i < 128; ++i)
          if (i >= from) x[i >> 5][i & 31] = 0xff800000u;  // -inf
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
      const bool grow = alive && top > ref + (kLazy + kShift<QT>);  // from -inf: any score
      if (__any_sync(0xffffffffu, grow)) {
        const float now = grow ? top - kShift<QT> : ref;
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
        unsigned p[32];
        exp_pack<QT>(x[2 * i], c, neg, p, 0, sum0);
        exp_pack<QT>(x[2 * i + 1], c, neg, p, 16, sum1);
        tmem_st32(s_col + i * 32, p);
      }
      sum0 = add2(sum0, sum1);
      l += sum0.x + sum0.y;
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&sh.p_ready[stream]);
    }
    if (T > 0 && ok) ok = wait(&sh.o_full[stream], 0);
    if (T == 0 && some) ok = wait(&sh.q_full, 0);  // the tile's memory is used below
    __syncwarp();
    tc_fence_after();
    if (!alive) l = 0.0f;
    const bool bad = n.bad || !ok || *reinterpret_cast<volatile int *>(&sh.gave_up) ||
                     *reinterpret_cast<volatile int *>(&sh.bad_page);
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
      if (T > 0) {
        tmem_ld32(o_col + i * 32, o);
        tmem_wait_ld();
      }
      float v[32];
#pragma unroll
      for (int k = 0; k < 32; ++k) v[k] = bad ? NAN : l == 0.0f ? 0.0f : __uint_as_float(o[k]) * inv;
      if (f.p.splits == 1) {
        stage32<QT>(out_tile, S::CHUNK, r, i * 32, v);
      } else if (row < a.Lq) {
        store_columns(f.part_o + (tile_at * DP + i * 32) * (S::NS * kRows) + threadIdx.x, S::NS * kRows, v);
      }
      __syncwarp();
    }
    if (f.p.splits == 1) {
      fence_async_shared();
      named_barrier<128>(1 + stream);
      if (r == 0 && row < a.Lq) {
        for (int ch = 0; ch < S::CHUNKS; ++ch)
          if (ch * 64 < a.D) tma_store_4d(&om, out_tile + ch * S::CHUNK, ch * 64, h0 * f.o_h, row, (int)b * f.o_b);
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
template <int QT, int DP>
__global__ void __launch_bounds__(256) paged_join_kernel(const __grid_constant__ TcArgs f, int rows) {
  const PagedArgs &a = f.a;
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
    if (row_of(rr) < a.Lq && d0 + d < a.D) {
      unsigned short *dst = static_cast<unsigned short *>(a.out) + b * a.so.b + row_of(rr) * a.so.l + head_of(rr) * a.so.h + d0 + d;
      *reinterpret_cast<uint4 *>(dst) = make_uint4(pack2<QT>(x[0], x[1]), pack2<QT>(x[2], x[3]), pack2<QT>(x[4], x[5]), pack2<QT>(x[6], x[7]));
    }
  }
}

TcPlan plan(long long B, long long Lq, long long most, int H, int G) {
  TcPlan p;
  p.P = attn_row_pack(G);
  p.packs = H / p.P;
  const long long rows = Lq * p.P;
  p.wide = rows > kRows;
  const int tile_rows = p.wide ? 2 * kRows : kRows;
  p.tiles = (int)((rows + tile_rows - 1) / tile_rows);
  // split the keys while the CTAs leave SMs idle, if that saves a CTA a dozen tiles' time: joining
  // costs about as much as eight take
  const long long ctas = B * p.packs * p.tiles, steps = (most + kRows - 1) / kRows;
  long long s = ctas > 0 ? (p.wide ? 1 : 2) * kSMs / ctas : 1;
  if (s > steps / 4) s = steps / 4;
  if (s > kMostSplits) s = kMostSplits;
  p.splits = s < 2 || steps - steps / s < 12 ? 1 : (int)s;
  return p;
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }
size_t part_rows(const TcPlan &p, long long B) {
  return p.splits == 1 ? 0 : (size_t)B * p.packs * p.tiles * p.splits * (p.wide ? 2 : 1) * kRows;
}

template <int QT, int DP, bool WIDE>
cudaError_t launch(const TcArgs &f, const TensorMap &q, const TensorMap &k, const TensorMap &v, const TensorMap &o,
                   cudaStream_t stream) {
  typedef TcShape<DP, WIDE> S;
  const size_t smem = S::BYTES + 1024;
  cudaError_t e = prepare_tc_kernel(reinterpret_cast<const void *>(paged_tc_kernel<QT, DP, WIDE>), smem, S::REGS);
  if (e != cudaSuccess) return e;
  const long long ctas = f.a.B * f.p.packs * f.p.tiles;
  paged_tc_kernel<QT, DP, WIDE>
      <<<(unsigned)(ctas * f.p.splits), S::THREADS, smem, stream>>>(q.map, k.map, v.map, o.map, f);
  e = cudaGetLastError();
  if (e != cudaSuccess || f.p.splits == 1) return e;
  const int rows = S::NS * kRows;
  return launch_follower(paged_join_kernel<QT, DP>, dim3((unsigned)(ctas * (rows / 32) * (DP / 32))), 256, 0, stream, f, rows);
}
template <int QT>
cudaError_t by_shape(const TcArgs &f, const TensorMap &q, const TensorMap &k, const TensorMap &v, const TensorMap &o,
                     cudaStream_t s) {
  if (f.a.D > 64)
    return f.p.wide ? launch<QT, 128, true>(f, q, k, v, o, s) : launch<QT, 128, false>(f, q, k, v, o, s);
  return f.p.wide ? launch<QT, 64, true>(f, q, k, v, o, s) : launch<QT, 64, false>(f, q, k, v, o, s);
}

}  // namespace

bool paged_tc_takes(const PagedArgs &a, int dtype) {
  auto pages_fit = [&](const Pages &p) {
    return map_fits(dtype, p.data, a.t.n_pages, 1LL << a.t.page_bits, a.Hkv, a.D, p.s.b, p.s.l, p.s.h);
  };
  return dtype != kF32 && a.D <= 128 && a.D % 8 == 0 && a.t.page_bits >= 3 && pages_fit(a.k) && pages_fit(a.v);
}

size_t paged_tc_workspace(long long B, long long Lq, long long most, int H, int Hkv, int D) {
  const size_t rows = part_rows(plan(B, Lq, most, H, H / Hkv), B);
  return align256(rows * (D <= 64 ? 64 : 128) * 4) + align256(rows * 4);
}

bool paged_tc_fits(const PagedArgs &a, int dtype) {
  auto rows_fit = [&](const void *p, const Strides &s) { return map_fits(dtype, p, a.B, a.Lq, a.H, a.D, s.b, s.l, s.h); };
  return paged_tc_takes(a, dtype) && rows_fit(a.q, a.sq) && rows_fit(a.out, a.so) && (attn_row_pack(a.G) == 1 || a.sq.h != 0);
}

cudaError_t launch_paged_tc(const PagedArgs &a, int dtype, void *workspace, cudaStream_t stream) {
  TcArgs f = {};
  f.a = a;
  const long long page_size = 1LL << a.t.page_bits;
  f.p = plan(a.B, a.Lq, (long long)a.t.max_pages << a.t.page_bits, a.H, a.G);
  const size_t rows = part_rows(f.p, a.B);
  f.part_o = static_cast<float *>(workspace);
  f.part_l = reinterpret_cast<float *>(static_cast<char *>(workspace) + align256(rows * (a.D <= 64 ? 64 : 128) * 4));
  TensorMap q, k, v, o;
  const int box = (int)(page_size < kRows ? page_size : kRows);
  if (!encode_map(&o, a.out, dtype, a.B, a.Lq, a.H, a.D, a.so.b, a.so.l, a.so.h, f.p.P, kRows / f.p.P) ||
      !encode_map(&q, a.q, dtype, a.B, a.Lq, a.H, a.D, a.sq.b, a.sq.l, a.sq.h, f.p.P, kRows / f.p.P) ||
      !encode_map(&k, a.k.data, dtype, a.t.n_pages, page_size, a.Hkv, a.D, a.k.s.b, a.k.s.l, a.k.s.h, 1, box) ||
      !encode_map(&v, a.v.data, dtype, a.t.n_pages, page_size, a.Hkv, a.D, a.v.s.b, a.v.s.l, a.v.s.h, 1, box))
    return cudaErrorInvalidValue;
  f.q_b = q.b_mul;
  f.q_h = q.h_mul;
  f.o_b = o.b_mul;
  f.o_h = o.h_mul;
  f.k_p = k.b_mul;
  f.k_h = k.h_mul;
  f.v_p = v.b_mul;
  f.v_h = v.h_mul;
  return dtype == kF16 ? by_shape<kF16>(f, q, k, v, o, stream) : by_shape<kBF16>(f, q, k, v, o, stream);
}

}  // namespace tdt
