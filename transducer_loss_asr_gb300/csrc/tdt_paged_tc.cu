// tdt_paged_tc.cu -- causal attention of many query rows over a paged cache on the 5th-generation tensor cores: float16 and
// bfloat16 queries over pages of their own type or of e4m3, heads up to 128.
//
// A tile is 128 rows, a row being a (query, head) pair: P heads (the largest power of two that divides the group of a key
// head, up to 16) of 128 / P queries share a tile and so share the keys that are loaded for it.  A stream is a walk over
// tiles of 128 keys, with 128 threads (thread = row) for its softmax:
//   S = Q K^T            128 x 128, float32 in TMEM, operands in shared memory
//   P = 2^(S c - m)      rounded to 16 bits, written over S in TMEM
//   O += P V             P from TMEM, O in TMEM
// and the products of one stream run while the threads of the SM's other one are at their softmax:
//   wide    (more than 128 rows): a CTA walks two row tiles over the same keys;
//   single  (at most 128 rows):   16-bit pages: one row tile, two CTAs an SM; e4m3: one row tile, two streams that take
//                                 every other key tile, joined in shared memory at the end.
// The reference m of a row moves only when its maximum has grown by 8 (in base 2): the factor cancels in O / l.  l adds the
// unrounded float32 weights.  A row sees the positions up to its own: a tile's walk ends at its last row's.
//
// 16-bit pages: one warp loads tiles with TMA, a box a page (pages of at least 8 places); a page that a tile does not need
// becomes one past the tensor's end, which TMA fills with zeros, and places past the utterance's end are zeroed in the last
// value tile, as they may hold anything.
// e4m3 pages: four warps load rows, turn them into float16 (exactly) times a power of two that makes 32 rows even, and place
// them as TMA would.  The 32 rows' common power of two multiplies their scores (keys), or lowers their weights against the
// largest so far (values), so it costs the softmax nothing an element.  q enters as float16 times a power of two a row.
//
// Few row tiles: the keys are split over several CTAs, whose results a second kernel joins in a fixed order.
#include "tdt_paged.cuh"
#include "tdt_tc.cuh"

namespace tdt {
namespace {

constexpr int kRows = 128;          // rows of a tile, keys of a tile
constexpr int kMostSplits = 64;
constexpr float kLazy = 8.0f;
// float16 weights start at 2^7 and so stay clear of the type's least numbers; at most 2^15
template <int DT> constexpr float kShift = DT == kF16 ? 7.0f : 0.0f;
constexpr int kUp = 6;              // e4m3 values are held 2^6 up: 448 * 2^6 < 65504
constexpr int kLeastShift = -60;    // of weights against the largest value rows; float16 ends far above

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
  int e8_align;                                // e4m3: bytes that every row is aligned to, 16 or 8
  float *part_o, *part_l;                      // splits > 1: [split][CTA row][DP], [split][CTA row]
};

template <int PT, int DP, bool WIDE> struct TcShape {
  static constexpr bool E8 = PT == kE4M3;
  static constexpr int CHUNKS = DP / 64;
  static constexpr int CHUNK = kRows * 128;          // bytes
  static constexpr int TILE = CHUNKS * CHUNK;
  static constexpr int NS = WIDE || E8 ? 2 : 1;      // streams
  static constexpr int QTILES = WIDE ? 2 : 1;
  static constexpr int SLOTS = DP == 64 ? (NS == 2 ? 8 : 5) : WIDE ? 4 : E8 ? 5 : 2;
  static constexpr int BYTES = (QTILES + SLOTS) * TILE;
  // softmax warps; TMA, MMA, tails, a spare one; e4m3: four that convert
  static constexpr int THREADS = NS * 128 + 128 + (E8 ? 128 : 0);
  static constexpr int CTAS = NS == 2 ? 1 : 2;       // of an SM
  static constexpr int TMEM = NS == 2 ? 512 : 256;   // columns: S and O of each stream
  // registers of a thread: at launch, then of the warpgroups, which adds up to the same:
  // 4 x 128 = 2 x 192 + 40 + 88, 3 x 168 = 2 x 208 + 88, 2 x 128 = 200 + 56
  static constexpr int REGS = E8 ? 128 : WIDE ? 168 : 128;
  static constexpr int SOFTMAX_REGS = E8 ? 192 : WIDE ? 208 : 200;
  static constexpr int OTHER_REGS = E8 ? 40 : WIDE ? 88 : 56;
  static constexpr int CONVERT_REGS = 88;
};

struct TcShared {
  unsigned long long full[8], empty[8], q_full, q_ready, s_full[2], p_ready[2], o_full[2], tail_full, drained;
  unsigned tmem;
  int gave_up, bad_page;
  unsigned k_bytes[8], v_bytes[8];  // e4m3: of a step, a byte for each 32 rows
  float q_scale[2 * kRows];         // e4m3: of each row of q
  float join_m[kRows], join_l[kRows];
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
// 2^(byte - 127) of a byte that is not NaN's
__device__ __forceinline__ float pow2_of(int byte) { return __uint_as_float(byte <= 0 ? 0x00400000u : (unsigned)byte << 23); }
__device__ __forceinline__ unsigned mul_half2(unsigned a, unsigned b) {
  unsigned d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

template <int QT, int PT, int DP, bool WIDE>
__global__ void __launch_bounds__(TcShape<PT, DP, WIDE>::THREADS, TcShape<PT, DP, WIDE>::CTAS)
    paged_tc_kernel(const __grid_constant__ CUtensorMap qm, const __grid_constant__ CUtensorMap km,
                    const __grid_constant__ CUtensorMap vm, const __grid_constant__ CUtensorMap om,
                    const __grid_constant__ TcArgs f) {
  typedef TcShape<PT, DP, WIDE> S;
  constexpr int CT = S::E8 ? (int)kF16 : QT;  // the products' type
  constexpr bool ALT = S::NS == 2 && !WIDE;   // streams take every other key tile
  extern __shared__ unsigned char raw[];
  __shared__ TcShared sh;
  unsigned char *tiles = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  unsigned char *q_tile = tiles, *slots = tiles + S::QTILES * S::TILE;
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
  const int P = f.p.P, per = kRows / P, i0 = tile * S::QTILES * per;
  const int h0 = pack * P, hk = h0 / a.G;
  const NewRows n = new_rows(a.t, b, a.Lq);
  const bool some = i0 < n.n;                                              // else no row takes part
  const int end = some ? n.first + min(n.n, i0 + S::QTILES * per) : 0;     // positions that some row sees
  const int kv_end = n.first + n.n;
  const int2 steps = share_of((end + kRows - 1) / kRows, split, f.p.splits);
  const int begin = steps.x * kRows, T = steps.y - steps.x;                // T tiles of keys from `begin`
  auto frame = [&](int s) { return begin + s * kRows; };
  // 16-bit pages: a warp zeroes what lies past the utterance's end in its last tile of v, which is the last tile
  // loaded: the load then arrives at tail_full, and that warp hands the tile on.
  const bool cut = !S::E8 && T > 0 && begin + T * kRows > kv_end;

  constexpr int kAux = S::NS * 4;  // the first warp past the softmax's: TMA
  const int stream = warp >> 2, r = threadIdx.x & 127;
  int row = 0, head = 0;
  int seen = 0;                    // positions that this thread's row sees
  if (warp < kAux) {
    row = i0 + (WIDE ? stream * per : 0) + r / P;
    head = h0 + r % P;
    seen = row < n.n ? n.first + row + 1 : 0;
  } else if (warp == kAux && lane == 0) {
    for (int i = 0; i < S::SLOTS; ++i) {
      mbar_init(&sh.full[i], S::E8 ? 4 : 1);
      mbar_init(&sh.empty[i], 1);
    }
    mbar_init(&sh.q_full, 1);
    mbar_init(&sh.q_ready, S::QTILES * 128);
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
      arrive_expect_tx(&sh.q_full, S::QTILES * S::TILE);
      for (int t = 0; t < S::QTILES; ++t)
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

  if (warp >= kAux + 4) {
    if constexpr (S::E8) {
      // ---- e4m3 rows to float16 tiles: a warp has 32 rows of each tile, L lanes a row of 16 bytes each
      warpgroup_give_registers<S::CONVERT_REGS>();
      constexpr int L = DP / 16, RPI = 32 / L, N = 32 / RPI;  // rows of a load, loads of a tile
      const int w = warp - (kAux + 4), piece = lane % L, sub = lane / L;
      const int place_mask = (1 << a.t.page_bits) - 1;
      const int left = a.D - piece * 16;  // bytes of this lane's piece
      const unsigned char *base[2] = {static_cast<const unsigned char *>(a.k.data) + hk * a.k.s.h + piece * 16,
                                      static_cast<const unsigned char *>(a.v.data) + hk * a.v.s.h + piece * 16};
      auto lookup = [&](int s) {  // the page of this lane's row of step s
        const int pos = frame(s) + w * 32 + lane;
        int page = -1;
        if (s < T && pos < end) {
          page = page_of(a.t, b, pos);
          if (page < 0) sh.bad_page = 1;
        }
        return page;
      };
      auto bytes_of = [&](int s, int page) {
        if (page < 0) return 0u;
        const int place = (frame(s) + w * 32 + lane) & place_mask;
        return __ldg(a.k.scales + row_at(a.k.ss, page, place, hk)) |
               (unsigned)__ldg(a.v.scales + row_at(a.v.ss, page, place, hk)) << 8;
      };
      uint4 x[N];
      auto load = [&](int s, int page, bool values, int i) {
        const int rr = i * RPI + sub, mine = __shfl_sync(0xffffffffu, page, rr);
        const Strides &st = values ? a.v.s : a.k.s;
        const unsigned char *p = base[values] + mine * st.b + ((frame(s) + w * 32 + rr) & place_mask) * st.l;
        x[i] = make_uint4(0, 0, 0, 0);
        if (mine >= 0) {
          if (f.e8_align == 16) {
            if (left >= 16) x[i] = __ldg(reinterpret_cast<const uint4 *>(p));
            else if (left > 0) {
              const uint2 h = __ldg(reinterpret_cast<const uint2 *>(p));
              x[i].x = h.x;
              x[i].y = h.y;
            }
          } else {
            if (left > 0) {
              const uint2 h = __ldg(reinterpret_cast<const uint2 *>(p));
              x[i].x = h.x;
              x[i].y = h.y;
            }
            if (left >= 16) {
              const uint2 h = __ldg(reinterpret_cast<const uint2 *>(p) + 1);
              x[i].z = h.x;
              x[i].w = h.y;
            }
          }
        }
      };
      int page = lookup(0), next = lookup(1);
      unsigned bytes = bytes_of(0, page);
      if (T > 0)
#pragma unroll
        for (int i = 0; i < N; ++i) load(0, page, false, i);
      bool ok = true;
      for (int s = 0; ok && s < T; ++s) {
        const unsigned next_bytes = bytes_of(s + 1, next);
        const int after = lookup(s + 2);
        const unsigned kb = bytes & 0xffu, vb = bytes >> 8;
        const unsigned kmost = __reduce_max_sync(0xffffffffu, kb == kByteNaN ? 0u : kb);
        const unsigned vmost = __reduce_max_sync(0xffffffffu, vb == kByteNaN ? 0u : vb);
#pragma unroll
        for (int values = 0; values < 2; ++values) {
          const int at = 2 * s + values, slot = at % S::SLOTS;
          ok = __all_sync(0xffffffffu, wait(&sh.empty[slot], ((unsigned)(at / S::SLOTS) & 1) ^ 1)) && ok;
          if (!values && lane == 0) {
            reinterpret_cast<unsigned char *>(&sh.k_bytes[s & 7])[w] = (unsigned char)kmost;
            reinterpret_cast<unsigned char *>(&sh.v_bytes[s & 7])[w] = (unsigned char)vmost;
          }
          // this lane's row's factor, relative to the 32 rows' largest
          const unsigned byte = values ? vb : kb, most = values ? vmost : kmost;
          const float factor = byte == kByteNaN ? NAN : pow2_of(127 + max((int)byte - (int)most + kUp, -40));
          const unsigned mine = pack2<kF16>(factor, factor);
          unsigned char *dst = slots + slot * S::TILE;
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const int rr = i * RPI + sub, at_row = w * 32 + rr;
            const unsigned by = __shfl_sync(0xffffffffu, mine, rr);
            const unsigned in[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
            unsigned h[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              h[2 * k] = mul_half2(e4m3x2_to_half2(in[k] & 0xffffu), by);
              h[2 * k + 1] = mul_half2(e4m3x2_to_half2(in[k] >> 16), by);
            }
            // 16 elements are two 16-byte units of a row; lanes of the second chunk start with the other one, so that
            // a row's eight lanes meet different banks
            const int u = piece % 4 * 2, swap = piece / 4;
            unsigned char *line = dst + piece / 4 * S::CHUNK + at_row * 128;
            const uint4 lo = make_uint4(h[0], h[1], h[2], h[3]), hi = make_uint4(h[4], h[5], h[6], h[7]);
            *reinterpret_cast<uint4 *>(line + (((u + swap) ^ (at_row & 7)) * 16)) = swap ? hi : lo;
            *reinterpret_cast<uint4 *>(line + (((u + 1 - swap) ^ (at_row & 7)) * 16)) = swap ? lo : hi;
            if (values)
              load(s + 1, next, false, i);
            else
              load(s, page, true, i);
          }
          fence_async_shared();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.full[slot]);
        }
        page = next;
        next = after;
        bytes = next_bytes;
      }
    }
  } else if (warp >= kAux) {
    warpgroup_give_registers<S::OTHER_REGS>();  // to the softmax warps, which hold a row of scores
    if (warp == kAux && some && T == 0) wait(&sh.q_full, 0);  // nobody else does
    if constexpr (!S::E8) {
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
    }
    if (warp == kAux + 1 && T > 0 && elect_one()) {
      constexpr unsigned i_s = mma_desc<CT>(kRows, false), i_o = mma_desc<CT>(DP, true);
      const unsigned q_addr = smem_u32(q_tile), s_addr = smem_u32(slots);
      bool ok = wait(S::E8 ? &sh.q_ready : &sh.q_full, 0);
      auto loaded = [&](int at) {
        ok = ok && wait(&sh.full[at % S::SLOTS], (unsigned)(at / S::SLOTS) & 1);
      };
      auto scores = [&](int w, int at) {  // S_w = Q_w K^T
        tc_fence_after();
        if (!ok) return;
        const int slot = at % S::SLOTS;
        mma_rows<DP>(tmem + w * kRows, q_addr + (WIDE ? w * S::TILE : 0), S::CHUNK, s_addr + slot * S::TILE, S::CHUNK,
                     i_s, false);
        mma_commit(&sh.s_full[w]);
        if (ALT || w == S::NS - 1) mma_commit(&sh.empty[slot]);
      };
      auto values = [&](int w, int k, int at, bool last) {  // O_w += P_w V, the stream's k-th
        const int slot = at % S::SLOTS;
        ok = ok && wait(&sh.p_ready[w], k & 1);
        tc_fence_after();
        if (!ok) return;
        mma_across<kRows>(tmem + S::NS * kRows + w * DP, tmem + w * kRows, s_addr + slot * S::TILE, S::CHUNK, i_o, k > 0);
        if (ALT || w == S::NS - 1) mma_commit(&sh.empty[slot]);
        if (last) mma_commit(&sh.o_full[w]);
      };
      if constexpr (ALT) {
        for (int s = 0; s < min(2, T); ++s) {
          loaded(2 * s);
          scores(s, 2 * s);
        }
        for (int s = 0; ok && s < T; ++s) {
          loaded(2 * s + 1);
          values(s & 1, s >> 1, 2 * s + 1, s + 2 >= T);
          if (s + 2 < T) {
            loaded(2 * s + 4);
            scores(s & 1, 2 * s + 4);
          }
        }
      } else {
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
    int top_e = 0;                    // e4m3: the largest byte of value rows so far; O is in units of 2^(top_e - 127 - kUp)
    const bool alive = seen > 0;
    const bool used = __any_sync(0xffffffffu, alive);  // warps without a row that takes part only pass the tiles on
    const int T_own = ALT ? (T - stream + 1) / 2 : T;
    bool ok = true;
    float c = a.scale * kLog2e;
    if constexpr (S::E8) {
      if (some) {
        ok = wait(&sh.q_full, 0);
        if (WIDE || stream == 0) {
          unsigned char *line = q_tile + stream * S::TILE + r * 128;
          float up = 1.0f;
          if (QT == kBF16 && ok) {  // a row as float16 times a power of two: its largest becomes at most 2^15
            unsigned most = 0;
#pragma unroll
            for (int k = 0; k < S::CHUNKS * 8; ++k) {
              const uint4 v = *reinterpret_cast<const uint4 *>(line + k / 8 * S::CHUNK + (k % 8) * 16);
              const unsigned x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int y = 0; y < 4; ++y) most = max(most, max(x[y] << 16 & 0x7fff0000u, x[y] & 0x7fff0000u));
            }
            const int e = min(max((int)(most >> 23) - 127 - 14, -110), 113);
            const float down = __uint_as_float((unsigned)(127 - e) << 23);
            up = __uint_as_float((unsigned)(127 + e) << 23);
#pragma unroll
            for (int k = 0; k < S::CHUNKS * 8; ++k) {
              uint4 *at = reinterpret_cast<uint4 *>(line + k / 8 * S::CHUNK + (k % 8) * 16);
              const uint4 v = *at;
              unsigned x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int y = 0; y < 4; ++y)
                x[y] = pack2<kF16>(__uint_as_float(x[y] << 16) * down, __uint_as_float(x[y] & 0xffff0000u) * down);
              *at = make_uint4(x[0], x[1], x[2], x[3]);
            }
          }
          sh.q_scale[stream * kRows + r] = up * (1.0f / (1 << kUp));
          fence_async_shared();
          mbar_arrive(&sh.q_ready);
        }
        ok = wait(&sh.q_ready, 0) && ok;
        c *= sh.q_scale[(WIDE ? stream * kRows : 0) + r];
      }
    }
    for (int k = 0; k < T_own; ++k) {
      const int s = ALT ? 2 * k + stream : k;
      ok = wait(&sh.s_full[stream], k & 1) && ok;
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
      // of each 32 keys: the factor of scores, and what lowers their weights
      float cg[S::E8 ? 4 : 1], lower[S::E8 ? 4 : 1];
      int most_e = top_e;
      if constexpr (S::E8) {
        const unsigned kb = sh.k_bytes[s & 7], vb = sh.v_bytes[s & 7];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          cg[i] = fmaxf(c * pow2_of(kb >> (8 * i) & 0xff), 1e-37f);  // above 0: it multiplies -inf where keys are masked
          most_e = max(most_e, (int)(vb >> (8 * i) & 0xff));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) lower[i] = (float)max((int)(vb >> (8 * i) & 0xff) - most_e, kLeastShift);
      } else {
        cg[0] = c;
        lower[0] = 0.0f;
      }
      tmem_wait_ld();
      if (masked) {
        const int from = seen - j0;
#pragma unroll
        for (int i = 0; i < 128; ++i)
          if (i >= from) x[i >> 5][i & 31] = 0xff800000u;  // -inf
      }
      float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int i = 0; i < 32; i += 2)
#pragma unroll
        for (int y = 0; y < 4; ++y) m[y] = max3(m[y], __uint_as_float(x[y][i]), __uint_as_float(x[y][i + 1]));
      float top;
      if constexpr (S::E8)
        top = fmaxf(fmaxf(m[0] * cg[0], m[1] * cg[1]), fmaxf(m[2] * cg[2], m[3] * cg[3]));
      else
        top = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])) * c;
      const bool grow = alive && top > ref + (kLazy + kShift<CT>);  // from -inf: any score
      if (__any_sync(0xffffffffu, grow || most_e > top_e)) {
        const float now = grow ? top - kShift<CT> : ref;
        float scale = grow ? fast_exp2(ref - now) : 1.0f;
        l *= scale;
        if (S::E8 && top_e > 0) scale *= pow2_nonpos(top_e - most_e);
        if (k > 0) {  // the products up to this stream's last tile are done: S of this one came after them
          unsigned o[32];
#pragma unroll
          for (int i = 0; i < DP / 32; ++i) {
            tmem_ld32(o_col + i * 32, o);
            tmem_wait_ld();
#pragma unroll
            for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * scale);
            tmem_st32(o_col + i * 32, o);
          }
        }
        ref = now;
        top_e = most_e;
      }
      const float neg = ref == -INFINITY ? 0.0f : -ref;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        unsigned p[32];
        float2 sum0 = make_float2(0.0f, 0.0f), sum1 = sum0;
        if constexpr (S::E8) {
          exp_pack<CT>(x[2 * i], cg[2 * i], neg + lower[2 * i], p, 0, sum0);
          exp_pack<CT>(x[2 * i + 1], cg[2 * i + 1], neg + lower[2 * i + 1], p, 16, sum1);
          l += (sum0.x + sum0.y) * pow2_of(127 - (int)lower[2 * i]) + (sum1.x + sum1.y) * pow2_of(127 - (int)lower[2 * i + 1]);
        } else {
          exp_pack<CT>(x[2 * i], c, neg, p, 0, sum0);
          exp_pack<CT>(x[2 * i + 1], c, neg, p, 16, sum1);
          sum0 = add2(sum0, sum1);
          l += sum0.x + sum0.y;
        }
        tmem_st32(s_col + i * 32, p);
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&sh.p_ready[stream]);
    }
    if (T_own > 0 && ok) ok = wait(&sh.o_full[stream], 0);
    if (T == 0 && some) ok = wait(&sh.q_full, 0);  // the tile's memory is used below
    __syncwarp();
    tc_fence_after();
    if (!alive) l = 0.0f;
    float unit = S::E8 ? pow2_of(top_e) : 1.0f;
    if constexpr (S::E8) unit *= 1.0f / (1 << kUp);
    unsigned char *out_tile = q_tile + (WIDE ? stream * S::TILE : 0);  // every product with q is done
    float weight_own = 1.0f, weight_other = 0.0f;
    float *other = reinterpret_cast<float *>(slots);  // the second stream's O, column by column
    if constexpr (ALT) {
      // Both streams have waited for their products before this barrier, so the slots are free behind it.
      named_barrier<256>(3);
      if (stream == 1) {
        sh.join_m[r] = T_own > 0 && ok ? ref : -INFINITY;
        sh.join_l[r] = ok ? (T_own > 0 ? l : 0.0f) : NAN;
        if (T_own > 0)
#pragma unroll
          for (int i = 0; i < DP / 32; ++i) {
            unsigned o[32];
            tmem_ld32(o_col + i * 32, o);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) other[(i * 32 + k) * kRows + r] = __uint_as_float(o[k]) * unit;
          }
        tc_fence_before();
      }
      named_barrier<256>(3);
      if (stream == 0) {
        const float m2 = sh.join_m[r], l2 = sh.join_l[r], both = fmaxf(ref, m2);
        if (both > -INFINITY) {
          weight_own = fast_exp2(ref - both);
          weight_other = T > 1 ? fast_exp2(m2 - both) : 0.0f;
          l = l * weight_own + l2 * weight_other;
          ref = both;
        }
        if (l2 != l2) l = NAN;
        if (!alive) l = 0.0f;
      }
    }
    if (!ALT || stream == 0) {
      const bool bad = n.bad || !ok || *reinterpret_cast<volatile int *>(&sh.gave_up) || *reinterpret_cast<volatile int *>(&sh.bad_page);
      const long long tile_at = (long long)split * f.p.tiles * f.p.packs * a.B + cta;  // of a partial result
      const int slot_row = WIDE ? (int)threadIdx.x : r;
      if (row < a.Lq) {
        const float total = bad ? NAN : l == 0.0f ? -INFINITY : ref + log2f(l);
        if (f.p.splits > 1)
          f.part_l[tile_at * (S::QTILES * kRows) + slot_row] = total;
        else if (a.lse)
          a.lse[(b * a.H + head) * a.Lq + row] = total * kLn2;
      }
      const float inv = bad ? NAN : l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
      for (int i = 0; i < DP / 32; ++i) {
        unsigned o[32];
        if (T > 0) {
          tmem_ld32(o_col + i * 32, o);
          tmem_wait_ld();
        }
        float v[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          float x = __uint_as_float(o[k]);
          if constexpr (S::E8) x *= unit;
          if constexpr (ALT) {
            x *= weight_own;
            if (T > 1) x = fmaf(weight_other, other[(i * 32 + k) * kRows + r], x);
          }
          v[k] = bad ? NAN : l == 0.0f ? 0.0f : x * inv;
        }
        if (f.p.splits == 1) {
          stage32<QT>(out_tile, S::CHUNK, r, i * 32, v);
        } else if (row < a.Lq) {
          store_columns(f.part_o + (tile_at * DP + i * 32) * (S::QTILES * kRows) + slot_row, S::QTILES * kRows, v);
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

TcPlan plan(long long B, long long Lq, long long most, int H, int G, bool e8) {
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
  long long s = ctas > 0 ? (p.wide || e8 ? 1 : 2) * kSMs / ctas : 1;
  if (s > steps / 4) s = steps / 4;
  if (s > kMostSplits) s = kMostSplits;
  p.splits = s < 2 || steps - steps / s < 12 ? 1 : (int)s;
  return p;
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }
size_t part_rows(const TcPlan &p, long long B) {
  return p.splits == 1 ? 0 : (size_t)B * p.packs * p.tiles * p.splits * (p.wide ? 2 : 1) * kRows;
}

template <int QT, int PT, int DP, bool WIDE>
cudaError_t launch(const TcArgs &f, const TensorMap &q, const TensorMap &k, const TensorMap &v, const TensorMap &o,
                   cudaStream_t stream) {
  typedef TcShape<PT, DP, WIDE> S;
  const size_t smem = S::BYTES + 1024;
  cudaError_t e = prepare_tc_kernel(reinterpret_cast<const void *>(paged_tc_kernel<QT, PT, DP, WIDE>), smem, S::REGS);
  if (e != cudaSuccess) return e;
  const long long ctas = f.a.B * f.p.packs * f.p.tiles;
  paged_tc_kernel<QT, PT, DP, WIDE>
      <<<(unsigned)(ctas * f.p.splits), S::THREADS, smem, stream>>>(q.map, k.map, v.map, o.map, f);
  e = cudaGetLastError();
  if (e != cudaSuccess || f.p.splits == 1) return e;
  const int rows = S::QTILES * kRows;
  return launch_follower(paged_join_kernel<QT, DP>, dim3((unsigned)(ctas * (rows / 32) * (DP / 32))), 256, 0, stream, f, rows);
}
template <int QT, int PT>
cudaError_t by_shape(const TcArgs &f, const TensorMap &q, const TensorMap &k, const TensorMap &v, const TensorMap &o,
                     cudaStream_t s) {
  if (f.a.D > 64)
    return f.p.wide ? launch<QT, PT, 128, true>(f, q, k, v, o, s) : launch<QT, PT, 128, false>(f, q, k, v, o, s);
  return f.p.wide ? launch<QT, PT, 64, true>(f, q, k, v, o, s) : launch<QT, PT, 64, false>(f, q, k, v, o, s);
}

int e8_alignment(const PagedArgs &a) {
  uintptr_t x = 0;
  for (const Pages *p : {&a.k, &a.v}) x |= (uintptr_t)p->data | (uintptr_t)p->s.b | (uintptr_t)p->s.l | (uintptr_t)p->s.h;
  return x % 16 == 0 ? 16 : x % 8 == 0 ? 8 : 1;
}

}  // namespace

bool paged_tc_takes(int dtype, int D) { return dtype != kF32 && D <= 128 && D % 8 == 0; }

size_t paged_tc_workspace(long long B, long long Lq, long long most, int H, int Hkv, int D, int cache_dtype) {
  const size_t rows = part_rows(plan(B, Lq, most, H, H / Hkv, cache_dtype == kE4M3), B);
  return align256(rows * (D <= 64 ? 64 : 128) * 4) + align256(rows * 4);
}

bool paged_tc_fits(const PagedArgs &a, int dtype, int cache_dtype) {
  if (!paged_tc_takes(dtype, a.D)) return false;
  auto rows_fit = [&](const void *p, const Strides &s) { return map_fits(dtype, p, a.B, a.Lq, a.H, a.D, s.b, s.l, s.h); };
  if (!rows_fit(a.q, a.sq) || !rows_fit(a.out, a.so) || (attn_row_pack(a.G) > 1 && a.sq.h == 0)) return false;
  if (cache_dtype == kE4M3) return e8_alignment(a) >= 8;
  auto pages_fit = [&](const Pages &p) {
    return map_fits(dtype, p.data, a.t.n_pages, 1LL << a.t.page_bits, a.Hkv, a.D, p.s.b, p.s.l, p.s.h);
  };
  return a.t.page_bits >= 3 && pages_fit(a.k) && pages_fit(a.v);
}

cudaError_t launch_paged_tc(const PagedArgs &a, int dtype, int cache_dtype, void *workspace, cudaStream_t stream) {
  TcArgs f = {};
  f.a = a;
  const bool e8 = cache_dtype == kE4M3;
  const long long page_size = 1LL << a.t.page_bits;
  f.p = plan(a.B, a.Lq, (long long)a.t.max_pages << a.t.page_bits, a.H, a.G, e8);
  const size_t rows = part_rows(f.p, a.B);
  f.part_o = static_cast<float *>(workspace);
  f.part_l = reinterpret_cast<float *>(static_cast<char *>(workspace) + align256(rows * (a.D <= 64 ? 64 : 128) * 4));
  TensorMap q, k = {}, v = {}, o;
  bool ok = encode_map(&o, a.out, dtype, a.B, a.Lq, a.H, a.D, a.so.b, a.so.l, a.so.h, f.p.P, kRows / f.p.P) &&
            encode_map(&q, a.q, dtype, a.B, a.Lq, a.H, a.D, a.sq.b, a.sq.l, a.sq.h, f.p.P, kRows / f.p.P);
  if (e8) {
    f.e8_align = e8_alignment(a);
  } else {
    const int box = (int)(page_size < kRows ? page_size : kRows);
    ok = ok &&
         encode_map(&k, a.k.data, dtype, a.t.n_pages, page_size, a.Hkv, a.D, a.k.s.b, a.k.s.l, a.k.s.h, 1, box) &&
         encode_map(&v, a.v.data, dtype, a.t.n_pages, page_size, a.Hkv, a.D, a.v.s.b, a.v.s.l, a.v.s.h, 1, box);
  }
  if (!ok) return cudaErrorInvalidValue;
  f.q_b = q.b_mul;
  f.q_h = q.h_mul;
  f.o_b = o.b_mul;
  f.o_h = o.h_mul;
  f.k_p = k.b_mul;
  f.k_h = k.h_mul;
  f.v_p = v.b_mul;
  f.v_h = v.h_mul;
  if (e8)
    return dtype == kF16 ? by_shape<kF16, kE4M3>(f, q, k, v, o, stream) : by_shape<kBF16, kE4M3>(f, q, k, v, o, stream);
  return dtype == kF16 ? by_shape<kF16, kF16>(f, q, k, v, o, stream) : by_shape<kBF16, kBF16>(f, q, k, v, o, stream);
}

}  // namespace tdt
