// tdt_paged_step.cu -- causal attention of few query rows over a paged cache (a decoding step, a small beam, a few drafted
// tokens): float16 and bfloat16 queries over pages of their own type or of e4m3, heads up to 128.
//
// With R = Lq * G rows a key head (G query heads share it), the work is to read k and v once.  A warp multiplies tiles of
// 16 keys in the pieces that its lanes load, by mma.sync m16n8k16, which adds over the lanes by itself, where
// products on the CUDA cores take R / 2 instructions an element and the exchange of partial scores.  (A tcgen05 product has 128 rows; its operands would have to go through shared memory first.)
//   S = Q K^T     A = q, in registers for the whole walk; B = k: lane (g, t) has key g of 8 and a quarter of its elements.
//                 A contraction may take its elements in any order, so a lane's quarter is what its 16-byte copies bring.
//   O^T = V^T P^T A = v: lane (g, t) holds keys 2t, 2t+1, 2t+8, 2t+9 and an eighth of their elements, two keys to a register by a
//                 byte permutation; B = p: exactly what S leaves in the lane (query g, keys 2t, 2t+1).
// Rows 8 to 15 of A and a second B take up to 16 query rows; more rows: more CTAs, which mostly find k and v in L2.
//
// e4m3 pages: values become float16 exactly, q is put into float16 by a power of two a row, a key's power of two
// multiplies its scores and a value row's its weight, relative to the largest so far (E); sums stay in float32.
// The reference m of a row moves only when its maximum has grown by 8 (in base 2), so O is rescaled rarely.
//
// A cluster of S CTAs has one (utterance, key head, group of rows); its warps take the keys in turns.  Each warp has 16 KB of
// shared memory for turns in flight, which TMA fills, a box a page, swizzled so that the lanes' pieces lie in different banks.
// Warps and then CTAs (over distributed shared memory) are joined in a fixed order.
//
// Bound by memory: 64 x 1 x 6,000 bfloat16, 32 heads on 8 of 128: 254 us, 6.2 TB/s of 6.8 measured; e4m3, 128 utterances: 292 us,
// 5.4 TB/s (issue slots 44 %, the rest waits for data: three CTAs an SM by shared memory).  64 ragged x 750, 16 heads of 64,
// float16: 34 us, short walks.  1 x 40, 8 heads of 64: 6 us, latency.  The same with rows loaded to registers a turn ahead (8 KB in
// flight a warp): 379 us for 292, 272 for 254, and 39 for 18 at 1 x 8,000, 8 heads; with cp.async into the ring: 381, 364 and 22.
#include <cooperative_groups.h>

#include <algorithm>

#include "tdt_paged.cuh"
#include "tdt_tc.cuh"

namespace tdt {
namespace {

namespace cg = cooperative_groups;

constexpr int kWarps = 4;
constexpr float kLazy = 8.0f;

struct StepArgs {
  PagedArgs a;
  int splits;  // CTAs of a cluster
  int groups;  // clusters that share the rows of a key head
  int q_whole; // q's rows suit 8-byte loads
  int k_p, k_h, v_p, v_h;  // 0 for repeated axes
};

// d += a b, 16 x 8 x 16, float32 sums; F16: float16 operands, else bfloat16
template <bool F16>
__device__ __forceinline__ void mma16(float (&d)[4], const unsigned (&a)[4], unsigned b0, unsigned b1) {
  if (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int QT, int PT, int DP, int RT> struct Shape {
  static constexpr bool E8 = PT == kE4M3;
  static constexpr bool F16 = E8 || PT == kF16;      // the products' type
  static constexpr int ES = E8 ? 1 : 2;
  static constexpr int KT = E8 || DP == 64 ? 32 : 16;  // keys of a turn
  static constexpr int NT = KT / 8;                  // tiles of 8 keys
  static constexpr int KL = DP * ES / 64;            // 16-byte loads of a key's quarter (64 bytes an instruction and key)
  static constexpr int VB = DP * ES / 8 >= 16 ? 16 : DP * ES / 8;  // bytes of a load of a value row's eighth
  static constexpr int VL = DP * ES / 8 / VB;
  static constexpr int KSTEPS = DP / 16;
  static constexpr int MTILES = DP / 16;
  static constexpr int ROW = DP * ES < 128 ? DP * ES : 128;  // bytes of a row in a box
  static constexpr int CHUNKS = DP * ES / ROW;       // boxes across a head
  static constexpr int CHUNK = KT * ROW;
  static constexpr int SIDE = CHUNKS * CHUNK;        // k or v of a turn
  static constexpr int TURN = 2 * SIDE;
  static constexpr int STAGES = 16384 / TURN;        // turns in flight
  static constexpr int CTAS = RT == 1 ? 3 : 2;       // of an SM, by shared memory
};

// The first of the four elements that lane t of a group contributes to step i of the contraction over a head.
template <int ES> __device__ __forceinline__ constexpr int step_element(int i, int t) {
  return ES == 1 ? i / 4 * 64 + t * 16 + i % 4 * 4 : i / 2 * 32 + t * 8 + i % 2 * 4;
}
// The first of the two elements that lane group g contributes to tile i of 16 elements of a value row.
template <int ES, int VB> __device__ __forceinline__ constexpr int tile_element(int i, int g) {
  constexpr int per = VB / ES / 2;  // tiles of a load
  return i / per * (8 * VB / ES) + g * (VB / ES) + i % per * 2;
}

template <int QT, int PT, int DP, int RT>
__global__ void __launch_bounds__(kWarps * 32, Shape<QT, PT, DP, RT>::CTAS)
    paged_step_kernel(const __grid_constant__ CUtensorMap km, const __grid_constant__ CUtensorMap vm,
                      const __grid_constant__ StepArgs f) {
  typedef Shape<QT, PT, DP, RT> S;
  typedef typename Elem<QT>::T E;
  constexpr int R = 8 * RT;
  constexpr float kShift = S::F16 ? 7.0f : 0.0f;  // float16 weights start at 2^7, at most 2^15
  const PagedArgs &a = f.a;
  // turns in flight of each warp; after the walk, the warps' partial results
  extern __shared__ unsigned char raw[];
  unsigned char *fifo = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  float(*part_o)[R][DP + 4] = reinterpret_cast<float(*)[R][DP + 4]>(fifo);
  __shared__ float part_m[kWarps][R], part_l[kWarps][R];
  __shared__ float cta_m[R], cta_l[R];
  __shared__ int cta_bad;
  __shared__ __align__(16) float cta_o[R][DP];
  __shared__ __align__(8) float key_f[kWarps][32], value_f[kWarps][32];  // e4m3: of a turn's rows
  __shared__ unsigned long long full[kWarps][S::STAGES][2];  // k, v of a turn have landed
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const unsigned cluster_id = blockIdx.x / f.splits, unit = cluster_id / f.groups;  // = b * Hkv + hk
  const int split = blockIdx.x % f.splits, hk = unit % a.Hkv;
  const long long b = unit / a.Hkv;
  const NewRows n = new_rows(a.t, b, a.Lq);
  const int row0 = cluster_id % f.groups * R;  // Lq * G < 2^31
  const int rows = min(R, a.Lq * a.G - row0);  // row r: query (row0 + r) / G, head hk * G + (row0 + r) % G
  const int used = min(n.n, (row0 + rows - 1) / a.G + 1);  // queries that take part, of those up to this group's last
  const int end = used > row0 / a.G ? n.first + used : 0;  // positions that some row sees
  __shared__ int gave_up;
  if (threadIdx.x == 0) cta_bad = gave_up = 0;
  if (lane == 0) {
    for (int i = 0; i < S::STAGES; ++i) {
      mbar_init(&full[warp][i][0], 1);
      mbar_init(&full[warp][i][1], 1);
    }
    fence_mbar_init_cluster();
  }
  __syncthreads();
  const Waiter wait{&gave_up};

  // q: rows g and g + 8, in the order of the contraction's steps
  unsigned q[S::KSTEPS][RT][2];
  float c[RT];
  int last[RT];  // the last position that the row sees
#pragma unroll
  for (int h = 0; h < RT; ++h) {
    const int r = g + 8 * h, i = (row0 + r) / a.G;
    const bool live = r < rows && i < n.n;
    last[h] = live ? n.first + i : -1;
    c[h] = a.scale * kLog2e;
    const E *src = static_cast<const E *>(a.q) + b * a.sq.b + i * a.sq.l + (hk * a.G + (row0 + r) % a.G) * a.sq.h;
#pragma unroll
    for (int x = 0; x < S::KSTEPS; ++x) {
      const int d = step_element<S::ES>(x, t);
      uint2 w = make_uint2(0, 0);
      if (live && d < a.D) {
        if (f.q_whole) {
          w = __ldg(reinterpret_cast<const uint2 *>(src + d));
        } else {
          const unsigned short *e = reinterpret_cast<const unsigned short *>(src + d);
          w = make_uint2(e[0] | (unsigned)e[1] << 16, e[2] | (unsigned)e[3] << 16);
        }
      }
      q[x][h][0] = w.x;
      q[x][h][1] = w.y;
    }
    if (QT == kBF16 && S::F16) {  // into float16 by a power of two: the row's largest becomes at most 2^15
      unsigned top = 0;
#pragma unroll
      for (int x = 0; x < S::KSTEPS; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y) top = max(top, max(q[x][h][y] << 16 & 0x7fff0000u, q[x][h][y] & 0x7fff0000u));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e = min(max((int)(top >> 23) - 127 - 14, -110), 113);
      const float down = __uint_as_float((unsigned)(127 - e) << 23);
      c[h] *= __uint_as_float((unsigned)(127 + e) << 23);
#pragma unroll
      for (int x = 0; x < S::KSTEPS; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y)
          q[x][h][y] = pack2<kF16>(__uint_as_float(q[x][h][y] << 16) * down, __uint_as_float(q[x][h][y] & 0xffff0000u) * down);
    }
  }
  const int least = __reduce_min_sync(0xffffffffu, min(last[0] < 0 ? 0x7fffffff : last[0], last[RT - 1] < 0 ? 0x7fffffff : last[RT - 1]));

  float o[S::MTILES][RT][4], m[RT], l[RT];
#pragma unroll
  for (int h = 0; h < RT; ++h) {
    m[h] = -INFINITY;
    l[h] = 0.0f;
#pragma unroll
    for (int x = 0; x < S::MTILES; ++x)
#pragma unroll
      for (int y = 0; y < 4; ++y) o[x][h][y] = 0.0f;
  }
  int top_e = -1;  // e4m3: the largest byte of the value rows so far, -1: none; o is in units of 2^(top_e - 127)
  bool bad = false;

  const int place_mask = (1 << a.t.page_bits) - 1, box_rows = min(1 << a.t.page_bits, S::KT);
  auto lookup = [&](int x) {  // the page of this lane's position (of KT) of turn x
    const int pos = x * S::KT + lane % S::KT;
    if (pos >= end) return -1;
    const int page = page_of(a.t, b, pos);
    bad |= page < 0;
    return page;
  };
  // k (or v) of turn x, whose page is `id`: a box for each page, by the lane of its first row.  A box without a page is one
  // past the tensor's end, which TMA fills with zeros; what lies past the utterance's end in its last page comes along.
  unsigned char *mine = fifo + warp * (S::STAGES * S::TURN);
  auto copy = [&](int x, int stage, int id, bool values) {
    unsigned long long *bar = &full[warp][stage][values];
    if (lane == 0) arrive_expect_tx(bar, S::SIDE);
    __syncwarp();
    if (lane < S::KT && lane % box_rows == 0) {
      const int page = id < 0 ? a.t.n_pages : id * (values ? f.v_p : f.k_p);
      const int place = (x * S::KT + lane) & place_mask;
#pragma unroll
      for (int i = 0; i < S::CHUNKS; ++i)
        tma_load_4d(values ? &vm : &km, mine + stage * S::TURN + (values ? S::SIDE : 0) + i * S::CHUNK + lane * S::ROW, bar,
                    i * (S::ROW / S::ES), hk * (values ? f.v_h : f.k_h), place, page);
    }
  };
  // where 16-byte unit u of a row lies
  auto unit_at = [](int row, int u) { return row * S::ROW + (S::ROW == 128 ? u ^ (row & 7) : u ^ (row >> 1 & 3)) * 16; };
  unsigned bytes = 0;  // e4m3: this lane's position's bytes of k and v
  auto load_bytes = [&](int x, int id) {
    if (!S::E8) return 0u;
    const int place = (x * S::KT + lane) & place_mask;
    return id < 0 ? 0u
                  : __ldg(a.k.scales + row_at(a.k.ss, id, place, hk)) |
                        (unsigned)__ldg(a.v.scales + row_at(a.v.ss, id, place, hk)) << 8;
  };

  const int turns = (end + S::KT - 1) / S::KT, step = f.splits * kWarps;
  int turn = split * kWarps + warp;
  // copies go STAGES turns ahead, and pages are looked up a turn before that
  int ids[S::STAGES + 1];
#pragma unroll
  for (int x = 0; x <= S::STAGES; ++x) ids[x] = lookup(turn + x * step);
#pragma unroll
  for (int x = 0; x < S::STAGES; ++x)
    if (turn + x * step < turns) {
      copy(turn + x * step, x, ids[x], false);
      copy(turn + x * step, x, ids[x], true);
    }
  bytes = load_bytes(turn, ids[0]);
  int stage = 0, parity = 0;
  bool ok = true;
  for (; turn < turns; turn += step) {
    const int base = turn * S::KT, ahead = turn + S::STAGES * step;
    const bool more = ahead < turns;
    const int after = lookup(ahead + step);
    const unsigned next_bytes = load_bytes(turn + step, ids[1]);
    const unsigned char *k_at = mine + stage * S::TURN, *v_at = k_at + S::SIDE;
    ok = __all_sync(0xffffffffu, wait(&full[warp][stage][0], parity)) && ok;
    // scores: rows g, g + 8; keys 8 j + 2 t, + 1
    float s[S::NT][4];
#pragma unroll
    for (int j = 0; j < S::NT; ++j) {
      s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.0f;
#pragma unroll
      for (int i = 0; i < S::KL; ++i) {
        const uint4 piece = *reinterpret_cast<const uint4 *>(k_at + i * 64 / S::ROW * S::CHUNK + unit_at(8 * j + g, i * 4 % (S::ROW / 16) + t));
        const unsigned w[4] = {piece.x, piece.y, piece.z, piece.w};
#pragma unroll
        for (int y = 0; y < (S::E8 ? 4 : 2); ++y) {
          const int x = i * (S::E8 ? 4 : 2) + y;
          const unsigned qa[4] = {q[x][0][0], RT == 2 ? q[x][RT - 1][0] : 0, q[x][0][1], RT == 2 ? q[x][RT - 1][1] : 0};
          if constexpr (S::E8)
            mma16<true>(s[j], qa, e4m3x2_to_half2(w[y] & 0xffffu), e4m3x2_to_half2(w[y] >> 16));
          else
            mma16<S::F16>(s[j], qa, w[2 * y], w[2 * y + 1]);
        }
      }
    }
    if constexpr (S::E8) {
      const unsigned kb = bytes & 0xffu, vb = bytes >> 8;
      const int most = (int)__reduce_max_sync(0xffffffffu, vb == kByteNaN ? 0u : vb);
      if (most > top_e) {
        if (top_e >= 0) {
          const float down = pow2_nonpos(top_e - most);
#pragma unroll
          for (int x = 0; x < S::MTILES; ++x)
#pragma unroll
            for (int h = 0; h < RT; ++h)
#pragma unroll
              for (int y = 0; y < 4; ++y) o[x][h][y] *= down;
        }
        top_e = most;
      }
      __syncwarp();
      key_f[warp][lane] = scale_of(kb);
      value_f[warp][lane] = vb == kByteNaN ? NAN : pow2_nonpos((int)vb - top_e);
      __syncwarp();
    }
    __syncwarp();  // every lane has read the keys
    if (more) copy(ahead, stage, ids[S::STAGES], false);
    // weights
    float top[RT];
#pragma unroll
    for (int h = 0; h < RT; ++h) {
      top[h] = -INFINITY;
      const bool masked = base + S::KT - 1 > least;
#pragma unroll
      for (int j = 0; j < S::NT; ++j) {
        float2 kf = make_float2(c[h], c[h]);
        if constexpr (S::E8) {
          const float2 two = *reinterpret_cast<const float2 *>(&key_f[warp][8 * j + 2 * t]);
          kf = make_float2(two.x * c[h], two.y * c[h]);
        }
        s[j][2 * h] *= kf.x;
        s[j][2 * h + 1] *= kf.y;
        if (masked) {
          const int key = base + 8 * j + 2 * t;
          if (key > last[h]) s[j][2 * h] = -INFINITY;
          if (key + 1 > last[h]) s[j][2 * h + 1] = -INFINITY;
        }
        top[h] = fmaxf(top[h], fmaxf(s[j][2 * h], s[j][2 * h + 1]));
      }
    }
    bool grow = false;
#pragma unroll
    for (int h = 0; h < RT; ++h) grow |= top[h] > m[h] + (kLazy + kShift);  // from -inf: any score
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int h = 0; h < RT; ++h) {
        top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
        top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2));
        const bool up = top[h] > m[h] + (kLazy + kShift);
        const float now = up ? top[h] - kShift : m[h], down = up ? fast_exp2(m[h] - now) : 1.0f;
        m[h] = now;
        l[h] *= down;
        // a lane's columns of o are the queries 2t, 2t + 1
        const float f0 = __shfl_sync(0xffffffffu, down, 8 * t), f1 = __shfl_sync(0xffffffffu, down, 8 * t + 4);
#pragma unroll
        for (int x = 0; x < S::MTILES; ++x) {
          o[x][h][0] *= f0;
          o[x][h][1] *= f1;
          o[x][h][2] *= f0;
          o[x][h][3] *= f1;
        }
      }
    }
    unsigned p[S::NT][RT];
#pragma unroll
    for (int h = 0; h < RT; ++h) {
      const float ref = m[h] == -INFINITY ? 0.0f : m[h];
#pragma unroll
      for (int j = 0; j < S::NT; ++j) {
        float p0 = fast_exp2(s[j][2 * h] - ref), p1 = fast_exp2(s[j][2 * h + 1] - ref);
        l[h] += p0 + p1;
        if constexpr (S::E8) {
          const float2 two = *reinterpret_cast<const float2 *>(&value_f[warp][8 * j + 2 * t]);
          p0 *= two.x;
          p1 *= two.y;
        }
        p[j][h] = pack2<S::F16 ? (int)kF16 : (int)kBF16>(p0, p1);
      }
    }
    ok = __all_sync(0xffffffffu, wait(&full[warp][stage][1], parity)) && ok;
    const bool cut = base + S::KT > end;  // rows past the end may hold anything: 0 times NaN is NaN
#pragma unroll
    for (int j = 0; j < S::KT / 16; ++j)
#pragma unroll
      for (int i = 0; i < S::VL; ++i) {
        constexpr int W = S::VB / 4;
        unsigned w[4][W];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int key = 16 * j + 2 * t + (y & 1) + (y >> 1) * 8;
          if constexpr (S::VB == 16) {
            const uint4 piece = *reinterpret_cast<const uint4 *>(v_at + i * S::CHUNK + unit_at(key, g));
            w[y][0] = piece.x;
            w[y][1] = piece.y;
            w[y][2] = piece.z;
            w[y][W - 1] = piece.w;
          } else {
            const uint2 piece = *reinterpret_cast<const uint2 *>(v_at + unit_at(key, g / 2) + g % 2 * 8);
            w[y][0] = piece.x;
            w[y][W - 1] = piece.y;
          }
          if (cut && base + key >= end)
#pragma unroll
            for (int z = 0; z < W; ++z) w[y][z] = 0;
        }
#pragma unroll
        for (int z = 0; z < W; ++z) {
#pragma unroll
          for (int half = 0; half < (S::E8 ? 2 : 1); ++half) {
            unsigned va[4];
            if constexpr (S::E8) {
              const int sel = half ? 0x7362 : 0x5140;
              const unsigned lo = __byte_perm(w[0][z], w[1][z], sel), hi = __byte_perm(w[2][z], w[3][z], sel);
              va[0] = e4m3x2_to_half2(lo & 0xffffu);
              va[1] = e4m3x2_to_half2(lo >> 16);
              va[2] = e4m3x2_to_half2(hi & 0xffffu);
              va[3] = e4m3x2_to_half2(hi >> 16);
            } else {
              va[0] = __byte_perm(w[0][z], w[1][z], 0x5410);
              va[1] = __byte_perm(w[0][z], w[1][z], 0x7632);
              va[2] = __byte_perm(w[2][z], w[3][z], 0x5410);
              va[3] = __byte_perm(w[2][z], w[3][z], 0x7632);
            }
            const int x = i * (S::MTILES / S::VL) + z * (S::E8 ? 2 : 1) + half;
#pragma unroll
            for (int h = 0; h < RT; ++h) mma16<S::F16>(o[x][h], va, p[2 * j][h], p[2 * j + 1][h]);
          }
        }
      }
    __syncwarp();
    if (more) copy(ahead, stage, ids[S::STAGES], true);
    bytes = next_bytes;
#pragma unroll
    for (int x = 0; x < S::STAGES; ++x) ids[x] = ids[x + 1];
    ids[S::STAGES] = after;
    if (++stage == S::STAGES) {
      stage = 0;
      parity ^= 1;
    }
  }

  if (!ok)  // copies in flight land before their memory is used for something else
    for (int i = 0; i < S::STAGES; ++i) {
      Waiter::drain(&full[warp][i][0], parity ^ (i < stage));
      Waiter::drain(&full[warp][i][1], parity ^ (i < stage));
    }

  // the warps of a CTA
  __syncthreads();  // the memory of turns in flight is free
  const float unit_f = S::E8 ? scale_of(max(top_e, 0)) : 1.0f;
#pragma unroll
  for (int h = 0; h < RT; ++h) {
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    if (t == 0) {
      part_m[warp][g + 8 * h] = m[h];
      part_l[warp][g + 8 * h] = l[h];
    }
#pragma unroll
    for (int x = 0; x < S::MTILES; ++x) {
      const int d = tile_element<S::ES, S::VB>(x, g);
#pragma unroll
      for (int y = 0; y < 2; ++y)
        *reinterpret_cast<float2 *>(&part_o[warp][8 * h + 2 * t + y][d]) = make_float2(o[x][h][y] * unit_f, o[x][h][y + 2] * unit_f);
    }
  }
  if (bad || !ok) cta_bad = 1;
  __syncthreads();
  for (int x = threadIdx.x; x < R * DP; x += kWarps * 32) {
    const int r = x / DP, d = x % DP;
    float top = -INFINITY, sum = 0.0f, out = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, part_m[w][r]);
    const float ref = top == -INFINITY ? 0.0f : top;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float e = fast_exp2(part_m[w][r] - ref);
      sum += e * part_l[w][r];
      out += e * part_o[w][r][d];
    }
    cta_o[r][d] = out;
    if (d == 0) {
      cta_m[r] = cta_bad ? NAN : top;
      cta_l[r] = sum;
    }
  }
  cg::cluster_group cluster = cg::this_cluster();
  if (f.splits > 1)
    cluster.sync();
  else
    __syncthreads();
  // the CTAs of the cluster: each writes its part of the elements
  for (int x = split * (kWarps * 32) + threadIdx.x; x < rows * DP; x += f.splits * kWarps * 32) {
    const int r = x / DP, d = x % DP;
    float top = -INFINITY, sum = 0.0f, out = 0.0f;
    bool lost = n.bad;
    if (f.splits == 1) {
      top = cta_m[r];
      sum = cta_l[r];
      out = cta_o[r][d];
      lost |= top != top;
    } else {
      for (int i = 0; i < f.splits; ++i) {
        const float x2 = *cluster.map_shared_rank(&cta_m[r], i);
        lost |= x2 != x2;
        top = fmaxf(top, x2);
      }
      const float ref = top == -INFINITY ? 0.0f : top;
      for (int i = 0; i < f.splits; ++i) {
        const float e = fast_exp2(*cluster.map_shared_rank(&cta_m[r], i) - ref);
        sum += e * *cluster.map_shared_rank(&cta_l[r], i);
        out += e * *cluster.map_shared_rank(&cta_o[r][d], i);
      }
    }
    const int i = (row0 + r) / a.G, h = hk * a.G + (row0 + r) % a.G;
    const bool live = i < n.n;
    if (d < a.D)
      static_cast<E *>(a.out)[b * a.so.b + i * a.so.l + h * a.so.h + d] =
          Elem<QT>::from_float(lost ? NAN : live ? out / sum : 0.0f);
    if (d == 0 && a.lse)
      a.lse[(b * a.H + h) * a.Lq + i] = lost ? NAN : live ? (top + log2f(sum)) * kLn2 : -INFINITY;
  }
  if (f.splits > 1) cluster.sync();  // nobody leaves while its memory may be read
}

template <int QT, int PT, int DP, int RT> cudaError_t launch(StepArgs f, cudaStream_t stream) {
  typedef Shape<QT, PT, DP, RT> S;
  const PagedArgs &a = f.a;
  TensorMap k, v;
  const int box = (int)std::min<long long>(1LL << a.t.page_bits, S::KT);
  auto encode = [&](TensorMap *m, const Pages &p) {
    return encode_rows(m, p.data, PT == kE4M3 ? 1 : 2, a.t.n_pages, 1LL << a.t.page_bits, a.Hkv, a.D, p.s.b, p.s.l, p.s.h, S::ROW, box);
  };
  if (!encode(&k, a.k) || !encode(&v, a.v)) return cudaErrorInvalidValue;
  f.k_p = k.b_mul;
  f.k_h = k.h_mul;
  f.v_p = v.b_mul;
  f.v_h = v.h_mul;
  constexpr int smem = 1024 + std::max(kWarps * S::STAGES * S::TURN, kWarps * 8 * RT * (DP + 4) * 4);
  const cudaError_t e = cudaFuncSetAttribute(paged_step_kernel<QT, PT, DP, RT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.B * a.Hkv * f.groups * f.splits));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = f.splits;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = f.splits > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, paged_step_kernel<QT, PT, DP, RT>, k.map, v.map, f);
}
template <int QT, int PT, int RT> cudaError_t by_width(const StepArgs &f, cudaStream_t s) {
  return f.a.D <= 64 ? launch<QT, PT, 64, RT>(f, s) : launch<QT, PT, 128, RT>(f, s);
}
template <int QT, int PT> cudaError_t by_rows(const StepArgs &f, cudaStream_t s) {
  return (long long)f.a.Lq * f.a.G <= 8 ? by_width<QT, PT, 1>(f, s) : by_width<QT, PT, 2>(f, s);
}

}  // namespace

bool paged_step_takes(const PagedArgs &a, int dtype, int cache_dtype) {
  const int es = cache_dtype == kE4M3 ? 1 : 2;
  auto fits = [&](const Pages &p) {
    return rows_fit(p.data, es, a.t.n_pages, 1LL << a.t.page_bits, a.Hkv, a.D, p.s.b, p.s.l, p.s.h);
  };
  return dtype != kF32 && a.D <= 128 && a.D % 8 == 0 && a.t.page_bits >= 3 && fits(a.k) && fits(a.v);
}

cudaError_t launch_paged_step(const PagedArgs &a, int dtype, int cache_dtype, cudaStream_t stream) {
  StepArgs f = {};
  f.a = a;
  f.q_whole = (uintptr_t)a.q % 8 == 0 && (a.B == 1 || a.sq.b % 4 == 0) && (a.Lq == 1 || a.sq.l % 4 == 0) && (a.H == 1 || a.sq.h % 4 == 0);
  const int R = (long long)a.Lq * a.G <= 8 ? 8 : 16;
  f.groups = (int)(((long long)a.Lq * a.G + R - 1) / R);
  // a cluster's CTAs: the split whose waves of CTAs take least, in turns of a warp (one CTA's start and end cost about
  // as much as three)
  const long long units = a.B * a.Hkv * f.groups, slots = (R == 8 ? 3 : 2) * kSMs;
  const long long turns = (((long long)a.t.max_pages << a.t.page_bits) + 31) / 32;
  long long least = -1;
  for (int s = 1; s <= 8 && (s == 1 || turns >= 2 * s); s *= 2) {
    const long long waves = (units * s + slots - 1) / slots, cost = waves * ((turns + s * kWarps - 1) / (s * kWarps) + 3);
    if (least < 0 || cost < least) {
      least = cost;
      f.splits = s;
    }
  }
  if (cache_dtype == kE4M3) return dtype == kF16 ? by_rows<kF16, kE4M3>(f, stream) : by_rows<kBF16, kE4M3>(f, stream);
  return dtype == kF16 ? by_rows<kF16, kF16>(f, stream) : by_rows<kBF16, kBF16>(f, stream);
}

}  // namespace tdt
