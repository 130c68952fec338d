// Projections y = act(x W^T + b) + res and their gradients: one tile product
// C[m, n] = sum_k A[m, k] B[n, k] whose operands lie with K contiguous (x, W, and
// dp in dx = dp W) or K-major (W in dx, dp and x in dW = dp^T x), and an epilogue
// on the finished fp32 tile.
#include "block.h"
#include "common.h"
#include "launch.h"
#include "ring.h"

#include <algorithm>
#include <type_traits>

#include "../../include/ipttt.h"

namespace ipttt {
namespace {

// ---------------------------------------------------------------- epilogue

// exp(-v^2 / 2) and, of |v|, the normal distribution's upper tail Q: the exponential
// times a polynomial in t = 1 / (1 + 0.27 |v|), fitted to Q exp(v^2 / 2) / t for the least
// relative error over |v| <= 16, 2.5e-8 (beyond, the exponential is 0).  -v^2 / (2 ln 2)
// rounded to fp32 is off by some 2^-24 of itself, which the exponential makes 7e-6 of the
// tail at |v| = 12.  For fp32 data (T) what the square and its product lose is taken along,
// e, so that the tail is good to some 12 roundings wherever it is a normal number (1999 x
// 1024 x 4096 with GELU and pre kept 136.5 us, without e 135.7); next to bf16's own rounding,
// 2^-9, the 7e-6 do not count, and e would cost 28.2 instead of 27.2 us.  Less than half of
// erfcf's instructions: GELU's gradient at 1999 x 4096 in bf16 12.6 us, with erfcf 18.
template <typename T>
__device__ __forceinline__ float normal_tail(float v, float& bell) {
  if constexpr (sizeof(T) == 4) {
    constexpr float C = -0.72134752044448170f;                              // -1 / (2 ln 2)
    constexpr float CL = (float)(-0.72134752044448170368 - (double)C);
    const float m = fminf(fabsf(v), 16.0f), s = m * m, x = s * C;
    const float e = fmaf(fmaf(m, m, -s), C, fmaf(s, CL, fmaf(s, C, -x)));
    bell = __builtin_amdgcn_exp2f(x);
    bell = fmaf(bell, 0.69314718055994531f * e, bell);
  } else {
    bell = __expf(-0.5f * v * v);
  }
  const float t = __builtin_amdgcn_rcpf(fmaf(0.27f, fabsf(v), 1.0f));
  float p = 0.02903915521f;
  p = fmaf(p, t, -0.126877247f);
  p = fmaf(p, t, 0.170622473f);
  p = fmaf(p, t, -0.07020300618f);
  p = fmaf(p, t, 0.1085386858f);
  p = fmaf(p, t, 0.07173266605f);
  p = fmaf(p, t, 0.1018954598f);
  p = fmaf(p, t, 0.1075303996f);
  p = fmaf(p, t, 0.1077214258f);
  return bell * (t * p);
}
// The normal distribution function at v, from the tail so that the small values of
// negative v are as good, relative to themselves, as the tail.
template <typename T>
__device__ __forceinline__ float normal_cdf(float v, float& bell) {
  const float q = normal_tail<T>(v, bell);
  return v > 0.0f ? 1.0f - q : q;
}
template <typename T>
__device__ __forceinline__ float act_f32(int act, float v) {
  float bell;
  if (act == IPTTT_ACT_SILU) return silu_f32(v);
  if (act == IPTTT_ACT_GELU) return v * normal_cdf<T>(v, bell);
  return v;
}
// The activation's derivative at v.
template <typename T>
__device__ __forceinline__ float slope_f32(int act, float v) {
  if (act == IPTTT_ACT_SILU) {
    const float s = __builtin_amdgcn_rcpf(1.0f + __expf(-v));
    return s * (1.0f + v * (1.0f - s));
  }
  if (act == IPTTT_ACT_GELU) {
    float bell;
    const float cdf = normal_cdf<T>(v, bell);
    return cdf + v * (0.39894228040143268f * bell);  // far out the bell is 0, and so is the product
  }
  return 1.0f;
}

// -------------------------------------------------------------------- tiles

// How a product is cut: `whole` tiles over all of K, then the rest in `parts` of
// `per` stages each, whose fp32 partial tiles a second launch joins.
struct RingPlan {
  int nw;                 // tiles of 32 nw x 32 nw
  int tiles_m, tiles_n;   // tiles_m: of both products, where there are two
  int whole, split, parts, per;
  int stages, legs;       // stages of a leg
};

// N neighbouring elements, 16-byte aligned (or less where they are fewer bytes).
template <typename T, int N>
struct Run {
  typedef T type __attribute__((ext_vector_type(N), aligned(N * sizeof(T) < 16 ? N * sizeof(T) : 16)));
};
template <typename T, int N>
using Vec = typename Run<T, N>::type;

// One row's NJ neighbouring columns of a finished tile; res: the residual's.  A tile's
// rows are stored past the caches (STREAM), which keeps the operands in them.  In bf16,
// so and through the caches, a product alone: 1999 x 1024 x 4096 20.9 and 22.1 us, 32768 x
// 4096 x 2560 with a residual 533 and 528; with the product that reads it next: 1024 ->
// 4096 -> 1024 of 4096 rows 89 and 86, of 8192 152 and 150, of 32768 512 and 545, 2560 ->
// 9728 -> 2560 of 4096 rows 387 and 415.  (The column by column stores of K-major products
// are short pieces that the L2 has to join.)
template <bool STREAM, typename T, int NJ>
__device__ __forceinline__ void finish_row(const GemmArgs& g, int64_t m, int64_t n, const float (&bias)[NJ],
                                           const Vec<T, NJ>& res, float (&v)[NJ]) {
  typedef Vec<T, NJ> vec;
#pragma unroll
  for (int j = 0; j < NJ; ++j) v[j] += bias[j];
  if (g.pre.p != nullptr) {
    vec o;
#pragma unroll
    for (int j = 0; j < NJ; ++j) o[j] = (T)v[j];
    vec* to = reinterpret_cast<vec*>(static_cast<T*>(g.pre.p) + m * g.pre.ld + n);
    if constexpr (STREAM) __builtin_nontemporal_store(o, to);
    else *to = o;
  }
  if (g.act != IPTTT_ACT_NONE) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) v[j] = act_f32<T>(g.act, v[j]);
  }
  if (g.res.p != nullptr) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) v[j] += (float)res[j];
  }
  vec o;
#pragma unroll
  for (int j = 0; j < NJ; ++j) o[j] = (T)v[j];
  vec* to = reinterpret_cast<vec*>(static_cast<T*>(g.c.p) + m * g.c.ld + n);
  if constexpr (STREAM) __builtin_nontemporal_store(o, to);
  else *to = o;
}

// Waits for x's loads here: left to a use in a branch they would have the compiler wait
// in the next tile's loop, for the tile's loads behind them too.
template <typename V>
__device__ __forceinline__ V settled(V x) {
  if constexpr (sizeof(V) == 4) {
    asm volatile("" : "+v"(x));
    return x;
  } else {
    typedef uint32_t words __attribute__((ext_vector_type(sizeof(V) / 4)));
    words w = __builtin_bit_cast(words, x);
    asm volatile("" : "+v"(w));
    return __builtin_bit_cast(V, w);
  }
}

// The residual's rows of block row i of a tile at (m0, n0), loaded ahead.
template <typename T, int NW>
__device__ __forceinline__ void load_res(const GemmArgs& g, int64_t m0, int64_t n0, int i,
                                         Vec<T, ring::Geo<T, NW>::NJ> (&res)[4]) {
  typedef ring::Geo<T, NW> G;
  if (g.res.p == nullptr) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wm = wave >> 1, wn = wave & 1;
  const int64_t m = m0 + wm * G::WM + i * 16 + 4 * (lane >> 4), n = n0 + wn * G::WN + (lane & 15) * G::NJ;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (n < g.N && m + e < g.M)
      res[e] = *reinterpret_cast<const Vec<T, G::NJ>*>(static_cast<const T*>(g.res.p) + (m + e) * g.res.ld + n);
}

// Finishes block row i of a tile at (m0, n0): this lane's four rows of it.  With B's
// rows in the order of PERM (K contiguous) a lane has NJ neighbouring columns and
// the whole epilogue; K-major products have none and store column by column.
template <typename T, int NW, bool BK>
__device__ __forceinline__ void finish_block(const GemmArgs& g, const Rows& c, int64_t m0, int64_t n0, int i,
                                             const Vec<T, ring::Geo<T, NW>::NJ> (&res)[4],
                                             ring::f4 (&acc)[ring::Geo<T, NW>::NJ]) {
  typedef ring::Geo<T, NW> G;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wm = wave >> 1, wn = wave & 1;
  const int64_t m = m0 + wm * G::WM + i * 16 + 4 * (lane >> 4);
  if constexpr (!BK) {
    const int64_t n = n0 + wn * G::WN + (lane & 15) * G::NJ;
    if (n >= g.N) return;
    float bias[G::NJ];
#pragma unroll
    for (int j = 0; j < G::NJ; ++j) bias[j] = g.bias != nullptr ? (float)static_cast<const T*>(g.bias)[n + j] : 0.0f;
#pragma unroll
    for (int j = 0; j < G::NJ; ++j) bias[j] = settled(bias[j]);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (m + e >= g.M) break;
      float v[G::NJ];
#pragma unroll
      for (int j = 0; j < G::NJ; ++j) v[j] = acc[j][e];
      finish_row<true, T, G::NJ>(g, m + e, n, bias, res[e], v);
    }
  } else {
    const int64_t n = n0 + wn * G::WN + (lane & 15);
    const int blocks = n < g.N ? (int)min((int64_t)G::NJ, (g.N - n + 15) / 16) : 0;
    auto store = [&](auto* to) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (m + e >= g.M) break;
        auto* row = to + (m + e) * c.ld + n;
#pragma unroll
        for (int j = 0; j < G::NJ; ++j)
          if (j < blocks) row[j * 16] = from_f32<std::remove_pointer_t<decltype(to)>>(acc[j][e]);
      }
    };
    if (g.c_f32) store(static_cast<float*>(c.p));
    else store(static_cast<T*>(c.p));
  }
}

// The tile of an item, and the part of it (-1: whole).  Of two products the second
// has the second half of the tile rows.
__device__ __forceinline__ bool ring_item(const GemmArgs& g, const RingPlan& p, int t, int64_t& m0, int64_t& n0,
                                          int& part) {
  int tile = t;
  part = -1;
  if (t >= p.whole) {
    tile = p.whole + (t - p.whole) / p.parts;
    part = (t - p.whole) % p.parts;
  }
  int tm, tn;
  // four rows of tiles walked together: an XCD's workgroups share both operands' panels
  grouped_tile(tile, p.tiles_m, p.tiles_n, 4, tm, tn);
  const bool second = g.two_products && tm >= p.tiles_m / 2;
  m0 = (int64_t)(second ? tm - p.tiles_m / 2 : tm) * p.nw * 32;
  n0 = (int64_t)tn * p.nw * 32;
  return second;
}

template <typename T, int NW, bool AK, bool BK, int LEGS>
__device__ __forceinline__ void ring_product(const T* __restrict__ A, const T* __restrict__ B, const T* __restrict__ A2,
                                             const T* __restrict__ B2, const GemmArgs& g, const RingPlan& p, int turn,
                                             char* lds) {
  typedef ring::Geo<T, NW> G;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  // an item's stages, counted through the legs, cut at the leg's ends
  auto stages = [&](int t, int leg, int& s0, int& n) {
    int from = 0, to = p.stages * LEGS;
    if (t >= p.whole) {
      from = (t - p.whole) % p.parts * p.per;
      to = min(to, from + p.per);
    }
    s0 = max(0, from - leg * p.stages);
    n = min(p.stages, to - leg * p.stages) - s0;
  };
  auto open_a = [&](int t, int leg, int s0, ring::Loader<T, NW, AK>& l) {
    int64_t m0, n0;
    int part;
    const bool second = ring_item(g, p, t, m0, n0, part);
    const T* from = (LEGS > 1 && leg == 1) || second ? A2 : A;
    l.init(from + (AK ? m0 : m0 * g.a.ld), g.a.ld, g.M - m0, g.K, s0, wave, lane, [](int r) { return r; });
  };
  auto open_b = [&](int t, int leg, int s0, ring::Loader<T, NW, BK>& l) {
    int64_t m0, n0;
    int part;
    ring_item(g, p, t, m0, n0, part);
    const T* from = LEGS > 1 && leg == 1 ? B2 : B;
    l.init(from + (BK ? n0 : n0 * g.b.ld), g.b.ld, g.N - n0, g.K, s0, wave, lane,
           [](int r) { return ring::perm_row<NW>(r); });
  };
  auto epilogue = [&](int t, ring::f4 (&acc)[G::MI][G::NJ], auto&&) {
    int64_t m0, n0;
    int part;
    const Rows& c = ring_item(g, p, t, m0, n0, part) ? g.c2 : g.c;
    if (part >= 0) {
      ring::f4* to = reinterpret_cast<ring::f4*>(g.part) + (int64_t)(t - p.whole) * G::MI * G::NJ * G::NT + threadIdx.x;
#pragma unroll
      for (int i = 0; i < G::MI; ++i)
#pragma unroll
        for (int j = 0; j < G::NJ; ++j) to[(i * G::NJ + j) * G::NT] = acc[i][j];
      return;
    }
    // the residual's loads two block rows at a time: waiting for each one's cost 26 us
    // of 222 at 8192 x 2560 x 6144
#pragma unroll
    for (int i = 0; i < G::MI; i += 2) {
      Vec<T, G::NJ> res[2][4];
      if constexpr (!BK) {
#pragma unroll
        for (int q = 0; q < 2; ++q) load_res<T, NW>(g, m0, n0, i + q, res[q]);
#pragma unroll
        for (int e = 0; e < 8; ++e) res[e / 4][e % 4] = settled(res[e / 4][e % 4]);
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) finish_block<T, NW, BK>(g, c, m0, n0, i + q, res[q], acc[i + q]);
    }
  };
  ring::run<T, NW, AK, BK, LEGS, false>(lds, p.whole, p.split * p.parts, turn, stages, open_a, open_b, epilogue);
}

template <typename T, int NW, bool AK, bool BK, int LEGS>
__global__ __launch_bounds__((ring::Geo<T, NW>::NT), (ring::Geo<T, NW>::GROUPS)) void ring_kernel(GemmArgs g, RingPlan p) {
  __shared__ __attribute__((aligned(1024))) char lds[ring::Geo<T, NW>::LDS_BYTES];
  ring_product<T, NW, AK, BK, LEGS>(static_cast<const T*>(g.a.p), static_cast<const T*>(g.b.p),
                                    static_cast<const T*>(g.a2.p), static_cast<const T*>(g.b2.p), g, p, 0, lds);
}

// Both gradients of a projection in one launch, tiles of 4 waves: a workgroup walks its
// items of the first product, then of the second, the workgroups that the first one's
// last round leaves without an item first.  (A wave may begin the second while others
// finish the first: the slots that it loads are read only for products that are not
// formed.)
template <typename T, int NW, int LEGS>
__global__ __launch_bounds__(256, (ring::Geo<T, NW>::GROUPS)) void ring_pair_kernel(GemmArgs g, RingPlan p, GemmArgs h, RingPlan q, int turn) {
  __shared__ __attribute__((aligned(1024))) char lds[ring::Geo<T, NW>::LDS_BYTES];
  ring_product<T, NW, false, true, LEGS>(static_cast<const T*>(g.a.p), static_cast<const T*>(g.b.p),
                                        static_cast<const T*>(g.a2.p), static_cast<const T*>(g.b2.p), g, p, 0, lds);
  ring_product<T, NW, true, true, 1>(static_cast<const T*>(h.a.p), static_cast<const T*>(h.b.p),
                                    static_cast<const T*>(h.a2.p), static_cast<const T*>(h.b2.p), h, q, turn, lds);
}

// Sums the parts of a split tile in order and finishes it; blockIdx.y takes a block
// row of it.
template <typename T, int NW, bool BK>
__global__ __launch_bounds__((ring::Geo<T, NW>::NT)) void ring_join_kernel(GemmArgs g, RingPlan p) {
  typedef ring::Geo<T, NW> G;
  const int i = blockIdx.y, t = p.whole + blockIdx.x * p.parts;
  int64_t m0, n0;
  int part;
  const Rows& c = ring_item(g, p, t, m0, n0, part) ? g.c2 : g.c;
  Vec<T, G::NJ> res[4];
  if constexpr (!BK) load_res<T, NW>(g, m0, n0, i, res);
  const ring::f4* from = reinterpret_cast<const ring::f4*>(g.part) +
                         ((int64_t)blockIdx.x * p.parts * G::MI + i) * G::NJ * G::NT + threadIdx.x;
  ring::f4 acc[G::NJ];
#pragma unroll
  for (int j = 0; j < G::NJ; ++j) acc[j] = from[j * G::NT];
  for (int q = 1; q < p.parts; ++q) {
    from += (int64_t)G::MI * G::NJ * G::NT;
#pragma unroll
    for (int j = 0; j < G::NJ; ++j) acc[j] += from[j * G::NT];
  }
  finish_block<T, NW, BK>(g, c, m0, n0, i, res, acc);
}

// A constant, not asked of the device, so that a workspace's size does not depend on the
// device that is current when it is asked for.
constexpr int kCus = 256;

// The cut for which an estimate of the product's time is least (in us); only: 0, or the
// one tile size to take.
RingPlan plan_ring(const GemmArgs& g, int only, double* us) {
  RingPlan best{};
  double least = 1e300;
  const bool h = g.dtype == 1;
  // us of a stage, of a workgroup alone on its CU and on a full one, of an item beside its
  // stages and of joining, fitted to some 1000 products of both types in all cuts (33 to
  // 16384 rows): over 240 others the cut so chosen takes 0.7 % longer than the best one on
  // average in bf16 and 0.5 % in fp32, 6 % at the ninth tenth, a third at most (dW of 4229
  // rows, 64 -> 256: 14.7 us, in 6 parts 11.0).  In bf16 small tiles are for few of them
  // (512 x 1024 x 1024 8.4 us on 64 x 64, 13.0 on 128 x 128; 1999 x 1024 x 4096 21.0 on 128 x
  // 128, 28 on 256 x 256); in fp32, where products take 16 times as long, 128 x 128 took 19 %
  // longer than 64 x 64 on average and up to 4 % less (8192 x 2560 x 2560), 256 x 256 up to
  // four times as long.
  const struct Cost {
    int nw;
    double lone, full, item;
  } costs[2][3] = {{{2, 0.55, 1.9, 2.0}}, {{8, 1.3, 1.35, 4.5}, {4, 0.5, 0.95, 1.9}, {2, 0.3, 0.77, 1.2}}};
  for (const Cost& c : costs[h]) {
    if (c.nw == 0 || (only != 0 && c.nw != only)) continue;
    const int64_t w = c.nw * 32, tm = (g.M + w - 1) / w * (g.two_products ? 2 : 1), tn = (g.N + w - 1) / w, tiles = tm * tn;
    const int64_t most = 8 / c.nw, groups = most * kCus;
    const int ks = h ? ring::kStage<bf16> : ring::kStage<float>, legs = g.two_pairs ? 2 : 1,
              leg = (int)((g.K + ks - 1) / ks), stages = legs * leg;
    auto consider = [&](int64_t whole, int parts) {
      const int per = (stages + parts - 1) / parts;
      parts = (stages + per - 1) / per;
      const int64_t split = tiles - whole, items = split * parts;
      const int64_t rounds = whole / groups;
      double t = rounds * (stages * c.full + c.item);
      const int64_t rest = whole % groups + items;
      // 8 waves: a half empty device
      const double share = most == 1 ? (rest > groups / 2 ? 1.0 : 0.0)
                                     : (double)(std::min((rest + kCus - 1) / kCus, most) - 1) / (double)(most - 1);
      t += (double)((rest + groups - 1) / groups) * (per * (c.lone + (c.full - c.lone) * share) + c.item);
      if (parts > 1) t += (h ? 2.8 : 4.0) + (double)items * w * w * 8 / (h ? 5.2e6 : 8.0e6);
      if (t >= least) return;
      least = t;
      best = RingPlan{c.nw, (int)tm, (int)tn, (int)(parts > 1 ? whole : tiles), (int)(parts > 1 ? split : 0), parts, per, leg, legs};
    };
    consider(tiles, 1);
    const int64_t whole = tiles / groups * groups, rem = tiles - whole;
    if (rem > 0)
      for (int64_t parts = 2; parts <= 32 && parts * 2 <= stages && rem * parts <= 2 * groups; ++parts) consider(whole, (int)parts);
  }
  *us = least;
  return best;
}
RingPlan plan_ring(const GemmArgs& g) {
  double us;
  return plan_ring(g, 0, &us);
}

// Both gradients of a projection: tiles of one size where neither's are of 8 waves, so
// that one launch can take both.
struct PairPlan {
  RingPlan g, h;
};
PairPlan plan_pair(const GemmArgs& g, const GemmArgs& h) {
  PairPlan best{plan_ring(g), plan_ring(h)};
  if (best.g.nw == best.h.nw || best.g.nw == 8 || best.h.nw == 8) return best;
  double least = 1e300;
  for (const int nw : {4, 2}) {
    double a, b;
    const PairPlan p{plan_ring(g, nw, &a), plan_ring(h, nw, &b)};
    if (a + b >= least) continue;
    least = a + b;
    best = p;
  }
  return best;
}

int64_t ring_items(const RingPlan& p) { return (int64_t)p.whole + (int64_t)p.split * p.parts; }

template <typename T, int NW>
hipError_t launch_join(const GemmArgs& g, const RingPlan& p, hipStream_t st) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.split == 0) return e;
  note_launch("linear_join", st);
  typedef ring::Geo<T, NW> G;
  const dim3 j((unsigned)p.split, G::MI);
  if (!g.b_kmaj) ring_join_kernel<T, NW, false><<<j, G::NT, 0, st>>>(g, p);
  else ring_join_kernel<T, NW, true><<<j, G::NT, 0, st>>>(g, p);
  return hipGetLastError();
}

template <typename T, int NW>
hipError_t launch_ring(const GemmArgs& g, const RingPlan& p, hipStream_t st) {
  typedef ring::Geo<T, NW> G;
  const unsigned grid = (unsigned)std::min<int64_t>(kCus * G::GROUPS, (ring_items(p) + 7) / 8 * 8);
  note_launch("linear", st);
  if (!g.a_kmaj && !g.b_kmaj) ring_kernel<T, NW, false, false, 1><<<grid, G::NT, 0, st>>>(g, p);
  else if (p.legs == 2) {
    if constexpr (sizeof(T) == 2) ring_kernel<T, NW, false, true, 2><<<grid, G::NT, 0, st>>>(g, p);
  } else if (!g.a_kmaj) ring_kernel<T, NW, false, true, 1><<<grid, G::NT, 0, st>>>(g, p);
  else ring_kernel<T, NW, true, true, 1><<<grid, G::NT, 0, st>>>(g, p);
  return launch_join<T, NW>(g, p, st);
}

template <typename T, int NW, int LEGS>
hipError_t launch_ring_pair(const GemmArgs& g, const RingPlan& p, const GemmArgs& h, const RingPlan& q,
                            hipStream_t st) {
  const unsigned grid = (unsigned)std::min<int64_t>(kCus * ring::Geo<T, NW>::GROUPS, (ring_items(p) + ring_items(q) + 7) / 8 * 8);
  // the items an XCD's workgroups walk last in the first product
  const int last = p.split > 0 ? p.split * p.parts : p.whole;
  note_launch("linear_pair", st);
  ring_pair_kernel<T, NW, LEGS><<<grid, 256, 0, st>>>(g, p, h, q, (last + 7) / 8 % (int)(grid / 8));
  const hipError_t e = launch_join<T, NW>(g, p, st);
  return e != hipSuccess ? e : launch_join<T, NW>(h, q, st);
}

size_t ring_bytes(const RingPlan& p) {
  return (size_t)p.split * p.parts * (p.nw * 32) * (p.nw * 32) * sizeof(float);
}

// ---------------------------------------------------------------- few rows

// Up to 16 MT rows of x: the weights stream from HBM once, straight to the
// fragments of 16x16 products (rows: 16 FB outputs, columns: rows of x), with all
// their loads in flight; 16 waves take every 16th slice of K and are summed through
// LDS.  A lane ends up with four neighbouring outputs of one row.
// Bound by the launch and the weights' way to the CUs: one row 2560 -> 6144 in bf16 8.5 us
// for 31 MB that the memory-side cache holds (3.7 TB/s) and 10.8 where they come from HBM
// (2.9 TB/s), as those of a decoder's layers do; 32 rows 4096 -> 2560 13.1 and 14.6 us,
// where each of 160 workgroups reads the 262 KB of x beside 131 KB of weights.  Two
// neighbouring slices a wave, so that it reads whole lines, changed nothing.
template <typename T, int MT, int FB>
__global__ __launch_bounds__(1024) void few_kernel(GemmArgs g) {
  constexpr int W = 16;
  typedef typename ring::Frag<T>::type frag;
  constexpr int VE = 16 / sizeof(T), CK = 4 * VE;                              // K of a slice: 16 bytes a lane
  constexpr int U = MT * FB >= 3 ? 4 : 8;  // slices in flight
  __shared__ ring::f4 red[W][MT * FB][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, kg = (lane >> 4) * VE;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * FB);
  const T *a[FB], *b[MT];
#pragma unroll
  for (int f = 0; f < FB; ++f) a[f] = static_cast<const T*>(g.b.p) + min(n0 + f * 16 + r, g.N - 1) * g.b.ld + kg;
#pragma unroll
  for (int t = 0; t < MT; ++t) b[t] = static_cast<const T*>(g.a.p) + min((int64_t)(t * 16 + r), g.M - 1) * g.a.ld + kg;
  ring::f4 acc[MT][FB];
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int f = 0; f < FB; ++f) acc[t][f] = ring::f4{0.0f, 0.0f, 0.0f, 0.0f};
  const int K = (int)g.K;
  for (int k0 = wave * CK; k0 < K; k0 += U * W * CK) {
    frag fa[U][FB], fb[U][MT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * W * CK;
      const bool on = k + kg < K;
#pragma unroll
      for (int f = 0; f < FB; ++f) fa[u][f] = on ? *reinterpret_cast<const frag*>(a[f] + k) : frag{};
#pragma unroll
      for (int t = 0; t < MT; ++t) fb[u][t] = on ? *reinterpret_cast<const frag*>(b[t] + k) : frag{};
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int f = 0; f < FB; ++f) acc[t][f] = ring::Frag<T>::mma(fa[u][f], fb[u][t], acc[t][f]);
  }
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int f = 0; f < FB; ++f) red[wave][t * FB + f][lane] = acc[t][f];
  __syncthreads();
  for (int i = wave; i < MT * FB; i += W) {
    ring::f4 v = red[0][i][lane];
#pragma unroll
    for (int w = 1; w < W; ++w) v += red[w][i][lane];
    const int64_t m = i / FB * 16 + r, n = n0 + i % FB * 16 + 4 * (lane >> 4);
    if (m >= g.M || n >= g.N) continue;
    float bias[4], y[4];
    Vec<T, 4> res = {};
    if (g.res.p != nullptr) res = *reinterpret_cast<const Vec<T, 4>*>(static_cast<const T*>(g.res.p) + m * g.res.ld + n);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      bias[e] = g.bias != nullptr ? to_f32(static_cast<const T*>(g.bias)[n + e]) : 0.0f;
      y[e] = v[e];
    }
    finish_row<false, T, 4>(g, m, n, bias, res, y);
  }
}

// Where the tiles take less: from 65 rows on, and before that for large weights, which
// every workgroup's reads of all of x hold up here (they grow with the rows and K; the
// outputs cost little until there are more than 256 workgroups).  Us here and on the
// tiles, with weights that the memory-side cache holds, and [with weights from HBM]:
//   bf16, 64 rows  1024 -> 4096 7.3, 7.6 [7.9, 14.0]    1024 -> 6144 12.7, 7.7 [13.7, 14.3]
//                  1280 -> 4096 8.3, 9.9 [9.7, 12.1]    2560 -> 2560 13.7, 10.5 [16.8, 13.6]
//         32 rows  2560 -> 6144 12.0, 13.1 [15.7, 15.4] 2560 -> 9728 22.5, 20.0 [25.9, 30.6]
//         16 rows  2560 -> 9728 17.2, 19.6 [20.1, 30.2] 9728 -> 2560 19.4, 17.5 [24.1, 21.0]
//   fp32, 32 rows  1024 -> 2048 11.3, 12.5 [11.9, 13.5] 2560 -> 2560 21.2, 17.0 [24.7, 19.4]
//         16 rows  4096 -> 2560 18.5, 22.7 [21.3, 23.3] 2560 -> 9728 39.9, 33.3 [48.0, 34.9]
//          8 rows  4096 -> 2560 15.9, 22.5 [18.1, 23.3] 2560 -> 9728 31.4, 33.2 [36.4, 34.8]
// The bounds are those of weights in the cache.  On their wrong side lie, in bf16, 64 rows
// 1536 -> 4096 (here 9.4, tiles 10.1), 32 rows 4096 -> 2560 (13.1, 11.2) and, from HBM, 32
// rows 2560 -> 9728.
bool few_rows(const GemmArgs& g) {
  if (g.a_kmaj || g.b_kmaj) return false;
  const bool h = g.dtype == 1;
  const int64_t weights = g.N * g.K;
  if (g.M > 32) return h && g.M <= 64 && g.K <= 1280 && g.N <= 4096;
  return g.M <= (h ? 16 : 8) || (g.M <= (h ? 32 : 16) && weights <= 20000000) || weights <= 4000000;
}

// Two blocks of outputs a workgroup halve the rows' reads; they pay where there are
// workgroups enough.
template <typename T>
void launch_few(const GemmArgs& g, hipStream_t st) {
  note_launch("linear_few", st);
  const auto groups = [&](int fb) { return (unsigned)((g.N + 16 * fb - 1) / (16 * fb)); };
  const bool wide = groups(2) >= 192;
  if (g.M <= 8) few_kernel<T, 1, 1><<<groups(1), 1024, 0, st>>>(g);
  else if (g.M <= 16 && !wide) few_kernel<T, 1, 1><<<groups(1), 1024, 0, st>>>(g);
  else if (g.M <= 16) few_kernel<T, 1, 2><<<groups(2), 1024, 0, st>>>(g);
  else if (g.M > 32) {
    if constexpr (sizeof(T) == 2) {
      if (g.M > 48) few_kernel<T, 4, 1><<<groups(1), 1024, 0, st>>>(g);
      else few_kernel<T, 3, 1><<<groups(1), 1024, 0, st>>>(g);
    }
  } else if (!wide) few_kernel<T, 2, 1><<<groups(1), 1024, 0, st>>>(g);
  else few_kernel<T, 2, 2><<<groups(2), 1024, 0, st>>>(g);
}

// ------------------------------------------------- the activation's gradient

// A thread takes 8 columns of every eighth row of a strip of rows, two of its rows at
// a time; the columns' sums stay in registers and each strip writes one partial.  dp is
// rounded to T, an operand of the matrix cores: in bf16 dx and dW are then 2.3e-3 of their
// norm off, sqrt(2) times their own rounding's 1.7e-3; a second bf16 term of dp would take
// that away and double both products, most of the gradient's time.  The columns' sums are
// of the unrounded values.
// Bound by the memory: 1999 x 4096 in bf16 with GELU 12.6 us for 49 MB (four rows at a
// time 13.3), 8192 x 6144 without an activation 17 us for 101 MB.
template <typename T>
__global__ __launch_bounds__(256) void act_grad_kernel(ActGradArgs a, int64_t strip) {
  typedef Vec<T, 8> vec;
  static_assert(alignof(vec) <= 16, "what the entries ask of a tensor");
  constexpr int U = 2;
  __shared__ float red[8][256];
  const int cg = threadIdx.x & 31, rg = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 256 + cg * 8;
  const int64_t end = min(a.rows, (blockIdx.y + 1) * strip);
  float s[8] = {};
  auto rows = [&](int64_t r, auto count) {
    constexpr int N = decltype(count)::value;
    vec dy[N], pre[N];
#pragma unroll
    for (int u = 0; u < N; ++u)
      dy[u] = *reinterpret_cast<const vec*>(static_cast<const T*>(a.dy.p) + (r + 8 * u) * a.dy.ld + c);
    if (a.pre.p != nullptr) {
#pragma unroll
      for (int u = 0; u < N; ++u)
        pre[u] = *reinterpret_cast<const vec*>(static_cast<const T*>(a.pre.p) + (r + 8 * u) * a.pre.ld + c);
    }
#pragma unroll
    for (int u = 0; u < N; ++u) {
      vec o;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float v = a.pre.p != nullptr ? (float)dy[u][e] * slope_f32<T>(a.act, (float)pre[u][e]) : (float)dy[u][e];
        s[e] += v;
        o[e] = (T)v;
      }
      if (a.dp.p != nullptr)
        *reinterpret_cast<vec*>(static_cast<T*>(a.dp.p) + (r + 8 * u) * a.dp.ld + c) = o;
    }
  };
  if (c < a.dim) {
    int64_t r = blockIdx.y * strip + rg;
    for (; r + 8 * (U - 1) < end; r += 8 * U) rows(r, std::integral_constant<int, U>());
    for (; r < end; r += 8) rows(r, std::integral_constant<int, 1>());
  }
  if (a.db == nullptr) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) red[rg][cg * 8 + e] = s[e];
  __syncthreads();
  const int64_t col = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (col >= a.dim) return;
  float x = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) x += red[i][threadIdx.x];
  a.part[blockIdx.y * a.dim + col] = x;
}

// The strips' partials of 16 columns a workgroup, 32 threads a column, in a fixed order.
__global__ __launch_bounds__(512) void column_sum_kernel(const float* part, int parts, int64_t dim, float* out) {
  __shared__ float red[32][17];
  const int64_t c = (int64_t)blockIdx.x * 16 + (threadIdx.x & 15);
  const int g = threadIdx.x >> 4;
  float x = 0.0f;
  if (c < dim)
    for (int p = g; p < parts; p += 32) x += part[p * dim + c];
  red[g][threadIdx.x & 15] = x;
  __syncthreads();
  if (g != 0 || c >= dim) return;
#pragma unroll
  for (int i = 1; i < 32; ++i) x += red[i][threadIdx.x];
  out[c] = x;
}

constexpr int kStrips = 256;  // most strips of rows of a column sum

}  // namespace

size_t gemm_workspace(const GemmArgs& g) { return few_rows(g) ? 0 : ring_bytes(plan_ring(g)); }

namespace {

hipError_t launch_plan(const GemmArgs& g, const RingPlan& p, hipStream_t st) {
  // products that no caller has
  if (g.a_kmaj && !g.b_kmaj) return hipErrorInvalidValue;
  if (g.two_pairs && (g.a_kmaj || !g.b_kmaj || g.two_products || g.dtype != 1)) return hipErrorInvalidValue;
  if (g.two_products && (!g.a_kmaj || g.dtype != 1)) return hipErrorInvalidValue;
  if (g.dtype == 1)
    return p.nw == 8   ? launch_ring<bf16, 8>(g, p, st)
           : p.nw == 4 ? launch_ring<bf16, 4>(g, p, st)
                       : launch_ring<bf16, 2>(g, p, st);
  return launch_ring<float, 2>(g, p, st);
}

}  // namespace

hipError_t launch_gemm(const GemmArgs& g, hipStream_t st) {
  if (!few_rows(g)) return launch_plan(g, plan_ring(g), st);
  if (g.dtype == 1) launch_few<bf16>(g, st);
  else launch_few<float>(g, st);
  return hipGetLastError();
}

void gemm_pair_workspace(const GemmArgs& g, const GemmArgs& h, size_t* of_g, size_t* of_h) {
  const PairPlan p = plan_pair(g, h);
  *of_g = ring_bytes(p.g);
  *of_h = ring_bytes(p.h);
}

hipError_t launch_gemm_pair(const GemmArgs& g, const GemmArgs& h, hipStream_t st) {
  const auto [p, q] = plan_pair(g, h);
  // Tiles of 4 waves together: 1999 x 1024 x 4096 in bf16 44.7 us, one after the other
  // 55.5; 4096 x 1024 x 1024 30.0 and 41.7; 6000 x 1024 x 2048 in fp32, which fills the
  // device twice each, 478 and 470.  Tiles of 8 waves, one workgroup a CU, fill the
  // device by themselves.
  if (g.c.p == nullptr || h.c.p == nullptr || p.nw == 8 || p.nw != q.nw || g.a_kmaj || !g.b_kmaj || !h.a_kmaj ||
      !h.b_kmaj || g.dtype != h.dtype) {
    const hipError_t e = g.c.p != nullptr ? launch_plan(g, p, st) : hipSuccess;
    return e != hipSuccess || h.c.p == nullptr ? e : launch_plan(h, q, st);
  }
  if (g.dtype == 1 && p.nw == 4)
    return g.two_pairs ? launch_ring_pair<bf16, 4, 2>(g, p, h, q, st) : launch_ring_pair<bf16, 4, 1>(g, p, h, q, st);
  if (g.dtype == 1)
    return g.two_pairs ? launch_ring_pair<bf16, 2, 2>(g, p, h, q, st) : launch_ring_pair<bf16, 2, 1>(g, p, h, q, st);
  if (g.two_pairs || h.two_products) return hipErrorInvalidValue;
  return launch_ring_pair<float, 2, 1>(g, p, h, q, st);
}

int act_grad_parts(int64_t rows, int64_t dim) {
  // about 2048 workgroups, of at least 32 rows each
  const int64_t want = std::max<int64_t>(1, 2048 / ((dim + 255) / 256));
  return (int)std::min<int64_t>({want, (rows + 31) / 32, kStrips});
}

hipError_t launch_act_grad(const ActGradArgs& a, hipStream_t st) {
  const int64_t parts = act_grad_parts(a.rows, a.dim), strip = (a.rows + parts - 1) / parts;
  // strips that hold no row write zeros
  note_launch("act_grad", st);
  const dim3 grid((unsigned)((a.dim + 255) / 256), (unsigned)parts);
  if (a.dtype == 1) act_grad_kernel<bf16><<<grid, 256, 0, st>>>(a, strip);
  else act_grad_kernel<float><<<grid, 256, 0, st>>>(a, strip);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.db == nullptr) return e;
  note_launch("column_sum", st);
  column_sum_kernel<<<(unsigned)((a.dim + 15) / 16), 512, 0, st>>>(a.part, (int)parts, a.dim, a.db);
  return hipGetLastError();
}

}  // namespace ipttt
