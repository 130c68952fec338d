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

constexpr float kRsqrt2 = 0.70710678118654752f;

// v times the normal distribution function; erfc keeps the small values of
// negative v, where 1 + erf cancels.
__device__ __forceinline__ float gelu_f32(float v) { return 0.5f * v * erfcf(-kRsqrt2 * v); }
__device__ __forceinline__ float act_f32(int act, float v) {
  if (act == IPTTT_ACT_SILU) return silu_f32(v);
  if (act == IPTTT_ACT_GELU) return gelu_f32(v);
  return v;
}
// The activation's derivative at v.
__device__ __forceinline__ float slope_f32(int act, float v) {
  if (act == IPTTT_ACT_SILU) {
    const float s = 1.0f / (1.0f + __expf(-v));
    return s * (1.0f + v * (1.0f - s));
  }
  // v phi(v): far out phi underflows to 0 and so must the product
  if (act == IPTTT_ACT_GELU) return 0.5f * erfcf(-kRsqrt2 * v) + v * (0.39894228040143268f * __expf(-0.5f * v * v));
  return 1.0f;
}

// Finishes element (m, n) of the product.
template <typename T>
__device__ __forceinline__ void finish(const GemmArgs& g, int64_t m, int n, float v) {
  if (g.bias != nullptr) v += to_f32(static_cast<const T*>(g.bias)[n]);
  if (g.pre.p != nullptr) static_cast<T*>(g.pre.p)[m * g.pre.ld + n] = from_f32<T>(v);
  v = act_f32(g.act, v);
  if (g.res.p != nullptr) v += to_f32(static_cast<const T*>(g.res.p)[m * g.res.ld + n]);
  if (g.c_f32)
    static_cast<float*>(g.c.p)[m * g.c.ld + n] = v;
  else
    static_cast<T*>(g.c.p)[m * g.c.ld + n] = from_f32<T>(v);
}

// ------------------------------------------------------------ general tiles

// A [BK x 128] slice of a K-major operand (K rows of the matrix, 128 of its
// columns) moved to the [128][LDK] LDS tile that stage_mma reads: 16-byte loads
// along the columns, one element a row stored.  Columns >= ncols (a multiple of
// the piece) and rows >= krows read as zero.
template <typename T>
struct KmajLoad {
  static constexpr int VE = 16 / sizeof(T), BK = 128 / sizeof(T), VPR = 128 / VE, NV = BK * VPR / kThreads;
  u32x4 v[NV];
  __device__ __forceinline__ void load(const T* __restrict__ base, int64_t ld, int ncols, int64_t k0, int64_t krows,
                                       int tid) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int idx = tid + j * kThreads;
      const int k = idx / VPR, c = (idx % VPR) * VE;
      v[j] = k0 + k < krows && c < ncols ? *reinterpret_cast<const u32x4*>(base + (k0 + k) * ld + c)
                                         : u32x4{0u, 0u, 0u, 0u};
    }
  }
  template <int LDK>
  __device__ __forceinline__ void store(T* lds, int tid) const {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int idx = tid + j * kThreads;
      const int k = idx / VPR, c = (idx % VPR) * VE;
      const T* e = reinterpret_cast<const T*>(&v[j]);
#pragma unroll
      for (int q = 0; q < VE; ++q) lds[(c + q) * LDK + k] = e[q];
    }
  }
};

// One operand's slices: rows [0, n) of it from `base` on, K contiguous or major.
template <typename T, bool KMAJ>
struct Side {
  typename std::conditional<KMAJ, KmajLoad<T>, TileLoad<T, 128>>::type t;
  __device__ __forceinline__ void load(const T* base, int64_t ld, int n, int64_t k0, int64_t K, int tid) {
    if constexpr (KMAJ) t.load(base, ld, n, k0, K, tid);
    else t.load(base, ld, n, (int)k0, (int)K, tid);
  }
};

// 128 x 128 tiles, 4 waves, one slice of each operand in LDS while the next is on
// its way to registers.  Takes every size (multiples of 8) and both types.
template <typename T, bool AK, bool BK>
__global__ __launch_bounds__(kThreads) void gemm_kernel(GemmArgs g) {
  typedef Geo<T, 128, 128> G;
  __shared__ __attribute__((aligned(16))) T lds[(G::BM + G::BN) * G::LDK];
  T *lA = lds, *lB = lds + G::BM * G::LDK;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave >> 1, wn = wave & 1;
  const int tiles_m = (int)((g.M + 127) / 128), tiles_n = (int)((g.N + 127) / 128);
  int tm, tn;
  grouped_tile(xcd_remap(blockIdx.x, gridDim.x), tiles_m, tiles_n, 16, tm, tn);
  const int64_t m0 = (int64_t)tm * 128, n0 = (int64_t)tn * 128;
  const int mrows = (int)min((int64_t)128, g.M - m0), nrows = (int)min((int64_t)128, g.N - n0);
  const T* A = static_cast<const T*>(g.a.p) + (AK ? m0 : m0 * g.a.ld);
  const T* B = static_cast<const T*>(g.b.p) + (BK ? n0 : n0 * g.b.ld);
  floatx16 acc[G::MB][G::NB];
  zero_acc<G>(acc);
  Side<T, AK> la;
  Side<T, BK> lb;
  la.load(A, g.a.ld, mrows, 0, g.K, tid);
  lb.load(B, g.b.ld, nrows, 0, g.K, tid);
  for (int64_t k0 = 0; k0 < g.K; k0 += G::BK) {
    la.t.template store<G::LDK>(lA, tid);
    lb.t.template store<G::LDK>(lB, tid);
    __syncthreads();
    if (k0 + G::BK < g.K) {
      la.load(A, g.a.ld, mrows, k0 + G::BK, g.K, tid);
      lb.load(B, g.b.ld, nrows, k0 + G::BK, g.K, tid);
    }
    stage_mma<T, G>(lA, lB, acc, wm, wn, lane);
    __syncthreads();
  }
#pragma unroll
  for (int mb = 0; mb < G::MB; ++mb)
#pragma unroll
    for (int nb = 0; nb < G::NB; ++nb)
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int r = wm * G::WM + mb * 32 + acc_row(j, lane), c = wn * G::WN + nb * 32 + (lane & 31);
        if (r < mrows && c < nrows) finish<T>(g, m0 + r, (int)n0 + c, acc[mb][nb][j]);
      }
}

// --------------------------------------------------------------- bf16 tiles

// How a product is cut: `whole` tiles over all of K, then the rest in `parts` of
// `per` stages each, whose fp32 partial tiles a second launch joins.
struct RingPlan {
  int nw;                 // 8: tiles of 256 x 256, 4: of 128 x 128
  int tiles_m, tiles_n, whole, split, parts, per, stages;
};

// One row's NJ neighbouring columns of a finished tile.
template <int NJ>
__device__ __forceinline__ void finish_row(const GemmArgs& g, int64_t m, int64_t n, const float (&bias)[NJ], float (&v)[NJ]) {
  typedef bf16 vec __attribute__((ext_vector_type(NJ)));
#pragma unroll
  for (int j = 0; j < NJ; ++j) v[j] += bias[j];
  if (g.pre.p != nullptr) {
    vec o;
#pragma unroll
    for (int j = 0; j < NJ; ++j) o[j] = (bf16)v[j];
    *reinterpret_cast<vec*>(static_cast<bf16*>(g.pre.p) + m * g.pre.ld + n) = o;
  }
  if (g.act != IPTTT_ACT_NONE) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) v[j] = act_f32(g.act, v[j]);
  }
  if (g.res.p != nullptr) {
    const vec r = *reinterpret_cast<const vec*>(static_cast<const bf16*>(g.res.p) + m * g.res.ld + n);
#pragma unroll
    for (int j = 0; j < NJ; ++j) v[j] += (float)r[j];
  }
  vec o;
#pragma unroll
  for (int j = 0; j < NJ; ++j) o[j] = (bf16)v[j];
  *reinterpret_cast<vec*>(static_cast<bf16*>(g.c.p) + m * g.c.ld + n) = o;
}

// Finishes block row i of a tile at (m0, n0): this lane's four rows of it.  With B's
// rows in the order of PERM (K contiguous) a lane has NJ neighbouring columns and
// the whole epilogue; K-major products have none and store column by column.
template <int NW, bool BK>
__device__ __forceinline__ void finish_block(const GemmArgs& g, int64_t m0, int64_t n0, int i,
                                             ring::f4 (&acc)[ring::Geo<NW>::NJ]) {
  typedef ring::Geo<NW> G;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wm = wave >> 1, wn = wave & 1;
  const int64_t m = m0 + wm * G::WM + i * 16 + 4 * (lane >> 4);
  if constexpr (!BK) {
    const int64_t n = n0 + wn * G::WN + (lane & 15) * G::NJ;
    if (n >= g.N) return;
    float bias[G::NJ];
#pragma unroll
    for (int j = 0; j < G::NJ; ++j) bias[j] = g.bias != nullptr ? (float)static_cast<const bf16*>(g.bias)[n + j] : 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (m + e >= g.M) break;
      float v[G::NJ];
#pragma unroll
      for (int j = 0; j < G::NJ; ++j) v[j] = acc[j][e];
      finish_row<G::NJ>(g, m + e, n, bias, v);
    }
  } else {
    const int64_t n = n0 + wn * G::WN + (lane & 15);
    const int blocks = n < g.N ? (int)min((int64_t)G::NJ, (g.N - n + 15) / 16) : 0;
    auto store = [&](auto* c) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (m + e >= g.M) break;
        auto* row = c + (m + e) * g.c.ld + n;
#pragma unroll
        for (int j = 0; j < G::NJ; ++j)
          if (j < blocks) row[j * 16] = from_f32<std::remove_pointer_t<decltype(c)>>(acc[j][e]);
      }
    };
    if (g.c_f32) store(static_cast<float*>(g.c.p));
    else store(static_cast<bf16*>(g.c.p));
  }
}

// The tile of an item, and the part of it (-1: whole).
__device__ __forceinline__ void ring_item(const RingPlan& p, int t, int64_t& m0, int64_t& n0, int& part) {
  int tile = t;
  part = -1;
  if (t >= p.whole) {
    tile = p.whole + (t - p.whole) / p.parts;
    part = (t - p.whole) % p.parts;
  }
  int tm, tn;
  // four rows of tiles walked together: an XCD's workgroups share both operands' panels
  grouped_tile(tile, p.tiles_m, p.tiles_n, 4, tm, tn);
  m0 = (int64_t)tm * p.nw * 32;
  n0 = (int64_t)tn * p.nw * 32;
}

template <int NW, bool AK, bool BK>
__device__ __forceinline__ void ring_product(const bf16* __restrict__ A, const bf16* __restrict__ B, const GemmArgs& g,
                                             const RingPlan& p, char* lds) {
  typedef ring::Geo<NW> G;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  auto stages = [&](int t, int& s0, int& n) {
    s0 = 0;
    n = p.stages;
    if (t >= p.whole) {
      s0 = (t - p.whole) % p.parts * p.per;
      n = min(p.per, p.stages - s0);
    }
  };
  auto open_a = [&](int t, int s0, ring::Loader<NW, AK>& l) {
    int64_t m0, n0;
    int part;
    ring_item(p, t, m0, n0, part);
    l.init(A + (AK ? m0 : m0 * g.a.ld), g.a.ld, g.M - m0, g.K, s0, wave, lane, [](int r) { return r; });
  };
  auto open_b = [&](int t, int s0, ring::Loader<NW, BK>& l) {
    int64_t m0, n0;
    int part;
    ring_item(p, t, m0, n0, part);
    l.init(B + (BK ? n0 : n0 * g.b.ld), g.b.ld, g.N - n0, g.K, s0, wave, lane,
           [](int r) { return ring::perm_row<NW>(r); });
  };
  auto epilogue = [&](int t, ring::f4 (&acc)[G::MI][G::NJ]) {
    int64_t m0, n0;
    int part;
    ring_item(p, t, m0, n0, part);
    if (part >= 0) {
      ring::f4* to = reinterpret_cast<ring::f4*>(g.part) + (int64_t)(t - p.whole) * G::MI * G::NJ * G::NT + threadIdx.x;
#pragma unroll
      for (int i = 0; i < G::MI; ++i)
#pragma unroll
        for (int j = 0; j < G::NJ; ++j) to[(i * G::NJ + j) * G::NT] = acc[i][j];
      return;
    }
#pragma unroll
    for (int i = 0; i < G::MI; ++i) finish_block<NW, BK>(g, m0, n0, i, acc[i]);
  };
  ring::run<NW, AK, BK>(lds, p.whole, p.split * p.parts, stages, open_a, open_b, epilogue);
}

template <int NW, bool AK, bool BK>
__global__ __launch_bounds__(ring::Geo<NW>::NT, ring::Geo<NW>::MAX_GROUPS) void ring_kernel(GemmArgs g, RingPlan p) {
  __shared__ __attribute__((aligned(1024))) char lds[ring::Geo<NW>::LDS_BYTES];
  ring_product<NW, AK, BK>(static_cast<const bf16*>(g.a.p), static_cast<const bf16*>(g.b.p), g, p, lds);
}

// Sums the parts of a split tile in order and finishes it; blockIdx.y takes a block
// row of it.
template <int NW, bool BK>
__global__ __launch_bounds__(ring::Geo<NW>::NT) void ring_join_kernel(GemmArgs g, RingPlan p) {
  typedef ring::Geo<NW> G;
  const int i = blockIdx.y, t = p.whole + blockIdx.x * p.parts;
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
  int64_t m0, n0;
  int part;
  ring_item(p, t, m0, n0, part);
  finish_block<NW, BK>(g, m0, n0, i, acc);
}

constexpr int kCus = 256;

// The cut for which an estimate of the product's time is least.
RingPlan plan_ring(const GemmArgs& g) {
  RingPlan best{};
  double least = 1e300;
  for (const int nw : {8, 4}) {
    const int64_t w = nw * 32, tm = (g.M + w - 1) / w, tn = (g.N + w - 1) / w, tiles = tm * tn;
    const int64_t groups = nw == 8 ? kCus : 2 * kCus;
    const int stages = (int)((g.K + ring::KS - 1) / ring::KS);
    const double stage = nw == 8 ? 1.6 : 1.0, lone = nw == 8 ? 1.2 : 0.7;   // us, on a full and a half empty device
    auto consider = [&](int64_t whole, int parts) {
      const int per = (stages + parts - 1) / parts;
      parts = (stages + per - 1) / per;
      const int64_t split = tiles - whole, items = split * parts;
      const int64_t full = whole / groups;
      double t = full * (stages * stage + 2.0);
      const int64_t rest = whole % groups + items;
      t += (double)((rest + groups - 1) / groups) * (per * (rest <= groups / 2 ? lone : stage) + 2.0);
      if (parts > 1) t += 5.0 + (double)items * w * w * 8 / 4.0e6;
      if (t >= least) return;
      least = t;
      best = RingPlan{nw, (int)tm, (int)tn, (int)(parts > 1 ? whole : tiles), (int)(parts > 1 ? split : 0), parts, per, stages};
    };
    consider(tiles, 1);
    const int64_t whole = tiles / groups * groups, rem = tiles - whole;
    if (rem > 0)
      for (int64_t parts = 2; parts <= 32 && parts * 2 <= stages && rem * parts <= 2 * groups; ++parts) consider(whole, (int)parts);
  }
  return best;
}

template <int NW>
hipError_t launch_ring(const GemmArgs& g, const RingPlan& p, hipStream_t st) {
  typedef ring::Geo<NW> G;
  const int64_t items = (int64_t)p.whole + (int64_t)p.split * p.parts;
  const unsigned grid = (unsigned)std::min<int64_t>(kCus * G::MAX_GROUPS, (items + 7) / 8 * 8);
  note_launch("linear", st);
  if (!g.a_kmaj && !g.b_kmaj) ring_kernel<NW, false, false><<<grid, G::NT, 0, st>>>(g, p);
  else if (!g.a_kmaj) ring_kernel<NW, false, true><<<grid, G::NT, 0, st>>>(g, p);
  else ring_kernel<NW, true, true><<<grid, G::NT, 0, st>>>(g, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.split == 0) return e;
  note_launch("linear_join", st);
  const dim3 j((unsigned)p.split, G::MI);
  if (!g.b_kmaj) ring_join_kernel<NW, false><<<j, G::NT, 0, st>>>(g, p);
  else ring_join_kernel<NW, true><<<j, G::NT, 0, st>>>(g, p);
  return hipGetLastError();
}

size_t ring_bytes(const RingPlan& p) {
  return (size_t)p.split * p.parts * (p.nw * 32) * (p.nw * 32) * sizeof(float);
}

// ------------------------------------------------- the activation's gradient

// A thread takes 8 columns of every eighth row of a strip of rows; the columns'
// sums stay in registers and each strip writes one partial.
template <typename T>
__global__ __launch_bounds__(256) void act_grad_kernel(ActGradArgs a, int64_t strip) {
  typedef T vec __attribute__((ext_vector_type(8)));
  __shared__ float red[8][256];
  const int cg = threadIdx.x & 31, rg = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 256 + cg * 8;
  const int64_t end = min(a.rows, (blockIdx.y + 1) * strip);
  float s[8] = {};
  if (c < a.dim) {
    for (int64_t r = blockIdx.y * strip + rg; r < end; r += 8) {
      const vec dy = *reinterpret_cast<const vec*>(static_cast<const T*>(a.dy.p) + r * a.dy.ld + c);
      vec pre, o;
      if (a.pre.p != nullptr) pre = *reinterpret_cast<const vec*>(static_cast<const T*>(a.pre.p) + r * a.pre.ld + c);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float v = a.pre.p != nullptr ? (float)dy[e] * slope_f32(a.act, (float)pre[e]) : (float)dy[e];
        s[e] += v;
        o[e] = (T)v;
      }
      if (a.dp.p != nullptr) *reinterpret_cast<vec*>(static_cast<T*>(a.dp.p) + r * a.dp.ld + c) = o;
    }
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

__global__ __launch_bounds__(256) void column_sum_kernel(const float* part, int parts, int64_t dim, float* out) {
  __shared__ float red[8][32];
  const int64_t c = (int64_t)blockIdx.x * 32 + (threadIdx.x & 31);
  const int g = threadIdx.x >> 5;
  float x = 0.0f;
  if (c < dim)
    for (int p = g; p < parts; p += 8) x += part[p * dim + c];
  red[g][threadIdx.x & 31] = x;
  __syncthreads();
  if (g != 0 || c >= dim) return;
#pragma unroll
  for (int i = 1; i < 8; ++i) x += red[i][threadIdx.x & 31];
  out[c] = x;
}

constexpr int kStrips = 256;  // most strips of rows of a column sum

template <typename T>
void launch_general(const GemmArgs& g, hipStream_t st) {
  const unsigned tiles = (unsigned)(((g.M + 127) / 128) * ((g.N + 127) / 128));
  if (!g.a_kmaj && !g.b_kmaj) gemm_kernel<T, false, false><<<tiles, kThreads, 0, st>>>(g);
  else if (!g.a_kmaj) gemm_kernel<T, false, true><<<tiles, kThreads, 0, st>>>(g);
  else gemm_kernel<T, true, true><<<tiles, kThreads, 0, st>>>(g);
}

}  // namespace

size_t gemm_workspace(const GemmArgs& g) { return g.dtype == 1 ? ring_bytes(plan_ring(g)) : 0; }

hipError_t launch_gemm(const GemmArgs& g, hipStream_t st) {
  if (g.a_kmaj && !g.b_kmaj) return hipErrorInvalidValue;  // no caller has such a product
  if (g.dtype == 1) {
    const RingPlan p = plan_ring(g);
    return p.nw == 8 ? launch_ring<8>(g, p, st) : launch_ring<4>(g, p, st);
  }
  note_launch("linear", st);
  launch_general<float>(g, st);
  return hipGetLastError();
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
  column_sum_kernel<<<(unsigned)((a.dim + 31) / 32), 256, 0, st>>>(a.part, (int)parts, a.dim, a.db);
  return hipGetLastError();
}

}  // namespace ipttt
