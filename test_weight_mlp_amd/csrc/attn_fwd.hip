// Causal attention forward over packed sequences with grouped heads.
//
// A workgroup takes one tile of flat (query, head of the group) rows of one key
// head, 32 rows a wave, and walks that sequence's keys 64 at a time with the
// running maximum m and sum l of the softmax (everything in fp32):
//   S^T = K Q^T       32x32 MFMA blocks, K rows from LDS, Q in registers
//   P   = 2^(S scale log2(e) - m)
//   O^T += V^T P^T    V read transposed from LDS, P straight from its registers
// In S^T and O^T a lane holds one query row, so m, l and the rescaling of O
// are per-lane scalars and the row maximum crosses lanes once (l and l ^ 32).
#include "attn_core.h"
#include "attn.h"
#include "launch.h"

#include <algorithm>
#include <type_traits>

namespace ipttt {
namespace attn {
namespace {

// The work of one wave on one step of NB blocks of 32 keys, in phases of MFMAs:
// the next step's scores, a phase a block, then this step's part of O from each
// block.  The vector units meanwhile raise this step's scores to probabilities,
// spread evenly over the phases of scores and the first half of the others (a
// block's phase must find its own raised), and take the next scores' maximum in
// the second half.  Fragments are read from LDS one group of four MFMAs ahead.
template <typename T, int DP, int NB>
struct Step {
  typedef Tile<T, DP> TL;
  typedef Groups<T, DP> GR;
  typedef typename Elt<T>::frag frag;
  static constexpr int EPL = Elt<T>::EPL, DB = DP / 32, H = GR::H;

  // scores [e0, e0 + n) of the step's 16 NB to probabilities
  template <int N>
  static __device__ __forceinline__ void raise(floatx16 (&s)[NB], int e0, float sl2, float m, float& l) {
#pragma unroll
    for (int e = e0; e < e0 + N; ++e) {
      s[e >> 4][e & 15] = __builtin_amdgcn_exp2f(fmaf(s[e >> 4][e & 15], sl2, -m));
      l += s[e >> 4][e & 15];
    }
  }

  // s: this step's scores in, the next step's out (if NEXT) and top their
  // largest; kt: the next step's keys, vt: this step's values; issue() starts
  // the loads of later steps
  template <bool NEXT, class Issue>
  static __device__ __forceinline__ void run(const char* kt, const char* vt, const frag (&qf)[TL::STEPS],
                                             floatx16 (&s)[NB], floatx16 (&o)[DB], float sl2, float m, float& l,
                                             float& top, const At<T, DP>& at, Issue issue) {
    frag f[2][4];
    floatx16 n[NB];
    int cur = 0;
    if constexpr (NEXT) {
      GR::rows(kt, at, 0, 0, f[0]);
#pragma unroll
      for (int kb = 0; kb < NB; ++kb) {
        fill16(n[kb], 0.0f);
#pragma unroll
        for (int g = 0; g < H; ++g) {
          if (g + 1 < H) GR::rows(kt, at, 32 * kb, g + 1, f[cur ^ 1]);
          else if (kb + 1 < NB) GR::rows(kt, at, 32 * (kb + 1), 0, f[cur ^ 1]);
          else GR::cols(vt, at, 0, 0, f[cur ^ 1]);
          raise<12 / H>(s, (kb * H + g) * (12 / H), sl2, m, l);
#pragma unroll
          for (int x = 0; x < 4; ++x) n[kb] = Elt<T>::mma(f[cur][x], qf[4 * g + x], n[kb]);
          cur ^= 1;
          __builtin_amdgcn_sched_barrier(0);
          if (kb == 0 && g == 0) issue();
        }
      }
    } else {
      GR::cols(vt, at, 0, 0, f[0]);
      raise<12 * NB>(s, 0, sl2, m, l);
    }
#pragma unroll
    for (int kb = 0; kb < NB; ++kb) {
      frag p[GR::NP];
#pragma unroll
      for (int j = 0; j < GR::NP; ++j) p[j] = pack<T>(s[kb], j * EPL);
#pragma unroll
      for (int g = 0; g < H; ++g) {
        if (g + 1 < H) GR::cols(vt, at, 32 * kb, g + 1, f[cur ^ 1]);
        else if (kb + 1 < NB) GR::cols(vt, at, 32 * (kb + 1), 0, f[cur ^ 1]);
        if (kb < NB / 2) {
          raise<8 / H>(s, 12 * NB + (kb * H + g) * (8 / H), sl2, m, l);
        } else if constexpr (NEXT) {
          const floatx16 &x = n[2 * (kb - NB / 2)], &y = n[2 * (kb - NB / 2) + 1];
          if (kb == NB / 2 && g == 0) top = x[0];
#pragma unroll
          for (int i = g * (16 / H); i < (g + 1) * (16 / H); ++i) top = fmaxf(fmaxf(top, x[i]), y[i]);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int y = 4 * g + x;
          o[y % DB] = Elt<T>::mma(f[cur][x], p[y / DB], o[y % DB]);
        }
        cur ^= 1;
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if constexpr (NEXT) {
#pragma unroll
      for (int kb = 0; kb < NB; ++kb) s[kb] = n[kb];
    }
  }
};

template <int NB>
__device__ __forceinline__ float largest(const floatx16 (&s)[NB]) {
  float x = s[0][0];
#pragma unroll
  for (int kb = 0; kb < NB; kb += 2)
#pragma unroll
    for (int i = 0; i < 16; ++i) x = fmaxf(fmaxf(x, s[kb][i]), s[kb + 1][i]);
  return x;
}

// Masks a step's scores (whose largest is top) and moves m up if a row's
// maximum passed it by more than 2^8: sums and O are relative to m, exact for any
// m near the maximum, so they are rescaled (one multiplication an element)
// only then, which after the first few steps is rare.  A row's own scores decide:
// its result does not depend on the other rows of its wave.
template <int NB, int DB>
__device__ __forceinline__ void settle(floatx16 (&s)[NB], float top, int key0, const Row& row, float sl2,
                                       floatx16 (&o)[DB], float& m, float& l, int lane) {
  if (key0 + 32 * NB > row.all) {
#pragma unroll
    for (int kb = 0; kb < NB; ++kb)
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (key0 + 32 * kb + 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3) >= row.lim) s[kb][i] = -INFINITY;
    top = largest(s);
  }
  const float x = half_max(top) * sl2;
  if (__any(x > m + 8.0f)) {
    const float mn = x > m + 8.0f ? x : m, c = __builtin_amdgcn_exp2f(m - mn);
    m = mn;
    l *= c;
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[db][i] *= c;
  }
}

template <typename T, int DP, int NB>
__device__ __forceinline__ void fwd_tile(const Args& a, const RowItem& it, int kvh, const char* __restrict__ K,
                                         const char* __restrict__ V, char* lds) {
  typedef Tile<T, DP> TL;
  typedef Step<T, DP, NB> ST;
  typedef typename Elt<T>::frag frag;
  constexpr int NW = 4, ES = sizeof(T), KT = 32 * NB, TB = TL::bytes(KT), DB = DP / 32;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), h = lane >> 5;
  const int D = a.D;
  const float sl2 = a.scale * kLog2e;
  const Row row(it, a.G, wave, lane);
  const int64_t at = it.q_start + (int64_t)row.t;
  const int head = kvh * a.G + row.g;

  const At<T, DP> here(lane);
  const RowStream<T, DP, NW, KT> ks(a.k.row, D, wave, lane), vs(a.v.row, D, wave, lane);
  const int k_len = it.off + it.q_len, steps = (it.k_end - it.k_begin + KT - 1) / KT;
  // keys in buffers 0 and 1, values in 2 and 3, step s in buffer s & 1
  auto keys = [&](int s) {
    const int key = it.k_begin + s * KT;
    ks.issue(K, (int64_t)it.k_start + key, k_len - key, lds + (s & 1) * TB, wave);
  };
  auto values = [&](int s) {
    const int key = it.k_begin + s * KT;
    vs.issue(V, (int64_t)it.k_start + key, k_len - key, lds + (2 + (s & 1)) * TB, wave);
  };
  if (steps > 0) keys(0);

  frag qf[TL::STEPS];
  row_frags<T, DP>(a.q, it, row, kvh, a.G, D, h, qf);
  floatx16 o[DB];
#pragma unroll
  for (int db = 0; db < DB; ++db) fill16(o[db], 0.0f);
  // m starts below every score and stays finite, so that masked scores (-inf)
  // of a row that has seen nothing give 0, not NaN
  float m = -1e38f, l = 0.0f;

  if (steps > 0) {
    tiles_landed();
    values(0);
    if (steps > 1) keys(1);
    floatx16 s[NB];
#pragma unroll
    for (int kb = 0; kb < NB; ++kb) {
      fill16(s[kb], 0.0f);
#pragma unroll
      for (int q = 0; q < TL::STEPS; ++q)
        s[kb] = Elt<T>::mma(TL::row(lds, here.row, 32 * kb, q), qf[q], s[kb]);
    }
    settle(s, largest(s), it.k_begin, row, sl2, o, m, l, lane);
    float top = 0.0f;
    // one step with another to follow; its buffers are known at compile time, so
    // that the LDS addresses of all fragments are a few registers plus immediate
    // offsets.  A wave whose rows see none of the next keys scores them all the
    // same (as -inf): at most the last step or two of a tile.
    auto step = [&](int st, auto odd) {
      constexpr int B = decltype(odd)::value;
      // this step's values and the next one's keys are here, and every wave is
      // done with the buffers that the loads below fill
      tiles_landed();
      ST::template run<true>(lds + (B ^ 1) * TB, lds + (2 + B) * TB, qf, s, o, sl2, m, l, top, here, [&] {
        values(st + 1);
        if (st + 2 < steps) keys(st + 2);
      });
      settle(s, top, it.k_begin + (st + 1) * KT, row, sl2, o, m, l, lane);
    };
    int st = 0;
    while (st < steps - 1) {
      step(st++, std::integral_constant<int, 0>());
      if (st >= steps - 1) break;
      step(st++, std::integral_constant<int, 1>());
    }
    tiles_landed();
    ST::template run<false>(lds, lds + (2 + (st & 1)) * TB, qf, s, o, sl2, m, l, top, here, [] {});
  }
  l = half_sum(l);
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  const float lse = l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2;
  if (!row.live) return;
  if (it.part >= 0) {
    const int64_t slot = part_row(it.part, a.kv_heads, kvh, row.r - it.r0);
    if (h == 0) a.part_lse[slot] = lse;
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int d = 32 * db + 8 * j + 4 * h;
        if (d < D)
          store4<float>(a.part_o + slot * D + d, o[db][4 * j] * inv, o[db][4 * j + 1] * inv, o[db][4 * j + 2] * inv,
                        o[db][4 * j + 3] * inv);
      }
    return;
  }
  if (h == 0) a.lse[at * a.heads + head] = lse;
  T* out = static_cast<T*>(a.o.p) + at * a.o.row + head * a.o.head;
#pragma unroll
  for (int db = 0; db < DB; ++db)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int d = 32 * db + 8 * j + 4 * h;
      if (d < D)
        store4<T>(out + d, o[db][4 * j] * inv, o[db][4 * j + 1] * inv, o[db][4 * j + 2] * inv, o[db][4 * j + 3] * inv);
    }
}

// Two waves a SIMD (256 registers a wave) where the tiles allow it; fp32 of
// width 128 needs the registers of one.  Bound by the matrix cores at the clock
// that the card's power allows, and by what keeps them waiting a third of the time:
// 32 heads over 8 of width 128, one sequence of 32768 tokens 7.7 ms, 1.14 PFLOP/s of
// what the mask leaves, matrix cores 65 % busy at 1.68 GHz (on zeros 67 % at 2.38
// GHz); of 8192 tokens 0.50 ms, 1.09 PFLOP/s.  (256 rows a tile with 8 waves: equal
// at 32768, slower below.)
template <typename T, int DP, int NB>
__global__ __launch_bounds__(256, sizeof(T) * DP > 256 ? 1 : 2) void fwd_kernel(Args a) {
  __shared__ __attribute__((aligned(16))) char lds[4 * Tile<T, DP>::bytes(32 * NB)];
  const int kvh = blockIdx.x % a.kv_heads;
  const RowItem it = static_cast<const RowItem*>(a.items)[blockIdx.x / a.kv_heads];
  fwd_tile<T, DP, NB>(a, it, kvh, static_cast<const char*>(a.k.p) + (int64_t)kvh * a.k.head * (int)sizeof(T),
                      static_cast<const char*>(a.v.p) + (int64_t)kvh * a.v.head * (int)sizeof(T), lds);
}

// Joins the partial results of one tile: with each part's lse, its weight is
// e^(lse_i - lse), lse = log sum e^(lse_i); parts in slot order, eight parts'
// loads in flight.  A tile of many rows: a thread takes four columns of one row.
// One of few rows, which has many parts: a wave takes one row, two columns a
// lane, and its lanes hold the weights of 64 parts (one token over 4097 keys, 22
// parts: 3.2 us; with 33 parts 4.3, and 5.2 as the other kind).
template <typename T>
__device__ __forceinline__ void join_many(const Args& a, const JoinItem& it, int kvh) {
  const int G = a.G, D = a.D, quads = D / 4, per = 256 / quads;
  const int i = blockIdx.z * per + threadIdx.x / quads, r = it.r0 + i, d = threadIdx.x % quads * 4;
  if ((int)threadIdx.x >= per * quads || i >= it.step * kPartRows || r >= it.q_len * G) return;
  const int64_t slot0 = part_row(it.part, a.kv_heads, kvh, i), step = (int64_t)it.step * a.kv_heads * kPartRows;
  const float* ls = a.part_lse + slot0;
  const float* x = a.part_o + slot0 * D + d;
  float m = -INFINITY;
#pragma unroll 8
  for (int p = 0; p < it.n; ++p) m = fmaxf(m, ls[p * step]);
  const float mu = m == -INFINITY ? 0.0f : m;
  float l = 0.0f;
  float4_t o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
  for (int p = 0; p < it.n; ++p) {
    const float w = __builtin_amdgcn_exp2f((ls[p * step] - mu) * kLog2e);
    l += w;
    o += w * *reinterpret_cast<const float4_t*>(x + p * step * D);
  }
  o *= l == 0.0f ? 0.0f : 1.0f / l;
  const int t = r / G, head = kvh * G + r - t * G;
  const int64_t row = it.q_start + (int64_t)t;
  if (d == 0) a.lse[row * a.heads + head] = l == 0.0f ? -INFINITY : mu + __builtin_amdgcn_logf(l) * kLn2;
  store4<T>(static_cast<T*>(a.o.p) + row * a.o.row + head * a.o.head + d, o[0], o[1], o[2], o[3]);
}

template <typename T>
__device__ __forceinline__ void join_few(const Args& a, const JoinItem& it, int kvh) {
  const int G = a.G, D = a.D, lane = threadIdx.x & 63, i = blockIdx.z * 4 + (threadIdx.x >> 6), r = it.r0 + i;
  if (i >= it.step * kPartRows || r >= it.q_len * G) return;
  const int t = r / G, head = kvh * G + r - t * G;
  const int64_t slot0 = part_row(it.part, a.kv_heads, kvh, i), step = (int64_t)it.step * a.kv_heads * kPartRows;
  float m = -INFINITY;
  for (int p = lane; p < it.n; p += 64) m = fmaxf(m, a.part_lse[slot0 + p * step]);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
  const float mu = m == -INFINITY ? 0.0f : m;
  const bool on = 2 * lane < D;
  const float* x = a.part_o + slot0 * D + (on ? 2 * lane : 0);
  float l = 0.0f, x0 = 0.0f, x1 = 0.0f;
  for (int p0 = 0; p0 < it.n; p0 += 64) {  // lane p holds part p0 + p's weight
    const int n = min(64, it.n - p0);
    const float w = lane < n ? __builtin_amdgcn_exp2f((a.part_lse[slot0 + (p0 + lane) * step] - mu) * kLog2e) : 0.0f;
    l += w;
    for (int p = 0; p < n; p += 8) {
      float2_t v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        v[j] = *reinterpret_cast<const float2_t*>(x + (p0 + min(p + j, n - 1)) * step * D);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float wj = __shfl(w, p + j, 64);  // 0 past the last part
        x0 = fmaf(wj, v[j][0], x0);
        x1 = fmaf(wj, v[j][1], x1);
      }
    }
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) l += __shfl_xor(l, o, 64);
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  const int64_t row = it.q_start + (int64_t)t;
  if (lane == 0) a.lse[row * a.heads + head] = l == 0.0f ? -INFINITY : mu + __builtin_amdgcn_logf(l) * kLn2;
  T* out = static_cast<T*>(a.o.p) + row * a.o.row + head * a.o.head;
  if (on) {
    out[2 * lane] = (T)(x0 * inv);
    out[2 * lane + 1] = (T)(x1 * inv);
  }
}

template <typename T>
__global__ __launch_bounds__(256) void join_kernel(Args a, const JoinItem* items) {
  const JoinItem it = items[blockIdx.x];
  if (it.step == 1) join_few<T>(a, it, blockIdx.y);
  else join_many<T>(a, it, blockIdx.y);
}

}  // namespace

hipError_t launch_forward(const Args& a, hipStream_t st) {
  const dim3 grid((unsigned)(a.n_items * a.kv_heads));
  note_launch("attn_fwd", st);
  // steps of 64 keys; bf16 of width 64, whose tiles are small, has steps of 128 and
  // half the barriers (3500 and 900 tokens, 16 heads over 8: 44.6 us, 48.6 with
  // 64), unless tiles are cut into parts (300 and 1000 tokens over 4000 and 9000: 65.2
  // us, 62.2 with 64; 700, 97 and 300 over 700, 1025 and 255: 14.9 and 14.4)
  if (a.dtype == 1 && a.D <= 64 && !a.cut) fwd_kernel<bf16, 64, 4><<<grid, 256, 0, st>>>(a);
  else if (a.dtype == 1 && a.D <= 64) fwd_kernel<bf16, 64, 2><<<grid, 256, 0, st>>>(a);
  else if (a.dtype == 1) fwd_kernel<bf16, 128, 2><<<grid, 256, 0, st>>>(a);
  else if (a.D <= 64) fwd_kernel<float, 64, 2><<<grid, 256, 0, st>>>(a);
  else fwd_kernel<float, 128, 2><<<grid, 256, 0, st>>>(a);
  return hipGetLastError();
}

hipError_t launch_join(const Args& a, const void* items, int n, int rows, hipStream_t st) {
  // rows of a block: 4 of a tile of few rows, per of one of many
  const int per = 256 / (a.D / 4), z = std::max((std::min(rows, kFewRows) + 3) / 4, (rows + per - 1) / per);
  const dim3 grid((unsigned)n, (unsigned)a.kv_heads, (unsigned)z);
  note_launch("attn_join", st);
  if (a.dtype == 1) join_kernel<bf16><<<grid, 256, 0, st>>>(a, static_cast<const JoinItem*>(items));
  else join_kernel<float><<<grid, 256, 0, st>>>(a, static_cast<const JoinItem*>(items));
  return hipGetLastError();
}

}  // namespace attn
}  // namespace ipttt
