// Causal attention backward over packed sequences with grouped heads.  With
// P = e^(scale q.k - lse), dP = dO V^T and delta = sum_d dO O:
//   dS = P (dP - delta),  dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dO.
// Every tile recomputes P from lse: tiles of rows form dQ, tiles of keys dK and
// dV (summed over the rows of every head of the group), all in one launch, so
// that the ends of the one kind are filled by the other.  Seven products instead
// of the five that tiles of keys with atomic adds to dQ would do, but every sum
// runs in a fixed order: the gradients are the same bits in every run.  A small
// launch before it forms delta.
#include "attn_core.h"
#include "attn.h"
#include "launch.h"

#include <type_traits>

namespace ipttt {
namespace attn {
namespace {

// Rows that see at most so many keys get delta = sum_j P dP from the keys
// themselves (one pass more over them); the others from the forward's O.  In
// bf16, O's rounding (2^-9 of it) goes into delta, and it is not small beside dP
// while O averages few values: dQ's error against 64 bits, random data of 2, 64 and
// 256 keys, is 0.0049, 0.0027, 0.0025 with O and 0.0024, 0.0024, 0.0023 without.
// Over whole sequences these bounds keep dQ within 1.5 times the error of rounding it
// alone, 1.41 to 1.45 of which are dS's and its own rounding (sequences of 333 to 1999
// tokens of width 64: 1.50 with a bound of 512, 1.46 of 1024, 1.45 of 2048; 1500 of
// width 128: 1.48 of 512, 1.45 of 1024), and this part short beside the rest (the same
// sequences, forward and backward: 97, 102 and 114 us).  Narrow heads average fewer
// roundings in delta and need more.
// fp32: where one probability is near 1, dP - delta is what dP's own rounding
// leaves unless delta was made of the same dP and of P's that add up to 1 (sequences
// of 9 tokens: dQ 1.0 times a plain fp32 form's error, 1.6 with O; of 120: 1.12 and
// 1.18; one of 300 and one of 30 tokens, forward and backward: 52.6 us and 47.8).
template <typename T>
__device__ __forceinline__ int exact_delta_keys(int D) {
  return sizeof(T) == 4 ? 64 : max(768, 73728 / D);
}

// Whether a sequence's P and dS go into bf16's products as two terms each, 16 bits in
// all: a few probabilities, each in many elements of a gradient, do not average their
// roundings (3 tokens: dQ 1.7 times the error of rounding it alone; in two terms 1.0).
// The sequence's own keys decide, whatever it is packed with (forward and backward, 32
// heads over 8 of width 128, in one term and two: 9 tokens 15.5 and 16.7 us, 100
// sequences of 9 tokens 41 and 45, 400 of 30 tokens 243 and 277).
__device__ __forceinline__ bool short_keys(int k_len) { return k_len <= kShortKeys; }

// Where lse and delta are taken off.  bf16: the accumulators start at -lse / scale
// and -delta, which costs no instruction.  fp32: after the products; sums that start
// ten times as large as the score round ten times as coarsely at every step (dQ's
// error against 64 bits, 2300 tokens of width 128: 1.1e-6, and 1.9e-6 from -lse /
// scale; a plain fp32 form's 0.9e-6).
template <typename T>
struct Shift {
  static constexpr bool kLate = sizeof(T) == 4;
  // of a row, from its lse
  static __device__ __forceinline__ float of(float lse, float scale) { return kLate ? -lse * kLog2e : -lse / scale; }
  // P and dS of one element, from what the accumulators hold
  static __device__ __forceinline__ float p(float s, float sl2, float shift) {
    return __builtin_amdgcn_exp2f(kLate ? fmaf(s, sl2, shift) : s * sl2);
  }
  static __device__ __forceinline__ float ds(float p, float dp, float ndelta) { return p * (kLate ? dp + ndelta : dp); }
};

// The shift (Shift::of) and -delta of one tile of 128 flat rows, 32 a wave.
template <typename T, int DP>
__device__ __forceinline__ void delta_tile(const Args& a, const RowItem& it, int kvh, const char* __restrict__ K,
                                           const char* __restrict__ V, char* lds) {
  typedef Tile<T, DP> TL;
  typedef typename Elt<T>::frag frag;
  constexpr int NW = 4, KT = sizeof(T) == 2 ? kKeys : kKeys / 2, TB = TL::bytes(KT), EPL = Elt<T>::EPL;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), h = lane >> 5;
  const int D = a.D;
  const Row row(it, a.G, wave, lane);
  const int64_t at = (it.q_start + (int64_t)row.t) * a.heads + kvh * a.G + row.g;
  float nlse = -INFINITY;
  if (row.live) {
    const float x = a.lse[at];
    if (x != -INFINITY) nlse = Shift<T>::of(x, a.scale);
  }
  frag df[TL::STEPS];
  row_frags<T, DP>(a.dO, it, row, kvh, a.G, D, h, df);
  float delta = 0.0f;
  if (it.k_end <= exact_delta_keys<T>(D)) {
    frag qf[TL::STEPS];
    row_frags<T, DP>(a.q, it, row, kvh, a.G, D, h, qf);
    const float sl2 = a.scale * kLog2e;
    const At<T, DP> here(lane);
    const RowStream<T, DP, NW, KT> ks(a.k.row, D, wave, lane), vs(a.v.row, D, wave, lane);
    auto load = [&](int key0, char* tile) {
      const int left = it.off + it.q_len - key0;
      ks.issue(K, (int64_t)it.k_start + key0, left, tile, wave);
      vs.issue(V, (int64_t)it.k_start + key0, left, tile + TB, wave);
    };
    float l = 0.0f, sum[4] = {};
    if (it.k_end > 0) load(0, lds);
    for (int key0 = 0, odd = 0; key0 < it.k_end; key0 += KT, odd ^= 1) {
      const char* tile = lds + odd * 2 * TB;
      tiles_landed();
      if (key0 + KT < it.k_end) load(key0 + KT, lds + (odd ^ 1) * 2 * TB);
      floatx16 x[KT / 32], dp[KT / 32];
#pragma unroll
      for (int kb = 0; kb < KT / 32; ++kb) {
        fill16(x[kb], Shift<T>::kLate ? 0.0f : nlse);
        fill16(dp[kb], 0.0f);
#pragma unroll
        for (int q = 0; q < TL::STEPS; ++q) {
          x[kb] = Elt<T>::mma(TL::row(tile, here.row, 32 * kb, q), qf[q], x[kb]);
          dp[kb] = Elt<T>::mma(TL::row(tile + TB, here.row, 32 * kb, q), df[q], dp[kb]);
        }
      }
      if (key0 + KT > row.all) {
#pragma unroll
        for (int kb = 0; kb < KT / 32; ++kb)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (key0 + 32 * kb + 8 * (i >> 2) + 4 * h + (i & 3) >= row.lim) x[kb][i] = -INFINITY;
      }
#pragma unroll
      for (int kb = 0; kb < KT / 32; ++kb)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float p = Shift<T>::p(x[kb][i], sl2, nlse);
          sum[i & 3] = fmaf(p, dp[kb][i], sum[i & 3]);
          l += p;
        }
    }
    delta = (sum[0] + sum[1]) + (sum[2] + sum[3]);
    if constexpr (Shift<T>::kLate) {  // P's sum is 1 only within lse's rounding; bf16's P are rounded anyhow
      l = half_sum(l);
      if (l > 0.0f) delta /= l;
    }
  } else {
    frag of[TL::STEPS];
    row_frags<T, DP>(a.o, it, row, kvh, a.G, D, h, of);
#pragma unroll
    for (int s = 0; s < TL::STEPS; ++s)
#pragma unroll
      for (int e = 0; e < EPL; ++e) delta = fmaf((float)of[s][e], (float)df[s][e], delta);
  }
  delta = half_sum(delta);
  if (row.live && h == 0) {
    a.nlse[at] = nlse;
    a.ndelta[at] = -delta;
  }
}

// Bound by reading O and dO once (8192 tokens, 32 heads of width 128: 29 us, 4.6 TB/s),
// where rows see few keys by the products (4 sequences of 333 to 1999 tokens, 16
// heads over 8 of width 64: 21 us).
template <typename T, int DP>
__global__ __launch_bounds__(256) void delta_kernel(Args a) {
  __shared__ __attribute__((aligned(16))) char lds[4 * Tile<T, DP>::bytes(sizeof(T) == 2 ? kKeys : kKeys / 2)];
  const int kvh = blockIdx.x % a.kv_heads;
  const RowItem it = static_cast<const RowItem*>(a.items)[blockIdx.x / a.kv_heads];
  delta_tile<T, DP>(a, it, kvh, static_cast<const char*>(a.k.p) + (int64_t)kvh * a.k.head * (int)sizeof(T),
                    static_cast<const char*>(a.v.p) + (int64_t)kvh * a.v.head * (int)sizeof(T), lds);
}

// dQ of one tile of 128 flat rows, 32 a wave: over the keys the rows see,
// S^T = K Q^T and dP^T = V dO^T, then dQ^T += K^T dS^T with K read transposed.
// bf16: what comes out of the products is ready for the exponential and for dS.
template <typename T, int DP, bool SHORT, bool TWICE>
__device__ __forceinline__ void dq_tile(const Args& a, const RowItem& it, int kvh, const char* __restrict__ K,
                                        const char* __restrict__ V, char* lds) {
  typedef Tile<T, DP> TL;
  typedef Groups<T, DP> GR;
  typedef typename Elt<T>::frag frag;
  constexpr int NW = 4, ES = sizeof(T), KT = ES == 2 ? kKeys : kKeys / 2, TB = TL::bytes(KT), EPL = Elt<T>::EPL;
  constexpr int DB = DP / 32, H = GR::H;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), h = lane >> 5;
  const int D = a.D;
  const float sl2 = a.scale * kLog2e;
  const Row row(it, a.G, wave, lane);
  const int64_t at = it.q_start + (int64_t)row.t;
  const int head = kvh * a.G + row.g;

  const At<T, DP> here(lane);
  const RowStream<T, DP, NW, KT> ks(a.k.row, D, wave, lane), vs(a.v.row, D, wave, lane);
  const int k_len = it.off + it.q_len, steps = (it.k_end - it.k_begin + KT - 1) / KT;
  auto load = [&](int s, int buf) {
    const int key = it.k_begin + s * KT;
    ks.issue(K, (int64_t)it.k_start + key, k_len - key, lds + 2 * buf * TB, wave);
    vs.issue(V, (int64_t)it.k_start + key, k_len - key, lds + (2 * buf + 1) * TB, wave);
  };
  if (steps > 0) load(0, 0);

  frag qf[TL::STEPS], df[TL::STEPS];
  row_frags<T, DP>(a.q, it, row, kvh, a.G, D, h, qf);
  row_frags<T, DP>(a.dO, it, row, kvh, a.G, D, h, df);
  // -inf (P = 0) on rows that see nothing, and past the sequence
  const float nlse = row.live ? a.nlse[at * a.heads + head] : -INFINITY;
  const float ndelta = row.live ? a.ndelta[at * a.heads + head] : 0.0f;

  floatx16 acc[DB];
#pragma unroll
  for (int db = 0; db < DB; ++db) fill16(acc[db], 0.0f);

  // One tile of keys, in blocks of 32: the products of a block run while the
  // vector units work on the scores or gradients of the block before.
  auto step = [&](int st, auto odd) {
    constexpr int B = decltype(odd)::value;
    constexpr int NB = KT / 32;
    tiles_landed();
    if (it.k_begin + st * KT >= row.any) {  // no row of this wave sees these keys
      if (st + 1 < steps) load(st + 1, B ^ 1);
      return;
    }
    const char *kt = lds + 2 * B * TB, *vt = kt + TB;
    frag f[2][4], p[NB][GR::NP], p2[NB][GR::NP];
    floatx16 s[NB], dp[NB];
    int cur = 0;
    GR::rows(kt, here, 0, 0, f[0]);
    // dS of block b from its P and dP - delta
    auto grad = [&](int b) {
#pragma unroll
      for (int i = 0; i < 16; ++i) s[b][i] = Shift<T>::ds(s[b][i], dp[b][i], ndelta);
      // a softmax over one key has no gradient: exactly 0, whatever rounding
      // put between dP and delta
      if (b == 0 && st == 0 && it.k_begin == 0 && row.all <= 1 && row.lim == 1) fill16(s[b], 0.0f);
#pragma unroll
      for (int j = 0; j < GR::NP; ++j) {
        p[b][j] = pack<T>(s[b], j * EPL);
        if constexpr (TWICE) p2[b][j] = rest<T>(s[b], j * EPL, p[b][j]);
      }
    };
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      start16(s[b], Shift<T>::kLate ? 0.0f : nlse);
      start16(dp[b], Shift<T>::kLate ? 0.0f : ndelta);
#pragma unroll
      for (int g = 0; g < H; ++g) {
        if (g + 1 < H) GR::rows(kt, here, 32 * b, g + 1, f[cur ^ 1]);
        else GR::rows(vt, here, 32 * b, 0, f[cur ^ 1]);
#pragma unroll
        for (int x = 0; x < 4; ++x) s[b] = Elt<T>::mma(f[cur][x], qf[4 * g + x], s[b]);
        if (b > 0 && g == 0) grad(b - 1);
        cur ^= 1;
        __builtin_amdgcn_sched_barrier(0);
        if (b == 0 && g == 0 && st + 1 < steps) load(st + 1, B ^ 1);
      }
      const int key0 = it.k_begin + st * KT + 32 * b;
      if (key0 + 32 > row.all) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (key0 + 8 * (i >> 2) + 4 * h + (i & 3) >= row.lim) s[b][i] = -INFINITY;
      }
#pragma unroll
      for (int g = 0; g < H; ++g) {
        if (g + 1 < H) GR::rows(vt, here, 32 * b, g + 1, f[cur ^ 1]);
        else if (b + 1 < NB) GR::rows(kt, here, 32 * (b + 1), 0, f[cur ^ 1]);
        else GR::cols(kt, here, 0, 0, f[cur ^ 1]);
#pragma unroll
        for (int i = g * (16 / H); i < (g + 1) * (16 / H); ++i) s[b][i] = Shift<T>::p(s[b][i], sl2, nlse);
#pragma unroll
        for (int x = 0; x < 4; ++x) dp[b] = Elt<T>::mma(f[cur][x], df[4 * g + x], dp[b]);
        cur ^= 1;
        __builtin_amdgcn_sched_barrier(0);
      }
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      if (NB == 1) grad(0);
#pragma unroll
      for (int g = 0; g < H; ++g) {
        if (g + 1 < H) GR::cols(kt, here, 32 * b, g + 1, f[cur ^ 1]);
        else if (b + 1 < NB) GR::cols(kt, here, 32 * (b + 1), 0, f[cur ^ 1]);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int y = 4 * g + x;
          acc[y % DB] = Elt<T>::mma(f[cur][x], p[b][y / DB], acc[y % DB]);
          if constexpr (TWICE) acc[y % DB] = Elt<T>::mma(f[cur][x], p2[b][y / DB], acc[y % DB]);
        }
        if (b + 1 < NB && g == 0) grad(b + 1);
        cur ^= 1;
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  int st = 0;
  while (st < steps) {
    step(st++, std::integral_constant<int, 0>());
    if (st >= steps) break;
    step(st++, std::integral_constant<int, 1>());
  }
  if (!row.live) return;
  if (it.part >= 0) {
    float* x = a.part_dq + part_row(it.part, a.kv_heads, kvh, row.r - it.r0) * D;
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int d = 32 * db + 8 * j + 4 * h;
        if (d < D) store4<float>(x + d, acc[db][4 * j], acc[db][4 * j + 1], acc[db][4 * j + 2], acc[db][4 * j + 3]);
      }
    return;
  }
  T* out = static_cast<T*>(a.dq.p) + at * a.dq.row + head * a.dq.head;
#pragma unroll
  for (int db = 0; db < DB; ++db)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int d = 32 * db + 8 * j + 4 * h;
      if (d < D)
        store4<T>(out + d, acc[db][4 * j] * a.scale, acc[db][4 * j + 1] * a.scale, acc[db][4 * j + 2] * a.scale,
                  acc[db][4 * j + 3] * a.scale);
    }
}

// dK and dV of one tile of 128 keys, 32 a wave: over the flat rows that see any
// of them (all heads of the group), 32 a step, S = Q K^T and dP = dO V^T (a lane
// holds one key), then dV^T += dO^T P and dK^T += Q^T dS with dO and Q read
// transposed.  K stays in registers; V stays in LDS, which keeps a wave within
// half a SIMD's registers, so that two run at once.
template <typename T, int DP>
struct KeyTile {
  typedef Tile<T, DP> TL;
  static constexpr int RT = kBwdRows, TB = TL::bytes(RT), VB = TL::bytes(kBwdKeys);
  static constexpr int STAT = VB + 4 * TB;           // [buffer][shift, -delta][row]
  static constexpr int LDS = STAT + 2 * 2 * RT * 4;
};

// The C block's rows of 32 row values: rows 8 j + 4 h + i in registers 4 j + i.
__device__ __forceinline__ void row_stats(const float* x, int h, floatx16& c) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float4_t v = *reinterpret_cast<const float4_t*>(x + 8 * j + 4 * h);
#pragma unroll
    for (int i = 0; i < 4; ++i) c[4 * j + i] = v[i];
  }
}

template <typename T, int DP, bool SHORT, bool TWICE>
__device__ __forceinline__ void dkv_tile(const Args& a, const KeyItem& it, int kvh, const char* __restrict__ Q,
                                         const char* __restrict__ dO, const float* __restrict__ nlse,
                                         const float* __restrict__ ndelta, const char* __restrict__ K,
                                         const char* __restrict__ V, char* lds) {
  typedef Tile<T, DP> TL;
  typedef Groups<T, DP> GR;
  typedef KeyTile<T, DP> KT;
  typedef typename Elt<T>::frag frag;
  constexpr int NW = 4, ES = sizeof(T), RT = KT::RT, TB = KT::TB, EPL = Elt<T>::EPL, DB = DP / 32, H = GR::H;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), h = lane >> 5;
  const int G = a.G, D = a.D, r_end = it.r_end, k_len = it.off + it.q_len;
  const float sl2 = a.scale * kLog2e;

  const At<T, DP> here(lane);
  const int wkey = it.key0 + wave * 32, key = wkey + (lane & 31);
  const bool live = key < k_len;
  const int64_t krow = (int64_t)it.k_start + key;
  {
    const RowStream<T, DP, NW, kBwdKeys> vs(a.v.row, D, wave, lane);
    vs.issue(V, (int64_t)it.k_start + it.key0, k_len - it.key0, lds, wave);
  }
  frag kf[TL::STEPS];
  row_frags<T, DP>(rsrc_of(K + ((int64_t)it.k_start + it.key0) * a.k.row * ES, kMaxBytes),
                   live ? (uint32_t)((key - it.key0) * (int)a.k.row) * ES : kOob, D, h, kf);
  // the first flat row that sees this key, the wave's first key, its last
  const int from = live ? max(0, key - it.off) * G : 0x7FFFFFFF;
  const int any = wkey < k_len ? max(0, wkey - it.off) * G : 0x7FFFFFFF;
  const int all = wkey + 32 > k_len ? 0x7FFFFFFF : max(0, wkey + 31 - it.off) * G;
  // the end of the flat rows that see key 0 alone (none before its first row)
  const int one = wkey == 0 && it.off <= 0 ? (1 - it.off) * G : 0;
  const int one_row = key == 0 ? one : 0;

  floatx16 dk[DB], dv[DB];
#pragma unroll
  for (int db = 0; db < DB; ++db) {
    fill16(dk[db], 0.0f);
    fill16(dv[db], 0.0f);
  }

  // Steps of 32 rows from r_begin, the last first: tiles of other keys of the
  // sequence end at the same row, so workgroups that start together read the
  // same rows at the same time.  Straight to LDS; rows past the end read as
  // zeros, which add nothing.
  const int r_last = it.r_begin + max(0, it.r_end - it.r_begin - 1) / RT * RT;
  RowMap rm(r_last, G);
  const int t_step = RT / G, g_step = RT - t_step * G;
  auto load = [&](int r0, int buf) {
    const int64_t row = it.q_start + (int64_t)rm.t0;
    const __amdgpu_buffer_rsrc_t rq = rsrc_of(Q + row * a.q.row * ES, kMaxBytes);
    const __amdgpu_buffer_rsrc_t rd = rsrc_of(dO + row * a.dO.row * ES, kMaxBytes);
    constexpr int N = RT / (NW * TL::RPI);
    static_assert(N > 0 && RT % (NW * TL::RPI) == 0, "rows per wave");
    char* qt = lds + KT::VB + 2 * buf * TB;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int blk = wave * N + j;
      int i, c, t, g;
      TL::source(lane, &i, &c);
      i += blk * TL::RPI;
      rm.of(i, &t, &g);
      const bool ok = r0 + i < r_end && c * 16 < D * ES;
      const uint32_t oq = (uint32_t)(t * (int)a.q.row + g * (int)a.q.head) * ES + (uint32_t)c * 16u;
      const uint32_t od = (uint32_t)(t * (int)a.dO.row + g * (int)a.dO.head) * ES + (uint32_t)c * 16u;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rq, (lds_ptr_t)(qt + blk * TL::PITCH), 16, ok ? oq : kOob, 0, 0, 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rd, (lds_ptr_t)(qt + TB + blk * TL::PITCH), 16, ok ? od : kOob, 0, 0, 0);
    }
    if (wave < 2) {  // the shift by wave 0, -delta by wave 1, 32 lanes each
      const __amdgpu_buffer_rsrc_t rs = rsrc_of((wave == 0 ? nlse : ndelta) + row * a.heads, kMaxBytes);
      int t, g;
      rm.of(lane & 31, &t, &g);
      const bool ok = r0 + (lane & 31) < r_end;
      if (lane < 32)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr_t)(lds + KT::STAT + (2 * buf + wave) * RT * 4), 4,
                                                 ok ? (uint32_t)(t * a.heads + g) * 4u : kOob, 0, 0, 0);
    }
    // the next step's first row
    rm.t0 -= t_step;
    rm.g0 -= g_step;
    if (rm.g0 < 0) {
      rm.g0 += G;
      --rm.t0;
    }
  };

  auto step = [&](int r0, auto odd) {
    constexpr int B = decltype(odd)::value;
    tiles_landed();
    if (r0 + RT <= any) {  // no row of these sees a key of this wave
      if (r0 > it.r_begin) load(r0 - RT, B ^ 1);
      return;
    }
    const char *qt = lds + KT::VB + 2 * B * TB, *ot = qt + TB;
    const float* stat = reinterpret_cast<const float*>(lds + KT::STAT + 2 * B * RT * 4);
    frag f[2][4];
    int cur = 0;
    GR::rows(qt, here, 0, 0, f[0]);
    floatx16 shift, ndelta;
    row_stats(stat, h, shift);
    row_stats(stat + RT, h, ndelta);
    floatx16 s = shift, dp = ndelta;
    if constexpr (Shift<T>::kLate) {
      fill16(s, 0.0f);
      fill16(dp, 0.0f);
    }
    auto pair = [&](int g, frag(&x)[4]) {  // two fragments of dO, two of V
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x[i] = TL::row(ot, here.row, 0, 2 * g + i);
        x[2 + i] = TL::row(lds, here.row + wave * TL::bytes(32), 0, 2 * g + i);
      }
    };
#pragma unroll
    for (int g = 0; g < H; ++g) {
      if (g + 1 < H) GR::rows(qt, here, 0, g + 1, f[cur ^ 1]);
      else pair(0, f[cur ^ 1]);
#pragma unroll
      for (int x = 0; x < 4; ++x) s = Elt<T>::mma(f[cur][x], kf[4 * g + x], s);
      cur ^= 1;
      __builtin_amdgcn_sched_barrier(0);
      // the next step's loads, while the matrix cores are busy
      if (g == 0 && r0 > it.r_begin) load(r0 - RT, B ^ 1);
    }
    if (r0 < all) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (r0 + 8 * (i >> 2) + 4 * h + (i & 3) < from) s[i] = -INFINITY;
    }
#pragma unroll
    for (int g = 0; g < 2 * H; ++g) {
      if (g + 1 < 2 * H) pair(g + 1, f[cur ^ 1]);
      else GR::cols(ot, here, 0, 0, f[cur ^ 1]);
      constexpr int EX = 16 / (2 * H);
#pragma unroll
      for (int i = g * EX; i < (g + 1) * EX; ++i) s[i] = Shift<T>::p(s[i], sl2, shift[i]);
#pragma unroll
      for (int x = 0; x < 2; ++x) dp = Elt<T>::mma(f[cur][x], f[cur][2 + x], dp);
      cur ^= 1;
      __builtin_amdgcn_sched_barrier(0);
    }
    frag p[GR::NP], d[GR::NP], p2[GR::NP], d2[GR::NP];
#pragma unroll
    for (int j = 0; j < GR::NP; ++j) {
      p[j] = pack<T>(s, j * EPL);
      if constexpr (TWICE) p2[j] = rest<T>(s, j * EPL, p[j]);
    }
#pragma unroll
    for (int g = 0; g < H; ++g) {
      if (g + 1 < H) GR::cols(ot, here, 0, g + 1, f[cur ^ 1]);
      else GR::cols(qt, here, 0, 0, f[cur ^ 1]);
#pragma unroll
      for (int i = g * (16 / H); i < (g + 1) * (16 / H); ++i)
        dp[i] = Shift<T>::ds(s[i], dp[i], ndelta[i]);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int y = 4 * g + x;
        dv[y % DB] = Elt<T>::mma(f[cur][x], p[y / DB], dv[y % DB]);
        if constexpr (TWICE) dv[y % DB] = Elt<T>::mma(f[cur][x], p2[y / DB], dv[y % DB]);
      }
      cur ^= 1;
      __builtin_amdgcn_sched_barrier(0);
    }
    // rows that see this one key have no gradient through the softmax
    if (r0 < one) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (r0 + 8 * (i >> 2) + 4 * h + (i & 3) < one_row) dp[i] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < GR::NP; ++j) {
      d[j] = pack<T>(dp, j * EPL);
      if constexpr (TWICE) d2[j] = rest<T>(dp, j * EPL, d[j]);
    }
#pragma unroll
    for (int g = 0; g < H; ++g) {
      if (g + 1 < H) GR::cols(qt, here, 0, g + 1, f[cur ^ 1]);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int y = 4 * g + x;
        dk[y % DB] = Elt<T>::mma(f[cur][x], d[y / DB], dk[y % DB]);
        if constexpr (TWICE) dk[y % DB] = Elt<T>::mma(f[cur][x], d2[y / DB], dk[y % DB]);
      }
      cur ^= 1;
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  if (it.r_begin < r_end) load(r_last, 0);
  for (int r0 = r_last; it.r_begin < r_end;) {
    step(r0, std::integral_constant<int, 0>());
    if ((r0 -= RT) < it.r_begin) break;
    step(r0, std::integral_constant<int, 1>());
    if ((r0 -= RT) < it.r_begin) break;
  }
  if (!live) return;
  if (it.part >= 0) {
    float* o = a.part_o + (((int64_t)it.part * a.kv_heads + kvh) * 2 * kBwdKeys + (key - it.key0)) * D;
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int d = 32 * db + 8 * j + 4 * h;
        if (d < D) {
          store4<float>(o + d, dk[db][4 * j], dk[db][4 * j + 1], dk[db][4 * j + 2], dk[db][4 * j + 3]);
          store4<float>(o + kBwdKeys * D + d, dv[db][4 * j], dv[db][4 * j + 1], dv[db][4 * j + 2], dv[db][4 * j + 3]);
        }
      }
    return;
  }
  T* ok = static_cast<T*>(a.dk.p) + krow * a.dk.row + (int64_t)kvh * a.dk.head;
  T* ov = static_cast<T*>(a.dv.p) + krow * a.dv.row + (int64_t)kvh * a.dv.head;
#pragma unroll
  for (int db = 0; db < DB; ++db)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int d = 32 * db + 8 * j + 4 * h;
      if (d < D) {
        store4<T>(ok + d, dk[db][4 * j] * a.scale, dk[db][4 * j + 1] * a.scale, dk[db][4 * j + 2] * a.scale,
                  dk[db][4 * j + 3] * a.scale);
        store4<T>(ov + d, dv[db][4 * j], dv[db][4 * j + 1], dv[db][4 * j + 2], dv[db][4 * j + 3]);
      }
    }
}

// The tiles of keys (longest first), then those of rows.  bf16: two waves a SIMD.
// Bound by the matrix cores at the clock that the card's power allows, and by what
// keeps them waiting: 8192 tokens, 32 heads over 8 of width 128: 1.61 ms, 1.19 PFLOP/s
// of its seven products, matrix cores 65 % busy at 1.77 GHz.
// SHORT: sequences of few keys, whose P and dS go in two terms, are among them; at
// width 128 both kinds of tile together do not fit a wave's registers (8180 tokens
// beside 12, forward and backward: 2.16 ms, 2.13 with one kind).  Its tiles have SHORT
// as a parameter too: hipcc's host pass takes one use of each.
template <typename T, int DP, bool SHORT = false>
__global__ __launch_bounds__(256, sizeof(T) == 4 ? 1 : 2) void bwd_kernel(Args a) {
  constexpr int ES = sizeof(T), DQ = 4 * Tile<T, DP>::bytes(ES == 2 ? kKeys : kKeys / 2);
  __shared__ __attribute__((aligned(16))) char lds[KeyTile<T, DP>::LDS > DQ ? KeyTile<T, DP>::LDS : DQ];
  const int kvh = blockIdx.x % a.kv_heads, i = blockIdx.x / a.kv_heads;
  const char* K = static_cast<const char*>(a.k.p) + (int64_t)kvh * a.k.head * ES;
  const char* V = static_cast<const char*>(a.v.p) + (int64_t)kvh * a.v.head * ES;
  if (i < a.n_items) {
    const int64_t q = (int64_t)kvh * a.G;
    const char* Q = static_cast<const char*>(a.q.p) + q * a.q.head * ES;
    const char* dO = static_cast<const char*>(a.dO.p) + q * a.dO.head * ES;
    const KeyItem it = static_cast<const KeyItem*>(a.items)[i];
    if constexpr (SHORT) {
      if (short_keys(it.off + it.q_len)) {
        dkv_tile<T, DP, SHORT, true>(a, it, kvh, Q, dO, a.nlse + q, a.ndelta + q, K, V, lds);
        return;
      }
    }
    dkv_tile<T, DP, SHORT, false>(a, it, kvh, Q, dO, a.nlse + q, a.ndelta + q, K, V, lds);
  } else {
    const RowItem it = static_cast<const RowItem*>(a.dq_items)[i - a.n_items];
    if constexpr (SHORT) {
      if (short_keys(it.off + it.q_len)) {
        dq_tile<T, DP, SHORT, true>(a, it, kvh, K, V, lds);
        return;
      }
    }
    dq_tile<T, DP, SHORT, false>(a, it, kvh, K, V, lds);
  }
}

// Sums the partial gradients of one tile in slot order, a block 16 rows or keys
// of it, a thread four columns of one at a time: dQ of the first n_dq items, dK
// and dV of the others.  Launch and latency: 6 us after 8192 tokens' backward.
template <typename T>
__global__ __launch_bounds__(256) void join_bwd_kernel(Args a, const JoinItem* dq_items, int n_dq,
                                                       const KeyJoin* key_items) {
  const int kvh = blockIdx.y, D = a.D, quads = D / 4, G = a.G, i0 = 16 * blockIdx.z;
  if ((int)blockIdx.x < n_dq) {
    const JoinItem it = dq_items[blockIdx.x];
    const int64_t step = (int64_t)it.step * a.kv_heads * kPartRows * D;
    const int rows = min(16, min(kRows, it.q_len * G - it.r0) - i0);
    for (int e = threadIdx.x; e < rows * quads; e += 256) {
      const int i = i0 + e / quads, d = e % quads * 4;
      const float* p = a.part_dq + part_row(it.part, a.kv_heads, kvh, i) * D + d;
      float4_t x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
      for (int j = 0; j < it.n; ++j) x += *reinterpret_cast<const float4_t*>(p + j * step);
      x *= a.scale;
      const int r = it.r0 + i, t = r / G, head = kvh * G + r - t * G;
      store4<T>(static_cast<T*>(a.dq.p) + (it.q_start + (int64_t)t) * a.dq.row + head * a.dq.head + d, x[0], x[1],
                x[2], x[3]);
    }
    return;
  }
  const KeyJoin it = key_items[blockIdx.x - n_dq];
  const int64_t step = (int64_t)a.kv_heads * 2 * kBwdKeys * D;
  const int keys = min(16, it.n_keys - i0);
  for (int e = threadIdx.x; e < keys * quads; e += 256) {
    const int i = i0 + e / quads, d = e % quads * 4;
    const float* p = a.part_o + (((int64_t)it.part * a.kv_heads + kvh) * 2 * kBwdKeys + i) * D + d;
    float4_t k = {0.0f, 0.0f, 0.0f, 0.0f}, v = k;
#pragma unroll 4
    for (int j = 0; j < it.n; ++j) {
      k += *reinterpret_cast<const float4_t*>(p + j * step);
      v += *reinterpret_cast<const float4_t*>(p + j * step + (int64_t)kBwdKeys * D);
    }
    const int64_t row = (int64_t)it.k_row + i;
    k *= a.scale;
    store4<T>(static_cast<T*>(a.dk.p) + row * a.dk.row + kvh * a.dk.head + d, k[0], k[1], k[2], k[3]);
    store4<T>(static_cast<T*>(a.dv.p) + row * a.dv.row + kvh * a.dv.head + d, v[0], v[1], v[2], v[3]);
  }
}

}  // namespace

hipError_t launch_delta(const Args& a, hipStream_t st) {
  const dim3 grid((unsigned)(a.n_items * a.kv_heads));
  note_launch("attn_delta", st);
  if (a.dtype == 1 && a.D <= 64) delta_kernel<bf16, 64><<<grid, 256, 0, st>>>(a);
  else if (a.dtype == 1) delta_kernel<bf16, 128><<<grid, 256, 0, st>>>(a);
  else if (a.D <= 64) delta_kernel<float, 64><<<grid, 256, 0, st>>>(a);
  else delta_kernel<float, 128><<<grid, 256, 0, st>>>(a);
  return hipGetLastError();
}

hipError_t launch_backward(const Args& a, hipStream_t st) {
  const dim3 grid((unsigned)((a.n_items + a.n_dq) * a.kv_heads));
  note_launch("attn_bwd", st);
  if (a.dtype == 1 && a.D <= 64 && a.shorts) bwd_kernel<bf16, 64, true><<<grid, 256, 0, st>>>(a);
  else if (a.dtype == 1 && a.D <= 64) bwd_kernel<bf16, 64><<<grid, 256, 0, st>>>(a);
  else if (a.dtype == 1 && a.shorts) bwd_kernel<bf16, 128, true><<<grid, 256, 0, st>>>(a);
  else if (a.dtype == 1) bwd_kernel<bf16, 128><<<grid, 256, 0, st>>>(a);
  else if (a.D <= 64) bwd_kernel<float, 64><<<grid, 256, 0, st>>>(a);
  else bwd_kernel<float, 128><<<grid, 256, 0, st>>>(a);
  return hipGetLastError();
}

hipError_t launch_join_backward(const Args& a, const void* dq_items, int n_dq, const void* key_items, int n_key,
                                hipStream_t st) {
  static_assert(kRows == kBwdKeys, "one grid for both kinds of tile");
  const dim3 grid((unsigned)(n_dq + n_key), (unsigned)a.kv_heads, kRows / 16);
  const JoinItem* q = static_cast<const JoinItem*>(dq_items);
  const KeyJoin* k = static_cast<const KeyJoin*>(key_items);
  note_launch("attn_join_bwd", st);
  if (a.dtype == 1) join_bwd_kernel<bf16><<<grid, 256, 0, st>>>(a, q, n_dq, k);
  else join_bwd_kernel<float><<<grid, 256, 0, st>>>(a, q, n_dq, k);
  return hipGetLastError();
}

}  // namespace attn
}  // namespace ipttt
