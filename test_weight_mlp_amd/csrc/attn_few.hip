// Causal attention forward for few rows over many keys: the single tokens (or a
// few) of decoding sequences.
//
// Bound by reading K and V once.  A workgroup takes one tile of at most 32 flat
// rows of one key head and a range of keys; each of its waves walks every
// NW-th block of 32 keys with its own running softmax and its own two pairs of
// LDS tiles, filled two blocks ahead straight from memory.  The waves never wait
// for each other until their results are joined at the end; ranges of one tile
// are joined by the join kernel.  32 sequences' next tokens over up to 16000 keys, 8
// key heads of width 128 (949 MB): 171 us, 5.5 TB/s; one over 4097 keys, where the
// chain of one load after the other counts: 7.1 us.  Four waves a workgroup: equal.
#include "attn_core.h"
#include "attn.h"
#include "launch.h"

namespace ipttt {
namespace attn {
namespace {

constexpr int kFewWaves = 2;

template <typename T, int DP>
struct Few {
  typedef Tile<T, DP> TL;
  static constexpr int NW = kFewWaves, KT = 32, TB = TL::bytes(KT);
  static constexpr int OP = DP + 4;  // pitch of a row of O in LDS: rows of a quad of banks apart
  static constexpr int WAVE = 4 * TB;
  static constexpr int LDS = NW * WAVE;
  static_assert(32 * OP * 4 + 64 * 4 <= WAVE, "a wave's result fits its tiles");
};

template <typename T, int DP>
__device__ __forceinline__ void few_tile(const Args& a, const RowItem& it, int kvh, const char* __restrict__ K,
                                         const char* __restrict__ V, char* lds) {
  typedef Tile<T, DP> TL;
  typedef Few<T, DP> F;
  typedef typename Elt<T>::frag frag;
  constexpr int ES = sizeof(T), TB = F::TB, NW = F::NW, EPL = Elt<T>::EPL, DB = DP / 32, KT = F::KT;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), h = lane >> 5;
  const int D = a.D;
  const float sl2 = a.scale * kLog2e;
  const Row row(it, a.G, 0, lane);
  const int64_t at = it.q_start + (int64_t)row.t;
  const int head = kvh * a.G + row.g;
  char* mine = lds + wave * F::WAVE;

  const At<T, DP> here(lane);
  typedef RowStream<T, DP, 1, KT> RS;
  const RS ks(a.k.row, D, 0, lane), vs(a.v.row, D, 0, lane);
  const int k_len = it.off + it.q_len;
  const int blocks = (it.k_end - it.k_begin + KT - 1) / KT, steps = (blocks - wave + NW - 1) / NW;
  auto load = [&](int s, int buf) {
    const int key = it.k_begin + (s * NW + wave) * KT;
    ks.issue(K, (int64_t)it.k_start + key, k_len - key, mine + 2 * buf * TB, 0);
    vs.issue(V, (int64_t)it.k_start + key, k_len - key, mine + (2 * buf + 1) * TB, 0);
  };
  frag qf[TL::STEPS];
  row_frags<T, DP>(a.q, it, row, kvh, a.G, D, h, qf);
  if (steps > 0) load(0, 0);
  if (steps > 1) load(1, 1);

  floatx16 o[DB];
#pragma unroll
  for (int db = 0; db < DB; ++db) fill16(o[db], 0.0f);
  float m = -1e38f, l = 0.0f;  // as in the tiles of many rows
  auto step = [&](int s, auto odd) {
    constexpr int B = decltype(odd)::value;
    // this block has landed once at most the next one's loads are pending
    if (s + 1 < steps) loads_pending<2 * RS::N>();
    else loads_pending<0>();
    const char *kt = mine + 2 * B * TB, *vt = kt + TB;
    const int key0 = it.k_begin + (s * NW + wave) * KT;
    floatx16 x;
    fill16(x, 0.0f);
#pragma unroll
    for (int q = 0; q < TL::STEPS; ++q) x = Elt<T>::mma(TL::row(kt, here.row, 0, q), qf[q], x);
    if (key0 + KT > row.all) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (key0 + 8 * (i >> 2) + 4 * h + (i & 3) >= row.lim) x[i] = -INFINITY;
    }
    float top = x[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) top = fmaxf(top, x[i]);
    top = half_max(top) * sl2;
    if (__any(top > m + 8.0f)) {
      const float mn = top > m + 8.0f ? top : m, c = __builtin_amdgcn_exp2f(m - mn);
      m = mn;
      l *= c;
#pragma unroll
      for (int db = 0; db < DB; ++db)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[db][i] *= c;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      x[i] = __builtin_amdgcn_exp2f(fmaf(x[i], sl2, -m));
      l += x[i];
    }
#pragma unroll
    for (int j = 0; j < 16 / EPL; ++j) {
      const frag p = pack<T>(x, j * EPL);
#pragma unroll
      for (int db = 0; db < DB; ++db) o[db] = Elt<T>::mma(TL::col(vt, here.col, 2 * EPL * j, db), p, o[db]);
    }
    // every read of this buffer has returned before it is filled again
    reads_done();
    if (s + 2 < steps) load(s + 2, B);
  };
  for (int s = 0; s < steps; s += 2) {
    step(s, std::integral_constant<int, 0>());
    if (s + 1 < steps) step(s + 1, std::integral_constant<int, 1>());
  }

  // the waves' results, joined: m and l per row, then O in the wave's tiles
  l = half_sum(l);
  float* ow = reinterpret_cast<float*>(mine);
  float* ml = ow + 32 * F::OP;
  if (h == 0) {
    ml[lane] = m;
    ml[32 + lane] = l;
  }
#pragma unroll
  for (int db = 0; db < DB; ++db)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *reinterpret_cast<float4_t*>(ow + (lane & 31) * F::OP + 32 * db + 8 * j + 4 * h) =
          float4_t{o[db][4 * j], o[db][4 * j + 1], o[db][4 * j + 2], o[db][4 * j + 3]};
  __syncthreads();
  const int rows = min(32, it.q_len * a.G - it.r0), quads = D / 4;
  const RowMap rm(it.r0, a.G);
  for (int e = threadIdx.x; e < rows * quads; e += 64 * NW) {
    const int i = e / quads, d = e % quads * 4;
    const float* o0 = reinterpret_cast<const float*>(lds) + i * F::OP + d;
    const float* s0 = reinterpret_cast<const float*>(lds) + 32 * F::OP + i;
    constexpr int W = F::WAVE / 4;
    float top = s0[0];
#pragma unroll
    for (int w = 1; w < NW; ++w) top = fmaxf(top, s0[w * W]);
    float sum = 0.0f;
    float4_t x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float c = __builtin_amdgcn_exp2f(s0[w * W] - top);
      sum = fmaf(c, s0[w * W + 32], sum);
      x += c * *reinterpret_cast<const float4_t*>(o0 + w * W);
    }
    x *= sum == 0.0f ? 0.0f : 1.0f / sum;
    const float lse = sum == 0.0f ? -INFINITY : (top + __builtin_amdgcn_logf(sum)) * kLn2;
    if (it.part >= 0) {
      const int64_t slot = part_row(it.part, a.kv_heads, kvh, i);
      if (d == 0) a.part_lse[slot] = lse;
      *reinterpret_cast<float4_t*>(a.part_o + slot * D + d) = x;
    } else {
      int t, g;
      rm.of(i, &t, &g);
      const int64_t out = it.q_start + (int64_t)rm.t0 + t;
      if (d == 0) a.lse[out * a.heads + kvh * a.G + g] = lse;
      store4<T>(static_cast<T*>(a.o.p) + out * a.o.row + (kvh * a.G + g) * a.o.head + d, x[0], x[1], x[2], x[3]);
    }
  }
}

template <typename T, int DP>
__global__ __launch_bounds__(64 * kFewWaves, 1) void few_kernel(Args a) {
  __shared__ __attribute__((aligned(16))) char lds[Few<T, DP>::LDS];
  const int kvh = blockIdx.x % a.kv_heads;
  const RowItem it = static_cast<const RowItem*>(a.items)[blockIdx.x / a.kv_heads];
  few_tile<T, DP>(a, it, kvh, static_cast<const char*>(a.k.p) + (int64_t)kvh * a.k.head * (int)sizeof(T),
                  static_cast<const char*>(a.v.p) + (int64_t)kvh * a.v.head * (int)sizeof(T), lds);
}

}  // namespace

hipError_t launch_few(const Args& a, hipStream_t st) {
  const dim3 grid((unsigned)(a.n_items * a.kv_heads));
  note_launch("attn_few", st);
  if (a.dtype == 1 && a.D <= 64) few_kernel<bf16, 64><<<grid, 64 * kFewWaves, 0, st>>>(a);
  else if (a.dtype == 1) few_kernel<bf16, 128><<<grid, 64 * kFewWaves, 0, st>>>(a);
  else if (a.D <= 64) few_kernel<float, 64><<<grid, 64 * kFewWaves, 0, st>>>(a);
  else few_kernel<float, 128><<<grid, 64 * kFewWaves, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace attn
}  // namespace ipttt
