// Causal attention backward over packed sequences with grouped heads.  With
// P = e^(scale q.k - lse), dP = dO V^T and delta = sum_d dO O:
//   dS = P (dP - delta),  dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dO.
// Two kernels, each recomputing P from lse: one per tile of rows (dQ, and delta
// on the way), one per tile of keys (dK, dV, summed over the rows of every head
// of the group).  Seven products instead of the five that one kernel with atomic
// adds to dQ would do, but every sum runs in a fixed order: the gradients are
// the same bits in every run.
#include "attn_core.h"
#include "attn.h"
#include "launch.h"

namespace ipttt {
namespace attn {
namespace {

// dQ of one tile of 128 flat rows, 32 a wave: over the keys the rows see,
// S^T = K Q^T and dP^T = V dO^T, then dQ^T += K^T dS^T with K read transposed.
template <typename T, int DP>
__global__ __launch_bounds__(256, 1) void dq_kernel(Args a) {
  typedef Tile<T, DP> TL;
  typedef typename Elt<T>::frag frag;
  constexpr int NW = 4, ES = sizeof(T), KT = sizeof(T) == 2 ? kKeys : kKeys / 2, TB = KT * TL::RB;
  constexpr int EPL = Elt<T>::EPL;
  __shared__ __attribute__((aligned(1024))) char lds[4 * TB];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, h = lane >> 5;
  const int kvh = blockIdx.x % a.kv_heads;
  const RowItem it = static_cast<const RowItem*>(a.items)[blockIdx.x / a.kv_heads];
  const int G = a.G, D = a.D, n_rows = it.q_len * G;
  const float sl2 = a.scale * kLog2e;

  const RowMap rm(it.r0 + wave * 32, G);
  const int r = it.r0 + wave * 32 + (lane & 31);
  int t, g;
  rm.of(lane & 31, &t, &g);
  t += rm.t0;
  const bool live = r < n_rows;
  const int lim = live ? min(it.off + t + 1, it.k_end) : 0;
  const int all = __builtin_amdgcn_readfirstlane(min(it.off + rm.t0 + 1, it.k_end));
  const int r_last = min(it.r0 + wave * 32 + 31, n_rows - 1);
  const int any = __builtin_amdgcn_readfirstlane(
      it.r0 + wave * 32 < n_rows ? min(it.off + r_last / G + 1, it.k_end) : 0);
  const int64_t row = it.q_start + (int64_t)t;
  const int head = kvh * G + g;

  frag qf[TL::STEPS], df[TL::STEPS];
  row_frags<T, DP>(static_cast<const char*>(a.q.p) + (row * a.q.row + head * a.q.head) * ES, live, D, h, qf);
  row_frags<T, DP>(static_cast<const char*>(a.dO.p) + (row * a.dO.row + head * a.dO.head) * ES, live, D, h, df);
  float delta = 0.0f;
  {
    frag of[TL::STEPS];
    row_frags<T, DP>(static_cast<const char*>(a.o.p) + (row * a.o.row + head * a.o.head) * ES, live, D, h, of);
#pragma unroll
    for (int s = 0; s < TL::STEPS; ++s)
#pragma unroll
      for (int e = 0; e < EPL; ++e) delta = fmaf((float)of[s][e], (float)df[s][e], delta);
    delta += other_half(delta);
  }
  float lse2 = INFINITY;  // P = 0 on rows that see nothing, and past the sequence
  if (live) {
    const float x = a.lse[row * a.heads + head];
    if (x != -INFINITY) lse2 = x * kLog2e;
    if (h == 0) a.delta[row * a.heads + head] = delta;
  }

  floatx16 acc[DP / 32];
#pragma unroll
  for (int db = 0; db < DP / 32; ++db)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[db][i] = 0.0f;

  const uint32_t ks = (uint32_t)(a.k.row * ES), vs = (uint32_t)(a.v.row * ES);
  const char* K = static_cast<const char*>(a.k.p) + (int64_t)kvh * a.k.head * ES;
  const char* V = static_cast<const char*>(a.v.p) + (int64_t)kvh * a.v.head * ES;
  const int k_len = it.off + it.q_len;
  auto issue = [&](int key0, int buf) {
    const int64_t at = (int64_t)it.k_start + key0, left = k_len - key0;
    load_rows<T, DP, NW, KT>(rsrc_of(K + at * (int64_t)ks, (left - 1) * (int64_t)ks + D * ES), ks, D,
                             lds + 2 * buf * TB, wave, lane);
    load_rows<T, DP, NW, KT>(rsrc_of(V + at * (int64_t)vs, (left - 1) * (int64_t)vs + D * ES), vs, D,
                             lds + (2 * buf + 1) * TB, wave, lane);
  };
  const int steps = (it.k_end + KT - 1) / KT;
  if (steps > 0) issue(0, 0);
  for (int st = 0; st < steps; ++st) {
    const int key0 = st * KT;
    __syncthreads();
    if (st + 1 < steps) issue(key0 + KT, (st + 1) & 1);
    if (key0 >= any) continue;
    const char* kt = lds + 2 * (st & 1) * TB;
    const char* vt = kt + TB;
#pragma unroll
    for (int kb = 0; kb < KT / 32; ++kb) {
      floatx16 s, dp;
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i] = dp[i] = 0.0f;
#pragma unroll
      for (int q = 0; q < TL::STEPS; ++q) {
        s = Elt<T>::mma(TL::row(kt, 32 * kb + (lane & 31), 2 * q + h), qf[q], s);
        dp = Elt<T>::mma(TL::row(vt, 32 * kb + (lane & 31), 2 * q + h), df[q], dp);
      }
      if (key0 + 32 * kb + 32 > all) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (key0 + 32 * kb + 8 * (i >> 2) + 4 * h + (i & 3) >= lim) s[i] = -INFINITY;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i] = __builtin_amdgcn_exp2f(fmaf(s[i], sl2, -lse2)) * (dp[i] - delta);
      // a softmax over one key has no gradient: exactly 0, whatever rounding
      // the stored O put between dP and delta
      if (key0 + 32 * kb == 0 && all <= 1 && lim == 1) {
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = 0.0f;
      }
#pragma unroll
      for (int j = 0; j < 16 / EPL; ++j) {
        const frag p = pack<T>(s, j * EPL);
#pragma unroll
        for (int db = 0; db < DP / 32; ++db)
          acc[db] = Elt<T>::mma(TL::col(kt, 32 * kb + 2 * EPL * j, db, lane), p, acc[db]);
      }
    }
  }
  if (!live) return;
  T* out = static_cast<T*>(a.dq.p) + row * a.dq.row + head * a.dq.head;
#pragma unroll
  for (int db = 0; db < DP / 32; ++db)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int d = 32 * db + 8 * j + 4 * h;
      if (d < D)
        store4<T>(out + d, acc[db][4 * j] * a.scale, acc[db][4 * j + 1] * a.scale, acc[db][4 * j + 2] * a.scale,
                  acc[db][4 * j + 3] * a.scale);
    }
}

// dK and dV of one tile of 128 keys, 32 a wave, K and V of the wave's keys in
// registers: over the flat rows that see any of them (all heads of the group),
// S = Q K^T and dP = dO V^T (a lane holds one key), then dV^T += dO^T P and
// dK^T += Q^T dS with dO and Q read transposed.
template <typename T, int DP>
__global__ __launch_bounds__(256, 1) void dkv_kernel(Args a) {
  typedef Tile<T, DP> TL;
  typedef typename Elt<T>::frag frag;
  constexpr int NW = 4, ES = sizeof(T), RT = sizeof(T) == 2 ? kBwdRows : kBwdRows / 2, TB = RT * TL::RB;
  constexpr int EPL = Elt<T>::EPL;
  __shared__ __attribute__((aligned(1024))) char lds[4 * TB];
  __shared__ __attribute__((aligned(16))) float stat[2][2][RT];  // [buffer][lse * log2(e), delta][row]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, h = lane >> 5;
  const int kvh = blockIdx.x % a.kv_heads;
  const KeyItem it = static_cast<const KeyItem*>(a.items)[blockIdx.x / a.kv_heads];
  const int G = a.G, D = a.D, n_rows = it.q_len * G;
  const float sl2 = a.scale * kLog2e;

  const int key = it.key0 + wave * 32 + (lane & 31);
  const bool live = key < it.k_len;
  const int64_t krow = (int64_t)it.k_start + key;
  frag kf[TL::STEPS], vf[TL::STEPS];
  row_frags<T, DP>(static_cast<const char*>(a.k.p) + (krow * a.k.row + (int64_t)kvh * a.k.head) * ES, live, D, h, kf);
  row_frags<T, DP>(static_cast<const char*>(a.v.p) + (krow * a.v.row + (int64_t)kvh * a.v.head) * ES, live, D, h, vf);
  // the first flat row that sees this key, the wave's first key, its last
  const int from = live ? max(0, key - it.off) * G : 0x7FFFFFFF;
  const int wkey = it.key0 + wave * 32;
  const int any = __builtin_amdgcn_readfirstlane(wkey < it.k_len ? max(0, wkey - it.off) * G : 0x7FFFFFFF);
  const int all = __builtin_amdgcn_readfirstlane(max(0, wkey + 31 - it.off) * G);
  // the end of the flat rows that see key 0 alone (none before its first row)
  const int one = wkey == 0 && it.off <= 0 ? (1 - it.off) * G : 0;
  const int one_row = key == 0 ? one : 0;

  floatx16 dk[DP / 32], dv[DP / 32];
#pragma unroll
  for (int db = 0; db < DP / 32; ++db)
#pragma unroll
    for (int i = 0; i < 16; ++i) dk[db][i] = dv[db][i] = 0.0f;

  // rows of a step: Q and dO straight to LDS, their lse and delta through registers
  auto issue = [&](int r0, int buf) {
    const RowMap rm(r0, G);
    const int64_t row = it.q_start + (int64_t)rm.t0;
    const __amdgpu_buffer_rsrc_t rq = rsrc_of(
        static_cast<const char*>(a.q.p) + (row * a.q.row + (int64_t)kvh * G * a.q.head) * ES, kMaxBytes);
    const __amdgpu_buffer_rsrc_t rd = rsrc_of(
        static_cast<const char*>(a.dO.p) + (row * a.dO.row + (int64_t)kvh * G * a.dO.head) * ES, kMaxBytes);
    constexpr int PER_WAVE = RT / (NW * TL::RPI);
    static_assert(RT % (NW * TL::RPI) == 0, "rows per wave");
#pragma unroll
    for (int j = 0; j < PER_WAVE; ++j) {
      const int blk = wave * PER_WAVE + j;
      const int i = blk * TL::RPI + lane / TL::SLOTS;
      const int c = (lane % TL::SLOTS) ^ TL::f(i);
      int t, g;
      rm.of(i, &t, &g);
      const bool ok = r0 + i < n_rows && c * 16 < D * ES;
      const uint32_t oq = (uint32_t)(t * (int)a.q.row + g * (int)a.q.head) * ES + (uint32_t)c * 16u;
      const uint32_t od = (uint32_t)(t * (int)a.dO.row + g * (int)a.dO.head) * ES + (uint32_t)c * 16u;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rq, (lds_ptr_t)(lds + 2 * buf * TB + blk * 1024), 16, ok ? oq : kOob, 0,
                                               0, 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rd, (lds_ptr_t)(lds + (2 * buf + 1) * TB + blk * 1024), 16,
                                               ok ? od : kOob, 0, 0, 0);
    }
  };
  auto stats = [&](int r0, float* x) {  // thread i of the first 2 RT: lse or delta of row r0 + i % RT
    const int i = threadIdx.x % RT;
    *x = threadIdx.x < RT ? INFINITY : 0.0f;
    if ((int)threadIdx.x < 2 * RT && r0 + i < n_rows) {
      const RowMap rm(r0, G);
      int t, g;
      rm.of(i, &t, &g);
      const int64_t at = (it.q_start + (int64_t)rm.t0 + t) * a.heads + kvh * G + g;
      if ((int)threadIdx.x >= RT) *x = a.delta[at];
      else *x = a.lse[at] * kLog2e;
    }
  };

  const int steps = it.r_begin < n_rows ? (n_rows - it.r_begin + RT - 1) / RT : 0;
  float x = 0.0f;
  if (steps > 0) {
    issue(it.r_begin, 0);
    stats(it.r_begin, &x);
  }
  for (int st = 0; st < steps; ++st) {
    const int r0 = it.r_begin + st * RT;
    if ((int)threadIdx.x < 2 * RT) stat[st & 1][threadIdx.x / RT][threadIdx.x % RT] = x;
    __syncthreads();
    if (st + 1 < steps) {
      issue(r0 + RT, (st + 1) & 1);
      stats(r0 + RT, &x);
    }
    const char* qt = lds + 2 * (st & 1) * TB;
    const char* ot = qt + TB;
#pragma unroll
    for (int rb = 0; rb < RT / 32; ++rb) {
      if (r0 + 32 * rb + 32 <= any) continue;  // no row of these sees a key of this wave
      floatx16 s, dp;
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i] = dp[i] = 0.0f;
#pragma unroll
      for (int q = 0; q < TL::STEPS; ++q) {
        s = Elt<T>::mma(TL::row(qt, 32 * rb + (lane & 31), 2 * q + h), kf[q], s);
        dp = Elt<T>::mma(TL::row(ot, 32 * rb + (lane & 31), 2 * q + h), vf[q], dp);
      }
      if (r0 + 32 * rb < all || wkey + 32 > it.k_len) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (r0 + 32 * rb + 8 * (i >> 2) + 4 * h + (i & 3) < from) s[i] = -INFINITY;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4_t ls = *reinterpret_cast<const float4_t*>(&stat[st & 1][0][32 * rb + 8 * j + 4 * h]);
        const float4_t de = *reinterpret_cast<const float4_t*>(&stat[st & 1][1][32 * rb + 8 * j + 4 * h]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // a masked entry is 0 whatever lse is (-inf on a row that sees nothing)
          const float e = fmaf(s[4 * j + i], sl2, -ls[i]);
          s[4 * j + i] = s[4 * j + i] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(e);
          dp[4 * j + i] = s[4 * j + i] * (dp[4 * j + i] - de[i]);
        }
      }
      // rows that see this one key have no gradient through the softmax
      if (r0 + 32 * rb < one) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (r0 + 32 * rb + 8 * (i >> 2) + 4 * h + (i & 3) < one_row) dp[i] = 0.0f;
      }
#pragma unroll
      for (int j = 0; j < 16 / EPL; ++j) {
        const frag p = pack<T>(s, j * EPL), d = pack<T>(dp, j * EPL);
#pragma unroll
        for (int db = 0; db < DP / 32; ++db) {
          dv[db] = Elt<T>::mma(TL::col(ot, 32 * rb + 2 * EPL * j, db, lane), p, dv[db]);
          dk[db] = Elt<T>::mma(TL::col(qt, 32 * rb + 2 * EPL * j, db, lane), d, dk[db]);
        }
      }
    }
  }
  if (!live) return;
  T* ok = static_cast<T*>(a.dk.p) + krow * a.dk.row + (int64_t)kvh * a.dk.head;
  T* ov = static_cast<T*>(a.dv.p) + krow * a.dv.row + (int64_t)kvh * a.dv.head;
#pragma unroll
  for (int db = 0; db < DP / 32; ++db)
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

}  // namespace

hipError_t launch_dq(const Args& a, hipStream_t st) {
  const dim3 grid((unsigned)(a.n_items * a.kv_heads));
  note_launch("attn_dq", st);
  if (a.dtype == 1 && a.D <= 64) dq_kernel<bf16, 64><<<grid, 256, 0, st>>>(a);
  else if (a.dtype == 1) dq_kernel<bf16, 128><<<grid, 256, 0, st>>>(a);
  else if (a.D <= 64) dq_kernel<float, 64><<<grid, 256, 0, st>>>(a);
  else dq_kernel<float, 128><<<grid, 256, 0, st>>>(a);
  return hipGetLastError();
}

hipError_t launch_dkv(const Args& a, hipStream_t st) {
  const dim3 grid((unsigned)(a.n_items * a.kv_heads));
  note_launch("attn_dkv", st);
  if (a.dtype == 1 && a.D <= 64) dkv_kernel<bf16, 64><<<grid, 256, 0, st>>>(a);
  else if (a.dtype == 1) dkv_kernel<bf16, 128><<<grid, 256, 0, st>>>(a);
  else if (a.D <= 64) dkv_kernel<float, 64><<<grid, 256, 0, st>>>(a);
  else dkv_kernel<float, 128><<<grid, 256, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace attn
}  // namespace ipttt
