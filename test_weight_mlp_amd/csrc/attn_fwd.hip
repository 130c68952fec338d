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

namespace ipttt {
namespace attn {
namespace {

template <typename T, int DP>
__global__ __launch_bounds__(256, 1) void fwd_kernel(Args a) {
  typedef Tile<T, DP> TL;
  typedef typename Elt<T>::frag frag;
  constexpr int NW = 4, ES = sizeof(T), TB = kKeys * TL::RB, EPL = Elt<T>::EPL;
  __shared__ __attribute__((aligned(1024))) char lds[4 * TB];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, h = lane >> 5;
  const int kvh = blockIdx.x % a.kv_heads;
  const RowItem it = static_cast<const RowItem*>(a.items)[blockIdx.x / a.kv_heads];
  const int G = a.G, D = a.D, n_rows = it.q_len * G;
  const float sl2 = a.scale * kLog2e;

  // this lane's row: query t of head kvh * G + g; it sees keys below lim
  const RowMap rm(it.r0 + wave * 32, G);
  const int r = it.r0 + wave * 32 + (lane & 31);
  int t, g;
  rm.of(lane & 31, &t, &g);
  t += rm.t0;
  const bool live = r < n_rows;
  const int lim = live ? min(it.off + t + 1, it.k_end) : 0;
  // the wave's first and last limits: keys every row sees, keys any row sees
  const int all = __builtin_amdgcn_readfirstlane(min(it.off + rm.t0 + 1, it.k_end));
  const int r_last = min(it.r0 + wave * 32 + 31, n_rows - 1);
  const int any = __builtin_amdgcn_readfirstlane(
      it.r0 + wave * 32 < n_rows ? min(it.off + r_last / G + 1, it.k_end) : 0);

  const int64_t row = it.q_start + (int64_t)t;
  const int head = kvh * G + g;
  frag qf[TL::STEPS];
  row_frags<T, DP>(static_cast<const char*>(a.q.p) + (row * a.q.row + head * a.q.head) * ES, live, D, h, qf);

  floatx16 o[DP / 32];
#pragma unroll
  for (int db = 0; db < DP / 32; ++db)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[db][i] = 0.0f;
  float m = -INFINITY, l = 0.0f;

  const uint32_t ks = (uint32_t)(a.k.row * ES), vs = (uint32_t)(a.v.row * ES);
  const char* K = static_cast<const char*>(a.k.p) + (int64_t)kvh * a.k.head * ES;
  const char* V = static_cast<const char*>(a.v.p) + (int64_t)kvh * a.v.head * ES;
  const int last_key = it.off + it.q_len;  // = k_len
  auto issue = [&](int key0, int buf) {
    const int64_t at = (int64_t)it.k_start + key0, left = last_key - key0;
    load_rows<T, DP, NW, kKeys>(rsrc_of(K + at * (int64_t)ks, (left - 1) * (int64_t)ks + D * ES), ks, D, lds + 2 * buf * TB,
                         wave, lane);
    load_rows<T, DP, NW, kKeys>(rsrc_of(V + at * (int64_t)vs, (left - 1) * (int64_t)vs + D * ES), vs, D,
                         lds + (2 * buf + 1) * TB, wave, lane);
  };
  const int steps = (it.k_end - it.k_begin + kKeys - 1) / kKeys;
  if (steps > 0) issue(it.k_begin, 0);
  for (int st = 0; st < steps; ++st) {
    const int key0 = it.k_begin + st * kKeys;
    __syncthreads();  // this step's tiles have landed; the other buffer's readers are done
    if (st + 1 < steps) issue(key0 + kKeys, (st + 1) & 1);
    if (key0 >= any) continue;  // no row of this wave sees these keys
    const char* kt = lds + 2 * (st & 1) * TB;
    const char* vt = kt + TB;
    floatx16 s[2];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
      for (int i = 0; i < 16; ++i) s[kb][i] = 0.0f;
#pragma unroll
      for (int q = 0; q < TL::STEPS; ++q)
        s[kb] = Elt<T>::mma(TL::row(kt, 32 * kb + (lane & 31), 2 * q + h), qf[q], s[kb]);
    }
    if (key0 + kKeys > all) {
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (key0 + 32 * kb + 8 * (i >> 2) + 4 * h + (i & 3) >= lim) s[kb][i] = -INFINITY;
    }
    float mx = s[0][0];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[kb][i]);
    mx = fmaxf(mx, other_half(mx)) * sl2;
    const float mn = fmaxf(m, mx);
    const float mu = mn == -INFINITY ? 0.0f : mn;  // a row that has seen nothing yet
    const float c = __builtin_amdgcn_exp2f(m - mu);
    m = mn;
    float sum = 0.0f;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[kb][i] = __builtin_amdgcn_exp2f(fmaf(s[kb][i], sl2, -mu));
        sum += s[kb][i];
      }
    l = l * c + sum;
#pragma unroll
    for (int db = 0; db < DP / 32; ++db)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[db][i] *= c;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int j = 0; j < 16 / EPL; ++j) {
        const frag p = pack<T>(s[kb], j * EPL);
#pragma unroll
        for (int db = 0; db < DP / 32; ++db)
          o[db] = Elt<T>::mma(TL::col(vt, 32 * kb + 2 * EPL * j, db, lane), p, o[db]);
      }
  }
  l += other_half(l);
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
  const float lse = l > 0.0f ? (m + __builtin_amdgcn_logf(l)) * kLn2 : -INFINITY;
  if (!live) return;
  if (it.part >= 0) {
    const int64_t slot = ((int64_t)it.part * a.kv_heads + kvh) * kRows + (r - it.r0);
    if (h == 0) a.part_lse[slot] = lse;
#pragma unroll
    for (int db = 0; db < DP / 32; ++db)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int d = 32 * db + 8 * j + 4 * h;
        if (d < D)
          store4<float>(a.part_o + slot * D + d, o[db][4 * j] * inv, o[db][4 * j + 1] * inv, o[db][4 * j + 2] * inv,
                        o[db][4 * j + 3] * inv);
      }
    return;
  }
  if (h == 0) a.lse[row * a.heads + head] = lse;
  T* out = static_cast<T*>(a.o.p) + row * a.o.row + head * a.o.head;
#pragma unroll
  for (int db = 0; db < DP / 32; ++db)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int d = 32 * db + 8 * j + 4 * h;
      if (d < D)
        store4<T>(out + d, o[db][4 * j] * inv, o[db][4 * j + 1] * inv, o[db][4 * j + 2] * inv, o[db][4 * j + 3] * inv);
    }
}

// Joins the partial results of one tile: with each part's lse, its weight is
// e^(lse_i - lse), lse = log sum e^(lse_i).  One wave a row, in slot order.
template <typename T>
__global__ __launch_bounds__(256) void join_kernel(Args a, const JoinItem* items) {
  const int kvh = blockIdx.y;
  const JoinItem it = items[blockIdx.x];
  const int G = a.G, D = a.D, lane = threadIdx.x & 63;
  const int rows = min(kRows, it.q_len * G - it.r0);
  for (int i = threadIdx.x >> 6; i < rows; i += 4) {
    const int r = it.r0 + i, t = r / G, head = kvh * G + r - t * G;
    const int64_t slot0 = ((int64_t)it.part * a.kv_heads + kvh) * kRows + i, step = (int64_t)a.kv_heads * kRows;
    float m = -INFINITY;
    for (int p = 0; p < it.n; ++p) m = fmaxf(m, a.part_lse[slot0 + p * step]);
    const float mu = m == -INFINITY ? 0.0f : m;
    float l = 0.0f, x0 = 0.0f, x1 = 0.0f;
    for (int p = 0; p < it.n; ++p) {
      const int64_t s = slot0 + p * step;
      const float w = __builtin_amdgcn_exp2f((a.part_lse[s] - mu) * kLog2e);
      l += w;
      if (w > 0.0f) {
        if (2 * lane < D) {
          x0 = fmaf(w, a.part_o[s * D + 2 * lane], x0);
          x1 = fmaf(w, a.part_o[s * D + 2 * lane + 1], x1);
        }
      }
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    const int64_t row = it.q_start + (int64_t)t;
    if (lane == 0) a.lse[row * a.heads + head] = l > 0.0f ? mu + __builtin_amdgcn_logf(l) * kLn2 : -INFINITY;
    T* out = static_cast<T*>(a.o.p) + row * a.o.row + head * a.o.head;
    if (2 * lane < D) {
      out[2 * lane] = (T)(x0 * inv);
      out[2 * lane + 1] = (T)(x1 * inv);
    }
  }
}

}  // namespace

hipError_t launch_forward(const Args& a, hipStream_t st) {
  const dim3 grid((unsigned)(a.n_items * a.kv_heads));
  note_launch("attn_fwd", st);
  if (a.dtype == 1 && a.D <= 64) fwd_kernel<bf16, 64><<<grid, 256, 0, st>>>(a);
  else if (a.dtype == 1) fwd_kernel<bf16, 128><<<grid, 256, 0, st>>>(a);
  else if (a.D <= 64) fwd_kernel<float, 64><<<grid, 256, 0, st>>>(a);
  else fwd_kernel<float, 128><<<grid, 256, 0, st>>>(a);
  return hipGetLastError();
}

hipError_t launch_join(const Args& a, const void* items, int n, hipStream_t st) {
  const dim3 grid((unsigned)n, (unsigned)a.kv_heads);
  note_launch("attn_join", st);
  if (a.dtype == 1) join_kernel<bf16><<<grid, 256, 0, st>>>(a, static_cast<const JoinItem*>(items));
  else join_kernel<float><<<grid, 256, 0, st>>>(a, static_cast<const JoinItem*>(items));
  return hipGetLastError();
}

}  // namespace attn
}  // namespace ipttt
