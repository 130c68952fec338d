// RMS norm of every query and key head fused with the position rotation, and
// its backward.
//
// A group of LG lanes holds one head of one token: lane i the elements VEC i ..
// of the first half and the same of the second, so that a rotation pair
// (d, d + D/2) sits in one lane and the norm's sum crosses log2(LG) lanes.  All
// arithmetic is fp32; the outputs are rounded once.
#include "attn.h"
#include "common.h"
#include "launch.h"

#include <algorithm>
#include <type_traits>

namespace ipttt {
namespace {

using attn::View;

template <typename T, int VEC> struct VecOf {
  typedef T type __attribute__((ext_vector_type(VEC)));
};

template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T* p, float (&x)[VEC]) {
  const auto v = *reinterpret_cast<const typename VecOf<T, VEC>::type*>(p);
#pragma unroll
  for (int i = 0; i < VEC; ++i) x[i] = (float)v[i];
}
template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T* p, const float (&x)[VEC]) {
  typename VecOf<T, VEC>::type v;
#pragma unroll
  for (int i = 0; i < VEC; ++i) v[i] = (T)x[i];
  *reinterpret_cast<typename VecOf<T, VEC>::type*>(p) = v;
}

template <int CTRL>
__device__ __forceinline__ float dpp_add(float x) {
  return x + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xF, 0xF, true));
}

// Sum over each group of LG lanes, in all of them: neighbours, then pairs, then
// (once quads are equal) the mirrored half and whole row of 16.
template <int LG>
__device__ __forceinline__ float group_sum(float x) {
  if constexpr (LG > 1) x = dpp_add<0xB1>(x);   // quad_perm 1 0 3 2
  if constexpr (LG > 2) x = dpp_add<0x4E>(x);   // quad_perm 2 3 0 1
  if constexpr (LG > 4) x = dpp_add<0x141>(x);  // row_half_mirror
  if constexpr (LG > 8) x = dpp_add<0x140>(x);  // row_mirror
  return x;
}

template <typename T>
__device__ __forceinline__ T* head_ptr(const View& v, int64_t row, int head) {
  return static_cast<T*>(v.p) + row * v.row + head * v.head;
}

// cos and sin of this lane's pairs; NaN (which the outputs then carry) where
// the position is outside the table.
template <int VEC>
__device__ __forceinline__ void load_angles(const QkArgs& a, int64_t t, int d, bool on, float (&c)[VEC],
                                            float (&s)[VEC]) {
  const int pos = a.pos[t];
  const bool ok = pos >= 0 && pos < a.table_rows;
#pragma unroll
  for (int i = 0; i < VEC; ++i) c[i] = s[i] = on ? __builtin_nanf("") : 0.0f;
  if (ok && on) {
    load_vec<float, VEC>(a.table + (int64_t)pos * a.D + d, c);
    load_vec<float, VEC>(a.table + (int64_t)pos * a.D + a.D / 2 + d, s);
  }
}

// One wave a token; blockIdx.y splits the token's heads when tokens are few.
// Bound by memory: 32768 tokens, 40 heads of width 128 in 126 us, 5.3 TB/s; one
// token's launch in 3.1 us.
template <typename T, int VEC, int LG>
__global__ __launch_bounds__(256) void qk_kernel(QkArgs a) {
  constexpr int GPW = 64 / LG;
  const int lane = threadIdx.x & 63, group = lane / LG, d = (lane % LG) * VEC, half = a.D / 2;
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= a.tokens) return;
  const bool on = d < half;
  float c[VEC], s[VEC];
  load_angles<VEC>(a, t, d, on, c, s);
  const int64_t out = a.rows != nullptr ? (int64_t)a.rows[t] : t;
  const bool keep = out >= 0 && out < a.out_rows;
  const int nq = a.heads, nk = a.kv_heads, n = nq + nk + (a.v.p != nullptr ? nk : 0);
  for (int hd = blockIdx.y * GPW + group; hd < n; hd += gridDim.y * GPW) {
    if (hd >= nq + nk) {  // V, copied to its row
      if (!on || !keep) continue;
      const T* v = head_ptr<T>(a.v, t, hd - nq - nk) + d;
      T* o = head_ptr<T>(a.v_out, out, hd - nq - nk) + d;
      typedef typename VecOf<T, VEC>::type vec;
      const vec lo = *reinterpret_cast<const vec*>(v), hi = *reinterpret_cast<const vec*>(v + half);
      *reinterpret_cast<vec*>(o) = lo;
      *reinterpret_cast<vec*>(o + half) = hi;
      continue;
    }
    const bool q = hd < nq;
    const T* x = (q ? head_ptr<T>(a.q, t, hd) : head_ptr<T>(a.k, t, hd - nq)) + d;
    const T* w = static_cast<const T*>(q ? a.w_q : a.w_k) + d;
    float lo[VEC], hi[VEC], wl[VEC], wh[VEC], sq = 0.0f;
#pragma unroll
    for (int i = 0; i < VEC; ++i) lo[i] = hi[i] = 0.0f;
    if (on) {
      load_vec<T, VEC>(x, lo);
      load_vec<T, VEC>(x + half, hi);
      load_vec<T, VEC>(w, wl);
      load_vec<T, VEC>(w + half, wh);
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) sq = fmaf(lo[i], lo[i], fmaf(hi[i], hi[i], sq));
    const float r = rsqrtf(group_sum<LG>(sq) / (float)a.D + a.eps);
    if (!on || (!q && !keep)) continue;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const float u = lo[i] * r * wl[i], v = hi[i] * r * wh[i];
      lo[i] = u * c[i] - v * s[i];
      hi[i] = v * c[i] + u * s[i];
    }
    T* o = (q ? head_ptr<T>(a.q_out, t, hd) : head_ptr<T>(a.k_out, out, hd - nq)) + d;
    store_vec<T, VEC>(o, lo);
    store_vec<T, VEC>(o + half, hi);
  }
}

// Backward: the rotation transposed, then the norm's; all query heads, then all
// key heads, so that only one of the weight gradients is in registers.  Each
// wave sums them over its tokens, each block writes one partial.  FULL: the
// group's lanes hold exactly one half (D of 64 and 128, for instance); otherwise
// the lanes past it hold nothing.  Bound by memory: 16k tokens, 40 heads of width
// 128 in 0.098 ms, 5.2 TB/s (two or four heads a group at once: 0.101, 0.118).
template <typename T, int VEC, int LG, bool FULL>
__global__ __launch_bounds__(256, 2) void qk_bwd_kernel(QkArgs a) {
  constexpr int GPW = 64 / LG;
  typedef typename VecOf<T, VEC>::type vec;
  __shared__ float red[4][2][LG * VEC];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, group = lane / LG, d = (lane % LG) * VEC;
  const int half = a.D / 2;
  const bool on = FULL || d < half;
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    const int heads = which == 0 ? a.heads : a.kv_heads;
    const View xv = which == 0 ? a.q : a.k, zv = which == 0 ? a.q_out : a.k_out, ov = which == 0 ? a.dq : a.dk;
    float dwl[VEC], dwh[VEC], wl[VEC], wh[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) dwl[i] = dwh[i] = wl[i] = wh[i] = 0.0f;
    if (on) {
      const T* w = static_cast<const T*>(which == 0 ? a.w_q : a.w_k) + d;
      load_vec<T, VEC>(w, wl);
      load_vec<T, VEC>(w + half, wh);
    }
#pragma unroll 1
    for (int64_t t = (int64_t)blockIdx.x * 4 + wave; t < a.tokens; t += (int64_t)gridDim.x * 4) {
      float c[VEC], s[VEC];
      load_angles<VEC>(a, t, d, on, c, s);
#pragma unroll 1
      for (int hd = group; hd < heads; hd += GPW) {
        vec raw[4] = {};
        if (on) {
          const T* x = head_ptr<T>(xv, t, hd) + d;
          const T* z = head_ptr<T>(zv, t, hd) + d;
          raw[0] = *reinterpret_cast<const vec*>(x);
          raw[1] = *reinterpret_cast<const vec*>(x + half);
          raw[2] = *reinterpret_cast<const vec*>(z);
          raw[3] = *reinterpret_cast<const vec*>(z + half);
        }
        float lo[VEC], hi[VEC], zl[VEC], zh[VEC], sq = 0.0f, dot = 0.0f;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          lo[i] = (float)raw[0][i];
          hi[i] = (float)raw[1][i];
          const float a0 = (float)raw[2][i], a1 = (float)raw[3][i];
          zl[i] = a0 * c[i] + a1 * s[i];
          zh[i] = a1 * c[i] - a0 * s[i];
          sq = fmaf(lo[i], lo[i], fmaf(hi[i], hi[i], sq));
          dot = fmaf(zl[i] * wl[i], lo[i], fmaf(zh[i] * wh[i], hi[i], dot));
        }
        const float r = rsqrtf(group_sum<LG>(sq) / (float)a.D + a.eps);
        const float k = group_sum<LG>(dot) * r * r / (float)a.D;
        if (!on) continue;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          dwl[i] = fmaf(zl[i], lo[i] * r, dwl[i]);
          dwh[i] = fmaf(zh[i], hi[i] * r, dwh[i]);
          lo[i] = r * (zl[i] * wl[i] - lo[i] * k);
          hi[i] = r * (zh[i] * wh[i] - hi[i] * k);
        }
        T* o = head_ptr<T>(ov, t, hd) + d;
        store_vec<T, VEC>(o, lo);
        store_vec<T, VEC>(o + half, hi);
      }
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      float x = dwl[i], y = dwh[i];
#pragma unroll
      for (int o = LG; o < 64; o <<= 1) {
        x += __shfl_xor(x, o, 64);
        y += __shfl_xor(y, o, 64);
      }
      if (group == 0) {
        red[wave][0][d + i] = x;
        red[wave][1][d + i] = y;
      }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.D; e += 256) {
      const int hf = e / half, at = e % half;
      a.part[((int64_t)blockIdx.x * 2 + which) * a.D + e] =
          red[0][hf][at] + red[1][hf][at] + red[2][hf][at] + red[3][hf][at];
    }
    __syncthreads();
  }
}

// dw[e] = sum of the blocks' partials, one block an element, in a fixed order: 4.1 us
// for 512 partials of width 128, half of it the launch.
__global__ __launch_bounds__(256) void qk_sum_kernel(const float* part, int n, int D, float* dw_q, float* dw_k) {
  __shared__ float red[256];
  const int e = blockIdx.x;
  float x = 0.0f;
  for (int p = threadIdx.x; p < n; p += 256) x += part[(int64_t)p * 2 * D + e];
  red[threadIdx.x] = x;
  __syncthreads();
#pragma unroll
  for (int o = 128; o > 0; o >>= 1) {
    if ((int)threadIdx.x < o) red[threadIdx.x] += red[threadIdx.x + o];
    __syncthreads();
  }
  if (threadIdx.x == 0) (e < D ? dw_q[e] : dw_k[e - D]) = red[0];
}

// Lanes of a head: its half in pieces of VEC elements, up to a power of two
// (D <= 128, so at most 16).
template <int LG, typename F>
void with_full(bool full, F&& f) {
  if (full) f(std::integral_constant<int, LG>(), std::true_type());
  else f(std::integral_constant<int, LG>(), std::false_type());
}
template <typename F>
void with_lanes(int half, int vec, F&& f) {
  const int lanes = (half + vec - 1) / vec;
  if (lanes <= 1) with_full<1>(half == vec, f);
  else if (lanes <= 2) with_full<2>(half == 2 * vec, f);
  else if (lanes <= 4) with_full<4>(half == 4 * vec, f);
  else if (lanes <= 8) with_full<8>(half == 8 * vec, f);
  else with_full<16>(half == 16 * vec, f);
}

// 16-byte pieces where half a head is whole 16-byte pieces (fp32 always, as D
// is a multiple of 8; bf16 with D a multiple of 16), else 8-byte ones.
template <typename F>
void with_types(const QkArgs& a, F&& f) {
  if (a.dtype != 1) f(float(), std::integral_constant<int, 4>());
  else if (a.D % 16 == 0) f(bf16(), std::integral_constant<int, 8>());
  else f(bf16(), std::integral_constant<int, 4>());
}

}  // namespace

hipError_t launch_qk(const QkArgs& a, hipStream_t st) {
  note_launch("qk", st);
  with_types(a, [&](auto type, auto vec) {
    constexpr int VEC = decltype(vec)::value;
    with_lanes(a.D / 2, VEC, [&](auto lg, auto) {
      constexpr int LG = decltype(lg)::value;
      const int heads = a.heads + a.kv_heads * (a.v.p != nullptr ? 2 : 1);
      const int64_t bx = (a.tokens + 3) / 4, trips = (heads + 64 / LG - 1) / (64 / LG);
      // the heads of a token go to more waves while the tokens leave CUs idle
      const int64_t by = std::min<int64_t>(trips, std::max<int64_t>(1, 1024 / bx));
      qk_kernel<decltype(type), VEC, LG><<<dim3((unsigned)bx, (unsigned)by), 256, 0, st>>>(a);
    });
  });
  return hipGetLastError();
}

hipError_t launch_qk_backward(const QkArgs& a, hipStream_t st) {
  const int blocks = (int)std::min<int64_t>(kQkParts, (a.tokens + 3) / 4);
  note_launch("qk_bwd", st);
  with_types(a, [&](auto type, auto vec) {
    constexpr int VEC = decltype(vec)::value;
    with_lanes(a.D / 2, VEC, [&](auto lg, auto full) {
      qk_bwd_kernel<decltype(type), VEC, decltype(lg)::value, decltype(full)::value><<<blocks, 256, 0, st>>>(a);
    });
  });
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  note_launch("qk_sum", st);
  qk_sum_kernel<<<2 * a.D, 256, 0, st>>>(a.part, blocks, a.D, a.dw_q, a.dw_k);
  return hipGetLastError();
}

}  // namespace ipttt
