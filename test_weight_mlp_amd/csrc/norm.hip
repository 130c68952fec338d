// Layer norm and RMS norm of rows, and their gradients.
//
// A row is held in the registers of one wave (or, wider rows, of a workgroup's
// four), in 16-byte pieces a lane, so that it is read once: the mean, the squares
// about it and the output come from the same registers.  All arithmetic is
// fp32; the outputs are rounded once.
#include "block.h"
#include "common.h"
#include "launch.h"

#include <algorithm>
#include <type_traits>

namespace ipttt {
namespace {

template <int CTRL>
__device__ __forceinline__ float dpp_add(float x) {
  return x + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xF, 0xF, true));
}

// Sum over the wave, in all lanes: neighbours, pairs, half rows and rows of 16
// lanes, then across the rows.
__device__ __forceinline__ float wave_sum(float x) {
  x = dpp_add<0xB1>(x);   // quad_perm 1 0 3 2
  x = dpp_add<0x4E>(x);   // quad_perm 2 3 0 1
  x = dpp_add<0x141>(x);  // row_half_mirror
  x = dpp_add<0x140>(x);  // row_mirror
  x += __shfl_xor(x, 16, 64);
  x += __shfl_xor(x, 32, 64);
  return x;
}

// N sums over a row's lanes: the wave's, or (NW = 4) the workgroup's through LDS.
// slot alternates between consecutive calls, so that one barrier a call is
// enough: a wave that writes a slot again has passed the barrier of the call
// between, which every wave meets after its reads of that slot.
template <int NW, int N>
__device__ __forceinline__ void row_sum(float (&x)[N], float (*red)[4][N], int slot, int wave) {
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = wave_sum(x[i]);
  if constexpr (NW > 1) {
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) red[slot][wave][i] = x[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = red[slot][0][i] + red[slot][1][i] + red[slot][2][i] + red[slot][3][i];
  }
}

template <typename T>
struct Piece {  // 16 bytes
  static constexpr int V = 16 / sizeof(T);
  typedef T vec __attribute__((ext_vector_type(V)));
};

template <typename T, int NW, int IT>
__global__ __launch_bounds__(256) void norm_kernel(NormArgs a) {
  constexpr int V = Piece<T>::V, L = NW * 64;
  typedef typename Piece<T>::vec vec;
  __shared__ float red[2][4][1];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x % L;
  for (int64_t row = (int64_t)blockIdx.x * (4 / NW) + wave / NW; row < a.rows; row += (int64_t)gridDim.x * (4 / NW)) {
    const T* x = static_cast<const T*>(a.x.p) + row * a.x.ld;
    vec raw[IT];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int c = (i * L + lane) * V;
      raw[i] = c < a.dim ? *reinterpret_cast<const vec*>(x + c) : vec{};
    }
    float mu[1] = {0.0f}, sq[1] = {0.0f};
    if (a.center) {
#pragma unroll
      for (int i = 0; i < IT; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) mu[0] += (float)raw[i][e];
      row_sum<NW>(mu, red, 0, wave);
      mu[0] /= (float)a.dim;
    }
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const bool on = (i * L + lane) * V < a.dim;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float d = on ? (float)raw[i][e] - mu[0] : 0.0f;
        sq[0] = fmaf(d, d, sq[0]);
      }
    }
    row_sum<NW>(sq, red, 1, wave);
    const float r = rsqrtf(sq[0] / (float)a.dim + a.eps);
    T* y = static_cast<T*>(a.y.p) + row * a.y.ld;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int c = (i * L + lane) * V;
      if (c >= a.dim) continue;
      vec w, b, o;
      if (a.w != nullptr) w = *reinterpret_cast<const vec*>(static_cast<const T*>(a.w) + c);
      if (a.b != nullptr) b = *reinterpret_cast<const vec*>(static_cast<const T*>(a.b) + c);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float v = ((float)raw[i][e] - mu[0]) * r;
        if (a.w != nullptr) v *= (float)w[e];
        if (a.b != nullptr) v += (float)b[e];
        o[e] = (T)v;
      }
      *reinterpret_cast<vec*>(y + c) = o;
    }
    if constexpr (NW > 1) __syncthreads();  // before the next row writes red
  }
}

// Rows of a grid's stride a wave (or workgroup); the weight gradients of a
// lane's columns stay in registers until its last row, and each workgroup writes
// one partial.
template <typename T, int NW, int IT>
__global__ __launch_bounds__(256, 1) void norm_bwd_kernel(NormArgs a) {
  constexpr int V = Piece<T>::V, L = NW * 64;
  typedef typename Piece<T>::vec vec;
  __shared__ float red[2][4][3];
  __shared__ float red1[2][4][1];
  __shared__ float sum[NW == 1 ? 4 : 1][NW == 1 ? IT * L * V : 1];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x % L;
  const bool grads = a.dw != nullptr || a.db != nullptr;
  float dw[IT][V], db[IT][V];
#pragma unroll
  for (int i = 0; i < IT; ++i)
#pragma unroll
    for (int e = 0; e < V; ++e) dw[i][e] = db[i][e] = 0.0f;
  int slot = 0;
  for (int64_t row = (int64_t)blockIdx.x * (4 / NW) + wave / NW; row < a.rows;
       row += (int64_t)gridDim.x * (4 / NW), slot ^= 1) {
    const T* xp = static_cast<const T*>(a.x.p) + row * a.x.ld;
    const T* yp = static_cast<const T*>(a.dy.p) + row * a.dy.ld;
    vec x[IT], dy[IT];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int c = (i * L + lane) * V;
      x[i] = c < a.dim ? *reinterpret_cast<const vec*>(xp + c) : vec{};
      dy[i] = c < a.dim ? *reinterpret_cast<const vec*>(yp + c) : vec{};
    }
    float mu[1] = {0.0f};
    if (a.center) {
#pragma unroll
      for (int i = 0; i < IT; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) mu[0] += (float)x[i][e];
      row_sum<NW>(mu, red1, slot, wave);
      mu[0] /= (float)a.dim;
    }
    float s[3] = {0.0f, 0.0f, 0.0f};  // squares, u, u (x - mu)
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int c = (i * L + lane) * V;
      const bool on = c < a.dim;
      vec w;
      if (a.w != nullptr) w = on ? *reinterpret_cast<const vec*>(static_cast<const T*>(a.w) + c) : vec{};
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float d = on ? (float)x[i][e] - mu[0] : 0.0f;
        const float u = a.w != nullptr ? (float)dy[i][e] * (float)w[e] : (float)dy[i][e];
        s[0] = fmaf(d, d, s[0]);
        s[1] += u;
        s[2] = fmaf(u, d, s[2]);
      }
    }
    row_sum<NW>(s, red, slot, wave);
    const float n = (float)a.dim, r = rsqrtf(s[0] / n + a.eps);
    const float mean_u = a.center ? s[1] / n : 0.0f, along = s[2] / n * r * r;
    const T* rp = a.dres.p != nullptr ? static_cast<const T*>(a.dres.p) + row * a.dres.ld : nullptr;
    T* op = static_cast<T*>(a.dx.p) + row * a.dx.ld;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int c = (i * L + lane) * V;
      if (c >= a.dim) continue;
      vec w, more, o;
      if (a.w != nullptr) w = *reinterpret_cast<const vec*>(static_cast<const T*>(a.w) + c);
      if (rp != nullptr) more = *reinterpret_cast<const vec*>(rp + c);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float g = (float)dy[i][e], d = (float)x[i][e] - mu[0];
        const float u = a.w != nullptr ? g * (float)w[e] : g;
        float v = r * (u - mean_u - d * along);
        if (rp != nullptr) v += (float)more[e];
        o[e] = (T)v;
        dw[i][e] = fmaf(g, d * r, dw[i][e]);
        db[i][e] += g;
      }
      *reinterpret_cast<vec*>(op + c) = o;
    }
  }
  if (!grads) return;
  float* part = a.part + (int64_t)blockIdx.x * 2 * a.dim;
  if constexpr (NW == 1) {
#pragma unroll
    for (int which = 0; which < 2; ++which) {
#pragma unroll
      for (int i = 0; i < IT; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) sum[wave][(i * L + lane) * V + e] = which == 0 ? dw[i][e] : db[i][e];
      __syncthreads();
      for (int c = threadIdx.x; c < a.dim; c += 256) part[which * a.dim + c] = sum[0][c] + sum[1][c] + sum[2][c] + sum[3][c];
      __syncthreads();
    }
  } else {
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int c = (i * L + lane) * V;
      if (c >= a.dim) continue;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        part[c + e] = dw[i][e];
        part[a.dim + c + e] = db[i][e];
      }
    }
  }
}

// dw and db: the partials of 32 columns a workgroup, eight threads a column, in a
// fixed order.
__global__ __launch_bounds__(256) void norm_sum_kernel(const float* part, int parts, int dim, float* dw, float* db) {
  __shared__ float red[8][32];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), g = threadIdx.x >> 5;
  float x = 0.0f;
  if (c < 2 * dim)
    for (int p = g; p < parts; p += 8) x += part[(int64_t)p * 2 * dim + c];
  red[g][threadIdx.x & 31] = x;
  __syncthreads();
  if (g != 0 || c >= 2 * dim) return;
#pragma unroll
  for (int i = 1; i < 8; ++i) x += red[i][threadIdx.x & 31];
  float* out = c < dim ? dw : db;
  if (out != nullptr) out[c < dim ? c : c - dim] = x;
}

// Rows of up to this many elements a lane go to one wave.
constexpr int kWaveElems = 40;

template <typename T, int NW, typename F>
void with_pieces(int it, F&& f) {
  constexpr int most = NW == 1 ? kWaveElems / Piece<T>::V : 16384 / 256 / Piece<T>::V;
  auto pick = [&](auto n) {
    constexpr int N = decltype(n)::value;
    if constexpr (N <= most) f(std::integral_constant<int, NW>(), n);
  };
  if (it <= 1) pick(std::integral_constant<int, 1>());
  else if (it <= 2) pick(std::integral_constant<int, 2>());
  else if (it <= 3) pick(std::integral_constant<int, 3>());
  else if (it <= 4) pick(std::integral_constant<int, 4>());
  else if (it <= 5) pick(std::integral_constant<int, 5>());
  else if (it <= 6) pick(std::integral_constant<int, 6>());
  else if (it <= 8) pick(std::integral_constant<int, 8>());
  else if (it <= 10) pick(std::integral_constant<int, 10>());
  else pick(std::integral_constant<int, 16>());
}

template <typename T>
bool one_wave(int dim) { return dim <= 64 * kWaveElems; }

template <typename T, typename F>
void with_row(int dim, bool wave, F&& f) {
  const int V = Piece<T>::V, L = wave ? 64 : 256, it = (dim + L * V - 1) / (L * V);
  if (wave) with_pieces<T, 1>(it, f);
  else with_pieces<T, 4>(it, f);
}

constexpr int kNormParts = 512;

}  // namespace

hipError_t launch_norm(const NormArgs& a, hipStream_t st) {
  note_launch("norm", st);
  auto go = [&](auto type) {
    typedef decltype(type) T;
    with_row<T>(a.dim, one_wave<T>(a.dim), [&](auto nw, auto it) {
      constexpr int NW = decltype(nw)::value;
      const unsigned g = (unsigned)std::min<int64_t>((a.rows + 4 / NW - 1) / (4 / NW), 1 << 20);
      norm_kernel<T, NW, decltype(it)::value><<<g, 256, 0, st>>>(a);
    });
  };
  if (a.dtype == 1) go(bf16());
  else go(float());
  return hipGetLastError();
}

int norm_parts(int dtype, int64_t rows, int dim) {
  const bool wave = dtype == 1 ? one_wave<bf16>(dim) : one_wave<float>(dim);
  return (int)std::min<int64_t>(kNormParts, wave ? (rows + 3) / 4 : rows);
}

hipError_t launch_norm_backward(const NormArgs& a, hipStream_t st) {
  const int parts = norm_parts(a.dtype, a.rows, a.dim);
  note_launch("norm_bwd", st);
  auto go = [&](auto type) {
    typedef decltype(type) T;
    with_row<T>(a.dim, one_wave<T>(a.dim), [&](auto nw, auto it) {
      norm_bwd_kernel<T, decltype(nw)::value, decltype(it)::value><<<parts, 256, 0, st>>>(a);
    });
  };
  if (a.dtype == 1) go(bf16());
  else go(float());
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || (a.dw == nullptr && a.db == nullptr)) return e;
  note_launch("norm_sum", st);
  norm_sum_kernel<<<(2 * a.dim + 31) / 32, 256, 0, st>>>(a.part, parts, a.dim, a.dw, a.db);
  return hipGetLastError();
}

}  // namespace ipttt
