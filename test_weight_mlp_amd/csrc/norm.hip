// Layer norm and RMS norm of rows, and their gradients.
//
// A row is held in the registers of one wave (narrow rows of 8 to 32 lanes, wide ones of
// several waves), in 16-byte pieces a lane, so that it is read once: the mean, the squares
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

// Sum over groups of L lanes (8 to 64), in all of them: neighbours, pairs, half rows and
// rows of 16 lanes, then across the rows.
template <int L>
__device__ __forceinline__ float lane_sum(float x) {
  x = dpp_add<0xB1>(x);   // quad_perm 1 0 3 2
  x = dpp_add<0x4E>(x);   // quad_perm 2 3 0 1
  x = dpp_add<0x141>(x);  // row_half_mirror
  if constexpr (L >= 16) x = dpp_add<0x140>(x);  // row_mirror
  if constexpr (L >= 32) x += __shfl_xor(x, 16, 64);
  if constexpr (L >= 64) x += __shfl_xor(x, 32, 64);
  return x;
}

// N sums over a row's L lanes: within the wave, or (L > 64) of neighbouring waves through
// LDS, red[slot][wave].  slot alternates between consecutive calls, so that one
// barrier a call is enough: a wave that writes a slot again has passed the barrier of
// the call between, which every wave meets after its reads of that slot.
template <int L, int N>
__device__ __forceinline__ void row_sum(float (&x)[N], float (*red)[8][N], int slot, int wave) {
  constexpr int NW = L / 64;
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = lane_sum<L < 64 ? L : 64>(x[i]);
  if constexpr (NW > 1) {
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) red[slot][wave][i] = x[i];
    }
    __syncthreads();
    const int first = wave / NW * NW;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      x[i] = red[slot][first][i];
#pragma unroll
      for (int q = 1; q < NW; ++q) x[i] += red[slot][first + q][i];
    }
  }
}

template <typename T>
struct Piece {  // 16 bytes
  static constexpr int V = 16 / sizeof(T);
  typedef T vec __attribute__((ext_vector_type(V)));
};

// L lanes a row, 256 / L rows a workgroup at a time.
template <typename T, int L, int IT>
__global__ __launch_bounds__(256) void norm_kernel(NormArgs a) {
  constexpr int V = Piece<T>::V, ROWS = 256 / L;
  typedef typename Piece<T>::vec vec;
  __shared__ float red[2][8][1];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x % L;
  for (int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / L; row < a.rows; row += (int64_t)gridDim.x * ROWS) {
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
      row_sum<L>(mu, red, 0, wave);
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
    row_sum<L>(sq, red, 1, wave);
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
    if constexpr (L > 64) __syncthreads();  // before the next row writes red
  }
}

// L lanes a row, 512 / L rows a workgroup at a time.  The weight gradients of a lane's
// columns stay in registers until its last row, and each workgroup writes one partial
// (a lone one the result).  Bound by the memory: 16384 x 2560 in bf16 with dres 83 us
// for 336 MB (4.0 TB/s), 32768 x 1024 58 us (4.6 TB/s).  Loading the next row's pieces
// before the current row's sums gained nothing (84 and 59 us): with 16 waves resident
// the others' loads fill the wait.
template <typename T, int L, int IT>
__global__ __launch_bounds__(512) void norm_bwd_kernel(NormArgs a) {
  constexpr int V = Piece<T>::V, ROWS = 512 / L;
  typedef typename Piece<T>::vec vec;
  __shared__ float red[2][8][3];
  __shared__ float red1[2][8][1];
  __shared__ float sum[L < 512 ? ROWS : 1][L < 512 ? IT * L * V : 1];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x % L, group = threadIdx.x / L;
  const bool grads = a.dw != nullptr || a.db != nullptr;
  float dw[IT][V], db[IT][V];
#pragma unroll
  for (int i = 0; i < IT; ++i)
#pragma unroll
    for (int e = 0; e < V; ++e) dw[i][e] = db[i][e] = 0.0f;
  auto load = [&](const Rows& t, int64_t row, vec (&to)[IT]) {
    const T* p = static_cast<const T*>(t.p) + row * t.ld;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int c = (i * L + lane) * V;
      to[i] = c < a.dim && row < a.rows ? *reinterpret_cast<const vec*>(p + c) : vec{};
    }
  };
  const int64_t step = (int64_t)gridDim.x * ROWS;
  vec x[IT], dy[IT];
  load(a.x, (int64_t)blockIdx.x * ROWS + group, x);
  load(a.dy, (int64_t)blockIdx.x * ROWS + group, dy);
  int slot = 0;
  // all groups make the same rounds (they meet in row_sum); rows past the end are zeros
  for (int64_t first = (int64_t)blockIdx.x * ROWS; first < a.rows; first += step, slot ^= 1) {
    const int64_t row = first + group;
    vec more[IT];
    if (a.dres.p != nullptr) load(a.dres, row, more);
    float mu[1] = {0.0f};
    if (a.center) {
#pragma unroll
      for (int i = 0; i < IT; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) mu[0] += (float)x[i][e];
      row_sum<L>(mu, red1, slot, wave);
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
    row_sum<L>(s, red, slot, wave);
    const float n = (float)a.dim, r = rsqrtf(s[0] / n + a.eps);
    const float mean_u = a.center ? s[1] / n : 0.0f, along = s[2] / n * r * r;
    T* op = static_cast<T*>(a.dx.p) + row * a.dx.ld;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int c = (i * L + lane) * V;
      if (c >= a.dim || row >= a.rows) continue;
      vec w, o;
      if (a.w != nullptr) w = *reinterpret_cast<const vec*>(static_cast<const T*>(a.w) + c);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float g = (float)dy[i][e], d = (float)x[i][e] - mu[0];
        const float u = a.w != nullptr ? g * (float)w[e] : g;
        float v = r * (u - mean_u - d * along);
        if (a.dres.p != nullptr) v += (float)more[i][e];
        o[e] = (T)v;
        dw[i][e] = fmaf(g, d * r, dw[i][e]);
        db[i][e] += g;
      }
      *reinterpret_cast<vec*>(op + c) = o;
    }
    load(a.x, row + step, x);
    load(a.dy, row + step, dy);
  }
  if (!grads) return;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float* to = which == 0 ? a.dw : a.db;
    if (gridDim.x > 1) to = a.part + ((int64_t)blockIdx.x * 2 + which) * a.dim;
    if constexpr (L < 512) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < IT; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) sum[group][(i * L + lane) * V + e] = which == 0 ? dw[i][e] : db[i][e];
      __syncthreads();
      for (int c = threadIdx.x; c < a.dim && to != nullptr; c += 512) {
        float t = sum[0][c];
#pragma unroll
        for (int q = 1; q < ROWS; ++q) t += sum[q][c];
        to[c] = t;
      }
    } else {
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        const int c = (i * L + lane) * V;
        if (c >= a.dim || to == nullptr) continue;
#pragma unroll
        for (int e = 0; e < V; ++e) to[c + e] = which == 0 ? dw[i][e] : db[i][e];
      }
    }
  }
}

// dw and db: the partials of 16 columns a workgroup, 32 threads a column, in a fixed
// order.
__global__ __launch_bounds__(512) void norm_sum_kernel(const float* part, int parts, int dim, float* dw, float* db) {
  __shared__ float red[32][17];
  const int c = blockIdx.x * 16 + (threadIdx.x & 15), g = threadIdx.x >> 4;
  float x = 0.0f;
  // (8 loads at a time: 256 partials of 2048 sums 2.8 us, one load at a time 4.5)
  for (int p = g; p < parts && c < 2 * dim; p += 32 * 8) {
    float v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = p + 32 * u < parts ? part[(int64_t)(p + 32 * u) * 2 * dim + c] : 0.0f;
#pragma unroll
    for (int u = 0; u < 8; ++u) x += v[u];
  }
  red[g][threadIdx.x & 15] = x;
  __syncthreads();
  if (threadIdx.x >= 16 || c >= 2 * dim) return;
#pragma unroll
  for (int i = 1; i < 32; ++i) x += red[i][threadIdx.x];
  float* out = c < dim ? dw : db;
  if (out != nullptr) out[c < dim ? c : c - dim] = x;
}

// Rows of up to this many elements a lane go to one wave.
constexpr int kWaveElems = 40;

// Rows of up to 32 pieces share a wave: the lanes, 8, 16 or 32, that hold one (20000 x 64
// in bf16 3.4 us and its gradient 7.7; with a wave a row 6.5 and 14.6).
template <typename T, typename F>
bool with_narrow_row(int dim, F&& f) {
  const int pieces = (dim + Piece<T>::V - 1) / Piece<T>::V;
  const std::integral_constant<int, 1> one;
  if (pieces <= 8) f(std::integral_constant<int, 8>(), one);
  else if (pieces <= 16) f(std::integral_constant<int, 16>(), one);
  else if (pieces <= 32) f(std::integral_constant<int, 32>(), one);
  return pieces <= 32;
}

template <typename T, int L, typename F>
void with_pieces(int dim, F&& f) {
  constexpr int V = Piece<T>::V, most = L == 64 ? kWaveElems / V : 16384 / 256 / V;
  const int it = (dim + L * V - 1) / (L * V);
  auto pick = [&](auto n) {
    constexpr int N = decltype(n)::value;
    if constexpr (N <= most) f(std::integral_constant<int, L>(), n);
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

template <typename T, typename F>
void with_row(int dim, F&& f) {
  if (with_narrow_row<T>(dim, f)) return;
  if (dim <= 64 * kWaveElems) with_pieces<T, 64>(dim, f);
  else with_pieces<T, 256>(dim, f);
}

// The gradient's waves a row: as few as hold it in kGradPieces 16-byte pieces a lane
// (16384 x 2560 in bf16 83 us; one wave with 5 pieces, its registers spilled, 112;
// 8192 x 2560 in fp32 74 with 4 waves and 3 pieces, 87 with 2 and 5).
constexpr int kGradPieces = 3;
int pieces_a_lane(int dtype, int nw, int dim) {
  const int v = dtype == 1 ? 8 : 4;
  return (dim + nw * 64 * v - 1) / (nw * 64 * v);
}
int grad_waves(int dtype, int dim) {
  int nw = 1;
  while (nw < 8 && pieces_a_lane(dtype, nw, dim) > kGradPieces) nw *= 2;
  return nw;
}

template <typename T, int L, typename F>
void with_grad_pieces(int it, F&& f) {
  constexpr int most = L < 512 ? kGradPieces : 16384 / (512 * Piece<T>::V);
  auto pick = [&](auto n) {
    if constexpr (decltype(n)::value <= most) f(std::integral_constant<int, L>(), n);
  };
  if (it <= 1) pick(std::integral_constant<int, 1>());
  else if (it <= 2) pick(std::integral_constant<int, 2>());
  else if (it <= 3) pick(std::integral_constant<int, 3>());
  else if (it <= 4) pick(std::integral_constant<int, 4>());
  else if (it <= 6) pick(std::integral_constant<int, 6>());
  else pick(std::integral_constant<int, 8>());
}

template <typename T, typename F>
void with_grad_row(int dtype, int dim, F&& f) {
  if (with_narrow_row<T>(dim, f)) return;
  const int nw = grad_waves(dtype, dim), it = pieces_a_lane(dtype, nw, dim);
  switch (nw) {
    case 1: return with_grad_pieces<T, 64>(it, f);
    case 2: return with_grad_pieces<T, 128>(it, f);
    case 4: return with_grad_pieces<T, 256>(it, f);
    default: return with_grad_pieces<T, 512>(it, f);
  }
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, hipStream_t st) {
  note_launch("norm", st);
  auto go = [&](auto type) {
    typedef decltype(type) T;
    with_row<T>(a.dim, [&](auto lanes, auto it) {
      constexpr int L = decltype(lanes)::value, ROWS = 256 / L;
      const unsigned g = (unsigned)std::min<int64_t>((a.rows + ROWS - 1) / ROWS, 1 << 20);
      norm_kernel<T, L, decltype(it)::value><<<g, 256, 0, st>>>(a);
    });
  };
  if (a.dtype == 1) go(bf16());
  else go(float());
  return hipGetLastError();
}

// As many workgroups as are resident: two a compute unit while a row's pieces and their
// gradients fit 128 registers a lane (16 elements in bf16, 12 in fp32), above that one:
// 32768 x 1024 in bf16 58 us with 512 and 65 with 256, 16384 x 2560 89 and 83.
int norm_parts(int dtype, int64_t rows, int dim) {
  const int nw = grad_waves(dtype, dim);
  int64_t groups = 8 / nw;
  const auto narrow = [&](auto lanes, auto) { groups = 512 / decltype(lanes)::value; };
  if (dtype == 1) with_narrow_row<bf16>(dim, narrow);
  else with_narrow_row<float>(dim, narrow);
  const int64_t most = pieces_a_lane(dtype, nw, dim) <= (dtype == 1 ? 2 : 3) ? 512 : 256;
  return (int)std::min<int64_t>(most, (rows + groups - 1) / groups);
}

hipError_t launch_norm_backward(const NormArgs& a, hipStream_t st) {
  const int parts = norm_parts(a.dtype, a.rows, a.dim);
  note_launch("norm_bwd", st);
  auto go = [&](auto type) {
    typedef decltype(type) T;
    with_grad_row<T>(a.dtype, a.dim, [&](auto lanes, auto it) {
      norm_bwd_kernel<T, decltype(lanes)::value, decltype(it)::value><<<parts, 512, 0, st>>>(a);
    });
  };
  if (a.dtype == 1) go(bf16());
  else go(float());
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || parts == 1 || (a.dw == nullptr && a.db == nullptr)) return e;
  note_launch("norm_sum", st);
  norm_sum_kernel<<<(2 * a.dim + 15) / 16, 512, 0, st>>>(a.part, parts, a.dim, a.dw, a.db);
  return hipGetLastError();
}

}  // namespace ipttt
