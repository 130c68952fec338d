// Z = SiLU(H W_gate^T) * (H W_up^T): the intermediate activation of the gated
// MLP (lijianxiong.blog "In-Place Test-Time Training", 方法 > 原地自适应 and
// 高效的块状更新机制; phi = SiLU).
//
// One workgroup computes a tile of Z: the same H tile is multiplied by the gate and
// the up tiles (a dual GEMM, K = d_model), both products stay in fp32 registers, and
// the epilogue applies SiLU(g) * u before rounding once to the output type.  Z is
// written row-major.
#include <algorithm>
#include <type_traits>

#include "epilogue.h"
#include "launch.h"
#include "mfma_core.h"
#include "ring.h"

namespace ipttt {

// What a Z kernel keeps of G = H W_gate^T and U = H W_up^T for the backward:
// nothing, both in dtype, or both in 8 bits (bf16 data) with their scales.
enum { KEEP_NONE = 0, KEEP_ALL = 1, KEEP_8 = 2 };
struct Kept {
  void *G, *U;
  float *sG, *sU;
};

// fp32 data: 128 x 128 tiles of 4 waves.
template <typename T, int KEEP>
__global__ __launch_bounds__(kThreads) void gated_z_kernel(const T* __restrict__ H, const T* __restrict__ Wg,
                                                           const T* __restrict__ Wu, T* __restrict__ Z,
                                                           Kept kept, int64_t M, int d, int f) {
  typedef Geo<T, 128, 128> G;
  constexpr int LDC = G::BN + G::VE;
  constexpr int kStage = (G::BM + 2 * G::BN) * G::LDK;
  constexpr int kEpi = G::BM * LDC;
  __shared__ __attribute__((aligned(16))) T lds[kStage > kEpi ? kStage : kEpi];
  T* lA = lds;
  T* lB0 = lds + G::BM * G::LDK;
  T* lB1 = lB0 + G::BN * G::LDK;

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave >> 1, wn = wave & 1;
  const int tiles_m = (int)((M + G::BM - 1) / G::BM), tiles_n = (f + G::BN - 1) / G::BN;
  int tm, tn;
  grouped_tile(xcd_remap(blockIdx.x, gridDim.x), tiles_m, tiles_n, 16, tm, tn);
  const int64_t m0 = (int64_t)tm * G::BM;
  const int n0 = tn * G::BN;
  const int mrows = (int)min((int64_t)G::BM, M - m0), nrows = min(G::BN, f - n0);
  const T* A = H + m0 * d;
  const T* B0 = Wg + (int64_t)n0 * d;
  const T* B1 = Wu + (int64_t)n0 * d;

  floatx16 ag[G::MB][G::NB], au[G::MB][G::NB];
  zero_acc<G>(ag);
  zero_acc<G>(au);
  TileLoad<T, G::BM> la;
  TileLoad<T, G::BN> lb0, lb1;
  la.load(A, d, mrows, 0, d, tid);
  lb0.load(B0, d, nrows, 0, d, tid);
  lb1.load(B1, d, nrows, 0, d, tid);
  for (int k0 = 0; k0 < d; k0 += G::BK) {
    la.template store<G::LDK>(lA, tid);
    lb0.template store<G::LDK>(lB0, tid);
    lb1.template store<G::LDK>(lB1, tid);
    __syncthreads();
    if (k0 + G::BK < d) {
      la.load(A, d, mrows, k0 + G::BK, d, tid);
      lb0.load(B0, d, nrows, k0 + G::BK, d, tid);
      lb1.load(B1, d, nrows, k0 + G::BK, d, tid);
    }
    stage_mma<T, G>(lA, lB0, ag, wm, wn, lane);
    stage_mma<T, G>(lA, lB1, au, wm, wn, lane);
    __syncthreads();
  }

  T* lC = lds;
  // which = 0: Z, 1: G, 2: U
  auto stage = [&](int which) {
#pragma unroll
    for (int mb = 0; mb < G::MB; ++mb)
#pragma unroll
      for (int nb = 0; nb < G::NB; ++nb)
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int r = wm * G::WM + mb * 32 + acc_row(j, lane);
          const int c = wn * G::WN + nb * 32 + (lane & 31);
          const float g = ag[mb][nb][j], u = au[mb][nb][j];
          lC[r * LDC + c] = from_f32<T>(which == 0 ? silu_f32(g) * u : which == 1 ? g : u);
        }
    __syncthreads();
  };
  stage(0);
  store_tile_rows<T, G::BM, G::BN, LDC>(lC, Z, m0, mrows, n0, nrows, f, tid);
  if constexpr (KEEP != KEEP_NONE) {
#pragma unroll
    for (int o = 0; o < 2; ++o) {
      __syncthreads();
      stage(1 + o);
      store_tile_rows<T, G::BM, G::BN, LDC>(lC, static_cast<T*>(o == 0 ? kept.G : kept.U), m0, mrows, n0, nrows, f, tid);
    }
  }
}

// bf16: NW * 32 tokens x NW * 16 features a tile on the ring (ring.h), the B rows of a
// stage being the tile's rows of W_gate and of W_up in the order that gives a lane
// NW / 2 neighbouring features of both products: SiLU(g) * u is formed and stored
// straight from the accumulators.  The tiles are grouped 4 token tiles at a time so
// that an XCD's workgroups share H and weight panels in its L2.
template <int NW, int KEEP>
__device__ __forceinline__ void gated_z_tiles(const bf16* __restrict__ H, const bf16* __restrict__ Wg,
                                              const bf16* __restrict__ Wu, bf16* Z, const Kept& kept, int64_t M, int d,
                                              int f, char* lds) {
  typedef ring::Geo<bf16, NW> G;
  constexpr int BF = G::BN / 2, WF = G::WN / 2, NF = G::NJ / 2;  // features of a tile, a wave, a lane
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int tiles_m = (int)((M + G::BM - 1) / G::BM), tiles_n = (f + BF - 1) / BF;
  auto origin = [&](int t, int64_t& m0, int& n0) {
    int tm, tn;
    grouped_tile(t, tiles_m, tiles_n, 4, tm, tn);
    m0 = (int64_t)tm * G::BM;
    n0 = tn * BF;
  };
  auto stages = [&](int, int, int& s0, int& n) {
    s0 = 0;
    n = (d + G::KS - 1) / G::KS;
  };
  auto open_a = [&](int t, int, int, ring::Loader<bf16, NW, false>& l) {
    int64_t m0;
    int n0;
    origin(t, m0, n0);
    l.init(H + m0 * d, d, M - m0, d, 0, wave, lane, [](int r) { return r; });
  };
  // LDS row r: block j of 16 rows of a wave's columns, the first half of the blocks of
  // W_gate, the second of W_up; a wave's loads (32 rows) are of one of them
  const bf16* W = wave * 32 % G::WN < WF ? Wg : Wu;
  auto open_b = [&](int t, int, int, ring::Loader<bf16, NW, false>& l) {
    int64_t m0;
    int n0;
    origin(t, m0, n0);
    l.init(W + (int64_t)n0 * d, d, f - n0, d, 0, wave, lane,
           [](int r) { return r / G::WN * WF + (r & 15) * NF + (r % WF >> 4); });
  };
  auto epilogue = [&](int t, ring::f4 (&acc)[G::MI][G::NJ], auto&& idle) {
    typedef bf16 vec __attribute__((ext_vector_type(NF)));
    int64_t m0;
    int n0;
    origin(t, m0, n0);
    const int n = n0 + wn * WF + (lane & 15) * NF;
    // 8 bits: the largest of a row's block of 64 features, this wave's 64 or (NW = 4) its
    // 32 and those of the wave beside it, exchanged through the idle slots
    auto largest = [&](int o, int i, int e) {
      uint32_t x = 0;
#pragma unroll
      for (int j = 0; j < NF; ++j) {
        // (of a vector's element itself the cast takes the vector's first)
        const float v = acc[i][o * NF + j][e];
        x = max(x, __builtin_bit_cast(uint32_t, v) & 0x7FFFFFFFu);
      }
      x = dpp_max<0xB1>(x);
      x = dpp_max<0x4E>(x);
      x = dpp_max<0x141>(x);
      return dpp_max<0x140>(x);  // row_mirror: all 16 lanes
    };
    static_assert(KEEP != KEEP_8 || (kKeep8 == 64 && (WF == 64 || BF == 64)), "a block is a wave's features, or a tile's");
    constexpr bool SHARE = KEEP == KEEP_8 && NW == 4;
    uint32_t top[2][SHARE ? G::MI : 1][4];
    if constexpr (SHARE) {
      uint32_t* share = reinterpret_cast<uint32_t*>(idle(0));
      auto at = [&](int w, int o, int i, int e) { return ((w * 2 + o) * G::MI + i) * 16 + 4 * (lane >> 4) + e; };
      core::lds_barrier();  // every wave is done with the stage in it
#pragma unroll
      for (int o = 0; o < 2; ++o)
#pragma unroll
        for (int i = 0; i < G::MI; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            top[o][i][e] = largest(o, i, e);
            if ((lane & 15) == 0) share[at(wave, o, i, e)] = top[o][i][e];
          }
      core::lds_barrier();
#pragma unroll
      for (int o = 0; o < 2; ++o)
#pragma unroll
        for (int i = 0; i < G::MI; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) top[o][i][e] = max(top[o][i][e], share[at(wave ^ 1, o, i, e)]);
    }
    // the scales: of the 16 lanes of a row each takes one of the 16 rows that they share
    // (2049 x 1024 x 4096 50 us; stored row by row by the first lane 54)
    uint32_t mine[2] = {};
    static_assert(G::MI * 4 == 16, "a scale a lane");
#pragma unroll
    for (int i = 0; i < G::MI; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t m = m0 + wm * G::WM + i * 16 + 4 * (lane >> 4) + e;
        uint32_t most[2] = {};
        if constexpr (KEEP == KEEP_8) {  // (by all lanes)
#pragma unroll
          for (int o = 0; o < 2; ++o) {
            if constexpr (SHARE) most[o] = top[o][i][e];
            else most[o] = largest(o, i, e);
            if ((lane & 15) == i * 4 + e) mine[o] = most[o];
          }
        }
        if (m >= M || n >= f) continue;
        vec z, v[2];
#pragma unroll
        for (int j = 0; j < NF; ++j) {
          z[j] = (bf16)(silu_f32(acc[i][j][e]) * acc[i][NF + j][e]);
          v[0][j] = (bf16)acc[i][j][e];
          v[1][j] = (bf16)acc[i][NF + j][e];
        }
        const int64_t at = m * f + n;
        __builtin_nontemporal_store(z, reinterpret_cast<vec*>(Z + at));
        if constexpr (KEEP == KEEP_ALL) {
          __builtin_nontemporal_store(v[0], reinterpret_cast<vec*>(static_cast<bf16*>(kept.G) + at));
          __builtin_nontemporal_store(v[1], reinterpret_cast<vec*>(static_cast<bf16*>(kept.U) + at));
        }
        if constexpr (KEEP == KEEP_8) {
#pragma unroll
          for (int o = 0; o < 2; ++o) {
            const Keep8Scale sc(most[o]);
            bf16 x[NF];
#pragma unroll
            for (int j = 0; j < NF; ++j) x[j] = v[o][j];
            const uint32_t q = sc.bytes(x);
            uint8_t* to = static_cast<uint8_t*>(o == 0 ? kept.G : kept.U) + at;
            if constexpr (NF == 4) __builtin_nontemporal_store(q, reinterpret_cast<uint32_t*>(to));
            else __builtin_nontemporal_store((uint16_t)q, reinterpret_cast<uint16_t*>(to));
          }
        }
      }
    if constexpr (KEEP == KEEP_8) {
      // (NW = 4: both waves of a block hold it, the first writes it)
      const int n64 = n0 + wn * WF;
      const int64_t m = m0 + wm * G::WM + (lane & 15) / 4 * 16 + 4 * (lane >> 4) + (lane & 3);
      if (m < M && n64 < f && n64 % kKeep8 == 0) {
        const int64_t at = m * ((f + kKeep8 - 1) / kKeep8) + n64 / kKeep8;
        kept.sG[at] = Keep8Scale(mine[0]).scale;
        kept.sU[at] = Keep8Scale(mine[1]).scale;
      }
    }
  };
  ring::run<bf16, NW, false, false, 1, KEEP == KEEP_8 && NW == 4>(lds, tiles_m * tiles_n, 0, 0, stages, open_a, open_b, epilogue);
}

template <int NW, int KEEP>
__global__ __launch_bounds__(NW * 64, NW == 8 ? 1 : 2) void gated_z_ring_kernel(const bf16* H, const bf16* Wg,
                                                                              const bf16* Wu, bf16* Z, Kept kept,
                                                                              int64_t M, int d, int f) {
  __shared__ __attribute__((aligned(1024))) char lds[ring::Geo<bf16, NW>::LDS_BYTES];
  gated_z_tiles<NW, KEEP>(H, Wg, Wu, Z, kept, M, d, f, lds);
}

namespace {

// Whether tiles of 8 waves end sooner than those of 4, from the rounds that each
// takes: a tile of 4 waves has a quarter of the products and, two on a CU, takes some
// 0.31 of the time.
bool wide_tiles(int64_t M, int f, int cus) {
  const auto rounds = [&](int64_t nw, int64_t groups) {
    return (((M + nw * 32 - 1) / (nw * 32)) * ((f + nw * 16 - 1) / (nw * 16)) + groups - 1) / groups;
  };
  return (double)rounds(8, cus) <= 0.62 * (double)rounds(4, 2 * cus);
}

template <int KEEP>
hipError_t launch_kept(const Prob& p, const void* H, const void* Wg, const void* Wu, void* Z, const Kept& kept,
                       hipStream_t st) {
  note_launch("gated_z", st);
  if (p.dtype == 1) {
    const auto go = [&](auto nw, int cus) {
      constexpr int NW = decltype(nw)::value;
      const int64_t tiles = ((p.M + NW * 32 - 1) / (NW * 32)) * ((p.f + NW * 16 - 1) / (NW * 16));
      const int64_t g = std::min<int64_t>(cus * (NW == 8 ? 1 : 2), (tiles + 7) / 8 * 8);
      gated_z_ring_kernel<NW, KEEP><<<(unsigned)g, NW * 64, 0, st>>>((const bf16*)H, (const bf16*)Wg, (const bf16*)Wu,
                                                                    (bf16*)Z, kept, p.M, p.d, p.f);
    };
    // one persistent workgroup of 8 waves a CU, or two of 4 (the walk needs a multiple
    // of 8)
    int dev = 0, cus = 256;
    if (hipGetDevice(&dev) == hipSuccess)
      (void)hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev);
    cus = std::max(8, cus / 8 * 8);
    if (wide_tiles(p.M, p.f, cus)) go(std::integral_constant<int, 8>(), cus);
    else go(std::integral_constant<int, 4>(), cus);
  } else if constexpr (KEEP == KEEP_8) {
    return hipErrorInvalidValue;  // 8 bits are for bf16 data
  } else {
    const int64_t tiles = ((p.M + 127) / 128) * ((p.f + 127) / 128);
    gated_z_kernel<float, KEEP><<<(unsigned)tiles, kThreads, 0, st>>>(
        (const float*)H, (const float*)Wg, (const float*)Wu, (float*)Z, kept, p.M, p.d, p.f);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gated_z(const Prob& p, const void* H, const void* Wg, const void* Wu, void* Z, void* GU,
                          hipStream_t st) {
  if (GU == nullptr) return launch_kept<KEEP_NONE>(p, H, Wg, Wu, Z, Kept{}, st);
  const size_t e = p.dtype == 1 ? 2 : 4;
  return launch_kept<KEEP_ALL>(p, H, Wg, Wu, Z, Kept{GU, static_cast<char*>(GU) + (size_t)p.M * p.f * e, nullptr, nullptr},
                               st);
}

hipError_t launch_gated_z8(const Prob& p, const void* H, const void* Wg, const void* Wu, void* Z, const Keep8& k,
                           hipStream_t st) {
  return launch_kept<KEEP_8>(p, H, Wg, Wu, Z, Kept{k.G, k.U, k.sG, k.sU}, st);
}

}  // namespace ipttt
