// Persistent tile products for gfx950 in bf16, C[m, n] = sum_k A[m, k] B[n, k]: tiles
// of 256 x 256 by 8 waves, or of 128 x 128 by 4 (two workgroups a CU), on
// v_mfma_f32_16x16x32_bf16.  Either operand may lie with K contiguous or K-major
// (A[m, k] at p[k * ld + m]).
//
// Operands go HBM/L2 -> LDS with direct loads into a ring of five slots, each the A
// or the B part of a stage of 64 K: stage q's A in slot 2q % 5, its B in slot
// (2q + 1) % 5.  While stage q is multiplied, B of stage q+1 and A of stage q+2 are
// issued, into the slots that stage q-1 left, so that A has a stage and a half to
// arrive, B a stage, and each memory phase issues four loads a wave.  The ring goes
// on over the ends of a workgroup's tiles: the next one's first stages are in flight
// while a tile is finished.
//
// 8 waves: two groups with one wave of each on every SIMD, one phase apart, so
// that one reads fragments and issues loads while the other multiplies; a barrier
// ends each phase.  4 waves: the CU's other workgroup fills the gaps.
//
// LDS layouts, both free of bank conflicts:
//   rows     128-byte rows of 64 K; 16-byte chunk c of LDS row r at slot
//            c ^ ((r >> 1) & 7).
//   K-major  a row of the tile's width for each K; its 32-byte unit u (16 columns)
//            at slot u ^ (2 (k & 3) + ((k >> 3) & 1)), read with the transposing
//            LDS loads.
// LDS row r of B's rows need not hold row r of the tile: with the order of PERM a
// lane ends up with neighbouring columns of C and stores 16 bytes at once.
//
// Measured (one MI355X, TFLOP/s; both K contiguous, B K-major, both K-major):
// 8192^3 1434, 1340, 1325; 8192 x 6144 x 2560 1339, 1256, 1213.  With two whole stages
// instead of the ring 1283, 1341, 1332 and 1294, 1251, 1265; with 32x32x16 products
// 1372 and 1271 (first only); both parts' loads issued in one phase 1354; four waves
// of 128 x 128 instead of eight 1040.
#pragma once

#include "common.h"
#include "mfma_core.h"

namespace ipttt {
namespace ring {

constexpr int KS = 64, NSLOT = 5;
typedef float4_t f4;

template <int NW>
struct Geo {
  static constexpr int BM = NW * 32, BN = NW * 32;          // 256 or 128
  static constexpr int WAVES_N = 2, WAVES_M = NW / 2;
  static constexpr int WM = 64, WN = BN / 2, MI = WM / 16, NJ = WN / 16;
  static_assert(BM == WAVES_M * WM, "wave grid");
  static constexpr int SLOT = BM * KS * 2;                  // bytes
  static constexpr int LDS_BYTES = NSLOT * SLOT;
  static constexpr int NT = NW * 64;
  static constexpr int NL = 4;                              // load instructions a wave and part
  static_assert(SLOT == NW * NL * 1024, "load split");
  static constexpr int MAX_GROUPS = NW == 8 ? 1 : 2;        // workgroups a CU
};

// Offsets past every buffer's end: such a load reads zeros.
constexpr uint32_t kOut = 0xFFFFFFF0u;

// One operand's loads.  init(): p at the tile's first row (or column), n rows (or
// columns) of it valid, K valid along k; stages count from k = 0.
template <int NW, bool KMAJ>
struct Loader {
  typedef Geo<NW> G;
  uint32_t voff[G::NL];
  uint32_t chunk;        // rows: K element of this lane's pieces within a stage, by load (4 bits each, in 8s)
  const char* base;
  int64_t left, step;    // bytes valid from base on; bytes a stage
  int K;                 // rows: valid k (K-major: unused)

  // row(r): the operand's row that LDS row r holds
  template <class Row>
  __device__ __forceinline__ void init(const bf16* p, int64_t ld, int64_t n, int64_t kvalid, int wave, int lane,
                                       Row&& row) {
    base = reinterpret_cast<const char*>(p);
    const uint32_t ldb = (uint32_t)ld * 2u;
    if constexpr (!KMAJ) {
      left = n > 0 ? (n - 1) * ld * 2 + kvalid * 2 : 0;
      step = KS * 2;
      K = (int)kvalid;
      chunk = 0;
#pragma unroll
      for (int j = 0; j < G::NL; ++j) {
        const int r = (wave * G::NL + j) * 8 + (lane >> 3), c = (lane & 7) ^ ((r >> 1) & 7);
        const int at = row(r);
        voff[j] = at < n ? (uint32_t)at * ldb + (uint32_t)c * 16u : kOut;
        chunk |= (uint32_t)c << (4 * j);
      }
    } else {
      left = n > 0 ? (kvalid - 1) * ld * 2 + n * 2 : 0;
      step = (int64_t)KS * ld * 2;
      constexpr int LPR = G::BM / 8, RPI = 64 / LPR;  // lanes a K row, K rows an instruction
#pragma unroll
      for (int j = 0; j < G::NL; ++j) {
        const int r = (wave * G::NL + j) * RPI + lane / LPR, s = lane % LPR;
        const int u = (s >> 1) ^ (((r & 3) << 1) | ((r >> 3) & 1)), col = u * 16 + (s & 1) * 8;
        voff[j] = col < n ? (uint32_t)r * ldb + (uint32_t)col * 2u : kOut;
      }
    }
  }
  __device__ __forceinline__ void issue(int s, char* slot, int wave) const {
    const int64_t off = (int64_t)s * step;
    const __amdgpu_buffer_rsrc_t rs = core::make_operand(base + off, 0, left - off).rsrc;
    char* to = slot + wave * G::NL * 1024;
    if (!KMAJ && (s + 1) * KS > K) {  // the last stage's pieces past K read as zero
#pragma unroll
      for (int j = 0; j < G::NL; ++j)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rs, (core::lds_ptr_t)(to + j * 1024), 16,
            s * KS + (int)((chunk >> (4 * j)) & 7) * 8 < K ? voff[j] : kOut, 0, 0, 0);
      return;
    }
#pragma unroll
    for (int j = 0; j < G::NL; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (core::lds_ptr_t)(to + j * 1024), 16, voff[j], 0, 0, 0);
  }
};

// Fragments of 16 rows x 32 K from a slot.
template <int NW, bool KMAJ>
struct Reader {
  typedef Geo<NW> G;
  int at, sw, unit;
  __device__ __forceinline__ void init(int row0, int lane) {
    if constexpr (!KMAJ) {
      const int r = row0 + (lane & 15);
      at = r * 128;
      sw = (r >> 1) & 7;
      unit = lane >> 4;
    } else {
      const int kg = lane >> 4, r = (lane >> 2) & 3;
      at = (8 * kg + r) * G::BM * 2 + (lane & 3) * 8;
      sw = (r << 1) | (kg & 1);
      unit = row0 >> 4;
    }
  }
  // block blk of 16 rows, half h of the stage's K
  __device__ __forceinline__ bf16x8 get(const char* slot, int blk, int h) const {
    if constexpr (!KMAJ) {
      return *reinterpret_cast<const bf16x8*>(slot + at + blk * 16 * 128 + (((h * 4 + unit) ^ sw) << 4));
    } else {
      typedef __attribute__((address_space(3))) short4_t* lp4;
      const char* p = slot + at + h * 32 * G::BM * 2 + (((unit + blk) ^ sw) << 5);
      const short4_t x0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp4)p);
      const short4_t x1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp4)(p + 4 * G::BM * 2));
      return __builtin_bit_cast(bf16x8, __builtin_shufflevector(x0, x1, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }
};

// The order of B's rows with which a lane's NJ blocks are NJ neighbouring columns.
template <int NW>
__device__ __forceinline__ int perm_row(int r) {
  constexpr int WN = Geo<NW>::WN, NJ = Geo<NW>::NJ;
  return r / WN * WN + (r & 15) * NJ + (r % WN >> 4);
}

// The items of a launch: [0, n1), then [n1, n1 + n2).  The hardware hands
// consecutive workgroups to the 8 XCDs in turn; each XCD's workgroups walk a
// contiguous range of either kind together.  Launches have a multiple of 8
// workgroups.
struct Walk {
  int n1, n2, t, end, per;
  bool second;
  __device__ __forceinline__ void range(int first, int n) {
    const int xcd = blockIdx.x & 7, slot = blockIdx.x >> 3, r = (n + 7) >> 3;
    end = first + min(n, (xcd + 1) * r);
    t = first + xcd * r + slot;
  }
  __device__ __forceinline__ void settle() {
    if (t < end || second) return;
    second = true;
    range(n1, n2);
  }
  __device__ __forceinline__ Walk(int a, int b) : n1(a), n2(b), per((int)gridDim.x >> 3), second(false) {
    range(0, n1);
    settle();
  }
  __device__ __forceinline__ bool on() const { return t < end; }
  __device__ __forceinline__ void next() {
    t += per;
    settle();
  }
};

// Walks the items.  stages(t) gives item t's first stage and their number (at least
// one); open_a(t, loader) and open_b(t, loader) set its operands;
// epilogue(t, acc) takes the finished tile: block (i, j), element e of a lane is
// row wm * 64 + i * 16 + 4 * (lane / 16) + e and LDS row wn * WN + j * 16 + lane % 16
// of B.  A and B are restrict so that the compiler tells the LDS reads apart from
// the direct loads and puts no wait for those in front of them; the ring's own
// waits order them.
template <int NW, bool AK, bool BK, class Stages, class OpenA, class OpenB, class Epilogue>
__device__ __forceinline__ void run(char* lds, int n1, int n2, Stages&& stages, OpenA&& open_a, OpenB&& open_b,
                                    Epilogue&& epilogue) {
  typedef Geo<NW> G;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1, grp = NW == 8 ? wave >> 2 : 0;
  Walk w(n1, n2), wa = w, wb = w;
  if (!w.on()) return;
  Loader<NW, AK> la;
  Loader<NW, BK> lb;
  Reader<NW, AK> ra;
  Reader<NW, BK> rb;
  ra.init(wm * G::WM, lane);
  rb.init(wn * G::WN, lane);
  auto m5 = [](int x) { return x >= NSLOT ? x - NSLOT : x; };
  int sa = 0, ea = 0, sb = 0, eb = 0;  // the next stages to issue, and the items' ends
  auto first = [&](const Walk& x, int& s, int& e) {
    int n;
    stages(x.t, s, n);
    e = s + n;
  };
  first(wa, sa, ea);
  first(wb, sb, eb);
  open_a(wa.t, la);
  open_b(wb.t, lb);
  int ia = 0, ib = 1;  // the slots they go to
  auto issue_a = [&]() {
    if (!wa.on()) return false;
    la.issue(sa, lds + ia * G::SLOT, wave);
    ia = m5(ia + 2);
    if (++sa == ea) {
      wa.next();
      if (wa.on()) {
        first(wa, sa, ea);
        open_a(wa.t, la);
      }
    }
    return true;
  };
  auto issue_b = [&]() {
    if (!wb.on()) return;
    lb.issue(sb, lds + ib * G::SLOT, wave);
    ib = m5(ib + 2);
    if (++sb == eb) {
      wb.next();
      if (wb.on()) {
        first(wb, sb, eb);
        open_b(wb.t, lb);
      }
    }
  };
  // all but the A part issued last have landed
  bool more = false;
  auto landed = [&]() {
    if (more) core::wait_vmcnt<G::NL>();
    else core::wait_vmcnt<0>();
  };
  issue_a();
  issue_b();
  more = issue_a();
  int a = 0;  // the slot of A of the stage to multiply
  if constexpr (NW == 8) {
    landed();
    core::lds_barrier();
  }
  for (; w.on(); w.next()) {
    f4 acc[G::MI][G::NJ];
#pragma unroll
    for (int i = 0; i < G::MI; ++i)
#pragma unroll
      for (int j = 0; j < G::NJ; ++j) acc[i][j] = f4{0.0f, 0.0f, 0.0f, 0.0f};
    bf16x8 fa[G::MI], fb[G::NJ];
    int s0, S;
    stages(w.t, s0, S);
    auto read = [&](int h) {
      const char *pa = lds + a * G::SLOT, *pb = lds + m5(a + 1) * G::SLOT;
#pragma unroll
      for (int i = 0; i < G::MI; ++i) fa[i] = ra.get(pa, i, h);
#pragma unroll
      for (int j = 0; j < G::NJ; ++j) fb[j] = rb.get(pb, j, h);
    };
    auto multiply = [&]() {
#pragma unroll
      for (int i = 0; i < G::MI; ++i)
#pragma unroll
        for (int j = 0; j < G::NJ; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[i], fb[j], acc[i][j], 0, 0, 0);
    };
    if constexpr (NW == 8) {
      auto phase_end = [&](bool wait) {
        __builtin_amdgcn_sched_barrier(0);
        if (wait) landed();
        core::lds_barrier();
        __builtin_amdgcn_sched_barrier(0);
      };
      // Group 1 meets one barrier more before its phases, group 0 one after.  A
      // wave's loads of stage s+1 have landed before the barrier ahead of group
      // 0's first read of it (group 0: after its last products of stage s; group
      // 1: after its last reads of it).
      if (grp == 1) phase_end(false);
      for (int s = 0; s < S; ++s) {
        issue_b();
        __builtin_amdgcn_sched_barrier(0);
        read(0);
        phase_end(false);
        multiply();
        phase_end(false);
        more = issue_a();
        __builtin_amdgcn_sched_barrier(0);
        read(1);
        phase_end(grp == 1);
        multiply();
        phase_end(grp == 0);
        a = m5(a + 2);
      }
      if (grp == 0) phase_end(false);
    } else {
      for (int s = 0; s < S; ++s) {
        // this wave's loads of stage s have landed, and every wave is done with
        // stage s-1
        landed();
        core::lds_barrier();
        __builtin_amdgcn_sched_barrier(0);
        issue_b();
        more = issue_a();
        __builtin_amdgcn_sched_barrier(0);
        read(0);
        multiply();
        read(1);
        multiply();
        __builtin_amdgcn_sched_barrier(0);
        a = m5(a + 2);
      }
    }
    epilogue(w.t, acc);
  }
}

}  // namespace ring
}  // namespace ipttt
