// Persistent tile products for gfx950, C[m, n] = sum_k A[m, k] B[n, k]: tiles of 256 x
// 256 by 8 waves, of 128 x 128 by 4 (two workgroups a CU) or of 64 x 64 by 4 (four), on
// v_mfma_f32_16x16x32_bf16 or v_mfma_f32_16x16x4_f32.  The smaller the tile, the more
// evenly a small product spreads and the more bytes it loads; in fp32, whose products take
// 8 times as long for the same bytes, that costs nothing.  Either operand may lie with K
// contiguous or K-major (A[m, k] at p[k * ld + m]).
//
// Operands go HBM/L2 -> LDS with direct loads into a ring of five slots, each the A
// or the B part of a stage of 128 bytes of K: stage q's A in slot 2q % 5, its B in slot
// (2q + 1) % 5.  The ring goes on over the ends of a workgroup's tiles: the next one's
// first stages are in flight while a tile is finished.
//
// 8 waves: two groups with one wave of each on every SIMD, one phase apart, so
// that one reads fragments and issues loads while the other multiplies; a barrier
// ends each phase.  While stage q is multiplied, B of stage q+1 and A of stage q+2 are
// issued, into the slots that stage q-1 left, so that A has a stage and a half to
// arrive, B a stage, and each memory phase issues four loads a wave.
// 4 waves: one barrier a stage, in its middle; each half is multiplied while the next
// half's fragments are read and one part's loads (A of stage q+2, B of stage q+2) are
// issued, spread over the products.  A CU's loads take as long as its products
// here in bf16 (32 KB and 512 cycles a stage), so that eight loads issued at once left the
// matrix units idle: a tile alone took 0.49 us a stage and now takes 0.36, 2049 x 2560 x
// 2560 40.5 us and now 35.5.  A ring twice as deep, one workgroup a CU, gained nothing
// (0.49): the loads' rate counts, not their latency.
//
// LDS layouts, both free of bank conflicts:
//   rows     128-byte rows; 16-byte chunk c of LDS row r at slot
//            c ^ ((r >> 1) & 7).
//   K-major  a row of the tile's width for each K.  bf16: its 32-byte unit u (16
//            columns) at slot u ^ kmajor_swizzle(k & 3, k >> 3), read with the
//            transposing LDS loads; fp32: its 64-byte unit at slot u ^ ((k >> 2) & 3),
//            read one element at a time.
// LDS row r of B's rows need not hold row r of the tile: with the order of PERM a
// lane ends up with neighbouring columns of C and stores 16 bytes at once.
//
// Measured (one MI355X, TFLOP/s; both K contiguous, B K-major, both K-major):
// 8192^3 1370, 1394, 1380; 8192 x 6144 x 2560 1366, 1255, 1279; fp32: 8192 x 6144 x 2560 139,
// 137, 136, 1021 x 4096 x 1024 128, 126.  Cards differ in their clock under load: on another,
// bf16 was 1519, 1501, 1474 and 1418, 1292, 1399, and there the steady loop without branches
// made these of 1434, 1340, 1325 and 1339, 1256, 1213; next to those stood, with
// two whole stages instead of the ring, 1283, 1341, 1332 and 1294, 1251, 1265; with
// 32x32x16 products 1372 and 1271 (first only); both parts' loads issued in one phase
// 1354; four waves of 128 x 128 instead of eight 1040.
#pragma once

#include <type_traits>

#include "common.h"
#include "mfma_core.h"

namespace ipttt {
namespace ring {

constexpr int SLOTS = 5;
typedef float4_t f4;

template <typename T>
constexpr int kStage = 128 / (int)sizeof(T);  // K of a stage

template <typename T, int NW>
struct Geo {
  static constexpr int KS = kStage<T>, ES = sizeof(T), VE = 16 / ES;
  static constexpr int BM = NW * 32, BN = NW * 32;          // 256, 128 or 64
  static constexpr int WAVES = NW == 8 ? 8 : 4, WAVES_N = 2, WAVES_M = WAVES / 2;
  static constexpr int WM = BM / WAVES_M, WN = BN / 2, MI = WM / 16, NJ = WN / 16;
  static constexpr int SLOT = BM * 128;                     // bytes
  static constexpr int LDS_BYTES = SLOTS * SLOT;
  static constexpr int NT = WAVES * 64;
  static constexpr int NL = SLOT / (WAVES * 1024);          // load instructions a wave and part
  static constexpr int GROUPS = 8 / NW;                     // workgroups a CU
  static_assert(NW == 8 || NW == 4 || NW == 2, "tiles");
  static_assert(NW == 8 || NL == MI, "a load for each block row of products");
};

// Offsets past every buffer's end: such a load reads zeros.  (A tile's rows end
// below 2^31: 255 strides of 2^22 elements, and K.)
constexpr uint32_t kOut = 0x80000000u;

// 16 bytes of an operand, and their products: bf16 32 of K; fp32 16 of K, element e of a
// lane being K = 4 (lane / 16) + e in both operands.
template <typename T> struct Frag;
template <> struct Frag<bf16> {
  typedef bf16x8 type;
  static __device__ __forceinline__ f4 mma(type a, type b, f4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};
template <> struct Frag<float> {
  typedef float4_t type;
  static __device__ __forceinline__ f4 mma(type a, type b, f4 c) {
#pragma unroll
    for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
    return c;
  }
};

// The exchange of the units of a K-major row in bf16, K = 8 kg + r or 8 kg + 4 + r: half a
// wave reads r = 0 .. 3 of two kg at once, one unit each, and those have to lie in
// different banks (a row of 64 columns is half the banks' width, so that two K share one).
template <int NW>
__device__ __forceinline__ int kmajor_swizzle(int r, int kg) {
  return NW == 2 ? (r >> 1 & 1) | (kg & 1) << 1 : r << 1 | (kg & 1);
}

// One operand's loads.  issue() loads the stage that the cursor stands at, and
// advance() moves it, so that the scalar work of a stage's addresses is done while
// the fragment reads behind the loads are on their way.
template <typename T, int NW, bool KMAJ>
struct Loader {
  typedef Geo<T, NW> G;
  static constexpr int KS = G::KS;
  uint32_t voff[G::NL];
  uint32_t chunk;              // rows: K element of this lane's pieces within a stage, by load (4 bits each, in 8s)
  __amdgpu_buffer_rsrc_t rs;   // rows: over the tile's rows, the stage's bytes into a row, and a row's valid bytes
  uint32_t at, kbytes;
  const char* base;            // K-major: the stage's first K row, the valid rows from it on, bytes a row
  int krows;
  uint32_t ldb, width;

  // p at the tile's first row (or column), n > 0 rows (or columns) of it valid, K
  // valid along k; row(r): the operand's row that LDS row r holds
  template <class Row>
  __device__ __forceinline__ void init(const T* p, int64_t ld, int64_t n, int64_t kvalid, int stage, int wave,
                                       int lane, Row&& row) {
    ldb = (uint32_t)ld * G::ES;
    const uint32_t here = (uint32_t)min(n, (int64_t)G::BM);
    if constexpr (!KMAJ) {
      kbytes = (uint32_t)kvalid * G::ES;
      at = (uint32_t)stage * 128;
      rs = core::make_operand(p, 0, (int64_t)(here - 1) * ldb + kbytes).rsrc;
      chunk = 0;
#pragma unroll
      for (int j = 0; j < G::NL; ++j) {
        const int r = (wave * G::NL + j) * 8 + (lane >> 3), c = (lane & 7) ^ ((r >> 1) & 7);
        const uint32_t from = (uint32_t)row(r);
        voff[j] = from < here ? from * ldb + (uint32_t)c * 16u : kOut;
        chunk |= (uint32_t)c << (4 * j);
      }
    } else {
      base = reinterpret_cast<const char*>(p) + (int64_t)stage * KS * ldb;
      krows = (int)kvalid - stage * KS;
      width = here * G::ES;
      constexpr int LPR = G::BM / G::VE, RPI = 64 / LPR;  // lanes a K row, K rows an instruction
#pragma unroll
      for (int j = 0; j < G::NL; ++j) {
        const int r = (wave * G::NL + j) * RPI + lane / LPR, s = lane % LPR;
        const int u = G::ES == 2 ? (s >> 1) ^ kmajor_swizzle<NW>(r & 3, r >> 3) : (s >> 2) ^ ((r >> 2) & 3);
        const int col = u * 16 + (G::ES == 2 ? (s & 1) * 8 : (s & 3) * 4);
        voff[j] = (uint32_t)col < here ? (uint32_t)r * ldb + (uint32_t)col * G::ES : kOut;
      }
    }
  }
  __device__ __forceinline__ void advance() {
    if constexpr (!KMAJ) {
      at += 128;
    } else {
      base += (int64_t)KS * ldb;
      krows -= KS;
    }
  }
  // Tells the compiler that the cursor is the same in all lanes: it cannot see that
  // after the branches that move a loader on to the next item.
  __device__ __forceinline__ void uniform() {
    if constexpr (!KMAJ) {
      at = __builtin_amdgcn_readfirstlane(at);
    } else {
      const uint64_t p = reinterpret_cast<uint64_t>(base);
      const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)p), hi = __builtin_amdgcn_readfirstlane((uint32_t)(p >> 32));
      base = reinterpret_cast<const char*>((uint64_t)hi << 32 | lo);
      krows = __builtin_amdgcn_readfirstlane(krows);
    }
  }
  // Load j of the stage's four.  last (a constant): the stage may be the last one, cut
  // short by K, so that its pieces past K read as zero.
  __device__ __forceinline__ void issue_one(char* slot, int wave, bool last, int j) const {
    core::lds_ptr_t to = (core::lds_ptr_t)(slot + (wave * G::NL + j) * 1024);
    if constexpr (!KMAJ) {
      const bool cut = last && at + ((chunk >> (4 * j)) & 7) * 16 >= kbytes;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, to, 16, cut ? kOut : voff[j], at, 0, 0);
    } else {
      // a resource over the stage's K rows
      int end = 0x7FFFFFFF;
      if (last && krows < KS) end = krows > 0 ? (int)((uint32_t)(krows - 1) * ldb + width) : 0;
      const __amdgpu_buffer_rsrc_t r =
          __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), (short)0, end, 0x00020000);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, to, 16, voff[j], 0, 0, 0);
    }
  }
  __device__ __forceinline__ void issue(char* slot, int wave, bool last) const {
#pragma unroll
    for (int j = 0; j < G::NL; ++j) issue_one(slot, wave, last, j);
  }
};

// Fragments of 16 rows and half a stage's K from a slot.
template <typename T, int NW, bool KMAJ>
struct Reader {
  typedef Geo<T, NW> G;
  typedef typename Frag<T>::type frag;
  int at, sw, unit;
  __device__ __forceinline__ void init(int row0, int lane) {
    if constexpr (!KMAJ) {
      const int r = row0 + (lane & 15);
      at = r * 128;
      sw = (r >> 1) & 7;
      unit = lane >> 4;
    } else if constexpr (G::ES == 4) {
      at = 4 * (lane >> 4) * G::BM * 4 + (lane & 15) * 4;
      sw = lane >> 4;
      unit = row0 >> 4;
    } else {
      const int kg = lane >> 4, r = (lane >> 2) & 3;
      at = (8 * kg + r) * G::BM * 2 + (lane & 3) * 8;
      sw = kmajor_swizzle<NW>(r, kg);
      unit = row0 >> 4;
    }
  }
  // block blk of 16 rows, half h of the stage's K
  __device__ __forceinline__ frag get(const char* slot, int blk, int h) const {
    if constexpr (!KMAJ) {
      return *reinterpret_cast<const frag*>(slot + at + blk * 16 * 128 + (((h * 4 + unit) ^ sw) << 4));
    } else if constexpr (G::ES == 4) {
      const char* p = slot + at + h * 16 * G::BM * 4 + (((unit + blk) ^ sw) << 6);
      frag x;
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = *reinterpret_cast<const float*>(p + e * G::BM * 4);
      return x;
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
  constexpr int WN = Geo<float, NW>::WN, NJ = Geo<float, NW>::NJ;
  return r / WN * WN + (r & 15) * NJ + (r % WN >> 4);
}

// The items of a launch: [0, n1), then [n1, n1 + n2).  The hardware hands
// consecutive workgroups to the 8 XCDs in turn; each XCD's workgroups walk a
// contiguous range of either kind together.  Launches have a multiple of 8
// workgroups.
struct Walk {
  int n1, n2, t, end, per, slot;
  bool second;
  __device__ __forceinline__ void range(int first, int n) {
    const int xcd = blockIdx.x & 7, r = (n + 7) >> 3;
    end = first + min(n, (xcd + 1) * r);
    t = first + xcd * r + slot;
  }
  __device__ __forceinline__ void settle() {
    if (t < end || second) return;
    second = true;
    range(n1, n2);
  }
  // turn: the workgroup of an XCD that begins
  __device__ __forceinline__ Walk(int a, int b, int turn)
      : n1(a), n2(b), per((int)gridDim.x >> 3), slot(((int)blockIdx.x >> 3) - turn), second(false) {
    if (slot < 0) slot += per;
    range(0, n1);
    settle();
  }
  __device__ __forceinline__ bool on() const { return t < end; }
  __device__ __forceinline__ void next() {
    t += per;
    settle();
  }
};

// Walks the items, from the XCD's workgroup `turn` on (a launch may walk the items of
// two products one after the other).  An item is summed over LEGS legs, pairs of operands:
// stages(t, leg, first, n) gives the first stage of one and their number (of some leg
// at least one), open_a(t, leg, first, loader) and open_b set its operands.
// epilogue(t, acc, idle) takes the finished tile, with idle two slots that nothing
// reads or loads until the next barrier that all waves meet after it (waves may
// still be reading them when it begins): block (i, j), element e of a lane is
// row wm * WM + i * 16 + 4 * (lane / 16) + e and LDS row wn * WN + j * 16 + lane % 16
// of B.  A and B are restrict so that the compiler tells the LDS reads apart from
// the direct loads and puts no wait for those in front of them; the ring's own
// waits order them.
template <typename T, int NW, bool AK, bool BK, int LEGS, bool HOLD, class Stages, class OpenA, class OpenB, class Epilogue>
__device__ __forceinline__ void run(char* lds, int n1, int n2, int turn, Stages&& stages, OpenA&& open_a, OpenB&& open_b,
                                    Epilogue&& epilogue) {
  typedef Geo<T, NW> G;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1, grp = NW == 8 ? wave >> 2 : 0;
  Walk w(n1, n2, turn), wa = w, wb = w;
  if (!w.on()) return;
  Loader<T, NW, AK> la;
  Loader<T, NW, BK> lb;
  Reader<T, NW, AK> ra;
  Reader<T, NW, BK> rb;
  ra.init(wm * G::WM, lane);
  rb.init(wn * G::WN, lane);
  // The legs that the loaders stand at, their stages left to issue, and whether
  // there is one.
  int na = 0, nb = 0, leg_a = -1, leg_b = -1;
  bool on_a = true, on_b = true;
  // to the next leg that has stages, of this item or the next
  auto enter_a = [&]() {
    int s;
    for (na = 0;;) {
      if (++leg_a == LEGS) {
        leg_a = 0;
        wa.next();
        on_a = wa.on();
        if (!on_a) return;
      }
      stages(wa.t, leg_a, s, na);
      if (LEGS == 1 || na > 0) break;
    }
    open_a(wa.t, leg_a, s, la);
  };
  auto enter_b = [&]() {
    int s;
    for (nb = 0;;) {
      if (++leg_b == LEGS) {
        leg_b = 0;
        wb.next();
        on_b = wb.on();
        if (!on_b) return;
      }
      stages(wb.t, leg_b, s, nb);
      if (LEGS == 1 || nb > 0) break;
    }
    open_b(wb.t, leg_b, s, lb);
  };
  enter_a();
  enter_b();
  constexpr int RING = G::LDS_BYTES;
  auto past = [](int x) { return x >= RING ? x - RING : x; };
  int a = 0;  // where A of the stage to multiply lies; the slots after it: B, the next A, the next B, the A after
  auto advance_a = [&]() {
    if (--na > 0) la.advance();
    else enter_a();
  };
  auto advance_b = [&]() {
    if (--nb > 0) lb.advance();
    else enter_b();
  };
  bool more;  // whether every part up to the one issued last was there to issue
  if constexpr (NW == 8) {
    la.issue(lds, wave, true);
    advance_a();
    lb.issue(lds + G::SLOT, wave, true);
    advance_b();
    more = on_a;
    if (on_a) {
      la.issue(lds + 2 * G::SLOT, wave, true);
      advance_a();
    }
    if (more) core::wait_vmcnt<G::NL>();
    else core::wait_vmcnt<0>();
  } else {
#pragma unroll
    for (int p = 0; p < SLOTS - 1; ++p) {
      more = p % 2 == 0 ? on_a : on_b;
      if (!more) break;
      if (p % 2 == 0) {
        la.issue(lds + p * G::SLOT, wave, true);
        advance_a();
      } else {
        lb.issue(lds + p * G::SLOT, wave, true);
        advance_b();
      }
    }
    if (more) core::wait_vmcnt<2 * G::NL>();
    else core::wait_vmcnt<0>();
  }
  core::lds_barrier();
  // 4 waves: the fragments of the two halves; half 0 of a stage is read ahead of it
  typename Frag<T>::type fa[NW == 8 ? 1 : 2][G::MI], fb[NW == 8 ? 1 : 2][G::NJ];
  auto read = [&](int stage_at, int h, int to) {
    const char *pa = lds + past(a + stage_at * G::SLOT), *pb = lds + past(a + (stage_at + 1) * G::SLOT);
#pragma unroll
    for (int i = 0; i < G::MI; ++i) fa[to][i] = ra.get(pa, i, h);
#pragma unroll
    for (int j = 0; j < G::NJ; ++j) fb[to][j] = rb.get(pb, j, h);
  };
  if constexpr (NW != 8) read(0, 0, 0);
  for (; w.on(); w.next()) {
    f4 acc[G::MI][G::NJ];
#pragma unroll
    for (int i = 0; i < G::MI; ++i)
#pragma unroll
      for (int j = 0; j < G::NJ; ++j) acc[i][j] = f4{0.0f, 0.0f, 0.0f, 0.0f};
    auto multiply = [&](int from) {
#pragma unroll
      for (int i = 0; i < G::MI; ++i)
#pragma unroll
        for (int j = 0; j < G::NJ; ++j) acc[i][j] = Frag<T>::mma(fa[from][i], fb[from][j], acc[i][j]);
    };
    // A part's loads into the slot `to` slots behind the stage's A.  STEADY: the loaders
    // stay in this item, short of its last stage, so that nothing is asked; otherwise
    // they may be at its last stage, in the next item or done.
    auto next_b = [&](auto steady, int to) {
      constexpr bool STEADY = decltype(steady)::value;
      if constexpr (STEADY) {
        lb.issue(lds + past(a + to * G::SLOT), wave, false);
      } else {
        more = on_b;
        if (on_b) lb.issue(lds + past(a + to * G::SLOT), wave, true);
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    auto next_a = [&](auto steady, int to) {
      constexpr bool STEADY = decltype(steady)::value;
      if constexpr (STEADY) {
        la.issue(lds + past(a + to * G::SLOT), wave, false);
      } else {
        more = on_a;
        if (on_a) la.issue(lds + past(a + to * G::SLOT), wave, true);
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    auto step_b = [&](auto steady) {
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (decltype(steady)::value) lb.advance();
      else if (on_b) advance_b();
    };
    auto step_a = [&](auto steady) {
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (decltype(steady)::value) la.advance();
      else if (on_a) advance_a();
    };
    // 4 waves: half h of the stage is multiplied while the other half's (h = 1: the next
    // stage's first) fragments are read and one part's loads are issued, spread over the
    // products: the loads of a CU take as long as its products.
    auto window = [&](auto steady, auto half, bool hold) {
      constexpr bool STEADY = decltype(steady)::value;
      constexpr int H = decltype(half)::value;
      // A to where B of the stage before lay, B to where this stage's A lay
      constexpr int TO = H == 0 ? SLOTS - 1 : 0;
      constexpr bool IS_A = H == 0;
      if (!STEADY && !hold) {
        if constexpr (IS_A) {
          next_a(steady, TO);
          step_a(steady);
        } else {
          next_b(steady, TO);
          step_b(steady);
        }
      }
      char* to = lds + past(a + TO * G::SLOT);
      const char *pa = lds + past(a + 2 * H * G::SLOT), *pb = lds + past(a + (2 * H + 1) * G::SLOT);
#pragma unroll
      for (int i = 0; i < G::MI; ++i) {
        if (STEADY) {
          if constexpr (IS_A) la.issue_one(to, wave, false, i);
          else lb.issue_one(to, wave, false, i);
        }
        if (i == 0) {
#pragma unroll
          for (int q = 0; q < G::MI; ++q) fa[1 - H][q] = ra.get(pa, q, 1 - H);
        }
        if (i == 1) {
#pragma unroll
          for (int q = 0; q < G::NJ; ++q) fb[1 - H][q] = rb.get(pb, q, 1 - H);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < G::NJ; ++j) acc[i][j] = Frag<T>::mma(fa[H][i], fb[H][j], acc[i][j]);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (STEADY) {
        if constexpr (IS_A) la.advance();
        else lb.advance();
      }
    };
    auto stage = [&](auto steady, bool hold) {
      constexpr bool STEADY = decltype(steady)::value;
      auto landed = [&]() {  // all but the A issued last
        if (STEADY || more) core::wait_vmcnt<G::NL>();
        else core::wait_vmcnt<0>();
      };
      auto phase_end = [&](bool wait) {
        __builtin_amdgcn_sched_barrier(0);
        if (wait) landed();
        core::lds_barrier();
        __builtin_amdgcn_sched_barrier(0);
      };
      if constexpr (NW == 8) {
        // A wave's loads of the next stage have landed before the barrier ahead of
        // group 0's first read of it (group 0: after its last products of this
        // stage; group 1: after its last reads of it).
        next_b(steady, 3);
        read(0, 0, 0);
        step_b(steady);
        phase_end(false);
        multiply(0);
        phase_end(false);
        next_a(steady, 4);
        read(0, 1, 0);
        step_a(steady);
        phase_end(grp == 1);
        multiply(0);
        phase_end(grp == 0);
      } else {
        window(steady, std::integral_constant<int, 0>(), false);
        // this wave's loads of the next stage have landed, and every wave has read
        // this one
        phase_end(true);
        window(steady, std::integral_constant<int, 1>(), hold);
      }
      if (!hold) a = past(a + 2 * G::SLOT);
    };
    // (a wait that the compiler sees: scalar loads left over from the epilogue would have
    // it wait for every LDS read in the loop)
    if constexpr (NW != 8) __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
    // Group 1 meets one barrier more before its phases, group 0 one after.
    if (NW == 8 && grp == 1) core::lds_barrier();
#pragma unroll
    for (int leg = 0; leg < LEGS; ++leg) {
      int s0, S, s = 0;
      stages(w.t, leg, s0, S);
      // the loaders are up to two stages ahead, in this leg
      const int steady = S - 3;
      if (steady > 0) {
        la.uniform();
        lb.uniform();
        for (; s < steady; ++s) stage(std::true_type(), false);
        na -= steady;
        nb -= steady;
      }
      const int rest = HOLD && leg == LEGS - 1 ? S - 1 : S;
      for (; s < rest; ++s) stage(std::false_type(), false);
    }
    if constexpr (HOLD) stage(std::false_type(), true);
    if (NW == 8 && grp == 0) core::lds_barrier();
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (NW == 8) {
      // the stage multiplied last lies in the two slots before a
      epilogue(w.t, acc, [&](int which) { return lds + past(a + (SLOTS - 2 + which) * G::SLOT); });
    } else {
      epilogue(w.t, acc, [&](int which) { return lds + past(a + which * G::SLOT); });
      if constexpr (HOLD) {
        core::lds_barrier();  // every wave is done with the idle slots
        next_b(std::false_type(), 0);
        step_b(std::false_type());
        a = past(a + 2 * G::SLOT);
      }
    }
  }
}

}  // namespace ring
}  // namespace ipttt
