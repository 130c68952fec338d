// Shared device helpers of the attention kernels (gfx950): one source for
// bf16 and fp32, built on 32x32 MFMA blocks.
//
// A head row is DP elements (head_dim padded with zeros to 64 or 128), RB =
// DP * sizeof(T) bytes, in LDS as RB / 16 chunks of 16 bytes.  One chunk is one
// lane's part of an operand that contracts over head_dim: lane l supplies
// chunk 2 s + l / 32 of row l % 32 for step s (bf16: one 32x32x16 MFMA; fp32:
// four 32x32x2 MFMAs, whose K order inside the step is permuted alike in both
// operands).
//
// The same tiles are read transposed for products that contract over rows
// (keys or queries).  The C block of a 32x32 MFMA holds, in lane l, column
// l % 32 and rows 8 (i / 4) + 4 (l / 32) + i % 4 for register i.  Used as the
// B operand of the next product, registers [EPL j, EPL j + EPL) are one
// step's fragment if the A operand takes its rows in the same order, so the
// probabilities never leave their registers: no LDS trip, no lane exchange.
#pragma once

#include "attn.h"
#include "common.h"

namespace ipttt {
namespace attn {

typedef __attribute__((address_space(3))) void* lds_ptr_t;
typedef __attribute__((address_space(3))) short4_t* lds_s4_t;

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr uint32_t kOob = 0x80000000u;        // a buffer offset past every resource's end: reads as zero
constexpr int64_t kMaxBytes = 0x7FFFFFF0LL;   // a resource's largest size

template <typename T> struct Elt;
template <> struct Elt<bf16> {
  static constexpr int EPL = 8;  // elements of a 16-byte chunk
  typedef bf16x8 frag;
  static __device__ __forceinline__ floatx16 mma(frag a, frag b, floatx16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
};
template <> struct Elt<float> {
  static constexpr int EPL = 4;
  typedef float4_t frag;
  static __device__ __forceinline__ floatx16 mma(frag a, frag b, floatx16 c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[i], b[i], c, 0, 0, 0);
    return c;
  }
};

// A tile of rows in LDS.  A 1 KB block, the 64 lanes' 16 bytes of one direct
// load, holds RPI rows; blocks follow at PITCH = 1024 + 16 (or 32) bytes.  In a
// block the rows alternate in units of 64 bytes (fp32 of width 128: 128 bytes),
// so that whatever step of head_dim, block of columns or group of rows a
// fragment takes only adds a constant: each kind of read has one address per
// lane and immediate offsets.  Free of bank conflicts (64 banks of 4 bytes) for
// the 16 lanes of a 16-byte read, one chunk of 16 rows each, and the 32 lanes
// of a transposed read, 64 bytes of 4 rows.
template <typename T, int DP>
struct Tile {
  static constexpr int RB = DP * (int)sizeof(T);
  static constexpr int STEPS = RB / 32;  // MFMA steps over head_dim
  static constexpr int RPI = 1024 / RB;  // rows of a block
  static constexpr int PITCH = RB == 128 ? 1056 : 1040;
  typedef typename Elt<T>::frag frag;
  static constexpr int bytes(int rows) { return rows / RPI * PITCH; }

  // Row and chunk that lane l's 16 bytes of a block hold.
  static __device__ __forceinline__ void source(int l, int* row, int* chunk) {
    if constexpr (RB == 512) {
      *row = (l >> 3) & 1;
      *chunk = 8 * (l >> 4) + (l & 7);
    } else if constexpr (RB == 256) {
      *row = (l >> 2) & 3;
      *chunk = 4 * (l >> 4) + (l & 3);
    } else {  // rows i and i + 4 share banks: their chunks 0, 1 (and 2, 3) change places
      *row = (l >> 2) & 7;
      *chunk = 4 * (l >> 5) + ((l & 3) ^ (*row >> 2));
    }
  }

  // Chunk 2 q + lane / 32 of row r0 + lane % 32, r0 a multiple of 32: a lane's
  // fragment of an operand contracted over head_dim.
  static __device__ __forceinline__ int row_base(int lane) {
    const int r = lane & 31, h = lane >> 5, i = r % RPI, at = r / RPI * PITCH;
    if constexpr (RB == 512) return at + 128 * i + 16 * h;
    if constexpr (RB == 256) return at + 64 * i + 16 * h;
    return at + 64 * i + 16 * (h ^ (i >> 2));
  }
  static constexpr int row_step(int q) {
    return RB == 512 ? 256 * (q >> 2) + 32 * (q & 3) : (RB == 256 ? 256 : 512) * (q >> 1) + 32 * (q & 1);
  }
  static __device__ __forceinline__ frag row(const char* t, int base, int r0, int q) {
    return *reinterpret_cast<const frag*>(t + base + r0 / RPI * PITCH + row_step(q));
  }

  // Fragment of the tile transposed, columns (head_dim) 32 db + lane % 32 as
  // the A rows, contracted over EPL rows (a C block's order) from r0, a
  // multiple of 2 EPL.
  static __device__ __forceinline__ int col_base(int lane) {
    const int h = lane >> 5;
    if constexpr (sizeof(T) == 2) {
      const int r = (lane >> 2) & 3, c = 2 * ((lane >> 4) & 1) + ((lane >> 1) & 1), b = 8 * (lane & 1);
      return RB == 256 ? h * PITCH + 64 * r + 16 * c + b : 64 * (4 * h + r) + 16 * (c ^ h) + b;
    } else {
      const int d = lane & 31;
      return RB == 512 ? 2 * h * PITCH + 4 * d : h * PITCH + 256 * (d >> 4) + 4 * (d & 15);
    }
  }
  static __device__ __forceinline__ frag col(const char* t, int base, int r0, int db) {
    const char* at = t + base + r0 / RPI * PITCH;
    if constexpr (sizeof(T) == 2) {
      at += (RB == 256 ? 256 : 512) * db;
      const short4_t x0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4_t)at);
      const short4_t x1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4_t)(at + 8 / RPI * PITCH));
      return __builtin_bit_cast(bf16x8, __builtin_shufflevector(x0, x1, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      frag x;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[i] = *reinterpret_cast<const float*>(RB == 512 ? at + 256 * db + (i >> 1) * PITCH + 128 * (i & 1)
                                                         : at + 512 * db + 64 * i);
      return x;
    }
  }
};

// Where this lane reads in any tile.
template <typename T, int DP>
struct At {
  int row, col;
  __device__ __forceinline__ explicit At(int lane)
      : row(Tile<T, DP>::row_base(lane)), col(Tile<T, DP>::col_base(lane)) {}
};

// One group of four row fragments (A operands contracted over head_dim), or of
// transposed ones (contracted over EPL rows each, DB blocks of head_dim).
template <typename T, int DP>
struct Groups {
  typedef Tile<T, DP> TL;
  typedef typename Elt<T>::frag frag;
  static constexpr int EPL = Elt<T>::EPL, DB = DP / 32, H = TL::STEPS / 4, NP = 16 / EPL;
  static_assert(NP * DB == 4 * H, "equal groups");
  static __device__ __forceinline__ void rows(const char* t, const At<T, DP>& at, int r0, int g, frag (&f)[4]) {
#pragma unroll
    for (int x = 0; x < 4; ++x) f[x] = TL::row(t, at.row, r0, 4 * g + x);
  }
  static __device__ __forceinline__ void cols(const char* t, const At<T, DP>& at, int r0, int g, frag (&f)[4]) {
#pragma unroll
    for (int x = 0; x < 4; ++x) f[x] = TL::col(t, at.col, r0 + 2 * EPL * ((4 * g + x) / DB), (4 * g + x) % DB);
  }
};

__device__ __forceinline__ void fill16(floatx16& x, float v) {
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = v;
}

// The same for a value that a loop does not change: without the empty asm the
// compiler keeps 16 copies of it in registers for the whole loop.
__device__ __forceinline__ void start16(floatx16& x, float v) {
  asm volatile("" : "+v"(v));
  fill16(x, v);
}

// EPL registers of a C block, from register i0, as a B fragment (bf16: rounded
// to nearest even, the one rounding of a probability or its gradient).
template <typename T>
__device__ __forceinline__ typename Elt<T>::frag pack(const floatx16& x, int i0) {
  typename Elt<T>::frag p;
#pragma unroll
  for (int i = 0; i < Elt<T>::EPL; ++i) p[i] = (T)x[i0 + i];
  return p;
}

// max and sum over lanes l and l ^ 32, in both
__device__ __forceinline__ void both_halves(float x, float* lo, float* hi) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  *lo = __builtin_bit_cast(float, (uint32_t)r[0]);
  *hi = __builtin_bit_cast(float, (uint32_t)r[1]);
}
__device__ __forceinline__ float half_max(float x) {
  float a, b;
  both_halves(x, &a, &b);
  return fmaxf(a, b);
}
__device__ __forceinline__ float half_sum(float x) {
  float a, b;
  both_halves(x, &a, &b);
  return a + b;
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const void* p, int64_t bytes) {
  const int n = (int)(bytes < 0 ? 0 : bytes > kMaxBytes ? kMaxBytes : bytes);
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, n, 0x00020000);
}

// Rows of one head streamed into LDS tiles of R rows, NW waves sharing each:
// 16 bytes a lane straight to LDS.  The resource is set to the tile's first row
// with 64-bit arithmetic, so that offsets inside it are 32-bit however long the
// cache; rows past the sequence's end and columns past D read as zero.
template <typename T, int DP, int NW, int R>
struct RowStream {
  typedef Tile<T, DP> TL;
  static constexpr int N = R / (NW * TL::RPI);  // loads per wave and tile
  static_assert(R % (NW * TL::RPI) == 0, "rows per wave");
  uint32_t off[N];
  uint32_t stride;  // bytes
  int tail;         // bytes of one row

  __device__ __forceinline__ RowStream(int64_t row_stride, int D, int wave, int lane)
      : stride((uint32_t)(row_stride * (int)sizeof(T))), tail(D * (int)sizeof(T)) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      int r, c;
      TL::source(lane, &r, &c);
      r += (wave * N + j) * TL::RPI;
      off[j] = c * 16 < tail ? (uint32_t)r * stride + (uint32_t)c * 16u : kOob;
    }
  }
  // tile <- rows [row, row + min(R, left)) of the head at base; left >= 1
  __device__ __forceinline__ void issue(const char* base, int64_t row, int left, char* tile, int wave) const {
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char*>(base + row * (int64_t)stride), (short)0, (min(left, R) - 1) * (int)stride + tail, 0x00020000);
#pragma unroll
    for (int j = 0; j < N; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr_t)(tile + (wave * N + j) * TL::PITCH), 16, off[j], 0, 0, 0);
  }
};

// What that rounding left of them, rounded in turn.
template <typename T>
__device__ __forceinline__ typename Elt<T>::frag rest(const floatx16& x, int i0, const typename Elt<T>::frag& p) {
  typename Elt<T>::frag r;
#pragma unroll
  for (int i = 0; i < Elt<T>::EPL; ++i) r[i] = (T)(x[i0 + i] - (float)p[i]);
  return r;
}

// Waits until at most N of this wave's vector-memory operations are pending.
template <int N>
__device__ __forceinline__ void loads_pending() {
  static_assert(N < 64, "vmcnt");
  __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
  asm volatile("" ::: "memory");
}

// Waits until every LDS read of this wave has returned.
__device__ __forceinline__ void reads_done() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// Row i of the partial results in slot part: slots hold kPartRows rows of every
// key head.
__device__ __forceinline__ int64_t part_row(int part, int kv_heads, int kvh, int i) {
  return ((int64_t)(part + i / kPartRows) * kv_heads + kvh) * kPartRows + i % kPartRows;
}

// Workgroup barrier after this wave's own loads to LDS have landed.
__device__ __forceinline__ void tiles_landed() {
  loads_pending<0>();
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// A lane's chunks of one row in global memory, its byte offset in the resource
// given (kOob: no row); zeros where it has none.
template <typename T, int DP>
__device__ __forceinline__ void row_frags(__amdgpu_buffer_rsrc_t rs, uint32_t off, int D, int h,
                                          typename Elt<T>::frag (&f)[Tile<T, DP>::STEPS]) {
#pragma unroll
  for (int s = 0; s < Tile<T, DP>::STEPS; ++s) {
    const uint32_t at = (uint32_t)(2 * s + h) * 16u;
    f[s] = __builtin_bit_cast(typename Elt<T>::frag,
                              __builtin_amdgcn_raw_buffer_load_b128(
                                  rs, at < (uint32_t)D * sizeof(T) && off != kOob ? off + at : kOob, 0, 0));
  }
}

// 4 consecutive elements from registers, rounded once.
template <typename T>
__device__ __forceinline__ void store4(T* p, float a, float b, float c, float d) {
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4_t*>(p) = float4_t{a, b, c, d};
  } else {
    *reinterpret_cast<bf16x4*>(p) = bf16x4{(bf16)a, (bf16)b, (bf16)c, (bf16)d};
  }
}

// Rows of a group's query tile: flat row r of a sequence is query t = r / G of
// head kvh * G + r % G.  All rows of a tile derive from the tile's first row
// (one scalar division), so that the per-lane division is of a small number:
// n * m >> 32 with m = ceil(2^32 / G) is exact while n * G < 2^32.
struct RowMap {
  int t0, g0;
  uint32_t m;
  int G;
  __device__ __forceinline__ RowMap(int r0, int group) : G(group) {
    t0 = r0 / group;
    g0 = r0 - t0 * group;
    m = group == 1 ? 0u : (uint32_t)(0xFFFFFFFFu / (uint32_t)group) + 1u;
  }
  // row r0 + i: its query relative to t0, and its head in the group
  __device__ __forceinline__ void of(int i, int* t, int* g) const {
    const int n = g0 + i;
    *t = G == 1 ? n : (int)__umulhi((uint32_t)n, m);
    *g = n - *t * G;
  }
};

// One lane's row of a tile, and what its wave's rows see.
struct Row {
  int r, t, g;      // flat row, query, head of the group
  bool live;
  int lim;          // it sees keys below lim
  int all, any;     // every row of the wave sees the keys below all, none those from any on
  int t0;           // the wave's first query

  __device__ __forceinline__ Row(const RowItem& it, int G, int wave, int lane) {
    const int n_rows = it.q_len * G, r0 = it.r0 + wave * 32;
    const RowMap rm(r0, G);
    t0 = rm.t0;
    r = r0 + (lane & 31);
    rm.of(lane & 31, &t, &g);
    t += rm.t0;
    live = r < n_rows;
    lim = live ? min(it.off + t + 1, it.k_end) : 0;
    all = __builtin_amdgcn_readfirstlane(min(it.off + rm.t0 + 1, it.k_end));
    any = __builtin_amdgcn_readfirstlane(
        r0 < n_rows ? max(0, min(it.off + min(r0 + 31, n_rows - 1) / G + 1, it.k_end)) : 0);
  }
};

// This lane's chunks of its row of a [rows, heads, D] tensor: the resource
// starts at the wave's first query, so that offsets are 32-bit.
template <typename T, int DP>
__device__ __forceinline__ void row_frags(const View& v, const RowItem& it, const Row& row, int kvh, int G, int D, int h,
                                          typename Elt<T>::frag (&f)[Tile<T, DP>::STEPS]) {
  constexpr int ES = sizeof(T);
  const char* base = static_cast<const char*>(v.p) +
                     ((it.q_start + (int64_t)row.t0) * v.row + (int64_t)kvh * G * v.head) * ES;
  const uint32_t off = (uint32_t)((row.t - row.t0) * (int)v.row + row.g * (int)v.head) * ES;
  row_frags<T, DP>(rsrc_of(base, kMaxBytes), row.live ? off : kOob, D, h, f);
}

}  // namespace attn
}  // namespace ipttt
