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

// Tile of R rows of RB bytes.  Chunk c of row r sits in slot c ^ f(r): the 16
// rows that 16 neighbouring lanes read with one chunk index fall on 16
// distinct bank quads (64 banks of 4 bytes), and so do the rows of a transposed
// read (bf16: 4 rows of 64 bytes; fp32: rows r and r + 4 of 128 bytes).
template <typename T, int DP>
struct Tile {
  static constexpr int RB = DP * (int)sizeof(T);
  static constexpr int SLOTS = RB / 16;
  static constexpr int STEPS = RB / 32;       // MFMA steps over head_dim
  static constexpr int RPI = 1024 / RB;       // rows of one wave-wide 16-byte load
  typedef typename Elt<T>::frag frag;

  static __device__ __forceinline__ int f(int r) {
    if constexpr (sizeof(T) == 4) return ((r & 7) << 1) | ((r >> 3) & 1);
    if constexpr (RB == 256) return ((r & 3) << 2) | ((r >> 2) & 3);
    return (((r >> 1) & 1) << 2) | ((r >> 2) & 3);  // RB 128: two rows per 256 bytes
  }
  static __device__ __forceinline__ int at(int r, int c) { return r * RB + ((c ^ f(r)) << 4); }

  // Chunk c of row r: a lane's fragment of an operand contracted over head_dim.
  static __device__ __forceinline__ frag row(const char* t, int r, int c) {
    return *reinterpret_cast<const frag*>(t + at(r, c));
  }

  // Fragment of the tile transposed, columns (head_dim) 32 db + lane % 32 as
  // the A rows, contracted over EPL rows of the tile from row0 in the C
  // block's order.
  static __device__ __forceinline__ frag col(const char* t, int row0, int db, int lane) {
    const int h = lane >> 5;
    if constexpr (sizeof(T) == 2) {
      const int r = row0 + 4 * h + ((lane >> 2) & 3), c = 4 * db + 2 * ((lane >> 4) & 1) + ((lane >> 1) & 1);
      const int b = 8 * (lane & 1);
      const short4_t x0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4_t)(t + at(r, c) + b));
      const short4_t x1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4_t)(t + at(r + 8, c) + b));
      return __builtin_bit_cast(bf16x8, __builtin_shufflevector(x0, x1, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      const int d = lane & 31, c = 8 * db + (d >> 2), b = 4 * (d & 3);
      frag x;
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float*>(t + at(row0 + 4 * h + i, c) + b);
      return x;
    }
  }
};

// EPL registers of a C block, from register i0, as a B fragment (bf16: rounded
// to nearest even, the one rounding of a probability or its gradient).
template <typename T>
__device__ __forceinline__ typename Elt<T>::frag pack(const floatx16& x, int i0) {
  typename Elt<T>::frag p;
#pragma unroll
  for (int i = 0; i < Elt<T>::EPL; ++i) p[i] = (T)x[i0 + i];
  return p;
}

__device__ __forceinline__ float other_half(float x) { return __shfl_xor(x, 32, 64); }

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const void* p, int64_t bytes) {
  const int n = (int)(bytes < 0 ? 0 : bytes > kMaxBytes ? kMaxBytes : bytes);
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, n, 0x00020000);
}

// Direct-to-LDS copy of R rows of one head into a tile, NW waves sharing it:
// row r of the resource at r * stride; rows past its end and columns past D
// read as zero.
template <typename T, int DP, int NW, int R>
__device__ __forceinline__ void load_rows(__amdgpu_buffer_rsrc_t rs, uint32_t stride, int D, char* tile, int wave,
                                          int lane) {
  typedef Tile<T, DP> TL;
  constexpr int PER_WAVE = R / (NW * TL::RPI);
  static_assert(R % (NW * TL::RPI) == 0, "rows per wave");
#pragma unroll
  for (int j = 0; j < PER_WAVE; ++j) {
    const int blk = wave * PER_WAVE + j;
    const int r = blk * TL::RPI + lane / TL::SLOTS;
    const int c = (lane % TL::SLOTS) ^ TL::f(r);
    const uint32_t off = c * 16 < D * (int)sizeof(T) ? (uint32_t)r * stride + (uint32_t)c * 16u : kOob;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr_t)(tile + blk * 1024), 16, off, 0, 0, 0);
  }
}

// A lane's chunks of one row in global memory (zeros where it has none).
template <typename T, int DP>
__device__ __forceinline__ void row_frags(const char* row, bool live, int D, int h,
                                          typename Elt<T>::frag (&f)[Tile<T, DP>::STEPS]) {
#pragma unroll
  for (int s = 0; s < Tile<T, DP>::STEPS; ++s) {
    const int c = 2 * s + h;
#pragma unroll
    for (int e = 0; e < Elt<T>::EPL; ++e) f[s][e] = (T)0.0f;
    if (live && c * 16 < D * (int)sizeof(T)) f[s] = *reinterpret_cast<const typename Elt<T>::frag*>(row + c * 16);
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

}  // namespace attn
}  // namespace ipttt
