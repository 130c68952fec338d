// Attention: the plan's items and the launchers the C ABI layer calls.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

namespace ipttt {
namespace attn {

// Tile sizes the plan cuts sequences into.  Rows are the flat (query, head of
// the group) rows of one key head: row r is query r / G, head r % G of the group.
constexpr int kRows = 128;      // rows of a forward tile, and of a dQ tile
constexpr int kKeys = 64;       // keys of one step
constexpr int kFewRows = 32;    // most rows of a sequence that the kernel of few rows takes, in one tile
constexpr int kPartRows = 32;   // rows of a slot of partial results (a forward tile takes kRows / kPartRows of them)
constexpr int kBwdKeys = 128;   // keys of a dK, dV tile
constexpr int kBwdRows = 32;    // rows of one step of it
constexpr int kShortKeys = 32;  // most keys of a sequence whose bf16 gradients take P and dS in two terms

// One forward (or dQ) tile: rows [r0, min(r0 + tile rows, q_len * G)) of one
// sequence over keys [k_begin, k_end) of it.  Query t sees keys below off + t + 1.
struct RowItem {
  int32_t q_start, q_len, r0;
  int32_t k_start, off;      // off = k_len - q_len
  int32_t k_begin, k_end;
  int32_t part;              // -1: the whole of the rows' keys; else the slot of this partial result
};

// The n partial results of one forward tile, in slots part, part + step, ...
struct JoinItem {
  int32_t q_start, q_len, r0, part, n, step;
};

// One dK, dV tile: keys [key0, min(key0 + kBwdKeys, k_len)) of one sequence
// against its rows [r_begin, r_end), both whole steps of kBwdRows but for the last.
struct KeyItem {
  int32_t q_start, q_len, r_begin, r_end;
  int32_t k_start, off, key0;
  int32_t part;              // -1: all rows that see the keys; else the slot of this partial result
};

// The partial results of one dK, dV tile, slots [part, part + n), for the
// n_keys rows of dK and dV from k_row on.
struct KeyJoin {
  int32_t k_row, n_keys, part, n;
};

// What the plan table starts with; the items follow at these offsets (bytes).
struct PlanHeader {
  int32_t magic, dtype, heads, kv_heads, head_dim, n_seqs;
  int32_t q_rows, k_rows;
  int32_t n_rows, n_join, n_dq, n_key;
  int32_t o_rows, o_join, o_dq, o_key;
  int32_t parts, overlap;    // partial slots; whether two sequences share keys
  int32_t bytes;
  int32_t n_key_join, o_key_join, key_parts;
  int32_t n_few, o_few;      // items of the kernel of few rows
  int32_t join_rows;         // most rows of a joined tile
  int32_t n_tiles, o_tiles;  // tiles of rows, uncut
  int32_t n_dq_join, o_dq_join, dq_parts;
  int32_t rows_cut;          // whether tiles of many rows are cut into parts
  int32_t shorts;            // whether a sequence with queries has at most kShortKeys keys
};
static_assert(sizeof(PlanHeader) == 128, "plan header");
constexpr int32_t kMagic = 0x41545031;

struct View {             // [rows, heads, D] with element strides
  void* p;
  int64_t row, head;
};

struct Args {
  int dtype, heads, kv_heads, G, D;
  float scale;
  bool shorts;            // sequences of at most kShortKeys keys are among those of the backward
  const void *items, *dq_items;  // device
  int n_items, n_dq;
  bool cut;               // tiles of the forward are cut into parts
  View q, k, v, o, dO, dq, dk, dv;
  float *lse;             // [q rows, heads]
  float *nlse, *ndelta;   // same: what is added to the scores (-inf on rows that see nothing), -delta
  float *part_o, *part_lse, *part_dq;
};

hipError_t launch_forward(const Args& a, hipStream_t st);
hipError_t launch_few(const Args& a, hipStream_t st);
hipError_t launch_join(const Args& a, const void* items, int n, int rows, hipStream_t st);
hipError_t launch_delta(const Args& a, hipStream_t st);
hipError_t launch_backward(const Args& a, hipStream_t st);
hipError_t launch_join_backward(const Args& a, const void* dq_items, int n_dq, const void* key_items, int n_key,
                                hipStream_t st);

}  // namespace attn

struct QkArgs {
  int dtype, heads, kv_heads, D;
  int64_t tokens, table_rows, out_rows;
  float eps;
  attn::View q, k, v, q_out, k_out, v_out;   // backward: q_out, k_out are the cotangents
  attn::View dq, dk;
  const void *w_q, *w_k;
  const int32_t *pos, *rows;
  const float* table;
  float *dw_q, *dw_k, *part;
};
constexpr int kQkParts = 512;   // partial weight gradients of the backward
hipError_t launch_qk(const QkArgs& a, hipStream_t st);
hipError_t launch_qk_backward(const QkArgs& a, hipStream_t st);

}  // namespace ipttt
