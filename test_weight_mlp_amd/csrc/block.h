// The rest of the block: arguments and launchers of the norm and of the
// projections, called by the C ABI layer.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

namespace ipttt {

struct Rows {             // [rows, columns] with a row stride in elements
  void* p;
  int64_t ld;
};

struct NormArgs {
  int dtype, dim;
  int64_t rows;
  bool center;            // layer norm
  float eps;
  Rows x, y;              // backward: y is unused
  const void *w, *b;
  Rows dy, dres, dx;
  float *dw, *db;
  float* part;            // [norm_parts, 2, dim]
};
hipError_t launch_norm(const NormArgs& a, hipStream_t st);
// Partial weight gradients of the backward.
int norm_parts(int dtype, int64_t rows, int dim);
hipError_t launch_norm_backward(const NormArgs& a, hipStream_t st);

// C[m, n] = sum_k A[m, k] B[n, k] with the projection's epilogue (which takes K
// contiguous in B).  A and B are
// row-major with K contiguous, or (a_kmaj, b_kmaj) K-major: A[m, k] at
// a.p[k * a.ld + m].
struct GemmArgs {
  int dtype;
  int64_t M, N, K;
  Rows a, b, c;
  int a_kmaj, b_kmaj;
  // A second pair of operands of the same sizes and strides, C = A B + A2 B2, or a
  // second product, C = A B and C2 = A2 B, in one launch.
  int two_pairs, two_products;
  Rows a2, b2, c2;
  int c_f32;              // C is float (else dtype)
  int act;                // ipttt_act
  const void* bias;       // [N] dtype, or NULL
  Rows res, pre;          // p NULL: none
  float* part;            // partial products where K is cut (gemm_workspace)
};
size_t gemm_workspace(const GemmArgs& g);
hipError_t launch_gemm(const GemmArgs& g, hipStream_t st);
// Two products that do not depend on each other, g with B K-major and h with both
// (dx and dW of a projection), each with its own part: in one launch where both are of
// small tiles.  One whose c is NULL is left out; the other has the same bits as with it.
void gemm_pair_workspace(const GemmArgs& g, const GemmArgs& h, size_t* of_g, size_t* of_h);
hipError_t launch_gemm_pair(const GemmArgs& g, const GemmArgs& h, hipStream_t st);

// dp = dy act'(pre) and db (each optional), in one pass over dy.
struct ActGradArgs {
  int dtype, act;
  int64_t rows, dim;
  Rows dy, pre, dp;       // dp.p NULL: not written
  float* db;
  float* part;            // [act_grad_parts, dim], where db is wanted
};
int act_grad_parts(int64_t rows, int64_t dim);
hipError_t launch_act_grad(const ActGradArgs& a, hipStream_t st);

}  // namespace ipttt
