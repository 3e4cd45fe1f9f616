// Dense operators: what the host dispatch (dense.cu) hands to the kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "coll.h"

namespace coll {

// Element (i, j) at p + i * rs + j * cs elements.
struct DenseMat {
  const void *p;
  int64_t rs, cs;
};

// What happens to a finished accumulator. One product: z = acc + bias, y = act(z) + residual,
// z kept in `pre`. Gated: h = act(g) u, g and u kept in `gate` and `up`.
struct DenseEpi {
  void *out[2];       // per batch
  int64_t out_rs[2];
  void *pre;
  int64_t pre_rs;
  void *gate, *up;
  int64_t gate_rs, up_rs;
  const void *bias;
  int64_t bias_stride;
  const void *res;
  int64_t res_rs, res_cs;
  int32_t type;      // COLL_BF16 / COLL_F16: bias, pre, gate, up
  int32_t out_type;  // type or COLL_F32: out, residual
  int32_t act;
  int32_t vec;       // 1: every array above has unit column stride, and its rows start on
                     // 32-byte boundaries
};

// out[b](m, n) = epilogue(sum over s of sum over k of A[b or s](m, k) B[s](n, k)).
//   nseg == 2: the sums of two products (A[0] B[0] + A[1] B[1]), one output
//   nbatch == 2: two products A[0] B[0] and A[1] B[0], two outputs
//   gated: g = A[0] B[0], u = A[0] B[1], one output
struct DenseJob {
  int64_t m, n, k;
  int32_t nseg, nbatch, gated, pad;
  DenseMat a[2], b[2];
  DenseEpi e;
  int32_t *status;
};

// Elementwise parts of the backward calls (dense_aux.cu).
struct DenseActBwd {
  int64_t m, n;
  DenseMat dy, pre, up;  // up: gated only
  void *dz, *du;         // [m][ld]; may be NULL when only db is wanted
  int64_t ld;
  void *db;              // NULL: no column sums
  float *part;           // column sums of each row block, [row_blocks][n]
  int32_t type, db_type, act, gated;
};
int64_t dense_act_bwd_row_blocks(int64_t m, int64_t n);
cudaError_t dense_act_bwd(const DenseActBwd &a, cudaStream_t s);


// dst[i * ld + j] = src(i, j): an operand whose strides or base no tensor map takes, laid out in
// rows of whole 16-byte runs.
cudaError_t dense_pack(const DenseMat &src, int64_t rows, int64_t cols, void *dst, int64_t ld,
                       cudaStream_t s);

// The job's epilogue over accumulators of zero (nothing to sum over).
cudaError_t dense_empty_sum(const DenseJob &j, cudaStream_t s);

}  // namespace coll
