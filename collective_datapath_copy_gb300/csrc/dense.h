// Dense operators: what the host dispatch (dense.cu) hands to the kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

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
  int32_t vec;       // 1: every array above has unit column stride, its rows start on 16 bytes
};

// out[b](m, n) = epilogue(sum over s of sum over k of A[b or s](m, k) B[s](n, k)).
//   nseg == 2: the sums of two products (A[0] B[0] + A[1] B[1]), one output
//   nbatch == 2: two products A[0] B[0] and A[1] B[0], two outputs
//   gated: g = A[0] B[0], u = A[0] B[1], one output
struct DenseJob {
  int64_t m, n, k;
  int32_t nseg, nbatch, gated;
  int32_t forward;  // 0: a gradient, kept to one kernel whichever others are asked for
  DenseMat a[2], b[2];
  DenseEpi e;
  int32_t *status;
};

// Column sums of row blocks still to be added, in order: db[c] = sum over b of part[b][c].
struct DenseJoin {
  const float *part;
  int64_t blocks, n;
  void *db;  // NULL: nothing to do
  int32_t type;
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
// dst[i * ld + j] = src(i, j): operands whose strides or base no tensor map takes, laid out in
// rows of whole 16-byte runs, all of a call's in one launch.
struct DensePack {
  DenseMat src[4];
  int64_t rows[4], cols[4], ld[4];
  unsigned ctas;  // for an operand (set at the launch)
  uint16_t *dst[4];
  int count;
};
int64_t dense_act_bwd_row_blocks(int64_t m, int64_t n, bool sums);
// Lays out `pack` in the same launch. With more than one row block, db is only complete after the
// join that `join` receives.
cudaError_t dense_act_bwd(const DenseActBwd &a, DensePack &pack, DenseJoin &join, cudaStream_t s);
cudaError_t dense_join(const DenseJoin &join, cudaStream_t s);
cudaError_t dense_pack(DensePack &p, cudaStream_t s);

// The job's epilogue over accumulators of zero (nothing to sum over).
cudaError_t dense_empty_sum(const DenseJob &j, cudaStream_t s);

// Launch a kernel that may be set up while its predecessor in the stream still runs. A call's first
// kernel waits for that (griddep_wait) before it touches memory, and every kernel waits before it ends.
// A later kernel of a call may read before its own wait what an earlier one of the call had waited for
// before it let its successor start (griddep_launch behind griddep_wait): the caller's arrays, or a plan
// made two kernels before.
template <typename... P, typename... A>
cudaError_t dense_launch(void (*kernel)(P...), dim3 grid, unsigned threads, uint32_t smem,
                         unsigned cluster, cudaStream_t s, A &&...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<A &&>(args)...);
}

// Shared memory past 48 KiB that a kernel may ask for: the runtime keeps the limit for each device,
// so it is set by the first launch on each (a stream capture then records the launch alone). One
// object for each kernel.
class DenseSmemLimit {
 public:
  cudaError_t operator()(const void *kernel, uint32_t bytes) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool kept = dev >= 0 && dev < kDevices;
    if (kept && set_[dev].load(std::memory_order_acquire)) return cudaSuccess;
    const cudaError_t r =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (r == cudaSuccess && kept) set_[dev].store(true, std::memory_order_release);
    return r;
  }

 private:
  static constexpr int kDevices = 64;
  std::atomic<bool> set_[kDevices] = {};
};

}  // namespace coll
