// Launch interface of the tensor-core products (dense_tc.cu).
#pragma once

#include <cuda.h>  // CUtensorMap (the type only; maps are encoded through the runtime)
#include <cudaTypedefs.h>

#include "dense.h"

namespace coll {

constexpr uint32_t kSms = 152;            // multiprocessors of a GB300: what shapes are chosen for
constexpr uint32_t kTcSmem = 226 * 1024;  // dynamic shared memory a CTA may ask for

// One product of a launch.
struct TcProb {
  CUtensorMap a[2], b[2];
  DenseEpi e;
  int64_t m, n;
  uint32_t tiles_m, tiles_n, tiles;
  int32_t tile_cols;         // of the output
  int32_t a_rows;            // rows of A a CTA loads: 128, or all there are
  int32_t b_rows, b_chunks;  // rows of B per CTA and operand, and 64-row chunks of them
  int32_t b_box;             // rows of B a CTA loads (k contiguous): b_rows, or all there are
  int32_t kblocks, nseg, nbatch;
  int32_t split;             // shares of k, each with its own tiles
  float *part;               // split > 1: their sums, [share][batch][gate, up][m][part_ld]
  int64_t part_ld;
  uint32_t idesc;
  int32_t a_mn[2], b_mn[2];  // 1: the operand's rows (not k) are contiguous
};

struct TcParams {
  TcProb prob[2];  // the second's tiles may be 0
  DenseJoin join;
  int32_t *status;
  uint32_t even;   // turns of the second product's tiles that only go to the clusters with one
                   // tile of the first product less
  uint32_t stages, stage_bytes;
};

// An operand as the tensor maps take it: rows x k, k contiguous (mn == 0) or rows contiguous.
struct TcOperand {
  const void *p;
  int64_t rows, k, ld;  // ld: elements between the lines of the contiguous axis, a multiple of 8
  int32_t mn;
};

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

// Map of an operand in boxes of 64 of k by `rows` rows (k contiguous) or 64 rows by 64 of k.
int tc_encode(CUtensorMap *map, const TcOperand &o, int64_t type, uint32_t rows);

// A job with its operands: a[nseg or nbatch], b[nseg, or 2 when gated].
struct TcJob {
  const DenseJob *j;
  TcOperand a[2], b[2];
};

// The shapes of `p` for one or two jobs (two: neither gated); part_bytes: room for each job's
// shares, 0 where k is not split. Makes no device call.
int tc_plan(TcParams &p, const TcJob *jobs, int count, uint64_t (&part_bytes)[2]);
// Tensor maps and the kernel's shared memory: what may be refused, before anything of the call is
// launched.
int tc_prepare(TcParams &p, const TcJob *jobs, int count);
// The launch (p.prob[i].part and p.join are set by now); the shares of split jobs join in a second
// one.
cudaError_t tc_run(const TcParams &p, const TcJob *jobs, int count, cudaStream_t s);


// A small batch against many output features (dense_skinny.cu): the weights are the 128-row
// operand, the m tokens its columns.
constexpr int64_t kSkinnyMost = 64;           // tokens
constexpr int64_t kSkinnyLeast = 64 * kSms;   // output features: 64 for every SM

struct SkinnyParams {
  CUtensorMap w[2], x;
  DenseEpi e;
  int64_t m, n;
  int32_t *status;
  int32_t rows, cols;          // output features of a CTA; tokens, rounded up to 16
  int32_t w_chunks, x_chunks;  // 64-row chunks of them
  int32_t kblocks, stages, w_mn, x_mn;
  uint32_t tiles;
  uint32_t w_bytes, stage_bytes, smem, idesc, tmem_cols;
};

// Shapes, tensor maps and shared memory: nothing is refused after it.
int skinny_plan(SkinnyParams &p, const DenseJob &j, const TcOperand *w, const TcOperand &x);
cudaError_t skinny_run(const SkinnyParams &p, bool gated, cudaStream_t s);


// One to a few tokens (dense_gemv.cu): A and B with unit stride along k, any row strides.
constexpr int64_t kGemvMost = 64;

struct GemvParams {
  const void *w[2], *x;
  int64_t ld[2], x_ld;
  DenseEpi e;
  int64_t m, n, k;
  uint32_t warps;
  int32_t x_align;  // what the rows of x start on; the weights' is the kernel's
};

cudaError_t gemv_run(const DenseJob &j, cudaStream_t s);

// The same with B's rows contiguous instead, up to 16 tokens.
constexpr int64_t kGemvTMost = 16;

struct GemvTParams {
  const void *w[2], *x;
  int64_t ld[2], x_ld;
  DenseEpi e;
  int64_t m, n, k;
  int32_t x_align;
};

cudaError_t gemv_t_run(const DenseJob &j, cudaStream_t s);

}  // namespace coll
