// Experts for a few tokens: what the host half (experts.cu) hands to the kernels.
#pragma once

#include "dense.h"
#include "dense_epi.cuh"

namespace coll {

// An inner value act(g) u as the sum of two numbers of the operands' type, off by 2^-16 of itself in bf16 and
// 2^-22 in f16: the sums' matrix instructions take 16 bits, and each weight that is read goes into both
// products. One number alone put the result 0.0019 to 0.0025 of its size off in bf16, where its own rounding is
// 0.0016 to 0.0017, and took 0 to 4 % less time (one token, 6 of 64 experts of 2048 x 176: 8.0 us, 8.1 with
// both; 128 of two, eight of 4096 x 14336 452, 463). What is infinite has no rest.
__device__ __forceinline__ void split_value(float v, int type, uint16_t &value, uint16_t &rest) {
  value = f2h(v, type);
  const float r = h2f(value, type);
  rest = fabsf(r) < INFINITY ? f2h(v - r, type) : (uint16_t)0;
}

constexpr int kExpertsMost = 1024;  // experts of a call
constexpr int kChosenMost = 32;     // choices of a token
constexpr int kExpertsGroup = 128;  // tokens that a launch takes

// The choices sorted by expert, in chunks of at most so many of one expert; each choice's token and
// weight in the order of the chunks.
struct ExpertsPlan {
  int32_t *chunks;   // their number
  int4 *chunk;       // {expert, first place, choices, the expert's first chunk | its chunks << 16}
  int32_t *token;
  float *weight;
};

// One to a few tokens of few choices (experts_direct.cu).
constexpr int kDirectChoices = 32;  // that a warp sorts by itself
constexpr int kDirectTokens = 32;

struct DirectParams {
  const uint16_t *w[2];  // gate and up, or down
  int64_t es[2], rs[2];
  const uint16_t *x;     // tokens, or the inner values in the order of the chunks
  int64_t x_ld;
  DenseMat ids, weights;
  int32_t first, experts, top, tokens;
  int32_t type, out_type, act;
  int32_t len;           // elements of a row of weights
  int32_t features;      // rows of weights of an expert
  int32_t x_align;       // inner: bytes that rows of x start on and are a multiple of
  uint16_t *h;           // inner: the output
  int64_t h_ld;
  int64_t rest;          // elements from an inner value to its rest
  uint32_t *counters;    // of the sums' tiles; the inner kernel sets them to 0
  int32_t tiles;
  void *y;               // sums: the output
  int64_t y_rs;
  DenseMat res;
  float *part;           // splits > 1: [split][tile][tokens][16]
  int32_t splits;
  uint32_t most_chunks, warps;
};

constexpr int kDirectInner = 8;   // inner features of a CTA
constexpr int kDirectOuter = 16;  // outputs of a CTA

// align: of the weights' rows, as x_align.
cudaError_t experts_direct_inner(const DirectParams &p, int align, cudaStream_t s);
cudaError_t experts_direct_outer(const DirectParams &p, int align, cudaStream_t s);

}  // namespace coll
