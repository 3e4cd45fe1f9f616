// Experts for a few tokens: what the host half (experts.cu) hands to the kernels.
#pragma once

#include "dense.h"

namespace coll {

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
  int32_t x_align;       // bytes that rows of x start on and are a multiple of
  uint16_t *h;           // inner: the output
  int64_t h_ld;
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
