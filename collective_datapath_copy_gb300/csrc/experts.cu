// A few tokens through their chosen gated experts: C ABI (include/coll.h) and kernels.
//
//   h_ij = act(gate_e x_i) (up_e x_i),  y_i = residual_i + sum over j of weights_ij down_e h_ij,
//   e = ids_ij - first
//
// Bound by HBM: the weights of every chosen expert are read once, 4 f k + 2 n f bytes each, and a token
// or a few an expert multiply them. Up to 32 choices go to experts_direct.cu. Here the weights are the
// 128-row operand of tcgen05 and an expert's tokens its columns: product_kernel<true> computes the
// inner values, product_kernel<false> the sums. Both are persistent, a CTA an SM, and share their work
// to the k block: the list of (expert, tile of 128 features) is one line of k blocks that is cut into
// 152 equal lengths, because whole tiles would leave SMs idle (8 experts of 2048 inner features are
// 128 tiles). The shares of a tile that was cut join in a launch behind, in the order of k: nothing
// waits, and results do not depend on timing. Measured: 128 tokens of two, eight experts of 4096 x 14336
// (2.8 GB) 463 us, 6.1 TB/s; 32 tokens of eight out of 256, 32 of these experts here, of 7168 x 2048,
// 281 us, 6.4 TB/s; 17 to 128 tokens over weights of some MB 21 to 27 us, which is the chain of the
// launches: plan 2 us, first weights 3, inner values, join 4, sums, join 4.
//
// The sums' columns are inner values and their rests, 16 of each in turn: one tensor copy brings both (two,
// 33 tokens of two, eight experts of 1024 x 512: 21.9 us, 21.0 so) and one matrix instruction takes them.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "dense.h"
#include "dense_check.h"
#include "dense_direct.cuh"
#include "dense_epi.cuh"
#include "dense_tc.h"
#include "experts.h"
#include "tcgen05.cuh"

namespace coll {
namespace {

// ---------------------------------------------------------------- choices sorted by expert

constexpr int kTileK = 64;
constexpr int kPlanThreads = 1024;

// Where the choices come from.
struct Choices {
  DenseMat ids, weights;
  int32_t tokens, top, experts, first, cols;
};

// The plan of up to TURNS choices a thread, by all threads of the CTA; the number of chunks. The
// choices go through the CTA 32 at a time, a warp after the other, each adding to its experts'
// counts: so they stay in order, and the plan does not depend on timing. base: a word an expert.
template <int TURNS>
__device__ __forceinline__ int make_plan(const Choices &p, int4 *chunk, int32_t *tokens,
                                         float *weights, uint32_t *base, uint32_t *sums) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  const int n = p.tokens * p.top;
  int expert[TURNS], token[TURNS], place[TURNS];
  float weight[TURNS];
#pragma unroll
  for (int r = 0; r < TURNS; ++r) {
    const int s = r * (int)blockDim.x + tid;
    expert[r] = -1;
    if (s < n) {
      const int i = s / p.top, j = s - i * p.top;
      const int id = static_cast<const int32_t *>(p.ids.p)[i * p.ids.rs + j * p.ids.cs];
      weight[r] = static_cast<const float *>(p.weights.p)[i * p.weights.rs + j * p.weights.cs];
      const int64_t e = (int64_t)id - p.first;
      token[r] = i;
      if (id >= 0 && e >= 0 && e < p.experts) expert[r] = (int)e;
    }
  }
  for (int i = tid; i < p.experts; i += blockDim.x) base[i] = 0u;
  __syncthreads();
#pragma unroll
  for (int r = 0; r < TURNS; ++r) {
    if (r * (int)blockDim.x >= n) break;
    const int e = expert[r];
    const uint32_t same = __match_any_sync(~0u, e);
    const int lead = __ffs(same) - 1, rank = __popc(same & ((1u << lane) - 1u));
    const int turns = min(warps, (n - r * (int)blockDim.x + 31) / 32);
    int before = 0;
    for (int w = 0; w < turns; ++w) {
      if (w == warp && e >= 0 && lane == lead) {
        before = (int)base[e];
        base[e] = (uint32_t)(before + __popc(same));
      }
      __syncthreads();
    }
    place[r] = __shfl_sync(~0u, before, lead) + rank;
  }
  // from counts to chunks before an expert << 16 | places before it
  uint32_t at = 0u;
  for (int e0 = 0; e0 < p.experts; e0 += (int)blockDim.x) {
    const int e = e0 + tid;
    const int c = e < p.experts ? (int)base[e] : 0;
    const int chunks = (c + p.cols - 1) / p.cols;
    const uint32_t mine = (uint32_t)chunks << 16 | (uint32_t)c;
    uint32_t run = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(~0u, run, o);
      if (lane >= o) run += v;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = run;
    __syncthreads();
    uint32_t first = at + run - mine;
    for (int w = 0; w < warps; ++w) {
      const uint32_t v = sums[w];
      if (w < warp) first += v;
      at += v;
    }
    if (e < p.experts) base[e] = first;
    const int q0 = (int)(first >> 16), s0 = (int)(first & 0xFFFFu);
    for (int q = 0; q < chunks; ++q)
      chunk[q0 + q] =
          make_int4(e, s0 + q * p.cols, min(p.cols, c - q * p.cols), q0 | chunks << 16);
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < TURNS; ++r)
    if (expert[r] >= 0) {
      const int s = (int)(base[expert[r]] & 0xFFFFu) + place[r];
      tokens[s] = token[r];
      weights[s] = weight[r];
    }
  return (int)(at >> 16);
}

struct PlanParams {
  Choices choices;        // of this group's tokens
  ExpertsPlan out;
  DenseMat x;             // rows to lay out; p NULL: none
  uint16_t *packed;
  int64_t k, packed_ld;
};

// CTA 0 plans; the others lay out x in rows of whole 16-byte runs where no tensor copy takes it as
// it lies.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanParams p) {
  __shared__ uint32_t base[kExpertsMost], sums[32];
  const int tid = threadIdx.x;
  griddep_wait();
  griddep_launch();
  if (blockIdx.x > 0) {
    const int64_t runs = p.packed_ld / 8, all = runs * p.choices.tokens;
    for (int64_t r = (int64_t)(blockIdx.x - 1) * blockDim.x + tid; r < all;
         r += (int64_t)(gridDim.x - 1) * blockDim.x) {
      const int64_t i = r / runs, k = r % runs * 8;
      const uint16_t *q = static_cast<const uint16_t *>(p.x.p) + i * p.x.rs + k * p.x.cs;
      uint32_t v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = k + j < p.k ? q[j * p.x.cs] : 0u;
      *reinterpret_cast<uint4 *>(p.packed + i * p.packed_ld + k) =
          make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
    }
    return;
  }
  const int chunks = make_plan<kExpertsGroup * kChosenMost / kPlanThreads>(
      p.choices, p.out.chunk, p.out.token, p.out.weight, base, sums);
  if (tid == 0) *p.out.chunks = chunks;
}

// ---------------------------------------------------------------- products

constexpr int kThreads = 192;  // warp 0 loads, 1 matrix instructions and TMEM, 2-5 epilogue
constexpr int kLoaders = 16;   // more warps, where no tensor copy takes the weights as they lie
template <bool COPY>
constexpr int kAllThreads = kThreads + (COPY ? 0 : 32 * kLoaders);
constexpr int kMaxStages = 16;
constexpr uint32_t kTile = 128 * 128;  // bytes of 128 rows of one k block
constexpr uint32_t kShort = 8;

struct ProductParams {
  // weights {k, rows, experts}; tokens {k, rows} by four rows, or inner values {k, rows, 2}, by 16 of
  // them and their rests
  CUtensorMap w[2], b;
  Choices choices;
  ExpertsPlan plan;     // plan.chunks NULL: every CTA makes its own
  DenseMat res;         // sums only
  void *out;            // inner values [place][out_rs], or y
  int64_t out_rs;
  int64_t rest;         // inner: elements from a value to its rest
  float *part;          // of cut tiles
  int32_t *status;
  int32_t rows;         // output features of a tile: at most 128
  int32_t features;     // of the product
  int32_t tiles, kblocks, cols, tokens;
  int32_t stages;
  uint32_t w_bytes, stage_bytes, ring, raw, smem;  // raw: where the loader warps' rings start
  int32_t type, out_type, act;
  int32_t nothing;      // sums of nothing: y = residual
  int32_t whole;        // inner: no tile is cut
  const uint16_t *stack[2];  // weights that loader warps bring, with their extent
  int64_t es[2], rs[2];
  uintptr_t stack_end[2];
  int32_t len;               // elements of a row of them
  int32_t lines;             // places of the loader warps' rings
};

// A plan of few choices, made by every CTA that goes by it: no launch and no way through memory
// before the first weights are asked for (32 choices of eight experts of 4096 x 1792: 71 us with
// plan_kernel, 67 so, when those came here).
constexpr int kOwnChoices = 256;

struct OwnPlan {
  int4 chunk[kOwnChoices];
  int32_t token[kOwnChoices];
  float weight[kOwnChoices];
  uint32_t base[kExpertsMost], sums[32];
};

struct PlanView {
  const int4 *chunk;
  const int32_t *token;
  const float *weight;
  int chunks;
};

// By all threads of the CTA. What the plan depends on is there: the caller has waited for it, or the
// kernel before it had before it let this one start.
template <int TURNS>
__device__ __forceinline__ PlanView view_plan(const ProductParams &p, OwnPlan &own) {
  if (p.plan.chunks) return PlanView{p.plan.chunk, p.plan.token, p.plan.weight, *p.plan.chunks};
  const int n = make_plan<TURNS>(p.choices, own.chunk, own.token, own.weight, own.base, own.sums);
  __syncthreads();
  return PlanView{own.chunk, own.token, own.weight, n};
}

struct Shared {
  uint64_t full[kMaxStages], empty[kMaxStages], ready[2], free[2];
  uint32_t tmem, abort;
};

__device__ __forceinline__ void tma_box3(uint32_t sdst, const void *map, int32_t x, int32_t y,
                                         int32_t z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(sdst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// Rows r of a two-dimensional map of boxes one row high, from column x on.
__device__ __forceinline__ void tma_gather4(uint32_t sdst, const void *map, int32_t x, int4 r,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4"
      ".mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(sdst),
      "l"(map), "r"(x), "r"(r.x), "r"(r.y), "r"(r.z), "r"(r.w), "r"(bar)
      : "memory");
}

// Bring a tensor map, whose first use would wait for it.
__device__ __forceinline__ void map_ahead(const void *map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// 16 columns of this warp's 32 lanes.
__device__ __forceinline__ void tmem_load16(uint32_t addr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// The line of k blocks, cut into `ctas` equal lengths of whole units.
struct Line {
  uint32_t units, unit, ctas;  // unit: k blocks
  __device__ uint32_t begin(uint32_t c) const {
    return (uint32_t)((uint64_t)units * c / ctas) * unit;
  }
  // whose length block u is in
  __device__ uint32_t owner(uint32_t u) const {
    return (uint32_t)((((uint64_t)(u / unit) + 1) * ctas - 1) / units);
  }
  __device__ uint32_t end() const { return units * unit; }
};

// A length is kShort blocks at least where there is too little for every CTA: shorter ones would
// come sooner, but a tile's shares take longer to join.
template <bool INNER>
__device__ __forceinline__ Line line_of(const ProductParams &p, int chunks) {
  Line l;
  l.unit = INNER && p.whole ? (uint32_t)p.kblocks : 1u;
  l.units = (uint32_t)chunks * (uint32_t)p.tiles * ((uint32_t)p.kblocks / l.unit);
  const uint32_t least = INNER && p.whole ? 1u : kShort;
  l.ctas = min(kSms, max(l.units / least, min(l.units, 1u)));
  return l;
}

// A CTA's share of a cut tile that CTA c0 begins: of one begun by an earlier CTA, or of one ended by a
// later one. Inner: [g, u][choice][128]; sums: [token][128].
template <bool INNER>
__device__ __forceinline__ float *share_of(const ProductParams &p, uint32_t cta, uint32_t c0) {
  return p.part + (2 * (int64_t)cta + (cta == c0)) * (INNER ? 2 * p.cols : p.tokens) * 128;
}

// Part of a tile: k blocks [k0, k1) of tile `tile` of chunk `chunk`.
struct Piece {
  int chunk, tile, k0, k1;
};

// INNER walks expert by expert, tile after tile, and in a tile the expert's chunks. The sums walk tile
// by tile, chunk after chunk, so that one tile's sums over the experts stay in the CTA. Either way an
// expert's chunks read the same weights one right after the other.
template <bool INNER>
__device__ __forceinline__ Piece piece_at(const ProductParams &p, const PlanView &plan, uint32_t u,
                                          uint32_t end) {
  const uint32_t item = u / (uint32_t)p.kblocks;
  Piece q;
  q.k0 = (int)(u - item * (uint32_t)p.kblocks);
  q.k1 = (int)min((uint32_t)p.kblocks, q.k0 + (end - u));
  if (INNER) {
    const uint32_t c = item / (uint32_t)p.tiles, w = (uint32_t)plan.chunk[c].w;
    const uint32_t first = w & 0xFFFFu, count = w >> 16, r = item - first * p.tiles;
    q.tile = (int)(r / count);
    q.chunk = (int)(first + r - (uint32_t)q.tile * count);
  } else {
    q.tile = (int)(item / (uint32_t)plan.chunks);
    q.chunk = (int)(item - (uint32_t)q.tile * plan.chunks);
  }
  return q;
}

// Loader warps: the weights of this CTA's k blocks from rows that start anywhere, into the layout that a
// tensor copy with a 128-byte swizzle gives. A row's 128-byte lines are copied asynchronously into a ring
// of the warp's own, each once: a k block's 128 bytes are the end of one and the start of the next. (Nine
// words around each k block instead straddle two lines, 13 shared-memory wavefronts a copy instruction
// where whole lines take four; loads into registers kept too little on its way, 2.1 TB/s.) From there a
// lane shifts two words into the 16 bytes it stores. A warp takes every eighth row, so that all of its
// rows start alike within 16 bytes and the shift is the warp's.
template <bool INNER>
constexpr int kLoaderRows = (INNER ? 2 : 1) * 128 / kLoaders;
template <bool INNER>
constexpr uint32_t kLineBytes = kLoaders * kLoaderRows<INNER> * 128;  // of one line of all rows

// The aligned 16-byte word at `from` to shared memory: those of its bytes that are [lo, hi), and zeros.
__device__ __forceinline__ void copy_word(uint32_t to, uintptr_t from, uintptr_t lo, uintptr_t hi) {
  if (from >= lo) {
    const uint32_t bytes = from + 16 <= hi ? 16u : from < hi ? (uint32_t)(hi - from) : 0u;
    if (bytes)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes)
                   : "memory");
    return;
  }
#pragma unroll 1
  for (uint32_t j = 0; j < 16; j += 2) {
    const uint16_t x = from + j >= lo && from + j < hi ? (uint16_t)ld_word2((const void *)(from + j))
                                                       : (uint16_t)0;
    asm volatile("st.shared.b16 [%0], %1;" ::"r"(to + j), "h"(x) : "memory");
  }
}

// 16 bytes that start 4 S bytes and `bits` bits into the first of two words, from shared memory to `to`,
// for `rows` rows of this lane, of which `left` elements each are there.
template <int S, int STEPS>
__device__ __forceinline__ void shift_words(uint32_t raw, const uint32_t (&at)[STEPS],
                                            const uint32_t (&next)[STEPS], uint32_t to, int rows,
                                            int left, uint32_t bits) {
#pragma unroll
  for (int j = 0; j < STEPS; ++j) {
    uint32_t e[8];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(e[4 * h]), "=r"(e[4 * h + 1]), "=r"(e[4 * h + 2]), "=r"(e[4 * h + 3])
                   : "r"(raw + (h ? next[j] : at[j])));
    uint32_t r[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) r[x] = __funnelshift_r(e[x + S], e[x + S + 1], bits);
    if (left < 8) {
#pragma unroll
      for (int x = 0; x < 4; ++x)
        r[x] = 2 * x + 1 < left ? r[x] : 2 * x < left ? r[x] & 0xFFFFu : 0u;
    }
    if (j < rows)
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to + j * 4096), "r"(r[0]),
                   "r"(r[1]), "r"(r[2]), "r"(r[3])
                   : "memory");
  }
}

// LINES: places of a warp's ring, a power of two. The k block that is next needs two lines in a row, and
// all that the ring has room for are asked for.
template <bool INNER, int LINES>
__device__ __forceinline__ void load_weights(const ProductParams &p, const PlanView &plan,
                                             uint32_t u, uint32_t end, uint32_t ring,
                                             uint32_t raw, uint32_t full0, uint32_t empty0,
                                             Shared &sh, int loader, int lane) {
  constexpr int ROWS = kLoaderRows<INNER>, STEPS = ROWS / 4;
  constexpr uint32_t LINE = ROWS * 128, ALL = LINES * LINE;
  const int w = INNER ? loader >> 3 : 0;
  // this warp's rows of a tile: first, first + 8, ...
  const int first = (loader & 7) + (INNER ? 0 : (loader >> 3) * 8 * ROWS);
  const int sub = lane >> 3, chunk = lane & 7;
  const uintptr_t lo = (uintptr_t)p.stack[w], hi = p.stack_end[w];
  const int64_t pitch = p.rs[w] * 16;  // bytes from one of them to the next
  raw += loader * ALL;
  // Two places on this CTA's length, `ahead` by lines and `now` by k blocks. All that does not change
  // from one to the next of a tile is made once.
  struct Place {
    uint32_t v;
    int kb, kb1, rows;
    uintptr_t row;
  } ahead = {u, 0, 0, 0, 0}, now = {u, 0, 0, 0, 0};
  auto begin = [&](Place &c) {
    const Piece q = piece_at<INNER>(p, plan, c.v, end);
    c.kb = q.k0, c.kb1 = q.k1;
    c.v += q.k1 - q.k0;
    const int f = q.tile * p.rows;
    c.rows = min(ROWS, (min(p.rows, p.features - f) - first + 7) >> 3);  // this warp's
    c.row = lo + (uintptr_t)(plan.chunk[q.chunk].x * p.es[w] + (int64_t)(f + first) * p.rs[w]) * 2;
  };
  uintptr_t word[STEPS];  // this lane's of the line ahead; of rows that are not there, the last one's
  bool inside = false;    // all of the warp's lines of this tile are the stack's
  int lines = 0;          // of it that are still to be asked for
  auto begin_ahead = [&]() {
    if (ahead.v >= end) return;
    begin(ahead);
    lines = ahead.kb1 - ahead.kb + 1;
#pragma unroll
    for (int j = 0; j < STEPS; ++j) {
      const int row = min(4 * j + sub, max(ahead.rows, 1) - 1);
      word[j] = ((ahead.row + row * pitch) & ~(uintptr_t)127) + (uintptr_t)ahead.kb * 128 + chunk * 16;
    }
    const uintptr_t last = ahead.row + (max(ahead.rows, 1) - 1) * pitch;
    inside = (ahead.row & ~(uintptr_t)127) >= lo &&
             (last & ~(uintptr_t)127) + ((uintptr_t)ahead.kb1 + 1) * 128 <= hi;
  };
  auto ask = [&](uint32_t place) {
    if (lines > 0) {
      const uint32_t to = raw + place + sub * 128 + chunk * 16;
      if (ahead.rows > 0) {
        if (inside) {
#pragma unroll
          for (int j = 0; j < STEPS; ++j)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + j * 512),
                         "l"(word[j])
                         : "memory");
        } else {
#pragma unroll
          for (int j = 0; j < STEPS; ++j) copy_word(to + j * 512, word[j], lo, hi);
        }
      }
#pragma unroll
      for (int j = 0; j < STEPS; ++j) word[j] += 128;
      if (--lines == 0) begin_ahead();
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  int shift = 0, rows = 0;           // elements; rows of this lane
  uint32_t at[STEPS], next[STEPS];   // its words of this k block in the ring
  uint32_t place = 0;                // of the k block's first line
  auto begin_now = [&]() {
    if (now.v >= end) return;
    begin(now);
    shift = (int)(now.row >> 1 & 7);
    rows = (now.rows - sub + 3) >> 2;
#pragma unroll
    for (int j = 0; j < STEPS; ++j) {
      const int64_t row = 4 * j + sub;
      const uint32_t off = (uint32_t)((now.row + row * pitch) & 112u) + chunk * 16;
      auto in_ring = [&](uint32_t o) {
        return (place + (o >> 7) * LINE) % ALL + (uint32_t)row * 128 + (o & 127u);
      };
      at[j] = in_ring(off);
      next[j] = in_ring(off + 16);
    }
  };
  const uint32_t n = end - u;
  begin_ahead();
  begin_now();
#pragma unroll
  for (int d = 0; d < LINES; ++d) ask(d * LINE);
  const uint32_t to0 = ring + w * p.w_bytes + (first + 8 * sub) * 128 + ((chunk ^ (loader & 7)) << 4);
  uint32_t s = 0, phase = 0;
  bool ok = true;
  for (uint32_t i = 0; i < n; ++i) {
    asm volatile("cp.async.wait_group %0;" ::"n"(LINES - 2) : "memory");
    __syncwarp();
    ok = ok && __all_sync(~0u, wait_bar(&sh.abort, empty0 + 8 * s, phase ^ 1u, p.status));
    if (ok) {
      const int left = p.len - now.kb * kTileK - chunk * 8;
      const uint32_t to = to0 + s * p.stage_bytes, bits = (uint32_t)(shift & 1) * 16;
      if (shift < 2) shift_words<0, STEPS>(raw, at, next, to, rows, left, bits);
      else if (shift < 4) shift_words<1, STEPS>(raw, at, next, to, rows, left, bits);
      else if (shift < 6) shift_words<2, STEPS>(raw, at, next, to, rows, left, bits);
      else shift_words<3, STEPS>(raw, at, next, to, rows, left, bits);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (elect_one())
        asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(full0 + 8 * s) : "memory");
    }
    __syncwarp();
    // the first line is done with, behind a tile's last k block the second too
    ask(place);
    place = (place + LINE) % ALL;
    if (++now.kb == now.kb1) {
      ask(place);
      place = (place + LINE) % ALL;
      begin_now();
    } else {
#pragma unroll
      for (int j = 0; j < STEPS; ++j) at[j] = (at[j] + LINE) % ALL, next[j] = (next[j] + LINE) % ALL;
    }
    if (++s == (uint32_t)p.stages) {
      s = 0;
      phase ^= 1u;
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

__device__ __forceinline__ void inner_out(const ProductParams &p, int64_t place, int f, int rows,
                                          float (&g)[16], const float (&u)[16]) {
  act_run(g, p.act);
  uint16_t *o = static_cast<uint16_t *>(p.out) + place * p.out_rs + f;
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (i < rows) split_value(g[i] * u[i], p.type, o[i * p.out_rs], o[i * p.out_rs + p.rest]);
}

template <bool INNER, bool COPY>
__global__ void __launch_bounds__(kAllThreads<COPY>, 1)
    product_kernel(const __grid_constant__ ProductParams p) {
  extern __shared__ uint8_t raw[];
  __shared__ Shared sh;
  __shared__ OwnPlan own;
  const uint32_t ring = (smem_u32(raw) + 1023u) & ~1023u;
  const int warp = __shfl_sync(~0u, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t full0 = smem_u32(&sh.full[0]), empty0 = smem_u32(&sh.empty[0]);
  const uint32_t ready0 = smem_u32(&sh.ready[0]), free0 = smem_u32(&sh.free[0]);
  constexpr int W = INNER ? 2 : 1;
  const uint32_t stages = p.stages, stage_bytes = p.stage_bytes;
  uint32_t tmem_cols = 32;
  while (tmem_cols < 4u * p.cols) tmem_cols *= 2;  // two accumulators of g and u, or values and rests

  if (threadIdx.x == 0) {
    if (!p.nothing) {
      if (COPY) {
        map_ahead(&p.w[0]);
        if (INNER) map_ahead(&p.w[1]);
      }
      map_ahead(&p.b);
    }
    for (uint32_t i = 0; i < stages; ++i) {
      mbar_init(&sh.full[i], COPY ? 1 : 1 + kLoaders);
      mbar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.ready[i], 1);
      mbar_init(&sh.free[i], 4);
    }
    sh.abort = 0u;
    mbar_init_fence();
  }
  if (warp == 1) tmem_alloc<1>(&sh.tmem, tmem_cols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  // The sums start as the inner values' CTAs leave, and bring weights for their whole ring then: the
  // plan they go by is done, because the inner kernel lets them start only after its own wait for it.
  if (INNER || p.nothing) griddep_wait();
  griddep_launch();
  PlanView plan = {};
  if (!p.nothing) plan = view_plan<(kOwnChoices + kThreads - 1) / kThreads>(p, own);
  if (!INNER && warp != 0 && warp < kThreads / 32) griddep_wait();
  const int chunks = plan.chunks;
  const Line line = line_of<INNER>(p, chunks);
  const uint32_t cta = blockIdx.x;
  uint32_t u = 0, end = 0;
  if (cta < line.ctas) {
    u = line.begin(cta);
    end = line.begin(cta + 1);
  }

  if (warp == 0) {
    uint32_t s = 0, phase = 0, early = 0;
    bool ok = true;
    auto weights = [&](const Piece &q, const int4 &c, int kb) {
      const uint32_t bar = full0 + 8 * s, at = ring + s * stage_bytes;
      bar_expect(bar, (COPY ? W * (uint32_t)p.rows * 128u : 0u) +
                          (INNER ? (uint32_t)((c.z + 3) / 4) * 512u
                                 : (uint32_t)((c.z + 15) / 16) * 4096u));
      if (!COPY) return;
#pragma unroll
      for (int w = 0; w < W; ++w)
        tma_box3(at + w * p.w_bytes, &p.w[w], kb * kTileK, q.tile * p.rows, c.x, bar);
    };
    for (uint32_t v = u; COPY && v < end && early < stages;) {
      const Piece q = piece_at<INNER>(p, plan, v, end);
      const int4 c = plan.chunk[q.chunk];
      for (int kb = q.k0; kb < q.k1 && early < stages; ++kb) {
        if (elect_one()) weights(q, c, kb);
        __syncwarp();
        ++early;
        ++s;
      }
      v += q.k1 - q.k0;
    }
    s = 0;
    if (!INNER) griddep_wait();
    while (u < end) {
      const Piece q = piece_at<INNER>(p, plan, u, end);
      const int4 c = plan.chunk[q.chunk];
      const int fours = (c.z + 3) / 4, sixteens = (c.z + 15) / 16;
      int4 tok = make_int4(0, 0, 0, 0);
      if (INNER && lane < fours) {  // behind the last choice the first again: its product is not used
        const int32_t *q4 = plan.token + c.y;
        const int i = 4 * lane;
        tok = make_int4(q4[i], q4[i + 1 < c.z ? i + 1 : 0], q4[i + 2 < c.z ? i + 2 : 0],
                        q4[i + 3 < c.z ? i + 3 : 0]);
      }
      for (int kb = q.k0; kb < q.k1; ++kb) {
        const uint32_t bar = full0 + 8 * s, at = ring + s * stage_bytes + W * p.w_bytes;
        if (early == 0) {
          ok = ok && wait_bar(&sh.abort, empty0 + 8 * s, phase ^ 1u, p.status);
          if (elect_one() && ok) weights(q, c, kb);
        } else {
          --early;
        }
        __syncwarp();
        if (INNER) {
          if (ok && lane < fours) tma_gather4(at + lane * 512u, &p.b, kb * kTileK, tok, bar);
        } else if (elect_one() && ok) {
          for (int i = 0; i < sixteens; ++i)
            tma_box3(at + i * 4096u, &p.b, kb * kTileK, c.y + 16 * i, 0, bar);
        }
        __syncwarp();
        if (++s == stages) {
          s = 0;
          phase ^= 1u;
        }
      }
      u += q.k1 - q.k0;
    }
  } else if (warp == 1) {
    const uint32_t hi = desc_hi(1024), step = stage_bytes >> 4;
    uint32_t a = desc_lo(ring, 16u), b = desc_lo(ring + W * p.w_bytes, 16u);
    const uint32_t second = p.w_bytes >> 4;
    uint32_t s = 0, phase = 0, d = 0, dphase = 0;
    bool ok = true;
    while (u < end) {
      const Piece q = piece_at<INNER>(p, plan, u, end);
      const uint32_t n = (uint32_t)(plan.chunk[q.chunk].z + 15) & ~15u;
      // sums: every 16 columns of values and the 16 of their rests
      const uint32_t idesc = mma_desc(p.type == COLL_BF16, false, false, 128, INNER ? n : 2 * n);
      const uint32_t d0 = tmem + d * 2 * p.cols, d1 = d0 + p.cols;
      ok = ok && wait_bar(&sh.abort, free0 + 8 * d, dphase ^ 1u, p.status);
      tc_fence_after();
      uint32_t add = 0;
      for (int kb = q.k0; kb < q.k1; ++kb) {
        ok = ok && wait_bar(&sh.abort, full0 + 8 * s, phase, p.status);
        tc_fence_after();
        if (elect_one() && ok) {
#pragma unroll
          for (uint32_t i = 0; i < 4; ++i) {
            mma_f16<1>(d0, a + 2 * i, hi, b + 2 * i, hi, idesc, i ? 1u : add);
            if (INNER)
              mma_f16<1>(d1, a + second + 2 * i, hi, b + 2 * i, hi, idesc, i ? 1u : add);
          }
          mma_commit<1>(empty0 + 8 * s, 0);
        }
        __syncwarp();
        add = 1;
        a += step;
        b += step;
        if (++s == stages) {
          s = 0;
          phase ^= 1u;
          a -= stages * step;
          b -= stages * step;
        }
      }
      if (elect_one() && ok) mma_commit<1>(ready0 + 8 * d, 0);
      __syncwarp();
      dphase ^= d;
      d ^= 1u;
      u += q.k1 - q.k0;
    }
  } else if (warp >= kThreads / 32) {
    if constexpr (!COPY) {
      const int loader = warp - kThreads / 32;
      if (!INNER && p.lines == 8)
        load_weights<INNER, 8>(p, plan, u, end, ring, ring + p.raw, full0, empty0, sh, loader, lane);
      else
        load_weights<INNER, 4>(p, plan, u, end, ring, ring + p.raw, full0, empty0, sh, loader, lane);
    }
  } else {
    const int quad = warp & 3, row = quad * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    const uint32_t step = INNER ? (uint32_t)p.kblocks : (uint32_t)p.kblocks * (uint32_t)chunks;
    float *sums = reinterpret_cast<float *>(raw + (ring - smem_u32(raw)) + p.ring) + row;
    uint32_t d = 0, dphase = 0;
    bool ok = true;
    if (!INNER && chunks == 0) {
      for (int t = (int)cta; t < p.tiles; t += (int)gridDim.x) {
        const int f = t * p.rows + row;
        if (row >= p.rows || f >= p.features) continue;
        for (int i = 0; i < p.tokens; ++i)
          st_elem(p.out, i * p.out_rs + f,
                  p.res.p ? ld_elem(p.res.p, i * p.res.rs + f * p.res.cs, p.out_type) : 0.0f,
                  p.out_type);
      }
    }
    while (u < end) {
      // a cut tile (sums: all of a tile's chunks) belongs to CTAs [c0, c1]
      const uint32_t job = u / step;
      const uint32_t c0 = line.owner(job * step), c1 = line.owner(job * step + step - 1);
      const uint32_t job_end = min(end, job * step + step);
      float *part = share_of<INNER>(p, cta, c0) + row;
      if (!INNER)
        for (int i = 0; i < p.tokens; ++i) sums[i * 128] = 0.0f;
      while (u < job_end) {
        const Piece q = piece_at<INNER>(p, plan, u, job_end);
        const int4 c = plan.chunk[q.chunk];
        const int f = q.tile * p.rows + row;
        const bool live = row < p.rows && f < p.features;
        ok = ok && __all_sync(~0u, wait_bar(&sh.abort, ready0 + 8 * d, dphase, p.status));
        tc_fence_after();
        const uint32_t from = lanes + d * 2 * p.cols;
        for (int i0 = 0; ok && i0 < c.z; i0 += 16) {
          const int rows = min(16, c.z - i0);
          float v[16];
          tmem_load16(from + (INNER ? i0 : 2 * i0), v);
          if constexpr (INNER) {
            float up[16];
            tmem_load16(from + p.cols + i0, up);
            if (c0 == c1) {
              if (live) inner_out(p, c.y + i0, f, rows, v, up);
            } else {
#pragma unroll
              for (int i = 0; i < 16; ++i)
                if (i < rows) {
                  __stcg(part + (i0 + i) * 128, v[i]);
                  __stcg(part + (p.cols + i0 + i) * 128, up[i]);
                }
            }
          } else {
            float rest[16];
            tmem_load16(from + 2 * i0 + 16, rest);
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] += rest[i];
            int tok = 0;
            float wt = 0.0f;
            if (lane < rows) {
              tok = plan.token[c.y + i0 + lane];
              wt = plan.weight[c.y + i0 + lane];
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int t = __shfl_sync(~0u, tok, i);
              const float w = __shfl_sync(~0u, wt, i);
              if (i < rows) sums[t * 128] = fmaf(w, v[i], sums[t * 128]);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (elect_one())
          asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(free0 + 8 * d) : "memory");
        dphase ^= d;
        d ^= 1u;
        u += q.k1 - q.k0;
      }
      if (!INNER && ok) {
        const int f = (int)job * p.rows + row;
        if (c0 != c1) {
#pragma unroll 8
          for (int i = 0; i < p.tokens; ++i) __stcg(part + i * 128, sums[i * 128]);
        } else if (row < p.rows && f < p.features) {
#pragma unroll 8
          for (int i = 0; i < p.tokens; ++i) {
            float v = sums[i * 128];
            if (p.res.p) v += ld_elem(p.res.p, i * p.res.rs + f * p.res.cs, p.out_type);
            st_elem(p.out, i * p.out_rs + f, v, p.out_type);
          }
        }
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (sh.abort) drain();
  if (warp == 1) {
    tc_fence_after();
    tmem_free<1>(tmem, tmem_cols);
  }
}

// The shares of cut tiles, in order of the line: inner values are finished, sums get the residual. A
// launch of its own (about 2.5 us), because the last CTA to arrive would do it with one SM's loads in
// flight, and after a fence and an atomic: 5 us a tile, and a CTA can have two. Inner values: a CTA for
// every CTA of the line, which takes the tile that one began last. Sums: a CTA for every tile and
// eight tokens.
constexpr int kJoinTokens = 8;

template <bool INNER>
__global__ void __launch_bounds__(512) join_kernel(const __grid_constant__ ProductParams p) {
  __shared__ OwnPlan own;
  griddep_launch();
  const PlanView plan = view_plan<kOwnChoices / 256>(p, own);
  const int chunks = plan.chunks;
  const Line line = line_of<INNER>(p, chunks);
  const uint32_t step = INNER ? (uint32_t)p.kblocks : (uint32_t)p.kblocks * (uint32_t)chunks;
  uint32_t job = 0, c0 = 0, c1 = 0;
  if (INNER ? blockIdx.x < line.ctas : chunks > 0) {
    job = INNER ? (line.begin(blockIdx.x + 1) - 1) / step : blockIdx.x;
    c0 = line.owner(job * step);
    c1 = line.owner(job * step + step - 1);
  }
  const bool cut = c1 > c0 && (!INNER || c0 == blockIdx.x);
  Piece q = {};
  int4 c = make_int4(0, 0, 0, 0);
  if (cut) {
    q = piece_at<INNER>(p, plan, job * step, line.end());
    if (INNER) c = plan.chunk[q.chunk];
  }
  griddep_wait();
  const int row = threadIdx.x & 127, groups = blockDim.x >> 7;
  const int f = q.tile * p.rows + row;
  if (!cut || row >= p.rows || f >= p.features) return;
  constexpr int R = 4;
  const int end = INNER ? c.z : min(p.tokens, ((int)blockIdx.y + 1) * kJoinTokens);
  for (int i0 = (INNER ? 0 : (int)blockIdx.y * kJoinTokens) + (threadIdx.x >> 7); i0 < end;
       i0 += R * groups) {
    float v[R], u[R];
#pragma unroll
    for (int i = 0; i < R; ++i) v[i] = u[i] = 0.0f;
#pragma unroll 4
    for (uint32_t w = c0; w <= c1; ++w) {
      const float *o = share_of<INNER>(p, w, c0) + i0 * 128 + row;
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (i0 + groups * i < end) {
          v[i] += __ldcg(o + groups * i * 128);
          if (INNER) u[i] += __ldcg(o + (p.cols + groups * i) * 128);
        }
    }
    if constexpr (INNER) act_run(v, p.act);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int64_t t = i0 + groups * i;
      if (t >= end) break;
      if constexpr (INNER) {
        uint16_t *h = static_cast<uint16_t *>(p.out) + (c.y + t) * p.out_rs + f;
        split_value(v[i] * u[i], p.type, h[0], h[p.rest]);
      } else {
        if (p.res.p) v[i] += ld_elem(p.res.p, t * p.res.rs + f * p.res.cs, p.out_type);
        st_elem(p.out, t * p.out_rs + f, v[i], p.out_type);
      }
    }
  }
}

// ---------------------------------------------------------------- host

int check_stack(const coll_stack_t &w, int64_t e, int64_t rows, int64_t cols, View &v) {
  const int64_t lim = (int64_t)kAddressable;
  v = View{w.ptr, 0, 0, 0, 1, 2};
  if (rows == 0 || cols == 0) return COLL_OK;
  if (!w.ptr || w.es < 0 || w.rs < 0) return COLL_EINVAL;
  if ((uintptr_t)w.ptr & 1u) return COLL_EALIGN;
  if ((e > 1 && w.es > lim / (e - 1)) || (rows > 1 && w.rs > lim / (rows - 1))) return COLL_EINVAL;
  // its extent, as e rows
  v.rows = e;
  v.rs = w.es;
  v.cols = (rows - 1) * w.rs + cols;
  return COLL_OK;
}

int check(const coll_experts_t &a) {
  const int64_t most = 0x7FFFFFFF - 4096;
  for (int64_t v : {a.m, a.n, a.k, a.f})
    if (v < 0 || v > most) return COLL_EINVAL;
  if (!is_half(a.dtype) || (a.out_dtype != a.dtype && a.out_dtype != COLL_F32)) return COLL_EINVAL;
  if (a.act < COLL_ACT_RELU || a.act > COLL_ACT_SIGMOID) return COLL_EINVAL;
  if (a.experts < 1 || a.experts > kExpertsMost || a.top < 1 || a.top > kChosenMost ||
      a.first < 0 || a.first > most)
    return COLL_EINVAL;
  const int oe = esize(a.out_dtype);
  Check k;
  k.output(view(a.y, a.m, a.n, oe));
  k.input(view(a.x, a.m, a.k, 2));
  k.input(view(a.ids, a.m, a.top, 4));
  k.input(view(a.weights, a.m, a.top, 4));
  const int res = k.input(view(a.residual, a.m, a.n, oe), false);
  if (k.code) return k.code;
  View v;
  int c = check_stack(a.w_gate, a.experts, a.f, a.k, v);
  if (!c) k.in[k.n_in++] = v, c = check_stack(a.w_up, a.experts, a.f, a.k, v);
  if (!c) k.in[k.n_in++] = v, c = check_stack(a.w_down, a.experts, a.n, a.f, v);
  if (c) return c;
  k.in[k.n_in++] = v;
  if ((uintptr_t)a.status % sizeof(int32_t)) return COLL_EALIGN;
  return k.finish(res);
}

int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// A stack that a tensor copy takes as it lies: its base and strides on 16 bytes.
bool copied(const coll_stack_t &w, int64_t e, int64_t rows) {
  return (uintptr_t)w.ptr % 16 == 0 && (e == 1 || (w.es > 0 && w.es % 8 == 0)) &&
         (rows == 1 || (w.rs > 0 && w.rs % 8 == 0));
}

// Rows of tokens the same.
bool copied(const coll_mat_t &x, int64_t rows, int64_t k) {
  return (uintptr_t)x.ptr % 16 == 0 && (x.cs == 1 || k == 1) &&
         (rows == 1 || (x.rs > 0 && x.rs % 8 == 0));
}

int encode(CUtensorMap *map, int64_t type, int rank, const void *base, const cuuint64_t *dims,
           const cuuint64_t *strides, uint32_t rows, uint32_t planes = 1) {
  const PFN_cuTensorMapEncodeTiled_v12000 fn = tensor_map_encoder();
  if (!fn) return COLL_ECUDA;
  const cuuint32_t box[3] = {kTileK, rows, planes}, step[3] = {1, 1, 1};
  return fn(map,
            type == COLL_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
            (cuuint32_t)rank, const_cast<void *>(base), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? COLL_OK
             : COLL_EINVAL;
}

int encode_stack(CUtensorMap *map, int64_t type, const coll_stack_t &w, int64_t e, int64_t rows,
                 int64_t k, int box) {
  // the stride of a dimension of one is not used, but has to be one that a map may have
  const int64_t line = round_up(k, 8);
  const cuuint64_t dims[3] = {(cuuint64_t)k, (cuuint64_t)rows, (cuuint64_t)e};
  const cuuint64_t strides[2] = {(cuuint64_t)(rows == 1 ? line : w.rs) * 2,
                                 (cuuint64_t)(e == 1 ? line : w.es) * 2};
  return encode(map, type, 3, w.ptr, dims, strides, (uint32_t)box);
}

// Rows of tokens, one at a time.
int encode_rows(CUtensorMap *map, int64_t type, const void *base, int64_t rows, int64_t k,
                int64_t ld) {
  const cuuint64_t dims[2] = {(cuuint64_t)k, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  return encode(map, type, 2, base, dims, strides, 1);
}

// Inner values and, behind them all, their rests.
int encode_pairs(CUtensorMap *map, int64_t type, const void *base, int64_t rows, int64_t k,
                 int64_t ld) {
  const cuuint64_t dims[3] = {(cuuint64_t)k, (cuuint64_t)rows, 2};
  const cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)(rows * ld) * 2};
  return encode(map, type, 3, base, dims, strides, 16, 2);
}

// The bytes that every row of a stack starts on and is a multiple of: 32, 16, 4 or 2.
int alignment(const void *base, int64_t es, int64_t e, int64_t rs, int64_t rows, int64_t len) {
  uint64_t v = (uintptr_t)base | (uint64_t)len * 2;
  if (e > 1) v |= (uint64_t)es * 2;
  if (rows > 1) v |= (uint64_t)rs * 2;
  return v % 32 == 0 ? 32 : v % 16 == 0 ? 16 : v % 4 == 0 ? 4 : 2;
}

// Shared memory for a product's CTA: an SM's. (Half of it, so that the sums' CTAs fit beside the inner
// values' and bring their weights early, left too few stages: 16 experts of 4096 x 4096, 60 tokens, 265 us
// against 252; a call of 20 us gained one.) Tensor copies leave room for a CTA of the join, which then makes
// its plan beside the products (64 experts of 2048 x 704, 16 tokens of six: 86.7 us without, 82.9 with), as
// long as four stages are left; loader warps need the room themselves (eight of 2001 x 5001, 128 tokens: 137
// us, 147 without it). All three before inner values had their rests.
constexpr uint32_t kSmem = 227 * 1024 - sizeof(OwnPlan) - sizeof(Shared) - 64;
constexpr uint32_t kJoinSmem = 1024 + sizeof(OwnPlan) + 512;

// The workspace of a group of tokens, and the shapes of its launches.
struct Layout {
  int64_t tokens, places, chunks, ld, packed_ld;
  int32_t cols;
  bool nothing, direct, planned, pack;
  bool inner_copied, outer_copied;  // the weights by tensor copies
  ProductParams inner, outer;
  DirectParams few, few_sums;
  int inner_align, outer_align;
  PlanParams plan;
  uint64_t bytes;
};

// Rows of the inner tiles. 128 and cut where a CTA's length ends, or fewer and whole, which saves the
// launch that joins them: whole if that takes less time for as many experts as uniform choices come to,
// one more and all of them. The times are a model's, a k block its bytes at 45 a ns or 300 ns to issue,
// cutting 6 us. Both ways measured (us, tokens, choices / experts, sizes):
//   left whole: 17, 2 / 8, 4096 x 1792 64.6 whole, 67.7 cut; 100 of the same 73.9, 79.9; 32, 6 / 64,
//   2048 x 176 38.0, 38.2; 64, 8 / 64, 2048 x 704 101, 106; 32, 8 / 32, 2048 x 768 60.7, 64.8; 40,
//   2 / 16, 2048 x 1024 44.9, 46.6; 40, 2 / 8, 1024 x 14336 120, 126; but 33, 2 / 8, 1024 x 512 21.0,
//   19.2, 20, 4 / 8, 1024 x 1024 24.5, 23.4 and 12, 4 / 16, 2048 x 512 31.4, 30.9
//   cut: 40, 2 / 64, 1024 x 512 37.9, 41.5; 48, 2 / 16, 4096 x 512 46.9, 47.6; 24, 6 / 64, 2048 x 704
//   88.6, 92.9; 60, 2 / 16, 4096 x 4096 249, 253; 128, 2 / 8, 4096 x 14336 455, 463
// so it is right to leave tiles whole where it does but for calls of 20 to 30 us, and cuts more than it
// should.
void inner_tiles(const coll_experts_t &a, Layout &l) {
  ProductParams &p = l.inner;
  const double choices = (double)l.tokens * a.top, e = (double)a.experts;
  const double likely = e * (1.0 - pow(1.0 - 1.0 / e, choices));
  const double most = e < choices ? e : choices;
  const double chunks[3] = {likely, likely + 1.0 < most ? likely + 1.0 : most, most};
  const double kblocks = (double)ceil_div(a.k, kTileK);
  auto set = [&](int64_t rows) {  // the time of a k block
    p.tiles = (int32_t)ceil_div(a.f, rows);
    p.rows = (int32_t)round_up(ceil_div(a.f, p.tiles), 8);
    const double ns = (p.rows * 256.0 + l.cols * 128.0) / 45.0;
    return ns > 300.0 ? ns : 300.0;
  };
  // two stages have to fit beside the loader warps' rings
  const int64_t full = l.inner_copied || l.cols < 128 ? 128 : 88;
  double cut[3], best = 0.97;  // nearly as long is not sure to save
  for (int i = 0; i < 3; ++i) {
    const double block = set(full), blocks = chunks[i] * p.tiles * kblocks / kSms;
    cut[i] = (blocks > kShort ? blocks : kShort) * block + 6000.0;
  }
  int64_t rows = full;
  for (int64_t r = 16; r <= full; r += 8) {
    const double block = set(r);
    double worst = 0.0;  // of the times whole in those cut
    for (int i = 0; i < 3; ++i) {
      const double part = ceil(chunks[i] * p.tiles / kSms - 1e-9) * kblocks * block / cut[i];
      if (part > worst) worst = part;
    }
    if (worst < best) {
      best = worst;
      rows = r;
      p.whole = 1;
    }
  }
  set(rows);
}

int lay_out(const coll_experts_t &a, Layout &l, char *base) {
  memset(&l, 0, sizeof(l));
  l.tokens = a.m < kExpertsGroup ? a.m : kExpertsGroup;
  l.nothing = a.k == 0 || a.f == 0;
  const int64_t choices = l.tokens * a.top;
  const bool rows = a.x.cs == 1 || a.k == 1;
  const int64_t chosen = a.experts < choices ? a.experts : choices;
  l.direct = !l.nothing && rows && l.tokens <= kDirectTokens && choices <= kDirectChoices &&
             ceil_div(a.f, kDirectInner) * (chosen + choices / 8) < 0x7FFFFFFF;
  l.inner_copied = copied(a.w_gate, a.experts, a.f) && copied(a.w_up, a.experts, a.f);
  l.outer_copied = copied(a.w_down, a.experts, a.n);
  // columns of a chunk: all tokens, or 64 or 32 where the experts have half as many each at most (100
  // tokens of two, eight experts of 4096 x 1792: 81 us with 128, 74 with 64, whose ring is deeper; 128 of
  // 4096 x 14336 468, 462); not more than 64 beside the loader warps' rings, where 128 leave one stage
  const bool spread = choices <= 16 * a.experts;
  l.cols = l.direct ? 8
           : l.tokens <= 16 ? 16
           : l.tokens <= 32 || spread ? 32
           : l.tokens <= 64 || choices <= 32 * a.experts || !l.outer_copied ? 64 : 128;
  l.planned = !l.nothing && !l.direct && (choices > kOwnChoices || !copied(a.x, a.m, a.k));
  l.pack = !l.nothing && !l.direct && !copied(a.x, a.m, a.k);
  l.chunks = chosen + choices / l.cols;
  l.places = l.direct ? 8 * l.chunks : choices;
  l.ld = round_up(a.f, 64);
  l.packed_ld = round_up(a.k, 64);
  uint64_t used = 0;
  bool over = false;
  auto take = [&](uint64_t bytes) -> char * {
    if (bytes > kAddressable - used) {
      over = true;
      return nullptr;
    }
    const uint64_t at = used;
    used += (bytes + 255) & ~(uint64_t)255;
    return base ? base + at : nullptr;
  };
  ProductParams &p = l.inner, &q = l.outer;
  DirectParams &d = l.few, &e = l.few_sums;
  PlanParams &s = l.plan;
  ExpertsPlan o = {};
  uint64_t part = 0, counters = 0;
  if (!l.direct) {
    if (!l.nothing) inner_tiles(a, l);
    q.tiles = (int32_t)ceil_div(a.n, 128);
    q.rows = (int32_t)round_up(ceil_div(a.n, q.tiles), 8);
    p.features = (int32_t)a.f;
    q.features = (int32_t)a.n;
    p.kblocks = (int32_t)ceil_div(a.k, kTileK);
    q.kblocks = (int32_t)ceil_div(a.f, kTileK);
    // the line of k blocks is counted in 32 bits
    if ((uint64_t)l.chunks * p.tiles * p.kblocks >> 32 ||
        (uint64_t)l.chunks * q.tiles * q.kblocks >> 32)
      return COLL_EINVAL;
    q.nothing = l.nothing;
    p.cols = q.cols = l.cols;
    p.type = q.type = (int32_t)a.dtype;
    p.out_type = (int32_t)a.dtype;
    q.out_type = (int32_t)a.out_dtype;
    p.act = (int32_t)a.act;
    p.status = q.status = a.status;
    // w stacks' rows and b tiles of tokens a stage
    auto ring = [&](ProductParams &r, int w, int b, uint32_t fixed, uint32_t raw) {
      r.w_bytes = (uint32_t)r.rows * 128u;
      r.stage_bytes = w * r.w_bytes + b * (uint32_t)l.cols * 128u;
      // a matrix instruction reads 128 rows whatever a tile has: slack behind the last stage's
      const uint32_t other = 1024 + kTile - r.w_bytes + fixed + raw;
      auto fit = [&](uint32_t room) {
        return room > other ? (int32_t)((room - other) / r.stage_bytes) : 0;
      };
      r.stages = fit(raw ? kSmem : kSmem - kJoinSmem);
      if (r.stages < 4) r.stages = fit(kSmem);
      if (r.stages > kMaxStages) r.stages = kMaxStages;
      r.ring = r.stages * r.stage_bytes;
      r.raw = r.ring + fixed;
      r.smem = r.ring + other;
    };
    auto by_hand = [&](ProductParams &r, int w, const coll_stack_t &m, int64_t rows, int64_t len) {
      r.stack[w] = static_cast<const uint16_t *>(m.ptr);
      r.es[w] = m.es, r.rs[w] = m.rs;
      r.stack_end[w] =
          (uintptr_t)m.ptr + 2 * (uintptr_t)((a.experts - 1) * m.es + (rows - 1) * m.rs + len);
      r.len = (int32_t)len;
    };
    by_hand(p, 0, a.w_gate, a.f, a.k);
    by_hand(p, 1, a.w_up, a.f, a.k);
    by_hand(q, 0, a.w_down, a.n, a.f);
    const uint32_t sums = (uint32_t)l.tokens * 512u;
    p.lines = 4;
    ring(p, 2, 1, 0, l.inner_copied ? 0 : 4 * kLineBytes<true>);
    for (q.lines = 8; q.lines >= 4; q.lines /= 2) {  // as long as two stages fit beside it
      ring(q, 1, 2, sums, l.outer_copied ? 0 : q.lines * kLineBytes<false>);
      if (q.stages >= 2) break;
    }
    const uint64_t inner = (uint64_t)2 * l.cols * 512, outer = (uint64_t)l.tokens * 512;
    part = l.nothing ? 0 : 2 * kSms * (inner > outer ? inner : outer);
  } else {
    l.inner_align = alignment(a.w_gate.ptr, a.w_gate.es, a.experts, a.w_gate.rs, a.f, a.k);
    const int up = alignment(a.w_up.ptr, a.w_up.es, a.experts, a.w_up.rs, a.f, a.k);
    if (up < l.inner_align) l.inner_align = up;
    l.outer_align = alignment(a.w_down.ptr, a.w_down.es, a.experts, a.w_down.rs, a.n, a.f);
    d.w[0] = static_cast<const uint16_t *>(a.w_gate.ptr), d.es[0] = a.w_gate.es;
    d.w[1] = static_cast<const uint16_t *>(a.w_up.ptr), d.es[1] = a.w_up.es;
    e.w[0] = static_cast<const uint16_t *>(a.w_down.ptr), e.es[0] = a.w_down.es;
    d.rs[0] = a.w_gate.rs, d.rs[1] = a.w_up.rs, e.rs[0] = a.w_down.rs;
    d.len = (int32_t)a.k, e.len = (int32_t)a.f;
    d.features = (int32_t)a.f, e.features = (int32_t)a.n;
    d.x_align = alignment(a.x.ptr, 0, 1, a.x.rs, a.m, a.k);
    for (DirectParams *r : {&d, &e}) {
      r->first = (int32_t)a.first, r->experts = (int32_t)a.experts, r->top = (int32_t)a.top;
      r->type = (int32_t)a.dtype, r->out_type = (int32_t)a.out_dtype, r->act = (int32_t)a.act;
      r->most_chunks = (uint32_t)l.chunks;
      r->tiles = (int32_t)ceil_div(a.n, kDirectOuter);
      r->splits = 1;
    }
    // two CTAs for every SM; warps that have four steps each, all in flight at once
    auto warps = [](int64_t steps) { return (uint32_t)(steps > 28 ? 8 : (steps + 3) / 4); };
    d.warps = warps(ceil_div(a.k, 64));
    const int64_t steps = l.chunks * ceil_div(a.f, 64);
    int64_t splits = 2 * kSms / e.tiles;
    if (splits > steps / 16) splits = steps / 16;
    if (splits > 32) splits = 32;
    if (splits < 1) splits = 1;
    e.warps = warps(ceil_div(steps, splits));
    if (splits > 1) {
      d.splits = e.splits = (int32_t)splits;
      counters = (uint64_t)e.tiles;
      part = (uint64_t)splits * e.tiles * l.tokens * 64;
    }
  }
  if (l.planned) {
    o.chunks = reinterpret_cast<int32_t *>(take(4));
    o.chunk = reinterpret_cast<int4 *>(take((uint64_t)l.chunks * 16));
    o.token = reinterpret_cast<int32_t *>(take((uint64_t)l.places * 4));
    o.weight = reinterpret_cast<float *>(take((uint64_t)l.places * 4));
  }
  d.counters = e.counters = reinterpret_cast<uint32_t *>(take(counters * 4));
  char *h = take((uint64_t)l.places * l.ld * 4);  // the values, then their rests
  p.part = q.part = e.part = reinterpret_cast<float *>(take(part));
  if (l.pack)
    s.packed = reinterpret_cast<uint16_t *>(take((uint64_t)l.tokens * l.packed_ld * 2));
  s.packed_ld = l.packed_ld;
  s.choices.top = (int32_t)a.top;
  s.choices.experts = (int32_t)a.experts;
  s.choices.first = (int32_t)a.first;
  s.choices.cols = l.cols;
  s.k = a.k;
  s.out = p.plan = q.plan = o;
  p.out = h;
  p.out_rs = l.ld;
  p.rest = d.rest = e.rest = l.places * l.ld;
  d.h = reinterpret_cast<uint16_t *>(h);
  d.h_ld = e.x_ld = l.ld;
  e.x = d.h;
  l.bytes = used;
  return over ? COLL_EINVAL : COLL_OK;
}

int64_t need(const coll_experts_t &a) {
  if (a.m == 0 || a.n == 0) return 0;
  Layout l;
  const int c = lay_out(a, l, nullptr);
  return c ? c : (int64_t)l.bytes + 128;  // room to start on 128 bytes
}

template <bool INNER, bool COPY>
int set_up() {
  static DenseSmemLimit limit;
  return limit((const void *)product_kernel<INNER, COPY>, kSmem) == cudaSuccess ? COLL_OK
                                                                                   : COLL_ECUDA;
}

template <bool INNER, bool COPY>
cudaError_t launch(const ProductParams &p, cudaStream_t s) {
  const cudaError_t e = dense_launch(product_kernel<INNER, COPY>, dim3(kSms), kAllThreads<COPY>,
                                     p.smem, 1, s, p);
  if (e != cudaSuccess || p.nothing || p.whole) return e;
  const dim3 grid = INNER ? dim3(kSms) : dim3(p.tiles, (unsigned)ceil_div(p.tokens, kJoinTokens));
  return dense_launch(join_kernel<INNER>, grid, INNER ? 512 : 256, 0, 1, s, p);
}

int run(const coll_experts_t &a, Layout &l, cudaStream_t s) {
  int c = COLL_OK;
  ProductParams &p = l.inner, &q = l.outer;
  DirectParams &d = l.few, &e = l.few_sums;
  if (!l.direct) {
    c = l.inner_copied ? set_up<true, true>() : set_up<true, false>();
    if (!c) c = l.outer_copied ? set_up<false, true>() : set_up<false, false>();
    if (!c && !l.nothing) {
      if (l.inner_copied) {
        c = encode_stack(&p.w[0], a.dtype, a.w_gate, a.experts, a.f, a.k, p.rows);
        if (!c) c = encode_stack(&p.w[1], a.dtype, a.w_up, a.experts, a.f, a.k, p.rows);
      }
      if (!c && l.outer_copied)
        c = encode_stack(&q.w[0], a.dtype, a.w_down, a.experts, a.n, a.f, q.rows);
      if (!c) c = encode_pairs(&q.b, a.dtype, p.out, l.places, a.f, l.ld);
      // the first group's rows as a trial of them all
      if (!c)
        c = l.pack ? encode_rows(&p.b, a.dtype, l.plan.packed, l.tokens, a.k, l.packed_ld)
                   : encode_rows(&p.b, a.dtype, a.x.ptr, l.tokens, a.k,
                                 a.m == 1 ? round_up(a.k, 8) : a.x.rs);
    }
    if (c) return c;
  }
  const int oe = esize(a.out_dtype);
  for (int64_t t = 0; t < a.m; t += l.tokens) {
    const int64_t tokens = a.m - t < l.tokens ? a.m - t : l.tokens;
    PlanParams &o = l.plan;
    Choices &ch = o.choices;
    ch.ids = DenseMat{static_cast<const int32_t *>(a.ids.ptr) + t * a.ids.rs, a.ids.rs, a.ids.cs};
    ch.weights = DenseMat{static_cast<const float *>(a.weights.ptr) + t * a.weights.rs,
                          a.weights.rs, a.weights.cs};
    ch.tokens = p.tokens = q.tokens = d.tokens = e.tokens = (int32_t)tokens;
    p.choices = q.choices = ch;
    const uint16_t *x = static_cast<const uint16_t *>(a.x.ptr) + t * a.x.rs;
    if (l.pack) o.x = DenseMat{x, a.x.rs, a.x.cs};
    else if (!l.direct && t && !l.nothing)
      c = encode_rows(&p.b, a.dtype, x, tokens, a.k, a.x.rs);
    if (c) return c;
    void *y = static_cast<char *>(a.y.ptr) + t * a.y.rs * oe;
    DenseMat res = {};
    if (a.residual.ptr)
      res = DenseMat{static_cast<const char *>(a.residual.ptr) + t * a.residual.rs * oe,
                     a.residual.rs, a.residual.cs};
    cudaError_t err = cudaSuccess;
    if (l.planned) {
      const int64_t most = tokens * a.top > a.experts ? tokens * a.top : a.experts;
      const unsigned threads = most >= kPlanThreads ? kPlanThreads : (unsigned)round_up(most, 32);
      const unsigned more = l.pack ? (unsigned)ceil_div(tokens * l.packed_ld / 8, threads) : 0;
      err = dense_launch(plan_kernel, dim3(1 + more), threads, 0, 1, s, o);
    }
    if (l.direct) {
      d.ids = e.ids = ch.ids;
      d.weights = e.weights = ch.weights;
      d.x = x;
      d.x_ld = a.x.rs;
      e.y = y;
      e.y_rs = a.y.rs;
      e.res = res;
      if (err == cudaSuccess) err = experts_direct_inner(d, l.inner_align, s);
      if (err == cudaSuccess) err = experts_direct_outer(e, l.outer_align, s);
    } else {
      q.out = y;
      q.out_rs = a.y.rs;
      q.res = res;
      if (err == cudaSuccess && !l.nothing)
        err = l.inner_copied ? launch<true, true>(p, s) : launch<true, false>(p, s);
      if (err == cudaSuccess)
        err = l.outer_copied ? launch<false, true>(q, s) : launch<false, false>(q, s);
    }
    if (err != cudaSuccess) return COLL_ECUDA;
  }
  return COLL_OK;
}

}  // namespace
}  // namespace coll

extern "C" int64_t coll_gated_experts_workspace(const coll_experts_t *a) {
  if (!a) return COLL_EINVAL;
  const int c = coll::check(*a);
  return c ? c : coll::need(*a);
}

extern "C" int coll_gated_experts(const coll_experts_t *a, void *stream) {
  if (!a) return COLL_EINVAL;
  int c = coll::check(*a);
  if (c || a->m == 0 || a->n == 0) return c;
  // laid out from where the workspace starts, whether or not it is there or large enough
  char *base = reinterpret_cast<char *>(((uintptr_t)a->workspace + 127) & ~(uintptr_t)127);
  coll::Layout l;
  c = coll::lay_out(*a, l, base);
  if (c) return c;
  if (!a->workspace || ((uintptr_t)a->workspace & 15u) || a->workspace_bytes < l.bytes + 128)
    return COLL_EWORKSPACE;
  return coll::run(*a, l, static_cast<cudaStream_t>(stream));
}
