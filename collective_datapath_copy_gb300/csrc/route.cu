// The router's choice of experts and its gradient: C ABI (include/coll.h) and kernels.
//
//   choice      the `top` largest logits of a token, largest first, ties to the lowest index
//   softmax     p_e = exp(l_e - max) / sum over all e;       sigmoid  s_e = 1 / (1 + exp(-l_e))
//   weights     scale score_j, or scale score_j / (sum over the chosen): then only the chosen logits
//               matter, and softmax scores are taken relative to the largest, exp(l_j - l_0) / sum;
//               sigmoids as they are where all chosen logits are above -60, else relative to the
//               largest too, exp(log s_j - log s_0) / sum, so that no sum of tiny scores vanishes
//
// A warp takes a token. Its logits stay in registers, as keys whose unsigned order is that of the
// numbers, or as they are; choosing is by them alone, so it depends on no computed score. Bound by the
// warps' instructions as much as by HBM (32768 x 256, eight chosen: 11.8 us, of which reading takes 5), so
// for many experts the chosen are not taken one by one: the k-th largest of the lanes' largest is reached
// by at least k logits and by few more, which a lane each then ranks.
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include "dense.h"
#include "dense_check.h"
#include "dense_epi.cuh"
#include "tma.cuh"

namespace coll {
namespace {

constexpr int kWarps = 8;
constexpr int kSmCount = 152;         // of a GB300
constexpr int kMostExperts = 1024;  // 32 a lane
constexpr int kMostChosen = 32;     // one a lane

struct RouteParams {
  DenseMat logits;
  int32_t *ids;
  int64_t ids_rs, ids_cs;
  float *weights;
  int64_t w_rs, w_cs;
  void *dlogits;  // backward
  int64_t dl_rs;
  int64_t t;
  int32_t e, top, type, score, norm;
  float scale;
};

// Order-preserving: a < b as numbers exactly where key(a) < key(b); -0 is 0, NaN the largest (as in
// a sort). 0 stands for what cannot be chosen: -inf, and places past the end.
__device__ __forceinline__ uint32_t order_key(float v) {
  v += 0.0f;
  if (v != v) return 0xFFFFFFFFu;
  if (v == -INFINITY) return 0u;
  const uint32_t u = __float_as_uint(v);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  if (k == 0u) return -INFINITY;
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}
// NaN only where every lane's is.
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// exp(d) for d <= 0, off by 2^-22 and d's rounding times log2 e, 2^-23 |d|, 0 below 2^-126: for sums and
// products over all experts, where a term so far below the largest is nothing, a third of expf's
// instructions.
__device__ __forceinline__ float exp_below(float d) { return exp2_fast(d * kLog2e); }

// a / b, off by two steps at most, for b up to 2^126 (0 past it). With exact divisions 32768 x 256 took
// 12.9 us in place of 11.8, the gradient of 777 x 60 2.8 in place of 2.4.
__device__ __forceinline__ float quotient(float a, float b) { return __fdividef(a, b); }

__device__ __forceinline__ float log_sigmoid(float l) {
  return fminf(l, 0.0f) - log1pf(expf(-fabsf(l)));
}
// Below -80 the exponential itself, which 1 added to its reciprocal would not change: the quotient over
// that is 0 from 2^-126 on, where scores still are numbers. Not x / (1 + x) throughout: s and 1 - s, which
// the gradient multiplies, would then share their errors (9.8e-8 of its size so, 7.2e-8 as they are).
__device__ __forceinline__ float sigmoid(float l) {
  const bool far = l < -80.0f;
  const float x = expf(far ? l : -l);
  return far ? x : quotient(1.0f, 1.0f + x);
}

// The sum over the first `top` lanes, which the others have to leave at 0, in those lanes.
__device__ __forceinline__ float chosen_sum(float v, int top) {
  if (top > 8) {
    v += __shfl_xor_sync(~0u, v, 16);
    v += __shfl_xor_sync(~0u, v, 8);
  }
#pragma unroll
  for (int o = 4; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

// Normalised weights over the chosen logits, one in each of the first `top` lanes; `there`: a choice
// was left for this lane. SORTED: the largest is lane 0's.
template <bool SORTED>
__device__ __forceinline__ float normalised(float l, bool there, int top, int score) {
  // sigmoids that are far from underflow as they are, without their logarithms (32768 x 128, six chosen:
  // a thirtieth of the time)
  if (score == COLL_SCORE_SIGMOID && __all_sync(~0u, !there || l > -60.0f)) {
    const float s = there ? sigmoid(l) : 0.0f;
    const float sum = chosen_sum(s, top);
    return there ? quotient(s, sum) : 0.0f;
  }
  const float a = score == COLL_SCORE_SIGMOID ? log_sigmoid(l) : l;
  const float most = SORTED ? __shfl_sync(~0u, a, 0) : warp_max(there ? a : -INFINITY);
  const float x = there ? expf(a - most) : 0.0f;
  const float sum = chosen_sum(x, top);
  return there ? quotient(x, sum) : 0.0f;
}

// How a row lies over a warp: lane l holds runs of L neighbouring logits, V / L of them. VEC: the runs
// are one load each, up to 16 bytes; else L is 1.
template <int V, int TYPE, bool VEC>
struct Row {
  static constexpr int kSize = TYPE == COLL_F32 ? 4 : 2;
  static constexpr int L = !VEC ? 1 : V < 16 / kSize ? V : 16 / kSize;
  static __device__ __forceinline__ int index(int i, int lane) {
    return (i / L * 32 + lane) * L + i % L;
  }
  static __device__ __forceinline__ const char *row(const RouteParams &p, int64_t row) {
    return static_cast<const char *>(p.logits.p) + row * p.logits.rs * kSize;
  }
  // -inf past the end
  static __device__ __forceinline__ void load(const RouteParams &p, const char *base, int lane,
                                              float (&v)[V]) {
    if (VEC && p.e == 32 * V) load_run<true>(p, base, lane, v);
    else load_run<false>(p, base, lane, v);
  }
  template <bool FULL>
  static __device__ __forceinline__ void load_run(const RouteParams &p, const char *base, int lane,
                                                  float (&v)[V]) {
    constexpr int kWords = L * kSize >= 4 ? L * kSize / 4 : 1;
#pragma unroll
    for (int i = 0; i < V; i += L) {
      const int e = index(i, lane);
      if constexpr (L * kSize < 4 || !VEC) {
        v[i] = e < p.e ? ld_elem(base, (int64_t)e * p.logits.cs, TYPE) : -INFINITY;
      } else {
        uint32_t w[kWords];
        const char *q = base + e * kSize;
        if (FULL || e < p.e) {
          if constexpr (kWords == 4) {
            const uint4 x = *reinterpret_cast<const uint4 *>(q);
            w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
          } else if constexpr (kWords == 2) {
            const uint2 x = *reinterpret_cast<const uint2 *>(q);
            w[0] = x.x, w[1] = x.y;
          } else {
            w[0] = *reinterpret_cast<const uint32_t *>(q);
          }
        }
#pragma unroll
        for (int j = 0; j < L; ++j) {
          const float x = TYPE == COLL_F32 ? __uint_as_float(w[j])
                                           : h2f((uint16_t)(w[j / 2] >> (16 * (j & 1))), TYPE);
          v[i + j] = FULL || e < p.e ? x : -INFINITY;
        }
      }
    }
  }
  static __device__ __forceinline__ void store(const RouteParams &p, int64_t row, int lane,
                                               const float (&v)[V]) {
    char *base = static_cast<char *>(p.dlogits) + row * p.dl_rs * kSize;
    constexpr int kWords = L * kSize >= 4 ? L * kSize / 4 : 1;
#pragma unroll
    for (int i = 0; i < V; i += L) {
      const int e = index(i, lane);
      if (e >= p.e) continue;
      if constexpr (L * kSize < 4 || !VEC) {
        st_elem(base, e, v[i], TYPE);
      } else {
        uint32_t w[kWords];
#pragma unroll
        for (int j = 0; j < kWords; ++j)
          w[j] = TYPE == COLL_F32 ? __float_as_uint(v[i + j])
                                  : f2h2(v[i + 2 * j], v[i + (2 * j + 1) % V], TYPE);
        char *q = base + e * kSize;
        if constexpr (kWords == 4)
          *reinterpret_cast<uint4 *>(q) = make_uint4(w[0], w[1], w[2], w[3]);
        else if constexpr (kWords == 2) *reinterpret_cast<uint2 *>(q) = make_uint2(w[0], w[1]);
        else *reinterpret_cast<uint32_t *>(q) = w[0];
      }
    }
  }
};

// One round for each choice: the largest key, of equal ones that of the lowest index. Lane j gets the
// j-th.
template <typename R, int V>
__device__ __forceinline__ void choose_in_turn(int top, int lane, const float (&v)[V], int &id,
                                               float &chosen) {
  uint32_t key[V];
  bool odd = false;  // NaN or an infinity among the logits
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const uint32_t u = __float_as_uint(v[i] + 0.0f);
    key[i] = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
    odd = odd || !(fabsf(v[i]) < INFINITY);
  }
  if (__any_sync(~0u, odd)) {
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = order_key(v[i]);
  }
  for (int j = 0; j < top; ++j) {
    uint32_t best = 0u;
    int at = 0;
#pragma unroll
    for (int i = V - 1; i >= 0; --i)
      if (key[i] >= best) best = key[i], at = R::index(i, lane);
    const uint32_t most = __reduce_max_sync(~0u, best);
    if (most == 0u) break;
    const uint32_t first = __reduce_min_sync(~0u, best == most ? (uint32_t)at : ~0u);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if ((uint32_t)R::index(i, lane) == first) key[i] = 0u;
    if (lane == j) {
      id = (int)first;
      chosen = key_value(most);
    }
  }
}

// NaN where one is.
__device__ __forceinline__ float max_of_three(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

struct Places {
  uint2 of[32];  // value, index
  float value[32];
};

// The same by rank among the logits that reach the top-th largest of the lanes' own largest: all that
// are chosen, and few more, a lane each. On the numbers themselves: only rows with a NaN need keys.
// False for those, and where more than 32 reach it.
template <typename R, int V>
__device__ __forceinline__ bool choose_by_rank(int top, int lane, const float (&v)[V], Places &mine,
                                               int &id, float &chosen) {
  static_assert(V % 2 == 0, "logits in pairs");
  float best = v[0];
#pragma unroll
  for (int i = 0; i < V; i += 2) best = max_of_three(best, v[i], v[i + 1]);
  if (__any_sync(~0u, best != best)) return false;
  // equal lanes go together, which only lowers what is left
  float least = 0.0f;
#pragma unroll 4
  for (int j = 0; j < top; ++j) {
    least = warp_max(best);
    best = best == least ? -INFINITY : best;
  }
  least = fmaxf(least, -FLT_MAX);  // lanes ran out: all but -inf are wanted
  int count = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) count += v[i] >= least;
  int at = count;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .s32 c;\n\tshfl.sync.up.b32 c|p, %0, %1, 0, 0xffffffff;\n\t"
        "@p add.s32 %0, %0, c;\n\t}"
        : "+r"(at)
        : "r"(o));
  const int n = __shfl_sync(~0u, at, 31);
  if (n > 32) return false;
  uint32_t to = smem_u32(mine.of + at - count);
#pragma unroll
  for (int i = 0; i < V; ++i)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ge.f32 p, %1, %2;\n\t"
        "@p st.shared.v2.b32 [%0], {%1, %3};\n\t@p add.u32 %0, %0, 8;\n\t}"
        : "+r"(to)
        : "f"(v[i]), "f"(least), "r"(R::index(i, lane))
        : "memory");
  __syncwarp();
  const bool one = lane < n;
  const uint2 own = mine.of[lane];
  const float value = one ? __uint_as_float(own.x) : -INFINITY;
  mine.value[lane] = value;
  __syncwarp();
  uint32_t rank = 0;
#pragma unroll 2
  for (int j = 0; j < n; j += 4) {
    const float4 o = *reinterpret_cast<const float4 *>(mine.value + j);
    rank += o.x > value;
    rank += o.y > value;
    rank += o.z > value;
    rank += o.w > value;
  }
  // different numbers have the ranks 0 to n - 1; of equal ones the lower index comes first
  if (__reduce_add_sync(~0u, one ? rank : 0u) != (uint32_t)(n * (n - 1) / 2)) {
    for (int j = 0; j < n; ++j) rank += mine.value[j] == value && mine.of[j].y < own.y;
    __syncwarp();
  }
  if (one && rank < (uint32_t)top) mine.of[rank] = own;
  __syncwarp();
  if (one && lane < top) {
    const uint2 o = mine.of[lane];
    chosen = __uint_as_float(o.x);
    id = (int)o.y;
  }
  __syncwarp();
  return true;
}

// CTAs that an SM is sure to hold, which bounds the registers: those of V logits, asked for ahead, and what
// lets a row's instructions overlap. With exact divisions: 8000 tokens of 1000 12.8 us with one, 10.6 with
// two; 8192 of 512 8.9 with two, 7.5 with three; 32768 of 256 12.8 with four, 13.9 with five; of 128 16.2
// with four, 13.3 with six; 5003 of 60 3.0 with four, 3.4 with six, 4.0 with eight (more fit, and the grid
// has eight an SM). A row of 1024 and the next one do not fit 128 registers: up to 304 bytes of a thread's
// go to local memory with two CTAs (168 in 16-byte loads), up to 36 of rows of 512 with three, and that is
// in these times.
template <int V>
constexpr int kPerSm = V <= 2 ? 4 : V <= 4 ? 6 : V <= 8 ? 4 : V <= 16 ? 3 : 2;

template <int V, int TYPE, bool VEC>
__global__ void __launch_bounds__(kWarps * 32, kPerSm<V>) route_kernel(const RouteParams p) {
  using R = Row<V, TYPE, VEC>;
  __shared__ __align__(16) Places places[kWarps];
  // by a shuffle, from which the compiler knows that it is the same for all lanes: the row's branches and
  // addresses are then the warp's (32768 x 256: an eighth of the time)
  const int warp = __shfl_sync(~0u, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int64_t step = (int64_t)gridDim.x * kWarps;
  int64_t row = (int64_t)blockIdx.x * kWarps + warp;
  const char *from = R::row(p, row);
  int32_t *ids = p.ids + row * p.ids_rs + lane * p.ids_cs;
  float *weights = p.weights + row * p.w_rs + lane * p.w_cs;
  griddep_launch();
  griddep_wait();
  float v[V], next[V];
  if (row < p.t) R::load(p, from, lane, next);
  for (; row < p.t; row += step) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = next[i];
    from += step * p.logits.rs * R::kSize;
    if (row + step < p.t) R::load(p, from, lane, next);
    float chosen = -INFINITY;
    int id = -1;
    bool done = false;
    if constexpr (V > 2) done = choose_by_rank<R, V>(p.top, lane, v, places[warp], id, chosen);
    if (!done) choose_in_turn<R, V>(p.top, lane, v, id, chosen);
    const bool there = id >= 0;
    float w;
    if (p.norm) {
      w = normalised<true>(chosen, there, p.top, p.score);
    } else if (p.score == COLL_SCORE_SIGMOID) {
      w = sigmoid(chosen);
    } else {
      const float most = __shfl_sync(~0u, chosen, 0);
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) sum += exp_below(v[i] - most);
      w = quotient(expf(chosen - most), warp_sum(sum));
    }
    if (lane < p.top) {
      *ids = id;
      *weights = there ? w * p.scale : 0.0f;
    }
    ids += step * p.ids_rs;
    weights += step * p.w_rs;
  }
}

// With g = scale dweights over the chosen, w the normalised weights, p or s the scores:
//   normalised softmax  dl_j = w_j (g_j - sum g w);      sigmoid, normalised  the same times 1 - s_j
//   softmax             dl_e = p_e ([e chosen] g_e - sum g p);        sigmoid  dl_j = g_j s_j (1 - s_j)
// 1 - s is the sigmoid of -l. Logits not chosen get 0 but for the plain softmax. Chosen twice, an
// expert gets both gradients (and a normalised weight for each). The row is written whole as if
// nothing were chosen, then the chosen logits' lanes write theirs over it.
template <int V, int TYPE, bool VEC>
__global__ void __launch_bounds__(kWarps * 32) route_bwd_kernel(const RouteParams p) {
  using R = Row<V, TYPE, VEC>;
  const int warp = __shfl_sync(~0u, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * kWarps + warp;
  griddep_launch();
  griddep_wait();
  if (row >= p.t) return;
  int id = -1;
  float g = 0.0f, l = -INFINITY;
  const bool plain = !p.norm && p.score == COLL_SCORE_SOFTMAX;
  if (lane < p.top) {
    id = p.ids[row * p.ids_rs + lane * p.ids_cs];
    g = p.weights[row * p.w_rs + lane * p.w_cs] * p.scale;
  }
  float v[V], d, rest = 0.0f;  // rest: what an expert gets beside its own gradients
  if (plain) R::load(p, R::row(p, row), lane, v);
  const bool there = (uint32_t)id < (uint32_t)p.e;
  if (there) l = ld_elem(p.logits.p, row * p.logits.rs + id * p.logits.cs, TYPE);
  else g = 0.0f;  // whatever stands there has no part in the sums
  if (p.norm) {
    const float w = normalised<false>(l, there, p.top, p.score);
    const float sum = chosen_sum(g * w, p.top);
    d = w * (g - sum);
    if (p.score == COLL_SCORE_SIGMOID) d *= sigmoid(-l);
  } else if (p.score == COLL_SCORE_SIGMOID) {
    d = g * sigmoid(l) * sigmoid(-l);
  } else {
    float most = v[0];
#pragma unroll
    for (int i = 1; i < V; ++i) most = fmaxf(most, v[i]);
    most = warp_max(most);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      v[i] = exp_below(v[i] - most);
      sum += v[i];
    }
    sum = warp_sum(sum);
    // a row of -inf has no probabilities, and no gradient
    const float r = most == -INFINITY ? 0.0f : quotient(1.0f, sum);
    const float own = there ? (most == -INFINITY ? 0.0f : expf(l - most) * r) : 0.0f;
    d = own * g;
    const float all = __shfl_sync(~0u, chosen_sum(d, p.top), 0);
    rest = -all * own;
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = most == -INFINITY ? 0.0f : v[i] * (-all * r);
  }
  if (!plain) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = 0.0f;
  }
  R::store(p, row, lane, v);
  if (!there) {
    d = 0.0f;
    id = -1;
  }
  // an expert that was chosen more than once: its first lane adds the others' up, in order
  const uint32_t same = __match_any_sync(~0u, id);
  const bool first = there && __ffs(same) - 1 == lane;
  float sum = d;
  if (__any_sync(~0u, first && __popc(same) > 1)) {
    for (int j = 0; j < p.top; ++j) {
      const float x = __shfl_sync(~0u, d, j);
      if (first && j > lane && (same >> j & 1u)) sum += x;
    }
  }
  __syncwarp();
  if (first) st_elem(p.dlogits, row * p.dl_rs + id, sum + rest, TYPE);
}

template <bool BWD, int TYPE, bool VEC>
cudaError_t launch(const RouteParams &p, cudaStream_t s) {
  // as many CTAs as the SMs hold, whose warps ask for their next row ahead (a second wave of a few: 18
  // us for 32768 x 256)
  const int64_t rows = (p.t + kWarps - 1) / kWarps;
  auto grid = [&](int per_sm) {
    return dim3((unsigned)(BWD || rows <= kSmCount * per_sm ? rows : kSmCount * per_sm));
  };
#define COLL_ROUTE(V)                                                                               \
  return BWD ? dense_launch(route_bwd_kernel<V, TYPE, VEC>, grid(0), kWarps * 32, 0, 1, s, p)       \
             : dense_launch(route_kernel<V, TYPE, VEC>, grid(V <= 2 ? 8 : kPerSm<V>), kWarps * 32, 0, 1, \
                            s, p)
  if (p.e <= 32) COLL_ROUTE(1);
  if (p.e <= 64) COLL_ROUTE(2);
  if (p.e <= 128) COLL_ROUTE(4);
  if (p.e <= 256) COLL_ROUTE(8);
  if (p.e <= 512) COLL_ROUTE(16);
  COLL_ROUTE(32);
#undef COLL_ROUTE
}

// Do rows lie so that every lane's runs are whole loads (and stores)? Runs are of at most 16 bytes
// and V elements.
bool whole_runs(const RouteParams &p, bool bwd) {
  const int size = esize(p.type), v = p.e <= 32 ? 1 : p.e <= 64 ? 2 : p.e <= 128 ? 4 : 8;
  const int run = v * size < 16 ? v * size : 16;
  auto fits = [&](const void *q, int64_t rs) {
    return ((uintptr_t)q | (p.t > 1 ? (uint64_t)(rs * size) : 0)) % run == 0;
  };
  return run >= 4 && p.e * size % run == 0 && p.logits.cs == 1 && fits(p.logits.p, p.logits.rs) &&
         (!bwd || fits(p.dlogits, p.dl_rs));
}

template <bool BWD>
cudaError_t launch(const RouteParams &p, cudaStream_t s) {
  const bool vec = whole_runs(p, BWD);
#define COLL_ROUTE(TYPE) return vec ? launch<BWD, TYPE, true>(p, s) : launch<BWD, TYPE, false>(p, s)
  if (p.type == COLL_F32) COLL_ROUTE(COLL_F32);
  if (p.type == COLL_BF16) COLL_ROUTE(COLL_BF16);
  COLL_ROUTE(COLL_F16);
#undef COLL_ROUTE
}

template <typename T>
int check_sizes(const T &a) {
  if (a.t < 0 || a.t > 0x7FFFFFFF - 4096 || a.top < 1 || a.top > kMostChosen || a.e < a.top ||
      a.e > kMostExperts)
    return COLL_EINVAL;
  if (!is_half(a.dtype) && a.dtype != COLL_F32) return COLL_EINVAL;
  if (a.score != COLL_SCORE_SOFTMAX && a.score != COLL_SCORE_SIGMOID) return COLL_EINVAL;
  // the weights are binary32, and so is what they are multiplied by
  return (a.normalize == 0 || a.normalize == 1) && fabs(a.scale) <= FLT_MAX ? COLL_OK : COLL_EINVAL;
}

int check(const coll_route_t &a) {
  const int c = check_sizes(a);
  if (c) return c;
  Check k;
  k.output(view(a.ids, a.t, a.top, 4));
  k.output(view(a.weights, a.t, a.top, 4));
  k.input(view(a.logits, a.t, a.e, esize(a.dtype)));
  return k.finish();
}

int check(const coll_route_bwd_t &a) {
  const int c = check_sizes(a);
  if (c) return c;
  Check k;
  k.output(view(a.dlogits, a.t, a.e, esize(a.dtype)));
  k.input(view(a.dweights, a.t, a.top, 4));
  k.input(view(a.logits, a.t, a.e, esize(a.dtype)));
  k.input(view(a.ids, a.t, a.top, 4));
  return k.finish();
}

template <typename T>
RouteParams params(const T &a, const coll_mat_t &w) {
  RouteParams p = {};
  p.logits = DenseMat{a.logits.ptr, a.logits.rs, a.logits.cs};
  p.ids = static_cast<int32_t *>(a.ids.ptr);
  p.ids_rs = a.ids.rs;
  p.ids_cs = a.ids.cs;
  p.weights = static_cast<float *>(w.ptr);
  p.w_rs = w.rs;
  p.w_cs = w.cs;
  p.t = a.t;
  p.e = (int32_t)a.e;
  p.top = (int32_t)a.top;
  p.type = (int32_t)a.dtype;
  p.score = (int32_t)a.score;
  p.norm = (int32_t)a.normalize;
  p.scale = (float)a.scale;
  return p;
}

}  // namespace
}  // namespace coll

extern "C" int coll_route(const coll_route_t *a, void *stream) {
  if (!a) return COLL_EINVAL;
  const int c = coll::check(*a);
  if (c || a->t == 0) return c;
  const coll::RouteParams p = coll::params(*a, a->weights);
  return coll::launch<false>(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? COLL_OK
                                                                                  : COLL_ECUDA;
}

extern "C" int coll_route_backward(const coll_route_bwd_t *a, void *stream) {
  if (!a) return COLL_EINVAL;
  const int c = coll::check(*a);
  if (c || a->t == 0) return c;
  coll::RouteParams p = coll::params(*a, a->dweights);
  p.dlogits = a->dlogits.ptr;
  p.dl_rs = a->dlogits.rs;
  return coll::launch<true>(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? COLL_OK
                                                                                 : COLL_ECUDA;
}
