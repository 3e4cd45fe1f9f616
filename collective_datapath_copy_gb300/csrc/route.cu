// The router's choice of experts and its gradient: C ABI (include/coll.h) and kernels.
//
//   choice      the `top` largest logits of a token, largest first, ties to the lowest index
//   softmax     p_e = exp(l_e - max) / sum over all e;       sigmoid  s_e = 1 / (1 + exp(-l_e))
//   weights     scale score_j, or scale score_j / (sum over the chosen): then only the chosen logits
//               matter, and both scores are taken relative to the largest, exp(a_j - a_0) / sum, with
//               a = l (softmax) or log s (sigmoid), so that no sum of tiny scores vanishes
//
// A warp takes a token. Its logits stay in registers, as keys whose unsigned order is that of the
// numbers; choosing is by the keys alone, so it depends on no computed score.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "dense.h"
#include "dense_check.h"
#include "dense_epi.cuh"
#include "tma.cuh"

namespace coll {
namespace {

constexpr int kWarps = 8;
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
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float w = __shfl_xor_sync(~0u, v, o);
    v = w > v || w != w ? w : v;
  }
  return v;
}

__device__ __forceinline__ float log_sigmoid(float l) {
  return fminf(l, 0.0f) - log1pf(expf(-fabsf(l)));
}
__device__ __forceinline__ float sigmoid(float l) { return 1.0f / (1.0f + expf(-l)); }

// Normalised weights over the chosen logits, one in each of the first `top` lanes; `there`: a choice
// was left for this lane.
__device__ __forceinline__ float normalised(float l, bool there, int score) {
  const float a = score == COLL_SCORE_SIGMOID ? log_sigmoid(l) : l;
  const float most = warp_max(there ? a : -INFINITY);
  const float x = there ? expf(a - most) : 0.0f;
  return there ? x / warp_sum(x) : (warp_sum(x), 0.0f);
}

// Expert i * 32 + lane in v[i].
template <int V>
__device__ __forceinline__ void load_row(const RouteParams &p, int64_t row, int lane,
                                         float (&v)[V]) {
  const int64_t at = row * p.logits.rs + (int64_t)lane * p.logits.cs;
#pragma unroll
  for (int i = 0; i < V; ++i)
    v[i] = i * 32 + lane < p.e ? ld_elem(p.logits.p, at + (int64_t)(i * 32) * p.logits.cs, p.type)
                               : -INFINITY;
}

template <int V>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(const RouteParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  griddep_launch();
  griddep_wait();
  if (row >= p.t) return;
  float v[V];
  load_row<V>(p, row, lane, v);
  uint32_t key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) key[i] = order_key(v[i]);
  float chosen = -INFINITY;
  int id = -1;
  for (int j = 0; j < p.top; ++j) {
    uint32_t best = 0u;
    int at = 0;
#pragma unroll
    for (int i = V - 1; i >= 0; --i)
      if (key[i] >= best) best = key[i], at = i;
    const uint32_t most = __reduce_max_sync(~0u, best);
    if (most == 0u) break;
    const uint32_t first =
        __reduce_min_sync(~0u, best == most ? (uint32_t)(at * 32 + lane) : ~0u);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if ((uint32_t)(i * 32 + lane) == first) key[i] = 0u;
    if (lane == j) {
      id = (int)first;
      chosen = key_value(most);
    }
  }
  const bool there = id >= 0;
  float w;
  if (p.norm) {
    w = normalised(chosen, there, p.score);
  } else if (p.score == COLL_SCORE_SIGMOID) {
    w = sigmoid(chosen);
  } else {
    const float most = __shfl_sync(~0u, chosen, 0);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) sum += expf(v[i] - most);
    w = expf(chosen - most) / warp_sum(sum);
  }
  if (lane < p.top) {
    p.ids[row * p.ids_rs + lane * p.ids_cs] = id;
    p.weights[row * p.w_rs + lane * p.w_cs] = there ? w * p.scale : 0.0f;
  }
}

// With g = scale dweights over the chosen, w the normalised weights, p or s the scores:
//   normalised softmax  dl_j = w_j (g_j - sum g w);      sigmoid, normalised  the same times 1 - s_j
//   softmax             dl_e = p_e ([e chosen] g_e - sum g p);        sigmoid  dl_j = g_j s_j (1 - s_j)
// 1 - s is the sigmoid of -l. Logits not chosen get 0 but for the plain softmax. Chosen twice, an
// expert gets both gradients (and a normalised weight for each).
template <int V>
__global__ void __launch_bounds__(kWarps * 32) route_bwd_kernel(const RouteParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  griddep_launch();
  griddep_wait();
  if (row >= p.t) return;
  int id = -1;
  float g = 0.0f, l = -INFINITY;
  if (lane < p.top) {
    id = p.ids[row * p.ids_rs + lane * p.ids_cs];
    g = p.weights[row * p.w_rs + lane * p.w_cs] * p.scale;
  }
  const bool there = (uint32_t)id < (uint32_t)p.e;
  if (there) l = ld_elem(p.logits.p, row * p.logits.rs + id * p.logits.cs, p.type);
  float v[V], d;
  if (p.norm) {
    const float w = normalised(l, there, p.score);
    const float sum = warp_sum(there ? g * w : 0.0f);
    d = w * (g - sum);
    if (p.score == COLL_SCORE_SIGMOID) d *= sigmoid(-l);
  } else if (p.score == COLL_SCORE_SIGMOID) {
    d = g * sigmoid(l) * sigmoid(-l);
  } else {
    load_row<V>(p, row, lane, v);
    float most = v[0];
#pragma unroll
    for (int i = 1; i < V; ++i) most = v[i] > most || v[i] != v[i] ? v[i] : most;
    most = warp_max(most);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      v[i] = most == -INFINITY ? 0.0f : expf(v[i] - most);
      sum += v[i];
    }
    sum = warp_sum(sum);
    const float r = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
    d = there && most != -INFINITY ? expf(l - most) * r * g : 0.0f;
    const float all = warp_sum(d);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] *= -all * r;
  }
  if (p.norm || p.score == COLL_SCORE_SIGMOID) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = 0.0f;
  }
  if (!there) d = 0.0f;
  for (int j = 0; j < p.top; ++j) {
    const int e = __shfl_sync(~0u, id, j);
    const float x = __shfl_sync(~0u, d, j);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i * 32 + lane == e) v[i] += x;
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (i * 32 + lane < p.e) st_elem(p.dlogits, row * p.dl_rs + i * 32 + lane, v[i], p.type);
}

template <bool BWD>
cudaError_t launch(const RouteParams &p, cudaStream_t s) {
  const dim3 grid((unsigned)((p.t + kWarps - 1) / kWarps));
#define COLL_ROUTE(V)                                                                        \
  return BWD ? dense_launch(route_bwd_kernel<V>, grid, kWarps * 32, 0, 1, s, p) \
             : dense_launch(route_kernel<V>, grid, kWarps * 32, 0, 1, s, p)
  if (p.e <= 32) COLL_ROUTE(1);
  if (p.e <= 64) COLL_ROUTE(2);
  if (p.e <= 128) COLL_ROUTE(4);
  if (p.e <= 256) COLL_ROUTE(8);
  if (p.e <= 512) COLL_ROUTE(16);
  COLL_ROUTE(32);
#undef COLL_ROUTE
}

template <typename T>
int check_sizes(const T &a) {
  if (a.t < 0 || a.t > 0x7FFFFFFF - 4096 || a.top < 1 || a.top > kMostChosen || a.e < a.top ||
      a.e > kMostExperts)
    return COLL_EINVAL;
  if (!is_half(a.dtype) && a.dtype != COLL_F32) return COLL_EINVAL;
  if (a.score != COLL_SCORE_SOFTMAX && a.score != COLL_SCORE_SIGMOID) return COLL_EINVAL;
  return (a.normalize == 0 || a.normalize == 1) && isfinite(a.scale) ? COLL_OK : COLL_EINVAL;
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
