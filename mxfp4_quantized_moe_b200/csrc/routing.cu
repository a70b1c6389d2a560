// Expert routing with softmax or sigmoid scores, a balance bias, groups and renormalised
// weights, its gradient, and the import of a caller's routing into the block's workspace.
// Definitions at mxfp4_moe_route and mxfp4_moe_route_backward in include/mxfp4_moe.h.
#include <cfloat>

#include "block_edge.h"
#include "common.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kWarps = 8;  // tokens in flight per block, one warp each

struct RouteArgs {
  int T, E, k;
  int groups, gsize, top_groups;
  uint32_t gmagic;   // e / gsize = e * gmagic >> 16 for e < 256
  bool sigmoid, best2, renorm;
  float scale, inv_scale;
  const float* logits;
  const float* bias;
  int32_t* idx;
  float* w;
  int32_t* counts;
};

// A masked logit or bias: NaN, -inf or the lowest finite value.
MOE_DEV bool absent(float v) { return !(v > -FLT_MAX); }

// Order-preserving integer keys, above 1 for every finite value that is not -FLT_MAX.  0 is
// kept for experts out of the choice, 1 for masked experts of the kept groups.
MOE_DEV uint32_t order_bits(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);  // -0 ranks with +0
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
MOE_DEV float order_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
MOE_DEV uint64_t order_bits(double x) {
  const uint64_t b = (uint64_t)__double_as_longlong(x + 0.0);
  return (b >> 63) ? ~b : (b | (1ull << 63));
}
MOE_DEV double order_value(uint64_t k) {
  return __longlong_as_double((long long)((k >> 63) ? (k & ~(1ull << 63)) : ~k));
}
template <class F> struct KeyOf;
template <> struct KeyOf<float> { using type = uint32_t; };
template <> struct KeyOf<double> { using type = uint64_t; };

MOE_DEV uint32_t warp_max(uint32_t v) { return __reduce_max_sync(kFull, v); }
MOE_DEV uint64_t warp_max(uint64_t v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const uint64_t u = __shfl_xor_sync(kFull, v, o);
    v = u > v ? u : v;
  }
  return v;
}
template <class F>
MOE_DEV F warp_sum(F v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
MOE_DEV float warp_maxf(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}
MOE_DEV float exp_of(float x) { return expf(x); }
MOE_DEV double exp_of(double x) { return exp(x); }

// Bounds on what the fp32 keys may be off.  A sigmoid or softmax score in [0, 1] is within
// 2^-20 of its value (expf 2 ulp, at most eight sums in sequence, a division, and the rounding
// of the exponent, |x| e^x 2^-24 <= 2^-25), and adding the bias rounds by 2^-24 of the key.
// Two keys further apart than twice that are in order; these are twice that again.
MOE_DEV float key_margin(float key) { return 0x1p-18f + 0x1p-22f * fabsf(key); }
MOE_DEV float group_margin(float score) { return 0x1p-17f + 0x1p-21f * fabsf(score); }

// One token's logits over the lanes of a warp: lane l holds experts l NG .. l NG + NG - 1.
template <int NG>
struct Token {
  float l[NG];       // +inf clamped to the largest finite value
  float b[NG];
  uint32_t present;  // bit i: expert exists
  uint32_t masked;   // bit i: left out of the choice (logit or bias)
  uint32_t lmasked;  // bit i: logit masked (scores 0)
};

// Selection slots: lane j % 32 holds selection j in slot j / 32.
template <int NS>
struct Picked {
  int e[NS];
  float l[NS];
  bool ok[NS];
};

// Softmax statistics of the token: maximum over the unmasked logits and the sum of exps.
template <class F, int NG>
MOE_DEV void softmax_stats(const Token<NG>& t, float& top, F& total) {
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < NG; ++i)
    if (!((t.lmasked >> i) & 1)) m = fmaxf(m, t.l[i]);
  top = warp_maxf(m);
  F z = 0;
#pragma unroll
  for (int i = 0; i < NG; ++i)
    if (!((t.lmasked >> i) & 1)) z += exp_of((F)t.l[i] - (F)top);
  total = warp_sum(z);
}

// The k selections with keys of type F.  Returns false when F = float cannot decide an order
// within its error (the caller repeats with double).  `buf`: E values of F per warp in shared
// memory (group scores).
template <class F, int NG, int NS>
MOE_DEV bool select(const RouteArgs& a, const Token<NG>& t, F* buf, Picked<NS>& p) {
  using K = typename KeyOf<F>::type;
  constexpr bool fast = sizeof(F) == 4;
  const int lane = threadIdx.x & 31;
  const bool approx = a.bias != nullptr;  // without a bias the keys are the logits, exact
  const bool score_groups = a.groups > 1;
  F s[NG];
  if (approx || (score_groups && a.best2)) {
    float top = 0.f;
    F total = 1;
    if (!a.sigmoid) softmax_stats<F, NG>(t, top, total);
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      const F x = (F)t.l[i];
      s[i] = ((t.lmasked >> i) & 1) ? (F)0
             : a.sigmoid            ? (F)1 / ((F)1 + exp_of(-x))
                                    : exp_of(x - (F)top) / total;
    }
  }
  K key[NG];
#pragma unroll
  for (int i = 0; i < NG; ++i) {
    const F v = approx ? s[i] + (F)t.b[i] : (F)t.l[i];
    key[i] = !((t.present >> i) & 1) ? (K)0 : ((t.masked >> i) & 1) ? (K)1 : order_bits(v);
  }
  if (score_groups) {
    // group scores: the keys (the scores, without a bias and for sums) through shared memory,
    // lane g scanning group g from a start of its own so that the lanes meet different banks
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      const int e = lane * NG + i;
      if (e < a.E)
        buf[e] = ((t.masked >> i) & 1) ? (F)-INFINITY
                 : approx              ? s[i] + (F)t.b[i]
                 : a.best2             ? s[i]
                                       : (F)t.l[i];
    }
    __syncwarp();
    F m1 = (F)-INFINITY, m2 = (F)-INFINITY;
    if (lane < a.groups) {
      const F* mine = buf + lane * a.gsize;
      int at = lane % a.gsize;
      for (int i = 0; i < a.gsize; ++i) {
        const F v = mine[at];
        at = at + 1 == a.gsize ? 0 : at + 1;
        m2 = v > m1 ? m1 : (v > m2 ? v : m2);
        m1 = v > m1 ? v : m1;
      }
    }
    __syncwarp();
    const F score = m1 + ((a.best2 && m2 > (F)-INFINITY) ? m2 : (F)0);
    int rank = 0;
    for (int g = 0; g < a.groups; ++g) {
      const F o = __shfl_sync(kFull, score, g);
      rank += (o > score || (o == score && g < lane)) ? 1 : 0;
    }
    const bool mine = lane < a.groups;
    const unsigned kept = __ballot_sync(kFull, mine && rank < a.top_groups);
    if (fast && (approx || a.best2) && a.top_groups < a.groups) {
      const unsigned in = __ballot_sync(kFull, mine && rank == a.top_groups - 1);
      const unsigned out = __ballot_sync(kFull, mine && rank == a.top_groups);
      const F si = __shfl_sync(kFull, score, __ffs(in) - 1);
      const F so = __shfl_sync(kFull, score, __ffs(out) - 1);
      if (so > (F)-INFINITY && si - so <= (F)group_margin((float)si)) return false;
    }
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      const uint32_t g = ((uint32_t)(lane * NG + i) * a.gmagic) >> 16;
      if (!((t.present >> i) & 1) || !((kept >> g) & 1u)) key[i] = 0;
    }
  }
  // k rounds: the lane's best remaining key (its first on a tie), the warp's largest, the
  // lowest lane that holds it
  K prev = 0;
  float prev_l = 0.f, prev_b = 0.f;
  for (int j = 0; j < a.k; ++j) {
    K best = key[0];
    int bi = 0;
#pragma unroll
    for (int i = 1; i < NG; ++i)
      if (key[i] > best) {
        best = key[i];
        bi = i;
      }
    const K top = warp_max(best);
    const int src = __ffs(__ballot_sync(kFull, best == top)) - 1;
    float bl = t.l[0], bb = t.b[0];
#pragma unroll
    for (int i = 1; i < NG; ++i)
      if (bi == i) {
        bl = t.l[i];
        bb = t.b[i];
      }
    if (lane == src) {
#pragma unroll
      for (int i = 0; i < NG; ++i)
        if (bi == i) key[i] = 0;
    }
    const int e = __shfl_sync(kFull, lane * NG + bi, src);
    const float l = __shfl_sync(kFull, bl, src);
    if (fast && approx && top > 1) {
      const float b = __shfl_sync(kFull, bb, src);
      if (j > 0) {
        const float v = (float)order_value(top);
        // experts with equal logit and bias tie in any precision
        if ((float)order_value(prev) - v <= key_margin(v) && !(l == prev_l && b == prev_b))
          return false;
      }
      prev = top;
      prev_l = l;
      prev_b = b;
    }
    if (lane == (j & 31)) {
#pragma unroll
      for (int q = 0; q < NS; ++q)
        if (q == (j >> 5)) {
          p.e[q] = e;
          p.l[q] = l;
          p.ok[q] = top > 1;
        }
    }
  }
  if (fast && approx && prev > 1) {  // an expert left out within reach of the last one chosen
    const float v = (float)order_value(prev);
    const float m = key_margin(v);
    bool near = false;
#pragma unroll
    for (int i = 0; i < NG; ++i)
      near |= key[i] > 1 && v - (float)order_value(key[i]) <= m &&
              !(t.l[i] == prev_l && t.b[i] == prev_b);
    if (__any_sync(kFull, near)) return false;
  }
  return true;
}

// One warp per token.  Reads 4 E bytes and writes 8 k bytes a token; the k rounds of warp
// reductions bound it, not the bytes.
template <int NG, int NS>
__global__ void __launch_bounds__(32 * kWarps) route_kernel(RouteArgs a) {
  __shared__ double s_buf[kWarps][32 * NG];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long row = (long long)blockIdx.x * kWarps + warp;
  if (row >= a.T) return;  // warp-uniform
  Token<NG> t;
  t.present = t.masked = t.lmasked = 0;
#pragma unroll
  for (int i = 0; i < NG; ++i) {
    const int e = lane * NG + i;
    const bool in = e < a.E;
    const float l = in ? __ldg(a.logits + row * a.E + e) : -INFINITY;
    const float b = in && a.bias ? __ldg(a.bias + e) : 0.f;
    const bool lm = absent(l);
    t.present |= (uint32_t)in << i;
    t.lmasked |= (uint32_t)lm << i;
    t.masked |= (uint32_t)(lm || absent(b)) << i;
    t.l[i] = fminf(l, FLT_MAX);
    t.b[i] = fminf(b, FLT_MAX);
  }
  Picked<NS> p;
#pragma unroll
  for (int q = 0; q < NS; ++q) p.ok[q] = false;
  if (!select<float, NG, NS>(a, t, reinterpret_cast<float*>(s_buf[warp]), p)) {
    __syncwarp();
    select<double, NG, NS>(a, t, s_buf[warp], p);
  }
  // weights of the lane's selections
  float w[NS];
  if (a.renorm) {
    // s_j / sum s_i as a softmax over log s_j: no score underflows.  log sigmoid(l) =
    // min(l, 0) - log(1 + e^-|l|); the softmax's own denominator cancels.
    float v[NS], m = -INFINITY;
#pragma unroll
    for (int q = 0; q < NS; ++q) {
      v[q] = -INFINITY;
      if (p.ok[q]) v[q] = a.sigmoid ? fminf(p.l[q], 0.f) - log1pf(expf(-fabsf(p.l[q]))) : p.l[q];
      m = fmaxf(m, v[q]);
    }
    m = warp_maxf(m);
    float sum = 0.f;
#pragma unroll
    for (int q = 0; q < NS; ++q) {
      w[q] = p.ok[q] ? expf(v[q] - m) : 0.f;
      sum += w[q];
    }
    sum = warp_sum(sum);
    const float c = m > -INFINITY ? a.scale / sum : 0.f;
#pragma unroll
    for (int q = 0; q < NS; ++q) w[q] *= c;
  } else if (a.sigmoid) {
#pragma unroll
    for (int q = 0; q < NS; ++q) w[q] = p.ok[q] ? a.scale / (1.f + expf(-p.l[q])) : 0.f;
  } else {
    float top, total;
    softmax_stats<float, NG>(t, top, total);
#pragma unroll
    for (int q = 0; q < NS; ++q) w[q] = p.ok[q] ? a.scale * (expf(p.l[q] - top) / total) : 0.f;
  }
#pragma unroll
  for (int q = 0; q < NS; ++q) {
    const int j = lane + 32 * q;
    if (j < a.k) {
      a.idx[row * a.k + j] = p.e[q];
      a.w[row * a.k + j] = w[q];
      if (a.counts) atomicAdd(a.counts + p.e[q], 1);
    }
  }
}

// One warp per token: the row of d_logits is filled by the lanes together (zeros, or the dense
// part of the softmax's gradient), then the k selected entries are added.
template <int NG>
__global__ void __launch_bounds__(32 * kWarps) route_backward_kernel(
    RouteArgs a, const float* __restrict__ d_w, float* __restrict__ d_logits) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long row = (long long)blockIdx.x * kWarps + warp;
  if (row >= a.T) return;  // warp-uniform
  const float* lg = a.logits + row * a.E;
  const int32_t* idx = a.idx + row * a.k;
  const float* w = a.w + row * a.k;
  const float* dw = d_w + row * a.k;
  float dot = 0.f;  // sum_j w_j dw_j; a weight of exactly 0 (masked) takes no part
  for (int j = lane; j < a.k; j += 32) {
    const float wj = w[j];
    dot += wj != 0.f ? wj * dw[j] : 0.f;
  }
  dot = warp_sum(dot);
  const bool dense = !a.sigmoid && !a.renorm;
  float out[NG];
#pragma unroll
  for (int i = 0; i < NG; ++i) out[i] = 0.f;
  if (dense) {
    float l[NG], m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      const int e = lane + 32 * i;
      const float v = e < a.E ? __ldg(lg + e) : -INFINITY;
      l[i] = absent(v) ? -INFINITY : fminf(v, FLT_MAX);
      m = fmaxf(m, l[i]);
    }
    m = warp_maxf(m);
    if (m > -INFINITY) {
      float z = 0.f;
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        l[i] = l[i] > -INFINITY ? expf(l[i] - m) : 0.f;
        z += l[i];
      }
      z = warp_sum(z);
      const float c = -dot / z;
#pragma unroll
      for (int i = 0; i < NG; ++i) out[i] = c * l[i];
    }
  }
  const float shared = a.renorm ? dot * a.inv_scale : 0.f;
  for (int j0 = 0; j0 < a.k; j0 += 32) {
    const int j = j0 + lane;
    int e = -1;
    float q = 0.f;
    if (j < a.k) {
      const float wj = w[j];
      e = idx[j];
      if (wj != 0.f && e >= 0 && e < a.E) {
        q = wj * (dw[j] - shared);
        if (a.sigmoid) q /= 1.f + expf(__ldg(lg + e));  // 1 - sigmoid(l)
      }
    }
    const int n = min(32, a.k - j0);
    for (int i0 = 0; i0 < n; ++i0) {
      const int ee = __shfl_sync(kFull, e, i0);
      const float qq = __shfl_sync(kFull, q, i0);
#pragma unroll
      for (int i = 0; i < NG; ++i)
        if (ee == lane + 32 * i) out[i] += qq;
    }
  }
  float* o = d_logits + row * a.E;
#pragma unroll
  for (int i = 0; i < NG; ++i)
    if (lane + 32 * i < a.E) o[lane + 32 * i] = out[i];
}

// One block per 32-token segment: slots copied, checked and counted per expert.
constexpr int kSegTokens = 32;
__global__ void __launch_bounds__(256) import_routing_kernel(
    const int32_t* __restrict__ topk_idx, const float* __restrict__ topk_w, int T, int E, int k,
    int32_t* __restrict__ idx, float* __restrict__ w, int32_t* __restrict__ hist, int* err) {
  __shared__ int s_hist[256];
  const int seg = blockIdx.x;
  for (int e = threadIdx.x; e < E; e += 256) s_hist[e] = 0;
  __syncthreads();
  const size_t s0 = (size_t)seg * kSegTokens * k;
  const int n = min(kSegTokens, T - seg * kSegTokens) * k;
  for (int i = threadIdx.x; i < n; i += 256) {
    int e = __ldg(topk_idx + s0 + i);
    float v = __ldg(topk_w + s0 + i);
    if (e < 0 || e >= E) {
      DevErr{err}.set(MXFP4_MOE_ERR_DEVICE_BOUNDS, 0x120);
      e = 0;
      v = 0.f;
    }
    idx[s0 + i] = e;
    w[s0 + i] = v;
    atomicAdd(s_hist + e, 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += 256) hist[(size_t)seg * E + e] = s_hist[e];
}

RouteArgs route_args(const mxfp4_moe_routing& r) {
  RouteArgs a{};
  a.T = r.T; a.E = r.E; a.k = r.k;
  a.groups = r.groups; a.gsize = r.E / r.groups; a.top_groups = r.top_groups;
  a.gmagic = (65536u + (uint32_t)a.gsize - 1) / (uint32_t)a.gsize;
  a.sigmoid = r.scores == MXFP4_MOE_SCORES_SIGMOID;
  a.best2 = r.group_best == 2;
  a.renorm = r.renormalize != 0;
  a.scale = r.scale;
  a.inv_scale = 1.f / r.scale;
  return a;
}

}  // namespace

cudaError_t launch_route(const mxfp4_moe_routing& r, const float* logits, const float* bias,
                         int32_t* idx, float* w, int32_t* counts, int, cudaStream_t st) {
  if (counts) {
    const cudaError_t e = cudaMemsetAsync(counts, 0, 4 * (size_t)r.E, st);
    if (e != cudaSuccess) return e;
  }
  if (r.T == 0) return cudaSuccess;
  RouteArgs a = route_args(r);
  a.logits = logits; a.bias = bias; a.idx = idx; a.w = w; a.counts = counts;
  const int ng = (r.E + 31) / 32;
  const bool one = r.k <= 32;
  auto kern = ng <= 1   ? route_kernel<1, 1>
              : ng <= 2 ? (one ? route_kernel<2, 1> : route_kernel<2, 2>)
              : ng <= 4 ? (one ? route_kernel<4, 1> : route_kernel<4, 4>)
                        : (one ? route_kernel<8, 1> : route_kernel<8, 8>);
  kern<<<(unsigned)(((long long)r.T + kWarps - 1) / kWarps), 32 * kWarps, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_route_backward(const mxfp4_moe_routing& r, const float* logits,
                                  const int32_t* idx, const float* w, const float* d_w,
                                  float* d_logits, cudaStream_t st) {
  if (r.T == 0) return cudaSuccess;
  RouteArgs a = route_args(r);
  a.logits = logits;
  a.idx = const_cast<int32_t*>(idx);
  a.w = const_cast<float*>(w);
  const int ng = (r.E + 31) / 32;
  auto kern = ng <= 1   ? route_backward_kernel<1>
              : ng <= 2 ? route_backward_kernel<2>
              : ng <= 4 ? route_backward_kernel<4>
                        : route_backward_kernel<8>;
  kern<<<(unsigned)(((long long)r.T + kWarps - 1) / kWarps), 32 * kWarps, 0, st>>>(a, d_w, d_logits);
  return cudaGetLastError();
}

cudaError_t launch_import_routing(const int32_t* topk_idx, const float* topk_w, int T, int E,
                                  int k, int32_t* idx, float* w, int32_t* scratch, int* err,
                                  cudaStream_t st) {
  import_routing_kernel<<<route_blocks(T), 256, 0, st>>>(topk_idx, topk_w, T, E, k, idx, w,
                                                          scratch, err);
  return cudaGetLastError();
}

}  // namespace moe
