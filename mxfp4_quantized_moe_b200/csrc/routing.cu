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

MOE_DEV bool valid_expert(int e, int E) { return e >= 0 && e < E; }

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
constexpr float kLog2e = 1.4426950408889634f;
MOE_DEV float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
MOE_DEV float exp_of(float x) { return expf(x); }
MOE_DEV double exp_of(double x) { return exp(x); }

// Bounds on what the fp32 keys may be off.  A sigmoid or softmax score in [0, 1] is within
// 2^-20 of its value (expf 2 ulp, at most eight sums in sequence, a division, and the rounding
// of the exponent, |x| e^x 2^-24 <= 2^-25), and adding the bias rounds by 2^-24 of the key.
// Two keys further apart than twice that are in order; this is twice that again.
MOE_DEV float key_margin(float key) { return 0x1p-18f + 0x1p-22f * fabsf(key); }
// A group's score is the sum of its keys m1 and m2 (m2 = 0: m1 alone).  Key i is off by what its
// score is, and rounds by 2^-24 |m_i|; the largest and the second largest of several keys are off by
// no more than that, since value + bound and value - bound rise with the value; and the sum rounds
// by 2^-24 (|m1| + |m2|).  In all `scores`, what two scores may be off together, and
// 2^-23 (|m1| + |m2|): relative to the keys, not to a sum in which they may cancel.  Twice the
// latter, for the rounding of score - slack and score + slack as well; each product by itself, so
// that keys near the largest value do not overflow.
MOE_DEV float group_slack(float m1, float m2, float scores) {
  return scores + (0x1p-22f * fabsf(m1) + 0x1p-22f * fabsf(m2));
}

// One token's logits over the lanes of a warp: lane l holds experts l NG .. l NG + NG - 1.
template <int NG>
struct Token {
  float l[NG];       // +inf clamped to the largest finite value
  float b[NG];
  uint32_t present;  // bit i: expert exists
  uint32_t masked;   // bit i: left out of the choice (logit or bias)
  uint32_t lmasked;  // bit i: logit masked (scores 0)
};

template <int NG>
MOE_DEV void load_token(const RouteArgs& a, long long row, Token<NG>& t) {
  t.present = t.masked = t.lmasked = 0;
#pragma unroll
  for (int i = 0; i < NG; ++i) {
    const int e = (threadIdx.x & 31) * NG + i;
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
}

// log s up to the token's constant: renormalised weights are a softmax over it, so that no score
// underflows.  log sigmoid(l) = min(l, 0) - log(1 + e^-|l|); the softmax's denominator cancels.
MOE_DEV float log_score(float l, bool sigmoid) {
  return sigmoid ? fminf(l, 0.f) - log1pf(expf(-fabsf(l))) : l;
}

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
    if (!(a.best2 && m2 > (F)-INFINITY)) m2 = 0;
    const F score = m1 + m2;
    int rank = 0;
    for (int g = 0; g < a.groups; ++g) {
      const F o = __shfl_sync(kFull, score, g);
      rank += (o > score || (o == score && g < lane)) ? 1 : 0;
    }
    const bool mine = lane < a.groups;
    const unsigned kept = __ballot_sync(kFull, mine && rank < a.top_groups);
    if (fast && (approx || a.best2) && a.top_groups < a.groups) {
      // Every kept group must lie above every other one by what both may be off.  Groups without
      // experts, at -inf, do not count; a sum below what fp32 holds is not one of those.
      const bool some = mine && m1 > (F)-INFINITY, sunk = some && !(score > (F)-INFINITY);
      const float slack = some ? group_slack((float)m1, (float)m2, 0x1p-18f) : 0.f;
      const float low = mine && rank < a.top_groups ? (float)score - slack : INFINITY;
      const float high = sunk ? INFINITY : some && rank >= a.top_groups ? (float)score + slack : -INFINITY;
      const uint32_t out = warp_max(order_bits(high)), in = ~warp_max(~order_bits(low));
      if (out > order_bits(-INFINITY) && in <= out) return false;
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

// One warp per token, for k > 8 and for groups that are no whole slots or more than 8.  Reads 4 E
// bytes and writes 8 k bytes a token; the k rounds of warp reductions bound it, and the scan of a
// group by one lane, not the bytes.  T = 32768: E = 256, k = 8, without groups (forced into this
// form) 61 us without a bias and 88 with one, against 14 and 21 in the form for four tokens below;
// E = 160, k = 6, 3 of 8 groups 84 and 105 us; E = 256, k = 8, 4 of 32 groups with a bias 120 us;
// k = 16 without groups 93 and 130 us.
template <int NG, int NS>
__global__ void __launch_bounds__(32 * kWarps) route_kernel(RouteArgs a) {
  __shared__ double s_buf[kWarps][32 * NG];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long row = (long long)blockIdx.x * kWarps + warp;
  if (row >= a.T) return;  // warp-uniform
  Token<NG> t;
  load_token<NG>(a, row, t);
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
    float v[NS], m = -INFINITY;
#pragma unroll
    for (int q = 0; q < NS; ++q) {
      v[q] = -INFINITY;
      if (p.ok[q]) v[q] = log_score(p.l[q], a.sigmoid);
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

// ---- four tokens per warp ---------------------------------------------------------------------
// The form for k <= 8 (and groups, if any, of whole slots): eight lanes hold a token, lane q its
// experts q, q + 8, ...  Each key becomes one 32-bit word, its place within the token's range of
// keys in 23 bits above 255 - expert, so that words order by key and then by lower index, and a
// compare-exchange is two instructions.  Words are sorted in registers (Batcher's odd-even merge
// sort of K2 at a time), and two descending lists merge by max(a_i, b_{K2-1-i}), the K2 largest
// of both, which a bitonic half-cleaner sorts; three such merges across lanes leave the token's
// K2 largest in all eight.  Where the 23 bits (or fp32 keys) cannot decide an order, sigmoid keys
// of the chosen experts and at most one other are compared in fp64; a token that needs more, or
// has fewer than k unmasked experts, goes through select() instead.  Bound by the ALU pipe
// (min / max, compares, selects: half its slots) and latency, not by the bytes.  T = 32768, E = 256,
// k = 8: softmax 14 us, sigmoid with a bias 21 us, with 4 of 8 groups 26-28 us (by the draw: a
// few rows go to fp64, and a wider margin, with more of them, measures slower), where the logits'
// bytes alone take 5.4 us.
template <int N>
MOE_DEV void exchange(uint32_t (&v)[N], int i, int j) {  // the larger to i
  const uint32_t a = max(v[i], v[j]), b = min(v[i], v[j]);
  v[i] = a;
  v[j] = b;
}
template <int N>
MOE_DEV void sort_words(uint32_t (&v)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) exchange(v, i + j, i + j + k);
}
template <int N>  // a := the N largest of a and b, both descending
MOE_DEV void merge_words(uint32_t (&a)[N], const uint32_t (&b)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) a[i] = max(a[i], b[N - 1 - i]);
#pragma unroll
  for (int d = N / 2; d >= 1; d /= 2)
#pragma unroll
    for (int i = 0; i < N; ++i)
      if ((i & d) == 0) exchange(a, i, i + d);
}
// Reductions over a token's eight lanes.
template <class F, class Op>
MOE_DEV F over8(F v, Op op) {
#pragma unroll
  for (int o = 1; o < 8; o *= 2) v = op(v, __shfl_xor_sync(kFull, v, o));
  return v;
}
MOE_DEV float max8(float v) { return over8(v, [](float a, float b) { return fmaxf(a, b); }); }
MOE_DEV float min8(float v) { return over8(v, [](float a, float b) { return fminf(a, b); }); }
MOE_DEV float sum8(float v) { return over8(v, [](float a, float b) { return a + b; }); }

// Two largest of a token's keys, joined.
MOE_DEV void join_two(float& m1, float& m2, float o1, float o2) {
  m2 = fmaxf(fminf(m1, o1), fmaxf(m2, o2));
  m1 = fmaxf(m1, o1);
}

// G: groups when a group is NS / G whole slots and E = 8 NS (a folded reduction then gives lane q
// the score of group q), 1 without groups, 0 for other groups of whole slots.  WHOLE: E = 8 NS.
template <int NS, int K2, int G, bool WHOLE>
__global__ void __launch_bounds__(128, NS == 32 ? 6 : 8) route4_kernel(RouteArgs a) {
  constexpr int NG = NS / 4;  // experts a lane holds in select()
  __shared__ double s_buf[4][32 * NG];
  __shared__ float s_bias[8 * NS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int q = lane & 7, tok = lane >> 3;
  const long long row0 = ((long long)blockIdx.x * (blockDim.x >> 5) + warp) * 4;
  const bool live = row0 + tok < a.T;
  const long long row = live ? row0 + tok : a.T - 1;  // dead lanes repeat the last token
  const float* lg = a.logits + row * a.E;
  // keys are scores where a bias or a group's sum needs them, else the logits
  const bool scored = a.bias != nullptr || (G != 1 && a.best2);
  // masked and missing experts hold the lowest finite value, below every other key; a token with
  // a logit of +inf is left to select()
  float x[NS];
#pragma unroll
  for (int i = 0; i < NS; ++i) x[i] = WHOLE || 8 * i + q < a.E ? __ldg(lg + 8 * i + q) : -FLT_MAX;
  if (scored) {
    float b[NS / 4];  // all requested before the first is stored (one warp alone takes them all)
#pragma unroll
    for (int i = 0; i < NS / 4; ++i) {
      const int e = threadIdx.x + i * blockDim.x;
      b[i] = a.bias && e < a.E ? __ldg(a.bias + e) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < NS / 4; ++i) {
      const int e = threadIdx.x + i * blockDim.x;
      if (e < 8 * NS) s_bias[e] = fminf(fmaxf(b[i], -FLT_MAX), FLT_MAX);
    }
    __syncthreads();
  }
  if (row0 >= a.T) return;  // warp-uniform
#pragma unroll
  for (int i = 0; i < NS; ++i) x[i] = fmaxf(x[i], -FLT_MAX);
  // softmax statistics where scores or weights need them
  float top = 0.f, total = 1.f;
  if (!a.sigmoid && (scored || !a.renorm)) {
    float m = x[0];
#pragma unroll
    for (int i = 1; i < NS; ++i) m = fmaxf(m, x[i]);
    top = max8(m);
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < NS; ++i) z += expf(x[i] - top);
    total = sum8(z);
  }
  // Scores as keys.  ex2.approx and rcp.approx are within 2 ulp and 1 ulp, the exponent's
  // rounding moves e^-l by |l| 2^-24: a sigmoid is within 4.3 2^-24 of its value.  A softmax score
  // is within 2^-22, plus what the sum of exps is off: at most 38 2^-24 of the score (31 + 3 sums,
  // expf), in the same direction for all scores of the token.  `unit_margin` bounds what two scores
  // may be off against one another, its double what two sums of two scores may.
  const float inv_total = 1.f / total;
  auto score = [&](float l) {
    if (!a.sigmoid) return exp2_approx((l - top) * kLog2e) * inv_total;
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + exp2_approx(-kLog2e * l)));
    return r;
  };
  if (scored) {
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      x[i] = x[i] > -FLT_MAX ? score(x[i]) + s_bias[8 * i + q] : -FLT_MAX;
    }
  }
  const float unit_margin = 0x1p-20f + (a.sigmoid ? 0.f : 0x1p-18f * inv_total);
  bool unsure = !(top < INFINITY);
  if constexpr (G != 1) {
    float mine = -FLT_MAX;  // lane q: score of group q, and how far it may be off
    float slack = 0.f;
    auto total_of = [&](float m1, float m2) {
      if (!(a.best2 && m2 > -FLT_MAX)) m2 = 0.f;
      mine = m1 + m2;
      slack = m1 > -FLT_MAX ? group_slack(m1, m2, unit_margin) : 0.f;
    };
    int span = 0;
    float v1[G ? G : 1], v2[G ? G : 1];
    if constexpr (G > 1) {
      constexpr int kSpan = NS / G;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        v1[g] = v2[g] = -FLT_MAX;
#pragma unroll
        for (int i = 0; i < kSpan; ++i) {
          const float v = x[g * kSpan + i];
          v2[g] = fmaxf(v2[g], fminf(v1[g], v));
          v1[g] = fmaxf(v1[g], v);
        }
      }
      // halve the groups a lane keeps while joining it with the lane that keeps the others
#pragma unroll
      for (int n = G / 2, o = 4; o >= 1; o /= 2, n /= 2) {
        const bool upper = q & o;
        if (n >= 1) {
#pragma unroll
          for (int g = 0; g < G / 2; ++g)
            if (g < n) {
              const float k1 = upper ? v1[g + n] : v1[g], k2 = upper ? v2[g + n] : v2[g];
              const float s1 = upper ? v1[g] : v1[g + n], s2 = upper ? v2[g] : v2[g + n];
              v1[g] = k1;
              v2[g] = k2;
              join_two(v1[g], v2[g], __shfl_xor_sync(kFull, s1, o), __shfl_xor_sync(kFull, s2, o));
            }
        } else {
          join_two(v1[0], v2[0], __shfl_xor_sync(kFull, v1[0], o), __shfl_xor_sync(kFull, v2[0], o));
        }
      }
      // lane q holds group q / (8 / G)
      const int from = (lane & 24) | (q * (8 / G) & 7);
      total_of(v1[0], v2[0]);
      if constexpr (G < 8) {
        mine = __shfl_sync(kFull, mine, from);
        slack = __shfl_sync(kFull, slack, from);
      }
    } else {
      span = a.gsize >> 3;  // slots of a group
      float m1 = -FLT_MAX, m2 = -FLT_MAX;
      int g = 0, left = span;
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        if (8 * i < a.E) {
          const float v = x[i];
          m2 = fmaxf(m2, fminf(m1, v));
          m1 = fmaxf(m1, v);
          if (--left == 0) {  // the group's two largest over the eight lanes
#pragma unroll
            for (int o = 1; o < 8; o *= 2)
              join_two(m1, m2, __shfl_xor_sync(kFull, m1, o), __shfl_xor_sync(kFull, m2, o));
            if (q == g) total_of(m1, m2);
            ++g;
            left = span;
            m1 = m2 = -FLT_MAX;
          }
        }
      }
    }
    int rank = 0;
#pragma unroll
    for (int o = 1; o < 8; ++o) {
      const int other = (q + o) & 7;
      const float v = __shfl_sync(kFull, mine, (lane & 24) | other);
      rank += other < a.groups && (v > mine || (v == mine && other < q)) ? 1 : 0;
    }
    const bool real = q < a.groups, kept = real && rank < a.top_groups;
    if (scored) {
      // (a sum below the lowest finite value ranks behind groups without experts here; keys that
      // low are beyond the words' range, and select() decides)
      const float in = min8(kept ? mine - slack : INFINITY);
      const float no = max8(real && !kept && mine > -FLT_MAX ? mine + slack : -INFINITY);
      unsure |= no > -INFINITY && !(in > no);
    }
    const uint32_t keep = __ballot_sync(kFull, kept) >> (lane & 24);
    if constexpr (G > 1) {
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int i = 0; i < NS / G; ++i) x[g * (NS / G) + i] = (keep >> g) & 1u ? x[g * (NS / G) + i] : -FLT_MAX;
    } else {
      int g = 0, left = span;
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        x[i] = (keep >> g) & 1u ? x[i] : -FLT_MAX;
        if (--left == 0) {
          ++g;
          left = span;
        }
      }
    }
  }
  // words: the key's place below the largest one, 1 .. 2^23 - 1, above 255 - expert.  The eight
  // lanes' largest keys are eight keys, so the k largest reach down to the least of these (lo):
  // they have the places above 1024, and place 1 (masked, dropped, far below) is never chosen.
  float hi = x[0];
#pragma unroll
  for (int i = 1; i < NS; ++i) hi = fmaxf(hi, x[i]);
  const float lo = min8(hi);
  hi = max8(hi);
  unsure |= !(hi > -FLT_MAX && hi < INFINITY);
  const float range = fminf(fmaxf(hi - lo, 1e-30f), 64.f);
  const float per = 8387582.f / range;
  uint32_t word[NS];
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    const float f = fmaxf(fmaf(x[i] - hi, per, 16777215.f), 8388609.f);
    word[i] = (__float_as_uint(f) << 8) + (uint32_t)(255 - 8 * i - q);
  }
  uint32_t best[K2];
#pragma unroll
  for (int i = 0; i < K2; ++i) best[i] = i < NS ? word[i] : 0u;
  sort_words(best);
#pragma unroll
  for (int c = K2; c < NS; c += K2) {
    uint32_t next[K2];
#pragma unroll
    for (int i = 0; i < K2; ++i) next[i] = word[c + i];
    sort_words(next);
    merge_words(best, next);
  }
#pragma unroll
  for (int o = 1; o < 8; o *= 2) {
    uint32_t next[K2];
#pragma unroll
    for (int i = 0; i < K2; ++i) next[i] = __shfl_xor_sync(kFull, best[i], o);
    merge_words(best, next);
  }
  // lane q takes selection q; the last one bounds what was left out
  uint32_t mine = best[0], last = best[0];
#pragma unroll
  for (int i = 1; i < K2; ++i) {
    mine = q == i ? best[i] : mine;
    last = a.k - 1 == i ? best[i] : last;
  }
  const bool slot = q < a.k;
  int e = slot ? 255 - (int)(mine & 255u) : 0;
  e = e < a.E ? e : 0;
  float l = fminf(__ldg(lg + e), FLT_MAX);
  const float b = a.bias ? __ldg(a.bias + e) : 0.f;
  {
    // places nearer than the keys' error (none for logits) need equal logits and biases
    const uint32_t near =
        scored ? (uint32_t)fminf((unit_margin + 0x1p-22f * (fabsf(hi) + range)) * per, 8388607.f) + 1u : 0u;
    const uint32_t below = __shfl_down_sync(kFull, mine, 1, 8);
    const float l1 = __shfl_down_sync(kFull, l, 1, 8), b1 = __shfl_down_sync(kFull, b, 1, 8);
    bool open = q + 1 < a.k && (mine >> 8) - (below >> 8) <= near && !(l == l1 && b == b1);
    // With place 1 chosen or within reach (masked, missing, too far below) select() decides;
    // else what is within reach has a place, and so a logit
    const bool floor_near = (last >> 8) <= near + 1u;
    unsure |= floor_near;
    const uint32_t reach = floor_near ? last : ((last >> 8) - near) << 8;
    bool close = false;
#pragma unroll
    for (int i = 0; i < NS; ++i) close |= word[i] - reach < last - reach;  // reach <= word < last
    int others = 0, other = 0;  // experts left out within reach of the last one chosen
    bool tied = false;          // one of them equals the last one chosen
    if (__any_sync(kFull, close)) {  // exact ties with the last one are in order
      const float lk = __shfl_sync(kFull, l, (lane & 24) | (a.k - 1));
      const float bk = __shfl_sync(kFull, b, (lane & 24) | (a.k - 1));
#pragma unroll
      for (int i = 0; i < NS; ++i)
        if (word[i] - reach < last - reach) {
          const int o = 8 * i + q;
          if (!(fminf(__ldg(lg + o), FLT_MAX) == lk && (!a.bias || __ldg(a.bias + o) == bk))) {
            ++others;
            other = o;
          } else {
            tied = true;
          }
        }
    }
    open |= others > 0;
    if (!(scored && a.sigmoid)) {
      unsure |= open;
    } else if (__any_sync(kFull, open)) {
      // one or no expert in question beside the chosen ones: all of them by their fp64 keys (an
      // equal of the last one, left out, goes ahead of whatever that one turns out to pass)
      const unsigned opens = (__ballot_sync(kFull, open) >> (lane & 24)) & 0xFFu;
      unsure |= tied && opens != 0u;
      const unsigned have = (__ballot_sync(kFull, others > 0) >> (lane & 24)) & 0xFFu;
      others = (int)sum8((float)others);
      unsure |= others > 1;
      const int oe = __shfl_sync(kFull, other, (lane & 24) | (have ? __ffs(have) - 1 : 0));
      auto key64 = [&](int i) {
        const double v = (double)fminf(__ldg(lg + i), FLT_MAX);
        if (!a.bias) return v;  // scores order like logits, which do not saturate
        return 1.0 / (1.0 + exp(-v)) + (double)fminf(__ldg(a.bias + i), FLT_MAX);
      };
      const double mykey = key64(e), okey = others ? key64(oe) : -1e300;
      const bool before = others && (okey > mykey || (okey == mykey && oe < e));
      int rank = before ? 1 : 0;  // this lane's place among the k chosen and the other one
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const double k = __shfl_sync(kFull, mykey, (lane & 24) | j);
        const int ke = __shfl_sync(kFull, e, (lane & 24) | j);
        rank += j < a.k && j != q && (k > mykey || (k == mykey && ke < e)) ? 1 : 0;
      }
      const unsigned ahead = (__ballot_sync(kFull, slot && !before) >> (lane & 24)) & 0xFFu;
      const int orank = others ? __popc(ahead) : 8;
      int ne = orank == q ? oe : e;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int r = __shfl_sync(kFull, rank, (lane & 24) | j);
        const int je = __shfl_sync(kFull, e, (lane & 24) | j);
        ne = j < a.k && r == q ? je : ne;
      }
      e = slot ? ne : 0;
      l = fminf(__ldg(lg + e), FLT_MAX);
    }
  }
  bool ok = true;
  unsigned again = __ballot_sync(kFull, unsure && live);
  if (again) {
    for (int t = 0; t < 4; ++t) {
      if (!((again >> (8 * t)) & 0xFFu)) continue;  // warp-uniform
      Token<NG> tk;
      load_token<NG>(a, row0 + t, tk);
      Picked<1> p;
      p.ok[0] = false;
      if (scored) select<double, NG, 1>(a, tk, s_buf[warp], p);
      else select<float, NG, 1>(a, tk, reinterpret_cast<float*>(s_buf[warp]), p);
      __syncwarp();
      float ttop = 0.f, ttotal = 1.f;  // infinite logits clamped
      if (!a.sigmoid && !a.renorm) softmax_stats<float, NG>(tk, ttop, ttotal);
      const int pe = __shfl_sync(kFull, p.e[0], q);
      const float pl = __shfl_sync(kFull, p.l[0], q);
      const bool po = __shfl_sync(kFull, (int)p.ok[0], q);
      if (tok == t) {
        e = pe;
        l = pl;
        ok = po;
        top = ttop;
        total = ttotal;
      }
    }
  }
  ok = ok && slot;
  float w;
  if (a.renorm) {
    const float v = !ok ? -INFINITY : log_score(l, a.sigmoid), m = max8(v);
    const float z = ok ? expf(v - m) : 0.f, sum = sum8(z);
    w = m > -INFINITY ? z * (a.scale / sum) : 0.f;
  } else if (a.sigmoid) {
    w = ok ? a.scale / (1.f + expf(-l)) : 0.f;
  } else {
    w = ok ? a.scale * (expf(l - top) / total) : 0.f;
  }
  if (slot && live) {
    a.idx[row * a.k + q] = e;
    a.w[row * a.k + q] = w;
    if (a.counts) atomicAdd(a.counts + e, 1);
  }
}

// Four tokens per warp, for k <= 8: eight lanes hold a token's slots and the vectors q, q + 8, ...
// of its row (V floats each: 4 where E and the pointers allow it).  The row is laid out in shared
// memory (zeros, or the dense part of the softmax's gradient), the selected entries are added
// there, and it leaves in vectors.  Bound by the rows of d_logits: T = 32768, E = 256, k = 8 in 8-10
// us (3.6-4.5 TB/s), 18 us with a warp per token.
template <int NV, int V>
__global__ void __launch_bounds__(128) route4_backward_kernel(RouteArgs a, const float* __restrict__ d_w,
                                                              float* __restrict__ d_logits) {
  struct alignas(4 * V) Vec { float f[V]; };
  __shared__ Vec s_row[4][4][8 * NV];
  __shared__ uint8_t s_tag[4][4][8 * NV * V];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int q = lane & 7, tok = lane >> 3;
  const long long row0 = ((long long)blockIdx.x * (blockDim.x >> 5) + warp) * 4;
  if (row0 >= a.T) return;  // warp-uniform
  const bool live = row0 + tok < a.T;
  const long long row = live ? row0 + tok : a.T - 1;  // dead lanes repeat the last token
  const float* lg = a.logits + row * a.E;
  const int vecs = a.E / V;
  const bool dense = !a.sigmoid && !a.renorm, has = q < a.k;
  const int e = has ? __ldg(a.idx + row * a.k + q) : -1;
  float w = has ? __ldg(a.w + row * a.k + q) : 0.f, dw = has ? __ldg(d_w + row * a.k + q) : 0.f;
  const bool put = valid_expert(e, a.E);
  const float le = a.sigmoid && put && w != 0.f ? __ldg(lg + e) : 0.f;
  Vec row_v[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int u = 0; u < V; ++u) row_v[i].f[u] = 0.f;
  dw = w != 0.f ? dw : 0.f;  // a weight of exactly 0 (masked) takes no part
  const float dot = sum8(w * dw);
  if (dense) {
    float m = -FLT_MAX, z = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = 8 * i + q;
      if (c < vecs) row_v[i] = *reinterpret_cast<const Vec*>(lg + V * c);
#pragma unroll
      for (int u = 0; u < V; ++u) {
        row_v[i].f[u] = c < vecs ? fminf(fmaxf(row_v[i].f[u], -FLT_MAX), FLT_MAX) : -FLT_MAX;
        m = fmaxf(m, row_v[i].f[u]);
      }
    }
    m = max8(m);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int u = 0; u < V; ++u) {
        row_v[i].f[u] = row_v[i].f[u] > -FLT_MAX ? expf(row_v[i].f[u] - m) : 0.f;
        z += row_v[i].f[u];
      }
    z = sum8(z);
    const float scale = z > 0.f ? -dot / z : 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int u = 0; u < V; ++u) row_v[i].f[u] *= scale;
  }
  Vec* mine = s_row[warp][tok];
  float* flat = mine[0].f;
#pragma unroll
  for (int i = 0; i < NV; ++i) mine[8 * i + q] = row_v[i];
  // two slots that name one expert see it in its tag; they are added one after another
  if (put) s_tag[warp][tok][e] = (uint8_t)q;
  float d = w != 0.f ? w * (dw - (a.renorm ? dot * a.inv_scale : 0.f)) : 0.f;
  if (a.sigmoid) d /= 1.f + expf(le);  // times 1 - sigmoid(l)
  __syncwarp();
  if (!__any_sync(kFull, put && s_tag[warp][tok][e] != q)) {
    if (put) flat[e] += d;
  } else {
    for (int j = 0; j < 8; ++j) {
      if (put && q == j) flat[e] += d;
      __syncwarp();
    }
  }
  __syncwarp();
  float* o = d_logits + row * a.E;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = 8 * i + q;
    if (c < vecs && live) *reinterpret_cast<Vec*>(o + V * c) = mine[c];
  }
}

// One warp per token.  The row of d_logits is laid out in shared memory (zeros, or the dense part
// of the softmax's gradient), the selected entries are added there, and the row leaves in vectors
// of V floats (4 where E and the pointers allow it).  Bound by the rows of d_logits.
template <int NV, int V>
__global__ void __launch_bounds__(32 * kWarps) route_backward_kernel(
    RouteArgs a, const float* __restrict__ d_w, float* __restrict__ d_logits) {
  struct alignas(4 * V) Vec { float f[V]; };
  __shared__ Vec s_row[kWarps][32 * NV];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long row = (long long)blockIdx.x * kWarps + warp;
  if (row >= a.T) return;  // warp-uniform
  const float* lg = a.logits + row * a.E;
  const int32_t* idx = a.idx + row * a.k;
  const float* w = a.w + row * a.k;
  const float* dw = d_w + row * a.k;
  const int vecs = a.E / V;
  const bool dense = !a.sigmoid && !a.renorm;
  float l[NV][V];
  if (dense) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = lane + 32 * i;
      Vec v;
#pragma unroll
      for (int u = 0; u < V; ++u) v.f[u] = -INFINITY;
      if (c < vecs) v = *reinterpret_cast<const Vec*>(lg + V * c);
#pragma unroll
      for (int u = 0; u < V; ++u) l[i][u] = absent(v.f[u]) ? -INFINITY : fminf(v.f[u], FLT_MAX);
    }
  }
  // the lane's slot; a weight of exactly 0 (masked) takes no part
  const bool has = lane < a.k;
  int e = has ? __ldg(idx + lane) : -1;
  const float w0 = has ? __ldg(w + lane) : 0.f, dw0 = has && w0 != 0.f ? __ldg(dw + lane) : 0.f;
  float dot = w0 * dw0;
  for (int j = lane + 32; j < a.k; j += 32) {
    const float wj = __ldg(w + j);
    dot += wj != 0.f ? wj * __ldg(dw + j) : 0.f;
  }
  const float rest = a.sigmoid && valid_expert(e, a.E) ? 1.f + expf(__ldg(lg + e)) : 1.f;  // 1 / (1 - sigmoid(l))
  dot = warp_sum(dot);
  Vec* mine = s_row[warp];
  float* flat = mine[0].f;
  float scale = 0.f;
  if (dense) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int u = 0; u < V; ++u) m = fmaxf(m, l[i][u]);
    m = warp_maxf(m);
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int u = 0; u < V; ++u) {
        l[i][u] = l[i][u] > -INFINITY ? expf(l[i][u] - m) : 0.f;
        z += l[i][u];
      }
    z = warp_sum(z);
    scale = z > 0.f ? -dot / z : 0.f;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    Vec v;
#pragma unroll
    for (int u = 0; u < V; ++u) v.f[u] = dense ? scale * l[i][u] : 0.f;
    mine[lane + 32 * i] = v;
  }
  const float shared = a.renorm ? dot * a.inv_scale : 0.f;
  float q = w0 != 0.f ? w0 * (dw0 - shared) / rest : 0.f;
  __syncwarp();
  for (int j0 = 0;;) {
    // slots that name the same expert are added one after another, in order
    const bool put = valid_expert(e, a.E);
    const unsigned same = __match_any_sync(kFull, put ? e : -1 - lane);
    if (!__any_sync(kFull, __popc(same) > 1)) {
      if (put) flat[e] += q;
    } else {
      for (int i = 0; i < 32; ++i) {
        if (lane == i && put) flat[e] += q;
        __syncwarp();
      }
    }
    __syncwarp();
    j0 += 32;
    if (j0 >= a.k) break;
    const int j = j0 + lane;
    e = -1;
    q = 0.f;
    if (j < a.k) {
      const float wj = __ldg(w + j);
      e = __ldg(idx + j);
      if (wj != 0.f && valid_expert(e, a.E)) {
        q = wj * (__ldg(dw + j) - shared);
        if (a.sigmoid) q /= 1.f + expf(__ldg(lg + e));
      }
    }
  }
  float* o = d_logits + row * a.E;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = lane + 32 * i;
    if (c < vecs) *reinterpret_cast<Vec*>(o + V * c) = mine[c];
  }
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

template <int N> struct Slots { static constexpr int value = N; };

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
                         int32_t* idx, float* w, int32_t* counts, int sms, cudaStream_t st) {
  if (counts) {
    const cudaError_t e = cudaMemsetAsync(counts, 0, 4 * (size_t)r.E, st);
    if (e != cudaSuccess) return e;
  }
  if (r.T == 0) return cudaSuccess;
  RouteArgs a = route_args(r);
  a.logits = logits; a.bias = bias; a.idx = idx; a.w = w; a.counts = counts;
  const int ng = (r.E + 31) / 32;
  if (r.k <= 8 && (r.groups == 1 || (a.gsize % 8 == 0 && r.groups <= 8))) {
    auto pick = [&](auto slots) {
      constexpr int kNS = decltype(slots)::value;
      const bool few = r.k <= 4;
      if (r.E == 8 * kNS) {
        if (r.groups == 1) return few ? route4_kernel<kNS, 4, 1, true> : route4_kernel<kNS, 8, 1, true>;
        if constexpr (kNS >= 8)
          if (r.groups == 8) return few ? route4_kernel<kNS, 4, 8, true> : route4_kernel<kNS, 8, 8, true>;
        if (r.groups == 4) return few ? route4_kernel<kNS, 4, 4, true> : route4_kernel<kNS, 8, 4, true>;
      }
      if (r.groups == 1) return few ? route4_kernel<kNS, 4, 1, false> : route4_kernel<kNS, 8, 1, false>;
      return few ? route4_kernel<kNS, 4, 0, false> : route4_kernel<kNS, 8, 0, false>;
    };
    auto kern = ng <= 1 ? pick(Slots<4>{}) : ng <= 2 ? pick(Slots<8>{}) : ng <= 4 ? pick(Slots<16>{}) : pick(Slots<32>{});
    const long long warps = ((long long)r.T + 3) / 4;
    const int per = warps >= 4 * sms ? 4 : 1;  // few tokens: a warp to an SM
    kern<<<(unsigned)((warps + per - 1) / per), 32 * per, 0, st>>>(a);
    return cudaGetLastError();
  }
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
  const bool vec = r.E % 4 == 0 && ((reinterpret_cast<uintptr_t>(logits) |
                                      reinterpret_cast<uintptr_t>(d_logits)) & 15u) == 0;
  if (r.k <= 8) {
    const int n = (r.E + 31) / 32;
    auto kern4 = vec ? (n <= 1   ? route4_backward_kernel<1, 4>
                        : n <= 2 ? route4_backward_kernel<2, 4>
                        : n <= 4 ? route4_backward_kernel<4, 4>
                                 : route4_backward_kernel<8, 4>)
                     : (n <= 1   ? route4_backward_kernel<4, 1>
                        : n <= 2 ? route4_backward_kernel<8, 1>
                        : n <= 4 ? route4_backward_kernel<16, 1>
                                 : route4_backward_kernel<32, 1>);
    const long long warps = ((long long)r.T + 3) / 4;
    kern4<<<(unsigned)((warps + 3) / 4), 128, 0, st>>>(a, d_w, d_logits);
    return cudaGetLastError();
  }
  const int nv = ((vec ? r.E / 4 : r.E) + 31) / 32;
  auto kern = vec       ? (nv <= 1 ? route_backward_kernel<1, 4> : route_backward_kernel<2, 4>)
              : nv <= 1 ? route_backward_kernel<1, 1>
              : nv <= 2 ? route_backward_kernel<2, 1>
              : nv <= 4 ? route_backward_kernel<4, 1>
                        : route_backward_kernel<8, 1>;
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
