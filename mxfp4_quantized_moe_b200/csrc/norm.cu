// Layer / rms norm of activation rows with the residual add and the 8-bit checkpoint fused in,
// its gradients (from the rows or from their checkpoint), and the checkpoint alone.
// Definitions at mxfp4_moe_norm_forward, mxfp4_moe_norm_backward and mxfp4_moe_checkpoint in
// include/mxfp4_moe.h.
#include <cuda_fp16.h>

#include "block_edge.h"
#include "common.cuh"

namespace moe {

namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;

// Where a pass reads its rows from.
enum Source : int { kBf16 = 0, kF32 = 1, kE4m3 = 2, kInt8 = 3 };

// The warp's index as a value that is the same in all its lanes for the compiler too, so that row
// numbers and row addresses are computed once per warp.
MOE_DEV int warp_index() { return __shfl_sync(kFull, (int)threadIdx.x >> 5, 0); }

MOE_DEV float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// Two values rounded to bf16 by one instruction.
MOE_DEV uint32_t pack_bf16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// ---- rows of bf16 or fp32 -----------------------------------------------------------------
// V consecutive features of a row as they come from memory: V = 8 in 16-byte vectors, V = 1
// alone.  A pass first issues every load it needs into such registers and only then computes:
// loads of a row must not wait for one another's arithmetic or stores.
template <int SRC, int V> struct Raw;
template <> struct Raw<kBf16, 8> { uint4 q; };
template <> struct Raw<kBf16, 1> { uint32_t q; };
template <> struct Raw<kF32, 8> { float4 a, b; };
template <> struct Raw<kF32, 1> { float a; };
template <int SRC> struct Raw<SRC, 8> { uint2 q; uint32_t byte; };  // checkpoints

template <int SRC, int V>
MOE_DEV void fetch(Raw<SRC, V>& r, const void* base, size_t at) {
  if constexpr (SRC == kF32 && V == 8) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
    r.a = __ldg(p);
    r.b = __ldg(p + 1);
  } else if constexpr (SRC == kF32) {
    r.a = __ldg(static_cast<const float*>(base) + at);
  } else if constexpr (V == 8) {
    r.q = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at));
  } else {
    r.q = __ldg(static_cast<const uint16_t*>(base) + at);
  }
}
// The same from a buffer that the kernel also writes (a gradient added in place).
template <int SRC, int V>
MOE_DEV void fetch_rw(Raw<SRC, V>& r, const void* base, size_t at) {
  if constexpr (SRC == kF32 && V == 8) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
    r.a = p[0];
    r.b = p[1];
  } else if constexpr (SRC == kF32) {
    r.a = static_cast<const float*>(base)[at];
  } else if constexpr (V == 8) {
    r.q = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at);
  } else {
    r.q = static_cast<const uint16_t*>(base)[at];
  }
}
template <int SRC, int V>
MOE_DEV void clear(Raw<SRC, V>& r) {
  if constexpr (SRC == kF32 && V == 8) r.a = r.b = make_float4(0.f, 0.f, 0.f, 0.f);
  else if constexpr (SRC == kF32) r.a = 0.f;
  else if constexpr (SRC == kBf16 && V == 8) r.q = make_uint4(0u, 0u, 0u, 0u);
  else if constexpr (SRC == kBf16) r.q = 0u;
  else {
    r.q = make_uint2(0u, 0u);
    r.byte = 127u;
  }
}
template <bool F32, int V> using Row = Raw<F32 ? kF32 : kBf16, V>;

template <bool F32, int V>
MOE_DEV void store_rows(void* base, size_t at, const float (&v)[V]) {
  if constexpr (F32) {
    float* p = static_cast<float*>(base) + at;
    if constexpr (V == 8) {
      reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      *p = v[0];
    }
  } else {
    uint16_t* p = static_cast<uint16_t*>(base) + at;
    if constexpr (V == 8)
      *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                                pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
    else
      *p = f_to_bf16(v[0]);
  }
}
// fp32 values as the row type holds them
template <bool F32, int V>
MOE_DEV void into_raw(const float (&v)[V], Row<F32, V>& r) {
  if constexpr (F32 && V == 8) {
    r.a = make_float4(v[0], v[1], v[2], v[3]);
    r.b = make_float4(v[4], v[5], v[6], v[7]);
  } else if constexpr (F32) {
    r.a = v[0];
  } else if constexpr (V == 8) {
    r.q = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                     pack_bf16(v[6], v[7]));
  } else {
    r.q = f_to_bf16(v[0]);
  }
}
template <bool F32, int V>
MOE_DEV void store_raw(void* base, size_t at, const Row<F32, V>& r) {
  if constexpr (F32 && V == 8) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
    p[0] = r.a;
    p[1] = r.b;
  } else if constexpr (F32) {
    static_cast<float*>(base)[at] = r.a;
  } else if constexpr (V == 8) {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at) = r.q;
  } else {
    static_cast<uint16_t*>(base)[at] = (uint16_t)r.q;
  }
}

// ---- checkpoint blocks ----------------------------------------------------------------------
// Four adjacent lanes hold a block of 32 features, 8 each.  The block's largest magnitude (as
// bits, which order like the magnitudes) gives the scale; x 2^-S is a product with a power of
// two, so the conversion's rounding is the only one.
MOE_DEV float pow2(int n) { return __uint_as_float((uint32_t)(n + 127) << 23); }  // [-126, 127]

template <int FMT>
MOE_DEV uint2 encode8(const float (&v)[8], uint32_t& scale_byte) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  m = max(m, __shfl_xor_sync(kFull, m, 1));
  m = max(m, __shfl_xor_sync(kFull, m, 2));
  const bool bad = m >= 0x7F800000u;  // an infinity or NaN
  const int e = (int)(m >> 23);
  const uint32_t frac = m & 0x7FFFFFu;
  uint2 q;
  if constexpr (FMT == kE4m3) {
    const int S = min(120, max(-126, e - 135 + (frac > 0x600000u ? 1 : 0)));  // 448 = 1.75 2^8
    const float inv = pow2(-S), lim = S == 120 ? 240.f : 448.f;
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = fminf(fmaxf(v[2 * i] * inv, -lim), lim);
      const float b = fminf(fmaxf(v[2 * i + 1] * inv, -lim), lim);
      uint16_t d;
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(b), "f"(a));
      h[i] = d;
    }
    q = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
    scale_byte = bad ? 255u : (uint32_t)(S + 127);
  } else {
    // 127 = 1.984375 2^6
    const int S = min(121, max(-126, e - 133 + (frac > 0x7E0000u ? 1 : 0)));
    const float inv = pow2(-S);
    uint32_t b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      b[i] = (uint32_t)__float2int_rn(fminf(fmaxf(v[i] * inv, -127.f), 127.f)) & 0xFFu;
    q.x = b[0] | (b[1] << 8) | (b[2] << 16) | (b[3] << 24);
    q.y = b[4] | (b[5] << 8) | (b[6] << 16) | (b[7] << 24);
    scale_byte = bad ? 255u : (uint32_t)(S + 133);
  }
  if (bad) q = make_uint2(0u, 0u);
  return q;
}

// 2^(byte - 127); byte 0 is the subnormal 2^-127, 255 is NaN
MOE_DEV float scale_value(uint32_t byte) {
  return byte == 255u ? __uint_as_float(0x7FC00000u)
                      : __uint_as_float(byte == 0u ? 0x00400000u : byte << 23);
}

template <int FMT>
MOE_DEV void decode8(uint2 q, uint32_t byte, float (&v)[8]) {
  const float s = scale_value(byte);
  const uint32_t w[2] = {q.x, q.y};
  if constexpr (FMT == kE4m3) {
    const uint64_t s2 = f2(s, s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t h2;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)(w[i >> 1] >> (16 * (i & 1)))));
      const __half2 hh = *reinterpret_cast<const __half2*>(&h2);
      const uint64_t p = f2mul(f2(__low2float(hh), __high2float(hh)), s2);
      v[2 * i] = f2lo(p);
      v[2 * i + 1] = f2hi(p);
    }
  } else {
    // the byte with its sign bit flipped is code + 128, set into the fraction of 2^23
    const float t = s * 0.015625f;
    const uint64_t t2 = f2(t, t), z2 = f2(-8388736.f, -8388736.f);
    const uint32_t x[2] = {w[0] ^ 0x80808080u, w[1] ^ 0x80808080u};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = prmt(x[i >> 1], 0x4B000000u, 0x7440u | (uint32_t)(2 * i & 3));
      const uint32_t hi = prmt(x[i >> 1], 0x4B000000u, 0x7440u | (uint32_t)(2 * i + 1 & 3));
      const uint64_t p = f2mul(f2add(f2(__uint_as_float(lo), __uint_as_float(hi)), z2), t2);
      v[2 * i] = f2lo(p);
      v[2 * i + 1] = f2hi(p);
    }
  }
}

// Loads of a pass's rows from any source, and their values.
template <int SRC, int V>
MOE_DEV void fetch_source(Raw<SRC, V>& r, const void* x, const mxfp4_moe_checkpoint& from, size_t at) {
  if constexpr (SRC == kBf16 || SRC == kF32) {
    fetch<SRC, V>(r, x, at);
  } else {
    r.q = __ldg(reinterpret_cast<const uint2*>(from.codes + at));
    r.byte = __ldg(from.scales + at / 32);
  }
}
template <int SRC, int V>
MOE_DEV void values(const Raw<SRC, V>& r, float (&v)[V]) {
  if constexpr (SRC == kF32 && V == 8) {
    v[0] = r.a.x; v[1] = r.a.y; v[2] = r.a.z; v[3] = r.a.w;
    v[4] = r.b.x; v[5] = r.b.y; v[6] = r.b.z; v[7] = r.b.w;
  } else if constexpr (SRC == kF32) {
    v[0] = r.a;
  } else if constexpr (SRC == kBf16 && V == 8) {
    v[0] = bf16_lo(r.q.x); v[1] = bf16_hi(r.q.x); v[2] = bf16_lo(r.q.y); v[3] = bf16_hi(r.q.y);
    v[4] = bf16_lo(r.q.z); v[5] = bf16_hi(r.q.z); v[6] = bf16_lo(r.q.w); v[7] = bf16_hi(r.q.w);
  } else if constexpr (SRC == kBf16) {
    v[0] = __uint_as_float(r.q << 16);
  } else {
    decode8<SRC>(r.q, r.byte, v);
  }
}
template <int V>
MOE_DEV void load_params(const void* base, bool f32, size_t at, float absent, float (&v)[V]) {
  if (!base) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = absent;
  } else if (f32) {
    Raw<kF32, V> r;
    fetch<kF32, V>(r, base, at);
    values<kF32, V>(r, v);
  } else {
    Raw<kBf16, V> r;
    fetch<kBf16, V>(r, base, at);
    values<kBf16, V>(r, v);
  }
}

// Feature of a thread's chunk c: chunks go round the lanes of the row's W warps.
template <int V>
MOE_DEV int feature(int c, int W, int wi, int lane) { return V * ((c * W + wi) * 32 + lane); }

MOE_DEV void group_barrier(int id, int W) {  // the W warps of a row
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(32 * W) : "memory");
}

// V features as fp32 in registers; pairs for the paired fp32 arithmetic where V = 8.
template <int V> struct Vals { float v[1]; };
template <> struct Vals<8> { uint64_t p[4]; };

template <int V>
MOE_DEV void set(Vals<V>& x, const float (&v)[V]) {
  if constexpr (V == 8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x.p[i] = f2(v[2 * i], v[2 * i + 1]);
  } else {
    x.v[0] = v[0];
  }
}
template <int V>
MOE_DEV void get(const Vals<V>& x, float (&v)[V]) {
  if constexpr (V == 8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = f2lo(x.p[i]);
      v[2 * i + 1] = f2hi(x.p[i]);
    }
  } else {
    v[0] = x.v[0];
  }
}
// Sums that keep two partial sums (even and odd features) where V = 8.
struct Pair {
  uint64_t p = 0;  // two zeros
  MOE_DEV float sum() const { return f2lo(p) + f2hi(p); }
};
template <int V>
MOE_DEV void add_sum(Pair& s, const Vals<V>& x) {
  if constexpr (V == 8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) s.p = f2add(s.p, x.p[i]);
  } else {
    s.p = f2(f2lo(s.p) + x.v[0], 0.f);
  }
}
// x - mean, in place, and the sum of its squares
template <int V>
MOE_DEV void center(Pair& s, Vals<V>& x, float mean) {
  if constexpr (V == 8) {
    const uint64_t m = f2(-mean, -mean);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x.p[i] = f2add(x.p[i], m);
      s.p = f2fma(x.p[i], x.p[i], s.p);
    }
  } else {
    x.v[0] -= mean;
    s.p = f2(fmaf(x.v[0], x.v[0], f2lo(s.p)), 0.f);
  }
}
template <int V>
MOE_DEV void scale_shift(Vals<V>& x, float rstd, const Vals<V>& g, const Vals<V>& b) {
  if constexpr (V == 8) {
    const uint64_t r = f2(rstd, rstd);
#pragma unroll
    for (int i = 0; i < 4; ++i) x.p[i] = f2fma(f2mul(x.p[i], r), g.p[i], b.p[i]);
  } else {
    x.v[0] = fmaf(x.v[0] * rstd, g.v[0], b.v[0]);
  }
}

// Totals of Q values over the warp: lane l ends with that of value l / (32 / Q).
template <int Q>
MOE_DEV float fold(float (&q)[Q]) {
  const int lane = threadIdx.x & 31;
  int n = Q;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    if (n > 1) {
      n >>= 1;
      const bool upper = lane & o;
#pragma unroll
      for (int i = 0; i < Q / 2; ++i)
        if (i < n) {
          const float mine = upper ? q[i + n] : q[i], other = upper ? q[i] : q[i + n];
          q[i] = mine + __shfl_xor_sync(kFull, other, o);
        }
    } else {
      q[0] += __shfl_xor_sync(kFull, q[0], o);
    }
  }
  return q[0];
}

// Eight features of a lane into the checkpoint; all lanes of the warp take part (H is a multiple
// of 32, so the four lanes of a block are inside the row together).
MOE_DEV void store_checkpoint(const mxfp4_moe_checkpoint& to, size_t at, bool in, const Vals<8>& v) {
  float f[8];
  get<8>(v, f);
  uint32_t byte;
  const uint2 q = to.format == MXFP4_MOE_CHECKPOINT_E4M3 ? encode8<kE4m3>(f, byte)
                                                         : encode8<kInt8>(f, byte);
  if (in) {
    *reinterpret_cast<uint2*>(to.codes + at) = q;
    if ((threadIdx.x & 3) == 0) to.scales[at / 32] = (uint8_t)byte;
  }
}

// ---- forward --------------------------------------------------------------------------------
// A row is held as fp32 in registers from its one read to its output: mean, then the variance
// about that mean, then the output.

template <int I> struct Index { static constexpr int value = I; };

// The form for few rows, for latency: a row over as many warps as it fills, every load of it in
// flight at once (one row of 2880: 2.6 us, of which 1.5 are a launch's).  Also takes rows of more
// than 8192 features that vectors cannot read.
template <int SRC, bool F32, int V, int NC>
__global__ void __launch_bounds__(512) norm_forward_kernel(NormArgs a, int W) {
  __shared__ __align__(16) float s_buf[2][16][16];
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int group = W == 1 ? warp : warp / W, wi = W == 1 ? 0 : warp % W;
  const long long row = (long long)blockIdx.x * (blockDim.x / (32 * W)) + group;
  if (row >= a.T) return;  // whole groups leave together
  constexpr bool kRows = SRC == kBf16 || SRC == kF32;
  const float inv_h = 1.f / (float)a.H;
  const int h0 = V * (wi * NC * 32 + lane);  // the lane's vectors are 32 V features apart
  const size_t at = (size_t)row * a.H + h0;
  bool in[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) in[c] = h0 + 32 * V * c < a.H;
  auto group_sum = [&](float v, int slot) {
    v = warp_sum(v);
    if (W == 1) return v;
    if (lane == 0) s_buf[slot][group][wi] = v;
    group_barrier(1 + group, W);
    const float4* b = reinterpret_cast<const float4*>(s_buf[slot][group]);
    float t = 0.f;
    for (int i = 0; i < W; i += 4) {
      const float4 f = b[i / 4];
      t += f.x;
      if (i + 1 < W) t += f.y;
      if (i + 2 < W) t += f.z;
      if (i + 3 < W) t += f.w;
    }
    return t;
  };
  Raw<SRC, V> r[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    clear(r[c]);
    if (in[c]) fetch_source<SRC, V>(r[c], a.x, a.from, at + 32 * V * c);
  }
  if constexpr (kRows) {
    if (a.y) {
      Raw<SRC, V> y[NC];
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        clear(y[c]);
        if (in[c]) fetch<SRC, V>(y[c], a.y, at + 32 * V * c);
      }
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        float f[V], u[V];
        values<SRC, V>(r[c], f);
        values<SRC, V>(y[c], u);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] += u[i];
        into_raw<F32, V>(f, r[c]);
        if (in[c]) store_raw<F32, V>(a.x_out, at + 32 * V * c, r[c]);
      }
    }
  }
  Vals<V> v[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    float f[V];
    values<SRC, V>(r[c], f);
    set<V>(v[c], f);
  }
  if constexpr (kRows && V == 8) {
    if (a.to.codes) {
#pragma unroll
      for (int c = 0; c < NC; ++c) store_checkpoint(a.to, at + 32 * V * c, in[c], v[c]);
    }
  }
  float mean = 0.f;
  if (!a.rms) {
    Pair s;
#pragma unroll
    for (int c = 0; c < NC; ++c) add_sum<V>(s, v[c]);
    mean = group_sum(s.sum(), 0) * inv_h;
  }
  Pair s;
#pragma unroll
  for (int c = 0; c < NC; ++c)
    if (in[c]) center<V>(s, v[c], mean);
  const float rstd = rsqrtf(group_sum(s.sum(), 1) * inv_h + a.eps);
  if (wi == 0 && lane == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }
  auto finish = [&](auto type) {  // parameters of either type, the branch outside the loops
    constexpr int kP = decltype(type)::value;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      if (!in[c]) continue;
      float f[V];
      Vals<V> g, b;
      Raw<kP, V> rg, rb;
      if (a.weight) fetch<kP, V>(rg, a.weight, h0 + 32 * V * c);
      if (a.bias) fetch<kP, V>(rb, a.bias, h0 + 32 * V * c);
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = 1.f;
      if (a.weight) values<kP, V>(rg, f);
      set<V>(g, f);
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = 0.f;
      if (a.bias) values<kP, V>(rb, f);
      set<V>(b, f);
      scale_shift<V>(v[c], rstd, g, b);
      get<V>(v[c], f);
      store_rows<F32, V>(a.out, at + 32 * V * c, f);
    }
  };
  if (a.param_f32) finish(Index<kF32>{});
  else finish(Index<kBf16>{});
}

// 16 (8) bytes to shared memory; with n == 0 nothing is read and zeros are written.  CA: by way
// of L1, for the two halves of a 32-byte sector that two copies take.
template <int DST, int SRC, bool CA>  // byte offsets known at compile time
MOE_DEV void copy_async16(uint32_t dst, const void* src, uint32_t n) {
  if constexpr (CA)
    asm volatile("cp.async.ca.shared.global [%0 + %3], [%1 + %4], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(n), "n"(DST), "n"(SRC) : "memory");
  else
    asm volatile("cp.async.cg.shared.global [%0 + %3], [%1 + %4], 16, %2;" ::"r"(dst), "l"(src),
               "r"(n), "n"(DST), "n"(SRC) : "memory");
}
template <int DST, int SRC>
MOE_DEV void copy_async8(uint32_t dst, const void* src, uint32_t n) {
  asm volatile("cp.async.ca.shared.global [%0 + %3], [%1 + %4], 8, %2;" ::"r"(dst), "l"(src),
               "r"(n), "n"(DST), "n"(SRC) : "memory");
}
MOE_DEV void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N = 0>  // all but the N latest groups have arrived
MOE_DEV void copy_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// for_n<N>(f): f(integral_constant 0), ..., f(integral_constant N - 1)
template <int N, int I = 0, class F>
MOE_DEV void for_n(const F& f) {
  if constexpr (I < N) {
    f(Index<I>{});
    for_n<N, I + 1>(f);
  }
}

// Totals of Q values over the W warps of a row group, in every lane: folded over each warp, then
// one exchange through `buf` (W Q floats) behind the group's barrier.
template <int Q>
MOE_DEV void group_totals(float (&q)[Q], int W, int wi, int bar, float* buf) {
  const int lane = threadIdx.x & 31;
  float t = fold<Q>(q);
  int step = 32 / Q;  // lanes between the totals of two values
  if (W > 1) {
    if ((lane & (step - 1)) == 0) buf[wi * Q + lane / step] = t;
    group_barrier(bar, W);
    t = lane < W * Q ? buf[lane] : 0.f;  // lane l holds value l % Q
#pragma unroll
    for (int i = 32; i < 16 * Q; i += 32) t += lane + i < W * Q ? buf[lane + i] : 0.f;
#pragma unroll
    for (int o = 16; o >= Q; o >>= 1) t += __shfl_xor_sync(kFull, t, o);
    step = 1;
  }
#pragma unroll
  for (int i = 0; i < Q; ++i) q[i] = __shfl_sync(kFull, t, i * step);
}

// The form for many rows: persistent blocks whose groups of W warps take RB rows in turn.  A
// lane copies the vectors that it will compute on into shared memory asynchronously (its own 16
// bytes of each 512, so no lane waits for another), takes them into registers, and at once
// requests the next rows' into the same place: the loads of a whole turn are in flight behind
// the arithmetic of the one before, without registers for them.  A lane keeps the same features
// throughout, so weight and bias stay in its registers; the RB rows share one folded reduction.
// Nothing branches per row: copies past a row's end read nothing and write zeros, rows past the
// last one repeat it.  (The instructions per feature bound the earlier forms, not the bytes: 24 of
// them with branches, 13 here.)  T = 32768, H = 2880, bf16: 60 us, 6.3 TB/s, 96 % of the measured
// copy; with the residual 133 us, 87 %; with the checkpoint as well 145-155 us.  One row a turn
// and warp-wide sums took 131 us, a row in one warp's registers 93 us.
template <int SRC> constexpr int kStage = SRC == kF32 ? 1024 : SRC == kBf16 ? 512 : 256;

// A lane's vector from its place in a stage (fp32: two planes of 512 bytes).
template <int SRC>
MOE_DEV void read_stage(uint32_t from, Raw<SRC, 8>& r) {
  if constexpr (SRC == kF32) {
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(r.a.x), "=f"(r.a.y), "=f"(r.a.z), "=f"(r.a.w) : "r"(from) : "memory");
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(r.b.x), "=f"(r.b.y), "=f"(r.b.z), "=f"(r.b.w) : "r"(from + 512) : "memory");
  } else if constexpr (SRC == kBf16) {
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.q.x), "=r"(r.q.y), "=r"(r.q.z), "=r"(r.q.w) : "r"(from) : "memory");
  } else {
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r.q.x), "=r"(r.q.y) : "r"(from) : "memory");
  }
}

template <int SRC, bool F32, bool RES, int NC, int RB, int NT, int BLOCKS>
__global__ void __launch_bounds__(NT, BLOCKS) norm_forward_many_kernel(NormArgs a, int W) {
  constexpr int V = 8;
  constexpr bool kRows = SRC == kBf16 || SRC == kF32;
  constexpr int kElem = SRC == kF32 ? 4 : SRC == kBf16 ? 2 : 1;  // bytes of a feature as read
  constexpr int kOut = F32 ? 4 : 2;
  constexpr int kTurn = RB * NC * kStage<SRC>;
  extern __shared__ __align__(16) uint8_t s_dyn[];  // the warps' stages
  __shared__ float s_buf[NT / 32][2][2][RB * (NT / 32)];
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int group = W == 1 ? warp : warp / W, wi = W == 1 ? 0 : warp % W;
  const int G = blockDim.x / (32 * W);
  const uint32_t stage = smem_u32(s_dyn) + (uint32_t)warp * (RES ? 2 * kTurn : kTurn) +
                         (kRows ? 16u : 8u) * lane;
  const float inv_h = 1.f / (float)a.H;
  const int h0 = V * (wi * NC * 32 + lane);  // the lane's vectors are 256 features apart
  bool in[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) in[c] = h0 + 256 * c < a.H;
  const int h0r = in[0] ? h0 : 0;
  uint32_t byte[kRows ? 1 : RB][kRows ? 1 : NC];
  // rows past the last one stand for it: they compute and store what it does
  const uint32_t rows = (uint32_t)a.T;
  auto offset = [&](uint32_t row, int j) { return (size_t)min(row + j, rows - 1) * (uint32_t)a.H; };

  auto request = [&](uint32_t row) {
    for_n<RB>([&](auto jj) {
      constexpr int j = decltype(jj)::value;
      const size_t at = offset(row, j);
      const uint8_t* x = (kRows ? static_cast<const uint8_t*>(a.x) + at * kElem : a.from.codes + at) + h0r * kElem;
      const uint8_t* y = RES ? static_cast<const uint8_t*>(a.y) + at * kElem + h0r * kElem : nullptr;
      for_n<NC>([&](auto cc) {
        constexpr int c = decltype(cc)::value, to = (j * NC + c) * kStage<SRC>, from = 256 * c * kElem;
        if constexpr (kRows) {
          const uint32_t n = in[c] ? 16u : 0u;
          copy_async16<to, from, SRC == kF32>(stage, x, n);
          if constexpr (SRC == kF32) copy_async16<to + 512, from + 16, SRC == kF32>(stage, x, n);
          if constexpr (RES) {
            copy_async16<kTurn + to, from, SRC == kF32>(stage, y, n);
            if constexpr (SRC == kF32) copy_async16<kTurn + to + 512, from + 16, SRC == kF32>(stage, y, n);
          }
        } else {
          copy_async8<to, from>(stage, x, in[c] ? 8u : 0u);
          byte[j][c] = __ldg(a.from.scales + at / 32 + (in[c] ? h0 / 32 + 8 * c : 0));
        }
      });
    });
    copy_async_commit();
  };
  const uint32_t step = gridDim.x * (uint32_t)(G * RB);
  uint32_t row = (blockIdx.x * (uint32_t)G + group) * RB;
  if (row < rows) request(row);
  Vals<V> pg[NC], pb[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    float f[V];
    load_params<V>(a.weight, a.param_f32, in[c] ? h0 + 256 * c : 0, 1.f, f);
    set<V>(pg[c], f);
    load_params<V>(a.bias, a.param_f32, in[c] ? h0 + 256 * c : 0, 0.f, f);
    set<V>(pb[c], f);
  }
  int turn = 0;
  for (; row < rows; row += step) {
    Vals<V> v[RB][NC];
    copy_async_wait<0>();
#pragma unroll
    for (int j = 0; j < RB; ++j) {
      uint8_t* x_out = RES ? static_cast<uint8_t*>(a.x_out) + offset(row, j) * kOut + h0 * kOut : nullptr;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const uint32_t from = stage + (uint32_t)(j * NC + c) * kStage<SRC>;
        Raw<SRC, V> r;
        float f[V];
        read_stage<SRC>(from, r);
        if constexpr (!kRows) r.byte = byte[j][c];
        values<SRC, V>(r, f);
        if constexpr (RES) {
          float u[V];
          read_stage<SRC>(from + kTurn, r);
          values<SRC, V>(r, u);
#pragma unroll
          for (int i = 0; i < V; ++i) f[i] += u[i];
          into_raw<F32, V>(f, r);
          if (in[c]) store_raw<F32, V>(x_out, 256 * c, r);
          values<SRC, V>(r, f);
        }
        set<V>(v[j][c], f);
      }
    }
    if (rows - row > step) request(row + step);  // this lane has read its places
    if constexpr (kRows) {
      if (a.to.codes) {
#pragma unroll
        for (int j = 0; j < RB; ++j)
#pragma unroll
          for (int c = 0; c < NC; ++c)
            store_checkpoint(a.to, offset(row, j) + h0 + 256 * c, in[c], v[j][c]);
      }
    }
    float mean[RB], q[RB];
#pragma unroll
    for (int j = 0; j < RB; ++j) mean[j] = 0.f;
    if (!a.rms) {
#pragma unroll
      for (int j = 0; j < RB; ++j) {
        Pair s;
#pragma unroll
        for (int c = 0; c < NC; ++c) add_sum<V>(s, v[j][c]);
        mean[j] = s.sum();
      }
      group_totals<RB>(mean, W, wi, 1 + group, s_buf[group][turn][0]);
    }
#pragma unroll
    for (int j = 0; j < RB; ++j) {
      mean[j] *= inv_h;
      q[j] = 0.f;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        Pair s;
        center<V>(s, v[j][c], mean[j]);
        q[j] += in[c] ? s.sum() : 0.f;
      }
    }
    group_totals<RB>(q, W, wi, 1 + group, s_buf[group][turn][1]);
    turn ^= 1;  // the next rows' exchange must not meet this one's readers
#pragma unroll
    for (int j = 0; j < RB; ++j) {
      q[j] = rsqrtf(q[j] * inv_h + a.eps);
      if (wi == 0 && lane == 0) {
        if (a.mean) a.mean[min(row + j, rows - 1)] = mean[j];
        if (a.rstd) a.rstd[min(row + j, rows - 1)] = q[j];
      }
      uint8_t* out = static_cast<uint8_t*>(a.out) + offset(row, j) * kOut + h0 * kOut;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        scale_shift<V>(v[j][c], q[j], pg[c], pb[c]);
        float f[V];
        get<V>(v[j][c], f);
        Row<F32, V> r;
        into_raw<F32, V>(f, r);
        if (in[c]) store_raw<F32, V>(out, 256 * c, r);
      }
    }
  }
}

// Rows that 16-byte vectors cannot read in place (H or a pointer without that alignment) are staged
// whole, by the warps of the row together: the 16-byte pieces that begin inside the row by cp.async
// (the last one with only its bytes of the row), what lies before the first of them by plain loads
// of single features.  The row then stands at 16 - head bytes in its place, and a lane reads the
// features lane, lane + 32, ... of every 256.  T = 16384, H = 1001, bf16: forward 24 us (2.7 TB/s),
// backward 40 us; read feature by feature from global memory they took 64 and 62 us.
template <int E>  // bytes of a feature
struct LooseRow {
  const uint8_t* from;
  uint32_t head, bytes;  // bytes before the first piece; bytes of the row
  MOE_DEV LooseRow(const void* base, size_t row, int H)
      : from(static_cast<const uint8_t*>(base) + row * (size_t)((uint32_t)H * E)), bytes((uint32_t)H * E) {
    head = min((16u - (uint32_t)(reinterpret_cast<uintptr_t>(from) & 15u)) & 15u, bytes);
  }
  static __host__ __device__ uint32_t place(int H) { return 16u + ((uint32_t)H * E + 15u) / 16u * 16u; }
  // PIECES pieces a thread cover the row; returns the thread's feature of the head
  template <int PIECES>
  MOE_DEV uint32_t request(uint32_t to, int tid, int threads) const {
    const uint32_t body = bytes - head;
#pragma unroll
    for (int c = 0; c < PIECES; ++c) {
      const uint32_t off = 16u * (uint32_t)(tid + c * threads);
      if (off < body)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(to + 16u + off),
                     "l"(from + head + off), "r"(min(16u, body - off)) : "memory");
    }
    if ((uint32_t)tid * E >= head) return 0u;
    if constexpr (E == 2) return reinterpret_cast<const uint16_t*>(from)[tid];
    else return reinterpret_cast<const uint32_t*>(from)[tid];
  }
  MOE_DEV void put_head(uint32_t to, int tid, uint32_t feature) const {
    if ((uint32_t)tid * E >= head) return;
    const uint32_t at = to + 16u - head + (uint32_t)tid * E;
    if constexpr (E == 2) asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"((uint16_t)feature) : "memory");
    else asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(feature) : "memory");
  }
  // features h, h + 32, ... of which n lie in the row; 0 past its end
  MOE_DEV void read(uint32_t to, int h, int n, float (&f)[8]) const {
    const uint32_t at = to + 16u - head + (uint32_t)h * E;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t v = 0;
      if constexpr (E == 2) {
        uint16_t u = 0;
        if (i < n) asm volatile("ld.shared.u16 %0, [%1];" : "=h"(u) : "r"(at + 64u * i) : "memory");
        v = (uint32_t)u << 16;
      } else {
        if (i < n) asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at + 128u * i) : "memory");
      }
      f[i] = __uint_as_float(v);
    }
  }
};
template <bool F32>
MOE_DEV void store_loose(void* base, size_t row, int H, int h, int n, const float (&f)[8]) {
  const size_t at = row * (size_t)(uint32_t)H + (uint32_t)h;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) {
      if constexpr (F32) static_cast<float*>(base)[at + 32 * i] = f[i];
      else static_cast<uint16_t*>(base)[at + 32 * i] = f_to_bf16(f[i]);
    }
}
// n features from h on, 32 apart, of a parameter; 0 past the end
MOE_DEV void loose_params(const void* base, bool f32, int h, int n, float absent, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float v[1] = {0.f};
    if (i < n) load_params<1>(base, f32, h + 32 * i, absent, v);
    f[i] = v[0];
  }
}
MOE_DEV int loose_count(int H, int h) { return max(0, min(8, (H - h + 31) / 32)); }

template <int SRC, bool F32, bool RES, int NC, int RB, int NT, int BLOCKS>
__global__ void __launch_bounds__(NT, BLOCKS) norm_forward_loose_kernel(NormArgs a, int W) {
  constexpr int V = 8, E = F32 ? 4 : 2, kPieces = NC * E / 2 + 1, kSets = RES ? 2 : 1;
  extern __shared__ __align__(16) uint8_t s_dyn[];  // per group: 2 turns x RB rows x (x, y)
  __shared__ float s_buf[NT / 32][2][2][RB * (NT / 32)];
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int group = W == 1 ? warp : warp / W, wi = W == 1 ? 0 : warp % W;
  const int G = blockDim.x / (32 * W), tid = wi * 32 + lane;
  const uint32_t place = LooseRow<E>::place(a.H);
  const uint32_t base = smem_u32(s_dyn) + (uint32_t)group * (2 * RB * kSets) * place;
  const float inv_h = 1.f / (float)a.H;
  int h[NC], n[NC];
  Vals<V> pg[NC], pb[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    h[c] = 256 * (wi * NC + c) + lane;
    n[c] = loose_count(a.H, h[c]);
    float f[V];
    loose_params(a.weight, a.param_f32, h[c], n[c], 1.f, f);
    set<V>(pg[c], f);
    loose_params(a.bias, a.param_f32, h[c], n[c], 0.f, f);
    set<V>(pb[c], f);
  }
  const uint32_t rows = (uint32_t)a.T;  // rows past the last one stand for it
  uint32_t hx[RB], hy[RES ? RB : 1];
  auto spot = [&](int turn, int j, int set) { return base + (uint32_t)((turn * RB + j) * kSets + set) * place; };
  auto request = [&](uint32_t row, int turn) {
#pragma unroll
    for (int j = 0; j < RB; ++j) {
      const size_t r = min(row + j, rows - 1);
      hx[j] = LooseRow<E>(a.x, r, a.H).template request<kPieces>(spot(turn, j, 0), tid, 32 * W);
      if constexpr (RES)
        hy[j] = LooseRow<E>(a.y, r, a.H).template request<kPieces>(spot(turn, j, 1), tid, 32 * W);
    }
    copy_async_commit();
  };
  const uint32_t step = gridDim.x * (uint32_t)(G * RB);
  uint32_t row = (blockIdx.x * (uint32_t)G + group) * RB;
  if (row < rows) request(row, 0);
  int turn = 0;
  for (; row < rows; row += step) {
    Vals<V> v[RB][NC];
    copy_async_wait<0>();
#pragma unroll
    for (int j = 0; j < RB; ++j) {
      const size_t r = min(row + j, rows - 1);
      LooseRow<E>(a.x, r, a.H).put_head(spot(turn, j, 0), tid, hx[j]);
      if constexpr (RES) LooseRow<E>(a.y, r, a.H).put_head(spot(turn, j, 1), tid, hy[j]);
    }
    // the rows have arrived, and every lane is done with the other turn's places
    if (W > 1) group_barrier(1 + group, W); else __syncwarp();
    if (rows - row > step) request(row + step, turn ^ 1);
#pragma unroll
    for (int j = 0; j < RB; ++j) {
      const size_t r = min(row + j, rows - 1);
      const LooseRow<E> lx(a.x, r, a.H);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        float f[V];
        lx.read(spot(turn, j, 0), h[c], n[c], f);
        if constexpr (RES) {
          float u[V];
          LooseRow<E>(a.y, r, a.H).read(spot(turn, j, 1), h[c], n[c], u);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            f[i] += u[i];
            if constexpr (!F32) f[i] = bf16_to_f(f_to_bf16(f[i]));
          }
          store_loose<F32>(a.x_out, r, a.H, h[c], n[c], f);
        }
        set<V>(v[j][c], f);
      }
    }
    float mean[RB], q[RB];
#pragma unroll
    for (int j = 0; j < RB; ++j) mean[j] = 0.f;
    if (!a.rms) {
#pragma unroll
      for (int j = 0; j < RB; ++j) {
        Pair t;
#pragma unroll
        for (int c = 0; c < NC; ++c) add_sum<V>(t, v[j][c]);
        mean[j] = t.sum();
      }
      group_totals<RB>(mean, W, wi, 1 + group, s_buf[group][turn][0]);
    }
#pragma unroll
    for (int j = 0; j < RB; ++j) {
      mean[j] *= inv_h;
      q[j] = 0.f;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        float f[V];
        get<V>(v[j][c], f);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = i < n[c] ? f[i] - mean[j] : 0.f;
        set<V>(v[j][c], f);
#pragma unroll
        for (int i = 0; i < V; ++i) q[j] = fmaf(f[i], f[i], q[j]);
      }
    }
    group_totals<RB>(q, W, wi, 1 + group, s_buf[group][turn][1]);
#pragma unroll
    for (int j = 0; j < RB; ++j) {
      const uint32_t r = min(row + j, rows - 1);
      q[j] = rsqrtf(q[j] * inv_h + a.eps);
      if (wi == 0 && lane == 0) {
        if (a.mean) a.mean[r] = mean[j];
        if (a.rstd) a.rstd[r] = q[j];
      }
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        scale_shift<V>(v[j][c], q[j], pg[c], pb[c]);
        float f[V];
        get<V>(v[j][c], f);
        store_loose<F32>(a.out, r, a.H, h[c], n[c], f);
      }
    }
    turn ^= 1;
  }
}

// ---- backward -------------------------------------------------------------------------------
// A thread keeps the same features over all rows of its block, so the parameters' gradients
// accumulate in its registers and leave once per block; a second kernel adds the blocks' partial
// sums in a fixed order.  The sums c1, c2 of the rows that go together are reduced in one folding
// pass over the warp and one exchange over the row's warps.
constexpr int kParts = 296;  // most blocks: two per SM of a B200

// Where a block's sums of d_weight (0) or d_bias (1) go: its row of the partial sums, or the
// gradient itself when there is no other block.
MOE_DEV float* partial_row(const NormGradArgs& a, int which) {
  if (gridDim.x == 1) return which ? a.d_bias : a.d_weight;
  return a.partial + ((size_t)blockIdx.x * 2 + which) * a.H;
}
// The kernel that adds the partial sums is launched while this one ends, and waits for it.
MOE_DEV void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
MOE_DEV void wait_for_launcher() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The form for rows of more than 8192 features: a block of W warps takes one row at a time into
// registers, V NC = 32 features a thread, and reads the weight again for each (from L1).  The sums
// of 32 features leave no room for more: T = 4096, H = 16384, bf16 133 us, 3.0 TB/s.
template <int SRC, bool F32, int V, bool HASG>
__global__ void __launch_bounds__(512) norm_backward_long_kernel(NormGradArgs a, int W, int rows_per_block) {
  constexpr int NC = 32 / V, kGrad = F32 ? kF32 : kBf16;
  __shared__ float s_buf[2][2 * 16];
  const int wi = warp_index(), lane = threadIdx.x & 31;
  const float inv_h = 1.f / (float)a.H;
  float acc_g[NC][V], acc_b[NC][V];
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < V; ++i) acc_g[c][i] = acc_b[c][i] = 0.f;
  const long long begin = (long long)blockIdx.x * rows_per_block;
  const long long end = min((long long)a.T, begin + rows_per_block);
  int turn = 0;
  for (long long row = begin; row < end; ++row) {
    Raw<SRC, V> x[NC];
    Row<F32, V> d[NC], g[HASG ? NC : 1];
    const size_t r0 = (size_t)row * a.H;
    const float mean = a.rms ? 0.f : __ldg(a.mean + row), rstd = __ldg(a.rstd + row);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int h = feature<V>(c, W, wi, lane);
      clear(x[c]);
      clear(d[c]);
      if (h < a.H) {
        fetch_source<SRC, V>(x[c], a.x, a.from, r0 + h);
        fetch<kGrad, V>(d[c], a.d_out, r0 + h);
        if constexpr (HASG) fetch_rw<kGrad, V>(g[c], a.g, r0 + h);
      }
    }
    float q[2] = {0.f, 0.f};  // c1, c2
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int h = feature<V>(c, W, wi, lane);
      if (h < a.H) {
        float xv[V], dv[V], w[V];
        values<SRC, V>(x[c], xv);
        values<kGrad, V>(d[c], dv);
        load_params<V>(a.weight, a.param_f32, h, 1.f, w);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float xh = (xv[i] - mean) * rstd, v = dv[i] * w[i];
          q[0] += v;
          q[1] = fmaf(v, xh, q[1]);
          acc_g[c][i] = fmaf(dv[i], xh, acc_g[c][i]);
          acc_b[c][i] += dv[i];
        }
      }
    }
    group_totals<2>(q, W, wi, 1, s_buf[turn]);
    turn ^= 1;  // the next row's exchange must not meet this one's readers
    const float c1 = a.rms ? 0.f : q[0] * inv_h, c2 = q[1] * inv_h;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int h = feature<V>(c, W, wi, lane);
      if (h < a.H) {
        float xv[V], dv[V], w[V];
        values<SRC, V>(x[c], xv);
        values<kGrad, V>(d[c], dv);
        load_params<V>(a.weight, a.param_f32, h, 1.f, w);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float xh = (xv[i] - mean) * rstd;
          dv[i] = rstd * (dv[i] * w[i] - c1 - xh * c2);
        }
        if constexpr (HASG) {
          float gv[V];
          values<kGrad, V>(g[c], gv);
#pragma unroll
          for (int i = 0; i < V; ++i) dv[i] += gv[i];
        }
        store_rows<F32, V>(a.dx, r0 + h, dv);
      }
    }
  }
  if (!a.d_weight && !a.d_bias) return;
  launch_dependents();
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float* part = partial_row(a, which);
    if (!part) continue;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int h = feature<V>(c, W, wi, lane);
      if (h < a.H) {
#pragma unroll
        for (int i = 0; i < V; ++i) part[h + i] = which ? acc_b[c][i] : acc_g[c][i];
      }
    }
  }
}

// The staged form, for aligned rows of up to 8192 features: as the forward's persistent form,
// the next rows of x and d_out travel into shared memory behind this turn's arithmetic (and
// those of g behind the next turn's first half), a lane keeps its features' sums, and rows past
// the block's last one read as zeros and store nothing.  x_hat and v stay in registers between
// the sums and dx.  Two rows a turn and 80 registers, so that two blocks share an SM: T = 32768,
// H = 2880, bf16 105 us (5.4 TB/s, 82 % of the measured copy), with g 125 us (92 %), from a
// checkpoint with g 124 us.  Four rows a turn and one block measured the same, one row of twice the
// features and three blocks 120 and 137 us.
template <int SRC, bool F32, bool HASG, int NC, int R, int NT, int BLOCKS>
__global__ void __launch_bounds__(NT, BLOCKS)
    norm_backward_staged_kernel(NormGradArgs a, int W, int rows_per_block) {
  constexpr int V = 8, Q = 2 * R;
  constexpr int kGrad = F32 ? kF32 : kBf16;
  constexpr bool kRows = SRC == kBf16 || SRC == kF32;
  constexpr int kX = kRows ? (SRC == kF32 ? 4 : 2) : 1, kD = F32 ? 4 : 2;  // bytes of a feature
  constexpr int kXTurn = R * NC * kStage<SRC>, kDTurn = R * NC * kStage<kGrad>;
  extern __shared__ __align__(16) uint8_t s_dyn[];  // per warp: x, d_out, g
  __shared__ float s_buf[NT / 32][2][Q * (NT / 32)];
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int group = W == 1 ? warp : warp / W, wi = W == 1 ? 0 : warp % W;
  const int G = blockDim.x / (32 * W);
  const uint32_t base = smem_u32(s_dyn) + (uint32_t)warp * (kXTurn + kDTurn + (HASG ? kDTurn : 0));
  const uint32_t stage_x = base + (kRows ? 16u : 8u) * lane, stage_d = base + kXTurn + 16u * lane;
  const float inv_h = 1.f / (float)a.H;
  const int h0 = V * (wi * NC * 32 + lane);  // the lane's vectors are 256 features apart
  bool in[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) in[c] = h0 + 256 * c < a.H;
  const int h0r = in[0] ? h0 : 0;
  Vals<V> acc_g[NC], acc_b[NC], pg[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    float f[V];
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = 0.f;
    set<V>(acc_g[c], f);
    set<V>(acc_b[c], f);
    load_params<V>(a.weight, a.param_f32, in[c] ? h0 + 256 * c : 0, 1.f, f);
    set<V>(pg[c], f);
  }
  const uint32_t begin = blockIdx.x * (uint32_t)rows_per_block;
  const uint32_t end = min((uint32_t)a.T, begin + (uint32_t)rows_per_block);
  auto offset = [&](uint32_t row, int j) { return (size_t)min(row + j, end - 1) * (uint32_t)a.H; };
  uint32_t byte[kRows ? 1 : R][kRows ? 1 : NC];
  float mean_next[R], rstd_next[R];

  auto request = [&](uint32_t row) {
    for_n<R>([&](auto jj) {
      constexpr int j = decltype(jj)::value;
      const size_t at = offset(row, j);
      const bool live = row + j < end;
      const uint8_t* x = (kRows ? static_cast<const uint8_t*>(a.x) + at * kX : a.from.codes + at) + h0r * kX;
      const uint8_t* d = static_cast<const uint8_t*>(a.d_out) + at * kD + h0r * kD;
      for_n<NC>([&](auto cc) {
        constexpr int c = decltype(cc)::value;
        constexpr int tx = (j * NC + c) * kStage<SRC>, td = (j * NC + c) * kStage<kGrad>;
        const uint32_t n = in[c] && live ? 16u : 0u;
        // Features past the row's end have d_out = 0, and for x the row's own (the lane's first
        // vector, or the row's): with x = 0 there x_hat = -mean rstd need not be a finite number.
        const uint8_t* xc = c == 0 || in[c] ? x : x - 256 * c * kX;
        const uint32_t nx = live ? 16u : 0u;
        if constexpr (kRows) {
          copy_async16<tx, 256 * c * kX, SRC == kF32>(stage_x, xc, nx);
          if constexpr (SRC == kF32) copy_async16<tx + 512, 256 * c * kX + 16, SRC == kF32>(stage_x, xc, nx);
        } else {
          copy_async8<tx, 256 * c>(stage_x, xc, nx / 2);
          byte[j][c] = __ldg(a.from.scales + at / 32 + h0r / 32 + (c == 0 || in[c] ? 8 * c : 0));
        }
        copy_async16<td, 256 * c * kD, F32>(stage_d, d, n);
        if constexpr (F32) copy_async16<td + 512, 256 * c * kD + 16, F32>(stage_d, d, n);
      });
      const uint32_t r = min(row + j, end - 1);
      mean_next[j] = a.rms ? 0.f : __ldg(a.mean + r);
      rstd_next[j] = live ? __ldg(a.rstd + r) : 0.f;
    });
    copy_async_commit();
  };
  auto request_g = [&](uint32_t row) {
    for_n<R>([&](auto jj) {
      constexpr int j = decltype(jj)::value;
      const uint8_t* g = static_cast<const uint8_t*>(a.g) + offset(row, j) * kD + h0r * kD;
      for_n<NC>([&](auto cc) {
        constexpr int c = decltype(cc)::value, td = kDTurn + (j * NC + c) * kStage<kGrad>;
        const uint32_t n = in[c] && row + j < end ? 16u : 0u;
        copy_async16<td, 256 * c * kD, F32>(stage_d, g, n);
        if constexpr (F32) copy_async16<td + 512, 256 * c * kD + 16, F32>(stage_d, g, n);
      });
    });
    copy_async_commit();
  };

  const uint32_t step = (uint32_t)(G * R);
  uint32_t row = begin + (uint32_t)(group * R);
  if (row < end) {
    request(row);
    if constexpr (HASG) request_g(row);
  }
  int turn = 0;
  for (; row < end; row += step) {
    if constexpr (HASG) copy_async_wait<1>(); else copy_async_wait<0>();  // x and d_out
    Vals<V> xh[R][NC], v[R][NC];
    float q[Q], rstd[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      rstd[j] = rstd_next[j];
      const uint64_t m2 = f2(-mean_next[j], -mean_next[j]), r2 = f2(rstd[j], rstd[j]);
      Pair c1, c2;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        Raw<SRC, V> rx;
        Raw<kGrad, V> rd;
        read_stage<SRC>(stage_x + (uint32_t)(j * NC + c) * kStage<SRC>, rx);
        read_stage<kGrad>(stage_d + (uint32_t)(j * NC + c) * kStage<kGrad>, rd);
        if constexpr (!kRows) rx.byte = byte[j][c];
        float f[V];
        values<SRC, V>(rx, f);
        set<V>(xh[j][c], f);
        values<kGrad, V>(rd, f);
        set<V>(v[j][c], f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          xh[j][c].p[i] = f2mul(f2add(xh[j][c].p[i], m2), r2);
          const uint64_t d = v[j][c].p[i];
          acc_g[c].p[i] = f2fma(d, xh[j][c].p[i], acc_g[c].p[i]);
          acc_b[c].p[i] = f2add(acc_b[c].p[i], d);
          v[j][c].p[i] = f2mul(d, pg[c].p[i]);
          c1.p = f2add(c1.p, v[j][c].p[i]);
          c2.p = f2fma(v[j][c].p[i], xh[j][c].p[i], c2.p);
        }
      }
      q[2 * j] = a.rms ? 0.f : c1.sum();
      q[2 * j + 1] = c2.sum();
    }
    const bool more = end - row > step;
    if (more) request(row + step);  // this lane has read its places
    group_totals<Q>(q, W, wi, 1 + group, s_buf[group][turn]);
    turn ^= 1;  // the next rows' exchange must not meet this one's readers
    if constexpr (HASG) {
      if (more) copy_async_wait<1>(); else copy_async_wait<0>();  // g
    }
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const float k1 = -rstd[j] * (q[2 * j] * inv_h), k2 = -rstd[j] * (q[2 * j + 1] * inv_h);
      const uint64_t p1 = f2(k1, k1), p2 = f2(k2, k2), r2 = f2(rstd[j], rstd[j]);
      uint8_t* dx = static_cast<uint8_t*>(a.dx) + offset(row, j) * kD + h0 * kD;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v[j][c].p[i] = f2fma(v[j][c].p[i], r2, f2fma(xh[j][c].p[i], p2, p1));
        float f[V];
        Row<F32, V> r;
        if constexpr (HASG) {
          read_stage<kGrad>(stage_d + kDTurn + (uint32_t)(j * NC + c) * kStage<kGrad>, r);
          Vals<V> g;
          values<kGrad, V>(r, f);
          set<V>(g, f);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[j][c].p[i] = f2add(v[j][c].p[i], g.p[i]);
        }
        get<V>(v[j][c], f);
        into_raw<F32, V>(f, r);
        if (in[c] && row + j < end) store_raw<F32, V>(dx, 256 * c, r);
      }
    }
    if constexpr (HASG) {
      if (more) request_g(row + step);
    }
  }
  if (!a.d_weight && !a.d_bias) return;
  launch_dependents();
  // the block's sum over its groups, in group order, to its row of the partial sums
  __syncthreads();
  float* s_sum = reinterpret_cast<float*>(s_dyn);  // the groups' sums of one kind, 32 V NC W each
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float* part = partial_row(a, which);
    if (!part) continue;
    // a caller's gradient is aligned to a feature; the partial sums are to vectors
    const bool whole = (reinterpret_cast<uintptr_t>(part) & 15u) == 0;
    const Vals<V>* acc = which ? acc_b : acc_g;
    if (G > 1) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        float f[V];
        get<V>(acc[c], f);
        float4* to = reinterpret_cast<float4*>(s_sum + (size_t)group * 256 * NC * W + h0 + 256 * c);
        to[0] = make_float4(f[0], f[1], f[2], f[3]);
        to[1] = make_float4(f[4], f[5], f[6], f[7]);
      }
      __syncthreads();
      for (int h = threadIdx.x; h < a.H; h += blockDim.x) {
        float t = 0.f;
        for (int g = 0; g < G; ++g) t += s_sum[(size_t)g * 256 * NC * W + h];
        part[h] = t;
      }
      __syncthreads();
    } else {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        float f[V];
        get<V>(acc[c], f);
        if (in[c] && whole) {
          float4* to = reinterpret_cast<float4*>(part + h0 + 256 * c);
          to[0] = make_float4(f[0], f[1], f[2], f[3]);
          to[1] = make_float4(f[4], f[5], f[6], f[7]);
        } else if (in[c]) {
#pragma unroll
          for (int i = 0; i < V; ++i) part[h0 + 256 * c + i] = f[i];
        }
      }
    }
  }
}

// The staged form for rows without vector alignment (see LooseRow): x, d_out and g of a turn are
// requested together, into the other of two places.
template <bool F32, bool HASG, int NC, int R, int NT, int BLOCKS>
__global__ void __launch_bounds__(NT, BLOCKS)
    norm_backward_loose_kernel(NormGradArgs a, int W, int rows_per_block) {
  constexpr int V = 8, Q = 2 * R, E = F32 ? 4 : 2, kPieces = NC * E / 2 + 1, kSets = HASG ? 3 : 2;
  extern __shared__ __align__(16) uint8_t s_dyn[];  // per group: 2 turns x R rows x (x, d_out, g)
  __shared__ float s_buf[NT / 32][2][Q * (NT / 32)];
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int group = W == 1 ? warp : warp / W, wi = W == 1 ? 0 : warp % W;
  const int G = blockDim.x / (32 * W), tid = wi * 32 + lane;
  const uint32_t place = LooseRow<E>::place(a.H);
  const uint32_t base = smem_u32(s_dyn) + (uint32_t)group * (2 * R * kSets) * place;
  const float inv_h = 1.f / (float)a.H;
  int h[NC], n[NC];
  Vals<V> acc_g[NC], acc_b[NC], pg[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    h[c] = 256 * (wi * NC + c) + lane;
    n[c] = loose_count(a.H, h[c]);
    float f[V];
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = 0.f;
    set<V>(acc_g[c], f);
    set<V>(acc_b[c], f);
    loose_params(a.weight, a.param_f32, h[c], n[c], 1.f, f);
    set<V>(pg[c], f);
  }
  const uint32_t begin = blockIdx.x * (uint32_t)rows_per_block;
  const uint32_t end = min((uint32_t)a.T, begin + (uint32_t)rows_per_block);
  auto spot = [&](int turn, int j, int set) { return base + (uint32_t)((turn * R + j) * kSets + set) * place; };
  uint32_t head[kSets][R];
  float mean_next[R], rstd_next[R];
  const void* from[3] = {a.x, a.d_out, a.g};
  auto request = [&](uint32_t row, int turn) {
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const uint32_t r = min(row + j, end - 1);
#pragma unroll
      for (int t = 0; t < kSets; ++t)
        head[t][j] = LooseRow<E>(from[t], r, a.H).template request<kPieces>(spot(turn, j, t), tid, 32 * W);
      mean_next[j] = a.rms ? 0.f : __ldg(a.mean + r);
      rstd_next[j] = __ldg(a.rstd + r);
    }
    copy_async_commit();
  };
  const uint32_t step = (uint32_t)(G * R);
  uint32_t row = begin + (uint32_t)(group * R);
  if (row < end) request(row, 0);
  int turn = 0;
  for (; row < end; row += step) {
    float mean[R], rstd[R];
    copy_async_wait<0>();
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const uint32_t r = min(row + j, end - 1);
      mean[j] = mean_next[j];
      rstd[j] = rstd_next[j];
#pragma unroll
      for (int t = 0; t < kSets; ++t)
        LooseRow<E>(from[t], r, a.H).put_head(spot(turn, j, t), tid, head[t][j]);
    }
    // the rows have arrived, and every lane is done with the other turn's places
    if (W > 1) group_barrier(1 + group, W); else __syncwarp();
    if (end - row > step) request(row + step, turn ^ 1);
    Vals<V> xh[R][NC], v[R][NC];
    float q[Q];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const uint32_t r = min(row + j, end - 1);
      const bool live = row + j < end;  // a row past the block's last one counts for nothing
      Pair c1, c2;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        float f[V];
        LooseRow<E>(a.x, r, a.H).read(spot(turn, j, 0), h[c], n[c], f);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = i < n[c] ? (f[i] - mean[j]) * rstd[j] : 0.f;
        set<V>(xh[j][c], f);
        LooseRow<E>(a.d_out, r, a.H).read(spot(turn, j, 1), h[c], live ? n[c] : 0, f);
        set<V>(v[j][c], f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint64_t d = v[j][c].p[i];
          acc_g[c].p[i] = f2fma(d, xh[j][c].p[i], acc_g[c].p[i]);
          acc_b[c].p[i] = f2add(acc_b[c].p[i], d);
          v[j][c].p[i] = f2mul(d, pg[c].p[i]);
          c1.p = f2add(c1.p, v[j][c].p[i]);
          c2.p = f2fma(v[j][c].p[i], xh[j][c].p[i], c2.p);
        }
      }
      q[2 * j] = a.rms ? 0.f : c1.sum();
      q[2 * j + 1] = c2.sum();
    }
    group_totals<Q>(q, W, wi, 1 + group, s_buf[group][turn]);
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const uint32_t r = min(row + j, end - 1);
      const float k1 = -rstd[j] * (q[2 * j] * inv_h), k2 = -rstd[j] * (q[2 * j + 1] * inv_h);
      const uint64_t p1 = f2(k1, k1), p2 = f2(k2, k2), r2 = f2(rstd[j], rstd[j]);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v[j][c].p[i] = f2fma(v[j][c].p[i], r2, f2fma(xh[j][c].p[i], p2, p1));
        float f[V];
        get<V>(v[j][c], f);
        if constexpr (HASG) {
          float g[V];
          LooseRow<E>(a.g, r, a.H).read(spot(turn, j, 2), h[c], n[c], g);
#pragma unroll
          for (int i = 0; i < V; ++i) f[i] += g[i];
        }
        store_loose<F32>(a.dx, r, a.H, h[c], row + j < end ? n[c] : 0, f);
      }
    }
    turn ^= 1;
  }
  if (!a.d_weight && !a.d_bias) return;
  launch_dependents();
  // the block's sum over its groups, in group order, to its row of the partial sums
  __syncthreads();
  float* s_sum = reinterpret_cast<float*>(s_dyn);
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float* part = partial_row(a, which);
    if (!part) continue;
    const Vals<V>* acc = which ? acc_b : acc_g;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      float f[V];
      get<V>(acc[c], f);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i < n[c]) {
          if (G > 1) s_sum[(size_t)group * a.H + h[c] + 32 * i] = f[i];
          else part[h[c] + 32 * i] = f[i];
        }
    }
    if (G > 1) {
      __syncthreads();
      for (int i = threadIdx.x; i < a.H; i += blockDim.x) {
        float t = 0.f;
        for (int g = 0; g < G; ++g) t += s_sum[(size_t)g * a.H + i];
        part[i] = t;
      }
      __syncthreads();
    }
  }
}

// d_weight (blockIdx.y 0) and d_bias (1) from the blocks' partial sums: 32 features per block,
// its warps over the parts.
constexpr int kReduceWarps = 16, kPerWarp = (kParts + kReduceWarps - 1) / kReduceWarps;
__global__ void __launch_bounds__(32 * kReduceWarps) norm_reduce_kernel(
    const float* __restrict__ partial, int parts, int H, float* __restrict__ d_weight,
    float* __restrict__ d_bias) {
  __shared__ float s[kReduceWarps][33];
  float* out = blockIdx.y ? d_bias : d_weight;
  if (!out) return;  // uniform in the block
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int h = blockIdx.x * 32 + lane;
  float v = 0.f;
  wait_for_launcher();
  if (h < H) {
    const float* p = partial + (size_t)blockIdx.y * H + h;
    float each[kPerWarp];  // all requested before the first is added
#pragma unroll
    for (int i = 0; i < kPerWarp; ++i) {
      const int part = warp + i * kReduceWarps;
      each[i] = part < parts ? p[(size_t)part * 2 * H] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < kPerWarp; ++i) v += each[i];
  }
  s[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && h < H) {
#pragma unroll
    for (int i = 1; i < kReduceWarps; ++i) v += s[i][lane];
    out[h] = v;
  }
}

// ---- the checkpoint alone -------------------------------------------------------------------
// Bound by the bytes; a thread takes kEach vectors, a block apart, so that their loads are in
// flight together: T = 32768, H = 2880, bf16 stored in 50 us (5.7 TB/s) and read in 44 us (6.4
// TB/s), 63 and 53 us with one vector a thread.
constexpr int kEach = 4;
template <int FMT, bool F32>
__global__ void __launch_bounds__(256) checkpoint_pack_kernel(const void* x, long long chunks,
                                                              mxfp4_moe_checkpoint to) {
  const long long c0 = (long long)blockIdx.x * (256 * kEach) + threadIdx.x;
  Row<F32, 8> r[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    clear(r[i]);
    if (c0 + 256 * i < chunks) fetch<F32 ? kF32 : kBf16, 8>(r[i], x, (size_t)(c0 + 256 * i) * 8);
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const long long c = c0 + 256 * i;  // whole blocks of four lanes
    float v[8];
    values<F32 ? kF32 : kBf16, 8>(r[i], v);
    uint32_t byte;
    const uint2 q = encode8<FMT>(v, byte);
    if (c < chunks) {
      reinterpret_cast<uint2*>(to.codes)[c] = q;
      if ((c & 3) == 0) to.scales[c >> 2] = (uint8_t)byte;
    }
  }
}

template <int FMT, bool F32>
__global__ void __launch_bounds__(256) checkpoint_unpack_kernel(mxfp4_moe_checkpoint from,
                                                                long long chunks, void* x) {
  const long long c0 = (long long)blockIdx.x * (256 * kEach) + threadIdx.x;
  uint2 q[kEach];
  uint32_t byte[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    q[i] = make_uint2(0u, 0u);
    byte[i] = 127u;
    if (c0 + 256 * i < chunks) {
      q[i] = __ldg(reinterpret_cast<const uint2*>(from.codes) + c0 + 256 * i);
      byte[i] = __ldg(from.scales + ((c0 + 256 * i) >> 2));
    }
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    float v[8];
    decode8<FMT>(q[i], byte[i], v);
    if (c0 + 256 * i < chunks) store_rows<F32, 8>(x, (size_t)(c0 + 256 * i) * 8, v);
  }
}

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Rows of a batch from which the forward takes its persistent form.  Few rows / persistent, bf16:
//   rows        150        300        600       1200       2400   (32768 of 2880: 93 / 60 us)
//   H = 256   2.0 / 2.6  2.1 / 2.7  2.2 / 2.7  2.2 / 2.8  3.0 / 2.8 us
//   1024      2.5 / 3.0  2.6 / 3.1  3.7 / 3.1  5.2 / 3.2  8.1 / 3.8
//   2880      2.7 / 3.1  3.3 / 3.1  4.9 / 3.6  7.6 / 4.8   13 / 6.5
//   4096      3.1 / 2.8  4.5 / 3.3  6.6 / 4.2   11 / 5.6   19 / 8.7
//   16384     6.3 / 5.3  8.8 / 7.0   14 / 10    24 / 16    56 / 32
// The forms meet at about 2000 warps of the first one (T H / 256 up to H = 4096), so one number of
// rows is a compromise: short rows lose 0.6 us from it on, rows of 4096 and more 1 to 4 us below
// it.  fp32 rows with a residual meet later (600 rows of 2880: 7.0 / 9.5 us), rows without vector
// alignment at 500 to 1000 (1001: 5.3 / 5.7).  Rows in L2, as a batch of this size just written is.
constexpr int kManyRows = 600;

// Leave for a launch of `bytes` of dynamic shared memory.  The leave belongs to the kernel, not to
// the launch, and other host threads launch it for rows of other lengths: so every call asks for
// the same, the most that any H of this kernel takes.
template <int MOST, class K>
cudaError_t allow_shared(K kern, int bytes) {
  if (bytes > MOST) return cudaErrorInvalidValue;
  if (MOST <= 32 * 1024) return cudaSuccess;  // static shared memory included: 48 KB need no leave
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, MOST);
}
// Bytes of the unaligned rows that the warps of a block (NT / 32, NC vectors of 8 features a lane)
// hold at a time, at most: fewer groups of more warps pad less.
template <int NC, int E, int NT> constexpr int kLoosePlaces = NT / 32 * (16 + 256 * NC * E);

template <int SRC, bool F32, bool RES, int NC, int RB, int NT, int BLOCKS>
cudaError_t forward_persistent(const NormArgs& a, int W, int sms, cudaStream_t st) {
  auto kern = norm_forward_many_kernel<SRC, F32, RES, NC, RB, NT, BLOCKS>;
  const int groups = NT / (32 * W);
  constexpr int kWarpBytes = RB * NC * kStage<SRC> * (RES ? 2 : 1);
  const int smem = W * groups * kWarpBytes;  // at most 128 KB
  const cudaError_t e = allow_shared<NT / 32 * kWarpBytes>(kern, smem);
  if (e != cudaSuccess) return e;
  const long long need = ((long long)a.T + RB * groups - 1) / (RB * groups);
  const long long most = (long long)sms * BLOCKS;
  kern<<<(unsigned)(need < most ? need : most), 32 * W * groups, smem, st>>>(a, W);
  return cudaGetLastError();
}
template <bool F32, bool RES, int NC, int RB, int NT, int BLOCKS>
cudaError_t forward_loose(const NormArgs& a, int W, int sms, cudaStream_t st) {
  auto kern = norm_forward_loose_kernel<F32 ? kF32 : kBf16, F32, RES, NC, RB, NT, BLOCKS>;
  const int groups = NT / (32 * W);
  constexpr int E = F32 ? 4 : 2, kRowsHeld = 2 * RB * (RES ? 2 : 1);
  const int smem = groups * kRowsHeld * (int)LooseRow<E>::place(a.H);
  const cudaError_t e = allow_shared<kRowsHeld * kLoosePlaces<NC, E, NT>>(kern, smem);
  if (e != cudaSuccess) return e;
  const long long need = ((long long)a.T + RB * groups - 1) / (RB * groups);
  const long long most = (long long)sms * BLOCKS;
  kern<<<(unsigned)(need < most ? need : most), 32 * W * groups, smem, st>>>(a, W);
  return cudaGetLastError();
}
template <bool F32, int NC, int RB, int NT, int BLOCKS>
cudaError_t forward_loose_pick(const NormArgs& a, int W, int sms, cudaStream_t st) {
  return a.y ? forward_loose<F32, true, NC, RB, NT, BLOCKS>(a, W, sms, st)
             : forward_loose<F32, false, NC, RB, NT, BLOCKS>(a, W, sms, st);
}
template <int SRC, bool F32, int NC, int RB, int NT, int BLOCKS>
cudaError_t forward_many(const NormArgs& a, int W, int sms, cudaStream_t st) {
  if constexpr (SRC == kBf16 || SRC == kF32)
    if (a.y) return forward_persistent<SRC, F32, true, NC, RB, NT, BLOCKS>(a, W, sms, st);
  return forward_persistent<SRC, F32, false, NC, RB, NT, BLOCKS>(a, W, sms, st);
}
template <int SRC, bool F32, int V, int NC>
cudaError_t forward_few(const NormArgs& a, int W, cudaStream_t st) {
  const int groups = W >= 4 ? 1 : 4 / W;
  norm_forward_kernel<SRC, F32, V, NC>
      <<<(unsigned)(((long long)a.T + groups - 1) / groups), 32 * W * groups, 0, st>>>(a, W);
  return cudaGetLastError();
}

template <int SRC, bool F32>
cudaError_t forward_from(const NormArgs& a, bool vec, int sms, cudaStream_t st) {
  if (vec) {
    const int units = a.H / 8;
    auto warps = [&](int nc) { return (units + 32 * nc - 1) / (32 * nc); };
    if (a.T >= kManyRows) {
      if (units <= 384) return forward_many<SRC, F32, 1, 4, 384, 2>(a, warps(1), sms, st);
      if (units <= 512) return forward_many<SRC, F32, 1, 2, 512, 2>(a, warps(1), sms, st);
      if (units <= 1024) return forward_many<SRC, F32, 2, 2, 512, 1>(a, warps(2), sms, st);
      return forward_many<SRC, F32, 4, 1, 512, 1>(a, warps(4), sms, st);
    }
    if (units <= 512) return forward_few<SRC, F32, 8, 1>(a, warps(1), st);
    if (units <= 1024) return forward_few<SRC, F32, 8, 2>(a, warps(2), st);
    return forward_few<SRC, F32, 8, 4>(a, warps(4), st);
  }
  if constexpr (SRC == kBf16 || SRC == kF32) {
    if (a.T >= kManyRows && a.H <= 8192) {
      const int W1 = (a.H + 255) / 256;
      if (W1 <= 12) return forward_loose_pick<F32, 1, F32 ? 2 : 4, 384, 2>(a, W1, sms, st);
      if (W1 <= 16) return forward_loose_pick<F32, 1, F32 ? 1 : 2, 512, 2>(a, W1, sms, st);
      return forward_loose_pick<F32, 2, 1, 512, 1>(a, (a.H + 511) / 512, sms, st);
    }
    if (a.H <= 4096) return forward_few<SRC, F32, 1, 8>(a, (a.H + 255) / 256, st);
    return forward_few<SRC, F32, 1, 32>(a, (a.H + 1023) / 1024, st);
  }
  return cudaErrorInvalidValue;  // checkpoints are aligned
}

// Rows that a block of the backward walks over, and the blocks of a batch of T: as many as run at
// once (a block's partial sums cost a row of fp32 and its part of the second kernel).
struct Share {
  int rows, blocks;
};
Share share_rows(int T, int step, int per_sm) {
  const int most = kParts / 2 * per_sm;
  if (T <= step) return {T, 1};
  long long rows = ((long long)T + most - 1) / most;
  if (rows > step) rows = (rows + step - 1) / step * step;
  return {(int)rows, (int)((T + rows - 1) / rows)};
}

template <int SRC, bool F32, int V, bool HASG>
cudaError_t backward_long(const NormGradArgs& a, int* parts, cudaStream_t st) {
  const int W = (a.H + 1023) / 1024;
  const Share sh = share_rows(a.T, 1, 1);
  *parts = sh.blocks;
  norm_backward_long_kernel<SRC, F32, V, HASG><<<sh.blocks, 32 * W, 0, st>>>(a, W, sh.rows);
  return cudaGetLastError();
}

template <int SRC, bool F32, bool HASG, int NC, int R, int NT, int BLOCKS>
cudaError_t backward_staged(const NormGradArgs& a, int W, int* parts, cudaStream_t st) {
  auto kern = norm_backward_staged_kernel<SRC, F32, HASG, NC, R, NT, BLOCKS>;
  constexpr int kGrad = F32 ? kF32 : kBf16;
  const int groups = NT / (32 * W);
  constexpr int kTurns = R * NC * (kStage<SRC> + kStage<kGrad> * (HASG ? 2 : 1));
  constexpr int kSums = 4 * 256 * NC;  // the groups' sums at the end
  constexpr int kWarpBytes = kTurns > kSums ? kTurns : kSums;
  const int smem = W * groups * kWarpBytes;
  const cudaError_t e = allow_shared<NT / 32 * kWarpBytes>(kern, smem);
  if (e != cudaSuccess) return e;
  const Share sh = share_rows(a.T, R * groups, BLOCKS);
  *parts = sh.blocks;
  kern<<<sh.blocks, 32 * W * groups, smem, st>>>(a, W, sh.rows);
  return cudaGetLastError();
}

template <bool F32, bool HASG, int NC, int R, int NT, int BLOCKS>
cudaError_t backward_loose(const NormGradArgs& a, int W, int* parts, cudaStream_t st) {
  auto kern = norm_backward_loose_kernel<F32, HASG, NC, R, NT, BLOCKS>;
  const int groups = NT / (32 * W);
  constexpr int E = F32 ? 4 : 2, kRowsHeld = 2 * R * (HASG ? 3 : 2);
  static_assert(kRowsHeld * E >= 4, "the groups' sums at the end fit the rows' places");
  const int smem = groups * kRowsHeld * (int)LooseRow<E>::place(a.H);
  const cudaError_t e = allow_shared<kRowsHeld * kLoosePlaces<NC, E, NT>>(kern, smem);
  if (e != cudaSuccess) return e;
  const Share sh = share_rows(a.T, R * groups, BLOCKS);
  *parts = sh.blocks;
  kern<<<sh.blocks, 32 * W * groups, smem, st>>>(a, W, sh.rows);
  return cudaGetLastError();
}

template <int SRC, bool F32, bool HASG>
cudaError_t backward_from(const NormGradArgs& a, bool vec, int* parts, cudaStream_t st) {
  if (vec) {
    const int W1 = (a.H + 255) / 256, W2 = (a.H + 511) / 512;
    if (W1 <= 12) return backward_staged<SRC, F32, HASG, 1, 2, 384, 2>(a, W1, parts, st);
    if (W1 <= 16) return backward_staged<SRC, F32, HASG, 1, F32 ? 2 : 4, 512, 1>(a, W1, parts, st);
    if (W2 <= 16) return backward_staged<SRC, F32, HASG, 2, 1, 512, 1>(a, W2, parts, st);
    return backward_long<SRC, F32, 8, HASG>(a, parts, st);
  }
  if constexpr (SRC == kBf16 || SRC == kF32) {
    const int W1 = (a.H + 255) / 256;
    if (W1 <= 12) return backward_loose<F32, HASG, 1, F32 ? 1 : 2, 384, 2>(a, W1, parts, st);
    if (W1 <= 16) return backward_loose<F32, HASG, 1, F32 ? 1 : 2, 512, 1>(a, W1, parts, st);
    if (W1 <= 32) return backward_loose<F32, HASG, 2, 1, 512, 1>(a, (a.H + 511) / 512, parts, st);
    return backward_long<SRC, F32, 1, HASG>(a, parts, st);
  }
  return cudaErrorInvalidValue;  // checkpoints are aligned
}

template <int SRC, bool F32>
cudaError_t backward_pick(const NormGradArgs& a, bool vec, int* parts, cudaStream_t st) {
  return a.g ? backward_from<SRC, F32, true>(a, vec, parts, st)
             : backward_from<SRC, F32, false>(a, vec, parts, st);
}

}  // namespace

cudaError_t launch_norm_forward(const NormArgs& a, int sms, cudaStream_t st) {
  if (a.T == 0) return cudaSuccess;
  const bool vec = a.H % 8 == 0 && al16(a.x) && al16(a.y) && al16(a.x_out) && al16(a.out) &&
                   al16(a.weight) && al16(a.bias);
  if (a.from.codes) {
    if (a.from.format == MXFP4_MOE_CHECKPOINT_E4M3)
      return a.rows_f32 ? forward_from<kE4m3, true>(a, vec, sms, st) : forward_from<kE4m3, false>(a, vec, sms, st);
    return a.rows_f32 ? forward_from<kInt8, true>(a, vec, sms, st) : forward_from<kInt8, false>(a, vec, sms, st);
  }
  return a.rows_f32 ? forward_from<kF32, true>(a, vec, sms, st) : forward_from<kBf16, false>(a, vec, sms, st);
}

size_t norm_scratch_bytes(int T, int H) {
  return 8 * (size_t)(T < kParts ? T : kParts) * (size_t)H;
}

cudaError_t launch_norm_backward(const NormGradArgs& a, int, cudaStream_t st) {
  int parts = 0;
  if (a.T > 0) {
    const bool vec = a.H % 8 == 0 && al16(a.x) && al16(a.d_out) && al16(a.g) && al16(a.dx) &&
                     al16(a.weight);
    cudaError_t e;
    if (a.from.codes && a.from.format == MXFP4_MOE_CHECKPOINT_E4M3)
      e = a.rows_f32 ? backward_pick<kE4m3, true>(a, vec, &parts, st)
                     : backward_pick<kE4m3, false>(a, vec, &parts, st);
    else if (a.from.codes)
      e = a.rows_f32 ? backward_pick<kInt8, true>(a, vec, &parts, st)
                     : backward_pick<kInt8, false>(a, vec, &parts, st);
    else
      e = a.rows_f32 ? backward_pick<kF32, true>(a, vec, &parts, st)
                     : backward_pick<kBf16, false>(a, vec, &parts, st);
    if (e != cudaSuccess) return e;
  }
  if (!a.d_weight && !a.d_bias) return cudaSuccess;
  if (parts == 1) return cudaSuccess;  // one block writes the gradients itself
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((a.H + 31) / 32, 2);
  cfg.blockDim = dim3(32 * kReduceWarps);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = parts > 0 ? 1 : 0;  // T = 0: no kernel to overlap
  return cudaLaunchKernelEx(&cfg, norm_reduce_kernel, (const float*)a.partial, parts, a.H,
                            a.d_weight, a.d_bias);
}

cudaError_t launch_checkpoint_pack(int T, int H, bool rows_f32, const void* x,
                                   const mxfp4_moe_checkpoint& to, cudaStream_t st) {
  const long long chunks = (long long)T * H / 8;
  if (chunks == 0) return cudaSuccess;
  const unsigned blocks = (unsigned)((chunks + 256 * kEach - 1) / (256 * kEach));
  auto kern = to.format == MXFP4_MOE_CHECKPOINT_E4M3
                  ? (rows_f32 ? checkpoint_pack_kernel<kE4m3, true> : checkpoint_pack_kernel<kE4m3, false>)
                  : (rows_f32 ? checkpoint_pack_kernel<kInt8, true> : checkpoint_pack_kernel<kInt8, false>);
  kern<<<blocks, 256, 0, st>>>(x, chunks, to);
  return cudaGetLastError();
}

cudaError_t launch_checkpoint_unpack(int T, int H, bool rows_f32,
                                     const mxfp4_moe_checkpoint& from, void* x, cudaStream_t st) {
  const long long chunks = (long long)T * H / 8;
  if (chunks == 0) return cudaSuccess;
  const unsigned blocks = (unsigned)((chunks + 256 * kEach - 1) / (256 * kEach));
  auto kern = from.format == MXFP4_MOE_CHECKPOINT_E4M3
                  ? (rows_f32 ? checkpoint_unpack_kernel<kE4m3, true> : checkpoint_unpack_kernel<kE4m3, false>)
                  : (rows_f32 ? checkpoint_unpack_kernel<kInt8, true> : checkpoint_unpack_kernel<kInt8, false>);
  kern<<<blocks, 256, 0, st>>>(from, chunks, x);
  return cudaGetLastError();
}

}  // namespace moe
