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

MOE_DEV float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// ---- rows of bf16 or fp32 -----------------------------------------------------------------
// V consecutive features as floats: V = 8 in 16-byte vectors, V = 1 alone.  Loads are plain
// (not the read-only path): an output may be the same buffer as the gradient it is added to.
template <bool F32, int V>
MOE_DEV void load_rows(const void* base, size_t at, float (&v)[V]) {
  if constexpr (F32) {
    const float* p = static_cast<const float*>(base) + at;
    if constexpr (V == 8) {
      const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
      v[0] = *p;
    }
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(base) + at;
    if constexpr (V == 8) {
      const uint4 q = *reinterpret_cast<const uint4*>(p);
      v[0] = bf16_lo(q.x); v[1] = bf16_hi(q.x); v[2] = bf16_lo(q.y); v[3] = bf16_hi(q.y);
      v[4] = bf16_lo(q.z); v[5] = bf16_hi(q.z); v[6] = bf16_lo(q.w); v[7] = bf16_hi(q.w);
    } else {
      v[0] = bf16_to_f(*p);
    }
  }
}
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
      *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    else
      *p = f_to_bf16(v[0]);
  }
}
// fp32 values as the row type holds them
template <bool F32, int V>
MOE_DEV void round_rows(float (&v)[V]) {
  if constexpr (!F32) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = bf16_to_f(f_to_bf16(v[i]));
  }
}
template <int V>
MOE_DEV void load_params(const void* base, bool f32, size_t at, float absent, float (&v)[V]) {
  if (!base) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = absent;
  } else if (f32) {
    load_rows<true, V>(base, at, v);
  } else {
    load_rows<false, V>(base, at, v);
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
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t h2;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)(w[i >> 1] >> (16 * (i & 1)))));
      const __half2 hh = *reinterpret_cast<const __half2*>(&h2);
      v[2 * i] = __low2float(hh) * s;
      v[2 * i + 1] = __high2float(hh) * s;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // the byte with its sign bit flipped is code + 128, set into the fraction of 2^23
      const uint32_t u = prmt(w[i >> 2] ^ 0x80808080u, 0x4B000000u, 0x7440u | (uint32_t)(i & 3));
      v[i] = (__uint_as_float(u) - 8388736.f) * 0.015625f * s;
    }
  }
}

// Rows of a pass from any source, 8 (or 1) features at a time.
template <int SRC, int V>
MOE_DEV void load_source(const void* x, const mxfp4_moe_checkpoint& from, size_t at, float (&v)[V]) {
  if constexpr (SRC == kBf16 || SRC == kF32) {
    load_rows<SRC == kF32, V>(x, at, v);
  } else {
    const uint2 q = __ldg(reinterpret_cast<const uint2*>(from.codes + at));
    decode8<SRC>(q, __ldg(from.scales + at / 32), v);
  }
}

// ---- forward --------------------------------------------------------------------------------
// A row is held in registers by W warps (V NC features a thread), so it is read once for the
// mean, the variance about that mean and the output.  W = 1 reduces by shuffles alone; larger
// rows add one exchange through shared memory per statistic behind a barrier of the row's own
// warps.  Bound by the rows' bytes.
struct RowGroup {  // the W warps of a row
  int W, warp, bar;
  float* buf;  // [2][32] floats of shared memory
  MOE_DEV float sum(float v, int slot) const {
    v = warp_sum(v);
    if (W == 1) return v;
    const int lane = threadIdx.x & 31;
    if (lane == 0) buf[32 * slot + warp] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(32 * W) : "memory");
    return warp_sum(lane < W ? buf[32 * slot + lane] : 0.f);
  }
};

constexpr int kNormThreads = 512;  // most threads of a block (16 warps)

template <int SRC, bool F32, int V, int NC>
__global__ void __launch_bounds__(kNormThreads) norm_forward_kernel(NormArgs a, int W) {
  __shared__ float s_buf[16][64];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = warp / W, wi = warp % W;
  const long long row = (long long)blockIdx.x * (blockDim.x / (32 * W)) + group;
  if (row >= a.T) return;  // whole groups leave together
  const RowGroup rg{W, wi, 1 + group, s_buf[group]};
  const size_t r0 = (size_t)row * a.H;
  float v[NC][V];
  float part = 0.f;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int h = V * ((c * W + wi) * 32 + lane);
    const bool in = h < a.H;
#pragma unroll
    for (int i = 0; i < V; ++i) v[c][i] = 0.f;
    if (in) load_source<SRC, V>(a.x, a.from, r0 + h, v[c]);
    if constexpr (SRC == kBf16 || SRC == kF32) {
      if (a.y) {
        if (in) {
          float y[V];
          load_rows<F32, V>(a.y, r0 + h, y);
#pragma unroll
          for (int i = 0; i < V; ++i) v[c][i] += y[i];
          round_rows<F32, V>(v[c]);
          store_rows<F32, V>(a.x_out, r0 + h, v[c]);
        }
      }
      if constexpr (V == 8) {
        if (a.to.codes) {  // all lanes take part: H is a multiple of 32, so a block's four do
          uint32_t byte;
          const uint2 q = a.to.format == MXFP4_MOE_CHECKPOINT_E4M3 ? encode8<kE4m3>(v[c], byte)
                                                                   : encode8<kInt8>(v[c], byte);
          if (in) {
            *reinterpret_cast<uint2*>(a.to.codes + r0 + h) = q;
            if ((lane & 3) == 0) a.to.scales[(r0 + h) / 32] = (uint8_t)byte;
          }
        }
      }
    }
    if (!a.rms) {
#pragma unroll
      for (int i = 0; i < V; ++i) part += v[c][i];
    }
  }
  const float mean = a.rms ? 0.f : rg.sum(part, 0) / (float)a.H;
  part = 0.f;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int h = V * ((c * W + wi) * 32 + lane);
    if (h < a.H) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        v[c][i] -= mean;
        part += v[c][i] * v[c][i];
      }
    }
  }
  const float rstd = 1.f / sqrtf(rg.sum(part, 1) / (float)a.H + a.eps);
  if (wi == 0 && lane == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int h = V * ((c * W + wi) * 32 + lane);
    if (h < a.H) {
      float g[V], b[V];
      load_params<V>(a.weight, a.param_f32, h, 1.f, g);
      load_params<V>(a.bias, a.param_f32, h, 0.f, b);
#pragma unroll
      for (int i = 0; i < V; ++i) v[c][i] = fmaf(v[c][i] * rstd, g[i], b[i]);
      store_rows<F32, V>(a.out, r0 + h, v[c]);
    }
  }
}

// ---- backward -------------------------------------------------------------------------------
// A block walks over its share of the rows; a thread keeps the same features throughout, so the
// parameters' gradients accumulate in its registers and leave once per block (a second kernel
// adds the blocks' partial sums in a fixed order).
constexpr int kParts = 296;  // most blocks, two per SM of a B200

template <int SRC, bool F32, int V, int NC>
__global__ void __launch_bounds__(kNormThreads) norm_backward_kernel(NormGradArgs a, int W,
                                                                     int rows_per_block) {
  __shared__ float s_buf[16][2][64];
  __shared__ float s_sum[kNormThreads * V * NC / 2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = blockDim.x / (32 * W), group = warp / W, wi = warp % W;
  float acc_g[NC][V], acc_b[NC][V];
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < V; ++i) acc_g[c][i] = acc_b[c][i] = 0.f;
  const long long row_end = min((long long)a.T, (long long)(blockIdx.x + 1) * rows_per_block);
  int turn = 0;
  for (long long row = (long long)blockIdx.x * rows_per_block + group; row < row_end; row += G) {
    const RowGroup rg{W, wi, 1 + group, s_buf[group][turn]};
    turn ^= 1;  // the next row's exchange must not meet this one's readers
    const size_t r0 = (size_t)row * a.H;
    const float mean = a.rms ? 0.f : __ldg(a.mean + row), rstd = __ldg(a.rstd + row);
    float xh[NC][V], v[NC][V];
    float c1 = 0.f, c2 = 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int h = V * ((c * W + wi) * 32 + lane);
      if (h < a.H) {
        float d[V], g[V];
        load_source<SRC, V>(a.x, a.from, r0 + h, xh[c]);
        load_rows<F32, V>(a.d_out, r0 + h, d);
        load_params<V>(a.weight, a.param_f32, h, 1.f, g);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          xh[c][i] = (xh[c][i] - mean) * rstd;
          v[c][i] = d[i] * g[i];
          c1 += v[c][i];
          c2 += v[c][i] * xh[c][i];
          acc_g[c][i] += d[i] * xh[c][i];
          acc_b[c][i] += d[i];
        }
      }
    }
    c1 = a.rms ? 0.f : rg.sum(c1, 0) / (float)a.H;
    c2 = rg.sum(c2, 1) / (float)a.H;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int h = V * ((c * W + wi) * 32 + lane);
      if (h < a.H) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[c][i] = rstd * (v[c][i] - c1 - xh[c][i] * c2);
        if (a.g) {
          float g[V];
          load_rows<F32, V>(a.g, r0 + h, g);
#pragma unroll
          for (int i = 0; i < V; ++i) v[c][i] += g[i];
        }
        store_rows<F32, V>(a.dx, r0 + h, v[c]);
      }
    }
  }
  if (!a.d_weight && !a.d_bias) return;
  // the block's sum over its groups, in group order, to its row of the partial sums
  float* part = a.partial + (size_t)blockIdx.x * 2 * a.H;
  for (int which = 0; which < 2; ++which) {
    // groups other than the first pass theirs through shared memory one at a time
    for (int other = 1; other < G; ++other) {
      __syncthreads();
      if (group == other) {
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int i = 0; i < V; ++i)
            s_sum[V * ((c * W + wi) * 32 + lane) + i] = which ? acc_b[c][i] : acc_g[c][i];
      }
      __syncthreads();
      if (group == 0) {
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float o = s_sum[V * ((c * W + wi) * 32 + lane) + i];
            if (which) acc_b[c][i] += o; else acc_g[c][i] += o;
          }
      }
    }
    if (group == 0) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int h = V * ((c * W + wi) * 32 + lane);
        if (h < a.H) {
#pragma unroll
          for (int i = 0; i < V; ++i) part[which * a.H + h + i] = which ? acc_b[c][i] : acc_g[c][i];
        }
      }
    }
  }
}

// d_weight (blockIdx.y 0) and d_bias (1) from the blocks' partial sums: 32 features per block,
// eight warps over the parts.
__global__ void __launch_bounds__(256) norm_reduce_kernel(const float* __restrict__ partial,
                                                          int parts, int H,
                                                          float* __restrict__ d_weight,
                                                          float* __restrict__ d_bias) {
  __shared__ float s[8][33];
  float* out = blockIdx.y ? d_bias : d_weight;
  if (!out) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int h = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (h < H)
    for (int p = warp; p < parts; p += 8) v += partial[((size_t)p * 2 + blockIdx.y) * H + h];
  s[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && h < H) {
#pragma unroll
    for (int i = 1; i < 8; ++i) v += s[i][lane];
    out[h] = v;
  }
}

// ---- the checkpoint alone -------------------------------------------------------------------
template <int FMT, bool F32>
__global__ void __launch_bounds__(256) checkpoint_pack_kernel(const void* x, long long chunks,
                                                              mxfp4_moe_checkpoint to) {
  const long long c = (long long)blockIdx.x * 256 + threadIdx.x;
  const bool in = c < chunks;  // whole blocks of four lanes
  float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (in) load_rows<F32, 8>(x, (size_t)c * 8, v);
  uint32_t byte;
  const uint2 q = encode8<FMT>(v, byte);
  if (in) {
    reinterpret_cast<uint2*>(to.codes)[c] = q;
    if ((c & 3) == 0) to.scales[c >> 2] = (uint8_t)byte;
  }
}

template <int FMT, bool F32>
__global__ void __launch_bounds__(256) checkpoint_unpack_kernel(mxfp4_moe_checkpoint from,
                                                                long long chunks, void* x) {
  const long long c = (long long)blockIdx.x * 256 + threadIdx.x;
  if (c >= chunks) return;
  float v[8];
  decode8<FMT>(__ldg(reinterpret_cast<const uint2*>(from.codes) + c), __ldg(from.scales + (c >> 2)), v);
  store_rows<F32, 8>(x, (size_t)c * 8, v);
}

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Features a thread holds, and the warps that hold a row, for rows of H features in vectors of V.
struct Split {
  int per_thread, W;
};
Split split_row(int H, int V, int most_warps) {
  const int units = (H + V - 1) / V;
  for (int nc = 8 / V; nc < 32 / V; nc *= 2) {
    const int W = (units + 32 * nc - 1) / (32 * nc);
    if (W <= most_warps) return {nc * V, W};
  }
  return {32, (units * V + 1023) / 1024};
}

template <int SRC, bool F32>
cudaError_t forward_from(const NormArgs& a, bool vec, cudaStream_t st) {
  const Split s = split_row(a.H, vec ? 8 : 1, 4);
  const int groups = s.W >= 8 ? 1 : 8 / s.W;
  const unsigned blocks = (unsigned)(((long long)a.T + groups - 1) / groups);
  const int threads = 32 * s.W * groups;
  if (vec) {
    if (s.per_thread == 8) norm_forward_kernel<SRC, F32, 8, 1><<<blocks, threads, 0, st>>>(a, s.W);
    else if (s.per_thread == 16) norm_forward_kernel<SRC, F32, 8, 2><<<blocks, threads, 0, st>>>(a, s.W);
    else norm_forward_kernel<SRC, F32, 8, 4><<<blocks, threads, 0, st>>>(a, s.W);
  } else if constexpr (SRC == kBf16 || SRC == kF32) {
    if (s.per_thread == 8) norm_forward_kernel<SRC, F32, 1, 8><<<blocks, threads, 0, st>>>(a, s.W);
    else if (s.per_thread == 16) norm_forward_kernel<SRC, F32, 1, 16><<<blocks, threads, 0, st>>>(a, s.W);
    else norm_forward_kernel<SRC, F32, 1, 32><<<blocks, threads, 0, st>>>(a, s.W);
  } else {
    return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

template <int SRC, bool F32>
cudaError_t backward_from(const NormGradArgs& a, bool vec, cudaStream_t st) {
  const Split s = split_row(a.H, vec ? 8 : 1, 16);
  const int groups = s.W >= 8 ? 1 : 8 / s.W;
  const int threads = 32 * s.W * groups;
  const int rows = (int)(((long long)a.T + kParts - 1) / kParts);
  const unsigned blocks = (unsigned)((a.T + (long long)rows - 1) / rows);
  if (vec) {
    if (s.per_thread == 8) norm_backward_kernel<SRC, F32, 8, 1><<<blocks, threads, 0, st>>>(a, s.W, rows);
    else if (s.per_thread == 16) norm_backward_kernel<SRC, F32, 8, 2><<<blocks, threads, 0, st>>>(a, s.W, rows);
    else norm_backward_kernel<SRC, F32, 8, 4><<<blocks, threads, 0, st>>>(a, s.W, rows);
  } else if constexpr (SRC == kBf16 || SRC == kF32) {
    if (s.per_thread == 8) norm_backward_kernel<SRC, F32, 1, 8><<<blocks, threads, 0, st>>>(a, s.W, rows);
    else if (s.per_thread == 16) norm_backward_kernel<SRC, F32, 1, 16><<<blocks, threads, 0, st>>>(a, s.W, rows);
    else norm_backward_kernel<SRC, F32, 1, 32><<<blocks, threads, 0, st>>>(a, s.W, rows);
  } else {
    return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_forward(const NormArgs& a, int, cudaStream_t st) {
  if (a.T == 0) return cudaSuccess;
  const bool vec = a.H % 8 == 0 && al16(a.x) && al16(a.y) && al16(a.x_out) && al16(a.out) &&
                   al16(a.weight) && al16(a.bias);
  if (a.from.codes) {
    if (a.from.format == MXFP4_MOE_CHECKPOINT_E4M3)
      return a.rows_f32 ? forward_from<kE4m3, true>(a, vec, st) : forward_from<kE4m3, false>(a, vec, st);
    return a.rows_f32 ? forward_from<kInt8, true>(a, vec, st) : forward_from<kInt8, false>(a, vec, st);
  }
  return a.rows_f32 ? forward_from<kF32, true>(a, vec, st) : forward_from<kBf16, false>(a, vec, st);
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
    if (a.from.codes)
      e = a.from.format == MXFP4_MOE_CHECKPOINT_E4M3
              ? (a.rows_f32 ? backward_from<kE4m3, true>(a, vec, st) : backward_from<kE4m3, false>(a, vec, st))
              : (a.rows_f32 ? backward_from<kInt8, true>(a, vec, st) : backward_from<kInt8, false>(a, vec, st));
    else
      e = a.rows_f32 ? backward_from<kF32, true>(a, vec, st) : backward_from<kBf16, false>(a, vec, st);
    if (e != cudaSuccess) return e;
    const int rows = (int)(((long long)a.T + kParts - 1) / kParts);
    parts = (a.T + rows - 1) / rows;
  }
  if (!a.d_weight && !a.d_bias) return cudaSuccess;
  norm_reduce_kernel<<<dim3((a.H + 31) / 32, 2), 256, 0, st>>>(a.partial, parts, a.H, a.d_weight,
                                                              a.d_bias);
  return cudaGetLastError();
}

cudaError_t launch_checkpoint_pack(int T, int H, bool rows_f32, const void* x,
                                   const mxfp4_moe_checkpoint& to, cudaStream_t st) {
  const long long chunks = (long long)T * H / 8;
  if (chunks == 0) return cudaSuccess;
  const unsigned blocks = (unsigned)((chunks + 255) / 256);
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
  const unsigned blocks = (unsigned)((chunks + 255) / 256);
  auto kern = from.format == MXFP4_MOE_CHECKPOINT_E4M3
                  ? (rows_f32 ? checkpoint_unpack_kernel<kE4m3, true> : checkpoint_unpack_kernel<kE4m3, false>)
                  : (rows_f32 ? checkpoint_unpack_kernel<kInt8, true> : checkpoint_unpack_kernel<kInt8, false>);
  kern<<<blocks, 256, 0, st>>>(from, chunks, x);
  return cudaGetLastError();
}

}  // namespace moe
