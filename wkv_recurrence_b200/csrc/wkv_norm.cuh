// RMS norm of the residual stream, by groups (heads) of a row, and its
// gradients. Per row of C columns, G groups of D = C / G:
//     s = round(x + residual)        (the type the residual stream is held in)
//     r = (mean over the group of s^2 + eps)^-1/2,   y = s r weight
// y in 16 or 32 bits, or in e4m3 with a scale for each block of columns (or
// each row): scale = max |y| / 448, q = y / scale.
//     p = gy weight,  ds = gs + r (p - s r^2 mean(p s)),  dweight = sum over rows of gy s r.
//
// y is the norm of the rounded s, the value that the stream carries on, so
// forward and backward are about the same s.
//
// Bound: memory traffic; every kernel reads its inputs once into registers
// (wkv_norm_row apart, see there) and reduces while they stay there.
#pragma once

#include <cuda_fp8.h>

#include "wkv_device.cuh"

namespace wkv {

constexpr float kE4m3Max = 448.f;
constexpr int kNV = 8;  // columns per vector: 16 bytes of bf16, 32 of fp32

// Eight adjacent columns as they lie in memory.
template <typename T>
struct Vec8;
template <>
struct Vec8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
  __device__ __forceinline__ static void store(float* p, const float (&x)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
};
template <>
struct Vec8<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    unpack_bf16x2(a.x, x[0], x[1]);
    unpack_bf16x2(a.y, x[2], x[3]);
    unpack_bf16x2(a.z, x[4], x[5]);
    unpack_bf16x2(a.w, x[6], x[7]);
  }
  __device__ __forceinline__ static void store(__nv_bfloat16* p, const float (&x)[8]) {
    uint4 o;
    __nv_bfloat162 t;
    t = __floats2bfloat162_rn(x[0], x[1]), o.x = *reinterpret_cast<uint32_t*>(&t);
    t = __floats2bfloat162_rn(x[2], x[3]), o.y = *reinterpret_cast<uint32_t*>(&t);
    t = __floats2bfloat162_rn(x[4], x[5]), o.z = *reinterpret_cast<uint32_t*>(&t);
    t = __floats2bfloat162_rn(x[6], x[7]), o.w = *reinterpret_cast<uint32_t*>(&t);
    *reinterpret_cast<uint4*>(p) = o;
  }
};

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// The scale of a block whose largest |y| is `top`: 1 for a block of zeros, and
// never below the smallest normal number, so its inverse is finite.
__device__ __forceinline__ float e4m3_scale(float top) {
  return top > 0.f ? fmaxf(top / kE4m3Max, 1.17549435e-38f) : 1.f;
}

enum { kOutF32 = 0, kOutBf16 = 1, kOutE4m3 = 2 };

struct NormParams {
  long long N;
  int C, G, D;
  float eps;
  const void* x;
  long long x_st;       // element stride of x's rows
  const void* res;      // or NULL
  long long res_st;
  const float* weight;  // [C]
  void* y;              // [N, C], by out_kind
  int out_kind;
  void* s;              // [N, C] in the residual's type, or NULL (no residual); may be res
  float* scale;         // [N, C / block], e4m3 only
  int block;            // columns per scale, C for the whole row
};

template <int W>
__device__ __forceinline__ float team_sum(float v) {
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float lanes_max(float v, int width) {  // over `width` (a power of two) adjacent lanes
  for (int o = width / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Sum (or maximum) over the CTA's threads, the same for every thread; red has 32 floats.
template <bool MAX>
__device__ __forceinline__ float cta_reduce(float v, float* red) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = (blockDim.x + 31) >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float u = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? fmaxf(v, u) : v + u;
  }
  __syncthreads();  // red may still be read from the reduction before
  if (lane == 0) red[w] = v;
  __syncthreads();
  v = lane < nw ? red[lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float u = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? fmaxf(v, u) : v + u;
  }
  return v;
}

// ---------------------------------------------------------------------------
// forward, one team of threads per group
// ---------------------------------------------------------------------------
// TW lanes (TW <= 32: several teams per warp) or the whole CTA (TW = 0) hold
// one group's D columns in registers, K vectors of 8 per thread; vector k of
// team lane l is columns 8 (k TW + l). Takes 16-byte aligned rows with D a
// multiple of 8, and e4m3 scales whose block lies inside a group (the whole
// group, or 32, 64 or 128 columns held by adjacent lanes in one k).
template <typename X, typename R, bool RES, int TW, int K>
__global__ void __launch_bounds__(TW ? 256 : 1024) wkv_norm_team(const NormParams p) {
  __shared__ float red[32];
  const int width = TW ? TW : (int)blockDim.x;
  const int tl = TW ? (int)(threadIdx.x % width) : (int)threadIdx.x;
  const long long seg = TW ? (long long)blockIdx.x * (256 / width) + threadIdx.x / width : (long long)blockIdx.x;
  const bool live = seg < p.N * p.G;
  const long long row = live ? seg / p.G : 0;
  const int g = live ? (int)(seg - row * p.G) : 0;
  const X* xp = static_cast<const X*>(p.x) + row * p.x_st + (long long)g * p.D;
  const R* rp = RES ? static_cast<const R*>(p.res) + row * p.res_st + (long long)g * p.D : nullptr;
  Vec8<X> xv[K];
  Vec8<R> rv[K];
  bool in[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int col = (k * width + tl) * kNV;
    in[k] = live && col < p.D;
    if (in[k]) {
      xv[k].load(xp + col);
      if (RES) rv[k].load(rp + col);
    }
  }
  float s[K][kNV];
  float sum = 0.f;
  const long long o = row * p.C + (long long)g * p.D;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (in[k]) {
      xv[k].get(s[k]);
      if (RES) {
        float r[kNV];
        rv[k].get(r);
#pragma unroll
        for (int e = 0; e < kNV; ++e) s[k][e] = Elem<R>::to_f32(Elem<R>::from_f32(s[k][e] + r[e]));
        Vec8<R>::store(static_cast<R*>(p.s) + o + (k * width + tl) * kNV, s[k]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < kNV; ++e) s[k][e] = 0.f;
    }
#pragma unroll
    for (int e = 0; e < kNV; ++e) sum = fmaf(s[k][e], s[k][e], sum);
  }
  sum = TW ? team_sum<TW ? TW : 32>(sum) : cta_reduce<false>(sum, red);
  const float r = 1.f / sqrtf(sum / (float)p.D + p.eps);
  const float* wp = p.weight + (long long)g * p.D;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (in[k]) {
      Vec8<float> wv;
      float w[kNV];
      wv.load(wp + (k * width + tl) * kNV);
      wv.get(w);
#pragma unroll
      for (int e = 0; e < kNV; ++e) s[k][e] = s[k][e] * r * w[e];
    }
  }
  if (p.out_kind != kOutE4m3) {
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (in[k]) {
        const long long at = o + (k * width + tl) * kNV;
        if (p.out_kind == kOutF32) Vec8<float>::store(static_cast<float*>(p.y) + at, s[k]);
        else Vec8<__nv_bfloat16>::store(static_cast<__nv_bfloat16*>(p.y) + at, s[k]);
      }
    return;
  }
  float top[K];
  float all = 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    top[k] = 0.f;
#pragma unroll
    for (int e = 0; e < kNV; ++e) top[k] = fmaxf(top[k], fabsf(s[k][e]));
    all = fmaxf(all, top[k]);
  }
  const bool whole = p.block == p.D;
  if (whole) all = TW ? lanes_max(all, width) : cta_reduce<true>(all, red);
  const int per = whole ? width : p.block / kNV;  // threads that share a scale
  const int nb = p.C / p.block;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const float m = whole ? all : lanes_max(top[k], per);
    const float sc = e4m3_scale(m), inv = 1.f / sc;
    if (in[k]) {
      const int col = (k * width + tl) * kNV;
      uint2 q;
      q.x = e4m3x4(s[k][0] * inv, s[k][1] * inv, s[k][2] * inv, s[k][3] * inv);
      q.y = e4m3x4(s[k][4] * inv, s[k][5] * inv, s[k][6] * inv, s[k][7] * inv);
      *reinterpret_cast<uint2*>(static_cast<unsigned char*>(p.y) + o + col) = q;
      if (tl % per == 0 && (!whole || k == 0)) p.scale[row * nb + ((long long)g * p.D + col) / p.block] = sc;
    }
  }
}

// ---------------------------------------------------------------------------
// forward, one CTA per row, any size, alignment and scale block
// ---------------------------------------------------------------------------
// Three walks over the row: s (written where there is a residual) and the
// groups' sums; the scales' maxima; the output. The second and third read the
// row again from L1/L2. Shared memory: one float per group.
__device__ __forceinline__ float load_any(const void* p, bool bf, long long i) {
  return bf ? Elem<__nv_bfloat16>::to_f32(static_cast<const __nv_bfloat16*>(p)[i]) : static_cast<const float*>(p)[i];
}

__global__ void __launch_bounds__(256) wkv_norm_row(const NormParams p, bool x_bf, bool r_bf) {
  extern __shared__ float rstd[];  // [G]
  __shared__ float red[32];
  const long long row = blockIdx.x;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const long long xo = row * p.x_st, ro = row * p.res_st, o = row * p.C;
  const bool has_res = p.res != nullptr;
  const void* src = has_res ? p.s : p.x;  // where s can be read again
  const bool src_bf = has_res ? r_bf : x_bf;
  const long long so = has_res ? o : xo;
  auto first = [&](int c) {
    float s = load_any(p.x, x_bf, xo + c);
    if (has_res) {
      s += load_any(p.res, r_bf, ro + c);
      if (r_bf) {
        const __nv_bfloat16 b = __float2bfloat16_rn(s);
        static_cast<__nv_bfloat16*>(p.s)[o + c] = b;
        s = __bfloat162float(b);
      } else {
        static_cast<float*>(p.s)[o + c] = s;
      }
    }
    return s;
  };
  if (p.G == 1) {
    float sum = 0.f;
    for (int c = threadIdx.x; c < p.C; c += blockDim.x) {
      const float s = first(c);
      sum = fmaf(s, s, sum);
    }
    sum = cta_reduce<false>(sum, red);
    if (threadIdx.x == 0) rstd[0] = 1.f / sqrtf(sum / (float)p.D + p.eps);
  } else {
    for (int g = w; g < p.G; g += nw) {  // a warp per group
      float sum = 0.f;
      for (int c = lane; c < p.D; c += 32) {
        const float s = first(g * p.D + c);
        sum = fmaf(s, s, sum);
      }
      sum = team_sum<32>(sum);
      if (lane == 0) rstd[g] = 1.f / sqrtf(sum / (float)p.D + p.eps);
    }
  }
  __threadfence_block();
  __syncthreads();  // rstd, and s as written above, are there for every thread
  auto value = [&](int c) {
    return load_any(src, src_bf, so + c) * rstd[p.G == 1 ? 0 : c / p.D] * __ldg(p.weight + c);
  };
  if (p.out_kind != kOutE4m3) {
    for (int c = threadIdx.x; c < p.C; c += blockDim.x) {
      const float y = value(c);
      if (p.out_kind == kOutF32) static_cast<float*>(p.y)[o + c] = y;
      else static_cast<__nv_bfloat16*>(p.y)[o + c] = __float2bfloat16_rn(y);
    }
    return;
  }
  auto put = [&](int c, float y, float inv) {
    static_cast<unsigned char*>(p.y)[o + c] = (unsigned char)__nv_cvt_float_to_fp8(y * inv, __NV_SATFINITE, __NV_E4M3);
  };
  if (p.block == p.C) {
    float top = 0.f;
    for (int c = threadIdx.x; c < p.C; c += blockDim.x) top = fmaxf(top, fabsf(value(c)));
    const float sc = e4m3_scale(cta_reduce<true>(top, red)), inv = 1.f / sc;
    if (threadIdx.x == 0) p.scale[row] = sc;
    for (int c = threadIdx.x; c < p.C; c += blockDim.x) put(c, value(c), inv);
  } else {
    const int nb = p.C / p.block;
    for (int b = w; b < nb; b += nw) {  // a warp per block of at most 128 columns
      float y[4], top = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y[i] = i * 32 + lane < p.block ? value(b * p.block + i * 32 + lane) : 0.f;
        top = fmaxf(top, fabsf(y[i]));
      }
      const float sc = e4m3_scale(lanes_max(top, 32)), inv = 1.f / sc;
      if (lane == 0) p.scale[row * nb + b] = sc;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i * 32 + lane < p.block) put(b * p.block + i * 32 + lane, y[i], inv);
    }
  }
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
struct NormBwdParams {
  long long N;
  int C, G, D;
  float eps;
  const void* gy;        // [N, C]
  const void* s;         // [N, C] (row stride s_st)
  long long s_st;
  const float* weight;
  const void* gs;        // [N, C] in s's type, or NULL
  void* ds;              // [N, C] in s's type
  float* part;           // [nparts, C] sums of gy s r over each part's rows
  float* rstd;           // [N, G], wkv_norm_bwd_row only
  int nparts;
};

// Rows are dealt to CTAs (row = CTA, CTA + grid, ...). A CTA holds whole rows:
// RPC rows at a time, each by its teams of TW lanes (one team per group) or by
// all threads (TW = 0, one group), K vectors of 8 columns per thread. A thread
// keeps the same columns from row to row and adds up its part of dweight in
// registers; the RPC rows' parts are joined through shared memory at the end,
// in a fixed order.
template <typename Y, typename S, bool GS, int TW, int K>
__global__ void __launch_bounds__(TW ? 512 : 1024) wkv_norm_bwd_team(const NormBwdParams p, int rpc) {
  extern __shared__ float acc[];  // [C], TW > 0 with rpc > 1
  __shared__ float red[64];
  const int tpr = TW ? TW * p.G : (int)blockDim.x;  // threads per row
  const int rl = TW ? (int)threadIdx.x / tpr : 0;   // row within the CTA's rpc rows
  const int tl = (int)threadIdx.x - rl * tpr;
  const int g = TW ? tl / TW : 0;
  const int l = TW ? tl % (TW ? TW : 1) : tl;
  const int width = TW ? TW : tpr;
  const bool lane_on = rl < rpc;
  const long long step = (long long)gridDim.x * rpc;
  float dw[K][kNV], w[K][kNV];
  bool in[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int col = (k * width + l) * kNV;
    in[k] = lane_on && col < p.D;
#pragma unroll
    for (int e = 0; e < kNV; ++e) dw[k][e] = 0.f, w[k][e] = 0.f;
    if (in[k]) {
      Vec8<float> wv;
      wv.load(p.weight + (long long)g * p.D + col);
      wv.get(w[k]);
    }
  }
  for (long long row0 = (long long)blockIdx.x * rpc; row0 < p.N; row0 += step) {
    const long long row = row0 + rl;
    const bool live = lane_on && row < p.N;
    Vec8<Y> yv[K];
    Vec8<S> sv[K], gv[K];
    const long long o = row * p.C + (long long)g * p.D;
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (live && in[k]) {
        const int col = (k * width + l) * kNV;
        yv[k].load(static_cast<const Y*>(p.gy) + o + col);
        sv[k].load(static_cast<const S*>(p.s) + row * p.s_st + (long long)g * p.D + col);
        if (GS) gv[k].load(static_cast<const S*>(p.gs) + o + col);
      }
    float s[K][kNV], gy[K][kNV];
    float ss = 0.f, ps = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (live && in[k]) {
        yv[k].get(gy[k]);
        sv[k].get(s[k]);
      } else {
#pragma unroll
        for (int e = 0; e < kNV; ++e) s[k][e] = gy[k][e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < kNV; ++e) {
        ss = fmaf(s[k][e], s[k][e], ss);
        ps = fmaf(gy[k][e] * w[k][e], s[k][e], ps);
      }
    }
    if (TW) {
      ss = team_sum<TW ? TW : 32>(ss);
      ps = team_sum<TW ? TW : 32>(ps);
    } else {  // both sums in one exchange
      const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5, nw = blockDim.x >> 5;
      ss = team_sum<32>(ss);
      ps = team_sum<32>(ps);
      __syncthreads();
      if (lane == 0) red[wp] = ss, red[32 + wp] = ps;
      __syncthreads();
      ss = team_sum<32>(lane < nw ? red[lane] : 0.f);
      ps = team_sum<32>(lane < nw ? red[32 + lane] : 0.f);
    }
    const float r = 1.f / sqrtf(ss / (float)p.D + p.eps);
    const float m = ps / (float)p.D * r * r;
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (live && in[k]) {
        float d[kNV];
        if (GS) gv[k].get(d);
#pragma unroll
        for (int e = 0; e < kNV; ++e) {
          d[e] = (GS ? d[e] : 0.f) + r * (gy[k][e] * w[k][e] - s[k][e] * m);
          dw[k][e] = fmaf(gy[k][e], s[k][e] * r, dw[k][e]);
        }
        Vec8<S>::store(static_cast<S*>(p.ds) + o + (k * width + l) * kNV, d);
      }
  }
  for (int turn = 0; turn < rpc; ++turn) {  // rows' parts join in order
    if (turn == rl && lane_on) {
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (in[k]) {
          const int col = g * p.D + (k * width + l) * kNV;
          if (turn > 0) {
#pragma unroll
            for (int e = 0; e < kNV; ++e) dw[k][e] += acc[col + e];
          }
          if (turn == rpc - 1) {
            Vec8<float>::store(p.part + (long long)blockIdx.x * p.C + col, dw[k]);
          } else {
#pragma unroll
            for (int e = 0; e < kNV; ++e) acc[col + e] = dw[k][e];
          }
        }
    }
    if (rpc > 1) __syncthreads();
  }
}

// Any size and alignment: ds of one row per CTA, and r of its groups.
__global__ void __launch_bounds__(256) wkv_norm_bwd_row(const NormBwdParams p, bool y_bf, bool s_bf) {
  __shared__ float red[32];
  const long long row = blockIdx.x;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const long long o = row * p.C, so = row * p.s_st;
  const int step = p.G == 1 ? (int)blockDim.x : 32;
  const int at = p.G == 1 ? (int)threadIdx.x : lane;
  for (int g = p.G == 1 ? 0 : w; g < p.G; g += p.G == 1 ? 1 : nw) {
    float ss = 0.f, ps = 0.f;
    for (int i = at; i < p.D; i += step) {
      const int c = g * p.D + i;
      const float s = load_any(p.s, s_bf, so + c);
      ss = fmaf(s, s, ss);
      ps = fmaf(load_any(p.gy, y_bf, o + c) * __ldg(p.weight + c), s, ps);
    }
    if (p.G == 1) {
      ss = cta_reduce<false>(ss, red);
      ps = cta_reduce<false>(ps, red);
    } else {
      ss = team_sum<32>(ss);
      ps = team_sum<32>(ps);
    }
    const float r = 1.f / sqrtf(ss / (float)p.D + p.eps);
    const float m = ps / (float)p.D * r * r;
    if (at == 0) p.rstd[row * p.G + g] = r;
    for (int i = at; i < p.D; i += step) {
      const int c = g * p.D + i;
      const float s = load_any(p.s, s_bf, so + c);
      const float d = (p.gs ? load_any(p.gs, s_bf, o + c) : 0.f) +
                      r * (load_any(p.gy, y_bf, o + c) * __ldg(p.weight + c) - s * m);
      if (s_bf) static_cast<__nv_bfloat16*>(p.ds)[o + c] = __float2bfloat16_rn(d);
      else static_cast<float*>(p.ds)[o + c] = d;
    }
  }
}

// dweight's parts for the same: columns by threads, rows blockIdx.y, + nparts, ...
__global__ void __launch_bounds__(256) wkv_norm_bwd_cols(const NormBwdParams p, bool y_bf, bool s_bf) {
  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= p.C) return;
  float dw = 0.f;
  for (long long row = blockIdx.y; row < p.N; row += p.nparts)
    dw = fmaf(load_any(p.gy, y_bf, row * p.C + c), load_any(p.s, s_bf, row * p.s_st + c) * p.rstd[row * p.G + c / p.D], dw);
  p.part[(long long)blockIdx.y * p.C + c] = dw;
}

// dweight = the parts' sum, in a fixed order: 8 warps add every eighth part of
// 32 columns, then join.
__global__ void __launch_bounds__(256) wkv_norm_bwd_join(const float* part, int nparts, int C, float* dw) {
  __shared__ float sm[8][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float a = 0.f;
  if (c < C)
    for (int i = w; i < nparts; i += 8) a += part[(long long)i * C + c];
  sm[w][lane] = a;
  __syncthreads();
  if (w == 0 && c < C) {
#pragma unroll
    for (int i = 1; i < 8; ++i) a += sm[i][lane];
    dw[c] = a;
  }
}

}  // namespace wkv
