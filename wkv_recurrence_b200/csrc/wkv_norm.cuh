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
// Bound: memory traffic; the kernels read their inputs once into registers
// (wkv_norm_row and wkv_norm_bwd_row apart, see there) and reduce while they
// stay there.
#pragma once

#include <cuda_fp8.h>

#include "wkv_device.cuh"
#include "wkv_pair.cuh"

namespace wkv {

constexpr float kE4m3Max = 448.f;
constexpr int kNV = 8;  // columns per vector: 16 bytes of bf16, 32 of fp32

// Eight columns of a thread as they lie in memory: adjacent (SC false: one or
// two 16-byte accesses), or `st` apart (SC true: element by element, adjacent
// lanes on adjacent columns, for rows that are not 16-byte aligned), the first
// `n` of them real.
template <typename T, bool SC>
struct Raw8;
template <>
struct Raw8<float, false> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p, int, int) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
    a = make_float4(x[0], x[1], x[2], x[3]);
    b = make_float4(x[4], x[5], x[6], x[7]);
  }
  __device__ __forceinline__ void put(float* p, int, int) const {
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
  }
};
template <>
struct Raw8<__nv_bfloat16, false> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p, int, int) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    unpack_bf16x2(a.x, x[0], x[1]);
    unpack_bf16x2(a.y, x[2], x[3]);
    unpack_bf16x2(a.z, x[4], x[5]);
    unpack_bf16x2(a.w, x[6], x[7]);
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {  // rounded to nearest even
    __nv_bfloat162 t;
    t = __floats2bfloat162_rn(x[0], x[1]), a.x = *reinterpret_cast<uint32_t*>(&t);
    t = __floats2bfloat162_rn(x[2], x[3]), a.y = *reinterpret_cast<uint32_t*>(&t);
    t = __floats2bfloat162_rn(x[4], x[5]), a.z = *reinterpret_cast<uint32_t*>(&t);
    t = __floats2bfloat162_rn(x[6], x[7]), a.w = *reinterpret_cast<uint32_t*>(&t);
  }
  __device__ __forceinline__ void put(__nv_bfloat16* p, int, int) const { *reinterpret_cast<uint4*>(p) = a; }
};
template <typename T>
struct Raw8<T, true> {
  T a[8];
  __device__ __forceinline__ void load(const T* p, int st, int n) {
#pragma unroll
    for (int e = 0; e < 8; ++e) a[e] = e < n ? p[e * st] : Elem<T>::from_f32(0.f);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = Elem<T>::to_f32(a[e]);
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) a[e] = Elem<T>::from_f32(x[e]);
  }
  __device__ __forceinline__ void put(T* p, int st, int n) const {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) p[e * st] = a[e];
  }
};

// x as T, rounded, to memory.
template <typename T, bool SC>
__device__ __forceinline__ void store8(T* p, int st, int n, const float (&x)[8]) {
  Raw8<T, SC> r;
  r.set(x);
  r.put(p, st, n);
}

// sum + the squares, in two partial sums; products by one number and by eight.
__device__ __forceinline__ float2 squares8(const float (&x)[8], float2 sum) {
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    const float2 v = make_float2(x[e], x[e + 1]);
    sum = fma2(v, v, sum);
  }
  return sum;
}
__device__ __forceinline__ void scale8(float (&x)[8], float f) {
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    const float2 v = mul2(make_float2(x[e], x[e + 1]), splat(f));
    x[e] = v.x, x[e + 1] = v.y;
  }
}
__device__ __forceinline__ void scale8(float (&x)[8], const float (&w)[8]) {
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    const float2 v = mul2(make_float2(x[e], x[e + 1]), make_float2(w[e], w[e + 1]));
    x[e] = v.x, x[e + 1] = v.y;
  }
}

// The columns of vector k of team lane l, `width` lanes in the team.
template <bool SC>
struct Cols {
  int at, st, n;  // first column, distance, how many of the eight exist
  __device__ __forceinline__ Cols(int k, int l, int width, int D) {
    at = SC ? k * kNV * width + l : (k * width + l) * kNV;
    st = SC ? width : 1;
    n = SC ? min(kNV, (D - at + width - 1) / width) : (at < D ? kNV : 0);
  }
};

// v^-1/2: the approximation and one Newton step (not for a sum that
// overflowed: 0 there)
__device__ __forceinline__ float inv_root(float v) {
  const float r = rsqrtf(v);
  return v <= 3.4028235e38f ? fmaf(0.5f * r, fmaf(-v * r, r, 1.f), r) : r;
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

template <bool SC>
__device__ __forceinline__ void store_e4m3(unsigned char* p, int st, int n, const float (&x)[8]) {
  if constexpr (SC) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) p[e * st] = (unsigned char)__nv_cvt_float_to_fp8(x[e], __NV_SATFINITE, __NV_E4M3);
  } else {
    *reinterpret_cast<uint2*>(p) = make_uint2(e4m3x4(x[0], x[1], x[2], x[3]), e4m3x4(x[4], x[5], x[6], x[7]));
  }
}

// The scale of a block whose largest |y| is `top`: 1 for a block of zeros, and
// never below the smallest normal number, so its inverse is finite.
__device__ __forceinline__ float e4m3_scale(float top) {
  return top > 0.f ? fmaxf(top * (1.f / kE4m3Max), 1.17549435e-38f) : 1.f;
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
  int nb;               // C / block
  float inv_d;          // 1 / D
};

template <int W>
__device__ __forceinline__ float team_sum(float v) {
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float lanes_max(float v, int width) {  // over `width` (a power of two from 4) adjacent lanes
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
  if (width > 4) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
  if (width > 8) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
  if (width > 16) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
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
// one group's D columns in registers, K vectors of 8 per thread. Vectors of 16
// bytes take aligned rows with D a multiple of 8; SC takes the others. e4m3
// scales here have their block inside a group: the whole group, or 32, 64 or
// 128 columns held by adjacent lanes in one k.
//
// What a row costs beside its bytes is paid per thread (index, root, scale), so
// wide rows have two vectors a thread and no divisions. Measured (of the 6521
// GB/s copy rate): 65536 x 4096 bf16 with residual 311 us (1.06), in e4m3 by
// 128 columns 274 us (1.05; 461 with one vector and IEEE divisions), e4m3
// without a residual 166 us (0.74: issue, at 3 bytes a column); 65536 x 12 x 64
// fp32 60 us (1.02); rows off 16 bytes: 40000 x 515 bf16 38 us (0.67: 2-byte
// accesses; 49 with a CTA per row), 65536 x 57 bf16 11 us (0.42; 68).
template <typename X, typename R, bool RES, int TW, int K, bool SC>
__global__ void __launch_bounds__(TW ? 256 : 512) wkv_norm_team(const NormParams p) {
  follow_on();
  __shared__ float red[32];
  const int width = TW ? TW : (int)blockDim.x;
  const int tl = TW ? (int)(threadIdx.x % width) : (int)threadIdx.x;
  const uint32_t seg = TW ? blockIdx.x * (256 / width) + threadIdx.x / width : blockIdx.x;
  const bool live = seg < (uint32_t)(p.N * p.G);
  const uint32_t row = !live ? 0 : p.G == 1 ? seg : seg / (uint32_t)p.G;
  const int gc = live ? (int)(seg - row * (uint32_t)p.G) * p.D : 0;  // the group's first column
  const X* xp = static_cast<const X*>(p.x) + row * p.x_st + gc;
  const R* rp = RES ? static_cast<const R*>(p.res) + row * p.res_st + gc : nullptr;
  Raw8<X, SC> xv[K];
  Raw8<R, SC> rv[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const Cols<SC> c(k, tl, width, p.D);
    if (live && c.n > 0) {
      xv[k].load(xp + c.at, c.st, c.n);
      if (RES) rv[k].load(rp + c.at, c.st, c.n);
    }
  }
  float s[K][kNV];
  float2 sums = splat(0.f);
  const long long o = (long long)row * p.C + gc;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const Cols<SC> c(k, tl, width, p.D);
    if (live && c.n > 0) {
      xv[k].get(s[k]);
      if (RES) {
        float r[kNV];
        rv[k].get(r);
#pragma unroll
        for (int e = 0; e < kNV; ++e) s[k][e] += r[e];
        rv[k].set(s[k]);  // the stream's rounding
        rv[k].put(static_cast<R*>(p.s) + o + c.at, c.st, c.n);
        rv[k].get(s[k]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < kNV; ++e) s[k][e] = 0.f;
    }
    sums = squares8(s[k], sums);
  }
  float sum = sums.x + sums.y;
  sum = TW ? team_sum<TW ? TW : 32>(sum) : cta_reduce<false>(sum, red);
  const float r = inv_root(fmaf(sum, p.inv_d, p.eps));
  const float* wp = p.weight + gc;
  const bool f8 = p.out_kind == kOutE4m3;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const Cols<SC> c(k, tl, width, p.D);
    if (live && c.n > 0) {
      Raw8<float, SC> wv;
      float w[kNV];
      wv.load(wp + c.at, c.st, c.n);
      wv.get(w);
      if (!f8) scale8(s[k], r);  // in e4m3 r joins the scale: one product less per column
      scale8(s[k], w);
      if (p.out_kind == kOutF32) store8<float, SC>(static_cast<float*>(p.y) + o + c.at, c.st, c.n, s[k]);
      if (p.out_kind == kOutBf16)
        store8<__nv_bfloat16, SC>(static_cast<__nv_bfloat16*>(p.y) + o + c.at, c.st, c.n, s[k]);
    }
  }
  if (!f8) return;
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
  const int per = p.block >> 3;  // threads that share a scale, where it is not the whole group
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const Cols<SC> c(k, tl, width, p.D);
    const float sc = e4m3_scale((whole ? all : lanes_max(top[k], per)) * r), inv = rcp(sc);
    if (live && c.n > 0) {
      if (sc < 1e-30f) {  // r / sc might overflow
        scale8(s[k], r);
        scale8(s[k], inv);
      } else {
        scale8(s[k], r * inv);
      }
      store_e4m3<SC>(static_cast<unsigned char*>(p.y) + o + c.at, c.st, c.n, s[k]);
      if (whole ? k == 0 && tl == 0 : (tl & (per - 1)) == 0)
        p.scale[(long long)row * p.nb + (whole ? (uint32_t)gc / (uint32_t)p.block : (uint32_t)(gc + c.at) / (uint32_t)p.block)] = sc;
    }
  }
}

// e4m3 whose scale blocks reach across groups (a row of several heads, blocks
// that straddle them): a CTA takes RPC rows, each by its groups' teams of TW
// lanes (one vector per thread), and the blocks' maxima meet in shared memory
// (the order of maxima does not matter).
template <typename X, typename R, bool RES, int TW>
__global__ void __launch_bounds__(1024) wkv_norm_cross(const NormParams p, int rpc) {
  follow_on();
  extern __shared__ int tops[];  // [rpc][nb]
  const int tpr = TW * p.G;
  const int rl = (int)threadIdx.x / tpr, tl = (int)threadIdx.x - rl * tpr;
  const int gc = tl / TW * p.D, c = (tl % TW) * kNV;
  const long long row = (long long)blockIdx.x * rpc + rl;
  const bool live = rl < rpc && row < p.N && c < p.D;
  for (int i = threadIdx.x; i < rpc * p.nb; i += blockDim.x) tops[i] = 0;
  float s[kNV];
  float sum = 0.f;
  const long long o = row * p.C + gc + c;
#pragma unroll
  for (int e = 0; e < kNV; ++e) s[e] = 0.f;
  if (live) {
    Raw8<X, false> xv;
    Raw8<R, false> rv;
    xv.load(static_cast<const X*>(p.x) + row * p.x_st + gc + c, 1, kNV);
    if (RES) rv.load(static_cast<const R*>(p.res) + row * p.res_st + gc + c, 1, kNV);
    xv.get(s);
    if (RES) {
      float r[kNV];
      rv.get(r);
#pragma unroll
      for (int e = 0; e < kNV; ++e) s[e] += r[e];
      rv.set(s);
      rv.put(static_cast<R*>(p.s) + o, 1, kNV);
      rv.get(s);
    }
    const float2 sums = squares8(s, splat(0.f));
    sum = sums.x + sums.y;
  }
  __syncthreads();  // tops is clear
  sum = team_sum<TW>(sum);
  const float r = inv_root(fmaf(sum, p.inv_d, p.eps));
  int* top = tops + rl * p.nb + (uint32_t)(gc + c) / (uint32_t)p.block;
  if (live) {
    Raw8<float, false> wv;
    float w[kNV], m = 0.f;
    wv.load(p.weight + gc + c, 1, kNV);
    wv.get(w);
    scale8(s, r);
    scale8(s, w);
#pragma unroll
    for (int e = 0; e < kNV; ++e) m = fmaxf(m, fabsf(s[e]));
    atomicMax(top, __float_as_int(m));  // bits of floats >= 0 are ordered as they are
  }
  __syncthreads();
  if (live) {
    const float sc = e4m3_scale(__int_as_float(*top)), f = rcp(sc);
    scale8(s, f);
    store_e4m3<false>(static_cast<unsigned char*>(p.y) + o, 1, kNV, s);
    if ((uint32_t)(gc + c) % (uint32_t)p.block == 0) p.scale[row * p.nb + (uint32_t)(gc + c) / (uint32_t)p.block] = sc;
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
    if (threadIdx.x == 0) rstd[0] = inv_root(fmaf(sum, p.inv_d, p.eps));
  } else {
    for (int g = w; g < p.G; g += nw) {  // a warp per group
      float sum = 0.f;
      for (int c = lane; c < p.D; c += 32) {
        const float s = first(g * p.D + c);
        sum = fmaf(s, s, sum);
      }
      sum = team_sum<32>(sum);
      if (lane == 0) rstd[g] = inv_root(fmaf(sum, p.inv_d, p.eps));
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
    const float sc = e4m3_scale(cta_reduce<true>(top, red)), inv = rcp(sc);
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
      const float sc = e4m3_scale(lanes_max(top, 32)), inv = rcp(sc);
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
  float inv_d;           // 1 / D
};

// Rows are dealt to CTAs (row = CTA, CTA + grid, ...). A CTA holds whole rows:
// RPC rows at a time, each by its teams of TW lanes (one team per group) or by
// all threads (TW = 0, one group), K vectors of 8 columns per thread; SC as in
// the forward. A thread keeps the same columns from row to row and adds up its
// part of dweight in registers; the RPC rows' parts are joined through shared
// memory at the end, pairwise. The next row is loaded while this one
// is reduced (K <= 2: registers).
//
// Measured: 65536 x 2048 bf16 with gs 180 us (0.91), fp32 310 us (1.06), 8191 x
// 12 x 64 fp32 15.4 us of inputs out of L2 (0.75: one wave of nine turns a CTA,
// and the parts' sum behind it).
template <typename Y, typename S, bool GS, int TW, int K, bool SC>
__global__ void __launch_bounds__(512) wkv_norm_bwd_team(const NormBwdParams p, int rpc, int half) {
  follow_on();
  extern __shared__ float acc[];  // [half][C], half the largest power of two below rpc (0: rpc = 1)
  __shared__ float2 red[2][16];
  constexpr bool kAhead = K <= 2;
  constexpr bool kKeepW = K == 1 || (K == 2 && sizeof(S) == 2);  // weights in registers, else from L1
  const int tpr = TW ? TW * p.G : (int)blockDim.x;  // threads per row
  const int rl = TW ? (int)threadIdx.x / tpr : 0;   // row within the CTA's rpc rows
  const int tl = (int)threadIdx.x - rl * tpr;
  const int gc = TW ? tl / TW * p.D : 0;            // the group's first column
  const int l = TW ? tl % (TW ? TW : 1) : tl;
  const int width = TW ? TW : tpr;
  const bool lane_on = rl < rpc;
  const long long step = (long long)gridDim.x * rpc;
  float dw[K][kNV], wk[kKeepW ? K : 1][kNV];
  auto weights = [&](int k, float (&w)[kNV]) {
    const Cols<SC> c(k, l, width, p.D);
#pragma unroll
    for (int e = 0; e < kNV; ++e) w[e] = 0.f;
    if (lane_on && c.n > 0) {
      Raw8<float, SC> wv;
      wv.load(p.weight + gc + c.at, c.st, c.n);
      wv.get(w);
    }
  };
#pragma unroll
  for (int k = 0; k < K; ++k) {
#pragma unroll
    for (int e = 0; e < kNV; ++e) dw[k][e] = 0.f;
    if (kKeepW) weights(k, wk[kKeepW ? k : 0]);
  }
  Raw8<Y, SC> yv[K];
  Raw8<S, SC> sv[K], gv[K];
  auto load_ys = [&](long long row) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const Cols<SC> c(k, l, width, p.D);
      if (lane_on && row < p.N && c.n > 0) {
        yv[k].load(static_cast<const Y*>(p.gy) + row * p.C + gc + c.at, c.st, c.n);
        sv[k].load(static_cast<const S*>(p.s) + row * p.s_st + gc + c.at, c.st, c.n);
      }
    }
  };
  auto load_g = [&](long long row) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const Cols<SC> c(k, l, width, p.D);
      if (GS && lane_on && row < p.N && c.n > 0)
        gv[k].load(static_cast<const S*>(p.gs) + row * p.C + gc + c.at, c.st, c.n);
    }
  };
  long long row0 = (long long)blockIdx.x * rpc;
  if (kAhead) load_ys(row0 + rl), load_g(row0 + rl);
  for (int par = 0; row0 < p.N; row0 += step, par ^= 1) {
    const long long row = row0 + rl;
    const bool live = lane_on && row < p.N;
    if (!kAhead) load_ys(row), load_g(row);
    float s[K][kNV], gy[K][kNV];
    float ss = 0.f, ps = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const Cols<SC> c(k, l, width, p.D);
      if (live && c.n > 0) {
        yv[k].get(gy[k]);
        sv[k].get(s[k]);
      } else {
#pragma unroll
        for (int e = 0; e < kNV; ++e) s[k][e] = gy[k][e] = 0.f;
      }
      float(&w)[kNV] = wk[kKeepW ? k : 0];
      if (!kKeepW) weights(k, w);
#pragma unroll
      for (int e = 0; e < kNV; ++e) {
        ss = fmaf(s[k][e], s[k][e], ss);
        ps = fmaf(gy[k][e] * w[e], s[k][e], ps);
      }
    }
    if (kAhead) load_ys(row + step);
    if (TW) {
      ss = team_sum<TW ? TW : 32>(ss);
      ps = team_sum<TW ? TW : 32>(ps);
    } else {  // both sums in one exchange; two buffers, one barrier per row
      const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5, nw = blockDim.x >> 5;
      ss = team_sum<32>(ss);
      ps = team_sum<32>(ps);
      if (lane == 0) red[par][wp] = make_float2(ss, ps);
      __syncthreads();
      const float2 v = lane < nw ? red[par][lane] : make_float2(0.f, 0.f);
      ss = team_sum<32>(v.x);
      ps = team_sum<32>(v.y);
    }
    const float r = inv_root(fmaf(ss, p.inv_d, p.eps));
    const float m = ps * p.inv_d * r * r;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const Cols<SC> c(k, l, width, p.D);
      if (live && c.n > 0) {
        float d[kNV];
        if (GS) gv[k].get(d);
        float(&w)[kNV] = wk[kKeepW ? k : 0];
        if (!kKeepW) weights(k, w);
#pragma unroll
        for (int e = 0; e < kNV; ++e) {
          const float t = gy[k][e] * w[e] - s[k][e] * m;
          d[e] = GS ? fmaf(r, t, d[e]) : r * t;
          dw[k][e] = fmaf(gy[k][e], s[k][e] * r, dw[k][e]);
        }
        store8<S, SC>(static_cast<S*>(p.ds) + row * p.C + gc + c.at, c.st, c.n, d);
      }
    }
    if (kAhead) load_g(row + step);
  }
  for (int h = half; h > 0; h >>= 1) {  // the rows' parts join pairwise, the upper half's onto the lower's
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const Cols<SC> c(k, l, width, p.D);
      if (lane_on && rl >= h && rl < 2 * h && c.n > 0) {
#pragma unroll
        for (int e = 0; e < kNV; ++e)
          if (!SC || e < c.n) acc[(rl - h) * p.C + gc + c.at + e * c.st] = dw[k][e];
      }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const Cols<SC> c(k, l, width, p.D);
      if (rl < h && rl + h < rpc && c.n > 0) {
#pragma unroll
        for (int e = 0; e < kNV; ++e)
          if (!SC || e < c.n) dw[k][e] += acc[rl * p.C + gc + c.at + e * c.st];
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const Cols<SC> c(k, l, width, p.D);
    if (lane_on && rl == 0 && c.n > 0)
      store8<float, SC>(p.part + (long long)blockIdx.x * p.C + gc + c.at, c.st, c.n, dw[k]);
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
    const float r = inv_root(fmaf(ss, p.inv_d, p.eps));
    const float m = ps * p.inv_d * r * r;
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

// dweight = the parts' sum, in a fixed order: of 32 columns, each of 32 warps
// adds every 32nd part, then a warp joins the 32 sums of a column.
__global__ void __launch_bounds__(1024) wkv_norm_bwd_join(const float* part, int nparts, int C, float* dw) {
  follow_on();
  __shared__ float sm[32][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float a = 0.f;
  if (c < C) {
#pragma unroll 8
    for (int i = w; i < nparts; i += 32) a += part[(long long)i * C + c];
  }
  sm[w][lane] = a;
  __syncthreads();
  // warp w joins column w's 32 sums, lane by lane
  a = team_sum<32>(sm[lane][w]);
  if (lane == 0 && blockIdx.x * 32 + w < C) dw[blockIdx.x * 32 + w] = a;
}

}  // namespace wkv
