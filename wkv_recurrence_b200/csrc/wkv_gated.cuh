// The gated linear recurrence: per channel, with a gate for every token,
//     h_t = f_t h_{t-1} + i_t x_t
//     sigmoid gate: f = sigmoid(z), i = 1 - f       decay gate: f = e^{-z}, i = 1
// and its backward, which runs the same recurrence from the end:
//     D_t = g_t + f_{t+1} D_{t+1}                    (D_t = dL/dh_t, all later tokens included)
//     dx_t = i_t D_t,   dz_t = D_t (h_{t-1} - x_t) f_t i_t   (decay: -D_t h_{t-1} f_t).
//
// One scan serves both directions. A span of tokens acts on the state as
// h -> P h + H (P the product of its f, H its own result from an empty state),
// and spans compose: (P2, H2) after (P1, H1) is (P2 P1, P2 H1 + H2).
//
//   CTA    a tile: 32 lanes x V channels by NW warps x J tokens. Every thread
//          loads its J tokens x V channels at once into registers (the loads
//          of a whole tile are in flight together), folds them into (P, H),
//          and the warps exchange theirs through shared memory.
//   chain  tiles of one channel group hand the state on through the
//          workspace. Tiles are numbered by a ticket with the position in the
//          sequence slowest, so a tile waits only for tiles that have already
//          started. Tiles form groups of G: a tile reads the state after the
//          group before its own (one record) and the totals of the tiles
//          before it in its group, so the sequence is walked in T/(L G) hops
//          and every sum has one fixed order.
//   replay with the state in front of its span, each warp runs its tokens
//          again from registers and stores. Inputs are read once, outputs
//          written once.
// A record is 16 bytes, {P, H, tag}, moved by one 128-bit access, so its tag
// (the launch's epoch) vouches for its data without a fence, and a reader
// polls the data itself.
//
// Bound: memory traffic (12 bytes per element fp32, 6 bf16; backward 20/10).
#pragma once

#include "wkv_device.cuh"

namespace wkv {

enum { kGateSigmoid = 0, kGateDecay = 1 };

// ---------------------------------------------------------------------------
// gate arithmetic
// ---------------------------------------------------------------------------
// A channel that remembers thousands of tokens has 1 - f ~ 1e-4, which f in
// fp32 holds to 2^-25 / 1e-4 = 3e-4 only, and the same error returns at every
// token. So a gate is carried as one number c whose sign says which of f and
// 1 - f it holds exactly to fp32:  c = -(1 - f) where 0 <= 1 - f < 1/2 (sign
// bit set, also for 1 - f = 0), else c = f. With base = 1 or 0 accordingly,
//     f h + b = base h + (c h + b),   f = base + c,   1 - f = (1 - base) - c,
// and a slow gate rounds the large h once a token, not twice.

// base: 1 where c holds f - 1, 0 where it holds f
__device__ __forceinline__ float gate_base(float c) { return __float_as_int(c) < 0 ? 1.f : 0.f; }

__device__ __forceinline__ float gate_pack(float m, float f) {  // m = 1 - f
  return (m >= 0.f && m < 0.5f) ? __int_as_float(__float_as_int(m) | (int)0x80000000) : f;
}

template <int GATE>
__device__ __forceinline__ float gate_coef(float z) {
  if constexpr (GATE == kGateSigmoid) {
    // e^z overflows to infinity for z > 88: m = 0, the state is held, and f
    // (then NaN) is not the number kept. z = -inf gives f = 0 exactly.
    const float e = ex2(z * kLog2e);
    const float m = rcp(1.f + e);
    return gate_pack(m, e * m);
  } else {
    const float f = ex2(-z * kLog2e);
    // 1 - e^{-z} by its series below 1/4, where the difference would cancel
    // (first term left out: z^7 / 7! < 2^-25 z)
    const float s = z * (1.f - z * (1.f / 2) * (1.f - z * (1.f / 3) * (1.f - z * (1.f / 4) * (1.f - z * (1.f / 5) * (1.f - z * (1.f / 6))))));
    return gate_pack(fabsf(z) < 0.25f ? s : 1.f - f, f);
  }
}

// f h + b
__device__ __forceinline__ float gate_step(float c, float base, float h, float b) {
  return fmaf(base, h, fmaf(c, h, b));
}
// f p
__device__ __forceinline__ float gate_mul(float c, float base, float p) { return fmaf(base, p, c * p); }
// what the token adds to the state, i_t x_t
template <int GATE>
__device__ __forceinline__ float gate_input(float c, float base, float x) {
  return GATE == kGateSigmoid ? ((1.f - base) - c) * x : x;
}

// ---------------------------------------------------------------------------
// V adjacent channels of one token, as they lie in memory
// ---------------------------------------------------------------------------
template <typename T, int V>
struct Pack;
template <>
struct Pack<float, 1> {
  float a;
  __device__ __forceinline__ void zero() { a = 0.f; }
  __device__ __forceinline__ void load(const float* p) { a = __ldg(p); }
  __device__ __forceinline__ void get(float (&x)[1]) const { x[0] = a; }
  __device__ __forceinline__ static void store(float* p, const float (&x)[1]) { *p = x[0]; }
};
template <>
struct Pack<float, 2> {
  float2 a;
  __device__ __forceinline__ void zero() { a = make_float2(0.f, 0.f); }
  __device__ __forceinline__ void load(const float* p) { a = __ldg(reinterpret_cast<const float2*>(p)); }
  __device__ __forceinline__ void get(float (&x)[2]) const { x[0] = a.x, x[1] = a.y; }
  __device__ __forceinline__ static void store(float* p, const float (&x)[2]) {
    *reinterpret_cast<float2*>(p) = make_float2(x[0], x[1]);
  }
};
template <>
struct Pack<__nv_bfloat16, 1> {
  unsigned short a;
  __device__ __forceinline__ void zero() { a = 0; }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = __ldg(reinterpret_cast<const unsigned short*>(p)); }
  __device__ __forceinline__ void get(float (&x)[1]) const { x[0] = __uint_as_float((uint32_t)a << 16); }
  __device__ __forceinline__ static void store(__nv_bfloat16* p, const float (&x)[1]) { *p = __float2bfloat16_rn(x[0]); }
};
template <>
struct Pack<__nv_bfloat16, 2> {
  uint32_t a;
  __device__ __forceinline__ void zero() { a = 0; }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = __ldg(reinterpret_cast<const uint32_t*>(p)); }
  __device__ __forceinline__ void get(float (&x)[2]) const { unpack_bf16x2(a, x[0], x[1]); }
  __device__ __forceinline__ static void store(__nv_bfloat16* p, const float (&x)[2]) {
    *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(x[0], x[1]);
  }
};

// ---------------------------------------------------------------------------
// the records of the chain
// ---------------------------------------------------------------------------
struct __align__(16) GatedRec {
  float P, H;
  uint64_t tag;
};

__device__ __forceinline__ void rec_store(GatedRec* r, float P, float H, uint64_t tag) {
  const uint64_t d = ((uint64_t)__float_as_uint(H) << 32) | __float_as_uint(P);
  asm volatile("{\n\t.reg .b128 t;\n\tmov.b128 t, {%1, %2};\n\tst.relaxed.gpu.global.b128 [%0], t;\n\t}" ::"l"(r),
               "l"(d), "l"(tag)
               : "memory");
}
__device__ __forceinline__ bool rec_load(const GatedRec* r, uint64_t tag, float& P, float& H) {
  uint64_t d, t;
  asm volatile("{\n\t.reg .b128 t;\n\tld.relaxed.gpu.global.b128 t, [%2];\n\tmov.b128 {%0, %1}, t;\n\t}"
               : "=l"(d), "=l"(t)
               : "l"(r)
               : "memory");
  P = __uint_as_float((uint32_t)d);
  H = __uint_as_float((uint32_t)(d >> 32));
  return t == tag;
}

constexpr uint64_t kGatedTag = 0x47415445ull << 32;  // tag = kGatedTag + the launch's number on this workspace

struct GatedParams {
  int B, T, C;
  int NG;      // channel groups of 32 V channels per batch row
  int nch;     // tiles per sequence
  int G;       // tiles per look-back group
  int ngrp;    // look-back groups per sequence
  const void* x;
  const void* z;
  long long x_sb, x_st, z_sb, z_st;  // element strides of the batch and token axes
  const float* h0;    // [B, C] state before the sequence, or NULL (zero)
  float* marks;       // [B, nch, C] the state in front of every tile: written by the forward (NULL: not), read by the
                      // backward
  // forward
  void* out;          // [B, T, C], or NULL (only the states are wanted)
  float* h_out;       // [B, C] or NULL
  // backward
  const void* g;      // [B, T, C]
  const float* dh_out;  // [B, C] gradient of the final state, or NULL (zero)
  void* dx;           // [B, T, C], type of x
  void* dz;           // [B, T, C], type of z
  float* dh0;         // [B, C] or NULL
  // chain
  WsHeader* hdr;
  GatedRec* tot;      // [items][nch][CG] totals of the tiles
  GatedRec* pre;      // [items][ngrp][CG] state after each look-back group
  uint64_t timeout_ns;
};

// Polls one record per channel until all V carry the tag, for at most the
// wait limit (then the status word says so and the values are whatever is
// there: finite work follows in any case).
template <int V>
__device__ __forceinline__ void rec_wait(const GatedRec* r, uint64_t tag, float (&P)[V], float (&H)[V],
                                         const GatedParams& p) {
  uint64_t t0 = 0;
  for (int spin = 0;; ++spin) {
    bool ok = true;
#pragma unroll
    for (int v = 0; v < V; ++v) ok &= rec_load(r + v, tag, P[v], H[v]);
    if (ok) return;
    if ((spin & 255) == 255) {
      const uint64_t now = global_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > p.timeout_ns) {
        atomicOr(&p.hdr->status, kStatusWaitTimeout);
        return;
      }
    }
  }
}

// The state in front of tile `pos` (counted along the scan's direction), for
// one channel group, by all warps of the CTA: the record after the previous
// look-back group (at pos = 0 `first`, the state before the sequence, which
// tile 0's total carries on to the others), then the totals of the tiles
// before `pos` in its own group. Shared memory: lb[NW][CG] and
// head[CG]. Ends with every thread holding its V channels' state in h.
template <int V>
__device__ __forceinline__ void gated_lookback(const GatedParams& p, int item, int pos, uint64_t tag,
                                               const float (&first)[V], float2* lb, float* head, float (&h)[V]) {
  constexpr int CG = 32 * V;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, NW = blockDim.x >> 5;
  const int grp = pos / p.G, n = pos - grp * p.G;  // n totals to read
  const int per = (n + NW - 1) / NW;
  if (w == 0) {
    float P[V], H[V];
    if (grp > 0) {
      rec_wait<V>(p.pre + ((size_t)item * p.ngrp + grp - 1) * CG + lane * V, tag, P, H, p);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) H[v] = first[v];
    }
#pragma unroll
    for (int v = 0; v < V; ++v) head[lane * V + v] = H[v];
  }
  if (w * per < n) {
    float Pa[V], Ha[V];
#pragma unroll
    for (int v = 0; v < V; ++v) Pa[v] = 1.f, Ha[v] = 0.f;
    for (int i = w * per; i < min(n, (w + 1) * per); ++i) {
      float P[V], H[V];
      rec_wait<V>(p.tot + ((size_t)item * p.nch + grp * p.G + i) * CG + lane * V, tag, P, H, p);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        Ha[v] = fmaf(P[v], Ha[v], H[v]);
        Pa[v] *= P[v];
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) lb[w * CG + lane * V + v] = make_float2(Pa[v], Ha[v]);
  }
  __syncthreads();
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = head[lane * V + v];
  for (int i = 0; i * per < n; ++i)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float2 a = lb[i * CG + lane * V + v];
      h[v] = fmaf(a.x, h[v], a.y);
    }
}

// Thread 0 counts the CTA out; the last one readies the header for the next
// launch on this workspace.
__device__ __forceinline__ void gated_leave(const GatedParams& p, uint32_t epoch) {
  if (threadIdx.x == 0) {
    const uint32_t prev = atomicAdd(&p.hdr->done, 1u);
    if (prev == gridDim.x - 1) {
      p.hdr->ticket = 0;
      p.hdr->done = 0;
      p.hdr->epoch = epoch + 1;
    }
  }
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
template <typename X, typename Z, typename O, int GATE, int V, int J, int NWMAX>
__global__ void __launch_bounds__(32 * NWMAX) gated_fwd(const GatedParams p) {
  constexpr int CG = 32 * V;
  __shared__ float2 s_agg[NWMAX * CG];
  __shared__ float2 s_lb[NWMAX * CG];
  __shared__ float s_head[CG];
  __shared__ uint32_t s_tick[2];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, NW = blockDim.x >> 5;
  const int L = NW * J;
  const int items = p.B * p.NG;
  uint32_t t = blockIdx.x, epoch = 0;
  if (p.nch > 1) {
    if (threadIdx.x == 0) {
      s_tick[0] = atomicAdd(&p.hdr->ticket, 1u);
      s_tick[1] = *reinterpret_cast<volatile uint32_t*>(&p.hdr->epoch);
    }
    __syncthreads();
    t = s_tick[0];
    epoch = s_tick[1];
  }
  const uint64_t tag = kGatedTag + epoch + 1u;
  const int pos = (int)(t / (uint32_t)items), item = (int)(t % (uint32_t)items);
  const int b = item / p.NG, c0 = (item % p.NG) * CG + lane * V;
  const bool on = c0 < p.C;  // C is a multiple of V
  const int t0 = pos * L + w * J;

  Pack<X, V> xr[J];
  Pack<Z, V> zr[J];
  const X* xp = static_cast<const X*>(p.x) + b * p.x_sb + t0 * p.x_st + c0;
  const Z* zp = static_cast<const Z*>(p.z) + b * p.z_sb + t0 * p.z_st + c0;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    if (on && t0 + j < p.T) {
      xr[j].load(xp + j * p.x_st);
      zr[j].load(zp + j * p.z_st);
    }
  }
  // The state before the sequence enters the scan at its first tile alone: its
  // total, which carries it on, depends on this load, so h_out may be h0. (In
  // a single tile the barrier below stands between this load and that store.)
  float first[V];
#pragma unroll
  for (int v = 0; v < V; ++v) first[v] = (p.h0 && on && pos == 0) ? p.h0[(size_t)b * p.C + c0 + v] : 0.f;

  // fold. A token past the end changes nothing: c = -0 (f = 1), b = 0.
  float c[J][V], in[J][V], P[V], H[V];
#pragma unroll
  for (int v = 0; v < V; ++v) P[v] = 1.f, H[v] = 0.f;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    float xf[V], zf[V];
    xr[j].get(xf);
    zr[j].get(zf);
    const bool tok = on && t0 + j < p.T;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      c[j][v] = tok ? gate_coef<GATE>(zf[v]) : -0.f;
      const float base = gate_base(c[j][v]);
      in[j][v] = tok ? gate_input<GATE>(c[j][v], base, xf[v]) : 0.f;
      H[v] = gate_step(c[j][v], base, H[v], in[j][v]);
      P[v] = gate_mul(c[j][v], base, P[v]);
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) s_agg[w * CG + lane * V + v] = make_float2(P[v], H[v]);
  __syncthreads();

  float h[V];
  if (p.nch > 1) {
    if (w == NW - 1 && pos % p.G != p.G - 1 && pos != p.nch - 1) {  // this tile's total, for the later tiles of its group
      float Pt[V], Ht[V];
#pragma unroll
      for (int v = 0; v < V; ++v) Pt[v] = pos == 0 ? 0.f : 1.f, Ht[v] = first[v];
      for (int i = 0; i < NW; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float2 a = s_agg[i * CG + lane * V + v];
          Ht[v] = fmaf(a.x, Ht[v], a.y);
          Pt[v] *= a.x;
        }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const size_t ri = ((size_t)item * p.nch + pos) * CG + lane * V + v;
        if (WKV_IN(p.hdr, ri, (size_t)items * p.nch * CG)) rec_store(p.tot + ri, Pt[v], Ht[v], tag);
      }
    }
    gated_lookback<V>(p, item, pos, tag, first, s_lb, s_head, h);
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = first[v];
  }
  if (p.marks && w == 0 && on) {
    const size_t mi = ((size_t)b * p.nch + pos) * p.C + c0;
    if (WKV_IN(p.hdr, mi + V - 1, (size_t)p.B * p.nch * p.C)) {
#pragma unroll
      for (int v = 0; v < V; ++v) p.marks[mi + v] = h[v];
    }
  }
  for (int i = 0; i < w; ++i)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float2 a = s_agg[i * CG + lane * V + v];
      h[v] = fmaf(a.x, h[v], a.y);
    }
  if (w == NW - 1 && pos % p.G == p.G - 1 && pos != p.nch - 1) {  // the state after this look-back group
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const size_t ri = ((size_t)item * p.ngrp + pos / p.G) * CG + lane * V + v;
      if (WKV_IN(p.hdr, ri, (size_t)items * p.ngrp * CG)) rec_store(p.pre + ri, 0.f, fmaf(P[v], h[v], H[v]), tag);
    }
  }
  // replay
  O* op = static_cast<O*>(p.out) + ((size_t)b * p.T + t0) * p.C + c0;
#pragma unroll
  for (int j = 0; j < J; ++j) {
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = gate_step(c[j][v], gate_base(c[j][v]), h[v], in[j][v]);
    if (p.out && on && t0 + j < p.T && WKV_IN(p.hdr, op + j * (size_t)p.C + V - 1 - static_cast<O*>(p.out),
                                             (size_t)p.B * p.T * p.C))
      Pack<O, V>::store(op + j * (size_t)p.C, h);
  }
  if (p.h_out && on && t0 < p.T && t0 + J >= p.T) {  // this span holds the last token
    const size_t si = (size_t)b * p.C + c0;
    if (WKV_IN(p.hdr, si + V - 1, (size_t)p.B * p.C)) {
#pragma unroll
      for (int v = 0; v < V; ++v) p.h_out[si + v] = h[v];
    }
  }
  if (p.nch > 1) gated_leave(p, epoch);
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
// Tiles are taken from the end of the sequence. The state in front of a tile
// comes from the forward's marks, so only the gradient travels along the
// chain, and the states inside the tile are computed again from x and z.
template <typename X, typename Z, typename O, int GATE, int V, int J, int NWMAX>
__global__ void __launch_bounds__(32 * NWMAX) gated_bwd(const GatedParams p) {
  constexpr int CG = 32 * V;
  __shared__ float2 s_fwd[NWMAX * CG];  // (P, H) of each warp's span
  __shared__ float s_rev[NWMAX * CG];   // its gradient from a zero gradient behind it (the P is the same)
  __shared__ float2 s_lb[NWMAX * CG];
  __shared__ float s_head[CG];
  __shared__ uint32_t s_tick[2];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, NW = blockDim.x >> 5;
  const int L = NW * J;
  const int items = p.B * p.NG;
  uint32_t t = blockIdx.x, epoch = 0;
  if (p.nch > 1) {
    if (threadIdx.x == 0) {
      s_tick[0] = atomicAdd(&p.hdr->ticket, 1u);
      s_tick[1] = *reinterpret_cast<volatile uint32_t*>(&p.hdr->epoch);
    }
    __syncthreads();
    t = s_tick[0];
    epoch = s_tick[1];
  }
  const uint64_t tag = kGatedTag + epoch + 1u;
  const int pos = (int)(t / (uint32_t)items), item = (int)(t % (uint32_t)items);  // pos counts from the end
  const int chunk = p.nch - 1 - pos;
  const int b = item / p.NG, c0 = (item % p.NG) * CG + lane * V;
  const bool on = c0 < p.C;
  const int t0 = chunk * L + w * J;

  Pack<X, V> xr[J];
  Pack<Z, V> zr[J];
  Pack<O, V> gr[J];
  const X* xp = static_cast<const X*>(p.x) + b * p.x_sb + t0 * p.x_st + c0;
  const Z* zp = static_cast<const Z*>(p.z) + b * p.z_sb + t0 * p.z_st + c0;
  const size_t o0 = ((size_t)b * p.T + t0) * p.C + c0;
  const O* gp = static_cast<const O*>(p.g) + o0;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    gr[j].zero();
    if (on && t0 + j < p.T) {
      xr[j].load(xp + j * p.x_st);
      zr[j].load(zp + j * p.z_st);
      gr[j].load(gp + j * (size_t)p.C);
    }
  }
  // gradient behind the sequence (read by the first tile of the scan alone, as
  // in the forward), state in front of the tile
  float first[V], h[V];
  const float* hp = p.nch > 1 ? p.marks + ((size_t)b * p.nch + chunk) * p.C : (p.h0 ? p.h0 + (size_t)b * p.C : nullptr);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    first[v] = (p.dh_out && on && pos == 0) ? p.dh_out[(size_t)b * p.C + c0 + v] : 0.f;
    h[v] = (hp && on) ? hp[c0 + v] : 0.f;
  }

  float c[J][V], e[J][V], P[V], H[V], Q[V];
#pragma unroll
  for (int v = 0; v < V; ++v) P[v] = 1.f, H[v] = 0.f, Q[v] = 0.f;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    float zf[V];
    xr[j].get(e[j]);
    zr[j].get(zf);
    const bool tok = on && t0 + j < p.T;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      c[j][v] = tok ? gate_coef<GATE>(zf[v]) : -0.f;
      e[j][v] = tok ? e[j][v] : 0.f;
      const float base = gate_base(c[j][v]);
      H[v] = gate_step(c[j][v], base, H[v], gate_input<GATE>(c[j][v], base, e[j][v]));
      P[v] = gate_mul(c[j][v], base, P[v]);
    }
  }
#pragma unroll
  for (int j = J - 1; j >= 0; --j) {
    float gf[V];
    gr[j].get(gf);
#pragma unroll
    for (int v = 0; v < V; ++v) Q[v] = gate_mul(c[j][v], gate_base(c[j][v]), gf[v] + Q[v]);
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    s_fwd[w * CG + lane * V + v] = make_float2(P[v], H[v]);
    s_rev[w * CG + lane * V + v] = Q[v];
  }
  __syncthreads();
  if (p.nch > 1 && w == 0 && pos % p.G != p.G - 1 && pos != p.nch - 1) {
    float Pt[V], Qt[V];
#pragma unroll
    for (int v = 0; v < V; ++v) Pt[v] = pos == 0 ? 0.f : 1.f, Qt[v] = first[v];
    for (int i = NW - 1; i >= 0; --i)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float pi = s_fwd[i * CG + lane * V + v].x;
        Qt[v] = fmaf(pi, Qt[v], s_rev[i * CG + lane * V + v]);
        Pt[v] *= pi;
      }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const size_t ri = ((size_t)item * p.nch + pos) * CG + lane * V + v;
      if (WKV_IN(p.hdr, ri, (size_t)items * p.nch * CG)) rec_store(p.tot + ri, Pt[v], Qt[v], tag);
    }
  }
  // the states of this span, and with them what D is multiplied by in dz
  for (int i = 0; i < w; ++i)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float2 a = s_fwd[i * CG + lane * V + v];
      h[v] = fmaf(a.x, h[v], a.y);
    }
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float base = gate_base(c[j][v]), f = base + c[j][v];
      const float hn = gate_step(c[j][v], base, h[v], gate_input<GATE>(c[j][v], base, e[j][v]));
      e[j][v] = GATE == kGateSigmoid ? (h[v] - e[j][v]) * f * ((1.f - base) - c[j][v]) : -h[v] * f;
      h[v] = hn;
    }
  float q[V];  // f_{t+1} D_{t+1}, what flows back into token t
  if (p.nch > 1) {
    gated_lookback<V>(p, item, pos, tag, first, s_lb, s_head, q);
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) q[v] = first[v];
  }
  for (int i = NW - 1; i > w; --i)
#pragma unroll
    for (int v = 0; v < V; ++v) q[v] = fmaf(s_fwd[i * CG + lane * V + v].x, q[v], s_rev[i * CG + lane * V + v]);
  if (w == 0 && pos % p.G == p.G - 1 && pos != p.nch - 1) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const size_t ri = ((size_t)item * p.ngrp + pos / p.G) * CG + lane * V + v;
      if (WKV_IN(p.hdr, ri, (size_t)items * p.ngrp * CG)) rec_store(p.pre + ri, 0.f, fmaf(P[v], q[v], Q[v]), tag);
    }
  }
  X* dxp = static_cast<X*>(p.dx) + o0;
  Z* dzp = static_cast<Z*>(p.dz) + o0;
#pragma unroll
  for (int j = J - 1; j >= 0; --j) {
    float gf[V], dxv[V], dzv[V];
    gr[j].get(gf);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float base = gate_base(c[j][v]), D = gf[v] + q[v];
      dxv[v] = gate_input<GATE>(c[j][v], base, D);
      dzv[v] = D * e[j][v];
      q[v] = gate_mul(c[j][v], base, D);
    }
    if (on && t0 + j < p.T && WKV_IN(p.hdr, o0 + j * (size_t)p.C + V - 1, (size_t)p.B * p.T * p.C)) {
      Pack<X, V>::store(dxp + j * (size_t)p.C, dxv);
      Pack<Z, V>::store(dzp + j * (size_t)p.C, dzv);
    }
  }
  if (p.dh0 && on && chunk == 0 && w == 0) {
    const size_t si = (size_t)b * p.C + c0;
    if (WKV_IN(p.hdr, si + V - 1, (size_t)p.B * p.C)) {
#pragma unroll
      for (int v = 0; v < V; ++v) p.dh0[si + v] = q[v];
    }
  }
  if (p.nch > 1) gated_leave(p, epoch);
}

// ---------------------------------------------------------------------------
// one token for S streams
// ---------------------------------------------------------------------------
struct GatedStepParams {
  long long n;   // vectors of V channels: S * C / V
  int CV;        // vectors per stream
  int C;
  const void* x;
  const void* z;
  long long x_ss, z_ss;  // element strides of the stream axis
  const float* h_in;
  float* h_out;  // may be h_in
  void* out;
};

// Elementwise and bound by memory (16 bytes per stream-channel in fp32, 14 in
// bf16); V channels per thread move as 16-byte accesses of the state.
template <typename X, typename Z, typename O, int GATE, int V>
__global__ void __launch_bounds__(256) gated_step_kernel(const GatedStepParams p) {
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= p.n) return;
  long long s;
  int cv;
  if (p.n < (1ll << 31)) {
    s = (uint32_t)i / (uint32_t)p.CV;
    cv = (int)((uint32_t)i % (uint32_t)p.CV);
  } else {
    s = i / p.CV;
    cv = (int)(i % p.CV);
  }
  float x[V], z[V], h[V];
  load_vec<X, V>(static_cast<const X*>(p.x) + s * p.x_ss + cv * V, x);
  load_vec<Z, V>(static_cast<const Z*>(p.z) + s * p.z_ss + cv * V, z);
  const long long o = s * p.C + (long long)cv * V;
  load_vec<float, V>(p.h_in + o, h);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const float c = gate_coef<GATE>(z[v]), base = gate_base(c);
    h[v] = gate_step(c, base, h[v], gate_input<GATE>(c, base, x[v]));
  }
  store_vec<float, V>(p.h_out + o, h);
  store_vec<O, V>(static_cast<O*>(p.out) + o, h);
}

}  // namespace wkv
