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
//   CTA    persistent; takes tiles of 64 channels (2 adjacent ones per lane)
//          by NW warps x J tokens. Each warp copies its own J x 64 inputs to
//          shared memory asynchronously, one tile ahead, folds them into
//          (P, H), and the warps exchange theirs through shared memory.
//   chain  tiles of one channel group hand the state on through the
//          workspace. Tiles are numbered by a ticket with the position in the
//          sequence slowest and every CTA works through its tickets in order,
//          so the tile with the smallest unfinished ticket never waits. Tiles
//          form groups of G: a tile reads the state after the group before
//          its own (one record) and the totals of the tiles before it in its
//          group, so the sequence is walked in T/(L G) hops and every sum has
//          one fixed order.
//   output with the state in front of its span, each warp has its tokens'
//          states from what the fold kept in registers (the backward runs its
//          tokens again). Inputs are read once, outputs written once.
// A record is 16 bytes, {P, H, tag}, moved by one 128-bit access, so its tag
// (the launch's number) vouches for its data without a fence, and a reader
// polls the data itself.
//
// Bound: memory traffic (12 bytes per element fp32, 6 bf16; backward 20/10) in
// fp32; in bf16, with half the bytes behind the same instructions (28 per
// element forward and 54 backward), latency: 16 warps per SM fill 55-60% of the
// issue slots and wait for copies, barriers and their own results. Pairs of
// channels are computed with the two-wide fp32 instructions, which took 14% off.
//
// Tile: 128 tokens by eight warps of 16, two CTAs per SM at 128 registers. What
// a warp spends on a tile besides its tokens (copies' addresses, joining spans,
// the chain) is about 250 instructions, so fewer, longer spans win as far as
// registers hold them: 16 warps of 8 tokens, as many CTAs, took 532 us for the
// 303 of 1 x 65536 x 2048 fp32 and 473 for the 340 of 16 x 4096 x 4096 bf16.
#pragma once

#include "wkv_device.cuh"
#include "wkv_pair.cuh"

namespace wkv {

enum { kGateSigmoid = 0, kGateDecay = 1 };

// ---------------------------------------------------------------------------
// gate arithmetic
// ---------------------------------------------------------------------------
// A channel that remembers thousands of tokens has 1 - f ~ 1e-4, which f in
// fp32 holds to 2^-25 / 1e-4 = 3e-4 only, and the same error returns at every
// token. So one number c is kept per gate, whose sign says which of 1 - f and f
// it holds to fp32's precision:
//     c = -(1 - f) < 0 near f = 1,  else c = f,
// and with A = 1 or 0 accordingly f = A + c, 1 - f = (1 - A) - c and
//     f h + b = A h + (c h + b),
// which rounds the large h of a slow gate once and holds a small f relative to
// itself (a state or gradient behind it may be large). A gate of f = 1 is kept
// as c = -2^-126, the smallest normal number, so that A is one saturated
// product and h stays what it is.
constexpr float kGateHeld = -1.17549435e-38f;
__device__ __forceinline__ float gate_base(float c) { return __saturatef(c * -3e38f); }
__device__ __forceinline__ float2 gate_base(float2 c) { return make_float2(gate_base(c.x), gate_base(c.y)); }

template <int GATE>
struct Gate;

template <>
struct Gate<kGateSigmoid> {
  // m = 1 - f = 1 / (1 + e^z), f = e^z m. z = -inf gives f = 0 and m = 1
  // exactly, z = +inf m = 0 (f is then NaN, and not the number kept). in =
  // i_t x.
  __device__ __forceinline__ static float2 coef(float2 z, float2 x, float2& in) {
    const float2 t = mul2(z, splat(kLog2e));
    const float2 e = make_float2(ex2(t.x), ex2(t.y));
    const float2 d = add2(e, splat(1.f));
    const float2 m = make_float2(rcp(d.x), rcp(d.y));
    const float2 f = mul2(e, m), n = fma2(m, splat(-1.f), splat(kGateHeld));
    in = mul2(m, x);
    return make_float2(m.x < 0.5f ? n.x : f.x, m.y < 0.5f ? n.y : f.y);
  }
  // i_t times x from c
  __device__ __forceinline__ static float2 input(float2 A, float2 c, float2 x) {
    return mul2(sub2(sub2(splat(1.f), A), c), x);
  }
  // dz_t / D_t, and i_t x
  __device__ __forceinline__ static float2 slope(float2 A, float2 c, float2 h, float2 x, float2& in) {
    const float2 m = sub2(sub2(splat(1.f), A), c);
    in = mul2(m, x);
    return mul2(mul2(sub2(h, x), add2(A, c)), m);
  }
};

template <>
struct Gate<kGateDecay> {
  // 1 - e^{-z} by its series for 0 <= z < 1/8 (first term left out z^6 / 720 <
  // 2^-24 z), where the difference would cancel.
  __device__ __forceinline__ static float2 coef(float2 z, float2 x, float2& in) {
    const float2 t = mul2(z, splat(-kLog2e));
    float2 n = fma2(z, splat(-1.f / 120), splat(1.f / 24));
    n = fma2(z, n, splat(-1.f / 6));
    n = fma2(z, n, splat(1.f / 2));
    n = fma2(z, n, splat(-1.f));
    n = fma2(z, n, splat(kGateHeld));
    in = x;
    return make_float2(z.x >= 0.f && z.x < 0.125f ? n.x : ex2(t.x), z.y >= 0.f && z.y < 0.125f ? n.y : ex2(t.y));
  }
  __device__ __forceinline__ static float2 input(float2, float2, float2 x) { return x; }
  __device__ __forceinline__ static float2 slope(float2 A, float2 c, float2 h, float2 x, float2& in) {
    in = x;
    return mul2(mul2(h, splat(-1.f)), add2(A, c));
  }
};

// Keeps the compiler from carrying what it derived from these numbers across
// this point (A of a whole span beside c would not fit in registers).
template <int J>
__device__ __forceinline__ void forget(float2 (&c)[J]) {
#pragma unroll
  for (int j = 0; j < J; ++j) asm volatile("" : "+f"(c[j].x), "+f"(c[j].y));
}

// f h + b and f h
__device__ __forceinline__ float2 gate_step(float2 A, float2 c, float2 h, float2 b) { return fma2(A, h, fma2(c, h, b)); }
__device__ __forceinline__ float2 gate_mul(float2 A, float2 c, float2 h) { return fma2(A, h, mul2(c, h)); }

// ---------------------------------------------------------------------------
// tiles in shared memory
// ---------------------------------------------------------------------------
constexpr int kGatedCG = 64;  // channels per tile: 32 lanes x 2

__device__ __forceinline__ float2 load2(const float* p) { return *reinterpret_cast<const float2*>(p); }
__device__ __forceinline__ float2 load2(const __nv_bfloat16* p) {
  float2 r;
  unpack_bf16x2(*reinterpret_cast<const uint32_t*>(p), r.x, r.y);
  return r;
}
// Two adjacent channels, as one access or, where the address does not take
// that, one by one, the second only if it exists.
__device__ __forceinline__ void store2(float* p, float2 v) { *reinterpret_cast<float2*>(p) = v; }
__device__ __forceinline__ void store2(__nv_bfloat16* p, float2 v) {
  *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(v.x, v.y);
}
template <typename T>
__device__ __forceinline__ void store_one(T* p, float2 v, bool second) {
  p[0] = Elem<T>::from_f32(v.x);
  if (second) p[1] = Elem<T>::from_f32(v.y);
}

template <int GR>
__device__ __forceinline__ void copy_async(void* dst, const void* src, bool real) {
  // bytes beyond the source size are filled with zeros
  const int n = real ? GR : 0;
  if constexpr (GR == 16) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(n) : "memory");
  } else {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(smem_u32(dst)), "l"(src), "n"(GR), "r"(n)
                 : "memory");
  }
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

template <typename T, int J, int GR>
__device__ __forceinline__ void copy_rows(T* dst, const T* src, const T* safe, long long st, int rows, int left) {
  constexpr int kPer = GR / (int)sizeof(T);  // elements per copy
  constexpr int kCols = kGatedCG / kPer;     // copies per row
  const int lane = threadIdx.x & 31;
  if constexpr (kCols <= 32) {  // 32 / kCols rows at a time, a lane stays in its column
    constexpr int kStep = 32 / kCols;
    const int row = lane / kCols, col = lane % kCols * kPer;
    const T* at = src + row * st + col;
    T* to = dst + row * kGatedCG + col;
    if (rows >= J && left >= kGatedCG) {
#pragma unroll
      for (int k = 0; k < J / kStep; ++k, at += kStep * st) copy_async<GR>(to + k * kStep * kGatedCG, at, true);
    } else {
#pragma unroll
      for (int k = 0; k < J / kStep; ++k, at += kStep * st) {
        const bool real = row + k * kStep < rows && col < left;
        copy_async<GR>(to + k * kStep * kGatedCG, real ? at : safe, real);
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < J * kCols / 32; ++k) {
      const int row = k * 32 / kCols, col = (k * 32 % kCols + lane) * kPer;
      const bool real = row < rows && col < left;
      copy_async<GR>(dst + row * kGatedCG + col, real ? src + row * st + col : safe, real);
    }
  }
}

// A warp's J rows of 64 channels into shared memory: `rows` rows and `left`
// channels exist from `src` on, the others are zeros (`safe`: an address for
// copies of nothing). gran: bytes that base, strides and row length are
// multiples of (16, 4, or 2: an element of bf16, copied through registers).
template <typename T, int J>
__device__ __forceinline__ void copy_span(T* dst, const T* src, const T* safe, long long st, int rows, int left, int gran) {
  if (gran == 16) {
    copy_rows<T, J, 16>(dst, src, safe, st, rows, left);
  } else if (gran == 4) {
    copy_rows<T, J, 4>(dst, src, safe, st, rows, left);
  } else if constexpr (sizeof(T) == 2) {
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int i = 0; i < 2 * J; i += 8) {  // eight loads in flight: what the callers' registers leave room for
      unsigned short v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int j = (i + k) >> 1, col = (k & 1) * 32 + lane;
        v[k] = j < rows && col < left ? reinterpret_cast<const unsigned short*>(src)[j * st + col] : (unsigned short)0;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k)
        reinterpret_cast<unsigned short*>(dst)[((i + k) >> 1) * kGatedCG + (k & 1) * 32 + lane] = v[k];
    }
  }
}

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

// t / d for t < 2^31 as floor(t m / 2^sh), sh = 31 + ceil(log2 d): m = ceil(2^sh
// / d) is less than 1 too large, so t m / 2^sh less than t / 2^sh < 1 / d, the
// least distance of t / d from the next whole number.
struct Divisor {
  uint32_t d, m;
  int sh;
  __device__ __forceinline__ uint32_t of(uint32_t t) const { return (uint32_t)(((uint64_t)t * m) >> sh); }
};

struct GatedParams {
  int B, T, C;
  int NG;      // channel groups of 64 per batch row
  int nch;     // tiles per sequence
  int G;       // tiles per look-back group
  int ngrp;    // look-back groups per sequence
  long long tiles;
  Divisor by_items, by_ng;  // B NG and NG
  const void* x;
  const void* z;
  long long x_sb, x_st, z_sb, z_st;  // element strides of the batch and token axes
  int x_gran, z_gran, g_gran;        // copy_span's gran
  int pair;           // whether outputs take two channels per store
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
  GatedRec* tot;      // [items][nch][64] totals of the tiles
  GatedRec* pre;      // [items][ngrp][64] state after each look-back group
  uint64_t timeout_ns;
};

// Two floats of a [B, C]-like row at channel c0 (zeros past C).
__device__ __forceinline__ float2 row_get(const float* p, long long o, int c0, int C) {
  return make_float2(c0 < C ? p[o + c0] : 0.f, c0 + 1 < C ? p[o + c0 + 1] : 0.f);
}
__device__ __forceinline__ void row_put(WsHeader* hdr, float* p, long long o, int c0, int C, size_t n, float2 v) {
  if (c0 < C && WKV_IN(hdr, o + c0, n)) p[o + c0] = v.x;
  if (c0 + 1 < C && WKV_IN(hdr, o + c0 + 1, n)) p[o + c0 + 1] = v.y;
}

// Polls a record pair until both carry the tag, for at most the wait limit
// (then the status word says so and the values are whatever is there: finite
// work follows in any case).
__device__ __forceinline__ void rec_wait(const GatedRec* r, uint64_t tag, float2& P, float2& H, const GatedParams& p) {
  uint64_t t0 = 0;
  for (int spin = 0;; ++spin) {
    bool ok = rec_load(r, tag, P.x, H.x);
    ok &= rec_load(r + 1, tag, P.y, H.y);
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
__device__ __forceinline__ void rec_put(const GatedParams& p, GatedRec* r, size_t i, size_t n, float2 P, float2 H,
                                        uint64_t tag) {
  if (!WKV_IN(p.hdr, i + 1, n)) return;
  rec_store(r + i, P.x, H.x, tag);
  rec_store(r + i + 1, P.y, H.y, tag);
}

// h -> P h + H of one span after another
struct Span {
  float2 P, H;
};
__device__ __forceinline__ float2 apply(const Span& s, float2 h) { return fma2(s.P, h, s.H); }
// Tiles joined: h -> 2^-32 P h + H. A product of several tiles' P may leave
// fp32's range at either end although each is in it, and so is the state it is
// applied to. It is kept 2^32 times too large, and as 0 below 2^-158, where it
// shrinks a state of less than 2^32 to nothing in fp32. Products that overflow,
// and larger states in front of such a 0 if later gates may be above 1 (GROWS),
// are found by `peak` and take the tiles one by one (1 x 65536 x 2048 fp32 decays
// with states of 1e12: 557 us forward for 311).
constexpr float kLift = 4294967296.f, kMaxF = 3.4028235e38f;
struct Joint {
  float2 P, H;
};
__device__ __forceinline__ float2 apply(const Joint& a, float2 h) {
  return fma2(mul2(a.P, h), splat(1.f / kLift), a.H);
}
__device__ __forceinline__ void join(Joint& a, const Span& s) {
  a.H = apply(s, a.H);
  a.P = mul2_ftz(a.P, s.P);
}
__device__ __forceinline__ void join(Joint& a, const Joint& s) {
  a.H = apply(s, a.H);
  a.P = mul2_ftz(mul2(a.P, s.P), splat(1.f / kLift));
}
// The larger of m and both magnitudes; NaN if one is.
__device__ __forceinline__ float peak(float m, float2 h) {
  asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(fabsf(h.x)), "f"(fabsf(h.y)));
  return m;
}

// The state in front of tile `pos` (counted along the scan's direction) comes
// from the record of the look-back group before it; at pos = 0 it is `first`,
// the state before the sequence, which tile 0's total carries on to the other
// tiles of its group.
//
// Groups of one tile (G = 1: many channel groups, the tile before is done):
// every warp asks for the record when it starts the tile and has it when the
// tile's own spans are folded.
struct Head {
  float2 H;
  bool got;
};
__device__ __forceinline__ const GatedRec* head_rec(const GatedParams& p, int item, int pos) {
  return p.pre + ((size_t)item * p.ngrp + pos / p.G - 1) * kGatedCG + (threadIdx.x & 31) * 2;
}
__device__ __forceinline__ Head head_ask(const GatedParams& p, int item, int pos, uint64_t tag) {
  Head r{splat(0.f), true};
  if (p.G == 1 && pos > 0) {
    float P;
    const GatedRec* rec = head_rec(p, item, pos);
    const bool a = rec_load(rec, tag, P, r.H.x), b = rec_load(rec + 1, tag, P, r.H.y);
    r.got = a && b;
  }
  return r;
}
__device__ __forceinline__ float2 head_get(const GatedParams& p, int item, int pos, uint64_t tag, float2 first, Head r) {
  if (pos == 0) return first;
  if (!r.got) {
    float2 P;
    rec_wait(head_rec(p, item, pos), tag, P, r.H, p);
  }
  return r.H;
}

// Groups of several tiles: the warps gather the totals of the tiles before
// `pos` in its group, which do not wait for the chain, and warp 0 the record.
// The tile that ends its group is a link of the chain: there warp 0 first joins
// all totals, its own tile's included, then waits for the record and hands the
// state on at once, before the other warps know it (1 x 65536 x 64, inputs in
// L2: 70 us without this, 20 with it).
template <int NWMAX>
struct Front {
  Joint part[NWMAX][32];
  float2 h[32];
};
// The state behind the first n tiles of a look-back group (`tot`: its first
// total) from the state in front of it, tile by tile. All have been waited for.
__device__ __forceinline__ float2 one_by_one(const GatedRec* tot, int n, uint64_t tag, float2 h) {
#pragma unroll 1
  for (int i = 0; i < n; ++i) {
    Span s;
    rec_load(tot + (size_t)i * kGatedCG, tag, s.P.x, s.H.x);
    rec_load(tot + (size_t)i * kGatedCG + 1, tag, s.P.y, s.H.y);
    h = apply(s, h);
  }
  return h;
}
template <bool GROWS, int NWMAX, typename Total>
__device__ __forceinline__ float2 gated_front(const GatedParams& p, int item, int pos, uint64_t tag, float2 first,
                                              Front<NWMAX>& fr, const Total& own) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, NW = blockDim.x >> 5;
  const int grp = pos / p.G, n = pos - grp * p.G;  // n totals to read
  const int per = (n + NW - 1) / NW;
  const bool group_end = n == p.G - 1, last = pos == p.nch - 1;
  if (w == NW - 1 && !group_end && !last) {  // this tile's total, for the later tiles of its group
    Span tot = own();
    if (pos == 0) tot.H = apply(tot, first), tot.P = splat(0.f);
    rec_put(p, p.tot, ((size_t)item * p.nch + pos) * kGatedCG + lane * 2, (size_t)p.B * p.NG * p.nch * kGatedCG, tot.P,
            tot.H, tag);
  }
  const GatedRec* tots = p.tot + ((size_t)item * p.nch + grp * p.G) * kGatedCG + lane * 2;
  if (w * per < n) {
    Joint a{splat(kLift), splat(0.f)};
    for (int i = w * per; i < min(n, (w + 1) * per); ++i) {
      Span s;
      rec_wait(tots + (size_t)i * kGatedCG, tag, s.P, s.H, p);
      join(a, s);
    }
    fr.part[w][lane] = a;
  }
  const bool hand_on = group_end && !last;
  if (w == 0 && !hand_on) {
    float2 P, H = first;
    if (grp > 0) rec_wait(head_rec(p, item, pos), tag, P, H, p);
    fr.h[lane] = H;
  }
  __syncthreads();
  if (hand_on) {
    if (w == 0) {
      Joint a{splat(kLift), splat(0.f)};
      float m = 0.f;
      for (int i = 0; i * per < n; ++i) {
        join(a, fr.part[i][lane]);
        m = peak(m, a.H);
      }
      const Span tot = own();
      join(a, tot);
      float2 P, H = first;
      if (grp > 0) rec_wait(head_rec(p, item, pos), tag, P, H, p);
      float2 after = apply(a, H);
      m = peak(peak(m, H), after);
      if (!(m < kLift) && !(m <= kMaxF && (!GROWS || (a.P.x > 0.f && a.P.y > 0.f))))
        after = apply(tot, one_by_one(tots, n, tag, H));
      rec_put(p, p.pre, ((size_t)item * p.ngrp + grp) * kGatedCG + lane * 2, (size_t)p.B * p.NG * p.ngrp * kGatedCG,
              splat(0.f), after, tag);
      fr.h[lane] = H;
    }
    __syncthreads();
  }
  float2 h = fr.h[lane];
  float m = peak(0.f, h);
  for (int i = 0; i * per < n; ++i) {
    h = apply(fr.part[i][lane], h);
    m = peak(m, h);
  }
  if (m < kLift) return h;
  bool whole = m <= kMaxF;
  for (int i = 0; GROWS && i * per < n; ++i) whole &= fr.part[i][lane].P.x > 0.f && fr.part[i][lane].P.y > 0.f;
  return whole ? h : one_by_one(tots, n, tag, fr.h[lane]);
}

// The tiles of a CTA. Several tiles per sequence: by tickets, so that every
// tile's predecessors have been taken before it. One: dealt out.
struct Tile {
  int pos, item, b, cg;  // position along the scan (-1: no more tiles), channel group, batch row, first channel
};
__device__ __forceinline__ Tile gated_tile(const GatedParams& p, long long t) {
  if (t >= p.tiles) return Tile{-1, 0, 0, 0};
  Tile r;
  r.pos = (int)p.by_items.of((uint32_t)t);
  r.item = (int)((uint32_t)t - (uint32_t)r.pos * p.by_items.d);
  r.b = (int)p.by_ng.of((uint32_t)r.item);
  r.cg = (r.item - r.b * p.NG) * kGatedCG;
  return r;
}
// The ticket after `last` (thread 0).
__device__ __forceinline__ long long gated_ticket(const GatedParams& p, long long last) {
  return p.nch > 1 ? (long long)atomicAdd(&p.hdr->ticket, 1u) : last + gridDim.x;
}

// Thread 0 counts the CTA out; the last one readies the header for the next
// launch on this workspace. (Every CTA has taken its last ticket by then.)
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

// Shared memory of a CTA beside its input tiles.
template <int NWMAX>
struct GatedShared {
  Span agg[2][NWMAX][32];   // the warps' spans, by parity of the tile
  float2 rev[2][NWMAX][32];  // backward: their gradients (the P is the same)
  Front<NWMAX> front;
  float2 first[2][32];      // by parity: the state (gradient) before the sequence, of a tile that starts it
  long long next[2];        // by parity: the ticket after this one
  uint32_t epoch;
};

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
// Measured (of the 6521 GB/s copy rate, for each input read and each output
// written once; inputs from DRAM): 1 x 65536 x 2048 fp32 310 us (0.80; 307
// with joined tiles' products unscaled), 16 x 4096 x 4096 with bf16 x and out
// and fp32 decays 344 us (0.96), all bf16 341 us (0.72), 8 x 1024 x 768 bf16
// 16.8 us (0.35: three rounds of tiles, about 5 us each; 14.3 us out of L2).
template <typename X, typename Z, int J, int NW>
constexpr size_t gated_fwd_smem() {
  return (size_t)J * NW * kGatedCG * (sizeof(X) + sizeof(Z));
}

template <typename X, typename Z, typename O, int GATE, int J, int NWMAX>
__global__ void __launch_bounds__(32 * NWMAX, 64 / (NWMAX * 4)) gated_fwd(const GatedParams p) {
  follow_on();
  using Gt = Gate<GATE>;
  extern __shared__ __align__(16) unsigned char tiles[];
  __shared__ GatedShared<NWMAX> sh;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, NW = blockDim.x >> 5;
  const int L = NW * J;
  const bool chained = p.nch > 1;
  X* sx = reinterpret_cast<X*>(tiles) + (size_t)w * J * kGatedCG;
  Z* sz = reinterpret_cast<Z*>(tiles + (size_t)NW * J * kGatedCG * sizeof(X)) + (size_t)w * J * kGatedCG;

  auto fetch = [&](const Tile& a) {  // this warp's inputs of a tile, on their way to shared memory
    if (a.pos >= 0) {
      const int t0 = a.pos * L + w * J;
      const int rows = min(J, p.T - t0), left = p.C - a.cg;
      copy_span<X, J>(sx, static_cast<const X*>(p.x) + a.b * p.x_sb + t0 * p.x_st + a.cg, static_cast<const X*>(p.x),
                      p.x_st, rows, left, p.x_gran);
      copy_span<Z, J>(sz, static_cast<const Z*>(p.z) + a.b * p.z_sb + t0 * p.z_st + a.cg, static_cast<const Z*>(p.z),
                      p.z_st, rows, left, p.z_gran);
    }
    copy_commit();
  };

  long long ticket = (long long)blockIdx.x - gridDim.x;  // thread 0's last one
  if (threadIdx.x == 0) {
    ticket = gated_ticket(p, ticket);
    sh.next[0] = ticket;
    sh.epoch = chained ? *reinterpret_cast<volatile uint32_t*>(&p.hdr->epoch) : 0;
  }
  __syncthreads();
  Tile a = gated_tile(p, sh.next[0]);
  const uint64_t tag = kGatedTag + sh.epoch + 1u;
  fetch(a);
  for (int par = 1; a.pos >= 0; par ^= 1) {
    const int t0 = a.pos * L + w * J;
    const int nt = p.T - t0;  // tokens from this span on
    const int c0 = a.cg + lane * 2;
    if (threadIdx.x == 0) ticket = gated_ticket(p, ticket);
    // The state before the sequence enters the scan at its first tile alone, by
    // one warp, and is in shared memory before the barrier: whatever the tile
    // hands on lies behind this load, so h_out may be h0.
    if (w == 0 && a.pos == 0) sh.first[par][lane] = p.h0 ? row_get(p.h0, (long long)a.b * p.C, c0, p.C) : splat(0.f);
    const Head ask = head_ask(p, a.item, a.pos, tag);

    copy_wait();
    __syncwarp();
    // fold, keeping for every token the span up to it: h_t = P_t h + H_t. A
    // token past the end (its x is 0) changes nothing: f = 1.
    Span s{splat(1.f), splat(0.f)};
    float2 P[J], H[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      P[j] = Gt::coef(load2(sz + j * kGatedCG + lane * 2), load2(sx + j * kGatedCG + lane * 2), H[j]);
      if (nt < J && j >= nt) P[j] = splat(kGateHeld);
      const float2 A = gate_base(P[j]);
      s.H = H[j] = gate_step(A, P[j], s.H, H[j]);
      s.P = P[j] = gate_mul(A, P[j], s.P);
    }
    sh.agg[par][w][lane] = s;
    if (threadIdx.x == 0) sh.next[par] = ticket;
    __syncthreads();
    const Tile an = gated_tile(p, sh.next[par]);
    fetch(an);  // every lane's reads of the tile lie before the barrier

    const float2 first = a.pos == 0 ? sh.first[par][lane] : splat(0.f);
    float2 h;  // the state in front of the tile
    if (chained && p.G > 1) {
      h = gated_front<GATE == kGateDecay>(p, a.item, a.pos, tag, first, sh.front, [&] {
        Span tot = sh.agg[par][0][lane];
        for (int i = 1; i < NW; ++i) {
          const Span u = sh.agg[par][i][lane];
          tot.H = apply(u, tot.H);
          tot.P = mul2(tot.P, u.P);
        }
        return tot;
      });
    } else {
      h = head_get(p, a.item, a.pos, tag, first, ask);
    }
    if (p.marks && w == 0)
      row_put(p.hdr, p.marks, ((long long)a.b * p.nch + a.pos) * p.C, c0, p.C, (size_t)p.B * p.nch * p.C, h);
    for (int i = 0; i < w; ++i) h = apply(sh.agg[par][i][lane], h);
    if (chained && p.G == 1 && w == NW - 1 && a.pos != p.nch - 1)  // the state after this tile
      rec_put(p, p.pre, ((size_t)a.item * p.ngrp + a.pos) * kGatedCG + lane * 2,
              (size_t)p.B * p.NG * p.ngrp * kGatedCG, splat(0.f), apply(s, h), tag);
    O* op = static_cast<O*>(p.out) + ((long long)a.b * p.T + t0) * p.C + c0;
    const bool store = p.out && c0 < p.C;
    if (nt >= J && p.pair) {
#pragma unroll
      for (int j = 0; j < J; ++j) {
        if (store && WKV_IN(p.hdr, op + 1 - static_cast<O*>(p.out), (size_t)p.B * p.T * p.C))
          store2(op, fma2(P[j], h, H[j]));
        op += p.C;
      }
    } else {
#pragma unroll
      for (int j = 0; j < J; ++j) {
        if (store && j < nt && WKV_IN(p.hdr, op - static_cast<O*>(p.out), (size_t)p.B * p.T * p.C))
          store_one(op, fma2(P[j], h, H[j]), c0 + 1 < p.C);
        op += p.C;
      }
    }
    h = apply(s, h);
    if (p.h_out && nt > 0 && nt <= J)  // this span holds the last token
      row_put(p.hdr, p.h_out, (long long)a.b * p.C, c0, p.C, (size_t)p.B * p.C, h);
    a = an;
  }
  if (chained) gated_leave(p, sh.epoch);
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
// Tiles are taken from the end of the sequence. The state in front of a tile
// comes from the forward's marks, so only the gradient travels along the
// chain, and the states inside the tile are computed again from x and z.
// x and z are fetched one tile ahead as soon as the states are done; g has two
// buffers where both fit beside another CTA (kGB), else it is fetched last.
//
// Measured: 1 x 65536 x 2048 fp32 488 us (0.84; 478 unscaled), 16 x 4096 x 4096
// bf16 with fp32 decays 627 us (0.92; 670-720 back to back under the power cap),
// all bf16 609 us (0.68), 8 x 1024 x 768 bf16 24.1 us (0.40; 22.1 out of L2).
template <typename X, typename Z, typename O, int J, int NW>
struct GatedBwdSmem {
  static constexpr size_t kRow = (size_t)J * NW * kGatedCG;
  static constexpr int kGB = kRow * (sizeof(X) + sizeof(Z) + 2 * sizeof(O)) <= 88 * 1024 ? 2 : 1;
  static constexpr size_t kBytes = kRow * (sizeof(X) + sizeof(Z) + kGB * sizeof(O));
};

template <typename X, typename Z, typename O, int GATE, int J, int NWMAX>
__global__ void __launch_bounds__(32 * NWMAX, 64 / (NWMAX * 4)) gated_bwd(const GatedParams p) {
  follow_on();
  using Gt = Gate<GATE>;
  constexpr int kGB = GatedBwdSmem<X, Z, O, J, NWMAX>::kGB;
  extern __shared__ __align__(16) unsigned char tiles[];
  __shared__ GatedShared<NWMAX> sh;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, NW = blockDim.x >> 5;
  const int L = NW * J;
  const bool chained = p.nch > 1;
  const size_t row = (size_t)NW * J * kGatedCG, mine = (size_t)w * J * kGatedCG;
  X* sx = reinterpret_cast<X*>(tiles) + mine;
  Z* sz = reinterpret_cast<Z*>(tiles + row * sizeof(X)) + mine;
  O* sg0 = reinterpret_cast<O*>(tiles + row * (sizeof(X) + sizeof(Z))) + mine;

  auto fetch_xz = [&](const Tile& a) {
    if (a.pos >= 0) {
      const int t0 = (p.nch - 1 - a.pos) * L + w * J;
      const int rows = min(J, p.T - t0), left = p.C - a.cg;
      copy_span<X, J>(sx, static_cast<const X*>(p.x) + a.b * p.x_sb + t0 * p.x_st + a.cg, static_cast<const X*>(p.x),
                      p.x_st, rows, left, p.x_gran);
      copy_span<Z, J>(sz, static_cast<const Z*>(p.z) + a.b * p.z_sb + t0 * p.z_st + a.cg, static_cast<const Z*>(p.z),
                      p.z_st, rows, left, p.z_gran);
    }
  };
  auto fetch_g = [&](const Tile& a, O* dst) {
    if (a.pos >= 0) {
      const int t0 = (p.nch - 1 - a.pos) * L + w * J;
      copy_span<O, J>(dst, static_cast<const O*>(p.g) + ((long long)a.b * p.T + t0) * p.C + a.cg,
                      static_cast<const O*>(p.g), p.C, min(J, p.T - t0), p.C - a.cg, p.g_gran);
    }
  };

  long long ticket = (long long)blockIdx.x - gridDim.x;  // thread 0's last one
  if (threadIdx.x == 0) {
    ticket = gated_ticket(p, ticket);
    sh.next[0] = ticket;
    sh.epoch = chained ? *reinterpret_cast<volatile uint32_t*>(&p.hdr->epoch) : 0;
  }
  __syncthreads();
  Tile a = gated_tile(p, sh.next[0]);
  const uint64_t tag = kGatedTag + sh.epoch + 1u;
  fetch_xz(a);
  fetch_g(a, sg0 + (kGB == 2 ? row : 0));
  copy_commit();
  for (int par = 1; a.pos >= 0; par ^= 1) {
    const int chunk = p.nch - 1 - a.pos;  // position in the sequence
    const int t0 = chunk * L + w * J;
    const int nt = p.T - t0;
    const int c0 = a.cg + lane * 2;
    O* sg = sg0 + (kGB == 2 && par ? row : 0);
    if (threadIdx.x == 0) ticket = gated_ticket(p, ticket);
    // gradient behind the sequence (as the state in the forward: dh0 may be
    // dh_out), state in front of the tile
    if (w == 0 && a.pos == 0)
      sh.first[par][lane] = p.dh_out ? row_get(p.dh_out, (long long)a.b * p.C, c0, p.C) : splat(0.f);
    float2 h = chained ? row_get(p.marks, ((long long)a.b * p.nch + chunk) * p.C, c0, p.C)
                       : (p.h0 ? row_get(p.h0, (long long)a.b * p.C, c0, p.C) : splat(0.f));
    const Head ask = head_ask(p, a.item, a.pos, tag);

    copy_wait();
    __syncwarp();
    Span s{splat(1.f), splat(0.f)};
    float2 Q = splat(0.f);  // the span's gradient in front of it, from none behind: the sum of P_t g_t, P_t = f_1 .. f_t
    float2 coef[J], e[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      float2 in;
      coef[j] = Gt::coef(load2(sz + j * kGatedCG + lane * 2), load2(sx + j * kGatedCG + lane * 2), in);
      if (nt < J && j >= nt) coef[j] = splat(kGateHeld);  // past the end: f = 1 (x and g are 0)
      const float2 A = gate_base(coef[j]);
      s.H = gate_step(A, coef[j], s.H, in);
      s.P = gate_mul(A, coef[j], s.P);
      Q = fma2(s.P, load2(sg + j * kGatedCG + lane * 2), Q);
      if (j % 4 == 3) asm volatile("" ::: "memory");  // four tokens' loads and exponentials at a time: registers
    }
    sh.agg[par][w][lane] = s;
    sh.rev[par][w][lane] = Q;
    if (threadIdx.x == 0) sh.next[par] = ticket;
    __syncthreads();
    forget(coef);
    const Tile an = gated_tile(p, sh.next[par]);
    // the states of this span, and with them what D is multiplied by in dz
    for (int i = 0; i < w; ++i) h = apply(sh.agg[par][i][lane], h);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const float2 A = gate_base(coef[j]);
      float2 in;
      e[j] = Gt::slope(A, coef[j], h, load2(sx + j * kGatedCG + lane * 2), in);
      h = gate_step(A, coef[j], h, in);
    }
    forget(coef);
    __syncwarp();
    fetch_xz(an);
    if (kGB == 2) fetch_g(an, sg0 + (par ? 0 : row));
    copy_commit();
    const float2 first = a.pos == 0 ? sh.first[par][lane] : splat(0.f);
    float2 q;  // f_{t+1} D_{t+1}, what flows back into token t
    if (chained && p.G > 1) {
      q = gated_front<GATE == kGateDecay>(p, a.item, a.pos, tag, first, sh.front, [&] {
        Span tot{sh.agg[par][NW - 1][lane].P, sh.rev[par][NW - 1][lane]};
        for (int i = NW - 2; i >= 0; --i) {
          const Span u{sh.agg[par][i][lane].P, sh.rev[par][i][lane]};
          tot.H = apply(u, tot.H);
          tot.P = mul2(tot.P, u.P);
        }
        return tot;
      });
    } else {
      q = head_get(p, a.item, a.pos, tag, first, ask);
    }
    for (int i = NW - 1; i > w; --i) q = fma2(sh.agg[par][i][lane].P, q, sh.rev[par][i][lane]);
    if (chained && p.G == 1 && w == 0 && a.pos != p.nch - 1)
      rec_put(p, p.pre, ((size_t)a.item * p.ngrp + a.pos) * kGatedCG + lane * 2,
              (size_t)p.B * p.NG * p.ngrp * kGatedCG, splat(0.f), fma2(s.P, q, Q), tag);
    long long o = ((long long)a.b * p.T + t0 + J - 1) * p.C + c0;
    const bool on = c0 < p.C;
    if (nt >= J && p.pair) {
#pragma unroll
      for (int j = J - 1; j >= 0; --j) {
        const float2 A = gate_base(coef[j]), D = add2(load2(sg + j * kGatedCG + lane * 2), q);
        q = gate_mul(A, coef[j], D);
        if (on && WKV_IN(p.hdr, o + 1, (size_t)p.B * p.T * p.C)) {
          store2(static_cast<X*>(p.dx) + o, Gt::input(A, coef[j], D));
          store2(static_cast<Z*>(p.dz) + o, mul2(D, e[j]));
        }
        o -= p.C;
      }
    } else {
#pragma unroll
      for (int j = J - 1; j >= 0; --j) {
        const float2 A = gate_base(coef[j]), D = add2(load2(sg + j * kGatedCG + lane * 2), q);
        q = gate_mul(A, coef[j], D);
        if (on && j < nt && WKV_IN(p.hdr, o, (size_t)p.B * p.T * p.C)) {
          store_one(static_cast<X*>(p.dx) + o, Gt::input(A, coef[j], D), c0 + 1 < p.C);
          store_one(static_cast<Z*>(p.dz) + o, mul2(D, e[j]), c0 + 1 < p.C);
        }
        o -= p.C;
      }
    }
    if (p.dh0 && chunk == 0 && w == 0) row_put(p.hdr, p.dh0, (long long)a.b * p.C, c0, p.C, (size_t)p.B * p.C, q);
    if (kGB == 1) {
      __syncwarp();
      fetch_g(an, sg0);
      copy_commit();
    }
    a = an;
  }
  if (chained) gated_leave(p, sh.epoch);
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

// Elementwise and bound by memory (20 bytes per stream-channel in fp32, 14 in
// bf16); four channels per thread move as 16-byte accesses of the state. Steps
// of 4096 x 768 bf16, one after the other: 6.7 us on the same 44 MB (in L2), 8.4
// us from DRAM (0.80 of the copy rate).
template <typename X, typename Z, typename O, int GATE, int V>
__global__ void __launch_bounds__(256) gated_step_kernel(const GatedStepParams p) {
  follow_on();
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
  for (int v = 0; v < V; v += 2) {
    constexpr int k = V > 1 ? 1 : 0;  // V = 1: the second half of the pair repeats the first
    float2 in;
    const float2 c = Gate<GATE>::coef(make_float2(z[v], z[v + k]), make_float2(x[v], x[v + k]), in);
    const float2 r = gate_step(gate_base(c), c, make_float2(h[v], h[v + k]), in);
    h[v + k] = r.y;
    h[v] = r.x;
  }
  store_vec<float, V>(p.h_out + o, h);
  store_vec<O, V>(static_cast<O*>(p.out) + o, h);
}

}  // namespace wkv
