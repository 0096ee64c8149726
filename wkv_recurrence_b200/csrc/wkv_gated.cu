// C ABI of the gated linear recurrence (declared in include/wkv.h): argument
// checks, tile sizes, workspace layout and launches of the kernels in
// wkv_gated.cuh. Nothing here allocates device memory.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "wkv_gated.cuh"
#include "wkv_host_util.h"

namespace wkv {
namespace {

constexpr int kGatedL = WKV_GATED_TILE;  // tokens per tile of a sequence of several tiles
constexpr int kGatedJ = 16;              // tokens per warp
constexpr int kGatedNW = kGatedL / kGatedJ;
constexpr int kMaxDevices = 64;

struct GatedPlan {
  int NG, nch, G, ngrp, NW;
  long long tiles;
  size_t off_tot, off_pre, bytes;
};

// Sizes as wkv_forward's: B, T, C >= 0, T < 2^24, B*T*C < 2^62; and fewer than
// 2^31 tiles.
bool gated_plan(int64_t B, int64_t T, int64_t C, GatedPlan* pl) {
  if (B < 0 || T < 0 || C < 0) return false;
  if (T >= (1ll << 24) || C >= (1ll << 31) - kGatedCG || B >= (1ll << 31)) return false;
  if (B > 0 && C > 0 && T > (int64_t)((1ull << 62) / (uint64_t)(B * C))) return false;
  const int64_t NG = (C + kGatedCG - 1) / kGatedCG, nch = (T + kGatedL - 1) / kGatedL;
  const int64_t items = B * NG;
  if (items >= (1ll << 31) || (items > 0 && nch > (int64_t)(((1ll << 31) - 1) / items))) return false;
  pl->NG = (int)NG;
  pl->nch = (int)nch;
  pl->NW = nch > 1 ? kGatedNW : (int)std::max<int64_t>(1, (T + kGatedJ - 1) / kGatedJ);
  // Tiles per look-back group: one where the tile before is long done when a
  // tile starts (about 300 run at once). Else a hop from group to group must
  // not limit, nor the G - 1 totals that a tile may have to read (1 x 65536 x
  // 2048 fp32, 32 channel groups, forward: G = 1 558 us, 2 360, 4 344, 8 332,
  // 16 311, 32 330; 1 x 65536 x 64: G = 16 24.9 us, 32 20.1, 64 21.0).
  int G = 1;
  if (items < 256)
    while (G < 32 && G * items < 512) G *= 2;
  pl->G = G;
  pl->ngrp = (int)((nch + pl->G - 1) / pl->G);
  pl->tiles = items * nch;
  size_t off = sizeof(WsHeader);
  pl->off_tot = off;
  if (nch > 1 && pl->G > 1) off = round_up(off + sizeof(GatedRec) * (size_t)(items * nch * kGatedCG), 256);
  pl->off_pre = off;
  if (nch > 1) off = round_up(off + sizeof(GatedRec) * (size_t)(items * pl->ngrp * kGatedCG), 256);
  pl->bytes = off;
  return true;
}

bool types_ok(int x, int z, int o) {
  if ((x != WKV_F32 && x != WKV_BF16) || (z != WKV_F32 && z != WKV_BF16) || (o != WKV_F32 && o != WKV_BF16)) return false;
  return x == WKV_BF16 || (z == WKV_F32 && o == WKV_F32);
}

size_t elem(int d) { return d == WKV_F32 ? 4 : 2; }

bool vec_ok(const void* p, int dt, int V, int64_t s0 = 0, int64_t s1 = 0) {
  return aligned(p, elem(dt) * V) && s0 % V == 0 && s1 % V == 0;
}

// The widest copy (16, 4 or 2 bytes) that base, strides and row length allow.
int granule(const void* p, int dt, int64_t C, int64_t s0, int64_t s1) {
  const int64_t es = (int64_t)elem(dt);
  for (const int g : {16, 4})
    if (aligned(p, g) && C * es % g == 0 && s0 * es % g == 0 && s1 * es % g == 0) return g;
  return 2;
}

// CTAs to launch: as many as are resident at once, at most one per tile. The
// kernel's shared memory limit is raised and its occupancy looked up once per
// device.
struct Resident {
  std::mutex mu;
  int ctas[kMaxDevices] = {};
};

template <typename F>
bool resident(Resident& r, F fn, int threads, size_t smem, int* ctas) {
  int dev = 0;
  if (!cuda_ok(cudaGetDevice(&dev)) || dev >= kMaxDevices) return false;
  std::lock_guard<std::mutex> lk(r.mu);
  if (r.ctas[dev] == 0) {
    int sms = 0, per = 0;
    if (!cuda_ok(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) ||
        !cuda_ok(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, fn, threads, smem)) ||
        !cuda_ok(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)))
      return false;
    r.ctas[dev] = std::max(1, per) * sms;
  }
  *ctas = r.ctas[dev];
  return true;
}

struct FwdLaunch {
  template <typename X, typename Z, typename O, int GATE>
  static wkv_status go(const GatedParams& p, const GatedPlan& pl, cudaStream_t st) {
    static Resident r;
    const auto fn = gated_fwd<X, Z, O, GATE, kGatedJ, kGatedNW>;
    int ctas;
    if (!resident(r, fn, 32 * kGatedNW, gated_fwd_smem<X, Z, kGatedJ, kGatedNW>(), &ctas)) return WKV_ERR_CUDA;
    // a single tile of fewer warps takes less shared memory: more CTAs fit
    const size_t smem = gated_fwd_smem<X, Z, kGatedJ, kGatedNW>() / kGatedNW * pl.NW;
    const long long most = (long long)ctas * (kGatedNW / pl.NW);
    return launch_follow_on(fn, (unsigned)std::min(pl.tiles, most), 32 * pl.NW, smem, st, p);
  }
};
struct BwdLaunch {
  template <typename X, typename Z, typename O, int GATE>
  static wkv_status go(const GatedParams& p, const GatedPlan& pl, cudaStream_t st) {
    static Resident r;
    const auto fn = gated_bwd<X, Z, O, GATE, kGatedJ, kGatedNW>;
    using Smem = GatedBwdSmem<X, Z, O, kGatedJ, kGatedNW>;
    int ctas;
    if (!resident(r, fn, 32 * kGatedNW, Smem::kBytes, &ctas)) return WKV_ERR_CUDA;
    const size_t smem = Smem::kBytes / kGatedNW * pl.NW;
    const long long most = (long long)ctas * (kGatedNW / pl.NW);
    return launch_follow_on(fn, (unsigned)std::min(pl.tiles, most), 32 * pl.NW, smem, st, p);
  }
};

template <typename F, typename X, typename Z, typename O>
wkv_status by_gate(int gate, const GatedParams& p, const GatedPlan& pl, cudaStream_t st) {
  return gate == WKV_GATE_SIGMOID ? F::template go<X, Z, O, kGateSigmoid>(p, pl, st)
                                  : F::template go<X, Z, O, kGateDecay>(p, pl, st);
}

template <typename F>
wkv_status by_type(int x, int z, int o, int gate, const GatedParams& p, const GatedPlan& pl, cudaStream_t st) {
  using bf = __nv_bfloat16;
  if (x == WKV_F32) return by_gate<F, float, float, float>(gate, p, pl, st);
  if (z == WKV_F32)
    return o == WKV_F32 ? by_gate<F, bf, float, float>(gate, p, pl, st) : by_gate<F, bf, float, bf>(gate, p, pl, st);
  return o == WKV_F32 ? by_gate<F, bf, bf, float>(gate, p, pl, st) : by_gate<F, bf, bf, bf>(gate, p, pl, st);
}

template <typename X, typename Z, typename O>
wkv_status step_launch(int gate, int V, const GatedStepParams& p, cudaStream_t st) {
  const unsigned grid = (unsigned)((p.n + 255) / 256);
  if (gate == WKV_GATE_SIGMOID) {
    if (V == 4) return launch_follow_on(gated_step_kernel<X, Z, O, kGateSigmoid, 4>, grid, 256, 0, st, p);
    else return launch_follow_on(gated_step_kernel<X, Z, O, kGateSigmoid, 1>, grid, 256, 0, st, p);
  } else {
    if (V == 4) return launch_follow_on(gated_step_kernel<X, Z, O, kGateDecay, 4>, grid, 256, 0, st, p);
    else return launch_follow_on(gated_step_kernel<X, Z, O, kGateDecay, 1>, grid, 256, 0, st, p);
  }
}

// A state passed through unchanged (no tokens): copied, or zeros.
wkv_status pass_state(const float* in, float* out, int64_t n, cudaStream_t st) {
  if (!out || out == in || n == 0) return WKV_OK;
  const size_t bytes = sizeof(float) * (size_t)n;
  const cudaError_t e =
      in ? cudaMemcpyAsync(out, in, bytes, cudaMemcpyDeviceToDevice, st) : cudaMemsetAsync(out, 0, bytes, st);
  return cuda_ok(e) ? WKV_OK : WKV_ERR_CUDA;
}

Divisor divisor(uint32_t d) {
  int s = 0;
  while ((1ull << s) < d) ++s;
  return Divisor{d, (uint32_t)(((1ull << (31 + s)) + d - 1) / d), 31 + s};
}

void chain(GatedParams* p, const GatedPlan& pl, void* workspace) {
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  p->NG = pl.NG;
  p->nch = pl.nch;
  p->G = pl.G;
  p->ngrp = pl.ngrp;
  p->tiles = pl.tiles;
  p->by_items = divisor((uint32_t)p->B * (uint32_t)pl.NG);
  p->by_ng = divisor((uint32_t)pl.NG);
  p->hdr = reinterpret_cast<WsHeader*>(ws);
  p->tot = reinterpret_cast<GatedRec*>(ws + pl.off_tot);
  p->pre = reinterpret_cast<GatedRec*>(ws + pl.off_pre);
  p->timeout_ns = kDefaultTimeoutNs;
}

// What forward and backward check alike.
wkv_status check_common(int64_t B, int64_t T, int64_t C, const void* x, int x_dtype, int64_t x_sb, int64_t x_st,
                        const void* z, int z_dtype, int64_t z_sb, int64_t z_st, int gate, int o_dtype) {
  GatedPlan pl;
  if (!gated_plan(B, T, C, &pl)) return WKV_ERR_INVALID_ARG;
  if (!types_ok(x_dtype, z_dtype, o_dtype)) return WKV_ERR_UNSUPPORTED_DTYPE;
  if (gate != WKV_GATE_SIGMOID && gate != WKV_GATE_DECAY) return WKV_ERR_INVALID_ARG;
  if (x_sb < 0 || x_st < 0 || z_sb < 0 || z_st < 0) return WKV_ERR_INVALID_ARG;
  if (B > 0 && T > 0 && C > 0) {
    if (!x || !z) return WKV_ERR_INVALID_ARG;
    if (!aligned(x, elem(x_dtype)) || !aligned(z, elem(z_dtype))) return WKV_ERR_MISALIGNED;
    // the last element of each input is addressed with 62 bits
    const uint64_t lim = 1ull << 62;
    for (const int64_t* s : {&x_sb, &z_sb})
      if (B > 1 && (uint64_t)*s > lim / (uint64_t)B) return WKV_ERR_INVALID_ARG;
    for (const int64_t* s : {&x_st, &z_st})
      if (T > 1 && (uint64_t)*s > lim / (uint64_t)T) return WKV_ERR_INVALID_ARG;
  }
  return WKV_OK;
}

wkv_status check_workspace(const GatedPlan& pl, void* workspace, size_t bytes) {
  if (pl.nch <= 1) return WKV_OK;  // nothing waits, nothing is kept
  if (!workspace) return WKV_ERR_INVALID_ARG;
  if (!aligned(workspace, 256)) return WKV_ERR_MISALIGNED;
  return bytes < pl.bytes ? WKV_ERR_WORKSPACE_TOO_SMALL : WKV_OK;
}

}  // namespace
}  // namespace wkv

using namespace wkv;

extern "C" {

size_t wkv_gated_workspace_size(int64_t B, int64_t T, int64_t C) {
  GatedPlan pl;
  return gated_plan(B, T, C, &pl) ? pl.bytes : 0;
}

wkv_status wkv_gated_forward(int64_t B, int64_t T, int64_t C, const void* x, wkv_dtype x_dtype, int64_t x_batch_stride,
                             int64_t x_token_stride, const void* z, wkv_dtype z_dtype, int64_t z_batch_stride,
                             int64_t z_token_stride, wkv_gate gate, void* out, wkv_dtype out_dtype,
                             const float* state_in, float* state_out, float* checkpoints, void* workspace,
                             size_t workspace_bytes, void* stream) {
  const wkv_status chk = check_common(B, T, C, x, x_dtype, x_batch_stride, x_token_stride, z, z_dtype, z_batch_stride,
                                      z_token_stride, gate, out_dtype);
  if (chk != WKV_OK) return chk;
  if (out && !aligned(out, elem(out_dtype))) return WKV_ERR_MISALIGNED;
  if (!aligned(state_in, 4) || !aligned(state_out, 4) || !aligned(checkpoints, 4)) return WKV_ERR_MISALIGNED;
  GatedPlan pl;
  if (!gated_plan(B, T, C, &pl)) return WKV_ERR_INVALID_ARG;
  const wkv_status wchk = check_workspace(pl, workspace, workspace_bytes);
  if (wchk != WKV_OK) return wchk;
  if (B == 0 || C == 0) return WKV_OK;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (T == 0) return pass_state(state_in, state_out, B * C, st);
  GatedParams p;
  std::memset(&p, 0, sizeof p);
  p.B = (int)B;
  p.T = (int)T;
  p.C = (int)C;
  p.x = x;
  p.z = z;
  p.x_sb = x_batch_stride;
  p.x_st = x_token_stride;
  p.z_sb = z_batch_stride;
  p.z_st = z_token_stride;
  p.h0 = state_in;
  p.marks = checkpoints;
  p.out = out;
  p.h_out = state_out;
  p.x_gran = granule(x, x_dtype, C, x_batch_stride, x_token_stride);
  p.z_gran = granule(z, z_dtype, C, z_batch_stride, z_token_stride);
  p.pair = C % 2 == 0 && vec_ok(out, out_dtype, 2);
  chain(&p, pl, workspace);
  return by_type<FwdLaunch>(x_dtype, z_dtype, out_dtype, gate, p, pl, st);
}

wkv_status wkv_gated_backward(int64_t B, int64_t T, int64_t C, const void* x, wkv_dtype x_dtype, int64_t x_batch_stride,
                              int64_t x_token_stride, const void* z, wkv_dtype z_dtype, int64_t z_batch_stride,
                              int64_t z_token_stride, wkv_gate gate, const void* gout, wkv_dtype g_dtype,
                              const float* state_in, const float* dstate_out, const float* checkpoints, void* dx,
                              void* dz, float* dstate_in, void* workspace, size_t workspace_bytes, void* stream) {
  const wkv_status chk = check_common(B, T, C, x, x_dtype, x_batch_stride, x_token_stride, z, z_dtype, z_batch_stride,
                                      z_token_stride, gate, g_dtype);
  if (chk != WKV_OK) return chk;
  const bool any = B > 0 && T > 0 && C > 0;
  if (any && (!gout || !dx || !dz)) return WKV_ERR_INVALID_ARG;
  if (any && (!aligned(gout, elem(g_dtype)) || !aligned(dx, elem(x_dtype)) || !aligned(dz, elem(z_dtype))))
    return WKV_ERR_MISALIGNED;
  if (!aligned(state_in, 4) || !aligned(dstate_out, 4) || !aligned(checkpoints, 4) || !aligned(dstate_in, 4))
    return WKV_ERR_MISALIGNED;
  GatedPlan pl;
  if (!gated_plan(B, T, C, &pl)) return WKV_ERR_INVALID_ARG;
  if (any && pl.nch > 1 && !checkpoints) return WKV_ERR_INVALID_ARG;
  const wkv_status wchk = check_workspace(pl, workspace, workspace_bytes);
  if (wchk != WKV_OK) return wchk;
  if (B == 0 || C == 0) return WKV_OK;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (T == 0) return pass_state(dstate_out, dstate_in, B * C, st);
  GatedParams p;
  std::memset(&p, 0, sizeof p);
  p.B = (int)B;
  p.T = (int)T;
  p.C = (int)C;
  p.x = x;
  p.z = z;
  p.x_sb = x_batch_stride;
  p.x_st = x_token_stride;
  p.z_sb = z_batch_stride;
  p.z_st = z_token_stride;
  p.h0 = state_in;
  p.marks = const_cast<float*>(checkpoints);
  p.g = gout;
  p.dh_out = dstate_out;
  p.dx = dx;
  p.dz = dz;
  p.dh0 = dstate_in;
  p.x_gran = granule(x, x_dtype, C, x_batch_stride, x_token_stride);
  p.z_gran = granule(z, z_dtype, C, z_batch_stride, z_token_stride);
  p.g_gran = granule(gout, g_dtype, C, 0, 0);
  p.pair = C % 2 == 0 && vec_ok(dx, x_dtype, 2) && vec_ok(dz, z_dtype, 2);
  chain(&p, pl, workspace);
  return by_type<BwdLaunch>(x_dtype, z_dtype, g_dtype, gate, p, pl, st);
}

wkv_status wkv_gated_step(int64_t S, int64_t C, const void* x, wkv_dtype x_dtype, int64_t x_stride, const void* z,
                          wkv_dtype z_dtype, int64_t z_stride, wkv_gate gate, void* out, wkv_dtype out_dtype,
                          const float* state_in, float* state_out, void* stream) {
  if (S < 0 || C < 0 || C >= (1ll << 31) || (S > 0 && C > (int64_t)((1ull << 38) / (uint64_t)S))) return WKV_ERR_INVALID_ARG;
  if (!types_ok(x_dtype, z_dtype, out_dtype)) return WKV_ERR_UNSUPPORTED_DTYPE;
  if (gate != WKV_GATE_SIGMOID && gate != WKV_GATE_DECAY) return WKV_ERR_INVALID_ARG;
  if (x_stride < 0 || z_stride < 0) return WKV_ERR_INVALID_ARG;
  if (S * C == 0) return WKV_OK;
  if (!x || !z || !out || !state_in || !state_out) return WKV_ERR_INVALID_ARG;
  if (!aligned(x, elem(x_dtype)) || !aligned(z, elem(z_dtype)) || !aligned(out, elem(out_dtype)) ||
      !aligned(state_in, 4) || !aligned(state_out, 4))
    return WKV_ERR_MISALIGNED;
  const int V = C % 4 == 0 && vec_ok(x, x_dtype, 4, x_stride) && vec_ok(z, z_dtype, 4, z_stride) &&
                        vec_ok(out, out_dtype, 4) && aligned(state_in, 16) && aligned(state_out, 16)
                    ? 4
                    : 1;
  GatedStepParams p;
  p.n = S * C / V;
  p.CV = (int)(C / V);
  p.C = (int)C;
  p.x = x;
  p.z = z;
  p.x_ss = x_stride;
  p.z_ss = z_stride;
  p.h_in = state_in;
  p.h_out = state_out;
  p.out = out;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  using bf = __nv_bfloat16;
  if (x_dtype == WKV_F32) return step_launch<float, float, float>(gate, V, p, st);
  if (z_dtype == WKV_F32)
    return out_dtype == WKV_F32 ? step_launch<bf, float, float>(gate, V, p, st)
                                : step_launch<bf, float, bf>(gate, V, p, st);
  return out_dtype == WKV_F32 ? step_launch<bf, bf, float>(gate, V, p, st) : step_launch<bf, bf, bf>(gate, V, p, st);
}

}  // extern "C"
