// C ABI of the RMS norm (declared in include/wkv.h): argument checks, the
// choice of kernel, workspace layout and launches of wkv_norm.cuh. Nothing
// here allocates device memory.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <new>
#include <utility>
#include <vector>

#include "wkv_host_util.h"
#include "wkv_norm.cuh"

namespace wkv {
namespace {

using bf = __nv_bfloat16;
constexpr int kSms = 148;
constexpr int64_t kMaxGroups = 8192;  // wkv_norm_row keeps one float per group in shared memory

size_t elem(int d) { return d == WKV_F32 ? 4 : 2; }
bool dtype_ok(int d) { return d == WKV_F32 || d == WKV_BF16; }

bool sizes_ok(int64_t N, int64_t C, int64_t G) {
  if (N < 0 || C < 0 || G < 1 || G > kMaxGroups || C % G != 0) return false;
  return N < (1ll << 31) && C < (1ll << 24);
}

// Rows that start on 16 bytes.
bool rows_ok(const void* p, int dt, int64_t stride) {
  return aligned(p, 16) && (stride * (int64_t)elem(dt)) % 16 == 0;
}

// The team that holds a group of D columns: TW lanes (0: a whole CTA of
// `threads`) with K vectors each, adjacent columns or (sc) strided ones. K = 0:
// too wide for registers.
struct Team {
  int TW, K, threads;
  bool sc;
};

Team cta_team(int64_t n8, int K, bool sc) { return Team{0, K, (int)round_up((size_t)((n8 + K - 1) / K), 32), sc}; }

Team fwd_team(int64_t D, bool vec) {
  const int64_t n8 = (D + 7) / 8;
  if (n8 > 4096) return Team{0, 0, 0, false};
  if (n8 <= 32) {
    // a power of two of lanes, or three vectors on a quarter as many where
    // that leaves none idle (96 columns: 4 lanes x 3 against 12 of 16 lanes)
    int tw = 4;
    while (tw < n8) tw *= 2;
    if (vec && n8 * 4 == 3ll * tw && tw >= 16) return Team{tw / 4, 3, 256, false};
    return Team{tw, 1, 256, !vec};
  }
  if (n8 <= 128) return Team{32, (int)((n8 + 31) / 32), 256, !vec};
  return cta_team(n8, n8 <= 256 ? 1 : n8 <= 1024 ? 2 : n8 <= 2048 ? 4 : 8, !vec);
}

// s_bf: s (and gs, ds) in bf16; gs: the stream's own gradient is added. Two
// vectors a thread keep more bytes under way and let half as many warps meet at
// a row's barrier, where the registers hold them (65536 x 2048, gs: bf16 199 us
// with one, 184 with two; fp32 376 and 310; 65536 x 12 x 64 bf16: 63 and 57).
// fp32 without gs does better with one (32768 x 4096, gy bf16: 209 and 259).
Team bwd_team(int64_t D, int64_t G, bool vec, bool s_bf, bool gs) {
  const int64_t n8 = (D + 7) / 8;
  if (n8 <= (vec ? 64 : 32)) {
    int tw = 4;
    while (tw < n8 && tw < 32) tw *= 2;
    const bool two = vec && (n8 > 32 || (s_bf && n8 > 4));
    if (two && n8 <= 32) tw /= 2;
    if (tw * G <= 512) return Team{tw, two ? 2 : 1, 0, !vec};
  }
  if (G == 1 && n8 <= 2048) return cta_team(n8, n8 <= (vec && (s_bf || gs) ? 96 : 512) ? 1 : n8 <= 1024 ? 2 : 4, !vec);
  return Team{0, 0, 0, false};
}

struct BwdPlan {
  Team team;
  int rpc, threads, nparts;
};

// vec: 16-byte aligned rows. Without a team (team.K = 0) the general kernels
// run, on nparts parts of the rows.
BwdPlan bwd_plan(int64_t N, int64_t C, int64_t G, bool vec, bool s_bf, bool gs) {
  BwdPlan pl;
  pl.team = bwd_team(C / G, G, vec && (C / G) % 8 == 0, s_bf, gs);
  pl.rpc = 1;
  pl.threads = pl.team.threads;
  if (!pl.team.K) {
    pl.nparts = (int)std::max<int64_t>(1, std::min<int64_t>(N, 256));
    return pl;
  }
  if (pl.team.TW) {
    const int tpr = pl.team.TW * (int)G;
    pl.rpc = std::max(1, 256 / tpr);
    pl.threads = (int)round_up((size_t)pl.rpc * tpr, 32);
  }
  // at most one wave; the launch takes as many of these as are resident
  const int per_sm = std::max(1, 1024 / pl.threads);
  pl.nparts = (int)std::max<int64_t>(1, std::min<int64_t>((N + pl.rpc - 1) / pl.rpc, (int64_t)kSms * per_sm));
  return pl;
}

// [parts][C] floats, then [N][G] for the general kernels: enough for whatever
// a call's alignment and types take.
size_t bwd_parts_bytes(int64_t N, int64_t C, int64_t G) {
  size_t most = 0;
  for (int k = 0; k < 8; ++k) most = std::max(most, (size_t)bwd_plan(N, C, G, k & 1, k & 2, k & 4).nparts);
  return round_up(sizeof(float) * std::max<size_t>(most, 256) * (size_t)C, 256);
}

template <typename X, typename R, bool RES, int TW, int K, bool SC = false>
wkv_status launch_team(const NormParams& p, int threads, cudaStream_t st) {
  const long long segs = p.N * p.G;
  const unsigned grid = (unsigned)(TW ? (segs * TW + 255) / 256 : segs);
  return launch_follow_on(wkv_norm_team<X, R, RES, TW, K, SC>, grid, (unsigned)threads, 0, st, p);
}

template <typename X, typename R, bool RES>
wkv_status fwd_shape(const NormParams& p, const Team& t, cudaStream_t st) {
  if (t.sc) {
    switch (t.TW * 16 + t.K) {
      case 4 * 16 + 1: return launch_team<X, R, RES, 4, 1, true>(p, t.threads, st);
      case 8 * 16 + 1: return launch_team<X, R, RES, 8, 1, true>(p, t.threads, st);
      case 16 * 16 + 1: return launch_team<X, R, RES, 16, 1, true>(p, t.threads, st);
      case 32 * 16 + 1: return launch_team<X, R, RES, 32, 1, true>(p, t.threads, st);
      case 32 * 16 + 2: return launch_team<X, R, RES, 32, 2, true>(p, t.threads, st);
      case 32 * 16 + 3: return launch_team<X, R, RES, 32, 3, true>(p, t.threads, st);
      case 32 * 16 + 4: return launch_team<X, R, RES, 32, 4, true>(p, t.threads, st);
      case 1: return launch_team<X, R, RES, 0, 1, true>(p, t.threads, st);
      case 2: return launch_team<X, R, RES, 0, 2, true>(p, t.threads, st);
      case 4: return launch_team<X, R, RES, 0, 4, true>(p, t.threads, st);
      default: return launch_team<X, R, RES, 0, 8, true>(p, t.threads, st);
    }
  }
  switch (t.TW * 16 + t.K) {
    case 4 * 16 + 1: return launch_team<X, R, RES, 4, 1>(p, t.threads, st);
    case 4 * 16 + 3: return launch_team<X, R, RES, 4, 3>(p, t.threads, st);
    case 8 * 16 + 1: return launch_team<X, R, RES, 8, 1>(p, t.threads, st);
    case 8 * 16 + 3: return launch_team<X, R, RES, 8, 3>(p, t.threads, st);
    case 16 * 16 + 1: return launch_team<X, R, RES, 16, 1>(p, t.threads, st);
    case 32 * 16 + 1: return launch_team<X, R, RES, 32, 1>(p, t.threads, st);
    case 32 * 16 + 2: return launch_team<X, R, RES, 32, 2>(p, t.threads, st);
    case 32 * 16 + 3: return launch_team<X, R, RES, 32, 3>(p, t.threads, st);
    case 32 * 16 + 4: return launch_team<X, R, RES, 32, 4>(p, t.threads, st);
    case 1: return launch_team<X, R, RES, 0, 1>(p, t.threads, st);
    case 2: return launch_team<X, R, RES, 0, 2>(p, t.threads, st);
    case 4: return launch_team<X, R, RES, 0, 4>(p, t.threads, st);
    default: return launch_team<X, R, RES, 0, 8>(p, t.threads, st);
  }
}

// e4m3 scales across groups: TW lanes per group, or 0 where that kernel does
// not fit.
int cross_lanes(int64_t D, int64_t G) {
  int tw = 4;
  while (tw < D / 8) tw *= 2;
  return tw <= 32 && tw * G <= 1024 ? tw : 0;
}

template <typename X, typename R, bool RES>
wkv_status cross_shape(const NormParams& p, int tw, cudaStream_t st) {
  const int tpr = tw * p.G, rpc = std::max(1, 256 / tpr);
  const unsigned grid = (unsigned)((p.N + rpc - 1) / rpc);
  const int threads = (int)round_up((size_t)rpc * tpr, 32);
  const size_t smem = sizeof(int) * (size_t)rpc * p.nb;
  if (tw == 4) return launch_follow_on(wkv_norm_cross<X, R, RES, 4>, grid, (unsigned)threads, smem, st, p, rpc);
  else if (tw == 8) return launch_follow_on(wkv_norm_cross<X, R, RES, 8>, grid, (unsigned)threads, smem, st, p, rpc);
  else if (tw == 16) return launch_follow_on(wkv_norm_cross<X, R, RES, 16>, grid, (unsigned)threads, smem, st, p, rpc);
  else return launch_follow_on(wkv_norm_cross<X, R, RES, 32>, grid, (unsigned)threads, smem, st, p, rpc);
}

template <typename X, typename R, bool RES>
wkv_status fwd_launch(const NormParams& p, const Team& t, int cross, cudaStream_t st) {
  return cross ? cross_shape<X, R, RES>(p, cross, st) : fwd_shape<X, R, RES>(p, t, st);
}

// A general row kernel may use 48 KB of shared memory without asking.
static_assert(kMaxGroups * sizeof(float) <= 40 * 1024, "one float per group");

wkv_status norm(int64_t N, int64_t C, int64_t G, float eps, const void* x, int x_dtype, int64_t x_stride, const void* res,
                int r_dtype, int64_t r_stride, const float* weight, void* y, int out_kind, void* s, float* scale,
                int64_t block, void* stream) {
  if (!sizes_ok(N, C, G)) return WKV_ERR_INVALID_ARG;
  if (!(eps > 0.f) || !std::isfinite(eps)) return WKV_ERR_INVALID_ARG;
  if (!dtype_ok(x_dtype) || (res && !dtype_ok(r_dtype)) || (res && x_dtype == WKV_F32 && r_dtype != WKV_F32))
    return WKV_ERR_UNSUPPORTED_DTYPE;
  if (x_stride < 0 || r_stride < 0 || x_stride > (1ll << 31) || r_stride > (1ll << 31)) return WKV_ERR_INVALID_ARG;
  if (out_kind == kOutE4m3) {
    if (block == 0) block = C;
    if (block != C && ((block != 32 && block != 64 && block != 128) || C % block != 0)) return WKV_ERR_INVALID_ARG;
  }
  if (N == 0 || C == 0) return WKV_OK;
  if (!x || !weight || !y || (res && !s) || (out_kind == kOutE4m3 && !scale)) return WKV_ERR_INVALID_ARG;
  if (!aligned(x, elem(x_dtype)) || !aligned(weight, 4) || (out_kind == kOutF32 && !aligned(y, 4)) ||
      (out_kind == kOutBf16 && !aligned(y, 2)) || (res && (!aligned(res, elem(r_dtype)) || !aligned(s, elem(r_dtype)))) ||
      (out_kind == kOutE4m3 && !aligned(scale, 4)))
    return WKV_ERR_MISALIGNED;
  NormParams p;
  std::memset(&p, 0, sizeof p);
  p.N = N;
  p.C = (int)C;
  p.G = (int)G;
  p.D = (int)(C / G);
  p.eps = eps;
  p.x = x;
  p.x_st = x_stride;
  p.res = res;
  p.res_st = r_stride;
  p.weight = weight;
  p.y = y;
  p.out_kind = out_kind;
  p.s = res ? s : nullptr;
  p.scale = scale;
  p.block = (int)block;
  p.nb = block ? (int)(C / block) : 0;
  p.inv_d = 1.f / (float)p.D;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int64_t D = p.D;
  const bool vec = D % 8 == 0 && rows_ok(x, x_dtype, x_stride) &&
                   (!res || (rows_ok(res, r_dtype, r_stride) && aligned(s, 16))) && aligned(weight, 16) && aligned(y, 16);
  Team t = fwd_team(D, vec);
  int cross = 0;
  if (out_kind == kOutE4m3 && block != D) {
    const int width = t.TW ? t.TW : t.threads;
    if (t.sc || D % block != 0 || block / 8 > width) {
      t.K = 0;
      cross = vec ? cross_lanes(D, G) : 0;
    }
  }
  if ((t.K || cross) && N * G < (1ll << 31)) {
    if (!res)
      return x_dtype == WKV_F32 ? fwd_launch<float, float, false>(p, t, cross, st) : fwd_launch<bf, bf, false>(p, t, cross, st);
    if (x_dtype == WKV_F32) return fwd_launch<float, float, true>(p, t, cross, st);
    return r_dtype == WKV_F32 ? fwd_launch<bf, float, true>(p, t, cross, st) : fwd_launch<bf, bf, true>(p, t, cross, st);
  }
  wkv_norm_row<<<(unsigned)N, 256, sizeof(float) * (size_t)G, st>>>(p, x_dtype == WKV_BF16, r_dtype == WKV_BF16);
  return launch_result();
}

// CTAs of `fn` that are resident on the device at once, looked up once per
// device and block size.
template <typename F>
bool resident(F fn, int threads, size_t smem, int* ctas) {
  struct Entry {
    int dev, threads, ctas;
    size_t smem;
  };
  static std::mutex mu;  // one of each per kernel type F; fn tells kernels of one type apart
  static std::vector<std::pair<F, Entry>> known;
  int dev = 0;
  if (!cuda_ok(cudaGetDevice(&dev))) return false;
  std::lock_guard<std::mutex> lk(mu);
  for (const auto& k : known)
    if (k.first == fn && k.second.dev == dev && k.second.threads == threads && k.second.smem == smem) {
      *ctas = k.second.ctas;
      return true;
    }
  int sms = 0, per = 0;
  if (!cuda_ok(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, fn, threads, smem)) ||
      !cuda_ok(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)))
    return false;
  *ctas = std::max(1, per) * sms;
  try {
    known.push_back({fn, Entry{dev, threads, *ctas, smem}});
  } catch (const std::bad_alloc&) {  // no exception leaves a C entry; looked up again next time
  }
  return true;
}

template <typename Y, typename S, bool GS, int TW, int K, bool SC>
bool bwd_launch(NormBwdParams& p, const BwdPlan& pl, cudaStream_t st) {
  int half = 0;  // the largest power of two below rpc, or 0
  while (std::max(1, 2 * half) < pl.rpc) half = std::max(1, 2 * half);
  const size_t smem = sizeof(float) * (size_t)half * p.C;
  int ctas;
  if (!resident(wkv_norm_bwd_team<Y, S, GS, TW, K, SC>, pl.threads, smem, &ctas)) return false;
  p.nparts = std::min(pl.nparts, ctas);
  return launch_follow_on(wkv_norm_bwd_team<Y, S, GS, TW, K, SC>, (unsigned)p.nparts, (unsigned)pl.threads, smem, st, p,
                          pl.rpc, half) == WKV_OK;
}

template <typename Y, typename S, bool GS>
bool bwd_shape(NormBwdParams& p, const BwdPlan& pl, cudaStream_t st) {
  if (pl.team.sc) {
    switch (pl.team.TW * 8 + pl.team.K) {
      case 4 * 8 + 1: return bwd_launch<Y, S, GS, 4, 1, true>(p, pl, st);
      case 8 * 8 + 1: return bwd_launch<Y, S, GS, 8, 1, true>(p, pl, st);
      case 16 * 8 + 1: return bwd_launch<Y, S, GS, 16, 1, true>(p, pl, st);
      case 32 * 8 + 1: return bwd_launch<Y, S, GS, 32, 1, true>(p, pl, st);
      case 1: return bwd_launch<Y, S, GS, 0, 1, true>(p, pl, st);
      case 2: return bwd_launch<Y, S, GS, 0, 2, true>(p, pl, st);
      default: return bwd_launch<Y, S, GS, 0, 4, true>(p, pl, st);
    }
  }
  switch (pl.team.TW * 8 + pl.team.K) {
    case 4 * 8 + 1: return bwd_launch<Y, S, GS, 4, 1, false>(p, pl, st);
    case 8 * 8 + 1: return bwd_launch<Y, S, GS, 8, 1, false>(p, pl, st);
    case 16 * 8 + 1: return bwd_launch<Y, S, GS, 16, 1, false>(p, pl, st);
    case 32 * 8 + 1: return bwd_launch<Y, S, GS, 32, 1, false>(p, pl, st);
    case 4 * 8 + 2: return bwd_launch<Y, S, GS, 4, 2, false>(p, pl, st);
    case 8 * 8 + 2: return bwd_launch<Y, S, GS, 8, 2, false>(p, pl, st);
    case 16 * 8 + 2: return bwd_launch<Y, S, GS, 16, 2, false>(p, pl, st);
    case 32 * 8 + 2: return bwd_launch<Y, S, GS, 32, 2, false>(p, pl, st);
    case 1: return bwd_launch<Y, S, GS, 0, 1, false>(p, pl, st);
    case 2: return bwd_launch<Y, S, GS, 0, 2, false>(p, pl, st);
    default: return bwd_launch<Y, S, GS, 0, 4, false>(p, pl, st);
  }
}

}  // namespace
}  // namespace wkv

using namespace wkv;

extern "C" {

wkv_status wkv_rms_norm(int64_t N, int64_t C, int64_t groups, float eps, const void* x, wkv_dtype x_dtype, int64_t x_stride,
                        const void* residual, wkv_dtype r_dtype, int64_t r_stride, const float* weight, void* y,
                        wkv_dtype y_dtype, void* sum, void* stream) {
  if (!dtype_ok(y_dtype) || (x_dtype == WKV_F32 && y_dtype != WKV_F32)) return WKV_ERR_UNSUPPORTED_DTYPE;
  return norm(N, C, groups, eps, x, x_dtype, x_stride, residual, r_dtype, r_stride, weight, y,
              y_dtype == WKV_F32 ? kOutF32 : kOutBf16, sum, nullptr, 0, stream);
}

wkv_status wkv_rms_norm_quant(int64_t N, int64_t C, int64_t groups, float eps, const void* x, wkv_dtype x_dtype,
                              int64_t x_stride, const void* residual, wkv_dtype r_dtype, int64_t r_stride,
                              const float* weight, void* q, float* scale, int64_t block, void* sum, void* stream) {
  return norm(N, C, groups, eps, x, x_dtype, x_stride, residual, r_dtype, r_stride, weight, q, kOutE4m3, sum, scale, block,
              stream);
}

size_t wkv_rms_norm_backward_workspace_size(int64_t N, int64_t C, int64_t groups) {
  if (!sizes_ok(N, C, groups)) return 0;
  if (C == 0) return 256;
  return std::max<size_t>(256, bwd_parts_bytes(N, C, groups) + sizeof(float) * (size_t)(N * groups));
}

wkv_status wkv_rms_norm_backward(int64_t N, int64_t C, int64_t groups, float eps, const void* gy, wkv_dtype gy_dtype,
                                 const void* sum, wkv_dtype s_dtype, int64_t s_stride, const float* weight, const void* gsum,
                                 void* dsum, float* dweight, void* workspace, size_t workspace_bytes, void* stream) {
  if (!sizes_ok(N, C, groups)) return WKV_ERR_INVALID_ARG;
  if (!(eps > 0.f) || !std::isfinite(eps)) return WKV_ERR_INVALID_ARG;
  if (!dtype_ok(gy_dtype) || !dtype_ok(s_dtype) || (gy_dtype == WKV_F32 && s_dtype != WKV_F32))
    return WKV_ERR_UNSUPPORTED_DTYPE;
  if (s_stride < 0 || s_stride > (1ll << 31)) return WKV_ERR_INVALID_ARG;
  if (C == 0) return WKV_OK;
  if (!weight || !dweight) return WKV_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (N == 0) return cuda_ok(cudaMemsetAsync(dweight, 0, sizeof(float) * (size_t)C, st)) ? WKV_OK : WKV_ERR_CUDA;
  if (!gy || !sum || !dsum || !workspace) return WKV_ERR_INVALID_ARG;
  if (workspace_bytes < wkv_rms_norm_backward_workspace_size(N, C, groups)) return WKV_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(workspace, 256) || !aligned(gy, elem(gy_dtype)) || !aligned(sum, elem(s_dtype)) ||
      !aligned(dsum, elem(s_dtype)) || (gsum && !aligned(gsum, elem(s_dtype))) || !aligned(weight, 4) || !aligned(dweight, 4))
    return WKV_ERR_MISALIGNED;
  NormBwdParams p;
  std::memset(&p, 0, sizeof p);
  p.N = N;
  p.C = (int)C;
  p.G = (int)groups;
  p.D = (int)(C / groups);
  p.eps = eps;
  p.gy = gy;
  p.s = sum;
  p.s_st = s_stride;
  p.weight = weight;
  p.gs = gsum;
  p.ds = dsum;
  p.part = static_cast<float*>(workspace);
  p.rstd = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + bwd_parts_bytes(N, C, groups));
  p.inv_d = 1.f / (float)p.D;
  const BwdPlan pl = bwd_plan(N, C, groups,
                              aligned(gy, 16) && rows_ok(sum, s_dtype, s_stride) && (!gsum || aligned(gsum, 16)) &&
                                  aligned(dsum, 16) && aligned(weight, 16),
                              s_dtype == WKV_BF16, gsum != nullptr);
  p.nparts = pl.nparts;
  if (pl.team.K) {
    bool ok;
    if (gy_dtype == WKV_F32) {
      ok = gsum ? bwd_shape<float, float, true>(p, pl, st) : bwd_shape<float, float, false>(p, pl, st);
    } else if (s_dtype == WKV_F32) {
      ok = gsum ? bwd_shape<bf, float, true>(p, pl, st) : bwd_shape<bf, float, false>(p, pl, st);
    } else {
      ok = gsum ? bwd_shape<bf, bf, true>(p, pl, st) : bwd_shape<bf, bf, false>(p, pl, st);
    }
    if (!ok) return WKV_ERR_CUDA;
  } else {
    wkv_norm_bwd_row<<<(unsigned)N, 256, 0, st>>>(p, gy_dtype == WKV_BF16, s_dtype == WKV_BF16);
    wkv_norm_bwd_cols<<<dim3((unsigned)((C + 255) / 256), (unsigned)p.nparts), 256, 0, st>>>(p, gy_dtype == WKV_BF16,
                                                                                             s_dtype == WKV_BF16);
  }
  if (launch_result() != WKV_OK) return WKV_ERR_CUDA;
  return launch_follow_on(wkv_norm_bwd_join, (unsigned)((C + 31) / 32), 1024, 0, st, (const float*)p.part, p.nparts, p.C,
                          dweight);
}

}  // extern "C"
