// blocks.cu -- entry points of the operators between a model's two ends when it
// is trained: the gated MLP block and its gradient, the gradient of the fused
// residual add + RMSNorm.  Argument checks, workspace layout, launch.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "../../include/gbfuse.h"
#include "../../include/gbfuse_debug.h"
#include "internal.h"

namespace gbf {

namespace {

constexpr int64_t kMaxInt = (int64_t(1) << 31) - 1;
constexpr int kMaxSms = 152;   // of the device this library is built for
constexpr int kMlpPairs = 76;  // CTA pairs that run at once
constexpr int kMlpRows = 256;  // of a pair's tile

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
bool aligned(const void* p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
gbf_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? GBF_OK : GBF_ERR_CUDA; }
int64_t ceil_div64(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Rows and products of one launch, without its tensor maps.
void set_job(MbJob* j, int mode, int64_t rows, int64_t cols, int64_t k, bool a_mn, bool b_mn) {
  j->mode = mode;
  j->rows = static_cast<int>(rows);
  j->cols = static_cast<int>(cols);
  j->a_mn = a_mn;
  j->b_mn = b_mn;
  j->num_kb = j->kb_first = static_cast<int>(ceil_div64(k, kBK));
  j->splits = 1;
  j->m_pad = 0;
}
int64_t mlp_m_pad(int64_t M) { return ceil_div64(M, 512) * 512; }
void set_dx(MbJob* j, int64_t M, int64_t D, int64_t F, int splits) {
  set_job(j, kMbStore, M, D, F, false, true);
  j->num_kb = 2 * j->kb_first;
  j->splits = splits;
  j->m_pad = static_cast<int>(mlp_m_pad(M));
}

// Row tiles per unit of work: one, or two that share a column tile where that is
// estimated to be faster.
int faster_streams(MbLaunch* l, int64_t M, int64_t* cycles) {
  const int64_t one = plan_mlp_launch(l, 1, kMlpPairs);
  const int64_t two = M > kMlpRows ? plan_mlp_launch(l, 2, kMlpPairs) : one + 1;
  if (cycles) *cycles = std::min(one, two);
  return two < one ? 2 : 1;
}

// The gradient of a weight: [rows][cols] over the M rows of both operands.
void set_dw_job(MbJob* j, int64_t rows, int64_t cols, int64_t M) {
  set_job(j, kMbStore, rows, cols, M, true, true);
  j->splits = static_cast<int>(std::max<int64_t>(1, ceil_div64(M, kGradChain)));
  j->m_pad = static_cast<int>(ceil_div64(rows, 32) * 32);
}
size_t dw_part_bytes(int64_t M, int64_t rows, int64_t cols) {  // of several parts of K
  MbJob j;
  set_dw_job(&j, rows, cols, M);
  return j.splits > 1 ? align256(static_cast<size_t>(j.splits) * j.m_pad * cols * 4) : 0;
}

// Parts of K of the product for dx, each with an fp32 buffer of its own: 16 at most and
// none shorter than 8 K blocks or longer than a chain.
int64_t dx_least_splits(int64_t F) { return std::max<int64_t>(1, ceil_div64(2 * F, kGradChain)); }
int64_t dx_most_splits(int64_t F) {
  return std::max<int64_t>(1, std::min<int64_t>(2 * ceil_div64(F, kBK) / 8, 16));
}
int64_t dx_few_splits(int64_t D, int64_t F) {  // with one row tile
  return std::max(dx_least_splits(F), std::min(dx_most_splits(F), kMlpPairs / ceil_div64(D, 256)));
}
// Bytes of all of them, for M rows and for any fewer: where there are several row tiles
// no more than this are taken (a quarter of a percent of sizes would take more, and lose
// up to 6 % by the estimate), so the size of a workspace never falls with M.
constexpr int64_t kDxPartBytes = int64_t(192) << 20;
int64_t dx_part_bytes(int64_t M, int64_t D, int64_t F, int64_t splits) {
  return splits > 1 ? splits * mlp_m_pad(M) * D * 4 : 0;
}
int64_t dx_part_limit(int64_t M, int64_t D, int64_t F) {
  const int64_t few = M > 0 ? dx_part_bytes(1, D, F, dx_few_splits(D, F)) : 0;
  if (M <= kMlpRows) return few;
  return std::max({few, dx_part_bytes(M, D, F, dx_least_splits(F)),
                   std::min(dx_part_bytes(M, D, F, dx_most_splits(F)), kDxPartBytes)});
}

// The launch of dx and the weights' gradients: row tiles per unit, and the parts of K
// of the product for dx.  With one row tile as many as give one round of units over
// the pairs (all of the gradient of 16 x 4096 x 14336: 3 parts 142 us, 4, one round, 122, 5
// 137, 9 121).  Else as the whole launch is fastest by the estimate; adding the parts
// costs a launch and their traffic (all of the gradient of 1021 x 1000 x 2728: none 58 us,
// 2 or 3 parts 49, 4 52.5).
struct MlpPlan {
  int streams, dx_splits;
};
MlpPlan plan_mlp(int64_t M, int64_t D, int64_t F) {
  MlpPlan p{};
  int64_t best = 0;
  if (M <= kMlpRows) return {1, static_cast<int>(dx_few_splits(D, F))};
  const int64_t most = dx_most_splits(F), limit = dx_part_limit(M, D, F);
  const int least = static_cast<int>(dx_least_splits(F));
  for (int splits = least; splits <= most && dx_part_bytes(M, D, F, splits) <= limit; ++splits) {
    MbLaunch l{};
    set_dx(&l.job[0], M, D, F, splits);
    set_dw_job(&l.job[1], F, D, M);
    set_dw_job(&l.job[2], F, D, M);
    set_dw_job(&l.job[3], D, F, M);
    int64_t cycles;
    const int streams = faster_streams(&l, M, &cycles);
    if (splits > 1) cycles += 6000 + 8 * splits * M * D / 2500;  // bytes at about 4.8 TB/s
    if (splits == least || cycles < best) {
      best = cycles;
      p.streams = streams;
      p.dx_splits = splits;
    }
  }
  return p;
}

// The bytes that a call needs: dg and du, and the parts of K of each result that has
// several.
struct MlpGradWs {
  __nv_bfloat16 *dg, *du;
  float *dx, *dw_gate, *dw_up, *dw_down;
};
size_t mlp_grad_sections(void* base, int64_t M, int64_t D, int64_t F, int dx_splits, bool dx,
                         bool dw_gate, bool dw_up, bool dw_down, MlpGradWs* w) {
  size_t at = 0;
  auto take = [&](size_t bytes) -> void* {
    void* p = base && bytes ? static_cast<uint8_t*>(base) + at : nullptr;
    at += bytes;
    return p;
  };
  const size_t act = dx || dw_gate || dw_up ? align256(static_cast<size_t>(M) * F * 2) : 0;
  w->dg = static_cast<__nv_bfloat16*>(take(act));
  w->du = static_cast<__nv_bfloat16*>(take(act));
  w->dx = static_cast<float*>(take(dx ? align256(dx_part_bytes(M, D, F, dx_splits)) : 0));
  w->dw_gate = static_cast<float*>(take(dw_gate ? dw_part_bytes(M, F, D) : 0));
  w->dw_up = static_cast<float*>(take(dw_up ? dw_part_bytes(M, F, D) : 0));
  w->dw_down = static_cast<float*>(take(dw_down ? dw_part_bytes(M, D, F) : 0));
  return at;
}
// What a call of all four gradients needs with M rows or fewer.
size_t mlp_grad_workspace(int64_t M, int64_t D, int64_t F) {
  return 2 * align256(static_cast<size_t>(M) * F * 2) + align256(dx_part_limit(M, D, F)) +
         2 * dw_part_bytes(M, F, D) + dw_part_bytes(M, D, F);
}

// Sizes that the kernels' 32-bit coordinates and unit counts hold.
bool mlp_sizes_held(int64_t M, int64_t D, int64_t F) {
  if (D < 8 || F < 8 || D % 8 != 0 || F % 8 != 0 || M > (int64_t(1) << 24) ||
      D > (int64_t(1) << 20) || F > (int64_t(1) << 20))
    return false;
  const int64_t m = ceil_div64(M, 256), d = ceil_div64(D, 256), f = ceil_div64(F, 128);
  return m * f <= kMaxInt / 4 && m * d * 16 <= kMaxInt / 4 &&
         d * f * ceil_div64(std::max<int64_t>(M, 1), kGradChain) <= kMaxInt / 4;
}

gbf_status_t check_mlp(int64_t M, int64_t D, int64_t F, int act) {
  if (M < 0 || D < 0 || F < 0 || act < GBF_ACT_IDENTITY || act > GBF_ACT_GELU_TANH)
    return GBF_ERR_INVALID_ARG;
  return mlp_sizes_held(M, D, F) ? GBF_OK : GBF_ERR_UNSUPPORTED_SHAPE;
}

gbf_status_t check_all(std::initializer_list<const void*> required,
                       std::initializer_list<const void*> optional) {
  for (const void* p : required)
    if (!p) return GBF_ERR_INVALID_ARG;
  for (const void* p : required)
    if (!aligned(p, 16)) return GBF_ERR_MISALIGNED;
  for (const void* p : optional)
    if (!aligned(p, 16)) return GBF_ERR_MISALIGNED;
  return GBF_OK;
}

// K-major operand (rows of `inner` values along K): 64 x 128 boxes.
bool map_k(CUtensorMap* m, const void* p, int64_t inner, int64_t outer) {
  return lib_tmap_2d(m, p, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, inner, outer, inner * 2, kBK, 128,
                     CU_TENSOR_MAP_SWIZZLE_128B);
}
// Operand with one row per k: 64 x 64 boxes.
bool map_mn(CUtensorMap* m, const void* p, int64_t inner, int64_t outer) {
  return lib_tmap_2d(m, p, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, inner, outer, inner * 2, 64, kBK,
                     CU_TENSOR_MAP_SWIZZLE_128B);
}
bool map_out(CUtensorMap* m, const void* p, int64_t inner, int64_t outer, bool wide) {
  return wide ? lib_tmap_2d(m, p, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, inner, outer, inner * 2, 64, 32,
                            CU_TENSOR_MAP_SWIZZLE_128B)
              : lib_tmap_2d(m, p, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, inner, outer, inner * 2, 32, 32,
                            CU_TENSOR_MAP_SWIZZLE_64B);
}
bool map_parts(CUtensorMap* m, const void* p, int64_t inner, int64_t outer) {
  return lib_tmap_2d(m, p, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, inner, outer, inner * 4, 16, 32,
                     CU_TENSOR_MAP_SWIZZLE_64B);
}

// The gradient of a weight: out [rows][cols] = a^T b over the M rows of a and b; parts: of
// its K, where there are several.
bool set_dw(MbJob* j, const void* a, const void* b, const void* out, float* parts, int64_t rows,
            int64_t cols, int64_t M) {
  set_dw_job(j, rows, cols, M);
  return map_mn(&j->a[0], a, rows, M) && map_mn(&j->b[0], b, cols, M) &&
         (j->splits > 1 ? map_parts(&j->o[0], parts, cols, static_cast<int64_t>(j->splits) * j->m_pad)
                        : map_out(&j->o[0], out, cols, rows, false));
}

// The kernel of the gate/up product, or of dh, and its launch where that is the CTA
// pairs'; M > 0.
enum MlpPath { kMlpOneSm = 1, kMlpSwap = 2, kMlpPairOne = 8, kMlpPairTwo = 9 };
MlpPath forward_path(int64_t M, int64_t D, int64_t F, int act, MbLaunch* l) {
  set_job(&l->job[1], kMbGlu, M, F, D, false, false);
  l->act = act;
  int64_t cycles;
  const int streams = faster_streams(l, M, &cycles);
  // Few rows or tiles: the weights' bytes or the latency count, and the swapped kernel
  // splits K over clusters (16 x 4096 x 14336: 38 us, pairs 54).  Else the one-SM kernel
  // where its tiles of 128 rows fill their rounds better (64 x 4096 x 14336: 47 us, pairs
  // 56; 257 x 2048 x 5632 21, 28; 256 x 4096 x 14336 64, 56).
  if (lib_glu_swap(M, F, D, true)) return kMlpSwap;
  const int64_t tiles = ceil_div64(M, 128) * ceil_div64(F, 128);
  if (ceil_div64(tiles, kMaxSms) * ceil_div64(D, kBK) * 680 + 9000 < cycles) return kMlpOneSm;
  return streams == 2 ? kMlpPairTwo : kMlpPairOne;
}
MlpPath dh_path(int64_t M, int64_t D, int64_t F, int act, MbLaunch* l) {
  // few rows or tiles, as in gbf_mlp_train (16 x 4096 x 14336, dh alone: 21 us, units of 256
  // rows 32)
  if (lib_glu_swap(M, F, D, false)) return kMlpSwap;
  set_job(&l->job[0], kMbGluGrad, M, F, D, false, true);
  l->act = act;
  return faster_streams(l, M, nullptr) == 2 ? kMlpPairTwo : kMlpPairOne;
}

gbf_status_t run_launch(MbLaunch* l, int streams, const DeviceInfo& dev, unsigned* err,
                        cudaStream_t s) {
  plan_mlp_launch(l, streams, dev.pairs);
  if (l->job[0].units + l->shorts == 0) return GBF_OK;
  return cuda_status(launch_mlp_train(*l, streams, lib_ctl(err, 2 * l->pairs), s));
}

}  // namespace

size_t blocks_workspace_size(int op, int64_t M, int64_t N, int64_t K) {
  if (op == GBF_OP_MLP_GRAD) {
    if (!mlp_sizes_held(M, N, K)) return 0;  // as the entry point refuses them
    return mlp_grad_workspace(M, N, K);
  }
  if (op == GBF_OP_ADD_RMSNORM_GRAD) {
    if (N % 8 != 0 || N > kRmsMaxN || M > kMaxInt) return 0;
    return align256(static_cast<size_t>(rms_grad_sums(M, static_cast<int>(N), kMaxSms)) * N * 4);
  }
  return 0;
}

}  // namespace gbf

using namespace gbf;

extern "C" {

gbf_status_t gbf_mlp_train(const void* x, const void* w_gate, const void* w_up,
                           const void* w_down, const void* residual, void* out, void* g, void* u,
                           void* h, int64_t M, int64_t D, int64_t F, int act,
                           gbf_stream_t stream) {
  gbf_status_t st = check_mlp(M, D, F, act);
  if (st != GBF_OK) return st;
  if (M == 0) {  // arrays without elements may be null
    if ((st = check_all({w_gate, w_up, w_down}, {x, residual, out, g, u, h})) != GBF_OK) return st;
  } else {
    st = check_all({x, w_gate, w_up, w_down, out, g, u, h}, {residual});
    if (st != GBF_OK) return st;
  }
  const DeviceInfo* dev;
  unsigned* err;
  if ((st = lib_device(&dev, &err)) != GBF_OK) return st;
  if (M == 0) return GBF_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  MbLaunch l{};
  MbJob& j = l.job[1];
  const MlpPath path = forward_path(M, D, F, act, &l);
  if (path == kMlpSwap || path == kMlpOneSm) {
    if ((st = lib_glu_keep(x, w_gate, w_up, h, g, u, M, F, D, act, s)) != GBF_OK) return st;
  } else {
    if (!map_k(&j.a[0], x, D, M) || !map_k(&j.b[0], w_gate, D, F) || !map_k(&j.b[1], w_up, D, F) ||
        !map_out(&j.o[0], h, F, M, false) || !map_out(&j.o[1], g, F, M, false) ||
        !map_out(&j.o[2], u, F, M, false))
      return GBF_ERR_CUDA;
    if ((st = run_launch(&l, path == kMlpPairTwo ? 2 : 1, *dev, err, s)) != GBF_OK) return st;
  }
  return lib_mlp_down(h, w_down, residual, out, M, D, F, s);
}

gbf_status_t gbf_mlp_grad(const void* dout, const void* x, const void* g, const void* u,
                          const void* h, const void* w_gate, const void* w_up, const void* w_down,
                          void* dx, void* dw_gate, void* dw_up, void* dw_down, int64_t M,
                          int64_t D, int64_t F, int act, void* workspace, size_t workspace_bytes,
                          gbf_stream_t stream) {
  gbf_status_t st = check_mlp(M, D, F, act);
  if (st != GBF_OK) return st;
  if (M == 0) {
    st = check_all({w_gate, w_up, w_down},
                   {dout, x, g, u, h, dx, dw_gate, dw_up, dw_down, workspace});
  } else {
    if (!dx && !dw_gate && !dw_up && !dw_down) return GBF_ERR_INVALID_ARG;
    st = check_all({dout, x, g, u, h, w_gate, w_up, w_down},
                   {dx, dw_gate, dw_up, dw_down, workspace});
  }
  if (st != GBF_OK) return st;
  const bool hidden = dx || dw_gate || dw_up;
  const MlpPlan plan = plan_mlp(M, D, F);
  const int splits = plan.dx_splits, streams = plan.streams;
  MlpGradWs ws;
  const size_t need = mlp_grad_sections(workspace, M, D, F, splits, dx, dw_gate, dw_up, dw_down, &ws);
  if (need && (!workspace || workspace_bytes < need)) return GBF_ERR_WORKSPACE;
  const DeviceInfo* dev;
  unsigned* err;
  if ((st = lib_device(&dev, &err)) != GBF_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (M == 0) {  // no rows: empty sums
    for (void* dw : {dw_gate, dw_up, dw_down})
      if (dw && (st = cuda_status(cudaMemsetAsync(dw, 0, static_cast<size_t>(D) * F * 2, s))) !=
                    GBF_OK)
        return st;
    return GBF_OK;
  }
  if (hidden) {
    MbLaunch l{};
    MbJob& j = l.job[0];
    const MlpPath path = dh_path(M, D, F, act, &l);
    if (path == kMlpSwap) {
      st = static_cast<gbf_status_t>(lib_glu_grad(dout, w_down, g, u, ws.dg, ws.du, M, F, D, act, s));
    } else {
      if (!map_k(&j.a[0], dout, D, M) || !map_mn(&j.b[0], w_down, F, D) ||
          !map_out(&j.a[1], g, F, M, true) || !map_out(&j.b[1], u, F, M, true) ||
          !map_out(&j.o[0], ws.dg, F, M, true) || !map_out(&j.o[1], ws.du, F, M, true))
        return GBF_ERR_CUDA;
      st = run_launch(&l, path == kMlpPairTwo ? 2 : 1, *dev, err, s);
    }
    if (st != GBF_OK) return st;
  }
  MbLaunch l{};
  if (dx) {
    MbJob& j = l.job[0];
    set_dx(&j, M, D, F, splits);
    if (!map_k(&j.a[0], ws.dg, F, M) || !map_k(&j.a[1], ws.du, F, M) ||
        !map_mn(&j.b[0], w_gate, D, F) || !map_mn(&j.b[1], w_up, D, F) ||
        !(splits > 1 ? map_parts(&j.o[0], ws.dx, D, splits * mlp_m_pad(M))
                     : map_out(&j.o[0], dx, D, M, false)))
      return GBF_ERR_CUDA;
  }
  if ((dw_gate && !set_dw(&l.job[1], ws.dg, x, dw_gate, ws.dw_gate, F, D, M)) ||
      (dw_up && !set_dw(&l.job[2], ws.du, x, dw_up, ws.dw_up, F, D, M)) ||
      (dw_down && !set_dw(&l.job[3], dout, h, dw_down, ws.dw_down, D, F, M)))
    return GBF_ERR_CUDA;
  if ((st = run_launch(&l, streams, *dev, err, s)) != GBF_OK) return st;
  const float* parts[kMbJobs] = {ws.dx, ws.dw_gate, ws.dw_up, ws.dw_down};
  void* out[kMbJobs] = {dx, dw_gate, dw_up, dw_down};
  for (int i = 0; i < kMbJobs; ++i) {
    const MbJob& j = l.job[i];
    if (!out[i] || j.splits == 1) continue;
    const int64_t cols = j.cols;
    st = cuda_status(launch_mlp_sum(parts[i], static_cast<__nv_bfloat16*>(out[i]), j.rows * cols,
                                    j.m_pad * cols, j.splits, dev->sms, s));
    if (st != GBF_OK) return st;
  }
  return GBF_OK;
}

int gbf_debug_mlp_path(int64_t M, int64_t D, int64_t F, int grad, int64_t* units) {
  if (units) *units = 0;
  if (M == 0 || check_mlp(M, D, F, GBF_ACT_SILU) != GBF_OK) return -1;
  MbLaunch l{};
  const MlpPath path = grad ? dh_path(M, D, F, GBF_ACT_SILU, &l) : forward_path(M, D, F, GBF_ACT_SILU, &l);
  if (path == kMlpPairOne || path == kMlpPairTwo) {
    plan_mlp_launch(&l, path == kMlpPairTwo ? 2 : 1, kMlpPairs);
    if (units) *units = l.job[0].units + l.shorts;
  }
  return path;
}

gbf_status_t gbf_add_rmsnorm_grad(const void* dnorm, const void* dresid, const void* resid,
                                  const void* weight, void* dr, void* dweight, int64_t M,
                                  int64_t N, float eps, void* workspace, size_t workspace_bytes,
                                  gbf_stream_t stream) {
  if (M < 0 || N < 0 || !(eps >= 0.0f)) return GBF_ERR_INVALID_ARG;
  gbf_status_t st =
      M == 0 || N == 0
          ? check_all({}, {dnorm, dresid, resid, weight, dr, dweight, workspace})
          : check_all({dnorm, resid, weight, dr}, {dresid, dweight, workspace});
  if (st != GBF_OK) return st;
  if (N % 8 != 0 || N > kRmsMaxN || M > kMaxInt) return GBF_ERR_UNSUPPORTED_SHAPE;
  const size_t need = dweight ? gbf_workspace_size(GBF_OP_ADD_RMSNORM_GRAD, M, N, 0, 1) : 0;
  if (need && (!workspace || workspace_bytes < need)) return GBF_ERR_WORKSPACE;
  const DeviceInfo* dev;
  unsigned* err;
  if ((st = lib_device(&dev, &err)) != GBF_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (N == 0) return GBF_OK;
  if (M == 0)
    return dweight ? cuda_status(cudaMemsetAsync(dweight, 0, static_cast<size_t>(N) * 2, s)) : GBF_OK;
  return cuda_status(launch_add_rmsnorm_grad(
      static_cast<const __nv_bfloat16*>(dnorm), static_cast<const __nv_bfloat16*>(dresid),
      static_cast<const __nv_bfloat16*>(resid), static_cast<const __nv_bfloat16*>(weight),
      static_cast<__nv_bfloat16*>(dr), static_cast<__nv_bfloat16*>(dweight), M,
      static_cast<int>(N), eps, static_cast<float*>(workspace), std::min(dev->sms, kMaxSms), s));
}

}  // extern "C"
