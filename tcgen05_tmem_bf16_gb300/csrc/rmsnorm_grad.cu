// rmsnorm_grad.cu -- the gradient of the fused residual add + RMSNorm.
//
// Per row, with s = rsqrt(mean(r^2) + eps) and n = r s w the forward's result:
//   dr = dresid + s (dn w - r s^2 mean(dn w r))
//   dweight = sum over the rows of dn r s
// Both row sums, of r^2 and of dn w r, are taken in one pass over the row, which
// stays on the SM; so r, dn and dresid are read once and dr is written once.
//
// HBM-bound.  A CTA takes rows in turn, short ones several at a time, and loads its next
// before it reduces the present ones.  A thread holds the same columns of every row, so dweight's
// sums stay in its registers in fp32 and leave the CTA once, as one row of
// partial sums; a second kernel adds those rows in their order (the same bits on
// every run).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace gbf {

namespace {

// ROW threads hold R 16-byte vectors each of a row: all T of a CTA, or fewer, which take
// rows of their own; PER_SM CTAs at a time.  STAGED: a thread keeps its vectors of the
// present row in shared memory, where it alone reads them, and only the next row's in
// registers.
template <int T, int ROW, int R, int PER_SM, bool STAGED>
__global__ void __launch_bounds__(T, PER_SM)
    rmsnorm_grad_kernel(const __nv_bfloat16* dnorm, const __nv_bfloat16* dresid,
                        const __nv_bfloat16* r, const __nv_bfloat16* w,
                        __nv_bfloat16* dr, float* __restrict__ partial, int64_t M, int N,
                        float eps) {
  constexpr int kRows = T / ROW;  // at a time
  constexpr int kWarps = ROW / 32;
  __shared__ float2 sums[2][T / 32];
  __shared__ float rows_acc[kRows > 1 ? kRows : 1][kRows > 1 ? ROW * R * 8 : 1];
  extern __shared__ uint4 staged[];  // STAGED: [3][R][T]
  griddep_launch_dependents();
  griddep_wait();
  const uint64_t pol = l2_evict_first_policy();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int place = threadIdx.x % ROW, mine = threadIdx.x / ROW;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kRows + mine;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  constexpr int kHeld = STAGED ? 1 : R;
  uint4 wv[R], vr[R], vn[R], vd[R];
  float acc[R][8];
#pragma unroll
  for (int v = 0; v < R; ++v) {
    const int col = (place + v * ROW) * 8;
    // (a plain load: the kernel before may still have been writing w when this one began)
    wv[v] = col < N ? ld_u4(w + col) : zero;
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[v][i] = 0.0f;
  }
  auto slot = [&](int k, int v) { return &staged[(k * R + v) * T + threadIdx.x]; };
  auto load_row = [&](int64_t row) {
#pragma unroll
    for (int v = 0; v < R; ++v) {
      const int col = (place + v * ROW) * 8;
      const bool ok = col < N && row < M;
      const int64_t at = row * N + col;
      vr[v] = ok ? ld_stream_u4(r + at, pol) : zero;
      vn[v] = ok ? ld_stream_u4(dnorm + at, pol) : zero;
      vd[v] = ok && dresid ? ld_stream_u4(dresid + at, pol) : zero;
    }
  };
  load_row(row0);
  int flip = 0;
  for (int64_t row = row0; row < M; row += step, flip ^= 1) {
    float ss = 0.0f, t = 0.0f;
    uint4 cr[kHeld], cn[kHeld], cd[kHeld];
#pragma unroll
    for (int v = 0; v < R; ++v) {
      if constexpr (STAGED) {
        *slot(0, v) = vr[v];
        *slot(1, v) = vn[v];
        *slot(2, v) = vd[v];
      } else {
        cr[v] = vr[v];
        cn[v] = vn[v];
        cd[v] = vd[v];
      }
    }
    if constexpr (STAGED) load_row(row + step);
#pragma unroll
    for (int v = 0; v < R; ++v) {
      float a[8], b[8], c[8];
      unpack8(STAGED ? *slot(0, v) : cr[v % kHeld], a);
      unpack8(STAGED ? *slot(1, v) : cn[v % kHeld], b);
      unpack8(wv[v], c);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ss = fmaf(a[i], a[i], ss);
        t = fmaf(b[i] * c[i], a[i], t);
      }
    }
    if constexpr (!STAGED) load_row(row + step);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
      t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
    }
    if constexpr (ROW > 32) {
      if (lane == 0) sums[flip][warp] = make_float2(ss, t);
      // one barrier of the row's threads: the other buffer is free once all have passed it
      if constexpr (kRows == 1) __syncthreads();
      else asm volatile("bar.sync %0, %1;" ::"r"(1 + mine), "n"(ROW) : "memory");
      ss = t = 0.0f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        ss += sums[flip][mine * kWarps + i].x;
        t += sums[flip][mine * kWarps + i].y;
      }
    }
    const float s = rsqrtf(ss / static_cast<float>(N) + eps);
    // one s at a time: s^2 leaves fp32 where the values are below 5e-20
    const float k = s * (s * (t / static_cast<float>(N)));
#pragma unroll
    for (int v = 0; v < R; ++v) {
      const int col = (place + v * ROW) * 8;
      float a[8], b[8], c[8], d[8];
      unpack8(STAGED ? *slot(0, v) : cr[v % kHeld], a);
      unpack8(STAGED ? *slot(1, v) : cn[v % kHeld], b);
      unpack8(wv[v], c);
      unpack8(STAGED ? *slot(2, v) : cd[v % kHeld], d);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        acc[v][i] = fmaf(b[i], a[i] * s, acc[v][i]);
        d[i] = fmaf(s, fmaf(-a[i], k, b[i] * c[i]), d[i]);
      }
      if (col < N) st_stream_u4(dr + row * N + col, pack8(d), pol);
    }
  }
  if (!partial) return;
  if constexpr (kRows > 1) {  // the rows' sums, in their order
#pragma unroll
    for (int v = 0; v < R; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) rows_acc[mine][(place + v * ROW) * 8 + i] = acc[v][i];
    __syncthreads();
    for (int col = threadIdx.x; col < N; col += T) {
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < kRows; ++i) sum += rows_acc[i][col];
      partial[static_cast<int64_t>(blockIdx.x) * N + col] = sum;
    }
    return;
  }
#pragma unroll
  for (int v = 0; v < R; ++v) {
    const int col = (place + v * ROW) * 8;
    if (col >= N) continue;
    float4* dst = reinterpret_cast<float4*>(partial + static_cast<int64_t>(blockIdx.x) * N + col);
    dst[0] = make_float4(acc[v][0], acc[v][1], acc[v][2], acc[v][3]);
    dst[1] = make_float4(acc[v][4], acc[v][5], acc[v][6], acc[v][7]);
  }
}

// dweight: 32 columns per CTA, whose warps share out the rows of partial sums.
constexpr int kJoinWarps = 16;
__global__ void __launch_bounds__(kJoinWarps * 32)
    rmsnorm_grad_join_kernel(const float* __restrict__ partial, __nv_bfloat16* __restrict__ dweight,
                             int rows, int N) {
  __shared__ float part[kJoinWarps][32];
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col = blockIdx.x * 32 + lane;
  float sum = 0.0f;
  if (col < N) {
#pragma unroll 8
    for (int i = warp; i < rows; i += kJoinWarps)
      sum += __ldcg(partial + static_cast<int64_t>(i) * N + col);
  }
  part[warp][lane] = sum;
  __syncthreads();
  if (warp != 0 || col >= N) return;
  sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kJoinWarps; ++i) sum += part[i][lane];
  dweight[col] = __float2bfloat16_rn(sum);
}

// 512 threads per SM, of up to 128 registers each, with two vectors of three rows per
// thread on their way, 48 KB per SM: short rows are taken several at a time (20000 x 1000:
// 31.7 us, one per CTA of 128 threads 37.7; 100000 x 256 48, 121).  Four vectors, for rows of
// more than 8192 values, find no room in registers (2000 x 16384: 96 us, staged 48.7).
int rms_grad_threads(int N) { return N <= 4096 ? 256 : 512; }
int rms_grad_rows(int N) { return N <= 512 ? 8 : N <= 1024 ? 4 : N <= 2048 ? 2 : 1; }

template <int T, int ROW, int R, bool STAGED>
cudaError_t run_rms_grad(const __nv_bfloat16* dnorm, const __nv_bfloat16* dresid,
                         const __nv_bfloat16* r, const __nv_bfloat16* weight, __nv_bfloat16* dr,
                         float* partial, int64_t M, int N, float eps, int grid,
                         cudaStream_t stream) {
  auto kernel = rmsnorm_grad_kernel<T, ROW, R, 512 / T, STAGED>;
  constexpr int smem = STAGED ? 3 * R * T * 16 : 0;
  if constexpr (STAGED) {
    static std::atomic<uint64_t> mask{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (!(mask.load(std::memory_order_acquire) & bit)) {
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e != cudaSuccess) return e;
      mask.fetch_or(bit, std::memory_order_acq_rel);
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(T, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, dnorm, dresid, r, weight, dr, partial, M, N, eps);
}

}  // namespace

int rms_grad_sums(int64_t M, int N, int sms) {
  return static_cast<int>(std::min<int64_t>(M, static_cast<int64_t>(sms) * (512 / rms_grad_threads(N))));
}

cudaError_t launch_add_rmsnorm_grad(const __nv_bfloat16* dnorm, const __nv_bfloat16* dresid,
                                    const __nv_bfloat16* r, const __nv_bfloat16* weight,
                                    __nv_bfloat16* dr, __nv_bfloat16* dweight, int64_t M, int N,
                                    float eps, float* partial, int sms, cudaStream_t stream) {
  const int rows = rms_grad_rows(N);
  const int grid = rms_grad_sums((M + rows - 1) / rows, N, sms);
  float* p = dweight ? partial : nullptr;
  cudaError_t e;
  if (N <= 512) e = run_rms_grad<256, 32, 2, false>(dnorm, dresid, r, weight, dr, p, M, N, eps, grid, stream);
  else if (N <= 1024) e = run_rms_grad<256, 64, 2, false>(dnorm, dresid, r, weight, dr, p, M, N, eps, grid, stream);
  else if (N <= 2048) e = run_rms_grad<256, 128, 2, false>(dnorm, dresid, r, weight, dr, p, M, N, eps, grid, stream);
  else if (N <= 4096) e = run_rms_grad<256, 256, 2, false>(dnorm, dresid, r, weight, dr, p, M, N, eps, grid, stream);
  else if (N <= 8192) e = run_rms_grad<512, 512, 2, false>(dnorm, dresid, r, weight, dr, p, M, N, eps, grid, stream);
  else e = run_rms_grad<512, 512, 4, true>(dnorm, dresid, r, weight, dr, p, M, N, eps, grid, stream);
  if (e != cudaSuccess || !dweight) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((N + 31) / 32), 1, 1);
  cfg.blockDim = dim3(kJoinWarps * 32, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rmsnorm_grad_join_kernel, static_cast<const float*>(partial),
                            dweight, grid, N);
}

}  // namespace gbf
