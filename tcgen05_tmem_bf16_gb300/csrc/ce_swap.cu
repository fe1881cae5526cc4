// ce_swap.cu -- the logits of the linear cross entropy for up to 128 rows.
//
// With few rows the weight's bytes are the work: W is read once from HBM at a
// few operations per byte.  So the roles are swapped against linear_ce.cu's
// tiles: 128 rows of W (columns of the vocabulary) are the MMA's M, the rows of
// x, padded to 16, 64 or 128, its N; a stage of the ring is 16 KB of W and 2 to
// 16 KB of x (from L2).  Two CTAs per SM, each persistent over tiles, so that
// one CTA's ending and the other's loads overlap; every tile's K blocks begin at
// another place, so that the CTAs do not all ask for the same lines of x.
//
// A tile's K blocks are dealt to several accumulators, which the ending adds in
// fp32: shorter chains of additions on the tensor cores, which cut.  Where a chain
// would still be longer than kCeChain blocks, K is taken in segments, and the
// ending keeps the sums of those before the last in a buffer of the CTA's own (128
// rows x 32000 x 4096: 58 us with lse off by 4e-7 of itself, in one segment 51 us and
// twice that).
//
// Endings, a thread per column of the vocabulary:
//   LSE   the tile is transposed 16 rows at a time through shared memory; per
//         row and 32 columns one (maximum, sum of powers), and the target's logit;
//   GRAD  G transposed: gt[v][m], one contiguous row per thread.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "epilogue.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace gbf {

namespace {

constexpr int kSwThreads = 192;  // producer, MMA issuer, four warps of the ending
constexpr int kSwWBytes = 128 * kBK * 2;

template <int MPAD>
struct SwCfg {
  static constexpr int kXBytes = MPAD * kBK * 2;
  static constexpr int kStageBytes = kSwWBytes + kXBytes;
  static constexpr int kStages = MPAD == 16 ? 5 : MPAD == 64 ? 4 : 3;
  static constexpr int kAccs = MPAD == 16 ? 8 : MPAD == 64 ? 4 : 2;  // accumulators
  static constexpr int kTmemCols = MPAD * kAccs;  // 128 or 256: two CTAs fit
  // Accumulators of a tile: four, or two where that leaves another tile in
  // tensor memory and their chains are short enough (64 rows x 128000 x 2048: 99
  // us, with four 102).
  static __host__ __device__ constexpr int groups(int num_kb) {
    return MPAD == 64 && num_kb <= 2 * kCeChain ? 2 : kAccs < 4 ? kAccs : 4;
  }
  static constexpr int kBarBytes = 256;
  static constexpr int kRowBytes = 3 * MPAD * 4;            // lse2, dl, targets
  static constexpr int kTurnBytes = 4 * 32 * 17 * 4;        // transposition, per warp
  static constexpr int kSmem = 1024 + kStages * kStageBytes + kBarBytes + kRowBytes + kTurnBytes;
  static_assert(2 * (kSmem + 1024) <= 227 * 1024, "two CTAs per SM");
  static_assert(kStageBytes % 1024 == 0, "stages stay 1024-byte aligned");
};

__device__ __forceinline__ float sw_pow2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int MPAD, bool GRAD>
__global__ void __launch_bounds__(kSwThreads, 2)
    ce_swap_kernel(const __grid_constant__ CeSwap a, const CeEnd e, const KernelCtl kctl) {
  using Cfg = SwCfg<MPAD>;
  constexpr int kStages = Cfg::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint8_t* stages = smem;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kStages * Cfg::kStageBytes);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* done = tempty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(done + 1);
  int* abort_flag = reinterpret_cast<int*>(tmem_holder + 1);
  uint8_t* after = smem + kStages * Cfg::kStageBytes + Cfg::kBarBytes;
  float* row_lse2 = reinterpret_cast<float*>(after);
  float* row_dl = row_lse2 + MPAD;
  int* row_tgt = reinterpret_cast<int*>(row_dl + MPAD);
  float* turn = reinterpret_cast<float*>(after + Cfg::kRowBytes);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 4);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&a.w);
    tma_prefetch_desc(&a.x[0]);
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, Cfg::kTmemCols);
    tmem_relinquish();
  }
  if (threadIdx.x == 0) griddep_launch_dependents();
  griddep_wait();  // the gradient's scored rows are listed by the kernel before
  const int count = GRAD ? *e.count : e.M;
  for (int i = threadIdx.x; i < MPAD; i += kSwThreads) {
    if (GRAD) {
      row_tgt[i] = i < count ? e.tgt[i] - a.v0 : -1;
      row_lse2[i] = i < count ? e.lse2[i] : 0.0f;
      row_dl[i] = i < count ? e.dl[i] : 0.0f;
    } else {
      const int64_t t = i < count ? ce_target(a.targets, a.ids64, i) : -1;
      row_tgt[i] = t >= 0 && t < a.cols ? static_cast<int>(t) : -1;
    }
  }
  if (!GRAD && blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0u;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  const WaitCtl ctl{kctl.err, kctl.timeout_ns, abort_flag, prof_slots(kctl.prof)};
  const long long t_start = clock64();
  const int tiles = (a.cols + 127) / 128;
  const int num_kb = a.num_kb;
  const int per_tile = Cfg::groups(num_kb);
  const int two_bufs = Cfg::kAccs / per_tile == 2 ? 1 : 0;  // segments in tensor memory: 2 or 1
  const int seg_kb = per_tile * kCeChain;
  const int step = static_cast<int>(gridDim.x);

  if (warp == 0) {
    if (lane == 0) {
      asm volatile("fence.proxy.async;" ::: "memory");  // the gathered rows: plain stores
      const CUtensorMap* mx = &a.x[!GRAD || count == e.M ? 1 : 0];
      uint32_t fills[kStages];
#pragma unroll
      for (int i = 0; i < kStages; ++i) fills[i] = 0;
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < tiles && ok; t += step) {
        // by the column of W, so that both passes add in the same order
        int kb = static_cast<int>(static_cast<unsigned>(a.v0 / 128 + t) * 13u %
                                  static_cast<unsigned>(num_kb));
        for (int i = 0; i < num_kb; ++i) {
          if (!wait_bar(&empty[s], ph ^ 1, ctl, kSiteProducerEmpty)) {
            ok = false;
            break;
          }
          uint8_t* sw = stages + s * Cfg::kStageBytes;
          mbar_arrive_expect_tx(&full[s], Cfg::kStageBytes);
          tma_load_2d(sw, &a.w, &full[s], kb * kBK, a.v0 + t * 128);
          tma_load_2d(sw + kSwWBytes, mx, &full[s], kb * kBK, 0);
          fills[s]++;
          if (++s == kStages) {
            s = 0;
            ph ^= 1;
          }
          if (++kb == num_kb) kb = 0;
        }
      }
      if (ok) {
        for (int i = 0; i < kStages; ++i)
          if (fills[i]) wait_bar(&empty[i], (fills[i] - 1) & 1, ctl, kSiteDrain, false);
      } else {
        const uint64_t t0 = globaltimer_ns();  // let the copies in flight land (bounded)
        while (globaltimer_ns() - t0 < 2000000ull) __nanosleep(1000);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_bf16(128, MPAD, false, false);
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      int l = 0, seg = 0;
      for (int t = blockIdx.x; t < tiles && ok; ++l) {
        const int buf = l & two_bufs;
        const int use = l >> two_bufs;
        if (!wait_bar(&tempty[buf], (use & 1) ^ 1, ctl, kSiteMmaAccEmpty)) break;
        tc_fence_after();
        const int seg_end = min(seg + seg_kb, num_kb);
        for (int i = seg; i < seg_end; ++i) {
          if (!wait_bar(&full[s], ph, ctl, kSiteMmaFull)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t w0 = smem_u32(stages + s * Cfg::kStageBytes);
          const uint32_t x0 = w0 + kSwWBytes;
          const uint32_t d = tmem_base + (buf * per_tile + (i & (per_tile - 1))) * MPAD;
#pragma unroll
          for (int k = 0; k < kBK / 16; ++k)
            mma_ss(d, sdesc_sw128(w0 + k * 32, 16, 1024), sdesc_sw128(x0 + k * 32, 16, 1024),
                   idesc, (i - seg >= per_tile || k != 0) ? 1u : 0u);
          mma_commit(&empty[s]);
          if (++s == kStages) {
            s = 0;
            ph ^= 1;
          }
        }
        if (!ok) break;
        if (!(kctl.inject && l == 0)) mma_commit(&tfull[buf]);
        seg = seg_end;
        if (seg == num_kb) {
          seg = 0;
          t += step;
        }
      }
      mma_commit(done);
      wait_bar(done, 0, ctl, kSiteDrain, false);
    }
    __syncwarp();
  } else {
    const int q = warp & 3;  // the quarter of tensor memory that this warp reads
    float* my_turn = turn + q * 32 * 17;
    const int chunks = (count + 15) / 16;  // of 16 rows
    // sums of the segments before: [row][column], this thread's column
    float* part = e.chain + static_cast<int64_t>(blockIdx.x) * MPAD * 128 + q * 32 + lane;
    int seg = 0;
    for (int t = blockIdx.x, l = 0; t < tiles; ++l) {
      const int buf = l & two_bufs;
      float before[16];  // of the next 16 rows, on their way meanwhile
      if (seg > 0) {
#pragma unroll
        for (int k = 0; k < 16; ++k) before[k] = __ldcg(part + k * 128);
      }
      if (!wait_bar(&tfull[buf], (l >> two_bufs) & 1, ctl, kSiteEpiAccFull)) break;
      tc_fence_after();
      const int groups = min(per_tile, num_kb - seg);
      const bool last = seg + seg_kb >= num_kb;
      const uint32_t tb =
          tmem_base + buf * per_tile * MPAD + (static_cast<uint32_t>(q * 32) << 16);
      const int col = t * 128 + q * 32 + lane;  // of the piece
#pragma unroll 1
      for (int c = 0; c < MPAD / 16; ++c) {
        float v[16];
        if (c < chunks) {
          uint32_t r[16];
          tmem_ld16(tb + c * 16, r);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 16; ++k) v[k] = __uint_as_float(r[k]);
          for (int g = 1; g < groups; ++g) {
            tmem_ld16(tb + g * MPAD + c * 16, r);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] += __uint_as_float(r[k]);
          }
          if (seg > 0) {
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = before[k] + v[k];
            if (c + 1 < chunks) {
#pragma unroll
              for (int k = 0; k < 16; ++k) before[k] = __ldcg(part + ((c + 1) * 16 + k) * 128);
            }
          }
        }
        if (!last) {
          if (c < chunks) {
#pragma unroll
            for (int k = 0; k < 16; ++k) __stcg(part + (c * 16 + k) * 128, v[k]);
          }
        } else if (GRAD) {
          float f[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const int m = c * 16 + k;
            f[k] = 0.0f;
            if (m < count) {
              const float p = sw_pow2(fmaf(v[k], e.c2, -row_lse2[m]));
              f[k] = row_dl[m] * (row_tgt[m] == col ? p - 1.0f : p);
            }
          }
          if (col < a.cols) {
            __nv_bfloat16* dst = a.gt + static_cast<int64_t>(col) * MPAD + c * 16;
            float lo[8], hi[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              lo[k] = f[k];
              hi[k] = f[8 + k];
            }
            st_u4(dst, pack8(lo));
            st_u4(dst + 8, pack8(hi));
          }
        } else if (c < chunks) {
#pragma unroll
          for (int k = 0; k < 16; ++k) my_turn[lane * 17 + k] = v[k];
          __syncwarp();
          // lanes 0-15: the first 16 columns of row c * 16 + lane; 16-31: the others
          const int m = c * 16 + (lane & 15);
          const int first = (lane >> 4) * 16;
          const int base = t * 128 + q * 32;
          float x[16], top = -INFINITY;
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            x[k] = my_turn[(first + k) * 17 + (lane & 15)];
            if (base + first + k < a.cols) top = fmaxf(top, x[k] * e.c2);
          }
          const float ref = top == -INFINITY ? 0.0f : top;
          float sum = 0.0f;
#pragma unroll
          for (int k = 0; k < 16; ++k)  // one rounding less than x c2 - ref
            if (base + first + k < a.cols) sum += sw_pow2(fmaf(x[k], e.c2, -ref));
          const float top2 = __shfl_xor_sync(0xFFFFFFFFu, top, 16);
          const float sum2 = __shfl_xor_sync(0xFFFFFFFFu, sum, 16);
          const float m2 = fmaxf(top, top2);
          const float ref2 = m2 == -INFINITY ? 0.0f : m2;
          sum = fmaf(sum, sw_pow2(top - ref2), sum2 * sw_pow2(top2 - ref2));
          if (lane < 16 && m < count) {
            e.part[static_cast<int64_t>(4 * t + q) * e.M + m] = make_float2(m2, sum);
            const int at = row_tgt[m] - base;
            if (row_tgt[m] >= 0 && at >= 0 && at < 32) e.tlog[m] = my_turn[at * 17 + lane];
          }
          __syncwarp();
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[buf]);
      seg += seg_kb;
      if (last) {
        seg = 0;
        t += step;
      }
    }
  }

  if (ctl.prof && threadIdx.x == 0)
    atomicAdd(&ctl.prof[31], static_cast<unsigned long long>(clock64() - t_start));
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, Cfg::kTmemCols);
  }
}

template <int MPAD, bool GRAD>
cudaError_t run_swap(const CeSwap& a, const CeEnd& end, const KernelCtl& ctl, int grid,
                     cudaStream_t stream) {
  static std::atomic<uint64_t> mask{0};
  auto kernel = ce_swap_kernel<MPAD, GRAD>;
  constexpr int smem = SwCfg<MPAD>::kSmem;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (!(mask.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    mask.fetch_or(bit, std::memory_order_acq_rel);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(kSwThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, end, ctl);
}

}  // namespace

int ce_swap_rows(int64_t M) { return M <= 16 ? 16 : M <= 64 ? 64 : M <= kCeSwapMax ? 128 : 0; }

int ce_swap_segments(int64_t M, int k_blocks) {
  const int n = M <= 16   ? SwCfg<16>::groups(k_blocks)
                : M <= 64 ? SwCfg<64>::groups(k_blocks)
                          : SwCfg<128>::groups(k_blocks);
  return (k_blocks + n * kCeChain - 1) / (n * kCeChain);
}

cudaError_t launch_ce_swap(const CeSwap& a, bool grad, const CeEnd& end, int sms,
                           const KernelCtl& ctl, cudaStream_t stream) {
  const int grid = std::min((a.cols + 127) / 128, 2 * sms);
  switch (ce_swap_rows(end.M)) {
    case 16: return grad ? run_swap<16, true>(a, end, ctl, grid, stream)
                         : run_swap<16, false>(a, end, ctl, grid, stream);
    case 64: return grad ? run_swap<64, true>(a, end, ctl, grid, stream)
                         : run_swap<64, false>(a, end, ctl, grid, stream);
    case 128: return grad ? run_swap<128, true>(a, end, ctl, grid, stream)
                          : run_swap<128, false>(a, end, ctl, grid, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace gbf
