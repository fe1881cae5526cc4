// pair_end.cuh -- parts of the endings of the CTA-pair product kernels beside
// gemm_pair.cu (linear_ce.cu, mlp_train.cu): a warp's chunk of a tile to global
// memory, and the return of an accumulator to the issuers.
#pragma once

#include <cstdint>
#include <cuda.h>

#include "common.cuh"
#include "epilogue.cuh"
#include "ptx.cuh"

namespace gbf {

// One warp's 32 rows x 32 columns of fp32 to the map's tensor, stored or added
// there by the TMA engine, through the warp's two staging buffers (16 columns
// each).  Every element is added to by one warp of one launch, so the sums do
// not depend on timing.
__device__ __forceinline__ void put_chunk_f32(uint8_t* bufs, int buf_bytes, int& flip,
                                              const uint32_t (&v)[32], const CUtensorMap* map,
                                              int row0, int col0, int n, bool some, bool add) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint8_t* buf = bufs + flip * buf_bytes;
    if (lane == 0) bulk_wait_read<1>();
    __syncwarp();
    uint32_t w[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) w[j] = v[16 * h + j];
    stage_row32(buf, lane, w);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      if (some && col0 + 16 * h < n) {
        if (add) tma_add_2d(map, buf, col0 + 16 * h, row0);
        else tma_store_2d(map, buf, col0 + 16 * h, row0, policy_evict_last());
      }
      bulk_commit();
    }
    flip ^= 1;
  }
}

// One warp's 32 rows x 32 bf16 columns through a staging buffer to the map's
// tensor, as store_chunk32 does; WIDE: two calls with c even and odd fill rows
// of 128 bytes (128-byte swizzle), which the second one stores.
template <bool WIDE>
__device__ __forceinline__ void put_chunk(uint8_t* bufs, int buf_bytes, int& flip, int c,
                                          const uint32_t (&w)[16], const CUtensorMap* map,
                                          int row0, int col0, int rows, int n, uint64_t pol) {
  const int lane = threadIdx.x & 31;
  uint8_t* buf = bufs + flip * buf_bytes;
  const bool first = !WIDE || (c & 1) == 0, last = !WIDE || (c & 1) == 1;
  if (first) {
    if (lane == 0) bulk_wait_read<1>();
    __syncwarp();
  }
  if (WIDE) {
    const uint32_t base = smem_u32(buf) + static_cast<uint32_t>(lane) * 128u;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t at = static_cast<uint32_t>((4 * (c & 1) + u) ^ (lane & 7)) << 4;
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(base + at), "r"(w[4 * u]),
                   "r"(w[4 * u + 1]), "r"(w[4 * u + 2]), "r"(w[4 * u + 3])
                   : "memory");
    }
  } else {
    stage_row32(buf, lane, w);
  }
  if (last) {
    const int at = WIDE ? col0 - 32 : col0;
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      if (row0 < rows && at < n) tma_store_2d(map, buf, at, row0, pol);
      bulk_commit();
    }
    flip ^= 1;
  }
}

// Eight columns of a product whose K was taken in n parts: at(i) is part i's address,
// f the sums in the parts' order.  Loads of four parts are in flight at a time.
template <typename At>
__device__ __forceinline__ void add_parts(float (&f)[8], int n, const At& at) {
#pragma unroll
  for (int k = 0; k < 8; ++k) f[k] = 0.0f;
  for (int i0 = 0; i0 < n; i0 += 4) {
    float4 x[4], y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i0 + i >= n) break;
      const float4* src = reinterpret_cast<const float4*>(at(i0 + i));
      x[i] = __ldcs(src);
      y[i] = __ldcs(src + 1);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i0 + i >= n) break;
      f[0] += x[i].x; f[1] += x[i].y; f[2] += x[i].z; f[3] += x[i].w;
      f[4] += y[i].x; f[5] += y[i].y; f[6] += y[i].z; f[7] += y[i].w;
    }
  }
}

// How a warp of the ending gives an accumulator back to the issuers.  What is handed
// over is tensor memory: its loads have completed (tcgen05.wait::ld) and are ordered by
// the fence, and no thread reads memory that the warp wrote because of this arrival.
// So the odd CTA's is relaxed: one that releases at the cluster's scope waits for the
// warp's stores in flight, the TMA engine's among them, and the next products wait for
// it (weights' gradients of 16 rows, 352 MB: 75 us, relaxed 53).
struct AccFree {
  uint64_t* mine;
  uint32_t lead;  // the even CTA's, as the odd one sees it
  bool leader;
  __device__ __forceinline__ void operator()() const {
    tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) {
      if (leader)
        mbar_arrive(mine);
      else
        asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(lead)
                     : "memory");
    }
  }
};

}  // namespace gbf
