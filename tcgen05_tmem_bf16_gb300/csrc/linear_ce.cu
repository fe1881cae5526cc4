// linear_ce.cu -- softmax cross entropy of a linear head over a large
// vocabulary, without the logits in memory, and its gradients.
//
//   l[m][v] = alpha * sum_d x[m][d] w[v][d]
//   lse[m] = log sum_v exp(l[m][v]),   loss[m] = lse[m] - l[m][t_m]
//   G[m][v] = dloss[m] * (exp(l[m][v] - lse[m]) - [v = t_m])
//   dx = alpha * scale * G W,   dw = alpha * scale * G^T X
//
// One matrix-product kernel (ce_gemm_kernel) with four endings does the work.
// Its main loop is the CTA-pair form of gemm_pair.cu: 256 x 256 tiles on two
// SMs (tcgen05.mma.cta_group::2), TMA-fed, one or two MMA streams.
//   kLse    the logits' tile ends as one (maximum, sum of powers) per row and
//           128 columns, and the target's logit: 8 bytes for 128 logits;
//   kGrad   the logits again, ending as G in bf16 for a piece of the
//           vocabulary;
//   kDx     G W over the piece, added to an fp32 buffer;
//   kDw     G^T X, the rows of dw of the piece, complete: written once.
// Bound by the tensor pipe (8192 x 65536 x 4096: loss and gradients, four
// products, 10.7 ms, 1.64 PFLOP/s under the power cap; 1024 rows x 128000 x 4096
// scored in 612 us, 1.76 PFLOP/s), below some 500 rows by W's bytes.
// Rows whose target is outside [0, V) are not scored: they take part in
// nothing.  ce_prep_kernel gathers the scored rows' x when there are others,
// so masked prompts cost no products, and whatever their rows of x hold (NaN
// included) reaches no result.
//
// G is rounded to bf16 without the mean's factor: the factor multiplies the
// fp32 sums, so it adds no rounding of its own.
//
// The sums of the products are the tensor cores' fp32, whose additions cut instead
// of rounding: one chain over all of K loses 1e-9 K of a logit, and up to 4e-9 K
// where its products have one sign (lse off by 1.5e-6 of itself at K = 4096, 6e-5
// at 65536).  So a logit's K is taken in chains of kCeChain blocks, whose sums the
// ending adds in fp32 (lse off by 3 to 4e-7 at any K).  Up to 1024 products one
// chain is enough, and the logits are tiles of two row tiles like the others.  Above
// that they run in units of one row tile (kCeChains), because a thread of the
// ending then holds its 128 sums in registers and one accumulator is emptied
// while the other is filled.  (Forward pass, 8192 x 65536 x 4096: 2.68 ms, one
// chain with two row tiles 2.47; 1024 x 128000 x 4096 612 and 593 us; 2868 x
// 50001 x 2048 388 and 397.  The sums of two row tiles do not fit in registers:
// kept in L2, 3.42 ms.)  Both passes cut K at the same places: the backward
// pass's powers then add up to the forward's sum, and a confident row's p - 1
// holds no error of the products.
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

constexpr float kLog2e = 1.4426950408889634f;
constexpr double kLn2 = 0.69314718055994531;

__device__ __forceinline__ float pow2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr int kCeThreads = 384;        // warps 0-3 roles, 4-11 ending
constexpr int kCeTile = 256;           // rows and columns of a pair's tile
constexpr int kCeABytes = kBM * kBK * 2;   // 16 KB: this CTA's 128 rows of A
constexpr int kCeBBytes = 128 * kBK * 2;   // 16 KB: this CTA's half of B
constexpr int kCeGroup = 8;            // raster group (units of rows)
constexpr int kCeUnitCost = 4;         // a unit's ending, in K blocks of its main loop

// Two row tiles per unit, a lone one, or a lone one of logits in chains.
enum CeForm { kCeTwo, kCeLone, kCeChains };

template <int FORM>
struct CeCfg {
  static constexpr int kStreams = FORM == kCeTwo ? 2 : 1;
  static constexpr int kStageBytes = kStreams * kCeABytes + kCeBBytes;
  static constexpr int kStages = FORM == kCeTwo ? 4 : FORM == kCeLone ? 5 : 6;
  static constexpr int kBarBytes = 1024;
  // Two staging buffers per warp of the ending, of 32 rows x 64 bytes.  Few rows
  // of x make dw a matter of writing: there the rows are 128 bytes.  (Stores of
  // 128 x 256 tiles of a 32000 x 4096 tensor, by bytes of a row per request: 16:
  // 97 us, 32: 58, 256: 41, a plain fill 38.)
  static constexpr bool kWide = FORM == kCeLone;
  static constexpr int kBufBytes = kWide ? 32 * 128 : 32 * 64;
  static constexpr int kStagingBytes = 8 * 2 * kBufBytes;
  static constexpr int kSmem = 1024 + kStages * kStageBytes + kBarBytes + kStagingBytes;
  static_assert(kSmem <= 227 * 1024, "shared memory per CTA");
};

// A unit of work: STREAMS row tiles x one column tile x a range of K blocks of
// one of the launch's products.
struct CeUnit {
  int job, mp, nb, split, kb0, kb1;
};

// What a launch's products come to on the device, where the number of scored
// rows is known, and which units a CTA pair works through, in order.
//
// The products for dx (job 0) have few, long units, the others many short
// ones.  The long units are dealt out first, one per pair and round; the pairs
// that got one more than the others (the first `extra`) then sit out `skip`
// rounds of short units, about as many as the long one takes.  Every role of a
// pair computes the same sequence for itself: no shared queue.
struct CeWork {
  int units[kCeJobs], m_units[kCeJobs], n_tiles[kCeJobs], num_kb[kCeJobs];
  int longs, extra, skip, shorts, npairs;
};

__device__ __forceinline__ CeWork ce_work(const CeLaunch& a, int count, int streams, int npairs) {
  CeWork w;
  int64_t blocks = 0;
#pragma unroll
  for (int i = 0; i < kCeJobs; ++i) {
    w.units[i] = w.m_units[i] = w.n_tiles[i] = w.num_kb[i] = 0;
    if (a.job[i].mode == kCeNone) continue;
    const CeJob& j = a.job[i];
    const int rows = j.mode == kCeDw ? j.cols : count;
    const int n = (j.mode == kCeLse || j.mode == kCeGrad) ? j.cols : a.d;
    const int k = j.mode == kCeDw ? count : (j.mode == kCeDx ? j.cols : a.d);
    w.m_units[i] = (rows + kCeTile * streams - 1) / (kCeTile * streams);
    w.n_tiles[i] = (n + j.bn - 1) / j.bn;
    w.num_kb[i] = (k + kBK - 1) / kBK;
    w.units[i] = w.m_units[i] * w.n_tiles[i] * j.splits;
    if (i > 0) blocks += static_cast<int64_t>(w.units[i]) * (w.num_kb[i] + kCeUnitCost);
  }
  w.npairs = npairs;
  w.longs = w.units[0];
  w.shorts = w.units[1] + w.units[2];
  w.extra = w.longs % npairs;
  w.skip = 0;
  if (w.extra > 0 && w.shorts > 0) {
    const int64_t len = w.num_kb[0] / a.job[0].splits + kCeUnitCost;
    const int64_t fit = static_cast<int64_t>(w.shorts) / (npairs - w.extra) + 1;
    w.skip = static_cast<int>(min(len * w.shorts / max(blocks, static_cast<int64_t>(1)), fit));
  }
  return w;
}

// The n-th unit of a pair; false after its last.
__device__ __forceinline__ bool ce_unit(const CeWork& w, const CeLaunch& a, int pair, int n,
                                        CeUnit& u) {
  const int mine = w.longs / w.npairs + (pair < w.extra ? 1 : 0);
  int t;
  if (n < mine) {
    t = n * w.npairs + pair;
    u.job = 0;
  } else {
    const int round = n - mine + (pair < w.extra ? w.skip : 0);
    if (round < w.skip)
      t = round * (w.npairs - w.extra) + pair - w.extra;
    else
      t = w.skip * (w.npairs - w.extra) + (round - w.skip) * w.npairs + pair;
    if (t >= w.shorts) return false;
    u.job = 1;
    if (t >= w.units[1]) {
      u.job = 2;
      t -= w.units[1];
    }
  }
  const int m_units = u.job == 0 ? w.m_units[0] : u.job == 1 ? w.m_units[1] : w.m_units[2];
  const int n_tiles = u.job == 0 ? w.n_tiles[0] : u.job == 1 ? w.n_tiles[1] : w.n_tiles[2];
  const int num_kb = u.job == 0 ? w.num_kb[0] : u.job == 1 ? w.num_kb[1] : w.num_kb[2];
  u.split = 0;
  u.kb0 = 0;
  u.kb1 = num_kb;
  if (u.job == 0) {  // the only product whose K is split; at most 16 parts of 2^20 blocks
    const unsigned splits = a.job[0].splits;
    const unsigned tiles = m_units * n_tiles;
    u.split = static_cast<unsigned>(t) / tiles;
    t -= u.split * tiles;
    u.kb0 = static_cast<unsigned>(u.split * num_kb) / splits;
    u.kb1 = static_cast<unsigned>((u.split + 1) * num_kb) / splits;
  }
  tile_coords(t, m_units, n_tiles, u.mp, u.nb, kCeGroup);
  return true;
}

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

// How a warp of the ending gives an accumulator back to the issuers.
struct CeFree {
  uint64_t* mine;
  uint32_t lead;  // the even CTA's, as the odd one sees it
  bool leader;
  __device__ __forceinline__ void operator()() const {
    tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) {
      if (leader) mbar_arrive(mine);
      else mbar_arrive_cluster(lead);
    }
  }
};

// A warp's 128 columns of an accumulator, which is then given back.
__device__ __forceinline__ void ce_read(uint32_t tb, const CeFree& release,
                                        uint32_t (&v)[4][32]) {
#pragma unroll
  for (int c = 0; c < 4; ++c) tmem_ld32(tb + 32 * c, v[c]);
  tmem_wait_ld();
  release();
}
// The same, added to v.
__device__ __forceinline__ void ce_add(uint32_t tb, const CeFree& release,
                                       uint32_t (&v)[4][32]) {
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    uint32_t o[16];
    tmem_ld16(tb + 16 * c, o);
    tmem_wait_ld();
    if (c == 7) release();
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      uint32_t& x = v[c / 2][16 * (c & 1) + k];
      x = __float_as_uint(__uint_as_float(x) + __uint_as_float(o[k]));
    }
  }
}

// What the ending of a tile needs: a thread holds one row, a warp 128 columns
// from col0 on.
struct CeTileArgs {
  const CUtensorMap* out;
  uint8_t* staging;
  uint64_t pol;
  int row, col0, cols, v0, d, count;
  int buf_row;  // kDx: row in the fp32 buffers
  bool row_ok, none, add;
  int tgt;      // the target's column, from col0 on
  float lse2, dl, out_scale;
};

template <int MODE, int FORM>
__device__ __forceinline__ void ce_chunk(int c, const uint32_t (&v)[32], const CeTileArgs& t,
                                         const CeEnd& e, int& flip, float& m, float& sum) {
  constexpr int kBuf = CeCfg<FORM>::kBufBytes;
  const int col0 = t.col0 + c * 32;
  const int row0 = t.row - static_cast<int>(threadIdx.x & 31);
  if constexpr (MODE == kCeLse) {
    if (col0 < t.cols) {
      if (static_cast<unsigned>(t.tgt - c * 32) < 32u) {
#pragma unroll
        for (int k = 0; k < 32; ++k)
          if (t.tgt - c * 32 == k) e.tlog[t.row] = __uint_as_float(v[k]);
      }
      float top = -INFINITY, add = 0.0f;
      if (col0 + 32 <= t.cols) {
        // the largest scaled value is the scaled largest (smallest) one
        float ext = __uint_as_float(v[0]);
        if (e.c2 >= 0.0f) {
#pragma unroll
          for (int k = 1; k < 32; ++k) ext = fmaxf(ext, __uint_as_float(v[k]));
        } else {
#pragma unroll
          for (int k = 1; k < 32; ++k) ext = fminf(ext, __uint_as_float(v[k]));
        }
        top = ext * e.c2;
      } else {
#pragma unroll
        for (int k = 0; k < 32; ++k)
          if (col0 + k < t.cols) top = fmaxf(top, __uint_as_float(v[k]) * e.c2);
      }
      const float m2 = fmaxf(m, top);
      const float ref = m2 == -INFINITY ? 0.0f : m2;  // no -inf - -inf
      if (col0 + 32 <= t.cols) {
#pragma unroll
        for (int k = 0; k < 32; ++k) add += pow2(fmaf(__uint_as_float(v[k]), e.c2, -ref));
      } else {
#pragma unroll
        for (int k = 0; k < 32; ++k)
          if (col0 + k < t.cols) add += pow2(fmaf(__uint_as_float(v[k]), e.c2, -ref));
      }
      sum = fmaf(sum, pow2(m - ref), add);
      m = m2;
    }
  } else if constexpr (MODE == kCeDx) {
    uint32_t w[32];
#pragma unroll
    for (int k = 0; k < 32; ++k) w[k] = t.none ? 0u : v[k];
    put_chunk_f32(t.staging, kBuf, flip, w, t.out, t.buf_row - t.row + row0, col0, t.d,
                  row0 < t.count, t.add);
  } else {
    uint32_t w[16];
    if constexpr (MODE == kCeGrad) {
      float g[32];
#pragma unroll
      for (int k = 0; k < 32; ++k) g[k] = pow2(fmaf(__uint_as_float(v[k]), e.c2, -t.lse2));
      if (static_cast<unsigned>(t.tgt - c * 32) < 32u) {
#pragma unroll
        for (int k = 0; k < 32; ++k)
          g[k] += t.tgt - c * 32 == k ? -1.0f : 0.0f;
      }
#pragma unroll
      for (int k = 0; k < 16; ++k)  // zeros in the rows up to a full K block of kDw
        w[k] = t.row_ok ? pack_bf16x2(t.dl * g[2 * k], t.dl * g[2 * k + 1]) : 0u;
    } else {
#pragma unroll
      for (int k = 0; k < 16; ++k)
        w[k] = t.none ? 0u  // no rows: an empty sum
                      : pack_bf16x2(__uint_as_float(v[2 * k]) * t.out_scale,
                                    __uint_as_float(v[2 * k + 1]) * t.out_scale);
    }
    if constexpr (MODE == kCeGrad)
      put_chunk<false>(t.staging, kBuf, flip, c, w, t.out, row0, col0, e.M, t.cols, t.pol);
    else
      put_chunk<CeCfg<FORM>::kWide>(t.staging, kBuf, flip, c, w, t.out, t.v0 + row0, col0,
                              t.v0 + t.cols, t.d, t.pol);
  }
}

// A warp's 128 columns, 32 at a time: the next are on their way from tensor
// memory while the ending works on the present ones; the accumulator is free
// once the last have arrived.
template <int MODE, int FORM>
__device__ __forceinline__ void ce_tile(uint32_t tb, const CeFree& release, const CeTileArgs& t,
                                        const CeEnd& e, int& flip, float& m, float& sum) {
  uint32_t va[32], vb[32];
  tmem_ld32(tb, va);
  tmem_wait_ld();
  tmem_ld32(tb + 32, vb);
  ce_chunk<MODE, FORM>(0, va, t, e, flip, m, sum);
  tmem_wait_ld();
  tmem_ld32(tb + 64, va);
  ce_chunk<MODE, FORM>(1, vb, t, e, flip, m, sum);
  tmem_wait_ld();
  tmem_ld32(tb + 96, vb);
  ce_chunk<MODE, FORM>(2, va, t, e, flip, m, sum);
  tmem_wait_ld();
  release();
  ce_chunk<MODE, FORM>(3, vb, t, e, flip, m, sum);
}

template <int FORM>
__global__ void __launch_bounds__(kCeThreads, 1)
    ce_gemm_kernel(const __grid_constant__ CeLaunch a, const CeEnd e, const KernelCtl kctl) {
  using Cfg = CeCfg<FORM>;
  constexpr int STREAMS = Cfg::kStreams;
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
  uint8_t* staging = smem + kStages * Cfg::kStageBytes + Cfg::kBarBytes;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();  // 0: the even CTA, which issues the MMAs
  const bool leader = rank == 0;
  const int pair = static_cast<int>(blockIdx.x >> 1);
  const int npairs = static_cast<int>(gridDim.x >> 1);

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], STREAMS);  // every issuer
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 16);  // 8 warps in each CTA of the pair
    }
    mbar_init(done, STREAMS);
    *abort_flag = 0;
    fence_mbar_init();
    for (int i = 0; i < kCeJobs; ++i) {
      if (a.job[i].mode == kCeNone) continue;
      tma_prefetch_desc(&a.job[i].a[0]);
      tma_prefetch_desc(&a.job[i].b[0]);
      if (a.job[i].mode != kCeLse) tma_prefetch_desc(&a.job[i].o);
    }
  }
  if (warp == 2) {
    tmem_alloc_pair(tmem_holder, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  const WaitCtl ctl{kctl.err, kctl.timeout_ns, abort_flag, prof_slots(kctl.prof)};
  const long long t_start = clock64();
  if (threadIdx.x == 0) griddep_launch_dependents();
  // the number of scored rows is an output of the kernel before
  griddep_wait();
  const int count = *e.count;
  const int all = count == e.M ? 1 : 0;  // every row is scored: x itself, not the gathered rows
  const CeWork work = ce_work(a, count, STREAMS, npairs);

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer (both CTAs)
    if (lane == 0) {
      asm volatile("fence.proxy.async;" ::: "memory");  // the gathered rows: plain stores
      uint32_t fills[kStages];
#pragma unroll
      for (int i = 0; i < kStages; ++i) fills[i] = 0;
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      CeUnit u;
      for (int n = 0; ok && ce_unit(work, a, pair, n, u); ++n) {
        const CeJob& j = a.job[u.job];
        // A is read along its columns: G for dw, its transpose for dx
        const bool a_mn = (j.mode == kCeDw && !j.gt) || (j.mode == kCeDx && j.gt);
        const bool b_mn = j.mode == kCeDw || j.mode == kCeDx;  // B holds one row per k
        const CUtensorMap* ma = &j.a[(j.mode == kCeLse || j.mode == kCeGrad) ? all : 0];
        const CUtensorMap* mb = &j.b[j.mode == kCeDw ? all : 0];
        const int n0 = u.nb * j.bn + static_cast<int>(rank) * (j.bn / 2);
        // into one CTA's stage; a box of W's rows holds bn / 2 of them
        const int load_bytes = STREAMS * kCeABytes + (b_mn ? kCeBBytes : (j.bn / 2) * kBK * 2);
        for (int kb = u.kb0; kb < u.kb1; ++kb) {
          if (!wait_bar(&empty[s], ph ^ 1, ctl, kSiteProducerEmpty)) {
            ok = false;
            break;
          }
          uint8_t* sa = stages + s * Cfg::kStageBytes;
          uint8_t* sb = sa + STREAMS * kCeABytes;
          const uint32_t bar = mapa_shared(smem_u32(&full[s]), 0);
          if (leader) mbar_arrive_expect_tx(&full[s], 2 * load_bytes);
#pragma unroll
          for (int i = 0; i < STREAMS; ++i) {
            const int m0 = (STREAMS * u.mp + i) * kCeTile + static_cast<int>(rank) * kBM;
            if (a_mn) {
              tma_load_2d_pair(sa + i * kCeABytes, ma, bar, m0, kb * kBK);
              tma_load_2d_pair(sa + i * kCeABytes + 8192, ma, bar, m0 + 64, kb * kBK);
            } else {
              tma_load_2d_pair(sa + i * kCeABytes, ma, bar, kb * kBK, m0);
            }
          }
          if (b_mn) {
            const int k0 = (j.mode == kCeDx ? j.v0 : 0) + kb * kBK;
            tma_load_2d_pair(sb, mb, bar, n0, k0);
            tma_load_2d_pair(sb + 8192, mb, bar, n0 + 64, k0);
          } else {
            tma_load_2d_pair(sb, mb, bar, kb * kBK, j.v0 + n0);
          }
          fills[s]++;
          if (++s == kStages) {
            s = 0;
            ph ^= 1;
          }
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
  } else if (warp == 1 || warp == 2) {
    // ------------------------------------------------------------ MMA issuers (even CTA)
    // Two row tiles per unit: warp 1 issues the first's, warp 2 the second's,
    // each into its own accumulator; both read every stage.  One row tile: warp 1
    // alone, accumulators in turn, so that a chain's ending overlaps the next one's
    // products.  One thread's MMAs complete one after another, about 150 cycles each,
    // where two threads' reach the tensor pipe's 128; with one row tile in all W's 8
    // KB per MMA are 7.9 TB/s over all pairs, more than HBM gives.
    // (Issuers that shared a unit's blocks would each have to wait for all of them
    // all the same: a barrier's parity says nothing to a thread that has missed a
    // phase.)
    const int st = warp - 1;
    if (lane == 0 && leader && st < STREAMS) {
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      bool first = true;
      int use0 = 0, use1 = 0;  // of the accumulators
      int turn = 0;
      CeUnit u;
      for (int n = 0; ok && ce_unit(work, a, pair, n, u); ++n) {
        const CeJob& j = a.job[u.job];
        const bool a_mn = (j.mode == kCeDw && !j.gt) || (j.mode == kCeDx && j.gt);
        const bool b_mn = j.mode == kCeDw || j.mode == kCeDx;
        const uint32_t idesc = idesc_bf16(kCeTile, j.bn, a_mn, b_mn);
        int acc = st;
        // the next accumulator, when the ending has emptied it
        auto take = [&]() -> bool {
          if (STREAMS == 1) {
            acc = turn;
            turn ^= 1;
          }
          if (!wait_bar(&tempty[acc], ((acc ? use1 : use0) & 1) ^ 1, ctl, kSiteMmaAccEmpty))
            return false;
          if (acc) ++use1;
          else ++use0;
          tc_fence_after();
          return true;
        };
        if (!take()) break;
        uint32_t accumulate = 0;
        for (int kb = u.kb0; kb < u.kb1; ++kb) {
          if (FORM == kCeChains && kb > 0 && kb % kCeChain == 0) {
            mma_commit_pair(&tfull[acc], 0x3);
            accumulate = 0;
            if (!take()) {
              ok = false;
              break;
            }
          }
          if (!wait_bar(&full[s], ph, ctl, kSiteMmaFull)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t s0 = smem_u32(stages + s * Cfg::kStageBytes);
          const uint32_t a0 = s0 + st * kCeABytes;
          const uint32_t b0 = s0 + STREAMS * kCeABytes;
#pragma unroll
          for (int k = 0; k < kBK / 16; ++k) {
            const uint64_t ad = a_mn ? sdesc_sw128(a0 + k * 2048, 8192, 1024)
                                     : sdesc_sw128(a0 + k * 32, 16, 1024);
            const uint64_t bd = b_mn ? sdesc_sw128(b0 + k * 2048, 8192, 1024)
                                     : sdesc_sw128(b0 + k * 32, 16, 1024);
            mma_ss_pair(tmem_base + acc * 256, ad, bd, idesc, accumulate);
            accumulate = 1;
          }
          mma_commit_pair(&empty[s], 0x3);
          if (++s == kStages) {
            s = 0;
            ph ^= 1;
          }
        }
        if (!ok) break;
        if (!(kctl.inject && first)) mma_commit_pair(&tfull[acc], 0x3);
        first = false;
      }
      mma_commit_pair(done, 1);
      wait_bar(done, 0, ctl, kSiteDrain, false);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------------------ ending (both CTAs)
    const int q = warp & 3;
    const int half = (warp - 4) >> 2;  // columns 128 * half .. of the tile
    const uint64_t pol = l2_evict_first_policy();
    const uint32_t lead_empty0 = mapa_shared(smem_u32(&tempty[0]), 0);
    const uint32_t lead_empty1 = mapa_shared(smem_u32(&tempty[1]), 0);
    uint8_t* my_staging = staging + (warp - 4) * 2 * Cfg::kBufBytes;
    int flip = 0;
    const float out_scale = e.mean ? e.scale / static_cast<float>(max(count, 1)) : e.scale;
    int use0 = 0, use1 = 0;  // of the accumulators
    int turn = 0;
    bool ok = true;
    CeUnit u;
    for (int n = 0; ok && ce_unit(work, a, pair, n, u); ++n) {
      const CeJob& j = a.job[u.job];
      const int mode = j.mode;
      CeTileArgs t;
      t.out = &j.o;
      t.staging = my_staging;
      t.pol = pol;
      t.col0 = u.nb * j.bn + half * 128;
      t.none = u.kb0 == u.kb1;  // also a split without a K block of a short piece
      // the forward pass takes the tile's columns only: a narrow one ends inside
      // the accumulator
      t.cols = mode == kCeLse ? min(j.cols, (u.nb + 1) * j.bn) : j.cols;
      t.v0 = j.v0;
      t.d = a.d;
      t.count = count;
      t.add = j.add != 0;
      t.out_scale = out_scale;
      // waits for the next sums of row tile i: their accumulator's index, or -1
      auto next = [&](int i) -> int {
        int acc = i;
        if (STREAMS == 1) {
          acc = turn;
          turn ^= 1;
        }
        if (!wait_bar(&tfull[acc], (acc ? use1 : use0) & 1, ctl, kSiteEpiAccFull)) return -1;
        if (acc) ++use1;
        else ++use0;
        tc_fence_after();
        return acc;
      };
      auto columns = [&](int acc) -> uint32_t {
        return tmem_base + acc * 256 + (static_cast<uint32_t>(q * 32) << 16) + half * 128;
      };
      auto free_of = [&](int acc) -> CeFree {
        return CeFree{acc ? &tempty[1] : &tempty[0], acc ? lead_empty1 : lead_empty0, leader};
      };
#pragma unroll 1
      for (int i = 0; i < STREAMS; ++i) {
        t.row = (STREAMS * u.mp + i) * kCeTile + static_cast<int>(rank) * kBM + q * 32 + lane;
        t.row_ok = t.row < count;
        t.buf_row = u.split * e.m_pad + t.row;
        t.tgt = -1;
        t.lse2 = t.dl = 0.0f;
        if ((mode == kCeLse || mode == kCeGrad) && t.row_ok) {
          t.tgt = e.tgt[t.row] - t.v0 - t.col0;
          if (mode == kCeGrad) {
            t.lse2 = e.lse2[t.row];
            t.dl = e.dl[t.row];
          }
        }
        const int acc = next(i);
        ok = acc >= 0;
        if (!ok) break;
        const uint32_t tb = columns(acc);
        const CeFree release = free_of(acc);
        float m = -INFINITY, sum = 0.0f;  // kLse
        if constexpr (FORM == kCeChains) {
          uint32_t v[4][32];  // the sums over the chains
          ce_read(tb, release, v);
          for (int kb = kCeChain; ok && kb < u.kb1; kb += kCeChain) {
            const int more = next(i);
            ok = more >= 0;
            if (ok) ce_add(columns(more), free_of(more), v);
          }
          if (!ok) break;
          if (mode == kCeLse) {
#pragma unroll
            for (int c = 0; c < 4; ++c) ce_chunk<kCeLse, FORM>(c, v[c], t, e, flip, m, sum);
            if (t.row_ok)
              e.part[static_cast<int64_t>(2 * u.nb + half) * e.M + t.row] = make_float2(m, sum);
          } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) ce_chunk<kCeGrad, FORM>(c, v[c], t, e, flip, m, sum);
          }
        } else if (mode == kCeLse) {
          ce_tile<kCeLse, FORM>(tb, release, t, e, flip, m, sum);
          if (t.row_ok)
            e.part[static_cast<int64_t>(2 * u.nb + half) * e.M + t.row] = make_float2(m, sum);
        } else if (mode == kCeGrad) {
          ce_tile<kCeGrad, FORM>(tb, release, t, e, flip, m, sum);
        } else if (mode == kCeDx) {
          ce_tile<kCeDx, FORM>(tb, release, t, e, flip, m, sum);
        } else {
          ce_tile<kCeDw, FORM>(tb, release, t, e, flip, m, sum);
        }
      }
    }
    if (lane == 0) bulk_wait<0>();
    __syncwarp();
  }

  if (ctl.prof && threadIdx.x == 0)
    atomicAdd(&ctl.prof[31], static_cast<unsigned long long>(clock64() - t_start));
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // no CTA leaves while its peer may still signal it or read its memory
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

// ---------------------------------------------------------------- before and after

constexpr int kPrepThreads = 256;

// Sum over the CTA of a pair of counts.
__device__ __forceinline__ int2 block_sum2(int a, int b) {
  __shared__ int part[2][kPrepThreads / 32];
  a = __reduce_add_sync(0xFFFFFFFFu, a);
  b = __reduce_add_sync(0xFFFFFFFFu, b);
  if ((threadIdx.x & 31) == 0) {
    part[0][threadIdx.x >> 5] = a;
    part[1][threadIdx.x >> 5] = b;
  }
  __syncthreads();
  int2 s = make_int2(0, 0);
  for (int w = 0; w < kPrepThreads / 32; ++w) {
    s.x += part[0][w];
    s.y += part[1][w];
  }
  return s;
}

// One row by one warp, four 16-byte vectors per lane in flight; zeros without src.
__device__ __forceinline__ void copy_row(__nv_bfloat16* dst, const __nv_bfloat16* src, int D) {
  for (int c0 = (threadIdx.x & 31) * 8; c0 < D; c0 += 4 * 256) {
    uint4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      v[k] = src && c0 + k * 256 < D ? ldg_u4(src + c0 + k * 256) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (c0 + k * 256 < D) st_u4(dst + c0 + k * 256, v[k]);
  }
}

// CTA b takes the rows [b * rows_per, ...): it counts the scored rows before
// them itself (all targets are a few KB in L2), so one launch lists the scored
// rows in order, gathers their x where not all are scored, and writes the
// results of the others (loss and lse 0, or a zero row of dx).
template <typename Id>
__global__ void __launch_bounds__(kPrepThreads)
    ce_prep_kernel(const Id* __restrict__ targets, const CePrep p) {
  griddep_launch_dependents();
  griddep_wait();
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * p.rows_per;
  const int64_t r1 = min(r0 + p.rows_per, static_cast<int64_t>(p.M));
  int total = 0, before = 0;
#pragma unroll 8
  for (int64_t i = threadIdx.x; i < p.M; i += kPrepThreads) {
    const int64_t t = static_cast<int64_t>(targets[i]);
    const int scored = t >= 0 && t < p.V;
    total += scored;
    before += scored && i < r0;
  }
  const int2 sums = block_sum2(total, before);
  total = sums.x;
  int slot = sums.y;
  const bool gather = total < p.M;
  const int zero_to = (total + kBK - 1) / kBK * kBK;  // the last K block of kDw
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *p.count = total;
    if (p.ticket) *p.ticket = 0u;
  }
  // 32 rows at a time: a lane's row in the lists, a warp's row in the copies
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int64_t b0 = r0; b0 < r1; b0 += 32) {
    const int n = static_cast<int>(min(r1 - b0, static_cast<int64_t>(32)));
    const int64_t t = lane < n ? static_cast<int64_t>(targets[b0 + lane]) : -1;
    const bool scored = t >= 0 && t < p.V;
    const unsigned mask = __ballot_sync(0xFFFFFFFFu, scored);
    if (warp == 0) {
      const int64_t r = b0 + lane;
      if (scored) {
        const int at = slot + __popc(mask & ((1u << lane) - 1u));
        p.rows[at] = static_cast<int>(r);
        p.tgt[at] = static_cast<int>(t);
        if (p.lse2) {
          p.lse2[at] = p.lse_in[r] * kLog2e;
          p.dl[at] = p.dloss ? p.dloss[r] : 1.0f;
        }
      } else if (lane < n && p.loss) {
        p.loss[r] = 0.0f;
        p.lse_out[r] = 0.0f;
      }
    }
    for (int i = warp; i < n; i += kPrepThreads / 32) {
      const int64_t r = b0 + i;
      if ((mask >> i) & 1u) {
        if (gather) copy_row(p.xc + (slot + __popc(mask & ((1u << i) - 1u))) *
                                        static_cast<int64_t>(p.D), p.x + r * p.D, p.D);
      } else if (p.dx) {
        copy_row(p.dx + r * p.D, nullptr, p.D);
      }
      if (gather && r >= total && r < zero_to)  // slots past the scored rows
        copy_row(p.xc + r * p.D, nullptr, p.D);
    }
    slot += __popc(mask);
  }
}

constexpr int kJoinThreads = 512;
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kJoinRows = 8;  // rows per CTA: 64-byte segments of the partial sums

// (m, s) stands for s * 2^m.
__device__ __forceinline__ float2 join(float2 a, float2 b) {
  const float m = fmaxf(a.x, b.x);
  const float ref = m == -INFINITY ? 0.0f : m;
  return make_float2(m, fmaf(a.y, pow2(a.x - ref), b.y * pow2(b.x - ref)));
}

__device__ __forceinline__ bool scored(const CeJoin& p, int row) {
  const int64_t t = ce_target(p.targets, p.ids64, row);
  return t >= 0 && t < p.V;
}
static_assert(kCeSwapMax <= kJoinThreads, "a thread for each row that is taken as it is");

// Eight scored rows per CTA, 64 threads each: adds up each row's partial sums,
// writes its loss and lse; the last CTA adds the CTAs' sums of losses in order
// for the mean.
__global__ void __launch_bounds__(kJoinThreads) ce_join_kernel(const CeJoin p) {
  __shared__ float2 part[kJoinWarps][kJoinRows];
  __shared__ double sums[kJoinWarps];
  __shared__ bool last;
  griddep_launch_dependents();
  griddep_wait();
  const int count = p.rows ? *p.count : p.M;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.x * kJoinRows + (lane & (kJoinRows - 1));
  // what the row's result takes beside the sums, on its way meanwhile
  float target = 0.0f;  // the target's product
  int r = row;
  bool counts = true;
  if (warp == 0 && lane < kJoinRows && row < count) {
    target = p.tlog[row];
    if (p.rows) r = p.rows[row];
    else counts = scored(p, row);
  }
  float2 a = make_float2(-INFINITY, 0.0f);
  if (row < count) {
    const float2* src = p.part + row;
    constexpr int kAhead = 16, kStep = kJoinThreads / kJoinRows;
    for (int n0 = threadIdx.x / kJoinRows; n0 < p.parts; n0 += kAhead * kStep) {
      float2 v[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (n0 + i * kStep < p.parts) v[i] = src[static_cast<int64_t>(n0 + i * kStep) * p.M];
      float m = a.x;
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (n0 + i * kStep < p.parts) m = fmaxf(m, v[i].x);
      const float ref = m == -INFINITY ? 0.0f : m;
      float sum = a.y * pow2(a.x - ref);
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (n0 + i * kStep < p.parts) sum = fmaf(v[i].y, pow2(v[i].x - ref), sum);
      a = make_float2(m, sum);
    }
  }
#pragma unroll
  for (int o = kJoinRows; o < 32; o <<= 1) {
    float2 b;
    b.x = __shfl_xor_sync(0xFFFFFFFFu, a.x, o);
    b.y = __shfl_xor_sync(0xFFFFFFFFu, a.y, o);
    a = join(a, b);
  }
  if (lane < kJoinRows) part[warp][lane] = a;
  __syncthreads();
  if (warp == 0) {
    // four lanes per row: each joins the parts of four warps, then they join
#pragma unroll
    for (int w = 0; w < kJoinWarps; w += 32 / kJoinRows) {
      const float2 b = part[w + lane / kJoinRows][lane & (kJoinRows - 1)];
      a = w == 0 ? b : join(a, b);
    }
#pragma unroll
    for (int o = kJoinRows; o < 32; o <<= 1) {
      float2 b;
      b.x = __shfl_xor_sync(0xFFFFFFFFu, a.x, o);
      b.y = __shfl_xor_sync(0xFFFFFFFFu, a.y, o);
      a = join(a, b);
    }
    double loss = 0.0;
    if (lane < kJoinRows && row < count) {
      // A confident row's loss is a small difference: in 64 bits, and of powers of
      // two by the same fp32 factor c2 (its rounding is then one of the loss, not
      // one of the logits that outlives the subtraction).  What is left is the
      // rounding of the powers, 2^-22; the exact loss is never below zero.
      const double sum2 = static_cast<double>(log2f(a.y));
      const double lse = (static_cast<double>(a.x) + sum2) * kLn2;
      if (counts) {
        loss = ((static_cast<double>(a.x) - static_cast<double>(p.c2) * target) + sum2) * kLn2;
        if (loss < 0.0) loss = 0.0;
      }
      p.loss[r] = static_cast<float>(loss);
      p.lse[r] = counts ? static_cast<float>(lse) : 0.0f;
    }
    if (p.mean) {
#pragma unroll
      for (int o = kJoinRows / 2; o > 0; o >>= 1) loss += __shfl_xor_sync(0xFFFFFFFFu, loss, o);
      if (lane == 0) {
        p.sums[blockIdx.x] = loss;
        if (gridDim.x > 1) {
          __threadfence();
          last = atomicAdd(p.ticket, 1u) == gridDim.x - 1;
        } else {
          last = true;
        }
      }
    }
  }
  if (!p.mean) return;
  __syncthreads();
  if (!last) return;
  if (gridDim.x > 1) __threadfence();
  double s = 0.0;
  for (unsigned i = threadIdx.x; i < gridDim.x; i += kJoinThreads) s += __ldcg(p.sums + i);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  if (lane == 0) sums[warp] = s;
  int n = count;
  if (!p.rows) n = __syncthreads_count(static_cast<int>(threadIdx.x) < p.M && scored(p, threadIdx.x));
  else __syncthreads();
  if (threadIdx.x == 0) {
    s = 0.0;
    for (int w = 0; w < kJoinWarps; ++w) s += sums[w];
    *p.mean = static_cast<float>(s / max(n, 1));
  }
}

constexpr int kOutThreads = 128;

// dx of the scored rows: the splits' sums added in order, scaled, rounded once.
// A warp per 256 columns of a row.
__global__ void __launch_bounds__(kOutThreads) ce_dx_kernel(const CeDxOut p) {
  griddep_launch_dependents();
  griddep_wait();
  const int count = *p.count;
  const float scale = p.mean ? p.scale / static_cast<float>(max(count, 1)) : p.scale;
  const int segs = (p.D + 255) / 256;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kOutThreads / 32);
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * (kOutThreads / 32) + (threadIdx.x >> 5);
       t < static_cast<int64_t>(count) * segs; t += step) {
    const int64_t row = t / segs;
    const int col = static_cast<int>(t - row * segs) * 256 + (threadIdx.x & 31) * 8;
    if (col >= p.D) continue;
    float f[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    for (int s = 0; s < p.splits; ++s) {
      const float4* src = reinterpret_cast<const float4*>(
          p.acc + (static_cast<int64_t>(s) * p.m_pad + row) * p.D + col);
      const float4 x = __ldcs(src), y = __ldcs(src + 1);
      f[0] += x.x; f[1] += x.y; f[2] += x.z; f[3] += x.w;
      f[4] += y.x; f[5] += y.y; f[6] += y.z; f[7] += y.w;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] *= scale;
    st_u4(p.dx + static_cast<int64_t>(p.rows[row]) * p.D + col, pack8(f));
  }
}

cudaLaunchConfig_t overlapped(int64_t grid, int threads, size_t smem, cudaStream_t stream,
                              cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

template <int FORM>
cudaError_t run_ce(const CeLaunch& launch, const CeEnd& end, const KernelCtl& ctl, int grid,
                   cudaStream_t stream) {
  static std::atomic<uint64_t> mask{0};
  auto kernel = ce_gemm_kernel<FORM>;
  constexpr int smem = CeCfg<FORM>::kSmem;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (!(mask.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    mask.fetch_or(bit, std::memory_order_acq_rel);
  }
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = overlapped(grid, kCeThreads, smem, stream, attr);
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, launch, end, ctl);
}

}  // namespace

cudaError_t launch_ce_gemm(const CeLaunch& launch, const CeEnd& end, int streams, bool chains,
                           int grid, const KernelCtl& ctl, cudaStream_t stream) {
  return chains         ? run_ce<kCeChains>(launch, end, ctl, grid, stream)
         : streams == 2 ? run_ce<kCeTwo>(launch, end, ctl, grid, stream)
                        : run_ce<kCeLone>(launch, end, ctl, grid, stream);
}

cudaError_t launch_ce_prep(const void* targets, bool ids64, CePrep p, int sms,
                           cudaStream_t stream) {
  // eight CTAs per SM; one row each up to that
  const int64_t most = static_cast<int64_t>(sms) * 8;
  p.rows_per = static_cast<int>((p.M + most - 1) / most);
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg =
      overlapped((p.M + p.rows_per - 1) / p.rows_per, kPrepThreads, 0, stream, attr);
  return ids64 ? cudaLaunchKernelEx(&cfg, ce_prep_kernel<int64_t>,
                                    static_cast<const int64_t*>(targets), p)
               : cudaLaunchKernelEx(&cfg, ce_prep_kernel<int>, static_cast<const int*>(targets), p);
}

cudaError_t launch_ce_join(const CeJoin& p, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = overlapped((p.M + kJoinRows - 1) / kJoinRows, kJoinThreads, 0, stream, attr);
  return cudaLaunchKernelEx(&cfg, ce_join_kernel, p);
}

cudaError_t launch_ce_dx(const CeDxOut& p, int M, int sms, cudaStream_t stream) {
  const int64_t warps = static_cast<int64_t>(M) * ((p.D + 255) / 256);
  const int64_t ctas = std::min<int64_t>((warps + 3) / 4, static_cast<int64_t>(sms) * 16);
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = overlapped(ctas, kOutThreads, 0, stream, attr);
  return cudaLaunchKernelEx(&cfg, ce_dx_kernel, p);
}

}  // namespace gbf
