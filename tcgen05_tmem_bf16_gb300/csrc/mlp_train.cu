// mlp_train.cu -- the products of a gated MLP block that is trained, and of its
// gradient, each with its ending.
//
//   g = x Wg^T, u = x Wu^T, h = act(g) u               (kMbGlu: all three stored)
//   dh = dout Wd;  dg = dh u act'(g), du = dh act(g)    (kMbGluGrad)
//   dx = dg Wg + du Wu                                  (one product over both halves of K)
//   dWg = dg^T x, dWu = du^T x, dWd = dout^T h
//
// One kernel does them all: the CTA-pair main loop of gemm_pair.cu (256 x 256
// tiles on two SMs, tcgen05.mma.cta_group::2, TMA-fed), working through a list of
// up to four products per launch that do not depend on one another.  dh never
// reaches memory: its tile ends as dg and du.  Every operand is read in the layout
// in which it lies, along rows or columns, so nothing is transposed in memory.
//
// The gradient takes two launches: dh, then {dx, dWg, dWu, dWd}, which fill each
// other's last round of units.
//
// Bound by the tensor pipe above some 500 rows, by the weights' bytes below.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "epilogue.cuh"
#include "glu_grad.cuh"
#include "internal.h"
#include "pair_end.cuh"
#include "ptx.cuh"

namespace gbf {

namespace {

constexpr int kMbThreads = 384;          // warps 0-3 roles, 4-11 ending
constexpr int kMbTile = 256;             // rows and columns of a pair's tile
constexpr int kMbABytes = kBM * kBK * 2;  // 16 KB: this CTA's 128 rows of A
constexpr int kMbBBytes = 128 * kBK * 2;  // 16 KB: this CTA's half of B
constexpr int kMbGroup = 8;              // raster group (units of rows)

// STREAMS row tiles per unit of work, as in linear_ce.cu: two that share each B
// tile, or a lone one.  (Sixteen warps for a lone one's ending, and rows of 128 bytes for
// its stores, change nothing: the three weights' gradients of 16 x 4096 x 14336, 352 MB,
// are 53 us either way, 6.6 TB/s.)
// GRAD: kMbGluGrad alone, with several pairs of buffers per two warps of the ending for
// g and u, which become dg and du.
constexpr int kGradBytes = 32 * 128;  // 32 rows x 64 columns
template <int STREAMS, bool GRAD>
struct MbCfg {
  static constexpr int kStageBytes = STREAMS * kMbABytes + kMbBBytes;
  static constexpr int kStages = STREAMS == 2 ? (GRAD ? 3 : 4) : GRAD ? 4 : 5;
  static constexpr int kSlots = STREAMS == 2 ? 2 : 3;
  static constexpr int kBarBytes = 1024;
  static constexpr int kWarpBytes = GRAD ? kSlots * kGradBytes : 2 * kStageChunkBytes;
  static constexpr int kStagingBytes = 8 * kWarpBytes;
  static constexpr int kSmem = 1024 + kStages * kStageBytes + kBarBytes + kStagingBytes;
  static_assert(kSmem <= 227 * 1024, "shared memory per CTA");
};

// A unit of work: STREAMS row tiles x one column tile x a range of K blocks of
// one of the launch's products.
struct MbUnit {
  int job, mp, nb, split, kb0, kb1;
};

// The n-th unit of a pair; false after its last.  The units of job 0 are long;
// they are dealt out first, one per pair and round, and the pairs that got one more
// than the others sit out `skip` rounds of the short ones.  (Every role of a CTA
// computes this for every unit, so it does without divisions: the divisors are the
// launch's, their reciprocals the host's.)
__device__ __forceinline__ uint32_t mb_div(uint32_t x, const MbDiv& d) {
  return d.by == 1 ? x : __umulhi(x, d.mul) >> d.shift;
}
__device__ __forceinline__ bool mb_unit(const MbLaunch& a, int pair, int npairs, int n, MbUnit& u) {
  const int mine = a.longs_each + (pair < a.extra ? 1 : 0);
  int t;
  if (n < mine) {
    t = n * npairs + pair;
    u.job = 0;
  } else {
    const int round = n - mine + (pair < a.extra ? a.skip : 0);
    if (round < a.skip)
      t = round * (npairs - a.extra) + pair - a.extra;
    else
      t = a.skip * (npairs - a.extra) + (round - a.skip) * npairs + pair;
    if (t >= a.shorts) return false;
    u.job = 1;
    while (t >= a.job[u.job].units) t -= a.job[u.job++].units;
  }
  const MbJob& j = a.job[u.job];
  u.split = 0;
  u.kb0 = 0;
  u.kb1 = j.num_kb;
  if (j.splits > 1) {
    u.split = mb_div(t, j.tiles);
    t -= u.split * j.tiles.by;
    u.kb0 = mb_div(u.split * j.num_kb, j.parts);
    u.kb1 = mb_div((u.split + 1) * j.num_kb, j.parts);
  }
  // as tile_coords: groups of kMbGroup units of rows, the column tile slowest
  const int g = mb_div(t, j.group);
  const int local = t - g * j.group.by;
  if (g < j.full_groups) {
    u.nb = local / kMbGroup;
    u.mp = g * kMbGroup + local % kMbGroup;
  } else {
    u.nb = mb_div(local, j.last);
    u.mp = g * kMbGroup + local - u.nb * j.last.by;
  }
  return true;
}

// 16 columns of this lane's row of a 32 x 64 chunk (128-byte rows, 128-byte swizzle),
// from column 16 at on: from and to a staging buffer.
__device__ __forceinline__ uint32_t staged_unit(const uint8_t* buf, uint32_t unit) {
  const uint32_t lane = threadIdx.x & 31;
  return smem_u32(buf) + lane * 128u + ((unit ^ (lane & 7u)) << 4);
}
__device__ __forceinline__ void staged_row16(uint4 (&d)[2], const uint8_t* buf, uint32_t at) {
#pragma unroll
  for (uint32_t v = 0; v < 2; ++v)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(d[v].x), "=r"(d[v].y), "=r"(d[v].z), "=r"(d[v].w)
                 : "r"(staged_unit(buf, 2 * at + v))
                 : "memory");
}
__device__ __forceinline__ void stage_row16(uint8_t* buf, uint32_t at, const uint32_t (&w)[8]) {
#pragma unroll
  for (uint32_t v = 0; v < 2; ++v)
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(staged_unit(buf, 2 * at + v)),
                 "r"(w[4 * v]), "r"(w[4 * v + 1]), "r"(w[4 * v + 2]), "r"(w[4 * v + 3])
                 : "memory");
}

// dg and du of 16 columns.
template <int ACT>
__device__ __forceinline__ void glu_grad_pack(const uint32_t (&dh)[16], const uint4 (&g2)[2],
                                              const uint4 (&u2)[2], uint32_t (&dg)[8],
                                              uint32_t (&du)[8]) {
  const uint32_t g[8] = {g2[0].x, g2[0].y, g2[0].z, g2[0].w, g2[1].x, g2[1].y, g2[1].z, g2[1].w};
  const uint32_t u[8] = {u2[0].x, u2[0].y, u2[0].z, u2[0].w, u2[1].x, u2[1].y, u2[1].z, u2[1].w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    f2 y, dy;
    act_both<ACT>(f2_of(bf16lo(g[i]), bf16hi(g[i])), y, dy);
    const f2 d = f2_of(__uint_as_float(dh[2 * i]), __uint_as_float(dh[2 * i + 1]));
    float lo, hi;
    f2_get(f2_mul(f2_mul(d, f2_of(bf16lo(u[i]), bf16hi(u[i]))), dy), lo, hi);
    dg[i] = pack_bf16x2(lo, hi);
    f2_get(f2_mul(d, y), lo, hi);
    du[i] = pack_bf16x2(lo, hi);
  }
}

// The chunks of g and u of the two warps that share 32 rows of a tile, 64 columns at
// a time, on their way ahead of the arithmetic: one lane asks the TMA engine for the
// next chunk of the next units, into a slot whose dg and du have been stored.
//
// dh of 4096 x 4096 x 14336 takes 275 us without g and u, 245 without an ending.  Read by
// the lanes themselves they cost the products their shared memory, which is the same as L1
// (16 bytes of 32 rows at a time 450 us, 64 of 8 rows 362); by the TMA engine its requests
// count, one per row of a box: 330 us with rows of 64 bytes, 314 with 128.
template <int STREAMS, int SLOTS>
struct GradLoads {
  MbUnit u;   // of the next chunk
  int n, c;   // its unit's number, its place in the unit: four per row tile
  int slot;
  bool more;
  __device__ __forceinline__ void start(const MbLaunch& a, int pair, int npairs) {
    n = c = slot = 0;
    more = mb_unit(a, pair, npairs, n, u);
  }
  __device__ __forceinline__ void next(const MbLaunch& a, int pair, int npairs, int row,
                                       uint8_t* slots, uint64_t* bars) {
    if (!more) return;
    if ((threadIdx.x & 31) == 0) {
      const MbJob& j = a.job[u.job];
      uint8_t* buf = slots + slot * 2 * kGradBytes;
      mbar_arrive_expect_tx(&bars[slot], 2 * kGradBytes);
      const int col0 = u.nb * kMbTile + (c & 3) * 64;
      const int row0 = (STREAMS * u.mp + (c >> 2)) * kMbTile + row;
      const uint64_t once = policy_evict_first();
      tma_load_2d_hint(buf, &j.a[1], &bars[slot], col0, row0, once);
      tma_load_2d_hint(buf + kGradBytes, &j.b[1], &bars[slot], col0, row0, once);
    }
    if (++slot == SLOTS) slot = 0;
    if (++c == 4 * STREAMS) {
      c = 0;
      more = mb_unit(a, pair, npairs, ++n, u);
    }
  }
};

// This warp's 32 of a chunk's 64 columns of dh (half 0 or 1): dg and du in the place of
// g and u.  `ask`, in the middle, asks for the chunk after the next.
template <int ACT, typename Ask>
__device__ __forceinline__ void glu_grad_chunk(uint32_t tb, uint8_t* buf, int half,
                                               const Ask& ask) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint4 g2[2], u2[2];
    uint32_t v[16], dg[8], du[8];
    const uint32_t at = 2 * half + h;
    tmem_ld16(tb + 16 * h, v);
    staged_row16(g2, buf, at);
    staged_row16(u2, buf + kGradBytes, at);
    tmem_wait_ld();
    glu_grad_pack<ACT>(v, g2, u2, dg, du);
    stage_row16(buf, at, dg);
    stage_row16(buf + kGradBytes, at, du);
    if (h == 0) ask();
  }
}

// A warp's 128 columns of a product, to the fp32 rows of its part of K.
__device__ __forceinline__ void store_part(uint32_t tb, const AccFree& release, const MbJob& j,
                                           uint8_t* bufs, int& flip, int row0, int col0, int part) {
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t v[32];
    tmem_ld32(tb + 32 * c, v);
    tmem_wait_ld();
    if (c == 3) release();
    put_chunk_f32(bufs, kStageChunkBytes, flip, v, &j.o[0], part * j.m_pad + row0, col0 + 32 * c,
                  j.cols, row0 < j.rows, false);
  }
}

__device__ __forceinline__ void pack32(const uint32_t (&v)[32], uint32_t (&w)[16]) {
#pragma unroll
  for (int k = 0; k < 16; ++k)
    w[k] = pack_bf16x2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1]));
}

// A warp's 128 columns to bf16, 32 at a time: the next are on their way from tensor
// memory meanwhile.
__device__ __forceinline__ void store_tile(uint32_t tb, const AccFree& release, const MbJob& j,
                                              uint8_t* bufs, int& flip, int row0, int col0,
                                              uint64_t pol) {
  auto put = [&](int c, const uint32_t (&v)[32]) {
    uint32_t w[16];
    pack32(v, w);
    put_chunk<false>(bufs, kStageChunkBytes, flip, c, w, &j.o[0], row0, col0 + c * 32, j.rows,
                     j.cols, pol);
  };
  uint32_t va[32], vb[32];
  tmem_ld32(tb, va);
  tmem_wait_ld();
  tmem_ld32(tb + 32, vb);
  put(0, va);
  tmem_wait_ld();
  tmem_ld32(tb + 64, va);
  put(1, vb);
  tmem_wait_ld();
  tmem_ld32(tb + 96, vb);
  put(2, va);
  tmem_wait_ld();
  release();
  put(3, vb);
}

template <int STREAMS, bool GRAD>
__global__ void __launch_bounds__(kMbThreads, 1)
    mlp_train_kernel(const __grid_constant__ MbLaunch a, const KernelCtl kctl) {
  using Cfg = MbCfg<STREAMS, GRAD>;
  constexpr int kStages = Cfg::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint8_t* stages = smem;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kStages * Cfg::kStageBytes);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* done = tempty + 2;
  uint64_t* loaded = done + 1;  // GRAD: slots of g and u, of each two warps
  uint64_t* made = loaded + 4 * Cfg::kSlots;  // dg and du by both warps
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(made + 4 * Cfg::kSlots);
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
    for (int i = 0; i < 4 * Cfg::kSlots; ++i) {
      mbar_init(&loaded[i], 1);
      mbar_init(&made[i], 2);
    }
    *abort_flag = 0;
    fence_mbar_init();
    for (int i = 0; i < kMbJobs; ++i) {
      if (a.job[i].mode == kMbNone) continue;
      tma_prefetch_desc(&a.job[i].a[0]);
      tma_prefetch_desc(&a.job[i].b[0]);
      tma_prefetch_desc(&a.job[i].o[0]);
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
  griddep_wait();  // operands may be the previous kernel's results

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer (both CTAs)
    if (lane == 0) {
      asm volatile("fence.proxy.async;" ::: "memory");
      const uint64_t stream = policy_evict_first();
      int fills = 0;
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      MbUnit u;
      for (int n = 0; ok && mb_unit(a, pair, npairs, n, u); ++n) {
        const MbJob& j = a.job[u.job];
        const bool glu = j.mode == kMbGlu;  // the even CTA's half of B is Wg's, the odd one's Wu's
        // A weight of few rows is read by one unit: the lines of the other operands, which
        // every unit reads, outlive its own in L2 (gradient of 16 x 4096 x 14336 123 us, the
        // weights as any operand 128.5).
        const bool once = (u.job == 0 || glu) && j.rows <= kMbTile;
        const int n0 = glu ? u.nb * 128 : u.nb * kMbTile + static_cast<int>(rank) * 128;
        for (int kb = u.kb0; kb < u.kb1; ++kb) {
          if (!wait_bar(&empty[s], ph ^ 1, ctl, kSiteProducerEmpty)) {
            ok = false;
            break;
          }
          const int second = kb >= j.kb_first ? 1 : 0;  // K blocks of the second pair of operands
          const int k0 = (kb - second * j.kb_first) * kBK;
          const CUtensorMap* ma = &j.a[second];
          const CUtensorMap* mb = &j.b[glu ? static_cast<int>(rank) : second];
          uint8_t* sa = stages + s * Cfg::kStageBytes;
          uint8_t* sb = sa + STREAMS * kMbABytes;
          const uint32_t bar = mapa_shared(smem_u32(&full[s]), 0);
          if (leader) mbar_arrive_expect_tx(&full[s], 2 * Cfg::kStageBytes);
#pragma unroll
          for (int i = 0; i < STREAMS; ++i) {
            const int m0 = (STREAMS * u.mp + i) * kMbTile + static_cast<int>(rank) * kBM;
            if (j.a_mn) {
              tma_load_2d_pair(sa + i * kMbABytes, ma, bar, m0, k0);
              tma_load_2d_pair(sa + i * kMbABytes + 8192, ma, bar, m0 + 64, k0);
            } else {
              tma_load_2d_pair(sa + i * kMbABytes, ma, bar, k0, m0);
            }
          }
          if (j.b_mn) {
            if (once) {
              tma_load_2d_pair_hint(sb, mb, bar, n0, k0, stream);
              tma_load_2d_pair_hint(sb + 8192, mb, bar, n0 + 64, k0, stream);
            } else {
              tma_load_2d_pair(sb, mb, bar, n0, k0);
              tma_load_2d_pair(sb + 8192, mb, bar, n0 + 64, k0);
            }
          } else if (once) {
            tma_load_2d_pair_hint(sb, mb, bar, k0, n0, stream);
          } else {
            tma_load_2d_pair(sb, mb, bar, k0, n0);
          }
          ++fills;
          if (++s == kStages) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      if (ok) {
        for (int i = 0; i < kStages && i < fills; ++i)  // stage i's last fill
          wait_bar(&empty[i], (fills - 1 - i) / kStages & 1, ctl, kSiteDrain, false);
      } else {
        const uint64_t t0 = globaltimer_ns();  // let the copies in flight land (bounded)
        while (globaltimer_ns() - t0 < 2000000ull) __nanosleep(1000);
      }
    }
    __syncwarp();
  } else if (warp == 1 || warp == 2) {
    // ------------------------------------------------------------ MMA issuers (even CTA)
    // Two row tiles per unit: warp 1 issues the first's, warp 2 the second's, each
    // into its own accumulator.  One row tile: warp 1 alone, accumulators in turn.
    const int st = warp - 1;
    if (lane == 0 && leader && st < STREAMS) {
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      MbUnit u;
      for (int n = 0; ok && mb_unit(a, pair, npairs, n, u); ++n) {
        const MbJob& j = a.job[u.job];
        const uint32_t idesc = idesc_bf16(kMbTile, 256, j.a_mn != 0, j.b_mn != 0);
        const int acc = STREAMS == 2 ? st : n & 1;
        const int use = STREAMS == 2 ? n : n >> 1;
        if (!wait_bar(&tempty[acc], (use & 1) ^ 1, ctl, kSiteMmaAccEmpty)) break;
        tc_fence_after();
        for (int kb = u.kb0; kb < u.kb1; ++kb) {
          if (!wait_bar(&full[s], ph, ctl, kSiteMmaFull)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t s0 = smem_u32(stages + s * Cfg::kStageBytes);
          const uint32_t a0 = s0 + st * kMbABytes;
          const uint32_t b0 = s0 + STREAMS * kMbABytes;
#pragma unroll
          for (int k = 0; k < kBK / 16; ++k) {
            const uint64_t ad = j.a_mn ? sdesc_sw128(a0 + k * 2048, 8192, 1024)
                                       : sdesc_sw128(a0 + k * 32, 16, 1024);
            const uint64_t bd = j.b_mn ? sdesc_sw128(b0 + k * 2048, 8192, 1024)
                                       : sdesc_sw128(b0 + k * 32, 16, 1024);
            mma_ss_pair(tmem_base + acc * 256, ad, bd, idesc, (kb != u.kb0 || k != 0) ? 1u : 0u);
          }
          mma_commit_pair(&empty[s], 0x3);
          if (++s == kStages) {
            s = 0;
            ph ^= 1;
          }
        }
        if (!ok) break;
        if (!(kctl.inject && n == 0)) mma_commit_pair(&tfull[acc], 0x3);
      }
      mma_commit_pair(done, 1);
      wait_bar(done, 0, ctl, kSiteDrain, false);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------------------ ending (both CTAs)
    const int q = warp & 3;
    const int slice = (warp - 4) >> 2;  // of the tile's columns
    const uint64_t first = l2_evict_first_policy();
    const uint32_t lead_empty0 = mapa_shared(smem_u32(&tempty[0]), 0);
    const uint32_t lead_empty1 = mapa_shared(smem_u32(&tempty[1]), 0);
    uint8_t* bufs = staging + (warp - 4) * Cfg::kWarpBytes;
    int flip = 0;
    bool ok = true;
    MbUnit u;
    GradLoads<STREAMS, Cfg::kSlots> loads;
    uint64_t* bars = loaded + q * Cfg::kSlots;
    uint8_t* slots = staging + q * 2 * Cfg::kWarpBytes;
    const int row_in = static_cast<int>(rank) * kBM + q * 32;  // of a row tile
    int slot = 0;  // GRAD: the present chunk's, and the phase of its barrier
    uint32_t phase = 0;
    if (GRAD && slice == 0) {
      loads.start(a, pair, npairs);
      for (int i = 1; i < Cfg::kSlots; ++i) loads.next(a, pair, npairs, row_in, slots, bars);
    }
    for (int n = 0; ok && mb_unit(a, pair, npairs, n, u); ++n) {
      const MbJob& j = a.job[u.job];
#pragma unroll 1
      for (int i = 0; i < STREAMS; ++i) {
        const int acc = STREAMS == 2 ? i : n & 1;
        const int use = STREAMS == 2 ? n : n >> 1;
        const int row0 = (STREAMS * u.mp + i) * kMbTile + row_in;
        const uint32_t tb = tmem_base + acc * 256 + (static_cast<uint32_t>(q * 32) << 16);
        const AccFree release{acc ? &tempty[1] : &tempty[0], acc ? lead_empty1 : lead_empty0,
                              leader};
        ok = wait_bar(&tfull[acc], use & 1, ctl, kSiteEpiAccFull);
        if (!ok) break;
        tc_fence_after();
        if constexpr (GRAD) {
          const uint64_t pol = policy_evict_last();  // the next launch's operands
          // the slot that the present chunk's predecessor leaves, once its stores have
          // read it
          auto ask = [&]() {
            if (slice != 0) return;
            if (lane == 0) bulk_wait_read<0>();
            loads.next(a, pair, npairs, row_in, slots, bars);
          };
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint8_t* buf = slots + slot * 2 * kGradBytes;
            ok = wait_bar(&bars[slot], phase, ctl, kSiteXformFull);
            if (!ok) break;
            const uint32_t t = tb + c * 64 + slice * 32;
            switch (a.act) {
              case kActRelu: glu_grad_chunk<kActRelu>(t, buf, slice, ask); break;
              case kActSilu: glu_grad_chunk<kActSilu>(t, buf, slice, ask); break;
              case kActGeluTanh: glu_grad_chunk<kActGeluTanh>(t, buf, slice, ask); break;
              default: glu_grad_chunk<kActIdentity>(t, buf, slice, ask); break;
            }
            if (c == 3) release();
            fence_proxy_async_smem();
            __syncwarp();
            uint64_t* both = &made[q * Cfg::kSlots + slot];
            if (lane == 0) mbar_arrive(both);
            if (slice == 0) {
              ok = wait_bar(both, phase, ctl, kSiteXformEmpty);
              if (!ok) break;
              if (lane == 0) {
                const int col = u.nb * kMbTile + c * 64;
                if (row0 < j.rows && col < j.cols) {
                  tma_store_2d(&j.o[0], buf, col, row0, pol);
                  tma_store_2d(&j.o[1], buf + kGradBytes, col, row0, pol);
                }
                bulk_commit();
              }
            }
            if (++slot == Cfg::kSlots) {
              slot = 0;
              phase ^= 1;
            }
          }
          if (!ok) break;
        } else if (j.mode == kMbGlu) {
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {  // 64 columns of h, g and u each
            uint32_t g[32], up[32], w[16];
            tmem_ld32(tb + slice * 64 + c * 32, g);
            tmem_ld32(tb + 128 + slice * 64 + c * 32, up);
            tmem_wait_ld();
            if (c == 1) release();
            const int col = u.nb * 128 + slice * 64 + c * 32;
            auto put = [&](int o) {
              put_chunk<false>(bufs, kStageChunkBytes, flip, 0, w, &j.o[o], row0, col, j.rows,
                               j.cols, first);
            };
            glu_pack(a.act, g, up, w);
            put(0);
            pack32(g, w);
            put(1);
            pack32(up, w);
            put(2);
          }
        } else {
          const int col0 = u.nb * kMbTile + slice * 128;
          const uint32_t t = tb + slice * 128;
          if (j.splits > 1)
            store_part(t, release, j, bufs, flip, row0, col0, u.split);
          else
            store_tile(t, release, j, bufs, flip, row0, col0, first);
        }
      }
    }
    if (GRAD && !ok && lane == 0) {
      const uint64_t t0 = globaltimer_ns();  // let the copies in flight land (bounded)
      while (globaltimer_ns() - t0 < 2000000ull) __nanosleep(1000);
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

// dx from the parts of its K: added in their order in fp32, rounded once.
constexpr int kSumThreads = 256;
__global__ void __launch_bounds__(kSumThreads)
    mlp_sum_kernel(const float* __restrict__ parts, __nv_bfloat16* __restrict__ dx, int64_t n,
                   int64_t stride, int splits) {
  griddep_launch_dependents();
  griddep_wait();
  const int64_t step = static_cast<int64_t>(gridDim.x) * kSumThreads * 8;
  for (int64_t i = (static_cast<int64_t>(blockIdx.x) * kSumThreads + threadIdx.x) * 8; i < n;
       i += step) {
    float f[8];
    add_parts(f, splits, [&](int s) { return parts + s * stride + i; });
    st_u4(dx + i, pack8(f));
  }
}

template <int STREAMS, bool GRAD>
cudaError_t run_mb(const MbLaunch& launch, const KernelCtl& ctl, int grid, cudaStream_t stream) {
  static std::atomic<uint64_t> mask{0};
  auto kernel = mlp_train_kernel<STREAMS, GRAD>;
  constexpr int smem = MbCfg<STREAMS, GRAD>::kSmem;
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
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(kMbThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, launch, ctl);
}

}  // namespace

namespace {

MbDiv div_by(int d) {  // exact for 31-bit numbers: the reciprocal is rounded up
  MbDiv r;
  r.by = std::max(d, 1);
  int bits = 0;
  while ((int64_t(1) << bits) < r.by) ++bits;
  r.shift = bits - 1;  // of 1, whose reciprocal does not fit, unused
  r.mul = static_cast<uint32_t>(((uint64_t(1) << (31 + bits)) + r.by - 1) / r.by);
  return r;
}

// About how many cycles a unit keeps its pair, by its K blocks and its ending: from
// measured totals over rounds of units (h of 257 to 1024 rows x 2048 x 5632 and x 4096 x
// 14336, dh of 4096 x 4096 x 14336 and 2048 x 2048 x 8192, weights' gradients of 512 x
// 4096 x 14336 and 1021 x 1000 x 2728).  A lone row tile's MMAs take 150 cycles each,
// its 64 KB of operands per K block come from L2 at about the same pace, and its ending
// overlaps the next unit's; two row tiles' MMAs share the tensor pipe at 128 cycles, and
// the next unit waits for the first one's ending, of kMbGluGrad for both.
int64_t unit_cycles(int mode, int64_t kb, int streams) {
  switch (mode) {
    case kMbGluGrad:
      return streams == 1 ? std::max<int64_t>(800 * kb, 14000) + 300 : 1024 * kb + 20000;
    case kMbGlu: return streams == 1 ? 640 * kb + 4000 : 1120 * kb + 6500;
    default:
      return streams == 1 ? std::max<int64_t>(760 * kb, 2600) + 300
                          : std::max<int64_t>(1060 * kb, 5200) + 2600;
  }
}

}  // namespace

int64_t plan_mlp_launch(MbLaunch* l, int streams, int npairs) {
  int64_t work = 0, cycles[kMbJobs] = {};
  for (int i = 0; i < kMbJobs; ++i) {
    MbJob& j = l->job[i];
    j.units = 0;
    if (j.mode == kMbNone) continue;
    const int bn = j.mode == kMbGlu ? 128 : kMbTile;
    const int m_units = (j.rows + kMbTile * streams - 1) / (kMbTile * streams);
    const int n_tiles = (j.cols + bn - 1) / bn;
    j.units = m_units * n_tiles * j.splits;
    j.full_groups = m_units / kMbGroup;
    j.group = div_by(kMbGroup * n_tiles);
    j.last = div_by(m_units % kMbGroup);
    j.tiles = div_by(m_units * n_tiles);
    j.parts = div_by(j.splits);
    cycles[i] = unit_cycles(j.mode, (j.num_kb + j.splits - 1) / j.splits, streams);
    if (i > 0) work += j.units * cycles[i];
  }
  const int longs = l->job[0].units;
  l->shorts = 0;
  for (int i = 1; i < kMbJobs; ++i) l->shorts += l->job[i].units;
  l->pairs = std::max(1, std::min(npairs, longs + l->shorts));
  l->longs_each = longs / l->pairs;
  l->extra = longs % l->pairs;
  l->skip = 0;
  const int64_t begun = l->longs_each * cycles[0];
  const int64_t later = l->extra > 0 ? cycles[0] : 0;  // of the pairs with one long unit more
  if (l->shorts == 0) return begun + later;
  // rounds of short units that the others finish meanwhile, to the nearest
  const int64_t each = std::max<int64_t>(1, work / l->shorts);
  const int others = l->pairs - l->extra;
  l->skip = static_cast<int>(std::min<int64_t>((later + each / 2) / each,
                                               l->extra > 0 ? l->shorts / others + 1 : 0));
  const int64_t left = std::max<int64_t>(0, l->shorts - int64_t(l->skip) * others);
  const int64_t rounds = (left + l->pairs - 1) / l->pairs;
  return begun + std::max(later, l->skip * each) + rounds * each;
}

cudaError_t launch_mlp_train(const MbLaunch& launch, int streams, const KernelCtl& ctl,
                             cudaStream_t stream) {
  const int grid = 2 * launch.pairs;
  if (launch.job[0].mode == kMbGluGrad)  // alone
    return streams == 2 ? run_mb<2, true>(launch, ctl, grid, stream)
                        : run_mb<1, true>(launch, ctl, grid, stream);
  return streams == 2 ? run_mb<2, false>(launch, ctl, grid, stream)
                      : run_mb<1, false>(launch, ctl, grid, stream);
}

cudaError_t launch_mlp_sum(const float* parts, __nv_bfloat16* dx, int64_t n, int64_t stride,
                           int splits, int sms, cudaStream_t stream) {
  const int64_t ctas = std::min<int64_t>((n / 8 + kSumThreads - 1) / kSumThreads,
                                         static_cast<int64_t>(sms) * 8);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
  cfg.blockDim = dim3(kSumThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, mlp_sum_kernel, parts, dx, n, stride, splits);
}

}  // namespace gbf
