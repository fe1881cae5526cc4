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

// LISTS: the backward pass over lists, which puts the entries in shared memory.
template <int MPAD, bool LISTS = false>
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
  // per warp: 32 x 17 values to be transposed, or LISTS: a mask of columns per row and
  // the shares that it stands for
  static constexpr int kTurnWords = LISTS ? 832 : 32 * 17;
  static constexpr int kTurnBytes = 4 * kTurnWords * 4;
  static constexpr int kSmem = 1024 + kStages * kStageBytes + kBarBytes + kRowBytes + kTurnBytes;
  static_assert(2 * (kSmem + 1024) <= 227 * 1024, "two CTAs per SM");
  static_assert(kStageBytes % 1024 == 0, "stages stay 1024-byte aligned");
};

__device__ __forceinline__ float sw_pow2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// PICK: lists of columns with their shares instead of one target per row (CePick).
template <int MPAD, bool GRAD, bool PICK>
__global__ void __launch_bounds__(kSwThreads, 2)
    ce_swap_kernel(const __grid_constant__ CeSwap a, const CeEnd e, const KernelCtl kctl) {
  using Cfg = SwCfg<MPAD, PICK && GRAD>;
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
  // A tile's first block of K: by the column of W, so that both passes add in the same order.
  auto first_block = [&](int t) {
    return static_cast<int>(static_cast<unsigned>(a.v0 / 128 + t) * 13u %
                            static_cast<unsigned>(a.num_kb));
  };
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
  // The gradient's scored rows are listed by the kernel before.  The forward pass over
  // lists is launched by the kernel that makes them, once everything before that one
  // has completed: x and w are read meanwhile, and only the ending waits.
  // (So the lists are written while this kernel runs: they are read by plain loads, not
  // by those for data that is constant meanwhile.)
  constexpr bool kEarly = PICK && !GRAD;
  // The gradient's CTAs wait while the rows are listed; meanwhile their first blocks of W
  // go to L2, which would update them (64 rows x 32000 x 4096 trained 205.5 us, 6 blocks
  // each 203.6, 16 202.2).
  constexpr int kAhead = 16;
  if (GRAD && threadIdx.x == 0 && blockIdx.x * 128u < static_cast<unsigned>(a.cols)) {
    int kb = first_block(blockIdx.x);
    for (int i = 0; i < min(a.num_kb, kAhead); ++i) {
      tma_prefetch_l2_2d(&a.w, kb * kBK, a.v0 + static_cast<int>(blockIdx.x) * 128);
      if (++kb == a.num_kb) kb = 0;
    }
  }
  if (!kEarly) griddep_wait();
  const int count = GRAD ? *e.count : e.M;
  for (int i = threadIdx.x; i < MPAD; i += kSwThreads) {
    if (GRAD) {
      row_tgt[i] = i < count ? (PICK ? e.rows[i] : e.tgt[i] - a.v0) : -1;
      row_lse2[i] = i < count ? e.lse2[i] : 0.0f;
      row_dl[i] = i < count ? e.dl[i] : 0.0f;
    } else if (!PICK) {
      const int64_t t = i < count ? ce_target(a.targets, a.ids64, i) : -1;
      row_tgt[i] = t >= 0 && t < a.cols ? static_cast<int>(t) : -1;
    }
  }
  if (!GRAD && !PICK && blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0u;
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
      const uint64_t stream = policy_evict_first();
      const CUtensorMap* mx = &a.x[!GRAD || count == e.M ? 1 : 0];
      int fills = 0;
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < tiles && ok; t += step) {
        int kb = first_block(t);
        for (int i = 0; i < num_kb; ++i) {
          if (!wait_bar(&empty[s], ph ^ 1, ctl, kSiteProducerEmpty)) {
            ok = false;
            break;
          }
          uint8_t* sw = stages + s * Cfg::kStageBytes;
          mbar_arrive_expect_tx(&full[s], Cfg::kStageBytes);
          // W streams past the other operands in L2, but for the last eighth of each of its
          // rows, which the next pass may still find (64 rows x 32000 x 4096 trained
          // 214 us, without the hint 222, all of W 216; 128 rows scored 65, 69.5, 62.5).
          if (i < num_kb - num_kb / 8)
            tma_load_2d_hint(sw, &a.w, &full[s], kb * kBK, a.v0 + t * 128, stream);
          else
            tma_load_2d(sw, &a.w, &full[s], kb * kBK, a.v0 + t * 128);
          tma_load_2d(sw + kSwWBytes, mx, &full[s], kb * kBK, 0);
          ++fills;
          if (++s == kStages) {
            s = 0;
            ph ^= 1;
          }
          if (++kb == num_kb) kb = 0;
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
    if (kEarly) {
      griddep_wait();
      if (blockIdx.x == 0 && threadIdx.x == 64) *a.ticket = 0u;
    }
    const int q = warp & 3;  // the quarter of tensor memory that this warp reads
    float* my_turn = turn + q * Cfg::kTurnWords;
    const int chunks = (count + 15) / 16;  // of 16 rows
    // sums of the segments before: [row][column], this thread's column
    float* part = e.chain + static_cast<int64_t>(blockIdx.x) * MPAD * 128 + q * 32 + lane;
    int seg = 0;
    for (int t = blockIdx.x, l = 0; t < tiles; ++l) {
      const int buf = l & two_bufs;
      float before[16];  // of the next 16 rows, on their way meanwhile
      // PICK: rows lane, lane + 32, ...: number, and entries in this warp's 32 columns
      constexpr int kRows = PICK ? (MPAD + 31) / 32 : 1;
      int pick_row[kRows], pick_at[kRows], pick_n[kRows];
      if constexpr (PICK) {
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          const int m = i * 32 + lane;
          pick_row[i] = pick_at[i] = pick_n[i] = 0;
          if (seg + seg_kb >= num_kb && m < count && t * 128 + q * 32 < a.cols) {
            pick_row[i] = GRAD ? row_tgt[m] : m;
            const uint16_t* at = e.pick.at + static_cast<int64_t>(pick_row[i]) * e.pick.stride +
                                 ((a.v0 + t * 128 + q * 32) >> 5);
            pick_at[i] = at[0];
            pick_n[i] = at[1] - pick_at[i];
          }
        }
      }
      // Those of one i, by masks: a choice of the language's puts the arrays in local memory.
      auto take = [&](bool it, int i, int& row, int& at, int& n) {
        const int mask = it ? -1 : 0;
        row |= pick_row[i] & mask;
        at |= pick_at[i] & mask;
        n |= pick_n[i] & mask;
      };
      // GRAD: one entry of each of the rows 8 g .. 8 g + 7 per lane, (-1, 0) where there
      // is none.
      auto entries = [&](int g, int2 (&x)[8]) {
        int row_g = 0, at_g = 0, n_g = 0;
#pragma unroll
        for (int i = 0; i < kRows; ++i)
          take(g / 4 == i, i, row_g, at_g, n_g);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int from = 8 * (g & 3) + k;
          const int64_t row = __shfl_sync(0xFFFFFFFFu, row_g, from);
          const int at = __shfl_sync(0xFFFFFFFFu, at_g, from);
          const int n = __shfl_sync(0xFFFFFFFFu, n_g, from);
          x[k] = make_int2(-1, 0);
          if (lane < n) x[k] = e.pick.list[row * (e.pick.K + 1) + at + lane];
        }
      };
      // The entries go to shared memory while the products are on their way: beside the
      // stream of W a load from L2 takes microseconds, also a second one of the same
      // line (64 rows x 32000 x 4096, read in the ending 58 us, staged 49).  Rows from
      // `staged` on, of a warp with more entries than there is room for, are read there.
      constexpr int kRoom = Cfg::kTurnWords - MPAD;
      uint32_t* masks = reinterpret_cast<uint32_t*>(my_turn);
      float* shares = my_turn + MPAD;
      int staged = MPAD;
      if constexpr (PICK && GRAD) {
        if (seg + seg_kb >= num_kb) {
          __syncwarp();
          int before_row = 0;  // entries of the rows before
#pragma unroll
          for (int i = 0; i < kRows; ++i) {  // a lane per row
            const int m = i * 32 + lane;
            int at = pick_n[i];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const int up = __shfl_up_sync(0xFFFFFFFFu, at, o);
              if (lane >= o) at += up;
            }
            const int all = __shfl_sync(0xFFFFFFFFu, at, 31);
            at += before_row - pick_n[i];
            before_row += all;
            const unsigned over = __ballot_sync(0xFFFFFFFFu, at + pick_n[i] > kRoom);
            if (over) staged = min(staged, i * 32 + __ffs(over) - 1);
            uint32_t cols = 0u;
            if (at + pick_n[i] <= kRoom) {
              const int2* list =
                  e.pick.list + static_cast<int64_t>(pick_row[i]) * (e.pick.K + 1) + pick_at[i];
              for (int k0 = 0; k0 < pick_n[i]; k0 += 4) {  // four loads in flight
                int2 x[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  if (k0 + k < pick_n[i]) x[k] = list[k0 + k];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  if (k0 + k >= pick_n[i]) continue;
                  cols |= 1u << (x[k].x - (a.v0 + t * 128 + q * 32));
                  shares[at + k0 + k] = __int_as_float(x[k].y);
                }
              }
            }
            if (m < MPAD) masks[m] = cols;
          }
          __syncwarp();
        }
      }
      int taken = 0;  // shares of the rows before
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
        // the same of the chunk's rows: lanes 16 (c & 1) + k
        int row_c = 0, at_c = 0, n_c = 0;
        if constexpr (PICK) {
#pragma unroll
          for (int i = 0; i < kRows; ++i)
            take(c / 2 == i, i, row_c, at_c, n_c);
        }
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
          float f[16], dl[16], lse2[16];
#pragma unroll
          for (int k = 0; k < 16; k += 4) {
            *reinterpret_cast<float4*>(dl + k) = *reinterpret_cast<const float4*>(row_dl + c * 16 + k);
            *reinterpret_cast<float4*>(lse2 + k) = *reinterpret_cast<const float4*>(row_lse2 + c * 16 + k);
          }
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const int m = c * 16 + k;
            f[k] = 0.0f;
            if (m < count) {
              const float p = sw_pow2(fmaf(v[k], e.c2, -lse2[k]));
              if constexpr (PICK) f[k] = p;
              else f[k] = dl[k] * (row_tgt[m] == col ? p - 1.0f : p);
            }
          }
          if constexpr (PICK) {
            // A row's entries here are at most 32, and their columns differ and ascend: a
            // lane finds its own column's by counting the columns below it.
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const unsigned some = __ballot_sync(0xFFFFFFFFu, n_c > 0) >> (16 * (c & 1) + 8 * h);
              if (!(some & 0xFFu)) continue;
              if (c * 16 + 8 * h + 8 <= staged) {
                uint32_t cols[8];
                *reinterpret_cast<uint4*>(cols) = *reinterpret_cast<const uint4*>(masks + c * 16 + 8 * h);
                *reinterpret_cast<uint4*>(cols + 4) =
                    *reinterpret_cast<const uint4*>(masks + c * 16 + 8 * h + 4);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  const int i = taken + __popc(cols[k] & ((1u << lane) - 1u));
                  if ((cols[k] >> lane) & 1u) f[8 * h + k] -= shares[i];
                  taken += __popc(cols[k]);
                }
                continue;
              }
              int2 x[8];
              entries(2 * c + h, x);
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const int m = c * 16 + 8 * h + k;
                uint32_t cols;
                float share;
                if (m < staged) {
                  cols = masks[m];
                  const int i = taken + __popc(cols & ((1u << lane) - 1u));
                  share = (cols >> lane) & 1u ? shares[i] : 0.0f;
                  taken += __popc(cols);
                } else {
                  cols = __reduce_or_sync(
                      0xFFFFFFFFu, x[k].x < 0 ? 0u : 1u << (x[k].x - (a.v0 + t * 128 + q * 32)));
                  share = __int_as_float(__shfl_sync(0xFFFFFFFFu, x[k].y,
                                                     __popc(cols & ((1u << lane) - 1u))));
                  if (!((cols >> lane) & 1u)) share = 0.0f;
                }
                f[8 * h + k] -= share;
              }
            }
#pragma unroll
            for (int k = 0; k < 16; ++k)
              if (c * 16 + k < count) f[k] *= dl[k];
          }
          if (col < a.cols) {
            constexpr bool kTwice = PICK && MPAD <= kCeTwiceRows;
            __nv_bfloat16* dst =
                a.gt + static_cast<int64_t>(col) * (kTwice ? 2 * MPAD : MPAD) + c * 16;
            float lo[8], hi[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              lo[k] = f[k];
              hi[k] = f[8 + k];
            }
            st_u4(dst, pack8(lo));
            st_u4(dst + 8, pack8(hi));
            if constexpr (kTwice) {  // what the first rounding left
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                lo[k] -= __bfloat162float(__float2bfloat16_rn(lo[k]));
                hi[k] -= __bfloat162float(__float2bfloat16_rn(hi[k]));
              }
              st_u4(dst + MPAD, pack8(lo));
              st_u4(dst + MPAD + 8, pack8(hi));
            }
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
          // each row's entries by the lane that holds their places
          if constexpr (PICK) {
            if (lane / 16 == (c & 1)) {
              const int2* list = e.pick.list + static_cast<int64_t>(row_c) * (e.pick.K + 1) + at_c;
              float* dots = e.pick.dots + static_cast<int64_t>(row_c) * e.pick.K + at_c;
              for (int i0 = 0; i0 < n_c; i0 += 8) {  // eight loads in flight
                int col8[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) col8[i] = i0 + i < n_c ? list[i0 + i].x : base;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  if (i0 + i < n_c) dots[i0 + i] = my_turn[(col8[i] - base) * 17 + (lane & 15)];
              }
            }
          }
          if (lane < 16 && m < count) {
            e.part[static_cast<int64_t>(4 * t + q) * e.M + m] = make_float2(m2, sum);
            if constexpr (!PICK) {
              const int at = row_tgt[m] - base;
              if (row_tgt[m] >= 0 && at >= 0 && at < 32) e.tlog[m] = my_turn[at * 17 + lane];
            }
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

template <int MPAD, bool GRAD, bool PICK>
cudaError_t run_swap(const CeSwap& a, const CeEnd& end, const KernelCtl& ctl, int grid,
                     cudaStream_t stream) {
  static std::atomic<uint64_t> mask{0};
  auto kernel = ce_swap_kernel<MPAD, GRAD, PICK>;
  constexpr int smem = SwCfg<MPAD, PICK && GRAD>::kSmem;
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

template <bool GRAD, bool PICK>
static cudaError_t run_swap_rows(const CeSwap& a, const CeEnd& end, const KernelCtl& ctl, int grid,
                                 cudaStream_t stream) {
  switch (ce_swap_rows(end.M)) {
    case 16: return run_swap<16, GRAD, PICK>(a, end, ctl, grid, stream);
    case 64: return run_swap<64, GRAD, PICK>(a, end, ctl, grid, stream);
    case 128: return run_swap<128, GRAD, PICK>(a, end, ctl, grid, stream);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_ce_swap(const CeSwap& a, bool grad, const CeEnd& end, int sms,
                           const KernelCtl& ctl, cudaStream_t stream) {
  const int grid = std::min((a.cols + 127) / 128, 2 * sms);
  if (end.pick.list)
    return grad ? run_swap_rows<true, true>(a, end, ctl, grid, stream)
                : run_swap_rows<false, true>(a, end, ctl, grid, stream);
  return grad ? run_swap_rows<true, false>(a, end, ctl, grid, stream)
              : run_swap_rows<false, false>(a, end, ctl, grid, stream);
}

}  // namespace gbf
