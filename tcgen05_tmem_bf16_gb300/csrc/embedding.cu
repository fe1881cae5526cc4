// embedding.cu -- the embedding lookup with scaling and its gradient.
//
// Lookup: out[m] = bf16(scale * table[id_m]), zeros for an id outside [0, V).
// HBM-bound: a warp moves 1024 columns of one row, four 16-byte vectors per
// lane in flight (16383 rows of 8192: 59 us, 334 MB of 510 from and to HBM).
//
// Gradient: dtable[v] (+)= scale * sum over {m : id_m = v} of dout[m], in
// fp32, in the order of m.  Summing with atomics would add in an order that
// changes from run to run, so the positions are sorted by id first and the
// sorted list is cut into pieces of equal length, however the ids repeat:
//   1. embed_sort_kernel: the positions in the order of (id, m), by a stable
//      radix sort inside one cluster of CTAs;
//   2. embed_sum_kernel: one piece of the list x 1024 columns per CTA.  A run
//      of equal ids inside the piece is summed and written; the part of a run
//      that continues from the previous piece or into the next one goes to the
//      workspace in fp32.  Without accumulation further CTAs write the
//      zero rows of the ids that do not occur;
//   3. embed_join_kernel: the runs over several pieces, their parts added in
//      order, written once.
// Up to 1024 positions one kernel does without sorting (embed_direct_kernel).
// HBM-bound but for the sort: 16384 x 4096 into a tied table of 128000 rows takes
// 64.5 us, 15 of them the sort (twelve short phases that wait on one another),
// 42 the sums (5 to 6.4 TB/s), 8 the join.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "internal.h"

namespace gbf {

namespace {

constexpr int kLookThreads = 128;
constexpr int kSegCols = 1024;  // columns per warp (lookup) or CTA (gradient)

template <typename Id>
__global__ void __launch_bounds__(kLookThreads)
    embed_lookup_kernel(const Id* __restrict__ ids, const __nv_bfloat16* __restrict__ table,
                        __nv_bfloat16* __restrict__ out, int64_t M, int64_t V, int D, int segs,
                        float scale) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t task =
      static_cast<int64_t>(blockIdx.x) * (kLookThreads / 32) + (threadIdx.x >> 5);
  const int64_t m = task / segs;
  if (m >= M) return;
  const int col0 = static_cast<int>(task - m * segs) * kSegCols + lane * 8;
  const int64_t id = static_cast<int64_t>(ids[m]);
  const bool known = id >= 0 && id < V;
  const __nv_bfloat16* src = table + (known ? id : 0) * D;
  __nv_bfloat16* dst = out + m * D;
  uint4 v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int col = col0 + i * 256;
    v[i] = (known && col < D) ? ldg_u4(src + col) : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int col = col0 + i * 256;
    if (col < D) {
      float f[8];
      unpack8(v[i], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] *= scale;
      // 0 * inf must not reach the row of an unknown id
      st_u4(dst + col, known ? pack8(f) : make_uint4(0u, 0u, 0u, 0u));
    }
  }
}

// ---------------------------------------------------------------- sort
//
// Stable least-significant-digit radix sort of (id, m) by one cluster: CTA c
// holds the c-th contiguous share of the list, warp w the w-th of the CTA's.
// Per pass: every warp counts its digits, the counts are summed over warps
// and CTAs (one CTA's totals are read by the others from its shared memory),
// and every warp writes its items to their places, 32 at a time, ranked among
// equal digits by lane.  Ids outside [0, V) get the key V and end the list.
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxDigitBits = 9;
constexpr int kMaxDigits = 1 << kMaxDigitBits;
constexpr int kSortCluster = 8;
constexpr size_t kSortSmem = (kSortWarps + 2) * kMaxDigits * sizeof(int);

__device__ __forceinline__ int ld_cg(const int* p) { return __ldcg(p); }

__device__ __forceinline__ int ld_dsmem_s32(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

template <typename Id>
__global__ void __launch_bounds__(kSortThreads)
    embed_sort_kernel(const Id* __restrict__ ids, int M, int V, int passes, int digit_bits,
                      int* key0, int* idx0, int* key1, int* idx1) {
  extern __shared__ int sort_smem[];
  __shared__ int warp_sum[kSortWarps];
  int* hist = sort_smem;                            // [warps][digits]
  int* total = sort_smem + kSortWarps * kMaxDigits;  // this CTA's digit counts
  int* base = total + kMaxDigits;                    // where this CTA's digits begin
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  constexpr int ctas = kSortCluster;
  const int rank = static_cast<int>(cluster_ctarank());
  const int digits = 1 << digit_bits;
  griddep_launch_dependents();
  griddep_wait();
  // contiguous shares, multiples of 32 so that a warp's steps are full but the last
  const int64_t share =
      ((static_cast<int64_t>(M) + ctas * kSortWarps - 1) / (ctas * kSortWarps) + 31) / 32 * 32;
  const int64_t lo64 = (static_cast<int64_t>(rank) * kSortWarps + warp) * share;
  const int lo = static_cast<int>(min(lo64, static_cast<int64_t>(M)));
  const int hi = static_cast<int>(min(lo64 + share, static_cast<int64_t>(M)));
  int* const my_hist = hist + warp * kMaxDigits;
  for (int pass = 0; pass < passes; ++pass) {
    const int shift = pass * digit_bits;
    const int* ksrc = (pass & 1) ? key0 : key1;
    const int* isrc = (pass & 1) ? idx0 : idx1;
    int* kdst = (pass & 1) ? key1 : key0;
    int* idst = (pass & 1) ? idx1 : idx0;
    auto key_at = [&](int i) -> int {
      if (pass > 0) return ld_cg(ksrc + i);
      const int64_t id = static_cast<int64_t>(ids[i]);
      return (id >= 0 && id < V) ? static_cast<int>(id) : V;
    };
    // the first steps' items stay in registers from counting to placing
    constexpr int kKept = 4;
    int kept_key[kKept], kept_idx[kKept];
#pragma unroll
    for (int k = 0; k < kKept; ++k) {
      const int i = lo + k * 32 + lane;
      kept_key[k] = i < hi ? key_at(i) : 0;
      kept_idx[k] = i < hi ? (pass > 0 ? ld_cg(isrc + i) : i) : 0;
    }
    for (int d = lane; d < digits; d += 32) my_hist[d] = 0;
    __syncwarp();
    // the lanes with an item of the same digit, by one vote per bit
    auto alike = [&](bool in, int key) -> unsigned {
      unsigned same = __ballot_sync(0xFFFFFFFFu, in);
      for (int b = 0; b < digit_bits; ++b) {
        const bool one = (key >> (shift + b)) & 1;
        const unsigned ones = __ballot_sync(0xFFFFFFFFu, one);
        same &= one ? ones : ~ones;
      }
      return same;
    };
    auto count = [&](bool in, int key) -> unsigned {
      const unsigned same = alike(in, key);
      if (in && lane == __ffs(same) - 1) my_hist[(key >> shift) & (digits - 1)] += __popc(same);
      __syncwarp();
      return same;
    };
    unsigned kept_same[kKept];
#pragma unroll
    for (int k = 0; k < kKept; ++k)
      if (lo + k * 32 < hi) kept_same[k] = count(lo + k * 32 + lane < hi, kept_key[k]);
    for (int i0 = lo + kKept * 32; i0 < hi; i0 += 32) {
      const bool in = i0 + lane < hi;
      count(in, in ? key_at(i0 + lane) : 0);
    }
    __syncthreads();
    // per digit: this CTA's count, and each warp's offset within it
    for (int d = threadIdx.x; d < digits; d += kSortThreads) {
      int n[kSortWarps];
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) n[w] = hist[w * kMaxDigits + d];
      int sum = 0;
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) {
        hist[w * kMaxDigits + d] = sum;
        sum += n[w];
      }
      total[d] = sum;
    }
    cluster_sync_all();  // every CTA's counts are written
    // per digit: the count over all CTAs and that of the CTAs before this one;
    // then where the digit begins: a scan over the digits of each warp's 32 and
    // over the warps
    {
      const int d = threadIdx.x;  // digits <= kSortThreads
      int all = 0, before = 0;
      if (d < digits) {
        const uint32_t at = smem_u32(&total[d]);
        int n[kSortCluster];
#pragma unroll
        for (int c = 0; c < kSortCluster; ++c)
          n[c] = ld_dsmem_s32(mapa_shared(at, c));
#pragma unroll
        for (int c = 0; c < kSortCluster; ++c) {
          if (c < rank) before += n[c];
          all += n[c];
        }
      }
      int x = all;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += y;
      }
      if (lane == 31) warp_sum[warp] = x;
      __syncthreads();
      int earlier = lane < warp ? warp_sum[lane] : 0;
      earlier = __reduce_add_sync(0xFFFFFFFFu, earlier);
      if (d < digits) base[d] = earlier + x - all + before;
    }
    __syncthreads();
    auto place = [&](bool in, int key, int idx, unsigned same) {
      const int d = (key >> shift) & (digits - 1);
      int at = 0;
      if (in) at = base[d] + my_hist[d] + __popc(same & ((1u << lane) - 1u));
      __syncwarp();
      if (in && lane == __ffs(same) - 1) my_hist[d] += __popc(same);
      __syncwarp();
      if (in) {
        kdst[at] = key;
        idst[at] = idx;
      }
    };
#pragma unroll
    for (int k = 0; k < kKept; ++k)
      if (lo + k * 32 < hi) place(lo + k * 32 + lane < hi, kept_key[k], kept_idx[k], kept_same[k]);
    for (int i0 = lo + kKept * 32; i0 < hi; i0 += 32) {
      const int i = i0 + lane;
      const bool in = i < hi;
      const int key = in ? key_at(i) : 0;
      place(in, key, in ? (pass > 0 ? ld_cg(isrc + i) : i) : 0, alike(in, key));
    }
    cluster_sync_all();  // the pass is written before the next one reads it
  }
}

// ---------------------------------------------------------------- sums

constexpr int kSumThreads = 128;
constexpr int kMaxPiece = 32;  // sorted positions per piece at most

struct SumArgs {
  const int* key;   // sorted ids, V for the unknown ones
  const int* idx;   // their positions
  const __nv_bfloat16* dout;
  __nv_bfloat16* dtable;
  float* head;      // [pieces][D]: the part of a run that began in an earlier piece
  float* tail;      // [pieces][D]: the part of a run that goes on in the next piece
  int M, V, D;
  int piece;        // positions per piece
  int pieces;
  int segs;         // column segments
  float scale;
  int accumulate;
};

// `old`: the row's present values, where they are added to.
__device__ __forceinline__ void write_row(const SumArgs& a, int64_t v, int col,
                                          const float (&sum)[8], const uint4& old) {
  __nv_bfloat16* p = a.dtable + v * a.D + col;
  float f[8];
  if (a.accumulate) {
    unpack8(old, f);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = fmaf(a.scale, sum[j], f[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = a.scale * sum[j];
  }
  st_u4(p, pack8(f));
}

__device__ __forceinline__ void store_part(float* p, const float (&sum)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(sum[0], sum[1], sum[2], sum[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(sum[4], sum[5], sum[6], sum[7]);
}

// The first position of the sorted list whose key is not under `key`, by one
// warp, 32 places looked at together.
__device__ __forceinline__ int lower_bound(const int* keys, int n, int key) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n;  // every position before lo is under, none from hi on
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32;
    const int64_t at = lo + static_cast<int64_t>(lane + 1) * step - 1;
    const bool under = at < hi && keys[at] < key;
    const int k = __popc(__ballot_sync(0xFFFFFFFFu, under));
    const int64_t next = lo + static_cast<int64_t>(k) * step;
    hi = static_cast<int>(min(static_cast<int64_t>(hi), next + step - 1));
    lo = static_cast<int>(min(next, static_cast<int64_t>(hi)));
  }
  return lo;
}

constexpr int kZeroRows = 1024;  // rows looked for at a time

// Writes the zero rows of the me-th of `ctas` equal shares of the table.
// mark(first, rows, found) sets a bit for each of the rows from `first` on that
// an id asks for.
template <typename Mark>
__device__ __forceinline__ void zero_rows(const SumArgs& a, int64_t me, int64_t ctas, Mark mark) {
  __shared__ unsigned found[kZeroRows / 32];
  const int64_t v0 = a.V * me / ctas, v1 = a.V * (me + 1) / ctas;
  for (int64_t first = v0; first < v1; first += kZeroRows) {
    const int rows = static_cast<int>(min(static_cast<int64_t>(kZeroRows), v1 - first));
    for (int i = threadIdx.x; i < kZeroRows / 32; i += kSumThreads) found[i] = 0u;
    __syncthreads();
    mark(first, rows, found);
    __syncthreads();
    for (int r = 0; r < rows; ++r) {
      if ((found[r >> 5] >> (r & 31)) & 1u) continue;
      for (int c = threadIdx.x * 8; c < a.D; c += kSumThreads * 8)
        st_u4(a.dtable + (first + r) * a.D + c, make_uint4(0u, 0u, 0u, 0u));
    }
    __syncthreads();
  }
}

// Up to 1024 positions nothing is sorted: the CTA of position m (x 1024
// columns) looks through all ids, leaves if one before m is the same, and else
// sums the rows of those that are, in order.  One launch, no parts to join.
// (1021 ids x 1024 into 32000 rows: 16.4 us, 21.3 sorted; 1024 x 4096 into a tied
// table 9.4, 11.7 sorted; 4096 x 4096 69.7, 24.2 sorted; 1024 ids all the same
// 55, 1025 sorted 18.)
constexpr int kDirectMax = 1024;

template <typename Id>
__global__ void __launch_bounds__(kSumThreads)
    embed_direct_kernel(const Id* __restrict__ ids, const SumArgs a) {
  __shared__ int keys[kDirectMax];
  __shared__ int same[kDirectMax];
  __shared__ int count;
  griddep_launch_dependents();
  griddep_wait();
  const int64_t sums = static_cast<int64_t>(a.M) * a.segs;
  if (static_cast<int64_t>(blockIdx.x) >= sums) {
    zero_rows(a, blockIdx.x - sums, gridDim.x - sums,
              [&](int64_t first, int rows, unsigned* found) {
                for (int i = threadIdx.x; i < a.M; i += kSumThreads) {
                  const int64_t r = static_cast<int64_t>(ids[i]) - first;
                  if (r >= 0 && r < rows) atomicOr(&found[r >> 5], 1u << (r & 31));
                }
              });
    return;
  }
  const int m = static_cast<int>(blockIdx.x / a.segs);
  const int seg = static_cast<int>(blockIdx.x - static_cast<int64_t>(m) * a.segs);
  for (int i = threadIdx.x; i < a.M; i += kSumThreads) {
    const int64_t id = static_cast<int64_t>(ids[i]);
    keys[i] = (id >= 0 && id < a.V) ? static_cast<int>(id) : a.V;
  }
  __syncthreads();
  const int key = keys[m];
  bool earlier = key == a.V;
  for (int i = threadIdx.x; i < m; i += kSumThreads) earlier |= keys[i] == key;
  if (__syncthreads_or(earlier)) return;
  if (threadIdx.x < 32) {
    int n = 0;
    for (int i0 = m; i0 < a.M; i0 += 32) {
      const int i = i0 + static_cast<int>(threadIdx.x);
      const bool hit = i < a.M && keys[i] == key;
      const unsigned hits = __ballot_sync(0xFFFFFFFFu, hit);
      if (hit) same[n + __popc(hits & ((1u << threadIdx.x) - 1u))] = i;
      n += __popc(hits);
    }
    if (threadIdx.x == 0) count = n;
  }
  __syncthreads();
  const int col = seg * kSegCols + threadIdx.x * 8;
  if (col >= a.D) return;
  const int n = count;
  const uint4 old = a.accumulate ? ld_u4(a.dtable + static_cast<int64_t>(key) * a.D + col)
                                 : make_uint4(0u, 0u, 0u, 0u);
  float sum[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) sum[j] = 0.0f;
  constexpr int kAhead = 8;
  for (int i0 = 0; i0 < n; i0 += kAhead) {
    uint4 v[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (i0 + u < n) v[u] = ldg_u4(a.dout + static_cast<int64_t>(same[i0 + u]) * a.D + col);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (i0 + u >= n) break;
      float f[8];
      unpack8(v[u], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] += f[j];
    }
  }
  write_row(a, key, col, sum, old);
}

// CTAs [0, pieces * segs): sums; the rest: the zero rows of equal shares of the
// table, those that the sorted list does not hold.
__global__ void __launch_bounds__(kSumThreads) embed_sum_kernel(const SumArgs a) {
  __shared__ int skey[kMaxPiece + 2];
  __shared__ int sidx[kMaxPiece];
  griddep_launch_dependents();
  griddep_wait();
  const int64_t sums = static_cast<int64_t>(a.pieces) * a.segs;
  if (static_cast<int64_t>(blockIdx.x) >= sums) {
    __shared__ int begin;
    zero_rows(a, blockIdx.x - sums, gridDim.x - sums,
              [&](int64_t first, int rows, unsigned* found) {
                if (threadIdx.x < 32) {
                  const int at = lower_bound(a.key, a.M, static_cast<int>(first));
                  if (threadIdx.x == 0) begin = at;
                }
                __syncthreads();
                for (int64_t i = static_cast<int64_t>(begin) + threadIdx.x; i < a.M;
                     i += kSumThreads) {
                  const int64_t r = a.key[i] - first;
                  if (r >= rows) break;
                  atomicOr(&found[r >> 5], 1u << (r & 31));
                }
              });
    return;
  }
  const int p = static_cast<int>(blockIdx.x / a.segs);
  const int seg = static_cast<int>(blockIdx.x - static_cast<int64_t>(p) * a.segs);
  const int64_t first = static_cast<int64_t>(p) * a.piece;
  const int n = static_cast<int>(min(static_cast<int64_t>(a.piece), a.M - first));
  // the keys before and after the piece tell whether its runs go on
  for (int i = threadIdx.x; i < n + 2; i += kSumThreads) {
    const int64_t at = first + i - 1;
    skey[i] = (at >= 0 && at < a.M) ? a.key[at] : -1;
  }
  for (int i = threadIdx.x; i < n; i += kSumThreads) sidx[i] = a.idx[first + i];
  __syncthreads();
  const int col = seg * kSegCols + threadIdx.x * 8;
  if (col >= a.D) return;
  float sum[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) sum[j] = 0.0f;
  bool began = skey[0] != skey[1];  // the current run began in this piece
  // eight positions' rows, and the table's rows that end a run among them, are
  // loaded before the first is added
  constexpr int kAhead = 8;
  for (int i0 = 0; i0 < n; i0 += kAhead) {
    uint4 v[kAhead], old[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (i0 + u < n && skey[i0 + u + 1] < a.V) {
        const int key = skey[i0 + u + 1];
        v[u] = ldg_u4(a.dout + static_cast<int64_t>(sidx[i0 + u]) * a.D + col);
        if (a.accumulate && skey[i0 + u + 2] != key)
          old[u] = ld_u4(a.dtable + static_cast<int64_t>(key) * a.D + col);
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = i0 + u;
      if (i >= n) break;
      const int key = skey[i + 1];
      if (key >= a.V) return;  // the unknown ids end the list
      float f[8];
      unpack8(v[u], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] += f[j];
      const bool ends = skey[i + 2] != key;
      if (ends || i + 1 == n) {
        if (began && ends)
          write_row(a, key, col, sum, old[u]);
        else
          store_part((began ? a.tail : a.head) + static_cast<int64_t>(p) * a.D + col, sum);
        began = true;
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] = 0.0f;
      }
    }
  }
}

// Adds up to sum the parts [q0, q1) of a run, in order, eight in flight.
__device__ __forceinline__ void add_parts(const SumArgs& a, const float* base, int q0, int q1,
                                          int col, float (&sum)[8]) {
  constexpr int kAhead = 8;
  for (; q0 < q1; q0 += kAhead) {
    float4 g[kAhead][2];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (q0 + u < q1) {
        const float4* t = reinterpret_cast<const float4*>(base + static_cast<int64_t>(q0 + u) * a.D + col);
        g[u][0] = t[0];
        g[u][1] = t[1];
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (q0 + u >= q1) break;
      sum[0] += g[u][0].x; sum[1] += g[u][0].y; sum[2] += g[u][0].z; sum[3] += g[u][0].w;
      sum[4] += g[u][1].x; sum[5] += g[u][1].y; sum[6] += g[u][1].z; sum[7] += g[u][1].w;
    }
  }
}

// How many pieces from `piece` on begin with `key`: as many as the CTA has
// threads looked at together.
__device__ __forceinline__ int pieces_begun(const SumArgs& a, int64_t piece, int key) {
  int n = 0;
  for (;;) {
    const int64_t at = (piece + n + threadIdx.x) * a.piece;
    const int here = __syncthreads_count(at < a.M && a.key[at] == key);
    n += here;
    if (here < static_cast<int>(blockDim.x)) return n;
  }
}

// Runs with parts in more than this many pieces after their first are long.
constexpr int kLongRun = 64;
constexpr int kLongCols = 256;  // columns of a CTA that joins a long run
constexpr int kRanges = kSumThreads / 32;

// A long run (an id that fills much of a long list, such as a padding token that
// is not -1): the run that goes on into piece 64 k, if it did not into the one 64
// before.  256 columns per CTA: the parts are cut into four ranges, one for each
// warp, whose sums are added in order.  (16384 ids, half of them the same, D =
// 1024: 122 us with the runs' own CTAs alone, 48 so.)
__device__ __forceinline__ void join_long(const SumArgs& a, int k, int block) {
  __shared__ float range_sum[kRanges - 1][8][32];
  const int b = k * kLongRun;  // a piece that begins inside the run
  const int64_t at = static_cast<int64_t>(b) * a.piece;
  if (at >= a.M) return;
  const int key = a.key[at];
  if (key >= a.V || a.key[at - 1] != key) return;
  const int64_t earlier = static_cast<int64_t>(b - kLongRun) * a.piece;
  if (earlier > 0 && a.key[earlier] == key && a.key[earlier - 1] == key) return;  // of k - 1
  // the run began in the piece before the earliest whose beginning is inside it
  const int64_t before = static_cast<int64_t>(b - static_cast<int>(threadIdx.x)) * a.piece;
  const int inside = __syncthreads_count(static_cast<int>(threadIdx.x) < kLongRun && before > 0 &&
                                         a.key[before > 0 ? before - 1 : 0] == key);
  const int p = b - inside;
  const int more = b - 1 - p + pieces_begun(a, b, key);
  if (more <= kLongRun) return;
  const int range = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int col = block * kLongCols + lane * 8;
  const bool in = col < a.D;
  float sum[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) sum[j] = 0.0f;
  if (in) {
    if (range == 0) add_parts(a, a.tail, p, p + 1, col, sum);
    const int each = (more + kRanges - 1) / kRanges;
    add_parts(a, a.head, p + 1 + range * each, p + 1 + min(more, (range + 1) * each), col, sum);
    if (range > 0)
#pragma unroll
      for (int j = 0; j < 8; ++j) range_sum[range - 1][j][lane] = sum[j];
  }
  __syncthreads();
  if (!in || range > 0) return;
#pragma unroll
  for (int r = 0; r < kRanges - 1; ++r)
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[j] += range_sum[r][j][lane];
  write_row(a, key, col, sum,
            a.accumulate ? ld_u4(a.dtable + static_cast<int64_t>(key) * a.D + col)
                         : make_uint4(0u, 0u, 0u, 0u));
}

// One CTA per piece x segment: where the piece's last run began in it and goes
// on, adds the run's parts in order and writes the row.  Long runs are left to
// the CTAs after those.
__global__ void __launch_bounds__(kSumThreads) embed_join_kernel(const SumArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int64_t runs = static_cast<int64_t>(a.pieces) * a.segs;
  if (static_cast<int64_t>(blockIdx.x) >= runs) {
    const int64_t t = blockIdx.x - runs;
    const int blocks = (a.D + kLongCols - 1) / kLongCols;
    const int k = static_cast<int>(t / blocks);
    join_long(a, k + 1, static_cast<int>(t - static_cast<int64_t>(k) * blocks));
    return;
  }
  const int p = static_cast<int>(blockIdx.x / a.segs);
  const int seg = static_cast<int>(blockIdx.x - static_cast<int64_t>(p) * a.segs);
  const int64_t next = static_cast<int64_t>(p + 1) * a.piece;  // first position after the piece
  if (next >= a.M) return;
  const int key = a.key[next - 1];
  if (key >= a.V || a.key[next] != key) return;                     // the last run ends here
  const int64_t first = static_cast<int64_t>(p) * a.piece;
  if (a.key[first] == key && first > 0 && a.key[first - 1] == key) return;  // began earlier
  const int more = pieces_begun(a, p + 1, key);
  const int col = seg * kSegCols + threadIdx.x * 8;
  if (more > kLongRun || col >= a.D) return;
  const uint4 old = a.accumulate ? ld_u4(a.dtable + static_cast<int64_t>(key) * a.D + col)
                                 : make_uint4(0u, 0u, 0u, 0u);
  float sum[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) sum[j] = 0.0f;
  add_parts(a, a.tail, p, p + 1, col, sum);
  add_parts(a, a.head, p + 1, p + 1 + more, col, sum);
  write_row(a, key, col, sum, old);
}

// A launch that may begin while the previous kernel of the stream finishes:
// every kernel here waits for it before it reads or writes memory.
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

int bit_length(int64_t x) {
  int n = 0;
  while (x > 0) {
    ++n;
    x >>= 1;
  }
  return n;
}

// Lets a kernel have `bytes` of dynamic shared memory, once per device.
template <auto KERNEL>
cudaError_t allow_smem(size_t bytes) {
  static std::atomic<uint64_t> mask{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (!(mask.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(bytes));
    if (e != cudaSuccess) return e;
    mask.fetch_or(bit, std::memory_order_acq_rel);
  }
  return cudaSuccess;
}

template <typename Id>
cudaError_t launch_sort(const Id* ids, int M, int V, const EmbedGradWs& ws, int* passes_out,
                        cudaStream_t stream) {
  auto kernel = embed_sort_kernel<Id>;
  const cudaError_t e = allow_smem<embed_sort_kernel<Id>>(kSortSmem);
  if (e != cudaSuccess) return e;
  const int bits = bit_length(V);  // keys 0 .. V
  const int passes = (bits + kMaxDigitBits - 1) / kMaxDigitBits;
  const int digit_bits = (bits + passes - 1) / passes;
  const int ctas = kSortCluster;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = overlapped(ctas, kSortThreads, kSortSmem, stream, attr);
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(ctas);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.numAttrs = 2;
  *passes_out = passes;
  return cudaLaunchKernelEx(&cfg, kernel, ids, M, V, passes, digit_bits, ws.key0, ws.idx0,
                            ws.key1, ws.idx1);
}

}  // namespace

cudaError_t launch_embedding_lookup(const void* ids, bool ids64, const __nv_bfloat16* table,
                                    __nv_bfloat16* out, int64_t M, int64_t V, int D, float scale,
                                    cudaStream_t stream) {
  const int segs = (D + kSegCols - 1) / kSegCols;
  const int64_t warps = M * segs;
  const int64_t per = kLookThreads / 32;
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = overlapped((warps + per - 1) / per, kLookThreads, 0, stream, attr);
  return ids64 ? cudaLaunchKernelEx(&cfg, embed_lookup_kernel<int64_t>,
                                    static_cast<const int64_t*>(ids), table, out, M, V, D, segs,
                                    scale)
               : cudaLaunchKernelEx(&cfg, embed_lookup_kernel<int>, static_cast<const int*>(ids),
                                    table, out, M, V, D, segs, scale);
}

// Positions per piece: 32 (16384 x 4096: 66 us in all, 74 with 16), fewer while
// that leaves under eight CTAs per SM.
int embed_piece(int64_t M, int D) {
  const int segs = (D + kSegCols - 1) / kSegCols;
  int piece = kMaxPiece;
  while (piece > 4 && (M + piece - 1) / piece * segs < 152 * 8) piece /= 2;
  return piece;
}

cudaError_t launch_embedding_grad(const void* ids, bool ids64, const __nv_bfloat16* dout,
                                  __nv_bfloat16* dtable, int M, int V, int D, float scale,
                                  bool accumulate, const EmbedGradWs& ws, int sms,
                                  cudaStream_t stream) {
  SumArgs a{};
  a.dout = dout;
  a.dtable = dtable;
  a.head = ws.head;
  a.tail = ws.tail;
  a.M = M;
  a.V = V;
  a.D = D;
  a.piece = embed_piece(M, D);
  a.pieces = (M + a.piece - 1) / a.piece;
  a.segs = (D + kSegCols - 1) / kSegCols;
  a.scale = scale;
  a.accumulate = accumulate ? 1 : 0;
  const int64_t zeros = accumulate ? 0 : std::min(V, sms * 8);
  cudaError_t e;
  if (M <= kDirectMax) {
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg =
        overlapped(static_cast<int64_t>(M) * a.segs + zeros, kSumThreads, 0, stream, attr);
    return ids64 ? cudaLaunchKernelEx(&cfg, embed_direct_kernel<int64_t>,
                                      static_cast<const int64_t*>(ids), a)
                 : cudaLaunchKernelEx(&cfg, embed_direct_kernel<int>, static_cast<const int*>(ids),
                                      a);
  }
  int passes = 0;
  e = ids64 ? launch_sort(static_cast<const int64_t*>(ids), M, V, ws, &passes, stream)
            : launch_sort(static_cast<const int*>(ids), M, V, ws, &passes, stream);
  if (e != cudaSuccess) return e;
  a.key = (passes & 1) ? ws.key0 : ws.key1;
  a.idx = (passes & 1) ? ws.idx0 : ws.idx1;
  const int64_t sums = static_cast<int64_t>(a.pieces) * a.segs;
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = overlapped(sums + zeros, kSumThreads, 0, stream, attr);
  if ((e = cudaLaunchKernelEx(&cfg, embed_sum_kernel, a)) != cudaSuccess) return e;
  cudaLaunchAttribute attr2[1];
  // and one for each place where a long run is looked for, x 256 columns
  const int64_t longs = static_cast<int64_t>((a.pieces - 1) / kLongRun) *
                        ((D + kLongCols - 1) / kLongCols);
  cudaLaunchConfig_t cfg2 = overlapped(sums + longs, kSumThreads, 0, stream, attr2);
  return cudaLaunchKernelEx(&cfg2, embed_join_kernel, a);
}

}  // namespace gbf
