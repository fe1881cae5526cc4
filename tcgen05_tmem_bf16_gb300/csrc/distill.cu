// distill.cu -- the lists of a distillation from a teacher's top logits: for each
// row the columns of the vocabulary it holds, in ascending order, each with its
// share q = softmax(beta * logits) over the row's valid entries.
//
// An entry is valid if its column is inside [0, V) and its logit is not minus
// infinity.  Entries of one column become one, with the sum of their shares.  The
// products' endings walk a row's list along with their columns (linear_ce.cu,
// ce_swap.cu): sorting it here, once, is what lets them find the next entry with one
// comparison, and `at`, the first entry of each 2^shift columns, lets a tile begin
// anywhere.  A row holds a few hundred entries at most, so an entry's
// place is the number of columns before its own, counted by its own thread: no
// exchange, no atomics, the same sums in the same order on every run.
//
// One CTA per row in turn.  Bound by the operations of the counting (K^2 per row) and
// by latency.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>

#include "internal.h"
#include "ptx.cuh"

namespace gbf {

namespace {

// What a row's CTA of THREADS holds of its entries, up to MOST of them.
template <int THREADS, int MOST>
struct ListRow {
  static constexpr int kListWarps = THREADS / 32;
  int4 col[MOST / 4];    // as given; INT_MAX where not valid, and up to a multiple of four
  float share[MOST];
  int sorted[MOST];      // the columns in ascending order
  float sorted_share[MOST];
  float part[2][kListWarps];
  int count[kListWarps];
};

// The row has a column twice: every entry looks for its column's others, and the first
// of them takes the sum of the shares in the entries' order.  Returns the number of
// different columns.
template <int THREADS, int MOST>
__device__ int merge_columns(ListRow<THREADS, MOST>& s, int K) {
  constexpr int kListThreads = THREADS, kListWarps = THREADS / 32, kSlots = MOST / THREADS;
  int* col = reinterpret_cast<int*>(s.col);
  const int quads = (K + 3) / 4;
  float all[kSlots];
  bool first[kSlots];
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    const int k = threadIdx.x + i * kListThreads;
    first[i] = false;
    if (k >= K) continue;
    const int c = col[k];
    first[i] = c != INT_MAX;
    all[i] = 0.0f;
    for (int j = 0; j < quads; ++j) {
      const int4 x = s.col[j];
      const int four[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        if (four[h] != c || c == INT_MAX) continue;
        first[i] = first[i] && 4 * j + h >= k;
        all[i] += s.share[4 * j + h];
      }
    }
  }
  __syncthreads();
  int n = 0;
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    const int k = threadIdx.x + i * kListThreads;
    if (k < K && !first[i]) col[k] = INT_MAX;
    n += first[i];
  }
  n = __reduce_add_sync(0xFFFFFFFFu, n);
  if ((threadIdx.x & 31) == 0) s.count[threadIdx.x >> 5] = n;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    const int k = threadIdx.x + i * kListThreads;
    if (!first[i]) continue;
    int before = 0;
    for (int j = 0; j < quads; ++j) {
      const int4 x = s.col[j];
      before += (x.x < col[k]) + (x.y < col[k]) + (x.z < col[k]) + (x.w < col[k]);
    }
    s.sorted[before] = col[k];
    s.sorted_share[before] = all[i];
  }
  n = 0;
  for (int w = 0; w < kListWarps; ++w) n += s.count[w];
  return n;
}

// SLOTS entries per thread.
template <int THREADS, int SLOTS>
__global__ void __launch_bounds__(THREADS) ce_lists_kernel(const CeLists p) {
  constexpr int kListThreads = THREADS, kListWarps = THREADS / 32;
  __shared__ ListRow<THREADS, SLOTS * THREADS> s;
  int* col = reinterpret_cast<int*>(s.col);
  griddep_wait();
  // From here on the kernels before this one have completed: the next may start, and
  // read all but this one's results before its own wait.
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quads = (p.K + 3) / 4;
  for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x) {
    float t[SLOTS];  // this thread's logits, then exponentials
    float top = -INFINITY;
    int n = 0;
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
      const int k = threadIdx.x + i * kListThreads;
      t[i] = -INFINITY;
      if (k >= 4 * quads) continue;
      bool ok = k < p.K;
      int64_t id = 0;
      if (ok) {
        const int64_t at = row * p.K + k;
        id = p.ids64 ? static_cast<const int64_t*>(p.ids)[at]
                     : static_cast<const int*>(p.ids)[at];
        const float x = p.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p.logits)[at])
                               : static_cast<const float*>(p.logits)[at];
        ok = id >= 0 && id < p.V && x != -INFINITY;
        if (ok) {
          t[i] = p.beta * x;
          top = fmaxf(top, t[i]);
          ++n;
        }
      }
      col[k] = ok ? static_cast<int>(id) : INT_MAX;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    n = __reduce_add_sync(0xFFFFFFFFu, n);
    if (lane == 0) {
      s.part[0][warp] = top;
      s.count[warp] = n;
    }
    __syncthreads();
    n = 0;
#pragma unroll
    for (int w = 0; w < kListWarps; ++w) {
      top = fmaxf(top, s.part[0][w]);
      n += s.count[w];
    }
    float sum = 0.0f;
    int before[SLOTS];
    bool twice = false;
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
      const int k = threadIdx.x + i * kListThreads;
      before[i] = 0;
      if (k >= p.K || col[k] == INT_MAX) continue;
      // a product that has left fp32's range downwards all the same has the largest
      // logit's place: no minus infinity less minus infinity
      t[i] = expf(t[i] == top ? 0.0f : t[i] - top);
      sum += t[i];
      const int c = col[k];
      int same = 0;
      for (int j = 0; j < quads; ++j) {
        const int4 x = s.col[j];
        before[i] += (x.x < c) + (x.y < c) + (x.z < c) + (x.w < c);
        same += (x.x == c) + (x.y == c) + (x.z == c) + (x.w == c);
      }
      twice = twice || same > 1;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (lane == 0) s.part[1][warp] = sum;
    const bool merge = __syncthreads_or(twice);
    sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kListWarps; ++w) sum += s.part[1][w];
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
      const int k = threadIdx.x + i * kListThreads;
      if (k >= p.K || col[k] == INT_MAX) continue;
      if (merge) {
        s.share[k] = t[i] / sum;
      } else {
        s.sorted[before[i]] = col[k];
        s.sorted_share[before[i]] = t[i] / sum;
      }
    }
    __syncthreads();
    if (merge) {
      n = merge_columns(s, p.K);
      __syncthreads();
    }
    int2* list = p.list + row * (p.K + 1);
    for (int i = threadIdx.x; i <= p.K; i += kListThreads)
      list[i] = i < n ? make_int2(s.sorted[i], __float_as_int(s.sorted_share[i]))
                      : make_int2(INT_MAX, 0);
    if (threadIdx.x == 0) p.tgt[row] = n > 0 ? s.sorted[0] : -1;
    // at[b] == i from behind the block of the entry before to its own block
    uint16_t* at = p.at + row * p.stride;
    for (int i = warp; i <= n; i += kListWarps) {
      const int from = i > 0 ? (s.sorted[i - 1] >> p.shift) + 1 : 0;
      const int to = i < n ? s.sorted[i] >> p.shift : p.stride - 1;
      for (int b = from + lane; b <= to; b += 32) at[b] = static_cast<uint16_t>(i);
    }
    __syncthreads();  // the arrays are the next row's
  }
}

}  // namespace

cudaError_t launch_ce_lists(const CeLists& p, int sms, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(p.M, static_cast<int64_t>(sms) * 16)), 1, 1);
  // threads of a row: lists of 100 rows of 1000 entries take 75 us with 128, 41 with 512
  const bool few = p.K <= 128;
  cfg.blockDim = dim3(few ? 128 : 512, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return few ? cudaLaunchKernelEx(&cfg, ce_lists_kernel<128, 1>, p)
             : cudaLaunchKernelEx(&cfg, ce_lists_kernel<512, kPickMax / 512>, p);
}

}  // namespace gbf
