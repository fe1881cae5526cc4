// distill.cu -- the lists of a distillation from a teacher's top logits: for each
// row the columns of the vocabulary it holds, in ascending order, each with its
// share q = softmax(beta * logits) over the row's valid entries.
//
// An entry is valid if its column is inside [0, V) and its logit is not minus
// infinity.  Entries of one column become one, with the sum of their shares.  The products' endings walk a row's list along with their columns
// (linear_ce.cu, ce_swap.cu): sorting it here, once, is what lets them find the next
// entry with one comparison, and `at`, the first entry of each 2^shift columns, lets
// a tile begin anywhere.  A row holds a few hundred entries at most, so an entry's
// place is the number of columns before its own, counted by its own thread: no
// exchange, no atomics, the same sums in the same order on every run.
//
// One CTA per row in turn.  Bound by latency and, for a large vocabulary, by writing
// `at` (2 bytes per 128 columns and row).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>

#include "internal.h"
#include "ptx.cuh"

namespace gbf {

namespace {

constexpr int kListThreads = 128;
constexpr int kListWarps = kListThreads / 32;

// SLOTS entries per thread: one for short lists (1 row of 8 entries x 32000: 6.1 us
// with the eight that the longest take, 4.3 with one).
template <int SLOTS>
__global__ void __launch_bounds__(kListThreads) ce_lists_kernel(const CeLists p) {
  constexpr int kMost = SLOTS * kListThreads;
  __shared__ int col[kMost];    // as given; INT_MAX where not valid
  __shared__ int lead[kMost];   // the same, but only at a column's first entry
  __shared__ float share[kMost];
  __shared__ int sorted[kMost];
  __shared__ float part[2][kListWarps];
  __shared__ int count[kListWarps];
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x) {
    float t[SLOTS];  // this thread's logits, then shares
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
      const int k = threadIdx.x + i * kListThreads;
      t[i] = -INFINITY;
      if (k >= p.K) continue;
      const int64_t at = row * p.K + k;
      const int64_t id = p.ids64 ? static_cast<const int64_t*>(p.ids)[at]
                                 : static_cast<const int*>(p.ids)[at];
      const float x = p.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p.logits)[at])
                             : static_cast<const float*>(p.logits)[at];
      const bool ok = id >= 0 && id < p.V && x != -INFINITY;
      col[k] = ok ? static_cast<int>(id) : INT_MAX;
      if (ok) {
        t[i] = p.beta * x;
        top = fmaxf(top, t[i]);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    if (lane == 0) part[0][warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kListWarps; ++w) top = fmaxf(top, part[0][w]);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
      const int k = threadIdx.x + i * kListThreads;
      if (k >= p.K || col[k] == INT_MAX) continue;
      // a product that has left fp32's range downwards all the same has the largest
      // logit's place: no minus infinity less minus infinity
      t[i] = expf(t[i] == top ? 0.0f : t[i] - top);
      sum += t[i];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (lane == 0) part[1][warp] = sum;
    __syncthreads();
    sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kListWarps; ++w) sum += part[1][w];
    int n = 0;
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
      const int k = threadIdx.x + i * kListThreads;
      if (k >= p.K) continue;
      share[k] = t[i] / sum;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
      const int k = threadIdx.x + i * kListThreads;
      if (k >= p.K) continue;
      const int c = col[k];
      bool first = c != INT_MAX;
      float all = 0.0f;
      for (int j = 0; j < p.K; ++j) {
        if (col[j] != c) continue;
        first = first && j >= k;
        all += share[j];
      }
      lead[k] = first ? c : INT_MAX;
      t[i] = all;
      n += first;
    }
    n = __reduce_add_sync(0xFFFFFFFFu, n);
    if (lane == 0) count[warp] = n;
    __syncthreads();
    n = 0;
#pragma unroll
    for (int w = 0; w < kListWarps; ++w) n += count[w];
    int2* list = p.list + row * (p.K + 1);
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
      const int k = threadIdx.x + i * kListThreads;
      if (k >= p.K) continue;
      const int c = lead[k];
      if (c != INT_MAX) {
        int before = 0;
        for (int j = 0; j < p.K; ++j) before += lead[j] < c;
        sorted[before] = c;
        list[before] = make_int2(c, __float_as_int(t[i]));
      }
      if (k >= n) list[k] = make_int2(INT_MAX, 0);
    }
    if (threadIdx.x == 0) list[p.K] = make_int2(INT_MAX, 0);
    __syncthreads();
    if (threadIdx.x == 0) p.tgt[row] = n > 0 ? sorted[0] : -1;
    uint16_t* at = p.at + row * p.stride;
    for (int b = threadIdx.x; b < p.stride; b += kListThreads) {
      const int64_t first = static_cast<int64_t>(b) << p.shift;
      int lo = 0, hi = n;  // the entries before column `first`
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (sorted[mid] < first) lo = mid + 1;
        else hi = mid;
      }
      at[b] = static_cast<uint16_t>(lo);
    }
    __syncthreads();  // the arrays are the next row's
  }
}

}  // namespace

cudaError_t launch_ce_lists(const CeLists& p, int sms, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(p.M, static_cast<int64_t>(sms) * 16)), 1, 1);
  cfg.blockDim = dim3(kListThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return p.K <= kListThreads ? cudaLaunchKernelEx(&cfg, ce_lists_kernel<1>, p)
                             : cudaLaunchKernelEx(&cfg, ce_lists_kernel<kPickMax / kListThreads>, p);
}

}  // namespace gbf
