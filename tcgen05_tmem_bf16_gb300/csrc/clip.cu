// clip.cu -- the global 2-norm over many gradient tensors, and clipping.
//
//   norm = sqrt(sum over all tensors of x^2),
//   factor = min(1, max_norm / (norm + eps)),  out = factor * x.
//
// HBM-bound (836M bf16 values: norm 231 us, 7.2 TB/s; scaling into other buffers
// 510 us, 6.5 TB/s; eight 16-byte loads in flight per thread, 835 us in all with
// four): one read of every tensor for the norm, then one read and one
// write where the factor is below 1 (in place with a factor of 1 nothing is
// touched again; into other buffers the values are copied).
//
// The tensors are cut into chunks of 2048 to 32768 elements, dealt to the CTAs in a
// fixed order, and every CTA writes its own partial sum, which the second
// kernel adds in a fixed order: no atomics, the same bits on every run.
//
// Squares outside fp32's range: a vector of eight values whose squares add up
// to more than 1e24 or less than 1e-30 is squared again scaled by 2^-96 or
// 2^96, into sums of their own, so that the norm neither overflows nor loses
// small gradients.  Beyond a chunk the sums are carried as pairs of fp32 values
// (a sum and what its roundings left out): fp64 would do, but is slow on this
// GPU (0.5M values in 171 chunks: 30.7 us with sums and root in fp64, 7.3 so).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace gbf {

namespace {

constexpr int kClipThreads = 256;
constexpr int kClipMinChunk = 2048, kClipMaxChunk = 32768;  // elements
constexpr int kClipList = 512;     // tensors per launch at most

struct ClipTensor {
  const void* in;
  void* out;
  int64_t n;
  int64_t first_chunk;  // chunks of the launch's tensors before this one
};

// Elements of a 16-byte block before p: the chunks of a tensor are cut where
// p - before would be, so that only the first of them begins inside a block.
int before_of(const void* p, int type) {
  return static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15u) / (type == 1 ? 4 : 2));
}
template <typename T>
__device__ __forceinline__ int before_of(const T* p) {
  return static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T));
}

template <int LIST>
struct ClipArgs {
  ClipTensor t[LIST];
  unsigned f32[LIST / 32];  // bit i: tensor i holds 32-bit values (else bf16)
  int tensors;
  int64_t chunks;
  int chunk;              // elements
  float2* partial;        // this launch's sums: [CTA][3]
  const float2* sums;     // every launch's sums, for the second kernel
  int num_sums;           // triples
  float* norm;
  float max_norm, eps;
  int in_place;
};

// The tensor that holds a chunk: the last one whose first chunk is not after it.
template <int LIST>
__device__ __forceinline__ int tensor_of(const ClipArgs<LIST>& a, int64_t chunk) {
  int lo = 0, hi = a.tensors - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.t[mid].first_chunk <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// A sum and the rounding errors of its additions.
struct Pair {
  float hi = 0.0f, lo = 0.0f;
  __device__ __forceinline__ void add(float x, float more = 0.0f) {
    const float s = __fadd_rn(hi, x);
    const float b = __fadd_rn(s, -hi);
    // an infinite or NaN sum has no error to keep
    const float e = __fadd_rn(__fadd_rn(hi, -__fadd_rn(s, -b)), __fadd_rn(x, -b));
    lo += (isfinite(s) ? e : 0.0f) + more;
    hi = s;
  }
  __device__ __forceinline__ void add(const Pair& o) { add(o.hi, o.lo); }
  __device__ __forceinline__ Pair shuffled(int mask) const {
    Pair o;
    o.hi = __shfl_xor_sync(0xFFFFFFFFu, hi, mask);
    o.lo = __shfl_xor_sync(0xFFFFFFFFu, lo, mask);
    return o;
  }
};

constexpr float kBigSum = 1e24f, kSmallSum = 1e-30f;
constexpr float kDown = 0x1p-96f, kUp = 0x1p96f;

struct Squares {
  float mid = 0.0f, high = 0.0f, low = 0.0f;
  template <int N>
  __device__ __forceinline__ void add(const float (&x)[N]) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) s = fmaf(x[i], x[i], s);
    if (s >= kSmallSum && s <= kBigSum) {
      mid += s;
    } else if (s < kSmallSum) {  // often all zeros
#pragma unroll
      for (int i = 0; i < N; ++i) low = fmaf(x[i] * kUp, x[i] * kUp, low);
    } else {  // large, infinite or NaN
#pragma unroll
      for (int i = 0; i < N; ++i) high = fmaf(x[i] * kDown, x[i] * kDown, high);
    }
  }
};

template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void unpack(const uint4& u, float (&f)[8]) { unpack8(u, f); }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) { return pack8(f); }
  static __device__ __forceinline__ float one(const __nv_bfloat16* p) { return ld_bf16f(p); }
  static __device__ __forceinline__ void put(__nv_bfloat16* p, float x) {
    *p = __float2bfloat16_rn(x);
  }
};
template <>
struct Vec<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void unpack(const uint4& u, float (&f)[4]) {
    f[0] = __uint_as_float(u.x);
    f[1] = __uint_as_float(u.y);
    f[2] = __uint_as_float(u.z);
    f[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
  static __device__ __forceinline__ float one(const float* p) { return *p; }
  static __device__ __forceinline__ void put(float* p, float x) { *p = x; }
};

// Elements of [p, p + n) before the first 16-byte boundary.
template <typename T>
__device__ __forceinline__ int head_of(const T* p, int n) {
  const int bytes = static_cast<int>((16u - (reinterpret_cast<uintptr_t>(p) & 15u)) & 15u);
  return min(n, bytes / static_cast<int>(sizeof(T)));
}

template <typename T>
__device__ __forceinline__ void square_range(const T* p, int n, Squares& s) {
  constexpr int kN = Vec<T>::kN;
  const int head = head_of(p, n);
  const int vecs = (n - head) / kN;
  const uint4* v = reinterpret_cast<const uint4*>(p + head);
  constexpr int kAhead = 8;
  int i = threadIdx.x;
  for (; i + (kAhead - 1) * kClipThreads < vecs; i += kAhead * kClipThreads) {
    uint4 u[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) u[k] = v[i + k * kClipThreads];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      float f[kN];
      Vec<T>::unpack(u[k], f);
      s.add(f);
    }
  }
  for (; i < vecs; i += kClipThreads) {
    float f[kN];
    Vec<T>::unpack(v[i], f);
    s.add(f);
  }
  const int rest = n - vecs * kN;  // the head and what follows the vectors
  if (static_cast<int>(threadIdx.x) < rest) {
    const int at = static_cast<int>(threadIdx.x) < head ? threadIdx.x : threadIdx.x + vecs * kN;
    float f[1] = {Vec<T>::one(p + at)};
    s.add(f);
  }
}

// The elements [at, at + n) of tensor i that chunk c holds, cut along the blocks
// of `by`.
template <typename T>
__device__ __forceinline__ int chunk_of(int64_t c, int chunk, int64_t count, const T* by,
                                        int64_t& at) {
  const int64_t from = c * chunk - before_of(by);
  at = from > 0 ? from : 0;
  return static_cast<int>(min(from + chunk, count) - at);
}

// Sums over the CTA, in the same order on every run; valid in thread 0.
__device__ __forceinline__ void block_sum(Pair (&sum)[3], Pair (&part)[kClipThreads / 32][3]) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < 3; ++k) sum[k].add(sum[k].shuffled(o));
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int k = 0; k < 3; ++k) part[threadIdx.x >> 5][k] = sum[k];
  __syncthreads();
  if (threadIdx.x == 0)
    for (int w = 1; w < kClipThreads / 32; ++w)
#pragma unroll
      for (int k = 0; k < 3; ++k) sum[k].add(part[w][k]);
}

template <int LIST>
__global__ void __launch_bounds__(kClipThreads)
    clip_norm_kernel(const __grid_constant__ ClipArgs<LIST> a) {
  __shared__ Pair part[kClipThreads / 32][3];
  griddep_launch_dependents();
  griddep_wait();
  Pair sum[3];  // the squares as they are, scaled down, scaled up
  for (int64_t c = blockIdx.x; c < a.chunks; c += gridDim.x) {
    const int i = tensor_of(a, c);
    int64_t at;
    Squares s;
    if ((a.f32[i >> 5] >> (i & 31)) & 1u) {
      const float* p = static_cast<const float*>(a.t[i].in);
      const int n = chunk_of(c - a.t[i].first_chunk, a.chunk, a.t[i].n, p, at);
      square_range(p + at, n, s);
    } else {
      const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(a.t[i].in);
      const int n = chunk_of(c - a.t[i].first_chunk, a.chunk, a.t[i].n, p, at);
      square_range(p + at, n, s);
    }
    sum[0].add(s.mid);
    sum[1].add(s.high);
    sum[2].add(s.low);
  }
  block_sum(sum, part);
  if (threadIdx.x == 0) {
#pragma unroll
    for (int k = 0; k < 3; ++k)
      a.partial[static_cast<int64_t>(blockIdx.x) * 3 + k] = make_float2(sum[k].hi, sum[k].lo);
  }
}

// Sixteen bytes from an address that need not be a multiple of 16 (but of the
// element's size): the two aligned vectors that hold them, shifted.  Each of
// the two holds at least one of the sixteen bytes, so neither lies outside the
// memory that the range is in; bytes of a neighbour are shifted out.
__device__ __forceinline__ uint4 load_across(const uint4* base, int i, int shift_bytes) {
  const uint4 x = base[i];
  const uint4 y = base[i + 1];
  uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
  if (shift_bytes & 8) {
#pragma unroll
    for (int k = 0; k < 6; ++k) w[k] = w[k + 2];
  }
  if (shift_bytes & 4) {
#pragma unroll
    for (int k = 0; k < 5; ++k) w[k] = w[k + 1];
  }
  const unsigned bits = (shift_bytes & 3) * 8;
  return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                    __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
}

template <typename T>
__device__ __forceinline__ void scale_range(const T* p, T* out, int n, float factor) {
  constexpr int kN = Vec<T>::kN;
  const int head = head_of(out, n);  // the stores are aligned
  const int vecs = (n - head) / kN;
  uint4* o = reinterpret_cast<uint4*>(out + head);
  const uintptr_t in = reinterpret_cast<uintptr_t>(p + head);
  const int shift = static_cast<int>(in & 15u);
  const uint4* v = reinterpret_cast<const uint4*>(in - shift);
  auto put = [&](int i, const uint4& u) {
    float f[kN];
    Vec<T>::unpack(u, f);
#pragma unroll
    for (int j = 0; j < kN; ++j) f[j] *= factor;
    o[i] = Vec<T>::pack(f);
  };
  constexpr int kAhead = 8;
  int i = threadIdx.x;
  if (shift == 0) {
    for (; i + (kAhead - 1) * kClipThreads < vecs; i += kAhead * kClipThreads) {
      uint4 u[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) u[k] = v[i + k * kClipThreads];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) put(i + k * kClipThreads, u[k]);
    }
    for (; i < vecs; i += kClipThreads) put(i, v[i]);
  } else {
    for (; i + (kAhead - 1) * kClipThreads < vecs; i += kAhead * kClipThreads) {
      uint4 u[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) u[k] = load_across(v, i + k * kClipThreads, shift);
#pragma unroll
      for (int k = 0; k < kAhead; ++k) put(i + k * kClipThreads, u[k]);
    }
    for (; i < vecs; i += kClipThreads) put(i, load_across(v, i, shift));
  }
  const int rest = n - vecs * kN;
  if (static_cast<int>(threadIdx.x) < rest) {
    const int at = static_cast<int>(threadIdx.x) < head ? threadIdx.x : threadIdx.x + vecs * kN;
    Vec<T>::put(out + at, Vec<T>::one(p + at) * factor);
  }
}

// Adds the partial sums (every CTA for itself, in the same order), then scales
// its chunks, the last ones first: they are the ones still in L2.
template <int LIST>
__global__ void __launch_bounds__(kClipThreads)
    clip_scale_kernel(const __grid_constant__ ClipArgs<LIST> a) {
  __shared__ Pair part[kClipThreads / 32][3];
  __shared__ float shared_factor;
  griddep_launch_dependents();
  griddep_wait();
  Pair sum[3];
  for (int i = threadIdx.x; i < a.num_sums; i += kClipThreads)
#pragma unroll
    for (int k = 0; k < 3; ++k) sum[k].add(a.sums[i * 3 + k].x, a.sums[i * 3 + k].y);
  block_sum(sum, part);
  if (threadIdx.x == 0) {
    float norm, factor;
    if (sum[1].hi == 0.0f && sum[0].hi >= 1e-12f) {
      // the squares scaled up are under 1e-30 for each vector: nothing next to this
      norm = __fsqrt_rn(sum[0].hi + sum[0].lo);
      const float ratio = __fdiv_rn(a.max_norm, norm + a.eps);
      factor = ratio >= 1.0f ? 1.0f : ratio;
    } else {
      double t[3];
#pragma unroll
      for (int k = 0; k < 3; ++k)
        t[k] = static_cast<double>(sum[k].hi) + static_cast<double>(sum[k].lo);
      const double wide = sqrt(t[1] * 0x1p192 + t[0] + t[2] * 0x1p-192);
      // a NaN norm makes the factor NaN
      const double ratio = static_cast<double>(a.max_norm) / (wide + static_cast<double>(a.eps));
      norm = static_cast<float>(wide);
      factor = ratio >= 1.0 ? 1.0f : static_cast<float>(ratio);
      if (wide == 0.0) factor = 1.0f;
    }
    if (isinf(a.max_norm)) factor = 1.0f;  // the norm alone
    shared_factor = factor;
    if (blockIdx.x == 0) *a.norm = norm;
  }
  __syncthreads();
  const float factor = shared_factor;
  if (a.in_place && factor == 1.0f) return;
  for (int64_t r = blockIdx.x; r < a.chunks; r += gridDim.x) {
    const int64_t c = a.chunks - 1 - r;
    const int i = tensor_of(a, c);
    int64_t at;
    if ((a.f32[i >> 5] >> (i & 31)) & 1u) {
      float* out = static_cast<float*>(a.t[i].out);
      const int n = chunk_of(c - a.t[i].first_chunk, a.chunk, a.t[i].n, out, at);
      scale_range(static_cast<const float*>(a.t[i].in) + at, out + at, n, factor);
    } else {
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.t[i].out);
      const int n = chunk_of(c - a.t[i].first_chunk, a.chunk, a.t[i].n, out, at);
      scale_range(static_cast<const __nv_bfloat16*>(a.t[i].in) + at, out + at, n, factor);
    }
  }
}

template <int LIST>
cudaError_t run_clip(const void* const* in, void* const* out, const int64_t* counts,
                     const int* types, int n, float max_norm, float eps, float* norm,
                     float2* partial, int sms, cudaStream_t stream) {
  const int launches = std::max(1, (n + LIST - 1) / LIST);
  const int most = clip_ctas(sms);
  // Long chunks save the way from one to the next, short ones keep every SM busy:
  // the longest of which there are two for each CTA.  (0.5M values in 51 tensors:
  // 7.3 us, 7.5 with 8192 as the shortest.)
  int64_t total = 0;
  for (int i = 0; i < n; ++i) total += counts[i];
  int chunk = kClipMaxChunk;
  while (chunk > kClipMinChunk && total / chunk < 2 * most) chunk /= 2;
  auto prepare = [&](int l, ClipArgs<LIST>& a, bool scale) {
    a = ClipArgs<LIST>{};
    const int first = l * LIST;
    const int last = std::min(n, first + LIST);
    for (int i = first; i < last; ++i) {
      if (counts[i] == 0) continue;
      const int k = a.tensors++;
      a.t[k] = ClipTensor{in[i], out ? out[i] : const_cast<void*>(in[i]), counts[i], a.chunks};
      if (types[i] == 1) a.f32[k >> 5] |= 1u << (k & 31);
      const int before = before_of(scale ? a.t[k].out : a.t[k].in, types[i]);
      a.chunks += (counts[i] + before + chunk - 1) / chunk;
    }
    a.chunk = chunk;
    a.max_norm = max_norm;
    a.eps = eps;
    a.norm = norm;
    a.sums = partial;
    a.in_place = out == nullptr;
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(a.chunks, most)));
  };
  auto launch = [&](void (*kernel)(ClipArgs<LIST>), int grid, const ClipArgs<LIST>& a) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(kClipThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
  };
  ClipArgs<LIST> a;
  int sums = 0;
  for (int l = 0; l < launches; ++l) {
    const int grid = prepare(l, a, false);
    a.partial = partial + 3 * static_cast<int64_t>(sums);
    const cudaError_t e = launch(clip_norm_kernel<LIST>, grid, a);
    if (e != cudaSuccess) return e;
    sums += grid;
  }
  for (int l = 0; l < launches; ++l) {
    const int grid = prepare(l, a, true);
    a.num_sums = sums;
    const cudaError_t e = launch(clip_scale_kernel<LIST>, grid, a);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

int clip_ctas(int sms) { return sms * 8; }
int clip_launches(int n) { return std::max(1, (n + kClipList - 1) / kClipList); }

cudaError_t launch_clip_grad_norm(const void* const* in, void* const* out, const int64_t* counts,
                                  const int* types, int n, float max_norm, float eps, float* norm,
                                  float2* partial, int sms, cudaStream_t stream) {
  // a short list keeps the launch's arguments small
  return n <= 64 ? run_clip<64>(in, out, counts, types, n, max_norm, eps, norm, partial, sms,
                                stream)
                 : run_clip<kClipList>(in, out, counts, types, n, max_norm, eps, norm, partial,
                                       sms, stream);
}

}  // namespace gbf
