// clip.cu -- the global 2-norm over many gradient tensors, and clipping.
//
//   norm = sqrt(sum over all tensors of x^2),
//   factor = min(1, max_norm / (norm + eps)),  out = factor * x.
//
// HBM-bound: one read of every tensor for the norm, then one read and one
// write where the factor is below 1 (in place with a factor of 1 nothing is
// touched again; into other buffers the values are copied).
//
// The tensors are cut into chunks of 32768 elements, dealt to the CTAs in a
// fixed order, and every CTA writes its own partial sum, which the second
// kernel adds in a fixed order: no atomics, the same bits on every run.
//
// Squares outside fp32's range: a vector of eight values whose squares add up
// to more than 1e30 or less than 1e-30 is squared again scaled by 2^-96 or
// 2^96, into sums of their own, so that the norm neither overflows nor loses
// small gradients.  Per chunk the sums are carried in 64 bits.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace gbf {

namespace {

constexpr int kClipThreads = 256;
constexpr int kClipChunk = 32768;  // elements
constexpr int kClipList = 512;     // tensors per launch at most

struct ClipTensor {
  const void* in;
  void* out;
  int64_t n;
  int64_t first_chunk;  // chunks of the launch's tensors before this one
};

template <int LIST>
struct ClipArgs {
  ClipTensor t[LIST];
  unsigned f32[LIST / 32];  // bit i: tensor i holds 32-bit values (else bf16)
  int tensors;
  int64_t chunks;
  double* partial;        // this launch's sums: [CTA][3]
  const double* sums;     // every launch's sums, for the second kernel
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

constexpr float kBigSum = 1e30f, kSmallSum = 1e-30f;
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
  constexpr int kAhead = 4;
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

template <int LIST>
__global__ void __launch_bounds__(kClipThreads)
    clip_norm_kernel(const __grid_constant__ ClipArgs<LIST> a) {
  __shared__ double part[kClipThreads / 32][3];
  griddep_launch_dependents();
  griddep_wait();
  double mid = 0.0, high = 0.0, low = 0.0;
  for (int64_t c = blockIdx.x; c < a.chunks; c += gridDim.x) {
    const int i = tensor_of(a, c);
    const int64_t at = (c - a.t[i].first_chunk) * kClipChunk;
    const int n = static_cast<int>(min(static_cast<int64_t>(kClipChunk), a.t[i].n - at));
    Squares s;
    if ((a.f32[i >> 5] >> (i & 31)) & 1u)
      square_range(static_cast<const float*>(a.t[i].in) + at, n, s);
    else
      square_range(static_cast<const __nv_bfloat16*>(a.t[i].in) + at, n, s);
    mid += s.mid;
    high += s.high;
    low += s.low;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    mid += __shfl_xor_sync(0xFFFFFFFFu, mid, o);
    high += __shfl_xor_sync(0xFFFFFFFFu, high, o);
    low += __shfl_xor_sync(0xFFFFFFFFu, low, o);
  }
  if ((threadIdx.x & 31) == 0) {
    part[threadIdx.x >> 5][0] = mid;
    part[threadIdx.x >> 5][1] = high;
    part[threadIdx.x >> 5][2] = low;
  }
  __syncthreads();
  if (threadIdx.x < 3) {
    double t = 0.0;
    for (int w = 0; w < kClipThreads / 32; ++w) t += part[w][threadIdx.x];
    a.partial[blockIdx.x * 3 + threadIdx.x] = t;
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
  constexpr int kAhead = 4;
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
  __shared__ double part[kClipThreads / 32][3];
  griddep_launch_dependents();
  griddep_wait();
  double s[3] = {0.0, 0.0, 0.0};
  for (int i = threadIdx.x; i < a.num_sums; i += kClipThreads)
#pragma unroll
    for (int k = 0; k < 3; ++k) s[k] += a.sums[i * 3 + k];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < 3; ++k) s[k] += __shfl_xor_sync(0xFFFFFFFFu, s[k], o);
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int k = 0; k < 3; ++k) part[threadIdx.x >> 5][k] = s[k];
  __syncthreads();
  double t[3] = {0.0, 0.0, 0.0};
  for (int w = 0; w < kClipThreads / 32; ++w)
#pragma unroll
    for (int k = 0; k < 3; ++k) t[k] += part[w][k];
  const double norm = sqrt(t[1] * 0x1p192 + t[0] + t[2] * 0x1p-192);
  // a NaN norm makes the factor NaN; an infinite limit means no clipping
  const double ratio = static_cast<double>(a.max_norm) / (norm + static_cast<double>(a.eps));
  float factor = ratio >= 1.0 ? 1.0f : static_cast<float>(ratio);
  if (isinf(a.max_norm) || norm == 0.0) factor = 1.0f;
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.norm = static_cast<float>(norm);
  if (a.in_place && factor == 1.0f) return;
  for (int64_t r = blockIdx.x; r < a.chunks; r += gridDim.x) {
    const int64_t c = a.chunks - 1 - r;
    const int i = tensor_of(a, c);
    const int64_t at = (c - a.t[i].first_chunk) * kClipChunk;
    const int n = static_cast<int>(min(static_cast<int64_t>(kClipChunk), a.t[i].n - at));
    if ((a.f32[i >> 5] >> (i & 31)) & 1u)
      scale_range(static_cast<const float*>(a.t[i].in) + at, static_cast<float*>(a.t[i].out) + at,
                  n, factor);
    else
      scale_range(static_cast<const __nv_bfloat16*>(a.t[i].in) + at,
                  static_cast<__nv_bfloat16*>(a.t[i].out) + at, n, factor);
  }
}

template <int LIST>
cudaError_t run_clip(const void* const* in, void* const* out, const int64_t* counts,
                     const int* types, int n, float max_norm, float eps, float* norm,
                     double* partial, int sms, cudaStream_t stream) {
  const int launches = std::max(1, (n + LIST - 1) / LIST);
  const int most = clip_ctas(sms);
  auto prepare = [&](int l, ClipArgs<LIST>& a) {
    a = ClipArgs<LIST>{};
    const int first = l * LIST;
    const int last = std::min(n, first + LIST);
    for (int i = first; i < last; ++i) {
      if (counts[i] == 0) continue;
      const int k = a.tensors++;
      a.t[k] = ClipTensor{in[i], out ? out[i] : const_cast<void*>(in[i]), counts[i], a.chunks};
      if (types[i] == 1) a.f32[k >> 5] |= 1u << (k & 31);
      a.chunks += (counts[i] + kClipChunk - 1) / kClipChunk;
    }
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
    const int grid = prepare(l, a);
    a.partial = partial + 3 * static_cast<int64_t>(sums);
    const cudaError_t e = launch(clip_norm_kernel<LIST>, grid, a);
    if (e != cudaSuccess) return e;
    sums += grid;
  }
  for (int l = 0; l < launches; ++l) {
    const int grid = prepare(l, a);
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
                                  double* partial, int sms, cudaStream_t stream) {
  // a short list keeps the launch's arguments small
  return n <= 64 ? run_clip<64>(in, out, counts, types, n, max_norm, eps, norm, partial, sms,
                                stream)
                 : run_clip<kClipList>(in, out, counts, types, n, max_norm, eps, norm, partial,
                                       sms, stream);
}

}  // namespace gbf
