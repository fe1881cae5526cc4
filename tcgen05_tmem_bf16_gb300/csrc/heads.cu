// heads.cu -- entry points of the operators at the two ends of a language
// model and of its training step: argument checks, workspace layout, launch.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/gbfuse.h"
#include "internal.h"

namespace gbf {

namespace {

constexpr int64_t kMaxInt = (int64_t(1) << 31) - 1;
constexpr int kMaxSms = 152;  // of the device this library is built for

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
bool aligned(const void* p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
gbf_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? GBF_OK : GBF_ERR_CUDA; }

// Sections of a workspace, each on a 256-byte boundary; with a null base it
// only adds up their sizes.
struct Sections {
  uint8_t* base;
  size_t at = 0;
  template <typename T>
  T* take(size_t count) {
    T* p = base ? reinterpret_cast<T*>(base + at) : nullptr;
    at += align256(count * sizeof(T));
    return p;
  }
};

gbf_status_t check_ids(const void* ids, int index_type, int64_t M, int64_t V, int64_t D) {
  if (!ids || M < 0 || V < 0 || D < 0) return GBF_ERR_INVALID_ARG;
  if (index_type != GBF_INDEX_I64 && index_type != GBF_INDEX_I32) return GBF_ERR_INVALID_ARG;
  if (!aligned(ids, index_type == GBF_INDEX_I64 ? 8 : 4)) return GBF_ERR_MISALIGNED;
  if (D % 8 != 0 || M > kMaxInt || V > kMaxInt - 1 || D > kMaxInt) return GBF_ERR_UNSUPPORTED_SHAPE;
  return GBF_OK;
}

constexpr int64_t kMaxSorted = int64_t(1) << 30;

size_t embed_grad_sections(void* base, int64_t M, int64_t V, int64_t D, EmbedGradWs* ws) {
  Sections s{static_cast<uint8_t*>(base)};
  const int64_t piece = embed_piece(M, static_cast<int>(D));
  const size_t parts = static_cast<size_t>((M + piece - 1) / piece) * D;
  ws->key0 = s.take<int>(M);
  ws->idx0 = s.take<int>(M);
  ws->key1 = s.take<int>(M);
  ws->idx1 = s.take<int>(M);
  ws->present = s.take<unsigned>((V + 31) / 32);
  ws->head = s.take<float>(parts);
  ws->tail = s.take<float>(parts);
  return s.at;
}

}  // namespace

size_t heads_workspace_size(int op, int64_t M, int64_t N, int64_t K) {
  switch (op) {
    case GBF_OP_EMBEDDING_GRAD: {
      if (M > kMaxSorted || N > kMaxInt || K > kMaxInt) return 0;
      EmbedGradWs ws;
      return embed_grad_sections(nullptr, M, N, K, &ws);
    }
    case GBF_OP_CLIP_GRAD_NORM:
      if (M > kMaxInt) return 0;
      return align256(static_cast<size_t>(clip_launches(static_cast<int>(M))) *
                      clip_ctas(kMaxSms) * 3 * sizeof(double));
    default: return 0;
  }
}

}  // namespace gbf

using namespace gbf;

extern "C" {

gbf_status_t gbf_embedding_lookup(const void* ids, int index_type, const void* table, void* out,
                              int64_t M, int64_t V, int64_t D, float scale, gbf_stream_t stream) {
  gbf_status_t st = check_ids(ids, index_type, M, V, D);
  if (st != GBF_OK) return st;
  if (!table || !out) return GBF_ERR_INVALID_ARG;
  if (!aligned(table, 16) || !aligned(out, 16)) return GBF_ERR_MISALIGNED;
  // one warp per 1024 columns of a row, four warps per CTA
  if (D > 0 && M > kMaxInt / ((D + 1023) / 1024)) return GBF_ERR_UNSUPPORTED_SHAPE;
  const DeviceInfo* dev;
  unsigned* err;
  if ((st = lib_device(&dev, &err)) != GBF_OK) return st;
  if (M == 0 || D == 0) return GBF_OK;
  return cuda_status(launch_embedding_lookup(
      ids, index_type == GBF_INDEX_I64, static_cast<const __nv_bfloat16*>(table),
      static_cast<__nv_bfloat16*>(out), M, V, static_cast<int>(D), scale,
      reinterpret_cast<cudaStream_t>(stream)));
}

gbf_status_t gbf_embedding_grad(const void* ids, int index_type, const void* dout, void* dtable,
                            int64_t M, int64_t V, int64_t D, float scale, int accumulate,
                            void* workspace, size_t workspace_bytes, gbf_stream_t stream) {
  gbf_status_t st = check_ids(ids, index_type, M, V, D);
  if (st != GBF_OK) return st;
  if (!dout || !dtable || (accumulate != 0 && accumulate != 1)) return GBF_ERR_INVALID_ARG;
  if (!aligned(dout, 16) || !aligned(dtable, 16) || !aligned(workspace, 16))
    return GBF_ERR_MISALIGNED;
  const int64_t segs = (D + 1023) / 1024;
  if (M > kMaxSorted || (D > 0 && M > kMaxInt / segs)) return GBF_ERR_UNSUPPORTED_SHAPE;
  EmbedGradWs ws;
  const size_t need = embed_grad_sections(workspace, M, V, D, &ws);
  if (need && (!workspace || workspace_bytes < need)) return GBF_ERR_WORKSPACE;
  const DeviceInfo* dev;
  unsigned* err;
  if ((st = lib_device(&dev, &err)) != GBF_OK) return st;
  if (V == 0 || D == 0) return GBF_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (M == 0) {  // no positions: an empty sum in every row
    if (accumulate) return GBF_OK;
    return cuda_status(cudaMemsetAsync(dtable, 0, static_cast<size_t>(V) * D * 2, s));
  }
  return cuda_status(launch_embedding_grad(
      ids, index_type == GBF_INDEX_I64, static_cast<const __nv_bfloat16*>(dout),
      static_cast<__nv_bfloat16*>(dtable), static_cast<int>(M), static_cast<int>(V),
      static_cast<int>(D), scale, accumulate == 1, ws, dev->sms, s));
}

gbf_status_t gbf_clip_grad_norm(const void* const* grads, void* const* out, const int64_t* counts,
                            const int* types, int tensors, float max_norm, float eps, float* norm,
                            void* workspace, size_t workspace_bytes, gbf_stream_t stream) {
  if (tensors < 0 || !norm || !(max_norm >= 0.0f) || !(eps >= 0.0f) || std::isinf(eps))
    return GBF_ERR_INVALID_ARG;
  if (tensors > 0 && (!grads || !counts || !types)) return GBF_ERR_INVALID_ARG;
  for (int i = 0; i < tensors; ++i) {
    if (counts[i] < 0 || (types[i] != GBF_TYPE_BF16 && types[i] != GBF_TYPE_F32))
      return GBF_ERR_INVALID_ARG;
    if (counts[i] == 0) continue;
    if (!grads[i] || (out && !out[i])) return GBF_ERR_INVALID_ARG;
    const size_t size = types[i] == GBF_TYPE_F32 ? 4 : 2;
    if (!aligned(grads[i], size) || (out && !aligned(out[i], size))) return GBF_ERR_MISALIGNED;
  }
  if (!aligned(norm, 4) || !aligned(workspace, 16)) return GBF_ERR_MISALIGNED;
  const DeviceInfo* dev;
  unsigned* err;
  gbf_status_t st;
  const size_t need = gbf_workspace_size(GBF_OP_CLIP_GRAD_NORM, tensors, 0, 0, 1);
  if (!workspace || workspace_bytes < need) return GBF_ERR_WORKSPACE;
  if ((st = lib_device(&dev, &err)) != GBF_OK) return st;
  return cuda_status(launch_clip_grad_norm(grads, out, counts, types, tensors, max_norm, eps, norm,
                                           static_cast<double*>(workspace),
                                           dev->sms < kMaxSms ? dev->sms : kMaxSms,
                                           reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
