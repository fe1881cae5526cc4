// heads.cu -- entry points of the operators at the two ends of a language
// model and of its training step: argument checks, workspace layout, launch.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
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

// The address of an array without elements may be null, as torch gives it.
gbf_status_t check_ids(const void* ids, int index_type, int64_t M, int64_t V, int64_t D) {
  if ((!ids && M != 0) || M < 0 || V < 0 || D < 0) return GBF_ERR_INVALID_ARG;
  if (index_type != GBF_INDEX_I64 && index_type != GBF_INDEX_I32) return GBF_ERR_INVALID_ARG;
  if (!aligned(ids, index_type == GBF_INDEX_I64 ? 8 : 4)) return GBF_ERR_MISALIGNED;
  if (D % 8 != 0 || M > kMaxInt || V > kMaxInt - 1 || D > kMaxInt) return GBF_ERR_UNSUPPORTED_SHAPE;
  return GBF_OK;
}

constexpr int64_t kMaxSorted = int64_t(1) << 30;

size_t embed_grad_sections(void* base, int64_t M, int64_t D, EmbedGradWs* ws) {
  Sections s{static_cast<uint8_t*>(base)};
  const int64_t piece = embed_piece(M, static_cast<int>(D));
  const size_t parts = static_cast<size_t>((M + piece - 1) / piece) * D;
  ws->key0 = s.take<int>(M);
  ws->idx0 = s.take<int>(M);
  ws->key1 = s.take<int>(M);
  ws->idx1 = s.take<int>(M);
  ws->head = s.take<float>(parts);
  ws->tail = s.take<float>(parts);
  return s.at;
}

// What that comes to with M positions or fewer, which may be cut into shorter pieces.
size_t embed_grad_workspace(int64_t M, int64_t D) {
  Sections s{nullptr};
  for (int i = 0; i < 4; ++i) s.take<int>(M);
  const size_t parts = static_cast<size_t>(embed_most_pieces(M, static_cast<int>(D))) * D;
  s.take<float>(parts);
  s.take<float>(parts);
  return s.at;
}

// ---- linear cross entropy

constexpr int kCePairs = 76;  // CTA pairs that run at once
constexpr int kCeTileRows = 256;

// Columns of the vocabulary per piece of the backward pass: as many whole
// tiles as keep G of the piece within 256 MB, at least 512, and no more than 16 chains
// of dx hold.
constexpr int64_t kPieceBytes = int64_t(256) << 20;
int64_t ce_piece(int64_t M, int64_t V) {
  const int64_t cols = std::max<int64_t>(512, kPieceBytes / 2 / std::max<int64_t>(M, 1) / 512 * 512);
  return std::min({cols, V, 16 * kGradChain});
}

int64_t ceil_div64(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Row tiles per unit of work: two that share a column tile, or a lone one where
// there is no second.
int ce_streams(int64_t M) { return M > kCeTileRows ? 2 : 1; }
// The same for lists, where a lone one is also taken if the rounds of units over the pairs
// are shorter so (a unit of two takes about 1.7 times as long): 300 rows x 4000 x 1000
// trained 66 us, two 80.5; 300 x 20000 x 512 86, 104; 1000 x 4000 x 1000 84, 101.
int ce_streams(int64_t M, int64_t cols, bool lists) {
  if (!lists || ce_streams(M) == 1) return ce_streams(M);
  const int64_t v = ceil_div64(cols, 256);
  const int64_t one = ceil_div64(ceil_div64(M, kCeTileRows) * v, kCePairs);
  const int64_t two = ceil_div64(ceil_div64(M, 2 * kCeTileRows) * v, kCePairs);
  return one * 10 < two * 17 ? 1 : 2;
}
// Whether the logits' K is taken in several chains (above kCeSwapMax rows): then in
// units of one row tile, by a launch of their own (linear_ce.cu).
bool ce_chained(int64_t D) { return ceil_div64(D, kBK) > kCeChain; }

// Parts of K of the product for dx, each with an fp32 buffer of its own, 16 at
// most and none shorter than 8 K blocks or longer than a chain.  With one row tile: as
// many as give one round of units over the pairs (64 rows, 32000 x 4096, dx alone: 4
// parts 103 us, 5 parts, a second round for four of 80 units, 129, 14 parts 108 and more
// beside dw).  Else: none longer than half of what a pair has to do in all, the
// logits among it also where their launch is another (without them there are more
// parts: 1024 x 32000 x 4096 491 us, 501; 4096 x 32000 x 8192 3.59 ms, 3.66).
int64_t ce_least_splits(int64_t cols) { return ceil_div64(cols, kGradChain); }
int64_t ce_most_splits(int64_t cols) {
  return std::max<int64_t>(1, std::min<int64_t>(ceil_div64(cols, 64) / 8, 16));
}
// Bytes of several of them: sizes come to 58 MB at most (of 3e7 random ones); held, so
// that the size of a workspace never falls with M.
constexpr int64_t kCePartBytes = int64_t(64) << 20;
int64_t ce_part_bytes(int64_t M, int64_t D) { return ceil_div64(M, 512) * 512 * D * 4; }
int ce_splits(int64_t M, int64_t D, int64_t cols) {
  const int64_t d = ceil_div64(D, kCeTileRows), k = ceil_div64(cols, 64);
  const int64_t most = ce_most_splits(cols);
  if (ce_streams(M) == 1)
    return static_cast<int>(std::max(ce_least_splits(cols), std::min(most, kCePairs / d)));
  const int64_t rows = 2 * kCeTileRows;
  const int64_t m = ceil_div64(M, rows), v = ceil_div64(cols, kCeTileRows);
  const int64_t all = m * d * k + m * v * ceil_div64(D, 64) +
                      ceil_div64(cols, rows) * d * ceil_div64(M, 64);
  const int64_t half = std::max<int64_t>(1, all / kCePairs / 2);
  const int64_t held = std::max<int64_t>(1, kCePartBytes / ce_part_bytes(M, D));
  return static_cast<int>(std::max(ce_least_splits(cols), std::min({most, ceil_div64(k, half), held})));
}
// The same of the product for dw, whose K are the rows; rows between the parts.
int ce_dw_splits(int64_t M) { return static_cast<int>(std::max<int64_t>(1, ceil_div64(M, kGradChain))); }
int64_t ce_dw_pad(int64_t cols) { return ceil_div64(cols, 32) * 32; }
size_t ce_dw_part_bytes(int64_t M, int64_t D, int64_t cols) {
  const int64_t n = ce_dw_splits(M);
  return n > 1 ? static_cast<size_t>(n * ce_dw_pad(cols)) * D * 4 : 0;
}

// Columns of a tile of the forward pass: 224 where the rounds of such tiles over
// the pairs are shorter than those of 256 (1024 rows x 32000 x 1024, four rounds
// either way: 59.5 us, 64.4 with 256; 700 x 50001 x 1024: 81.5, 87.6).  In chains,
// units of one row tile, an MMA takes as long for 224 columns as for 256.
int ce_tile_cols(int64_t M, int64_t V, int64_t D) {
  if (ce_streams(M) == 1 || ce_chained(D)) return 256;
  const int64_t m = ceil_div64(M, 2 * kCeTileRows);
  const int64_t wide = ceil_div64(m * ceil_div64(V, 256), kCePairs) * 256;
  const int64_t narrow = ceil_div64(m * ceil_div64(V, 224), kCePairs) * 224;
  return narrow * 102 < wide * 100 ? 224 : 256;
}

// Partial sums per row of the forward pass: two per tile, with swapped roles one
// per 32 columns.
int64_t ce_parts(int64_t M, int64_t V, int64_t D) {
  return M <= kCeSwapMax ? 4 * ceil_div64(V, 128) : 2 * ceil_div64(V, ce_tile_cols(M, V, D));
}

struct CeWs {
  int *count, *rows, *tgt;
  unsigned* ticket;
  float *lse2, *dl, *tlog, *dxacc, *dwacc, *chain;
  float2* part;
  double* sums;
  __nv_bfloat16 *xc, *g[2];
};

// Sums over the segments before the last of a logit's K: for each CTA the padded
// rows x 128 columns.
size_t ce_chain_floats(int64_t M, int64_t D) {
  if (M > kCeSwapMax || ce_swap_segments(M, static_cast<int>(ceil_div64(D, kBK))) == 1) return 0;
  return size_t(2) * kMaxSms * ce_swap_rows(M) * 128;
}

size_t ce_sections(void* base, int64_t M, int64_t V, int64_t D, bool grad, CeWs* w,
                   bool twice = false) {
  Sections s{static_cast<uint8_t*>(base)};
  *w = CeWs{};
  w->count = s.take<int>(1);
  w->ticket = s.take<unsigned>(1);
  w->rows = s.take<int>(M);
  w->tgt = s.take<int>(M);
  w->xc = s.take<__nv_bfloat16>(static_cast<size_t>(M) * D);
  w->chain = s.take<float>(ce_chain_floats(M, D));
  if (!grad) {
    w->part = s.take<float2>(static_cast<size_t>(ce_parts(M, V, D)) * M);
    w->tlog = s.take<float>(M);
    w->sums = s.take<double>(ceil_div64(M, 8));  // one per CTA of the join
  } else {
    const int64_t cols = ce_piece(M, V);
    const int64_t m_pad = ceil_div64(M, 512) * 512;
    w->lse2 = s.take<float>(M);
    w->dl = s.take<float>(M);
    // G of two pieces: one is written while the other's products run
    const size_t g = M <= kCeSwapMax ? static_cast<size_t>(ce_swap_rows(M)) * cols * (twice ? 2 : 1)
                                     : static_cast<size_t>(M) * (ceil_div64(cols, 8) * 8);
    w->g[0] = s.take<__nv_bfloat16>(g);
    w->g[1] = cols < V ? s.take<__nv_bfloat16>(g) : w->g[0];
    w->dxacc = s.take<float>(static_cast<size_t>(ce_splits(M, D, cols)) * m_pad * D);
    w->dwacc = s.take<float>(ce_dw_part_bytes(M, D, cols) / 4);
  }
  return s.at;
}

// What ce_sections comes to with M rows or fewer, by the largest of each section.
// lists: two bf16 per value of G up to kCeTwiceRows rows.
size_t ce_workspace(int64_t M, int64_t V, int64_t D, bool grad, bool lists) {
  Sections s{nullptr};
  const int64_t few = std::min<int64_t>(M, kCeSwapMax);
  s.take<int>(1);
  s.take<unsigned>(1);
  s.take<int>(M);
  s.take<int>(M);
  s.take<__nv_bfloat16>(static_cast<size_t>(M) * D);
  size_t chain = 0;
  for (int64_t m : {int64_t(16), int64_t(64), int64_t(kCeSwapMax)})  // a size for all rows up to each
    if (ce_swap_rows(few) >= m) chain = std::max(chain, ce_chain_floats(m, D));
  s.take<float>(chain);
  if (!grad) {
    const int64_t part = 4 * ceil_div64(V, 128) * few;
    s.take<float2>(M > few ? std::max(part, 2 * ceil_div64(V, 224) * M) : part);
    s.take<float>(M);
    s.take<double>(ceil_div64(M, 8));
    return s.at;
  }
  s.take<float>(M);
  s.take<float>(M);
  // G of one piece, or of two
  int64_t one = 0, two = 0;
  for (int64_t m = few; m >= 0; --m) {
    const int64_t cols = ce_piece(m, V);
    const int64_t g = ce_swap_rows(m) * cols * (lists && m <= kCeTwiceRows ? 2 : 1);
    one = std::max(one, g);
    if (cols < V) two = std::max(two, g);
  }
  if (M > few) {
    if (ce_piece(M, V) == V) {
      one = std::max(one, M * (ceil_div64(V, 8) * 8));
    } else {
      const int64_t most = std::max(512 * M, kPieceBytes / 2);
      one = std::max(one, most + 8 * M);
      two = std::max(two, most);
    }
  }
  s.take<__nv_bfloat16>(one);
  s.take<__nv_bfloat16>(two);
  const int64_t lone = std::max(ce_least_splits(ce_piece(1, V)),
                                std::min(ce_most_splits(V), kCePairs / ceil_div64(D, kCeTileRows)));
  int64_t acc = lone * ce_part_bytes(std::min<int64_t>(M, kCeTileRows), D);
  if (M > kCeTileRows) {
    const int64_t part = ce_part_bytes(M, D);
    acc = std::max({acc, part, std::min(ce_most_splits(V) * part, kCePartBytes)});
    for (int64_t m = kCeTileRows + 1; m <= std::min<int64_t>(M, 1024); m += 256)  // the least, in steps of 512 rows
      acc = std::max(acc, ce_least_splits(ce_piece(m, V)) * ce_part_bytes(m, D));
  }
  s.take<uint8_t>(acc);
  s.take<uint8_t>(ce_dw_part_bytes(M, D, ce_piece(M, V)));
  return s.at;
}

// Sizes that the kernels' 32-bit coordinates and unit counts hold.
bool ce_sizes_held(int64_t M, int64_t V, int64_t D) {
  if (V < 1 || D < 8 || D % 8 != 0 || M > (int64_t(1) << 24) || V > (int64_t(1) << 26) ||
      D > (int64_t(1) << 20))
    return false;
  const int64_t m = ceil_div64(M, 256), v = ceil_div64(V, 256), d = ceil_div64(D, 256);
  return m * v <= kMaxInt / 2 && m * d * 16 <= kMaxInt / 2 && v * d <= kMaxInt / 2;
}

gbf_status_t check_ce(const void* x, const void* w, const void* targets, int index_type,
                      int64_t M, int64_t V, int64_t D, float alpha) {
  gbf_status_t st = check_ids(targets, index_type, M, V, D);
  if (st != GBF_OK) return st;
  if ((!x && M > 0) || !w || !std::isfinite(alpha)) return GBF_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(w, 16)) return GBF_ERR_MISALIGNED;
  return ce_sizes_held(M, V, D) ? GBF_OK : GBF_ERR_UNSUPPORTED_SHAPE;
}

// K-major operand: rows of D values, 64 x 128 boxes (half a tile's columns of W).
bool ce_map_k(CUtensorMap* m, const void* p, int64_t inner, int64_t outer, int64_t ld,
              uint32_t rows = 128) {
  return lib_tmap_2d(m, p, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, inner, outer, ld * 2, kBK, rows,
                     CU_TENSOR_MAP_SWIZZLE_128B);
}
// Operand with one row per k: 64 x 64 boxes.
bool ce_map_mn(CUtensorMap* m, const void* p, int64_t inner, int64_t outer, int64_t ld) {
  return lib_tmap_2d(m, p, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, inner, outer, ld * 2, 64, kBK,
                     CU_TENSOR_MAP_SWIZZLE_128B);
}
// Operands of the swapped roles: boxes of 64 x the padded rows, 64 x 128.
bool ce_maps_swap(CeSwap* a, const void* w, const void* xc, const void* x, int64_t M, int64_t V,
                  int64_t D) {
  const uint32_t rows = static_cast<uint32_t>(ce_swap_rows(M));
  return ce_map_k(&a->w, w, D, V, D) &&
         lib_tmap_2d(&a->x[0], xc, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, D, M, D * 2, kBK, rows,
                     CU_TENSOR_MAP_SWIZZLE_128B) &&
         lib_tmap_2d(&a->x[1], x, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, D, M, D * 2, kBK, rows,
                     CU_TENSOR_MAP_SWIZZLE_128B);
}
bool ce_map_out(CUtensorMap* m, const void* p, int64_t inner, int64_t outer, int64_t ld) {
  return lib_tmap_2d(m, p, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, inner, outer, ld * 2, 32, 32,
                     CU_TENSOR_MAP_SWIZZLE_64B);
}
// With one row tile per unit the ending stores rows of 128 bytes.
bool ce_map_dw(CUtensorMap* m, const void* p, int64_t D, int64_t V, bool wide) {
  return wide ? lib_tmap_2d(m, p, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, D, V, D * 2, 64, 32,
                            CU_TENSOR_MAP_SWIZZLE_128B)
              : ce_map_out(m, p, D, V, D);
}
bool ce_map_out_f32(CUtensorMap* m, const void* p, int64_t inner, int64_t outer) {
  return lib_tmap_2d(m, p, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, inner, outer, inner * 4, 16, 32,
                     CU_TENSOR_MAP_SWIZZLE_64B);
}

// One launch: a CTA pair per unit of work at most, with M rows scored.
gbf_status_t run_ce_gemm(const CeLaunch& launch, const CeEnd& end, int64_t M, int streams,
                         bool chains, const DeviceInfo& dev, unsigned* err, cudaStream_t s) {
  int64_t units = 0;
  for (const CeJob& j : launch.job) {
    if (j.mode == kCeNone) continue;
    const int64_t rows = j.mode == kCeDw ? j.cols : M;
    const int64_t n = j.mode == kCeLse || j.mode == kCeGrad ? j.cols : launch.d;
    units += ceil_div64(rows, kCeTileRows * streams) * ceil_div64(n, j.bn) * j.splits;
  }
  const int grid = 2 * static_cast<int>(std::min<int64_t>(units, dev.pairs));
  return cuda_status(launch_ce_gemm(launch, end, streams, chains, grid, lib_ctl(err, grid), s));
}

// The sizes and arrays that both passes of both losses work on; pick.list null: the
// hard targets' loss.
struct CeCall {
  const void *x, *w, *targets;
  bool ids64;
  int64_t M, V, D;
  float alpha;
  CeWs ws;
  CePick pick;
  const DeviceInfo* dev;
  unsigned* err;
  cudaStream_t s;
};

// Forward pass of rows > 0.
gbf_status_t ce_forward(const CeCall& call, float* loss, float* lse, float* mean) {
  const auto [x, w, targets, ids64, M, V, D, alpha, ws, pick, dev, err, s] = call;
  const int swap_sms = std::min(dev->sms, kMaxSms);
  gbf_status_t st;
  CePrep p{};
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.xc = ws.xc;
  p.loss = loss;
  p.lse_out = lse;
  p.count = ws.count;
  p.rows = ws.rows;
  p.tgt = ws.tgt;
  p.ticket = ws.ticket;
  p.M = static_cast<int>(M);
  p.V = static_cast<int>(V);
  p.D = static_cast<int>(D);
  const bool few = M <= kCeSwapMax, chains = ce_chained(D);
  CeLaunch launch{};
  for (CeJob& j : launch.job) j.bn = 256;
  CeSwap swap{};
  if (few) {
    if (!ce_maps_swap(&swap, w, ws.xc, x, M, V, D)) return GBF_ERR_CUDA;
    swap.cols = p.V;
    swap.num_kb = static_cast<int>(ceil_div64(D, kBK));
    swap.targets = targets;
    swap.ids64 = ids64;
    swap.ticket = ws.ticket;
  } else {
    launch.d = p.D;
    CeJob& job = launch.job[1];
    job.bn = pick.list ? 256 : ce_tile_cols(M, V, D);
    if (!ce_map_k(&job.a[0], ws.xc, D, M, D) || !ce_map_k(&job.a[1], x, D, M, D) ||
        !ce_map_k(&job.b[0], w, D, V, D, job.bn / 2))
      return GBF_ERR_CUDA;
    job.mode = kCeLse;
    job.cols = p.V;
    job.splits = 1;
  }
  CeEnd end{};
  end.count = ws.count;
  end.tgt = ws.tgt;
  end.part = ws.part;
  end.tlog = ws.tlog;
  end.chain = ws.chain;
  end.c2 = static_cast<float>(alpha * 1.4426950408889634);
  end.M = p.M;
  end.rows = ws.rows;
  end.pick = pick;
  CeJoin join{};
  join.count = ws.count;
  join.rows = few ? nullptr : ws.rows;
  join.targets = targets;
  join.ids64 = ids64;
  join.V = p.V;
  join.part = ws.part;
  join.tlog = ws.tlog;
  join.ticket = ws.ticket;
  join.sums = ws.sums;
  join.loss = loss;
  join.lse = lse;
  join.mean = mean;
  join.c2 = end.c2;
  join.M = p.M;
  join.parts = static_cast<int>(few || !pick.list ? ce_parts(M, V, D) : 2 * ceil_div64(V, 256));
  join.pick = pick;
  if (!few && (st = cuda_status(launch_ce_prep(targets, ids64, p, dev->sms,
                                               s))) != GBF_OK)
    return st;
  st = few ? cuda_status(launch_ce_swap(swap, false, end, swap_sms, lib_ctl(err, 2 * swap_sms), s))
           : run_ce_gemm(launch, end, M, chains ? 1 : ce_streams(M, V, pick.list != nullptr), chains,
                         *dev, err, s);
  if (st != GBF_OK) return st;
  return cuda_status(launch_ce_join(join, s));
}

// Backward pass of rows > 0.
gbf_status_t ce_backward(const CeCall& call, const float* lse, const float* dloss, void* dx,
                         void* dw, float scale, int reduction) {
  const auto [x, w, targets, ids64, M, V, D, alpha, ws, pick, dev, err, s] = call;
  const int swap_sms = std::min(dev->sms, kMaxSms);
  gbf_status_t st;
  CePrep p{};
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.xc = ws.xc;
  p.lse_in = lse;
  p.dloss = dloss;
  p.dx = static_cast<__nv_bfloat16*>(dx);
  p.count = ws.count;
  p.rows = ws.rows;
  p.tgt = ws.tgt;
  p.lse2 = ws.lse2;
  p.dl = ws.dl;
  p.M = static_cast<int>(M);
  p.V = static_cast<int>(V);
  p.D = static_cast<int>(D);
  if ((st = cuda_status(launch_ce_prep(targets, ids64, p, dev->sms, s))) !=
      GBF_OK)
    return st;
  const int64_t piece = ce_piece(M, V);
  const bool few = M <= kCeSwapMax;  // G transposed, by the swapped roles
  const bool chains = !few && ce_chained(D);
  const bool twice = pick.list && M <= kCeTwiceRows;
  const int64_t rows = ce_swap_rows(M);
  const int64_t ld = few ? (twice ? 2 : 1) * rows : ceil_div64(piece, 8) * 8;
  const int64_t m_pad = ceil_div64(M, 512) * 512;
  const int splits = ce_splits(M, D, piece), dw_splits = ce_dw_splits(M);
  const int streams = ce_streams(M, piece, pick.list != nullptr);
  CeEnd end{};
  end.count = ws.count;
  end.tgt = ws.tgt;
  end.lse2 = ws.lse2;
  end.dl = ws.dl;
  end.chain = ws.chain;
  end.c2 = static_cast<float>(alpha * 1.4426950408889634);
  end.scale = alpha * scale;
  end.mean = reduction == GBF_REDUCE_MEAN;
  end.M = p.M;
  end.m_pad = static_cast<int>(m_pad);
  end.rows = ws.rows;
  end.pick = pick;
  // Launch n: G of piece n, and the products of piece n - 1's G.
  const int64_t pieces = ceil_div64(V, piece);
  for (int64_t n = 0; n <= pieces; ++n) {
    CeLaunch launch{}, logits{};
    launch.d = logits.d = p.D;
    launch.twice = twice;
    for (CeJob& j : launch.job) j.bn = 256;
    for (CeJob& j : logits.job) j.bn = 256;
    if (n < pieces && few) {
      const int64_t v0 = n * piece;
      CeSwap swap{};
      if (!ce_maps_swap(&swap, w, ws.xc, x, M, V, D)) return GBF_ERR_CUDA;
      swap.gt = ws.g[n & 1];
      swap.v0 = static_cast<int>(v0);
      swap.cols = static_cast<int>(std::min(piece, V - v0));
      swap.num_kb = static_cast<int>(ceil_div64(D, kBK));
      st = cuda_status(launch_ce_swap(swap, true, end, swap_sms, lib_ctl(err, 2 * swap_sms), s));
      if (st != GBF_OK) return st;
    } else if (n < pieces) {
      CeJob& job = chains ? logits.job[1] : launch.job[1];
      const int64_t v0 = n * piece, cols = std::min(piece, V - v0);
      job.mode = kCeGrad;
      job.cols = static_cast<int>(cols);
      job.v0 = static_cast<int>(v0);
      job.splits = 1;
      if (!ce_map_k(&job.a[0], ws.xc, D, M, D) || !ce_map_k(&job.a[1], x, D, M, D) ||
          !ce_map_k(&job.b[0], w, D, V, D) || !ce_map_out(&job.o, ws.g[n & 1], cols, M, ld))
        return GBF_ERR_CUDA;
      if (chains && (st = run_ce_gemm(logits, end, M, 1, true, *dev, err, s)) != GBF_OK) return st;
    }
    if (n > 0) {
      const int64_t v0 = (n - 1) * piece, cols = std::min(piece, V - v0);
      const __nv_bfloat16* g = ws.g[(n - 1) & 1];
      if (dx) {
        CeJob& job = launch.job[0];
        job.mode = kCeDx;
        job.cols = static_cast<int>(cols);
        job.v0 = static_cast<int>(v0);
        job.splits = splits;
        job.add = n > 1;
        job.gt = few;
        if (!(few ? ce_map_mn(&job.a[0], g, ld, cols, ld) : ce_map_k(&job.a[0], g, cols, M, ld)) ||
            !ce_map_mn(&job.b[0], w, D, V, D) ||
            !ce_map_out_f32(&job.o, ws.dxacc, D, splits * m_pad))
          return GBF_ERR_CUDA;
      }
      if (dw) {
        CeJob& job = launch.job[2];
        job.mode = kCeDw;
        job.cols = static_cast<int>(cols);
        job.v0 = static_cast<int>(v0);
        job.splits = dw_splits;
        job.pad = static_cast<int>(ce_dw_pad(piece));
        job.gt = few;
        if (!(few ? ce_map_k(&job.a[0], g, rows, cols, ld) : ce_map_mn(&job.a[0], g, cols, M, ld)) ||
            (twice && !ce_map_k(&job.a[1], g + rows, rows, cols, ld)) ||
            !ce_map_mn(&job.b[0], ws.xc, D, M, D) ||
            !ce_map_mn(&job.b[1], x, D, M, D) ||
            !(dw_splits > 1 ? ce_map_out_f32(&job.o, ws.dwacc, D, dw_splits * job.pad)
                            : ce_map_dw(&job.o, dw, D, V, streams == 1)))
          return GBF_ERR_CUDA;
      }
    }
    if ((few || chains) && n == 0) continue;  // no G yet
    if ((st = run_ce_gemm(launch, end, M, streams, false, *dev, err, s)) != GBF_OK) return st;
    if (n > 0 && dw && dw_splits > 1) {
      const CeJob& job = launch.job[2];
      CeDxOut out{};
      out.count = ws.count;
      out.acc = ws.dwacc;
      out.dx = static_cast<__nv_bfloat16*>(dw) + job.v0 * D;
      out.scale = end.scale;
      out.mean = end.mean;
      out.m_pad = job.pad;
      out.splits = dw_splits;
      out.D = p.D;
      out.dw_rows = job.cols;
      if ((st = cuda_status(launch_ce_dx(out, job.cols, dev->sms, s))) != GBF_OK) return st;
    }
  }
  if (!dx) return GBF_OK;
  CeDxOut out{};
  out.count = ws.count;
  out.rows = ws.rows;
  out.acc = ws.dxacc;
  out.dx = p.dx;
  out.scale = end.scale;
  out.mean = end.mean;
  out.m_pad = end.m_pad;
  out.splits = splits;
  out.D = p.D;
  out.twice = twice;
  return cuda_status(launch_ce_dx(out, p.M, dev->sms, s));
}

// ---- distillation from a teacher's top logits

struct DistillWs {
  CeWs ce;
  int2* list;
  uint16_t* at;
  int* tgt;
  float* dots;
};
// Columns per entry of `at`: those that a warp of the ending holds at a time.
int pick_shift(int64_t M) { return M <= kCeSwapMax ? 5 : 7; }
int64_t pick_stride(int64_t M, int64_t V) { return (V >> pick_shift(M)) + 2; }

size_t distill_sections(void* base, int64_t M, int64_t V, int64_t D, int64_t K, bool grad,
                        DistillWs* w) {
  const size_t at = ce_sections(base, M, V, D, grad, &w->ce, M <= kCeTwiceRows);
  Sections s{static_cast<uint8_t*>(base), at};
  w->list = s.take<int2>(static_cast<size_t>(M) * (K + 1));
  w->at = s.take<uint16_t>(static_cast<size_t>(M) * pick_stride(M, V));
  w->tgt = s.take<int>(M);
  w->dots = grad ? nullptr : s.take<float>(static_cast<size_t>(M) * K);
  return s.at;
}

// With M rows or fewer.
size_t distill_workspace(int64_t M, int64_t V, int64_t D, int64_t K, bool grad) {
  Sections s{nullptr, ce_workspace(M, V, D, grad, true)};
  const int64_t few = std::min<int64_t>(M, kCeSwapMax);
  s.take<int2>(static_cast<size_t>(M) * (K + 1));
  s.take<uint16_t>(M > few ? std::max(few * pick_stride(few, V), M * pick_stride(M, V))
                           : M * pick_stride(M, V));
  s.take<int>(M);
  if (!grad) s.take<float>(static_cast<size_t>(M) * K);
  return s.at;
}

gbf_status_t check_distill(const void* x, const void* w, const void* ids, const void* logits,
                           int index_type, int teacher_type, int64_t M, int64_t V, int64_t D,
                           int64_t K, float alpha, float beta) {
  gbf_status_t st = check_ce(x, w, ids, index_type, M, V, D, alpha);
  if (st != GBF_OK) return st;
  if ((!logits && M > 0) || K < 0 || !std::isfinite(beta) || !(beta > 0.0f) ||
      (teacher_type != GBF_TYPE_BF16 && teacher_type != GBF_TYPE_F32))
    return GBF_ERR_INVALID_ARG;
  if (!aligned(logits, teacher_type == GBF_TYPE_F32 ? 4 : 2)) return GBF_ERR_MISALIGNED;
  return K >= 1 && K <= kPickMax ? GBF_OK : GBF_ERR_UNSUPPORTED_SHAPE;
}

// Launches the lists and fills in what a pass takes of them.
gbf_status_t make_lists(const void* ids, const void* logits, int teacher_type, float beta,
                        int64_t K, const DistillWs& ws, CeCall* call) {
  CeLists p{};
  p.ids = ids;
  p.logits = logits;
  p.ids64 = call->ids64;
  p.bf16 = teacher_type == GBF_TYPE_BF16;
  p.beta = beta;
  p.list = ws.list;
  p.at = ws.at;
  p.tgt = ws.tgt;
  p.M = call->M;
  p.V = static_cast<int>(call->V);
  p.K = static_cast<int>(K);
  p.stride = static_cast<int>(pick_stride(call->M, call->V));
  p.shift = pick_shift(call->M);
  call->pick = CePick{ws.list, ws.at, ws.dots, p.K, p.stride, p.shift};
  call->targets = ws.tgt;
  call->ids64 = false;
  return cuda_status(launch_ce_lists(p, call->dev->sms, call->s));
}

}  // namespace

size_t heads_workspace_size(int op, int64_t M, int64_t N, int64_t K) {
  switch (op) {
    case GBF_OP_EMBEDDING_GRAD: {
      if (M > kMaxSorted || N > kMaxInt || K > kMaxInt) return 0;
      return embed_grad_workspace(M, K);
    }
    case GBF_OP_CLIP_GRAD_NORM:
      if (M > kMaxInt) return 0;
      return align256(static_cast<size_t>(clip_launches(static_cast<int>(M))) *
                      clip_ctas(kMaxSms) * 3 * sizeof(float2));
    case GBF_OP_LINEAR_CE:
    case GBF_OP_LINEAR_CE_GRAD: {
      if (!ce_sizes_held(M, N, K)) return 0;  // as the entry points refuse them
      return ce_workspace(M, N, K, op == GBF_OP_LINEAR_CE_GRAD, false);
    }
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
  if ((!table && V > 0 && D > 0) || (!out && M > 0 && D > 0)) return GBF_ERR_INVALID_ARG;
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
  if ((!dout && M > 0 && D > 0) || (!dtable && V > 0 && D > 0) ||
      (accumulate != 0 && accumulate != 1))
    return GBF_ERR_INVALID_ARG;
  if (!aligned(dout, 16) || !aligned(dtable, 16) || !aligned(workspace, 16))
    return GBF_ERR_MISALIGNED;
  const int64_t segs = (D + 1023) / 1024;
  if (M > kMaxSorted || (D > 0 && M > kMaxInt / segs)) return GBF_ERR_UNSUPPORTED_SHAPE;
  EmbedGradWs ws;
  const size_t need = embed_grad_sections(workspace, M, D, &ws);
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
                                           static_cast<float2*>(workspace),
                                           dev->sms < kMaxSms ? dev->sms : kMaxSms,
                                           reinterpret_cast<cudaStream_t>(stream)));
}

gbf_status_t gbf_linear_ce(const void* x, const void* w, const void* targets, int index_type,
                           float* loss, float* lse, float* mean, int64_t M, int64_t V, int64_t D,
                           float alpha, void* workspace, size_t workspace_bytes,
                           gbf_stream_t stream) {
  gbf_status_t st = check_ce(x, w, targets, index_type, M, V, D, alpha);
  if (st != GBF_OK) return st;
  if (M > 0 && (!loss || !lse)) return GBF_ERR_INVALID_ARG;
  if (!aligned(loss, 4) || !aligned(lse, 4) || !aligned(mean, 4) || !aligned(workspace, 16))
    return GBF_ERR_MISALIGNED;
  CeWs ws;
  const size_t need = ce_sections(workspace, M, V, D, false, &ws);
  if (!workspace || workspace_bytes < need) return GBF_ERR_WORKSPACE;
  const DeviceInfo* dev;
  unsigned* err;
  if ((st = lib_device(&dev, &err)) != GBF_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (M == 0) return mean ? cuda_status(cudaMemsetAsync(mean, 0, 4, s)) : GBF_OK;
  return ce_forward({x, w, targets, index_type == GBF_INDEX_I64, M, V, D, alpha, ws, CePick{}, dev, err, s},
                    loss, lse, mean);
}

gbf_status_t gbf_linear_ce_grad(const void* x, const void* w, const void* targets, int index_type,
                                const float* lse, const float* dloss, void* dx, void* dw,
                                int64_t M, int64_t V, int64_t D, float alpha, float scale,
                                int reduction, void* workspace, size_t workspace_bytes,
                                gbf_stream_t stream) {
  gbf_status_t st = check_ce(x, w, targets, index_type, M, V, D, alpha);
  if (st != GBF_OK) return st;
  if ((M > 0 && (!lse || (!dx && !dw))) ||
      (reduction != GBF_REDUCE_SUM && reduction != GBF_REDUCE_MEAN))
    return GBF_ERR_INVALID_ARG;
  if (!aligned(lse, 4) || !aligned(dloss, 4) || !aligned(dx, 16) || !aligned(dw, 16) ||
      !aligned(workspace, 16))
    return GBF_ERR_MISALIGNED;
  CeWs ws;
  const size_t need = ce_sections(workspace, M, V, D, true, &ws);
  if (!workspace || workspace_bytes < need) return GBF_ERR_WORKSPACE;
  const DeviceInfo* dev;
  unsigned* err;
  if ((st = lib_device(&dev, &err)) != GBF_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (M == 0)
    return dw ? cuda_status(cudaMemsetAsync(dw, 0, static_cast<size_t>(V) * D * 2, s)) : GBF_OK;
  return ce_backward({x, w, targets, index_type == GBF_INDEX_I64, M, V, D, alpha, ws, CePick{}, dev, err, s},
                     lse, dloss, dx, dw, scale, reduction);
}

size_t gbf_linear_distill_workspace_size(int64_t M, int64_t V, int64_t D, int64_t K, int grad) {
  if (M < 0 || K < 1 || K > kPickMax || !ce_sizes_held(M, V, D)) return 0;  // as refused
  return distill_workspace(M, V, D, K, grad != 0);
}

gbf_status_t gbf_linear_distill(const void* x, const void* w, const void* ids, int index_type,
                                const void* logits, int teacher_type, float* loss, float* lse,
                                float* mean, int64_t M, int64_t V, int64_t D, int64_t K,
                                float alpha, float beta, void* workspace, size_t workspace_bytes,
                                gbf_stream_t stream) {
  gbf_status_t st =
      check_distill(x, w, ids, logits, index_type, teacher_type, M, V, D, K, alpha, beta);
  if (st != GBF_OK) return st;
  if (M > 0 && (!loss || !lse)) return GBF_ERR_INVALID_ARG;
  if (!aligned(loss, 4) || !aligned(lse, 4) || !aligned(mean, 4) || !aligned(workspace, 16))
    return GBF_ERR_MISALIGNED;
  DistillWs ws;
  const size_t need = distill_sections(workspace, M, V, D, K, false, &ws);
  if (!workspace || workspace_bytes < need) return GBF_ERR_WORKSPACE;
  const DeviceInfo* dev;
  unsigned* err;
  if ((st = lib_device(&dev, &err)) != GBF_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (M == 0) return mean ? cuda_status(cudaMemsetAsync(mean, 0, 4, s)) : GBF_OK;
  CeCall call{x, w, nullptr, index_type == GBF_INDEX_I64, M, V, D, alpha, ws.ce, CePick{}, dev, err, s};
  if ((st = make_lists(ids, logits, teacher_type, beta, K, ws, &call)) != GBF_OK) return st;
  return ce_forward(call, loss, lse, mean);
}

gbf_status_t gbf_linear_distill_grad(const void* x, const void* w, const void* ids, int index_type,
                                     const void* logits, int teacher_type, const float* lse,
                                     const float* dloss, void* dx, void* dw, int64_t M, int64_t V,
                                     int64_t D, int64_t K, float alpha, float beta, float scale,
                                     int reduction, void* workspace, size_t workspace_bytes,
                                     gbf_stream_t stream) {
  gbf_status_t st =
      check_distill(x, w, ids, logits, index_type, teacher_type, M, V, D, K, alpha, beta);
  if (st != GBF_OK) return st;
  if ((M > 0 && (!lse || (!dx && !dw))) ||
      (reduction != GBF_REDUCE_SUM && reduction != GBF_REDUCE_MEAN))
    return GBF_ERR_INVALID_ARG;
  if (!aligned(lse, 4) || !aligned(dloss, 4) || !aligned(dx, 16) || !aligned(dw, 16) ||
      !aligned(workspace, 16))
    return GBF_ERR_MISALIGNED;
  DistillWs ws;
  const size_t need = distill_sections(workspace, M, V, D, K, true, &ws);
  if (!workspace || workspace_bytes < need) return GBF_ERR_WORKSPACE;
  const DeviceInfo* dev;
  unsigned* err;
  if ((st = lib_device(&dev, &err)) != GBF_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (M == 0)
    return dw ? cuda_status(cudaMemsetAsync(dw, 0, static_cast<size_t>(V) * D * 2, s)) : GBF_OK;
  CeCall call{x, w, nullptr, index_type == GBF_INDEX_I64, M, V, D, alpha, ws.ce, CePick{}, dev, err, s};
  if ((st = make_lists(ids, logits, teacher_type, beta, K, ws, &call)) != GBF_OK) return st;
  return ce_backward(call, lse, dloss, dx, dw, scale, reduction);
}

}  // extern "C"
