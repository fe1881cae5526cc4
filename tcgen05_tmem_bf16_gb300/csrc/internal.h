// internal.h -- declarations shared by the library's translation units
// (kernel launchers and the C-ABI layer).  Not installed; not part of the ABI.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace gbf {

// Pointwise ending of a product: act(alpha*acc + beta*C + bias) + residual.
struct EpiParams {
  const __nv_bfloat16* C;         // [M][N] or null
  const __nv_bfloat16* bias;      // [N] or null
  const __nv_bfloat16* residual;  // [M][N] or null (may alias out)
  __nv_bfloat16* out;             // [M][N]
  float alpha;
  float beta;
  int act;
};

// Per-launch control: the device error word, the wait limit and the
// test-only timeout injection.
struct KernelCtl {
  unsigned* err;
  unsigned long long timeout_ns;
  int inject;
  unsigned long long* prof;  // per-CTA wait-time counters (kProfSlots each) or null
};
constexpr int kProfSlots = 32;  // [2*site] cycles waited, [2*site+1] waits; [31] CTA cycles

// Kernel families (gbf_kernel_path codes).
enum Path {
  kPathNone = 0,
  kPathPersistent = 1,
  kPathSwap = 2,
  kPathW4 = 3,
  kPathPair = 4,
  kPathPersistentSplit = 5,  // the one-SM persistent kernel, K split over a CTA pair per tile
  kPathPairOne = 6,          // the CTA-pair kernel with one MMA stream (units of one M-tile)
  kPathPairSplit = 7,        // the one-stream CTA-pair kernel, K split over two pairs per tile
};

struct GemmPlan {
  int path = kPathNone;
  int mpad = 0;      // swapped kernels: MMA N (padded rows of A per tile)
  int splits = 1;    // swapped kernels: cluster split-K size
  int m_tiles = 0;
  int n_tiles = 0;
  int num_kb = 0;    // 64-wide K blocks
  int grid = 0;      // persistent kernels: CTAs
  int bn = 256;      // pair kernel: tile width (MMA N)
  int streams = 2;   // pair kernel: M-tiles (MMA streams) per unit of work
  bool kpar = false; // one-stream pair kernel: two MMA streams over alternate K blocks
};

struct DeviceInfo {
  int sms = 0;
  int pairs = 0;  // CTA pairs (clusters of two 1-SM CTAs) that fit at once
  int quads = 0;  // clusters of four 1-SM CTAs (two pairs) that fit at once
  int cc_major = 0;
  int cc_minor = 0;
};

// ---- argument checks (api.cu) -------------------------------------------------
// The status gemm_epilogue / gemm_epilogue_unfused return for these arguments
// before any workspace or device check (a GBF_* code; 0 = acceptable).
int check_gemm_call(const void* A, const void* B, int b_layout, const void* C, const void* bias,
                    const void* residual, const void* out, int64_t M, int64_t N, int64_t K,
                    int act);

// ---- planning (api.cu) -------------------------------------------------------
GemmPlan plan_gemm(int64_t M, int64_t N, int64_t K, bool dual, bool kn, const DeviceInfo& dev);
GemmPlan plan_w4a16(int64_t M, int64_t N, int64_t K, const DeviceInfo& dev);

// ---- launchers ---------------------------------------------------------------
// Dense bf16 GEMM with fused ending (gemm_tc.cu).  tmA: activations [M][K];
// tmW / tmW2: weights (tmW2 = up weights of the dual GEMM); tmO: the output
// [M][N] in boxes of 32 x 32 with the 64-byte swizzle (used by the
// persistent kernel's TMA stores; the swapped kernel writes directly).
cudaError_t launch_gemm(const GemmPlan& plan, bool w_kn, bool dual, const CUtensorMap& tmA,
                        const CUtensorMap& tmW, const CUtensorMap& tmW2, const CUtensorMap& tmO,
                        const EpiParams& ep, int M, int N, int K, const KernelCtl& ctl,
                        cudaStream_t stream);

// The same on CTA pairs with tcgen05.mma.cta_group::2 (gemm_pair.cu).  tmO:
// the output [M][N] bf16 in boxes of 32 x 32 with the 64-byte swizzle (the
// epilogue writes it with TMA stores).
cudaError_t launch_gemm_pair(const GemmPlan& plan, bool w_kn, bool dual, const CUtensorMap& tmA,
                             const CUtensorMap& tmW, const CUtensorMap& tmW2,
                             const CUtensorMap& tmO, const EpiParams& ep, int M, int N, int K,
                             const KernelCtl& ctl, cudaStream_t stream);
int max_active_pairs();
int max_active_quads();

// Weight-only quantised GEMM (wq_gemm.cu).  tmA: activations; tmQ: the
// weight codes (int4, nvfp4: [K][N/2] bytes; fp8: [K][N]); tmS: scales
// (int4, fp8: bf16 [K/G][N]; nvfp4: E4M3 bytes [K/16][N]).
enum WqFmt { kWqInt4 = 0, kWqFp8 = 1, kWqNvfp4 = 2 };
cudaError_t launch_wq_gemm(int fmt, const GemmPlan& plan, const CUtensorMap& tmA,
                           const CUtensorMap& tmQ, const CUtensorMap& tmS, const EpiParams& ep,
                           int M, int N, int K, int group, const KernelCtl& ctl,
                           cudaStream_t stream);

// Pointwise kernels of the unfused compositions (pointwise.cu).  D == null
// means a zero product (used for K == 0).
cudaError_t launch_pointwise_epilogue(const __nv_bfloat16* D, const EpiParams& ep, int64_t M,
                                      int64_t N, int sms, cudaStream_t stream);
cudaError_t launch_swiglu_pointwise(const __nv_bfloat16* g, const __nv_bfloat16* u,
                                    const EpiParams& ep, int64_t M, int64_t N, int sms,
                                    cudaStream_t stream);
cudaError_t launch_dequant_int4(const uint8_t* Wq, const __nv_bfloat16* scales, int group,
                                int64_t K, int64_t N, __nv_bfloat16* w, int sms,
                                cudaStream_t stream);
// FP8 (bf16 group scales) and NVFP4 (E4M3 block scales) weights -> bf16 [K][N].
cudaError_t launch_dequant_fp8(const uint8_t* Wq, const __nv_bfloat16* scales, int group,
                               int64_t K, int64_t N, __nv_bfloat16* w, int sms,
                               cudaStream_t stream);
cudaError_t launch_dequant_nvfp4(const uint8_t* Wq, const uint8_t* scales, int64_t K, int64_t N,
                                 __nv_bfloat16* w, int sms, cudaStream_t stream);

// Fused residual add + RMSNorm (rmsnorm.cu).  x == null: no add (plain
// RMSNorm of a); resid == null: the residual is not written.  N <= 16384.
cudaError_t launch_add_rmsnorm(const __nv_bfloat16* a, const __nv_bfloat16* x,
                               const __nv_bfloat16* w, __nv_bfloat16* norm,
                               __nv_bfloat16* resid, int64_t M, int N, float eps, int sms,
                               cudaStream_t stream);
constexpr int kRmsMaxN = 16384;

// Embedding lookup and its gradient (embedding.cu).  ids: int64 or int32;
// one outside [0, V) reads zeros and gets no gradient.
cudaError_t launch_embedding_lookup(const void* ids, bool ids64, const __nv_bfloat16* table,
                                    __nv_bfloat16* out, int64_t M, int64_t V, int D, float scale,
                                    cudaStream_t stream);
struct EmbedGradWs {
  int *key0, *idx0, *key1, *idx1;  // [M] each: the sorted list, twice
  float *head, *tail;              // [pieces][D]: parts of runs over several pieces
};
int embed_piece(int64_t M, int D);  // sorted positions per piece
cudaError_t launch_embedding_grad(const void* ids, bool ids64, const __nv_bfloat16* dout,
                                  __nv_bfloat16* dtable, int M, int V, int D, float scale,
                                  bool accumulate, const EmbedGradWs& ws, int sms,
                                  cudaStream_t stream);

// Global norm and clipping (clip.cu).  out == null: in place.  partial: three
// float2 for each of clip_ctas() CTAs of each of clip_launches() launches.
int clip_ctas(int sms);
int clip_launches(int n);
cudaError_t launch_clip_grad_norm(const void* const* in, void* const* out, const int64_t* counts,
                                  const int* types, int n, float max_norm, float eps, float* norm,
                                  float2* partial, int sms, cudaStream_t stream);

// Linear cross entropy (linear_ce.cu).  One product of the kernel with its
// ending; the scored rows are numbered 0 .. count-1 in their order.
enum CeMode { kCeNone = 0, kCeLse = 1, kCeGrad = 2, kCeDx = 3, kCeDw = 4 };
struct CeJob {
  // a[1] / b[1]: x itself, where it is an operand, for when every row is
  // scored; [0] the gathered rows (or the operand's only map)
  CUtensorMap a[2], b[2], o;
  int mode;
  int bn;      // columns of a tile: 256, or for kLse 224
  int cols;    // columns of the vocabulary: all (kCeLse) or the piece's
  int v0;      // first column of the piece
  int splits;  // parts of K (kCeDx), each with its own fp32 buffer
  int add;     // kCeDx: add to the buffer (a later piece)
  int gt;      // kCeDx, kCeDw: G is stored transposed, [cols][rows]
};
// The products of one launch, none of which reads what another writes.  Job 0:
// the one with the longest units, if any.
constexpr int kCeJobs = 3;
struct CeLaunch {
  CeJob job[kCeJobs];
  int d;  // hidden width
};
struct CeEnd {
  const int* count;   // scored rows
  const int* tgt;     // [count] targets
  const float* lse2;  // [count] lse / ln 2
  const float* dl;    // [count] gradient of each loss
  float2* part;       // [2 per column tile][M] (maximum, sum), powers of two
  float* tlog;        // [count] the targets' products
  float c2;           // alpha / ln 2
  float* chain;       // ce_swap.cu: sums over the segments before the last
  float scale;        // of dw
  int mean;           // divide by the number of scored rows
  int M;
  int m_pad;          // rows between the splits' fp32 buffers
};
#ifdef __CUDACC__
// Target i of an array of int64 or int32.
__device__ __forceinline__ int64_t ce_target(const void* targets, int ids64, int64_t i) {
  return ids64 ? static_cast<const int64_t*>(targets)[i]
               : static_cast<int64_t>(static_cast<const int*>(targets)[i]);
}
#endif
// The logits for up to kCeSwapMax rows, with swapped roles (ce_swap.cu).
constexpr int kCeSwapMax = 128;
// K blocks whose products the tensor cores add up in one chain for a logit.  Each
// addition cuts 2^-25 off the running sum on average, so that a sum of 16 K blocks
// of 64 is low by 1e-6 of itself (measured: 9.8e-10 per product for random signs,
// up to 3.9e-9 for one sign).
constexpr int kCeChain = 16;
int ce_swap_segments(int64_t M, int k_blocks);  // parts of K between which the ending adds
int ce_swap_rows(int64_t M);  // rows padded to: 16, 64, 128; 0 above kCeSwapMax
struct CeSwap {
  CUtensorMap w, x[2];  // x[1]: x itself, for when every row is scored (and forward)
  __nv_bfloat16* gt;    // gradient: [cols][padded rows]
  // forward: all rows as they are, scored or not (they fill the padding anyway)
  const void* targets;
  int ids64;
  unsigned* ticket;     // zeroed for the join
  int cols, v0, num_kb;
};
cudaError_t launch_ce_swap(const CeSwap& a, bool grad, const CeEnd& end, int sms,
                           const KernelCtl& ctl, cudaStream_t stream);
struct CePrep {
  const __nv_bfloat16* x;
  __nv_bfloat16* xc;      // gathered rows
  const float* lse_in;    // gradient: the forward's lse
  const float* dloss;     // gradient, may be null (1)
  float *loss, *lse_out;  // forward
  __nv_bfloat16* dx;      // gradient: zero rows where not scored
  int *count, *rows, *tgt;
  unsigned* ticket;
  float *lse2, *dl;
  int M, V, D, rows_per;
};
struct CeJoin {
  const int* count;
  const int* rows;      // null: the rows as they are, scored by these targets
  const void* targets;
  int ids64, V;
  const float2* part;
  const float* tlog;
  unsigned* ticket;
  double* sums;  // per 8 rows
  float *loss, *lse, *mean;
  float c2;      // as in CeEnd: what the maxima were made with
  int M, parts;
};
struct CeDxOut {
  const int* count;
  const int* rows;
  const float* acc;
  __nv_bfloat16* dx;
  float scale;
  int mean, m_pad, splits, D;
};
// chains: one product, the logits, in units of one row tile (streams 1).
cudaError_t launch_ce_gemm(const CeLaunch& launch, const CeEnd& end, int streams, bool chains,
                           int grid, const KernelCtl& ctl, cudaStream_t stream);
cudaError_t launch_ce_prep(const void* targets, bool ids64, CePrep p, int sms,
                           cudaStream_t stream);
cudaError_t launch_ce_join(const CeJoin& p, cudaStream_t stream);
cudaError_t launch_ce_dx(const CeDxOut& p, int M, int sms, cudaStream_t stream);

// ---- shared with the other entry-point files (api.cu) ---------------------------
// The current device and the address of its error word (a GBF_* status).
int lib_device(const DeviceInfo** info, unsigned** err);
// Row-major 2-D tensor map; false if the driver refuses it.
bool lib_tmap_2d(CUtensorMap* m, const void* base, CUtensorMapDataType dt, uint64_t inner,
                 uint64_t outer, uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer,
                 CUtensorMapSwizzle swz);
// Launch control of a grid of `ctas`.
KernelCtl lib_ctl(unsigned* err, int64_t ctas);
// gbf_workspace_size() of the operators in heads.cu.
size_t heads_workspace_size(int op, int64_t M, int64_t N, int64_t K);

// Tile geometry shared by the planner and the kernels.
constexpr int kBM = 128;        // MMA M: rows of TMEM / output tile height
constexpr int kBK = 64;         // K per pipeline stage (one 128-byte swizzle row of bf16)
constexpr int kPersistBN = 256; // persistent kernel: MMA N
constexpr int kSwapBN = 128;    // swapped kernel: output columns per tile (= MMA M)
constexpr int kSwapDualMaxM = 32;  // gate/up GEMM on the swapped kernel up to this M
constexpr int kW4BN = 512;      // W4A16 kernel: output columns per tile
constexpr int kMaxSplits = 8;   // portable cluster size limit

}  // namespace gbf
