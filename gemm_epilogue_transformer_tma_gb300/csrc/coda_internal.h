// Host-side plumbing shared by the translation units of libcoda: tensor-map
// construction, the launch context, and the internal launchers each .cu file
// provides.  Not part of the public ABI (that is include/coda.h).
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace coda {

struct LaunchCtx {
  int num_sms;
  int* status;          // device status word
  uint64_t timeout_ns;  // bound on every in-kernel wait
  cudaStream_t stream;
  int skip_first_stage;  // test hook, see coda_debug_skip_first_stage
  int pair;              // 1: 2-SM GEMM kernel (CTA pairs), 0: 1-SM kernel
  const float* scale_a;  // FP8 operands: device pointers to the per-tensor scales
  const float* scale_b;
  uint32_t f8_fmt;       // FP8 operands: format bits of A and B (f8_format_bits; 0 = both e4m3)
  float scale_host;      // FP8 operands: a further accumulator scale known on the host (1 otherwise)
  float* sk_parts;       // split-tile scratch (coda_set_split_workspace), or null: no tile is split
  int* sk_flags;
  int sk_slots;          // clusters the scratch has slots for
  int wide_lead;         // > 0: long-K launches take 256 x 512 pair tiles with this lead J (coda_set_wide_tiles)
};

// Whether a bf16 GEMM over K with tiles_n 256-column output tiles takes the
// wide-tile pair kernel: the handle asks for it (a lead J > 0), the pair
// kernel is on, the column tiles pair up, and K is long: at least
// kWideMinKb k-blocks of 64 (K >= 16384), and enough that the 2J single-half
// k-blocks of a tile are at most a quarter of its 2 nkb half k-blocks.  Only
// the long-K backward programs are compiled for it.  Each tile boundary
// exposes part of an accumulator half's drain, so short-K GEMMs, with many
// tiles per SM pair, lose more there than the smaller operand traffic gains:
// measured, the 7B / 70B weight gradient (K = 8192 / 4096) ran 1-9 % slower
// on wide tiles and the data gradient (K = 28672 / 57344) 3 % faster.
constexpr int kWideMinKb = 256;
bool wide_tiles_fit(const LaunchCtx& c, int K, int tiles_n);

// 2-D bf16 tensor map with 128-byte swizzle.  The tensor is `outer` rows of
// `inner` contiguous elements with a row pitch of `ld` elements; the box is
// box_inner x box_outer elements (box_inner * 2 bytes must be <= 128).
// Returns false if the driver rejects it.
bool make_tmap_bf16(CUtensorMap* m, const void* base, uint64_t inner, uint64_t outer, uint64_t ld,
                    uint32_t box_inner, uint32_t box_outer);
// Tensor maps for the epilogue's TMA stores: `rows` x `cols` elements with a
// row pitch of `ld` elements, 32 x 32 boxes (bf16: 64-byte swizzle; fp32:
// 128-byte swizzle), matching the staging layout of the GEMM epilogue.
bool make_tmap_store_bf16(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint64_t ld);
bool make_tmap_store_f32(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint64_t ld);
// 1-byte codes (32 x 32 boxes, 32-byte swizzle), matching stage_e5m2x32
bool make_tmap_store_u8_sw32(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint64_t ld);
// The same for 1-byte elements (e4m3 codes): box_inner <= 128.
bool make_tmap_u8(CUtensorMap* m, const void* base, uint64_t inner, uint64_t outer, uint64_t ld, uint32_t box_inner,
                  uint32_t box_outer);

// Packed block scales as `chunks` rows of 512 bytes, loaded one at a time.
bool make_tmap_scale_chunks(CUtensorMap* m, const void* base, uint64_t chunks);

// Launch `kern` on c.stream with programmatic stream serialization: its
// prologue may overlap the tail of the previous kernel in the stream.  Every
// library kernel calls griddep_wait() before its first global-memory access,
// so the ordering of memory effects is that of a plain stream launch.
template <typename... KArgs, typename... Args>
cudaError_t launch_chained(const LaunchCtx& c, void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem,
                           Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = c.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

// Dynamic shared memory above 48 KB is granted per kernel and device; asking
// again on every call costs more than a launch.
template <class Kern>
inline cudaError_t allow_smem(Kern kern, int bytes, bool (&done)[64]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev < 0 || dev >= 64) return e != cudaSuccess ? e : cudaErrorInvalidDevice;
  if (done[dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  done[dev] = e == cudaSuccess;
  return e;
}

// Handle accessors (api.cu), for translation units that only see the
// opaque coda_handle_t.
LaunchCtx launch_ctx_of_handle(void* handle, void* stream);
int device_of_handle(void* handle);
// Partial-accumulator slots the split-tile scratch needs on a GPU with
// num_sms SMs (gemm_fwd.cu, beside the split plan it serves).
int split_scratch_slots(int num_sms);
// The handle's slot for the device address of the allocation-free call's
// scratch array (noalloc.cu); null until that call first runs on the handle.
void** noalloc_scratch_slot(void* handle);

// ---- GEMM launchers (gemm_*.cu) --------------------------------------------
// Operand majors: A K-major = [M][K], MN-major = [K][M]; B K-major = [N][K],
// MN-major = [K][N].  All row pitches equal the extents (dense tensors).

// C = bf16(row_scale[m] * col_scale[n] * sum_k A B); scales may be null.
cudaError_t gemm_store(const LaunchCtx& c, const __nv_bfloat16* A, bool a_mn, const __nv_bfloat16* B, bool b_mn,
                       __nv_bfloat16* C, int M, int N, int K, const float* row_scale,
                       const __nv_bfloat16* col_scale);

// C = bf16(row_scale[m] (A B)[m][n] + add[m][n]), A [M][K], B [K][N]
cudaError_t gemm_scale_add(const LaunchCtx& c, const __nv_bfloat16* A, const __nv_bfloat16* B, const float* row_scale,
                           const __nv_bfloat16* add, __nv_bfloat16* C, int M, int N, int K);

// C (fp32) = A B  or  C += A B.
cudaError_t gemm_store_f32(const LaunchCtx& c, const __nv_bfloat16* A, bool a_mn, const __nv_bfloat16* B, bool b_mn,
                           float* C, int M, int N, int K, bool accumulate);

// h = bf16(X W1 + R); psum[m, j] = sum of h^2 over column block j; with
// Hg != null also Hg = bf16(h * g).
cudaError_t gemm_res_prms(const LaunchCtx& c, const __nv_bfloat16* X, const __nv_bfloat16* W1t,
                          const __nv_bfloat16* R, __nv_bfloat16* H, float* psum, int M, int K1, int d, int T,
                          const __nv_bfloat16* g = nullptr, __nv_bfloat16* Hg = nullptr);

// z = rstd * (H W2g); out = silu(z_gate) * z_up (swiglu) or z (plain).
// With psum != null the row scale comes from the partial sums of squares
// (1 / sqrt(sum_j psum / d + eps)) instead of rstd, and is also written to
// rstd_out when that is not null.
cudaError_t gemm_rowscale_swiglu(const LaunchCtx& c, const __nv_bfloat16* H, const __nv_bfloat16* W2gt,
                                 const float* rstd, __nv_bfloat16* out, __nv_bfloat16* zsave, int M, int d, int N2,
                                 bool swiglu, const float* psum = nullptr, int T = 0, float eps = 0.f,
                                 float* rstd_out = nullptr);

// acc = dP W2^T; dH = g*acc - c*h; dgpart[4*tm+q, n] = sum_rows acc*h.
// With cpart != null, c comes from the SwiGLU-backward epilogue's partial
// sums: c[m] = rstd[m]^2 / d * sum_j cpart[m, j] (Tc columns); cvec unused.
cudaError_t gemm_dgrad_rms(const LaunchCtx& c, const __nv_bfloat16* dP, const __nv_bfloat16* W2t,
                           const __nv_bfloat16* H, const __nv_bfloat16* g, const float* cvec, __nv_bfloat16* dH,
                           float* dgpart, int M, int N2, int d, const float* cpart = nullptr, int Tc = 0,
                           const float* rstd = nullptr);

// dY = dYb W3 computed on chip, then the SwiGLU backward in the epilogue:
// dP = bf16(rstd dZ), cpart[m, j] = sum over 256-column tile j of dZ z.
cudaError_t gemm_dgrad_swiglu_bwd(const LaunchCtx& c, const __nv_bfloat16* dYb, const __nv_bfloat16* W3t,
                                  const __nv_bfloat16* z, const float* rstd, __nv_bfloat16* dP, float* cpart, int M,
                                  int d, int F, int T);

// per (row, vocab tile) max / sum-exp / argmax, label logit.
cudaError_t gemm_ce_stats(const LaunchCtx& c, const __nv_bfloat16* H, const __nv_bfloat16* Wt, const int32_t* labels,
                          float* pmax, float* psum, int32_t* parg, float* zy, int M, int d, int V, int T);

// per (row, 128-column block) max / sum-exp of c.scale_host H Wt^T, and the
// label's logit where the label lies in [0, V); the contraction summed in
// pieces (gemm_logits.cuh).  kept: exp(logit - its block's max) in bf16 of the
// first kept_cols columns (whole chunks, V or 0), vocabulary chunk c of `chunk`
// columns [M][its columns] from kept + c * chunk * (M rounded up to 32)
cudaError_t gemm_logit_stats(const LaunchCtx& c, const __nv_bfloat16* H, const __nv_bfloat16* Wt,
                             const int32_t* labels, float* pmax, float* psum, float* zy, __nv_bfloat16* kept, int chunk,
                             int kept_cols, int M, int d, int V, int T);

// Scoring (logits_score.cuh): blocks of a row and what is kept of each.
struct ScoreStats {
  float* pmax;    // [M][T]: the block's largest logit
  float* psum;    // [M][T]: sum of exp((L - pmax) / temperature), less 1
  float* pdot;    // [M][T]: sum of (L - pmax) exp((L - pmax) / temperature)
  float* zy;      // [M]: the logit of the row's token
  float* logits;  // [M][V], or null: no alternatives
  float* sub;     // [M][4 T]: maxima of sub_cols columns each, with logits
  float* bound;   // [M], or null: below it a row's logits from score_first_columns on need not be there
  int k;          // alternatives
  int T;          // blocks of a row
  int sub_cols;   // a quarter of a block
};
// Up to kScoreFew rows take the kernel of gemm_score_few.cuh, whose blocks have
// score_few_rows(V) columns: 128 or less, a multiple of 4, such that the blocks
// fill the SMs of a GB300 evenly (a constant: a workspace is sized without a
// device).  Others have blocks of 128.  At d = 4096, V = 128256 with 8
// alternatives: 64 rows 208 us, 128 (of a kernel for so many) 293; 129 by the
// other kernel 210.
constexpr int64_t kScoreFew = 64, kScoreSms = 152;
int score_few_rows(int64_t V);
cudaError_t gemm_score(const LaunchCtx& c, const __nv_bfloat16* H, const __nv_bfloat16* Wt, const int32_t* labels,
                       const ScoreStats& s, float log2e_over_t, int M, int d, int V);
// Columns whose logits are all kept, a multiple of 256, or V; a bound on each row's
// k-th largest from their sub-blocks' maxima is in s.bound for the others.
int score_first_columns(int64_t M, int64_t V, int64_t k);
cudaError_t launch_score_bound(const LaunchCtx& c, const ScoreStats& s, int64_t M, int64_t first);
// logp, entropy, the k highest logits' tokens and log-probabilities of M rows
// (score.cu); any of the outputs may be null, top_ids and top_logp together
constexpr int kScoreMaxTop = 256;
struct ScoreOut {
  const int32_t* labels;  // or null, with logp
  float* logp;
  float* entropy;
  int32_t* top_ids;       // [M][k]
  float* top_logp;
  int k;
  float temperature, log2e_over_t;
  int* status;
};
cudaError_t launch_score_rows(const LaunchCtx& c, const ScoreStats& s, const ScoreOut& o, int64_t M, int64_t V);

// Distillation from a teacher's list (distill.cu, logits_distill.cuh).
constexpr int kDistillMaxList = 256;
// So few rows take part in dW's contraction twice, the second time with what the
// rounding of factor H to bf16 takes from their listed entries: the error of dW,
// 1.4 times that of rounding it alone on average, spreads to 1.7 where few rows make
// it.  8 tokens, d = 2048, V = 50280: 140 us, 139 without; 64, d = 1024, V = 32000: 67
// and 64; 128 of d = 4096, V = 128256: 615 and 557, which is not done.
constexpr int64_t kDistillTwice = 64;
constexpr uint32_t kNoEntry = 0xFFFFFFFFu;
struct DistillIn {
  const int32_t* ids;   // [M][k], an entry outside [0, V) is not used
  const float* val;     // [M][k]
  const float* weight;  // [M], or null: uniform
  float uniform;
  int mode;             // CODA_DISTILL_*
  float temperature, log2e_over_t, log2e_over_t_low;  // the quotient in two parts
  int* status;
};
struct DistillWork {
  int k, T;             // entries of a list, 128-column blocks of the vocabulary
  int32_t* ids;         // [M][k]: the list's tokens, each once, -1 for other entries
  float2* t;            // [M][k]: those entries' targets, in two parts
  uint32_t* at;         // [G][T], G = ceil(M / 32): where the entries of 32 rows in a block begin | how many << 16
  uint32_t* entry;      // [G][32 k]: row of the 32 | column of the block << 5 | position in the row's list << 12, or
                        // kNoEntry for a token that an earlier entry of its row has
  float4* mass;         // [M]: P, r, P + r - 1, what P's fp32 leaves of it
  float* n;             // [M]: the exponent of the row's kept values, NaN: no weight
  float* listed;        // [M][k]: the student's logits of the entries
  float* pn;            // [M][T], logits_distill.cuh
  float* psum;          // [M][T]
  float4* terms;        // [M]: shares of the statistics
  int* done;            // rows finished
  // with gradients, dH = factor kept Wt + add, dW = kept^T scaled: [M][V], [M], [M][d]
  // and [M][d].  Up to kDistillTwice rows as many more behind kept and scaled: the
  // listed entries of kept alone, and what bf16 takes from scaled
  __nv_bfloat16* kept;
  float* factor;
  __nv_bfloat16* add;
  __nv_bfloat16* scaled;
  float2* carry;          // [M][k], or null.  Else add is left to gemm_splitk, by this list
  int* carry_n;           // [M]
};
struct DistillOut {
  float* stats;     // or null: the shares stay in DistillWork::terms
  float* row_loss;  // or null
};
cudaError_t launch_distill_list(const LaunchCtx& c, const DistillIn& in, const DistillWork& w, const __nv_bfloat16* H,
                                const __nv_bfloat16* Wt, int64_t M, int64_t d, int64_t V);
cudaError_t gemm_distill(const LaunchCtx& c, const __nv_bfloat16* H, const __nv_bfloat16* Wt, const DistillWork& w,
                         float log2e_over_t, int M, int d, int V);
cudaError_t launch_distill_rows(const LaunchCtx& c, const DistillIn& in, const DistillWork& w, const DistillOut& o,
                                const __nv_bfloat16* H, const __nv_bfloat16* Wt, int64_t M, int64_t d, int64_t V);
// dH = diag(factor) E Wt + add of the first M rows of E and dW = E^T scaled of all
// (E [rows][V], scaled [rows][d]), one grouped launch
cudaError_t gemm_group_scaled_bwd(const LaunchCtx& c, const __nv_bfloat16* E, const float* factor,
                                  const __nv_bfloat16* Wt, const __nv_bfloat16* add, const __nv_bfloat16* scaled,
                                  __nv_bfloat16* dH, __nv_bfloat16* dW, int M, int rows, int d, int V);

// out[m] = bf16(sum of factor times row of Wt over list[m][0 .. n[m])), rows of 8 d8
struct RowSums {
  const float2* list;  // [M][k]: a factor and, as its bits, a row
  const int* n;        // [M]
  int k;
  const uint4* Wt;
  int64_t n8, d8;      // n8 = M d8
  uint4* out;
};
// parts_buf [parts][M rounded up to 256][N] fp32 (+)= the K ranges of A B, A
// [M][K], B [K][N] (gemm_splitk.cuh); parts <= the k-blocks of 64 in K; beside them
// the sums, if there are any
cudaError_t gemm_splitk(const LaunchCtx& c, const __nv_bfloat16* A, const __nv_bfloat16* B, float* parts_buf, int parts,
                        bool accumulate, int M, int N, int K, const RowSums& sums = RowSums{});

// dL chunk = (softmax - onehot) / M for vocabulary rows [v0, v0 + Vc).
cudaError_t gemm_ce_grad(const LaunchCtx& c, const __nv_bfloat16* H, const __nv_bfloat16* Wt_chunk,
                         const int32_t* labels, const float* lse, __nv_bfloat16* dL, int M, int d, int Vc, int v0,
                         float inv_M);
// The same as row_scale[m] (softmax - onehot) of the logits c.scale_host H Wt^T;
// lost[m] = what the bf16 rounding takes from the entry of a label in the chunk.
cudaError_t gemm_policy_grad(const LaunchCtx& c, const __nv_bfloat16* H, const __nv_bfloat16* Wt_chunk,
                             const int32_t* labels, const float* lse, __nv_bfloat16* dL, int M, int d, int Vc, int v0,
                             const float* row_scale, float* lost);

// qkv = X Wqkv with RoPE (head_dim 128) on the first rot_cols columns.
cudaError_t gemm_qkv_rope(const LaunchCtx& c, const __nv_bfloat16* X, const __nv_bfloat16* Wqkv_t,
                          const float* cos_t, const float* sin_t, __nv_bfloat16* qkv, int M, int d, int N,
                          int rot_cols, int S);

// FP8 (e4m3, per-tensor scales sa / sb) forms of the forward GEMMs; operands
// K-major: A [M][K] codes, B [N][K] codes.
cudaError_t gemm_res_prms_fp8(const LaunchCtx& c, const uint8_t* Xq, const float* sX, const uint8_t* W1q,
                              const float* sW1, const __nv_bfloat16* R, __nv_bfloat16* H, float* psum, int M, int K1,
                              int d, int T);
cudaError_t gemm_rowscale_swiglu_fp8(const LaunchCtx& c, const uint8_t* Hq, const float* sH, const uint8_t* W2q,
                                     const float* sW2, const float* rstd, __nv_bfloat16* out, __nv_bfloat16* zsave,
                                     int M, int d, int N2, bool swiglu);

// Independent GEMM pairs in one launch (SM-pair kernel; two launches of the
// 1-SM kernel when pairing is off):
//   dX = dH W1t (W1t [d][K1]) and dW1t = dH^T X (any such pair: A [M][d]
//   K-major with B [d][K1], and A^T with X [M][K1]);
cudaError_t gemm_group_store(const LaunchCtx& c, const __nv_bfloat16* dH, const __nv_bfloat16* W1t,
                             const __nv_bfloat16* X, __nv_bfloat16* dX, __nv_bfloat16* dW1t, int M, int K1, int d);
//   LM-head chunk: dH32 (+)= dL Wc (Wc [Vc][d]) in fp32 and dWc = dL^T H.
cudaError_t gemm_group_ce_bwd(const LaunchCtx& c, const __nv_bfloat16* dL, const __nv_bfloat16* Wc,
                              const __nv_bfloat16* H, float* dH32, bool accumulate, __nv_bfloat16* dWc, int M, int d,
                              int Vc);
//   the same with rows[slot[v]] (fp32, d wide) added to row v of dWc before
//   it is rounded, where slot[v] != kNoSlot; and the dW GEMM of it alone
cudaError_t gemm_group_policy_bwd(const LaunchCtx& c, const __nv_bfloat16* dL, const __nv_bfloat16* Wc,
                                  const __nv_bfloat16* H, float* dH32, bool accumulate, __nv_bfloat16* dWc,
                                  const uint32_t* slot, const float* rows, int M, int d, int Vc);
//   (slot null: dWc = dL^T H).  It can take on the end of a split data gradient:
struct SplitDh {
  const float4* parts;  // [num][stride4], of which n4 are used
  int num;
  int64_t stride4, n4, d4;
  const float* factor;  // [n4 / d4]
  const uint2* add;     // bf16
  uint2* out;           // bf16
  const float4* terms;  // [n4 / d4], or null: their sum to stats
  float* stats;
};
cudaError_t gemm_store_plus_rows(const LaunchCtx& c, const __nv_bfloat16* dL, const __nv_bfloat16* H,
                                 __nv_bfloat16* dWc, const uint32_t* slot, const float* rows, int M, int d, int Vc,
                                 const SplitDh& dh = SplitDh{});
//   the same first-layer pair on 8-bit codes: dX = sdH sW1 dHq W1q and
//   dW1t = sdH sX dHq^T Xq (dH format dh_fmt; W1 and X in w_fmt); two
//   launches when pairing is off.
cudaError_t gemm_group_store_fp8(const LaunchCtx& c, const uint8_t* dHq, int dh_fmt, const float* sdH,
                                 const uint8_t* W1q, const float* sW1, const uint8_t* Xq, const float* sX, int w_fmt,
                                 __nv_bfloat16* dX, __nv_bfloat16* dW1t, int M, int K1, int d);
// Host check of the grouped tile schedule (0 = every tile visited once).
int group_schedule_violations(int P, int heavy, int nH, int nL, int q);
// Tensor map of an 8-bit operand: K-major [rows][K] (boxes of 128 K x
// box_rows) or MN-major [K][mn] (boxes of 128 x 128).
bool make_f8_operand_map(CUtensorMap* m, const uint8_t* p, bool mn_major, int mn, int K, int box_rows);

// C = bf16(row_scale * col_scale * sA * sB * A B) on 8-bit operands: A
// [M][K] (K-major) or [K][M] (MN-major), B [N][K] or [K][N]; formats 0 =
// e4m3, 1 = e5m2; sA / sB device pointers to the scales (null = 1).
cudaError_t gemm_store_fp8(const LaunchCtx& c, const uint8_t* A, bool a_mn, int a_fmt, const float* sA,
                           const uint8_t* B, bool b_mn, int b_fmt, const float* sB, __nv_bfloat16* C, int M, int N,
                           int K, const float* row_scale, const __nv_bfloat16* col_scale);

// dgrad2 with the RMSNorm-backward epilogue (as gemm_dgrad_rms) on 8-bit
// operands: dP codes [M][N2] (format dp_fmt, scale sdP), W2t codes [N2][d]
// (format w_fmt, scale sW2).
cudaError_t gemm_dgrad_rms_fp8(const LaunchCtx& c, const uint8_t* dPq, int dp_fmt, const float* sdP,
                               const uint8_t* W2q, int w_fmt, const float* sW2, const __nv_bfloat16* H,
                               const __nv_bfloat16* g, const float* cvec, __nv_bfloat16* dH, float* dgpart, int M,
                               int N2, int d);

// LM-head GEMMs on 8-bit operands: the statistics GEMM on e4m3 H and W
// codes; the chunk's recomputed logits writing dL as e5m2 codes of
// dL * code_inv; the chunk's dH (+)= and dW GEMMs on those codes (scale s_dL)
cudaError_t gemm_ce_stats_fp8(const LaunchCtx& c, const uint8_t* Hq, const float* sH, const uint8_t* Wq,
                              const float* sW, const int32_t* labels, float* pmax, float* psum, int32_t* parg,
                              float* zy, int M, int d, int V, int T);
cudaError_t gemm_ce_grad_fp8(const LaunchCtx& c, const uint8_t* Hq, const float* sH, const uint8_t* Wq_chunk,
                             const float* sW, const int32_t* labels, const float* lse, uint8_t* dLq, float code_inv,
                             int M, int d, int Vc, int v0, float inv_M);
cudaError_t gemm_ce_bwd_fp8(const LaunchCtx& c, const uint8_t* dLq, float s_dL, const uint8_t* Wq_chunk,
                            const float* sW, const uint8_t* Hq, const float* sH, float* dH32, bool accumulate,
                            __nv_bfloat16* dWc, int M, int d, int Vc);
// the same two GEMMs in one grouped SM-pair launch (the two launches above
// on single SMs)
cudaError_t gemm_group_ce_bwd_fp8(const LaunchCtx& c, const uint8_t* dLq, float s_dL, const uint8_t* Wq_chunk,
                                  const float* sW, const uint8_t* Hq, const float* sH, float* dH32, bool accumulate,
                                  __nv_bfloat16* dWc, int M, int d, int Vc);

// C = bf16(A B) on 8-bit operands with packed power-of-two scales for blocks
// of 128 along K (gemm_block.cuh); operands and formats as gemm_store_fp8.
cudaError_t gemm_fp8_block(const LaunchCtx& c, const uint8_t* A, bool a_mn, int a_fmt, const uint8_t* sA,
                           const uint8_t* B, bool b_mn, int b_fmt, const uint8_t* sB, __nv_bfloat16* C, int M, int N,
                           int K);

int ce_tile_cols();    // vocabulary columns per CE statistics tile
int prms_tile_cols();  // columns per partial-RMS tile of GEMM1

// ---- memory-bound kernels (mem_kernels.cu) ---------------------------------
cudaError_t launch_fold(const LaunchCtx& c, const __nv_bfloat16* W2t, const __nv_bfloat16* g, __nv_bfloat16* W2gt,
                        int64_t N2, int64_t d);
cudaError_t launch_rstd_combine(const LaunchCtx& c, const float* psum, int64_t M, int64_t T, int64_t d, float eps,
                                float* rstd);
cudaError_t launch_swiglu_bwd(const LaunchCtx& c, const __nv_bfloat16* dY, const __nv_bfloat16* z,
                              const float* rstd, __nv_bfloat16* dP, float* cvec, int64_t M, int64_t F, int64_t d);
cudaError_t launch_col_combine(const LaunchCtx& c, const float* part, int64_t rows, int64_t d, float* out);
cudaError_t launch_ce_combine(const LaunchCtx& c, const float* pmax, const float* psum, const int32_t* parg,
                              const float* zy, const int32_t* labels, int64_t M, int64_t T, int64_t V, float* lse,
                              int32_t* argmax, float* row_loss);
cudaError_t launch_mean(const LaunchCtx& c, const float* v, int64_t n, float* out);
cudaError_t launch_f32_to_bf16(const LaunchCtx& c, const float* in, __nv_bfloat16* out, int64_t n);
// cos / sin tables [S, head_dim/2] of the rotary embedding, computed in fp64
cudaError_t launch_rope_table(const LaunchCtx& c, float* cos_t, float* sin_t, int64_t S, int64_t head_dim, double base);
// RoPE in place on the first rot_cols columns of qkv [M, N] (standalone, unfused)
cudaError_t launch_rope_apply(const LaunchCtx& c, __nv_bfloat16* qkv, const float* cos_t, const float* sin_t,
                              int64_t M, int64_t N, int64_t rot_cols, int64_t head_dim, int64_t S);
// per-tensor fp8 quantisation: ws[0] = amax of src (times g[col] if g),
// ws[1] = scale = the smallest power of two with amax / scale <= fmax (1 if
// amax == 0); dst = fp8(src * g / scale), e4m3 (fmax 448) or, with
// e5m2 != 0, e5m2 (fmax 57344)
cudaError_t launch_fp8_quantize(const LaunchCtx& c, const __nv_bfloat16* src, int64_t rows, int64_t cols,
                                const __nv_bfloat16* g, float* ws, uint8_t* dst, int e5m2 = 0);
// the SwiGLU backward straight to fp8 codes of bf16(dP) (two passes over dY
// and z; ws as launch_fp8_quantize)
cudaError_t launch_swiglu_bwd_fp8(const LaunchCtx& c, const __nv_bfloat16* dY, const __nv_bfloat16* z,
                                  const float* rstd, float* ws, uint8_t* dPq, float* cvec, int64_t M, int64_t F,
                                  int64_t d, int e5m2);
// the same with delayed scaling: state = {amax, scale}; on entry state[0] is
// the previous dP's amax, on exit {this dP's amax, the scale used} (one pass)
cudaError_t launch_swiglu_bwd_fp8_delayed(const LaunchCtx& c, const __nv_bfloat16* dY, const __nv_bfloat16* z,
                                          const float* rstd, float* state, uint8_t* dPq, float* cvec, int64_t M,
                                          int64_t F, int64_t d, int e5m2);
// block quantisation (fp8_block.cu): codes and packed scales of blocks along
// the rows (q_row, s_row) and / or along the columns (q_col, s_col); with
// tile, 128 x 128 blocks: codes q_row, scales s_row and, transposed, s_col
cudaError_t launch_fp8_block_quantize(const LaunchCtx& c, const __nv_bfloat16* src, bool e5m2, uint8_t* q_row,
                                      uint8_t* s_row, uint8_t* q_col, uint8_t* s_col, bool tile, int64_t rows,
                                      int64_t cols);
cudaError_t launch_fp8_block_dequantize(const LaunchCtx& c, const uint8_t* q, const uint8_t* s, bool e5m2, bool col,
                                        __nv_bfloat16* dst, int64_t rows, int64_t cols);
// norm of the q and k heads, then RoPE (qknorm.cu); x may be out
cudaError_t launch_qknorm_rope(const LaunchCtx& c, const __nv_bfloat16* x, const __nv_bfloat16* gq,
                               const __nv_bfloat16* gk, const float* cos_t, const float* sin_t, const int32_t* pos,
                               __nv_bfloat16* out, int64_t M, int n_q, int n_kv, int D, int64_t S, float eps);
// its backward; part: fp32 [qknorm_max_parts()][2][D]; dx may be dy or x
cudaError_t launch_qknorm_rope_bwd(const LaunchCtx& c, const __nv_bfloat16* dy, const __nv_bfloat16* x,
                                   const __nv_bfloat16* gq, const __nv_bfloat16* gk, const float* cos_t,
                                   const float* sin_t, const int32_t* pos, __nv_bfloat16* dx, float* dgq, float* dgk,
                                   float* part, int64_t M, int n_q, int n_kv, int D, int64_t S, float eps);
int qknorm_max_parts();
// the policy loss's row kernels (policy.cu)
struct PolicyRows {
  const int32_t* labels;
  const float* adv;
  const float* weight;       // or null: uniform
  const float* old;          // or null: the current log-probabilities (ratio 1)
  const float* ref;          // or null: no KL term
  float uniform;             // weight of every row when weight is null
  float lo, hi, beta, inv_temp;
  float* lse;
  float* logp;
  float* row_scale;          // factor of (softmax - onehot), or null
  float* lost;               // set to 0, with row_scale
  uint32_t* slot;            // [2][V], with row_scale: the first of the tokens that carry the label and a
                             // weight, and the complement of the last (so both are minima)
  float4* terms;
  int* status;
};
// dL of a vocabulary chunk in place of its kept exponentials [M][Vc], and
// lost, as gemm_policy_grad; pmax [M][T]
cudaError_t launch_policy_dl(const LaunchCtx& c, __nv_bfloat16* dL, const float* pmax, const int32_t* labels,
                             const float* lse, const float* logp, const float* row_scale, float* lost, int64_t M,
                             int64_t T, int64_t v0, int64_t Vc);
// rows[m] = sum of lost[t] H[t] over the tokens t with m's label, for every m
// that is the first token of a label in [v0, v0 + Vc) (slot[label] == m;
// ~not_last[label] is its last)
cudaError_t launch_label_rows(const LaunchCtx& c, const int32_t* labels, const uint32_t* slot,
                              const uint32_t* not_last, const float* lost, const __nv_bfloat16* H, float* rows,
                              int64_t M, int64_t d, int64_t v0, int64_t Vc);
// dH[m] = bf16(sum_p parts[p][m] + lost[m] Wt[labels[m]]), `stride` values
// between parts
cudaError_t launch_policy_dh(const LaunchCtx& c, const float* parts, int num, int64_t stride, const float* lost,
                             const int32_t* labels, const __nv_bfloat16* Wt, __nv_bfloat16* dH, int64_t M, int64_t d);
cudaError_t launch_policy_rows(const LaunchCtx& c, const float* pmax, const float* psum, const float* zy,
                               const PolicyRows& p, int64_t M, int64_t T, int64_t V, float* stats);
// unfused ablation kernels
cudaError_t launch_add_rmsnorm(const LaunchCtx& c, const __nv_bfloat16* A, const __nv_bfloat16* R,
                               const __nv_bfloat16* g, __nv_bfloat16* H, float* rstd, __nv_bfloat16* Nrm, int64_t M,
                               int64_t d, float eps);
cudaError_t launch_swiglu(const LaunchCtx& c, const __nv_bfloat16* z, __nv_bfloat16* out, int64_t M, int64_t F);
cudaError_t launch_swiglu_bwd_plain(const LaunchCtx& c, const __nv_bfloat16* dY, const __nv_bfloat16* z,
                                    __nv_bfloat16* dZ, int64_t M, int64_t F);
cudaError_t launch_rmsnorm_bwd(const LaunchCtx& c, const __nv_bfloat16* dN, const __nv_bfloat16* H,
                               const float* rstd, const __nv_bfloat16* g, __nv_bfloat16* dH, int64_t M, int64_t d);
cudaError_t launch_rmsnorm_bwd_dg(const LaunchCtx& c, const __nv_bfloat16* dN, const __nv_bfloat16* H,
                                  const float* rstd, float* dgpart, int64_t M, int64_t d, int64_t rows_per_part);

}  // namespace coda
