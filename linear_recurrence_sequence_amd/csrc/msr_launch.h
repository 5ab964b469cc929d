// Host-side launchers of the libmsr kernels (internal; the public ABI is
// include/msr.h).  Every launcher only enqueues on `stream`.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "msr_device.h"

namespace msr {

enum Elt { kF32 = 0, kBF16 = 1 };

// Brackets one kernel launch with HIP events on its stream while tracing is
// enabled (msr_trace_enable); a no-op otherwise.
class TraceScope {
 public:
  TraceScope(const char* name, hipStream_t stream);
  ~TraceScope();
  TraceScope(const TraceScope&) = delete;
  TraceScope& operator=(const TraceScope&) = delete;

 private:
  const char* name_;
  hipStream_t stream_;
  hipEvent_t start_{}, stop_{};
  bool active_ = false;
};

struct ChunkArgs {
  Elt elt;
  int d_k, d_v;
  int batch, seqlen, heads;
  int chunk;                 // tokens per chunk (multiple of 32)
  const void* Q; int64_t ldq;   // token stride in elements
  const void* K; int64_t ldk;
  const void* V; int64_t ldv;
  void* O; int64_t ldo;
  const void* G; int64_t ldg;   // gate (only with fused GroupNorm + gate)
  float scale, eps;
  bool fuse_gn_gate;
  const float* S_in; float* S_out;
  const float* sout_scale;   // host array [heads]: S_out = sout_scale[h] * final state (null: factor 1)
  void* dR;                  // [B, H, NC, d_v, d_k] elt: each chunk's own state contribution
  void* Rx;                  // [B, H, NC, d_v, d_k] elt: R_{i-1} per chunk (aliases dR)
  bool rev_out;              // write output row t of each sequence to row seqlen-1-t
  bool rev_in;               // read Q, K, V row t of each sequence from row seqlen-1-t
  // Rx already holds every chunk's R_{i-1} (state and scan kernels skipped);
  // reuse_seeded: chunk 0's R_{-1} is a seed (else zero)
  bool reuse_rx, reuse_seeded;
  // with reuse_rx, on the direct-copy path only (chunk_out_direct): Rx
  // holds each chunk's R_{i-1} itself, [d_k rows][d_v cols], instead of its
  // transpose
  bool rx_kv;
  // (cos, sin) table [seqlen][d_k / 2] of the positions of the sequence's
  // rows: the output kernel rotates Q with it as it loads Q (only where
  // chunk_out_o16 holds; K must then already be rotated); null: Q as given
  const float2* q_rope_tab;
  // (cos, sin) table of the rows' positions for K (forward passes only):
  // the state kernel rotates the K rows it stages with it and writes them
  // to k_rot (row stride ld_k_rot), which the output kernel then reads in
  // place of K; null: K as given
  const float2* k_rope_tab;
  void* k_rot; int64_t ld_k_rot;
};

// Whether the forward output kernel for these dims and chunk rotates Q
// itself from ChunkArgs::q_rope_tab (all but the bf16 direct-copy kernel
// of d_v <= 256).
bool chunk_out_rotates_q(Elt elt, int d_k, int d_v, int chunk);

// Whether the chunkwise form of these dims and chunk runs the bf16
// direct-copy output kernel (the one that can read Rx as R_{i-1} itself).
bool chunk_out_direct(Elt elt, int d_k, int d_v, int chunk);

// Whether the forward output kernel with 16 query rows per wave runs these
// dims and chunk (bf16, d_k 256, d_v 256 or 512, chunk a multiple of 128).
bool chunk_out_o16(Elt elt, int d_k, int d_v, int chunk);
// That kernel: the chunkwise form's outputs (state: Rx holds R_{i-1}^T per
// chunk) or the parallel form's (one chunk of chunk = TPC * 128 rows); with
// rev_in (and rev_out) set, those of the time-reversed sequence (no fused
// GroupNorm or rotation).
hipError_t launch_out_o16(const ChunkArgs& a, bool state, int chunk, int NC, int TPC, int has_sin,
                          const HeadTab& tab, hipStream_t stream);

// Chunkwise retention: state contributions, fp32 scan, outputs.
hipError_t launch_chunkwise(const ChunkArgs& a, const HeadTab& tab, hipStream_t stream);
// Parallel form: one "chunk" spanning the whole sequence, no state.
hipError_t launch_parallel(const ChunkArgs& a, const HeadTab& tab, hipStream_t stream);

// One decode step: S <- gamma S + k^T v; o = scale q S (q, k rotated at pos).
// Operands of a decode step: one row per batch element (head h at column
// h * d of the row), row strides in elements; o is float32 when o_f32.
struct StepIO {
  const void* q; int64_t ldq;
  const void* k; int64_t ldk;
  const void* v; int64_t ldv;
  void* o; int64_t ldo;
  bool o_f32;
};
hipError_t launch_recurrent_step(Elt elt, int d_k, int d_v, int batch, int heads, const StepIO& io, float* S,
                                 float scale, int64_t pos, float base, const HeadTab& tab, hipStream_t stream);
// z = swish(g) (.) GroupNorm_h(o) per (batch element, head) over d_v; o float32.
hipError_t launch_gn_gate(Elt elt, int d_v, int batch, int heads, const float* o, int64_t ldo, const void* g,
                          int64_t ldg, void* z, int64_t ldz, float eps, hipStream_t stream);

// RG-LRU scan over gates already formed: G = [r | i], [batch*seqlen, 2*width]
// (row stride ldg), X and Y [batch*seqlen, width] (row strides ldx, ldy),
// lam [width] float32, h0 / hT [batch, width] float32 (nullable).  width a
// multiple of 64.
hipError_t launch_rglru_scan(Elt elt, const void* X, int64_t ldx, const void* G, int64_t ldg, const float* lam,
                             float c, const float* h0, float* hT, void* Y, int64_t ldy, int batch, int seqlen,
                             int width, hipStream_t stream);

// In-place transpose of nblocks contiguous d x d blocks of elt (d a multiple
// of 64 for bf16, of 32 for float32).
hipError_t launch_transpose_blocks(Elt elt, void* base, int d, int64_t nblocks, hipStream_t stream);
// The same from src to dst (disjoint, or equal for the in-place transpose).
hipError_t launch_transpose_blocks_to(Elt elt, const void* src, void* dst, int d, int64_t nblocks, hipStream_t stream);
// Per-head factors of launch_state_xform.
struct HeadScale {
  float c[kMaxHeads];
};
// Every chunk's R_{i-1} (Rx, [B, H, NC, d_v, d_k]) and the final state in
// one kernel that walks the chunks of each state tile in order (bf16,
// (d_k, d_v) in {(128, 128), (256, 256), (256, 512)}, chunk a multiple of
// 64, enough (batch, head) pairs bh; K as given; rev_in: the time-reversed
// sequence).
bool chunk_rscan_ok(Elt elt, int dk, int dv, int chunk, int bh);
hipError_t launch_chunk_rscan(const ChunkArgs& a, const HeadTab& tab, const HeadScale& so, hipStream_t st);
// dst[bh] (rows x cols float32) = c[bh % heads] * (transpose ? src[bh]^T :
// src[bh]) for bh < nbh; src == nullptr writes zeros; dst may equal src
// only without transpose.  rows and cols multiples of 32.
hipError_t launch_state_xform(const float* src, float* dst, int nbh, int heads, int rows, int cols, bool transpose,
                              const HeadScale& hs, hipStream_t stream);

// cos/sin table: tab[n * (d/2) + j] = (cos, sin)((pos0 + n) * theta_j),
// theta_j = base^(-2j/d), n = 0..npos-1.
hipError_t launch_rope_table(float2* tab, int npos, int d, int64_t pos0, float base,
                             hipStream_t stream);
// Rotate the first d columns of every head of a [rows, heads * d] block
// (rows = batch * seqlen tokens, token n = row % seqlen) from src to dst
// (dst may equal src).  Strides in elements.
// inverse: rotate by the negative angle (the adjoint, for gradients).
hipError_t launch_rope_apply(Elt elt, const void* src, int64_t lds, void* dst, int64_t ldd,
                             int rows, int seqlen, int heads, int d, const float2* tab,
                             hipStream_t stream, bool inverse = false);

// B operand of launch_gemm: up to four column segments, segment s covering
// output columns [start[s], start[s+1]) (start[0] = 0, unused entries set to
// INT_MAX), each a row-major [K, width] block at ptr[s] with row stride
// ld[s] (elements; multiples of 8).  The first rope_segs segments get the
// rotation epilogue with head dim rope_d and table rope_tab ([seqlen][rope_d/2]
// (cos, sin)); output row m is token m % seqlen.
struct GemmB {
  const void* ptr[4];
  int64_t ld[4];
  int start[4];
  int rope_segs, rope_d, seqlen;
  const float2* rope_tab;
  // split-K: when set, workgroup z of the launch's z dimension sums K rows
  // [z K_s, (z + 1) K_s) and stores float32 partials to part + z M N (no
  // rotation); launch_gemm_splitk adds them up.
  float* part;
  // launch_gemm_parts: the first kextra slices take 64 more K rows; the K
  // rows from tail0 on are those of `tail` (row stride ld[0])
  int kextra, tail0;
  const void* tail;
  // epilogue: C = act(A B + bias) + resid, act = gelu when act == 1 and
  // sigmoid when act == 2 (after any rotation), bias[s] a float32 vector
  // over segment s's columns (nullable), resid an [M, N] matrix with row
  // stride ldr (nullable).  Not with split-K.
  const float* bias[4];
  int act;
  const void* resid;
  int64_t ldr;
};

// C[M, N] = A[M, K] * B[K, N] (row-major A and B segments), fp32
// accumulation, C (row stride ldc) in elt.  K must be a multiple of 64.
hipError_t launch_gemm(Elt elt, const void* A, int64_t lda, const GemmB& b, void* C, int64_t ldc, int M, int N,
                       int K, hipStream_t stream);
// The same product for few rows (M <= 256): the K range split over
// `splits` workgroups per output tile (K a multiple of 64 * splits), float32
// partials in `part` ([splits, M, N]), then summed and rounded once into C.
hipError_t launch_gemm_splitk(Elt elt, const void* A, int64_t lda, const GemmB& b, void* C, int64_t ldc, int M,
                              int N, int K, int splits, float* part, hipStream_t stream);
// How many K splits launch_gemm_splitk should use for an M x N x K product.
int gemm_splits(Elt elt, int M, int N, int K);
// Row-wise LayerNorm over d columns (biased variance, identity affine):
// Y = (X - mean) / sqrt(var + eps); d a multiple of 8, at most 8192.
hipError_t launch_layer_norm(Elt elt, const void* X, int64_t ldx, void* Y, int64_t ldy, int rows, int d, float eps,
                             hipStream_t stream);

// ---- norms between retention cores, with gate and residual (k_norm.hip) ----
// fmt: kQNone (activations in elt) or the 8-bit format of the *_q / *_qs
// pairs (msr_q8.h).  Nullable pointers are named.
struct ResidNormArgs {
  Elt elt;
  int fmt;
  bool layer;                                        // mean subtracted
  int64_t rows;
  int d;                                             // multiple of 64, at most 8192
  float alpha, eps;
  const void* X; const void* B;                      // B null: h = alpha x
  const float* scale; const float* weight; const float* bias;   // [d], null: 1, 1, 0
  void* H; void* Y;                                  // H null: not written
  float* mean; float* rstd;                          // [rows], null: not written
  uint8_t* H_q; uint8_t* H_qs;                       // with fmt
  uint8_t* B_q; uint8_t* B_qs;                       // with fmt, null: not written
  int chunk;                                         // set by the launcher
};
hipError_t launch_resid_norm_fwd(const ResidNormArgs& a, hipStream_t st);
struct ResidNormBwdArgs {
  Elt elt;
  int fmt;                                           // of H and B
  bool layer;
  int64_t rows;
  int d;
  float alpha;
  const void* dY; const void* dH_in;                 // dH_in null: 0
  const void* H; const uint8_t* H_qs;
  const void* B; const uint8_t* B_qs;                // only with dscale
  const float* mean; const float* rstd;
  const float* scale; const float* weight;
  void* dX; void* dB;                                // dB null: not written
  float* part;                                       // resid_norm_bwd_parts() rows of d per requested sum
  bool sum_w, sum_c;                                 // set by the launcher
  int tpr;
};
int resid_norm_bwd_parts(int64_t rows, int d);
// dscale, dweight, dbias null: not computed
hipError_t launch_resid_norm_bwd(const ResidNormBwdArgs& a, float* dscale, float* dweight, float* dbias,
                                 hipStream_t st);
struct GatedNormArgs {
  Elt elt;
  int fmt;
  bool layer;
  int64_t rows;
  int heads, d_v;                                    // d_v 64, 128, 256 or 512
  float eps;
  const void* O; const void* G;
  const float* weight; const float* bias;            // [heads, d_v], nullable
  void* Z;
  float* mean; float* rstd;                          // [rows, heads], nullable
  uint8_t* O_q; uint8_t* O_qs; uint8_t* G_q; uint8_t* G_qs;   // with fmt
  int R;                                             // set by the launcher
};
hipError_t launch_gated_norm_fwd(const GatedNormArgs& a, hipStream_t st);
struct GatedNormBwdArgs {
  Elt elt;
  int fmt;                                           // of O and G
  bool layer;
  int64_t rows;
  int heads, d_v;
  const void* dZ;
  const void* O; const uint8_t* O_qs;
  const void* G; const uint8_t* G_qs;
  const float* mean; const float* rstd;
  const float* weight; const float* bias;
  void* dO; void* dG; void* Z;                       // Z null: not written
  float* part;                                       // gated_norm_bwd_parts() rows of heads * d_v per requested sum
  bool sum_w, sum_c;                                 // set by the launcher
  int R;
};
int gated_norm_bwd_parts(int64_t rows, int heads, int d_v);
hipError_t launch_gated_norm_bwd(const GatedNormBwdArgs& a, float* dweight, float* dbias, hipStream_t st);
// out.v[i][j] = sum over p < P of part[i][p][j], i < vecs <= 3, j < n.
struct ColSumOut {
  float* v[3];
};
hipError_t launch_col_sums(const float* part, int P, int n, const ColSumOut& out, int vecs, hipStream_t st);

// ---- activations held in 8 bits (k_ckpt.hip) ----
hipError_t launch_ckpt_pack(Elt elt, int fmt, int64_t rows, int cols, const void* X, uint8_t* q, uint8_t* qs,
                            hipStream_t st);
// The values read back, optionally normalised: ((x - mean[row]) rstd[row])
// weight[col] + bias[col] (each nullable: 0, 1, 1, 0).
struct CkptArgs {
  int64_t rows;
  int cols;
  const uint8_t* q; const uint8_t* qs;
  const float* mean; const float* rstd; const float* weight; const float* bias;
};
hipError_t launch_ckpt_unpack(Elt elt, int fmt, const CkptArgs& a, void* X, hipStream_t st);
// A weight gradient X^T dY as a sum of products of bf16 pieces (see
// k_ckpt.hip): terms 1 (bf16 tensors), 3 (float32) or 6 (float32, normalised
// X) of X's and dY's pieces.
struct WgradPieces {
  int x, dy;
};
constexpr WgradPieces wgrad_pieces(int terms) { return {terms == 6 ? 3 : 1, terms == 1 ? 1 : 3}; }
// Its operands, of P pieces each: token t's piece p stands at index ((t / 64)
// P + p) 64 + t % 64; tokens past the last, up to 64 slabs, hold zeros.
// XT[col][index] bf16; a.cols a multiple of 64.
struct WgradOperands {
  CkptArgs a;
  uint16_t* XT;
  int64_t slabs;                     // of 64 tokens
  // dY [dy_rows, dy_cols] (dy_cols a multiple of 8).  float32: its pieces in
  // dYt[index][dy_cols].  bf16: the product reads it in place, but for a last
  // slab that it does not fill: with zeros behind it in dYt [64, dy_cols].
  const void* dY;
  int64_t dy_rows;
  int dy_cols;
  uint16_t* dYt;
};
hipError_t launch_wgrad_operands(Elt elt, int fmt, int terms, const WgradOperands& w, hipStream_t st);
// out[i] = (accumulate ? out[i] : 0) + sum over z < parts of part[z n + i], n a multiple of 4.
hipError_t launch_sum_parts(const float* part, int parts, float* out, int64_t n, bool accumulate, hipStream_t st);
// float32 products of K slices of bf16 matrices: the 64 slabs rows of K are
// cut into `splits` slices of whole slabs (the first slabs % splits one slab
// longer), slice z's product of A[m][k] B[k][n] in part[z M N + m N + n].  The
// last slab's rows of B are `tail` (row stride ldb) where that is given.  N a
// multiple of 64; on 256 x 256 tiles, or small_tiles: 128 x 64.
// terms 3 or 6 (no tail): `slabs` counts terms, A and B are a weight
// gradient's operands in pieces; terms of a token slab follow each other: 3:
// X with hi, mid, lo of dY; 6: hi hi, hi mid, mid hi, hi lo, mid mid, lo hi.
hipError_t launch_gemm_parts(const void* A, int64_t lda, const void* B, int64_t ldb, float* part, int M, int N,
                             int slabs, const void* tail, int terms, int splits, bool small_tiles, hipStream_t st);

}  // namespace msr
