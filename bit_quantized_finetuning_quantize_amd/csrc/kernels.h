// Internal launch interface between the C ABI (api.cpp) and the kernels.
// Launchers enqueue on `stream`, never synchronize, and return the launch
// status. Shapes have been validated by the caller.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "common.h"

namespace qlora {

struct Nf4Weight {
  const uint8_t* codes;
  const uint8_t* absmax_q;
  const float* absmax_s2;
  int store_type = 0;  // kStoreFP4 | kStoreDqFp8 (common.h); 0 is NF4, linear code
};

// The level table and constant code the kernels use for a store. A store
// without double quantization keeps float32 constants, so the constant code
// does not apply (the loaders read it with the 8-bit code forced to 255,
// whose linear value is exactly 1).
inline Codebook codebook_of(const Nf4Weight& W) {
  return make_codebook(W.absmax_q ? W.store_type : (W.store_type & kStoreFP4));
}

hipError_t launch_nf4_quantize(const uint16_t* w, int64_t numel, uint8_t* codes,
                               uint8_t* absmax_q, float* absmax_s2, int store_type,
                               hipStream_t stream);

hipError_t launch_nf4_dequantize(Nf4Weight W, int64_t numel, void* out, bool bf16,
                                 hipStream_t stream);

// Merged 16-bit weight: bf16(w' + s (A B)^T), [N x K] row-major.
hipError_t launch_nf4_merge(Nf4Weight W, int64_t N, int64_t K, const uint16_t* A,
                            const uint16_t* B, int r, float scale, uint16_t* out,
                            hipStream_t stream);

// One AdamW step over n float32 parameters with float32 moments (in place);
// p16 (optional) receives bf16(p).
hipError_t launch_adamw(float* p, float* m, float* v, const float* g, int64_t n, float lr,
                        float beta1, float beta2, float eps, float weight_decay, int64_t step,
                        uint16_t* p16, hipStream_t stream);

// The same step with 8-bit moments: per block of 256 parameters, E4M3 codes
// of m with scale sm[b] and E5M2 codes of v with scale sv[b] (updated in
// place).
hipError_t launch_adamw8(float* p, uint8_t* m8, float* sm, uint8_t* v8, float* sv, const float* g,
                         int64_t n, float lr, float beta1, float beta2, float eps,
                         float weight_decay, int64_t step, uint16_t* p16, hipStream_t stream);

// ---- LoRA dropout -------------------------------------------------------------

// Keep mask of an [M x K] adapter input (K a multiple of 32): Philox4x32-10
// with the 64-bit seed as key and (group, offset) as counter, one 16-bit
// value per element compared with thr; bits packed [M][K/32].
hipError_t launch_dropout_mask(int64_t M, int64_t K, uint32_t thr, uint64_t seed,
                               uint64_t offset, uint32_t* mask, hipStream_t stream);

// The mask and the inverse keep probability of one linear call; a null mask
// means no dropout.
struct Dropout {
  const uint32_t* mask = nullptr;
  float keep_scale = 1.0f;
};

// ---- linear layer -----------------------------------------------------------

// Workspace carve-up for the forward and backward of one linear call.
size_t linear_workspace_bytes(int64_t M, int64_t N, int64_t K, int r);

// Small-M forward (M <= kGemvMaxM): one launch; workgroups that form split
// partials of T = X A (a copy per XCD), and workgroups over row tiles of the
// whole K that wait for them, add s T B and write Y.
constexpr int kGemvMaxM = 16;
int64_t gemv_partial_elems(int64_t M, int64_t N, int64_t K, int r);
void set_gemv_wait_us(int64_t us);
hipError_t launch_fwd_gemv(const uint16_t* X, Nf4Weight W, const uint16_t* A,
                           const uint16_t* B, int M, int64_t N, int64_t K, int r,
                           float scale, uint16_t* Y, float* T_out, void* ws,
                           hipStream_t stream, hipEvent_t ev0 = nullptr,
                           hipEvent_t ev1 = nullptr);

// Large-M forward: T = X A, then Y = [X | s T] [W' | B^T]^T on MFMA tiles.
hipError_t launch_fwd_gemm(const uint16_t* X, Nf4Weight W, const uint16_t* A,
                           const uint16_t* B, int64_t M, int64_t N, int64_t K,
                           int r, float scale, uint16_t* Y, float* T_out, void* ws,
                           hipStream_t stream, hipEvent_t ev0 = nullptr,
                           hipEvent_t ev1 = nullptr, Dropout dr = Dropout{});

// Backward: G = dY B^T, dX = [dY | s G] [W' ; A^T], dA = s X^T G, dB = s T^T dY.
hipError_t launch_bwd(const uint16_t* dY, const uint16_t* X, const float* T,
                      Nf4Weight W, const uint16_t* A, const uint16_t* B,
                      int64_t M, int64_t N, int64_t K, int r, float scale,
                      uint16_t* dX, float* dA, float* dB, void* ws,
                      hipStream_t stream, hipEvent_t ev0 = nullptr,
                      hipEvent_t ev1 = nullptr, Dropout dr = Dropout{});

// ---- 8-bit blocks -------------------------------------------------------------

struct Act8 {
  uint8_t* codes;
  uint8_t* scales;
};
struct ConstAct8 {
  const uint8_t* codes;
  const uint8_t* scales;
};

// fmt: 0 E4M3, 1 E5M2 (include/qlora.h, "8-bit blocks"); ld: elements between rows.
hipError_t launch_act8_quantize(const uint16_t* X, int64_t M, int64_t K, int64_t ldx, int fmt,
                                uint8_t* codes, uint8_t* scales, hipStream_t stream);
hipError_t launch_act8_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t M, int64_t K,
                                  int fmt, uint16_t* X, int64_t ldx, hipStream_t stream);
hipError_t launch_fp8_weight_quantize(const uint16_t* W, int64_t N, int64_t K, Act8 w8, Act8 w8t,
                                      hipStream_t stream);
hipError_t launch_swiglu_act8_fwd(const uint16_t* g, int64_t ldg, const uint16_t* u, int64_t ldu,
                                  int64_t M, int64_t F, int fmt, uint16_t* h, int64_t ldh, Act8 h8,
                                  Act8 g8, Act8 u8, hipStream_t stream);
hipError_t launch_swiglu_act8_bwd(const uint16_t* dh, int64_t lddh, ConstAct8 g8, ConstAct8 u8,
                                  int64_t M, int64_t F, int fmt, uint16_t* dg, int64_t lddg,
                                  uint16_t* du, int64_t lddu, hipStream_t stream);

namespace lr8 {
struct ColPair;
}

// Memory for tiles that several workgroups share: kTileSums counts, 0 before,
// and 64 * 64 floats for each of at most kTileSums workgroups; or nulls.
constexpr int kTileSums = 256;
struct TileSums {
  uint32_t* done = nullptr;
  float* sums = nullptr;
};

// Y [M x N] = dec(x) dec(w)^T + U V^T; x [M x K], w [N x K] in 128 x 128
// blocks (E4M3), U bf16 [M x r64] and V bf16 [N x r64] or null; and the column
// products `cols` (or null).
hipError_t launch_fp8_gemm(ConstAct8 x, int xfmt, ConstAct8 w, int64_t M, int64_t N, int64_t K,
                           const uint16_t* U, const uint16_t* V, int r64, uint16_t* Y, TileSums sums,
                           const lr8::ColPair* cols, hipStream_t stream);

// The same for bf16 x [M x K] and w [N x K], K a multiple of 64, with a keep
// mask [M][N / 32] over the U V^T term (or null).
hipError_t launch_bf16_gemm(const uint16_t* x, const uint16_t* w, int64_t M, int64_t N, int64_t K,
                            const uint16_t* U, const uint16_t* V, int r64, const uint32_t* keep,
                            uint16_t* Y, TileSums sums, const lr8::ColPair* cols, hipStream_t stream);

// The same product where its output is small (fp8_few), the adapter's term
// from split partials of T (launch_rows_act8; null without an adapter) or, where
// fp8_few_forms_t, from A (else null); writes T_out. For few_t_shape
// launch_rows_act8 sums kFewWaves runs along K as that kernel does, so that
// both give T the same bits.
bool fp8_few(int64_t M, int64_t N);
bool few_t_shape(int64_t M, int64_t K, int r);
bool fp8_few_forms_t(const uint16_t* A, int64_t M, int64_t K, int r);
constexpr int kFewWaves = 8;
hipError_t launch_fp8_few(ConstAct8 x, int xfmt, ConstAct8 w, int64_t M, int64_t N, int64_t K,
                          const uint16_t* A, const float* part, int splits, const uint16_t* B, int r,
                          float scale, uint16_t* Y, float* T_out, hipStream_t stream);

// The adapter's products beside an 8-bit input (lowrank8.hip).
// Columns of a low-rank partial or term matrix: r rounded up to 16, 32 or a
// multiple of 64.
int lowrank_cols(int r);
// Split partials [splits][M][lowrank_cols(r)] of D(dec x) A (A [K x r]) and
// of S B^T (S bf16 [M x C], B [r x C]); K and C multiples of 64, at most
// max(256 * 64 * 64, M * lowrank_cols(r)) elements with M rounded up to 64.
hipError_t launch_rows_act8(ConstAct8 x, int fmt, int64_t M, int64_t K, const uint32_t* mask,
                            const uint16_t* A, int r, float* part, int* splits, hipStream_t stream);
hipError_t launch_rows_bf16(const uint16_t* S, int64_t M, int64_t C, const uint16_t* B, int r,
                            float* part, int* splits, hipStream_t stream);
// V = f * (sum of partials, rows ldp apart), as float32 [M x r], as bf16(s V)
// [Mp x r64], and as s V in the order launch_columns reads it (Mp x
// lowrank_cols(r) floats); each output may be null. Up to two of them and one padded copy per launch:
// dst [rows x r64] from src [rows x r], or from the columns of src [r x rows].
struct LowrankOut {
  const float* part;  // or null, with
  const uint16_t *s, *w;  // the factors of V = S W^T: S bf16 [M x C], W [r x C], C a multiple of 64
  int64_t C;
  int splits;
  int64_t ldp;
  float f;
  float* out32;
  uint16_t* u;
  float* vf;
};
struct LowrankPad {
  const uint16_t* src = nullptr;
  bool columns = false;
  int64_t rows = 0;
  uint16_t* dst = nullptr;
};
// Beside them in the same launch, none or one of:
//   codes, scales  8-bit blocks in fmt of bf16 s [M x C], 16-byte aligned, C a multiple of 8
//   w [K x N]      bf16(w')^T of a store of W [N x K], N and K multiples of 64
struct LowrankBeside {
  const uint16_t* s = nullptr;
  int64_t C = 0;
  int fmt = 0;
  uint8_t *codes = nullptr, *scales = nullptr;
  Nf4Weight W{};
  int64_t N = 0, K = 0;
  uint16_t* w = nullptr;
};
// `done`: the counts of a TileSums, set to 0 (or null).
hipError_t launch_lowrank_out(const LowrankOut* o, int n, LowrankPad pad, int64_t M, int r, float s,
                              uint32_t* done, hipStream_t stream, const LowrankBeside& beside = LowrankBeside{});
// dA = D(dec x)^T g, dB = t^T dY, g and t as launch_lowrank_out's vf (lowrank8.h).
hipError_t launch_columns(const lr8::ColPair& p, hipStream_t stream);

// Workspace of the three calls below (r may be 0 for the 8-bit weight's): the
// adapter's factors alone (the forward, a backward pass without dX), with dY in
// 8 bits (the 8-bit weight's dX), or with that or the bf16 copy of a 4-bit weight.
enum class Act8Ws { kFactors, kDy8, kWeight };
size_t act8_workspace_bytes(int64_t M, int64_t N, int64_t K, int r, Act8Ws what);
// launch_bwd with the input in 8-bit blocks.
hipError_t launch_bwd_act8(const uint16_t* dY, ConstAct8 x, int fmt, const float* T, Nf4Weight W,
                           const uint16_t* A, const uint16_t* B, int64_t M, int64_t N, int64_t K,
                           int r, float scale, uint16_t* dX, float* dA, float* dB, void* ws,
                           hipStream_t stream, Dropout dr = Dropout{});
// Y = dec(x) dec(w)^T + s T B, T = dec(x) A (no adapter when r = 0).
hipError_t launch_fp8_fwd(ConstAct8 x, int fmt, ConstAct8 w, const uint16_t* A, const uint16_t* B,
                          int64_t M, int64_t N, int64_t K, int r, float scale, uint16_t* Y,
                          float* T_out, void* ws, hipStream_t stream);
// dX = dec(q(dY)) dec(w) + s G A^T, dA = s dec(x)^T G, dB = s T^T dY; w^T given.
hipError_t launch_fp8_bwd(const uint16_t* dY, int dyfmt, ConstAct8 x, int fmt, const float* T,
                          ConstAct8 w_t, const uint16_t* A, const uint16_t* B, int64_t M, int64_t N,
                          int64_t K, int r, float scale, uint16_t* dX, float* dA, float* dB,
                          void* ws, hipStream_t stream);

// ---- rows of logits (logits.hip) ------------------------------------------------

// Z [T x V], rows ldz elements apart, bf16 or float32.
struct Logits {
  const void* Z;
  bool f32;
  int64_t T, V, ldz;
  double temperature;
};
// A teacher's k largest logits of each row and their ids, [T x k].
struct TopLogits {
  const int64_t* ids;
  const void* values;
  bool f32;
  int k;
};
size_t logits_workspace_bytes(int64_t T, int64_t V, int n_top);
hipError_t launch_logprobs_fwd(const Logits& z, const int64_t* target, float* logp, float* entropy, int n_top,
                               int64_t* top_ids, float* top_logp, float* stats, void* ws, hipStream_t stream);
hipError_t launch_logprobs_bwd(const Logits& z, const int64_t* target, const float* stats, const float* g_logp,
                               const float* g_entropy, void* dZ, int64_t lddz, hipStream_t stream);
hipError_t launch_distill_fwd(const Logits& z, const TopLogits& t, const float* teacher_lse, float* loss,
                              float* stats, void* ws, hipStream_t stream);
hipError_t launch_distill_bwd(const Logits& z, const TopLogits& t, const float* stats, const float* g, void* dZ,
                              int64_t lddz, hipStream_t stream);

// ---- 4 bits in groups (int4.hip) --------------------------------------------------

// [N x K] codes, scales bf16 and zero points (null: 8) [N x ceil(K / group)].
struct Int4Weight {
  const uint8_t* codes;
  const uint16_t* scales;
  const uint8_t* zeros;
  int64_t N, K;
  int group;  // 32, 64 or 128
};
hipError_t launch_int4_quantize(const uint16_t* W, int64_t N, int64_t K, int64_t ldw, int group, uint8_t* codes,
                                uint16_t* scales, uint8_t* zeros, hipStream_t stream);
hipError_t launch_int4_dequantize(const Int4Weight& w, uint16_t* out, int64_t ldo, hipStream_t stream);
hipError_t launch_int4_linear_fwd(const uint16_t* X, int64_t M, int64_t ldx, const Int4Weight& w, void* Y, bool f32,
                                  int64_t ldy, hipStream_t stream);

// Forward with the library's own scratch array (one per device, this many
// bytes) in place of a caller workspace.
constexpr size_t kNoAllocScratchBytes = (size_t)32 << 20;
hipError_t launch_fwd_noalloc(const uint16_t* X, Nf4Weight W, const uint16_t* A,
                              const uint16_t* B, int64_t M, int64_t N, int64_t K, int r,
                              float scale, uint16_t* Y, float* T_out, hipStream_t stream);

// Records `ev` on `stream` when it is not null (profiling hooks around the
// dominant launch of a call).
inline hipError_t record_if(hipEvent_t ev, hipStream_t stream) {
  return ev ? hipEventRecord(ev, stream) : hipSuccess;
}

}  // namespace qlora
