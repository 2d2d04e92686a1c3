// C ABI of the library: argument validation, dispatch, status codes.
// Every check runs before anything is enqueued; a rejected call has no side
// effects and makes no HIP call.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/qlora.h"
#include "act8.h"
#include "common.h"
#include "kernels.h"

namespace {

thread_local int g_last_hip_error = 0;

int hip_status(hipError_t e) {
  if (e == hipSuccess) return QLORA_OK;
  g_last_hip_error = (int)e;
  return QLORA_ERR_HIP;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int64_t kMaxGroups = 0x7fffffffLL;  // grid limit of the quantize launch

// absmax_q may be null: a store without double quantization
int check_store(const uint8_t* codes, const uint8_t* absmax_q, const float* absmax_s2) {
  (void)absmax_q;
  if (!codes || !absmax_s2) return QLORA_ERR_INVALID_ARG;
  if (!aligned(codes, 16) || !aligned(absmax_s2, 4)) return QLORA_ERR_UNSUPPORTED;
  return QLORA_OK;
}

bool valid_store_type(int32_t t) { return t >= 0 && t <= (QLORA_STORE_FP4 | QLORA_STORE_DQ_FP8); }

int check_linear_shape(int64_t M, int64_t N, int64_t K, int32_t r) {
  if (M <= 0 || N <= 0 || K <= 0) return QLORA_ERR_INVALID_ARG;
  if (K % QLORA_NF4_BLOCK != 0 || N % QLORA_NF4_BLOCK != 0) return QLORA_ERR_UNSUPPORTED;
  if (r < 1 || r > QLORA_MAX_RANK) return QLORA_ERR_UNSUPPORTED;
  if (M > (int64_t)1 << 30 || N > (int64_t)1 << 30 || K > (int64_t)1 << 30) return QLORA_ERR_UNSUPPORTED;
  // The kernels address their operands with 32-bit buffer offsets: every
  // bf16 activation matrix stays below 2^30 elements (2 GiB), the NF4 codes
  // below 2 GiB, and a row below 2^21 elements (a 256-row tile spans at most
  // 1 GiB).
  if (N > (int64_t)1 << 21 || K > (int64_t)1 << 21) return QLORA_ERR_UNSUPPORTED;
  if (M * N >= (int64_t)1 << 30 || M * K >= (int64_t)1 << 30 || N * K >= (int64_t)1 << 32)
    return QLORA_ERR_UNSUPPORTED;
  return QLORA_OK;
}

// 16-bit keep threshold of a drop probability p in [0, 1): floor(p 2^16 + 1/2)
// (p * 2^16 is exact in double). Returns -1 for p outside [0, 1) or NaN, and
// 65536 when p rounds to certain dropping.
int64_t keep_threshold(float p) {
  if (!(p >= 0.0f && p < 1.0f)) return -1;
  return (int64_t)std::floor((double)p * 65536.0 + 0.5);
}

int check_dropout(const uint32_t* mask, float p, qlora::Dropout* dr) {
  if (!mask) return QLORA_ERR_INVALID_ARG;
  const int64_t thr = keep_threshold(p);
  if (thr < 0) return QLORA_ERR_INVALID_ARG;
  if (thr >= 65536) return QLORA_ERR_UNSUPPORTED;
  if (!aligned(mask, 4)) return QLORA_ERR_UNSUPPORTED;
  dr->mask = mask;
  dr->keep_scale = (float)(65536.0 / (double)(65536 - thr));
  return QLORA_OK;
}

bool valid_fmt(int32_t f) { return f == QLORA_ACT8_E4M3 || f == QLORA_ACT8_E5M2; }

// Shape of a matrix in 8-bit blocks: one lane group per block of 128 in one
// launch (32-bit block index), and rows that 32-bit offsets can reach.
int check_act8_shape(int64_t M, int64_t K) {
  if (M <= 0 || K <= 0) return QLORA_ERR_INVALID_ARG;
  if (M > (int64_t)1 << 30 || K > (int64_t)1 << 21) return QLORA_ERR_UNSUPPORTED;
  const int64_t kb = (K + QLORA_ACT8_BLOCK - 1) / QLORA_ACT8_BLOCK;
  if (M * kb > (int64_t)1 << 30) return QLORA_ERR_UNSUPPORTED;
  return QLORA_OK;
}

int check_act8(const uint8_t* codes, const uint8_t* scales) {
  if (!codes || !scales) return QLORA_ERR_INVALID_ARG;
  if (!aligned(codes, 16) || !aligned(scales, 4)) return QLORA_ERR_UNSUPPORTED;
  return QLORA_OK;
}

// Shapes of the linear calls on 8-bit inputs; r = 0 is a call without an adapter.
int check_fp8_shape(int64_t M, int64_t N, int64_t K, int32_t r) {
  if (M <= 0 || N <= 0 || K <= 0) return QLORA_ERR_INVALID_ARG;
  if (r) return check_linear_shape(M, N, K, r);
  if (N > (int64_t)1 << 21 || K > (int64_t)1 << 21 || M > (int64_t)1 << 30)
    return QLORA_ERR_UNSUPPORTED;
  const int64_t np = (N + 127) / 128 * 128, kp = (K + 127) / 128 * 128;
  if (M * np >= (int64_t)1 << 30 || M * kp >= (int64_t)1 << 30 || np * kp >= (int64_t)1 << 32)
    return QLORA_ERR_UNSUPPORTED;
  return QLORA_OK;
}

// A weight in groups of 4-bit codes.
int check_int4(const void* codes, const void* scales, int64_t N, int64_t K, int32_t group) {
  if (!codes || !scales || N <= 0 || K <= 0) return QLORA_ERR_INVALID_ARG;
  if (group != 32 && group != 64 && group != 128) return QLORA_ERR_UNSUPPORTED;
  if (K % 32 || N > (int64_t)1 << 21 || K > (int64_t)1 << 21 || N * K >= (int64_t)1 << 32)
    return QLORA_ERR_UNSUPPORTED;
  return aligned(codes, 16) && aligned(scales, 2) ? QLORA_OK : QLORA_ERR_UNSUPPORTED;
}

// Rows of logits.
int check_logits(const void* Z, int32_t dtype, int64_t T, int64_t V, int64_t ldz, double temperature,
                 qlora::Logits* z) {
  if (!Z || T <= 0 || V <= 0 || ldz < V) return QLORA_ERR_INVALID_ARG;
  if (dtype != QLORA_LOGITS_BF16 && dtype != QLORA_LOGITS_F32) return QLORA_ERR_INVALID_ARG;
  if (!(temperature > 0.0) || std::isinf(temperature)) return QLORA_ERR_INVALID_ARG;
  if (T > (int64_t)1 << 23 || V > (int64_t)1 << 21 || ldz > (int64_t)1 << 32) return QLORA_ERR_UNSUPPORTED;
  if (temperature < 0x1p-40 || temperature > 0x1p40) return QLORA_ERR_UNSUPPORTED;
  if (!aligned(Z, dtype == QLORA_LOGITS_F32 ? 4 : 2)) return QLORA_ERR_UNSUPPORTED;
  *z = qlora::Logits{Z, dtype == QLORA_LOGITS_F32, T, V, ldz, temperature};
  return QLORA_OK;
}

int check_top_logits(const int64_t* ids, const void* values, int32_t dtype, int32_t k, qlora::TopLogits* t) {
  if (!ids || !values || k <= 0) return QLORA_ERR_INVALID_ARG;
  if (dtype != QLORA_LOGITS_BF16 && dtype != QLORA_LOGITS_F32) return QLORA_ERR_INVALID_ARG;
  if (k > QLORA_MAX_TEACHER_LOGITS) return QLORA_ERR_UNSUPPORTED;
  if (!aligned(ids, 8) || !aligned(values, dtype == QLORA_LOGITS_F32 ? 4 : 2)) return QLORA_ERR_UNSUPPORTED;
  *t = qlora::TopLogits{ids, values, dtype == QLORA_LOGITS_F32, k};
  return QLORA_OK;
}

int check_dlogits(const void* dZ, int64_t lddz, const qlora::Logits& z) {
  if (!dZ || lddz < z.V) return QLORA_ERR_INVALID_ARG;
  if (lddz > (int64_t)1 << 32 || !aligned(dZ, z.f32 ? 4 : 2)) return QLORA_ERR_UNSUPPORTED;
  // in place each workgroup writes only what itself has read
  return dZ == z.Z && z.T > 1 && lddz != z.ldz ? QLORA_ERR_INVALID_ARG : QLORA_OK;
}

int check_logits_ws(const qlora::Logits& z, int n_top, const void* ws, size_t ws_bytes) {
  if (!ws || ws_bytes < qlora::logits_workspace_bytes(z.T, z.V, n_top)) return QLORA_ERR_WORKSPACE;
  return aligned(ws, 256) ? QLORA_OK : QLORA_ERR_UNSUPPORTED;
}

}  // namespace

extern "C" {

int64_t qlora_nf4_codes_bytes(int64_t numel) { return numel < 0 ? -1 : (numel + 1) / 2; }
int64_t qlora_nf4_num_blocks(int64_t numel) {
  return numel < 0 ? -1 : (numel + QLORA_NF4_BLOCK - 1) / QLORA_NF4_BLOCK;
}
int64_t qlora_nf4_num_groups(int64_t numel) {
  return numel < 0 ? -1 : (qlora_nf4_num_blocks(numel) + QLORA_NF4_GROUP - 1) / QLORA_NF4_GROUP;
}

void qlora_nf4_codebook(float* levels) {
  if (!levels) return;
  std::memcpy(levels, qlora::kNF4, sizeof(qlora::kNF4));
}

int qlora_nf4_quantize_ex(const uint16_t* w, int64_t numel, uint8_t* codes, uint8_t* absmax_q,
                          float* absmax_s2, int32_t store_type, void* stream) {
  if (!w || numel <= 0) return QLORA_ERR_INVALID_ARG;
  if (!codes || !absmax_s2) return QLORA_ERR_INVALID_ARG;  // absmax_q null: no DQ
  if (!valid_store_type(store_type)) return QLORA_ERR_INVALID_ARG;
  if (!aligned(w, 2) || !aligned(codes, 4) || !aligned(absmax_s2, 4)) return QLORA_ERR_UNSUPPORTED;
  if (qlora_nf4_num_groups(numel) > kMaxGroups) return QLORA_ERR_UNSUPPORTED;
  return hip_status(qlora::launch_nf4_quantize(w, numel, codes, absmax_q, absmax_s2, store_type,
                                               reinterpret_cast<hipStream_t>(stream)));
}

int qlora_nf4_quantize(const uint16_t* w, int64_t numel, uint8_t* codes, uint8_t* absmax_q,
                       float* absmax_s2, void* stream) {
  return qlora_nf4_quantize_ex(w, numel, codes, absmax_q, absmax_s2, QLORA_STORE_NF4, stream);
}

static int dequant_common(const uint8_t* codes, const uint8_t* absmax_q, const float* absmax_s2,
                          int64_t numel, int32_t store_type, void* out, bool bf16, void* stream) {
  if (!codes || !absmax_s2 || !out || numel <= 0) return QLORA_ERR_INVALID_ARG;
  if (!valid_store_type(store_type)) return QLORA_ERR_INVALID_ARG;
  if (!aligned(codes, 4) || !aligned(absmax_s2, 4) || !aligned(out, 16)) return QLORA_ERR_UNSUPPORTED;
  return hip_status(qlora::launch_nf4_dequantize(qlora::Nf4Weight{codes, absmax_q, absmax_s2,
                                                                  store_type},
                                                 numel, out, bf16,
                                                 reinterpret_cast<hipStream_t>(stream)));
}

int qlora_nf4_dequantize_ex(const uint8_t* codes, const uint8_t* absmax_q,
                            const float* absmax_s2, int64_t numel, int32_t store_type,
                            float* out, void* stream) {
  return dequant_common(codes, absmax_q, absmax_s2, numel, store_type, out, false, stream);
}

int qlora_nf4_dequantize_bf16_ex(const uint8_t* codes, const uint8_t* absmax_q,
                                 const float* absmax_s2, int64_t numel, int32_t store_type,
                                 uint16_t* out, void* stream) {
  return dequant_common(codes, absmax_q, absmax_s2, numel, store_type, out, true, stream);
}

int qlora_nf4_dequantize(const uint8_t* codes, const uint8_t* absmax_q, const float* absmax_s2,
                         int64_t numel, float* out, void* stream) {
  return dequant_common(codes, absmax_q, absmax_s2, numel, QLORA_STORE_NF4, out, false, stream);
}

int qlora_nf4_dequantize_bf16(const uint8_t* codes, const uint8_t* absmax_q,
                              const float* absmax_s2, int64_t numel, uint16_t* out,
                              void* stream) {
  return dequant_common(codes, absmax_q, absmax_s2, numel, QLORA_STORE_NF4, out, true, stream);
}

int qlora_nf4_merge(const uint8_t* codes, const uint8_t* absmax_q, const float* absmax_s2,
                    int64_t N, int64_t K, const uint16_t* A, const uint16_t* B, int32_t r,
                    float scale, uint16_t* out, void* stream) {
  return qlora_nf4_merge_ex(codes, absmax_q, absmax_s2, N, K, A, B, r, scale, QLORA_STORE_NF4,
                            out, stream);
}

int qlora_nf4_merge_ex(const uint8_t* codes, const uint8_t* absmax_q, const float* absmax_s2,
                       int64_t N, int64_t K, const uint16_t* A, const uint16_t* B, int32_t r,
                       float scale, int32_t store_type, uint16_t* out, void* stream) {
  if (!A || !B || !out) return QLORA_ERR_INVALID_ARG;
  if (!valid_store_type(store_type)) return QLORA_ERR_INVALID_ARG;
  int st = check_store(codes, absmax_q, absmax_s2);
  if (st != QLORA_OK) return st;
  if (N <= 0 || K <= 0) return QLORA_ERR_INVALID_ARG;
  if (K % QLORA_NF4_BLOCK != 0 || r < 1 || r > QLORA_MAX_RANK) return QLORA_ERR_UNSUPPORTED;
  if (N > (int64_t)1 << 30 || K > (int64_t)1 << 30 || (N + 63) / 64 > 65535)
    return QLORA_ERR_UNSUPPORTED;
  if (!aligned(A, 2) || !aligned(B, 2) || !aligned(out, 16)) return QLORA_ERR_UNSUPPORTED;
  return hip_status(qlora::launch_nf4_merge(qlora::Nf4Weight{codes, absmax_q, absmax_s2, store_type},
                                            N, K, A, B, r, scale, out,
                                            reinterpret_cast<hipStream_t>(stream)));
}

int qlora_adamw_step(float* p, float* m, float* v, const float* g, int64_t n, float lr,
                     float beta1, float beta2, float eps, float weight_decay, int64_t step,
                     uint16_t* p_bf16, void* stream) {
  if (!p || !m || !v || !g || n <= 0 || step < 1) return QLORA_ERR_INVALID_ARG;
  if (!(beta1 >= 0.0f && beta1 < 1.0f) || !(beta2 >= 0.0f && beta2 < 1.0f) || !(eps > 0.0f))
    return QLORA_ERR_INVALID_ARG;
  if (!aligned(p, 4) || !aligned(m, 4) || !aligned(v, 4) || !aligned(g, 4) ||
      (p_bf16 && !aligned(p_bf16, 2)))
    return QLORA_ERR_UNSUPPORTED;
  return hip_status(qlora::launch_adamw(p, m, v, g, n, lr, beta1, beta2, eps, weight_decay, step,
                                        p_bf16, reinterpret_cast<hipStream_t>(stream)));
}

int qlora_adamw8_step(float* p, uint8_t* m8, float* m_scale, uint8_t* v8, float* v_scale,
                      const float* g, int64_t n, float lr, float beta1, float beta2, float eps,
                      float weight_decay, int64_t step, uint16_t* p_bf16, void* stream) {
  if (!p || !m8 || !m_scale || !v8 || !v_scale || !g || n <= 0 || step < 1)
    return QLORA_ERR_INVALID_ARG;
  if (!(beta1 >= 0.0f && beta1 < 1.0f) || !(beta2 >= 0.0f && beta2 < 1.0f) || !(eps > 0.0f))
    return QLORA_ERR_INVALID_ARG;
  if (!aligned(p, 4) || !aligned(g, 4) || !aligned(m_scale, 4) || !aligned(v_scale, 4) ||
      (p_bf16 && !aligned(p_bf16, 2)))
    return QLORA_ERR_UNSUPPORTED;
  return hip_status(qlora::launch_adamw8(p, m8, m_scale, v8, v_scale, g, n, lr, beta1, beta2, eps,
                                         weight_decay, step, p_bf16,
                                         reinterpret_cast<hipStream_t>(stream)));
}

size_t qlora_linear_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t r) {
  if (check_linear_shape(M, N, K, r) != QLORA_OK) return 0;
  return qlora::linear_workspace_bytes(M, N, K, r);
}

static int linear_fwd_impl(const uint16_t* X, const uint8_t* codes, const uint8_t* absmax_q,
                           const float* absmax_s2, const uint16_t* A, const uint16_t* B,
                           int64_t M, int64_t N, int64_t K, int32_t r, float scale, uint16_t* Y,
                           float* T_out, void* ws, size_t ws_bytes, int32_t store_type,
                           void* stream, void* ev_begin, void* ev_end) {
  if (!X || !A || !B || !Y) return QLORA_ERR_INVALID_ARG;
  if (!valid_store_type(store_type)) return QLORA_ERR_INVALID_ARG;
  int st = check_store(codes, absmax_q, absmax_s2);
  if (st != QLORA_OK) return st;
  st = check_linear_shape(M, N, K, r);
  if (st != QLORA_OK) return st;
  if (!aligned(X, 16) || !aligned(B, 16) || !aligned(A, 2) || !aligned(Y, 2) ||
      (T_out && !aligned(T_out, 4)))
    return QLORA_ERR_UNSUPPORTED;
  const size_t need = qlora::linear_workspace_bytes(M, N, K, r);
  if (!ws || ws_bytes < need) return QLORA_ERR_WORKSPACE;
  if (!aligned(ws, 256)) return QLORA_ERR_UNSUPPORTED;
  qlora::Nf4Weight W{codes, absmax_q, absmax_s2, store_type};
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  hipEvent_t e0 = reinterpret_cast<hipEvent_t>(ev_begin);
  hipEvent_t e1 = reinterpret_cast<hipEvent_t>(ev_end);
  if (M <= qlora::kGemvMaxM)
    return hip_status(
        qlora::launch_fwd_gemv(X, W, A, B, (int)M, N, K, r, scale, Y, T_out, ws, s, e0, e1));
  return hip_status(qlora::launch_fwd_gemm(X, W, A, B, M, N, K, r, scale, Y, T_out, ws, s, e0, e1));
}

int qlora_linear_fwd_profiled(const uint16_t* X, const uint8_t* codes, const uint8_t* absmax_q,
                              const float* absmax_s2, const uint16_t* A, const uint16_t* B,
                              int64_t M, int64_t N, int64_t K, int32_t r, float scale,
                              uint16_t* Y, float* T_out, void* ws, size_t ws_bytes, void* stream,
                              void* ev_begin, void* ev_end) {
  return linear_fwd_impl(X, codes, absmax_q, absmax_s2, A, B, M, N, K, r, scale, Y, T_out, ws,
                         ws_bytes, QLORA_STORE_NF4, stream, ev_begin, ev_end);
}

int qlora_linear_fwd(const uint16_t* X, const uint8_t* codes, const uint8_t* absmax_q,
                     const float* absmax_s2, const uint16_t* A, const uint16_t* B, int64_t M,
                     int64_t N, int64_t K, int32_t r, float scale, uint16_t* Y, float* T_out,
                     void* ws, size_t ws_bytes, void* stream) {
  return linear_fwd_impl(X, codes, absmax_q, absmax_s2, A, B, M, N, K, r, scale, Y, T_out, ws,
                         ws_bytes, QLORA_STORE_NF4, stream, nullptr, nullptr);
}

int qlora_linear_fwd_ex(const uint16_t* X, const uint8_t* codes, const uint8_t* absmax_q,
                        const float* absmax_s2, const uint16_t* A, const uint16_t* B, int64_t M,
                        int64_t N, int64_t K, int32_t r, float scale, uint16_t* Y, float* T_out,
                        void* ws, size_t ws_bytes, int32_t store_type, void* stream) {
  return linear_fwd_impl(X, codes, absmax_q, absmax_s2, A, B, M, N, K, r, scale, Y, T_out, ws,
                         ws_bytes, store_type, stream, nullptr, nullptr);
}

int qlora_linear_fwd_noalloc(const uint16_t* X, const uint8_t* codes, const uint8_t* absmax_q,
                             const float* absmax_s2, const uint16_t* A, const uint16_t* B,
                             int64_t M, int64_t N, int64_t K, int32_t r, float scale, uint16_t* Y,
                             float* T_out, void* stream) {
  static_assert(QLORA_NOALLOC_SCRATCH_BYTES == qlora::kNoAllocScratchBytes, "scratch size");
  if (!X || !A || !B || !Y) return QLORA_ERR_INVALID_ARG;
  int st = check_store(codes, absmax_q, absmax_s2);
  if (st != QLORA_OK) return st;
  st = check_linear_shape(M, N, K, r);
  if (st != QLORA_OK) return st;
  if (!aligned(X, 16) || !aligned(B, 16) || !aligned(A, 2) || !aligned(Y, 2) ||
      (T_out && !aligned(T_out, 4)))
    return QLORA_ERR_UNSUPPORTED;
  if (qlora::linear_workspace_bytes(M, N, K, r) > qlora::kNoAllocScratchBytes)
    return QLORA_ERR_WORKSPACE;
  qlora::Nf4Weight W{codes, absmax_q, absmax_s2};
  return hip_status(qlora::launch_fwd_noalloc(X, W, A, B, M, N, K, r, scale, Y, T_out,
                                              reinterpret_cast<hipStream_t>(stream)));
}

static int linear_bwd_impl(const uint16_t* dY, const uint16_t* X, const float* T,
                           const uint8_t* codes, const uint8_t* absmax_q, const float* absmax_s2,
                           const uint16_t* A, const uint16_t* B, int64_t M, int64_t N, int64_t K,
                           int32_t r, float scale, uint16_t* dX, float* dA, float* dB, void* ws,
                           size_t ws_bytes, int32_t store_type, void* stream, void* ev_begin,
                           void* ev_end) {
  if (!dY || !X || !A || !B || !dA || !dB) return QLORA_ERR_INVALID_ARG;
  if (!valid_store_type(store_type)) return QLORA_ERR_INVALID_ARG;
  int st = check_store(codes, absmax_q, absmax_s2);
  if (st != QLORA_OK) return st;
  st = check_linear_shape(M, N, K, r);
  if (st != QLORA_OK) return st;
  if (!aligned(dY, 16) || !aligned(X, 16) || !aligned(B, 16) || !aligned(A, 2) ||
      (T && !aligned(T, 4)) || (dX && !aligned(dX, 2)) || !aligned(dA, 4) || !aligned(dB, 4))
    return QLORA_ERR_UNSUPPORTED;
  const size_t need = qlora::linear_workspace_bytes(M, N, K, r);
  if (!ws || ws_bytes < need) return QLORA_ERR_WORKSPACE;
  if (!aligned(ws, 256)) return QLORA_ERR_UNSUPPORTED;
  qlora::Nf4Weight W{codes, absmax_q, absmax_s2, store_type};
  return hip_status(qlora::launch_bwd(dY, X, T, W, A, B, M, N, K, r, scale, dX, dA, dB, ws,
                                      reinterpret_cast<hipStream_t>(stream),
                                      reinterpret_cast<hipEvent_t>(ev_begin),
                                      reinterpret_cast<hipEvent_t>(ev_end)));
}

int qlora_linear_bwd_profiled(const uint16_t* dY, const uint16_t* X, const float* T,
                              const uint8_t* codes, const uint8_t* absmax_q,
                              const float* absmax_s2, const uint16_t* A, const uint16_t* B,
                              int64_t M, int64_t N, int64_t K, int32_t r, float scale,
                              uint16_t* dX, float* dA, float* dB, void* ws, size_t ws_bytes,
                              void* stream, void* ev_begin, void* ev_end) {
  return linear_bwd_impl(dY, X, T, codes, absmax_q, absmax_s2, A, B, M, N, K, r, scale, dX, dA,
                         dB, ws, ws_bytes, QLORA_STORE_NF4, stream, ev_begin, ev_end);
}

int qlora_linear_bwd(const uint16_t* dY, const uint16_t* X, const float* T, const uint8_t* codes,
                     const uint8_t* absmax_q, const float* absmax_s2, const uint16_t* A,
                     const uint16_t* B, int64_t M, int64_t N, int64_t K, int32_t r, float scale,
                     uint16_t* dX, float* dA, float* dB, void* ws, size_t ws_bytes,
                     void* stream) {
  return linear_bwd_impl(dY, X, T, codes, absmax_q, absmax_s2, A, B, M, N, K, r, scale, dX, dA,
                         dB, ws, ws_bytes, QLORA_STORE_NF4, stream, nullptr, nullptr);
}

int qlora_linear_bwd_ex(const uint16_t* dY, const uint16_t* X, const float* T,
                        const uint8_t* codes, const uint8_t* absmax_q, const float* absmax_s2,
                        const uint16_t* A, const uint16_t* B, int64_t M, int64_t N, int64_t K,
                        int32_t r, float scale, uint16_t* dX, float* dA, float* dB, void* ws,
                        size_t ws_bytes, int32_t store_type, void* stream) {
  return linear_bwd_impl(dY, X, T, codes, absmax_q, absmax_s2, A, B, M, N, K, r, scale, dX, dA,
                         dB, ws, ws_bytes, store_type, stream, nullptr, nullptr);
}

int qlora_dropout_mask(int64_t M, int64_t K, float p, uint64_t seed, uint64_t offset,
                       uint32_t* mask, void* stream) {
  if (!mask || M <= 0 || K <= 0) return QLORA_ERR_INVALID_ARG;
  const int64_t thr = keep_threshold(p);
  if (thr < 0) return QLORA_ERR_INVALID_ARG;
  if (thr >= 65536 || K % 32 != 0 || !aligned(mask, 4)) return QLORA_ERR_UNSUPPORTED;
  if (M > ((int64_t)1 << 40) / K) return QLORA_ERR_UNSUPPORTED;
  return hip_status(qlora::launch_dropout_mask(M, K, (uint32_t)thr, seed, offset, mask,
                                               reinterpret_cast<hipStream_t>(stream)));
}

int qlora_linear_fwd_dropout(const uint16_t* X, const uint8_t* codes, const uint8_t* absmax_q,
                             const float* absmax_s2, const uint16_t* A, const uint16_t* B,
                             int64_t M, int64_t N, int64_t K, int32_t r, float scale,
                             const uint32_t* keep_mask, float p, uint16_t* Y, float* T_out,
                             void* ws, size_t ws_bytes, void* stream) {
  if (!X || !A || !B || !Y) return QLORA_ERR_INVALID_ARG;
  int st = check_store(codes, absmax_q, absmax_s2);
  if (st != QLORA_OK) return st;
  st = check_linear_shape(M, N, K, r);
  if (st != QLORA_OK) return st;
  qlora::Dropout dr;
  st = check_dropout(keep_mask, p, &dr);
  if (st != QLORA_OK) return st;
  if (!aligned(X, 16) || !aligned(B, 16) || !aligned(A, 2) || !aligned(Y, 2) ||
      (T_out && !aligned(T_out, 4)))
    return QLORA_ERR_UNSUPPORTED;
  const size_t need = qlora::linear_workspace_bytes(M, N, K, r);
  if (!ws || ws_bytes < need) return QLORA_ERR_WORKSPACE;
  if (!aligned(ws, 256)) return QLORA_ERR_UNSUPPORTED;
  qlora::Nf4Weight W{codes, absmax_q, absmax_s2};
  // every M takes the MFMA path: the keep mask enters the X A contraction
  return hip_status(qlora::launch_fwd_gemm(X, W, A, B, M, N, K, r, scale, Y, T_out, ws,
                                           reinterpret_cast<hipStream_t>(stream), nullptr,
                                           nullptr, dr));
}

int qlora_linear_bwd_dropout(const uint16_t* dY, const uint16_t* X, const float* T,
                             const uint8_t* codes, const uint8_t* absmax_q,
                             const float* absmax_s2, const uint16_t* A, const uint16_t* B,
                             int64_t M, int64_t N, int64_t K, int32_t r, float scale,
                             const uint32_t* keep_mask, float p, uint16_t* dX, float* dA,
                             float* dB, void* ws, size_t ws_bytes, void* stream) {
  if (!dY || !X || !A || !B || !dA || !dB) return QLORA_ERR_INVALID_ARG;
  int st = check_store(codes, absmax_q, absmax_s2);
  if (st != QLORA_OK) return st;
  st = check_linear_shape(M, N, K, r);
  if (st != QLORA_OK) return st;
  qlora::Dropout dr;
  st = check_dropout(keep_mask, p, &dr);
  if (st != QLORA_OK) return st;
  if (dX && r > QLORA_MAX_DROPOUT_RANK) return QLORA_ERR_UNSUPPORTED;
  if (!aligned(dY, 16) || !aligned(X, 16) || !aligned(B, 16) || !aligned(A, 2) ||
      (T && !aligned(T, 4)) || (dX && !aligned(dX, 2)) || !aligned(dA, 4) || !aligned(dB, 4))
    return QLORA_ERR_UNSUPPORTED;
  const size_t need = qlora::linear_workspace_bytes(M, N, K, r);
  if (!ws || ws_bytes < need) return QLORA_ERR_WORKSPACE;
  if (!aligned(ws, 256)) return QLORA_ERR_UNSUPPORTED;
  qlora::Nf4Weight W{codes, absmax_q, absmax_s2};
  return hip_status(qlora::launch_bwd(dY, X, T, W, A, B, M, N, K, r, scale, dX, dA, dB, ws,
                                      reinterpret_cast<hipStream_t>(stream), nullptr, nullptr,
                                      dr));
}

int64_t qlora_act8_row_bytes(int64_t K) { return K < 0 ? -1 : qlora::act8_row_bytes(K); }
int64_t qlora_act8_scale_row_bytes(int64_t K) {
  return K < 0 ? -1 : qlora::act8_scale_row_bytes(K);
}

int qlora_act8_quantize(const uint16_t* X, int64_t M, int64_t K, int64_t ldx, int32_t fmt,
                        uint8_t* codes, uint8_t* scales, void* stream) {
  if (!X || !valid_fmt(fmt)) return QLORA_ERR_INVALID_ARG;
  int st = check_act8_shape(M, K);
  if (st != QLORA_OK) return st;
  if (ldx < K) return QLORA_ERR_INVALID_ARG;
  st = check_act8(codes, scales);
  if (st != QLORA_OK) return st;
  if (!aligned(X, 2)) return QLORA_ERR_UNSUPPORTED;
  return hip_status(qlora::launch_act8_quantize(X, M, K, ldx, fmt, codes, scales,
                                                reinterpret_cast<hipStream_t>(stream)));
}

int qlora_act8_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t M, int64_t K,
                          int32_t fmt, uint16_t* X, int64_t ldx, void* stream) {
  if (!X || !valid_fmt(fmt)) return QLORA_ERR_INVALID_ARG;
  int st = check_act8_shape(M, K);
  if (st != QLORA_OK) return st;
  if (ldx < K) return QLORA_ERR_INVALID_ARG;
  st = check_act8(codes, scales);
  if (st != QLORA_OK) return st;
  if (!aligned(X, 2)) return QLORA_ERR_UNSUPPORTED;
  return hip_status(qlora::launch_act8_dequantize(codes, scales, M, K, fmt, X, ldx,
                                                  reinterpret_cast<hipStream_t>(stream)));
}

int qlora_swiglu_act8_fwd(const uint16_t* G, int64_t ldg, const uint16_t* U, int64_t ldu, int64_t M,
                          int64_t F, int32_t fmt, uint16_t* H, int64_t ldh, uint8_t* h_codes,
                          uint8_t* h_scales, uint8_t* g_codes, uint8_t* g_scales, uint8_t* u_codes,
                          uint8_t* u_scales, void* stream) {
  if (!G || !U || !valid_fmt(fmt)) return QLORA_ERR_INVALID_ARG;
  int st = check_act8_shape(M, F);
  if (st != QLORA_OK) return st;
  if (ldg < F || ldu < F || (H && ldh < F)) return QLORA_ERR_INVALID_ARG;
  // each 8-bit output comes whole or not at all, and there is some output
  const uint8_t* pairs[3][2] = {{h_codes, h_scales}, {g_codes, g_scales}, {u_codes, u_scales}};
  bool any = H != nullptr;
  for (const auto& p : pairs) {
    if (!p[0] && !p[1]) continue;
    st = check_act8(p[0], p[1]);
    if (st != QLORA_OK) return st;
    any = true;
  }
  if (!any) return QLORA_ERR_INVALID_ARG;
  if (!aligned(G, 2) || !aligned(U, 2) || !aligned(H, 2)) return QLORA_ERR_UNSUPPORTED;
  return hip_status(qlora::launch_swiglu_act8_fwd(
      G, ldg, U, ldu, M, F, fmt, H, ldh, qlora::Act8{h_codes, h_scales},
      qlora::Act8{g_codes, g_scales}, qlora::Act8{u_codes, u_scales},
      reinterpret_cast<hipStream_t>(stream)));
}

int qlora_swiglu_act8_bwd(const uint16_t* dH, int64_t lddh, const uint8_t* g_codes,
                          const uint8_t* g_scales, const uint8_t* u_codes, const uint8_t* u_scales,
                          int64_t M, int64_t F, int32_t fmt, uint16_t* dG, int64_t lddg,
                          uint16_t* dU, int64_t lddu, void* stream) {
  if (!dH || !dG || !dU || !valid_fmt(fmt)) return QLORA_ERR_INVALID_ARG;
  int st = check_act8_shape(M, F);
  if (st != QLORA_OK) return st;
  if (lddh < F || lddg < F || lddu < F) return QLORA_ERR_INVALID_ARG;
  st = check_act8(g_codes, g_scales);
  if (st == QLORA_OK) st = check_act8(u_codes, u_scales);
  if (st != QLORA_OK) return st;
  if (!aligned(dH, 2) || !aligned(dG, 2) || !aligned(dU, 2)) return QLORA_ERR_UNSUPPORTED;
  return hip_status(qlora::launch_swiglu_act8_bwd(
      dH, lddh, qlora::ConstAct8{g_codes, g_scales}, qlora::ConstAct8{u_codes, u_scales}, M, F, fmt,
      dG, lddg, dU, lddu, reinterpret_cast<hipStream_t>(stream)));
}

int qlora_fp8_weight_quantize(const uint16_t* W, int64_t N, int64_t K, uint8_t* codes,
                              uint8_t* scales, uint8_t* codes_t, uint8_t* scales_t, void* stream) {
  if (!W || N <= 0 || K <= 0) return QLORA_ERR_INVALID_ARG;
  if (N > (int64_t)1 << 21 || K > (int64_t)1 << 21 ||
      (N + 127) / 128 * ((K + 127) / 128) >= (int64_t)1 << 18)
    return QLORA_ERR_UNSUPPORTED;
  int st = check_act8(codes, scales);
  if (st == QLORA_OK && (codes_t || scales_t)) st = check_act8(codes_t, scales_t);
  if (st != QLORA_OK) return st;
  if (!aligned(W, 2)) return QLORA_ERR_UNSUPPORTED;
  return hip_status(qlora::launch_fp8_weight_quantize(W, N, K, qlora::Act8{codes, scales},
                                                      qlora::Act8{codes_t, scales_t},
                                                      reinterpret_cast<hipStream_t>(stream)));
}

size_t qlora_act8_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t r) {
  if (check_fp8_shape(M, N, K, r) != QLORA_OK) return 0;
  return qlora::act8_workspace_bytes(M, N, K, r, qlora::Act8Ws::kWeight);
}

size_t qlora_fp8_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t r, int32_t backward) {
  if (check_fp8_shape(M, N, K, r) != QLORA_OK) return 0;
  return qlora::act8_workspace_bytes(M, N, K, r, backward ? qlora::Act8Ws::kDy8 : qlora::Act8Ws::kFactors);
}

static int check_act8_ws(int64_t M, int64_t N, int64_t K, int32_t r, qlora::Act8Ws what, const void* ws,
                         size_t ws_bytes) {
  if (!ws || ws_bytes < qlora::act8_workspace_bytes(M, N, K, r, what)) return QLORA_ERR_WORKSPACE;
  return aligned(ws, 256) ? QLORA_OK : QLORA_ERR_UNSUPPORTED;
}

int qlora_linear_bwd_act8(const uint16_t* dY, const uint8_t* x_codes, const uint8_t* x_scales,
                          int32_t fmt, const float* T, const uint8_t* codes,
                          const uint8_t* absmax_q, const float* absmax_s2, const uint16_t* A,
                          const uint16_t* B, int64_t M, int64_t N, int64_t K, int32_t r,
                          float scale, const uint32_t* keep_mask, float p, uint16_t* dX, float* dA,
                          float* dB, void* ws, size_t ws_bytes, int32_t store_type, void* stream) {
  if (!dY || !A || !B || !dA || !dB || !valid_fmt(fmt)) return QLORA_ERR_INVALID_ARG;
  if (!valid_store_type(store_type)) return QLORA_ERR_INVALID_ARG;
  int st = check_act8(x_codes, x_scales);
  // the weight is read for dX only
  if (st == QLORA_OK && dX) st = check_store(codes, absmax_q, absmax_s2);
  if (st == QLORA_OK && M > 0 && N > 0 && K > 0 && r == 0) st = QLORA_ERR_UNSUPPORTED;
  if (st == QLORA_OK) st = check_fp8_shape(M, N, K, r);
  if (st != QLORA_OK) return st;
  qlora::Dropout dr;
  if (keep_mask) {
    st = check_dropout(keep_mask, p, &dr);
    if (st != QLORA_OK) return st;
    if (dX && r > QLORA_MAX_DROPOUT_RANK) return QLORA_ERR_UNSUPPORTED;
  }
  if (!aligned(dY, 16) || !aligned(B, 16) || !aligned(A, 2) || (T && !aligned(T, 4)) ||
      (dX && !aligned(dX, 2)) || !aligned(dA, 4) || !aligned(dB, 4))
    return QLORA_ERR_UNSUPPORTED;
  st = check_act8_ws(M, N, K, r, dX ? qlora::Act8Ws::kWeight : qlora::Act8Ws::kFactors, ws, ws_bytes);
  if (st != QLORA_OK) return st;
  qlora::Nf4Weight W{codes, absmax_q, absmax_s2, store_type};
  return hip_status(qlora::launch_bwd_act8(dY, qlora::ConstAct8{x_codes, x_scales}, fmt, T, W, A, B,
                                           M, N, K, r, scale, dX, dA, dB, ws,
                                           reinterpret_cast<hipStream_t>(stream), dr));
}

int qlora_fp8_linear_fwd(const uint8_t* x_codes, const uint8_t* x_scales, int32_t fmt,
                         const uint8_t* w_codes, const uint8_t* w_scales, const uint16_t* A,
                         const uint16_t* B, int64_t M, int64_t N, int64_t K, int32_t r, float scale,
                         uint16_t* Y, float* T_out, void* ws, size_t ws_bytes, void* stream) {
  if (!Y || !valid_fmt(fmt)) return QLORA_ERR_INVALID_ARG;
  if (r ? (!A || !B) : (A || B || T_out)) return QLORA_ERR_INVALID_ARG;
  int st = check_act8(x_codes, x_scales);
  if (st == QLORA_OK) st = check_act8(w_codes, w_scales);
  if (st == QLORA_OK) st = check_fp8_shape(M, N, K, r);
  if (st != QLORA_OK) return st;
  if (!aligned(B, 16) || !aligned(A, 2) || !aligned(Y, 2) || !aligned(T_out, 4))
    return QLORA_ERR_UNSUPPORTED;
  st = check_act8_ws(M, N, K, r, qlora::Act8Ws::kFactors, ws, ws_bytes);
  if (st != QLORA_OK) return st;
  return hip_status(qlora::launch_fp8_fwd(qlora::ConstAct8{x_codes, x_scales}, fmt,
                                          qlora::ConstAct8{w_codes, w_scales}, A, B, M, N, K, r,
                                          scale, Y, T_out, ws,
                                          reinterpret_cast<hipStream_t>(stream)));
}

int qlora_fp8_linear_bwd(const uint16_t* dY, int32_t dy_fmt, const uint8_t* x_codes,
                         const uint8_t* x_scales, int32_t fmt, const float* T,
                         const uint8_t* w_codes_t, const uint8_t* w_scales_t, const uint16_t* A,
                         const uint16_t* B, int64_t M, int64_t N, int64_t K, int32_t r, float scale,
                         uint16_t* dX, float* dA, float* dB, void* ws, size_t ws_bytes,
                         void* stream) {
  if (!dY || !valid_fmt(fmt) || !valid_fmt(dy_fmt)) return QLORA_ERR_INVALID_ARG;
  if (r ? (!A || !B || !dA || !dB) : (A || B || T || dA || dB || !dX)) return QLORA_ERR_INVALID_ARG;
  int st = r ? check_act8(x_codes, x_scales) : QLORA_OK;
  if (st == QLORA_OK && dX) st = check_act8(w_codes_t, w_scales_t);
  if (st == QLORA_OK) st = check_fp8_shape(M, N, K, r);
  if (st != QLORA_OK) return st;
  if (!aligned(dY, r ? 16 : 2) || !aligned(B, 16) || !aligned(A, 2) || !aligned(T, 4) ||
      !aligned(dX, 2) || !aligned(dA, 4) || !aligned(dB, 4))
    return QLORA_ERR_UNSUPPORTED;
  st = check_act8_ws(M, N, K, r, dX ? qlora::Act8Ws::kDy8 : qlora::Act8Ws::kFactors, ws, ws_bytes);
  if (st != QLORA_OK) return st;
  return hip_status(qlora::launch_fp8_bwd(dY, dy_fmt, qlora::ConstAct8{x_codes, x_scales}, fmt, T,
                                          qlora::ConstAct8{w_codes_t, w_scales_t}, A, B, M, N, K, r,
                                          scale, dX, dA, dB, ws,
                                          reinterpret_cast<hipStream_t>(stream)));
}

int qlora_int4_quantize(const uint16_t* W, int64_t N, int64_t K, int64_t ldw, int32_t group,
                        uint8_t* codes, uint16_t* scales, uint8_t* zeros, void* stream) {
  if (!W || ldw < K) return QLORA_ERR_INVALID_ARG;
  const int st = check_int4(codes, scales, N, K, group);
  if (st != QLORA_OK) return st;
  if (!aligned(W, 2) || ldw > (int64_t)1 << 32) return QLORA_ERR_UNSUPPORTED;
  return hip_status(qlora::launch_int4_quantize(W, N, K, ldw, group, codes, scales, zeros,
                                                reinterpret_cast<hipStream_t>(stream)));
}

int qlora_int4_dequantize(const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros,
                          int64_t N, int64_t K, int32_t group, uint16_t* W, int64_t ldw,
                          void* stream) {
  if (!W || ldw < K) return QLORA_ERR_INVALID_ARG;
  const int st = check_int4(codes, scales, N, K, group);
  if (st != QLORA_OK) return st;
  if (!aligned(W, 2) || ldw > (int64_t)1 << 32) return QLORA_ERR_UNSUPPORTED;
  return hip_status(qlora::launch_int4_dequantize(qlora::Int4Weight{codes, scales, zeros, N, K, group}, W,
                                                  ldw, reinterpret_cast<hipStream_t>(stream)));
}

int qlora_int4_linear_fwd(const uint16_t* X, int64_t M, int64_t ldx, const uint8_t* codes,
                          const uint16_t* scales, const uint8_t* zeros, int64_t N, int64_t K,
                          int32_t group, void* Y, int32_t y_dtype, int64_t ldy, void* stream) {
  if (!X || !Y || M <= 0 || ldx < K || ldy < N) return QLORA_ERR_INVALID_ARG;
  if (y_dtype != QLORA_LOGITS_BF16 && y_dtype != QLORA_LOGITS_F32) return QLORA_ERR_INVALID_ARG;
  const int st = check_int4(codes, scales, N, K, group);
  if (st != QLORA_OK) return st;
  // 32-bit offsets into X; a token tile per row of the grid
  if (M > (int64_t)1 << 20 || ldx >= (int64_t)1 << 30 || M * ldx >= (int64_t)1 << 30 || ldx % 8 ||
      ldy > (int64_t)1 << 32)
    return QLORA_ERR_UNSUPPORTED;
  if (!aligned(X, 16) || !aligned(Y, y_dtype == QLORA_LOGITS_F32 ? 4 : 2)) return QLORA_ERR_UNSUPPORTED;
  return hip_status(qlora::launch_int4_linear_fwd(X, M, ldx, qlora::Int4Weight{codes, scales, zeros, N, K, group},
                                                  Y, y_dtype == QLORA_LOGITS_F32, ldy,
                                                  reinterpret_cast<hipStream_t>(stream)));
}

size_t qlora_logits_workspace_bytes(int64_t T, int64_t V, int32_t n_top) {
  if (T <= 0 || V <= 0 || T > (int64_t)1 << 23 || V > (int64_t)1 << 21) return 0;
  if (n_top < 0 || n_top > QLORA_MAX_TOP_LOGITS || n_top > V) return 0;
  return qlora::logits_workspace_bytes(T, V, n_top);
}

int qlora_logprobs_fwd(const void* Z, int32_t dtype, int64_t T, int64_t V, int64_t ldz,
                       const int64_t* target, double temperature, float* logp, float* entropy,
                       int32_t n_top, int64_t* top_ids, float* top_logp, float* stats, void* ws,
                       size_t ws_bytes, void* stream) {
  qlora::Logits z;
  int st = check_logits(Z, dtype, T, V, ldz, temperature, &z);
  if (st != QLORA_OK) return st;
  if (logp && !target) return QLORA_ERR_INVALID_ARG;
  if (n_top < 0 || n_top > V || (n_top ? !top_ids || !top_logp : top_ids || top_logp)) return QLORA_ERR_INVALID_ARG;
  if (!logp && !entropy && !n_top && !stats) return QLORA_ERR_INVALID_ARG;
  if (n_top > QLORA_MAX_TOP_LOGITS) return QLORA_ERR_UNSUPPORTED;
  if (!aligned(target, 8) || !aligned(top_ids, 8) || !aligned(logp, 4) || !aligned(entropy, 4) ||
      !aligned(top_logp, 4) || !aligned(stats, 4))
    return QLORA_ERR_UNSUPPORTED;
  st = check_logits_ws(z, n_top, ws, ws_bytes);
  if (st != QLORA_OK) return st;
  return hip_status(qlora::launch_logprobs_fwd(z, target, logp, entropy, n_top, top_ids, top_logp, stats, ws,
                                               reinterpret_cast<hipStream_t>(stream)));
}

int qlora_logprobs_bwd(const void* Z, int32_t dtype, int64_t T, int64_t V, int64_t ldz,
                       const int64_t* target, double temperature, const float* stats,
                       const float* g_logp, const float* g_entropy, void* dZ, int64_t lddz,
                       void* stream) {
  qlora::Logits z;
  int st = check_logits(Z, dtype, T, V, ldz, temperature, &z);
  if (st == QLORA_OK) st = check_dlogits(dZ, lddz, z);
  if (st != QLORA_OK) return st;
  if (!stats || (!g_logp && !g_entropy) || (g_logp && !target)) return QLORA_ERR_INVALID_ARG;
  if (!aligned(target, 8) || !aligned(stats, 4) || !aligned(g_logp, 4) || !aligned(g_entropy, 4))
    return QLORA_ERR_UNSUPPORTED;
  return hip_status(qlora::launch_logprobs_bwd(z, target, stats, g_logp, g_entropy, dZ, lddz,
                                               reinterpret_cast<hipStream_t>(stream)));
}

int qlora_distill_fwd(const void* Z, int32_t dtype, int64_t T, int64_t V, int64_t ldz,
                      const int64_t* ids, const void* values, int32_t values_dtype, int32_t k,
                      const float* teacher_lse, double temperature, float* loss, float* stats,
                      void* ws, size_t ws_bytes, void* stream) {
  qlora::Logits z;
  qlora::TopLogits t;
  int st = check_logits(Z, dtype, T, V, ldz, temperature, &z);
  if (st == QLORA_OK) st = check_top_logits(ids, values, values_dtype, k, &t);
  if (st != QLORA_OK) return st;
  if (!loss) return QLORA_ERR_INVALID_ARG;
  if (!aligned(teacher_lse, 4) || !aligned(loss, 4) || !aligned(stats, 4)) return QLORA_ERR_UNSUPPORTED;
  st = check_logits_ws(z, 0, ws, ws_bytes);
  if (st != QLORA_OK) return st;
  return hip_status(qlora::launch_distill_fwd(z, t, teacher_lse, loss, stats, ws,
                                              reinterpret_cast<hipStream_t>(stream)));
}

int qlora_distill_bwd(const void* Z, int32_t dtype, int64_t T, int64_t V, int64_t ldz,
                      const int64_t* ids, const void* values, int32_t values_dtype, int32_t k,
                      double temperature, const float* stats, const float* g, void* dZ,
                      int64_t lddz, void* stream) {
  qlora::Logits z;
  qlora::TopLogits t;
  int st = check_logits(Z, dtype, T, V, ldz, temperature, &z);
  if (st == QLORA_OK) st = check_top_logits(ids, values, values_dtype, k, &t);
  if (st == QLORA_OK) st = check_dlogits(dZ, lddz, z);
  if (st != QLORA_OK) return st;
  if (!stats || !g) return QLORA_ERR_INVALID_ARG;
  if (!aligned(stats, 4) || !aligned(g, 4)) return QLORA_ERR_UNSUPPORTED;
  return hip_status(qlora::launch_distill_bwd(z, t, stats, g, dZ, lddz, reinterpret_cast<hipStream_t>(stream)));
}

int qlora_gemv_wait_limit(int64_t microseconds) {
  if (microseconds < 0 || microseconds > 1000000) return QLORA_ERR_INVALID_ARG;
  qlora::set_gemv_wait_us(microseconds);
  return QLORA_OK;
}

const char* qlora_status_string(int status) {
  switch (status) {
    case QLORA_OK: return "ok";
    case QLORA_ERR_INVALID_ARG: return "invalid argument";
    case QLORA_ERR_UNSUPPORTED: return "unsupported shape, rank or alignment";
    case QLORA_ERR_WORKSPACE: return "workspace missing or too small";
    case QLORA_ERR_HIP: return "HIP launch failed";
    default: return "unknown status";
  }
}

int qlora_last_hip_error(void) { return g_last_hip_error; }

}  // extern "C"
