// The linear layer on 8-bit inputs: backward of the NF4 layer from an 8-bit
// copy of its input, and forward and backward of a frozen weight held in
// 8-bit blocks, both with a LoRA adapter beside it.
//
//   forward   T = dec(X8) A, split along K             row product
//             T (float32), bf16(s T), B^T padded       one launch
//             Y = dec(X8) dec(W8)^T + (s T) B          8-bit product
//             (few tokens: T, or its partials summed,  8-bit product
//             and s T in float32 there)
//   backward  G = dY B^T, split along N (a short N:    row product
//             in the next launch)
//             bf16(s G); float32 s G and s T; beside   one launch
//             them the weight to bf16 (NF4) or dY to
//             8 bits (8-bit weight)
//             dX                                       bf16 or 8-bit product
//             dA and dB                                column products, one launch
#include "lowrank8.h"

#include <algorithm>

namespace qlora {

namespace {

#define QLORA_TRY(x)                       \
  do {                                     \
    hipError_t e_ = (x);                   \
    if (e_ != hipSuccess) return e_;       \
  } while (0)

// dX of the NF4 layer: the weight decoded to bf16 once, transposed, beside the
// adapter's factors, and a bf16 product on it. The contraction that decodes
// tiles on their way in decodes each of them once per row tile (whole backward,
// r = 64: 80 us against 47 at 64 x 4096 x 4096, 616 against 506 at
// 4096 x 8192 x 8192; dX alone 9.1 us against 3.6 at 16 x 256 x 256).
struct Ws8 {
  int64_t r64;
  size_t v, u, g, t, part, done, dy8, dys, wt, total;
};

// Byte offsets in the workspace, 256-aligned. Each part grows with every
// size (the split partials by their bound of one workgroup per compute
// unit), so a workspace for a larger call serves a smaller one. What only
// some calls need is last, so that the others need not bring it.
Ws8 ws8_layout(int64_t M, int64_t N, int64_t K, int r, Act8Ws what) {
  Ws8 w{};
  w.r64 = ((int64_t)r + 63) / 64 * 64;
  const int64_t Mp = (M + 63) / 64 * 64;
  size_t off = 0;
  auto take = [&](int64_t bytes) { size_t o = off; off += ((size_t)bytes + 255) / 256 * 256; return o; };
  w.v = take(std::max(N, K) * w.r64 * 2);   // B^T or A, padded
  w.u = take(Mp * w.r64 * 2);               // bf16(s T) or bf16(s G)
  w.g = take(w.r64 * Mp * 4);               // s G and s T for dA and dB
  w.t = take(w.r64 * Mp * 4);
  // splits * M * columns: 256 tiles of 64 x 64 at most, or one split
  w.part = take(r ? std::max<int64_t>(256 * 64 * 64, Mp * w.r64) * 4 : 0);
  w.done = take(r ? kTileSums * 4 : 0);
  // the NF4 backward's decoded weight, in the place of the 8-bit dY
  w.wt = off;
  w.total = std::max<size_t>(off, 256);  // 0 is a rejected shape
  if (what == Act8Ws::kFactors) return w;
  w.dy8 = take(M * act8_row_bytes(N));
  w.dys = take(M * act8_scale_row_bytes(N));
  if (r && what == Act8Ws::kWeight) off = std::max(off, w.wt + (size_t)(N * K * 2));
  w.total = off;
  return w;
}

struct Ptrs {
  uint16_t *v, *u;
  float *g, *t, *part;
  uint8_t *dy8, *dys;
  uint16_t* wt;
  TileSums sums;
};
Ptrs carve(void* ws_, const Ws8& w) {
  char* ws = reinterpret_cast<char*>(ws_);
  auto at = [&](size_t o) { return reinterpret_cast<uint16_t*>(ws + o); };
  auto atf = [&](size_t o) { return reinterpret_cast<float*>(ws + o); };
  return Ptrs{at(w.v), at(w.u), atf(w.g), atf(w.t), atf(w.part),
              reinterpret_cast<uint8_t*>(ws + w.dy8), reinterpret_cast<uint8_t*>(ws + w.dys), at(w.wt),
              // the partials' place serves the product's tiles after them
              TileSums{reinterpret_cast<uint32_t*>(ws + w.done), atf(w.part)}};
}

// The adapter's rows serve as they are when they are whole 64-column tiles.
bool in_place(const uint16_t* A, int r) {
  return r % 64 == 0 && (reinterpret_cast<uintptr_t>(A) & 15) == 0;
}

// Whether G = dY B^T is formed where it is written out, in one launch less
// (whole 8-bit backward from a graph, us, so and with its own launch:
// 16 x 256 x 256 r = 8 10.3 and 12.9, 2048 x 512 x 2048 r = 64 33.0 and 37.6,
// 257 x 1024 x 1024 r = 64 22.0 and 23.0, 16 x 2048 x 1024 r = 64 28.6 and 21.4,
// 2048 x 1024 x 1024 r = 256 43.4 and 39.6).
bool factor_in_place(int64_t N, int r) { return N <= 1024 && r <= 64; }

// The adapter's part of a backward pass before dX: bf16(s G) in u, A padded
// in v (unless it serves as it is), float32 s G and s T for dA and dB.
hipError_t bwd_front(const uint16_t* dY, ConstAct8 x, int fmt, const float* T, const uint16_t* A,
                     const uint16_t* B, int64_t M, int64_t N, int64_t K, int r, float scale,
                     const Ptrs& w, const Dropout& dr, const LowrankBeside& beside, hipStream_t stream) {
  const float f = dr.mask ? dr.keep_scale : 1.0f;
  const int ldp = lowrank_cols(r);
  int splits = 0;
  if (!T) {  // recomputed from the 8-bit input
    QLORA_TRY(launch_rows_act8(x, fmt, M, K, dr.mask, A, r, w.part, &splits, stream));
    const LowrankOut t{w.part, nullptr, nullptr, 0, splits, ldp, f, nullptr, nullptr, w.t};
    QLORA_TRY(launch_lowrank_out(&t, 1, LowrankPad{}, M, r, scale, nullptr, stream));
  }
  const bool here = factor_in_place(N, r);
  if (!here) QLORA_TRY(launch_rows_bf16(dY, M, N, B, r, w.part, &splits, stream));
  const LowrankOut o[2] = {{here ? nullptr : w.part, here ? dY : nullptr, B, N, splits, ldp, f, nullptr, w.u, w.g},
                           {T, nullptr, nullptr, 0, 1, r, 1.0f, nullptr, nullptr, w.t}};
  const LowrankPad pad = in_place(A, r) ? LowrankPad{} : LowrankPad{A, false, K, w.v};
  return launch_lowrank_out(o, T ? 2 : 1, pad, M, r, scale, w.sums.done, stream, beside);
}

}  // namespace

size_t act8_workspace_bytes(int64_t M, int64_t N, int64_t K, int r, Act8Ws what) {
  return ws8_layout(M, N, K, r, what).total;
}

hipError_t launch_bwd_act8(const uint16_t* dY, ConstAct8 x, int fmt, const float* T, Nf4Weight W,
                           const uint16_t* A, const uint16_t* B, int64_t M, int64_t N, int64_t K,
                           int r, float scale, uint16_t* dX, float* dA, float* dB, void* ws,
                           hipStream_t stream, Dropout dr) {
  const Ws8 l = ws8_layout(M, N, K, r, dX ? Act8Ws::kWeight : Act8Ws::kFactors);
  const Ptrs w = carve(ws, l);
  LowrankBeside beside;
  if (dX) beside.W = W, beside.N = N, beside.K = K, beside.w = w.wt;
  QLORA_TRY(bwd_front(dY, x, fmt, T, A, B, M, N, K, r, scale, w, dr, beside, stream));
  const lr8::ColPair cols = lr8::column_pair(x, fmt, dr.mask, dY, w.g, w.t, M, N, K, r, dA, dB);
  return dX ? launch_bf16_gemm(dY, w.wt, M, K, N, w.u, in_place(A, r) ? A : w.v, (int)l.r64, dr.mask, dX,
                               w.sums, &cols, stream)
            : launch_columns(cols, stream);
}

hipError_t launch_fp8_fwd(ConstAct8 x, int fmt, ConstAct8 w8, const uint16_t* A, const uint16_t* B,
                          int64_t M, int64_t N, int64_t K, int r, float scale, uint16_t* Y,
                          float* T_out, void* ws, hipStream_t stream) {
  const Ws8 l = ws8_layout(M, N, K, r, Act8Ws::kFactors);
  const Ptrs w = carve(ws, l);
  const bool few = fp8_few(M, N);
  if (!r)
    return few ? launch_fp8_few(x, fmt, w8, M, N, K, nullptr, nullptr, 0, nullptr, 0, scale, Y, nullptr, stream)
               : launch_fp8_gemm(x, fmt, w8, M, N, K, nullptr, nullptr, 0, Y, TileSums{}, nullptr, stream);
  if (few && fp8_few_forms_t(A, M, K, r))
    return launch_fp8_few(x, fmt, w8, M, N, K, A, nullptr, 0, B, r, scale, Y, T_out, stream);
  int splits = 0;
  QLORA_TRY(launch_rows_act8(x, fmt, M, K, nullptr, A, r, w.part, &splits, stream));
  if (few)
    return launch_fp8_few(x, fmt, w8, M, N, K, nullptr, w.part, splits, B, r, scale, Y, T_out, stream);
  const LowrankOut t{w.part, nullptr, nullptr, 0, splits, lowrank_cols(r), 1.0f, T_out, w.u, nullptr};
  QLORA_TRY(launch_lowrank_out(&t, 1, LowrankPad{B, true, N, w.v}, M, r, scale, w.sums.done, stream));
  return launch_fp8_gemm(x, fmt, w8, M, N, K, w.u, w.v, (int)l.r64, Y, w.sums, nullptr, stream);
}

hipError_t launch_fp8_bwd(const uint16_t* dY, int dyfmt, ConstAct8 x, int fmt, const float* T,
                          ConstAct8 w8t, const uint16_t* A, const uint16_t* B, int64_t M, int64_t N,
                          int64_t K, int r, float scale, uint16_t* dX, float* dA, float* dB,
                          void* ws, hipStream_t stream) {
  const Ws8 l = ws8_layout(M, N, K, r, dX ? Act8Ws::kDy8 : Act8Ws::kFactors);
  const Ptrs w = carve(ws, l);
  const ConstAct8 dy8{w.dy8, w.dys};
  if (!r) {
    QLORA_TRY(launch_act8_quantize(dY, M, N, N, dyfmt, w.dy8, w.dys, stream));
    return launch_fp8_gemm(dy8, dyfmt, w8t, M, K, N, nullptr, nullptr, 0, dX, TileSums{}, nullptr, stream);
  }
  LowrankBeside beside;
  if (dX) beside.s = dY, beside.C = N, beside.fmt = dyfmt, beside.codes = w.dy8, beside.scales = w.dys;
  QLORA_TRY(bwd_front(dY, x, fmt, T, A, B, M, N, K, r, scale, w, Dropout{}, beside, stream));
  const lr8::ColPair cols = lr8::column_pair(x, fmt, nullptr, dY, w.g, w.t, M, N, K, r, dA, dB);
  return dX ? launch_fp8_gemm(dy8, dyfmt, w8t, M, K, N, w.u, in_place(A, r) ? A : w.v, (int)l.r64, dX,
                              w.sums, &cols, stream)
            : launch_columns(cols, stream);
}

}  // namespace qlora
