// The 8-bit block format: quantization and decoding of activation rows (one
// scale per 1 x 128), quantization of a weight (one scale per 128 x 128, in
// both orders), and the SwiGLU activation that writes and reads its
// checkpoints in it.
//
// Sixteen lanes own one block of 128: eight values per lane (one 16-byte
// load), the block maximum over one DPP row of 16 lanes. Blocks are taken in
// flat order b = row * ceil(K/128) + column block, so that a wave's codes
// are 512 consecutive bytes whatever K is.
//
// All of them pass over memory once with a few operations per value and are
// bound by it. At 2048 x 11008 (kernel time; a copy of 512 MiB reaches 5.3 TB/s):
//   quantize    13.0 us   68 MB  5.2 TB/s
//   dequantize  11.7 us   68 MB  5.8 TB/s
//   SwiGLU      41.4 us  203 MB  4.9 TB/s (H and three sets of blocks)
//   its backward  29.2 us  181 MB  6.2 TB/s
// and a weight of 11008 x 4096 in both orders takes 40 us (180 MB, 4.5 TB/s).
// Small calls (16 x 4096) take 2.4 us, a launch's own time.
#include "act8.h"
#include "kernels.h"

#include <algorithm>

namespace qlora {

namespace {

constexpr int kThreads = 256;
constexpr int kGroups = kThreads / 16;  // blocks per workgroup

template <int kFmt, bool kVec>
__global__ void __launch_bounds__(kThreads)
act8_quantize_kernel(const uint16_t* __restrict__ X, int64_t ldx, int64_t K, uint32_t blocks, int KB,
                     int sb, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  const uint32_t b = blockIdx.x * kGroups + (threadIdx.x >> 4);
  if (b < blocks) act8_quantize_block<kFmt, kVec>(X, ldx, K, b, KB, sb, codes, scales);
}

template <int kFmt, bool kVec>
__global__ void __launch_bounds__(kThreads)
act8_dequantize_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                       int64_t K, uint32_t blocks, int KB, int sb, uint16_t* __restrict__ X,
                       int64_t ldx) {
  const uint32_t b = blockIdx.x * kGroups + (threadIdx.x >> 4);
  if (b >= blocks) return;
  const uint32_t row = b / (uint32_t)KB;
  const int kb = (int)(b - row * (uint32_t)KB);
  const int l = threadIdx.x & 15;
  const u32x2 c = *reinterpret_cast<const u32x2*>(codes + (int64_t)b * kAct8Block + l * 8);
  const float s = act8_scale(scales[(int64_t)row * sb + kb]);
  store8<kVec>(X + (int64_t)row * ldx, (int64_t)kb * kAct8Block + l * 8, K, act8_decode8<kFmt>(c, s));
}

// ---------------------------------------------------------------------------
// SwiGLU: h = g s(g) u with s(g) = 1 / (1 + exp(-g)).

__device__ __forceinline__ float sigmoid(float g) { return 1.0f / (1.0f + __expf(-g)); }

struct SwigluFwd {
  const uint16_t *g, *u;
  int64_t ldg, ldu;
  uint16_t* h;  // or null
  int64_t ldh;
  uint8_t *h8, *hs, *g8, *gs, *u8, *us;  // each pair may be null
  int64_t F;
  uint32_t blocks;
  int KB, sb;
};

template <int kFmt, bool kVec>
__global__ void __launch_bounds__(kThreads) swiglu_act8_fwd_kernel(SwigluFwd p) {
  const uint32_t b = blockIdx.x * kGroups + (threadIdx.x >> 4);
  if (b >= p.blocks) return;
  const uint32_t row = b / (uint32_t)p.KB;
  const int kb = (int)(b - row * (uint32_t)p.KB);
  const int64_t c = (int64_t)kb * kAct8Block + (threadIdx.x & 15) * 8;
  const u32x4 g = load8<kVec>(p.g + (int64_t)row * p.ldg, c, p.F);
  const u32x4 u = load8<kVec>(p.u + (int64_t)row * p.ldu, c, p.F);
  u32x4 h;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float g0 = bf16_lo(g[i]), g1 = bf16_hi(g[i]);
    h[i] = pack_bf16x2(g0 * sigmoid(g0) * bf16_lo(u[i]), g1 * sigmoid(g1) * bf16_hi(u[i]));
  }
  if (p.h) store8<kVec>(p.h + (int64_t)row * p.ldh, c, p.F, h);
  if (p.h8) put_block<kFmt>(h, b, kb, p.KB, p.sb, row, p.h8, p.hs);
  if (p.g8) put_block<kFmt>(g, b, kb, p.KB, p.sb, row, p.g8, p.gs);
  if (p.u8) put_block<kFmt>(u, b, kb, p.KB, p.sb, row, p.u8, p.us);
}

struct SwigluBwd {
  const uint16_t* dh;
  int64_t lddh;
  const uint8_t *g8, *gs, *u8, *us;
  uint16_t *dg, *du;
  int64_t lddg, lddu, F;
  uint32_t blocks;
  int KB, sb;
};

// dg = dh u s (1 + g (1 - s)),  du = dh g s
template <int kFmt, bool kVec>
__global__ void __launch_bounds__(kThreads) swiglu_act8_bwd_kernel(SwigluBwd p) {
  const uint32_t b = blockIdx.x * kGroups + (threadIdx.x >> 4);
  if (b >= p.blocks) return;
  const uint32_t row = b / (uint32_t)p.KB;
  const int kb = (int)(b - row * (uint32_t)p.KB);
  const int l = threadIdx.x & 15;
  const int64_t c = (int64_t)kb * kAct8Block + l * 8;
  const int64_t at = (int64_t)b * kAct8Block + l * 8;
  const u32x4 dh = load8<kVec>(p.dh + (int64_t)row * p.lddh, c, p.F);
  const u32x4 g = act8_decode8<kFmt>(*reinterpret_cast<const u32x2*>(p.g8 + at),
                                     act8_scale(p.gs[(int64_t)row * p.sb + kb]));
  const u32x4 u = act8_decode8<kFmt>(*reinterpret_cast<const u32x2*>(p.u8 + at),
                                     act8_scale(p.us[(int64_t)row * p.sb + kb]));
  u32x4 dg, du;
  auto one = [](float d, float gg, float uu, float& og, float& ou) {
    const float s = sigmoid(gg);
    og = d * uu * (s * (1.0f + gg * (1.0f - s)));
    ou = d * (gg * s);
  };
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a0, a1, b0, b1;
    one(bf16_lo(dh[i]), bf16_lo(g[i]), bf16_lo(u[i]), a0, b0);
    one(bf16_hi(dh[i]), bf16_hi(g[i]), bf16_hi(u[i]), a1, b1);
    dg[i] = pack_bf16x2(a0, a1);
    du[i] = pack_bf16x2(b0, b1);
  }
  store8<kVec>(p.dg + (int64_t)row * p.lddg, c, p.F, dg);
  store8<kVec>(p.du + (int64_t)row * p.lddu, c, p.F, du);
}

// ---------------------------------------------------------------------------
// Weight quantization: one 128 x 128 block per workgroup; the codes in row
// order and, through LDS, in column order.
__global__ void __launch_bounds__(kThreads)
fp8_weight_quantize_kernel(const uint16_t* __restrict__ W, int64_t N, int64_t K,
                           uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                           uint8_t* __restrict__ codes_t, uint8_t* __restrict__ scales_t,
                           bool vec) {
  constexpr int kPitch = 132;  // bytes per LDS row: the column reads fall on distinct banks
  __shared__ uint32_t s_tile[128 * kPitch / 4];
  __shared__ uint32_t s_max[4];
  uint8_t* tile = reinterpret_cast<uint8_t*>(s_tile);
  const int KB = (int)((K + 127) / 128), NB = (int)((N + 127) / 128);
  const int kb = (int)(blockIdx.x % (unsigned)KB), nb = (int)(blockIdx.x / (unsigned)KB);
  const int t = threadIdx.x, l = t & 15, g = t >> 4;
  const int64_t c = (int64_t)kb * 128 + l * 8;
  u32x4 x[8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t n = (int64_t)nb * 128 + i * 16 + g;
    x[i] = u32x4{0u, 0u, 0u, 0u};
    if (n < N) x[i] = vec ? load8<true>(W + n * K, c, K) : load8<false>(W + n * K, c, K);
    m = max(m, finite_max8(x[i]));
  }
  m = row16_max(m);
  m = max(m, (uint32_t)__shfl_xor((int)m, 16));
  m = max(m, (uint32_t)__shfl_xor((int)m, 32));
  if ((t & 63) == 0) s_max[t >> 6] = m;
  __syncthreads();
  m = max(max(s_max[0], s_max[1]), max(s_max[2], s_max[3]));
  const int byte = act8_scale_byte<0>(m);
  const float s = act8_scale(byte);
  const int64_t Kp = act8_row_bytes(K), Np = act8_row_bytes(N);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = i * 16 + g;
    const int64_t n = (int64_t)nb * 128 + row;
    const u32x2 q = act8_encode8<0>(x[i], s);
    if (n < N) *reinterpret_cast<u32x2*>(codes + n * Kp + c) = q;
    s_tile[(row * kPitch + l * 8) / 4] = q[0];
    s_tile[(row * kPitch + l * 8) / 4 + 1] = q[1];
  }
  if (t == 0) {
    const int sb = (int)act8_scale_row_bytes(K);
    put_scale(scales + (int64_t)nb * sb, kb, KB, sb, byte);
  }
  if (!codes_t) return;
  __syncthreads();
  if (t == 0) {
    const int sb = (int)act8_scale_row_bytes(N);
    put_scale(scales_t + (int64_t)kb * sb, nb, NB, sb, byte);
  }
  // output row k (a source column), 16 source rows per store
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int id = t + i * kThreads;
    const int col = id & 127, part = id >> 7;
    const int64_t k = (int64_t)kb * 128 + col;
    u32x4 o;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t w = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w |= (uint32_t)tile[(part * 16 + j * 4 + e) * kPitch + col] << (8 * e);
      o[j] = w;
    }
    if (k < K) *reinterpret_cast<u32x4*>(codes_t + k * Np + (int64_t)nb * 128 + part * 16) = o;
  }
}

bool vec16(const void* p, int64_t ld) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % 8 == 0;
}

}  // namespace

hipError_t launch_act8_quantize(const uint16_t* X, int64_t M, int64_t K, int64_t ldx, int fmt,
                                uint8_t* codes, uint8_t* scales, hipStream_t stream) {
  const int KB = (int)((K + kAct8Block - 1) / kAct8Block);
  const uint32_t blocks = (uint32_t)(M * KB);
  const dim3 grid((blocks + kGroups - 1) / kGroups), block(kThreads);
  const int sb = (int)act8_scale_row_bytes(K);
  auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, grid, block, 0, stream, X, ldx, K, blocks, KB, sb, codes, scales);
    return hipGetLastError();
  };
  if (vec16(X, ldx)) return fmt ? go(act8_quantize_kernel<1, true>) : go(act8_quantize_kernel<0, true>);
  return fmt ? go(act8_quantize_kernel<1, false>) : go(act8_quantize_kernel<0, false>);
}

hipError_t launch_act8_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t M, int64_t K,
                                  int fmt, uint16_t* X, int64_t ldx, hipStream_t stream) {
  const int KB = (int)((K + kAct8Block - 1) / kAct8Block);
  const uint32_t blocks = (uint32_t)(M * KB);
  const dim3 grid((blocks + kGroups - 1) / kGroups), block(kThreads);
  const int sb = (int)act8_scale_row_bytes(K);
  auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, grid, block, 0, stream, codes, scales, K, blocks, KB, sb, X, ldx);
    return hipGetLastError();
  };
  if (vec16(X, ldx)) return fmt ? go(act8_dequantize_kernel<1, true>) : go(act8_dequantize_kernel<0, true>);
  return fmt ? go(act8_dequantize_kernel<1, false>) : go(act8_dequantize_kernel<0, false>);
}

hipError_t launch_swiglu_act8_fwd(const uint16_t* g, int64_t ldg, const uint16_t* u, int64_t ldu,
                                  int64_t M, int64_t F, int fmt, uint16_t* h, int64_t ldh, Act8 h8,
                                  Act8 g8, Act8 u8, hipStream_t stream) {
  SwigluFwd p{g, u, ldg, ldu, h, ldh, h8.codes, h8.scales, g8.codes, g8.scales, u8.codes, u8.scales,
              F, 0, (int)((F + kAct8Block - 1) / kAct8Block), (int)act8_scale_row_bytes(F)};
  p.blocks = (uint32_t)(M * p.KB);
  const dim3 grid((p.blocks + kGroups - 1) / kGroups), block(kThreads);
  auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, grid, block, 0, stream, p);
    return hipGetLastError();
  };
  if (vec16(g, ldg) && vec16(u, ldu) && (!h || vec16(h, ldh)))
    return fmt ? go(swiglu_act8_fwd_kernel<1, true>) : go(swiglu_act8_fwd_kernel<0, true>);
  return fmt ? go(swiglu_act8_fwd_kernel<1, false>) : go(swiglu_act8_fwd_kernel<0, false>);
}

hipError_t launch_swiglu_act8_bwd(const uint16_t* dh, int64_t lddh, ConstAct8 g8, ConstAct8 u8,
                                  int64_t M, int64_t F, int fmt, uint16_t* dg, int64_t lddg,
                                  uint16_t* du, int64_t lddu, hipStream_t stream) {
  SwigluBwd p{dh, lddh, g8.codes, g8.scales, u8.codes, u8.scales, dg, du, lddg, lddu,
              F, 0, (int)((F + kAct8Block - 1) / kAct8Block), (int)act8_scale_row_bytes(F)};
  p.blocks = (uint32_t)(M * p.KB);
  const dim3 grid((p.blocks + kGroups - 1) / kGroups), block(kThreads);
  auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, grid, block, 0, stream, p);
    return hipGetLastError();
  };
  if (vec16(dh, lddh) && vec16(dg, lddg) && vec16(du, lddu))
    return fmt ? go(swiglu_act8_bwd_kernel<1, true>) : go(swiglu_act8_bwd_kernel<0, true>);
  return fmt ? go(swiglu_act8_bwd_kernel<1, false>) : go(swiglu_act8_bwd_kernel<0, false>);
}

hipError_t launch_fp8_weight_quantize(const uint16_t* W, int64_t N, int64_t K, Act8 w8, Act8 w8t,
                                      hipStream_t stream) {
  const int64_t KB = (K + 127) / 128, NB = (N + 127) / 128;
  hipLaunchKernelGGL(fp8_weight_quantize_kernel, dim3((unsigned)(KB * NB)), dim3(kThreads), 0,
                     stream, W, N, K, w8.codes, w8.scales, w8t.codes, w8t.scales, vec16(W, K));
  return hipGetLastError();
}

}  // namespace qlora
