// Product of two matrices in the 8-bit block format, on gfx950's scaled
// matrix instructions:
//
//   Y[m][n] = sum_b 2^(ex[m][b] + ew[n/128][b]) sum_{k in b} x[m][k] w[n][k]
//             + sum_j U[m][j] V[n][j]
//
// v_mfma_scale_f32_32x32x64_f8f6f4 takes the two scale bytes beside the
// operands and applies their product to its sum, so the block scales cost no
// vector arithmetic and no extra accumulator. Inside one block the order of
// the 128 products is free, which lets each lane take whole 16-byte pieces.
#include "act8.h"
#include "gemm.h"
#include "kernels.h"

#include <algorithm>
#include <atomic>

namespace qlora {

namespace fp8 {

typedef int i32x8 __attribute__((ext_vector_type(8)));

struct Fp8Gemm {
  const uint8_t *x, *xs, *w, *ws;
  int64_t M, N, ldc;   // ldc: bytes of a row of codes (both operands)
  int KB, sb;          // blocks along K, bytes of a row of scales
  const uint16_t *U, *V;  // bf16 [M x r64], [N x r64], or null
  int r64;
  uint16_t* Y;         // [M x N]
  int nM, nN;
};

// 128-byte LDS rows, the 16-byte piece c of row r at position c ^ swz(r).
using gemm::lds_u32x4;
using gemm::lds_void;
using gemm::make_rsrc;
using gemm::tile_off;
using gemm::wait_vmcnt;

template <int kSel, int kXFmt>
__device__ __forceinline__ floatx16 mma(i32x8 w, i32x8 x, floatx16 c, uint32_t sw, uint32_t sx) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, x, c, 0, kXFmt, kSel, (int)sw, kSel,
                                                         (int)sx);
}

// Tile of TN weight rows by TM activation rows; each wave WN x WM of it.
template <int TN, int TM, int WN, int WM, int kXFmt>
__global__ void __launch_bounds__((TN / WN) * (TM / WM) * 64) fp8_gemm_kernel(Fp8Gemm p) {
#ifdef __HIP_DEVICE_COMPILE__  // the host pass needs the stub alone
  constexpr int kWaves = (TN / WN) * (TM / WM);
  constexpr int BN = WN / 32, BM = WM / 32;
  constexpr int kStage = (TN + TM) * 128;
  constexpr int kLoadW = TN / 8 / kWaves, kLoadX = TM / 8 / kWaves;
  static_assert(kLoadW * kWaves * 8 == TN && kLoadX * kWaves * 8 == TM, "whole loads per wave");
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const uint32_t lds0 = (uint32_t)(uintptr_t)((__attribute__((address_space(3))) uint8_t*)smem);

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave % (TN / WN), wm = wave / (TN / WN);
  const int r = lane & 31, half = lane >> 5;
  const int tm = blockIdx.x % p.nM, tn = blockIdx.x / p.nM;
  const int64_t n0 = (int64_t)tn * TN, m0 = (int64_t)tm * TM;

  // operand moves: 8 rows of 128 bytes per instruction
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(p.w + n0 * p.ldc, (p.N - n0) * p.ldc);
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(p.x + m0 * p.ldc, (p.M - m0) * p.ldc);
  int vw[kLoadW], vx[kLoadX];
#pragma unroll
  for (int i = 0; i < kLoadW; ++i) {
    const int row = (wave * kLoadW + i) * 8 + (lane >> 3);
    vw[i] = (int)(row * p.ldc) + (((lane & 7) ^ gemm::swz(row)) << 4);
  }
#pragma unroll
  for (int i = 0; i < kLoadX; ++i) {
    const int row = (wave * kLoadX + i) * 8 + (lane >> 3);
    vx[i] = (int)(row * p.ldc) + (((lane & 7) ^ gemm::swz(row)) << 4);
  }
  auto issue = [&](int kb, int st) {
    const uint32_t a = lds0 + (uint32_t)(st * kStage);
#pragma unroll
    for (int i = 0; i < kLoadW; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rw, (lds_void*)(uintptr_t)(a + (uint32_t)((wave * kLoadW + i) * 1024)), 16, vw[i],
          kb * 128, 0, 0);
#pragma unroll
    for (int i = 0; i < kLoadX; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rx, (lds_void*)(uintptr_t)(a + (uint32_t)(TN * 128 + (wave * kLoadX + i) * 1024)), 16,
          vx[i], kb * 128, 0, 0);
  };

  // scale bytes: four blocks per dword
  const int64_t NBl = (p.N + 127) / 128;
  const __amdgpu_buffer_rsrc_t rsw = make_rsrc(p.ws, NBl * p.sb);
  const __amdgpu_buffer_rsrc_t rsx = make_rsrc(p.xs + m0 * p.sb, (p.M - m0) * p.sb);
  int osw[BN], osx[BM];
#pragma unroll
  for (int i = 0; i < BN; ++i) osw[i] = (int)((n0 + wn * WN + i * 32) / 128) * p.sb;
#pragma unroll
  for (int j = 0; j < BM; ++j) osx[j] = (wm * WM + j * 32 + r) * p.sb;
  uint32_t sw[BN], sx[BM];

  issue(0, 0);

  floatx16 acc[BN][BM];
#pragma unroll
  for (int i = 0; i < BN; ++i)
#pragma unroll
    for (int j = 0; j < BM; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;

  // the low-rank term first, straight from memory
  if (p.U) {
    const __amdgpu_buffer_rsrc_t ru =
        make_rsrc(p.U + m0 * p.r64, (p.M - m0) * (int64_t)p.r64 * 2);
    const __amdgpu_buffer_rsrc_t rv =
        make_rsrc(p.V + n0 * p.r64, (p.N - n0) * (int64_t)p.r64 * 2);
    for (int j0 = 0; j0 < p.r64; j0 += 16) {
      bf16x8 a[BN], b[BM];
#pragma unroll
      for (int i = 0; i < BN; ++i)
        a[i] = as_bf16x8(__builtin_bit_cast(
            u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                       rv, ((wn * WN + i * 32 + r) * p.r64 + half * 8) * 2, j0 * 2, 0)));
#pragma unroll
      for (int j = 0; j < BM; ++j)
        b[j] = as_bf16x8(__builtin_bit_cast(
            u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                       ru, ((wm * WM + j * 32 + r) * p.r64 + half * 8) * 2, j0 * 2, 0)));
#pragma unroll
      for (int i = 0; i < BN; ++i)
#pragma unroll
        for (int j = 0; j < BM; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[i], b[j], acc[i][j], 0, 0, 0);
    }
  }

  auto frag = [&](uint32_t base, int row, int h) {
    // pieces 4 h + 2 half and the next one
    const u32x4 a = *(const lds_u32x4*)(uintptr_t)(base + (uint32_t)tile_off(row, 4 * h + 2 * half));
    const u32x4 b = *(const lds_u32x4*)(uintptr_t)(base + (uint32_t)tile_off(row, 4 * h + 2 * half + 1));
    return i32x8{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
  };
  auto block = [&](int kb, auto sel) {
    constexpr int kSel = decltype(sel)::value;
    wait_vmcnt<0>();
    gemm::stage_barrier();
    if (kb + 1 < p.KB) issue(kb + 1, (kb + 1) & 1);
    const uint32_t aw = lds0 + (uint32_t)((kb & 1) * kStage), ax = aw + TN * 128;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      i32x8 fw[BN], fx[BM];
#pragma unroll
      for (int i = 0; i < BN; ++i) fw[i] = frag(aw, wn * WN + i * 32 + r, h);
#pragma unroll
      for (int j = 0; j < BM; ++j) fx[j] = frag(ax, wm * WM + j * 32 + r, h);
#pragma unroll
      for (int i = 0; i < BN; ++i)
#pragma unroll
        for (int j = 0; j < BM; ++j)
          acc[i][j] = mma<kSel, kXFmt>(fw[i], fx[j], acc[i][j], sw[i], sx[j]);
    }
  };
  for (int kb = 0; kb < p.KB; kb += 4) {
#pragma unroll
    for (int i = 0; i < BN; ++i) sw[i] = __builtin_amdgcn_raw_buffer_load_b32(rsw, osw[i], kb, 0);
#pragma unroll
    for (int j = 0; j < BM; ++j) sx[j] = __builtin_amdgcn_raw_buffer_load_b32(rsx, osx[j], kb, 0);
    block(kb, std::integral_constant<int, 0>{});
    if (kb + 1 < p.KB) block(kb + 1, std::integral_constant<int, 1>{});
    if (kb + 2 < p.KB) block(kb + 2, std::integral_constant<int, 2>{});
    if (kb + 3 < p.KB) block(kb + 3, std::integral_constant<int, 3>{});
  }

  const bool vec = p.N % 4 == 0 && (reinterpret_cast<uintptr_t>(p.Y) & 7) == 0;
#pragma unroll
  for (int j = 0; j < BM; ++j) {
    const int64_t m = m0 + wm * WM + j * 32 + r;
    if (m >= p.M) continue;
#pragma unroll
    for (int i = 0; i < BN; ++i)
#pragma unroll
      for (int v = 0; v < 16; v += 4) {
        const int64_t n = n0 + wn * WN + i * 32 + (v >> 2) * 8 + half * 4;
        const u32x2 d = {pack_bf16x2(acc[i][j][v], acc[i][j][v + 1]),
                         pack_bf16x2(acc[i][j][v + 2], acc[i][j][v + 3])};
        uint16_t* y = p.Y + m * p.N + n;
        if (vec && n < p.N) {
          *reinterpret_cast<u32x2*>(y) = d;
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (n + e < p.N) y[e] = (uint16_t)(d[e >> 1] >> (16 * (e & 1)));
        }
      }
  }
#endif
}

}  // namespace fp8

using namespace fp8;

namespace {

// Dynamic LDS above the default limit, raised once per device and kernel.
hipError_t allow_lds(const void* kern, size_t lds, std::atomic<uint64_t>& raised) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (raised.load(std::memory_order_acquire) & bit) return hipSuccess;
  e = hipFuncSetAttribute(kern, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (e == hipSuccess) raised.fetch_or(bit, std::memory_order_acq_rel);
  return e;
}

template <int TN, int TM, int WN, int WM, int kXFmt>
hipError_t run_tile(Fp8Gemm p, hipStream_t stream) {
  static std::atomic<uint64_t> raised{0};
  auto kern = fp8_gemm_kernel<TN, TM, WN, WM, kXFmt>;
  constexpr size_t lds = 2 * (TN + TM) * 128;
  if (lds > 65536) {
    hipError_t e = allow_lds(reinterpret_cast<const void*>(kern), lds, raised);
    if (e != hipSuccess) return e;
  }
  p.nM = (int)((p.M + TM - 1) / TM);
  p.nN = (int)((p.N + TN - 1) / TN);
  hipLaunchKernelGGL(kern, dim3((unsigned)p.nM * (unsigned)p.nN),
                     dim3((TN / WN) * (TM / WM) * 64), lds, stream, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_fp8_gemm(ConstAct8 x, int xfmt, ConstAct8 w, int64_t M, int64_t N, int64_t K,
                           const uint16_t* U, const uint16_t* V, int r64, uint16_t* Y,
                           hipStream_t stream) {
  Fp8Gemm p{};
  p.x = x.codes; p.xs = x.scales; p.w = w.codes; p.ws = w.scales;
  p.M = M; p.N = N; p.ldc = act8_row_bytes(K);
  p.KB = (int)(p.ldc / kAct8Block);
  p.sb = (int)act8_scale_row_bytes(K);
  p.U = U; p.V = V; p.r64 = r64; p.Y = Y;
  if (xfmt) return run_tile<128, 128, 64, 64, 1>(p, stream);
  return run_tile<128, 128, 64, 64, 0>(p, stream);
}

}  // namespace qlora
