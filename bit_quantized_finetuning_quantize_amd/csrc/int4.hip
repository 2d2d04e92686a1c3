// Weights in 4 bits with a scale and a zero point for each group of 32, 64 or
// 128 columns of a row, w = s (q - z): quantization, decoding, and the product
// of few tokens with them.
#include "common.h"
#include "kernels.h"

#include <algorithm>

namespace qlora {

namespace {

constexpr int kThreads = 256;

typedef u32x4 u32x4_row __attribute__((aligned(2)));

__device__ __forceinline__ uint32_t bits_of(float f) { return __builtin_bit_cast(uint32_t, f); }
// bf16(f), as a float.
__device__ __forceinline__ float to_bf16(float f) { return bf16_lo(pack_bf16x2(f, 0.0f)); }

// ---------------------------------------------------------------------------
// Quantization: kG / 8 lanes own a group, eight values each.
//   asymmetric  lo = min(w, 0), hi = max(w, 0), s = bf16((hi - lo) / 15),
//               z = rint(-lo / s) in [0, 15]
//   symmetric   s = bf16(max|w| / 7), z = 8
//   q = rint(w / s) + z in [0, 15]; where s = 0, z = 0 (symmetric 8) and q = z.
template <int kG, bool kSym>
__global__ void __launch_bounds__(kThreads)
int4_quantize_kernel(const uint16_t* __restrict__ W, int64_t ldw, int K, int ng, int64_t groups,
                     uint8_t* __restrict__ codes, uint16_t* __restrict__ scales, uint8_t* __restrict__ zeros) {
#pragma clang fp contract(off)
  constexpr int kLanes = kG / 8;
  const int64_t b = (int64_t)blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
  if (b >= groups) return;
  const int l = threadIdx.x % kLanes;
  const int64_t row = b / ng;
  const int g = (int)(b - row * ng), col = g * kG + l * 8;
  u32x4 v = {0, 0, 0, 0};
  if (col < K) v = *reinterpret_cast<const u32x4_row*>(W + row * ldw + col);
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = v[i];
    x[2 * i] = bf16_lo(w);
    x[2 * i + 1] = bf16_hi(w);
  }
  float lo = 0.0f, hi = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo = fminf(lo, x[i]);
    hi = fmaxf(hi, x[i]);
  }
#pragma unroll
  for (int d = 1; d < kLanes; d <<= 1) {
    lo = fminf(lo, __shfl_xor(lo, d));
    hi = fmaxf(hi, __shfl_xor(hi, d));
  }
  const float s = to_bf16(kSym ? fmaxf(-lo, hi) / 7.0f : (hi - lo) / 15.0f);
  const float z = kSym ? 8.0f : s > 0.0f ? fminf(__builtin_rintf(-lo / s), 15.0f) : 0.0f;
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = s > 0.0f ? __builtin_rintf(x[i] / s) + z : z;
    word |= (uint32_t)fminf(fmaxf(q, 0.0f), 15.0f) << (4 * i);
  }
  if (col < K) *reinterpret_cast<uint32_t*>(codes + (row * K + col) / 2) = word;
  if (l == 0) {
    scales[b] = (uint16_t)(bits_of(s) >> 16);
    if (!kSym) zeros[b] = (uint8_t)z;
  }
}

// bf16(s (q - z)): the product of 8 and 5 bits is exact before that.
template <int kG>
__global__ void __launch_bounds__(kThreads)
int4_dequantize_kernel(const uint8_t* __restrict__ codes, const uint16_t* __restrict__ scales,
                       const uint8_t* __restrict__ zeros, int K, int ng, int64_t units,
                       uint16_t* __restrict__ W, int64_t ldw) {
  const int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x;  // eight values
  if (u >= units) return;
  const int per = K / 8;
  const int64_t row = u / per;
  const int col = (int)(u - row * per) * 8;
  const int64_t b = row * ng + col / kG;
  const uint32_t w = *reinterpret_cast<const uint32_t*>(codes + (row * K + col) / 2);
  const float s = bf16_to_f32(scales[b]), z = zeros ? (float)zeros[b] : 8.0f;
  u32x4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = pack_bf16x2(((float)((w >> (8 * i)) & 15u) - z) * s, ((float)((w >> (8 * i + 4)) & 15u) - z) * s);
  *reinterpret_cast<u32x4_row*>(W + row * ldw + col) = v;
}

// ---------------------------------------------------------------------------
// Y [M x N] = X [M x K] W^T. A workgroup owns 16 kNR weight rows and 16 kMT
// tokens over the whole K, its waves taking runs of 128 columns in turn. The
// codes go to the matrix units as bf16 integers, without a table: a nibble
// moved to bits 3-6 of 0x4180 (16.0) is 16 + q, and a second product with
// the constant -(16 + z) takes the offset and the zero point away, all of it
// exact up to the float32 sums; each group's sum is then scaled in float32.
// The nibbles of a code word come out in the order 0, 4, 1, 5, 2, 6, 3, 7, and
// the tokens' eight values are put in that order too.

constexpr int kWaves = 8;
constexpr int kOut = 0x7ffffff0;  // an offset past every range: the load returns 0

struct Int4Args {
  const uint16_t* X;
  const uint8_t* codes;
  const uint16_t* scales;
  const uint8_t* zeros;  // or null: 8
  int64_t M, N, K, ng, ldx, ldy;
  void* Y;
  int f32;
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const void* base, int64_t bytes) {
  if (bytes > 0x7ffffff0LL) bytes = 0x7ffffff0LL;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}

__device__ __forceinline__ u32x4 nibbles_bf16(uint32_t w) {
  constexpr uint32_t kMask = 0x00780078u, kBase = 0x41804180u;
  return u32x4{((w << 3) & kMask) | kBase, ((w >> 1) & kMask) | kBase, ((w >> 5) & kMask) | kBase,
               ((w >> 9) & kMask) | kBase};
}
__device__ __forceinline__ u32x4 nibble_order(const u32x4& v) {
  return u32x4{__builtin_amdgcn_perm(v[2], v[0], 0x05040100u), __builtin_amdgcn_perm(v[2], v[0], 0x07060302u),
               __builtin_amdgcn_perm(v[3], v[1], 0x05040100u), __builtin_amdgcn_perm(v[3], v[1], 0x07060302u)};
}

template <int kG, int kMT, int kNR>
__global__ void __launch_bounds__(kWaves * 64) int4_linear_kernel(Int4Args a) {
  constexpr int kGroups = 128 / kG;  // groups of a run
  constexpr int kWords = kG / 32;    // code words a lane holds of a group
  __shared__ floatx4 s_red[kWaves][kMT * kNR][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * kNR), m0 = (int64_t)blockIdx.y * (16 * kMT);
  const int K = (int)a.K;
  const __amdgpu_buffer_rsrc_t rc = rsrc_of(a.codes, a.N * a.K / 2);
  const __amdgpu_buffer_rsrc_t rs = rsrc_of(a.scales, a.N * a.ng * 2);
  const __amdgpu_buffer_rsrc_t rz = rsrc_of(a.zeros, a.zeros ? a.N * a.ng : 0);
  const __amdgpu_buffer_rsrc_t rx = rsrc_of(a.X, ((a.M - 1) * a.ldx + K) * 2);
  const floatx4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  floatx4 acc[kMT][kNR];
#pragma unroll
  for (int m = 0; m < kMT; ++m)
#pragma unroll
    for (int r = 0; r < kNR; ++r) acc[m][r] = zero;

  for (int k0 = wave * 128; k0 < K; k0 += kWaves * 128) {
    uint32_t w[kNR][kGroups][kWords];
    uint32_t s[kNR][kGroups], z[kNR][kGroups];
    u32x4 x[kMT][kGroups][kWords];
#pragma unroll
    for (int r = 0; r < kNR; ++r) {
      const int64_t n = n0 + 16 * r + c;
#pragma unroll
      for (int j = 0; j < kGroups; ++j) {
        const int k = k0 + kG * j + (kG / 4) * g;
        const int at = n < a.N && k < K ? (int)((n * K + k) / 2) : kOut;
        if constexpr (kWords == 4) {
          const u32x4 v = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rc, at, 0, 0));
          w[r][j][0] = v[0]; w[r][j][1] = v[1]; w[r][j][2] = v[2]; w[r][j][3] = v[3];
        } else if constexpr (kWords == 2) {
          const u32x2 v = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(rc, at, 0, 0));
          w[r][j][0] = v[0]; w[r][j][1] = v[1];
        } else {
          w[r][j][0] = __builtin_amdgcn_raw_buffer_load_b32(rc, at, 0, 0);
        }
        const int b = n < a.N && k0 + kG * j < K ? (int)(n * a.ng + k0 / kG + j) : -1;
        s[r][j] = __builtin_amdgcn_raw_buffer_load_b16(rs, b >= 0 ? b * 2 : kOut, 0, 0);
        z[r][j] = a.zeros ? __builtin_amdgcn_raw_buffer_load_b8(rz, b >= 0 ? b : kOut, 0, 0) : 8u;
      }
    }
#pragma unroll
    for (int m = 0; m < kMT; ++m) {
      const int64_t t = m0 + 16 * m + c;
#pragma unroll
      for (int j = 0; j < kGroups; ++j)
#pragma unroll
        for (int e = 0; e < kWords; ++e) {
          const int k = k0 + kG * j + (kG / 4) * g + 8 * e;
          x[m][j][e] = __builtin_bit_cast(
              u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                         rx, t < a.M && k < K ? (int)((t * a.ldx + k) * 2) : kOut, 0, 0));
        }
    }
#pragma unroll
    for (int j = 0; j < kGroups; ++j) {
      bf16x8 xf[kMT][kWords];
#pragma unroll
      for (int m = 0; m < kMT; ++m)
#pragma unroll
        for (int e = 0; e < kWords; ++e) xf[m][e] = as_bf16x8(nibble_order(x[m][j][e]));
#pragma unroll
      for (int r = 0; r < kNR; ++r) {
        const float sc = __builtin_bit_cast(float, s[r][j] << 16);
        const uint32_t off = (0xc180u | ((z[r][j] & 15u) << 3)) * 0x10001u;  // -(16 + z), twice
        const bf16x8 of = as_bf16x8(u32x4{off, off, off, off});
        floatx4 p[kMT];
#pragma unroll
        for (int e = 0; e < kWords; ++e) {
          const bf16x8 q = as_bf16x8(nibbles_bf16(w[r][j][e]));
#pragma unroll
          for (int m = 0; m < kMT; ++m) {
            p[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[m][e], q, e ? p[m] : zero, 0, 0, 0);
            p[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[m][e], of, p[m], 0, 0, 0);
          }
        }
#pragma unroll
        for (int m = 0; m < kMT; ++m)
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[m][r][v] = __builtin_fmaf(sc, p[m][v], acc[m][r][v]);
      }
    }
  }
  // the waves' sums, added in the order of the waves; lane (c, g) holds tokens
  // 4 g .. 4 g + 3 of weight row c
#pragma unroll
  for (int m = 0; m < kMT; ++m)
#pragma unroll
    for (int r = 0; r < kNR; ++r) s_red[wave][m * kNR + r][lane] = acc[m][r];
  __syncthreads();
  for (int i = wave; i < kMT * kNR; i += kWaves) {
    floatx4 y = s_red[0][i][lane];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) {
      const floatx4 u = s_red[w][i][lane];
#pragma unroll
      for (int v = 0; v < 4; ++v) y[v] += u[v];
    }
    const int64_t n = n0 + 16 * (i % kNR) + c;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int64_t t = m0 + 16 * (i / kNR) + 4 * g + v;
      if (n >= a.N || t >= a.M) continue;
      if (a.f32)
        reinterpret_cast<float*>(a.Y)[t * a.ldy + n] = y[v];
      else
        reinterpret_cast<uint16_t*>(a.Y)[t * a.ldy + n] = (uint16_t)(pack_bf16x2(y[v], 0.0f) & 0xffffu);
    }
  }
}

template <int kG, int kMT, int kNR>
hipError_t run_linear(const Int4Args& a, hipStream_t stream) {
  const dim3 grid((unsigned)((a.N + 16 * kNR - 1) / (16 * kNR)), (unsigned)((a.M + 16 * kMT - 1) / (16 * kMT)));
  int4_linear_kernel<kG, kMT, kNR><<<grid, dim3(kWaves * 64), 0, stream>>>(a);
  return hipGetLastError();
}

template <typename F>
hipError_t by_group(int group, F f) {
  if (group == 32) return f(std::integral_constant<int, 32>{});
  if (group == 64) return f(std::integral_constant<int, 64>{});
  return f(std::integral_constant<int, 128>{});
}

}  // namespace

hipError_t launch_int4_quantize(const uint16_t* W, int64_t N, int64_t K, int64_t ldw, int group, uint8_t* codes,
                                uint16_t* scales, uint8_t* zeros, hipStream_t stream) {
  const int64_t ng = (K + group - 1) / group, groups = N * ng, per = kThreads * 8 / group;
  return by_group(group, [&](auto g) {
    constexpr int kG = decltype(g)::value;
    const dim3 grid((unsigned)((groups + per - 1) / per));
    if (zeros)
      int4_quantize_kernel<kG, false><<<grid, dim3(kThreads), 0, stream>>>(W, ldw, (int)K, (int)ng, groups, codes, scales, zeros);
    else
      int4_quantize_kernel<kG, true><<<grid, dim3(kThreads), 0, stream>>>(W, ldw, (int)K, (int)ng, groups, codes, scales, zeros);
    return hipGetLastError();
  });
}

hipError_t launch_int4_dequantize(const Int4Weight& w, uint16_t* out, int64_t ldo, hipStream_t stream) {
  const int64_t units = w.N * w.K / 8;
  return by_group(w.group, [&](auto g) {
    constexpr int kG = decltype(g)::value;
    int4_dequantize_kernel<kG><<<dim3((unsigned)((units + kThreads - 1) / kThreads)), dim3(kThreads), 0, stream>>>(
        w.codes, w.scales, w.zeros, (int)w.K, (int)((w.K + kG - 1) / kG), units, out, ldo);
    return hipGetLastError();
  });
}

hipError_t launch_int4_linear_fwd(const uint16_t* X, int64_t M, int64_t ldx, const Int4Weight& w, void* Y, bool f32,
                                  int64_t ldy, hipStream_t stream) {
  Int4Args a{X, w.codes, w.scales, w.zeros, M, w.N, w.K, (w.K + w.group - 1) / w.group, ldx, ldy, Y, f32};
  return by_group(w.group, [&](auto g) {
    constexpr int kG = decltype(g)::value;
    if (M <= 16) return run_linear<kG, 1, 1>(a, stream);
    if (M <= 32) return run_linear<kG, 2, 1>(a, stream);
    if (M <= 48) return run_linear<kG, 3, 1>(a, stream);
    return run_linear<kG, 4, 1>(a, stream);
  });
}

}  // namespace qlora
