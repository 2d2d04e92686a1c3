// Column products of the adapter's gradients (lowrank8.hip says how they and
// the row products work), for a launch of their own and beside another kernel's
// workgroups.
#pragma once

#include "act8.h"
#include "gemm.h"
#include "kernels.h"

namespace qlora {

namespace lr8 {

using gemm::keep_mask8;
using gemm::lds_u32x4;
using gemm::make_rsrc;

constexpr int kWaves = 8;
constexpr int kThreads = kWaves * 64;
constexpr int kTerms = 3;
constexpr int kPitch = 144;  // bytes of a transposing tile's row: 64 bf16 and 16 bytes
                             // of padding, which keeps four rows on distinct banks

typedef __attribute__((address_space(3))) float lds_f32;
typedef __attribute__((address_space(3))) floatx4 lds_floatx4;

// How S is held: 8-bit blocks in either format, or bf16; kAct8: 8-bit blocks in
// the format that Stream names.
enum Src { kE4M3 = 0, kE5M2 = 1, kBf16 = 2, kAct8 = 3 };

struct Stream {
  const void* s;          // codes or bf16 values
  const uint8_t* scales;  // 8-bit only
  int64_t ld, sld;        // bytes between rows of s, of scales
  int64_t rows, cols;
  const uint32_t* mask;   // dropout keep bits [rows][cols / 32], or null
  int fmt;                // 8-bit only: E4M3 or E5M2
};

// Place of element (m, j) in the fragment order of V: blocks of 32 rows; in a
// block by 16 columns; there as the matrix instruction takes it, lane
// (m / 8 % 4) * 16 + j % 16 with eight consecutive m, so that one fragment is
// 2 KiB of consecutive memory.
__device__ __forceinline__ int64_t frag_index(int64_t m, int64_t j, int64_t rp) {
  return (((m >> 5) * (rp >> 4) + (j >> 4)) * 64 + ((m >> 3) & 3) * 16 + (j & 15)) * 8 + (m & 7);
}

// The waves' accumulators of one 64 x 16 NJ tile (block f * NJ + jt holds rows
// f * 16 + 4 g + e, column jt * 16 + i) added in a fixed order: wave w takes
// wave w + 4's, and the four sums go to LDS as [sum][column][kRowPitch rows],
// where tile_sum adds them. Every thread of the workgroup takes part.
constexpr int kRowPitch = 68;  // floats; 16 columns' 16-byte pieces on distinct banks
constexpr int tile_bytes(int NJ) { return 4 * 16 * NJ * kRowPitch * 4; }

template <int NJ>
__device__ __forceinline__ void reduce_waves(floatx4 (&acc)[4 * NJ], uint32_t buf, int wave, int lane) {
  const uint32_t mine = buf + (uint32_t)((((wave & 3) * 16 * NJ + (lane & 15)) * kRowPitch + (lane >> 4) * 4) * 4);
  __syncthreads();
#pragma unroll
  for (int pass = 0; pass < 2; ++pass) {
    if ((pass == 0) == (wave >= 4)) {
#pragma unroll
      for (int b = 0; b < 4 * NJ; ++b)
        *(lds_floatx4*)(uintptr_t)(mine + (uint32_t)(((b % NJ) * 16 * kRowPitch + (b / NJ) * 16) * 4)) = acc[b];
    }
    __syncthreads();
    if (pass == 0 && wave < 4) {
#pragma unroll
      for (int b = 0; b < 4 * NJ; ++b) {
        const floatx4 o =
            *(const lds_floatx4*)(uintptr_t)(mine + (uint32_t)(((b % NJ) * 16 * kRowPitch + (b / NJ) * 16) * 4));
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[b][e] += o[e];
      }
    }
  }
}
template <int NJ>
__device__ __forceinline__ float tile_sum(uint32_t buf, int row, int col) {
  float v = 0.0f;
#pragma unroll
  for (int w = 0; w < 4; ++w)
    v += *(const lds_f32*)(uintptr_t)(buf + (uint32_t)(((w * 16 * NJ + col) * kRowPitch + row) * 4));
  return v;
}

// ---------------------------------------------------------------------------
// Column products: 64 columns of S by 16 NJ columns of V per workgroup; the
// waves take 32 rows of S at a time in turn.
struct ColProd {
  Stream s;
  const float* v;      // V in fragment order
  float* out;          // element (c, j) at c * oc + j * oj
  int64_t oc, oj;
};
struct ColPair {
  ColProd a, b;   // a: 8-bit S, b: bf16 S
  int ta, tiles;  // column tiles of a, of both
  int jobs;       // workgroups: tiles by tiles of 64 columns of V
  int r, rp;
};

// Eight floats as three bf16 terms each: every remainder is exact, so the
// terms' sum is the float to 24 bits. The first term is cut towards zero, since
// rounded it would be an infinity above the largest bf16; the others are
// rounded. An infinity's remainder is a NaN.
__device__ __forceinline__ void split3(const floatx4 (&v)[2], u32x4 (&term)[kTerms]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float a = v[e >> 1][(e & 1) * 2], b = v[e >> 1][(e & 1) * 2 + 1];
#pragma unroll
    for (int c = 0; c < kTerms; ++c) {
      const uint32_t w = c ? pack_bf16x2(a, b)
                           : __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, b),
                                                   __builtin_bit_cast(uint32_t, a), 0x07060302u);  // upper halves
      term[c][e] = w;
      a -= __builtin_bit_cast(float, w << 16);
      b -= __builtin_bit_cast(float, w & 0xffff0000u);
    }
  }
}

template <int kSrc, int NJ>
__device__ __forceinline__ void column_product(const ColProd& p, int ct, int j0, int r, int rp,
                                                uint32_t lds, int wave, int lane) {
#ifdef __HIP_DEVICE_COMPILE__
  constexpr int NF = 4 * NJ;
  const int i = lane & 15, g = lane >> 4;
  const int64_t c0 = (int64_t)ct * 64;
  const uint32_t tile = lds + (uint32_t)(wave * 32 * kPitch);
  constexpr int kBytes = kSrc == kBf16 ? 2 : 1;
  const __amdgpu_buffer_rsrc_t rs = make_rsrc((const uint8_t*)p.s.s + c0 * kBytes, p.s.rows * p.s.ld - c0 * kBytes);
  const __amdgpu_buffer_rsrc_t rsc = make_rsrc(p.s.scales + (c0 >> 7), p.s.rows * p.s.sld - (c0 >> 7));
  const int64_t mld = p.s.cols / 32;
  const __amdgpu_buffer_rsrc_t rm = make_rsrc(p.s.mask + (c0 >> 5), p.s.rows * mld * 4 - (c0 >> 5) * 4);
  // fragments of one block of 32 rows: rp / 16 of 2 KiB
  const float* vb = p.v + (int64_t)(j0 >> 4) * 512 + lane * 8;
  const int64_t vblock = (int64_t)rp * 32;

  floatx4 acc[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f) acc[f] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};

  constexpr int kS = kSrc == kBf16 ? 4 : 2;
  const bool e5m2 = kSrc == kAct8 ? p.s.fmt != 0 : kSrc == kE5M2, masked = p.s.mask != nullptr;  // uniform
  struct Regs {
    u32x4 s[kS];
    uint32_t sc[2], keep[2];
    floatx4 v[NJ][2];
  };
  const int steps = (int)((p.s.rows + 31) / 32);
  // One step's loads: 32 rows of S by 64 columns, and V's fragments.
  auto load = [&](int st) {
    Regs q;
    if constexpr (kSrc == kBf16) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        q.s[e] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
            rs, (int)((st * 32 + e * 8 + (lane >> 3)) * p.s.ld) + (lane & 7) * 16, 0, 0));
    } else {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int m = st * 32 + e * 16 + (lane >> 2), ch = lane & 3;
        q.s[e] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
            rs, (int)(m * p.s.ld) + ch * 16, 0, 0));
        q.sc[e] = __builtin_amdgcn_raw_buffer_load_b8(rsc, (int)(m * p.s.sld), 0, 0);
        if (masked)
          q.keep[e] = __builtin_amdgcn_raw_buffer_load_b32(rm, (int)(m * mld * 4) + (ch >> 1) * 4, 0, 0);
      }
    }
    const float* v = vb + st * vblock;
#pragma unroll
    for (int jt = 0; jt < NJ; ++jt)
#pragma unroll
      for (int h = 0; h < 2; ++h) q.v[jt][h] = *reinterpret_cast<const floatx4*>(v + jt * 512 + h * 4);
    return q;
  };
  for (int st = wave; st < steps; st += kWaves) {
    const Regs q = load(st);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (kSrc == kBf16) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *(lds_u32x4*)(uintptr_t)(tile + (uint32_t)((e * 8 + (lane >> 3)) * kPitch + (lane & 7) * 16)) = q.s[e];
    } else {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = e * 16 + (lane >> 2), ch = lane & 3;
        const float sc = act8_scale((int)q.sc[e]);
        const u32x2 c0{q.s[e][0], q.s[e][1]}, c1{q.s[e][2], q.s[e][3]};
        u32x4 lo = e5m2 ? act8_decode8<1>(c0, sc) : act8_decode8<0>(c0, sc);
        u32x4 hi = e5m2 ? act8_decode8<1>(c1, sc) : act8_decode8<0>(c1, sc);
        if (masked) {
          const uint32_t bits = q.keep[e] >> ((ch & 1) * 16);
          lo &= keep_mask8(bits);
          hi &= keep_mask8(bits >> 8);
        }
        *(lds_u32x4*)(uintptr_t)(tile + (uint32_t)(row * kPitch + ch * 32)) = lo;
        *(lds_u32x4*)(uintptr_t)(tile + (uint32_t)(row * kPitch + ch * 32 + 16)) = hi;
      }
    }
    bf16x8 x[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) x[f] = tr_frag<kPitch>(tile, 8 * g, f * 16, lane);
#pragma unroll
    for (int jt = 0; jt < NJ; ++jt) {
      u32x4 term[kTerms];
      split3(q.v[jt], term);
#pragma unroll
      for (int c = kTerms - 1; c >= 0; --c)  // smallest terms first
#pragma unroll
        for (int f = 0; f < 4; ++f)
          acc[f * NJ + jt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[f], as_bf16x8(term[c]),
                                                                     acc[f * NJ + jt], 0, 0, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  reduce_waves<NJ>(acc, lds, wave, lane);
  // dA's rows run along j, dB's along the columns of S
#pragma unroll
  for (int q = 0; q < 2 * NJ; ++q) {
    const int o = q * kThreads + threadIdx.x;
    const int j = kSrc == kBf16 ? o / 64 : o % (16 * NJ), c = kSrc == kBf16 ? o % 64 : o / (16 * NJ);
    const float v = tile_sum<NJ>(lds, c, j);
    if (j0 + j < r) p.out[(c0 + c) * p.oc + (j0 + j) * p.oj] = v;
  }
#endif
}

// Workgroup `id` of a pair (kSrc: how the 8-bit S is held), kThreads threads and column_lds(NJ) bytes of LDS.
constexpr int column_lds(int NJ) {
  return kWaves * 32 * kPitch > tile_bytes(NJ) ? kWaves * 32 * kPitch : tile_bytes(NJ);
}
template <int kSrc, int NJ>
__device__ __forceinline__ void column_job(const ColPair& p, int id, uint32_t lds) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int b = id % p.tiles, j0 = id / p.tiles * 64;
  if (b < p.ta) column_product<kSrc, NJ>(p.a, b, j0, p.r, p.rp, lds, wave, lane);
  else column_product<kBf16, NJ>(p.b, b - p.ta, j0, p.r, p.rp, lds, wave, lane);
}

// Both products of a backward pass: dA [K x r] = D(dec x)^T g and
// dB [r x N] = t^T dY.
ColPair column_pair(ConstAct8 x, int fmt, const uint32_t* mask, const uint16_t* dY, const float* g,
                    const float* t, int64_t M, int64_t N, int64_t K, int r, float* dA, float* dB);

// Columns of V per workgroup in tiles of 16: f(integral_constant<int, NJ>).
template <class F>
hipError_t by_nj(int r, F&& f) {
  using std::integral_constant;
  if (r <= 16) return f(integral_constant<int, 1>{});
  if (r <= 32) return f(integral_constant<int, 2>{});
  return f(integral_constant<int, 4>{});
}

}  // namespace lr8

}  // namespace qlora
