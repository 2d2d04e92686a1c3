// The adapter's products beside an 8-bit input, on bf16 matrix instructions.
//
// Row products   V[m][j] = sum_c S[m][c] W[j][c]      T = dec(X8) A, G = dY B^T
// Column products P[c][j] = sum_m S[m][c] V[m][j]     dA = dec(X8)^T (s G), dB^T = dY^T (s T)
//
// S streams past once: codes are decoded in registers (a code times its
// power-of-two scale is an exact bf16 value). Both are bound by reading S
// and by the small factor's traffic through the caches; the matrix work is
// r columns wide.
//
// v_mfma_f32_16x16x32_bf16 takes eight contraction elements per lane. A row
// product finds them next to each other in memory (S and B rows), except for
// A [K x r]; a column product contracts down the rows of S. Those operands
// pass through a wave's own LDS tile, row-major, and come back transposed by
// ds_read_b64_tr_b16 (16 lanes read a 4 x 16 piece by rows and receive it by
// columns), with no barrier.
//
// dA and dB are float32: V enters the column product as three bf16 terms
// whose sum is the float32 value to 24 bits, so the products of bf16 values
// carry float32 accuracy. The results of the waves of a workgroup, which
// take turns along the contraction, are added in a fixed order.
#include "act8.h"
#include "gemm.h"
#include "kernels.h"

#include <algorithm>

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

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) float lds_f32;
typedef __attribute__((address_space(3))) floatx4 lds_floatx4;

// How S is held: 8-bit blocks in either format, or bf16.
enum Src { kE4M3 = 0, kE5M2 = 1, kBf16 = 2 };

struct Stream {
  const void* s;          // codes or bf16 values
  const uint8_t* scales;  // 8-bit only
  int64_t ld, sld;        // bytes between rows of s, of scales
  int64_t rows, cols;
  const uint32_t* mask;   // dropout keep bits [rows][cols / 32], or null
};

// The eight transposed elements of a fragment from a row-major tile: lane l
// receives column (l & 15) + c0 and rows r0 .. r0 + 7 of its own 16-lane
// group's row base.
__device__ __forceinline__ bf16x8 tr_frag(uint32_t tile, int row0, int c0, int lane) {
  const int p = lane & 15;
  const uint32_t a = tile + (uint32_t)((row0 + (p >> 2)) * kPitch + (c0 + (p & 3) * 4) * 2);
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(uintptr_t)a);
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(uintptr_t)(a + 4 * kPitch));
  const u32x2 l2 = __builtin_bit_cast(u32x2, lo), h2 = __builtin_bit_cast(u32x2, hi);
  return as_bf16x8(u32x4{l2[0], l2[1], h2[0], h2[1]});
}

// Sum of the waves' accumulators in a fixed order (a tree), left in wave 0's
// registers. `buf` holds kWaves / 2 accumulators. Every wave takes part.
template <int NF>
__device__ __forceinline__ void reduce_waves(floatx4 (&acc)[NF], uint32_t buf, int wave, int lane) {
#pragma unroll
  for (int n = kWaves / 2; n >= 1; n >>= 1) {
    __syncthreads();
    if (wave >= n && wave < 2 * n) {
#pragma unroll
      for (int f = 0; f < NF; ++f)
        *(lds_floatx4*)(uintptr_t)(buf + (uint32_t)((((wave - n) * NF + f) * 64 + lane) * 16)) = acc[f];
    }
    __syncthreads();
    if (wave < n) {
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        const floatx4 o = *(const lds_floatx4*)(uintptr_t)(buf + (uint32_t)(((wave * NF + f) * 64 + lane) * 16));
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[f][e] += o[e];
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Row products: 64 rows by 16 NJ columns per workgroup; the waves take the
// contraction 64 elements at a time in turn. Inside such a step the lanes of
// group g hold elements 16 g .. 16 g + 15 (one 16-byte piece of codes), which
// make two matrix instructions of eight elements per lane.
struct RowProd {
  Stream s;
  const uint16_t* w;  // kTrans: A [cols x r], row-major; else B [r x cols]
  int r;
  bool wvec;          // kTrans: rows of w are 16-byte aligned
  int steps;          // steps of 64 in all, and per workgroup
  int per;
  int ldp;            // columns of a partial row
  float* part;        // [splits][rows][ldp]
  int tiles;          // row tiles of 64
};

template <int kSrc, bool kMask, bool kTrans, int NJ>
__global__ void __launch_bounds__(kThreads) row_product_kernel(RowProd p) {
#ifdef __HIP_DEVICE_COMPILE__  // the host pass needs the stub alone
  constexpr int NF = 4 * NJ;
  constexpr int kTile = 64 * kPitch;
  constexpr int kRed = kWaves / 2 * NF * 1024;
  __shared__ __attribute__((aligned(16))) uint8_t smem[kTrans && kWaves * kTile > kRed ? kWaves * kTile : kRed];
  const uint32_t lds = (uint32_t)(uintptr_t)((__attribute__((address_space(3))) uint8_t*)smem);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = lane & 15, g = lane >> 4;
  const int tile = blockIdx.x % p.tiles, split = blockIdx.x / p.tiles;
  const int j0 = blockIdx.y * 64;
  const int64_t m0 = (int64_t)tile * 64;

  const int64_t rows = p.s.rows - m0;
  const __amdgpu_buffer_rsrc_t rs = make_rsrc((const uint8_t*)p.s.s + m0 * p.s.ld, rows * p.s.ld);
  const __amdgpu_buffer_rsrc_t rsc = make_rsrc(p.s.scales + m0 * p.s.sld, rows * p.s.sld);
  const int64_t mld = p.s.cols / 32;
  const __amdgpu_buffer_rsrc_t rm = make_rsrc(p.s.mask + m0 * mld, rows * mld * 4);
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(p.w, (int64_t)p.r * p.s.cols * 2);
  const uint32_t wt = lds + (uint32_t)(wave * kTile);

  floatx4 acc[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f) acc[f] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};

  const int end = min(p.steps, (split + 1) * p.per);
  for (int st = split * p.per + wave; st < end; st += kWaves) {
    u32x4 x[4][2];  // bf16 pairs: two matrix steps of 8 elements, four row blocks
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      const int row = f * 16 + i;
      if constexpr (kSrc == kBf16) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          x[f][h] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
              rs, (int)(row * p.s.ld) + g * 32 + h * 16, st * 128, 0));
      } else {
        const u32x4 c = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
            rs, (int)(row * p.s.ld) + g * 16, st * 64, 0));
        const float sc = act8_scale(__builtin_amdgcn_raw_buffer_load_b8(rsc, (int)(row * p.s.sld), st >> 1, 0));
        x[f][0] = act8_decode8<kSrc>(u32x2{c[0], c[1]}, sc);
        x[f][1] = act8_decode8<kSrc>(u32x2{c[2], c[3]}, sc);
        if constexpr (kMask) {
          const uint32_t bits = __builtin_amdgcn_raw_buffer_load_b32(
              rm, (int)(row * mld * 4) + (g >> 1) * 4, st * 8, 0) >> ((g & 1) * 16);
          x[f][0] &= keep_mask8(bits);
          x[f][1] &= keep_mask8(bits >> 8);
        }
      }
    }
    bf16x8 w[NJ][2];
    if constexpr (kTrans) {
      // rows st * 64 .. + 63 of A, columns j0 .. j0 + 16 NJ - 1, by way of LDS
      if (p.wvec) {
#pragma unroll
        for (int q = 0; q < 2 * NJ; ++q) {
          const int id = q * 64 + lane, row = id / (2 * NJ), ch = id % (2 * NJ);
          const bool ok = j0 + ch * 8 < p.r;  // r is a multiple of 8 here
          const u32x4 v = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
              rw, ok ? (row * p.r + j0 + ch * 8) * 2 : 0x7ffffff0, st * 64 * p.r * 2, 0));
          *(lds_u32x4*)(uintptr_t)(wt + (uint32_t)(row * kPitch + ch * 16)) = v;
        }
      } else {
        for (int e = lane; e < 64 * 16 * NJ; e += 64) {
          const int row = e / (16 * NJ), j = e % (16 * NJ);
          uint16_t v = 0;
          if (j0 + j < p.r) v = p.w[((int64_t)st * 64 + row) * p.r + j0 + j];
          *(gemm::lds_u16*)(uintptr_t)(wt + (uint32_t)(row * kPitch + j * 2)) = v;
        }
      }
#pragma unroll
      for (int jt = 0; jt < NJ; ++jt)
#pragma unroll
        for (int h = 0; h < 2; ++h) w[jt][h] = tr_frag(wt, 16 * g + 8 * h, jt * 16, lane);
    } else {
#pragma unroll
      for (int jt = 0; jt < NJ; ++jt) {
        const int j = j0 + jt * 16 + i;
        const int off = j < p.r ? (int)(j * p.s.cols * 2) + g * 32 : 0x7ffffff0;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          w[jt][h] = as_bf16x8(__builtin_bit_cast(
              u32x4, __builtin_amdgcn_raw_buffer_load_b128(rw, off + h * 16, st * 128, 0)));
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int f = 0; f < 4; ++f)
#pragma unroll
        for (int jt = 0; jt < NJ; ++jt)
          acc[f * NJ + jt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(x[f][h]), w[jt][h],
                                                                     acc[f * NJ + jt], 0, 0, 0);
  }
  reduce_waves<NF>(acc, lds, wave, lane);
  if (wave != 0) return;
#pragma unroll
  for (int f = 0; f < 4; ++f)
#pragma unroll
    for (int jt = 0; jt < NJ; ++jt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t m = m0 + f * 16 + g * 4 + e;
        if (m < p.s.rows)
          p.part[((int64_t)split * p.s.rows + m) * p.ldp + j0 + jt * 16 + i] = acc[f * NJ + jt][e];
      }
#endif
}

// ---------------------------------------------------------------------------
// What follows a row product: V = f * (sum of the partials, in split order),
// written as any of
//   out32  float32 V [M x r]
//   u      bf16(s V), [Mp x r64], 0 past M and r
//   v3     three bf16 terms of s V, transposed: [3][rp][Mp], 0 past M and r
// 64 x 64 tiles, through LDS for the transposed form.
struct OutJob {
  const float* part;  // null: no job
  int splits;
  int64_t ldp;
  float f;
  float* out32;
  uint16_t* u;
  uint16_t* v3;
};
// Padded copies of adapter operands: dst [rows x r64] from A [rows x r]
// (row-major), or from the columns of B [r x rows].
struct PadJob {
  const uint16_t* src;  // null: no job
  bool columns;
  int64_t rows;
  uint16_t* dst;
};

constexpr int kOutThreads = 256;

__device__ __forceinline__ void out_tile(const OutJob& jb, int64_t mt, int jc, int64_t M, int64_t Mp,
                                         int r, int64_t r64, int64_t rp, float s, float (&tile)[64][65]) {
  const int t = threadIdx.x;
#pragma unroll 4
  for (int q = 0; q < 16; ++q) {
    const int jl = t & 63, ml = (t >> 6) + 4 * q;
    const int64_t m = mt * 64 + ml;
    const int j = jc * 64 + jl;
    float v = 0.0f;
    if (m < M && j < r) {
      for (int sp = 0; sp < jb.splits; ++sp) v += jb.part[((int64_t)sp * M + m) * jb.ldp + j];
      v *= jb.f;
      if (jb.out32) jb.out32[m * r + j] = v;
    }
    v *= s;
    if (jb.u) jb.u[m * r64 + j] = (uint16_t)(pack_bf16x2(v, 0.0f) & 0xffffu);
    tile[ml][jl] = v;
  }
  if (!jb.v3) return;
  __syncthreads();
#pragma unroll 4
  for (int q = 0; q < 16; ++q) {
    const int ml = t & 63, jl = (t >> 6) + 4 * q;
    const int64_t j = jc * 64 + jl;
    if (j >= rp) continue;
    float rest = tile[ml][jl];
#pragma unroll
    for (int c = 0; c < kTerms; ++c) {
      const uint32_t b = pack_bf16x2(rest, 0.0f) & 0xffffu;
      jb.v3[(c * rp + j) * Mp + mt * 64 + ml] = (uint16_t)b;
      // exact; nothing is left of an infinity or NaN, which the first term carries
      const float top = __builtin_bit_cast(float, b << 16);
      rest = __builtin_isfinite(top) ? rest - top : 0.0f;
    }
  }
}

__device__ __forceinline__ void pad_tile(const PadJob& jb, int64_t rt, int jc, int r, int64_t r64,
                                         float (&tile)[64][65]) {
  const int t = threadIdx.x;
  if (!jb.columns) {
#pragma unroll 4
    for (int q = 0; q < 16; ++q) {
      const int64_t row = rt * 64 + (t >> 6) + 4 * q;
      const int j = jc * 64 + (t & 63);
      if (row < jb.rows) jb.dst[row * r64 + j] = j < r ? jb.src[row * r + j] : (uint16_t)0;
    }
    return;
  }
#pragma unroll 4
  for (int q = 0; q < 16; ++q) {  // read along the rows of B
    const int64_t row = rt * 64 + (t & 63);
    const int jl = (t >> 6) + 4 * q, j = jc * 64 + jl;
    uint32_t v = 0;
    if (row < jb.rows && j < r) v = jb.src[(int64_t)j * jb.rows + row];
    tile[t & 63][jl] = __builtin_bit_cast(float, v);
  }
  __syncthreads();
#pragma unroll 4
  for (int q = 0; q < 16; ++q) {
    const int rl = (t >> 6) + 4 * q;
    const int64_t row = rt * 64 + rl;
    if (row < jb.rows)
      jb.dst[row * r64 + jc * 64 + (t & 63)] = (uint16_t)__builtin_bit_cast(uint32_t, tile[rl][t & 63]);
  }
}

struct OutArgs {
  OutJob o[2];
  PadJob pad;
  int64_t M, Mp;
  int r;
  int64_t r64, rp;
  float s;
  int mtiles, blocks0, blocks1;  // row tiles of M; blocks of the two out jobs
};

__global__ void __launch_bounds__(kOutThreads) lowrank_out_kernel(OutArgs p) {
  __shared__ float tile[64][65];
  int b = blockIdx.x;
  const int jc = blockIdx.y;
  if (b < p.blocks0) return out_tile(p.o[0], b, jc, p.M, p.Mp, p.r, p.r64, p.rp, p.s, tile);
  b -= p.blocks0;
  if (b < p.blocks1) return out_tile(p.o[1], b, jc, p.M, p.Mp, p.r, p.r64, p.rp, p.s, tile);
  b -= p.blocks1;
  pad_tile(p.pad, b, jc, p.r, p.r64, tile);
}

// ---------------------------------------------------------------------------
// Column products: 64 columns of S by 16 NJ columns of V per workgroup; the
// waves take 32 rows of S at a time in turn.
struct ColProd {
  Stream s;
  const uint16_t* v3;  // [3][rp][Mp]
  float* out;          // element (c, j) at c * oc + j * oj
  int64_t oc, oj;
};
struct ColPair {
  ColProd a, b;   // a: 8-bit S, b: bf16 S
  int ta;         // column tiles of a
  int64_t Mp;
  int r, rp;
};

template <int kSrc, bool kMask, int NJ>
__device__ __forceinline__ void column_product(const ColProd& p, int ct, int j0, int64_t Mp, int r,
                                               int rp, uint32_t lds, int wave, int lane) {
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
  const __amdgpu_buffer_rsrc_t rv = make_rsrc(p.v3, (int64_t)kTerms * rp * Mp * 2);
  int ov[NJ];
#pragma unroll
  for (int jt = 0; jt < NJ; ++jt) ov[jt] = (int)(((int64_t)(j0 + jt * 16 + i) * Mp + g * 8) * 2);
  const int term = (int)((int64_t)rp * Mp * 2);

  floatx4 acc[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f) acc[f] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};

  const int steps = (int)((p.s.rows + 31) / 32);
  for (int st = wave; st < steps; st += kWaves) {
    if constexpr (kSrc == kBf16) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int row = q * 8 + (lane >> 3), ch = lane & 7;
        const u32x4 v = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
            rs, (int)((st * 32 + row) * p.s.ld) + ch * 16, 0, 0));
        *(lds_u32x4*)(uintptr_t)(tile + (uint32_t)(row * kPitch + ch * 16)) = v;
      }
    } else {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int row = q * 16 + (lane >> 2), ch = lane & 3;
        const int64_t m = (int64_t)st * 32 + row;
        const u32x4 c = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
            rs, (int)(m * p.s.ld) + ch * 16, 0, 0));
        const float sc = act8_scale(__builtin_amdgcn_raw_buffer_load_b8(rsc, (int)(m * p.s.sld), 0, 0));
        u32x4 lo = act8_decode8<kSrc>(u32x2{c[0], c[1]}, sc);
        u32x4 hi = act8_decode8<kSrc>(u32x2{c[2], c[3]}, sc);
        if constexpr (kMask) {
          const uint32_t bits = __builtin_amdgcn_raw_buffer_load_b32(
              rm, (int)(m * mld * 4) + (ch >> 1) * 4, 0, 0) >> ((ch & 1) * 16);
          lo &= keep_mask8(bits);
          hi &= keep_mask8(bits >> 8);
        }
        *(lds_u32x4*)(uintptr_t)(tile + (uint32_t)(row * kPitch + ch * 32)) = lo;
        *(lds_u32x4*)(uintptr_t)(tile + (uint32_t)(row * kPitch + ch * 32 + 16)) = hi;
      }
    }
    bf16x8 v[kTerms][NJ];
#pragma unroll
    for (int t = 0; t < kTerms; ++t)
#pragma unroll
      for (int jt = 0; jt < NJ; ++jt)
        v[t][jt] = as_bf16x8(__builtin_bit_cast(
            u32x4, __builtin_amdgcn_raw_buffer_load_b128(rv, ov[jt] + t * term, st * 64, 0)));
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      const bf16x8 x = tr_frag(tile, 8 * g, f * 16, lane);
#pragma unroll
      for (int jt = 0; jt < NJ; ++jt)
#pragma unroll
        for (int t = kTerms - 1; t >= 0; --t)
          acc[f * NJ + jt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, v[t][jt], acc[f * NJ + jt], 0, 0, 0);
    }
  }
  reduce_waves<NF>(acc, lds, wave, lane);
  if (wave != 0) return;
#pragma unroll
  for (int f = 0; f < 4; ++f)
#pragma unroll
    for (int jt = 0; jt < NJ; ++jt) {
      const int j = j0 + jt * 16 + i;
      if (j >= r) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        p.out[(c0 + f * 16 + g * 4 + e) * p.oc + j * p.oj] = acc[f * NJ + jt][e];
    }
#endif
}

template <int kSrc, bool kMask, int NJ>
__global__ void __launch_bounds__(kThreads) column_products_kernel(ColPair p) {
  constexpr int kRed = kWaves / 2 * 4 * NJ * 1024, kTiles = kWaves * 32 * kPitch;
  __shared__ __attribute__((aligned(16))) uint8_t smem[kTiles > kRed ? kTiles : kRed];
  const uint32_t lds = (uint32_t)(uintptr_t)((__attribute__((address_space(3))) uint8_t*)smem);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int b = blockIdx.x, j0 = blockIdx.y * 64;
  if (b < p.ta) column_product<kSrc, kMask, NJ>(p.a, b, j0, p.Mp, p.r, p.rp, lds, wave, lane);
  else column_product<kBf16, false, NJ>(p.b, b - p.ta, j0, p.Mp, p.r, p.rp, lds, wave, lane);
}

}  // namespace lr8

using namespace lr8;

namespace {

constexpr int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Splits of a row product's contraction across workgroups: enough for about
// one workgroup per compute unit, each with a step for every wave.
int row_splits(int64_t M, int64_t C, int r) {
  const int64_t tiles = ceil_div(M, 64) * ceil_div(r, 64), steps = ceil_div(C, 64);
  const int64_t s = std::max<int64_t>(1, std::min(256 / tiles, steps / kWaves));
  return (int)ceil_div(steps, ceil_div(steps, s));
}

template <class F>
hipError_t by_nj(int r, F&& f) {
  using std::integral_constant;
  if (r <= 16) return f(integral_constant<int, 1>{});
  if (r <= 32) return f(integral_constant<int, 2>{});
  return f(integral_constant<int, 4>{});
}

template <int kSrc, bool kMask, bool kTrans>
hipError_t run_rows(RowProd p, int splits, hipStream_t stream) {
  return by_nj(p.r, [&](auto nj) {
    auto kern = row_product_kernel<kSrc, kMask, kTrans, decltype(nj)::value>;
    hipLaunchKernelGGL(kern, dim3((unsigned)(p.tiles * splits), (unsigned)ceil_div(p.r, 64)),
                       dim3(kThreads), 0, stream, p);
    return hipGetLastError();
  });
}

RowProd row_args(Stream s, const uint16_t* w, int r, float* part, int* splits) {
  RowProd p{};
  p.s = s;
  p.w = w;
  p.r = r;
  p.wvec = r % 8 == 0 && (reinterpret_cast<uintptr_t>(w) & 15) == 0;
  p.steps = (int)ceil_div(s.cols, 64);
  *splits = row_splits(s.rows, s.cols, r);
  p.per = (int)ceil_div(p.steps, *splits);
  p.ldp = lowrank_cols(r);
  p.part = part;
  p.tiles = (int)ceil_div(s.rows, 64);
  return p;
}

Stream act8_stream(ConstAct8 x, int64_t M, int64_t K, const uint32_t* mask) {
  return Stream{x.codes, x.scales, act8_row_bytes(K), act8_scale_row_bytes(K), M, K, mask};
}

}  // namespace

int lowrank_cols(int r) { return r <= 16 ? 16 : r <= 32 ? 32 : (int)ceil_div(r, 64) * 64; }

hipError_t launch_rows_act8(ConstAct8 x, int fmt, int64_t M, int64_t K, const uint32_t* mask,
                            const uint16_t* A, int r, float* part, int* splits, hipStream_t stream) {
  const RowProd p = row_args(act8_stream(x, M, K, mask), A, r, part, splits);
  if (mask) return fmt ? run_rows<kE5M2, true, true>(p, *splits, stream) : run_rows<kE4M3, true, true>(p, *splits, stream);
  return fmt ? run_rows<kE5M2, false, true>(p, *splits, stream) : run_rows<kE4M3, false, true>(p, *splits, stream);
}

hipError_t launch_rows_bf16(const uint16_t* S, int64_t M, int64_t C, const uint16_t* B, int r,
                            float* part, int* splits, hipStream_t stream) {
  const RowProd p = row_args(Stream{S, nullptr, C * 2, 0, M, C, nullptr}, B, r, part, splits);
  return run_rows<kBf16, false, false>(p, *splits, stream);
}

hipError_t launch_lowrank_out(const LowrankOut* o, int n, LowrankPad pad, int64_t M, int r, float s,
                              hipStream_t stream) {
  OutArgs p{};
  p.M = M;
  p.Mp = ceil_div(M, 64) * 64;
  p.r = r;
  p.r64 = ceil_div(r, 64) * 64;
  p.rp = lowrank_cols(r);
  p.s = s;
  p.mtiles = (int)ceil_div(M, 64);
  for (int i = 0; i < n; ++i)
    p.o[i] = OutJob{o[i].part, o[i].splits, o[i].ldp, o[i].f, o[i].out32, o[i].u, o[i].v3};
  p.pad = PadJob{pad.src, pad.columns, pad.rows, pad.dst};
  p.blocks0 = p.mtiles;
  p.blocks1 = n > 1 ? p.mtiles : 0;
  const int64_t blocks = p.blocks0 + p.blocks1 + (pad.src ? ceil_div(pad.rows, 64) : 0);
  hipLaunchKernelGGL(lowrank_out_kernel, dim3((unsigned)blocks, (unsigned)(p.r64 / 64)),
                     dim3(kOutThreads), 0, stream, p);
  return hipGetLastError();
}

hipError_t launch_columns(ConstAct8 x, int fmt, const uint32_t* mask, const uint16_t* dY,
                          const uint16_t* g3, const uint16_t* t3, int64_t M, int64_t N, int64_t K,
                          int r, float* dA, float* dB, hipStream_t stream) {
  ColPair p{};
  p.a = ColProd{act8_stream(x, M, K, mask), g3, dA, (int64_t)r, 1};
  p.b = ColProd{Stream{dY, nullptr, N * 2, 0, M, N, nullptr}, t3, dB, 1, N};
  p.ta = (int)(K / 64);
  p.Mp = ceil_div(M, 64) * 64;
  p.r = r;
  p.rp = lowrank_cols(r);
  const dim3 grid((unsigned)(K / 64 + N / 64), (unsigned)ceil_div(r, 64)), block(kThreads);
  return by_nj(r, [&](auto nj) {
    constexpr int NJ = decltype(nj)::value;
    auto go = [&](auto kern) {
      hipLaunchKernelGGL(kern, grid, block, 0, stream, p);
      return hipGetLastError();
    };
    if (mask) return fmt ? go(column_products_kernel<kE5M2, true, NJ>) : go(column_products_kernel<kE4M3, true, NJ>);
    return fmt ? go(column_products_kernel<kE5M2, false, NJ>) : go(column_products_kernel<kE4M3, false, NJ>);
  });
}

}  // namespace qlora
