// Device helpers of the 8-bit block format (include/qlora.h, "8-bit blocks"):
// codes in E4M3 or E5M2, one power-of-two scale 2^e per block of 128, kept
// as the byte e + 127.
#pragma once

#include "common.h"

namespace qlora {

constexpr int kAct8Block = 128;
constexpr int kAct8MinByte = 127 - 110;  // scale byte of e = -110

// Bytes of one row of codes, and of its scales: K rounded up to whole
// blocks, and the block count rounded up to a whole dword.
__host__ __device__ constexpr int64_t act8_row_bytes(int64_t K) {
  return (K + kAct8Block - 1) / kAct8Block * kAct8Block;
}
__host__ __device__ constexpr int64_t act8_scale_row_bytes(int64_t K) {
  return ((K + kAct8Block - 1) / kAct8Block + 3) / 4 * 4;
}

// An offset past every range that the products read through a buffer descriptor
// (a tile of 256 rows, or an adapter matrix of 256): a load there gives zeros. A
// tile's row offset, up to 48 rows, may come on top and leaves it in 31 bits.
constexpr int kPastEnd = 0x70000000;
constexpr int64_t kMaxRowBytes = (int64_t)2 << 21;  // bf16, the longest row the calls take
static_assert(kPastEnd >= 256 * kMaxRowBytes && kPastEnd + 48 * kMaxRowBytes <= 0x7fffffff, "past every tile, 31 bits");

typedef short s16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Scale byte of a block whose largest finite magnitude has the bf16 bits
// `amax` (sign cleared): the least e with amax <= 1.75 * 2^(e + top), at
// least -110. With amax = (1 + f / 128) 2^(E - 127) that is
// e = E - 127 - top, plus one when f > 96.
template <int kFmt>
__device__ __forceinline__ int act8_scale_byte(uint32_t amax) {
  constexpr int kTop = kFmt ? 15 : 8;
  const int b = (int)(amax >> 7) - kTop + ((amax & 127u) > 96u ? 1 : 0);
  return b < kAct8MinByte ? kAct8MinByte : b;
}
__device__ __forceinline__ float act8_scale(int byte) {
  return __builtin_bit_cast(float, (uint32_t)byte << 23);
}

// Two bf16 values (bits) to two codes of x / scale, in the low or high half
// of `old`; nearest, ties to even. One conversion instruction.
template <int kFmt, bool kHigh>
__device__ __forceinline__ s16x2 act8_encode2(s16x2 old, uint32_t x, float scale) {
  const bf16x2 v = __builtin_bit_cast(bf16x2, x);
  if constexpr (kFmt == 0) return __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(old, v, scale, kHigh);
  else return __builtin_amdgcn_cvt_scalef32_pk_bf8_bf16(old, v, scale, kHigh);
}
// Eight bf16 values to eight codes.
template <int kFmt>
__device__ __forceinline__ u32x2 act8_encode8(u32x4 x, float scale) {
  s16x2 a = {0, 0}, b = {0, 0};
  a = act8_encode2<kFmt, false>(a, x[0], scale);
  a = act8_encode2<kFmt, true>(a, x[1], scale);
  b = act8_encode2<kFmt, false>(b, x[2], scale);
  b = act8_encode2<kFmt, true>(b, x[3], scale);
  return u32x2{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b)};
}
// Four codes to four bf16 values (exact: a code has at most 4 significant
// bits, and e >= -110 keeps the value a normal bf16).
template <int kFmt>
__device__ __forceinline__ u32x2 act8_decode4(uint32_t c, float scale) {
  bf16x2 lo, hi;
  if constexpr (kFmt == 0) {
    lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, scale, false);
    hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, scale, true);
  } else {
    lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(c, scale, false);
    hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(c, scale, true);
  }
  return u32x2{__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
}
template <int kFmt>
__device__ __forceinline__ u32x4 act8_decode8(u32x2 c, float scale) {
  const u32x2 a = act8_decode4<kFmt>(c[0], scale), b = act8_decode4<kFmt>(c[1], scale);
  return u32x4{a[0], a[1], b[0], b[1]};
}

// bf16 bits of |x| where finite, else 0, of both halves of a word.
__device__ __forceinline__ uint32_t finite_abs2(uint32_t x) {
  const uint32_t lo = x & 0x7fffu, hi = x & 0x7fff0000u;
  return (lo < 0x7f80u ? lo : 0u) | (hi < 0x7f800000u ? hi : 0u);
}
// Largest of eight magnitudes (two 16-bit maxima side by side, then one).
__device__ __forceinline__ uint32_t finite_max8(u32x4 x) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = finite_abs2(x[i]);
    m = max(m, max(a & 0xffffu, a >> 16));
  }
  return m;
}
// Maximum over the 16 lanes of a DPP row, in every lane of the row.
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
  auto step = [](uint32_t a, uint32_t b) { return a > b ? a : b; };
  v = step(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xb1, 0xf, 0xf, true));   // quad xor 1
  v = step(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4e, 0xf, 0xf, true));   // quad xor 2
  v = step(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xf, 0xf, true));  // half mirror
  v = step(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xf, 0xf, true));  // mirror
  return v;
}

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// The eight transposed elements of a fragment from a row-major tile of bf16 in
// LDS, rows kPitch bytes apart: lane l
// receives column (l & 15) + c0 and rows r0 .. r0 + 7 of its own 16-lane
// group's row base.
template <int kPitch>
__device__ __forceinline__ bf16x8 tr_frag(uint32_t tile, int row0, int c0, int lane) {
  const int p = lane & 15;
  const uint32_t a = tile + (uint32_t)((row0 + (p >> 2)) * kPitch + (c0 + (p & 3) * 4) * 2);
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(uintptr_t)a);
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(uintptr_t)(a + 4 * kPitch));
  const u32x2 l2 = __builtin_bit_cast(u32x2, lo), h2 = __builtin_bit_cast(u32x2, hi);
  return as_bf16x8(u32x4{l2[0], l2[1], h2[0], h2[1]});
}

// Eight bf16 of a row at column c (zero past `cols`).
template <bool kVec>
__device__ __forceinline__ u32x4 load8(const uint16_t* row, int64_t c, int64_t cols) {
  u32x4 v = {0u, 0u, 0u, 0u};
  if (c + 8 <= cols) {
    if constexpr (kVec) return *reinterpret_cast<const u32x4*>(row + c);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = (uint32_t)row[c + 2 * i] | ((uint32_t)row[c + 2 * i + 1] << 16);
    return v;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c + i < cols) v[i >> 1] |= (uint32_t)row[c + i] << (16 * (i & 1));
  return v;
}
template <bool kVec>
__device__ __forceinline__ void store8(uint16_t* row, int64_t c, int64_t cols, u32x4 v) {
  if (kVec && c + 8 <= cols) {
    *reinterpret_cast<u32x4*>(row + c) = v;
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c + i < cols) row[c + i] = (uint16_t)(v[i >> 1] >> (16 * (i & 1)));
}

// Scale byte of block kb of a row; the row's last block also clears the
// bytes up to the padded row end. Called by one lane of the block.
__device__ __forceinline__ void put_scale(uint8_t* row, int kb, int KB, int sb, int byte) {
  row[kb] = (uint8_t)byte;
  if (kb == KB - 1)
    for (int i = KB; i < sb; ++i) row[i] = 0;
}

// One block's codes from its lane's eight bf16 values.
template <int kFmt>
__device__ __forceinline__ void put_block(u32x4 x, uint32_t b, int kb, int KB, int sb, int64_t row,
                                          uint8_t* codes, uint8_t* scales) {
  const int l = threadIdx.x & 15;
  const int byte = act8_scale_byte<kFmt>(row16_max(finite_max8(x)));
  const u32x2 c = act8_encode8<kFmt>(x, act8_scale(byte));
  *reinterpret_cast<u32x2*>(codes + (int64_t)b * kAct8Block + l * 8) = c;
  if (l == 0) put_scale(scales + row * sb, kb, KB, sb, byte);
}

// Block b of the 8-bit blocks of X, in flat order b = row * KB + column block,
// by the sixteen lanes that call with it.
template <int kFmt, bool kVec>
__device__ __forceinline__ void act8_quantize_block(const uint16_t* X, int64_t ldx, int64_t K, uint32_t b,
                                                    int KB, int sb, uint8_t* codes, uint8_t* scales) {
  const uint32_t row = b / (uint32_t)KB;
  const int kb = (int)(b - row * (uint32_t)KB);
  const int64_t c = (int64_t)kb * kAct8Block + (threadIdx.x & 15) * 8;
  put_block<kFmt>(load8<kVec>(X + (int64_t)row * ldx, c, K), b, kb, KB, sb, row, codes, scales);
}

}  // namespace qlora
