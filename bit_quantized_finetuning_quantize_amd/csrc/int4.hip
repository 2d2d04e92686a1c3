// Weights in 4 bits with a scale and a zero point for each group of 32, 64 or
// 128 columns of a row, w = s (q - z): quantization, decoding, and the product
// of few tokens with them.
#include "common.h"
#include "kernels.h"

#include <algorithm>
#include <atomic>
#include <type_traits>

namespace qlora {

namespace {

constexpr int kThreads = 256;

typedef u32x4 u32x4_row __attribute__((aligned(2)));

__device__ __forceinline__ uint32_t bits_of(float f) { return __builtin_bit_cast(uint32_t, f); }
// bf16(f), as a float.
__device__ __forceinline__ float to_bf16(float f) { return bf16_lo(pack_bf16x2(f, 0.0f)); }

// Largest with that of another lane (update_dpp's control).
template <int kCtrl>
__device__ __forceinline__ uint32_t max_dpp(uint32_t v) {
  const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, 0xf, 0xf, true);
  return v > o ? v : o;
}

// Row and group of flat group index b = first + i, first the same in the whole
// workgroup and i below kPer: a scalar division unless rows are short.
template <uint32_t kPer>
__device__ __forceinline__ void split_index(uint32_t first, uint32_t i, uint32_t ng, uint32_t& row, uint32_t& g) {
  if (ng >= kPer) {
    row = first / ng;
    g = first - row * ng + i;
    if (g >= ng) {
      g -= ng;
      ++row;
    }
  } else {
    row = (first + i) / ng;
    g = first + i - row * ng;
  }
}

// ---------------------------------------------------------------------------
// Quantization: kG / 16 lanes own a group, two vectors of eight values each, so that
// what a group costs once is shared by 16 values.
//   asymmetric  lo = min(w, 0), hi = max(w, 0), s = bf16((hi - lo) / 15),
//               z = rint(-lo / s) in [0, 15]
//   symmetric   s = bf16(max|w| / 7), z = 8
//   q = rint(w / s) + z in [0, 15]; where s = 0, z = 0 (symmetric 8) and q = z.
// Bounded by memory: 4096 x 11008 in groups of 128 24 us, 4.8 TB/s, a copy's rate
// (with 8 values to a lane, a division to each value and shifts 43).
template <int kG, bool kSym>
__global__ void __launch_bounds__(kThreads)
int4_quantize_kernel(const uint16_t* __restrict__ W, int64_t ldw, int K, uint32_t ng, uint32_t groups,
                     uint8_t* __restrict__ codes, uint16_t* __restrict__ scales, uint8_t* __restrict__ zeros) {
#pragma clang fp contract(off)
  constexpr uint32_t kLanes = kG / 16, kPer = kThreads / kLanes;
  const uint32_t first = blockIdx.x * kPer, b = first + threadIdx.x / kLanes;
  if (b >= groups) return;
  const uint32_t l = threadIdx.x % kLanes;
  uint32_t row, g;
  split_index<kPer>(first, threadIdx.x / kLanes, ng, row, g);
  const int col = (int)(g * kG + l * 8);  // and kG / 2 columns on
  const uint16_t* w = W + (int64_t)row * ldw + col;
  u32x4 v[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (col + h * (kG / 2) < K) v[h] = *reinterpret_cast<const u32x4_row*>(w + h * (kG / 2));
  float x[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t p = v[i / 4][i % 4];
    x[2 * i] = bf16_lo(p);
    x[2 * i + 1] = bf16_hi(p);
  }
  float lo = 0.0f, hi = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    lo = fminf(lo, x[i]);
    hi = fmaxf(hi, x[i]);
  }
  // -lo and hi over two lanes, four and eight: the bits of numbers
  // that are not negative have their order
  uint32_t lob = bits_of(lo) & 0x7fffffffu, hib = bits_of(hi) & 0x7fffffffu;
  auto join = [&](auto ctrl) {
    lob = max_dpp<decltype(ctrl)::value>(lob);
    hib = max_dpp<decltype(ctrl)::value>(hib);
  };
  join(std::integral_constant<int, 0xb1>{});
  if constexpr (kLanes >= 4) join(std::integral_constant<int, 0x4e>{});
  if constexpr (kLanes >= 8) join(std::integral_constant<int, 0x141>{});
  lo = __builtin_bit_cast(float, lob);  // -lo from here on
  hi = __builtin_bit_cast(float, hib);
  // The quotient by 7 or 15, correctly rounded: the product with the rounded
  // inverse and one step from its exact remainder (a division for values whose
  // remainder float32 does not hold).
  constexpr float kD = kSym ? 7.0f : 15.0f, kInv = 1.0f / kD;
  const float span = kSym ? fmaxf(lo, hi) : hi + lo;
  float s = span * kInv;
  s = __builtin_fmaf(__builtin_fmaf(-kD, s, span), kInv, s);
  if (__any(span < 0x1p-90f)) s = span / kD;
  s = to_bf16(s);
  // rint(x / s) without a division to each value. x and s have 8 significant
  // bits: x / s below 32 is half-way between two integers or at least 2^-10 from
  // it. x times the hardware's inverse (one unit in the last place) is within
  // 2^-17 of x / s; rounded to multiples of 2^-12 it is exactly half-way in the
  // first case, and on the right side in the second. Scales whose inverse
  // float32 does not hold are taken 2^64 times, and the values with them.
  float sk = s;
  if (s < 0x1p-100f) {
    sk *= 0x1p64f;
    lo *= 0x1p64f;
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] *= 0x1p64f;
  }
  const float r = s > 0.0f ? __builtin_amdgcn_rcpf(sk) : 0.0f;
  auto near = [&](float v) { return __builtin_fmaf(v, r, 0x1.8p11f) - 0x1.8p11f; };
  const float z = kSym ? 8.0f : fminf(__builtin_rintf(near(lo)), 15.0f);
  // q - z in [-z, 15 - z], then its integer in the low bits of 1.5 2^23 + q - z
  // (ties to even); the eight integers in one word, modulo 2^32, and z to each
  uint8_t* c = codes + ((int64_t)row * K + col) / 2;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t word = (uint32_t)z * 0x11111111u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float q = __builtin_amdgcn_fmed3f(near(x[8 * h + i]), -z, 15.0f - z) + 0x1.8p23f;
      word += (bits_of(q) << (4 * i)) - (0x4b400000u << (4 * i));
    }
    if (col + h * (kG / 2) < K) *reinterpret_cast<uint32_t*>(c + h * (kG / 4)) = word;
  }
  if (l == 0) {
    scales[b] = (uint16_t)(bits_of(s) >> 16);
    if (!kSym) zeros[b] = (uint8_t)z;
  }
}

// bf16(s (q - z)): the product of 8 and 5 bits is exact before that. Bounded by
// memory: 4096 x 11008 19 us, 6.0 TB/s.
template <int kG>
__global__ void __launch_bounds__(kThreads)
int4_dequantize_kernel(const uint8_t* __restrict__ codes, const uint16_t* __restrict__ scales,
                       const uint8_t* __restrict__ zeros, int K, uint32_t ng, uint32_t units,
                       uint16_t* __restrict__ W, int64_t ldw) {
  const uint32_t u = blockIdx.x * kThreads + threadIdx.x;  // eight values
  if (u >= units) return;
  const uint32_t per = (uint32_t)K / 8;
  const int64_t row = u / per;
  const int col = (int)(u % per) * 8;
  const uint32_t b = (uint32_t)row * ng + col / kG;
  const uint32_t w = *reinterpret_cast<const uint32_t*>(codes + (row * K + col) / 2);
  const float s = bf16_to_f32(scales[b]), z = zeros ? (float)(zeros[b] & 15u) : 8.0f;
  u32x4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = pack_bf16x2(((float)((w >> (8 * i)) & 15u) - z) * s, ((float)((w >> (8 * i + 4)) & 15u) - z) * s);
  *reinterpret_cast<u32x4_row*>(W + row * ldw + col) = v;
}

// ---------------------------------------------------------------------------
// Y [M x N] = X [M x K] W^T. A workgroup owns 16 kNR weight rows and 16 kMT
// tokens over the whole K, its waves taking steps of 128 kRuns columns in turn,
// the next step's loads in flight while one is computed.
//
// Loads are of whole lines, four neighbouring lanes to 64 bytes of a row, and
// the values reach the lanes that multiply them, (c, g) = (lane & 15, lane >> 4),
// by way of LDS rows of the wave's own (no barrier: LDS accesses of one wave
// complete in order). Loaded by the lanes that multiply them, 16 bytes each from
// another row than its neighbour's, they took one pass of the memory pipe a
// lane, which bounded the kernel (32768 x 8192, one token: 39 us).
//
// Codes. A lane multiplies 16 bytes of weight row c, the 32 columns at 32 g of
// each run of 128; where a group is shorter, the code words change lanes so
// that the four lanes of a row hold words of one group at a time. They go to
// the matrix units as bf16 integers, without a table: a byte times 0x8008 has
// its two nibbles at bits 3-6 and 19-22, where 0x4180 (16.0) beneath makes them
// 16 + q. A second product with the constant -(16 + z) takes the offset and the
// zero point away, all of it exact up to the float32 sums, and each group's sum
// is scaled in float32.
//
// Rows and tokens past the end repeat the last one; their sums are not stored.
//
// What bounds it (us from a graph, where a launch takes 4). Few tokens: the loads;
// 32768 x 8192, one token, 31 us, 4.6 TB/s, without its sums 28; 4096 x 4096 5.4. More
// tokens: the few steps of each wave, one after the other; 48 x 11008 x 4096 in
// groups of 32 18.6, of which the matrix units work 3.5 and the vector
// instructions 6; in groups of 128 16.2, without the sums 12.3, without the tokens' and
// scales' loads 12.5, without either 8.9. Two steps' loads in flight: 1 x 32768 x
// 8192 29.8 for 30.1, but 2 x 8192 x 8192 14.6 for 12.3.

constexpr int kWaves = 8;

struct Int4Args {
  const uint16_t* X;
  const uint8_t* codes;
  const uint16_t* scales;
  const uint8_t* zeros;  // or null: 8
  int64_t M, N, K, ng, ldx, ldy;
  void* Y;
  int f32;
};

// The code word's eight values 16 + q, in order. mask 0x00780078 and base
// 0x41804180 come in registers: as constants they make two instructions of one
// for want of operands.
__device__ __forceinline__ u32x4 nibbles_bf16(uint32_t w, uint32_t mask, uint32_t base) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = (__umul24((w >> (8 * i)) & 0xffu, 0x8008u) & mask) | base;
  return r;
}

// kBytes (a power of two) at any address, as words (the last one's upper bytes 0).
template <int kBytes>
__device__ __forceinline__ void load_bytes(uint32_t* w, const void* p) {
  typedef uint16_t u16_1 __attribute__((aligned(1)));
  typedef uint32_t u32_1 __attribute__((aligned(1)));
  typedef u32x2 u32x2_1 __attribute__((aligned(1)));
  typedef u32x4 u32x4_1 __attribute__((aligned(1)));
  if constexpr (kBytes == 1) {
    w[0] = *reinterpret_cast<const uint8_t*>(p);
  } else if constexpr (kBytes == 2) {
    w[0] = *reinterpret_cast<const u16_1*>(p);
  } else if constexpr (kBytes == 4) {
    w[0] = *reinterpret_cast<const u32_1*>(p);
  } else if constexpr (kBytes == 8) {
    const u32x2 v = *reinterpret_cast<const u32x2_1*>(p);
    w[0] = v[0];
    w[1] = v[1];
  } else {
#pragma unroll
    for (int n = 0; n < kBytes / 16; ++n) {
      const u32x4 v = *(reinterpret_cast<const u32x4_1*>(p) + n);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[4 * n + i] = v[i];
    }
  }
}

__device__ __forceinline__ void load_lds(uint32_t (&w)[4], const uint8_t* p) {
  const u32x4 v = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = v[i];
}

// Swaps the upper 32 lanes of a with the lower 32 of b; the odd rows of 16
// lanes of a with the even ones of b.
__device__ __forceinline__ void swap32(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}
__device__ __forceinline__ void swap16(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}

// First column, within a run, of the eight of lane group g in product t (of
// four): those of its own code word t, or of the word that comes to it.
template <int kG>
__device__ __forceinline__ int column_of(int t, int g) {
  if constexpr (kG == 128) return 32 * g + 8 * t;
  if constexpr (kG == 64) return 64 * (t >> 1) + 32 * (g & 1) + 16 * (g >> 1) + 8 * (t & 1);
  return 32 * t + 8 * g;
}
template <int kG>
__device__ __forceinline__ void to_groups(uint32_t (&w)[4]) {
  if constexpr (kG < 128) {
    swap32(w[0], w[2]);
    swap32(w[1], w[3]);
  }
  if constexpr (kG == 32) {
    swap16(w[0], w[1]);
    swap16(w[2], w[3]);
  }
}

// Where a lane loads and what LDS bytes it takes its operands from.
template <int kX, int kNR>
struct Lane {
  uint32_t code[kNR];   // byte of its first code
  uint32_t group[kNR];  // its row's first group
  int token[kX];        // byte in x of its first value of each load
  __amdgpu_buffer_rsrc_t x;
  uint32_t put;      // of its first load's token values
  uint32_t get[4];   // of its token operands in a run
  uint32_t code_get; // of its codes in a run
  int from;          // the lane, times 4, that loads its row's scales
};

// Four lanes load a row's 64 bytes of a run; lane i of them takes piece
// i ^ swizzle(row), so that the reads, one piece of 16 rows, spread over the
// banks.
__device__ __forceinline__ int swizzle(int row) { return (row >> 2) & 3; }

template <int kG, int kMT, int kNR, int kRuns, int kX>
struct Int4Step {
  static constexpr int kColumns = 128 * kRuns;
  static constexpr int kGroups = kColumns / kG;
  static constexpr int kPitch = kColumns * 2 + 16;  // LDS bytes of a token's row
  static constexpr int kPer = 512 / kColumns;       // tokens of a load
  static constexpr int kTokenLds = kX * kPer * kPitch;
  static constexpr int kLds = kTokenLds + kNR * kRuns * 1024;  // of a wave: tokens, codes
  using At = Lane<kX, kNR>;
  struct Scales {
    uint32_t s[kNR][(kGroups + 1) / 2], z[kNR][(kGroups + 3) / 4];
  };
  uint32_t w[kNR][kRuns][4];
  uint32_t s[kNR][(kGroups + 1) / 2], z[kNR][(kGroups + 3) / 4];
  u32x4 x[kX];

  // kTail: the end of the rows; what lies past it is 0.
  template <bool kTail>
  __device__ __forceinline__ void load(const Int4Args& a, int k0, const At& at, int lane) {
    const int K = (int)a.K;
    const uint8_t* codes = a.codes + k0 / 2;
    const uint16_t* scales = a.scales + k0 / kG;
    const uint8_t* zeros = a.zeros + k0 / kG;
#pragma unroll
    for (int r = 0; r < kNR; ++r) {
#pragma unroll
      for (int n = 0; n < kRuns; ++n) {
        if (kTail && k0 + 128 * n + 32 * ((lane & 3) ^ swizzle(lane >> 2)) >= K) {
#pragma unroll
          for (int e = 0; e < 4; ++e) w[r][n][e] = 0;
        } else {
          load_bytes<16>(w[r][n], codes + at.code[r] + n * 64);
        }
      }
      if constexpr (kTail) {
#pragma unroll
        for (int j = 0; j < kGroups; ++j) {
          if (j % 2 == 0) s[r][j / 2] = 0;
          if (j % 4 == 0) z[r][j / 4] = 0;
          if (k0 + kG * j < K) {
            s[r][j / 2] |= (uint32_t)scales[at.group[r] + j] << (16 * (j & 1));
            z[r][j / 4] |= (a.zeros ? (uint32_t)zeros[at.group[r] + j] : 8u) << (8 * (j & 3));
          }
        }
      } else {
        load_bytes<kGroups * 2>(s[r], scales + at.group[r]);
#pragma unroll
        for (int j = 0; j < (kGroups + 3) / 4; ++j) z[r][j] = 0x08080808u;
        if (a.zeros) load_bytes<kGroups>(z[r], zeros + at.group[r]);
      }
    }
    const bool in = !kTail || k0 + (lane % (kColumns / 8)) * 8 < K;
#pragma unroll
    for (int m = 0; m < kX; ++m) {
      if (kTail) x[m] = u32x4{0, 0, 0, 0};
      if (in) x[m] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(at.x, at.token[m], k0 * 2, 0));
    }
  }

  // The loaded values to the wave's LDS, its rows' scales and zero points to cur.
  __device__ __forceinline__ void stage(const At& at, uint8_t* lds, int lane, Scales& cur) const {
    uint8_t* lds_codes = lds + kTokenLds;
    asm volatile("" ::: "memory");
#pragma unroll
    for (int r = 0; r < kNR; ++r)
#pragma unroll
      for (int n = 0; n < kRuns; ++n)
        *reinterpret_cast<u32x4*>(lds_codes + (r * kRuns + n) * 1024 + lane * 16) =
            u32x4{w[r][n][0], w[r][n][1], w[r][n][2], w[r][n][3]};
#pragma unroll
    for (int m = 0; m < kX; ++m) *reinterpret_cast<u32x4*>(lds + at.put + m * (kPer * kPitch)) = x[m];
#pragma unroll
    for (int r = 0; r < kNR; ++r) {
#pragma unroll
      for (int j = 0; j < (kGroups + 1) / 2; ++j) cur.s[r][j] = __builtin_amdgcn_ds_bpermute(at.from, s[r][j]);
#pragma unroll
      for (int j = 0; j < (kGroups + 3) / 4; ++j) cur.z[r][j] = __builtin_amdgcn_ds_bpermute(at.from, z[r][j]);
    }
    asm volatile("" ::: "memory");
  }

  __device__ __forceinline__ static void add(floatx4 (&acc)[kMT][kNR], const At& at, const uint8_t* lds,
                                             const Scales& cur, uint32_t mask, uint32_t base) {
    const floatx4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
    const uint8_t* lds_codes = lds + kTokenLds;
#pragma unroll
    for (int n = 0; n < kRuns; ++n) {
      bf16x8 t[kMT][4];
#pragma unroll
      for (int m = 0; m < kMT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          t[m][i] = as_bf16x8(*reinterpret_cast<const u32x4*>(lds + at.get[i] + m * (16 * kPitch) + n * 256));
#pragma unroll
      for (int r = 0; r < kNR; ++r) {
        uint32_t c[4];
        load_lds(c, lds_codes + (r * kRuns + n) * 1024 + at.code_get);
        to_groups<kG>(c);
        floatx4 p[kMT];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = (128 * n + 32 * i) / kG;  // the product's group
          const bool begins = (32 * i) % kG == 0, ends = (32 * (i + 1)) % kG == 0;
          const uint32_t off = (0xc180u | (((cur.z[r][j / 4] >> (8 * (j & 3))) & 15u) << 3)) * 0x10001u;  // -(16 + z), twice
          const bf16x8 of = as_bf16x8(u32x4{off, off, off, off});
          const bf16x8 q = as_bf16x8(nibbles_bf16(c[i], mask, base));
#pragma unroll
          for (int m = 0; m < kMT; ++m) {
            p[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(t[m][i], q, begins ? zero : p[m], 0, 0, 0);
            p[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(t[m][i], of, p[m], 0, 0, 0);
          }
          if (ends) {
            const uint32_t sw = cur.s[r][j / 2];
            const float sc = (j & 1) ? bf16_hi(sw) : bf16_lo(sw);
#pragma unroll
            for (int m = 0; m < kMT; ++m)
#pragma unroll
              for (int v = 0; v < 4; ++v) acc[m][r][v] = __builtin_fmaf(sc, p[m][v], acc[m][r][v]);
          }
        }
      }
    }
    asm volatile("" ::: "memory");
  }
};

template <int kG, int kMT, int kNR, int kRuns, int kX>
__global__ void __launch_bounds__(kWaves * 64) int4_linear_kernel(Int4Args a) {
  using Step = Int4Step<kG, kMT, kNR, kRuns, kX>;
  constexpr int kColumns = Step::kColumns, kPitch = Step::kPitch;
  extern __shared__ __attribute__((aligned(16))) uint8_t s_mem[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * kNR), m0 = (int64_t)blockIdx.y * (16 * kMT);
  const int K = (int)a.K;
  uint8_t* lds = s_mem + wave * Step::kLds;
  typename Step::At at;
  at.x = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(a.X), (short)0, (int)(((a.M - 1) * a.ldx + K) * 2), 0x00020000);
  {
    const int row = lane >> 2, piece = (lane & 3) ^ swizzle(row);
#pragma unroll
    for (int r = 0; r < kNR; ++r) {
      const int64_t n = n0 + 16 * r + row < a.N ? n0 + 16 * r + row : a.N - 1;
      at.code[r] = (uint32_t)(n * K / 2) + 16 * piece;
      at.group[r] = (uint32_t)(n * a.ng);
    }
    at.from = c * 16;  // lane 4 c
    at.code_get = (uint32_t)(c * 64 + (g ^ swizzle(c)) * 16);
    constexpr int kLanes = kColumns / 8;  // lanes to a token's row
#pragma unroll
    for (int m = 0; m < kX; ++m) {
      const int64_t t = m0 + m * Step::kPer + lane / kLanes;
      at.token[m] = (int)(((t < a.M ? t : a.M - 1) * a.ldx + (lane % kLanes) * 8) * 2);
    }
    at.put = (uint32_t)((lane / kLanes) * kPitch + (lane % kLanes) * 16);
    // fewer tokens than 16 are loaded where kX kPer is less: the last repeats
    const int t = kX * Step::kPer < 16 && c >= kX * Step::kPer ? kX * Step::kPer - 1 : c;
#pragma unroll
    for (int i = 0; i < 4; ++i) at.get[i] = (uint32_t)(t * kPitch + column_of<kG>(i, g) * 2);
  }
  floatx4 acc[kMT][kNR];
#pragma unroll
  for (int m = 0; m < kMT; ++m)
#pragma unroll
    for (int r = 0; r < kNR; ++r) acc[m][r] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};

  uint32_t mask = 0x00780078u, base = 0x41804180u;
  asm("" : "+v"(mask));
  asm("" : "+s"(base));
  const int whole = K / kColumns;                         // steps; this wave's are wave, wave + kWaves, ...
  const int left = (whole - wave + kWaves - 1) / kWaves;  // ... so many
  auto column = [&](int i) { return (wave + i * kWaves) * kColumns; };
  Step step;
  typename Step::Scales cur;
  if (left > 0) step.template load<false>(a, column(0), at, lane);
  for (int i = 0; i < left; ++i) {
    step.stage(at, lds, lane, cur);
    if (i + 1 < left) step.template load<false>(a, column(i + 1), at, lane);
    __builtin_amdgcn_sched_barrier(0);  // the loads stay ahead of the sums
    Step::add(acc, at, lds, cur, mask, base);
  }
  if (whole * kColumns < K && wave == whole % kWaves) {
    step.template load<true>(a, whole * kColumns, at, lane);
    step.stage(at, lds, lane, cur);
    Step::add(acc, at, lds, cur, mask, base);
  }
  // the waves' sums, added in the order of the waves; lane (c, g) holds tokens
  // 4 g .. 4 g + 3 of weight row c
  constexpr int kSums = kMT * kNR;
  floatx4* s_red = reinterpret_cast<floatx4*>(s_mem);
  __syncthreads();  // the steps' LDS is done with
#pragma unroll
  for (int i = 0; i < kSums; ++i) s_red[(wave * kSums + i) * 64 + lane] = acc[i / kNR][i % kNR];
  __syncthreads();
  for (int i = wave; i < kSums; i += kWaves) {
    floatx4 y = s_red[i * 64 + lane];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) {
      const floatx4 u = s_red[(w * kSums + i) * 64 + lane];
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

template <int kG, int kMT, int kNR, int kRuns, int kX>
hipError_t run_linear(const Int4Args& a, hipStream_t stream) {
  using Step = Int4Step<kG, kMT, kNR, kRuns, kX>;
  constexpr int kLds = kWaves * std::max(Step::kLds, kMT * kNR * 1024);
  static_assert(kLds <= 160 * 1024);
  auto kern = int4_linear_kernel<kG, kMT, kNR, kRuns, kX>;
  if constexpr (kLds > 65536) {  // the limit on dynamic LDS, raised once per device
    static std::atomic<uint64_t> raised{0};
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(raised.load(std::memory_order_acquire) & bit)) {
      e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
      if (e != hipSuccess) return e;
      raised.fetch_or(bit, std::memory_order_acq_rel);
    }
  }
  const dim3 grid((unsigned)((a.N + 16 * kNR - 1) / (16 * kNR)), (unsigned)((a.M + 16 * kMT - 1) / (16 * kMT)));
  kern<<<grid, dim3(kWaves * 64), kLds, stream>>>(a);
  return hipGetLastError();
}

// Workgroups of 16 kNR weight rows and 16 kMT tokens.
int64_t blocks(const Int4Args& a, int kMT, int kNR) {
  return ((a.N + 16 * kNR - 1) / (16 * kNR)) * ((a.M + 16 * kMT - 1) / (16 * kMT));
}
constexpr int64_t kUnits = 256;  // compute units, each of which holds one

// 16, 32 or 48 weight rows to a workgroup: as few as leave one workgroup to a
// compute unit, since every workgroup reads all of its tokens (us from a graph,
// with 16, 32 and 48: 48 tokens x 11008 x 4096 25.3, 24.9, 18.8; x 4096 x 4096
// 10.4, 12.2, 14.5; 16 x 11008 x 4096 11.8, 12.6, 11.1). Four tokens or fewer
// cost little to read, and 16 rows do better at any size (4 x 11008 x 4096 8.9,
// 10.1, 9.3). Up to 16 tokens with 16 weight rows, each step takes two runs of 128
// columns if every wave has two such steps (one run and two: 8 x 4096 x 4096 6.1,
// 5.2; 12 x 4096 x 11008 12.6, 10.8; 5 x 1001 x 1504 3.5, 3.8).
template <int kG, int kMT, int kX>
hipError_t run_rows(const Int4Args& a, hipStream_t stream) {
  if (blocks(a, kMT, 1) <= kUnits) {
    if constexpr (kMT == 1)
      if (a.K >= 2 * kWaves * 256) return run_linear<kG, kMT, 1, 2, 2 * kX>(a, stream);
    return run_linear<kG, kMT, 1, 1, kX>(a, stream);
  }
  if (blocks(a, kMT, 2) <= kUnits) return run_linear<kG, kMT, 2, 1, kX>(a, stream);
  return run_linear<kG, kMT, 3, 1, kX>(a, stream);
}
// More tokens than 48: 64 of them with 16 or 32 weight rows (48 do not fit the
// registers), or 32 with 48, whose workgroups take 4/5 of the time of 64 with 32
// and are the better choice if they come in few rounds more (us with 64 x 32 and
// 32 x 48: 64 x 11008 x 4096 26.8, 21.8; 64 x 32768 x 8192 98, 112; 128 x 8192 x
// 4096 26.5, 33.5).
template <int kG>
hipError_t run_many(const Int4Args& a, hipStream_t stream) {
  const auto rounds = [&](int kMT, int kNR) { return (blocks(a, kMT, kNR) + kUnits - 1) / kUnits; };
  if (blocks(a, 4, 1) <= kUnits) return run_linear<kG, 4, 1, 1, 16>(a, stream);
  if (5 * rounds(4, 2) <= 4 * rounds(2, 3)) return run_linear<kG, 4, 2, 1, 16>(a, stream);
  return run_linear<kG, 2, 3, 1, 8>(a, stream);
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
  const int64_t ng = (K + group - 1) / group, groups = N * ng, per = kThreads * 16 / group;
  return by_group(group, [&](auto g) {
    constexpr int kG = decltype(g)::value;
    const dim3 grid((unsigned)((groups + per - 1) / per));
    if (zeros)
      int4_quantize_kernel<kG, false><<<grid, dim3(kThreads), 0, stream>>>(W, ldw, (int)K, (uint32_t)ng, (uint32_t)groups, codes, scales, zeros);
    else
      int4_quantize_kernel<kG, true><<<grid, dim3(kThreads), 0, stream>>>(W, ldw, (int)K, (uint32_t)ng, (uint32_t)groups, codes, scales, zeros);
    return hipGetLastError();
  });
}

hipError_t launch_int4_dequantize(const Int4Weight& w, uint16_t* out, int64_t ldo, hipStream_t stream) {
  const int64_t units = w.N * w.K / 8;
  return by_group(w.group, [&](auto g) {
    constexpr int kG = decltype(g)::value;
    int4_dequantize_kernel<kG><<<dim3((unsigned)((units + kThreads - 1) / kThreads)), dim3(kThreads), 0, stream>>>(
        w.codes, w.scales, w.zeros, (int)w.K, (uint32_t)((w.K + kG - 1) / kG), (uint32_t)units, out, ldo);
    return hipGetLastError();
  });
}

hipError_t launch_int4_linear_fwd(const uint16_t* X, int64_t M, int64_t ldx, const Int4Weight& w, void* Y, bool f32,
                                  int64_t ldy, hipStream_t stream) {
  Int4Args a{X, w.codes, w.scales, w.zeros, M, w.N, w.K, (w.K + w.group - 1) / w.group, ldx, ldy, Y, f32};
  return by_group(w.group, [&](auto g) {
    constexpr int kG = decltype(g)::value;
    if (M <= 2) return run_linear<kG, 1, 1, 2, 1>(a, stream);
    if (M <= 4) return run_linear<kG, 1, 1, 2, 2>(a, stream);
    if (M <= 8) return run_rows<kG, 1, 2>(a, stream);
    if (M <= 16) return run_rows<kG, 1, 4>(a, stream);
    if (M <= 32) return run_rows<kG, 2, 8>(a, stream);
    if (M <= 48) return run_rows<kG, 3, 12>(a, stream);
    return run_many<kG>(a, stream);
  });
}

}  // namespace qlora
