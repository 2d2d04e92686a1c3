// The adapter's products beside an 8-bit input, on bf16 matrix instructions.
//
// Row products   V[m][j] = sum_c S[m][c] W[j][c]      T = dec(X8) A, G = dY B^T
// Column products P[c][j] = sum_m S[m][c] V[m][j]     dA = dec(X8)^T (s G), dB^T = dY^T (s T)
//
// S streams past once: codes are decoded in registers (a code times its
// power-of-two scale is an exact bf16 value). The matrix work is r columns
// wide, so both are bound by reading S and by the small factor, which every
// workgroup reads again through the caches. Kernel times at r = 64:
//   dY B^T, 2048 x 11008 (bf16, 45 MB)       16 to 19 us, 2.4 to 2.8 TB/s of S
//   dec(X8) A, 4096 x 8192 (33.5 MB)         18 us, 1.9 TB/s (A is r K values,
//                                            decoded X passes the vector units)
//   dA and dB at K = 11008, N = 4096, 2048 rows (39 MB)   19 to 23 us
// At 257 rows or fewer they take 3 to 5 us, mostly the launch and one round
// trip to memory.
//
// v_mfma_f32_16x16x32_bf16 takes eight contraction elements per lane. A row
// product finds them next to each other in memory (S and B rows), except for
// A [K x r]; a column product contracts down the rows of S. Those operands
// pass through a wave's own LDS tile, row-major, and come back transposed by
// ds_read_b64_tr_b16 (16 lanes read a 4 x 16 piece by rows and receive it by
// columns), with no barrier.
//
// dA and dB are float32: V stays float32 in memory and enters the column
// product as three bf16 terms whose sum is the value to 24 bits, so the
// products of bf16 values carry float32 accuracy. The terms are formed in
// registers: V passes once per 64 columns of S and is most of the cache
// traffic, 4 bytes an element so instead of 6 (terms formed beforehand took the
// same time and half as much memory again). The results of the waves of a
// workgroup, which take turns along the contraction, are added in a fixed order.
#include "lowrank8.h"

#include <algorithm>

namespace qlora {

namespace lr8 {

// ---------------------------------------------------------------------------
// Row products: 64 rows by 16 NJ columns per workgroup (so that S is read once
// for r up to 64), split along the contraction into about one workgroup per
// compute unit (512 halves: 22 us instead of 16 for dY B^T); the waves take the
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
  constexpr int kRed = tile_bytes(NJ);
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

  // One step's loads, all on their way before the first is waited for: S
  // (codes, scales and keep bits, or values) and W. The other waves cover the
  // wait; the next step's loads a step early took more registers and time.
  struct Regs {
    u32x4 s[4][kSrc == kBf16 ? 2 : 1];
    uint32_t sc[4], keep[4];
    u32x4 w[2 * NJ];
  };
  auto load = [&](int st) {
    Regs q;
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      const int row = f * 16 + i;
      if constexpr (kSrc == kBf16) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          q.s[f][h] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
              rs, (int)(row * p.s.ld) + g * 32 + h * 16, st * 128, 0));
      } else {
        q.s[f][0] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
            rs, (int)(row * p.s.ld) + g * 16, st * 64, 0));
        q.sc[f] = __builtin_amdgcn_raw_buffer_load_b8(rsc, (int)(row * p.s.sld), st >> 1, 0);
        if constexpr (kMask)
          q.keep[f] = __builtin_amdgcn_raw_buffer_load_b32(rm, (int)(row * mld * 4) + (g >> 1) * 4, st * 8, 0);
      }
    }
    if constexpr (kTrans) {
      // rows st * 64 .. + 63 of A, columns j0 .. j0 + 16 NJ - 1
      if (p.wvec) {
#pragma unroll
        for (int e = 0; e < 2 * NJ; ++e) {
          const int id = e * 64 + lane, row = id / (2 * NJ), ch = id % (2 * NJ);
          const bool ok = j0 + ch * 8 < p.r;  // r is a multiple of 8 here
          q.w[e] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
              rw, ok ? (row * p.r + j0 + ch * 8) * 2 : kPastEnd, st * 64 * p.r * 2, 0));
        }
      }
    } else {
#pragma unroll
      for (int jt = 0; jt < NJ; ++jt) {
        const int j = j0 + jt * 16 + i;
        const int off = j < p.r ? (int)(j * p.s.cols * 2) + g * 32 : kPastEnd;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          q.w[jt * 2 + h] = __builtin_bit_cast(
              u32x4, __builtin_amdgcn_raw_buffer_load_b128(rw, off + h * 16, st * 128, 0));
      }
    }
    return q;
  };
  const int end = min(p.steps, (split + 1) * p.per);
  const int begin = split * p.per + wave;
  for (int st = begin; st < end; st += kWaves) {
    const Regs q = load(st);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (kTrans) {  // A's rows to LDS, back by columns
      if (p.wvec) {
#pragma unroll
        for (int e = 0; e < 2 * NJ; ++e) {
          const int id = e * 64 + lane, row = id / (2 * NJ), ch = id % (2 * NJ);
          *(lds_u32x4*)(uintptr_t)(wt + (uint32_t)(row * kPitch + ch * 16)) = q.w[e];
        }
      } else {
        for (int e = lane; e < 64 * 16 * NJ; e += 64) {
          const int row = e / (16 * NJ), j = e % (16 * NJ);
          uint16_t v = 0;
          if (j0 + j < p.r) v = p.w[((int64_t)st * 64 + row) * p.r + j0 + j];
          *(gemm::lds_u16*)(uintptr_t)(wt + (uint32_t)(row * kPitch + j * 2)) = v;
        }
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      bf16x8 w[NJ];
#pragma unroll
      for (int jt = 0; jt < NJ; ++jt) {
        if constexpr (kTrans) w[jt] = tr_frag<kPitch>(wt, 16 * g + 8 * h, jt * 16, lane);
        else w[jt] = as_bf16x8(q.w[jt * 2 + h]);
      }
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        u32x4 x;
        if constexpr (kSrc == kBf16) {
          x = q.s[f][h];
        } else {
          x = act8_decode8<kSrc>(u32x2{q.s[f][0][2 * h], q.s[f][0][2 * h + 1]}, act8_scale((int)q.sc[f]));
          if constexpr (kMask) x &= keep_mask8(q.keep[f] >> ((g & 1) * 16 + 8 * h));
        }
#pragma unroll
        for (int jt = 0; jt < NJ; ++jt)
          acc[f * NJ + jt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(x), w[jt],
                                                                     acc[f * NJ + jt], 0, 0, 0);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  reduce_waves<NJ>(acc, lds, wave, lane);
#pragma unroll
  for (int q = 0; q < 2 * NJ; ++q) {
    const int o = q * kThreads + threadIdx.x, j = o % (16 * NJ), ml = o / (16 * NJ);
    const float v = tile_sum<NJ>(lds, ml, j);
    if (m0 + ml < p.s.rows) p.part[((int64_t)split * p.s.rows + m0 + ml) * p.ldp + j0 + j] = v;
  }
#endif
}

// ---------------------------------------------------------------------------
// What follows a row product: V = f * (sum of the partials, in split order),
// written as any of
//   out32  float32 V [M x r]
//   u      bf16(s V), [M rounded up to 64 x r64], 0 past M and r
//   vf     s V in float32 in the order a column product reads it
//          (frag_index), 0 past M and r
// 16 x 64 tiles, through LDS for the last form. 4.5 to 5.5 us up to 4096 rows:
// a launch and one round trip, whence the other work in the same launch (8-bit
// blocks of dY at 2048 x 4096 beside it: 7.0 us, 5.8 in a launch of its own).
struct OutJob {
  const float* part;  // null: no job, or the product below
  const uint16_t *sm, *w;  // the partials' place: V = S W^T formed here, S [M x C], W [r x C]
  int64_t C;
  int splits;
  int64_t ldp;
  float f;
  float* out32;
  uint16_t* u;
  float* vf;
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
constexpr int kOutRows = 16;  // rows of M per workgroup

// A tile of V = S W^T in place of summed partials, a wave per 16 columns, over
// the whole of C: for the C at which a launch costs more than the few trips to
// memory that one wave then makes.
__device__ __forceinline__ void out_product(const OutJob& jb, int64_t mt, int jc, int64_t M, int r,
                                            float (*tile)[65]) {
#ifdef __HIP_DEVICE_COMPILE__
  const int t = threadIdx.x, lane = t & 63, i = lane & 15, g = lane >> 4, ja = jc * 64 + (t >> 6) * 16 + i;
  const int64_t first = mt * kOutRows;
  const __amdgpu_buffer_rsrc_t rs = make_rsrc(jb.sm + first * jb.C, min(M - first, (int64_t)kOutRows) * jb.C * 2);
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(jb.w, r * jb.C * 2);
  const int so = (int)(i * jb.C * 2) + g * 16, wo = ja < r ? (int)(ja * jb.C * 2) + g * 16 : kPastEnd;
  floatx4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
  constexpr int kU = 8;  // pieces of 32 elements in flight
  for (int c = 0; c < (int)jb.C * 2; c += kU * 64) {
    u32x4 x[kU], w[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int off = c + u * 64 < (int)jb.C * 2 ? c + u * 64 : kPastEnd;  // past the row: zeros
      x[u] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, so, off, 0));
      w[u] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rw, wo, off, 0));
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < kU; ++u)
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(x[u]), as_bf16x8(w[u]), acc, 0, 0, 0);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) tile[4 * g + e][(t >> 6) * 16 + i] = acc[e];
#endif
}

__device__ __forceinline__ void out_tile(const OutJob& jb, int64_t mt, int jc, int64_t M, int r,
                                         int64_t r64, int64_t rp, float s, float (*tile)[65]) {
  const int t = threadIdx.x;
  float v[4];
  const int jl = t & 63, j = jc * 64 + jl;
  const int64_t m0 = mt * kOutRows + (t >> 6);
  if (jb.sm) {
    out_product(jb, mt, jc, M, r, tile);
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = tile[(t >> 6) + 4 * q][jl];
    __syncthreads();
  } else {
    // loads inside the product's rows and columns, so that none is conditional;
    // more splits at a time would take registers from the work beside
    const float* at[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[q] = 0.0f;
      at[q] = jb.part + min(m0 + 4 * q, M - 1) * jb.ldp + min(j, r - 1);
    }
    const int64_t stride = M * jb.ldp;
#pragma unroll 2
    for (int sp = 0; sp < jb.splits; ++sp)
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] += at[q][sp * stride];
  }
  // 0 past M and r: what stands there is a copy, or an infinity's product with 0
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (m0 + 4 * q >= M || j >= r) v[q] = 0.0f;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int64_t m = m0 + 4 * q;
    v[q] *= jb.f;
    if (jb.out32 && m < M && j < r) jb.out32[m * r + j] = v[q];
    v[q] *= s;
    if (jb.u) jb.u[m * r64 + j] = (uint16_t)(pack_bf16x2(v[q], 0.0f) & 0xffffu);
    tile[(t >> 6) + 4 * q][jl] = v[q];
  }
  if (!jb.vf) return;
  __syncthreads();
  // four consecutive m of one j per thread
  const int ja = t >> 2, ml = (t & 3) * 4;
  if (jc * 64 + ja >= rp) return;
  floatx4 o;
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] = tile[ml + e][ja];
  *reinterpret_cast<floatx4*>(jb.vf + frag_index(mt * kOutRows + ml, jc * 64 + ja, rp)) = o;
}

__device__ __forceinline__ void pad_tile(const PadJob& jb, int64_t rt, int jc, int r, int64_t r64,
                                         float (*tile)[65]) {
  const int t = threadIdx.x;
  uint32_t v[16];
  if (!jb.columns) {
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      const int64_t row = rt * 64 + (t >> 6) + 4 * q;
      const int j = jc * 64 + (t & 63);
      v[q] = row < jb.rows && j < r ? jb.src[row * r + j] : 0u;
    }
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      const int64_t row = rt * 64 + (t >> 6) + 4 * q;
      if (row < jb.rows) jb.dst[row * r64 + jc * 64 + (t & 63)] = (uint16_t)v[q];
    }
    return;
  }
#pragma unroll
  for (int q = 0; q < 16; ++q) {  // read along the rows of B
    const int64_t row = rt * 64 + (t & 63);
    const int j = jc * 64 + (t >> 6) + 4 * q;
    v[q] = row < jb.rows && j < r ? jb.src[(int64_t)j * jb.rows + row] : 0u;
  }
#pragma unroll
  for (int q = 0; q < 16; ++q) tile[t & 63][(t >> 6) + 4 * q] = __builtin_bit_cast(float, v[q]);
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    const int rl = (t >> 6) + 4 * q;
    const int64_t row = rt * 64 + rl;
    if (row < jb.rows)
      jb.dst[row * r64 + jc * 64 + (t & 63)] = (uint16_t)__builtin_bit_cast(uint32_t, tile[rl][t & 63]);
  }
}

// ---------------------------------------------------------------------------
// bf16(w') of a 4-bit store, transposed: one tile of 64 weight rows by 128
// columns per workgroup. A thread decodes 16 codes of two neighbouring rows
// (inside one block of 64 each) and writes them to LDS as pairs; the tile is
// stored by its columns, 128 bytes each. Bound by its writes: 11008 x 4096, 90 MB
// written and 24 MB read, takes 25 us with the jobs beside it (4.6 TB/s).
constexpr int kTPitch = 136;  // bytes of an LDS row: 64 bf16 and 8 bytes of padding
constexpr int kDecodeLds = 64 + 128 * kTPitch;

__device__ __forceinline__ void nf4_decode_t(const Nf4Weight& W, int64_t N, int64_t K, const Codebook& cb,
                                             uint16_t* __restrict__ out, unsigned tile, uint8_t* lds) {
#pragma clang fp contract(off)
  float* s_lv = reinterpret_cast<float*>(lds);
  uint8_t* s_t = lds + 64;
  const int t = threadIdx.x;
  if (t < 16) s_lv[t] = cb.lv[t];
  const int64_t kt = (K + 127) / 128;
  const int64_t n0 = tile / kt * 64, k0 = tile % kt * 128;
  const int np = t >> 3, q = t & 7;
  const int64_t k = k0 + q * 16;
  const bool ok = k < K;  // K is a multiple of 64: a piece of 16 is inside or outside
  u32x2 c[2];
  float cs[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t e = (n0 + 2 * np + h) * K + (ok ? k : 0);
    c[h] = *reinterpret_cast<const u32x2*>(W.codes + e / 2);
    const int64_t b = e / kBlock;
    cs[h] = !W.absmax_q ? W.absmax_s2[b]
            : cb.dq_fp8 ? block_scale_fp8(W.absmax_q[b], W.absmax_s2[b / kGroup])
                        : block_scale(W.absmax_q[b], W.absmax_s2[b / kGroup]);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float lo = s_lv[(c[0][i >> 3] >> (4 * (i & 7))) & 15u] * cs[0];
    const float hi = s_lv[(c[1][i >> 3] >> (4 * (i & 7))) & 15u] * cs[1];
    *reinterpret_cast<uint32_t*>(s_t + (q * 16 + i) * kTPitch + np * 4) = pack_bf16x2(lo, hi);
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int id = e * kOutThreads + t, row = id >> 3, ch = id & 7;
    const u32x2 a = *reinterpret_cast<const u32x2*>(s_t + row * kTPitch + ch * 16);
    const u32x2 b = *reinterpret_cast<const u32x2*>(s_t + row * kTPitch + ch * 16 + 8);
    if (k0 + row < K)
      *reinterpret_cast<u32x4*>(out + (k0 + row) * N + n0 + ch * 8) = u32x4{a[0], a[1], b[0], b[1]};
  }
}

// ---------------------------------------------------------------------------
struct OutArgs {
  OutJob o[2];
  PadJob pad;
  int64_t M;
  int r;
  int64_t r64, rp;
  float s;
  int cols;                      // column tiles of the jobs
  int blocks0, blocks1, blocks;  // workgroups of the first out job, of both, of all jobs
  uint32_t* done;                // kTileSums words to clear, or null
};
// What the same launch does beside the jobs: an 8-bit copy of S, or a weight
// to bf16 (decode_t). Both are what the launch after this one reads.
struct BesideArgs {
  const uint16_t* s;
  int64_t C;
  uint32_t blocks;
  int KB, sb;
  uint8_t *codes, *scales;
  Nf4Weight W;
  int64_t N, K;
  Codebook cb;
  uint16_t* w;
};
enum Beside { kNothing = 0, kQuantizeE4M3 = 1, kQuantizeE5M2 = 2, kDecode = 3 };

template <int kBeside>
__global__ void __launch_bounds__(kOutThreads) lowrank_out_kernel(OutArgs p, BesideArgs q) {
  constexpr int kTile = 64 * 65 * 4;
  __shared__ __attribute__((aligned(16))) uint8_t smem[kBeside == kDecode && kDecodeLds > kTile ? kDecodeLds : kTile];
  auto tile = reinterpret_cast<float(*)[65]>(smem);
  const int id = blockIdx.x;
  static_assert(kTileSums == kOutThreads, "a word per thread");
  if (id == 0 && p.done) p.done[threadIdx.x] = 0;
  if (id < p.blocks) {
    const int b = id / p.cols, jc = id % p.cols;
    if (b < p.blocks0) out_tile(p.o[0], b, jc, p.M, p.r, p.r64, p.rp, p.s, tile);
    else if (b < p.blocks1) out_tile(p.o[1], b - p.blocks0, jc, p.M, p.r, p.r64, p.rp, p.s, tile);
    else pad_tile(p.pad, b - p.blocks1, jc, p.r, p.r64, tile);
    return;
  }
  if constexpr (kBeside == kDecode) {
    nf4_decode_t(q.W, q.N, q.K, q.cb, q.w, id - p.blocks, smem);
  } else if constexpr (kBeside != kNothing) {
    const uint32_t b = (uint32_t)(id - p.blocks) * (kOutThreads / 16) + (threadIdx.x >> 4);
    if (b < q.blocks)
      act8_quantize_block<kBeside == kQuantizeE5M2, true>(q.s, q.C, q.C, b, q.KB, q.sb, q.codes, q.scales);
  }
}

template <int kSrc, int NJ>
__global__ void __launch_bounds__(kThreads) column_products_kernel(ColPair p) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[column_lds(NJ)];
  column_job<kSrc, NJ>(p, blockIdx.x, (uint32_t)(uintptr_t)((__attribute__((address_space(3))) uint8_t*)smem));
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

template <int kSrc, bool kMask, bool kTrans>
hipError_t run_rows(RowProd p, int splits, hipStream_t stream) {
  return by_nj(p.r, [&](auto nj) {
    auto kern = row_product_kernel<kSrc, kMask, kTrans, decltype(nj)::value>;
    hipLaunchKernelGGL(kern, dim3((unsigned)(p.tiles * splits), (unsigned)ceil_div(p.r, 64)),
                       dim3(kThreads), 0, stream, p);
    return hipGetLastError();
  });
}

// `per`: steps of a split, or 0 for row_splits' choice.
RowProd row_args(Stream s, const uint16_t* w, int r, int per, float* part, int* splits) {
  RowProd p{};
  p.s = s;
  p.w = w;
  p.r = r;
  p.wvec = r % 8 == 0 && (reinterpret_cast<uintptr_t>(w) & 15) == 0;
  p.steps = (int)ceil_div(s.cols, 64);
  *splits = per ? (int)ceil_div(p.steps, per) : row_splits(s.rows, s.cols, r);
  p.per = per ? per : (int)ceil_div(p.steps, *splits);
  p.ldp = lowrank_cols(r);
  p.part = part;
  p.tiles = (int)ceil_div(s.rows, 64);
  return p;
}

Stream act8_stream(ConstAct8 x, int fmt, int64_t M, int64_t K, const uint32_t* mask) {
  return Stream{x.codes, x.scales, act8_row_bytes(K), act8_scale_row_bytes(K), M, K, mask, fmt};
}

}  // namespace

int lowrank_cols(int r) { return r <= 16 ? 16 : r <= 32 ? 32 : (int)ceil_div(r, 64) * 64; }

hipError_t launch_rows_act8(ConstAct8 x, int fmt, int64_t M, int64_t K, const uint32_t* mask,
                            const uint16_t* A, int r, float* part, int* splits, hipStream_t stream) {
  // where the 8-bit product for few tokens may form T itself, its order
  const int per = few_t_shape(M, K, r) ? 2 * (int)ceil_div(act8_row_bytes(K) / kAct8Block, kFewWaves) : 0;
  const RowProd p = row_args(act8_stream(x, fmt, M, K, mask), A, r, per, part, splits);
  if (mask) return fmt ? run_rows<kE5M2, true, true>(p, *splits, stream) : run_rows<kE4M3, true, true>(p, *splits, stream);
  return fmt ? run_rows<kE5M2, false, true>(p, *splits, stream) : run_rows<kE4M3, false, true>(p, *splits, stream);
}

hipError_t launch_rows_bf16(const uint16_t* S, int64_t M, int64_t C, const uint16_t* B, int r,
                            float* part, int* splits, hipStream_t stream) {
  const RowProd p = row_args(Stream{S, nullptr, C * 2, 0, M, C, nullptr, 0}, B, r, 0, part, splits);
  return run_rows<kBf16, false, false>(p, *splits, stream);
}

hipError_t launch_lowrank_out(const LowrankOut* o, int n, LowrankPad pad, int64_t M, int r, float s,
                              uint32_t* done, hipStream_t stream, const LowrankBeside& beside) {
  OutArgs p{};
  p.done = done;
  p.M = M;
  p.r = r;
  p.r64 = ceil_div(r, 64) * 64;
  p.rp = lowrank_cols(r);
  p.s = s;
  for (int i = 0; i < n; ++i)
    p.o[i] = OutJob{o[i].part, o[i].s, o[i].w, o[i].C, o[i].splits, o[i].ldp, o[i].f, o[i].out32, o[i].u, o[i].vf};
  p.pad = PadJob{pad.src, pad.columns, pad.rows, pad.dst};
  p.cols = (int)(p.r64 / 64);
  p.blocks0 = (int)(ceil_div(M, 64) * 64 / kOutRows);
  p.blocks1 = n * p.blocks0;
  p.blocks = p.cols * (p.blocks1 + (pad.src ? (int)ceil_div(pad.rows, 64) : 0));
  BesideArgs q{};
  int64_t more = 0;
  if (beside.codes) {
    q.s = beside.s;
    q.C = beside.C;
    q.KB = (int)ceil_div(beside.C, kAct8Block);
    q.sb = (int)act8_scale_row_bytes(beside.C);
    q.blocks = (uint32_t)(M * q.KB);
    q.codes = beside.codes;
    q.scales = beside.scales;
    more = ceil_div(q.blocks, kOutThreads / 16);
  } else if (beside.w) {
    q.W = beside.W;
    q.N = beside.N;
    q.K = beside.K;
    q.cb = codebook_of(beside.W);
    q.w = beside.w;
    more = beside.N / 64 * ceil_div(beside.K, 128);
  }
  auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, dim3((unsigned)(p.blocks + more)), dim3(kOutThreads), 0, stream, p, q);
    return hipGetLastError();
  };
  if (beside.codes) return beside.fmt ? go(lowrank_out_kernel<kQuantizeE5M2>) : go(lowrank_out_kernel<kQuantizeE4M3>);
  return beside.w ? go(lowrank_out_kernel<kDecode>) : go(lowrank_out_kernel<kNothing>);
}

lr8::ColPair lr8::column_pair(ConstAct8 x, int fmt, const uint32_t* mask, const uint16_t* dY, const float* g,
                              const float* t, int64_t M, int64_t N, int64_t K, int r, float* dA, float* dB) {
  ColPair p{};
  p.a = ColProd{act8_stream(x, fmt, M, K, mask), g, dA, (int64_t)r, 1};
  p.b = ColProd{Stream{dY, nullptr, N * 2, 0, M, N, nullptr, 0}, t, dB, 1, N};
  p.ta = (int)(K / 64);
  p.tiles = (int)(K / 64 + N / 64);
  p.jobs = p.tiles * (int)ceil_div(r, 64);
  p.r = r;
  p.rp = lowrank_cols(r);
  return p;
}

hipError_t launch_columns(const ColPair& p, hipStream_t stream) {
  return by_nj(p.r, [&](auto nj) {
    constexpr int NJ = decltype(nj)::value;
    hipLaunchKernelGGL((p.a.s.fmt ? column_products_kernel<kE5M2, NJ> : column_products_kernel<kE4M3, NJ>),
                       dim3((unsigned)p.jobs), dim3(kThreads), 0, stream, p);
    return hipGetLastError();
  });
}

}  // namespace qlora
