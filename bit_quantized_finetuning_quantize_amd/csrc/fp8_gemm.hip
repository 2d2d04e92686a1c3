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
// The instruction sums its products in groups of eight, each to 13 bits below
// the group's largest product, and the groups in float32.
//
// The same tiles serve bf16 operands (launch_bf16_gemm).
//
// Large products are bound by the matrix units at the clock that their power
// allows: 8192^3 takes 375 to 387 us on random data (2.8 to 2.9 PFLOP/s, about
// 1.77 GHz) and 305 to 325 us on zeros; the units are busy 79 % of the clocks and
// the waves wait for operands and barriers 20 %. Where 256 x 128 tiles are left
// (2048 x 4096 x 11008, 76 to 90 us between cards) it is 62 % and 28 %: half the
// products per step to cover the loads' latency, and LDS for no more stages.
// With all operands in the L2 these two take 3 and 6 % less. 4096 x 22016 x 8192
// takes 520 to 560 us. Not kept: the tiles of a last round cut along K and their
// sums exchanged through memory (256 x 256 tiles instead of 256 x 128; the
// exchange took 17 us, more than the larger tiles gained), the waves of a tile
// splitting K (2048 x 4096 x 11008 75.2 us to 74.0).
#include "lowrank8.h"

#include <algorithm>
#include <atomic>

namespace qlora {

namespace fp8 {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) float lds_f32;
typedef __attribute__((address_space(3))) uint32_t lds_u32;

struct Fp8Gemm {
  const uint8_t *x, *xs, *w, *ws;
  int64_t M, N, ldc;   // ldc: bytes of a row of codes (both operands)
  int KB, sb;          // blocks along K, bytes of a row of scales
  const uint16_t *U, *V;  // bf16 [M x r64], [N x r64], or null
  int r64;
  uint16_t* Y;         // [M x N]
  const uint32_t* keep;   // bf16 only: mask [M][N / 32] over the U V term, or null
  bool stream;         // Y is stored past the caches
  int nM, nN, group;   // tiles, and row tiles per group of the walk
  int full, cut;       // 256 x 256 tiles done whole; parts of each other one
  // Small tiles: workgroups that share a tile, a run of K each; their counts
  // of workgroups done (0 before) and sums, 4096 floats a workgroup.
  int splits;
  uint32_t* done;
  float* sums;
};

// 128-byte LDS rows, the 16-byte piece c of row r at position c ^ swz(r).
using gemm::lds_u32x2;
using gemm::lds_u32x4;
using gemm::lds_void;
using gemm::make_rsrc;
using gemm::tile_off;
using gemm::wait_vmcnt;

// Format of the operands: weights E4M3 and activations E4M3 or E5M2, or both
// bf16 (then a step of 128 bytes is 64 elements, without scales).
enum Fmt { kE4M3 = 0, kE5M2 = 1, kBf16 = 2 };

// Product of two 32-row fragments of 64 bytes per row.
template <int kFmt>
__device__ __forceinline__ floatx16 mma(const u32x4 (&w)[2], const u32x4 (&x)[2], floatx16 c,
                                        uint32_t sw, uint32_t sx) {
  if constexpr (kFmt == kBf16) {
    c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(w[0]), as_bf16x8(x[0]), c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(w[1]), as_bf16x8(x[1]), c, 0, 0, 0);
  } else {
    auto whole = [](const u32x4 (&f)[2]) {
      return i32x8{(int)f[0][0], (int)f[0][1], (int)f[0][2], (int)f[0][3],
                   (int)f[1][0], (int)f[1][1], (int)f[1][2], (int)f[1][3]};
    };
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(whole(w), whole(x), c, 0, kFmt, 0, (int)sw, 0, (int)sx);
  }
}

// Tiles are walked in groups of `group` row tiles, column tile outermost in
// the group, so that neighbours in the walk share operands.
__device__ __forceinline__ void tile_at(const Fp8Gemm& p, int t, int& tm, int& tn) {
  const int per = p.group * p.nN;
  const int g = t / per, in = t - g * per;
  const int rows = min(p.group, p.nM - g * p.group);
  tm = g * p.group + in % rows;
  tn = in / rows;
}
// Workgroup id runs on XCD id % 8: each XCD takes a consecutive run of the
// walk (runs differ by one tile at most), whose operands then meet in its L2.
__device__ __forceinline__ int xcd_order(int id, int count) {
  const int x = id & 7;
  return x * (count >> 3) + min(x, count & 7) + (id >> 3);
}

// Issue order: kN times one product (kP matrix instructions) and, beside it, kV
// loads and kD LDS reads.
template <int kN, int kP, int kV, int kD>
__device__ __forceinline__ void pace() {
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, kP, 0);
    __builtin_amdgcn_sched_group_barrier(0x020, kV, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, kD, 0);
  }
}
// LDS of a tile: its ring, or the output staged in its place.
constexpr int lds_bytes(int TN, int TM, int stages, int groups) {
  const int ring = groups * stages * (TN + TM) * 128, out = TM * 2 * (TN + 16);
  return ring > out ? ring : out;
}

// The sum of a tile's splits. Every workgroup stores its sums and counts itself;
// the last one to do so adds them all, in the order of the splits, whichever it
// is, and is the one to go on (true). No workgroup waits for another. They may
// sit on different XCDs, whose L2s are separate: the sc1 bit makes a store
// write through to memory and a load pass over the L2.
__device__ __forceinline__ bool join_splits(floatx16& acc, const Fp8Gemm& p, int tile, int split, uint32_t lds) {
#ifdef __HIP_DEVICE_COMPILE__
  constexpr int kSc1 = 16, kBytes = 64 * 64 * 4;
  const __amdgpu_buffer_rsrc_t at = make_rsrc(p.sums + (int64_t)tile * p.splits * 4096, p.splits * kBytes);
  const int v = (int)threadIdx.x * 16;  // 256 threads
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const floatx4 o{acc[4 * e], acc[4 * e + 1], acc[4 * e + 2], acc[4 * e + 3]};
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, o), at, v, split * kBytes + e * 4096, kSc1);
  }
  // every store of the workgroup acknowledged before it counts itself
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  lds_u32* word = (lds_u32*)(uintptr_t)lds;
  if (threadIdx.x == 0)
    *word = __hip_atomic_fetch_add(p.done + tile, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  const bool last = __builtin_amdgcn_readfirstlane((int)*word) == p.splits - 1;
  __syncthreads();
  if (!last) return false;
  asm volatile("" ::: "memory");
  floatx16 sum;
#pragma unroll
  for (int i = 0; i < 16; ++i) sum[i] = 0.0f;
  constexpr int kU = 4;  // splits in flight; past the last they read zeros
  for (int s0 = 0; s0 < p.splits; s0 += kU) {
    floatx4 o[kU][4];
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        o[u][e] = __builtin_bit_cast(
            floatx4, __builtin_amdgcn_raw_buffer_load_b128(at, v, (s0 + u) * kBytes + e * 4096, kSc1));
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int i = 0; i < 16; ++i) sum[i] += o[u][i >> 2][i & 3];
  }
  acc = sum;
#endif
  return true;
}

// Tile of TN weight rows by TM activation rows, 2 x 2 waves, each a
// (TN / 2) x (TM / 2) part of it in 32 x 32 accumulators.
//
// A step is one block of 128 along K, in two halves of 64. The fragments of
// the next half are read from LDS while the matrix cores work on the present
// one, so two sets of fragments take turns. The operand tiles sit in a ring of
// LDS stages. In the middle of a step every wave has read all of the step's
// stage (its second half's fragments are in registers) and the loads of the
// next step have landed: one barrier there frees the stage for the step
// kStages ahead and lets the fragments of the next step be read under the second
// half's products. No load or LDS latency is then waited for inside the loop.
//
// With kGroups > 1 the workgroup has that many sets of 2 x 2 waves, each with
// a ring of its own, that take a run of the steps each; the sums of the other
// sets are added to the first's in order at the end. For grids that leave
// compute units idle: a step's latency then covers kGroups blocks along K.
//
// With kJoin, `split` is this workgroup's run of K in the tile `tile` that
// p.splits of them share: see join_splits.
template <int TN, int TM, int kStages, int kGroups, int kFmt, bool kJoin = false>
__device__ __forceinline__ void gemm_tile(const Fp8Gemm& p, int64_t n0, int64_t m0, uint32_t lds_all,
                                          int tile = 0, int split = 0) {
#ifdef __HIP_DEVICE_COMPILE__  // the host pass needs the kernels' stubs alone
  constexpr int WN = TN / 2, WM = TM / 2;
  constexpr int BN = WN / 32, BM = WM / 32;
  constexpr int kStage = (TN + TM) * 128;
  constexpr int kLoadW = TN / 32, kLoadX = TM / 32;  // per wave and step
  const int lane = threadIdx.x & 63;
  const int wave_all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wave = wave_all & 3, group = wave_all >> 2;
  const uint32_t lds0 = lds_all + (uint32_t)(group * kStages * kStage);
  const int wn = wave & 1, wm = wave >> 1;
  const int r = lane & 31, half = lane >> 5;

  // this set's steps: [first, first + KB); every set walks KB steps, and those
  // past the end of K read zeros
  const int run = kJoin ? (p.KB + p.splits - 1) / p.splits : p.KB, start = split * run;
  const int KB = (run + kGroups - 1) / kGroups;
  const int first = start + group * KB, valid = min(p.KB, start + run) - first;
  // The low-rank term comes first, through the same ring: a step of it is 64
  // columns of V and U, 128 bytes of a row as in the steps along K.
  const int LR = p.U && split == 0 ? p.r64 / 64 : 0;

  // operand moves: 8 rows of 128 bytes per instruction. The swizzle of rows 16
  // apart is the same: one lane offset serves every second instruction.
  const int row0 = wave * (kLoadW * 8) + (lane >> 3), row1 = wave * (kLoadX * 8) + (lane >> 3);
  struct Source {
    __amdgpu_buffer_rsrc_t w, x;
    int vw[2], vx[2], step16;
  };
  auto source = [&](const uint8_t* w, const uint8_t* x, int64_t ld) {
    Source s;
    // the tile's rows alone (2 GiB at most), so that a step past the end of
    // K is out of range however large the matrices are
    s.w = make_rsrc(w + n0 * ld, min(p.N - n0, (int64_t)TN) * ld);
    s.x = make_rsrc(x + m0 * ld, min(p.M - m0, (int64_t)TM) * ld);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      s.vw[i] = (int)((row0 + i * 8) * ld) + (((lane & 7) ^ gemm::swz(row0 + i * 8)) << 4);
      s.vx[i] = (int)((row1 + i * 8) * ld) + (((lane & 7) ^ gemm::swz(row1 + i * 8)) << 4);
    }
    s.step16 = (int)(16 * ld);
    return s;
  };
  const Source operands = source(p.w, p.x, p.ldc);
  // byte offset of a step in its rows; past the end out of range
  auto at_step = [&](int kb) { return kb < min(KB, valid) ? (first + kb) * 128 : kPastEnd; };
  // move i of a step: weight rows first, then activation rows
  auto move = [&](const Source& s, int off, uint32_t st, int i) {
    if (i < kLoadW)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          s.w, (lds_void*)(uintptr_t)(st + (uint32_t)((wave * kLoadW + i) * 1024)), 16, s.vw[i & 1],
          off + (i >> 1) * s.step16, 0, 0);
    else
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          s.x, (lds_void*)(uintptr_t)(st + (uint32_t)(TN * 128 + (wave * kLoadX + i - kLoadW) * 1024)),
          16, s.vx[(i - kLoadW) & 1], off + ((i - kLoadW) >> 1) * s.step16, 0, 0);
  };

  constexpr bool kRuns = kGroups > 1 || kJoin;  // steps may begin anywhere
  // scale bytes, a dword for four steps; the low byte is the present step's. A
  // set that begins inside a dword takes four steps' bytes from two of them.
  const __amdgpu_buffer_rsrc_t rsw = make_rsrc(p.ws, (p.N + 127) / 128 * p.sb);
  const __amdgpu_buffer_rsrc_t rsx = make_rsrc(p.xs + m0 * p.sb, (p.M - m0) * p.sb);
  struct Scales { uint32_t w, x[BM]; };
  auto scales = [&](int kb) {
    Scales s{};
    if constexpr (kFmt == kBf16) return s;
    const int at = (kRuns ? first & ~3 : 0) + kb;
    s.w = __builtin_amdgcn_raw_buffer_load_b32(rsw, (int)((n0 + wn * WN) / 128) * p.sb, at, 0);
#pragma unroll
    for (int j = 0; j < BM; ++j)
      s.x[j] = __builtin_amdgcn_raw_buffer_load_b32(rsx, (wm * WM + j * 32 + r) * p.sb, at, 0);
    return s;
  };
  auto four = [&](const Scales& lo, const Scales& hi) {
    Scales s = lo;
    if constexpr (kRuns) {
      const uint32_t by = (uint32_t)(first & 3) * 8;
      s.w = __builtin_amdgcn_alignbit(hi.w, lo.w, by);
#pragma unroll
      for (int j = 0; j < BM; ++j) s.x[j] = __builtin_amdgcn_alignbit(hi.x[j], lo.x[j], by);
    }
    return s;
  };

  // Every load of the loops and of this prologue is issued whatever KB is: past
  // the end it reads nothing, and its stage is not used.
  const Source lowrank = source(reinterpret_cast<const uint8_t*>(p.V), reinterpret_cast<const uint8_t*>(p.U),
                                (int64_t)p.r64 * 2);
  auto at_lowrank = [&](int q) { return group == 0 ? q * 128 : kPastEnd; };
  auto issue = [&](int q, uint32_t st) {  // step q of the low-rank steps and those along K
    if (q < LR) {
#pragma unroll
      for (int i = 0; i < kLoadW + kLoadX; ++i) move(lowrank, at_lowrank(q), st, i);
    } else {
#pragma unroll
      for (int i = 0; i < kLoadW + kLoadX; ++i) move(operands, at_step(q - LR), st, i);
    }
  };
#pragma unroll
  for (int k = 0; k < kStages; ++k) issue(k, lds0 + (uint32_t)(k * kStage));
  Scales s, dw0 = scales(0), dw1{};
  if constexpr (kRuns) dw1 = scales(4);

  floatx16 acc[BN][BM];
#pragma unroll
  for (int i = 0; i < BN; ++i)
#pragma unroll
    for (int j = 0; j < BM; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;

  // LDS offsets of a fragment's two 16-byte pieces, 4 h + 2 half and the
  // next, in row r of the wave's part; rows 32 apart share the swizzle
  uint32_t ow[2][2], ox[2][2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      ow[h][c] = lds0 + (uint32_t)tile_off(wn * WN + r, 4 * h + 2 * half + c);
      ox[h][c] = lds0 + (uint32_t)(TN * 128 + tile_off(wm * WM + r, 4 * h + 2 * half + c));
    }
  // Fragments in the order the products use them: weight block 0, the
  // activation blocks, the other weight blocks. Two pieces each.
  struct Frags { u32x4 f[BN + BM][2]; };
  auto read1 = [&](Frags& f, uint32_t st, int h, int i, int c) {
    const bool act = i >= 1 && i <= BM;
    const int block = act ? i - 1 : i ? i - BM : 0;
    f.f[i][c] = *(const lds_u32x4*)(uintptr_t)((act ? ox[h][c] : ow[h][c]) + st + (uint32_t)(block * 4096));
  };
  auto product = [&](auto fmt, const Frags& f) {
#pragma unroll
    for (int i = 0; i < BN; ++i)
#pragma unroll
      for (int j = 0; j < BM; ++j)
        acc[i][j] = mma<decltype(fmt)::value>(f.f[i ? i + BM : 0], f.f[1 + j], acc[i][j], s.w, s.x[j]);
  };
  // Issue order of a half: after each product the LDS reads and the loads
  // that fit beside it, the reads in the first half of the products so that
  // their data is there when the next half begins.
  constexpr int kM = BN * BM, kR = 2 * (BN + BM), kL = kLoadW + kLoadX;

  uint32_t cur = 0, nxt = kStage;  // stages of steps kb and kb + 1
  wait_vmcnt<(kStages - 1) * kL>();
  gemm::stage_barrier();
  Frags f0, f1;
#pragma unroll
  for (int i = 0; i < 2 * (BN + BM); ++i) read1(f0, 0, 0, i / 2, i % 2);
  // One step; `from` and `off` are those of the step kStages ahead.
  auto step = [&](auto fmt, const Source& from, int off) {
    constexpr int kP = decltype(fmt)::value == kBf16 ? 2 : 1;
#pragma unroll
    for (int i = 0; i < 2 * (BN + BM); ++i) read1(f1, cur, 1, i / 2, i % 2);
    product(fmt, f0);
    if constexpr (kM >= 4) {
      pace<kM / 2, kP, 0, 2 * kR / kM>();
      pace<kM / 2, kP, 0, 0>();
    }
    __builtin_amdgcn_sched_barrier(0);
    // The next step has landed when at most the moves of the kStages - 2 steps
    // after it are outstanding (they complete in order; a scale load among
    // them only makes this wait longer).
    wait_vmcnt<(kStages - 2) * kL>();
    gemm::stage_barrier();
    __builtin_amdgcn_sched_barrier(0);
    // The moves into the stage that is now free, and the reads of the next
    // step, in turn (their order is kept: both touch LDS).
#pragma unroll
    for (int i = 0; i < kL; ++i) {
      move(from, off, lds0 + cur, i);
      read1(f0, nxt, 0, i / 2, i % 2);
    }
    static_assert(kL == kR, "one move per piece");
    product(fmt, f1);
    if constexpr (kM >= 4) pace<kM, kP, kL / kM, kR / kM>();
    __builtin_amdgcn_sched_barrier(0);
    cur = nxt;
    nxt = nxt + kStage == kStages * kStage ? 0 : nxt + kStage;
  };
  constexpr std::integral_constant<int, kFmt> main_fmt;
  constexpr std::integral_constant<int, kBf16> low_fmt;
#pragma unroll 1
  for (int q = 0; q < LR; ++q) {
    const bool low = q + kStages < LR;
    const Source from = low ? lowrank : operands;
    step(low_fmt, from, low ? at_lowrank(q + kStages) : at_step(q + kStages - LR));
  }
  if constexpr (kFmt == kBf16) {
    if (p.keep) {  // dropped elements of the term become 0
      const int64_t mld = p.N / 32;
      const __amdgpu_buffer_rsrc_t rk = make_rsrc(p.keep + m0 * mld, (p.M - m0) * mld * 4);
#pragma unroll
      for (int j = 0; j < BM; ++j)
#pragma unroll
        for (int i = 0; i < BN; ++i) {
          const int word = (int)(n0 / 32) + wn * (WN / 32) + i;
          const uint32_t bits = __builtin_amdgcn_raw_buffer_load_b32(
              rk, (int)((wm * WM + j * 32 + r) * mld * 4), word * 4, 0) >> (half * 4);
#pragma unroll
          for (int v = 0; v < 16; ++v)
            if (!((bits >> ((v >> 2) * 8 + (v & 3))) & 1u)) acc[i][j][v] = 0.0f;
        }
    }
  }
  for (int kb4 = 0; kb4 < KB; kb4 += 4) {
    const Scales ahead = scales(kb4 + (kRuns ? 8 : 4));
    s = four(dw0, dw1);
    const int end = min(kb4 + 4, KB);
    for (int kb = kb4; kb < end; ++kb) {
      step(main_fmt, operands, at_step(kb + kStages));
      s.w >>= 8;
#pragma unroll
      for (int j = 0; j < BM; ++j) s.x[j] >>= 8;
    }
    dw0 = kRuns ? dw1 : ahead;
    dw1 = ahead;
  }
  wait_vmcnt<0>();  // no direct load may outlive the workgroup's LDS

  if constexpr (kGroups > 1) {
    constexpr int kAcc = BN * BM * 16;  // floats per lane
    const uint32_t at = lds_all + (uint32_t)(((wave * kAcc) * 64 + lane) * 4);
    for (int g = 1; g < kGroups; ++g) {
      __syncthreads();
      if (group == g) {
#pragma unroll
        for (int e = 0; e < kAcc; ++e)
          *(lds_f32*)(uintptr_t)(at + (uint32_t)(e * 256)) = acc[e / 16 / BM][e / 16 % BM][e % 16];
      }
      __syncthreads();
      if (group == 0) {
#pragma unroll
        for (int e = 0; e < kAcc; ++e)
          acc[e / 16 / BM][e / 16 % BM][e % 16] += *(const lds_f32*)(uintptr_t)(at + (uint32_t)(e * 256));
      }
    }
    if (group != 0) return;
  }
  if constexpr (kJoin) {
    static_assert(BN * BM == 1, "one accumulator");
    if (p.splits > 1 && !join_splits(acc[0][0], p, tile, split, lds_all)) return;
  }

  // Output by way of LDS (the ring is done with): a lane holds four
  // consecutive n of one row, 8 bytes; read back, 16 lanes hold a whole row
  // segment of the wave's part, and the stores are whole cache lines. Stored
  // straight from the accumulators, 8192^3 took 391 us, of which 30 were the
  // stores' 16-byte requests.
  constexpr int kOutPitch = WN * 2 + 16;
  constexpr int kOutBase = kGroups > 1 ? 4 * BN * BM * 16 * 256 : 0;
  static_assert(kOutBase + 4 * WM * kOutPitch <= lds_bytes(TN, TM, kStages, kGroups), "output fits the ring's LDS");
  const uint32_t ob = lds_all + (uint32_t)(kOutBase + wave * WM * kOutPitch);
  if constexpr (kGroups == 1) gemm::stage_barrier();
#pragma unroll
  for (int j = 0; j < BM; ++j)
#pragma unroll
    for (int i = 0; i < BN; ++i)
#pragma unroll
      for (int v = 0; v < 16; v += 4)
        *(lds_u32x2*)(uintptr_t)(ob + (uint32_t)((j * 32 + r) * kOutPitch + (i * 32 + (v >> 2) * 8 + half * 4) * 2)) =
            u32x2{pack_bf16x2(acc[i][j][v], acc[i][j][v + 1]), pack_bf16x2(acc[i][j][v + 2], acc[i][j][v + 3])};
  constexpr int kPieces = WN / 8;  // 16-byte pieces of a row
  auto put = [&](auto how) {  // 0: stores of single elements, 1: of pieces, 2: of pieces past the caches
    constexpr int kHow = decltype(how)::value;
#pragma unroll 8
    for (int q = 0; q < WM * kPieces / 64; ++q) {
      const int id = q * 64 + lane, row = id / kPieces, ch = id % kPieces;
      const u32x4 d = *(const lds_u32x4*)(uintptr_t)(ob + (uint32_t)(row * kOutPitch + ch * 16));
      const int64_t m = m0 + wm * WM + row, n = n0 + wn * WN + ch * 8;
      if (m >= p.M) continue;
      uint16_t* y = p.Y + m * p.N + n;
      if constexpr (kHow == 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (n + e < p.N) y[e] = (uint16_t)(d[e >> 1] >> (16 * (e & 1)));
      } else if (n < p.N) {
        if constexpr (kHow == 2) __builtin_nontemporal_store(d, reinterpret_cast<u32x4*>(y));
        else *reinterpret_cast<u32x4*>(y) = d;
      }
    }
  };
  if (p.N % 8 != 0 || (reinterpret_cast<uintptr_t>(p.Y) & 15) != 0) put(std::integral_constant<int, 0>{});
  else if (p.stream) put(std::integral_constant<int, 2>{});
  else put(std::integral_constant<int, 1>{});
#endif
}

__device__ __forceinline__ uint32_t lds_base() {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  return (uint32_t)(uintptr_t)((__attribute__((address_space(3))) uint8_t*)smem);
}

// 256 x 256 tiles, one workgroup per compute unit: the first `full` of the
// walk. The tiles that do not fill a last round are cut in `cut` parts (1, 2
// or 4), a workgroup each, so that more compute units share them.
template <int kXFmt>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1)))
fp8_gemm_kernel(Fp8Gemm p) {
  const uint32_t lds = lds_base();
  const int id = blockIdx.x;
  int tm, tn;
  if (id < p.full) {
    tile_at(p, xcd_order(id, p.full), tm, tn);
    gemm_tile<256, 256, 2, 1, kXFmt>(p, (int64_t)tn * 256, (int64_t)tm * 256, lds);
    return;
  }
  const int u = xcd_order(id - p.full, (int)gridDim.x - p.full);
  tile_at(p, p.full + u / p.cut, tm, tn);
  const int part = u % p.cut;
  const int64_t n0 = (int64_t)tn * 256, m0 = (int64_t)tm * 256;
  if (p.cut == 2) gemm_tile<256, 128, 3, 1, kXFmt>(p, n0, m0 + part * 128, lds);
  else gemm_tile<128, 128, 4, 1, kXFmt>(p, n0 + (part & 1) * 128, m0 + (part >> 1) * 128, lds);
}

// One tile size; several workgroups per compute unit. With NJ, the workgroups
// past the tiles do the column products of a backward pass, which need nothing
// of this product: they fill the compute units that a small one leaves idle.
template <int TN, int TM, int kStages, int kGroups, int kXFmt, int NJ>
__global__ void __launch_bounds__(NJ ? lr8::kThreads : 256 * kGroups)
__attribute__((amdgpu_waves_per_eu(2, kGroups > 2 ? 4 : 2)))
fp8_gemm_small_kernel(Fp8Gemm p, lr8::ColPair cols) {
  constexpr bool kJoin = TN == 64 && TM == 64;
  const int tiles = p.nM * p.nN, count = kJoin ? tiles * p.splits : tiles;
  if constexpr (NJ != 0) {
    if ((int)blockIdx.x >= count) return lr8::column_job<lr8::kAct8, NJ>(cols, blockIdx.x - count, lds_base());
    if (kGroups == 1 && threadIdx.x >= 256) return;
  }
  int tm, tn, tile = xcd_order(blockIdx.x, count), split = 0;
  if constexpr (kJoin) {  // an XCD's workgroups share runs of K
    split = tile / tiles;
    tile -= split * tiles;
  }
  tile_at(p, tile, tm, tn);
  gemm_tile<TN, TM, kStages, kGroups, kXFmt, kJoin>(p, (int64_t)tn * TN, (int64_t)tm * TM, lds_base(), tile, split);
}

// ---------------------------------------------------------------------------
// Few tokens: the time is that of a launch and of streaming the weight once
// (1 x 4096 x 4096, 17 MB: 6.4 us; 7.8 us where it forms T for r = 16). A
// workgroup owns 16 RN weight rows and 16 tokens over the whole of K, its eight
// waves a run of blocks each; both operands go from memory straight to registers
// (v_mfma_scale_f32_16x16x128_f8f6f4 takes a whole block), four blocks' loads
// in flight together, and the waves' sums meet in LDS in a fixed order. Two sets
// of four blocks in flight gained 2 to 5 % with 16 weight rows and spilled with
// 32. The adapter's term is added there in float32, from the split partials of T.
struct Fp8Few {
  Fp8Gemm g;
  const float* part;   // [splits][M][ldp] partials of T, or null
  const uint16_t* A;   // kR: [K x kR], 16-byte aligned
  int64_t K;
  int splits, ldp, r;
  float scale;
  const uint16_t* B;   // [r x N]
  float* T_out;        // [M x r] or null
};

// kR = 8 or 16: an adapter of that rank, T formed here by every workgroup, from
// A read beside the weight (A's rows pass through a wave's own LDS tile and
// come back by columns).
template <int RN, int kXFmt, int kR>
__global__ void __launch_bounds__(kFewWaves * 64) fp8_few_kernel(Fp8Few q) {
#ifdef __HIP_DEVICE_COMPILE__
  const Fp8Gemm& p = q.g;
  constexpr int kM = 16, kN = 16 * RN, kJ = 64;
  __shared__ floatx4 s_acc[kFewWaves][RN][64];
  __shared__ float s_t[kM][kJ + 1];
  __shared__ float s_y[kR ? 1 : kFewWaves * 64];
  constexpr int kPitch = 40;  // bytes of a row of the wave's tile of A
  __shared__ __attribute__((aligned(16))) uint8_t s_a[kR ? kFewWaves * 128 * kPitch : 16];
  __shared__ floatx4 s_tacc[kR ? kFewWaves : 1][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int i = lane & 15, g = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * kN, m0 = (int64_t)blockIdx.y * kM;

  const __amdgpu_buffer_rsrc_t rw = make_rsrc(p.w + n0 * p.ldc, min(p.N - n0, (int64_t)kN) * p.ldc);
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(p.x + m0 * p.ldc, min(p.M - m0, (int64_t)kM) * p.ldc);
  const __amdgpu_buffer_rsrc_t rsw = make_rsrc(p.ws + n0 / 128 * p.sb, p.sb);  // the tile is in one block row
  const __amdgpu_buffer_rsrc_t rsx = make_rsrc(p.xs + m0 * p.sb, (p.M - m0) * p.sb);
  floatx4 acc[RN];
#pragma unroll
  for (int a = 0; a < RN; ++a) acc[a] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};

  constexpr int kA = kR / 4;  // 16-byte pieces per lane of 128 rows of A
  const __amdgpu_buffer_rsrc_t ra = make_rsrc(q.A, q.K * kR * 2);
  const uint32_t at = (uint32_t)(uintptr_t)((__attribute__((address_space(3))) uint8_t*)s_a) +
                      (uint32_t)(wave * 128 * kPitch);
  // a sum for every eighth step of 64, in the order of row_product_kernel's
  // waves: T has the bits that a backward pass recomputes
  floatx4 tacc[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) tacc[c] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};

  // one output per thread: n = n0 + tid % kN, m = m0 + tid / kN; with kR its
  // column of B comes with the operands
  static_assert(kM * kN <= kFewWaves * 64, "a thread per output");
  const int nl = tid % kN, ml = tid / kN;
  const int64_t n = n0 + nl, m = m0 + ml;
  const bool mine = ml < kM && n < p.N && m < p.M;
  uint16_t b[kR ? kR : 1];
  if constexpr (kR != 0) {
    const __amdgpu_buffer_rsrc_t rb = make_rsrc(q.B, (int64_t)kR * p.N * 2);
#pragma unroll
    for (int j = 0; j < kR; ++j) b[j] = __builtin_amdgcn_raw_buffer_load_b16(rb, (int)n * 2, j * (int)p.N * 2, 0);
  }

  const int per = (p.KB + kFewWaves - 1) / kFewWaves;
  const int begin = wave * per, end = min(p.KB, begin + per);
  constexpr int kU = 4;
  for (int kb = begin; kb < end; kb += kU) {
    u32x4 w[kU][RN][2], x[kU][2], av[kU][kA ? kA : 1];
    uint32_t sw[kU], sx[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      // past the wave's run every offset is out of range: zeros
      const bool in = kb + u < end;
      const int off = in ? (kb + u) * 128 : kPastEnd;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int a = 0; a < RN; ++a)
          w[u][a][c] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
              rw, (int)((a * 16 + i) * p.ldc) + g * 16 + c * 64, off, 0));
        x[u][c] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
            rx, (int)(i * p.ldc) + g * 16 + c * 64, off, 0));
      }
      sw[u] = __builtin_amdgcn_raw_buffer_load_b8(rsw, 0, kb + u, 0);
      sx[u] = __builtin_amdgcn_raw_buffer_load_b8(rsx, i * p.sb, kb + u, 0);
#pragma unroll
      for (int e = 0; e < kA; ++e)
        av[u][e] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
            ra, (e * 64 + lane) * 16, in ? (kb + u) * (128 * kR * 2) : kPastEnd, 0));
    }
    // every load is on its way before the first product waits
    __builtin_amdgcn_sched_barrier(0);
    auto whole = [](const u32x4 (&f)[2]) {
      return i32x8{(int)f[0][0], (int)f[0][1], (int)f[0][2], (int)f[0][3],
                   (int)f[1][0], (int)f[1][1], (int)f[1][2], (int)f[1][3]};
    };
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int a = 0; a < RN; ++a)
        acc[a] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
            whole(w[u][a]), whole(x[u]), acc[a], 0, kXFmt, 0, (int)sw[u], 0, (int)sx[u]);
    if constexpr (kR != 0) {
      static_assert(kU == 4, "eight steps of 64 per turn of the loop");
#pragma unroll
      for (int u = 0; u < kU; ++u) {
#pragma unroll
        for (int e = 0; e < kA; ++e) {
          const int id = (e * 64 + lane) * 8;
          const uint32_t to = at + (uint32_t)(id / kR * kPitch + id % kR * 2);
          *(lds_u32x2*)(uintptr_t)to = u32x2{av[u][e][0], av[u][e][1]};
          *(lds_u32x2*)(uintptr_t)(to + 8) = u32x2{av[u][e][2], av[u][e][3]};
        }
        const float s = act8_scale((int)sx[u]);
#pragma unroll
        for (int c = 0; c < 4; ++c) {  // rows 64 (c / 2) + 16 g + 8 (c % 2) of the block
          const u32x4 xd = act8_decode8<kXFmt>(
              u32x2{x[u][c >> 1][2 * (c & 1)], x[u][c >> 1][2 * (c & 1) + 1]}, s);
          floatx4& t = tacc[2 * u + (c >> 1)];
          t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              as_bf16x8(xd), tr_frag<kPitch>(at, 64 * (c >> 1) + 16 * g + 8 * (c & 1), 0, lane), t, 0, 0, 0);
        }
      }
    }
  }
  if constexpr (kR != 0) {
    floatx4 t = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int v = 0; v < 4; ++v) t[v] += tacc[c][v] + tacc[c + 4][v];
    s_tacc[wave][lane] = t;
  }
#pragma unroll
  for (int a = 0; a < RN; ++a) s_acc[wave][a][lane] = acc[a];

  float y = 0.0f;
  if constexpr (kR != 0) {
    __syncthreads();
    if (tid < kM * kR) {
      // T's element (row 4 g + v, column i)
      const int tm = tid / kR, j = tid % kR;
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kFewWaves; ++w) v += s_tacc[w][(tm >> 2) * 16 + j][tm & 3];
      if (q.T_out && blockIdx.x == 0 && m0 + tm < p.M) q.T_out[(m0 + tm) * kR + j] = v;
      s_t[tm][j] = q.scale * v;
    }
    __syncthreads();
    if (mine) {
#pragma unroll
      for (int j = 0; j < kR; ++j) y += s_t[ml][j] * __builtin_bit_cast(float, (uint32_t)b[j] << 16);
    }
  } else if (q.part) {
    // The live rows (up to a power of two) by kN outputs, and as many threads
    // for each as there are then, every one with its own run of ranks
    // (1 x 4096 x 4096 from a graph: r = 64 14.3 -> 13.5 us, r = 256 22.6 -> 16.9).
    // Up to 16 ranks one thread, whose sum has the order of the one above.
    const int live = (int)min(p.M - m0, (int64_t)kM);
    const int rows = 1 << (32 - __builtin_clz(2 * live - 1)) >> 1, outs = rows * kN;
    const int js = q.r > 16 ? kFewWaves * 64 / outs : 1, o = tid & (outs - 1), jg = tid / outs, om = o / kN;
    const int64_t on = n0 + o % kN;
    for (int j0 = 0; j0 < q.r; j0 += kJ) {
      const int nj = min(kJ, q.r - j0);
      __syncthreads();
      for (int e = tid; e < rows * kJ; e += kFewWaves * 64) {
        const int64_t tm = m0 + e / kJ;
        const int j = e % kJ;
        float v = 0.0f;
        if (tm < p.M && j < nj) {
          const float* at = q.part + tm * q.ldp + j0 + j;
#pragma unroll 8
          for (int sp = 0; sp < q.splits; ++sp) v += at[(int64_t)sp * p.M * q.ldp];
          if (q.T_out && blockIdx.x == 0) q.T_out[tm * q.r + j0 + j] = v;
        }
        s_t[e / kJ][j] = q.scale * v;
      }
      __syncthreads();
      if (on < p.N && om < live && jg < js) {
        const int w = kJ / js, first = jg * w, many = min(w, nj - first);
        const uint16_t* bj = q.B + (int64_t)(j0 + first) * p.N + on;
#pragma unroll 16
        for (int j = 0; j < many; ++j)
          y += s_t[om][first + j] * __builtin_bit_cast(float, (uint32_t)bj[j * p.N] << 16);
      }
    }
    if (js > 1) {
      s_y[tid] = y;
      __syncthreads();
      y = 0.0f;
      if (tid < outs)
        for (int g = 0; g < js; ++g) y += s_y[g * outs + tid];
    }
  }
  __syncthreads();
  if (!mine) return;
  // accumulator (row 4 g + v, column i) of block a: n by row, m by column
  const int l = ((nl & 15) >> 2) * 16 + ml;
  float v = 0.0f;
#pragma unroll
  for (int w = 0; w < kFewWaves; ++w) v += s_acc[w][nl >> 4][l][nl & 3];
  p.Y[m * p.N + n] = (uint16_t)(pack_bf16x2(v + y, 0.0f) & 0xffffu);
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

template <int kXFmt>
hipError_t run_big(Fp8Gemm p, hipStream_t stream) {
  static std::atomic<uint64_t> raised{0};
  auto kern = fp8_gemm_kernel<kXFmt>;
  constexpr size_t lds = std::max({lds_bytes(256, 256, 2, 1), lds_bytes(256, 128, 3, 1), lds_bytes(128, 128, 4, 1)});
  hipError_t e = allow_lds(reinterpret_cast<const void*>(kern), lds, raised);
  if (e != hipSuccess) return e;
  p.nM = (int)((p.M + 255) / 256);
  p.nN = (int)((p.N + 255) / 256);
  p.group = 4;
  const int tiles = p.nM * p.nN;
  p.full = tiles / 256 * 256;
  const int rest = tiles - p.full;
  p.cut = rest <= 64 ? 4 : rest <= 128 ? 2 : 1;
  if (p.cut == 1) p.full = tiles;
  const int grid = p.full + (tiles - p.full) * p.cut;
  hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(256), lds, stream, p);
  return hipGetLastError();
}

template <int TN, int TM, int kStages, int kGroups, int kXFmt, int NJ>
hipError_t run_small(Fp8Gemm p, const lr8::ColPair& cols, hipStream_t stream) {
  static std::atomic<uint64_t> raised{0};
  auto kern = fp8_gemm_small_kernel<TN, TM, kStages, kGroups, kXFmt, NJ>;
  constexpr size_t lds = std::max(lds_bytes(TN, TM, kStages, kGroups), NJ ? lr8::column_lds(NJ) : 0);
  if (lds > 65536) {
    hipError_t e = allow_lds(reinterpret_cast<const void*>(kern), lds, raised);
    if (e != hipSuccess) return e;
  }
  p.nM = (int)((p.M + TM - 1) / TM);
  p.nN = (int)((p.N + TN - 1) / TN);
  p.group = 4;
  hipLaunchKernelGGL(kern, dim3((unsigned)(p.nM * p.nN * p.splits + (NJ ? cols.jobs : 0))),
                     dim3(NJ ? lr8::kThreads : 256 * kGroups), lds, stream, p, cols);
  return hipGetLastError();
}

template <int RN, int kXFmt, int kR>
hipError_t run_few(const Fp8Few& q, hipStream_t stream) {
  auto kern = fp8_few_kernel<RN, kXFmt, kR>;
  const dim3 grid((unsigned)((q.g.N + 16 * RN - 1) / (16 * RN)), (unsigned)((q.g.M + 15) / 16));
  hipLaunchKernelGGL(kern, grid, dim3(kFewWaves * 64), 0, stream, q);
  return hipGetLastError();
}

// Tile by the number of workgroups it gives. 256 x 256 moves the fewest
// operand bytes per product and is fastest once the chip is full (8192^3 with
// this tile 398 us when 128 x 128 in two workgroups per compute unit took 497);
// smaller tiles
// spread a small output over more compute units. From a graph of calls on
// rotating weights (us per call, 2 to 3 of them the graph's):
//   M x N x K            64 x 64   128 x 64   256 x 256 in parts
//   64 x 4096 x 4096     13.8 (14.4)  16.8 (17.5)   20.8
//   512 x 4096 x 4096    25.6 (20.7)  19.4 (20.4)   23.9
//   300 x 11008 x 4096   47.0 (33.7)  35.5 (29.7)   33.2
//   1000 x 512 x 512      5.4 (4.3)    6.7 (5.1)     6.9
// with two sets of waves, in brackets with one: two sets pay from about 16
// steps on, while every workgroup has a compute unit of its own.
//
// Up to 128 tiles of 64 x 64 are shared by several workgroups where each has 24
// steps or more (us in a graph, so and without): 64 x 4096 x 11008 r = 64 28.6
// and 37.0, 512 x 1024 x 11008 32.5 and 37.1; with 16 steps 512 x 1024 x 4096
// takes 22.1 instead of 20.8. Column products in the same launch keep some of
// the compute units (backward of 32 x 11008 x 4096 30.0 us, 31.5 if they do not
// and 35.1 without sharing).
//
// `cols`: column products to do besides, or null. They share the launch of a
// grid that leaves compute units idle, else they follow in their own (whole
// 8-bit backward, us in a graph, so and in two launches: 16 x 256 x 256 r = 8
// 7.8 and 10.3, 257 x 4096 x 4096 r = 8 26.9 and 30.8, 64 x 4096 x 4096 r = 64
// 23.6 and 28.3, 512 x 4096 x 4096 r = 64 with its 256 workgroups 36.5 and 37.2).
template <int kXFmt>
hipError_t run_fmt(Fp8Gemm p, const lr8::ColPair* cols, hipStream_t stream) {
  const int64_t mt = (p.M + 63) / 64;
  const int64_t t64 = mt * ((p.N + 63) / 64), t128 = mt * ((p.N + 127) / 128);
  const int64_t room = cols ? 160 : 256;  // workgroups
  p.splits = t64 <= 128 && p.done ? (int)std::max<int64_t>(1, std::min<int64_t>(room / t64, p.KB / 24)) : 1;
  const bool two = p.KB / p.splits >= 16;
  if (t128 <= 256) {
    auto small = [&](auto nj) {
      constexpr int NJ = decltype(nj)::value;
      const lr8::ColPair none{};
      const lr8::ColPair& c = NJ ? *cols : none;
      if (t64 <= 256)
        return two ? run_small<64, 64, 4, 2, kXFmt, NJ>(p, c, stream) : run_small<64, 64, 4, 1, kXFmt, NJ>(p, c, stream);
      return two ? run_small<128, 64, 3, 2, kXFmt, NJ>(p, c, stream) : run_small<128, 64, 3, 1, kXFmt, NJ>(p, c, stream);
    };
    return cols ? lr8::by_nj(cols->r, small) : small(std::integral_constant<int, 0>{});
  }
  const hipError_t e = t128 < 512 ? run_small<128, 64, 3, 1, kXFmt, 0>(p, lr8::ColPair{}, stream)
                                  : run_big<kXFmt>(p, stream);
  return cols && e == hipSuccess ? launch_columns(*cols, stream) : e;
}

// Y past the caches when it and the operands together outgrow the 256 MiB
// last-level cache: it would push out the operands, which every round of tiles
// reads again (4096 x 22016 x 8192: 514 us against 552; 8192 x 8192 x 1024,
// which fits, 73 us against 68).
bool streams_out(int64_t M, int64_t N, int64_t row_bytes) {
  return 2 * M * N + (M + N) * row_bytes > ((int64_t)256 << 20);
}

Fp8Gemm gemm_args(ConstAct8 x, ConstAct8 w, int64_t M, int64_t N, int64_t K, uint16_t* Y) {
  Fp8Gemm p{};
  p.x = x.codes; p.xs = x.scales; p.w = w.codes; p.ws = w.scales;
  p.M = M; p.N = N; p.ldc = act8_row_bytes(K);
  p.KB = (int)(p.ldc / kAct8Block);
  p.sb = (int)act8_scale_row_bytes(K);
  p.Y = Y;
  p.stream = streams_out(M, N, p.ldc);
  return p;
}

}  // namespace

hipError_t launch_fp8_gemm(ConstAct8 x, int xfmt, ConstAct8 w, int64_t M, int64_t N, int64_t K,
                           const uint16_t* U, const uint16_t* V, int r64, uint16_t* Y, TileSums sums,
                           const lr8::ColPair* cols, hipStream_t stream) {
  Fp8Gemm p = gemm_args(x, w, M, N, K, Y);
  p.U = U; p.V = V; p.r64 = r64; p.done = sums.done; p.sums = sums.sums;
  return xfmt ? run_fmt<1>(p, cols, stream) : run_fmt<0>(p, cols, stream);
}

hipError_t launch_bf16_gemm(const uint16_t* x, const uint16_t* w, int64_t M, int64_t N, int64_t K,
                            const uint16_t* U, const uint16_t* V, int r64, const uint32_t* keep,
                            uint16_t* Y, TileSums sums, const lr8::ColPair* cols, hipStream_t stream) {
  Fp8Gemm p{};
  p.x = reinterpret_cast<const uint8_t*>(x);
  p.w = reinterpret_cast<const uint8_t*>(w);
  p.M = M; p.N = N; p.ldc = K * 2;
  p.KB = (int)(K / 64);
  p.U = U; p.V = V; p.r64 = r64; p.keep = keep; p.Y = Y; p.done = sums.done; p.sums = sums.sums;
  p.stream = streams_out(M, N, p.ldc);
  return run_fmt<kBf16>(p, cols, stream);
}

bool fp8_few(int64_t M, int64_t N) { return (M + 15) / 16 * ((N + 15) / 16) <= 512; }

// Every workgroup reads all of A for it, beside its weight rows: worth a launch
// up to about 128 Ki elements (us per call from a graph, formed in the kernel
// and before it: 1 x 4096 x 4096 r = 16 9.8 and 11.4, 64 x 2048 x 2048 r = 16
// 9.3 and 13.7, 16 x 512 x 8192 r = 16 15.6 and 17.1, 1 x 4096 x 11008 r = 16
// 20.3 and 18.9).
bool few_t_shape(int64_t M, int64_t K, int r) {
  return M <= 64 && (r == 8 || r == 16) && K * r <= (int64_t)1 << 17;
}
bool fp8_few_forms_t(const uint16_t* A, int64_t M, int64_t K, int r) {
  return few_t_shape(M, K, r) && (reinterpret_cast<uintptr_t>(A) & 15) == 0;
}

hipError_t launch_fp8_few(ConstAct8 x, int xfmt, ConstAct8 w, int64_t M, int64_t N, int64_t K,
                          const uint16_t* A, const float* part, int splits, const uint16_t* B, int r,
                          float scale, uint16_t* Y, float* T_out, hipStream_t stream) {
  const Fp8Few q{gemm_args(x, w, M, N, K, Y), part, A, K, splits, lowrank_cols(r), r, scale, B, T_out};
  // 16 weight rows per workgroup while that leaves one per compute unit, else
  // 32 (32 x 4096 x 4096: 11.6 us against 13.8)
  const bool narrow = (M + 15) / 16 * ((N + 15) / 16) <= 256;
  auto go = [&](auto fmt, auto rank) {
    constexpr int kFmt = decltype(fmt)::value, kR = decltype(rank)::value;
    return narrow ? run_few<1, kFmt, kR>(q, stream) : run_few<2, kFmt, kR>(q, stream);
  };
  auto by_rank = [&](auto fmt) {
    if (!A) return go(fmt, std::integral_constant<int, 0>{});
    return r == 8 ? go(fmt, std::integral_constant<int, 8>{}) : go(fmt, std::integral_constant<int, 16>{});
  };
  return xfmt ? by_rank(std::integral_constant<int, 1>{}) : by_rank(std::integral_constant<int, 0>{});
}

}  // namespace qlora
