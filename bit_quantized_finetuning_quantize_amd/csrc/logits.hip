// Rows of logits: log-probabilities of given tokens with the row's entropy
// and its largest entries, distillation from a teacher's top logits, and the
// gradients of both.
//
// For a row z and a temperature t let x = (z - m) / t with m = max z, l = log
// sum exp x, p_j = exp(x_j - l). The forward passes read a row once and keep,
// per thread, a running maximum m, s = sum 2^y and (for the entropy) u = sum
// 2^y y, y = (z - m) log2(e) / t; a new maximum m' multiplies s by 2^d and
// turns u into 2^d (u + s d), d = (m - m') log2(e) / t. Then
//   l = ln s,   H = l - ln(2) u / s.
// z - m is formed before the product, so that logits near the type's lowest
// value, or far from zero, lose nothing.
#include "common.h"
#include "handover.h"
#include "kernels.h"

#include <algorithm>

namespace qlora {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kVecs = 4;             // vectors of 16 bytes a thread loads at once
constexpr int kUnit = 8192;          // parts of a row are multiples of this many elements
constexpr int kMaxUnits = 16;        // ... and at most this many of them
constexpr int kMaxParts = 32;
constexpr int kMaxTop = 64;
constexpr int kMaxItems = 2048;
constexpr int kMaxCand = kMaxParts * kMaxTop;
constexpr float kInf = __builtin_huge_valf();
constexpr float kLow = -1e30f;       // 0 * kLow is 0 where 0 * -inf would be NaN
constexpr double kLn2 = 0.693147180559945309417;

// A vector is 16 bytes at any element of a row: the loads and stores need no
// more than the elements' alignment, and cost the same (copying 512 MiB: 190 us
// aligned, 193 to 195 at odd elements; reading it 87 and 99).
typedef u32x4 u32x4_row __attribute__((aligned(2)));

template <bool kF32>
struct Elem {
  static constexpr int kE = kF32 ? 4 : 8;                       // elements of a vector
  static constexpr int kChunk = kThreads * kVecs * kE;          // a workgroup's loads of one step
  static constexpr int kBytes = kF32 ? 4 : 2;
};

template <bool kF32>
__device__ __forceinline__ u32x4 load_vec(const char* part, int v, int n);
// A thread's vectors of a step, the first of them v0: without a branch to a load
// where the whole step lies in the part.
template <bool kF32>
__device__ __forceinline__ void load_step(u32x4 (&r)[kVecs], const char* part, int c, int v0, int n) {
  if ((c + 1) * Elem<kF32>::kChunk <= n) {  // uniform
#pragma unroll
    for (int u = 0; u < kVecs; ++u)
      r[u] = *reinterpret_cast<const u32x4_row*>(part + (int64_t)(v0 + u * kThreads) * 16);
  } else {
#pragma unroll
    for (int u = 0; u < kVecs; ++u) r[u] = load_vec<kF32>(part, v0 + u * kThreads, n);
  }
}

// Vector v of a row part of n elements; elements past the end are -inf.
template <bool kF32>
__device__ __forceinline__ u32x4 load_vec(const char* part, int v, int n) {
  constexpr int kE = Elem<kF32>::kE;
  const int left = n - v * kE;
  if (left >= kE) return *reinterpret_cast<const u32x4_row*>(part + (int64_t)v * 16);
  if constexpr (kF32) {
    u32x4 r = {0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u};
    const uint32_t* e = reinterpret_cast<const uint32_t*>(part + (int64_t)v * 16);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) r[i] = e[i];
    return r;
  } else {
    u32x4 r = {0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u};
    const uint16_t* e = reinterpret_cast<const uint16_t*>(part + (int64_t)v * 16);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) {
        const uint32_t keep = (i & 1) ? 0x0000ffffu : 0xffff0000u;
        r[i >> 1] = (r[i >> 1] & keep) | ((uint32_t)e[i] << (16 * (i & 1)));
      }
    return r;
  }
}
template <bool kF32>
__device__ __forceinline__ void store_vec(char* part, int v, int n, u32x4 r) {
  constexpr int kE = Elem<kF32>::kE;
  const int left = n - v * kE;
  if (left >= kE) {
    *reinterpret_cast<u32x4_row*>(part + (int64_t)v * 16) = r;
    return;
  }
  if constexpr (kF32) {
    uint32_t* e = reinterpret_cast<uint32_t*>(part + (int64_t)v * 16);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) e[i] = r[i];
  } else {
    uint16_t* e = reinterpret_cast<uint16_t*>(part + (int64_t)v * 16);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) e[i] = (uint16_t)(r[i >> 1] >> (16 * (i & 1)));
  }
}

template <bool kF32>
__device__ __forceinline__ float elem(const u32x4& r, int i) {
  const uint32_t w = r[kF32 ? i : i >> 1];  // a copy: a bit cast of the element itself takes the first one's
  if constexpr (kF32) return __builtin_bit_cast(float, w);
  return (i & 1) ? bf16_hi(w) : bf16_lo(w);
}
template <bool kF32>
__device__ __forceinline__ float load_elem(const void* p, int64_t i) {
  if constexpr (kF32) return reinterpret_cast<const float*>(p)[i];
  return bf16_to_f32(reinterpret_cast<const uint16_t*>(p)[i]);
}
__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float base_of(float m) { return m == -kInf ? 0.0f : m; }

// A row part's statistics. u is used for the entropy only.
struct Soft {
  float m, s, u;
};
constexpr Soft kNone{-kInf, 0.0f, 0.0f};
__device__ __forceinline__ Soft rescaled(const Soft& a, float m, float c2) {
  const float d = (a.m - base_of(m)) * c2, r = exp2_(d);
  return Soft{m, a.s * r, r * (a.u + a.s * fmaxf(d, kLow))};
}
__device__ __forceinline__ Soft joined(const Soft& a, const Soft& b, float c2) {
  const float m = fmaxf(a.m, b.m);
  const Soft x = rescaled(a, m, c2), y = rescaled(b, m, c2);
  return Soft{m, x.s + y.s, x.u + y.u};
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}
template <typename T>
__device__ __forceinline__ T wave_sum(T v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
  return v;
}
__device__ __forceinline__ Soft wave_join(const Soft& a, float c2) {
  Soft r = rescaled(a, wave_max(a.m), c2);
  r.s = wave_sum(r.s);
  r.u = wave_sum(r.u);
  return r;
}

// ---------------------------------------------------------------------------
// Order of a row's entries: larger first, of equal ones the lower index first.
// key: unsigned order of floats, -0 and +0 alike, NaN below everything.
__device__ __forceinline__ uint32_t key_of(float z) {
  if (z != z) return 0;
  const uint32_t u = __builtin_bit_cast(uint32_t, z + 0.0f);
  return (u >> 31) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float of_key(uint32_t k) {
  if (k == 0) return __builtin_nanf("");
  return __builtin_bit_cast(float, (k >> 31) ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ uint64_t pair_of(uint32_t key, uint32_t idx) {
  return ((uint64_t)key << 32) | (0xffffffffu - idx);
}
__device__ __forceinline__ uint32_t idx_of(uint64_t pair) { return 0xffffffffu - (uint32_t)pair; }

template <int kCtrl, int kRows>
__device__ __forceinline__ uint64_t dpp64(uint64_t v) {
  const int lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)v, kCtrl, kRows, 0xf, true);
  const int hi = __builtin_amdgcn_update_dpp(0, (int)(v >> 32), kCtrl, kRows, 0xf, true);
  return ((uint64_t)(uint32_t)hi << 32) | (uint32_t)lo;
}
__device__ __forceinline__ uint64_t larger(uint64_t a, uint64_t b) { return a > b ? a : b; }
// Largest over the wave (every lane active), the same in every lane.
__device__ __forceinline__ uint64_t wave_largest(uint64_t v) {
  v = larger(v, dpp64<0x111, 0xf>(v));  // row_shr 1, 2, 4, 8
  v = larger(v, dpp64<0x112, 0xf>(v));
  v = larger(v, dpp64<0x114, 0xf>(v));
  v = larger(v, dpp64<0x118, 0xf>(v));
  v = larger(v, dpp64<0x142, 0xa>(v));  // row_bcast 15, 31
  v = larger(v, dpp64<0x143, 0xc>(v));
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)v, 63);
  const uint32_t hi = __builtin_amdgcn_readlane((int)(v >> 32), 63);
  return ((uint64_t)hi << 32) | lo;
}
// The r-th largest of the lanes' values (with multiplicity).
__device__ __forceinline__ uint64_t wave_rth(uint64_t v, int r) {
  uint64_t top = wave_largest(v);
  for (int i = 1; i < r; ++i) {
    const uint64_t at = __ballot(v == top);
    if ((int)(threadIdx.x & 63) == __builtin_ctzll(at)) v = 0;
    top = wave_largest(v);
  }
  return top;
}

// ---------------------------------------------------------------------------
// Forward.

enum { kLogprobs, kDistill, kDistillRest };

struct RowsFwd {
  const char* Z;
  int64_t ldz;  // in bytes
  int V, S, part;  // parts of a row, elements of a part
  float c2, inv_t;
  float* stats;
  // log-probabilities
  const int64_t* target;
  float *logp, *entropy;
  int n_top;
  int64_t* top_ids;
  float* top_logp;
  // distillation
  const int64_t* ids;
  const void* values;
  int values_f32, k;
  const float* teacher_lse;
  double inv_t64;
  float* loss;
  // where rows are split
  uint64_t* flags;  // [T][S]
  float* sums;      // [T][S][4]
  uint64_t* lists;  // [T][S][n_top]
};

__device__ __forceinline__ void put_agent(float* p, float v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float get_agent(const float* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// LDS of the selection of a part's largest entries.
struct TopLds {
  uint64_t cand[kMaxCand];
  uint64_t wave[kWaves];
  uint16_t items[kMaxItems];
  int n_items, n_cand;
};

// Ranks the candidates (all pairs differ) and hands the first `need` to put.
template <typename Put>
__device__ __forceinline__ void rank_candidates(const TopLds& t, int count, int need, Put put) {
  for (int i = threadIdx.x; i < count; i += kThreads) {
    const uint64_t mine = t.cand[i];
    int rank = 0;
    for (int j = 0; j < count; ++j) rank += t.cand[j] > mine;
    if (rank < need) put(rank, mine);
  }
}

// The `need` largest entries of a part. bins [chunks][kThreads]: key of the
// maximum of each thread's vectors of each step; best: the thread's largest
// bin as (key, first index of the step), an upper bound in that coarser order
// for all its entries, and attained by one of them unless they are all NaN.
// The r-th largest of them in each of w full waves, r = need / w rounded up,
// has r entries at or above it in that wave, so the smallest of the waves'
// has `need`: only the bins that reach it are read again (from the L2), and
// what reaches it there is ranked.
template <bool kF32, typename Put>
__device__ __forceinline__ void select_top(const char* part, int n, int first, int chunks,
                                           const uint32_t* bins, uint64_t best, int need, TopLds& t,
                                           Put put) {
  constexpr int kE = Elem<kF32>::kE, kChunk = Elem<kF32>::kChunk;
  const int tid = threadIdx.x, wave = tid >> 6;
  const int full = min(kWaves, n / kE / 64);  // waves whose lanes all hold an entry
  if (full) {
    const uint64_t r = wave_rth(best, (need + full - 1) / full);
    if ((tid & 63) == 0) t.wave[wave] = r;
  }
  if (tid == 0) t.n_items = t.n_cand = 0;
  __syncthreads();
  uint64_t t0 = full ? ~0ull : 0;
  for (int w = 0; w < full; ++w) t0 = t.wave[w] < t0 ? t.wave[w] : t0;
  auto coarse = [&](uint32_t key, int b) { return pair_of(key, (uint32_t)(first + b * kChunk)); };
  for (int b = 0; b < chunks; ++b) {
    const uint32_t key = bins[b * kThreads + tid];
    if (key && coarse(key, b) >= t0) {
      const int i = atomicAdd(&t.n_items, 1);
      if (i < kMaxItems) t.items[i] = (uint16_t)(b * kThreads + tid);
    }
  }
  __syncthreads();
  const int items = t.n_items;
  // f(key, index, step) over the entries of the bins listed, or of all
  auto each = [&](bool all, auto f) {
    const int units = (all ? chunks * kThreads : items) * kVecs;
    for (int w = tid; w < units; w += kThreads) {
      const int it = all ? w / kVecs : t.items[w / kVecs];
      const int b = it / kThreads, v = (b * kVecs + w % kVecs) * kThreads + it % kThreads;
      if (v * kE >= n) continue;
      const u32x4 x = load_vec<kF32>(part, v, n);
#pragma unroll
      for (int i = 0; i < kE; ++i)
        if (v * kE + i < n) f(key_of(elem<kF32>(x, i)), (uint32_t)(first + v * kE + i), b);
    }
  };
  bool all = items > kMaxItems;
  if (!all)
    each(false, [&](uint32_t key, uint32_t idx, int b) {
      if (coarse(key, b) < t0) return;
      const int i = atomicAdd(&t.n_cand, 1);
      if (i < kMaxCand) t.cand[i] = pair_of(key, idx);
    });
  __syncthreads();
  const int count = t.n_cand;
  if (!all && count >= need && count <= kMaxCand) {
    rank_candidates(t, count, need, put);
    return;
  }
  // Many equal entries, or NaN: one entry after another.
  all = all || count < need;
  uint64_t prev = ~0ull;
  for (int r = 0; r < need; ++r) {
    uint64_t top = 0;
    each(all, [&](uint32_t key, uint32_t idx, int) {
      const uint64_t p = pair_of(key, idx);
      if (p < prev && p > top) top = p;
    });
    top = wave_largest(top);
    __syncthreads();
    if ((tid & 63) == 0) t.wave[wave] = top;
    __syncthreads();
    for (int w = 0; w < kWaves; ++w) top = larger(top, t.wave[w]);
    if (tid == 0) put(r, top);
    prev = top;
  }
}

// One (row, part) per workgroup. Where a row has several, each stores its
// statistics and then a flag holding the dispatch's tag, and looks at all the
// row's flags: stores and looks are performed in one memory, so the workgroup
// whose flag comes last sees them all, and goes on with the row (if two see
// them all, both write the same values). None waits for another, and the
// flags need no clearing.
// kBins: steps whose maxima are kept for the largest entries; 0 for none.
template <bool kF32, int kOp, bool kTop>
__global__ void __launch_bounds__(kThreads) rows_fwd_kernel(RowsFwd a) {
  constexpr int kE = Elem<kF32>::kE, kChunk = Elem<kF32>::kChunk;
  extern __shared__ __attribute__((aligned(16))) uint8_t dyn[];
  __shared__ Soft s_soft[2][kWaves];
  __shared__ int s_last;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t row = blockIdx.x / (uint32_t)a.S;
  const int split = (int)(blockIdx.x - (uint32_t)row * (uint32_t)a.S);
  const int first = split * a.part, n = min(a.part, a.V - first);
  const char* zrow = a.Z + row * a.ldz;
  const char* part = zrow + (int64_t)first * Elem<kF32>::kBytes;
  const int chunks = (n + kChunk - 1) / kChunk;
  const float c2 = a.c2;

  TopLds& top = *reinterpret_cast<TopLds*>(dyn);
  uint32_t* bins = reinterpret_cast<uint32_t*>(dyn + sizeof(TopLds));
  uint32_t* mask = reinterpret_cast<uint32_t*>(dyn);  // bit i: entry first + i is on the list
  if constexpr (kOp == kDistillRest) {
    const int words = (n + 127) / 128 * 4;
    for (int i = tid * 4; i < words; i += kThreads * 4) *reinterpret_cast<u32x4*>(mask + i) = u32x4{0, 0, 0, 0};
    __syncthreads();
    for (int i = tid; i < a.k; i += kThreads) {
      const int64_t at = a.ids[row * a.k + i] - first;
      if (at >= 0 && at < n) atomicOr(mask + (at >> 5), 1u << (at & 31));
    }
    __syncthreads();
  }

  Soft acc = kNone, list = kNone;  // list: the listed entries, where they are kept apart
  uint64_t best = 0;
  for (int c = 0; c < chunks; ++c) {
    u32x4 r[kVecs];
    const int v0 = c * kVecs * kThreads + tid;
    load_step<kF32>(r, part, c, v0, n);
    float z[kVecs * kE];
#pragma unroll
    for (int u = 0; u < kVecs; ++u)
#pragma unroll
      for (int i = 0; i < kE; ++i) z[u * kE + i] = elem<kF32>(r[u], i);
    if constexpr (kOp == kDistillRest) {
#pragma unroll
      for (int u = 0; u < kVecs; ++u) {
        const int v = v0 + u * kThreads;
        uint32_t b = 0;
        if (v * kE < n)
          b = kF32 ? (reinterpret_cast<const uint8_t*>(mask)[v >> 1] >> (4 * (v & 1))) & 15u
                   : reinterpret_cast<const uint8_t*>(mask)[v];
        if (b) {
#pragma unroll
          for (int i = 0; i < kE; ++i)
            if ((b >> i) & 1) {
              list = joined(list, Soft{z[u * kE + i], z[u * kE + i] == -kInf ? 0.0f : 1.0f, 0.0f}, c2);
              z[u * kE + i] = -kInf;
            }
        }
      }
    }
    float m = z[0];
#pragma unroll
    for (int i = 1; i < kVecs * kE; ++i) m = fmaxf(m, z[i]);
    if constexpr (kTop) {
      const uint32_t key = v0 * kE < n ? key_of(m) : 0;
      bins[c * kThreads + tid] = key;
      if (key) best = larger(best, pair_of(key, (uint32_t)(first + c * kChunk)));
    }
    m = fmaxf(m, acc.m);
    const float base = base_of(m);
    float s[4] = {0, 0, 0, 0}, q[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < kVecs * kE; ++i) {
      const float y = (z[i] - base) * c2;
      const float e = exp2_(y);
      s[i & 3] += e;
      if constexpr (kOp == kLogprobs) q[i & 3] = __builtin_fmaf(e, fmaxf(y, kLow), q[i & 3]);
    }
    acc = rescaled(acc, m, c2);
    acc.s += (s[0] + s[1]) + (s[2] + s[3]);
    acc.u += (q[0] + q[1]) + (q[2] + q[3]);
  }

  // the workgroup's statistics, the same in every thread
  acc = wave_join(acc, c2);
  if (lane == 0) s_soft[0][wave] = acc;
  if constexpr (kOp == kDistillRest) {
    list = wave_join(list, c2);
    if (lane == 0) s_soft[1][wave] = list;
  }
  __syncthreads();
  acc = s_soft[0][0];
  for (int w = 1; w < kWaves; ++w) acc = joined(acc, s_soft[0][w], c2);
  if constexpr (kOp == kDistillRest) {
    list = s_soft[1][0];
    for (int w = 1; w < kWaves; ++w) list = joined(list, s_soft[1][w], c2);
  }

  if (a.S > 1) {
    const int64_t at = row * a.S + split;
    if constexpr (kTop) {
      const int need = min(a.n_top, n);
      uint64_t* mine = a.lists + at * a.n_top;
      auto put = [&](int r, uint64_t p) {
        __hip_atomic_store(mine + r, p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      };
      if (tid >= need && tid < a.n_top) put(tid, 0);
      select_top<kF32>(part, n, first, chunks, bins, best, need, top, put);
    }
    if (tid == 0) {
      put_agent(a.sums + at * 4, acc.m);
      put_agent(a.sums + at * 4 + 1, acc.s);
      put_agent(a.sums + at * 4 + 2, kOp == kLogprobs ? acc.u : list.m);
      put_agent(a.sums + at * 4 + 3, list.s);
    }
    // every store of the workgroup acknowledged before its flag
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (wave == 0) {
      const uint64_t tag = call_tag();
      uint64_t* flags = a.flags + row * a.S;
      if (lane == 0) {
        const uint64_t was = __hip_atomic_exchange(flags + split, tag, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        asm volatile("" ::"v"((uint32_t)was));  // performed before the looks below
      }
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      const uint64_t zero = (uint64_t)(a.V >> 30);  // an addition that the compiler keeps
      const bool there = lane >= a.S || __hip_atomic_fetch_add(flags + (lane < a.S ? lane : 0), zero, __ATOMIC_RELAXED,
                                                               __HIP_MEMORY_SCOPE_AGENT) == tag;
      if (lane == 0) s_last = 0;
      if (__all(there) && lane == 0) s_last = 1;
    }
    __syncthreads();
    if (!s_last) return;
    acc = list = kNone;
    if (lane < a.S) {
      const float* p = a.sums + (row * a.S + lane) * 4;
      acc.m = get_agent(p);
      acc.s = get_agent(p + 1);
      (kOp == kLogprobs ? acc.u : list.m) = get_agent(p + 2);
      list.s = get_agent(p + 3);
    }
    acc = wave_join(acc, c2);
    if constexpr (kOp == kDistillRest) list = wave_join(list, c2);
  }

  if constexpr (kOp == kLogprobs) {
    const bool empty = acc.m == -kInf && acc.s == 0.0f;
    const float l = empty ? 0.0f : logf(acc.s);
    auto logp_of = [&](float z) { return empty ? -kInf : (z - acc.m) * a.inv_t - l; };
    if (tid == 0) {
      const float H = empty ? 0.0f : l - (float)kLn2 * (acc.u / acc.s);
      if (a.entropy) a.entropy[row] = H;
      if (a.stats) {
        a.stats[row * 3] = acc.m;
        a.stats[row * 3 + 1] = l;
        a.stats[row * 3 + 2] = H;
      }
      if (a.logp) {
        const int64_t y = a.target[row];
        a.logp[row] = y >= 0 && y < a.V ? logp_of(load_elem<kF32>(zrow, y)) : 0.0f;
      }
    }
    if constexpr (kTop) {
      auto put = [&](int r, uint64_t p) {
        a.top_ids[row * a.n_top + r] = (int64_t)idx_of(p);
        a.top_logp[row * a.n_top + r] = logp_of(of_key((uint32_t)(p >> 32)));
      };
      if (a.S == 1) {
        select_top<kF32>(part, n, 0, chunks, bins, best, a.n_top, top, put);
      } else {
        // the parts' lists are sorted, and all but the last are whole: each has
        // r = n_top / (S - 1) rounded up entries at or above its r-th
        const uint64_t* lists = a.lists + row * a.S * a.n_top;
        const int r = (a.n_top + a.S - 2) / (a.S - 1);
        auto get = [&](int i) {
          return __hip_atomic_load(lists + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        };
        const uint64_t t0 = ~wave_largest(lane < a.S - 1 ? ~get(lane * a.n_top + r - 1) : 0);
        __syncthreads();
        if (tid == 0) top.n_cand = 0;
        __syncthreads();
        for (int i = tid; i < a.S * a.n_top; i += kThreads) {
          const uint64_t p = get(i);
          if (p && p >= t0) top.cand[atomicAdd(&top.n_cand, 1)] = p;
        }
        __syncthreads();
        rank_candidates(top, top.n_cand, a.n_top, put);
      }
    }
  } else {
    // one wave: up to four list entries a lane, in 64 bits
    if (wave) return;
    constexpr int kPer = 4;
    const int64_t at = row * a.k;
    bool ok[kPer];
    float t[kPer], z[kPer];
    float tm = -kInf;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = i * 64 + lane;
      const int64_t id = e < a.k ? a.ids[at + e] : -1;
      ok[i] = id >= 0 && id < a.V;
      t[i] = z[i] = -kInf;
      if (ok[i]) {
        t[i] = a.values_f32 ? load_elem<true>(a.values, at + e) : load_elem<false>(a.values, at + e);
        z[i] = load_elem<kF32>(zrow, id);
      }
      ok[i] = ok[i] && t[i] != -kInf;
      tm = fmaxf(tm, t[i]);
    }
    tm = wave_max(tm);
    if (tm == -kInf) tm = 0.0f;
    double rel[kPer], sum = 0.0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      rel[i] = ((double)t[i] - tm) * a.inv_t64;
      if (kOp == kDistill && ok[i]) sum += exp(rel[i]);
    }
    double tl;
    if constexpr (kOp == kDistillRest) {
      tl = (double)a.teacher_lse[row] - (double)tm * a.inv_t64;
    } else {
      sum = wave_sum(sum);
      tl = sum > 0.0 ? log(sum) : 0.0;
    }
    // the student's log sums over m = the larger maximum: of the rest, of the list
    const float m = kOp == kDistillRest ? fmaxf(acc.m, list.m) : acc.m;
    const bool empty = m == -kInf && acc.s == 0.0f && list.s == 0.0f;
    double l = 0.0, logr = 0.0;
    bool rest = false;
    if (!empty) {
      if constexpr (kOp == kDistillRest) {
        rest = acc.s != 0.0f;
        const double r = rest ? log((double)acc.s) + ((double)acc.m - m) * a.inv_t64 : -(double)kInf;
        const double g = list.s != 0.0f ? log((double)list.s) + ((double)list.m - m) * a.inv_t64 : -(double)kInf;
        const double hi = r > g ? r : g, lo = r > g ? g : r, d = log1p(exp(lo - hi));
        l = hi + d;
        logr = r > g ? -d : (r - g) - d;
        if (r != r || g != g) l = logr = r + g;
      } else {
        l = log((double)acc.s);
      }
    }
    double q_sum = 0.0, loss = 0.0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (!ok[i]) continue;
      const double q = exp(rel[i] - tl);
      const double logp = empty ? -(double)kInf : ((double)z[i] - m) * a.inv_t64 - l;
      q_sum += q;
      if (!(q <= 0.0)) loss += q * (rel[i] - tl - logp);
    }
    q_sum = wave_sum(q_sum);
    loss = wave_sum(loss);
    double w = q_sum, off = q_sum;
    if constexpr (kOp == kDistillRest) {
      double qr = 1.0 - q_sum;
      if (qr < 0.0) qr = 0.0;
      if (rest && !(qr <= 0.0)) {
        const double logq = log(qr);
        loss += qr * (logq - logr);
        w += qr;
        off = w - exp(logq - logr);
      }
    }
    if (lane == 0) {
      constexpr double kTop32 = 3.402823466e38;
      a.loss[row] = (float)loss;
      if (a.stats) {
        float* s = a.stats + row * 6;
        s[0] = m;
        s[1] = (float)l;
        s[2] = (float)w;
        s[3] = (float)(off < -kTop32 ? -kTop32 : off);
        s[4] = tm;
        s[5] = (float)tl;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Backward: one pass, dz in z's place if the caller wants it.

struct RowsBwd {
  const char* Z;
  int64_t ldz;  // in bytes
  char* dZ;
  int64_t lddz;
  int V, S, part;
  float c2, inv_t;
  const float* stats;
  const int64_t* target;
  const float *g_logp, *g_entropy;
  const int64_t* ids;
  const void* values;
  int values_f32, k;
  const float* g;
};

template <bool kF32>
__device__ __forceinline__ u32x4 pack_vec(const float* f) {
  if constexpr (kF32) {
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = __builtin_bit_cast(uint32_t, f[i]);
    return r;
  } else {
    return u32x4{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])};
  }
}

// f(v, value) over the vectors of a part: the new value of each element.
template <bool kF32, typename F>
__device__ __forceinline__ void map_part(const char* z, char* dz, int n, F f) {
  constexpr int kE = Elem<kF32>::kE, kChunk = Elem<kF32>::kChunk;
  for (int c = 0; c * kChunk < n; ++c) {
    const int v0 = c * kVecs * kThreads + (int)threadIdx.x;
    u32x4 r[kVecs];
    load_step<kF32>(r, z, c, v0, n);
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      const int v = v0 + u * kThreads;
      if (v * kE >= n) continue;
      float x[kE];
#pragma unroll
      for (int i = 0; i < kE; ++i) x[i] = elem<kF32>(r[u], i);
      f(v, x);
      store_vec<kF32>(dz, v, n, pack_vec<kF32>(x));
    }
  }
}
template <bool kF32>
__device__ __forceinline__ void zero_part(char* dz, int n) {
  for (int v = threadIdx.x; v * Elem<kF32>::kE < n; v += kThreads)
    store_vec<kF32>(dz, v, n, u32x4{0, 0, 0, 0});
}

// dz_j = (g ([j = target] - p_j) - h p_j (log p_j + H)) / t.
template <bool kF32>
__global__ void __launch_bounds__(kThreads) logprobs_bwd_kernel(RowsBwd a) {
  constexpr int kE = Elem<kF32>::kE;
  const int64_t row = blockIdx.x / (uint32_t)a.S;
  const int first = (int)(blockIdx.x - (uint32_t)row * (uint32_t)a.S) * a.part, n = min(a.part, a.V - first);
  const char* z = a.Z + row * a.ldz + (int64_t)first * Elem<kF32>::kBytes;
  char* dz = a.dZ + row * a.lddz + (int64_t)first * Elem<kF32>::kBytes;
  const float m = a.stats[row * 3], l = a.stats[row * 3 + 1], H = a.stats[row * 3 + 2];
  const int64_t y = a.target ? a.target[row] : -1;
  const float g = a.g_logp && y >= 0 && y < a.V ? a.g_logp[row] : 0.0f;
  const float h = a.g_entropy ? a.g_entropy[row] : 0.0f;
  if ((m == -kInf && l == 0.0f) || (g == 0.0f && h == 0.0f)) {
    zero_part<kF32>(dz, n);
    return;
  }
  const float c2 = a.c2, l2 = l * 1.44269504088896340736f;
  const float ca = -(g + h * H) * a.inv_t, cb = -h * (float)kLn2 * a.inv_t, one = g * a.inv_t;
  const int hot = (int)(y - first);  // may lie outside the part
  map_part<kF32>(z, dz, n, [&](int v, float* x) {
#pragma unroll
    for (int i = 0; i < kE; ++i) {
      const float p2 = __builtin_fmaf(x[i] - m, c2, -l2);
      x[i] = exp2_(p2) * __builtin_fmaf(cb, fmaxf(p2, kLow), ca);
    }
    if (y >= 0 && hot >= 0 && hot / kE == v) {
#pragma unroll
      for (int i = 0; i < kE; ++i) x[i] += hot % kE == i ? one : 0.0f;
    }
  });
}

// dz_j = g / t (w p_j - q_j) on the list, g / t off p_j off it. Every element
// is first written as one off the list; the listed ones, whose logits were
// read before, after that.
template <bool kF32>
__global__ void __launch_bounds__(kThreads) distill_bwd_kernel(RowsBwd a) {
  __shared__ int s_id[kThreads];
  __shared__ float s_q[kThreads];
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x / (uint32_t)a.S;
  const int first = (int)(blockIdx.x - (uint32_t)row * (uint32_t)a.S) * a.part, n = min(a.part, a.V - first);
  const char* z = a.Z + row * a.ldz + (int64_t)first * Elem<kF32>::kBytes;
  char* dz = a.dZ + row * a.lddz + (int64_t)first * Elem<kF32>::kBytes;
  const float* s = a.stats + row * 6;
  const float m = s[0], l2 = s[1] * 1.44269504088896340736f, w = s[2], off = s[3];
  const float gt = a.g[row] * a.inv_t;
  if ((m == -kInf && s[1] == 0.0f) || gt == 0.0f) {
    zero_part<kF32>(dz, n);
    return;
  }
  const float c2 = a.c2;
  int id = -1;
  float zi = -kInf, q = 0.0f;
  if (tid < a.k) {
    const int64_t at = row * a.k + tid, j = a.ids[at] - first;
    if (j >= 0 && j < n) {
      id = (int)j;
      zi = load_elem<kF32>(z, j);
      const float t = a.values_f32 ? load_elem<true>(a.values, at) : load_elem<false>(a.values, at);
      if (t != -kInf) q = exp2_(__builtin_fmaf(t - s[4], c2, -s[5] * 1.44269504088896340736f));
    }
  }
  s_id[tid] = id;
  s_q[tid] = q;
  // the listed logits are in registers before any wave writes over them
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  bool mine = id >= 0;
  if (mine) {  // an id twice: its first entry takes the sum
    q = 0.0f;
    for (int i = 0; i < a.k; ++i) {
      const bool same = s_id[i] == id;
      q += same ? s_q[i] : 0.0f;
      mine = mine && !(same && i < tid);
    }
  }
  // off p_j as one power of two: off may be as large as p_j is small
  const float go = off < 0.0f ? -gt : gt, shift = __log2f(fabsf(off)) - l2;
  map_part<kF32>(z, dz, n, [&](int, float* x) {
#pragma unroll
    for (int i = 0; i < Elem<kF32>::kE; ++i) x[i] = exp2_(__builtin_fmaf(x[i] - m, c2, shift)) * go;
  });
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (mine) {
    const float p = exp2_(__builtin_fmaf(zi - m, c2, -l2));
    const float v = gt * __builtin_fmaf(p, w, -q);
    if constexpr (kF32)
      reinterpret_cast<float*>(dz)[id] = v;
    else
      reinterpret_cast<uint16_t*>(dz)[id] = (uint16_t)(pack_bf16x2(v, 0.0f) & 0xffffu);
  }
}

// Parts of a row in the forward passes.
struct Parts {
  int S, part;
};
Parts fwd_parts(int64_t T, int64_t V) {
  const int64_t units = (V + kUnit - 1) / kUnit;
  int64_t S = std::min<int64_t>({(int64_t)kMaxParts, units, (1024 + T - 1) / T});
  S = std::max(S, (units + kMaxUnits - 1) / kMaxUnits);
  const int64_t per = (units + S - 1) / S;
  return Parts{(int)((units + per - 1) / per), (int)(per * kUnit)};
}
// ... and in the backward passes: more of it to a workgroup where there are many rows.
Parts bwd_parts(int64_t T, int64_t V) {
  const int64_t units = (V + kUnit - 1) / kUnit, per = T * units >= 4096 ? 4 : 1;
  return Parts{(int)((units + per - 1) / per), (int)(per * kUnit)};
}

int64_t up256(int64_t n) { return (n + 255) / 256 * 256; }

void carve(RowsFwd& a, int64_t T, int n_top, void* ws) {
  char* p = reinterpret_cast<char*>(ws);
  a.flags = reinterpret_cast<uint64_t*>(p);
  p += up256(T * a.S * 8);
  a.sums = reinterpret_cast<float*>(p);
  p += up256(T * a.S * 16);
  a.lists = reinterpret_cast<uint64_t*>(p);
}

template <bool kF32, int kOp, bool kTop>
hipError_t run_fwd(const RowsFwd& a, int64_t T, hipStream_t stream) {
  size_t lds = 0;
  if (kOp == kDistillRest) lds = ((size_t)std::min(a.part, a.V) + 127) / 128 * 16;
  if (kTop) lds = sizeof(TopLds) + (size_t)((std::min(a.part, a.V) + Elem<kF32>::kChunk - 1) / Elem<kF32>::kChunk) * kThreads * 4;
  rows_fwd_kernel<kF32, kOp, kTop><<<dim3((unsigned)(T * a.S)), dim3(kThreads), lds, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

size_t logits_workspace_bytes(int64_t T, int64_t V, int n_top) {
  const Parts p = fwd_parts(T, V);
  if (p.S == 1) return 256;
  return (size_t)(up256(T * p.S * 8) + up256(T * p.S * 16) + up256(T * p.S * 8 * n_top));
}

hipError_t launch_logprobs_fwd(const Logits& z, const int64_t* target, float* logp, float* entropy, int n_top,
                               int64_t* top_ids, float* top_logp, float* stats, void* ws, hipStream_t stream) {
  const Parts p = fwd_parts(z.T, z.V);
  RowsFwd a{};
  a.Z = reinterpret_cast<const char*>(z.Z);
  a.ldz = z.ldz * (z.f32 ? 4 : 2);
  a.V = (int)z.V; a.S = p.S; a.part = p.part;
  a.inv_t64 = 1.0 / z.temperature;
  a.inv_t = (float)a.inv_t64;
  a.c2 = (float)(a.inv_t64 / kLn2);
  a.stats = stats;
  a.target = target; a.logp = logp; a.entropy = entropy;
  a.n_top = n_top; a.top_ids = top_ids; a.top_logp = top_logp;
  carve(a, z.T, n_top, ws);
  if (n_top) return z.f32 ? run_fwd<true, kLogprobs, true>(a, z.T, stream) : run_fwd<false, kLogprobs, true>(a, z.T, stream);
  return z.f32 ? run_fwd<true, kLogprobs, false>(a, z.T, stream) : run_fwd<false, kLogprobs, false>(a, z.T, stream);
}

hipError_t launch_distill_fwd(const Logits& z, const TopLogits& t, const float* teacher_lse, float* loss,
                              float* stats, void* ws, hipStream_t stream) {
  const Parts p = fwd_parts(z.T, z.V);
  RowsFwd a{};
  a.Z = reinterpret_cast<const char*>(z.Z);
  a.ldz = z.ldz * (z.f32 ? 4 : 2);
  a.V = (int)z.V; a.S = p.S; a.part = p.part;
  a.inv_t64 = 1.0 / z.temperature;
  a.inv_t = (float)a.inv_t64;
  a.c2 = (float)(a.inv_t64 / kLn2);
  a.stats = stats;
  a.ids = t.ids; a.values = t.values; a.values_f32 = t.f32; a.k = t.k;
  a.teacher_lse = teacher_lse; a.loss = loss;
  carve(a, z.T, 0, ws);
  if (teacher_lse)
    return z.f32 ? run_fwd<true, kDistillRest, false>(a, z.T, stream) : run_fwd<false, kDistillRest, false>(a, z.T, stream);
  return z.f32 ? run_fwd<true, kDistill, false>(a, z.T, stream) : run_fwd<false, kDistill, false>(a, z.T, stream);
}

static RowsBwd bwd_args(const Logits& z, const float* stats, void* dZ, int64_t lddz) {
  const Parts p = bwd_parts(z.T, z.V);
  RowsBwd a{};
  a.Z = reinterpret_cast<const char*>(z.Z);
  a.ldz = z.ldz * (z.f32 ? 4 : 2);
  a.dZ = reinterpret_cast<char*>(dZ);
  a.lddz = lddz * (z.f32 ? 4 : 2);
  a.V = (int)z.V; a.S = p.S; a.part = p.part;
  a.inv_t = (float)(1.0 / z.temperature);
  a.c2 = (float)(1.0 / (z.temperature * kLn2));
  a.stats = stats;
  return a;
}

hipError_t launch_logprobs_bwd(const Logits& z, const int64_t* target, const float* stats, const float* g_logp,
                               const float* g_entropy, void* dZ, int64_t lddz, hipStream_t stream) {
  RowsBwd a = bwd_args(z, stats, dZ, lddz);
  a.target = target; a.g_logp = g_logp; a.g_entropy = g_entropy;
  const dim3 grid((unsigned)(z.T * a.S));
  if (z.f32)
    logprobs_bwd_kernel<true><<<grid, dim3(kThreads), 0, stream>>>(a);
  else
    logprobs_bwd_kernel<false><<<grid, dim3(kThreads), 0, stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_distill_bwd(const Logits& z, const TopLogits& t, const float* stats, const float* g, void* dZ,
                              int64_t lddz, hipStream_t stream) {
  RowsBwd a = bwd_args(z, stats, dZ, lddz);
  a.ids = t.ids; a.values = t.values; a.values_f32 = t.f32; a.k = t.k; a.g = g;
  const dim3 grid((unsigned)(z.T * a.S));
  if (z.f32)
    distill_bwd_kernel<true><<<grid, dim3(kThreads), 0, stream>>>(a);
  else
    distill_bwd_kernel<false><<<grid, dim3(kThreads), 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace qlora
