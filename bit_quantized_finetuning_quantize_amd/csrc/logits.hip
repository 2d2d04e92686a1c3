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
#include <type_traits>

namespace qlora {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kUnit = 8192;          // entries of a step of a workgroup; parts of a row are multiples of it
constexpr int kMaxUnits = 16;        // ... and at most this many of them
constexpr int kMaxParts = 32;
constexpr int64_t kMaxGrid = ((int64_t)1 << 32) / kThreads - 1;
constexpr int kMaxTop = 64;
constexpr int kMaxItems = 2048;
constexpr int kMaxCand = kMaxParts * kMaxTop;
constexpr float kInf = __builtin_huge_valf();
// 2^y is 0 below this, where 2^y y would be NaN for -inf: a bound no lower than
// needed, since a gradient's factor times it must stay finite as well.
constexpr float kLow = -1000.0f;
constexpr double kLn2 = 0.693147180559945309417;

// A row is cut into vectors of 16 bytes where its addresses are multiples of 16:
// `shift` elements of the first vector lie before the row, and a position is an
// element's index plus shift. (Vectors at any element are allowed, and cost
// the same at multiples of 4 bytes; at odd bf16 elements each lane's 16 bytes
// take a pass of their own: 1024 rows of 100001 53 us forward and 106
// backward, of 100000 42 and 92.) Where a gradient's rows start at another
// offset than the logits', its stores are the ones not aligned.
typedef u32x4 u32x4_row __attribute__((aligned(2)));

template <bool kF32>
struct Elem {
  static constexpr int kE = kF32 ? 4 : 8;                       // elements of a vector
  static constexpr int kVecs = kUnit / kThreads / kE;           // vectors a thread loads at once
  static constexpr int kBytes = kF32 ? 4 : 2;
};

// kPast: past the caches, for logits that outgrow the last-level one (256 MiB)
// together with what is written: us without and with, forward 4096 x 32768 52
// and 46, 2048 x 131072 95 and 86, backward 98 and 92, 186 and 181; forward and
// backward of 1024 x 32768, which fits, 39 and 41.
constexpr int64_t kPastBytes = (int64_t)128 << 20;

// Positions [lo, n) of a part hold elements of the row; of vector v those
// outside are -inf.
template <bool kF32>
__device__ __forceinline__ u32x4 load_vec(const char* part, int v, int lo, int n) {
  constexpr int kE = Elem<kF32>::kE;
  const int from = lo - v * kE, to = n - v * kE;
  if (from <= 0 && to >= kE) return *reinterpret_cast<const u32x4_row*>(part + (int64_t)v * 16);
  const uint32_t none = kF32 ? 0xff800000u : 0xff80ff80u;
  u32x4 r = {none, none, none, none};
  if constexpr (kF32) {
    const uint32_t* e = reinterpret_cast<const uint32_t*>(part + (int64_t)v * 16);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i >= from && i < to) r[i] = e[i];
  } else {
    const uint16_t* e = reinterpret_cast<const uint16_t*>(part + (int64_t)v * 16);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i >= from && i < to) {
        const uint32_t keep = (i & 1) ? 0x0000ffffu : 0xffff0000u;
        r[i >> 1] = (r[i >> 1] & keep) | ((uint32_t)e[i] << (16 * (i & 1)));
      }
  }
  return r;
}
template <bool kF32, bool kPast>
__device__ __forceinline__ void store_vec(char* part, int v, int lo, int n, u32x4 r) {
  constexpr int kE = Elem<kF32>::kE;
  const int from = lo - v * kE, to = n - v * kE;
  if (from <= 0 && to >= kE) {
    u32x4_row* to = reinterpret_cast<u32x4_row*>(part + (int64_t)v * 16);
    if constexpr (kPast) __builtin_nontemporal_store(r, to);
    else *to = r;
    return;
  }
  if constexpr (kF32) {
    uint32_t* e = reinterpret_cast<uint32_t*>(part + (int64_t)v * 16);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i >= from && i < to) e[i] = r[i];
  } else {
    uint16_t* e = reinterpret_cast<uint16_t*>(part + (int64_t)v * 16);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i >= from && i < to) e[i] = (uint16_t)(r[i >> 1] >> (16 * (i & 1)));
  }
}
// A thread's vectors of a step, the first of them v0: without a branch to a load
// where the whole step lies in the row.
template <bool kF32, bool kPast>
__device__ __forceinline__ void load_step(u32x4 (&r)[Elem<kF32>::kVecs], const char* part, int c, int v0, int lo, int n) {
  constexpr int kVecs = Elem<kF32>::kVecs;
  if (c * kUnit >= lo && (c + 1) * kUnit <= n) {  // uniform
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      const u32x4_row* from = reinterpret_cast<const u32x4_row*>(part + (int64_t)(v0 + u * kThreads) * 16);
      if constexpr (kPast) r[u] = __builtin_nontemporal_load(from);
      else r[u] = *from;
    }
  } else {
#pragma unroll
    for (int u = 0; u < kVecs; ++u) r[u] = load_vec<kF32>(part, v0 + u * kThreads, lo, n);
  }
}

// A workgroup's part of a row: positions [first, first + n), of which the first lo
// hold nothing.
struct Part {
  int64_t row;
  int shift, first, lo, n;
};
template <bool kF32>
__device__ __forceinline__ Part part_of(const char* Z, int64_t ldz, int S, int part, int V) {
  Part p;
  const uint32_t row = blockIdx.x / (uint32_t)S;
  p.row = row;
  p.shift = (int)((uintptr_t)(Z + row * ldz) & 15) / Elem<kF32>::kBytes;
  p.first = (int)(blockIdx.x - row * (uint32_t)S) * part;
  p.lo = p.first == 0 ? p.shift : 0;
  p.n = max(0, min(part, V + p.shift - p.first));
  return p;
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
// Reductions over a wave whose lanes are all active, the same in every lane: by
// rows of 16 lanes, then of the rows; the last lane holds the result.
template <int kCtrl, int kRows, typename T>
__device__ __forceinline__ T dpp(T v, T none) {
  if constexpr (sizeof(T) == 4) {
    return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, none), __builtin_bit_cast(int, v),
                                                             kCtrl, kRows, 0xf, false));
  } else {
    const uint64_t w = __builtin_bit_cast(uint64_t, v), n = __builtin_bit_cast(uint64_t, none);
    const uint32_t lo = __builtin_amdgcn_update_dpp((int)(uint32_t)n, (int)(uint32_t)w, kCtrl, kRows, 0xf, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp((int)(n >> 32), (int)(w >> 32), kCtrl, kRows, 0xf, false);
    return __builtin_bit_cast(T, ((uint64_t)hi << 32) | lo);
  }
}
template <typename T, typename F>
__device__ __forceinline__ T wave_reduce(T v, T none, F f) {
  v = f(v, dpp<0x111, 0xf>(v, none));  // row_shr 1, 2, 4, 8
  v = f(v, dpp<0x112, 0xf>(v, none));
  v = f(v, dpp<0x114, 0xf>(v, none));
  v = f(v, dpp<0x118, 0xf>(v, none));
  v = f(v, dpp<0x142, 0xa>(v, none));  // row_bcast 15, 31
  v = f(v, dpp<0x143, 0xc>(v, none));
  if constexpr (sizeof(T) == 4) {
    return __builtin_bit_cast(T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
  } else {
    const uint64_t w = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)w, 63), hi = __builtin_amdgcn_readlane((int)(w >> 32), 63);
    return __builtin_bit_cast(T, ((uint64_t)hi << 32) | lo);
  }
}
__device__ __forceinline__ double lane_of(double v, int lane) {
  const uint64_t w = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)w, lane), hi = __builtin_amdgcn_readlane((int)(w >> 32), lane);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ float wave_max(float v) {
  return wave_reduce(v, -kInf, [](float a, float b) { return fmaxf(a, b); });
}
template <typename T>
__device__ __forceinline__ T wave_sum(T v) {
  return wave_reduce(v, T(0), [](T a, T b) { return a + b; });
}
__device__ __forceinline__ Soft wave_join(const Soft& a, float c2) {
  Soft r = rescaled(a, wave_max(a.m), c2);
  r.s = wave_sum(r.s);
  r.u = wave_sum(r.u);
  return r;
}

// The mass of a part of a distillation's row, sum s 2^((z - m) c), s in 64 bits: the
// loss is a difference of values near each other.
struct Mass {
  float m;
  double s;
};
constexpr Mass kNoMass{-kInf, 0.0};
// The lanes' masses as one, in every lane.
__device__ __forceinline__ Mass wave_join(const Mass& a, double c) {
  const float m = wave_max(a.m);
  // 2^d by the hardware's exp2 of d's fraction, 1 where d is 0
  const double d = fmax(((double)a.m - base_of(m)) * c, -1100.0), n = rint(d);
  return Mass{m, wave_sum(a.s * ldexp((double)exp2_((float)(d - n)), (int)n))};
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

__device__ __forceinline__ uint64_t larger(uint64_t a, uint64_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint64_t wave_largest(uint64_t v) { return wave_reduce(v, (uint64_t)0, larger); }
// Of the lanes' pairs of a key and a step, the r-th in the order larger keys, lower
// steps first (with multiplicity; r at most the lanes).
template <bool kF32>
__device__ __forceinline__ void wave_rth(uint32_t& key, uint32_t& step, int r) {
  uint32_t v = key, top;
  const uint32_t mine = step;
  if (r <= 2) {  // the largest, and perhaps the next
    for (;;) {
      top = wave_reduce(v, 0u, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
      const int c = __builtin_popcountll(__ballot(v == top));
      if (r <= c) break;
      r -= c;
      if (v == top) v = 0;
    }
  } else {
    // bit by bit, the lanes whose key may be it (the keys of bf16 logits differ in
    // their upper 16 bits if at all)
    uint64_t left = ~0ull;
#pragma unroll 1
    for (int bit = 31; bit >= (kF32 ? 0 : 16); --bit) {
      const uint64_t ones = __ballot((v >> bit) & 1) & left;
      const int c = __builtin_popcountll(ones);
      left = c >= r ? ones : left & ~ones;
      r -= c >= r ? 0 : c;
    }
    top = __builtin_amdgcn_readlane((int)v, __builtin_ctzll(left));
  }
  uint32_t s = 0;
#pragma unroll 1
  while (__builtin_popcountll(__ballot(v == top && mine <= s)) < r) ++s;
  key = top;
  step = s;
}

// ---------------------------------------------------------------------------
// 1 / d, exp x and log of a positive s in 64 bits, to 3e-13 of the value: two of Newton's
// steps from the hardware's inverse; Taylor's series of x less its nearest multiple of
// ln 2 (at most 0.35) up to the tenth power; 2 artanh((m - 1) / (m + 1)), s = 2^e m, m
// in [sqrt(1/2), sqrt 2), up to the 15th. A dozen or two operations one after the
// other, for a row's end waits for them (the library's took 1.3 us more of 4096 x
// 1000 with 32 entries, 0.3 of 7 x 50001).
__device__ __forceinline__ double inverse(double d) {
  double r = __builtin_amdgcn_rcp(d);
  r = __builtin_fma(__builtin_fma(-d, r, 1.0), r, r);
  return __builtin_fma(__builtin_fma(-d, r, 1.0), r, r);
}
__device__ __forceinline__ double exp_(double x) {
  x = x < -800.0 ? -800.0 : x > 800.0 ? 800.0 : x;  // 0 and infinity; keeps a NaN
  const double n = rint(x * 1.44269504088896340736);
  constexpr double kHi = 2977044471.0 / 4294967296.0, kLo = 1.9082149292705877e-10;  // ln 2 to 32 bits, and the rest
  const double r = __builtin_fma(n, -kLo, __builtin_fma(n, -kHi, x));
  double p = 1.0 / 3628800;
  constexpr double kInverse[10] = {1.0,       1.0,       1.0 / 2,    1.0 / 6,     1.0 / 24,
                                   1.0 / 120, 1.0 / 720, 1.0 / 5040, 1.0 / 40320, 1.0 / 362880};  // of i!
#pragma unroll
  for (int i = 9; i >= 0; --i) p = __builtin_fma(p, r, kInverse[i]);
  return ldexp(p, (int)n);
}
__device__ __forceinline__ double log_(double s) {
  double m = __builtin_amdgcn_frexp_mant(s);
  int e = __builtin_amdgcn_frexp_exp(s);
  const bool low = m < 0.70710678118654752440;
  m = low ? 2.0 * m : m;
  e -= low;
  const double f = (m - 1.0) * inverse(m + 1.0), g = f * f;
  double p = 2.0 / 15;
#pragma unroll
  for (int i = 13; i >= 3; i -= 2) p = __builtin_fma(p, g, 2.0 / i);
  return __builtin_fma((double)e, kLn2, __builtin_fma(p * g, f, 2.0 * f));
}

// A teacher's list in LDS: ids (-1: no entry), the teacher's and the student's logits,
// kThreads each.
constexpr int kPer = kThreads / 64;  // entries to a lane
__device__ __forceinline__ float list_logit(const int* list, int which, int e) {
  return __builtin_bit_cast(float, list[which * kThreads + e]);
}
// The student's mass on the list over its largest logit zm where an id is on it twice:
// each token once.
__device__ __noinline__ double list_mass(const int* list, int k, int lane, float zm, double inv_t) {
  double on = 0.0;
#pragma unroll 1
  for (int i = lane; i < k; i += 64) {
    bool once = list[i] >= 0;
    for (int e = 0; e < i && once; ++e) once = list[e] != list[i];
    if (once) on += exp_(((double)list_logit(list, 2, i) - base_of(zm)) * inv_t);
  }
  return wave_sum(on);
}
// What a row's end takes of its list, by one wave, in 64 bits (a loss is a sum of
// values that nearly cancel): the largest logits tm and zm (tm 0 for none), tl, the
// student's mass `on` over zm if no id is on it twice, e = sum e_i with e_i = exp((t_i -
// tm) / t), d = sum e_i ((t_i - tm) - (z_i - zm)) / t, scale and tl (q_i = e_i scale, log
// scale = -tl), w = sum q_i, and with kRest q_r and its logarithm.
struct ListSums {
  float tm, zm;
  double on, e, d, scale, tl, w, qr, ln_qr;
};
template <bool kRest>
__device__ __forceinline__ ListSums list_sums(const int* list, int k, int lane, double inv_t, const float* teacher_lse,
                                              int64_t row) {
  float tm = -kInf, zm = -kInf;
#pragma unroll 1
  for (int i = lane; i < k; i += 64) {
    tm = fmaxf(tm, list_logit(list, 1, i));
    zm = fmaxf(zm, list_logit(list, 2, i));
  }
  tm = base_of(wave_max(tm));
  zm = wave_max(zm);
  const double base = base_of(zm);
  double on = 0.0, e = 0.0, d = 0.0;
#pragma unroll 1
  for (int i = lane; i < k; i += 64) {
    // no entry and a teacher's logit of -inf have e_i = 0
    const double x = ((double)list_logit(list, 1, i) - tm) * inv_t, u = ((double)list_logit(list, 2, i) - base) * inv_t;
    const double y = exp_(x);
    on += exp_(u);
    e += y;
    d += y <= 0.0 ? 0.0 : y * (x - u);
  }
  on = wave_sum(on);
  e = wave_sum(e);
  d = wave_sum(d);
  ListSums s{tm, zm, on, e, d, 0.0, 0.0, 0.0, 0.0, 0.0};
  if (kRest) s.tl = (double)teacher_lse[row] - (double)tm * inv_t;
  else if (e > 0.0) s.tl = log_(e);
  s.scale = kRest ? exp_(-s.tl) : inverse(e);
  s.w = e == 0.0 ? 0.0 : e * s.scale;
  if (kRest) {
    s.qr = 1.0 - s.w;
    if (s.qr < 0.0) s.qr = 0.0;
    s.ln_qr = log_(s.qr);
  }
  return s;
}

// ---------------------------------------------------------------------------
// Forward.

enum { kLogprobs, kDistill, kDistillRest };
// a distillation has a wave more, for its list
constexpr int fwd_threads(int op) { return kThreads + (op == kLogprobs ? 0 : 64); }

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
  double inv_t64, c64;
  float* loss;
  // where rows are split
  uint64_t* flags;  // [T][S]
  float* sums;      // [T][S][4]: m, s, u, or m, s in 64 bits, whether an id is twice on the list
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

// The `need` largest entries of a part, among the returned number of candidates in
// t.cand (all different). bins [steps][kThreads]: key of the maximum of each
// thread's vectors of each step; best: the thread's largest bin as (key, first
// position of the step), an upper bound in that coarser order for all its
// entries, and attained by one of them unless they are all NaN. The r-th largest
// of them in each of w full waves, r = need / w rounded up, has r entries at or
// above it in that wave, so the smallest of the waves' has `need`: only the
// bins that reach it are read again (from the L2).
// Equal entries at t0 beyond what t.cand holds take a pass to each entry, and so
// do parts with fewer numbers than `need`. Masked logits are such entries where a
// part has fewer others than the bound asks for: one row of 131072 with 200 of its
// tokens allowed, 1, 5, 20 and 64 entries, 25, 54, 165 and 486 us from a graph,
// against 9.6, 10.2, 11.8 and 15.7 with 20000 allowed.
// The code is kept short: a few rows run all of it once, and fetching it costs
// as much as running it (one row of 131072 with 20 entries 12.4 us from a graph,
// 14.1 with the steps below unrolled and entries taken from registers; 6.0
// without entries, where a launch alone takes 4).
template <bool kF32>
__device__ __forceinline__ int select_top(const char* part, int lo, int n, int first, int steps,
                                          const uint32_t* bins, uint64_t best, int need, TopLds& t) {
  constexpr int kE = Elem<kF32>::kE, kVecs = Elem<kF32>::kVecs;
  const int tid = threadIdx.x, wave = tid >> 6;
  // waves whose lanes all hold an entry; a part that fills none has as many lanes as vectors
  const int full = n / kE >= 64 ? min(kWaves, n / kE / 64) : (n + kE - 1) / kE >= need;
  if (full) {
    uint32_t key = (uint32_t)(best >> 32), step = best ? (idx_of(best) - (uint32_t)first) / kUnit : 0;
    wave_rth<kF32>(key, step, (need + full - 1) / full);
    if ((tid & 63) == 0) t.wave[wave] = pair_of(key, (uint32_t)first + step * kUnit);
  }
  if (tid == 0) t.n_items = t.n_cand = 0;
  __syncthreads();
  uint64_t t0 = full ? ~0ull : 0;
#pragma unroll 1
  for (int w = 0; w < full; ++w) t0 = t.wave[w] < t0 ? t.wave[w] : t0;
  auto coarse = [&](uint32_t key, int b) { return pair_of(key, (uint32_t)(first + b * kUnit)); };
#pragma unroll 1
  for (int b = 0; b < steps; ++b) {
    const uint32_t key = bins[b * kThreads + tid];
    if (key && coarse(key, b) >= t0) {
      const int i = atomicAdd(&t.n_items, 1);
      if (i < kMaxItems) t.items[i] = (uint16_t)(b * kThreads + tid);
    }
  }
  __syncthreads();
  // Pass -1 collects the numbers at or above t0 of the bins listed. Where those are
  // too many (equal entries), each further pass takes the next entry in order of
  // the bins listed; where the part has fewer numbers than `need`, of all its
  // bins, since the NaNs that come next lie in bins not listed too.
  bool all = t.n_items > kMaxItems;
  uint64_t prev = ~0ull;
#pragma unroll 1
  for (int pass = all ? 0 : -1; pass < need; ++pass) {
    const int bins_here = all ? steps * kThreads : t.n_items;
    const float zt = all ? -kInf : of_key((uint32_t)(t0 >> 32));  // NaN for 0: everything
    uint64_t top = 0;
#pragma unroll 1
    for (int w = tid; w < bins_here * kVecs; w += kThreads) {
      const int it = all ? w / kVecs : t.items[w / kVecs], b = it / kThreads;
      const int v = (b * kVecs + w % kVecs) * kThreads + it % kThreads;
      if (v * kE >= n) continue;
      const u32x4 x = load_vec<kF32>(part, v, lo, n);
      uint32_t hits = 0;
#pragma unroll
      for (int i = 0; i < kE; ++i) hits |= !(elem<kF32>(x, i) < zt) ? 1u << i : 0u;
#pragma unroll 1
      while (hits) {
        const int at = v * kE + __builtin_ctz(hits);
        hits &= hits - 1;
        if (at < lo || at >= n) continue;
        const uint32_t key = key_of(load_elem<kF32>(part, at));
        const uint64_t p = pair_of(key, (uint32_t)(first + at));
        if (pass >= 0) {
          if (p < prev && p > top) top = p;
        } else if (key && coarse(key, b) >= t0) {
          const int c = atomicAdd(&t.n_cand, 1);
          if (c < kMaxCand) t.cand[c] = p;
        }
      }
    }
    if (pass >= 0) {
      top = wave_largest(top);
      if ((tid & 63) == 0) t.wave[wave] = top;
    }
    __syncthreads();
    if (pass < 0) {
      const int count = t.n_cand;
      if (count >= need && count <= kMaxCand) return count;
      all = count < need;
    } else {
#pragma unroll 1
      for (int w = 0; w < kWaves; ++w) top = larger(top, t.wave[w]);
      if (tid == 0) t.cand[pass] = top;
      prev = top;
      __syncthreads();
    }
  }
  return need;
}

// One (row, part) per workgroup. Rows that do not fit 16 steps (131072 positions)
// are split, and where there are fewer than 1024 rows also shorter ones, into about
// 1024 workgroups (with 2048 and 4096: 600 x 50000 with 20 entries 26.5 us -> 29.5
// and 36, 1030 x 32000 17.5 -> 17.9 and 18.9, 449 x 30637 13.3 -> 11.8).
// Large calls are bounded by memory: 4096 x 32768 in bf16 48 us in a graph, 5.6
// TB/s, where reads alone reach 6.2; the operations, nine a logit, take 29 us
// of that. A row of 131072 takes 6.0 us, where a launch takes 4, and 9.4, 11.9
// and 16.0 with 1, 20 and 64 entries: the selection's latency.
//
// Where a row has several workgroups, each stores its statistics and then a
// flag holding the dispatch's tag, and looks at all the row's flags: stores and
// looks are performed in one memory, so the workgroup whose flag comes last
// sees them all, and goes on with the row (if two see them all, both write the
// same values). None waits for another. Whoever goes on sets the row's flags to
// 0; before a call they may hold anything.
//
// A distillation's loss is a difference of values near each other, so the tokens of
// the list, which hold most of the mass, are left out of the float32 sums and taken in
// 64 bits, and what the sums hold moves the loss by their error times |w p_r - q_r|
// only: of 1500 drawn calls the losses were off by 3e-8 at the median and 1.1e-6 at
// most, at 2e-4; with the list in the sums 2e-7 and 5e-5, at 3e-3. A wave of its own makes the list's mask while the row's first loads are in
// flight, and its sums beside the row's; without it (the list with the row's waves)
// 1024 x 18000 with 64 entries and the rest 15.8 us and 300 x 100003 19.8, with it
// 14.2 and 18.3; 4096 x 1000 with 32 20.7 and 21.0.
// kTop: with the largest entries. kPast: loads past the caches.
template <bool kF32, int kOp, bool kTop, bool kPast>
__global__ void __launch_bounds__(fwd_threads(kOp)) rows_fwd_kernel(RowsFwd a) {
  constexpr int kE = Elem<kF32>::kE, kVecs = Elem<kF32>::kVecs;
  extern __shared__ __attribute__((aligned(16))) uint8_t dyn[];
  __shared__ Soft s_soft[kWaves];
  __shared__ Mass s_mass[kWaves];
  __shared__ ListSums s_sums;
  __shared__ int s_last, s_twice, s_list[kOp == kLogprobs ? 1 : 3 * kThreads];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const Part in = part_of<kF32>(a.Z, a.ldz, a.S, a.part, a.V);
  const int64_t row = in.row;
  const int shift = in.shift, first = in.first, lo = in.lo, n = in.n, split = first / a.part;
  const char* zrow = a.Z + row * a.ldz;
  const char* part = zrow + (int64_t)(first - shift) * Elem<kF32>::kBytes;
  const int steps = (n + kUnit - 1) / kUnit;
  const float c2 = a.c2;

  float zy = 0.0f;  // the target's logit
  bool counts = false;
  if (kOp == kLogprobs && a.logp) {
    const int64_t y = a.target[row];
    counts = y >= 0 && y < a.V;
    if (counts) zy = load_elem<kF32>(zrow, y);
  }
  TopLds& top = *reinterpret_cast<TopLds*>(dyn);
  uint32_t* bins = reinterpret_cast<uint32_t*>(dyn + sizeof(TopLds));
  uint64_t* s_lists = reinterpret_cast<uint64_t*>(bins);  // after the part's own selection: [S][n_top]
  uint32_t* mask = reinterpret_cast<uint32_t*>(dyn);  // bit i: position first + i is on the list
  u32x4 r[kVecs];
  if constexpr (kOp != kLogprobs) {
    if (wave == kWaves) {
      // the list's wave, up to four entries to a lane
      int id[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        id[i] = -1;
        if (i * 64 + lane < a.k) {
          const int64_t j = a.ids[row * a.k + i * 64 + lane];
          if (j >= 0 && j < a.V) id[i] = (int)j;
        }
      }
      // LDS accesses of one wave complete in order
      const int words = (n + 127) / 128 * 4;
      for (int i = lane * 4; i < words; i += 256) *reinterpret_cast<u32x4*>(mask + i) = u32x4{0, 0, 0, 0};
      asm volatile("" ::: "memory");
      bool twice = false;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int at = id[i] + shift - first;
        const uint32_t bit = 1u << (at & 31);
        if (id[i] >= 0 && at >= lo && at < n) twice |= (atomicOr(mask + (at >> 5), bit) & bit) != 0;
      }
      twice = __any(twice);
      if (lane == 0) s_twice = twice;
      __syncthreads();
      float t[kPer], z[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        t[i] = z[i] = -kInf;
        const int64_t entry = row * a.k + i * 64 + lane;
        if (id[i] < 0) continue;
        t[i] = a.values_f32 ? load_elem<true>(a.values, entry) : load_elem<false>(a.values, entry);
        z[i] = load_elem<kF32>(zrow, id[i]);
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        s_list[i * 64 + lane] = id[i];
        s_list[kThreads + i * 64 + lane] = __builtin_bit_cast(int, t[i]);
        s_list[2 * kThreads + i * 64 + lane] = __builtin_bit_cast(int, z[i]);
      }
      asm volatile("" ::: "memory");
      const ListSums sums = list_sums<kOp == kDistillRest>(s_list, a.k, lane, a.inv_t64, a.teacher_lse, row);
      if (lane == 0) s_sums = sums;
      __syncthreads();
      return;
    }
    if (steps > 0) load_step<kF32, kPast>(r, part, 0, tid, lo, n);  // in flight while the mask is made
    __syncthreads();
  }

  Soft acc = kNone;  // in a distillation without the listed entries
  uint64_t best = 0;
  for (int c = 0; c < steps; ++c) {
    float z[kVecs * kE];
    const int v0 = c * kVecs * kThreads + tid;
    if (kOp == kLogprobs || c > 0) load_step<kF32, kPast>(r, part, c, v0, lo, n);
#pragma unroll
    for (int u = 0; u < kVecs; ++u)
#pragma unroll
      for (int i = 0; i < kE; ++i) z[u * kE + i] = elem<kF32>(r[u], i);
    if constexpr (kOp != kLogprobs) {
      uint32_t b[kVecs];  // all read before the branches
#pragma unroll
      for (int u = 0; u < kVecs; ++u) {
        const int v = v0 + u * kThreads < (n + kE - 1) / kE ? v0 + u * kThreads : 0;
        const uint8_t byte = reinterpret_cast<const uint8_t*>(mask)[kF32 ? v >> 1 : v];
        b[u] = kF32 ? (byte >> (4 * (v & 1))) & 15u : byte;
      }
#pragma unroll
      for (int u = 0; u < kVecs; ++u)
        if (b[u]) {
#pragma unroll
          for (int i = 0; i < kE; ++i) z[u * kE + i] = (b[u] >> i) & 1 ? -kInf : z[u * kE + i];
        }
    }
    float m = z[0];
#pragma unroll
    for (int i = 1; i < kVecs * kE; ++i) m = fmaxf(m, z[i]);
    if constexpr (kTop) {
      const uint32_t key = v0 * kE < n ? key_of(m) : 0;
      bins[c * kThreads + tid] = key;
      if (key) best = larger(best, pair_of(key, (uint32_t)(first + c * kUnit)));
    }
    m = fmaxf(m, acc.m);
    const float base = base_of(m);
    float s[4] = {0, 0, 0, 0}, q[4] = {0, 0, 0, 0};
    auto sums = [&](auto y_of) {
#pragma unroll
      for (int i = 0; i < kVecs * kE; ++i) {
        const float y = y_of(z[i]);
        const float e = exp2_(y);
        s[i & 3] += e;
        if constexpr (kOp == kLogprobs) q[i & 3] = __builtin_fmaf(e, fmaxf(y, kLow), q[i & 3]);
      }
    };
    // z c2 - b, b = fl(m c2), is one operation to (z - m) c2's two, and off by what
    // b was rounded by: d for every entry, taken out of the sums below. Far from
    // zero (a row of the type's lowest values, say) d would not be small.
    const float b = base * c2;
    float d = 0.0f;
    if (__all(fabsf(b) < 1024.0f)) {
      d = __builtin_fmaf(base, c2, -b);
      sums([&](float v) { return __builtin_fmaf(v, c2, -b); });
    } else {
      sums([&](float v) { return (v - base) * c2; });
    }
    const float f = exp2_(-d), sc = (s[0] + s[1]) + (s[2] + s[3]), qc = (q[0] + q[1]) + (q[2] + q[3]);
    acc = rescaled(acc, m, c2);
    acc.s = __builtin_fmaf(sc, f, acc.s);
    acc.u = __builtin_fmaf(qc - sc * d, f, acc.u);
  }

  // the workgroup's statistics; one wave goes on with them, all where a selection
  // is to come
  Mass mass = kNoMass;
  if constexpr (kOp == kLogprobs) {
    acc = wave_join(acc, c2);
    if (lane == 0) s_soft[wave] = acc;
  } else {
    mass = wave_join(Mass{acc.m, acc.s}, a.c64);
    if (lane == 0) s_mass[wave] = mass;
  }
  __syncthreads();
  if (!kTop && wave) return;
  if constexpr (kOp == kLogprobs) {
    acc = s_soft[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) acc = joined(acc, s_soft[w], c2);
  } else {
    mass = wave_join(lane < kWaves ? s_mass[lane] : kNoMass, a.c64);
  }
  bool twice = kOp != kLogprobs && s_twice;  // an id is twice on the list

  int count = 0, need = kTop ? min(a.n_top, n - lo) : 0;
  if (kTop && need > 0) count = select_top<kF32>(part, lo, n, first, steps, bins, best, need, top);
  bool whole = a.S == 1;  // the row's statistics, and not a part's
#pragma unroll 1
  for (;;) {
    const bool empty = acc.m == -kInf && acc.s == 0.0f;
    float l = 0.0f;
    if (kOp == kLogprobs && whole) {
      // s holds the largest logit's 1, whatever it was rounded to
      const float s = acc.s < 1.0f ? 1.0f : acc.s;
      l = empty ? 0.0f : logf(s);
      if (tid == 0) {
        float H = empty ? 0.0f : l - (float)kLn2 * (acc.u / s);
        H = H < 0.0f ? 0.0f : H;
        if (a.entropy) a.entropy[row] = H;
        if (a.stats) {
          a.stats[row * 3] = acc.m;
          a.stats[row * 3 + 1] = l;
          a.stats[row * 3 + 2] = H;
        }
        if (a.logp) a.logp[row] = !counts ? 0.0f : empty ? -kInf : (zy - acc.m) * a.inv_t - l;
      }
    }
    if constexpr (kTop) {  // the candidates' ranks, and the first of them to their places
      __syncthreads();
#pragma unroll 1
      for (int i = tid; i < count; i += kThreads) {
        const uint64_t mine = top.cand[i];
        int rank = 0;
#pragma unroll 4
        for (int j = 0; j < count; ++j) rank += top.cand[j] > mine;
        if (rank >= need) continue;
        if (whole) {
          a.top_ids[row * a.n_top + rank] = (int64_t)idx_of(mine) - shift;
          a.top_logp[row * a.n_top + rank] = empty ? -kInf : (of_key((uint32_t)(mine >> 32)) - acc.m) * a.inv_t - l;
        } else {
          __hip_atomic_store(a.lists + (int64_t)blockIdx.x * a.n_top + rank, mine, __ATOMIC_RELAXED,
                             __HIP_MEMORY_SCOPE_AGENT);
        }
      }
    }
    if (whole) break;
    if (kTop && tid >= need && tid < a.n_top)
      __hip_atomic_store(a.lists + (int64_t)blockIdx.x * a.n_top + tid, (uint64_t)0, __ATOMIC_RELAXED,
                         __HIP_MEMORY_SCOPE_AGENT);
    if (tid == 0) {
      float* p = a.sums + (int64_t)blockIdx.x * 4;
      if constexpr (kOp == kLogprobs) {
        put_agent(p, acc.m);
        put_agent(p + 1, acc.s);
        put_agent(p + 2, acc.u);
      } else {
        const uint64_t s = __builtin_bit_cast(uint64_t, mass.s);
        put_agent(p, mass.m);
        put_agent(p + 1, __builtin_bit_cast(float, (uint32_t)s));
        put_agent(p + 2, __builtin_bit_cast(float, (uint32_t)(s >> 32)));
        put_agent(p + 3, twice ? 1.0f : 0.0f);
      }
    }
    // every store of the workgroup acknowledged before its flag
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    if constexpr (kTop) __syncthreads();
    bool last = true;
    if (wave == 0) {
      const uint64_t tag = call_tag();
      uint64_t* flags = a.flags + row * a.S;
      if (lane == 0) {
        const uint64_t was = __hip_atomic_exchange(flags + split, tag, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        asm volatile("" ::"v"((uint32_t)was));  // performed before the looks below
      }
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      const uint64_t zero = (uint64_t)(a.V >> 30);  // an addition that the compiler keeps
      last = lane >= a.S || __hip_atomic_fetch_add(flags + (lane < a.S ? lane : 0), zero, __ATOMIC_RELAXED,
                                                   __HIP_MEMORY_SCOPE_AGENT) == tag;
      last = __all(last);
      if (kTop && lane == 0) s_last = last;
    }
    if constexpr (kTop) {
      __syncthreads();
      last = s_last;
    }
    if (!last) return;
    // whoever looks later sees no full set and leaves, and no later call finds one
    // that it could take for its own
    if (wave == 0 && lane < a.S)
      __hip_atomic_store(a.flags + row * a.S + lane, (uint64_t)0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    acc = kNone;
    mass = kNoMass;
    float last_of = 0.0f;
    if (lane < a.S) {
      const float* p = a.sums + (row * a.S + lane) * 4;
      if constexpr (kOp == kLogprobs) {
        acc = Soft{get_agent(p), get_agent(p + 1), get_agent(p + 2)};
      } else {
        const uint32_t s0 = __builtin_bit_cast(uint32_t, get_agent(p + 1)), s1 = __builtin_bit_cast(uint32_t, get_agent(p + 2));
        mass = Mass{get_agent(p), __builtin_bit_cast(double, ((uint64_t)s1 << 32) | s0)};
        last_of = get_agent(p + 3);
      }
    }
    if constexpr (kTop) {
      // the parts' lists are sorted, and all but the last are whole: each has
      // r = n_top / (S - 1) rounded up entries at or above its r-th
      const uint64_t* lists = a.lists + row * a.S * a.n_top;
      need = a.n_top;
      const int total = a.S * need, r = (need + a.S - 2) / (a.S - 1);
#pragma unroll 1
      for (int i = tid; i < total; i += kThreads)
        s_lists[i] = __hip_atomic_load(lists + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      if (tid == 0) top.n_cand = 0;
      __syncthreads();
      uint64_t t0 = ~0ull;
#pragma unroll 4
      for (int w = 0; w < a.S - 1; ++w) t0 = s_lists[w * need + r - 1] < t0 ? s_lists[w * need + r - 1] : t0;
#pragma unroll 1
      for (int i = tid; i < total; i += kThreads) {
        const uint64_t p = s_lists[i];
        if (p && p >= t0) top.cand[atomicAdd(&top.n_cand, 1)] = p;
      }
      __syncthreads();
      count = top.n_cand;
    }
    if constexpr (kOp == kLogprobs) {
      acc = wave_join(acc, c2);
    } else {
      twice = __any(last_of != 0.0f);
      mass = wave_join(mass, a.c64);
    }
    whole = true;
  }

  if constexpr (kOp != kLogprobs) {
    const ListSums at = s_sums;
    const double on = twice ? list_mass(s_list, a.k, lane, at.zm, a.inv_t64) : at.on;  // uniform
    // The student's mass over m, the larger maximum: of the rest and of the list. Two
    // lanes take the two exponentials, and the two logarithms.
    const float m = fmaxf(mass.m, at.zm);
    const bool empty = m == -kInf && mass.s == 0.0 && on == 0.0, odd = lane & 1;
    const double base = base_of(m);
    const double f = exp_(((double)(odd ? at.zm : mass.m) - base) * a.inv_t64);
    const double r = mass.s * lane_of(f, 0), s = r + on * lane_of(f, 1);
    const double ln = log_(odd ? mass.s : s);
    double l = lane_of(ln, 0), loss = 0.0, w = at.w;
    if (empty || l < 0.0) l = 0.0;  // below 0 by rounding of the sums alone
    const double far = empty ? (double)kInf : l - ((double)base_of(at.zm) - base) * a.inv_t64;
    if (!(w <= 0.0)) loss = at.scale * (at.d + at.e * (far - at.tl));
    double off = w;
    if (kOp == kDistillRest && mass.s != 0.0 && !(at.qr <= 0.0)) {
      loss += at.qr * (at.ln_qr - (lane_of(ln, 1) + ((double)mass.m - base) * a.inv_t64 - l));
      w += at.qr;
      off = w - at.qr * s / r;
    }
    if (lane == 0) {
      constexpr double kTop32 = 3.402823466e38;
      a.loss[row] = (float)loss;
      if (a.stats) {
        float* p = a.stats + row * 6;
        p[0] = m;
        p[1] = (float)l;
        p[2] = (float)w;
        p[3] = (float)(off < -kTop32 ? -kTop32 : off);
        p[4] = at.tm;
        p[5] = (float)at.tl;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Backward: one pass, dz in z's place if the caller wants it, and bounded by
// memory, at or above the rate of a copy (5.2 TB/s for 1 GiB): in bf16 1023 rows
// of 100003, all but one in eight of them unaligned, 74 us in a graph, 5.5 TB/s;
// a distillation's 2048 x 131072 with 64 entries 180 us, 6.0 TB/s.

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

// f(v, value) over the vectors of a part, mostly one step: the new value of each
// element.
template <bool kF32, bool kPast, typename F>
__device__ __forceinline__ void map_part(const char* z, char* dz, int lo, int n, F f) {
  constexpr int kE = Elem<kF32>::kE, kVecs = Elem<kF32>::kVecs;
  const int tid = (int)threadIdx.x;
  for (int c = 0; c * kUnit < n; ++c) {
    const int v0 = c * kVecs * kThreads + tid;
    u32x4 r[kVecs];
    load_step<kF32, kPast>(r, z, c, v0, lo, n);
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      const int v = v0 + u * kThreads;
      if (v * kE >= n) continue;
      float x[kE];
#pragma unroll
      for (int i = 0; i < kE; ++i) x[i] = elem<kF32>(r[u], i);
      f(v, x);
      store_vec<kF32, kPast>(dz, v, lo, n, pack_vec<kF32>(x));
    }
  }
}
template <bool kF32>
__device__ __forceinline__ void zero_part(char* dz, int lo, int n) {
  for (int v = threadIdx.x; v * Elem<kF32>::kE < n; v += kThreads)
    store_vec<kF32, false>(dz, v, lo, n, u32x4{0, 0, 0, 0});
}

// dz_j = (g ([j = target] - p_j) - h p_j (log p_j + H)) / t.
template <bool kF32, bool kPast>
__global__ void __launch_bounds__(kThreads) logprobs_bwd_kernel(RowsBwd a) {
  constexpr int kE = Elem<kF32>::kE;
  const Part in = part_of<kF32>(a.Z, a.ldz, a.S, a.part, a.V);
  const int64_t row = in.row;
  const int shift = in.shift, first = in.first, lo = in.lo, n = in.n;
  const char* z = a.Z + row * a.ldz + (int64_t)(first - shift) * Elem<kF32>::kBytes;
  char* dz = a.dZ + row * a.lddz + (int64_t)(first - shift) * Elem<kF32>::kBytes;
  const float m = a.stats[row * 3], l = a.stats[row * 3 + 1], H = a.stats[row * 3 + 2];
  const int64_t y = a.target ? a.target[row] : -1;
  const float g = a.g_logp && y >= 0 && y < a.V ? a.g_logp[row] : 0.0f;
  const float h = a.g_entropy ? a.g_entropy[row] : 0.0f;
  if ((m == -kInf && l == 0.0f) || (g == 0.0f && h == 0.0f)) {
    zero_part<kF32>(dz, lo, n);
    return;
  }
  const float c2 = a.c2, l2 = l * 1.44269504088896340736f;
  const float ca = -(g + h * H) * a.inv_t, cb = -h * (float)kLn2 * a.inv_t, one = g * a.inv_t;
  const int hot = (int)(y + shift - first);  // may lie outside the part
  map_part<kF32, kPast>(z, dz, lo, n, [&](int v, float* x) {
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
template <bool kF32, bool kPast>
__global__ void __launch_bounds__(kThreads) distill_bwd_kernel(RowsBwd a) {
  __shared__ __attribute__((aligned(16))) int s_id[kThreads];
  __shared__ float s_q[kThreads];
  const int tid = threadIdx.x;
  const Part in = part_of<kF32>(a.Z, a.ldz, a.S, a.part, a.V);
  const int64_t row = in.row;
  const int shift = in.shift, first = in.first, lo = in.lo, n = in.n;
  const char* z = a.Z + row * a.ldz + (int64_t)(first - shift) * Elem<kF32>::kBytes;
  char* dz = a.dZ + row * a.lddz + (int64_t)(first - shift) * Elem<kF32>::kBytes;
  const float* s = a.stats + row * 6;
  const float m = s[0], l2 = s[1] * 1.44269504088896340736f, w = s[2], off = s[3];
  const float gt = a.g[row] * a.inv_t;
  if ((m == -kInf && s[1] == 0.0f) || gt == 0.0f) {
    zero_part<kF32>(dz, lo, n);
    return;
  }
  const float c2 = a.c2;
  int id = -1;
  float zi = -kInf, q = 0.0f;
  if (tid < a.k) {
    const int64_t at = row * a.k + tid, j = a.ids[at] + shift - first;
    if (j >= lo && j < n) {
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
  int times = 0;
  if (mine) {
#pragma unroll 4
    for (int i = 0; i < a.k; i += 4) {
      const u32x4 v = *reinterpret_cast<const u32x4*>(s_id + i);
#pragma unroll
      for (int e = 0; e < 4; ++e) times += (int)v[e] == id;
    }
  }
  if (times > 1) {  // its first entry takes the sum
    q = 0.0f;
    for (int i = 0; i < a.k; ++i) {
      const bool same = s_id[i] == id;
      q += same ? s_q[i] : 0.0f;
      mine = mine && !(same && i < tid);
    }
  }
  // off p_j as one power of two: off may be as large as p_j is small
  const float go = off < 0.0f ? -gt : gt, up = __log2f(fabsf(off)) - l2;
  map_part<kF32, kPast>(z, dz, lo, n, [&](int, float* x) {
#pragma unroll
    for (int i = 0; i < Elem<kF32>::kE; ++i) x[i] = exp2_(__builtin_fmaf(x[i] - m, c2, up)) * go;
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

// Parts of a row, for positions up to V and the largest shift of its rows.
struct Parts {
  int S, part;
};
Parts split_row(int64_t units, int64_t S) {
  const int64_t per = (units + S - 1) / S;
  return Parts{(int)((units + per - 1) / per), (int)(per * kUnit)};
}
int64_t units_of(int64_t V, int shift) { return (V + shift + kUnit - 1) / kUnit; }
Parts fwd_parts(int64_t T, int64_t V, int shift) {
  const int64_t units = units_of(V, shift);
  const int64_t S = std::min<int64_t>({(int64_t)kMaxParts, units, (1024 + T - 1) / T});
  return split_row(units, std::max(S, (units + kMaxUnits - 1) / kMaxUnits));
}
// In the backward passes one unit to a workgroup (us with one, two and four:
// 4096 x 32768 98, 106, 111, 1024 x 98304 76, 81, 87), as long as a grid holds
// them: its threads are counted in 32 bits.
Parts bwd_parts(int64_t T, int64_t V, int shift) {
  const int64_t units = units_of(V, shift), most = std::max<int64_t>(kMaxGrid / T, 1);
  return split_row(units, std::min(units, most));
}
int largest_shift(const Logits& z) {
  const int64_t bytes = z.f32 ? 4 : 2;
  const bool aligned = reinterpret_cast<uintptr_t>(z.Z) % 16 == 0 && (z.T == 1 || z.ldz * bytes % 16 == 0);
  return aligned ? 0 : (int)(16 / bytes - 1);
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

bool past_caches(const Logits& z) { return z.T * z.V * (z.f32 ? 4 : 2) > kPastBytes; }

// f(type is float32, past the caches), both as constants.
template <typename F>
hipError_t by_kind(const Logits& z, F f) {
  const auto of = [&](auto f32) {
    return past_caches(z) ? f(f32, std::true_type{}) : f(f32, std::false_type{});
  };
  return z.f32 ? of(std::true_type{}) : of(std::false_type{});
}

template <int kOp, bool kTop>
hipError_t run_fwd(const RowsFwd& a, const Logits& z, hipStream_t stream) {
  return by_kind(z, [&](auto f32, auto past) {
    constexpr bool kF32 = decltype(f32)::value;
    const size_t n = (size_t)std::min(a.part, a.V + 7);  // positions of a part
    size_t lds = 0;
    if (kOp != kLogprobs) lds = (n + 127) / 128 * 16;
    if (kTop) {
      const size_t bins = (n + kUnit - 1) / kUnit * kThreads * 4;
      const size_t lists = a.S > 1 ? (size_t)a.S * a.n_top * 8 : 0;
      lds = sizeof(TopLds) + std::max(bins, lists);
    }
    rows_fwd_kernel<kF32, kOp, kTop, decltype(past)::value>
        <<<dim3((unsigned)(z.T * a.S)), dim3(fwd_threads(kOp)), lds, stream>>>(a);
    return hipGetLastError();
  });
}

}  // namespace

size_t logits_workspace_bytes(int64_t T, int64_t V, int n_top) {
  const int64_t S = std::max(fwd_parts(T, V, 0).S, fwd_parts(T, V, 7).S);
  return (size_t)(up256(T * S * 8) + up256(T * S * 16) + up256(T * S * 8 * n_top));
}

hipError_t launch_logprobs_fwd(const Logits& z, const int64_t* target, float* logp, float* entropy, int n_top,
                               int64_t* top_ids, float* top_logp, float* stats, void* ws, hipStream_t stream) {
  const Parts p = fwd_parts(z.T, z.V, largest_shift(z));
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
  return n_top ? run_fwd<kLogprobs, true>(a, z, stream) : run_fwd<kLogprobs, false>(a, z, stream);
}

hipError_t launch_distill_fwd(const Logits& z, const TopLogits& t, const float* teacher_lse, float* loss,
                              float* stats, void* ws, hipStream_t stream) {
  const Parts p = fwd_parts(z.T, z.V, largest_shift(z));
  RowsFwd a{};
  a.Z = reinterpret_cast<const char*>(z.Z);
  a.ldz = z.ldz * (z.f32 ? 4 : 2);
  a.V = (int)z.V; a.S = p.S; a.part = p.part;
  a.inv_t64 = 1.0 / z.temperature;
  a.c64 = a.inv_t64 / kLn2;
  a.inv_t = (float)a.inv_t64;
  a.c2 = (float)a.c64;
  a.stats = stats;
  a.ids = t.ids; a.values = t.values; a.values_f32 = t.f32; a.k = t.k;
  a.teacher_lse = teacher_lse; a.loss = loss;
  carve(a, z.T, 0, ws);
  return teacher_lse ? run_fwd<kDistillRest, false>(a, z, stream) : run_fwd<kDistill, false>(a, z, stream);
}

static RowsBwd bwd_args(const Logits& z, const float* stats, void* dZ, int64_t lddz) {
  const Parts p = bwd_parts(z.T, z.V, largest_shift(z));
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
  return by_kind(z, [&](auto f32, auto past) {
    logprobs_bwd_kernel<decltype(f32)::value, decltype(past)::value>
        <<<dim3((unsigned)(z.T * a.S)), dim3(kThreads), 0, stream>>>(a);
    return hipGetLastError();
  });
}

hipError_t launch_distill_bwd(const Logits& z, const TopLogits& t, const float* stats, const float* g, void* dZ,
                              int64_t lddz, hipStream_t stream) {
  RowsBwd a = bwd_args(z, stats, dZ, lddz);
  a.ids = t.ids; a.values = t.values; a.values_f32 = t.f32; a.k = t.k; a.g = g;
  return by_kind(z, [&](auto f32, auto past) {
    distill_bwd_kernel<decltype(f32)::value, decltype(past)::value>
        <<<dim3((unsigned)(z.T * a.S)), dim3(kThreads), 0, stream>>>(a);
    return hipGetLastError();
  });
}

}  // namespace qlora
