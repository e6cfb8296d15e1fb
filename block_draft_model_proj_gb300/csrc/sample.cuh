// Filtered sampling of logits rows, and speculative-sampling verification against the
// filtered target distribution.
//
// "DFlash: drafting, verification, and speed", Sampling with temperature is not argmax
// matching: acceptance needs the ACTUAL proposal distribution q (after any top-k,
// temperature or selector on the draft side) and the target's p.  dflash_sample_tokens draws
// the proposals and writes q; dflash_verify_sampling_filtered tests them against a target
// filtered the same way.
//
// Per row, with logits l and their maximum M: w_v = exp((l_v - M) / T).  Kept tokens: those
// with w_v >= min_p; of those the top_k largest; of those, in the order (logit descending,
// index ascending), every token whose predecessors' mass is below top_p of the mass so far
// kept.  All three cuts keep a prefix of that order, so the kept set is always
//   { v : l_v > pivot, or l_v == pivot and v <= cut }
// and a row's whole outcome is (M, pivot, cut, Z = sum of the kept w).  The sampled token is
// the lowest v whose inclusive sum of kept w, in index order, exceeds u Z.
//
// Numbers next to a border (a token whose predecessors hold almost exactly top_p of the
// mass, a u that falls on the seam of two tokens) decide whole tokens, so masses are exact
// integers: w is computed to about 2^-31 (weight_parts) and held in units of 2^-44, sums are
// 64-bit integer sums.  They do not depend on how a row is split or on the order of atomics.
//
// One thread-block cluster of 1 to 8 CTAs per row (row_shape): each CTA reads its slice of the
// row from HBM once, for its maximum; later passes find it in L2 (a copy in shared memory made
// no call faster and left room for fewer CTAs).  The CTAs join maxima, counts and sums through
// distributed shared memory.
//
// Most rows keep few tokens, and then only those need exact weights.  A threshold that the
// kept tokens certainly reach is found cheaply -- top-k: from the maxima of groups of threads;
// min-p: it is the threshold; top-p: like a top-k of kGuess -- the tokens above it (at most
// kList) are gathered in one CTA, which ranks them and finishes the row.  For top-p this needs
// the row's total, and an unfiltered draw needs the tokens' running sum: both are taken with
// fast fp32 weights, whose error is bounded (kFastBits, kRoughBits), and the outcome stands
// when no border lies within that bound.
//
// Rows that keep more, and undecided ones: bf16 tokens are counted per value (there are few),
// with one exact weight per value (value_cut).  For fp32, counts per bucket of the weight find
// nuclei of up to kList tokens; beyond that every weight is computed exactly: a histogram of
// masses over buckets of 1/32 octave finds the bucket that holds the cut, which is sorted, or
// cut by a radix selection on the logit's bits and then by index when it is large (long ties,
// tokens beyond 2^-64 of the maximum).
//
// Measured (GB300, 151936 logits a row, temperature 0.85, device us of a call; "with q":
// probabilities written too; the floor of 960 rows is 43 / 129 us in bf16, 86 / 172 in fp32).
// Rows: N(0, 1.5) and 200 tokens falling off from 18 by 2 ln(rank), "broad" from 9 by ln(rank);
// up to 120 rows are found in L2.
//   bf16 rows             1      15     120    960    960 with q
//   greedy                5.4    6.2    9.8    57     154
//   min-p 0.05            10     11     16     94     196
//   top-k 50              12     13     18     104    206
//   top-p 0.9             13     14     22     131    225
//   unfiltered            11     15     28     162    286
//   min-p 0.001, broad    25     35     79     283    397
//   top-k 400             27     29     70     293    487    (a list that is sorted)
//   top-k 600 or 5000     30     35     83     458    615    (by value)
//   top-p 0.9, broad      41     45     96     551    824    (tens of thousands kept)
//   fp32 rows
//   greedy                5.6    6.6    18     94     192
//   top-k 50              11     12     28     190    310
//   top-p 0.9             13     14     33     287    376
//   unfiltered            12     14     41     259    412
//   top-k 600 or 5000     27     31     94     584    706    (exact)
//   min-p 0.001, broad    26     32     87     335    439
//   top-p 0.9, broad      85     99     243    1247   1479   (exact)
// Few rows are bound by dependent phases of about 1 us (cluster barriers, the gather, the
// list).  Many rows that keep few tokens wait for loads in both passes and at barriers (issue
// slots 31 to 41 % used); broad nuclei are bound by issue (64 %) with one shared-memory atomic
// per token, fp32 ones by four of them and an exact weight per token.
//
// This header holds what a row's CTAs do; sample_*.cu compile filter_kernel for one type and
// purpose each (side by side: the kernel is long), sample.cu holds the rest of the two calls.
#pragma once

#include <cooperative_groups.h>

#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace cg = cooperative_groups;

namespace dflash {

typedef unsigned long long u64;

// One row's filtered distribution; z = 0: nothing is kept.
struct RowStats {
  float mx, pivot, chi, clo;  // chi + clo = log2(e) / T
  int cut;
  int pad;
  u64 z;                      // sum of the kept w, units of 2^-44
};

struct FilterArgs {
  const void* logits;
  long ld;                    // elements between rows
  int V, C, per;              // per: rows that share one request's settings
  const float* temperature;   // [rows / per], optional as the next three
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  // sampling
  const float* uniforms;
  int32_t* tokens;
  float* probs;               // [rows][V] or nullptr
  // verification
  const float* q;
  const int32_t* draft;
  RowStats* stats;
  uint8_t* accept;
  int gamma;
  unsigned* status;
};

// Defined for <bf16 or float, sampling or verification, 512 or 256 threads> in sample_*.cu.
template <typename T, bool kVerify, int kNT>
cudaError_t launch_filter_nt(const FilterArgs& a, long rows, cudaStream_t stream);

namespace {

constexpr int kMaxNT = 512;          // threads per CTA: 512 or 256
constexpr int kBuckets = 2048;       // 64 octaves of 32 buckets
constexpr int kList = 1024;          // tokens a CTA sorts
constexpr int kSlots = 2048;         // places for gathered tokens
// Up to here the list is ranked by counting, else sorted (one row, top-k 50: 11.5 against 15.7
// us; top-k 100: 13.8 against 17.7).
constexpr int kCountList = 256;
// Tokens that a nucleus is first tried with: the list then holds about twice as many.  960 rows
// under top-p 0.9: 127 us with 48, 142 with 96, 172 with 160 (longer lists to rank); a nucleus
// that the list does not hold costs the next tier (one row: 45 us).
constexpr int kGuess = 64;
// Bins of one bf16 value each, largest first: magnitudes in [2^-9, 2^6) of either sign, with
// one bin above, one for the small magnitudes between the signs, and one below.
constexpr int kValueOctaves = 15 * 128, kValueLowest = 0x3B00;  // 2^-9 as bf16 bits
constexpr int kValueBins = 2 * kValueOctaves + 3, kValueSmall = kValueOctaves + 1;
constexpr int kMaxSteps = 1040;      // 32-vector steps of one CTA's slice
constexpr int kMaxC = 8;             // CTAs per row (portable cluster size)
constexpr int kOneBits = 44;         // w = 1 is 2^44: sums of 2^19 tokens stay below 2^63
constexpr float kMinTemp = 1e-6f, kMaxTemp = 1e6f;
constexpr float kFastLogit = 1e30f;   // fast weights need |M| below this (no overflow in x)
// Error of a sum of fast weights over any of a row's tokens, relative to the row's total, in
// units of 2^-24: ex2.approx 4, its correction's rounding 1, the additions of a step 8, and the
// rounding of l - M, |x| ln 2 for a weight 2^x.  By weight |x| is 14.3 on average at most: beside
// M's own weight, n weights of 2^-y have the mean a with n 2^-y (y - a) = a, largest at
// y = a + 1 / ln 2, and n = 2^19 gives 14.26 -- 9.9 units.  23 in all: below 2^-19.
constexpr int kFastBits = 19;
// ... and of rough weights: the roundings of x and of chi, 9.9 units each, are left in: 4 + 3
// additions + 3 * 9.9, below 2^-18.
constexpr int kRoughBits = 17;

// round(2^(31 + j/32))
__device__ const uint32_t kExp2Table[32] = {
    2147483648u, 2194507417u, 2242560872u, 2291666561u, 2341847524u, 2393127307u, 2445529972u,
    2499080105u, 2553802834u, 2609723834u, 2666869345u, 2725266179u, 2784941738u, 2845924021u,
    2908241642u, 2971923842u, 3037000500u, 3103502151u, 3171459999u, 3240905930u, 3311872529u,
    3384393094u, 3458501653u, 3534232978u, 3611622603u, 3690706840u, 3771522796u, 3854108391u,
    3938502376u, 4024744348u, 4112874773u, 4202935003u};

struct Exp2Table {
  uint32_t fix[32];   // 2^(31 + j/32)
  float flt[32];
};

// w = exp((l - mx) / T) = mant * 2^(n - 31), mant in [2^31, 2^32): relative error about
// 2^-30.5.  l - mx as a sum of two floats, times chi + clo; 2^x by the nearest 32nd (table)
// and the Taylor series of 2^f - 1, |f| <= 1/64, whose fp32 rounding is 2^-31 absolute.
// Returns false below 2^-150 (and for NaN).
__device__ __forceinline__ bool weight_parts(float l, float mx, float chi, float clo,
                                             const Exp2Table& tab, uint32_t& mant, int& n) {
  float d = l - mx;
  const float bv = d - l, av = d - bv;
  float e = (l - av) - (mx + bv);
  if (l == mx) d = e = 0.f;
  const float x = d * chi;
  const float xl = fmaf(d, chi, -x) + fmaf(d, clo, e * chi);
  if (!(x > -150.f)) return false;
  const float m = x + 393216.f;  // 1.5 * 2^18: one unit in the last place is 1/32
  const int k = __float_as_int(m) - __float_as_int(393216.f);
  const float f = (x - (m - 393216.f)) + xl;
  const float p = f * fmaf(f, fmaf(f, fmaf(f, 0.009618129f, 0.055504109f), 0.240226507f),
                           0.693147181f);
  const int j = k & 31;
  n = k >> 5;
  mant = tab.fix[j] + (uint32_t)__float2int_rn(tab.flt[j] * p);
  return true;
}

// w in units of 2^-44, rounded to nearest.
__device__ __forceinline__ u64 weight_units(float l, float mx, float chi, float clo,
                                            const Exp2Table& tab) {
  uint32_t mant;
  int n;
  if (!weight_parts(l, mx, chi, clo, tab, mant, n)) return 0;
  const u64 w = (u64)mant << (kOneBits - 31);
  if (n >= 0) return w;         // n = 0: x is at most 0
  const int s = -n;
  if (s > kOneBits + 1) return 0;
  return (w + (1ull << (s - 1))) >> s;
}

// The smallest float l with (l - mx) / T >= ln(min_p), ln to about 2^-30: logf's value y and
// the rest of min_p over exp(y) (as weight_parts finds it), T times their sum as a sum of two
// floats.
__device__ __forceinline__ float min_p_threshold(float mx, float temp, float min_p,
                                                 const Exp2Table& tab) {
  const float y = fminf(logf(min_p), 0.f);
  uint32_t mant = 0x80000000u;
  int n = 0;
  weight_parts(y, 0.f, 1.44269502f, 1.92596299e-8f, tab, mant, n);  // min_p > 2^-150
  // min_p 2^(31 - n), an integer near 2^31: two factors, each a normal float
  const int h = (31 - n) / 2;
  const float m = min_p * __int_as_float((h + 127) << 23) * __int_as_float((31 - n - h + 127) << 23);
  const float rest = (float)((long long)m - (long long)mant) / (float)mant;
  const float hi = temp * y, lo = fmaf(temp, y, -hi) + temp * rest;
  const float s = mx + hi, bv = s - mx;
  const float e = ((mx - (s - bv)) + (hi - bv)) + lo;
  const float t = s + e;
  if (!(fabsf(t) < INFINITY)) return fmaxf(t, -3.402823466e38f);
  if ((s - t) + e <= 0.f) return t;
  // the next float up
  const int b = __float_as_int(t);
  return t == 0.f ? __int_as_float(1) : __int_as_float(t > 0.f ? b + 1 : b - 1);
}

// f * z for f in [0, 1), rounded down or up, exactly.
__device__ __forceinline__ u64 mul_fraction(float f, u64 z, bool up) {
  const uint32_t b = __float_as_uint(f);
  const int ex = (int)(b >> 23);
  const u64 m = ex ? (b & 0x7fffffu) | 0x800000u : b & 0x7fffffu;
  const int sh = 150 - (ex ? ex : 1);  // f = m 2^-sh, sh >= 24
  const u64 lo = m * z, hi = __umul64hi(m, z);
  u64 r;
  bool rest;
  if (sh < 64) {
    r = hi << (64 - sh) | lo >> sh;
    rest = (lo & ((1ull << sh) - 1)) != 0;
  } else {
    const int t = sh - 64;             // hi < 2^24
    r = t < 64 ? hi >> t : 0;
    rest = lo != 0 || (t < 64 ? (hi & ((1ull << t) - 1)) != 0 : hi != 0);
  }
  return r + (up && rest ? 1 : 0);
}

// 2^107 / z for z in [2^44, 2^63], to about 2^-60: a reciprocal in fp32 and two Newton steps
// on 64-bit integers.
__device__ __forceinline__ u64 reciprocal(u64 z) {
  const int s = __clzll((long long)z);      // z 2^s in [2^63, 2^64)
  const u64 n = z << s;
  const float y = __fdiv_rn(8388608.f, (float)(uint32_t)(n >> 40));   // in (1/2, 1]
  long long i = (long long)(y * 4611686018427387904.f) << 1;          // 2^126 / n, 23 bits
  if (i < 0) i = 0x7fffffffffffffffll;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const long long e = (1ll << 62) - (long long)__umul64hi(n, (u64)i);
    const long long d = __mul64hi(i, e) << 2;
    i = e > 0 && i > 0x7fffffffffffffffll - d ? 0x7fffffffffffffffll : i + d;
  }
  return (u64)i >> (19 - s);
}

// top_p's share of a total, at least one unit and at most all of it
__device__ __forceinline__ u64 share_of(float top_p, u64 total) {
  const u64 n = mul_fraction(top_p, total, true);
  return n < 1 ? 1 : n > total ? total : n;
}

// ---- pairs of fp32 operations ----
__device__ __forceinline__ u64 pack2(float a, float b) {
  u64 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(u64 v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ u64 add2(u64 a, u64 b) {
  u64 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ u64 mul2(u64 a, u64 b) {
  u64 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ u64 fma2(u64 a, u64 b, u64 c) {
  u64 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Fast weights: 2^x, x = (l - M) * chi in fp32, corrected by what the product's rounding and
// chi's low part leave out -- rough ones without that.  Logits are first clamped to lmin
// (unpack_clamped), whose weight is 0: no -inf and no NaN gets here.
struct FastScale {
  u64 nmx, chi, nchi, nclo;
  float lmin;
  __device__ __forceinline__ FastScale(float mx, float c, float cl) {
    nmx = pack2(-mx, -mx);
    chi = pack2(c, c);
    nchi = pack2(-c, -c);
    nclo = pack2(-cl, -cl);
    lmin = __fsub_rd(mx, 200.f / c);
  }
  __device__ __forceinline__ u64 two(float a, float b) const {
    const u64 d = add2(pack2(a, b), nmx);
    const u64 x = mul2(d, chi);
    const u64 left = fma2(d, nclo, fma2(d, nchi, x));  // x - d (chi + clo)
    float x0, x1;
    unpack2(x, x0, x1);
    const u64 e = pack2(ex2f(x0), ex2f(x1));
    return fma2(mul2(e, left), pack2(-0.693147181f, -0.693147181f), e);
  }
  __device__ __forceinline__ u64 two_rough(float a, float b) const {
    float x0, x1;
    unpack2(mul2(add2(pack2(a, b), nmx), chi), x0, x1);
    return pack2(ex2f(x0), ex2f(x1));
  }
  // the weights of a vector of logits, added up
  template <int kN, bool kRough>
  __device__ __forceinline__ float sum(const float* v) const {
    u64 w[kN / 2];
#pragma unroll
    for (int e = 0; e < kN / 2; ++e)
      w[e] = kRough ? two_rough(v[2 * e], v[2 * e + 1]) : two(v[2 * e], v[2 * e + 1]);
    u64 s = add2(w[0], w[1]);
    if constexpr (kN == 8) s = add2(s, add2(w[2], w[3]));
    float s0, s1;
    unpack2(s, s0, s1);
    return s0 + s1;
  }
};

// a total order in which larger logits come first (finite logits and +inf)
__device__ __forceinline__ uint32_t desc_key(float l) {
  const uint32_t b = __float_as_uint(l + 0.f);  // -0 and +0 are one value
  return ~((b & 0x80000000u) ? ~b : (b | 0x80000000u));
}
__device__ __forceinline__ float key_value(uint32_t k) {
  k = ~k;
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void unpack(const uint4& u, float* v) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = __uint_as_float(w[e] << 16);
      v[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
    }
  }
  // largest element (a NaN operand is dropped)
  static __device__ __forceinline__ __nv_bfloat162 pair_max(const uint4& u) {
    __nv_bfloat162 w[4];
    memcpy(w, &u, sizeof(w));
    return __hmax2(__hmax2(w[0], w[1]), __hmax2(w[2], w[3]));
  }
  static __device__ __forceinline__ float largest(const uint4& u) {
    const __nv_bfloat162 m = pair_max(u);
    return fmaxf(__low2float(m), __high2float(m));
  }
  // a running maximum
  struct Max {
    __nv_bfloat162 m = __float2bfloat162_rn(-INFINITY);
    __device__ __forceinline__ void push(const uint4& u) { m = __hmax2(m, pair_max(u)); }
    __device__ __forceinline__ float value() const {
      const float v = fmaxf(__low2float(m), __high2float(m));
      return v == v ? v : -INFINITY;
    }
  };
  // is an element >= lo?  (lo rounded up to a bf16 tests the same)
  struct AtLeast {
    __nv_bfloat162 lo;
    __device__ __forceinline__ explicit AtLeast(float x) {
      lo = __bfloat162bfloat162(__float2bfloat16_ru(x));
    }
    __device__ __forceinline__ bool any(const uint4& u) const {
      return !__hbltu2(pair_max(u), lo);
    }
  };
  // elements below lo (and NaN) become lo, rounded down to T
  static __device__ __forceinline__ void unpack_clamped(const uint4& u, float lo, float* v) {
    const __nv_bfloat162 l2 = __bfloat162bfloat162(__float2bfloat16_rd(lo));
    __nv_bfloat162 w[4];
    memcpy(w, &u, sizeof(w));
    uint4 c;
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = __hmax2(w[e], l2);
    memcpy(&c, w, sizeof(c));
    unpack(c, v);
  }
};
template <>
struct Vec<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void unpack(const uint4& u, float* v) {
    v[0] = __uint_as_float(u.x);
    v[1] = __uint_as_float(u.y);
    v[2] = __uint_as_float(u.z);
    v[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ float largest(const uint4& u) {
    return fmaxf(fmaxf(__uint_as_float(u.x), __uint_as_float(u.y)),
                 fmaxf(__uint_as_float(u.z), __uint_as_float(u.w)));
  }
  struct Max {
    float m = -INFINITY;
    __device__ __forceinline__ void push(const uint4& u) { m = fmaxf(m, largest(u)); }
    __device__ __forceinline__ float value() const { return m; }
  };
  struct AtLeast {
    float lo;
    __device__ __forceinline__ explicit AtLeast(float x) : lo(x) {}
    __device__ __forceinline__ bool any(const uint4& u) const { return largest(u) >= lo; }
  };
  static __device__ __forceinline__ void unpack_clamped(const uint4& u, float lo, float* v) {
    unpack(u, v);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = fmaxf(v[e], lo);
  }
};

// A CTA's slice of a logits row as 16-byte vectors on 16-byte boundaries of global memory
// whatever the row's own alignment: vector j holds elements first + j*kN + e, and elements
// outside [c0, c1) read as -inf.
template <typename T, int kNT>
struct Slice {
  static constexpr int kN = Vec<T>::kN;
  const T* row = nullptr;
  int c0 = 0, c1 = 0;         // elements of this CTA
  int first = 0;              // index of vector 0's first element (may be below c0)
  int nv = 0;

  __device__ __forceinline__ void init(const T* r, int lo, int hi) {
    row = r;
    c0 = lo;
    c1 = hi > lo ? hi : lo;
    const int pre = (int)(((uintptr_t)(r + lo) & 15) / sizeof(T));
    first = lo - pre;
    nv = c1 > c0 ? (c1 - first + kN - 1) / kN : 0;
  }
  __device__ __forceinline__ uint4 load(int j) const {
    const int i0 = first + j * kN;
    if (i0 >= c0 && i0 + kN <= c1) return __ldg(reinterpret_cast<const uint4*>(row + i0));
    union {
      uint4 u;
      T t[kN];
    } r;
#pragma unroll
    for (int e = 0; e < kN; ++e) {
      const int i = i0 + e;
      r.t[e] = (i >= c0 && i < c1) ? row[i] : from_f<T>(-INFINITY);
    }
    return r.u;
  }
  __device__ __forceinline__ float at(int i) const {  // -inf outside the slice
    if (i < c0 || i >= c1) return -INFINITY;
    return to_f(row[i]);
  }
  __device__ __forceinline__ void values(int j, float* v) const { Vec<T>::unpack(load(j), v); }
  // f(s, j, vector) for the steps s = warp, warp + kNT / 32, ... of 32 vectors, each warp taking
  // the vectors j = 32 s + lane of its steps, four steps' loads at a time (-inf past the end)
  template <typename F>
  __device__ __forceinline__ void each_step(F f) const {
    constexpr int kW = kNT / 32;
    const uint32_t none = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;
    const int lane = threadIdx.x & 31, steps = (nv + 31) / 32;
    for (int s = threadIdx.x >> 5; s < steps; s += 4 * kW) {
      uint4 r[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int j = (s + q * kW) * 32 + lane;
        r[q] = j < nv ? load(j) : make_uint4(none, none, none, none);
      }
      // one copy of f: it can be long, and cold instructions cost more than the moves
#pragma unroll 1
      for (int t = s; t < min(steps, s + 4 * kW); t += kW) {
        f(t, t * 32 + lane, r[0]);
        r[0] = r[1];
        r[1] = r[2];
        r[2] = r[3];
      }
    }
  }
  // f(j, vector) for this thread's vectors j = tid, tid + kNT, ..., kU loads at a time; past
  // the end f may get vectors of -inf.  Blocks of kU * kNT vectors that lie whole in the slice
  // are loaded without a look at its edges.
  template <int kU, typename F>
  __device__ __forceinline__ void each(F f) const {
    const uint32_t none = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;
    const int e0 = first == c0 ? 0 : 1;
    const int e1 = first + nv * kN == c1 ? nv : nv - 1;
    const uint4* p = reinterpret_cast<const uint4*>(row + first);
    for (int b = 0; b < nv; b += kU * kNT) {
      const int j = b + threadIdx.x;
      uint4 r[kU];
      if (b >= e0 && b + kU * kNT <= e1) {
#pragma unroll
        for (int q = 0; q < kU; ++q) r[q] = p[j + q * kNT];
      } else {
#pragma unroll
        for (int q = 0; q < kU; ++q)
          r[q] = j + q * kNT < nv ? load(j + q * kNT) : make_uint4(none, none, none, none);
      }
#pragma unroll
      for (int q = 0; q < kU; ++q) f(j + q * kNT, r[q]);
    }
  }
};

struct Shared {
  Exp2Table tab;
  union {
    uint32_t hist[4][kBuckets];  // count, and w in three 15-bit pieces
    struct {                     // CTA 0
      u64 slot[kSlots];          // gathered tokens, kSlots / C places for each CTA
      u64 key[kList];
      u64 mass[kList];
    } list;
    struct {
      uint32_t count[2 * kValueOctaves];  // by value_index
      uint32_t zone_count[3];    // the bins that hold several values, and their masses
      u64 mass[3];
    } val;
    u64 weight[2 * kValueOctaves];        // by value_index, 0 where it is not kept
  };
  u64 step[kMaxSteps];
  u64 warp64[kMaxNT / 32];
  uint32_t warp32[kMaxNT / 32];
  alignas(16) float gmax[kMaxNT];   // read four at a time
  int warpi[kMaxNT / 32];
  // written by the row's CTAs into each other
  float cmax[kMaxC], cthr[kMaxC];
  u64 cmass[kMaxC];
  uint32_t ccnt[kMaxC], clist[kMaxC];
  struct Found {
    int bucket;
    uint32_t cnt_before, cnt_in;
    u64 mass_before, total;
  } found;
  struct Pivot {
    float value;
    int cut;
  } pivot;
  int index;
  int verdict;
  uint32_t list_n;
  u64 last_key, last_z;  // the last kept token of the list, and the mass up to it
};

__device__ __forceinline__ u64 shfl_xor64(u64 v, int o) {
  return __shfl_xor_sync(0xffffffffu, v, o);
}
__device__ __forceinline__ u64 warp_sum64(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += shfl_xor64(v, o);
  return v;
}

// Inclusive scans over the block's threads, and the totals.
template <int kNT>
__device__ __forceinline__ void block_scan(uint32_t& c, u64& m, uint32_t& ctot, u64& mtot,
                                           Shared& sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t c2 = __shfl_up_sync(0xffffffffu, c, o);
    const u64 m2 = __shfl_up_sync(0xffffffffu, m, o);
    if (lane >= o) {
      c += c2;
      m += m2;
    }
  }
  __syncthreads();
  if (lane == 31) {
    sh.warp32[warp] = c;
    sh.warp64[warp] = m;
  }
  __syncthreads();
  ctot = 0;
  mtot = 0;
  for (int w = 0; w < kNT / 32; ++w) {
    if (w == warp) {
      c += ctot;
      m += mtot;
    }
    ctot += sh.warp32[w];
    mtot += sh.warp64[w];
  }
  // the callers' next write of warp32 / warp64 is behind another __syncthreads
}

// value -> slot [rank] of the array at the same place in every CTA of the cluster
template <typename X>
__device__ __forceinline__ void publish(cg::cluster_group& cl, X* arr, int rank, int C, X v) {
  if ((int)threadIdx.x < C) cl.map_shared_rank(arr, threadIdx.x)[rank] = v;
}

// Lowest index whose inclusive sum of weights exceeds target(total), over the whole row in
// index order; -1 when the total is 0.  weight(value, index, e) must be the same on both
// passes.  Every CTA of the cluster returns the index; *total_out the total.  whole(vector,
// index of its first element): a cheaper way to the sum of a vector's weights, as a u64, or as
// a uint32_t where they are 0 and 1.
struct NoWhole {};
template <typename T, int kNT, typename W, typename G, typename Q = NoWhole>
__device__ int search(cg::cluster_group& cl, Shared& sh, const Slice<T, kNT>& sl, int rank, int C,
                      W weight, G target, u64* total_out, Q whole = Q()) {
  constexpr int kN = Slice<T, kNT>::kN;

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int steps = (sl.nv + 31) / 32;
  auto vec_sum = [&](int j, const uint4& r) {
    u64 s = 0;
    float v[kN];
    Vec<T>::unpack(r, v);
#pragma unroll
    for (int e = 0; e < kN; ++e) s += weight(v[e], sl.first + j * kN + e);
    return s;
  };
  sl.each_step([&](int s, int j, const uint4& r) {
    u64 t;
    if constexpr (std::is_same<Q, NoWhole>::value) {
      t = warp_sum64(vec_sum(j, r));
    } else {
      const auto w = whole(r, sl.first + j * kN);
      if constexpr (sizeof(w) == 4) t = __reduce_add_sync(0xffffffffu, w);
      else t = warp_sum64(w);
    }
    if (lane == 0) sh.step[s] = t;
  });
  __syncthreads();
  u64 mine = 0;
  for (int s = threadIdx.x; s < steps; s += kNT) mine += sh.step[s];
  uint32_t c = 0, ct;
  u64 mt;
  block_scan<kNT>(c, mine, ct, mt, sh);
  publish(cl, sh.cmass, rank, C, mt);
  cl.sync();
  u64 total = 0, before = 0;
  for (int r = 0; r < C; ++r) {
    if (r == rank) before = total;
    total += sh.cmass[r];
  }
  const u64 own = sh.cmass[rank];
  *total_out = total;
  if (total == 0) {
    cl.sync();
    return -1;
  }
  const u64 t = target(total);
  if (t >= before && t < before + own && warp == 0) {
    u64 acc = before;
    int s = 0;
    for (int s0 = 0; s0 < steps; s0 += 32) {
      const u64 x = s0 + lane < steps ? sh.step[s0 + lane] : 0;
      u64 incl = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const u64 up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, acc + incl > t);
      if (hit) {
        const int h = __ffs(hit) - 1;
        s = s0 + h;
        acc += __shfl_sync(0xffffffffu, incl - x, h);
        break;
      }
      acc += __shfl_sync(0xffffffffu, incl, 31);
    }
    // the step's tokens in order, 32 at a time (one short copy of the weight's code: this is
    // one warp's work while the row waits)
    int idx = -1;
#pragma unroll 1
    for (int r = 0; r < kN && idx < 0; ++r) {
      const int i = sl.first + s * 32 * kN + r * 32 + lane;
      u64 incl = weight(sl.at(i), i);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const u64 up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, acc + incl > t);
      if (hit) idx = i - lane + __ffs(hit) - 1;
      acc += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane < C) *cl.map_shared_rank(&sh.index, lane) = idx;
  }
  cl.sync();
  return sh.index;
}

// search() over the kept tokens' weights with fast sums: *total_out has their relative error
// of 2^-kFastBits.  The token when no seam lies within the error of u Z and of the sum before
// it, else -2.  some: not every logit above -inf is kept.
template <typename T, int kNT, typename K, typename L, typename U>
__device__ int search_fast(cg::cluster_group& cl, Shared& sh, const Slice<T, kNT>& sl, int rank,
                           int C, bool some, K kept, L least_kept, const FastScale& fs, U units, float u,
                           u64* total_out) {
  constexpr int kN = Slice<T, kNT>::kN;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int steps = (sl.nv + 31) / 32;
  sl.each_step([&](int s, int j, const uint4& r) {
    float v[kN];
    Vec<T>::unpack_clamped(r, fs.lmin, v);
    if (some) {
      const int i0 = sl.first + j * kN;
      const float least = least_kept(i0);
      if (least == least) {
#pragma unroll
        for (int e = 0; e < kN; ++e) v[e] = v[e] >= least ? v[e] : fs.lmin;
      } else {
#pragma unroll 1
        for (int e = 0; e < kN; ++e)
          if (!kept(v[e], i0 + e)) v[e] = fs.lmin;
      }
    }
    const float sum = warp_sum(fs.template sum<kN, false>(v));
    if (lane == 0) sh.step[s] = __float2ull_rn(sum * 17592186044416.f);
  });
  __syncthreads();
  u64 mine = 0, mt;
  for (int s = threadIdx.x; s < steps; s += kNT) mine += sh.step[s];
  uint32_t c = 0, ct;
  block_scan<kNT>(c, mine, ct, mt, sh);
  publish(cl, sh.cmass, rank, C, mt);
  if (threadIdx.x == 0) sh.index = -2;
  cl.sync();
  u64 total = 0, before = 0;
  for (int r = 0; r < C; ++r) {
    if (r == rank) before = total;
    total += sh.cmass[r];
  }
  *total_out = total;
  const u64 t = mul_fraction(u, total, false);
  const u64 err = (total >> (kFastBits - 1)) + 1;  // of the sum before a token and of u Z
  if (t >= before && t < before + sh.cmass[rank] && warp == 0) {
    u64 acc = before;
    int s = 0;
    for (int s0 = 0; s0 < steps; s0 += 32) {
      const u64 x = s0 + lane < steps ? sh.step[s0 + lane] : 0;
      u64 incl = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const u64 up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, acc + incl > t);
      if (hit) {
        const int h = __ffs(hit) - 1;
        s = s0 + h;
        acc += __shfl_sync(0xffffffffu, incl - x, h);
        break;
      }
      acc += __shfl_sync(0xffffffffu, incl, 31);
    }
    int idx = -2;
#pragma unroll 1
    for (int r = 0; r < kN; ++r) {
      const int i = sl.first + s * 32 * kN + r * 32 + lane;
      const float l = sl.at(i);
      const u64 w = kept(l, i) ? units(l) : 0;
      u64 incl = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const u64 up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
      }
      // (q, q + w] holds t, and stays clear of it by err (nothing weighs before it: exact)
      const u64 q = acc + incl - w;
      if (w && t + err < q + w && (q == 0 || q + err <= t)) idx = i;
      acc += __shfl_sync(0xffffffffu, incl, 31);
      if (acc > t) break;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, idx >= 0);
    if (hit) {
      idx = __shfl_sync(0xffffffffu, idx, __ffs(hit) - 1);
      if (lane < C) *cl.map_shared_rank(&sh.index, lane) = idx;
    }
  }
  cl.sync();
  return sh.index;
}

// Sorts keys in ascending order, thread t holding keys t + r * kNT of which only the first n
// (<= kList) can differ from ~0: a bitonic network whose steps between lanes are shuffles and
// whose wider steps go through sh.list.key.  On return sh.list.key holds the sorted keys as
// well.
template <int kNT, int kKeys>
__device__ __forceinline__ void sort_keys(Shared& sh, u64 (&k)[kKeys], int n) {
  static_assert(kList == kKeys * kNT, "every place of the list has a thread");
  const int tid = threadIdx.x;
  int n2 = 1;
  while (n2 < n) n2 <<= 1;
  for (int size = 2; size <= n2; size <<= 1) {
    for (int j = size >> 1; j > 0; j >>= 1) {
      if (j >= 32) {
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kKeys; ++r)
          if (tid + r * kNT < n2) sh.list.key[tid + r * kNT] = k[r];
        __syncthreads();
      }
#pragma unroll
      for (int r = 0; r < kKeys; ++r) {
        const int i = tid + r * kNT;
        if (r > 0 && n2 <= r * kNT) break;
        u64 o;
        if (j >= 32)
          o = i < n2 ? sh.list.key[i ^ j] : ~0ull;
        else
          o = __shfl_xor_sync(0xffffffffu, k[r], j);
        const bool up = (i & size) == 0, low = (i & j) == 0;
        const bool take_min = up == low;
        k[r] = take_min ? (o < k[r] ? o : k[r]) : (o > k[r] ? o : k[r]);
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kKeys; ++r)
    if (tid + r * kNT < n2) sh.list.key[tid + r * kNT] = k[r];
  __syncthreads();
}

}  // namespace

}  // namespace dflash
