// Expert routing from scores (include/moe_route.h): one wave per token.
//
// Mathematics.  The weights need the scores of the k chosen experts only, and
// the denominator of a softmax where it is not divided out again.  The order
// needs more: with a bias, or groups, experts are compared by sums of scores,
// and fp32 scores of 512 experts lie so close that another rounding swaps two
// of them in about one token in a thousand.  So those scores are formed in
// double precision for all E experts; without bias and groups every score
// grows with its logit and the logits are compared instead.  Most tokens need
// neither: fp32 scores with a proven bound on their error decide wherever the
// keys that matter lie further apart than the bound.  Where neighbours do not,
// the few candidates alone are ranked again in double precision (sigmoid); where
// groups do not, or a softmax's terms, all E scores are formed so.  That
// is many times the usual work (rows that the mask leaves empty, 2% of them,
// and near ties together took 15 of 46 us that way), so the bound is kept close:
// a softmax's falls with its denominator, and with the largest value.
//
// Organisation.  A token's E logits are spread over one wave (a lane holds
// every 64th expert, or groups of four neighbours where E fills the wave and
// rows are aligned), and a block is four tokens whose choices are independent.
//   - The groups' scores: their values go through LDS once; 64 / G lanes scan
//     one group each for its two largest and merge by lane exchanges.
//   - Top-k: the largest threshold with at least k lane maxima at or above it
//     bounds the k-th key from below; it is found on the upper bits of an
//     order-preserving 32-bit image of the key (doubles are rounded to fp32
//     first, which keeps the order up to ties).  The few experts at or above
//     it are ranked against each other exactly, by (key, -id).  More than 64
//     of them (many equal keys) take k rounds of a wave arg-max.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdio>

#include "device_common.h"
#include "moe_internal.h"
#include "moe_route.h"
#include "topk_wave.h"

namespace moe {
namespace {

constexpr int kRtWaves = 4;   // tokens per block

struct RouteArgs {
  const void* logits;
  const float* bias;
  int32_t* ids;
  float* w;
  int64_t stride;   // elements between rows
  int T, E, k, G, tg, gt, renorm;
  int gsize;        // experts per group
  uint32_t ginv;    // ceil(2^20 / gsize): e / gsize = (e ginv) >> 20 for e < 1024
  float scale;
};

__device__ __forceinline__ double dbl(uint32_t hi, uint32_t lo) {
  return __longlong_as_double((static_cast<long long>(hi) << 32) | lo);
}

template <int S>
__device__ __forceinline__ double lane_xor_d(double v, int lane) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v));
  const uint32_t hi = lane_xor<S>(static_cast<uint32_t>(b >> 32), lane);
  return dbl(hi, lane_xor<S>(static_cast<uint32_t>(b), lane));
}

// Sums and maxima over the wave; every lane ends with the same bits.
__device__ __forceinline__ double wave_sum_d(double v, int lane) {
  v += lane_xor_d<1>(v, lane);
  v += lane_xor_d<2>(v, lane);
  v += lane_xor_d<4>(v, lane);
  v += lane_xor_d<8>(v, lane);
  v += lane_xor_d<16>(v, lane);
  return v + lane_xor_d<32>(v, lane);
}

__device__ __forceinline__ float wave_max_f(float v, int lane) {
#define STEP(S) v = fmaxf(v, __uint_as_float(lane_xor<S>(__float_as_uint(v), lane)))
  STEP(1); STEP(2); STEP(4); STEP(8); STEP(16); STEP(32);
#undef STEP
  return v;
}

// 64-bit order key of a double: larger value, larger key; both zeros alike.
// The caller has turned NaN into -inf.
__device__ __forceinline__ uint64_t order_key64(double d) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(d));
  if ((b << 1) == 0) return 0x8000000000000000ull;
  return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}

struct WaveLds {
  uint64_t key[2 * kCandMax];   // candidates; behind them a place per lane for what is none
  int32_t id[kCandMax];
};

// A wave's experts: slot j of a lane.  VEC: four neighbours a load (E = 64 NJ).
template <bool VEC>
__device__ __forceinline__ int expert_of(int lane, int j) {
  return VEC ? 4 * lane + 256 * (j >> 2) + (j & 3) : lane + j * kWave;
}
template <bool VEC>
__device__ __forceinline__ int lane_of(int e) { return VEC ? (e >> 2) & (kWave - 1) : e & (kWave - 1); }
template <bool VEC>
__device__ __forceinline__ int slot_of(int e) { return VEC ? (e >> 8) * 4 + (e & 3) : e / kWave; }

__device__ __forceinline__ int mbcnt(uint64_t m) {
  return static_cast<int>(__builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(m >> 32),
                                                    __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(m), 0u)));
}

// The largest threshold (on the key's upper 18 bits) that at least k lanes'
// largest keys reach: a lower bound of the k-th largest key.  Nine bits of the
// fp32 mantissa are told apart, since scores crowd below 1.
template <int NJ>
__device__ __forceinline__ uint32_t kth_bound(const uint32_t (&key)[NJ], int k) {
  uint32_t lm = 0;
#pragma unroll
  for (int j = 0; j < NJ; ++j) lm = key[j] > lm ? key[j] : lm;
  uint32_t theta = 0;
#pragma unroll
  for (int b = 30; b >= 14; b -= 2) {
    const uint32_t c1 = theta | (1u << b), c2 = theta | (2u << b), c3 = theta | (3u << b);
    const int n1 = __popcll(__ballot(lm >= c1)), n2 = __popcll(__ballot(lm >= c2)), n3 = __popcll(__ballot(lm >= c3));
    theta = n3 >= k ? c3 : n2 >= k ? c2 : n1 >= k ? c1 : theta;
  }
  return theta;
}

// Candidates: entries with key >= theta >= 1 (key 0: no entry), ranked by (key,
// -id).  Returns their number; if at most 64, lane r < number holds the id and
// key of rank r.
template <int NJ, bool VEC>
__device__ __forceinline__ int rank32(const uint32_t (&key)[NJ], uint32_t theta, int lane, WaveLds* lds, int* id_out,
                                      uint32_t* key_out) {
  lds->key[lane] = 0;   // padding; a wave's LDS accesses land in order
  int cnt = 0;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const bool in = key[j] >= theta;
    const uint64_t m = __ballot(in);
    const int pos = cnt + mbcnt(m);
    // no branch: a lane without a candidate, and one past the 64th, writes to its own place behind them
    lds->key[in && pos < kCandMax ? pos : kCandMax + lane] =
        (static_cast<uint64_t>(key[j]) << 32) | static_cast<uint32_t>(~expert_of<VEC>(lane, j));
    cnt += __popcll(m);
  }
  if (cnt > kCandMax) return cnt;
  wave_sync_lds();
  const uint64_t mine = lds->key[lane];
  int rank = 0;
  for (int c = 0; c < cnt; c += 8) {
    uint64_t o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = lds->key[c + i];
#pragma unroll
    for (int i = 0; i < 8; ++i) rank += o[i] > mine ? 1 : 0;
  }
  // the candidates' ranks and the other lanes' own numbers are a permutation
  const int dst = 4 * (lane < cnt ? rank : lane);
  *id_out = __builtin_amdgcn_ds_permute(dst, static_cast<int>(~static_cast<uint32_t>(mine)));
  *key_out = static_cast<uint32_t>(__builtin_amdgcn_ds_permute(dst, static_cast<int>(mine >> 32)));
  wave_sync_lds();
  return cnt;
}

// The same on 64-bit keys, bounded by their 32-bit images: lane r < k returns
// the id of rank r.  More than 64 candidates (many equal keys) take k rounds
// of a wave arg-max.
template <int NJ, bool VEC>
__device__ __forceinline__ int topk64(const uint32_t (&key32)[NJ], const uint64_t (&key64)[NJ], int k, int lane,
                                      WaveLds* lds) {
  const uint32_t theta = kth_bound<NJ>(key32, k);
  int cnt = 0;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const bool in = key32[j] != 0u && key32[j] >= theta;
    const uint64_t m = __ballot(in);
    const int pos = cnt + mbcnt(m);
    if (in && pos < kCandMax) {
      lds->key[pos] = key64[j];
      lds->id[pos] = expert_of<VEC>(lane, j);
    }
    cnt += __popcll(m);
  }
  int myid = 0;
  if (cnt <= kCandMax) {
    wave_sync_lds();
    const uint64_t mine = lane < cnt ? lds->key[lane] : 0;
    const int id = lane < cnt ? lds->id[lane] : 0;
    int rank = 0;
    for (int c = 0; c < cnt; ++c) {
      const uint64_t o = lds->key[c];
      rank += (o > mine || (o == mine && lds->id[c] < id)) ? 1 : 0;
    }
    myid = __builtin_amdgcn_ds_permute(4 * (lane < cnt ? rank : lane), id);
    wave_sync_lds();
    return myid;
  }
  uint32_t taken = 0;
  for (int i = 0; i < k; ++i) {
    uint64_t best = 0;
    int bid = 0x7fffffff;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      if (!((taken >> j) & 1u) && key32[j] != 0u && key64[j] > best) {   // equal keys: the lower slot is the lower id
        best = key64[j];
        bid = expert_of<VEC>(lane, j);
      }
    }
#define ARGMAX(S)                                                                                            \
  {                                                                                                          \
    const uint64_t o = (static_cast<uint64_t>(lane_xor<S>(static_cast<uint32_t>(best >> 32), lane)) << 32) | \
                       lane_xor<S>(static_cast<uint32_t>(best), lane);                                       \
    const int oid = static_cast<int>(lane_xor<S>(static_cast<uint32_t>(bid), lane));                         \
    if (o > best || (o == best && oid < bid)) {                                                              \
      best = o;                                                                                              \
      bid = oid;                                                                                             \
    }                                                                                                        \
  }
    ARGMAX(1) ARGMAX(2) ARGMAX(4) ARGMAX(8) ARGMAX(16) ARGMAX(32)
#undef ARGMAX
    if (lane_of<VEC>(bid) == lane) taken |= 1u << slot_of<VEC>(bid);
    if (lane == i) myid = bid;
  }
  return myid;
}

__device__ __forceinline__ float second_of(float hi, float lo, float v) { return __builtin_amdgcn_fmed3f(hi, lo, v); }
__device__ __forceinline__ double second_of(double hi, double lo, double v) { return v > hi ? hi : (v > lo ? v : lo); }
// Of two numbers (no NaN comes here) in one instruction each, as the middle of
// three: fmaxf and fminf would first quiet both.
__device__ __forceinline__ float larger(float a, float b) { return __builtin_amdgcn_fmed3f(a, b, INFINITY); }
__device__ __forceinline__ double larger(double a, double b) { return a > b ? a : b; }
__device__ __forceinline__ float smaller(float a, float b) { return __builtin_amdgcn_fmed3f(a, b, -INFINITY); }
__device__ __forceinline__ double smaller(double a, double b) { return a < b ? a : b; }

template <int S>
__device__ __forceinline__ float lane_xor_f(float v, int lane) {
  return __uint_as_float(lane_xor<S>(__float_as_uint(v), lane));
}
template <int S>
__device__ __forceinline__ double lane_xor_f(double v, int lane) { return lane_xor_d<S>(v, lane); }

// The two largest of two lanes' two largest (lo <= hi).
template <int S, typename F>
__device__ __forceinline__ void merge_two(F& hi, F& lo, int lane) {
  const F oh = lane_xor_f<S>(hi, lane), ol = lane_xor_f<S>(lo, lane);
  lo = larger(smaller(hi, oh), larger(lo, ol));
  hi = larger(hi, oh);
}

// Scores of the groups from the experts' values in LDS (-inf: not counted).
// L lanes (64 over the power of two at or above G) share a group; all of them
// return its score, lanes of no group -inf.
template <typename F>
__device__ __forceinline__ F group_score(const F* val, const RouteArgs& a, int L, int lane) {
  typedef F F4 __attribute__((ext_vector_type(4)));
  const int g = lane / L;
  F hi = -INFINITY, lo = -INFINITY;
  const F* v = val + g * a.gsize;
  if (a.gsize % (4 * L) == 0) {
    if (g < a.G) {
      for (int x = 4 * (lane & (L - 1)); x < a.gsize; x += 4 * L) {
        const F4 w = *reinterpret_cast<const F4*>(v + x);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          lo = second_of(hi, lo, w[i]);
          hi = larger(hi, w[i]);
        }
      }
    }
  } else if (g < a.G) {
    for (int x = lane & (L - 1); x < a.gsize; x += L) {
      lo = second_of(hi, lo, v[x]);
      hi = larger(hi, v[x]);
    }
  }
  if (L > 1) merge_two<1>(hi, lo, lane);
  if (L > 2) merge_two<2>(hi, lo, lane);
  if (L > 4) merge_two<4>(hi, lo, lane);
  if (L > 8) merge_two<8>(hi, lo, lane);
  if (L > 16) merge_two<16>(hi, lo, lane);
  return a.gt == 2 && hi != -INFINITY && lo != -INFINITY ? hi + lo : hi;
}

__device__ __forceinline__ float readlane_f(float v, int l) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l));
}

__device__ __forceinline__ double readlane_f(double v, int l) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v));
  return dbl(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(b >> 32), l)),
             static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(b & 0xffffffffu), l)));
}

// 1 for the experts of the groups in `keep` (bit g L: group g), else 0.
template <int NJ, bool VEC>
__device__ __forceinline__ void mark_groups(uint64_t keep, const RouteArgs& a, int L, int lane, uint32_t (&mark)[NJ]) {
  const uint32_t n = static_cast<uint32_t>(a.E);
  const auto kept = [&](uint32_t e) { return e < n && ((keep >> (((e * a.ginv) >> 20) * L)) & 1ull) ? 1u : 0u; };
  if (VEC && (a.gsize & 3) == 0) {   // four neighbours are of one group
#pragma unroll
    for (int j = 0; j < NJ; j += 4)
      mark[j] = mark[j + 1] = mark[j + 2] = mark[j + 3] = kept(static_cast<uint32_t>(expert_of<VEC>(lane, j)));
  } else {
#pragma unroll
    for (int j = 0; j < NJ; ++j) mark[j] = kept(static_cast<uint32_t>(expert_of<VEC>(lane, j)));
  }
}

struct Chosen {
  int id;         // lane r < k: the id of rank r
  double denom;   // the softmax denominator
};

// The choice by double-precision scores.
template <int NJ, bool SIGMOID, bool VEC>
__device__ __forceinline__ Chosen choose_exact(const RouteArgs& a, const float (&l)[NJ], const float (&bias)[NJ], float mx,
                                               int L, int lane, WaveLds* lds, double* val) {
  Chosen c;
  double s[NJ], sum = 0.0;
  c.denom = 1.0;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const double x = static_cast<double>(l[j]);
    if (SIGMOID) s[j] = 1.0 / (1.0 + exp(-x));
    else s[j] = l[j] == -INFINITY ? 0.0 : exp(x - static_cast<double>(mx));
    sum += s[j];
  }
  if (!SIGMOID) {
    c.denom = wave_sum_d(sum, lane);
    if (c.denom == 0.0) c.denom = 1.0;   // a row whose mask leaves nothing
#pragma unroll
    for (int j = 0; j < NJ; ++j) s[j] /= c.denom;
  }
  uint32_t key32[NJ];
  uint64_t key64[NJ];
  if (a.G > 1) {
    wave_sync_lds();
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int e = expert_of<VEC>(lane, j);
      const double v = s[j] + static_cast<double>(bias[j]);
      if (e < a.E) val[e] = (l[j] == -INFINITY || v != v) ? -INFINITY : v;
    }
    wave_sync_lds();
    const double sc = group_score<double>(val, a, L, lane);
    const int g = lane / L;
    int rank = 0;   // among all groups, ties to the lower group
    for (int o = 0; o < a.G; ++o) {
      const double v = readlane_f(sc, o * L);
      rank += (v > sc || (v == sc && o < g)) ? 1 : 0;
    }
    mark_groups<NJ, VEC>(__ballot(g < a.G && rank < a.tg && (lane & (L - 1)) == 0), a, L, lane, key32);
    wave_sync_lds();
  } else {
#pragma unroll
    for (int j = 0; j < NJ; ++j) key32[j] = expert_of<VEC>(lane, j) < a.E ? 1u : 0u;
  }
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    double key = a.bias ? s[j] + static_cast<double>(bias[j]) : static_cast<double>(l[j]);
    if (l[j] == -INFINITY || key != key) key = -INFINITY;
    key64[j] = order_key64(key);
    key32[j] = key32[j] ? order_key(static_cast<float>(key)) : 0u;   // order_key is never 0 for a number
  }
  c.id = topk64<NJ, VEC>(key32, key64, a.k, lane, lds);
  return c;
}

// The same choice from fp32 scores, where it is certain.  With u = 2^-24:
//   sigmoid   exp2 of a rounded product, a sum and a reciprocal of 1 ulp each
//             leave |error of s| <= (0.45 + 0.5 + 1 + 2) u < 8 u
//   softmax   a term exp(d) <= 1 is off by exp(d) (2 |d| + 2) u <= 3 u; the
//             denominator D, whose terms are off by 2 |d| + 2 u and whose mean
//             |d| is at most the entropy, 6.94, by (14 + 2 + 16 + 6) u of
//             itself, the quotient by 3 u of itself; |error of s| <= (3 + 41) u
//             / D < 64 u / D
// and a bias adds a rounding of u |v|; `eps` is that bound.  A group's score is
// off by 2 eps + u |sum| at most.  Groups: one that stays has fewer than
// top_groups others that may lie above it, one that goes at least that many
// that do, by more than twice the bound.  Experts: every entry within 2 eps of
// the bound on the k-th largest is a candidate, and neighbours among the first
// k + 1 have to differ by more than 2 eps (a logit is exact), or the candidates
// are ranked by double precision.
// Returns false where it is not certain (groups within the bound, more than 64
// candidates).
template <int NJ, int DT, bool SIGMOID, bool VEC>
__device__ __forceinline__ bool choose_fast(const RouteArgs& a, int64_t row, const float (&l)[NJ], const float (&bias)[NJ],
                                            float mx, int L, int lane, WaveLds* lds, float* val, int* id) {
  constexpr float kLog2e = 1.4426950408889634f, u = 5.9604644775390625e-8f;
  float v[NJ], eps = 8.f * u;
  if (SIGMOID) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) v[j] = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-l[j] * kLog2e));
  } else {
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      v[j] = l[j] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((l[j] - mx) * kLog2e);
      sum += v[j];
    }
#define STEP(S) sum += lane_xor_f<S>(sum, lane)
    STEP(1); STEP(2); STEP(4); STEP(8); STEP(16); STEP(32);
#undef STEP
    const float r = __builtin_amdgcn_rcpf(sum);
#pragma unroll
    for (int j = 0; j < NJ; ++j) v[j] *= r;
    eps = 64.f * u * r;
  }
  // the largest magnitude as whole numbers: infinities and NaN come out on top
  uint32_t top = 0;
  uint64_t empty = ~0ull;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const bool out = l[j] == -INFINITY;
    const float x = v[j] + bias[j];
    const uint32_t m = __float_as_uint(x) & 0x7fffffffu;
    top = m > top ? m : top;
    empty &= __ballot(out);
    v[j] = out ? -INFINITY : x;
  }
  if (empty == ~0ull) {   // the mask leaves nothing: all keys are equal, the lowest ids stay
    *id = lane;
    return true;
  }
  // most values lie below 1 or 4; others take an exchange
  float big = 1.f;
  if (__ballot(top >= 0x3f800000u)) {
    big = 4.f;
    if (__ballot(top >= 0x40800000u)) {
      big = wave_max_f(__uint_as_float(top), lane);   // passes NaN over, which is not below itself
      if (__ballot(!(__uint_as_float(top) < 1e30f))) return false;
    }
  }
  eps += 2.f * u * big;
  uint32_t key[NJ];
  if (a.G > 1) {
    if (VEC) {
      typedef float f32x4 __attribute__((ext_vector_type(4)));
#pragma unroll
      for (int j = 0; j < NJ; j += 4) *reinterpret_cast<f32x4*>(val + expert_of<VEC>(lane, j)) = f32x4{v[j], v[j + 1], v[j + 2], v[j + 3]};
    } else {
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        if (expert_of<VEC>(lane, j) < a.E) val[expert_of<VEC>(lane, j)] = v[j];
    }
    wave_sync_lds();
    const float sc = group_score<float>(val, a, L, lane);
    const float margin = 4.f * eps + 8.f * u * big, low = sc - margin, high = sc + margin;
    int maybe = -1, surely = 0;   // the group itself lies above low
    for (int o = 0; o < a.G; ++o) {
      const float x = readlane_f(sc, o * L);
      maybe += x > low ? 1 : 0;
      surely += x > high ? 1 : 0;
    }
    if (sc == -INFINITY) maybe = 64;
    const bool real = lane / L < a.G;
    if (__ballot(real && maybe >= a.tg && surely < a.tg)) return false;
    mark_groups<NJ, VEC>(__ballot(real && maybe < a.tg && (lane & (L - 1)) == 0), a, L, lane, key);
  } else {
#pragma unroll
    for (int j = 0; j < NJ; ++j) key[j] = VEC || expert_of<VEC>(lane, j) < a.E ? 1u : 0u;
  }
  const bool by_score = a.bias != nullptr;
  const auto key_of = [](float x) {   // order_key of a number that is not -0
    const uint32_t b = __float_as_uint(x);
    return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
  };
  // a NaN logit has not come this far: its magnitude was refused above
  if (by_score) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) key[j] = key[j] ? key_of(v[j]) : 0u;   // a score is not -0, nor is its sum with a bias
  } else {
#pragma unroll
    for (int j = 0; j < NJ; ++j) key[j] = key[j] ? key_of(l[j] + 0.f) : 0u;
  }
  const uint32_t theta = kth_bound<NJ>(key, a.k);
  uint32_t from = theta > 1u ? theta : 1u;
  if (by_score) {
    if (theta < 0x00800000u) from = 1u;   // below every number's key
    else from = order_key(key_float(theta) - 2.5f * eps);
  }
  uint32_t mykey = 0;
  const int cnt = rank32<NJ, VEC>(key, from, lane, lds, id, &mykey);
  if (cnt > kCandMax) return false;
  if (!by_score) return true;
  const float mine = key_float(mykey), below = __shfl_down(mine, 1);
  const bool sure = lane >= a.k || lane + 1 >= cnt || mine - below > 2.f * eps;
  if (__ballot(!sure) == 0) return true;
  if (!SIGMOID) return false;
  // the candidates hold the first k for certain
  double exact = -INFINITY;
  if (lane < cnt) {
    const float x = load_scalar<DT>(a.logits, static_cast<size_t>(row + *id));
    if (x != -INFINITY) exact = 1.0 / (1.0 + exp(-static_cast<double>(x))) + static_cast<double>(a.bias[*id]);
  }
  int rank = lane < cnt ? 0 : lane;
  for (int o = 0; o < cnt; ++o) {
    const double v = readlane_f(exact, o);
    const int i = __builtin_amdgcn_readlane(*id, o);
    if (lane < cnt) rank += v > exact || (v == exact && i < *id) ? 1 : 0;
  }
  *id = __builtin_amdgcn_ds_permute(4 * rank, *id);
  return true;
}

// One token's logits on the wave.
template <int NJ, int DT, bool VEC>
__device__ __forceinline__ void load_row(const RouteArgs& a, int64_t t, int lane, float (&l)[NJ]) {
  const int64_t row = t * a.stride;
  if constexpr (VEC) {
#pragma unroll
    for (int j = 0; j < NJ; j += 4) {
      const int64_t at = row + expert_of<VEC>(lane, j);
      if constexpr (DT == kF32) {
        const float4 w = *reinterpret_cast<const float4*>(static_cast<const float*>(a.logits) + at);
        l[j] = w.x; l[j + 1] = w.y; l[j + 2] = w.z; l[j + 3] = w.w;
      } else {
        const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.logits) + at);
        l[j] = __uint_as_float(w.x << 16);
        l[j + 1] = __uint_as_float(w.x & 0xffff0000u);
        l[j + 2] = __uint_as_float(w.y << 16);
        l[j + 3] = __uint_as_float(w.y & 0xffff0000u);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int e = lane + j * kWave;
      l[j] = e < a.E ? load_scalar<DT>(a.logits, static_cast<size_t>(row + e)) : -INFINITY;
    }
  }
}

// The row's largest logit, NaN if one is: then every score of a softmax is NaN,
// also where the NaN is not chosen.
template <int NJ>
__device__ __forceinline__ float row_max(const float (&l)[NJ], int lane) {
  float m = l[0];
#pragma unroll
  for (int j = 1; j < NJ; ++j) m = __builtin_elementwise_maximum(m, l[j]);
#define STEP(S) m = __builtin_elementwise_maximum(m, lane_xor_f<S>(m, lane))
  STEP(1); STEP(2); STEP(4); STEP(8); STEP(16); STEP(32);
#undef STEP
  return m;
}

// NJ: logits per lane (E <= 64 NJ).  WIDE: experts or groups are compared by
// scores (a bias or groups).  VEC: E = 64 NJ and aligned rows.
// Bound by the instructions of a token's wave: 32768 tokens of 512 bf16 logits
// in 8 groups (sigmoid) take 31 us, six times the time of reading them; 16384
// of 512 fp32 logits with a softmax, bias and groups 23.7 us renormalised, 31.5
// with the exact denominator, with a bias alone 17.5; one token of 256 takes
// 3.6 us, 2048 of 512 without groups 4.5 us, both little over a launch.
// The double-precision weights of a block's four tokens are one wave's work
// (33.4 against 35.0 us at that point).  Several tokens per wave throughout,
// sharing the bias too, were slower (four 62, eight 65, sixteen 87 us against
// one's 59): fewer waves hide less of each other's exchanges.
template <int NJ, int DT, bool SIGMOID, bool WIDE, bool VEC>
__global__ __launch_bounds__(kRtWaves* kWave) void k_route(RouteArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ WaveLds wave_lds[kRtWaves];
  __shared__ int32_t chosen[kRtWaves][kWave / kRtWaves];
  __shared__ float maxima[kRtWaves];
  __shared__ double denoms[kRtWaves];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  int64_t t = static_cast<int64_t>(blockIdx.x) * kRtWaves + wave;
  float mx = 0.f;
  Chosen c{0, 1.0};
  if (t < a.T) {
    WaveLds* lds = &wave_lds[wave];

    float l[NJ];
    load_row<NJ, DT, VEC>(a, t, lane, l);
    if (!SIGMOID) mx = row_max<NJ>(l, lane);
    if constexpr (WIDE) {
      double* val = reinterpret_cast<double*>(smem) + static_cast<size_t>(wave) * a.E;
      float bias[NJ] = {};
      if (a.bias) {
        if constexpr (VEC) {
#pragma unroll
          for (int j = 0; j < NJ; j += 4) __builtin_memcpy(bias + j, a.bias + expert_of<VEC>(lane, j), 16);
        } else {
#pragma unroll
          for (int j = 0; j < NJ; ++j) bias[j] = lane + j * kWave < a.E ? a.bias[lane + j * kWave] : 0.f;
        }
      }
      int L = kWave;   // lanes per group
      while (L * a.G > kWave) L >>= 1;
      if (!choose_fast<NJ, DT, SIGMOID, VEC>(a, t * a.stride, l, bias, mx, L, lane, lds, reinterpret_cast<float*>(val), &c.id)) {
        c = choose_exact<NJ, SIGMOID, VEC>(a, l, bias, mx, L, lane, lds, val);
        if (!SIGMOID && c.denom != c.denom) mx = NAN;   // +inf (choose_fast leaves such rows), chosen or not
      } else if (!SIGMOID && !a.renorm) {
        double sum = 0.0;
#pragma unroll
        for (int j = 0; j < NJ; ++j) sum += l[j] == -INFINITY ? 0.0 : exp(static_cast<double>(l[j]) - static_cast<double>(mx));
        c.denom = wave_sum_d(sum, lane);
        if (c.denom == 0.0) c.denom = 1.0;
      }
  } else {
      if (!SIGMOID && !a.renorm) {
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < NJ; ++j) sum += l[j] == -INFINITY ? 0.f : expf(l[j] - mx);
        c.denom = wave_sum_d(static_cast<double>(sum), lane);
        if (c.denom == 0.0) c.denom = 1.0;
      }
      uint32_t key[NJ];
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        key[j] = VEC || lane + j * kWave < a.E ? order_key(l[j] != l[j] ? -INFINITY : l[j]) : 0u;
      const uint32_t theta = kth_bound<NJ>(key, a.k);
      bool empty = false;   // no number in the row: the lowest ids stay
      if (theta < 0x00800000u) {
        uint64_t numbers = 0;
#pragma unroll
        for (int j = 0; j < NJ; ++j) numbers |= __ballot(key[j] >= 0x00800000u);
        empty = numbers == 0;
      }
      uint32_t mykey = 0;
      if (empty) {
        c.id = lane;
      } else if (rank32<NJ, VEC>(key, theta > 1u ? theta : 1u, lane, lds, &c.id, &mykey) > kCandMax) {
        uint64_t key64[NJ];
#pragma unroll
        for (int j = 0; j < NJ; ++j) key64[j] = key[j];
        c.id = topk64<NJ, VEC>(key, key64, a.k, lane, lds);
      }
    }
  }

  // weights of the chosen, in double precision (one exp per lane): up to 16 of
  // each of the block's tokens by one wave, not the same in neighbouring blocks
  int rank = lane;
  if (a.k <= kWave / kRtWaves) {
    if (lane < a.k) chosen[wave][lane] = c.id;
    if (lane == 0) { maxima[wave] = mx; denoms[wave] = c.denom; }
    __syncthreads();
    if (wave != static_cast<int>((blockIdx.x >> 3) & 3)) return;
    const int part = lane / (kWave / kRtWaves);
    rank = lane % (kWave / kRtWaves);
    t = static_cast<int64_t>(blockIdx.x) * kRtWaves + part;
    c.id = chosen[part][rank];
    mx = maxima[part];
    c.denom = denoms[part];
  }
  const bool on = rank < a.k && t < a.T;
  const float lc = on ? load_scalar<DT>(a.logits, static_cast<size_t>(t * a.stride + c.id)) : -INFINITY;
  double sc = 0.0;
  if (on && (lc != -INFINITY || (!SIGMOID && mx != mx))) {
    if (SIGMOID) sc = 1.0 / (1.0 + exp(-static_cast<double>(lc)));
    else sc = exp(static_cast<double>(lc) - static_cast<double>(mx));
  }
  if (a.renorm) {
    double sum = sc;
    sum += lane_xor_d<1>(sum, lane);
    sum += lane_xor_d<2>(sum, lane);
    sum += lane_xor_d<4>(sum, lane);
    sum += lane_xor_d<8>(sum, lane);
    if (a.k > 16) {
      sum += lane_xor_d<16>(sum, lane);
      sum += lane_xor_d<32>(sum, lane);
    }
    sc = sum == 0.0 ? 0.0 : sc / sum;
  } else if (!SIGMOID) {
    sc /= c.denom;
  }
  if (on) {
    a.ids[t * a.k + rank] = c.id;
    a.w[t * a.k + rank] = static_cast<float>(sc * static_cast<double>(a.scale));
  }
}

template <int NJ, int DT, bool SIGMOID, bool WIDE, bool VEC>
void launch_route(const RouteArgs& a, hipStream_t s) {
  const uint32_t lds = WIDE && a.G > 1 ? kRtWaves * static_cast<uint32_t>(a.E) * 8u : 0u;
  const dim3 grid(static_cast<uint32_t>((a.T + kRtWaves - 1) / kRtWaves)), block(kRtWaves * kWave);
  launch_kernel(k_route<NJ, DT, SIGMOID, WIDE, VEC>, grid, block, lds, s, a);
}

template <int NJ, int DT, bool SIGMOID>
void launch_route_wide(const RouteArgs& a, bool wide, hipStream_t s) {
  constexpr uintptr_t kAlign = DT == kF32 ? 16 : 8;
  const bool vec = a.E == 64 * NJ && a.stride % 4 == 0 && (reinterpret_cast<uintptr_t>(a.logits) & (kAlign - 1)) == 0;
  if (wide && vec) launch_route<NJ, DT, SIGMOID, true, true>(a, s);
  else if (wide) launch_route<NJ, DT, SIGMOID, true, false>(a, s);
  else if (vec) launch_route<NJ, DT, SIGMOID, false, true>(a, s);
  else launch_route<NJ, DT, SIGMOID, false, false>(a, s);
}

template <int DT, bool SIGMOID>
void launch_route_size(const RouteArgs& a, bool wide, hipStream_t s) {
  if (a.E <= 4 * kWave) launch_route_wide<4, DT, SIGMOID>(a, wide, s);
  else if (a.E <= 8 * kWave) launch_route_wide<8, DT, SIGMOID>(a, wide, s);
  else launch_route_wide<16, DT, SIGMOID>(a, wide, s);
}

template <int DT>
void launch_route_dt(const RouteArgs& a, bool sigmoid, bool wide, hipStream_t s) {
  if (sigmoid) launch_route_size<DT, true>(a, wide, s);
  else launch_route_size<DT, false>(a, wide, s);
}

int bad(const char* fmt, long long x = 0, long long y = 0) {
  char buf[256];
  snprintf(buf, sizeof(buf), fmt, x, y);
  return api_fail(MOE_EINVAL, buf);
}

bool overlaps(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
  return a && b && na > 0 && nb > 0 && pa < pb + static_cast<uintptr_t>(nb) && pb < pa + static_cast<uintptr_t>(na);
}

bool at(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace

int check_route(const moe_route_desc* r) {
  if (!r) return bad("routing descriptor is NULL");
  if (r->n_experts < 1 || r->n_experts > kMaxExperts) return bad("n_experts=%lld must be in [1, 1024]", r->n_experts);
  if (r->n_groups < 1 || r->n_groups > 64 || r->n_experts % r->n_groups)
    return bad("n_groups=%lld must be in [1, 64] and divide n_experts=%lld", r->n_groups, r->n_experts);
  if (r->top_groups < 1 || r->top_groups > r->n_groups)
    return bad("top_groups=%lld must be in [1, n_groups=%lld]", r->top_groups, r->n_groups);
  if (r->top_k < 1 || r->top_k > 64 || r->top_k > r->top_groups * (r->n_experts / r->n_groups))
    return bad("top_k=%lld must be in [1, 64] and at most the %lld experts of the groups that stay", r->top_k,
               r->top_groups * static_cast<long long>(r->n_experts / r->n_groups));
  if (r->score != MOE_SCORE_SOFTMAX && r->score != MOE_SCORE_SIGMOID) return bad("score=%lld is not a MOE_SCORE_* code", r->score);
  if (r->group_top != 1 && r->group_top != 2) return bad("group_top=%lld must be 1 or 2", r->group_top);
  if (r->renormalize != 0 && r->renormalize != 1) return bad("renormalize=%lld must be 0 or 1", r->renormalize);
  if (r->logit_dtype != MOE_F32 && r->logit_dtype != MOE_BF16)
    return bad("logit_dtype=%lld is neither MOE_F32 nor MOE_BF16", r->logit_dtype);
  if (!std::isfinite(r->scale)) return bad("scale must be finite");
  return MOE_OK;
}

int route_forward(const moe_route_desc* r, int32_t T, const void* logits, int64_t stride, const float* bias,
                  int32_t* ids, float* w, hipStream_t s) {
  RouteArgs a{};
  a.logits = logits;
  a.bias = bias;
  a.ids = ids;
  a.w = w;
  a.stride = stride;
  a.T = T;
  a.E = r->n_experts;
  a.k = r->top_k;
  a.G = r->n_groups;
  a.tg = r->top_groups;
  a.gt = r->group_top;
  a.renorm = r->renormalize;
  a.gsize = a.E / a.G;
  a.ginv = ((1u << 20) + a.gsize - 1) / a.gsize;
  a.scale = r->scale;
  // all groups staying is no choice of groups
  if (a.tg == a.G) a.G = 1;
  const bool sigmoid = r->score == MOE_SCORE_SIGMOID, wide = bias != nullptr || a.G > 1;
  if (r->logit_dtype == MOE_F32) launch_route_dt<kF32>(a, sigmoid, wide, s);
  else launch_route_dt<kBF16>(a, sigmoid, wide, s);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) {
    char buf[256];
    snprintf(buf, sizeof(buf), "routing launch failed: %s", hipGetErrorString(e));
    return api_fail(MOE_EHIP, buf);
  }
  return api_ok();
}

int check_route_out(const moe_route_desc* r, int32_t T, const float* bias, const int32_t* ids, const float* w) {
  if (!ids || !w) return bad("NULL topk_ids or topk_w");
  if (!at(ids, 4) || !at(w, 4) || !at(bias, 4)) return bad("bias, topk_ids and topk_w must be 4-byte aligned");
  const int64_t n_o = static_cast<int64_t>(T) * r->top_k * 4, n_b = static_cast<int64_t>(r->n_experts) * 4;
  if (overlaps(ids, n_o, w, n_o) || overlaps(ids, n_o, bias, n_b) || overlaps(w, n_o, bias, n_b))
    return bad("topk_ids and topk_w overlap each other or the bias");
  return MOE_OK;
}

}  // namespace moe

extern "C" int moe_route_forward(const moe_route_desc* r, int32_t T, const void* logits, int64_t logits_stride,
                                 const float* bias, int32_t* topk_ids, float* topk_w, void* stream) {
  using namespace moe;
  MarkScope marks;
  int rc;
  if ((rc = check_route(r))) return rc;
  if (T < 0 || T > (1 << 20)) return bad("T=%lld must be in [0, 2^20]", T);
  if (T == 0) return api_ok();
  if (T > 1 && (logits_stride < r->n_experts || logits_stride > (int64_t(1) << 40)))
    return bad("logits_stride=%lld is smaller than n_experts=%lld or too large", logits_stride, r->n_experts);
  if (!logits) return bad("NULL logits");
  const int64_t sz = r->logit_dtype == MOE_F32 ? 4 : 2;
  if (!at(logits, sz)) return bad("logits must be aligned to their type's %lld bytes", sz);
  if ((rc = check_route_out(r, T, bias, topk_ids, topk_w))) return rc;
  const int64_t n_l = ((T - 1) * logits_stride + r->n_experts) * sz, n_o = static_cast<int64_t>(T) * r->top_k * 4;
  if (overlaps(topk_ids, n_o, logits, n_l) || overlaps(topk_w, n_o, logits, n_l))
    return bad("topk_ids or topk_w overlaps the logits");
  return route_forward(r, T, logits, T > 1 ? logits_stride : 0, bias, topk_ids, topk_w, static_cast<hipStream_t>(stream));
}
