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
// keys that matter lie further apart than the bound, and only the other tokens
// (a group or a neighbour within 2^-18 or so) go through double precision.
//
// Organisation.  A token's E logits are spread over one wave, lane l holding
// experts l, l + 64, ... (coalesced loads), nothing crosses waves, and a
// block is four independent tokens.
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
  uint64_t key[kCandMax];
  int32_t id[kCandMax];
};

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

// Candidates: entries with key >= theta (key 0: no entry), ranked by (key,
// -id).  Returns their number; if at most 64, lane r < number holds the id and
// key of rank r.
template <int NJ>
__device__ __forceinline__ int rank32(const uint32_t (&key)[NJ], uint32_t theta, int lane, WaveLds* lds, int* id_out,
                                      uint32_t* key_out) {
  lds->key[lane] = 0;   // padding; a wave's LDS accesses land in order
  int cnt = 0;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const bool in = key[j] != 0u && key[j] >= theta;
    const uint64_t m = __ballot(in);
    const int pos = cnt + mbcnt(m);
    if (in && pos < kCandMax) lds->key[pos] = (static_cast<uint64_t>(key[j]) << 32) | static_cast<uint32_t>(~(lane + j * kWave));
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
template <int NJ>
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
      lds->id[pos] = lane + j * kWave;
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
      if (!((taken >> j) & 1u) && key32[j] != 0u && key64[j] > best) {
        best = key64[j];
        bid = lane + j * kWave;
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
    if ((bid & (kWave - 1)) == lane) taken |= 1u << (bid / kWave);
    if (lane == i) myid = bid;
  }
  return myid;
}

// Scores of the groups from the experts' values in LDS (-inf: not counted).
// L lanes (64 over the power of two at or above G) share a group; all of them
// return its score, lanes of no group -inf.
template <typename F>
__device__ __forceinline__ F group_score(const F* val, const RouteArgs& a, int L, int lane) {
  const int g = lane / L;
  F hi = -INFINITY, lo = -INFINITY;
  if (g < a.G) {
    for (int x = lane & (L - 1); x < a.gsize; x += L) {
      const F v = val[g * a.gsize + x];
      lo = v > hi ? hi : (v > lo ? v : lo);
      hi = v > hi ? v : hi;
    }
  }
  for (int st = 1; st < L; st <<= 1) {
    const F oh = __shfl_xor(hi, st), ol = __shfl_xor(lo, st);
    const F mid = oh > hi ? hi : oh;       // the smaller of the two largest
    const F second = oh > hi ? ol : lo;    // the second of the side with the larger first
    hi = oh > hi ? oh : hi;
    lo = mid > second ? mid : second;
  }
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

// Rank of this lane's group among all, ties to the lower group.
template <typename F>
__device__ __forceinline__ int group_rank(F sc, const RouteArgs& a, int L, int lane) {
  const int g = lane / L;
  int rank = 0;
  for (int o = 0; o < a.G; ++o) {
    const F v = readlane_f(sc, o * L);
    rank += (v > sc || (v == sc && o < g)) ? 1 : 0;
  }
  return rank;
}

// 1 for the experts of the groups in `keep` (bit g L: group g), else 0.
template <int NJ>
__device__ __forceinline__ void mark_groups(uint64_t keep, const RouteArgs& a, int L, int lane, uint32_t (&mark)[NJ]) {
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const uint32_t e = static_cast<uint32_t>(lane + j * kWave), n = static_cast<uint32_t>(a.E);
    const uint32_t g = e < n ? (e * a.ginv) >> 20 : 0u;
    mark[j] = e < n && ((keep >> (g * L)) & 1ull) ? 1u : 0u;
  }
}

// The choice by double-precision scores.  Lane r < k returns the id of rank r;
// *denom_out: the softmax denominator.
template <int NJ, bool SIGMOID>
__device__ __forceinline__ int choose_exact(const RouteArgs& a, const float (&l)[NJ], const float (&bias)[NJ], float mx,
                                         int lane, WaveLds* lds, double* val, double* denom_out) {
  double s[NJ], sum = 0.0, denom = 1.0;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const double x = static_cast<double>(l[j]);
    if (SIGMOID) s[j] = 1.0 / (1.0 + exp(-x));
    else s[j] = l[j] == -INFINITY ? 0.0 : exp(x - static_cast<double>(mx));
    sum += s[j];
  }
  if (!SIGMOID) {
    denom = wave_sum_d(sum, lane);
    if (denom == 0.0) denom = 1.0;   // a row whose mask leaves nothing
#pragma unroll
    for (int j = 0; j < NJ; ++j) s[j] /= denom;
  }
  *denom_out = denom;
  uint32_t key32[NJ];
  uint64_t key64[NJ];
  if (a.G > 1) {
    wave_sync_lds();
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int e = lane + j * kWave;
      const double v = s[j] + static_cast<double>(bias[j]);
      if (e < a.E) val[e] = (l[j] == -INFINITY || v != v) ? -INFINITY : v;
    }
    wave_sync_lds();
    int L = kWave;
    while (L * a.G > kWave) L >>= 1;
    const double sc = group_score<double>(val, a, L, lane);
    const int rank = group_rank<double>(sc, a, L, lane);
    mark_groups<NJ>(__ballot(lane / L < a.G && rank < a.tg && (lane & (L - 1)) == 0), a, L, lane, key32);
  } else {
#pragma unroll
    for (int j = 0; j < NJ; ++j) key32[j] = lane + j * kWave < a.E ? 1u : 0u;
  }
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    double key = a.bias ? s[j] + static_cast<double>(bias[j]) : static_cast<double>(l[j]);
    if (l[j] == -INFINITY || key != key) key = -INFINITY;
    key64[j] = order_key64(key);
    key32[j] = key32[j] ? order_key(static_cast<float>(key)) : 0u;   // order_key is never 0 for a number
  }
  return topk64<NJ>(key32, key64, a.k, lane, lds);
}

// The same choice from fp32 scores, where it is certain.  With u = 2^-24:
//   sigmoid   exp2 of a rounded product, a sum and a reciprocal of 1 ulp each
//             leave |error of s| <= (0.23 + 1 + 1 + 2) u < 8 u
//   softmax   a term exp(d) <= 1 is off by exp(d) (2 |d| + 2) u <= 3 u; the
//             denominator, whose terms are off by 2 |d| + 2 u and whose mean
//             |d| is at most the entropy, 6.94, by (14 + 2 + 16 + 6) u of
//             itself; |error of s| < 64 u
// and a bias adds a rounding of u |v|; `eps` is that bound.  A group's score is
// off by 2 eps + u |sum| at most.  Groups: the worst that stays has to lead the
// best that goes by more than twice the bound.  Experts: every entry within
// 2 eps of the bound on the k-th largest is a candidate, and neighbours among
// the first k + 1 have to differ by more than 2 eps (a logit is exact).
// Returns false where it is not certain (equal keys, empty groups).
template <int NJ, bool SIGMOID>
__device__ __forceinline__ bool choose_fast(const RouteArgs& a, const float (&l)[NJ], const float (&bias)[NJ], float mx,
                                            int lane, WaveLds* lds, float* val, int* id) {
  constexpr float kLog2e = 1.4426950408889634f, u = 5.9604644775390625e-8f;
  float v[NJ], big = 0.f;
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
#define STEP(S) sum += __uint_as_float(lane_xor<S>(__float_as_uint(sum), lane))
    STEP(1); STEP(2); STEP(4); STEP(8); STEP(16); STEP(32);
#undef STEP
    const float r = __builtin_amdgcn_rcpf(sum);
#pragma unroll
    for (int j = 0; j < NJ; ++j) v[j] *= r;
  }
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    v[j] = l[j] == -INFINITY ? -INFINITY : v[j] + bias[j];
    if (v[j] != v[j]) big = INFINITY;
    else if (v[j] != -INFINITY) big = fmaxf(big, fabsf(v[j]));
  }
  big = wave_max_f(big, lane);
  if (!(big < 1e30f)) return false;
  const float eps = (SIGMOID ? 8.f : 64.f) * u + 2.f * u * big;
  uint32_t key[NJ];
  if (a.G > 1) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int e = lane + j * kWave;
      if (e < a.E) val[e] = v[j];
    }
    wave_sync_lds();
    int L = kWave;
    while (L * a.G > kWave) L >>= 1;
    const float sc = group_score<float>(val, a, L, lane);
    const int rank = group_rank<float>(sc, a, L, lane);
    const bool real = lane / L < a.G;
    const float lead = -wave_max_f(real && rank < a.tg ? -sc : -INFINITY, lane);
    const float next = wave_max_f(real && rank >= a.tg ? sc : -INFINITY, lane);
    if (!(lead - next > 4.f * eps + 8.f * u * big)) return false;
    mark_groups<NJ>(__ballot(real && rank < a.tg && (lane & (L - 1)) == 0), a, L, lane, key);
  } else {
#pragma unroll
    for (int j = 0; j < NJ; ++j) key[j] = lane + j * kWave < a.E ? 1u : 0u;
  }
  const bool by_score = a.bias != nullptr;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const float x = by_score || l[j] != l[j] ? v[j] : l[j];
    key[j] = key[j] ? order_key(x) : 0u;
  }
  const uint32_t theta = kth_bound<NJ>(key, a.k);
  uint32_t from = theta > 1u ? theta : 1u;
  if (by_score) {
    if (theta < 0x00800000u) from = 1u;   // below every number's key
    else from = order_key(key_float(theta) - 2.5f * eps);
  }
  uint32_t mykey = 0;
  const int cnt = rank32<NJ>(key, from, lane, lds, id, &mykey);
  if (cnt > kCandMax) return false;
  if (!by_score) return true;
  const float mine = key_float(mykey), below = __shfl_down(mine, 1);
  const bool sure = lane >= a.k || lane + 1 >= cnt || mine - below > 2.f * eps;
  return __ballot(!sure) == 0;
}

// NJ: logits per lane (E <= 64 NJ).  WIDE: experts or groups are compared by
// scores (a bias or groups).
template <int NJ, int DT, bool SIGMOID, bool WIDE>
__global__ __launch_bounds__(kRtWaves* kWave) void k_route(RouteArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = threadIdx.x / kWave;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kRtWaves + wave;
  if (t >= a.T) return;   // no barrier below: waves are independent
  WaveLds* lds = reinterpret_cast<WaveLds*>(smem) + wave;
  double* val = reinterpret_cast<double*>(smem + kRtWaves * sizeof(WaveLds)) + static_cast<size_t>(wave) * (WIDE ? a.E : 0);

  const int64_t row = t * a.stride;
  float l[NJ];
  float bias[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int e = lane + j * kWave;
    l[j] = e < a.E ? load_scalar<DT>(a.logits, static_cast<size_t>(row + e)) : -INFINITY;
    bias[j] = (WIDE && a.bias && e < a.E) ? a.bias[e] : 0.f;
  }
  float mx = l[0];   // fmaxf passes NaN over
#pragma unroll
  for (int j = 1; j < NJ; ++j) mx = fmaxf(mx, l[j]);
  mx = wave_max_f(mx, lane);

  int id = 0;
  double denom = 1.0;   // of a softmax that is not divided out again
  if constexpr (WIDE) {
    const bool sum_too = !SIGMOID && !a.renorm;
    if (sum_too || !choose_fast<NJ, SIGMOID>(a, l, bias, mx, lane, lds, reinterpret_cast<float*>(val), &id))
      id = choose_exact<NJ, SIGMOID>(a, l, bias, mx, lane, lds, val, &denom);
  } else {
    if (!SIGMOID && !a.renorm) {
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < NJ; ++j) sum += l[j] == -INFINITY ? 0.f : expf(l[j] - mx);
      denom = wave_sum_d(static_cast<double>(sum), lane);
      if (denom == 0.0) denom = 1.0;
    }
    uint32_t key[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      key[j] = lane + j * kWave < a.E ? order_key(l[j] != l[j] ? -INFINITY : l[j]) : 0u;
    const uint32_t theta = kth_bound<NJ>(key, a.k);
    uint32_t mykey = 0;
    if (rank32<NJ>(key, theta, lane, lds, &id, &mykey) > kCandMax) {
      uint64_t key64[NJ];
#pragma unroll
      for (int j = 0; j < NJ; ++j) key64[j] = key[j];
      id = topk64<NJ>(key, key64, a.k, lane, lds);
    }
  }

  // weights of the chosen, in double precision (one exp per lane)
  const bool on = lane < a.k;
  const float lc = on ? load_scalar<DT>(a.logits, static_cast<size_t>(row + id)) : -INFINITY;
  double sc = 0.0;
  if (on && lc != -INFINITY) {
    if (SIGMOID) sc = 1.0 / (1.0 + exp(-static_cast<double>(lc)));
    else sc = exp(static_cast<double>(lc) - static_cast<double>(mx));
  }
  if (a.renorm) {
    const double sum = wave_sum_d(sc, lane);
    sc = sum == 0.0 ? 0.0 : sc / sum;
  } else if (!SIGMOID) {
    sc /= denom;
  }
  if (on) {
    a.ids[t * a.k + lane] = id;
    a.w[t * a.k + lane] = static_cast<float>(sc * static_cast<double>(a.scale));
  }
}

template <int NJ, int DT, bool SIGMOID>
void launch_route_wide(const RouteArgs& a, bool wide, dim3 grid, dim3 block, hipStream_t s) {
  const uint32_t lds = kRtWaves * (sizeof(WaveLds) + (wide && a.G > 1 ? static_cast<uint32_t>(a.E) * 8u : 0u));
  if (wide) launch_kernel(k_route<NJ, DT, SIGMOID, true>, grid, block, lds, s, a);
  else launch_kernel(k_route<NJ, DT, SIGMOID, false>, grid, block, lds, s, a);
}

template <int NJ, int DT>
void launch_route_score(const RouteArgs& a, bool sigmoid, bool wide, dim3 grid, dim3 block, hipStream_t s) {
  if (sigmoid) launch_route_wide<NJ, DT, true>(a, wide, grid, block, s);
  else launch_route_wide<NJ, DT, false>(a, wide, grid, block, s);
}

template <int DT>
void launch_route_dt(const RouteArgs& a, bool sigmoid, bool wide, dim3 grid, dim3 block, hipStream_t s) {
  if (a.E <= 4 * kWave) launch_route_score<4, DT>(a, sigmoid, wide, grid, block, s);
  else if (a.E <= 8 * kWave) launch_route_score<8, DT>(a, sigmoid, wide, grid, block, s);
  else launch_route_score<16, DT>(a, sigmoid, wide, grid, block, s);
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
  const dim3 grid(static_cast<uint32_t>((T + kRtWaves - 1) / kRtWaves)), block(kRtWaves * kWave);
  if (r->logit_dtype == MOE_F32) launch_route_dt<kF32>(a, sigmoid, wide, grid, block, s);
  else launch_route_dt<kBF16>(a, sigmoid, wide, grid, block, s);
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
