// Norms of the query and key heads, position rotation, and the append of k and
// v to the paged cache (include/attention.h), in one pass (gfx950).
//
// A head is 16 bytes a lane: L = head_dim * size / 16 lanes, so a wave takes
// 64 / L heads of one token at once, a group.  The norm is one sum of squares over
// L lanes; the partner of a rotated pair is in the same lane (adjacent pairs) or
// read again from the row, which the load before has brought to the cache.  The
// angles of a token are formed once by the wave, a pair a lane, and handed out
// through LDS; with the weights of the norm they make two factors a value.
//
// A prompt is bound by memory and by its instructions, about 1000 a token for place
// and angles and 130 a group (16384 tokens of 16 + 2 heads of 256: 100 us, 3.3 TB/s
// of the copy's 4.7; fp32 heads of 128 without norms 6.2 TB/s, part of it in the
// last-level cache).  A token takes 4.7 us, two trips to memory after each other.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdio>
#include <type_traits>

#include "attn_internal.h"
#include "moe_internal.h"
#include "topk_wave.h"

namespace moe {
namespace {

struct AppendArgs {
  AttnBatch at;
  const int32_t* positions;
  const void* q;
  const void* k;
  const void* v;
  int64_t qs, ks, vs;
  const float* qw;
  const float* kw;
  const float* inv_freq;
  void* q_out;
  void* pages;
  int nq, nkv, R, adjacent;
  int per_wave;         // groups of 64 / L heads that a wave takes
  float eps, offset;
};

template <int L>
__device__ __forceinline__ float lanes_sum(float x, int lane) {
  if constexpr (L > 1) x += __uint_as_float(lane_xor<1>(__float_as_uint(x), lane));
  if constexpr (L > 2) x += __uint_as_float(lane_xor<2>(__float_as_uint(x), lane));
  if constexpr (L > 4) x += __uint_as_float(lane_xor<4>(__float_as_uint(x), lane));
  if constexpr (L > 8) x += __uint_as_float(lane_xor<8>(__float_as_uint(x), lane));
  if constexpr (L > 16) x += __uint_as_float(lane_xor<16>(__float_as_uint(x), lane));
  if constexpr (L > 32) x += __uint_as_float(lane_xor<32>(__float_as_uint(x), lane));
  return x;
}

// 1 / sqrt(x) by the instruction, within one unit in the last place; it takes
// denormals for zero, so small x are brought up.
__device__ __forceinline__ float inverse_root(float x) {
  const bool small = x < 0x1p-96f;
  return __builtin_amdgcn_rsqf(small ? x * 0x1p64f : x) * (small ? 0x1p32f : 1.f);
}

// The sequence of row t, with the number of the row's token in it; false if it
// has none.  64 entries of cu a step, in equal distances until 64 are left.
__device__ __forceinline__ bool find_sequence(const AttnBatch& at, int t, int lane, int& b, int64_t& number) {
  int lo = 0, n = at.B;
  while (n > kWave) {
    const int step = (n + kWave - 1) / kWave, j = lane * step;
    const int hits = __popcll(__ballot(j < n && at.cu[lo + (j < n ? j : 0)] <= t));
    if (hits == 0) return false;
    lo += (hits - 1) * step;
    n = n - (hits - 1) * step < step ? n - (hits - 1) * step : step;
  }
  const int j = lo + (lane < n ? lane : n - 1);
  const int begin = at.cu[j], end = at.cu[j + 1], len = at.lens[j];
  const uint64_t hit = __ballot(lane < n && begin <= t && t < end);
  if (hit == 0) return false;
  const int first = __builtin_ctzll(hit);
  b = lo + first;
  number = static_cast<int64_t>(__builtin_amdgcn_readlane(len, first)) - __builtin_amdgcn_readlane(end, first) + t;
  return true;
}

template <int DT, int V>
__device__ __forceinline__ void unpack(const u32x4& w, float (&x)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if constexpr (DT == kF32) x[i] = __uint_as_float(w[i]);
    else x[i] = __uint_as_float((i & 1) ? (w[i / 2] & 0xffff0000u) : (w[i / 2] << 16));
  }
}

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

template <int DT, int V>
__device__ __forceinline__ u32x4 pack(const float (&x)[V]) {
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == kF32) w[i] = __float_as_uint(x[i]);
    else w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{x[2 * i], x[2 * i + 1]}), bf16x2));
  }
  return w;
}

template <int DT, int D>
__global__ __launch_bounds__(256) void k_attn_append(AppendArgs a) {
  constexpr int V = DT == kF32 ? 4 : 8;      // values a lane
  constexpr int L = D / V;                   // lanes a head
  constexpr int H = kWave / L;               // heads a group
  constexpr int G = 4;                       // groups requested at once
  constexpr int kSize = DT == kF32 ? 4 : 2;
  __shared__ __align__(16) float turns[4][2][D];   // by wave: cosines and sines, the sign of the pair's first on the sine
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int nq = a.q ? a.nq : 0;
  const int qgroups = (nq + H - 1) / H, groups = qgroups + (2 * a.nkv + H - 1) / H;
  const int waves = (groups + a.per_wave - 1) / a.per_wave;      // per token
  const uint32_t w = blockIdx.x * 4 + wave;
  const int t = static_cast<int>(w / waves);
  if (t >= a.at.N) return;
  const int first = static_cast<int>(w % waves) * a.per_wave, last = first + a.per_wave < groups ? first + a.per_wave : groups;

  const int sub = lane / L, e0 = (lane % L) * V;                 // this lane's values of a head
  const int half = a.R / 2;
  const bool turned = e0 < a.R, apart = turned && !a.adjacent;
  u32x4 raw[G], other[G];
  const uint8_t* src[G];
  // Groups g0 .. of those up to `to`: heads of q, or of k and then v.
  const auto request = [&](auto kind, int g0, int to) {
    constexpr bool IS_Q = decltype(kind)::value;
    const int base = IS_Q ? 0 : qgroups, heads = IS_Q ? nq : 2 * a.nkv;
#pragma unroll
    for (int y = 0; y < G; ++y) {
      int head = (g0 + y < to ? g0 + y - base : to - 1 - base) * H + sub;
      head = head < heads ? head : heads - 1;
      const bool is_v = !IS_Q && head >= a.nkv;
      const int64_t row = static_cast<int64_t>(t) * (IS_Q ? a.qs : (is_v ? a.vs : a.ks));
      src[y] = static_cast<const uint8_t*>(IS_Q ? a.q : (is_v ? a.v : a.k)) + (row + static_cast<int64_t>(is_v ? head - a.nkv : head) * D) * kSize;
      raw[y] = load16(src[y] + e0 * kSize);
      if (apart && half % V == 0) other[y] = load16(src[y] + (e0 < half ? e0 + half : e0 - half) * kSize);
    }
  };
  if (first < qgroups) request(std::true_type{}, first, last < qgroups ? last : qgroups);
  else request(std::false_type{}, first, last);

  int b;
  int64_t number;
  if (!find_sequence(a.at, t, lane, b, number)) return;
  int64_t page = -1;
  if (number >= 0 && (number >> a.at.shift) < a.at.max_pages)
    page = a.at.table[static_cast<int64_t>(b) * a.at.max_pages + (number >> a.at.shift)];
  const bool kept = page >= 0 && page < a.at.n_pages;
  const int64_t place = number & ((1 << a.at.shift) - 1);

  float* const cosines = turns[wave][0];
  float* const sines = turns[wave][1];
  for (int p = lane; p < half; p += kWave) {
    // turns, reduced to [-1/2, 1/2] before the step down to fp32
    const double whole = static_cast<double>(a.positions[t]) * (static_cast<double>(a.inv_freq[p]) * 0.15915494309189535);
    float sn, cs;
    sincospif(2.f * static_cast<float>(whole - rint(whole)), &sn, &cs);
    const int i = a.adjacent ? 2 * p : p, j = a.adjacent ? 2 * p + 1 : p + half;
    cosines[i] = cosines[j] = cs;
    sines[i] = -sn;                          // first of a pair: x cos - partner sin; second: x cos + partner sin
    sines[j] = sn;
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  const auto partner = [&](int e) { return a.adjacent ? e ^ 1 : (e < half ? e + half : e - half); };

  const auto take = [&](auto kind, int from, int to) {
    constexpr bool IS_Q = decltype(kind)::value;
    const int base = IS_Q ? 0 : qgroups, heads = IS_Q ? nq : 2 * a.nkv;
    const float* const wt = IS_Q ? a.qw : a.kw;
    float c[V], s[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = e0 + i;
      c[i] = e < a.R ? cosines[e] : 1.f;
      s[i] = e < a.R ? sines[e] : 0.f;
      if (wt) {
        c[i] *= a.offset + wt[e];
        if (e < a.R) s[i] *= a.offset + wt[partner(e)];
      }
    }
    for (int g0 = from; g0 < to; g0 += G) {
      if (g0 > first) request(kind, g0, to);
#pragma unroll
      for (int y = 0; y < G; ++y) {
        const int head = (g0 + y - base) * H + sub;
        if (g0 + y >= to || head >= heads) continue;
        const bool is_v = !IS_Q && head >= a.nkv;
        if (!is_v && (wt || turned)) {
          float x[V], z[V], r = 1.f;
          unpack<DT, V>(raw[y], x);
          if (wt) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i) ss = fmaf(x[i], x[i], ss);
            ss = lanes_sum<L>(ss, lane);
            r = inverse_root(fmaf(ss, 1.0f / D, a.eps));
#pragma unroll
            for (int i = 0; i < V; ++i) x[i] *= r;
          }
          if (turned) {
            if (!apart) {
#pragma unroll
              for (int i = 0; i < V; ++i) z[i] = x[i ^ 1];
            } else {
              if (half % V == 0) {
                unpack<DT, V>(other[y], z);
              } else {
#pragma unroll
                for (int i = 0; i < V; ++i) z[i] = load_scalar<DT>(src[y], e0 + i < a.R ? partner(e0 + i) : e0 + i);
              }
#pragma unroll
              for (int i = 0; i < V; ++i) z[i] *= r;
            }
          }
#pragma unroll
          for (int i = 0; i < V; ++i) {
            x[i] *= c[i];
            if (e0 + i < a.R) x[i] = fmaf(z[i], s[i], x[i]);
          }
          raw[y] = pack<DT, V>(x);
        }
        uint8_t* to_row;
        if (IS_Q) {
          to_row = static_cast<uint8_t*>(a.q_out) + (static_cast<int64_t>(t) * nq + head) * D * kSize;
        } else {
          if (!kept) continue;
          to_row = static_cast<uint8_t*>(a.pages) + (page * a.at.page_elems + (is_v ? a.at.half_elems : 0) +
                   ((static_cast<int64_t>(is_v ? head - a.nkv : head) << a.at.shift) + place) * D) * kSize;
        }
        *reinterpret_cast<u32x4*>(to_row + e0 * kSize) = raw[y];
      }
    }
  };
  if (first < qgroups) take(std::true_type{}, first, last < qgroups ? last : qgroups);
  if (last > qgroups) take(std::false_type{}, first > qgroups ? first : qgroups, last);
}

// Groups that a wave takes: one for few tokens, so that as many loads as can be
// are under way at once, and with more of them as many as leave ten waves a CU,
// so that a token's place and angles are formed less often.  Microseconds with
// 1, 2, 5 and 10 groups a wave, 16 + 2 heads of 256: a token 4.8, 5.3, 9.0, 12.0;
// 512 tokens 12.8, 9.0, 10.4, 13.4; 1024 21, 14.6, 12.9, 14.1; 4096 73, 43, 34, 27.
int append_per_wave(int groups, int N) {
  const int64_t v = (static_cast<int64_t>(groups) * N + 2559) / 2560;
  return v < groups ? static_cast<int>(v) : groups;
}

template <int DT>
void launch_append(AppendArgs a, int D, hipStream_t s) {
  const int V = DT == kF32 ? 4 : 8, H = kWave / (D / V);
  const int groups = ((a.q ? a.nq : 0) + H - 1) / H + (2 * a.nkv + H - 1) / H;
  a.per_wave = append_per_wave(groups, a.at.N);
  const int64_t waves = static_cast<int64_t>((groups + a.per_wave - 1) / a.per_wave) * a.at.N;
  const dim3 grid(static_cast<uint32_t>((waves + 3) / 4));
  if (D == 64) launch_kernel(k_attn_append<DT, 64>, grid, dim3(256), 0, s, a);
  else if (D == 128) launch_kernel(k_attn_append<DT, 128>, grid, dim3(256), 0, s, a);
  else launch_kernel(k_attn_append<DT, 256>, grid, dim3(256), 0, s, a);
}

}  // namespace

int attn_bad(const char* fmt, long long x, long long y) {
  char buf[256];
  snprintf(buf, sizeof(buf), fmt, x, y);
  return api_fail(MOE_EINVAL, buf);
}

int check_attn(const attn_desc* d) {
  if (!d) return attn_bad("attention descriptor is NULL");
  if (d->n_kv_heads < 1 || d->n_q_heads < 1 || d->n_q_heads > 256 || d->n_q_heads % d->n_kv_heads)
    return attn_bad("n_q_heads=%lld must be in [1, 256] and a multiple of n_kv_heads=%lld", d->n_q_heads, d->n_kv_heads);
  if (d->head_dim != 64 && d->head_dim != 128 && d->head_dim != 256)
    return attn_bad("head_dim=%lld must be 64, 128 or 256", d->head_dim);
  if (d->dtype != MOE_F32 && d->dtype != MOE_BF16) return attn_bad("dtype=%lld is neither MOE_F32 nor MOE_BF16", d->dtype);
  if (d->page_size < 1 || d->page_size > 1024 || (d->page_size & (d->page_size - 1)))
    return attn_bad("page_size=%lld must be a power of two in [1, 1024]", d->page_size);
  if (d->max_pages < 1 || d->max_pages > (1 << 24)) return attn_bad("max_pages=%lld must be in [1, 2^24]", d->max_pages);
  if (d->rotary_dim < 0 || d->rotary_dim > d->head_dim || d->rotary_dim % 2)
    return attn_bad("rotary_dim=%lld must be even and in [0, head_dim=%lld]", d->rotary_dim, d->head_dim);
  if (d->rotary_pairs != ATTN_ROTARY_HALF && d->rotary_pairs != ATTN_ROTARY_ADJACENT)
    return attn_bad("rotary_pairs=%lld is not an ATTN_ROTARY_* code", d->rotary_pairs);
  if (d->n_pages < 1 || d->n_pages > 0x7fffffffLL) return attn_bad("n_pages=%lld must be in [1, 2^31)", d->n_pages);
  if (!std::isfinite(d->scale)) return attn_bad("scale must be finite");
  if (!(d->eps >= 0.f) || !std::isfinite(d->eps)) return attn_bad("eps must be finite and >= 0");
  if (!std::isfinite(d->norm_offset)) return attn_bad("norm_offset must be finite");
  return MOE_OK;
}

int check_attn_batch(int32_t B, int32_t N, const int32_t* cu, const int32_t* lens, const int32_t* table) {
  if (!cu || !lens || !table) return attn_bad("NULL cu, lens or table");
  if (!attn_aligned(cu, 4) || !attn_aligned(lens, 4) || !attn_aligned(table, 4))
    return attn_bad("cu, lens and table must be 4-byte aligned");
  return MOE_OK;
}

}  // namespace moe

extern "C" int attn_append(const attn_desc* d, int32_t B, int32_t N, const int32_t* cu, const int32_t* lens,
                           const int32_t* table, const int32_t* positions, const void* q, int64_t q_stride,
                           const void* k, int64_t k_stride, const void* v, int64_t v_stride, const float* q_norm,
                           const float* k_norm, const float* inv_freq, void* q_out, void* pages, void* stream) {
  using namespace moe;
  MarkScope marks;
  int rc;
  if ((rc = check_attn(d))) return rc;
  if (B < 0 || B > (1 << 16) || N < 0 || N > (1 << 20)) return attn_bad("B=%lld must be in [0, 2^16], N=%lld in [0, 2^20]", B, N);
  if (B == 0 || N == 0) return api_ok();
  if ((rc = check_attn_batch(B, N, cu, lens, table))) return rc;
  if (!k || !v || !pages) return attn_bad("NULL k, v or pages");
  if (!q != !q_out) return attn_bad("q and q_out are given together or not at all");
  if (d->rotary_dim > 0 && (!positions || !inv_freq)) return attn_bad("positions and inv_freq are needed for rotary_dim=%lld", d->rotary_dim);
  const int64_t sz = d->dtype == MOE_F32 ? 4 : 2, D = d->head_dim;
  const int64_t nqD = d->n_q_heads * D, nkD = d->n_kv_heads * D;
  const int64_t most = int64_t(1) << 32;
  if (q && (q_stride < nqD || q_stride > most || q_stride * sz % 16))
    return attn_bad("q_stride=%lld must be at least %lld elements and a multiple of 16 bytes", q_stride, nqD);
  if (k_stride < nkD || k_stride > most || k_stride * sz % 16 || v_stride < nkD || v_stride > most || v_stride * sz % 16)
    return attn_bad("k_stride=%lld and v_stride=%lld must hold a row and be multiples of 16 bytes", k_stride, v_stride);
  if (!attn_aligned(q, 16) || !attn_aligned(k, 16) || !attn_aligned(v, 16) || !attn_aligned(q_out, 16) || !attn_aligned(pages, 16))
    return attn_bad("q, k, v, q_out and pages must be 16-byte aligned");
  if (!attn_aligned(positions, 4) || !attn_aligned(q_norm, 4) || !attn_aligned(k_norm, 4) || !attn_aligned(inv_freq, 4))
    return attn_bad("positions, norms and inv_freq must be 4-byte aligned");
  const AttnBatch at = attn_batch(d, B, N, cu, lens, table);
  const int64_t n_pages = d->n_pages * at.page_elems * sz, n_qo = q ? N * nqD * sz : 0;
  const void* ins[] = {q, k, v, cu, lens, table, positions, q_norm, k_norm, inv_freq};
  const int64_t in_n[] = {((N - 1) * q_stride + nqD) * sz, ((N - 1) * k_stride + nkD) * sz, ((N - 1) * v_stride + nkD) * sz,
                          (B + 1) * int64_t(4), B * int64_t(4), static_cast<int64_t>(B) * d->max_pages * 4, N * int64_t(4),
                          D * 4, D * 4, d->rotary_dim * int64_t(2)};
  for (int i = 0; i < 10; ++i)
    if (attn_overlaps(pages, n_pages, ins[i], in_n[i]) || attn_overlaps(q_out, n_qo, ins[i], in_n[i]))
      return attn_bad("pages or q_out overlaps input %lld", i);
  if (attn_overlaps(pages, n_pages, q_out, n_qo)) return attn_bad("pages and q_out overlap");

  AppendArgs a{};
  a.at = at;
  a.positions = positions;
  a.q = q; a.k = k; a.v = v;
  a.qs = q_stride; a.ks = k_stride; a.vs = v_stride;
  a.qw = q_norm; a.kw = k_norm;
  a.inv_freq = inv_freq;
  a.q_out = q_out;
  a.pages = pages;
  a.nq = d->n_q_heads; a.nkv = d->n_kv_heads;
  a.R = d->rotary_dim;
  a.adjacent = d->rotary_pairs == ATTN_ROTARY_ADJACENT;
  a.eps = d->eps;
  a.offset = d->norm_offset;
  if (d->dtype == MOE_F32) launch_append<kF32>(a, d->head_dim, static_cast<hipStream_t>(stream));
  else launch_append<kBF16>(a, d->head_dim, static_cast<hipStream_t>(stream));
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) {
    char buf[256];
    snprintf(buf, sizeof(buf), "append launch failed: %s", hipGetErrorString(e));
    return api_fail(MOE_EHIP, buf);
  }
  return api_ok();
}
