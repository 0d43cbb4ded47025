// Norms of the query and key heads, position rotation, and the append of k and
// v to the paged cache (include/attention.h), in one pass (gfx950).
//
// A head is 16 bytes a lane: L = head_dim * size / 16 lanes, so a wave takes
// 64 / L heads of one token at once.  The norm is one sum of squares over L
// lanes; the partner of a rotated pair is in the same lane (adjacent pairs) or
// read again from the row, which the load before has brought to the cache.
// Angles are formed once per lane and used for all heads that the wave takes.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdio>

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

// Number of entries of cu[0 .. B] that are at most t, less one: the last
// sequence that begins at or before row t (-1: none).  All lanes, 64 entries a
// step.
__device__ __forceinline__ int sequence_of(const int32_t* cu, int B, int t, int lane) {
  int n = 0;
  for (int i = 0; i <= B; i += kWave) {
    const int j = i + lane;
    n += __popcll(__ballot(j <= B && cu[j] <= t));
  }
  return n - 1;
}

template <int DT, int V>
__device__ __forceinline__ void unpack(const u32x4& w, float (&x)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if constexpr (DT == kF32) x[i] = __uint_as_float(w[i]);
    else x[i] = __uint_as_float((i & 1) ? (w[i / 2] & 0xffff0000u) : (w[i / 2] << 16));
  }
}

template <int DT, int V>
__device__ __forceinline__ u32x4 pack(const float (&x)[V]) {
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == kF32) w[i] = __float_as_uint(x[i]);
    else w[i] = f32_to_bf16(x[2 * i]) | (static_cast<uint32_t>(f32_to_bf16(x[2 * i + 1])) << 16);
  }
  return w;
}

template <int DT, int D>
__global__ __launch_bounds__(256) void k_attn_append(AppendArgs a) {
  constexpr int V = DT == kF32 ? 4 : 8;      // values a lane
  constexpr int L = D / V;                   // lanes a head
  constexpr int H = kWave / L;               // heads a wave takes at once
  constexpr int kSize = DT == kF32 ? 4 : 2;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = threadIdx.x / kWave;
  const int heads = (a.q ? a.nq : 0) + 2 * a.nkv;
  const int groups = (heads + H - 1) / H;
  const int waves = (groups + a.per_wave - 1) / a.per_wave;      // per token
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + wave;
  const int t = static_cast<int>(w / waves);
  if (t >= a.at.N) return;
  const int first = static_cast<int>(w % waves) * a.per_wave;

  const int b = sequence_of(a.at.cu, a.at.B, t, lane);
  if (b < 0 || b >= a.at.B) return;          // a row of no sequence
  const int begin = a.at.cu[b], end = a.at.cu[b + 1];
  const int64_t number = static_cast<int64_t>(a.at.lens[b]) - end + t;
  int64_t page = -1;
  if (number >= 0 && (number >> a.at.shift) < a.at.max_pages)
    page = a.at.table[static_cast<int64_t>(b) * a.at.max_pages + (number >> a.at.shift)];
  const bool kept = page >= 0 && page < a.at.n_pages;
  const int64_t place = number & ((1 << a.at.shift) - 1);

  const int sub = lane / L;
  const int e0 = (lane % L) * V;             // this lane's values of a head
  const bool turned = e0 < a.R;
  float cs[V], sn[V];
  if (turned) {
    const double pos = a.positions[t];
    const int half = a.R / 2;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = e0 + i;
      const int pair = a.adjacent ? e / 2 : (e < half ? e : e - half);
      const bool second = a.adjacent ? (i & 1) != 0 : e >= half;
      float c = 1.f, s = 0.f;
      if (a.adjacent && second) {
        c = cs[i - 1];
        s = -sn[i - 1];
      } else if (e < a.R) {
        // turns, reduced to [-1/2, 1/2] before the step down to fp32
        const double turns = pos * (static_cast<double>(a.inv_freq[pair]) * 0.15915494309189535);
        sincospif(2.f * static_cast<float>(turns - rint(turns)), &s, &c);
      }
      cs[i] = c;
      sn[i] = second ? s : -s;               // first of a pair: x cos - partner sin; second: x cos + partner sin
    }
  }

  for (int gidx = first; gidx < first + a.per_wave && gidx < groups; ++gidx) {
    const int head = gidx * H + sub;         // queries, then keys, then values
    if (head >= heads) continue;
    const int nq = heads - 2 * a.nkv;
    const bool is_q = head < nq, is_v = head >= nq + a.nkv;
    const int h = is_q ? head : (is_v ? head - nq - a.nkv : head - nq);
    const uint8_t* src = static_cast<const uint8_t*>(is_q ? a.q : (is_v ? a.v : a.k)) +
                         (static_cast<int64_t>(t) * (is_q ? a.qs : (is_v ? a.vs : a.ks)) + static_cast<int64_t>(h) * D) * kSize;
    u32x4 raw = *reinterpret_cast<const u32x4*>(src + e0 * kSize);
    if (!is_v) {
      float x[V], y[V];
      unpack<DT, V>(raw, x);
      const bool apart = turned && !a.adjacent;
      const int half = a.R / 2;
      if (apart) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int e = e0 + i;
          const int p = e < half ? e + half : (e < a.R ? e - half : e);
          y[i] = load_scalar<DT>(src, p);
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) y[i] = x[i ^ 1];
      }
      const float* wt = is_q ? a.qw : a.kw;
      if (wt) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) ss = fmaf(x[i], x[i], ss);
        ss = lanes_sum<L>(ss, lane);
        const float r = 1.0f / sqrtf(ss * (1.0f / D) + a.eps);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int e = e0 + i;
          const int p = apart ? (e < half ? e + half : (e < a.R ? e - half : e)) : (e0 + (i ^ 1));
          x[i] = x[i] * r * (a.offset + wt[e]);
          y[i] = y[i] * r * (a.offset + wt[p]);
        }
      }
      if (turned) {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (e0 + i < a.R) x[i] = fmaf(x[i], cs[i], y[i] * sn[i]);
      }
      raw = pack<DT, V>(x);
    }
    if (is_q) {
      *reinterpret_cast<u32x4*>(static_cast<uint8_t*>(a.q_out) + ((static_cast<int64_t>(t) * a.nq + h) * D + e0) * kSize) = raw;
    } else if (kept) {
      const int64_t o = page * a.at.page_elems + (is_v ? a.at.half_elems : 0) +
                        ((static_cast<int64_t>(h) << a.at.shift) + place) * D + e0;
      *reinterpret_cast<u32x4*>(static_cast<uint8_t*>(a.pages) + o * kSize) = raw;
    }
  }
}

template <int DT>
void launch_append(const AppendArgs& a, int D, hipStream_t s) {
  const int V = DT == kF32 ? 4 : 8, H = kWave / (D / V);
  const int heads = (a.q ? a.nq : 0) + 2 * a.nkv, groups = (heads + H - 1) / H;
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
  // one group of heads a wave: the most waves for few tokens; more where a
  // launch would need 2^32 threads
  const int per_group = kWave / static_cast<int>(D * sz / 16), heads = (q ? d->n_q_heads : 0) + 2 * d->n_kv_heads;
  const int64_t groups = (heads + per_group - 1) / per_group;
  a.per_wave = static_cast<int>((groups * N + (1 << 25) - 1) >> 25);
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
