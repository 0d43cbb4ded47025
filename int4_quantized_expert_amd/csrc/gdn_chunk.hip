// Gated delta rule over prompts in chunks of 64 tokens (include/gdn_chunk.h, gfx950).
//
// Two kernels.  k_gdc_prep forms, for every chunk and value head at once, what
// does not depend on the state: with A and P as in the header, T = (I + A)^-1,
//   Z-matrix  diag(w) T diag(beta),  w_i = D_Ci / |k_i|
//   O-matrix  P T diag(beta)
// and the row factors e_i = g_i / |k_i|, f_i = g_i scale / |q_i|.  k_gdc_scan
// then walks the chunks of a sequence with 16 rows of a head's state on chip:
//   X = V - diag(e) K S^T,  O = diag(f) Q S^T + (O-matrix) X,
//   Zt = (Z-matrix) X,      S <- g_C S + Zt^T K
// with K and Q as they are stored (their norms are in the factors).
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdio>

#include "device_common.h"
#include "gdn_chunk.h"
#include "moe_internal.h"
#include "topk_wave.h"

namespace moe {
namespace {

constexpr int kC = 64;                        // tokens a chunk
constexpr int kRowsS = 16;                    // state rows a block
constexpr int64_t kPassBytes = int64_t(256) << 20;   // workspace a pass may take
typedef float f32x4 __attribute__((ext_vector_type(4)));

// One chunk and value head in the workspace.
constexpr int kSlotMat = kC * kC;             // floats of each matrix
constexpr int kSlotVec = 4 * kC;              // e, f, then g_C and whether the chunk runs token by token
constexpr int kSlotFloats = 2 * kSlotMat + kSlotVec;

struct GdcArgs {
  const int32_t* cu;
  const void* q;
  const void* k;
  const void* v;
  const float* alpha;
  const float* beta;
  const float* state_in;
  float* state_out;
  void* out;
  float* ws;
  int B, N, T_max;
  int nk, nv, dv;
  int first;            // first chunk of this pass in every sequence
  int per_pass;         // chunks a pass and sequence; 0: all of them, packed
  int slots;
  float scale, eps;
};

__device__ __forceinline__ void sequence(const GdcArgs& a, int b, int& begin, int& n) {
  const int s = a.cu[b], e = a.cu[b + 1];
  begin = s;
  n = s >= 0 && e <= a.N && e > s ? e - s : 0;
  if (n > a.T_max) n = a.T_max;
}

// Slot of chunk c of a sequence that begins at row `begin`.  Packed: chunks of
// sequence b come after begin / 64 + b, which leaves room for those before it.
__device__ __forceinline__ int64_t slot_of(const GdcArgs& a, int b, int begin, int c) {
  return a.per_pass ? static_cast<int64_t>(b) * a.per_pass + (c - a.first) : static_cast<int64_t>(begin / kC) + b + c;
}

// Four values of a row from element c on, as fp32.
template <int ACT>
__device__ __forceinline__ f32x4 load4(const void* base, int64_t c) {
  if constexpr (ACT == kF32) {
    return *reinterpret_cast<const f32x4*>(static_cast<const float*>(base) + c);
  } else {
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + c);
    return f32x4{__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                 __uint_as_float(w.y & 0xffff0000u)};
  }
}

__device__ __forceinline__ float xor16_add(float x, int lane) {
  x = x + __uint_as_float(lane_xor<16>(__float_as_uint(x), lane));
  return x + __uint_as_float(lane_xor<32>(__float_as_uint(x), lane));
}

__device__ __forceinline__ bool finite4(const f32x4& v) {
  return isfinite(v[0]) && isfinite(v[1]) && isfinite(v[2]) && isfinite(v[3]);
}

template <int DK, int ACT>
__global__ __launch_bounds__(256) void k_gdc_prep(GdcArgs a) {
  constexpr int KS = DK / 16;
  constexpr int kLd = kC + 4;
  __shared__ __align__(16) float As[kC * kLd];
  __shared__ __align__(16) float Ts[kC * kLd];   // its blocks on and below the diagonal
  __shared__ __align__(16) float Ps[kC * kLd];
  __shared__ float rk[kC], rq[kC], be[kC];
  __shared__ double Lg[kC];
  __shared__ int odd;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), w = tid / kWave;
  const int n16 = lane & 15, g = lane >> 4;
  const int slot = blockIdx.x / a.nv, h = blockIdx.x % a.nv, kh = h / (a.nv / a.nk);

  // the sequence and chunk of this slot
  int b;
  if (a.per_pass) {
    b = slot / a.per_pass;
  } else {
    int cnt = 0;
    for (int i = 0; i < a.B; i += kWave) {
      const int j = i + lane;
      cnt += __popcll(__ballot(j < a.B && a.cu[j] / kC + j <= slot));
    }
    b = cnt - 1;
  }
  if (b < 0 || b >= a.B) return;
  int begin, n;
  sequence(a, b, begin, n);
  const int c = a.per_pass ? a.first + slot % a.per_pass : slot - begin / kC - b;
  if (c < 0 || static_cast<int64_t>(c) * kC >= n) return;
  const int t0 = c * kC;
  const int len = n - t0 < kC ? n - t0 : kC;
  const int64_t row0 = static_cast<int64_t>(begin) + t0;

  if (tid == 0) odd = 0;
  __syncthreads();
  if (w == 0) {                                // gates: logarithms summed in double precision
    const bool in = lane < len;
    const float al = in ? a.alpha[(row0 + lane) * a.nv + h] : 1.f;
    const float bt = in ? a.beta[(row0 + lane) * a.nv + h] : 0.f;
    if (!(al >= 9.5367431640625e-7f && al <= 1.f && bt >= 0.f && bt <= 2.f)) odd = 1;
    double s = static_cast<double>(log2f(al));
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const double o = __shfl_up(s, d);
      if (lane >= d) s += o;
    }
    Lg[lane] = s;
    be[lane] = bt;
  }

  // K K^T and Q K^T, the lower blocks; rows of tile w, columns of tiles up to w
  const int64_t st = static_cast<int64_t>(a.nk) * DK;
  const bool live = 16 * w + n16 < len;
  const int64_t mine = (row0 + (live ? 16 * w + n16 : 0)) * st + static_cast<int64_t>(kh) * DK;
  f32x4 Ka[KS], Qa[KS];
  float sk = 0.f, sq = 0.f;
  bool fine = true;
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    Ka[s] = load4<ACT>(a.k, mine + 16 * s + 4 * g);
    Qa[s] = load4<ACT>(a.q, mine + 16 * s + 4 * g);
    if (!live) Ka[s] = Qa[s] = f32x4{0.f, 0.f, 0.f, 0.f};
    fine = fine && finite4(Ka[s]) && finite4(Qa[s]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sk = fmaf(Ka[s][i], Ka[s][i], sk);
      sq = fmaf(Qa[s][i], Qa[s][i], sq);
    }
  }
  for (int i = tid; i < len * (a.dv / 4); i += 256) {
    const f32x4 v = load4<ACT>(a.v, ((row0 + i / (a.dv / 4)) * a.nv + h) * static_cast<int64_t>(a.dv) + (i % (a.dv / 4)) * 4);
    fine = fine && finite4(v);
  }
  sk = xor16_add(sk, lane);
  sq = xor16_add(sq, lane);
  const float rkv = 1.0f / sqrtf(sk + a.eps), rqv = a.scale / sqrtf(sq + a.eps);
  if (!fine || (live && !(isfinite(rkv) && isfinite(rqv) && isfinite(sk) && isfinite(sq)))) odd = 1;
  if (g == 0) {
    rk[16 * w + n16] = live ? rkv : 0.f;
    rq[16 * w + n16] = live ? rqv : 0.f;
  }
  f32x4 G[4], H[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    G[j] = H[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (j > w) continue;
    const bool lj = 16 * j + n16 < len;
    const int64_t at = (row0 + (lj ? 16 * j + n16 : 0)) * st + static_cast<int64_t>(kh) * DK;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      f32x4 Kb = load4<ACT>(a.k, at + 16 * s + 4 * g);
      if (!lj) Kb = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        G[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(Ka[s][i], Kb[i], G[j], 0, 0, 0);
        H[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(Qa[s][i], Kb[i], H[j], 0, 0, 0);
      }
    }
  }
  __syncthreads();
  float* slot_p = a.ws + (static_cast<int64_t>(slot) * a.nv + h) * kSlotFloats;
  if (odd) {
    if (tid == 0) slot_p[2 * kSlotMat + 2 * kC + 1] = 1.f;
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int i = 16 * w + 4 * g + r, jj = 16 * j + n16;
      const float D = i >= jj ? exp2f(static_cast<float>(Lg[i] - Lg[jj])) : 0.f;
      As[i * kLd + jj] = i > jj ? be[i] * D * rk[i] * rk[jj] * G[j][r] : 0.f;
      Ps[i * kLd + jj] = D * rq[i] * rk[jj] * H[j][r];
    }
  __syncthreads();
  // T = (I + A)^-1: the diagonal blocks by substitution, a column a lane ...
  {
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s = i == n16 ? 1.f : 0.f;
#pragma unroll
      for (int l = 0; l < i; ++l) s = fmaf(-As[(16 * w + i) * kLd + 16 * w + l], x[l], s);
      x[i] = s;
    }
    if (g == 0)
#pragma unroll
      for (int i = 0; i < 16; ++i) Ts[(16 * w + i) * kLd + 16 * w + n16] = x[i];
  }
  __syncthreads();
  // ... those below from the ones nearer to it: T_ij = -T_ii sum_l A_il T_lj
  for (int d = 1; d < 4; ++d) {
    const int bj = w - d;
    if (bj >= 0) {
      f32x4 s = {0.f, 0.f, 0.f, 0.f}, o = {0.f, 0.f, 0.f, 0.f};
      for (int l = bj; l < w; ++l)
#pragma unroll
        for (int i = 0; i < 4; ++i)          // k = 4 g + i of block l
          s = __builtin_amdgcn_mfma_f32_16x16x4f32(As[(16 * w + n16) * kLd + 16 * l + 4 * g + i],
                                                   Ts[(16 * l + 4 * g + i) * kLd + 16 * bj + n16], s, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < 4; ++i)            // s[i] is row 4 g + i: the operand's k
        o = __builtin_amdgcn_mfma_f32_16x16x4f32(Ts[(16 * w + n16) * kLd + 16 * w + 4 * g + i], s[i], o, 0, 0, 0);
#pragma unroll
      for (int r = 0; r < 4; ++r) Ts[(16 * w + 4 * g + r) * kLd + 16 * bj + n16] = -o[r];
    }
    __syncthreads();
  }
  // P T, and both matrices out
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
    for (int l = j; l <= w; ++l)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        o = __builtin_amdgcn_mfma_f32_16x16x4f32(Ps[(16 * w + n16) * kLd + 16 * l + 4 * g + i],
                                                 Ts[(16 * l + 4 * g + i) * kLd + 16 * j + n16], o, 0, 0, 0);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int i = 16 * w + 4 * g + r, jj = 16 * j + n16;
      const float wi = exp2f(static_cast<float>(Lg[kC - 1] - Lg[i])) * rk[i];
      slot_p[i * kC + jj] = j <= w ? wi * Ts[i * kLd + jj] * be[jj] : 0.f;
      slot_p[kSlotMat + i * kC + jj] = o[r] * be[jj];
    }
  }
  if (tid < kC) {
    const float gi = exp2f(static_cast<float>(Lg[tid]));
    slot_p[2 * kSlotMat + tid] = gi * rk[tid];
    slot_p[2 * kSlotMat + kC + tid] = gi * rq[tid];
    if (tid == kC - 1) {
      slot_p[2 * kSlotMat + 2 * kC] = gi;
      slot_p[2 * kSlotMat + 2 * kC + 1] = 0.f;
    }
  }
}

template <int DK, int ACT, int OUT>
__global__ __launch_bounds__(256) void k_gdc_scan(GdcArgs a) {
  constexpr int KS = DK / 16;
  constexpr int NT = DK / 64;                  // tiles of 16 state columns a wave
  constexpr int kLs = DK + 4, kLx = kC + 4;
  __shared__ __align__(16) float Ss[kRowsS * kLs];
  __shared__ __align__(16) float Ks[kC * kLs];
  __shared__ __align__(16) float Xs[kRowsS * kLx];
  __shared__ __align__(16) float Zs[kRowsS * kLx];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), w = tid / kWave;
  const int n16 = lane & 15, g = lane >> 4;
  const int nz = a.dv / kRowsS;
  const int z = blockIdx.x % nz;
  const int bh = blockIdx.x / nz;
  const int h = bh % a.nv, b = bh / a.nv, kh = h / (a.nv / a.nk);
  int begin, n;
  sequence(a, b, begin, n);
  const int dv0 = z * kRowsS;
  const int64_t so = (static_cast<int64_t>(b) * a.nv + h) * a.dv * static_cast<int64_t>(DK) + static_cast<int64_t>(dv0) * DK;
  const int c0 = a.first;
  int c1 = (n + kC - 1) / kC;
  if (a.per_pass && c1 > c0 + a.per_pass) c1 = c0 + a.per_pass;
  if (c0 > 0 && c0 >= c1) return;              // done in an earlier pass
  const float* src = c0 > 0 ? a.state_out : a.state_in;
  for (int i = tid; i < kRowsS * (DK / 4); i += 256) {
    const int r = i / (DK / 4), cc = (i % (DK / 4)) * 4;
    *reinterpret_cast<f32x4*>(Ss + r * kLs + cc) =
        src ? *reinterpret_cast<const f32x4*>(src + so + r * DK + cc) : f32x4{0.f, 0.f, 0.f, 0.f};
  }
  const int64_t st = static_cast<int64_t>(a.nk) * DK;
  __syncthreads();
  for (int c = c0; c < c1; ++c) {
    const int t0 = c * kC;
    const int len = n - t0 < kC ? n - t0 : kC;
    const int64_t row0 = static_cast<int64_t>(begin) + t0;
    const float* slot_p = a.ws + (slot_of(a, b, begin, c) * a.nv + h) * kSlotFloats;
    if (slot_p[2 * kSlotMat + 2 * kC + 1] != 0.f) {
      // token by token, 16 lanes a row of the state
      const int r = 4 * w + g;
      float S[DK / 16];
#pragma unroll
      for (int i = 0; i < DK / 16; ++i) S[i] = Ss[r * kLs + n16 * (DK / 16) + i];
      for (int t = 0; t < len; ++t) {
        const int64_t at = (row0 + t) * st + static_cast<int64_t>(kh) * DK + n16 * (DK / 16);
        float kv[DK / 16], qv[DK / 16], sk = 0.f, sq = 0.f;
#pragma unroll
        for (int i = 0; i < DK / 16; ++i) {
          kv[i] = load_scalar<ACT>(a.k, at + i);
          qv[i] = load_scalar<ACT>(a.q, at + i);
          sk = fmaf(kv[i], kv[i], sk);
          sq = fmaf(qv[i], qv[i], sq);
        }
        const auto sum16 = [&](float x) {
          x += __shfl_xor(x, 1);
          x += __shfl_xor(x, 2);
          x += __shfl_xor(x, 4);
          return x + __shfl_xor(x, 8);
        };
        const float fk = 1.0f / sqrtf(sum16(sk) + a.eps), fq = a.scale / sqrtf(sum16(sq) + a.eps);
        const float al = a.alpha[(row0 + t) * a.nv + h], bt = a.beta[(row0 + t) * a.nv + h];
        const int64_t vo = ((row0 + t) * a.nv + h) * static_cast<int64_t>(a.dv) + dv0 + r;
        float x = 0.f, o = 0.f;
#pragma unroll
        for (int i = 0; i < DK / 16; ++i) {
          kv[i] *= fk;
          qv[i] *= fq;
          x = fmaf(S[i], kv[i], x);
        }
        const float u = bt * (load_scalar<ACT>(a.v, vo) - al * sum16(x));
#pragma unroll
        for (int i = 0; i < DK / 16; ++i) {
          S[i] = fmaf(u, kv[i], al * S[i]);
          o = fmaf(S[i], qv[i], o);
        }
        o = sum16(o);
        if (n16 == 0) {
          if constexpr (OUT == kF32) static_cast<float*>(a.out)[vo] = o;
          else static_cast<uint16_t*>(a.out)[vo] = f32_to_bf16(o);
        }
      }
#pragma unroll
      for (int i = 0; i < DK / 16; ++i) Ss[r * kLs + n16 * (DK / 16) + i] = S[i];
      __syncthreads();
      continue;
    }
    // K S^T and Q S^T for the 16 tokens of this wave
    const bool live = 16 * w + n16 < len;
    const int64_t mine = (row0 + (live ? 16 * w + n16 : 0)) * st + static_cast<int64_t>(kh) * DK;
    f32x4 ks = {0.f, 0.f, 0.f, 0.f}, qs = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      f32x4 Ka = load4<ACT>(a.k, mine + 16 * s + 4 * g), Qa = load4<ACT>(a.q, mine + 16 * s + 4 * g);
      if (!live) Ka = Qa = f32x4{0.f, 0.f, 0.f, 0.f};
      *reinterpret_cast<f32x4*>(Ks + (16 * w + n16) * kLs + 16 * s + 4 * g) = Ka;
      const f32x4 Sb = *reinterpret_cast<const f32x4*>(Ss + n16 * kLs + 16 * s + 4 * g);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ks = __builtin_amdgcn_mfma_f32_16x16x4f32(Ka[i], Sb[i], ks, 0, 0, 0);
        qs = __builtin_amdgcn_mfma_f32_16x16x4f32(Qa[i], Sb[i], qs, 0, 0, 0);
      }
    }
    f32x4 x;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int i = 16 * w + 4 * g + r;
      const float v = i < len ? load_scalar<ACT>(a.v, ((row0 + i) * a.nv + h) * static_cast<int64_t>(a.dv) + dv0 + n16) : 0.f;
      x[r] = v - slot_p[2 * kSlotMat + i] * ks[r];
      qs[r] *= slot_p[2 * kSlotMat + kC + i];
    }
    *reinterpret_cast<f32x4*>(Xs + n16 * kLx + 16 * w + 4 * g) = x;
    __syncthreads();
    f32x4 zt = {0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s <= w; ++s) {
      const f32x4 Tz = *reinterpret_cast<const f32x4*>(slot_p + (16 * w + n16) * kC + 16 * s + 4 * g);
      const f32x4 To = *reinterpret_cast<const f32x4*>(slot_p + kSlotMat + (16 * w + n16) * kC + 16 * s + 4 * g);
      const f32x4 Xb = *reinterpret_cast<const f32x4*>(Xs + n16 * kLx + 16 * s + 4 * g);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        zt = __builtin_amdgcn_mfma_f32_16x16x4f32(Tz[i], Xb[i], zt, 0, 0, 0);
        qs = __builtin_amdgcn_mfma_f32_16x16x4f32(To[i], Xb[i], qs, 0, 0, 0);
      }
    }
    *reinterpret_cast<f32x4*>(Zs + n16 * kLx + 16 * w + 4 * g) = zt;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int i = 16 * w + 4 * g + r;
      if (i < len) {
        const int64_t oi = ((row0 + i) * a.nv + h) * static_cast<int64_t>(a.dv) + dv0 + n16;
        if constexpr (OUT == kF32) static_cast<float*>(a.out)[oi] = qs[r];
        else static_cast<uint16_t*>(a.out)[oi] = f32_to_bf16(qs[r]);
      }
    }
    __syncthreads();
    // S^T, the columns of this wave
    const float gc = slot_p[2 * kSlotMat + 2 * kC];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int d0 = 16 * (NT * w + t);
      f32x4 s = *reinterpret_cast<const f32x4*>(Ss + n16 * kLs + d0 + 4 * g);
      s *= gc;
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const f32x4 Zb = *reinterpret_cast<const f32x4*>(Zs + n16 * kLx + 16 * y + 4 * g);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          s = __builtin_amdgcn_mfma_f32_16x16x4f32(Ks[(16 * y + 4 * g + i) * kLs + d0 + n16], Zb[i], s, 0, 0, 0);
      }
      *reinterpret_cast<f32x4*>(Ss + n16 * kLs + d0 + 4 * g) = s;
    }
    __syncthreads();
  }
  for (int i = tid; i < kRowsS * (DK / 4); i += 256) {
    const int r = i / (DK / 4), cc = (i % (DK / 4)) * 4;
    *reinterpret_cast<f32x4*>(a.state_out + so + r * DK + cc) = *reinterpret_cast<const f32x4*>(Ss + r * kLs + cc);
  }
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

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int check(const gdn_desc* d, int32_t B, int32_t N) {
  if (!d) return bad("descriptor is NULL");
  if (d->n_k_heads < 1 || d->n_v_heads < 1 || d->n_v_heads > 1024 || d->n_v_heads % d->n_k_heads != 0)
    return bad("n_v_heads=%lld must be in [1, 1024] and a multiple of n_k_heads=%lld", d->n_v_heads, d->n_k_heads);
  if (d->d_k != 64 && d->d_k != 128) return bad("d_k=%lld must be 64 or 128", d->d_k);
  if (d->d_v < 16 || d->d_v > 256 || d->d_v % 16 != 0) return bad("d_v=%lld must be a multiple of 16 in [16, 256]", d->d_v);
  if ((d->act_dtype != MOE_F32 && d->act_dtype != MOE_BF16) || (d->out_dtype != MOE_F32 && d->out_dtype != MOE_BF16))
    return bad("act_dtype=%lld / out_dtype=%lld must be MOE_F32 or MOE_BF16", d->act_dtype, d->out_dtype);
  if (!std::isfinite(d->scale)) return bad("scale must be finite");
  if (!(d->eps >= 0.f) || !std::isfinite(d->eps)) return bad("eps must be finite and >= 0");
  if (B < 0 || B > (1 << 16) || N < 0 || N > (1 << 24)) return bad("B=%lld must be in [0, 2^16], N=%lld in [0, 2^24]", B, N);
  return MOE_OK;
}

// Slots of a pass: all chunks where they fit kPassBytes, else as many of each
// sequence as do (at least one).
struct GdcPlan {
  int per_pass;         // 0: one pass
  int slots;
  size_t bytes;
};

GdcPlan plan(const gdn_desc* d, int32_t B, int32_t N) {
  GdcPlan p;
  const int64_t each = static_cast<int64_t>(d->n_v_heads) * kSlotFloats * 4;
  const int64_t all = static_cast<int64_t>(N) / kC + B;
  if (all * each <= kPassBytes || all <= B) {
    p.per_pass = 0;
    p.slots = static_cast<int>(all);
  } else {
    int64_t per = kPassBytes / each / B;
    if (per < 1) per = 1;
    p.per_pass = static_cast<int>(per);
    p.slots = static_cast<int>(per * B);
  }
  p.bytes = static_cast<size_t>(p.slots) * each;
  return p;
}

template <int DK, int ACT>
void launch(const GdcArgs& a, int out, uint32_t prep, uint32_t scan, hipStream_t s) {
  if (prep > 0) launch_kernel(k_gdc_prep<DK, ACT>, dim3(prep), dim3(256), 0, s, a);
  if (out == MOE_F32) launch_kernel(k_gdc_scan<DK, ACT, kF32>, dim3(scan), dim3(256), 0, s, a);
  else launch_kernel(k_gdc_scan<DK, ACT, kBF16>, dim3(scan), dim3(256), 0, s, a);
}

}  // namespace
}  // namespace moe

extern "C" size_t gdn_chunk_workspace_bytes(const gdn_desc* d, int32_t B, int32_t N) {
  using namespace moe;
  if (check(d, B, N) != MOE_OK) return static_cast<size_t>(-1);
  api_ok();
  return B == 0 || N == 0 ? 0 : plan(d, B, N).bytes;
}

extern "C" int gdn_chunk_forward(const gdn_desc* d, int32_t B, int32_t N, int32_t T_max, const int32_t* cu, const void* q,
                                 const void* k, const void* v, const float* alpha, const float* beta,
                                 const float* state_in, float* state_out, void* out, void* workspace, size_t ws_bytes,
                                 void* stream) {
  using namespace moe;
  MarkScope marks;
  int rc;
  if ((rc = check(d, B, N))) return rc;
  if (T_max < 0) return bad("T_max=%lld must not be negative", T_max);
  if (B == 0) return api_ok();
  if (!cu || !state_out || (N > 0 && (!q || !k || !v || !alpha || !beta || !out))) return bad("NULL pointer argument");
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(state_in, 16) || !aligned(state_out, 16) ||
      !aligned(out, 16) || !aligned(alpha, 4) || !aligned(beta, 4) || !aligned(cu, 4))
    return bad("q, k, v, states and out must be 16-byte aligned, alpha, beta and cu 4-byte aligned");
  const GdcPlan p = plan(d, B, N);
  const size_t need = N > 0 ? p.bytes : 0;
  if (need > 0) {
    if (!workspace || !aligned(workspace, 256)) return bad("the workspace is NULL or not 256-byte aligned");
    if (ws_bytes < need) {
      char buf[256];
      snprintf(buf, sizeof(buf), "workspace of %zu bytes, %zu needed", ws_bytes, need);
      return api_fail(MOE_ENOMEM, buf);
    }
  }
  const int64_t act = d->act_dtype == MOE_F32 ? 4 : 2, osz = d->out_dtype == MOE_F32 ? 4 : 2, n = N;
  const int64_t n_q = n * d->n_k_heads * d->d_k * act, n_v = n * d->n_v_heads * d->d_v * act, n_g = n * d->n_v_heads * 4;
  const int64_t n_o = n * d->n_v_heads * d->d_v * osz, n_s = static_cast<int64_t>(B) * d->n_v_heads * d->d_v * d->d_k * 4;
  const int64_t n_w = static_cast<int64_t>(need);
  const void* ins[] = {q, k, v, alpha, beta, cu, state_in};
  const int64_t in_n[] = {n_q, n_q, n_v, n_g, n_g, (static_cast<int64_t>(B) + 1) * 4, n_s};
  for (int i = 0; i < 7; ++i) {
    const bool same = i == 6 && state_in == state_out;
    if ((!same && overlaps(state_out, n_s, ins[i], in_n[i])) || overlaps(out, n_o, ins[i], in_n[i]) ||
        overlaps(workspace, n_w, ins[i], in_n[i]))
      return bad("state_out, out or the workspace overlaps input %lld", i);
  }
  if (overlaps(state_out, n_s, out, n_o) || overlaps(workspace, n_w, out, n_o) || overlaps(workspace, n_w, state_out, n_s))
    return bad("state_out, out and the workspace overlap");

  GdcArgs a{};
  a.cu = cu;
  a.q = q; a.k = k; a.v = v; a.alpha = alpha; a.beta = beta;
  a.state_in = state_in; a.state_out = state_out; a.out = out;
  a.ws = static_cast<float*>(workspace);
  a.B = B; a.N = N; a.T_max = T_max < N ? T_max : N;
  a.nk = d->n_k_heads; a.nv = d->n_v_heads; a.dv = d->d_v;
  a.scale = d->scale; a.eps = d->eps;
  a.per_pass = p.per_pass;
  a.slots = p.slots;
  const int64_t scan = static_cast<int64_t>(B) * d->n_v_heads * (d->d_v / kRowsS), prep = static_cast<int64_t>(p.slots) * d->n_v_heads;
  if (scan >= (1 << 24) || prep >= (1 << 24)) return bad("B=%lld sequences of N=%lld tokens are too many blocks for one launch", B, N);
  const int chunks = (a.T_max + kC - 1) / kC;
  hipStream_t s = static_cast<hipStream_t>(stream);
  for (a.first = 0; a.first == 0 || a.first < chunks; a.first += a.per_pass) {
    const uint32_t np = chunks > 0 ? static_cast<uint32_t>(prep) : 0u, nb = static_cast<uint32_t>(scan);
    if (d->d_k == 128) {
      if (d->act_dtype == MOE_F32) launch<128, kF32>(a, d->out_dtype, np, nb, s);
      else launch<128, kBF16>(a, d->out_dtype, np, nb, s);
    } else {
      if (d->act_dtype == MOE_F32) launch<64, kF32>(a, d->out_dtype, np, nb, s);
      else launch<64, kBF16>(a, d->out_dtype, np, nb, s);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) {
      char buf[256];
      snprintf(buf, sizeof(buf), "chunked delta rule launch failed: %s", hipGetErrorString(e));
      return api_fail(MOE_EHIP, buf);
    }
    if (a.per_pass == 0) break;
  }
  return api_ok();
}
