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
//
// Single precision on the bf16 matrix units.  An fp32 value is the sum of three
// bf16 (8 bits each, 24 together); K and Q are bf16 as they come.  So K S^T takes
// three products, and (Z-matrix) X the six whose terms are above 2^-24: 1 1, 1 2,
// 2 1, 1 3, 2 2, 3 1.  That is 5 to 10 times the rate of the fp32 instruction,
// which fp32 activations run on.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdio>
#include <type_traits>

#include "device_common.h"
#include "gdn_chunk.h"
#include "moe_internal.h"
#include "topk_wave.h"

namespace moe {
namespace {

constexpr int kC = 64;                        // tokens a chunk
constexpr int kRowsS = 16;                    // state rows a block
constexpr int64_t kPassBytes = int64_t(512) << 20;   // workspace a pass may take
typedef float f32x4 __attribute__((ext_vector_type(4)));

// One chunk and value head in the workspace: the row factors e, f, then g_C and
// whether the chunk runs token by token; the two matrices.  For fp32 activations
// they are rows of fp32; for bf16 planes of bf16 as the matrix unit's
// operand has them, 16 rows by 32 columns a kilobyte, those that lie above the
// diagonal left out (rows in the order of token_of).
constexpr int kVec = 4 * kC;                  // floats
constexpr int kPieces = 6;                    // (tiles 0 .. 3 by columns 0; 2, 3 by 32)
constexpr int kMatF32 = kC * kC * 4, kMatBf16 = kPieces * 1024;   // of one plane
// Planes of the O-matrix, and of S in Q S^T: outputs in bf16 keep 8 bits, so two.
constexpr int o_planes(int out) { return out == kF32 ? 3 : 2; }
constexpr int slot_bytes(int act, int out) { return kVec * 4 + (act == kF32 ? 2 * kMatF32 : (3 + o_planes(out)) * kMatBf16); }
// Row m of tile i is this token of the chunk: the eight values that a lane holds
// of the results of two tiles are then eight tokens in a row, which is the
// operand of the next product as it stands.
__host__ __device__ constexpr int token_of(int tile, int m) { return 32 * (tile >> 1) + 8 * (m >> 2) + 4 * (tile & 1) + (m & 3); }
__host__ __device__ constexpr int piece_of(int tile, int step) { return tile < 2 ? tile : 2 * tile - 2 + step; }

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
  uint8_t* ws;
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

// Sum over the L lanes that hold a row; every lane ends with it.
template <int L>
__device__ __forceinline__ float lanes_sum(float x, int lane) {
  x += __uint_as_float(lane_xor<1>(__float_as_uint(x), lane));
  x += __uint_as_float(lane_xor<2>(__float_as_uint(x), lane));
  x += __uint_as_float(lane_xor<4>(__float_as_uint(x), lane));
  if constexpr (L > 8) x += __uint_as_float(lane_xor<8>(__float_as_uint(x), lane));
  if constexpr (L > 16) x += __uint_as_float(lane_xor<16>(__float_as_uint(x), lane));
  return x;
}

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// Two values as the sums of three bf16 each, a word a plane.
__device__ __forceinline__ void split3(float x, float y, uint32_t& p0, uint32_t& p1, uint32_t& p2) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const auto step = [&]() {
    const uint32_t p = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{x, y}), bf16x2));
    x -= __uint_as_float(p << 16);
    y -= __uint_as_float(p & 0xffff0000u);
    return p;
  };
  p0 = step();
  p1 = step();
  p2 = step();
}

// Eight values, four of each argument, as an operand in three planes.
__device__ __forceinline__ void split3(const f32x4& lo, const f32x4& hi, bf16x8 (&p)[3]) {
  u32x4 w[3];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t a0, a1, a2;
    split3(lo[2 * i], lo[2 * i + 1], a0, a1, a2);
    w[0][i] = a0; w[1][i] = a1; w[2][i] = a2;
    split3(hi[2 * i], hi[2 * i + 1], a0, a1, a2);
    w[0][2 + i] = a0; w[1][2 + i] = a1; w[2][2 + i] = a2;
  }
#pragma unroll
  for (int x = 0; x < 3; ++x) p[x] = __builtin_bit_cast(bf16x8, w[x]);
}

// The part of a row of K or Q that a lane feeds to a product over 32 (bf16) or
// 16 (fp32) dims, from LDS.
template <int ACT>
using Operand = std::conditional_t<ACT == kF32, f32x4, bf16x8>;

__device__ __forceinline__ f32x4 dot_step(f32x4 a, f32x4 b, f32x4 c) {
#pragma unroll
  for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], c, 0, 0, 0);
  return c;
}
__device__ __forceinline__ f32x4 dot_step(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// The matrices of one chunk and value head.  Four waves: K K^T and Q K^T below the
// diagonal on the matrix units, T by substitution in the diagonal blocks of 16 and
// block by block below them in fp32, P T, then both out.  Its phases, with a
// barrier after each, bound it: three blocks on a CU hide part of them (8 sequences
// of 1024 tokens by 32 heads, 4096 blocks: 70 us; 210 MB read and written, 3 TB/s).
// Everything it reads is requested before the first use: 145 us instead of 243
// for 16 prompts of 60 to 4000 tokens.
template <int DK, int ACT, int OUT>
__global__ __launch_bounds__(256) void k_gdc_prep(GdcArgs a) {
  constexpr int kSize = ACT == kF32 ? 4 : 2;
  constexpr int kRow = DK * kSize + 16;          // bytes of a row of K or Q in LDS
  constexpr int kPer = DK * kSize / 16;          // 16-byte pieces a row: the lanes that load it
  constexpr int KS = DK * kSize / 64;            // steps of 64 bytes
  constexpr int kLd = kC + 4;
  // K and Q, then in their place P and T
  constexpr int kKq = 2 * kC * kRow, kMats = 2 * kC * kLd * 4;
  __shared__ __align__(16) uint8_t kq[kKq > kMats ? kKq : kMats];
  __shared__ __align__(16) float As[kC * kLd];
  __shared__ float rk[kC], rq[kC];
  __shared__ __align__(16) float be[kC];
  __shared__ double Lg[kC];
  __shared__ int odd;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), w = __builtin_amdgcn_readfirstlane(tid / kWave);
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
      cnt += __popcll(__ballot(j < a.B && a.cu[j < a.B ? j : 0] / kC + j <= slot));
    }
    b = cnt - 1;
  }
  if (b < 0 || b >= a.B) return;
  b = __builtin_amdgcn_readfirstlane(b);
  int begin, n;
  sequence(a, b, begin, n);
  const int c = a.per_pass ? a.first + slot % a.per_pass : slot - begin / kC - b;
  if (c < 0 || static_cast<int64_t>(c) * kC >= n) return;
  const int t0 = c * kC;
  const int len = n - t0 < kC ? n - t0 : kC;
  const int64_t row0 = static_cast<int64_t>(begin) + t0;

  if (tid == 0) odd = 0;
  // everything that is read, requested at once
  constexpr int kLoads = kC * kPer / 256;
  const int64_t st = static_cast<int64_t>(a.nk) * DK;
  u32x4 kv[kLoads], qv[kLoads];
#pragma unroll
  for (int x = 0; x < kLoads; ++x) {
    const int i = tid + 256 * x, r = i / kPer;
    const int64_t off = ((row0 + (r < len ? r : len - 1)) * st + static_cast<int64_t>(kh) * DK) * kSize + (i % kPer) * 16;
    kv[x] = load16(static_cast<const uint8_t*>(a.k) + off);
    qv[x] = load16(static_cast<const uint8_t*>(a.q) + off);
  }
  float al = 1.f, bt = 0.f;
  if (w == 0 && lane < len) {
    al = a.alpha[(row0 + lane) * a.nv + h];
    bt = a.beta[(row0 + lane) * a.nv + h];
  }
  __syncthreads();
  bool fine = true;
  // K and Q into LDS, and the norms of their rows over the lanes that load one
#pragma unroll
  for (int x = 0; x < kLoads; ++x) {
    const int i = tid + 256 * x, r = i / kPer, at = (i % kPer) * 16;
    if (r >= len) kv[x] = qv[x] = u32x4{0, 0, 0, 0};
    *reinterpret_cast<u32x4*>(kq + r * kRow + at) = kv[x];
    *reinterpret_cast<u32x4*>(kq + kC * kRow + r * kRow + at) = qv[x];
    float sk = 0.f, sq = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (ACT == kF32) {
        sk = fmaf(__uint_as_float(kv[x][j]), __uint_as_float(kv[x][j]), sk);
        sq = fmaf(__uint_as_float(qv[x][j]), __uint_as_float(qv[x][j]), sq);
      } else {
        const float k0 = __uint_as_float(kv[x][j] << 16), k1 = __uint_as_float(kv[x][j] & 0xffff0000u);
        const float q0 = __uint_as_float(qv[x][j] << 16), q1 = __uint_as_float(qv[x][j] & 0xffff0000u);
        sk = fmaf(k1, k1, fmaf(k0, k0, sk));
        sq = fmaf(q1, q1, fmaf(q0, q0, sq));
      }
    }
    sk = lanes_sum<kPer>(sk, lane);
    sq = lanes_sum<kPer>(sq, lane);
    const float rkv = 1.0f / sqrtf(sk + a.eps), rqv = a.scale / sqrtf(sq + a.eps);
    // a row that is not finite has a norm that is not
    fine = fine && (r >= len || (isfinite(sk) && isfinite(sq) && isfinite(rkv) && isfinite(rqv)));
    if (i % kPer == 0) {
      rk[r] = r < len ? rkv : 0.f;
      rq[r] = r < len ? rqv : 0.f;
    }
  }
  if (w == 0) {                                // gates: logarithms summed in double precision
    if (!(al >= 9.5367431640625e-7f && al <= 1.f && bt >= 0.f && bt <= 2.f)) fine = false;
    double s = static_cast<double>(log2f(al));
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const double o = __shfl_up(s, d);
      if (lane >= d) s += o;
    }
    Lg[lane] = s;
    be[lane] = bt;
  }
  if (!fine) odd = 1;
  __syncthreads();
  uint8_t* const out = a.ws + (static_cast<int64_t>(slot) * a.nv + h) * slot_bytes(ACT, OUT);
  float* const vec = reinterpret_cast<float*>(out);
  if (odd) {
    if (tid == 0) vec[2 * kC + 1] = 1.f;
    return;
  }
  // K K^T and Q K^T: the ten blocks (i, j) of 16 x 16 on and below the diagonal
  constexpr int I[12] = {0, 1, 2, 3, 1, 2, 3, 2, 3, 3, 0, 0}, J[12] = {0, 1, 2, 3, 0, 1, 2, 0, 1, 0, 0, 0};
  f32x4 H[3];
#pragma unroll
  for (int x = 0; x < 3; ++x) {
    const int p = w + 4 * x;
    if (p >= 10) continue;
    const int bi = I[p], bj = J[p];
    f32x4 G = {0.f, 0.f, 0.f, 0.f};
    H[x] = G;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const auto Ka = *reinterpret_cast<const Operand<ACT>*>(kq + (16 * bi + n16) * kRow + 64 * s + 16 * g);
      const auto Qa = *reinterpret_cast<const Operand<ACT>*>(kq + kC * kRow + (16 * bi + n16) * kRow + 64 * s + 16 * g);
      const auto Kb = *reinterpret_cast<const Operand<ACT>*>(kq + (16 * bj + n16) * kRow + 64 * s + 16 * g);
      G = dot_step(Ka, Kb, G);
      H[x] = dot_step(Qa, Kb, H[x]);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int i = 16 * bi + 4 * g + r, j = 16 * bj + n16;
      const float D = i >= j ? __builtin_amdgcn_exp2f(static_cast<float>(Lg[i] - Lg[j])) * rk[j] : 0.f;
      As[i * kLd + j] = i > j ? be[i] * D * rk[i] * G[r] : 0.f;
      H[x][r] *= D * rq[i];
    }
  }
  __syncthreads();                               // K and Q have been read
  float* const Ps = reinterpret_cast<float*>(kq);
  float* const Ts = Ps + kC * kLd;
  float* const PT = As;                          // A has done its part by then
#pragma unroll
  for (int x = 0; x < 3; ++x) {
    const int p = w + 4 * x;
    if (p < 10)
#pragma unroll
      for (int r = 0; r < 4; ++r) Ps[(16 * I[p] + 4 * g + r) * kLd + 16 * J[p] + n16] = H[x][r];
  }
  // T = (I + A)^-1: the diagonal blocks by substitution, a column a lane ...
  {
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s0 = i == n16 ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
      for (int l = 0; l < i; ++l) {
        float& s = l & 1 ? s1 : s0;
        s = fmaf(-As[(16 * w + i) * kLd + 16 * w + l], x[l], s);
      }
      x[i] = s0 + s1;
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
      for (int l = bj; l < w; ++l) {
        const f32x4 Al = *reinterpret_cast<const f32x4*>(As + (16 * w + n16) * kLd + 16 * l + 4 * g);
#pragma unroll
        for (int i = 0; i < 4; ++i)          // k = 4 g + i of block l
          s = __builtin_amdgcn_mfma_f32_16x16x4f32(Al[i], Ts[(16 * l + 4 * g + i) * kLd + 16 * bj + n16], s, 0, 0, 0);
      }
      const f32x4 Tw = *reinterpret_cast<const f32x4*>(Ts + (16 * w + n16) * kLd + 16 * w + 4 * g);
#pragma unroll
      for (int i = 0; i < 4; ++i)            // s[i] is row 4 g + i: the operand's k
        o = __builtin_amdgcn_mfma_f32_16x16x4f32(Tw[i], s[i], o, 0, 0, 0);
#pragma unroll
      for (int r = 0; r < 4; ++r) Ts[(16 * w + 4 * g + r) * kLd + 16 * bj + n16] = -o[r];
    }
    __syncthreads();
  }
  // P T, block by block; entry (i, j) takes i - j + 1 products, and each wave five
  constexpr int PI[12] = {3, 2, 3, 3, 0, 1, 2, 1, 0, 0, 0, 2}, PJ[12] = {0, 0, 1, 2, 0, 0, 1, 1, 0, 0, 0, 2};
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    // wave 3 has (3, 2), (1, 1), (2, 2), (3, 3); the others two blocks
    int bi, bj;
    if (x < 2) {
      bi = PI[w + 4 * x];
      bj = PJ[w + 4 * x];
    } else {
      if (w != 3) continue;
      bi = bj = x;
    }
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
    for (int l = bj; l <= bi; ++l) {
      const f32x4 Pl = *reinterpret_cast<const f32x4*>(Ps + (16 * bi + n16) * kLd + 16 * l + 4 * g);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        o = __builtin_amdgcn_mfma_f32_16x16x4f32(Pl[i], Ts[(16 * l + 4 * g + i) * kLd + 16 * bj + n16], o, 0, 0, 0);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) PT[(16 * bi + 4 * g + r) * kLd + 16 * bj + n16] = o[r];
  }
  __syncthreads();
  // both matrices out, 16 rows a wave, scaled by w_i and beta_j
  {
    const int i = ACT == kF32 ? 16 * w + n16 : token_of(w, n16);
    const float wi = exp2f(static_cast<float>(Lg[kC - 1] - Lg[i])) * rk[i];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if (ACT == kBF16 && s > w / 2) continue;
      f32x4 tz[2], to[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int j0 = 32 * s + 8 * g + 4 * x;
        const f32x4 t = *reinterpret_cast<const f32x4*>(Ts + i * kLd + j0), p = *reinterpret_cast<const f32x4*>(PT + i * kLd + j0);
        const f32x4 b4 = *reinterpret_cast<const f32x4*>(be + j0);
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const bool in = j0 + y <= i;
          tz[x][y] = in ? wi * t[y] * b4[y] : 0.f;
          to[x][y] = in ? p[y] * b4[y] : 0.f;
        }
      }
      if constexpr (ACT == kF32) {
        float* m = vec + kVec + i * kC + 32 * s + 8 * g;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          *reinterpret_cast<f32x4*>(m + 4 * x) = tz[x];
          *reinterpret_cast<f32x4*>(m + kC * kC + 4 * x) = to[x];
        }
      } else {
        bf16x8 z[3], o[3];
        split3(tz[0], tz[1], z);
        split3(to[0], to[1], o);
        uint8_t* m = out + kVec * 4 + piece_of(w, s) * 1024 + lane * 16;   // [plane][piece]
#pragma unroll
        for (int x = 0; x < 3; ++x) {
          *reinterpret_cast<bf16x8*>(m + x * kMatBf16) = z[x];
          if (x < o_planes(OUT)) *reinterpret_cast<bf16x8*>(m + (3 + x) * kMatBf16) = o[x];
        }
      }
    }
  }
  if (tid < kC) {
    const float gi = exp2f(static_cast<float>(Lg[tid]));
    vec[tid] = gi * rk[tid];
    vec[kC + tid] = gi * rq[tid];
    if (tid == kC - 1) {
      vec[2 * kC] = gi;
      vec[2 * kC + 1] = 0.f;
    }
  }
}

// Whether one of the values is not finite, or so large (2^96) that the products
// of a chunk could leave the range where those of single tokens do not.
__device__ __forceinline__ bool far4(const f32x4& v) {
  const uint32_t a = __float_as_uint(v[0]) & 0x7fffffffu, b = __float_as_uint(v[1]) & 0x7fffffffu;
  const uint32_t c = __float_as_uint(v[2]) & 0x7fffffffu, d = __float_as_uint(v[3]) & 0x7fffffffu;
  const uint32_t x = a > b ? a : b, y = c > d ? c : d;
  return (x > y ? x : y) > 0x6f800000u;
}

// A chunk token by token, 16 lanes a row of the 16 of the state in LDS (S, rows
// kLs apart), every wave four of them.
template <int DK, int ACT, int OUT>
__device__ __forceinline__ void chunk_by_token(const GdcArgs& a, float* Ss, int kLs, int64_t row0, int len, int h, int kh, int dv0, int lane, int w) {
  constexpr int NC = DK / 16;
  const int n16 = lane & 15, r = 4 * w + (lane >> 4);
  const int64_t st = static_cast<int64_t>(a.nk) * DK;
  float S[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) S[i] = Ss[r * kLs + n16 * NC + i];
  const auto sum16 = [&](float x) {
    x += __shfl_xor(x, 1);
    x += __shfl_xor(x, 2);
    x += __shfl_xor(x, 4);
    return x + __shfl_xor(x, 8);
  };
  for (int t = 0; t < len; ++t) {
    const int64_t at = (row0 + t) * st + static_cast<int64_t>(kh) * DK + n16 * NC;
    float kv[NC], qv[NC], sk = 0.f, sq = 0.f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      kv[i] = load_scalar<ACT>(a.k, at + i);
      qv[i] = load_scalar<ACT>(a.q, at + i);
      sk = fmaf(kv[i], kv[i], sk);
      sq = fmaf(qv[i], qv[i], sq);
    }
    const float fk = 1.0f / sqrtf(sum16(sk) + a.eps), fq = a.scale / sqrtf(sum16(sq) + a.eps);
    const float al = a.alpha[(row0 + t) * a.nv + h], bt = a.beta[(row0 + t) * a.nv + h];
    const int64_t vo = ((row0 + t) * a.nv + h) * static_cast<int64_t>(a.dv) + dv0 + r;
    float x = 0.f, o = 0.f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      kv[i] *= fk;
      qv[i] *= fq;
      x = fmaf(S[i], kv[i], x);
    }
    const float u = bt * (load_scalar<ACT>(a.v, vo) - al * sum16(x));
#pragma unroll
    for (int i = 0; i < NC; ++i) {
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
  for (int i = 0; i < NC; ++i) Ss[r * kLs + n16 * NC + i] = S[i];
}

// What a block of a scan works on: head h of sequence b, state rows from dv0 on.
struct Scan {
  int h, kh, b, dv0, begin, n, c0, c1;
  int64_t state;        // offset of its rows in the states
};

// The blocks of a head, which read the same matrices, go to one XCD (blocks
// are dealt out in turns over eight).
template <int WIDTH>
__device__ __forceinline__ bool find_scan(const GdcArgs& a, int dk, Scan& s) {
  const int nz = (a.dv + WIDTH - 1) / WIDTH;
  const int q = blockIdx.x / 8;
  const int bh = (q / nz) * 8 + blockIdx.x % 8;
  if (bh >= a.B * a.nv) return false;
  s.dv0 = (q % nz) * WIDTH;
  s.h = bh % a.nv;
  s.b = bh / a.nv;
  // the longest sequences first, where a wave holds all of them: theirs are the last to end
  if (a.B > 1 && a.B <= kWave) {
    const int lane = threadIdx.x & (kWave - 1);
    int begin, n = -1, rank = 0;
    if (lane < a.B) sequence(a, lane, begin, n);
    for (int j = 0; j < a.B; ++j) {
      const int o = __builtin_amdgcn_readlane(n, j);
      rank += o > n || (o == n && j < lane);
    }
    const uint64_t hit = __ballot(lane < a.B && rank == s.b);
    s.b = __builtin_ctzll(hit);
  }
  s.kh = s.h / (a.nv / a.nk);
  sequence(a, s.b, s.begin, s.n);
  s.state = (static_cast<int64_t>(s.b) * a.nv + s.h) * a.dv * static_cast<int64_t>(dk) + static_cast<int64_t>(s.dv0) * dk;
  s.c0 = a.first;
  s.c1 = (s.n + kC - 1) / kC;
  if (a.per_pass && s.c1 > s.c0 + a.per_pass) s.c1 = s.c0 + a.per_pass;
  return s.c0 == 0 || s.c0 < s.c1;             // else done in an earlier pass
}

// bf16 activations, few heads: four waves share 16 rows of a state.  Wave w has
// the tokens of tile w of a chunk in the first two products and state columns
// DK / 4 w .. in the third; S, X and Zt pass from one to the next through LDS, split
// in three.  What a product takes of the next chunk is requested a chunk ahead,
// between the products: the memory unit takes 64 bytes a cycle.
//
// Its own chain bounds it, 2.2 us a chunk alone on a CU, of which a wave's 50
// products are a sixth: the rest are their operands' way through LDS, the splits and
// three barriers (one sequence of 2048 tokens, 32 heads of 128 x 128: 68 us; 78 with
// every address formed from the chunk's number).
template <int DK, int OUT>
__global__ __launch_bounds__(256, 2) void k_gdc_scan_few(GdcArgs a) {
  constexpr int OP = o_planes(OUT);
  constexpr int KS = DK / 32;                  // steps of 32 state columns
  constexpr int NT = DK / 64;                  // tiles of 16 state columns a wave
  constexpr int kLs = DK + 4;
  constexpr int kPer = DK / 8;                 // 16-byte pieces of a row of K
  constexpr int kKl = kC * kPer / 256;         // of them a thread
  constexpr int kPlaneS = kRowsS * DK * 2, kPlaneX = kRowsS * kC * 2;
  __shared__ __align__(16) uint8_t Sp[3 * kPlaneS];        // S, X and Zt: [plane][state row][column or token]
  __shared__ __align__(16) uint8_t Xp[3 * kPlaneX];
  __shared__ __align__(16) uint8_t Zp[3 * kPlaneX];
  __shared__ __align__(16) uint8_t Kp[2][kC * DK * 2];
  __shared__ int far[4];                       // whether a wave's part of X is out of range
  const int lane = threadIdx.x & (kWave - 1), w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int n16 = lane & 15, g = lane >> 4;
  Scan sc;
  if (!find_scan<kRowsS>(a, DK, sc)) return;
  // Pieces of 16 bytes turned by their row against bank conflicts: rows of S
  // (256 or 128 bytes), of X and Zt (128), and of K (read by rows and, four rows of
  // 32 bytes at once, transposed).
  const auto s_at = [&](int row, int col) { return row * DK * 2 + (((col >> 3) ^ (row & (kPer - 1))) << 4) + (col & 7) * 2; };
  const auto x_at = [&](int row, int tok) { return row * kC * 2 + (((tok >> 3) ^ (row & 7)) << 4) + (tok & 7) * 2; };
  const auto k_at = [&](int tok, int piece) { return tok * DK * 2 + ((piece ^ (((tok & 3) + ((tok >> 1) & 4)) * (DK == 128 ? 2 : 1))) << 4); };

  // this wave's columns of S^T: tile t, lane: state row n16, columns 16 (NT w + t) + 4 g ..
  f32x4 S[NT];
  const float* src = sc.c0 > 0 ? a.state_out : a.state_in;
#pragma unroll
  for (int t = 0; t < NT; ++t)
    S[t] = src ? *reinterpret_cast<const f32x4*>(src + sc.state + n16 * DK + 16 * (NT * w + t) + 4 * g) : f32x4{0.f, 0.f, 0.f, 0.f};
  const auto put_s = [&]() {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      uint32_t p[3], q[3];
      split3(S[t][0], S[t][1], p[0], p[1], p[2]);
      split3(S[t][2], S[t][3], q[0], q[1], q[2]);
#pragma unroll
      for (int x = 0; x < 3; ++x) *reinterpret_cast<uint2*>(Sp + x * kPlaneS + s_at(n16, 16 * (NT * w + t) + 4 * g)) = uint2{p[x], q[x]};
    }
  };
  const int t4 = token_of(w, 4 * g);           // this lane's four tokens of a result
  const auto put_x = [&](uint8_t* to, const f32x4& v) {
    uint32_t p[3], q[3];
    split3(v[0], v[1], p[0], p[1], p[2]);
    split3(v[2], v[3], q[0], q[1], q[2]);
#pragma unroll
    for (int x = 0; x < 3; ++x) *reinterpret_cast<uint2*>(to + x * kPlaneX + x_at(n16, t4)) = uint2{p[x], q[x]};
  };

  const int64_t st = static_cast<int64_t>(a.nk) * DK;
  const int64_t vst = static_cast<int64_t>(a.nv) * a.dv;
  constexpr int kOut = OUT == kF32 ? 4 : 2;
  // where the chunks to request next begin, and the one to write
  const int kst = static_cast<int>(st) * 2, vbytes = static_cast<int>(vst) * 2, ost = static_cast<int>(vst) * kOut;
  const int64_t row = static_cast<int64_t>(sc.begin) + static_cast<int64_t>(sc.c0) * kC, to_v = static_cast<int64_t>(sc.h) * a.dv + sc.dv0;
  const uint8_t* kn = static_cast<const uint8_t*>(a.k) + row * kst + static_cast<int64_t>(sc.kh) * DK * 2;
  const uint8_t* qn = static_cast<const uint8_t*>(a.q) + row * kst + static_cast<int64_t>(sc.kh) * DK * 2;
  const uint8_t* vn = static_cast<const uint8_t*>(a.v) + row * vbytes + to_v * 2;
  const uint8_t* mn = a.ws + (slot_of(a, sc.b, sc.begin, sc.c0) * a.nv + sc.h) * slot_bytes(kBF16, OUT);
  uint8_t* on = static_cast<uint8_t*>(a.out) + row * ost + to_v * kOut;
  // Offsets within a chunk.  The descriptors end with the last token: rows behind
  // it arrive as zeros, and are not written.
  uint32_t koff[kKl], voff[4];
#pragma unroll
  for (int i = 0; i < kKl; ++i) {
    const int p = threadIdx.x + 256 * i;
    koff[i] = (p / kPer) * static_cast<uint32_t>(kst) + (p % kPer) * 16;
  }
  const uint32_t qoff = token_of(w, n16) * static_cast<uint32_t>(kst) + g * 16;
#pragma unroll
  for (int r = 0; r < 4; ++r) voff[r] = (t4 + r) * static_cast<uint32_t>(vbytes) + n16 * 2;
  const auto length = [&](int c) { return sc.n - c * kC < kC ? sc.n - c * kC : kC; };
  const auto buffer = [](const void* base, int bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, bytes, 0x00020000);
  };
  const auto load = [](auto rs, uint32_t off, int at) { return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, off, at, 0)); };
  u32x4 Kn[kKl];
  bf16x8 Tz[2][3], To[2][OP];
  struct First {                               // what the first product takes
    bf16x8 Q[KS];
    uint16_t V[4];                             // as stored: converted where it is used, or the load would be waited for here
    f32x4 e, f;
    float2 gc;                                 // g_C, and whether the chunk runs token by token
  };
  First even, odd;                             // by the chunk's number
  const auto ask_k = [&](int c) {
    const auto rs = buffer(kn, (length(c) - 1) * kst + DK * 2);
#pragma unroll
    for (int i = 0; i < kKl; ++i) Kn[i] = load(rs, koff[i], 0);
  };
  const auto put_k = [&](int half) {
#pragma unroll
    for (int i = 0; i < kKl; ++i) {
      const int p = threadIdx.x + 256 * i;
      *reinterpret_cast<u32x4*>(Kp[half] + k_at(p / kPer, p % kPer)) = Kn[i];
    }
  };
  const auto ask_q = [&](int c, First& o, int s) {
    const auto rq = buffer(qn, (length(c) - 1) * kst + DK * 2);
    o.Q[s] = __builtin_bit_cast(bf16x8, load(rq, qoff + 64 * s, 0));
  };
  const auto ask_rest = [&](int c, First& o) {
    const auto rv = buffer(vn, (length(c) - 1) * vbytes + kRowsS * 2);
    const auto rf = buffer(mn, kVec * 4);
#pragma unroll
    for (int r = 0; r < 4; ++r) o.V[r] = __builtin_amdgcn_raw_buffer_load_b16(rv, voff[r], 0, 0);
    o.e = __builtin_bit_cast(f32x4, load(rf, t4 * 4, 0));
    o.f = __builtin_bit_cast(f32x4, load(rf, t4 * 4, kC * 4));
    o.gc = __builtin_bit_cast(float2, __builtin_amdgcn_raw_buffer_load_b64(rf, 0, 2 * kC * 4, 0));
  };
  const auto ask_second = [&](int s) {         // for the second, 32 columns of the matrices
    const auto rm = buffer(mn, slot_bytes(kBF16, OUT));
    if (s <= w / 2)
#pragma unroll
      for (int x = 0; x < 3; ++x) {
        Tz[s][x] = __builtin_bit_cast(bf16x8, load(rm, lane * 16, kVec * 4 + x * kMatBf16 + piece_of(w, s) * 1024));
        if (x < OP) To[s][x] = __builtin_bit_cast(bf16x8, load(rm, lane * 16, kVec * 4 + (3 + x) * kMatBf16 + piece_of(w, s) * 1024));
      }
  };
  put_s();
  if (sc.c0 < sc.c1) {
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      ask_q(sc.c0, even, s);
    }
    ask_k(sc.c0);
    ask_rest(sc.c0, even);
    ask_second(0);
    ask_second(1);
    put_k(0);
    if (sc.c0 + 1 < sc.c1) kn += static_cast<int64_t>(kC) * kst;
    ask_k(sc.c0 + 1 < sc.c1 ? sc.c0 + 1 : sc.c0);
  }
  __syncthreads();
  // chunk c, whose rows of K lie in stage `half`
  const auto chunk = [&](int c, int half, const First& one, First& then) {
    const int64_t row0 = static_cast<int64_t>(sc.begin) + c * kC;
    const int len = sc.n - c * kC < kC ? sc.n - c * kC : kC;
    // requests without a condition (the last chunk asks for itself again), so that no copy of a register waits for one
    const int next = c + 1 < sc.c1 ? c + 1 : c;
    if (c + 1 < sc.c1) {
      qn += static_cast<int64_t>(kC) * kst;
      vn += static_cast<int64_t>(kC) * vbytes;
      mn += static_cast<int64_t>(a.nv) * slot_bytes(kBF16, OUT);
    }
    const uint8_t* K = Kp[half];
    const float gC = one.gc.x;
    bool by_token = __builtin_amdgcn_readfirstlane(__float_as_int(one.gc.y)) != 0;
    f32x4 qs = {0.f, 0.f, 0.f, 0.f};
    const auto run_tokens = [&]() {            // in fp32 through the place of S
      static_assert(3 * kPlaneS >= kRowsS * kLs * 4, "room for the state");
      float* Ss = reinterpret_cast<float*>(Sp);
#pragma unroll
      for (int t = 0; t < NT; ++t) *reinterpret_cast<f32x4*>(Ss + n16 * kLs + 16 * (NT * w + t) + 4 * g) = S[t];
      __syncthreads();
      chunk_by_token<DK, kBF16, OUT>(a, Ss, kLs, row0, len, sc.h, sc.kh, sc.dv0, lane, w);
      __syncthreads();
#pragma unroll
      for (int t = 0; t < NT; ++t) S[t] = *reinterpret_cast<const f32x4*>(Ss + n16 * kLs + 16 * (NT * w + t) + 4 * g);
      __syncthreads();
    };
    if (by_token) {
      run_tokens();
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        ask_q(next, then, s);
      }
      ask_rest(next, then);
    } else {
      // K S^T and Q S^T
      f32x4 ks = {0.f, 0.f, 0.f, 0.f}, ks2 = ks, qs2 = ks;   // two chains each: a product waits for the one before it
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const bf16x8 Ka = *reinterpret_cast<const bf16x8*>(K + k_at(token_of(w, n16), 4 * s + g));
        ask_q(next, then, s);
#pragma unroll
        for (int x = 2; x >= 0; --x) {
          const bf16x8 Sb = *reinterpret_cast<const bf16x8*>(Sp + x * kPlaneS + s_at(n16, 32 * s + 8 * g));
          f32x4& kd = s & 1 ? ks2 : ks;
          f32x4& qd = (s & 1) && OP == 2 ? qs2 : qs;       // with three planes its chain is as long as the other
          kd = __builtin_amdgcn_mfma_f32_16x16x32_bf16(Ka, Sb, kd, 0, 0, 0);
          if (x < OP) qd = __builtin_amdgcn_mfma_f32_16x16x32_bf16(one.Q[s], Sb, qd, 0, 0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);     // requests between the products: the memory unit takes 64 bytes a cycle
      }
      f32x4 x;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        x[r] = bf16_to_f32(one.V[r]) - one.e[r] * (ks[r] + ks2[r]);
        qs[r] = (qs[r] + qs2[r]) * one.f[r];
      }
      put_x(Xp, x);
      ask_rest(next, then);
      if (lane == 0) far[w] = 0;
      if (far4(x)) far[w] = 1;
    }
    __syncthreads();
    if (!by_token && (far[0] | far[1] | far[2] | far[3]) != 0) {
      by_token = true;                         // out of range: S is as it was
      __syncthreads();                         // before the next chunk's flags
      run_tokens();
    }
    if (!by_token) {
      // (Z-matrix) X and (O-matrix) X
      f32x4 zt = {0.f, 0.f, 0.f, 0.f}, zt2 = zt;
#pragma unroll
      for (int s = 0; s < 2; ++s)
        if (s <= w / 2) {
          bf16x8 Xb[3];
#pragma unroll
          for (int y = 0; y < 3; ++y) Xb[y] = *reinterpret_cast<const bf16x8*>(Xp + y * kPlaneX + x_at(n16, 32 * s + 8 * g));
#pragma unroll
          for (int y = 2; y >= 0; --y)         // the smallest terms first
#pragma unroll
            for (int z = 2 - y; z >= 0; --z) {
              f32x4& zd = z & 1 ? zt2 : zt;
              zd = __builtin_amdgcn_mfma_f32_16x16x32_bf16(Tz[s][z], Xb[y], zd, 0, 0, 0);
              if (z + y < OP) qs = __builtin_amdgcn_mfma_f32_16x16x32_bf16(To[s][z], Xb[y], qs, 0, 0, 0);
            }
        }
      put_x(Zp, zt + zt2);
    }
    ask_second(0);
    __syncthreads();
    if (!by_token) {
      const auto ro = buffer(on, (len - 1) * ost + kRowsS * kOut);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if constexpr (OUT == kF32) __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(qs[r]), ro, voff[r] * 2, 0, 0);
        else __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, static_cast<__bf16>(qs[r])), ro, voff[r], 0, 0);
      }
      // S^T, the columns of this wave
      bf16x8 Zb[2][3];
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int y = 0; y < 3; ++y) Zb[s][y] = *reinterpret_cast<const bf16x8*>(Zp + y * kPlaneX + x_at(n16, 32 * s + 8 * g));
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int piece = 2 * (NT * w + t) + ((n16 & 3) >> 1);
        f32x4 d[2] = {};
        if (t == 0) ask_second(1);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          bf16x8 Ka;                           // column n16 of the tile, tokens 32 s + 8 g + 0 .. 7
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
            const int tok = 32 * s + 8 * g + 4 * y + (n16 >> 2);
            const bf16x4 v = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(K + k_at(tok, piece) + (n16 & 1) * 8)));
#pragma unroll
            for (int i = 0; i < 4; ++i) Ka[4 * y + i] = v[i];
          }
#pragma unroll
          for (int y = 2; y >= 0; --y) d[s] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(Ka, Zb[s][y], d[s], 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) S[t][i] = fmaf(gC, S[t][i], d[0][i] + d[1][i]);
      }
    } else {
      ask_second(1);
    }
    put_s();
    put_k(half ^ 1);
    if (c + 2 < sc.c1) kn += static_cast<int64_t>(kC) * kst;
    on += static_cast<int64_t>(kC) * ost;
    ask_k(c + 2 < sc.c1 ? c + 2 : sc.c1 - 1);  // a chunk ahead: what has to come from HBM takes half of one
    __syncthreads();
  };
  for (int c = sc.c0; c < sc.c1; c += 2) {
    chunk(c, 0, even, odd);
    if (c + 1 < sc.c1) chunk(c + 1, 1, odd, even);
  }
#pragma unroll
  for (int t = 0; t < NT; ++t)
    *reinterpret_cast<f32x4*>(a.state_out + sc.state + n16 * DK + 16 * (NT * w + t) + 4 * g) = S[t];
}

// bf16 activations, many heads.  A wave walks the chunks with 16 rows of the state to itself,
// all in registers: a product's result, four tokens (or columns) of a state row
// a lane and tile, is split in three and is the next one's operand as it
// stands, by the order of tokens and columns within two tiles (token_of).  The four
// waves of a block, 64 rows of one head, share K, Q, V, the factors and the
// matrices in LDS, where the next chunk's arrive by direct loads meanwhile: one
// barrier a chunk.
//
// A wave's 216 products of 16 x 16 x 32 a chunk, 16 cycles each, and the 80 KB of
// operands that it reads from LDS bound it; two waves on a SIMD overlap them in
// part: a chunk of 128 rows takes 6.0 us, of which the products are 2.9 and the reads
// 2.1 (128 x 128 states; 8 sequences of 1024 tokens by 32 heads 96 us, 16 prompts of
// 60 to 4000 tokens 286; 106 and 324 with pointers converted and addresses formed anew
// for every load).
// lds_load<16> to an address as a number: no conversion of a pointer, with its check for NULL, before each load.
__device__ __forceinline__ void lds_load16(u32x4 rs, uint32_t to, uint32_t voff, uint32_t soff) {
  const uint32_t la = __builtin_amdgcn_readfirstlane(to), so = __builtin_amdgcn_readfirstlane(soff);
  uint32_t saved;
  asm volatile(
      "s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tbuffer_load_dwordx4 %2, %3, %4 offen lds\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(saved)
      : "s"(la), "v"(voff), "s"(rs), "s"(so)
      : "memory");
}

template <int DK, int OUT, int NW>
struct ScanLds {
  static constexpr int kK = 0, kQ = kC * DK * 2, kV = 2 * kC * DK * 2, kF = kV + kC * 16 * NW * 2, kM = kF + kVec * 4;
  static constexpr int kStage = kM + (3 + o_planes(OUT)) * kMatBf16, kBytes = 2 * kStage;
};

template <int DK, int OUT, int NW>
__global__ __launch_bounds__(64 * NW, NW / 4) void k_gdc_scan_bf16(GdcArgs a) {
  using L = ScanLds<DK, OUT, NW>;
  constexpr int OP = o_planes(OUT);
  constexpr int KS = DK / 32;                  // steps of 32 state columns
  constexpr int kPer = DK / 8;                 // 16-byte pieces of a row of K
  constexpr int kRpl = 64 / kPer;              // rows a direct load
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & (kWave - 1), w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int n16 = lane & 15, g = lane >> 4;
  Scan sc;
  if (!find_scan<16 * NW>(a, DK, sc)) return;
  const int dv0 = sc.dv0 + 16 * w;             // this wave's state rows
  const bool idle = dv0 >= a.dv;               // none: it only fetches
  // Pieces of K and Q are turned by their row, so that the 16 rows of a tile, and
  // eight of the sixteen of a transposing read, fall into different banks.
  const auto turn = [](int tok) { return DK == 128 ? (tok & 3) | ((tok >> 1) & 12) : (tok & 3) | ((tok >> 1) & 4); };

  // this wave's rows of S^T: tile pair s, lane: row n16, columns 32 s + 8 g + 0 .. 3, then + 4 .. 7
  f32x4 S[2 * KS];
  const float* src = sc.c0 > 0 ? a.state_out : a.state_in;
  const int64_t so = sc.state + static_cast<int64_t>(16 * w + n16) * DK;
#pragma unroll
  for (int t = 0; t < 2 * KS; ++t)
    S[t] = src && !idle ? *reinterpret_cast<const f32x4*>(src + so + 32 * (t >> 1) + 8 * g + 4 * (t & 1)) : f32x4{0.f, 0.f, 0.f, 0.f};
  // waited for here: a wait in the loop would be for the direct loads as well
#pragma unroll
  for (int t = 0; t < 2 * KS; ++t) asm volatile("" : "+v"(S[t]));

  const int64_t st = static_cast<int64_t>(a.nk) * DK, vst = static_cast<int64_t>(a.nv) * a.dv;
  const uint16_t* const kb = static_cast<const uint16_t*>(a.k) + static_cast<int64_t>(sc.begin) * st + static_cast<int64_t>(sc.kh) * DK;
  const uint16_t* const qb = static_cast<const uint16_t*>(a.q) + static_cast<int64_t>(sc.begin) * st + static_cast<int64_t>(sc.kh) * DK;
  const uint16_t* const vb = static_cast<const uint16_t*>(a.v) + static_cast<int64_t>(sc.begin) * vst + static_cast<int64_t>(sc.h) * a.dv + sc.dv0;
  const int vcols = a.dv - sc.dv0 < 16 * NW ? a.dv - sc.dv0 : 16 * NW;
  // Load i of a wave is kilobyte NW i + w: of K and Q kRpl rows each, of V kRpv.
  constexpr int kKq = kC / kRpl / NW, kRpv = 1024 / (32 * NW), kVl = kC / kRpv / NW, kMl = 1 + (3 + OP) * kPieces;
  uint32_t koff[kKq], voff[kVl];
#pragma unroll
  for (int i = 0; i < kKq; ++i) {
    const int row = (NW * i + w) * kRpl + lane / kPer;
    koff[i] = static_cast<uint32_t>(row) * static_cast<uint32_t>(st) * 2u + (((lane % kPer) ^ turn(row)) << 4);
  }
#pragma unroll
  for (int i = 0; i < kVl; ++i)
    voff[i] = static_cast<uint32_t>((NW * i + w) * kRpv + lane / (2 * NW)) * static_cast<uint32_t>(vst) * 2u + (lane % (2 * NW)) * 16;
  const auto length = [&](int c) { return sc.n - c * kC < kC ? sc.n - c * kC : kC; };
  // The requests for a chunk, in parts: the memory unit takes 64 bytes a cycle, so
  // all at once would hold the wave up.  The descriptors end with the last token:
  // rows behind it arrive as zeros.
  constexpr int kParts = 4;
  const int kst = static_cast<int>(st) * 2, vbytes = static_cast<int>(vst) * 2;      // from token to token
  const uint8_t* kn = reinterpret_cast<const uint8_t*>(kb) + static_cast<int64_t>(sc.c0) * kC * kst;   // of the chunk to request
  const uint8_t* qn = reinterpret_cast<const uint8_t*>(qb) + static_cast<int64_t>(sc.c0) * kC * kst;
  const uint8_t* vn = reinterpret_cast<const uint8_t*>(vb) + static_cast<int64_t>(sc.c0) * kC * vbytes;
  const uint8_t* mn = a.ws + (slot_of(a, sc.b, sc.begin, sc.c0) * a.nv + sc.h) * slot_bytes(kBF16, OUT);
  const auto request = [&](int c, uint32_t to, int part) {
    const int len = length(c);
    if (part == 0) {
      const u32x4 rk = raw_rsrc(kn, (len - 1) * kst + DK * 2);
#pragma unroll
      for (int i = 0; i < kKq; ++i) lds_load16(rk, to + L::kK + (NW * i + w) * 1024, koff[i], 0);
    } else if (part == 1) {
      const u32x4 rq = raw_rsrc(qn, (len - 1) * kst + DK * 2), rv = raw_rsrc(vn, (len - 1) * vbytes + vcols * 2);
#pragma unroll
      for (int i = 0; i < kKq; ++i) lds_load16(rq, to + L::kQ + (NW * i + w) * 1024, koff[i], 0);
#pragma unroll
      for (int i = 0; i < kVl; ++i) lds_load16(rv, to + L::kV + (NW * i + w) * 1024, voff[i], 0);
    } else {
      // the factors and the matrices lie as they do in the slot
      const u32x4 rm = raw_rsrc(mn, slot_bytes(kBF16, OUT));
      constexpr int kEach = (kMl + NW - 1) / NW, kHalf = kEach / 2;
#pragma unroll
      for (int i = part == 2 ? 0 : kHalf; i < (part == 2 ? kHalf : kEach); ++i)
        if (NW * i + w < kMl) lds_load16(rm, to + L::kF + (NW * i + w) * 1024, lane * 16, (NW * i + w) * 1024);
      if (part == kParts - 1) {
        kn += static_cast<int64_t>(kC) * kst;
        qn += static_cast<int64_t>(kC) * kst;
        vn += static_cast<int64_t>(kC) * vbytes;
        mn += static_cast<int64_t>(a.nv) * slot_bytes(kBF16, OUT);
      }
    }
  };
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  const auto transposed = [&](const uint8_t* p) { return __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p)); };

  // A chunk token by token: a lane has a quarter of a row's columns.
  const auto tokens = [&](int c, const uint8_t* in) {
    const int64_t row0 = static_cast<int64_t>(sc.begin) + static_cast<int64_t>(c) * kC;
    const auto sum4 = [&](float x) {
      x += __uint_as_float(lane_xor<16>(__float_as_uint(x), lane));
      return x + __uint_as_float(lane_xor<32>(__float_as_uint(x), lane));
    };
    const int len = length(c);
#pragma unroll 1
    for (int t = 0; t < len; ++t) {
      u32x4 kr[KS], qr[KS];
      float sk = 0.f, sq = 0.f;
      const auto lo = [](uint32_t x) { return __uint_as_float(x << 16); };
      const auto hi = [](uint32_t x) { return __uint_as_float(x & 0xffff0000u); };
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const int off = t * DK * 2 + (((4 * s + g) ^ turn(t)) << 4);
        kr[s] = *reinterpret_cast<const u32x4*>(in + L::kK + off);
        qr[s] = *reinterpret_cast<const u32x4*>(in + L::kQ + off);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sk = fmaf(hi(kr[s][i]), hi(kr[s][i]), fmaf(lo(kr[s][i]), lo(kr[s][i]), sk));
          sq = fmaf(hi(qr[s][i]), hi(qr[s][i]), fmaf(lo(qr[s][i]), lo(qr[s][i]), sq));
        }
      }
      const float fk = 1.0f / sqrtf(sum4(sk) + a.eps), fq = a.scale / sqrtf(sum4(sq) + a.eps);
      const float al = a.alpha[(row0 + t) * a.nv + sc.h], bt = a.beta[(row0 + t) * a.nv + sc.h];
      const float v = bf16_to_f32(*reinterpret_cast<const uint16_t*>(in + L::kV + t * 32 * NW + (16 * w + n16) * 2));
      float x = 0.f, y = 0.f;
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x = fmaf(S[2 * s + i / 2][2 * (i % 2)], lo(kr[s][i]) * fk, x);
          x = fmaf(S[2 * s + i / 2][2 * (i % 2) + 1], hi(kr[s][i]) * fk, x);
        }
      const float u = bt * (v - al * sum4(x));
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float s0 = fmaf(u, lo(kr[s][i]) * fk, al * S[2 * s + i / 2][2 * (i % 2)]);
          const float s1 = fmaf(u, hi(kr[s][i]) * fk, al * S[2 * s + i / 2][2 * (i % 2) + 1]);
          S[2 * s + i / 2][2 * (i % 2)] = s0;
          S[2 * s + i / 2][2 * (i % 2) + 1] = s1;
          y = fmaf(s0, lo(qr[s][i]) * fq, y);
          y = fmaf(s1, hi(qr[s][i]) * fq, y);
        }
      y = sum4(y);
      if (g == 0) {
        const int64_t oi = ((row0 + t) * a.nv + sc.h) * static_cast<int64_t>(a.dv) + dv0 + n16;
        if constexpr (OUT == kF32) static_cast<float*>(a.out)[oi] = y;
        else static_cast<uint16_t*>(a.out)[oi] = f32_to_bf16(y);
      }
    }
  };

  const uint32_t base = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_u8*)smem));
  int stage = 0;
  if (sc.c0 < sc.c1)
#pragma unroll
    for (int i = 0; i < kParts; ++i) request(sc.c0, base, i);
  constexpr int kOut = OUT == kF32 ? 4 : 2;
  const int ost = static_cast<int>(vst) * kOut;
  const uint32_t ooff = 8 * g * static_cast<uint32_t>(ost) + n16 * kOut;
  uint8_t* on = static_cast<uint8_t*>(a.out) +
                ((static_cast<int64_t>(sc.begin) + static_cast<int64_t>(sc.c0) * kC) * vst + static_cast<int64_t>(sc.h) * a.dv + dv0) * kOut;
  for (int c = sc.c0; c < sc.c1; ++c) {
    uint8_t* const in = smem + stage * L::kStage;
    stage ^= 1;
    const uint32_t other = base + stage * L::kStage;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();                           // the chunk is there, and nobody reads the other stage any more
    const bool more = c + 1 < sc.c1;
    if (idle) {
      if (more)
#pragma unroll
        for (int i = 0; i < kParts; ++i) request(c + 1, other, i);
      continue;
    }
    const float* const vec = reinterpret_cast<const float*>(in + L::kF);
    const int len = length(c);
    bool by_token = __builtin_amdgcn_readfirstlane(__float_as_int(vec[2 * kC + 1])) != 0;
    // K S^T and Q S^T
    bf16x8 Sp[KS][3];
#pragma unroll
    for (int s = 0; s < KS; ++s) split3(S[2 * s], S[2 * s + 1], Sp[s]);
    f32x4 ks[4], o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      ks[i] = o[i] = f32x4{0.f, 0.f, 0.f, 0.f};
      const int tok = token_of(i, n16);
      if (more) request(c + 1, other, i);
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const int off = tok * DK * 2 + (((4 * s + g) ^ turn(tok)) << 4);
        const bf16x8 Ka = *reinterpret_cast<const bf16x8*>(in + L::kK + off), Qa = *reinterpret_cast<const bf16x8*>(in + L::kQ + off);
#pragma unroll
        for (int x = 2; x >= 0; --x) {
          ks[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(Ka, Sp[s][x], ks[i], 0, 0, 0);
          if (x < OP) o[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(Qa, Sp[s][x], o[i], 0, 0, 0);
        }
      }
    }
    // X: tokens 8 g + 0 .. 3 and 4 .. 7 of each half of the chunk
    bf16x8 Xp[2][3];
    bool far = false;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      f32x4 x[2];
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int tok = 32 * s + 8 * g + 4 * y;
        const bf16x4 v = transposed(in + L::kV + (tok + (n16 >> 2)) * 32 * NW + (16 * w + 4 * (n16 & 3)) * 2);
        const f32x4 e = *reinterpret_cast<const f32x4*>(vec + tok), f = *reinterpret_cast<const f32x4*>(vec + kC + tok);
#pragma unroll
        for (int r = 0; r < 4; ++r) x[y][r] = static_cast<float>(v[r]) - e[r] * ks[2 * s + y][r];
        o[2 * s + y] *= f;
        far |= far4(x[y]);
      }
      split3(x[0], x[1], Xp[s]);
    }
    if (by_token || __ballot(far)) {           // outside the range of the matrices, or not finite
      tokens(c, in);
      on += static_cast<int64_t>(kC) * ost;
      continue;
    }
    // (Z-matrix) X and (O-matrix) X, the smallest terms first
    f32x4 z[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      z[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s <= i / 2; ++s) {
        const uint8_t* m = in + L::kM + piece_of(i, s) * 1024 + lane * 16;
        bf16x8 Tz[3], To[OP];
#pragma unroll
        for (int x = 0; x < 3; ++x) Tz[x] = *reinterpret_cast<const bf16x8*>(m + x * kMatBf16);
#pragma unroll
        for (int x = 0; x < OP; ++x) To[x] = *reinterpret_cast<const bf16x8*>(m + (3 + x) * kMatBf16);
#pragma unroll
        for (int y = 2; y >= 0; --y)
#pragma unroll
          for (int x = 2 - y; x >= 0; --x) {
            z[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(Tz[x], Xp[s][y], z[i], 0, 0, 0);
            if (x + y < OP) o[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(To[x], Xp[s][y], o[i], 0, 0, 0);
          }
      }
    }
    // rows 32 s + 8 g + 4 y + r; those behind the last token are beyond the descriptor's end
    const auto ro = __builtin_amdgcn_make_buffer_rsrc(on, 0, (len - 1) * ost + kRowsS * kOut, 0x00020000);
    on += static_cast<int64_t>(kC) * ost;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint32_t off = ooff + static_cast<uint32_t>((32 * (i >> 1) + 4 * (i & 1) + r) * ost);
        if constexpr (OUT == kF32) __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(o[i][r]), ro, off, 0, 0);
        else __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, static_cast<__bf16>(o[i][r])), ro, off, 0, 0);
      }
    // S^T
    bf16x8 Zp[2][3];
#pragma unroll
    for (int s = 0; s < 2; ++s) split3(z[2 * s], z[2 * s + 1], Zp[s]);
    const float gC = vec[2 * kC];
#pragma unroll
    for (int t = 0; t < 2 * KS; ++t) {
      f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        bf16x8 Ka;                             // row m of the tile is column 32 (t / 2) + 8 (m / 4) + 4 (t % 2) + m % 4; tokens 32 s + 8 g ..
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int tok = 32 * s + 8 * g + 4 * y + (n16 >> 2);
          const bf16x4 v = transposed(in + L::kK + tok * DK * 2 + (((4 * (t >> 1) + (n16 & 3)) ^ turn(tok)) << 4) + 8 * (t & 1));
#pragma unroll
          for (int i = 0; i < 4; ++i) Ka[4 * y + i] = v[i];
        }
#pragma unroll
        for (int x = 2; x >= 0; --x) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(Ka, Zp[s][x], d, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) S[t][i] = fmaf(gC, S[t][i], d[i]);
    }
  }
  if (!idle)
#pragma unroll
    for (int t = 0; t < 2 * KS; ++t) *reinterpret_cast<f32x4*>(a.state_out + so + 32 * (t >> 1) + 8 * g + 4 * (t & 1)) = S[t];
}

// fp32 activations, on the fp32 matrix instruction.
template <int DK, int OUT>
__global__ __launch_bounds__(256) void k_gdc_scan_f32(GdcArgs a) {
  constexpr int ACT = kF32;
  constexpr int KS = DK / 16;
  constexpr int NT = DK / 64;                  // tiles of 16 state columns a wave
  constexpr int kLs = DK + 4, kLx = kC + 4;
  __shared__ __align__(16) float Ss[kRowsS * kLs];
  __shared__ __align__(16) float Ks[kC * kLs];
  __shared__ __align__(16) float Xs[kRowsS * kLx];
  __shared__ __align__(16) float Zs[kRowsS * kLx];
  __shared__ int far[4];                       // whether a wave's part of X is out of range
  const int tid = threadIdx.x, lane = tid & (kWave - 1), w = tid / kWave;
  const int n16 = lane & 15, g = lane >> 4;
  Scan sc;
  if (!find_scan<kRowsS>(a, DK, sc)) return;
  const int h = sc.h, kh = sc.kh, b = sc.b, begin = sc.begin, n = sc.n, c0 = sc.c0, c1 = sc.c1, dv0 = sc.dv0;
  const int64_t so = sc.state;
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
    const float* vec = reinterpret_cast<const float*>(a.ws + (slot_of(a, b, begin, c) * a.nv + h) * slot_bytes(kF32, OUT));
    const float* slot_p = vec + kVec;
    if (vec[2 * kC + 1] != 0.f) {
      chunk_by_token<DK, ACT, OUT>(a, Ss, kLs, row0, len, h, kh, dv0, lane, w);
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
      x[r] = v - vec[i] * ks[r];
      qs[r] *= vec[kC + i];
    }
    *reinterpret_cast<f32x4*>(Xs + n16 * kLx + 16 * w + 4 * g) = x;
    if (lane == 0) far[w] = 0;
    if (far4(x)) far[w] = 1;
    __syncthreads();
    if ((far[0] | far[1] | far[2] | far[3]) != 0) {   // out of range: S is as it was
      chunk_by_token<DK, ACT, OUT>(a, Ss, kLs, row0, len, h, kh, dv0, lane, w);
      __syncthreads();
      continue;
    }
    f32x4 zt = {0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s <= w; ++s) {
      const f32x4 Tz = *reinterpret_cast<const f32x4*>(slot_p + (16 * w + n16) * kC + 16 * s + 4 * g);
      const f32x4 To = *reinterpret_cast<const f32x4*>(slot_p + kC * kC + (16 * w + n16) * kC + 16 * s + 4 * g);
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
    const float gc = vec[2 * kC];
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
  const int64_t each = static_cast<int64_t>(d->n_v_heads) * slot_bytes(d->act_dtype, d->out_dtype);
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

// Whether two stages of a block of eight waves fit the LDS of a CU.
template <int DK, int OUT>
constexpr bool kHasWide = ScanLds<DK, OUT, 8>::kBytes <= 160 * 1024;

// Launch with dynamic LDS, whose size is set once per kernel and device.
template <void (*KERNEL)(GdcArgs), int BYTES, int NW>
bool launch_scan(const GdcArgs& a, uint32_t blocks, hipStream_t s) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return false;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (!bit || !(done.load(std::memory_order_relaxed) & bit)) {
    if (hipFuncSetAttribute(reinterpret_cast<const void*>(KERNEL), hipFuncAttributeMaxDynamicSharedMemorySize, BYTES) != hipSuccess)
      return false;
    done.fetch_or(bit, std::memory_order_relaxed);
  }
  launch_kernel(KERNEL, dim3(blocks), dim3(64 * NW), BYTES, s, a);
  return true;
}

// State rows a block of the scan takes.  A chunk takes a block of 16 rows 3.0 us
// (two on a CU; 2.2 alone), one of 64 rows 4.0 and one of 128 rows 6.2 (128 x 128
// states, one on a CU).  The longest sequence's chunks run one after the other, and
// all of them share the chip: the larger of the two is what a width takes, and the
// smallest wins.  1, 2, 3, 4 and 8 sequences of 1024 tokens by 32 heads: 16 rows 35,
// 47, 75, 86 and 196 us; 64 rows 59, 62, 62, 64 and 126; 128 rows 79, 81, 83, 83 and 96.
int scan_width(const gdn_desc* d, int32_t B, int32_t N, int T_max) {
  if (d->act_dtype == MOE_F32) return kRowsS;
  const bool fits = d->d_k == 64 ? kHasWide<64, kF32> : (d->out_dtype == MOE_F32 ? kHasWide<128, kF32> : kHasWide<128, kBF16>);
  const double chain = (T_max + kC - 1) / kC, mean = static_cast<double>(N) / kC / B + 0.5, heads = static_cast<double>(B) * d->n_v_heads;
  int best = kRowsS;
  double least = 1e300;
  for (const int w : {16, 64, 128}) {
    if (w == 128 && (!fits || d->d_v <= 64)) continue;
    const double t = w == 16 ? 3.0 : (w == 64 ? 4.0 : 6.2), slots = w == 16 ? 512 : 256;
    const double blocks = heads * ((d->d_v + w - 1) / w);
    const double one = w == 16 && blocks <= 256 ? 2.2 : t;
    const double took = std::max(chain * one, std::ceil(blocks / slots) * mean * t);
    if (took < least) {
      least = took;
      best = w;
    }
  }
  return best;
}

template <int DK, int OUT>
bool launch_out(const GdcArgs& a, bool f32, int width, uint32_t prep, uint32_t scan, hipStream_t s) {
  if (f32) {
    if (prep > 0) launch_kernel(k_gdc_prep<DK, kF32, OUT>, dim3(prep), dim3(256), 0, s, a);
    launch_kernel(k_gdc_scan_f32<DK, OUT>, dim3(scan), dim3(256), 0, s, a);
    return true;
  }
  if (prep > 0) launch_kernel(k_gdc_prep<DK, kBF16, OUT>, dim3(prep), dim3(256), 0, s, a);
  if (width == kRowsS) {
    launch_kernel(k_gdc_scan_few<DK, OUT>, dim3(scan), dim3(256), 0, s, a);
    return true;
  }
  if constexpr (kHasWide<DK, OUT>)
    if (width == 128) return launch_scan<k_gdc_scan_bf16<DK, OUT, 8>, ScanLds<DK, OUT, 8>::kBytes, 8>(a, scan, s);
  return launch_scan<k_gdc_scan_bf16<DK, OUT, 4>, ScanLds<DK, OUT, 4>::kBytes, 4>(a, scan, s);
}

bool launch(const GdcArgs& a, const gdn_desc* d, int width, uint32_t prep, uint32_t scan, hipStream_t s) {
  const bool f32 = d->act_dtype == MOE_F32;
  if (d->d_k == 128)
    return d->out_dtype == MOE_F32 ? launch_out<128, kF32>(a, f32, width, prep, scan, s) : launch_out<128, kBF16>(a, f32, width, prep, scan, s);
  return d->out_dtype == MOE_F32 ? launch_out<64, kF32>(a, f32, width, prep, scan, s) : launch_out<64, kBF16>(a, f32, width, prep, scan, s);
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
  a.ws = static_cast<uint8_t*>(workspace);
  a.B = B; a.N = N; a.T_max = T_max < N ? T_max : N;
  a.nk = d->n_k_heads; a.nv = d->n_v_heads; a.dv = d->d_v;
  a.scale = d->scale; a.eps = d->eps;
  a.per_pass = p.per_pass;
  a.slots = p.slots;
  const int width = scan_width(d, B, N, a.T_max);
  const int64_t heads = static_cast<int64_t>(B) * d->n_v_heads;
  const int64_t scan = (heads + 7) / 8 * 8 * ((d->d_v + width - 1) / width), prep = static_cast<int64_t>(p.slots) * d->n_v_heads;
  // a launch takes fewer than 2^32 threads
  if (scan >= (width == 128 ? 1 << 23 : 1 << 24) || prep >= (1 << 24)) return bad("B=%lld sequences of N=%lld tokens are too many blocks for one launch", B, N);
  const int chunks = (a.T_max + kC - 1) / kC;
  hipStream_t s = static_cast<hipStream_t>(stream);
  for (a.first = 0; a.first == 0 || a.first < chunks; a.first += a.per_pass) {
    const uint32_t np = chunks > 0 ? static_cast<uint32_t>(prep) : 0u, nb = static_cast<uint32_t>(scan);
    const bool sent = launch(a, d, width, np, nb, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !sent) {
      char buf[256];
      snprintf(buf, sizeof(buf), "chunked delta rule launch failed: %s", hipGetErrorString(e));
      return api_fail(MOE_EHIP, buf);
    }
    if (a.per_pass == 0) break;
  }
  return api_ok();
}
