// Attention of new tokens over the paged cache (include/attention.h, gfx950).
//
//   out_r = sum_j p_rj v_j / sum_j p_rj,   p_rj = exp(scale q_r . k_j - m_r)
//
// in one pass over the keys with the running maximum m and sum l of a row; O is
// scaled by exp(m_old - m_new) where a maximum grows.  The query heads that
// share a key head, and the new tokens of a sequence, are the rows of one
// product: row r stands for token r / each, query head h each + r % each.
//
// Both products run transposed, S^T = K Q^T and O^T = V^T P^T: a lane of the
// matrix unit's result then holds four consecutive keys (or dims) of ONE row,
// so a row's maximum, sum and scale are one value a lane, and P^T, as it comes
// out of S^T, is already the operand that the second product takes.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdio>

#include "attn_internal.h"
#include "moe_internal.h"
#include "topk_wave.h"

namespace moe {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

struct AttnArgs {
  AttnBatch at;
  const uint64_t* tree;
  const void* q;
  const void* pages;
  void* out;
  float* part;          // [N n_q][splits][D] sums, where keys are split
  float* ml;            // [N n_q][splits][2] their maxima and denominators
  int nq, nkv, each;
  int new_max, len_max;
  int tiles;            // row tiles a sequence and key head
  int splits, chunk;    // keys a split, a multiple of what a block takes a step
  float scale2;         // scale log2 e
};

// What one block works on; false: nothing.
struct Rows {
  int b, h, tile, split;
  int begin, n;         // first row of the sequence, its new tokens (at most new_max)
  int prefix;           // tokens before the new ones (negative: the first new ones are not in the sequence)
  int len;              // tokens that may be seen
};

__device__ __forceinline__ bool find_rows(const AttnArgs& a, int64_t blk, Rows& r) {
  // the row tiles that read the same keys go to one XCD (blocks are dealt out
  // in turns over eight)
  int64_t unit;
  if (a.tiles > 1) {
    const int64_t pos = blk / 8;
    unit = (pos / a.tiles) * 8 + blk % 8;
    r.tile = static_cast<int>(pos % a.tiles);
  } else {
    unit = blk;
    r.tile = 0;
  }
  if (unit >= static_cast<int64_t>(a.at.B) * a.nkv * a.splits) return false;
  r.split = static_cast<int>(unit % a.splits);
  const int64_t bh = unit / a.splits;
  r.h = static_cast<int>(bh % a.nkv);
  r.b = static_cast<int>(bh / a.nkv);
  const int begin = a.at.cu[r.b], end = a.at.cu[r.b + 1];
  if (begin < 0 || end > a.at.N || end <= begin) return false;
  r.begin = begin;
  const int n = end - begin;
  r.n = n < a.new_max ? n : a.new_max;
  const int64_t room = static_cast<int64_t>(a.at.max_pages) << a.at.shift;
  const int len = a.at.lens[r.b];
  r.prefix = (len > 0 ? len : 0) - n;
  int64_t seen = len < a.len_max ? len : a.len_max;
  if (seen > room) seen = room;
  r.len = seen > 0 ? static_cast<int>(seen) : 0;
  return true;
}

__device__ __forceinline__ int page_at(const AttnArgs& a, int b, int key) {
  return a.at.table[static_cast<int64_t>(b) * a.at.max_pages + (key >> a.at.shift)];
}

// Offset in elements of a key of head h; page 0 stands in for one that is not there.
template <int D>
__device__ __forceinline__ int64_t key_at(const AttnArgs& a, int page, int h, int key) {
  const int64_t p = page >= 0 && page < a.at.n_pages ? page : 0;
  return p * a.at.page_elems + ((static_cast<int64_t>(h) << a.at.shift) + (key & ((1 << a.at.shift) - 1))) * D;
}

// Whether new token i sees new token j (negative: one before the new ones, seen
// by all), 0 or 1: what the tree says, or the tokens up to itself.  Without
// branches.
__device__ __forceinline__ uint32_t sees(bool tree, uint64_t mask, int i, int j) {
  const uint32_t bit = (static_cast<uint32_t>(mask >> (j & 63)) & 1u) & static_cast<uint32_t>(j < 64);
  return static_cast<uint32_t>(j < 0) | (tree ? bit : static_cast<uint32_t>(j <= i));
}

__device__ __forceinline__ float xor_max(float x, int lane) {
  x = fmaxf(x, __uint_as_float(lane_xor<16>(__float_as_uint(x), lane)));
  return fmaxf(x, __uint_as_float(lane_xor<32>(__float_as_uint(x), lane)));
}
__device__ __forceinline__ float xor_add(float x, int lane) {
  x = x + __uint_as_float(lane_xor<16>(__float_as_uint(x), lane));
  return x + __uint_as_float(lane_xor<32>(__float_as_uint(x), lane));
}

// Four bf16 of consecutive rows of one column from a wave's tile of V in LDS:
// lane 4 r + c of 16 names row r, columns 4 c .. 4 c + 3 and gets column
// 4 r + c of the four rows.
__device__ __forceinline__ bf16x4 read_tr(const uint8_t* p) {
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  return __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p));
}

// The joined sums of a block's waves go out: divided and rounded, or as one
// split's part.  `sum` holds dims [c0, c0 + 4) of row r of the tile.
template <int DT, int D>
__device__ __forceinline__ void store_row(const AttnArgs& a, const Rows& r, int row, int c0, const float (&sum)[4], float m, float l) {
  const int64_t token = r.begin + row / a.each;
  const int64_t o = token * a.nq + r.h * a.each + row % a.each;
  if (a.splits > 1) {
    *reinterpret_cast<f32x4*>(a.part + (o * a.splits + r.split) * D + c0) = f32x4{sum[0], sum[1], sum[2], sum[3]};
    if (c0 == 0) {
      a.ml[(o * a.splits + r.split) * 2] = m;
      a.ml[(o * a.splits + r.split) * 2 + 1] = l;
    }
    return;
  }
  const float inv = l == 0.f ? 0.f : 1.0f / l;
  if constexpr (DT == kF32) {
    *reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + o * D + c0) = f32x4{sum[0] * inv, sum[1] * inv, sum[2] * inv, sum[3] * inv};
  } else {
    uint2 w;
    w.x = f32_to_bf16(sum[0] * inv) | (static_cast<uint32_t>(f32_to_bf16(sum[1] * inv)) << 16);
    w.y = f32_to_bf16(sum[2] * inv) | (static_cast<uint32_t>(f32_to_bf16(sum[3] * inv)) << 16);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + o * D + c0) = w;
  }
}

// Weight of a part whose maximum is m among parts whose largest is M.
__device__ __forceinline__ float part_weight(float m, float l, float M) { return l == 0.f ? 0.f : __builtin_amdgcn_exp2f(m - M); }

// ---------------------------------------------------------------------------
// Few rows: a block takes 16 RT rows of a key head and a run of its keys, its
// four waves in turn 32 keys each; they join at the end.
//
// The reads of K and V bound it.  K goes from memory straight into the operand
// of S^T (a lane reads 16 bytes of one key), V through registers and LDS, where
// the transposing read gives four keys of a dim; the next 32 keys are
// requested before the current ones are worked on.
template <int D, int RT>
struct FewLds {
  static constexpr int kKeys = 32;
  static constexpr int kV = kKeys * D * 2;                 // a wave's tile of V
  static constexpr int kCut = RT == 4 ? 32 : 64;           // dims joined at once
  static constexpr int kRow = kCut + 4;
  static constexpr int kJoin = 4 * 16 * RT * kRow * 4 + 4 * 16 * RT * 2 * 4;
  static constexpr int kBytes = 4 * kV > kJoin ? 4 * kV : kJoin;
};

template <int D, int RT>
__global__ __launch_bounds__(256) void k_attn_few(AttnArgs a) {
  using L = FewLds<D, RT>;
  constexpr int KS = D / 32;                 // steps of 32 dims
  constexpr int DT = D / 16;                 // tiles of 16 dims
  constexpr int VL = D * 2 * 32 / 16 / 64;   // 16-byte pieces of a V tile a lane
  __shared__ __align__(16) uint8_t smem[L::kBytes];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = threadIdx.x / kWave;
  const int n16 = lane & 15, g = lane >> 4;
  Rows r;
  if (!find_rows(a, blockIdx.x, r)) return;
  const int rows = r.n * a.each;
  const int row0 = r.tile * 16 * RT;
  if (row0 >= rows) return;
  const bool tree = a.tree != nullptr;

  // what the tile's last row sees at most
  int kend = r.len;
  if (!tree) {
    const int last = (row0 + 16 * RT < rows ? row0 + 16 * RT : rows) - 1;
    const int most = r.prefix + last / a.each + 1;
    if (most < kend) kend = most > 0 ? most : 0;
  }
  const int64_t k0 = static_cast<int64_t>(r.split) * a.chunk;
  const int kbeg = k0 < kend ? static_cast<int>(k0) : kend;
  if (kend - kbeg > a.chunk) kend = kbeg + a.chunk;

  // this lane's row of each of the RT tiles
  bf16x8 Q[RT][KS];
  int itok[RT];
  uint64_t mask[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int row = row0 + 16 * t + n16;
    const int rr = row < rows ? row : rows - 1;
    itok[t] = rr / a.each;
    const int64_t token = r.begin + itok[t];
    mask[t] = tree ? a.tree[token] : 0;
    const uint16_t* q = static_cast<const uint16_t*>(a.q) + (token * a.nq + r.h * a.each + rr % a.each) * D;
#pragma unroll
    for (int s = 0; s < KS; ++s) Q[t][s] = __builtin_bit_cast(bf16x8, load16(q + 32 * s + 8 * g));
  }
  f32x4 O[RT][DT];
  float m[RT], l[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    m[t] = -INFINITY;
    l[t] = 0.f;
#pragma unroll
    for (int d = 0; d < DT; ++d) O[t][d] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  const uint16_t* pool = static_cast<const uint16_t*>(a.pages);
  uint8_t* vt = smem + wave * L::kV;
  // piece j of a V tile: 16 bytes at (row, column) of lane + 64 j in row order,
  // kept at the column turned by the row so that the transposing reads of
  // eight rows fall into different banks
  constexpr int kPer = D * 2 / 16;           // pieces a row
  const auto turn = [](int row) { return D == 64 ? ((row >> 1) & 3) * 2 : (row & 7) * 2; };

  u32x4 Kn[2][KS], Vn[VL];
  bool okn[2];
  const auto request = [&](int kt) {         // the 32 keys from kt on
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      int key = kt + 16 * t + n16;
      key = key < kend ? key : kend - 1;
      const int page = page_at(a, r.b, key);
      okn[t] = page >= 0 && page < a.at.n_pages;
      const uint16_t* p = pool + key_at<D>(a, page, r.h, key);
#pragma unroll
      for (int s = 0; s < KS; ++s) Kn[t][s] = load16(p + 32 * s + 8 * g);
    }
#pragma unroll
    for (int j = 0; j < VL; ++j) {
      const int piece = lane + 64 * j;
      int key = kt + piece / kPer;
      key = key < kend ? key : kend - 1;
      const uint16_t* p = pool + a.at.half_elems + key_at<D>(a, page_at(a, r.b, key), r.h, key);
      Vn[j] = load16(p + (piece % kPer) * 8);
    }
  };

  int kt = kbeg + 32 * wave;
  if (kt < kend) request(kt);
  for (; kt < kend; kt += 128) {
    f32x4 S[RT][2];
    const bool ok0 = okn[0], ok1 = okn[1];
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        S[t][x] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < KS; ++s)
          S[t][x] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, Kn[x][s]), Q[t][s], S[t][x], 0, 0, 0);
      }
#pragma unroll
    for (int j = 0; j < VL; ++j) {
      const int piece = lane + 64 * j, row = piece / kPer, col = piece % kPer;
      *reinterpret_cast<u32x4*>(vt + row * D * 2 + ((col ^ turn(row)) << 4)) = Vn[j];
    }
    // keys that some row of the tile does not see, or that are not there
    const uint32_t there = (static_cast<uint32_t>(__ballot(ok0)) & 0xffffu) | (static_cast<uint32_t>(__ballot(ok1)) << 16);
    const bool careful = there != 0xffffffffu || kt + 32 > kend || kt + 32 > r.prefix;
    bool bad = false;                        // such a tile holds a value that is not finite
    if (careful) {
      typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
      u16x2 big = {0, 0};
#pragma unroll
      for (int j = 0; j < VL; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) big = __builtin_elementwise_max(big, __builtin_bit_cast(u16x2, Vn[j][i] & 0x7fff7fffu));
      bad = __ballot(big[0] >= 0x7f80u || big[1] >= 0x7f80u) != 0;
    }
    if (kt + 128 < kend) request(kt + 128);
    wave_sync_lds();

    bf16x8 P[RT], Plo[RT];
    uint32_t seen[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      seen[t] = 0xffu;
      if (careful) {
        seen[t] = 0;
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int at = 16 * x + 4 * g + i;
            const uint32_t in = static_cast<uint32_t>(kt + at < kend) & (there >> at);
            seen[t] |= (in & sees(tree, mask[t], itok[t], kt + at - r.prefix)) << (4 * x + i);
          }
      }
      float mx = -INFINITY;
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          S[t][x][i] *= a.scale2;
          if (careful && !((seen[t] >> (4 * x + i)) & 1u)) S[t][x][i] = -INFINITY;
          mx = fmaxf(mx, S[t][x][i]);
        }
      mx = xor_max(mx, lane);
      if (__ballot(mx > m[t])) {             // some row's maximum grows
        const float mn = fmaxf(m[t], mx);
        const float f = mn == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(m[t] - mn);
        m[t] = mn;
        l[t] *= f;
#pragma unroll
        for (int d = 0; d < DT; ++d) O[t][d] *= f;
      }
      const float mu = m[t] == -INFINITY ? 0.f : m[t];
      float add = 0.f;
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float p = __builtin_amdgcn_exp2f(S[t][x][i] - mu);
          add += p;
          // P in two bf16 parts: one alone would add an error as large as the output's own rounding
          const __bf16 hi = static_cast<__bf16>(p);
          P[t][4 * x + i] = hi;
          Plo[t][4 * x + i] = static_cast<__bf16>(p - static_cast<float>(hi));
        }
      l[t] += add;                           // this lane's keys; the four lanes of a row are joined at the end
    }
    if (!bad) {
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        // rows 4 g + r, then 16 + 4 g + r; this lane names row (n16 / 4), columns 4 (n16 % 4) ..
        bf16x8 V;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int row = 16 * x + 4 * g + (n16 >> 2);
          const int col = 2 * d + ((n16 & 3) >> 1);
          const bf16x4 v = read_tr(vt + row * D * 2 + ((col ^ turn(row)) << 4) + (n16 & 1) * 8);
#pragma unroll
          for (int i = 0; i < 4; ++i) V[4 * x + i] = v[i];
        }
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          O[t][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(V, Plo[t], O[t][d], 0, 0, 0);
          O[t][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(V, P[t], O[t][d], 0, 0, 0);
        }
      }
    } else {
      // only the rows that see a value that is not finite may take it (in the
      // product above 0 times it is NaN): key by key
      for (int kk = 0; kk < 32; ++kk) {
        const int from = n16 + 16 * ((kk & 15) >> 2), idx = 4 * (kk >> 4) + (kk & 3);
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          float p = 0.f;
#pragma unroll
          for (int x = 0; x < 8; ++x) p = x == idx ? static_cast<float>(P[t][x]) + static_cast<float>(Plo[t][x]) : p;
          p = __shfl(p, from);
          const bool s = (__shfl(static_cast<int>(seen[t]), from) >> idx) & 1;
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            const uint2 w = *reinterpret_cast<const uint2*>(vt + kk * D * 2 + (((2 * d + (g >> 1)) ^ turn(kk)) << 4) + (g & 1) * 8);
            if (s) {
              O[t][d][0] = fmaf(p, __uint_as_float(w.x << 16), O[t][d][0]);
              O[t][d][1] = fmaf(p, __uint_as_float(w.x & 0xffff0000u), O[t][d][1]);
              O[t][d][2] = fmaf(p, __uint_as_float(w.y << 16), O[t][d][2]);
              O[t][d][3] = fmaf(p, __uint_as_float(w.y & 0xffff0000u), O[t][d][3]);
            }
          }
        }
      }
    }
    wave_sync_lds();                         // the tile's reads before the next one's writes
  }

  // join the waves
  float* mlw = reinterpret_cast<float*>(smem + 4 * 16 * RT * L::kRow * 4);
  float* ow = reinterpret_cast<float*>(smem);
  __syncthreads();
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    l[t] = xor_add(l[t], lane);
    if (g == 0) {
      mlw[(wave * 16 * RT + 16 * t + n16) * 2] = m[t];
      mlw[(wave * 16 * RT + 16 * t + n16) * 2 + 1] = l[t];
    }
  }
#pragma unroll
  for (int c = 0; c < D / L::kCut; ++c) {
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int d = 0; d < L::kCut / 16; ++d)
        *reinterpret_cast<f32x4*>(ow + (wave * 16 * RT + 16 * t + n16) * L::kRow + 16 * d + 4 * g) = O[t][c * (L::kCut / 16) + d];
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * RT * (L::kCut / 4); i += 256) {
      const int row = i / (L::kCut / 4), cc = (i % (L::kCut / 4)) * 4;
      if (row0 + row < rows) {
        float M = -INFINITY, ll = 0.f, sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < 4; ++w) M = fmaxf(M, mlw[(w * 16 * RT + row) * 2]);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float lw = mlw[(w * 16 * RT + row) * 2 + 1];
          const float f = part_weight(mlw[(w * 16 * RT + row) * 2], lw, M);
          ll = fmaf(lw, f, ll);
          const f32x4 v = *reinterpret_cast<const f32x4*>(ow + (w * 16 * RT + row) * L::kRow + cc);
          if (lw != 0.f)
#pragma unroll
            for (int j = 0; j < 4; ++j) sum[j] = fmaf(v[j], f, sum[j]);
        }
        store_row<kBF16, D>(a, r, row0 + row, c * L::kCut + cc, sum, M, ll);
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// fp32: the same split of the work on the fp32 matrix instruction (16x16x4).
// Everything goes from memory to its operand: of the four dims of a 16-byte
// piece of a key, one for each of four products; V likewise, four dims of one
// key for four tiles.
template <int D, int RT>
struct F32Lds {
  static constexpr int kCut = RT == 2 ? 32 : 64;
  static constexpr int kRow = kCut + 4;
  static constexpr int kBytes = 4 * 16 * RT * kRow * 4 + 4 * 16 * RT * 2 * 4;
};

template <int D, int RT>
__global__ __launch_bounds__(256) void k_attn_f32(AttnArgs a) {
  using L = F32Lds<D, RT>;
  constexpr int KS = D / 16;                 // 16-byte pieces of a row for a lane's quarter
  constexpr int DQ = D / 64;                 // groups of 64 dims
  __shared__ __align__(16) uint8_t smem[L::kBytes];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = threadIdx.x / kWave;
  const int n16 = lane & 15, g = lane >> 4;
  Rows r;
  if (!find_rows(a, blockIdx.x, r)) return;
  const int rows = r.n * a.each;
  const int row0 = r.tile * 16 * RT;
  if (row0 >= rows) return;
  const bool tree = a.tree != nullptr;

  int kend = r.len;
  if (!tree) {
    const int last = (row0 + 16 * RT < rows ? row0 + 16 * RT : rows) - 1;
    const int most = r.prefix + last / a.each + 1;
    if (most < kend) kend = most > 0 ? most : 0;
  }
  const int64_t k0 = static_cast<int64_t>(r.split) * a.chunk;
  const int kbeg = k0 < kend ? static_cast<int>(k0) : kend;
  if (kend - kbeg > a.chunk) kend = kbeg + a.chunk;

  f32x4 Q[RT][KS];
  int itok[RT];
  uint64_t mask[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int row = row0 + 16 * t + n16;
    const int rr = row < rows ? row : rows - 1;
    itok[t] = rr / a.each;
    const int64_t token = r.begin + itok[t];
    mask[t] = tree ? a.tree[token] : 0;
    const float* q = static_cast<const float*>(a.q) + (token * a.nq + r.h * a.each + rr % a.each) * D;
#pragma unroll
    for (int s = 0; s < KS; ++s) Q[t][s] = *reinterpret_cast<const f32x4*>(q + 16 * s + 4 * g);
  }
  f32x4 O[RT][DQ][4];                        // tile (q, i): dims 64 q + 4 m + i
  float m[RT], l[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    m[t] = -INFINITY;
    l[t] = 0.f;
#pragma unroll
    for (int d = 0; d < DQ; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i) O[t][d][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  const float* pool = static_cast<const float*>(a.pages);
  for (int kt = kbeg + 16 * wave; kt < kend; kt += 64) {
    int key = kt + n16;
    key = key < kend ? key : kend - 1;
    int page = page_at(a, r.b, key);
    const uint32_t there = static_cast<uint32_t>(__ballot(page >= 0 && page < a.at.n_pages)) & 0xffffu;
    const float* kp = pool + key_at<D>(a, page, r.h, key);
    f32x4 K[KS];
#pragma unroll
    for (int s = 0; s < KS; ++s) K[s] = *reinterpret_cast<const f32x4*>(kp + 16 * s + 4 * g);
    f32x4 V[4][DQ];                          // keys 4 g + r, dims 64 q + 4 n16 ..
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      int vk = kt + 4 * g + i;
      vk = vk < kend ? vk : kend - 1;
      const float* vp = pool + a.at.half_elems + key_at<D>(a, page_at(a, r.b, vk), r.h, vk);
#pragma unroll
      for (int d = 0; d < DQ; ++d) V[i][d] = *reinterpret_cast<const f32x4*>(vp + 64 * d + 4 * n16);
    }
    const bool careful = there != 0xffffu || kt + 16 > kend || kt + 16 > r.prefix;
    bool bad = false;
    if (careful) {
      uint32_t big = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int d = 0; d < DQ; ++d)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t w = __float_as_uint(V[i][d][j]) & 0x7fffffffu;
            big = w > big ? w : big;
          }
      bad = __ballot(big >= 0x7f800000u) != 0;
    }
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      f32x4 S = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) S = __builtin_amdgcn_mfma_f32_16x16x4f32(K[s][i], Q[t][s][i], S, 0, 0, 0);
      uint32_t seen = 0xfu;
      if (careful) {
        seen = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = 4 * g + i;
          const uint32_t in = static_cast<uint32_t>(kt + at < kend) & (there >> at);
          seen |= (in & sees(tree, mask[t], itok[t], kt + at - r.prefix)) << i;
        }
      }
      float mx = -INFINITY;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        S[i] = (seen >> i) & 1u ? S[i] * a.scale2 : -INFINITY;
        mx = fmaxf(mx, S[i]);
      }
      mx = xor_max(mx, lane);
      if (__ballot(mx > m[t])) {
        const float mn = fmaxf(m[t], mx);
        const float f = mn == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(m[t] - mn);
        m[t] = mn;
        l[t] *= f;
#pragma unroll
        for (int d = 0; d < DQ; ++d)
#pragma unroll
          for (int i = 0; i < 4; ++i) O[t][d][i] *= f;
      }
      const float mu = m[t] == -INFINITY ? 0.f : m[t];
      f32x4 p;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        p[i] = __builtin_amdgcn_exp2f(S[i] - mu);
        l[t] += p[i];
      }
      if (!bad) {
#pragma unroll
        for (int d = 0; d < DQ; ++d)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) O[t][d][i] = __builtin_amdgcn_mfma_f32_16x16x4f32(V[k][d][i], p[k], O[t][d][i], 0, 0, 0);
      } else {
        // as above: key 4 kg + k for its rows only; dim 64 d + 4 (4 g + j) + i of it is with lane 4 g + j of group kg
        for (int kg = 0; kg < 4; ++kg)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float pk = __shfl(p[k], n16 + 16 * kg);
            const bool s = (__shfl(static_cast<int>(seen), n16 + 16 * kg) >> k) & 1;
#pragma unroll
            for (int d = 0; d < DQ; ++d)
#pragma unroll
              for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const float v = __shfl(V[k][d][i], 16 * kg + 4 * g + j);
                  if (s) O[t][d][i][j] = fmaf(pk, v, O[t][d][i][j]);
                }
          }
      }
    }
  }

  float* mlw = reinterpret_cast<float*>(smem + 4 * 16 * RT * L::kRow * 4);
  float* ow = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    l[t] = xor_add(l[t], lane);
    if (g == 0) {
      mlw[(wave * 16 * RT + 16 * t + n16) * 2] = m[t];
      mlw[(wave * 16 * RT + 16 * t + n16) * 2 + 1] = l[t];
    }
  }
#pragma unroll
  for (int c = 0; c < D / L::kCut; ++c) {
    // dims [kCut c, kCut (c + 1)): a lane holds 16 dims from 64 q + 16 g on
    const int q = c * L::kCut / 64;
    const int lo = c * L::kCut - 64 * q;     // 0, or 32 in the second half of 64
#pragma unroll
    for (int t = 0; t < RT; ++t)
      if (L::kCut == 64 || (16 * g >= lo && 16 * g < lo + 32))
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<f32x4*>(ow + (wave * 16 * RT + 16 * t + n16) * L::kRow + 16 * g - lo + 4 * j) =
              f32x4{O[t][q][0][j], O[t][q][1][j], O[t][q][2][j], O[t][q][3][j]};
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * RT * (L::kCut / 4); i += 256) {
      const int row = i / (L::kCut / 4), cc = (i % (L::kCut / 4)) * 4;
      if (row0 + row < rows) {
        float M = -INFINITY, ll = 0.f, sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < 4; ++w) M = fmaxf(M, mlw[(w * 16 * RT + row) * 2]);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float lw = mlw[(w * 16 * RT + row) * 2 + 1];
          const float f = part_weight(mlw[(w * 16 * RT + row) * 2], lw, M);
          ll = fmaf(lw, f, ll);
          const f32x4 v = *reinterpret_cast<const f32x4*>(ow + (w * 16 * RT + row) * L::kRow + cc);
          if (lw != 0.f)
#pragma unroll
            for (int j = 0; j < 4; ++j) sum[j] = fmaf(v[j], f, sum[j]);
        }
        store_row<kF32, D>(a, r, row0 + row, c * L::kCut + cc, sum, M, ll);
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// The splits of a row joined: D / 4 lanes a row, four dims each.
template <int DT, int D>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a) {
  constexpr int LR = D / 4;
  const int per = 256 / LR;                  // rows a block
  const int64_t steps = (static_cast<int64_t>(a.new_max) * a.nq + per - 1) / per;
  const int b = static_cast<int>(blockIdx.x / steps);
  const int64_t row = (blockIdx.x % steps) * per + threadIdx.x / LR;
  const int c0 = (threadIdx.x % LR) * 4;
  const int begin = a.at.cu[b], end = a.at.cu[b + 1];
  if (begin < 0 || end > a.at.N || end <= begin) return;
  const int n = end - begin < a.new_max ? end - begin : a.new_max;
  if (row >= static_cast<int64_t>(n) * a.nq) return;
  const int64_t o = static_cast<int64_t>(begin) * a.nq + row;
  const float* ml = a.ml + o * a.splits * 2;
  const float* part = a.part + o * a.splits * D + c0;
  float M = -INFINITY;
  for (int s = 0; s < a.splits; ++s) M = fmaxf(M, ml[2 * s]);
  float l = 0.f, sum[4] = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < a.splits; ++s) {
    const float ls = ml[2 * s + 1];
    if (ls == 0.f) continue;
    const float f = part_weight(ml[2 * s], ls, M);
    l = fmaf(ls, f, l);
    const f32x4 v = *reinterpret_cast<const f32x4*>(part + static_cast<int64_t>(s) * D);
#pragma unroll
    for (int j = 0; j < 4; ++j) sum[j] = fmaf(v[j], f, sum[j]);
  }
  const float inv = l == 0.f ? 0.f : 1.0f / l;
  if constexpr (DT == kF32) {
    *reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + o * D + c0) = f32x4{sum[0] * inv, sum[1] * inv, sum[2] * inv, sum[3] * inv};
  } else {
    uint2 w;
    w.x = f32_to_bf16(sum[0] * inv) | (static_cast<uint32_t>(f32_to_bf16(sum[1] * inv)) << 16);
    w.y = f32_to_bf16(sum[2] * inv) | (static_cast<uint32_t>(f32_to_bf16(sum[3] * inv)) << 16);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + o * D + c0) = w;
  }
}

// ---------------------------------------------------------------------------
struct AttnPlan {
  int rt;               // tiles of 16 rows a block
  int tiles;            // row tiles a sequence and key head
  int splits, chunk;
  int64_t blocks;
  size_t part, total;   // workspace: sums, then maxima and denominators
};

int attn_plan(const attn_desc* d, int32_t B, int32_t N, int32_t new_max, int32_t len_max, AttnPlan* p) {
  if (B < 0 || B > (1 << 16) || N < 0 || N > (1 << 20)) return attn_bad("B=%lld must be in [0, 2^16], N=%lld in [0, 2^20]", B, N);
  if (new_max < 0 || len_max < 0 || len_max > 0x7ffff000) return attn_bad("new_max=%lld and len_max=%lld must not be negative or too large", new_max, len_max);
  const int each = d->n_q_heads / d->n_kv_heads;
  const int most = new_max < N ? new_max : N;
  const int64_t rows = static_cast<int64_t>(most) * each;
  const int cap = d->dtype == MOE_F32 ? 2 : (d->head_dim == 256 ? 2 : 4);
  p->rt = rows <= 16 ? 1 : (rows <= 32 || cap == 2 ? 2 : 4);
  p->tiles = static_cast<int>((rows + 16 * p->rt - 1) / (16 * p->rt));
  if (p->tiles < 1) p->tiles = 1;
  const int step = d->dtype == MOE_F32 ? 64 : 128;
  const int64_t units = static_cast<int64_t>(B) * d->n_kv_heads * p->tiles;
  int64_t splits = units > 0 ? 1024 / units : 1;
  if (splits > 64) splits = 64;
  if (splits < 1) splits = 1;
  int64_t chunk = (len_max + splits - 1) / splits;
  chunk = (chunk + step - 1) / step * step;
  if (chunk < step) chunk = step;
  p->chunk = static_cast<int>(chunk);
  p->splits = static_cast<int>((len_max + chunk - 1) / chunk);
  if (p->splits < 1) p->splits = 1;
  const int64_t groups = static_cast<int64_t>(B) * d->n_kv_heads * p->splits;
  p->blocks = (p->tiles > 1 ? (groups + 7) / 8 * 8 : groups) * p->tiles;
  if (p->blocks >= (int64_t(1) << 24)) return attn_bad("%lld blocks are too many for one launch", p->blocks);
  p->part = 0;
  p->total = 0;
  if (p->splits > 1) {
    p->part = static_cast<size_t>(N) * d->n_q_heads * p->splits * d->head_dim * 4;
    p->total = p->part + static_cast<size_t>(N) * d->n_q_heads * p->splits * 8;
  }
  return MOE_OK;
}

template <int D>
void launch_attn_d(const AttnArgs& a, const AttnPlan& p, int dtype, hipStream_t s) {
  const dim3 grid(static_cast<uint32_t>(p.blocks)), block(256);
  if (dtype == MOE_F32) {
    if (p.rt == 1) launch_kernel(k_attn_f32<D, 1>, grid, block, 0, s, a);
    else launch_kernel(k_attn_f32<D, 2>, grid, block, 0, s, a);
  } else {
    if (p.rt == 1) launch_kernel(k_attn_few<D, 1>, grid, block, 0, s, a);
    else if (p.rt == 2) launch_kernel(k_attn_few<D, 2>, grid, block, 0, s, a);
    else if constexpr (D < 256) launch_kernel(k_attn_few<D, 4>, grid, block, 0, s, a);
  }
  if (p.splits > 1) {
    const int64_t per = 256 / (D / 4);
    const int64_t steps = (static_cast<int64_t>(a.new_max) * a.nq + per - 1) / per;
    const dim3 jg(static_cast<uint32_t>(steps * a.at.B));
    if (dtype == MOE_F32) launch_kernel(k_attn_join<kF32, D>, jg, block, 0, s, a);
    else launch_kernel(k_attn_join<kBF16, D>, jg, block, 0, s, a);
  }
}

}  // namespace
}  // namespace moe

extern "C" size_t attn_workspace_bytes(const attn_desc* d, int32_t B, int32_t N, int32_t new_max, int32_t len_max) {
  using namespace moe;
  AttnPlan p;
  if (check_attn(d) != MOE_OK || attn_plan(d, B, N, new_max, len_max, &p) != MOE_OK) return static_cast<size_t>(-1);
  api_ok();
  return B == 0 || N == 0 || new_max == 0 ? 0 : p.total;
}

extern "C" int attn_forward(const attn_desc* d, int32_t B, int32_t N, int32_t new_max, int32_t len_max, const int32_t* cu,
                            const int32_t* lens, const int32_t* table, const uint64_t* tree, const void* q,
                            const void* pages, void* out, void* workspace, size_t ws_bytes, void* stream) {
  using namespace moe;
  MarkScope marks;
  int rc;
  AttnPlan p;
  if ((rc = check_attn(d)) || (rc = attn_plan(d, B, N, new_max, len_max, &p))) return rc;
  if (B == 0 || N == 0 || new_max == 0) return api_ok();
  if ((rc = check_attn_batch(B, N, cu, lens, table))) return rc;
  if (!q || !pages || !out) return attn_bad("NULL q, pages or out");
  if (!attn_aligned(q, 16) || !attn_aligned(pages, 16) || !attn_aligned(out, 16)) return attn_bad("q, pages and out must be 16-byte aligned");
  if (!attn_aligned(tree, 8)) return attn_bad("tree must be 8-byte aligned");
  if (tree && new_max > 64) return attn_bad("new_max=%lld: a tree brings at most 64 tokens a sequence", new_max);
  if (p.total > 0) {
    if (!workspace || !attn_aligned(workspace, 256)) return attn_bad("the workspace is NULL or not 256-byte aligned");
    if (ws_bytes < p.total) {
      char buf[256];
      snprintf(buf, sizeof(buf), "workspace of %zu bytes, %zu needed", ws_bytes, p.total);
      return api_fail(MOE_ENOMEM, buf);
    }
  }
  const AttnBatch at = attn_batch(d, B, N, cu, lens, table);
  const int64_t sz = d->dtype == MOE_F32 ? 4 : 2, n_q = static_cast<int64_t>(N) * d->n_q_heads * d->head_dim * sz;
  const void* ins[] = {q, pages, cu, lens, table, tree};
  const int64_t in_n[] = {n_q, d->n_pages * at.page_elems * sz, (B + 1) * int64_t(4), B * int64_t(4),
                          static_cast<int64_t>(B) * d->max_pages * 4, N * int64_t(8)};
  for (int i = 0; i < 6; ++i)
    if (attn_overlaps(out, n_q, ins[i], in_n[i]) || attn_overlaps(workspace, static_cast<int64_t>(p.total), ins[i], in_n[i]))
      return attn_bad("out or the workspace overlaps input %lld", i);
  if (attn_overlaps(workspace, static_cast<int64_t>(p.total), out, n_q)) return attn_bad("out overlaps the workspace");

  AttnArgs a{};
  a.at = at;
  a.tree = tree;
  a.q = q;
  a.pages = pages;
  a.out = out;
  a.part = static_cast<float*>(workspace);
  a.ml = p.total ? reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + p.part) : nullptr;
  a.nq = d->n_q_heads;
  a.nkv = d->n_kv_heads;
  a.each = a.nq / a.nkv;
  a.new_max = new_max < N ? new_max : N;
  a.len_max = len_max;
  a.tiles = p.tiles;
  a.splits = p.splits;
  a.chunk = p.chunk;
  a.scale2 = d->scale * 1.4426950408889634f;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (d->head_dim == 64) launch_attn_d<64>(a, p, d->dtype, s);
  else if (d->head_dim == 128) launch_attn_d<128>(a, p, d->dtype, s);
  else launch_attn_d<256>(a, p, d->dtype, s);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) {
    char buf[256];
    snprintf(buf, sizeof(buf), "attention launch failed: %s", hipGetErrorString(e));
    return api_fail(MOE_EHIP, buf);
  }
  return api_ok();
}
