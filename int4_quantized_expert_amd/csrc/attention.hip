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

#include <atomic>
#include <cfloat>
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
  float* part;          // even: [blocks][2][rows of a tile][D] sums
  float* ml;            // even: [blocks][2][rows of a tile][2] their maxima and denominators
  int* shares;          // even: steps a block, then the steps up to and with each sequence
  int nq, nkv, each;
  int new_max, len_max;
  int tiles;            // row tiles a sequence and key head, at most
  int blocks;
  float scale2;         // |scale| log2 e, not 0
  uint32_t flip;        // the sign bits of q, set where scale is negative
};

// One unit of work: a tile of rows of one key head of one sequence.
struct Rows {
  int b, h, tile;
  int begin, n;         // first row of the sequence, its new tokens (at most new_max)
  int prefix;           // tokens before the new ones (negative: the first new ones are not in the sequence)
  int len;              // tokens that may be seen
};

// Sequence b; false: it brings no token, or does not fit the rows.
__device__ __forceinline__ bool sequence(const AttnArgs& a, int b, Rows& r) {
  const int begin = a.at.cu[b], end = a.at.cu[b + 1], len = a.at.lens[b];
  r.b = b;
  r.begin = begin;
  const int n = end - begin;
  r.n = n < a.new_max ? n : a.new_max;
  const int64_t room = static_cast<int64_t>(a.at.max_pages) << a.at.shift;
  r.prefix = (len > 0 ? len : 0) - n;
  int64_t seen = len < a.len_max ? len : a.len_max;
  if (seen > room) seen = room;
  r.len = seen > 0 ? static_cast<int>(seen) : 0;
  return begin >= 0 && end <= a.at.N && end > begin;
}

// What the rows [row0, row0 + count) of a sequence see at most.
__device__ __forceinline__ int last_key(const AttnArgs& a, const Rows& r, int row0, int count) {
  if (a.tree) return r.len;
  const int rows = r.n * a.each;
  const int last = (row0 + count < rows ? row0 + count : rows) - 1;
  const int most = r.prefix + last / a.each + 1;
  return most < r.len ? (most > 0 ? most : 0) : r.len;
}

// Even shares.  The units in order (sequence, key head, tile) have as many
// steps of STEP keys each as the sequence has; every block takes a share of
// all steps, so a long context is many blocks' work and a block takes many
// short ones.  A block finishes all units but, at most, the first and the last
// of its share; their sums go to the workspace and are joined by a second launch,
// which finds the share and the steps before each sequence there too.
template <int STEP>
__device__ __forceinline__ int steps_of(const Rows& r) { return (r.len + STEP - 1) / STEP; }
template <int ROWS>
__device__ __forceinline__ int tiles_of(const AttnArgs& a, const Rows& r) { return (r.n * a.each + ROWS - 1) / ROWS; }

// Steps of sequence b; all of them together are below 2^31 (the host sees to that).
template <int ROWS, int STEP>
__device__ __forceinline__ int work_of(const AttnArgs& a, int b) {
  Rows r;
  if (b >= a.at.B || !sequence(a, b, r)) return 0;
  return a.nkv * tiles_of<ROWS>(a, r) * steps_of<STEP>(r);
}

__device__ __forceinline__ int wave_scan(int x, int lane) {      // inclusive
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const int o = __shfl_up(x, d);
    x += lane >= d ? o : 0;
  }
  return x;
}

// Calls unit(rows, first key, last key + 1, whole, slot) for everything that
// this block works on; not whole: the sums go to its slot.
template <int ROWS, int STEP, bool EVEN, typename F>
__device__ __forceinline__ void walk(const AttnArgs& a, int lane, F unit) {
  Rows r;
  if constexpr (!EVEN) {
    // The last row tiles first: they see the most keys.  Blocks are dealt out in
    // turns over eight XCDs; with a power of two of heads the tiles that read the
    // same keys meet in the same XCDs' caches.
    const int heads = a.at.B * a.nkv;
    const int bh = blockIdx.x % heads;
    r.tile = a.tiles - 1 - static_cast<int>(blockIdx.x / heads);
    r.h = bh % a.nkv;
    if (!sequence(a, bh / a.nkv, r) || r.tile >= tiles_of<ROWS>(a, r)) return;
    unit(r, 0, last_key(a, r, r.tile * ROWS, ROWS), true, 0);
  } else {
    const bool writes = blockIdx.x == 0 && threadIdx.x < kWave;
    // all steps, and with a batch that one wave holds the steps up to each sequence
    int in = wave_scan(work_of<ROWS, STEP>(a, lane), lane);
    int total = __shfl(in, kWave - 1);
    if (writes && lane < a.at.B) a.shares[1 + lane] = in;
    for (int i = kWave; i < a.at.B; i += kWave) {
      const int more = total + wave_scan(work_of<ROWS, STEP>(a, i + lane), lane);
      if (writes && i + lane < a.at.B) a.shares[1 + i + lane] = more;
      total = __shfl(more, kWave - 1);
    }
    total = __builtin_amdgcn_readfirstlane(total);
    const int per = total > 0 ? (total + a.blocks - 1) / a.blocks : 1;
    if (writes && lane == 0) a.shares[0] = per;
    // neighbouring shares, which may be of one sequence, are neighbouring blocks and go to different XCDs
    if (static_cast<int64_t>(blockIdx.x) * per >= total) return;
    const int first = static_cast<int>(blockIdx.x) * per;
    const int end = total - first < per ? total : first + per;
    int pos = first, b = 0, rem = first;
    for (int i = 0;; i += kWave) {
      const int n = __popcll(__ballot(in <= first));         // sequences that end before the share
      b = i + n;
      if (n > 0) rem = first - __shfl(in, n - 1);
      if (n < kWave || i + kWave >= a.at.B) break;
      in = __shfl(in, kWave - 1) + wave_scan(work_of<ROWS, STEP>(a, i + kWave + lane), lane);
    }
    b = __builtin_amdgcn_readfirstlane(b);
    rem = __builtin_amdgcn_readfirstlane(rem);
    while (pos < end && b < a.at.B) {
      const bool ok = sequence(a, b, r);
      const int steps = ok ? steps_of<STEP>(r) : 0, tiles = tiles_of<ROWS>(a, r);
      const int all = a.nkv * tiles * steps;
      if (rem >= all) {
        rem -= all;
        ++b;
        continue;
      }
      const int idx = rem / steps, step = rem % steps;
      const int count = steps - step < end - pos ? steps - step : end - pos;
      r.h = idx / tiles;
      r.tile = idx % tiles;
      const int most = last_key(a, r, r.tile * ROWS, ROWS);
      const int k1 = (step + count) * STEP;
      unit(r, step * STEP, k1 < most ? k1 : most, count == steps, pos == first ? 0 : 1);
      pos += count;
      rem += count;
    }
  }
}

__device__ __forceinline__ int page_at(const AttnArgs& a, int b, int key) {
  return a.at.table[static_cast<int64_t>(b) * a.at.max_pages + (key >> a.at.shift)];
}

// The page that holds a key, 0 in place of one that is not there.
__device__ __forceinline__ bool there(const AttnArgs& a, int page) {
  return (static_cast<uint32_t>(page >= 0) & static_cast<uint32_t>(page < a.at.n_pages)) != 0;
}

// Offset in elements of a key of head h.
template <int D>
__device__ __forceinline__ int64_t key_at(const AttnArgs& a, int page, int h, int key) {
  const int64_t p = there(a, page) ? page : 0;
  return p * a.at.page_elems + ((static_cast<int64_t>(h) << a.at.shift) + (key & ((1 << a.at.shift) - 1))) * D;
}

// A direct load of 16 bytes a lane as lds_load<16>, each lane from an address of its own.
__device__ __forceinline__ void lds_load_at(const void* p, uint8_t* lds) {
  const uint32_t la = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_u8*)lds)));
  uint32_t saved;
  asm volatile(
      "s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, off\n\ts_mov_b32 m0, %0"
      : "=&s"(saved)
      : "s"(la), "v"(p)
      : "memory");
}

__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// Whether new token i sees new token j (negative: one before the new ones, seen
// by all), 0 or 1: what the tree says, or the tokens up to itself.  Without
// branches.
__device__ __forceinline__ uint32_t sees(bool tree, uint64_t mask, int i, int j) {
  const uint32_t bit = (static_cast<uint32_t>(mask >> (j & 63)) & 1u) & static_cast<uint32_t>(j < 64);
  return static_cast<uint32_t>(j < 0) | (tree ? bit : static_cast<uint32_t>(j <= i));
}

// A row's maximum may be exceeded by this much (in powers of two) before its
// sums are scaled again: weights of up to 2^8 lose nothing in fp32 or bf16.
constexpr float kSlack = 8.f;

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

// Values that are not finite.  0 times them is NaN, so a product over all keys
// would carry them to rows that do not see them.  Where a tile with unseen keys
// holds one, the product runs over the finite values (the others as 0), and a
// second one counts what each row sees of the others: +inf as 1, -inf as 128,
// NaN as 129 (both), exact in bf16 and in sums over 64 keys.
__device__ __forceinline__ bf16x8 finite_part(bf16x8 v) {
  u32x4 w = __builtin_bit_cast(u32x4, v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = (w[i] & 0x7f80u) == 0x7f80u ? 0u : w[i] & 0xffffu;
    const uint32_t hi = (w[i] & 0x7f800000u) == 0x7f800000u ? 0u : w[i] & 0xffff0000u;
    w[i] = lo | hi;
  }
  return __builtin_bit_cast(bf16x8, w);
}
__device__ __forceinline__ uint32_t odd_code(uint32_t h) { // of a bf16's bits: 0 for a finite one
  const uint32_t inf = (h & 0x8000u) ? 0x4300u : 0x3f80u;  // 128 or 1
  const uint32_t c = (h & 0x7fu) ? 0x4301u : inf;          // 129
  return (h & 0x7f80u) == 0x7f80u ? c : 0u;
}
__device__ __forceinline__ bf16x8 odd_part(bf16x8 v) {
  u32x4 w = __builtin_bit_cast(u32x4, v);
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = odd_code(w[i] & 0xffffu) | (odd_code(w[i] >> 16) << 16);
  return __builtin_bit_cast(bf16x8, w);
}
__device__ __forceinline__ float odd_code_f32(float f) {
  const float inf = f < 0.f ? 128.f : 1.f;
  return isnan(f) ? 129.f : (isinf(f) ? inf : 0.f);
}
// What the counted values add up to.
__device__ __forceinline__ float odd_sum(float count) {
  const float neg = floorf(count * (1.0f / 128.0f)), pos = count - 128.0f * neg;
  const float one = neg > 0.f ? -INFINITY : (pos > 0.f ? INFINITY : 0.f);
  return neg > 0.f && pos > 0.f ? __uint_as_float(0x7fc00000u) : one;
}
// Eight bits as eight bf16, 0 or 1.
__device__ __forceinline__ bf16x8 bits_bf16(uint32_t bits) {
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = ((bits >> (2 * i)) & 1u) * 0x3f80u + ((bits >> (2 * i + 1)) & 1u) * 0x3f800000u;
  return __builtin_bit_cast(bf16x8, w);
}

// Four sums over their denominator, rounded; no denominator: zeros.
template <int DT>
__device__ __forceinline__ void put_row(void* out, int64_t at, const f32x4& sum, float l) {
  const f32x4 y = sum * (l == 0.f ? 0.f : 1.0f / l);
  if constexpr (DT == kF32) {
    *reinterpret_cast<f32x4*>(static_cast<float*>(out) + at) = y;
  } else {
    uint2 w;
    w.x = f32_to_bf16(y[0]) | (static_cast<uint32_t>(f32_to_bf16(y[1])) << 16);
    w.y = f32_to_bf16(y[2]) | (static_cast<uint32_t>(f32_to_bf16(y[3])) << 16);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) = w;
  }
}

// The joined sums of a block's waves go out: divided and rounded, or as one
// share's part.  `sum` holds dims [c0, c0 + 4) of row `row` of the sequence's.
template <int DT, int D, int ROWS>
__device__ __forceinline__ void store_row(const AttnArgs& a, const Rows& r, int row, int c0, const f32x4& sum, float m, float l,
                                          bool whole, int slot) {
  if (!whole) {
    const int64_t at = (static_cast<int64_t>(blockIdx.x) * 2 + slot) * ROWS + row - r.tile * ROWS;
    *reinterpret_cast<f32x4*>(a.part + at * D + c0) = sum;
    if (c0 == 0) *reinterpret_cast<float2*>(a.ml + at * 2) = float2{m, l};
    return;
  }
  const int64_t o = (r.begin + static_cast<int64_t>(row / a.each)) * a.nq + r.h * a.each + row % a.each;
  put_row<DT>(a.out, o * D + c0, sum, l);
}

// What sums are scaled by when the maximum grows from m to M; not 0, times which
// an infinite sum would be NaN.
__device__ __forceinline__ float grown(float m, float M) { return M == -INFINITY ? 1.f : fmaxf(__builtin_amdgcn_exp2f(m - M), 1e-37f); }

// Weight of a part whose maximum is m among parts whose largest is M.
__device__ __forceinline__ float part_weight(float m, float l, float M) { return l == 0.f ? 0.f : grown(m, M); }

// ---------------------------------------------------------------------------
// Few rows: a block takes 16 RT rows of a key head and a run of its keys, its
// four waves in turn 16 X keys each; they join at the end.
//
// The reads of K and V bound it (64 contexts of 100 to 32768 tokens, 16 query and 2 key
// heads of 256: 763 MB in 142 us, 5.4 TB/s; 256 of 2000 tokens, 8 key heads of 128:
// 5.8 TB/s; a pure read reaches 6.4).  K goes from memory straight into the operand
// of S^T (a lane reads 16 bytes of one key), V by direct loads into the wave's
// own part of LDS, where the transposing read gives four keys of a dim; the
// next keys are under way while the current ones are worked on.  Pieces of
// 16 bytes lie turned by their row, so that the transposing reads of eight rows
// fall into different banks.  A step is 32 keys a wave, for 256 dims 16, which
// leaves room for two blocks on a CU: a block's start (lengths, then pages, then
// keys: three trips to memory) hides behind the other's work.
//
// WHOLE: 16 keys from a multiple of 16 on lie in one page (pages of 16 tokens or
// more), so their address is one for the wave.  Other pages are looked up key
// by key.
template <int D, int RT>
struct FewLds {
  static constexpr int kX = D == 256 ? 1 : 2;              // runs of 16 keys a step
  static constexpr int kV = 16 * kX * D * 2;               // a wave's tile of V
  static constexpr int kCut = 64;                          // dims joined at once
  static constexpr int kRow = kCut + 4;
  static constexpr int kJoin = 4 * 16 * RT * kRow * 4 + 4 * 16 * RT * 2 * 4;
  static constexpr int kBytes = 8 * kV > kJoin ? 8 * kV : kJoin;
};

template <int D, int RT, bool WHOLE, bool EVEN>
__global__ __launch_bounds__(256, RT == 1 ? 2 : 1) void k_attn_few(AttnArgs a) {
  using L = FewLds<D, RT>;
  constexpr int KS = D / 32;                 // steps of 32 dims
  constexpr int DT = D / 16;                 // tiles of 16 dims
  constexpr int kPer = D / 8;                // 16-byte pieces a row
  constexpr int kRpl = 64 / kPer;            // rows a direct load
  constexpr int X = L::kX, kKeys = 16 * X;
  constexpr int VL = kKeys / kRpl;           // direct loads a tile of V
  constexpr int kVary = D == 256 ? 4 : (D == 128 ? 2 : 1);   // loads until the turn comes round
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int n16 = lane & 15, g = lane >> 4;
  walk<16 * RT, 4 * 16 * L::kX, EVEN>(a, lane, [&](const Rows& r, int kbeg, int kend, bool whole, int slot) {
  const int rows = r.n * a.each;
  const int row0 = r.tile * 16 * RT;
  const bool tree = a.tree != nullptr;
  const int clear = r.prefix + (tree ? 0 : row0 / a.each + 1);   // keys that all rows see

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
    for (int s = 0; s < KS; ++s) Q[t][s] = __builtin_bit_cast(bf16x8, load16(q + 32 * s + 8 * g) ^ a.flip);
  }
  // waited for here: a wait in the loop would be for the direct loads as well
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int s = 0; s < KS; ++s) asm volatile("" : "+v"(Q[t][s]));
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
  const auto turn = [](int row) { return D == 64 ? ((row >> 1) & 3) * 2 : (row & 7) * 2; };
  uint32_t voff[kVary];
#pragma unroll
  for (int j = 0; j < kVary; ++j)
    voff[j] = (lane / kPer) * D * 2 + (((lane % kPer) ^ turn(j * kRpl + lane / kPer)) << 4);
  const int koff = n16 * D + 8 * g;

  u32x4 Kn[X][KS];
  int ids[X];                                // WHOLE: pages of the runs of 16 keys
  const auto look = [&](int kt) {
    if constexpr (WHOLE) {
#pragma unroll
      for (int t = 0; t < X; ++t) ids[t] = page_at(a, r.b, kt + 16 * t < kend ? kt + 16 * t : kend - 1);
    }
  };
  const auto request = [&](int kt, uint8_t* vt) {   // the keys of a step from kt on
    if constexpr (WHOLE) {
#pragma unroll
      for (int t = 0; t < X; ++t) {
        // keys behind the end: rows of the last one's page, or of the run's own, that nobody sees
        const uint16_t* p = pool + key_at<D>(a, ids[t], r.h, kt + 16 * t);
        const u32x4 rs = raw_rsrc(p + a.at.half_elems, 16 * D * 2);
#pragma unroll
        for (int j = t * VL / X; j < (t + 1) * VL / X; ++j)
          lds_load<16>(rs, vt + j * 1024, voff[j % kVary], ((j * kRpl) & 15) * D * 2);
      }
#pragma unroll
      for (int t = 0; t < X; ++t) {
        const uint16_t* p = pool + key_at<D>(a, ids[t], r.h, kt + 16 * t);
#pragma unroll
        for (int s = 0; s < KS; ++s) Kn[t][s] = load16(p + koff + 32 * s);
      }
    } else {
#pragma unroll
      for (int j = 0; j < VL; ++j) {
        const int row = j * kRpl + lane / kPer;
        const int key = kt + row < kend ? kt + row : kend - 1;
        lds_load_at(pool + a.at.half_elems + key_at<D>(a, page_at(a, r.b, key), r.h, key) + ((lane % kPer) ^ turn(row)) * 8, vt + j * 1024);
      }
#pragma unroll
      for (int t = 0; t < X; ++t) {
        const int key = kt + 16 * t + n16 < kend ? kt + 16 * t + n16 : kend - 1;
        const uint16_t* p = pool + key_at<D>(a, page_at(a, r.b, key), r.h, key) + 8 * g;
#pragma unroll
        for (int s = 0; s < KS; ++s) Kn[t][s] = load16(p + 32 * s);
      }
    }
  };

  constexpr int kStep = 4 * kKeys;
  int kt = kbeg + kKeys * wave;
  uint8_t* const part = smem + wave * 2 * L::kV;
  int stage = 0;
  uint32_t gone = 0;                         // WHOLE: runs of 16 keys whose page is not there
  const auto missing = [&]() {
    uint32_t w = 0;
    if constexpr (WHOLE) {
#pragma unroll
      for (int t = 0; t < X; ++t) w |= static_cast<uint32_t>(!there(a, ids[t])) << t;
    }
    return w;
  };
  if (kt < kend) {
    look(kt);
    request(kt, part);
    gone = missing();
    look(kt + kStep);
  }
  for (; kt < kend; kt += kStep) {
    uint8_t* vt = part + stage * L::kV;
    const auto value = [&](int d) {          // rows 4 g + r, then 16 + 4 g + r (or again); this lane names row (n16 / 4), columns 4 (n16 % 4) ..
      bf16x8 V;
#pragma unroll
      for (int x = 0; x < X; ++x) {
        const int row = 16 * x + 4 * g + (n16 >> 2);
        const int col = 2 * d + ((n16 & 3) >> 1);
        const bf16x4 v = read_tr(vt + row * D * 2 + ((col ^ turn(row)) << 4) + (n16 & 1) * 8);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          V[4 * x + i] = v[i];
          if constexpr (X == 1) V[4 + i] = v[i];
        }
      }
      return V;
    };
    wait_loads();
    f32x4 S[RT][X];
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int x = 0; x < X; ++x) {
        S[t][x] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < KS; ++s)
          S[t][x] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, Kn[x][s]), Q[t][s], S[t][x], 0, 0, 0);
      }
    const uint32_t none = WHOLE ? gone : 0;
    stage ^= 1;
    if (kt + kStep < kend) {
      request(kt + kStep, part + stage * L::kV);
      gone = missing();
      look(kt + 2 * kStep);
    }

    // keys that some row of the tile does not see, or that are not there
    const bool careful = !WHOLE || none != 0 || kt + kKeys > kend || kt + kKeys > clear;
    uint32_t seen[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) seen[t] = 0xffu;
    if (careful) {
      uint32_t in = 0;
#pragma unroll
      for (int x = 0; x < X; ++x)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = kt + 16 * x + 4 * g + i;
          uint32_t ok = static_cast<uint32_t>(key < kend);
          if constexpr (WHOLE) ok &= ~(none >> x);
          else ok &= static_cast<uint32_t>(there(a, page_at(a, r.b, key < kend ? key : kend - 1)));
          in |= ok << (4 * x + i);
        }
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        uint32_t of = 0;
#pragma unroll
        for (int x = 0; x < X; ++x)
#pragma unroll
          for (int i = 0; i < 4; ++i) of |= sees(tree, mask[t], itok[t], kt + 16 * x + 4 * g + i - r.prefix) << (4 * x + i);
        seen[t] = in & of;
      }
      typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
      u16x2 big = {0, 0};
#pragma unroll
      for (int j = 0; j < VL; ++j) {
        const u32x4 w = *reinterpret_cast<const u32x4*>(vt + j * 1024 + lane * 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) big = __builtin_elementwise_max(big, __builtin_bit_cast(u16x2, w[i] & 0x7fff7fffu));
      }
      if (__ballot(big[0] >= 0x7f80u || big[1] >= 0x7f80u)) {
        // values that are not finite: counted by the rows that see them, then taken out of the tile
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int t = 0; t < RT; ++t) {
            f32x4 c = {0.f, 0.f, 0.f, 0.f};
            c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(odd_part(value(d)), bits_bf16(seen[t]), c, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i) O[t][d][i] += odd_sum(c[i]);
          }
        wave_sync_lds();
        for (int j = 0; j < VL; ++j) {
          u32x4* w = reinterpret_cast<u32x4*>(vt + j * 1024 + lane * 16);
          *w = __builtin_bit_cast(u32x4, finite_part(__builtin_bit_cast(bf16x8, *w)));
        }
        wave_sync_lds();
      }
    }
    // P in two bf16 parts: one alone would add an error as large as the output's
    // own rounding.  With 16 keys a step both go into one product, V twice.
    bf16x8 P[RT], Plo[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      float mx = -INFINITY;
#pragma unroll
      for (int x = 0; x < X; ++x)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (careful) S[t][x][i] = ((seen[t] >> (4 * x + i)) & 1u) ? S[t][x][i] : -INFINITY;
          mx = fmaxf(mx, S[t][x][i]);
        }
      mx = xor_max(mx, lane) * a.scale2;
      if (__ballot(mx > m[t] + kSlack)) {    // some row's maximum grows
        const float mn = fmaxf(m[t], mx);
        const float f = grown(m[t], mn);
        m[t] = mn;
        l[t] *= f;
#pragma unroll
        for (int d = 0; d < DT; ++d) O[t][d] *= f;
      }
      const float mu = m[t] == -INFINITY ? 0.f : m[t];
      float add = 0.f;
#pragma unroll
      for (int x = 0; x < X; ++x)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float p = __builtin_amdgcn_exp2f(fmaf(S[t][x][i], a.scale2, -mu));
          add += p;
          const __bf16 hi = static_cast<__bf16>(p), lo = static_cast<__bf16>(p - static_cast<float>(hi));
          P[t][4 * x + i] = hi;
          if constexpr (X == 2) Plo[t][4 * x + i] = lo;
          else P[t][4 + i] = lo;
        }
      l[t] += add;                           // this lane's keys; the four lanes of a row are joined at the end
    }
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      const bf16x8 V = value(d);
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        if constexpr (X == 2) O[t][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(V, Plo[t], O[t][d], 0, 0, 0);
        O[t][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(V, P[t], O[t][d], 0, 0, 0);
      }
    }
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
        float M = -INFINITY, ll = 0.f;
        f32x4 sum = {0.f, 0.f, 0.f, 0.f};
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
        store_row<kBF16, D, 16 * RT>(a, r, row0 + row, c * L::kCut + cc, sum, M, ll, whole, slot);
      }
    }
    __syncthreads();
  }
  });
}

// ---------------------------------------------------------------------------
// Many rows: a block takes 128 rows of a key head, 32 a wave, and walks their
// keys 64 at a time through LDS, which all four waves read; the next 64 are
// under way by direct loads meanwhile.  32x32x16 products: a lane has 16 of a
// tile's 32 keys of one row, its partner (lane ^ 32) the others.
//
// The matrix units and the reads of LDS bound it alike (each wave reads the
// whole tile for its 32 rows): 8192 tokens behind 809, 16 heads of 256, 1150 us,
// 570 TF/s; 4096 tokens, 32 heads of 128, 187 us, 735 TF/s.  Pieces of 16 bytes lie turned by their row so
// that the 16 rows, or the four rows of a transposing read, that are read at
// once fall into different banks.
//
// WHOLE as above, with runs of 16 keys (32 for 64 dims).
template <int D>
struct TileLds {
  static constexpr int kTile = 64 * D * 2;                 // bytes of K, and of V
  static constexpr int kBytes = 4 * kTile;                 // two stages
};

template <int D>
__device__ __forceinline__ int k_turn(int key) { return D == 64 ? (key >> 1) & 7 : key & 15; }
template <int D>
__device__ __forceinline__ int v_turn(int key) { return D == 64 ? ((key >> 1) & 1) * 4 : (key & 3) * 4; }

typedef float f32x16 __attribute__((ext_vector_type(16)));

template <int D, bool WHOLE, bool EVEN>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void k_attn_tile(AttnArgs a) {
  using L = TileLds<D>;
  constexpr int KS = D / 16;                 // steps of 16 dims
  constexpr int DT = D / 32;                 // tiles of 32 dims
  constexpr int kPer = D / 8;                // 16-byte pieces a row
  constexpr int kRpl = 64 / kPer;            // rows a direct load
  constexpr int kRun = D == 64 ? 32 : 16;    // keys whose page is one
  constexpr int kRuns = 64 / kRun;
  constexpr int kLoads = kRun / kRpl / 4;    // direct loads of a wave for a run of K, and of V
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int n32 = lane & 31, g = lane >> 5;
  walk<128, 64, EVEN>(a, lane, [&](const Rows& r, int kbeg, int kend, bool whole, int slot) {
  const int rows = r.n * a.each;
  const int row0 = r.tile * 128;
  const bool tree = a.tree != nullptr;
  const int clear = r.prefix + (tree ? 0 : row0 / a.each + 1);   // keys that all rows see

  const int row = row0 + 32 * wave + n32;
  const int rr = row < rows ? row : rows - 1;
  const int itok = rr / a.each;
  const int64_t token = r.begin + itok;
  const uint64_t mask = tree ? a.tree[token] : 0;
  const bool idle = row0 + 32 * wave >= rows;              // a wave without rows only fetches
  bf16x8 Q[KS];
  {
    const uint16_t* q = static_cast<const uint16_t*>(a.q) + (token * a.nq + r.h * a.each + rr % a.each) * D;
#pragma unroll
    for (int s = 0; s < KS; ++s) Q[s] = __builtin_bit_cast(bf16x8, load16(q + 16 * s + 8 * g) ^ a.flip);
  }
  // Q is waited for here: a wait in the loop would be for the direct loads as well.
  // 256 dims: in accumulation registers, so that O, which is scaled, stays in the others.
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    if constexpr (D == 256) asm volatile("" : "+a"(Q[s]));
    else asm volatile("" : "+v"(Q[s]));
  }
  f32x16 O[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) O[d][i] = 0.f;
  float m = -INFINITY, l = 0.f;

  // Row (i 4 + wave) kRpl + lane / kPer of a run is load i's; its turn is the same in every run.
  const uint16_t* pool = static_cast<const uint16_t*>(a.pages);
  uint32_t koff[kLoads], voff[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int rw = (4 * i + wave) * kRpl + lane / kPer;
    koff[i] = rw * D * 2 + (((lane % kPer) ^ k_turn<D>(rw)) << 4);
    voff[i] = rw * D * 2 + (((lane % kPer) ^ v_turn<D>(rw)) << 4);
  }
  int ids[kRuns];
  const auto look = [&](int kt) {
    if constexpr (WHOLE) {
#pragma unroll
      for (int c = 0; c < kRuns; ++c) ids[c] = page_at(a, r.b, kt + kRun * c < kend ? kt + kRun * c : kend - 1);
    }
  };
  const auto request = [&](int kt, uint8_t* st) {
#pragma unroll
    for (int c = 0; c < kRuns; ++c) {
      if constexpr (WHOLE) {
        // keys behind the end: rows of the last one's page, or of the run's own, that nobody sees
        const uint16_t* p = pool + key_at<D>(a, ids[c], r.h, kt + kRun * c);
        const u32x4 rk = raw_rsrc(p, kRun * D * 2), rv = raw_rsrc(p + a.at.half_elems, kRun * D * 2);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          uint8_t* to = st + (c * kRun + (4 * i + wave) * kRpl) * D * 2;
          lds_load<16>(rk, to, koff[i], 0);
          lds_load<16>(rv, to + L::kTile, voff[i], 0);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          const int rw = c * kRun + (4 * i + wave) * kRpl + lane / kPer;
          const int key = kt + rw < kend ? kt + rw : kend - 1;
          const uint16_t* p = pool + key_at<D>(a, page_at(a, r.b, key), r.h, key);
          uint8_t* to = st + (c * kRun + (4 * i + wave) * kRpl) * D * 2;
          lds_load_at(p + ((lane % kPer) ^ k_turn<D>(rw)) * 8, to);
          lds_load_at(p + a.at.half_elems + ((lane % kPer) ^ v_turn<D>(rw)) * 8, to + L::kTile);
        }
      }
    }
  };
  const auto missing = [&]() {               // runs whose page is not there
    uint32_t w = 0;
    if constexpr (WHOLE) {
#pragma unroll
      for (int c = 0; c < kRuns; ++c) w |= static_cast<uint32_t>(!there(a, ids[c])) << c;
    }
    return w;
  };

  int stage = 0;
  uint32_t gone = 0;
  if (kbeg < kend) {
    look(kbeg);
    request(kbeg, smem);
    gone = missing();
    look(kbeg + 64);
  }
  for (int kt = kbeg; kt < kend; kt += 64) {
    const uint8_t* Kt = smem + stage * 2 * L::kTile;
    const uint8_t* Vt = Kt + L::kTile;
    stage ^= 1;
    wait_loads();
    __syncthreads();                         // the tile is there, and nobody reads the other stage any more
    const uint32_t none = gone;
    if (kt + 64 < kend) {
      request(kt + 64, smem + stage * 2 * L::kTile);
      gone = missing();
      look(kt + 128);
    }
    const bool careful = !WHOLE || none != 0 || kt + 64 > kend || kt + 64 > clear;
    uint32_t seen[2] = {0xffffu, 0xffffu};   // of 32 keys each, bit i: key 8 (i / 4) + 4 g + i % 4
    const auto value = [&](int key0, int d) {    // keys key0 + 8 y + 4 g + 0 .. 3, dims 32 d + 16 (lane / 16 % 2) ..
      bf16x8 V;
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int key = key0 + 8 * y + 4 * g + ((lane & 15) >> 2);
        const int col = 4 * d + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
        const bf16x4 v = read_tr(Vt + key * D * 2 + ((col ^ v_turn<D>(key)) << 4) + (lane & 1) * 8);
#pragma unroll
        for (int i = 0; i < 4; ++i) V[4 * y + i] = v[i];
      }
      return V;
    };
    if (careful) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        seen[x] = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int at = kt + 32 * x + 8 * (i >> 2) + 4 * g + (i & 3);
          uint32_t in = static_cast<uint32_t>(at < kend);
          if constexpr (WHOLE) in &= ~(none >> ((32 * x + 8 * (i >> 2)) / kRun));
          else in &= static_cast<uint32_t>(there(a, page_at(a, r.b, at < kend ? at : kend - 1)));
          seen[x] |= (in & sees(tree, mask, itok, at - r.prefix)) << i;
        }
      }
      typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
      u16x2 big = {0, 0};
      for (int i = lane; i < 64 * kPer; i += kWave) {
        const u32x4 w = *reinterpret_cast<const u32x4*>(Vt + i * 16);
#pragma unroll
        for (int j = 0; j < 4; ++j) big = __builtin_elementwise_max(big, __builtin_bit_cast(u16x2, w[j] & 0x7fff7fffu));
      }
      if (__ballot(big[0] >= 0x7f80u || big[1] >= 0x7f80u)) {
        // values that are not finite (all four waves see them): counted by the
        // rows that see them, then taken out of the tile
#pragma unroll 1
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            f32x16 c;
#pragma unroll
            for (int i = 0; i < 16; ++i) c[i] = 0.f;
#pragma unroll
            for (int j = 0; j < 2; ++j)
              c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(odd_part(value(32 * x + 16 * j, d)), bits_bf16(seen[x] >> (8 * j)), c, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 16; ++i) O[d][i] += odd_sum(c[i]);
          }
        __syncthreads();
        for (int i = threadIdx.x; i < 64 * kPer; i += 256) {
          u32x4* w = reinterpret_cast<u32x4*>(const_cast<uint8_t*>(Vt) + i * 16);
          *w = __builtin_bit_cast(u32x4, finite_part(__builtin_bit_cast(bf16x8, *w)));
        }
        __syncthreads();
      }
    }
    if (idle) continue;
#pragma unroll
    for (int x = 0; x < 2; ++x) {            // 32 keys each
      f32x16 S;
#pragma unroll
      for (int i = 0; i < 16; ++i) S[i] = 0.f;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const int key = 32 * x + n32;
        const u32x4 kv = *reinterpret_cast<const u32x4*>(Kt + key * D * 2 + (((2 * s + g) ^ k_turn<D>(key)) << 4));
        S = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, kv), Q[s], S, 0, 0, 0);
      }
      __builtin_amdgcn_sched_barrier(0);     // or the reads of V are moved up until registers run out
      if (careful) {
#pragma unroll
        for (int i = 0; i < 16; ++i) S[i] = ((seen[x] >> i) & 1u) ? S[i] : -INFINITY;
      }
      float mx = -INFINITY;
#pragma unroll
      for (int i = 0; i < 16; ++i) mx = fmaxf(mx, S[i]);
      mx = fmaxf(mx, __uint_as_float(lane_xor<32>(__float_as_uint(mx), lane))) * a.scale2;
      if (__ballot(mx > m + kSlack)) {
        const float mn = fmaxf(m, mx);
        const float f = grown(m, mn);
        m = mn;
        l *= f;
#pragma unroll
        for (int d = 0; d < DT; ++d) O[d] *= f;
      }
      const float mu = m == -INFINITY ? 0.f : m;
      bf16x8 P[2];                           // 16 keys each, in the order of the lane's S
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float p = __builtin_amdgcn_exp2f(fmaf(S[i], a.scale2, -mu));
        l += p;
        P[i >> 3][i & 7] = static_cast<__bf16>(p);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int j = 0; j < 2; ++j) O[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(value(32 * x + 16 * j, d), P[j], O[d], 0, 0, 0);
    }
  }
  l += __uint_as_float(lane_xor<32>(__float_as_uint(l), lane));
  if (row < rows)
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        store_row<kBF16, D, 128>(a, r, row, 32 * d + 8 * i + 4 * g,
                                 f32x4{O[d][4 * i], O[d][4 * i + 1], O[d][4 * i + 2], O[d][4 * i + 3]}, m, l, whole, slot);
  __syncthreads();                           // nobody reads this unit's tiles when the next one's arrive
  });
}

// ---------------------------------------------------------------------------
// fp32: the same split of the work on the fp32 matrix instruction (16x16x4).
// Everything goes from memory to its operand: of the four dims of a 16-byte
// piece of a key, one for each of four products; V likewise, four dims of one
// key for four tiles.  Few rows are bound by the reads of K and V (64 tokens behind
// 4000, 2 key heads of 256: 200 us, 5.2 TB/s), prompts by the instruction's rate and the
// loads that each wave repeats (2048 tokens, 16 heads of 128: 222 us, 77 TF/s).
template <int D, int RT>
struct F32Lds {
  static constexpr int kCut = RT == 2 ? 32 : 64;
  static constexpr int kRow = kCut + 4;
  static constexpr int kBytes = 4 * 16 * RT * kRow * 4 + 4 * 16 * RT * 2 * 4;
};

template <int D, int RT, bool EVEN>
__global__ __launch_bounds__(256, RT == 1 ? 2 : 1) void k_attn_f32(AttnArgs a) {
  using L = F32Lds<D, RT>;
  constexpr int KS = D / 16;                 // 16-byte pieces of a row for a lane's quarter
  constexpr int DQ = D / 64;                 // groups of 64 dims
  __shared__ __align__(16) uint8_t smem[L::kBytes];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = threadIdx.x / kWave;
  const int n16 = lane & 15, g = lane >> 4;
  walk<16 * RT, 64, EVEN>(a, lane, [&](const Rows& r, int kbeg, int kend, bool whole, int slot) {
  const int rows = r.n * a.each;
  const int row0 = r.tile * 16 * RT;
  const bool tree = a.tree != nullptr;
  const int clear = r.prefix + (tree ? 0 : row0 / a.each + 1);   // keys that all rows see

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
    for (int s = 0; s < KS; ++s) Q[t][s] = __builtin_bit_cast(f32x4, load16(q + 16 * s + 4 * g) ^ a.flip);
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
    f32x4 S[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      S[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) S[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(K[s][i], Q[t][s][i], S[t], 0, 0, 0);
    }
    __builtin_amdgcn_sched_barrier(0);       // V takes the registers of K: a second block on the CU hides more than an earlier request
    f32x4 V[4][DQ];                          // keys 4 g + r, dims 64 q + 4 n16 ..
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      int vk = kt + 4 * g + i;
      vk = vk < kend ? vk : kend - 1;
      const float* vp = pool + a.at.half_elems + key_at<D>(a, page_at(a, r.b, vk), r.h, vk);
#pragma unroll
      for (int d = 0; d < DQ; ++d) V[i][d] = *reinterpret_cast<const f32x4*>(vp + 64 * d + 4 * n16);
    }
    const bool careful = there != 0xffffu || kt + 16 > kend || kt + 16 > clear;
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
        if (careful) S[t][i] = (seen >> i) & 1u ? S[t][i] : -INFINITY;
        mx = fmaxf(mx, S[t][i]);
      }
      mx = xor_max(mx, lane) * a.scale2;
      if (__ballot(mx > m[t] + kSlack)) {
        const float mn = fmaxf(m[t], mx);
        const float f = grown(m[t], mn);
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
        p[i] = __builtin_amdgcn_exp2f(fmaf(S[t][i], a.scale2, -mu));
        l[t] += p[i];
      }
#pragma unroll
      for (int d = 0; d < DQ; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float v = V[k][d][i];
            if (bad) v = (__float_as_uint(v) & 0x7f800000u) == 0x7f800000u ? 0.f : v;
            O[t][d][i] = __builtin_amdgcn_mfma_f32_16x16x4f32(v, p[k], O[t][d][i], 0, 0, 0);
          }
      if (bad) {
#pragma unroll
        for (int d = 0; d < DQ; ++d)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            f32x4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              c = __builtin_amdgcn_mfma_f32_16x16x4f32(odd_code_f32(V[k][d][i]), static_cast<float>((seen >> k) & 1u), c, 0, 0, 0);
#pragma unroll
            for (int j = 0; j < 4; ++j) O[t][d][i][j] += odd_sum(c[j]);
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
        float M = -INFINITY, ll = 0.f;
        f32x4 sum = {0.f, 0.f, 0.f, 0.f};
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
        store_row<kF32, D, 16 * RT>(a, r, row0 + row, c * L::kCut + cc, sum, M, ll, whole, slot);
      }
    }
    __syncthreads();
  }
  });
}

// ---------------------------------------------------------------------------
// The parts of a row joined, where blocks shared its keys, and zeros for rows
// without any.  A wave takes 128 dims of a row (heads of 64 dims: 64), 32 or 16 lanes a
// part, two or four parts at once, four loads each on the way; WIDE, for many parts of few
// rows: the block's four waves share those of 64 dims.  Bound
// by the parts' reads, and by the launch where there are few (1 token of 16 heads
// 4.0 us; 248 tokens of 32 heads of 128, 32 MB of parts, 9.4, and 14 with 64 dims a wave).
constexpr int join_dims(int D, bool wide) { return wide || D == 64 ? 64 : 128; }

template <int DT, int D, int ROWS, int STEP, bool WIDE>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a) {
  constexpr int W = join_dims(D, WIDE), LP = W / 4;    // dims a wave, lanes a part
  constexpr int kSlices = D / W;
  __shared__ f32x4 sums[4][LP];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int64_t item = WIDE ? blockIdx.x : static_cast<int64_t>(blockIdx.x) * 4 + wave;
  const int64_t per = static_cast<int64_t>(a.new_max) * a.nq * kSlices;
  if (item >= per * a.at.B) return;
  const int b = static_cast<int>(item / per), slice = static_cast<int>(item % kSlices);
  const int idx = static_cast<int>((item % per) / kSlices);
  const int h = idx / (a.new_max * a.each), row = idx % (a.new_max * a.each);
  Rows r;
  if (!sequence(a, b, r) || row >= r.n * a.each) return;
  const int steps = steps_of<STEP>(r);
  const int64_t o = ((r.begin + static_cast<int64_t>(row / a.each)) * a.nq + h * a.each + row % a.each) * D + slice * W + lane % LP * 4;
  if (steps == 0) {
    if (lane < LP && (!WIDE || wave == 0)) put_row<DT>(a.out, o, f32x4{0.f, 0.f, 0.f, 0.f}, 0.f);
    return;
  }
  const int share = a.shares[0], before = b > 0 ? a.shares[b] : 0;
  const int w0 = before + (h * tiles_of<ROWS>(a, r) + row / ROWS) * steps;
  const int k0 = w0 / share, k1 = (w0 + steps - 1) / share;
  if (k0 == k1) return;                      // one block had all of it
  const int parts = k1 - k0 + 1;
  const auto place = [&](int p) {            // the first block's part lies in slot 1 unless its share begins with it
    return (static_cast<int64_t>(k0 + p) * 2 + (p == 0 && w0 != k0 * share ? 1 : 0)) * ROWS + row % ROWS;
  };
  float M = -INFINITY;
  for (int p = lane; p < parts; p += kWave) M = fmaxf(M, a.ml[place(p) * 2]);
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) M = fmaxf(M, __shfl_xor(M, d));
  const auto over_parts = [&](float x) {     // lanes that hold the same dims of other parts
    if constexpr (LP == 16) x += __uint_as_float(lane_xor<16>(__float_as_uint(x), lane));
    return x + __uint_as_float(lane_xor<32>(__float_as_uint(x), lane));
  };
  f32x4 sum = {0.f, 0.f, 0.f, 0.f};
  float l = 0.f;
  constexpr int kGroups = (WIDE ? 4 : 1) * (kWave / LP);
  for (int p0 = (WIDE ? wave * (kWave / LP) : 0) + lane / LP; p0 < parts; p0 += 4 * kGroups) {
    f32x4 v[4];
    float2 ml[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int p = p0 + kGroups * i < parts ? p0 + kGroups * i : p0;
      const int64_t at = place(p);
      ml[i] = *reinterpret_cast<const float2*>(a.ml + at * 2);
      v[i] = *reinterpret_cast<const f32x4*>(a.part + at * D + slice * W + lane % LP * 4);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (p0 + kGroups * i < parts && ml[i].y != 0.f) {
        const float f = part_weight(ml[i].x, ml[i].y, M);
        l = fmaf(ml[i].y, f, l);
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[j] = fmaf(v[i][j], f, sum[j]);
      }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) sum[j] = over_parts(sum[j]);
  l = over_parts(l);
  if constexpr (WIDE) {
    __shared__ float ls[4];
    if (lane < LP) sums[wave][lane] = sum;
    if (lane == 0) ls[wave] = l;
    __syncthreads();
    sum = sums[0][lane % LP] + sums[1][lane % LP] + sums[2][lane % LP] + sums[3][lane % LP];
    l = ls[0] + ls[1] + ls[2] + ls[3];
    if (wave != 0) return;
  }
  if (lane < LP) put_row<DT>(a.out, o, sum, l);
}

// ---------------------------------------------------------------------------
struct AttnPlan {
  int rt;               // bf16: 1 or 2 times 16 rows a block (few), 8 (tiles); fp32: 1 or 2
  int tiles;            // row tiles a sequence and key head
  bool even, wide;
  int64_t blocks, join;
  size_t part, ml, total;   // workspace: sums, maxima and denominators, shares
};

int attn_plan(const attn_desc* d, int32_t B, int32_t N, int32_t new_max, int32_t len_max, AttnPlan* p) {
  if (B < 0 || B > (1 << 16) || N < 0 || N > (1 << 20)) return attn_bad("B=%lld must be in [0, 2^16], N=%lld in [0, 2^20]", B, N);
  if (new_max < 0 || len_max < 0 || len_max > 0x7ffff000) return attn_bad("new_max=%lld and len_max=%lld must not be negative or too large", new_max, len_max);
  const int each = d->n_q_heads / d->n_kv_heads, D = d->head_dim;
  const int most = new_max < N ? new_max : N;
  const int64_t rows = static_cast<int64_t>(most) * each;
  const bool f32 = d->dtype == MOE_F32;
  p->rt = f32 ? (rows <= 16 || D == 256 ? 1 : 2) : (rows <= 16 ? 1 : (rows <= 32 && D < 256 ? 2 : 8));
  p->tiles = static_cast<int>((rows + 16 * p->rt - 1) / (16 * p->rt));
  if (p->tiles < 1) p->tiles = 1;
  const int step = f32 || p->rt == 8 || D == 256 ? 64 : 128;   // keys a block takes at once
  // Even shares go to as many blocks as the chip holds at once, by their
  // registers and LDS.  64 contexts of 100 to 32768 tokens, 16 heads of 256: half as
  // many blocks 176 us, these 151, twice as many 155; a block for each (sequence, key
  // head) with its keys cut in runs of 2048 181.
  const int fit = f32 ? (p->rt == 1 ? (D == 64 ? 4 : (D == 128 ? 3 : 2)) : (D == 64 ? 2 : 1))
                      : (D == 64 && p->rt < 8 ? 5 - p->rt : (D == 256 && p->rt == 8 ? 1 : 2));
  const int64_t slots = 256 * fit;
  const int64_t units = static_cast<int64_t>(B) * d->n_kv_heads * p->tiles;
  const int64_t steps = (static_cast<int64_t>(len_max) + step - 1) / step;
  p->even = steps > 4 && units * steps < (int64_t(1) << 31) && (p->tiles == 1 || units < slots);
  p->blocks = units;
  p->join = 0;
  p->part = p->ml = p->total = 0;
  p->wide = false;
  if (p->even) {
    if (units * steps < slots) p->blocks = units * steps;
    else p->blocks = slots;
    // 32 parts of few rows: 6.8 us by four waves and 8.1 by one (4 sequences of 8
    // tokens, 16 heads of 256), 4.5 and 7.8 (2 of 6, 32 heads of 128); 8 parts of
    // 7936 rows take one wave each 9.4.
    p->wide = p->blocks > 12 * units;
    const int64_t items = static_cast<int64_t>(B) * rows * d->n_kv_heads * (D / join_dims(D, p->wide));
    p->join = p->wide ? items : (items + 3) / 4;
    const size_t at = static_cast<size_t>(p->blocks) * 2 * 16 * p->rt;
    p->part = at * D * 4;
    p->ml = at * 8;
    p->total = p->part + p->ml + (static_cast<size_t>(B) + 1) * 4;
  }
  if (p->blocks >= (int64_t(1) << 24) || p->join >= (int64_t(1) << 24))
    return attn_bad("B=%lld sequences of new_max=%lld tokens are too many blocks for one launch", B, new_max);
  return MOE_OK;
}

// Launch with dynamic LDS, whose size is set once per kernel and device.
template <void (*KERNEL)(AttnArgs), int BYTES>
bool launch_lds(const AttnArgs& a, hipStream_t s) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return false;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (!bit || !(done.load(std::memory_order_relaxed) & bit)) {
    if (hipFuncSetAttribute(reinterpret_cast<const void*>(KERNEL), hipFuncAttributeMaxDynamicSharedMemorySize, BYTES) != hipSuccess)
      return false;
    done.fetch_or(bit, std::memory_order_relaxed);
  }
  launch_kernel(KERNEL, dim3(a.blocks), dim3(256), BYTES, s, a);
  return true;
}

template <int D, bool WHOLE, bool EVEN>
bool launch_bf16(const AttnArgs& a, int rt, hipStream_t s) {
  if (rt == 1) return launch_lds<k_attn_few<D, 1, WHOLE, EVEN>, FewLds<D, 1>::kBytes>(a, s);
  if constexpr (D < 256)
    if (rt == 2) return launch_lds<k_attn_few<D, 2, WHOLE, EVEN>, FewLds<D, 2>::kBytes>(a, s);
  return launch_lds<k_attn_tile<D, WHOLE, EVEN>, TileLds<D>::kBytes>(a, s);
}

template <int D, bool EVEN>
bool launch_keys(const AttnArgs& a, int rt, int dtype, hipStream_t s) {
  if (dtype == MOE_F32) {
    if (rt == 1) launch_kernel(k_attn_f32<D, 1, EVEN>, dim3(a.blocks), dim3(256), 0, s, a);
    else if constexpr (D < 256) launch_kernel(k_attn_f32<D, 2, EVEN>, dim3(a.blocks), dim3(256), 0, s, a);
    return true;
  }
  const bool whole = a.at.shift >= (rt == 8 && D == 64 ? 5 : 4);
  return whole ? launch_bf16<D, true, EVEN>(a, rt, s) : launch_bf16<D, false, EVEN>(a, rt, s);
}

template <int DT, int D, int ROWS, int STEP>
void launch_join(const AttnArgs& a, const AttnPlan& p, hipStream_t s) {
  const dim3 grid(static_cast<uint32_t>(p.join));
  if (p.wide) launch_kernel(k_attn_join<DT, D, ROWS, STEP, true>, grid, dim3(256), 0, s, a);
  else launch_kernel(k_attn_join<DT, D, ROWS, STEP, false>, grid, dim3(256), 0, s, a);
}

template <int D>
bool launch_attn_d(const AttnArgs& a, const AttnPlan& p, int dtype, hipStream_t s) {
  if (!(p.even ? launch_keys<D, true>(a, p.rt, dtype, s) : launch_keys<D, false>(a, p.rt, dtype, s))) return false;
  if (!p.even) return true;
  if (dtype == MOE_F32) {
    if (p.rt == 1) launch_join<kF32, D, 16, 64>(a, p, s);
    else if constexpr (D < 256) launch_join<kF32, D, 32, 64>(a, p, s);
  } else {
    if (p.rt == 1) launch_join<kBF16, D, 16, D == 256 ? 64 : 128>(a, p, s);
    else if (p.rt == 8) launch_join<kBF16, D, 128, 64>(a, p, s);
    else if constexpr (D < 256) launch_join<kBF16, D, 32, 128>(a, p, s);
  }
  return true;
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
  a.shares = p.total ? reinterpret_cast<int*>(static_cast<uint8_t*>(workspace) + p.part + p.ml) : nullptr;
  a.nq = d->n_q_heads;
  a.nkv = d->n_kv_heads;
  a.each = a.nq / a.nkv;
  a.new_max = new_max < N ? new_max : N;
  a.len_max = len_max;
  a.tiles = p.tiles;
  a.blocks = static_cast<int>(p.blocks);
  // a positive factor, so that the largest product is the largest score: q takes the sign
  a.scale2 = fmaxf(fabsf(d->scale) * 1.4426950408889634f, FLT_MIN);
  a.flip = d->scale < 0.f ? (d->dtype == MOE_F32 ? 0x80000000u : 0x80008000u) : 0u;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool sent = d->head_dim == 64    ? launch_attn_d<64>(a, p, d->dtype, s)
                    : d->head_dim == 128 ? launch_attn_d<128>(a, p, d->dtype, s)
                                         : launch_attn_d<256>(a, p, d->dtype, s);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !sent) {
    char buf[256];
    snprintf(buf, sizeof(buf), "attention launch failed: %s", hipGetErrorString(e));
    return api_fail(MOE_EHIP, buf);
  }
  return api_ok();
}
