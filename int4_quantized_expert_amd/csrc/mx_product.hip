// Products of microscaled 4-bit matrices, dense and by routed expert
// (include/mxfp4.h).
//
// Mathematics.  v_mfma_scale_f32_16x16x128 multiplies 16 rows of W with 16
// rows of A over 128 values of k and scales every 32 of them by the two rows'
// powers of two.  Lane l holds 32 values (16 bytes) of row l mod 16 and their
// scale; which 32 of the 128 is free as long as both operands agree.  A chunk
// of 256 values (128 bytes of a row) is two such products: quarter l / 16
// holds values 64 q .. 64 q + 63 of the chunk, 32 in each product, so that a
// lane's 32 bytes and its two scale bytes are contiguous.  With W as the first
// operand a lane's four results are four consecutive outputs of one row of A.
#include <hip/hip_runtime.h>

#include <atomic>
#include <cstdio>

#include "mx_common.h"
#include "mx_internal.h"
#include "topk_wave.h"

namespace moe {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kMxF4 = 2;                 // a_dtype code MX_FP4
constexpr int kChunk = kMxPad;           // k values per step
// Pairs up to which the blocks find their expert's pairs by themselves (one id a
// lane) instead of a grouping launch, and up to which a token's weighted sum is
// one block's work, unless the pairs' codes of W are so many bytes that the
// tiles, whose loads run further ahead, make up for the launches.  Measured
// (bf16, here against tiles, us):
//   gate and up rows, 512 outputs, k = 2048: 20 pairs 10.3, 13.0; 40 pairs 14.2,
//     15.8; 50 pairs (52 MB) 16.6, 16.4; 60 pairs 18.6, 17.3
//   512 outputs, k = 512: 48 pairs 7.2, 10.0
//   sums of 2048 outputs, k = 512: 80 pairs 14.5, 18.5; 120 pairs (63 MB) 17.6,
//     22.1; of 2048 x 2048: 64 pairs (134 MB) 33.9, 30.2
//   sums of 512 outputs, k = 512: 256 pairs (34 MB) 13.4, 14.9; 384 pairs 15.4,
//     16.2, through 16 experts 14.8, 14.2; of 128 outputs: 1024 pairs 12.7, 13.5
constexpr int kDirectPairs = 64, kSumPairs = 1024;
constexpr int64_t kDirectBytes = 3 << 24, kSumBytes = 1 << 26;

enum Mode { kDense, kDirect, kTiles, kSum };

// A tile of the grouped path: up to PrepArgs::rows pairs of one expert.
struct MxTile {
  int64_t off;    // the expert's blob in the pool; -1: unusable, the rows are zero
  int32_t first;  // place of its first pair in the list
  int32_t count;
};

struct MxArgs {
  const void* a;
  const uint8_t* as;
  const uint8_t* wc;        // dense
  const uint8_t* wsc;
  const int64_t* slots;     // by expert
  const uint8_t* pool;
  int64_t codes_off, scales_off, need, pool_bytes;
  const int32_t* ids;
  const float* wts;
  void* out;
  uint32_t* flags;
  const int32_t* plist;
  const MxTile* tiles;
  const int32_t* ntiles;
  int M;                    // rows of A (dense), pairs
  int arows;                // rows of A that exist
  int N, K, chunks;
  int nblk;                 // blocks along N; the grid is flat, these fastest
  int k, E, pair_rows, out_bf16;
};

// The blob offset of expert e, -1 if the id or the slot is unusable.
__device__ __forceinline__ int64_t blob_of(const int64_t* slots, int e, int E, int64_t need, int64_t pool_bytes) {
  if (e < 0 || e >= E) return -1;
  const int64_t off = slots[e];
  return (off >= 0 && (off & 255) == 0 && off <= pool_bytes - need) ? off : -1;
}

__device__ __forceinline__ v4f mfma4(v4i a, v4i b, v4f c, int sa, int sb, int s) {
  const v8i A = {a[0], a[1], a[2], a[3], 0, 0, 0, 0}, B = {b[0], b[1], b[2], b[3], 0, 0, 0, 0};
  return s == 0 ? __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A, B, c, 4, 4, 0, sa, 0, sb)
                : __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A, B, c, 4, 4, 1, sa, 1, sb);
}

// A lane's part of a row's chunk: two blocks of codes and their scale bytes
// (in the low half of `sc`).
struct Part {
  v4i c[2];
  int sc;
};

template <int SRC>
struct Stored {
  typedef uint32_t T;
};
template <>
struct Stored<kBF16> {
  typedef uint16_t T;
};

// The same as it is stored: an MX matrix's codes, or values still to quantise.
template <int SRC>
struct RawPart {
  Eight<SRC> v[2][4];
};
template <>
struct RawPart<kMxF4> {
  Part p;
};

// A part from a wave-uniform base and a lane's offset (scalar base, 32-bit
// offset loads; the address arithmetic of cold kernels counts).  Codes: bytes
// from the chunk's first; values: elements from the row's chunk, `left` of them
// to the row's end.
__device__ __forceinline__ void load_codes(const uint8_t* codes, const uint8_t* scales, uint32_t co, uint32_t so, bool on,
                                           Part& p) {
  if (on) {
    const v4i* c = reinterpret_cast<const v4i*>(codes + co);
    p.c[0] = c[0];
    p.c[1] = c[1];
    p.sc = *reinterpret_cast<const uint16_t*>(scales + so);
  } else {
    p.c[0] = p.c[1] = v4i{0, 0, 0, 0};
    p.sc = 0;
  }
}

template <int SRC>
__device__ __forceinline__ void load_values(const void* base, int64_t at, int left, bool on, RawPart<SRC>& p) {
  // one test for the lane's 64 values, so that the usual path is short and in
  // one piece (a cold kernel waits for its instructions)
  const auto* src = static_cast<const typename Stored<SRC>::T*>(base) + at;
  if (on && left >= 64) {
    __builtin_memcpy(p.v, src, sizeof(p.v));
  } else {
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (on) mx_load8<SRC>(src, 0, b * 32 + i * 8, left, p.v[b][i]);
        else p.v[b][i] = Eight<SRC>{};
      }
  }
}

template <int SRC>
__device__ __forceinline__ Part finish_part(const RawPart<SRC>& p) {
  if constexpr (SRC == kMxF4) {
    return p.p;
  } else {
    Part o;
    o.sc = 0;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t x = mx_mag8(p.v[b][i]);
        m = x > m ? x : m;
      }
      const uint32_t byte = mx_scale_byte(m);
#pragma unroll
      for (int i = 0; i < 4; ++i) o.c[b][i] = static_cast<int>(mx_codes8(p.v[b][i], byte));
      o.sc |= static_cast<int>(byte) << (8 * b);
    }
    return o;
  }
}

__device__ __forceinline__ int64_t readlane64(int64_t v, int l) {
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(v & 0xffffffff), l);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(v >> 32), l);
  return static_cast<int64_t>((static_cast<uint64_t>(hi) << 32) | lo);
}

__device__ __forceinline__ float readlane_f(float v, int l) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l));
}

__device__ __forceinline__ float silu(float g) { return g / (1.0f + expf(-g)); }

// Round to nearest even in one instruction.
__device__ __forceinline__ uint16_t to_bf16(float y) { return __builtin_bit_cast(uint16_t, static_cast<__bf16>(y)); }

__device__ __forceinline__ void store_out(void* out, int64_t i, float y, int bf16) {
  if (bf16) static_cast<uint16_t*>(out)[i] = to_bf16(y);
  else static_cast<float*>(out)[i] = y;
}

// Few rows of A: a block forms 16 outputs of up to 16 MT rows (kSum: of one
// token), its waves take the chunks of k in turn and their sums are joined in
// LDS.  Bound by the reads of W and the chain of dependent loads before them
// (ids, slots); every block reads A while W is on its way, and quantises it where
// that is cheaper than a launch before (quantise_in_place).
// One token by 4096 x 2048: 4.3 us; through ten experts' gate and up rows (512
// outputs, k = 2048): 7.1 us, 1.6 TB/s; its sum over eight experts (2048 outputs,
// k = 512): 5.7 us.  64 rows by 4096 x 4096: 10.2 us.
//   kDense   rows 16 MT y .. of A
//   kDirect  y is a pair; the block of the first pair of an expert takes all
//            of that expert's pairs, the others end
//   kTiles   y is a tile of the grouped list
//   kSum     y is a token; its experts' products are summed with their weights
template <int SRC, int ACT, int MODE, int MT, int NW>
__global__ __launch_bounds__(NW* kWave) void k_mx_narrow(MxArgs a) {
  constexpr int NM = ACT == MX_ACT_SWIGLU ? 2 : 1;
  static_assert(MODE != kSum || ACT == MX_ACT_NONE, "a gated product is not linear in its sums");
  static_assert(MODE != kTiles || SRC == kMxF4, "grouped rows are quantised beside the grouping");
  static_assert(MT == 1 || (MODE == kDense && (MT == 2 || SRC == kMxF4)), "more row tiles are for dense products, more than two for codes");
  __shared__ __align__(16) float red[NM][NW][16][20];   // 20: four-float stores, fewer bank conflicts
  __shared__ int32_t list[kDirectPairs];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int r = lane & 15, q = lane >> 4;
  const int y = blockIdx.x / a.nblk, bx = blockIdx.x % a.nblk;
  const int n0 = bx * 16;
  const uint32_t pitch = a.chunks * 128u, spitch = a.chunks * 8u;
  const uint32_t wr = n0 + r < a.N ? r : a.N - 1 - n0;   // a row past the end is read again and not stored
  const uint32_t wco = wr * pitch + q * 32, wso = wr * spitch + q * 2;
  const int64_t wc0 = n0 * static_cast<int64_t>(pitch), ws0 = n0 * static_cast<int64_t>(spitch);

  // where the rows come from, and where they go
  int count = 0;
  int64_t off = 0;
  const int32_t* pairs = nullptr;
  int64_t offs = 0;    // kSum: lane i has expert i's blob and weight
  float wts = 0.f;
  if constexpr (MODE == kDense) {
    count = a.M - y * 16 * MT;
    count = count < 16 * MT ? count : 16 * MT;
  } else if constexpr (MODE == kDirect) {
    const int id = a.ids[lane < a.M ? lane : 0];
    const int e = __builtin_amdgcn_readlane(id, y);
    const uint64_t same = __ballot(lane < a.M && id == e);
    if (__ffsll(static_cast<unsigned long long>(same)) - 1 != y) return;
    off = blob_of(a.slots, e, a.E, a.need, a.pool_bytes);
    count = __popcll(same);
    if (wave == 0 && ((same >> lane) & 1ull)) list[__popcll(same & lane_mask_lt(lane))] = lane;
    __syncthreads();
    pairs = list;
    if (off < 0 && tid == 0 && bx == 0) atomicOr(a.flags, 1u);
  } else if constexpr (MODE == kTiles) {
    if (y >= *a.ntiles) return;
    const MxTile t = a.tiles[y];
    count = t.count;
    off = t.off;
    pairs = a.plist + t.first;
  } else {
    count = 1;
    if (lane < a.k) {
      const int e = a.ids[y * a.k + lane];
      wts = a.wts[y * a.k + lane];
      offs = blob_of(a.slots, e, a.E, a.need, a.pool_bytes);
      if (offs < 0 && wave == 0 && bx == 0) atomicOr(a.flags, 1u);
    }
  }

  static_assert(kDirectPairs <= kWave, "one id per lane");
  for (int g0 = 0; g0 < (MODE == kDirect ? count : 1); g0 += 16) {
    const int here = MODE == kDirect ? (count - g0 < 16 ? count - g0 : 16) : count;
    // A's rows: kDense and kSum from a uniform base, the others by the list
    int64_t row0 = 0;
    int64_t row[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) row[t] = t * 16 + r;
    if constexpr (MODE == kDense) row0 = static_cast<int64_t>(y) * 16 * MT;
    if constexpr (MODE == kDirect || MODE == kTiles) {
      const int p = r < here ? pairs[g0 + r] : 0;
      row[0] = a.pair_rows ? p : p / a.k;
    }
    v4f acc[MT][NM];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int m = 0; m < NM; ++m) acc[t][m] = v4f{0.f, 0.f, 0.f, 0.f};
    const int tasks = MODE == kSum ? a.k * a.chunks : a.chunks;

    // one task: a chunk of k (kSum: of one expert)
    RawPart<SRC> A[MT];
    RawPart<kMxF4> W[NM];
    float w = 1.f;
    bool usable = true;
    const auto load = [&](int task) {
      int chunk = task;
      const uint8_t *wc = a.wc, *wsc = a.wsc;
      int64_t o = off;
      if constexpr (MODE == kSum) {
        const int i = task / a.chunks;
        chunk = task - i * a.chunks;
        row0 = a.pair_rows ? static_cast<int64_t>(y) * a.k + i : y;
        o = readlane64(offs, i);
        w = readlane_f(wts, i);
      }
      if constexpr (SRC == kMxF4) {
        const uint8_t* ac = static_cast<const uint8_t*>(a.a) + row0 * pitch + chunk * 128;
        const uint8_t* as = a.as + row0 * spitch + chunk * 8;
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          if constexpr (MODE == kTiles) load_codes(ac + row[t] * pitch, as + row[t] * spitch, q * 32, q * 2, r < here, A[t].p);
          else load_codes(ac, as, static_cast<uint32_t>(row[t]) * pitch + q * 32, static_cast<uint32_t>(row[t]) * spitch + q * 2,
                          t * 16 + r < here, A[t].p);
        }
      } else {
        const int c0 = chunk * kChunk + q * 64;
        const auto* av = static_cast<const typename Stored<SRC>::T*>(a.a) + row0 * a.K;
#pragma unroll
        for (int t = 0; t < MT; ++t) load_values<SRC>(av, row[t] * a.K + c0, a.K - c0, t * 16 + r < here, A[t]);
      }
      if constexpr (MODE != kDense) {
        usable = o >= 0;   // an unusable expert's product is zero, whatever A holds
        wc = a.pool + o + a.codes_off;
        wsc = a.pool + o + a.scales_off;
      }
      wc += wc0 + chunk * 128;
      wsc += ws0 + chunk * 8;
#pragma unroll
      for (int m = 0; m < NM; ++m)
        load_codes(wc + m * a.N * static_cast<int64_t>(pitch), wsc + m * a.N * static_cast<int64_t>(spitch), wco, wso, usable,
                   W[m].p);
    };
    // the next task's loads are requested before this one is multiplied
    bool have = false;
    for (int task = wave;; task += NW) {
      Part pa[MT], pw[NM];
      const float w0 = w;
      const bool product = have && usable;
      if (product) {
#pragma unroll
        for (int t = 0; t < MT; ++t) pa[t] = finish_part<SRC>(A[t]);
#pragma unroll
        for (int m = 0; m < NM; ++m) pw[m] = W[m].p;
      }
      const bool more = task < tasks;
      if (more) load(task);
      if (product) {
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int m = 0; m < NM; ++m) {
            v4f d = MODE == kSum ? v4f{0.f, 0.f, 0.f, 0.f} : acc[t][m];
            d = mfma4(pw[m].c[0], pa[t].c[0], d, pw[m].sc, pa[t].sc, 0);
            d = mfma4(pw[m].c[1], pa[t].c[1], d, pw[m].sc, pa[t].sc, 1);
            if constexpr (MODE == kSum) {
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[t][m][i] = fmaf(w0, d[i], acc[t][m][i]);
            } else {
              acc[t][m] = d;
            }
          }
      }
      if (!more) break;
      have = true;
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      if (t > 0) __syncthreads();
#pragma unroll
      for (int m = 0; m < NM; ++m) *reinterpret_cast<v4f*>(&red[m][wave][r][4 * q]) = acc[t][m];
      __syncthreads();
      if (tid < 256) {
        const int tr = tid >> 4, n = tid & 15;
        if (t * 16 + tr < here && n0 + n < a.N) {
          float v[NM];
#pragma unroll
          for (int m = 0; m < NM; ++m) {
            v[m] = 0.f;
#pragma unroll
            for (int x = 0; x < NW; ++x) v[m] += red[m][x][tr][n];
          }
          int64_t to;
          if constexpr (MODE == kDense) to = static_cast<int64_t>(y) * 16 * MT + t * 16 + tr;
          else if constexpr (MODE == kSum) to = y;
          else to = pairs[g0 + tr];
          store_out(a.out, to * a.N + n0 + n, NM == 2 ? silu(v[0]) * v[NM - 1] : v[0], a.out_bf16);
        }
      }
    }
    if (MODE == kDirect) __syncthreads();
  }
}

// Many rows of A: a block forms BM rows of A x BN rows of W.  Both operands'
// codes (128 bytes of a row per chunk) go to LDS with direct loads, through S
// stages: while a chunk is multiplied the next S - 1 are on their way.  Their
// scales go with every second chunk, 16 bytes of a row for two chunks (4-byte
// loads with every chunk touched as many lines as the codes: 8192^3 took 308
// instead of 282 us).  Of a row's eight 16-byte pieces, piece c lies at c ^ (row
// mod 8) ^ (row / 8 mod 2), so that sixteen lanes reading one piece of sixteen
// rows use all 64 banks once (without the last term half of them twice: five
// times the bank conflicts, 301 against 299 us for 8192^3, 11.8 against 11.2
// for 256 x 4096 x 4096).
//   Rows of W past N and rows of A past M read as zeros (the buffer
//   descriptors end there; a row's offset is in the lane's part of the
//   address, which the bounds check compares with what the scalar part leaves)
//   and are not stored; with SWIGLU the first half of a block's W rows are gate
//   rows and the second half the up rows of the same outputs.
//   Every wave issues the same number of loads for a chunk (a wave without a
//   share repeats the last one, the same bytes to the same place), so that all
//   but the newest chunk's have landed once no more than that number is left.
//   Bound: 8192^3 by the clock that its power leaves (2.0 GHz, the matrix units
// busy 40% of the time; the same instructions on registers alone, with random
// codes, reach 7.1 PFLOP/s): 282 to 320 us by what ran before it, 3.4 to 3.9
// PFLOP/s (the figures above, "instead of", were taken in turn on one card);
// experts by the reads of W, 4.4 TB/s where a pure read reaches 6.4.
//   KS = 2: a stage is two chunks, and two groups of waves multiply one each,
//   their sums joined at the end.  For long rows of tiles that do not fill the
//   GPU.  512 x 2048 outputs, one group and two, us in the product: 4 chunks
//   5.75, 5.81; 5 chunks 6.31, 6.45; 6 chunks 6.88, 6.63; 8 chunks 7.99, 7.40; 12
//   chunks 10.3, 8.95; 16 chunks 12.6, 10.5; 32 chunks 21.7, 17.0; the same steps
//   with 8 to 256 tiles.  mx_linear_forward takes two from 16 chunks on, which
//   leaves out 6 to 15, where two are faster too.
template <int WM, int WN, int TM, int TN, int S, int KS>
struct TileCfg {
  static constexpr int kGroup = WM * WN, kWaves = KS * kGroup;
  static constexpr int kBM = WM * TM * 16, kBN = WN * TN * 16, kRows = kBM + kBN;
  static constexpr int kStage = KS * kRows * 128;           // the codes of a stage's chunks
  // rows of a direct load: 8 of codes, 64 of scales, each of one operand
  static constexpr int kCodeGroups = kRows / 8, kAScales = (kBM + 63) / 64, kScaleGroups = kAScales + kBN / 64;
  static constexpr int kScales = kScaleGroups * 1024;       // the scales of two chunks
  static constexpr int kPC = (KS * kCodeGroups + kWaves - 1) / kWaves, kPS = (kScaleGroups + kWaves - 1) / kWaves;
  static constexpr int kSBufs = KS == 1 ? S / 2 + 1 : S;    // chunk pairs that S stages in a row can touch
  static constexpr size_t kLds = S * static_cast<size_t>(kStage) + kSBufs * static_cast<size_t>(kScales);
  // loads of the S - 2 stages after an even and after an odd one: every stage,
  // with KS = 1 every even one, brings scales
  static constexpr int kNewEven = (S - 2) * kPC + (KS == 1 ? (S - 2) / 2 : S - 2) * kPS;
  static constexpr int kNewOdd = (S - 2) * kPC + (KS == 1 ? (S - 1) / 2 : S - 2) * kPS;
  static_assert(S >= 2 && kNewOdd < 64, "the wait counter has six bits");
  static_assert(kBM % 8 == 0 && kBN % 64 == 0 && (KS == 1 || KS == 2), "whole groups");
  static_assert(KS == 1 || kGroup * TM * TN * 1024 <= S * kStage, "the joined sums fit the stages");
};

// A direct load of 16 bytes a lane (lane l's land at lds + 16 l), as lds_load<16>
// of device_common.h but with the five wait states that a vector memory
// instruction needs behind a vector instruction that wrote one of its scalar
// operands: the compiler does not look into the assembly, and the offset may
// come from v_readfirstlane.
__device__ __forceinline__ void lds_copy(u32x4 rs, uint8_t* lds, uint32_t voff, int soff) {
  const uint32_t la = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_u8*)lds)));
  const uint32_t so = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(soff));
  uint32_t saved;
  asm volatile(
      "s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 4\n\tbuffer_load_dwordx4 %2, %3, %4 offen lds\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(saved)
      : "s"(la), "v"(voff), "s"(rs), "s"(so)
      : "memory");
}

__device__ __forceinline__ int64_t clamp32(int64_t n) { return n < 0xfffffff0ll ? n : 0xfffffff0ll; }

template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

template <int WM, int WN, int TM, int TN, int S, int KS, int ACT, bool EXPERTS>
__global__ __launch_bounds__(KS* WM* WN* kWave) void k_mx_tile(MxArgs a) {
  using C = TileCfg<WM, WN, TM, TN, S, KS>;
  constexpr int NM = ACT == MX_ACT_SWIGLU ? 2 : 1;
  constexpr int kCols = C::kBN / NM;                       // outputs of a block
  static_assert(kCols % 64 == 0, "a group of scales is of one matrix");
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int r = lane & 15, q = lane >> 4;
  const int kg = wave / C::kGroup, wm = wave % C::kGroup / WN, wn = wave % WN;
  const int pitch = a.chunks * 128, spitch = a.chunks * 8;

  // which tile: an XCD (blockIdx mod 8) runs a contiguous range of them, so
  // that neighbours share rows through its L2
  int mt, nb, count = 0;
  int64_t blob = 0;
  const int32_t* pairs = nullptr;
  {
    const int tiles = EXPERTS ? *a.ntiles : (a.M + C::kBM - 1) / C::kBM;
    const int total = tiles * a.nblk, per = (total + 7) / 8;
    const int idx = static_cast<int>(blockIdx.x & 7) * per + static_cast<int>(blockIdx.x >> 3);
    if (static_cast<int>(blockIdx.x >> 3) >= per || idx >= total) return;
    if constexpr (EXPERTS) {
      mt = idx / a.nblk;
      nb = idx % a.nblk;
      const MxTile t = a.tiles[mt];
      count = t.count;
      blob = t.off;
      pairs = a.plist + t.first;
    } else {
      // bands of eight row tiles, columns outermost inside a band
      const int band = idx / (8 * a.nblk), in = idx % (8 * a.nblk);
      const int high = tiles - band * 8 < 8 ? tiles - band * 8 : 8;
      mt = band * 8 + in % high;
      nb = in / high;
      count = a.M - mt * C::kBM;
    }
  }
  const int n0 = nb * kCols;
  const int64_t m0 = static_cast<int64_t>(mt) * C::kBM;

  v4f acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

  if (blob >= 0) {
    const uint8_t* wc = EXPERTS ? a.pool + blob + a.codes_off : a.wc;
    const uint8_t* wsc = EXPERTS ? a.pool + blob + a.scales_off : a.wsc;
    const int64_t left = a.N - n0;
    u32x4 rw[NM], rws[NM];
#pragma unroll
    for (int m = 0; m < NM; ++m) {
      const int64_t row = n0 + m * static_cast<int64_t>(a.N);
      rw[m] = raw_rsrc(wc + row * pitch, clamp32(left * pitch));
      rws[m] = raw_rsrc(wsc + row * spitch, clamp32(left * spitch));
    }
    const uint8_t* ab = static_cast<const uint8_t*>(a.a);
    const u32x4 ra = EXPERTS ? raw_rsrc(ab, clamp32(static_cast<int64_t>(a.arows) * pitch))
                             : raw_rsrc(ab + m0 * pitch, clamp32(static_cast<int64_t>(count) * pitch));
    const u32x4 ras = EXPERTS ? raw_rsrc(a.as, clamp32(static_cast<int64_t>(a.arows) * spitch))
                              : raw_rsrc(a.as + m0 * spitch, clamp32(static_cast<int64_t>(count) * spitch));
    // a stage's row -> its row in its operand
    const auto row_at = [&](int row) {
      if (row < C::kBM) {
        if constexpr (EXPERTS) {
          const int p = pairs[row < count ? row : count - 1];
          return static_cast<uint32_t>(a.pair_rows ? p : p / a.k);
        }
        return static_cast<uint32_t>(row);
      }
      row -= C::kBM;
      return static_cast<uint32_t>(NM == 2 && row >= kCols ? row - kCols : row);
    };
    // this wave's loads: a lane takes piece lane mod 8 of row lane / 8 of its
    // group; of scales 16 bytes of row lane (with an odd number of chunks the
    // last 8 of them lie past the row's end and are not used)
    uint32_t vc[C::kPC], vs[C::kPS];
#pragma unroll
    for (int i = 0; i < C::kPC; ++i) {
      int g = wave + i * C::kWaves;
      g = (g < KS * C::kCodeGroups ? g : KS * C::kCodeGroups - 1) % C::kCodeGroups;
      vc[i] = row_at(g * 8 + (lane >> 3)) * pitch + static_cast<uint32_t>(((lane & 7) ^ (lane >> 3) ^ (g & 1)) << 4);
    }
#pragma unroll
    for (int i = 0; i < C::kPS; ++i) {
      int g = wave + i * C::kWaves;
      g = g < C::kScaleGroups ? g : C::kScaleGroups - 1;
      const int row = g * 64 + lane;
      vs[i] = row_at(g >= C::kAScales ? row - C::kAScales * 64 + C::kBM : row < C::kBM ? row : C::kBM - 1) * spitch;
    }
    int sput = 0, sget = 0;   // buffers of scales
    const auto fetch = [&](int stage, int buf) {
      uint8_t* st = smem + buf * C::kStage;
#pragma unroll
      for (int i = 0; i < C::kPC; ++i) {
        int g = wave + i * C::kWaves;
        g = g < KS * C::kCodeGroups ? g : KS * C::kCodeGroups - 1;
        const int row = g % C::kCodeGroups * 8;
        int chunk = stage * KS + g / C::kCodeGroups;
        if (KS == 2 && chunk >= a.chunks) chunk = a.chunks - 1;   // not multiplied
        const u32x4 rs = row < C::kBM ? ra : (NM == 2 && row >= C::kBM + kCols ? rw[NM - 1] : rw[0]);
        lds_copy(rs, st + g * 1024, vc[i], chunk * 128);
      }
      if (KS == 1 && (stage & 1)) return;
      uint8_t* ss = smem + S * C::kStage + sput * C::kScales;
      sput = sput + 1 == C::kSBufs ? 0 : sput + 1;
#pragma unroll
      for (int i = 0; i < C::kPS; ++i) {
        int g = wave + i * C::kWaves;
        g = g < C::kScaleGroups ? g : C::kScaleGroups - 1;
        const int row = (g - C::kAScales) * 64;   // of W
        const u32x4 rs = g < C::kAScales ? ras : (NM == 2 && row >= kCols ? rws[NM - 1] : rws[0]);
        lds_copy(rs, ss + g * 1024, vs[i], stage * KS * 8);
      }
    };

    const int stages = (a.chunks + KS - 1) / KS;
#pragma unroll
    for (int c = 0; c < S - 1; ++c)
      if (c < stages) fetch(c, c);
    int buf = 0;
    for (int stage = 0; stage < stages; ++stage) {
      // the loads of the next S - 2 stages may be on their way still
      if (stage + S - 2 >= stages) wait_loads<0>();
      else if (stage & 1) wait_loads<C::kNewOdd>();
      else wait_loads<C::kNewEven>();
      __syncthreads();   // the stage has arrived everywhere, and the one before it is read to its end
      if (stage + S - 1 < stages) fetch(stage + S - 1, buf == 0 ? S - 1 : buf - 1);
      const uint8_t* st = smem + buf * C::kStage + kg * C::kRows * 128;
      const uint8_t* ss = smem + S * C::kStage + sget * C::kScales + (KS == 1 ? stage & 1 : kg) * 8;
      if (KS == 2 || (stage & 1)) sget = sget + 1 == C::kSBufs ? 0 : sget + 1;
      buf = buf + 1 == S ? 0 : buf + 1;
      if (KS == 2 && stage * KS + kg >= a.chunks) continue;
      int sa[TM], sw[TN];
#pragma unroll
      for (int i = 0; i < TM; ++i)
        sa[i] = *reinterpret_cast<const uint16_t*>(ss + ((wm * TM + i) * 16 + r) * 16 + q * 2);
      const auto wrow = [&](int j) {   // W rows of this wave's tile j: with SWIGLU gate and up tiles in turn
        return NM == 1 ? (wn * TN + j) * 16 : (j & 1) * kCols + (wn * (TN / 2) + j / 2) * 16;
      };
#pragma unroll
      for (int j = 0; j < TN; ++j)
        sw[j] = *reinterpret_cast<const uint16_t*>(ss + (C::kAScales * 64 + wrow(j) + r) * 16 + q * 2);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int at = ((2 * q + s) ^ (r & 7) ^ (r >> 3)) << 4;
        v4i fa[TM], fw[TN];
#pragma unroll
        for (int j = 0; j < TN; ++j) fw[j] = *reinterpret_cast<const v4i*>(st + (C::kBM + wrow(j) + r) * 128 + at);
#pragma unroll
        for (int i = 0; i < TM; ++i) fa[i] = *reinterpret_cast<const v4i*>(st + ((wm * TM + i) * 16 + r) * 128 + at);
        // one W tile with all of A's: 281 against 287 us for 8192^3 the other way round
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
          for (int i = 0; i < TM; ++i) acc[i][j] = mfma4(fw[j], fa[i], acc[i][j], sw[j], sa[i], s);
      }
    }
  }

  if constexpr (KS == 2) {
    __syncthreads();   // every stage is read to its end (or there was none)
    v4f* part = reinterpret_cast<v4f*>(smem) + (wave % C::kGroup) * TM * TN * kWave + lane;
    if (kg == 1)
#pragma unroll
      for (int i = 0; i < TM * TN; ++i) part[i * kWave] = acc[i / TN][i % TN];
    __syncthreads();
    if (kg == 1) return;
#pragma unroll
    for (int i = 0; i < TM * TN; ++i) acc[i / TN][i % TN] += part[i * kWave];
  }

  // a lane holds four consecutive outputs of one row
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int m = (wm * TM + i) * 16 + r;
    if (m >= count) continue;
    const int64_t to = (EXPERTS ? static_cast<int64_t>(pairs[m]) : m0 + m) * a.N;
#pragma unroll
    for (int j = 0; j < TN; j += NM) {
      const int n = n0 + (NM == 1 ? (wn * TN + j) * 16 : (wn * (TN / 2) + j / 2) * 16) + 4 * q;
      float y[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) y[x] = NM == 2 ? silu(acc[i][j][x]) * acc[i][j + NM - 1][x] : acc[i][j][x];
      if (n + 4 <= a.N) {   // aligned to an element only if N is not a multiple of four (element
                            // stores: 35.4 instead of 25.7 us for 4082 x 2683 x 1020)
        if (a.out_bf16) {
          uint32_t w[2];
          w[0] = to_bf16(y[0]) | (static_cast<uint32_t>(to_bf16(y[1])) << 16);
          w[1] = to_bf16(y[2]) | (static_cast<uint32_t>(to_bf16(y[3])) << 16);
          __builtin_memcpy(static_cast<uint16_t*>(a.out) + to + n, w, 8);
        } else {
          __builtin_memcpy(static_cast<float*>(a.out) + to + n, y, 16);
        }
      } else {
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (n + x < a.N) store_out(a.out, to + n + x, y[x], a.out_bf16);
      }
    }
  }
}

// Before the tiles: block 0 groups the pairs by expert, the others quantise A.
//
// Grouping is one block's work: count (LDS atomics, which hand out each pair's
// place within its expert), scan, place.  The order of an expert's pairs does
// not change any result, since every pair has its own column of the product.
// Up to kPrepThr * 4 * NI pairs stay in registers between the passes (four
// consecutive ids a load, all requested at once) and are placed in LDS, from
// where the list is written in order (scattered 4-byte stores to memory took
// half of 18 us for 20480 pairs); more are read again and placed in memory
// (NI = 0).  20480 pairs and 2048 x 2048 bf16 values take 11 us, 512 pairs and
// 512 x 512 values 4.0 us.
constexpr int kPrepThr = 1024;

struct PrepArgs {
  MxArgs g;
  int P, rows;            // pairs; most pairs of a tile
  int32_t* place;
  int32_t* plist;
  MxTile* tiles;
  int32_t* ntiles;
  const void* x;          // A, fp32 or bf16, to quantise; NULL: nothing
  int64_t pieces, cols;
  uint32_t per_row;
  uint32_t* codes;
  uint8_t* scales;
};

template <int NI>
__device__ __forceinline__ void group_pairs(const PrepArgs& p) {
  __shared__ int32_t cnt[kMaxExperts + 1];       // the last: pairs whose id is unusable
  __shared__ int32_t sum_p[kPrepThr / kWave], sum_t[kPrepThr / kWave];
  __shared__ int32_t start[kMaxExperts + 1];
  __shared__ __align__(16) uint16_t listed[NI > 0 ? NI * 4 * kPrepThr : 1];
  const MxArgs& a = p.g;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const int P = p.P, E = a.E;
  const auto bucket = [&](int id) { return id >= 0 && id < E ? id : E; };
  // bucket (11 bits) and place of each pair
  uint32_t kept[NI > 0 ? NI : 1][4];
  if constexpr (NI > 0) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int at = (i * kPrepThr + tid) * 4;
      if (at + 4 <= P) __builtin_memcpy(kept[i], a.ids + at, 16);
      else
#pragma unroll
        for (int x = 0; x < 4; ++x) kept[i][x] = at + x < P ? static_cast<uint32_t>(a.ids[at + x]) : 0u;
    }
  }
  // the slots of this thread's expert, requested before they are needed
  const int64_t off = tid < E ? blob_of(a.slots, tid, E, a.need, a.pool_bytes) : -1;
  for (int e = tid; e <= E; e += kPrepThr) cnt[e] = 0;
  __syncthreads();
  if constexpr (NI > 0) {
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if ((i * kPrepThr + tid) * 4 + x < P) {
          const uint32_t b = static_cast<uint32_t>(bucket(static_cast<int>(kept[i][x])));
          kept[i][x] = b | (static_cast<uint32_t>(atomicAdd(&cnt[b], 1)) << 11);
        }
  } else {
    for (int i = tid; i < P; i += kPrepThr) p.place[i] = atomicAdd(&cnt[bucket(a.ids[i])], 1);
  }
  __syncthreads();
  // exclusive scans of the pair and tile counts; the bucket of unusable ids
  // (index E <= 1024, one past the threads at most) comes last
  const int c = tid < E ? cnt[tid] : 0;
  const int nt = (c + p.rows - 1) / p.rows;
  int ip = c, it = nt;
  for (int s = 1; s < kWave; s <<= 1) {
    const int op = __shfl_up(ip, s), ot = __shfl_up(it, s);
    if (lane >= s) { ip += op; it += ot; }
  }
  if (lane == kWave - 1) { sum_p[wave] = ip; sum_t[wave] = it; }
  __syncthreads();
  int bp = 0, bt = 0, tp = 0, tt = 0;
#pragma unroll
  for (int w = 0; w < kPrepThr / kWave; ++w) {
    if (w < wave) { bp += sum_p[w]; bt += sum_t[w]; }
    tp += sum_p[w];
    tt += sum_t[w];
  }
  const int sp = bp + ip - c, st = bt + it - nt;
  if (tid < E) start[tid] = sp;
  const int lost = cnt[E], lost_t = (lost + p.rows - 1) / p.rows;
  if (tid == 0) {
    *p.ntiles = tt + lost_t;
    start[E] = tp;
    if (lost) atomicOr(a.flags, 1u);
  }
  __syncthreads();
  if constexpr (NI > 0) {
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int at = (i * kPrepThr + tid) * 4 + x;
        if (at < P) listed[start[kept[i][x] & 2047u] + (kept[i][x] >> 11)] = static_cast<uint16_t>(at);
      }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int at = (i * kPrepThr + tid) * 4;
      int32_t four[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) four[x] = listed[at + x];
      if (at + 4 <= P) *reinterpret_cast<int4*>(p.plist + at) = int4{four[0], four[1], four[2], four[3]};
      else
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (at + x < P) p.plist[at + x] = four[x];
    }
  } else {
    for (int i = tid; i < P; i += kPrepThr) p.plist[start[bucket(a.ids[i])] + p.place[i]] = i;
  }
  if (c > 0) {
    if (off < 0) atomicOr(a.flags, 1u);
    for (int i = 0; i < nt; ++i) {
      const int left = c - i * p.rows;
      p.tiles[st + i] = MxTile{off, sp + i * p.rows, left < p.rows ? left : p.rows};
    }
  }
  for (int i = tid; i < lost_t; i += kPrepThr) {
    const int left = lost - i * p.rows;
    p.tiles[tt + i] = MxTile{-1, tp + i * p.rows, left < p.rows ? left : p.rows};
  }
}

template <int SRC, int NI>
__global__ __launch_bounds__(kPrepThr) void k_mx_prep(PrepArgs p) {
  if (blockIdx.x == 0) {
    group_pairs<NI>(p);
    return;
  }
  if constexpr (SRC != kMxF4) {
    mx_quantize_piece<SRC>(p.x, p.cols, p.cols, p.per_row, static_cast<int64_t>(blockIdx.x - 1) * kPrepThr + threadIdx.x,
                           p.pieces, p.codes, p.scales);
  }
}

// out[t] = sum_i w[t, i] rows[t k + i], i ascending, over the pairs that have an
// expert (a weight of another pair may be anything).  The rows are fp32: half
// the bytes would round every product before the sum.  Ids, rows and slots are
// requested in this order, so that the rows come while the slots are looked up.
// 64 tokens' 8 rows of 2048: 4.0 to 4.6 us, little over a launch; 2048 tokens'
// 10 rows: 36 us, 5.2 TB/s.
__global__ __launch_bounds__(256) void k_mx_combine(MxArgs a, const float* rows) {
  constexpr int kStep = 8;
  const int t = blockIdx.x / a.nblk, lane = threadIdx.x & (kWave - 1);
  const int n = (blockIdx.x % a.nblk) * 256 + threadIdx.x;
  const int64_t p0 = static_cast<int64_t>(t) * a.k;
  const int at = lane < a.k ? lane : 0;   // k <= 64
  const int id = a.ids[p0 + at];
  const float w = a.wts[p0 + at];
  const float* row = rows + p0 * a.N + (n < a.N ? n : a.N - 1);
  float v[kStep], y = 0.f;
  const auto load = [&](int i0) {
#pragma unroll
    for (int x = 0; x < kStep; ++x) v[x] = row[static_cast<int64_t>(i0 + x < a.k ? i0 + x : a.k - 1) * a.N];
  };
  load(0);
  const uint64_t usable = __ballot(lane < a.k && blob_of(a.slots, id, a.E, a.need, a.pool_bytes) >= 0);
  for (int i0 = 0;;) {
#pragma unroll
    for (int x = 0; x < kStep; ++x) {
      const int i = i0 + x < kWave ? i0 + x : kWave - 1;
      if (i0 + x < a.k && ((usable >> i) & 1ull)) y = fmaf(readlane_f(w, i), v[x], y);
    }
    i0 += kStep;
    if (i0 >= a.k) break;
    load(i0);
  }
  if (n < a.N) store_out(a.out, static_cast<int64_t>(t) * a.N + n, y, a.out_bf16);
}

// ---------------------------------------------------------------------------

int bad(const char* fmt, long long x = 0, long long y = 0) {
  char buf[256];
  snprintf(buf, sizeof(buf), fmt, x, y);
  return api_fail(MOE_EINVAL, buf);
}

bool at(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int check_product(const mx_product_desc* d, bool experts) {
  if (!d) return bad("product descriptor is NULL");
  if (d->n < 1 || d->n > (1 << 20) || d->k < 1 || d->k > (1 << 20)) return bad("n=%lld and k=%lld must be in [1, 2^20]", d->n, d->k);
  if (d->a_dtype != MOE_F32 && d->a_dtype != MOE_BF16 && d->a_dtype != MX_FP4)
    return bad("a_dtype=%lld is not MOE_F32, MOE_BF16 or MX_FP4", d->a_dtype);
  if (d->out_dtype != MOE_F32 && d->out_dtype != MOE_BF16) return bad("out_dtype=%lld is neither MOE_F32 nor MOE_BF16", d->out_dtype);
  if (d->act != MX_ACT_NONE && d->act != MX_ACT_SWIGLU) return bad("act=%lld is not a MX_ACT_* code", d->act);
  if (!experts) {
    if (d->n_experts || d->top_k || d->pair_rows || d->codes_off || d->scales_off || d->pool_bytes)
      return bad("the fields of a product by expert must be 0 for a dense one");
    return MOE_OK;
  }
  if (d->n_experts < 1 || d->n_experts > kMaxExperts) return bad("n_experts=%lld must be in [1, 1024]", d->n_experts);
  if (d->top_k < 1 || d->top_k > 64) return bad("top_k=%lld must be in [1, 64]", d->top_k);
  if (d->pair_rows != 0 && d->pair_rows != 1) return bad("pair_rows=%lld must be 0 or 1", d->pair_rows);
  if (d->codes_off < 0 || d->codes_off % 16 || d->scales_off < 0 || d->scales_off % 16 || d->codes_off > (int64_t(1) << 40) ||
      d->scales_off > (int64_t(1) << 40))
    return bad("codes_off=%lld and scales_off=%lld must be multiples of 16 in [0, 2^40]", d->codes_off, d->scales_off);
  const int64_t rows = static_cast<int64_t>(d->n) * (d->act == MX_ACT_SWIGLU ? 2 : 1);
  const int64_t nc = mx_codes_bytes(rows, d->k), ns = mx_scales_bytes(rows, d->k);
  if (d->codes_off < d->scales_off + ns && d->scales_off < d->codes_off + nc) return bad("a blob's codes and scales overlap");
  if (d->pool_bytes < d->codes_off + nc || d->pool_bytes < d->scales_off + ns)
    return bad("pool_bytes=%lld is smaller than one blob", d->pool_bytes);
  return MOE_OK;
}

// The tiles' offsets into A have 32 bits.
bool far_rows(int64_t rows, int k) { return rows * (mx_padded(k) / 2) >= (int64_t(1) << 32) - 65536; }

constexpr int64_t kMostThreads = int64_t(1) << 32;   // a launch holds fewer

// How P pairs are grouped: rows per tile, the most tiles, and the threads of
// their launch.
//   By the pairs that an expert has on average (gate and up rows, 512 outputs,
// k = 2048; tiles of 32, 64 and 128 rows): 16 pairs 63, 65, 76 us; 32 pairs 77,
// 72, 83; 64 pairs 102, 90, 92; 96 pairs 70, 61, 56; 256 pairs 76, 63, 58.
// Where the launch would hold too many threads the tiles are higher.  An A
// beyond 4 GiB takes the kernel of few rows.
struct Grouping {
  int bm;
  int64_t tiles, threads;
};

Grouping grouping(const mx_product_desc& d, int64_t P, int64_t rows) {
  const int64_t some = P < d.n_experts + 1 ? P : d.n_experts + 1;   // experts with pairs, and the pairs without one
  if (far_rows(rows, d.k)) {
    const int64_t tiles = some + P / 16;
    return {16, tiles, tiles * ((d.n + 15) / 16) * (8 * kWave)};
  }
  const int64_t each = P / d.n_experts;
  const int cols = d.act == MX_ACT_SWIGLU ? 64 : 128;   // outputs of a tile; its block is four waves
  for (int bm = each >= 96 ? 128 : each >= 24 ? 64 : 32;; bm *= 2) {
    const int64_t tiles = some + P / bm, threads = (tiles * ((d.n + cols - 1) / cols) + 7) / 8 * 8 * (4 * kWave);
    if (threads < kMostThreads || bm == 128) return {bm, tiles, threads};
  }
}

int check_rows(const mx_product_desc& d, int32_t T, bool experts) {
  if (T < 0 || T > (experts ? 65536 : (1 << 20))) return bad("%lld rows are negative or too many", T);
  const int64_t P = static_cast<int64_t>(T) * (experts ? d.top_k : 1), rows = experts && !d.pair_rows ? T : P;
  if (P * ((d.n + 15) / 16) >= (int64_t(1) << 31)) return bad("%lld rows of %lld columns are too many for one launch", P, d.n);
  // every launch that may follow: the quantisation (of a launch before a dense
  // product four pieces a thread, with the grouping one), the sums over a
  // token's experts, the products of grouped rows
  const int64_t pieces = rows * (mx_padded(d.k) / 8);
  if (d.a_dtype != MX_FP4 && pieces / (experts ? 1 : 4) >= kMostThreads - 2048)
    return bad("%lld rows of %lld values are too many to quantise in one launch", rows, d.k);
  if (!experts) return MOE_OK;
  if (P >= (1 << 22)) return bad("T * top_k = %lld must be below 2^22", P);
  if (T * ((d.n + 255) / 256 * int64_t(256)) >= kMostThreads) return bad("%lld rows of %lld columns are too many for one launch", T, d.n);
  if (grouping(d, P, rows).threads >= kMostThreads) return bad("%lld pairs of %lld columns are too many for one launch", P, d.n);
  return MOE_OK;
}

struct MxWs {
  size_t codes, scales;      // A as an MX matrix
  size_t place, plist, tiles, ntiles;
  size_t rows;               // fp32 rows of the pairs
  size_t total;
  int max_tiles;
};

// The regions lie behind those at fixed offsets that moe_layer.h's calls keep
// across calls (control words, tagged words), so that one workspace serves both.
MxWs mx_ws(const mx_product_desc& d, int32_t T, bool experts) {
  MxWs w{};
  moe_desc any{};
  any.hidden = any.inter = any.shared_inter = 64;
  any.n_experts = any.top_k = 1;
  size_t o = ws_layout(any, 0).logits;
  auto take = [&](size_t bytes) { const size_t p = o; o += align256(bytes > 0 ? bytes : 1); return p; };
  const int64_t P = static_cast<int64_t>(T) * (experts ? d.top_k : 1);
  const int64_t rows = experts && !d.pair_rows ? T : P;
  const bool quant = d.a_dtype != MX_FP4;
  w.codes = take(quant ? mx_codes_bytes(rows, d.k) : 0);
  w.scales = take(quant ? mx_scales_bytes(rows, d.k) : 0);
  if (experts) {
    w.place = take(P * 4);
    w.plist = take(P * 4);
    w.max_tiles = static_cast<int>((P < d.n_experts + 1 ? P : d.n_experts + 1) + P / 16);
    w.tiles = take(static_cast<size_t>(w.max_tiles) * sizeof(MxTile));
    w.ntiles = take(4);
    w.rows = take(static_cast<size_t>(P) * d.n * 4);
  }
  w.total = o;
  return w;
}

int check_call(const mx_product_desc& d, const void* a, const void* as, int64_t rows, const void* out, int64_t out_rows,
               const void* ws, size_t ws_bytes, const MxWs& L) {
  if (!a || !out) return bad("NULL a or out");
  if (d.a_dtype == MX_FP4) {
    if (!as) return bad("a_scales is NULL");
    if (!at(a, 16) || !at(as, 16)) return bad("codes and scales must be 16-byte aligned");
  } else {
    if (as) return bad("a_scales must be NULL unless a_dtype is MX_FP4");
    if (!at(a, d.a_dtype == MOE_F32 ? 4 : 2)) return bad("a is not aligned to its element");
  }
  if (!at(out, d.out_dtype == MOE_F32 ? 4 : 2)) return bad("out is not aligned to its element");
  if (!ws || !at(ws, 256)) return bad("workspace is NULL or not 256-byte aligned");
  if (ws_bytes < L.total) {
    char buf[160];
    snprintf(buf, sizeof(buf), "workspace has %zu bytes, %zu needed", ws_bytes, L.total);
    return api_fail(MOE_ENOMEM, buf);
  }
  const int64_t n_a = d.a_dtype == MX_FP4 ? mx_codes_bytes(rows, d.k) : rows * d.k * (d.a_dtype == MOE_F32 ? 4 : 2);
  const int64_t n_as = d.a_dtype == MX_FP4 ? mx_scales_bytes(rows, d.k) : 0;
  const int64_t n_o = out_rows * d.n * (d.out_dtype == MOE_F32 ? 4 : 2);
  if (mx_overlaps(out, n_o, a, n_a) || mx_overlaps(out, n_o, as, n_as) || mx_overlaps(out, n_o, ws, ws_bytes) ||
      mx_overlaps(a, n_a, ws, ws_bytes) || mx_overlaps(as, n_as, ws, ws_bytes))
    return bad("out or the workspace overlaps another argument");
  return MOE_OK;
}

int launched() {
  const hipError_t e = hipGetLastError();
  if (e == hipSuccess) return api_ok();
  char buf[256];
  snprintf(buf, sizeof(buf), "product launch failed: %s", hipGetErrorString(e));
  return api_fail(MOE_EHIP, buf);
}

template <int SRC, int MODE, int MT, int NW>
void narrow_act(const MxArgs& a, int act, uint32_t blocks, hipStream_t s) {
  const dim3 grid(blocks), block(NW * kWave);
  if constexpr (MODE != kSum) {
    if (act == MX_ACT_SWIGLU) {
      launch_kernel(k_mx_narrow<SRC, MX_ACT_SWIGLU, MODE, MT, NW>, grid, block, 0, s, a);
      return;
    }
  }
  launch_kernel(k_mx_narrow<SRC, MX_ACT_NONE, MODE, MT, NW>, grid, block, 0, s, a);
}

// Row tiles of more than two take codes (their values do not fit the
// registers), and so do grouped rows.
template <int MODE, int MT, int NW>
void narrow_src(const MxArgs& a, int src, int act, uint32_t blocks, hipStream_t s) {
  if constexpr (MT <= 2 && MODE != kTiles) {
    if (src == kF32) return narrow_act<kF32, MODE, MT, NW>(a, act, blocks, s);
    if (src == kBF16) return narrow_act<kBF16, MODE, MT, NW>(a, act, blocks, s);
  }
  narrow_act<kMxF4, MODE, MT, NW>(a, act, blocks, s);
}

template <int MODE, int MT = 1>
void narrow(MxArgs a, int src, int act, int ny, hipStream_t s) {
  a.nblk = (a.N + 15) / 16;
  const uint32_t blocks = static_cast<uint32_t>(a.nblk) * ny;
  const int tasks = a.chunks * (MODE == kSum ? a.k : 1);
  // a wave's instructions cost more than its loads: four waves with two tasks
  // each take 8.1 us where eight with one take 10.2 (ten experts' gate and up
  // rows, 512 outputs, k = 2048); longer rows need eight to hide their loads
  if (tasks <= 8) narrow_src<MODE, MT, 4>(a, src, act, blocks, s);
  else narrow_src<MODE, MT, 8>(a, src, act, blocks, s);
}

template <int WM, int WN, int TM, int TN, int S, int KS, bool EXPERTS>
int tile(MxArgs a, int act, int64_t tiles, hipStream_t s) {
  using C = TileCfg<WM, WN, TM, TN, S, KS>;
  const int cols = act == MX_ACT_SWIGLU ? C::kBN / 2 : C::kBN;
  a.nblk = (a.N + cols - 1) / cols;
  const dim3 grid(static_cast<uint32_t>((tiles * a.nblk + 7) / 8 * 8)), block(C::kWaves * kWave);
  const auto kernel = act == MX_ACT_SWIGLU ? &k_mx_tile<WM, WN, TM, TN, S, KS, MX_ACT_SWIGLU, EXPERTS>
                                           : &k_mx_tile<WM, WN, TM, TN, S, KS, MX_ACT_NONE, EXPERTS>;
  if (C::kLds > 65536) {
    // once per device (a bit each) and activation
    static std::atomic<uint64_t> done[2];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return MOE_EHIP;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (!(done[act].load(std::memory_order_relaxed) & bit) || !bit) {
      if (hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(C::kLds)) != hipSuccess)
        return MOE_EHIP;
      done[act].fetch_or(bit, std::memory_order_relaxed);
    }
  }
  launch_kernel(kernel, grid, block, static_cast<uint32_t>(C::kLds), s, a);
  return MOE_OK;
}

template <int SRC>
void prep_src(const PrepArgs& p, uint32_t blocks, hipStream_t s) {
  const dim3 grid(blocks), block(kPrepThr);
  if (p.P <= 4 * kPrepThr) launch_kernel(k_mx_prep<SRC, 1>, grid, block, 0, s, p);
  else if (p.P <= 8 * kPrepThr) launch_kernel(k_mx_prep<SRC, 2>, grid, block, 0, s, p);
  else if (p.P <= 24 * kPrepThr) launch_kernel(k_mx_prep<SRC, 6>, grid, block, 0, s, p);
  else launch_kernel(k_mx_prep<SRC, 0>, grid, block, 0, s, p);
}

// Whether blocks of the kernel of few rows quantise A themselves, which saves a
// launch: `rows` of them (a multiple of 16, others cost as much) in each of
// `blocks`.  A block's own part must not hold it up (16 rows of 1024 x 8192 in
// bf16 take 12.2 us against 10.4 with A quantised before, in fp32 20.2) and all
// of them together not the GPU (16 rows of 16384 x 2048 12.8 and 20.7 against
// 10.4).  16 rows of 4096 x 2048 take 5.6 us in bf16 and 7.1 in fp32 against 6.8
// and 6.7 in a row of launches (7.0 and 7.1 against 9.3 where a program's calls
// are as slow as its host: a launch more is 2 us of it), one row 3.8 and 4.7
// against 6.1 and 6.3.  By expert the part may be twice as large, while ids and
// slots are looked up (one token's sum over 8 experts, 2048 outputs, k = 512 in
// fp32: 9.2 us a call against 11.0).
bool quantise_in_place(const mx_product_desc& d, int64_t rows, int64_t blocks, int64_t most) {
  const int64_t bytes = rows * d.k * (d.a_dtype == MOE_F32 ? 4 : 2);
  return d.a_dtype != MX_FP4 && bytes <= most && bytes * blocks <= (3 << 24);
}

MxArgs common_args(const mx_product_desc& d, const void* a, const void* as, void* out, void* ws) {
  MxArgs g{};
  g.a = a;
  g.as = static_cast<const uint8_t*>(as);
  g.out = out;
  g.flags = static_cast<uint32_t*>(ws);
  g.N = d.n;
  g.K = d.k;
  g.chunks = static_cast<int>(mx_padded(d.k) / kChunk);
  g.out_bf16 = d.out_dtype == MOE_BF16;
  return g;
}

}  // namespace
}  // namespace moe

extern "C" {

size_t mx_workspace_bytes(const mx_product_desc* d, int32_t T_max) {
  using namespace moe;
  const bool experts = d && d->n_experts != 0;
  if (check_product(d, experts) != MOE_OK || check_rows(*d, T_max, experts) != MOE_OK) return 0;
  return mx_ws(*d, T_max, experts).total;
}

int mx_linear_forward(const mx_product_desc* d, int32_t M, const void* a, const void* a_scales, const void* w_codes,
                      const void* w_scales, void* out, void* workspace, size_t ws_bytes, void* stream) {
  using namespace moe;
  MarkScope marks;
  int rc;
  if ((rc = check_product(d, false)) || (rc = check_rows(*d, M, false))) return rc;
  if (M == 0) return api_ok();
  const MxWs L = mx_ws(*d, M, false);
  if ((rc = check_call(*d, a, a_scales, M, out, M, workspace, ws_bytes, L))) return rc;
  if (!w_codes || !w_scales || !at(w_codes, 16) || !at(w_scales, 16)) return bad("w_codes and w_scales must be 16-byte aligned and not NULL");
  const int64_t wrows = static_cast<int64_t>(d->n) * (d->act == MX_ACT_SWIGLU ? 2 : 1);
  const int64_t n_o = static_cast<int64_t>(M) * d->n * (d->out_dtype == MOE_F32 ? 4 : 2);
  const int64_t n_c = mx_codes_bytes(wrows, d->k), n_s = mx_scales_bytes(wrows, d->k);
  if (mx_overlaps(out, n_o, w_codes, n_c) || mx_overlaps(out, n_o, w_scales, n_s) ||
      mx_overlaps(workspace, ws_bytes, w_codes, n_c) || mx_overlaps(workspace, ws_bytes, w_scales, n_s))
    return bad("out or the workspace overlaps w_codes or w_scales");
  MxArgs g = common_args(*d, a, a_scales, out, workspace);
  g.M = M;
  g.wc = static_cast<const uint8_t*>(w_codes);
  g.wsc = static_cast<const uint8_t*>(w_scales);
  hipStream_t s = static_cast<hipStream_t>(stream);
  g.arows = M;
  const bool few = M <= 32 && quantise_in_place(*d, M <= 16 ? 16 : 32, (d->n + 15) / 16, 1 << 17);
  if (!few && d->a_dtype != MX_FP4) {
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    launch_mx_quantize(d->a_dtype, M, d->k, a, d->k, ws + L.codes, ws + L.scales, s);
    g.a = ws + L.codes;
    g.as = ws + L.scales;
  }
  if (M <= 64) {
    const int src = few ? d->a_dtype : MX_FP4;
    if (M <= 16) narrow<kDense>(g, src, d->act, 1, s);
    else if (M <= 32) narrow<kDense, 2>(g, src, d->act, 1, s);
    else narrow<kDense, 4>(g, MX_FP4, d->act, 1, s);
    return launched();
  }
  const auto tiles = [&](int bm, int bn) {
    return static_cast<int64_t>((M + bm - 1) / bm) * ((wrows + bn - 1) / bn);
  };
  // the largest tile that still gives most of the 256 CUs one (a 256 x 256 tile
  // reads half as much per product as a 128 x 128 one: 8192^3 takes 309 against
  // 454 us).  us in the product by k = 1024 and 4096, 256 x 256 against 128 x 128:
  // 160 of the larger tiles 17.9, 16.4 and 38.6, 38.4; 176 tiles 18.2, 16.3 and
  // 38.9, 39.0; 208 tiles 18.5, 19.9 and 39.1, 44.0; 256 tiles 19.3, 21.0 and
  // 41.2, 49.6.  128 x 128 against 64 x 128: 176 of the larger 8.0, 7.4 and 17.4,
  // 17.2; 256 tiles 8.6, 8.0 and 18.0, 18.0; 384 tiles 11.5, 11.7 and 23.8, 27.8
  if (tiles(256, 256) >= 192) rc = tile<2, 4, 8, 4, 2, 1, false>(g, d->act, (M + 255) / 256, s);
  else if (tiles(128, 128) >= 192) rc = tile<2, 2, 4, 4, 2, 1, false>(g, d->act, (M + 127) / 128, s);
  else if (tiles(64, 128) > 256 || g.chunks < 16) rc = tile<1, 4, 4, 2, 3, 1, false>(g, d->act, (M + 63) / 64, s);
  else rc = tile<1, 4, 4, 2, 3, 2, false>(g, d->act, (M + 63) / 64, s);
  return rc == MOE_OK ? launched() : api_fail(MOE_EHIP, "the product kernel's LDS size was refused");
}

int mx_experts_forward(const mx_product_desc* d, int32_t T, const void* a, const void* a_scales,
                       const int32_t* topk_ids, const float* topk_w, const int64_t* slot_table, const void* pool_base,
                       void* out, void* workspace, size_t ws_bytes, void* stream) {
  using namespace moe;
  MarkScope marks;
  int rc;
  if ((rc = check_product(d, true)) || (rc = check_rows(*d, T, true))) return rc;
  if (T == 0) return api_ok();
  const MxWs L = mx_ws(*d, T, true);
  const int P = T * d->top_k;
  const int64_t rows = d->pair_rows ? P : T, out_rows = topk_w ? T : P;
  if ((rc = check_call(*d, a, a_scales, rows, out, out_rows, workspace, ws_bytes, L))) return rc;
  if (!topk_ids || !slot_table || !pool_base) return bad("NULL topk_ids, slot_table or pool_base");
  if (!at(topk_ids, 4) || !at(topk_w, 4) || !at(slot_table, 8) || !at(pool_base, 256))
    return bad("misaligned pointer (topk_ids/topk_w 4, slot_table 8, pool_base 256)");
  const int64_t n_o = out_rows * d->n * (d->out_dtype == MOE_F32 ? 4 : 2), n_i = static_cast<int64_t>(P) * 4;
  const int64_t n_t = static_cast<int64_t>(d->n_experts) * 8;
  const void* ins[4] = {topk_ids, topk_w, slot_table, pool_base};
  const int64_t in_n[4] = {n_i, n_i, n_t, d->pool_bytes};
  for (int i = 0; i < 4; ++i)
    if (mx_overlaps(out, n_o, ins[i], in_n[i]) || mx_overlaps(workspace, ws_bytes, ins[i], in_n[i]))
      return bad("out or the workspace overlaps the routing, the slot table or the pool");
  hipStream_t s = static_cast<hipStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  MxArgs g = common_args(*d, a, a_scales, out, workspace);
  const int64_t wrows = static_cast<int64_t>(d->n) * (d->act == MX_ACT_SWIGLU ? 2 : 1);
  const int64_t end_c = d->codes_off + mx_codes_bytes(wrows, d->k), end_s = d->scales_off + mx_scales_bytes(wrows, d->k);
  g.M = P;
  g.k = d->top_k;
  g.E = d->n_experts;
  g.pair_rows = d->pair_rows;
  g.ids = topk_ids;
  g.wts = topk_w;
  g.slots = slot_table;
  g.pool = static_cast<const uint8_t*>(pool_base);
  g.codes_off = d->codes_off;
  g.scales_off = d->scales_off;
  g.need = end_c > end_s ? end_c : end_s;
  g.pool_bytes = d->pool_bytes;
  // a gated product is not linear in its sums, so the weighted sum of a token
  // in one block is for the plain one
  const int nblk = (d->n + 15) / 16;
  const int64_t w_bytes = P * mx_codes_bytes(wrows, d->k);
  const bool sum = topk_w && d->act == MX_ACT_NONE && P <= kSumPairs && w_bytes < kSumBytes;
  const bool direct = !sum && P <= kDirectPairs && w_bytes < kDirectBytes;
  int src = d->a_dtype;
  if ((sum || direct) && src != MX_FP4 &&
      !quantise_in_place(*d, sum ? 16 * d->top_k : 16, static_cast<int64_t>(nblk) * (sum ? T : P), 1 << 18)) {
    launch_mx_quantize(src, rows, d->k, a, d->k, ws + L.codes, ws + L.scales, s);
    g.a = ws + L.codes;
    g.as = ws + L.scales;
    src = MX_FP4;
  }
  if (sum) {
    narrow<kSum>(g, src, d->act, T, s);
    return launched();
  }
  if (topk_w) {
    g.out = ws + L.rows;
    g.out_bf16 = 0;
  }
  if (direct) {
    narrow<kDirect>(g, src, d->act, P, s);
  } else {
    g.arows = static_cast<int>(rows);
    const Grouping by = grouping(*d, P, rows);
    PrepArgs p{};
    p.g = g;
    p.P = P;
    p.rows = by.bm;
    p.place = reinterpret_cast<int32_t*>(ws + L.place);
    p.plist = reinterpret_cast<int32_t*>(ws + L.plist);
    p.tiles = reinterpret_cast<MxTile*>(ws + L.tiles);
    p.ntiles = reinterpret_cast<int32_t*>(ws + L.ntiles);
    if (d->a_dtype == MX_FP4) {
      prep_src<kMxF4>(p, 1, s);
    } else {
      p.x = a;
      p.cols = d->k;
      p.per_row = static_cast<uint32_t>(mx_padded(d->k) / 8);
      p.pieces = rows * p.per_row;
      p.codes = reinterpret_cast<uint32_t*>(ws + L.codes);
      p.scales = ws + L.scales;
      const uint32_t blocks = static_cast<uint32_t>(1 + (p.pieces + kPrepThr - 1) / kPrepThr);
      if (d->a_dtype == MOE_F32) prep_src<kF32>(p, blocks, s);
      else prep_src<kBF16>(p, blocks, s);
      g.a = p.codes;
      g.as = p.scales;
    }
    g.plist = p.plist;
    g.tiles = p.tiles;
    g.ntiles = p.ntiles;
    if (by.bm == 16) narrow<kTiles>(g, MX_FP4, d->act, static_cast<int>(by.tiles), s);
    else if (by.bm == 32) rc = tile<1, 4, 2, 2, 3, 1, true>(g, d->act, by.tiles, s);
    else if (by.bm == 64) rc = tile<1, 4, 4, 2, 3, 1, true>(g, d->act, by.tiles, s);
    else rc = tile<2, 2, 4, 4, 2, 1, true>(g, d->act, by.tiles, s);
    if (rc != MOE_OK) return api_fail(MOE_EHIP, "the product kernel's LDS size was refused");
  }
  if (topk_w) {
    const float* sums = static_cast<const float*>(g.out);
    g.out = out;
    g.out_bf16 = d->out_dtype == MOE_BF16;
    g.nblk = (d->n + 255) / 256;
    launch_kernel(k_mx_combine, dim3(static_cast<uint32_t>(g.nblk) * T), dim3(256), 0, s, g, sums);
  }
  return launched();
}

}  // extern "C"
