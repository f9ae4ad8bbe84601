// The 16-bit matrix-core tile (gfx950): BM x BN outputs of one workgroup, fp32 sums, operands of
// bf16 or fp16 staged through LDS 64 contraction values at a time.
//
// Operands come in two storages: "K" holds the contraction axis contiguous (rows x 64 values a
// stage), "M" holds the output axis contiguous (64 contraction rows x COLS values a stage; its
// fragments are turned by the LDS transpose read).  Both fill LDS by direct global-to-LDS loads of
// 16 bytes a lane; LDS is written lane after lane, so the bank swizzle is applied to the global
// address.  With D = sum_k N[n,k] M[m,k] each v_mfma_f32_16x16x32 takes the n side as its first
// operand: a lane then holds consecutive n of one m.  Fragment f (0..3) of a block of 64 rows
// takes rows 16*(r/4) + 4*f + r%4 (r = lane % 16), so that over a block's four fragments a lane
// owns 16 consecutive n: whole 128-byte lines for four lanes of a 16-bit row.
#pragma once
#include "device.h"
#include "ffn.h"

namespace moe {

enum : int { T_F32 = 0, T_BF16 = 1, T_F16 = 2 };

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// LDS by byte offset (the direct loads take offsets, and so do the fragment reads)
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// Element type DT (T_BF16 or T_F16).
template <int DT>
struct El {
  static __device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    if constexpr (DT == T_BF16)
      return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
      return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
  // nearest even, the one rounding of a finished sum
  static __device__ __forceinline__ uint32_t bits(float v) {
    if constexpr (DT == T_BF16) return __builtin_bit_cast(uint16_t, (__bf16)v);
    else return __builtin_bit_cast(uint16_t, (_Float16)v);
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) { return bits(lo) | (bits(hi) << 16); }
  static __device__ __forceinline__ float lo(uint32_t w) {
    if constexpr (DT == T_BF16) return bf16_bits_to_float(w & 0xFFFFu);
    else return half_bits_to_float(w & 0xFFFFu);
  }
  static __device__ __forceinline__ float hi(uint32_t w) {
    if constexpr (DT == T_BF16) return __uint_as_float(w & 0xFFFF0000u);
    else return half_bits_to_float(w >> 16);
  }
};

// 16 zero bytes: what a lane loads in place of contraction values past the end (the other operand
// gets zeros there as well, so an infinity or NaN beyond the end never enters a sum).
__device__ const uint4 kZero16 = {0, 0, 0, 0};

constexpr int kStageK = 64;                 // contraction values a stage
constexpr int kRowB = kStageK * 2;          // bytes of an LDS row of a "K" operand

// LDS chunk swizzles (16-byte chunks).  "K" rows are 128 bytes: the 16 rows 16*(r/4)+4f+r%4 of a
// fragment differ in bits 0, 1, 4 and 5; bit 0 selects the half of the 256-byte bank line, the
// others pick one of 8 chunks, so the 16 lanes of a fragment column touch 16 distinct bank groups.
__device__ __forceinline__ int swz_k(int row) { return ((row >> 1) & 1) | (((row >> 4) & 3) << 1); }
// "M" rows are whole bank lines: a transpose read takes 4 contraction rows x 4 segments of 32
// bytes apart; the row's low bits go to chunk bits 0 and 3, which the segments leave free.
__device__ __forceinline__ int swz_m(int k) { return (k & 1) | ((k & 2) << 2); }

// A tensor whose rows are addressed by grouped position p: its row is p, or the slot slots[p], or
// the slot's token slots[p] / div.  Read rows are clamped into the tensor, written ones checked.
struct RowMap {
  const char* base;
  int64_t ld;               // bytes
  const int32_t* slots;     // NULL: position p is row p
  int div;
  int nrows;
  __device__ __forceinline__ int row(int p) const {
    if (!slots) return p;
    const int s = slots[p];
    return div == 1 ? s : (s < 0 ? -1 : (int)((unsigned)s / (unsigned)div));
  }
  __device__ __forceinline__ const char* read(int p) const {
    return base + (int64_t)max(0, min(row(p), nrows - 1)) * ld;
  }
  __device__ __forceinline__ char* write(int p) const {   // NULL: not a row of the tensor
    const int r = row(p);
    return (unsigned)r < (unsigned)nrows ? const_cast<char*>(base) + (int64_t)r * ld : nullptr;
  }
};

// Stage of a "K" operand: ROWS rows x 64 contraction values.
template <int ROWS, int WAVES>
struct StageK {
  static constexpr int NI = ROWS * kRowB / 1024 / WAVES;   // direct loads of a wave
  static constexpr int BYTES = ROWS * kRowB;
  static_assert(NI >= 1, "rows per wave");
  const char* p[NI];
  int K;

  // rowptr(r): address of tile row r's contraction value 0 (valid for every r in 0..ROWS-1)
  template <class F>
  __device__ __forceinline__ void init(int lane, int wave, int K_, F&& rowptr) {
    K = K_;
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const int r = (wave * NI + j) * 8 + (lane >> 3);
      p[j] = rowptr(r) + (((lane & 7) ^ swz_k(r)) << 4);
    }
  }
  __device__ __forceinline__ void advance(int64_t bytes) {
#pragma unroll
    for (int j = 0; j < NI; ++j) p[j] += bytes;
  }
  // stage k0..k0+63 (the pointers stand at k0) into LDS byte offset `lds`
  __device__ __forceinline__ void issue(uint32_t lds, int k0, int lane, int wave) const {
    const bool tail = k0 + kStageK > K;
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const char* q = p[j];
      if (tail) {
        const int r = (wave * NI + j) * 8 + (lane >> 3);
        if (k0 + (((lane & 7) ^ swz_k(r)) << 3) >= K) q = reinterpret_cast<const char*>(&kZero16);
      }
      dma16(q, lds + (uint32_t)((wave * NI + j) * 1024));
    }
  }
  // fragment addresses: the lane's base for rows at `row0` (a multiple of 64); + 512 f + 8192 block
  struct Frag {
    uint32_t a[2];
    __device__ __forceinline__ void init(uint32_t lds, int row0, int lane) {
      const int r = lane & 15, q = lane >> 4;
      const int row = row0 + 16 * (r >> 2) + (r & 3);
#pragma unroll
      for (int s = 0; s < 2; ++s) a[s] = lds + row * kRowB + (((4 * s + q) ^ swz_k(row)) << 4);
    }
    __device__ __forceinline__ u32x4 load(uint32_t buf, int s, int blk, int f) const {
      return *(const lds_u32x4*)(a[s] + buf + blk * 64 * kRowB + f * 4 * kRowB);
    }
  };
};

// Stage of an "M" operand: 64 contraction rows x COLS values.
template <int COLS, int WAVES>
struct StageM {
  static constexpr int LPR = COLS / 8;                   // lanes a row
  static constexpr int RPI = 64 / LPR;                   // rows a load
  static constexpr int NI = kStageK / RPI / WAVES;
  static constexpr int BYTES = COLS * kRowB;
  static_assert(NI >= 1 && COLS >= 128, "columns per wave");
  RowMap map;
  int first, count;       // contraction rows are positions first..first+count-1
  int col[2];             // byte offset of the lane's chunk for even and odd loads
  int idx[NI];            // next stage's rows (indexed maps)

  __device__ __forceinline__ int kr(int j, int lane, int wave) const { return (wave * NI + j) * RPI + lane / LPR; }
  // col0: first column of the tile, ncols: columns of the tensor (a multiple of 8; chunks past it
  // read column 0 instead: those outputs are not stored)
  __device__ __forceinline__ void init(int lane, int wave, const RowMap& m, int first_, int count_, int col0, int ncols) {
    map = m;
    first = first_;
    count = count_;
#pragma unroll
    for (int o = 0; o < 2; ++o) {
      const int c = col0 + ((((lane % LPR) ^ swz_m(o * RPI + lane / LPR))) << 3);
      col[o] = c < ncols ? c * 2 : 0;
    }
  }
  __device__ __forceinline__ void fetch(int k0, int lane, int wave) {
    if (!map.slots) return;
#pragma unroll
    for (int j = 0; j < NI; ++j) idx[j] = k0 + kr(j, lane, wave) < count ? map.row(first + k0 + kr(j, lane, wave)) : 0;
  }
  __device__ __forceinline__ void issue(uint32_t lds, int k0, int lane, int wave) const {
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const int k = k0 + kr(j, lane, wave);
      const int row = map.slots ? max(0, min(idx[j], map.nrows - 1)) : first + k;
      // (kr mod 4 is the lane's row plus RPI for odd loads; wave * NI * RPI is a multiple of 4 when
      // NI is even, and RPI = 4 leaves the row alone)
      const char* q = map.base + (int64_t)row * map.ld + col[RPI == 4 ? 0 : (j & 1)];
      if (k >= count) q = reinterpret_cast<const char*>(&kZero16);
      dma16(q, lds + (uint32_t)((wave * NI + j) * 1024));
    }
  }
  struct Frag {
    uint32_t a[2][2];   // [f / 2][block parity]
    __device__ __forceinline__ void init(uint32_t lds, int row0, int lane) {
      const int j = lane & 15, q = lane >> 4, k = 8 * q + (j >> 2);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int b = 0; b < 2; ++b)
          a[h][b] = lds + k * (COLS * 2) + (((row0 / 8 + 8 * b + 2 * (j & 3) + h) ^ swz_m(k)) << 4);
    }
    __device__ __forceinline__ u32x4 load(uint32_t buf, int s, int blk, int f) const {
      const uint32_t p = a[f >> 1][blk & 1] + buf + (blk >> 1) * 256 + (f & 1) * 8 + s * 32 * COLS * 2;
      const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
      const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * COLS * 2));
      return __builtin_bit_cast(u32x4, (s16x8)__builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  };
};

// ---- ragged groups ------------------------------------------------------------------------------

// Rows grouped by expert: positions offsets[e]..offsets[e+1]-1 of expert e (clamped into
// 0..n_slots, so bad offsets never leave the tensors); g2l as in moe_expert_forward.  offsets NULL:
// one group of n_slots rows (a dense product).
struct Groups {
  const int32_t* offsets;
  const int32_t* g2l;
  int E, E_local, n_slots;
};

struct Span {
  int local, first, count;   // local expert, first position, rows
};

__device__ __forceinline__ Span span_of(const Groups& g, int e) {
  const int a = max(0, min(g.offsets[e], g.n_slots)), b = max(a, min(g.offsets[e + 1], g.n_slots));
  const int l = g.g2l ? g.g2l[e] : e;
  return Span{l, a, (unsigned)l < (unsigned)g.E_local ? b - a : 0};
}

// The group and row tile of row tile number t, numbered group by group (ceil(rows / BM) tiles
// each), and the number of tiles of all groups.  Every wave finds it by itself: a lane counts the
// tiles of ceil(E / 64) experts, a wave scan places them (inclusive count returned, the lane's own in *mine).
__device__ __forceinline__ int group_tiles(const Groups& g, int lane, int BM, int* mine) {
  const int per = (g.E + kWave - 1) / kWave;
  int n = 0;
  for (int i = 0; i < per; ++i) {
    const int e = lane * per + i;
    if (e < g.E) n += (span_of(g, e).count + BM - 1) / BM;
  }
  *mine = n;
  int sum = n;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const int v = __shfl_up(sum, d, kWave);
    if (lane >= d) sum += v;
  }
  return sum;   // inclusive
}

// The span and row tile of tile t; false past the last one.
__device__ __forceinline__ bool find_tile(const Groups& g, int lane, int BM, int incl, int mine, int t, Span* sp, int* mt) {
  const uint64_t past = __ballot(incl > t);
  if (!past) return false;
  const int src = __builtin_ctzll(past);
  int left = t - __builtin_amdgcn_readlane(incl - mine, src);
  const int per = (g.E + kWave - 1) / kWave;
  for (int i = 0; i < per; ++i) {
    const int e = src * per + i;
    if (e >= g.E) break;
    const Span s = span_of(g, e);
    const int n = (s.count + BM - 1) / BM;
    if (left < n) {
      *sp = s;
      *mt = left;
      return true;
    }
    left -= n;
  }
  return false;
}

}  // namespace moe
