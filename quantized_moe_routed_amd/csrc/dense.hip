// The 16-bit products: rows grouped by expert times the expert's weight (plain, with SwiGLU, as the
// gradient of the rows), the dense product with bias, activation and residual, the two vocabulary
// passes of the cross entropy, and the products over rows that give weight gradients.  All of them
// are one tile loop (tile16.h) with another operand storage or epilogue.  Sums are fp32 in the
// matrix cores' order over the contraction; no atomics, so calls repeat bit for bit.
#include <algorithm>

#include "dense.h"
#include "device.h"
#include "launch.h"
#include "tile16.h"

namespace moe {

namespace {

__device__ __forceinline__ RowMap row_map(const RowsArg& r) {
  return RowMap{static_cast<const char*>(r.base), r.ld, r.slots, r.div, r.nrows};
}
__device__ __forceinline__ Groups groups(const GroupsArg& g) { return Groups{g.offsets, g.g2l, g.E, g.E_local, g.n_slots}; }

// ---- 16 consecutive values of an output row -----------------------------------------------------
template <int DT>
__device__ __forceinline__ void load16(const char* p, int n, float (&v)[16]) {   // n = 8 or 16 values
  if constexpr (DT == T_F32) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (4 * i < n) {
        const float4 w = reinterpret_cast<const float4*>(p)[i];
        v[4 * i] = w.x; v[4 * i + 1] = w.y; v[4 * i + 2] = w.z; v[4 * i + 3] = w.w;
      }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (8 * i < n) {
        const u32x4 w = reinterpret_cast<const u32x4*>(p)[i];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          v[8 * i + 2 * c] = El<DT>::lo(w[c]);
          v[8 * i + 2 * c + 1] = El<DT>::hi(w[c]);
        }
      }
  }
}
template <int DT>
__device__ __forceinline__ void store16(char* p, int n, const float (&v)[16]) {
  if constexpr (DT == T_F32) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (4 * i < n) reinterpret_cast<float4*>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (8 * i < n) {
        u32x4 w;
#pragma unroll
        for (int c = 0; c < 4; ++c) w[c] = El<DT>::pack(v[8 * i + 2 * c], v[8 * i + 2 * c + 1]);
        reinterpret_cast<u32x4*>(p)[i] = w;
      }
  }
}

// act(z) and act'(z).  The exact gelu z Phi(z), by erff.
__device__ __forceinline__ float fn_value(int fn, float z) {
  switch (fn) {
    case FN_RELU: return z > 0.0f ? z : (z != z ? z : 0.0f);
    case FN_SILU: return silu(z);
    case FN_GELU: return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
    default: return z;
  }
}
__device__ __forceinline__ float fn_slope(int fn, float z) {
  switch (fn) {
    case FN_RELU: return z > 0.0f ? 1.0f : 0.0f;
    case FN_SILU: {
      const float p = 1.0f / (1.0f + expf(-z));
      return p * (1.0f + z * (1.0f - p));
    }
    case FN_GELU:
      return 0.5f * (1.0f + erff(z * 0.70710678118654752f)) + z * expf(-0.5f * z * z) * 0.39894228040143268f;
    default: return 1.0f;
  }
}

// Workgroup number to tile number: workgroup i runs on XCD i mod 8, and each XCD takes a contiguous
// range of the tiles, so that tiles which share rows or weights meet in one L2.
__device__ __forceinline__ int xcd_order(int i, int total) {
  const int x = i & 7, q = total >> 3, r = total & 7;
  return x * q + min(x, r) + (i >> 3);
}

// ---- the tile loop --------------------------------------------------------------------------------
// n stages; next(i) moves the stagers to stage i's addresses and issues it into LDS buffer i & 1.
template <int DT, int FM, int FN, class FragM, class FragN, class Next>
__device__ __forceinline__ void tile_loop(int n, uint32_t bytes, const FragM& fm, const FragN& fn, f32x4 (&acc)[FM][FN],
                                          Next&& next) {
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  if (n <= 0) return;
  next(0);
  for (int it = 0; it < n; ++it) {
    wait_vmem();        // this wave's part of stage `it` has landed
    __syncthreads();    // every wave's has, and no wave reads the other buffer any more
    if (it + 1 < n) next(it + 1);
    const uint32_t buf = (it & 1) * bytes;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      u32x4 b[FN], a[FM];
#pragma unroll
      for (int j = 0; j < FN; ++j) b[j] = fn.load(buf, s, j >> 2, j & 3);
#pragma unroll
      for (int i = 0; i < FM; ++i) a[i] = fm.load(buf, s, i >> 2, i & 3);
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = El<DT>::mfma(b[j], a[i], acc[i][j]);
    }
  }
}

template <int BM, int BN, int WM, int WN>
struct Shape {
  static constexpr int WAVES = WM * WN, FM = BM / WM / 16, FN = BN / WN / 16;
  static constexpr uint32_t BYTES = (BM + BN) * kRowB;
  static_assert(FM % 4 == 0 && FN % 4 == 0, "blocks of 64");
};

constexpr int kGroupM = 8;   // row tiles taken together along the columns (they share weights in L2)

// ---- y rows = x rows times the group's weight -----------------------------------------------------
template <int DT, int BM, int BN, int WM, int WN, bool WK, int EPI>
__global__ __launch_bounds__(64 * WM * WN) void rows_kernel(const RowsProduct a, const int NT) {
  using S = Shape<BM, BN, WM, WN>;
  extern __shared__ __align__(1024) char smem[];
  const uint32_t lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)smem;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % WM, wn = wave / WM;

  Span sp;
  int mt, nt;
  {
    const Groups g = groups(a.g);
    int id, rem;
    if (g.offsets) {
      int mine;
      const int incl = group_tiles(g, lane, BM, &mine);
      const int total = __builtin_amdgcn_readlane(incl, 63) * NT;
      if ((int)blockIdx.x >= total) return;
      id = xcd_order(blockIdx.x, total);
      if (!find_tile(g, lane, BM, incl, mine, id / NT, &sp, &mt)) return;
      rem = mt * NT + id % NT;
    } else {
      sp = Span{0, 0, g.n_slots};
      rem = xcd_order(blockIdx.x, gridDim.x);
    }
    const int MT = (sp.count + BM - 1) / BM;
    const int gq = rem / (kGroupM * NT), gr = rem % (kGroupM * NT), gm = min(kGroupM, MT - gq * kGroupM);
    mt = gq * kGroupM + gr % gm;
    nt = gr / gm;
  }
  const int row0 = mt * BM, K = a.K, N = a.N;
  const RowMap xm = row_map(a.x);

  StageK<BM, S::WAVES> sa;
  const int last = sp.count - 1;
  sa.init(lane, wave, (K + 7) & ~7, [&](int r) { return xm.read(sp.first + min(row0 + r, last)); });
  typename StageK<BM, S::WAVES>::Frag fa;
  fa.init(lds, wm * (BM / WM), lane);

  const char* w = static_cast<const char*>(a.w) + (int64_t)sp.local * (WK ? N : K) * a.w_ld;
  const char* w2 = a.w2 ? static_cast<const char*>(a.w2) + (int64_t)sp.local * (WK ? N : K) * a.w_ld : nullptr;
  f32x4 acc[S::FM][S::FN];
  const int n1 = (K + kStageK - 1) / kStageK;

  if constexpr (WK) {
    StageK<BN, S::WAVES> sb;
    sb.init(lane, wave, (K + 7) & ~7, [&](int r) {
      if constexpr (EPI == EPI_SWIGLU) {
        // a block of 64 tile rows is 32 columns of gate (fragments 0, 1) and of up (2, 3): a lane's 16
        // values are then gate and up of the same 8 columns
        const int c = nt * (BN / 2) + (r >> 6) * 32 + 8 * ((r >> 4) & 3) + 4 * ((r >> 2) & 1) + (r & 3);
        return ((r >> 3) & 1 ? w2 : w) + (int64_t)min(c, N - 1) * a.w_ld;
      } else {
        return w + (int64_t)min(nt * BN + r, N - 1) * a.w_ld;
      }
    });
    typename StageK<BN, S::WAVES>::Frag fb;
    fb.init(lds + StageK<BM, S::WAVES>::BYTES, wn * (BN / WN), lane);
    tile_loop<DT, S::FM, S::FN>(n1, S::BYTES, fa, fb, acc, [&](int i) {
      const uint32_t at = lds + (i & 1) * S::BYTES;
      sa.issue(at, i * kStageK, lane, wave);
      sb.issue(at + StageK<BM, S::WAVES>::BYTES, i * kStageK, lane, wave);
      sa.advance(kRowB);
      sb.advance(kRowB);
    });
  } else {
    StageM<BN, S::WAVES> sb;
    sb.init(lane, wave, RowMap{w, a.w_ld, nullptr, 1, K}, 0, K, nt * BN, N);
    typename StageM<BN, S::WAVES>::Frag fb;
    fb.init(lds + StageK<BM, S::WAVES>::BYTES, wn * (BN / WN), lane);
    const int64_t seg = a.x2 ? static_cast<const char*>(a.x2) - static_cast<const char*>(a.x.base) : 0;
    tile_loop<DT, S::FM, S::FN>(a.x2 ? 2 * n1 : n1, S::BYTES, fa, fb, acc, [&](int i) {
      const uint32_t at = lds + (i & 1) * S::BYTES;
      if (i == n1) {   // the second product's contraction follows the first's
        sa.advance(seg - (int64_t)n1 * kRowB);
        sb.map.base = w2;
      }
      const int k0 = (i < n1 ? i : i - n1) * kStageK;
      sa.issue(at, k0, lane, wave);
      sb.issue(at + StageK<BM, S::WAVES>::BYTES, k0, lane, wave);
      sa.advance(kRowB);
    });
  }

  // ---- epilogue: a lane holds, of row m, 16 consecutive columns of every block of 64 ----
  const int r = lane & 15, q = lane >> 4;
  const float scale = EPI == EPI_STORE && a.scale ? *a.scale : 1.0f;
  float ce_scale = 1.0f;
  if constexpr (EPI == EPI_CE_GRAD) ce_scale = *a.ds_scale;
  if constexpr (EPI == EPI_CE_SUM) __syncthreads();   // the stages' LDS is free for the row sums
#pragma unroll
  for (int i = 0; i < S::FM; ++i) {
    const int ml = wm * (BM / WM) + (i >> 2) * 64 + 16 * (r >> 2) + 4 * (i & 3) + (r & 3);
    const int mr = row0 + ml;                 // row of the group
    const bool live = mr < sp.count;
    const int p = sp.first + (live ? mr : 0);
    if constexpr (EPI == EPI_CE_SUM) {
      // the row's maximum and sum over the tile's columns: 16 values a block here, the other three
      // lanes of the row by lane exchange, the other waves through LDS
      const int tgt = a.target[p];
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < S::FN; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int n = nt * BN + wn * (BN / WN) + (j >> 2) * 64 + 16 * q + 4 * (j & 3) + c;
          if (n < N) {
            mx = fmaxf(mx, acc[i][j][c]);
            if (live && n == tgt) a.hit[p] = acc[i][j][c];
          }
        }
      mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
      mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
      const float top = mx == INFINITY || mx == -INFINITY ? 0.0f : mx;
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < S::FN; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int n = nt * BN + wn * (BN / WN) + (j >> 2) * 64 + 16 * q + 4 * (j & 3) + c;
          if (n < N) sum += __expf(acc[i][j][c] - top);
        }
      sum += __shfl_xor(sum, 16, 64);
      sum += __shfl_xor(sum, 32, 64);
      if (q == 0) reinterpret_cast<float2*>(smem)[wn * BM + ml] = make_float2(mx == -INFINITY ? mx : top, sum);
      continue;
    }
    if (!live) continue;
#pragma unroll
    for (int b = 0; b < S::FN / 4; ++b) {
      float v[16];
#pragma unroll
      for (int c = 0; c < 16; ++c) v[c] = acc[i][b * 4 + (c >> 2)][c & 3];
      if constexpr (EPI == EPI_SWIGLU) {
        const int n = nt * (BN / 2) + (wn * (BN / WN) + b * 64) / 2 + 8 * q;
        if (n >= N) continue;
        float h[16];
#pragma unroll
        for (int c = 0; c < 8; ++c) h[c] = silu(v[c]) * v[8 + c];
        if (char* o = row_map(a.y).write(p)) store16<DT>(o + 2 * (int64_t)n, 8, h);
        if (a.keep_g.base) store16<DT>(row_map(a.keep_g).write(p) + 2 * (int64_t)n, 8, v);
        if (a.keep_u.base) {
#pragma unroll
          for (int c = 0; c < 8; ++c) h[c] = v[8 + c];
          store16<DT>(row_map(a.keep_u).write(p) + 2 * (int64_t)n, 8, h);
        }
        continue;
      }
      const int n = nt * BN + wn * (BN / WN) + b * 64 + 16 * q;
      if constexpr (EPI == EPI_CE_GRAD) {
        // ds = (exp(z - lse) - [target]) dnll, scaled; columns up to the next multiple of 8 are zeros
        const int cnt = min(16, ((N + 7) & ~7) - n);
        if (cnt <= 0) continue;
        const int t = xm.row(p), tgt = a.target[t];
        const float up = a.dnll[t] * ce_scale, l = a.lse[t];
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float pr = __expf(v[c] - l) - (a.v0 + n + c == tgt ? 1.0f : 0.0f);
          v[c] = n + c < N ? pr * up : 0.0f;
        }
        store16<DT>(row_map(a.y).write(p) + 2 * (int64_t)n, cnt, v);
        continue;
      }
      const int cnt = min(16, N - n);
      if (cnt <= 0) continue;
      if constexpr (EPI == EPI_LINEAR) {
        if (a.bias) {
          float w16[16];
          load16<T_F32>(reinterpret_cast<const char*>(a.bias + n), cnt, w16);
#pragma unroll
          for (int c = 0; c < 16; ++c) v[c] += w16[c];
        }
        if (a.pre.base) store16<DT>(row_map(a.pre).write(p) + 2 * (int64_t)n, cnt, v);
        if (a.fn != FN_NONE) {
#pragma unroll
          for (int c = 0; c < 16; ++c) v[c] = fn_value(a.fn, v[c]);
        }
        if (a.res.base) {
          float w16[16];
          load16<DT>(row_map(a.res).write(p) + 2 * (int64_t)n, cnt, w16);
#pragma unroll
          for (int c = 0; c < 16; ++c) v[c] += w16[c];
        }
      } else {
#pragma unroll
        for (int c = 0; c < 16; ++c) v[c] *= scale;
        if (a.add) {
          float w16[16];
          load16<T_F32>(reinterpret_cast<const char*>(a.add + (int64_t)p * N + n), cnt, w16);
#pragma unroll
          for (int c = 0; c < 16; ++c) v[c] += w16[c];
        }
      }
      if (char* o = row_map(a.y).write(p)) {
        if (a.y.dt == T_F32) store16<T_F32>(o + 4 * (int64_t)n, cnt, v);
        else store16<DT>(o + 2 * (int64_t)n, cnt, v);
      }
    }
  }
  if constexpr (EPI == EPI_CE_SUM) {
    __syncthreads();
    for (int ml = threadIdx.x; ml < BM; ml += 64 * S::WAVES) {
      if (row0 + ml >= sp.count) continue;
      float mx = -INFINITY;
#pragma unroll
      for (int k = 0; k < WN; ++k) mx = fmaxf(mx, reinterpret_cast<const float2*>(smem)[k * BM + ml].x);
      float sum = 0.0f;
      if (mx != -INFINITY) {
#pragma unroll
        for (int k = 0; k < WN; ++k) {
          const float2 w16 = reinterpret_cast<const float2*>(smem)[k * BM + ml];
          sum += w16.y * __expf(w16.x - mx);
        }
      }
      a.part[(int64_t)nt * a.g.n_slots + row0 + ml] = make_float2(mx, sum);
    }
  }
}

// ---- w[e] = sum over the group's rows of a[p]^T b[p] ------------------------------------------------
template <int DT, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void cols_kernel(const ColsProduct a, const int MT, const int NT) {
  using S = Shape<BM, BN, WM, WN>;
  extern __shared__ __align__(1024) char smem[];
  const uint32_t lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)smem;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % WM, wn = wave / WM;
  const int id = xcd_order(blockIdx.x, gridDim.x);
  const int local = id / (MT * NT), rem = id % (MT * NT);
  const int gq = rem / (kGroupM * NT), gr = rem % (kGroupM * NT), gm = min(kGroupM, MT - gq * kGroupM);
  const int mt = gq * kGroupM + gr % gm, nt = gr / gm;
  Span sp{local, 0, a.g.n_slots};
  if (a.g.offsets) {
    const Groups g = groups(a.g);
    int e = local;
    if (g.g2l) {   // the global expert of local id `local` (none: no rows)
      e = -1;
      for (int e0 = 0; e0 < g.E; e0 += 64) {
        const uint64_t hit = __ballot(e0 + lane < g.E && g.g2l[min(e0 + lane, g.E - 1)] == local);
        if (hit) {
          e = e0 + __builtin_ctzll(hit);
          break;
        }
      }
    }
    sp = e < 0 || e >= g.E ? Span{local, 0, 0} : span_of(g, e);
  }

  using SA = StageM<BM, S::WAVES>;
  using SB = StageM<BN, S::WAVES>;
  SA sa;
  SB sb;
  sa.init(lane, wave, row_map(a.a), sp.first, sp.count, mt * BM, (a.M + 7) & ~7);
  sb.init(lane, wave, row_map(a.b), sp.first, sp.count, nt * BN, a.N);
  typename SA::Frag fa;
  typename SB::Frag fb;
  fa.init(lds, wm * (BM / WM), lane);
  fb.init(lds + SA::BYTES, wn * (BN / WN), lane);
  f32x4 acc[S::FM][S::FN];
  sa.fetch(0, lane, wave);
  sb.fetch(0, lane, wave);
  tile_loop<DT, S::FM, S::FN>((sp.count + kStageK - 1) / kStageK, S::BYTES, fa, fb, acc, [&](int i) {
    const uint32_t at = lds + (i & 1) * S::BYTES;
    sa.issue(at, i * kStageK, lane, wave);
    sb.issue(at + SA::BYTES, i * kStageK, lane, wave);
    sa.fetch((i + 1) * kStageK, lane, wave);   // the next stage's rows arrive during this one's products
    sb.fetch((i + 1) * kStageK, lane, wave);
  });

  const int r = lane & 15, q = lane >> 4;
  const float scale = a.scale ? *a.scale : 1.0f;
#pragma unroll
  for (int i = 0; i < S::FM; ++i) {
    const int m = mt * BM + wm * (BM / WM) + (i >> 2) * 64 + 16 * (r >> 2) + 4 * (i & 3) + (r & 3);
    if (m >= a.M) continue;
#pragma unroll
    for (int b = 0; b < S::FN / 4; ++b) {
      const int n = nt * BN + wn * (BN / WN) + b * 64 + 16 * q, cnt = min(16, a.N - n);
      if (cnt <= 0) continue;
      float v[16];
#pragma unroll
      for (int c = 0; c < 16; ++c) v[c] = acc[i][b * 4 + (c >> 2)][c & 3] * scale;
      char* o = static_cast<char*>(a.w) + (((int64_t)local * a.M + m) * a.N + n) * (a.w_dt == T_F32 ? 4 : 2);
      if (a.accumulate) {
        float w16[16] = {};
        if (a.w_dt == T_F32) load16<T_F32>(o, cnt, w16);
        else load16<DT>(o, cnt, w16);
#pragma unroll
        for (int c = 0; c < 16; ++c) v[c] += w16[c];
      }
      if (a.w_dt == T_F32) store16<T_F32>(o, cnt, v);
      else store16<DT>(o, cnt, v);
    }
  }
}

template <class Kern>
hipError_t lds_limit(Kern k, uint32_t bytes) {
  return hipFuncSetAttribute(reinterpret_cast<const void*>(k), hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <int DT, int BM, int BN, int WM, int WN, bool WK, int EPI>
hipError_t go_rows(const RowsProduct& a, hipStream_t s) {
  using S = Shape<BM, BN, WM, WN>;
  const int cols = EPI == EPI_SWIGLU ? BN / 2 : BN;
  const int NT = (a.N + cols - 1) / cols;
  // row tiles: every group may end inside a tile
  int64_t mt = (a.g.n_slots + BM - 1) / BM;
  if (a.g.offsets) mt = (a.g.n_slots + BM - 1) / BM + std::min(a.g.E_local, a.g.n_slots);
  auto k = rows_kernel<DT, BM, BN, WM, WN, WK, EPI>;
  if (hipError_t e = lds_limit(k, 2 * S::BYTES)) return e;
  hipLaunchKernelGGL(k, dim3((uint32_t)(mt * NT)), dim3(64 * S::WAVES), 2 * S::BYTES, s, a, NT);
  return hipGetLastError();
}

template <int DT>
hipError_t rows_dt(const RowsProduct& a, hipStream_t s) {
  if (!a.w_k) return go_rows<DT, 128, 128, 2, 2, false, EPI_STORE>(a, s);
  switch (a.epi) {
    case EPI_SWIGLU: return go_rows<DT, 128, 128, 2, 2, true, EPI_SWIGLU>(a, s);
    case EPI_LINEAR: return go_rows<DT, 128, 128, 2, 2, true, EPI_LINEAR>(a, s);
    case EPI_CE_SUM: return go_rows<DT, 128, 128, 2, 2, true, EPI_CE_SUM>(a, s);
    case EPI_CE_GRAD: return go_rows<DT, 128, 128, 2, 2, true, EPI_CE_GRAD>(a, s);
    default: return go_rows<DT, 128, 128, 2, 2, true, EPI_STORE>(a, s);
  }
}

template <int DT>
hipError_t cols_dt(const ColsProduct& a, hipStream_t s) {
  constexpr int BM = 128, BN = 128;
  using S = Shape<BM, BN, 2, 2>;
  const int MT = (a.M + BM - 1) / BM, NT = (a.N + BN - 1) / BN;
  const int E = a.g.offsets ? a.g.E_local : 1;
  auto k = cols_kernel<DT, BM, BN, 2, 2>;
  if (hipError_t e = lds_limit(k, 2 * S::BYTES)) return e;
  hipLaunchKernelGGL(k, dim3((uint32_t)((int64_t)E * MT * NT)), dim3(64 * S::WAVES), 2 * S::BYTES, s, a, MT, NT);
  return hipGetLastError();
}

// ---- elementwise -----------------------------------------------------------------------------------
template <int DT>
__global__ __launch_bounds__(256) void swiglu_grad_kernel(const RowsArg dh, const RowsArg g, const RowsArg u, int R,
                                                          int I, uint16_t* __restrict__ dg, uint16_t* __restrict__ du) {
  const int p = blockIdx.y + blockIdx.z * gridDim.y, c = (blockIdx.x * 256 + threadIdx.x) * 8;
  if (p >= R || c >= I) return;
  float d[16], gv[16], uv[16];
  load16<DT>(row_map(dh).read(p) + 2 * c, 8, d);
  load16<DT>(row_map(g).read(p) + 2 * c, 8, gv);
  load16<DT>(row_map(u).read(p) + 2 * c, 8, uv);
  float a[16], b[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float sg = 1.0f / (1.0f + expf(-gv[i]));
    a[i] = d[i] * uv[i] * (sg * (1.0f + gv[i] * (1.0f - sg)));
    b[i] = d[i] * (gv[i] * sg);
  }
  store16<DT>(reinterpret_cast<char*>(dg + (int64_t)p * I + c), 8, a);
  store16<DT>(reinterpret_cast<char*>(du + (int64_t)p * I + c), 8, b);
}

// dz = dy act'(pre) for kBiasRows rows and 8 columns a thread, with the columns' sums over the rows
// (fp32, of the unrounded values)
template <int DT>
__global__ __launch_bounds__(64) void linear_dz_kernel(const RowsArg dy, const RowsArg pre, int fn, int T, int N,
                                                       uint16_t* __restrict__ dz, float* __restrict__ part) {
  const int c = (blockIdx.x * 64 + threadIdx.x) * 8;
  if (c >= N) return;
  const int t0 = blockIdx.y * kBiasRows, t1 = min(T, t0 + kBiasRows);
  float sum[16] = {};
  for (int t = t0; t < t1; ++t) {
    float d[16], z[16];
    load16<DT>(row_map(dy).read(t) + 2 * c, 8, d);
    if (fn != FN_NONE) {
      load16<DT>(row_map(pre).read(t) + 2 * c, 8, z);
#pragma unroll
      for (int i = 0; i < 8; ++i) d[i] *= fn_slope(fn, z[i]);
    }
    if (dz) store16<DT>(reinterpret_cast<char*>(dz + (int64_t)t * N + c), 8, d);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] += d[i];
  }
  if (part) store16<T_F32>(reinterpret_cast<char*>(part + (int64_t)blockIdx.y * N + c), 8, sum);
}

__global__ __launch_bounds__(256) void bias_sum_kernel(const float* __restrict__ part, int chunks, int N,
                                                       float* __restrict__ dbias, bool accumulate) {
  const int n = blockIdx.x * 256 + threadIdx.x;
  if (n >= N) return;
  float s = 0.0f;
  for (int c = 0; c < chunks; ++c) s += part[(int64_t)c * N + n];
  dbias[n] = accumulate ? dbias[n] + s : s;
}

// One wave a row: the partial sums brought to the largest maximum.
__global__ __launch_bounds__(256) void ce_finish_kernel(const float2* __restrict__ part, int tiles,
                                                        const float* __restrict__ hit, const int32_t* __restrict__ target,
                                                        int T, int V, float* __restrict__ nll, float* __restrict__ lse) {
  const int t = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (t >= T) return;
  float mx = -INFINITY;
  for (int i = lane; i < tiles; i += 64) mx = fmaxf(mx, part[(int64_t)i * T + t].x);
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) mx = fmaxf(mx, __shfl_xor(mx, m, 64));
  float sum = 0.0f;
  if (mx != -INFINITY)
    for (int i = lane; i < tiles; i += 64) {
      const float2 v = part[(int64_t)i * T + t];
      sum += v.y * expf(v.x - mx);
    }
  sum = wave_sum(sum);
  if (lane == 0) {
    const float l = mx == -INFINITY ? mx : mx + logf(sum);
    lse[t] = l;
    nll[t] = (unsigned)target[t] < (unsigned)V ? l - hit[t] : 0.0f;
  }
}

// The counted tokens in order (one workgroup: 1024 tokens at a time, placed by ballots and a sum
// over the waves), and the power of two that brings their largest |dnll| to [2^14, 2^15) with its
// inverse (1 where there is none, or it is not finite: the gradients then are not either).
__global__ __launch_bounds__(1024) void ce_plan_kernel(const float* __restrict__ dnll, const int32_t* __restrict__ target,
                                                       int T, int V, int32_t* __restrict__ keep,
                                                       int32_t* __restrict__ offsets, float* __restrict__ scale) {
  __shared__ float top[16];
  __shared__ int cnt[16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float mx = 0.0f;
  int base = 0;
  for (int t0 = 0; t0 < T; t0 += 1024) {
    const int t = t0 + threadIdx.x;
    const bool in = t < T && (unsigned)target[t] < (unsigned)V;
    if (in) mx = fmaxf(mx, fabsf(dnll[t]));
    const uint64_t b = __ballot(in);
    if (lane == 0) cnt[wave] = __popcll(b);
    __syncthreads();
    int at = base, all = 0;
    for (int i = 0; i < 16; ++i) {
      if (i < wave) at += cnt[i];
      all += cnt[i];
    }
    if (in) keep[at + __popcll(b & lanemask_lt())] = t;
    base += all;
    __syncthreads();
  }
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) mx = fmaxf(mx, __shfl_xor(mx, m, 64));
  if (lane == 0) top[wave] = mx;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 0; i < 16; ++i) mx = fmaxf(mx, top[i]);
    int a = 0;
    if (mx > 0.0f && mx < INFINITY) {
      (void)frexpf(mx, &a);
      a = max(-111, min(15 - a, 125));   // both powers stay normal numbers
    }
    scale[0] = ldexpf(1.0f, a);
    scale[1] = ldexpf(1.0f, -a);
    offsets[0] = 0;
    offsets[1] = base;
  }
}

// Rows of dx of ignored tokens: zeros, 16 bytes a thread.
__global__ __launch_bounds__(256) void ce_zero_kernel(const int32_t* __restrict__ target, int V, const RowsArg dx,
                                                      int chunks) {
  const int t = blockIdx.x;
  if ((unsigned)target[t] < (unsigned)V) return;
  u32x4* o = reinterpret_cast<u32x4*>(static_cast<char*>(dx.base) + (int64_t)t * dx.ld);
  for (int c = threadIdx.x; c < chunks; c += 256) o[c] = u32x4{0, 0, 0, 0};
}

__global__ __launch_bounds__(256) void zero16_kernel(u32x4* __restrict__ p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) p[i] = u32x4{0, 0, 0, 0};
}

}  // namespace

hipError_t launch_zero16(void* p, int64_t n, hipStream_t s) {
  hipLaunchKernelGGL(zero16_kernel, dim3((uint32_t)std::min<int64_t>((n + 255) / 256, 4096)), dim3(256), 0, s,
                     static_cast<u32x4*>(p), n);
  return hipGetLastError();
}

int ce_tile_cols(int T) {
  (void)T;
  return 128;
}

hipError_t launch_rows_product(const RowsProduct& a, hipStream_t s) {
  trace_pre("rows_product", s);
  const hipError_t e = a.dt == T_BF16 ? rows_dt<T_BF16>(a, s) : rows_dt<T_F16>(a, s);
  trace_post("rows_product", s);
  return e;
}

hipError_t launch_cols_product(const ColsProduct& a, hipStream_t s) {
  trace_pre("cols_product", s);
  const hipError_t e = a.dt == T_BF16 ? cols_dt<T_BF16>(a, s) : cols_dt<T_F16>(a, s);
  trace_post("cols_product", s);
  return e;
}

hipError_t launch_swiglu_grad(int dt, const RowsArg& dh, const RowsArg& g, const RowsArg& u, int R, int I, void* dg,
                              void* du, hipStream_t s) {
  const int gy = std::min(R, 65535);
  const dim3 grid((I / 8 + 255) / 256, gy, (R + gy - 1) / gy);
  if (dt == T_BF16)
    hipLaunchKernelGGL(swiglu_grad_kernel<T_BF16>, grid, dim3(256), 0, s, dh, g, u, R, I, (uint16_t*)dg, (uint16_t*)du);
  else
    hipLaunchKernelGGL(swiglu_grad_kernel<T_F16>, grid, dim3(256), 0, s, dh, g, u, R, I, (uint16_t*)dg, (uint16_t*)du);
  return hipGetLastError();
}

hipError_t launch_linear_dz(int dt, const RowsArg& dy, const RowsArg& pre, int fn, int T, int N, void* dz, float* part,
                            float* dbias, bool accumulate, hipStream_t s) {
  const int chunks = (T + kBiasRows - 1) / kBiasRows;
  const dim3 grid((N / 8 + 63) / 64, chunks);
  if (dt == T_BF16)
    hipLaunchKernelGGL(linear_dz_kernel<T_BF16>, grid, dim3(64), 0, s, dy, pre, fn, T, N, (uint16_t*)dz, part);
  else
    hipLaunchKernelGGL(linear_dz_kernel<T_F16>, grid, dim3(64), 0, s, dy, pre, fn, T, N, (uint16_t*)dz, part);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !dbias) return e;
  hipLaunchKernelGGL(bias_sum_kernel, dim3((N + 255) / 256), dim3(256), 0, s, part, chunks, N, dbias, accumulate);
  return hipGetLastError();
}

hipError_t launch_ce_finish(const float2* part, int tiles, const float* hit, const int32_t* target, int T, int V,
                            float* nll, float* lse, hipStream_t s) {
  hipLaunchKernelGGL(ce_finish_kernel, dim3((T + 3) / 4), dim3(256), 0, s, part, tiles, hit, target, T, V, nll, lse);
  return hipGetLastError();
}

hipError_t launch_ce_plan(const float* dnll, const int32_t* target, int T, int V, int32_t* keep, int32_t* offsets,
                          float* scale, const RowsArg& dx, int H, hipStream_t s) {
  hipLaunchKernelGGL(ce_plan_kernel, dim3(1), dim3(1024), 0, s, dnll, target, T, V, keep, offsets, scale);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !dx.base) return e;
  hipLaunchKernelGGL(ce_zero_kernel, dim3(T), dim3(256), 0, s, target, V, dx, H / (dx.dt == T_F32 ? 4 : 8));
  return hipGetLastError();
}

}  // namespace moe
