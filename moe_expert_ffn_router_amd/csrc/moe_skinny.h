// Products of a few rows of x with a few rows of w over a long K, on the matrix
// cores: acc[nt][mt] = w rows (16 nt ..) . x rows (16 mt ..), for the router
// projection and the adapters' first factor.
//
// K is split over the waves of a workgroup, in chunks of 64: no two waves read
// the same bytes, each runs its own pipeline without barriers, and the waves'
// sums are added once at the end. A wave loads the D next chunks of its rows
// into registers, 16 bytes per lane with consecutive lanes along a row, and
// passes them one chunk at a time through its own piece of LDS, where it reads
// the MFMA fragments. (Loading fragments directly takes a different row in
// every lane of a quad: measured 36 GB/s per CU from L2 against 100 for loads
// along the rows.) Rows past the end are read from a row inside: a row or
// column of D depends on its own row of w or x alone, and those are not stored.
//
// fp32 operands enter exactly, as three bf16 planes each (round to nearest, the
// remainder again, and what is left: 8 + 8 + 8 bits). The products of planes
// p + q <= 2 are summed; the dropped ones are below 2^-23 of the product. (A value
// that rounds to a bf16 infinity, 3.39e38 or more, gives one less itself: NaN. The
// planes end at 2^-133, the smallest bf16; the matrix cores keep subnormal ones.)
#pragma once

#include "moe_common.h"

namespace moe {
namespace skinny {

constexpr int kChunk = 64;  // k per step of a wave

// 8 floats -> PLANES bf16 fragments whose sum is the floats (3 planes: exactly).
template <int PLANES>
__device__ __forceinline__ void split8(const float (&v)[8], bf16x8 (&out)[PLANES]) {
  u32x4 w[PLANES];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a = v[2 * i], b = v[2 * i + 1];
#pragma unroll
    for (int p = 0; p < PLANES; ++p) {
      const uint32_t u = pack_bf16(a, b);
      w[p][i] = u;
      a -= __uint_as_float(u << 16);
      b -= __uint_as_float(u & 0xffff0000u);
    }
  }
#pragma unroll
  for (int p = 0; p < PLANES; ++p) out[p] = __builtin_bit_cast(bf16x8, w[p]);
}

// The lanes of a wave exchange data through LDS without a barrier: the hardware
// performs a wave's LDS accesses in order, and this keeps the compiler from
// reordering them (no instruction).
__device__ __forceinline__ void wave_lds_order() {
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_wave_barrier();
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// A tile of R rows, one chunk wide: as loaded (kLoads 16-byte words per lane,
// load i covering rows i * kRows ..) and in LDS, where column c (16 bytes) of
// row r is kept at column c ^ (r % kCols), so that the 8 rows a fragment read
// meets at a time lie in different banks.
// R = 16: the two halves of a chunk are an MFMA each. R = 8: one MFMA takes both,
// the first half in rows 0 .. 7 of its operands and the second in rows 8 .. 15;
// of its output the quarters row, column < 8 and row, column >= 8 are the two
// halves' sums, the others mean nothing.
template <typename T, int R>
struct Tile {
  static constexpr int kPlanes = sizeof(T) == 2 ? 1 : 3;
  static constexpr int kRowBytes = kChunk * sizeof(T);
  static constexpr int kCols = kRowBytes / 16;   // lanes along a row
  static constexpr int kRows = 64 / kCols;       // rows per load
  static constexpr int kLoads = R / kRows;
  static constexpr int kBytes = R * kRowBytes;
  static constexpr int kSteps = R / 8;           // MFMAs of a chunk

  __device__ __forceinline__ static int col() { return (threadIdx.x & 63) % kCols; }
  __device__ __forceinline__ static int row(int i) {
    return i * kRows + (threadIdx.x & 63) / kCols;
  }
  // the chunk's first k this lane loads
  __device__ __forceinline__ static int at() { return col() * (16 / (int)sizeof(T)); }

  __device__ __forceinline__ static void put(char* lds, const u32x4 (&v)[kLoads]) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      *(u32x4*)(lds + row(i) * kRowBytes + ((col() ^ (row(i) % kCols)) << 4)) = v[i];
  }
  // this lane's fragment of a step: 8 elements of its row at k-group l >> 4
  __device__ __forceinline__ static void frag(const char* lds, int step,
                                              bf16x8 (&out)[kPlanes]) {
    const int l = threadIdx.x & 15, g = (threadIdx.x >> 4) & 3;
    const int r = l % R, half = R == 16 ? step : l / 8;
    const char* base = lds + r * kRowBytes;
    if constexpr (sizeof(T) == 2) {
      out[0] = __builtin_bit_cast(
          bf16x8, *(const u32x4*)(base + (((half * 4 + g) ^ (r % kCols)) << 4)));
    } else {
      const int c = half * 8 + g * 2;
      const f32x4 a =
          __builtin_bit_cast(f32x4, *(const u32x4*)(base + ((c ^ (r % kCols)) << 4)));
      const f32x4 b =
          __builtin_bit_cast(f32x4, *(const u32x4*)(base + (((c + 1) ^ (r % kCols)) << 4)));
      const float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
      split8<kPlanes>(v, out);
    }
  }
};

// The rows of one operand: N tiles, as per-lane pointers at k = at().
template <typename T, int N, int R>
struct Rows {
  const T* p[N][Tile<T, R>::kLoads];

  // row(i): the address of row i of the R N
  template <typename F>
  __device__ __forceinline__ void set(F row) {
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int i = 0; i < Tile<T, R>::kLoads; ++i)
        p[n][i] = row(n * R + Tile<T, R>::row(i)) + Tile<T, R>::at();
  }
};

template <typename T, int N, int R>
struct Chunk {
  u32x4 v[N][Tile<T, R>::kLoads];

  __device__ __forceinline__ void load(const Rows<T, N, R>& rows, int k) {
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int i = 0; i < Tile<T, R>::kLoads; ++i) v[n][i] = *(const u32x4*)(rows.p[n][i] + k);
  }
  // the partial chunk at the end of K: zeros from there on (K a multiple of 8,
  // so a load lies inside or outside as a whole)
  __device__ __forceinline__ void load_tail(const Rows<T, N, R>& rows, int k, int K) {
    const bool in = k + Tile<T, R>::at() < K;
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int i = 0; i < Tile<T, R>::kLoads; ++i) {
        v[n][i] = u32x4{0, 0, 0, 0};
        if (in) v[n][i] = *(const u32x4*)(rows.p[n][i] + k);
      }
  }
  __device__ __forceinline__ void put(char* lds) const {
#pragma unroll
    for (int n = 0; n < N; ++n) Tile<T, R>::put(lds + n * Tile<T, R>::kBytes, v[n]);
  }
};

template <int MT, int NT, int R, typename XT, typename WT>
struct Product {
  typedef Tile<XT, R> XTile;
  typedef Tile<WT, R> WTile;
  static constexpr int kLdsBytes = MT * XTile::kBytes + NT * WTile::kBytes;  // per wave

  Rows<XT, MT, R> x;
  Rows<WT, NT, R> w;
  f32x4 acc[NT][MT];
  char* lds;  // this wave's kLdsBytes

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < MT; ++i) acc[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  template <int D>
  struct Group {
    Chunk<XT, MT, R> x[D];
    Chunk<WT, NT, R> w[D];
  };

  template <int D>
  __device__ __forceinline__ void load(Group<D>& g, int c, int step) const {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      g.w[d].load(w, (c + d * step) * kChunk);
      g.x[d].load(x, (c + d * step) * kChunk);
    }
  }
  // A chunk through LDS into acc: one piece of LDS serves every chunk.
  __device__ __forceinline__ void put(const Chunk<XT, MT, R>& cx, const Chunk<WT, NT, R>& cw) {
    wave_lds_order();
    cx.put(lds);
    cw.put(lds + MT * XTile::kBytes);
    wave_lds_order();
  }
  __device__ __forceinline__ void multiply() {
#pragma unroll
    for (int step = 0; step < XTile::kSteps; ++step) {
      bf16x8 xf[MT][XTile::kPlanes];
#pragma unroll
      for (int i = 0; i < MT; ++i) XTile::frag(lds + i * XTile::kBytes, step, xf[i]);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        bf16x8 wf[WTile::kPlanes];
        WTile::frag(lds + MT * XTile::kBytes + j * WTile::kBytes, step, wf);
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int p = WTile::kPlanes - 1; p >= 0; --p)
#pragma unroll
            for (int q = XTile::kPlanes - 1; q >= 0; --q)
              if (p + q <= 2) acc[j][i] = mfma_bf16(wf[p], xf[i][q], acc[j][i]);
      }
    }
  }

  // `count` whole chunks c, c + step, ...: groups of D, the next group's loads
  // issued before a group's last chunk is multiplied, then the rest with smaller
  // groups. No load is conditional, so none is waited for early.
  template <int D>
  __device__ __forceinline__ void whole(int c, int step, int count) {
    if (count >= D) {
      Group<D> g;
      load(g, c, step);
      for (; count >= 2 * D; count -= D) {
#pragma unroll
        for (int d = 0; d < D - 1; ++d) {
          put(g.x[d], g.w[d]);
          multiply();
        }
        put(g.x[D - 1], g.w[D - 1]);
        c += D * step;
        load(g, c, step);
        multiply();
      }
#pragma unroll
      for (int d = 0; d < D; ++d) {
        put(g.x[d], g.w[d]);
        multiply();
      }
      c += D * step;
      count -= D;
    }
    if constexpr (D > 1) whole<D / 2>(c, step, count);
  }

  // The chunks first, first + step, ... below `end` of all K.
  template <int D>
  __device__ __forceinline__ void accumulate(int K, int first, int end, int step) {
    const int full = min(end, K / kChunk);
    whole<D>(first, step, first < full ? (full - first + step - 1) / step : 0);
    // the partial last chunk, by the wave whose turn it is
    if (full < end && full >= first && (full - first) % step == 0) {
      Chunk<XT, MT, R> cx;
      Chunk<WT, NT, R> cw;
      cx.load_tail(x, full * kChunk, K);
      cw.load_tail(w, full * kChunk, K);
      put(cx, cw);
      multiply();
    }
  }
};

// LDS of a workgroup of NW waves: their pieces, then (in the same place) their sums.
template <int MT, int NT, int R, int NW, typename XT, typename WT>
constexpr int lds_bytes() {
  constexpr int stage = NW * Product<MT, NT, R, XT, WT>::kLdsBytes;
  constexpr int sums = NW * NT * MT * 1024;
  return stage > sums ? stage : sums;
}

// Sums the accumulators of the NW waves of a workgroup in wave order and calls
// store(w row, x row, sum) for every row of the R MT of x and the R NT of w. A
// sum is four consecutive w rows' (f32x4) where that leaves every thread one,
// else a single value, so that a small tile has many threads at it.
template <int MT, int NT, int R, int NW, typename F>
__device__ __forceinline__ void reduce_waves(const f32x4 (&acc)[NT][MT], char* lds, F store) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float* part = (float*)lds;
  constexpr int kOne = NT * MT * 256;  // values of a wave
  __syncthreads();  // the pieces of all waves are done with
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < MT; ++i)
      ((f32x4*)part)[wave * (kOne / 4) + (j * MT + i) * 64 + lane] = acc[j][i];
  __syncthreads();
  if constexpr (R == 16 && kOne >= NW * 256) {
    for (int u = threadIdx.x; u < kOne / 4; u += NW * 64) {
      f32x4 s = ((const f32x4*)part)[u];
#pragma unroll
      for (int w = 1; w < NW; ++w) s += ((const f32x4*)part)[w * (kOne / 4) + u];
      const int tile = u >> 6, l = u & 63;
      store(tile / MT * R + (l >> 4) * 4, tile % MT * R + (l & 15), s);
    }
  } else if constexpr (R == 16) {
    for (int u = threadIdx.x; u < kOne; u += NW * 64) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) s += part[w * kOne + u];
      const int tile = u >> 8, l = (u >> 2) & 63;
      store(tile / MT * R + (l >> 4) * 4 + (u & 3), tile % MT * R + (l & 15), s);
    }
  } else {
    // the 8 x 8 values of a tile in a wave's lanes 0 .. 31 and in the next
    // iteration's; lanes 32 .. 63 add up the other half of K: rows and columns 8 on
    for (int u = threadIdx.x; u < NT * MT * 128; u += NW * 64) {
      const int tile = u >> 7, v = (u >> 6 & 1) * 32 + (u & 31), half = u >> 5 & 1;
      const int wr = v & 7, xr = v >> 3;
      const int at = tile * 256 + (half * 32 + (wr >> 2) * 16 + half * 8 + xr) * 4 + (wr & 3);
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) s += part[w * kOne + at];
      s += __shfl_xor(s, 32);
      if (half == 0) store(tile / MT * R + wr, tile % MT * R + xr, s);
    }
  }
}

}  // namespace skinny
}  // namespace moe
