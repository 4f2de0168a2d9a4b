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
// p + q <= 2 are summed; the dropped ones are below 2^-23 of the product.
#pragma once

#include "moe_common.h"

namespace moe {
namespace skinny {

constexpr int kChunk = 64;  // k per step of a wave

// 8 floats -> PLANES bf16 fragments whose sum is the floats (3 planes: exactly,
// 2 planes: to 2^-16).
template <int PLANES>
__device__ __forceinline__ void split8(const float (&v)[8], bf16x8 (&out)[PLANES]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float rest = v[i];
#pragma unroll
    for (int p = 0; p < PLANES; ++p) {
      const __bf16 b = (__bf16)rest;
      out[p][i] = b;
      if (p + 1 < PLANES) rest -= (float)b;
    }
  }
}

// A tile of 16 rows, one chunk wide: as loaded (kLoads 16-byte words per lane,
// load i covering rows i * kRows ..) and in LDS, where column c (16 bytes) of
// row r is kept at column c ^ (r % kCols), so that the 8 rows a fragment read
// meets at a time lie in different banks.
template <typename T>
struct Tile {
  static constexpr int kPlanes = sizeof(T) == 2 ? 1 : 3;
  static constexpr int kRowBytes = kChunk * sizeof(T);
  static constexpr int kCols = kRowBytes / 16;   // lanes along a row
  static constexpr int kRows = 64 / kCols;       // rows per load
  static constexpr int kLoads = 16 / kRows;
  static constexpr int kBytes = 16 * kRowBytes;

  __device__ __forceinline__ static int col() { return (threadIdx.x & 63) % kCols; }
  __device__ __forceinline__ static int row(int i) { return i * kRows + (threadIdx.x & 63) / kCols; }
  // the chunk's first k this lane loads
  __device__ __forceinline__ static int at() { return col() * (16 / (int)sizeof(T)); }

  __device__ __forceinline__ static void put(char* lds, const u32x4 (&v)[kLoads]) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      *(u32x4*)(lds + row(i) * kRowBytes + ((col() ^ (row(i) % kCols)) << 4)) = v[i];
  }
  // this lane's fragment of a half: 8 elements of row l & 15 at k-group l >> 4
  __device__ __forceinline__ static void frag(const char* lds, int half, bf16x8 (&out)[kPlanes]) {
    const int r = threadIdx.x & 15, g = (threadIdx.x >> 4) & 3;
    const char* base = lds + r * kRowBytes;
    if constexpr (sizeof(T) == 2) {
      out[0] = *(const bf16x8*)(base + (((half * 4 + g) ^ (r % kCols)) << 4));
    } else {
      const int c = half * 8 + g * 2;
      const f32x4 a = *(const f32x4*)(base + ((c ^ (r % kCols)) << 4));
      const f32x4 b = *(const f32x4*)(base + (((c + 1) ^ (r % kCols)) << 4));
      const float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
      split8<kPlanes>(v, out);
    }
  }
};

// The rows of one operand: N tiles of 16, as per-lane pointers at k = at().
template <typename T, int N>
struct Rows {
  const T* p[N][Tile<T>::kLoads];

  // row(i): the address of row i of the 16 N, i < 16 N
  template <typename F>
  __device__ __forceinline__ void set(F row) {
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int i = 0; i < Tile<T>::kLoads; ++i)
        p[n][i] = row(n * 16 + Tile<T>::row(i)) + Tile<T>::at();
  }
};

template <typename T, int N>
struct Chunk {
  u32x4 v[N][Tile<T>::kLoads];

  __device__ __forceinline__ void load(const Rows<T, N>& rows, int k) {
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int i = 0; i < Tile<T>::kLoads; ++i) v[n][i] = *(const u32x4*)(rows.p[n][i] + k);
  }
  // the partial chunk at the end of K: zeros from there on (K a multiple of 8,
  // so a load lies inside or outside as a whole)
  __device__ __forceinline__ void load_tail(const Rows<T, N>& rows, int k, int K) {
    const bool in = k + Tile<T>::at() < K;
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int i = 0; i < Tile<T>::kLoads; ++i) {
        v[n][i] = u32x4{0, 0, 0, 0};
        if (in) v[n][i] = *(const u32x4*)(rows.p[n][i] + k);
      }
  }
  __device__ __forceinline__ void put(char* lds) const {
#pragma unroll
    for (int n = 0; n < N; ++n) Tile<T>::put(lds + n * Tile<T>::kBytes, v[n]);
  }
};

template <int MT, int NT, typename XT, typename WT>
struct Product {
  static constexpr int kLdsBytes = MT * Tile<XT>::kBytes + NT * Tile<WT>::kBytes;  // per wave

  Rows<XT, MT> x;
  Rows<WT, NT> w;
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
    Chunk<XT, MT> x[D];
    Chunk<WT, NT> w[D];
  };

  template <int D>
  __device__ __forceinline__ void load(Group<D>& g, int c, int step) const {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      g.w[d].load(w, (c + d * step) * kChunk);
      g.x[d].load(x, (c + d * step) * kChunk);
    }
  }
  // Passes chunk d of the group through LDS into acc. The LDS accesses of a
  // wave are performed in order, so one piece of LDS serves every chunk.
  __device__ __forceinline__ void put(const Chunk<XT, MT>& cx, const Chunk<WT, NT>& cw) {
    cx.put(lds);
    cw.put(lds + MT * Tile<XT>::kBytes);
  }
  __device__ __forceinline__ void multiply() {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      bf16x8 xf[MT][Tile<XT>::kPlanes];
#pragma unroll
      for (int i = 0; i < MT; ++i) Tile<XT>::frag(lds + i * Tile<XT>::kBytes, half, xf[i]);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        bf16x8 wf[Tile<WT>::kPlanes];
        Tile<WT>::frag(lds + MT * Tile<XT>::kBytes + j * Tile<WT>::kBytes, half, wf);
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int p = Tile<WT>::kPlanes - 1; p >= 0; --p)
#pragma unroll
            for (int q = Tile<XT>::kPlanes - 1; q >= 0; --q)
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
      Chunk<XT, MT> cx;
      Chunk<WT, NT> cw;
      cx.load_tail(x, full * kChunk, K);
      cw.load_tail(w, full * kChunk, K);
      put(cx, cw);
      multiply();
    }
  }
};

// LDS of a workgroup of NW waves: their pieces, then (in the same place) their sums.
template <int MT, int NT, int NW, typename XT, typename WT>
constexpr int lds_bytes() {
  constexpr int stage = NW * Product<MT, NT, XT, WT>::kLdsBytes;
  constexpr int sums = NW * NT * MT * 1024;
  return stage > sums ? stage : sums;
}

// Sums the accumulators of the NW waves of a workgroup in wave order and calls
// store(nt, mt, lane, sum) for every tile and lane; sum holds w rows
// 16 nt + 4 (lane >> 4) .. + 3 of x row 16 mt + (lane & 15).
template <int MT, int NT, int NW, typename F>
__device__ __forceinline__ void reduce_waves(const f32x4 (&acc)[NT][MT], char* lds, F store) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  f32x4* part = (f32x4*)lds;
  constexpr int kOne = NT * MT * 64;
  __syncthreads();  // the pieces of all waves are done with
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < MT; ++i) part[wave * kOne + (j * MT + i) * 64 + lane] = acc[j][i];
  __syncthreads();
  for (int u = threadIdx.x; u < kOne; u += NW * 64) {
    f32x4 s = part[u];
#pragma unroll
    for (int w = 1; w < NW; ++w) s += part[w * kOne + u];
    const int tile = u >> 6;
    store(tile / MT, tile % MT, u & 63, s);
  }
}

}  // namespace skinny
}  // namespace moe
