// Low-rank adapters of many requests beside a shared projection:
// out[s] = y[s] + scale[g] * b[g] (a[g] x[s]) for the rows s of adapter g.
//
// Two launches over the aligned row lists, both bound by memory (2 r flops per
// element of x, y, a or b): the shrink z = a x, split over K, leaves fp32
// partial sums in the workspace (r numbers per row: nothing next to x and y);
// the expansion adds them up and works b into the rows of y. Small batches run
// both in one launch.
// Measured (captured into a graph): 16 requests with r 16 beside 4096 x 4096 6.8
// us, one 4.3 us; 512 slots of 8 adapters x 128 experts, r 8, 2048
// -> 7168, 16.9 us = 3.5 TB/s; 4096 rows of prompts, 8 adapters of r 64, 4096 x
// 4096, 26.2 us = 3.1 TB/s.
#include "../../include/moe.h"
#include "moe_common.h"
#include "moe_launch.h"
#include "moe_skinny.h"

namespace moe {
namespace lora {

using skinny::kChunk;

// How a problem is cut: decided on the host from its sizes alone.
struct Plan {
  int log2m;
  bool many;   // rows of an adapter on average: 32 or more
  bool tiles;  // the expansion shares b between rows
  int slices;  // of K, a power of two
  int rows;    // of a group of the expansion: consecutive positions of a block
  int rows_a;  // of a group of the shrink
};

// Some rows of an adapter: lane l < count has the l-th.
struct Group {
  int adapter, count, row;
};
// The rows of the lanes in `which`. The alignment puts a block's rows first; should
// a list not, they are brought together here.
__device__ __forceinline__ Group group_of(int adapter, int row, uint64_t which) {
  Group r;
  r.adapter = adapter;
  r.count = __builtin_popcountll(which);
  if (which & (which + 1)) {
    int from = 0, i = 0;
    for (uint64_t left = which; left; left &= left - 1, ++i)
      if ((int)(threadIdx.x & 63) == i) from = __builtin_ctzll(left);
    row = __shfl(row, from);
  }
  r.row = row;
  return r;
}
// The group's row i, or its last one past the end.
__device__ __forceinline__ int row_at(const Group& g, int i) {
  return __shfl(g.row, min(i, g.count - 1));
}
// The rows at g * rows .. of the lists.
__device__ __forceinline__ Group group_at(const LoraProblem& p, const Plan& c, long g, int rows) {
  const long pos = g * rows;
  const int lane = threadIdx.x & 63;
  // the loads do not wait for each other: past *num_padded the lists still
  // hold what the alignment wrote there
  const int padded = p.num_padded[0];
  const int adapter = p.block_adapter[pos >> c.log2m];
  const int row = p.sorted_ids[pos + min(lane, rows - 1)];
  return group_of(adapter, row,
                  __ballot(lane < rows && (unsigned)row < (unsigned)p.S && pos < padded &&
                           (unsigned)adapter < (unsigned)p.n));
}

// A workgroup's pieces of N rows: the piece 0 of its group, the piece 1 of the group
// an eighth of them further on, and so forth. A block of few rows has a piece 0
// alone; the pieces of a full one, a much-used adapter's, are in as many workgroups
// (256 rows of 4 of 256 adapters, r 16 beside 4096 x 4096: 14.3 us, 46 with the
// pieces of a group in turn; groups of 8 rows each take 18, but 36 instead of 15.7
// where every row has an adapter of its own).
template <int N>
struct Pieces {
  int row, adapter;  // of lane l: piece l / N, position l % N
  uint64_t left;     // lanes with a row, of the pieces still to do

  // the first position of piece j (j * shift < groups)
  __device__ __forceinline__ static long position(int g, int rows, int groups, int j) {
    int at = g + j * (groups / 8);
    if (at >= groups) at -= groups;
    return (long)at * rows + j * N;
  }
  __device__ __forceinline__ Pieces(const LoraProblem& p, const Plan& c, int g, int rows,
                                    int groups) {
    const int me = threadIdx.x & 63, lane = min(me, rows - 1);
    const long pos = position(g, rows, groups, lane / N) + lane % N;
    const int padded = p.num_padded[0];
    adapter = p.block_adapter[pos >> c.log2m];
    row = p.sorted_ids[pos];
    left = __ballot(me < rows && (unsigned)row < (unsigned)p.S && pos < padded &&
                    (unsigned)adapter < (unsigned)p.n);
  }
  // the next piece's number; its rows
  __device__ __forceinline__ int next() const { return __builtin_ctzll(left) / N; }
  __device__ __forceinline__ Group take(int j) {
    const uint64_t mine = left >> (j * N) & ((1ull << N) - 1);
    left &= ~(((1ull << N) - 1) << (j * N));
    return group_of(__builtin_amdgcn_readlane(adapter, j * N),
                    __shfl(row, min(j * N + (int)(threadIdx.x & 63), 63)), mine);
  }
};

// ---------------------------------------------------------------- shrink ---
// A workgroup: R NT ranks of a group's adapter, one slice of K, R MT rows at a
// time. Bound by reading x and, for few rows, a; every 16 or 32 rows read a again,
// from L2 (the prompts above: 9.3 us, 5 of them for x at the rate of a copy).
constexpr int kShrinkWaves = 8;

template <int MT, int NT, int R, typename XT>
__global__ __launch_bounds__(kShrinkWaves * 64) void shrink_kernel(LoraProblem p, Plan c,
                                                                   int rank_tiles, int groups) {
  constexpr int NW = kShrinkWaves;
  __shared__ __align__(16) char lds[skinny::lds_bytes<MT, NT, R, NW, XT, uint16_t>()];
  __shared__ int rows[R * MT];
  const int slice = blockIdx.x / rank_tiles, q0 = blockIdx.x % rank_tiles * NT * R;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int chunks = (p.K + kChunk - 1) / kChunk;
  const int first = (int)((long)chunks * slice / c.slices);
  const int end = (int)((long)chunks * (slice + 1) / c.slices);
  float* z = (float*)p.workspace + (size_t)slice * p.S * p.r;
  for (int gi = blockIdx.y; gi < groups; gi += gridDim.y) {
    Pieces<R * MT> pieces(p, c, gi, c.rows_a, groups);
    while (pieces.left) {  // the whole workgroup
      const Group g = pieces.take(pieces.next());
      if (threadIdx.x < R * MT) rows[threadIdx.x] = g.row;
      const uint16_t* a = p.a + (size_t)g.adapter * p.r * p.K;
      skinny::Product<MT, NT, R, XT, uint16_t> m;
      m.lds = lds + wave * m.kLdsBytes;
      m.x.set([&](int i) { return (const XT*)p.x + (size_t)row_at(g, i) * p.ldx; });
      m.w.set([&](int i) { return a + (size_t)min(q0 + i, p.r - 1) * p.K; });
      m.clear();
      // two chunks in flight where their registers allow it
      constexpr int D = MT * (int)sizeof(XT) / 2 + NT <= 5 ? 2 : 1;
      m.template accumulate<D>(p.K, first + wave, end, NW);
      skinny::reduce_waves<MT, NT, R, NW>(m.acc, lds, [&](int wr, int xr, auto s) {
        // (rows: the lanes that hold them need not be here; 4 divides the rank)
        const int q = q0 + wr;
        if (xr < g.count && q < p.r) *(decltype(s)*)(z + (size_t)rows[xr] * p.r + q) = s;
      });
      __syncthreads();  // the sums and rows are read before the next ones
    }
  }
}

// ---------------------------------------------------------------- expand ---
// D = z (rows) x b (columns), 16 rows and 16 J columns at a time, with column
// J cc + j in column cc of tile j: a lane then holds J consecutive columns of 4
// rows, 16 bytes of y, and 16 lanes 256 bytes of a row. (J 4 and half of that for
// bf16 rows and ranks past 64, whose b takes the registers.)
// STEPS: MFMAs over the rank, 32 of it each.

// z enters the matrix cores exactly, as three bf16 planes. (Two, 16 bits, would take 25.5 us
// instead of 26.1 for the prompts above, and show 2^-16 of b z where y cancels it.)
constexpr int kZPlanes = 3;

// z of rows 16 t .. of a group: 8 ranks from q of row lane & 15 in each step (any
// values past the rank, where b is zero).
template <int STEPS>
struct Z16 {
  bf16x8 f[STEPS][kZPlanes];

  __device__ __forceinline__ void load(const LoraProblem& p, const Plan& c, const Group& g, int t,
                                       int q) {
    const size_t slice = (size_t)p.S * p.r;
    const float* zp =
        (const float*)p.workspace + (size_t)row_at(g, t * 16 + (threadIdx.x & 15)) * p.r;
    float v[STEPS][8] = {};
    constexpr int kTogether = STEPS < 4 ? 4 / STEPS : 1;  // slices whose loads are in flight
    if (c.slices < kTogether) {
      for (int k = 0; k < c.slices; ++k) add<1>(v, zp + k * slice, 0, q, p.r);
    } else {  // powers of two both
      for (int k = 0; k < c.slices; k += kTogether)
        add<kTogether>(v, zp + k * slice, slice, q, p.r);
    }
#pragma unroll
    for (int s = 0; s < STEPS; ++s) skinny::split8<kZPlanes>(v[s], f[s]);
  }
  // N slices, their loads together
  template <int N>
  __device__ __forceinline__ static void add(float (&v)[STEPS][8], const float* zp, size_t slice,
                                             int q, int r) {
    f32x4 w[N][STEPS][2];
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        const f32x4* from = (const f32x4*)(zp + k * slice + min(s * 32 + q, r - 8));
        w[k][s][0] = from[0];
        w[k][s][1] = from[1];
      }
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
      for (int s = 0; s < STEPS; ++s)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[s][e] += w[k][s][e >> 2][e & 3];
  }
};

// J columns from n of rows 16 t + 4 (lane >> 4) .. + 3 of a group, of y.
template <int J, typename YT>
struct Y4 {
  static constexpr int kWords = J * (int)sizeof(YT) / 4;  // 32-bit words of a row
  uint32_t w[4][kWords];

  __device__ __forceinline__ void load(const LoraProblem& p, const Group& g, int t, int n) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = t * 16 + ((threadIdx.x >> 4) & 3) * 4 + i, row = row_at(g, at);
      const YT* yp = (const YT*)p.y + (size_t)row * p.ldy + n;
#pragma unroll
      for (int q = 0; q < kWords; ++q) w[i][q] = 0;
      if (at < g.count && n < p.N) {
        if constexpr (kWords == 2) {
          const u32x2 v = *(const u32x2*)yp;
          w[i][0] = v[0];
          w[i][1] = v[1];
        } else {
#pragma unroll
          for (int q = 0; q < kWords; q += 4) {
            const u32x4 v = ((const u32x4*)yp)[q / 4];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[i][q + e] = v[e];
          }
        }
      }
    }
  }
};

// out = y + scale * z b for those rows and columns; frag(s, j): b's fragments.
// Two of the J tiles at a time: their sums go into y's registers.
template <int J, int STEPS, typename YT, typename F>
__device__ __forceinline__ void add_rows(const LoraProblem& p, const Group& g, int t,
                                         const Z16<STEPS>& z, Y4<J, YT>& y, float scale, int n,
                                         F frag) {
  constexpr int kWords = Y4<J, YT>::kWords;
#pragma unroll
  for (int j = 0; j < J; j += 2) {
    f32x4 lo = {0.f, 0.f, 0.f, 0.f}, hi = lo;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const bf16x8 b0 = frag(s, j), b1 = frag(s, j + 1);
#pragma unroll
      for (int q = kZPlanes - 1; q >= 0; --q) {
        lo = mfma_bf16(z.f[s][q], b0, lo);
        hi = mfma_bf16(z.f[s][q], b1, hi);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(YT) == 2) {
        const uint32_t w = y.w[i][j / 2];
        y.w[i][j / 2] = pack_bf16(bf16_bits_to_f32(w & 0xffffu) + scale * lo[i],
                                  __uint_as_float(w & 0xffff0000u) + scale * hi[i]);
      } else {
        y.w[i][j] = __float_as_uint(__uint_as_float(y.w[i][j]) + scale * lo[i]);
        y.w[i][j + 1] = __float_as_uint(__uint_as_float(y.w[i][j + 1]) + scale * hi[i]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int at = t * 16 + ((threadIdx.x >> 4) & 3) * 4 + i, row = row_at(g, at);
    if (at < g.count && n < p.N) {
      YT* op = (YT*)p.out + (size_t)row * p.ldo + n;
      const uint32_t* o = y.w[i];
      if constexpr (kWords == 2) {
        *(u32x2*)op = u32x2{o[0], o[1]};
      } else {
#pragma unroll
        for (int q = 0; q < kWords; q += 4)
          ((u32x4*)op)[q / 4] = u32x4{o[q], o[q + 1], o[q + 2], o[q + 3]};
      }
    }
  }
}

// Few rows of an adapter and a rank above 32: b is most of the traffic and each
// of its rows is used once or little more. A wave keeps the b of 16 J columns in
// registers and takes the group's rows 16 at a time (16 requests of r 64, an adapter
// each, beside 2048 -> 8192: 12.3 us with the shrink, 14.6 with b shared through LDS).
template <int J, int STEPS, typename YT>
__global__ __launch_bounds__(256) void expand_kernel(LoraProblem p, Plan c, int groups) {
  const int g4 = (threadIdx.x >> 4) & 3;
  const int n0 = (blockIdx.x * 4 + (threadIdx.x >> 6)) * 16 * J;
  if (n0 >= p.N) return;  // whole waves
  const int n = n0 + (threadIdx.x & 15) * J;
  for (int gi = blockIdx.y; gi < groups; gi += gridDim.y) {
    Pieces<16> pieces(p, c, gi, c.rows, groups);
    while (pieces.left) {
      const Group g = pieces.take(pieces.next());
      const float scale = p.scale ? p.scale[g.adapter] : 1.f;
      const uint16_t* b = p.b + ((size_t)g.adapter * p.N + min(n, p.N - J)) * p.r;  // J divides N
      u32x4 bq[STEPS][J];
#pragma unroll
      for (int s = 0; s < STEPS; ++s)
#pragma unroll
        for (int j = 0; j < J; ++j)
          bq[s][j] = *(const u32x4*)(b + (size_t)j * p.r + min(s * 32 + g4 * 8, p.r - 8));
      Z16<STEPS> z;
      Y4<J, YT> y;
      y.load(p, g, 0, n);
      z.load(p, c, g, 0, g4 * 8);
      add_rows(p, g, 0, z, y, scale, n, [&](int s, int j) {
        return __builtin_bit_cast(bf16x8, s * 32 + g4 * 8 < p.r ? bq[s][j] : u32x4{0, 0, 0, 0});
      });
    }
  }
}

// Few rows and a rank of at most 32 (PIECES = r / 8 pieces of 16 bytes): a lane
// takes whole rows of b, one column of the output each, and fp32 FMAs do the
// little there is to compute; z lies in LDS, read by all lanes alike, and 8 KB of
// b per wave are in flight. On matrix tiles, one row of 16 of them used, a wave
// had 2 KB in flight and the expert slots above took 21 us; they take 11.3 here,
// where 45 MB at the rate of a copy are 9.
template <int PIECES, typename YT>
struct Columns {
  static constexpr int U = 8 / PIECES;  // columns of a lane: n0, n0 + 64, ...
  static constexpr int R = PIECES * 8;  // rank
  static constexpr int RB = 2;          // rows of y in flight
  u32x4 b[U][PIECES];
  YT y[RB][U];

  __device__ __forceinline__ void load_b(const LoraProblem& p, const Group& g, int n0) {
    const uint16_t* from = p.b + (size_t)g.adapter * p.N * R;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int q = 0; q < PIECES; ++q)
        b[u][q] = ((const u32x4*)(from + (size_t)min(n0 + u * 64, p.N - 1) * R))[q];
  }
  __device__ __forceinline__ void load_y(const LoraProblem& p, const Group& g, int i0, int n0) {
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      if (i0 + i < g.count) {
        const YT* yp = (const YT*)p.y + (size_t)row_at(g, i0 + i) * p.ldy;
#pragma unroll
        for (int u = 0; u < U; ++u) y[i][u] = yp[min(n0 + u * 64, p.N - 1)];
      }
    }
  }
  // rows i0 .. of the group, RB of them; z: theirs, in LDS
  __device__ __forceinline__ void add(const LoraProblem& p, const Group& g, int i0, int n0,
                                      float scale, const float* z) const {
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      if (i0 + i < g.count) {
        YT* op = (YT*)p.out + (size_t)row_at(g, i0 + i) * p.ldo;
        float acc[U] = {};
#pragma unroll
        for (int q = 0; q < PIECES; ++q) {
          const f32x4 lo = *(const f32x4*)(z + i * R + q * 8);
          const f32x4 hi = *(const f32x4*)(z + i * R + q * 8 + 4);
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t w = b[u][q][e];
              acc[u] += (e < 2 ? lo : hi)[e * 2 & 3] * bf16_bits_to_f32(w & 0xffffu);
              acc[u] += (e < 2 ? lo : hi)[(e * 2 & 3) + 1] * __uint_as_float(w & 0xffff0000u);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (n0 + u * 64 < p.N) {
            if constexpr (sizeof(YT) == 2)
              op[n0 + u * 64] = (YT)pack_bf16(bf16_bits_to_f32(y[i][u]) + scale * acc[u], 0.f);
            else
              op[n0 + u * 64] = y[i][u] + scale * acc[u];
          }
        }
      }
    }
  }
};

template <int PIECES, typename YT>
__global__ __launch_bounds__(256) void expand_columns_kernel(LoraProblem p, Plan c, int groups) {
  typedef Columns<PIECES, YT> Cols;
  constexpr int R = Cols::R;
  __shared__ __align__(16) float zl[8 * R];
  const int n0 = (blockIdx.x * 4 + (threadIdx.x >> 6)) * Cols::U * 64 + (threadIdx.x & 63);
  for (int gi = blockIdx.y; gi < groups; gi += gridDim.y) {
    Pieces<8> pieces(p, c, gi, c.rows, groups);
    while (pieces.left) {  // the whole workgroup
      const Group g = pieces.take(pieces.next());
      const float scale = p.scale ? p.scale[g.adapter] : 1.f;
      Cols m;
      m.load_b(p, g, n0);
      m.load_y(p, g, 0, n0);
      const int e = threadIdx.x;  // R of 8 rows: 256 values at most
      const size_t at = (size_t)row_at(g, e / R) * R + e % R, slice = (size_t)p.S * R;
      const float* z = (const float*)p.workspace + at;
      float v = z[0];
      if (c.slices == 2) v += z[slice];
      if (c.slices >= 4) {  // a power of two: the loads of four together
        v = 0.f;
        for (int k = 0; k < c.slices; k += 4)
          v += (z[k * slice] + z[(k + 1) * slice]) + (z[(k + 2) * slice] + z[(k + 3) * slice]);
      }
      if (e < g.count * R) zl[e] = v;
      __syncthreads();
      for (int i0 = 0; i0 < g.count; i0 += Cols::RB) {
        if (i0) m.load_y(p, g, i0, n0);
        m.add(p, g, i0, n0, scale, zl + i0 * R);
      }
      __syncthreads();  // z is read before the next piece's comes in
    }
  }
}

// Both steps in one launch, for batches whose groups do not fill the chip: there
// a second launch costs more than reading a once per 8 waves' columns. A
// workgroup forms z of 8 rows at a time (all of K, split over its waves, as the
// shrink does) and adds its columns, whose b and y are on their way while the
// waves' sums are added (asked for before the products, b's registers slow those:
// by 0.5 us). 16 requests of r 16 beside 4096 x 4096 6.8 us, 7.8 in two launches;
// one 4.3, 5.7.
constexpr int kOneWaves = 8;

template <int PIECES, typename XT, typename YT>
__global__ __launch_bounds__(kOneWaves * 64) void one_launch_kernel(LoraProblem p, Plan c,
                                                                    int groups) {
  constexpr int NW = kOneWaves;
  typedef Columns<PIECES, YT> Cols;
  typedef skinny::Product<1, PIECES, 8, XT, uint16_t> Shrink;
  constexpr int R = Cols::R;
  __shared__ __align__(16) char lds[skinny::lds_bytes<1, PIECES, 8, NW, XT, uint16_t>()];
  __shared__ __align__(16) float zl[8 * R];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = (blockIdx.x * NW + wave) * Cols::U * 64 + (threadIdx.x & 63);
  const int chunks = (p.K + kChunk - 1) / kChunk;
  for (int gi = blockIdx.y; gi < groups; gi += gridDim.y) {
    Pieces<8> pieces(p, c, gi, c.rows, groups);
    while (pieces.left) {  // the whole workgroup
      const Group g = pieces.take(pieces.next());
      const uint16_t* a = p.a + (size_t)g.adapter * R * p.K;
      Cols cols;
      Shrink m;
      m.lds = lds + wave * m.kLdsBytes;
      m.x.set([&](int i) { return (const XT*)p.x + (size_t)row_at(g, i) * p.ldx; });
      m.w.set([&](int i) { return a + (size_t)i * p.K; });
      m.clear();
      m.template accumulate<PIECES * (int)sizeof(XT) <= 8 ? 4 : 2>(p.K, wave, chunks, NW);
      cols.load_b(p, g, n0);
      cols.load_y(p, g, 0, n0);
      const float scale = p.scale ? p.scale[g.adapter] : 1.f;
      skinny::reduce_waves<1, PIECES, 8, NW>(m.acc, lds, [&](int wr, int xr, float s) {
        zl[xr * R + wr] = s;
      });
      __syncthreads();
      for (int i = 0; i < g.count; i += Cols::RB) {
        if (i) cols.load_y(p, g, i, n0);
        cols.add(p, g, i, n0, scale, zl + i * R);
      }
      __syncthreads();  // z is read before the next piece's comes in
    }
  }
}

// More rows of an adapter: a workgroup takes up to 64 rows of it, 16 to a wave,
// and every stride-th 16 J columns, whose rows of b it brings into LDS once for
// all its rows, 16 bytes per lane along b. z stays in registers from one set of
// columns to the next (it is as large as y's columns from a rank of 64 on), and
// the next ones' b and y are in flight while these are worked on. The prompts
// above: 16 us, 10 of them for y and out at the rate of a copy.
// The registers are what it needs: held to 128 a rank of 16 spills four and takes
// 28.7 us instead of 27.8 (4096 rows of 64 adapters), and so does a rank of 64 held
// to 168, three waves a SIMD instead of two: 14, the prompts above 28.3 instead of 26.1.
template <int J, int STEPS, typename YT>
__global__ __launch_bounds__(256, 1) void expand_tiles_kernel(LoraProblem p, Plan c, int groups) {
  // rows of b at (n % J) * 16 + n / J, so that a tile's are together; 16 bytes
  // of padding spread a column of them over the banks
  constexpr int kStride = STEPS * 64 + 16;
  constexpr int kLoads = J * STEPS / 4;  // of a thread: 16 J rows of 64 STEPS bytes at most
  __shared__ __align__(16) char lds[16 * J * kStride];
  const int g4 = (threadIdx.x >> 4) & 3, cc = threadIdx.x & 15, wave = threadIdx.x >> 6;
  const int units = (p.N + 16 * J - 1) / (16 * J), stride = gridDim.x;
  const int pieces = p.r / 8;  // 16-byte pieces of a row of b
  int to[kLoads];              // where this thread's pieces go
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int e = threadIdx.x + i * 256, row = e / pieces;
    to[i] = ((row % J) * 16 + row / J) * kStride + (e - row * pieces) * 16;
  }
  for (int gi = blockIdx.y; gi < groups; gi += gridDim.y) {
    const Group g = group_at(p, c, gi, c.rows);
    if (g.count == 0) continue;  // the whole workgroup
    const float scale = p.scale ? p.scale[g.adapter] : 1.f;
    const u32x4* b = (const u32x4*)(p.b + (size_t)g.adapter * p.N * p.r);
    auto column = [&](int u) { return (u * 16 + cc) * J; };
    auto pieces_of = [&](int u) { return min(16 * J, p.N - u * 16 * J) * pieces; };
    u32x4 bq[kLoads];
    auto load_b = [&](int u) {
      const u32x4* from = b + (size_t)u * 16 * J * pieces;
      const int last = pieces_of(u) - 1;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) bq[i] = from[min((int)threadIdx.x + i * 256, last)];
    };
    const bool mine = wave * 16 < g.count;
    Z16<STEPS> z;
    Y4<J, YT> even, odd;
    load_b(blockIdx.x);
    if (mine) {
      even.load(p, g, wave, column(blockIdx.x));
      z.load(p, c, g, wave, g4 * 8);
    }
    auto step = [&](int u, Y4<J, YT>& now, Y4<J, YT>& next) {
      const int rows_b = min(16 * J, p.N - u * 16 * J);
      __syncthreads();  // the previous columns' b is read
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
        if ((int)threadIdx.x + i * 256 < rows_b * pieces) *(u32x4*)(lds + to[i]) = bq[i];
      __syncthreads();
      if (u + stride < units) {
        load_b(u + stride);
        if (mine) next.load(p, g, wave, column(u + stride));
      }
      if (mine)
        add_rows(p, g, wave, z, now, scale, column(u), [&](int s, int j) {
          // zero past the rank and past the last column
          u32x4 v = {0, 0, 0, 0};
          if (s * 4 + g4 < pieces && cc * J < rows_b)
            v = *(const u32x4*)(lds + (j * 16 + cc) * kStride + (s * 4 + g4) * 16);
          return __builtin_bit_cast(bf16x8, v);
        });
    };
    for (int u = blockIdx.x; u < units; u += 2 * stride) {
      step(u, even, odd);  // two sets of registers in turn: a copy would wait for the loads
      if (u + stride < units) step(u + stride, odd, even);
    }
  }
}

// ------------------------------------------------------------------ host ---

// Rows of z that the slices of K may add up to, where a call's own are fewer.
constexpr long kSliceRows = 16384;
constexpr int kMaxSlices = 16;

static int max_slices(int K) {
  const int chunks = (K + kChunk - 1) / kChunk;
  const int most = chunks / kShrinkWaves;  // a chunk for every wave
  return most < 1 ? 1 : most > kMaxSlices ? kMaxSlices : most;
}

static int groups_of(const LoraProblem& p, int rows) {
  return (int)(align_capacity(p.S, p.n, p.block_m) / rows);
}

static Plan plan_of(const LoraProblem& p) {
  Plan c{};
  while ((1 << c.log2m) < p.block_m) ++c.log2m;
  c.rows = p.block_m < 64 ? p.block_m : 64;
  c.many = p.block_m >= 32 && (long)p.S >= 32L * p.n;
  // b shared between rows from 8 rows an adapter on (4096 x 4096, r 16, a quarter of
  // the rows without an adapter and some adapters popular: 512 adapters x 4 rows 59
  // us so, 46.8 row by row; 16 adapters x 8 8.0, 13.6); with so few adapters that
  // their groups do not fill the chip, from 2 and up to a rank of 64 (16 adapters x 2
  // rows 7.6, 7.7, x 6 8.0, 10.0; r 64 x 2 11.3, 12.2; a rank of 128 x 4 22.7, 17.8).
  // Of how the rows are spread the host knows nothing: with two for every adapter a
  // rank of 16 takes 7.8 and 6.5.
  c.tiles = (long)p.S >= 8L * p.n || (p.n <= 16 && p.S >= 2 * p.n && p.r <= 64);
  // 16 rows to a group of the shrink until 32 of them are 256 groups
  if (c.many) c.rows_a = p.S >= 4096 ? 32 : 16;
  // and 16 where fewer than 8 groups cannot share out their pieces (28 rows of an
  // adapter of r 128, 936 -> 360, 8.6 us instead of 9.7)
  else c.rows_a = c.tiles && c.rows > 16 && groups_of(p, c.rows) < 8 ? 16 : c.rows;
  // slices of K until some 256 workgroups (of much-used adapters) or 512 have work;
  // fewer past a rank of 64, since the expansion reads the rows' z of every slice
  // once per 128 columns (512 rows of 8 adapters, 4096 x 4096: r 128 18.9 us, 32 with
  // as many as for r 64; r 256 32, 62), and past 32 where it takes rows 16 at a time
  // of which few are there (64 rows of 64 adapters, r 64: 17.2 us, 20.2)
  const long groups = c.many ? p.S / c.rows_a + 1 : p.S / 16 + (p.n < p.S ? p.n : p.S) / 2 + 1;
  const long weight = p.r > 64 || (p.r > 32 && !c.tiles) ? (p.r + 31) / 32 : 1;
  const long most = max_slices(p.K), want = c.many ? 320 : 512;
  c.slices = 1;
  while (c.slices * 2 <= most && c.slices * 2 * groups * weight <= want) c.slices *= 2;
  return c;
}

static int grid_y(int groups) { return groups < 65535 ? groups : 65535; }

template <int MT, int NT, int R, typename XT>
static void shrink(const LoraProblem& p, const Plan& c, hipStream_t stream) {
  const int rank_tiles = (p.r + NT * R - 1) / (NT * R), groups = groups_of(p, c.rows_a);
  shrink_kernel<MT, NT, R, XT><<<dim3(c.slices * rank_tiles, grid_y(groups)), kShrinkWaves * 64, 0,
                              stream>>>(p, c, rank_tiles, groups);
}

template <typename XT>
static void run_shrink(const LoraProblem& p, const Plan& c, hipStream_t stream) {
  const bool pairs = c.many && c.rows_a == 32;
  // 16 ranks to a workgroup while those are one a CU at most (the same 28 rows 8.6 us
  // instead of 10.0; with 208 of them, 96 rows of 12 adapters of r 64, 2048 -> 8192,
  // 13.5 and 14.3; with 272, 128 rows of 16 of r 24, 4096 x 4096, 8.7 both; with 288,
  // 100 rows of 4 of r 128, 2048 x 2048, 11.2 and 10.9)
  const long narrow =
      (p.S / 16 + (p.n < p.S ? p.n : p.S) / 2 + 1) * (long)c.slices * ((p.r + 15) / 16);
  if (c.tiles && !pairs && p.r > 16 && narrow <= 256) shrink<1, 1, 16, XT>(p, c, stream);
  else if (p.r > 32)
    pairs ? shrink<2, 4, 16, XT>(p, c, stream) : shrink<1, 4, 16, XT>(p, c, stream);
  else if (p.r > 16)
    pairs ? shrink<2, 2, 16, XT>(p, c, stream) : shrink<1, 2, 16, XT>(p, c, stream);
  else if (pairs) shrink<2, 1, 16, XT>(p, c, stream);
  else if (c.tiles) shrink<1, 1, 16, XT>(p, c, stream);
  else if (p.r > 8) shrink<1, 2, 8, XT>(p, c, stream);
  else shrink<1, 1, 8, XT>(p, c, stream);
}

template <int J, int STEPS, typename YT>
static void expand(const LoraProblem& p, const Plan& c, hipStream_t stream) {
  const int groups = groups_of(p, c.rows), units = (p.N + 16 * J - 1) / (16 * J);
  // some 1024 workgroups at work; beyond, one takes several sets of columns, all
  // of them as many (4096 rows r 128: 36.8 us; 2048 workgroups 37.6, 4096 46)
  const long live = p.S / c.rows + (p.n < p.S ? p.n : p.S) / 2 + 1;
  const int want = (int)((1024 + live - 1) / live), each = units > want ? units / want : 1;
  if (c.tiles)
    expand_tiles_kernel<J, STEPS, YT>
        <<<dim3((units + each - 1) / each, grid_y(groups)), 256, 0, stream>>>(p, c, groups);
  else if constexpr (STEPS > 1)
    expand_kernel<J, STEPS, YT>
        <<<dim3((units + 3) / 4, grid_y(groups)), 256, 0, stream>>>(p, c, groups);
}

template <int PIECES, typename YT>
static void expand_columns(const LoraProblem& p, const Plan& c, hipStream_t stream) {
  constexpr int kColumns = 4 * 64 * Columns<PIECES, YT>::U;  // of a workgroup
  const int groups = groups_of(p, c.rows);
  expand_columns_kernel<PIECES, YT>
      <<<dim3((p.N + kColumns - 1) / kColumns, grid_y(groups)), 256, 0, stream>>>(p, c, groups);
}

template <typename YT>
static void run_expand(const LoraProblem& p, const Plan& c, hipStream_t stream) {
  constexpr int J = 16 / sizeof(YT);  // 16 bytes of a row per lane
  if (!c.tiles && p.r == 8) expand_columns<1, YT>(p, c, stream);
  else if (!c.tiles && p.r == 16) expand_columns<2, YT>(p, c, stream);
  else if (!c.tiles && p.r == 24) expand_columns<3, YT>(p, c, stream);
  else if (!c.tiles && p.r == 32) expand_columns<4, YT>(p, c, stream);
  else if (p.r <= 32) expand<J, 1, YT>(p, c, stream);
  else if (p.r <= 64) expand<J, 2, YT>(p, c, stream);
  else if (p.r <= 128) expand<4, 4, YT>(p, c, stream);
  else expand<4, 8, YT>(p, c, stream);
}

// Whether both steps run in one launch: up to 512 readings of 8 ranks of a (2048 ->
// 7168, r 8: 256 slots of 512 adapters 11.4 us in one, 12.2 in two; 4096 x 4096: 128
// requests of r 16 9.5 and 11.4, 256 15.0 and 14.6, 128 of r 32 19.6 and 14.0).
static bool one_launch(const LoraProblem& p, const Plan& c) {
  if (c.tiles || p.r > 32) return false;
  const int pieces = p.r / 8, columns = kOneWaves * 64 * (8 / pieces);
  return (long)(p.n < p.S ? p.n : p.S) * ((p.N + columns - 1) / columns) * pieces <= 512;
}

template <int PIECES, typename XT, typename YT>
static void run_one(const LoraProblem& p, const Plan& c, hipStream_t stream) {
  constexpr int kColumns = kOneWaves * 64 * Columns<PIECES, YT>::U;
  const int groups = groups_of(p, c.rows);
  one_launch_kernel<PIECES, XT, YT>
      <<<dim3((p.N + kColumns - 1) / kColumns, grid_y(groups)), kOneWaves * 64, 0, stream>>>(
          p, c, groups);
}

template <typename XT, typename YT>
static hipError_t run(const LoraProblem& p, const Plan& c, hipStream_t stream) {
  if (one_launch(p, c)) {
    if (p.r == 8) run_one<1, XT, YT>(p, c, stream);
    else if (p.r == 16) run_one<2, XT, YT>(p, c, stream);
    else if (p.r == 24) run_one<3, XT, YT>(p, c, stream);
    else run_one<4, XT, YT>(p, c, stream);
    return hipGetLastError();
  }
  run_shrink<XT>(p, c, stream);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  run_expand<YT>(p, c, stream);
  return hipGetLastError();
}

}  // namespace lora

size_t lora_workspace_bytes(int S, int n, int K, int r, int block_m) {
  (void)n, (void)block_m;
  // slices * S <= max(S, kSliceRows): 512 / (S / 32) slices at most. Stated so
  // that a workspace for some batch holds for every smaller one.
  const long few = (long)S * lora::max_slices(K);
  const long rows = few < lora::kSliceRows ? few : S > lora::kSliceRows ? S : lora::kSliceRows;
  return ((size_t)rows * r * sizeof(float) + 255) / 256 * 256;
}

hipError_t launch_lora_add(const LoraProblem& p, hipStream_t stream) {
  const lora::Plan c = lora::plan_of(p);
  if (p.x_dtype == MOE_DTYPE_BF16)
    return p.y_dtype == MOE_DTYPE_BF16 ? lora::run<uint16_t, uint16_t>(p, c, stream)
                                       : lora::run<uint16_t, float>(p, c, stream);
  return p.y_dtype == MOE_DTYPE_BF16 ? lora::run<float, uint16_t>(p, c, stream)
                                     : lora::run<float, float>(p, c, stream);
}

}  // namespace moe
