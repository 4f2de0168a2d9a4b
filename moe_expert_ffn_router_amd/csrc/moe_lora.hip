// Low-rank adapters of many requests beside a shared projection:
// out[s] = y[s] + scale[g] * b[g] (a[g] x[s]) for the rows s of adapter g.
//
// Two launches over the aligned row lists, both bound by memory (2 r flops per
// element of x, y, a or b): the shrink z = a x, split over K, leaves fp32
// partial sums in the workspace (r numbers per row: nothing next to x and y);
// the expansion adds them up and works b into the rows of y.
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
  int slices;      // of K
  int rows_a, rows_b;  // rows of a group of the shrink, of the expansion
  int groups_a, groups_b;  // of all blocks
};

// A group of `rows` consecutive positions of a block (a power of two at most
// block_m): whether it has a row, its adapter and first position.
struct Group {
  int adapter;
  long pos;
  bool live;
};
__device__ __forceinline__ Group group_at(const LoraProblem& p, const Plan& c, long g, int rows) {
  Group r{0, g * rows, false};
  if (r.pos >= p.num_padded[0]) return r;
  r.adapter = p.block_adapter[r.pos >> c.log2m];
  // a block's rows come first in it
  r.live = (unsigned)p.sorted_ids[r.pos] < (unsigned)p.S && (unsigned)r.adapter < (unsigned)p.n;
  return r;
}

// ---------------------------------------------------------------- shrink ---
// A workgroup: 16 MT rows of one adapter, 16 NT of its ranks, one slice of K.
constexpr int kShrinkWaves = 8;

template <int MT, int NT, typename XT>
__global__ __launch_bounds__(kShrinkWaves * 64) void shrink_kernel(LoraProblem p, Plan c,
                                                                   int rank_tiles) {
  constexpr int NW = kShrinkWaves;
  __shared__ __align__(16) char lds[skinny::lds_bytes<MT, NT, NW, XT, uint16_t>()];
  const int slice = blockIdx.x / rank_tiles, q0 = blockIdx.x % rank_tiles * NT * 16;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int chunks = (p.K + kChunk - 1) / kChunk;
  const int first = (int)((long)chunks * slice / c.slices);
  const int end = (int)((long)chunks * (slice + 1) / c.slices);
  float* z = (float*)p.workspace + (size_t)slice * p.S * p.r;
  for (int gi = blockIdx.y; gi < c.groups_a; gi += gridDim.y) {
    const Group g = group_at(p, c, gi, c.rows_a);
    if (!g.live) continue;  // the whole workgroup
    const int some = p.sorted_ids[g.pos];
    skinny::Product<MT, NT, XT, uint16_t> m;
    m.lds = lds + wave * m.kLdsBytes;
    m.x.set([&](int i) {
      int row = i < c.rows_a ? p.sorted_ids[g.pos + i] : some;
      if ((unsigned)row >= (unsigned)p.S) row = some;
      return (const XT*)p.x + (size_t)row * p.ldx;
    });
    const uint16_t* a = p.a + (size_t)g.adapter * p.r * p.K;
    m.w.set([&](int i) { return a + (size_t)min(q0 + i, p.r - 1) * p.K; });
    m.clear();
    // two chunks in flight where their registers allow it
    constexpr int D = MT * (int)sizeof(XT) / 2 + NT <= 5 ? 2 : 1;
    m.template accumulate<D>(p.K, first + wave, end, NW);
    skinny::reduce_waves<MT, NT, NW>(m.acc, lds, [&](int j, int i, int lane, f32x4 s) {
      const int at = i * 16 + (lane & 15), q = q0 + j * 16 + (lane >> 4) * 4;
      if (at >= c.rows_a || q >= p.r) return;
      const int row = p.sorted_ids[g.pos + at];
      if ((unsigned)row < (unsigned)p.S) *(f32x4*)(z + (size_t)row * p.r + q) = s;
    });
    __syncthreads();  // the sums are read before the next group's chunks
  }
}

// ---------------------------------------------------------------- expand ---
// A wave: TT tiles of 16 rows, 16 J columns. D = z (rows) x b (columns) with
// column 16 J u + J cc + j in column cc of tile j: a lane then holds J
// consecutive columns of 4 rows, 16 bytes of y, and 16 lanes 256 bytes of a row.
// STEPS: MFMAs over the rank, 32 of it each. A rank of 8 or 16 fills only one or
// two of an MFMA's four k-groups: there one load brings PACK = 4 or 2 tiles of
// b, a tile to a k-group (or two), and a tile's fragment is the load with the
// others' groups zero (z is the same in every group).
template <int J, int STEPS, int PACK, int TT, typename YT>
__global__ __launch_bounds__(256) void expand_kernel(LoraProblem p, Plan c) {
  // z enters as bf16 planes: exactly (3) for fp32 rows, to 2^-16 (2) for bf16
  // rows, whose own rounding is 2^-8
  constexpr int kPlanes = sizeof(YT) == 2 ? 2 : 3;
  constexpr int kWords = J * (int)sizeof(YT) / 4;  // 32-bit words of y of a lane and row
  const int lane = threadIdx.x & 63, cc = lane & 15, g4 = lane >> 4;
  const int n0 = (blockIdx.x * 4 + (threadIdx.x >> 6)) * 16 * J;
  if (n0 >= p.N) return;  // whole waves
  const int n = n0 + cc * J;
  constexpr int kGroups = 4 / PACK;  // k-groups of a tile
  const int kg = PACK > 1 ? g4 % kGroups : g4;
  const size_t zslice = (size_t)p.S * p.r;
  for (int gi = blockIdx.y; gi < c.groups_b; gi += gridDim.y) {
    const Group g = group_at(p, c, gi, c.rows_b);
    if (!g.live) continue;
    const float scale = p.scale ? p.scale[g.adapter] : 1.f;
    // the rows: as z's row (lane & 15) and as the 4 of D this lane holds
    int zrow[TT], row[TT][4];
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      zrow[t] = -1;
      if (t * 16 + cc < c.rows_b) zrow[t] = p.sorted_ids[g.pos + t * 16 + cc];
#pragma unroll
      for (int i = 0; i < 4; ++i) row[t][i] = __shfl(zrow[t], g4 * 4 + i);
    }
    u32x4 bq[STEPS][J];
    const uint16_t* b = p.b + (size_t)g.adapter * p.N * p.r;
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
      for (int j = 0; j < J; j += PACK) {
        const int nb = min(n + j + (PACK > 1 ? g4 / kGroups : 0), p.N - 1);
        u32x4 v = {0, 0, 0, 0};
        if (s * 32 + kg * 8 < p.r) v = *(const u32x4*)(b + (size_t)nb * p.r + s * 32 + kg * 8);
#pragma unroll
        for (int pk = 0; pk < PACK; ++pk)
          bq[s][j + pk] = PACK == 1 || g4 / kGroups == pk ? v : u32x4{0, 0, 0, 0};
      }
    uint32_t yw[TT][4][kWords];
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if ((unsigned)row[t][i] < (unsigned)p.S && n < p.N) {
          const u32x4* yp = (const u32x4*)((const YT*)p.y + (size_t)row[t][i] * p.ldy + n);
#pragma unroll
          for (int q = 0; q < kWords; q += 4) {
            const u32x4 v = yp[q / 4];
#pragma unroll
            for (int e = 0; e < 4; ++e) yw[t][i][q + e] = v[e];
          }
        }
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      f32x4 acc[J];
#pragma unroll
      for (int j = 0; j < J; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        float zv[8] = {};
        if ((unsigned)zrow[t] < (unsigned)p.S && s * 32 + kg * 8 < p.r) {
          const float* zp = (const float*)p.workspace + (size_t)zrow[t] * p.r + s * 32 + kg * 8;
          for (int k = 0; k < c.slices; ++k) {
            const f32x4 lo = *(const f32x4*)(zp + k * zslice);
            const f32x4 hi = *(const f32x4*)(zp + k * zslice + 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              zv[e] += lo[e];
              zv[4 + e] += hi[e];
            }
          }
        }
        bf16x8 zf[kPlanes];
        skinny::split8<kPlanes>(zv, zf);
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
          for (int q = kPlanes - 1; q >= 0; --q)
            acc[j] = mfma_bf16(zf[q], __builtin_bit_cast(bf16x8, bq[s][j]), acc[j]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if ((unsigned)row[t][i] < (unsigned)p.S && n < p.N) {
          YT* op = (YT*)p.out + (size_t)row[t][i] * p.ldo + n;
          uint32_t o[kWords];
#pragma unroll
          for (int q = 0; q < kWords; ++q) {
            if constexpr (sizeof(YT) == 2) {
              const float lo = bf16_bits_to_f32(yw[t][i][q] & 0xffffu) + scale * acc[2 * q][i];
              const float hi = __uint_as_float(yw[t][i][q] & 0xffff0000u) + scale * acc[2 * q + 1][i];
              o[q] = f32_to_bf16_rne(lo) | (f32_to_bf16_rne(hi) << 16);
            } else {
              o[q] = __float_as_uint(__uint_as_float(yw[t][i][q]) + scale * acc[q][i]);
            }
          }
          if constexpr (kWords == 2) {
            *(u32x2*)op = u32x2{o[0], o[1]};
          } else {
#pragma unroll
            for (int q = 0; q < kWords; q += 4)
              *(u32x4*)(op + q * 4 / (int)sizeof(YT)) = u32x4{o[q], o[q + 1], o[q + 2], o[q + 3]};
          }
        }
    }
  }
}

// ------------------------------------------------------------------ host ---

// Rows of a call: up to kSliceRows of z (in slices of K and rows) are kept.
constexpr long kSliceRows = 8192;
constexpr int kMaxSlices = 16;

static int max_slices(int K) {
  const int chunks = (K + kChunk - 1) / kChunk;
  const int most = chunks / kShrinkWaves;  // a chunk for every wave
  return most < 1 ? 1 : most > kMaxSlices ? kMaxSlices : most;
}

static Plan plan_of(const LoraProblem& p) {
  Plan c{};
  while ((1 << c.log2m) < p.block_m) ++c.log2m;
  const bool many = (long)p.S >= 32L * p.n;  // rows of an adapter on average
  const int rows = p.block_m < 16 ? p.block_m : many && p.block_m >= 32 ? 32 : 16;
  c.rows_a = p.r <= 64 ? rows : rows < 16 ? rows : 16;
  c.rows_b = rows;
  const long cap = (long)align_capacity(p.S, p.n, p.block_m);
  c.groups_a = (int)(cap / c.rows_a);
  c.groups_b = (int)(cap / c.rows_b);
  // slices of K until some 512 workgroups have work: every adapter in use and
  // every 16 rows give one
  const long groups = p.S / 16 + (p.n < p.S ? p.n : p.S) / 2 + 1;
  const int want = (int)(512 / groups), most = max_slices(p.K);
  c.slices = want < 1 ? 1 : want > most ? most : want;
  return c;
}

template <int MT, int NT, typename XT>
static void shrink(const LoraProblem& p, const Plan& c, hipStream_t stream) {
  const int rank_tiles = (p.r + NT * 16 - 1) / (NT * 16);
  const dim3 grid(c.slices * rank_tiles, c.groups_a < 65535 ? c.groups_a : 65535);
  shrink_kernel<MT, NT, XT><<<grid, kShrinkWaves * 64, 0, stream>>>(p, c, rank_tiles);
}

template <typename XT>
static void run_shrink(const LoraProblem& p, const Plan& c, hipStream_t stream) {
  if (p.r > 64) shrink<1, 8, XT>(p, c, stream);
  else if (p.r > 32) c.rows_a == 32 ? shrink<2, 4, XT>(p, c, stream) : shrink<1, 4, XT>(p, c, stream);
  else if (p.r > 16) c.rows_a == 32 ? shrink<2, 2, XT>(p, c, stream) : shrink<1, 2, XT>(p, c, stream);
  else c.rows_a == 32 ? shrink<2, 1, XT>(p, c, stream) : shrink<1, 1, XT>(p, c, stream);
}

template <int J, int STEPS, int PACK, typename YT>
static void expand(const LoraProblem& p, const Plan& c, hipStream_t stream) {
  const int units = (p.N + 16 * J - 1) / (16 * J);
  const dim3 grid((units + 3) / 4, c.groups_b < 65535 ? c.groups_b : 65535);
  if (c.rows_b == 32) expand_kernel<J, STEPS, PACK, 2, YT><<<grid, 256, 0, stream>>>(p, c);
  else expand_kernel<J, STEPS, PACK, 1, YT><<<grid, 256, 0, stream>>>(p, c);
}

template <typename YT>
static void run_expand(const LoraProblem& p, const Plan& c, hipStream_t stream) {
  constexpr int J = 16 / sizeof(YT);  // 16 bytes of a row per lane
  if (p.r == 8) expand<J, 1, 4, YT>(p, c, stream);
  else if (p.r == 16) expand<J, 1, 2, YT>(p, c, stream);
  else if (p.r <= 32) expand<J, 1, 1, YT>(p, c, stream);
  else if (p.r <= 64) expand<J, 2, 1, YT>(p, c, stream);
  else if (p.r <= 128) expand<4, 4, 1, YT>(p, c, stream);
  else expand<4, 8, 1, YT>(p, c, stream);
}

}  // namespace lora

size_t lora_workspace_bytes(int S, int n, int K, int r, int block_m) {
  (void)n, (void)block_m;
  // slices * S <= max(S, kSliceRows): 512 / (S / 16) slices at most. Stated so
  // that a workspace for some batch holds for every smaller one.
  const long few = (long)S * lora::max_slices(K);
  const long rows = few < lora::kSliceRows ? few : S > lora::kSliceRows ? S : lora::kSliceRows;
  return ((size_t)rows * r * sizeof(float) + 255) / 256 * 256;
}

hipError_t launch_lora_add(const LoraProblem& p, hipStream_t stream) {
  const lora::Plan c = lora::plan_of(p);
  if (p.x_dtype == MOE_DTYPE_BF16) lora::run_shrink<uint16_t>(p, c, stream);
  else lora::run_shrink<float>(p, c, stream);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  if (p.y_dtype == MOE_DTYPE_BF16) lora::run_expand<uint16_t>(p, c, stream);
  else lora::run_expand<float>(p, c, stream);
  return hipGetLastError();
}

}  // namespace moe
