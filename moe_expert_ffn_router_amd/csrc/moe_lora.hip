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
  int slices;  // of K
  int rows;    // of a group: consecutive positions of a block, at most 64
  int groups;  // of all blocks
};

// A group: its adapter, first position and this lane's row (lane l: position
// pos + l; -1 where there is none). A block's rows come first in it, so count
// rows are in lanes 0 .. count - 1.
struct Group {
  int adapter, count, row;
};
__device__ __forceinline__ Group group_at(const LoraProblem& p, const Plan& c, long g) {
  const long pos = g * c.rows;
  const int lane = threadIdx.x & 63;
  // the loads do not wait for each other: past *num_padded the lists still
  // hold what the alignment wrote there
  const int padded = p.num_padded[0];
  Group r;
  r.adapter = p.block_adapter[pos >> c.log2m];
  r.row = p.sorted_ids[pos + min(lane, c.rows - 1)];
  if (lane >= c.rows || (unsigned)r.row >= (unsigned)p.S || pos >= padded ||
      (unsigned)r.adapter >= (unsigned)p.n)
    r.row = -1;
  r.count = __builtin_popcountll(__ballot(r.row >= 0));
  return r;
}
// The row of the group's position i, or of its last row past the end.
__device__ __forceinline__ int row_at(const Group& g, int i) {
  return __shfl(g.row, min(i, g.count - 1));
}

// ---------------------------------------------------------------- shrink ---
// A workgroup: 16 NT ranks of a group's adapter, one slice of K, 16 MT rows at a
// time.
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
  for (int gi = blockIdx.y; gi < c.groups; gi += gridDim.y) {
    const Group g = group_at(p, c, gi);
    const uint16_t* a = p.a + (size_t)g.adapter * p.r * p.K;
    for (int t = 0; t < g.count; t += 16 * MT) {  // the whole workgroup
      skinny::Product<MT, NT, XT, uint16_t> m;
      m.lds = lds + wave * m.kLdsBytes;
      m.x.set([&](int i) { return (const XT*)p.x + (size_t)row_at(g, t + i) * p.ldx; });
      m.w.set([&](int i) { return a + (size_t)min(q0 + i, p.r - 1) * p.K; });
      m.clear();
      // two chunks in flight where their registers allow it
      constexpr int D = MT * (int)sizeof(XT) / 2 + NT <= 5 ? 2 : 1;
      m.template accumulate<D>(p.K, first + wave, end, NW);
      skinny::reduce_waves<MT, NT, NW>(m.acc, lds, [&](int j, int i, int lane, f32x4 s) {
        const int at = t + i * 16 + (lane & 15), q = q0 + j * 16 + (lane >> 4) * 4;
        const int row = row_at(g, at);
        if (at < g.count && q < p.r) *(f32x4*)(z + (size_t)row * p.r + q) = s;
      });
      __syncthreads();  // the sums are read before the next rows' chunks
    }
  }
}

// ---------------------------------------------------------------- expand ---
// A wave: 16 J columns of a group, 16 rows at a time with the next ones' y and z
// loaded ahead. D = z (rows) x b (columns) with column 16 J u + J cc + j in
// column cc of tile j: a lane then holds J consecutive columns of 4 rows, 16
// bytes of y, and 16 lanes 256 bytes of a row.
// STEPS: MFMAs over the rank, 32 of it each. A rank of 8 or 16 fills only one or
// two of an MFMA's four k-groups: there one load brings PACK = 4 or 2 tiles of
// b, a tile to a k-group (or two), and a tile's fragment is the load with the
// others' groups zero (z is the same in every group).
template <int J, int STEPS, typename YT>
struct Rows16 {
  static constexpr int kWords = J * (int)sizeof(YT) / 4;  // 32-bit words of y, lane and row
  float z[STEPS][8];
  uint32_t y[4][kWords];

  // rows 16 t .. of the group; zq: this lane's first rank, n: its first column
  __device__ __forceinline__ void load(const LoraProblem& p, const Plan& c, const Group& g, int t,
                                       int zq, int n) {
    const int lane = threadIdx.x & 63;
    const float* zp = (const float*)p.workspace + (size_t)row_at(g, t * 16 + (lane & 15)) * p.r;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      // past the rank: any values, b is zero there (clamped to stay in the row)
      const f32x4* q = (const f32x4*)(zp + min(s * 32 + zq, p.r - 8));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        z[s][e] = q[0][e];
        z[s][4 + e] = q[1][e];
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const YT* yp = (const YT*)p.y + (size_t)row_at(g, t * 16 + (lane >> 4) * 4 + i) * p.ldy + n;
      if constexpr (kWords == 2) {
        const u32x2 v = *(const u32x2*)yp;
        y[i][0] = v[0];
        y[i][1] = v[1];
      } else {
#pragma unroll
        for (int q = 0; q < kWords; q += 4) {
          const u32x4 v = ((const u32x4*)yp)[q / 4];
#pragma unroll
          for (int e = 0; e < 4; ++e) y[i][q + e] = v[e];
        }
      }
    }
    for (int k = 1; k < c.slices; ++k) {
      zp += (size_t)p.S * p.r;
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        const f32x4* q = (const f32x4*)(zp + min(s * 32 + zq, p.r - 8));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          z[s][e] += q[0][e];
          z[s][4 + e] += q[1][e];
        }
      }
    }
  }
};

template <int J, int STEPS, int PACK, typename YT>
__global__ __launch_bounds__(256) void expand_kernel(LoraProblem p, Plan c) {
  // z enters as bf16 planes: exactly (3) for fp32 rows, to 2^-16 (2) for bf16
  // rows, whose own rounding is 2^-8
  constexpr int kPlanes = sizeof(YT) == 2 ? 2 : 3;
  constexpr int kWords = Rows16<J, STEPS, YT>::kWords;
  const int lane = threadIdx.x & 63, cc = lane & 15, g4 = lane >> 4;
  const int n0 = (blockIdx.x * 4 + (threadIdx.x >> 6)) * 16 * J;
  if (n0 >= p.N) return;  // whole waves
  const int n = n0 + cc * J, n_in = min(n, p.N - J);  // N and J: whole groups of J
  constexpr int kGroups = 4 / PACK;  // k-groups of a tile
  const int kq = g4 % kGroups * 8;
  for (int gi = blockIdx.y; gi < c.groups; gi += gridDim.y) {
    const Group g = group_at(p, c, gi);
    if (g.count == 0) continue;
    const float scale = p.scale ? p.scale[g.adapter] : 1.f;
    const uint16_t* b = p.b + (size_t)g.adapter * p.N * p.r;
    u32x4 bq[STEPS][J];
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
      for (int j = 0; j < J; j += PACK) {
        const int q = s * 32 + kq;
        const u32x4 v = *(const u32x4*)(b + (size_t)(n_in + j + g4 / kGroups) * p.r +
                                        min(q, p.r - 8));
#pragma unroll
        for (int pk = 0; pk < PACK; ++pk)
          bq[s][j + pk] = q < p.r && g4 / kGroups == pk ? v : u32x4{0, 0, 0, 0};
      }
    Rows16<J, STEPS, YT> now;
    auto work = [&](int t) {
      f32x4 acc[J];
#pragma unroll
      for (int j = 0; j < J; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        bf16x8 zf[kPlanes];
        skinny::split8<kPlanes>(now.z[s], zf);
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
          for (int q = kPlanes - 1; q >= 0; --q)
            acc[j] = mfma_bf16(zf[q], __builtin_bit_cast(bf16x8, bq[s][j]), acc[j]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = t * 16 + g4 * 4 + i, row = row_at(g, at);
        uint32_t o[kWords];
#pragma unroll
        for (int q = 0; q < kWords; ++q) {
          const uint32_t w = now.y[i][q];
          if constexpr (sizeof(YT) == 2) {
            const float lo = bf16_bits_to_f32(w & 0xffffu) + scale * acc[2 * q][i];
            const float hi = __uint_as_float(w & 0xffff0000u) + scale * acc[2 * q + 1][i];
            o[q] = f32_to_bf16_rne(lo) | (f32_to_bf16_rne(hi) << 16);
          } else {
            o[q] = __float_as_uint(__uint_as_float(w) + scale * acc[q][i]);
          }
        }
        if (at < g.count && n < p.N) {
          YT* op = (YT*)p.out + (size_t)row * p.ldo + n;
          if constexpr (kWords == 2) {
            *(u32x2*)op = u32x2{o[0], o[1]};
          } else {
#pragma unroll
            for (int q = 0; q < kWords; q += 4)
              ((u32x4*)op)[q / 4] = u32x4{o[q], o[q + 1], o[q + 2], o[q + 3]};
          }
        }
      }
    };
    const int tiles = (g.count + 15) / 16;
    now.load(p, c, g, 0, kq, n_in);
    for (int t = 0; t + 1 < tiles; ++t) {
      Rows16<J, STEPS, YT> next;
      next.load(p, c, g, t + 1, kq, n_in);
      work(t);
      now = next;
    }
    work(tiles - 1);
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
  c.rows = p.block_m < 64 ? p.block_m : 64;
  c.groups = (int)(align_capacity(p.S, p.n, p.block_m) / c.rows);
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
  const dim3 grid(c.slices * rank_tiles, c.groups < 65535 ? c.groups : 65535);
  shrink_kernel<MT, NT, XT><<<grid, kShrinkWaves * 64, 0, stream>>>(p, c, rank_tiles);
}

template <typename XT>
static void run_shrink(const LoraProblem& p, const Plan& c, hipStream_t stream) {
  const bool pairs = c.rows >= 32 && (long)p.S >= 32L * p.n;  // rows of an adapter on average
  if (p.r > 32) pairs ? shrink<2, 4, XT>(p, c, stream) : shrink<1, 4, XT>(p, c, stream);
  else if (p.r > 16) pairs ? shrink<2, 2, XT>(p, c, stream) : shrink<1, 2, XT>(p, c, stream);
  else pairs ? shrink<2, 1, XT>(p, c, stream) : shrink<1, 1, XT>(p, c, stream);
}

template <int J, int STEPS, int PACK, typename YT>
static void expand(const LoraProblem& p, const Plan& c, hipStream_t stream) {
  const int units = (p.N + 16 * J - 1) / (16 * J);
  const dim3 grid((units + 3) / 4, c.groups < 65535 ? c.groups : 65535);
  expand_kernel<J, STEPS, PACK, YT><<<grid, 256, 0, stream>>>(p, c);
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
