// Norms around the expert FFN: before it (residual add, RMS norm) and after it
// (top-k combine, gated shared expert, RMS norm, residual add, next norm).
//
// Every kernel is one pass: a row is held in registers as fp32 from its loads
// to its stores, so each input is read once and each output written once, and
// the only other work is one (norm_in) or up to two (norm_out) sums of squares
// per row. Bound by HBM: 2 bytes per bf16 element and stream; for norm_out the
// k expert rows per token are the largest of them. Measured (captured into a
// graph): norm_in 4096 x 4096 bf16 with residual 21.4 us = 6.3 TB/s, 16 x 4096
// 2.7 us; norm_out 4096 x top-8 x 4096 bf16, everything on, 61.3 us = 6.6 TB/s,
// 64 x top-8 x 7168 fp32 7.9 us (a row per CU: 64 of them, 330 KB each),
// 16 x top-8 x 4096 bf16 3.8 us.
//
// W waves serve a row: thread i of the row's 64 W holds the vectors i,
// i + 64 W, ... of VEC elements, NV of them. VEC is what 16 bytes of the largest
// input hold (y; x of norm_in): with 32 bytes of fp32 to a lane a load of 16
// would touch every other piece of a line.
#include <type_traits>

#include "../../include/moe.h"
#include "moe_common.h"
#include "moe_launch.h"
#include "moe_rows.h"

namespace moe {
namespace norm {

using namespace rows;

template <int NV, int VEC>
__device__ __forceinline__ float sum_squares(const float (&v)[NV][VEC]) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int q = 0; q < VEC; ++q) s += v[i][q] * v[i][q];
  return s;
}

// The row this thread works on: W > 1 waves: one row per workgroup; W = 1:
// a row per wave, four to a workgroup. Workgroups lie in a grid of kGridX
// columns (a launch counts its threads in 32 bits along a dimension).
constexpr int kGridX = 1 << 20;
template <int W>
__device__ __forceinline__ int my_row() {
  const int group = blockIdx.y * kGridX + blockIdx.x;
  if constexpr (W == 1)
    return __builtin_amdgcn_readfirstlane(group * 4 + (threadIdx.x >> 6));
  else
    return group;
}

template <int W, int NV, int VEC, typename IO>
__global__ __launch_bounds__(W == 1 ? 256 : W * 64) void norm_in_kernel(NormInProblem p) {
  __shared__ float red[W];
  const int row = my_row<W>();
  if (row >= p.T) return;  // whole waves, and W = 1 has no barrier
  const Place<W, NV> c(p.H / VEC);
  const size_t base = (size_t)row * p.H;
  Vec<IO, VEC> xr[NV], rr[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) xr[i] = load_vec<IO, VEC>((const IO*)p.x + base + c.at[i] * VEC);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    rr[i] = Vec<IO, VEC>{};
    if (p.residual) rr[i] = load_vec<IO, VEC>((const IO*)p.residual + base + c.at[i] * VEC);
  }
  Vec<float, VEC> w[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    w[i] = load_vec<float, VEC>(p.weight + c.at[i] * VEC);
    keep_vec<IO, VEC>(xr[i], c.mask[i]);
    keep_vec<IO, VEC>(rr[i], c.mask[i]);
  }
  float s[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int q = 0; q < VEC; ++q)
      s[i][q] = p.alpha * elem<IO, VEC>(xr[i], q) + elem<IO, VEC>(rr[i], q);
  const float ms = row_sum<W>(sum_squares<NV, VEC>(s), red) / (float)p.H;
  const float inv = 1.0f / sqrtf(ms + p.eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (c.mask[i]) {
      const size_t at = base + c.at[i] * VEC;
      if (p.residual_out) store_vec<IO, VEC>((IO*)p.residual_out + at, s[i]);
      float o[VEC];
#pragma unroll
      for (int q = 0; q < VEC; ++q) o[q] = s[i][q] * inv * elem<float, VEC>(w[i], q);
      store_vec<IO, VEC>((IO*)p.out + at, o);
    }
  }
}

// y rows of a token loaded together: as many as fill 64 registers, at most 8.
template <int NV, int VEC, typename YT>
constexpr int batch() {
  constexpr int regs = NV * VEC * (int)sizeof(YT) / 4;  // of one row
  return regs >= 64 ? 1 : regs <= 8 ? 8 : 64 / regs;
}

template <int W, int NV, int VEC, bool NT, typename YT, typename IO>
__global__ __launch_bounds__(W == 1 ? 256 : W * 64) void norm_out_kernel(NormOutProblem p) {
  constexpr int B = batch<NV, VEC, YT>();
  __shared__ float red[2][W];
  const int row = my_row<W>();
  if (row >= p.T) return;  // whole waves, and W = 1 has no barrier
  const Place<W, NV> c(p.H / VEC);
  const size_t base = (size_t)row * p.H;
  // what does not depend on the routing is loaded first
  Vec<IO, VEC> res[NV], sh[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    res[i] = sh[i] = Vec<IO, VEC>{};
    if (p.residual) res[i] = load_vec<IO, VEC>((const IO*)p.residual + base + c.at[i] * VEC);
    if (p.shared) sh[i] = load_vec<IO, VEC>((const IO*)p.shared + base + c.at[i] * VEC);
  }
  // (the weights of the norms too where a row is one vector per thread)
  constexpr bool kEarly = NV == 1;
  Vec<float, VEC> w1[NV], w2[NV];
  auto load_weight = [&](const float* from, Vec<float, VEC>(&to)[NV]) {
#pragma unroll
    for (int i = 0; i < NV; ++i) to[i] = load_vec<float, VEC>(from + c.at[i] * VEC);
  };
  if (kEarly && p.weight) load_weight(p.weight, w1);
  if (kEarly && p.next) load_weight(p.next_weight, w2);
  float v[NV][VEC] = {};
  // the combine, 64 slots at a time: lane l holds slot l's id and weight, and
  // the slots of other shards are left out without reading their rows
  const int lane = threadIdx.x & 63;
  for (int j0 = 0; j0 < p.k; j0 += 64) {
    const int j = j0 + lane;
    bool mine = j < p.k;
    float wl = 1.f;
    if (mine) {
      const size_t s = (size_t)row * p.k + j;
      if (p.topk_weights) wl = p.topk_weights[s];
      if (p.topk_ids) mine = (unsigned)p.topk_ids[s] < (unsigned)p.E;
    }
    uint64_t left = __ballot(mine);
    // B slots; where fewer are left the last one again, as zeros (its weight too,
    // which may be infinite). Full batches without that: 61.1 us of the largest case
    // above instead of 68.4.
    auto batch_of = [&](auto full) {
      constexpr bool kFull = decltype(full)::value;
      int u[B], some = 0;
      uint32_t keep[B];
#pragma unroll
      for (int q = 0; q < B; ++q) {
        keep[q] = kFull || left ? ~0u : 0u;
        if (kFull || left) some = __builtin_ctzll(left);
        left &= left - 1;
        u[q] = some;
      }
      Vec<YT, VEC> r[B][NV];
#pragma unroll
      for (int q = 0; q < B; ++q) {
        const YT* yr = (const YT*)p.y + ((size_t)row * p.k + j0 + u[q]) * p.H;
#pragma unroll
        for (int i = 0; i < NV; ++i) r[q][i] = load_vec<YT, VEC, NT>(yr + c.at[i] * VEC);
      }
#pragma unroll
      for (int q = 0; q < B; ++q) {
        const float wj =
            __uint_as_float(__builtin_amdgcn_readlane(__float_as_int(wl), u[q]) & keep[q]);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          keep_vec<YT, VEC>(r[q][i], keep[q] & c.mask[i]);
#pragma unroll
          for (int e = 0; e < VEC; ++e) v[i][e] += wj * elem<YT, VEC>(r[q][i], e);
        }
      }
    };
    for (int n = __builtin_popcountll(left); n >= B; n -= B) batch_of(std::true_type{});
    if (left) batch_of(std::false_type{});
  }
  if (p.shared) {
    const float g = p.gate ? 1.0f / (1.0f + expf(-p.gate[row])) : 1.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      keep_vec<IO, VEC>(sh[i], c.mask[i]);
#pragma unroll
      for (int q = 0; q < VEC; ++q) v[i][q] += g * elem<IO, VEC>(sh[i], q);
    }
  }
  if (p.weight) {
    if (!kEarly) load_weight(p.weight, w1);
    const float ms = row_sum<W>(sum_squares<NV, VEC>(v), red[0]) / (float)p.H;
    const float inv = 1.0f / sqrtf(ms + p.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      keep_vec<float, VEC>(w1[i], c.mask[i]);
#pragma unroll
      for (int q = 0; q < VEC; ++q) v[i][q] = v[i][q] * inv * elem<float, VEC>(w1[i], q);
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    keep_vec<IO, VEC>(res[i], c.mask[i]);
#pragma unroll
    for (int q = 0; q < VEC; ++q) v[i][q] = p.scale * v[i][q] + elem<IO, VEC>(res[i], q);
    if (c.mask[i]) store_vec<IO, VEC>((IO*)p.out + base + c.at[i] * VEC, v[i]);
  }
  if (p.next) {
    if (!kEarly) load_weight(p.next_weight, w2);
    const float ms = row_sum<W>(sum_squares<NV, VEC>(v), red[1]) / (float)p.H;
    const float inv = 1.0f / sqrtf(ms + p.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float o[VEC];
#pragma unroll
      for (int q = 0; q < VEC; ++q) o[q] = v[i][q] * inv * elem<float, VEC>(w2[i], q);
      if (c.mask[i]) store_vec<IO, VEC>((IO*)p.next + base + c.at[i] * VEC, o);
    }
  }
}

// y rows that together pass this are read around the caches: 268 MB of them
// leave nothing in the 256 MB cache that a later kernel would find, and read so
// they take 61.2 us instead of 75.7 (4096 x 8 rows of 4096 bf16, everything on; 64.2
// instead of 79.5 right after another kernel has written them). 15 MB that FC2 has
// just written are still there, and take 12.1 us instead of 10.1; 59 MB 16.9 instead
// of 15.7. From 92 to 161 MB the better side depends on the shape and on what ran
// before: 134 MB in turn with others 33.6 instead of 37.4, just written 43.7 and 42.4.
constexpr size_t kStreamBytes = (size_t)128 << 20;

// Calls f(W, NV) as compile-time constants for rows of H elements: the fewest
// waves that hold a row with one vector per thread, where they are at most 8, then
// two vectors per thread: half the waves of a row leave room for twice the rows on
// a CU. Rows of 513 .. 1024 vectors with two instead of one: norm_in 8192 x 7168
// bf16 84 us instead of 90, 16 x 4096 fp32 2.97 instead of 2.87; norm_out 4096 x
// top-8 x 7168 bf16 119 instead of 137, 16 x top-8 5.6 instead of 6.0.
template <int V>
struct Int {
  static constexpr int value = V;
};
template <int VEC, typename F>
static void by_row_length(int H, F f) {
  const int vecs = H / VEC;
  if (vecs <= 64) f(Int<1>{}, Int<1>{});
  else if (vecs <= 128) f(Int<1>{}, Int<2>{});
  else if (vecs <= 256) f(Int<4>{}, Int<1>{});
  else if (vecs <= 512) f(Int<8>{}, Int<1>{});
  else if (vecs <= 1024) f(Int<8>{}, Int<2>{});
  else if (VEC == 8 || vecs <= 2048) f(Int<16>{}, Int<2>{});
  else if constexpr (VEC == 4) f(Int<16>{}, Int<4>{});
}

template <int W>
static dim3 grid_of(int T) {
  const int groups = W == 1 ? (T + 3) / 4 : T;
  return dim3(groups < kGridX ? groups : kGridX, (groups + kGridX - 1) / kGridX);
}

template <int VEC, typename IO>
static void run_in(const NormInProblem& p, hipStream_t stream) {
  by_row_length<VEC>(p.H, [&](auto w, auto nv) {
    constexpr int W = decltype(w)::value, NV = decltype(nv)::value;
    norm_in_kernel<W, NV, VEC, IO>
        <<<grid_of<W>(p.T), W == 1 ? 256 : W * 64, 0, stream>>>(p);
  });
}

template <int VEC, typename YT, typename IO>
static void run_out(const NormOutProblem& p, hipStream_t stream) {
  by_row_length<VEC>(p.H, [&](auto w, auto nv) {
    constexpr int W = decltype(w)::value, NV = decltype(nv)::value;
    const dim3 grid = grid_of<W>(p.T);
    const int threads = W == 1 ? 256 : W * 64;
    if ((size_t)p.T * p.k * p.H * sizeof(YT) > kStreamBytes)
      norm_out_kernel<W, NV, VEC, true, YT, IO><<<grid, threads, 0, stream>>>(p);
    else
      norm_out_kernel<W, NV, VEC, false, YT, IO><<<grid, threads, 0, stream>>>(p);
  });
}

}  // namespace norm

hipError_t launch_norm_in(const NormInProblem& p, hipStream_t stream) {
  if (p.dtype == MOE_DTYPE_BF16) norm::run_in<8, uint16_t>(p, stream);
  else norm::run_in<4, float>(p, stream);
  return hipGetLastError();
}

hipError_t launch_norm_out(const NormOutProblem& p, hipStream_t stream) {
  if (p.dtype == MOE_DTYPE_BF16) {
    if (p.y_dtype == MOE_DTYPE_BF16) norm::run_out<8, uint16_t, uint16_t>(p, stream);
    else norm::run_out<4, float, uint16_t>(p, stream);
  } else {
    if (p.y_dtype == MOE_DTYPE_BF16) norm::run_out<8, uint16_t, float>(p, stream);
    else norm::run_out<4, float, float>(p, stream);
  }
  return hipGetLastError();
}

}  // namespace moe
