// Layer norm with the residual add in front of it, and its gradients.
//
// Forward: one pass; a row is held in registers as fp32 from its loads to its stores,
// its mean and then its squares about the mean are summed in turn. Backward: one pass
// over the rows with the sums s as the forward pass stored them: with u = (s - mean) /
// sqrt(var + eps) and g = dout weight,
//   ds = (g - mean(g) - u mean(g u)) / sqrt(var + eps)  [+ dresidual_out]
// takes two sums over the row twice (s and g, then (s - mean)^2 and g (s - mean)); the
// gradients of weight and bias are sums over all rows, which every worker (W waves with
// one row after the other) keeps in registers for its own rows; a workgroup writes its sums
// once, for a second kernel that adds the workgroups' in a fixed order. Bound by HBM, small
// calls by their launches. Measured (captured into a graph), bf16 with residual: forward 16 x
// 4096 2.5 us, 4096 x 4096 22.7 us = 5.9 TB/s; backward 4096 x 4096 39 us (35 = 5.2 TB/s with its
// 16 MB of sums, and 4 the second kernel), 8192 x 7168 120 us = 4.9 TB/s, 4096 x 16384 149, 8192 x
// 1024 18, 100 x 4096 7.6, 16 x 512 3.6; fp32 777 x 1031 forward 3.1 us, backward 11.
#include <algorithm>

#include "../../include/moe.h"
#include "moe_common.h"
#include "moe_launch.h"
#include "moe_rows.h"

namespace moe {
namespace layer_norm {

using namespace rows;

// The forward pass's row of this thread: W > 1 waves: one row per workgroup; W = 1: a row per
// wave, four to a workgroup. Workgroups lie in a grid of kGridX columns (a launch counts its
// threads in 32 bits along a dimension).
constexpr int kGridX = 1 << 20;
template <int W>
__device__ __forceinline__ int my_row() {
  const int group = blockIdx.y * kGridX + blockIdx.x;
  if constexpr (W == 1)
    return __builtin_amdgcn_readfirstlane(group * 4 + (threadIdx.x >> 6));
  else
    return group;
}
template <int W>
static dim3 grid_of(int T) {
  const int groups = W == 1 ? (T + 3) / 4 : T;
  return dim3(std::min(groups, kGridX), (groups + kGridX - 1) / kGridX);
}

template <int W, int NV, int VEC, bool ANY, typename IO>
__global__ __launch_bounds__(W == 1 ? 256 : W * 64) void forward_kernel(LayerNormProblem p) {
  __shared__ float red[2][W];
  const int row = my_row<W>();
  if (row >= p.T) return;  // whole waves, and W = 1 has no barrier
  const Span<W, NV, VEC, ANY> c(p.H, W == 1 ? threadIdx.x & 63 : threadIdx.x);
  const size_t base = (size_t)row * p.H;
  Vec<IO, VEC> xr[NV], rr[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i)
    xr[i] = load_vec<IO, VEC, false, ANY>((const IO*)p.x + base + c.at[i]);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    rr[i] = Vec<IO, VEC>{};
    if (p.residual) rr[i] = load_vec<IO, VEC, false, ANY>((const IO*)p.residual + base + c.at[i]);
  }
  float s[NV][VEC], sum = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int q = 0; q < VEC; ++q) {
      s[i][q] = p.alpha * elem<IO, VEC>(xr[i], q) + elem<IO, VEC>(rr[i], q);
      sum += c.has(i, q) ? s[i][q] : 0.f;
    }
    if (p.residual_out) c.store(i, (IO*)p.residual_out + base, s[i]);
  }
  const float mean = row_sum<W>(sum, red[0]) / (float)p.H;
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int q = 0; q < VEC; ++q) {
      s[i][q] -= mean;
      ss += c.has(i, q) ? s[i][q] * s[i][q] : 0.f;
    }
  const float inv = 1.0f / sqrtf(row_sum<W>(ss, red[1]) / (float)p.H + p.eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    Vec<float, VEC> w, b{};
    if (p.weight) w = load_vec<float, VEC, false, ANY>(p.weight + c.at[i]);
    if (p.bias) b = load_vec<float, VEC, false, ANY>(p.bias + c.at[i]);
    float o[VEC];
#pragma unroll
    for (int q = 0; q < VEC; ++q) {
      o[q] = s[i][q] * inv;
      if (p.weight) o[q] *= elem<float, VEC>(w, q);
      o[q] += elem<float, VEC>(b, q);
    }
    c.store(i, (IO*)p.out + base, o);
  }
}

// Two sums over the W waves of a row at once; `slot` as in row_sum.
template <int W>
__device__ __forceinline__ void row_sums(float& a, float& b, f32x2* slot) {
  a = wave_sum(a);
  b = wave_sum(b);
  if constexpr (W > 1) {
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = f32x2{a, b};
    __syncthreads();
    a = b = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      a += slot[i][0];
      b += slot[i][1];
    }
  }
}

// A worker of W waves takes the rows w, w + workers, ... . W > 1: it is a workgroup; W = 1:
// 16 of them are one. At the end a workgroup's sums for the weight and the bias (16 workers'
// side by side in LDS, added up in order) go to partial[workgroup] ([2, H]), or are the
// gradients where it is the only one. The slots of the two sums over a row are each written
// again only past the other's barrier, when all have read them. (Two workers of 8 waves to a
// workgroup, for half the partials, hold each other up at the barriers: 41.4 us instead of
// 38.8 for 4096 x 4096 bf16.)
template <int W>
constexpr int group_waves() {
  return W == 1 ? 16 : W;
}
template <int W, int NV, int VEC, bool ANY, typename IO>
__global__ __launch_bounds__(group_waves<W>() * 64) void backward_kernel(
    LayerNormBackwardProblem p) {
  constexpr int kWorkers = group_waves<W>() / W, kLength = W * 64 * NV * VEC;
  __shared__ f32x2 red[2][W];
  __shared__ __attribute__((aligned(16))) float sums[2][kWorkers][kWorkers > 1 ? kLength : 1];
  const int mine = kWorkers == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Span<W, NV, VEC, ANY> c(p.H, threadIdx.x - mine * 64);
  Vec<float, VEC> w[NV];
  float dw[NV][VEC] = {}, db[NV][VEC] = {};
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (p.weight) w[i] = load_vec<float, VEC, false, ANY>(p.weight + c.at[i]);
  const float n = 1.0f / (float)p.H;
  auto weighted = [&](float g, int i, int q) __attribute__((always_inline)) {
    return p.weight ? g * elem<float, VEC>(w[i], q) : g;
  };
  for (int row = blockIdx.x * kWorkers + mine; row < p.T; row += gridDim.x * kWorkers) {
    const size_t base = (size_t)row * p.H;
    Vec<IO, VEC> sr[NV], gr[NV], rr[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      sr[i] = load_vec<IO, VEC, false, ANY>((const IO*)p.s + base + c.at[i]);
      gr[i] = load_vec<IO, VEC, false, ANY>((const IO*)p.dout + base + c.at[i]);
      rr[i] = Vec<IO, VEC>{};
      if (p.dresidual_out)
        rr[i] = load_vec<IO, VEC, false, ANY>((const IO*)p.dresidual_out + base + c.at[i]);
    }
    float s[NV][VEC], g[NV][VEC], sum = 0.f, sg = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int q = 0; q < VEC; ++q) {
        s[i][q] = c.has(i, q) ? elem<IO, VEC>(sr[i], q) : 0.f;
        g[i][q] = c.has(i, q) ? elem<IO, VEC>(gr[i], q) : 0.f;
        db[i][q] += g[i][q];
        sum += s[i][q];
        sg += weighted(g[i][q], i, q);
      }
    }
    row_sums<W>(sum, sg, red[0]);
    const float mean = sum * n;
    float ss = 0.f, sgs = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int q = 0; q < VEC; ++q) {
        s[i][q] = c.has(i, q) ? s[i][q] - mean : 0.f;
        ss += s[i][q] * s[i][q];
        sgs += weighted(g[i][q], i, q) * s[i][q];
      }
    row_sums<W>(ss, sgs, red[1]);
    const float inv = 1.0f / sqrtf(ss * n + p.eps);
    const float mg = sg * n, mgu = sgs * n * inv;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float d[VEC];
#pragma unroll
      for (int q = 0; q < VEC; ++q) {
        const float u = s[i][q] * inv;
        dw[i][q] += g[i][q] * u;
        d[q] = (weighted(g[i][q], i, q) - mg - u * mgu) * inv + elem<IO, VEC>(rr[i], q);
      }
      if (p.dresidual) c.store(i, (IO*)p.dresidual + base, d);
#pragma unroll
      for (int q = 0; q < VEC; ++q) d[q] *= p.alpha;
      c.store(i, (IO*)p.dx + base, d);
    }
  }
  if (!p.dweight && !p.dbias) return;
  float* to_w = p.partial + (size_t)blockIdx.x * 2 * p.H;
  float* to_b = to_w + p.H;
  if (gridDim.x == 1) {
    to_w = p.dweight;
    to_b = p.dbias;
  }
  if constexpr (kWorkers > 1) {
    // a lane's vectors where it has them among the 64 lanes', what is another's as zeros
    const int me = (threadIdx.x - mine * 64) * VEC;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      store_vec<float, VEC>(&sums[0][mine][me + i * 64 * VEC], dw[i]);
      store_vec<float, VEC>(&sums[1][mine][me + i * 64 * VEC], db[i]);
    }
    __syncthreads();
    const int last = (p.H - 1) / VEC * VEC;  // the vector that ends with the row is kept here
    for (int i = threadIdx.x; i < 2 * p.H; i += blockDim.x) {
      const int half = i >= p.H, col = i - half * p.H;
      const int at = ANY && col >= last ? col - (p.H - VEC) + last : col;
      float v = 0.f;
#pragma unroll
      for (int t = 0; t < kWorkers; ++t) v += sums[half][t][at];
      float* to = half ? to_b : to_w;
      if (to) to[col] = v;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (to_w) c.store(i, to_w, dw[i]);
      if (to_b) c.store(i, to_b, db[i]);
    }
  }
}

// The workgroups' sums added up: 32 columns of one of the two to a workgroup here, whose 32
// half waves take those of the workgroups h, h + 32, ...; then the halves' in order.
__global__ __launch_bounds__(1024) void finish_kernel(const float* __restrict__ partial,
                                                      int partials, int H,
                                                      float* __restrict__ dweight,
                                                      float* __restrict__ dbias) {
  __shared__ float part[32][32];
  float* out = blockIdx.y ? dbias : dweight;
  if (!out) return;
  const int at = threadIdx.x & 31, half = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + at;
  const float* from = partial + (blockIdx.y ? H : 0) + min(col, H - 1);
  float v = 0.f;
#pragma unroll 8
  for (int i = half; i < partials; i += 32) v += from[(size_t)i * 2 * H];
  part[half][at] = v;
  __syncthreads();
  if (half == 0 && col < H) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += part[i][at];
    out[col] = v;
  }
}

// Calls f(W, NV) as compile-time constants for rows of H elements: up to 8 waves with a vector a
// lane, as few as hold the row (of 4 and 8 alone 4096 x 2560 bf16 took 17.1 us forward and
// 28.5 backward instead of 16.4 and 26.2). The longest rows of the backward pass (BACK) take 8
// waves: 16 leave a wave 128 registers, from which more of a row spills (4096 x 16384 bf16 202
// us instead of 149, 2048 x 16384 fp32 180 instead of 169). fp32 rows past 8192 spill with 8
// too, 26 registers of a lane, off the 16-byte grid 131 (2048 x 16383 195 us), bf16 ones there
// 4 (4096 x 16383 185), and rows of 65 to 128 vectors off it 1.
template <int V>
struct Int {
  static constexpr int value = V;
};
template <int VEC, bool BACK, typename F>
static void by_row_length(int H, F f) {
  const int vecs = (H + VEC - 1) / VEC;
  if (VEC == 1 || vecs <= 64) {
    f(Int<1>{}, Int<1>{});
  } else if constexpr (VEC > 1) {
    if (vecs <= 128) f(Int<1>{}, Int<2>{});
    else if (vecs <= 192) f(Int<3>{}, Int<1>{});
    else if (vecs <= 256) f(Int<4>{}, Int<1>{});
    else if (vecs <= 320) f(Int<5>{}, Int<1>{});
    else if (vecs <= 384) f(Int<6>{}, Int<1>{});
    else if (vecs <= 448) f(Int<7>{}, Int<1>{});
    else if (vecs <= 512) f(Int<8>{}, Int<1>{});
    else if (vecs <= 1024) f(Int<8>{}, Int<2>{});
    else if constexpr (BACK) {
      if (VEC == 8 || vecs <= 2048) f(Int<8>{}, Int<4>{});
      else if constexpr (VEC == 4) f(Int<8>{}, Int<8>{});
    } else if (VEC == 8 || vecs <= 2048) f(Int<16>{}, Int<2>{});
    else if constexpr (VEC == 4) f(Int<16>{}, Int<4>{});
  }
}

// Calls f(VEC, ANY, type): 16 bytes to a lane; ANY where rows do not start at multiples of
// 16; rows shorter than that element by element.
template <typename F>
static void by_type(int H, int dtype, std::initializer_list<const void*> ptrs, F f) {
  const int vec = dtype == MOE_DTYPE_BF16 ? 8 : 4;
  bool any = H % vec != 0;
  for (const void* p : ptrs) any = any || (uintptr_t)p % 16;
  const uint16_t b = 0;
  const float s = 0;
  if (dtype == MOE_DTYPE_BF16) {
    if (H < vec) f(Int<1>{}, Int<0>{}, b);
    else if (any) f(Int<8>{}, Int<1>{}, b);
    else f(Int<8>{}, Int<0>{}, b);
  } else {
    if (H < vec) f(Int<1>{}, Int<0>{}, s);
    else if (any) f(Int<4>{}, Int<1>{}, s);
    else f(Int<4>{}, Int<0>{}, s);
  }
}

// Workgroups of the backward pass for rows of H elements.
// More of them keep more rows in flight, fewer have fewer sums to write and add up (2 H floats
// each): a quarter of the rows (an eighth: 2385 x 1704 17.9 us instead of 16.5, 5446 x 1168 22.1
// instead of 20.2), at least 256 and at most what these measured (us, bf16): 8192 x 2048 256
// 36.9, 512 28.1, 768 27.4; 4096 x 4096 256 40.1, 512 38.8, 768 45.7; 1000 x 4096 256 15.9, 512
// 19.6; 8192 x 7168 256 121, 512 129. Rows of one wave: a wave for each as far as 256 workgroups
// go, one workgroup alone up to 16 rows (with 64, four to a wave, 64 x 512 took 8.7 instead of
// 5.8 with a second kernel).
static int partials_of(int T, int H, int dtype) {
  const int vec = dtype == MOE_DTYPE_BF16 ? 8 : 4, vecs = (H + vec - 1) / vec;
  if (H < vec || vecs <= 128) return std::min((T + 15) / 16, 256);
  const int most = vecs <= 256 ? 768 : vecs <= 512 ? 512 : 256;
  return std::min(T, std::min(std::max(T / 4, 256), most));
}

}  // namespace layer_norm

size_t layer_norm_backward_workspace_bytes(int T, int H) {
  const int most = std::max(layer_norm::partials_of(T, H, MOE_DTYPE_BF16),
                            layer_norm::partials_of(T, H, MOE_DTYPE_F32));
  return ((size_t)most * 2 * H * sizeof(float) + 255) / 256 * 256;
}

hipError_t launch_layer_norm(const LayerNormProblem& p, hipStream_t stream) {
  using namespace layer_norm;
  by_type(p.H, p.dtype, {p.x, p.residual, p.weight, p.bias, p.residual_out, p.out},
          [&](auto v, auto any, auto io) {
            constexpr int VEC = decltype(v)::value;
            by_row_length<VEC, false>(p.H, [&](auto w, auto nv) {
              constexpr int W = decltype(w)::value, NV = decltype(nv)::value;
              forward_kernel<W, NV, VEC, decltype(any)::value != 0, decltype(io)>
                  <<<grid_of<W>(p.T), W == 1 ? 256 : W * 64, 0, stream>>>(p);
            });
          });
  return hipGetLastError();
}

hipError_t launch_layer_norm_backward(const LayerNormBackwardProblem& p, hipStream_t stream) {
  using namespace layer_norm;
  const int partials = partials_of(p.T, p.H, p.dtype);
  if (p.T > 0) {
    const bool alone = partials == 1;
    by_type(p.H, p.dtype,
            {p.dout, p.s, p.weight, p.dresidual_out, p.dx, p.dresidual,
             alone ? p.dweight : nullptr, alone ? p.dbias : nullptr},
            [&](auto v, auto any, auto io) {
              constexpr int VEC = decltype(v)::value;
              by_row_length<VEC, true>(p.H, [&](auto w, auto nv) {
                constexpr int W = decltype(w)::value, NV = decltype(nv)::value;
                backward_kernel<W, NV, VEC, decltype(any)::value != 0, decltype(io)>
                    <<<partials, group_waves<W>() * 64, 0, stream>>>(p);
              });
            });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (partials != 1 && (p.dweight || p.dbias))
    finish_kernel<<<dim3((p.H + 31) / 32, 2), 1024, 0, stream>>>(p.partial, partials, p.H,
                                                                p.dweight, p.dbias);
  return hipGetLastError();
}

}  // namespace moe
