// Layer norm with the residual add in front of it, and its gradients.
//
// Forward: one pass; a row is held in registers as fp32 from its loads to its stores,
// its mean and then its squares about the mean are summed in turn. Backward: one pass
// over the rows with the sums s as the forward pass stored them: with u = (s - mean) /
// sqrt(var + eps) and g = dout weight,
//   ds = (g - mean(g) - u mean(g u)) / sqrt(var + eps)  [+ dresidual_out]
// takes two sums over the row twice (s and g, then (s - mean)^2 and g (s - mean)); the
// gradients of weight and bias are sums over all rows, which every worker (W waves with
// one row after the other) keeps in registers for its own rows and writes once, for a
// second kernel that adds the workers' in a fixed order. Bound by HBM.
#include <algorithm>

#include "../../include/moe.h"
#include "moe_common.h"
#include "moe_launch.h"
#include "moe_rows.h"

namespace moe {
namespace layer_norm {

using namespace rows;

constexpr int kGridX = 1 << 20;
// Worker of this thread: W > 1 waves make a workgroup; W = 1: four to one.
template <int W>
__device__ __forceinline__ int my_worker() {
  const int group = blockIdx.y * kGridX + blockIdx.x;
  if constexpr (W == 1)
    return __builtin_amdgcn_readfirstlane(group * 4 + (threadIdx.x >> 6));
  else
    return group;
}
template <int W>
static dim3 grid_of(int workers) {
  const int groups = W == 1 ? (workers + 3) / 4 : workers;
  return dim3(std::min(groups, kGridX), (groups + kGridX - 1) / kGridX);
}

template <int W, int NV, int VEC, typename IO>
__global__ __launch_bounds__(W == 1 ? 256 : W * 64) void forward_kernel(LayerNormProblem p) {
  __shared__ float red[2][W];
  const int row = my_worker<W>();
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
  float s[NV][VEC], sum = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    keep_vec<IO, VEC>(xr[i], c.mask[i]);
    keep_vec<IO, VEC>(rr[i], c.mask[i]);
#pragma unroll
    for (int q = 0; q < VEC; ++q) {
      s[i][q] = p.alpha * elem<IO, VEC>(xr[i], q) + elem<IO, VEC>(rr[i], q);
      sum += s[i][q];
    }
    if (c.mask[i] && p.residual_out)
      store_vec<IO, VEC>((IO*)p.residual_out + base + c.at[i] * VEC, s[i]);
  }
  const float mean = row_sum<W>(sum, red[0]) / (float)p.H;
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int q = 0; q < VEC; ++q) {
      s[i][q] -= mean;
      ss += c.mask[i] ? s[i][q] * s[i][q] : 0.f;
    }
  const float inv = 1.0f / sqrtf(row_sum<W>(ss, red[1]) / (float)p.H + p.eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (!c.mask[i]) continue;
    Vec<float, VEC> w, b{};
    if (p.weight) w = load_vec<float, VEC>(p.weight + c.at[i] * VEC);
    if (p.bias) b = load_vec<float, VEC>(p.bias + c.at[i] * VEC);
    float o[VEC];
#pragma unroll
    for (int q = 0; q < VEC; ++q) {
      o[q] = s[i][q] * inv;
      if (p.weight) o[q] *= elem<float, VEC>(w, q);
      o[q] += elem<float, VEC>(b, q);
    }
    store_vec<IO, VEC>((IO*)p.out + base + c.at[i] * VEC, o);
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

// Worker w takes the rows w, w + workers, ... and writes its sums for the weight and
// the bias to partial[w] ([2, H]). The slots of the two sums are each written again
// only past the other's barrier, when all have read them.
template <int W, int NV, int VEC, typename IO>
__global__ __launch_bounds__(W == 1 ? 256 : W * 64) void backward_kernel(
    LayerNormBackwardProblem p, int workers) {
  __shared__ f32x2 red[2][W];
  const int worker = my_worker<W>();
  if (worker >= workers) return;  // whole waves, and W = 1 has no barrier
  const Place<W, NV> c(p.H / VEC);
  Vec<float, VEC> w[NV];
  float dw[NV][VEC] = {}, db[NV][VEC] = {};
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (p.weight) w[i] = load_vec<float, VEC>(p.weight + c.at[i] * VEC);
  const float n = 1.0f / (float)p.H;
  for (int row = worker; row < p.T; row += workers) {
    const size_t base = (size_t)row * p.H;
    Vec<IO, VEC> sr[NV], gr[NV], rr[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      sr[i] = load_vec<IO, VEC>((const IO*)p.s + base + c.at[i] * VEC);
      gr[i] = load_vec<IO, VEC>((const IO*)p.dout + base + c.at[i] * VEC);
      rr[i] = Vec<IO, VEC>{};
      if (p.dresidual_out)
        rr[i] = load_vec<IO, VEC>((const IO*)p.dresidual_out + base + c.at[i] * VEC);
    }
    float s[NV][VEC], g[NV][VEC], sum = 0.f, sg = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      keep_vec<IO, VEC>(sr[i], c.mask[i]);
      keep_vec<IO, VEC>(gr[i], c.mask[i]);
#pragma unroll
      for (int q = 0; q < VEC; ++q) {
        s[i][q] = elem<IO, VEC>(sr[i], q);
        g[i][q] = elem<IO, VEC>(gr[i], q);
        db[i][q] += g[i][q];
        sum += s[i][q];
        sg += p.weight ? g[i][q] * elem<float, VEC>(w[i], q) : g[i][q];
      }
    }
    row_sums<W>(sum, sg, red[0]);
    const float mean = sum * n;
    float ss = 0.f, sgs = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int q = 0; q < VEC; ++q) {
        s[i][q] = c.mask[i] ? s[i][q] - mean : 0.f;
        ss += s[i][q] * s[i][q];
        sgs += (p.weight ? g[i][q] * elem<float, VEC>(w[i], q) : g[i][q]) * s[i][q];
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
        const float gw = p.weight ? g[i][q] * elem<float, VEC>(w[i], q) : g[i][q];
        d[q] = (gw - mg - u * mgu) * inv + elem<IO, VEC>(rr[i], q);
      }
      if (!c.mask[i]) continue;
      const size_t at = base + c.at[i] * VEC;
      if (p.dresidual) store_vec<IO, VEC>((IO*)p.dresidual + at, d);
#pragma unroll
      for (int q = 0; q < VEC; ++q) d[q] *= p.alpha;
      store_vec<IO, VEC>((IO*)p.dx + at, d);
    }
  }
  if (!p.dweight && !p.dbias) return;
  float* mine = p.partial + (size_t)worker * 2 * p.H;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (!c.mask[i]) continue;
    store_vec<float, VEC>(mine + c.at[i] * VEC, dw[i]);
    store_vec<float, VEC>(mine + p.H + c.at[i] * VEC, db[i]);
  }
}

// The workers' sums added up: a workgroup takes 64 columns of one of the two, wave w
// the workers w, w + 16, ...; then the waves' in order.
__global__ __launch_bounds__(1024) void finish_kernel(const float* __restrict__ partial,
                                                      int workers, int H,
                                                      float* __restrict__ dweight,
                                                      float* __restrict__ dbias) {
  __shared__ float part[16][64];
  float* out = blockIdx.y ? dbias : dweight;
  if (!out) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = blockIdx.x * 64 + lane;
  const float* from = partial + (blockIdx.y ? H : 0) + min(col, H - 1);
  float v = 0.f;
#pragma unroll 4
  for (int i = wave; i < workers; i += 16) v += from[(size_t)i * 2 * H];
  part[wave][lane] = v;
  __syncthreads();
  if (wave == 0 && col < H) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) v += part[i][lane];
    out[col] = v;
  }
}

// Calls f(W, NV) as compile-time constants for rows of H elements.
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
  else if (VEC == 4 || vecs <= 4096) f(Int<16>{}, Int<4>{});
  else if constexpr (VEC == 1) f(Int<16>{}, Int<16>{});
}

static int workers_of(int T) { return std::min(T, 512); }

template <int VEC, typename IO>
static void run_forward(const LayerNormProblem& p, hipStream_t stream) {
  by_row_length<VEC>(p.H, [&](auto w, auto nv) {
    constexpr int W = decltype(w)::value, NV = decltype(nv)::value;
    forward_kernel<W, NV, VEC, IO><<<grid_of<W>(p.T), W == 1 ? 256 : W * 64, 0, stream>>>(p);
  });
}

template <int VEC, typename IO>
static void run_backward(const LayerNormBackwardProblem& p, hipStream_t stream) {
  const int workers = workers_of(p.T);
  by_row_length<VEC>(p.H, [&](auto w, auto nv) {
    constexpr int W = decltype(w)::value, NV = decltype(nv)::value;
    backward_kernel<W, NV, VEC, IO>
        <<<grid_of<W>(workers), W == 1 ? 256 : W * 64, 0, stream>>>(p, workers);
  });
}

// 16 bytes to a lane where every row starts at a multiple of 16, else one element.
static bool wide(int H, int dtype, std::initializer_list<const void*> ptrs) {
  if (H % (dtype == MOE_DTYPE_BF16 ? 8 : 4)) return false;
  for (const void* p : ptrs)
    if ((uintptr_t)p % 16) return false;
  return true;
}

}  // namespace layer_norm

size_t layer_norm_backward_workspace_bytes(int T, int H) {
  return ((size_t)layer_norm::workers_of(T) * 2 * H * sizeof(float) + 255) / 256 * 256;
}

hipError_t launch_layer_norm(const LayerNormProblem& p, hipStream_t stream) {
  using namespace layer_norm;
  const bool v = wide(p.H, p.dtype, {p.x, p.residual, p.weight, p.bias, p.residual_out, p.out});
  if (p.dtype == MOE_DTYPE_BF16)
    v ? run_forward<8, uint16_t>(p, stream) : run_forward<1, uint16_t>(p, stream);
  else
    v ? run_forward<4, float>(p, stream) : run_forward<1, float>(p, stream);
  return hipGetLastError();
}

hipError_t launch_layer_norm_backward(const LayerNormBackwardProblem& p, hipStream_t stream) {
  using namespace layer_norm;
  const bool v = wide(p.H, p.dtype, {p.dout, p.s, p.weight, p.dresidual_out, p.dx, p.dresidual});
  if (p.T > 0) {
    if (p.dtype == MOE_DTYPE_BF16)
      v ? run_backward<8, uint16_t>(p, stream) : run_backward<1, uint16_t>(p, stream);
    else
      v ? run_backward<4, float>(p, stream) : run_backward<1, float>(p, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (p.dweight || p.dbias)
    finish_kernel<<<dim3((p.H + 63) / 64, 2), 1024, 0, stream>>>(p.partial, workers_of(p.T), p.H,
                                                                p.dweight, p.dbias);
  return hipGetLastError();
}

}  // namespace moe
