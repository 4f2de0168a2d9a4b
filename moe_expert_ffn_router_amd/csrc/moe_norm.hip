// Norms around the expert FFN: before it (residual add, RMS norm) and after it
// (top-k combine, gated shared expert, RMS norm, residual add, next norm).
//
// Every kernel is one pass: a row is held in registers as fp32 from its loads
// to its stores, so each input is read once and each output written once, and
// the only other work is one (norm_in) or up to two (norm_out) sums of squares
// per row. Bound by HBM: 2 bytes per bf16 element and stream; for norm_out the
// k expert rows per token are the largest of them.
//
// W waves serve a row: thread i of the row's 64 W holds the vectors i,
// i + 64 W, ... of VEC elements (8: one 16-byte load of bf16, two of fp32; 4
// where an fp32 row length asks for it), NV of them.
#include "../../include/moe.h"
#include "moe_common.h"
#include "moe_launch.h"

namespace moe {
namespace norm {

// VEC elements of one thread as loaded (16-byte words), and their fp32 values.
template <typename T, int VEC>
struct Vec {
  static constexpr int kWords = VEC * (int)sizeof(T) / 16;
  u32x4 w[kWords];
};

template <typename T, int VEC>
__device__ __forceinline__ Vec<T, VEC> load_vec(const T* p) {
  Vec<T, VEC> v;
#pragma unroll
  for (int i = 0; i < Vec<T, VEC>::kWords; ++i) v.w[i] = ((const u32x4*)p)[i];
  return v;
}

template <typename T, int VEC>
__device__ __forceinline__ float elem(const Vec<T, VEC>& v, int i) {
  if constexpr (sizeof(T) == 2) {
    const uint32_t u = v.w[i >> 3][(i >> 1) & 3];
    return __uint_as_float((i & 1) ? (u & 0xffff0000u) : (u << 16));
  } else {
    return __uint_as_float(v.w[i >> 2][i & 3]);
  }
}

template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T* p, const float (&v)[VEC]) {
#pragma unroll
  for (int i = 0; i < Vec<T, VEC>::kWords; ++i) {
    u32x4 o;
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        o[q] = f32_to_bf16_rne(v[i * 8 + 2 * q]) | (f32_to_bf16_rne(v[i * 8 + 2 * q + 1]) << 16);
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) o[q] = __float_as_uint(v[i * 4 + q]);
    }
    ((u32x4*)p)[i] = o;
  }
}

// Sum over the W waves of a row, in a fixed order; `slot`: W words of LDS of
// this use alone (no barrier protects them from an earlier use).
template <int W>
__device__ __forceinline__ float row_sum(float v, float* slot) {
  v = wave_sum(v);
  if constexpr (W > 1) {
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) v += slot[i];
  }
  return v;
}

template <int NV, int VEC>
__device__ __forceinline__ float sum_squares(const float (&v)[NV][VEC]) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int q = 0; q < VEC; ++q) s += v[i][q] * v[i][q];
  return s;
}

// The row this thread works on: W >= 4 waves: one row per workgroup; W = 1:
// a row per wave, four to a workgroup.
template <int W>
__device__ __forceinline__ int my_row() {
  if constexpr (W == 1)
    return __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
  else
    return blockIdx.x;
}
template <int W>
__device__ __forceinline__ int my_thread() {
  return W == 1 ? (threadIdx.x & 63) : threadIdx.x;
}

template <int W, int NV, int VEC, typename IO>
__global__ __launch_bounds__(W == 1 ? 256 : W * 64) void norm_in_kernel(NormInProblem p) {
  __shared__ float red[W];
  const int row = my_row<W>();
  if (row >= p.T) return;  // whole waves, and W = 1 has no barrier
  const int vecs = p.H / VEC;
  const size_t base = (size_t)row * p.H;
  Vec<IO, VEC> xr[NV], rr[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = my_thread<W>() + i * W * 64;
    xr[i] = rr[i] = Vec<IO, VEC>{};
    if (c < vecs) {
      xr[i] = load_vec<IO, VEC>((const IO*)p.x + base + (size_t)c * VEC);
      if (p.residual) rr[i] = load_vec<IO, VEC>((const IO*)p.residual + base + (size_t)c * VEC);
    }
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
    const int c = my_thread<W>() + i * W * 64;
    if (c < vecs) {
      const size_t at = base + (size_t)c * VEC;
      if (p.residual_out) store_vec<IO, VEC>((IO*)p.residual_out + at, s[i]);
      const Vec<float, VEC> g = load_vec<float, VEC>(p.weight + (size_t)c * VEC);
      float o[VEC];
#pragma unroll
      for (int q = 0; q < VEC; ++q) o[q] = s[i][q] * inv * elem<float, VEC>(g, q);
      store_vec<IO, VEC>((IO*)p.out + at, o);
    }
  }
}

template <int W, int NV, int VEC, typename YT, typename IO>
__global__ __launch_bounds__(W == 1 ? 256 : W * 64) void norm_out_kernel(NormOutProblem p) {
  __shared__ float red[2][W];
  const int row = my_row<W>();
  if (row >= p.T) return;  // whole waves, and W = 1 has no barrier
  const int vecs = p.H / VEC;
  const size_t base = (size_t)row * p.H;
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
      if (p.topk_ids) mine = (unsigned)p.topk_ids[s] < (unsigned)p.E;
      if (p.topk_weights) wl = p.topk_weights[s];
    }
    uint64_t left = __ballot(mine);
    while (left) {
      const int u = __builtin_ctzll(left);
      left &= left - 1;
      const float wj = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(wl), u));
      const YT* yr = (const YT*)p.y + ((size_t)row * p.k + j0 + u) * p.H;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = my_thread<W>() + i * W * 64;
        if (c < vecs) {
          const Vec<YT, VEC> r = load_vec<YT, VEC>(yr + (size_t)c * VEC);
#pragma unroll
          for (int q = 0; q < VEC; ++q) v[i][q] += wj * elem<YT, VEC>(r, q);
        }
      }
    }
  }
  if (p.shared) {
    const float g = p.gate ? 1.0f / (1.0f + expf(-p.gate[row])) : 1.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = my_thread<W>() + i * W * 64;
      if (c < vecs) {
        const Vec<IO, VEC> r = load_vec<IO, VEC>((const IO*)p.shared + base + (size_t)c * VEC);
#pragma unroll
        for (int q = 0; q < VEC; ++q) v[i][q] += g * elem<IO, VEC>(r, q);
      }
    }
  }
  if (p.weight) {
    const float ms = row_sum<W>(sum_squares<NV, VEC>(v), red[0]) / (float)p.H;
    const float inv = 1.0f / sqrtf(ms + p.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = my_thread<W>() + i * W * 64;
      if (c < vecs) {
        const Vec<float, VEC> g = load_vec<float, VEC>(p.weight + (size_t)c * VEC);
#pragma unroll
        for (int q = 0; q < VEC; ++q) v[i][q] = v[i][q] * inv * elem<float, VEC>(g, q);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = my_thread<W>() + i * W * 64;
    if (c < vecs) {
      Vec<IO, VEC> r{};
      if (p.residual) r = load_vec<IO, VEC>((const IO*)p.residual + base + (size_t)c * VEC);
#pragma unroll
      for (int q = 0; q < VEC; ++q) v[i][q] = p.scale * v[i][q] + elem<IO, VEC>(r, q);
      store_vec<IO, VEC>((IO*)p.out + base + (size_t)c * VEC, v[i]);
    }
  }
  if (p.next) {
    const float ms = row_sum<W>(sum_squares<NV, VEC>(v), red[1]) / (float)p.H;
    const float inv = 1.0f / sqrtf(ms + p.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = my_thread<W>() + i * W * 64;
      if (c < vecs) {
        const Vec<float, VEC> g = load_vec<float, VEC>(p.next_weight + (size_t)c * VEC);
        float o[VEC];
#pragma unroll
        for (int q = 0; q < VEC; ++q) o[q] = v[i][q] * inv * elem<float, VEC>(g, q);
        store_vec<IO, VEC>((IO*)p.next + base + (size_t)c * VEC, o);
      }
    }
  }
}

// Calls f(W, NV) as compile-time constants for a row of `vecs` vectors: the
// fewest waves that hold it in at most two vectors per thread.
template <int V>
struct Int {
  static constexpr int value = V;
};
template <typename F>
static void by_row_length(int vecs, F f) {
  if (vecs <= 64) f(Int<1>{}, Int<1>{});
  else if (vecs <= 128) f(Int<1>{}, Int<2>{});
  else if (vecs <= 256) f(Int<4>{}, Int<1>{});
  else if (vecs <= 512) f(Int<4>{}, Int<2>{});
  else if (vecs <= 1024) f(Int<16>{}, Int<1>{});
  else if (vecs <= 2048) f(Int<16>{}, Int<2>{});
  else f(Int<16>{}, Int<4>{});
}

template <int W>
static dim3 grid_of(int T) {
  return dim3(W == 1 ? (T + 3) / 4 : T);
}

template <int VEC, typename IO>
static void run_in(const NormInProblem& p, hipStream_t stream) {
  by_row_length(p.H / VEC, [&](auto w, auto nv) {
    constexpr int W = decltype(w)::value, NV = decltype(nv)::value;
    norm_in_kernel<W, NV, VEC, IO>
        <<<grid_of<W>(p.T), W == 1 ? 256 : W * 64, 0, stream>>>(p);
  });
}

template <int VEC, typename YT, typename IO>
static void run_out(const NormOutProblem& p, hipStream_t stream) {
  by_row_length(p.H / VEC, [&](auto w, auto nv) {
    constexpr int W = decltype(w)::value, NV = decltype(nv)::value;
    norm_out_kernel<W, NV, VEC, YT, IO>
        <<<grid_of<W>(p.T), W == 1 ? 256 : W * 64, 0, stream>>>(p);
  });
}

}  // namespace norm

hipError_t launch_norm_in(const NormInProblem& p, hipStream_t stream) {
  if (p.dtype == MOE_DTYPE_BF16) norm::run_in<8, uint16_t>(p, stream);
  else if (p.H % 8 == 0) norm::run_in<8, float>(p, stream);
  else norm::run_in<4, float>(p, stream);
  return hipGetLastError();
}

hipError_t launch_norm_out(const NormOutProblem& p, hipStream_t stream) {
  if (p.dtype == MOE_DTYPE_BF16) {
    if (p.y_dtype == MOE_DTYPE_BF16) norm::run_out<8, uint16_t, uint16_t>(p, stream);
    else norm::run_out<8, float, uint16_t>(p, stream);
  } else if (p.y_dtype == MOE_DTYPE_BF16) {
    norm::run_out<8, uint16_t, float>(p, stream);
  } else if (p.H % 8 == 0) {
    norm::run_out<8, float, float>(p, stream);
  } else {
    norm::run_out<4, float, float>(p, stream);
  }
  return hipGetLastError();
}

}  // namespace moe
