// Rows held in registers: vectors of a row's elements as loaded and as fp32, which
// of them a thread holds, and sums over the waves of a row. For the norms and the
// other kernels that pass over rows.
#pragma once

#include "moe_common.h"

namespace moe {
namespace rows {

// VEC elements of one thread as loaded (32-bit words), and their fp32 values. VEC = 1
// is for rows off the 16-byte grid: one bf16 in the low half of its word.
template <typename T, int VEC>
struct Vec {
  static constexpr int kWords = VEC == 1 ? 1 : VEC * (int)sizeof(T) / 4;  // 1, 2 or 4 n
  uint32_t w[kWords];
};

// Vectors that need not start at a multiple of their size (the hardware's loads and stores
// need not either).
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));

// ANY: p is aligned to an element only.
template <typename T, int VEC, bool NT = false, bool ANY = false>
__device__ __forceinline__ Vec<T, VEC> load_vec(const T* p) {
  constexpr int N = Vec<T, VEC>::kWords;
  Vec<T, VEC> v;
  if constexpr (N == 1) {
    if constexpr (sizeof(T) == 2) v.w[0] = *p;
    else v.w[0] = __float_as_uint(*p);
  } else if constexpr (N == 2) {
    const u32x2 r = ANY ? *(const u32x2_any*)p : *(const u32x2*)p;
    v.w[0] = r[0];
    v.w[1] = r[1];
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      u32x4 r;
      if constexpr (ANY) r = ((const u32x4_any*)p)[i / 4];
      else if constexpr (NT) r = __builtin_nontemporal_load((const u32x4*)p + i / 4);
      else r = ((const u32x4*)p)[i / 4];
#pragma unroll
      for (int q = 0; q < 4; ++q) v.w[i + q] = r[q];
    }
  }
  return v;
}

template <typename T, int VEC>
__device__ __forceinline__ float elem(const Vec<T, VEC>& v, int i) {
  if constexpr (sizeof(T) == 2) {
    const uint32_t u = v.w[i >> 1];
    return __uint_as_float((i & 1) ? (u & 0xffff0000u) : (u << 16));
  } else {
    return __uint_as_float(v.w[i]);
  }
}

template <typename T, int VEC, bool NT = false, bool ANY = false>
__device__ __forceinline__ void store_vec(T* p, const float (&v)[VEC]) {
  constexpr int N = Vec<T, VEC>::kWords;
  if constexpr (N == 1) {
    if constexpr (sizeof(T) == 2) *p = (T)pack_bf16(v[0], v[0]);
    else *p = v[0];
  } else {
    uint32_t o[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (sizeof(T) == 2)
        o[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
      else
        o[i] = __float_as_uint(v[i]);
    }
    if constexpr (N == 2) {
      if constexpr (ANY) *(u32x2_any*)p = u32x2{o[0], o[1]};
      else *(u32x2*)p = u32x2{o[0], o[1]};
    } else {
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        const u32x4 r{o[i], o[i + 1], o[i + 2], o[i + 3]};
        if constexpr (ANY) ((u32x4_any*)p)[i / 4] = r;
        else if constexpr (NT) __builtin_nontemporal_store(r, (u32x4*)p + i / 4);
        else ((u32x4*)p)[i / 4] = r;
      }
    }
  }
}

template <typename T, int VEC>
__device__ __forceinline__ void keep_vec(Vec<T, VEC>& v, uint32_t mask) {
#pragma unroll
  for (int i = 0; i < Vec<T, VEC>::kWords; ++i) v.w[i] &= mask;
}

// The NV vectors of this thread: vector at[i] of the row and mask ~0, or, past
// the end of the row, the last one and mask 0: loads are never conditional (a
// branch around one would have it waited for early), and what the mask clears
// counts as zero in the sums of squares.
template <int W, int NV>
struct Place {
  int at[NV];
  uint32_t mask[NV];
  __device__ __forceinline__ explicit Place(int vecs) {
    const int me = W == 1 ? (threadIdx.x & 63) : threadIdx.x;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = me + i * W * 64;
      at[i] = min(c, vecs - 1);
      mask[i] = c < vecs ? ~0u : 0u;
    }
  }
};

// The same for rows of any H >= VEC elements: at[i] counts elements, and the vector that
// would pass the row's end ends with it instead; its first skip[i] elements are the vector's
// before it (all VEC of a vector past the end) and belong to that one's thread.
template <int W, int NV, int VEC, bool ANY>
struct Span {
  int at[NV], skip[NV];
  // me: the thread's place among the row's
  __device__ __forceinline__ Span(int H, int me) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (me + i * W * 64) * VEC;
      at[i] = min(c, H - VEC);
      skip[i] = ANY ? min(c - at[i], VEC) : c < H ? 0 : VEC;
    }
  }
  __device__ __forceinline__ bool has(int i, int e) const { return ANY ? e >= skip[i] : skip[i] == 0; }
  // this thread's elements of vector i
  template <typename T>
  __device__ __forceinline__ void store(int i, T* row, const float (&v)[VEC]) const {
    if (skip[i] == 0) {
      store_vec<T, VEC, false, ANY>(row + at[i], v);
    } else if (ANY && skip[i] < VEC) {
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (e >= skip[i]) store_vec<T, 1>(row + at[i] + e, {v[e]});
    }
  }
};

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

}  // namespace rows
}  // namespace moe
