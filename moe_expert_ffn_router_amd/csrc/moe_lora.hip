// Low-rank adapters of many requests beside a shared projection:
// out[s] = y[s] + scale[g] * b[g] (a[g] x[s]) for the rows s of adapter g.
//
// Two launches over the aligned row lists: z = a x (fp32, in the workspace),
// then the expansion by b into the rows of y.
#include "../../include/moe.h"
#include "moe_common.h"
#include "moe_launch.h"

namespace moe {
namespace lora {

__device__ __forceinline__ float val(const float* p) { return *p; }
__device__ __forceinline__ float val(const uint16_t* p) { return bf16_bits_to_f32(*p); }

// Row of sorted position pos, or -1 (a sentinel, or past the lists); its adapter in g.
__device__ __forceinline__ int row_at(const LoraProblem& p, int log2m, long pos, int& g) {
  if (pos >= p.num_padded[0]) return -1;
  const int row = p.sorted_ids[pos];
  g = p.block_adapter[pos >> log2m];
  return (unsigned)row < (unsigned)p.S && (unsigned)g < (unsigned)p.n ? row : -1;
}

// One wave per (position, rank).
template <typename XT>
__global__ __launch_bounds__(256) void shrink_kernel(LoraProblem p, int log2m, long units) {
  const long u = (long)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (u >= units) return;  // uniform per wave
  int g = 0;
  const int row = row_at(p, log2m, u / p.r, g), q = (int)(u % p.r);
  if (row < 0) return;
  const XT* xr = (const XT*)p.x + (size_t)row * p.ldx;
  const uint16_t* ar = p.a + ((size_t)g * p.r + q) * p.K;
  float s = 0.f;
  for (int c = threadIdx.x & 63; c < p.K; c += 64) s += val(xr + c) * val(ar + c);
  s = wave_sum(s);
  if ((threadIdx.x & 63) == 0) ((float*)p.workspace)[(size_t)row * p.r + q] = s;
}

// One thread per (position, column).
template <typename YT>
__global__ __launch_bounds__(256) void expand_kernel(LoraProblem p, int log2m) {
  int g = 0;
  const int row = row_at(p, log2m, blockIdx.x, g);
  const int c = blockIdx.y * 256 + threadIdx.x;
  if (row < 0 || c >= p.N) return;
  const float* z = (const float*)p.workspace + (size_t)row * p.r;
  const uint16_t* br = p.b + ((size_t)g * p.N + c) * p.r;
  float s = 0.f;
  for (int q = 0; q < p.r; ++q) s += z[q] * val(br + q);
  const float v = val((const YT*)p.y + (size_t)row * p.ldy + c) + (p.scale ? p.scale[g] * s : s);
  YT* o = (YT*)p.out + (size_t)row * p.ldo + c;
  if constexpr (sizeof(YT) == 2) *o = (YT)f32_to_bf16_rne(v);
  else *o = v;
}

}  // namespace lora

size_t lora_workspace_bytes(int S, int n, int K, int r, int block_m) {
  (void)n, (void)K, (void)block_m;
  return ((size_t)S * r * sizeof(float) + 255) / 256 * 256;
}

hipError_t launch_lora_add(const LoraProblem& p, hipStream_t stream) {
  int log2m = 0;
  while ((1 << log2m) < p.block_m) ++log2m;
  const size_t cap = align_capacity(p.S, p.n, p.block_m);
  const long units = (long)cap * p.r;
  const dim3 shrink((unsigned)((units + 3) / 4));
  if (p.x_dtype == MOE_DTYPE_BF16)
    lora::shrink_kernel<uint16_t><<<shrink, 256, 0, stream>>>(p, log2m, units);
  else
    lora::shrink_kernel<float><<<shrink, 256, 0, stream>>>(p, log2m, units);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const dim3 expand((unsigned)cap, (p.N + 255) / 256);
  if (p.y_dtype == MOE_DTYPE_BF16)
    lora::expand_kernel<uint16_t><<<expand, 256, 0, stream>>>(p, log2m);
  else
    lora::expand_kernel<float><<<expand, 256, 0, stream>>>(p, log2m);
  return hipGetLastError();
}

}  // namespace moe
