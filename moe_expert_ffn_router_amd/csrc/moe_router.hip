// Router projection: logits[t, e] = x[t] . w[e] + bias[e] in fp32.
//
// One wave per (token, expert), lanes splitting H.
#include "../../include/moe.h"
#include "moe_common.h"
#include "moe_launch.h"

namespace moe {
namespace router {

__device__ __forceinline__ float val(const float* p) { return *p; }
__device__ __forceinline__ float val(const uint16_t* p) { return bf16_bits_to_f32(*p); }

template <typename XT, typename WT>
__global__ __launch_bounds__(256) void router_kernel(const XT* __restrict__ x,
                                                     const WT* __restrict__ w,
                                                     const float* __restrict__ bias, long n,
                                                     int E, int H, float* __restrict__ logits) {
  const long u = (long)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (u >= n) return;  // uniform per wave
  const XT* xr = x + (size_t)(u / E) * H;
  const WT* wr = w + (size_t)(u % E) * H;
  float s = 0.f;
  for (int c = threadIdx.x & 63; c < H; c += 64) s += val(xr + c) * val(wr + c);
  s = wave_sum(s);
  if ((threadIdx.x & 63) == 0) logits[u] = bias ? s + bias[u % E] : s;
}

}  // namespace router

hipError_t launch_router_logits(const void* x, int x_dtype, const void* w, int w_dtype,
                                const float* bias, int T, int E, int H, float* logits,
                                hipStream_t stream) {
  const long n = (long)T * E;
  const dim3 grid((unsigned)((n + 3) / 4));
  if (x_dtype == MOE_DTYPE_F32)
    router::router_kernel<<<grid, 256, 0, stream>>>((const float*)x, (const float*)w, bias, n, E,
                                                    H, logits);
  else if (w_dtype == MOE_DTYPE_F32)
    router::router_kernel<<<grid, 256, 0, stream>>>((const uint16_t*)x, (const float*)w, bias, n,
                                                    E, H, logits);
  else
    router::router_kernel<<<grid, 256, 0, stream>>>((const uint16_t*)x, (const uint16_t*)w, bias,
                                                    n, E, H, logits);
  return hipGetLastError();
}

}  // namespace moe
