// Router projection: logits[t, e] = x[t] . w[e] + bias[e] in fp32, on the matrix
// cores with K split over the waves of a workgroup (moe_skinny.h), so that one
// launch serves a single token as well as a prompt and needs no workspace.
#include "../../include/moe.h"
#include "moe_common.h"
#include "moe_launch.h"
#include "moe_skinny.h"

namespace moe {
namespace router {

template <int MT, int NT, int NW, int D, typename XT, typename WT>
__global__ __launch_bounds__(NW * 64) void router_kernel(const XT* __restrict__ x,
                                                         const WT* __restrict__ w,
                                                         const float* __restrict__ bias, int T,
                                                         int E, int H, int e_tiles,
                                                         float* __restrict__ logits) {
  __shared__ __align__(16) char lds[skinny::lds_bytes<MT, NT, NW, XT, WT>()];
  // the expert tiles of one token tile are 8 workgroups apart: on one XCD, whose
  // L2 then serves the token rows to all but the first
  const int tile = blockIdx.x / (8 * e_tiles) * 8 + blockIdx.x % 8;
  const int t0 = tile * MT * 16, e0 = blockIdx.x / 8 % e_tiles * NT * 16;
  if (t0 >= T) return;  // the whole workgroup
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  skinny::Product<MT, NT, XT, WT> m;
  m.lds = lds + wave * m.kLdsBytes;
  m.x.set([&](int i) { return x + (size_t)min(t0 + i, T - 1) * H; });
  m.w.set([&](int i) { return w + (size_t)min(e0 + i, E - 1) * H; });
  m.clear();
  m.template accumulate<D>(H, wave, (H + skinny::kChunk - 1) / skinny::kChunk, NW);
  skinny::reduce_waves<MT, NT, NW>(m.acc, lds, [&](int j, int i, int lane, f32x4 s) {
    const int t = t0 + i * 16 + (lane & 15), e = e0 + j * 16 + (lane >> 4) * 4;
    if (t >= T) return;
    float* o = logits + (size_t)t * E + e;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (e + q < E) o[q] = bias ? s[q] + bias[e + q] : s[q];
  });
}

template <int MT, int NT, int NW, int D, typename XT, typename WT>
static void run(const XT* x, const WT* w, const float* bias, int T, int E, int H, float* logits,
                hipStream_t stream) {
  const int tt = (T + MT * 16 - 1) / (MT * 16), et = (E + NT * 16 - 1) / (NT * 16);
  router_kernel<MT, NT, NW, D><<<(tt + 7) / 8 * 8 * et, NW * 64, 0, stream>>>(x, w, bias, T, E, H,
                                                                    et, logits);
}

template <typename XT, typename WT>
static void dispatch(const XT* x, const WT* w, const float* bias, int T, int E, int H,
                     float* logits, hipStream_t stream) {
  const long big = (long)((T + 31) / 32) * ((E + 63) / 64);
  // fp32 operands take twice the registers of bf16: half the depth
  constexpr int kHalf = sizeof(XT) == 4 ? 2 : 1;
  if (big >= 128)
    run<2, 4 / kHalf, 8, 1>(x, w, bias, T, E, H, logits, stream);
  else
    run<1, 1, 16, sizeof(WT) == 4 ? 2 : 4>(x, w, bias, T, E, H, logits, stream);
}

}  // namespace router

hipError_t launch_router_logits(const void* x, int x_dtype, const void* w, int w_dtype,
                                const float* bias, int T, int E, int H, float* logits,
                                hipStream_t stream) {
  if (x_dtype == MOE_DTYPE_F32)
    router::dispatch((const float*)x, (const float*)w, bias, T, E, H, logits, stream);
  else if (w_dtype == MOE_DTYPE_F32)
    router::dispatch((const uint16_t*)x, (const float*)w, bias, T, E, H, logits, stream);
  else
    router::dispatch((const uint16_t*)x, (const uint16_t*)w, bias, T, E, H, logits, stream);
  return hipGetLastError();
}

}  // namespace moe
