// Router projection: logits[t, e] = x[t] . w[e] + bias[e] in fp32, on the matrix
// cores with K split over the waves of a workgroup (moe_skinny.h), so that one
// launch serves a single token as well as a prompt and needs no workspace.
// Bound by what a CU reads: R (MT + NT) rows of x and w per workgroup. Measured
// (captured into a graph): 16 tokens x 64 experts x 4096 bf16 3.4 us, 64 x 128 x
// 7168 with fp32 w 8.4 us (the split of w into planes included), 512 x 128 x 4096
// 5.6 us, 4096 x 128 x 4096 14.9 us: 786 KB per CU at 63 GB/s, where 32 x 64
// tiles, one per CU, are the largest that fill the chip.
#include "../../include/moe.h"
#include "moe_common.h"
#include "moe_launch.h"
#include "moe_skinny.h"

namespace moe {
namespace router {

// A workgroup: MT tiles of R tokens x NT tiles of R experts, K split over its NW
// waves, D chunks of a wave in flight.
template <int MT, int NT, int R, int NW, int D, typename XT, typename WT>
__global__ __launch_bounds__(NW * 64) void router_kernel(const XT* __restrict__ x,
                                                         const WT* __restrict__ w,
                                                         const float* __restrict__ bias, int T,
                                                         int E, int H, int e_tiles,
                                                         float* __restrict__ logits) {
  __shared__ __align__(16) char lds[skinny::lds_bytes<MT, NT, R, NW, XT, WT>()];
  // the expert tiles of one token tile are 8 workgroups apart: on one XCD, whose
  // L2 then serves the token rows to all but the first
  const int tile = blockIdx.x / (8 * e_tiles) * 8 + blockIdx.x % 8;
  const int t0 = tile * MT * R, e0 = blockIdx.x / 8 % e_tiles * NT * R;
  if (t0 >= T) return;  // the whole workgroup
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  skinny::Product<MT, NT, R, XT, WT> m;
  m.lds = lds + wave * m.kLdsBytes;
  m.x.set([&](int i) { return x + (size_t)min(t0 + i, T - 1) * H; });
  m.w.set([&](int i) { return w + (size_t)min(e0 + i, E - 1) * H; });
  m.clear();
  m.template accumulate<D>(H, wave, (H + skinny::kChunk - 1) / skinny::kChunk, NW);
  const bool whole = E % 4 == 0 && (uintptr_t)logits % 16 == 0;  // rows of 16-byte words
  skinny::reduce_waves<MT, NT, R, NW>(m.acc, lds, [&](int wr, int xr, auto s) {
    const int t = t0 + xr, e = e0 + wr;
    if (t >= T || e >= E) return;
    float* o = logits + (size_t)t * E + e;
    if constexpr (sizeof(s) == 4) {
      *o = bias ? s + bias[e] : s;
    } else {
      if (bias) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (e + q < E) s[q] += bias[e + q];
      }
      if (whole) {
        *(f32x4*)o = s;
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (e + q < E) o[q] = s[q];
      }
    }
  });
}

template <int MT, int NT, int R, int NW, int D, typename XT, typename WT>
static void run(const XT* x, const WT* w, const float* bias, int T, int E, int H, float* logits,
                hipStream_t stream) {
  const int tt = (T + MT * R - 1) / (MT * R), et = (E + NT * R - 1) / (NT * R);
  router_kernel<MT, NT, R, NW, D>
      <<<(tt + 7) / 8 * 8 * et, NW * 64, 0, stream>>>(x, w, bias, T, E, H, et, logits);
}

template <typename XT, typename WT>
static void dispatch(const XT* x, const WT* w, const float* bias, int T, int E, int H,
                     float* logits, hipStream_t stream) {
  // fp32 tokens take twice the registers of bf16: half the tiles, half the depth
  constexpr int kHalf = sizeof(XT) == 4 ? 2 : 1;
  // the largest tiles of which there are 96 (x 4096, 128 experts, bf16): 1024
  // tokens in 64 of 32 x 64 tokens and experts 11.7 us, in 512 of 16 x 16 9.5; 1536
  // 11.9 and 13.0; 128 tokens in 64 of 16 x 16 4.8, in 256 of 8 x 8 3.9; 240 5.0
  // and 5.8
  const long big = (long)((T + 31) / 32) * ((E + 63) / 64);
  const long small = (long)((T + 15) / 16) * ((E + 15) / 16);
  if (big >= 96)
    run<2, 4 / kHalf, 16, 8, 1>(x, w, bias, T, E, H, logits, stream);
  else if (small >= 96)
    run<1, 1, 16, 16, sizeof(XT) == 4 ? 1 : sizeof(WT) == 4 ? 2 : 4>(x, w, bias, T, E, H, logits,
                                                                     stream);
  else
    run<1, 1, 8, 16, sizeof(XT) == 4 ? 2 : 4>(x, w, bias, T, E, H, logits, stream);
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
