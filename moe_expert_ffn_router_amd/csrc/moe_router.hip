// Router projection: logits[t, e] = x[t] . w[e] + bias[e] in fp32, on the matrix
// cores with K split over the waves of a workgroup (moe_skinny.h), so that one
// launch serves a single token as well as a prompt and needs no workspace.
// Bound by what a CU reads: R (MT + NT) rows of x and w per workgroup. Measured
// (captured into a graph): 16 tokens x 64 experts x 4096 bf16 3.4 us, 64 x 128 x
// 7168 with fp32 w 8.4 us (the split of w into planes included), 1024 x 128 x 4096
// 7.3 us, 4096 x 128 x 4096 14.9 us: 786 KB per CU at 63 GB/s, where 32 x 64
// tiles, one per CU, are the largest that fill the chip; with fp32 w 19.6 us.
#include <limits.h>

#include <algorithm>

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
                                                         int E, int H, int t_tiles, int e_tiles,
                                                         float* __restrict__ logits) {
  __shared__ __align__(16) char lds[skinny::lds_bytes<MT, NT, R, NW, XT, WT>()];
  // the expert tiles of one token tile are 8 workgroups apart: on one XCD, whose
  // L2 then serves the token rows to all but the first; those of the last t_tiles % 8
  // token tiles go round the XCDs, which would else have more to do than others (1
  // token, 512 experts x 7168 4.4 us instead of 9.7 on one XCD; 653 x 191 x 7744 12.0
  // instead of 18.9)
  const int even = t_tiles & ~7, b = blockIdx.x, past = b - even * e_tiles;
  const int q = (past < 0 ? b >> 3 : past) / e_tiles;
  const int e_tile = (past < 0 ? b >> 3 : past) - q * e_tiles;
  const int tile = past < 0 ? q * 8 + (b & 7) : even + q;
  const int t0 = tile * MT * R, e0 = e_tile * NT * R;
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
      <<<tt * et, NW * 64, 0, stream>>>(x, w, bias, T, E, H, tt, et, logits);
}

template <typename XT, typename WT>
static void dispatch(const XT* x, const WT* w, const float* bias, int T, int E, int H,
                     float* logits, hipStream_t stream) {
  constexpr bool kX4 = sizeof(XT) == 4, kW4 = sizeof(WT) == 4;
  // fp32 w beside bf16 x: its rows are twice as long and every workgroup splits
  // them into planes, so tiles take half the experts and twice the tokens (4096
  // tokens x 4096, 128 experts 19.6 us instead of 27.5)
  constexpr bool kTall = kW4 && !kX4;
  // The tiles for which a CU reads the least of x and w, the larger where that is
  // the same. x 4096, bf16: 128 experts, 128 tokens 8 x 8 tiles 3.9 us (16 x 16
  // 4.8), 1024 16 x 32 7.3 (16 x 16 9.6), 1536 32 x 32 9.0 (32 x 64 11.9, 16 x 16
  // 13.0); 16384 32 x 64 59.5; 8 experts, 4096 tokens 16 x 16 7.8 (32 x 64 12.9).
  auto bytes = [&](int t, int e) {
    const long tiles = (long)((T + t - 1) / t) * ((E + e - 1) / e);
    return (tiles + 255) / 256 * (t * sizeof(XT) + e * sizeof(WT));
  };
  const long big = kX4 ? LONG_MAX : kTall ? bytes(64, 32) : bytes(32, 64);
  const long square = bytes(32, 32), wide = kTall ? bytes(32, 16) : bytes(16, 32);
  const long mid = bytes(16, 16), small = bytes(8, 8);
  const long least = std::min({big, square, wide, mid, small});
  // with fp32 operands fewer waves or chunks in flight: registers and LDS
  if constexpr (!kX4) {
    if (big == least)
      return run<kTall ? 4 : 2, kTall ? 2 : 4, 16, 8, 1>(x, w, bias, T, E, H, logits, stream);
  }
  if (square == least)
    run<2, 2, 16, kW4 ? 8 : 16, kW4 ? 1 : 2>(x, w, bias, T, E, H, logits, stream);
  else if (wide == least)
    run<kTall ? 2 : 1, kTall ? 1 : 2, 16, kX4 ? 8 : 16, kW4 ? 1 : 2>(x, w, bias, T, E, H, logits,
                                                                     stream);
  else if (mid == least)
    run<1, 1, 16, 16, kX4 ? 1 : kW4 ? 2 : 4>(x, w, bias, T, E, H, logits, stream);
  else
    run<1, 1, 8, 16, kX4 ? 2 : 4>(x, w, bias, T, E, H, logits, stream);
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
