// Tokens in expert order and back: dispatch copies every token's row to the places
// that the alignment gave its slots, combine sums the rows of a token's slots with the
// routing weights, and each has its gradient. With at[s] the place of slot s (-1: none)
//   dispatch           rows[at[t,j]] = x[t], zeros in the places that pad a run
//   its gradient       dx[t] = sum_j drows[at[t,j]]: the combine without weights
//   combine            out[t] = sum_j w[t,j] rows[at[t,j]]
//   its gradient       drows[at[t,j]] = w[t,j] dout[t], dw[t,j] = dout[t] . rows[at[t,j]]
//
// Bound by HBM: each kernel reads and writes a row once, 16 bytes to a lane; a wave takes a
// row (or a piece of it), lanes along it, sums in a fixed order in fp32. Measured (captured
// into a graph), 4096 tokens x top-8 x 4096 bf16, runs padded to 128: dispatch 73 us = 5.0
// TB/s, combine 53 us = 5.7 TB/s, its gradient 131 us = 4.9 TB/s (a copy of 1 GiB: 5.1); 16
// tokens: dispatch 2.8 us, combine 2.3.
#include <algorithm>
#include <type_traits>

#include "../../include/moe.h"
#include "moe_common.h"
#include "moe_launch.h"
#include "moe_rows.h"

namespace moe {
namespace dispatch {

using namespace rows;

// Waves of a launch in workgroups of four, these in a grid of kGridX columns (a launch
// counts its threads in 32 bits along a dimension).
constexpr int kGridX = 1 << 20;
__device__ __forceinline__ int my_wave() {
  const int group = blockIdx.y * kGridX + blockIdx.x;
  return __builtin_amdgcn_readfirstlane(group * 4 + (threadIdx.x >> 6));
}
static dim3 grid_of(long waves, int pieces = 1) {
  const long groups = (waves + 3) / 4;
  return dim3((unsigned)std::min<long>(groups, kGridX), (unsigned)((groups + kGridX - 1) / kGridX),
              pieces);
}

// Rows that together pass this are read and written around the caches: they leave nothing
// there that a later kernel would find (the cache before HBM holds 256 MB). 268 MB of rows:
// dispatch 72.7 us instead of 78.9, combine 52.0 instead of 56.9, its gradient 130 instead of
// 140. The host knows T, k and H but not the ids: slots of another shard count as rows too.
constexpr size_t kStreamBytes = (size_t)128 << 20;

// How the rows of a call are copied: in words (U) of 16 bytes; where rows do not start at
// multiples of 16 (ANY) the last of them ends with the row, and copies part of the one before
// it again; rows shorter than that by elements.
template <typename U, bool ANY>
struct Words {
  typedef U Word;
  size_t row;  // bytes
  int count;   // words of a row
  template <typename P>
  __device__ __forceinline__ P* at(P* rows, size_t r) const {
    if constexpr (ANY) return rows + r * row;  // (P: a byte)
    else return rows + r * count;
  }
  __device__ __forceinline__ U load(const U* from, int c) const { return from[c]; }
  __device__ __forceinline__ U load(const uint8_t* from, int c) const {
    return *(const u32x4_any*)(from + min((size_t)c * 16, row - 16));
  }
  template <bool NT>
  __device__ __forceinline__ void store(U* to, int c, U v) const {
    if constexpr (NT) __builtin_nontemporal_store(v, to + c);
    else to[c] = v;
  }
  template <bool NT>
  __device__ __forceinline__ void store(uint8_t* to, int c, U v) const {
    *(u32x4_any*)(to + min((size_t)c * 16, row - 16)) = v;
  }
};
template <bool NT, typename P, typename W>
__device__ __forceinline__ void clear_row(P* to, const W& w) {
  for (int c = threadIdx.x & 63; c < w.count; c += 64)
    w.template store<NT>(to, c, typename W::Word{});
}

// kCopy words of 64 lanes each, those past the row's end its last one.
constexpr int kCopy = 8;
template <typename P, typename W>
__device__ __forceinline__ void load_piece(const P* from, int c0, const W& w,
                                           typename W::Word (&v)[kCopy]) {
#pragma unroll
  for (int i = 0; i < kCopy; ++i) v[i] = w.load(from, min(c0 + i * 64, w.count - 1));
}
template <bool NT, typename P, typename W>
__device__ __forceinline__ void store_piece(P* to, int c0, const W& w,
                                            const typename W::Word (&v)[kCopy]) {
#pragma unroll
  for (int i = 0; i < kCopy; ++i)
    if (c0 + i * 64 < w.count) w.template store<NT>(to, c0 + i * 64, v[i]);
}

struct Lists {
  const int32_t* topk_ids;    // [S]
  const int32_t* sorted_ids;  // [R]
  const int32_t* num_padded;
  int32_t* slot_rows;  // [S]
  int S, E, R;
};

// Dispatch in one launch, place by place: one wave per place (the first R waves), its
// token's row or zeros where it pads a run; then a wave for every 64 slots: -1 for those of
// another shard's experts. Places at and past num_padded are left alone.
template <typename P, typename W>
__global__ __launch_bounds__(256) void places_kernel(const P* __restrict__ x, Lists l, W words,
                                                     int k, P* __restrict__ rows) {
  const int w = my_wave(), lane = threadIdx.x & 63;
  if (w >= l.R) {
    const long s = (long)(w - l.R) * 64 + lane;
    if (s < l.S && (unsigned)l.topk_ids[s] >= (unsigned)l.E) l.slot_rows[s] = -1;
    return;
  }
  if (w >= l.num_padded[0]) return;
  const int slot = __builtin_amdgcn_readfirstlane(l.sorted_ids[w]);
  if ((unsigned)slot >= (unsigned)l.S) {
    clear_row<false>(words.at(rows, w), words);
    return;
  }
  if (lane == 0) l.slot_rows[slot] = w;
  for (int c = lane; c < words.count; c += 64 * kCopy) {
    typename W::Word v[kCopy];
    load_piece(words.at(x, slot / k), c, words, v);
    store_piece<false>(words.at(rows, w), c, words, v);
  }
}

// Dispatch in two launches, token by token: the slots' places first, then each token is
// read once and written to all of its places; behind the tokens' waves a wave for every 8
// places clears those that pad a run. (Place by place a token is read k times, out of the
// cache at best.)
__global__ __launch_bounds__(256) void slots_kernel(Lists l) {
  const long i = (long)blockIdx.x * 256 + threadIdx.x;
  if (i < l.S && (unsigned)l.topk_ids[i] >= (unsigned)l.E) l.slot_rows[i] = -1;
  if (i < l.R && i < l.num_padded[0]) {
    const int slot = l.sorted_ids[i];
    if ((unsigned)slot < (unsigned)l.S) l.slot_rows[slot] = (int)i;
  }
}
template <bool NT, typename P, typename W>
__global__ __launch_bounds__(256) void tokens_kernel(const P* __restrict__ x, Lists l, W words,
                                                     int T, int k, P* __restrict__ rows) {
  const int w = my_wave(), lane = threadIdx.x & 63;
  if (w >= T) {
    const long p0 = (long)(w - T) * 8;
    const int n = (int)min((long)min(l.num_padded[0], l.R) - p0, 8L);
    for (int i = 0; i < n; ++i) {
      const int slot = __builtin_amdgcn_readfirstlane(l.sorted_ids[p0 + i]);
      if ((unsigned)slot >= (unsigned)l.S) clear_row<NT>(words.at(rows, p0 + i), words);
    }
    return;
  }
  // The lanes go on together, those past the row's end too: each brings a slot's place.
  for (int c0 = 0; c0 < words.count; c0 += 64 * kCopy) {
    const int c = c0 + lane;
    typename W::Word v[kCopy];
    load_piece(words.at(x, w), c, words, v);
    for (int j0 = 0; j0 < k; j0 += 64) {
      const int at = j0 + lane < k ? l.slot_rows[(size_t)w * k + j0 + lane] : -1;
      for (uint64_t left = __ballot((unsigned)at < (unsigned)l.R); left; left &= left - 1) {
        const int row = __builtin_amdgcn_readlane(at, __builtin_ctzll(left));
        store_piece<NT>(words.at(rows, row), c, words, v);
      }
    }
  }
}

// The combine, and without weights the dispatch's gradient: the sum over a token's slots, 64 at
// a time, lane l holding slot l's place and weight. A wave takes 64 vectors of a token's row,
// the last of which ends with the row (ANY: it may sum some of the one before it again);
// slots without a place are not read.
constexpr int kBatch = 8;
template <int VEC, bool ANY, bool NT, bool WEIGHTED, typename YT, typename IO>
__global__ __launch_bounds__(256) void combine_kernel(const YT* __restrict__ y,
                                                      const int32_t* __restrict__ slot_rows,
                                                      const float* __restrict__ weights, int T,
                                                      int H, int k, int R, int pieces,
                                                      IO* __restrict__ out) {
  const int w = my_wave(), lane = threadIdx.x & 63;
  const int t = w / pieces, c = ((w - t * pieces) * 64 + lane) * VEC, col = min(c, H - VEC);
  if (t >= T) return;
  float v[VEC] = {};
  for (int j0 = 0; j0 < k; j0 += 64) {
    const int j = j0 + lane;
    int at = -1;
    float wl = 1.f;
    if (j < k) {
      at = slot_rows[(size_t)t * k + j];
      if (WEIGHTED) wl = weights[(size_t)t * k + j];
    }
    uint64_t left = __ballot((unsigned)at < (unsigned)R);
    while (left) {
      // where fewer than kBatch are left the last one again, its values and weight as zeros
      int row[kBatch], some = 0;
      uint32_t keep[kBatch];
      float wj[kBatch];
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        keep[q] = left ? ~0u : 0u;
        if (left) some = __builtin_ctzll(left);
        left &= left - 1;
        row[q] = __builtin_amdgcn_readlane(at, some);
        wj[q] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_int(wl), some) & keep[q]);
      }
      Vec<YT, VEC> r[kBatch];
#pragma unroll
      for (int q = 0; q < kBatch; ++q)
        r[q] = load_vec<YT, VEC, NT, ANY>(y + (size_t)row[q] * H + col);
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        keep_vec<YT, VEC>(r[q], keep[q]);
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] += wj[q] * elem<YT, VEC>(r[q], e);
      }
    }
  }
  if (c < H) store_vec<IO, VEC, false, ANY>(out + (size_t)t * H + col, v);
}

// The combine's gradient. One wave per slot (the first S waves): its row of the gradient and its
// weight's, the dot product of the token's gradient with the row; then a wave for every 8
// places: zeros in those that pad a run. kPiece: vectors of a lane in flight.
template <int VEC, bool ANY, int kPiece, bool NT, typename YT, typename IO>
__global__ __launch_bounds__(256) void combine_backward_kernel(CombineBackwardProblem p) {
  const int w = my_wave(), lane = threadIdx.x & 63, S = p.T * p.k;
  if (w >= S) {
    const long p0 = (long)(w - S) * 8;
    const int n = (int)min((long)min(p.num_padded[0], p.R) - p0, 8L);
    for (int i = 0; i < n; ++i) {
      const int slot = __builtin_amdgcn_readfirstlane(p.sorted_ids[p0 + i]);
      if ((unsigned)slot < (unsigned)S) continue;
      const float zero[VEC] = {};
      YT* to = (YT*)p.drows + (size_t)(p0 + i) * p.H;
      for (int c = lane * VEC; c < p.H; c += 64 * VEC)
        store_vec<YT, VEC, NT, ANY>(to + min(c, p.H - VEC), zero);
    }
    return;
  }
  const int at = __builtin_amdgcn_readfirstlane(p.slot_rows[w]);
  if ((unsigned)at >= (unsigned)p.R) {
    if (lane == 0 && p.dweights) p.dweights[w] = 0.f;
    return;
  }
  const float wt = p.topk_weights ? p.topk_weights[w] : 1.f;
  const IO* g = (const IO*)p.dout + (size_t)(w / p.k) * p.H;
  const YT* y = (const YT*)p.rows + (size_t)at * p.H;
  YT* dy = (YT*)p.drows + (size_t)at * p.H;
  float dot = 0.f;
  for (int c0 = lane * VEC; c0 < p.H; c0 += 64 * VEC * kPiece) {
    Vec<IO, VEC> gv[kPiece];
    Vec<YT, VEC> yv[kPiece];
#pragma unroll
    for (int i = 0; i < kPiece; ++i) {
      const int at = min(c0 + i * 64 * VEC, p.H - VEC);
      gv[i] = load_vec<IO, VEC, false, ANY>(g + at);
      if (p.dweights) yv[i] = load_vec<YT, VEC, NT, ANY>(y + at);
    }
#pragma unroll
    for (int i = 0; i < kPiece; ++i) {
      const int c = c0 + i * 64 * VEC, at = min(c, p.H - VEC);
      if (c >= p.H) break;
      if (p.dweights) {
        // the last vector's first elements may be those of the one before it, whose lane has
        // counted them (and, in place, may have written their gradient by now)
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if (!ANY || at + e >= c) dot += elem<IO, VEC>(gv[i], e) * elem<YT, VEC>(yv[i], e);
      }
      float d[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) d[e] = wt * elem<IO, VEC>(gv[i], e);
      store_vec<YT, VEC, NT, ANY>(dy + at, d);
    }
  }
  dot = wave_sum(dot);
  if (lane == 0 && p.dweights) p.dweights[w] = dot;
}

template <int V>
struct Int {
  static constexpr int value = V;
};

template <int VEC, bool ANY, typename YT, typename IO>
static void run_combine(const CombineProblem& p, hipStream_t stream) {
  const int pieces = (p.H + 64 * VEC - 1) / (64 * VEC);
  const dim3 grid = grid_of((long)p.T * pieces);
  constexpr bool kStream = VEC > 1 && !ANY;
  auto run = [&](auto nt, auto weighted) {
    combine_kernel<VEC, ANY, decltype(nt)::value, decltype(weighted)::value>
        <<<grid, 256, 0, stream>>>((const YT*)p.rows, p.slot_rows, p.topk_weights, p.T, p.H, p.k,
                                   p.R, pieces, (IO*)p.out);
  };
  const bool nt = kStream && (size_t)p.T * p.k * p.H * sizeof(YT) > kStreamBytes;
  if (p.topk_weights) nt ? run(Int<kStream>{}, Int<1>{}) : run(Int<0>{}, Int<1>{});
  else nt ? run(Int<kStream>{}, Int<0>{}) : run(Int<0>{}, Int<0>{});
}

template <int VEC, bool ANY, typename YT, typename IO>
static void run_combine_backward(const CombineBackwardProblem& p, hipStream_t stream) {
  const dim3 grid = grid_of((long)p.T * p.k + (p.R + 7) / 8);
  // Eight vectors of a lane in flight for rows of more than four a lane: 32768 rows of 4096
  // bf16 129.7 us instead of 135.4 with two; 2250 rows of 2048 bf16 8.9 instead of 8.4. Shorter
  // rows also where they pass kStreamBytes: 131072 of 1024 bf16 115.9 us instead of 146.8 with
  // eight around the caches (65536 of 2048, the longest with two, 118.9 and 116.4).
  constexpr bool kStream = VEC > 1 && !ANY;
  const bool nt = kStream && (size_t)p.T * p.k * p.H * sizeof(YT) > kStreamBytes;
  if (p.H <= 256 * VEC)
    combine_backward_kernel<VEC, ANY, 2, false, YT, IO><<<grid, 256, 0, stream>>>(p);
  else if (nt)
    combine_backward_kernel<VEC, ANY, 8, kStream, YT, IO><<<grid, 256, 0, stream>>>(p);
  else
    combine_backward_kernel<VEC, ANY, 8, false, YT, IO><<<grid, 256, 0, stream>>>(p);
}

// Calls f(VEC, ANY, rows' type, tokens' type) for the types of a call: 16 bytes of the
// narrower type to a lane, ANY where a row of either does not start at a multiple of 16; rows
// shorter than that element by element.
template <typename F>
static void by_type(int rows_dtype, int dtype, int H, bool aligned, F f) {
  const uint16_t b = 0;
  const float s = 0;
  const bool rb = rows_dtype == MOE_DTYPE_BF16, tb = dtype == MOE_DTYPE_BF16;
  auto go = [&](auto vec, auto y, auto io) {
    constexpr int VEC = decltype(vec)::value;
    if (H < VEC) f(Int<1>{}, Int<0>{}, y, io);
    else if (aligned && H % VEC == 0) f(vec, Int<0>{}, y, io);
    else f(vec, Int<1>{}, y, io);
  };
  if (rb && tb) go(Int<8>{}, b, b);
  else if (rb) go(Int<8>{}, b, s);
  else if (tb) go(Int<8>{}, s, b);
  else go(Int<4>{}, s, s);
}

static bool aligned16(std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if ((uintptr_t)p % 16) return false;
  return true;
}

}  // namespace dispatch

hipError_t launch_dispatch(const DispatchProblem& p, hipStream_t stream) {
  using namespace dispatch;
  const int bytes = p.dtype == MOE_DTYPE_BF16 ? 2 : 4;
  const Lists l{p.topk_ids, p.sorted_ids, p.num_padded, p.slot_rows, p.T * p.k, p.E, p.R};
  // Token by token from kTokenBytes on (all slots counted, as above): the second launch costs
  // 3 us. 65 MB of rows 20.7 us instead of 21.4, 59 MB 17.7 instead of 18.4; 268 MB 78.9
  // instead of 90.8; 15 MB 10.5 instead of 7.1.
  constexpr size_t kTokenBytes = (size_t)64 << 20;
  const size_t all = (size_t)l.S * p.H * bytes;
  // P: what the kernels count rows' addresses in
  auto run = [&](auto* p0, auto words) {
    typedef std::remove_pointer_t<decltype(p0)> P;
    words.row = (size_t)p.H * bytes;
    words.count = (int)((words.row + sizeof(typename decltype(words)::Word) - 1) /
                        sizeof(typename decltype(words)::Word));
    const P* x = (const P*)p.x;
    P* rows = (P*)p.rows;
    if (all < kTokenBytes) {
      places_kernel<<<grid_of((long)p.R + (l.S + 63) / 64), 256, 0, stream>>>(x, l, words, p.k,
                                                                             rows);
      return;
    }
    slots_kernel<<<(unsigned)((std::max(l.S, l.R) + 255L) / 256), 256, 0, stream>>>(l);
    const dim3 grid = grid_of((long)p.T + (p.R + 7) / 8);
    if (all > kStreamBytes)
      tokens_kernel<true><<<grid, 256, 0, stream>>>(x, l, words, p.T, p.k, rows);
    else
      tokens_kernel<false><<<grid, 256, 0, stream>>>(x, l, words, p.T, p.k, rows);
  };
  if ((size_t)p.H * bytes % 16 == 0 && aligned16({p.x, p.rows}))
    run((u32x4*)nullptr, Words<u32x4, false>{});
  else if (p.H * bytes >= 16) run((uint8_t*)nullptr, Words<u32x4, true>{});
  else if (bytes == 4) run((uint32_t*)nullptr, Words<uint32_t, false>{});
  else run((uint16_t*)nullptr, Words<uint16_t, false>{});
  return hipGetLastError();
}

hipError_t launch_combine(const CombineProblem& p, hipStream_t stream) {
  using namespace dispatch;
  by_type(p.rows_dtype, p.dtype, p.H, aligned16({p.rows, p.out}),
          [&](auto v, auto any, auto y, auto io) {
            run_combine<decltype(v)::value, decltype(any)::value != 0, decltype(y), decltype(io)>(
                p, stream);
          });
  return hipGetLastError();
}

hipError_t launch_combine_backward(const CombineBackwardProblem& p, hipStream_t stream) {
  using namespace dispatch;
  by_type(p.rows_dtype, p.dtype, p.H, aligned16({p.dout, p.rows, p.drows}),
          [&](auto v, auto any, auto y, auto io) {
            run_combine_backward<decltype(v)::value, decltype(any)::value != 0, decltype(y),
                                 decltype(io)>(p, stream);
          });
  return hipGetLastError();
}

}  // namespace moe
