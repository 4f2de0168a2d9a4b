// Matrix product with its epilogue: out = residual + act(x w^T + bias), or gated
// residual + act(x wg^T + bg) (x wu^T + bu), on the bf16 matrix cores with fp32 sums; fp32
// operands enter exactly, as three bf16 planes each, of whose nine products six are taken (the
// other three are 2^-24 of the whole). (The fp32 matrix instructions run at a sixteenth of the
// bf16 rate, and are no closer: both round as a chain of K additions does, 17 to 18 u rms at
// K = 4096.)
//
// Few rows of x: K over the waves of a workgroup, which streams its w rows from HBM. Else
// tiles of 32 NI w rows x 64 MI x rows, with K in parts over workgroups and a second kernel
// that joins them where there are few tiles. Past the operands' ends (rows, and the last
// stage's columns past K) a load's offset lies outside its buffer and gives zeros.
//
// Measured (captured into a graph), bf16: 16 rows x gated 2048 x 7168 11.4 us = 5.2 TB/s of
// weights, 1 x 4096 x 4096 7.1 us; 509 x 4100 x 4096 with gelu 29 us = 586 TFLOP/s (132 tiles of 256
// CUs); 4096 x 7168 x 4096 187 us = 1286 TFLOP/s, with bias and residual 200-208 us; 8192^3 1397-1430
// TFLOP/s (the vendor library's plain product 1478-1550), where the chip's power and the LDS
// (256 KB through it for 2048 cycles of products a stage) are the bounds. fp32: 16 x 4096 x
// 4096 16 us = 4.1 TB/s, 2048 x 4096 x 4096 296-307 us = 224-232 TFLOP/s of the 420 that six
// products leave.
#include <algorithm>
#include <type_traits>

#include "../../include/moe.h"
#include "moe_common.h"
#include "moe_launch.h"
#include "moe_skinny.h"

namespace moe {
namespace linear {

typedef __attribute__((address_space(3))) void* lds_ptr_t;
constexpr int kRsrcWord3 = 0x00020000;     // raw buffer, 32-bit data format
// A tile's rows lie within 2^31 bytes (256 rows of less than 2^23); a lane whose offset
// starts at kOOB is past them whatever row of the tile is added: zeros, no memory read.
constexpr uint32_t kOOB = 0x80000000u;
constexpr int kLds = 160 * 1024;

__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ const uint8_t* uni_ptr(const uint8_t* v) {
  const uint64_t a = (uint64_t)v;
  return (const uint8_t*)(((uint64_t)(uint32_t)uni((int)(a >> 32)) << 32) |
                          (uint32_t)uni((int)(uint32_t)a));
}

// Waits until at most VM vector loads of this wave are in flight (and, LGKM = 0, no LDS read).
template <int VM, int LGKM = 15>
__device__ __forceinline__ void wait_loads() {
  static_assert(VM >= 0 && VM < 64, "vmcnt");
  __builtin_amdgcn_s_waitcnt((VM & 15) | ((VM >> 4) << 14) | (0x7 << 4) | (LGKM << 8));
}
__device__ __forceinline__ void ring_barrier() {
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_barrier();
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// ---------------------------------------------------------- epilogue ---

// With the hardware's exp2 and reciprocal, an ulp each; the product in exp2's argument is
// off by |v| u, which counts for nothing where v is large: v exp(-|v|) is small there.
__device__ __forceinline__ float exp_of(float v) {
  return __builtin_amdgcn_exp2f(v * 1.44269504088896341f);
}
__device__ __forceinline__ float logistic(float v) {
  return __builtin_amdgcn_rcpf(1.0f + exp_of(-v));
}
// v times the normal distribution at v. Its tail at x = |v| / sqrt 2 is erfc(x) / 2 = t P(1 - t)
// exp(-x^2), t = 1 / (1 + 0.49 x), with P of degree 8 fitted to what that leaves of erfc
// for the least relative error, 2.3e-8 (0.4 u) for x to 9.4, where exp(-x^2) ends. In 1 - t, so
// that its terms do not cancel near 0: the tail is off by (20 + v^2) u of itself at most, 7 of
// them t's steps, and for |v| < 1 the result by 3.1 u of v at most, 0.6 u rms. (A polynomial of
// degree 5 in t that holds to an absolute 1.5e-7: 5.5 u and 1.2 u, and 0.2 % of the tail at 4;
// 4096 x 7168 x 4096 with gelu 208.7 us instead of 210.3.)
__device__ __forceinline__ float gelu(float v) {
  const float t = __builtin_amdgcn_rcpf(1.0f + 0.34648232278141387f * fabsf(v));
  const float s = 1.0f - t;
  float p = 0.084097139533734436f + s * -0.028645332902669907f;
  p = -0.053465139120817184f + s * p;
  p = -0.020093560218811035f + s * p;
  p = -0.069017730653285980f + s * p;
  p = 0.097168847918510437f + s * p;
  p = 0.279573887586593628f + s * p;
  p = -0.651405036449432373f + s * p;
  p = 0.5f + s * p;
  const float tail = t * p * __builtin_amdgcn_exp2f(v * (v * -0.72134752044448170f));
  return v * (v < 0.f ? tail : 1.0f - tail);
}
// The activation of all of a lane's values in one branch, not one a value: what is executed
// of the epilogue is straight code of a few lines (jumps from value to value, each to a line
// that the instruction cache does not hold yet, took 14 us of every workgroup).
template <int N>
__device__ __forceinline__ void activate(int act, f32x4 (&v)[N]) {
  auto each = [&](auto f) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) v[i][q] = f(v[i][q]);
  };
  if (act == MOE_ACT_NONE) return;
  if (act == MOE_ACT_RELU)
    each([](float x) { return x < 0.f ? 0.f : x; });  // a NaN stays
  else if (act == MOE_ACT_SILU)
    each([](float x) { return x * logistic(x); });
  else if (act == MOE_ACT_GELU)
    each([](float x) { return gelu(x); });
  else  // (1 + tanh z) / 2 is the logistic function of 2 z
    each([](float x) {
      return x * logistic(x * (1.5957691216057307f + 0.071354816272600251f * x * x));
    });
}

// Four consecutive values of out or residual as they are in memory, where they need not start
// at a multiple of more than their type.
template <typename OT>
struct Four {
  typedef u32x2 type;
  typedef type any __attribute__((aligned(2)));
};
template <>
struct Four<float> {
  typedef f32x4 type;
  typedef type any __attribute__((aligned(4)));
};
__device__ __forceinline__ f32x4 value(const u32x2& r) {
  return f32x4{__uint_as_float(r[0] << 16), __uint_as_float(r[0] & 0xffff0000u),
               __uint_as_float(r[1] << 16), __uint_as_float(r[1] & 0xffff0000u)};
}
__device__ __forceinline__ f32x4 value(const f32x4& r) { return r; }
__device__ __forceinline__ void store_four(uint16_t* p, f32x4 v) {
  *(Four<uint16_t>::any*)p = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
}
__device__ __forceinline__ void store_four(float* p, f32x4 v) { *(Four<float>::any*)p = v; }
__device__ __forceinline__ float load_one(const uint16_t* p) { return bf16_bits_to_f32(*p); }
__device__ __forceinline__ float load_one(const float* p) { return *p; }
__device__ __forceinline__ void store_one(uint16_t* p, float v) { *p = (uint16_t)pack_bf16(v, v); }
__device__ __forceinline__ void store_one(float* p, float v) { *p = v; }

// Four columns n .. n + 3 < N of some rows: their biases once, then row by row.
template <bool GATED, typename OT>
struct Columns {
  int n;
  bool whole;  // N cuts none of the fours of the wave, nor is it less than four
  f32x4 bias, up_bias;

  __device__ __forceinline__ Columns(const LinearProblem& p, int n)
      : n(n), whole(p.N >= 4 && __ballot(n < p.N && n + 4 > p.N) == 0), bias{}, up_bias{} {
    if (!p.bias || n >= p.N) return;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int c = min(n + q, p.N - 1);
      bias[q] = p.bias[c];
      if (GATED) up_bias[q] = p.bias[p.N + c];
    }
  }
  // The sums of a part of K as they are: [part, T, columns of w rounded up to fours] fp32.
  template <int R, typename F>
  __device__ __forceinline__ void store_sums(const LinearProblem& p, F m, const f32x4 (&v)[R],
                                             const f32x4 (&up)[R]) const {
    const size_t fours = (p.N + 3) / 4 * (GATED ? 2 : 1);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (m(i) >= p.T || n >= p.N) continue;
      f32x4* to = (f32x4*)p.workspace + ((size_t)blockIdx.y * p.T + m(i)) * fours + n / 4;
      *to = v[i];
      if (GATED) to[fours / 2] = up[i];
    }
  }
  // What residual holds of rows m(i), ahead of their sums: loads that nothing waits for yet
  // (those past the ends from inside, never used). Only where the fours are whole.
  template <int R, typename F>
  __device__ __forceinline__ void fetch(const LinearProblem& p, F m,
                                        typename Four<OT>::type (&raw)[R]) const {
    if (!p.residual || !whole) return;
#pragma unroll
    for (int i = 0; i < R; ++i)
      raw[i] = *(const typename Four<OT>::any*)((const OT*)p.residual +
                                                (size_t)min(m(i), p.T - 1) * p.ldr +
                                                min(n, p.N - 4));
  }
  // Rows m(i) of them from their sums (and, gated, those of the up rows) and what fetch has
  // brought. m(i) >= T: none.
  template <int R, typename F>
  __device__ __forceinline__ void store(const LinearProblem& p, F m, f32x4 (&v)[R],
                                        const f32x4 (&up)[R],
                                        const typename Four<OT>::type (&raw)[R]) const {
#pragma unroll
    for (int i = 0; i < R; ++i) v[i] += bias;
    activate(p.activation, v);
    if (GATED) {
#pragma unroll
      for (int i = 0; i < R; ++i) v[i] *= up[i] + up_bias;
    }
    if (whole) {
      if (p.residual) {
#pragma unroll
        for (int i = 0; i < R; ++i) v[i] += value(raw[i]);
      }
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (m(i) < p.T && n < p.N) store_four((OT*)p.out + (size_t)m(i) * p.ldo + n, v[i]);
      return;
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (m(i) >= p.T) continue;
      OT* out = (OT*)p.out + (size_t)m(i) * p.ldo + n;
      const OT* res = (const OT*)p.residual + (size_t)m(i) * p.ldr + n;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (n + q < p.N) store_one(out + q, p.residual ? load_one(res + q) + v[i][q] : v[i][q]);
    }
  }
};

// -------------------------------------------------------------- tiles ---

// A workgroup of 8 waves, two along the w rows and four along the x rows, each 16 NI w rows x
// 16 MI x rows.
constexpr int kWaves = 8;

// Row in LDS of row r of w tile i of the waves wn. Gated: tile after tile, gate rows in the
// even ones and their up rows in the odd. Else row r of tile i of a pair lies at (r / 4) 8 +
// 4 (i odd) + r % 4 of the pair's 32, so that a lane's eight sums of a pair are those of
// eight consecutive rows.
template <int NI, bool GATED>
__device__ __forceinline__ int w_row(int wn, int i, int r) {
  if (GATED) return (wn * NI + i) * 16 + r;
  return (wn * (NI / 2) + (i >> 1)) * 32 + (r >> 2) * 8 + (i & 1) * 4 + (r & 3);
}
// The row of w (from the tile's first, gated: of gate or of up rows) at row r of LDS.
template <bool GATED>
__device__ __forceinline__ int w_at(int r) {
  return GATED ? (r >> 5) * 16 + (r & 15) : r;
}
template <bool GATED>
__device__ __forceinline__ bool w_up(int r) {
  return GATED && (r & 16);
}
// Column (16 bytes) c of a row lies at column c ^ key in LDS, so that eight lanes of a read,
// one column of eight rows (of x, and gated of w, in a row; else two times four, eight
// apart), meet the eight columns of 128 bytes: one row, or two of BYTES = 64.
template <int BYTES, bool PAIRS>
__device__ __forceinline__ int key_of(int row) {
  const int r = PAIRS ? (row & 3) | ((row >> 1) & 4) : row & 7;
  return BYTES == 128 ? r : r >> 1;
}

// Workgroups go round the 8 XCDs: the b-th gets a tile of its XCD's share, a run of
// consecutive tiles (shares differ by one at most).
__device__ __forceinline__ int xcd_order(int b, int tiles) {
  const int per = tiles >> 3, rest = tiles & 7, q = b & 7;
  return q * per + min(q, rest) + (b >> 3);
}
// Tiles run down panels of kPanel columns, row by row: consecutive tiles share the rows of w
// and x that an XCD's L2 then holds (8192^3: 1249 TFLOP/s, with panels of 4 1204, of 16 1183).
constexpr int kPanel = 8;
__device__ __forceinline__ void panel(int t, int m_tiles, int n_tiles, int& m, int& n) {
  const int q = t / (kPanel * m_tiles), in = t - q * kPanel * m_tiles;
  const int wide = min(kPanel, n_tiles - q * kPanel);
  m = in / wide;
  n = q * kPanel + in - m * wide;
}

// What a workgroup works on: its tile, its part of K (blockIdx.y of gridDim.y) in stages of
// 128 bytes of every row.
constexpr int kRowBytes = 128;
template <int MI, int NI, bool GATED, typename T>
struct Tile {
  static constexpr int kRowsW = 32 * NI, kRowsX = 64 * MI;
  static constexpr int kCols = GATED ? kRowsW / 2 : kRowsW;  // outputs of a row
  static_assert(NI % 2 == 0, "pairs of tiles");
  int wave, lane, wn, wm, m0, n0, first, stages;
  int bytes;              // of K from its first stage on
  uint32_t wstep, xstep;  // bytes from row to row

  __device__ __forceinline__ Tile(const LinearProblem& p, int n_tiles)
      : wave(uni(threadIdx.x >> 6)), lane(threadIdx.x & 63), wn(wave & 1), wm(wave >> 1) {
    int tile_m, tile_n;
    panel(xcd_order(blockIdx.x, gridDim.x), gridDim.x / n_tiles, n_tiles, tile_m, tile_n);
    m0 = tile_m * kRowsX;
    n0 = tile_n * kCols;
    const int row = p.K * (int)sizeof(T), all = (row + kRowBytes - 1) / kRowBytes;
    first = (int)((long)all * blockIdx.y / gridDim.y);
    stages = (int)((long)all * (blockIdx.y + 1) / gridDim.y) - first;
    bytes = min(row - first * kRowBytes, stages * kRowBytes);
    wstep = (uint32_t)p.K * sizeof(T);
    xstep = (uint32_t)p.ldx * sizeof(T);
  }
  // The tile's first row of w (or of the up rows) and of x, at the part's first stage, and the
  // bytes from there to the end of a stage of the last row that is there (of the row itself
  // where a stage is longer: rows that follow are not there).
  __device__ __forceinline__ const uint8_t* w(const LinearProblem& p, bool up) const {
    return uni_ptr((const uint8_t*)p.w + (size_t)(n0 + (up ? p.N : 0)) * wstep +
                   (size_t)first * kRowBytes);
  }
  __device__ __forceinline__ const uint8_t* x(const LinearProblem& p) const {
    return uni_ptr((const uint8_t*)p.x + (size_t)m0 * xstep + (size_t)first * kRowBytes);
  }
  __device__ __forceinline__ uint32_t w_size(const LinearProblem& p) const {
    return uni((min(kCols, p.N - n0) - 1) * wstep + min(kRowBytes, bytes));
  }
  __device__ __forceinline__ uint32_t x_size(const LinearProblem& p) const {
    return uni((min(kRowsX, p.T - m0) - 1) * xstep + min(kRowBytes, bytes));
  }
};

// A product added in place, where it stands: the reads and loads of the loop are placed
// among the products by hand. (As a builtin the compiler moved them together, and gave sums
// new registers, 184 copies a step with 256 of them to a wave: 1249 TFLOP/s for 8192^3
// instead of 1331.) It knows nothing of the matrix instruction in here: what writes the sums
// before the first and reads them after the last goes through settle(), and the operands are
// registers that LDS reads fill. A vector instruction that wrote one would have to be two states
// ahead: the compiled loops have none, which tests/test_compiled_linear_cpu.py checks in the
// library as built.
__device__ __forceinline__ void mfma_in_place(f32x4& acc, const u32x4& a, const u32x4& b) {
  asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
}
// Orders everything else that touches the sums before or after the products, by more than
// the 16 wait states that a product's registers may need.
template <int I, int NI, int MI>
__device__ __forceinline__ void settle(f32x4 (&acc)[NI][MI]) {
  if constexpr (I == 0) asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
  if constexpr (I < NI) {
#pragma unroll
    for (int j = 0; j < MI; ++j) asm volatile("" : "+a"(acc[I][j]));
    settle<I + 1>(acc);
  }
}

// bf16: direct-to-LDS loads fill a ring of stages, two steps of 32 k each. A load takes 8 rows
// and the waves' loads 64; every wave has the same number of them, so that what is in flight
// is known.
template <int MI, int NI, bool GATED>
struct Sums16 {
  typedef Tile<MI, NI, GATED, uint16_t> Where;
  static constexpr int kLoadsW = Where::kRowsW / 64, kLoadsX = Where::kRowsX / 64;
  static constexpr int kLoads = kLoadsW + kLoadsX;
  static constexpr int kStage = (Where::kRowsW + Where::kRowsX) * kRowBytes;
  static constexpr int kStages = kLds / kStage < 5 ? kLds / kStage : 5;
  static constexpr int kLdsBytes = kStages * kStage;

  static __device__ __forceinline__ void run(const LinearProblem& p, const Where& t, uint8_t* lds,
                                             f32x4 (&acc)[NI][MI]) {
    // This wave's loads: lane l the 16 bytes that belong at column l % 8 of row l / 8, from the
    // rows of the tile that are there (a buffer of that size). Few registers for them: the sums
    // and two steps' operands take nearly all that a wave has.
    const int lane = t.lane, row = t.wave * 8 + (lane >> 3);  // of the first load of w and of x
    const uint8_t* wbase = t.w(p, w_up<GATED>(t.wave * 8));   // (rows 64 on are alike)
    const uint8_t* xbase = t.x(p);
    const uint32_t wsize = t.w_size(p), xsize = t.x_size(p);
    const int wcol = ((lane & 7) ^ key_of<128, !GATED>(row)) * 16;
    const int xcol = ((lane & 7) ^ key_of<128, false>(row)) * 16;
    const uint32_t woff = w_at<GATED>(row) * t.wstep + wcol, xoff = row * t.xstep + xcol;
    const uint32_t wnext = w_at<GATED>(64) * t.wstep, xnext = 64 * t.xstep;
    // the i-th load of stage c; past the last stage all zeros
    auto issue = [&](int i, int c, int slot) __attribute__((always_inline)) {
      const int left = t.bytes - c * kRowBytes;  // bytes of K from this stage on
      const bool is_w = i < kLoadsW;
      const int q = is_w ? i : i - kLoadsW;
      const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
          (void*)((is_w ? wbase : xbase) + (size_t)c * kRowBytes), (short)0,
          (int)(is_w ? wsize : xsize), kRsrcWord3);
      const uint32_t o = (is_w ? wcol : xcol) < left ? (is_w ? woff : xoff) : kOOB;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rs,
          (lds_ptr_t)(lds + slot * kStage +
                      ((is_w ? 0 : Where::kRowsW) + q * 64 + t.wave * 8) * kRowBytes),
          16, (int)(o + q * (is_w ? wnext : xnext)), 0, 0, 0);
    };
    // operand q of a step (h of the stage): the x tiles', then the w tiles'; lane l the k-group
    // l / 16 of row l % 16
    const int r = lane & 15, g = lane >> 4;
    auto read = [&](u32x4(&wf)[NI], u32x4(&xf)[MI], int q, int slot, int h)
        __attribute__((always_inline)) {
      const uint8_t* at = lds + slot * kStage;
      if (q < MI) {
        const int x = Where::kRowsW + (t.wm * MI + q) * 16 + r;
        xf[q] = *(const u32x4*)(at + x * kRowBytes + (((h * 4 + g) ^ key_of<128, false>(r)) << 4));
      } else {
        const int w = w_row<NI, GATED>(t.wn, q - MI, r);
        wf[q - MI] = *(const u32x4*)(at + w * kRowBytes +
                                     (((h * 4 + g) ^ key_of<128, !GATED>(w)) << 4));
      }
    };
#pragma unroll
    for (int c = 0; c < kStages; ++c)
#pragma unroll
      for (int i = 0; i < kLoads; ++i) issue(i, c, c);
    int slot = 0;
    u32x4 w0[NI], x0[MI], w1[NI], x1[MI];
    // A step's products, with the reads of the next one's operands among the first of them
    // and, in a stage's last step, the loads that fill its slot again. The stage's own
    // operands are all read by then, and the next stage's loads have landed: in this wave
    // where it waits, in all past the barrier.
    auto step = [&](const u32x4(&wa)[NI], const u32x4(&xa)[MI], u32x4(&wb)[NI], u32x4(&xb)[MI],
                    bool last, int c) __attribute__((always_inline)) {
      const int here = slot;
      if (last) {
        wait_loads<(kStages - 2) * kLoads, 0>();
        ring_barrier();
        slot = slot == kStages - 1 ? 0 : slot + 1;
      }
      constexpr int kReads = NI + MI, kMma = NI * MI;
      constexpr int kPer = kMma >= 2 * kReads ? 2 : 1, kGap = kMma >= 2 * kLoads ? 2 : 1;
#pragma unroll
      for (int n = 0; n < kMma || n / kPer < kReads || n / kGap < kLoads; ++n) {
        if (n < kMma) mfma_in_place(acc[n / MI][n % MI], wa[n / MI], xa[n % MI]);
        if (n % kPer == 0 && n / kPer < kReads) read(wb, xb, n / kPer, slot, last ? 0 : 1);
        if (last && n % kGap == kGap - 1 && n / kGap < kLoads)
          issue(n / kGap, c + kStages, here);
      }
    };
    wait_loads<(kStages - 1) * kLoads>();
    ring_barrier();
#pragma unroll
    for (int q = 0; q < NI + MI; ++q) read(w0, x0, q, 0, 0);
    settle<0>(acc);
    for (int c = 0; c < t.stages; ++c) {
      step(w0, x0, w1, x1, false, c);
      step(w1, x1, w0, x0, true, c);
    }
    settle<0>(acc);
  }
};

// Two bf16 in one word, infinities as the largest finite values: as 16-bit numbers the positive
// ones are below that of 0x7f7f, the negative ones (unsigned) below that of 0xff7f. (A NaN too:
// what is left of its float is one.) A clamp of the two floats instead: 1 to 4 % of a product.
__device__ __forceinline__ uint32_t finite_bf16(uint32_t u) {
  typedef short s16x2 __attribute__((ext_vector_type(2)));
  typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
  const s16x2 v =
      __builtin_elementwise_min(__builtin_bit_cast(s16x2, u), s16x2{0x7f7f, 0x7f7f});
  return __builtin_bit_cast(
      uint32_t, __builtin_elementwise_min(__builtin_bit_cast(u16x2, v), u16x2{0xff7f, 0xff7f}));
}
// fp32: 8 floats are three bf16 planes of 8 significant bits each, rounded to nearest, the
// remainder again and what is left, as in skinny::split8: exact, and the products that are left
// out (p + q > 2) add up to 2^-24 of one, of either sign. (Cut off instead of rounded the planes
// all have the value's sign and are twice as large: up to 2^-21 is left out, always towards
// zero, 0.6 u of every product in the mean.) The first plane stops at the largest bf16, so
// that no value is rounded up to an infinity; the second has what is above.
__device__ __forceinline__ void planes8(const u32x4& lo, const u32x4& hi, u32x4 (&out)[3]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a = __uint_as_float(i < 2 ? lo[2 * i] : hi[2 * i - 4]);
    float b = __uint_as_float(i < 2 ? lo[2 * i + 1] : hi[2 * i - 3]);
#pragma unroll
    for (int p = 0; p < 3; ++p) {
      const uint32_t u = p == 0 ? finite_bf16(pack_bf16(a, b)) : pack_bf16(a, b);
      out[p][i] = u;
      a -= __uint_as_float(u << 16);
      b -= __uint_as_float(u & 0xffff0000u);
    }
  }
}

// A stage (32 k) is loaded into registers, split into planes and written to one of two slots
// of LDS, every value once for the whole workgroup; the products of planes p + q <= 2 are
// summed. Two stages are under way in registers while one is multiplied.
template <int MI, int NI, bool GATED>
struct Sums32 {
  typedef Tile<MI, NI, GATED, float> Where;
  static constexpr int kRows = Where::kRowsW + Where::kRowsX;
  static constexpr int kPlane = kRows * 64, kStage = 3 * kPlane, kLdsBytes = 2 * kStage;
  static constexpr int kLoads = kRows / 128;  // of 8 floats a thread, four threads to a row
  static_assert(kRows % 128 == 0 && kLdsBytes <= kLds, "whole loads");
  struct Stage {
    u32x4 v[kLoads][2];
  };

  static __device__ __forceinline__ void run(const LinearProblem& p, const Where& t, uint8_t* lds,
                                             f32x4 (&acc)[NI][MI]) {
    const int lane = t.lane, g4 = lane & 3;
    const uint8_t* base[kLoads];
    uint32_t size[kLoads], off[kLoads];
    int to[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int row0 = i * 128 + t.wave * 16, row = row0 + (lane >> 2);  // 16 rows of one kind
      const bool is_w = row0 < Where::kRowsW;
      const int r = is_w ? w_at<GATED>(row) : row - Where::kRowsW;
      base[i] = is_w ? t.w(p, w_up<GATED>(row0)) : t.x(p);
      size[i] = is_w ? t.w_size(p) : t.x_size(p);
      off[i] = r * (is_w ? t.wstep : t.xstep) + g4 * 32;
      const int key = is_w ? key_of<64, !GATED>(row) : key_of<64, false>(row - Where::kRowsW);
      to[i] = row * 64 + ((g4 ^ key) << 4);
    }
    auto load = [&](Stage& s, int c) __attribute__((always_inline)) {
      const int left = t.bytes - c * kRowBytes;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
            (void*)(base[i] + (size_t)c * kRowBytes), (short)0, (int)size[i], kRsrcWord3);
        const uint32_t o = g4 * 32 < left ? off[i] : kOOB;  // (K a multiple of 8)
        s.v[i][0] = __builtin_amdgcn_raw_buffer_load_b128(rs, (int)o, 0, 0);
        s.v[i][1] = __builtin_amdgcn_raw_buffer_load_b128(rs, (int)o, 16, 0);
      }
    };
    auto split = [&](const Stage& s, int slot) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        u32x4 plane[3];
        planes8(s.v[i][0], s.v[i][1], plane);
#pragma unroll
        for (int q = 0; q < 3; ++q)
          *(u32x4*)(lds + slot * kStage + q * kPlane + to[i]) = plane[q];
      }
    };
    const int r = lane & 15, g = lane >> 4;
    auto operand = [&](int slot, int plane, int row, int key) __attribute__((always_inline)) {
      return __builtin_bit_cast(
          bf16x8,
          *(const u32x4*)(lds + slot * kStage + plane * kPlane + row * 64 + ((g ^ key) << 4)));
    };
    // Stage c: its slot is written in this wave, past the barrier in all; all have read the
    // other slot by then, too, which the next stage goes to.
    auto stage = [&](Stage& s, int c) __attribute__((always_inline)) {
      const int slot = c & 1;
      wait_loads<63, 0>();
      ring_barrier();
      bf16x8 wf[NI][3], xf[MI][3];
#pragma unroll
      for (int q = 0; q < 3; ++q) {
#pragma unroll
        for (int j = 0; j < MI; ++j)
          xf[j][q] = operand(slot, q, Where::kRowsW + (t.wm * MI + j) * 16 + r,
                             key_of<64, false>(r));
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const int row = w_row<NI, GATED>(t.wn, i, r);
          wf[i][q] = operand(slot, q, row, key_of<64, !GATED>(row));
        }
      }
      // (the small tile: not among the operands' reads, for the registers, see tile_kernel)
      if constexpr (MI == 1) __builtin_amdgcn_sched_barrier(0);
      split(s, slot ^ 1);
      load(s, c + 3);
#pragma unroll
      for (int a = 2; a >= 0; --a)
#pragma unroll
        for (int b = 2 - a; b >= 0; --b)
#pragma unroll
          for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int j = 0; j < MI; ++j) acc[i][j] = mfma_bf16(wf[i][a], xf[j][b], acc[i][j]);
    };
    Stage s0, s1;
    load(s0, 0);
    load(s1, 1);
    split(s0, 0);
    load(s0, 2);
    for (int c = 0; c < t.stages; c += 2) {  // (a stage more than there are: zeros)
      stage(s1, c);
      stage(s0, c + 1);
    }
  }
};

// The small fp32 tile (48 KB of LDS) with registers for three workgroups a CU: 128 x 4096 x 4096
// 37.7 us instead of 41.2 with 86 of them, 128 x gated 2048 x 4096 38.7 instead of 40.1.
template <int MI, int NI, bool GATED, typename T, typename OT>
__global__ __launch_bounds__(kWaves * 64, sizeof(T) == 4 && MI == 1 ? 6 : 2) void tile_kernel(
    LinearProblem p, int n_tiles) {
  typedef std::conditional_t<sizeof(T) == 2, Sums16<MI, NI, GATED>, Sums32<MI, NI, GATED>> Sums;
  __shared__ __attribute__((aligned(16))) uint8_t lds[Sums::kLdsBytes];
  const Tile<MI, NI, GATED, T> t(p, n_tiles);
  f32x4 acc[NI][MI];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < MI; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  Sums::run(p, t, lds, acc);

  // A wave's sums, as many of its 16-row tiles at a time as its piece of LDS holds, and back
  // along rows: whole lines of out and residual, and one copy of the epilogue's code.
  constexpr int kCell = 16 * NI * 4 + 16;  // bytes of a row, a column of banks apart
  constexpr int kAt = Sums::kLdsBytes / kWaves / (16 * kCell);
  constexpr int kGroup = kAt >= MI ? MI : kAt >= 2 && MI % 2 == 0 ? 2 : 1;
  constexpr int kFours = GATED ? 2 * NI : 4 * NI;  // of a row's outputs
  constexpr int kRows = 64 / kFours;               // rows at a time, a lane to four columns
  constexpr int kTurns = (kGroup * 16 + kRows - 1) / kRows;
  static_assert(kAt >= 1 && MI % kGroup == 0, "LDS of a wave");
  const int lane = t.lane;
  uint8_t* mine = lds + t.wave * kGroup * 16 * kCell;
  const int row0 = lane / kFours, q = lane - row0 * kFours;
  const Columns<GATED, OT> cols(
      p, row0 < kRows ? t.n0 + t.wn * (GATED ? 8 : 16) * NI + q * 4 : p.N);
  const uint8_t* cell = mine + (GATED ? (q >> 2) * 128 + (q & 3) * 16 : q * 16);
  const int m1 = t.m0 + t.wm * MI * 16 + row0;
  typename Four<OT>::type raw[2][kTurns];
  auto at = [&](int j0, int a) __attribute__((always_inline)) {
    return kGroup * 16 % kRows == 0 || row0 + a * kRows < kGroup * 16 ? m1 + j0 * 16 + a * kRows
                                                                      : p.T;
  };
  const bool whole = gridDim.y == 1;
  wait_loads<0, 0>();  // no load may still write the ring, which the sums go through now
  if (whole) cols.fetch(p, [&](int a) { return at(0, a); }, raw[0]);
  ring_barrier();
#pragma unroll
  for (int j0 = 0; j0 < MI; j0 += kGroup) {
    skinny::wave_lds_order();
#pragma unroll
    for (int j = j0; j < j0 + kGroup; ++j)
#pragma unroll
      for (int i = 0; i < NI; ++i)
        *(f32x4*)(mine + ((j - j0) * 16 + (lane & 15)) * kCell +
                  w_row<NI, GATED>(0, i, (lane >> 4) * 4) * 4) = acc[i][j];
    if (whole && j0 + kGroup < MI)
      cols.fetch(p, [&](int a) { return at(j0 + kGroup, a); }, raw[(j0 / kGroup + 1) & 1]);
    skinny::wave_lds_order();
    f32x4 v[kTurns], up[kTurns];
#pragma unroll
    for (int a = 0; a < kTurns; ++a) {
      const uint8_t* from = cell + min(row0 + a * kRows, kGroup * 16 - 1) * kCell;
      v[a] = *(const f32x4*)from;
      up[a] = GATED ? *(const f32x4*)(from + 64) : f32x4{};
    }
    if (whole)
      cols.store(p, [&](int a) { return at(j0, a); }, v, up, raw[(j0 / kGroup) & 1]);
    else
      cols.store_sums(p, [&](int a) { return at(j0, a); }, v, up);
  }
}

// The parts' sums added in order, and the epilogue: a thread for four columns of a row.
template <bool GATED, typename OT>
__global__ __launch_bounds__(256) void join_kernel(LinearProblem p, int parts) {
  const int fours = (p.N + 3) / 4;
  const long u = (long)blockIdx.x * 256 + threadIdx.x;
  const int m = (int)(u / fours), q = (int)(u - (long)m * fours);
  if (m >= p.T) return;
  const size_t step = (size_t)p.T * fours * (GATED ? 2 : 1);
  const f32x4* from = (const f32x4*)p.workspace + (size_t)m * fours * (GATED ? 2 : 1) + q;
  const Columns<GATED, OT> cols(p, q * 4);
  typename Four<OT>::type raw[1];
  cols.fetch(p, [&](int) { return m; }, raw);
  f32x4 v[1] = {}, up[1] = {};
#pragma unroll 4
  for (int i = 0; i < parts; ++i) {
    v[0] += from[i * step];
    if (GATED) up[0] += from[i * step + fours];
  }
  cols.store(p, [&](int) { return m; }, v, up, raw);
}

// -------------------------------------------------------------- few rows ---

// Up to R MT rows of x: K over the waves of a workgroup (moe_skinny.h), R NT rows of w each:
// gated half of them gate rows, half their up rows. No second launch, no padding to a tile.
// Bound by the stream of w: 58.7 MB in 11.4 us (16 x gated 2048 x 7168), which in tiles with K
// in parts takes 14.5.
template <int MT, int NT, int R, int NW, int D, bool GATED, typename T, typename OT>
__global__ __launch_bounds__(NW * 64) void few_kernel(LinearProblem p) {
  constexpr int kSums = R * MT * R * NT * 4;
  constexpr int kPieces = skinny::lds_bytes<MT, NT, R, NW, T, T>();
  __shared__ __attribute__((aligned(16))) char lds[kPieces + kSums];
  constexpr int kCols = R * NT / (GATED ? 2 : 1);
  const int n0 = blockIdx.x * kCols;
  const int wave = uni(threadIdx.x >> 6);
  skinny::Product<MT, NT, R, T, T> product;
  product.lds = lds + wave * product.kLdsBytes;
  product.x.set([&](int i) { return (const T*)p.x + (size_t)min(i, p.T - 1) * p.ldx; });
  product.w.set([&](int i) {
    const int n = min(n0 + (GATED ? i % kCols : i), p.N - 1);
    return (const T*)p.w + (size_t)(n + (GATED && i >= kCols ? p.N : 0)) * p.K;
  });
  product.clear();
  product.template accumulate<D>(p.K, wave, (p.K + skinny::kChunk - 1) / skinny::kChunk, NW);
  float* sums = (float*)(lds + kPieces);  // [x row][w row]
  skinny::reduce_waves<MT, NT, R, NW>(product.acc, lds, [&](int wr, int xr, auto s) {
    if constexpr (sizeof(s) == 4) sums[xr * R * NT + wr] = s;
    else *(f32x4*)(sums + xr * R * NT + wr) = s;
  });
  __syncthreads();
  for (int u = threadIdx.x; u < R * MT * kCols / 4; u += NW * 64) {
    const int m = u / (kCols / 4), q = u - m * (kCols / 4);
    const float* at = sums + m * R * NT + q * 4;
    f32x4 v[1] = {*(const f32x4*)at}, up[1] = {GATED ? *(const f32x4*)(at + kCols) : f32x4{}};
    const Columns<GATED, OT> cols(p, n0 + q * 4);
    typename Four<OT>::type raw[1];
    cols.fetch(p, [&](int) { return m; }, raw);
    cols.store(p, [&](int) { return m; }, v, up, raw);
  }
}

// ------------------------------------------------------------------ plan ---

template <int MI, int NI, bool GATED, typename T, typename OT>
static void run_tiles(const LinearProblem& p, int parts, hipStream_t stream) {
  typedef Tile<MI, NI, GATED, T> Where;
  const int mt = (p.T + Where::kRowsX - 1) / Where::kRowsX;
  const int nt = (p.N + Where::kCols - 1) / Where::kCols;
  tile_kernel<MI, NI, GATED, T, OT><<<dim3(mt * nt, parts), kWaves * 64, 0, stream>>>(p, nt);
  if (parts > 1) {
    const long fours = (long)p.T * ((p.N + 3) / 4);
    join_kernel<GATED, OT><<<(unsigned)((fours + 255) / 256), 256, 0, stream>>>(p, parts);
  }
}

template <int MT, int NT, int R, int NW, int D, bool GATED, typename T, typename OT>
static void run_few(const LinearProblem& p, hipStream_t stream) {
  const int cols = R * NT / (GATED ? 2 : 1);
  few_kernel<MT, NT, R, NW, D, GATED, T, OT>
      <<<(p.N + cols - 1) / cols, NW * 64, 0, stream>>>(p);
}

template <int V>
struct Int {
  static constexpr int value = V;
};

struct TileCost {
  int mi, ni;
  float fixed, alone, full;  // us: of a tile beside its stages; of a stage, one tile and all CUs
};
// The least of these estimates, in us. Tiles: measured with K 2048 and 4096 on 32 .. 256
// tiles (alone and full), e.g. 512 x 4096 x 4096 1 x 4 23.9 (1 x 2 30.3, 2 x 4 27.3), 1024 rows
// 2 x 4 35.5 (2 x 8 43.8, 1 x 4 46.8), 2048 rows 2 x 8 60.6 (4 x 8 76.1), 4096 rows 4 x 8 102.7
// (2 x 8 117.7), 3000 x 1500 x 2000 2 x 6 28.9 (2 x 8 32.2, 2 x 4 43.0). Parts of K where
// tiles are few: 64 x gated 2048 x 7168 in 4 15.8 (whole 27.0), 700 x 700 x 8192 in 2 21.5 (30.8);
// the joining kernel takes 3.2 and its bytes. Few rows: w streams at 90 GB/s a CU and 7.5 TB/s
// in all, x comes from L2 at 140: 16 x gated 2048 x 7168 11.5 (tiles 14.5), 16 x 4096 x 4096 7.7
// (10.9), 64 x 512 x 512 3.3 (4.7), but 64 x 7168 x 2048 14.5 (10.0). fp32: 2048 x 4096 x 4096 4 x 4
// 306 (2 x 4 340, 1 x 2 434), 256 rows 2 x 4 in 4 53 (1 x 2 67), 300 x 512 x 512 1 x 2 in 4 8.5 (whole
// 10.6), 16 x 4096 x 4096 few rows 15.6 (tiles 27). A CU counts as holding one tile at a time,
// and tiles past 256 as a round more, as measured for the large ones; the small ones' LDS
// leaves room for more (fp32 1 x 2: three, bf16 1 x 2: two), whose rounds were not measured.
static const TileCost kTiles[] = {{1, 2, 3.3f, 0.21f, 0.255f}, {1, 4, 3.8f, 0.24f, 0.31f},
                                  {2, 4, 4.5f, 0.34f, 0.48f},  {2, 6, 5.0f, 0.46f, 0.68f},
                                  {2, 8, 5.5f, 0.57f, 0.86f},  {4, 8, 8.0f, 1.05f, 1.5f}};
static const TileCost kTilesF32[] = {{1, 2, 3.3f, 0.42f, 0.48f}, {2, 4, 4.5f, 0.9f, 1.25f},
                                     {4, 4, 5.5f, 1.6f, 2.3f}};
struct FewCost {
  int mt, nt, r;
  float f32;  // fp32 takes that much longer than its bytes say: fewer waves (0: not at all)
};
static const FewCost kFew[] = {{1, 1, 8, 1.15f}, {1, 1, 16, 1.f}, {1, 2, 16, 0.f},
                               {2, 1, 16, 1.f}, {2, 2, 16, 0.f}, {4, 1, 16, 1.8f}};
constexpr int kCus = 256;

static LinearPlan plan_of(int T, int N, int K, bool gated, int dtype) {
  const bool f32 = dtype == MOE_DTYPE_F32;
  const int size = f32 ? 4 : 2, half = gated ? 2 : 1;
  LinearPlan best{};
  float least = 3.0e38f;
  auto take = [&](float t, const LinearPlan& p) {
    if (t < least) {
      least = t;
      best = p;
    }
  };
  for (const FewCost& f : kFew) {
    if (T > f.mt * f.r || (f32 && f.f32 == 0.f)) continue;
    const int cols = f.nt * f.r / half;
    const long tiles = ((long)N + cols - 1) / cols;
    const float w = 1e-3f * f.nt * f.r * K * size, x = 1e-3f * f.mt * f.r * K * size;  // KB
    const float all = w * std::min<long>(tiles, kCus) / (f32 ? 6000.f : 7500.f);
    const float round = std::max(w / 90.f, all) + x / 140.f;
    take(2.5f + (float)((tiles + kCus - 1) / kCus) * round * (f32 ? f.f32 : 1.f),
         LinearPlan{true, f.mt, f.nt, f.r, 1});
  }
  const int stages = (K * size + 127) / 128;
  auto price = [&](const TileCost& c) {
    const int rows = 64 * c.mi, cols = 32 * c.ni / half;
    const long tiles = ((long)T + rows - 1) / rows * (((long)N + cols - 1) / cols);
    for (int parts = 1; parts <= 16; parts += parts < 4 ? 1 : parts / 2) {
      if (parts > 1 && 2 * parts > stages) break;
      const long groups = tiles * parts, whole = groups / kCus;
      const float part = (float)(groups - whole * kCus) / kCus, n = (stages + parts - 1) / parts;
      float t = 2.5f + whole * (c.fixed - 2.5f + n * c.full);
      if (part > 0) t += c.fixed - 2.5f + n * (c.alone + (c.full - c.alone) * part);
      if (parts > 1) t += 3.2f + 2e-6f * parts * T * ((float)N * half);  // 8 bytes at 4 TB/s
      take(t, LinearPlan{false, c.mi, c.ni, 0, parts});
      if (groups > 2 * kCus) break;  // more parts: more rounds
    }
  };
  if (f32) {
    for (const TileCost& c : kTilesF32) price(c);
  } else {
    for (const TileCost& c : kTiles) price(c);
  }
  return best;
}

template <bool GATED, typename T, typename OT>
static void dispatch(const LinearProblem& p, const LinearPlan& plan, hipStream_t stream) {
  constexpr bool kF32 = sizeof(T) == 4;
  auto tiles = [&](auto mi, auto ni) {
    constexpr int MI = decltype(mi)::value, NI = decltype(ni)::value;
    if (!plan.few && plan.a == MI && plan.b == NI)
      run_tiles<MI, NI, GATED, T, OT>(p, plan.parts, stream);
  };
  // NW waves with D chunks in flight each (fp32: less, for registers and LDS)
  auto few = [&](auto mt, auto nt, auto r, auto nw, auto d) {
    constexpr int MT = decltype(mt)::value, NT = decltype(nt)::value, R = decltype(r)::value;
    if (plan.few && plan.a == MT && plan.b == NT && plan.r == R)
      run_few<MT, NT, R, decltype(nw)::value, decltype(d)::value, GATED, T, OT>(p, stream);
  };
  few(Int<1>{}, Int<1>{}, Int<8>{}, Int<16>{}, Int<kF32 ? 2 : 4>{});
  few(Int<1>{}, Int<1>{}, Int<16>{}, Int<16>{}, Int<kF32 ? 1 : 4>{});
  few(Int<2>{}, Int<1>{}, Int<16>{}, Int<kF32 ? 8 : 16>{}, Int<kF32 ? 1 : 2>{});
  few(Int<4>{}, Int<1>{}, Int<16>{}, Int<kF32 ? 4 : 8>{}, Int<kF32 ? 1 : 2>{});
  if constexpr (!kF32) {
    few(Int<1>{}, Int<2>{}, Int<16>{}, Int<16>{}, Int<2>{});
    few(Int<2>{}, Int<2>{}, Int<16>{}, Int<16>{}, Int<2>{});
  }
  tiles(Int<1>{}, Int<2>{});
  tiles(Int<2>{}, Int<4>{});
  if constexpr (kF32) {
    tiles(Int<4>{}, Int<4>{});
  } else {
    tiles(Int<1>{}, Int<4>{});
    tiles(Int<2>{}, Int<6>{});
    tiles(Int<2>{}, Int<8>{});
    tiles(Int<4>{}, Int<8>{});
  }
}

}  // namespace linear

LinearPlan linear_plan(int T, int N, int K, bool gated, int dtype) {
  return linear::plan_of(T, N, K, gated, dtype);
}

size_t linear_workspace_bytes(const LinearPlan& plan, int T, int N, bool gated) {
  if (plan.few || plan.parts == 1) return 0;
  const size_t n = (size_t)(N + 3) / 4 * 4 * (gated ? 2 : 1);
  return (plan.parts * T * n * sizeof(float) + 255) / 256 * 256;
}

hipError_t launch_linear(const LinearProblem& p, const LinearPlan& plan, hipStream_t stream) {
  using namespace linear;
  const bool b = p.dtype == MOE_DTYPE_BF16, ob = p.out_dtype == MOE_DTYPE_BF16;
  if (p.gated) {
    if (b) ob ? dispatch<true, uint16_t, uint16_t>(p, plan, stream)
              : dispatch<true, uint16_t, float>(p, plan, stream);
    else ob ? dispatch<true, float, uint16_t>(p, plan, stream)
            : dispatch<true, float, float>(p, plan, stream);
  } else {
    if (b) ob ? dispatch<false, uint16_t, uint16_t>(p, plan, stream)
              : dispatch<false, uint16_t, float>(p, plan, stream);
    else ob ? dispatch<false, float, uint16_t>(p, plan, stream)
            : dispatch<false, float, float>(p, plan, stream);
  }
  return hipGetLastError();
}

}  // namespace moe
