// Matrix product with its epilogue: out = residual + act(x w^T + bias), or gated
// residual + act(x wg^T + bg) (x wu^T + bu), on the bf16 matrix cores with fp32 sums; fp32
// operands enter exactly, as three bf16 planes each of which six products are taken.
// (The fp32 matrix instructions run at a sixteenth of the bf16 rate, and are no closer: both
// round as a chain of K additions does, 17 to 18 u rms at K = 4096.)
//
// Tile kernel: a workgroup of 8 waves (2 along the w rows, 4 along the x rows) makes
// 32 NI w rows x 64 MI x rows, wave by wave 16 NI x 16 MI. 128 bytes of every row (a
// chunk: 64 bf16, 32 fp32) are a stage of a ring in LDS that direct-to-LDS loads fill
// ahead of the chunk in work, one barrier a chunk. Past the operands' ends (rows, and
// the last chunk's columns past K) a load's offset lies outside its buffer and gives
// zeros.
#include <algorithm>

#include "../../include/moe.h"
#include "moe_common.h"
#include "moe_launch.h"
#include "moe_skinny.h"

namespace moe {
namespace linear {

typedef __attribute__((address_space(3))) void* lds_ptr_t;
constexpr int kRsrcWord3 = 0x00020000;     // raw buffer, 32-bit data format
// Offsets of a tile's rows stay below kBufferBytes (255 rows of less than 2^24 bytes); one
// past it, kOOB, gives zeros and reads no memory.
constexpr uint32_t kBufferBytes = 0xFF800000u, kOOB = 0xFFFF0000u;
constexpr int kRowBytes = 128;             // of a row in a stage
constexpr int kWaves = 8, kWavesN = 2, kWavesM = 4;
constexpr int kLds = 160 * 1024;

__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }

template <int VM>
__device__ __forceinline__ void wait_loads() {
  static_assert(VM >= 0 && VM < 64, "vmcnt");
  __builtin_amdgcn_s_waitcnt((VM & 15) | ((VM >> 4) << 14) | (0x7 << 4) | (15 << 8));
}
__device__ __forceinline__ void ring_barrier() {
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_barrier();
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// ---------------------------------------------------------- epilogue ---

__device__ __forceinline__ float activate(int act, float v) {
  switch (act) {
    case MOE_ACT_RELU: return v < 0.f ? 0.f : v;  // a NaN stays
    case MOE_ACT_SILU: return v / (1.0f + expf(-v));
    case MOE_ACT_GELU: return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
    case MOE_ACT_GELU_TANH: {
      // (1 + tanh z) / 2 = 1 / (1 + exp(-2 z))
      const float z = v * (0.79788456080286536f + 0.035677408136300125f * v * v);
      return v / (1.0f + expf(-2.0f * z));
    }
    default: return v;
  }
}

__device__ __forceinline__ float load_one(const uint16_t* p) { return bf16_bits_to_f32(*p); }
__device__ __forceinline__ float load_one(const float* p) { return *p; }
__device__ __forceinline__ void store_one(uint16_t* p, float v) { *p = (uint16_t)pack_bf16(v, v); }
__device__ __forceinline__ void store_one(float* p, float v) { *p = v; }
__device__ __forceinline__ f32x4 load_four(const uint16_t* p) {
  const u32x2 r = *(const u32x2*)p;
  return f32x4{__uint_as_float(r[0] << 16), __uint_as_float(r[0] & 0xffff0000u),
               __uint_as_float(r[1] << 16), __uint_as_float(r[1] & 0xffff0000u)};
}
__device__ __forceinline__ f32x4 load_four(const float* p) { return *(const f32x4*)p; }
__device__ __forceinline__ void store_four(uint16_t* p, f32x4 v) {
  *(u32x2*)p = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
}
__device__ __forceinline__ void store_four(float* p, f32x4 v) { *(f32x4*)p = v; }

// Four columns n .. n + 3 of row m from their sums (and, gated, those of the up rows).
template <bool GATED, typename OT>
__device__ __forceinline__ void finish(const LinearProblem& p, int m, int n, f32x4 v, f32x4 up) {
  if (m >= p.T || n >= p.N) return;
  OT* out = (OT*)p.out + (size_t)m * p.ldo + n;
  const OT* res = p.residual ? (const OT*)p.residual + (size_t)m * p.ldr + n : nullptr;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int c = min(n + q, p.N - 1);
    if (p.bias) {
      v[q] += p.bias[c];
      if (GATED) up[q] += p.bias[p.N + c];
    }
    v[q] = activate(p.activation, v[q]);
    if (GATED) v[q] *= up[q];
  }
  if (p.by_four) {
    if (res) v += load_four(res);
    store_four(out, v);
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (n + q < p.N) store_one(out + q, res ? load_one(res + q) + v[q] : v[q]);
  }
}

// -------------------------------------------------------------- tiles ---

// A lane's share of 32 k of its row: 16 bytes of bf16, 32 of fp32 as three bf16 planes
// whose sum it is (moe_skinny.h).
template <typename T>
struct Frag {
  static constexpr int kPlanes = sizeof(T) == 2 ? 1 : 3;
  bf16x8 plane[kPlanes];

  // step: which 32 of the chunk's k; row, key: the row in LDS and its columns' key
  __device__ __forceinline__ void read(const uint8_t* row, int key, int step) {
    const int g = (threadIdx.x >> 4) & 3;
    if constexpr (sizeof(T) == 2) {
      plane[0] = __builtin_bit_cast(
          bf16x8, *(const u32x4*)(row + (((step * 4 + g) ^ key) << 4)));
    } else {
      const f32x4 a = *(const f32x4*)(row + (((2 * g) ^ key) << 4));
      const f32x4 b = *(const f32x4*)(row + (((2 * g + 1) ^ key) << 4));
      const float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
      skinny::split8<kPlanes>(v, plane);
    }
  }
};
template <typename T>
__device__ __forceinline__ void multiply(f32x4& acc, const Frag<T>& w, const Frag<T>& x) {
#pragma unroll
  for (int a = Frag<T>::kPlanes - 1; a >= 0; --a)
#pragma unroll
    for (int b = Frag<T>::kPlanes - 1; b >= 0; --b)
      if (a + b <= 2) acc = mfma_bf16(w.plane[a], x.plane[b], acc);
}

// Rows of a wave's NI w tiles in LDS. Gated: tile after tile, gate rows in the even ones
// and their up rows in the odd. Else row r of tile i of a pair lies at (r / 4) 8 + 4 (i
// odd) + r % 4 of the pair's 32, so that a lane's eight sums of a pair are those of eight
// consecutive rows (16 bytes of bf16); a last tile without a partner keeps its order.
template <int NI, bool GATED>
__device__ __forceinline__ int w_row(int i, int r) {
  if (GATED || (NI % 2 && i == NI - 1)) return i * 16 + r;
  return (i >> 1) * 32 + (r >> 2) * 8 + (i & 1) * 4 + (r & 3);
}
// Column (16 bytes) c of a row lies at column c ^ key in LDS, so that eight lanes of a
// read, one column of eight rows, meet eight columns.
template <int NI, bool GATED>
__device__ __forceinline__ int w_key(int row) {
  if (GATED) return row & 7;
  const int r = row % (16 * NI);
  if (NI % 2 && r >= 16 * (NI - 1)) return r & 7;
  return (r & 3) | ((r >> 1) & 4);
}

template <int MI, int NI>
struct Shape {
  static constexpr int kRowsW = 16 * NI * kWavesN, kRowsX = 16 * MI * kWavesM;
  // loads (8 rows) of a wave and stage; the same for every wave, so that what is in
  // flight is known: loads past the last row fill the stage's padding with zeros
  static constexpr int kLoads = (kRowsW + kRowsX + 8 * kWaves - 1) / (8 * kWaves);
  static constexpr int kStage = kLoads * kWaves * 1024;
  static constexpr int kStages = kLds / kStage < 4 ? kLds / kStage : 4;
};

template <int MI, int NI, bool GATED, typename T, typename OT>
__global__ __launch_bounds__(kWaves * 64, 2) void tile_kernel(LinearProblem p, int n_tiles) {
  typedef Shape<MI, NI> S;
  static_assert(!GATED || NI % 2 == 0, "pairs of tiles");
  __shared__ __attribute__((aligned(16))) uint8_t lds[S::kStages * S::kStage];
  const int wave = uni(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int wn = wave & 1, wm = wave >> 1;
  const int tile_m = blockIdx.x / n_tiles, tile_n = blockIdx.x - tile_m * n_tiles;
  constexpr int kCols = GATED ? S::kRowsW / 2 : S::kRowsW;  // outputs of a row
  const int m0 = tile_m * S::kRowsX, n0 = tile_n * kCols;

  // this wave's loads, 8 rows each, the w rows first: lane l the 16 bytes that belong at
  // column l % 8 of row l / 8
  const size_t wstep = (size_t)p.K * sizeof(T), xstep = p.ldx * sizeof(T);
  const uint8_t* wbase = (const uint8_t*)p.w + n0 * wstep;
  const uint8_t* ubase = wbase + p.N * wstep;  // gated: the up rows
  const uint8_t* xbase = (const uint8_t*)p.x + m0 * xstep;
  uint32_t off[S::kLoads];
  int col[S::kLoads];
#pragma unroll
  for (int i = 0; i < S::kLoads; ++i) {
    const int row = (i * kWaves + wave) * 8 + (lane >> 3);
    int key = row & 7;
    off[i] = kOOB;
    if (row < S::kRowsW) {
      key = w_key<NI, GATED>(row);
      const int n = GATED ? (row >> 5) * 16 + (row & 15) : row;
      if (n0 + n < p.N) off[i] = (uint32_t)n * (uint32_t)wstep;
    } else if (row < S::kRowsW + S::kRowsX) {
      const int m = row - S::kRowsW;
      if (m0 + m < p.T) off[i] = (uint32_t)m * (uint32_t)xstep;
    }
    col[i] = ((lane & 7) ^ key) * 16;
    if (off[i] != kOOB) off[i] += col[i];
  }
  const int bytes = p.K * (int)sizeof(T);
  const int chunks = (bytes + kRowBytes - 1) / kRowBytes;
  auto issue = [&](int c, int slot) {
    const int left = bytes - c * kRowBytes;  // bytes of K from this chunk on
#pragma unroll
    for (int i = 0; i < S::kLoads; ++i) {
      const int first = (i * kWaves + wave) * 8;
      const uint8_t* base = first >= S::kRowsW ? xbase : GATED && (first & 16) ? ubase : wbase;
      const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
          (void*)(base + (size_t)c * kRowBytes), (short)0, (int)kBufferBytes, kRsrcWord3);
      const uint32_t o = left >= kRowBytes || col[i] < left ? off[i] : kOOB;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rs, (lds_ptr_t)(lds + slot * S::kStage + first * kRowBytes), 16, (int)o, 0, 0, 0);
    }
  };

  f32x4 acc[NI][MI];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < MI; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  int fill = 0, slot = 0;  // slots of the next chunk to load and of the one in work
  for (; fill < S::kStages - 1; ++fill) issue(fill, fill);
  for (int c = 0; c < chunks; ++c) {
    // this wave's loads of chunk c have landed, then all waves': and all have read what
    // lay in the slot that the next loads fill
    wait_loads<(S::kStages - 2) * S::kLoads>();
    ring_barrier();
    issue(c + S::kStages - 1, fill);
    fill = fill == S::kStages - 1 ? 0 : fill + 1;
    const uint8_t* w = lds + slot * S::kStage + wn * 16 * NI * kRowBytes;
    const uint8_t* x = lds + slot * S::kStage + (S::kRowsW + wm * 16 * MI) * kRowBytes;
    slot = slot == S::kStages - 1 ? 0 : slot + 1;
#pragma unroll
    for (int step = 0; step < (sizeof(T) == 2 ? 2 : 1); ++step) {
      Frag<T> wf[NI], xf[MI];
      const int r = lane & 15;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int row = w_row<NI, GATED>(i, r);
        wf[i].read(w + row * kRowBytes, w_key<NI, GATED>(row), step);
      }
#pragma unroll
      for (int j = 0; j < MI; ++j) xf[j].read(x + (j * 16 + r) * kRowBytes, r & 7, step);
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < MI; ++j) multiply<T>(acc[i][j], wf[i], xf[j]);
    }
  }
  wait_loads<0>();  // no load may still write this workgroup's LDS at its end
  const int g = lane >> 4;
#pragma unroll
  for (int j = 0; j < MI; ++j) {
    const int m = m0 + (wm * MI + j) * 16 + (lane & 15);
    if constexpr (GATED) {
#pragma unroll
      for (int i = 0; i < NI; i += 2)
        finish<true, OT>(p, m, n0 + wn * 8 * NI + i * 8 + g * 4, acc[i][j], acc[i + 1][j]);
    } else {
#pragma unroll
      for (int i = 0; i < NI; ++i)
        finish<false, OT>(p, m, n0 + wn * 16 * NI + w_row<NI, GATED>(i, g * 4), acc[i][j],
                          f32x4{});
    }
  }
}

template <int MI, int NI, bool GATED, typename T, typename OT>
static void run_tiles(const LinearProblem& p, hipStream_t stream) {
  typedef Shape<MI, NI> S;
  const int mt = (p.T + S::kRowsX - 1) / S::kRowsX;
  const int cols = GATED ? S::kRowsW / 2 : S::kRowsW;
  const int nt = (p.N + cols - 1) / cols;
  tile_kernel<MI, NI, GATED, T, OT><<<mt * nt, kWaves * 64, 0, stream>>>(p, nt);
}

template <bool GATED, typename T, typename OT>
static void dispatch(const LinearProblem& p, hipStream_t stream) {
  if (p.T > 512) run_tiles<4, 8, GATED, T, OT>(p, stream);
  else run_tiles<1, 2, GATED, T, OT>(p, stream);
}

}  // namespace linear

size_t linear_workspace_bytes(int, int, int, int, int) { return 0; }

hipError_t launch_linear(const LinearProblem& p, hipStream_t stream) {
  using namespace linear;
  const bool b = p.dtype == MOE_DTYPE_BF16, ob = p.out_dtype == MOE_DTYPE_BF16;
  if (p.gated) {
    if (b) ob ? dispatch<true, uint16_t, uint16_t>(p, stream)
              : dispatch<true, uint16_t, float>(p, stream);
    else ob ? dispatch<true, float, uint16_t>(p, stream) : dispatch<true, float, float>(p, stream);
  } else {
    if (b) ob ? dispatch<false, uint16_t, uint16_t>(p, stream)
              : dispatch<false, uint16_t, float>(p, stream);
    else ob ? dispatch<false, float, uint16_t>(p, stream)
            : dispatch<false, float, float>(p, stream);
  }
  return hipGetLastError();
}

}  // namespace moe
