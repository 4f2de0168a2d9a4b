// C ABI of libmoe.so: argument validation, then the launchers. Declared in
// include/moe.h; every export is listed there with its meaning and limits.
#include <hip/hip_runtime.h>

#include <limits.h>

#include <initializer_list>

#include "../../include/moe.h"
#include "moe_launch.h"

#define MOE_EXPORT extern "C" __attribute__((visibility("default")))

namespace {

constexpr int kMaxE = 1024;
constexpr long kMaxSlots = 1L << 24;

bool is_pow2_le256(int v) { return v >= 1 && v <= 256 && (v & (v - 1)) == 0; }
bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

moe_status hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

moe_status check_common(int T, int E, int k) {
  if (T < 0 || E < 1 || E > kMaxE || k < 1 || k > E) return MOE_ERR_SHAPE;
  if ((long)T * k >= kMaxSlots || (long)T * E > INT_MAX) return MOE_ERR_SHAPE;
  return MOE_OK;
}

size_t capacity(long S, int E, int block_m) { return moe::align_capacity(S, E, block_m); }

// Validation shared by the FFN entry points; H and I must be multiples of
// mult (f32: 4; bf16 and fp8: 8; weight-only and block-scaled fp8: 128).
moe_status check_ffn(const void* x, const void* w1, const void* w2, const int32_t* topk_ids,
                     const float* topk_weights, const int32_t* sorted_ids,
                     const int32_t* block_expert, const int32_t* num_padded, int T, int E, int H,
                     int I, int k, int block_m, unsigned flags, const void* workspace,
                     size_t workspace_bytes, const void* out, int dtype, int mult) {
  moe_status s = check_common(T, E, k);
  if (s != MOE_OK) return s;
  if (H < mult || I < mult || H % mult != 0 || I % mult != 0) return MOE_ERR_SHAPE;
  if (!is_pow2_le256(block_m)) return MOE_ERR_SHAPE;
  const unsigned known = MOE_FFN_STAGE_PREP | MOE_FFN_STAGE_FC1 | MOE_FFN_STAGE_FC2 |
                         MOE_FFN_STAGE_COMBINE | MOE_FFN_PREPARED | MOE_FFN_NO_XCD_REMAP |
                         MOE_FFN_RANGE_GEMM;
  if (flags & ~known) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!x || !w1 || !w2 || !topk_ids || !topk_weights || !sorted_ids || !block_expert ||
      !num_padded || !workspace || !out)
    return MOE_ERR_NULL;
  if (!aligned(x, 16) || !aligned(w1, 16) || !aligned(w2, 16) || !aligned(out, 16) ||
      !aligned(workspace, 256) || !aligned(topk_ids, 4) || !aligned(topk_weights, 4) ||
      !aligned(sorted_ids, 4) || !aligned(block_expert, 4) || !aligned(num_padded, 4))
    return MOE_ERR_ALIGN;
  if (workspace_bytes < moe::ffn_workspace_layout(T, E, H, I, k, dtype).total)
    return MOE_ERR_WORKSPACE;
  return MOE_OK;
}

moe::FfnProblem problem(const void* x, const void* w1, const float* w1s, const void* w2,
                        const float* w2s, const int32_t* topk_ids, const float* topk_weights,
                        const int32_t* sorted_ids, const int32_t* block_expert,
                        const int32_t* num_padded, int T, int E, int H, int I, int k,
                        int block_m, unsigned flags, void* workspace, void* out) {
  return moe::FfnProblem{x, w1, w1s, w2, w2s, topk_ids, topk_weights, sorted_ids, block_expert,
                         num_padded, T, E, H, I, k, block_m, flags, workspace, out};
}

}  // namespace

MOE_EXPORT const char* moe_status_str(moe_status s) {
  switch (s) {
    case MOE_OK: return "MOE_OK";
    case MOE_ERR_NULL: return "MOE_ERR_NULL: a required pointer is NULL";
    case MOE_ERR_SHAPE: return "MOE_ERR_SHAPE: a size is out of range or inconsistent";
    case MOE_ERR_ALIGN: return "MOE_ERR_ALIGN: a pointer is not suitably aligned";
    case MOE_ERR_WORKSPACE: return "MOE_ERR_WORKSPACE: workspace too small";
    case MOE_ERR_UNSUPPORTED: return "MOE_ERR_UNSUPPORTED: request not served by this library";
    case MOE_ERR_HIP: return "MOE_ERR_HIP: a HIP runtime call or kernel launch failed";
  }
  return "MOE_ERR_UNKNOWN: not a moe_status value";
}

MOE_EXPORT int moe_abi_version(void) { return MOE_ABI_VERSION; }

MOE_EXPORT moe_status moe_route_topk(const float* logits, int T, int E, int k, int renormalize,
                                     int32_t* topk_ids, float* topk_weights,
                                     moe_stream_t stream) {
  moe_status s = check_common(T, E, k);
  if (s != MOE_OK) return s;
  if (T == 0) return MOE_OK;
  if (!logits || !topk_ids || !topk_weights) return MOE_ERR_NULL;
  if (!aligned(logits, 4) || !aligned(topk_ids, 4) || !aligned(topk_weights, 4))
    return MOE_ERR_ALIGN;
  return hip_status(moe::launch_route_topk(logits, T, E, k, renormalize ? 1 : 0, topk_ids,
                                           topk_weights, (hipStream_t)stream));
}

MOE_EXPORT size_t moe_align_capacity(int T, int k, int E, int block_m) {
  if (check_common(T, E, k) != MOE_OK || !is_pow2_le256(block_m)) return 0;
  return capacity((long)T * k, E, block_m);
}

MOE_EXPORT moe_status moe_align_block(const int32_t* topk_ids, int T, int k, int E, int block_m,
                                      int32_t* sorted_ids, int32_t* block_expert,
                                      int32_t* num_padded, moe_stream_t stream) {
  moe_status s = check_common(T, E, k);
  if (s != MOE_OK) return s;
  if (!is_pow2_le256(block_m)) return MOE_ERR_SHAPE;
  const long S = (long)T * k;
  const size_t cap = capacity(S, E, block_m);
  if (!num_padded) return MOE_ERR_NULL;
  if (S > 0 && !topk_ids) return MOE_ERR_NULL;
  if (cap > 0 && (!sorted_ids || !block_expert)) return MOE_ERR_NULL;
  if (!aligned(topk_ids, 4) || !aligned(sorted_ids, 4) || !aligned(block_expert, 4) ||
      !aligned(num_padded, 4))
    return MOE_ERR_ALIGN;
  return hip_status(moe::launch_align(topk_ids, (int)S, E, block_m, (int)cap, sorted_ids,
                                      block_expert, num_padded, (hipStream_t)stream));
}

MOE_EXPORT moe_status moe_route_align(const float* logits, int T, int E, int k, int renormalize,
                                      int block_m, int32_t* topk_ids, float* topk_weights,
                                      int32_t* sorted_ids, int32_t* block_expert,
                                      int32_t* num_padded, moe_stream_t stream) {
  moe_status s = check_common(T, E, k);
  if (s != MOE_OK) return s;
  if (!is_pow2_le256(block_m)) return MOE_ERR_SHAPE;
  const long S = (long)T * k;
  const size_t cap = capacity(S, E, block_m);
  if (!num_padded) return MOE_ERR_NULL;
  if (T > 0 && (!logits || !topk_ids || !topk_weights)) return MOE_ERR_NULL;
  if (cap > 0 && (!sorted_ids || !block_expert)) return MOE_ERR_NULL;
  if (!aligned(logits, 4) || !aligned(topk_ids, 4) || !aligned(topk_weights, 4) ||
      !aligned(sorted_ids, 4) || !aligned(block_expert, 4) || !aligned(num_padded, 4))
    return MOE_ERR_ALIGN;
  hipStream_t st = (hipStream_t)stream;
  if (moe::route_align_fusable(T, E, k))
    return hip_status(moe::launch_route_align(logits, T, E, k, renormalize ? 1 : 0, topk_ids,
                                              topk_weights, block_m, (int)cap, sorted_ids,
                                              block_expert, num_padded, st));
  if (T > 0) {
    const hipError_t e = moe::launch_route_topk(logits, T, E, k, renormalize ? 1 : 0, topk_ids,
                                                topk_weights, st);
    if (e != hipSuccess) return MOE_ERR_HIP;
  }
  return hip_status(moe::launch_align(topk_ids, (int)S, E, block_m, (int)cap, sorted_ids,
                                      block_expert, num_padded, st));
}

MOE_EXPORT int moe_small_max_tokens(void) { return moe::kSmallTokens; }

static moe_status check_small(int T, int E, int H, int I, int k, int dtype, unsigned flags) {
  moe_status s = check_common(T, E, k);
  if (s != MOE_OK) return s;
  if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_FP8) return MOE_ERR_UNSUPPORTED;
  if (T > moe::kSmallTokens || E > moe::kSmallExperts || (long)T * k > moe::kSmallSlots)
    return MOE_ERR_SHAPE;
  if (H < 128 || I < 128 || H % 128 != 0 || I % 128 != 0) return MOE_ERR_SHAPE;
  if (flags & ~(unsigned)(MOE_FFN_NO_XCD_REMAP | MOE_FORWARD_ONE_KERNEL)) return MOE_ERR_UNSUPPORTED;
  // the single cooperative kernel exists for the small kernels' batches only
  if ((flags & MOE_FORWARD_ONE_KERNEL) && !moe::small_kernels(T, k)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

MOE_EXPORT size_t moe_forward_small_workspace_bytes(int T, int E, int H, int I, int k,
                                                    int dtype) {
  if (check_small(T, E, H, I, k, dtype, 0) != MOE_OK) return 0;
  return moe::small_workspace_bytes(T, E, H, I, k, dtype);
}

MOE_EXPORT moe_status moe_forward_small(const float* logits, const uint16_t* x, const void* w1,
                                        const float* w1_scale, const void* w2,
                                        const float* w2_scale, int T, int E, int H, int I,
                                        int k, int renormalize, int dtype, unsigned flags,
                                        int32_t* topk_ids, float* topk_weights, void* workspace,
                                        size_t workspace_bytes, uint16_t* out,
                                        moe_stream_t stream) {
  moe_status s = check_small(T, E, H, I, k, dtype, flags);
  if (s != MOE_OK || T == 0) return s;
  const bool fp8 = dtype == MOE_DTYPE_FP8;
  if (!logits || !x || !w1 || !w2 || !topk_ids || !topk_weights || !workspace || !out)
    return MOE_ERR_NULL;
  if (fp8 && (!w1_scale || !w2_scale)) return MOE_ERR_NULL;
  if (!aligned(logits, 4) || !aligned(x, 16) || !aligned(w1, 16) || !aligned(w2, 16) ||
      !aligned(out, 16) || !aligned(topk_ids, 4) || !aligned(topk_weights, 4) ||
      !aligned(workspace, 256) || (fp8 && (!aligned(w1_scale, 16) || !aligned(w2_scale, 16))))
    return MOE_ERR_ALIGN;
  if (workspace_bytes < moe::small_workspace_bytes(T, E, H, I, k, dtype)) return MOE_ERR_WORKSPACE;
  moe::SmallProblem p{logits, x, w1, fp8 ? w1_scale : nullptr, w2, fp8 ? w2_scale : nullptr,
                      T, E, H, I, k, renormalize ? 1 : 0, flags, dtype, topk_ids, topk_weights,
                      workspace, out};
  return hip_status(moe::launch_forward_small(p, (hipStream_t)stream));
}

MOE_EXPORT moe_status moe_forward_small_static(const float* logits, const uint16_t* x,
                                               const void* w1, const float* w1_scale,
                                               const void* w2, const float* w2_scale, int T,
                                               int E, int H, int I, int k, int renormalize,
                                               int dtype, unsigned flags, int32_t* topk_ids,
                                               float* topk_weights, uint16_t* out,
                                               moe_stream_t stream) {
  static_assert(moe::kStaticScratchBytes == MOE_STATIC_SCRATCH_BYTES, "scratch size");
  moe_status s = check_small(T, E, H, I, k, dtype, flags);
  if (s != MOE_OK || T == 0) return s;
  if (moe::small_workspace_bytes(T, E, H, I, k, dtype) > moe::kStaticScratchBytes)
    return MOE_ERR_WORKSPACE;
  const bool fp8 = dtype == MOE_DTYPE_FP8;
  if (!logits || !x || !w1 || !w2 || !topk_ids || !topk_weights || !out) return MOE_ERR_NULL;
  if (fp8 && (!w1_scale || !w2_scale)) return MOE_ERR_NULL;
  if (!aligned(logits, 4) || !aligned(x, 16) || !aligned(w1, 16) || !aligned(w2, 16) ||
      !aligned(out, 16) || !aligned(topk_ids, 4) || !aligned(topk_weights, 4) ||
      (fp8 && (!aligned(w1_scale, 16) || !aligned(w2_scale, 16))))
    return MOE_ERR_ALIGN;
  void* ws = nullptr;
  if (moe::static_scratch(&ws) != hipSuccess) return MOE_ERR_HIP;
  moe::SmallProblem p{logits, x, w1, fp8 ? w1_scale : nullptr, w2, fp8 ? w2_scale : nullptr,
                      T, E, H, I, k, renormalize ? 1 : 0, flags, dtype, topk_ids, topk_weights,
                      ws, out};
  return hip_status(moe::launch_forward_small(p, (hipStream_t)stream));
}

MOE_EXPORT int moe_default_block_m(int T, int E, int k) {
  if (check_common(T, E, k) != MOE_OK) return 0;
  return moe::default_block_m(T, E, k);
}

MOE_EXPORT size_t moe_ffn_workspace_bytes(int T, int E, int H, int I, int k, int block_m,
                                          int dtype) {
  (void)block_m;
  if (dtype != MOE_DTYPE_F32 && dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_FP8 &&
      dtype != MOE_DTYPE_W8A16 && dtype != MOE_DTYPE_FP8_BLOCK)
    return 0;
  if (T < 0 || E < 1 || H < 1 || I < 1 || k < 1) return 0;
  // W8A16 keeps the bf16 path's intermediates
  return moe::ffn_workspace_layout(T, E, H, I, k,
                                   dtype == MOE_DTYPE_W8A16 ? MOE_DTYPE_BF16 : dtype)
      .total;
}

MOE_EXPORT moe_status moe_ffn_bf16(const uint16_t* x, const uint16_t* w1, const uint16_t* w2,
                                   const int32_t* topk_ids, const float* topk_weights,
                                   const int32_t* sorted_ids, const int32_t* block_expert,
                                   const int32_t* num_padded, int T, int E, int H, int I, int k,
                                   int block_m, unsigned flags, void* workspace,
                                   size_t workspace_bytes, uint16_t* out, moe_stream_t stream) {
  moe_status s = check_ffn(x, w1, w2, topk_ids, topk_weights, sorted_ids, block_expert,
                           num_padded, T, E, H, I, k, block_m, flags, workspace, workspace_bytes,
                           out, MOE_DTYPE_BF16, 8);
  if (s != MOE_OK || T == 0) return s;
  return hip_status(moe::launch_ffn_bf16(
      problem(x, w1, nullptr, w2, nullptr, topk_ids, topk_weights, sorted_ids, block_expert,
              num_padded, T, E, H, I, k, block_m, flags, workspace, out),
      (hipStream_t)stream));
}

MOE_EXPORT moe_status moe_ffn_fp8(const uint16_t* x, const uint8_t* w1, const float* w1_scale,
                                  const uint8_t* w2, const float* w2_scale,
                                  const int32_t* topk_ids, const float* topk_weights,
                                  const int32_t* sorted_ids, const int32_t* block_expert,
                                  const int32_t* num_padded, int T, int E, int H, int I, int k,
                                  int block_m, unsigned flags, void* workspace,
                                  size_t workspace_bytes, uint16_t* out, moe_stream_t stream) {
  moe_status s = check_ffn(x, w1, w2, topk_ids, topk_weights, sorted_ids, block_expert,
                           num_padded, T, E, H, I, k, block_m, flags, workspace, workspace_bytes,
                           out, MOE_DTYPE_FP8, 8);
  if (s != MOE_OK || T == 0) return s;
  if (!w1_scale || !w2_scale) return MOE_ERR_NULL;
  if (!aligned(w1_scale, 16) || !aligned(w2_scale, 16)) return MOE_ERR_ALIGN;
  return hip_status(moe::launch_ffn_fp8(
      problem(x, w1, w1_scale, w2, w2_scale, topk_ids, topk_weights, sorted_ids, block_expert,
              num_padded, T, E, H, I, k, block_m, flags, workspace, out),
      (hipStream_t)stream));
}

MOE_EXPORT moe_status moe_ffn_w8a16(const uint16_t* x, const uint8_t* w1, const float* w1_scale,
                                    const uint8_t* w2, const float* w2_scale,
                                    const int32_t* topk_ids, const float* topk_weights,
                                    const int32_t* sorted_ids, const int32_t* block_expert,
                                    const int32_t* num_padded, int T, int E, int H, int I, int k,
                                    int block_m, unsigned flags, void* workspace,
                                    size_t workspace_bytes, uint16_t* out, moe_stream_t stream) {
  // the bf16 path's shape rules (H, I multiples of 128: whole 128-byte lines of codes) and
  // its workspace
  moe_status s = check_ffn(x, w1, w2, topk_ids, topk_weights, sorted_ids, block_expert, num_padded, T, E,
                H, I, k, block_m, flags, workspace, workspace_bytes, out, MOE_DTYPE_BF16, 128);
  if (s != MOE_OK || T == 0) return s;
  if (!w1_scale || !w2_scale) return MOE_ERR_NULL;
  if (!aligned(w1_scale, 16) || !aligned(w2_scale, 16)) return MOE_ERR_ALIGN;
  return hip_status(moe::launch_ffn_w8a16(
      problem(x, w1, w1_scale, w2, w2_scale, topk_ids, topk_weights, sorted_ids, block_expert,
              num_padded, T, E, H, I, k, block_m, flags, workspace, out),
      (hipStream_t)stream));
}

MOE_EXPORT moe_status moe_ffn_fp8_block(const uint16_t* x, const uint8_t* w1,
                                        const float* w1_scale, const uint8_t* w2,
                                        const float* w2_scale, const int32_t* topk_ids,
                                        const float* topk_weights, const int32_t* sorted_ids,
                                        const int32_t* block_expert, const int32_t* num_padded,
                                        int T, int E, int H, int I, int k, int block_m,
                                        unsigned flags, void* workspace, size_t workspace_bytes,
                                        uint16_t* out, moe_stream_t stream) {
  moe_status s = check_ffn(x, w1, w2, topk_ids, topk_weights, sorted_ids, block_expert,
                           num_padded, T, E, H, I, k, block_m, flags, workspace, workspace_bytes,
                           out, MOE_DTYPE_FP8_BLOCK, 128);
  if (s != MOE_OK || T == 0) return s;
  if (!w1_scale || !w2_scale) return MOE_ERR_NULL;
  if (!aligned(w1_scale, 4) || !aligned(w2_scale, 4)) return MOE_ERR_ALIGN;
  return hip_status(moe::launch_ffn_fp8_block(
      problem(x, w1, w1_scale, w2, w2_scale, topk_ids, topk_weights, sorted_ids, block_expert,
              num_padded, T, E, H, I, k, block_m, flags, workspace, out),
      (hipStream_t)stream));
}

MOE_EXPORT moe_status moe_ffn_f32(const float* x, const float* w1, const float* w2,
                                  const int32_t* topk_ids, const float* topk_weights,
                                  const int32_t* sorted_ids, const int32_t* block_expert,
                                  const int32_t* num_padded, int T, int E, int H, int I, int k,
                                  int block_m, unsigned flags, void* workspace,
                                  size_t workspace_bytes, float* out, moe_stream_t stream) {
  moe_status s = check_ffn(x, w1, w2, topk_ids, topk_weights, sorted_ids, block_expert,
                           num_padded, T, E, H, I, k, block_m, flags, workspace, workspace_bytes,
                           out, MOE_DTYPE_F32, 4);
  if (s != MOE_OK || T == 0) return s;
  return hip_status(moe::launch_ffn_f32(
      problem(x, w1, nullptr, w2, nullptr, topk_ids, topk_weights, sorted_ids, block_expert,
              num_padded, T, E, H, I, k, block_m, flags, workspace, out),
      (hipStream_t)stream));
}

// ---------------------------------------------------- around the FFN ---

namespace {

bool bf16_or_f32(int dtype) { return dtype == MOE_DTYPE_BF16 || dtype == MOE_DTYPE_F32; }
size_t elem_bytes(int dtype) { return dtype == MOE_DTYPE_BF16 ? 2 : 4; }
constexpr int kMaxLength = 1 << 24;  // of a row, where the kernels count in 32 bits

// Whether two buffers share a byte.
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return a && b && x < y + nb && y < x + na;
}

// Whether an output shares a byte with an input of as many bytes without being its
// buffer: rows of one would then be written while others of the launch read them.
bool shifted(const void* out, const void* in, size_t n) {
  return out != in && overlap(out, n, in, n);
}

// Whether an output shares a byte with any of some operands that every row of the launch
// reads: weights, gates, lists.
struct Span {
  const void* p;
  size_t n;
};
bool meets(const void* out, size_t n, std::initializer_list<Span> operands) {
  for (const Span& s : operands)
    if (overlap(out, n, s.p, s.n)) return true;
  return false;
}

// Whether S rows of wa bytes, sa apart, share a byte with S rows of wb bytes, sb
// apart: interleaved column slices of one matrix do not. (Interleaved rows of
// different strides count as sharing.)
bool rows_overlap(const void* a, size_t sa, size_t wa, const void* b, size_t sb, size_t wb,
                  int S) {
  if (!overlap(a, sa * (S - 1) + wa, b, sb * (S - 1) + wb)) return false;
  if (S == 1 || sa != sb) return true;
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  const size_t d = y >= x ? (y - x) % sa : (sa - (x - y) % sa) % sa;  // of b's rows in a's
  return d < wa || d + wb > sa;
}

// Whether S rows of wa bytes, sa apart, share a byte with a span.
bool rows_meet(const void* a, size_t sa, size_t wa, int S, const Span& span) {
  if (!overlap(a, sa * (S - 1) + wa, span.p, span.n)) return false;
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)span.p;
  const size_t first = y < x + wa ? 0 : (y - x - wa) / sa + 1;  // row that ends past its start
  return first < (size_t)S && x + first * sa < y + span.n;
}

// Rows and row length of a norm; mult: what H is a multiple of.
moe_status check_norm(int T, int H, int mult, float eps) {
  if (T < 0 || (long)T >= kMaxSlots) return MOE_ERR_SHAPE;
  if (H < mult || H % mult != 0 || H > MOE_NORM_MAX_H) return MOE_ERR_SHAPE;
  if (!(eps >= 0.f) || eps > 3.0e38f) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace

MOE_EXPORT moe_status moe_norm_in(const void* x, const void* residual, const float* weight,
                                  float alpha, float eps, int T, int H, int dtype,
                                  void* residual_out, void* out, moe_stream_t stream) {
  static_assert(moe::kNormMaxH == MOE_NORM_MAX_H, "row length");
  if (!bf16_or_f32(dtype)) return MOE_ERR_UNSUPPORTED;
  moe_status s = check_norm(T, H, dtype == MOE_DTYPE_F32 ? 4 : 8, eps);
  if (s != MOE_OK || T == 0) return s;
  if (!x || !weight || !out) return MOE_ERR_NULL;
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) ||
      !aligned(residual_out, 16) || !aligned(out, 16))
    return MOE_ERR_ALIGN;
  const size_t bytes = (size_t)T * H * elem_bytes(dtype);
  if (overlap(out, bytes, residual_out, bytes) || shifted(out, x, bytes) ||
      shifted(out, residual, bytes) || shifted(residual_out, x, bytes) ||
      shifted(residual_out, residual, bytes))
    return MOE_ERR_UNSUPPORTED;
  const Span w{weight, H * sizeof(float)};
  if (meets(out, bytes, {w}) || meets(residual_out, bytes, {w})) return MOE_ERR_UNSUPPORTED;
  return hip_status(moe::launch_norm_in(
      moe::NormInProblem{x, residual, weight, alpha, eps, T, H, dtype, residual_out, out},
      (hipStream_t)stream));
}

MOE_EXPORT moe_status moe_norm_out(const void* y, int y_dtype, const int32_t* topk_ids,
                                   const float* topk_weights, const void* shared,
                                   const float* gate, const void* residual, const float* weight,
                                   const float* next_weight, float scale, float eps, int T, int E,
                                   int H, int k, int dtype, void* out, void* next,
                                   moe_stream_t stream) {
  if (!bf16_or_f32(dtype) || !bf16_or_f32(y_dtype)) return MOE_ERR_UNSUPPORTED;
  const int mult = dtype == MOE_DTYPE_F32 && y_dtype == MOE_DTYPE_F32 ? 4 : 8;
  moe_status s = check_norm(T, H, mult, eps);
  if (s != MOE_OK) return s;
  if (k < 1 || (long)T * k >= kMaxSlots || (topk_ids && E < 1)) return MOE_ERR_SHAPE;
  if (T == 0) return MOE_OK;
  if (!y || !out || (!topk_weights && k > 1) || (gate && !shared) || !next != !next_weight)
    return MOE_ERR_NULL;
  if (!aligned(y, 16) || !aligned(shared, 16) || !aligned(residual, 16) || !aligned(weight, 16) ||
      !aligned(next_weight, 16) || !aligned(out, 16) || !aligned(next, 16) ||
      !aligned(topk_ids, 4) || !aligned(topk_weights, 4) || !aligned(gate, 4))
    return MOE_ERR_ALIGN;
  const size_t bytes = (size_t)T * H * elem_bytes(dtype);
  const size_t y_bytes = (size_t)T * k * H * elem_bytes(y_dtype);
  if (overlap(out, bytes, next, bytes) || overlap(y, y_bytes, out, bytes) ||
      overlap(y, y_bytes, next, bytes) || shifted(out, residual, bytes) ||
      shifted(out, shared, bytes) || shifted(next, residual, bytes) ||
      shifted(next, shared, bytes))
    return MOE_ERR_UNSUPPORTED;
  const size_t row = H * sizeof(float), slots = (size_t)T * k * 4;
  const Span w{weight, row}, nw{next_weight, row}, g{gate, T * sizeof(float)},
      wts{topk_weights, slots}, ids{topk_ids, slots};
  if (meets(out, bytes, {w, nw, g, wts, ids}) || meets(next, bytes, {w, nw, g, wts, ids}))
    return MOE_ERR_UNSUPPORTED;
  return hip_status(moe::launch_norm_out(
      moe::NormOutProblem{y, y_dtype, topk_ids, topk_weights, shared, gate, residual, weight,
                          next_weight, scale, eps, T, E, H, k, dtype, out, next},
      (hipStream_t)stream));
}

MOE_EXPORT moe_status moe_router_logits(const void* x, int x_dtype, const void* w, int w_dtype,
                                        const float* bias, int T, int E, int H, float* logits,
                                        moe_stream_t stream) {
  if (!bf16_or_f32(x_dtype) || !bf16_or_f32(w_dtype) ||
      (x_dtype == MOE_DTYPE_F32 && w_dtype != MOE_DTYPE_F32))
    return MOE_ERR_UNSUPPORTED;
  moe_status s = check_common(T, E, 1);
  if (s != MOE_OK) return s;
  if (H < 8 || H % 8 != 0 || H >= kMaxLength) return MOE_ERR_SHAPE;
  if (T == 0) return MOE_OK;
  if (!x || !w || !logits) return MOE_ERR_NULL;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(bias, 4) || !aligned(logits, 4))
    return MOE_ERR_ALIGN;
  const size_t bytes = (size_t)T * E * sizeof(float);
  if (meets(logits, bytes, {{x, (size_t)T * H * elem_bytes(x_dtype)},
                            {w, (size_t)E * H * elem_bytes(w_dtype)},
                            {bias, E * sizeof(float)}}))
    return MOE_ERR_UNSUPPORTED;
  return hip_status(moe::launch_router_logits(x, x_dtype, w, w_dtype, bias, T, E, H, logits,
                                              (hipStream_t)stream));
}

static moe_status check_lora(int S, int n, int K, int r, int block_m) {
  if (S < 0 || (long)S >= kMaxSlots || n < 1 || n > kMaxE) return MOE_ERR_SHAPE;
  if (K < 8 || K % 8 != 0 || K >= kMaxLength || r < 8 || r % 8 != 0 || r > 256)
    return MOE_ERR_SHAPE;
  if (!is_pow2_le256(block_m)) return MOE_ERR_SHAPE;
  return MOE_OK;
}

MOE_EXPORT size_t moe_lora_workspace_bytes(int S, int n, int K, int r, int block_m) {
  if (check_lora(S, n, K, r, block_m) != MOE_OK) return 0;
  return moe::lora_workspace_bytes(S, n, K, r, block_m);
}

MOE_EXPORT moe_status moe_lora_add(const void* x, int x_dtype, size_t ldx, const uint16_t* a,
                                   const uint16_t* b, const float* scale,
                                   const int32_t* sorted_ids, const int32_t* block_adapter,
                                   const int32_t* num_padded, int S, int n, int K, int N, int r,
                                   int block_m, void* workspace, size_t workspace_bytes,
                                   const void* y, int y_dtype, size_t ldy, void* out, size_t ldo,
                                   moe_stream_t stream) {
  if (!bf16_or_f32(x_dtype) || !bf16_or_f32(y_dtype)) return MOE_ERR_UNSUPPORTED;
  moe_status s = check_lora(S, n, K, r, block_m);
  if (s != MOE_OK) return s;
  const size_t mx = 16 / elem_bytes(x_dtype), my = 16 / elem_bytes(y_dtype);
  if (N < 8 || N % 8 != 0 || N >= kMaxLength) return MOE_ERR_SHAPE;
  if (ldx < (size_t)K || ldy < (size_t)N || ldo < (size_t)N || ldx % mx != 0 || ldy % my != 0 ||
      ldo % my != 0)
    return MOE_ERR_SHAPE;
  if (S == 0) return MOE_OK;
  if (!x || !a || !b || !sorted_ids || !block_adapter || !num_padded || !workspace || !y || !out)
    return MOE_ERR_NULL;
  if (!aligned(x, 16) || !aligned(a, 16) || !aligned(b, 16) || !aligned(y, 16) ||
      !aligned(out, 16) || !aligned(scale, 4) || !aligned(sorted_ids, 4) ||
      !aligned(block_adapter, 4) || !aligned(num_padded, 4) || !aligned(workspace, 256))
    return MOE_ERR_ALIGN;
  if (workspace_bytes < moe::lora_workspace_bytes(S, n, K, r, block_m)) return MOE_ERR_WORKSPACE;
  const size_t bx = elem_bytes(x_dtype), by = elem_bytes(y_dtype);
  if (rows_overlap(x, ldx * bx, K * bx, out, ldo * by, N * by, S) ||
      ((y != out || ldy != ldo) &&
       rows_overlap(y, ldy * by, N * by, out, ldo * by, N * by, S)))
    return MOE_ERR_UNSUPPORTED;
  const size_t rows = moe::align_capacity(S, n, block_m);
  const Span operands[] = {{a, (size_t)n * r * K * 2},
                           {b, (size_t)n * r * N * 2},
                           {scale, n * sizeof(float)},
                           {sorted_ids, rows * sizeof(int32_t)},
                           {block_adapter, rows / block_m * sizeof(int32_t)},
                           {num_padded, sizeof(int32_t)}};
  const Span ws{workspace, moe::lora_workspace_bytes(S, n, K, r, block_m)};
  for (const Span& o : operands)
    if (rows_meet(out, ldo * by, N * by, S, o) || meets(ws.p, ws.n, {o}))
      return MOE_ERR_UNSUPPORTED;
  if (rows_meet(x, ldx * bx, K * bx, S, ws) || rows_meet(y, ldy * by, N * by, S, ws) ||
      rows_meet(out, ldo * by, N * by, S, ws))
    return MOE_ERR_UNSUPPORTED;
  return hip_status(moe::launch_lora_add(
      moe::LoraProblem{x, x_dtype, ldx, a, b, scale, sorted_ids, block_adapter, num_padded, S, n,
                       K, N, r, block_m, workspace, y, y_dtype, ldy, out, ldo},
      (hipStream_t)stream));
}

MOE_EXPORT moe_status moe_ffn_intermediates(int T, int E, int H, int I, int k, int block_m,
                                            int dtype, size_t* h_offset, int* h_dtype,
                                            size_t* y_offset, int* y_dtype) {
  if (!h_offset || !h_dtype || !y_offset || !y_dtype) return MOE_ERR_NULL;
  int mult = 8;
  if (dtype == MOE_DTYPE_F32) mult = 4;
  else if (dtype == MOE_DTYPE_W8A16 || dtype == MOE_DTYPE_FP8_BLOCK) mult = 128;
  else if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_FP8) return MOE_ERR_UNSUPPORTED;
  moe_status s = check_common(T, E, k);
  if (s != MOE_OK) return s;
  if (H < mult || I < mult || H % mult != 0 || I % mult != 0) return MOE_ERR_SHAPE;
  if (!is_pow2_le256(block_m)) return MOE_ERR_SHAPE;
  // W8A16 keeps the bf16 path's intermediates, the W8A8 grouped-GEMM tiles
  // leave theirs in bf16 in the places of the fp32 ones
  const int layout = dtype == MOE_DTYPE_W8A16 ? MOE_DTYPE_BF16 : dtype;
  const bool bf16 = layout == MOE_DTYPE_BF16 ||
                    (dtype == MOE_DTYPE_FP8 && moe::fp8_dense(H, I, block_m));
  const moe::FfnWorkspace L = moe::ffn_workspace_layout(T, E, H, I, k, layout);
  *h_offset = L.h_off;
  *y_offset = L.y_off;
  *h_dtype = *y_dtype = bf16 ? MOE_DTYPE_BF16 : MOE_DTYPE_F32;
  return MOE_OK;
}

// ---------------------------------------------------- beside the FFN ---

// Sizes of rows in expert order (of a backward or a way back: without E).
static moe_status check_rows(int T, int E, int H, int k, int R) {
  if (T < 0 || E < 1 || k < 1 || (long)T * k >= kMaxSlots) return MOE_ERR_SHAPE;
  if (H < 1 || H > 1 << 20 || R < (T > 0 ? 1 : 0) || R >= 1 << 25) return MOE_ERR_SHAPE;
  if ((long)T * k * H >= 1L << 37 || (long)R * H >= 1L << 37) return MOE_ERR_SHAPE;
  return MOE_OK;
}

MOE_EXPORT moe_status moe_dispatch(const void* x, const int32_t* topk_ids,
                                   const int32_t* sorted_ids, const int32_t* num_padded, int T,
                                   int E, int H, int k, int R, int dtype, void* rows,
                                   int32_t* slot_rows, moe_stream_t stream) {
  if (!bf16_or_f32(dtype)) return MOE_ERR_UNSUPPORTED;
  moe_status s = check_rows(T, E, H, k, R);
  if (s != MOE_OK || T == 0) return s;
  if (!x || !topk_ids || !sorted_ids || !num_padded || !rows || !slot_rows) return MOE_ERR_NULL;
  const size_t b = elem_bytes(dtype);
  if (!aligned(x, b) || !aligned(rows, b) || !aligned(topk_ids, 4) || !aligned(sorted_ids, 4) ||
      !aligned(num_padded, 4) || !aligned(slot_rows, 4))
    return MOE_ERR_ALIGN;
  const size_t slots = (size_t)T * k * 4, row_bytes = (size_t)R * H * b;
  const Span in[] = {{x, (size_t)T * H * b}, {topk_ids, slots}, {sorted_ids, (size_t)R * 4},
                     {num_padded, 4}};
  if (overlap(rows, row_bytes, slot_rows, slots)) return MOE_ERR_UNSUPPORTED;
  for (const Span& o : in)
    if (meets(rows, row_bytes, {o}) || meets(slot_rows, slots, {o})) return MOE_ERR_UNSUPPORTED;
  return hip_status(moe::launch_dispatch(
      moe::DispatchProblem{x, topk_ids, sorted_ids, num_padded, T, E, H, k, R, dtype, rows,
                           slot_rows},
      (hipStream_t)stream));
}

MOE_EXPORT moe_status moe_combine(const void* rows, int rows_dtype, const int32_t* slot_rows,
                                  const float* topk_weights, int T, int H, int k, int R, int dtype,
                                  void* out, moe_stream_t stream) {
  if (!bf16_or_f32(dtype) || !bf16_or_f32(rows_dtype)) return MOE_ERR_UNSUPPORTED;
  moe_status s = check_rows(T, 1, H, k, R);
  if (s != MOE_OK || T == 0) return s;
  if (!rows || !slot_rows || !out) return MOE_ERR_NULL;
  const size_t b = elem_bytes(dtype), rb = elem_bytes(rows_dtype);
  if (!aligned(rows, rb) || !aligned(out, b) || !aligned(slot_rows, 4) ||
      !aligned(topk_weights, 4))
    return MOE_ERR_ALIGN;
  const size_t slots = (size_t)T * k * 4;
  if (meets(out, (size_t)T * H * b,
            {{rows, (size_t)R * H * rb}, {slot_rows, slots}, {topk_weights, slots}}))
    return MOE_ERR_UNSUPPORTED;
  return hip_status(moe::launch_combine(
      moe::CombineProblem{rows, rows_dtype, slot_rows, topk_weights, T, H, k, R, dtype, out},
      (hipStream_t)stream));
}

MOE_EXPORT moe_status moe_dispatch_backward(const void* drows, const int32_t* slot_rows, int T,
                                            int H, int k, int R, int dtype, void* dx,
                                            moe_stream_t stream) {
  return moe_combine(drows, dtype, slot_rows, nullptr, T, H, k, R, dtype, dx, stream);
}

MOE_EXPORT moe_status moe_combine_backward(const void* dout, int dtype, const void* rows,
                                           int rows_dtype, const int32_t* slot_rows,
                                           const float* topk_weights, const int32_t* sorted_ids,
                                           const int32_t* num_padded, int T, int H, int k, int R,
                                           void* drows, float* dweights, moe_stream_t stream) {
  if (!bf16_or_f32(dtype) || !bf16_or_f32(rows_dtype)) return MOE_ERR_UNSUPPORTED;
  moe_status s = check_rows(T, 1, H, k, R);
  if (s != MOE_OK || T == 0) return s;
  if (!dout || (!rows && dweights) || !slot_rows || !sorted_ids || !num_padded || !drows)
    return MOE_ERR_NULL;
  const size_t b = elem_bytes(dtype), rb = elem_bytes(rows_dtype);
  if (!aligned(dout, b) || !aligned(rows, rb) || !aligned(drows, rb) || !aligned(slot_rows, 4) ||
      !aligned(topk_weights, 4) || !aligned(sorted_ids, 4) || !aligned(num_padded, 4) ||
      !aligned(dweights, 4))
    return MOE_ERR_ALIGN;
  const size_t slots = (size_t)T * k * 4, row_bytes = (size_t)R * H * rb;
  const Span in[] = {{dout, (size_t)T * H * b}, {slot_rows, slots}, {topk_weights, slots},
                     {sorted_ids, (size_t)R * 4}, {num_padded, 4}};
  if (shifted(drows, rows, row_bytes) || overlap(drows, row_bytes, dweights, slots) ||
      overlap(dweights, slots, rows, row_bytes))
    return MOE_ERR_UNSUPPORTED;
  for (const Span& o : in)
    if (meets(drows, row_bytes, {o}) || meets(dweights, slots, {o})) return MOE_ERR_UNSUPPORTED;
  return hip_status(moe::launch_combine_backward(
      moe::CombineBackwardProblem{dout, dtype, rows, rows_dtype, slot_rows, topk_weights,
                                  sorted_ids, num_padded, T, H, k, R, drows, dweights},
      (hipStream_t)stream));
}

MOE_EXPORT moe_status moe_layer_norm(const void* x, const void* residual, const float* weight,
                                     const float* bias, float alpha, float eps, int T, int H,
                                     int dtype, void* residual_out, void* out,
                                     moe_stream_t stream) {
  if (!bf16_or_f32(dtype)) return MOE_ERR_UNSUPPORTED;
  moe_status s = check_norm(T, H, 1, eps);
  if (s != MOE_OK || T == 0) return s;
  if (!x || !out) return MOE_ERR_NULL;
  const size_t b = elem_bytes(dtype), bytes = (size_t)T * H * b;
  if (!aligned(x, b) || !aligned(residual, b) || !aligned(residual_out, b) || !aligned(out, b) ||
      !aligned(weight, 4) || !aligned(bias, 4))
    return MOE_ERR_ALIGN;
  if (overlap(out, bytes, residual_out, bytes) || shifted(out, x, bytes) ||
      shifted(out, residual, bytes) || shifted(residual_out, x, bytes) ||
      shifted(residual_out, residual, bytes))
    return MOE_ERR_UNSUPPORTED;
  const Span w{weight, H * sizeof(float)}, bi{bias, H * sizeof(float)};
  if (meets(out, bytes, {w, bi}) || meets(residual_out, bytes, {w, bi}))
    return MOE_ERR_UNSUPPORTED;
  return hip_status(moe::launch_layer_norm(
      moe::LayerNormProblem{x, residual, weight, bias, alpha, eps, T, H, dtype, residual_out, out},
      (hipStream_t)stream));
}

MOE_EXPORT size_t moe_layer_norm_backward_workspace_bytes(int T, int H) {
  if (check_norm(T, H, 1, 0.f) != MOE_OK) return 0;
  return moe::layer_norm_backward_workspace_bytes(T, H);
}

MOE_EXPORT moe_status moe_layer_norm_backward(const void* dout, const void* s,
                                              const float* weight, const void* dresidual_out,
                                              float alpha, float eps, int T, int H, int dtype,
                                              void* dx, void* dresidual, float* dweight,
                                              float* dbias, void* workspace,
                                              size_t workspace_bytes, moe_stream_t stream) {
  if (!bf16_or_f32(dtype)) return MOE_ERR_UNSUPPORTED;
  moe_status st = check_norm(T, H, 1, eps);
  if (st != MOE_OK) return st;
  const bool sums = dweight || dbias;
  const size_t used = sums ? moe::layer_norm_backward_workspace_bytes(T, H) : 0;
  if ((T > 0 && (!dout || !s || !dx)) || (used && !workspace)) return MOE_ERR_NULL;
  const size_t b = elem_bytes(dtype), bytes = (size_t)T * H * b, vec = H * sizeof(float);
  if (!aligned(dout, b) || !aligned(s, b) || !aligned(dresidual_out, b) || !aligned(dx, b) ||
      !aligned(dresidual, b) || !aligned(weight, 4) || !aligned(dweight, 4) ||
      !aligned(dbias, 4) || (used && !aligned(workspace, 16)))
    return MOE_ERR_ALIGN;
  if (workspace_bytes < used) return MOE_ERR_WORKSPACE;
  const Span w{weight, vec};
  const void* in[] = {dout, s, dresidual_out};
  if (overlap(dx, bytes, dresidual, bytes) || meets(dx, bytes, {w}) || meets(dresidual, bytes, {w}))
    return MOE_ERR_UNSUPPORTED;
  for (const void* p : in)
    if (shifted(dx, p, bytes) || shifted(dresidual, p, bytes)) return MOE_ERR_UNSUPPORTED;
  const Span rows[] = {{dout, bytes}, {s, bytes}, {dresidual_out, bytes}, {dx, bytes},
                       {dresidual, bytes}, w};
  for (const Span& o : rows)
    if (meets(dweight, vec, {o}) || meets(dbias, vec, {o}) || (used && meets(workspace, used, {o})))
      return MOE_ERR_UNSUPPORTED;
  if (overlap(dweight, vec, dbias, vec) ||
      (used && meets(workspace, used, {{dweight, vec}, {dbias, vec}})))
    return MOE_ERR_UNSUPPORTED;
  return hip_status(moe::launch_layer_norm_backward(
      moe::LayerNormBackwardProblem{dout, s, weight, dresidual_out, alpha, eps, T, H, dtype, dx,
                                    dresidual, dweight, dbias, (float*)workspace},
      (hipStream_t)stream));
}

static moe_status check_linear(int T, int N, int K, int gated, int dtype) {
  if (!bf16_or_f32(dtype)) return MOE_ERR_UNSUPPORTED;
  if (T < 0 || (long)T >= kMaxSlots || N < 1) return MOE_ERR_SHAPE;
  if ((long)N * (gated ? 2 : 1) >= kMaxLength) return MOE_ERR_SHAPE;
  if (K < 8 || K % 8 != 0 || K >= 1 << 21 || (long)T * N >= 1L << 37) return MOE_ERR_SHAPE;
  // A launch counts its threads in 32 bits, and of the largest tiles gated fp32 ones hold the
  // fewest outputs, 256 x 64 to 512 threads. (All others' 2^37 are 2^22 of them and their edges.)
  if (gated && dtype == MOE_DTYPE_F32 && ((long)T + 255) / 256 * (((long)N + 63) / 64) >= 1 << 23)
    return MOE_ERR_SHAPE;
  return MOE_OK;
}

MOE_EXPORT size_t moe_linear_workspace_bytes(int T, int N, int K, int gated, int dtype) {
  if (check_linear(T, N, K, gated, dtype) != MOE_OK) return 0;
  return moe::linear_workspace_bytes(moe::linear_plan(T, N, K, gated != 0, dtype), T, N, gated != 0);
}

MOE_EXPORT moe_status moe_linear(const void* x, size_t ldx, const void* w, const float* bias,
                                 int activation, int gated, const void* residual, size_t ldr,
                                 int T, int N, int K, int dtype, int out_dtype, void* workspace,
                                 size_t workspace_bytes, void* out, size_t ldo,
                                 moe_stream_t stream) {
  if (!bf16_or_f32(out_dtype) || activation < MOE_ACT_NONE || activation > MOE_ACT_GELU_TANH)
    return MOE_ERR_UNSUPPORTED;
  moe_status s = check_linear(T, N, K, gated, dtype);
  if (s != MOE_OK) return s;
  const size_t b = elem_bytes(dtype), ob = elem_bytes(out_dtype);
  if (ldx < (size_t)K || ldx >= 1 << 21 || ldx % (16 / b) != 0) return MOE_ERR_SHAPE;
  if (ldo < (size_t)N || ldo > INT_MAX || (residual && (ldr < (size_t)N || ldr > INT_MAX)))
    return MOE_ERR_SHAPE;
  if (T == 0) return MOE_OK;
  const moe::LinearPlan plan = moe::linear_plan(T, N, K, gated != 0, dtype);
  const size_t used = moe::linear_workspace_bytes(plan, T, N, gated != 0);
  if (!x || !w || !out || (used && !workspace)) return MOE_ERR_NULL;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(bias, 4) || !aligned(residual, ob) ||
      !aligned(out, ob) || (used && !aligned(workspace, 256)))
    return MOE_ERR_ALIGN;
  if (workspace_bytes < used) return MOE_ERR_WORKSPACE;
  const size_t n = gated ? 2 * (size_t)N : N, ldrb = ldr * ob;
  const Span ws{used ? workspace : nullptr, used};
  const Span vecs[] = {{w, n * K * b}, {bias, n * sizeof(float)}, ws};
  for (const Span& o : vecs)
    if (o.p && rows_meet(out, ldo * ob, N * ob, T, o)) return MOE_ERR_UNSUPPORTED;
  if (rows_overlap(x, ldx * b, K * b, out, ldo * ob, N * ob, T) ||
      (residual && (residual != out || ldr != ldo) &&
       rows_overlap(residual, ldrb, N * ob, out, ldo * ob, N * ob, T)))
    return MOE_ERR_UNSUPPORTED;
  if (used && (meets(ws.p, ws.n, {vecs[0], vecs[1]}) || rows_meet(x, ldx * b, K * b, T, ws) ||
               (residual && rows_meet(residual, ldrb, N * ob, T, ws))))
    return MOE_ERR_UNSUPPORTED;
  return hip_status(moe::launch_linear(
      moe::LinearProblem{x, ldx, w, bias, activation, gated != 0, residual, ldr, T, N, K, dtype,
                         out_dtype, workspace, out, ldo},
      plan, (hipStream_t)stream));
}
