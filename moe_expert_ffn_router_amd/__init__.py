"""Thin Python binding of libmoe.so (fused MoE expert FFN on MI355X / gfx950).

Argument marshalling only: every step of the path runs in the HIP kernels of
libmoe.so; torch supplies device memory and the current stream. Importing the
package loads the library and raises if it has not been built; nothing here
computes a result on the CPU.

The names mirror the C ABI in include/moe.h:

    route_topk(logits, k, renormalize=False)           -> (topk_ids, topk_weights)
    align_block(topk_ids, E, block_m)                   -> (sorted_ids, block_expert, num_padded)
    ffn_bf16(x, w1, w2, ids, wts, sorted_ids, block_expert, num_padded, block_m, ...) -> out
    ffn_fp8(x, w1, w1_scale, w2, w2_scale, ids, wts, ..., block_m, ...)              -> out
    ffn_w8a16(x, w1, w1_scale, w2, w2_scale, ids, wts, ..., block_m, ...)            -> out
    ffn_fp8_block(x, w1, w1_scale, w2, w2_scale, ids, wts, ..., block_m, ...)        -> out
    ffn_f32(x, w1, w2, ids, wts, ..., block_m, ...)                                 -> out
    forward(x, logits, w1, w2, k, ...)   convenience chaining of the three calls
    forward_small(logits, x, w1, w2, k, ...) -> (out, topk_ids, topk_weights)   one launch, T <= 16
    forward_small_static(logits, x, w1, w2, k, ...)   the same without a workspace (allocates nothing)
    norm_in(x, weight, residual=None, ...) -> (out, residual_out)      residual add + norm before the block
    router_logits(x, w, bias=None, ...)    -> logits                   router projection
    lora_add(y, x, a, b, sorted_ids, block_adapter, num_padded, block_m, ...) -> out   adapters of many requests
    norm_out(y, topk_weights, ...)         -> (out, next)              combine + shared expert + norms + residual
    ffn_intermediates(workspace, ...)      -> (h, y)                   an FFN workspace's tensors, for the two above
    dispatch(x, topk_ids, E, sorted_ids, num_padded, ...) -> (rows, slot_rows)   tokens in expert order
    dispatch_backward(drows, slot_rows, ...)              -> dx
    combine(rows, slot_rows, topk_weights, ...)           -> out                 and back, weighted
    combine_backward(dout, rows, slot_rows, topk_weights, sorted_ids, num_padded, ...) -> (drows, dweights)
    layer_norm(x, weight, bias, residual=None, ...)       -> (out, residual_out)
    layer_norm_backward(dout, s, weight, ...)             -> (dx, dresidual, dweight, dbias)
    linear(x, w, bias=None, activation=ACT_NONE, gated=False, residual=None, ...) -> out
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Tuple

import torch  # loads torch's HIP runtime first; libmoe.so then binds to the same one

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe.so")

MOE_OK = 0
MOE_DTYPE_F32, MOE_DTYPE_BF16, MOE_DTYPE_FP8, MOE_DTYPE_W8A16, MOE_DTYPE_FP8_BLOCK = 0, 1, 2, 3, 4
STAGE_FC1, STAGE_FC2, STAGE_COMBINE, STAGE_PREP = 1 << 0, 1 << 1, 1 << 2, 1 << 3
PREPARED = 1 << 11  # with STAGE_FC1: an earlier call ran STAGE_PREP (see include/moe.h)
NO_XCD_REMAP = 1 << 8
FORWARD_ONE_KERNEL = 1 << 9  # forward_small: the whole layer as one cooperative launch
ACT_NONE, ACT_RELU, ACT_SILU, ACT_GELU, ACT_GELU_TANH = 0, 1, 2, 3, 4  # activations of linear
RANGE_GEMM = 1 << 10  # bf16 prefill blocks: 256 x 256 tiles over per-expert token ranges
ABI_VERSION = 1

EXPORTS = ("moe_status_str", "moe_abi_version", "moe_route_topk", "moe_align_capacity",
           "moe_align_block", "moe_route_align", "moe_default_block_m",
           "moe_ffn_workspace_bytes", "moe_ffn_bf16", "moe_ffn_fp8", "moe_ffn_w8a16",
           "moe_ffn_fp8_block", "moe_ffn_f32", "moe_small_max_tokens",
           "moe_forward_small_workspace_bytes", "moe_forward_small", "moe_forward_small_static",
           "moe_norm_in", "moe_norm_out", "moe_router_logits", "moe_lora_workspace_bytes",
           "moe_lora_add", "moe_ffn_intermediates", "moe_dispatch", "moe_dispatch_backward",
           "moe_combine", "moe_combine_backward", "moe_layer_norm",
           "moe_layer_norm_backward_workspace_bytes", "moe_layer_norm_backward",
           "moe_linear_workspace_bytes", "moe_linear")
STATIC_SCRATCH_BYTES = 32 << 20  # MOE_STATIC_SCRATCH_BYTES


class MoEError(RuntimeError):
    """A libmoe call returned a non-OK status."""

    def __init__(self, status: int, msg: str):
        super().__init__(msg)
        self.status = status


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run __graft_entry__.build() "
                          "(or python moe_expert_ffn_router_amd/build.py)")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, U, Z, F = (ctypes.c_void_p, ctypes.c_int, ctypes.c_uint, ctypes.c_size_t,
                     ctypes.c_float)
    lib.moe_status_str.restype = ctypes.c_char_p
    lib.moe_status_str.argtypes = [I]
    lib.moe_abi_version.restype = I
    lib.moe_abi_version.argtypes = []
    lib.moe_route_topk.restype = I
    lib.moe_route_topk.argtypes = [P, I, I, I, I, P, P, P]
    lib.moe_align_capacity.restype = Z
    lib.moe_align_capacity.argtypes = [I, I, I, I]
    lib.moe_align_block.restype = I
    lib.moe_align_block.argtypes = [P, I, I, I, I, P, P, P, P]
    lib.moe_route_align.restype = I
    lib.moe_route_align.argtypes = [P, I, I, I, I, I, P, P, P, P, P, P]
    lib.moe_default_block_m.restype = I
    lib.moe_default_block_m.argtypes = [I, I, I]
    lib.moe_ffn_workspace_bytes.restype = Z
    lib.moe_ffn_workspace_bytes.argtypes = [I, I, I, I, I, I, I]
    ffn_tail = [P, P, P, P, P, I, I, I, I, I, I, U, P, Z, P, P]
    lib.moe_ffn_bf16.restype = I
    lib.moe_ffn_bf16.argtypes = [P, P, P] + ffn_tail
    lib.moe_ffn_f32.restype = I
    lib.moe_ffn_f32.argtypes = [P, P, P] + ffn_tail
    lib.moe_ffn_fp8.restype = I
    lib.moe_ffn_fp8.argtypes = [P, P, P, P, P] + ffn_tail
    lib.moe_ffn_w8a16.restype = I
    lib.moe_ffn_w8a16.argtypes = [P, P, P, P, P] + ffn_tail
    lib.moe_ffn_fp8_block.restype = I
    lib.moe_ffn_fp8_block.argtypes = [P, P, P, P, P] + ffn_tail
    lib.moe_small_max_tokens.restype = I
    lib.moe_small_max_tokens.argtypes = []
    lib.moe_forward_small_workspace_bytes.restype = Z
    lib.moe_forward_small_workspace_bytes.argtypes = [I, I, I, I, I, I]
    lib.moe_forward_small.restype = I
    lib.moe_forward_small.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, I, U, P, P, P, Z, P, P]
    lib.moe_forward_small_static.restype = I
    lib.moe_forward_small_static.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, I, U, P, P, P, P]
    lib.moe_norm_in.restype = I
    lib.moe_norm_in.argtypes = [P, P, P, F, F, I, I, I, P, P, P]
    lib.moe_norm_out.restype = I
    lib.moe_norm_out.argtypes = [P, I, P, P, P, P, P, P, P, F, F, I, I, I, I, I, P, P, P]
    lib.moe_router_logits.restype = I
    lib.moe_router_logits.argtypes = [P, I, P, I, P, I, I, I, P, P]
    lib.moe_lora_workspace_bytes.restype = Z
    lib.moe_lora_workspace_bytes.argtypes = [I, I, I, I, I]
    lib.moe_lora_add.restype = I
    lib.moe_lora_add.argtypes = [P, I, Z, P, P, P, P, P, P, I, I, I, I, I, I, P, Z, P, I, Z, P, Z,
                                 P]
    lib.moe_ffn_intermediates.restype = I
    lib.moe_ffn_intermediates.argtypes = [I, I, I, I, I, I, I, P, P, P, P]
    lib.moe_dispatch.restype = I
    lib.moe_dispatch.argtypes = [P, P, P, P, I, I, I, I, I, I, P, P, P]
    lib.moe_dispatch_backward.restype = I
    lib.moe_dispatch_backward.argtypes = [P, P, I, I, I, I, I, P, P]
    lib.moe_combine.restype = I
    lib.moe_combine.argtypes = [P, I, P, P, I, I, I, I, I, P, P]
    lib.moe_combine_backward.restype = I
    lib.moe_combine_backward.argtypes = [P, I, P, I, P, P, P, P, I, I, I, I, P, P, P]
    lib.moe_layer_norm.restype = I
    lib.moe_layer_norm.argtypes = [P, P, P, P, F, F, I, I, I, P, P, P]
    lib.moe_layer_norm_backward_workspace_bytes.restype = Z
    lib.moe_layer_norm_backward_workspace_bytes.argtypes = [I, I]
    lib.moe_layer_norm_backward.restype = I
    lib.moe_layer_norm_backward.argtypes = [P, P, P, P, F, F, I, I, I, P, P, P, P, P, Z, P]
    lib.moe_linear_workspace_bytes.restype = Z
    lib.moe_linear_workspace_bytes.argtypes = [I, I, I, I, I]
    lib.moe_linear.restype = I
    lib.moe_linear.argtypes = [P, Z, P, P, I, I, P, Z, I, I, I, I, I, P, Z, P, Z, P]
    if lib.moe_abi_version() != ABI_VERSION:
        raise ImportError(f"libmoe ABI {lib.moe_abi_version()} != binding ABI {ABI_VERSION}")
    return lib


lib = _load()


def status_str(s: int) -> str:
    return lib.moe_status_str(s).decode()


def _check(s: int) -> None:
    if s != MOE_OK:
        raise MoEError(s, status_str(s))


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


# The handle of a device's current stream without a Stream object around it: the
# object costs 2.4 us of every call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
# The current device, where a tensor on one shows that the runtime is up.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream: Optional[torch.cuda.Stream]) -> int:
    if stream is None and _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _need(t: torch.Tensor, name: str, dtypes, device=None, shape=None,
          min_numel: Optional[int] = None) -> None:
    """Check one tensor argument before its pointer reaches the library (the C
    ABI sees only addresses, so a wrong shape, dtype or device would be read or
    written out of bounds on the GPU): a contiguous device tensor of one of
    ``dtypes``, on ``device``, of exactly ``shape`` and/or at least
    ``min_numel`` elements."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a device (cuda/hip) tensor, got {t.device}")
    if device is not None and t.device != torch.device(device):
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if min_numel is not None and t.numel() < min_numel:
        raise ValueError(f"{name} holds {t.numel()} elements, needs at least {min_numel}")


def _dims(t: torch.Tensor, name: str, ndim: int) -> tuple:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got shape {tuple(t.shape)}")
    return tuple(t.shape)


_FP8 = (torch.uint8, torch.float8_e4m3fn)


# ------------------------------------------------------------- routing ---

def _routing_outputs(out, T, k, dev):
    if out is None:
        return (torch.empty((T, k), dtype=torch.int32, device=dev),
                torch.empty((T, k), dtype=torch.float32, device=dev))
    ids, wts = out
    _need(ids, "topk_ids", (torch.int32,), dev, (T, k))
    _need(wts, "topk_weights", (torch.float32,), dev, (T, k))
    return ids, wts


def _align_outputs(out, T, k, E, block_m, dev):
    cap = align_capacity(T, k, E, block_m)
    nblk = cap // block_m if block_m > 0 else 0
    if out is None:
        return (torch.empty(cap, dtype=torch.int32, device=dev),
                torch.empty(nblk, dtype=torch.int32, device=dev),
                torch.empty(1, dtype=torch.int32, device=dev))
    sorted_ids, block_expert, num_padded = out
    _need(sorted_ids, "sorted_ids", (torch.int32,), dev, min_numel=cap)
    _need(block_expert, "block_expert", (torch.int32,), dev, min_numel=nblk)
    _need(num_padded, "num_padded", (torch.int32,), dev, min_numel=1)
    return sorted_ids, block_expert, num_padded


def route_topk(logits: torch.Tensor, k: int, renormalize: bool = False, out=None,
               stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Router softmax + top-k (moe_route_topk). logits [T, E] float32; ``out``
    = (topk_ids [T, k] int32, topk_weights [T, k] float32) to write into."""
    T, E = _dims(logits, "logits", 2)
    _need(logits, "logits", (torch.float32,))
    ids, wts = _routing_outputs(out, T, k, logits.device)
    _check(lib.moe_route_topk(_ptr(logits), T, E, k, int(bool(renormalize)), _ptr(ids),
                              _ptr(wts), _stream(stream)))
    return ids, wts


def align_capacity(T: int, k: int, E: int, block_m: int) -> int:
    return int(lib.moe_align_capacity(T, k, E, block_m))


def default_block_m(T: int, E: int, k: int) -> int:
    """moe_default_block_m: the block size of the fast regime for this batch."""
    return int(lib.moe_default_block_m(T, E, k))


def align_block(topk_ids: torch.Tensor, E: int, block_m: int, out=None, stream=None):
    """Token-to-expert alignment (moe_align_block). Returns device tensors
    (sorted_ids [cap], block_expert [cap/block_m], num_padded [1]); ``out`` may
    supply them (at least that many elements each)."""
    T, k = _dims(topk_ids, "topk_ids", 2)
    _need(topk_ids, "topk_ids", (torch.int32,))
    sorted_ids, block_expert, num_padded = _align_outputs(out, T, k, E, block_m,
                                                          topk_ids.device)
    _check(lib.moe_align_block(_ptr(topk_ids), T, k, E, block_m, _ptr(sorted_ids),
                               _ptr(block_expert), _ptr(num_padded), _stream(stream)))
    return sorted_ids, block_expert, num_padded


align = align_block  # the alignment step under its short name


def route_align(logits: torch.Tensor, k: int, block_m: int, renormalize: bool = False,
                out=None, stream=None, prepare: bool = False):
    """Routing and alignment in one call (moe_route_align). logits [T, E] float32.
    Returns (topk_ids, topk_weights, sorted_ids, block_expert, num_padded), or
    fills `out`, a tuple of those five tensors."""
    T, E = _dims(logits, "logits", 2)
    _need(logits, "logits", (torch.float32,))
    dev = logits.device
    if out is None:
        ids, wts = _routing_outputs(None, T, k, dev)
        sorted_ids, block_expert, num_padded = _align_outputs(None, T, k, E, block_m, dev)
    else:
        ids, wts = _routing_outputs(out[:2], T, k, dev)
        sorted_ids, block_expert, num_padded = _align_outputs(out[2:], T, k, E, block_m, dev)
    keep = (logits, ids, wts, sorted_ids, block_expert, num_padded)
    args = (_ptr(logits), T, E, k, int(bool(renormalize)), block_m, _ptr(ids), _ptr(wts),
            _ptr(sorted_ids), _ptr(block_expert), _ptr(num_padded), _stream(stream))
    return _run(lib.moe_route_align, args, keep, prepare,
                (ids, wts, sorted_ids, block_expert, num_padded))


# ------------------------------------------------------- prepared calls ---

class Prepared:
    """A library call whose arguments were checked and marshalled once (pass
    ``prepare=True`` to route_align, the ffn_* calls or forward_small): calling
    it makes only the C call, which validates its arguments again on the host,
    and checks the status. For loops that launch the same call many times; it
    keeps its tensors alive, and they must not be resized or reallocated."""
    __slots__ = ("_fn", "_args", "_keep")

    def __init__(self, fn, args, keep):
        self._fn, self._args, self._keep = fn, args, keep

    def __call__(self):
        _check(self._fn(*self._args))


def _run(fn, args, keep, prepare, result):
    if prepare:
        return Prepared(fn, args, keep)
    _check(fn(*args))
    return result


# ----------------------------------------------------------------- FFN ---

def workspace_bytes(T: int, E: int, H: int, I: int, k: int, block_m: int, dtype: int) -> int:
    return int(lib.moe_ffn_workspace_bytes(T, E, H, I, k, block_m, dtype))


def alloc_workspace(T, E, H, I, k, block_m, dtype, device) -> torch.Tensor:
    n = workspace_bytes(T, E, H, I, k, block_m, dtype)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def _ffn_args(x, w1, w2, wdtypes, xdtypes, topk_ids, topk_weights, sorted_ids, block_expert,
              num_padded, block_m):
    """Shapes of an FFN call, checked against each other: x [T, H], w1 [E, 2I, H],
    w2 [E, H, I], routing [T, k], alignment buffers that hold the capacity of
    ``block_m``. Returns (T, E, H, I, k)."""
    T, H = _dims(x, "x", 2)
    _need(x, "x", xdtypes)
    dev = x.device
    E, I2, H1 = _dims(w1, "w1", 3)
    if H1 != H or I2 % 2:
        raise ValueError(f"w1 has shape {tuple(w1.shape)}, expected [E, 2I, H={H}]")
    I = I2 // 2
    _need(w1, "w1", wdtypes, dev)
    _need(w2, "w2", wdtypes, dev, (E, H, I))
    Tk = _dims(topk_ids, "topk_ids", 2)
    if Tk[0] != T:
        raise ValueError(f"topk_ids has {Tk[0]} rows, x has {T}")
    k = Tk[1]
    _need(topk_ids, "topk_ids", (torch.int32,), dev, (T, k))
    _need(topk_weights, "topk_weights", (torch.float32,), dev, (T, k))
    _align_outputs((sorted_ids, block_expert, num_padded), T, k, E, block_m, dev)
    return T, E, H, I, k


def _ffn_buffers(x, T, E, H, I, k, block_m, dtype, out_dtype, workspace, out):
    dev = x.device
    if workspace is None:
        workspace = alloc_workspace(T, E, H, I, k, block_m, dtype, dev)
    else:
        _need(workspace, "workspace", (torch.uint8,), dev,
              min_numel=workspace_bytes(T, E, H, I, k, block_m, dtype))
    if out is None:
        out = torch.empty((T, H), dtype=out_dtype, device=dev)
    else:
        _need(out, "out", (out_dtype,), dev, (T, H))
    return workspace, out


def ffn_bf16(x, w1, w2, topk_ids, topk_weights, sorted_ids, block_expert, num_padded,
             block_m: int, flags: int = 0, workspace=None, out=None, stream=None,
             prepare: bool = False):
    """moe_ffn_bf16: x [T,H], w1 [E,2I,H], w2 [E,H,I] bfloat16 -> out [T,H] bfloat16."""
    T, E, H, I, k = _ffn_args(x, w1, w2, (torch.bfloat16,), (torch.bfloat16,), topk_ids,
                              topk_weights, sorted_ids, block_expert, num_padded, block_m)
    workspace, out = _ffn_buffers(x, T, E, H, I, k, block_m, MOE_DTYPE_BF16, torch.bfloat16,
                                  workspace, out)
    keep = (x, w1, w2, topk_ids, topk_weights, sorted_ids, block_expert, num_padded, workspace,
            out)
    args = (_ptr(x), _ptr(w1), _ptr(w2), _ptr(topk_ids), _ptr(topk_weights), _ptr(sorted_ids),
            _ptr(block_expert), _ptr(num_padded), T, E, H, I, k, block_m, flags,
            _ptr(workspace), workspace.numel(), _ptr(out), _stream(stream))
    return _run(lib.moe_ffn_bf16, args, keep, prepare, out)


def _scale_shapes(dtype, E, H, I):
    if dtype == MOE_DTYPE_FP8_BLOCK:
        return (E, 2 * I // 128, H // 128), (E, H // 128, I // 128)
    return (E, 2 * I), (E, H)


def _ffn_scaled(fn, dtype, x, w1, w1_scale, w2, w2_scale, topk_ids, topk_weights, sorted_ids,
                block_m, flags, workspace, out, stream, block_expert, num_padded,
                prepare=False):
    T, E, H, I, k = _ffn_args(x, w1, w2, _FP8, (torch.bfloat16,), topk_ids, topk_weights,
                              sorted_ids, block_expert, num_padded, block_m)
    s1, s2 = _scale_shapes(dtype, E, H, I)
    _need(w1_scale, "w1_scale", (torch.float32,), x.device, s1)
    _need(w2_scale, "w2_scale", (torch.float32,), x.device, s2)
    workspace, out = _ffn_buffers(x, T, E, H, I, k, block_m, dtype, torch.bfloat16,
                                  workspace, out)
    keep = (x, w1, w1_scale, w2, w2_scale, topk_ids, topk_weights, sorted_ids, block_expert,
            num_padded, workspace, out)
    args = (_ptr(x), _ptr(w1), _ptr(w1_scale), _ptr(w2), _ptr(w2_scale), _ptr(topk_ids),
            _ptr(topk_weights), _ptr(sorted_ids), _ptr(block_expert), _ptr(num_padded), T, E,
            H, I, k, block_m, flags, _ptr(workspace), workspace.numel(), _ptr(out),
            _stream(stream))
    return _run(fn, args, keep, prepare, out)


def ffn_fp8(x, w1, w1_scale, w2, w2_scale, topk_ids, topk_weights, sorted_ids, block_expert,
            num_padded, block_m: int, flags: int = 0, workspace=None, out=None, stream=None,
            prepare: bool = False):
    """moe_ffn_fp8: x [T,H] bfloat16; w1 [E,2I,H], w2 [E,H,I] e4m3fn codes (uint8 or
    float8_e4m3fn) with float32 per-output-row scales -> out [T,H] bfloat16."""
    return _ffn_scaled(lib.moe_ffn_fp8, MOE_DTYPE_FP8, x, w1, w1_scale, w2, w2_scale, topk_ids,
                       topk_weights, sorted_ids, block_m, flags, workspace, out, stream,
                       block_expert, num_padded, prepare)


def ffn_w8a16(x, w1, w1_scale, w2, w2_scale, topk_ids, topk_weights, sorted_ids, block_expert,
              num_padded, block_m: int, flags: int = 0, workspace=None, out=None, stream=None,
              prepare: bool = False):
    """moe_ffn_w8a16: weight-only fp8. Arguments as ffn_fp8; activations stay
    bfloat16 -> out [T,H] bfloat16."""
    return _ffn_scaled(lib.moe_ffn_w8a16, MOE_DTYPE_W8A16, x, w1, w1_scale, w2, w2_scale,
                       topk_ids, topk_weights, sorted_ids, block_m, flags, workspace, out,
                       stream, block_expert, num_padded, prepare)


def ffn_fp8_block(x, w1, w1_scale, w2, w2_scale, topk_ids, topk_weights, sorted_ids,
                  block_expert, num_padded, block_m: int, flags: int = 0, workspace=None,
                  out=None, stream=None, prepare: bool = False):
    """moe_ffn_fp8_block: x [T,H] bfloat16; w1 [E,2I,H], w2 [E,H,I] e4m3fn codes with
    float32 scales per 128x128 block (w1_scale [E,2I/128,H/128], w2_scale [E,H/128,I/128])
    -> out [T,H] bfloat16."""
    return _ffn_scaled(lib.moe_ffn_fp8_block, MOE_DTYPE_FP8_BLOCK, x, w1, w1_scale, w2,
                       w2_scale, topk_ids, topk_weights, sorted_ids, block_m, flags, workspace,
                       out, stream, block_expert, num_padded, prepare)


def ffn_f32(x, w1, w2, topk_ids, topk_weights, sorted_ids, block_expert, num_padded,
            block_m: int, flags: int = 0, workspace=None, out=None, stream=None,
            prepare: bool = False):
    """moe_ffn_f32: float32 throughout."""
    T, E, H, I, k = _ffn_args(x, w1, w2, (torch.float32,), (torch.float32,), topk_ids,
                              topk_weights, sorted_ids, block_expert, num_padded, block_m)
    workspace, out = _ffn_buffers(x, T, E, H, I, k, block_m, MOE_DTYPE_F32, torch.float32,
                                  workspace, out)
    keep = (x, w1, w2, topk_ids, topk_weights, sorted_ids, block_expert, num_padded, workspace,
            out)
    args = (_ptr(x), _ptr(w1), _ptr(w2), _ptr(topk_ids), _ptr(topk_weights), _ptr(sorted_ids),
            _ptr(block_expert), _ptr(num_padded), T, E, H, I, k, block_m, flags,
            _ptr(workspace), workspace.numel(), _ptr(out), _stream(stream))
    return _run(lib.moe_ffn_f32, args, keep, prepare, out)


def forward(x, logits, w1, w2, k: int, block_m: Optional[int] = None, renormalize: bool = False,
            w1_scale=None, w2_scale=None, flags: int = 0, weight_only: bool = False,
            stream=None):
    """route_align -> ffn_{f32,bf16,fp8,w8a16,fp8_block}, dtype taken from w1 (fp8
    codes with 3-d block scales run ffn_fp8_block; with per-row scales ffn_w8a16
    if ``weight_only``, else ffn_fp8); block_m defaults to moe_default_block_m."""
    E = _dims(w1, "w1", 3)[0]
    if block_m is None:
        block_m = default_block_m(x.shape[0], E, k)
    ids, wts, sorted_ids, block_expert, num_padded = route_align(logits, k, block_m, renormalize,
                                                                 stream=stream)
    if w1.dtype in _FP8:
        if w1_scale is not None and w1_scale.dim() == 3:
            return ffn_fp8_block(x, w1, w1_scale, w2, w2_scale, ids, wts, sorted_ids,
                                 block_expert, num_padded, block_m, flags, stream=stream)
        return (ffn_w8a16 if weight_only else ffn_fp8)(x, w1, w1_scale, w2, w2_scale, ids, wts,
                                                       sorted_ids, block_expert, num_padded,
                                                       block_m, flags, stream=stream)
    if w1.dtype == torch.bfloat16:
        return ffn_bf16(x, w1, w2, ids, wts, sorted_ids, block_expert, num_padded, block_m,
                        flags, stream=stream)
    return ffn_f32(x, w1, w2, ids, wts, sorted_ids, block_expert, num_padded, block_m, flags,
                   stream=stream)


# ----------------------------------------------------- small-batch path ---

def small_max_tokens() -> int:
    return int(lib.moe_small_max_tokens())


def forward_small_workspace_bytes(T, E, H, I, k, dtype) -> int:
    return int(lib.moe_forward_small_workspace_bytes(T, E, H, I, k, dtype))


def _small_args(logits, x, w1, w2, k, fp8, w1_scale, w2_scale):
    """Shapes of a small-batch forward, checked against each other: logits
    [T, E], x [T, H], w1 [E, 2I, H], w2 [E, H, I], fp8 scales [E, 2I] and
    [E, H]. Returns (T, H, E, I, dtype)."""
    T, H = _dims(x, "x", 2)
    _need(x, "x", (torch.bfloat16,))
    dev = x.device
    E, I2, H1 = _dims(w1, "w1", 3)
    if H1 != H or I2 % 2:
        raise ValueError(f"w1 has shape {tuple(w1.shape)}, expected [E, 2I, H={H}]")
    I = I2 // 2
    _need(logits, "logits", (torch.float32,), dev, (T, E))
    wdt = _FP8 if fp8 else (torch.bfloat16,)
    _need(w1, "w1", wdt, dev)
    _need(w2, "w2", wdt, dev, (E, H, I))
    if fp8:
        _need(w1_scale, "w1_scale", (torch.float32,), dev, (E, 2 * I))
        _need(w2_scale, "w2_scale", (torch.float32,), dev, (E, H))
    return T, H, E, I, MOE_DTYPE_FP8 if fp8 else MOE_DTYPE_BF16


def _small_outputs(x, T, H, k, out, topk_ids, topk_weights):
    dev = x.device
    if topk_ids is None:
        topk_ids = torch.empty((T, k), dtype=torch.int32, device=dev)
    else:
        _need(topk_ids, "topk_ids", (torch.int32,), dev, (T, k))
    if topk_weights is None:
        topk_weights = torch.empty((T, k), dtype=torch.float32, device=dev)
    else:
        _need(topk_weights, "topk_weights", (torch.float32,), dev, (T, k))
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    else:
        _need(out, "out", (torch.bfloat16,), dev, (T, H))
    return out, topk_ids, topk_weights


def forward_small(logits, x, w1, w2, k: int, renormalize: bool = False, w1_scale=None,
                  w2_scale=None, flags: int = 0, out=None, topk_ids=None, topk_weights=None,
                  workspace=None, stream=None, prepare: bool = False):
    """moe_forward_small: the whole layer in one call for T <= small_max_tokens():
    up to 16 tokens (and 256 slots) without an alignment step (separate
    launches; one cooperative launch with flags | FORWARD_ONE_KERNEL), beyond
    that routing, alignment and the FFN launches in its workspace. bf16 weights,
    or e4m3fn codes with per-row float32 scales (W8A8). Returns
    (out [T,H] bfloat16, topk_ids [T,k] int32, topk_weights [T,k] float32)."""
    fp8 = w1.dtype in _FP8
    T, H, E, I, dtype = _small_args(logits, x, w1, w2, k, fp8, w1_scale, w2_scale)
    out, topk_ids, topk_weights = _small_outputs(x, T, H, k, out, topk_ids, topk_weights)
    n = forward_small_workspace_bytes(T, E, H, I, k, dtype)
    if workspace is None:
        workspace = torch.empty(max(n, 256), dtype=torch.uint8, device=x.device)
    else:
        _need(workspace, "workspace", (torch.uint8,), x.device, min_numel=n)
    keep = (logits, x, w1, w2, w1_scale, w2_scale, topk_ids, topk_weights, workspace, out)
    args = (_ptr(logits), _ptr(x), _ptr(w1), _ptr(w1_scale) if fp8 else None, _ptr(w2),
            _ptr(w2_scale) if fp8 else None, T, E, H, I, k, 1 if renormalize else 0, dtype,
            flags, _ptr(topk_ids), _ptr(topk_weights), _ptr(workspace), workspace.numel(),
            _ptr(out), _stream(stream))
    return _run(lib.moe_forward_small, args, keep, prepare, (out, topk_ids, topk_weights))


def forward_small_static(logits, x, w1, w2, k: int, renormalize: bool = False, w1_scale=None,
                         w2_scale=None, flags: int = 0, out=None, topk_ids=None,
                         topk_weights=None, stream=None):
    """moe_forward_small_static: forward_small with the intermediates in the
    library's static per-GPU scratch (STATIC_SCRATCH_BYTES) instead of a
    workspace; the library call allocates nothing (pass ``out``, ``topk_ids``
    and ``topk_weights`` to allocate nothing here either). Calls that overlap
    in time on one GPU race. Returns (out, topk_ids, topk_weights)."""
    fp8 = w1.dtype in (torch.uint8, torch.float8_e4m3fn)
    T, H, E, I, dtype = _small_args(logits, x, w1, w2, k, fp8, w1_scale, w2_scale)
    out, topk_ids, topk_weights = _small_outputs(x, T, H, k, out, topk_ids, topk_weights)
    _check(lib.moe_forward_small_static(
        _ptr(logits), _ptr(x), _ptr(w1), _ptr(w1_scale) if fp8 else None, _ptr(w2),
        _ptr(w2_scale) if fp8 else None, T, E, H, I, k, 1 if renormalize else 0, dtype, flags,
        _ptr(topk_ids), _ptr(topk_weights), _ptr(out), _stream(stream)))
    return out, topk_ids, topk_weights


# ------------------------------------------------------- around the FFN ---

# These calls are microseconds of kernel each, so their checks are kept short: a
# tensor that is as expected costs one comparison of each property; for any
# other _need finds the words.

_ACT = {torch.bfloat16: MOE_DTYPE_BF16, torch.float32: MOE_DTYPE_F32}
_F32, _I32 = (torch.float32,), (torch.int32,)


def _act(t: torch.Tensor, name: str) -> int:
    """The library's dtype code of an activation tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    code = _ACT.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {tuple(_ACT)}")
    return code


def _same(t, name: str, dtypes, dev: int, shape: tuple) -> None:
    """_need for a tensor of exactly ``shape`` on the device of index ``dev``."""
    if (isinstance(t, torch.Tensor) and t.dtype in dtypes and t.get_device() == dev >= 0
            and t.shape == shape and t.is_contiguous()):
        return
    _need(t, name, dtypes, None if dev < 0 else torch.device("cuda", dev), shape)


def _launch_stream(dev: int, stream: Optional[torch.cuda.Stream]) -> int:
    """The stream a call on tensors of device ``dev`` runs on. The library
    launches on the current device, so its tensors (and a stream that is passed)
    are there."""
    if dev != _current_device():
        raise ValueError(f"tensors are on cuda:{dev}, the current device is "
                         f"cuda:{torch.cuda.current_device()}")
    if stream is None:
        return _raw_stream(dev) if _raw_stream is not None else _stream(None)
    if stream.device.index != dev:
        raise ValueError(f"stream is on {stream.device}, tensors are on cuda:{dev}")
    return stream.cuda_stream


def _empty(like: torch.Tensor, shape, dtype, stream: Optional[torch.cuda.Stream]) -> torch.Tensor:
    """A new tensor on ``like``'s device for a call on ``stream``, allocated
    there: memory that another stream still uses cannot be handed to it."""
    if stream is None:
        if like.dtype is dtype and like.shape == shape and like.is_contiguous():
            return torch.empty_like(like)
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _like(t: torch.Tensor, stream: Optional[torch.cuda.Stream]) -> torch.Tensor:
    """_empty of the contiguous tensor ``t``'s own shape and type."""
    if stream is None:
        return torch.empty_like(t)
    with torch.cuda.stream(stream):
        return torch.empty_like(t)


def _matrix(t: torch.Tensor, name: str) -> tuple:
    """Check a contiguous matrix of activations on a device. Returns its dtype code, its device's
    index and its shape."""
    if isinstance(t, torch.Tensor):
        code, dev, shape = _ACT.get(t.dtype), t.get_device(), t.shape
        if code is not None and dev >= 0 and len(shape) == 2 and t.is_contiguous():
            return code, dev, shape
    shape = _dims(t, name, 2)
    code = _act(t, name)
    _need(t, name, (t.dtype,))
    return code, t.get_device(), shape


def _need_rows(t: torch.Tensor, name: str, dtypes, dev: Optional[int] = None, shape=None) -> int:
    """Check a matrix of contiguous rows that may lie apart (a slice of columns
    of a wider one): a device tensor of one of ``dtypes`` with stride 1 along the
    rows. Returns its row stride in elements."""
    rows, cols = _dims(t, name, 2)
    if (t.dtype in dtypes and t.get_device() == (t.get_device() if dev is None else dev) >= 0
            and (shape is None or (rows, cols) == shape) and t.is_contiguous()):
        return cols
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device (cuda/hip) tensor, got {t.device}")
    if dev is not None and t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if shape is not None and (rows, cols) != shape:
        raise ValueError(f"{name} has shape {(rows, cols)}, expected {shape}")
    step, one = t.stride()
    if cols > 1 and one != 1:
        raise ValueError(f"{name} must have contiguous rows, got strides {t.stride()}")
    if rows <= 1:
        return cols
    if step < cols:
        raise ValueError(f"the rows of {name} overlap: strides {t.stride()}")
    return step


def norm_in(x, weight, residual=None, alpha: float = 1.0, eps: float = 1e-6, out=None,
            residual_out=None, stream=None, prepare: bool = False):
    """moe_norm_in: s = residual + alpha * x; out = RMS norm of s times ``weight``;
    residual_out = s. x, residual [T, H] bfloat16 or float32, weight [H] float32.
    Returns (out, residual_out); residual_out is None (and s not stored) without
    a residual unless a buffer is given. out or residual_out may be x or
    residual itself."""
    T, H = shape = _dims(x, "x", 2)
    code = _act(x, "x")
    dev, like = x.get_device(), (x.dtype,)
    _same(x, "x", like, dev, shape)
    _same(weight, "weight", _F32, dev, (H,))
    if residual is not None:
        _same(residual, "residual", like, dev, shape)
    raw = _launch_stream(dev, stream)
    if residual_out is not None:
        _same(residual_out, "residual_out", like, dev, shape)
    elif residual is not None:
        residual_out = _empty(x, shape, x.dtype, stream)
    if out is None:
        out = _empty(x, shape, x.dtype, stream)
    else:
        _same(out, "out", like, dev, shape)
    keep = (x, weight, residual, out, residual_out)
    args = (x.data_ptr(), _ptr(residual), weight.data_ptr(), alpha, eps, T, H, code,
            _ptr(residual_out), out.data_ptr(), raw)
    return _run(lib.moe_norm_in, args, keep, prepare, (out, residual_out))


def norm_out(y, topk_weights=None, topk_ids=None, num_experts: Optional[int] = None, shared=None,
             gate=None, residual=None, weight=None, next_weight=None, scale: float = 1.0,
             eps: float = 1e-6, dtype=None, out=None, next_out=None, stream=None,
             prepare: bool = False):
    """moe_norm_out: v = sum_j topk_weights[t, j] * y[t*k+j] + sigmoid(gate) * shared;
    out = residual + scale * (RMS norm of v times ``weight``, or v without it);
    next = RMS norm of the unrounded out times ``next_weight``.

    y [T*k, H] (or [T, k, H]) bfloat16 or float32; topk_weights, topk_ids [T, k]
    (k = 1 and weight 1 without topk_weights); slots with an id outside
    [0, num_experts) add nothing. shared, residual [T, H] of one type (``dtype``,
    by default theirs, else y's), gate [T], weight, next_weight [H] float32.
    Returns (out, next); next is None without next_weight."""
    code_y = _act(y, "y")
    dev, H = y.get_device(), y.shape[-1] if y.dim() else 0
    _same(y, "y", (y.dtype,), dev, y.shape)
    if topk_weights is None:
        T, k = y.numel() // H if H else 0, 1
    else:
        T, k = _dims(topk_weights, "topk_weights", 2)
        _same(topk_weights, "topk_weights", _F32, dev, (T, k))
    if y.shape != (T * k, H) and y.shape != (T, k, H):
        raise ValueError(f"y has shape {tuple(y.shape)}, expected {(T * k, H)} or {(T, k, H)}")
    if topk_ids is not None:
        _same(topk_ids, "topk_ids", _I32, dev, (T, k))
        if num_experts is None:
            raise ValueError("topk_ids needs num_experts")
    if dtype is None:
        like = residual if residual is not None else shared if shared is not None else out
        dtype = y.dtype if like is None else like.dtype
    if dtype not in _ACT:
        raise TypeError(f"dtype is {dtype}, expected one of {tuple(_ACT)}")
    for name, t in (("shared", shared), ("residual", residual), ("out", out),
                    ("next_out", next_out)):
        if t is not None:
            _same(t, name, (dtype,), dev, (T, H))
    if gate is not None:
        _same(gate, "gate", _F32, dev, (T,))
    if weight is not None:
        _same(weight, "weight", _F32, dev, (H,))
    if next_weight is not None:
        _same(next_weight, "next_weight", _F32, dev, (H,))
    raw = _launch_stream(dev, stream)
    like = y if residual is None else residual
    if out is None:
        out = _empty(like, (T, H), dtype, stream)
    if next_out is None and next_weight is not None:
        next_out = _empty(like, (T, H), dtype, stream)
    keep = (y, topk_ids, topk_weights, shared, gate, residual, weight, next_weight, out, next_out)
    args = (y.data_ptr(), code_y, _ptr(topk_ids), _ptr(topk_weights), _ptr(shared), _ptr(gate),
            _ptr(residual), _ptr(weight), _ptr(next_weight), scale, eps, T, num_experts or 0, H,
            k, _ACT[dtype], out.data_ptr(), _ptr(next_out), raw)
    return _run(lib.moe_norm_out, args, keep, prepare, (out, next_out))


def router_logits(x, w, bias=None, out=None, stream=None, prepare: bool = False):
    """moe_router_logits: logits [T, E] float32 = x [T, H] @ w [E, H]^T + bias [E].
    x bfloat16 with w bfloat16 or float32, or both float32."""
    T, H = _dims(x, "x", 2)
    E = _dims(w, "w", 2)[0]
    code_x, code_w = _act(x, "x"), _act(w, "w")
    dev = x.get_device()
    _same(x, "x", (x.dtype,), dev, (T, H))
    _same(w, "w", (w.dtype,), dev, (E, H))
    if bias is not None:
        _same(bias, "bias", _F32, dev, (E,))
    raw = _launch_stream(dev, stream)
    if out is None:
        out = _empty(x, (T, E), torch.float32, stream)
    else:
        _same(out, "out", _F32, dev, (T, E))
    args = (x.data_ptr(), code_x, w.data_ptr(), code_w, _ptr(bias), T, E, H, out.data_ptr(), raw)
    return _run(lib.moe_router_logits, args, (x, w, bias, out), prepare, out)


def lora_workspace_bytes(S: int, n: int, K: int, r: int, block_m: int) -> int:
    return int(lib.moe_lora_workspace_bytes(S, n, K, r, block_m))


def lora_add(y, x, a, b, sorted_ids, block_adapter, num_padded, block_m: int, scale=None,
             out=None, workspace=None, stream=None, prepare: bool = False):
    """moe_lora_add: out[s] = y[s] + scale[g] * b[g] (a[g] x[s]) for the rows s of
    adapter g in the lists (align_block of the rows' adapter ids [S, 1], or of
    any ids whose flat slots are the rows; -1 for slots of experts that another
    shard serves); the other rows of ``out`` are left as they are. x [S, K], y [S, N] bfloat16 or float32, a [n, r, K], b [n, N, r]
    bfloat16, scale [n] float32. ``out`` defaults to y (in place). x, y and out
    may be column slices of wider matrices."""
    S, K = _dims(x, "x", 2)
    n, r, _ = _dims(a, "a", 3)
    N = _dims(y, "y", 2)[1]
    code_x, code_y = _act(x, "x"), _act(y, "y")
    dev, bf16 = x.get_device(), (torch.bfloat16,)
    ldx = _need_rows(x, "x", (x.dtype,))
    ldy = _need_rows(y, "y", (y.dtype,), dev, (S, N))
    _same(a, "a", bf16, dev, (n, r, K))
    _same(b, "b", bf16, dev, (n, N, r))
    if scale is not None:
        _same(scale, "scale", _F32, dev, (n,))
    # what the lists of S slots hold, however these split into tokens and k
    m = max(block_m, 1)
    blocks = (S + min(n, S) * (m - 1) + m - 1) // m
    for name, t, least in (("sorted_ids", sorted_ids, blocks * m),
                           ("block_adapter", block_adapter, blocks),
                           ("num_padded", num_padded, 1)):
        if not (isinstance(t, torch.Tensor) and t.dtype is torch.int32 and t.get_device() == dev
                and t.numel() >= least and t.is_contiguous()):
            _need(t, name, _I32, x.device, min_numel=least)
    if out is None:
        out, ldo = y, ldy
    else:
        ldo = _need_rows(out, "out", (y.dtype,), dev, (S, N))
    raw = _launch_stream(dev, stream)
    need = lora_workspace_bytes(S, n, K, r, block_m)
    if workspace is None:
        workspace = _empty(x, (max(need, 256),), torch.uint8, stream)
    else:
        _need(workspace, "workspace", (torch.uint8,), x.device, min_numel=need)
    keep = (y, x, a, b, sorted_ids, block_adapter, num_padded, scale, out, workspace)
    args = (x.data_ptr(), code_x, ldx, a.data_ptr(), b.data_ptr(), _ptr(scale),
            sorted_ids.data_ptr(), block_adapter.data_ptr(), num_padded.data_ptr(), S, n, K, N, r,
            block_m, workspace.data_ptr(), workspace.numel(), y.data_ptr(), code_y, ldy,
            out.data_ptr(), ldo, raw)
    return _run(lib.moe_lora_add, args, keep, prepare, out)


def ffn_intermediates(workspace, T: int, E: int, H: int, I: int, k: int, block_m: int,
                      dtype: int) -> Tuple[torch.Tensor, torch.Tensor]:
    """moe_ffn_intermediates: the h [T*k, I] and y [T*k, H] that the FFN call of
    ``dtype`` (MOE_DTYPE_*) and block_m keeps in ``workspace``, as views of it
    (bfloat16 or float32)."""
    h_at, y_at = ctypes.c_size_t(), ctypes.c_size_t()
    h_dt, y_dt = ctypes.c_int(), ctypes.c_int()
    _check(lib.moe_ffn_intermediates(T, E, H, I, k, block_m, dtype, ctypes.byref(h_at),
                                     ctypes.byref(h_dt), ctypes.byref(y_at), ctypes.byref(y_dt)))
    _need(workspace, "workspace", (torch.uint8,),
          min_numel=workspace_bytes(T, E, H, I, k, block_m, dtype))

    def view(at, code, cols):
        t = torch.bfloat16 if code.value == MOE_DTYPE_BF16 else torch.float32
        size = 2 if code.value == MOE_DTYPE_BF16 else 4
        return workspace[at.value:at.value + T * k * cols * size].view(t).view(T * k, cols)

    return view(h_at, h_dt, I), view(y_at, y_dt, H)


# ------------------------------------------------------- beside the FFN ---

def _rows_lists(sorted_ids, num_padded, dev: int) -> int:
    """The lists of an alignment as the rows in expert order take them; their length R."""
    if not (isinstance(num_padded, torch.Tensor) and num_padded.dtype is torch.int32
            and num_padded.get_device() == dev >= 0 and num_padded.numel() >= 1):
        _need(num_padded, "num_padded", _I32, torch.device("cuda", max(dev, 0)), min_numel=1)
    R = _dims(sorted_ids, "sorted_ids", 1)[0]
    _same(sorted_ids, "sorted_ids", _I32, dev, (R,))
    return R


def dispatch(x, topk_ids, E: int, sorted_ids, num_padded, out=None, slot_rows=None, stream=None,
             prepare: bool = False):
    """moe_dispatch: the rows of x [T, H] (bfloat16 or float32) in expert order, and every slot's
    place among them. topk_ids [T, k] and E as given to align_block, sorted_ids [R] and num_padded
    as it returned them. Returns (rows [R, H], slot_rows [T, k] int32): rows that pad an expert's
    run are zeros, those from num_padded on are not written; slot_rows is -1 for a slot whose id is
    outside [0, E)."""
    code, dev, (T, H) = _matrix(x, "x")
    k = _dims(topk_ids, "topk_ids", 2)[1]
    _same(topk_ids, "topk_ids", _I32, dev, (T, k))
    R = _rows_lists(sorted_ids, num_padded, dev)
    raw = _launch_stream(dev, stream)
    if out is None:
        out = _empty(x, (R, H), x.dtype, stream)
    else:
        _same(out, "out", (x.dtype,), dev, (R, H))
    if slot_rows is None:
        slot_rows = _like(topk_ids, stream)
    else:
        _same(slot_rows, "slot_rows", _I32, dev, (T, k))
    keep = (x, topk_ids, sorted_ids, num_padded, out, slot_rows)
    args = (x.data_ptr(), topk_ids.data_ptr(), sorted_ids.data_ptr(), num_padded.data_ptr(), T, E,
            H, k, R, code, out.data_ptr(), slot_rows.data_ptr(), raw)
    return _run(lib.moe_dispatch, args, keep, prepare, (out, slot_rows))


def dispatch_backward(drows, slot_rows, out=None, stream=None, prepare: bool = False):
    """moe_dispatch_backward: dx [T, H] from the gradient drows [R, H] of the rows and the slots'
    places slot_rows [T, k]; the rows of no slot are not read."""
    code, dev, (R, H) = _matrix(drows, "drows")
    T, k = _dims(slot_rows, "slot_rows", 2)
    _same(slot_rows, "slot_rows", _I32, dev, (T, k))
    raw = _launch_stream(dev, stream)
    if out is None:
        out = _empty(drows, (T, H), drows.dtype, stream)
    else:
        _same(out, "out", (drows.dtype,), dev, (T, H))
    args = (drows.data_ptr(), slot_rows.data_ptr(), T, H, k, R, code, out.data_ptr(), raw)
    return _run(lib.moe_dispatch_backward, args, (drows, slot_rows, out), prepare, out)


def combine(rows, slot_rows, topk_weights=None, dtype=None, out=None, stream=None,
            prepare: bool = False):
    """moe_combine: out[t] = sum_j topk_weights[t, j] * rows[slot_rows[t, j]] (weight 1 without
    topk_weights); slots without a place add nothing. rows [R, H] bfloat16 or float32, out [T, H]
    of ``dtype`` (by default the rows')."""
    code_r, dev, (R, H) = _matrix(rows, "rows")
    T, k = _dims(slot_rows, "slot_rows", 2)
    _same(slot_rows, "slot_rows", _I32, dev, (T, k))
    if topk_weights is not None:
        _same(topk_weights, "topk_weights", _F32, dev, (T, k))
    if dtype is None:
        dtype = rows.dtype if out is None else out.dtype
    if dtype not in _ACT:
        raise TypeError(f"dtype is {dtype}, expected one of {tuple(_ACT)}")
    raw = _launch_stream(dev, stream)
    if out is None:
        out = _empty(rows, (T, H), dtype, stream)
    else:
        _same(out, "out", (dtype,), dev, (T, H))
    args = (rows.data_ptr(), code_r, slot_rows.data_ptr(), _ptr(topk_weights), T, H, k, R,
            _ACT[dtype], out.data_ptr(), raw)
    return _run(lib.moe_combine, args, (rows, slot_rows, topk_weights, out), prepare, out)


def combine_backward(dout, rows, slot_rows, topk_weights, sorted_ids, num_padded, drows=None,
                     dweights=None, stream=None, prepare: bool = False):
    """moe_combine_backward: the gradients of combine's rows and weights from dout [T, H]. Returns
    (drows [R, H] of the rows' type, dweights [T, k] float32); topk_weights None: weight 1. Rows of
    drows that pad a run are zeros, those from num_padded on are not written; drows may be rows
    itself."""
    code, dev, (T, H) = _matrix(dout, "dout")
    code_r = _act(rows, "rows")
    k = _dims(slot_rows, "slot_rows", 2)[1]
    _same(slot_rows, "slot_rows", _I32, dev, (T, k))
    R = _rows_lists(sorted_ids, num_padded, dev)
    _same(rows, "rows", (rows.dtype,), dev, (R, H))
    if topk_weights is not None:
        _same(topk_weights, "topk_weights", _F32, dev, (T, k))
    raw = _launch_stream(dev, stream)
    if drows is None:
        drows = _like(rows, stream)
    else:
        _same(drows, "drows", (rows.dtype,), dev, (R, H))
    if dweights is None:
        dweights = _empty(slot_rows, (T, k), torch.float32, stream)
    else:
        _same(dweights, "dweights", _F32, dev, (T, k))
    keep = (dout, rows, slot_rows, topk_weights, sorted_ids, num_padded, drows, dweights)
    args = (dout.data_ptr(), code, rows.data_ptr(), code_r, slot_rows.data_ptr(),
            _ptr(topk_weights), sorted_ids.data_ptr(), num_padded.data_ptr(), T, H, k, R,
            drows.data_ptr(), dweights.data_ptr(), raw)
    return _run(lib.moe_combine_backward, args, keep, prepare, (drows, dweights))


def layer_norm(x, weight=None, bias=None, residual=None, alpha: float = 1.0, eps: float = 1e-5,
               out=None, residual_out=None, stream=None, prepare: bool = False):
    """moe_layer_norm: s = residual + alpha * x; out = layer norm of s times ``weight`` plus
    ``bias`` (either None: 1 and 0); residual_out = s. x, residual [T, H] bfloat16 or float32,
    weight, bias [H] float32. Returns (out, residual_out); residual_out is None (and s not stored)
    without a residual unless a buffer is given. out or residual_out may be x or residual itself."""
    code, dev, shape = _matrix(x, "x")
    (T, H), like = shape, (x.dtype,)
    if weight is not None:
        _same(weight, "weight", _F32, dev, (H,))
    if bias is not None:
        _same(bias, "bias", _F32, dev, (H,))
    if residual is not None:
        _same(residual, "residual", like, dev, shape)
    raw = _launch_stream(dev, stream)
    if residual_out is not None:
        _same(residual_out, "residual_out", like, dev, shape)
    elif residual is not None:
        residual_out = _like(x, stream)
    if out is None:
        out = _like(x, stream)
    else:
        _same(out, "out", like, dev, shape)
    keep = (x, residual, weight, bias, out, residual_out)
    args = (x.data_ptr(), _ptr(residual), _ptr(weight), _ptr(bias), alpha, eps, T, H, code,
            _ptr(residual_out), out.data_ptr(), raw)
    return _run(lib.moe_layer_norm, args, keep, prepare, (out, residual_out))


def layer_norm_backward_workspace_bytes(T: int, H: int) -> int:
    return int(lib.moe_layer_norm_backward_workspace_bytes(T, H))


def layer_norm_backward(dout, s, weight=None, dresidual_out=None, alpha: float = 1.0,
                        eps: float = 1e-5, dx=None, dresidual=None, dweight=None, dbias=None,
                        workspace=None, stream=None, prepare: bool = False):
    """moe_layer_norm_backward: the gradients of layer_norm from dout [T, H], the sum s [T, H] it
    normalised (its residual_out, or x) and what arrives at residual_out. Returns (dx, dresidual,
    dweight, dbias): dx = alpha * ds; dresidual = ds, None without dresidual_out unless a buffer is
    given; dweight [H] float32, None without a weight unless a buffer is given; dbias [H] float32.
    dx or dresidual may be dout, s or dresidual_out itself."""
    code, dev, shape = _matrix(dout, "dout")
    (T, H), like = shape, (dout.dtype,)
    _same(s, "s", like, dev, shape)
    if weight is not None:
        _same(weight, "weight", _F32, dev, (H,))
    if dresidual_out is not None:
        _same(dresidual_out, "dresidual_out", like, dev, shape)
    raw = _launch_stream(dev, stream)
    if dresidual is not None:
        _same(dresidual, "dresidual", like, dev, shape)
    elif dresidual_out is not None:
        dresidual = _like(dout, stream)
    if dx is None:
        dx = _like(dout, stream)
    else:
        _same(dx, "dx", like, dev, shape)
    if dweight is not None:
        _same(dweight, "dweight", _F32, dev, (H,))
    elif weight is not None:
        dweight = _like(weight, stream)
    if dbias is None:
        dbias = _empty(dout, (H,), torch.float32, stream) if weight is None else _like(weight, stream)
    else:
        _same(dbias, "dbias", _F32, dev, (H,))
    need = layer_norm_backward_workspace_bytes(T, H)
    if workspace is None:
        workspace = _empty(dout, (max(need, 256),), torch.uint8, stream)
    else:
        _need(workspace, "workspace", (torch.uint8,), dout.device, min_numel=need)
    keep = (dout, s, weight, dresidual_out, dx, dresidual, dweight, dbias, workspace)
    args = (dout.data_ptr(), s.data_ptr(), _ptr(weight), _ptr(dresidual_out), alpha, eps, T, H,
            code, dx.data_ptr(), _ptr(dresidual), _ptr(dweight), dbias.data_ptr(),
            workspace.data_ptr(), workspace.numel(), raw)
    return _run(lib.moe_layer_norm_backward, args, keep, prepare, (dx, dresidual, dweight, dbias))


def linear_workspace_bytes(T: int, N: int, K: int, gated: bool, dtype: int) -> int:
    return int(lib.moe_linear_workspace_bytes(T, N, K, int(bool(gated)), dtype))


def linear(x, w, bias=None, activation: int = ACT_NONE, gated: bool = False, residual=None,
           dtype=None, out=None, workspace=None, stream=None, prepare: bool = False):
    """moe_linear: out [T, N] = residual + act(x w^T + bias), or gated residual + act(x wg^T + bg)
    * (x wu^T + bu) with w [2 N, K] and bias [2 N] holding the gate rows, then the up rows. x [T, K]
    and w bfloat16 or float32 (the same), bias float32, activation ACT_*; residual and out of
    ``dtype`` (by default the residual's, else x's). x, residual and out may be column slices of
    wider matrices; out may be residual itself."""
    if isinstance(x, torch.Tensor) and x.is_contiguous():
        code, dev, (T, K) = _matrix(x, "x")
        ldx = K
    else:
        T, K = _dims(x, "x", 2)
        code, dev = _act(x, "x"), x.get_device()
        ldx = _need_rows(x, "x", (x.dtype,))
    wcode, wdev, (n, wk) = _matrix(w, "w")
    if wcode != code or wdev != dev or wk != K:
        _same(w, "w", (x.dtype,), dev, (n, K))
    if gated and n % 2:
        raise ValueError(f"w has shape {tuple(w.shape)}, expected [2 N, K={K}]")
    N = n // 2 if gated else n
    if bias is not None:
        _same(bias, "bias", _F32, dev, (n,))
    if dtype is None:
        like = residual if residual is not None else x if out is None else out
        dtype = like.dtype
    if dtype not in _ACT:
        raise TypeError(f"dtype is {dtype}, expected one of {tuple(_ACT)}")
    ldr = 0 if residual is None else _need_rows(residual, "residual", (dtype,), dev, (T, N))
    raw = _launch_stream(dev, stream)
    if out is None:
        out, ldo = _empty(x, (T, N), dtype, stream), N
    else:
        ldo = _need_rows(out, "out", (dtype,), dev, (T, N))
    need = linear_workspace_bytes(T, N, K, gated, code)
    if workspace is not None:
        _need(workspace, "workspace", (torch.uint8,), x.device, min_numel=need)
    elif need:
        workspace = _empty(x, (need,), torch.uint8, stream)
    keep = (x, w, bias, residual, out, workspace)
    args = (x.data_ptr(), ldx, w.data_ptr(), _ptr(bias), activation, int(bool(gated)),
            _ptr(residual), ldr, T, N, K, code, _ACT[dtype], _ptr(workspace),
            0 if workspace is None else workspace.numel(), out.data_ptr(), ldo, raw)
    return _run(lib.moe_linear, args, keep, prepare, out)
