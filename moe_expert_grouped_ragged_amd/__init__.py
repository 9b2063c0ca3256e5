"""Python binding of libgg, the MI355X (gfx950) grouped GEMM for frozen MoE experts.

Argument marshalling only: every step of the computation runs in the HIP
kernels behind ``include/gg.h``.  PyTorch supplies device memory and the
current stream.  The functions carry the C names:

  gg_pack_weights(w1, w2)                        -> packed weight buffer
  gg_forward_fc1_swiglu(x, offsets, packed, ...) -> (h1, a)
  gg_forward_fc2(a, offsets, packed, ...)        -> y
  gg_dgrad(dy, h1, offsets, packed, ...)         -> dx  (dH1 left in the workspace)
  gg_forward_fc1_glu(x, offsets, packed, ..., activation, probs) -> (h1, a)
  gg_dgrad_glu(dy, h1, offsets, packed, ..., activation, probs)  -> (dx, dprobs)
  gg_dgrad_recompute(dy, x, offsets, packed, ...)                 -> (dx, dprobs)
        (no saved H1: FC1 is recomputed from x inside the call)
  gg_pack_frag(packed, E, H, F)                  -> opt-in fragment buffer
  gg_forward_fc2_frag(a, offsets, packed, frag, ...) -> y
        (the *_glu, recompute and fc2_frag calls take `frag`: fragment-ordered
        weight copies that speed up the GEMMs for H % 256 == 0 and
        F % 128 == 0, at 12*E*H*F more bytes)

The *_glu calls add the QuickGeGLU activation and the weighting of the
activation by each row's router probability (fp32 [M]), with dp of that
weight from the input gradient.  The probability can instead scale the FC1
input rows:

  gg_scale_rows(x, probs)                        -> x' = bf16(p_r * x_r)
  gg_scale_rows_backward(dxs, x, probs)          -> (dx, dprobs)
        (ScaleRows is the autograd form, to compose with FrozenExpertMLP)

Expert products over 8-bit copies of the frozen weights, tokens quantized on
the way (half the weight bytes, twice the matrix rate), and the trainable
low-rank adapters added to a product's output (both products of the 8-bit MLP;
the bf16 calls make H1 and A, and dA and dH1, in one launch each, with no place for
an adapter between them):

  gg_int8_quantize_rows(x)                       -> (q, s), one scale a row
  gg_int8_pack(wq, ws) / gg_int8_pack_transposed -> laid out for forward / dgrad
  gg_int8_forward(x, offsets, packed, ...)       -> (y, A or None)
  gg_int8_dgrad(dy, offsets, packed_t, ...)      -> (dx, dH1 or None)
  gg_adapter_forward(x, offsets, a, b, scale, base)           -> (y, u)
  gg_adapter_backward(dy, x, u, offsets, a, b, scale, base)   -> (dx, da, db)
        (Int8AdapterExpertMLP runs the gated MLP of both, with autograd;
        int8_experts prepares its weights)

The other calls take frozen, bias-free bf16 expert weights only: the Megatron-LM pull request
"perf(moe): add frozen grouped GEMM for adapter training" (section "Why
existing behavior remains safe") accepts only grouped, frozen, bias-free BF16
expert weights and fails during preparation otherwise; ``gg_pack_weights``
raises ValueError for other dtypes and for weights that require grad.

There is no fallback: if libgg.so is missing, importing this package raises.
"""
from __future__ import annotations

import ctypes
import functools
import inspect
import os
from typing import NamedTuple, Optional, Sequence, Tuple, Union

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgg.so")

GG_OK = 0
GG_ERR_INVALID_ARGUMENT = 1
GG_ERR_MISALIGNED = 2
GG_ERR_UNSUPPORTED_DEVICE = 3
GG_ERR_WORKSPACE_TOO_SMALL = 4
GG_ERR_ALIASING = 5
GG_ERR_HIP = 6

GG_ACT_SWIGLU = 0
GG_ACT_QGEGLU = 1
GG_ACT_NONE = -1
ACTIVATIONS = {"swiglu": GG_ACT_SWIGLU, "qgeglu": GG_ACT_QGEGLU}

EXPORTED = ("gg_status_string", "gg_packed_bytes", "gg_dgrad_workspace_bytes", "gg_pack_weights",
            "gg_forward_fc1_swiglu", "gg_forward_fc2", "gg_dgrad", "gg_round_bf16",
            "gg_dgrad_glu_workspace_bytes", "gg_forward_fc1_glu", "gg_dgrad_glu", "gg_dgrad_recompute",
            "gg_frag_bytes", "gg_pack_frag", "gg_forward_fc2_frag", "gg_dgrad_noalloc",
            "gg_scale_rows", "gg_scale_rows_backward",
            "gg_int8_quantize_rows", "gg_int8_packed_bytes", "gg_int8_pack", "gg_int8_workspace_bytes",
            "gg_int8_forward", "gg_int8_dgrad",
            "gg_adapter_forward", "gg_adapter_workspace_bytes", "gg_adapter_backward")


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run "
                          "`python -m moe_expert_grouped_ragged_amd._build` (or __graft_entry__.build())")
    lib = ctypes.CDLL(LIB_PATH)
    p, i64, sz, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
    lib.gg_status_string.argtypes = [i32]
    lib.gg_status_string.restype = ctypes.c_char_p
    lib.gg_packed_bytes.argtypes = [i64, i64, i64]
    lib.gg_packed_bytes.restype = sz
    lib.gg_frag_bytes.argtypes = [i64, i64, i64]
    lib.gg_frag_bytes.restype = sz
    lib.gg_dgrad_workspace_bytes.argtypes = [i64, i64]
    lib.gg_dgrad_workspace_bytes.restype = sz
    lib.gg_pack_weights.argtypes = [i64, i64, i64, ctypes.POINTER(p), ctypes.POINTER(p), p, sz, p]
    lib.gg_pack_frag.argtypes = [i64, i64, i64, p, sz, p, sz, p]
    lib.gg_forward_fc1_swiglu.argtypes = [p, p, i64, p, i64, i64, i64, p, p, p]
    lib.gg_forward_fc2.argtypes = [p, p, i64, p, i64, i64, i64, p, p]
    lib.gg_forward_fc2_frag.argtypes = [p, p, i64, p, p, i64, i64, i64, p, p]
    lib.gg_dgrad.argtypes = [p, p, p, i64, p, i64, i64, i64, p, sz, p, p]
    lib.gg_round_bf16.argtypes = [p, p, i64, p]
    lib.gg_dgrad_noalloc.argtypes = [p, p, p, i64, p, i64, i64, i64, p, p]
    lib.gg_dgrad_glu_workspace_bytes.argtypes = [i64, i64, i32]
    lib.gg_dgrad_glu_workspace_bytes.restype = sz
    lib.gg_forward_fc1_glu.argtypes = [p, p, i64, p, p, i64, i64, i64, i32, p, p, p, p]
    lib.gg_dgrad_glu.argtypes = [p, p, p, i64, p, p, i64, i64, i64, i32, p, p, sz, p, p, p]
    lib.gg_dgrad_recompute.argtypes = [p, p, p, i64, p, p, i64, i64, i64, i32, p, p, sz, p, p, p]
    lib.gg_scale_rows.argtypes = [p, p, i64, i64, p, p]
    lib.gg_scale_rows_backward.argtypes = [p, p, p, i64, i64, p, p, p]
    lib.gg_int8_quantize_rows.argtypes = [p, i64, i64, p, p, p]
    lib.gg_int8_packed_bytes.argtypes = [i64, i64, i64, i32]
    lib.gg_int8_packed_bytes.restype = sz
    lib.gg_int8_pack.argtypes = [p, p, i64, i64, i64, i32, p, sz, p]
    lib.gg_int8_workspace_bytes.argtypes = [i64, i64]
    lib.gg_int8_workspace_bytes.restype = sz
    lib.gg_int8_forward.argtypes = [p, p, i64, p, i64, i64, i64, i32, p, p, sz, p, p]
    lib.gg_int8_dgrad.argtypes = [p, p, p, i64, p, i64, i64, i64, i32, p, p, sz, p, p]
    f32 = ctypes.c_float
    lib.gg_adapter_forward.argtypes = [p, p, i64, p, p, i64, i64, i64, i64, f32, p, p, p, p]
    lib.gg_adapter_workspace_bytes.argtypes = [i64, i64, i64, i64, i64]
    lib.gg_adapter_workspace_bytes.restype = sz
    lib.gg_adapter_backward.argtypes = [p, p, p, p, i64, p, p, i64, i64, i64, i64, f32, p, p, sz, p, p, p, i32, p]
    for name in ("gg_pack_weights", "gg_pack_frag", "gg_forward_fc1_swiglu", "gg_forward_fc2",
                 "gg_forward_fc2_frag", "gg_dgrad", "gg_round_bf16", "gg_forward_fc1_glu", "gg_dgrad_glu",
                 "gg_dgrad_recompute", "gg_dgrad_noalloc", "gg_scale_rows", "gg_scale_rows_backward",
                 "gg_int8_quantize_rows", "gg_int8_pack", "gg_int8_forward", "gg_int8_dgrad",
                 "gg_adapter_forward", "gg_adapter_backward"):
        getattr(lib, name).restype = i32
    return lib


lib = _load()


class GGError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {lib.gg_status_string(status).decode()}")


def _check(status: int, what: str) -> None:
    if status != GG_OK:
        raise GGError(status, what)


def _stream_ptr(stream: Optional[torch.cuda.Stream], device: torch.device) -> int:
    """The given stream, or the current stream of the tensors' device; the
    library runs on the stream's device, so a stream of another device is
    refused."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device.index)   # current_stream(device).cuda_stream, 2 us sooner
    if stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    return int(stream.cuda_stream)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else int(t.data_ptr())


def _bf16_cuda(t: torch.Tensor, name: str, shape=None, device=None) -> torch.Tensor:
    """A contiguous bf16 device tensor (of the given shape, on the given device)."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch tensor")
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be bfloat16, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    return t


def _offsets(offsets: torch.Tensor, E: int, device) -> torch.Tensor:
    """The split offsets as given (no copy: a strided tensor is refused)."""
    if (not isinstance(offsets, torch.Tensor) or offsets.dtype != torch.int64 or not offsets.is_cuda
            or offsets.shape != (E + 1,) or offsets.device != device or not offsets.is_contiguous()):
        raise ValueError(f"offsets must be a contiguous int64 tensor of shape [E+1] on {device}")
    return offsets


def _packed(packed: torch.Tensor, E: int, H: int, F: int, device) -> torch.Tensor:
    """The packed weights: a contiguous bf16 buffer of at least packed_bytes(E, H, F)."""
    _bf16_cuda(packed, "packed", device=device)
    need = packed_bytes(E, H, F)
    if need == 0 or packed.numel() * 2 < need:
        raise ValueError(f"packed holds {packed.numel() * 2} bytes; E={E}, H={H}, F={F} needs {need}")
    return packed


def _frag(frag: Optional[torch.Tensor], E: int, H: int, F: int, device) -> Optional[torch.Tensor]:
    """An optional fragment buffer of at least frag_bytes(E, H, F)."""
    if frag is None:
        return None
    _bf16_cuda(frag, "frag", device=device)
    need = frag_bytes(E, H, F)
    if need == 0:
        raise ValueError(f"H={H}, F={F} has no fragment-ordered copies (needs H % 256 == 0 and F % 128 == 0)")
    if frag.numel() * 2 < need:
        raise ValueError(f"frag holds {frag.numel() * 2} bytes; E={E}, H={H}, F={F} needs {need}")
    return frag


def _out(t: Optional[torch.Tensor], shape, name: str, device) -> torch.Tensor:
    """A caller-given output (checked) or a new one."""
    if t is None:
        return torch.empty(*shape, dtype=torch.bfloat16, device=device)
    return _bf16_cuda(t, name, shape=shape, device=device)


def _workspace(ws: Optional[torch.Tensor], nbytes: int, device) -> torch.Tensor:
    """A caller-given workspace (contiguous, on the device, any dtype, >= nbytes) or a new one."""
    if ws is None:
        return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)
    if not isinstance(ws, torch.Tensor) or not ws.is_cuda or not ws.is_contiguous() or ws.device != device:
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    if ws.numel() * ws.element_size() < nbytes:
        raise ValueError(f"workspace holds {ws.numel() * ws.element_size()} bytes, {nbytes} needed")
    return ws


def packed_bytes(E: int, H: int, F: int) -> int:
    return int(lib.gg_packed_bytes(E, H, F))


def frag_bytes(E: int, H: int, F: int) -> int:
    """Bytes of the opt-in fragment-ordered copies (0 when the shape has none)."""
    return int(lib.gg_frag_bytes(E, H, F))


def has_frag(H: int, F: int) -> bool:
    return frag_bytes(1, H, F) > 0


def dgrad_workspace_bytes(M: int, F: int) -> int:
    return int(lib.gg_dgrad_workspace_bytes(M, F))


def gg_pack_weights(w1: Union[torch.Tensor, Sequence[torch.Tensor]],
                    w2: Union[torch.Tensor, Sequence[torch.Tensor]],
                    packed: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Pack frozen expert weights (w1[e]: [2F, H], gate rows then up rows;
    w2[e]: [H, F]) into one expert-major bf16 buffer of exactly the weights'
    size.  Returns the packed buffer (1-D, packed_bytes(E, H, F) / 2
    elements).  Per-expert views into it: ``expert_views(packed, E, H, F)``."""
    w1s = list(w1.unbind(0)) if isinstance(w1, torch.Tensor) else list(w1)
    w2s = list(w2.unbind(0)) if isinstance(w2, torch.Tensor) else list(w2)
    if len(w1s) != len(w2s) or not w1s:
        raise ValueError("w1 and w2 need the same, nonzero number of experts")
    for t in w1s + w2s:
        if t.dtype != torch.bfloat16:
            raise ValueError(f"expert weights must be bfloat16 (got {t.dtype}); "
                             "fp8/fp4/fp32 expert weights are not supported")
        if t.requires_grad:
            raise ValueError("expert base weights must be frozen (requires_grad=False)")
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("expert weights must be contiguous device tensors")
        if t.device != w1s[0].device:
            raise ValueError("expert weights must all be on one device")
    E = len(w1s)
    twoF, H = w1s[0].shape
    F = twoF // 2
    if twoF != 2 * F or any(t.shape != (2 * F, H) for t in w1s) or any(t.shape != (H, F) for t in w2s):
        raise ValueError("w1[e] must be [2F, H] and w2[e] must be [H, F] for every expert")
    nbytes = packed_bytes(E, H, F)
    if packed is None:
        packed = torch.empty(nbytes // 2, dtype=torch.bfloat16, device=w1s[0].device)
    _packed(packed, E, H, F, w1s[0].device)
    arr1 = (ctypes.c_void_p * E)(*[t.data_ptr() for t in w1s])
    arr2 = (ctypes.c_void_p * E)(*[t.data_ptr() for t in w2s])
    _check(lib.gg_pack_weights(E, H, F, arr1, arr2, packed.data_ptr(), packed.numel() * 2,
                               _stream_ptr(stream, w1s[0].device)), "gg_pack_weights")
    return packed


def gg_pack_frag(packed: torch.Tensor, E: int, H: int, F: int, frag: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Opt-in fragment-ordered copies of the packed weights (H % 256 == 0 and
    F % 128 == 0 only): returns the fragment buffer (frag_bytes(E, H, F) / 2
    bf16 elements) to pass as ``frag`` to the extended calls."""
    _packed(packed, E, H, F, packed.device)
    need = frag_bytes(E, H, F)
    if need == 0:
        raise ValueError(f"H={H}, F={F} has no fragment-ordered copies (needs H % 256 == 0 and F % 128 == 0)")
    if frag is None:
        frag = torch.empty(need // 2, dtype=torch.bfloat16, device=packed.device)
    _frag(frag, E, H, F, packed.device)
    _check(lib.gg_pack_frag(E, H, F, packed.data_ptr(), packed.numel() * 2, frag.data_ptr(), frag.numel() * 2,
                            _stream_ptr(stream, packed.device)), "gg_pack_frag")
    return frag


def expert_views(packed: torch.Tensor, E: int, H: int, F: int):
    """(w1_views, w2_views): per-expert views into the packed buffer.  A
    fragment buffer derived from it does not follow writes through them: call
    gg_pack_frag again."""
    per = packed_bytes(1, H, F) // 2
    w1 = [packed[e * per:e * per + 2 * F * H].view(2 * F, H) for e in range(E)]
    w2 = [packed[e * per + 2 * F * H:e * per + 3 * F * H].view(H, F) for e in range(E)]
    return w1, w2


def gg_forward_fc1_swiglu(x: torch.Tensor, offsets: torch.Tensor, packed: torch.Tensor,
                          E: int, H: int, F: int, save_h1: bool = True,
                          h1_out: Optional[torch.Tensor] = None, a_out: Optional[torch.Tensor] = None,
                          stream: Optional[torch.cuda.Stream] = None
                          ) -> Tuple[Optional[torch.Tensor], torch.Tensor]:
    """FC1 (x [M, H] -> H1 [M, 2F]) with the fused SwiGLU -> A [M, F]."""
    _bf16_cuda(x, "x")
    M, dev = x.shape[0], x.device
    _bf16_cuda(x, "x", shape=(M, H))
    _packed(packed, E, H, F, dev)
    off = _offsets(offsets, E, dev)
    if h1_out is not None:
        _bf16_cuda(h1_out, "h1_out", shape=(M, 2 * F), device=dev)
    a_out = _out(a_out, (M, F), "a_out", dev)
    if h1_out is None and save_h1:
        h1_out = _out(None, (M, 2 * F), "h1_out", dev)
    _check(lib.gg_forward_fc1_swiglu(x.data_ptr(), off.data_ptr(), M, packed.data_ptr(), E, H, F,
                                     _ptr(h1_out), a_out.data_ptr(), _stream_ptr(stream, dev)),
           "gg_forward_fc1_swiglu")
    return h1_out, a_out


def gg_forward_fc2(a: torch.Tensor, offsets: torch.Tensor, packed: torch.Tensor,
                   E: int, H: int, F: int, y: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """FC2: a [M, F] -> y [M, H]."""
    return gg_forward_fc2_frag(a, offsets, packed, None, E, H, F, y=y, stream=stream)


def gg_forward_fc2_frag(a: torch.Tensor, offsets: torch.Tensor, packed: torch.Tensor,
                        frag: Optional[torch.Tensor], E: int, H: int, F: int, y: Optional[torch.Tensor] = None,
                        stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """FC2 with an optional fragment buffer (gg_pack_frag): a [M, F] -> y [M, H]."""
    _bf16_cuda(a, "a")
    M, dev = a.shape[0], a.device
    _bf16_cuda(a, "a", shape=(M, F))
    _packed(packed, E, H, F, dev)
    fr = _frag(frag, E, H, F, dev)
    off = _offsets(offsets, E, dev)
    y = _out(y, (M, H), "y", dev)
    if fr is None:
        st = lib.gg_forward_fc2(a.data_ptr(), off.data_ptr(), M, packed.data_ptr(), E, H, F, y.data_ptr(),
                                _stream_ptr(stream, dev))
        _check(st, "gg_forward_fc2")
    else:
        st = lib.gg_forward_fc2_frag(a.data_ptr(), off.data_ptr(), M, packed.data_ptr(), fr.data_ptr(), E, H, F,
                                     y.data_ptr(), _stream_ptr(stream, dev))
        _check(st, "gg_forward_fc2_frag")
    return y


def gg_dgrad(dy: torch.Tensor, h1: torch.Tensor, offsets: torch.Tensor, packed: torch.Tensor,
             E: int, H: int, F: int, workspace: Optional[torch.Tensor] = None,
             dx: Optional[torch.Tensor] = None,
             stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Input gradient: dy [M, H], saved h1 [M, 2F] -> dx [M, H].  The
    workspace (bf16 [M, 2F] or any buffer of dgrad_workspace_bytes) receives dH1."""
    _bf16_cuda(dy, "dy")
    M, dev = dy.shape[0], dy.device
    _bf16_cuda(dy, "dy", shape=(M, H))
    _bf16_cuda(h1, "h1", shape=(M, 2 * F), device=dev)
    _packed(packed, E, H, F, dev)
    off = _offsets(offsets, E, dev)
    if dx is not None:
        _bf16_cuda(dx, "dx", shape=(M, H), device=dev)
    if workspace is not None:
        _workspace(workspace, dgrad_workspace_bytes(M, F), dev)
    else:
        workspace = torch.empty(M, 2 * F, dtype=torch.bfloat16, device=dev)
    dx = _out(dx, (M, H), "dx", dev)
    _check(lib.gg_dgrad(dy.data_ptr(), h1.data_ptr(), off.data_ptr(), M, packed.data_ptr(), E, H, F,
                        workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                        dx.data_ptr(), _stream_ptr(stream, dev)), "gg_dgrad")
    return dx


NOALLOC_SCRATCH_BYTES = 128 << 20    # GG_NOALLOC_SCRATCH_BYTES of include/gg.h


def gg_dgrad_noalloc(dy: torch.Tensor, h1: torch.Tensor, offsets: torch.Tensor, packed: torch.Tensor,
                     E: int, H: int, F: int, dx: Optional[torch.Tensor] = None,
                     stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """gg_dgrad with dH1 kept in the library's static per-GPU scratch (no
    workspace; 4*M*F <= NOALLOC_SCRATCH_BYTES).  Calls that overlap on one GPU
    race; with dx given, nothing is allocated."""
    _bf16_cuda(dy, "dy")
    M, dev = dy.shape[0], dy.device
    _bf16_cuda(dy, "dy", shape=(M, H))
    _bf16_cuda(h1, "h1", shape=(M, 2 * F), device=dev)
    _packed(packed, E, H, F, dev)
    off = _offsets(offsets, E, dev)
    dx = _out(dx, (M, H), "dx", dev)
    _check(lib.gg_dgrad_noalloc(dy.data_ptr(), h1.data_ptr(), off.data_ptr(), M, packed.data_ptr(), E, H, F,
                                dx.data_ptr(), _stream_ptr(stream, dev)), "gg_dgrad_noalloc")
    return dx


def _activation(activation) -> int:
    if isinstance(activation, str):
        if activation not in ACTIVATIONS:
            raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}")
        return ACTIVATIONS[activation]
    return int(activation)


def _probs_cuda(probs: Optional[torch.Tensor], M: int, device, name: str = "probs") -> Optional[torch.Tensor]:
    if probs is None:
        return None
    if (probs.dtype != torch.float32 or not probs.is_cuda or probs.shape != (M,) or not probs.is_contiguous()
            or probs.device != device):
        raise ValueError(f"{name} must be a contiguous float32 tensor of shape [M] on {device}")
    return probs


def dgrad_glu_workspace_bytes(M: int, F: int, with_dprobs: bool) -> int:
    return int(lib.gg_dgrad_glu_workspace_bytes(M, F, int(bool(with_dprobs))))


def gg_forward_fc1_glu(x: torch.Tensor, offsets: torch.Tensor, packed: torch.Tensor,
                       E: int, H: int, F: int, activation="swiglu", probs: Optional[torch.Tensor] = None,
                       save_h1: bool = True, h1_out: Optional[torch.Tensor] = None,
                       a_out: Optional[torch.Tensor] = None, frag: Optional[torch.Tensor] = None,
                       stream: Optional[torch.cuda.Stream] = None
                       ) -> Tuple[Optional[torch.Tensor], torch.Tensor]:
    """FC1 with the fused activation ("swiglu" | "qgeglu"), optionally scaled
    per row by probs (float32 [M]) -> (H1 or None, A).  frag: optional
    fragment buffer (gg_pack_frag) of the same weights."""
    _bf16_cuda(x, "x")
    M, dev = x.shape[0], x.device
    _bf16_cuda(x, "x", shape=(M, H))
    _packed(packed, E, H, F, dev)
    fr = _frag(frag, E, H, F, dev)
    off = _offsets(offsets, E, dev)
    pr = _probs_cuda(probs, M, dev)
    if h1_out is not None:
        _bf16_cuda(h1_out, "h1_out", shape=(M, 2 * F), device=dev)
    a_out = _out(a_out, (M, F), "a_out", dev)
    if h1_out is None and save_h1:
        h1_out = _out(None, (M, 2 * F), "h1_out", dev)
    _check(lib.gg_forward_fc1_glu(x.data_ptr(), off.data_ptr(), M, packed.data_ptr(), _ptr(fr), E, H, F,
                                  _activation(activation), _ptr(pr), _ptr(h1_out), a_out.data_ptr(),
                                  _stream_ptr(stream, dev)), "gg_forward_fc1_glu")
    return h1_out, a_out


def gg_dgrad_glu(dy: torch.Tensor, h1: torch.Tensor, offsets: torch.Tensor, packed: torch.Tensor,
                 E: int, H: int, F: int, activation="swiglu", probs: Optional[torch.Tensor] = None,
                 want_dprobs: bool = True, workspace: Optional[torch.Tensor] = None,
                 dx: Optional[torch.Tensor] = None, dprobs: Optional[torch.Tensor] = None,
                 frag: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None
                 ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Input gradient of gg_forward_fc1_glu + FC2 -> (dx, dprobs or None).
    The workspace (a byte buffer of dgrad_glu_workspace_bytes) keeps dH1 [M, 2F]
    bf16 at its start.  frag: optional fragment buffer (gg_pack_frag)."""
    _bf16_cuda(dy, "dy")
    M, dev = dy.shape[0], dy.device
    _bf16_cuda(dy, "dy", shape=(M, H))
    _bf16_cuda(h1, "h1", shape=(M, 2 * F), device=dev)
    _packed(packed, E, H, F, dev)
    fr = _frag(frag, E, H, F, dev)
    off = _offsets(offsets, E, dev)
    pr = _probs_cuda(probs, M, dev)
    dprobs = _probs_cuda(dprobs, M, dev, "dprobs")
    if dx is not None:
        _bf16_cuda(dx, "dx", shape=(M, H), device=dev)
    with_dp = dprobs is not None or want_dprobs
    if workspace is not None:
        _workspace(workspace, dgrad_glu_workspace_bytes(M, F, with_dp), dev)
    if dprobs is None and want_dprobs:
        dprobs = torch.empty(M, dtype=torch.float32, device=dev)
    workspace = _workspace(workspace, dgrad_glu_workspace_bytes(M, F, with_dp), dev)
    dx = _out(dx, (M, H), "dx", dev)
    _check(lib.gg_dgrad_glu(dy.data_ptr(), h1.data_ptr(), off.data_ptr(), M, packed.data_ptr(), _ptr(fr), E, H, F,
                            _activation(activation), _ptr(pr), workspace.data_ptr(),
                            workspace.numel() * workspace.element_size(), dx.data_ptr(), _ptr(dprobs),
                            _stream_ptr(stream, dev)), "gg_dgrad_glu")
    return dx, dprobs


def gg_dgrad_recompute(dy: torch.Tensor, x: torch.Tensor, offsets: torch.Tensor, packed: torch.Tensor,
                       E: int, H: int, F: int, activation="swiglu", probs: Optional[torch.Tensor] = None,
                       want_dprobs: bool = False, workspace: Optional[torch.Tensor] = None,
                       dx: Optional[torch.Tensor] = None, dprobs: Optional[torch.Tensor] = None,
                       frag: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None
                       ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Input gradient without a saved H1: FC1 is recomputed from the forward
    input x [M, H] inside the call -> (dx, dprobs or None).  The workspace
    ends up holding dH1 [M, 2F] bf16 at its start."""
    _bf16_cuda(dy, "dy")
    M, dev = dy.shape[0], dy.device
    _bf16_cuda(dy, "dy", shape=(M, H))
    _bf16_cuda(x, "x", shape=(M, H), device=dev)
    _packed(packed, E, H, F, dev)
    fr = _frag(frag, E, H, F, dev)
    off = _offsets(offsets, E, dev)
    pr = _probs_cuda(probs, M, dev)
    dprobs = _probs_cuda(dprobs, M, dev, "dprobs")
    if dx is not None:
        _bf16_cuda(dx, "dx", shape=(M, H), device=dev)
    with_dp = dprobs is not None or want_dprobs
    if workspace is not None:
        _workspace(workspace, dgrad_glu_workspace_bytes(M, F, with_dp), dev)
    if dprobs is None and want_dprobs:
        dprobs = torch.empty(M, dtype=torch.float32, device=dev)
    workspace = _workspace(workspace, dgrad_glu_workspace_bytes(M, F, with_dp), dev)
    dx = _out(dx, (M, H), "dx", dev)
    _check(lib.gg_dgrad_recompute(dy.data_ptr(), x.data_ptr(), off.data_ptr(), M, packed.data_ptr(), _ptr(fr),
                                  E, H, F, _activation(activation), _ptr(pr), workspace.data_ptr(),
                                  workspace.numel() * workspace.element_size(), dx.data_ptr(), _ptr(dprobs),
                                  _stream_ptr(stream, dev)), "gg_dgrad_recompute")
    return dx, dprobs


def gg_round_bf16(x: torch.Tensor, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Diagnostic: device fp32 -> bf16 rounding as used by the epilogues."""
    if x.dtype != torch.float32 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous float32 device tensor")
    out = torch.empty(x.shape, dtype=torch.bfloat16, device=x.device)
    _check(lib.gg_round_bf16(x.data_ptr(), out.data_ptr(), x.numel(), _stream_ptr(stream, x.device)),
           "gg_round_bf16")
    return out


def gg_scale_rows(x: torch.Tensor, probs: torch.Tensor, out: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Router probability on the FC1 input: out [M, H] = bf16(probs[r] * x[r])
    for every row (out may be x).  x bf16 [M, H]; probs fp32 [M]."""
    x = _bf16_cuda(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be [M, H]")
    M, H = x.shape
    pr = _probs_cuda(probs, M, x.device)
    if pr is None:
        raise ValueError("probs is required")
    out = _out(out, (M, H), "out", x.device)
    _check(lib.gg_scale_rows(x.data_ptr(), pr.data_ptr(), M, H, out.data_ptr(), _stream_ptr(stream, x.device)),
           "gg_scale_rows")
    return out


def gg_scale_rows_backward(dxs: torch.Tensor, x: torch.Tensor, probs: torch.Tensor, want_dprobs: bool = True,
                           dx: Optional[torch.Tensor] = None, dprobs: Optional[torch.Tensor] = None,
                           stream: Optional[torch.cuda.Stream] = None):
    """Input gradient of gg_scale_rows given dxs = dL/dx' [M, H] and the
    unscaled x: (dx = bf16(probs[r] * dxs[r]), dprobs[r] = sum_h dxs*x in fp32
    or None).  dx may be dxs."""
    dxs = _bf16_cuda(dxs, "dxs")
    if dxs.dim() != 2:
        raise ValueError("dxs must be [M, H]")
    M, H = dxs.shape
    x = _bf16_cuda(x, "x", (M, H), dxs.device)
    pr = _probs_cuda(probs, M, dxs.device)
    if pr is None:
        raise ValueError("probs is required")
    dx = _out(dx, (M, H), "dx", dxs.device)
    dprobs = _probs_cuda(dprobs, M, dxs.device, "dprobs")
    if dprobs is None and want_dprobs:
        dprobs = torch.empty(M, dtype=torch.float32, device=dxs.device)
    _check(lib.gg_scale_rows_backward(dxs.data_ptr(), x.data_ptr(), pr.data_ptr(), M, H, dx.data_ptr(),
                                      _ptr(dprobs), _stream_ptr(stream, dxs.device)), "gg_scale_rows_backward")
    return dx, dprobs


def _allocates_on_stream(fn):
    """For a call with a `stream`: what it allocates comes from that stream's
    memory, so nothing queued elsewhere still uses it when the call's kernels run, and
    what it returns is not given out again before the current stream's work on it is done."""
    at = list(inspect.signature(fn).parameters).index("stream")

    @functools.wraps(fn)
    def call(*args, **kw):
        stream = kw.get("stream") if len(args) <= at else args[at]
        if stream is None:
            return fn(*args, **kw)
        current = torch.cuda.current_stream(stream.device)
        with torch.cuda.stream(stream):
            out = fn(*args, **kw)
        for t in out if isinstance(out, tuple) else (out,):
            if t is not None:
                t.record_stream(current)
        return out

    return call


def _typed_cuda(t: torch.Tensor, dtype, name: str, shape, device) -> torch.Tensor:
    """A contiguous device tensor of the given dtype and shape (None: any size there), on the given device."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch tensor")
    if t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} device tensor")
    if t.dim() != len(shape) or any(w is not None and n != w for n, w in zip(t.shape, shape)):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    return t


def int8_packed_bytes(E: int, N: int, K: int, transposed: bool = False) -> int:
    return int(lib.gg_int8_packed_bytes(E, N, K, int(bool(transposed))))


def int8_workspace_bytes(M: int, width: int) -> int:
    """Workspace of gg_int8_forward (width = K) or gg_int8_dgrad (width = N)."""
    return int(lib.gg_int8_workspace_bytes(M, width))


@_allocates_on_stream
def gg_int8_quantize_rows(x: torch.Tensor, q: Optional[torch.Tensor] = None, s: Optional[torch.Tensor] = None,
                          stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Rows of x (bf16 [M, K]) to int8 with one scale each: (q int8 [M, K], s
    float32 [M]), x ~ s[:, None] * q.  Frozen weights [E, N, K] are quantized
    for each output channel as x = w.view(E * N, K)."""
    _bf16_cuda(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be [M, K]")
    M, K = x.shape
    q = torch.empty(M, K, dtype=torch.int8, device=x.device) if q is None else _typed_cuda(q, torch.int8, "q", (M, K), x.device)
    s = torch.empty(M, dtype=torch.float32, device=x.device) if s is None else _probs_cuda(s, M, x.device, "s")
    _check(lib.gg_int8_quantize_rows(x.data_ptr(), M, K, q.data_ptr(), s.data_ptr(), _stream_ptr(stream, x.device)),
           "gg_int8_quantize_rows")
    return q, s


def _int8_pack(wq, ws, transposed, packed, stream):
    _typed_cuda(wq, torch.int8, "wq", (None, None, None), None)
    E, N, K = wq.shape
    _typed_cuda(ws, torch.float32, "ws", (E, N), wq.device)
    need = int8_packed_bytes(E, N, K, transposed)
    if need == 0:
        raise ValueError(f"E={E}, N={N}, K={K} is outside the limits of the int8 calls")
    if packed is None:
        packed = torch.empty(need, dtype=torch.uint8, device=wq.device)
    _workspace(packed, need, wq.device)
    _check(lib.gg_int8_pack(wq.data_ptr(), ws.data_ptr(), E, N, K, int(transposed), packed.data_ptr(),
                            packed.numel() * packed.element_size(), _stream_ptr(stream, wq.device)), "gg_int8_pack")
    if not packed.is_inference():       # those have no version
        torch.autograd.graph.increment_version(packed)      # as for any write to it; its views see it too
        packed._gg_int8_holds = (E, N, K, bool(transposed)), packed._version
    return packed


@_allocates_on_stream
def gg_int8_pack(wq: torch.Tensor, ws: torch.Tensor, packed: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """8-bit weights wq (int8 [E, N, K]) with channel scales ws (float32
    [E, N]), laid out once for gg_int8_forward: a byte buffer of
    int8_packed_bytes(E, N, K).  The tensor returned is refused where another layout is needed."""
    return _int8_pack(wq, ws, False, packed, stream)


@_allocates_on_stream
def gg_int8_pack_transposed(wq: torch.Tensor, ws: torch.Tensor, packed: Optional[torch.Tensor] = None,
                            stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The same weights laid out for gg_int8_dgrad (int8_packed_bytes(E, N, K, True) bytes)."""
    return _int8_pack(wq, ws, True, packed, stream)


def _int8_packed(packed: torch.Tensor, E: int, N: int, K: int, transposed: bool, device) -> torch.Tensor:
    need = int8_packed_bytes(E, N, K, transposed)
    if need == 0:
        raise ValueError(f"E={E}, N={N}, K={K} is outside the limits of the int8 calls")
    if not isinstance(packed, torch.Tensor) or not packed.is_cuda or not packed.is_contiguous() or packed.device != device:
        raise ValueError(f"packed must be a contiguous tensor on {device}")
    if packed.numel() * packed.element_size() < need:
        raise ValueError(f"packed holds {packed.numel() * packed.element_size()} bytes, {need} needed")
    # The two layouts of a matrix may be equally large: a tensor that was packed, and not written since, says what it
    # holds (a copy or a view of one does not).
    holds = getattr(packed, "_gg_int8_holds", None)
    if holds is not None and holds[0] != (E, N, K, transposed) and holds[1] == packed._version:
        raise ValueError(f"packed holds (E, N, K, transposed) = {holds[0]}, not {(E, N, K, transposed)}")
    return packed


@_allocates_on_stream
def gg_int8_forward(x: torch.Tensor, offsets: torch.Tensor, packed: torch.Tensor, E: int, N: int, K: int,
                    activation=None, save_a: bool = False, a_out: Optional[torch.Tensor] = None,
                    y: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """(y [M, N], A or None): the rows quantized to 8 bits, times each expert's
    8-bit matrix (gg_int8_pack).  activation None: x is [M, K]; "swiglu" |
    "qgeglu": x is H1 [M, 2K], the product's operand is A = act(gate) * up
    [M, K], returned with save_a (or given a_out)."""
    _bf16_cuda(x, "x")
    dev, M = x.device, x.shape[0]
    act = GG_ACT_NONE if activation is None else _activation(activation)
    _bf16_cuda(x, "x", shape=(M, K if act == GG_ACT_NONE else 2 * K))
    _int8_packed(packed, E, N, K, False, dev)
    off = _offsets(offsets, E, dev)
    if a_out is not None:
        _bf16_cuda(a_out, "a_out", shape=(M, K), device=dev)
    if act == GG_ACT_NONE and (save_a or a_out is not None):
        raise ValueError("A exists with an activation only")
    workspace = _workspace(workspace, int8_workspace_bytes(M, K), dev)
    if a_out is None and save_a:
        a_out = _out(None, (M, K), "a_out", dev)
    y = _out(y, (M, N), "y", dev)
    _check(lib.gg_int8_forward(x.data_ptr(), off.data_ptr(), M, packed.data_ptr(), E, N, K, act, _ptr(a_out),
                               workspace.data_ptr(), workspace.numel() * workspace.element_size(), y.data_ptr(),
                               _stream_ptr(stream, dev)), "gg_int8_forward")
    return y, a_out


@_allocates_on_stream
def gg_int8_dgrad(dy: torch.Tensor, offsets: torch.Tensor, packed: torch.Tensor, E: int, N: int, K: int,
                  h1: Optional[torch.Tensor] = None, activation=None, save_dh1: bool = True,
                  dh1_out: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None
                  ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """(dx [M, K], dH1 or None): input gradient through 8-bit weights
    (gg_int8_pack_transposed).  activation None: dy is [M, N]; else N = 2F, dy
    is dA [M, F], h1 the saved [M, 2F], and dH1 [M, 2F] is returned unless
    save_dh1 is False."""
    _bf16_cuda(dy, "dy")
    dev, M = dy.device, dy.shape[0]
    act = GG_ACT_NONE if activation is None else _activation(activation)
    if (act == GG_ACT_NONE) != (h1 is None):
        raise ValueError("h1 and an activation go together")
    _bf16_cuda(dy, "dy", shape=(M, N if act == GG_ACT_NONE else N // 2))
    if h1 is not None:
        _bf16_cuda(h1, "h1", shape=(M, N), device=dev)
    _int8_packed(packed, E, N, K, True, dev)
    off = _offsets(offsets, E, dev)
    if dh1_out is not None:
        if h1 is None:
            raise ValueError("dH1 exists with an activation only")
        _bf16_cuda(dh1_out, "dh1_out", shape=(M, N), device=dev)
    workspace = _workspace(workspace, int8_workspace_bytes(M, N), dev)
    if dh1_out is None and h1 is not None and save_dh1:
        dh1_out = _out(None, (M, N), "dh1_out", dev)
    dx = _out(dx, (M, K), "dx", dev)
    _check(lib.gg_int8_dgrad(dy.data_ptr(), _ptr(h1), off.data_ptr(), M, packed.data_ptr(), E, N, K, act,
                             _ptr(dh1_out), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                             dx.data_ptr(), _stream_ptr(stream, dev)), "gg_int8_dgrad")
    return dx, dh1_out


ADAPTER_MAX_RANK = 64    # GG_ADAPTER_MAX_RANK of include/gg.h


def adapter_workspace_bytes(M: int, E: int, N: int, K: int, r: int) -> int:
    return int(lib.gg_adapter_workspace_bytes(M, E, N, K, r))


def _adapter(x, offsets, a, b):
    """The checked operands' sizes (M, E, N, K, r)."""
    _bf16_cuda(x, "x")
    _bf16_cuda(a, "a", device=x.device)
    if x.dim() != 2 or a.dim() != 3 or a.shape[2] != x.shape[1]:
        raise ValueError("x must be [M, K] and a [E, r, K]")
    E, r, K = a.shape
    _bf16_cuda(b, "b", device=x.device)
    if b.dim() != 3 or b.shape[0] != E or b.shape[2] != r:
        raise ValueError(f"b must be [E, N, r] with E={E}, r={r}, got {tuple(b.shape)}")
    if not 1 <= r <= ADAPTER_MAX_RANK:
        raise ValueError(f"the rank must be 1 .. {ADAPTER_MAX_RANK}, got {r}")
    _offsets(offsets, E, x.device)
    return x.shape[0], E, b.shape[1], K, r


@_allocates_on_stream
def gg_adapter_forward(x: torch.Tensor, offsets: torch.Tensor, a: torch.Tensor, b: torch.Tensor, scale: float,
                       base: Optional[torch.Tensor] = None, u: Optional[torch.Tensor] = None,
                       y: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None
                       ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Low-rank adapters: y = base + scale * (x a_e^T) b_e^T for the rows of
    each expert -> (y [M, N], u = x a_e^T [M, r] for the backward).  a [E, r, K],
    b [E, N, r], all bf16.  y may be base (in place)."""
    M, E, N, K, r = _adapter(x, offsets, a, b)
    dev = x.device
    if base is not None:
        _bf16_cuda(base, "base", shape=(M, N), device=dev)
    if u is not None:
        _bf16_cuda(u, "u", shape=(M, r), device=dev)
    y = _out(y, (M, N), "y", dev)
    u = _out(u, (M, r), "u", dev)
    _check(lib.gg_adapter_forward(x.data_ptr(), offsets.data_ptr(), M, a.data_ptr(), b.data_ptr(), E, N, K, r, scale,
                                  _ptr(base), u.data_ptr(), y.data_ptr(), _stream_ptr(stream, dev)),
           "gg_adapter_forward")
    return y, u


@_allocates_on_stream
def gg_adapter_backward(dy: torch.Tensor, x: torch.Tensor, u: torch.Tensor, offsets: torch.Tensor, a: torch.Tensor,
                        b: torch.Tensor, scale: float, base: Optional[torch.Tensor] = None,
                        dx: Optional[torch.Tensor] = None, da: Optional[torch.Tensor] = None,
                        db: Optional[torch.Tensor] = None, accumulate: bool = False,
                        workspace: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None
                        ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Gradients of gg_adapter_forward: (dx = base + du a_e [M, K] bf16, da
    [E, r, K] float32, db [E, N, r] float32) with du = scale * dy b_e.  base is
    the frozen product's input gradient (dx may be base).  accumulate: da and
    db are given and added to."""
    M, E, N, K, r = _adapter(x, offsets, a, b)
    dev = x.device
    _bf16_cuda(dy, "dy", shape=(M, N), device=dev)
    _bf16_cuda(u, "u", shape=(M, r), device=dev)
    if base is not None:
        _bf16_cuda(base, "base", shape=(M, K), device=dev)
    if accumulate and (da is None or db is None):
        raise ValueError("accumulate needs da and db")
    if da is not None:
        _typed_cuda(da, torch.float32, "da", (E, r, K), dev)
    if db is not None:
        _typed_cuda(db, torch.float32, "db", (E, N, r), dev)
    if dx is not None:
        _bf16_cuda(dx, "dx", shape=(M, K), device=dev)
    workspace = _workspace(workspace, adapter_workspace_bytes(M, E, N, K, r), dev)
    dx = _out(dx, (M, K), "dx", dev)
    da = torch.empty(E, r, K, dtype=torch.float32, device=dev) if da is None else da
    db = torch.empty(E, N, r, dtype=torch.float32, device=dev) if db is None else db
    _check(lib.gg_adapter_backward(dy.data_ptr(), x.data_ptr(), u.data_ptr(), offsets.data_ptr(), M, a.data_ptr(),
                                   b.data_ptr(), E, N, K, r, scale, _ptr(base), workspace.data_ptr(),
                                   workspace.numel() * workspace.element_size(), dx.data_ptr(), da.data_ptr(),
                                   db.data_ptr(), int(bool(accumulate)), _stream_ptr(stream, dev)),
           "gg_adapter_backward")
    return dx, da, db


class ScaleRows(torch.autograd.Function):
    """Autograd wrapper of gg_scale_rows: x' = bf16(probs[r] * x[r]); the
    backward gives dx and, when probs requires grad, dprobs."""

    @staticmethod
    def forward(ctx, x, probs):
        ctx.save_for_backward(x, probs)
        return gg_scale_rows(x, probs.detach())

    @staticmethod
    def backward(ctx, g):
        x, probs = ctx.saved_tensors
        dx, dprobs = gg_scale_rows_backward(g.contiguous(), x, probs.detach(),
                                            want_dprobs=ctx.needs_input_grad[1])
        return dx, dprobs


class FrozenExpertMLP(torch.autograd.Function):
    """Autograd wrapper: forward FC1 -> SwiGLU -> FC2, backward = input
    gradient only (the packed base weights are frozen)."""

    @staticmethod
    def forward(ctx, x, offsets, packed, E, H, F):
        h1, a = gg_forward_fc1_swiglu(x, offsets, packed, E, H, F, save_h1=True)
        y = gg_forward_fc2(a, offsets, packed, E, H, F)
        ctx.save_for_backward(h1, offsets, packed)
        ctx.shape = (E, H, F)
        return y

    @staticmethod
    def backward(ctx, dy):
        h1, offsets, packed = ctx.saved_tensors
        E, H, F = ctx.shape
        dx = gg_dgrad(dy.contiguous(), h1, offsets, packed, E, H, F)
        return dx, None, None, None, None, None


class Int8Experts(NamedTuple):
    """Frozen gated expert MLPs in 8 bits: W1 [E, 2F, H] and W2 [E, H, F] laid
    out for the forward (fc1, fc2) and for the input gradient (fc1_t, fc2_t)."""
    E: int
    H: int
    F: int
    fc1: torch.Tensor
    fc2: torch.Tensor
    fc1_t: torch.Tensor
    fc2_t: torch.Tensor


def int8_experts(w1: torch.Tensor, w2: torch.Tensor) -> Int8Experts:
    """Quantize frozen bf16 weights w1 [E, 2F, H] (gate rows, then up rows) and
    w2 [E, H, F] for each output channel and lay them out for Int8AdapterExpertMLP."""
    if w1.requires_grad or w2.requires_grad:
        raise ValueError("expert base weights must be frozen (requires_grad=False)")
    if w1.dim() != 3 or w2.dim() != 3 or w1.shape[0] != w2.shape[0] or w1.shape[1] != 2 * w2.shape[2] \
            or w1.shape[2] != w2.shape[1]:
        raise ValueError("w1 must be [E, 2F, H] and w2 [E, H, F]")
    E, H, F = w2.shape
    packs = []
    for w in (w1, w2):
        q, s = gg_int8_quantize_rows(w.reshape(-1, w.shape[2]))
        q, s = q.view(w.shape), s.view(w.shape[0], w.shape[1])
        packs.append((gg_int8_pack(q, s), gg_int8_pack_transposed(q, s)))
    return Int8Experts(E, H, F, packs[0][0], packs[1][0], packs[0][1], packs[1][1])


class Int8AdapterExpertMLP(torch.autograd.Function):
    """The gated expert MLP over frozen 8-bit weights with a low-rank adapter on
    each of its two products:

      H1 = int8(X) W1^T + scale (X a1^T) b1^T      A = act(gate) * up
      Y  = int8(A) W2^T + scale (A a2^T) b2^T

    apply(x, offsets, experts, a1, b1, a2, b2, scale, activation) with experts
    from int8_experts, a1 [E, r1, H], b1 [E, 2F, r1], a2 [E, r2, F],
    b2 [E, H, r2] (bf16).  The backward gives dX and the adapters' gradients,
    those that are needed (FC1's part is left out where neither x, a1 nor b1
    need one); the base weights have none."""

    @staticmethod
    def forward(ctx, x, offsets, experts, a1, b1, a2, b2, scale, activation="swiglu"):
        E, H, F = experts.E, experts.H, experts.F
        a1, b1, a2, b2 = (t.detach() for t in (a1, b1, a2, b2))
        h1, _ = gg_int8_forward(x, offsets, experts.fc1, E, 2 * F, H)
        h1, u1 = gg_adapter_forward(x, offsets, a1, b1, scale, base=h1, y=h1)
        y, a = gg_int8_forward(h1, offsets, experts.fc2, E, H, F, activation=activation, save_a=True)
        y, u2 = gg_adapter_forward(a, offsets, a2, b2, scale, base=y, y=y)
        ctx.save_for_backward(x, offsets, h1, a, u1, u2, a1, b1, a2, b2)
        ctx.experts, ctx.scale, ctx.activation = experts, scale, activation
        return y

    @staticmethod
    def backward(ctx, dy):
        x, offsets, h1, a, u1, u2, a1, b1, a2, b2 = ctx.saved_tensors
        w, scale = ctx.experts, ctx.scale
        need = ctx.needs_input_grad
        fc1 = need[0] or need[3] or need[4]      # something that lies before A
        dy, da, dx, ga1, gb1 = dy.contiguous(), None, None, None, None
        if fc1:
            da, _ = gg_int8_dgrad(dy, offsets, w.fc2_t, w.E, w.H, w.F)
        da, ga2, gb2 = gg_adapter_backward(dy, a, u2, offsets, a2, b2, scale, base=da, dx=da)
        if fc1:
            dx, dh1 = gg_int8_dgrad(da, offsets, w.fc1_t, w.E, 2 * w.F, w.H, h1=h1, activation=ctx.activation)
            dx, ga1, gb1 = gg_adapter_backward(dh1, x, u1, offsets, a1, b1, scale, base=dx, dx=dx)
        grads = [g.to(torch.bfloat16) if n else None for g, n in zip((ga1, gb1, ga2, gb2), need[3:7])]
        return dx if need[0] else None, None, None, *grads, None, None
