"""GB300 (sm_103a) flash-CCE ORPO head: Python binding of liborpo_head.

The functions here carry the C entry points' names and only marshal arguments:
every step of the head runs in the library's CUDA kernels.  PyTorch supplies
device memory and the current CUDA stream.  If the library has not been built
(``python -c "import __graft_entry__ as g; g.build()"``) the calls raise; there
is no fallback implementation.
"""

from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import warnings

import torch

from . import build as _build

__all__ = [
    "OrpoError", "load", "lib_path", "orpo_head_workspace_bytes", "orpo_head_fwd", "orpo_loss",
    "orpo_head_bwd", "orpo_status_string", "orpo_debug_gemm", "OrpoHead", "STATUS_BITS",
    "orpo_profile_start", "orpo_profile_stop", "orpo_head_fwd_static", "orpo_debug_wait_timeout",
    "orpo_pref_loss", "PREF_KINDS", "orpo_head_q_workspace_bytes", "orpo_head_fwd_q", "orpo_head_bwd_q",
    "use_bounds_checked_library", "orpo_head_logits_q", "orpo_head_logits_q_workspace_bytes", "orpo_beam_select", "orpo_beam_select_workspace_bytes",
    "orpo_beam_reorder", "BeamDecoder", "orpo_logits_adjust", "orpo_beam_history", "orpo_pages_workspace_bytes",
    "orpo_pages_advance", "orpo_pages_copy", "orpo_pages_release", "orpo_pages_compact", "PagedStates",
]

STATUS_BITS = {"target": 1 << 4, "seqid": 1 << 5, "empty": 1 << 6, "nonfinite": 1 << 7, "timeout": 1 << 8,
               "bounds": 1 << 9, "parent": 1 << 10, "page": 1 << 11, "full": 1 << 12, "mask": 1 << 13}
MAX_PAIRS = 2048
MAX_BEAMS = 64
MAX_SELECT = 64

_lib = None
_fast = None


class OrpoError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {orpo_status_string(code)} (code {code})")
        self.code = code


_variant = "release"


def lib_path() -> str:
    return _build.DEBUG_LIB_PATH if _variant == "debug" else _build.LIB_PATH


def use_bounds_checked_library() -> None:
    """Bind this process to liborpo_head_debug.so (build(debug=True)) instead of liborpo_head.so.

    The bounds-checked build checks every computed index against its buffer and reports a miss
    as ORPO_STATUS_BOUNDS; its arithmetic is the release build's.  Call before the first use."""
    global _variant
    if _lib is not None and _variant != "debug":
        raise RuntimeError("the release library is already loaded in this process")
    _variant = "debug"


def load():
    """Load the library (built in-tree); raises if it is missing."""
    global _lib, _fast
    if _lib is not None:
        return _lib
    path = lib_path()
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with orpo_preference_loss_gb300.build.build()")
    L = ctypes.CDLL(path)
    vp, i64, i32, f32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
    L.orpo_head_workspace_bytes.argtypes = [i64, i64, i64]
    L.orpo_head_workspace_bytes.restype = sz
    L.orpo_head_fwd.argtypes = [vp, vp, vp, vp, i64, i64, i64, f32, vp, vp, vp, sz, vp, vp]
    L.orpo_head_fwd.restype = ctypes.c_int
    L.orpo_loss.argtypes = [vp, vp, vp, i64, i32, f32, vp, vp, vp, vp, vp]
    L.orpo_loss.restype = ctypes.c_int
    L.orpo_head_bwd.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, f32, vp, vp, ctypes.c_int, vp, sz, vp, vp]
    L.orpo_head_bwd.restype = ctypes.c_int
    L.orpo_status_string.argtypes = [ctypes.c_int]
    L.orpo_status_string.restype = ctypes.c_char_p
    L.orpo_debug_gemm.argtypes = [vp, vp, vp, i64, i64, i64, ctypes.c_int, ctypes.c_int, vp, vp]
    L.orpo_debug_gemm.restype = ctypes.c_int
    L.orpo_pref_loss.argtypes = [ctypes.c_int, vp, vp, vp, i64, i32, f32, f32, vp, vp, vp, vp, vp, vp]
    L.orpo_pref_loss.restype = ctypes.c_int
    L.orpo_head_q_workspace_bytes.argtypes = [i64, i64, i64]
    L.orpo_head_q_workspace_bytes.restype = sz
    L.orpo_head_fwd_q.argtypes = [vp, vp, vp, vp, ctypes.c_int, ctypes.c_int, vp, vp, i64, i64, i64, f32, vp, vp, vp,
                                  sz, vp, vp]
    L.orpo_head_fwd_q.restype = ctypes.c_int
    L.orpo_head_bwd_q.argtypes = [vp, vp, vp, vp, ctypes.c_int, ctypes.c_int, vp, vp, vp, vp, i64, i64, i64, f32, vp,
                                  vp, ctypes.c_int, vp, sz, vp, vp]
    L.orpo_head_bwd_q.restype = ctypes.c_int
    L.orpo_head_fwd_static.argtypes = [vp, vp, vp, vp, i64, i64, i64, f32, vp, vp, vp, vp]
    L.orpo_head_fwd_static.restype = ctypes.c_int
    L.orpo_debug_wait_timeout.argtypes = [vp, i64, vp]
    L.orpo_debug_wait_timeout.restype = ctypes.c_int
    L.orpo_head_block_max_elems.argtypes = [i64, i64]
    L.orpo_head_block_max_elems.restype = sz
    L.orpo_head_fwd_bmax.argtypes = [vp, vp, vp, vp, i64, i64, i64, f32, vp, vp, vp, vp, sz, vp, vp]
    L.orpo_head_fwd_bmax.restype = ctypes.c_int
    L.orpo_head_bwd_skip.argtypes = [vp, vp, vp, vp, vp, vp, vp, f32, i64, i64, i64, f32, vp, vp, ctypes.c_int, vp,
                                     sz, vp, vp]
    L.orpo_head_bwd_skip.restype = ctypes.c_int
    L.orpo_head_fwd_q_bmax.argtypes = [vp, vp, vp, vp, ctypes.c_int, ctypes.c_int, vp, vp, i64, i64, i64, f32, vp,
                                       vp, vp, vp, sz, vp, vp]
    L.orpo_head_fwd_q_bmax.restype = ctypes.c_int
    L.orpo_head_bwd_q_skip.argtypes = [vp, vp, vp, vp, ctypes.c_int, ctypes.c_int, vp, vp, vp, vp, vp, f32, i64, i64,
                                       i64, f32, vp, vp, ctypes.c_int, vp, sz, vp, vp]
    L.orpo_head_bwd_q_skip.restype = ctypes.c_int
    L.orpo_head_logits_q.argtypes = [vp, i64, vp, vp, vp, ctypes.c_int, ctypes.c_int, i64, i64, i64, f32, vp, i64,
                                     ctypes.c_int, vp, sz, vp, vp]
    L.orpo_head_logits_q.restype = ctypes.c_int
    L.orpo_head_logits_q_workspace_bytes.argtypes = [i64, i64, ctypes.c_int]
    L.orpo_head_logits_q_workspace_bytes.restype = sz
    L.orpo_beam_select_workspace_bytes.argtypes = [i64, ctypes.c_int, i64, ctypes.c_int]
    L.orpo_beam_select_workspace_bytes.restype = sz
    L.orpo_beam_select.argtypes = [vp, i64, ctypes.c_int, vp, vp, i32, i64, ctypes.c_int, i64, ctypes.c_int, vp, vp,
                                   vp, vp, vp, sz, vp, vp]
    L.orpo_beam_select.restype = ctypes.c_int
    L.orpo_beam_reorder.argtypes = [vp, vp, i64, vp, i64, i64, ctypes.c_int, i64, i64, i64, vp, vp]
    L.orpo_beam_reorder.restype = ctypes.c_int
    L.orpo_logits_adjust.argtypes = [vp, i64, ctypes.c_int, i64, ctypes.c_int, i64, vp, i64, i64, vp, vp, f32, f32, f32,
                                     ctypes.c_int, vp, vp, i64, i64, vp, i64, i64, vp, vp, vp]
    L.orpo_logits_adjust.restype = ctypes.c_int
    L.orpo_beam_history.argtypes = [vp, i64, i64, vp, i64, vp, i64, vp, i64, ctypes.c_int, vp, vp]
    L.orpo_beam_history.restype = ctypes.c_int
    L.orpo_pages_workspace_bytes.argtypes = [i64, i64, i64, i64]
    L.orpo_pages_workspace_bytes.restype = sz
    L.orpo_pages_advance.argtypes = [vp, i64, i64, vp, i64, i64, vp, i64, vp, vp, i64, i64, ctypes.c_int, vp, i64, vp, vp, sz,
                                     vp, vp]
    L.orpo_pages_advance.restype = ctypes.c_int
    L.orpo_pages_copy.argtypes = [vp, i64, i64, i64, i64, i64, vp, i64, vp, vp, vp]
    L.orpo_pages_copy.restype = ctypes.c_int
    L.orpo_pages_release.argtypes = [vp, i64, i64, vp, i64, vp, i64, ctypes.c_int, vp, vp]
    L.orpo_pages_release.restype = ctypes.c_int
    L.orpo_pages_compact.argtypes = [vp, i64, i64, i64, vp, i64, i64, vp, i64, vp, vp, vp, i64, vp, vp, sz, vp, vp]
    L.orpo_pages_compact.restype = ctypes.c_int
    L.orpo_profile_start.argtypes = []
    L.orpo_profile_start.restype = ctypes.c_int
    L.orpo_profile_stop.argtypes = [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int64), ctypes.c_int]
    L.orpo_profile_stop.restype = ctypes.c_int
    L.orpo_profile_kind_name.argtypes = [ctypes.c_int]
    L.orpo_profile_kind_name.restype = ctypes.c_char_p
    _fast = _load_binding(L)
    _lib = L
    return L


class _NoBinding:
    """Where csrc/binding.cpp's module is not there: answers as that does to arguments it does not take, so all go through ctypes."""

    adjust = history = advance = copy = release = compact = staticmethod(lambda *args: -1)


def _load_binding(L):
    """The module of csrc/binding.cpp, bound to the library's entry points.  It saves time and nothing else, so the library does
    without one: another PyTorch than it was built for, or none of PyTorch's headers."""
    path = _build.binding_path(_variant == "debug")
    try:
        loader = importlib.machinery.ExtensionFileLoader("orpo_binding", path)
        module = importlib.util.module_from_spec(importlib.machinery.ModuleSpec("orpo_binding", loader, origin=path))
        loader.exec_module(module)
    except ImportError as e:
        warnings.warn(f"the binding {path} cannot be loaded ({e}): calls take some microseconds more; "
                      "orpo_preference_loss_gb300.build.build() makes it", RuntimeWarning, stacklevel=3)
        return _NoBinding()
    module.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (L.orpo_logits_adjust, L.orpo_beam_history, L.orpo_pages_advance,
                                                                  L.orpo_pages_copy, L.orpo_pages_release, L.orpo_pages_compact)))
    return module


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# The current stream's handle without building a Stream object (3 us a call); torch's own code generators
# use the same two functions.  The public way where they are missing.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None and _raw_device is not None:
            return _raw_stream(_raw_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _check(code, what):
    if code != 0:
        raise OrpoError(code, what)


def _dev(t, name, dtypes, shape=None):
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != shape and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t


BF16 = (torch.bfloat16, torch.int16, torch.uint16) if hasattr(torch, "uint16") else (torch.bfloat16, torch.int16)


def orpo_status_string(code: int) -> str:
    return load().orpo_status_string(int(code)).decode()


def orpo_head_workspace_bytes(M: int, V: int, d: int) -> int:
    return int(load().orpo_head_workspace_bytes(M, V, d))


def orpo_head_fwd(h, W, targets, mask, softcap, logp, lse, workspace, status, stream=None):
    M, d = h.shape
    V = W.shape[0]
    _dev(h, "h", BF16)
    _dev(W, "W", BF16, (V, d))
    _dev(targets, "targets", (torch.int32,), (M,))
    _dev(mask, "mask", (torch.uint8, torch.bool), (M,))
    _dev(logp, "logp", (torch.float32,), (M,))
    _dev(lse, "lse", (torch.float32,), (M,))
    _dev(workspace, "workspace", (torch.uint8,))
    _dev(status, "status", (torch.int32,))
    _check(load().orpo_head_fwd(_ptr(h), _ptr(W), _ptr(targets), _ptr(mask), M, V, d, float(softcap),
                                _ptr(logp), _ptr(lse), _ptr(workspace), workspace.numel(), _ptr(status),
                                _stream(stream)), "orpo_head_fwd")


FWD_STATIC_MAX_ROWS = 65536


def orpo_head_fwd_static(h, W, targets, mask, softcap, logp, lse, status, stream=None):
    """orpo_head_fwd without a workspace argument, for callers that may not allocate
    device memory: the split partials use a fixed array inside the library."""
    M, d = h.shape
    V = W.shape[0]
    _dev(h, "h", BF16)
    _dev(W, "W", BF16, (V, d))
    _dev(targets, "targets", (torch.int32,), (M,))
    _dev(mask, "mask", (torch.uint8, torch.bool), (M,))
    _dev(logp, "logp", (torch.float32,), (M,))
    _dev(lse, "lse", (torch.float32,), (M,))
    _dev(status, "status", (torch.int32,))
    _check(load().orpo_head_fwd_static(_ptr(h), _ptr(W), _ptr(targets), _ptr(mask), M, V, d, float(softcap),
                                       _ptr(logp), _ptr(lse), _ptr(status), _stream(stream)),
           "orpo_head_fwd_static")


def orpo_loss(logp, seq_id, mask, n_pairs, lam, out, ell, g, status, stream=None):
    M = logp.shape[0]
    _dev(logp, "logp", (torch.float32,), (M,))
    _dev(seq_id, "seq_id", (torch.int32,), (M,))
    _dev(mask, "mask", (torch.uint8, torch.bool), (M,))
    _dev(out, "out", (torch.float32,), (5,))
    _dev(ell, "ell", (torch.float32,), (2 * n_pairs,))
    _dev(g, "g", (torch.float32,), (M,))
    _dev(status, "status", (torch.int32,))
    _check(load().orpo_loss(_ptr(logp), _ptr(seq_id), _ptr(mask), M, int(n_pairs), float(lam), _ptr(out),
                            _ptr(ell), _ptr(g), _ptr(status), _stream(stream)), "orpo_loss")


PREF_KINDS = {"orpo": 0, "simpo": 1, "dpo": 2, "ipo": 3, "hinge": 4, "orpo_full": 5}


def orpo_pref_loss(kind, logp, seq_id, mask, n_pairs, beta, gamma, ref_logp, out, ell, g, status, stream=None):
    """Sibling preference objective `kind` (orpo, simpo, dpo, ipo, hinge) on per-token logp."""
    M = logp.shape[0]
    k = PREF_KINDS[kind] if isinstance(kind, str) else int(kind)
    _dev(logp, "logp", (torch.float32,), (M,))
    _dev(seq_id, "seq_id", (torch.int32,), (M,))
    _dev(mask, "mask", (torch.uint8, torch.bool), (M,))
    _dev(out, "out", (torch.float32,), (5,))
    _dev(ell, "ell", (torch.float32,), (2 * n_pairs,))
    _dev(g, "g", (torch.float32,), (M,))
    _dev(status, "status", (torch.int32,))
    if ref_logp is not None:
        _dev(ref_logp, "ref_logp", (torch.float32,), (2 * n_pairs,))
    _check(load().orpo_pref_loss(k, _ptr(logp), _ptr(seq_id), _ptr(mask), M, int(n_pairs), float(beta), float(gamma),
                                 _ptr(ref_logp), _ptr(out), _ptr(ell), _ptr(g), _ptr(status), _stream(stream)),
           "orpo_pref_loss")


def orpo_head_bwd(h, W, targets, mask, lse, g, softcap, dh, dW, accumulate_dW, workspace, status,
                  stream=None):
    M, d = h.shape
    V = W.shape[0]
    _dev(h, "h", BF16)
    _dev(W, "W", BF16, (V, d))
    _dev(targets, "targets", (torch.int32,), (M,))
    _dev(mask, "mask", (torch.uint8, torch.bool), (M,))
    _dev(lse, "lse", (torch.float32,), (M,))
    _dev(g, "g", (torch.float32,), (M,))
    _dev(dh, "dh", (torch.float32,), (M, d))
    if dW is not None:
        _dev(dW, "dW", (torch.float32,), (V, d))
    _dev(workspace, "workspace", (torch.uint8,))
    _dev(status, "status", (torch.int32,))
    _check(load().orpo_head_bwd(_ptr(h), _ptr(W), _ptr(targets), _ptr(mask), _ptr(lse), _ptr(g), M, V, d,
                                float(softcap), _ptr(dh), _ptr(dW), 1 if accumulate_dW else 0, _ptr(workspace),
                                workspace.numel(), _ptr(status), _stream(stream)), "orpo_head_bwd")


def orpo_head_block_max_elems(M: int, V: int) -> int:
    return int(load().orpo_head_block_max_elems(M, V))


def block_max_shape(M: int, V: int):
    """[ceil(M / 32), ceil(V / 256)]: the block-max array of the backward skips."""
    return (-(-M // 32), -(-V // 256))


def orpo_head_fwd_bmax(h, W, targets, mask, softcap, logp, lse, block_max, workspace, status, stream=None):
    """orpo_head_fwd that also writes the block maxima the backward's block skip reads."""
    M, d = h.shape
    V = W.shape[0]
    _dev(h, "h", BF16)
    _dev(W, "W", BF16, (V, d))
    _dev(targets, "targets", (torch.int32,), (M,))
    _dev(mask, "mask", (torch.uint8, torch.bool), (M,))
    _dev(logp, "logp", (torch.float32,), (M,))
    _dev(lse, "lse", (torch.float32,), (M,))
    _dev(block_max, "block_max", (torch.float32,), block_max_shape(M, V))
    _dev(workspace, "workspace", (torch.uint8,))
    _dev(status, "status", (torch.int32,))
    _check(load().orpo_head_fwd_bmax(_ptr(h), _ptr(W), _ptr(targets), _ptr(mask), M, V, d, float(softcap),
                                     _ptr(logp), _ptr(lse), _ptr(block_max), _ptr(workspace), workspace.numel(),
                                     _ptr(status), _stream(stream)), "orpo_head_fwd_bmax")


def orpo_head_bwd_skip(h, W, targets, mask, lse, g, block_max, eps, softcap, dh, dW, accumulate_dW, workspace,
                       status, stream=None):
    """orpo_head_bwd with the backward skips: the coefficient filter at eps, and the block skip when
    block_max (from orpo_head_fwd_bmax) is given (None: filter alone)."""
    M, d = h.shape
    V = W.shape[0]
    _dev(h, "h", BF16)
    _dev(W, "W", BF16, (V, d))
    _dev(targets, "targets", (torch.int32,), (M,))
    _dev(mask, "mask", (torch.uint8, torch.bool), (M,))
    _dev(lse, "lse", (torch.float32,), (M,))
    _dev(g, "g", (torch.float32,), (M,))
    if block_max is not None:
        _dev(block_max, "block_max", (torch.float32,), block_max_shape(M, V))
    _dev(dh, "dh", (torch.float32,), (M, d))
    if dW is not None:
        _dev(dW, "dW", (torch.float32,), (V, d))
    _dev(workspace, "workspace", (torch.uint8,))
    _dev(status, "status", (torch.int32,))
    _check(load().orpo_head_bwd_skip(_ptr(h), _ptr(W), _ptr(targets), _ptr(mask), _ptr(lse), _ptr(g),
                                     _ptr(block_max), float(eps), M, V, d, float(softcap), _ptr(dh), _ptr(dW),
                                     1 if accumulate_dW else 0, _ptr(workspace), workspace.numel(), _ptr(status),
                                     _stream(stream)), "orpo_head_bwd_skip")


def orpo_head_q_workspace_bytes(M: int, V: int, d: int) -> int:
    return int(load().orpo_head_q_workspace_bytes(M, V, d))


def _quant_args(wq, scales, biases, V, d, bits, group):
    _dev(wq, "wq", (torch.uint8,), (V, d * bits // 8))
    _dev(scales, "scales", BF16, (V, d // group))
    _dev(biases, "biases", BF16, (V, d // group))


def orpo_head_fwd_q(h, wq, scales, biases, bits, group, targets, mask, softcap, logp, lse, workspace, status,
                    stream=None):
    """orpo_head_fwd on an affine group-quantised head (wq, scales, biases)."""
    M, d = h.shape
    V = wq.shape[0]
    _dev(h, "h", BF16)
    _quant_args(wq, scales, biases, V, d, bits, group)
    _dev(targets, "targets", (torch.int32,), (M,))
    _dev(mask, "mask", (torch.uint8, torch.bool), (M,))
    _dev(logp, "logp", (torch.float32,), (M,))
    _dev(lse, "lse", (torch.float32,), (M,))
    _dev(workspace, "workspace", (torch.uint8,))
    _check(load().orpo_head_fwd_q(_ptr(h), _ptr(wq), _ptr(scales), _ptr(biases), int(bits), int(group), _ptr(targets),
                                  _ptr(mask), M, V, d, float(softcap), _ptr(logp), _ptr(lse), _ptr(workspace),
                                  workspace.numel(), _ptr(status), _stream(stream)), "orpo_head_fwd_q")


def orpo_head_bwd_q(h, wq, scales, biases, bits, group, targets, mask, lse, g, softcap, dh, dW, accumulate_dW,
                    workspace, status, stream=None):
    """orpo_head_bwd on an affine group-quantised head; dW (optional) is w.r.t. the dequantised weight."""
    M, d = h.shape
    V = wq.shape[0]
    _dev(h, "h", BF16)
    _quant_args(wq, scales, biases, V, d, bits, group)
    _dev(lse, "lse", (torch.float32,), (M,))
    _dev(g, "g", (torch.float32,), (M,))
    _dev(dh, "dh", (torch.float32,), (M, d))
    if dW is not None:
        _dev(dW, "dW", (torch.float32,), (V, d))
    _check(load().orpo_head_bwd_q(_ptr(h), _ptr(wq), _ptr(scales), _ptr(biases), int(bits), int(group), _ptr(targets),
                                  _ptr(mask), _ptr(lse), _ptr(g), M, V, d, float(softcap), _ptr(dh), _ptr(dW),
                                  1 if accumulate_dW else 0, _ptr(workspace), workspace.numel(), _ptr(status),
                                  _stream(stream)), "orpo_head_bwd_q")


def orpo_head_fwd_q_bmax(h, wq, scales, biases, bits, group, targets, mask, softcap, logp, lse, block_max,
                         workspace, status, stream=None):
    """orpo_head_fwd_q that also writes the block maxima of the backward skips."""
    M, d = h.shape
    V = wq.shape[0]
    _dev(h, "h", BF16)
    _quant_args(wq, scales, biases, V, d, bits, group)
    _dev(targets, "targets", (torch.int32,), (M,))
    _dev(mask, "mask", (torch.uint8, torch.bool), (M,))
    _dev(logp, "logp", (torch.float32,), (M,))
    _dev(lse, "lse", (torch.float32,), (M,))
    _dev(block_max, "block_max", (torch.float32,), block_max_shape(M, V))
    _dev(workspace, "workspace", (torch.uint8,))
    _check(load().orpo_head_fwd_q_bmax(_ptr(h), _ptr(wq), _ptr(scales), _ptr(biases), int(bits), int(group),
                                       _ptr(targets), _ptr(mask), M, V, d, float(softcap), _ptr(logp), _ptr(lse),
                                       _ptr(block_max), _ptr(workspace), workspace.numel(), _ptr(status),
                                       _stream(stream)), "orpo_head_fwd_q_bmax")


def orpo_head_bwd_q_skip(h, wq, scales, biases, bits, group, targets, mask, lse, g, block_max, eps, softcap, dh, dW,
                         accumulate_dW, workspace, status, stream=None):
    """orpo_head_bwd_q with the backward skips (block_max may be None: filter alone)."""
    M, d = h.shape
    V = wq.shape[0]
    _dev(h, "h", BF16)
    _quant_args(wq, scales, biases, V, d, bits, group)
    _dev(lse, "lse", (torch.float32,), (M,))
    _dev(g, "g", (torch.float32,), (M,))
    if block_max is not None:
        _dev(block_max, "block_max", (torch.float32,), block_max_shape(M, V))
    _dev(dh, "dh", (torch.float32,), (M, d))
    if dW is not None:
        _dev(dW, "dW", (torch.float32,), (V, d))
    _check(load().orpo_head_bwd_q_skip(_ptr(h), _ptr(wq), _ptr(scales), _ptr(biases), int(bits), int(group),
                                       _ptr(targets), _ptr(mask), _ptr(lse), _ptr(g), _ptr(block_max), float(eps), M, V,
                                       d, float(softcap), _ptr(dh), _ptr(dW), 1 if accumulate_dW else 0,
                                       _ptr(workspace), workspace.numel(), _ptr(status), _stream(stream)),
           "orpo_head_bwd_q_skip")


def _rows(t, name, dtypes, cols=None, rows=None):
    """A 2-D CUDA tensor whose rows are contiguous; returns its row pitch in elements."""
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    shape = t.shape
    if len(shape) != 2 or (cols is not None and shape[1] != cols) or (rows is not None and shape[0] != rows):
        raise ValueError(f"{name} has shape {tuple(shape)}, expected "
                         f"({'rows' if rows is None else rows}, {'columns' if cols is None else cols})")
    r, c = shape
    pitch, step = t.stride()
    if r <= 1:
        pitch = c
    if (step != 1 and c > 1) or pitch < c:
        raise ValueError(f"{name} must have contiguous rows that do not overlap")
    return pitch


LOGITS = (torch.float32, torch.bfloat16)
F32, I32, U8, FLAGS = (torch.float32,), (torch.int32,), (torch.uint8,), (torch.uint8, torch.bool)
MASKS = (torch.int32, torch.uint32) if hasattr(torch, "uint32") else (torch.int32,)


def orpo_head_logits_q_workspace_bytes(M: int, d: int, bits: int) -> int:
    return int(load().orpo_head_logits_q_workspace_bytes(M, d, bits))


def orpo_head_logits_q(h, wq, scales, biases, bits, group, softcap, logits, status, stream=None, workspace=None):
    """Logits [M, V] (fp32 or bf16) of the rows of h [M, d] under the affine group-quantised head.

    h and logits may have any row pitch, e.g. hidden[:, -1] of [M, T, d] hidden states.  workspace: uint8,
    orpo_head_logits_q_workspace_bytes(M, d, bits) of them; None takes what is needed from PyTorch's
    allocator, on the call's stream."""
    M, d = h.shape
    V = wq.shape[0]
    if workspace is not None:
        _dev(workspace, "workspace", U8)
    elif M > 16 or d > 2048:
        need = (_lib or load()).orpo_head_logits_q_workspace_bytes(M, d, bits)
        if need:
            # from the pool of the stream that the kernels run on: a block of another stream's may have been freed
            # with work on it still to come there
            with torch.cuda.stream(stream):
                workspace = torch.empty(need, dtype=torch.uint8, device=h.device)
    # A decode step is a few microseconds of GPU work, so the usual, right arguments pass one plain test;
    # whatever fails it is looked at in full for its message.
    hp, hs = h.stride()
    if M <= 1:
        hp = d  # where a next row would start does not matter
    lp, ls = logits.stride()
    if not (h.is_cuda and h.dtype in BF16 and hs == 1 and hp >= d and wq.is_cuda and wq.dtype is torch.uint8
            and wq.is_contiguous() and wq.shape == (V, d * bits // 8) and scales.is_cuda and scales.dtype in BF16
            and scales.is_contiguous() and scales.shape == (V, d // group) and biases.is_cuda and biases.dtype in BF16
            and biases.is_contiguous() and biases.shape == (V, d // group) and logits.is_cuda
            and logits.dtype in LOGITS and logits.shape == (M, V) and ls == 1 and lp >= V and status.is_cuda
            and status.dtype is torch.int32):
        hp = _rows(h, "h", BF16)
        _quant_args(wq, scales, biases, V, d, bits, group)
        lp = _rows(logits, "logits", LOGITS, cols=V, rows=M)
        _dev(status, "status", I32)
    code = (_lib or load()).orpo_head_logits_q(
        h.data_ptr(), hp, wq.data_ptr(), scales.data_ptr(), biases.data_ptr(), bits, group, M, V, d, softcap,
        logits.data_ptr(), lp, logits.dtype is torch.bfloat16, None if workspace is None else workspace.data_ptr(),
        0 if workspace is None else workspace.numel(), status.data_ptr(), _stream(stream))
    if code:
        raise OrpoError(code, "orpo_head_logits_q")


def orpo_beam_select_workspace_bytes(batch: int, beams: int, V: int, n: int) -> int:
    return int(load().orpo_beam_select_workspace_bytes(batch, beams, V, n))


def orpo_beam_select(logits, score, finished, eos, beams, out_score, out_parent, out_token, out_finished, workspace,
                     status, stream=None):
    """The n best continuations (out_* are [batch, n]) over beams x vocabulary of logits [batch * beams, V].

    finished and out_finished may be None; eos is -1 when no token ends a response."""
    rows, V = logits.shape
    batch, n = out = out_score.shape
    pitch, step = logits.stride()
    if not (rows == batch * beams and logits.is_cuda and logits.dtype in LOGITS and step == 1 and pitch >= V
            and score.is_cuda and score.dtype is torch.float32 and score.is_contiguous() and score.numel() == rows
            and (finished is None or (finished.is_cuda and finished.dtype in FLAGS and finished.is_contiguous()
                                      and finished.numel() == rows))
            and out_score.is_cuda and out_score.dtype is torch.float32 and out_score.is_contiguous()
            and out_parent.is_cuda and out_parent.dtype is torch.int32 and out_parent.is_contiguous()
            and out_parent.shape == out and out_token.is_cuda and out_token.dtype is torch.int32
            and out_token.is_contiguous() and out_token.shape == out
            and (out_finished is None or (out_finished.is_cuda and out_finished.dtype in FLAGS
                                          and out_finished.is_contiguous() and out_finished.shape == out))
            and workspace.is_cuda and workspace.dtype is torch.uint8 and workspace.is_contiguous() and status.is_cuda
            and status.dtype is torch.int32):
        rows = batch * beams
        pitch = _rows(logits, "logits", LOGITS, rows=rows)
        _dev(score, "score", F32)
        if score.numel() != rows:
            raise ValueError(f"score has {score.numel()} elements, expected batch * beams = {rows}")
        if finished is not None:
            _dev(finished, "finished", FLAGS)
            if finished.numel() != rows:
                raise ValueError(f"finished has {finished.numel()} elements, expected batch * beams = {rows}")
        _dev(out_score, "out_score", F32)
        _dev(out_parent, "out_parent", I32, (batch, n))
        _dev(out_token, "out_token", I32, (batch, n))
        if out_finished is not None:
            _dev(out_finished, "out_finished", FLAGS, (batch, n))
        _dev(workspace, "workspace", U8)
        _dev(status, "status", I32)
    code = (_lib or load()).orpo_beam_select(
        logits.data_ptr(), pitch, logits.dtype is torch.bfloat16, score.data_ptr(),
        None if finished is None else finished.data_ptr(), eos, batch, beams, V, n, out_score.data_ptr(),
        out_parent.data_ptr(), out_token.data_ptr(), None if out_finished is None else out_finished.data_ptr(),
        workspace.data_ptr(), workspace.numel(), status.data_ptr(), _stream(stream))
    if code:
        raise OrpoError(code, "orpo_beam_select")


def orpo_beam_reorder(state, parent, length, status, stream=None):
    """state [outer, batch * beams, rows, capacity, unit] (any dtype) follows parent [batch, beams] in place.

    Only positions t < length[b] (int32 [batch]; None: all) of the capacity dimension move."""
    batch, beams = parent.shape
    pitch, step = parent.stride()
    if not (state.is_cuda and state.is_contiguous() and state.dim() == 5 and state.shape[1] == batch * beams
            and parent.is_cuda and parent.dtype is torch.int32 and step == 1 and pitch >= beams
            and (length is None or (length.is_cuda and length.dtype is torch.int32 and length.is_contiguous()
                                    and length.shape == (batch,)))
            and status.is_cuda and status.dtype is torch.int32):
        if not state.is_cuda or not state.is_contiguous() or state.dim() != 5:
            raise ValueError("state must be a contiguous CUDA tensor [outer, batch * beams, rows, capacity, unit]")
        pitch = _rows(parent, "parent", I32)
        if state.shape[1] != batch * beams:
            raise ValueError(f"state has {state.shape[1]} beams, expected batch * beams = {batch * beams}")
        if length is not None:
            _dev(length, "length", I32, (batch,))
        _dev(status, "status", I32)
    outer, _, rows, capacity, unit = state.shape
    code = (_lib or load()).orpo_beam_reorder(
        state.data_ptr(), parent.data_ptr(), pitch, None if length is None else length.data_ptr(), outer, batch,
        beams, rows, capacity, unit * state.element_size(), status.data_ptr(), _stream(stream))
    if code:
        raise OrpoError(code, "orpo_beam_reorder")


def _now():
    """The current device's number."""
    return torch.cuda.current_device() if _raw_device is None else _raw_device()


def _bound():
    """The module of csrc/binding.cpp, once the library is loaded."""
    load()
    return _fast


def _here(first, *others):
    """The tensors (None: not given) are on the device that is current, where the call's kernels run."""
    at = first.get_device()
    if at < 0:
        raise ValueError("the tensors must be CUDA tensors")
    now = _now()
    if at != now:
        raise ValueError(f"the tensors are on cuda:{at}, but the current device is cuda:{now}")
    for t in others:
        if t is not None and t.get_device() != at:
            raise ValueError(f"the tensors are on different devices: {first.device} and {t.device}")


def _fits(bits, **numbers):
    """ctypes cuts a whole number to its C type without a word: 2^32 + 2 would pass for 2."""
    for name, n in numbers.items():
        if isinstance(n, int) and not -(1 << bits - 1) <= n < 1 << bits - 1:
            raise ValueError(f"{name} = {n} is out of range")


# Each of the calls below goes through csrc/binding.cpp, which looks at the tensors in a fraction of the time.  Where that
# finds one that is not of the usual kind (-1), the arguments are looked at here one by one, for the message.


def orpo_logits_adjust(logits, beams, status, history=None, length=None, prompt=None, repetition=1.0, presence=0.0, frequency=0.0,
                       no_repeat=0, bias_token=None, bias_value=None, masks=None, mask_row=None, stream=None):
    """Penalties for repeated tokens, biases and grammar masks, in place on logits [batch * beams, V] (fp32 or bf16).

    history: int32 [batch * beams, capacity], of which the first length[b] (int32 [batch]) are tokens of the row, the first
    prompt[b] of those (None: 0) the prompt's.  bias_token, bias_value: int32, fp32 [batch, n], or [n] for every entry.  masks:
    int32 or uint32 [n_masks, ceil(V / 32)], bit set = allowed; mask_row: int32 [batch * beams], -1 for a row without a mask."""
    code = (_fast or _bound()).adjust(stream, logits, beams, status, history, length, prompt, repetition, presence, frequency, no_repeat,
                                      bias_token, bias_value, masks, mask_row)
    if code < 0:
        code = _adjust(logits, beams, status, history, length, prompt, repetition, presence, frequency, no_repeat, bias_token,
                       bias_value, masks, mask_row, stream)
    if code:
        raise OrpoError(code, "orpo_logits_adjust")


def _adjust(logits, beams, status, history, length, prompt, repetition, presence, frequency, no_repeat, bias_token, bias_value,
            masks, mask_row, stream):
    rows, V = logits.shape
    if beams < 1 or rows % beams:
        raise ValueError(f"logits has {rows} rows, expected a multiple of beams = {beams}")
    batch = rows // beams
    _fits(32, beams=beams, no_repeat=no_repeat)
    _here(logits, status, history, length, prompt, bias_token, bias_value, masks, mask_row)
    pitch = _rows(logits, "logits", LOGITS)
    _dev(status, "status", I32)
    ld_history = capacity = 0
    if history is not None:
        ld_history, capacity = _rows(history, "history", I32, rows=rows), history.shape[1]
        _dev(length, "length", I32, (batch,))
        if prompt is not None:
            _dev(prompt, "prompt", I32, (batch,))
    ld_bias = n_bias = 0
    if bias_token is not None or bias_value is not None:
        if bias_token is None or bias_value is None or bias_token.shape != bias_value.shape:
            raise ValueError("bias_token and bias_value must be given together, in one shape")
        if bias_token.dim() == 1:
            _dev(bias_token, "bias_token", I32)
            _dev(bias_value, "bias_value", F32)
        else:
            ld_bias = _rows(bias_token, "bias_token", I32, rows=batch)
            if _rows(bias_value, "bias_value", F32) != ld_bias:
                raise ValueError("bias_token and bias_value must have the same row pitch")
        n_bias = bias_token.shape[-1]
    ld_masks = n_masks = 0
    if masks is not None or mask_row is not None:
        ld_masks, n_masks = _rows(masks, "masks", MASKS, cols=-(-V // 32)), masks.shape[0]
        _dev(mask_row, "mask_row", I32, (rows,))
    return load().orpo_logits_adjust(
        _ptr(logits), pitch, logits.dtype is torch.bfloat16, batch, beams, V, _ptr(history), ld_history, capacity, _ptr(length),
        _ptr(prompt), repetition, presence, frequency, no_repeat, _ptr(bias_token), _ptr(bias_value), ld_bias, n_bias, _ptr(masks),
        ld_masks, n_masks, _ptr(mask_row), _ptr(status), _stream(stream))


def orpo_beam_history(history, parent, token, length, status, stream=None):
    """Token histories [batch * beams, capacity] (int32) follow parent [batch, beams] in place, up to length[b], where
    token [batch, beams] is then put.  length is not changed."""
    code = (_fast or _bound()).history(stream, history, parent, token, length, status)
    if code < 0:
        batch, beams = parent.shape
        _here(history, parent, token, length, status)
        ld = _rows(history, "history", I32, rows=batch * beams)
        ld_parent = _rows(parent, "parent", I32)
        ld_token = _rows(token, "token", I32, cols=beams, rows=batch)
        _dev(length, "length", I32, (batch,))
        _dev(status, "status", I32)
        code = load().orpo_beam_history(_ptr(history), ld, history.shape[1], _ptr(parent), ld_parent, _ptr(token), ld_token,
                                        _ptr(length), batch, beams, _ptr(status), _stream(stream))
    if code:
        raise OrpoError(code, "orpo_beam_history")


def orpo_pages_workspace_bytes(table_rows: int, pages: int, page: int, most: int = 1) -> int:
    _fits(64, table_rows=table_rows, pages=pages, page=page, most=most)
    return int(load().orpo_pages_workspace_bytes(table_rows, pages, page, most))


def _moves(moves, n_moves, workspace, status):
    _dev(moves, "moves", I32)
    if moves.dim() != 2 or moves.shape[1] != 3:
        raise ValueError(f"moves has shape {tuple(moves.shape)}, expected (max_moves, 3)")
    _dev(n_moves, "n_moves", I32, (1,))
    if workspace is not None:
        _dev(workspace, "workspace", U8)
    _dev(status, "status", I32)


def orpo_pages_advance(table, refs, page, parent, length, more, most, moves, n_moves, workspace, status, stream=None):
    """Page tables [batch * beams, columns] follow parent [batch, beams] (None: they stay), and positions length[b] ..
    length[b] + more[b] - 1 (more None: `most` of them) of each row become writable.

    Pages are taken and let go of in refs (int32 [pages]); pages to be copied are listed in moves (int32 [max_moves, 3], n_moves
    int32 [1]) for orpo_pages_copy.  workspace: uint8, orpo_pages_workspace_bytes(batch * beams, pages, page, most)."""
    code = (_fast or _bound()).advance(stream, table, refs, page, parent, length, more, most, moves, n_moves, workspace, status)
    if code < 0:
        rows, columns = table.shape
        batch = length.shape[0]
        beams = rows // batch if batch else 1
        if rows != batch * beams:
            raise ValueError(f"table has {rows} rows, expected a multiple of the {batch} lengths")
        _fits(64, page=page, most=most)
        _here(table, refs, parent, length, more, moves, n_moves, workspace, status)
        ld = _rows(table, "table", I32)
        _dev(refs, "refs", I32, (refs.numel(),))
        ld_parent = 0 if parent is None else _rows(parent, "parent", I32, cols=beams, rows=batch)
        _dev(length, "length", I32, (batch,))
        if more is not None:
            _dev(more, "more", I32, (batch,))
        _moves(moves, n_moves, workspace, status)
        code = load().orpo_pages_advance(
            _ptr(table), ld, columns, _ptr(refs), refs.numel(), page, _ptr(parent), ld_parent, _ptr(length), _ptr(more), most, batch,
            beams, _ptr(moves), moves.shape[0], _ptr(n_moves), _ptr(workspace), workspace.numel(), _ptr(status), _stream(stream))
    if code:
        raise OrpoError(code, "orpo_pages_advance")


def orpo_pages_copy(pool, moves, n_moves, status, stream=None):
    """Carries out the copies of moves in pool [outer, pages, rows, page, unit] (any dtype)."""
    code = (_fast or _bound()).copy(stream, pool, moves, n_moves, status)
    if code < 0:
        _here(pool, moves, n_moves, status)
        if not pool.is_contiguous() or pool.dim() != 5:
            raise ValueError("pool must be a contiguous CUDA tensor [outer, pages, rows, page, unit]")
        _moves(moves, n_moves, None, status)
        outer, pages, rows, page, unit = pool.shape
        code = load().orpo_pages_copy(_ptr(pool), outer, pages, rows, page, unit * pool.element_size(), _ptr(moves), moves.shape[0],
                                      _ptr(n_moves), _ptr(status), _stream(stream))
    if code:
        raise OrpoError(code, "orpo_pages_copy")


def orpo_pages_release(table, refs, ended, status, stream=None):
    """The rows of entries with ended[b] != 0 (uint8 or bool [batch]; None: all rows) let go of their pages."""
    code = (_fast or _bound()).release(stream, table, refs, ended, status)
    if code < 0:
        rows, columns = table.shape
        batch = rows if ended is None else ended.shape[0]
        beams = rows // batch if batch else 1
        if rows != batch * beams:
            raise ValueError(f"table has {rows} rows, expected a multiple of the {batch} entries of ended")
        _here(table, refs, ended, status)
        ld = _rows(table, "table", I32)
        _dev(refs, "refs", I32, (refs.numel(),))
        if ended is not None:
            _dev(ended, "ended", FLAGS, (batch,))
        _dev(status, "status", I32)
        code = load().orpo_pages_release(_ptr(table), ld, columns, _ptr(refs), refs.numel(), _ptr(ended), batch, beams, _ptr(status),
                                         _stream(stream))
    if code:
        raise OrpoError(code, "orpo_pages_release")


def orpo_pages_compact(table, refs, page, new_table, new_refs, live, moves, n_moves, workspace, status, stream=None):
    """Numbers the pages in use 0 .. live[0] - 1: those at live[0] or above take the free numbers below, in order.

    new_table and new_refs may be table and refs themselves; moves (at least pages / 2 of them) are for orpo_pages_copy."""
    code = (_fast or _bound()).compact(stream, table, refs, page, new_table, new_refs, live, moves, n_moves, workspace, status)
    if code < 0:
        rows, columns = table.shape
        _fits(64, page=page)
        _here(table, refs, new_table, new_refs, live, moves, n_moves, workspace, status)
        ld = _rows(table, "table", I32)
        ld_new = _rows(new_table, "new_table", I32, cols=columns, rows=rows)
        _dev(refs, "refs", I32, (refs.numel(),))
        _dev(new_refs, "new_refs", I32, (refs.numel(),))
        _dev(live, "live", I32, (1,))
        _moves(moves, n_moves, workspace, status)
        code = load().orpo_pages_compact(
            _ptr(table), ld, columns, rows, _ptr(refs), refs.numel(), page, _ptr(new_table), ld_new, _ptr(new_refs), _ptr(live),
            _ptr(moves), moves.shape[0], _ptr(n_moves), _ptr(workspace), workspace.numel(), _ptr(status), _stream(stream))
    if code:
        raise OrpoError(code, "orpo_pages_compact")


def orpo_debug_gemm(A, B, C, M, N, K, a_mn_major, b_mn_major, status, stream=None):
    _dev(A, "A", BF16)
    _dev(B, "B", BF16)
    _dev(C, "C", (torch.float32,), (M, N))
    _check(load().orpo_debug_gemm(_ptr(A), _ptr(B), _ptr(C), M, N, K, int(a_mn_major), int(b_mn_major),
                                  _ptr(status), _stream(stream)), "orpo_debug_gemm")


def orpo_debug_wait_timeout(status, limit_ns, stream=None):
    _dev(status, "status", (torch.int32,))
    _check(load().orpo_debug_wait_timeout(_ptr(status), int(limit_ns), _stream(stream)), "orpo_debug_wait_timeout")


PROFILE_KINDS = 15


def orpo_profile_start():
    _check(load().orpo_profile_start(), "orpo_profile_start")


def orpo_profile_stop():
    """Per kernel kind: {name: (total_ms, launches)} for the launches since orpo_profile_start()."""
    ms = (ctypes.c_double * PROFILE_KINDS)()
    cnt = (ctypes.c_int64 * PROFILE_KINDS)()
    _check(load().orpo_profile_stop(ms, cnt, PROFILE_KINDS), "orpo_profile_stop")
    return {load().orpo_profile_kind_name(k).decode(): (ms[k], int(cnt[k])) for k in range(PROFILE_KINDS)}


class OrpoHead:
    """Owns the per-size device buffers (workspace, outputs) and runs one head step.

    All tensors come from PyTorch's allocator; the step itself is the three C
    entry points in order on the current stream.
    """

    def __init__(self, M: int, V: int, d: int, n_pairs: int, device="cuda", skip_eps: float = 0.0):
        """skip_eps > 0 turns on the backward skips (coefficient filter and block skip) at that eps."""
        self.M, self.V, self.d, self.P = M, V, d, n_pairs
        self.skip_eps = float(skip_eps)
        dev = torch.device(device)
        self.block_max = (torch.empty(block_max_shape(M, V), dtype=torch.float32, device=dev)
                          if self.skip_eps > 0 else None)
        self.workspace = torch.empty(orpo_head_workspace_bytes(M, V, d), dtype=torch.uint8, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.logp = torch.empty(M, dtype=torch.float32, device=dev)
        self.lse = torch.empty(M, dtype=torch.float32, device=dev)
        self.out = torch.empty(5, dtype=torch.float32, device=dev)
        self.ell = torch.empty(2 * n_pairs, dtype=torch.float32, device=dev)
        self.g = torch.empty(M, dtype=torch.float32, device=dev)
        self.dh = torch.empty((M, d), dtype=torch.float32, device=dev)
        self.dW = torch.empty((V, d), dtype=torch.float32, device=dev)

    def step(self, h, W, targets, mask, seq_id, softcap, lam, accumulate_dW=False, stream=None):
        if self.skip_eps > 0:
            orpo_head_fwd_bmax(h, W, targets, mask, softcap, self.logp, self.lse, self.block_max, self.workspace,
                               self.status, stream)
        else:
            orpo_head_fwd(h, W, targets, mask, softcap, self.logp, self.lse, self.workspace, self.status, stream)
        orpo_loss(self.logp, seq_id, mask, self.P, lam, self.out, self.ell, self.g, self.status, stream)
        if self.skip_eps > 0:
            orpo_head_bwd_skip(h, W, targets, mask, self.lse, self.g, self.block_max, self.skip_eps, softcap,
                               self.dh, self.dW, accumulate_dW, self.workspace, self.status, stream)
        else:
            orpo_head_bwd(h, W, targets, mask, self.lse, self.g, softcap, self.dh, self.dW, accumulate_dW,
                          self.workspace, self.status, stream)
        return self.out

    def capture(self, h, W, targets, mask, seq_id, softcap, lam, accumulate_dW=False):
        """Record one step on these tensors into a CUDA graph and return it.

        Each ``graph.replay()`` reruns the whole step (forward, loss, backward: 5 or more launches)
        on whatever the given tensors hold at that moment, for the price of one launch; this matters
        for small batches, whose step is a few launches of microseconds.  The step runs once eagerly
        first, on a side stream, so that the library's one-time device set-up happens outside the
        capture.  Fill the same input tensors before each replay; the outputs land in this head's
        buffers as with step()."""
        args = (h, W, targets, mask, seq_id, softcap, lam, accumulate_dW)
        side = torch.cuda.Stream(self.workspace.device)
        side.wait_stream(torch.cuda.current_stream(self.workspace.device))
        with torch.cuda.stream(side):
            self.step(*args)
        torch.cuda.current_stream(self.workspace.device).wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.step(*args)
        return graph


class PagedStates:
    """Owns the page table of beam states kept in shared pages, and runs the calls of orpo_pages.h on it.

    The pools themselves, [outer, pages, rows, page, unit] of any dtype and any number of them, are the caller's: position
    t of beam r is position t % page of page table[r, t // page] in every pool.  table [batch * beams, columns], refs [pages],
    moves and status stay on the device; nothing waits on the host.  The constructor fills them on the current stream.
    A call that raises for its arguments has changed nothing.  most: the largest number of positions that advance or admit is
    asked for at once."""

    def __init__(self, batch: int, beams: int, columns: int, pages: int, page: int, most: int = 1, status=None, device="cuda"):
        self.batch, self.beams, self.columns, self.pages, self.page, self.most = batch, beams, columns, pages, page, most
        dev = torch.device(device)
        ws = orpo_pages_workspace_bytes(batch * beams, pages, page, most)
        if ws == 0:
            raise ValueError(f"batch {batch}, beams {beams}, pages {pages}, page {page}, most {most} are out of orpo_pages.h's range")
        self.workspace = torch.empty(ws, dtype=torch.uint8, device=dev)
        self.table = torch.full((batch * beams, columns), -1, dtype=torch.int32, device=dev)
        self.refs = torch.zeros(pages, dtype=torch.int32, device=dev)
        self.moves = torch.empty((max(batch * beams, pages // 2), 3), dtype=torch.int32, device=dev)
        self.n_moves = torch.zeros(1, dtype=torch.int32, device=dev)
        self.live = torch.zeros(1, dtype=torch.int32, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev) if status is None else status

    def _check_pools(self, pools):
        """The pools as a tuple.  Raises where one does not fit the table: a plan changes the table in place, so by the time a
        copy is refused it would be too late."""
        pools, at = tuple(pools), self.table.get_device()
        for pool in pools:
            shape = pool.shape
            if (len(shape) != 5 or shape[1] != self.pages or shape[3] != self.page or not pool.is_contiguous() or pool.get_device() != at
                    or self.page * shape[4] * pool.element_size() >= 1 << 31):
                raise ValueError(f"a pool has shape {tuple(shape)} of {pool.dtype} on {pool.device}, expected a contiguous tensor [outer, {self.pages}, "
                                 f"rows, {self.page}, unit] on {self.table.device} with less than 2^31 bytes per page and row")
        return pools

    def _copy(self, pools, stream):
        for pool in pools:
            orpo_pages_copy(pool, self.moves, self.n_moves, self.status, stream)

    def advance(self, length, parent=None, more=None, most=1, pools=(), stream=None):
        """The beams' tables follow parent [batch, beams] up to length[b], and positions length[b] .. length[b] + more[b] - 1
        (more None: `most` of them) of every beam can be written in all pools."""
        self._advance(length, parent, more, most, self._check_pools(pools), stream)

    def _advance(self, length, parent, more, most, pools, stream):
        orpo_pages_advance(self.table, self.refs, self.page, parent, length, more, most, self.moves, self.n_moves,
                           self.workspace, self.status, stream)
        self._copy(pools, stream)

    def admit(self, length, more, most, pools=(), stream=None):
        """As advance without parents, for beam 0 of each entry alone: a prompt, which the other beams take with their
        first advance (all parents 0)."""
        pools = self._check_pools(pools)
        orpo_pages_advance(self.table[::self.beams], self.refs, self.page, None, length, more, most, self.moves, self.n_moves,
                           self.workspace, self.status, stream)
        self._copy(pools, stream)

    def release(self, ended=None, stream=None):
        """Entries with ended[b] != 0 (None: all) let go of their pages."""
        if ended is not None and ended.shape != (self.batch,):
            raise ValueError(f"ended has shape {tuple(ended.shape)}, expected ({self.batch},)")
        orpo_pages_release(self.table, self.refs, ended, self.status, stream)

    def compact(self, pools=(), stream=None):
        """Pages in use move to the lowest numbers, 0 .. live[0] - 1, in all pools."""
        pools = self._check_pools(pools)
        orpo_pages_compact(self.table, self.refs, self.page, self.table, self.refs, self.live, self.moves, self.n_moves,
                           self.workspace, self.status, stream)
        self._copy(pools, stream)


class BeamDecoder:
    """Owns the buffers of beam search on the quantised head and runs one decode step.

    A step is the C entry points of orpo_decode.h in order on the current stream: logits of the beams' last hidden
    rows, their penalties, biases and masks where any are given, selection of each batch entry's `beams` best
    continuations, and the states and histories following their parents.  score, finished, parent and token stay on the
    device; nothing waits on the host, so a step can be recorded in a CUDA graph.  The constructor and reset fill the buffers
    on the current stream: a step on another stream has to be ordered behind them.

    repetition, presence, frequency, no_repeat: orpo_logits_adjust's; any of them makes step need a history."""

    def __init__(self, batch: int, beams: int, V: int, d: int, bits: int = 4, group: int = 64, softcap: float = 0.0,
                 eos: int = -1, logits_dtype=torch.float32, device="cuda", repetition: float = 1.0, presence: float = 0.0,
                 frequency: float = 0.0, no_repeat: int = 0):
        self.batch, self.beams, self.V, self.d = batch, beams, V, d
        self.bits, self.group, self.softcap, self.eos = bits, group, float(softcap), int(eos)
        self.repetition, self.presence, self.frequency = float(repetition), float(presence), float(frequency)
        self.no_repeat = int(no_repeat)
        self._penalties = self.repetition != 1.0 or self.presence != 0.0 or self.frequency != 0.0 or self.no_repeat != 0
        dev = torch.device(device)
        ws = orpo_beam_select_workspace_bytes(batch, beams, V, beams)
        if ws == 0:
            raise ValueError(f"batch {batch}, beams {beams}, V {V} are out of orpo_beam_select's range")
        self.workspace = torch.empty(ws, dtype=torch.uint8, device=dev)
        self.logits_workspace = torch.empty(orpo_head_logits_q_workspace_bytes(batch * beams, d, bits), dtype=torch.uint8,
                                            device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.logits = torch.empty((batch * beams, V), dtype=logits_dtype, device=dev)
        self.score = torch.empty((batch, beams), dtype=torch.float32, device=dev)
        self.finished = torch.empty((batch, beams), dtype=torch.uint8, device=dev) if self.eos >= 0 else None
        self.parent = torch.empty((batch, beams), dtype=torch.int32, device=dev)
        self.token = torch.empty((batch, beams), dtype=torch.int32, device=dev)
        self.reset()

    def reset(self):
        """Start new responses: all beams of an entry hold the same prompt, so only beam 0 may propose."""
        self.score.fill_(float("-inf"))
        self.score[:, 0] = 0.0
        if self.finished is not None:
            self.finished.zero_()

    def step(self, h, wq, scales, biases, states=(), length=None, stream=None, history=None, prompt=None, bias_token=None,
             bias_value=None, masks=None, mask_row=None, pages=None, pools=(), more=None):
        """One step from the hidden rows h [batch * beams, d]; returns (parent, token) [batch, beams].

        states: tensors [outer, batch * beams, rows, capacity, unit] that follow their parents, up to
        position length[b] of each entry.  history: int32 [batch * beams, capacity], each beam's length[b] tokens so far (the
        first prompt[b] of them the prompt's); it follows its parent and gets the new token at length[b].  bias_token,
        bias_value, masks, mask_row: as for orpo_logits_adjust.  pages, pools: a PagedStates and the pools of it, which follow
        and in which position length[b] can then be written.  more: int32 [batch], 0 for entries that get no such position (they
        ended and were released, or all their positions are in use), else 1; None: 1 for all.  length itself is the caller's to
        raise."""
        if length is None and (history is not None or pages is not None):
            raise ValueError("a history or pages need length")
        if self._penalties and history is None:
            raise ValueError("penalties for repeated tokens need a history")
        if pages is not None and (pages.batch != self.batch or pages.beams != self.beams):
            raise ValueError(f"pages is for {pages.batch} x {pages.beams} beams, expected {self.batch} x {self.beams}")
        if (bias_token is None) != (bias_value is None) or (masks is None) != (mask_row is None):
            raise ValueError("bias_token and bias_value, and masks and mask_row, must be given together")
        pools = () if pools is None else tuple(pools)
        if pages is None and (pools or more is not None):
            raise ValueError("pools and more need pages")
        # The selection replaces the scores, so whatever the calls behind it would refuse is looked at before the first.
        rows, at = self.batch * self.beams, self.score.get_device()
        states = tuple(states)
        if length is not None and (states or history is not None or pages is not None):
            if not (length.dtype is torch.int32 and length.shape == (self.batch,) and length.is_contiguous() and length.get_device() == at):
                _dev(length, "length", I32, (self.batch,))
                raise ValueError(f"length is on {length.device}, expected {self.score.device}")
        for state in states:
            shape = state.shape
            if (len(shape) != 5 or shape[1] != rows or not state.is_contiguous() or state.get_device() != at
                    or (self.batch * shape[2] > 1 << 30 and state.numel() > 0)):
                raise ValueError(f"a state has shape {tuple(shape)} on {state.device}, expected a contiguous tensor [outer, {rows}, rows, "
                                 f"capacity, unit] on {self.score.device}")
        if history is not None:
            _rows(history, "history", I32, rows=rows)
            if not 1 <= history.shape[1] < 1 << 28 or history.get_device() != at:
                raise ValueError(f"history has room for {history.shape[1]} tokens on {history.device}, expected at least 1 and less than 2^28 on "
                                 f"{self.score.device}")
        if more is not None:
            _dev(more, "more", I32, (self.batch,))
        if pages is not None:
            pools = pages._check_pools(pools)
            if pages.table.get_device() != at:
                raise ValueError(f"pages is on {pages.table.device}, expected {self.score.device}")
        orpo_head_logits_q(h, wq, scales, biases, self.bits, self.group, self.softcap, self.logits, self.status,
                           stream, self.logits_workspace)
        if self._penalties or bias_token is not None or masks is not None:
            orpo_logits_adjust(self.logits, self.beams, self.status, history, length, prompt, self.repetition, self.presence,
                               self.frequency, self.no_repeat, bias_token, bias_value, masks, mask_row, stream)
        orpo_beam_select(self.logits, self.score, self.finished, self.eos, self.beams, self.score, self.parent,
                         self.token, self.finished, self.workspace, self.status, stream)
        for state in states:
            orpo_beam_reorder(state, self.parent, length, self.status, stream)
        if history is not None:
            orpo_beam_history(history, self.parent, self.token, length, self.status, stream)
        if pages is not None:
            pages._advance(length, self.parent, more, 1, pools, stream)
        return self.parent, self.token
