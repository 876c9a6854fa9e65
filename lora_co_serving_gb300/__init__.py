"""Python binding of the mixed-batch multi-adapter LoRA layer library (``liblora_mixed.so``).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels.  PyTorch supplies device memory and streams.  The entry points mirror
``include/lora_mixed.h``:

    forward(x, Wt, pool, segs, ...)         -> y   (and the saved xA when asked)
    backward(x, Wt, pool, segs, dY, ...)    -> dX, dA, dB
    sliced_forward / sliced_backward        -> the same for a fused projection of several slices
                                               (q|k|v, gate|up) over one input

and, around the layer in a fine-tuning step (``include/lora_fp8.h``, ``include/lora_preference.h``):

    fp8_quantize / fp8_quantize_weight      -> e4m3 codes and their block scales
    fp8_linear(x, w, w_scales)              -> y = x W^T of a frozen weight in 8 bits
    swiglu_forward / swiglu_backward        -> the MLP activation with an 8-bit checkpoint of the fine-tuning rows
    token_logprob                           -> log probability of each row's label
    preference_forward / preference_backward-> paired log-ratio loss and the gradient of the logits

``segs`` is an int32 array (or list) of rows {start, len, adapter_id, is_train};
``Pool`` holds the stacked adapter factors (A blocks [r_a, K], B blocks [r_a, N])
on the device plus their host-side offsets, ranks and scales.

If the compiled library is missing, calls raise ``LibraryNotBuilt``: there is no
fallback path.
"""
import ctypes
import functools
import os
from collections import namedtuple

import numpy as np

from . import _build

__all__ = ["Pool", "forward", "backward", "sliced_forward", "sliced_backward", "sliced_workspace_size",
           "sliced_xa_size", "workspace_size", "xa_size", "workspace_status", "plan_describe",
           "LoraError", "LibraryNotBuilt", "library", "build", "SAVE_XA", "RECOMPUTE_XA", "ACCUMULATE_GRAD",
           "DEBUG_CHECKS", "plan_check", "static_status", "set_wait_limit", "fp8_quantize", "fp8_quantize_weight",
           "fp8_linear", "fp8_workspace_size", "checkpoint_rows", "swiglu_forward", "swiglu_backward",
           "token_logprob", "preference_forward", "preference_backward", "Preference"]

SAVE_XA = 1
RECOMPUTE_XA = 2
ACCUMULATE_GRAD = 4
DEBUG_CHECKS = 8
BF16 = 0
F32 = 1

ERRORS = {0: "LORA_OK", -1: "LORA_ERR_INVALID_ARG", -2: "LORA_ERR_SEGMENTS", -3: "LORA_ERR_ADAPTER",
          -4: "LORA_ERR_TRAIN_BASE", -5: "LORA_ERR_ALIGNMENT", -6: "LORA_ERR_WORKSPACE", -7: "LORA_ERR_DTYPE",
          -8: "LORA_ERR_CUDA", -9: "LORA_ERR_RANK", -10: "LORA_ERR_LIMIT", -11: "LORA_ERR_TIMEOUT",
          -12: "LORA_ERR_BOUNDS"}

EXPORTED = ["lora_workspace_size", "lora_xa_size", "lora_mixed_forward", "lora_mixed_backward", "lora_last_error",
            "lora_workspace_status", "lora_plan_describe", "lora_set_trace_events", "lora_mixed_forward_static",
            "lora_selftest_wait_timeout", "lora_adamw_step", "lora_mixed_backward_flagged",
            "lora_sliced_workspace_size", "lora_sliced_xa_size", "lora_sliced_forward", "lora_sliced_backward",
            "lora_latency_terms", "lora_latency_features", "lora_latency_fit", "lora_latency_predict",
            "lora_static_status", "lora_plan_check", "lora_set_wait_limit", "lora_fp8_quantize",
            "lora_fp8_quantize_weight", "lora_fp8_workspace_size", "lora_fp8_linear", "lora_checkpoint_rows",
            "lora_swiglu_forward", "lora_swiglu_backward", "lora_token_logprob", "lora_preference_forward",
            "lora_preference_backward"]


class LoraError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__("%s (%d): %s" % (ERRORS.get(code, "?"), code, msg))
        self.code = code


class LibraryNotBuilt(ImportError):
    pass


class _Segment(ctypes.Structure):
    _fields_ = [("start", ctypes.c_int32), ("len", ctypes.c_int32), ("adapter_id", ctypes.c_int32),
                ("is_train", ctypes.c_int32)]


class _Pool(ctypes.Structure):
    _fields_ = [("A", ctypes.c_void_p), ("B", ctypes.c_void_p), ("a_off", ctypes.c_void_p),
                ("b_off", ctypes.c_void_p), ("rank", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("n_adapters", ctypes.c_int32)]


class _Slices(ctypes.Structure):
    _fields_ = [("n_slices", ctypes.c_int32), ("col_bounds", ctypes.c_void_p)]


_LIB = None


def build(force=False):
    """Compile the CUDA library for sm_103a (in-tree) and return its path."""
    return _build.build(force=force)


def library(path=None):
    """The loaded ``liblora_mixed.so`` (ctypes); raises LibraryNotBuilt if it has not been built."""
    global _LIB
    if _LIB is not None and path is None:
        return _LIB
    p = path or _build.LIB
    if not os.path.exists(p):
        raise LibraryNotBuilt("liblora_mixed.so is not built; run lora_co_serving_gb300.build()")
    lib = ctypes.CDLL(p)
    P, I32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    lib.lora_workspace_size.argtypes = [I32, I32, I32, ctypes.c_int, P, P, I32]
    lib.lora_workspace_size.restype = SZ
    lib.lora_xa_size.argtypes = [ctypes.c_int, P, P, I32]
    lib.lora_xa_size.restype = SZ
    lib.lora_mixed_forward.argtypes = [I32, I32, I32, ctypes.c_int, P, P, P, P, I32, P, P, ctypes.c_uint32, P, SZ, P]
    lib.lora_mixed_forward.restype = ctypes.c_int
    lib.lora_mixed_backward.argtypes = [I32, I32, I32, ctypes.c_int, P, P, P, P, I32, P, P, P, P, P, ctypes.c_uint32,
                                        P, SZ, P]
    lib.lora_mixed_backward.restype = ctypes.c_int
    lib.lora_last_error.argtypes = []
    lib.lora_last_error.restype = ctypes.c_char_p
    lib.lora_workspace_status.argtypes = [P, P]
    lib.lora_workspace_status.restype = ctypes.c_int
    lib.lora_plan_describe.argtypes = [I32, I32, I32, P, P, I32, P, P, P, I32]
    lib.lora_plan_describe.restype = ctypes.c_int
    lib.lora_set_trace_events.argtypes = [P]
    lib.lora_set_trace_events.restype = ctypes.c_int
    lib.lora_mixed_forward_static.argtypes = [I32, I32, I32, ctypes.c_int, P, P, P, P, I32, P, P, ctypes.c_uint32, P]
    lib.lora_mixed_forward_static.restype = ctypes.c_int
    lib.lora_plan_check.argtypes = [I32, I32, I32, P, P, P, I32, I32]
    lib.lora_plan_check.restype = ctypes.c_int
    lib.lora_static_status.argtypes = [P]
    lib.lora_static_status.restype = ctypes.c_int
    lib.lora_set_wait_limit.argtypes = [ctypes.c_uint64]
    lib.lora_set_wait_limit.restype = ctypes.c_int
    lib.lora_selftest_wait_timeout.argtypes = [P, SZ, P]
    lib.lora_selftest_wait_timeout.restype = ctypes.c_int
    lib.lora_adamw_step.argtypes = [ctypes.c_int, P, I32, I32, P, P, P, P, P, P, P, P, P, P, P, I32, P, P]
    lib.lora_adamw_step.restype = ctypes.c_int
    lib.lora_mixed_backward_flagged.argtypes = [I32, I32, I32, ctypes.c_int, P, P, P, P, I32, P, P, P, P, P, P,
                                                ctypes.c_uint32, P, SZ, P]
    lib.lora_mixed_backward_flagged.restype = ctypes.c_int
    lib.lora_sliced_workspace_size.argtypes = [I32, I32, I32, ctypes.c_int, P, P, P, I32]
    lib.lora_sliced_workspace_size.restype = SZ
    lib.lora_sliced_xa_size.argtypes = [ctypes.c_int, P, P, P, I32]
    lib.lora_sliced_xa_size.restype = SZ
    lib.lora_sliced_forward.argtypes = [I32, I32, I32, ctypes.c_int, P, P, P, P, P, I32, P, P, ctypes.c_uint32, P, SZ,
                                        P]
    lib.lora_sliced_forward.restype = ctypes.c_int
    lib.lora_sliced_backward.argtypes = [I32, I32, I32, ctypes.c_int, P, P, P, P, P, I32, P, P, P, P, P,
                                         ctypes.c_uint32, P, SZ, P]
    lib.lora_sliced_backward.restype = ctypes.c_int
    lib.lora_latency_terms.argtypes = [I32]
    lib.lora_latency_terms.restype = I32
    lib.lora_latency_features.argtypes = [I32, P, I32, ctypes.c_double, P]
    lib.lora_latency_features.restype = ctypes.c_int
    lib.lora_latency_fit.argtypes = [I32, P, P, I32, P]
    lib.lora_latency_fit.restype = ctypes.c_int
    lib.lora_latency_predict.argtypes = [I32, P, P]
    lib.lora_latency_predict.restype = ctypes.c_double
    I64, F, INT = ctypes.c_int64, ctypes.c_float, ctypes.c_int
    for name, res, args in (
            ("lora_fp8_quantize", INT, [I32, I32, INT, P, I64, P, I64, P, P]),
            ("lora_fp8_quantize_weight", INT, [I32, I32, INT, P, I64, P, P, P]),
            ("lora_fp8_workspace_size", SZ, [I32, I32, I32, I32]),
            ("lora_fp8_linear", INT, [I32, I32, I32, INT, P, I64, P, P, P, P, I64, P, SZ, P]),
            ("lora_checkpoint_rows", I64, [I32, P, I32]),
            ("lora_swiglu_forward", INT, [I32, I32, INT, P, I64, P, I32, P, I64, P, P, P, P]),
            ("lora_swiglu_backward", INT, [I32, I32, INT, P, P, P, I64, P, I64, P, P]),
            ("lora_token_logprob", INT, [I32, I32, INT, P, I64, P, P, P, P]),
            ("lora_preference_forward", INT, [I32, I32, INT, P, I64, P, P, P, I32, F, F, P, P, P, P, P, P]),
            ("lora_preference_backward", INT, [I32, I32, INT, P, I64, P, P, P, P, I32, P, P, I64, P])):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    if path is None:
        _LIB = lib
    return lib


def _check(rc):
    if rc != 0:
        raise LoraError(rc, library().lora_last_error().decode())


def _ptr(t):
    """Raw address of a torch tensor / numpy array (None -> NULL)."""
    if t is None:
        return None
    if isinstance(t, np.ndarray):
        return t.ctypes.data
    return t.data_ptr()


def _dtype_code(t):
    import torch
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError("unsupported dtype %s (bf16 or float32)" % t.dtype)


def _stream_ptr(stream):
    import torch
    if stream is None:      # torch.cuda.current_stream().cuda_stream without its 2.9 us of Stream object
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def segments(segs):
    """Segment table as a contiguous int32 [n, 4] numpy array."""
    a = np.ascontiguousarray(np.asarray(segs, dtype=np.int32).reshape(-1, 4))
    return a


class AdamW(ctypes.Structure):
    """lora_adamw_t: AdamW hyperparameters (step is 1-based)."""
    _fields_ = [("lr", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float),
                ("eps", ctypes.c_float), ("weight_decay", ctypes.c_float), ("step", ctypes.c_int32)]


def adamw_step(pool, K, N, dA, dB, mA, vA, mB, vB, adapters, step, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8,
               weight_decay=0.01, A_master=None, B_master=None, stream=None):
    """AdamW on the listed adapters' blocks of pool.A / pool.B (and fp32 masters if given), in place."""
    code = _dtype_code(pool.A)
    ids = np.ascontiguousarray(adapters, dtype=np.int32)
    hp = AdamW(lr, beta1, beta2, eps, weight_decay, step)
    _check(library().lora_adamw_step(code, pool.cptr(), K, N, _ptr(pool.A), _ptr(pool.B), _ptr(A_master),
                                     _ptr(B_master), _ptr(dA), _ptr(dB), _ptr(mA), _ptr(vA), _ptr(mB), _ptr(vB),
                                     _ptr(ids), ids.shape[0], ctypes.addressof(hp), _stream_ptr(stream)))


class Pool:
    """Stacked adapter pool: A (concatenated [r_a, K] blocks) and B (concatenated [r_a, N] blocks) on the device,
    with host arrays of element offsets, ranks and scales."""

    def __init__(self, A, B, a_off, b_off, rank, scale):
        self.A = A
        self.B = B
        self.a_off = np.ascontiguousarray(a_off, dtype=np.int64)
        self.b_off = np.ascontiguousarray(b_off, dtype=np.int64)
        self.rank = np.ascontiguousarray(rank, dtype=np.int32)
        self.scale = np.ascontiguousarray(scale, dtype=np.float32)
        n = self.rank.shape[0]
        self._c = _Pool(_ptr(A), _ptr(B), _ptr(self.a_off), _ptr(self.b_off), _ptr(self.rank), _ptr(self.scale), n)

    @property
    def n_adapters(self):
        return int(self.rank.shape[0])

    def cptr(self):
        return ctypes.addressof(self._c)


def workspace_size(T, K, N, dtype_code, pool, segs):
    s = segments(segs)
    n = library().lora_workspace_size(T, K, N, dtype_code, pool.cptr(), _ptr(s), s.shape[0])
    if n == 0:
        raise LoraError(-1, library().lora_last_error().decode())
    return int(n)


def xa_size(dtype_code, pool, segs):
    s = segments(segs)
    return int(library().lora_xa_size(dtype_code, pool.cptr(), _ptr(s), s.shape[0]))


def _workspace(T, K, N, code, pool, s, workspace, device):
    """The caller's workspace, or a new one of the size this call needs (the library checks a given one)."""
    import torch
    if workspace is None:
        workspace = torch.empty(workspace_size(T, K, N, code, pool, s), dtype=torch.uint8, device=device)
    return workspace


def forward(x, Wt, pool, segs, y=None, xa_save=None, save_xa=False, workspace=None, stream=None, debug=False,
            check_status=False):
    """y [T, N] = x W + per-segment LoRA; returns y, or (y, xa_save) when save_xa is set.

    debug: LORA_DEBUG_CHECKS (host plan check, in-kernel bounds checks on every store).  check_status: wait for the
    call and raise LoraError if a kernel reported a problem in the workspace status word (a bounded wait that gave
    up, or a debug bounds check)."""
    import torch
    T, K = x.shape
    N = Wt.shape[0]
    code = _dtype_code(x)
    s = segments(segs)
    if y is None:
        y = torch.empty((T, N), dtype=x.dtype, device=x.device)
    if save_xa and xa_save is None:
        n = xa_size(code, pool, s) // x.element_size()
        xa_save = torch.empty(max(n, 1), dtype=x.dtype, device=x.device)
    ws = _workspace(T, K, N, code, pool, s, workspace, x.device)
    flags = (SAVE_XA if save_xa else 0) | (DEBUG_CHECKS if debug else 0)
    _check(library().lora_mixed_forward(T, K, N, code, _ptr(x), _ptr(Wt), pool.cptr(), _ptr(s), s.shape[0], _ptr(y),
                                        _ptr(xa_save), flags, _ptr(ws), ws.numel(), _stream_ptr(stream)))
    if check_status:
        workspace_status(ws, stream)
    return (y, xa_save) if save_xa else y


def forward_static(x, Wt, pool, segs, y=None, xa_save=None, save_xa=False, stream=None):
    """forward() with the library's fixed device scratch instead of a caller workspace (allocates nothing in
    the library; see lora_mixed_forward_static).  Returns y, or (y, xa_save) when save_xa is set."""
    import torch
    T, K = x.shape
    N = Wt.shape[0]
    code = _dtype_code(x)
    s = segments(segs)
    if y is None:
        y = torch.empty((T, N), dtype=x.dtype, device=x.device)
    if save_xa and xa_save is None:
        n = xa_size(code, pool, s) // x.element_size()
        xa_save = torch.empty(max(n, 1), dtype=x.dtype, device=x.device)
    flags = SAVE_XA if save_xa else 0
    _check(library().lora_mixed_forward_static(T, K, N, code, _ptr(x), _ptr(Wt), pool.cptr(), _ptr(s), s.shape[0],
                                               _ptr(y), _ptr(xa_save), flags, _stream_ptr(stream)))
    return (y, xa_save) if save_xa else y


def set_wait_limit(seconds):
    """Limit of every bounded wait in the library's kernels on the current device (1 ms to 60 s; default 1 s)."""
    _check(library().lora_set_wait_limit(int(round(seconds * 1e9))))


def static_status(stream=None):
    """Raise LoraError if a kernel of the last lora_mixed_forward_static call on this device gave up a wait."""
    _check(library().lora_static_status(_stream_ptr(stream)))


def backward(x, Wt, pool, segs, dY, xa_saved=None, dX=None, dA=None, dB=None, want_dx=True, want_grads=True,
             recompute=False, accumulate=False, workspace=None, stream=None, debug=False, check_status=False):
    """LoRA backward of the fine-tuning segments; returns (dX, dA, dB) (dA/dB float32, pool-shaped).
    debug / check_status: as in forward()."""
    import torch
    T, K = x.shape
    N = Wt.shape[0]
    code = _dtype_code(x)
    s = segments(segs)
    if want_dx and dX is None:
        dX = torch.zeros((T, K), dtype=x.dtype, device=x.device)
    if want_grads and dA is None:
        dA = torch.zeros(pool.A.numel(), dtype=torch.float32, device=x.device)
    if want_grads and dB is None:
        dB = torch.zeros(pool.B.numel(), dtype=torch.float32, device=x.device)
    ws = _workspace(T, K, N, code, pool, s, workspace, x.device)
    flags = (RECOMPUTE_XA if recompute else 0) | (ACCUMULATE_GRAD if accumulate else 0) | (DEBUG_CHECKS if debug else 0)
    _check(library().lora_mixed_backward(T, K, N, code, _ptr(x), _ptr(Wt), pool.cptr(), _ptr(s), s.shape[0],
                                         _ptr(dY), _ptr(xa_saved), _ptr(dX) if want_dx else None,
                                         _ptr(dA) if want_grads else None, _ptr(dB) if want_grads else None, flags,
                                         _ptr(ws), ws.numel(), _stream_ptr(stream)))
    if check_status:
        workspace_status(ws, stream)
    return dX, dA, dB


def backward_flagged(x, Wt, pool, segs, dY, xa_saved, xa_valid, dX=None, dA=None, dB=None, accumulate=False,
                     workspace=None, stream=None):
    """backward() with a device flag table choosing, per fine-tuning segment (increasing start order), the saved
    xA (nonzero) or a recompute (zero)."""
    import torch
    T, K = x.shape
    N = Wt.shape[0]
    code = _dtype_code(x)
    s = segments(segs)
    if dX is None:
        dX = torch.zeros((T, K), dtype=x.dtype, device=x.device)
    if dA is None:
        dA = torch.zeros(pool.A.numel(), dtype=torch.float32, device=x.device)
    if dB is None:
        dB = torch.zeros(pool.B.numel(), dtype=torch.float32, device=x.device)
    ws = _workspace(T, K, N, code, pool, s, workspace, x.device)
    flags = ACCUMULATE_GRAD if accumulate else 0
    _check(library().lora_mixed_backward_flagged(T, K, N, code, _ptr(x), _ptr(Wt), pool.cptr(), _ptr(s), s.shape[0],
                                                 _ptr(dY), _ptr(xa_saved), _ptr(xa_valid), _ptr(dX), _ptr(dA),
                                                 _ptr(dB), flags, _ptr(ws), ws.numel(), _stream_ptr(stream)))
    return dX, dA, dB


def workspace_status(workspace, stream=None):
    """Raise LoraError if a kernel of the last call on this workspace gave up a bounded wait."""
    _check(library().lora_workspace_status(_ptr(workspace), _stream_ptr(stream)))


def set_trace_events(events):
    """Record 8 torch.cuda.Event objects around the four launch groups of later calls (None: off)."""
    if events is None:
        _check(library().lora_set_trace_events(None))
        return
    assert len(events) == 8
    arr = (ctypes.c_void_p * 8)(*[e.cuda_event for e in events])
    _check(library().lora_set_trace_events(ctypes.cast(arr, ctypes.c_void_p)))


def plan_check(T, K, N, pool, segs, backward=False, bounds=None):
    """Host check of the bf16 plan of this table (LORA_DEBUG_CHECKS' host half); raises LoraError on a violation."""
    s = segments(segs)
    sl = None if bounds is None else _slices(bounds)
    _check(library().lora_plan_check(T, K, N, pool.cptr(), None if sl is None else sl.cptr(), _ptr(s), s.shape[0],
                                     1 if backward else 0))


def plan_describe(T, K, N, pool, segs, cap=None):
    """(rows [n_tiles, 128], info [n_tiles, 4]) of the forward tile plan; info = gathered, adapters, LoRA cols, x row."""
    s = segments(segs)
    cap = cap or (T // 128 + 2 * s.shape[0] + 8)
    rows = np.zeros((cap, 128), np.int32)
    info = np.zeros((cap, 4), np.int32)
    nt = ctypes.c_int32(0)
    _check(library().lora_plan_describe(T, K, N, pool.cptr(), _ptr(s), s.shape[0], ctypes.addressof(nt), _ptr(rows),
                                        _ptr(info), cap))
    return rows[:nt.value], info[:nt.value]


class Slices:
    """Output-column bounds of a sliced (fused) projection: slice i = columns [bounds[i], bounds[i+1])."""

    def __init__(self, bounds):
        self.bounds = np.ascontiguousarray(bounds, dtype=np.int32)
        self._c = _Slices(self.bounds.shape[0] - 1, _ptr(self.bounds))

    @property
    def n_slices(self):
        return int(self.bounds.shape[0]) - 1

    def cptr(self):
        return ctypes.addressof(self._c)


def _slices(bounds):
    return bounds if isinstance(bounds, Slices) else Slices(bounds)


def sliced_workspace_size(T, K, N, dtype_code, pool, bounds, segs):
    s = segments(segs)
    sl = _slices(bounds)
    n = library().lora_sliced_workspace_size(T, K, N, dtype_code, pool.cptr(), sl.cptr(), _ptr(s), s.shape[0])
    if n == 0:
        raise LoraError(-1, library().lora_last_error().decode())
    return int(n)


def sliced_xa_size(dtype_code, pool, bounds, segs):
    s = segments(segs)
    return int(library().lora_sliced_xa_size(dtype_code, pool.cptr(), _slices(bounds).cptr(), _ptr(s), s.shape[0]))


def sliced_forward(x, Wt, pool, bounds, segs, y=None, xa_save=None, save_xa=False, workspace=None, stream=None):
    """Forward of a sliced projection (Wt [N, K] = the slices' weights stacked; pool laid out per
    lora_sliced_forward).  Returns y, or (y, xa_save) when save_xa is set."""
    import torch
    T, K = x.shape
    N = Wt.shape[0]
    code = _dtype_code(x)
    s = segments(segs)
    sl = _slices(bounds)
    if y is None:
        y = torch.empty((T, N), dtype=x.dtype, device=x.device)
    if save_xa and xa_save is None:
        n = sliced_xa_size(code, pool, sl, s) // x.element_size()
        xa_save = torch.empty(max(n, 1), dtype=x.dtype, device=x.device)
    if workspace is None:
        workspace = torch.empty(sliced_workspace_size(T, K, N, code, pool, sl, s), dtype=torch.uint8, device=x.device)
    flags = SAVE_XA if save_xa else 0
    _check(library().lora_sliced_forward(T, K, N, code, _ptr(x), _ptr(Wt), pool.cptr(), sl.cptr(), _ptr(s),
                                         s.shape[0], _ptr(y), _ptr(xa_save), flags, _ptr(workspace),
                                         workspace.numel(), _stream_ptr(stream)))
    return (y, xa_save) if save_xa else y


def sliced_backward(x, Wt, pool, bounds, segs, dY, xa_saved=None, dX=None, dA=None, dB=None, want_dx=True,
                    want_grads=True, recompute=False, accumulate=False, workspace=None, stream=None):
    """LoRA backward of a sliced projection; dX sums every slice's contribution.  Returns (dX, dA, dB)."""
    import torch
    T, K = x.shape
    N = Wt.shape[0]
    code = _dtype_code(x)
    s = segments(segs)
    sl = _slices(bounds)
    if want_dx and dX is None:
        dX = torch.zeros((T, K), dtype=x.dtype, device=x.device)
    if want_grads and dA is None:
        dA = torch.zeros(pool.A.numel(), dtype=torch.float32, device=x.device)
    if want_grads and dB is None:
        dB = torch.zeros(pool.B.numel(), dtype=torch.float32, device=x.device)
    if workspace is None:
        workspace = torch.empty(sliced_workspace_size(T, K, N, code, pool, sl, s), dtype=torch.uint8, device=x.device)
    flags = (RECOMPUTE_XA if recompute else 0) | (ACCUMULATE_GRAD if accumulate else 0)
    _check(library().lora_sliced_backward(T, K, N, code, _ptr(x), _ptr(Wt), pool.cptr(), sl.cptr(), _ptr(s),
                                          s.shape[0], _ptr(dY), _ptr(xa_saved), _ptr(dX) if want_dx else None,
                                          _ptr(dA) if want_grads else None, _ptr(dB) if want_grads else None, flags,
                                          _ptr(workspace), workspace.numel(), _stream_ptr(stream)))
    return dX, dA, dB


# ----------------------------------------------------------------------------------------------- latency model
EQ_I = 1
EQ_II = 2


def latency_features(model, segs, kv_size=0.0):
    """Feature vector of one step (Eq. I: {sum (n_i+B_d)^2, T_in+B_d, T_ft, K, 1}; Eq. II: {B_d, K, 1})."""
    s = segments(segs)
    p = library().lora_latency_terms(model)
    out = np.zeros(p, np.float64)
    _check(library().lora_latency_features(model, _ptr(s), s.shape[0], float(kv_size), _ptr(out)))
    return out


def latency_fit(model, feats, times):
    """Least-squares coefficients of the model over measured steps (feats [n, terms], times [n])."""
    f = np.ascontiguousarray(feats, dtype=np.float64)
    t = np.ascontiguousarray(times, dtype=np.float64)
    p = library().lora_latency_terms(model)
    coef = np.zeros(p, np.float64)
    _check(library().lora_latency_fit(model, _ptr(f), _ptr(t), t.shape[0], _ptr(coef)))
    return coef


def latency_predict(model, coef, feat):
    c = np.ascontiguousarray(coef, dtype=np.float64)
    f = np.ascontiguousarray(feat, dtype=np.float64)
    return float(library().lora_latency_predict(model, _ptr(c), _ptr(f)))


# ------------------------------------------------------------------------------------ 8-bit products and checkpoints
FP8_BLOCK = 128     # columns (and weight rows) that share a scale


def _blocks(n):
    return -(-n // FP8_BLOCK)


def _matrix(t, name, dtype=None, rows=None, cols=None, contiguous=False):
    """Check a 2-D tensor argument (unit column stride) and return its row distance in elements."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError("%s must have two dimensions, got %d" % (name, len(shape)))
    r, c = shape
    if (rows is not None and r != rows) or (cols is not None and c != cols):
        raise ValueError("%s must be [%s, %s], got [%d, %d]" % (name, "T" if rows is None else rows,
                                                                "K" if cols is None else cols, r, c))
    if dtype is not None and t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.is_contiguous():
        return c
    ld, unit = t.stride()
    if contiguous or (unit != 1 and c > 1):
        raise ValueError("%s must %s" % (name, "be contiguous" if contiguous else "have unit column stride"))
    return ld if r > 1 else max(ld, c)


def _on_stream(fn):
    """fn(..., stream=s) runs with s current, so that what it allocates belongs to s as well: memory that the caller's
    stream has just given back, or takes again after the call, is none of it."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if stream is None:
            return fn(*args, **kw)
        import torch
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(getattr(stream, "cuda_stream", stream))
        with torch.cuda.stream(stream):
            return fn(*args, **kw)
    return call


def _one_device(*tensors):
    """Refuse tensors off the current device: the launch goes to its stream, which no other device's work waits for."""
    import torch
    d = tensors[0].get_device()
    for t in tensors:
        if t is not None and (d < 0 or t.get_device() != d):
            raise ValueError("tensors must lie on one CUDA device")
    if d != torch._C._cuda_getDevice():
        raise ValueError("tensors must lie on one CUDA device, the current one: they lie on cuda:%d, cuda:%d is current"
                         % (d, torch._C._cuda_getDevice()))


def _table(rows):
    """A table of four int32 a row as (bytes, number of rows): bytes cross the ABI without a numpy pointer object."""
    a = np.asarray(rows, dtype=np.int32).reshape(-1, 4)
    return a.tobytes(), a.shape[0]


def _vector(t, name, dtype, n):
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.numel() != n or not t.is_contiguous():
        raise ValueError("%s must be contiguous with %d elements, got %s" % (name, n, tuple(t.shape)))


@_on_stream
def fp8_quantize(x, codes=None, scales=None):
    """x [T, K] (bf16 or float32) -> (codes [T, K] float8_e4m3fn, scales [T, ceil(K / 128)] float32).

    A scale is the smallest power of two that brings its block of 128 columns within e4m3's largest number, 448."""
    import torch
    code, ld = _dtype_code(x), _matrix(x, "x")
    T, K = x.shape
    if codes is None:
        codes = torch.empty((T, K), dtype=torch.float8_e4m3fn, device=x.device)
    if scales is None:
        scales = torch.empty((T, _blocks(K)), dtype=torch.float32, device=x.device)
    ldc = _matrix(codes, "codes", torch.float8_e4m3fn, T, K)
    _one_device(x, codes, scales)
    _matrix(scales, "scales", torch.float32, T, _blocks(K), contiguous=True)
    _check(library().lora_fp8_quantize(T, K, code, _ptr(x), ld, _ptr(codes), ldc, _ptr(scales), _stream_ptr(None)))
    return codes, scales


@_on_stream
def fp8_quantize_weight(W):
    """W [N, K] (bf16 or float32) -> (codes [N, K] float8_e4m3fn, scales [ceil(N / 128), ceil(K / 128)]), a scale for
    each 128 x 128 block.  For the input's gradient pass the transposed weight's (codes.t() and scales.t(), made
    contiguous once: a block of the transposed weight is the transposed block)."""
    import torch
    code, ld = _dtype_code(W), _matrix(W, "W")
    _one_device(W)
    N, K = W.shape
    codes = torch.empty((N, K), dtype=torch.float8_e4m3fn, device=W.device)
    scales = torch.empty((_blocks(N), _blocks(K)), dtype=torch.float32, device=W.device)
    _check(library().lora_fp8_quantize_weight(N, K, code, _ptr(W), ld, _ptr(codes), _ptr(scales),
                                              _stream_ptr(None)))
    return codes, scales


@functools.lru_cache(maxsize=4096)
def fp8_workspace_size(T, K, N, x_fp8=False):
    """Bytes of workspace that fp8_linear needs for these sizes (x given in 8 bits or not)."""
    n = library().lora_fp8_workspace_size(T, K, N, 1 if x_fp8 else 0)
    if n == 0:
        raise LoraError(-1, library().lora_last_error().decode())
    return int(n)


_STATUS_BYTES = 256
_status_workspaces = {}


def _status_workspace(stream_ptr, device):
    """A stream's own workspace for calls that need no more than the status word and do not read it: calls on one stream
    run one after another, but a thread's call may clear the word before another thread has read it.  None while a CUDA
    graph is captured (its replays may run beside the stream's later calls)."""
    import torch
    if torch._C._cuda_isCurrentStreamCapturing():
        return None
    key = (device.index, stream_ptr)
    ws = _status_workspaces.get(key)
    if ws is None:
        ws = _status_workspaces[key] = torch.empty(_STATUS_BYTES, dtype=torch.uint8, device=device)
    return ws


@_on_stream
def fp8_linear(x, w, w_scales, x_scales=None, y=None, workspace=None, check_status=False):
    """y [T, N] (bf16) = x W^T for a frozen weight in 8 bits (w [N, K] codes, w_scales [ceil(N/128), ceil(K/128)]).

    x [T, K] is bf16 or float32 and is quantized on the way, or float8_e4m3fn codes with their x_scales
    [T, ceil(K / 128)].  check_status: as in forward()."""
    import torch
    ld = _matrix(x, "x")
    T, K = x.shape
    N = w.shape[0]
    _matrix(w, "w", torch.float8_e4m3fn, N, K, contiguous=True)
    _matrix(w_scales, "w_scales", torch.float32, _blocks(N), _blocks(K), contiguous=True)
    if x_scales is None:
        code = _dtype_code(x)
    else:
        code = BF16
        _matrix(x, "x", torch.float8_e4m3fn)
        _matrix(x_scales, "x_scales", torch.float32, T, _blocks(K), contiguous=True)
    if y is None:
        y, ldy = torch.empty((T, N), dtype=torch.bfloat16, device=x.device), N
    else:
        ldy = _matrix(y, "y", torch.bfloat16, T, N)
    _one_device(x, w, w_scales, x_scales, y, workspace)
    st = _stream_ptr(None)
    if workspace is None:
        need = fp8_workspace_size(T, K, N, x_scales is not None)
        workspace = _status_workspace(st, x.device) if need <= _STATUS_BYTES and not check_status else None
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    rc = library().lora_fp8_linear(T, K, N, code, x.data_ptr(), ld, _ptr(x_scales), w.data_ptr(), w_scales.data_ptr(),
                                   y.data_ptr(), ldy, workspace.data_ptr(), workspace.numel(), st)
    if rc != 0:
        _check(rc)
    if check_status and T > 0:      # a call without rows launches nothing and leaves the status word as it was
        workspace_status(workspace)
    return y


def checkpoint_rows(T, segs):
    """Rows of the 8-bit checkpoint of a segment table: the tokens of its fine-tuning segments."""
    n = library().lora_checkpoint_rows(T, *_table(segs))
    if n < 0:
        raise LoraError(int(n), library().lora_last_error().decode())
    return int(n)


@_on_stream
def swiglu_forward(gu, segs=None, checkpoint=False, fp8_out=False, h=None, h_scales=None):
    """h [T, I] = silu(gate) * up of gu [T, 2 I] = gate|up.

    checkpoint: also keep gate|up of the fine-tuning rows of `segs` in 8 bits; returns (h, saved) with saved =
    (codes [R, 2 I], scales [R, 2 ceil(I / 128)]), rows in increasing segment order.  fp8_out: h is (codes, scales)
    for the next fp8_linear instead of a tensor of gu's type."""
    import torch
    code, ld = _dtype_code(gu), _matrix(gu, "gu")
    T, I2 = gu.shape
    if I2 % 2:
        raise ValueError("gu must hold gate|up, an even number of columns; got %d" % I2)
    I = I2 // 2
    s, n_segs = (None, 0) if segs is None else _table(segs)
    ck = cs = None
    if checkpoint:
        if s is None:
            raise ValueError("a checkpoint needs the batch's segment table")
        R = library().lora_checkpoint_rows(T, s, n_segs)
        if R < 0:
            _check(R)
        ck = torch.empty((R, I2), dtype=torch.float8_e4m3fn, device=gu.device)
        cs = torch.empty((R, 2 * _blocks(I)), dtype=torch.float32, device=gu.device)
    out = torch.float8_e4m3fn if fp8_out else gu.dtype
    if h is None:
        h, ldh = torch.empty((T, I), dtype=out, device=gu.device), I
    else:
        ldh = _matrix(h, "h", out, T, I)
    if fp8_out and h_scales is None:
        h_scales = torch.empty((T, _blocks(I)), dtype=torch.float32, device=gu.device)
    if fp8_out:
        _matrix(h_scales, "h_scales", torch.float32, T, _blocks(I), contiguous=True)
    keep = ck is not None and ck.numel() > 0
    _one_device(gu, h, h_scales)
    rc = library().lora_swiglu_forward(T, I, code, gu.data_ptr(), ld, s, n_segs, h.data_ptr(), ldh,
                                       h_scales.data_ptr() if fp8_out else None, ck.data_ptr() if keep else None,
                                       cs.data_ptr() if keep else None, _stream_ptr(None))
    if rc != 0:
        _check(rc)
    h = (h, h_scales) if fp8_out else h
    return (h, (ck, cs)) if checkpoint else h


@_on_stream
def swiglu_backward(saved, dh, fp8_out=False, dgu=None, dgu_scales=None):
    """Gradient of gate|up [R, 2 I] from the checkpoint `saved` of swiglu_forward and dh [R, I], the gradient of h for
    the checkpoint's rows.  fp8_out: (codes, scales) for the next fp8_linear (I a multiple of 128)."""
    import torch
    ck, cs = saved
    code, ld = _dtype_code(dh), _matrix(dh, "dh")
    R, I = dh.shape
    _matrix(ck, "the checkpoint's codes", torch.float8_e4m3fn, R, 2 * I, contiguous=True)
    _matrix(cs, "the checkpoint's scales", torch.float32, R, 2 * _blocks(I), contiguous=True)
    out = torch.float8_e4m3fn if fp8_out else dh.dtype
    if dgu is None:
        dgu, ldo = torch.empty((R, 2 * I), dtype=out, device=dh.device), 2 * I
    else:
        ldo = _matrix(dgu, "dgu", out, R, 2 * I)
    if fp8_out and dgu_scales is None:
        dgu_scales = torch.empty((R, 2 * _blocks(I)), dtype=torch.float32, device=dh.device)
    if fp8_out:
        _matrix(dgu_scales, "dgu_scales", torch.float32, R, 2 * _blocks(I), contiguous=True)
    _one_device(dh, ck, cs, dgu, dgu_scales)
    rc = library().lora_swiglu_backward(R, I, code, ck.data_ptr(), cs.data_ptr(), dh.data_ptr(), ld, dgu.data_ptr(), ldo,
                                        dgu_scales.data_ptr() if fp8_out else None, _stream_ptr(None))
    if rc != 0:
        _check(rc)
    return (dgu, dgu_scales) if fp8_out else dgu


# -------------------------------------------------------------------------------------------------- preference loss
Preference = namedtuple("Preference", ["loss", "rewards", "logp", "lse", "coef"])


@_on_stream
def token_logprob(logits, labels, logp=None, lse=None):
    """(logp [T], lse [T]) float32: log probability of each row's label, and the row's log-sum-exp.  labels int64 [T];
    a negative label's row is not read and gives zeros."""
    import torch
    code, ld = _dtype_code(logits), _matrix(logits, "logits")
    T, V = logits.shape
    _vector(labels, "labels", torch.int64, T)
    if logp is None:
        logp = torch.empty(T, dtype=torch.float32, device=logits.device)
    if lse is None:
        lse = torch.empty(T, dtype=torch.float32, device=logits.device)
    _vector(logp, "logp", torch.float32, T)
    _vector(lse, "lse", torch.float32, T)
    _one_device(logits, labels, logp, lse)
    _check(library().lora_token_logprob(T, V, code, _ptr(logits), ld, _ptr(labels), _ptr(logp), _ptr(lse),
                                        _stream_ptr(None)))
    return logp, lse


@_on_stream
def preference_forward(logits, labels, ref_logp, pairs, beta=0.1, label_smoothing=0.0):
    """Paired log-ratio loss of a policy's logits [T, V] against a reference's ref_logp [T].

    pairs: int32 rows {chosen start, chosen length, rejected start, rejected length} over the batch's rows.  Returns
    Preference(loss [P], rewards [P, 2], logp [T], lse [T], coef [P, 2]), float32; lse and coef are the backward's."""
    import torch
    code, ld = _dtype_code(logits), _matrix(logits, "logits")
    T, V = logits.shape
    _vector(labels, "labels", torch.int64, T)
    _vector(ref_logp, "ref_logp", torch.float32, T)
    _one_device(logits, labels, ref_logp)
    p, n = _table(pairs)
    new = ref_logp.new_empty
    logp, lse, loss, rewards, coef = new(T), new(T), new(n), new((n, 2)), new((n, 2))
    rc = library().lora_preference_forward(T, V, code, logits.data_ptr(), ld, labels.data_ptr(), ref_logp.data_ptr(),
                                           p, n, beta, label_smoothing, loss.data_ptr(), rewards.data_ptr(),
                                           logp.data_ptr(), lse.data_ptr(), coef.data_ptr(), _stream_ptr(None))
    if rc != 0:
        _check(rc)
    return Preference(loss, rewards, logp, lse, coef)


@_on_stream
def preference_backward(logits, labels, lse, coef, pairs, dloss=None, dlogits=None):
    """Gradient of the logits [T, V] in their type: every row is written, zeros where a row is not counted.

    dloss [P] float32: the gradient of each pair's loss (default: 1 / P each, the mean's).  dlogits may be `logits`
    itself: the gradient then takes the logits' place.  Rows whose |lse| is 256 or more are read twice: one float32 number
    no longer holds it well enough for their probabilities."""
    import torch
    code, ld = _dtype_code(logits), _matrix(logits, "logits")
    T, V = logits.shape
    p, n = _table(pairs)
    _vector(labels, "labels", torch.int64, T)
    _vector(lse, "lse", torch.float32, T)
    _vector(coef, "coef", torch.float32, 2 * n)
    if dloss is not None:
        _vector(dloss, "dloss", torch.float32, n)
    if dlogits is None:
        dlogits, ldd = torch.empty((T, V), dtype=logits.dtype, device=logits.device), V
    else:
        ldd = _matrix(dlogits, "dlogits", logits.dtype, T, V)
    _one_device(logits, labels, lse, coef, dloss, dlogits)
    rc = library().lora_preference_backward(T, V, code, logits.data_ptr(), ld, labels.data_ptr(), lse.data_ptr(),
                                            coef.data_ptr(), p, n, _ptr(dloss), dlogits.data_ptr(), ldd,
                                            _stream_ptr(None))
    if rc != 0:
        _check(rc)
    return dlogits
