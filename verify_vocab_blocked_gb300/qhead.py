"""Thin ctypes binding of libqhead.so (include/qhead.h).

Argument marshalling only: every step of the head runs in the library's CUDA
kernels.  PyTorch provides device memory and the current stream.  If the
library has not been built, the first call raises -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
from array import array
from dataclasses import dataclass

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libqhead.so")

QHEAD_OK, QHEAD_EINVAL, QHEAD_EUNSUPPORTED, QHEAD_ECUDA = 0, 1, 2, 3
QHEAD_SB_F16, QHEAD_SB_BF16, QHEAD_SB_F32 = 0, 1, 2
_SB_CODE = {torch.float16: QHEAD_SB_F16, torch.bfloat16: QHEAD_SB_BF16,
            torch.float32: QHEAD_SB_F32}

# Every symbol include/qhead.h declares.
EXPORTS = ("qhead_fwd_workspace", "qhead_bwd_workspace", "qhead_fwd", "qhead_bwd",
           "qhead_last_error", "qhead_version", "qhead_time_next_head_kernel",
           "qhead_fwd_noalloc", "qhead_test_stall_next_call", "qhead_verify",
           "qhead_bwd_dw_workspace", "qhead_bwd_dw", "qhead_fwd_blockmax_workspace",
           "qhead_fwd_blockmax", "qhead_bwd_blockskip_workspace", "qhead_bwd_blockskip",
           "qhead_bwd_filter_workspace", "qhead_bwd_filter", "qhead_embed",
           "qhead_embed_bwd_workspace", "qhead_embed_bwd", "qhead_layer_norm",
           "qhead_layer_norm_bwd_workspace", "qhead_layer_norm_bwd",
           "qhead_distill_fwd_workspace", "qhead_distill_fwd", "qhead_distill_bwd_workspace",
           "qhead_distill_bwd", "qhead_distill_kept", "qhead_linear_workspace", "qhead_linear",
           "qhead_linear_bwd_workspace", "qhead_linear_bwd", "qhead_linear_bwd_dbias", "qhead_add_norm", "qhead_norm_8bit",
           "qhead_add_norm_bwd", "qhead_grad_norm_workspace", "qhead_grad_norm", "qhead_clip_grads")


class CHead(ctypes.Structure):
    _fields_ = [("wq", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("biases", ctypes.c_void_p), ("V", ctypes.c_int64), ("H", ctypes.c_int32),
                ("bits", ctypes.c_int32), ("group", ctypes.c_int32),
                ("sb_dtype", ctypes.c_int32), ("softcap", ctypes.c_float)]


class QheadError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"qhead error {code}: {msg}")
        self.code = code


_lib = None


def lib() -> ctypes.CDLL:
    """Load libqhead.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -m verify_vocab_blocked_gb300.build` (no CPU fallback exists)")
    L = ctypes.CDLL(LIB_PATH)
    vp, i64, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
    hp = ctypes.POINTER(CHead)
    L.qhead_fwd_workspace.argtypes = [hp, i64]
    L.qhead_fwd_workspace.restype = sz
    L.qhead_bwd_workspace.argtypes = [hp, i64]
    L.qhead_bwd_workspace.restype = sz
    L.qhead_bwd_dw_workspace.argtypes = [hp, i64]
    L.qhead_bwd_dw_workspace.restype = sz
    L.qhead_fwd.argtypes = [hp, vp, i64, vp, vp, vp, vp, vp, vp, sz, vp]
    L.qhead_fwd.restype = ctypes.c_int
    L.qhead_bwd.argtypes = [hp, vp, i64, vp, vp, vp, vp, vp, vp, sz, vp]
    L.qhead_bwd.restype = ctypes.c_int
    L.qhead_bwd_dw.argtypes = [hp, vp, i64, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.qhead_bwd_dw.restype = ctypes.c_int
    for name in ("qhead_fwd_blockmax_workspace", "qhead_bwd_blockskip_workspace",
                 "qhead_bwd_filter_workspace"):
        getattr(L, name).argtypes = [hp, i64]
        getattr(L, name).restype = sz
    L.qhead_fwd_blockmax.argtypes = [hp, vp, i64, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.qhead_fwd_blockmax.restype = ctypes.c_int
    L.qhead_bwd_blockskip.argtypes = [hp, vp, i64, vp, vp, vp, vp, vp, ctypes.c_float, vp, vp,
                                      sz, vp]
    L.qhead_bwd_blockskip.restype = ctypes.c_int
    L.qhead_bwd_filter.argtypes = [hp, vp, i64, vp, vp, vp, vp, ctypes.c_float, vp, vp, vp, sz,
                                   vp]
    L.qhead_bwd_filter.restype = ctypes.c_int
    L.qhead_verify.argtypes = [hp, vp, i64, i64, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.qhead_verify.restype = ctypes.c_int
    i32, f32 = ctypes.c_int, ctypes.c_float
    L.qhead_embed.argtypes = [hp, vp, i64, vp, f32, vp, i32, vp]
    L.qhead_embed.restype = i32
    L.qhead_embed_bwd_workspace.argtypes = [hp, i64]
    L.qhead_embed_bwd_workspace.restype = sz
    L.qhead_embed_bwd.argtypes = [hp, vp, i64, vp, f32, vp, i32, vp, i32, vp, sz, vp]
    L.qhead_embed_bwd.restype = i32
    L.qhead_layer_norm.argtypes = [vp, i32, i64, i64, i64, vp, vp, i32, f32, i32, vp, i32, vp, vp,
                                   vp]
    L.qhead_layer_norm.restype = i32
    L.qhead_layer_norm_bwd_workspace.argtypes = [i64, i64]
    L.qhead_layer_norm_bwd_workspace.restype = sz
    L.qhead_layer_norm_bwd.argtypes = [vp, i32, i64, i64, i64, vp, i32, vp, vp, vp, i32, i64, vp,
                                       vp, vp, vp, sz, vp]
    L.qhead_layer_norm_bwd.restype = i32
    for name in ("qhead_distill_fwd_workspace", "qhead_distill_bwd_workspace"):
        getattr(L, name).argtypes = [hp, i64, i64]
        getattr(L, name).restype = sz
    L.qhead_distill_kept.argtypes = [hp, i64, i64]
    L.qhead_distill_kept.restype = i64
    L.qhead_distill_fwd.argtypes = [hp, vp, i64, vp, vp, i32, i64, f32, vp, vp, vp, vp, vp, sz, vp]
    L.qhead_distill_fwd.restype = i32
    L.qhead_distill_bwd.argtypes = [hp, vp, i64, vp, vp, i32, i64, f32, vp, vp, vp, vp, vp, vp, sz,
                                    vp]
    L.qhead_distill_bwd.restype = i32
    size = [vp, i32, i64, i64, i64, vp, i64, i64]
    for name in ("qhead_linear_workspace", "qhead_linear_bwd_workspace"):
        getattr(L, name).argtypes = size
        getattr(L, name).restype = sz
    L.qhead_linear.argtypes = size + [vp, vp, vp, i32, i32, vp, i32, i64, vp, i32, vp, vp, sz, vp]
    L.qhead_linear.restype = i32
    L.qhead_linear_bwd.argtypes = size + [vp, i32, i64, vp, i32, vp, vp, vp, vp, sz, vp]
    L.qhead_linear_bwd.restype = i32
    L.qhead_linear_bwd_dbias.argtypes = size + [vp, i32, i64, vp, i32, vp, vp, vp, i32, vp, sz, vp]
    L.qhead_linear_bwd_dbias.restype = i32
    added = [vp, i32, i64, vp, i32, i64, i64, i64, vp, vp, i32, f32, i32, vp]
    L.qhead_add_norm.argtypes = added + [vp, i32, vp, vp, vp]
    L.qhead_add_norm.restype = i32
    L.qhead_norm_8bit.argtypes = added + [vp, vp, vp]
    L.qhead_norm_8bit.restype = i32
    L.qhead_add_norm_bwd.argtypes = [vp, i32, i64, i64, i64, vp, i32, vp, vp, vp, i32, i64, vp, i64, vp,
                                     vp, vp, vp, sz, vp]
    L.qhead_add_norm_bwd.restype = i32
    L.qhead_grad_norm_workspace.argtypes = [i64]
    L.qhead_grad_norm_workspace.restype = sz
    L.qhead_grad_norm.argtypes = [vp, vp, vp, i64, vp, vp, sz, vp]
    L.qhead_grad_norm.restype = i32
    L.qhead_clip_grads.argtypes = [vp, vp, vp, i64, f32, vp, vp, vp, vp, sz, vp]
    L.qhead_clip_grads.restype = i32
    L.qhead_last_error.argtypes = []
    L.qhead_last_error.restype = ctypes.c_char_p
    L.qhead_version.argtypes = []
    L.qhead_version.restype = ctypes.c_char_p
    L.qhead_time_next_head_kernel.argtypes = [vp, vp]
    L.qhead_time_next_head_kernel.restype = None
    L.qhead_test_stall_next_call.argtypes = [ctypes.c_int]
    L.qhead_test_stall_next_call.restype = None
    L.qhead_fwd_noalloc.argtypes = [hp, vp, i64, vp, vp, vp, vp, vp, vp]
    L.qhead_fwd_noalloc.restype = ctypes.c_int
    _lib = L
    return L


def test_stall_next_call(armed: bool = True) -> None:
    """Arm the library's one-shot stall switch on this thread: the next fwd/bwd
    call's pipelined head kernel gets no loads, its bounded waits expire and
    the call's active rows come back NaN (argmax -1)."""
    lib().qhead_test_stall_next_call(1 if armed else 0)


def time_next_head_kernel(start: torch.cuda.Event, stop: torch.cuda.Event) -> None:
    """Arm the library's one-shot hook: the next fwd/bwd call on this thread
    records `start` / `stop` around its head kernel on the call's stream.
    Both events must already exist (record them once beforehand)."""
    lib().qhead_time_next_head_kernel(start.cuda_event, stop.cuda_event)


def last_error() -> str:
    return lib().qhead_last_error().decode()


def _check(rc: int):
    if rc != QHEAD_OK:
        raise QheadError(rc, last_error())


@dataclass
class Head:
    """A quantized head resident on the GPU (FlashCceHead layout)."""
    wq: torch.Tensor        # int32 (uint32 bit patterns) [V, H*bits/32]
    scales: torch.Tensor    # float16, bfloat16 or float32 [V, H/group]
    biases: torch.Tensor    # the same type as scales, [V, H/group]
    bits: int
    group: int = 64
    softcap: float = 0.0

    @property
    def V(self) -> int:
        return int(self.wq.shape[0])

    @property
    def H(self) -> int:
        return int(self.wq.shape[1]) * 32 // self.bits

    def c(self) -> CHead:
        wq, scales, biases, bits = self.wq, self.scales, self.biases, self.bits
        if not (wq.is_contiguous() and scales.is_contiguous() and biases.is_contiguous()):
            raise ValueError("head tensors must be contiguous")
        if scales.device != wq.device or biases.device != wq.device:
            raise ValueError("head tensors must be on one device")
        dtype = scales.dtype
        code = _SB_CODE.get(dtype)
        if code is None or biases.dtype != dtype:
            raise ValueError("scales and biases must share one type: float16, bfloat16 or "
                             "float32")
        V, words = wq.shape
        H = words * 32 // bits
        groups = H // self.group if self.group > 0 else 0
        if scales.numel() != V * groups or biases.numel() != V * groups:
            raise ValueError(f"scales and biases must have shape [{V}, {groups}]")
        return CHead(wq.data_ptr(), scales.data_ptr(), biases.data_ptr(), V,
                     H, bits, self.group, code, self.softcap)

    @staticmethod
    def from_numpy(wq, scales, biases, bits, group=64, softcap=0.0, device="cuda",
                   sb_dtype: str = "f16"):
        """Scales and biases: float16 or float32 arrays, or uint16 bf16 bit
        patterns with sb_dtype="bf16"."""
        import numpy as np

        def sb(x):
            x = np.ascontiguousarray(x)
            if sb_dtype == "bf16":
                return torch.from_numpy(x.astype(np.uint16).view(np.int16)).view(
                    torch.bfloat16).to(device)
            want = {"f16": np.float16, "f32": np.float32}[sb_dtype]
            if x.dtype != want:
                raise ValueError(f"scales/biases are {x.dtype}, sb_dtype is {sb_dtype}")
            return torch.from_numpy(x).to(device)

        return Head(torch.from_numpy(np.ascontiguousarray(wq).view(np.int32)).to(device),
                    sb(scales), sb(biases), bits, group, softcap)


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _usable(dev: torch.device, stream, workspace: torch.Tensor | None = None) -> None:
    """The checked tensors' device must be the GPU whose stream the kernels are
    launched on: an address of another device, or of the host, is not for them."""
    if dev.type != "cuda":
        raise ValueError(f"the tensors are on {dev}: they must be on a GPU")
    if dev.index != torch.cuda.current_device():
        raise ValueError(f"the tensors are on {dev} but the current device is "
                         f"cuda:{torch.cuda.current_device()}: call under torch.cuda.device")
    if stream is not None and stream.device != dev:
        raise ValueError(f"the tensors are on {dev} but the stream is of {stream.device}")
    if workspace is not None:
        if workspace.device != dev:
            raise ValueError(f"the tensors are on {dev} but the workspace is on {workspace.device}")
        if not workspace.is_contiguous():  # (an expanded one has less memory than elements)
            raise ValueError("workspace must be contiguous")


# The current stream's handle without a Stream object around it, where torch has it
# (building one is a fifth of a small call's time).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, dev: torch.device) -> int:
    """The handle of the given stream, or of the current one."""
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is None:
        return torch.cuda.current_stream(dev).cuda_stream
    return _raw_stream(dev.index)


def _check_h(head: Head, h: torch.Tensor, what: str = "[M, H]") -> int:
    """h must be a contiguous bf16 matrix with head.H columns, on the head's
    device; returns M."""
    if not isinstance(h, torch.Tensor) or h.dtype != torch.bfloat16 or h.dim() != 2 \
            or not h.is_contiguous():
        raise ValueError(f"h must be a contiguous bf16 {what} tensor")
    M, H = h.shape
    wq = head.wq
    if H != wq.shape[1] * 32 // head.bits:
        raise ValueError(f"h has {H} columns but the head's hidden size H is {head.H}")
    if wq.device != h.device:
        raise ValueError(f"h is on {h.device} but the head is on {wq.device}")
    return M


def _check_vec(name: str, t: torch.Tensor | None, n: int, dtypes, dev, required: bool = True):
    """A per-row argument: contiguous, shape [n], one of `dtypes`, on `dev`.
    Returns the tensor to pass (bool masks are passed as their uint8 bytes)."""
    if t is None:
        if required:
            raise ValueError(f"{name} is required")
        return None
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch tensor")
    if t.dtype not in dtypes:
        names = " or ".join(str(d).replace("torch.", "") for d in dtypes)
        raise ValueError(f"{name} must be {names}, got {str(t.dtype).replace('torch.', '')}")
    if t.dim() != 1 or t.shape[0] != n:
        raise ValueError(f"{name} must have shape [{n}], got {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, h on {dev}")
    return t.view(torch.uint8) if t.dtype == torch.bool else t


def _targets(t, M, dev, required):
    return _check_vec("targets", t, M, (torch.int32,), dev, required)


def _mask(mk, M, dev):
    return _check_vec("mask", mk, M, (torch.uint8, torch.bool), dev, required=False)


def _f32(name, t, M, dev):
    return _check_vec(name, t, M, (torch.float32,), dev)


def fwd_workspace(head: Head, M: int) -> int:
    n = lib().qhead_fwd_workspace(ctypes.byref(head.c()), M)
    if n == ctypes.c_size_t(-1).value:
        raise QheadError(QHEAD_EINVAL, last_error())
    return int(n)


def bwd_workspace(head: Head, M: int) -> int:
    n = lib().qhead_bwd_workspace(ctypes.byref(head.c()), M)
    if n == ctypes.c_size_t(-1).value:
        raise QheadError(QHEAD_EINVAL, last_error())
    return int(n)


def bwd_dw_workspace(head: Head, M: int) -> int:
    n = lib().qhead_bwd_dw_workspace(ctypes.byref(head.c()), M)
    if n == ctypes.c_size_t(-1).value:
        raise QheadError(QHEAD_EINVAL, last_error())
    return int(n)


def alloc_workspace(nbytes: int, device) -> torch.Tensor:
    """A 256-byte aligned device buffer of at least nbytes (torch allocations are)."""
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)


# Memory of a call on a stream given to it.  The caller has ordered that stream
# behind whatever makes the inputs (stream.wait_stream(...)) and orders what reads
# the outputs behind it; whose memory a block is, is settled here, so that any tensor
# of the call may be dropped as soon as the call has returned:
#   * a workspace and the outputs come from the given stream's own pool: a block that
#     the current stream's queued work still uses is not among them;
#   * the outputs are recorded on the current stream, which goes on to use them;
#   * the inputs are recorded on the given stream, which reads them after the call.

def _scratch(nbytes: int, dev, stream) -> torch.Tensor:
    """A workspace of this call's own."""
    if stream is None:
        return alloc_workspace(nbytes, dev)
    with torch.cuda.stream(stream):
        return alloc_workspace(nbytes, dev)


def _out(shape, dtype, dev, stream, fill: float | None = None) -> torch.Tensor:
    """An output of the call (filled, on the call's stream, if `fill` is given)."""
    if stream is None:
        t = torch.empty(shape, dtype=dtype, device=dev)
        return t if fill is None else t.fill_(fill)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=dev)
        if fill is not None:
            t.fill_(fill)
    t.record_stream(torch.cuda.current_stream(dev))
    return t


def _reads(stream, head: "Head | None", *tensors) -> None:
    """Records the call's inputs (and a buffer or workspace given to it) on its stream."""
    if stream is None:
        return
    for t in (head.wq, head.scales, head.biases) if head is not None else ():
        t.record_stream(stream)
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


def fwd(head: Head, h: torch.Tensor, targets: torch.Tensor | None = None,
        mask: torch.Tensor | None = None, *, want_logp: bool = True, want_lse: bool = True,
        want_argmax: bool = True, workspace: torch.Tensor | None = None, stream=None):
    """Returns (logp or None, lse or None, argmax or None) for every row of h."""
    M = _check_h(head, h)
    dev = h.device
    targets = _targets(targets, M, dev, required=False)
    mask = _mask(mask, M, dev)
    want_logp = want_logp and targets is not None
    _usable(dev, stream, workspace)
    logp = _out(M, torch.float32, dev, stream) if want_logp else None
    lse = _out(M, torch.float32, dev, stream) if want_lse else None
    am = _out(M, torch.int32, dev, stream) if want_argmax else None
    _reads(stream, head, h, targets, mask, workspace)
    if workspace is None:
        workspace = _scratch(fwd_workspace(head, M), dev, stream)
    _check(lib().qhead_fwd(ctypes.byref(head.c()), h.data_ptr(), M, _ptr(targets), _ptr(mask),
                           _ptr(logp), _ptr(lse), _ptr(am), workspace.data_ptr(),
                           workspace.numel(), _stream(stream, dev)))
    return logp, lse, am


def bwd(head: Head, h: torch.Tensor, targets: torch.Tensor, lse: torch.Tensor,
        dlogp: torch.Tensor, mask: torch.Tensor | None = None, *,
        workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """dh [M, H] float32 of sum_m dlogp[m] * logp[m]."""
    M = _check_h(head, h)
    dev = h.device
    targets = _targets(targets, M, dev, required=True)
    mask = _mask(mask, M, dev)
    lse, dlogp = _f32("lse", lse, M, dev), _f32("dlogp", dlogp, M, dev)
    _usable(dev, stream, workspace)
    dh = _out((M, head.H), torch.float32, dev, stream)
    _reads(stream, head, h, targets, lse, dlogp, mask, workspace)
    if workspace is None:
        workspace = _scratch(bwd_workspace(head, M), dev, stream)
    _check(lib().qhead_bwd(ctypes.byref(head.c()), h.data_ptr(), M, _ptr(targets), _ptr(mask),
                           lse.data_ptr(), dlogp.data_ptr(), dh.data_ptr(), workspace.data_ptr(),
                           workspace.numel(), _stream(stream, dev)))
    return dh


def bwd_dw(head: Head, h: torch.Tensor, targets: torch.Tensor, lse: torch.Tensor,
           dlogp: torch.Tensor, mask: torch.Tensor | None = None, *, want_dh: bool = False,
           workspace: torch.Tensor | None = None, stream=None):
    """(dh [M, H] float32 or None, dw [V, H] float32): the gradients of
    sum_m dlogp[m] * logp[m] with respect to h and to the dequantized head."""
    M = _check_h(head, h)
    dev = h.device
    targets = _targets(targets, M, dev, required=True)
    mask = _mask(mask, M, dev)
    lse, dlogp = _f32("lse", lse, M, dev), _f32("dlogp", dlogp, M, dev)
    _usable(dev, stream, workspace)
    dh = _out((M, head.H), torch.float32, dev, stream) if want_dh else None
    dw = _out((head.V, head.H), torch.float32, dev, stream)
    _reads(stream, head, h, targets, lse, dlogp, mask, workspace)
    if workspace is None:
        workspace = _scratch(bwd_dw_workspace(head, M), dev, stream)
    _check(lib().qhead_bwd_dw(ctypes.byref(head.c()), h.data_ptr(), M, targets.data_ptr(),
                              _ptr(mask), lse.data_ptr(), dlogp.data_ptr(), _ptr(dh),
                              dw.data_ptr(), workspace.data_ptr(), workspace.numel(),
                              _stream(stream, dev)))
    return dh, dw


def _ws_size(fn_name: str, head: Head, M: int) -> int:
    n = getattr(lib(), fn_name)(ctypes.byref(head.c()), M)
    if n == ctypes.c_size_t(-1).value:
        raise QheadError(QHEAD_EINVAL, last_error())
    return int(n)


def fwd_blockmax(head: Head, h: torch.Tensor, targets: torch.Tensor | None = None,
                 mask: torch.Tensor | None = None, *, workspace: torch.Tensor | None = None,
                 stream=None):
    """(logp or None, lse, argmax, block_max [M, ceil(V / 256)]): the forward
    plus each row's maximum capped logit per 256-row vocab tile."""
    M = _check_h(head, h)
    dev = h.device
    targets = _targets(targets, M, dev, required=False)
    mask = _mask(mask, M, dev)
    _usable(dev, stream, workspace)
    logp = _out(M, torch.float32, dev, stream) if targets is not None else None
    lse = _out(M, torch.float32, dev, stream)
    am = _out(M, torch.int32, dev, stream)
    bm = _out((M, (head.V + 255) // 256), torch.float32, dev, stream, fill=float("-inf"))
    _reads(stream, head, h, targets, mask, workspace)
    if workspace is None:
        workspace = _scratch(_ws_size("qhead_fwd_blockmax_workspace", head, M), dev, stream)
    _check(lib().qhead_fwd_blockmax(ctypes.byref(head.c()), h.data_ptr(), M, _ptr(targets),
                                    _ptr(mask), _ptr(logp), lse.data_ptr(), am.data_ptr(),
                                    bm.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                    _stream(stream, dev)))
    return logp, lse, am, bm


def bwd_blockskip(head: Head, h: torch.Tensor, targets: torch.Tensor, lse: torch.Tensor,
                  dlogp: torch.Tensor, block_max: torch.Tensor, eps: float,
                  mask: torch.Tensor | None = None, *, workspace: torch.Tensor | None = None,
                  stream=None) -> torch.Tensor:
    """Approximate dh [M, H] float32: the blocks below eps (see
    qhead_bwd_blockskip) are left out of both backward phases."""
    M = _check_h(head, h)
    dev = h.device
    targets = _targets(targets, M, dev, required=True)
    mask = _mask(mask, M, dev)
    lse, dlogp = _f32("lse", lse, M, dev), _f32("dlogp", dlogp, M, dev)
    nvt = (head.V + 255) // 256
    if (not isinstance(block_max, torch.Tensor) or block_max.dtype != torch.float32
            or tuple(block_max.shape) != (M, nvt) or not block_max.is_contiguous()
            or block_max.device != dev):
        raise ValueError(f"block_max must be a contiguous float32 [{M}, {nvt}] tensor on {dev}")
    _usable(dev, stream, workspace)
    dh = _out((M, head.H), torch.float32, dev, stream)
    _reads(stream, head, h, targets, lse, dlogp, block_max, mask, workspace)
    if workspace is None:
        workspace = _scratch(_ws_size("qhead_bwd_blockskip_workspace", head, M), dev, stream)
    _check(lib().qhead_bwd_blockskip(ctypes.byref(head.c()), h.data_ptr(), M, targets.data_ptr(),
                                     _ptr(mask), lse.data_ptr(), dlogp.data_ptr(),
                                     block_max.data_ptr(), float(eps), dh.data_ptr(),
                                     workspace.data_ptr(), workspace.numel(), _stream(stream, dev)))
    return dh


def bwd_filter(head: Head, h: torch.Tensor, targets: torch.Tensor, lse: torch.Tensor,
               dlogp: torch.Tensor, eps: float, mask: torch.Tensor | None = None, *,
               want_cold: bool = False, workspace: torch.Tensor | None = None, stream=None):
    """(dh [M, H] float32, cold or None): the approximate dh of the
    coefficient filter (see qhead_bwd_filter) and, when asked for, its block
    decisions uint8 [ceil(M / 32), ceil(V / 32)] (1 = cold)."""
    M = _check_h(head, h)
    dev = h.device
    targets = _targets(targets, M, dev, required=True)
    mask = _mask(mask, M, dev)
    lse, dlogp = _f32("lse", lse, M, dev), _f32("dlogp", dlogp, M, dev)
    _usable(dev, stream, workspace)
    dh = _out((M, head.H), torch.float32, dev, stream)
    cold = _out(((M + 31) // 32, (head.V + 31) // 32), torch.uint8, dev, stream) if want_cold else None
    _reads(stream, head, h, targets, lse, dlogp, mask, workspace)
    if workspace is None:
        workspace = _scratch(_ws_size("qhead_bwd_filter_workspace", head, M), dev, stream)
    _check(lib().qhead_bwd_filter(ctypes.byref(head.c()), h.data_ptr(), M, targets.data_ptr(),
                                  _ptr(mask), lse.data_ptr(), dlogp.data_ptr(), float(eps),
                                  dh.data_ptr(), _ptr(cold), workspace.data_ptr(),
                                  workspace.numel(), _stream(stream, dev)))
    return dh, cold


def verify(head: Head, h: torch.Tensor, W: int, draft: torch.Tensor | None,
           mask: torch.Tensor | None = None, *, want_lse: bool = False,
           workspace: torch.Tensor | None = None, stream=None):
    """Verify B = h.shape[0] / W windows of W = gamma + 1 rows against their
    drafts (int32 [B, W - 1]).  Returns (n_accept [B], next_token [B],
    argmax [B * W], lse [B * W] or None), all on the device."""
    M = _check_h(head, h, "[B * W, H]")
    if W < 1 or M % W:
        raise ValueError("the row count must be a multiple of W >= 1")
    B = M // W
    if draft is not None and (draft.dtype != torch.int32 or not draft.is_contiguous()
                              or draft.numel() != B * (W - 1)):
        raise ValueError("draft must be a contiguous int32 [B, W - 1] tensor")
    dev = h.device
    if draft is not None and draft.device != dev:
        raise ValueError(f"draft is on {draft.device}, h on {dev}")
    mask = _mask(mask, M, dev)
    _usable(dev, stream, workspace)
    am = _out(M, torch.int32, dev, stream)
    lse = _out(M, torch.float32, dev, stream) if want_lse else None
    n_acc = _out(B, torch.int32, dev, stream)
    nxt = _out(B, torch.int32, dev, stream)
    _reads(stream, head, h, draft, mask, workspace)
    if workspace is None:
        workspace = _scratch(fwd_workspace(head, M), dev, stream)
    _check(lib().qhead_verify(ctypes.byref(head.c()), h.data_ptr(), B, W, _ptr(draft),
                              _ptr(mask), _ptr(lse), am.data_ptr(), n_acc.data_ptr(),
                              nxt.data_ptr(), workspace.data_ptr(), workspace.numel(),
                              _stream(stream, dev)))
    return n_acc, nxt, am, lse


# ------------------------------------------------- the operators beside the head

def _check_matrix(name: str, t: torch.Tensor, dev, contiguous: bool = True):
    """A float matrix on `dev` whose rows are contiguous (rows too, unless
    contiguous is off: then their stride may exceed the width)."""
    if not isinstance(t, torch.Tensor) or t.dtype not in _SB_CODE or t.dim() != 2:
        raise ValueError(f"{name} must be a float16, bfloat16 or float32 matrix")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if t.is_contiguous():
        return
    if contiguous:
        raise ValueError(f"{name} must be contiguous")
    if t.shape[1] > 1 and t.stride(1) != 1 or t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        raise ValueError(f"{name} must have contiguous rows that do not overlap")


def _row_stride(t: torch.Tensor, M: int, H: int) -> int:
    return H if M <= 1 else max(t.stride(0), H)


def _tokens(head: Head, t: torch.Tensor) -> int:
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or t.dim() != 1 \
            or not t.is_contiguous():
        raise ValueError("tokens must be a contiguous int32 vector")
    if t.device != head.wq.device:
        raise ValueError(f"tokens are on {t.device} but the head is on {head.wq.device}")
    return int(t.shape[0])


def _out_code(dtype, name: str = "out_dtype") -> int:
    code = _SB_CODE.get(dtype)
    if code is None:
        raise ValueError(f"{name} must be float16, bfloat16 or float32")
    return code


def _size(n: int) -> int:
    if n == ctypes.c_size_t(-1).value:
        raise QheadError(QHEAD_EINVAL, last_error())
    return int(n)


def embed(head: Head, tokens: torch.Tensor, scale: float = 1.0, mask: torch.Tensor | None = None, *,
          out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """[M, H] rows of the dequantized table, times scale: zeros where the mask
    is off, NaN where a token lies outside [0, V)."""
    M = _tokens(head, tokens)
    dev = tokens.device
    if mask is not None:
        mask = _mask(mask, M, dev)
    code = _out_code(out_dtype)
    c = head.c()
    _usable(dev, stream)
    out = _out((M, c.H), out_dtype, dev, stream)
    _reads(stream, head, tokens, mask)
    _check(lib().qhead_embed(ctypes.byref(c), tokens.data_ptr(), M, _ptr(mask), scale,
                             out.data_ptr(), code, _stream(stream, dev)))
    return out


def embed_bwd(head: Head, tokens: torch.Tensor, dout: torch.Tensor, scale: float = 1.0,
              mask: torch.Tensor | None = None, *, dw: torch.Tensor | None = None,
              workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The gradient of embed() with respect to the dequantized table, float32
    [V, H]: added into dw (and dw returned) when it is given -- bwd_dw()'s, for
    a tied table -- else into a new tensor whose other rows are 0."""
    M = _tokens(head, tokens)
    dev = tokens.device
    mask = _mask(mask, M, dev)
    _check_matrix("dout", dout, dev)
    if tuple(dout.shape) != (M, head.H):
        raise ValueError(f"dout must have shape [{M}, {head.H}], got {list(dout.shape)}")
    add = dw is not None
    if add and (not isinstance(dw, torch.Tensor) or dw.dtype != torch.float32 or dw.device != dev
                or tuple(dw.shape) != (head.V, head.H) or not dw.is_contiguous()):
        raise ValueError(f"dw must be a contiguous float32 [{head.V}, {head.H}] tensor on {dev}")
    _usable(dev, stream, workspace)
    if not add:
        dw = _out((head.V, head.H), torch.float32, dev, stream)
    c = head.c()
    _reads(stream, None, tokens, dout, mask, dw if add else None, workspace)
    if workspace is None:
        workspace = _scratch(_size(lib().qhead_embed_bwd_workspace(ctypes.byref(c), M)), dev,
                             stream)
    _check(lib().qhead_embed_bwd(ctypes.byref(c), tokens.data_ptr(), M, _ptr(mask), scale,
                                 dout.data_ptr(), _SB_CODE[dout.dtype], dw.data_ptr(), int(add),
                                 workspace.data_ptr(), workspace.numel(), _stream(stream, dev)))
    return dw


def _check_param(name: str, t: torch.Tensor | None, H: int, dev, dtype=None):
    if t is None:
        return
    if not isinstance(t, torch.Tensor) or t.dtype not in _SB_CODE or t.dim() != 1 \
            or t.shape[0] != H or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float16, bfloat16 or float32 [{H}] tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must have weight's type")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, x on {dev}")


def layer_norm(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None,
               eps: float = 1e-6, *, center: bool = True, out_dtype: torch.dtype = torch.bfloat16,
               stream=None):
    """(y [M, H] of out_dtype, mean [M] or None, rstd [M]): the layer norm of
    x's rows (any float type; the row stride may exceed H), or with center off
    its root-mean-square form.  y in bfloat16 is the head's h."""
    if not isinstance(x, torch.Tensor):
        raise ValueError("x must be a torch tensor")
    dev = x.device
    _check_matrix("x", x, dev, contiguous=False)
    M, H = x.shape
    if weight is None:
        raise ValueError("weight is required")
    _check_param("weight", weight, H, dev)
    _check_param("bias", bias, H, dev, weight.dtype)
    code = _out_code(out_dtype)
    _usable(dev, stream)
    y = _out((M, H), out_dtype, dev, stream)
    rstd = _out(M, torch.float32, dev, stream)
    mean = _out(M, torch.float32, dev, stream) if center else None
    _reads(stream, None, x, weight, bias)
    _check(lib().qhead_layer_norm(x.data_ptr(), _SB_CODE[x.dtype], _row_stride(x, M, H), M, H,
                                  weight.data_ptr(), _ptr(bias), _SB_CODE[weight.dtype], eps,
                                  int(center), y.data_ptr(), code, _ptr(mean), rstd.data_ptr(),
                                  _stream(stream, dev)))
    return y, mean, rstd


def layer_norm_bwd(x: torch.Tensor, weight: torch.Tensor, mean: torch.Tensor | None,
                   rstd: torch.Tensor, dy: torch.Tensor, *, want_dbias: bool = True,
                   workspace: torch.Tensor | None = None, stream=None):
    """(dx [M, H] of x's type, dweight [H] float32, dbias [H] float32 or None)
    for dy = d/dy (any float type: bwd()'s float32 dh as it is); mean and rstd
    are layer_norm()'s (mean None: the uncentred form)."""
    if not isinstance(x, torch.Tensor):
        raise ValueError("x must be a torch tensor")
    dev = x.device
    _check_matrix("x", x, dev, contiguous=False)
    M, H = x.shape
    _check_matrix("dy", dy, dev, contiguous=False)
    if dy.shape != x.shape:
        raise ValueError(f"dy must have shape [{M}, {H}], got {list(dy.shape)}")
    if weight is None:
        raise ValueError("weight is required")
    _check_param("weight", weight, H, dev)
    mean = _check_vec("mean", mean, M, (torch.float32,), dev, required=False)
    rstd = _f32("rstd", rstd, M, dev)
    _usable(dev, stream, workspace)
    dx = _out((M, H), x.dtype, dev, stream)
    dw = _out(H, torch.float32, dev, stream)
    db = _out(H, torch.float32, dev, stream) if want_dbias else None
    _reads(stream, None, x, weight, mean, rstd, dy, workspace)
    if workspace is None:
        workspace = _scratch(_size(lib().qhead_layer_norm_bwd_workspace(M, H)), dev, stream)
    _check(lib().qhead_layer_norm_bwd(x.data_ptr(), _SB_CODE[x.dtype], _row_stride(x, M, H), M, H,
                                      weight.data_ptr(), _SB_CODE[weight.dtype], _ptr(mean),
                                      rstd.data_ptr(), dy.data_ptr(), _SB_CODE[dy.dtype],
                                      _row_stride(dy, M, H), dx.data_ptr(), dw.data_ptr(), _ptr(db),
                                      workspace.data_ptr(), workspace.numel(), _stream(stream, dev)))
    return dx, dw, db


def _check_teacher(ids: torch.Tensor, tlogits: torch.Tensor, M: int, dev) -> int:
    if not isinstance(ids, torch.Tensor) or ids.dtype != torch.int32 or ids.dim() != 2 \
            or not ids.is_contiguous() or ids.shape[0] != M or ids.device != dev:
        raise ValueError(f"ids must be a contiguous int32 [{M}, K] tensor on {dev}")
    _check_matrix("tlogits", tlogits, dev)
    shape = ids.shape
    if tlogits.shape != shape:
        raise ValueError(f"tlogits must have ids' shape {list(shape)}, got {list(tlogits.shape)}")
    return shape[1]


_distill_sizes: dict = {}  # (query, device, head's shape, M, K) -> its answer


def _distill_size(query: str, c: CHead, M: int, K: int, dev) -> int:
    """A size that the library gives for a shape, asked for once (the queries are a
    tenth of a small step's time)."""
    key = (query, dev, c.V, c.H, c.bits, c.group, c.sb_dtype, M, K)
    n = _distill_sizes.get(key)
    if n is None:
        n = getattr(lib(), query)(ctypes.byref(c), M, K)
        if n in (-1, ctypes.c_size_t(-1).value):
            raise QheadError(QHEAD_EINVAL, last_error())
        if len(_distill_sizes) >= 1024:
            _distill_sizes.clear()
        _distill_sizes[key] = n
    return n


def distill_fwd(head: Head, h: torch.Tensor, ids: torch.Tensor, tlogits: torch.Tensor,
                temperature: float = 1.0, mask: torch.Tensor | None = None, *,
                workspace: torch.Tensor | None = None, stream=None):
    """(loss [M], lse [M], kept [M, ...]), float32: each row's cross entropy of
    the head against a teacher's top logits (ids int32 [M, K], negative =
    padding; tlogits [M, K]), less the teacher's entropy; see
    qhead_distill_fwd.  lse is of the logits over the temperature; kept begins
    with the listed tokens' exact logits; distill_bwd() takes both."""
    M = _check_h(head, h)
    dev = h.device
    K = _check_teacher(ids, tlogits, M, dev)
    mask = _mask(mask, M, dev)
    _usable(dev, stream, workspace)
    loss = _out(M, torch.float32, dev, stream)
    lse = _out(M, torch.float32, dev, stream)
    c = head.c()
    kept = _out((M, _distill_size("qhead_distill_kept", c, M, K, dev)), torch.float32, dev, stream)
    _reads(stream, head, h, ids, tlogits, mask, workspace)
    if workspace is None:
        n = _distill_size("qhead_distill_fwd_workspace", c, M, K, dev)
        workspace = _scratch(n, dev, stream)
    _check(lib().qhead_distill_fwd(ctypes.byref(c), h.data_ptr(), M, ids.data_ptr(),
                                   tlogits.data_ptr(), _SB_CODE[tlogits.dtype], K, temperature,
                                   _ptr(mask), loss.data_ptr(), lse.data_ptr(), kept.data_ptr(),
                                   workspace.data_ptr(), workspace.numel(), _stream(stream, dev)))
    return loss, lse, kept


def distill_bwd(head: Head, h: torch.Tensor, ids: torch.Tensor, tlogits: torch.Tensor,
                kept: torch.Tensor, lse: torch.Tensor, dloss: torch.Tensor, temperature: float = 1.0,
                mask: torch.Tensor | None = None, *, workspace: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
    """dh [M, H] bfloat16 of sum_m dloss[m] * loss[m], from distill_fwd()'s kept
    and lse."""
    M = _check_h(head, h)
    dev = h.device
    K = _check_teacher(ids, tlogits, M, dev)
    mask = _mask(mask, M, dev)
    lse, dloss = _f32("lse", lse, M, dev), _f32("dloss", dloss, M, dev)
    _check_matrix("kept", kept, dev)
    c = head.c()
    cols = _distill_size("qhead_distill_kept", c, M, K, dev)
    if kept.dtype != torch.float32 or kept.shape != (M, cols):
        raise ValueError(f"kept must be a float32 [{M}, {cols}] tensor")
    _usable(dev, stream, workspace)
    dh = _out(h.shape, h.dtype, dev, stream)
    _reads(stream, head, h, ids, tlogits, kept, lse, dloss, mask, workspace)
    if workspace is None:
        n = _distill_size("qhead_distill_bwd_workspace", c, M, K, dev)
        workspace = _scratch(n, dev, stream)
    _check(lib().qhead_distill_bwd(ctypes.byref(c), h.data_ptr(), M, ids.data_ptr(),
                                   tlogits.data_ptr(), _SB_CODE[tlogits.dtype], K, temperature,
                                   _ptr(mask), kept.data_ptr(), lse.data_ptr(), dloss.data_ptr(),
                                   dh.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                   _stream(stream, dev)))
    return dh


# ------------------------------------------------- the block between norm and head

QHEAD_E4M3 = 3
ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
_HALF_CODE = {torch.float16: QHEAD_SB_F16, torch.bfloat16: QHEAD_SB_BF16}
_OPERAND_CODE = {**_HALF_CODE, torch.float8_e4m3fn: QHEAD_E4M3}


def _act_code(act: str) -> int:
    code = ACTIVATIONS.get(act)
    if code is None:
        raise ValueError(f"act must be one of {', '.join(ACTIVATIONS)}, got {act!r}")
    return code


def _rows_of(name: str, t: torch.Tensor, n: int, K: int) -> int:
    """The row stride of a matrix [n, K] whose rows are contiguous."""
    if t.is_contiguous():
        return K
    if K > 1 and t.stride(1) != 1 or n > 1 and t.stride(0) < K:
        raise ValueError(f"{name} must have contiguous rows that do not overlap")
    return K if n <= 1 else max(t.stride(0), K)


def _check_operands(x: torch.Tensor, weight: torch.Tensor, codes) -> tuple:
    """x [M, K] and weight [N, K], of one of the types of `codes`: what the library's
    calls and queries take of them (address, type, row stride, M, K, address, row
    stride, N)."""
    if not isinstance(x, torch.Tensor) or not isinstance(weight, torch.Tensor):
        raise ValueError("x and weight must be torch tensors")
    dtype = x.dtype
    code = codes.get(dtype)
    if code is None or weight.dtype != dtype:
        names = ", ".join(str(t).replace("torch.", "") for t in codes)
        raise ValueError(f"x and weight must share one type of {names}, got {dtype} and {weight.dtype}")
    xs, ws = x.shape, weight.shape
    if len(xs) != 2 or len(ws) != 2 or xs[1] != ws[1]:
        raise ValueError(f"x must be [M, K] and weight [N, K], got {list(xs)} and {list(ws)}")
    if weight.device != x.device:
        raise ValueError(f"weight is on {weight.device}, x on {x.device}")
    (M, K), N = xs, ws[0]
    return x.data_ptr(), code, _rows_of("x", x, M, K), M, K, weight.data_ptr(), _rows_of("weight", weight, N, K), N


_linear_sizes: dict = {}  # (query, device, what the operands' place and shape decide) -> its answer


def _linear_size(query: str, place: tuple, dev) -> int:
    """The workspace that the library asks for, asked for once a shape and alignment."""
    p, code, ldx, M, K, q, ldw, N = place
    key = (query, dev, p & 15, code, ldx, M, K, q & 15, ldw, N)
    n = _linear_sizes.get(key)
    if n is None:
        n = _size(getattr(lib(), query)(*place))
        if len(_linear_sizes) >= 1024:
            _linear_sizes.clear()
        _linear_sizes[key] = n
    return n


def linear(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None, act: str = "none",
           residual: torch.Tensor | None = None, *, x_scale: torch.Tensor | None = None,
           w_scale: torch.Tensor | None = None, out_dtype: torch.dtype | None = None, want_pre: bool = False,
           workspace: torch.Tensor | None = None, stream=None):
    """y [M, N] = act(x @ weight.T + bias) + residual, of out_dtype (x's, or
    bfloat16 for 8-bit operands, if not given); see qhead_linear.  x [M, K] and
    weight [N, K] in bfloat16 or float16, or in float8_e4m3fn with a float32
    scale for each row of both (norm_8bit()'s codes and scale for x).  With
    want_pre (y, pre): what linear_bwd() takes."""
    place = _check_operands(x, weight, _OPERAND_CODE)
    code, M, N, dev = place[1], place[3], place[7], x.device
    a = _act_code(act)
    if (code == QHEAD_E4M3) != (x_scale is not None and w_scale is not None) \
            or (x_scale is None) != (w_scale is None):
        raise ValueError("x_scale and w_scale belong to float8_e4m3fn operands, which need both")
    if x_scale is not None:
        x_scale, w_scale = _f32("x_scale", x_scale, M, dev), _f32("w_scale", w_scale, N, dev)
    b = b_code = r = r_code = None
    if bias is not None:
        _check_param("bias", bias, N, dev)
        b, b_code = bias.data_ptr(), _SB_CODE[bias.dtype]
    ldr = N
    if residual is not None:
        _check_matrix("residual", residual, dev, contiguous=False)
        if residual.shape != (M, N):
            raise ValueError(f"residual must have shape [{M}, {N}], got {list(residual.shape)}")
        r, r_code, ldr = residual.data_ptr(), _SB_CODE[residual.dtype], _row_stride(residual, M, N)
    if out_dtype is None:
        out_dtype = torch.bfloat16 if code == QHEAD_E4M3 else x.dtype
    out = _out_code(out_dtype)
    _usable(dev, stream, workspace)
    y = _out((M, N), out_dtype, dev, stream)
    pre = _out((M, N), torch.float16, dev, stream) if want_pre else None
    _reads(stream, None, x, weight, x_scale, w_scale, bias, residual, workspace)
    if workspace is None:
        n = _linear_size("qhead_linear_workspace", place, dev)
        workspace = _scratch(n, dev, stream) if n else None
    _check(lib().qhead_linear(*place, _ptr(x_scale), _ptr(w_scale), b, b_code or 0, a, r, r_code or 0, ldr,
                              y.data_ptr(), out, _ptr(pre), _ptr(workspace),
                              0 if workspace is None else workspace.numel(), _stream(stream, dev)))
    return (y, pre) if want_pre else y


def linear_bwd(x: torch.Tensor, weight: torch.Tensor, dy: torch.Tensor, pre: torch.Tensor | None = None,
               act: str = "none", dbias_dtype: torch.dtype | None = None, *, want_dx: bool = True,
               want_dw: bool = True, want_dbias: bool = True, workspace: torch.Tensor | None = None, stream=None):
    """(dx [M, K], dweight [N, K], dbias [N]), None where not wanted, for dy = d/dy
    (any float type) and linear()'s pre (act "none" needs none): dx and dweight of
    x's type, dbias of dbias_dtype (if not given, float32 where dy is and else x's).
    The residual's gradient is dy."""
    place = _check_operands(x, weight, _HALF_CODE)
    M, K, N, dev = place[3], place[4], place[7], x.device
    a = _act_code(act)
    _check_matrix("dy", dy, dev, contiguous=False)
    if dy.shape != (M, N):
        raise ValueError(f"dy must have shape [{M}, {N}], got {list(dy.shape)}")
    if a and (not isinstance(pre, torch.Tensor) or pre.dtype != torch.float16 or pre.shape != (M, N)
              or not pre.is_contiguous() or pre.device != dev):
        raise ValueError(f"pre must be a contiguous float16 [{M}, {N}] tensor on {dev}")
    if dbias_dtype is None:
        dbias_dtype = dy.dtype if dy.dtype == torch.float32 else x.dtype
    db_code = _out_code(dbias_dtype, "dbias_dtype")
    _usable(dev, stream, workspace)
    dx = _out((M, K), x.dtype, dev, stream) if want_dx else None
    dw = _out((N, K), x.dtype, dev, stream) if want_dw else None
    db = _out(N, dbias_dtype, dev, stream) if want_dbias else None
    _reads(stream, None, x, weight, dy, pre, workspace)
    if workspace is None:
        workspace = _scratch(_linear_size("qhead_linear_bwd_workspace", place, dev), dev, stream)
    _check(lib().qhead_linear_bwd_dbias(*place, dy.data_ptr(), _SB_CODE[dy.dtype], _row_stride(dy, M, N),
                                        _ptr(pre) if a else None, a, _ptr(dx), _ptr(dw), _ptr(db), db_code,
                                        workspace.data_ptr(), workspace.numel(), _stream(stream, dev)))
    return dx, dw, db


def _check_added(x, residual, weight, bias):
    """The operands of a norm behind an addition (residual None: of the norm alone)."""
    if not isinstance(x, torch.Tensor):
        raise ValueError("x must be a torch tensor")
    dev = x.device
    _check_matrix("x", x, dev, contiguous=False)
    M, H = x.shape
    if residual is not None:
        _check_matrix("residual", residual, dev, contiguous=False)
        if residual.shape != x.shape:
            raise ValueError(f"residual must have x's shape [{M}, {H}], got {list(residual.shape)}")
    if weight is None:
        raise ValueError("weight is required")
    _check_param("weight", weight, H, dev)
    _check_param("bias", bias, H, dev, weight.dtype)
    return dev, M, H


def _added(x, residual, weight, bias, eps, center, total, M, H):
    """The arguments that both forms of the norm behind an addition begin with."""
    return (x.data_ptr(), _SB_CODE[x.dtype], _row_stride(x, M, H), _ptr(residual),
            0 if residual is None else _SB_CODE[residual.dtype],
            H if residual is None else _row_stride(residual, M, H), M, H, weight.data_ptr(), _ptr(bias),
            _SB_CODE[weight.dtype], eps, int(center), _ptr(total))


def add_norm(x: torch.Tensor, residual: torch.Tensor, weight: torch.Tensor,
             bias: torch.Tensor | None = None, eps: float = 1e-6, *, center: bool = True,
             out_dtype: torch.dtype = torch.bfloat16, stream=None):
    """(y [M, H] of out_dtype, total [M, H] of residual's type, mean [M] or None,
    rstd [M]): total = x + residual, and layer_norm() of it, taken before it is
    rounded.  Both may have any float type and a row stride above H."""
    dev, M, H = _check_added(x, residual, weight, bias)
    if residual is None:
        raise ValueError("residual is required")
    code = _out_code(out_dtype)
    _usable(dev, stream)
    y = _out((M, H), out_dtype, dev, stream)
    total = _out((M, H), residual.dtype, dev, stream)
    rstd = _out(M, torch.float32, dev, stream)
    mean = _out(M, torch.float32, dev, stream) if center else None
    _reads(stream, None, x, residual, weight, bias)
    _check(lib().qhead_add_norm(*_added(x, residual, weight, bias, eps, center, total, M, H), y.data_ptr(), code,
                                _ptr(mean), rstd.data_ptr(), _stream(stream, dev)))
    return y, total, mean, rstd


def norm_8bit(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None, eps: float = 1e-6, *,
              residual: torch.Tensor | None = None, center: bool = True, stream=None):
    """(codes float8_e4m3fn [M, H], scale float32 [M], total or None): the norm of
    x (of x + residual, which total then holds) as 8-bit codes with a scale for each
    row, codes * scale = y: linear()'s x and x_scale."""
    dev, M, H = _check_added(x, residual, weight, bias)
    _usable(dev, stream)
    codes = _out((M, H), torch.float8_e4m3fn, dev, stream)
    scale = _out(M, torch.float32, dev, stream)
    total = None if residual is None else _out((M, H), residual.dtype, dev, stream)
    _reads(stream, None, x, residual, weight, bias)
    _check(lib().qhead_norm_8bit(*_added(x, residual, weight, bias, eps, center, total, M, H), codes.data_ptr(),
                                 scale.data_ptr(), _stream(stream, dev)))
    return codes, scale, total


def add_norm_bwd(total: torch.Tensor, weight: torch.Tensor, mean: torch.Tensor | None, rstd: torch.Tensor,
                 dy: torch.Tensor, dtotal: torch.Tensor | None = None, *, want_dbias: bool = True,
                 workspace: torch.Tensor | None = None, stream=None):
    """(dx [M, H] of total's type, dweight [H] float32, dbias [H] float32 or None)
    for dy = d/dy and dtotal = d/dtotal (total's type; None: nothing arrives
    there).  dx is the gradient of x and of the residual; total, mean and rstd are
    add_norm()'s."""
    if dtotal is None:
        return layer_norm_bwd(total, weight, mean, rstd, dy, want_dbias=want_dbias, workspace=workspace,
                              stream=stream)
    if not isinstance(total, torch.Tensor):
        raise ValueError("total must be a torch tensor")
    dev = total.device
    _check_matrix("total", total, dev, contiguous=False)
    M, H = total.shape
    for name, t in (("dy", dy), ("dtotal", dtotal)):
        _check_matrix(name, t, dev, contiguous=False)
        if t.shape != total.shape:
            raise ValueError(f"{name} must have shape [{M}, {H}], got {list(t.shape)}")
    if dtotal.dtype != total.dtype:
        raise ValueError("dtotal must have total's type")
    if weight is None:
        raise ValueError("weight is required")
    _check_param("weight", weight, H, dev)
    mean = _check_vec("mean", mean, M, (torch.float32,), dev, required=False)
    rstd = _f32("rstd", rstd, M, dev)
    _usable(dev, stream, workspace)
    dx = _out((M, H), total.dtype, dev, stream)
    dw = _out(H, torch.float32, dev, stream)
    db = _out(H, torch.float32, dev, stream) if want_dbias else None
    _reads(stream, None, total, weight, mean, rstd, dy, dtotal, workspace)
    if workspace is None:
        workspace = _scratch(_size(lib().qhead_layer_norm_bwd_workspace(M, H)), dev, stream)
    _check(lib().qhead_add_norm_bwd(total.data_ptr(), _SB_CODE[total.dtype], _row_stride(total, M, H), M, H,
                                    weight.data_ptr(), _SB_CODE[weight.dtype], _ptr(mean), rstd.data_ptr(),
                                    dy.data_ptr(), _SB_CODE[dy.dtype], _row_stride(dy, M, H), dtotal.data_ptr(),
                                    _row_stride(dtotal, M, H), dx.data_ptr(), dw.data_ptr(), _ptr(db),
                                    workspace.data_ptr(), workspace.numel(), _stream(stream, dev)))
    return dx, dw, db


# ------------------------------------------------- the gradients of a whole model

def _grad_list(name: str, tensors, dev=None):
    """(tensors as a list, their device, addresses, sizes and type codes as C arrays)."""
    ts = list(tensors)
    n = len(ts)
    codes = [_SB_CODE.get(t.dtype, -1) if isinstance(t, torch.Tensor) else -1 for t in ts]
    if -1 in codes or not all([t.is_contiguous() for t in ts]):
        raise ValueError(f"{name} must be contiguous float16, bfloat16 or float32 tensors")
    if ts and dev is None:
        dev = ts[0].device
    if len({t.get_device() for t in ts}) > 1 or ts and ts[0].device != dev:
        raise ValueError(f"{name} must be on one GPU{'' if dev is None else f', {dev}'}")
    return (ts, dev, array("Q", [t.data_ptr() for t in ts]), array("q", [t.numel() for t in ts]),
            array("i", codes))


def _at(a) -> int | None:
    return None if a is None else a.buffer_info()[0]


def grad_norm(tensors, *, workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The 2-norm over all elements of the tensors (contiguous, any float types, on
    one GPU), as a float32 scalar on the device."""
    ts, dev, ptrs, sizes, types = _grad_list("tensors", tensors)
    if not ts:
        raise ValueError("tensors is empty")
    _usable(dev, stream, workspace)
    norm = _out((), torch.float32, dev, stream)
    _reads(stream, None, *ts, workspace)
    if workspace is None:
        workspace = _scratch(_size(lib().qhead_grad_norm_workspace(len(ts))), dev, stream)
    _check(lib().qhead_grad_norm(_at(ptrs), _at(sizes), _at(types), len(ts), norm.data_ptr(), workspace.data_ptr(),
                                 workspace.numel(), _stream(stream, dev)))
    return norm


def clip_grads(tensors, max_norm: float, *, out=None, workspace: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """Scales the tensors by min(1, max_norm / (norm + 1e-6)) and returns
    grad_norm() of them as they were: in place, or into `out`, as many tensors of
    the same sizes and any float types (16-bit copies of float32 gradients, for
    example).  In place nothing is written when the norm is within max_norm."""
    ts, dev, ptrs, sizes, types = _grad_list("tensors", tensors)
    if not ts:
        raise ValueError("tensors is empty")
    os_, optrs, otypes = [], None, None
    if out is not None:
        os_, _, optrs, osizes, otypes = _grad_list("out", out, dev)
        if osizes != sizes:
            raise ValueError("out must hold as many elements as tensors, tensor by tensor")
    _usable(dev, stream, workspace)
    norm = _out((), torch.float32, dev, stream)
    _reads(stream, None, *ts, *os_, workspace)
    if workspace is None:
        workspace = _scratch(_size(lib().qhead_grad_norm_workspace(len(ts))), dev, stream)
    _check(lib().qhead_clip_grads(_at(ptrs), _at(sizes), _at(types), len(ts), max_norm, _at(optrs), _at(otypes),
                              norm.data_ptr(), workspace.data_ptr(), workspace.numel(), _stream(stream, dev)))
    # (written behind autograd's back: what it has saved of them is no longer theirs)
    torch.autograd.graph.increment_version([t for t in os_ or ts if not t.is_inference()])
    return norm
