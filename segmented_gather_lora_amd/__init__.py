"""Python binding of liblora_mi355x.so (segmented-gather multi-LoRA on MI355X).

Argument marshalling only: every step runs in the library's HIP kernels.
Torch tensors supply device memory and the current HIP stream.  The names
mirror the C ABI in include/lora_mi355x.h:

    lora_meta_bytes, lora_meta_bind, lora_prepare_meta, lora_shrink,
    lora_expand, lora_shrink_expand, lora_prepare_shrink_expand,
    lora_shrink_expand_noalloc, lora_linear, lora_linear_backward,
    lora_linear_workspace_bytes, lora_cross_entropy,
    lora_cross_entropy_backward, lora_cross_entropy_workspace_bytes,
    lora_mx_quantize, lora_mx_dequantize, lora_linear_mx,
    lora_linear_mx_backward, lora_linear_mx_workspace_bytes,
    lora_clip_gradients, lora_clip_gradients_workspace_bytes,
    lora_status_string, and the measurement aids
    lora_shrink_expand_launches, lora_prepare_meta_launches, lora_probe_read,
    lora_probe_empty

plus ``LoraMeta``, a holder that owns one device region sized by
``lora_meta_bytes`` (LoRAKernelMeta.make on the "lora_kernel_metadata" page)
and exposes its arrays as tensor views, and ``LoraGradients``, the tensors of a
training step's gradients as lora_clip_gradients takes them.

The library is loaded on the first call; that call raises ImportError if the
library has not been built (``python -m segmented_gather_lora_amd._build``):
there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import os
from operator import attrgetter
from typing import Optional, Sequence

from ._build import LIB as _LIB_PATH

LORA_OK = 0
LORA_ERR_NULL = -1
LORA_ERR_NUM_TOKENS = -2
LORA_ERR_SHAPE = -3
LORA_ERR_MAX_LORAS = -4
LORA_ERR_BUFFER = -5
LORA_ERR_ALIGN = -6
LORA_ERR_SLICES = -7
LORA_ERR_LAUNCH = -8
LORA_ERR_ID_RANGE = -9
LORA_ERR_SYNC = -10
LORA_ERR_SCRATCH = -11

LORA_MAX_LORAS = 1023
LORA_MAX_SLICES = 8
LORA_MAX_RANK = 128

LORA_BF16 = 0
LORA_F32 = 1

EXPORTED = ("lora_meta_bytes", "lora_meta_bind", "lora_prepare_meta", "lora_shrink",
            "lora_expand", "lora_shrink_expand", "lora_prepare_shrink_expand", "lora_shrink_expand_launches",
            "lora_prepare_meta_launches",
            "lora_status_string", "lora_probe_read", "lora_probe_empty", "lora_shrink_expand_noalloc",
            "lora_linear", "lora_linear_backward", "lora_linear_workspace_bytes",
            "lora_mx_quantize", "lora_mx_dequantize", "lora_linear_mx", "lora_linear_mx_backward",
            "lora_linear_mx_workspace_bytes", "lora_clip_gradients", "lora_clip_gradients_workspace_bytes",
            "lora_cross_entropy", "lora_cross_entropy_backward", "lora_cross_entropy_workspace_bytes")


class LoraError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s: %s (%d)" % (where, lora_status_string(status), status))


class lora_meta_t(ctypes.Structure):
    _fields_ = [
        ("token_lora_mapping", ctypes.c_void_p),
        ("token_indices_sorted", ctypes.c_void_p),
        ("active_lora_ids", ctypes.c_void_p),
        ("num_tokens_per_lora", ctypes.c_void_p),
        ("lora_token_start_loc", ctypes.c_void_p),
        ("no_lora_flag", ctypes.c_void_p),
        ("status", ctypes.c_void_p),
        ("sync", ctypes.c_void_p),
        ("host_no_lora", ctypes.c_void_p),
        ("max_loras", ctypes.c_int32),
        ("max_num_tokens", ctypes.c_int32),
        ("num_tokens", ctypes.c_int32),
    ]


def _load() -> ctypes.CDLL:
    if not os.path.exists(_LIB_PATH):
        raise ImportError("liblora_mi355x.so is not built (%s); run "
                          "`python -m segmented_gather_lora_amd._build`" % _LIB_PATH)
    lib = ctypes.CDLL(_LIB_PATH)
    P, i32, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
    lib.lora_meta_bytes.restype = ctypes.c_size_t
    lib.lora_meta_bytes.argtypes = [i32, i32]
    lib.lora_meta_bind.restype = i32
    lib.lora_meta_bind.argtypes = [P, ctypes.c_size_t, i32, i32, ctypes.POINTER(lora_meta_t)]
    lib.lora_prepare_meta.restype = i32
    lib.lora_prepare_meta.argtypes = [P, i32, ctypes.POINTER(lora_meta_t), P]
    lib.lora_shrink.restype = i32
    lib.lora_shrink.argtypes = [P, i64, i32, i32, P, i32, i32, P, ctypes.POINTER(lora_meta_t),
                                ctypes.c_float, P]
    lib.lora_expand.restype = i32
    lib.lora_expand.argtypes = [P, i32, i32, P, P, P, i32, P, i64, i32, i32,
                                ctypes.POINTER(lora_meta_t), P]
    lib.lora_shrink_expand.restype = i32
    lib.lora_shrink_expand.argtypes = [P, i64, i32, i32, P, P, P, P, i32, i32, P, P, i64, i32, i32,
                                       ctypes.POINTER(lora_meta_t), ctypes.c_float, P]
    lib.lora_shrink_expand_noalloc.restype = i32
    lib.lora_shrink_expand_noalloc.argtypes = [P, i64, i32, i32, P, P, P, P, i32, i32, P, i64, i32, i32,
                                               ctypes.POINTER(lora_meta_t), ctypes.c_float, P]
    lib.lora_prepare_shrink_expand.restype = i32
    lib.lora_prepare_shrink_expand.argtypes = [P, i32, P, i64, i32, P, P, P, P, i32, i32, P, P, i64, i32, i32,
                                               ctypes.POINTER(lora_meta_t), ctypes.c_float, P]
    lib.lora_shrink_expand_launches.restype = i32
    lib.lora_shrink_expand_launches.argtypes = [i32, i32, i32, i32, i32, i32]
    lib.lora_prepare_meta_launches.restype = i32
    lib.lora_prepare_meta_launches.argtypes = [i32, i32]
    Z = ctypes.c_size_t
    META = ctypes.POINTER(lora_meta_t)
    lib.lora_linear_workspace_bytes.restype = Z
    lib.lora_linear_workspace_bytes.argtypes = [i32, i32, i32, P, i32, i32, i32]
    lib.lora_linear.restype = i32
    lib.lora_linear.argtypes = [P, i64, i32, i32, P, i64, i32, P, P, P, P, P, i32, i32, P, P, i64, i32, META,
                                ctypes.c_float, P, Z, P]
    lib.lora_linear_backward.restype = i32
    lib.lora_linear_backward.argtypes = [P, i64, P, i64, i32, i32, P, i64, i32, P, P, P, i32, i32, P, P, P, i64, P, P,
                                         P, i32, META, ctypes.c_float, P, Z, P]
    lib.lora_cross_entropy_workspace_bytes.restype = Z
    lib.lora_cross_entropy_workspace_bytes.argtypes = [i32, i32, i32, i32]
    lib.lora_cross_entropy.restype = i32
    lib.lora_cross_entropy.argtypes = [P, i64, i32, i32, P, i64, i32, P, P, P, P, Z, P]
    lib.lora_cross_entropy_backward.restype = i32
    lib.lora_cross_entropy_backward.argtypes = [P, i64, i32, i32, P, i64, i32, P, P, P, P, i64, P, i64, P, Z, P]
    lib.lora_mx_quantize.restype = i32
    lib.lora_mx_quantize.argtypes = [P, i32, i64, i64, i32, P, i64, P, i64, P]
    lib.lora_mx_dequantize.restype = i32
    lib.lora_mx_dequantize.argtypes = [P, i64, P, i64, i64, i32, P, i32, i64, P]
    lib.lora_linear_mx_workspace_bytes.restype = Z
    lib.lora_linear_mx_workspace_bytes.argtypes = [i32, i32, i32, i32, P, i32, i32, i32]
    lib.lora_linear_mx.restype = i32
    lib.lora_linear_mx.argtypes = [P, i64, i32, i32, P, i64, P, i64, i32, P, P, P, P, P, i32, i32, P, P, i64, i32, META,
                                   ctypes.c_float, i32, P, Z, P]
    lib.lora_linear_mx_backward.restype = i32
    lib.lora_linear_mx_backward.argtypes = [P, i64, P, i64, i32, i32, P, i64, P, i64, i32, P, P, P, i32, i32, P, P, P,
                                            i64, P, P, P, i32, META, ctypes.c_float, P, Z, P]
    lib.lora_clip_gradients_workspace_bytes.restype = Z
    lib.lora_clip_gradients_workspace_bytes.argtypes = [P, P, i32, i32]
    lib.lora_clip_gradients.restype = i32
    lib.lora_clip_gradients.argtypes = [P, P, P, P, i32, i32, ctypes.c_double, P, P, Z, P]
    lib.lora_status_string.restype = ctypes.c_char_p
    lib.lora_status_string.argtypes = [i32]
    lib.lora_probe_read.restype = i32
    lib.lora_probe_read.argtypes = [P, ctypes.c_size_t, i32, P, P]
    lib.lora_probe_empty.restype = i32
    lib.lora_probe_empty.argtypes = [i32, P]
    return lib


_handle = None


def _lib() -> ctypes.CDLL:
    """The library, loaded on first use (the builder imports this package
    before any library exists); raises ImportError when it is not built."""
    global _handle
    if _handle is None:
        _handle = _load()
    return _handle


def __getattr__(name):
    if name == "lib":
        return _lib()
    raise AttributeError(name)


def lora_status_string(status: int) -> str:
    return _lib().lora_status_string(int(status)).decode()


def lora_shrink_expand_launches(num_tokens: int, max_loras: int, hidden: int, num_slices: int, rank: int,
                                with_prepare: bool) -> int:
    """Kernel launches of lora_shrink_expand / lora_prepare_shrink_expand for
    such a layer: 1 inside the one-launch range, else the separate calls'
    count (host only)."""
    st = _lib().lora_shrink_expand_launches(int(num_tokens), int(max_loras), int(hidden), int(num_slices),
                                            int(rank), 1 if with_prepare else 0)
    if st < 0:
        raise LoraError(st, "lora_shrink_expand_launches")
    return st


def lora_prepare_meta_launches(num_tokens: int, max_loras: int) -> int:
    """Kernel launches of lora_prepare_meta for a batch of this size (host only)."""
    st = _lib().lora_prepare_meta_launches(int(num_tokens), int(max_loras))
    if st < 0:
        raise LoraError(st, "lora_prepare_meta_launches")
    return st


def lora_probe_read(src, workgroups: int, sink, stream=None) -> None:
    """Measurement aid: one streaming read of every byte of the device tensor
    `src` by `workgroups` workgroups (sink: device float32 [>= workgroups])."""
    import torch
    _need(src.is_cuda and src.is_contiguous(), LORA_ERR_SHAPE, "lora_probe_read", "src must be a contiguous device tensor")
    _need(sink.is_cuda and sink.dtype == torch.float32 and sink.numel() >= workgroups, LORA_ERR_SHAPE,
          "lora_probe_read", "sink must be a device float32 tensor of >= workgroups elements")
    nbytes = src.numel() * src.element_size()
    _check(_lib().lora_probe_read(src.data_ptr(), nbytes, int(workgroups), sink.data_ptr(), _stream(stream)),
           "lora_probe_read")


def lora_probe_empty(workgroups: int, stream=None) -> None:
    """Measurement aid: one launch of `workgroups` workgroups that do nothing."""
    _check(_lib().lora_probe_empty(int(workgroups), _stream(stream)), "lora_probe_empty")


def _check(st: int, where: str) -> None:
    if st != LORA_OK:
        raise LoraError(st, where)


def _stream(stream) -> Optional[int]:
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    import torch
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _stream_on(stream, device, where: str) -> Optional[int]:
    """The stream for tensors on `device`, which has to be the current one: a kernel
    launched on another device would not reach them."""
    import torch
    current = torch.cuda.current_device()
    _need(device.index == current, LORA_ERR_SHAPE, where,
          "the tensors are on %s, the current device is cuda:%d" % (device, current))
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(current)


def _need(ok: bool, status: int, where: str, what: str) -> None:
    if not ok:
        raise LoraError(status, "%s: %s" % (where, what))


def _dev(t, dtype, meta, where: str, name: str) -> None:
    """A tensor the kernels read or write through a raw pointer: on meta's
    device, of the element type the C ABI takes, rows of unit element stride.
    What the C ABI cannot see is checked here, so that a host tensor or a
    wrong element type raises instead of reaching a kernel."""
    if not (t.is_cuda and t.device == meta.region.device):
        raise TypeError("%s: %s must be on %s (got %s)" % (where, name, meta.region.device, t.device))
    if t.dtype != dtype:
        raise TypeError("%s: %s must be %s (got %s)" % (where, name, dtype, t.dtype))
    _need(t.dim() == 0 or t.stride(-1) == 1 or t.numel() <= 1, LORA_ERR_SHAPE, where,
          "%s needs unit stride in its last dimension" % name)


def _weights(ts, meta, where: str, name: str, last: Optional[int], mid: Optional[Sequence] = None) -> None:
    """Per-slice weight tensors [>= max_loras][rows][last], contiguous: every
    id below max_loras indexes a whole matrix."""
    import torch
    for i, t in enumerate(ts):
        _dev(t, torch.bfloat16, meta, where, "%s[%d]" % (name, i))
        _need(t.dim() == 3 and t.is_contiguous(), LORA_ERR_SHAPE, where, "%s[%d] must be a contiguous 3-d tensor" % (name, i))
        _need(t.shape[0] >= meta.max_loras, LORA_ERR_SHAPE, where,
              "%s[%d] holds %d LoRAs, fewer than max_loras %d" % (name, i, t.shape[0], meta.max_loras))
        if last is not None:
            _need(t.shape[2] == last, LORA_ERR_SHAPE, where, "%s[%d] last dimension %d != %d" % (name, i, t.shape[2], last))
        if mid is not None:
            _need(t.shape[1] == mid[i], LORA_ERR_SHAPE, where, "%s[%d] rows %d != %d" % (name, i, t.shape[1], mid[i]))


def _bias(bias, widths, meta, where: str) -> None:
    import torch
    if bias is None:
        return
    _need(len(bias) == len(widths), LORA_ERR_SLICES, where, "one bias entry per slice")
    for i, t in enumerate(bias):
        if t is None:
            continue
        _dev(t, torch.bfloat16, meta, where, "bias[%d]" % i)
        _need(t.dim() == 2 and t.is_contiguous() and t.shape[0] >= meta.max_loras and t.shape[1] == widths[i],
              LORA_ERR_SHAPE, where, "bias[%d] must be contiguous [>= max_loras][%d]" % (i, widths[i]))


def _layer_checks(where: str, meta, n: int, x=None, lora_a=None, lora_b=None, bias=None, buf=None, y=None,
                  offset_start: int = 0) -> None:
    """The tensors of one layer call, checked before the library sees them.
    The token count is checked against the batch first, with the status the
    library gives it."""
    import torch
    _need(n == meta.num_tokens, LORA_ERR_NUM_TOKENS, where, "%d tokens, the batch has %d" % (n, meta.num_tokens))
    rank = None
    if buf is not None:
        _dev(buf, torch.float32, meta, where, "buf")
        _need(buf.dim() == 3 and buf.is_contiguous() and buf.shape[1] == n, LORA_ERR_SHAPE, where,
              "buf must be contiguous [S][%d][r]" % n)
        rank = buf.shape[2]
    if x is not None:
        _dev(x, torch.bfloat16, meta, where, "x")
        _need(x.dim() == 2 and x.shape[0] == n, LORA_ERR_SHAPE, where, "x must be [%d][H]" % n)
    if lora_a is not None:
        _weights(lora_a, meta, where, "lora_a", x.shape[1] if x is not None else None,
                 [rank] * len(lora_a) if rank is not None else None)
    if lora_b is not None:
        _weights(lora_b, meta, where, "lora_b", rank)
        widths = [int(t.shape[1]) for t in lora_b]
        _bias(bias, widths, meta, where)
        if y is not None:
            _dev(y, torch.bfloat16, meta, where, "y")
            _need(y.dim() == 2 and y.shape[0] >= n and y.shape[1] >= offset_start + sum(widths), LORA_ERR_SHAPE,
                  where, "y must be [>= %d][>= %d]" % (n, offset_start + sum(widths)))


def _ptr_array(tensors) -> ctypes.Array:
    return (ctypes.c_void_p * len(tensors))(*[None if t is None else t.data_ptr() for t in tensors])


def lora_meta_bytes(max_loras: int, max_num_tokens: int) -> int:
    return int(_lib().lora_meta_bytes(int(max_loras), int(max_num_tokens)))


def lora_meta_bind(dev_ptr: int, nbytes: int, max_loras: int, max_num_tokens: int) -> lora_meta_t:
    m = lora_meta_t()
    _check(_lib().lora_meta_bind(dev_ptr, nbytes, int(max_loras), int(max_num_tokens), ctypes.byref(m)),
           "lora_meta_bind")
    return m


class LoraMeta:
    """One device region holding a batch's kernel metadata (make() on the
    "lora_kernel_metadata" page: allocated once at maximum sizes, reused)."""

    def __init__(self, max_loras: int, max_num_tokens: int, device="cuda"):
        import torch
        nbytes = lora_meta_bytes(max_loras, max_num_tokens)
        if nbytes == 0:
            raise LoraError(LORA_ERR_MAX_LORAS, "lora_meta_bytes")
        # torch's caching allocator returns 512-byte aligned blocks; zero-filled
        # once so that the fused calls' counters start at zero
        self.region = torch.zeros(nbytes, dtype=torch.uint8, device=device)
        self.struct = lora_meta_bind(self.region.data_ptr(), nbytes, max_loras, max_num_tokens)
        self.max_loras, self.max_num_tokens = max_loras, max_num_tokens

    def _view(self, field: str, n: int):
        off = getattr(self.struct, field) - self.region.data_ptr()
        return self.region[off:off + 4 * n].view(__import__("torch").int32)

    @property
    def num_tokens(self) -> int:
        return self.struct.num_tokens

    def views(self) -> dict:
        """Tensor views of the metadata arrays (sizes as make() allocates)."""
        L, T = self.max_loras, self.max_num_tokens
        return dict(token_lora_mapping=self._view("token_lora_mapping", T),
                    token_indices_sorted=self._view("token_indices_sorted", T),
                    active_lora_ids=self._view("active_lora_ids", L + 1),
                    num_tokens_per_lora=self._view("num_tokens_per_lora", L + 1),
                    lora_token_start_loc=self._view("lora_token_start_loc", L + 2),
                    no_lora_flag=self._view("no_lora_flag", 1),
                    status=self._view("status", 1),
                    sync=self._view("sync", 1))


def lora_prepare_meta(mapping, meta: LoraMeta, stream=None) -> None:
    """mapping: int32 device tensor [N] of LoRA ids (-1 = none)."""
    import torch
    n = mapping.numel()
    if n:
        _dev(mapping, torch.int32, meta, "lora_prepare_meta", "mapping")
        _need(mapping.is_contiguous(), LORA_ERR_SHAPE, "lora_prepare_meta", "mapping must be contiguous")
    _check(_lib().lora_prepare_meta(mapping.data_ptr() if n else None, n, ctypes.byref(meta.struct),
                                 _stream(stream)), "lora_prepare_meta")


def lora_shrink(x, lora_a: Sequence, buf, meta: LoraMeta, scale: float, stream=None) -> None:
    """buf[i][t] += scale * x[t] @ lora_a[i][id_t]^T.
    x bf16 [N][H] (row stride x.stride(0)); lora_a: bf16 [max_loras][r][H] per
    slice; buf fp32 [S][N][r] contiguous."""
    n, h = x.shape
    r = lora_a[0].shape[1]
    _layer_checks("lora_shrink", meta, n, x=x, lora_a=lora_a, buf=buf)
    _need(buf.shape[0] == len(lora_a) and buf.shape[2] == r, LORA_ERR_SHAPE, "lora_shrink", "buf must be [S][N][r]")
    ptrs = _ptr_array(lora_a)
    _check(_lib().lora_shrink(x.data_ptr(), x.stride(0), n, h, ptrs, len(lora_a), r, buf.data_ptr(),
                           ctypes.byref(meta.struct), float(scale), _stream(stream)), "lora_shrink")


def lora_expand(buf, lora_b: Sequence, bias: Optional[Sequence], y, meta: LoraMeta,
                offset_start: int = 0, add_inputs: bool = True, stream=None) -> None:
    """y[t, off_i:off_i+O_i] = (add_inputs ? y : 0) + buf[i][t] @ lora_b[i][id_t]^T + bias[i][id_t].
    buf fp32 [S][N][r]; lora_b bf16 [max_loras][O_i][r] per slice; bias None
    or per slice (None | bf16 [max_loras][O_i]); y bf16 [N][ldy]."""
    s, n, r = buf.shape
    _layer_checks("lora_expand", meta, n, lora_b=lora_b, bias=bias, buf=buf, y=y, offset_start=offset_start)
    _need(len(lora_b) == s, LORA_ERR_SLICES, "lora_expand", "one lora_b entry per buf slice")
    widths = (ctypes.c_int * s)(*[int(t.shape[1]) for t in lora_b])
    bptrs = _ptr_array(lora_b)
    biasptrs = None if bias is None else _ptr_array(bias)
    _check(_lib().lora_expand(buf.data_ptr(), n, r, bptrs, biasptrs, widths, s, y.data_ptr(), y.stride(0),
                           int(offset_start), int(bool(add_inputs)), ctypes.byref(meta.struct),
                           _stream(stream)), "lora_expand")


def lora_shrink_expand(x, lora_a: Sequence, lora_b: Sequence, bias: Optional[Sequence], buf, y,
                       meta: LoraMeta, scale: float, offset_start: int = 0, add_inputs: bool = True,
                       stream=None) -> None:
    """add_lora_linear in one call (one launch for decode-like batches): buf
    is written as a fresh buffer, buf[i][t] = scale * x[t] @ lora_a[i][id_t]^T
    (its entry contents are ignored, rows of -1 tokens untouched), then y as
    lora_expand computes it.  Arguments as for the two calls."""
    n, h = x.shape
    s, _, r = buf.shape
    _layer_checks("lora_shrink_expand", meta, n, x=x, lora_a=lora_a, lora_b=lora_b, bias=bias, buf=buf, y=y,
                  offset_start=offset_start)
    _need(len(lora_a) == s and len(lora_b) == s, LORA_ERR_SLICES, "lora_shrink_expand", "one weight per buf slice")
    widths = (ctypes.c_int * s)(*[int(t.shape[1]) for t in lora_b])
    biasptrs = None if bias is None else _ptr_array(bias)
    _check(_lib().lora_shrink_expand(x.data_ptr(), x.stride(0), n, h, _ptr_array(lora_a), _ptr_array(lora_b),
                                  biasptrs, widths, s, r, buf.data_ptr(), y.data_ptr(), y.stride(0),
                                  int(offset_start), int(bool(add_inputs)), ctypes.byref(meta.struct),
                                  float(scale), _stream(stream)), "lora_shrink_expand")


def lora_shrink_expand_noalloc(x, lora_a: Sequence, lora_b: Sequence, bias: Optional[Sequence], y,
                               meta: LoraMeta, scale: float, offset_start: int = 0, add_inputs: bool = True,
                               stream=None) -> None:
    """lora_shrink_expand without a buffer argument, for callers that cannot
    allocate: the fp32 buffer is the library's static device array (at most
    8388608 floats, S * N * r; larger calls raise LORA_ERR_SCRATCH)."""
    n, h = x.shape
    r = lora_a[0].shape[1]
    s = len(lora_a)
    where = "lora_shrink_expand_noalloc"
    _layer_checks(where, meta, n, x=x, lora_a=lora_a, lora_b=lora_b, bias=bias, y=y, offset_start=offset_start)
    _need(len(lora_b) == s, LORA_ERR_SLICES, where, "one lora_b entry per lora_a entry")
    _need(all(int(t.shape[2]) == r for t in lora_b) and all(int(t.shape[1]) == r for t in lora_a),
          LORA_ERR_SHAPE, where, "lora_a and lora_b must share the rank")
    widths = (ctypes.c_int * s)(*[int(t.shape[1]) for t in lora_b])
    biasptrs = None if bias is None else _ptr_array(bias)
    _check(_lib().lora_shrink_expand_noalloc(x.data_ptr(), x.stride(0), n, h, _ptr_array(lora_a),
                                             _ptr_array(lora_b), biasptrs, widths, s, r, y.data_ptr(), y.stride(0),
                                             int(offset_start), int(bool(add_inputs)), ctypes.byref(meta.struct),
                                             float(scale), _stream(stream)), where)


def lora_prepare_shrink_expand(mapping, x, lora_a: Sequence, lora_b: Sequence, bias: Optional[Sequence], buf, y,
                               meta: LoraMeta, scale: float, offset_start: int = 0, add_inputs: bool = True,
                               stream=None) -> None:
    """lora_prepare_meta(mapping) then lora_shrink_expand (buf written as a
    fresh buffer), in one call (one launch for small decode-like batches)."""
    import torch
    n = mapping.numel()
    _, h = x.shape
    s, _, r = buf.shape
    where = "lora_prepare_shrink_expand"
    if n:
        _dev(mapping, torch.int32, meta, where, "mapping")
        _need(mapping.is_contiguous(), LORA_ERR_SHAPE, where, "mapping must be contiguous")
    _need(n <= meta.max_num_tokens, LORA_ERR_NUM_TOKENS, where, "more tokens than the metadata holds")
    saved = meta.struct.num_tokens
    meta.struct.num_tokens = n          # the layer is checked against the batch about to be prepared
    try:
        _layer_checks(where, meta, n, x=x, lora_a=lora_a, lora_b=lora_b, bias=bias, buf=buf, y=y,
                      offset_start=offset_start)
    finally:
        meta.struct.num_tokens = saved
    _need(len(lora_a) == s and len(lora_b) == s, LORA_ERR_SLICES, where, "one weight per buf slice")
    widths = (ctypes.c_int * s)(*[int(t.shape[1]) for t in lora_b])
    biasptrs = None if bias is None else _ptr_array(bias)
    _check(_lib().lora_prepare_shrink_expand(mapping.data_ptr() if n else None, n, x.data_ptr(), x.stride(0), h,
                                          _ptr_array(lora_a), _ptr_array(lora_b), biasptrs, widths, s, r,
                                          buf.data_ptr(), y.data_ptr(), y.stride(0), int(offset_start),
                                          int(bool(add_inputs)), ctypes.byref(meta.struct), float(scale),
                                          _stream(stream)), "lora_prepare_shrink_expand")


def _widths_array(widths) -> ctypes.Array:
    return (ctypes.c_int * len(widths))(*[int(w) for w in widths])


def lora_linear_workspace_bytes(num_tokens: int, max_loras: int, hidden: int, widths: Sequence, rank: int,
                                backward: bool = False) -> int:
    """Bytes of the workspace of lora_linear (backward: and of
    lora_linear_backward) for batches of up to num_tokens tokens: a uint8 device
    tensor, whose contents do not matter."""
    n = int(_lib().lora_linear_workspace_bytes(int(num_tokens), int(max_loras), int(hidden), _widths_array(widths),
                                               len(widths), int(rank), 1 if backward else 0))
    if n == 0:
        raise LoraError(LORA_ERR_SHAPE, "lora_linear_workspace_bytes")
    return n


def _workspace(t, device, where: str) -> None:
    import torch
    if not (t.is_cuda and t.device == device):
        raise TypeError("%s: workspace must be on %s (got %s)" % (where, device, t.device))
    if t.dtype != torch.uint8:
        raise TypeError("%s: workspace must be torch.uint8 (got %s)" % (where, t.dtype))
    _need(t.dim() == 1 and t.is_contiguous(), LORA_ERR_BUFFER, where, "workspace must be a contiguous 1-d tensor")


# The calls on the products accept what is plainly right in one look and go
# through the checks that name the fault only otherwise: for a few tokens the
# checks, spelled out, take longer than the kernels.

def _whole(t, dtype, device: int, shape) -> bool:
    return t.dtype is dtype and t.get_device() == device and t.shape == shape and t.is_contiguous()


def _matrix(t, dtype, device: int, shape) -> bool:
    """Rows of unit stride, any distance apart."""
    return t.dtype is dtype and t.get_device() == device and t.shape == shape and t.stride(1) == 1


def _linear_plain(meta, x, out: int, wide, lora_a, lora_b, bufs, widths, r: int, workspace, offset_start: int) -> bool:
    """All but the shared projection's matrix, which has `out` rows."""
    import torch
    n, h = x.shape
    device, loras, bf16 = meta.region.get_device(), lora_a[0].shape[0], torch.bfloat16
    if not (device >= 0 and n == meta.num_tokens and loras >= meta.max_loras and len(lora_a) == len(lora_b)
            and 0 <= offset_start and offset_start + sum(widths) <= out
            and _matrix(x, bf16, device, (n, h)) and _matrix(wide, bf16, device, (n, out)) and workspace.dtype is torch.uint8
            and workspace.get_device() == device and workspace.dim() == 1 and workspace.is_contiguous()):
        return False
    for t in bufs:
        if not _whole(t, torch.float32, device, (len(lora_a), n, r)):
            return False
    for a, b, width in zip(lora_a, lora_b, widths):
        if not (_whole(a, bf16, device, (loras, r, h)) and _whole(b, bf16, device, (loras, width, r))):
            return False
    return True


def _projection(where: str, meta, h: int, w) -> None:
    """The shared projection's matrix [out][hidden]."""
    import torch
    if _matrix(w, torch.bfloat16, meta.region.get_device(), (w.shape[0], h)) and w.is_cuda:
        return
    _dev(w, torch.bfloat16, meta, where, "w")
    _need(w.dim() == 2 and w.shape[1] == h, LORA_ERR_SHAPE, where, "w must be [out][%d]" % h)


def _projected(where: str, meta, out: int, wide, name: str, offset_start: int, widths) -> None:
    """The activations of the projection's output side (y or dy)."""
    import torch
    _dev(wide, torch.bfloat16, meta, where, name)
    _need(wide.dim() == 2 and wide.shape[0] == meta.num_tokens and wide.shape[1] == out, LORA_ERR_SHAPE, where,
          "%s must be [%d][%d]" % (name, meta.num_tokens, out))
    _need(offset_start >= 0 and offset_start + sum(widths) <= out, LORA_ERR_SHAPE, where,
          "the slices end past w's rows")


def _w_bias(t, out: int, meta, where: str) -> None:
    import torch
    if t is not None:
        _dev(t, torch.bfloat16, meta, where, "w_bias")
        _need(t.dim() == 1 and t.shape[0] == out, LORA_ERR_SHAPE, where, "w_bias must be [%d]" % out)


def _forward_checks(where: str, meta, x, out: int, y, lora_a, lora_b, buf, widths, r: int, workspace,
                    offset_start: int) -> None:
    s = len(lora_a)
    if not _linear_plain(meta, x, out, y, lora_a, lora_b, (buf,), widths, r, workspace, offset_start):
        _layer_checks(where, meta, x.shape[0], x=x, lora_a=lora_a, lora_b=lora_b, buf=buf, offset_start=offset_start)
        _need(len(lora_b) == s and buf.shape[0] == s, LORA_ERR_SLICES, where, "one weight per buf slice")
        _projected(where, meta, out, y, "y", offset_start, widths)
        _workspace(workspace, meta.region.device, where)


def lora_linear(x, w, w_bias, lora_a: Sequence, lora_b: Sequence, bias: Optional[Sequence], buf, y, meta: LoraMeta,
                scale: float, workspace, offset_start: int = 0, stream=None) -> None:
    """y = x @ w^T + w_bias, plus in slice i's columns buf[i][t] @ lora_b[i][id_t]^T
    + bias[i][id_t] for tokens with an adapter, in one product (y is written,
    rounded once); buf[i][t] = scale * x[t] @ lora_a[i][id_t]^T is written too.
    x bf16 [N][H]; w bf16 [out][H]; w_bias None or bf16 [out]; lora_a, lora_b,
    bias, buf as for lora_shrink_expand; y bf16 [N][out]; workspace uint8 of
    lora_linear_workspace_bytes."""
    where = "lora_linear"
    n, h = x.shape
    s, r = len(lora_a), lora_a[0].shape[1]
    widths = [t.shape[1] for t in lora_b]
    _forward_checks(where, meta, x, w.shape[0], y, lora_a, lora_b, buf, widths, r, workspace, offset_start)
    _projection(where, meta, h, w)
    _bias(bias, widths, meta, where)
    _w_bias(w_bias, w.shape[0], meta, where)
    _check(_lib().lora_linear(x.data_ptr(), x.stride(0), n, h, w.data_ptr(), w.stride(0), w.shape[0],
                              None if w_bias is None else w_bias.data_ptr(), _ptr_array(lora_a), _ptr_array(lora_b),
                              None if bias is None else _ptr_array(bias), _widths_array(widths), s, r, buf.data_ptr(),
                              y.data_ptr(), y.stride(0), int(offset_start), ctypes.byref(meta.struct), float(scale),
                              workspace.data_ptr(), workspace.numel(), _stream(stream)), where)


def _grads(ts, like, meta, where: str, name: str) -> None:
    import torch
    _need(len(ts) == len(like), LORA_ERR_SLICES, where, "one %s per slice" % name)
    device = meta.region.get_device()
    for i, (t, shape) in enumerate(zip(ts, like)):
        if device >= 0 and _whole(t, torch.bfloat16, device, shape):
            continue
        _dev(t, torch.bfloat16, meta, where, "%s[%d]" % (name, i))
        _need(tuple(t.shape) == tuple(shape) and t.is_contiguous(), LORA_ERR_SHAPE, where,
              "%s[%d] must be contiguous %s" % (name, i, tuple(shape)))


def _backward_checks(where: str, meta, dy, x, out: int, lora_a, lora_b, buf, dbuf, dx, da, db, dbias, widths, r: int,
                     workspace, offset_start: int) -> None:
    import torch
    n, h = x.shape
    s = len(lora_a)
    if not _linear_plain(meta, x, out, dy, lora_a, lora_b, (buf, dbuf), widths, r, workspace, offset_start):
        _layer_checks(where, meta, n, x=x, lora_a=lora_a, lora_b=lora_b, buf=buf)
        _need(len(lora_b) == s and buf.shape[0] == s, LORA_ERR_SLICES, where, "one weight per buf slice")
        _projected(where, meta, out, dy, "dy", offset_start, widths)
        _dev(dbuf, torch.float32, meta, where, "dbuf")
        _need(dbuf.shape == buf.shape and dbuf.is_contiguous(), LORA_ERR_SHAPE, where, "dbuf must be contiguous like buf")
        _workspace(workspace, meta.region.device, where)
    if dx is not None:
        _dev(dx, torch.bfloat16, meta, where, "dx")
        _need(tuple(dx.shape) == (n, h), LORA_ERR_SHAPE, where, "dx must be [%d][%d]" % (n, h))
    _grads(da, [t.shape for t in lora_a], meta, where, "da")
    _grads(db, [t.shape for t in lora_b], meta, where, "db")
    if dbias is not None:
        _need(len(dbias) == s, LORA_ERR_SLICES, where, "one dbias entry per slice")
        for i, t in enumerate(dbias):
            if t is not None:
                _grads([t], [lora_b[i].shape[:2]], meta, where, "dbias")


def lora_linear_backward(dy, x, w, lora_a: Sequence, lora_b: Sequence, buf, dbuf, dx, da: Sequence, db: Sequence,
                         dbias: Optional[Sequence], meta: LoraMeta, scale: float, workspace, offset_start: int = 0,
                         stream=None) -> None:
    """The gradients of lora_linear: dx = dy @ w + the adapters' part (dx may be
    None), da[i], db[i] and dbias[i] (None: not wanted) like lora_a[i],
    lora_b[i] and bias[i], zeros for ids without tokens.  buf is the forward
    pass's; dbuf (like buf) is written: scale * dy_i[t] @ lora_b[i][id_t].
    Matrices of ids from max_loras on are not touched."""
    where = "lora_linear_backward"
    n, h = x.shape
    s, r = len(lora_a), lora_a[0].shape[1]
    widths = [t.shape[1] for t in lora_b]
    _backward_checks(where, meta, dy, x, w.shape[0], lora_a, lora_b, buf, dbuf, dx, da, db, dbias, widths, r, workspace,
                     offset_start)
    _projection(where, meta, h, w)
    _check(_lib().lora_linear_backward(dy.data_ptr(), dy.stride(0), x.data_ptr(), x.stride(0), n, h, w.data_ptr(),
                                       w.stride(0), w.shape[0], _ptr_array(lora_a), _ptr_array(lora_b),
                                       _widths_array(widths), s, r, buf.data_ptr(), dbuf.data_ptr(),
                                       None if dx is None else dx.data_ptr(), 0 if dx is None else dx.stride(0),
                                       _ptr_array(da), _ptr_array(db), None if dbias is None else _ptr_array(dbias),
                                       int(offset_start), ctypes.byref(meta.struct), float(scale),
                                       workspace.data_ptr(), workspace.numel(), _stream(stream)), where)


def lora_cross_entropy_workspace_bytes(num_tokens: int, hidden: int, vocab: int, backward: bool = False) -> int:
    """Bytes of the workspace of lora_cross_entropy (backward: of both calls) for
    batches of up to num_tokens tokens: a uint8 device tensor."""
    n = int(_lib().lora_cross_entropy_workspace_bytes(int(num_tokens), int(hidden), int(vocab), 1 if backward else 0))
    if n == 0:
        raise LoraError(LORA_ERR_SHAPE, "lora_cross_entropy_workspace_bytes")
    return n


def _on(t, dtype, device, shape, where: str, name: str, contiguous: bool = True) -> None:
    """A tensor of this type and shape on `device`; rows of unit stride, or contiguous."""
    if t.is_cuda and t.device == device and (_whole if contiguous else _matrix)(t, dtype, t.get_device(), shape):
        return
    if not (t.is_cuda and t.device == device):
        raise TypeError("%s: %s must be on one GPU with w (got %s)" % (where, name, t.device))
    if t.dtype != dtype:
        raise TypeError("%s: %s must be %s (got %s)" % (where, name, dtype, t.dtype))
    _need(tuple(t.shape) == tuple(shape), LORA_ERR_SHAPE, where, "%s must be %s" % (name, tuple(shape)))
    _need(t.is_contiguous() if contiguous else t.stride(-1) == 1 or t.numel() <= 1, LORA_ERR_SHAPE, where,
          "%s must be contiguous%s" % (name, "" if contiguous else " in its last dimension"))


def _loss_checks(where: str, x, w, targets, workspace):
    import torch
    if not w.is_cuda:
        raise TypeError("%s: w must be on a GPU (got %s)" % (where, w.device))
    _need(x.dim() == 2 and w.dim() == 2, LORA_ERR_SHAPE, where, "x and w must be matrices")
    n, h = x.shape
    _on(w, torch.bfloat16, w.device, (w.shape[0], h), where, "w", False)
    _on(x, torch.bfloat16, w.device, (n, h), where, "x", False)
    _on(targets, torch.int32, w.device, (n,), where, "targets")
    _workspace(workspace, w.device, where)
    return n, h, w.shape[0]


def lora_cross_entropy(x, w, targets, loss, lse, workspace, stream=None) -> None:
    """loss[t] = lse[t] - (x @ w^T)[t][targets[t]] (0 where targets[t] is -1) and
    lse[t] = logsumexp of x @ w^T, without the logits in memory.  x bf16
    [N][H]; w bf16 [V][H]; targets int32 [N]; loss, lse float32 [N];
    workspace uint8 of lora_cross_entropy_workspace_bytes, whose first int32
    reports targets outside [-1, V) (LORA_ERR_ID_RANGE; they are ignored) where
    there are tokens at all."""
    import torch
    where = "lora_cross_entropy"
    n, h, v = _loss_checks(where, x, w, targets, workspace)
    _on(loss, torch.float32, w.device, (n,), where, "loss")
    _on(lse, torch.float32, w.device, (n,), where, "lse")
    _check(_lib().lora_cross_entropy(x.data_ptr(), x.stride(0), n, h, w.data_ptr(), w.stride(0), v, targets.data_ptr(),
                                     loss.data_ptr(), lse.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                     _stream(stream)), where)


def lora_cross_entropy_backward(x, w, targets, lse, dloss, dx, dw, workspace, stream=None) -> None:
    """The gradients of lora_cross_entropy for dloss float32 [N], from its lse:
    dx bf16 [N][H] and dw bf16 [V][H] are written (either may be None)."""
    import torch
    where = "lora_cross_entropy_backward"
    n, h, v = _loss_checks(where, x, w, targets, workspace)
    _on(lse, torch.float32, w.device, (n,), where, "lse")
    _on(dloss, torch.float32, w.device, (n,), where, "dloss")
    if dx is not None:
        _on(dx, torch.bfloat16, w.device, (n, h), where, "dx", False)
    if dw is not None:
        _on(dw, torch.bfloat16, w.device, (v, h), where, "dw", False)
    _check(_lib().lora_cross_entropy_backward(x.data_ptr(), x.stride(0), n, h, w.data_ptr(), w.stride(0), v,
                                              targets.data_ptr(), lse.data_ptr(), dloss.data_ptr(),
                                              None if dx is None else dx.data_ptr(), 0 if dx is None else dx.stride(0),
                                              None if dw is None else dw.data_ptr(), 0 if dw is None else dw.stride(0),
                                              workspace.data_ptr(), workspace.numel(), _stream(stream)), where)


def lora_mx_row_bytes(cols: int) -> tuple:
    """Bytes of a row of `cols` numbers in 4 bits: of its codes, and of its scales."""
    _need(cols >= 8 and cols % 8 == 0, LORA_ERR_SHAPE, "lora_mx_row_bytes", "cols must be a multiple of 8")
    blocks = (int(cols) + 31) // 32
    return 16 * blocks, (blocks + 3) // 4 * 4


def _mx_codes(where: str, device, codes, scales, rows: int, cols: int) -> tuple:
    """Checks the codes and scales of [rows][cols] numbers; their rows' distances."""
    import torch
    code_bytes, scale_bytes = (cols + 31) // 32 * 16, (cols + 127) // 128 * 4
    at, uint8 = device.index, torch.uint8
    if (codes.dtype is uint8 and scales.dtype is uint8 and codes.get_device() == at and scales.get_device() == at
            and codes.shape == (rows, code_bytes) and scales.shape == (rows, scale_bytes) and codes.is_contiguous()
            and scales.is_contiguous()):
        return code_bytes, scale_bytes
    for t, wide, name in ((codes, code_bytes, "codes"), (scales, scale_bytes, "scales")):
        if not (t.is_cuda and t.device == device):
            raise TypeError("%s: %s must be on %s (got %s)" % (where, name, device, t.device))
        if t.dtype != uint8:
            raise TypeError("%s: %s must be torch.uint8 (got %s)" % (where, name, t.dtype))
        _need(t.dim() == 2 and t.shape[0] == rows and t.shape[1] >= wide, LORA_ERR_SHAPE, where,
              "%s must be [%d][>= %d]" % (name, rows, wide))
        _need(t.stride(1) == 1, LORA_ERR_SHAPE, where, "%s needs unit stride in its last dimension" % name)
    return _pitch(codes), _pitch(scales)


def _type(t, where: str, name: str) -> int:
    import torch
    if t.dtype is torch.bfloat16:
        return LORA_BF16
    if t.dtype is torch.float32:
        return LORA_F32
    raise TypeError("%s: %s must be torch.bfloat16 or torch.float32 (got %s)" % (where, name, t.dtype))


def _pitch(t) -> int:
    """Distance of a matrix's rows; of a single row, its length rounded up as the
    library's checks want it (there is no next row)."""
    return t.stride(0) if t.shape[0] > 1 else (t.shape[1] + 15) // 16 * 16


def _mx_numbers(where: str, t, name: str) -> None:
    if not t.is_cuda:
        raise TypeError("%s: %s must be on a GPU (got %s)" % (where, name, t.device))
    _need(t.dim() == 2 and (t.stride(1) == 1 or t.numel() <= 1), LORA_ERR_SHAPE, where,
          "%s must be a matrix with unit stride in its last dimension" % name)


def lora_mx_quantize(x, codes, scales, stream=None) -> None:
    """Rows of x (bf16 or float32 [N][K], K % 8 == 0) to microscaled 4-bit numbers:
    codes uint8 [N][>= 16 ceil(K / 32)] (row distance a multiple of 16), two a byte,
    and scales uint8 [N][>= ceil(K / 32), rounded up to 4] (a multiple of 4), a
    power of two for every 32: the sizes of lora_mx_row_bytes."""
    where = "lora_mx_quantize"
    _mx_numbers(where, x, "x")
    kind = _type(x, where, "x")
    n, k = x.shape
    ldc, lds = _mx_codes(where, x.device, codes, scales, n, k)
    _check(_lib().lora_mx_quantize(x.data_ptr(), kind, _pitch(x), n, k, codes.data_ptr(), ldc, scales.data_ptr(), lds,
                                   _stream_on(stream, x.device, where)), where)


def lora_mx_dequantize(codes, scales, out, stream=None) -> None:
    """out (bf16 or float32 [N][K]) = the numbers that codes and scales stand for."""
    where = "lora_mx_dequantize"
    _mx_numbers(where, out, "out")
    kind = _type(out, where, "out")
    n, k = out.shape
    ldc, lds = _mx_codes(where, out.device, codes, scales, n, k)
    _check(_lib().lora_mx_dequantize(codes.data_ptr(), ldc, scales.data_ptr(), lds, n, k, out.data_ptr(), kind,
                                     _pitch(out), _stream_on(stream, out.device, where)), where)


def lora_linear_mx_workspace_bytes(num_tokens: int, max_loras: int, hidden: int, out_features: int, widths: Sequence,
                                   rank: int, backward: bool = False) -> int:
    """Bytes of the workspace of lora_linear_mx (backward: and of
    lora_linear_mx_backward) for batches of up to num_tokens tokens: a uint8 device
    tensor, whose contents do not matter."""
    n = int(_lib().lora_linear_mx_workspace_bytes(int(num_tokens), int(max_loras), int(hidden), int(out_features),
                                                  _widths_array(widths), len(widths), int(rank), 1 if backward else 0))
    if n == 0:
        raise LoraError(LORA_ERR_SHAPE, "lora_linear_mx_workspace_bytes")
    return n


def lora_linear_mx(x, codes, scales, w_bias, lora_a: Sequence, lora_b: Sequence, bias: Optional[Sequence], buf, y,
                   meta: LoraMeta, scale: float, workspace, offset_start: int = 0, quantize_x: bool = False,
                   stream=None) -> None:
    """lora_linear with the shared projection's matrix [out][H] in microscaled 4-bit
    numbers: codes and scales as lora_mx_quantize writes them.  quantize_x: x is
    rounded to such numbers too for the product with that matrix (the adapters read
    it as it is).  Everything else as for lora_linear; workspace uint8 of
    lora_linear_mx_workspace_bytes."""
    where = "lora_linear_mx"
    n, h = x.shape
    s, r = len(lora_a), lora_a[0].shape[1]
    out = codes.shape[0]
    widths = [t.shape[1] for t in lora_b]
    _forward_checks(where, meta, x, out, y, lora_a, lora_b, buf, widths, r, workspace, offset_start)
    ldc, lds = _mx_codes(where, meta.region.device, codes, scales, out, h)
    _bias(bias, widths, meta, where)
    _w_bias(w_bias, out, meta, where)
    _check(_lib().lora_linear_mx(x.data_ptr(), x.stride(0), n, h, codes.data_ptr(), ldc, scales.data_ptr(), lds, out,
                                 None if w_bias is None else w_bias.data_ptr(), _ptr_array(lora_a),
                                 _ptr_array(lora_b), None if bias is None else _ptr_array(bias), _widths_array(widths), s,
                                 r, buf.data_ptr(), y.data_ptr(), y.stride(0), int(offset_start),
                                 ctypes.byref(meta.struct), float(scale), 1 if quantize_x else 0, workspace.data_ptr(),
                                 workspace.numel(), _stream_on(stream, meta.region.device, where)), where)


def lora_linear_mx_backward(dy, x, codes, scales, lora_a: Sequence, lora_b: Sequence, buf, dbuf, dx, da: Sequence,
                            db: Sequence, dbias: Optional[Sequence], meta: LoraMeta, scale: float, workspace,
                            offset_start: int = 0, stream=None) -> None:
    """lora_linear_backward over such a matrix, which is frozen.  The gradient goes
    straight through the rounding of x, if the forward pass rounded it."""
    where = "lora_linear_mx_backward"
    n, h = x.shape
    s, r = len(lora_a), lora_a[0].shape[1]
    out = codes.shape[0]
    widths = [t.shape[1] for t in lora_b]
    _backward_checks(where, meta, dy, x, out, lora_a, lora_b, buf, dbuf, dx, da, db, dbias, widths, r, workspace,
                     offset_start)
    ldc, lds = _mx_codes(where, meta.region.device, codes, scales, out, h)
    _check(_lib().lora_linear_mx_backward(dy.data_ptr(), dy.stride(0), x.data_ptr(), x.stride(0), n, h, codes.data_ptr(),
                                          ldc, scales.data_ptr(), lds, out, _ptr_array(lora_a),
                                          _ptr_array(lora_b), _widths_array(widths), s, r, buf.data_ptr(),
                                          dbuf.data_ptr(), None if dx is None else dx.data_ptr(),
                                          0 if dx is None else dx.stride(0), _ptr_array(da), _ptr_array(db),
                                          None if dbias is None else _ptr_array(dbias), int(offset_start),
                                          ctypes.byref(meta.struct), float(scale), workspace.data_ptr(),
                                          workspace.numel(), _stream_on(stream, meta.region.device, where)), where)


class LoraGradients:
    """The tensors of a training step's gradients (bf16 or float32, contiguous, on one
    GPU), and of the scaled ones: `out`, tensors like them, or None to scale in
    place.  Made once for buffers that stay; a call looks whether any of them has
    another address, size, type or order than in the call before, and goes by them as
    they are."""

    def __init__(self, grads: Sequence, out: Optional[Sequence] = None):
        self.grads = list(grads)
        self.out = self.grads if out is None else list(out)
        self._marshal()

    def _seen(self, shapes: bool) -> list:
        """What a call goes by; with one norm a tensor's shape does not matter beside its size."""
        import torch
        ts, one = self.grads if self.out is self.grads else self.grads + self.out, torch.Tensor
        return [list(map(f, ts)) for f in (one.data_ptr, one.size if shapes else one.numel, attrgetter("dtype"),
                                           one.is_contiguous)]

    def _marshal(self) -> None:
        where, n, flat = "LoraGradients", len(self.grads), self._seen(False)
        _need(len(self.out) == n, LORA_ERR_SHAPE, where, "one result per gradient")
        device = self.grads[0].device if n else None
        kinds = []
        for i, (t, o) in enumerate(zip(self.grads, self.out)):
            if not (t.is_cuda and t.device == device and o.device == device):
                raise TypeError("%s: gradient and result %d must be on %s" % (where, i, device))
            kinds.append(_type(t, where, "grads[%d]" % i))
            if o.dtype != t.dtype:
                raise TypeError("%s: out[%d] must be %s (got %s)" % (where, i, t.dtype, o.dtype))
            _need(t.is_contiguous() and o.is_contiguous() and o.shape == t.shape, LORA_ERR_SHAPE, where,
                  "gradient and result %d must be contiguous and of one shape" % i)
        self.device, self._as = device, (flat, self._seen(True))
        self._in = (ctypes.c_void_p * n)(*flat[0][:n])
        self._out = self._in if self.out is self.grads else (ctypes.c_void_p * n)(*flat[0][n:])
        self._sizes = (ctypes.c_int64 * n)(*flat[1][:n])
        self._types = (ctypes.c_int * n)(*kinds)
        self._heads = {t.shape[0] if t.dim() else 1 for t in self.grads}

    def _current(self, groups: int) -> "LoraGradients":
        if self._seen(groups > 1) != self._as[groups > 1]:
            self._marshal()
        return self


def _gradients(grads, groups: int, out=None) -> LoraGradients:
    if isinstance(grads, LoraGradients):
        _need(out is None, LORA_ERR_SHAPE, "lora_clip_gradients", "a LoraGradients holds its results")
        return grads._current(groups)
    return LoraGradients(grads, out)


def lora_clip_gradients_workspace_bytes(grads, groups: int = 1) -> int:
    """Bytes of the workspace of lora_clip_gradients for these gradients (a sequence
    of tensors, or a LoraGradients) and so many norms: a uint8 device tensor, whose
    contents do not matter."""
    g = _gradients(grads, int(groups))
    n = int(_lib().lora_clip_gradients_workspace_bytes(g._sizes, g._types, len(g.grads), int(groups)))
    if n == 0:
        raise LoraError(LORA_ERR_SHAPE, "lora_clip_gradients_workspace_bytes")
    return n


def lora_clip_gradients(grads, norms, max_norm: float, workspace, out: Optional[Sequence] = None, stream=None) -> None:
    """Norms of gradients over many tensors, and the gradients times
    min(1, max_norm / (norm + 1e-6)), into `out` (like grads) or in place.  grads: a
    sequence of bf16 or float32 tensors, or a LoraGradients.  norms float32 [groups]
    is written: one norm over everything for groups 1, else norms[g] is that of the
    tensors' entries [g] (the gradients of adapter g: every tensor's first dimension
    is groups).  max_norm infinity: the norms alone.  A group with an infinity or a NaN
    in it keeps its gradients.  workspace uint8 of lora_clip_gradients_workspace_bytes."""
    import torch
    where = "lora_clip_gradients"
    _need(norms.dim() == 1 and norms.shape[0] >= 1, LORA_ERR_SHAPE, where, "norms must be [groups]")
    groups = norms.shape[0]
    g = _gradients(grads, groups, out)
    if not norms.is_cuda or (g.device is not None and norms.device != g.device):
        raise TypeError("%s: norms must be on one GPU with the gradients (got %s)" % (where, norms.device))
    _on(norms, torch.float32, norms.device, norms.shape, where, "norms")
    _need(groups == 1 or g._heads <= {groups}, LORA_ERR_SHAPE, where,
          "every gradient's first dimension must be the number of norms, %d" % groups)
    _workspace(workspace, norms.device, where)
    _check(_lib().lora_clip_gradients(g._in, g._out, g._sizes, g._types, len(g.grads), groups, float(max_norm),
                                      norms.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                      _stream_on(stream, norms.device, where)), where)
