"""Torch-facing call of the fused RMSNorm: tensors in, the C ABI underneath.

``rms_norm`` only checks shapes, allocates missing outputs with torch (the
caller's allocator, on the tensors' device) and passes raw pointers and the
current stream to ``rmsnorm_fwd``.  CPU tensors are refused: there is no
fallback path.
"""
from __future__ import annotations

import ctypes
import functools
import importlib.util
import os
import struct
import warnings
from typing import NamedTuple, Optional, Sequence

import torch

from . import _native as N

_CODES = {torch.bfloat16: N.RMSNORM_BF16, torch.float32: N.RMSNORM_F32}


def dtype_code(dtype: torch.dtype) -> int:
    try:
        return _CODES[dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {dtype}: bf16 or fp32 only") from None


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _check_tensor(t, name, x):
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path)")
    if t.device != x.device:
        raise ValueError(f"{name} is on {t.device}, x on {x.device}")
    if t.dtype != x.dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, x has {x.dtype}: one I/O type for all tensors")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def rms_norm(x: torch.Tensor, w: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
             eps: float = 1e-6, out: Optional[torch.Tensor] = None,
             residual_out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None,
             plan: Optional[N.Plan] = None, weight_bias: float = 0.0, cast_before_weight: bool = False):
    """y = x * rsqrt(mean(x^2) + eps) * (w + weight_bias) over the last dimension.

    With ``residual``: h = x + residual (rounded to the I/O type) is written to
    ``residual_out`` and normalised; returns ``(y, residual_out)``.  Without:
    returns ``y``.  ``plan`` forces a launch plan (see ``rmsnorm_fwd_plan``).
    ``weight_bias`` = 1 gives the (1 + w) weight form.  ``cast_before_weight``
    rounds the normalised value to the I/O type before the weight multiply
    (``rmsnorm_fwd_cast``, the eager op-by-op order; no weight bias).
    """
    if x.dim() < 1:
        raise ValueError("x must have at least one dimension")
    _check_tensor(x, "x", x)
    code = dtype_code(x.dtype)
    hidden = x.shape[-1]
    rows = x.numel() // hidden if hidden else 0
    for name, t in (("residual", residual), ("out", out), ("residual_out", residual_out)):
        if t is not None and t.shape != x.shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, x has {tuple(x.shape)}")
    if w is not None and tuple(w.shape) != (hidden,):
        raise ValueError(f"w must have shape ({hidden},), got {tuple(w.shape)}")
    y = torch.empty_like(x) if out is None else out
    if residual is not None and residual_out is None:
        residual_out = torch.empty_like(x)
    for name, t in (("w", w), ("residual", residual), ("out", y), ("residual_out", residual_out)):
        _check_tensor(t, name, x)
    with torch.cuda.device(x.device):
        s = stream if stream is not None else torch.cuda.current_stream(x.device)
        args = (_ptr(x), _ptr(residual), _ptr(w), _ptr(y), _ptr(residual_out), rows, hidden,
                float(eps))
        if cast_before_weight:
            if weight_bias:
                raise ValueError("cast_before_weight takes no weight_bias")
            N.rmsnorm_fwd_cast(*args, code, plan, s.cuda_stream)
        elif weight_bias:
            N.rmsnorm_fwd_ex(*args, float(weight_bias), code, plan, s.cuda_stream)
        elif plan is None:
            N.rmsnorm_fwd(*args, code, s.cuda_stream)
        else:
            N.rmsnorm_fwd_plan(*args, code, plan, s.cuda_stream)
    return (y, residual_out) if residual is not None else y


def rms_norm_host(x: torch.Tensor, w: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
                  eps: float = 1e-6, out: Optional[torch.Tensor] = None, residual_out: Optional[torch.Tensor] = None,
                  chunk_rows: int = 4096, workspace: Optional[torch.Tensor] = None,
                  device: Optional[torch.device] = None, stream: Optional[torch.cuda.Stream] = None):
    """``rms_norm`` on CPU tensors, streamed through a GPU in chunks of
    ``chunk_rows`` rows (``rmsnorm_fwd_host``): uploads, launches and
    read-backs overlap when the tensors are in pinned memory.  ``workspace``
    is a CUDA uint8 tensor of at least ``rmsnorm_host_workspace_bytes(...)``
    bytes
    (allocated on ``device`` when not given).  Returns after the work is
    queued on ``stream``: synchronise it before reading the outputs."""
    if x.dim() < 1:
        raise ValueError("x must have at least one dimension")
    code = dtype_code(x.dtype)
    hidden = x.shape[-1]
    rows = x.numel() // hidden if hidden else 0
    y = torch.empty_like(x) if out is None else out
    if residual is not None and residual_out is None:
        residual_out = torch.empty_like(x)
    for name, t in (("x", x), ("w", w), ("residual", residual), ("out", y), ("residual_out", residual_out)):
        if t is None:
            continue
        if t.is_cuda:
            raise ValueError(f"{name} must be a CPU tensor (use rms_norm for device tensors)")
        if t.dtype != x.dtype or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous with dtype {x.dtype}")
        if name != "w" and t.shape != x.shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, x has {tuple(x.shape)}")
    if w is not None and tuple(w.shape) != (hidden,):
        raise ValueError(f"w must have shape ({hidden},), got {tuple(w.shape)}")
    dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    need = N.rmsnorm_host_workspace_bytes(chunk_rows, hidden, code, residual is not None)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    if not workspace.is_cuda or workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace must be a CUDA tensor of at least {need} bytes")
    with torch.cuda.device(workspace.device):
        s = stream if stream is not None else torch.cuda.current_stream(workspace.device)
        N.rmsnorm_fwd_host(_ptr(x), _ptr(residual), _ptr(w), _ptr(y), _ptr(residual_out), rows, hidden,
                           float(eps), code, workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                           chunk_rows, s.cuda_stream)
    return (y, residual_out) if residual is not None else y


def _token_view(t: torch.Tensor, name: str):
    """(tokens, token_stride) of a [tokens, width] tensor with a contiguous last dimension."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D [tokens, width] tensor")
    if t.stride(1) != 1 and t.shape[1] > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return t.shape[0], t.stride(0), t


def qk_norm(qkv: torch.Tensor, q_heads: int, k_heads: int, head_dim: int, q_w: Optional[torch.Tensor] = None,
            k_w: Optional[torch.Tensor] = None, eps: float = 1e-6, weight_bias: float = 0.0,
            out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None,
            plan: Optional[N.Plan] = None) -> torch.Tensor:
    """Per-head RMSNorm of the query and key heads of packed token rows in one launch.

    ``qkv`` is [tokens, width] (last dimension contiguous, token rows evenly
    strided, e.g. a view of a fused projection) holding q_heads query heads, then
    k_heads key heads of head_dim elements, then anything else (value heads),
    which is left alone.  Query heads take ``q_w``, key heads ``k_w``.  The
    result goes to ``out`` (same layout; pass ``out=qkv`` to normalise in
    place) or to a new tensor whose other columns are copied from ``qkv``.
    """
    _check_tensor(qkv, "qkv", qkv)
    code = dtype_code(qkv.dtype)
    tokens, xs, rows = _token_view(qkv, "qkv")
    if out is None:
        out = qkv.clone()
    if out.shape != qkv.shape:
        raise ValueError("out must have the shape of qkv")
    _, ys, _ = _token_view(out, "out")
    for name, t in (("q_w", q_w), ("k_w", k_w)):
        if t is not None:
            _check_tensor(t, name, qkv)
            if tuple(t.shape) != (head_dim,):
                raise ValueError(f"{name} must have shape ({head_dim},)")
    if out.device != qkv.device or out.dtype != qkv.dtype:
        raise ValueError("out must match qkv's device and dtype")
    with torch.cuda.device(qkv.device):
        s = stream if stream is not None else torch.cuda.current_stream(qkv.device)
        N.rmsnorm_qk_fwd(_ptr(qkv), _ptr(out), tokens, xs, ys, int(q_heads), int(k_heads), int(head_dim),
                         _ptr(q_w), _ptr(k_w), float(weight_bias), float(eps), code, plan, s.cuda_stream)
    return out


def _empty(shape, dtype, device, stream):
    """An output or workspace allocated for work on ``stream`` (None: the
    current one), so that its memory is not handed out again before that work
    is done."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


# The calls below are made once a layer and token batch, and their kernels may
# take two microseconds.  The extension module ``_fastcall`` makes their checks
# and calls in native code; what it finds out of the ordinary it leaves to the
# Python bodies here (``None``), which say what is wrong or do it themselves.
_fast = None
_FAST_NAMES = ("rmsnorm_qk_rope_fwd", "rmsnorm_qk_rope_bwd", "rmsnorm_qk_rope_bwd_workspace_bytes",
               "rmsnorm_qkv_append", "rmsnorm_dropout_fwd", "rmsnorm_bwd", "rmsnorm_bwd_workspace_bytes",
               "rmsnorm_dropout_bwd", "rmsnorm_embedding_fwd", "rmsnorm_embedding_bwd",
               "rmsnorm_embedding_bwd_workspace_bytes", "rmsnorm_logprobs_fwd", "rmsnorm_logprobs_bwd",
               "rmsnorm_grad_norm", "rmsnorm_clip_grads", "rmsnorm_grad_norm_workspace_bytes")


class _PythonCalls:
    """In place of the extension module where there is none that the running
    torch and Python can load: every call is left to the Python bodies."""

    def __getattr__(self, name):
        return lambda *args: None


def _load_fast():
    from . import build
    path = build.fastcall_path()
    try:
        if not os.path.exists(path):
            raise ImportError(f"{path} does not exist")
        spec = importlib.util.spec_from_file_location(f"{__package__}._fastcall", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        return module
    except ImportError as e:
        warnings.warn(f"no native Python calls for this torch and Python ({e}): the same kernels are called several "
                      "microseconds slower; python -m row_reduction_norm_gb300.build makes them", RuntimeWarning,
                      stacklevel=4)
        return _PythonCalls()


def _bind_fast():
    global _fast
    lib = N.load()
    fast = _load_fast()
    fast.bind(*(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in _FAST_NAMES))
    _fast = fast
    return fast


def _took(result, where: str) -> bool:
    """Whether the native call was made; a status it came back with is raised."""
    if result is None:
        return False
    if type(result) is int:
        raise N.RmsNormError(result, where)
    return True


_raw_stream = torch._C._cuda_getCurrentRawStream      # the current stream's handle, by device number
_current_device = torch._C._cuda_getDevice


def _launch(dev: int, stream, call, *args):
    """call(*args, stream handle) with device number ``dev`` current."""
    if stream is None:
        s = _raw_stream(dev)
    elif stream.device.index != dev:
        raise ValueError(f"stream is on {stream.device}, the tensors on cuda:{dev}")
    else:
        s = stream.cuda_stream
    if _current_device() == dev:
        call(*args, s)
    else:
        with torch.cuda.device(dev):
            call(*args, s)


def _device_of(t: torch.Tensor, name: str) -> int:
    dev = t.get_device()
    if dev < 0 or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path)")
    return dev


def _head_rows(t: torch.Tensor, name: str, width: int, tokens: int, dtype, dev: int) -> int:
    """Token stride of a [tokens, >= width] tensor of packed heads (the last
    dimension contiguous)."""
    if t.get_device() != dev or t.dtype is not dtype:
        raise ValueError(f"{name} must be a {dtype} tensor on cuda:{dev} (no CPU path)")
    shape = t.shape
    if len(shape) != 2 or shape[0] != tokens or shape[1] < width:
        raise ValueError(f"{name} must be [{tokens}, at least {width}], got {tuple(shape)}")
    s0, s1 = t.stride()
    if s1 != 1 and shape[1] > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return s0 if tokens > 1 else max(s0, shape[1])


def _vector(t, name, size, dtype, dev: int):
    """Address of a contiguous [size] tensor (None for None)."""
    if t is None:
        return None
    if t.get_device() != dev or t.dtype is not dtype or t.shape != (size,) or (size > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous [{size}] tensor of {dtype} on cuda:{dev}")
    return t.data_ptr()


_pack_rope = struct.Struct("=QQqiiiiiiii").pack
_no_sections = (0, 0, 0)


def _rope_arg(positions, inv_freq, sections, interleaved, tokens, head_dim, dev: int) -> N.Rope:
    pairs = inv_freq.numel()
    freq = _vector(inv_freq, "inv_freq", pairs, torch.float32, dev)
    if not 1 <= pairs <= head_dim // 2:
        raise ValueError(f"inv_freq must hold 1..{head_dim // 2} frequencies, one for each rotated pair")
    if sections is None:
        axes, four = 1, (pairs, 0, 0, 0)
    else:
        axes = len(sections)
        if not 1 <= axes <= 4 or min(sections) < 0 or sum(sections) != pairs:
            raise ValueError(f"sections must be 1..4 counts that add up to {pairs}")
        four = (*sections, *_no_sections)[:4]
    at = stride = 0
    size = 4
    if positions is not None:
        shape, strides = positions.shape, positions.stride()
        kind = positions.dtype
        if positions.get_device() != dev or (kind is not torch.int64 and kind is not torch.int32):
            raise ValueError(f"positions must be an int32 or int64 tensor on cuda:{dev}")
        if shape != ((axes, tokens) if len(shape) == 2 else (tokens,)) or (tokens > 1 and strides[-1] != 1) or (
                axes > 1 and len(shape) != 2):
            raise ValueError(f"positions must be [{axes}, {tokens}] with a contiguous last dimension, "
                             f"got {tuple(shape)}")
        at = positions.data_ptr()
        size = 8 if kind is torch.int64 else 4
        if axes > 1:
            stride = strides[0] if tokens > 1 else max(strides[0], tokens)
    return N.Rope.from_buffer_copy(_pack_rope(at, freq, stride, size, axes, 2 * pairs, 1 if interleaved else 0, *four))


def qk_norm_rope(qkv: torch.Tensor, q_heads: int, k_heads: int, head_dim: int, positions: torch.Tensor,
                 inv_freq: torch.Tensor, q_w: Optional[torch.Tensor] = None, k_w: Optional[torch.Tensor] = None,
                 eps: float = 1e-6, weight_bias: float = 0.0, norm: bool = True, sections=None,
                 interleaved: bool = False, out: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """``qk_norm`` with the rotary positions applied to the normalised heads, in one launch.

    ``positions`` is [tokens] or [axes, tokens] (int32 or int64), ``inv_freq``
    (fp32) holds one frequency for each rotated pair: the first
    2 * len(inv_freq) elements of a head turn.  ``sections`` shares the pairs
    out to the axes in order (default: all to one axis); pairs are
    (i, i + len(inv_freq)), or neighbours with ``interleaved``.  ``norm=False``
    turns the heads as they are.  The result goes to ``out``, whose first
    q_heads + k_heads heads are written (``out=qkv`` works in place), or to a
    new [tokens, (q_heads + k_heads) * head_dim] tensor.
    """
    if stream is None and qkv.is_cuda:
        y = (_fast or _bind_fast()).qk_norm_rope(qkv, q_heads, k_heads, head_dim, positions, inv_freq, q_w, k_w, eps,
                                                 weight_bias, norm, sections, interleaved, out)
        if _took(y, "rmsnorm_qk_rope_fwd"):
            return y
    q_heads, k_heads, head_dim = int(q_heads), int(k_heads), int(head_dim)
    t = qkv.dtype
    code = dtype_code(t)
    dev = _device_of(qkv, "qkv")
    width = (q_heads + k_heads) * head_dim
    tokens = qkv.shape[0]
    xs = _head_rows(qkv, "qkv", width, tokens, t, dev)
    qw, kw = _vector(q_w, "q_w", head_dim, t, dev), _vector(k_w, "k_w", head_dim, t, dev)
    rope = _rope_arg(positions, inv_freq, sections, interleaved, tokens, head_dim, dev)
    if out is None:
        out = _empty((tokens, width), t, qkv.device, stream)
    ys = _head_rows(out, "out", width, tokens, t, dev)
    _launch(dev, stream, N.rmsnorm_qk_rope_fwd, qkv.data_ptr(), out.data_ptr(), tokens, xs, ys, q_heads, k_heads,
            head_dim, qw, kw, float(weight_bias), float(eps), 1 if norm else 0, rope, code)
    return out


def qk_norm_rope_backward(dout: torch.Tensor, qkv: Optional[torch.Tensor], q_heads: int, k_heads: int, head_dim: int,
                          positions: torch.Tensor, inv_freq: torch.Tensor, q_w: Optional[torch.Tensor] = None,
                          k_w: Optional[torch.Tensor] = None, eps: float = 1e-6, weight_bias: float = 0.0,
                          norm: bool = True, sections=None, interleaved: bool = False,
                          out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                          stream: Optional[torch.cuda.Stream] = None):
    """Gradient of ``qk_norm_rope``: returns (dqkv, dq_w, dk_w).

    ``dout`` holds the gradient of the rotated heads, ``qkv`` the forward's
    input (None with ``norm=False``).  dqkv goes to ``out`` (its first
    q_heads + k_heads heads; ``out=dout`` works in place) or to a new tensor;
    dq_w and dk_w are None without weights.  ``workspace`` is a CUDA uint8
    tensor of ``rmsnorm_qk_rope_bwd_workspace_bytes(head_dim)`` bytes
    (allocated when not given).
    """
    if stream is None and dout.is_cuda:
        r = (_fast or _bind_fast()).qk_norm_rope_backward(dout, qkv, q_heads, k_heads, head_dim, positions, inv_freq,
                                                          q_w, k_w, eps, weight_bias, norm, sections, interleaved, out,
                                                          workspace)
        if _took(r, "rmsnorm_qk_rope_bwd"):
            return r
    q_heads, k_heads, head_dim = int(q_heads), int(k_heads), int(head_dim)
    t = dout.dtype
    code = dtype_code(t)
    dev = _device_of(dout, "dout")
    width = (q_heads + k_heads) * head_dim
    tokens = dout.shape[0]
    gs = _head_rows(dout, "dout", width, tokens, t, dev)
    if qkv is None and norm:
        raise ValueError("the norm's gradient needs qkv")
    xs = _head_rows(qkv, "qkv", width, tokens, t, dev) if qkv is not None else width
    qw, kw = _vector(q_w, "q_w", head_dim, t, dev), _vector(k_w, "k_w", head_dim, t, dev)
    rope = _rope_arg(positions, inv_freq, sections, interleaved, tokens, head_dim, dev)
    if out is None:
        out = _empty((tokens, width), t, dout.device, stream)
    ds = _head_rows(out, "out", width, tokens, t, dev)
    dq_w = dk_w = dq = dk = None
    ws = need = 0
    if qw is not None and kw is not None:
        dq_w, dk_w = (_empty((head_dim,), t, dout.device, stream) for _ in range(2))
        dq, dk = dq_w.data_ptr(), dk_w.data_ptr()
        need = _rope_workspace_bytes(head_dim)
        workspace = _workspace(workspace, need, dout.device, stream)
        ws = workspace.data_ptr()
    _launch(dev, stream, N.rmsnorm_qk_rope_bwd, dout.data_ptr(), _ptr(qkv), out.data_ptr(), tokens, gs, xs, ds, q_heads,
            k_heads, head_dim, qw, kw, dq, dk, float(weight_bias), float(eps), 1 if norm else 0, rope, code, ws, need)
    return out, dq_w, dk_w


@functools.lru_cache(maxsize=64)
def _rope_workspace_bytes(head_dim: int) -> int:
    return N.rmsnorm_qk_rope_bwd_workspace_bytes(head_dim)


@functools.lru_cache(maxsize=256)
def _bwd_workspace_bytes(rows: int, hidden: int, code: int, dev: int) -> int:
    with torch.cuda.device(dev):
        return N.rmsnorm_bwd_workspace_bytes(rows, hidden, code)


def _workspace(workspace, need, device, stream):
    if workspace is None:
        return _empty((need,), torch.uint8, device, stream)
    if workspace.device != device or not workspace.is_contiguous() or \
            workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace must be a contiguous tensor of at least {need} bytes on {device}")
    return workspace


_pack_kv = struct.Struct("=QQQQQQqqqqiiiiiff4x").pack
_CACHE_CODES = {torch.bfloat16: N.RMSNORM_BF16, torch.float32: N.RMSNORM_F32, torch.float8_e4m3fn: N.RMSNORM_E4M3}


def qkv_append(qkv: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor,
               cu_tokens: torch.Tensor, cache_lens: torch.Tensor, q_heads: int, kv_heads: int, head_dim: int,
               inv_freq: torch.Tensor, positions: Optional[torch.Tensor] = None, q_w: Optional[torch.Tensor] = None,
               k_w: Optional[torch.Tensor] = None, eps: float = 1e-6, weight_bias: float = 0.0, norm: bool = True,
               sections=None, interleaved: bool = False, k_scale: float = 1.0, v_scale: float = 1.0,
               q_out: Optional[torch.Tensor] = None, dropped: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None) -> Optional[torch.Tensor]:
    """Appends a ragged batch to a paged cache: Q+K norm and rotation as in
    ``qk_norm_rope``, queries to ``q_out`` (returned), keys and values to the
    cache, in one launch.

    ``qkv`` is [tokens, (q_heads + 2 * kv_heads) * head_dim].  The caches are
    [num_pages, page_size, kv_heads, head_dim] tensors of any strides with a
    contiguous last dimension (so a permuted view of a cache kept head by head
    too), in qkv's type or float8_e4m3fn, where a code stands for
    code * ``k_scale`` (``v_scale``; 2^-100 .. 2^100).  Sequence s brings the tokens
    cu_tokens[s] .. cu_tokens[s + 1] - 1 (int32, [seqs + 1]) and has
    cache_lens[s] rows (int32) in the pages page_table[s] (int32, [seqs,
    max_pages], -1: no page); cache_lens is left as it is.  ``positions``
    defaults to the row's index in its sequence.  Rows behind the last
    sequence are left alone; rows without a page are not written and counted
    in ``dropped`` (int32, [1], added to) where given.
    """
    if stream is None and qkv.is_cuda:
        r = (_fast or _bind_fast()).qkv_append(qkv, k_cache, v_cache, page_table, cu_tokens, cache_lens, q_heads,
                                               kv_heads, head_dim, inv_freq, positions, q_w, k_w, eps, weight_bias,
                                               norm, sections, interleaved, k_scale, v_scale, q_out, dropped)
        if _took(r, "rmsnorm_qkv_append"):
            return r
    q_heads, kv_heads, head_dim = int(q_heads), int(kv_heads), int(head_dim)
    t = qkv.dtype
    code = dtype_code(t)
    dev = _device_of(qkv, "qkv")
    tokens = qkv.shape[0]
    xs = _head_rows(qkv, "qkv", (q_heads + 2 * kv_heads) * head_dim, tokens, t, dev)
    qw, kw = _vector(q_w, "q_w", head_dim, t, dev), _vector(k_w, "k_w", head_dim, t, dev)
    rope = _rope_arg(positions, inv_freq, sections, interleaved, tokens, head_dim, dev)
    shape, strides, kind = k_cache.shape, k_cache.stride(), k_cache.dtype
    if len(shape) != 4 or shape[2] != kv_heads or shape[3] != head_dim or strides[3] != 1:
        raise ValueError(f"k_cache must be [num_pages, page_size, {kv_heads}, {head_dim}] with a contiguous last "
                         f"dimension, got {tuple(shape)}")
    if v_cache.shape != shape or v_cache.stride() != strides or v_cache.dtype is not kind:
        raise ValueError("v_cache must have the shape, strides and dtype of k_cache")
    if k_cache.get_device() != dev or v_cache.get_device() != dev:
        raise ValueError(f"the caches must be on cuda:{dev}")
    if kind is not t and kind is not torch.float8_e4m3fn:
        raise TypeError(f"caches of {kind}: {t} or float8_e4m3fn only")
    if page_table.dim() != 2 or page_table.dtype is not torch.int32 or page_table.get_device() != dev:
        raise ValueError(f"page_table must be a 2-D int32 tensor on cuda:{dev}")
    seqs, max_pages = page_table.shape
    p0, p1 = page_table.stride()
    if p1 != 1 and max_pages > 1:
        raise ValueError("page_table: the last dimension must be contiguous")
    cu = _vector(cu_tokens, "cu_tokens", seqs + 1, torch.int32, dev)
    lens = _vector(cache_lens, "cache_lens", seqs, torch.int32, dev)
    drop = _vector(dropped, "dropped", 1, torch.int32, dev) or 0
    qs = 0
    q_at = None
    if q_heads > 0:
        if q_out is None:
            q_out = _empty((tokens, q_heads * head_dim), t, qkv.device, stream)
        qs = _head_rows(q_out, "q_out", q_heads * head_dim, tokens, t, dev)
        q_at = q_out.data_ptr()
    # strides of dimensions of one place are never used: 0 keeps them from
    # narrowing the accesses
    kv = N.PagedKV.from_buffer_copy(_pack_kv(
        k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(), cu, lens, drop,
        p0 if seqs > 1 else max(p0, max_pages), strides[0] if shape[0] > 1 else 0, strides[1] if shape[1] > 1 else 0,
        strides[2] if shape[2] > 1 else 0, seqs, max_pages, shape[0], shape[1], _CACHE_CODES[kind], float(k_scale),
        float(v_scale)))
    _launch(dev, stream, N.rmsnorm_qkv_append, qkv.data_ptr(), q_at, tokens, xs, qs, q_heads, kv_heads, head_dim, qw,
            kw, float(weight_bias), float(eps), 1 if norm else 0, rope, kv, code)
    return q_out


def _rows_of(t: torch.Tensor, name: str):
    """(device number, rows, hidden) of a contiguous CUDA tensor."""
    dev = _device_of(t, name)
    shape = t.shape
    if not shape or shape[-1] < 1:
        raise ValueError(f"{name} must have a last dimension of at least one element")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return dev, t.numel() // shape[-1], shape[-1]


def _like(t, name, x, dev: int) -> int:
    """Address of a contiguous tensor of the shape and type of ``x``."""
    if t.get_device() != dev or t.dtype is not x.dtype or t.shape != x.shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {tuple(x.shape)} tensor of {x.dtype} on cuda:{dev}")
    return t.data_ptr()


def _rng_arg(rng, p, dev: int):
    if rng is None:
        if p:
            raise ValueError("dropout needs rng, an int64 tensor of seed and offset")
        return None
    if rng.get_device() != dev or rng.dtype not in (torch.int64, torch.uint64) or rng.shape != (2,) or \
            rng.stride(0) != 1:
        raise ValueError(f"rng must be a contiguous [2] int64 tensor of seed and offset on cuda:{dev}")
    return rng.data_ptr()


def rms_norm_dropout(x: torch.Tensor, residual: torch.Tensor, p: float, rng: Optional[torch.Tensor],
                     w: Optional[torch.Tensor] = None, eps: float = 1e-6, weight_bias: float = 0.0,
                     out: Optional[torch.Tensor] = None, residual_out: Optional[torch.Tensor] = None,
                     stream: Optional[torch.cuda.Stream] = None):
    """Residual dropout and RMSNorm in one launch: returns (y, residual_out),
    residual_out = residual + dropout(x), y = its norm.

    ``rng`` is a CUDA int64 tensor (seed, offset), read when the kernel runs;
    the same values give the same mask, which is never stored, so a step that
    wants another mask changes the offset.  ``p`` is rounded to a multiple of
    2^-16, and kept elements are scaled by the inverse of the probability that
    makes.
    """
    if stream is None and x.is_cuda:
        r = (_fast or _bind_fast()).rms_norm_dropout(x, residual, p, rng, w, eps, weight_bias, out, residual_out)
        if _took(r, "rmsnorm_dropout_fwd"):
            return r
    code = dtype_code(x.dtype)
    dev, rows, hidden = _rows_of(x, "x")
    res = _like(residual, "residual", x, dev)
    wp = _vector(w, "w", hidden, x.dtype, dev)
    r = _rng_arg(rng, p, dev)
    if out is None:
        out = _empty(x.shape, x.dtype, x.device, stream)
    if residual_out is None:
        residual_out = _empty(x.shape, x.dtype, x.device, stream)
    _launch(dev, stream, N.rmsnorm_dropout_fwd, x.data_ptr(), res, wp, _like(out, "out", x, dev),
            _like(residual_out, "residual_out", x, dev), rows, hidden, float(eps), float(weight_bias), float(p), r,
            code)
    return out, residual_out


def _backward_args(dy, h, w, dresidual_out, workspace, stream):
    t = dy.dtype
    code = dtype_code(t)
    dev, rows, hidden = _rows_of(dy, "dy")
    at = (dy.data_ptr(), _like(h, "h", dy, dev), _vector(w, "w", hidden, t, dev),
          None if dresidual_out is None else _like(dresidual_out, "dresidual_out", dy, dev))
    if w is None:
        return dev, code, rows, hidden, at, None, None, 0, None
    dw = _empty((hidden,), t, dy.device, stream)
    need = _bwd_workspace_bytes(rows, hidden, code, dev)
    workspace = _workspace(workspace, need, dy.device, stream)
    # the workspace stays referenced until the call is made
    return dev, code, rows, hidden, at, dw, workspace.data_ptr(), need, workspace


def rms_norm_backward(dy: torch.Tensor, h: torch.Tensor, w: Optional[torch.Tensor] = None,
                      dresidual_out: Optional[torch.Tensor] = None, eps: float = 1e-6, weight_bias: float = 0.0,
                      out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                      stream: Optional[torch.cuda.Stream] = None):
    """Gradient of ``rms_norm``: returns (dx, dw), dw None without a weight.

    ``h`` is what was normalised: x, or residual_out with a residual, whose
    gradient dx then is too.  ``dresidual_out``, the gradient that reaches h
    past the norm, is added.  ``workspace``: a CUDA uint8 tensor of
    ``rmsnorm_bwd_workspace_bytes(rows, hidden, dtype)`` bytes (allocated when
    not given).
    """
    if stream is None and dy.is_cuda:
        r = (_fast or _bind_fast()).rms_norm_backward(dy, h, w, dresidual_out, eps, weight_bias, out, workspace)
        if _took(r, "rmsnorm_bwd"):
            return r
    dev, code, rows, hidden, at, dw, ws, need, keep = _backward_args(dy, h, w, dresidual_out, workspace, stream)
    if out is None:
        out = _empty(dy.shape, dy.dtype, dy.device, stream)
    _launch(dev, stream, N.rmsnorm_bwd, *at, _like(out, "out", dy, dev), None if dw is None else dw.data_ptr(), rows,
            hidden, float(eps), float(weight_bias), code, ws, need)
    return out, dw


def rms_norm_dropout_backward(dy: torch.Tensor, h: torch.Tensor, p: float, rng: Optional[torch.Tensor],
                              w: Optional[torch.Tensor] = None, dresidual_out: Optional[torch.Tensor] = None,
                              eps: float = 1e-6, weight_bias: float = 0.0, dresidual: Optional[torch.Tensor] = None,
                              dx: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                              stream: Optional[torch.cuda.Stream] = None):
    """Gradient of ``rms_norm_dropout`` (``h``: its residual_out, with the same
    ``p`` and ``rng``): returns (dresidual, dx, dw), dw None without a weight.
    Other arguments as ``rms_norm_backward``."""
    if stream is None and dy.is_cuda:
        r = (_fast or _bind_fast()).rms_norm_dropout_backward(dy, h, p, rng, w, dresidual_out, eps, weight_bias,
                                                              dresidual, dx, workspace)
        if _took(r, "rmsnorm_dropout_bwd"):
            return r
    dev, code, rows, hidden, at, dw, ws, need, keep = _backward_args(dy, h, w, dresidual_out, workspace, stream)
    r = _rng_arg(rng, p, dev)
    if dresidual is None:
        dresidual = _empty(dy.shape, dy.dtype, dy.device, stream)
    if dx is None:
        dx = _empty(dy.shape, dy.dtype, dy.device, stream)
    _launch(dev, stream, N.rmsnorm_dropout_bwd, *at, _like(dresidual, "dresidual", dy, dev), _like(dx, "dx", dy, dev),
            None if dw is None else dw.data_ptr(), rows, hidden, float(eps), float(weight_bias), float(p), r,
            code, ws, need)
    return dresidual, dx, dw


def _ids(t: torch.Tensor, name: str, shape, dev: int):
    """(address, bytes of an id) of a contiguous tensor of token ids."""
    kind = t.dtype
    if t.get_device() != dev or (kind is not torch.int64 and kind is not torch.int32) or not t.is_contiguous() or (
            shape is not None and t.shape != shape):
        raise ValueError(f"{name} must be a contiguous int32 or int64 tensor on cuda:{dev}"
                         + ("" if shape is None else f" of shape {tuple(shape)}"))
    return t.data_ptr(), 8 if kind is torch.int64 else 4


def _row_stride(t: torch.Tensor, name: str) -> int:
    """Elements between the rows of a 2-D tensor (the last dimension contiguous)."""
    shape = t.shape
    if len(shape) != 2 or shape[1] < 1:
        raise ValueError(f"{name} must be a 2-D tensor with rows of at least one element, got {tuple(shape)}")
    s0, s1 = t.stride()
    if s1 != 1 and shape[1] > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return s0 if shape[0] > 1 else max(s0, shape[1])


def embedding(tokens: torch.Tensor, table: torch.Tensor, scale: float = 1.0, out: Optional[torch.Tensor] = None,
              stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Rows of ``table`` times ``scale`` for each token: an fp32 product, rounded to
    the table's type.

    ``tokens`` is an int32 or int64 tensor of any shape, ``table`` [vocab,
    width] (last dimension contiguous, rows evenly strided); the result is
    [*tokens.shape, width].  A token outside 0 .. vocab - 1 (-1 marks padding)
    gives a row of zeros.  ``out`` must not overlap the table.
    """
    if stream is None and table.is_cuda:
        y = (_fast or _bind_fast()).embedding(tokens, table, scale, out)
        if _took(y, "rmsnorm_embedding_fwd"):
            return y
    t = table.dtype
    code = dtype_code(t)
    dev = _device_of(table, "table")
    stride = _row_stride(table, "table")
    at, size = _ids(tokens, "tokens", None, dev)
    vocab, width = table.shape
    shape = (*tokens.shape, width)
    if out is None:
        out = _empty(shape, t, table.device, stream)
    elif out.get_device() != dev or out.dtype is not t or out.shape != shape or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous {shape} tensor of {t} on cuda:{dev}")
    _launch(dev, stream, N.rmsnorm_embedding_fwd, at, size, table.data_ptr(), out.data_ptr(), tokens.numel(), vocab,
            width, stride, float(scale), code)
    return out


def embedding_backward(dout: torch.Tensor, tokens: torch.Tensor, vocab: int, scale: float = 1.0,
                       out: Optional[torch.Tensor] = None, accumulate: bool = False,
                       workspace: Optional[torch.Tensor] = None,
                       stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Gradient of ``embedding`` in its table: [vocab, width], a token's row the
    sum of its places' ``dout`` times ``scale``, other rows zeros.

    ``out`` (dout's type, or float32; the last dimension contiguous, rows
    evenly strided) takes the gradient; with ``accumulate`` it is added to what
    ``out`` holds, and only rows of tokens that occur are touched.  Sums are
    fp32 in an order that follows from the tokens and the sizes alone.
    ``workspace`` is a CUDA uint8 tensor of
    ``rmsnorm_embedding_bwd_workspace_bytes(tokens, vocab, width)`` bytes
    (allocated when not given).
    """
    if stream is None and dout.is_cuda:
        r = (_fast or _bind_fast()).embedding_backward(dout, tokens, vocab, scale, out, accumulate, workspace)
        if _took(r, "rmsnorm_embedding_bwd"):
            return r
    vocab = int(vocab)
    t = dout.dtype
    code = dtype_code(t)
    dev, count, width = _rows_of(dout, "dout")
    at, size = _ids(tokens, "tokens", dout.shape[:-1], dev)
    if vocab < 1:
        raise ValueError("vocab must be at least 1")
    if out is None:
        if accumulate:
            raise ValueError("accumulate adds to out, which is not given")
        out = _empty((vocab, width), t, dout.device, stream)
    if out.get_device() != dev or out.shape != (vocab, width) or (out.dtype is not t and out.dtype is not torch.float32):
        raise ValueError(f"out must be a {(vocab, width)} tensor of {t} or float32 on cuda:{dev}")
    need = N.rmsnorm_embedding_bwd_workspace_bytes(count, vocab, width)
    workspace = _workspace(workspace, need, dout.device, stream)
    _launch(dev, stream, N.rmsnorm_embedding_bwd, dout.data_ptr(), at, size, out.data_ptr(), count, vocab, width,
            _row_stride(out, "out"), float(scale), 1 if accumulate else 0, code, dtype_code(out.dtype),
            workspace.data_ptr(), need)
    return out


class TokenLogprobs(NamedTuple):
    """What ``token_logprobs`` returns; None for what was not asked for."""
    logprobs: Optional[torch.Tensor]       # [rows] float32
    stats: torch.Tensor                    # [rows, 2] float32: the largest logit, and the log of the sum relative to it
    entropy: Optional[torch.Tensor]        # [rows] float32
    top_logprobs: Optional[torch.Tensor]   # [rows, top] float32
    top_ids: Optional[torch.Tensor]        # [rows, top] int32


def _logits_args(logits, tokens, name):
    code = dtype_code(logits.dtype)
    dev = _device_of(logits, name)
    stride = _row_stride(logits, name)
    rows, vocab = logits.shape
    at, size = (None, 4) if tokens is None else _ids(tokens, "tokens", (rows,), dev)
    return code, dev, stride, rows, vocab, at, size


def token_logprobs(logits: torch.Tensor, tokens: Optional[torch.Tensor], temperature: float = 1.0, top: int = 0,
                   entropy: bool = False, stream: Optional[torch.cuda.Stream] = None) -> TokenLogprobs:
    """Log probabilities of the given tokens under softmax(logits / temperature),
    and on request the entropy of each row and the ``top`` (up to 32) likeliest
    tokens with theirs, in one pass over the logits.

    ``logits`` is [rows, vocab] (last dimension contiguous, rows evenly
    strided, so a view of padded rows too), ``tokens`` int32 or int64 [rows], or
    None for no log probabilities; places whose token lies outside 0 .. vocab -
    1 get 0.  -infinity masks a token; a row of nothing else has log
    probabilities of -infinity and an entropy of 0.  Equal logits are ordered by
    the lower id.  ``stats`` is what ``token_logprobs_backward`` starts from.
    A row that holds a NaN or +infinity has NaN for all of these; among the
    alternatives a NaN counts as -infinity.  What is returned may share one
    allocation: any of it keeps all of it, and ``torch.save`` writes all of it
    (``clone`` what is to be kept by itself).
    """
    if stream is None and logits.is_cuda:
        r = (_fast or _bind_fast()).token_logprobs(logits, tokens, temperature, top, entropy)
        if _took(r, "rmsnorm_logprobs_fwd"):
            return TokenLogprobs._make(r)
    top = int(top)
    code, dev, stride, rows, vocab, at, size = _logits_args(logits, tokens, "logits")
    if not 0 <= top <= min(32, vocab):
        raise ValueError(f"top must be 0 .. {min(32, vocab)}")
    f32, there = torch.float32, logits.device
    made = TokenLogprobs(None if tokens is None else _empty((rows,), f32, there, stream),
                         _empty((rows, 2), f32, there, stream),
                         _empty((rows,), f32, there, stream) if entropy else None,
                         _empty((rows, top), f32, there, stream) if top else None,
                         _empty((rows, top), torch.int32, there, stream) if top else None)
    _launch(dev, stream, N.rmsnorm_logprobs_fwd, logits.data_ptr(), at, size, *(_ptr(t) for t in made), rows, vocab,
            stride, top, float(temperature), code)
    return made


def token_logprobs_backward(logits: torch.Tensor, tokens: Optional[torch.Tensor], stats: torch.Tensor,
                            dlogprobs: Optional[torch.Tensor], entropy: Optional[torch.Tensor] = None,
                            dentropy: Optional[torch.Tensor] = None, temperature: float = 1.0,
                            out: Optional[torch.Tensor] = None,
                            stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Gradient of ``token_logprobs`` in the logits, of the log probabilities
    (``dlogprobs``, float32 [rows], or None) and of the entropies (``dentropy``
    with the forward's ``entropy``).  ``stats`` is the forward's.  Goes to
    ``out`` (``out=logits`` works in place) or a new [rows, vocab] tensor."""
    if stream is None and logits.is_cuda:
        r = (_fast or _bind_fast()).token_logprobs_backward(logits, tokens, stats, dlogprobs, entropy, dentropy,
                                                            temperature, out)
        if _took(r, "rmsnorm_logprobs_bwd"):
            return r
    code, dev, stride, rows, vocab, at, size = _logits_args(logits, tokens, "logits")
    f32 = torch.float32
    if stats.get_device() != dev or stats.dtype is not f32 or stats.shape != (rows, 2) or not stats.is_contiguous():
        raise ValueError(f"stats must be a contiguous [{rows}, 2] float32 tensor on cuda:{dev}")
    if dlogprobs is not None and tokens is None:
        raise ValueError("dlogprobs needs the tokens")
    if dentropy is not None and entropy is None:
        raise ValueError("dentropy needs the forward's entropy")
    if out is None:
        out = _empty((rows, vocab), logits.dtype, logits.device, stream)
    if out.get_device() != dev or out.dtype is not logits.dtype or out.shape != logits.shape:
        raise ValueError(f"out must be a {(rows, vocab)} tensor of {logits.dtype} on cuda:{dev}")
    _launch(dev, stream, N.rmsnorm_logprobs_bwd, logits.data_ptr(), at, size, stats.data_ptr(),
            _vector(dlogprobs, "dlogprobs", rows, f32, dev), _vector(entropy, "entropy", rows, f32, dev),
            _vector(dentropy, "dentropy", rows, f32, dev), out.data_ptr(), rows, vocab, stride,
            _row_stride(out, "out"), float(temperature), code)
    return out


def _grads_arg(grads, out):
    """(device number, device, array of the tensors that are there)."""
    pairs = [(g, g if out is None else out[i]) for i, g in enumerate(grads) if g is not None]
    if not pairs:
        raise ValueError("no gradients: every entry is None, or there are none")
    dev = _device_of(pairs[0][0], "grads[0]")
    array = (N.Grad * len(pairs))()
    for a, (g, o) in zip(array, pairs):
        if g.get_device() != dev or not g.is_contiguous():
            raise ValueError(f"gradients must be contiguous tensors on cuda:{dev}")
        if o is not g and (o is None or o.get_device() != dev or o.dtype is not g.dtype or o.shape != g.shape
                           or not o.is_contiguous()):
            raise ValueError("out must hold a contiguous tensor like each gradient")
        a.grad, a.out, a.count, a.dtype = g.data_ptr(), o.data_ptr(), g.numel(), dtype_code(g.dtype)
    return dev, pairs[0][0].device, array


def grad_norm(grads: Sequence[Optional[torch.Tensor]], workspace: Optional[torch.Tensor] = None,
              stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The 2-norm of all the tensors together, float32 [1] on their device (see ``clip_grad_norm``)."""
    return _norm_or_clip(grads, None, None, workspace, stream)


def clip_grad_norm(grads: Sequence[Optional[torch.Tensor]], max_norm: float,
                   out: Optional[Sequence[Optional[torch.Tensor]]] = None, workspace: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Scales the gradients by min(1, max_norm / norm), norm the 2-norm of all of
    them together, and returns the norm: float32 [1] on their device, not
    waited for.

    ``grads`` is a list of contiguous bf16 and float32 tensors of one device
    (None entries are passed over), changed in place, or written to ``out``, a
    tensor like each; none may be written twice.  An infinite element makes the
    factor 0, NaN everything NaN: a caller that skips such steps looks at the
    norm (infinite too where it is past float32's range).  ``workspace`` is a CUDA uint8 tensor of
    ``rmsnorm_grad_norm_workspace_bytes()`` bytes (allocated when not given).
    """
    if max_norm is None:
        raise ValueError("max_norm must be a number (grad_norm takes the norm alone)")
    return _norm_or_clip(grads, max_norm, out, workspace, stream)


def _norm_or_clip(grads, max_norm, out, workspace, stream):
    """``max_norm`` None for the norm alone."""
    if out is not None and len(out) != len(grads):
        raise ValueError(f"out holds {len(out)} tensors, grads {len(grads)}")
    if stream is None:
        r = (_fast or _bind_fast()).clip_grad_norm(grads, max_norm, out, workspace)
        if _took(r, "rmsnorm_grad_norm" if max_norm is None else "rmsnorm_clip_grads"):
            return r
    dev, device, array = _grads_arg(grads, out)
    norm = _empty((1,), torch.float32, device, stream)
    need = N.rmsnorm_grad_norm_workspace_bytes()
    workspace = _workspace(workspace, need, device, stream)
    if max_norm is None:
        _launch(dev, stream, N.rmsnorm_grad_norm, array, len(array), norm.data_ptr(), workspace.data_ptr(), need)
    else:
        _launch(dev, stream, N.rmsnorm_clip_grads, array, len(array), float(max_norm), norm.data_ptr(),
                workspace.data_ptr(), need)
    return norm


def qk_plan_for(qkv: torch.Tensor, q_heads: int, k_heads: int, head_dim: int, q_w=None, k_w=None,
                out=None) -> N.Plan:
    """The plan ``qk_norm`` would launch for these tensors."""
    tokens, xs, _ = _token_view(qkv, "qkv")
    y = qkv if out is None else out
    _, ys, _ = _token_view(y, "out")
    with torch.cuda.device(qkv.device):
        return N.rmsnorm_qk_plan_for(_ptr(qkv), _ptr(y), tokens, xs, ys, int(q_heads), int(k_heads),
                                     int(head_dim), _ptr(q_w), _ptr(k_w), dtype_code(qkv.dtype))


def plan_for(x: torch.Tensor, w=None, residual=None, out=None, residual_out=None) -> N.Plan:
    """The plan ``rms_norm`` would launch for these tensors."""
    hidden = x.shape[-1]
    rows = x.numel() // hidden
    y = out if out is not None else x
    ro = residual_out if residual_out is not None else residual
    with torch.cuda.device(x.device):
        return N.rmsnorm_plan_for(_ptr(x), _ptr(residual), _ptr(w), _ptr(y), _ptr(ro), rows, hidden,
                                  dtype_code(x.dtype))


def layer_norm(x: torch.Tensor, w: Optional[torch.Tensor] = None, b: Optional[torch.Tensor] = None,
               residual: Optional[torch.Tensor] = None, eps: float = 1e-5, out: Optional[torch.Tensor] = None,
               residual_out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None,
               plan: Optional[N.Plan] = None):
    """y = (h - mean(h)) / sqrt(var(h) + eps) * w + b over the last dimension
    (h = x, or x + residual written to ``residual_out``).  Returns y, or
    (y, residual_out) with a residual."""
    _check_tensor(x, "x", x)
    code = dtype_code(x.dtype)
    hidden = x.shape[-1]
    rows = x.numel() // hidden if hidden else 0
    for name, t in (("residual", residual), ("out", out), ("residual_out", residual_out)):
        if t is not None and t.shape != x.shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, x has {tuple(x.shape)}")
    for name, t in (("w", w), ("b", b)):
        if t is not None and tuple(t.shape) != (hidden,):
            raise ValueError(f"{name} must have shape ({hidden},)")
    y = torch.empty_like(x) if out is None else out
    if residual is not None and residual_out is None:
        residual_out = torch.empty_like(x)
    for name, t in (("w", w), ("b", b), ("residual", residual), ("out", y), ("residual_out", residual_out)):
        _check_tensor(t, name, x)
    with torch.cuda.device(x.device):
        s = stream if stream is not None else torch.cuda.current_stream(x.device)
        N.layernorm_fwd(_ptr(x), _ptr(residual), _ptr(w), _ptr(b), _ptr(y), _ptr(residual_out), rows, hidden,
                        float(eps), code, plan, s.cuda_stream)
    return (y, residual_out) if residual is not None else y


def layer_norm_plan_for(x, w=None, b=None, residual=None, out=None, residual_out=None) -> N.Plan:
    hidden = x.shape[-1]
    rows = x.numel() // hidden
    y = out if out is not None else x
    ro = residual_out if residual_out is not None else residual
    with torch.cuda.device(x.device):
        return N.layernorm_plan_for(_ptr(x), _ptr(residual), _ptr(w), _ptr(b), _ptr(y), _ptr(ro), rows, hidden,
                                    dtype_code(x.dtype))


def rms_norm_mxfp8(x: torch.Tensor, w: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
                   eps: float = 1e-6, weight_bias: float = 0.0, codes: Optional[torch.Tensor] = None,
                   scales: Optional[torch.Tensor] = None, residual_out: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None, plan: Optional[N.Plan] = None):
    """RMSNorm with MXFP8 output: returns (codes uint8 [rows, hidden] E4M3,
    scales uint8 [rows, hidden/32] E8M0) and, with a residual, residual_out."""
    _check_tensor(x, "x", x)
    code = dtype_code(x.dtype)
    hidden = x.shape[-1]
    rows = x.numel() // hidden if hidden else 0
    if w is not None and tuple(w.shape) != (hidden,):
        raise ValueError(f"w must have shape ({hidden},)")
    if codes is None:
        codes = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty(tuple(x.shape[:-1]) + (hidden // 32,), dtype=torch.uint8, device=x.device)
    if residual is not None and residual_out is None:
        residual_out = torch.empty_like(x)
    for name, t in (("w", w), ("residual", residual), ("residual_out", residual_out)):
        _check_tensor(t, name, x)
    for name, t in (("codes", codes), ("scales", scales)):
        if not t.is_cuda or t.dtype != torch.uint8 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA uint8 tensor")
    with torch.cuda.device(x.device):
        s = stream if stream is not None else torch.cuda.current_stream(x.device)
        N.rmsnorm_fwd_mxfp8(_ptr(x), _ptr(residual), _ptr(w), _ptr(codes), _ptr(scales), _ptr(residual_out), rows,
                            hidden, float(eps), float(weight_bias), code, plan, s.cuda_stream)
    return (codes, scales, residual_out) if residual is not None else (codes, scales)


def rms_norm_mxfp8_plan_for(x, w=None, residual=None) -> N.Plan:
    hidden = x.shape[-1]
    rows = x.numel() // hidden
    codes = torch.empty(1, dtype=torch.uint8, device=x.device)   # only its alignment matters
    with torch.cuda.device(x.device):
        return N.rmsnorm_mxfp8_plan_for(_ptr(x), _ptr(residual), _ptr(w), codes.data_ptr(), codes.data_ptr(),
                                        _ptr(residual), rows, hidden, dtype_code(x.dtype))


def rms_norm_nvfp4(x: torch.Tensor, w: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
                   eps: float = 1e-6, tensor_scale: float = 1.0, weight_bias: float = 0.0,
                   codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
                   residual_out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None,
                   plan: Optional[N.Plan] = None):
    """RMSNorm with NVFP4 output (bf16 input): returns (codes uint8 [rows,
    hidden/2] with two E2M1 codes a byte, scales uint8 [rows, hidden/16]
    E4M3) and, with a residual, residual_out."""
    _check_tensor(x, "x", x)
    code = dtype_code(x.dtype)
    hidden = x.shape[-1]
    rows = x.numel() // hidden if hidden else 0
    if w is not None and tuple(w.shape) != (hidden,):
        raise ValueError(f"w must have shape ({hidden},)")
    if codes is None:
        codes = torch.empty(tuple(x.shape[:-1]) + (hidden // 2,), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty(tuple(x.shape[:-1]) + (hidden // 16,), dtype=torch.uint8, device=x.device)
    if residual is not None and residual_out is None:
        residual_out = torch.empty_like(x)
    for name, t in (("w", w), ("residual", residual), ("residual_out", residual_out)):
        _check_tensor(t, name, x)
    for name, t in (("codes", codes), ("scales", scales)):
        if not t.is_cuda or t.dtype != torch.uint8 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA uint8 tensor")
    with torch.cuda.device(x.device):
        s = stream if stream is not None else torch.cuda.current_stream(x.device)
        N.rmsnorm_fwd_nvfp4(_ptr(x), _ptr(residual), _ptr(w), _ptr(codes), _ptr(scales), _ptr(residual_out), rows,
                            hidden, float(eps), float(weight_bias), float(tensor_scale), code, plan, s.cuda_stream)
    return (codes, scales, residual_out) if residual is not None else (codes, scales)


def rms_norm_nvfp4_plan_for(x, w=None, residual=None) -> N.Plan:
    hidden = x.shape[-1]
    rows = x.numel() // hidden
    codes = torch.empty(1, dtype=torch.uint8, device=x.device)
    with torch.cuda.device(x.device):
        return N.rmsnorm_nvfp4_plan_for(_ptr(x), _ptr(residual), _ptr(w), codes.data_ptr(), codes.data_ptr(),
                                        _ptr(residual), rows, hidden, dtype_code(x.dtype))
