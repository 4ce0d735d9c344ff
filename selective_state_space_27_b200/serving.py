"""Mamba-2 serving operators and norms: packed sequences, states in cache slots.

The calls that a serving step makes for every layer: on small batches they are
bound by the host, so this module marshals lean. Tensors are checked once, by the
compiled ``_binding`` (``csrc/binding.cpp``), and their pointers and strides packed
into the C structs of ``include/mambascan.h`` with :mod:`struct` (the norms' in the
compiled module); the structs' ctypes mirrors (``ConvPackedArgs`` and so on) describe
the same layouts. Outputs are allocated by the call unless ``out`` is given.

``stream``: the torch.cuda.Stream that the call runs on, in place of the current one, as
in a ``with torch.cuda.stream(stream)`` block: its scratch and outputs are that stream's.
Ordering it against the streams that make the inputs and read the outputs, and keeping the
inputs until it is done with them, is the caller's part.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import MS_BF16, MS_F32, SSD_DSTATE, SSD_HEADDIM, MambaScanError, _given, load_library, ssd_check

try:
    from . import _binding
    from ._binding import empty_like as _empty_like, rows as _rows, vector as _vector
except ImportError as e:
    raise RuntimeError("the compiled tensor checks are not built or do not fit this torch "
                       "(run python -m selective_state_space_27_b200.build)") from e

# struct layouts, field by field as in the header (P: pointer, q: int64, i: int32, f: float, B: uint8)
CONV_PACKED = struct.Struct("@4q2i Pq Pq Pqq PPP")
CONV1D = struct.Struct("@PPii")
SSD_PACKED = struct.Struct("@6q2i Pq Pq Pq Pq Pq Pq PPP Pq PPP Ii")
SSD_UPDATE = struct.Struct("@6q2i Pq Pq Pq Pq Pq Pq Pq PPPP")

_F32 = torch.float32
_DTYPES = {torch.float32: MS_F32, torch.bfloat16: MS_BF16}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_fns = {}


def _fn(name, *argtypes):
    """An entry point that takes its structs as bytes (a function object of its own)."""
    f = _fns.get(name)
    if f is None:
        f = load_library()[name]
        f.restype = ctypes.c_int
        f.argtypes = argtypes
        _fns[name] = f
    return f


_addresses = {}


def _address(name):
    """Address of an entry point, for the calls that the compiled module makes itself."""
    a = _addresses.get(name)
    if a is None:
        a = _addresses[name] = ctypes.cast(load_library()[name], ctypes.c_void_p).value
    return a


def _stream(x):
    """Handle of the current stream of x's device."""
    if not x.is_cuda:
        return 0
    if _raw_stream is not None:
        return _raw_stream(x.device.index)
    return torch.cuda.current_stream(x.device).cuda_stream


_str, _ptr = ctypes.c_char_p, ctypes.c_void_p


def _run(device, fn, *args):
    """``fn(*args, stream)`` with ``device`` current, on its current stream."""
    if device.index != _current_device():
        with torch.cuda.device(device):
            return _run(device, fn, *args)
    if _raw_stream is not None:
        s = _raw_stream(device.index)
    else:
        s = torch.cuda.current_stream(device).cuda_stream
    status = fn(*args, s)
    if status:
        raise MambaScanError(status, load_library().mamba_last_error().decode(errors="replace"))


def _cuda(x, ndim, what):
    """Device and dtype code of the leading tensor of a call."""
    if not x.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    if x.dim() != ndim:
        raise ValueError(f"{what} must have {ndim} dimensions")
    code = _DTYPES.get(x.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {x.dtype} (float32 or bfloat16)")
    return x.device, code


def _slots(nseq, state_indices, has_initial_state, device):
    """Pointers of the index table and the flags."""
    flags = 0
    if has_initial_state is not None:
        kind = torch.uint8 if has_initial_state.dtype is torch.uint8 else torch.bool
        flags = _vector("has_initial_state", has_initial_state, nseq, device, kind)
    return _vector("state_indices", state_indices, nseq, device, torch.int32), flags


def _offsets(cu_seqlens, device):
    """(pointer, number of sequences) of the row offsets."""
    n = cu_seqlens.numel()
    if n < 1:
        raise ValueError("cu_seqlens must hold nseq + 1 values")
    return _vector("cu_seqlens", cu_seqlens, n, device, torch.int32), n - 1


# ---- convolution ---------------------------------------------------------------

def _conv(x, weight, bias, silu, cu, nseq, state, state_indices, has_initial_state, out, stream):
    if stream is not None:
        return _given(stream, x, _conv, locals())
    device, code = _cuda(x, 2, "x")
    tokens, channels = shape = x.shape
    y = _empty_like(x) if out is None else out
    if weight.dim() != 2:
        raise ValueError("conv weight must be (channels, width)")
    width = weight.shape[1]
    wp, ws = _rows("conv weight", weight, torch.float32, (channels, width), device)
    if ws != width:
        raise ValueError("conv weight must be contiguous with one row per channel")
    idx, flags = _slots(nseq, state_indices, has_initial_state, device)
    st = slot_stride = row_stride = slots = 0
    if state is not None:
        slots = state.shape[0] if state.dim() == 3 else -1
        if state.shape != (slots, width - 1, channels) or state.dtype is not x.dtype or state.device != device:
            _rows("state", state, x.dtype, ("slots", width - 1, channels), device)   # (raises)
        slot_stride, row_stride, last = state.stride()
        if last != 1 and channels > 1:
            raise ValueError("state must be contiguous along the channels")
        if width <= 2:
            row_stride = max(row_stride, channels)   # (one row per slot: its stride is not used)
        st = state.data_ptr()
    xp, xs = _rows("x", x, x.dtype, shape, device)
    yp, ys = _rows("out", y, x.dtype, shape, device)
    args = CONV_PACKED.pack(tokens, channels, nseq, slots, code, 0, xp, xs, yp, ys, st, slot_stride, row_stride,
                            cu, idx, flags)
    conv = CONV1D.pack(wp, _vector("conv bias", bias, channels, device, _F32), width, 1 if silu else 0)
    _run(device, _fn("mamba_conv_packed_fwd", _str, _str, _ptr), args, conv)
    return y


def conv_packed_fwd(x, weight, cu_seqlens, bias=None, silu=True, state=None, state_indices=None,
                    has_initial_state=None, out=None, stream=None):
    """Causal depthwise convolution (and SiLU) over packed sequences.

    ``x`` (tokens, channels) float32 or bfloat16, channels contiguous: the
    sequences' tokens one behind the other, sequence s in rows
    ``cu_seqlens[s]`` to ``cu_seqlens[s + 1]`` (int32, nseq + 1 values on the
    device). ``weight`` (channels, width <= 4) and ``bias`` (channels,)
    float32. ``state`` (slots, width - 1, channels) in x's dtype holds each
    request's last width - 1 inputs, oldest first, and is updated in place:
    sequence s uses slot ``state_indices[s]`` (int32; None: slot s) and
    continues from it where ``has_initial_state[s]`` (bool; None: nowhere).
    Sequences with an index outside the cache, or an earlier sequence's, are
    skipped: their rows of the output and the cache stay as they were. Returns
    y (tokens, channels); rows of no sequence are not written. ``out`` must not
    overlap x (the same or other rows): x's rows are read again for later ones.
    """
    cu, nseq = _offsets(cu_seqlens, x.device)
    return _conv(x, weight, bias, silu, cu, nseq, state, state_indices, has_initial_state, out, stream)


def conv_packed_update(state, x, weight, bias=None, silu=True, state_indices=None, out=None, stream=None):
    """The same for one token per request: ``x`` (batch, channels), row b
    continuing from slot ``state_indices[b]`` (None: slot b) of ``state``,
    which takes the token in place. Skipped rows as :func:`conv_packed_fwd`."""
    return _conv(x, weight, bias, silu, 0, x.shape[0], state, state_indices, None, out, stream)


# ---- SSD -----------------------------------------------------------------------

def _ssd_state(state, nheads, headdim, dstate, device):
    """(slots, pointer, slot stride) of a cache of float32 states."""
    slots = state.shape[0] if state.dim() == 4 else -1
    shape = (slots, nheads, headdim, dstate)
    if slots < 0:
        shape = ("slots", nheads, headdim, dstate)
    ptr, stride = _rows("state", state, torch.float32, shape, device)
    return slots, ptr, stride


def _ssd_packed(args, x, workspace, replace):
    """The call with its device current; returns the workspace it used."""
    status, used = _binding.ssd_packed(_address("mamba_ssd_packed_fwd"), _address("mamba_ssd_packed_workspace_size"),
                                       _stream(x), args, x, workspace, replace)
    if status:
        raise MambaScanError(status, load_library().mamba_last_error().decode(errors="replace"))
    return used


def ssd_packed_fwd(x, dt, A, B, C, cu_seqlens, D=None, z=None, dt_bias=None, dt_softplus=True, state=None,
                   state_indices=None, has_initial_state=None, max_seqlen=0, out=None, workspace=None, check=True,
                   stream=None, wait_limit_us=0):
    """Mamba-2 scalar-decay SSM over packed sequences (chunked SSD on the tensor cores).

    The recurrence of :func:`ssd_fwd` for sequences packed one behind the
    other: x, z (tokens, nheads, 64), dt (tokens, nheads), B, C (tokens,
    ngroups, 128) bfloat16, the axes behind the tokens contiguous (slices of a
    wider row are fine); A, D, dt_bias (nheads,) float32. ``cu_seqlens``,
    ``state_indices`` and ``has_initial_state`` as :func:`conv_packed_fwd`;
    ``state`` (slots, nheads, 64, 128) float32 is updated in place (None:
    every sequence starts from zero and leaves no state). ``max_seqlen``: the
    longest sequence if the host knows it; it steers the schedule only.
    Returns y (tokens, nheads, 64); rows of no or of a skipped sequence are not
    written. ``out`` may be x or z itself, but overlap no other input, nor them
    in part. ``workspace``: a uint8 CUDA tensor, allocated here when None. With
    ``check`` the call synchronizes the stream (so it cannot be captured) and
    raises if the kernel reported a failed wait (a workspace that is too small
    is then replaced); without it, pass a workspace and call :func:`ssd_check`
    on it later (one that is too small is refused: the status would not be in
    it), or call ``ssd_check()`` after a number of calls without one.
    """
    if stream is not None:
        return _given(stream, x, ssd_packed_fwd, locals())
    device, code = _cuda(x, 3, "x")
    dtype = x.dtype
    tokens, nheads, headdim = shape = x.shape
    if headdim != SSD_HEADDIM:
        raise ValueError(f"x must be (tokens, nheads, {SSD_HEADDIM})")
    cu, nseq = _offsets(cu_seqlens, device)
    if B.dim() != 3:
        raise ValueError(f"B must be (tokens, ngroups, {SSD_DSTATE})")
    y = _empty_like(x) if out is None else out
    bc = (tokens, B.shape[1], SSD_DSTATE)
    idx, flags = _slots(nseq, state_indices, has_initial_state, device)
    slots, st, slot_stride = (0, 0, 0) if state is None else _ssd_state(state, nheads, headdim, SSD_DSTATE, device)
    args = SSD_PACKED.pack(
        tokens, nseq, nheads, bc[1], slots, int(max_seqlen), code, 1 if dt_softplus else 0,
        *_rows("x", x, dtype, shape, device), *_rows("dt", dt, dtype, (tokens, nheads), device),
        *_rows("B", B, dtype, bc, device), *_rows("C", C, dtype, bc, device), *_rows("z", z, dtype, shape, device),
        *_rows("out", y, dtype, shape, device), _vector("A", A, nheads, device, _F32), _vector("D", D, nheads, device, _F32),
        _vector("dt_bias", dt_bias, nheads, device, _F32), st, slot_stride, cu, idx, flags, int(wait_limit_us), 0)
    if device.index != _current_device():
        with torch.cuda.device(device):
            used = _ssd_packed(args, x, workspace, check)
    else:
        used = _ssd_packed(args, x, workspace, check)
    if check:
        ssd_check(used)
    return y


def ssd_state_update(state, x, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus=True, state_indices=None,
                     out=None, stream=None):
    """One Mamba-2 decode step for a batch of requests, states in cache slots.

    ``state`` (slots, nheads, headdim, dstate) float32 is updated in place, row
    b in slot ``state_indices[b]`` (int32; None: slot b); x, z (batch, nheads,
    headdim), dt (batch, nheads), B, C (batch, ngroups, dstate) all float32 or
    all bfloat16, the axes behind the batch contiguous; A, D, dt_bias
    (nheads,) float32. Any headdim, dstate up to 256. Returns y (batch,
    nheads, headdim); rows whose index lies outside the cache, or is an earlier
    row's, are skipped (output row and cache stay as they were). ``out`` may be
    x or z itself, but overlap no other input.
    """
    if stream is not None:
        return _given(stream, x, ssd_state_update, locals())
    device, code = _cuda(x, 3, "x")
    dtype = x.dtype
    batch, nheads, headdim = shape = x.shape
    if B.dim() != 3:
        raise ValueError("B must be (batch, ngroups, dstate)")
    y = _empty_like(x) if out is None else out
    bc = (batch, B.shape[1], B.shape[2])
    slots, st, slot_stride = _ssd_state(state, nheads, headdim, bc[2], device)
    args = SSD_UPDATE.pack(
        batch, nheads, bc[1], headdim, bc[2], slots, code, 1 if dt_softplus else 0, st, slot_stride,
        *_rows("x", x, dtype, shape, device), *_rows("dt", dt, dtype, (batch, nheads), device),
        *_rows("B", B, dtype, bc, device), *_rows("C", C, dtype, bc, device), *_rows("z", z, dtype, shape, device),
        *_rows("out", y, dtype, shape, device), _vector("A", A, nheads, device, _F32), _vector("D", D, nheads, device, _F32),
        _vector("dt_bias", dt_bias, nheads, device, _F32), _vector("state_indices", state_indices, batch, device, torch.int32))
    _run(device, _fn("mamba_ssd_state_update", _str, _ptr), args)
    return y


# ---- norm ----------------------------------------------------------------------

def norm_fwd(x, weight=None, z=None, residual=None, residual_scale=1.0, eps=1e-5, group_size=None, gate_first=True,
             out=None, residual_out=None, stream=None):
    """RMS norm of each row's groups of ``group_size`` channels (None: the row).

    v = x, or x * silu(z) with ``z`` and ``gate_first``; with ``residual``
    v = residual + residual_scale * v, which is also returned (in residual's
    dtype, x's or float32); y = v / sqrt(mean(v^2) + eps) * weight, times
    silu(z) when the gate comes last. x, z (rows, dim) float32 or bfloat16,
    rows of any stride; weight (dim,) float32 or None. Returns ``(y,
    residual_out)``, residual_out None without a residual. ``out`` may be x or
    z itself and ``residual_out`` residual; they overlap no other input.
    """
    if stream is not None:
        return _given(stream, x, norm_fwd, locals())
    if x.is_cuda and x.device.index != _current_device():
        with torch.cuda.device(x.device):
            return norm_fwd(x, weight, z, residual, residual_scale, eps, group_size, gate_first, out, residual_out)
    status, y, total = _binding.norm_fwd(_address("mamba_norm_fwd"), _stream(x), x, weight, z, residual,
                                         residual_scale, eps, group_size, gate_first, out, residual_out)
    if status:
        raise MambaScanError(status, load_library().mamba_last_error().decode(errors="replace"))
    return y, total


def norm_bwd(dy, x, weight=None, z=None, residual_out=None, dresidual_out=None, residual_scale=1.0, eps=1e-5,
             group_size=None, gate_first=True, workspace=None, stream=None):
    """Gradients of :func:`norm_fwd` for the loss sum(y * dy) + sum(residual_out * dresidual_out).

    ``residual_out`` is the sum that the forward returned (None: it had no
    residual); ``dresidual_out``, in its dtype, may be None. Returns a dict:
    dx, dz (None without z) in x's dtype, dresidual (None without a residual)
    in the residual's, dweight (dim,) float32 (None without weight).
    ``workspace``: optional uint8 CUDA tensor, allocated here when needed.
    """
    if stream is not None:
        return _given(stream, x, norm_bwd, locals())
    if x.is_cuda and x.device.index != _current_device():
        with torch.cuda.device(x.device):
            return norm_bwd(dy, x, weight, z, residual_out, dresidual_out, residual_scale, eps, group_size, gate_first,
                            workspace)
    status, dx, dz, dresidual, dweight = _binding.norm_bwd(
        _address("mamba_norm_bwd"), _address("mamba_norm_bwd_workspace_size"), _stream(x), dy, x, weight, z,
        residual_out, dresidual_out, residual_scale, eps, group_size, gate_first, workspace)
    if status:
        raise MambaScanError(status, load_library().mamba_last_error().decode(errors="replace"))
    return {"dx": dx, "dz": dz, "dresidual": dresidual, "dweight": dweight}
