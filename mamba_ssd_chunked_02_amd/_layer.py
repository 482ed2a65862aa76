"""ctypes binding of the operators around the scan (include/ssd.h): layer
norm, the short causal convolution, the selective scan and the single-token
forms.  Argument marshalling only, as in ``_binding``: every operator runs in
the HIP library on torch's current stream of the tensors' device, outputs and
workspaces are allocated with torch.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from ._binding import _DTYPES, SsdDims, SsdError, SsdLayout, _apart, library

_P = ctypes.c_void_p
_I32, _I64, _F32, _SIZE = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t


class SsdNormDims(ctypes.Structure):
    """Mirror of ``ssd_norm_dims`` in include/ssd.h."""
    _fields_ = [("rows", _I64), ("x_row", _I64), ("y_row", _I64), ("dy_row", _I64),
                ("width", _I32), ("dtype", _I32), ("eps", _F32), ("reserved", _I32)]


class SsdConvDims(ctypes.Structure):
    """Mirror of ``ssd_conv_dims``."""
    _fields_ = [("batch", _I32), ("seqlen", _I64), ("channels", _I32), ("width", _I32),
                ("nseq", _I32), ("dtype", _I32)]


class SsdConvLayout(ctypes.Structure):
    """Mirror of ``ssd_conv_layout`` (element strides)."""
    _fields_ = [("x_token", _I64), ("y_token", _I64), ("dy_token", _I64)]


class SsdSelscanDims(ctypes.Structure):
    """Mirror of ``ssd_selscan_dims``."""
    _fields_ = [("batch", _I32), ("seqlen", _I64), ("channels", _I32), ("d_state", _I32),
                ("ngroups", _I32), ("nseq", _I32), ("dtype", _I32), ("reserved", _I32)]


class SsdSelscanLayout(ctypes.Structure):
    """Mirror of ``ssd_selscan_layout`` (element strides)."""
    _fields_ = [(n, _I64) for n in ("x_token", "d_raw_token", "z_token", "B_token", "B_group",
                                    "C_token", "C_group", "y_token", "dy_token")]


@functools.lru_cache(maxsize=1024)
def _struct(cls, *fields):
    """The struct of these sizes; the library only reads it, so calls of the same
    sizes share one."""
    return cls(*fields)


def _pointer(struct):
    return ctypes.POINTER(struct)


_SIGNATURES = {
    "ssd_norm_fwd": [_pointer(SsdNormDims)] + [_P] * 7,
    "ssd_norm_bwd": [_pointer(SsdNormDims)] + [_P] * 9 + [_SIZE, _P],
    "ssd_conv_fwd": [_pointer(SsdConvDims), _pointer(SsdConvLayout)] + [_P] * 8,
    "ssd_conv_bwd": [_pointer(SsdConvDims), _pointer(SsdConvLayout)] + [_P] * 12 + [_SIZE, _P],
    "ssd_conv_step": [_pointer(SsdConvDims), _pointer(SsdConvLayout)] + [_P] * 5 + [_I32] + [_P] * 3,
    "ssd_selscan_fwd": [_pointer(SsdSelscanDims), _pointer(SsdSelscanLayout)] + [_P] * 13
                       + [_SIZE, _P],
    "ssd_selscan_bwd": [_pointer(SsdSelscanDims), _pointer(SsdSelscanLayout)] + [_P] * 22
                       + [_SIZE, _P],
    "ssd_selscan_step": [_pointer(SsdSelscanDims), _pointer(SsdSelscanLayout)] + [_P] * 10
                        + [_I32] + [_P] * 3,
    "ssd_step": [_pointer(SsdDims), _pointer(SsdLayout), _P, _P, _F32, _P, _P, _P, _P, _I32,
                 _P, _P, _P],
}
_WORKSPACES = {
    "ssd_norm_bwd_workspace_bytes": SsdNormDims,
    "ssd_conv_bwd_workspace_bytes": SsdConvDims,
    "ssd_selscan_fwd_workspace_bytes": SsdSelscanDims,
    "ssd_selscan_bwd_workspace_bytes": SsdSelscanDims,
}
_entries = {}


def _entry(name):
    f = _entries.get(name)
    if f is None:
        f = getattr(library(), name)
        if name in _WORKSPACES:
            f.restype, f.argtypes = _SIZE, [_pointer(_WORKSPACES[name])]
        else:
            f.restype, f.argtypes = ctypes.c_int, _SIGNATURES[name]
        _entries[name] = f
    return f


# The current stream of a device as an integer.  torch.cuda.current_stream
# builds a Stream object first, 2 us of a call whose kernel takes 5.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _launch(name, x, *args):
    """Call the entry point on the current stream of x's device."""
    f = _entries.get(name) or _entry(name)
    index = x.get_device()
    if index < 0:
        raise ValueError(f"{name} needs tensors on a GPU, got {x.device}")
    if index == torch.cuda.current_device():
        rc = f(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            rc = f(*args, _raw_stream(index))
    if rc != 0:
        raise SsdError(rc, name)


def _at(t):
    return None if t is None else t.data_ptr()


def _dtype_of(x, name):
    code = _DTYPES.get(x.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {x.dtype} of {name}")
    return code


def _same(x, *named):
    """(tensor, name) pairs: tensors of x's dtype on x's device."""
    dt, dev = x.dtype, x.get_device()
    for t, name in named:
        if t is not None and (t.dtype is not dt or t.get_device() != dev):
            raise ValueError(f"{name} must be on {x.device} with dtype {x.dtype}")


_FLOAT = torch.float32


def _floats(x, *named):
    """(tensor, shape, name): contiguous float32 tensors on x's device."""
    dev = x.get_device()
    for t, shape, name in named:
        if t is not None and (t.dtype is not _FLOAT or t.get_device() != dev
                              or t.shape != shape or not t.is_contiguous()):
            raise ValueError(f"{name} must be contiguous float32 {list(shape)} on {x.device}")


# Of a dimension of size 1 torch keeps any stride; the helpers below give the dense one.

def _tokens(t, name, shape):
    """Token stride of a [b, L, E] tensor whose rows are contiguous and whose
    batch rows are L tokens apart."""
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {list(shape)}")
    b, L, E = shape
    if t.is_contiguous() or t.numel() == 0:
        return E
    sb, st, se = t.stride()
    if E > 1 and se != 1:
        raise ValueError(f"{name} needs a contiguous last dimension")
    if L == 1:
        # one token a row: the batch stride is the token stride
        return sb if b > 1 else E
    if b > 1 and sb != L * st:
        raise ValueError(f"{name} needs batch stride L * token stride")
    return st


def _groups(t, name, shape):
    """(token, group) strides of a [b, L, G, N] tensor."""
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {list(shape)}")
    b, L, G, N = shape
    if t.is_contiguous() or t.numel() == 0:
        return G * N, N
    sb, st, sg, sn = t.stride()
    if N > 1 and sn != 1:
        raise ValueError(f"{name} needs a contiguous last dimension")
    if G == 1:
        sg = N
    if L == 1:
        return (sb if b > 1 else G * N), sg
    if b > 1 and sb != L * st:
        raise ValueError(f"{name} needs batch stride L * token stride")
    return st, sg


def _rows(t, name, shape):
    """Row stride of a [b, E] tensor with contiguous rows."""
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {list(shape)}")
    if t.is_contiguous():
        return shape[1]
    if shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} needs a contiguous last dimension")
    return t.stride(0) if shape[0] > 1 else shape[1]


def _heads(t, name, shape):
    """(row, head) strides of a [b, H, P] tensor with contiguous last dimension."""
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {list(shape)}")
    b, H, P = shape
    if t.is_contiguous():
        return H * P, P
    if P > 1 and t.stride(2) != 1:
        raise ValueError(f"{name} needs a contiguous last dimension")
    return t.stride(0) if b > 1 else H * P, t.stride(1) if H > 1 else P


def _output(x):
    """An uninitialized contiguous tensor of x's shape and dtype (empty_like is the
    cheapest way to one, but keeps a dense x's own order)."""
    return torch.empty_like(x) if x.is_contiguous() else x.new_empty(x.shape)


def _like(t):
    """An uninitialized tensor with t's shape and strides."""
    return torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device=t.device)


def _workspace(name, dims, x, given):
    """(tensor to keep, address, bytes) of the workspace: the caller's, or one of the
    size that the library names (none where that is 0)."""
    if given is None:
        need = _entry(name)(ctypes.byref(dims))
        if need == 0:
            return None, None, 0
        given = torch.empty(need, dtype=torch.uint8, device=x.device)
        return given, given.data_ptr(), need
    if given.get_device() != x.get_device() or given.device.type != x.device.type \
            or not given.is_contiguous():
        raise ValueError(f"workspace must be contiguous on {x.device}")
    return given, given.data_ptr(), given.nbytes


def _sequences(x, cu_seqlens, b):
    """cu_seqlens checked, and the number of sequences."""
    if cu_seqlens is None:
        return None, b
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.device != x.device or cu_seqlens.dim() != 1:
        raise ValueError("cu_seqlens must be a 1-D int32 tensor on the same device")
    if b != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens needs batch 1 and at least one sequence")
    cu_seqlens = cu_seqlens.contiguous()
    return cu_seqlens, cu_seqlens.numel() - 1


def _pools(x, state, new_state, row, dtype, slots):
    """The pools of a single-token call: ``state`` [nslots, *row], and
    ``new_state`` (``state`` itself where not given)."""
    if new_state is None:
        new_state = state
    dev, shape = x.get_device(), state.shape
    if new_state.shape != shape:
        raise ValueError("state and new_state must have the same shape")
    if shape[1:] != row or state.dtype is not dtype or new_state.dtype is not dtype \
            or state.get_device() != dev or new_state.get_device() != dev \
            or not state.is_contiguous() or not new_state.is_contiguous():
        raise ValueError(f"state and new_state must be contiguous {dtype} [nslots, "
                         f"{', '.join(map(str, row))}] on {x.device}")
    if slots is None:
        if shape[0] < x.shape[0]:
            raise ValueError("without slots the pool needs a row for every sequence")
    elif slots.dtype is not torch.int32 or slots.get_device() != dev or slots.shape != x.shape[:1] \
            or not slots.is_contiguous():
        raise ValueError(f"slots must be contiguous int32 [{x.shape[0]}] on {x.device}")
    return new_state


# ---- layer norm ----------------------------------------------------------------------------

def _matrix(t, name, width):
    """t [..., width] as rows: (rows, row stride)."""
    if t.dim() < 1 or t.shape[-1] != width:
        raise ValueError(f"{name} must have a last dimension of {width}")
    if t.is_contiguous():
        return t.numel() // width, width
    m = t.view(-1, width)  # raises where the leading dimensions do not form one stride
    if width > 1 and m.stride(1) != 1:
        raise ValueError(f"{name} needs a contiguous last dimension")
    return m.shape[0], (m.stride(0) if m.shape[0] > 1 else width)


def ssd_norm_fwd(x, weight=None, bias=None, eps=1e-5, y=None):
    """Layer norm over x's last dimension (bf16 or fp32; rows may be strided).
    weight, bias [width] fp32 or None; ``y`` may be preallocated (x itself for
    in place).  Returns (y, mean, rstd) with mean and rstd fp32 of x's leading
    shape, for ``ssd_norm_bwd``."""
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x [..., width] expected")
    width = x.shape[-1]
    code = _dtype_of(x, "x")
    _floats(x, (weight, (width,), "weight"), (bias, (width,), "bias"))
    rows, xs = _matrix(x, "x", width)
    if y is None:
        y, ys = _output(x), width
    else:
        _same(x, (y, "y"))
        if y.shape != x.shape:
            raise ValueError("y must have x's shape")
        ys = _matrix(y, "y", width)[1]
    mean, rstd = torch.empty((2,) + x.shape[:-1], dtype=torch.float32, device=x.device).unbind(0)
    dims = _struct(SsdNormDims, rows, xs, ys, width, width, code, eps, 0)
    _launch("ssd_norm_fwd", x, dims, x.data_ptr(), _at(weight), _at(bias), y.data_ptr(),
            mean.data_ptr(), rstd.data_ptr())
    return y, mean, rstd


def ssd_norm_bwd(x, weight, mean, rstd, dy, workspace=None):
    """Gradients of ``ssd_norm_fwd`` from its x, weight (or None), mean and
    rstd: a dict with dx (laid out like x), dweight and dbias [width] fp32."""
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x [..., width] expected")
    width = x.shape[-1]
    code = _dtype_of(x, "x")
    _same(x, (dy, "dy"))
    if dy.shape != x.shape:
        raise ValueError("dy must have x's shape")
    _floats(x, (weight, (width,), "weight"), (mean, x.shape[:-1], "mean"), (rstd, x.shape[:-1], "rstd"))
    rows, xs = _matrix(x, "x", width)
    dx = _like(x)
    dweight, dbias = torch.empty((2, width), dtype=torch.float32, device=x.device).unbind(0)
    dims = _struct(SsdNormDims, rows, xs, width, _matrix(dy, "dy", width)[1], width, code, 0.0, 0)
    workspace, *ws = _workspace("ssd_norm_bwd_workspace_bytes", dims, x, workspace)
    _launch("ssd_norm_bwd", x, dims, x.data_ptr(), _at(weight), mean.data_ptr(), rstd.data_ptr(),
            dy.data_ptr(), dx.data_ptr(), dweight.data_ptr(), dbias.data_ptr(),
            *ws)
    return {"dx": dx, "dweight": dweight, "dbias": dbias}


# ---- convolution ---------------------------------------------------------------------------

def _conv_arguments(x, weight, bias, init_state, cu_seqlens, dims_of):
    if x.dim() != dims_of or weight.dim() != 2 or x.shape[-1] != weight.shape[1]:
        raise ValueError("x [b, L, E] ([b, E] for one token) and weight [W, E] expected")
    W, E = weight.shape
    code = _dtype_of(x, "x")
    _floats(x, (weight, (W, E), "weight"), (bias, (E,), "bias"))
    cu, S = _sequences(x, cu_seqlens, x.shape[0])
    if init_state is not None:
        _same(x, (init_state, "init_state"))
        if init_state.shape != (S, W - 1, E) or not init_state.is_contiguous():
            raise ValueError(f"init_state must be contiguous [{S}, {W - 1}, {E}]")
    return W, E, code, cu, S


def ssd_conv_fwd(x, weight, bias=None, init_state=None, cu_seqlens=None, y=None,
                 final_state=True):
    """Short causal convolution with bias and SiLU per channel.

    x [b, L, E] (bf16 or fp32, strided tokens allowed), weight [W, E] and bias
    [E] fp32 (W 2 to 4; the last tap meets the token itself), init_state
    [S, W - 1, E] of x's dtype or None for zeros; cu_seqlens int32 [nseq + 1]
    (b must be 1) or None.  ``y`` may be preallocated; ``final_state``: True,
    False or a [S, W - 1, E] tensor to fill.  Returns (y, final_state or None)."""
    W, E, code, cu, S = _conv_arguments(x, weight, bias, init_state, cu_seqlens, 3)
    b, L, _ = x.shape
    xs = _tokens(x, "x", x.shape)
    if y is None:
        y, ys = _output(x), E
    else:
        _same(x, (y, "y"))
        ys = _tokens(y, "y", x.shape)
    if final_state is True:
        final_state = x.new_empty((S, W - 1, E))
    elif final_state is False:
        final_state = None
    elif final_state is not None:
        _same(x, (final_state, "final_state"))
        if final_state.shape != (S, W - 1, E) or not final_state.is_contiguous():
            raise ValueError(f"final_state must be contiguous [{S}, {W - 1}, {E}]")
    dims = _struct(SsdConvDims, b, L, E, W, 0 if cu is None else S, code)
    _launch("ssd_conv_fwd", x, dims, _struct(SsdConvLayout, xs, ys, E), x.data_ptr(),
            weight.data_ptr(), _at(bias), _at(init_state), _at(cu), y.data_ptr(), _at(final_state))
    return y, final_state


def ssd_conv_bwd(x, weight, bias, dy, init_state=None, cu_seqlens=None, d_final=None,
                 workspace=None):
    """Gradients of ``ssd_conv_fwd``: a dict with dx (laid out like x), dweight
    [W, E], dbias [E] (fp32) and dinit_state [S, W - 1, E] (x's dtype; the
    gradient at zeros without an init_state).  ``d_final`` is the gradient of
    final_state or None for zeros."""
    W, E, code, cu, S = _conv_arguments(x, weight, bias, init_state, cu_seqlens, 3)
    b, L, _ = x.shape
    _same(x, (dy, "dy"), (d_final, "d_final"))
    if d_final is not None and (d_final.shape != (S, W - 1, E) or not d_final.is_contiguous()):
        raise ValueError(f"d_final must be contiguous [{S}, {W - 1}, {E}]")
    lay = _struct(SsdConvLayout, _tokens(x, "x", x.shape), E, _tokens(dy, "dy", x.shape))
    dx = _like(x)
    sums = torch.empty((W + 1, E), dtype=torch.float32, device=x.device)
    dinit = torch.empty((S, W - 1, E), dtype=x.dtype, device=x.device)
    dims = _struct(SsdConvDims, b, L, E, W, 0 if cu is None else S, code)
    workspace, *ws = _workspace("ssd_conv_bwd_workspace_bytes", dims, x, workspace)
    dweight, dbias = sums[:W], sums[W]
    _launch("ssd_conv_bwd", x, dims, lay, x.data_ptr(), weight.data_ptr(), _at(bias),
            _at(init_state), _at(cu), dy.data_ptr(), _at(d_final), dx.data_ptr(),
            dweight.data_ptr(), dbias.data_ptr(), dinit.data_ptr(), *ws)
    return {"dx": dx, "dweight": dweight, "dbias": dbias, "dinit_state": dinit}


def ssd_conv_step(x, state, weight, bias=None, slots=None, new_state=None, y=None):
    """One new token x [b, E] for each of b sequences: their states are the rows
    ``slots`` (int32 [b], all different; None: row i) of the pool ``state``
    [nslots, W - 1, E].  The new states go to the same rows of ``new_state``
    (None: ``state`` itself, in place).  A slot outside the pool marks a padding
    row: its y is 0 and no state is touched.  Returns y [b, E]."""
    W, E, code, _, _ = _conv_arguments(x, weight, bias, None, None, 2)
    new_state = _pools(x, state, new_state, (W - 1, E), x.dtype, slots)
    xs = _rows(x, "x", x.shape)
    if y is None:
        y, ys = _output(x), E
    else:
        _same(x, (y, "y"))
        ys = _rows(y, "y", x.shape)
    dims = _struct(SsdConvDims, x.shape[0], 1, E, W, 0, code)
    _launch("ssd_conv_step", x, dims, _struct(SsdConvLayout, xs, ys, E), x.data_ptr(),
            weight.data_ptr(), _at(bias), state.data_ptr(), _at(slots), state.shape[0],
            y.data_ptr(), new_state.data_ptr())
    return y


# ---- selective scan ------------------------------------------------------------------------

def _selscan_arguments(x, d_raw, d_init, A, B, C, D, z, cu_seqlens, y, dy):
    if x.dim() != 3 or A.dim() != 2 or B.dim() != 4:
        raise ValueError("x [b, L, E], A [N, E] and B, C [b, L, G, N] expected")
    b, L, E = x.shape
    N, G = A.shape[0], B.shape[2]
    code = _dtype_of(x, "x")
    _same(x, (d_raw, "d_raw"), (B, "B"), (C, "C"), (z, "z"), (y, "y"), (dy, "dy"))
    _floats(x, (d_init, (E,), "d_init"), (A, (N, E), "A"), (D, (E,), "D"))
    cu, S = _sequences(x, cu_seqlens, b)
    shape = (b, L, G, N)
    lay = _struct(
        SsdSelscanLayout, _tokens(x, "x", x.shape), _tokens(d_raw, "d_raw", x.shape),
        E if z is None else _tokens(z, "z", x.shape), *_groups(B, "B", shape),
        *_groups(C, "C", shape), E if y is None else _tokens(y, "y", x.shape),
        E if dy is None else _tokens(dy, "dy", x.shape))
    dims = _struct(SsdSelscanDims, b, L, E, N, G, 0 if cu is None else S, code, 0)
    return dims, lay, cu, (S, N, E)


def ssd_selscan_fwd(x, d_raw, d_init, A, B, C, D=None, z=None, init_state=None, cu_seqlens=None,
                    y=None, final_state=True, workspace=None):
    """Selective scan with a decay per channel and state entry:
    ``d = softplus(d_raw + d_init)``, ``h = exp(d A) h + d B x``,
    ``y = (C h + D x) silu(z)``.

    x, d_raw, z [b, L, E] and B, C [b, L, G, N] (bf16 or fp32, one dtype, strided
    tokens allowed; N up to 64), d_init, D [E] and A [N, E] fp32, init_state
    [S, N, E] fp32 or None for zeros; D and z may be None.  cu_seqlens int32
    [nseq + 1] (b must be 1) or None.  ``y`` may be preallocated; ``final_state``:
    True, False or a [S, N, E] fp32 tensor to fill.  Returns (y, final_state or
    None)."""
    dims, lay, cu, state = _selscan_arguments(x, d_raw, d_init, A, B, C, D, z, cu_seqlens, y, None)
    _floats(x, (init_state, state, "init_state"))
    if y is None:
        y = _output(x)
    if final_state is True:
        final_state = torch.empty(state, dtype=torch.float32, device=x.device)
    elif final_state is False:
        final_state = None
    else:
        _floats(x, (final_state, state, "final_state"))
    workspace, *ws = _workspace("ssd_selscan_fwd_workspace_bytes", dims, x, workspace)
    _launch("ssd_selscan_fwd", x, dims, lay, x.data_ptr(), d_raw.data_ptr(), _at(d_init), _at(A), _at(B),
            _at(C), _at(D), _at(z), _at(init_state), _at(cu), y.data_ptr(), _at(final_state),
            *ws)
    return y, final_state


def ssd_selscan_bwd(x, d_raw, d_init, A, B, C, dy, D=None, z=None, init_state=None,
                    cu_seqlens=None, d_final=None, workspace=None):
    """Gradients of ``ssd_selscan_fwd``: a dict with dx, dd_raw, dB, dC (and dz
    with a gate), each laid out like its input (dB and dC dense where B or C is
    an expanded view: every token and group has its own gradient), and in fp32
    dA [N, E], dd_init, dD [E] (the gradient at zeros without a D) and
    dinit_state [S, N, E] (at zeros without an init_state).  ``d_final`` is the
    gradient of final_state or None for zeros."""
    B, C = _apart(B), _apart(C)
    dims, lay, cu, state = _selscan_arguments(x, d_raw, d_init, A, B, C, D, z, cu_seqlens, None, dy)
    _floats(x, (init_state, state, "init_state"), (d_final, state, "d_final"))
    N, E = A.shape
    g = {"dx": _like(x), "dd_raw": _like(d_raw), "dB": _like(B), "dC": _like(C)}
    if z is not None:
        g["dz"] = _like(z)
    sums = torch.empty((N + 2, E), dtype=torch.float32, device=x.device)
    g |= {"dA": sums[:N], "dD": sums[N], "dd_init": sums[N + 1],
          "dinit_state": torch.empty(state, dtype=torch.float32, device=x.device)}
    workspace, *ws = _workspace("ssd_selscan_bwd_workspace_bytes", dims, x, workspace)
    _launch("ssd_selscan_bwd", x, dims, lay, x.data_ptr(), d_raw.data_ptr(), _at(d_init), _at(A), _at(B),
            _at(C), _at(D), _at(z), _at(init_state), _at(cu), dy.data_ptr(), _at(d_final),
            _at(g["dx"]), _at(g["dd_raw"]), _at(g["dB"]), _at(g["dC"]), _at(g.get("dz")),
            _at(g["dA"]), _at(g["dD"]), _at(g["dd_init"]), _at(g["dinit_state"]),
            *ws)
    return g


def ssd_selscan_step(x, d_raw, d_init, A, B, C, state, D=None, z=None, slots=None, new_state=None,
                     y=None):
    """One new token of the selective scan for each of b sequences: x, d_raw, z
    [b, E], B, C [b, G, N]; state [nslots, N, E] fp32, slots and new_state as
    ``ssd_conv_step``'s.  Returns y [b, E]."""
    if x.dim() != 2 or A.dim() != 2 or B.dim() != 3:
        raise ValueError("x [b, E], A [N, E] and B, C [b, G, N] expected")
    b, E = x.shape
    N, G = A.shape[0], B.shape[1]
    code = _dtype_of(x, "x")
    _same(x, (d_raw, "d_raw"), (B, "B"), (C, "C"), (z, "z"))
    _floats(x, (d_init, (E,), "d_init"), (A, (N, E), "A"), (D, (E,), "D"))
    new_state = _pools(x, state, new_state, (N, E), torch.float32, slots)
    if y is None:
        y, ys = _output(x), E
    else:
        _same(x, (y, "y"))
        ys = _rows(y, "y", x.shape)
    lay = _struct(
        SsdSelscanLayout, _rows(x, "x", x.shape), _rows(d_raw, "d_raw", x.shape),
        E if z is None else _rows(z, "z", x.shape), *_heads(B, "B", (b, G, N)),
        *_heads(C, "C", (b, G, N)), ys, E)
    dims = _struct(SsdSelscanDims, b, 1, E, N, G, 0, code, 0)
    _launch("ssd_selscan_step", x, dims, lay, x.data_ptr(), d_raw.data_ptr(), _at(d_init), _at(A), _at(B),
            _at(C), _at(D), _at(z), state.data_ptr(), _at(slots), state.shape[0], y.data_ptr(),
            new_state.data_ptr())
    return y


# ---- SSD, one token ------------------------------------------------------------------------

def ssd_step(x, d_raw, d_init, B, C, state, slots=None, new_state=None, y=None):
    """One new token of ``ssd_fwd``'s scan for each of b sequences: x [b, H, P],
    d_raw [b, H], B, C [b, G, N] (bf16 or fp32; strided views allowed); state
    [nslots, H, N, P] fp32, slots and new_state as ``ssd_conv_step``'s.  Returns
    y [b, H, P]."""
    if x.dim() != 3 or d_raw.dim() != 2 or B.dim() != 3:
        raise ValueError("x [b, H, P], d_raw [b, H] and B, C [b, G, N] expected")
    b, H, P = x.shape
    G, N = B.shape[1], B.shape[2]
    code = _dtype_of(x, "x")
    _same(x, (d_raw, "d_raw"), (B, "B"), (C, "C"))
    if d_raw.shape != (b, H):
        raise ValueError(f"d_raw must have shape [{b}, {H}]")
    new_state = _pools(x, state, new_state, (H, N, P), torch.float32, slots)
    if y is None:
        y = _output(x)
    else:
        _same(x, (y, "y"))
    raw = (H, 1) if d_raw.is_contiguous() else (d_raw.stride(0) if b > 1 else H,
                                                d_raw.stride(1) if H > 1 else 1)
    lay = _struct(SsdLayout, *_heads(x, "x", x.shape), *raw, *_heads(B, "B", (b, G, N)),
                    *_heads(C, "C", (b, G, N)), *_heads(y, "y", x.shape))
    dims = _struct(SsdDims, b, 1, H, P, N, G, 64, 0, code)
    _launch("ssd_step", x, dims, lay, x.data_ptr(), d_raw.data_ptr(), float(d_init), _at(B), _at(C),
            state.data_ptr(), _at(slots), state.shape[0], y.data_ptr(), new_state.data_ptr())
    return y
