"""The operators around the mixer: norm, short convolution, selective scan.

Thin wrappers over the C ABI, as the package's own module has them for the
mixer: they check devices, types and shapes, allocate outputs and scratch with
PyTorch, and pass device pointers and the current stream.

    y, scale, h   = norm_fwd(x, weight, residual, out8=True)   # block entry
    q, conv_state = conv_fwd(xq, w, bias, heads=H, want_state=True)  # [B,H,L,d]
    y, h_L        = scan_fwd(x, dt, A, Bm, Cm, D, z, dt_bias)   # [B,L,C]

and ``norm_bwd``, ``conv_bwd``, ``scan_bwd`` for training, ``conv_step`` and
``scan_step`` for one token.  Formulas and layouts are in ``include/efla.h``.
Parameters (weight, bias, A, D, dt_bias) and scan states are float32;
activations are float32 or bfloat16.  Tokens of x, z, dt, Bm and Cm may lie
apart in memory (column slices of one projection); all else is contiguous.
``lengths`` [B] int32: tokens from there on are padding and come out as zeros.
"""
from __future__ import annotations

import ctypes

import torch

from . import EFLA_BF16, EFLA_F32, _check, _lib

_p, _i, _l, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_float, ctypes.c_size_t
_lib.efla_norm_fwd.argtypes = [_p, _i, _p, _i, _p, _f, _p, _p, _p, _i, _p, _l, _i, _p]
_lib.efla_norm_bwd_workspace_size.restype = _sz
_lib.efla_norm_bwd_workspace_size.argtypes = [_l, _i]
_lib.efla_norm_bwd.argtypes = [_p, _i, _p, _i, _p, _f, _p, _p, _p, _p, _l, _i, _p, _sz, _p]
_lib.efla_conv_fwd.argtypes = [_p, _l, _i, _p, _p, _p, _p, _i, _p, _i, _p, _i, _i, _i, _i, _p]
_lib.efla_conv_bwd_workspace_size.restype = _sz
_lib.efla_conv_bwd_workspace_size.argtypes = [_i, _i, _i, _i]
_lib.efla_conv_bwd.argtypes = [_p, _p, _l, _i, _p, _p, _p, _p, _i, _i, _p, _p, _p, _p, _p, _i, _i, _i, _i, _p, _sz, _p]
_lib.efla_conv_step.argtypes = [_p, _l, _i, _p, _p, _p, _i, _p, _i, _i, _i, _p]
_lib.efla_scan_fwd_workspace_size.restype = _sz
_lib.efla_scan_fwd_workspace_size.argtypes = [_i, _i, _i, _i, _i]
_lib.efla_scan_fwd.argtypes = [_p, _l, _p, _l, _p, _p, _l, _p, _l, _p, _p, _l, _p, _p, _p, _i, _i, _p, _p,
                               _i, _i, _i, _i, _i, _p, _sz, _p]
_lib.efla_scan_bwd_workspace_size.restype = _sz
_lib.efla_scan_bwd_workspace_size.argtypes = [_i, _i, _i, _i, _i]
_lib.efla_scan_bwd.argtypes = [_p, _p, _l, _p, _l, _p, _p, _l, _p, _l, _p, _p, _l, _p, _p, _p, _p, _i, _i,
                               _p, _p, _p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _p, _sz, _p]
_lib.efla_scan_step.argtypes = [_p, _l, _p, _l, _p, _p, _l, _p, _l, _p, _p, _l, _p, _i, _i, _p, _p, _i, _i, _i, _i, _p]
for _name in ("norm_fwd", "norm_bwd", "conv_fwd", "conv_bwd", "conv_step", "scan_fwd", "scan_bwd", "scan_step"):
    getattr(_lib, "efla_" + _name).restype = _i

_F32 = torch.float32
_CODE = {torch.float32: EFLA_F32, torch.bfloat16: EFLA_BF16}
# current_stream() and current_device() build objects and check initialisation: several microseconds that a
# one-token step does not have.  A tensor on the device is proof of the latter.
_raw_stream, _get_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice


def _refuse(t, shape, dtype, dev, name):
    if t.shape != shape or t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, as the first argument is")
    raise ValueError(f"{name} must be contiguous")


def _want(t, shape, dtype, dev, name):
    """A contiguous tensor of this shape, type and device, or None."""
    if t is not None and (t.shape != shape or t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous()):
        _refuse(t, shape, dtype, dev, name)


def _act(t, name):
    """Device index and type of the activation that the others are held to."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in _CODE:
        raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    return t.get_device(), t.dtype


def _rows(t, shape, lead, dtype, dev, name):
    """Elements from one token to the next of a tensor whose first ``lead``
    dimensions count tokens: each token's values are contiguous, and the
    tokens evenly spaced."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev:
        _refuse(t, shape, dtype, dev, name)
    width = 1
    for n in shape[lead:]:
        width *= n
    if t.is_contiguous():
        return width
    stride = t.stride()
    step, ld = 1, None
    for i in range(len(shape) - 1, lead - 1, -1):  # inside a token
        if shape[i] != 1 and stride[i] != step:
            raise ValueError(f"the values of one token of {name} must be contiguous")
        step *= shape[i]
    for i in range(lead - 1, -1, -1):  # from token to token
        if shape[i] == 1:
            continue
        if ld is None:
            ld, step = stride[i], stride[i] * shape[i]
            if ld < width:
                raise ValueError(f"the tokens of {name} must not overlap")
        elif stride[i] != step:
            raise ValueError(f"the tokens of {name} must be evenly spaced over the batch")
        else:
            step *= shape[i]
    return width if ld is None else ld


def _at(t):
    return None if t is None else t.data_ptr()


def _call(fn, dev, *args):
    """Call with the current stream of the tensors' device, made current if it is not."""
    if _get_device() == dev:
        status = fn(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _raw_stream(dev))
    if status:
        _check(status, fn.__name__)


def _scratch(need, workspace, x):
    """(workspace, its bytes): the caller's where it is large enough, else a new one on x's device."""
    if not need:
        return None, 0
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        return x.new_empty(need, dtype=torch.uint8), need
    if workspace.device != x.device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on {x.device}")
    return workspace, workspace.numel() * workspace.element_size()


# ------------------------------------------------------------------------------------------------- norm

def norm_fwd(x, weight, residual=None, eps: float = 1e-6, out8: bool = False, group: int = 128, y=None, scale=None,
             res_out=None):
    """Root-mean-square norm over the last dimension of ``h = x + residual``.
    Returns (y, scale, res_out): y in x's dtype, or with ``out8`` in
    float8_e4m3fn with one float32 scale per ``group`` columns (128, or 0: per
    row) in [..., ceil(C / group)]; scale is None otherwise.  res_out is h in
    the residual's dtype (x's, or float32), None without a residual; it may be
    passed as ``residual`` itself, to update the stream in place."""
    dev, T = _act(x, "x")
    shape = x.shape
    if not shape:
        raise ValueError("x must have a last dimension to norm over")
    C = shape[-1]
    rows = x.numel() // C if C else 0
    _want(x, shape, T, dev, "x")
    _want(weight, (C,), _F32, dev, "weight")
    if residual is not None:
        if residual.dtype is not T and residual.dtype is not _F32:
            raise TypeError(f"residual must be float32 or {T}, got {residual.dtype}")
        _want(residual, shape, residual.dtype, dev, "residual")
        if res_out is None:
            res_out = torch.empty_like(residual)
        else:
            _want(res_out, shape, residual.dtype, dev, "res_out")
    elif res_out is not None:
        raise ValueError("res_out needs a residual")
    if group not in (0, 128):
        raise ValueError("group must be 128 or 0")
    Y = torch.float8_e4m3fn if out8 else T
    if y is None:
        y = x.new_empty(shape, dtype=Y)
    else:
        _want(y, shape, Y, dev, "y")
    if out8:
        groups = shape[:-1] + ((C + 127) // 128 if group else 1,)
        if scale is None:
            scale = x.new_empty(groups, dtype=_F32)
        else:
            _want(scale, groups, _F32, dev, "scale")
    elif scale is not None:
        raise ValueError("scale is written with out8 only")
    _call(_lib.efla_norm_fwd, dev, x.data_ptr(), _CODE[T], _at(residual),
          _CODE[T if residual is None else residual.dtype], weight.data_ptr(), eps, None if out8 else y.data_ptr(),
          y.data_ptr() if out8 else None, _at(scale), group, _at(res_out), rows, C)
    return y, scale, res_out


def norm_bwd(dy, h, weight, dres_out=None, eps: float = 1e-6, workspace=None):
    """Gradients of ``norm_fwd``: h is the sum that was normed (res_out, or x
    without a residual), dres_out the gradient of res_out (or None).  Returns
    (dx, dres, dweight): the gradient of x in dy's dtype and of the residual in
    h's - one tensor where the dtypes agree - and of the weight in float32."""
    dev, T = _act(dy, "dy")
    shape = dy.shape
    if not shape:
        raise ValueError("dy must have a last dimension")
    C = shape[-1]
    rows = dy.numel() // C if C else 0
    if h.dtype is not T and h.dtype is not _F32:
        raise TypeError(f"h must be float32 or {T}, got {h.dtype}")
    _want(dy, shape, T, dev, "dy")
    _want(h, shape, h.dtype, dev, "h")
    _want(dres_out, shape, h.dtype, dev, "dres_out")
    _want(weight, (C,), _F32, dev, "weight")
    dx = torch.empty_like(dy)
    dres = dx if h.dtype is T else torch.empty_like(h)
    dw = dy.new_empty(C, dtype=_F32)
    ws, n = _scratch(_lib.efla_norm_bwd_workspace_size(rows, C), workspace, dy)
    _call(_lib.efla_norm_bwd, dev, dy.data_ptr(), _CODE[T], h.data_ptr(), _CODE[h.dtype], weight.data_ptr(), eps,
          _at(dres_out), dx.data_ptr(), None if dres is dx else dres.data_ptr(), dw.data_ptr(), rows, C, _at(ws), n)
    return dx, dres, dw


# ------------------------------------------------------------------------------------------------- conv

def _conv_args(x, weight, bias, state, lengths, heads):
    dev, T = _act(x, "x")
    if x.dim() != 3 or weight.dim() != 2:
        raise ValueError("x must be [B,L,C] and weight [C,K]")
    B, L, C = x.shape
    K = weight.shape[1]
    ldx = _rows(x, x.shape, 2, T, dev, "x")
    _want(weight, (C, K), _F32, dev, "weight")
    _want(bias, (C,), _F32, dev, "bias")
    _want(state, (B, K - 1, C), T, dev, "state")
    _want(lengths, (B,), torch.int32, dev, "lengths")
    if heads < 0 or (heads and C % heads):
        raise ValueError("heads must divide the channels")
    return dev, T, B, L, C, K, ldx, (B, heads, L, C // heads) if heads else (B, L, C)


def conv_fwd(x, weight, bias=None, state=None, lengths=None, silu: bool = True, heads: int = 0, want_state: bool = False,
             y=None, state_out=None):
    """Causal convolution of x [B,L,C] with weight [C,K] (K = 2, 3, 4), then
    SiLU.  state [B,K-1,C]: the inputs before x, oldest first (None: zeros).
    Returns (y, state_out): y [B,L,C], or [B,heads,L,C/heads] as the mixer
    reads it, and the last K-1 inputs of each sequence (None unless wanted;
    ``state_out=state`` updates it in place)."""
    dev, T, B, L, C, K, ldx, out = _conv_args(x, weight, bias, state, lengths, heads)
    if y is None:
        y = x.new_empty(out)
    else:
        _want(y, out, T, dev, "y")
    if state_out is not None:
        _want(state_out, (B, K - 1, C), T, dev, "state_out")
    elif want_state:
        state_out = x.new_empty((B, K - 1, C))
    _call(_lib.efla_conv_fwd, dev, x.data_ptr(), ldx, _CODE[T], weight.data_ptr(), _at(bias), _at(state),
          _at(lengths), silu, y.data_ptr(), heads, _at(state_out), B, L, C, K)
    return y, state_out


def conv_bwd(dy, x, weight, bias=None, state=None, lengths=None, silu: bool = True, heads: int = 0, dstate_out=None,
             workspace=None):
    """Gradients of ``conv_fwd``: (dx, dweight, dbias, dstate); dbias and
    dstate are None without a bias and a state.  dstate_out is the gradient of
    state_out (or None)."""
    dev, T, B, L, C, K, ldx, out = _conv_args(x, weight, bias, state, lengths, heads)
    _want(dy, out, T, dev, "dy")
    _want(dstate_out, (B, K - 1, C), T, dev, "dstate_out")
    dx = x.new_empty((B, L, C))
    dw = x.new_empty((C, K), dtype=_F32)
    db = None if bias is None else x.new_empty(C, dtype=_F32)
    ds = None if state is None else x.new_empty((B, K - 1, C))
    ws, n = _scratch(_lib.efla_conv_bwd_workspace_size(B, L, C, K), workspace, x)
    _call(_lib.efla_conv_bwd, dev, dy.data_ptr(), x.data_ptr(), ldx, _CODE[T], weight.data_ptr(),
          _at(bias), _at(state), _at(lengths), silu, heads, _at(dstate_out), dx.data_ptr(), dw.data_ptr(), _at(db),
          _at(ds), B, L, C, K, _at(ws), n)
    return dx, dw, db, ds


def conv_step(x, state, weight, bias=None, silu: bool = True, y=None):
    """One token: x [B,C], state [B,K-1,C] updated in place.  Returns y [B,C]."""
    dev, T = _act(x, "x")
    if x.dim() != 2 or weight.dim() != 2:
        raise ValueError("x must be [B,C] and weight [C,K]")
    B, C = x.shape
    K = weight.shape[1]
    ldx = _rows(x, x.shape, 1, T, dev, "x")
    _want(weight, (C, K), _F32, dev, "weight")
    _want(bias, (C,), _F32, dev, "bias")
    if state is None:
        raise ValueError("state must be given")
    _want(state, (B, K - 1, C), T, dev, "state")
    if y is None:
        y = x.new_empty((B, C))
    else:
        _want(y, (B, C), T, dev, "y")
    _call(_lib.efla_conv_step, dev, x.data_ptr(), ldx, _CODE[T], state.data_ptr(), weight.data_ptr(),
          _at(bias), silu, y.data_ptr(), B, C, K)
    return y


# ------------------------------------------------------------------------------------------------- scan

def _scan_args(x, dt, A, Bm, Cm, D, z, dt_bias, lengths, lead):
    """Checks shared by the scan's calls; lead is ("B", "L") or ("B",)."""
    dev, T = _act(x, "x")
    k = len(lead)
    if x.dim() != k + 1 or A.dim() != 2 or Bm.dim() != k + 2:
        raise ValueError(f"x must be [{','.join(lead)},C], A [C,N] and Bm [{','.join(lead)},G,N]")
    shape = x.shape
    head = shape[:k]
    C, N, G = shape[k], A.shape[1], Bm.shape[k]
    bc = head + (G, N)
    ld = (_rows(x, shape, k, T, dev, "x"), _rows(dt, shape, k, T, dev, "dt"), _rows(Bm, bc, k, T, dev, "Bm"),
          _rows(Cm, bc, k, T, dev, "Cm"), C if z is None else _rows(z, shape, k, T, dev, "z"))
    _want(A, (C, N), _F32, dev, "A")
    _want(D, (C,), _F32, dev, "D")
    _want(dt_bias, (C,), _F32, dev, "dt_bias")
    _want(lengths, head[:1], torch.int32, dev, "lengths")
    if G == 0 or C % G:
        raise ValueError("the groups of Bm and Cm must divide the channels")
    return dev, T, head, C, G, N, ld


def scan_fwd_workspace_size(B: int, L: int, C: int, G: int, N: int) -> int:
    return int(_lib.efla_scan_fwd_workspace_size(B, L, C, G, N))


def scan_bwd_workspace_size(B: int, L: int, C: int, G: int, N: int) -> int:
    return int(_lib.efla_scan_bwd_workspace_size(B, L, C, G, N))


def scan_fwd(x, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, h0=None, lengths=None, softplus: bool = True,
             want_state: bool = True, y=None, h_L=None, workspace=None):
    """Selective scan of x [B,L,C] with steps dt [B,L,C], decays A [C,N], inputs
    and read-outs Bm, Cm [B,L,G,N], skip D [C] and gate z [B,L,C], from the
    state h0 [B,C,N].  Returns (y [B,L,C], h_L [B,C,N] or None).
    ``h_L=h0`` updates the state in place."""
    dev, T, (B, L), C, G, N, ld = _scan_args(x, dt, A, Bm, Cm, D, z, dt_bias, lengths, ("B", "L"))
    _want(h0, (B, C, N), _F32, dev, "h0")
    if y is None:
        y = x.new_empty((B, L, C))
    else:
        _want(y, (B, L, C), T, dev, "y")
    if h_L is not None:
        _want(h_L, (B, C, N), _F32, dev, "h_L")
    elif want_state:
        h_L = x.new_empty((B, C, N), dtype=_F32)
    ws, n = _scratch(_lib.efla_scan_fwd_workspace_size(B, L, C, G, N), workspace, x)
    _call(_lib.efla_scan_fwd, dev, x.data_ptr(), ld[0], dt.data_ptr(), ld[1], A.data_ptr(),
          Bm.data_ptr(), ld[2], Cm.data_ptr(), ld[3], _at(D), _at(z), ld[4], _at(dt_bias), _at(h0), _at(lengths), _CODE[T],
          softplus, y.data_ptr(), _at(h_L), B, L, C, G, N, _at(ws), n)
    return y, h_L


def scan_bwd(dy, x, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, h0=None, lengths=None, softplus: bool = True, dh_L=None,
             workspace=None):
    """Gradients of ``scan_fwd``: (dx, ddt, dA, dB, dC, dD, dz, ddt_bias, dh0);
    dD, dz and ddt_bias are None where that input is (dh0 is not: a state of
    zeros has a gradient too).  dh_L is the gradient of h_L (or None)."""
    dev, T, (B, L), C, G, N, ld = _scan_args(x, dt, A, Bm, Cm, D, z, dt_bias, lengths, ("B", "L"))
    _want(h0, (B, C, N), _F32, dev, "h0")
    _want(dh_L, (B, C, N), _F32, dev, "dh_L")
    _want(dy, (B, L, C), T, dev, "dy")
    dx, ddt = x.new_empty((B, L, C)), x.new_empty((B, L, C))
    dB, dC = x.new_empty((B, L, G, N)), x.new_empty((B, L, G, N))
    dz = None if z is None else x.new_empty((B, L, C))
    dA = x.new_empty((C, N), dtype=_F32)
    dD = None if D is None else x.new_empty(C, dtype=_F32)
    db = None if dt_bias is None else x.new_empty(C, dtype=_F32)
    dh0 = x.new_empty((B, C, N), dtype=_F32)
    ws, n = _scratch(_lib.efla_scan_bwd_workspace_size(B, L, C, G, N), workspace, x)
    _call(_lib.efla_scan_bwd, dev, dy.data_ptr(), x.data_ptr(), ld[0], dt.data_ptr(), ld[1],
          A.data_ptr(), Bm.data_ptr(), ld[2], Cm.data_ptr(), ld[3], _at(D), _at(z), ld[4], _at(dt_bias), _at(h0),
          _at(lengths), _at(dh_L), _CODE[T], softplus, dx.data_ptr(), ddt.data_ptr(), dA.data_ptr(), dB.data_ptr(),
          dC.data_ptr(), _at(dD), _at(dz), _at(db), _at(dh0), B, L, C, G, N, _at(ws), n)
    return dx, ddt, dA, dB, dC, dD, dz, db, dh0


def scan_step(x, dt, A, Bm, Cm, h, D=None, z=None, dt_bias=None, softplus: bool = True, y=None):
    """One token: x, dt, z [B,C], Bm, Cm [B,G,N], h [B,C,N] updated in place.
    Returns y [B,C]."""
    dev, T, (B,), C, G, N, ld = _scan_args(x, dt, A, Bm, Cm, D, z, dt_bias, None, ("B",))
    if h is None:
        raise ValueError("h must be given")
    _want(h, (B, C, N), _F32, dev, "h")
    if y is None:
        y = x.new_empty((B, C))
    else:
        _want(y, (B, C), T, dev, "y")
    _call(_lib.efla_scan_step, dev, x.data_ptr(), ld[0], dt.data_ptr(), ld[1], A.data_ptr(),
          Bm.data_ptr(), ld[2], Cm.data_ptr(), ld[3], _at(D), _at(z), ld[4], _at(dt_bias), _CODE[T], softplus,
          h.data_ptr(), y.data_ptr(), B, C, G, N)
    return y
