"""The operators around the mixer: norm, short convolution, selective scan.

    y, scale, h   = norm_fwd(x, weight, residual, out8=True)   # block entry
    q, conv_state = conv_fwd(xq, w, bias, heads=H, want_state=True)  # [B,H,L,d]
    y, h_L        = scan_fwd(x, dt, A, Bm, Cm, D, z, dt_bias)   # [B,L,C]

and ``norm_bwd``, ``conv_bwd``, ``scan_bwd`` for training, ``conv_step`` and
``scan_step`` for one token.  Formulas and layouts are in ``include/efla.h``.
Parameters (weight, bias, A, D, dt_bias) and scan states are float32;
activations are float32 or bfloat16.  Tokens of x, z, dt, Bm and Cm may lie
apart in memory (column slices of one projection); all else is contiguous.
``lengths`` [B] int32: tokens from there on are padding and come out as zeros.

The functions run on the current stream of their tensors' device.  Outputs
and scratch are allocated with PyTorch unless passed in.  The checks and
calls are compiled (``csrc/efla_block_binding.cpp``): in Python they took
longer than a one-token step does on the GPU.
"""
from __future__ import annotations

import ctypes

import torch  # before the extension, which needs its libraries

from . import _check, _lib


class _Unusable:
    """Stands for a binding that cannot be loaded: the mixer, which needs none, goes on, and each call of this module says why it fails."""

    def __init__(self, why):
        self._why = why

    def __getattr__(self, name):
        raise ImportError(f"delta_rule_linear_03_b200/_efla_block.so cannot be used ({self._why}): build it with "
                          "`python delta_rule_linear_03_b200/build.py`. There is no fallback implementation.")


def _load():
    try:
        from . import _efla_block as ext
    except ImportError as e:  # missing, or built against another PyTorch's libraries
        return _Unusable(e)
    if ext.torch_version != torch.__version__:  # its C++ interface is one version's
        return _Unusable(f"it is built for PyTorch {ext.torch_version}, this is {torch.__version__}")
    return ext


_ext = _load()

# The C ABI's own signatures, for callers with raw pointers.
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
_lib.efla_diag_conv_run.restype = _i
_lib.efla_diag_conv_run.argtypes = [_i, _i, _i, _i, _i, _i]
_lib.efla_scan_fwd_workspace_size.restype = _sz
_lib.efla_scan_fwd_workspace_size.argtypes = [_i, _i, _i, _i, _i]
_lib.efla_scan_fwd.argtypes = [_p, _l, _p, _l, _p, _p, _l, _p, _l, _p, _p, _l, _p, _p, _p, _i, _i, _p, _p,
                               _i, _i, _i, _i, _i, _p, _sz, _p]
_lib.efla_scan_bwd_workspace_size.restype = _sz
_lib.efla_scan_bwd_workspace_size.argtypes = [_i, _i, _i, _i, _i]
_lib.efla_scan_bwd.argtypes = [_p, _p, _l, _p, _l, _p, _p, _l, _p, _l, _p, _p, _l, _p, _p, _p, _p, _i, _i,
                               _p, _p, _p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _p, _sz, _p]
_lib.efla_diag_scan_plan.argtypes = [_i, _i, _i, _i, _i, _i, ctypes.POINTER(_i)]
_lib.efla_scan_step.argtypes = [_p, _l, _p, _l, _p, _p, _l, _p, _l, _p, _p, _l, _p, _i, _i, _p, _p, _i, _i, _i, _i, _p]
for _name in ("norm_fwd", "norm_bwd", "conv_fwd", "conv_bwd", "conv_step", "scan_fwd", "scan_bwd", "scan_step", "diag_scan_plan"):
    getattr(_lib, "efla_" + _name).restype = _i


# ------------------------------------------------------------------------------------------------- norm

def norm_fwd(x, weight, residual=None, eps: float = 1e-6, out8: bool = False, group: int = 128, y=None, scale=None,
             res_out=None):
    """Root-mean-square norm over the last dimension of ``h = x + residual``.
    Returns (y, scale, res_out): y in x's dtype, or with ``out8`` in
    float8_e4m3fn with one float32 scale per ``group`` columns (128, or 0: per
    row) in [..., ceil(C / group)]; scale is None otherwise.  res_out is h in
    the residual's dtype (x's, or float32), None without a residual; it may be
    passed as ``residual`` itself, to update the stream in place."""
    status, y, scale, res_out = _ext.norm_fwd(x, weight, residual, eps, out8, group, y, scale, res_out)
    if status:
        _check(status, "efla_norm_fwd")
    return y, scale, res_out


def norm_bwd(dy, h, weight, dres_out=None, eps: float = 1e-6, workspace=None):
    """Gradients of ``norm_fwd``: h is the sum that was normed (res_out, or x
    without a residual), dres_out the gradient of res_out (or None).  Returns
    (dx, dres, dweight): the gradient of x in dy's dtype and of the residual in
    h's - one tensor where the dtypes agree - and of the weight in float32."""
    status, dx, dres, dw = _ext.norm_bwd(dy, h, weight, dres_out, eps, workspace)
    if status:
        _check(status, "efla_norm_bwd")
    return dx, dres, dw


# ------------------------------------------------------------------------------------------------- conv

def conv_fwd(x, weight, bias=None, state=None, lengths=None, silu: bool = True, heads: int = 0, want_state: bool = False,
             y=None, state_out=None):
    """Causal convolution of x [B,L,C] with weight [C,K] (K = 2, 3, 4), then
    SiLU.  state [B,K-1,C]: the inputs before x, oldest first (None: zeros).
    Returns (y, state_out): y [B,L,C], or [B,heads,L,C/heads] as the mixer
    reads it, and the last K-1 inputs of each sequence (None unless wanted;
    ``state_out=state`` updates it in place)."""
    status, y, so = _ext.conv_fwd(x, weight, bias, state, lengths, silu, heads, want_state, y, state_out)
    if status:
        _check(status, "efla_conv_fwd")
    return y, so


def conv_bwd(dy, x, weight, bias=None, state=None, lengths=None, silu: bool = True, heads: int = 0, dstate_out=None,
             workspace=None):
    """Gradients of ``conv_fwd``: (dx, dweight, dbias, dstate); dbias and
    dstate are None without a bias and a state.  dstate_out is the gradient of
    state_out (or None)."""
    status, *grads = _ext.conv_bwd(dy, x, weight, bias, state, lengths, silu, heads, dstate_out, workspace)
    if status:
        _check(status, "efla_conv_bwd")
    return tuple(grads)


def conv_step(x, state, weight, bias=None, silu: bool = True, y=None):
    """One token: x [B,C], state [B,K-1,C] updated in place.  Returns y [B,C]."""
    status, y = _ext.conv_step(x, state, weight, bias, silu, y)
    if status:
        _check(status, "efla_conv_step")
    return y


# ------------------------------------------------------------------------------------------------- scan

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
    status, y, h_L = _ext.scan_fwd(x, dt, A, Bm, Cm, D, z, dt_bias, h0, lengths, softplus, want_state, y, h_L, workspace)
    if status:
        _check(status, "efla_scan_fwd")
    return y, h_L


def scan_bwd(dy, x, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, h0=None, lengths=None, softplus: bool = True, dh_L=None,
             workspace=None):
    """Gradients of ``scan_fwd``: (dx, ddt, dA, dB, dC, dD, dz, ddt_bias, dh0);
    dD, dz and ddt_bias are None where that input is (dh0 is not: a state of
    zeros has a gradient too).  dh_L is the gradient of h_L (or None)."""
    status, *grads = _ext.scan_bwd(dy, x, dt, A, Bm, Cm, D, z, dt_bias, h0, lengths, softplus, dh_L, workspace)
    if status:
        _check(status, "efla_scan_bwd")
    return tuple(grads)


def scan_step(x, dt, A, Bm, Cm, h, D=None, z=None, dt_bias=None, softplus: bool = True, y=None):
    """One token: x, dt, z [B,C], Bm, Cm [B,G,N], h [B,C,N] updated in place.
    Returns y [B,C]."""
    status, y = _ext.scan_step(x, dt, A, Bm, Cm, h, D, z, dt_bias, softplus, y)
    if status:
        _check(status, "efla_scan_step")
    return y
