"""Plain float64 implementations (torch, CPU) of the operators around the
mixer, token by token from their formulas, with their gradients, and the
tolerances that the kernels' arithmetic allows.

``mag=True`` runs a formula on magnitudes: every product and sum with the
absolute values of its terms.  What comes out bounds the size of everything
that was added up on the way to a value, so that k rounded operations on the
way change the value by at most k u times it (u = 2^-24 for fp32 operations, to
first order), whatever cancels.  Tolerances are written as such counts.
"""
import math

import torch

U = 2.0 ** -24
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float8_e4m3fn: 2.0 ** -4}


def w(t):
    return None if t is None else t.detach().cpu().double()


def close(got, ref, mag, ops, what):
    """|got - ref| <= ops u mag + half a step of got's type of |ref|; NaN and
    infinities at the same places."""
    g, r = w(got), ref
    assert g.shape == r.shape, (what, g.shape, r.shape)
    fine = torch.isfinite(r)
    assert torch.equal(torch.isnan(g), torch.isnan(r)), f"{what}: NaN at other places"
    assert torch.equal(g[~fine & ~torch.isnan(r)], r[~fine & ~torch.isnan(r)]), f"{what}: infinities differ"
    # the value is rounded after its own error, so the half step is of |ref| + error; 2^-149: the smallest fp32 step
    err = ops * U * mag
    tol = err + HALF_STEP[got.dtype] * (r.abs() + err) + 2.0 ** -140
    bad = ((g - r).abs() > tol) & fine
    if bad.any():
        i = int(((g - r).abs() - tol)[fine].argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {g[fine][i]:.9g} for {r[fine][i]:.9g} "
                             f"(allowed {tol[fine][i]:.3g})")


# --------------------------------------------------------------------------------- norm

def norm_fwd(x, weight, res=None, eps=1e-6):
    h = w(x) if res is None else w(x) + w(res)
    return h * (h.pow(2).mean(-1, keepdim=True) + eps).rsqrt() * w(weight), h


def norm_scale(y, group):
    C = y.shape[-1]
    g = group or C
    n = -(-C // g)
    pad = torch.nn.functional.pad(y, (0, n * g - C)).unflatten(-1, (n, g)).abs().amax(-1)
    return torch.maximum(pad / 448, torch.tensor(2.0 ** -126, dtype=torch.float64))


def norm_bwd(dy, h, weight, dres=None, eps=1e-6, mag=False):
    f = torch.abs if mag else (lambda t: t)
    dy, h, wt = f(w(dy)), f(w(h)), f(w(weight))
    r = (h.pow(2).mean(-1, keepdim=True) + eps).rsqrt()
    u = dy * wt
    m = h * r.pow(3) * (u * h).mean(-1, keepdim=True)
    dh = u * r + m if mag else u * r - m
    if dres is not None:
        dh = dh + f(w(dres))
    return dh, (dy * h * r).flatten(0, -2).sum(0)


# --------------------------------------------------------------------------------- conv

def lens(lengths, B, L):
    return [L] * B if lengths is None else [min(max(int(n), 0), L) for n in lengths]


def conv_fwd(x, weight, bias=None, state=None, lengths=None, silu=True, mag=False):
    """(y, state_out, pre, inputs with the state in front)."""
    f = torch.abs if mag else (lambda t: t)
    x, wt = f(w(x)), f(w(weight))
    B, L, C = x.shape
    K = wt.shape[1]
    n = lens(lengths, B, L)
    front = f(w(state)) if state is not None else x.new_zeros(B, K - 1, C)
    xs = torch.cat([front, x.clone()], 1)
    for b in range(B):
        xs[b, K - 1 + n[b]:] = 0
    pre = x.new_zeros(B, L, C) if bias is None else f(w(bias)).expand(B, L, C).clone()
    for j in range(K):
        pre = pre + xs[:, j:j + L] * wt[:, j]
    y = pre * torch.sigmoid(pre) if silu and not mag else pre.clone()
    for b in range(B):
        y[b, n[b]:] = 0
    return y, torch.stack([xs[b, n[b]:n[b] + K - 1] for b in range(B)]), pre, xs


def dsilu(v):
    s = torch.sigmoid(v)
    return s * (1 + v * (1 - s))


def conv_bwd(dy, x, weight, bias=None, state=None, lengths=None, silu=True, dstate_out=None, mag=False):
    """(dx, dweight, dbias, dstate)."""
    f = torch.abs if mag else (lambda t: t)
    _, _, pre, xs = conv_fwd(x, weight, bias, state, lengths, silu)
    B, L, C = pre.shape
    K, n = weight.shape[1], lens(lengths, B, L)
    wt, xs = f(w(weight)), f(xs)
    d = f(w(dy) * (dsilu(pre) if silu else 1.0))
    if mag and silu:
        # silu' changes by at most 1/2 a unit of its argument, which is off by what pre's terms allow
        d = d + w(dy).abs() * (1 + conv_fwd(x, weight, bias, state, lengths, silu, mag=True)[2])
    for b in range(B):
        d[b, n[b]:] = 0
    dxs, dw = torch.zeros_like(xs), torch.zeros_like(wt)
    for j in range(K):
        dxs[:, j:j + L] += d * wt[:, j]
        dw[:, j] = (d * xs[:, j:j + L]).sum((0, 1))
    if dstate_out is not None:
        for b in range(B):
            dxs[b, n[b]:n[b] + K - 1] += f(w(dstate_out[b]))
    return dxs[:, K - 1:], dw, d.sum((0, 1)), dxs[:, :K - 1]


# --------------------------------------------------------------------------------- scan

def scan(x, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, h0=None, lengths=None, softplus=True, dy=None, dh_L=None,
         mag=False):
    """Forward, and backward where dy is given: a dict of y, h_L and the
    gradients dx, ddt, dA, dB, dC, dD, dz, ddt_bias, dh0."""
    f = torch.abs if mag else (lambda t: t)
    B, L, C = x.shape
    G, N = Bm.shape[2:]
    x, Bm, Cm = f(w(x)), f(w(Bm)), f(w(Cm))
    A_, Dk = w(A), f(w(D)) if D is not None else torch.zeros(C, dtype=torch.float64)
    raw = w(dt) + (w(dt_bias) if dt_bias is not None else 0.0)
    step = torch.logaddexp(raw, torch.zeros_like(raw)) if softplus else raw
    slope = torch.sigmoid(raw) if softplus else torch.ones_like(raw)
    stp = f(step)
    n = lens(lengths, B, L)
    on = torch.zeros(B, L, 1, dtype=torch.bool)
    for b in range(B):
        on[b, :n[b]] = True
    to = torch.arange(C) // (C // G)
    gate = w(z) * torch.sigmoid(w(z)) if z is not None else torch.ones_like(x)
    h = f(w(h0)) if h0 is not None else x.new_zeros(B, C, N)
    hs, out = [h], {}
    y = x.new_zeros(B, L, C)
    core = x.new_zeros(B, L, C)
    for t in range(L):
        e = torch.exp(step[:, t, :, None] * A_)
        new = e * h + (stp[:, t] * x[:, t])[..., None] * Bm[:, t, to]
        h = torch.where(on[:, t, :, None], new, h)
        hs.append(h)
        core[:, t] = torch.where(on[:, t], (h * Cm[:, t, to]).sum(-1) + Dk * x[:, t], 0.0)
        y[:, t] = torch.where(on[:, t], core[:, t] * f(gate[:, t]), 0.0)
    out.update(y=y, h_L=h)
    if dy is None:
        return out
    dy = torch.where(on, f(w(dy)), 0.0)
    g = torch.where(on, dy * f(gate), 0.0)
    p = f(w(dh_L)) if dh_L is not None else x.new_zeros(B, C, N)
    dx, ddt = torch.zeros_like(x), torch.zeros_like(x)
    dB, dC = torch.zeros_like(Bm), torch.zeros_like(Cm)
    dA = torch.zeros_like(A_)
    for t in reversed(range(L)):
        m = on[:, t, :, None]
        full = p + Cm[:, t, to] * g[:, t, :, None]
        e = torch.exp(step[:, t, :, None] * A_)
        back = full * e * hs[t]
        q = (full * Bm[:, t, to]).sum(-1)
        dx[:, t] = torch.where(on[:, t], stp[:, t] * q + Dk * g[:, t], 0.0)
        ddt[:, t] = torch.where(on[:, t], ((back * f(A_)).sum(-1) + x[:, t] * q) * slope[:, t], 0.0)
        dA += torch.where(m, back * stp[:, t, :, None], 0.0).sum(0)
        dB[:, t] = torch.where(m, full * (stp[:, t] * x[:, t])[..., None], 0.0).view(B, G, C // G, N).sum(2)
        dC[:, t] = torch.where(m, hs[t + 1] * g[:, t, :, None], 0.0).view(B, G, C // G, N).sum(2)
        p = torch.where(m, full * e, p)
    out.update(dx=dx, ddt=ddt, dA=dA, dB=dB, dC=dC, dD=(g * torch.where(on, x, 0.0)).sum((0, 1)), ddt_bias=ddt.sum((0, 1)), dh0=p)
    if z is not None:
        out["dz"] = torch.where(on, dy * core * f(dsilu(w(z))), 0.0)
    return out


def scan_ops(L, N, C, B, decay):
    """Rounded operations, in units u, between the inputs and a value of the
    scan, to first order.  Per step: a decay exp(D A) has the error of ex2 (2
    ulp, 4 u) and of its argument (D: softplus 16 u, its product with A and
    log2 e 3 u, times |D A| <= decay), a term D x B 18 u, the update 1 u.  A
    value depends on up to 2 L steps (a gradient: forward and back), and ends
    in a sum over N state values and, at most, over C channels or B L tokens."""
    per_step = 4 + 20 * decay + 1
    return 2 * L * per_step + 64 + N + C + B * L


def max_decay(dt, A, dt_bias=None, softplus=True):
    raw = w(dt) + (w(dt_bias) if dt_bias is not None else 0.0)
    step = torch.logaddexp(raw, torch.zeros_like(raw)) if softplus else raw
    return float(step.abs().max() * w(A).abs().max()) if step.numel() else 0.0


def scan_inputs(B, L, C, N, G=1, dtype=torch.float32, seed=0, lengths=None):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    step = torch.exp(torch.rand(C, generator=g) * math.log(100.0) + math.log(1e-3))
    return dict(x=r(B, L, C).to(dtype), dt=(0.5 * r(B, L, C)).to(dtype),
                A=-torch.arange(1, N + 1.0) * torch.exp(0.2 * r(C, N)), Bm=r(B, L, G, N).to(dtype), Cm=r(B, L, G, N).to(dtype),
                D=1 + 0.2 * r(C), z=r(B, L, C).to(dtype), dt_bias=step + torch.log(-torch.expm1(-step)), h0=0.3 * r(B, C, N),
                lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32))
