"""The selective scan in float64 with a bound on the error of its fp32
evaluation, carried through the recurrence itself: an error made at one token is
forgotten with the decay of the tokens behind it, and each step is charged by
its own |D A|.  To first order in u = 2^-24 (the bound is taken 2% larger):

  D         softplus 12 u D, and the rounding of dt + bias, u |dt + bias| softplus'
  e^(D A)   2^v 4.5 u; its argument 3 u |D A| (A log2 e, the constant, the product), and |A| times the error of D
  D x B     two products, 2 u
  h         e h + D x B rounded once: u |h|
  sums over the state index: two products in turn, their pair, four halvings: 8 u of the terms' magnitudes
  sigmoid, silu (8 + 2 |v|) u

Where the sequence is cut into segments, the state that enters a segment is
composed of the earlier segments' own states (from zero) and of the decay over
a whole segment, e^(A sum D): squared from its half (9 u, products 2 u), its
argument off by the additions of D in turn, u times each partial sum.  What a
segment makes by itself and what it passes on may cancel, so both count.

``scan(...)`` gives {name: (value, error bound)}."""
import torch

from block_ref import HALF_STEP, U, lens, w


def close(got, value, err, what):
    """got is value but for err and half a step of its type."""
    g = got.detach().cpu().double()
    assert g.shape == value.shape, (what, g.shape, value.shape)
    assert bool(torch.isfinite(g).all()), f"{what}: not finite"
    err = 1.02 * err
    tol = err + HALF_STEP[got.dtype] * (value.abs() + err) + 2.0 ** -140
    over = (g - value).abs() - tol
    if bool((over > 0).any()):
        i = int(over.argmax())
        raise AssertionError(f"{what}: {int((over > 0).sum())} of {g.numel()} off, worst {g.flatten()[i]:.9g} for {value.flatten()[i]:.9g} "
                             f"(allowed {tol.flatten()[i]:.3g})")


def _sigmoid(v):
    s = torch.sigmoid(v)
    return s, (8 + 2 * v.abs()) * U * s


def scan(x, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, h0=None, lengths=None, softplus=True, dy=None, dh_L=None, seg=None, seg_bwd=None,
         tiles=1):
    """seg, seg_bwd: tokens of a segment of the forward and the backward pass
    (None: the whole); tiles: of channels, whose dB and dC are added in turn."""
    B, L, C = x.shape
    G, N = Bm.shape[2:]
    x, Bm, Cm, A = w(x), w(Bm), w(Cm), w(A)
    Dk = w(D) if D is not None else torch.zeros(C, dtype=torch.float64)
    raw = w(dt) + (w(dt_bias) if dt_bias is not None else 0.0)
    slope, slope_err = _sigmoid(raw) if softplus else (torch.ones_like(raw), torch.zeros_like(raw))
    step = torch.logaddexp(raw, torch.zeros_like(raw)) if softplus else raw
    step_err = U * (12 * step + raw.abs() * slope) if softplus else U * raw.abs()
    n = lens(lengths, B, L)
    on = torch.arange(L)[None, :, None] < torch.tensor(n)[:, None, None]  # [B, L, 1]
    step, step_err, x = (torch.where(on, t, 0.0) for t in (step, step_err, x))
    Bm, Cm = (torch.where(on[..., None], t, 0.0) for t in (Bm, Cm))
    to = torch.arange(C) // (C // G)
    if z is not None:
        zz = torch.where(on, w(z), 0.0)
        s, s_err = _sigmoid(zz)
        gate, gate_err = zz * s, (9 + 2 * zz.abs()) * U * (zz * s).abs()
        slope_z = s + zz * s * (1 - s)
        slope_z_err = s_err * (1 + 2 * zz.abs()) + 4 * U * (s + (zz * s).abs())
    else:
        gate, gate_err = torch.ones_like(x), torch.zeros_like(x)
    zero = torch.zeros(B, C, N, dtype=torch.float64)

    def decay(t):
        d, e = step[:, t, :, None], step_err[:, t, :, None]
        a = torch.exp(d * A)
        return a, torch.where(on[:, t, :, None], 4.5 * U + 3 * U * (d * A).abs() + e * A.abs(), 0.0)

    def walk(order, start, start_err, size, term, late, get):
        """v = a v + term, or a (v + term) where late, over the tokens of `order`, in segments of `size`.  get(t, v, v_err)
        sees what `a` is multiplied with, and else what it gives."""
        own, passed, err = zero, start, start_err
        total, partial, inner = zero[..., 0], zero[..., 0], zero  # of a segment: sum of D, sum of its partial sums, error of D
        for k, t in enumerate(order):
            if k and size and (k % size == 0 if order[0] == 0 else (t + 1) % size == 0):
                whole = total[..., None] * A.abs()
                err = err + passed.abs() * (11 * U + 3 * U * whole + U * partial[..., None] * A.abs() + inner)
                own, passed = zero, own + passed
                total, partial, inner = zero[..., 0], zero[..., 0], zero
            a, a_err = decay(t)
            v, v_err = term(t)
            m = on[:, t, :, None]
            both = own + passed
            if late:
                err = torch.where(m, err + v_err + U * (both + v).abs(), err)
                get(t, both + v, err)
                own = own + v
                err = a * err + a_err * a * (own.abs() + passed.abs()) + torch.where(m, U * (a * (own + passed)).abs(), 0.0)
                own, passed = a * own, a * passed
            else:
                err = torch.where(m, a * err + a_err * a * (own.abs() + passed.abs()) + v_err + U * (a * both + v).abs(), err)
                own, passed = a * own + v, a * passed
                get(t, own + passed, err)
            total = total + step[:, t]
            partial = partial + torch.where(on[:, t], total, 0.0)
            inner = inner + step_err[:, t, :, None] * A.abs()
        return own + passed, err

    h, h_err = w(h0) if h0 is not None else zero, zero
    hs, hs_err = [h], [h_err]

    def forward_term(t):
        xb = x[:, t, :, None] * Bm[:, t, to]
        return step[:, t, :, None] * xb, step_err[:, t, :, None] * xb.abs() + 2 * U * (step[:, t, :, None] * xb).abs()

    def keep(t, v, e):
        hs.append(v)
        hs_err.append(e)

    def states(size):
        del hs[1:], hs_err[1:]
        return walk(range(L), h, h_err, size, forward_term, False, keep)

    end, end_err = states(seg)
    core, core_err = torch.zeros_like(x), torch.zeros_like(x)

    def cores():
        for t in range(L):
            c = Cm[:, t, to]
            core[:, t] = (hs[t + 1] * c).sum(-1) + Dk * x[:, t]
            core_err[:, t] = (hs_err[t + 1] * c.abs() + 8 * U * (hs[t + 1] * c).abs()).sum(-1) + U * core[:, t].abs()

    cores()
    mask = lambda p, q: (torch.where(on, p, 0.0), torch.where(on, q, 0.0))  # noqa: E731
    out = dict(y=mask(core * gate, core_err * gate.abs() + core.abs() * gate_err + U * (core * gate).abs()), h_L=(end, end_err))
    if dy is None:
        return out
    if seg_bwd != seg:
        states(seg_bwd)
        cores()
    dy = torch.where(on, w(dy), 0.0)
    g = dy * gate
    g_err = dy.abs() * gate_err + U * g.abs()
    names = ("dx", "ddt", "dB", "dC")
    val = {k: torch.zeros_like(x if k[1:] in ("x", "dt") else Bm) for k in names}
    err = {k: torch.zeros_like(v) for k, v in val.items()}
    sums = {k: [torch.zeros(C, N, dtype=torch.float64) for _ in range(3)] for k in ("dA",)}  # value, error of the terms, their magnitudes
    group = lambda v: v.view(B, G, C // G, N).sum(2)  # noqa: E731

    def back_term(t):
        c = Cm[:, t, to]
        gt = g[:, t, :, None]
        return c * gt, c.abs() * g_err[:, t, :, None] + U * (c * gt).abs()

    def gradients(t, p, p_err):
        d, d_err = step[:, t, :, None], step_err[:, t, :, None]
        a, a_err = decay(t)
        b, xt = Bm[:, t, to], x[:, t]
        q = (p * b).sum(-1)
        q_err = (p_err * b.abs() + 8 * U * (p * b).abs()).sum(-1)
        val["dx"][:, t] = step[:, t] * q + Dk * g[:, t]
        err["dx"][:, t] = step[:, t] * q_err + step_err[:, t] * q.abs() + Dk.abs() * g_err[:, t] + 2 * U * ((Dk * g[:, t]).abs() + (step[:, t] * q).abs())
        back = p * a * hs[t]
        back_err = p_err * a * hs[t].abs() + p.abs() * a * hs_err[t] + back.abs() * (a_err + 2 * U)
        dd = (back * A).sum(-1) + xt * q
        dd_err = (back_err * A.abs() + 8 * U * (back * A).abs()).sum(-1) + xt.abs() * q_err + U * (dd.abs() + (xt * q).abs())
        val["ddt"][:, t] = dd * slope[:, t]
        err["ddt"][:, t] = dd_err * slope[:, t] + dd.abs() * slope_err[:, t] + U * (dd * slope[:, t]).abs()
        m = on[:, t, :, None]
        for total, more in zip(sums["dA"], (back * d, back_err * d + back.abs() * d_err, (back * d).abs())):
            total += torch.where(m, more, 0.0).sum(0)
        dx = step[:, t] * xt
        u, u_err = dx[..., None], (step_err[:, t] * xt.abs() + U * dx.abs())[..., None]
        gt, gt_err = g[:, t, :, None], g_err[:, t, :, None]
        count = (12 + tiles) * U
        val["dB"][:, t] = group(p * u)
        err["dB"][:, t] = group(p_err * u.abs() + p.abs() * u_err + count * (p * u).abs())
        val["dC"][:, t] = group(hs[t + 1] * gt)
        err["dC"][:, t] = group(hs_err[t + 1] * gt.abs() + hs[t + 1].abs() * gt_err + count * (hs[t + 1] * gt).abs())

    first = w(dh_L) if dh_L is not None else zero
    out["dh0"] = walk(range(L - 1, -1, -1), first, zero, seg_bwd, back_term, True, gradients)
    for k in ("dx", "ddt"):
        out[k] = mask(val[k], err[k])
    for k in ("dB", "dC"):
        out[k] = tuple(torch.where(on[..., None], t, 0.0) for t in (val[k], err[k]))
    cuts = -(-L // seg_bwd) if seg_bwd else 1
    rows = cuts * B / 32 + 6  # partial sums of sequences and segments, added by 32s in turn and a tree
    v, e, m = sums["dA"]
    out["dA"] = (v, e + (12 + rows) * U * m)  # up to eight tokens in turn, the rest compensated
    count = (L / cuts / 16 + 18 + rows) * U  # a thread's tokens, a tile's, the rows
    ddt, ddt_err = out["ddt"]
    out["ddt_bias"] = (ddt.sum((0, 1)), (ddt_err + count * ddt.abs()).sum((0, 1)))
    gx = g * x
    out["dD"] = (gx.sum((0, 1)), (g_err * x.abs() + count * gx.abs()).sum((0, 1)))
    if z is not None:
        out["dz"] = mask(dy * core * slope_z, dy.abs() * (core_err * slope_z.abs() + core.abs() * slope_z_err) + 2 * U * (dy * core * slope_z).abs())
    return out
