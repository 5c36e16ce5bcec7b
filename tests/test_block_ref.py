"""The float64 references of the operators around the mixer: their gradients
against torch.autograd and against central differences (CPU)."""
import pytest
import torch

import block_ref as R


def _leaf(t):
    return None if t is None else t.double().requires_grad_()


def test_norm_gradient_matches_autograd():
    g = torch.Generator().manual_seed(0)
    x, wt, dy, dr = (torch.randn(s, generator=g) for s in ((5, 33), (33,), (5, 33), (5, 33)))
    h, wl = _leaf(x), _leaf(wt)
    y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + 1e-6) * wl
    ((y * dy.double()).sum() + (h * dr.double()).sum()).backward()
    dh, dw = R.norm_bwd(dy, x, wt, dr)
    torch.testing.assert_close(dh, h.grad, rtol=1e-12, atol=1e-12)
    torch.testing.assert_close(dw, wl.grad, rtol=1e-12, atol=1e-12)


def _conv_auto(x, wt, bias, state, lengths, silu):
    """Convolution from leaves, through unfold."""
    B, L, C = x.shape
    K = wt.shape[1]
    keep = torch.arange(L)[None, :] < torch.tensor(R.lens(lengths, B, L))[:, None]
    xs = torch.cat([state, torch.where(keep[..., None], x, 0.0)], 1)
    y = (xs.unfold(1, K, 1) * wt).sum(-1) + bias
    y = torch.nn.functional.silu(y) if silu else y
    n = R.lens(lengths, B, L)
    return torch.where(keep[..., None], y, 0.0), torch.stack([xs[b, n[b]:n[b] + K - 1] for b in range(B)])


@pytest.mark.parametrize("K,lengths,silu", [(2, None, True), (4, [7, 0, 2], True), (3, [1, 7, 9], False)])
def test_conv_gradient_matches_autograd(K, lengths, silu):
    g = torch.Generator().manual_seed(K)
    B, L, C = 3, 7, 5
    x, wt, bias, state, dy, ds = (torch.randn(s, generator=g) for s in
                                  ((B, L, C), (C, K), (C,), (B, K - 1, C), (B, L, C), (B, K - 1, C)))
    ls = [_leaf(t) for t in (x, wt, bias, state)]
    y, so = _conv_auto(*ls, lengths, silu)
    ((y * dy.double()).sum() + (so * ds.double()).sum()).backward()
    ry, rs, _, _ = R.conv_fwd(x, wt, bias, state, lengths, silu)
    torch.testing.assert_close(ry, y.detach(), rtol=1e-12, atol=1e-12)
    torch.testing.assert_close(rs, so.detach(), rtol=1e-12, atol=1e-12)
    for r, leaf in zip(R.conv_bwd(dy, x, wt, bias, state, lengths, silu, ds), ls):
        torch.testing.assert_close(r, leaf.grad, rtol=1e-11, atol=1e-11)


def _scan_case(lengths, softplus, gate):
    B, L, C, N, G = 3, 6, 4, 8, 2
    s = R.scan_inputs(B, L, C, N, G, seed=7, lengths=lengths)
    if not gate:
        s["z"] = None
    if not softplus:
        s["dt"] = s["dt"].abs() * 0.1
        s["dt_bias"] = None
    g = torch.Generator().manual_seed(8)
    return s, torch.randn(B, L, C, generator=g), torch.randn(B, C, N, generator=g)


@pytest.mark.parametrize("lengths,softplus,gate", [(None, True, True), ([6, 0, 3], True, True), ([1, 6, 6], False, False)])
def test_scan_gradient_matches_autograd(lengths, softplus, gate):
    s, dy, dh = _scan_case(lengths, softplus, gate)
    names = [k for k in ("x", "dt", "A", "Bm", "Cm", "D", "z", "dt_bias", "h0") if s[k] is not None]
    v = {k: _leaf(s[k]) for k in names}
    B, L, C = s["x"].shape
    to = torch.arange(C) // (C // s["Bm"].shape[2])
    h, ys = v["h0"], []
    n = R.lens(lengths, B, L)
    for t in range(L):
        raw = v["dt"][:, t] + v.get("dt_bias", 0.0)
        step = torch.nn.functional.softplus(raw, threshold=1e9) if softplus else raw
        new = torch.exp(step[..., None] * v["A"]) * h + (step * v["x"][:, t])[..., None] * v["Bm"][:, t, to]
        on = torch.tensor([t < k for k in n])[:, None]
        h = torch.where(on[..., None], new, h)
        y = (h * v["Cm"][:, t, to]).sum(-1) + v["D"] * v["x"][:, t]
        ys.append(torch.where(on, y * (torch.nn.functional.silu(v["z"][:, t]) if gate else 1.0), 0.0))
    y = torch.stack(ys, 1)
    ((y * dy.double()).sum() + (h * dh.double()).sum()).backward()
    r = R.scan(**s, softplus=softplus, dy=dy, dh_L=dh)
    torch.testing.assert_close(r["y"], y.detach(), rtol=1e-11, atol=1e-11)
    to_name = dict(x="dx", dt="ddt", A="dA", Bm="dB", Cm="dC", D="dD", z="dz", dt_bias="ddt_bias", h0="dh0")
    for k in names:
        torch.testing.assert_close(r[to_name[k]], v[k].grad, rtol=1e-10, atol=1e-10, msg=lambda m: f"{k}: {m}")


@pytest.mark.parametrize("name", ["x", "dt", "A", "Bm", "Cm", "D", "z", "dt_bias", "h0"])
def test_scan_gradient_matches_differences(name):
    s, dy, dh = _scan_case([6, 2, 5], True, True)
    to_name = dict(x="dx", dt="ddt", A="dA", Bm="dB", Cm="dC", D="dD", z="dz", dt_bias="ddt_bias", h0="dh0")
    grad = R.scan(**s, dy=dy, dh_L=dh)[to_name[name]]
    s = {k: (t.double() if t is not None and t.dtype.is_floating_point else t) for k, t in s.items()}
    d = torch.randn(s[name].shape, generator=torch.Generator().manual_seed(1), dtype=torch.float64)

    def loss(e):
        r = R.scan(**dict(s, **{name: s[name] + e * d}))
        return float((r["y"] * dy.double()).sum() + (r["h_L"] * dh.double()).sum())

    # central differences of step 1e-5: the cut-off is of order 1e-10, the cancellation 1e-16 / 1e-5 of the loss
    quotient = (loss(1e-5) - loss(-1e-5)) / 2e-5
    assert quotient == pytest.approx(float((grad * d).sum()), rel=1e-6, abs=1e-7)


def test_norm_and_conv_gradients_match_differences():
    g = torch.Generator().manual_seed(3)
    x, wt, dy = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((4, 9), (9,), (4, 9)))
    dx = torch.randn(4, 9, generator=g, dtype=torch.float64)
    dh, _ = R.norm_bwd(dy, x, wt)
    quotient = sum(s * float((R.norm_fwd(x + s * 1e-5 * dx, wt)[0] * dy).sum()) for s in (1, -1)) / 2e-5
    assert quotient == pytest.approx(float((dh * dx).sum()), rel=1e-6, abs=1e-7)
    x, wt, b, st, dy, d = (torch.randn(s, generator=g, dtype=torch.float64) for s in
                           ((2, 6, 3), (3, 4), (3,), (2, 3, 3), (2, 6, 3), (2, 6, 3)))
    dxs = R.conv_bwd(dy, x, wt, b, st)[0]
    quotient = sum(s * float((R.conv_fwd(x + s * 1e-5 * d, wt, b, st)[0] * dy).sum()) for s in (1, -1)) / 2e-5
    assert quotient == pytest.approx(float((dxs * d).sum()), rel=1e-6, abs=1e-7)
