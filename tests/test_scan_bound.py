"""The scan's error bound (CPU): its values are the reference's, fp32 arithmetic
keeps within it, and results that are a little wrong do not."""
import pytest
import torch

import block_ref as R
import scan_bound as S

NAMES = ("y", "h_L", "dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dh0")


def _case(B, L, C, N, G=1, lengths=None, T=torch.float32, seed=0):
    s = R.scan_inputs(B, L, C, N, G, T, seed=seed, lengths=lengths)
    g = torch.Generator().manual_seed(seed + 1)
    return s, torch.randn(B, L, C, generator=g).to(T), torch.randn(B, C, N, generator=g)


@pytest.mark.parametrize("B,L,C,N,G,lengths,seg", [(2, 9, 6, 8, 2, [9, 4], None), (3, 40, 4, 16, 1, [0, 33, 40], 32), (1, 100, 4, 8, 1, None, 32)])
def test_values_are_the_references(B, L, C, N, G, lengths, seg):
    s, dy, dh = _case(B, L, C, N, G, lengths)
    ref, got = R.scan(**s, dy=dy, dh_L=dh), S.scan(**s, dy=dy, dh_L=dh, seg=seg, seg_bwd=seg)
    for k in NAMES:
        torch.testing.assert_close(got[k][0], ref[k], rtol=1e-11, atol=1e-12, msg=lambda m: f"{k}: {m}")
        assert bool((got[k][1] >= 0).all())


def _fp32(s, dy, dh, seg=None, drop=None):
    """The scan in fp32 operations, in segments as the kernels compose them; drop: the segment whose entering state is lost."""
    x, dt, A, z = s["x"].float(), s["dt"].float(), s["A"], s["z"].float()
    Bm, Cm = s["Bm"].float(), s["Cm"].float()
    B, L, C = x.shape
    to = torch.arange(C) // (C // Bm.shape[2])
    step = torch.nn.functional.softplus(dt + s["dt_bias"], threshold=1e9)
    h, ys, hs = s["h0"].clone(), [], [s["h0"]]
    for t in range(L):
        if drop is not None and t == drop * seg:
            h = torch.zeros_like(h)
        h = torch.exp(step[:, t, :, None] * A) * h + (step[:, t] * x[:, t])[..., None] * Bm[:, t, to]
        hs.append(h)
        ys.append(((h * Cm[:, t, to]).sum(-1) + s["D"] * x[:, t]) * torch.nn.functional.silu(z[:, t]))
    out = dict(y=torch.stack(ys, 1), h_L=h)
    p = dh
    g = dy.float() * torch.nn.functional.silu(z)
    dB, dh0 = [], None
    for t in reversed(range(L)):
        p = p + Cm[:, t, to] * g[:, t, :, None]
        dB.append((p * (step[:, t] * x[:, t])[..., None]).view(B, Bm.shape[2], -1, A.shape[1]).sum(2))
        p = p * torch.exp(step[:, t, :, None] * A)
    out.update(dB=torch.stack(dB[::-1], 1), dh0=p)
    return out


CASES = [(3, 100, 96, 16, 4, None), (1, 257, 40, 32, 1, None), (1, 1000, 16, 16, 1, 64)]


@pytest.mark.parametrize("B,L,C,N,G,seg", CASES)
def test_fp32_keeps_within(B, L, C, N, G, seg):
    s, dy, dh = _case(B, L, C, N, G)
    bound = S.scan(**s, dy=dy, dh_L=dh, seg=seg, seg_bwd=seg)
    for k, v in _fp32(s, dy, dh).items():
        S.close(v, *bound[k], k)


def _refused(got, bound, k):
    with pytest.raises(AssertionError, match="off"):
        S.close(got, *bound[k], k)


@pytest.mark.parametrize("B,L,C,N,G,seg", CASES + [(1, 5000, 64, 32, 1, 128)])
def test_small_mistakes_are_seen(B, L, C, N, G, seg):
    s, dy, dh = _case(B, L, C, N, G)
    back = L < 5000
    bound = S.scan(**s, dy=dy if back else None, dh_L=dh, seg=seg, seg_bwd=seg)
    ref = {k: v[0] for k, v in bound.items()}
    for k in ref:  # a value off by a thousandth
        _refused((ref[k] * 1.001).float(), bound, k)
    rounded = {k: v.bfloat16().float() if k in ("x", "dt", "Bm", "Cm", "z") else v for k, v in s.items()}
    low = R.scan(**rounded, dy=dy if back else None, dh_L=dh)
    for k in ref:
        _refused(low[k].float(), bound, k)
    slower = R.scan(**dict(s, A=s["A"] * 1.001), dy=dy if back else None, dh_L=dh)  # decays off by a thousandth of their exponent
    for k in ("y", "h_L"):
        _refused(slower[k].float(), bound, k)
    if seg:
        lost = _fp32(s, dy, dh, seg, drop=L // seg // 2)  # the state that enters one segment is dropped
        _refused(lost["y"], bound, "y")
        _refused(_fp32(s, dy, dh, seg, drop=(L - 1) // seg)["h_L"], bound, "h_L")

