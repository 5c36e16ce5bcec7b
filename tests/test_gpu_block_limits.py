"""Batches whose states are gigabytes: every sequence comes out as it does in a
small batch."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def efla():
    import delta_rule_linear_03_b200 as m
    return m


def _like(p, q):
    """Of one token: equal but for the order of sums of N terms and the roundings of a decay's argument (|D A| < 8),
    well under 1e-5 of the largest, and, in bf16, one rounding that fell the other way."""
    p, q = p.float(), q.float()
    assert float((p - q).abs().max()) <= 2.0 ** -7 * float(q.abs().max())


@pytest.mark.parametrize("B,C,N", [(4096, 4096, 16), (300, 4096, 64), (20000, 200, 32)])
def test_scan_large_batches(efla, B, C, N):
    g = torch.Generator(device="cuda").manual_seed(B)
    r = lambda *s, to=BF: torch.randn(s, generator=g, device="cuda").to(to)  # noqa: E731
    s = dict(x=r(B, C), dt=r(B, C), z=r(B, C), Bm=r(B, 1, N), Cm=r(B, 1, N))
    h0, dy, dh, A = r(B, C, N, to=torch.float32), r(B, 1, C), r(B, C, N, to=torch.float32), -torch.rand(C, N, device="cuda", generator=g) - 0.1
    part = torch.cat([torch.arange(4), torch.arange(B // 2, B // 2 + 4), torch.arange(B - 4, B)]).cuda()
    few = {k: t[part] for k, t in s.items()}
    h, hf = h0.clone(), h0[part]
    y, yf = efla.scan_step(A=A, h=h, **s), efla.scan_step(A=A, h=hf, **few)
    assert torch.equal(y[part], yf) and torch.equal(h[part], hf)
    one = lambda d: {k: t[:, None] for k, t in d.items()}  # noqa: E731
    y1, h1 = efla.scan_fwd(A=A, h0=h0, **one(s))
    _like(y1[:, 0], y)
    assert float((h1 - h).abs().max()) <= 1e-5 * float(h.abs().max())
    dx, ddt, _, dB, dC, _, dz, _, dh0 = efla.scan_bwd(dy, A=A, h0=h0, dh_L=dh, **one(s))
    few = efla.scan_bwd(dy[part], A=A, h0=h0[part], dh_L=dh[part], **one(few))
    for p, i in ((dx, 0), (ddt, 1), (dB, 3), (dC, 4), (dz, 6)):
        _like(p[part], few[i])
    assert float((dh0[part] - few[8]).abs().max()) <= 1e-5 * float(few[8].abs().max())
