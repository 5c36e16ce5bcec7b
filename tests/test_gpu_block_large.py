"""Element offsets past 32 bits: the ends of large tensors come out as the
same rows do alone."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
C = 2048
ROWS = (1 << 31) // C + 64  # the last 64 rows lie past 2^31 elements


@pytest.fixture(scope="module")
def efla():
    import delta_rule_linear_03_b200 as m
    return m


def _rows(*shape, seed, std=1.0):
    t = torch.empty(shape, dtype=BF, device="cuda")
    return t.normal_(0, std, generator=torch.Generator(device="cuda").manual_seed(seed))


def _like(p, q):
    """Equal but for a rounding to bf16 that fell the other way: sums may be taken in another order."""
    p, q = p.float(), q.float()
    assert float((p - q).abs().max()) <= 2 ** -7 * float(q.abs().max())


def test_norm_large(efla):
    x, w = _rows(ROWS, C, seed=1), torch.rand(C, device="cuda") + 0.5
    y, _, _ = efla.norm_fwd(x, w)
    assert torch.equal(y[-64:], efla.norm_fwd(x[-64:].clone(), w)[0])
    y8, scale, _ = efla.norm_fwd(x, w, out8=True)
    z8, zs, _ = efla.norm_fwd(x[-64:].clone(), w, out8=True)
    assert torch.equal(y8[-64:].view(torch.uint8), z8.view(torch.uint8)) and torch.equal(scale[-64:], zs)
    dx, _, _ = efla.norm_bwd(y, x, w)
    assert torch.equal(dx[-64:], efla.norm_bwd(y[-64:].clone(), x[-64:].clone(), w)[0])


def test_conv_large(efla):
    x, w = _rows(1, ROWS, C, seed=2), torch.randn(C, 4, device="cuda")
    y, state = efla.conv_fwd(x, w, want_state=True)
    tail, before = x[:, -64:].clone(), x[:, -67:-64].clone()
    assert torch.equal(y[:, -64:], efla.conv_fwd(tail, w, state=before)[0]) and torch.equal(state, tail[:, -3:])
    dx = efla.conv_bwd(y, x, w)[0]
    _like(dx[:, -64:], efla.conv_bwd(y[:, -64:].clone(), tail, w, state=before)[0])


def test_scan_large(efla):
    N, cut = 8, ROWS - 64
    x, dt, Bm, Cm = _rows(1, ROWS, C, seed=3), _rows(1, ROWS, C, seed=4), _rows(1, ROWS, 1, N, seed=5), _rows(1, ROWS, 1, N, seed=6)
    A = -torch.rand(C, N, device="cuda") - 0.1
    y, h = efla.scan_fwd(x, dt, A, Bm, Cm)
    tail = [t[:, cut:].clone() for t in (x, dt, Bm, Cm)]
    _, mid = efla.scan_fwd(x[:, :cut], dt[:, :cut], A, Bm[:, :cut], Cm[:, :cut])
    y2, h2 = efla.scan_fwd(tail[0], tail[1], A, tail[2], tail[3], h0=mid)
    _like(y[:, cut:], y2)
    _like(h, h2)
    grads = efla.scan_bwd(y, x, dt, A, Bm, Cm)
    again = efla.scan_bwd(y2, tail[0], tail[1], A, tail[2], tail[3], h0=mid)
    for i in (0, 1, 3, 4):  # dx, ddt, dB, dC
        _like(grads[i][:, cut:], again[i])


def test_strides_large(efla):
    """Column slices of a projection whose rows are wide."""
    N, Ci, L = 16, 64, 70000
    wide = _rows(1, L, 32768, seed=7)
    assert wide.numel() > 1 << 31
    x, dt, z = wide[..., :Ci], wide[..., 8192:8192 + Ci], wide[..., -Ci:]
    Bm, Cm = (wide[..., i:i + N].unflatten(-1, (1, N)) for i in (1024, 2048))
    A, w = -torch.rand(Ci, N, device="cuda"), torch.randn(Ci, 4, device="cuda")
    args, copies = [x, dt, A, Bm, Cm], [t.contiguous() for t in (x, dt, A, Bm, Cm)]
    for p, q in zip(efla.scan_fwd(*args, z=z), efla.scan_fwd(*copies, z=z.contiguous())):
        assert torch.equal(p, q)
    assert torch.equal(efla.conv_fwd(z, w)[0], efla.conv_fwd(z.contiguous(), w)[0])
    step = wide[0, -8:]
    h = torch.rand(8, Ci, N, device="cuda")
    g = h.clone()
    args = [step[:, :Ci], step[:, 64:64 + Ci], A, step[:, 256:256 + N].unflatten(-1, (1, N)), step[:, 512:512 + N].unflatten(-1, (1, N))]
    copies = [t.contiguous() for t in args]
    assert torch.equal(efla.scan_step(*args, h), efla.scan_step(*copies, g)) and torch.equal(h, g)
