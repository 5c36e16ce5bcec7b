"""efla_norm_fwd where a thread has several rows in flight, and where rows do not
fill the last block, against float64 on the GPU; and the 8-bit values of many
rows next to the border of two."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32
U = 2.0 ** -24
HALF = {F: 2.0 ** -24, BF: 2.0 ** -8}


@pytest.fixture(scope="module")
def efla():
    import delta_rule_linear_03_b200 as m
    return m


def _draw(rows, C, T, RT):
    g = torch.Generator(device="cuda").manual_seed(rows + C)
    r = lambda *s: torch.randn(s, device="cuda", generator=g)  # noqa: E731
    return r(rows, C).to(T), 1 + 0.3 * r(C), None if RT is None else (2 * r(rows, C)).to(RT)


def _exact(x, wt, res):
    h = x.double() if res is None else x.double() + res.double()
    return h, h * torch.rsqrt(h.pow(2).mean(-1, keepdim=True) + 1e-6) * wt.double()


def _near(got, value, ops, what):
    err = ops * U * value.abs()
    over = (got.double() - value).abs() - err - HALF[got.dtype] * (value.abs() + err) - 2.0 ** -140
    assert float(over.max()) <= 0, (what, int((over > 0).sum()))


def _quotient(y, group):
    """y in units of its group's scale, and the scale."""
    rows, C = y.shape
    g = group or C
    n = -(-C // g)
    scale = (torch.nn.functional.pad(y, (0, n * g - C)).view(rows, n, g).abs().amax(-1) / 448).clamp_min(2.0 ** -126)
    return y / scale.repeat_interleave(g, 1)[:, :C], scale


def _eight(y8, scale, y, group):
    """Both sides' quotients are off by at most 16 u (the norm's root is common to y and the scale: two products each, the
    scale's two more and its reciprocal's 2 u, and the first sum h), so that a value may land one step away only where
    the exact quotient is within 16 u of the border between the two."""
    q, s = _quotient(y, group)
    assert float(((scale.double() - s).abs() - 66 * U * s - HALF[F] * s).max()) <= 0
    want = q.clamp(-448, 448).float().to(torch.float8_e4m3fn)
    off = y8.view(torch.uint8) != want.view(torch.uint8)
    off &= (y8.float() != 0) | (want.float() != 0)  # the sign of a zero
    a, b, exact = y8[off].double(), want[off].double(), q[off]
    border = (a + b) / 2
    step = (y8.view(torch.uint8)[off].int() - want.view(torch.uint8)[off].int()).abs()
    assert bool((step == 1).all())
    assert bool(((exact - border).abs() <= 16 * U * border.abs()).all())
    # 32 u out of steps of 2^-4 and more of a value, of 2^-9 below 2^-6: less than one in 10^4
    assert int(off.sum()) <= 1e-4 * off.numel() + 3


def _flies(rows, C, T):
    """Whether the rows are so many that a thread has four of them (two past 32 vectors) in flight: 512 threads an SM, of
    148, for each.  Past 512 vectors there is one, but to 8 bits."""
    vectors = C * T.itemsize // 16
    threads = 16 if vectors <= 16 else 32 if vectors <= 64 else -(-vectors // 64) * 32
    return vectors <= 1024 and rows * threads >= 512 * 148 * (4 if vectors <= 32 else 2)


@pytest.mark.parametrize("rows,C", [(131008, 128), (20003, 256), (40001, 64), (11111, 512), (5003, 2048), (3001, 4096), (50002, 8)])
@pytest.mark.parametrize("T,RT", [(BF, None), (BF, BF), (BF, F), (F, None), (F, F)])
def test_norm_rows_in_flight(efla, rows, C, T, RT):
    assert _flies(rows, C, T)
    x, wt, res = _draw(rows, C, T, RT)
    h, y = _exact(x, wt, res)
    got, _, out = efla.norm_fwd(x, wt, res)
    _near(got, y, 64, "y")
    if res is not None:
        _near(out, h, 1, "res_out")
    for group in (0, 128):
        y8, scale, out8 = efla.norm_fwd(x, wt, res, out8=True, group=group)
        _eight(y8, scale, y, group)
        if res is not None:
            assert torch.equal(out8, out)
        again = efla.norm_fwd(x, wt, res, out8=True, group=group)
        assert torch.equal(again[0].view(torch.uint8), y8.view(torch.uint8)) and torch.equal(again[1], scale)
    for n in (1, 5, 33):  # the same rows without the others
        few, _, _ = efla.norm_fwd(x[-n:].contiguous(), wt, None if res is None else res[-n:].contiguous())
        assert torch.equal(few, got[-n:])


@pytest.mark.parametrize("rows,C", [(65536, 2048), (20000, 1001), (8190, 4097)])
@pytest.mark.parametrize("T,RT", [(BF, BF), (F, F)])
@pytest.mark.parametrize("group", [0, 128])
def test_norm_eight_bits_of_many_rows(efla, rows, C, T, RT, group):
    x, wt, res = _draw(rows, C, T, RT)
    y8, scale, _ = efla.norm_fwd(x, wt, res, out8=True, group=group)
    _eight(y8, scale, _exact(x, wt, res)[1], group)


@pytest.mark.parametrize("rows,C", [(20011, 256), (50001, 64), (5003, 2048), (3001, 4096), (2001, 8192), (1501, 16384), (4001, 1001), (9001, 130)])
@pytest.mark.parametrize("T,HT,stream", [(BF, BF, True), (BF, F, True), (F, F, False)])
def test_norm_bwd_many_rows(efla, rows, C, T, HT, stream):
    """Rows in plenty for each of two blocks an SM.  A dweight adds a slot's rows in turn (of at least 296 slots), up to
    16 slots, and the blocks by 32s in turn and a tree: 64 + rows / 296 + 32 with the products."""
    dy, wt, h = _draw(rows, C, T, HT)
    dr = _draw(rows + 1, C, HT, None)[0][1:].clone() if stream else None
    dx, ds, dw = efla.norm_bwd(dy, h, wt, dr)
    y, hh, ww = dy.double(), h.double(), wt.double()
    r = torch.rsqrt(hh.pow(2).mean(-1, keepdim=True) + 1e-6)
    u = y * ww
    mean = hh * r.pow(3) * (u * hh).mean(-1, keepdim=True)
    size = (u * r).abs() + hh.abs() * r.pow(3) * (u * hh).abs().mean(-1, keepdim=True)
    dh = u * r - mean
    if dr is not None:
        dh, size = dh + dr.double(), size + dr.double().abs()
    for got, name in ((dx, "dx"), (ds, "dres")):
        over = (got.double() - dh).abs() - 128 * U * size - HALF[got.dtype] * (dh.abs() + 128 * U * size)
        assert float(over.max()) <= 0, name
    term = y * hh * r
    over = (dw.double() - term.sum(0)).abs() - (96 + rows / 296 + 1) * U * term.abs().sum(0)
    assert float(over.max()) <= 0
