"""efla_norm_fwd and efla_norm_bwd on the GPU against float64.

Rounded operations between the inputs and a value: the sum of squares takes a
thread's up to 32 terms in turn and then a tree of 10 levels, half of whose
error reaches 1/sqrt, with a division, an addition, the root, a reciprocal and
two products behind it: under 64.  The gradient has two such sums: 128.  dweight
adds a block's rows in turn and then the blocks: under 64 + rows."""
import pytest
import torch

import block_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def efla():
    import delta_rule_linear_03_b200 as m
    return m


BF, F = torch.bfloat16, torch.float32
SIZES = [(1, 1), (3, 7), (2, 8), (5, 64), (700, 128), (33, 129), (3, 200), (17, 256), (2000, 512), (9, 1000), (7, 1001), (300, 1024), (700, 2048),
         (5, 2056), (3, 4096), (600, 4104), (2, 8192), (3, 8193), (2, 16383), (2, 16384)]
TYPES = [(BF, None), (BF, BF), (BF, F), (F, None), (F, F)]


def _draw(rows, C, T, RT, seed=0):
    g = torch.Generator().manual_seed(seed + rows + C)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    return r(rows, C).to(T), (1 + 0.3 * r(C)), None if RT is None else (2 * r(rows, C)).to(RT)


@pytest.mark.parametrize("rows,C", SIZES)
@pytest.mark.parametrize("T,RT", TYPES)
def test_norm_fwd(efla, rows, C, T, RT):
    x, wt, res = _draw(rows, C, T, RT)
    y, scale, out = efla.norm_fwd(x.cuda(), wt.cuda(), None if res is None else res.cuda())
    ry, rh = R.norm_fwd(x, wt, res)
    assert scale is None and y.dtype == T
    R.close(y, ry, ry.abs(), 64, "y")
    if res is None:
        assert out is None
    else:
        assert out.dtype == RT
        R.close(out, rh, rh.abs(), 1, "res_out")


@pytest.mark.parametrize("rows,C", SIZES)
@pytest.mark.parametrize("T,RT", TYPES)
@pytest.mark.parametrize("group", [0, 128])
def test_norm_fwd_eight_bits(efla, rows, C, T, RT, group):
    x, wt, res = _draw(rows, C, T, RT, seed=1)
    y8, scale, out = efla.norm_fwd(x.cuda(), wt.cuda(), None if res is None else res.cuda(), out8=True, group=group)
    ry, rh = R.norm_fwd(x, wt, res)
    rs = R.norm_scale(ry, group)
    assert y8.dtype == torch.float8_e4m3fn and tuple(scale.shape) == tuple(rs.shape)
    R.close(scale, rs, rs, 66, "scale")
    cols = torch.arange(C) // (group or C)
    s = R.w(scale)[:, cols]
    # half a step of e4m3, at least half of its smallest, 2^-10, in units of the scale
    tol = torch.maximum(2.0 ** -4 * ry.abs(), 2.0 ** -10 * s) * (1 + 2.0 ** -10) + 70 * R.U * ry.abs()
    assert bool(((R.w(y8) * s - ry).abs() <= tol).all())
    if res is not None:
        R.close(out, rh, rh.abs(), 1, "res_out")


@pytest.mark.parametrize("rows,C", [(9, 130), (70, 255), (9, 385), (9, 511), (9, 514), (9, 1029), (700, 1001), (9, 2047), (9, 4099), (9, 6145), (9, 12289),
                                    (9, 16369), (9, 16371)])
@pytest.mark.parametrize("T,RT", [(BF, None), (BF, F), (F, F)])
def test_norm_fwd_rows_off_their_boundary(efla, rows, C, T, RT):
    """Rows that begin at every offset from a 16-byte boundary."""
    test_norm_fwd(efla, rows, C, T, RT)
    for group in (0, 128):
        test_norm_fwd_eight_bits(efla, rows, C, T, RT, group)


@pytest.mark.parametrize("rows,C", SIZES)
@pytest.mark.parametrize("T,HT,dres", [(BF, BF, True), (BF, BF, False), (BF, F, True), (BF, F, False), (F, F, True), (F, F, False)])
def test_norm_bwd(efla, rows, C, T, HT, dres):
    dy, wt, h = _draw(rows, C, T, HT, seed=2)
    dr = _draw(rows, C, HT, None, seed=3)[0] if dres else None
    dx, ds, dw = efla.norm_bwd(dy.cuda(), h.cuda(), wt.cuda(), None if dr is None else dr.cuda())
    rdh, rdw = R.norm_bwd(dy, h, wt, dr)
    mdh, mdw = R.norm_bwd(dy, h, wt, dr, mag=True)
    assert dx.dtype == T and ds.dtype == HT and (ds is dx) == (HT == T)
    R.close(dx, rdh, mdh, 128, "dx")
    R.close(ds, rdh, mdh, 128, "dres")
    R.close(dw, rdw, mdw, 64 + rows, "dweight")


def test_norm_no_rows(efla):
    z = torch.zeros(0, 256, device="cuda", dtype=BF)
    wt = torch.ones(256, device="cuda")
    y, scale, _ = efla.norm_fwd(z, wt, out8=True)
    assert y.shape == (0, 256) and scale.shape == (0, 2)
    dx, _, dw = efla.norm_bwd(z, z, wt)
    assert dx.shape == (0, 256) and not dw.any()


def test_norm_leading_dimensions(efla):
    """The mixer's output [B,H,L,d] is normed per head."""
    x, wt, _ = _draw(2 * 3 * 5, 64, F, None)
    y, scale, _ = efla.norm_fwd(x.view(2, 3, 5, 64).cuda(), wt.cuda(), out8=True)
    assert y.shape == (2, 3, 5, 64) and scale.shape == (2, 3, 5, 1)


@pytest.mark.parametrize("C", [100, 1001, 1024, 4096])
def test_norm_in_place(efla, C):
    x, wt, res = _draw(50, C, BF, BF)
    y, _, out = efla.norm_fwd(x.cuda(), wt.cuda(), res.cuda())
    stream = res.cuda()
    y2, _, out2 = efla.norm_fwd(x.cuda(), wt.cuda(), stream, res_out=stream)
    assert out2 is stream and torch.equal(out2, out) and torch.equal(y2, y)
    xs = x.cuda()
    y3, _, out3 = efla.norm_fwd(xs, wt.cuda(), res.cuda(), y=xs)
    assert torch.equal(y3, y) and torch.equal(out3, out)
    xs = x.cuda()
    y4, _, out4 = efla.norm_fwd(xs, wt.cuda(), res.cuda(), res_out=xs)
    assert torch.equal(y4, y) and torch.equal(out4, out)


@pytest.mark.parametrize("C", [300, 512, 513])
@pytest.mark.parametrize("group", [0, 128])
def test_norm_values_at_the_edge(efla, C, group):
    """Rows of zeros, of tiny values, with a NaN, with an infinity, beside an ordinary one."""
    g = torch.Generator().manual_seed(5)
    x = torch.randn(6, C, generator=g)
    x[0] = 0
    x[1] *= 1e-20
    x[2, 3] = float("nan")
    x[3, C - 1] = float("inf")
    wt = torch.ones(C)
    wt[:] = 1.0
    y, _, _ = efla.norm_fwd(x.cuda(), wt.cuda())
    y8, scale, _ = efla.norm_fwd(x.cuda(), wt.cuda(), out8=True, group=group)
    y, y8, scale = y.cpu(), y8.float().cpu(), scale.cpu()
    assert not y[0].any() and not y8[0].any() and bool((scale[0] == 2.0 ** -126).all())
    ry, _ = R.norm_fwd(x[[1, 4, 5]], wt)
    R.close(y[[1, 4, 5]], ry, ry.abs(), 64, "y")
    assert bool(torch.isnan(y[2]).all()) and bool(torch.isnan(y8[2]).all()) and bool(torch.isnan(scale[2]).all())
    # 1 / sqrt(inf) is 0: the finite values are 0, the infinite one is 0 inf = NaN, and so is its group
    assert not y[3, :-1].any() and bool(torch.isnan(y[3, -1]))
    last = (C - 1) // 128 * 128 if group else 0
    assert bool(torch.isnan(y8[3, last:]).all()) and not y8[3, :last].any()
    # the ordinary rows are what they are without their neighbours
    alone, s1, _ = efla.norm_fwd(x[4:].cuda(), wt.cuda(), out8=True, group=group)
    assert torch.equal(alone.float().cpu(), y8[4:]) and torch.equal(s1.cpu(), scale[4:])


def test_norm_refuses(efla):
    x, wt = torch.zeros(4, 64, device="cuda"), torch.ones(64, device="cuda")
    for bad in (lambda: efla.norm_fwd(x.double(), wt), lambda: efla.norm_fwd(x, wt, x.bfloat16()), lambda: efla.norm_bwd(x, x.half(), wt)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: efla.norm_fwd(x, wt[:32]), lambda: efla.norm_fwd(x, wt.double()), lambda: efla.norm_fwd(x.t(), wt[:4]),
                lambda: efla.norm_fwd(x, wt, group=32), lambda: efla.norm_fwd(x, wt, x[:2]), lambda: efla.norm_fwd(x, wt.cpu()),
                lambda: efla.norm_fwd(x, wt, res_out=x), lambda: efla.norm_fwd(x, wt, scale=wt), lambda: efla.norm_bwd(x, x, wt, x[:1])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(efla.EflaError):
        efla.norm_fwd(torch.zeros(2, 20000, device="cuda"), torch.ones(20000, device="cuda"))
    with pytest.raises(efla.EflaError):  # y over the residual
        efla.norm_fwd(x, wt, x.clone(), y=x, res_out=x)
