"""efla_conv_fwd, efla_conv_bwd and efla_conv_step on the GPU against float64.

Rounded operations of y: K products and sums, and the SiLU, whose exponential is
off by 2 ulp and by its argument's rounding, |v| log2 e u, with a division of
2 ulp behind it: 16 + 2 |v| u.  The gradients add K (dx) or all tokens (dweight)
of such terms in turn."""
import pytest
import torch

import block_ref as R

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def efla():
    import delta_rule_linear_03_b200 as m
    return m


def _draw(B, L, C, K, T, seed=0):
    g = torch.Generator().manual_seed(seed + 7 * L + C + K)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    return r(B, L, C).to(T), r(C, K) * 0.5, r(C) * 0.5, r(B, K - 1, C).to(T)


def _heads(t, H):
    B, L, C = t.shape
    return t.view(B, L, H, C // H).transpose(1, 2).contiguous() if H else t


def _c(t):
    return None if t is None else t.cuda()


SIZES = [(1, 1, 1), (2, 2, 3), (3, 3, 8), (2, 15, 32), (1, 16, 33), (2, 17, 256), (3, 127, 264), (2, 128, 40), (1, 129, 1001), (2, 300, 64), (1, 1030, 16)]
OPTIONS = [dict(), dict(bias=False, silu=False), dict(state=True), dict(state=True, ragged=True), dict(ragged=True, silu=False)]


def _case(B, L, C, K, T, bias=True, silu=True, state=False, ragged=False):
    x, wt, b, st = _draw(B, L, C, K, T)
    lengths = torch.tensor([[L // 2, L, 0, 1][i % 4] for i in range(B)], dtype=torch.int32) if ragged else None
    return x, wt, b if bias else None, st if state else None, lengths, silu


def _ops(pre):
    return 32 + 2 * float(pre.abs().max()) if pre.numel() else 32


@pytest.mark.parametrize("B,L,C", SIZES)
@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("T", [BF, F])
@pytest.mark.parametrize("opt", OPTIONS)
def test_conv_fwd(efla, B, L, C, K, T, opt):
    x, wt, b, st, lengths, silu = _case(B, L, C, K, T, **opt)
    if lengths is not None:  # padding holds anything
        for i, n in enumerate(lengths.tolist()):
            x[i, n:] = float("nan")
    y, so = efla.conv_fwd(_c(x), _c(wt), _c(b), _c(st), _c(lengths), silu, want_state=True)
    ry, rs, pre, _ = R.conv_fwd(x, wt, b, st, lengths, silu)
    mag = R.conv_fwd(x, wt, b, st, lengths, silu, mag=True)[0]
    R.close(y, ry, 1.1 * mag + ry.abs(), _ops(pre), "y")
    assert torch.equal(R.w(so), rs)


@pytest.mark.parametrize("B,L,C", SIZES)
@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("T", [BF, F])
@pytest.mark.parametrize("opt", OPTIONS)
def test_conv_bwd(efla, B, L, C, K, T, opt):
    x, wt, b, st, lengths, silu = _case(B, L, C, K, T, **opt)
    dy = _draw(B, L, C, K, T, seed=1)[0]
    ds = _draw(B, L, C, K, T, seed=2)[3] if st is not None else None
    if lengths is not None:
        for i, n in enumerate(lengths.tolist()):
            x[i, n:] = float("nan")
            dy[i, n:] = float("inf")
        dy_ref = torch.where(torch.isinf(dy), 0.0, dy.float()).to(T)
        x_ref = torch.where(torch.isnan(x), 0.0, x.float()).to(T)
    else:
        dy_ref, x_ref = dy, x
    got = efla.conv_bwd(_c(dy), _c(x), _c(wt), _c(b), _c(st), _c(lengths), silu, dstate_out=_c(ds))
    ref = R.conv_bwd(dy_ref, x_ref, wt, b, st, lengths, silu, ds)
    mag = R.conv_bwd(dy_ref, x_ref, wt, b, st, lengths, silu, ds, mag=True)
    ops = _ops(R.conv_fwd(x_ref, wt, b, st, lengths, silu)[2])
    R.close(got[0], ref[0], mag[0], ops, "dx")
    R.close(got[1], ref[1], mag[1], ops + B * L, "dweight")
    if b is None:
        assert got[2] is None
    else:
        R.close(got[2], ref[2], mag[2], ops + B * L, "dbias")
    if st is None:
        assert got[3] is None
    else:
        R.close(got[3], ref[3], mag[3], ops, "dstate")


@pytest.mark.parametrize("H,d", [(1, 32), (3, 64), (2, 128), (4, 6)])
@pytest.mark.parametrize("T", [BF, F])
def test_conv_head_layout(efla, H, d, T):
    """[B,H,L,d] holds the same values, and its gradients are the same."""
    x, wt, b, st = _draw(2, 37, H * d, 4, T)
    y, _ = efla.conv_fwd(_c(x), _c(wt), _c(b), _c(st))
    yh, _ = efla.conv_fwd(_c(x), _c(wt), _c(b), _c(st), heads=H)
    assert yh.shape == (2, H, 37, d) and torch.equal(yh, _heads(y, H))
    dy = _draw(2, 37, H * d, 4, T, seed=1)[0].cuda()
    for p, q in zip(efla.conv_bwd(dy, _c(x), _c(wt), _c(b), _c(st)), efla.conv_bwd(_heads(dy, H), _c(x), _c(wt), _c(b), _c(st), heads=H)):
        assert torch.equal(p, q)


@pytest.mark.parametrize("off,C", [(8, 64), (3, 64), (0, 30)])
@pytest.mark.parametrize("T", [BF, F])
def test_conv_strided_rows(efla, off, C, T):
    """A column slice of a wider projection, aligned for vectors or not."""
    wide = _draw(2, 50, 104, 4, T)[0].cuda()
    _, wt, b, st = (_c(t) for t in _draw(2, 50, C, 4, T))
    x = wide[..., off:off + C]
    dense = x.contiguous()
    for p, q in zip(efla.conv_fwd(x, wt, b, st, want_state=True), efla.conv_fwd(dense, wt, b, st, want_state=True)):
        assert torch.equal(p, q)
    for p, q in zip(efla.conv_bwd(dense, x, wt, b, st), efla.conv_bwd(dense, dense, wt, b, st)):
        assert torch.equal(p, q)
    s1, s2 = st.clone(), st.clone()
    assert torch.equal(efla.conv_step(x[:, 0], s1, wt, b), efla.conv_step(dense[:, 0].contiguous(), s2, wt, b)) and torch.equal(s1, s2)


@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("T", [BF, F])
@pytest.mark.parametrize("cuts", [[1, 1, 1, 40], [20, 23], [2, 0, 41]])
def test_conv_in_pieces_and_steps(efla, K, T, cuts):
    """A prompt in pieces, each from the state of the one before (updated in
    place), and then single tokens give the bits of one pass: every y is the
    same sum in the same order."""
    x, wt, b, st = (_c(t) for t in _draw(2, 47, 40, K, T))
    whole, end = efla.conv_fwd(x, wt, b, st, want_state=True)
    state, at, out = st.clone(), 0, []
    for n in cuts:
        y, s = efla.conv_fwd(x[:, at:at + n].contiguous(), wt, b, state, state_out=state)
        assert s is state
        out.append(y)
        at += n
    for t in range(at, 47):
        out.append(efla.conv_step(x[:, t], state, wt, b)[:, None])
    assert torch.equal(torch.cat(out, 1), whole) and torch.equal(state, end)


def test_conv_lengths_are_taken_into_range(efla):
    x, wt, b, st = (_c(t) for t in _draw(3, 20, 16, 4, BF))
    lengths = torch.tensor([-5, 1000, 20], dtype=torch.int32, device="cuda")
    fit = torch.tensor([0, 20, 20], dtype=torch.int32, device="cuda")
    for p, q in zip(efla.conv_fwd(x, wt, b, st, lengths, want_state=True), efla.conv_fwd(x, wt, b, st, fit, want_state=True)):
        assert torch.equal(p, q)


def test_conv_refuses(efla):
    x, wt = torch.zeros(2, 8, 16, device="cuda"), torch.zeros(16, 4, device="cuda")
    st = torch.zeros(2, 3, 16, device="cuda")
    for bad in (lambda: efla.conv_fwd(x[0], wt), lambda: efla.conv_fwd(x, wt[:8]), lambda: efla.conv_fwd(x, wt.bfloat16()),
                lambda: efla.conv_fwd(x, wt, state=st.bfloat16()), lambda: efla.conv_fwd(x, wt, state=st[:1]), lambda: efla.conv_fwd(x, wt, heads=3),
                lambda: efla.conv_fwd(x, wt, lengths=torch.zeros(2, dtype=torch.int64, device="cuda")), lambda: efla.conv_fwd(x[:, :4], wt),
                lambda: efla.conv_step(x[:, 0], None, wt), lambda: efla.conv_step(x[:, 0], st[:, :2], wt), lambda: efla.conv_bwd(x[:1], x, wt)):
        with pytest.raises(ValueError):
            bad()
    for K in (1, 5):
        with pytest.raises(efla.EflaError):
            efla.conv_fwd(x, torch.zeros(16, K, device="cuda"))
    with pytest.raises(efla.EflaError):
        efla.conv_fwd(x, wt, y=x)
