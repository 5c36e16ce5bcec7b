"""efla_scan_fwd, efla_scan_bwd and efla_scan_step on the GPU against float64.
The tolerances count rounded operations (``block_ref.scan_ops``) on magnitudes."""
import pytest
import torch

import block_ref as R

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32
GRADS = ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dh0")


@pytest.fixture(scope="module")
def efla():
    import delta_rule_linear_03_b200 as m
    return m


def _c(s):
    return {k: None if t is None else t.cuda() for k, t in s.items()}


def _fwd(efla, s, **kw):
    return efla.scan_fwd(**_c(s), **kw)


def _check_fwd(efla, s, softplus=True):
    y, h = _fwd(efla, s, softplus=softplus)
    ref, mag = R.scan(**s, softplus=softplus), R.scan(**s, softplus=softplus, mag=True)
    B, L, C = s["x"].shape
    ops = R.scan_ops(L, s["A"].shape[1], 0, 0, R.max_decay(s["dt"], s["A"], s["dt_bias"], softplus)) + 64
    R.close(y, ref["y"], mag["y"], ops, "y")
    R.close(h, ref["h_L"], mag["h_L"], ops, "h_L")


def _check_bwd(efla, s, dy, dh, softplus=True):
    got = dict(zip(GRADS, efla.scan_bwd(dy.cuda(), **_c(s), softplus=softplus, dh_L=None if dh is None else dh.cuda())))
    ref, mag = (R.scan(**s, softplus=softplus, dy=dy, dh_L=dh, mag=m) for m in (False, True))
    B, L, C = s["x"].shape
    ops = R.scan_ops(L, s["A"].shape[1], C, B, R.max_decay(s["dt"], s["A"], s["dt_bias"], softplus)) + 64
    skip = dict(dD="D", dz="z", ddt_bias="dt_bias")
    for k in GRADS:
        if k in skip and s[skip[k]] is None:
            assert got[k] is None
        else:
            R.close(got[k], ref[k], mag[k], ops, k)


def _cot(s, seed=9):
    g = torch.Generator().manual_seed(seed)
    B, L, C = s["x"].shape
    return torch.randn(B, L, C, generator=g).to(s["x"].dtype), torch.randn(B, C, s["A"].shape[1], generator=g)


SHAPES = [(1, 1, 1, 8, 1), (2, 2, 5, 16, 1), (1, 31, 32, 16, 1), (2, 32, 33, 8, 1), (1, 33, 70, 32, 2), (2, 65, 24, 64, 3), (3, 100, 96, 16, 4),
          (1, 17, 130, 64, 1), (2, 48, 200, 8, 2), (1, 257, 40, 32, 1)]


@pytest.mark.parametrize("B,L,C,N,G", SHAPES)
@pytest.mark.parametrize("T", [BF, F])
@pytest.mark.parametrize("ragged", [False, True])
def test_scan_fwd(efla, B, L, C, N, G, T, ragged):
    s = R.scan_inputs(B, L, C, N, G, T, lengths=[[L // 2, 0, L][b % 3] for b in range(B)] if ragged else None)
    _check_fwd(efla, s)


@pytest.mark.parametrize("B,L,C,N,G", SHAPES)
@pytest.mark.parametrize("T", [BF, F])
@pytest.mark.parametrize("ragged", [False, True])
def test_scan_bwd(efla, B, L, C, N, G, T, ragged):
    s = R.scan_inputs(B, L, C, N, G, T, lengths=[[L // 2, 0, L][b % 3] for b in range(B)] if ragged else None)
    _check_bwd(efla, s, *_cot(s))


@pytest.mark.parametrize("without", ["D", "z", "dt_bias", "h0"])
@pytest.mark.parametrize("softplus", [True, False])
def test_scan_options(efla, without, softplus):
    s = R.scan_inputs(2, 40, 24, 16)
    s[without] = None
    if not softplus:
        s["dt"] = 0.1 * s["dt"].abs()
        if s["dt_bias"] is not None:
            s["dt_bias"] = s["dt_bias"].abs() * 0.01
    _check_fwd(efla, s, softplus)
    dy, dh = _cot(s)
    _check_bwd(efla, s, dy, dh if without != "h0" else None, softplus)


def test_scan_many_channels(efla):
    """Channels enough that every SM has a block of four state values a lane."""
    s = R.scan_inputs(4, 35, 1288, 16, 1, BF, lengths=[35, 20, 0, 33])
    assert 4 * -(-1288 // 32) >= 148
    _check_fwd(efla, s)
    _check_bwd(efla, s, *_cot(s))


@pytest.mark.parametrize("B,L,C,N,G,lengths", [(1, 1000, 16, 16, 1, None), (2, 700, 40, 8, 2, [700, 130]), (3, 1030, 8, 64, 1, [0, 1, 1030]),
                                               (1, 5000, 64, 32, 1, None)])
@pytest.mark.parametrize("T", [BF, F])
def test_scan_in_segments(efla, B, L, C, N, G, lengths, T):
    """Few channels and a long sequence: cut into segments (scratch is asked for)."""
    assert efla.scan_fwd_workspace_size(B, L, C, G, N) > 0
    s = R.scan_inputs(B, L, C, N, G, T, lengths=lengths)
    _check_fwd(efla, s)
    if L <= 1030:
        _check_bwd(efla, s, *_cot(s))
    h = s["h0"].cuda()
    y, hl = _fwd(efla, s)
    y2, h2 = efla.scan_fwd(**dict(_c(s), h0=h), h_L=h)  # the state in place
    assert h2 is h and torch.equal(h, hl) and torch.equal(y2, y)


def test_scan_segments_grow_and_decay_out_of_range(efla):
    """A segment's whole decay may overflow or underflow where no state does."""
    B, L, C, N = 1, 1000, 16, 16
    assert efla.scan_fwd_workspace_size(B, L, C, 1, N) > 0
    s = R.scan_inputs(B, L, C, N, 1, F)
    s["A"] = torch.linspace(0.5, 1.0, C * N).reshape(C, N)  # growth of e^90 and more a segment, of a state of zeros
    s["h0"] = torch.zeros(B, C, N)
    s["x"][:, :690] = 0
    s["dt"][:, :690], s["dt"][:, 690:], s["dt_bias"] = 1.0, -3.0, torch.zeros(C)
    _check_fwd(efla, s)
    # Decay of e^-96 in the first 160 tokens, from 10^30.  Each step is off by 2^-22 of itself at most and a sum of
    # 160 of them by 160 2^-24, so the exponent by 96 (160 2^-24 + 2^-22) < 10^-3.
    s["A"], s["h0"] = torch.full((C, N), -1.0), torch.full((B, C, N), 1e30)
    s["x"][:], s["dt"][:, :160], s["dt"][:, 160:] = 0, -0.195, -300.0
    _, h = _fwd(efla, s)
    want = 1e30 * torch.exp(-160 * torch.nn.functional.softplus(s["dt"][0, 0, 0].double()))
    assert 1e-20 < float(want) < 1e-10 and float((h.cpu().double() / want - 1).abs().max()) <= 1e-3


def test_scan_padding_holds_anything(efla):
    s = R.scan_inputs(2, 70, 40, 16, 1, F, lengths=[33, 0])
    base = [t for t in _fwd(efla, s)] + [t for t in efla.scan_bwd(_cot(s)[0].cuda(), **_c(s))]
    dy = _cot(s)[0]
    for b, n in enumerate([33, 0]):
        for k in ("x", "dt", "z", "Bm", "Cm"):
            s[k][b, n:] = float("nan")
        dy[b, n:] = float("inf")
    again = [t for t in _fwd(efla, s)] + [t for t in efla.scan_bwd(dy.cuda(), **_c(s))]
    for p, q in zip(base, again):
        assert torch.equal(p, q) and bool(torch.isfinite(p).all())


def test_scan_values_at_the_edge(efla):
    """Steps that softplus takes to 0 and to large values, decays that vanish
    at once and never, an infinite input that reaches its own channel alone."""
    s = R.scan_inputs(1, 40, 36, 16, 1, F)
    s["dt"][0, 3] = -200.0
    s["dt"][0, 4] = 60.0
    s["dt"][0, 5] = 15.0
    s["A"][0] = 0.0
    s["A"][1] = -1e4
    _check_fwd(efla, s)
    y0, h0 = _fwd(efla, s)
    s["x"][0, 7, 5] = float("inf")
    y1, h1 = _fwd(efla, s)
    other = [c for c in range(36) if c != 5]
    assert torch.equal(y1[..., other], y0[..., other]) and torch.equal(h1[:, other], h0[:, other])
    assert torch.equal(y1[:, :7], y0[:, :7]) and not bool(torch.isfinite(y1[0, 7, 5]))


@pytest.mark.parametrize("T", [BF, F])
@pytest.mark.parametrize("off", [0, 16, 3])
def test_scan_strided_rows(efla, T, off):
    """Column slices of wider projections, aligned for vectors or not."""
    B, L, C, N, G = 2, 45, 48, 16, 2
    s = _c(R.scan_inputs(B, L, C, N, G, T))
    g = torch.Generator().manual_seed(4)
    xz = torch.randn(B, L, 2 * C + 32, generator=g).to(T).cuda()
    bc = torch.randn(B, L, 2 * G * N + 32, generator=g).to(T).cuda()
    v = dict(x=xz[..., off:off + C], z=xz[..., off + C:off + 2 * C], Bm=bc[..., off:off + G * N].unflatten(-1, (G, N)),
             Cm=bc[..., off + G * N:off + 2 * G * N].unflatten(-1, (G, N)))
    dense = {k: t.contiguous() for k, t in v.items()}
    dy = torch.randn(B, L, C, generator=g).to(T).cuda()
    for p, q in zip(efla.scan_fwd(**{**s, **v}), efla.scan_fwd(**{**s, **dense})):
        assert torch.equal(p, q)
    for p, q in zip(efla.scan_bwd(dy, **{**s, **v}), efla.scan_bwd(dy, **{**s, **dense})):
        assert torch.equal(p, q)
    one = lambda d: {k: t[:, 0] for k, t in d.items()}  # noqa: E731
    par = {k: s[k] for k in ("A", "D", "dt_bias")}
    h1, h2 = s["h0"].clone(), s["h0"].clone()
    dt1 = s["dt"][:, 0]
    y1 = efla.scan_step(dt=dt1, h=h1, **par, **one(v))
    y2 = efla.scan_step(dt=dt1.contiguous(), h=h2, **par, **{k: t.contiguous() for k, t in one(dense).items()})
    assert torch.equal(y1, y2) and torch.equal(h1, h2)


@pytest.mark.parametrize("B,C,N,G", [(1, 1, 8, 1), (3, 33, 16, 3), (2, 200, 32, 1), (5, 72, 64, 2), (70, 2048, 16, 1)])
@pytest.mark.parametrize("T", [BF, F])
@pytest.mark.parametrize("gate", [True, False])
def test_scan_step(efla, B, C, N, G, T, gate):
    s = R.scan_inputs(B, 1, C, N, G, T)
    if not gate:
        s["z"] = None
    h = s["h0"].cuda()
    one = {k: None if s[k] is None else s[k][:, 0].cuda() for k in ("x", "dt", "Bm", "Cm", "z")}
    y = efla.scan_step(h=h, A=s["A"].cuda(), D=s["D"].cuda(), dt_bias=s["dt_bias"].cuda(), **one)
    ref, mag = R.scan(**s), R.scan(**s, mag=True)
    ops = R.scan_ops(1, N, 0, 0, R.max_decay(s["dt"], s["A"], s["dt_bias"])) + 64
    R.close(y[:, None], ref["y"], mag["y"], ops, "y")
    R.close(h, ref["h_L"], mag["h_L"], ops, "h")


@pytest.mark.parametrize("C,L", [(96, 60), (1288 * 4, 12), (16, 900)])
def test_scan_in_pieces_and_steps(efla, C, L):
    """Pieces of a prompt, each from the state of the one before, then single
    tokens, against one pass: both within the tolerance of the whole."""
    s = R.scan_inputs(1, L, C, 16, 1, F)
    g = _c(s)
    h, at, ys = g["h0"].clone(), 0, []
    for n in (L // 2, 1, L // 3):
        part = {k: g[k][:, at:at + n].contiguous() for k in ("x", "dt", "z", "Bm", "Cm")}
        y, h = efla.scan_fwd(**part, A=g["A"], D=g["D"], dt_bias=g["dt_bias"], h0=h, h_L=h)
        ys.append(y)
        at += n
    for t in range(at, L):
        one = {k: g[k][:, t].contiguous() for k in ("x", "dt", "z", "Bm", "Cm")}
        ys.append(efla.scan_step(h=h, A=g["A"], D=g["D"], dt_bias=g["dt_bias"], **one)[:, None])
    ref, mag = R.scan(**s), R.scan(**s, mag=True)
    ops = R.scan_ops(L, 16, 0, 0, R.max_decay(s["dt"], s["A"], s["dt_bias"])) + 64
    R.close(torch.cat(ys, 1), ref["y"], mag["y"], ops, "y")
    R.close(h, ref["h_L"], mag["h_L"], ops, "h")


def test_scan_empty(efla):
    B, C, N = 2, 24, 16
    e = torch.zeros(B, 0, C, device="cuda")
    bc = torch.zeros(B, 0, 1, N, device="cuda")
    A, h0 = -torch.ones(C, N, device="cuda"), torch.randn(B, C, N, device="cuda")
    y, h = efla.scan_fwd(e, e, A, bc, bc, h0=h0)
    assert y.shape == (B, 0, C) and torch.equal(h, h0)
    dh = torch.randn(B, C, N, device="cuda")
    got = dict(zip(GRADS, efla.scan_bwd(e, e, e, A, bc, bc, D=A[:, 0].contiguous(), h0=h0, dh_L=dh)))
    assert not got["dA"].any() and not got["dD"].any() and torch.equal(got["dh0"], dh)


def test_scan_refuses(efla):
    s = _c(R.scan_inputs(2, 8, 16, 16, 2))
    for k, bad in [("x", s["x"][0]), ("dt", s["dt"].bfloat16()), ("dt", s["dt"][:1]), ("A", s["A"].double()), ("A", s["A"][:8]), ("Bm", s["Bm"][:, :4]),
                   ("Cm", s["Cm"].bfloat16()), ("D", s["D"][:3]), ("z", s["z"].cpu()), ("h0", s["h0"].bfloat16()),
                   ("lengths", torch.zeros(3, dtype=torch.int32, device="cuda")), ("x", s["x"].transpose(1, 2).contiguous().transpose(1, 2))]:
        with pytest.raises(ValueError):
            efla.scan_fwd(**{**s, k: bad})
    with pytest.raises(TypeError):
        efla.scan_fwd(**{**s, "x": s["x"].half()})
    with pytest.raises(ValueError):
        efla.scan_step(*(s[k][:, 0] for k in ("x", "dt")), s["A"], s["Bm"][:, 0], s["Cm"][:, 0], None)
    with pytest.raises(efla.EflaError):  # a state size that is not offered
        efla.scan_fwd(s["x"], s["dt"], s["A"][:, :12].contiguous(), s["Bm"][..., :12].contiguous(), s["Cm"][..., :12].contiguous())
    with pytest.raises(efla.EflaError):
        efla.scan_fwd(**s, y=s["x"])


@pytest.mark.parametrize("B,L,C,N", [(2, 90, 24, 16), (1, 40, 5000, 16), (1, 1000, 16, 64)])
def test_scan_steps_of_zero_leave_the_state(efla, B, L, C, N):
    """Tokens whose step underflows to 0, and padding, keep every bit of the state."""
    s = R.scan_inputs(B, L, C, N, 1, F)
    n = 33
    cut = {k: (t[:, :n].contiguous() if k in ("x", "dt", "Bm", "Cm", "z") else t) for k, t in s.items()}
    _, h = _fwd(efla, cut)
    s["dt"][:, n:] = -300.0
    _, h1 = _fwd(efla, s)
    s["lengths"] = torch.full((B,), n, dtype=torch.int32)
    y2, h2 = _fwd(efla, s)
    assert torch.equal(h, h1) and torch.equal(h, h2) and not y2[:, n:].any()
