"""The operators together, as a block uses them, and under streams, graphs and
repetition."""
import pytest
import torch

import block_ref as R
import oracle
from parity import np64

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def efla():
    import delta_rule_linear_03_b200 as m
    return m


def _randn(g, *s, std=1.0):
    return torch.randn(s, generator=g, device="cuda") * std


def _block(B, L, H, d, N, seed=0):
    """Weights and inputs of a block with a mixer half and a scan half of width H d."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    C = H * d
    p = dict(H=H, w1=1 + 0.1 * _randn(g, C), proj=_randn(g, C, 4 * C, std=C ** -0.5).to(BF), cw=_randn(g, 4 * C, 4, std=0.5), cb=_randn(g, 4 * C, std=0.1),
             A=-torch.arange(1, N + 1, device="cuda") * torch.exp(0.1 * _randn(g, C, N)), bc=_randn(g, C, 2 * N, std=C ** -0.5).to(BF),
             wdt=_randn(g, C, C, std=0.3 * C ** -0.5).to(BF), dt_bias=torch.full((C,), -4.0, device="cuda"), D=torch.ones(C, device="cuda"),
             w2=1 + 0.1 * _randn(g, d), w3=1 + 0.1 * _randn(g, C))
    return p, _randn(g, B, L, C).to(BF), _randn(g, B, L, C).to(BF)


def _prompt(efla, p, x, res, conv_state=None, S=None, h=None):
    """norm -> projection -> convolutions -> mixer and scan -> per-head and row norms in 8 bits."""
    H = p["H"]
    B, L, C = x.shape
    N = p["A"].shape[1]
    n1, _, res = efla.norm_fwd(x, p["w1"], res)
    u = n1 @ p["proj"]
    cs, outs = [], []
    for i in range(4):
        w, b = p["cw"][i * C:(i + 1) * C], p["cb"][i * C:(i + 1) * C]
        y, s = efla.conv_fwd(u[..., i * C:(i + 1) * C], w, b, None if conv_state is None else conv_state[i], heads=H if i < 3 else 0, want_state=True)
        outs.append(y)
        cs.append(s)
    q, k, v, xs = outs
    beta = torch.full((B, H, L), 0.5, device="cuda")
    o, S = efla.chunk_fwd(q, (k * 0.1).contiguous(), v, beta, S, out_dtype=BF)
    o8, oscale, _ = efla.norm_fwd(o, p["w2"], out8=True)
    bc = (xs @ p["bc"]).view(B, L, 2, N)
    y, h = efla.scan_fwd(xs, xs @ p["wdt"], p["A"], bc[:, :, :1], bc[:, :, 1:], D=p["D"], z=u[..., 3 * C:], dt_bias=p["dt_bias"], h0=h)
    y8, yscale, _ = efla.norm_fwd(y, p["w3"], out8=True)
    return dict(res=res, q=q, k=k, v=v, o=o, o8=o8, oscale=oscale, xs=xs, u=u, bc=bc, y=y, y8=y8, yscale=yscale), cs, S, h


def test_block_prompt_against_float64(efla):
    """Each stage of the block against float64 on the stage's own inputs."""
    p, x, res = _block(2, 70, 2, 128, 16)
    r, cs, S, h = _prompt(efla, p, x, res)
    C = x.shape[2]
    ry, rh = R.norm_fwd(x, p["w1"], res)
    R.close(r["res"], rh, rh.abs(), 1, "residual stream")
    for i, name in enumerate(("q", "k", "v", "xs")):
        part = r["u"][..., i * C:(i + 1) * C]
        cy, st, pre, _ = R.conv_fwd(part, p["cw"][i * C:(i + 1) * C], p["cb"][i * C:(i + 1) * C])
        mag = R.conv_fwd(part, p["cw"][i * C:(i + 1) * C], p["cb"][i * C:(i + 1) * C], mag=True)[0]
        got = r[name] if name == "xs" else r[name].transpose(1, 2).reshape(2, 70, C)
        R.close(got, cy, 1.1 * mag + cy.abs(), 32 + 2 * float(pre.abs().max()), name)
        assert torch.equal(R.w(cs[i]), st)
    o, _ = oracle.recurrence(r["q"].cpu(), (r["k"] * 0.1).contiguous().cpu(), r["v"].cpu(), torch.full((2, 2, 70), 0.5), None)
    assert abs(np64(r["o"]) - o).max() <= 2e-2 * (o ** 2).mean() ** 0.5 + 2.0 ** -8 * abs(o).max()
    s = dict(x=r["xs"], dt=r["xs"] @ p["wdt"], A=p["A"], Bm=r["bc"][:, :, :1], Cm=r["bc"][:, :, 1:], D=p["D"], z=r["u"][..., 3 * C:], dt_bias=p["dt_bias"])
    ref, mag = R.scan(**s), R.scan(**s, mag=True)
    ops = R.scan_ops(70, 16, 0, 0, R.max_decay(s["dt"], s["A"], s["dt_bias"])) + 64
    R.close(r["y"], ref["y"], mag["y"], ops, "scan")
    R.close(h, ref["h_L"], mag["h_L"], ops, "scan state")
    for src, w8, y8, sc in ((r["o"], p["w2"], r["o8"], r["oscale"]), (r["y"], p["w3"], r["y8"], r["yscale"])):
        ry, _ = R.norm_fwd(src, w8)
        s = R.w(sc).repeat_interleave(128, -1)
        tol = torch.maximum(2.0 ** -4 * ry.abs(), 2.0 ** -10 * s) * (1 + 2.0 ** -10) + 70 * R.U * ry.abs()
        assert bool(((R.w(y8) * s - ry).abs() <= tol).all())


def test_block_prompt_then_tokens(efla):
    """A prompt, then single tokens from its states: the scan half and the
    convolutions against one pass over all tokens."""
    p, x, res = _block(2, 40, 2, 64, 16, seed=3)
    C, n = x.shape[2], 33
    whole, _, _, h_all = _prompt(efla, p, x, res)
    _, cs, _, h = _prompt(efla, p, x[:, :n].contiguous(), res[:, :n].contiguous())
    for t in range(n, 40):
        n1, _, _ = efla.norm_fwd(x[:, t].contiguous(), p["w1"], res[:, t].contiguous())
        u = whole["u"][:, t]  # the projection's own rounding depends on its shape
        outs = [efla.conv_step(u[:, i * C:(i + 1) * C], cs[i], p["cw"][i * C:(i + 1) * C], p["cb"][i * C:(i + 1) * C]) for i in range(4)]
        for got, name in zip(outs[:3], "qkv"):
            assert torch.equal(got.view(2, 2, 64), whole[name][:, :, t])
        assert torch.equal(outs[3], whole["xs"][:, t])
        bc = whole["bc"][:, t]
        y = efla.scan_step(outs[3], (whole["xs"] @ p["wdt"])[:, t], p["A"], bc[:, :1], bc[:, 1:], h, D=p["D"], z=u[:, 3 * C:], dt_bias=p["dt_bias"])
        # two orders of fp32 sums, each rounded to bf16 once: a step of bf16 apart at most, beside the sums' own 1e-5
        d = (y.float() - whole["y"][:, t].float()).abs()
        assert bool((d <= 2.0 ** -7 * whole["y"][:, t].float().abs() + 1e-4).all())
    assert float((h - h_all).abs().max()) <= 1e-4 * float(h_all.abs().max())


def test_block_training_gradient_against_differences(efla):
    """conv -> scan -> norm in fp32: the chained gradients against central
    differences of the chained float64 formulas along a random direction."""
    g = torch.Generator().manual_seed(11)
    B, L, C, N, K = 2, 24, 20, 8, 4
    s = R.scan_inputs(B, L, C, N, 1, torch.float32, seed=12)
    x, cw, cb, nw, dy, d = (torch.randn(k, generator=g) for k in ((B, L, C), (C, K), (C,), (C,), (B, L, C), (B, L, C)))
    par = {k: s[k] for k in ("dt", "A", "Bm", "Cm", "D", "z", "dt_bias")}

    def loss(xx):
        u = R.conv_fwd(xx, cw, cb)[0]
        y = R.scan(x=u, **par)["y"]
        return float((R.norm_fwd(y, nw)[0] * dy.double()).sum())

    quotient = (loss(x.double() + 1e-5 * d.double()) - loss(x.double() - 1e-5 * d.double())) / 2e-5
    c = lambda t: t.cuda()  # noqa: E731
    u, _ = efla.conv_fwd(c(x), c(cw), c(cb))
    pc = {k: c(t) for k, t in par.items()}
    y, _ = efla.scan_fwd(u, **pc)
    dn, _, _ = efla.norm_bwd(c(dy), y, c(nw))
    du = efla.scan_bwd(dn, u, **pc)[0]
    dx = efla.conv_bwd(du, c(x), c(cw), c(cb))[0]
    got = float((R.w(dx) * d.double()).sum())
    # fp32 through three operators of some hundred operations each, against the sum of the terms' magnitudes
    assert abs(got - quotient) <= 1000 * R.U * float((R.w(dx) * d.double()).abs().sum())


def _calls(efla, seed=0, lead=1):
    """Every operator once: name -> call on fixed inputs."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, L, C, N = 2, 400, 64, 16
    x, dt, z, dy, r = (_randn(g, B, L, C).to(BF) for _ in range(5))
    A, cw, w = -torch.exp(_randn(g, C, N, std=0.3)), _randn(g, C, 4), _randn(g, C)
    Bm, Cm = _randn(g, B, L, 1, N).to(BF), _randn(g, B, L, 1, N).to(BF)
    h0, cs = _randn(g, B, C, N), _randn(g, B, 3, C).to(BF)
    lengths = torch.tensor([400, 123], dtype=torch.int32, device="cuda")
    hs, ct = h0.clone(), cs.clone()
    return {
        "norm_fwd": lambda: efla.norm_fwd(x, w, r), "norm_fwd8": lambda: efla.norm_fwd(x, w, r, out8=True), "norm_bwd": lambda: efla.norm_bwd(dy, x, w, r),
        "conv_fwd": lambda: efla.conv_fwd(x, cw, w, cs, lengths, want_state=True), "conv_bwd": lambda: efla.conv_bwd(dy, x, cw, w, cs, lengths),
        "conv_step": lambda: (efla.conv_step(x[:, 0], ct.copy_(cs), cw, w), ct),
        "scan_fwd": lambda: efla.scan_fwd(x, dt, A, Bm, Cm, D=w, z=z, dt_bias=w, h0=h0, lengths=lengths),
        "scan_bwd": lambda: efla.scan_bwd(dy, x, dt, A, Bm, Cm, D=w, z=z, dt_bias=w, h0=h0, lengths=lengths, dh_L=h0),
        "scan_step": lambda: (efla.scan_step(x[:, 0], dt[:, 0], A, Bm[:, 0], Cm[:, 0], hs.copy_(h0), D=w, z=z[:, 0], dt_bias=w), hs)}


NAMES = ("norm_fwd", "norm_fwd8", "norm_bwd", "conv_fwd", "conv_bwd", "conv_step", "scan_fwd", "scan_bwd", "scan_step")


def _same(a, b):
    return all((p is None and q is None) or torch.equal(p.view(torch.uint8) if p.dtype.itemsize == 1 else p,
                                                         q.view(torch.uint8) if q.dtype.itemsize == 1 else q) for p, q in zip(a, b))


def _copy(out):
    return [None if t is None else t.clone() for t in out]


@pytest.mark.parametrize("name", NAMES)
def test_same_bits_again(efla, name):
    call = _calls(efla)[name]
    first = _copy(call())
    for _ in range(3):
        assert _same(first, call())


@pytest.mark.parametrize("name", NAMES)
def test_captured_and_replayed(efla, name):
    """A captured call gives the eager bits, with other inputs in between; two
    graphs of one process do not share scratch."""
    one, two = _calls(efla, 0)[name], _calls(efla, 1)[name]
    e1, e2 = _copy(one()), _copy(two())
    torch.cuda.synchronize()
    graphs, outs = [], []
    for call in (one, two):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(call())
        graphs.append(gr)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        with torch.cuda.stream(s1):
            graphs[0].replay()
        with torch.cuda.stream(s2):
            graphs[1].replay()
    torch.cuda.synchronize()
    assert _same(e1, outs[0]) and _same(e2, outs[1])


@pytest.mark.parametrize("name", NAMES)
def test_two_streams_at_once(efla, name):
    """Calls run on the current stream: after work queued there, and beside another stream's."""
    one, two = _calls(efla, 0)[name], _calls(efla, 1)[name]
    e1, e2 = _copy(one()), _copy(two())
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(4):
        with torch.cuda.stream(s1):
            a = one()
        with torch.cuda.stream(s2):
            b = two()
    torch.cuda.synchronize()
    assert _same(e1, a) and _same(e2, b)
    assert efla.last_error() == 0
