"""The operators around the token mixer, as cases to be measured: the root-mean-square norm with the residual's
addition, the short causal convolution, and the selective state space scan, each with its backward pass and, for
the recurrent ones, its form for single tokens.

``run`` computes them from elementary torch operations, or, where ``own`` is true, with this library's calls.
"""
import math

import torch

own = False
EPS = 1e-6
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -126


def _lib():
    import delta_rule_linear_03_b200 as efla
    return efla


def listed():
    return [
        # one decode step of 64 sequences at the 1.3B-class width: residual added, 8-bit rows for the projections
        dict(name="norm_step_64x2048_fp8", op="norm_fwd", rows=64, C=2048, dtype="bf16", res="bf16", out8=True, group=128),
        # the same block on the long-context prompt of 65536 tokens
        dict(name="norm_prompt_65536x2048_fp8", op="norm_fwd", rows=65536, C=2048, dtype="bf16", res="bf16", out8=True, group=128),
        # the mixer's fp32 output normalised per head of 128, 340M-class layer at an odd length (8 x 8 heads x 2047 tokens)
        dict(name="norm_heads_131008x128_f32", op="norm_fwd", rows=131008, C=128, dtype="f32", res="none", out8=False, group=0),
        # training backward of the 1.3B-class layer's norm with the residual stream kept in fp32
        dict(name="norm_bwd_16384x2048", op="norm_bwd", rows=16384, C=2048, dtype="bf16", res="f32"),
        # one decode step of 64 sequences
        dict(name="conv_step_64x2048", op="conv_step", B=64, C=2048, K=4, dtype="bf16", bias=True, silu=True),
        # the 1.3B-class layer's prompt: q, k or v before the mixer, written per head as the mixer reads it
        dict(name="conv_prompt_4x4096x2048", op="conv_fwd", B=4, L=4096, C=2048, K=4, dtype="bf16", bias=True, silu=True, heads=16, state=True, ragged=False),
        # training backward of a padded batch, fp32, odd length and width, no vector width divides the row
        dict(name="conv_bwd_8x2047x1001_f32", op="conv_bwd", B=8, L=2047, C=1001, K=3, dtype="f32", bias=True, silu=True, heads=0, state=False, ragged=True),
        # one decode step of 64 sequences, twice the model width as such layers have it
        dict(name="scan_step_64x4096x16", op="scan_step", B=64, C=4096, N=16, G=1, dtype="bf16", z=True),
        # a small padded fp32 batch in two groups, continued from a state
        dict(name="scan_ragged_3x333x200x8_f32", op="scan_fwd", B=3, L=333, C=200, N=8, G=2, dtype="f32", z=True, h0=True, ragged=True),
        # the 1.3B-class layer's training forward
        dict(name="scan_fwd_4x4096x2048x16", op="scan_fwd", B=4, L=4096, C=2048, N=16, G=1, dtype="bf16", z=True, h0=False, ragged=False),
        # the long-context prompt: one sequence, so that only channels and time are left to work on
        dict(name="scan_prompt_1x65536x2048x16", op="scan_fwd", B=1, L=65536, C=2048, N=16, G=1, dtype="bf16", z=True, h0=True, ragged=False),
        # training backward at the 340M-class batch and length
        dict(name="scan_bwd_8x2048x1024x16", op="scan_bwd", B=8, L=2048, C=1024, N=16, G=1, dtype="bf16", z=True, h0=True, ragged=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def _width(rng, lo, hi):
    """A width: a multiple of 128, of 8, or any number."""
    c = _log(rng, lo, hi)
    m = rng.choice([128, 128, 8, 1])
    return max(1, c // m * m) if c >= m else c


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "conv_fwd", "conv_bwd", "conv_step", "scan_fwd", "scan_fwd", "scan_bwd", "scan_step"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("norm_fwd", "norm_bwd"):
        C = _width(rng, 32, 8192)
        rows = _log(rng, 1, min(65536, (1 << 26) // C))
        res = rng.choice(["none", "f32", dtype])
        if op == "norm_bwd":
            return dict(op=op, rows=rows, C=C, dtype=dtype, res=res)
        return dict(op=op, rows=rows, C=C, dtype=dtype, res=res, out8=rng.random() < 0.5, group=rng.choice([0, 128]))
    if op in ("conv_fwd", "conv_bwd"):
        heads = rng.choice([0, 0, 4, 16])
        C = heads * rng.choice([32, 64, 128]) if heads else _width(rng, 32, 8192)
        B = _log(rng, 1, 32)
        L = _log(rng, 1, min(65536, max(1, (1 << 25) // (B * C))))
        return dict(op=op, B=B, L=L, C=C, K=rng.choice([2, 3, 4, 4]), dtype=dtype, bias=rng.random() < 0.7, silu=rng.random() < 0.8,
                    heads=heads, state=rng.random() < 0.5, ragged=rng.random() < 0.4)
    if op == "conv_step":
        return dict(op=op, B=_log(rng, 1, 256), C=_width(rng, 32, 8192), K=rng.choice([2, 3, 4, 4]), dtype=dtype, bias=rng.random() < 0.7, silu=rng.random() < 0.8)
    N = rng.choice([8, 16, 16, 32, 64])
    G = rng.choice([1, 1, 2, 4])
    C = max(1, _width(rng, 32, 8192) // G) * G
    if op == "scan_step":
        return dict(op=op, B=_log(rng, 1, max(1, min(256, (1 << 25) // (C * N)))), C=C, N=N, G=G, dtype=dtype, z=rng.random() < 0.7)
    B = _log(rng, 1, 8)
    L = _log(rng, 1, min(65536, max(1, (1 << (28 if op == "scan_fwd" else 27)) // (B * C * N))))
    return dict(op=op, B=B, L=L, C=C, N=N, G=G, dtype=dtype, z=rng.random() < 0.7, h0=rng.random() < 0.5, ragged=rng.random() < 0.4)


# ---------------------------------------------------------------------------------------------------- inputs

def _type(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T = _type(case["dtype"])

    def normal(*shape, std=1.0, mean=0.0, to=None):
        return torch.randn(shape, generator=g, device="cuda").mul_(std).add_(mean).to(to or T)

    def uniform(lo, hi, *shape):
        return torch.rand(shape, generator=g, device="cuda").mul_(hi - lo).add_(lo)

    s = dict(case)
    op = case["op"]
    if op.startswith("norm"):
        rows, C = case["rows"], case["C"]
        s["w"] = uniform(0.5, 1.5, C)
        R = None if case["res"] == "none" else _type(case["res"])
        if op == "norm_fwd":
            s["x"] = normal(rows, C)
            s["r"] = None if R is None else normal(rows, C, std=2.0, to=R)
        else:
            s["dy"] = normal(rows, C)
            s["h"] = normal(rows, C, std=2.0, to=R or T)
            s["dr"] = None if R is None else normal(rows, C, to=R)
        return s
    if op.startswith("conv"):
        B, C, K = case["B"], case["C"], case["K"]
        s["w"] = uniform(-1 / math.sqrt(K), 1 / math.sqrt(K), C, K)
        s["bias"] = uniform(-0.5, 0.5, C) if case["bias"] else None
        if op == "conv_step":
            s["x"] = normal(B, C)
            s["state"] = normal(B, K - 1, C)
            return s
        L, H = case["L"], case["heads"]
        s["x"] = normal(B, L, C)
        s["state"] = normal(B, K - 1, C) if case["state"] else None
        s["lengths"] = torch.randint(0, L + 1, (B,), generator=g, device="cuda", dtype=torch.int32) if case["ragged"] else None
        if op == "conv_bwd":
            s["dy"] = normal(B, H, L, C // H) if H else normal(B, L, C)
            s["dstate"] = normal(B, K - 1, C) if case["state"] else None
        return s
    B, C, N, G = case["B"], case["C"], case["N"], case["G"]
    # decay rates 1..N with a spread, steps between 1e-3 and 1e-1: what such layers start from and stay near
    s["A"] = -torch.arange(1, N + 1, device="cuda", dtype=torch.float32) * torch.exp(uniform(-0.2, 0.2, C, N))
    step = torch.exp(uniform(math.log(1e-3), math.log(1e-1), C))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    s["D"] = uniform(0.5, 1.5, C)
    if op == "scan_step":
        s["x"], s["dt"] = normal(B, C), normal(B, C, std=0.5)
        s["Bm"], s["Cm"] = normal(B, G, N), normal(B, G, N)
        s["zz"] = normal(B, C) if case["z"] else None
        s["h"] = normal(B, C, N, std=0.3, to=torch.float32)
        return s
    L = case["L"]
    s["x"], s["dt"] = normal(B, L, C), normal(B, L, C, std=0.5)
    s["Bm"], s["Cm"] = normal(B, L, G, N), normal(B, L, G, N)
    s["zz"] = normal(B, L, C) if case["z"] else None
    s["h0_"] = normal(B, C, N, std=0.3, to=torch.float32) if case["h0"] else None
    s["lengths"] = torch.randint(0, L + 1, (B,), generator=g, device="cuda", dtype=torch.int32) if case["ragged"] else None
    if op == "scan_bwd":
        s["dy"] = normal(B, L, C)
        s["dh_L"] = normal(B, C, N, to=torch.float32) if case["h0"] else None
    return s


# ------------------------------------------------------------------------------------------------- plain forms

def _plain_norm_fwd(s):
    wide = torch.float64 if s["out8"] else torch.float32  # 8-bit values next to a border
    h = s["x"].to(wide) if s["r"] is None else s["x"].to(wide) + s["r"].to(wide)
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["w"].to(wide)
    out = {} if s["r"] is None else {"res_out": h.to(s["r"].dtype)}
    if not s["out8"]:
        return dict(out, y=y.to(s["x"].dtype))
    rows, C = y.shape
    g = s["group"] or C
    n = -(-C // g)
    full = torch.nn.functional.pad(y, (0, n * g - C)).view(rows, n, g)
    scale = (full.abs().amax(-1) / E4M3_MAX).clamp_min(SCALE_MIN).float()
    y8 = (full / scale.to(wide)[..., None]).view(rows, n * g)[:, :C]
    return dict(out, y8=y8.clamp(-E4M3_MAX, E4M3_MAX).float().to(torch.float8_e4m3fn), scale=scale)


def _plain_norm_bwd(s):
    h, dy = s["h"].float(), s["dy"].float()
    rstd = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    u = dy * s["w"]
    dh = rstd * (u - h * (rstd * rstd * (u * h).mean(-1, keepdim=True)))
    if s["dr"] is not None:
        dh = dh + s["dr"].float()
    out = dict(dx=dh.to(s["dy"].dtype), dweight=(dy * h * rstd).double().sum(0).float())
    return dict(out, dres=dh.to(s["h"].dtype)) if s["h"].dtype != s["dy"].dtype else out


def _silu(v):
    return v * torch.sigmoid(v)


def _dsilu(v):
    q = torch.sigmoid(v)
    return q * (1 + v * (1 - q))


def _inside(lengths, L):
    """[B, L, 1] truth values: the tokens that belong to their sequence."""
    t = torch.arange(L, device="cuda")
    return (t[None, :] < (lengths[:, None] if lengths is not None else L))[..., None]


def _heads_last(v, H):
    """[B, H, L, d] -> [B, L, H d]."""
    return v.transpose(1, 2).flatten(2) if H else v


def _window(s):
    """The inputs with the state in front, [B, K-1+L, C]."""
    x = s["x"].float()
    B, L, C = x.shape
    if s["lengths"] is not None:
        x = torch.where(_inside(s["lengths"], L), x, 0.0)
    front = s["state"].float() if s["state"] is not None else x.new_zeros(B, s["K"] - 1, C)
    return torch.cat([front, x], 1)


def _conv(s, xs, L):
    pre = (xs.unfold(1, s["K"], 1) * s["w"]).sum(-1)
    return pre if s["bias"] is None else pre + s["bias"]


def _plain_conv_fwd(s):
    B, L, C = s["x"].shape
    xs = _window(s)
    y = _conv(s, xs, L)
    y = _silu(y) if s["silu"] else y
    if s["lengths"] is not None:
        y = torch.where(_inside(s["lengths"], L), y, 0.0)
    n = s["lengths"].long() if s["lengths"] is not None else torch.full((B,), L, device="cuda")
    at = n[:, None] + torch.arange(s["K"] - 1, device="cuda")
    state = torch.gather(xs, 1, at[..., None].expand(-1, -1, C))
    y = y.to(s["x"].dtype)
    if s["heads"]:
        y = y.view(B, L, s["heads"], -1).transpose(1, 2).contiguous()
    return dict(y=y, state_out=state.to(s["x"].dtype))


def _plain_conv_bwd(s):
    B, L, C = s["x"].shape
    K = s["K"]
    xs = _window(s)
    d = _heads_last(s["dy"], s["heads"]).float()
    if s["silu"]:
        d = d * _dsilu(_conv(s, xs, L))
    if s["lengths"] is not None:
        d = torch.where(_inside(s["lengths"], L), d, 0.0)
    pad = torch.nn.functional.pad(d, (0, 0, K - 1, K - 1))
    dxs = (pad.unfold(1, K, 1) * s["w"].flip(1)).sum(-1)  # [B, K-1+L, C]
    if s["dstate"] is not None:
        n = s["lengths"].long() if s["lengths"] is not None else torch.full((B,), L, device="cuda")
        at = n[:, None] + torch.arange(K - 1, device="cuda")
        dxs = dxs.scatter_add(1, at[..., None].expand(-1, -1, C), s["dstate"].float())
    dw = (xs.unfold(1, K, 1) * d[..., None]).sum((0, 1), dtype=torch.float64).float()
    out = dict(dx=dxs[:, K - 1:].to(s["x"].dtype), dweight=dw)
    if s["bias"] is not None:
        out["dbias"] = d.sum((0, 1), dtype=torch.float64).float()
    if s["state"] is not None:
        out["dstate"] = dxs[:, :K - 1].to(s["x"].dtype)
    return out


def _plain_conv_step(s):
    xs = torch.cat([s["state"], s["x"][:, None]], 1)
    pre = (xs.float() * s["w"].t()).sum(1)
    pre = pre if s["bias"] is None else pre + s["bias"]
    s["state"].copy_(xs[:, 1:])
    return dict(y=(_silu(pre) if s["silu"] else pre).to(s["x"].dtype), state=s["state"])


def _recur(a, b):
    """h_t = a_t h_{t-1} + b_t along dimension 1, by doubling."""
    step, L = 1, a.shape[1]
    while step < L:
        b = torch.cat([b[:, :step], torch.addcmul(b[:, step:], a[:, step:], b[:, :-step])], 1)
        a = torch.cat([a[:, :step], a[:, step:] * a[:, :-step]], 1) if 2 * step < L else a
        step *= 2
    return b


def _per_channel(v, C):
    """[B, L, G, N] -> [B, L, C, N] without a copy where G is 1."""
    B, L, G, N = v.shape
    return v.float().unsqueeze(3).expand(B, L, G, C // G, N).reshape(B, L, C, N) if G > 1 else v.float()


def _scan_terms(s):
    x = s["x"].float()
    B, L, C = x.shape
    raw = s["dt"].float() + s["dt_bias"]
    step = torch.where(raw > 0, raw, 0.0) + torch.log1p(torch.exp(-raw.abs()))
    if s["lengths"] is not None:  # a step of zero leaves the state as it is
        step = torch.where(_inside(s["lengths"], L), step, 0.0)
        x = torch.where(_inside(s["lengths"], L), x, 0.0)
    a = torch.exp(step[..., None] * s["A"])
    b = (step * x)[..., None] * _per_channel(s["Bm"], C)
    if s["h0_"] is not None:
        b[:, 0] += a[:, 0] * s["h0_"]
    return x, raw, step, a, _recur(a, b)


def _plain_scan_fwd(s):
    B, L, C = s["x"].shape
    x, _, _, a, h = _scan_terms(s)
    del a
    y = (h * _per_channel(s["Cm"], C)).sum(-1) + s["D"] * x
    if s["zz"] is not None:
        y = y * _silu(s["zz"].float())
    if s["lengths"] is not None:
        y = torch.where(_inside(s["lengths"], L), y, 0.0)
    return dict(y=y.to(s["x"].dtype), h_L=h[:, -1].clone())


def _over_group(v, G, dtype):
    """[B, L, C, N] -> [B, L, G, N], summed over each group's channels."""
    B, L, C, N = v.shape
    return v.view(B, L, G, C // G, N).sum(3).to(dtype)


def _plain_scan_bwd(s):
    B, L, C = s["x"].shape
    G, T = s["G"], s["x"].dtype
    x, raw, step, a, h = _scan_terms(s)
    dy = s["dy"].float()
    if s["lengths"] is not None:
        dy = torch.where(_inside(s["lengths"], L), dy, 0.0)
    out = {}
    gy = dy
    if s["zz"] is not None:
        z = s["zz"].float()
        if s["lengths"] is not None:
            z = torch.where(_inside(s["lengths"], L), z, 0.0)
        out["dz"] = (dy * _dsilu(z) * ((h * _per_channel(s["Cm"], C)).sum(-1) + s["D"] * x)).to(T)
        gy = dy * _silu(z)
    out["dC"] = _over_group(gy[..., None] * h, G, T)
    # adjoint of the states, run from the end; the decay that takes step t to t + 1
    dh = gy[..., None] * _per_channel(s["Cm"], C)
    if s["dh_L"] is not None:
        dh[:, -1] += s["dh_L"]
    after = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    dh = _recur(after.flip(1), dh.flip(1)).flip(1)
    del after
    before = torch.cat([(s["h0_"] if s["h0_"] is not None else torch.zeros_like(h[:, 0]))[:, None], h[:, :-1]], 1)
    decayed = dh * a * before
    dhB = (dh * _per_channel(s["Bm"], C)).sum(-1)
    out["dx"] = (step * dhB + s["D"] * gy).to(T)
    dstep = (decayed * s["A"]).sum(-1) + x * dhB
    draw_ = dstep * torch.sigmoid(raw)
    if s["lengths"] is not None:
        draw_ = torch.where(_inside(s["lengths"], L), draw_, 0.0)
    out["ddt"] = draw_.to(T)
    out["ddt_bias"] = draw_.sum((0, 1), dtype=torch.float64).float()
    out["dA"] = (decayed * step[..., None]).sum(1).sum(0)
    out["dB"] = _over_group((step * x)[..., None] * dh, G, T)
    out["dD"] = (gy * x).sum((0, 1), dtype=torch.float64).float()
    out["dh0"] = a[:, 0] * dh[:, 0]
    return out


def _plain_scan_step(s):
    raw = s["dt"].float() + s["dt_bias"]
    step = torch.where(raw > 0, raw, 0.0) + torch.log1p(torch.exp(-raw.abs()))
    x, C = s["x"].float(), s["x"].shape[1]
    Bm, Cm = _per_channel(s["Bm"][:, None], C)[:, 0], _per_channel(s["Cm"][:, None], C)[:, 0]
    s["h"].mul_(torch.exp(step[..., None] * s["A"])).add_((step * x)[..., None] * Bm)
    y = (s["h"] * Cm).sum(-1) + s["D"] * x
    return dict(y=(y if s["zz"] is None else y * _silu(s["zz"].float())).to(s["x"].dtype), h=s["h"])


# -------------------------------------------------------------------------------------------- the library's calls

def _own_norm_fwd(s):
    y, scale, res_out = _lib().norm_fwd(s["x"], s["w"], s["r"], eps=EPS, out8=s["out8"], group=s["group"])
    out = {} if res_out is None else {"res_out": res_out}
    return dict(out, y8=y, scale=scale) if s["out8"] else dict(out, y=y)


def _own_norm_bwd(s):
    dx, dres, dw = _lib().norm_bwd(s["dy"], s["h"], s["w"], s["dr"], eps=EPS)
    out = dict(dx=dx, dweight=dw)
    return dict(out, dres=dres) if s["h"].dtype != s["dy"].dtype else out


def _own_conv_fwd(s):
    y, state = _lib().conv_fwd(s["x"], s["w"], s["bias"], state=s["state"], lengths=s["lengths"], silu=s["silu"], heads=s["heads"], want_state=True)
    return dict(y=y, state_out=state)


def _own_conv_bwd(s):
    dx, dw, db, dstate = _lib().conv_bwd(s["dy"], s["x"], s["w"], s["bias"], state=s["state"], lengths=s["lengths"], silu=s["silu"], heads=s["heads"],
                                         dstate_out=s["dstate"])
    out = dict(dx=dx, dweight=dw)
    if s["bias"] is not None:
        out["dbias"] = db
    if s["state"] is not None:
        out["dstate"] = dstate
    return out


def _own_conv_step(s):
    return dict(y=_lib().conv_step(s["x"], s["state"], s["w"], s["bias"], silu=s["silu"]), state=s["state"])


def _own_scan_fwd(s):
    y, h = _lib().scan_fwd(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], D=s["D"], z=s["zz"], dt_bias=s["dt_bias"], h0=s["h0_"], lengths=s["lengths"])
    return dict(y=y, h_L=h)


def _own_scan_bwd(s):
    g = _lib().scan_bwd(s["dy"], s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], D=s["D"], z=s["zz"], dt_bias=s["dt_bias"], h0=s["h0_"], lengths=s["lengths"],
                        dh_L=s["dh_L"])
    names = ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dh0")
    return {k: v for k, v in zip(names, g) if v is not None}


def _own_scan_step(s):
    return dict(y=_lib().scan_step(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["h"], D=s["D"], z=s["zz"], dt_bias=s["dt_bias"]), h=s["h"])


PLAIN = dict(norm_fwd=_plain_norm_fwd, norm_bwd=_plain_norm_bwd, conv_fwd=_plain_conv_fwd, conv_bwd=_plain_conv_bwd, conv_step=_plain_conv_step,
             scan_fwd=_plain_scan_fwd, scan_bwd=_plain_scan_bwd, scan_step=_plain_scan_step)
OWN = dict(norm_fwd=_own_norm_fwd, norm_bwd=_own_norm_bwd, conv_fwd=_own_conv_fwd, conv_bwd=_own_conv_bwd, conv_step=_own_conv_step,
           scan_fwd=_own_scan_fwd, scan_bwd=_own_scan_bwd, scan_step=_own_scan_step)


def run(state):
    return (OWN if own else PLAIN)[state["op"]](state)


# ------------------------------------------------------------------------------------------------------ work

def work(case):
    op, e = case["op"], 4 if case["dtype"] == "f32" else 2
    if op.startswith("norm"):
        n, C = case["rows"] * case["C"], case["C"]
        r = {"none": 0, "f32": 4, "bf16": 2}[case["res"]]
        if op == "norm_fwd":
            groups = case["rows"] * -(-C // (case["group"] or C))
            return {"bytes": n * (e + 2 * r + (1 if case["out8"] else e)) + (4 * groups if case["out8"] else 0) + 4 * C, "flops": 6 * n}
        h = r or e
        return {"bytes": n * (e + h + r + e + (h if h != e else 0)) + 8 * C, "flops": 12 * n}
    if op.startswith("conv"):
        K, C = case["K"], case["C"]
        small = 4 * C * (K + 1)
        if op == "conv_step":
            return {"bytes": case["B"] * C * e * (2 + 2 * (K - 1)) + small, "flops": case["B"] * C * (2 * K + 4)}
        n = case["B"] * case["L"] * C
        states = case["B"] * (K - 1) * C * e * (2 if case["state"] else 1)
        if op == "conv_fwd":
            return {"bytes": 2 * n * e + states + small, "flops": n * (2 * K + 4)}
        return {"bytes": 3 * n * e + states + 2 * small, "flops": n * (6 * K + 10)}
    B, C, N, G = case["B"], case["C"], case["N"], case["G"]
    params = 4 * C * (N + 2)
    if op == "scan_step":
        return {"bytes": B * C * (8 * N + e * (4 if case["z"] else 3)) + 2 * B * G * N * e + params, "flops": B * C * (7 * N + 10)}
    n = B * case["L"]
    if op == "scan_fwd":
        return {"bytes": n * (C * e * (4 if case["z"] else 3) + 2 * G * N * e) + 4 * B * C * N * (2 if case["h0"] else 1) + params, "flops": n * C * (7 * N + 10)}
    return {"bytes": n * (C * e * (7 if case["z"] else 5) + 4 * G * N * e) + 4 * B * C * N * (3 if case["h0"] else 1) + 2 * params, "flops": n * C * (20 * N + 30)}


# --------------------------------------------------------------------------------- the definition in 64 bits

def _wide(v):
    return None if v is None else v.double()


def exact(case, seed):
    if case["op"] == "scan_bwd" and case["L"] > 20000:  # some 40 operations a token
        return None
    s = prepare(case, seed)
    with torch.no_grad():
        return globals()["_exact_" + case["op"]](s)


def _exact_norm_fwd(s):
    h = _wide(s["x"])
    out = {}
    if s["r"] is not None:
        h = h + _wide(s["r"])
        out["res_out"] = h
    y = h / torch.sqrt(h.pow(2).sum(1, keepdim=True) / s["C"] + EPS) * _wide(s["w"])
    if not s["out8"]:
        return dict(out, y=y)
    g = s["group"] or s["C"]
    cols = torch.arange(s["C"], device="cuda") // g
    n = int(cols[-1]) + 1
    top = y.new_zeros(y.shape[0], n).scatter_reduce(1, cols.expand_as(y), y.abs(), "amax")
    scale = torch.maximum(top / E4M3_MAX, torch.tensor(SCALE_MIN, device="cuda", dtype=torch.float64))
    return dict(out, y8=y / scale[:, cols], scale=scale)


def _exact_norm_bwd(s):
    dy, h, w = _wide(s["dy"]), _wide(s["h"]), _wide(s["w"])
    ms = h.pow(2).sum(1, keepdim=True) / s["C"] + EPS
    dh = dy * w / ms.sqrt() - h * (dy * w * h).sum(1, keepdim=True) / (s["C"] * ms * ms.sqrt())
    if s["dr"] is not None:
        dh = dh + _wide(s["dr"])
    out = dict(dx=dh, dweight=(dy * h / ms.sqrt()).sum(0))
    return dict(out, dres=dh) if s["h"].dtype != s["dy"].dtype else out


def _exact_conv(s):
    """Inputs with the state in front, one row at a time cut to its length, and the pre-activation."""
    x = _wide(s["x"]).clone()
    B, L, C = x.shape
    n = [L] * B if s["lengths"] is None else s["lengths"].tolist()
    for b in range(B):
        x[b, n[b]:] = 0
    front = _wide(s["state"]) if s["state"] is not None else x.new_zeros(B, s["K"] - 1, C)
    xs = torch.cat([front, x], 1)
    w = _wide(s["w"])
    pre = x.new_zeros(B, L, C)
    for j in range(s["K"]):
        pre += xs[:, j:j + L] * w[:, j]
    if s["bias"] is not None:
        pre += _wide(s["bias"])
    return xs, pre, n


def _exact_conv_fwd(s):
    xs, pre, n = _exact_conv(s)
    B, L, C = pre.shape
    y = pre / (1 + torch.exp(-pre)) if s["silu"] else pre
    for b in range(B):
        y[b, n[b]:] = 0
    state = torch.stack([xs[b, n[b]:n[b] + s["K"] - 1] for b in range(B)])
    H = s["heads"]
    return dict(y=y.view(B, L, H, C // H).permute(0, 2, 1, 3) if H else y, state_out=state)


def _exact_conv_bwd(s):
    xs, pre, n = _exact_conv(s)
    B, L, C = pre.shape
    K, w = s["K"], _wide(s["w"])
    d = _wide(s["dy"])
    d = d.permute(0, 2, 1, 3).reshape(B, L, C) if s["heads"] else d.clone()
    if s["silu"]:
        q = 1 / (1 + torch.exp(-pre))
        d = d * (q + pre * q * (1 - q))
    for b in range(B):
        d[b, n[b]:] = 0
    dxs, dw = torch.zeros_like(xs), torch.zeros_like(w)
    for j in range(K):
        dxs[:, j:j + L] += d * w[:, j]
        dw[:, j] = (d * xs[:, j:j + L]).sum((0, 1))
    if s["dstate"] is not None:
        for b in range(B):
            dxs[b, n[b]:n[b] + K - 1] += _wide(s["dstate"][b])
    out = dict(dx=dxs[:, K - 1:], dweight=dw)
    if s["bias"] is not None:
        out["dbias"] = d.sum((0, 1))
    if s["state"] is not None:
        out["dstate"] = dxs[:, :K - 1]
    return out


def _exact_conv_step(s):
    K, w = s["K"], _wide(s["w"])
    xs = [_wide(s["state"][:, j]) for j in range(K - 1)] + [_wide(s["x"])]
    pre = sum(xs[j] * w[:, j] for j in range(K))
    if s["bias"] is not None:
        pre = pre + _wide(s["bias"])
    return dict(y=pre / (1 + torch.exp(-pre)) if s["silu"] else pre, state=torch.stack(xs[1:], 1))


def _exact_scan_at(s, t, to_c):
    """Step t of the scan for all rows: its step sizes, inputs and, per channel, Bm and Cm."""
    raw = _wide(s["dt"][:, t]) + _wide(s["dt_bias"])
    step = torch.logaddexp(raw, torch.zeros_like(raw))
    return raw, step, _wide(s["x"][:, t]), _wide(s["Bm"][:, t])[:, to_c], _wide(s["Cm"][:, t])[:, to_c]


def _exact_scan_fwd(s, keep=None):
    B, L, C = s["x"].shape
    A, D = _wide(s["A"]), _wide(s["D"])
    to_c = torch.arange(C, device="cuda") // (C // s["G"])
    h = _wide(s["h0_"]) if s["h0_"] is not None else A.new_zeros(B, C, s["N"])
    y = A.new_zeros(B, L, C)
    n = None if s["lengths"] is None else s["lengths"].long()
    for t in range(L):
        raw, step, x, Bt, Ct = _exact_scan_at(s, t, to_c)
        new = torch.exp(step[..., None] * A).mul_(h).addcmul_((step * x)[..., None], Bt)
        on = None if n is None else (t < n)[:, None]
        h = new if on is None else torch.where(on[..., None], new, h)
        if keep is not None:
            keep.append(h)
        v = torch.linalg.vecdot(h, Ct) + D * x
        y[:, t] = v if on is None else torch.where(on, v, 0.0)
    if s["zz"] is not None:
        z = _wide(s["zz"])
        y *= z / (1 + torch.exp(-z))
    return dict(y=y, h_L=h)


def _exact_scan_bwd(s):
    B, L, C = s["x"].shape
    G, N, A, D = s["G"], s["N"], _wide(s["A"]), _wide(s["D"])
    to_c = torch.arange(C, device="cuda") // (C // G)
    hs = []
    _exact_scan_fwd(dict(s, zz=None), keep=hs)
    zero = A.new_zeros(B, C, N)
    h0 = _wide(s["h0_"]) if s["h0_"] is not None else zero
    dh = _wide(s["dh_L"]).clone() if s["dh_L"] is not None else zero.clone()
    n = None if s["lengths"] is None else s["lengths"].long()
    out = {k: A.new_zeros(B, L, C) for k in ("dx", "ddt", "dz")}
    out["dB"], out["dC"] = A.new_zeros(B, L, G, N), A.new_zeros(B, L, G, N)
    dA, dD, db = torch.zeros_like(A), torch.zeros_like(D), torch.zeros_like(D)
    for t in reversed(range(L)):
        raw, step, x, Bt, Ct = _exact_scan_at(s, t, to_c)
        on = torch.ones(B, 1, dtype=torch.bool, device="cuda") if n is None else (t < n)[:, None]
        dy = torch.where(on, _wide(s["dy"][:, t]), 0.0)
        g = dy
        if s["zz"] is not None:
            z = _wide(s["zz"][:, t])
            q = 1 / (1 + torch.exp(-z))
            out["dz"][:, t] = torch.where(on, dy * ((hs[t] * Ct).sum(-1) + D * x) * (q + z * q * (1 - q)), 0.0)
            g = dy * z * q
        full = dh + Ct * g[..., None]
        before = hs[t - 1] if t else h0
        e = torch.exp(step[..., None] * A)
        eb = full * e * before
        dstep = (eb * A).sum(-1) + x * (full * Bt).sum(-1)
        dr = torch.where(on, dstep / (1 + torch.exp(-raw)), 0.0)
        out["dx"][:, t] = torch.where(on, step * (full * Bt).sum(-1) + D * g, 0.0)
        out["ddt"][:, t] = dr
        db += dr.sum(0)
        dA += torch.where(on[..., None], eb * step[..., None], 0.0).sum(0)
        dD += torch.where(on, g * x, 0.0).sum(0)
        out["dB"][:, t] = torch.where(on[..., None], full * (step * x)[..., None], 0.0).view(B, G, C // G, N).sum(2)
        out["dC"][:, t] = (hs[t] * g[..., None]).view(B, G, C // G, N).sum(2)
        dh = torch.where(on[..., None], full * e, dh)
    out.update(dA=dA, dD=dD, ddt_bias=db, dh0=dh)
    if s["zz"] is None:
        del out["dz"]
    return out


def _exact_scan_step(s):
    A, C = _wide(s["A"]), s["C"]
    to_c = torch.arange(C, device="cuda") // (C // s["G"])
    one = {k: s[k][:, None] for k in ("x", "dt", "Bm", "Cm")}
    _, step, x, Bt, Ct = _exact_scan_at(dict(s, **one), 0, to_c)
    h = torch.exp(step[..., None] * A) * _wide(s["h"]) + (step * x)[..., None] * Bt
    y = (h * Ct).sum(-1) + _wide(s["D"]) * x
    if s["zz"] is not None:
        z = _wide(s["zz"])
        y = y * z / (1 + torch.exp(-z))
    return dict(y=y, h=h)
