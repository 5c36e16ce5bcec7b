"""Synchronous argument checks of the operators around the mixer: every bad
call is refused before anything is launched (fake addresses, no GPU)."""
import ctypes

import pytest

P = ctypes.c_void_p
NULL, SHAPE, DTYPE, ALIGN, UNSUPPORTED, WORKSPACE, ALIAS = 1, 2, 3, 4, 5, 8, 9
F32, BF16 = 0, 1


def at(i, off=0):
    return P((i + 1 << 32) + off)  # distinct, aligned, far apart


@pytest.fixture(scope="module")
def so():
    import delta_rule_linear_03_b200 as efla
    return efla._lib


def norm_fwd(so, **kw):
    a = dict(x=at(0), dt=BF16, res=at(1), rdt=BF16, w=at(2), eps=1e-6, y=at(3), y8=at(4), scale=at(5), group=128,
             res_out=at(6), rows=0, C=256)
    a.update(kw)
    return so.efla_norm_fwd(*a.values(), None)


def test_norm_fwd_refusals(so):
    assert norm_fwd(so) == 0 and norm_fwd(so, rows=5, C=0) == 0  # nothing to do
    go = dict(rows=4)
    for kw, status in [
            (dict(dt=7), DTYPE), (dict(rdt=2), DTYPE), (dict(dt=F32, rdt=BF16), UNSUPPORTED),
            (dict(rows=-1), SHAPE), (dict(C=-1), SHAPE), (dict(rows=1 << 40, C=16384), SHAPE), (dict(rows=1 << 31, C=1), SHAPE),
            (dict(C=16385), UNSUPPORTED), (dict(group=64), UNSUPPORTED),
            (dict(x=None), NULL), (dict(w=None), NULL), (dict(y=None, y8=None), NULL), (dict(scale=None), NULL), (dict(res=None), NULL),
            (dict(x=at(0, 2)), ALIGN), (dict(w=at(2, 4)), ALIGN), (dict(y8=at(4, 8)), ALIGN), (dict(scale=at(5, 4)), ALIGN),
            (dict(y=at(1)), ALIAS), (dict(y=at(0, 16)), ALIAS), (dict(y8=at(0)), ALIAS), (dict(scale=at(2)), ALIAS),
            (dict(res_out=at(1, 16)), ALIAS), (dict(res_out=at(3)), ALIAS), (dict(rdt=F32, res_out=at(0)), ALIAS),
            (dict(y=at(0), res_out=at(0)), ALIAS), (dict(res=at(0), res_out=at(0), y=at(3)), ALIAS)]:
        assert norm_fwd(so, **{**go, **kw}) == status, kw


def norm_bwd(so, **kw):
    a = dict(dy=at(0), dt=BF16, h=at(1), hdt=F32, w=at(2), eps=1e-6, dr=at(3), dx=at(4), dres=at(5), dw=at(6), rows=64,
             C=256, ws=at(7), n=1 << 30)
    a.update(kw)
    return so.efla_norm_bwd(*a.values(), None)


def test_norm_bwd_refusals(so):
    assert norm_bwd(so, C=0) == 0
    need = so.efla_norm_bwd_workspace_size(64, 256)  # a row of sums a block, at most two blocks an SM
    assert need == 64 * 256 * 4 and so.efla_norm_bwd_workspace_size(0, 256) == 0 == so.efla_norm_bwd_workspace_size(4, 16385)
    for kw, status in [
            (dict(dt=3), DTYPE), (dict(dt=F32, hdt=BF16), UNSUPPORTED), (dict(C=20000), UNSUPPORTED), (dict(rows=-2), SHAPE),
            (dict(dy=None), NULL), (dict(h=None), NULL), (dict(dw=None), NULL), (dict(dx=None, dres=None), NULL),
            (dict(dx=at(4, 2)), ALIGN), (dict(ws=at(7, 8)), ALIGN), (dict(ws=None), WORKSPACE), (dict(n=need - 1), WORKSPACE),
            (dict(dx=at(0)), ALIAS), (dict(dres=at(1)), ALIAS), (dict(dw=at(2)), ALIAS), (dict(dres=at(4)), ALIAS), (dict(ws=at(3)), ALIAS)]:
        assert norm_bwd(so, **kw) == status, kw


def conv_fwd(so, **kw):
    a = dict(x=at(0), ldx=256, dt=BF16, w=at(1), b=at(2), state=at(3), lengths=at(4), silu=1, y=at(5), heads=2, s_out=at(6),
             B=2, L=64, C=256, K=4)
    a.update(kw)
    return so.efla_conv_fwd(*a.values(), None)


def test_conv_fwd_refusals(so):
    assert conv_fwd(so, B=0) == 0 and conv_fwd(so, C=0, heads=0) == 0 and conv_fwd(so, L=0, s_out=None) == 0
    for kw, status in [
            (dict(dt=2), DTYPE), (dict(K=1), UNSUPPORTED), (dict(K=5), UNSUPPORTED), (dict(K=0), SHAPE), (dict(L=-1), SHAPE),
            (dict(heads=3), SHAPE), (dict(heads=-1), SHAPE), (dict(ldx=255), SHAPE), (dict(ldx=1 << 50), SHAPE),
            (dict(x=None), NULL), (dict(w=None), NULL), (dict(y=None), NULL),
            (dict(x=at(0, 1)), ALIGN), (dict(lengths=at(4, 2)), ALIGN), (dict(state=at(3, 2)), ALIGN), (dict(y=at(5, 8)), ALIGN),
            (dict(y=at(0)), ALIAS), (dict(y=at(3)), ALIAS), (dict(s_out=at(5)), ALIAS), (dict(s_out=at(3, 16)), ALIAS), (dict(s_out=at(4)), ALIAS)]:
        assert conv_fwd(so, **kw) == status, kw


def conv_bwd(so, **kw):
    a = dict(dy=at(0), x=at(1), ldx=256, dt=BF16, w=at(2), b=at(3), state=at(4), lengths=at(5), silu=1, heads=0, dso=at(6),
             dx=at(7), dw=at(8), db=at(9), ds=at(10), B=2, L=64, C=256, K=4, ws=at(11), n=1 << 30)
    a.update(kw)
    return so.efla_conv_bwd(*a.values(), None)


def test_conv_bwd_refusals(so):
    assert conv_bwd(so, C=0) == 0
    need = so.efla_conv_bwd_workspace_size(2, 64, 256, 4)
    assert need >= 2 * 256 * 5 * 4 and so.efla_conv_bwd_workspace_size(2, 64, 256, 5) == 0
    for kw, status in [
            (dict(dt=2), DTYPE), (dict(K=9), UNSUPPORTED), (dict(B=-1), SHAPE), (dict(dy=None), NULL), (dict(dx=None), NULL),
            (dict(dw=None), NULL), (dict(dy=at(0, 2)), ALIGN), (dict(db=at(9, 4)), ALIGN), (dict(ws=None), WORKSPACE),
            (dict(n=need - 1), WORKSPACE), (dict(dx=at(1)), ALIAS), (dict(ds=at(4)), ALIAS), (dict(ds=at(6)), ALIAS), (dict(ws=at(0)), ALIAS)]:
        assert conv_bwd(so, **kw) == status, kw


def conv_step(so, **kw):
    a = dict(x=at(0), ldx=256, dt=F32, state=at(1), w=at(2), b=at(3), silu=1, y=at(4), B=2, C=256, K=4)
    a.update(kw)
    return so.efla_conv_step(*a.values(), None)


def test_conv_step_refusals(so):
    assert conv_step(so, B=0) == 0
    for kw, status in [(dict(dt=4), DTYPE), (dict(K=1), UNSUPPORTED), (dict(ldx=8), SHAPE), (dict(state=None), NULL),
                       (dict(x=at(0, 2)), ALIGN), (dict(state=at(1, 4)), ALIGN), (dict(y=at(0)), ALIAS), (dict(state=at(0)), ALIAS)]:
        assert conv_step(so, **kw) == status, kw


def scan_fwd(so, **kw):
    a = dict(x=at(0), ldx=64, dt=at(1), lddt=64, A=at(2), Bm=at(3), ldb=32, Cm=at(4), ldc=32, D=at(5), z=at(6), ldz=64, bias=at(7),
             h0=at(8), lengths=at(9), dtype=BF16, softplus=1, y=at(10), hL=at(11), B=2, L=4096, C=64, G=2, N=16, ws=at(12), n=1 << 30)
    a.update(kw)
    return so.efla_scan_fwd(*a.values(), None)


SCAN_BAD = [
    (dict(dtype=2), DTYPE), (dict(N=12), UNSUPPORTED), (dict(N=128), UNSUPPORTED), (dict(N=0), SHAPE), (dict(G=3), SHAPE), (dict(G=0), SHAPE),
    (dict(B=-1), SHAPE), (dict(ldx=63), SHAPE), (dict(ldb=31), SHAPE), (dict(ldz=1), SHAPE), (dict(ldc=1 << 48), SHAPE),
    (dict(x=None), NULL), (dict(A=None), NULL), (dict(Bm=None), NULL),
    (dict(x=at(0, 1)), ALIGN), (dict(A=at(2, 4)), ALIGN), (dict(h0=at(8, 8)), ALIGN), (dict(lengths=at(9, 2)), ALIGN),
]


def test_scan_fwd_refusals(so):
    assert scan_fwd(so, B=0) == 0 and scan_fwd(so, C=0) == 0 and scan_fwd(so, L=0, hL=None) == 0
    assert scan_fwd(so, L=0, hL=at(8)) == 0  # in place: nothing to do
    need = so.efla_scan_fwd_workspace_size(2, 4096, 64, 2, 16)
    assert need > 0  # few channels, long: cut into segments
    for kw, status in SCAN_BAD + [(dict(y=None), NULL), (dict(ws=None), WORKSPACE), (dict(n=need - 1), WORKSPACE), (dict(y=at(0)), ALIAS),
                                  (dict(y=at(8)), ALIAS), (dict(hL=at(8, 16)), ALIAS), (dict(hL=at(10)), ALIAS), (dict(ws=at(6)), ALIAS)]:
        assert scan_fwd(so, **kw) == status, kw


def scan_bwd(so, **kw):
    a = dict(dy=at(20), x=at(0), ldx=64, dt=at(1), lddt=64, A=at(2), Bm=at(3), ldb=32, Cm=at(4), ldc=32, D=at(5), z=at(6), ldz=64,
             bias=at(7), h0=at(8), lengths=at(9), dhL=at(10), dtype=BF16, softplus=1, dx=at(11), ddt=at(12), dA=at(13), dB=at(14),
             dC=at(15), dD=at(16), dz=at(17), db=at(18), dh0=at(19), B=2, L=4096, C=64, G=2, N=16, ws=at(30), n=1 << 30)
    a.update(kw)
    return so.efla_scan_bwd(*a.values(), None)


def test_scan_bwd_refusals(so):
    assert scan_bwd(so, C=0) == 0
    need = so.efla_scan_bwd_workspace_size(2, 4096, 64, 2, 16)
    assert need > 0
    for kw, status in SCAN_BAD + [(dict(dy=None), NULL), (dict(dx=None), NULL), (dict(dA=None), NULL), (dict(dB=None), NULL), (dict(dz=None), NULL),
                                  (dict(dh0=at(19, 4)), ALIGN), (dict(ws=None), WORKSPACE), (dict(n=need - 1), WORKSPACE),
                                  (dict(dx=at(0)), ALIAS), (dict(dh0=at(10)), ALIAS), (dict(dB=at(15)), ALIAS), (dict(ws=at(20)), ALIAS)]:
        assert scan_bwd(so, **kw) == status, kw


def scan_step(so, **kw):
    a = dict(x=at(0), ldx=64, dt=at(1), lddt=64, A=at(2), Bm=at(3), ldb=32, Cm=at(4), ldc=32, D=at(5), z=at(6), ldz=64, bias=at(7),
             dtype=BF16, softplus=1, h=at(8), y=at(9), B=2, C=64, G=2, N=16)
    a.update(kw)
    return so.efla_scan_step(*a.values(), None)


def test_scan_step_refusals(so):
    assert scan_step(so, B=0) == 0
    for kw, status in [x for x in SCAN_BAD if not {"h0", "lengths"} & set(x[0])] + [
            (dict(B=65536), SHAPE), (dict(h=None), NULL), (dict(h=at(8, 4)), ALIGN), (dict(y=at(8)), ALIAS), (dict(h=at(2)), ALIAS)]:
        assert scan_step(so, **kw) == status, kw


def test_workspace_sizes_depend_on_the_arguments_alone(so):
    for fn in (so.efla_scan_fwd_workspace_size, so.efla_scan_bwd_workspace_size):
        assert fn(2, 4096, 64, 2, 16) == fn(2, 4096, 64, 2, 16)
        assert fn(0, 4096, 64, 2, 16) == fn(2, 0, 64, 2, 16) == fn(2, 4096, 64, 2, 12) == fn(2, 4096, 64, 3, 16) == 0
    # channels enough for every SM: one segment, no scratch for the forward pass
    assert so.efla_scan_fwd_workspace_size(8, 2048, 1024, 1, 16) == 0


def test_wrappers_refuse_host_tensors():
    import torch

    import delta_rule_linear_03_b200 as efla
    x = torch.zeros(2, 4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        efla.norm_fwd(x, torch.ones(8))
    with pytest.raises(ValueError, match="CUDA"):
        efla.conv_fwd(x, torch.ones(8, 4))
    with pytest.raises(ValueError, match="CUDA"):
        efla.scan_fwd(x, x, torch.ones(8, 8), torch.ones(2, 4, 1, 8), torch.ones(2, 4, 1, 8))


def test_lengths_that_tiles_cannot_count(so):
    """A sequence so long that the tokens of its last tile pass 32 bits is refused."""
    L = (1 << 31) - 1
    assert conv_fwd(so, L=L, B=1) == SHAPE and conv_bwd(so, L=L, B=1) == SHAPE
    assert scan_fwd(so, L=L, B=1) == SHAPE and scan_bwd(so, L=L, B=1) == SHAPE
    assert so.efla_conv_bwd_workspace_size(1, L, 8, 4) == 0 == so.efla_scan_bwd_workspace_size(1, L, 8, 1, 8)


def test_row_strides():
    """Tokens may lie apart evenly, a token's values may not."""
    import torch

    import delta_rule_linear_03_b200  # noqa: F401
    from delta_rule_linear_03_b200 import _efla_block

    def ld(t, lead, tail):
        assert tuple(t.shape) == lead + tail
        return _efla_block.token_stride(t, len(lead))

    wide = torch.zeros(3, 5, 40)
    assert ld(wide, (3, 5), (40,)) == 40 and ld(wide[..., 8:24], (3, 5), (16,)) == 40
    assert ld(wide[..., 8:24].unflatten(-1, (2, 8)), (3, 5), (2, 8)) == 40
    assert ld(wide[:1, :, 3:4], (1, 5), (1,)) == 40 and ld(wide[:, :1, :7], (3, 1), (7,)) == 200
    assert ld(wide[:1, :1, :7], (1, 1), (7,)) == 7
    for bad, tail in [(wide[:, :4, :16], (16,)), (wide[:, ::2, :16], (16,)), (wide[..., ::2], (20,)), (wide[:, :, :16].flip(1).transpose(0, 1), (16,)),
                      (torch.zeros(1, 1, 16).expand(3, 5, 16), (16,)), (torch.zeros(3, 1, 16).expand(3, 5, 16), (16,))]:
        with pytest.raises(ValueError):
            ld(bad, tuple(bad.shape[:2]), tail)
