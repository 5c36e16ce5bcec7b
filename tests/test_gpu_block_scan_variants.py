"""Every way in which the scan is cut - channels and state values of a lane,
widths of access, segments - against float64, within the error bound that the
recurrence itself carries (``scan_bound``)."""
import ctypes

import pytest
import torch

import block_ref as R
import scan_bound as S

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32
GRADS = ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dh0")


@pytest.fixture(scope="module")
def efla():
    import delta_rule_linear_03_b200 as m
    return m


def _plan(efla, B, L, C, G, N, backward):
    p = (ctypes.c_int * 5)()
    assert efla._lib.efla_diag_scan_plan(B, L, C, G, N, backward, p) == 0
    return list(p)


def _check(efla, s, seed=9):
    B, L, C = s["x"].shape
    G, N = s["Bm"].shape[2:]
    g = torch.Generator().manual_seed(seed)
    dy, dh = torch.randn(B, L, C, generator=g).to(s["x"].dtype), torch.randn(B, C, N, generator=g)
    fwd, bwd = _plan(efla, B, L, C, G, N, 0), _plan(efla, B, L, C, G, N, 1)
    size = lambda p: p[3] if p[2] > 1 else None  # noqa: E731
    bound = S.scan(**s, dy=dy, dh_L=dh, seg=size(fwd), seg_bwd=size(bwd), tiles=bwd[4])
    d = {k: None if t is None else t.cuda() for k, t in s.items()}
    got = dict(zip(("y", "h_L"), efla.scan_fwd(**d)))
    got.update(zip(GRADS, efla.scan_bwd(dy.cuda(), **d, dh_L=dh.cuda())))
    for k, v in got.items():
        S.close(v, *bound[k], k)


# batch, length, channels, state values, groups, and what a lane takes of them (state values, channels) forward and
# backward.  Widths are whole vectors of eight channels a group, of four, odd, and odd with a half-empty pair.
CASES = [(8, 20, 3584, 16, 1, (4, 2), (4, 1)), (8, 20, 3580, 16, 1, (4, 2), (4, 1)), (8, 19, 3521, 16, 1, (4, 2), (4, 1)), (4, 35, 7102, 16, 2, (4, 2), (4, 1)),
         (8, 20, 3584, 8, 1, (2, 2), (4, 1)), (8, 17, 3533, 8, 1, (2, 2), (4, 1)), (4, 40, 7112, 8, 2, (2, 2), (4, 1)),
         (8, 33, 1800, 32, 1, (4, 2), (4, 2)), (8, 20, 1795, 32, 1, (4, 2), (4, 2)), (4, 18, 3604, 32, 2, (4, 2), (4, 2)),
         (2, 40, 600, 64, 1, (4, 2), (4, 2)), (2, 35, 603, 64, 1, (4, 2), (4, 2)), (1, 30, 1212, 64, 2, (4, 2), (4, 2)), (3, 33, 406, 64, 2, (4, 2), (4, 2)),
         (8, 33, 704, 32, 1, (4, 1), (4, 1)), (8, 20, 701, 32, 1, (4, 1), (4, 1)), (4, 20, 2400, 8, 1, (4, 1), (4, 1)), (4, 33, 1289, 16, 1, (4, 1), (4, 1)),
         (2, 50, 300, 16, 1, (2, 1), (2, 1)), (2, 50, 301, 8, 1, (2, 1), (2, 1)), (2, 50, 304, 32, 1, (2, 1), (2, 1)), (2, 33, 100, 64, 1, (4, 1), (4, 1))]


@pytest.mark.parametrize("B,L,C,N,G,fwd,bwd", CASES)
@pytest.mark.parametrize("T,ragged", [(BF, True), (F, True), (F, False)])
def test_scan_variants(efla, B, L, C, N, G, fwd, bwd, T, ragged):
    for back, lane in ((0, fwd), (1, bwd)):
        plan = _plan(efla, B, L, C, G, N, back)
        assert tuple(plan[:2]) == lane and plan[2] == 1
    _check(efla, R.scan_inputs(B, L, C, N, G, T, lengths=[[L // 2, L, 0, L - 1, 1][b % 5] for b in range(B)] if ragged else None))


@pytest.mark.parametrize("B,L,C,N,G,lengths", [(1, 1030, 24, 32, 1, None), (2, 900, 40, 16, 2, [900, 333]), (1, 1500, 23, 8, 1, None), (2, 700, 24, 64, 1, [160, 700]),
                                               (1, 5000, 64, 32, 1, None)])
@pytest.mark.parametrize("T", [BF, F])
def test_scan_segments(efla, B, L, C, N, G, lengths, T):
    for back in (0, 1):
        assert _plan(efla, B, L, C, G, N, back)[2] > 1
    _check(efla, R.scan_inputs(B, L, C, N, G, T, lengths=lengths))


@pytest.mark.parametrize("B,L,C,N,G", [(1, 1, 1, 8, 1), (2, 2, 5, 16, 1), (1, 31, 32, 16, 1), (2, 32, 33, 8, 1), (1, 33, 70, 32, 2), (2, 65, 24, 64, 3),
                                       (3, 100, 96, 16, 4), (1, 17, 130, 64, 1), (2, 48, 200, 8, 2), (1, 257, 40, 32, 1), (3, 333, 200, 8, 2), (1, 2000, 300, 16, 1)])
@pytest.mark.parametrize("T", [BF, F])
def test_scan_sizes(efla, B, L, C, N, G, T):
    _check(efla, R.scan_inputs(B, L, C, N, G, T))


@pytest.mark.parametrize("off", [1, 3, 4])
@pytest.mark.parametrize("C,N", [(3584, 16), (600, 64)])
@pytest.mark.parametrize("T", [BF, F])
def test_scan_pairs_from_unaligned_rows(efla, off, C, N, T):
    """Two channels a lane, read as columns of wider projections in single channels or in fours."""
    B, L = (8, 19) if N == 16 else (2, 19)
    assert _plan(efla, B, L, C, 1, N, 0)[1] == 2
    s = R.scan_inputs(B, L, C, N, 1, T)
    for k in ("x", "dt", "z"):
        wide = torch.zeros(B, L, C + 8, dtype=T)
        wide[..., off:off + C] = s[k]
        s[k] = wide.cuda()[..., off:off + C]
    _check(efla, s)


@pytest.mark.parametrize("B,C,N,G", [(1, 1, 8, 1), (3, 33, 16, 3), (2, 200, 32, 1), (5, 72, 64, 2), (70, 2048, 16, 1)])
@pytest.mark.parametrize("T", [BF, F])
def test_scan_step_within_the_bound(efla, B, C, N, G, T):
    s = R.scan_inputs(B, 1, C, N, G, T)
    bound = S.scan(**s)
    h = s["h0"].cuda()
    one = {k: s[k][:, 0].cuda() for k in ("x", "dt", "Bm", "Cm", "z")}
    y = efla.scan_step(h=h, A=s["A"].cuda(), D=s["D"].cuda(), dt_bias=s["dt_bias"].cuda(), **one)
    value, err = bound["y"]
    S.close(y[:, None], value, err, "y")
    S.close(h, *bound["h_L"], "h")
