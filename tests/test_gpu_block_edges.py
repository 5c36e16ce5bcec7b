"""Values at the edges of the operators around the mixer, on the GPU."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def efla():
    import delta_rule_linear_03_b200 as m
    return m


@pytest.mark.parametrize("C", [100, 1001, 1003, 1024, 4101])
@pytest.mark.parametrize("T", [BF, F])
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("end", [0, -1])
def test_norm_infinite_weight_at_a_row_end(efla, C, T, group, end):
    """An infinite weight in the first or last column gives infinities there alone, and its group's scale is infinite and
    not NaN: the finite values are 0, the infinite one is inf / inf.  Vectors of odd rows reach past those columns."""
    g = torch.Generator().manual_seed(C)
    x = (0.5 + torch.rand(9, C, generator=g)).to(T).cuda()
    wt = torch.ones(C, device="cuda")
    y0, _, _ = efla.norm_fwd(x, wt)
    z0, s0, _ = efla.norm_fwd(x, wt, out8=True, group=group)
    wt[end] = float("inf")
    y, _, _ = efla.norm_fwd(x, wt)
    z, s, _ = efla.norm_fwd(x, wt, out8=True, group=group)
    at = torch.arange(C, device="cuda") == C + end if end else torch.arange(C, device="cuda") == 0
    assert torch.equal(y[:, ~at], y0[:, ~at]) and bool(torch.isposinf(y[:, at]).all())
    cols = torch.arange(C, device="cuda") // (group or C)
    hit = cols == cols[end]
    z, z0 = z.float(), z0.float()
    assert bool(torch.isposinf(s[:, int(cols[end])]).all())
    rest = torch.arange(s.shape[1], device="cuda") != cols[end]
    assert torch.equal(s[:, rest], s0[:, rest]) and torch.equal(z[:, ~hit], z0[:, ~hit])
    assert bool(torch.isnan(z[:, at]).all()) and not z[:, hit & ~at].any()


@pytest.mark.parametrize("eighth", range(8))
@pytest.mark.parametrize("step", [False, True])
def test_scan_decays_have_no_mean_error(efla, eighth, step):
    """The state of a thousand tokens multiplies a decay's mean error by a thousand.  The approximate 2^v is 0.6 to
    2.6 10^-8 too small on average for v from -1 to 0; centred, -1.2 to 0.9 10^-8 remain.  Means of 131072 decays, of
    spread 5 10^-8, are known to 1.4 10^-10: an eighth of the range each, 64 times the same decay."""
    C, N, L = 8192, 16, 64
    g = torch.Generator(device="cuda").manual_seed(eighth)
    v = -(eighth + torch.rand(C, N, device="cuda", generator=g, dtype=torch.float64)) / 8
    d = 0.6 + 0.8 * torch.rand(C, device="cuda", generator=g)
    A = (v * 0.6931471805599453 / d.double()[:, None]).float()
    dt, none, bc, h = d.expand(1, L, C).contiguous(), torch.zeros(1, L, C, device="cuda"), torch.zeros(1, L, 1, N, device="cuda"), torch.ones(1, C, N, device="cuda")
    if step:
        for t in range(L):
            efla.scan_step(none[:, t], dt[:, t], A, bc[:, t], bc[:, t], h, softplus=False)
    else:
        efla.scan_fwd(none, dt, A, bc, bc, h0=h, h_L=h, softplus=False)
    mean = float((h.double().log() / L - A.double() * d.double()[:, None]).mean())
    assert -1.3e-8 <= mean <= 1.0e-8
