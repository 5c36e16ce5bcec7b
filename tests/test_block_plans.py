"""How calls of the operators around the mixer are cut (no GPU: 148 SMs are
assumed), and the references of the tests at large sizes."""
import itertools

import pytest
import torch

import block_ref as R
import conv_wide


@pytest.fixture(scope="module")
def so():
    import delta_rule_linear_03_b200 as efla
    return efla._lib


def test_conv_run_goes_by_the_channels_of_a_thread(so):
    """Single channels take the runs that suit their blocks whatever the parity of the width: heads or rows may be odd
    where it is even."""
    run = so.efla_diag_conv_run
    for B, L, C in [(16, 1000, 2050), (8, 4096, 1002), (4, 2000, 1350), (2, 300, 1002)]:
        for lengths in (0, 1):
            assert run(B, L, C, 1, 1, lengths) in (run(B, L, C - 1, 1, 1, lengths), run(B, L, C + 1, 1, 1, lengths))
    assert run(16, 1000, 2050, 1, 1, 0) == 128 and run(16, 1000, 2050, 2, 1, 0) == 256
    assert run(0, 5, 5, 1, 1, 0) == run(1, 5, 5, 4, 1, 0) == run(1, 5, 5, 2, 0, 0) == run(1, -1, 5, 1, 1, 0) == 0
    for B, L, C, channels in itertools.product((1, 7, 300), (1, 22, 999, 70000), (1, 64, 999, 8192), (1, 2)):
        assert run(B, L, C, channels, 1, 0) in (8, 16, 32, 64, 128, 256) and run(B, L, C, channels, 1, 1) in (8, 16, 32, 64, 128)
        assert run(B, L, C, 1, 0, 0) in range(8, 129, 8) and run(B, L, C, 4, 0, 0) in range(8, 129, 8)


def test_conv_workspace_holds_every_run(so):
    for B, L, C, K in itertools.product((1, 5, 64), (1, 100, 4097), (1, 2, 130, 1001, 4096), (2, 4)):
        size = so.efla_conv_bwd_workspace_size(B, L, C, K)
        for channels, lengths in itertools.product((1, 2), (0, 1)):
            if C % channels == 0:
                tokens = 4 * so.efla_diag_conv_run(B, L, C, channels, 1, lengths)
                assert size >= B * -(-L // tokens) * C * (K + 1) * 4, (B, L, C, K, channels, lengths)


@pytest.mark.parametrize("K,lengths,silu,state", [(2, None, True, True), (4, [9, 0, 3], True, True), (3, [1, 9, 8], False, False)])
def test_conv_wide_is_the_reference(K, lengths, silu, state):
    g = torch.Generator().manual_seed(K)
    B, L, C = 3, 9, 5
    x, wt, b, st, dy, ds = (torch.randn(s, generator=g) for s in ((B, L, C), (C, K), (C,), (B, K - 1, C), (B, L, C), (B, K - 1, C)))
    if not state:
        st = None
    ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int32)
    got, _ = conv_wide.conv(x, wt, b, st, ln, silu, dy, ds)
    y, so_, pre, _ = R.conv_fwd(x, wt, b, st, ln, silu)
    want = dict(zip(("dx", "dweight", "dbias", "dstate"), R.conv_bwd(dy, x, wt, b, st, ln, silu, ds)), y=y, state_out=so_)
    for k, v in want.items():
        torch.testing.assert_close(got[k][0], v, rtol=1e-12, atol=1e-12)
    mags = R.conv_bwd(dy, x, wt, b, st, ln, silu, ds, mag=True)
    for k, v in zip(("dx", "dweight", "dbias", "dstate"), mags):
        torch.testing.assert_close(got[k][1], v, rtol=1e-12, atol=1e-12)
