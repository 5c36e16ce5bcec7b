"""How large the scan's calls may be: what fits the kernels' grids and 32-bit
counts is taken, what does not is refused (fake addresses, no GPU)."""
import pytest

from test_block_abi import NULL, SHAPE, conv_bwd, conv_fwd, scan_bwd, scan_fwd, scan_step, so  # noqa: F401


@pytest.mark.parametrize("B,C,N", [(4096, 4096, 16), (1024, 4096, 64), (512, 8192, 64), (65535, 1024, 64)])
def test_large_batches_are_taken(so, B, C, N):  # noqa: F811
    """States of 1 to 17 GB; the missing x is the next thing that a call is refused for."""
    assert so.efla_scan_bwd_workspace_size(B, 1, C, 1, N) > 0
    kw = dict(B=B, C=C, N=N, G=1, ldx=C, lddt=C, ldz=C, ldb=N, ldc=N, x=None)
    assert scan_step(so, **kw) == NULL and scan_fwd(so, L=1, **kw) == NULL and scan_bwd(so, L=1, **kw) == NULL


def test_what_cannot_be_counted_is_refused(so):  # noqa: F811
    wide = dict(B=1, C=1 << 28, N=8, G=1, ldx=1 << 28, lddt=1 << 28, ldz=1 << 28, ldb=8, ldc=8)  # C N = 2^31
    groups = dict(B=1 << 19, C=4096, N=8, G=4096, ldx=4096, lddt=4096, ldz=4096, ldb=1 << 15, ldc=1 << 15)  # 2^31 blocks
    for kw in (wide, groups):
        assert scan_fwd(so, L=1, **kw) == SHAPE and scan_bwd(so, L=1, **kw) == SHAPE
        assert so.efla_scan_fwd_workspace_size(kw["B"], 1, kw["C"], kw["G"], 8) == 0 == so.efla_scan_bwd_workspace_size(kw["B"], 1, kw["C"], kw["G"], 8)
    assert scan_step(so, **wide) == SHAPE
    fewer = dict(groups, B=(1 << 19) - 16, x=None)
    assert scan_fwd(so, L=1, **fewer) == NULL


def test_batches_that_their_sums_cannot_count(so):  # noqa: F811
    """The sums over sequences go on by 32 rows past the last one, in 32 bits."""
    for B in (0x7fffffff, 0x7fff0001):
        assert conv_fwd(so, B=B, L=1, C=1, K=2, ldx=1, heads=0, x=None) == conv_bwd(so, B=B, L=1, C=1, K=2, ldx=1, x=None) == SHAPE
        one = dict(B=B, L=1, C=1, N=8, G=1, ldx=1, lddt=1, ldz=1, ldb=8, ldc=8, x=None)
        assert scan_fwd(so, **one) == scan_bwd(so, **one) == SHAPE
    assert conv_bwd(so, B=0x7fff0000, L=1, C=1, K=2, ldx=1, x=None) == NULL
    assert scan_bwd(so, **dict(one, B=0x7fff0000)) == NULL
