"""efla_conv_fwd and efla_conv_bwd where a thread's run is long, as at real
sizes, against float64 on the GPU: batches without conditions inside a run,
sequences that end inside one, at its edge, and within K - 1 tokens of it.

Tolerances count rounded operations as in ``test_gpu_block_conv``; dweight and
dbias add a run's tokens in turn, four runs of a block, and then P blocks' rows
by 32s in turn and a tree of five levels: run + 4 + P / 32 + 6."""
import pytest
import torch

from conv_wide import close, conv

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def efla():
    import delta_rule_linear_03_b200 as m
    return m


def _lengths(B, L, r, K):
    """Ends at a run's edge, beside it, within K - 1 of it, inside it, nowhere, at once."""
    at = [L, 2 * r, 2 * r + 1, 3 * r - 1, r + K - 2, 3 * r + r // 2, 4 * r + K - 1, 0, 1, L - 1, 4 * r, L - K + 1, r - 1, 5 * r + 3, L // 2, r]
    return torch.tensor([min(max(at[b % len(at)], 0), L) for b in range(B)], dtype=torch.int32, device="cuda")


# batch, length, channels, heads, columns that x begins at in wider rows; channels of a thread; its run backward, without
# lengths and with, and forward
CASES = [(16, 1100, 32, 0, 0, 2, 16, 8, 8), (16, 600, 200, 2, 0, 2, 32, 16, 16), (8, 4100, 130, 0, 0, 2, 64, 64, 40), (16, 4100, 132, 11, 0, 2, 128, 128, 64),
         (4, 4096, 2048, 16, 0, 2, 256, 64, 120), (3, 70, 4096, 0, 3, 1, 32, 16, 8), (3, 130, 4095, 0, 0, 1, 64, 32, 16), (3, 260, 4095, 45, 0, 1, 32, 64, 24),
         (16, 1000, 2050, 82, 0, 1, 128, 128, 128), (3, 4100, 1000, 8, 0, 1, 256, 128, 88)]


@pytest.mark.parametrize("B,L,C,H,off,channels,whole_run,ragged_run,fwd_run", CASES)
@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("T", [BF, F])
@pytest.mark.parametrize("full", [True, False])
def test_conv_long_runs(efla, B, L, C, H, off, channels, whole_run, ragged_run, fwd_run, K, T, full):
    diag = efla._lib.efla_diag_conv_run
    wide = channels == 2 and (C // H if H else C) % 4 == 0
    run = whole_run if full else ragged_run
    assert diag(B, L, C, channels, 1, 0 if full else 1) == run and diag(B, L, C, 4 if wide else 1, 0, 0) == fwd_run
    g = torch.Generator(device="cuda").manual_seed(L + C + K)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x = r(B, L, C + off).to(T)[..., off:]
    wt, b, st, dst, dy = 0.5 * r(C, K), 0.5 * r(C), r(B, K - 1, C).to(T), r(B, K - 1, C).to(T), r(B, L, C).to(T)
    lengths = None if full else _lengths(B, L, run, K)
    if full:
        b = st = None
    ref, top = conv(x, wt, b, st, lengths, True, dy, dst)
    if not full:  # padding holds anything
        pad = torch.arange(L, device="cuda")[None, :, None] >= lengths[:, None, None]
        x.masked_fill_(pad, float("nan"))
        dy.masked_fill_(pad, float("inf"))
    ops = 32 + 2 * top
    split = lambda t: t.view(B, L, H, C // H).transpose(1, 2) if H else t  # noqa: E731
    y, so = efla.conv_fwd(x, wt, b, st, lengths, heads=H, want_state=True)
    close(y, split(ref["y"][0]), split(ref["y"][1]), ops, "y")
    assert torch.equal(so.double(), ref["state_out"][0])
    work = torch.empty(efla._lib.efla_conv_bwd_workspace_size(B, L, C, K), dtype=torch.uint8, device="cuda").fill_(255)
    dx, dw, db, ds = efla.conv_bwd(split(dy).contiguous(), x, wt, b, st, lengths, heads=H, dstate_out=dst, workspace=work)
    blocks = B * -(-L // (4 * run))
    adds = run + 4 + blocks / 32 + 6
    for name, got, more in (("dx", dx, 0), ("dweight", dw, adds), ("dbias", db, adds), ("dstate", ds, 0)):
        if got is None:
            assert full and name in ("dbias", "dstate")
        else:
            close(got, *ref[name], ops + more, name)
