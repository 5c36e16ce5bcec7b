"""The short convolution and its gradients in float64 on the tensors' own
device, for sizes that take the token-by-token reference too long, with the
magnitudes that ``block_ref`` describes."""
import torch

from block_ref import HALF_STEP, U, dsilu


def close(got, ref, mag, ops, what):
    """``block_ref.close`` where the tensors are."""
    g = got.double()
    err = ops * U * mag
    tol = err + HALF_STEP[got.dtype] * (ref.abs() + err) + 2.0 ** -140
    assert bool(torch.isfinite(g).all()), f"{what}: not finite"
    over = (g - ref).abs() - tol
    assert float(over.max()) <= 0, (what, int((over > 0).sum()), over.numel(), float((g - ref).abs()[over > 0].max()), float(tol[over > 0].min()))


def inside(lengths, B, L, device):
    """[B, L, 1]: tokens that belong to their sequence."""
    n = torch.full((B,), L, device=device) if lengths is None else lengths.to(device).long()
    return (torch.arange(L, device=device) < n[:, None])[..., None], n


def conv(x, wt, bias, state, lengths, silu, dy, dstate_out):
    """{name: (value, magnitude)} of y, state_out, dx, dweight, dbias, dstate, and the largest |pre|."""
    B, L, C = x.shape
    K = wt.shape[1]
    on, n = inside(lengths, B, L, x.device)
    wt, bias = wt.double(), bias.double() if bias is not None else wt.new_zeros(C, dtype=torch.float64)
    front = state.double() if state is not None else torch.zeros(B, K - 1, C, dtype=torch.float64, device=x.device)
    xs = torch.cat([front, torch.where(on, x.double(), 0.0)], 1)
    pre, size = bias.expand(B, L, C).clone(), bias.abs().expand(B, L, C).clone()
    for j in range(K):
        term = xs[:, j:j + L] * wt[:, j]
        pre += term
        size += term.abs()
    y = torch.where(on, pre * torch.sigmoid(pre) if silu else pre, 0.0)
    rows = n[:, None] + torch.arange(K - 1, device=x.device)
    kept = torch.gather(xs, 1, rows[..., None].expand(-1, -1, C))
    out = dict(y=(y, 1.1 * torch.where(on, size, 0.0) + y.abs()), state_out=(kept, kept.abs()))
    dy = torch.where(on, dy.double(), 0.0)
    d = dy * dsilu(pre) if silu else dy
    dm = d.abs() + (dy.abs() * (1 + size) if silu else 0.0)  # silu' changes by at most 1/2 a unit of its argument
    dxs, dxm = torch.zeros_like(xs), torch.zeros_like(xs)
    dw, dwm = torch.zeros_like(wt), torch.zeros_like(wt)
    for j in range(K):
        dxs[:, j:j + L] += d * wt[:, j]
        dxm[:, j:j + L] += dm * wt[:, j].abs()
        dw[:, j] = (d * xs[:, j:j + L]).sum((0, 1))
        dwm[:, j] = (dm * xs[:, j:j + L].abs()).sum((0, 1))
    if dstate_out is not None:
        g = dstate_out.double()
        dxs.scatter_add_(1, rows[..., None].expand(-1, -1, C), g)
        dxm.scatter_add_(1, rows[..., None].expand(-1, -1, C), g.abs())
    out.update(dx=(dxs[:, K - 1:], dxm[:, K - 1:]), dstate=(dxs[:, :K - 1], dxm[:, :K - 1]), dweight=(dw, dwm), dbias=(d.sum((0, 1)), dm.sum((0, 1))))
    return out, float(pre.abs().max())
