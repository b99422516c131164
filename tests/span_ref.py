"""Plain float64 attention of query rows over given key/value rows, and how far the kernels may be
from it.  Test infrastructure: elementary torch operations, nothing of the library."""
import torch


def attend64(q, k, v, scale):
    """q [H_q, d] over k, v [n, H_kv, d], all of them; zeros for n = 0."""
    H_q, d = q.shape
    n, H_kv, _ = k.shape
    if n == 0:
        return torch.zeros((H_q, d), dtype=torch.float64, device=q.device)
    kk = k.double().repeat_interleave(H_q // H_kv, 1)
    vv = v.double().repeat_interleave(H_q // H_kv, 1)
    x = torch.einsum("hd,nhd->hn", q.double(), kk) * scale
    w = torch.exp(x - x.amax(1, keepdim=True))
    return torch.einsum("hn,nhd->hd", w / w.sum(1, keepdim=True), vv)


def tolerance(q, ks, vs, scale, rows):
    """Bound of an output's error.

    A score is a sum of d products in fp32: off by at most (d + 2) 2^-23 sum|q k|, and as much of a
    weight (twice: numerator and denominator); sums over the rows in fp32, off by at most 2^-23 a
    row; for bf16 the weights are kept as two bf16 parts, 2^-8 * 2^-8 of a weight is lost.
    """
    big = max([float(v.abs().nan_to_num(0).max()) for v in vs if v.numel()] + [0.0])
    mag = max([float(k.float().nan_to_num(0).norm(dim=-1).max()) for k in ks if k.numel()] + [0.0])
    d = q.shape[-1]
    dots = float(q.float().norm(dim=-1).max()) * mag * abs(scale)
    cut = 2.0 ** -16 if q.dtype == torch.bfloat16 else 0.0
    return big * (cut + 2 * (d + 2) * 2.0 ** -23 * dots + 2 * rows * 2.0 ** -23 + 2.0 ** -20)


def normal(shape, gen, dtype, std=1.0):
    return (torch.randn(shape, generator=gen) * std).to(dtype)
