"""How far an output row of the span kernels may be from float64, element by element, and how far all of
them together may lean towards zero.  Test infrastructure: elementary torch operations, nothing of the library.

With x_t the scores, p their softmax and out = sum_t p_t v_t, a kernel's weights are p_t (1 + e_t) with
|e_t| <= eps_t:
  scores       a sum of d products in float32: tensor cores add 16 at a time and round towards zero, at most
               2^-23 of the partial sum each, which sum_i |q_i k_i| bounds; d roundings of half that, of either
               sign, grow no faster on CUDA cores: |scale| (d/16 + 2) 2^-23 sum_i |q_i k_i|
  exponents    the scale and x - max are rounded once each: 2^-23 (|x| + |x - max|)
  exponentials ex2.approx is good to 2^-22, the weight's own and those of up to seven rescalings (maxima that
               rise, joins): 2^-19
  two parts    bf16 only, and not in the sum of weights: what the first bf16 part leaves is at most 2^-8 of the
               weight, what the second leaves of that 2^-8: 2^-16
The e_t of different rows are independent, so what they do to an element is a sum of n independent terms below
eps_t p_t |v_t|: at most 8 sqrt(sum (eps_t p_t v_t)^2) -- certainly when 64 rows or fewer share the weight, and
else 8 sqrt(3) = 13.8 standard deviations.  Likewise the sum of weights, which divides.  The additions: in a
tile 16 roundings towards zero of 2^-23 of sums whose size is sqrt(sum (p v)^2), and one rounding to nearest a
tile and a row outside.
"""
import torch

SIGMAS = 8.0


def attend_and_bound(q, k, v, scale, parts):
    """(out, bound) in float64 of q [R, d] over k, v [n, d]; ``parts``: the weights are kept as two bf16 parts."""
    q, k, v = q.double(), k.double(), v.double()
    n, d = k.shape
    x = q @ k.T * scale
    p = torch.softmax(x, -1)
    out = p @ v
    eps = abs(scale) * (d / 16 + 2) * 2.0 ** -23 * (q.abs() @ k.abs().T) + 2.0 ** -23 * (x.abs() + x.amax(-1, keepdim=True) - x) + 2.0 ** -19
    spread = lambda e: ((e * p) ** 2 @ v ** 2).sqrt()  # noqa: E731
    total = ((eps * p) ** 2).sum(-1, keepdim=True).sqrt() + n ** 0.5 * 2.0 ** -24
    ones = torch.ones_like(eps)
    bound = SIGMAS * (spread(eps + (2.0 ** -16 if parts else 0.0)) + (32 + n ** 0.5) * 2.0 ** -24 * spread(ones) + out.abs() * total)
    return out, bound


def lean(out, ref):
    """How much the outputs are too large (negative: too small) in all, as a share of their size."""
    return float(((out.double() - ref) * ref.sign()).sum() / ref.abs().sum())


def lean_bound(d):
    """A tile's 16 additions towards zero take at most 16 * 2^-23 of a tile's sum, and a score's d / 16 take
    (d / 16) 2^-23 of the score, which for scores of variance 1 moves outputs of random values by as much; the
    rest is rounded to nearest or divides out.  Kept over L tiles, a sum would lose ~L times the first part."""
    return (16 + d / 16) * 2.0 ** -23
