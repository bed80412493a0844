"""The latent-attention operators in 64 bits, from their formulas, on whatever
device the inputs live on; and the error that their roundings allow."""
import math

import torch


def frequencies(d, base=10000.0, scaling="plain", factor=1.0, original=4096, fast=32.0, slow=1.0):
    """(angle per position of each pair, factor on cos and sin)."""
    f = [base ** (-2.0 * i / d) for i in range(d // 2)]
    if scaling == "linear":
        return [x / factor for x in f], 1.0
    if scaling == "yarn":
        pair_of = lambda turns: d * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(pair_of(fast)), 0), min(math.ceil(pair_of(slow)), d - 1)
        g = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001))) for i in range(d // 2)]
        return [x * (1 - w) + x / factor * w for x, w in zip(f, g)], 0.1 * math.log(factor) + 1.0
    return f, 1.0


def rotate(x, positions, half, freq, mul=1.0):
    """x [n, d] (any dtype) rotated by positions [n], in 64 bits."""
    d = x.shape[-1]
    angle = positions.double()[:, None] * torch.tensor(freq, dtype=torch.float64, device=x.device)
    c, s = angle.cos() * mul, angle.sin() * mul
    i = torch.arange(d // 2, device=x.device)
    e0, e1 = (i, i + d // 2) if half else (2 * i, 2 * i + 1)
    y = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    a, b = x[:, e0].double(), x[:, e1].double()
    y[:, e0] = a * c - b * s
    y[:, e1] = a * s + b * c
    return y


def slots_of(cache, block_table, q, slots):
    """Cache entries of a request's slots, in 64 bits."""
    b = cache.shape[1]
    return cache[block_table[q].long()[slots // b], slots % b].double()


def attend(q, k, v, scale):
    """One softmax over the tokens: q [n, W], k [t, W], v [t, dv] in 64 bits ->
    (out [n, dv], lse [n], sum p |v|, sqrt(sum p^2 v^2), max_j scale |q| . |k_j|)."""
    if k.shape[0] == 0:
        z = torch.zeros((q.shape[0], v.shape[1]), dtype=torch.float64, device=q.device)
        return z, torch.full((q.shape[0],), -math.inf, dtype=torch.float64, device=q.device), z, z, z[:, 0]
    s = q @ k.T * scale
    lse = torch.logsumexp(s, dim=-1)
    p = (s - lse[:, None]).exp()
    return p @ v, lse, p @ v.abs(), (p.square() @ v.square()).sqrt(), (q.abs() @ k.abs().T).amax(-1) * scale


def half_step(dtype):
    """The largest relative error of one rounding."""
    return torch.finfo(dtype).eps / 2


def attention_bounds(out, lse, a, r, z, dtype, width):
    """Allowed |error| of each output element and lse, and of the outputs' 2-norm.

    Roundings: the weights (to dtype, half a step each: u), the output (u), and
    in fp32 the dot products (width terms, each product and sum half a step of
    2^-24, against sum |q||k| = z), exp2 and the sums (a few 2^-24 each, taken
    as 16 together).  A logit off by e changes a weight by the factor 1 + e and
    the normalisation by as much again.  The errors of the weights' roundings
    are independent, so their 2-norm over many elements is at most u *
    sqrt(sum p^2 v^2) (u bounds each, their spread is u / sqrt 3), while the
    logits' errors are taken at their bound."""
    u = half_step(dtype)
    e = z * width * 2.0 ** -24 + 16 * 2.0 ** -24
    elem = u * (a + out.abs()) + 2.1 * e[..., None] * a + 1e-30
    norm = u * (r.norm() + out.norm()) + 2.1 * (e[..., None] * a).norm() + 1e-30
    return elem, e + lse.abs().nan_to_num(posinf=0, neginf=0) * 2.0 ** -23, norm


def check(got, want, elem, norm=None, what=""):
    err = (got.double() - want).abs()
    assert torch.isfinite(got).all(), what
    worst = (err - elem).max().item()
    assert worst <= 0, (what, "element", worst, err.max().item())
    if norm is not None:
        assert err.norm() <= norm, (what, "2-norm", err.norm().item(), float(norm))
