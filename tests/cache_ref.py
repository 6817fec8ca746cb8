"""The paged int8 cache on the host: the append rule in fp32 as it is stated (numpy, every operation rounded), and
attention over the codes in fp64."""
import math

import numpy as np
import torch

PAGE = 64
F = np.float32


def rotate(x, cos, sin, dim, interleaved):
    """x float32 [..., d]; cos, sin float32 [..., dim / 2]: the leading dim columns rotated, products and sums rounded."""
    y = x.copy()
    i = np.arange(0, dim, 2) if interleaved else np.arange(dim // 2)
    j = i + 1 if interleaved else i + dim // 2
    a, b = x[..., i], x[..., j]
    y[..., i] = a * cos - b * sin
    y[..., j] = b * cos + a * sin
    return y


class HostCache:
    """The cache's contents and its append rule, page by page."""

    def __init__(self, k, v, k_scale, v_scale):
        self.codes = {"k": k.copy(), "v": v.copy()}
        self.scale = {"k": k_scale.copy(), "v": v_scale.copy()}

    def append(self, which, rows, table, start):
        """rows float32 [H, n, d] (already rotated) at positions start.. of the sequence with pages `table`."""
        codes, scale = self.codes[which], self.scale[which]
        n = rows.shape[1]
        for p in range(start // PAGE, (start + n - 1) // PAGE + 1) if n else []:
            lo, hi = max(start, p * PAGE), min(start + n, (p + 1) * PAGE)
            held = lo - p * PAGE
            g = table[p]
            for h in range(rows.shape[0]):
                y = rows[h, lo - start:hi - start]
                old = scale[g, h] if held else F(0)
                if not np.all(np.isfinite(y)) or not np.isfinite(old):
                    scale[g, h] = np.nan
                    codes[g, h, held:held + hi - lo] = 0
                    continue
                new = max(old, np.abs(y).max() / F(127), F(2.0 ** -100))
                if new > old and held:
                    codes[g, h, :held] = np.rint(codes[g, h, :held].astype(F) * (old / new)).astype(np.int8)
                codes[g, h, held:held + hi - lo] = np.clip(np.rint(y * (F(1) / new)), -127, 127).astype(np.int8)
                scale[g, h] = new


def values(codes, scale, table, length):
    """fp64 [H, length, d]: the rows of one sequence."""
    g = torch.as_tensor(table, dtype=torch.long)[: -(-length // PAGE)]
    x = codes[g].double() * scale[g].double()[:, :, None, None]
    return x.permute(1, 0, 2, 3).reshape(codes.shape[1], -1, codes.shape[3])[:, :length]


def attend(q, k, v, causal=False, bias=None):
    """q fp64 [H, n, d] over k, v fp64 [Hkv, len, d]; bias [n, len] is added to the scores.  Returns o [H, n, d], lse
    [H, n], and what the error bounds need: sum p |v| / sum p, and the largest sum |q k| / sqrt(d) of each row."""
    H, n, d = q.shape
    g = H // k.shape[0]
    k, v = k.repeat_interleave(g, 0), v.repeat_interleave(g, 0)
    x = q @ k.transpose(1, 2) / math.sqrt(d)
    if bias is not None:
        x = x + bias
    if causal:
        L = k.shape[1]
        x = x.masked_fill(torch.arange(L) > L - n + torch.arange(n)[:, None], -math.inf)
    if x.shape[2] == 0:
        z = torch.zeros(H, n, d, dtype=torch.float64)
        return z, torch.full((H, n), -math.inf, dtype=torch.float64), z, torch.zeros(H, n, dtype=torch.float64)
    lse = torch.logsumexp(x, dim=-1)
    w = torch.exp(x - torch.where(torch.isinf(lse), 0.0, lse)[..., None])
    reach = (q.abs() @ k.abs().transpose(1, 2)).amax(-1) / math.sqrt(d)
    return w @ v, lse, w @ v.abs(), reach


def bounds(o, lse, spread, reach, keys, d):
    """How far a kernel with bf16 probabilities and output and fp32 sums may be from attend()'s values.
    Scores: d + 4 roundings of 2^-24 of at most `reach`; penalty, exponent arguments (at most 2^7 in magnitude, with
    the scale's logarithm folded in) and exp2 itself: 2^-16 of a probability; the sum of `keys` terms: keys 2^-24.
    A probability is then rounded to bf16 (2^-8 of it) and so is the output (2^-8)."""
    p = (d + 4) * 2.0 ** -24 * reach + 2.0 ** -16 + keys * 2.0 ** -24
    tol_o = (2.0 ** -8 + 2 * p)[..., None] * spread * (1 + 2.0 ** -7) + 2.0 ** -8 * o.abs() + 1e-30
    tol_l = p + 2.0 ** -22 * lse.abs().clamp(max=1e30)
    return tol_o, tol_l
