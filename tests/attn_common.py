"""64-bit forms of the attention calls for their tests: the stored form of a
group of channels, attention by its definition, and how far a kernel may be
off.

Tolerances count roundings.  An output is rounded to bf16 once (at most 2^-8
of it); ``p_step`` is the rounding of a weight before it meets its value, per
key at most p_step * p_j |v_j|, which sums to p_step * A with A = sum p_j |v_j|;
fp32 sums of n terms are off by at most n 2^-24 A; a score is off by at most
(D + 8) 2^-24 scale sum_d |q_d k_d| =: e at most.  With scores s_j + d_j, |d_j|
<= e, a weight exp(s_j + d_j) / sum exp(s_i + d_i) lies between p_j exp(-2e)
and p_j exp(2e), which moves y by (exp(2e) - 1) A at most: 2e A for a small e,
where another 2e A is left for the exponentials and their sum (a few 2^-23),
but not 4e A for a large one (e = 2.8 allows 270 A, queries of 1024 against
keys near 100).
"""
import numpy as np
import torch

P_BF16, P_F16 = 2.0 ** -8, 2.0 ** -11


def stored(x, group):
    """The values (float64) that the cache holds for rows x (bf16)."""
    g = x.detach().cpu().double().numpy().reshape(x.shape[0], -1, group)
    out = np.empty_like(g)
    for idx in np.ndindex(*g.shape[:2]):
        v = g[idx]
        if not np.all(np.isfinite(v)):
            out[idx] = np.nan
            continue
        lo = v.min()
        s = torch.tensor(np.float32((v.max() - lo) / 15)).to(torch.bfloat16).double().item()
        code = np.minimum(np.rint((v - lo) / s), 15) if s > 0 else np.zeros_like(v)
        out[idx] = lo + code * s
    return torch.from_numpy(out.reshape(x.shape))


def attend(q, k, v, heads, kv_heads, scale, seen):
    """(y, A, e): rows q [n, heads * d] over k, v [keys, kv_heads * d] in
    float64; seen: bool [n, keys].  Hidden keys are left out of every sum."""
    n, keys = q.shape[0], k.shape[0]
    d = q.shape[1] // heads
    q, k, v = (t.detach().cpu().double() for t in (q, k, v))
    y, amount = torch.zeros(n, heads, d, dtype=torch.float64), torch.zeros(n, heads, d, dtype=torch.float64)
    err = torch.zeros(n, heads, 1, dtype=torch.float64)
    for h in range(heads):
        c = h // (heads // kv_heads)
        qh, kh, vh = q[:, h * d:(h + 1) * d], k[:, c * d:(c + 1) * d], v[:, c * d:(c + 1) * d]
        for i in range(n):
            at = torch.nonzero(seen[i])[:, 0]
            if not len(at):
                continue
            s = kh[at] @ qh[i] * scale
            p = torch.softmax(s, dim=0)
            y[i, h] = p @ vh[at]
            amount[i, h] = p @ vh[at].abs()
            mag = (kh[at].abs() @ qh[i].abs()) * abs(scale)
            err[i, h] = (d + 8) * 2.0 ** -24 * mag.max()
    return y.reshape(n, -1), amount.reshape(n, -1), err.expand(n, heads, d).reshape(n, -1)


def visible(n, keys, causal=True, window=0):
    p = torch.arange(n)[:, None] + keys - n
    j = torch.arange(keys)[None, :]
    seen = torch.ones(n, keys, dtype=torch.bool)
    if causal:
        seen &= j <= p
    if window:
        seen &= j > p - window
    return seen


def bound(y, amount, err, keys, p_step, floor=0.0):
    return floor + 2.0 ** -8 * y.abs() + (p_step * 1.01 + (keys + 64) * 2.0 ** -24 + 2 * err + torch.expm1(2 * err)) * amount + 1e-37


def cache_floor(v, keys):
    """How far attention over the cache may be off beside its roundings: a
    product of a weight and a scale is held as two fp16 numbers in units of
    2^(E - 8), so it is off by half a subnormal step, 2^-25 units, where 2^E is
    at most twice the greatest scale or minimum among the tokens seen (at most
    the greatest |v|): 2^-32 of it a key, times a code of 15 at most, over a sum
    of weights of at least 1."""
    return keys * 2.0 ** -28 * v.abs().max().item()


def check(got, want, amount, err, keys, p_step, label="", floor=0.0):
    got = got.detach().cpu().double()
    off = (got - want).abs()
    lim = bound(want, amount, err, keys, p_step, floor)
    bad = ~(off <= lim)
    assert not bad.any(), (f"{label}: {int(bad.sum())} of {bad.numel()} outside, first {torch.nonzero(bad)[0].tolist()}: "
                           f"{got[bad][0].item()} for {want[bad][0].item()}, bound {lim[bad][0].item()}")
