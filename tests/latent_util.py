"""Latent attention in float64 (torch on the host), for the tests: from the formulas,
sequence by sequence, with the bounds that the tests hold results to.

A result differs from the exact one by
  - the rounding of the output to bf16, at most 2^-8 of its size;
  - the rounding of the softmax weights to bf16, operands of the second product: at most 2^-8 of
    each weight, so 2^-8 of A = sum of p |v|;
  - fp32 sums: a score of K products in steps of 16 is off by at most (K / 16 + 16) 2^-23 of
    G = scale * sum |q k|, the weights by that share, the second sum likewise by its steps.
    With K <= 576 the first is at most 52 * 2^-23 G; G is taken from the inputs.
"""
import math

import torch

HALF_STEP = 2.0 ** -8  # of a bf16 value, relative


def rotate(v, positions, inv_freq, pairs):
    """v [T, ..., D] in float64, turned by its tokens' angles."""
    a = positions.double()[:, None] * inv_freq.double()
    shape = (v.shape[0],) + (1,) * (v.dim() - 2) + (a.shape[1],)
    c, s = a.cos().view(shape), a.sin().view(shape)
    out = torch.empty_like(v)
    half = v.shape[-1] // 2
    first, second = (slice(0, half), slice(half, None)) if pairs == "halves" else \
        (slice(0, None, 2), slice(1, None, 2))
    x, y = v[..., first], v[..., second]
    out[..., first] = x * c - y * s
    out[..., second] = y * c + x * s
    return out


def rows_of(kv, R, positions, inv_freq, gamma, eps, pairs):
    """Normed and rotated latent rows in float64."""
    kv = kv.double()
    c = kv[:, :R]
    c = c / torch.sqrt((c * c).mean(1, keepdim=True) + eps)
    if gamma is not None:
        c = c * gamma.double()
    return torch.cat([c, rotate(kv[:, R:], positions, inv_freq, pairs)], 1)


def softmax_rows(s, allowed, v, mag):
    """s [n, H, k] scores, allowed [n, k], v [H or 1, k, d], mag [n, H, k] sums of magnitudes.
    Returns out [n, H, d], lse [n, H] and their bounds; rows without keys: 0 and -inf."""
    s = s.masked_fill(~allowed[:, None], -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[..., None])
    out = torch.einsum("nhk,hkd->nhd", p, v.expand(s.shape[1], -1, -1))
    weight = torch.einsum("nhk,hkd->nhd", p, v.abs().expand(s.shape[1], -1, -1))
    worst = mag.masked_fill(~allowed[:, None], 0).amax(-1) if s.shape[-1] else lse * 0
    # scores: as above; the exponent's argument and the exponential: 2^-22 of up to 2 G + 2
    ds = 52 * 2.0 ** -23 * worst + 2.0 ** -22 * (2 * worst + 2)
    keys = s.shape[-1]
    sums = (keys / 16 + 16) * 2.0 ** -23
    bound = HALF_STEP * out.abs() + (HALF_STEP + 2 * ds[..., None] + sums) * weight * 1.01
    return out, lse, bound + 1e-30, 2 * ds + sums + 2.0 ** -22 * lse.abs().nan_to_num(0, 0, 0) + 1e-6


def attend(q, rows_by_seq, queries, R, scale):
    """Absorbed form: q [T, H, R + D], rows_by_seq: each sequence's rows (its length), queries:
    (first, last + 1) of each.  Returns out, lse and bounds for all of q; rows of no sequence nan."""
    q = q.double()
    T, H = q.shape[:2]
    out = torch.full((T, H, R), math.nan, dtype=torch.float64)
    lse = torch.full((T, H), math.nan, dtype=torch.float64)
    ob, lb = out.clone(), lse.clone()
    for rows, (lo, hi) in zip(rows_by_seq, queries):
        if hi <= lo:
            continue
        rows = rows.double()
        n, k = hi - lo, rows.shape[0]
        allowed = torch.arange(k)[None] <= torch.arange(k - n, k)[:, None]
        s = scale * torch.einsum("nhd,kd->nhk", q[lo:hi], rows)
        mag = scale * torch.einsum("nhd,kd->nhk", q[lo:hi].abs(), rows.abs())
        out[lo:hi], lse[lo:hi], ob[lo:hi], lb[lo:hi] = softmax_rows(s, allowed, rows[None, :, :R],
                                                                    mag)
    return out, lse, ob, lb


def prefill(q, k, v, k_rope, cu_q, cu_k, scale, causal):
    q, k, v, k_rope = (t.double() for t in (q, k, v, k_rope))
    T, H = q.shape[:2]
    nope = k.shape[2]
    out = torch.full((T, H, v.shape[2]), math.nan, dtype=torch.float64)
    lse = torch.full((T, H), math.nan, dtype=torch.float64)
    ob, lb = out.clone(), lse.clone()
    for b in range(len(cu_q) - 1):
        lo, hi, k0, k1 = cu_q[b], cu_q[b + 1], cu_k[b], cu_k[b + 1]
        if hi <= lo:
            continue
        n, m = hi - lo, k1 - k0
        allowed = torch.arange(m)[None] <= torch.arange(m - n, m)[:, None] if causal else \
            torch.ones(n, m, dtype=torch.bool)
        args = (q[lo:hi, :, :nope], k[k0:k1]), (q[lo:hi, :, nope:], k_rope[k0:k1])
        s = scale * (torch.einsum("nhd,khd->nhk", *args[0]) +
                     torch.einsum("nhd,kd->nhk", *args[1]))
        mag = scale * (torch.einsum("nhd,khd->nhk", *(t.abs() for t in args[0])) +
                       torch.einsum("nhd,kd->nhk", *(t.abs() for t in args[1])))
        out[lo:hi], lse[lo:hi], ob[lo:hi], lb[lo:hi] = softmax_rows(
            s, allowed, v[k0:k1].transpose(0, 1), mag)
    return out, lse, ob, lb


def check(got, want, bound, what):
    """Every element of got within its bound of want; equal infinities and nan pairs pass."""
    got = got.double().cpu()
    same = (got == want) | (got.isnan() & want.isnan())
    ok = same | ((got - want).abs() <= bound)
    if not bool(ok.all()):
        i = int((~ok).flatten().nonzero()[0])
        worst = ((got - want).abs() / bound).nan_to_num(math.inf)[~ok].max()
        raise AssertionError(
            f"{what}: {int((~ok).sum())} of {ok.numel()} out of bounds, first at {i}: "
            f"{got.flatten()[i]} for {want.flatten()[i]} +- {bound.flatten()[i]}; worst {worst}")
