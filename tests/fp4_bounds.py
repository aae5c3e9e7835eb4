"""Rounding bounds of the 4-bit attention and weights, per query, head and entry.

With z_s = scale q . v_s, a_s = scale sum_d |q_d v_sd| and zmax = max_s |z_s|,
the exponent of an entry's softmax weight is off by at most
    e_s = c 2^-24 a_s              the fp32 sum of c exact products
        + 2^-21 (|z_s| + zmax + 2) the scale's, the shift's and the exponential's roundings
(at most eight roundings of 2^-24 each). Sums of k weights: one addition per 64
entries and at most 80 more to join threads, warps and splits, (k/64 + 80)
2^-24; the second product's, k + 80 steps of 2^-23 (a tensor core may cut what it
does not round). Weights and outputs are rounded to bf16, half a step each:
2^-8. With p_s = e^(z_s - lse) and E = sum_s p_s e_s + (k/64 + 80) 2^-24:
    |out - ref| <= (1 + 2^-8) (sum_s p_s |v_s| (2^-8 + e_s + (k + 80) 2^-23) + |ref| E) + 2^-8 |ref|
    |lse - ref| <= E + 2^-21 (1 + |ref|)
(queries of zeros: every softmax weight is 1, which bf16 holds; the first 2^-8 is then left out)
    |w_s - ref| <= sum_h p_hs (e^(e_hs + 2^-21 |lse_h|) - 1 + (H + 16) 2^-24)
"""
import numpy as np

H_ = 2.0 ** -8


def attention(q, V, idx, scale, sink=None, seq=None):
    """(out, lse, their bounds) in 64 bits: q [nq, H, c], V [B, N, c], idx [nq, k] (< 0: empty), sink [H]."""
    nq, H, c = q.shape
    out, lim = np.zeros((nq, H, c)), np.full((nq, H, c), 1e-37)
    lse, lim_l = np.full((nq, H), -np.inf), np.zeros((nq, H))
    for t in range(nq):
        s = idx[t][idx[t] >= 0]
        b = 0 if seq is None else seq[t]
        rows = V[b, s]
        z = scale * q[t] @ rows.T
        zmax = np.abs(z).max(1, keepdims=True) if len(s) else np.zeros((H, 1))
        e = c * 2.0 ** -24 * scale * (np.abs(q[t]) @ np.abs(rows).T) + 2.0 ** -21 * (np.abs(z) + zmax + 2)
        if sink is not None:
            z = np.concatenate((z, sink[:, None]), 1)
            e = np.concatenate((e, 2.0 ** -21 * (np.abs(sink)[:, None] + zmax + 2)), 1)
        if z.shape[1] == 0:
            continue
        m = z.max(1, keepdims=True)
        lse[t] = m[:, 0] + np.log(np.exp(z - m).sum(1))
        p = np.exp(z - lse[t][:, None])
        E = (p * e).sum(1) + (len(s) / 64 + 80) * 2.0 ** -24
        lim_l[t] = E + 2.0 ** -21 * (1 + np.abs(lse[t]))
        p, e = p[:, :len(s)], e[:, :len(s)]
        out[t] = p @ rows
        step = H_ if q[t].any() else 0.0
        lim[t] = (1 + H_) * ((p * (step + e + (len(s) + 80) * 2.0 ** -23)) @ np.abs(rows) + np.abs(out[t]) * E[:, None]) \
            + H_ * np.abs(out[t]) + 1e-37
    return out, lse, lim, lim_l


def outside(got, ref, lim):
    """The largest excess over the bound, as a multiple of it (<= 1: within). Infinities and NaN have to be equal."""
    got, fin = np.asarray(got, float), np.isfinite(ref)
    if not np.array_equal(got[~fin], ref[~fin], equal_nan=True):
        return np.inf
    r = np.abs(got[fin] - ref[fin]) / lim[fin]
    return np.inf if np.isnan(r).any() else r.max(initial=0.0)


def check_attention(out, lse, q, V, idx, scale, sink, seq):
    ref, ref_l, lim, lim_l = attention(q, V, idx, scale, sink, seq)
    worst, worst_l = outside(out, ref, lim), outside(lse, ref_l, lim_l)
    assert worst <= 1, f"out {worst:.2f} of the bound"
    assert worst_l <= 1, f"lse {worst_l:.2f} of the bound"


def weights(q, lse, rows, scale):
    """(weights, bounds) of rows [n, c], summed over the heads of q [H, c]; lse [H] (-inf: a head without weight)."""
    live = ~np.isneginf(lse)
    q, l = q[live], lse[live][:, None]
    z = scale * q @ rows.T
    e = q.shape[-1] * 2.0 ** -24 * scale * (np.abs(q) @ np.abs(rows).T) + 2.0 ** -21 * (2 * np.abs(z) + np.abs(l) + 2)
    p = np.exp(z - l)
    return p.sum(0), (p * (np.expm1(e) + (len(lse) + 16) * 2.0 ** -24)).sum(0) + 1e-37
