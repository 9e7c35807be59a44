"""Plain 64-bit form of linear attention with a decay for each head, with bounds as tight as what the kernels promise.

Every output is a sum of products of inputs and decays e^D over pairs of a token s and a later or equal one t (and over the
initial state and the final gradient). To first order its error is the sum of the terms' magnitudes, each times
    ULP (2 |D| + dk + dv + m + 64), m the sequence's tokens: the decay's exponent, of magnitude |D| log2 e, is rounded twice, its
        exponential has an ulp or two; at most dk + dv + m additions, each half an ulp of a partial sum that the magnitudes bound;
        64 for the other roundings
    2^-16 in bf16: the factors that are fp32 (decayed scores, states, decayed values) enter a product as two or three bf16
        parts. Two leave at most 2^-17 of the factor, and a term has at most two such factors.
Outputs in bf16 add their rounding, at most 2^-8 of the value.

The decays' gradient dg_t = sum of the pairs s < t <= u. It may be formed from the block's end, as the sum of q . dq - k . dk
over the tokens from t on and the value behind them; the pairs of two tokens from t on cancel there but for their rounding. What
is promised is that such a sum reaches at most 127 tokens behind t, and none past a token whose factor is 0. So the bound is the largest,
over the token e = t .. t + 127 (before the next such token) where the sum may start, of the magnitudes of the value behind e and of
every q . dq and k . dk from t to e. Each factor of the value is itself a state or a gradient (m additions each, 4 |D|), its
product dk dv / 64 + 16 additions in one lane and the tree."""
import numpy as np

from block_reference import TINY, ULP

PARTS = 2.0 ** -16
REACH = 127
NO_FACTOR = -104.0


def _t(a):
    return a.transpose(0, 2, 1)


def linattn(q, k, v, g, scale, bounds, h0=None, reverse=False, dy=None, dh_last=None, bf16=False):
    """q, k (tokens, G, dk), v (tokens, H, dv), g (tokens, H) or (H,), h0 and dh_last (sequences, H, dk, dv), all float64.
    Returns a dict of name -> (value, bound); the gradients where dy or dh_last is given."""
    n, G, dk = q.shape
    H, dv = v.shape[1:]
    rep = H // G
    grads = dy is not None or dh_last is not None
    gt = np.maximum(np.broadcast_to(g, (n, H)), -200.0)
    shapes = dict(y=v.shape, h_last=(len(bounds), H, dk, dv))
    if grads:
        shapes.update(dq=(n, H, dk), dk=(n, H, dk), dv=v.shape, dg=(n, H), dh0=(len(bounds), H, dk, dv))
    out = {name: (np.zeros(s), np.zeros(s)) for name, s in shapes.items()}
    parts = PARTS if bf16 else 0.0
    for j, (lo, hi) in enumerate(bounds):
        rows = np.arange(hi - 1, lo - 1, -1) if reverse else np.arange(lo, hi)
        for h in range(H):
            one = _head(q[rows, h // rep], k[rows, h // rep], v[rows, h], gt[rows, h], scale,
                        h0[j, h] if h0 is not None else np.zeros((dk, dv)),
                        (dy[rows, h] if dy is not None else np.zeros((len(rows), dv))) if grads else None,
                        dh_last[j, h] if dh_last is not None else np.zeros((dk, dv)), parts)
            for name, (val, err) in one.items():
                at = (j, h) if name in ("h_last", "dh0") else (rows, h)
                out[name][0][at], out[name][1][at] = val, err
    if grads:
        for name in ("dq", "dk"):
            out[name] = tuple(t.reshape(n, G, rep, dk).sum(2) for t in out[name])
        if g.ndim == 1:
            out["dg"] = tuple(t.sum(0) for t in out["dg"])
    return {name: (val, err * 1.01 + ULP * np.abs(val) + TINY) for name, (val, err) in out.items()}


def _head(Q, K, V, g, scale, S0, Y, E, parts):
    m, dk, dv = len(Q), Q.shape[1], V.shape[1]
    cum = np.cumsum(g)
    end = cum[-1] if m else 0.0
    D = cum[:, None] - cum[None, :]
    M = np.where(np.tril(np.ones((m, m), dtype=bool)), np.exp(np.minimum(D, 700.0)), 0.0)
    c = dk + dv + m + 64

    def rel(d, times=2, more=0):
        return ULP * (times * np.abs(d) + c + more) + parts

    MR = M * rel(D)
    into, left, whole = np.exp(cum)[:, None], np.exp(end - cum)[:, None], np.exp(end)
    intoR, leftR, wholeR = into * rel(cum)[:, None], left * rel(end - cum)[:, None], whole * rel(end)
    aQ, aK, aV, aS0 = np.abs(Q), np.abs(K), np.abs(V), np.abs(S0)
    A, aA = Q @ K.T, aQ @ aK.T
    out = dict(y=(scale * ((A * M) @ V + into * (Q @ S0)), abs(scale) * ((aA * MR) @ aV + intoR * (aQ @ aS0))),
               h_last=(whole * S0 + (K * left).T @ V, wholeR * aS0 + (aK * leftR).T @ aV))
    if Y is None:
        return out
    Y = scale * Y
    aY, aE = np.abs(Y), np.abs(E)
    P, aP = Y @ V.T, aY @ aV.T
    out["dq"] = (P * M) @ K + into * (Y @ S0.T), (aP * MR) @ aK + intoR * (aY @ aS0.T)
    out["dk"] = (P * M).T @ Q + left * (V @ E.T), (aP * MR).T @ aQ + leftR * (aV @ aE.T)
    out["dv"] = (A * M).T @ Y + left * (K @ E), (aA * MR).T @ aY + leftR * (aK @ aE)
    out["dh0"] = (Q * into).T @ Y + whole * E, (aQ * intoR).T @ aY + wholeR * aE
    if m == 0:
        out["dg"] = np.zeros(0), np.zeros(0)
        return out
    # dg: the pairs (u, s), without a token's own; the initial state read at u; the final gradient of s; both
    more = m + dk * dv / 64 + 16

    def across(pair, read, kept, both):
        """Sum over s < t <= u for every t, by two-dimensional sums; t = 0 .. m (m: behind the last token)."""
        F = np.zeros((m + 1, m + 1))
        F[:m, 1:] = np.cumsum(np.cumsum(pair[::-1], 0)[::-1], 1)       # F[t, t']: u >= t, s < t'
        i = np.arange(m + 1)
        tail = np.append(np.cumsum(read[::-1])[::-1], 0.0)
        head = np.concatenate([[0.0], np.cumsum(kept)])
        return F[i, i] + tail + head + both

    off = ~np.eye(m, dtype=bool)
    read, kept, both = (Q * (into * (Y @ S0.T))).sum(1), (K * (left * (V @ E.T))).sum(1), (whole * S0 * E).sum()
    dg = across(A * P * M * off, read, kept, both)[:m]
    R = rel(D, 4, more) * off
    pair = aA * aP * M * R
    read = (aQ * (into * (aY @ aS0.T))).sum(1) * rel(cum, 4, more)
    kept = (aK * (left * (aV @ aE.T))).sum(1) * rel(end - cum, 4, more)
    both = (whole * aS0 * aE).sum() * rel(end, 4, more)
    value = across(pair, read, kept, both)                              # behind token e: value[e + 1]
    terms = pair.sum(1) + read + pair.sum(0) + kept                     # of q . dq and k . dk
    err = value[:m].copy()
    for t in range(m):
        total = 0.0
        for e in range(t, min(t + REACH + 1, m)):
            if e > t and g[e] < NO_FACTOR:
                break
            total += terms[e]
            err[t] = max(err[t], total + value[e + 1])
        if g[t] < NO_FACTOR:
            err[t] = value[t]
    out["dg"] = dg, err + ULP * np.abs(dg)
    return out
