"""Plain 64-bit form of linear attention with a decay for each head for the tests, each output with a bound on the
error that the kernels' arithmetic may leave in it.

Every output is a sum over pairs of a token s and a later one t (and over the initial state or the final gradient) of
products of inputs and a decay e^D. To first order its error is the sum of the terms' magnitudes, each times what its own
factors may be off by:
    ULP (2 |D| + dk + dv + tokens + 64): the decay's exponent, of magnitude up to |D| log2 e, is rounded twice and its
        exponential has an ulp or two; a term passes through at most dk + dv + tokens additions, each half an ulp
        of a partial sum that the magnitudes bound; 64 more for its other roundings (scales, decays of whole chunks)
    2^-16 in bf16, where fp32 factors of a product are the sum of three bf16 parts (2^-26 lost of each; the bound is that of two)
    2^-8 more in bf16 for outputs that are bf16 themselves and enter no fp32 output (y, dv; dq and dk where no gradient of the
        decays is formed): a term's score, or the state it is read from, is rounded to one bf16 part, half a step of which is 2^-8
Outputs in bf16 add their rounding, at most 2^-8 of the value."""
import numpy as np

from block_reference import TINY, ULP

SPLIT = 2.0 ** -16
ONE_PART = 2.0 ** -8


def rows_of(lo, hi, reverse):
    return np.arange(hi - 1, lo - 1, -1) if reverse else np.arange(lo, hi)


def linattn(q, k, v, g, scale, bounds, h0=None, reverse=False, dy=None, dh_last=None, bf16=False, decays=True):
    """q, k (tokens, G, dk), v (tokens, H, dv), g (tokens, H) or (H,), h0 and dh_last (sequences, H, dk, dv), all
    float64. Returns a dict of name -> (value, bound); gradients where dy or dh_last is given (decays: the decays' among them)."""
    n, G, dk = q.shape
    H, dv = v.shape[1:]
    rep = H // G
    by_head = g.ndim == 1
    gt = np.maximum(np.broadcast_to(g, (n, H)), -200.0)
    grads = dy is not None or dh_last is not None
    out = {}

    def slot(name, shape):
        out[name] = (np.zeros(shape), np.zeros(shape))

    slot("y", v.shape)
    slot("h_last", (len(bounds), H, dk, dv))
    if grads:
        for name, shape in (("dq", (n, H, dk)), ("dk", (n, H, dk)), ("dv", v.shape), ("dg", (n, H)),
                            ("dh0", (len(bounds), H, dk, dv))):
            slot(name, shape)

    def put(name, at, value, err):
        out[name][0][at], out[name][1][at] = value, err

    for j, (lo, hi) in enumerate(bounds):
        rows = rows_of(lo, hi, reverse)
        m = len(rows)
        Q, K = (np.repeat(t[rows], rep, 1).transpose(1, 0, 2) for t in (q, k))
        V = v[rows].transpose(1, 0, 2)                      # (H, m, d)
        S0 = h0[j] if h0 is not None else np.zeros((H, dk, dv))
        cum = np.cumsum(gt[rows], 0).T                      # (H, m)
        D = cum[:, :, None] - cum[:, None, :]
        tri = np.tril(np.ones((m, m), dtype=bool))
        M = np.where(tri, np.exp(np.where(tri, D, 0.0)), 0.0)
        c = dk + dv + m + 64
        extra = SPLIT if bf16 else 0.0
        MR = M * (ULP * (2 * np.abs(D) + c) + extra)
        into = np.exp(cum)[..., None]
        intoR = into * (ULP * (2 * np.abs(cum)[..., None] + c) + extra)
        end = cum[:, -1:] if m else np.zeros((H, 1))
        left = np.exp(end - cum)[..., None]
        leftR = left * (ULP * (2 * np.abs(end - cum)[..., None] + c) + extra)
        whole = np.exp(end)[..., None]
        wholeR = whole * (ULP * (2 * np.abs(end)[..., None] + c) + extra)
        aQ, aK, aV, aS0 = np.abs(Q), np.abs(K), np.abs(V), np.abs(S0)
        one = ONE_PART if bf16 else 0.0
        MO, intoO, leftO = MR + one * M, intoR + one * into, leftR + one * left
        MG, intoG, leftG = (MR, intoR, leftR) if decays else (MO, intoO, leftO)

        def T(t):
            return t.transpose(0, 2, 1)

        A, aA = Q @ T(K), aQ @ T(aK)
        put("y", rows, (scale * ((A * M) @ V + into * (Q @ S0))).transpose(1, 0, 2),
            abs(scale) * ((aA * MO) @ aV + intoO * (aQ @ aS0)).transpose(1, 0, 2))
        put("h_last", j, whole * S0 + T(K * left) @ V, wholeR * aS0 + T(aK * leftR) @ aV)
        if not grads:
            continue
        Y = scale * dy[rows].transpose(1, 0, 2) if dy is not None else np.zeros_like(V)
        E = dh_last[j] if dh_last is not None else np.zeros((H, dk, dv))
        aY, aE = np.abs(Y), np.abs(E)
        P, aP = Y @ T(V), aY @ T(aV)
        dq = (P * M) @ K + into * (Y @ T(S0))
        dq_e = (aP * MG) @ aK + intoG * (aY @ T(aS0))
        put("dq", rows, dq.transpose(1, 0, 2), dq_e.transpose(1, 0, 2))
        dk_ = T(P * M) @ Q + left * (V @ T(E))
        dk_e = T(aP * MG) @ aQ + leftG * (aV @ T(aE))
        put("dk", rows, dk_.transpose(1, 0, 2), dk_e.transpose(1, 0, 2))
        put("dv", rows, (T(A * M) @ Y + left * (K @ E)).transpose(1, 0, 2),
            (T(aA * MO) @ aY + leftO * (aK @ aE)).transpose(1, 0, 2))
        put("dh0", j, T(Q * into) @ Y + whole * E, T(aQ * intoR) @ aY + wholeR * aE)
        # dg_t: pairs s < t <= u, the initial state read at u >= t, the final gradient of s < t, both
        pairs, pairs_e = A * P * M, aA * aP * MR
        i = np.arange(m)
        pairs[:, i, i] = pairs_e[:, i, i] = 0.0

        def tail(t):
            return np.cumsum(t[:, ::-1], 1)[:, ::-1]

        read = (Q * (into * (Y @ T(S0)))).sum(-1)
        read_e = (aQ * (intoR * (aY @ T(aS0)))).sum(-1)
        kept = (K * (left * (V @ T(E)))).sum(-1)
        kept_e = (aK * (leftR * (aV @ T(aE)))).sum(-1)
        both, both_e = (whole * S0 * E).sum((-1, -2)), (wholeR * aS0 * aE).sum((-1, -2))
        last = both + kept.sum(-1)
        dg = tail(pairs.sum(2) + read) - tail(pairs.sum(1) + kept) + last[:, None]
        dg_e = tail(pairs_e.sum(2) + read_e) + tail(pairs_e.sum(1) + kept_e) + (both_e + kept_e.sum(-1))[:, None]
        put("dg", rows, dg.T, (dg_e + ULP * np.abs(dg)).T)
    if grads:
        for name in ("dq", "dk"):
            out[name] = tuple(t.reshape(n, G, rep, dk).sum(2) for t in out[name])
        if by_head:
            out["dg"] = tuple(t.sum(0) for t in out["dg"])
    return {name: (val, err * 1.01 + ULP * np.abs(val) + TINY) for name, (val, err) in out.items()}
