"""Plain 64-bit forms of the gated recurrence and the block norm for the tests, each output with a
bound on the error that 32-bit arithmetic may leave in it.

The bounds follow the rounding errors of a 32-bit evaluation to first order: ULP = 2^-23 is the
relative error allowed to one operation (the hardware's exp2, log2, rcp, rsq and sqrt have 1 ulp,
fma and mul half), a sigmoid of v costs |v| + 8 of them (the argument's rounding, scaled by |v|,
and its four operations), and errors are carried through the recurrence as it carries its values.
Outputs in bf16 (8 significant bits) add their rounding to nearest, at most 2^-8 of the value."""
import numpy as np

ULP = 2.0 ** -23
BF16_HALF = 2.0 ** -8
TINY = 1e-37      # the 32-bit range's end: results below it may be flushed to zero


def sigmoid(v):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-v))


def softplus(v):
    return np.maximum(v, 0.0) + np.log1p(np.exp(-np.abs(v)))


def bounds_of(nseq, length, offsets=None):
    if offsets is not None:
        return [(int(a), int(b)) for a, b in zip(offsets[:-1], offsets[1:])]
    return [(k * length, (k + 1) * length) for k in range(nseq)]


def gated(x, r, i, lam, c, bounds, h0=None, reverse=False, dy=None, dh_last=None, want_grads=False):
    """x, r, i (tokens, D), lam (D,), h0 and dh_last (sequences, D), all float64. Returns a dict of
    name -> (value, error bound)."""
    n, d = x.shape
    s, g, ng, ns = sigmoid(r), sigmoid(i), sigmoid(-i), sigmoid(-r)
    rate = c * softplus(lam)
    u = -rate * s
    a = np.exp(u)
    m2 = -np.expm1(2 * u)
    m = np.sqrt(m2)
    b = m * g * x
    # relative errors, in ulps: of u, of a, of m, of the input term
    ku = np.abs(r) + 8 + 6
    ka = np.abs(u) * ku + 2
    safe = np.where(m2 > 0, m2, 1.0)
    km = 0.5 * (ku + 8 + np.where(-2 * u >= 0.24, (2 * a * a * ka + 2) / safe, 0.0)) + 1
    kb = km + np.abs(i) + 8 + 2
    y, ye = np.zeros((n, d)), np.zeros((n, d))
    before, before_e = np.zeros((n, d)), np.zeros((n, d))
    h_last, h_last_e = np.zeros((len(bounds), d)), np.zeros((len(bounds), d))
    for q, (lo, hi) in enumerate(bounds):
        h = h0[q].copy() if h0 is not None else np.zeros(d)
        e = np.zeros(d)
        order = range(hi - 1, lo - 1, -1) if reverse else range(lo, hi)
        for t in order:
            before[t], before_e[t] = h, e
            e = a[t] * e + ULP * ((ka[t] + 2) * np.abs(a[t] * h) + (kb[t] + 1) * np.abs(b[t]))
            h = a[t] * h + b[t]
            y[t], ye[t] = h, e
        h_last[q], h_last_e[q] = h, e
    out = {"y": (y, ye + TINY), "h_last": (h_last, h_last_e + TINY)}
    if not want_grads:
        return out
    dl, dle = np.zeros((n, d)), np.zeros((n, d))
    dh0, dh0_e = np.zeros((len(bounds), d)), np.zeros((len(bounds), d))
    for q, (lo, hi) in enumerate(bounds):
        e = dh_last[q].copy() if dh_last is not None else np.zeros(d)
        err = np.zeros(d)
        order = range(lo, hi) if reverse else range(hi - 1, lo - 1, -1)
        for t in order:
            v = (dy[t] if dy is not None else 0.0) + e
            err = err + ULP * np.abs(v)
            dl[t], dle[t] = v, err
            e, err = a[t] * v, a[t] * err + ULP * (ka[t] + 1) * np.abs(a[t] * v)
        dh0[q], dh0_e[q] = e, err
    um = np.where(m > 0, u / np.where(m > 0, m, 1.0), 0.0)
    dx = dl * m * g
    dx_e = m * g * dle + ULP * kb * np.abs(dx)
    di = dx * x * ng
    di_e = np.abs(x * ng) * dx_e + ULP * (np.abs(i) + 10) * np.abs(di)
    t1, t2 = u * a * before, -g * x * a * a * um
    w = dl * (t1 + t2)
    w_e = (np.abs(t1 + t2) * dle + np.abs(dl) * np.abs(u * a) * before_e
           + ULP * np.abs(dl) * ((ku + ka + 4) * np.abs(t1) + (ku + 2 * ka + km + np.abs(i) + 14) * np.abs(t2)))
    dr = w * ns
    dr_e = ns * w_e + ULP * (np.abs(r) + 10) * np.abs(dr)
    share = sigmoid(lam) / softplus(lam)
    dlam = w.sum(0) * share
    # a sum in groups of 64 tokens, then over the groups
    dlam_e = (w_e.sum(0) + ULP * (128 + n / 64) * np.abs(w).sum(0)) * share + ULP * (np.abs(lam) + 16) * np.abs(dlam)
    out.update(dx=(dx, dx_e + TINY), di=(di, di_e + TINY), dr=(dr, dr_e + TINY), dlam=(dlam, dlam_e + TINY),
               dh0=(dh0, dh0_e + TINY))
    return out


def norm(x, z=None, w_post=None, residual=None, gamma=None, w_pre=None, eps=1e-5, gate_after=False, dsum=None,
         dn=None, want_grads=False):
    """x, z, residual (rows, D), weights (D,), float64. Returns a dict of name -> (value, bound). The
    bounds take a row's sum to be added in a tree with at most 64 additions in a row per lane."""
    rows, d = x.shape
    depth = 64 + 16
    gate = np.ones_like(x)
    kg = 0.0
    if z is not None:
        sg = sigmoid(z)
        gate = z * sg
        kg = np.abs(z) + 10
    v = x if gate_after else x * gate
    kv = 0.0 if gate_after else kg + 1
    rho1, kr1 = 1.0, 0.0
    q, kq = v, kv
    if w_post is not None:
        ss = (v * v).mean(1, keepdims=True) + eps
        kss = ((2 * kv + depth) * v * v).mean(1, keepdims=True) / ss + 4
        rho1, kr1 = 1 / np.sqrt(ss), 0.5 * kss + 2
        q, kq = v * rho1 * w_post, kv + kr1 + 2
    p, kp = (q * gate, kq + kg + 1) if gate_after else (q, kq)
    t, kt = (p * gamma, kp + 1) if gamma is not None else (p, kp)
    s = t + residual if residual is not None else t
    se = ULP * (kt * np.abs(t) + np.abs(s))
    out = {"sum": (s, se + TINY)}
    if w_pre is not None:
        ss2 = (s * s).mean(1, keepdims=True) + eps
        ess2 = (2 * np.abs(s) * se).mean(1, keepdims=True) + ULP * (depth + 4) * ss2
        rho2 = 1 / np.sqrt(ss2)
        rho2_e = 0.5 * rho2 / ss2 * ess2 + 2 * ULP * rho2
        n = s * rho2 * w_pre
        out["n"] = (n, np.abs(w_pre) * (se * rho2 + np.abs(s) * rho2_e) + 2 * ULP * np.abs(n) + TINY)
    if not want_grads:
        return out
    ds = dsum.copy() if dsum is not None else np.zeros_like(x)
    dse = ULP * np.abs(ds)
    if dn is not None:
        tw = dn * w_pre
        mt = (tw * s).mean(1, keepdims=True)
        mt_e = (np.abs(tw) * se).mean(1, keepdims=True) + ULP * depth * np.abs(tw * s).mean(1, keepdims=True)
        k2 = rho2 ** 3 * mt
        k2_e = rho2 ** 3 * mt_e + 3 * rho2 ** 2 * np.abs(mt) * rho2_e + 6 * ULP * np.abs(k2)
        ds = ds + rho2 * tw - s * k2
        dse = (dse + np.abs(tw) * rho2_e + np.abs(s) * k2_e + np.abs(k2) * se
               + 4 * ULP * (np.abs(rho2 * tw) + np.abs(s * k2) + np.abs(ds)))
    dp, dpe = (ds * gamma, np.abs(gamma) * dse + ULP * np.abs(ds * gamma)) if gamma is not None else (ds, dse)
    dq, dqe = dp, dpe
    if gate_after:
        dq = dp * gate
        dqe = np.abs(gate) * dpe + ULP * (kg + 1) * np.abs(dq)
    dv, dve = dq, dqe
    if w_post is not None:
        t1 = dq * w_post
        t1e = np.abs(w_post) * dqe + ULP * np.abs(t1)
        mt = (t1 * v).mean(1, keepdims=True)
        mt_e = (np.abs(v) * t1e).mean(1, keepdims=True) + ULP * ((kv + depth) * np.abs(t1 * v)).mean(1, keepdims=True)
        k1 = rho1 ** 3 * mt
        k1_e = rho1 ** 3 * mt_e + ULP * (3 * kr1 + 6) * rho1 ** 3 * np.abs(mt)
        dv = rho1 * t1 - v * k1
        dve = (rho1 * t1e + np.abs(v) * k1_e
               + ULP * ((kr1 + 3) * np.abs(rho1 * t1) + (kv + 3) * np.abs(v * k1) + np.abs(dv)))
        # sums over rows, in groups, then over the groups
        terms = dq * v * rho1
        out["dw_post"] = (terms.sum(0), (np.abs(v) * rho1 * dqe + ULP * (kv + kr1 + 4) * np.abs(terms)).sum(0)
                          + ULP * (64 + rows) * np.abs(terms).sum(0) + TINY)
    dx, dxe = dv, dve
    if z is not None:
        slope = sg * (1 + z * (1 - sg))
        slope_e = ULP * (np.abs(z) + 16) * sg * (1 + np.abs(z) * (1 - sg) * (np.abs(z) + 4))
        if gate_after:
            dz = dp * q * slope
            dze = np.abs(q * slope) * dpe + np.abs(dp * q) * slope_e + ULP * (kq + 4) * np.abs(dz)
        else:
            dx = dv * gate
            dxe = np.abs(gate) * dve + ULP * (kg + 1) * np.abs(dx)
            dz = dv * x * slope
            dze = np.abs(x * slope) * dve + np.abs(dv * x) * slope_e + ULP * 4 * np.abs(dz)
        out["dz"] = (dz, dze + TINY)
    out["dx"] = (dx, dxe + TINY)
    if residual is not None:
        out["dresidual"] = (ds, dse + TINY)
    if gamma is not None:
        terms = p * ds
        out["dgamma"] = (terms.sum(0), (np.abs(p) * dse + ULP * (kp + 4) * np.abs(terms)).sum(0)
                         + ULP * (64 + rows) * np.abs(terms).sum(0) + TINY)
    if w_pre is not None:
        g = dn if dn is not None else np.zeros_like(x)
        terms = g * s * rho2
        out["dw_pre"] = (terms.sum(0), (np.abs(g) * (se * rho2 + np.abs(s) * rho2_e) + 4 * ULP * np.abs(terms)).sum(0)
                         + ULP * (64 + rows) * np.abs(terms).sum(0) + TINY)
    return out


def check(got, want, bf16=False, what=""):
    """got: a torch tensor; want: (value, bound). NaN counts as a difference."""
    ref, err = want
    g = got.detach().double().cpu().numpy().reshape(ref.shape)
    bound = err + (BF16_HALF * (np.abs(ref) + err) if bf16 else 0.0)
    bad = ~(np.abs(g - ref) <= bound)
    if bad.any():
        k = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside the bound; first at {k}: got {g[k]!r}, want "
                             f"{ref[k]!r} +- {bound[k]:.3e}; worst {np.nanmax(np.abs(g - ref) / bound):.2f} bounds")
