"""The bounds that linear attention is tested with (linattn_bounds) are met by two bf16 parts of a score and not by one, and
their sums for the decays' gradient are those of its definition."""
import numpy as np
import torch

import linattn_bounds
from block_reference import BF16_HALF


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(torch.bfloat16).double().numpy()


def problem(m=300, d=64, seed=0):
    rng = np.random.default_rng(seed)
    q, k, v, dy = (bf16(rng.standard_normal((m, 1, d))) for _ in range(4))
    return q, k, v, -np.abs(rng.standard_normal((m, 1))), dy


def test_one_part_of_a_score_is_outside_the_bounds():
    q, k, v, g, _ = problem()
    m, _, d = q.shape
    scale = float(np.float32(d ** -0.5))
    val, err = linattn_bounds.linattn(q, k, v, g, scale, [(0, m)], bf16=True)["y"]
    cum = np.cumsum(g[:, 0])
    M = np.where(np.tril(np.ones((m, m), dtype=bool)), np.exp(np.minimum(cum[:, None] - cum[None], 0.0)), 0.0)
    P = q[:, 0] @ k[:, 0].T * M * scale
    own = np.linalg.norm(bf16(val) - val)
    parts = np.zeros_like(P)
    for n in (1, 2):
        parts = parts + bf16(P - parts)
        y = bf16(parts @ v[:, 0])[:, None]
        inside = (np.abs(y - val) <= err + BF16_HALF * np.abs(val)).all()
        near = np.linalg.norm(y - val) <= 1.1 * own
        assert (inside, near) == (n == 2, n == 2), n


def test_the_decays_gradient_is_that_of_the_definition():
    q, k, v, g, dy = problem(60, 8, 1)
    rng = np.random.default_rng(2)
    h0, dh = rng.standard_normal((2, 1, 1, 8, 8))
    for reverse in (False, True):
        val, _ = linattn_bounds.linattn(q, k, v, g, 0.5, [(0, 60)], h0, reverse, dy, dh)["dg"]
        S, states, order = h0[0, 0], [], list(range(60))[::-1 if reverse else 1]
        for t in order:
            states.append(S)
            S = np.exp(g[t, 0]) * S + np.outer(k[t, 0], v[t, 0])
        E = dh[0, 0]
        for S, t in zip(states[::-1], order[::-1]):
            D = E + 0.5 * np.outer(q[t, 0], dy[t, 0])
            E = np.exp(g[t, 0]) * D
            assert abs((S * E).sum() - val[t, 0]) <= 1e-12 * max(1.0, abs(val[t, 0]))
