"""Pins of the oracle's attention (attend_fp64)."""
import math

import numpy as np
import pytest

import oracle as o


def brute(q, k, v, scale, causal):
    """The definition, one number at a time."""
    n, H, D = len(q), len(q[0]), len(q[0][0])
    m, Hkv = len(k), len(k[0]) if k else 1
    out = [[[0.0] * D for _ in range(H)] for _ in range(n)]
    for i in range(n):
        for h in range(H):
            g = h // (H // Hkv)
            seen = [j for j in range(m) if not causal or j <= i + m - n]
            if not seen:
                continue
            s = [scale * math.fsum(q[i][h][d] * k[j][g][d] for d in range(D)) for j in seen]
            w = [math.exp(x - max(s)) for x in s]
            for d in range(D):
                out[i][h][d] = math.fsum(wj * v[j][g][d] for wj, j in zip(w, seen)) / math.fsum(w)
    return out


@pytest.mark.parametrize("n,m,H,Hkv,causal", [(1, 1, 1, 1, True), (4, 4, 4, 2, True), (3, 7, 2, 1, True),
                                              (5, 2, 2, 2, True), (3, 0, 1, 1, False), (3, 5, 6, 2, False)])
def test_attend_matches_the_definition(n, m, H, Hkv, causal):
    rng = np.random.default_rng([n, m, H])
    q, k, v = rng.standard_normal((n, H, 8)), rng.standard_normal((m, Hkv, 8)), rng.standard_normal((m, Hkv, 8))
    got, a, e = o.attend_fp64(q, k, v, 0.7, causal)
    want = np.array(brute(q.tolist(), k.tolist(), v.tolist(), 0.7, causal)).reshape(got.shape)
    assert np.allclose(got, want, rtol=1e-13, atol=1e-13)
    assert np.all(a >= np.abs(got) - 1e-13) and np.all(e >= 0)
    if n > m and causal:
        assert not got[: n - m].any()


def test_attend_does_not_read_what_a_query_does_not_see():
    rng = np.random.default_rng(5)
    q, k, v = (rng.standard_normal((6, 2, 8)) for _ in range(3))
    want, _, _ = o.attend_fp64(q, k, v, 0.5)
    k[4], v[4] = np.nan, np.inf
    got, _, _ = o.attend_fp64(q, k, v, 0.5)
    assert np.array_equal(got[:4], want[:4]) and not np.isfinite(got[4:]).any()
