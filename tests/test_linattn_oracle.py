"""The float64 oracle of the linear attention and of the head norms: against closed forms and differences (CPU)."""

import numpy as np
import pytest

import oracle.linattn as O


def _inputs(seed, B, T, Hk, H, Dk, Dv):
    r = np.random.default_rng(seed)
    return (r.standard_normal((B, T, Hk, Dk)), r.standard_normal((B, T, Hk, Dk)), r.standard_normal((B, T, H, Dv)),
            -np.abs(r.standard_normal(H)), r.standard_normal((B, H, Dk, Dv)))


def test_linattn_forward_is_the_masked_sum():
    q, k, v, ld, S0 = _inputs(0, 2, 9, 2, 4, 3, 5)
    o, S = O.linattn_forward(q, k, v, ld, S0, 0.7)
    for b in range(2):
        for h in range(4):
            g = np.exp(ld[h])
            for t in range(9):
                want = g ** (t + 1) * q[b, t, h // 2] @ S0[b, h]
                want = want + sum(g ** (t - j) * (q[b, t, h // 2] @ k[b, j, h // 2]) * v[b, j, h] for j in range(t + 1))
                np.testing.assert_allclose(o[b, t, h], 0.7 * want, rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(S[1, 3], np.exp(9 * ld[3]) * S0[1, 3] + sum(
        np.exp((8 - j) * ld[3]) * np.outer(k[1, j, 1], v[1, j, 3]) for j in range(9)), rtol=1e-12)


@pytest.mark.parametrize("T", [1, 5])
def test_linattn_backward_against_differences(T):
    q, k, v, ld, S0 = _inputs(1, 1, T, 1, 2, 3, 4)
    r = np.random.default_rng(2)
    dO, dS = r.standard_normal(v.shape), r.standard_normal(S0.shape)

    def loss(q, k, v, S0):
        o, S = O.linattn_forward(q, k, v, ld, S0, 0.3)
        return (dO * o).sum() + (dS * S).sum()

    g = O.linattn_backward(q, k, v, ld, dO, S0, dS, 0.3)
    x = {"dq": q, "dk": k, "dv": v, "dS0": S0}
    for n in x:
        for at in np.ndindex(x[n].shape):
            d = np.zeros_like(x[n])
            d[at] = 1e-5
            up, down = ({m: x[m] + (d * s if m == n else 0) for m in x} for s in (1, -1))
            diff = (loss(up["dq"], up["dk"], up["dv"], up["dS0"]) - loss(down["dq"], down["dk"], down["dv"], down["dS0"]))
            assert abs(diff / 2e-5 - g[n][at]) < 1e-7, (n, at)


@pytest.mark.parametrize("l2", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope_against_differences(l2, interleaved):
    r = np.random.default_rng(3)
    x, dy, w = r.standard_normal((3, 2, 16)), r.standard_normal((3, 2, 16)), r.standard_normal(16)
    pos, f = np.array([0, 7, 1000]), r.random(4)
    kw = dict(eps=0.1, l2=l2, interleaved=interleaved, scale=1.3)
    dx, dw = O.qk_norm_rope_backward(dy, x, pos, f, w, **kw)
    loss = lambda x, w: (dy * O.qk_norm_rope(x, pos, f, w, **kw)).sum()  # noqa: E731
    for at in np.ndindex(x.shape):
        d = np.zeros_like(x)
        d[at] = 1e-5
        assert abs((loss(x + d, w) - loss(x - d, w)) / 2e-5 - dx[at]) < 1e-7
    for at in range(16):
        d = np.zeros(16)
        d[at] = 1e-5
        assert abs((loss(x, w + d) - loss(x, w - d)) / 2e-5 - dw[at]) < 1e-7


def test_rotation_depends_on_the_distance_alone():
    r = np.random.default_rng(4)
    q, k, f = r.standard_normal((1, 1, 32)), r.standard_normal((1, 1, 32)), r.random(16)
    score = lambda p, s: (O.rotate(q, np.array([p]), f) * O.rotate(k, np.array([s]), f)).sum()  # noqa: E731
    assert abs(score(5, 2) - score(1005, 1002)) < 1e-11
