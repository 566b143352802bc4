"""The fp64 oracle of the gated delta rule and of the group norm (CPU):
against the C oracle of the plain delta rule, hand-worked values and central
differences."""
import numpy as np
import pytest

import oracle
from oracle import gated


def _inputs(B=2, Hk=2, H=4, L=5, d_k=6, d_v=3, seed=0):
    r = np.random.default_rng(seed)
    return dict(q=r.standard_normal((B, Hk, L, d_k)), k=r.standard_normal((B, Hk, L, d_k)),
                v=r.standard_normal((B, H, L, d_v)), g=-r.random((B, H, L)), beta=r.random((B, H, L)),
                W0=r.standard_normal((B, H, d_v, d_k)))


def test_without_decay_it_is_the_delta_rule():
    d = _inputs(Hk=2, H=2, d_k=8, L=9)
    y, W = oracle.delta_forward(d["q"], d["k"], d["v"], d["beta"], np.ones((2, 2, 3, 16)), 1, 1e-6)
    yg, Wg = gated.gated_forward(oracle.dpfp(d["q"], 1, 1e-6), oracle.dpfp(d["k"], 1, 1e-6), d["v"], 0 * d["g"],
                                 d["beta"], np.ones((2, 2, 3, 16)), l2norm=False)
    assert np.allclose(y, yg, rtol=1e-12, atol=1e-14) and np.allclose(W, Wg, rtol=1e-12, atol=1e-14)


def test_one_token_by_hand():
    # unit key (3, 4) / 5; W0 k = 5, decayed by 1/2 to 2.5; u = 0.5 (7 - 2.5) = 2.25
    y, W = gated.gated_forward([[[[5.0, 0.0]]]], [[[[3.0, 4.0]]]], [[[[7.0]]]], [[[np.log(0.5)]]], [[[0.5]]],
                               [[[[3.0, 4.0]]]], scale=2.0, eps=0.0)
    assert np.allclose(W, [[[[1.5 + 2.25 * 0.6, 2 + 2.25 * 0.8]]]])
    assert np.allclose(y, 2 * (1.5 + 2.25 * 0.6))


def test_a_gate_of_minus_infinity_forgets():
    d = _inputs()
    d["g"][:, :, 2] = -np.inf
    y, W = gated.gated_forward(**d)
    d2 = {n: (x if n == "W0" else x[:, :, 2:]) for n, x in d.items()}
    d2["W0"] = None
    d2["g"] = np.where(np.isinf(d2["g"]), 0, d2["g"])
    y2, W2 = gated.gated_forward(**d2)
    assert np.allclose(y[:, :, 2:], y2) and np.allclose(W, W2)


@pytest.mark.parametrize("l2norm", [True, False])
@pytest.mark.parametrize("lengths", [None, [3, 0]])
def test_gradients_are_the_differences(l2norm, lengths):
    d = _inputs(seed=3)
    r = np.random.default_rng(4)
    dy, dW = r.standard_normal((2, 4, 5, 3)), r.standard_normal((2, 4, 3, 6))
    opt = dict(lengths=lengths, l2norm=l2norm, scale=0.7)

    def loss(x):
        y, W = gated.gated_forward(**x, **opt)
        return (y * dy).sum() + (W * dW).sum()

    got = dict(zip(("q", "k", "v", "g", "beta", "W0"),
                   gated.gated_backward(d["q"], d["k"], d["v"], d["g"], d["beta"], dy, d["W0"], dW, **opt)))
    for n in d:
        for _ in range(3):
            way = r.standard_normal(d[n].shape)
            up, dn = (loss({**d, n: d[n] + s * way}) for s in (1e-5, -1e-5))
            assert abs((up - dn) / 2e-5 - (got[n] * way).sum()) <= 1e-7 * max(1, abs((got[n] * way).sum())), n


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("gate", [True, False])
def test_norm_gradients_are_the_differences(act, gate):
    r = np.random.default_rng(5)
    B, H, L, d = 2, 3, 4, 6
    a = dict(x=r.standard_normal((B, H, L, d)), gamma=r.standard_normal(H * d), beta=r.standard_normal(H * d))
    if gate:
        a["gate"] = r.standard_normal((B, L, H * d))
    do = r.standard_normal((B, L, H * d))
    dx, dgate, dgamma, dbeta = gated.group_norm_act(**a, act=act, dout=do)
    for n, got in (("x", dx), ("gate", dgate), ("gamma", dgamma), ("beta", dbeta)):
        if n not in a:
            assert got is None
            continue
        way = r.standard_normal(a[n].shape)
        up, dn = ((gated.group_norm_act(**{**a, n: a[n] + s * way}, act=act) * do).sum() for s in (1e-6, -1e-6))
        assert abs((up - dn) / 2e-6 - (got * way).sum()) <= 1e-6 * max(1, abs((got * way).sum())), n


def test_norm_of_one_row_by_hand():
    # (1, 3): mean 2, variance 1; relu((-1, 1) * 2 + 0.5)
    out = gated.group_norm_act([[[[1.0, 3.0]]]], [2.0, 2.0], [0.5, 0.5], act="relu", eps=0.0)
    assert np.allclose(out, [[[0.0, 2.5]]])
