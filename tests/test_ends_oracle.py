"""The fp64 oracle of the embedding, the layer norm and the vocabulary loss:
its gradients against differences of its own values (CPU only)."""
import numpy as np
import pytest

from oracle import ends


def differences(f, x, step=1e-5):
    g = np.zeros_like(x)
    it = np.nditer(x, flags=["multi_index"])
    for _ in it:
        i = it.multi_index
        keep = x[i]
        x[i] = keep + step
        up = f()
        x[i] = keep - step
        g[i] = (up - f()) / (2 * step)
        x[i] = keep
    return g


def test_embedding():
    r = np.random.default_rng(0)
    table, ids = r.standard_normal((5, 8)), [3, -1, 0, 3, -7, 4]
    do = r.standard_normal((6, 8))
    f = lambda: float((ends.embedding(ids, table, 1.5) * do).sum())  # noqa: E731
    assert np.allclose(ends.embedding_backward(ids, do, 5, 1.5), differences(f, table), atol=1e-8)
    assert np.all(ends.embedding(ids, table)[[1, 4]] == 0) and np.isnan(ends.embedding([5], table)).all()


@pytest.mark.parametrize("residual", [False, True])
def test_layer_norm(residual):
    r = np.random.default_rng(1)
    x, gamma, beta, do = (r.standard_normal(s) for s in ((3, 8), (8,), (8,), (3, 8)))
    res, ds = (r.standard_normal((3, 8)), r.standard_normal((3, 8))) if residual else (None, None)

    def f():
        out, s = ends.layer_norm(x, gamma, beta, res)
        return float((out * do).sum() + (0 if ds is None else (s * ds).sum()))

    s = ends.layer_norm(x, gamma, beta, res)[1]
    dx, dgamma, dbeta = ends.layer_norm_backward(s, gamma, do, ds)
    assert np.allclose(dx, differences(f, x), atol=1e-8)
    assert np.allclose(dgamma, differences(f, gamma), atol=1e-8)
    assert np.allclose(dbeta, differences(f, beta), atol=1e-8)


@pytest.mark.parametrize("bias", [False, True])
def test_vocab_loss(bias):
    r = np.random.default_rng(2)
    h, W, dl = r.standard_normal((4, 8)), r.standard_normal((7, 8)), r.standard_normal(4)
    b = r.standard_normal(7) if bias else None
    t = [2, -1, 6, 0]
    f = lambda: float((ends.vocab_loss(h, W, t, b)[0] * dl).sum())  # noqa: E731
    dh, dW, db = ends.vocab_loss_backward(h, W, t, dl, b)
    assert np.allclose(dh, differences(f, h), atol=1e-8) and np.all(dh[1] == 0)
    assert np.allclose(dW, differences(f, W), atol=1e-8)
    if bias:
        assert np.allclose(db, differences(f, b), atol=1e-8)
