"""Planted mistakes in the oracle of the embedding, the layer norm and the
vocabulary loss must fail its tests (CPU only): each case changes one place of
its source, as a plausible slip would, and runs the tests of
test_ends_oracle.py, and values worked out by hand, against the result."""
import inspect
import math
import types

import numpy as np
import pytest

from oracle import ends
from tests import test_ends_oracle as pins

MUTANTS = {
    "embedding_unscaled": ("out[n] = scale * table[t]", "out[n] = table[t]"),
    "embedding_padding_wraps": ("if t >= 0:\n            out[n]", "if True:\n            out[n]"),
    "embedding_past_the_end_is_zero": ("else np.nan\n    return out", "else 0.0\n    return out"),
    "embedding_gradient_unscaled": ("d[t] += scale * dout[n]", "d[t] += dout[n]"),
    "embedding_gradient_keeps_the_last": ("d[t] += scale * dout[n]", "d[t] = scale * dout[n]"),
    "embedding_gradient_of_padding": ("if 0 <= t < V:\n            d[t]", "if t < V:\n            d[t]"),
    "embedding_gradient_not_added": ("if start is None else _f64(start)", "if True else _f64(start)"),
    "norm_without_residual": ("_f64(x) + _f64(residual)", "_f64(x)"),
    "norm_unbiased": ("n = c / np.sqrt((c * c).mean(-1, keepdims=True) + eps)\n    return",
                      "n = c / np.sqrt((c * c).sum(-1, keepdims=True) / (c.shape[-1] - 1) + eps)\n    return"),
    "norm_eps_outside": ("n = c / np.sqrt((c * c).mean(-1, keepdims=True) + eps)\n    return",
                         "n = c / (np.sqrt((c * c).mean(-1, keepdims=True)) + eps)\n    return"),
    "norm_without_beta": ("(0.0 if beta is None else _f64(beta))", "0.0"),
    "norm_gradient_without_mean": ("r * (g - g.mean(-1, keepdims=True) -", "r * (g -"),
    "norm_gradient_without_projection": (" - n * (g * n).mean(-1, keepdims=True))", ")"),
    "norm_gradient_without_sum": ("(dx if dsum is None else dx + _f64(dsum))", "dx"),
    "norm_dgamma_of_the_centred": ("(dout * n).sum(0)", "(dout * c).sum(0)"),
    "norm_dbeta_with_gamma": ("dout.sum(0)\n\n\ndef vocab_loss", "g.sum(0)\n\n\ndef vocab_loss"),
    "loss_without_bias": ("W @ h[n] + (0.0 if bias is None else _f64(bias))", "W @ h[n]"),
    "loss_without_top": ("lse[n] = top + np.log(np.exp(z - top).sum())", "lse[n] = np.log(np.exp(z).sum())"),
    "loss_of_padding": ("if t < 0:\n            continue\n        z", "z"),
    "loss_sign": ("loss[n] = lse[n] - z[t]", "loss[n] = z[t] - lse[n]"),
    "loss_gradient_target_kept": ("g[n, targets[n]] -= 1", "g[n, targets[n]] -= 0"),
    "loss_gradient_unweighted": ("g[n] *= dloss[n]", "g[n] *= 1"),
    "loss_gradient_of_dbias_softmax": ("g.sum(0)", "p.sum(0)"),
    "loss_gradient_dW_of_all": ("g[live].T @ h[live]", "p.T @ h"),
}


def by_hand(m):
    out = m.embedding([1, -1, 0, 2], np.array([[1.0, 2.0], [3.0, 4.0]]), 2.0)
    assert np.array_equal(out[:3], [[6, 8], [0, 0], [2, 4]]) and np.isnan(out[3]).all()
    d = m.embedding_backward([1, -1, 1, 2], np.array([[1.0, 2.0], [9.0, 9.0], [3.0, 4.0], [9.0, 9.0]]), 2, 2.0,
                             np.array([[1.0, 1.0], [1.0, 1.0]]))
    assert np.array_equal(d, [[1, 1], [9, 13]])
    out, s = m.layer_norm([[1.0, 3.0]], [2.0, 2.0], [5.0, 5.0], [[1.0, 1.0]], eps=3.0)  # deviations of 1, root of 1 + 3
    assert np.array_equal(s, [[2, 4]]) and np.allclose(out, [[4, 6]], atol=1e-12)
    h, W = np.zeros((2, 3)), np.ones((4, 3))
    loss, lse, p = m.vocab_loss(h, W, [3, -1], np.log([1.0, 2.0, 3.0, 4.0]) + 800)
    assert np.allclose(loss, [math.log(2.5), 0], atol=1e-12) and np.allclose(lse, [math.log(10) + 800, 0], atol=1e-9)
    assert np.allclose(p, [[0.1, 0.2, 0.3, 0.4], [0, 0, 0, 0]], atol=1e-12)


def run_pins(m, monkeypatch):
    monkeypatch.setattr(pins, "ends", m)
    by_hand(m)
    pins.test_embedding()
    for flag in (False, True):
        pins.test_layer_norm(flag)
        pins.test_vocab_loss(flag)


def test_the_oracle_itself(monkeypatch):
    run_pins(ends, monkeypatch)


@pytest.mark.parametrize("name", MUTANTS)
def test_a_mistake_is_seen(name, monkeypatch):
    source, (old, new) = inspect.getsource(ends), MUTANTS[name]
    assert old in source, f"{name}: the oracle no longer reads so"
    mutant = types.ModuleType("mutant")
    exec(source.replace(old, new, 1), mutant.__dict__)
    with np.errstate(all="ignore"), pytest.raises((AssertionError, IndexError)):
        run_pins(mutant, monkeypatch)
