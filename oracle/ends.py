"""fp64 oracle of a model's two ends and the norm between its parts: the
embedding, the layer norm and the vocabulary loss, with their gradients.  TEST
INFRASTRUCTURE ONLY (numpy, no code of the CUDA library).

Negative tokens are padding; tokens at or past V give NaN and no gradient.
"""
import numpy as np


def _f64(a):
    return None if a is None else np.array(a, dtype=np.float64)


def embedding(ids, table, scale=1.0):
    table = _f64(table)
    out = np.zeros((len(ids), table.shape[1]))
    for n, t in enumerate(ids):
        if t >= 0:
            out[n] = scale * table[t] if t < len(table) else np.nan
    return out


def embedding_backward(ids, dout, V, scale=1.0, start=None):
    dout = _f64(dout)
    d = np.zeros((V, dout.shape[1])) if start is None else _f64(start)
    for n, t in enumerate(ids):
        if 0 <= t < V:
            d[t] += scale * dout[n]
    return d


def layer_norm(x, gamma=None, beta=None, residual=None, eps=1e-5):
    """(out, x + residual)."""
    s = _f64(x) if residual is None else _f64(x) + _f64(residual)
    c = s - s.mean(-1, keepdims=True)
    n = c / np.sqrt((c * c).mean(-1, keepdims=True) + eps)
    return n * (1.0 if gamma is None else _f64(gamma)) + (0.0 if beta is None else _f64(beta)), s


def layer_norm_backward(s, gamma, dout, dsum=None, eps=1e-5):
    """(dx, dgamma, dbeta)."""
    s, dout = _f64(s), _f64(dout)
    c = s - s.mean(-1, keepdims=True)
    r = 1 / np.sqrt((c * c).mean(-1, keepdims=True) + eps)
    n = c * r
    g = dout if gamma is None else dout * _f64(gamma)
    dx = r * (g - g.mean(-1, keepdims=True) - n * (g * n).mean(-1, keepdims=True))
    return (dx if dsum is None else dx + _f64(dsum)), (dout * n).sum(0), dout.sum(0)


def vocab_loss(h, W, targets, bias=None):
    """(loss, lse, softmax [N, V] with zero rows for padding)."""
    h, W = _f64(h), _f64(W)
    N, V = len(h), len(W)
    loss, lse, p = np.zeros(N), np.zeros(N), np.zeros((N, V))
    for n, t in enumerate(targets):
        if t < 0:
            continue
        z = W @ h[n] + (0.0 if bias is None else _f64(bias))
        top = z.max()
        lse[n] = top + np.log(np.exp(z - top).sum())
        p[n] = np.exp(z - lse[n])
        loss[n] = lse[n] - z[t] if t < V else np.nan
    return loss, lse, p


def vocab_loss_backward(h, W, targets, dloss, bias=None):
    """(dh, dW, dbias) of sum(dloss loss)."""
    h, W, dloss = _f64(h), _f64(W), _f64(dloss)
    _, _, p = vocab_loss(h, W, targets, bias)
    g = np.zeros_like(p)
    live = [n for n, t in enumerate(targets) if 0 <= t < len(W)]
    for n in live:
        g[n] = p[n]
        g[n, targets[n]] -= 1
        g[n] *= dloss[n]
    return g @ W, g[live].T @ h[live], g.sum(0)
