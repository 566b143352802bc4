"""fp64 oracle of the gated delta rule and of the group norm behind it.  TEST
INFRASTRUCTURE ONLY (numpy, no code of the CUDA library).

Per value head, with a_t = exp(g_t):
  W_t = a_t W_{t-1} + beta_t (v_t - a_t W_{t-1} k_t) k_t^T,  y_t = scale W_t q_t,
keys and queries as given or divided by sqrt(sum x^2 + eps); the gradients by
a reverse sweep over the kept states.  All arrays are numpy float64.
"""
import math

import numpy as np


def _f64(a):
    return None if a is None else np.array(a, dtype=np.float64)


def _unit(x, eps):
    s = np.sqrt((x * x).sum(-1, keepdims=True) + eps)
    return np.divide(1.0, s, out=np.zeros_like(s), where=s > 0)


def _ends(lengths, B, L):
    return [L] * B if lengths is None else [min(max(int(n), 0), L) for n in lengths]


def gated_forward(q, k, v, g, beta, W0=None, lengths=None, l2norm=True, scale=1.0, eps=1e-6, keep=None):
    """(y [B,H,L,d_v], W_final [B,H,d_v,d_k]); keep: a list that receives, per
    (b, h), the states before each token."""
    q, k, v, g, beta, W0 = (_f64(x) for x in (q, k, v, g, beta, W0))
    B, Hk, L, d_k = q.shape
    H, d_v = v.shape[1], v.shape[3]
    y = np.zeros((B, H, L, d_v))
    W = np.zeros((B, H, d_v, d_k)) if W0 is None else W0.copy()
    for b, n in enumerate(_ends(lengths, B, L)):
        for h in range(H):
            S, kept = W[b, h].copy(), []
            for t in range(n):
                kt, qt = k[b, h // (H // Hk), t], q[b, h // (H // Hk), t]
                if l2norm:
                    kt, qt = kt * _unit(kt, eps), qt * _unit(qt, eps)
                kept.append(S)
                S = math.exp(g[b, h, t]) * S
                S = S + beta[b, h, t] * np.outer(v[b, h, t] - S @ kt, kt)
                y[b, h, t] = scale * (S @ qt)
            W[b, h] = S
            if keep is not None:
                keep.append(kept)
    return y, W


def gated_backward(q, k, v, g, beta, dy, W0=None, dW=None, lengths=None, l2norm=True, scale=1.0, eps=1e-6):
    """(dq, dk, dv, dg, dbeta, dW0) of sum(y dy) + sum(W_final dW)."""
    kept = []
    gated_forward(q, k, v, g, beta, W0, lengths, l2norm, scale, eps, kept)
    q, k, v, g, beta, dy, dW = (_f64(x) for x in (q, k, v, g, beta, dy, dW))
    B, Hk, L, d_k = q.shape
    H, d_v = v.shape[1], v.shape[3]
    dq, dk, dv, dg, db = (np.zeros_like(x) for x in (q, k, v, g, beta))
    dW0 = np.zeros((B, H, d_v, d_k))
    for b, n in enumerate(_ends(lengths, B, L)):
        for h in range(H):
            j = h // (H // Hk)
            D = np.zeros((d_v, d_k)) if dW is None else dW[b, h].copy()
            for t in range(n - 1, -1, -1):
                rk = _unit(k[b, j, t], eps) if l2norm else 1.0
                rq = _unit(q[b, j, t], eps) if l2norm else 1.0
                kt, qt, a, be = rk * k[b, j, t], rq * q[b, j, t], math.exp(g[b, h, t]), beta[b, h, t]
                S = a * kept[b * H + h][t]
                e = v[b, h, t] - S @ kt
                S1 = S + be * np.outer(e, kt)
                D = D + scale * np.outer(dy[b, h, t], qt)
                gq = scale * (S1.T @ dy[b, h, t])
                du = D @ kt
                gk = D.T @ (be * e) - S.T @ (be * du)
                dv[b, h, t] = be * du
                db[b, h, t] = du @ e
                D = D - be * np.outer(du, kt)
                dg[b, h, t] = (D * S).sum()
                D = a * D
                if l2norm:
                    gq, gk = rq * (gq - qt * (qt @ gq)), rk * (gk - kt * (kt @ gk))
                dq[b, j, t] += gq
                dk[b, j, t] += gk
            dW0[b, h] = D
    return dq, dk, dv, dg, db, dW0


def _act(x, act):
    """(act(x), its derivative)."""
    if act == "relu":
        return x * (x > 0), (x > 0).astype(np.float64)
    if act == "silu":
        p = 1 / (1 + np.exp(-x))
        return x * p, p * (1 + x * (1 - p))
    if act == "gelu":
        p = 0.5 * (1 + np.vectorize(math.erf)(x / math.sqrt(2)))
        return x * p, p + x * np.exp(-x * x / 2) / math.sqrt(2 * math.pi)
    return x, np.ones_like(x)


def group_norm_act(x, gamma, beta, gate=None, act="none", eps=1e-5, dout=None):
    """out [B,L,H d], or with dout (dx, dgate or None, dgamma, dbeta)."""
    x, gamma, beta, gate, dout = (_f64(t) for t in (x, gamma, beta, gate, dout))
    B, H, L, d = x.shape
    c = x - x.mean(-1, keepdims=True)
    r = 1 / np.sqrt((c * c).mean(-1, keepdims=True) + eps)
    n = (c * r).transpose(0, 2, 1, 3)
    z = n * gamma.reshape(H, d) + beta.reshape(H, d)
    f, df = _act(z if gate is None else gate.reshape(B, L, H, d), act)
    if dout is None:
        return (f if gate is None else z * f).reshape(B, L, H * d)
    do = dout.reshape(B, L, H, d)
    dz = do * df if gate is None else do * f
    dn = dz * gamma.reshape(H, d)
    dx = r.transpose(0, 2, 1, 3) * (dn - dn.mean(-1, keepdims=True) - n * (dn * n).mean(-1, keepdims=True))
    return (dx.transpose(0, 2, 1, 3), None if gate is None else (do * z * df).reshape(B, L, H * d),
            (dz * n).sum((0, 1)).reshape(-1), dz.sum((0, 1)).reshape(-1))
