"""Cases for the gated delta rule and the group norm that follows it.

A fast-weight layer with a forget gate answers a token with a state that
first decays, then takes the delta rule's correction:

    W_t = a_t W_{t-1} + beta_t (v_t - a_t W_{t-1} k_t) k_t^T,   a_t = exp(g_t)
    y_t = scale W_t q_t

and normalises each head's answer, with a gate, on its way to the output map.
Five calls: the sequence (`forward`), its gradients (`backward`), one token
against a kept state (`decode`), the norm (`norm`) and its gradients
(`norm_backward`).  `run` computes each in plain torch where `own` is false
and through the library where it is true; `exact` computes the definitions,
token by token, in 64 bits.
"""
import math

import torch

own = False

L2_EPS = 1e-6     # inside the root of the keys' and queries' norm
NORM_EPS = 1e-5   # inside the root of the group norm
G_MIN = -200.0    # exp() of it is 0 in 32 bits: a gate of -inf is one that forgets everything
CHUNK = 64
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # a short prompt of three requests padded to the longest, no state yet
        dict(name="forward_b3h8_l130_padded", op="forward", B=3, Hk=8, H=8, L=130, d_k=64, d_v=64, io="bf16", keys="l2",
             state=False, padded=True),
        # the layer's benchmark length, keys and queries mapped by DPFP (d_key 64, nu 1), memory passed in and on
        dict(name="forward_b2h8_l2048_dpfp", op="forward", B=2, Hk=8, H=8, L=2048, d_k=128, d_v=64, io="bf16",
             keys="dpfp", state=True, padded=False),
        # one long document, two value heads to a key head, an odd length
        dict(name="forward_b1h16_l16381_shared", op="forward", B=1, Hk=8, H=16, L=16381, d_k=128, d_v=128, io="bf16",
             keys="l2", state=True, padded=False),
        # 32-bit tensors: what a numerical check of a model runs
        dict(name="forward_b1h4_l333_f32", op="forward", B=1, Hk=4, H=4, L=333, d_k=64, d_v=48, io="f32", keys="l2",
             state=True, padded=False),
        # a training step's backward at the benchmark's small shape
        dict(name="backward_b4h8_l512", op="backward", B=4, Hk=8, H=8, L=512, d_k=64, d_v=64, io="bf16", keys="l2",
             state=False, padded=False),
        # the same at a full training shape: shared key heads, a state carried between segments, ragged rows
        dict(name="backward_b8h16_l2048_shared", op="backward", B=8, Hk=8, H=16, L=2048, d_k=128, d_v=128, io="bf16",
             keys="l2", state=True, padded=True),
        # one user's next token: latency
        dict(name="decode_b1h8", op="decode", B=1, Hk=8, H=8, L=1, d_k=64, d_v=64, io="bf16", keys="l2"),
        # a full serving batch's next token: 268 MB of state read and written
        dict(name="decode_b256h16_shared", op="decode", B=256, Hk=8, H=16, L=1, d_k=128, d_v=128, io="bf16", keys="l2"),
        # the norm of one decoded token, and of a training batch
        dict(name="norm_b1h8_l1", op="norm", B=1, H=8, L=1, d=64, io="bf16", act="silu", gate=True),
        dict(name="norm_b16h8_l2048", op="norm", B=16, H=8, L=2048, d=128, io="bf16", act="silu", gate=True),
        # its gradients: a small odd batch in 32 bits without a gate, and the training batch
        dict(name="norm_backward_b3h5_l211_f32", op="norm_backward", B=3, H=5, L=211, d=48, io="f32", act="gelu",
             gate=False),
        dict(name="norm_backward_b16h8_l2048", op="norm_backward", B=16, H=8, L=2048, d=128, io="bf16", act="silu",
             gate=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["forward", "backward", "decode", "norm", "norm_backward"])
    io = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op in ("norm", "norm_backward"):
        B, H, d = _log_int(rng, 1, 16), rng.choice([1, 3, 4, 5, 8, 16]), rng.choice([8, 24, 32, 48, 64, 96, 128, 256])
        most = min(4096, (16 * 8 * 2048 * 128 if io == "bf16" else 8 * 8 * 2048 * 128) // (B * H * d))
        return dict(op=op, B=B, H=H, L=_log_int(rng, 1, max(1, most)), d=d, io=io,
                    act=rng.choice(["none", "relu", "silu", "gelu"]), gate=rng.random() < 0.6)
    Hk = rng.choice([1, 2, 4, 8])
    H = Hk * rng.choice([1, 1, 2, 3])
    d_k, d_v = rng.choice([16, 32, 64, 128]), rng.choice([16, 32, 48, 64, 96, 128])
    keys = "l2" if rng.random() < 0.7 else "dpfp"
    if op == "decode":
        return dict(op=op, B=_log_int(rng, 1, 4096 // max(H, 16)), Hk=Hk, H=H, L=1, d_k=d_k, d_v=d_v, io=io, keys=keys)
    B = _log_int(rng, 1, 8)
    most = (16 * 16381 if op == "forward" else 8 * 16 * 2048) // (B * H) // (1 if io == "bf16" else 16)
    return dict(op=op, B=B, Hk=Hk, H=H, L=_log_int(rng, 1, max(1, min(most, 16381 if op == "forward" else 2048))), d_k=d_k,
                d_v=d_v, io=io, keys=keys, state=rng.random() < 0.5, padded=rng.random() < 0.4)


# --------------------------------------------------------------- the inputs
def _dpfp(x):
    """DPFP with one roll: twice the width, non-negative, entries summing to 1."""
    r = torch.relu(torch.cat([x, -x], -1))
    p = r * torch.roll(r, 1, -1)
    return p / (p.sum(-1, keepdim=True) + 1e-6)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = DTYPES[case["io"]]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)

    s = dict(case)
    if case["op"] in ("norm", "norm_backward"):
        B, H, L, d = (case[n] for n in ("B", "H", "L", "d"))
        s["x"] = (0.5 * randn(B, H, L, d) + 0.1 * randn(H, 1, 1)).to(dt)
        s["gate"] = randn(B, L, H * d).to(dt) if case["gate"] else None
        s["gamma"] = 1 + 0.1 * randn(H * d)
        s["beta"] = 0.1 * randn(H * d)
        if case["op"] == "norm_backward":
            s["dout"] = randn(B, L, H * d).to(dt)
        return s
    B, Hk, H, L, d_k, d_v = (case[n] for n in ("B", "Hk", "H", "L", "d_k", "d_v"))
    t = () if case["op"] == "decode" else (L,)
    for n in ("q", "k"):
        x = randn(B, Hk, *t, d_k // 2 if case["keys"] == "dpfp" else d_k)
        s[n] = (_dpfp(x) if case["keys"] == "dpfp" else x).to(dt)
    s["v"] = randn(B, H, *t, d_v).to(dt)
    # each head forgets at a rate of its own, from a few tokens to a few thousand, moved by the token
    rate = torch.exp(-6.0 * torch.rand(H, *([1] * len(t)), generator=gen, device="cuda"))
    s["g"] = (-rate * torch.nn.functional.softplus(randn(B, H, *t))).to(dt)
    s["beta"] = torch.sigmoid(randn(B, H, *t)).to(dt)
    s["l2norm"] = case["keys"] == "l2"
    s["scale"] = d_k ** -0.5 if s["l2norm"] else 1.0
    if case["op"] == "decode":
        s["W"] = 0.3 * randn(B, H, d_v, d_k)
        return s
    s["W0"] = 0.3 * randn(B, H, d_v, d_k) if case["state"] else None
    s["lengths"] = None
    if case["padded"]:
        lens = torch.randint(L // 2, L + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
        lens[0] = L
        s["lengths"] = lens
    if case["op"] == "backward":
        s["dy"] = randn(B, H, L, d_v).to(dt)
        s["dW"] = 0.1 * randn(B, H, d_v, d_k) if case["state"] else None
    return s


# ------------------------------------------------------------ the plain form
def _unit(x):
    return x * torch.rsqrt((x * x).sum(-1, keepdim=True) + L2_EPS)


def _unit_lower_inverse(A):
    """(I + A)^-1 of strictly lower triangular A, by halves."""
    n = A.shape[-1]
    if n == 1:
        return torch.ones_like(A)
    h = n // 2
    a, b = _unit_lower_inverse(torch.stack([A[..., :h, :h], A[..., h:, h:]])).unbind(0)
    low = -(b @ A[..., h:, :h] @ a)
    return torch.cat([torch.cat([a, torch.zeros_like(a)], -1), torch.cat([low, b], -1)], -2)


def _plain_sequence(q, k, v, g, beta, W0, lengths, l2norm, scale):
    """(y, W_final) of 32-bit tensors, in chunks of 64 tokens."""
    B, Hk, L, d_k = q.shape
    H, d_v = v.shape[1], v.shape[-1]
    if lengths is not None:
        there = (torch.arange(L, device=q.device) < lengths[:, None])[:, None]
        zero = torch.zeros((), device=q.device)
        q, k, v = (torch.where(there[..., None], x, zero) for x in (q, k, v))
        g, beta = (torch.where(there, x, zero) for x in (g, beta))
    if l2norm:
        q, k = _unit(q), _unit(k)
    q, k = (x.repeat_interleave(H // Hk, 1) for x in (q, k))
    n = -(-L // CHUNK)
    pad = n * CHUNK - L
    q, k, v = (torch.nn.functional.pad(x, (0, 0, 0, pad)).reshape(B, H, n, CHUNK, -1) for x in (q, k, v))
    g, beta = (torch.nn.functional.pad(x, (0, pad)).reshape(B, H, n, CHUNK) for x in (g, beta))
    G = g.clamp(min=G_MIN).double().cumsum(-1)  # differences of long sums: 64 bits
    seen = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=q.device).tril()
    decay = torch.exp(torch.where(seen, G[..., :, None] - G[..., None, :], -math.inf)).float()
    M = (scale * q @ k.transpose(-1, -2)) * decay
    T = _unit_lower_inverse((beta[..., None] * (k @ k.transpose(-1, -2)) * decay).tril(-1))
    since, until = torch.exp(G).float()[..., None], torch.exp(G[..., -1:] - G).float()[..., None]
    whole = torch.exp(G[..., -1]).float()[..., None, None]
    W = torch.zeros(B, H, d_v, d_k, device=q.device) if W0 is None else W0
    ys = []
    for c in range(n):
        Wt = W.transpose(-1, -2)
        u = T[:, :, c] @ (beta[:, :, c, :, None] * (v[:, :, c] - since[:, :, c] * (k[:, :, c] @ Wt)))
        ys.append(scale * since[:, :, c] * (q[:, :, c] @ Wt) + M[:, :, c] @ u)
        W = whole[:, :, c] * W + (until[:, :, c] * u).transpose(-1, -2) @ k[:, :, c]
    y = torch.cat(ys, 2)[:, :, :L]
    return (y if lengths is None else torch.where(there[..., None], y, torch.zeros((), device=y.device))), W


def _plain_act(x, act):
    if act == "relu":
        return torch.relu(x)
    if act == "silu":
        return x * torch.sigmoid(x)
    if act == "gelu":
        return 0.5 * x * (1 + torch.erf(x * 0.5 ** 0.5))
    return x


def _plain_norm(x, gate, gamma, beta, act):
    """[B, H, L, d] -> [B, L, H d]: each head's channels normalised for each token."""
    B, H, L, d = x.shape
    c = x - x.mean(-1, keepdim=True)
    n = c * torch.rsqrt((c * c).mean(-1, keepdim=True) + NORM_EPS)
    z = n.transpose(1, 2).reshape(B, L, H * d) * gamma + beta
    return _plain_act(z, act) if gate is None else z * _plain_act(gate, act)


def _wide(*xs):
    return [None if x is None else x.float() for x in xs]


def _leaves(xs):
    return [None if x is None else x.detach().float().requires_grad_() for x in xs]


def _gradients(outs, grads, leaves, like):
    pairs = [(o, d.float()) for o, d in zip(outs, grads) if d is not None]
    got = torch.autograd.grad([o for o, _ in pairs], [x for x in leaves if x is not None], [d for _, d in pairs])
    it = iter(got)
    return [None if x is None else next(it).to(t.dtype) for x, t in zip(leaves, like)]


def _run_plain(s):
    dt = DTYPES[s["io"]]
    if s["op"] == "norm":
        return {"out": _plain_norm(*_wide(s["x"], s["gate"], s["gamma"], s["beta"]), s["act"]).to(dt)}
    if s["op"] == "norm_backward":
        like = [s["x"], s["gate"], s["gamma"], s["beta"]]
        ls = _leaves(like)
        got = _gradients([_plain_norm(*ls, s["act"])], [s["dout"]], ls, like)
        return dict(zip(("dx", "dgate", "dgamma", "dbeta"), got))
    if s["op"] == "decode":
        q, k, v, g, beta = _wide(s["q"], s["k"], s["v"], s["g"], s["beta"])
        if s["l2norm"]:
            q, k = _unit(q), _unit(k)
        q, k = (x.repeat_interleave(s["H"] // s["Hk"], 1) for x in (q, k))
        W = torch.exp(g)[..., None, None] * s["W"]
        u = beta[..., None] * (v - (W @ k[..., None])[..., 0])
        W = W + u[..., :, None] * k[..., None, :]
        s["W"].copy_(W)
        return {"y": (s["scale"] * (W @ q[..., None])[..., 0]).to(dt), "W": s["W"]}
    if s["op"] == "forward":
        y, W = _plain_sequence(*_wide(s["q"], s["k"], s["v"], s["g"], s["beta"], s["W0"]), s["lengths"], s["l2norm"],
                               s["scale"])
        return {"y": y.to(dt), "W_final": W}
    like = [s["q"], s["k"], s["v"], s["g"], s["beta"], s["W0"]]
    ls = _leaves(like)
    outs = _plain_sequence(*ls, s["lengths"], s["l2norm"], s["scale"])
    got = _gradients(outs, [s["dy"], s["dW"]], ls, like)
    return dict(zip(("dq", "dk", "dv", "dg", "dbeta", "dW0"), got))


def _run_own(s):
    from delta_rule_linear_dpfp_gb300 import binding as fw
    if s["op"] == "norm":
        return {"out": fw.fw_group_norm_act(s["x"], s["gamma"], s["beta"], gate=s["gate"], act=s["act"], eps=NORM_EPS)}
    if s["op"] == "norm_backward":
        got = fw.fw_group_norm_act_backward(s["x"], s["gamma"], s["beta"], s["dout"], gate=s["gate"], act=s["act"],
                                            eps=NORM_EPS)
        return dict(zip(("dx", "dgate", "dgamma", "dbeta"), got))
    if s["op"] == "decode":
        y = fw.fw_gated_delta_decode_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["W"], l2norm=s["l2norm"],
                                          scale=s["scale"], eps=L2_EPS)
        return {"y": y, "W": s["W"]}
    if s["op"] == "forward":
        y, W = fw.fw_gated_delta_forward(s["q"], s["k"], s["v"], s["g"], s["beta"], W0=s["W0"], lengths=s["lengths"],
                                         l2norm=s["l2norm"], scale=s["scale"], eps=L2_EPS)
        return {"y": y, "W_final": W}
    got = fw.fw_gated_delta_backward(s["q"], s["k"], s["v"], s["g"], s["beta"], s["dy"], W0=s["W0"], dW_final=s["dW"],
                                     lengths=s["lengths"], l2norm=s["l2norm"], scale=s["scale"], eps=L2_EPS,
                                     return_dW0=s["W0"] is not None)
    return dict(zip(("dq", "dk", "dv", "dg", "dbeta", "dW0"), got))


def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


# ------------------------------------------------------ what it cannot do without
def work(case):
    e = 2 if case["io"] == "bf16" else 4
    if case["op"] in ("norm", "norm_backward"):
        n, C = case["B"] * case["H"] * case["L"] * case["d"], case["H"] * case["d"]
        gate = n if case["gate"] else 0
        if case["op"] == "norm":
            return {"bytes": e * (2 * n + gate) + 8 * C, "flops": 12 * n}
        return {"bytes": e * (3 * n + 2 * gate) + 16 * C, "flops": 30 * n}
    B, Hk, H, L, d_k, d_v = (case[n] for n in ("B", "Hk", "H", "L", "d_k", "d_v"))
    keys, values, gates, state = 2 * B * Hk * L * d_k, B * H * L * d_v, 2 * B * H * L, 4 * B * H * d_v * d_k
    steps = B * H * L * d_k * d_v
    if case["op"] == "decode":
        return {"bytes": e * (keys + 2 * values + gates) + 2 * state, "flops": 7 * steps}
    s0 = state if case["state"] else 0
    if case["op"] == "forward":
        return {"bytes": e * (keys + 2 * values + gates) + s0 + state, "flops": 6 * steps}
    return {"bytes": e * (2 * keys + 3 * values + 2 * gates) + 3 * s0, "flops": 16 * steps}


# ------------------------------------------------------------------- 64 bits
def _exact_norm(s):
    x, gate, gamma, beta = (None if t is None else t.double() for t in (s["x"], s["gate"], s["gamma"], s["beta"]))
    B, H, L, d = x.shape
    x = x.permute(0, 2, 1, 3)
    mean = x.sum(-1, keepdim=True) / d
    var = ((x - mean) ** 2).sum(-1, keepdim=True) / d
    r = 1 / torch.sqrt(var + NORM_EPS)
    n = (x - mean) * r
    z = n * gamma.view(H, d) + beta.view(H, d)
    t = z if gate is None else gate.view(B, L, H, d)
    if s["act"] == "relu":
        f, df = t * (t > 0), (t > 0).double()
    elif s["act"] == "silu":
        p = 1 / (1 + torch.exp(-t))
        f, df = t * p, p * (1 + t * (1 - p))
    elif s["act"] == "gelu":
        p = 0.5 * torch.erfc(-t / math.sqrt(2.0))
        f, df = t * p, p + t * torch.exp(-t * t / 2) / math.sqrt(2 * math.pi)
    else:
        f, df = t, torch.ones_like(t)
    if s["op"] == "norm":
        return {"out": (f if gate is None else z * f).reshape(B, L, H * d)}
    do = s["dout"].double().view(B, L, H, d)
    dz, dgate = (do * df, None) if gate is None else (do * f, (do * z * df).reshape(B, L, H * d))
    dn = dz * gamma.view(H, d)
    dx = r * (dn - dn.sum(-1, keepdim=True) / d - n * (dn * n).sum(-1, keepdim=True) / d)
    return {"dx": dx.permute(0, 2, 1, 3), "dgate": dgate, "dgamma": (dz * n).sum((0, 1)).reshape(-1),
            "dbeta": dz.sum((0, 1)).reshape(-1)}


def _exact_rows(q, k, v, g, beta, W, scale, dy=None, dW=None):
    """The recurrence over rows of heads: q, k [N, L, d_k], v [N, L, d_v], g, beta [N, L], W [N, d_v, d_k]."""
    L = q.shape[1]
    a = torch.exp(g)
    ys, kept = [], []
    for t in range(L):
        if dy is not None:
            kept.append(W)
        W = a[:, t, None, None] * W
        e = v[:, t] - torch.einsum("nij,nj->ni", W, k[:, t])
        W = W + torch.einsum("ni,nj->nij", beta[:, t, None] * e, k[:, t])
        if dy is None:
            ys.append(scale * torch.einsum("nij,nj->ni", W, q[:, t]))
    if dy is None:
        return torch.stack(ys, 1), W
    D = torch.zeros_like(W) if dW is None else dW
    grads = [torch.zeros_like(x) for x in (q, k, v, g, beta)]
    for t in range(L - 1, -1, -1):
        before = a[:, t, None, None] * kept[t]
        e = v[:, t] - torch.einsum("nij,nj->ni", before, k[:, t])
        after = before + torch.einsum("ni,nj->nij", beta[:, t, None] * e, k[:, t])
        D = D + scale * torch.einsum("ni,nj->nij", dy[:, t], q[:, t])
        grads[0][:, t] = scale * torch.einsum("nij,ni->nj", after, dy[:, t])
        Dk = torch.einsum("nij,nj->ni", D, k[:, t])
        de = beta[:, t, None] * Dk
        grads[1][:, t] = torch.einsum("nij,ni->nj", D, beta[:, t, None] * e) - torch.einsum("nij,ni->nj", before, de)
        grads[2][:, t] = de
        grads[4][:, t] = (Dk * e).sum(-1)
        D = D - torch.einsum("ni,nj->nij", de, k[:, t])
        grads[3][:, t] = (D * before).sum((1, 2))
        D = a[:, t, None, None] * D
    return (*grads, D)


def _exact_delta(s):
    decode, B, Hk, H = s["op"] == "decode", s["B"], s["Hk"], s["H"]
    q, k, v, g, beta = (s[n].double() for n in ("q", "k", "v", "g", "beta"))
    if decode:
        q, k, v, g, beta = q[:, :, None], k[:, :, None], v[:, :, None], g[:, :, None], beta[:, :, None]
    L, d_k, d_v = q.shape[2], q.shape[3], v.shape[3]
    W0 = s["W"] if decode else s["W0"]
    W0 = torch.zeros(B, H, d_v, d_k, dtype=torch.float64, device=q.device) if W0 is None else W0.double()
    lens = None if decode or s["lengths"] is None else s["lengths"].tolist()
    if lens is not None:
        for b, n in enumerate(lens):
            for x in (q, k, v, g, beta):
                x[b, :, n:] = 0
    if s["l2norm"]:
        rq, rk = (1 / torch.sqrt((x * x).sum(-1, keepdim=True) + L2_EPS) for x in (q, k))
    else:
        rq = rk = torch.ones((), dtype=torch.float64, device=q.device)
    qn, kn = q * rq, k * rk
    qs, ks = (x.repeat_interleave(H // Hk, 1).reshape(B * H, L, d_k) for x in (qn, kn))
    vs, gs, bs, Ws = v.reshape(B * H, L, d_v), g.reshape(B * H, L), beta.reshape(B * H, L), W0.reshape(B * H, d_v, d_k)
    if s["op"] != "backward":
        y, W = _exact_rows(qs, ks, vs, gs, bs, Ws, s["scale"])
        y = y.reshape(B, H, L, d_v)
        if lens is not None:
            for b, n in enumerate(lens):
                y[b, :, n:] = 0
        W = W.reshape(B, H, d_v, d_k)
        return {"y": y[:, :, 0], "W": W} if decode else {"y": y, "W_final": W}
    dy = s["dy"].double()
    if lens is not None:
        for b, n in enumerate(lens):
            dy[b, :, n:] = 0
    dy = dy.reshape(B * H, L, d_v)
    dW = None if s["dW"] is None else s["dW"].double().reshape(B * H, d_v, d_k)
    step = max(1, int(20e9 // (8 * L * d_k * d_v)))  # heads at a time: every token's state is kept
    parts = [_exact_rows(qs[i:i + step], ks[i:i + step], vs[i:i + step], gs[i:i + step], bs[i:i + step], Ws[i:i + step],
                         s["scale"], dy[i:i + step], None if dW is None else dW[i:i + step])
             for i in range(0, B * H, step)]
    dq, dk, dv, dg, db, dW0 = (torch.cat(p) for p in zip(*parts))
    dq, dk = (x.reshape(B, Hk, H // Hk, L, d_k).sum(2) for x in (dq, dk))
    if s["l2norm"]:
        dq = rq * (dq - qn * (qn * dq).sum(-1, keepdim=True))
        dk = rk * (dk - kn * (kn * dk).sum(-1, keepdim=True))
    out = {"dq": dq, "dk": dk, "dv": dv.reshape(B, H, L, d_v), "dg": dg.reshape(B, H, L), "dbeta": db.reshape(B, H, L)}
    if lens is not None:
        for b, n in enumerate(lens):
            for x in out.values():
                x[b, :, n:] = 0
    out["dW0"] = dW0.reshape(B, H, d_v, d_k) if s["W0"] is not None else None
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_norm(s) if case["op"] in ("norm", "norm_backward") else _exact_delta(s)
