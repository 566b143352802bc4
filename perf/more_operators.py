"""Cases for the two ends of a fast-weight language model, and the norm between its parts.

    e_n = scale E[id_n]                                       (`embedding`)
    s = x + residual,  o = (s - mean(s)) / sqrt(var(s) + eps) gamma + beta   (`layer_norm`)
    z_n = W h_n + b,  loss_n = log sum_v exp(z_nv) - z_n,target_n            (`vocab_loss`)

and the gradients of the three (`..._backward`).  A negative id or target is
padding: a row of zeros, a loss of zero, no gradient, whatever the row holds.
`run` computes each in plain torch where `own` is false and through the
library where it is true; `exact` computes the definitions in 64 bits.
"""
import math

import torch

own = False

NORM_EPS = 1e-5   # inside the root of the norm
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # the next token of a serving batch of 256 sequences, scaled by the root of the width
        dict(name="embedding_n256_d512", op="embedding", N=256, V=32000, D=512, io="bf16", scaled=True, padded=False),
        # a training batch of padded rows
        dict(name="embedding_n32768_d1024", op="embedding", N=32768, V=50001, D=1024, io="bf16", scaled=False, padded=True),
        # 16 sequences of 128 characters: every row of the table is met many times
        dict(name="embedding_backward_n2048_v65_d512_f32", op="embedding_backward", N=2048, V=65, D=512, io="f32", scaled=True,
             padded=False),
        # words: a few are met all the time, most of the table never
        dict(name="embedding_backward_n16384_v50001_d1024", op="embedding_backward", N=16384, V=50001, D=1024, io="bf16",
             scaled=True, padded=True),
        # one decoded token's residual stream and its norm: latency
        dict(name="layer_norm_n1_d512", op="layer_norm", N=1, D=512, io="bf16", residual=True),
        # a training batch's
        dict(name="layer_norm_n32768_d1024", op="layer_norm", N=32768, D=1024, io="bf16", residual=True),
        # gradients in 32 bits, as a check of a model runs them: odd sizes, no residual
        dict(name="layer_norm_backward_n777_d1000_f32", op="layer_norm_backward", N=777, D=1000, io="f32", residual=False),
        # a training batch's gradients, the residual stream's own joining them
        dict(name="layer_norm_backward_n16384_d2048", op="layer_norm_backward", N=16384, D=2048, io="bf16", residual=True),
        # how likely one token is: latency, and the whole vocabulary to read
        dict(name="vocab_loss_n1_v32000_d512", op="vocab_loss", N=1, V=32000, D=512, bias=False, padded=False, weighted=False),
        # a training batch's losses over a vocabulary of words
        dict(name="vocab_loss_n8192_v50001_d1024", op="vocab_loss", N=8192, V=50001, D=1024, bias=False, padded=True,
             weighted=False),
        # the character model: 16 sequences of 128, 65 characters, an output map with a bias
        dict(name="vocab_loss_backward_n2048_v65_d512", op="vocab_loss_backward", N=2048, V=65, D=512, bias=True, padded=False,
             weighted=False),
        # a training batch's gradients over a vocabulary of words
        dict(name="vocab_loss_backward_n8192_v50001_d2048", op="vocab_loss_backward", N=8192, V=50001, D=2048, bias=False,
             padded=True, weighted=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["embedding", "embedding_backward", "layer_norm", "layer_norm_backward", "vocab_loss",
                     "vocab_loss_backward"])
    io = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("layer_norm"):
        D = 8 * _log_int(rng, 1, 1024)
        most = (32768 * 1024 if op == "layer_norm" else 16384 * 2048) // D // (1 if io == "bf16" else 2)
        return dict(op=op, N=_log_int(rng, 1, max(1, min(65536, most))), D=D, io=io, residual=rng.random() < 0.6)
    if op.startswith("embedding"):
        D = 8 * _log_int(rng, 1, 512)
        V = _log_int(rng, 33, min(65536, 50001 * 1024 // D))
        most = (32768 * 1024 if op == "embedding" else 16384 * 1024) // D // (1 if io == "bf16" else 2)
        return dict(op=op, N=_log_int(rng, 1, max(1, min(65536, most))), V=V, D=D, io=io, scaled=rng.random() < 0.6,
                    padded=rng.random() < 0.5)
    D = 8 * _log_int(rng, 2, 256)
    V = _log_int(rng, 33, 65536)
    most = (8192 * 50001 * 1024 * (1 if op == "vocab_loss" else 2)) // (V * D)
    return dict(op=op, N=_log_int(rng, 1, max(1, min(8192, most))), V=V, D=D, bias=rng.random() < 0.5,
                padded=rng.random() < 0.5, weighted=rng.random() < 0.3)


# --------------------------------------------------------------- the inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)

    def rand(*shape):
        return torch.rand(*shape, generator=gen, device="cuda", dtype=torch.float32)

    def tokens(N, V):
        """Tokens as a tokenizer orders them, the frequent ones first: the r-th with a probability of about 1 / r."""
        return torch.exp(rand(N).double() * math.log(V + 1.0)).long().sub_(1).clamp_(0, V - 1)

    s, op, N, D = dict(case), case["op"], case["N"], case["D"]
    there = rand(N) < 0.9 if case.get("padded") else None  # a tenth of a padded batch is padding
    if op.startswith("layer_norm"):
        dt = DTYPES[case["io"]]
        s["x"] = (randn(N, D) + 0.5 * randn(N, 1)).to(dt)
        s["gamma"], s["beta"] = 1 + 0.1 * randn(D), 0.1 * randn(D)
        s["other"] = randn(N, D).to(dt) if case["residual"] else None  # the residual stream, or its gradient
        if op == "layer_norm_backward":
            s["dout"] = randn(N, D).to(dt)
        return s
    V = case["V"]
    ids = tokens(N, V)
    if op.startswith("embedding"):
        dt = DTYPES[case["io"]]
        s["scale"] = math.sqrt(D) if case["scaled"] else 1.0
        s["ids"] = ids if there is None else torch.where(there, ids, -1)
        if op == "embedding":
            s["table"] = (randn(V, D) * D ** -0.5).to(dt)
        else:
            s["dout"] = (1e-2 * randn(N, D)).to(dt)
        return s
    # an output map of unit rows, and answers that know some of their tokens well and others not at all
    s["W"] = (randn(V, D) * D ** -0.5).bfloat16()
    s["h"] = (randn(N, D) + 12 * rand(N, 1) * s["W"][ids]).bfloat16()
    s["bias"] = 0.1 * randn(V) if case["bias"] else None
    s["targets"] = ids if there is None else torch.where(there, ids, -1)
    if op == "vocab_loss_backward":
        z = s["h"].float() @ s["W"].float().T
        if s["bias"] is not None:
            z += s["bias"]
        lse = torch.logsumexp(z, -1)
        live = s["targets"] >= 0
        # what the forward pass has left
        s["loss"] = torch.where(live, lse - z.gather(1, ids[:, None])[:, 0], 0.0)
        s["lse"] = torch.where(live, lse, 0.0)
        weights = live.float() if not case["weighted"] else live * rand(N)
        s["dloss"] = weights / live.sum().clamp(min=1)  # the mean over the batch's tokens
    return s


# ------------------------------------------------------------ the plain form
def _plain_logits(s):
    z = s["h"].float() @ s["W"].float().T
    return z if s["bias"] is None else z.add_(s["bias"])


def _run_plain(s):
    op = s["op"]
    if op == "embedding":
        rows = s["table"][s["ids"].clamp(min=0)].float() * s["scale"]
        return {"out": torch.where(s["ids"][:, None] >= 0, rows, 0.0).to(s["table"].dtype)}
    if op == "embedding_backward":
        V, D = s["V"], s["D"]
        at = torch.where(s["ids"] >= 0, s["ids"], V)  # padding goes to a row behind the table
        total = torch.zeros(V + 1, D, device=at.device).index_add_(0, at, s["dout"].float())
        return {"dtable": (total[:V] * s["scale"]).to(s["dout"].dtype)}
    if op == "layer_norm":
        x = s["x"].float()
        if s["other"] is not None:
            x = x + s["other"].float()
        c = x - x.mean(-1, keepdim=True)
        n = c * torch.rsqrt((c * c).mean(-1, keepdim=True) + NORM_EPS)
        out = (n * s["gamma"] + s["beta"]).to(s["x"].dtype)
        return {"out": out} if s["other"] is None else {"out": out, "sum": x.to(out.dtype)}
    if op == "layer_norm_backward":
        x, dout = s["x"].float(), s["dout"].float()
        c = x - x.mean(-1, keepdim=True)
        r = torch.rsqrt((c * c).mean(-1, keepdim=True) + NORM_EPS)
        n = c * r
        dn = dout * s["gamma"]
        dx = r * (dn - dn.mean(-1, keepdim=True) - n * (dn * n).mean(-1, keepdim=True))
        if s["other"] is not None:
            dx = dx + s["other"].float()
        return {"dx": dx.to(s["x"].dtype), "dgamma": (dout * n).sum(0), "dbeta": dout.sum(0)}
    live = s["targets"] >= 0
    at = s["targets"].clamp(min=0)[:, None]
    z = _plain_logits(s)
    if op == "vocab_loss":
        top = z.max(-1, keepdim=True).values
        own_z = z.gather(1, at)
        total = torch.exp(z - top).sum(-1, keepdim=True).log()
        loss, lse = (top - own_z) + total, top + total
        return {"loss": torch.where(live, loss[:, 0], 0.0), "lse": torch.where(live, lse[:, 0], 0.0)}
    p = z.sub_(s["lse"][:, None]).exp_()
    p.scatter_add_(1, at, torch.full_like(at, -1, dtype=torch.float32))
    g = p.mul_(torch.where(live, s["dloss"], 0.0)[:, None])
    out = {"dh": (g @ s["W"].float()).bfloat16(), "dW": (g.T @ s["h"].float()).bfloat16()}
    if s["bias"] is not None:
        out["dbias"] = g.sum(0)
    return out


def _run_own(s):
    from delta_rule_linear_dpfp_gb300 import binding as fw
    op = s["op"]
    if op == "embedding":
        return {"out": fw.fw_embedding(s["ids"], s["table"], scale=s["scale"])}
    if op == "embedding_backward":
        return {"dtable": fw.fw_embedding_backward(s["ids"], s["dout"], s["V"], scale=s["scale"])}
    if op == "layer_norm":
        got = fw.fw_layer_norm(s["x"], s["gamma"], s["beta"], residual=s["other"], eps=NORM_EPS)
        return {"out": got} if s["other"] is None else {"out": got[0], "sum": got[1]}
    if op == "layer_norm_backward":
        return dict(zip(("dx", "dgamma", "dbeta"),
                        fw.fw_layer_norm_backward(s["x"], s["gamma"], s["dout"], dsum=s["other"], eps=NORM_EPS)))
    if op == "vocab_loss":
        return dict(zip(("loss", "lse"), fw.fw_vocab_loss(s["h"], s["W"], s["targets"], bias=s["bias"])))
    dh, dW, dbias = fw.fw_vocab_loss_backward(s["h"], s["W"], s["targets"], s["loss"], s["lse"], s["dloss"],
                                              bias=s["bias"])
    return {"dh": dh, "dW": dW} if dbias is None else {"dh": dh, "dW": dW, "dbias": dbias}


def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


# ------------------------------------------------------ what it cannot do without
def work(case):
    N, D, op = case["N"], case["D"], case["op"]
    e = 4 if case.get("io") == "f32" else 2
    if op == "layer_norm":
        return {"bytes": e * N * D * (4 if case["residual"] else 2) + 8 * D, "flops": 9 * N * D}
    if op == "layer_norm_backward":
        return {"bytes": e * N * D * (4 if case["residual"] else 3) + 12 * D, "flops": 20 * N * D}
    V = case["V"]
    if op == "embedding":
        return {"bytes": e * (N + min(N, V)) * D + 8 * N, "flops": N * D}
    if op == "embedding_backward":
        return {"bytes": e * (N + V) * D + 8 * N, "flops": N * D}
    vocab = 4 * V if case["bias"] else 0
    if op == "vocab_loss":
        return {"bytes": 2 * (N + V) * D + 16 * N + vocab, "flops": 2 * N * V * D + 4 * N * V}
    return {"bytes": 4 * (N + V) * D + 16 * N + 2 * vocab, "flops": 6 * N * V * D + 4 * N * V}


# ------------------------------------------------------------------- 64 bits
def _exact_embedding(s):
    live = s["ids"] >= 0
    if s["op"] == "embedding":
        out = torch.zeros(s["N"], s["D"], dtype=torch.float64, device="cuda")
        out[live] = s["scale"] * s["table"].double()[s["ids"][live]]
        return {"out": out}
    ids, order = torch.sort(s["ids"][live], stable=True)
    rows = s["scale"] * s["dout"].double()[live][order]
    run_sums = torch.cat([torch.zeros(1, s["D"], dtype=torch.float64, device="cuda"), rows.cumsum(0)])
    ends = torch.searchsorted(ids, torch.arange(s["V"], device="cuda"), right=True)
    begins = torch.searchsorted(ids, torch.arange(s["V"], device="cuda"))
    return {"dtable": run_sums[ends] - run_sums[begins]}


def _exact_norm(s):
    x, gamma, beta = s["x"].double(), s["gamma"].double(), s["beta"].double()
    other = None if s["other"] is None else s["other"].double()
    D = s["D"]
    if s["op"] == "layer_norm":
        y = x if other is None else x + other
        mean = y.sum(1) / D
        root = torch.sqrt(((y - mean[:, None]) ** 2).sum(1) / D + NORM_EPS)
        out = {"out": (y - mean[:, None]) / root[:, None] * gamma + beta}
        return out if other is None else {**out, "sum": y}
    mean = x.sum(1) / D
    root = torch.sqrt(((x - mean[:, None]) ** 2).sum(1) / D + NORM_EPS)[:, None]
    n, dout = (x - mean[:, None]) / root, s["dout"].double()
    t = dout * gamma / root
    dx = t - t.sum(1, keepdim=True) / D - n * ((t * n).sum(1, keepdim=True) / D)
    return {"dx": dx if other is None else dx + other, "dgamma": torch.einsum("nd,nd->d", dout, n), "dbeta": dout.sum(0)}


def _exact_vocab(s):
    N, V, D = s["N"], s["V"], s["D"]
    W = s["W"].double()
    bias = torch.zeros(V, dtype=torch.float64, device="cuda") if s["bias"] is None else s["bias"].double()
    step = max(1, 2 ** 28 // V)  # tokens at a time
    loss, lse = (torch.zeros(N, dtype=torch.float64, device="cuda") for _ in range(2))
    dh, dW, db = torch.zeros(N, D, dtype=torch.float64, device="cuda"), torch.zeros_like(W), torch.zeros_like(bias)
    for i in range(0, N, step):
        part = torch.arange(i, min(N, i + step), device="cuda")
        part = part[s["targets"][part] >= 0]
        if not len(part):
            continue
        h, t = s["h"][part].double(), s["targets"][part]
        z = torch.addmm(bias, h, W.T)
        total = torch.logsumexp(z, 1)
        here = torch.arange(len(part), device="cuda")
        if s["op"] == "vocab_loss":
            lse[part], loss[part] = total, total - z[here, t]
            continue
        g = torch.softmax(z, 1)
        g[here, t] -= 1
        g *= s["dloss"][part].double()[:, None]
        dh[part] = g @ W
        dW += g.T @ h
        db += g.sum(0)
    if s["op"] == "vocab_loss":
        return {"loss": loss, "lse": lse}
    return {"dh": dh, "dW": dW} if s["bias"] is None else {"dh": dh, "dW": dW, "dbias": db}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("embedding"):
        return _exact_embedding(s)
    return _exact_norm(s) if case["op"].startswith("layer_norm") else _exact_vocab(s)
