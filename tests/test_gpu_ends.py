"""GPU parity of the embedding, the layer norm and the vocabulary loss, and of
their gradients, against the fp64 oracle.

Tolerances, from the arithmetic (u = 2^-24 is half a step of fp32):
 * Every bf16 output is rounded once: 2^-8 of its value.
 * Embedding: one product, u.  Its gradient: a run of n rows is added 32 at a
   time, at most 62 of them one by one and n / 32 parts: (96 + n / 32) u of the
   sum of the terms' sizes, and u for the scale (twice with the sum added).
 * Layer norm: a row's sums are trees of 3 + 5 + 5 additions; with the root, the
   divisions and the exchange between the warps 2^-18 of the row's scale, and the
   mean's own size over the deviation times 8 u beside it.  Its parameters'
   gradients: a term's 2^-18, and as many additions as a thread's rows, the
   CTA's and the CTAs' parts: 2^-15 of the terms' sizes.
 * Logits: products of bf16 are exact in fp32; each step of 16 of them is added
   with an error of at most 2^-22 of the sum of the products' sizes so far (the
   tensor core truncates): (D / 16 + 1) 2^-22 S with S = sum |h| |W| of the row.
   The loss takes two logits' errors, the exponentials' 2^-21, their sum's
   additions and the logarithm's: 2^-18 of 1 + |lse|.
 * Gradients of the loss: p is off by twice the logits' error and 2^-18 (1 + |lse|)
   of itself; G is rounded by 2^-8 of each entry but the target's, w h by 2^-8,
   and the sums' steps of 16 are as above."""
import numpy as np
import pytest
import torch

from delta_rule_linear_dpfp_gb300 import binding as fw
from delta_rule_linear_dpfp_gb300 import build
from oracle import ends
from tests.parity_util import f64

pytestmark = pytest.mark.gpu
U, HALF = 2.0 ** -24, {torch.bfloat16: 2.0 ** -8, torch.float32: 0.0}
BOTH = pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build.build()
    fw.load()
    yield
    assert fw.fw_device_status() == fw.FW_OK


def near(name, got, ref, lim):
    """|got - ref| <= lim + what rounding the output costs, element by element."""
    g, ref = f64(got), np.asarray(ref)
    assert g.shape == ref.shape, (name, g.shape, ref.shape)
    lim = lim + (HALF[got.dtype] + 2 * U) * np.abs(ref)
    off = np.abs(g - ref)
    assert np.all(off <= lim), (name, float(off.max()), float((off / np.maximum(lim, 1e-300)).max()))


def draws(seed):
    r = torch.Generator().manual_seed(seed)
    return r, lambda *s: torch.randn(*s, generator=r)


# ----------------------------------------------------------------- layer norm
def norm_check(rows, d, dtype, residual, seed, eps=1e-5, shift=0.5, params=True):
    r, n = draws(seed)
    x, gamma, beta, do = (n(rows, d) + shift * n(rows, 1)).to(dtype), 1 + 0.3 * n(d), 0.3 * n(d), n(rows, d).to(dtype)
    res, ds = (n(rows, d).to(dtype), n(rows, d).to(dtype)) if residual else (None, None)
    if not params:
        gamma = beta = None
    dv = lambda t: None if t is None else t.cuda()  # noqa: E731
    got = fw.fw_layer_norm(dv(x), dv(gamma), dv(beta), residual=dv(res), eps=eps)
    o = lambda t: None if t is None else f64(t)  # noqa: E731
    ref, s = ends.layer_norm(o(x), o(gamma), o(beta), o(res), eps)
    out, kept = got if residual else (got, x)
    c = s - s.mean(-1, keepdims=True)
    dev = np.sqrt((c * c).mean(-1, keepdims=True) + eps)
    tol = 2.0 ** -18 + 8 * U * np.abs(s).max(-1, keepdims=True) / dev
    near("out", out, ref, tol * (np.abs(ref).max(-1, keepdims=True) + 1))
    if residual:
        near("sum", kept, s, 2 * U * np.abs(s))
    dx, dgamma, dbeta = fw.fw_layer_norm_backward(dv(kept), dv(gamma), dv(do), dsum=dv(ds), eps=eps)
    kept = f64(kept)
    rx, rg, rb = ends.layer_norm_backward(kept, o(gamma), o(do), o(ds), eps)
    c = kept - kept.mean(-1, keepdims=True)
    dev = np.sqrt((c * c).mean(-1, keepdims=True) + eps)
    big = np.abs(f64(do)).max(-1, keepdims=True) * (1 if gamma is None else np.abs(o(gamma)).max()) * 4 / dev
    big = big * (1 + np.abs(c / dev).max(-1, keepdims=True))
    tol = 2.0 ** -18 + 8 * U * np.abs(kept).max(-1, keepdims=True) / dev
    near("dx", dx, rx, tol * big + (0 if ds is None else U * np.abs(o(ds))))
    terms = (np.abs(f64(do)) * (1 + np.abs(c / dev))).sum(0)
    # (the parameters' gradients carry the statistics' relative errors too)
    near("dgamma", dgamma, rg, (2.0 ** -15 + float(tol.max())) * terms)
    near("dbeta", dbeta, rb, 2.0 ** -15 * terms)


@pytest.mark.parametrize("rows, d", [(1, 8), (1, 512), (3, 16), (5, 64), (33, 72), (130, 128), (2, 200), (77, 256), (9, 264),
                                     (50, 512), (1, 1000), (40, 1024), (17, 1032), (11, 2048), (3, 2056), (6, 4096),
                                     (2, 4104), (1, 8184), (5, 8192), (2001, 24), (1500, 520)], ids=str)
@BOTH
@pytest.mark.parametrize("residual", [True, False])
def test_layer_norm(rows, d, dtype, residual):
    norm_check(rows, d, dtype, residual, rows + d)


@pytest.mark.parametrize("d", [40, 512, 1000])
@BOTH
def test_layer_norm_without_parameters(d, dtype):
    norm_check(7, d, dtype, True, d, params=False)


@pytest.mark.parametrize("d", [8, 96, 256, 1000, 8192])
def test_layer_norm_large_mean(d):
    norm_check(9, d, torch.float32, False, d, shift=300.0)


@pytest.mark.parametrize("rows, d", [(1, 8), (65, 32), (300, 256), (5, 1024), (700, 2048)], ids=str)
@BOTH
def test_layer_norm_without_eps(rows, d, dtype):
    norm_check(rows, d, dtype, False, rows, eps=0.0)


@pytest.mark.parametrize("d", [64, 512, 1024])
def test_layer_norm_rows_alone(d):
    """A NaN stays in its row, a row's bits do not depend on the others, equal channels give beta."""
    _, n = draws(d)
    x, gamma, beta = n(700, d), 1 + 0.1 * n(d), n(d)
    x[3] = 2.5
    x[5, 7] = float("nan")
    x[6, 0] = float("inf")
    out = fw.fw_layer_norm(x.cuda(), gamma.cuda(), beta.cuda())
    bad = torch.isnan(out).any(-1).cpu()
    assert bad[5] and bad[6] and bad.sum() == 2
    assert torch.equal(out[3].cpu(), beta)
    assert torch.equal(fw.fw_layer_norm(x[600:].cuda(), gamma.cuda(), beta.cuda()), out[600:])
    do = n(700, d)
    dx = fw.fw_layer_norm_backward(x.cuda(), gamma.cuda(), do.cuda())[0]
    bad = torch.isnan(dx).any(-1).cpu()
    assert bad[5] and bad[6] and bad.sum() == 2


def test_layer_norm_in_place_and_skipped():
    _, n = draws(3)
    x, res, gamma, do, ds = n(90, 256).cuda(), n(90, 256).cuda(), n(256).cuda(), n(90, 256).cuda(), n(90, 256).cuda()
    out, s = fw.fw_layer_norm(x, gamma, None, residual=res)
    x2, r2 = x.clone(), res.clone()
    got = fw.fw_layer_norm(x2, gamma, None, residual=r2, out=x2, sum=r2)
    assert got[0] is x2 and got[1] is r2 and torch.equal(x2, out) and torch.equal(r2, s)
    dx, dgamma, _ = fw.fw_layer_norm_backward(s, gamma, do, dsum=ds)
    d2 = ds.clone()
    got = fw.fw_layer_norm_backward(s, gamma, do, dsum=d2, dx=d2, return_params=False)
    assert got[1] is None and got[2] is None and torch.equal(d2, dx)
    # any number of axes, none of the rows
    assert torch.equal(fw.fw_layer_norm(x.view(9, 10, 256), gamma), fw.fw_layer_norm(x, gamma).view(9, 10, 256))
    assert fw.fw_layer_norm(x[:0], gamma).shape == (0, 256)
    _, dgamma, dbeta = fw.fw_layer_norm_backward(x[:0], gamma, do[:0])
    assert torch.all(dgamma == 0) and torch.all(dbeta == 0)


# ------------------------------------------------------------------ embedding
@pytest.mark.parametrize("N, V, D", [(1, 1, 8), (1, 65, 512), (7, 9, 24), (64, 300, 64), (257, 33, 1000), (33, 70000, 16),
                                     (1000, 65, 512), (5, 10, 2056), (3, 4, 4096)], ids=str)
@BOTH
@pytest.mark.parametrize("index", [torch.int32, torch.int64], ids=["i32", "i64"])
def test_embedding(N, V, D, dtype, index):
    r, n = draws(N + V + D)
    table, ids = n(V, D).to(dtype), torch.randint(0, V, (N,), generator=r, dtype=index)
    if N > 4:
        ids[::5] = -1
        ids[1] = V - 1
    out = fw.fw_embedding(ids.cuda(), table.cuda(), scale=1.75)
    ref = ends.embedding(ids.tolist(), f64(table), 1.75)
    near("out", out, ref, 0 * ref)
    assert torch.all(out.cpu()[ids < 0] == 0)


def tokens(N, V, kind, r):
    if kind == "one":
        return torch.full((N,), V // 2, dtype=torch.int64)
    if kind == "few":  # a few tokens all the time, and padding
        t = torch.randint(0, V, (N,), generator=r) % 3
        t[::7] = -100
        return t
    if kind == "none":
        return torch.full((N,), -1, dtype=torch.int64)
    t = torch.randint(0, V, (N,), generator=r)
    if N > 8:
        t[3], t[4] = V - 1, 0
    return t


@pytest.mark.parametrize("N, V, D", [(1, 1, 8), (2, 300, 16), (31, 5, 24), (32, 5, 64), (33, 255, 512), (64, 256, 40),
                                     (65, 257, 128), (1000, 65, 520), (4096, 65535, 32), (4097, 65536, 8), (40000, 70001, 16),
                                     (33000, 3, 8), (300, 7, 2056)], ids=str)
@BOTH
@pytest.mark.parametrize("kind", ["any", "few", "one", "none"])
def test_embedding_backward(N, V, D, dtype, kind):
    r, n = draws(N + V + D)
    ids, do = tokens(N, V, kind, r), n(N, D).to(dtype)
    do[ids < 0] = float("nan")                     # what padding holds reaches nothing
    start = n(V, D).to(dtype)
    dev = ids.cuda(), do.cuda()
    clean = torch.where((ids < 0)[:, None], torch.zeros((), dtype=dtype), do)
    idx = torch.where(ids < 0, V, ids)
    wide = torch.zeros(V + 1, D, dtype=torch.float64).index_add_(0, idx, clean.double())[:V]
    size = torch.zeros(V + 1, D, dtype=torch.float64).index_add_(0, idx, clean.double().abs())[:V].numpy()
    count = torch.bincount(idx, minlength=V + 1)[:V].double().numpy()[:, None]
    lim = (96 + count / 32) * U * size * 0.5
    got = fw.fw_embedding_backward(*dev, V, scale=0.5)
    near("dtable", got, 0.5 * wide.numpy(), lim)
    assert torch.all(got.cpu()[count[:, 0] == 0] == 0)
    assert torch.equal(got, fw.fw_embedding_backward(ids.int().cuda(), dev[1], V, scale=0.5))
    more = start.cuda()
    fw.fw_embedding_backward(*dev, V, scale=0.5, dtable=more, accumulate=True)
    near("accumulated", more, start.double().numpy() + 0.5 * wide.numpy(), lim + 2 * U * np.abs(start.double().numpy()))
    assert torch.equal(more.cpu()[count[:, 0] == 0], start[count[:, 0] == 0])


def test_embedding_backward_against_the_oracle():
    r, n = draws(5)
    ids, do = torch.randint(-2, 12, (200,), generator=r), n(200, 16)
    got = fw.fw_embedding_backward(ids.cuda(), do.cuda(), 10, scale=2.0)   # ids of 10 and 11 have no row
    ref = ends.embedding_backward(ids.tolist(), f64(do), 10, 2.0)
    near("dtable", got, ref, 200 * U * 2 * np.abs(f64(do)).max() * 200)
    out = fw.fw_embedding(ids.cuda(), n(10, 16).cuda())
    assert torch.equal(torch.isnan(out).all(-1).cpu(), ids >= 10) and torch.all(out.cpu()[ids < 0] == 0)


def test_embedding_shapes_and_empty():
    _, n = draws(6)
    table, ids = n(10, 16).cuda(), torch.tensor([[1, 2, -1], [9, 0, 3]]).cuda()
    out = fw.fw_embedding(ids, table)
    assert out.shape == (2, 3, 16) and torch.equal(out[0, 1], table[2])
    assert torch.equal(fw.fw_embedding_backward(ids, out, 10)[9], table[9])
    none = ids[:0]
    assert fw.fw_embedding(none, table).shape == (0, 3, 16)
    assert torch.all(fw.fw_embedding_backward(none, out[:0], 10) == 0)
    keep = table.clone()
    assert torch.equal(fw.fw_embedding_backward(none, out[:0], dtable=keep, accumulate=True), table)


# ------------------------------------------------------------ vocabulary loss
def loss_inputs(N, V, D, seed, bias=False, padded=False, known=6.0, weights=False, dtype=torch.bfloat16):
    r, n = draws(seed)
    W = (n(V, D) * D ** -0.5).to(dtype)
    t = torch.randint(0, V, (N,), generator=r)
    t[0] = V - 1
    h = (n(N, D) + known * torch.rand(N, 1, generator=r) * W[t].float()).to(dtype)
    b = n(V) if bias else None
    dl = torch.full((N,), 1.0 / N) if not weights else n(N)
    if padded:
        gone = torch.rand(N, generator=r) < 0.3
        t[gone] = -100
        h[gone] = float("nan")
        dl[gone] = float("nan")
    return h, W, t, b, dl


def loss_check(N, V, D, seed, index=torch.int64, **kw):
    h, W, t, b, dl = loss_inputs(N, V, D, seed, **kw)
    dv = lambda x: None if x is None else x.cuda()  # noqa: E731
    args = dv(h), dv(W), t.to(index).cuda()
    loss, lse = fw.fw_vocab_loss(*args, bias=dv(b))
    dh, dW, db = fw.fw_vocab_loss_backward(*args, loss, lse, dl.cuda(), bias=dv(b))
    live = (t >= 0).numpy()
    h0 = torch.where((t >= 0)[:, None], h.double(), 0.0).numpy()
    W0, tl, d0 = W.double().numpy(), t.tolist(), torch.where(t >= 0, dl.double(), 0.0).numpy()
    rl, rs, p = ends.vocab_loss(h0, W0, tl, None if b is None else b.double().numpy())
    S = np.abs(h0) @ np.abs(W0).T + (0 if b is None else np.abs(b.double().numpy()))
    half = HALF[h.dtype]
    # (fp32: a sum of n products takes n roundings of u of the terms' sizes at most)
    steps = lambda n: (n / 16 + 40) * 2.0 ** -22 if half else (n + 40) * U  # noqa: E731
    zerr = ((D / 16 + 1) * 2.0 ** -22 * S.max(-1) if half else (D + 1) * U * S.max(-1)) + 2.0 ** -18 * (1 + np.abs(rs))
    zerr = zerr * live
    near("loss", loss, rl, 2 * zerr)
    near("lse", lse, rs, 2 * zerr)
    rh, rW, rb = ends.vocab_loss_backward(h0, W0, tl, d0, None if b is None else b.double().numpy())
    g = p.copy()
    hot = np.zeros_like(p)
    hot[np.nonzero(live)[0], t.numpy()[live]] = 1
    g = np.abs(p - hot) * np.abs(d0)[:, None]            # the entries' sizes
    gerr = np.abs(d0)[:, None] * (p + hot) * 4 * zerr[:, None]   # what the logits and 1 - exp(-loss) leave
    off = g * (1 - hot) * half                            # G's rounding
    near("dh", dh, rh, (off + gerr) @ np.abs(W0) + steps(V) * (g @ np.abs(W0)))
    near("dW", dW, rW, (off + gerr + g * half).T @ np.abs(h0) + steps(N) * (g.T @ np.abs(h0)))
    if b is not None:
        near("dbias", db, rb, gerr.sum(0) + (N / 32 + 40) * U * g.sum(0))
    else:
        assert db is None
    assert torch.all(dh.cpu()[t < 0] == 0)


@pytest.mark.parametrize("N, V, D", [(1, 1, 8), (1, 2, 64), (1, 1000, 512), (2, 31, 24), (2, 20000, 264), (4, 3001, 2816),
                                     (3, 40, 2824), (1, 70, 11264), (1, 70, 11272), (3, 33, 16), (5, 255, 72), (64, 256, 128),
                                     (100, 257, 64), (127, 65, 512), (128, 128, 1024), (129, 129, 136), (256, 300, 256),
                                     (257, 511, 264), (300, 1025, 40), (520, 65, 512), (700, 770, 2048)], ids=str)
@pytest.mark.parametrize("bias", [False, True])
@BOTH
def test_vocab_loss(N, V, D, bias, dtype):
    loss_check(N, V, D, N + V + D, bias=bias, dtype=dtype)


@pytest.mark.parametrize("N, V, D", [(4, 9, 24), (130, 300, 64), (600, 70, 512)], ids=str)
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("index", [torch.int32, torch.int64], ids=["i32", "i64"])
@BOTH
def test_vocab_loss_padded(N, V, D, bias, index, dtype):
    """Padding's rows hold NaN: they reach nothing."""
    loss_check(N, V, D, N, index=index, bias=bias, padded=True, weights=True, dtype=dtype)


@pytest.mark.parametrize("known", [0.0, 40.0])
@BOTH
def test_vocab_loss_confident(known, dtype):
    """Tokens that nothing, and that everything, is known about."""
    loss_check(200, 500, 128, 7, known=known, bias=True, dtype=dtype)


@pytest.mark.parametrize("N", [1, 3, 70, 300])
@BOTH
def test_vocab_loss_all_but_certain(N, dtype):
    """A loss far below the logits' size keeps its digits: log(1 + sum exp(z_v - z_t)) is off by what the differences of
    logits are, relative to itself, and the exponentials' and the sum's 2^-19."""
    h, W, t, _, _ = loss_inputs(N, 400, 64, N, known=30.0, dtype=dtype)
    loss, _ = fw.fw_vocab_loss(h.cuda(), W.cuda(), t.cuda())
    z = h.double().numpy() @ W.double().numpy().T
    at = np.arange(N), t.numpy()
    d = z - z[at][:, None]
    d[at] = -np.inf
    ref = np.log1p(np.exp(d).sum(1))
    S = (np.abs(h.double().numpy()) @ np.abs(W.double().numpy()).T).max(1)
    rel = 4 * ((64 / 16 + 1) * 2.0 ** -22 if dtype == torch.bfloat16 else 65 * U) * S + 2.0 ** -19
    assert np.all(np.abs(f64(loss) - ref) <= rel * ref + 1e-300)
    assert ref.min() < 1e-3 or N < 70


@BOTH
def test_vocab_loss_masked_entries(dtype):
    """A bias of -infinity takes entries out, whole tiles of them; a target among them costs infinity."""
    h, W, t, b, dl = loss_inputs(70, 900, 64, 8, bias=True, dtype=dtype)
    b[100:700] = -float("inf")
    t[:] = 3
    t[5] = 200
    args = h.cuda(), W.cuda(), t.cuda()
    loss, lse = fw.fw_vocab_loss(*args, bias=b.cuda())
    kept = torch.cat([torch.arange(100), torch.arange(700, 900)])
    z = h.double() @ W[kept].double().T + b[kept].double()
    assert torch.all((lse.cpu().double() - z.logsumexp(1)).abs() < 1e-4)
    assert loss[5] == float("inf") and torch.isfinite(loss).sum() == 69
    dh, dW, db = fw.fw_vocab_loss_backward(*args, loss, lse, dl.cuda(), bias=b.cuda())
    out = torch.ones(900, dtype=torch.bool)
    out[kept] = False
    out[200] = False                    # (the target that was taken out pulls its row all the same)
    assert torch.all(dW.cpu()[out] == 0) and torch.all(db.cpu()[out] == 0)
    assert torch.isfinite(dh).all() and torch.isfinite(dW).all()
    none = torch.full_like(b, -float("inf"))
    loss, _ = fw.fw_vocab_loss(*args, bias=none.cuda())
    assert torch.isnan(loss).all()


@BOTH
def test_vocab_loss_past_the_vocabulary(dtype):
    h, W, t, _, dl = loss_inputs(40, 50, 32, 9, dtype=dtype)
    good = fw.fw_vocab_loss(h.cuda(), W.cuda(), t.cuda())[0]
    bad = t.clone()
    bad[7], bad[8] = 50, 2 ** 40
    loss, lse = fw.fw_vocab_loss(h.cuda(), W.cuda(), bad.cuda())
    assert torch.isnan(loss[7:9]).all() and torch.equal(loss[9:], good[9:])
    dh, dW, _ = fw.fw_vocab_loss_backward(h.cuda(), W.cuda(), bad.cuda(), loss, lse, dl.cuda())
    gone = t.clone()
    gone[7:9] = -1
    l2, s2 = fw.fw_vocab_loss(h.cuda(), W.cuda(), gone.cuda())
    dh2, dW2, _ = fw.fw_vocab_loss_backward(h.cuda(), W.cuda(), gone.cuda(), l2, s2, dl.cuda())
    assert torch.equal(dh, dh2) and torch.equal(dW, dW2)


@BOTH
def test_vocab_loss_parts_and_repeats(dtype):
    """Each gradient alone has the bits of all together, and every run the same."""
    h, W, t, b, dl = (None if x is None else x.cuda() for x in loss_inputs(300, 700, 256, 10, bias=True, dtype=dtype))
    loss, lse = fw.fw_vocab_loss(h, W, t, bias=b)
    dh, dW, db = fw.fw_vocab_loss_backward(h, W, t, loss, lse, dl, bias=b)
    assert torch.equal(fw.fw_vocab_loss_backward(h, W, t, loss, lse, dl, bias=b, return_dW=False)[0], dh)
    got = fw.fw_vocab_loss_backward(h, W, t, loss, lse, dl, bias=b, return_dh=False)
    assert got[0] is None and torch.equal(got[1], dW) and torch.equal(got[2], db)
    ws = torch.empty(fw.fw_vocab_loss_backward_workspace_size(300, 700, 256, dtype), dtype=torch.uint8, device="cuda")
    for fill in (0, 255):
        ws.fill_(fill)
        again = fw.fw_vocab_loss_backward(h, W, t, loss, lse, dl, bias=b, workspace=ws)
        assert all(torch.equal(x, y) for x, y in zip(again, (dh, dW, db)))
    # one token and a few at a time (summed on CUDA cores): off by the errors of two forms
    S = (h.double().abs() @ W.double().abs().T + b.double().abs()).max(1).values
    lim = 4 * ((256 / 16 + 1) * 2.0 ** -22 * S + 2.0 ** -18 * (1 + lse.double().abs()))
    for n in (0, 150, 299):
        one = fw.fw_vocab_loss(h[n], W, t[n], bias=b)
        assert one[0].shape == () and abs(one[0] - loss[n]) <= lim[n] and abs(one[1] - lse[n]) <= lim[n]
    for n in (2, 3, 4, 5):
        some = fw.fw_vocab_loss(h[:n], W, t[:n], bias=b)
        assert torch.all((some[0] - loss[:n]).abs() <= lim[:n]) and torch.all((some[1] - lse[:n]).abs() <= lim[:n])
    none = fw.fw_vocab_loss_backward(h[:0], W, t[:0], loss[:0], lse[:0], dl[:0], bias=b)
    assert none[0].shape == (0, 256) and torch.all(none[1] == 0) and torch.all(none[2] == 0)
    assert fw.fw_vocab_loss(h[:0], W, t[:0])[0].shape == (0,)


def plain_loss(h, W, t, dl, b=None):
    """In 64 bits on the GPU (elementary torch)."""
    z = h.double() @ W.double().T
    if b is not None:
        z += b.double()
    lse = z.logsumexp(1)
    loss = lse - z.gather(1, t[:, None])[:, 0]
    g = (z - lse[:, None]).exp_()
    g[torch.arange(len(t), device=t.device), t] -= 1
    g *= dl.double()[:, None]
    return loss, lse, g @ W.double(), g.T @ h.double(), g.sum(0)


@pytest.mark.parametrize("N, V, D", [(2500, 9001, 520), (70, 33000, 64), (20000, 300, 128), (33, 20011, 1024), (9000, 60001, 64)], ids=str)
@BOTH
def test_vocab_loss_many_tiles(N, V, D, dtype):
    """More tiles than pairs of SMs, long contractions, splits of them, pieces of the vocabulary: errors in the 2-norm.  bf16: an output's own
    rounding leaves at most 2^-8 of it, G's and w h's as much each, the sums' steps less: 2^-6.  fp32: p is off by the
    logits' error, at most 1e-5 here, and a sum of n terms by sqrt(n) u to n u of their sizes, n <= 60 000: 1e-4."""
    tol = 2.0 ** -6 if dtype == torch.bfloat16 else 1e-4
    h, W, t, b, dl = (None if x is None else x.cuda() for x in loss_inputs(N, V, D, N, bias=True, dtype=dtype))
    loss, lse = fw.fw_vocab_loss(h, W, t, bias=b)
    got = fw.fw_vocab_loss_backward(h, W, t, loss, lse, dl, bias=b)
    want = plain_loss(h, W, t, dl, b)
    rel = lambda a, w: float((a.double() - w).norm() / w.norm())  # noqa: E731
    assert rel(loss, want[0]) < 1e-5 and rel(lse, want[1]) < 1e-5
    assert rel(got[0], want[2]) < tol and rel(got[1], want[3]) < tol and rel(got[2], want[4]) < 1e-4
    # no tile is off by itself
    for x, w in ((got[0], want[2]), (got[1], want[3])):
        for i in range(0, len(w), 128):
            assert rel(x[i:i + 128], w[i:i + 128]) < 2 * tol, i


def test_graphs_and_streams():
    """Two captured graphs replayed in turn and two streams at once: every call has scratch of its own."""
    r, n = draws(13)
    ins = [tuple(None if x is None else x.cuda() for x in loss_inputs(N, V, 128, V, bias=True)) for N, V in ((200, 900), (333, 70))]

    def run(a):
        h, W, t, b, dl = a
        loss, lse = fw.fw_vocab_loss(h, W, t, bias=b)
        grads = fw.fw_vocab_loss_backward(h, W, t, loss, lse, dl, bias=b)
        out = fw.fw_embedding(t, W, scale=2.0)
        dE = fw.fw_embedding_backward(t, out, W.shape[0])
        o, s = fw.fw_layer_norm(out, residual=h)
        return (loss, lse, *grads, out, dE, o, s, *fw.fw_layer_norm_backward(s, None, o, dsum=h))

    want = [run(a) for a in ins]
    graphs, kept = [], []
    for a in ins:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            kept.append(run(a))
    for i in (0, 1, 1, 0):
        for x in kept[i]:
            x.zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(kept[i], want[i]))
    streams = [torch.cuda.Stream() for _ in ins]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = run(ins[i])
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(x, y) for x, y in zip(got[i], want[i]))
    # a stream given to the call: its outputs belong to it
    h, W, t, b, dl = ins[0]
    loss, lse = fw.fw_vocab_loss(h, W, t, bias=b, stream=streams[0])
    grads = fw.fw_vocab_loss_backward(h, W, t, loss, lse, dl, bias=b, stream=streams[0])
    out = fw.fw_embedding(t, W, scale=2.0, stream=streams[0])
    dE = fw.fw_embedding_backward(t, out, W.shape[0], stream=streams[0])
    o, s = fw.fw_layer_norm(out, residual=h, stream=streams[0])
    last = fw.fw_layer_norm_backward(s, None, o, dsum=h, stream=streams[0])
    streams[0].synchronize()
    assert all(torch.equal(x, y) for x, y in zip((loss, lse, *grads, out, dE, o, s, *last), want[0]))


def room(gigabytes):
    if torch.cuda.mem_get_info()[0] < gigabytes * 1e9:
        pytest.skip(f"needs {gigabytes} GB")


def test_offsets_past_32_bits():
    """More than 2^31 values: the last rows have the bits of calls of their own."""
    room(70)
    r = torch.Generator(device="cuda").manual_seed(14)
    rows, d = 2 ** 31 // 512 + 70, 512
    x = torch.randn(rows, d, generator=r, device="cuda", dtype=torch.bfloat16)
    g = torch.randn(d, generator=r, device="cuda")
    out, s = fw.fw_layer_norm(x, g, residual=x)
    dx, _, _ = fw.fw_layer_norm_backward(s, g, out, dsum=x)
    end = slice(rows - 60, rows)
    o1, s1 = fw.fw_layer_norm(x[end], g, residual=x[end])
    assert torch.equal(out[end], o1) and torch.equal(s[end], s1)
    assert torch.equal(dx[end], fw.fw_layer_norm_backward(s1, g, o1, dsum=x[end], return_params=False)[0])
    del out, s, dx
    # the same values as a table, and as the gradients of a batch
    ids = torch.tensor([0, rows - 1, -1, rows // 2, rows - 1], device="cuda")
    assert torch.equal(fw.fw_embedding(ids, x)[[0, 1, 3, 4]], x[ids[[0, 1, 3, 4]]])
    dE = fw.fw_embedding_backward(ids, x[:5].contiguous(), rows)
    assert torch.equal(dE[0], x[0]) and torch.equal(dE[rows // 2], x[3]) and dE[1:rows // 2].count_nonzero() == 0
    assert torch.equal(dE[-1], (x[1].float() + x[4].float()).bfloat16())
    del dE
    big = torch.randint(0, 9, (rows,), generator=r, device="cuda")
    out = fw.fw_embedding(big, x[:9].contiguous())
    assert torch.equal(out[end], x[big[end]])
    dE = fw.fw_embedding_backward(big, out, 9)
    count = torch.bincount(big, minlength=9).double()
    want = count[:, None] * x[:9].double()
    assert torch.all((dE.double() - want).abs() <= (2.0 ** -8 + (96 + rows / 32) * U) * want.abs())
    del out, x, dE
    torch.cuda.empty_cache()


def test_vocab_loss_offsets_past_32_bits():
    """An output map of more than 2^31 values, its last entries met: as the same map's halves."""
    room(40)
    r = torch.Generator(device="cuda").manual_seed(15)
    N, V, D = 40, 70001, 32768
    W = torch.randn(V, D, generator=r, device="cuda", dtype=torch.bfloat16).mul_(D ** -0.5)
    h = torch.randn(N, D, generator=r, device="cuda", dtype=torch.bfloat16)
    t = torch.randint(0, V, (N,), generator=r, device="cuda")
    t[:20] = V - 1 - torch.arange(20, device="cuda")
    dl = torch.full((N,), 1.0 / N, device="cuda")
    loss, lse = fw.fw_vocab_loss(h, W, t)
    dh, dW, _ = fw.fw_vocab_loss_backward(h, W, t, loss, lse, dl)
    z = torch.cat([h.double() @ W[i:i + 10000].double().T for i in range(0, V, 10000)], 1)
    want = z.logsumexp(1)
    assert torch.all((lse - want).abs() < 1e-4)
    assert torch.all((loss - (want - z.gather(1, t[:, None])[:, 0])).abs() < 1e-4)
    g = torch.softmax(z, 1)
    g[torch.arange(N, device="cuda"), t] -= 1
    g /= N
    rel = lambda a, w: float((a.double() - w).norm() / w.norm())  # noqa: E731
    for i in (0, 35000, V - 100):
        assert rel(dW[i:i + 100], g[:, i:i + 100].T @ h.double()) < 2.0 ** -6
    wh = sum(g[:, i:i + 10000] @ W[i:i + 10000].double() for i in range(0, V, 10000))
    assert rel(dh, wh) < 2.0 ** -6
    one = fw.fw_vocab_loss(h[:1, :8192].contiguous(), W[:, :8192].contiguous(), t[:1])
    assert torch.isfinite(one[0]).all()
    del W, dW, z, g
    torch.cuda.empty_cache()


# ------------------------------------------------------------- a run of them
def test_a_model_end_to_end():
    """Embedding, a gated layer between residual sums and norms, the loss over the same (tied) table, and every gradient
    back to it, against fp64 automatic differentiation; then the step as a graph, and on a stream of its own."""
    B, L, H, d, V = 2, 70, 2, 32, 90
    D = H * d
    r, n = draws(11)
    table = (n(V, D) * D ** -0.5).bfloat16().cuda()
    gamma, beta = (1 + 0.1 * n(D)).cuda(), (0.1 * n(D)).cuda()
    ids = torch.randint(0, V, (B, L), generator=r).cuda()
    targets = torch.randint(0, V, (B, L), generator=r).cuda()
    ids[1, 60:] = targets[1, 60:] = -1
    g = (-0.1 * torch.rand(B, H, L, generator=r)).bfloat16().cuda()
    be = torch.rand(B, H, L, generator=r).bfloat16().cuda()
    scale = D ** 0.5
    dl = torch.where(targets >= 0, 1.0 / (targets >= 0).sum(), 0.0)

    def heads(x):
        return x.view(B, L, H, d).transpose(1, 2).contiguous()

    def step():
        x = fw.fw_embedding(ids, table, scale=scale)
        q = heads(x)
        y, _ = fw.fw_gated_delta_forward(q, q, q, g, be, scale=d ** -0.5)
        a = y.transpose(1, 2).reshape(B, L, D).contiguous()
        o, s = fw.fw_layer_norm(a, gamma, beta, residual=x)
        loss, lse = fw.fw_vocab_loss(o, table, targets)
        do, dtable, _ = fw.fw_vocab_loss_backward(o, table, targets, loss, lse, dl)
        ds, dgamma, dbeta = fw.fw_layer_norm_backward(s, gamma, do)
        dq, dk, dv, dg, db, _ = fw.fw_gated_delta_backward(q, q, q, g, be, heads(ds), scale=d ** -0.5)
        dx = ds + (dq + dk + dv).transpose(1, 2).reshape(B, L, D)
        fw.fw_embedding_backward(ids, dx, dtable=dtable, scale=scale, accumulate=True)
        return loss, dtable, dgamma, dbeta

    got = step()
    E, ga, bt = (t.double().cpu().requires_grad_() for t in (table, gamma, beta))
    i, tt = ids.cpu(), targets.cpu()
    x = torch.where((i >= 0)[..., None], scale * E[i.clamp(min=0)], 0.0)
    q = x.view(B, L, H, d).transpose(1, 2)
    k = q / torch.sqrt((q * q).sum(-1, keepdim=True) + 1e-6)
    a, bw = torch.exp(g.double().cpu()), be.double().cpu()
    W, ys = torch.zeros(B, H, d, d, dtype=torch.float64), []
    for t in range(L):
        kt = k[:, :, t]
        W = a[:, :, t, None, None] * W
        u = bw[:, :, t, None] * (q[:, :, t] - (W @ kt[..., None])[..., 0])
        W = W + u[..., None] * kt[..., None, :]
        ys.append(d ** -0.5 * (W @ kt[..., None])[..., 0])
    s = x + torch.stack(ys, 2).transpose(1, 2).reshape(B, L, D)
    o = torch.nn.functional.layer_norm(s, (D,), ga, bt, 1e-5)
    z = o @ E.T
    live = tt >= 0
    loss = torch.where(live, z.logsumexp(-1) - z.gather(-1, tt.clamp(min=0)[..., None])[..., 0], 0.0)
    want = torch.autograd.grad((loss * dl.double().cpu()).sum(), [E, ga, bt])
    rel = lambda a, w: float((a.double().cpu() - w).norm() / w.norm())  # noqa: E731
    # each stage rounds its bf16 output by at most 2^-8 of it, and there are nine in a row
    assert rel(got[0], loss.detach()) < 9 * 2.0 ** -8
    assert all(rel(a, w) < 9 * 2.0 ** -8 for a, w in zip(got[1:], want))
    assert torch.all(got[0][1, 60:] == 0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(again, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    for _ in range(2):
        for x in kept:
            x.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(kept, got))
    if torch.cuda.device_count() > 1:
        with pytest.raises(ValueError):
            fw.fw_embedding(ids, table.to("cuda:1"))


def test_refused():
    _, n = draws(12)
    x, gamma = n(4, 32).cuda(), n(32).cuda()
    for bad in (dict(residual=x[:3]), dict(residual=x.bfloat16()), dict(sum=x), dict(out=x.bfloat16()), dict(gamma=gamma[:8]),
                dict(gamma=gamma.bfloat16())):
        with pytest.raises(ValueError):
            fw.fw_layer_norm(x, **{"gamma": gamma, **bad})
    with pytest.raises(ValueError):
        fw.fw_layer_norm(x.t(), gamma)
    with pytest.raises(TypeError):
        fw.fw_layer_norm(x.half(), gamma)
    with pytest.raises(fw.FwError):
        fw.fw_layer_norm(x[:, :12].contiguous(), gamma[:12].contiguous())
    ids = torch.tensor([1, 2, 3, 4]).cuda()
    with pytest.raises(TypeError):
        fw.fw_embedding(ids.float(), x)
    with pytest.raises(ValueError):
        fw.fw_embedding_backward(ids, x)
    with pytest.raises(ValueError):
        fw.fw_embedding_backward(ids, x, 9, accumulate=True)
    with pytest.raises(ValueError):
        fw.fw_embedding_backward(ids[:3], x, 9)
    h, W = x.bfloat16(), n(9, 32).bfloat16().cuda()
    f = n(4).cuda()
    for bad in (dict(h=h.half(), W=W.half()), dict(targets=ids.float())):
        with pytest.raises(TypeError):
            fw.fw_vocab_loss(**{"h": h, "W": W, "targets": ids, **bad})
    for bad in (dict(h=x), dict(W=W.float()), dict(targets=ids[:3]), dict(bias=f), dict(bias=n(9).bfloat16().cuda()), dict(loss=f.double()), dict(W=W.t())):
        with pytest.raises(ValueError):
            fw.fw_vocab_loss(**{"h": h, "W": W, "targets": ids, **bad})
    with pytest.raises(ValueError):
        fw.fw_vocab_loss_backward(h, W, ids, f, f, f[:3])
