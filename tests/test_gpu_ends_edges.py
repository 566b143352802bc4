"""Calls of the vocabulary loss at the edges of its numbers: masks of low finite
values, long sums of one sign, log-sum-exps of any size.

Tolerances as in test_gpu_ends.py (u = 2^-24 is half a step of fp32), each
derived where it stands."""
import numpy as np
import pytest
import torch

from delta_rule_linear_dpfp_gb300 import binding as fw
from delta_rule_linear_dpfp_gb300 import build
from tests.parity_util import f64

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BOTH = pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build.build()
    fw.load()
    yield
    assert fw.fw_device_status() == fw.FW_OK


def draws(seed):
    r = torch.Generator(device="cuda").manual_seed(seed)
    return r, lambda *s: torch.randn(*s, generator=r, device="cuda")


@pytest.mark.parametrize("mask", [torch.finfo(torch.float32).min, -1e38, -2e37, -1e30, -1e29, -1e20, -1e10, -1e9, -1e4])
@pytest.mark.parametrize("N", [1, 3, 70, 300])
@BOTH
def test_a_finite_mask_is_a_mask(mask, N, dtype):
    """Entries whose bias is a low finite number, whole parts of the vocabulary of them: the bits of a bias of -infinity."""
    V, D = 900, 64
    r, n = draws(N)
    W, h = (n(V, D) * D ** -0.5).to(dtype), n(N, D).to(dtype)
    t = torch.randint(0, 100, (N,), generator=r, device="cuda")
    dl = torch.rand(N, generator=r, device="cuda")
    b = n(V)
    b[100:700] = -float("inf")
    low = torch.where(torch.isinf(b), mask, b)
    want = fw.fw_vocab_loss(h, W, t, bias=b)
    got = fw.fw_vocab_loss(h, W, t, bias=low)
    assert torch.isfinite(want[0]).all()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    grads = (fw.fw_vocab_loss_backward(h, W, t, *want, dl, bias=x) for x in (b, low))
    assert all(torch.equal(x, y) for x, y in zip(*grads))
    # a target among them costs what it is below the others: two roundings of the mask's size, the logits beside it
    t[0] = 333
    loss, lse = fw.fw_vocab_loss(h, W, t, bias=low)
    z = h[0].double() @ W[333].double() + low[333].double()
    assert abs(float(loss[0]) - (float(lse[0]) - float(z))) <= 4 * U * abs(float(z)) + 2.0 ** -18 * 10
    dW = fw.fw_vocab_loss_backward(h, W, t, loss, lse, dl, bias=low)[1]
    assert torch.isfinite(dW).all()


@pytest.mark.parametrize("N", [2, 40])
@BOTH
def test_all_taken_out(N, dtype):
    _, n = draws(N)
    W, h = n(100, 16).to(dtype), n(N, 16).to(dtype)
    t = torch.arange(N, device="cuda")
    for mask in (-float("inf"), torch.finfo(torch.float32).min, -1e20):
        b = torch.full((100,), mask, device="cuda")
        assert torch.isnan(fw.fw_vocab_loss(h, W, t, bias=b)[0]).all()
        b[7] = 1.0  # one is left: it is certain
        loss, lse = fw.fw_vocab_loss(h, W, torch.full_like(t, 7), bias=b)
        z = h.double() @ W[7].double() + 1
        assert torch.all(loss == 0) and torch.all((lse - z).abs() < 1e-4)


@BOTH
def test_gradients_in_place(dtype):
    """What the header allows: dx in place of x, dout or dsum, dgamma of gamma; sum and out of x or the residual."""
    _, n = draws(31)
    rows, d = 300, 520
    x, do, ds = (n(rows, d).to(dtype) for _ in range(3))
    gamma, beta = n(d), n(d)
    want = fw.fw_layer_norm_backward(x, gamma, do, dsum=ds)
    lib, code = fw.load(), fw._dtype_code(dtype)
    for place in range(3):
        t = [x.clone(), do.clone(), ds.clone()]
        g, db = gamma.clone(), torch.empty_like(gamma)
        ws = torch.empty(fw.fw_layer_norm_backward_workspace_size(rows, d), dtype=torch.uint8, device="cuda")
        rc = lib.fw_layer_norm_backward(t[0].data_ptr(), g.data_ptr(), t[1].data_ptr(), t[2].data_ptr(), t[place].data_ptr(),
                                        g.data_ptr(), db.data_ptr(), ws.data_ptr(), ws.numel(), rows, d, 1e-5, code,
                                        torch.cuda.current_stream().cuda_stream)
        assert rc == fw.FW_OK
        assert torch.equal(t[place], want[0]) and torch.equal(g, want[1]) and torch.equal(db, want[2])
    out, s = fw.fw_layer_norm(x, gamma, beta, residual=do)
    for swap in (False, True):
        a, b = x.clone(), do.clone()
        to = (b, a) if swap else (a, b)
        fw.fw_layer_norm(a, gamma, beta, residual=b, out=to[0], sum=to[1])
        assert torch.equal(to[0], out) and torch.equal(to[1], s)
    for bad in (dict(out=x, sum=x), dict(out=x.view(-1)[d:].view(rows - 1, d))):
        with pytest.raises((fw.FwError, ValueError)):
            fw.fw_layer_norm(x, gamma, beta, residual=do, **bad)
    # a row behind: the next row's values would be gone before they are read
    both = torch.cat([x, x[:1]])
    with pytest.raises(fw.FwError):
        fw.fw_layer_norm(both[:rows], gamma, beta, out=both[1:])


@BOTH
def test_bias_gradient_in_place(dtype):
    """dbias in place of bias, over several tiles; the other outputs' places are refused."""
    r, n = draws(32)
    N, V, D = 130, 700, 64
    h, W, b, dl = n(N, D).to(dtype), n(V, D).to(dtype), n(V), n(N)
    t = torch.randint(0, V, (N,), generator=r, device="cuda")
    loss, lse = fw.fw_vocab_loss(h, W, t, bias=b)
    dh, dW, db = fw.fw_vocab_loss_backward(h, W, t, loss, lse, dl, bias=b)
    c, dh2, dW2 = b.clone(), torch.empty_like(h), torch.empty_like(W)
    ws = torch.empty(fw.fw_vocab_loss_backward_workspace_size(N, V, D, dtype), dtype=torch.uint8, device="cuda")
    rc = fw.load().fw_vocab_loss_backward(h.data_ptr(), W.data_ptr(), c.data_ptr(), t.data_ptr(), loss.data_ptr(), lse.data_ptr(),
                                          dl.data_ptr(), dh2.data_ptr(), dW2.data_ptr(), c.data_ptr(), ws.data_ptr(), ws.numel(),
                                          N, V, D, 1, fw._dtype_code(dtype), torch.cuda.current_stream().cuda_stream)
    assert rc == fw.FW_OK
    assert torch.equal(dh2, dh) and torch.equal(dW2, dW) and torch.equal(c, db)
    with pytest.raises(fw.FwError):
        fw.fw_vocab_loss(h, W, t, bias=b, loss=loss, lse=loss)
    with pytest.raises(fw.FwError):
        fw.fw_embedding_backward(t, h, dtable=h, scale=1.0)


def room(gigabytes):
    if torch.cuda.mem_get_info()[0] < gigabytes * 1e9:
        pytest.skip(f"needs {gigabytes} GB")


def uniform(n, d, r):
    """[n, d] of one sign in bf16, each column with a scale of its own."""
    scale = 1 + torch.rand(d, generator=r, device="cuda")
    x = torch.empty(n, d, dtype=torch.bfloat16, device="cuda")
    for i in range(0, n, 2 ** 17):
        x[i:i + 2 ** 17] = torch.rand(x[i:i + 2 ** 17].shape, generator=r, device="cuda") * scale
    return x


def column_sums(x):
    return sum(x[i:i + 2 ** 17].double().sum(0) for i in range(0, len(x), 2 ** 17))


def test_long_sums_of_one_sign():
    """dW over 2^20 tokens and dh over 2^20 entries, all terms of one sign, too many tiles for the contraction to be split.
    Equal logits make G (2^-10, 2^-20) and w h exact, so that what is off is the sum and the output's own rounding.  Of a
    sum of 8192 terms at most the tensor core truncates 512 steps by 2^-22 of what there is so far: 2^-14 on average.  A
    column's rounding is spread over 2^-8 either way, with a deviation of at most 2^-8 / sqrt(3); the mean of D of them
    is within six of its own."""
    room(30)
    r, _ = draws(33)
    D = 2560
    lim = 2.0 ** -14 + 6 * 2.0 ** -8 / (3 * D) ** 0.5
    N, V = 2 ** 20, 1025
    h, W = uniform(N, D, r), torch.zeros(V, D, dtype=torch.bfloat16, device="cuda")
    t = torch.zeros(N, dtype=torch.int64, device="cuda")
    loss, lse = fw.fw_vocab_loss(h, W, t)
    dl = torch.full((N,), V / (V - 1), device="cuda")
    dW = fw.fw_vocab_loss_backward(h, W, t, loss, lse, dl, return_dh=False)[1]
    want = column_sums(h) / (V - 1)
    off = (dW[1:].double() - want) / want
    assert abs(float(off[0].mean())) <= lim and float(off.abs().max()) <= 2.0 ** -8 + 2.0 ** -13
    off = dW[0].double() / (-want * (V - 1)) - 1
    assert abs(float(off.mean())) <= lim and float(off.abs().max()) <= 2.0 ** -8 + 2.0 ** -13
    del h, dW
    N, V = 300, 2 ** 20 + 1
    h, W = torch.zeros(N, D, dtype=torch.bfloat16, device="cuda"), uniform(V, D, r)
    W[0] = 0
    t = torch.zeros(N, dtype=torch.int64, device="cuda")
    loss, lse = fw.fw_vocab_loss(h, W, t)
    dh = fw.fw_vocab_loss_backward(h, W, t, loss, lse, torch.ones(N, device="cuda"), return_dW=False)[0]
    want = column_sums(W) / V
    off = (dh.double() - want) / want
    assert torch.equal(dh, dh[:1].expand(N, D))
    assert abs(float(off[0].mean())) <= lim and float(off.abs().max()) <= 2.0 ** -8 + 2.0 ** -13
    del W
    torch.cuda.empty_cache()


@pytest.mark.parametrize("base", [0, 20, 1000, 30000])
@BOTH
def test_bias_gradient_of_large_logits(base, dtype):
    """Logits that are the bias alone, exact at any size: dbias, with the log-sum-exp as it was handed over, is off by the
    exponent's rounding (2^-21 for entries down to 2^-16 of the sum), the exponential's 2^-22, the constants' few u and the
    additions', and by the conversion to powers of two: 2^-25 of the distance to the log-sum-exp twice."""
    N, V, D = 70, 300, 8
    r, _ = draws(base)
    b = base + torch.randint(0, 40, (V,), generator=r, device="cuda") / 8
    h, W = (torch.zeros(n, D, dtype=dtype, device="cuda") for n in (N, V))
    t = torch.randint(0, V, (N,), generator=r, device="cuda")
    dl = torch.rand(N, generator=r, device="cuda")
    loss, lse = fw.fw_vocab_loss(h, W, t, bias=b)
    db = fw.fw_vocab_loss_backward(h, W, t, loss, lse, dl, bias=b)[2]
    p = torch.exp(b.double()[None] - lse.double()[:, None])
    want = (p * dl.double()[:, None]).sum(0)
    off = torch.ones(V, dtype=torch.bool, device="cuda")
    off[t] = False
    rel = ((db.double() - want) / want).abs()[off]
    assert off.sum() > 200 and float(rel.max()) <= 2.0 ** -21 + 2.0 ** -22 + 2 * 16 * 2.0 ** -25 + 16 * U


@pytest.mark.parametrize("N", [1, 70])
@pytest.mark.parametrize("D", [504, 512, 520, 1024, 16384, 65536])
def test_fp32_sums_of_equal_terms(N, D):
    """Logits that are sums of D equal terms, whose roundings all go one way: chunks of 512, then the chunks', each addition
    off by u of the sum so far at most.  (One token of up to 11264 channels: a lane's channels in two sums, then the lanes'.)"""
    V = 130
    r, _ = draws(D)
    c = (1 + torch.rand(V, generator=r, device="cuda")) * 8 / D
    W, h = c[:, None].expand(V, D).contiguous(), torch.ones(N, D, device="cuda")
    t = torch.arange(N, device="cuda")
    loss, lse = fw.fw_vocab_loss(h, W, t)
    z = W.double().sum(1)
    want = z.logsumexp(0)
    lim = (min(D, 512) + D / 512 + 8) * U * 16 + 2.0 ** -18
    assert float((lse - want).abs().max()) <= lim and float((loss - (want - z[t])).abs().max()) <= 2 * lim


def test_fp32_gradients_of_equal_terms():
    """The same of the products with g (2^-11 and the like for every entry but the target), not split."""
    r, _ = draws(34)
    for N, V, D in ((20000, 2049, 2560), (2560, 20001, 2560)):
        c = 1 + torch.rand(D, generator=r, device="cuda")
        h, W = c[None].expand(N, D).contiguous(), torch.zeros(V, D, device="cuda")
        t = torch.zeros(N, dtype=torch.int64, device="cuda")
        bias = torch.zeros(V, device="cuda")
        if V > N:  # for dh: the logits are equal all the same
            h, W = torch.zeros_like(h), c[None].expand(V, D).contiguous()
            W[0] = 0
        loss, lse = fw.fw_vocab_loss(h, W, t, bias=bias)
        dh, dW, _ = fw.fw_vocab_loss_backward(h, W, t, loss, lse, torch.ones(N, device="cuda"), bias=bias)
        n = max(N, V)
        lim = (512 + n / 512 + 8) * U + 2.0 ** -18  # (g: the logarithm's and the exponential's)
        if V > N:
            want = c.double() * (V - 1) / V
            assert float((dh.double() / want - 1).abs().max()) <= lim
        else:
            want = c.double() * N / V
            assert float((dW[1:].double() / want - 1).abs().max()) <= lim


@pytest.mark.parametrize("N, V, D", [(2, 129, 8), (64, 129, 64), (130, 1025, 72), (256, 4097, 64), (258, 129, 512),
                                     (2048, 65, 512), (8192, 129, 512)], ids=str)
def test_second_terms_of_the_answers(N, V, D):
    """Pairs of tokens with the same answer and weights of opposite sign, 2^-12 apart: dW is 2^-12 of either's part, which one
    rounding of w h to bf16 (2^-8 of it) would lose.  Equal logits make G exact (1 / (V - 1), and -1 for the target).  Two
    terms leave 2^-16 of each token's part; w itself is off by 4 u, the sums by two steps of 2^-22 of the parts so far."""
    r, n = draws(N)
    half = n(N // 2, D).bfloat16()
    half[16:] = 0  # (and the sum of 32 tokens' parts at most: zeros leave it as it is)
    h = torch.stack([half, half], 1).view(N, D)
    W = torch.zeros(V, D, dtype=torch.bfloat16, device="cuda")
    t = torch.zeros(N, dtype=torch.int64, device="cuda")
    up = V / (V - 1)
    dl = torch.tensor([(1 + 2.0 ** -12) * up, -up], device="cuda").repeat(N // 2)
    loss, lse = fw.fw_vocab_loss(h, W, t)
    dW = fw.fw_vocab_loss_backward(h, W, t, loss, lse, dl, return_dh=False)[1]
    w = dl.double() / up
    want = (w[:, None] * h.double()).sum(0)
    size = h.double().abs().sum(0)
    lim = (2.0 ** -16 + 4 * U) * size + 2 * 2.0 ** -22 * size + 2.0 ** -8 * want.abs()
    assert torch.all((dW[1:].double() * (V - 1) - want).abs() <= lim)
    assert torch.all((dW[0].double() + want).abs() <= lim)
    if N == 2:
        assert float(want.abs().max()) > 4 * float(lim.max())


@pytest.mark.parametrize("N, most", [(64, 128), (600, 512)])
def test_logits_of_one_sign(N, most):
    """Logits of 32 768 products of one sign: an accumulator takes 128 channels (up to 256 tokens) or 512, whose steps of 16
    truncate at most 2^-22 of the sum so far each, and the accumulators are added with roundings of u each.  One accumulator
    for all channels would fall short by 2048 steps of 2^-24 of half the sum, which is past the bound."""
    V, D = 300, 32768
    r, _ = draws(N)
    h, W = uniform(N, D, r), (uniform(V, D, r).float() * 2.0 ** -6).bfloat16()
    t = torch.randint(0, V, (N,), generator=r, device="cuda")
    loss, lse = fw.fw_vocab_loss(h, W, t)
    z = h.double() @ W.double().T
    want = z.logsumexp(1)
    lim = (most / 16 / 2 * 2.0 ** -22 + D / most * U) * z.max(1).values + 2.0 ** -18 * 10 + 2 * U * want
    assert 2.0 * float(lim.max()) < 2048 / 2 * 2.0 ** -24 * float(z.max())
    assert torch.all((lse - want).abs() <= lim)


# ------------------------------------------------------- calls of other kinds
@pytest.mark.parametrize("N", [1, 4, 5, 300])
@BOTH
def test_nothing_but_padding(N, dtype):
    _, n = draws(N)
    V, D = 200, 64
    h, W, b = torch.full((N, D), float("nan"), device="cuda").to(dtype), n(V, D).to(dtype), n(V)
    t = torch.full((N,), -1, dtype=torch.int32, device="cuda")
    loss, lse = fw.fw_vocab_loss(h, W, t, bias=b)
    assert torch.all(loss == 0) and torch.all(lse == 0)
    nan = torch.full((N,), float("nan"), device="cuda")
    for x in fw.fw_vocab_loss_backward(h, W, t, loss, lse, nan, bias=b):
        assert torch.all(x == 0)
    assert torch.all(fw.fw_embedding(t, W) == 0) and torch.all(fw.fw_embedding_backward(t, h, V) == 0)


@pytest.mark.parametrize("index", [torch.int32, torch.int64])
@BOTH
def test_slices_of_a_batch_of_tokens(index, dtype):
    """Ids and targets are read one at a time: a batch's sequence shifted by one is an argument as it is."""
    r, n = draws(41)
    V, D = 70, 32
    W = n(V, D).to(dtype)
    ids = torch.randint(-1, V, (91,), generator=r, device="cuda", dtype=index)
    h, dl = n(90, D).to(dtype), n(90)
    for a, b in ((ids[:90], ids[1:]), (ids[1:], ids[:90])):
        x, e = fw.fw_embedding(a, W), fw.fw_embedding(a.clone(), W)
        assert torch.equal(x, e)
        assert torch.equal(fw.fw_embedding_backward(a, h, V), fw.fw_embedding_backward(a.clone(), h, V))
        got, want = fw.fw_vocab_loss(h, W, b), fw.fw_vocab_loss(h, W, b.clone())
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        got = fw.fw_vocab_loss_backward(h, W, b, *want, dl)
        want = fw.fw_vocab_loss_backward(h, W, b.clone(), *want, dl)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("N, V", [(1, 9), (3, 300), (40, 70)])
@BOTH
def test_the_widest(N, V, dtype):
    """D 65536 in every call; errors as sums of D, N or V products (the bounds of test_gpu_ends.py, in the 2-norm)."""
    r, n = draws(N)
    D = 65536
    W, h = (n(V, D) * D ** -0.5).to(dtype), n(N, D).to(dtype)
    t, dl = torch.randint(0, V, (N,), generator=r, device="cuda"), n(N)
    loss, lse = fw.fw_vocab_loss(h, W, t)
    z = h.double() @ W.double().T
    want = z.logsumexp(1)
    S = (h.double().abs() @ W.double().abs().T).max()
    lim = 520 * U * S + 2.0 ** -18 * (1 + want.abs().max())
    assert torch.all((lse - want).abs() <= lim)
    assert torch.all((loss - (want - z.gather(1, t[:, None])[:, 0])).abs() <= 2 * lim)
    dh, dW, _ = fw.fw_vocab_loss_backward(h, W, t, loss, lse, dl)
    g = torch.softmax(z, 1)
    g[torch.arange(N, device="cuda"), t] -= 1
    g *= dl.double()[:, None]
    tol = 3 * 2.0 ** -8 if dtype == torch.bfloat16 else float(2 * lim)
    for x, w in ((dh, g @ W.double()), (dW, g.T @ h.double())):
        assert float((x.double() - w).norm()) <= tol * float(w.norm())
    out = fw.fw_embedding(t, W, scale=2.0)
    assert torch.equal(out, 2 * W[t])
    dE = fw.fw_embedding_backward(t, h, V)
    w = torch.zeros(V, D, dtype=torch.float64, device="cuda").index_add_(0, t, h.double())
    assert torch.all((dE.double() - w).abs() <= (2.0 ** -8 if dtype == torch.bfloat16 else 0) * w.abs() + 40 * U * 40)


def test_one_workspace_of_two_graphs():
    """Two captured steps of different sizes on one workspace, replayed in turn, with new inputs in the same places."""
    r, n = draws(42)
    sizes = ((600, 700, 512), (33, 3000, 64))
    need = max(max(fw.fw_vocab_loss_backward_workspace_size(*s), fw.fw_vocab_loss_workspace_size(*s),
                   fw.fw_embedding_backward_workspace_size(*s), fw.fw_layer_norm_backward_workspace_size(s[0], s[2]))
               for s in sizes)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def step(h, W, t, dl, w):
        loss, lse = fw.fw_vocab_loss(h, W, t, workspace=w)
        dh, dW, _ = fw.fw_vocab_loss_backward(h, W, t, loss, lse, dl, workspace=w)
        dx, dg, db = fw.fw_layer_norm_backward(h, None, dh, workspace=w)
        fw.fw_embedding_backward(t, dx, dtable=dW, accumulate=True, workspace=w)
        return loss, lse, dh, dW, dx, dg, db

    def fresh(N, V, D):
        return n(N, D).bfloat16(), (n(V, D) * D ** -0.5).bfloat16(), torch.randint(-1, V, (N,), generator=r, device="cuda"), n(N)

    ins = [fresh(*s) for s in sizes]
    graphs, kept = [], []
    for i in ins:
        step(*i, ws)
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            kept.append(step(*i, ws))
    for turn in range(3):
        for s, i in zip(sizes, ins):
            for a, b in zip(i, fresh(*s)):
                a.copy_(b)
        for k in kept:
            for x in k:
                x.fill_(float("nan"))
        ws.fill_(255)
        for g in (graphs if turn % 2 else graphs[::-1]):
            g.replay()
        want = [step(*i, None) for i in ins]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for k, w in zip(kept, want) for x, y in zip(k, w))


@pytest.mark.parametrize("d", [8, 4104, 8192])
@BOTH
def test_more_rows_than_threads_of_rows(d, dtype):
    """Every group of threads walks many rows, the last walk ragged; gradients against the 64-bit formula in the 2-norm."""
    _, n = draws(d)
    rows = 2 ** 22 // d + 77
    x, do = (n(rows, d) + 0.5).to(dtype), n(rows, d).to(dtype)
    gamma = 1 + 0.1 * n(d)
    dx, dg, db = fw.fw_layer_norm_backward(x, gamma, do, dsum=do)
    a, g = x.double(), do.double() * gamma.double()
    c = a - a.mean(-1, keepdim=True)
    r1 = torch.rsqrt((c * c).mean(-1, keepdim=True) + 1e-5)
    m = c * r1
    want = r1 * (g - g.mean(-1, keepdim=True) - m * (g * m).mean(-1, keepdim=True)) + do.double()
    rel = lambda p, q: float((p.double() - q).norm() / q.norm())  # noqa: E731
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
    assert rel(dx, want) <= half + 2.0 ** -18
    assert rel(dg, (do.double() * m).sum(0)) <= 2.0 ** -15 and rel(db, do.double().sum(0)) <= 2.0 ** -15
    out = fw.fw_layer_norm(x, gamma)
    assert rel(out, m * gamma.double()) <= half + 2.0 ** -18


@pytest.mark.parametrize("base", [1e4, 1e6, 5e8, 1.07e9, -1e6, -1.07e9])
@pytest.mark.parametrize("N", [3, 70])
@BOTH
def test_the_loss_of_large_logits(base, N, dtype):
    """Logits that are the bias alone, up to 2^30 in size: the losses are those of their differences, which are exact.  The
    exponents take one rounding, of the few units that the differences are, and a reference's own, up to 2^6, is in both
    terms of the quotient; lse is as its own size allows."""
    V, D = 300, 8
    r, _ = draws(N)
    step = max(2.0 ** -4, 2.0 ** (np.floor(np.log2(abs(base))) - 23))   # of fp32 at that size
    b = base + torch.randint(0, 60, (V,), generator=r, device="cuda") * step
    h, W = (torch.zeros(n, D, dtype=dtype, device="cuda") for n in (N, V))
    t = torch.randint(0, V, (N,), generator=r, device="cuda")
    loss, lse = fw.fw_vocab_loss(h, W, t, bias=b)
    z = b.double()
    want = z.logsumexp(0) - z[t]
    span = float(z.max() - z.min())
    # (the constant of the conversion is off by 2^-26 of a difference, an exponent rounded by 2^-24 of it)
    lim = 2.0 ** -18 * (1 + want) + 2.0 ** -22 * span
    assert torch.all((loss - want).abs() <= lim)
    assert torch.all((lse - z.logsumexp(0)).abs() <= 4 * U * abs(base) + 2.0 ** -18 * 10 + lim)


@pytest.mark.parametrize("N, V, D", [(2500, 9001, 520), (300, 33000, 64), (20000, 300, 128), (9000, 60001, 64), (2048, 65, 512),
                                     (4096, 250, 1024)], ids=str)
@BOTH
def test_large_gradients_to_the_last_rounding(N, V, D, dtype):
    """In the 2-norm.  bf16: an element's rounding is spread over 2^-8 of it either way at most, with a deviation of
    2^-8 / sqrt(3); an output has its own, G's and that of w h (none of the latter in two terms), which are independent:
    2^-8 in all, 2^-8 sqrt(2/3) without it, and 2^-12 beside them for the sums and the logits.  fp32: a sum of n terms goes by
    chunks of 512 and by splits; roundings are independent, too, so that sqrt(512 + n / 512 + 64) u of the terms' size is
    above what they leave; logits D products in the same way, twice, the constants and the exponential 2^-20."""
    from tests.test_gpu_ends import loss_inputs, plain_loss
    h, W, t, b, dl = (None if x is None else x.cuda() for x in loss_inputs(N, V, D, N + 1, bias=True, dtype=dtype))
    loss, lse = fw.fw_vocab_loss(h, W, t, bias=b)
    got = fw.fw_vocab_loss_backward(h, W, t, loss, lse, dl, bias=b)
    want = plain_loss(h, W, t, dl, b)
    rel = lambda a, w: float((a.double() - w).norm() / w.norm())  # noqa: E731
    if dtype == torch.bfloat16:
        two = N <= 256 or (V <= 256 and N * D <= 2 ** 22)
        assert rel(got[0], want[2]) <= 2.0 ** -8 * (2 / 3) ** 0.5 + 2.0 ** -12
        assert rel(got[1], want[3]) <= 2.0 ** -8 * ((2 if two else 3) / 3) ** 0.5 + 2.0 ** -12
    else:
        S = float((h.abs() @ W.abs().T).max()) + 5
        logits = 2 * (512 + D / 512 + 64) ** 0.5 * U * S + 2.0 ** -20
        for x, w, n in ((got[0], want[2], V), (got[1], want[3], N)):
            assert rel(x, w) <= 4 * (512 + n / 512 + 64) ** 0.5 * U + logits
    assert rel(got[2], want[4]) <= 1e-5
