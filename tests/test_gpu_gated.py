"""GPU parity of the gated delta rule (sequence, gradients, one token) against
the fp64 oracle, and the calls its documentation allows.

Tolerances, from the arithmetic.  fp32 I/O: sums of at most 256 products a
term, 2^-24 each, so 2^-16 of the terms' sizes; the terms may cancel by a
factor of four: 2^-14 of the largest value.  bf16 I/O: an operand that is not
bf16 already may enter a product as two bf16 terms (2^-8 of it is left by the
first, 2^-8 of that by the second: 2^-16); the state, X, T, U and one dropped
product make 5 2^-16 of the terms' sizes, and with cancellation by three
2^-12 of the largest value; gradients pass twice as many: 2^-11.  A bf16
output is rounded once more, by at most 2^-8 of its own value.  dg is a
difference: what the answers lose when the state decays less what the token
itself wrote, so its terms are as large as dy.y of a token even where nothing
is left (a first token without a state has dg = 0)."""
import numpy as np
import pytest
import torch

from delta_rule_linear_dpfp_gb300 import binding as fw
from delta_rule_linear_dpfp_gb300 import build
from oracle import gated
from tests.parity_util import f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build.build()
    fw.load()
    yield
    assert fw.fw_device_status() == fw.FW_OK


def near(name, got, ref, grad=False, bf16=None, terms=0.0):
    bf16 = got.dtype == torch.bfloat16 if bf16 is None else bf16
    tol = (2.0 ** -11 if grad else 2.0 ** -12) if bf16 else 2.0 ** -14
    ref = np.asarray(ref)
    assert tuple(got.shape) == ref.shape, name
    g = f64(got)
    assert np.all(np.isfinite(g)), name
    lim = tol * max(np.abs(ref).max() if ref.size else 0, terms, 1e-30)
    if got.dtype == torch.bfloat16:
        lim = lim + 2.0 ** -8 * np.abs(ref)
    off = np.abs(g - ref)
    assert np.all(off <= lim), (name, off.max(), np.abs(ref).max())


def make(B, Hk, H, L, d_k, d_v, dtype, state, seed, keys="normal"):
    r = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=r)  # noqa: E731
    d = dict(q=n(B, Hk, L, d_k), k=n(B, Hk, L, d_k), v=n(B, H, L, d_v),
             g=-torch.rand(B, H, L, generator=r) * torch.exp(-4 * torch.rand(H, 1, generator=r)),
             beta=torch.rand(B, H, L, generator=r))
    if keys == "positive":   # strongly alike, as a feature map's are: T is far from the identity
        d["k"] = d["k"].abs() / d_k ** 0.5
        d["q"] = d["q"].abs() / d_k ** 0.5
    d = {x: t.to(dtype) for x, t in d.items()}
    d["W0"] = n(B, H, d_v, d_k) if state else None
    return d


def dev(d):
    return {n: None if t is None else t.cuda() for n, t in d.items()}


def host(d):
    return {n: None if t is None else f64(t) for n, t in d.items()}


# B, Hk, H, L, d_k, d_v, state, padded
CASES = [
    (1, 1, 1, 1, 16, 16, False, False),
    (2, 1, 2, 2, 32, 48, True, False),
    (1, 2, 2, 63, 64, 64, True, False),
    (2, 1, 3, 64, 128, 32, False, False),
    (1, 2, 4, 65, 64, 16, True, True),
    (3, 2, 2, 130, 128, 128, True, True),
    (1, 1, 1, 200, 16, 256, True, False),
    (2, 2, 6, 257, 32, 80, False, True),
    (1, 1, 2, 640, 128, 96, True, False),
    (5, 2, 6, 70, 128, 80, True, True),       # more CTAs than SMs, an odd number of 32-channel slices
    (10, 3, 3, 65, 64, 96, False, False),
    (1, 1, 2, 130, 128, 256, True, False),    # the widest state
    (2, 4, 8, 1600, 64, 48, True, True),      # long enough for the forward to go in segments
]


def _lengths(B, L, seed):
    r = np.random.default_rng(seed)
    lens = r.integers(0, L + 1, B)
    lens[0] = [L, L + 5, max(L - 1, 0)][seed % 3]       # past the end counts as the end
    if B > 1:
        lens[-1] = [0, -3, 1][seed % 3]                  # nothing at all
    return lens


@pytest.mark.parametrize("case", CASES, ids=lambda c: "b{}k{}h{}l{}dk{}dv{}s{:d}p{:d}".format(*c))
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("l2norm", [True, False])
def test_forward_and_gradients(case, dtype, l2norm):
    B, Hk, H, L, d_k, d_v, state, padded = case
    d = make(B, Hk, H, L, d_k, d_v, dtype, state, sum(case), "normal" if l2norm else "positive")
    lens = _lengths(B, L, sum(case)) if padded else None
    lt = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    x = dev(d)
    if lens is not None:                                  # whatever lies behind the end is not used
        for b, n in enumerate(lens):
            for t in ("q", "k", "v", "g", "beta"):
                x[t][b, :, max(int(n), 0):] = float("nan")
    opt = dict(l2norm=l2norm, scale=0.6)
    y, W = fw.fw_gated_delta_forward(**x, lengths=lt, **opt)
    ref = host(d)
    if lens is not None:                                  # (the oracle reads none of it either)
        for b, n in enumerate(lens):
            for t in ("q", "k", "v", "g", "beta"):
                ref[t][b, :, max(int(n), 0):] = np.nan
    yr, Wr = gated.gated_forward(**ref, lengths=lens, **opt)
    bf16 = dtype == torch.bfloat16
    near("y", y, yr)
    near("W", W, Wr, bf16=bf16)
    if lens is not None:
        for b, n in enumerate(lens):
            assert torch.all(y[b, :, max(int(n), 0):] == 0)

    r = torch.Generator().manual_seed(1)
    dy = torch.randn(B, H, L, d_v, generator=r).to(dtype)
    dW = torch.randn(B, H, d_v, d_k, generator=r) if state else None
    dyd = dy.cuda()
    if lens is not None:
        for b, n in enumerate(lens):
            dyd[b, :, max(int(n), 0):] = float("inf")
    got = fw.fw_gated_delta_backward(x["q"], x["k"], x["v"], x["g"], x["beta"], dyd, W0=x["W0"],
                                     dW_final=None if dW is None else dW.cuda(), lengths=lt, **opt)
    want = gated.gated_backward(ref["q"], ref["k"], ref["v"], ref["g"], ref["beta"], f64(dy), ref["W0"],
                                None if dW is None else f64(dW), lengths=lens, **opt)
    if lens is not None:                                  # zeros there, on both sides
        want = list(want)
        for w in want[:5]:
            for b, n in enumerate(lens):
                w[b, :, max(int(n), 0):] = 0
    terms = np.abs(f64(dy) * yr).sum(-1).max()
    for n, a, w in zip(("dq", "dk", "dv", "dg", "dbeta", "dW0"), got, want):
        near(n, a, w, grad=True, bf16=bf16, terms=terms if n == "dg" else 0.0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_strong_gates(dtype):
    """Tokens that forget everything (-inf, and sums far past exp's range)
    between others: no NaN, and the later tokens' decays keep their bits."""
    d = make(2, 2, 2, 150, 64, 32, dtype, True, 7)
    d["g"][:, :, 20] = -float("inf")
    d["g"][:, 0, 70:75] = -90.0
    d["g"][0, 1, 130] = -1e30
    x = dev(d)
    y, W = fw.fw_gated_delta_forward(**x)
    yr, Wr = gated.gated_forward(**host(d))
    near("y", y, yr)
    near("W", W, Wr, bf16=dtype == torch.bfloat16)
    dy = torch.randn(2, 2, 150, 32, generator=torch.Generator().manual_seed(2)).to(dtype)
    got = fw.fw_gated_delta_backward(x["q"], x["k"], x["v"], x["g"], x["beta"], dy.cuda(), W0=x["W0"])
    h = host(d)
    want = gated.gated_backward(h["q"], h["k"], h["v"], h["g"], h["beta"], f64(dy), h["W0"])
    for n, a, w in zip(("dq", "dk", "dv", "dg", "dbeta", "dW0"), got, want):
        near(n, a, w, grad=True, bf16=dtype == torch.bfloat16)


@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_keys_of_zeros(eps):
    d = make(1, 1, 2, 70, 32, 16, torch.bfloat16, True, 8)
    d["k"][:, :, 3] = 0
    d["q"][:, :, 66] = 0
    x = dev(d)
    y, W = fw.fw_gated_delta_forward(**x, eps=eps)
    yr, Wr = gated.gated_forward(**host(d), eps=eps)
    near("y", y, yr)
    near("W", W, Wr, bf16=True)
    assert torch.all(y[:, :, 66] == 0)
    got = fw.fw_gated_delta_backward(x["q"], x["k"], x["v"], x["g"], x["beta"], torch.ones_like(x["v"]), W0=x["W0"], eps=eps)
    assert all(torch.isfinite(t).all() for t in got)


def test_a_nan_gate_is_not_hidden():
    d = dev(make(1, 1, 2, 70, 32, 16, torch.bfloat16, True, 8))
    d["g"][0, 0, 65] = float("nan")
    y, _ = fw.fw_gated_delta_forward(**d)
    assert torch.isfinite(y[0, 0, :64]).all() and torch.isnan(y[0, 0, 65:]).all() and torch.isfinite(y[0, 1]).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("case", [(1, 1, 1, 16, 16), (3, 2, 4, 32, 48), (2, 1, 3, 64, 64), (5, 4, 4, 128, 256),
                                  (2, 2, 2, 64, 208)], ids=str)
def test_decode_is_the_sequence(case, dtype):
    B, Hk, H, d_k, d_v = case
    T = 5
    d = make(B, Hk, H, T, d_k, d_v, dtype, True, sum(case))
    x = dev(d)
    W = x["W0"].clone()
    ys = []
    for t in range(T):
        one = [x[n][:, :, t].clone() for n in ("q", "k", "v", "g", "beta")]
        ys.append(fw.fw_gated_delta_decode_step(*one, W, scale=0.5))
    yr, Wr = gated.gated_forward(**host(d), scale=0.5)
    near("y", torch.stack(ys, 2), yr)
    near("W", W, Wr, bf16=False)


def test_decode_extremes():
    d = make(2, 1, 2, 1, 64, 32, torch.bfloat16, True, 3)
    d["g"][0] = -float("inf")
    d["k"][1] = 0
    one = {n: t[:, :, 0].contiguous().cuda() for n, t in d.items() if n != "W0"}
    W = d["W0"].cuda()
    y = fw.fw_gated_delta_decode_step(**one, W=W, eps=0.0)
    yr, Wr = gated.gated_forward(**host(d), eps=0.0)
    near("y", y, yr[:, :, 0])
    near("W", W, Wr, bf16=False)


def test_in_place_state_and_no_state():
    d = dev(make(2, 2, 2, 100, 64, 48, torch.bfloat16, True, 9))
    y, W = fw.fw_gated_delta_forward(**d)
    W2 = d["W0"].clone()
    y2, out = fw.fw_gated_delta_forward(**{**d, "W0": W2}, W_final=W2)
    assert out is W2 and torch.equal(W, W2) and torch.equal(y, y2)
    y3, none = fw.fw_gated_delta_forward(**d, return_state=False)
    assert none is None and torch.equal(y, y3)


def test_split_sequence_and_repeats():
    """Two calls with the state passed on are one call; every repeat has the same bits."""
    d = dev(make(2, 1, 2, 192, 128, 64, torch.bfloat16, True, 10))
    y, W = fw.fw_gated_delta_forward(**d)
    for _ in range(3):
        y1, W1 = fw.fw_gated_delta_forward(**d)
        assert torch.equal(y, y1) and torch.equal(W, W1)
    a = {n: t[:, :, :128].contiguous() for n, t in d.items() if n != "W0"}
    b = {n: t[:, :, 128:].contiguous() for n, t in d.items() if n != "W0"}
    ya, Wa = fw.fw_gated_delta_forward(**a, W0=d["W0"])
    yb, Wb = fw.fw_gated_delta_forward(**b, W0=Wa)
    assert torch.equal(torch.cat([ya, yb], 2), y) and torch.equal(Wb, W)
    dy = torch.randn_like(d["v"])
    args = [d[n] for n in ("q", "k", "v", "g", "beta")]
    first = fw.fw_gated_delta_backward(*args, dy, W0=d["W0"])
    again = fw.fw_gated_delta_backward(*args, dy, W0=d["W0"])
    assert all(torch.equal(s, t) for s, t in zip(first, again))


@pytest.mark.parametrize("L", [0, 1])
def test_empty(L):
    d = dev(make(2, 1, 2, L, 32, 16, torch.bfloat16, True, 11))
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    y, W = fw.fw_gated_delta_forward(**d, lengths=lens)
    assert torch.equal(W, d["W0"]) and torch.all(y == 0)
    dW = torch.randn_like(d["W0"])
    got = fw.fw_gated_delta_backward(*[d[n] for n in ("q", "k", "v", "g", "beta")], torch.ones_like(d["v"]), W0=d["W0"],
                                     dW_final=dW, lengths=lens)
    assert torch.equal(got[5], dW) and all(torch.all(t == 0) for t in got[:5])
    e = {n: t[:0] for n, t in d.items()}
    y, W = fw.fw_gated_delta_forward(**e)
    assert y.shape[0] == 0 and W.shape[0] == 0


def test_graphs_and_streams():
    """Captured and replayed with new inputs, two graphs at once on two
    streams, and a call on a stream that is not the current one."""
    d = dev(make(2, 2, 2, 130, 64, 32, torch.bfloat16, True, 12))
    e = dev(make(2, 2, 2, 130, 64, 32, torch.bfloat16, True, 13))
    args = ("q", "k", "v", "g", "beta")

    def both(x):
        y, W = fw.fw_gated_delta_forward(**x)
        return (y, W) + fw.fw_gated_delta_backward(*[x[n] for n in args], x["v"], W0=x["W0"])

    want_d, want_e = both(d), both(e)
    one = {n: t.clone() for n, t in d.items()}
    two = {n: t.clone() for n, t in d.items()}
    graphs = []
    for x in (one, two):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = both(x)
        graphs.append((g, out))
    for n in one:
        two[n].copy_(e[n])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for s, (g, _) in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for (_, out), want in zip(graphs, (want_d, want_e)):
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y, W = fw.fw_gated_delta_forward(**e, stream=s)
    s.synchronize()
    assert torch.equal(y, want_e[0]) and torch.equal(W, want_e[1])


def test_refused_tensors():
    d = dev(make(2, 1, 2, 20, 32, 16, torch.bfloat16, True, 14))
    call = fw.fw_gated_delta_forward
    for bad in (dict(q=d["q"].transpose(0, 1)), dict(k=d["k"][:, :, :19]), dict(g=d["g"].float()), dict(v=d["v"].cpu()),
                dict(W0=d["W0"].bfloat16()), dict(W0=d["W0"][:1]), dict(v=d["v"][:, :1]), dict(beta=d["beta"][..., None])):
        with pytest.raises(ValueError):
            call(**{**d, **bad})
    with pytest.raises(ValueError):
        call(**d, lengths=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        call(**d, y=torch.empty(2, 2, 20, 32, dtype=torch.bfloat16, device="cuda"))
    three = dev(make(2, 2, 3, 20, 32, 16, torch.bfloat16, True, 14))
    with pytest.raises(ValueError):
        call(**three)
    odd = dev(make(2, 1, 2, 20, 32, 24, torch.bfloat16, True, 14))
    with pytest.raises(fw.FwError) as err:
        call(**odd)
    assert err.value.code == fw.FW_ERR_UNSUPPORTED
    with pytest.raises(fw.FwError):
        call(**d, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    buf = torch.empty(2 * 1 * 20 * 32 + 8, dtype=torch.bfloat16, device="cuda")[1:1 + 2 * 20 * 32].view(2, 1, 20, 32)
    with pytest.raises(fw.FwError):
        call(**{**d, "q": buf})


def test_gradients_are_the_differences():
    """Central differences of the fp32 forward along random directions.  The
    loss is summed in 64 bits; y's error of 2^-14 of its size over a step of
    2^-6 leaves 2^-7 of the slope's scale."""
    d = dev(make(1, 1, 2, 90, 32, 32, torch.float32, True, 15))
    gen = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda t: torch.randn(t.shape, generator=gen, device="cuda")  # noqa: E731
    dy, dW = rnd(d["v"]), rnd(d["W0"])
    got = dict(zip(("q", "k", "v", "g", "beta", "W0"),
                   fw.fw_gated_delta_backward(*[d[n] for n in ("q", "k", "v", "g", "beta")], dy, W0=d["W0"], dW_final=dW)))

    def loss(x):
        y, W = fw.fw_gated_delta_forward(**x)
        return float((y.double() * dy).sum() + (W.double() * dW).sum())

    for n in d:
        way = torch.sign(got[n])                          # the steepest of the box: a large slope
        step = 2.0 ** -8 * float(d[n].abs().mean())
        diff = (loss({**d, n: d[n] + step * way}) - loss({**d, n: d[n] - step * way})) / (2 * step)
        slope = float((got[n].double() * way).sum())
        assert abs(diff - slope) <= 2.0 ** -6 * abs(slope), (n, diff, slope)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", [(2, 1, 2, 130, 64, 48), (5, 2, 6, 70, 128, 80), (1, 1, 1, 3, 16, 16)], ids=str)
def test_a_workspace_of_anything(shape, dtype):
    """What a workspace holds on entry does not matter: all ones (NaN in every type) gives the same bits."""
    B, Hk, H, L, d_k, d_v = shape
    d = dev(make(B, Hk, H, L, d_k, d_v, dtype, True, 16))
    args = [d[n] for n in ("q", "k", "v", "g", "beta")]
    lens = torch.full((B,), max(L - 20, 1), dtype=torch.int32, device="cuda")
    got = []
    for fill in (0, 255):
        n = fw.fw_gated_delta_forward_workspace_size(B, Hk, H, L, d_k, d_v, dtype)
        m = fw.fw_gated_delta_backward_workspace_size(B, Hk, H, L, d_k, d_v, dtype)
        ws = torch.full((max(n, m),), fill, dtype=torch.uint8, device="cuda")
        out = fw.fw_gated_delta_forward(*args, W0=d["W0"], lengths=lens, workspace=ws)
        ws.fill_(fill)
        out += fw.fw_gated_delta_backward(*args, d["v"], W0=d["W0"], dW_final=d["W0"], lengths=lens, workspace=ws)
        got.append(out)
    assert all(torch.isfinite(t).all() for t in got[0])
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_two_streams_at_once():
    """Calls with workspaces of their own on two streams: the bits of the calls alone."""
    ds = [dev(make(2, 2, 4, 1600, 64, 64, torch.bfloat16, True, s)) for s in (17, 18)]
    args = ("q", "k", "v", "g", "beta")

    def work(d):
        y, W = fw.fw_gated_delta_forward(**d)
        return (y, W) + fw.fw_gated_delta_backward(*[d[n] for n in args], y, W0=d["W0"])

    want = [work(d) for d in ds]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ds]
    outs = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(work(ds[i]))
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(a, b) for r in o for a, b in zip(r, w))


def test_decode_in_a_graph():
    """One captured step replayed for token after token: the sequence's answers."""
    d = make(3, 1, 2, 6, 64, 32, torch.bfloat16, True, 19)
    x = dev(d)
    one = {n: x[n][:, :, 0].clone() for n in ("q", "k", "v", "g", "beta")}
    W = x["W0"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = fw.fw_gated_delta_decode_step(**one, W=W)
    ys = []
    for t in range(6):
        for n in one:
            one[n].copy_(x[n][:, :, t])
        graph.replay()
        ys.append(y.clone())
    yr, Wr = gated.gated_forward(**host(d))
    near("y", torch.stack(ys, 2), yr)
    near("W", W, Wr, bf16=False)


def test_lengths_are_refused_unaligned():
    d = dev(make(3, 1, 2, 20, 32, 16, torch.bfloat16, True, 20))
    lens = torch.full((4,), 5, dtype=torch.int32, device="cuda")[1:]
    with pytest.raises(fw.FwError):
        fw.fw_gated_delta_forward(**d, lengths=lens)


# ---- a forward in several segments: preparation beside the walk over the segment before

def segments(B, H, L, d_v):
    """How many segments the forward takes (the rule of csrc/fw_gated_tc.cu)."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    chunks, heads = -(-L // 64), B * H
    walkers = heads * -(-d_v // 32)
    if 2 * walkers > sms:
        return 1
    wave = max(1, 2 * (sms - walkers) // heads)
    seg = -(-12 // wave) * wave
    n = (chunks + seg // 2) // seg
    return 1 if n < 2 else -(-chunks // -(-chunks // n))


# B, Hk, H, L, d_k, d_v
LONG = [(3, 3, 6, 2301, 64, 48), (2, 8, 8, 3800, 128, 64), (1, 8, 16, 4500, 128, 128)]


def by_parts(d, lens, chunks=8):
    """The same sequence in calls of a few chunks each, which take one segment each."""
    L, W, ys = d["v"].shape[2], d["W0"], []
    for t in range(0, L, 64 * chunks):
        part = {n: x[:, :, t:t + 64 * chunks].contiguous() for n, x in d.items() if n != "W0"}
        left = None if lens is None else (lens - t).clamp(min=0).to(torch.int32)
        y, W = fw.fw_gated_delta_forward(**part, W0=W, lengths=left)
        ys.append(y)
    return torch.cat(ys, 2), W


@pytest.mark.parametrize("case", LONG, ids=str)
@pytest.mark.parametrize("ends", [None, 0.2, 0.5, 0.9, 0.0], ids=str)
def test_segments_are_the_parts(case, ends):
    """One call in three segments and more has the bits of its parts, called one
    by one: sequences that end in the first, a middle, the last segment, or
    before any; every repeat as well, and the state in place."""
    B, Hk, H, L, d_k, d_v = case
    assert segments(B, H, L, d_v) >= 3
    d = dev(make(B, Hk, H, L, d_k, d_v, torch.bfloat16, True, 21))
    lens = None
    if ends is not None:
        lens = torch.full((B,), int(ends * L), dtype=torch.int32, device="cuda")
        lens[-1] = L - 3 if B > 1 else lens[-1]
    y, W = by_parts(d, lens)
    for _ in range(3):
        y1, W1 = fw.fw_gated_delta_forward(**d, lengths=lens)
        assert torch.equal(y, y1) and torch.equal(W, W1)
    same = d["W0"].clone()
    y1, _ = fw.fw_gated_delta_forward(**{**d, "W0": same}, W_final=same, lengths=lens)
    assert torch.equal(y, y1) and torch.equal(W, same)


def test_segments_against_the_oracle():
    B, Hk, H, L, d_k, d_v = LONG[0]
    d = make(B, Hk, H, L, d_k, d_v, torch.bfloat16, True, 22)
    y, W = fw.fw_gated_delta_forward(**dev(d))
    yr, Wr = gated.gated_forward(**host(d))
    near("y", y, yr)
    near("W", W, Wr, bf16=True)


@pytest.mark.parametrize("case", LONG, ids=str)
def test_segments_in_graphs_and_on_streams(case):
    """Captured and replayed on new inputs, a workspace of one call reused by the
    next, and two calls at once on two streams."""
    B, Hk, H, L, d_k, d_v = case
    ds = [dev(make(B, Hk, H, L, d_k, d_v, torch.bfloat16, True, s)) for s in (23, 24)]
    want = [by_parts(d, None) for d in ds]
    x = {n: t.clone() for n, t in ds[0].items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fw.fw_gated_delta_forward(**x)
    for i in (0, 1, 1, 0):
        for n in x:
            x[n].copy_(ds[i][n])
        graph.replay()
        graph.replay()                                    # (at once behind the first, in the same workspace)
        assert all(torch.equal(a, b) for a, b in zip(got, want[i]))
    ws = torch.empty(fw.fw_gated_delta_forward_workspace_size(B, Hk, H, L, d_k, d_v, torch.bfloat16), dtype=torch.uint8,
                     device="cuda")
    outs = [fw.fw_gated_delta_forward(**ds[i & 1], workspace=ws) for i in range(6)]
    for i, out in enumerate(outs):
        assert all(torch.equal(a, b) for a, b in zip(out, want[i & 1]))
    streams, outs = [torch.cuda.Stream() for _ in ds], []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for i, s in enumerate(streams):
            outs.append((i, fw.fw_gated_delta_forward(**ds[i], stream=s)))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for i, out in outs for a, b in zip(out, want[i]))


def test_features_written_by_the_kernel_before():
    """Keys and queries that fw_dpfp writes immediately before, into the same
    buffers again and again, a long (segmented) call and gates and betas written by a copy: no
    call sees what a buffer held before."""
    B, H, L, d_key, d_v = 2, 4, 6400, 32, 32
    assert segments(B, H, L, d_v) >= 2
    r = torch.Generator(device="cuda").manual_seed(25)
    raw = [torch.randn(2, B, H, L, d_key, generator=r, device="cuda").bfloat16() for _ in range(3)]
    v = torch.randn(B, H, L, d_v, generator=r, device="cuda").bfloat16()
    g = -torch.rand(3, B, H, L, generator=r, device="cuda").bfloat16()
    be = torch.rand(3, B, H, L, generator=r, device="cuda").bfloat16()

    def alone(i):
        q, k = fw.fw_dpfp(raw[i][0]), fw.fw_dpfp(raw[i][1])
        torch.cuda.synchronize()
        out = fw.fw_gated_delta_forward(q, k, v, g[i].clone(), be[i].clone())
        torch.cuda.synchronize()
        return out

    want = [alone(i) for i in range(3)]
    q, k = (torch.empty(B, H, L, 2 * d_key, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    gi, bi = g[0].clone(), be[0].clone()
    outs = []
    for i in (0, 1, 2, 0, 2, 1):
        gi.copy_(g[i])
        bi.copy_(be[i])
        fw.fw_dpfp(raw[i][0], out=q)
        fw.fw_dpfp(raw[i][1], out=k)
        outs.append((i, fw.fw_gated_delta_forward(q, k, v, gi, bi)))
    assert all(torch.equal(a, b) for i, out in outs for a, b in zip(out, want[i]))


# ---- how much the states keep

def off_by(got, ref):
    ref = np.asarray(ref)
    return np.linalg.norm(f64(got) - ref) / np.linalg.norm(ref)


@pytest.mark.parametrize("case", [(2, 2, 4, 640, 128, 96), (2, 4, 4, 500, 64, 64), (1, 1, 2, 900, 32, 128)], ids=str)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_states_keep_their_bits(case, dtype):
    """The 2-norm of the states' errors.  bf16 tensors: a value in two bf16 terms
    is off by 2^-18 of itself (root mean square: each term leaves 2^-9.3, the
    dropped product of the second terms is as large); five operands of that kind
    lie between the inputs and the state (T, M, W', S, U), their errors add in
    squares, and the difference v - S k takes terms of up to sqrt(2) of its own
    size: sqrt(5) sqrt(2) 2^-18 < 2^-16.  The gradient goes through as many
    again: 2^-15.  fp32 tensors: six products of up to 128 terms, each off by
    sqrt(128) 2^-25, the same difference: below 2^-19, and 2^-18 for the gradient."""
    B, Hk, H, L, d_k, d_v = case
    d = make(B, Hk, H, L, d_k, d_v, dtype, True, sum(case))
    x, h = dev(d), host(d)
    bits = 16 if dtype == torch.bfloat16 else 19
    y, W = fw.fw_gated_delta_forward(**x, scale=0.5)
    yr, Wr = gated.gated_forward(**h, scale=0.5)
    assert off_by(W, Wr) <= 2.0 ** -bits
    if dtype == torch.float32:
        assert off_by(y, yr) <= 2.0 ** -19
    else:
        # An answer off by 2^-16 of the answers' size before its rounding goes to the other neighbour where the
        # exact one lies that near the middle of two: for normal answers 2^-7 sqrt(2 / pi) (1 + ln 2^7) = 4 % at most.
        there = torch.from_numpy(yr).float().bfloat16()
        other = (y.cpu() != there).float().mean()
        assert other <= 0.04, float(other)
    r = torch.Generator().manual_seed(1)
    dy, dW = torch.randn(B, H, L, d_v, generator=r).to(dtype), torch.randn(B, H, d_v, d_k, generator=r)
    args = ("q", "k", "v", "g", "beta")
    got = fw.fw_gated_delta_backward(*[x[n] for n in args], dy.cuda(), W0=x["W0"], dW_final=dW.cuda(), scale=0.5)
    want = gated.gated_backward(*[h[n] for n in args], f64(dy), h["W0"], f64(dW), scale=0.5)
    assert off_by(got[5], want[5]) <= 2.0 ** -(bits - 1)
    if dtype == torch.float32:
        for n, a, w in zip(("dq", "dk", "dv"), got, want):
            assert off_by(a, w) <= 2.0 ** -18, n


# ---- other calls that the documentation allows

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_decode_with_keys_as_given(dtype):
    d = make(3, 2, 4, 4, 64, 48, dtype, True, 26, "positive")
    x, W, ys = dev(d), d["W0"].cuda(), []
    for t in range(4):
        one = [x[n][:, :, t].contiguous() for n in ("q", "k", "v", "g", "beta")]
        ys.append(fw.fw_gated_delta_decode_step(*one, W, l2norm=False, scale=-0.5))
    yr, Wr = gated.gated_forward(**host(d), l2norm=False, scale=-0.5)
    near("y", torch.stack(ys, 2), yr)
    near("W", W, Wr, bf16=False)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("given", [(False, True), (True, False), (False, False)], ids=["dW", "W0", "neither"])
def test_gradients_of_either_state(given, dtype):
    """A gradient of the last state without a first state, and the other way round."""
    d = make(2, 1, 3, 100, 32, 48, dtype, given[0], 27)
    x, h = dev(d), host(d)
    r = torch.Generator().manual_seed(4)
    dy = torch.randn(2, 3, 100, 48, generator=r).to(dtype)
    dW = torch.randn(2, 3, 48, 32, generator=r) if given[1] else None
    args = ("q", "k", "v", "g", "beta")
    call = dict(W0=x["W0"], dW_final=None if dW is None else dW.cuda(), scale=-0.7)
    got = fw.fw_gated_delta_backward(*[x[n] for n in args], dy.cuda(), **call)
    want = gated.gated_backward(*[h[n] for n in args], f64(dy), h["W0"], None if dW is None else f64(dW), scale=-0.7)
    yr, _ = gated.gated_forward(**h, scale=-0.7)
    terms = np.abs(f64(dy) * yr).sum(-1).max()
    for n, a, w in zip(("dq", "dk", "dv", "dg", "dbeta", "dW0"), got, want):
        near(n, a, w, grad=True, bf16=dtype == torch.bfloat16, terms=terms if n == "dg" else 0.0)
    less = fw.fw_gated_delta_backward(*[x[n] for n in args], dy.cuda(), **call, return_dW0=False)
    assert less[5] is None and all(torch.equal(a, b) for a, b in zip(got[:5], less[:5]))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_a_scale_of_nothing(dtype):
    d = dev(make(1, 1, 2, 70, 32, 16, dtype, True, 28))
    y, W = fw.fw_gated_delta_forward(**d, scale=0.0)
    _, W1 = fw.fw_gated_delta_forward(**d)
    assert torch.all(y == 0) and torch.equal(W, W1)


def test_the_most_heads():
    """B H = 65 535, the last the grid takes: the bits of the batch in two parts; one more is refused."""
    B, L = 65535, 2
    r = torch.Generator(device="cuda").manual_seed(29)
    q, k, v, dy = (torch.randn(B, 1, L, 16, generator=r, device="cuda").bfloat16() for _ in range(4))
    g, be = (torch.rand(B, 1, L, generator=r, device="cuda").bfloat16() for _ in range(2))
    ins = (q, k, v, -g, be)

    def both(lo, hi):
        part = [t[lo:hi].contiguous() for t in ins]
        return fw.fw_gated_delta_forward(*part) + fw.fw_gated_delta_backward(*part, dy[lo:hi].contiguous())

    whole, a, b = both(0, B), both(0, 30000), both(30000, B)
    assert all(torch.equal(w, torch.cat(p)) for w, p in zip(whole, zip(a, b)))
    one = [t[:, :, 0].contiguous() for t in ins]
    W = torch.randn(B, 1, 16, 16, generator=r, device="cuda")
    halves = [W[:30000].clone(), W[30000:].clone()]
    y = fw.fw_gated_delta_decode_step(*one, W)
    ys = [fw.fw_gated_delta_decode_step(*[t[s].contiguous() for t in one], w)
          for s, w in zip((slice(0, 30000), slice(30000, B)), halves)]
    assert torch.equal(y, torch.cat(ys)) and torch.equal(W, torch.cat(halves))
    more = [torch.cat([t, t[:1]]) for t in ins]
    with pytest.raises(fw.FwError) as err:
        fw.fw_gated_delta_forward(*more)
    assert err.value.code == fw.FW_ERR_UNSUPPORTED


def test_offsets_past_32_bits():
    """More than 2^31 values and 2^34 bytes of workspace: the bits of the sequence in two calls."""
    H, L, d_v, cut = 2, 4200001, 256, 64 * 65000
    if torch.cuda.mem_get_info()[0] < 80e9:
        pytest.skip("needs 60 GB")
    r = torch.Generator(device="cuda").manual_seed(30)
    n = lambda *s: torch.randn(*s, generator=r, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    ins = (n(1, 1, L, 16), n(1, 1, L, 16), n(1, H, L, d_v), -torch.rand(1, H, L, generator=r, device="cuda").bfloat16(),
           torch.rand(1, H, L, generator=r, device="cuda").bfloat16())
    assert ins[2].numel() > 2 ** 31
    y, W = fw.fw_gated_delta_forward(*ins)
    y1, W1 = fw.fw_gated_delta_forward(*[t[:, :, :cut].contiguous() for t in ins])
    assert torch.equal(y[:, :, :cut], y1)
    y2, W2 = fw.fw_gated_delta_forward(*[t[:, :, cut:].contiguous() for t in ins], W0=W1)
    assert torch.equal(y[:, :, cut:], y2) and torch.equal(W, W2)
    del y, y1, y2, ins
    torch.cuda.empty_cache()


# ---- the gates' gradients

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("case", [(2, 1, 2, 1, 16, 16), (1, 2, 2, 1, 128, 64), (3, 2, 4, 5, 64, 48), (1, 1, 2, 130, 32, 80),
                                  (2, 2, 4, 200, 128, 128)], ids=str)
def test_nothing_to_forget(case, dtype):
    """Where nothing was there before a token its gate does not matter: dg is 0
    there, not what rounding leaves; so too behind a gate of -inf."""
    B, Hk, H, L, d_k, d_v = case
    d = make(B, Hk, H, L, d_k, d_v, dtype, False, sum(case))
    if L > 4:
        d["g"][:, 0, [3, L - 1]] = -float("inf")
    if L > 64:
        d["g"][:, 1, 64] = -float("inf")                  # a chunk's first token
    x = dev(d)
    args = ("q", "k", "v", "g", "beta")
    r = torch.Generator().manual_seed(31)
    dy, dW = torch.randn(B, H, L, d_v, generator=r).to(dtype), torch.randn(B, H, d_v, d_k, generator=r)
    dg = fw.fw_gated_delta_backward(*[x[n] for n in args], dy.cuda(), dW_final=dW.cuda())[3]
    assert torch.all(dg[:, :, 0] == 0)
    assert torch.all(dg[torch.isinf(x["g"])] == 0)
    want = gated.gated_backward(*[host(d)[n] for n in args], f64(dy), dW=f64(dW))[3]
    assert L == 1 or np.count_nonzero(want) > 0
    assert torch.all((dg.cpu() != 0) == torch.from_numpy(np.abs(want) > 1e-30))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("case", [(1, 1, 1, 70, 16, 16), (2, 1, 3, 150, 64, 48), (1, 2, 4, 200, 128, 128), (1, 1, 2, 257, 32, 80)],
                         ids=str)
def test_gradients_of_strong_gates(case, dtype):
    """Gates that leave e^-8 to e^-16 of everything: dg carries that factor, and
    so do its errors (no difference of large terms): dg e^-g within 2^-11 of its largest, as the other gradients
    (fp32 tensors: 2^-14), the exponent's rounding of 2^-19 among it."""
    B, Hk, H, L, d_k, d_v = case
    d = make(B, Hk, H, L, d_k, d_v, dtype, True, sum(case))
    r = torch.Generator().manual_seed(32)
    d["g"] = (-8 - 8 * torch.rand(B, H, L, generator=r)).to(dtype)
    x, h = dev(d), host(d)
    args = ("q", "k", "v", "g", "beta")
    dy, dW = torch.randn(B, H, L, d_v, generator=r).to(dtype), torch.randn(B, H, d_v, d_k, generator=r)
    got = fw.fw_gated_delta_backward(*[x[n] for n in args], dy.cuda(), W0=x["W0"], dW_final=dW.cuda(), scale=0.7)
    want = gated.gated_backward(*[h[n] for n in args], f64(dy), h["W0"], f64(dW), scale=0.7)
    rise = np.exp(-h["g"])
    off, ref = np.abs(f64(got[3]) - want[3]) * rise, np.abs(want[3]) * rise
    bf16 = dtype == torch.bfloat16
    assert np.all(off <= (2.0 ** -11 if bf16 else 2.0 ** -14) * ref.max() + (2.0 ** -8 * ref if bf16 else 0)), (off.max(), ref.max())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("case", [(2, 2, 4, 640, 128, 96), (2, 4, 4, 500, 64, 64), (1, 1, 2, 900, 32, 128)], ids=str)
def test_gate_gradients_keep_their_bits(case, dtype):
    """The 2-norm of dg's errors: bf16 tensors, the rounding's 2^-9 (root mean
    square at most) and 2^-13 of sums of 64 and more two-term products; fp32
    tensors, as the other gradients, 2^-18."""
    B, Hk, H, L, d_k, d_v = case
    d = make(B, Hk, H, L, d_k, d_v, dtype, True, sum(case))
    x, h = dev(d), host(d)
    args = ("q", "k", "v", "g", "beta")
    r = torch.Generator().manual_seed(33)
    dy, dW = torch.randn(B, H, L, d_v, generator=r).to(dtype), torch.randn(B, H, d_v, d_k, generator=r)
    got = fw.fw_gated_delta_backward(*[x[n] for n in args], dy.cuda(), W0=x["W0"], dW_final=dW.cuda(), scale=0.5)
    want = gated.gated_backward(*[h[n] for n in args], f64(dy), h["W0"], f64(dW), scale=0.5)
    assert off_by(got[3], want[3]) <= (2.0 ** -9 + 2.0 ** -13 if dtype == torch.bfloat16 else 2.0 ** -18)
