"""GPU parity of the group norm with its activation, forward and backward,
against the fp64 oracle, and the whole output path of a gated layer.

Tolerances, from the arithmetic: a row's statistics are sums of at most 256
values in a tree of 8 + 5 additions (13 2^-24), the root and the divisions add
a few units, the activations' functions two: 2^-18 of the row's scale, and the
mean's own size over the deviation times 2^-24 beside it (inputs here: at most
64).  dgamma and dbeta add up to B L rows more in 32 bits: 2^-16 of the sum of
the terms' sizes.  A bf16 output is rounded once, by at most 2^-8 of its
value."""
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


def near(name, got, ref, scale, tol):
    g = f64(got)
    assert g.shape == np.asarray(ref).shape, name
    lim = tol * scale + (2.0 ** -8 * np.abs(ref) if got.dtype == torch.bfloat16 else 0)
    off = np.abs(g - ref)
    assert np.all(off <= lim), (name, off.max(), np.max(scale))


def make(B, H, L, d, dtype, gate, seed, shift=1.0):
    r = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=r)  # noqa: E731
    x = (n(B, H, L, d) + shift * n(H, 1, 1)).to(dtype)
    return (x, 1 + 0.3 * n(H * d), 0.3 * n(H * d), n(B, L, H * d).to(dtype) if gate else None,
            n(B, L, H * d).to(dtype))


def check(B, H, L, d, dtype, act, gate, seed, shift=1.0):
    x, gamma, beta, z, do = make(B, H, L, d, dtype, gate, seed, shift)
    dv = lambda t: None if t is None else t.cuda()  # noqa: E731
    kw = dict(act=act, gate=dv(z))
    out = fw.fw_group_norm_act(dv(x), dv(gamma), dv(beta), **kw)
    dx, dgate, dgamma, dbeta = fw.fw_group_norm_act_backward(dv(x), dv(gamma), dv(beta), dv(do), **kw)
    o = [None if t is None else f64(t) for t in (x, gamma, beta, z, do)]
    ref = gated.group_norm_act(o[0], o[1], o[2], o[3], act)
    rx, rz, rg, rb = gated.group_norm_act(o[0], o[1], o[2], o[3], act, dout=o[4])
    tol = 2.0 ** -18 + 2.0 ** -24 * 64
    near("out", out, ref, np.abs(ref).max() + 1, tol)
    # dx carries 1 / deviation of its row
    big = np.abs(rx).max(-1, keepdims=True) + np.abs(rx).max() * 1e-3
    near("dx", dx, rx, np.maximum(big, np.abs(rx).max() * 0.1), 8 * tol)
    if gate:
        near("dgate", dgate, rz, np.abs(rz).max() + 1, 4 * tol)
    else:
        assert dgate is None
    terms = B * L * max(1.0, float(np.abs(o[4]).mean())) * 4
    near("dgamma", dgamma, rg, terms, 2.0 ** -16)
    near("dbeta", dbeta, rb, terms, 2.0 ** -16)


@pytest.mark.parametrize("shape", [(1, 1, 1, 8), (2, 3, 5, 16), (1, 8, 1, 64), (3, 5, 33, 48), (2, 2, 130, 96),
                                   (1, 3, 70, 128), (2, 1, 9, 200), (1, 2, 17, 256), (7, 16, 1, 24)], ids=str)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("gate", [True, False])
def test_shapes(shape, dtype, gate):
    check(*shape, dtype, "silu", gate, sum(shape))


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_activations(act, gate, dtype):
    check(2, 4, 40, 64, dtype, act, gate, 3)


def test_large_mean():
    """The deviation is taken from differences to the mean: a mean of 60 deviations costs its own 2^-24 only."""
    check(2, 3, 20, 64, torch.float32, "none", False, 4, shift=20.0)


def test_many_rows():
    check(4, 3, 3000, 32, torch.bfloat16, "silu", True, 5)


def test_constant_rows_and_extremes():
    x, gamma, beta, z, do = make(1, 2, 4, 32, torch.bfloat16, True, 6)
    x[:, :, 1] = 3.0                                      # no deviation: n = 0, out = beta act(gate)
    z[0, 2] = -1e4                                        # silu of a gate far out is 0, of one far up itself
    z[0, 3] = 1e4
    kw = dict(gate=z.cuda(), act="silu")
    out = fw.fw_group_norm_act(x.cuda(), gamma.cuda(), beta.cuda(), **kw)
    got = fw.fw_group_norm_act_backward(x.cuda(), gamma.cuda(), beta.cuda(), do.cuda(), **kw)
    assert torch.isfinite(out).all() and all(torch.isfinite(t).all() for t in got)
    assert torch.all(out[0, 2] == 0)
    want = (beta * (z[0, 1].float() * torch.sigmoid(z[0, 1].float()))).cuda()
    assert torch.all((out[0, 1].float() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-6)


def test_nan_stays_in_its_row():
    x, gamma, beta, _, _ = make(2, 2, 4, 32, torch.float32, False, 7)
    x[1, 0, 2, 5] = float("nan")
    for act in ("none", "relu"):
        out = fw.fw_group_norm_act(x.cuda(), gamma.cuda(), beta.cuda(), act=act).view(2, 4, 2, 32)
        assert torch.isnan(out[1, 2, 0]).all()
        out[1, 2, 0] = 0
        assert torch.isfinite(out).all()


def test_empty_and_refused():
    x, gamma, beta, z, do = (t.cuda() for t in make(2, 2, 4, 32, torch.bfloat16, True, 8))
    assert fw.fw_group_norm_act(x[:0], gamma, beta).shape == (0, 4, 64)
    got = fw.fw_group_norm_act_backward(x[:0], gamma, beta, do[:0])
    assert torch.all(got[2] == 0) and torch.all(got[3] == 0)
    for bad in (dict(gate=z.float()), dict(gate=z[:, :3]), dict(act="tanh"), dict(out=torch.empty_like(x))):
        with pytest.raises(ValueError):
            fw.fw_group_norm_act(x, gamma, beta, **bad)
    with pytest.raises(ValueError):
        fw.fw_group_norm_act(x.transpose(1, 2), gamma, beta)
    with pytest.raises(ValueError):
        fw.fw_group_norm_act(x, gamma.bfloat16(), beta)


def test_a_layer_end_to_end():
    """DPFP features, the gated rule, the norm and its gate, and all gradients
    back through the three; then the same tokens one at a time; then the
    forward as a graph."""
    from oracle import dpfp
    B, H, L, d_key, d_v = 2, 2, 70, 32, 32
    r = torch.Generator().manual_seed(9)
    n = lambda *s: torch.randn(*s, generator=r)  # noqa: E731
    q0, k0 = (n(B, H, L, d_key).bfloat16().cuda() for _ in range(2))
    v, z = n(B, H, L, d_v).bfloat16().cuda(), n(B, L, H * d_v).bfloat16().cuda()
    g = (-0.1 * torch.rand(B, H, L, generator=r)).bfloat16().cuda()
    be = torch.rand(B, H, L, generator=r).bfloat16().cuda()
    gamma, beta = (1 + 0.1 * n(H * d_v)).cuda(), (0.1 * n(H * d_v)).cuda()
    do = n(B, L, H * d_v).bfloat16().cuda()

    def forward():
        q, k = fw.fw_dpfp(q0, nu=1), fw.fw_dpfp(k0, nu=1)
        y, W = fw.fw_gated_delta_forward(q, k, v, g, be, l2norm=True)
        return q, k, y, W, fw.fw_group_norm_act(y, gamma, beta, gate=z, act="silu")

    q, k, y, W, out = forward()
    assert torch.isfinite(out).all()
    # each stage against the oracle on that stage's own bf16 inputs
    qf = dpfp(f64(q0), 1, 1e-6)
    assert np.abs(f64(q) - qf).max() <= 2.0 ** -8 * np.abs(qf).max() + 1e-6
    yr, Wr = gated.gated_forward(f64(q), f64(k), f64(v), f64(g), f64(be))
    assert np.abs(f64(y) - yr).max() <= 2.0 ** -7 * np.abs(yr).max()
    near("out", out, gated.group_norm_act(f64(y), f64(gamma), f64(beta), f64(z), "silu"), 4.0, 2.0 ** -17)
    dy, dz, dgamma, dbeta = fw.fw_group_norm_act_backward(y, gamma, beta, do, gate=z, act="silu")
    got = fw.fw_gated_delta_backward(q, k, v, g, be, dy, return_dW0=False)
    want = gated.gated_backward(f64(q), f64(k), f64(v), f64(g), f64(be), f64(dy))
    for a, w in zip(got[:5], want):
        assert np.all(np.abs(f64(a) - w) <= 2.0 ** -8 * np.abs(w) + 2.0 ** -11 * np.abs(w).max())
    # token by token: the norm of one token's answers is the sequence's row
    S = torch.zeros_like(W)
    for t in range(3):
        yt = fw.fw_gated_delta_decode_step(q[:, :, t].contiguous(), k[:, :, t].contiguous(), v[:, :, t].contiguous(),
                                           g[:, :, t].contiguous(), be[:, :, t].contiguous(), S)
        ot = fw.fw_group_norm_act(yt[:, :, None], gamma, beta, gate=z[:, t:t + 1].contiguous(), act="silu")
        assert torch.all((ot.float() - out[:, t:t + 1].float()).abs() <= 0.05)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = forward()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(again[4], out) and torch.equal(again[3], W)


def sizes_of_terms(x, gamma, beta, z, do, act, eps):
    """Per channel, the sums of |dz| (|n| + 1) over the tokens: what dgamma and dbeta add up."""
    x, gamma, beta, z, do = (None if t is None else f64(t) for t in (x, gamma, beta, z, do))
    B, H, L, d = x.shape
    c = x - x.mean(-1, keepdims=True)
    n = (c / np.sqrt((c * c).mean(-1, keepdims=True) + eps)).transpose(0, 2, 1, 3)
    f, df = gated._act(n * gamma.reshape(H, d) + beta.reshape(H, d) if z is None else z.reshape(B, L, H, d), act)
    dz = do.reshape(B, L, H, d) * (df if z is None else f)
    return (np.abs(dz) * (np.abs(n) + 1)).sum((0, 1)).reshape(-1)


# dgamma and dbeta: a term is off by 2^-19 of |dz| (|n| + 1) (the mean's 13 2^-24 of twice the deviation,
# the root, the activation), and goes through at most 300 additions of 2^-24 each: 2^-15 of the terms' sizes.
TERMS = 2.0 ** -15


@pytest.mark.parametrize("shape", [(1, 1, 1, 8), (1, 2, 63, 32), (1, 2, 64, 32), (1, 2, 65, 32), (1, 2, 129, 32), (2, 3, 130, 48),
                                   (3, 2, 70, 256), (5, 1, 700, 128)], ids=str)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("act, gate", [("none", False), ("silu", False), ("gelu", False), ("silu", True)])
def test_without_eps(shape, dtype, act, gate):
    """eps 0: rows past the last one have no deviation and no part in the sums over the rows."""
    x, gamma, beta, z, do = make(*shape, dtype, gate, sum(shape))
    dv = lambda t: None if t is None else t.cuda()  # noqa: E731
    kw = dict(act=act, gate=dv(z), eps=0.0)
    out = fw.fw_group_norm_act(dv(x), dv(gamma), dv(beta), **kw)
    dx, dgate, dgamma, dbeta = fw.fw_group_norm_act_backward(dv(x), dv(gamma), dv(beta), dv(do), **kw)
    o = [None if t is None else f64(t) for t in (x, gamma, beta, z)]
    ref = gated.group_norm_act(*o, act, eps=0.0)
    rx, rz, rg, rb = gated.group_norm_act(*o, act, eps=0.0, dout=f64(do))
    tol = 2.0 ** -18 + 2.0 ** -24 * 64
    near("out", out, ref, np.abs(ref).max() + 1, tol)
    # dx of a row is of the size of what goes into it, over the row's deviation
    c = o[0] - o[0].mean(-1, keepdims=True)
    near("dx", dx, rx, np.abs(f64(do)).max() * np.abs(o[1]).max() * 4 / np.sqrt((c * c).mean(-1, keepdims=True)), 8 * tol)
    if gate:
        near("dgate", dgate, rz, np.abs(rz).max() + 1, 4 * tol)
    big = sizes_of_terms(x, gamma, beta, z, do, act, 0.0)
    near("dgamma", dgamma, rg, big, TERMS)
    near("dbeta", dbeta, rb, big, TERMS)


@pytest.mark.parametrize("shape", [(4, 3, 3000, 32), (2, 5, 1111, 96), (1, 1, 9000, 8)], ids=str)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("act, gate", [("none", False), ("gelu", False), ("silu", True)])
def test_parameters_by_the_terms(shape, dtype, act, gate):
    x, gamma, beta, z, do = make(*shape, dtype, gate, sum(shape))
    dv = lambda t: None if t is None else t.cuda()  # noqa: E731
    _, _, dgamma, dbeta = fw.fw_group_norm_act_backward(dv(x), dv(gamma), dv(beta), dv(do), act=act, gate=dv(z))
    o = [None if t is None else f64(t) for t in (x, gamma, beta, z)]
    _, _, rg, rb = gated.group_norm_act(*o, act, dout=f64(do))
    big = sizes_of_terms(x, gamma, beta, z, do, act, 1e-5)
    near("dgamma", dgamma, rg, big, TERMS)
    near("dbeta", dbeta, rb, big, TERMS)


@pytest.mark.parametrize("row", [0, 63, 64, 2431, 2432, 2495, 4863, 4864, 4868])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_one_row_alone(row, dtype):
    """Only one token has a gradient: the parameters' are its terms, once, and
    no other row gets any (8 heads of 32 channels: 64 rows a CTA, 38 CTAs a head)."""
    B, H, L, d = 1, 8, 4869, 32
    x, gamma, beta, _, do = make(B, H, L, d, dtype, False, 11)
    only = torch.zeros_like(do)
    only[:, row] = do[:, row]
    dx, _, dgamma, dbeta = fw.fw_group_norm_act_backward(x.cuda(), gamma.cuda(), beta.cuda(), only.cuda())
    o = [f64(x), f64(gamma), f64(beta), None]
    _, _, rg, rb = gated.group_norm_act(*o, "none", dout=f64(only))
    big = sizes_of_terms(x, gamma, beta, None, only, "none", 1e-5)
    near("dgamma", dgamma, rg, big, TERMS)
    near("dbeta", dbeta, rb, big, TERMS)
    assert torch.all(dx[:, :, row] != 0)
    dx[:, :, row] = 0
    assert torch.all(dx == 0)


def test_offsets_past_32_bits():
    """More than 2^31 values: the last tokens have the bits of a call of their own."""
    H, L, d = 16, 1100003, 128
    if torch.cuda.mem_get_info()[0] < 60e9:
        pytest.skip("needs 40 GB")
    r = torch.Generator(device="cuda").manual_seed(12)
    x = torch.randn(1, H, L, d, generator=r, device="cuda", dtype=torch.bfloat16)
    gate = torch.randn(1, L, H * d, generator=r, device="cuda", dtype=torch.bfloat16)
    gamma, beta = (torch.randn(H * d, generator=r, device="cuda") for _ in range(2))
    assert x.numel() > 2 ** 31
    out = fw.fw_group_norm_act(x, gamma, beta, gate=gate, act="silu")
    dx, dgate, dgamma, _ = fw.fw_group_norm_act_backward(x, gamma, beta, out, gate=gate, act="silu")
    assert torch.isfinite(dgamma).all()
    for s in (slice(0, 500), slice(L - 500, L)):
        xs, zs, os = x[:, :, s].contiguous(), gate[:, s].contiguous(), out[:, s].contiguous()
        assert torch.equal(fw.fw_group_norm_act(xs, gamma, beta, gate=zs, act="silu"), os)
        dxs, dzs, _, _ = fw.fw_group_norm_act_backward(xs, gamma, beta, os, gate=zs, act="silu")
        assert torch.equal(dx[:, :, s], dxs) and torch.equal(dgate[:, s], dzs)
    del x, gate, out, dx, dgate
    torch.cuda.empty_cache()
