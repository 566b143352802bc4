"""Refusals of the embedding's, the layer norm's and the vocabulary loss's
entry points (host only: every call fails its checks before any CUDA call)."""
import ctypes

import pytest

from delta_rule_linear_dpfp_gb300 import binding, build

FAKE, MISALIGNED, ODD = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008), ctypes.c_void_p(0x10002)
TO, TO2 = ctypes.c_void_p(0x20000), ctypes.c_void_p(0x30000)  # outputs
E, U, OK = binding.FW_ERR_INVALID_ARG, binding.FW_ERR_UNSUPPORTED, binding.FW_OK


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def _call(fn, base):
    def call(**kw):
        assert set(kw) <= set(base)
        return fn(*{**base, **kw}.values())
    return call


def test_embedding_refusals(lib):
    call = _call(lib.fw_embedding, dict(ids=FAKE, table=FAKE, out=TO, N=5, V=9, D=64, scale=1.0, index=1, io=1, st=None))
    need = lib.fw_embedding_backward_workspace_size(5, 9, 64)
    assert need > 0
    back = _call(lib.fw_embedding_backward,
                 dict(ids=FAKE, dout=FAKE, dtable=TO, ws=FAKE, wsb=need, N=5, V=9, D=64, scale=1.0, acc=0, index=1, io=1,
                      st=None))
    for n in ("table", "out"):
        assert call(**{n: None}) == E and call(**{n: MISALIGNED}) == E, n
    for n in ("dout", "dtable", "ws"):
        assert back(**{n: None}) == E and back(**{n: MISALIGNED}) == E, n
    for c in (call, back):
        assert c(ids=None) == E and c(ids=ODD) == E and c(ids=ODD, index=0) == E and c(index=2) == E and c(io=2) == E
        assert c(N=-1) == E and c(V=0) == E and c(D=0) == E and c(scale=float("nan")) == E and c(scale=float("inf")) == E
        assert c(D=12) == U and c(D=65544) == U and c(V=2**31 - 1) == U and c(N=2**40) == U
    assert back(wsb=need - 1) == E and back(acc=2) == E and back(N=2**31 - 1) == U
    assert call(out=FAKE) == E                                   # the table itself
    assert call(N=0, ids=None, table=None, out=None) == OK
    assert back(N=0, ids=None, dout=None, ws=None, wsb=0, acc=1) == OK and back(N=0, dtable=None) == E


def test_layer_norm_refusals(lib):
    call = _call(lib.fw_layer_norm, dict(x=FAKE, res=None, gamma=FAKE, beta=FAKE, out=TO, sum=None, rows=5, d=64, eps=1e-5,
                                         io=1, st=None))
    need = lib.fw_layer_norm_backward_workspace_size(5, 64)
    assert need > 0
    back = _call(lib.fw_layer_norm_backward,
                 dict(x=FAKE, gamma=FAKE, dout=FAKE, dsum=None, dx=FAKE, dgamma=FAKE, dbeta=FAKE, ws=FAKE, wsb=need, rows=5,
                      d=64, eps=1e-5, io=1, st=None))
    for n in ("x", "out"):
        assert call(**{n: None}) == E and call(**{n: MISALIGNED}) == E, n
    for n in ("x", "dout", "dx", "ws"):
        assert back(**{n: None}) == E and back(**{n: MISALIGNED}) == E, n
    for n in ("gamma", "beta"):
        assert call(**{n: MISALIGNED}) == E, n
    assert call(res=MISALIGNED, sum=FAKE) == E and call(res=FAKE, sum=MISALIGNED) == E
    assert call(res=FAKE) == E and call(sum=FAKE) == E           # sum goes with residual
    assert call(res=FAKE, sum=TO) == E                           # two outputs in one place
    for n in ("gamma", "dsum", "dgamma", "dbeta"):
        assert back(**{n: MISALIGNED}) == E, n
    assert back(dgamma=None) == E and back(dbeta=None) == E and back(wsb=need - 1) == E
    for c in (call, back):
        assert c(rows=-1) == E and c(d=0) == E and c(io=2) == E and c(eps=-1.0) == E and c(eps=float("nan")) == E
        assert c(d=12) == U and c(d=8200) == U
    assert call(rows=0, x=None, out=None) == OK and back(rows=0, x=None, dgamma=None, dbeta=None, ws=None, wsb=0) == OK


@pytest.mark.parametrize("io", [0, 1])
def test_vocab_loss_refusals(lib, io):
    need = lib.fw_vocab_loss_workspace_size(5, 9, 64, io)
    call = _call(lib.fw_vocab_loss, dict(h=FAKE, W=FAKE, bias=None, targets=FAKE, loss=FAKE, lse=FAKE, ws=FAKE, wsb=need, N=5,
                                         V=9, D=64, index=1, io=io, st=None))
    bneed = lib.fw_vocab_loss_backward_workspace_size(5, 9, 64, io)
    back = _call(lib.fw_vocab_loss_backward,
                 dict(h=FAKE, W=FAKE, bias=None, targets=FAKE, loss=FAKE, lse=FAKE, dloss=FAKE, dh=TO, dW=TO2, dbias=None,
                      ws=FAKE, wsb=bneed, N=5, V=9, D=64, index=1, io=io, st=None))
    assert need > 0 and bneed > need
    for c, more in ((call, ()), (back, ("dloss",))):
        for n in ("h", "W", "loss", "lse", "ws", *more):
            assert c(**{n: None}) == E and c(**{n: MISALIGNED}) == E, n
        assert c(bias=MISALIGNED) == E and c(targets=None) == E and c(targets=ODD) == E and c(index=7) == E and c(io=2) == E
        assert c(N=-1) == E and c(V=0) == E and c(D=0) == E and c(D=20) == U and c(D=65544) == U
        assert c(N=2**31 - 1) == U and c(V=2**31 - 1) == U and c(N=2**30, V=2**30) == U
    for n in ("dh", "dW", "dbias"):
        assert back(**{n: MISALIGNED}) == E, n
    assert call(wsb=need - 1) == E and back(wsb=bneed - 1) == E
    assert back(dh=FAKE) == E and back(dW=FAKE) == E             # the inputs themselves
    assert call(N=0, h=None, targets=None, loss=None, lse=None, ws=None, wsb=0) == OK
    assert back(N=0, h=None, targets=None, dW=None, ws=None, wsb=0) == OK


def test_workspace_queries(lib):
    f = lib.fw_embedding_backward_workspace_size
    assert f(5, 9, 12) == 0 and f(0, 9, 16) == 0 and f(-1, 9, 16) == 0 and f(2**31 - 1, 9, 16) == 0 and f(1, 1, 8) > 0
    assert f(10**9, 9, 1024) > 2**37                      # 32-bit sums of every 32 rows: past 32 bits of bytes
    f = lib.fw_layer_norm_backward_workspace_size
    assert f(5, 12) == 0 and f(0, 16) == 0 and f(2**40, 8192) == f(2**20, 8192) > 0
    f = lib.fw_vocab_loss_backward_workspace_size
    for io in (0, 1):
        assert f(5, 9, 12, io) == 0 and f(0, 9, 16, io) == 0 and f(1, 1, 8, io) > 0 and f(1, 1, 8, 2) == 0
        assert f(8192, 10**6, 512, io) < 2**31 < 2 * 8192 * 10**6      # pieces of the vocabulary
    f = lib.fw_vocab_loss_workspace_size
    assert f(8192, 10**6, 512, 1) < 2**31 and f(2**20, 2**16, 512, 1) > 2**32 and f(1, 1, 8, 0) > 0 == f(1, 1, 8, 2)
