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


# ------------------------------------------------------------- shared memory
def _spread(fn, args, nbytes):
    """A call whose tensors lie apart from one another, and each one's address by name; `nbytes`: their sizes."""
    at = {n: 0x100000 * (i + 1) for i, n in enumerate(nbytes)}
    ptr = {n: ctypes.c_void_p(a) for n, a in at.items()}

    def call(**kw):
        assert set(kw) <= set(args)
        return fn(*{**args, **ptr, **kw}.values())
    return call, at


def _refused(call, at, nbytes, out, allowed=(), with_=None):
    """Each output on each other tensor: at its start, at its last 16 bytes, and with its own last 16 on the start."""
    with_ = with_ or {}
    for o in out:
        for n in nbytes:
            if n == o:
                continue
            for where in (at[n], at[n] + nbytes[n] - 16, at[n] - nbytes[o] + 16):
                if where == at[n] and (o, n) in allowed:
                    continue
                assert call(**{**with_, o: ctypes.c_void_p(where)}) == E, (o, n, hex(where))


@pytest.mark.parametrize("io", [0, 1])
def test_embedding_outputs_apart(lib, io):
    e, N, V, D = 2 if io else 4, 24, 10, 64
    size = dict(ids=8 * N, table=e * V * D, out=e * N * D)
    call, at = _spread(lib.fw_embedding, dict(ids=0, table=0, out=0, N=N, V=V, D=D, scale=1.0, index=1, io=io, st=None), size)
    _refused(call, at, size, ["out"])
    need = lib.fw_embedding_backward_workspace_size(N, V, D)
    size = dict(ids=8 * N, dout=e * N * D, dtable=e * V * D, ws=need)
    call, at = _spread(lib.fw_embedding_backward, dict(ids=0, dout=0, dtable=0, ws=0, wsb=need, N=N, V=V, D=D, scale=1.0, acc=0,
                                                       index=1, io=io, st=None), size)
    for acc in (0, 1):
        _refused(call, at, size, ["dtable", "ws"], with_=dict(acc=acc))


@pytest.mark.parametrize("io", [0, 1])
def test_layer_norm_outputs_apart(lib, io):
    e, rows, d = 2 if io else 4, 24, 64
    row, par = e * rows * d, 4 * d
    size = dict(x=row, res=row, gamma=par, beta=par, out=row, sum=row)
    call, at = _spread(lib.fw_layer_norm, dict(x=0, res=0, gamma=0, beta=0, out=0, sum=0, rows=rows, d=d, eps=1e-5, io=io,
                                               st=None), size)
    _refused(call, at, size, ["out", "sum"], allowed=[(o, n) for o in ("out", "sum") for n in ("x", "res")])
    need = lib.fw_layer_norm_backward_workspace_size(rows, d)
    size = dict(x=row, gamma=par, dout=row, dsum=row, dx=row, dgamma=par, dbeta=par, ws=need)
    call, at = _spread(lib.fw_layer_norm_backward, dict(x=0, gamma=0, dout=0, dsum=0, dx=0, dgamma=0, dbeta=0, ws=0, wsb=need,
                                                        rows=rows, d=d, eps=1e-5, io=io, st=None), size)
    _refused(call, at, size, ["dx", "dgamma", "dbeta", "ws"],
             allowed=[("dx", n) for n in ("x", "dout", "dsum")] + [("dgamma", "gamma")])


@pytest.mark.parametrize("io", [0, 1])
@pytest.mark.parametrize("N", [3, 24])
def test_vocab_loss_outputs_apart(lib, io, N):
    e, V, D = 2 if io else 4, 16, 64
    given = dict(h=e * N * D, W=e * V * D, bias=4 * V, targets=8 * N)
    need = lib.fw_vocab_loss_workspace_size(N, V, D, io)
    size = dict(given, loss=16 * ((4 * N + 15) // 16), lse=16 * ((4 * N + 15) // 16), ws=need)
    call, at = _spread(lib.fw_vocab_loss, dict(h=0, W=0, bias=0, targets=0, loss=0, lse=0, ws=0, wsb=need, N=N, V=V, D=D, index=1,
                                               io=io, st=None), size)
    out = ["loss", "lse", "ws"]
    if N % 4:  # (what ends between two aligned places has none before its end)
        size = {n: b for n, b in size.items() if n in ("loss", "lse", "ws", "h", "W")}
        for o in out:
            for n in size:
                if n != o:
                    assert call(**{o: ctypes.c_void_p(at[n])}) == E, (o, n)
    else:
        _refused(call, at, size, out)
    need = lib.fw_vocab_loss_backward_workspace_size(N, V, D, io)
    size = dict(given, loss=4 * N, lse=4 * N, dloss=4 * N, dh=e * N * D, dW=e * V * D, dbias=4 * V, ws=need)
    call, at = _spread(lib.fw_vocab_loss_backward, dict(h=0, W=0, bias=0, targets=0, loss=0, lse=0, dloss=0, dh=0, dW=0, dbias=0,
                                                        ws=0, wsb=need, N=N, V=V, D=D, index=1, io=io, st=None), size)
    if N % 4 == 0:
        _refused(call, at, size, ["dh", "dW", "dbias", "ws"], allowed=[("dbias", "bias")])
    # without tokens there is nothing to share but the map and its gradient
    assert call(N=0, dW=ctypes.c_void_p(at["W"])) == E
