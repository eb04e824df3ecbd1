"""Outputs of the linear map that would share memory with what the call reads, or
with one another, are refused by the library before anything is launched.  (No
GPU: addresses are made up, and every call here is a refused one.)"""
import ctypes as C

import pytest

from dynamic_block_sparse_stats_b200 import _lib

N, IN, OUT = 16, 128, 128                      # every matrix below is 4096 bytes, a checkpoint 2048 + 64
BIG = 1 << 20


def _at(k, off=0):
    """The k-th of many buffers, a megabyte apart."""
    return C.c_void_p((k + 1) * BIG + off)


def _ck(k, off=0):
    return C.byref(_lib.PrismCkpt8((k + 1) * BIG + off, (k + 1) * BIG + BIG // 2 + off, OUT))


def _said(rc, *names):
    msg = _lib.load().prism_last_error().decode()
    assert rc == _lib.PRISM_ERR_INVALID_ARG and "overlap" in msg and all(n in msg for n in names), (rc, msg)


def _fwd(n=N, X=_at(0), ldx=IN, W=_at(1), bias=_at(2), R=_at(3), ldr=OUT, Y=_at(4), ldy=OUT, Z=_at(5), Z8=None, ws=_at(6)):
    return _lib.load().prism_linear_fwd(C.byref(_lib.PrismLinear(n, IN, OUT, 0)), X, ldx, W, bias, R, ldr, Y, ldy, Z, Z8,
                                        ws, 256, None)


@pytest.mark.parametrize("kw,names", [
    (dict(Y=_at(0)), ("Y", "X")),
    (dict(Y=_at(0, 4096 - 16)), ("Y", "X")),           # the first bytes of Y in the last of X
    (dict(Y=_at(0, -4096 + 16)), ("Y", "X")),
    (dict(Y=_at(1)), ("Y", "W")),
    (dict(Y=_at(1, 2 * IN * OUT - 16)), ("Y", "W")),
    (dict(Y=_at(2, -16)), ("Y", "bias")),
    (dict(Y=_at(3), ldy=OUT + 8), ("Y", "R")),          # the residual's address with another stride
    (dict(Y=_at(3, 16)), ("Y", "R")),
    (dict(Y=_at(3, 2 * OUT)), ("Y", "R")),              # a row further on
    (dict(Z=_at(0)), ("Z", "X")),
    (dict(Z=_at(1)), ("Z", "W")),
    (dict(Z=_at(2)), ("Z", "bias")),
    (dict(Z=_at(3)), ("Z", "R")),
    (dict(Z=_at(4)), ("Z", "Y")),
    (dict(Z=_at(3), Y=_at(3)), ("Z", "R")),
    (dict(Z=None, Z8=_ck(0)), ("Z8", "X")),
    (dict(Z=None, Z8=_ck(4, 4096 - 128)), ("Z8", "Y")),
    (dict(Z=None, Z8=_ck(0, -BIG // 2)), ("Z8", "X")),  # the scales alone
    (dict(ws=_at(0)), ("workspace", "X")),
    (dict(ws=_at(4)), ("workspace", "Y")),
    # column slices of one buffer whose strides agree but whose columns meet
    (dict(X=_at(0), ldx=IN + OUT - 8, Y=_at(0, 2 * (IN - 8)), ldy=IN + OUT - 8), ("Y", "X")),
    (dict(X=_at(0), ldx=256, Y=_at(0, 2 * 200), ldy=256), ("Y", "X")),     # Y's rows run into X's next ones
    (dict(X=_at(0), ldx=256, Y=_at(0, -2 * 56), ldy=256), ("Y", "X")),     # Y begins before X and runs into it
    (dict(X=_at(0), ldx=256, Y=_at(0, 2 * IN), ldy=264), ("Y", "X")),      # strides that differ
    (dict(n=1, Y=_at(3, 16)), ("Y", "R")),
])
def test_forward(kw, names):
    _said(_fwd(**kw), *names)


def _bwd(n=N, act=3, dY=_at(0), X=_at(1), X8=None, W=_at(2), Z=_at(3), Z8=None, dX=_at(4), dW=_at(5), db=_at(6),
         fp32=0, ws=_at(8), size=BIG // 2):
    return _lib.load().prism_linear_bwd(C.byref(_lib.PrismLinear(n, IN, OUT, act)), dY, OUT, X, IN, X8, W, Z, OUT, Z8, dX,
                                        dW, db, fp32, ws, size, None)


@pytest.mark.parametrize("kw,names", [
    (dict(dX=_at(1)), ("dX", "X")),                     # the input's buffer: dW would read dX
    (dict(dX=_at(1, 4096 - 16)), ("dX", "X")),
    (dict(dX=_at(1), X=None, X8=_ck(1)), ("dX", "X8")),
    (dict(dX=_at(1, BIG // 2), X=None, X8=_ck(1)), ("dX", "X8")),
    (dict(dX=_at(0)), ("dX", "dY")),
    (dict(dX=_at(0), act=0), ("dX", "dY")),
    (dict(dX=_at(2)), ("dX", "W")),
    (dict(dX=_at(3)), ("dX", "Z")),
    (dict(dX=_at(3), Z=None, Z8=_ck(3)), ("dX", "Z8")),
    (dict(dW=_at(0)), ("dW", "dY")),
    (dict(dW=_at(1)), ("dW", "X")),
    (dict(dW=_at(2)), ("dW", "W")),
    (dict(dW=_at(2, 2 * IN * OUT - 16)), ("dW", "W")),
    (dict(dW=_at(2, -4 * IN * OUT + 16), fp32=1), ("dW", "W")),
    (dict(dW=_at(3)), ("dW", "Z")),
    (dict(db=_at(0)), ("db", "dY")),
    (dict(db=_at(1)), ("db", "X")),
    (dict(db=_at(2)), ("db", "W")),
    (dict(db=_at(3)), ("db", "Z")),
    (dict(dW=_at(4)), ("dW", "dX")),
    (dict(db=_at(4)), ("db", "dX")),
    (dict(db=_at(5, 4 * IN * OUT - 16), fp32=1), ("db", "dW")),
    (dict(ws=_at(0)), ("workspace", "dY")),
    (dict(ws=_at(5)), ("workspace", "dW")),
])
def test_backward(kw, names):
    _said(_bwd(**kw), *names)


def _pack(x=_at(0), n=N, ld=IN, c=None):
    return _lib.load().prism_ckpt8_pack(x, n, IN, ld, c or _ck(1), None)


def _unpack(x=_at(0), n=N, ld=IN, c=None):
    return _lib.load().prism_ckpt8_unpack(c or _ck(1), n, IN, x, ld, None)


@pytest.mark.parametrize("call", [_pack, _unpack])
@pytest.mark.parametrize("kw", [dict(x=_at(1)), dict(x=_at(1, BIG // 2)), dict(x=_at(1, 2048 - 16)), dict(x=_at(1, -4096 + 16)),
                                dict(x=_at(1, -512 * 8), ld=256), dict(x=_at(1, 2048 - 16), n=1 << 12, ld=1 << 20)])
def test_checkpoints(call, kw):
    _said(call(**kw), "ckpt8")


@pytest.mark.parametrize("call", [_pack, _unpack])
def test_codes_on_their_scales(call):
    _said(call(c=C.byref(_lib.PrismCkpt8(2 * BIG, 2 * BIG + 1024, OUT))), "ckpt8")
