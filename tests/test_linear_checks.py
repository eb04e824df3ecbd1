"""Argument checks of the linear map and the checkpoints, through the C ABI and
through the binding, and the float64 statement they are held to (no GPU: every
refusal returns before any CUDA call)."""
import ctypes as C

import numpy as np
import pytest
import torch

from dynamic_block_sparse_stats_b200 import _lib, api
from oracle import linear_oracle as L

OK = C.c_void_p(256)
BAD = _lib.PRISM_ERR_INVALID_ARG


def _lin(n=16, i=64, o=128, act=0):
    return C.byref(_lib.PrismLinear(n, i, o, act))


def _ck(ld=128, codes=256, scales=256):
    return C.byref(_lib.PrismCkpt8(codes, scales, ld))


def _fwd(lin=None, X=OK, ldx=64, W=OK, bias=OK, R=None, ldr=0, Y=OK, ldy=128, Z=None, Z8=None, ws=OK, size=256):
    return _lib.load().prism_linear_fwd(lin if lin is not None else _lin(), X, ldx, W, bias, R, ldr, Y, ldy, Z, Z8, ws,
                                        size, None)


def _bwd(lin=None, dY=OK, lddy=128, X=OK, ldx=64, X8=None, W=OK, Z=None, ldz=0, Z8=None, dX=OK, dW=OK, db=OK, fp32=0,
         ws=OK, size=1 << 40):
    return _lib.load().prism_linear_bwd(lin if lin is not None else _lin(), dY, lddy, X, ldx, X8, W, Z, ldz, Z8, dX,
                                        dW, db, fp32, ws, size, None)


def test_struct_layouts():
    assert C.sizeof(_lib.PrismCkpt8) == 24 and C.sizeof(_lib.PrismLinear) == 24


@pytest.mark.parametrize("kw", [dict(n=-1), dict(n=1 << 30), dict(i=0), dict(i=12), dict(i=1 << 17), dict(o=-8), dict(o=4),
                                dict(act=4), dict(act=-1)])
def test_bad_descriptions(kw):
    lib = _lib.load()
    for backward in (0, 1, 2):
        assert lib.prism_linear_workspace_size(_lin(**kw), backward) == 0
    assert _fwd(_lin(**kw)) == BAD and _bwd(_lin(**kw)) == BAD
    assert "linear" in lib.prism_last_error().decode()
    assert lib.prism_linear_workspace_size(None, 0) == 0


def test_sizes_past_2_40_values():
    big = _lin(n=(1 << 30) - 8, i=64, o=1 << 16)
    assert _lib.load().prism_linear_workspace_size(big, 1) == 0
    assert _fwd(big, ldy=1 << 16) == _lib.PRISM_ERR_UNSUPPORTED
    assert _bwd(big, lddy=1 << 16) == _lib.PRISM_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(X=None), dict(W=None), dict(Y=None), dict(ldx=56), dict(ldx=68), dict(ldy=120),
                                dict(ldy=132), dict(X=C.c_void_p(264)), dict(W=C.c_void_p(264)), dict(bias=C.c_void_p(264)),
                                dict(Y=C.c_void_p(264)), dict(R=OK, ldr=64), dict(R=C.c_void_p(258), ldr=128),
                                dict(Z=C.c_void_p(264)), dict(Z=OK, Z8=_ck()), dict(Z8=_ck(ld=256)), dict(Z8=_ck(ld=64)),
                                dict(Z8=_ck(codes=264)), dict(Z8=_ck(scales=258)), dict(Z8=_ck(codes=None)), dict(ws=None),
                                dict(ws=C.c_void_p(264))])
def test_forward_refusals(kw):
    assert _fwd(**kw) == BAD


@pytest.mark.parametrize("kw", [dict(dY=None), dict(W=None), dict(X=None), dict(X8=_ck()), dict(X=None, X8=_ck(ld=64)),
                                dict(dX=None, dW=None, db=None), dict(fp32=2), dict(lddy=64), dict(ldx=60),
                                dict(lin=_lin(act=1)), dict(lin=_lin(act=2), Z=OK, ldz=128, Z8=_ck()),
                                dict(lin=_lin(act=2), Z=OK, ldz=64), dict(dX=C.c_void_p(264)), dict(dW=C.c_void_p(264)),
                                dict(db=C.c_void_p(264)), dict(dY=C.c_void_p(264)), dict(ws=None)])
def test_backward_refusals(kw):
    assert _bwd(**kw) == BAD


def test_workspaces():
    lib = _lib.load()
    assert lib.prism_linear_workspace_size(_lin(), 0) == 256
    assert _fwd(size=255) == _lib.PRISM_ERR_CAPACITY
    plain = lib.prism_linear_workspace_size(_lin(n=4096, i=512, o=256), 1)
    act = lib.prism_linear_workspace_size(_lin(n=4096, i=512, o=256, act=3), 1)
    assert act - plain == 2 * 4096 * 256          # dZ
    assert _bwd(_lin(n=4096, i=512, o=256), lddy=256, ldx=512, size=plain - 1) == _lib.PRISM_ERR_CAPACITY
    x8 = lib.prism_linear_workspace_size(_lin(n=4096, i=512, o=2048), 2)
    assert x8 >= lib.prism_linear_workspace_size(_lin(n=4096, i=512, o=2048), 1) + 2 * 4096 * 512   # X restored
    assert lib.prism_linear_workspace_size(_lin(), 3) == 0
    assert api.linear_workspace_size(4096, 512, 2048, backward=True, x8=True) == x8
    assert api.linear_workspace_size(4096, 512, 256, api.ACT_GELU, True) == act
    with pytest.raises(_lib.PrismError):
        api.linear_workspace_size(4096, 12, 256)


@pytest.mark.parametrize("kw", [dict(n=-1), dict(n=1 << 31), dict(width=12), dict(width=0), dict(ld=56), dict(ld=68),
                                dict(x=C.c_void_p(264)), dict(x=None), dict(c=None), dict(c=_ck(ld=256)),
                                dict(c=_ck(ld=64)), dict(c=_ck(codes=264)), dict(c=_ck(scales=258))])
def test_checkpoint_refusals(kw):
    a = dict(x=OK, n=4, width=64, ld=64, c=_ck())
    a.update(kw)
    lib = _lib.load()
    assert lib.prism_ckpt8_pack(a["x"], a["n"], a["width"], a["ld"], a["c"], None) == BAD
    assert lib.prism_ckpt8_unpack(a["c"], a["n"], a["width"], a["x"], a["ld"], None) == BAD
    assert "ckpt8" in lib.prism_last_error().decode()


def test_empty_checkpoint_calls_need_no_gpu():
    lib = _lib.load()
    assert lib.prism_ckpt8_pack(None, 0, 64, 64, _ck(codes=None, scales=None), None) == _lib.PRISM_OK
    assert lib.prism_ckpt8_unpack(_ck(codes=None, scales=None), 0, 64, None, 64, None) == _lib.PRISM_OK


# ------------------------------------------------------------------------------------------------ binding
def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def _same(n=4, c=8):
    t = _t(n, c)
    return t, t


def _fwd_onto_itself():
    x, y = _same()
    return api.linear_fwd(x, _t(8, 8), Y=y)


def _bwd_onto_itself():
    dy, dx = _same()
    return api.linear_bwd(dy, _t(4, 8), _t(8, 8), out=(dx, None, None))


def test_outputs_onto_inputs_are_refused():
    for call in (_fwd_onto_itself, _bwd_onto_itself):
        with pytest.raises(ValueError, match="may not be"):
            call()


@pytest.mark.parametrize("make,err", [
    (lambda: api.linear_fwd(_t(4, 8), _t(16, 16)), ValueError),
    (lambda: api.linear_fwd(_t(4, 8, dtype=torch.float32), _t(16, 8)), ValueError),
    (lambda: api.linear_fwd(_t(4, 2, 8), _t(16, 8)), ValueError),
    (lambda: api.linear_fwd([[1.0]], _t(16, 8)), TypeError),
    (lambda: api.linear_fwd(_t(8, 4).t(), _t(16, 8)), ValueError),
    (lambda: api.linear_fwd(_t(1, 8).expand(4, 8), _t(16, 8)), ValueError),
    (lambda: api.linear_fwd(_t(4, 8), _t(8, 16).t()), ValueError),
    (lambda: api.linear_fwd(_t(4, 8), _t(16, 8), bias=_t(8)), ValueError),
    (lambda: api.linear_fwd(_t(4, 8), _t(16, 8), residual=_t(4, 8)), ValueError),
    (lambda: api.linear_fwd(_t(4, 8), _t(16, 8), Y=_t(5, 16)), ValueError),
    (lambda: api.linear_fwd(_t(4, 8), _t(16, 8), save="fp8"), ValueError),
    (lambda: api.linear_fwd(_t(4, 8), _t(16, 8), Z=_t(4, 16)), ValueError),
    (lambda: api.linear_fwd(_t(4, 8), _t(16, 8), save="ckpt8", Z=_t(4, 16)), TypeError),
    (lambda: api.linear_fwd(_t(4, 8), _t(16, 8), ws=_t(256)), ValueError),
    (lambda: api.linear_fwd(_t(4, 8), _t(16, 8)), ValueError),                      # CPU tensors
    (lambda: api.linear_bwd(_t(4, 16), _t(4, 8), _t(8, 16)), ValueError),
    (lambda: api.linear_bwd(_t(4, 16), _t(5, 8), _t(16, 8)), ValueError),
    (lambda: api.linear_bwd(_t(4, 16), None, _t(16, 8)), ValueError),
    (lambda: api.linear_bwd(_t(4, 16), [[1.0]], None, need=("dW",)), TypeError),
    (lambda: api.linear_bwd(_t(4, 16), _t(4, 8), _t(16, 8), need=("dX", "dX")), ValueError),
    (lambda: api.linear_bwd(_t(4, 16), _t(4, 8), None), ValueError),
    (lambda: api.linear_bwd(_t(4, 16), _t(4, 8), _t(16, 8), act=api.ACT_GELU), ValueError),
    (lambda: api.linear_bwd(_t(4, 16), _t(4, 8), _t(16, 8), _t(4, 8), api.ACT_GELU), ValueError),
    (lambda: api.linear_bwd(_t(4, 16), _t(4, 8), _t(16, 8), need=()), ValueError),
    (lambda: api.linear_bwd(_t(4, 16), _t(4, 8), _t(16, 8), need=("dR",)), ValueError),
    (lambda: api.linear_bwd(_t(4, 16), _t(4, 8), _t(16, 8), out=(None, _t(16, 8))), ValueError),
    (lambda: api.linear_bwd(_t(4, 16), _t(4, 8), _t(16, 8), grad_fp32=True, out=(None, _t(16, 8), None)), ValueError),
    (lambda: api.linear_bwd(_t(4, 16), _t(4, 8), _t(16, 8), need=("dX",), out=(None, _t(16, 8), None)), ValueError),
    (lambda: api.linear_bwd(_t(4, 16), api.alloc_ckpt8(4, 16, "cpu"), _t(16, 8)), ValueError),
    (lambda: api.linear_bwd(_t(4, 16), api.alloc_ckpt8(5, 8, "cpu"), _t(16, 8)), ValueError),
    (lambda: api.ckpt8_pack(_t(4, 8, dtype=torch.float16)), ValueError),
    (lambda: api.ckpt8_pack(_t(4, 8)), ValueError),
    (lambda: api.ckpt8_unpack(_t(4, 8)), TypeError),
    (lambda: api.ckpt8_unpack(api.alloc_ckpt8(4, 8, "cpu"), out=_t(4, 16)), ValueError),
    (lambda: api.ckpt8_unpack(api.Ckpt8(_t(4, 64, dtype=torch.int8), _t(4, 2, dtype=torch.uint8), 64)), ValueError),
])
def test_binding_refuses(make, err):
    with pytest.raises(err):
        make()


# ------------------------------------------------------------------------------------------------ oracle
@pytest.mark.parametrize("kind", [L.NONE, L.RELU, L.SILU, L.GELU])
def test_oracle_gradients_against_differences(kind):
    """Central differences of sum(dY * Y) along random directions; step 1e-5 of
    order-one values in float64: truncation ~1e-10, rounding ~1e-11."""
    r = np.random.default_rng(kind)
    X, W, b, dY = r.normal(size=(9, 6)), r.normal(size=(5, 6)), r.normal(size=5), r.normal(size=(9, 5))
    Z, _ = L.forward(X, W, b, kind)
    _, dX, dW, db = L.backward(dY, X, W, Z, kind)
    f = lambda X, W, b: (dY * L.forward(X, W, b, kind)[1]).sum()  # noqa: E731
    h = 1e-5
    for i, g in enumerate((dX, dW, db)):
        d = r.normal(size=g.shape)
        a = [X, W, b]
        up, dn = list(a), list(a)
        up[i], dn[i] = a[i] + h * d, a[i] - h * d
        assert abs((f(*up) - f(*dn)) / (2 * h) - (g * d).sum()) < 1e-7


def test_oracle_checkpoint_by_hand():
    x = np.zeros((1, 40))
    x[0, :4] = [127.0, 0.5, 1.5, -2.5]         # scale 1: ties to even
    x[0, 32] = 127.5                           # scale 2
    c, s = L.ckpt8_pack(x)
    assert c.shape == (1, 128) and s.shape == (1, 4)
    assert list(c[0, :4]) == [127, 0, 2, -2] and s[0, 0] == 127
    assert c[0, 32] == 64 and s[0, 1] == 128
    assert s[0, 2] == 1                        # an empty block
    v = L.ckpt8_unpack(c, s, 40)
    assert v[0, 32] == 128.0 and v[0, 2] == 2.0
