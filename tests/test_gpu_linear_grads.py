"""The linear map's gradients against difference quotients of the forward formula
in float64, sharp enough that a wrong gradient does not pass: a gradient that is
zero, negated or lacks the activation's slope is held to the same bound, and has
to fail it.

The quotient is taken of
    f(X, W, b) = sum dY * act(Z0 + (X W^T + b - (X W^T + b at the start))),
Z0 the pre-activation as it was saved (rounded to bf16, or a checkpoint's value):
its derivative at the start is the gradient that linear_bwd states, so that the
rounding of Z does not enter.  Directions are those in which a mistake shows: along
the difference of the wrong gradient from the formula's (for zero and negated ones,
along the gradient), and v = sign(g) |normal|, where the terms of <g, v> add up.

Tolerance, |<got, v> - quotient| <= |v| |err| (Cauchy-Schwarz) with err per value:
  * dZ rounded to bf16 where there is an activation: 2^-8 |dZ|; its slope's fp32
    error 2^-19 max(1, |Z|) |dY|; both times |W| or |X|, summed; db takes the
    slope's error alone;
  * K products summed in fp32: K 2^-23 sum|a b|; the output's own rounding, 2^-8 of
    the value in bf16;
  * the quotient's truncation: h^2 / 6 max|act'''| sum|dY| |dz|^3, with |act'''| < 2
    for gelu and silu (0 without an activation), and its rounding, 2^-50 of sum|terms|
    over h."""
import numpy as np
import pytest
import torch

from dynamic_block_sparse_stats_b200 import api
from oracle import linear_oracle as L

pytestmark = pytest.mark.gpu

STEP = 2.0 ** -23


def _np(t):
    return t.double().cpu().numpy()


def _case(n, cin, cout, act, z8, fp32, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s, k=1.0: (k * torch.randn(*s, generator=g, device="cuda")).to(torch.bfloat16)  # noqa: E731
    X, W, b, dY = r(n, cin), r(cout, cin, k=cin ** -0.5), r(cout), r(n, cout)
    f = api.linear_fwd(X, W, b, act, save="ckpt8" if z8 else "bf16")
    d = api.linear_bwd(dY, X, W, f.Z, act, grad_fp32=fp32)
    Z0 = _np(api.ckpt8_unpack(f.Z) if z8 else f.Z)
    return (_np(X), _np(W), _np(b)), _np(dY), Z0, [_np(t) for t in (d.dX, d.dW, d.db)]


def _errors(args, dY, Z0, act, fp32):
    """Per value, how far each gradient may be from the formula's."""
    X, W, _ = args
    dZ = dY * L.slope(Z0, act)
    slope = 2.0 ** -19 * np.abs(dY) * np.maximum(1, np.abs(Z0)) if act else 0 * dY
    err = slope + (2.0 ** -8 * (np.abs(dZ) + slope) if act else 0)
    n, cout = dY.shape
    ex = err @ np.abs(W) + cout * STEP * (np.abs(dZ) @ np.abs(W))
    ew = err.T @ np.abs(X) + n * STEP * (np.abs(dZ).T @ np.abs(X))
    eb = slope.sum(0) + n * STEP * np.abs(dZ).sum(0)
    half = 0 if fp32 else 2.0 ** -8
    g = (dZ @ W, dZ.T @ X, dZ.sum(0))
    return [e + o * (np.abs(v) + e) for e, o, v in zip((ex, ew, eb), (2.0 ** -8, half, half), g)], g


def _passes(got, i, v, args, dY, Z0, act, err):
    """Whether <got, v> agrees with the quotient of f along v in argument i."""
    h = 1e-4
    X, W, b = args
    dz = v @ W.T if i == 0 else X @ v.T if i == 1 else np.broadcast_to(v, dY.shape)     # Z is linear in each argument
    up, dn = (dY * L.act(Z0 + h * dz, act)), (dY * L.act(Z0 - h * dz, act))
    quotient = (up.sum() - dn.sum()) / (2 * h)
    cut = (h * h / 6 * 2 * (np.abs(dY) * np.abs(dz) ** 3).sum() if act else 0) + 2.0 ** -50 * (np.abs(up) + np.abs(dn)).sum() / h
    tol = np.linalg.norm(v) * np.linalg.norm(err) + cut
    off = abs((got * v).sum() - quotient)
    return off <= tol, off / tol


@pytest.mark.parametrize("n,cin,cout", [(37, 64, 48), (1, 64, 96), (300, 136, 72)])
@pytest.mark.parametrize("act,z8", [(api.ACT_NONE, False), (api.ACT_SILU, False), (api.ACT_SILU, True), (api.ACT_GELU, False),
                                    (api.ACT_GELU, True)])
@pytest.mark.parametrize("fp32", [False, True])
def test_gradients_along_themselves(n, cin, cout, act, z8, fp32):
    args, dY, Z0, got = _case(n, cin, cout, act, z8, fp32, seed=n + act)
    errs, exact = _errors(args, dY, Z0, act, fp32)
    X, W, _ = args
    bare = (dY @ W, dY.T @ X, dY.sum(0))                         # without the slope
    rng = np.random.default_rng(n)
    for i, name in enumerate(("dX", "dW", "db")):
        held = lambda t, v: _passes(t, i, v, args, dY, Z0, act, errs[i])  # noqa: E731,B023
        wrong = [0 * exact[i], -exact[i]] + ([bare[i]] if act else [])
        for bad in wrong:
            # the direction in which this mistake shows: for the first two, along the gradient
            v = (bad - exact[i]) / np.linalg.norm(bad - exact[i])
            ok, off = held(got[i], v)
            print(f"{name}: {off:.3f} of the tolerance, the wrong one {held(bad, v)[1]:.1f}")
            assert ok, name
            assert not held(bad, v)[0], name
        v = np.sign(exact[i]) * np.abs(rng.normal(size=exact[i].shape))
        assert held(got[i], v)[0] and not held(0 * got[i], v)[0] and not held(-got[i], v)[0], name


@pytest.mark.parametrize("act", [api.ACT_NONE, api.ACT_RELU, api.ACT_SILU, api.ACT_GELU])
def test_what_fp32_weight_gradients_are_good_to(act):
    """Without an activation, and with relu, the operands are exact: 16 additions of 2^-23 of the sum
    for the chains and their joining.  With one, dZ's rounding to bf16 is in it: 2^-8
    / sqrt(3) of the norm in the mean square at most, and more than a hundredth of it
    for dZ's values are not bf16's."""
    g = torch.Generator(device="cuda")
    g.manual_seed(act)
    n, cin, cout = 20000, 264, 520
    X, W, dY = (torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16) for s in ((n, cin), (cout, cin), (n, cout)))
    Z = torch.randn(n, cout, generator=g, device="cuda").to(torch.bfloat16)
    got = api.linear_bwd(dY, X, W, Z, act, need=("dW",), grad_fp32=True)
    dZ = dY.double() * torch.from_numpy(L.slope(_np(Z), act)).cuda()
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())  # noqa: E731
    dw = rel(got.dW, dZ.t() @ X.double())
    rms = 2.0 ** -8 / 3 ** 0.5
    if act <= api.ACT_RELU:                      # relu's slopes are 0 and 1
        assert dw < 16 * STEP
    else:
        assert rms / 100 < dw < rms
