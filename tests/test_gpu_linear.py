"""GPU parity of prism_linear_fwd / prism_linear_bwd with the float64 oracle.

Tolerances, per value:
  * bf16 outputs are rounded once: half a step, 2^-8 of the value;
  * products are exact in fp32; a sum of K of them, in any order and with every
    addition rounded or truncated (at most 2^-23 of the running magnitude),
    is off by at most K 2^-23 sum|a b|; bias and residual add two roundings;
  * the activations' slopes are at most 1.13, their own fp32 error at most
    2^-19 of max(1, |z|) (exp, a division, a polynomial: a few units of 2^-23
    each, the exponential's argument up to 2^3 larger than z);
  * dZ is rounded to bf16 where there is an activation: 2^-8 sum|dZ||w| more in
    dX and dW;
  * a checkpoint of Z is off by half its scale, plus the error of Z itself."""
import numpy as np
import pytest
import torch

from dynamic_block_sparse_stats_b200 import _lib, api
from oracle import linear_oracle as L

pytestmark = pytest.mark.gpu

ACTS = [api.ACT_NONE, api.ACT_RELU, api.ACT_SILU, api.ACT_GELU]
STEP = 2.0 ** -23


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rand(g, *shape, s=1.0):
    return (s * torch.randn(*shape, generator=g, device="cuda")).to(torch.bfloat16)


def _np(t):
    return t.double().cpu().numpy()


def _inputs(n, cin, cout, seed=0):
    g = _gen(1000 * seed + n + 7 * cin + 13 * cout)
    return dict(X=_rand(g, n, cin), W=_rand(g, cout, cin, s=cin ** -0.5), b=_rand(g, cout), R=_rand(g, n, cout),
                dY=_rand(g, n, cout), Z=_rand(g, n, cout, s=2.0))


def _within(got, want, tol, what):
    err = np.abs(_np(got) - want)
    worst = float((err / tol).max()) if err.size else 0.0
    print(f"{what}: max err / tolerance = {worst:.3f}")
    assert (err <= tol).all(), what


def _check_fwd(d, f, act, bias=True, res=True):
    X, W = _np(d["X"]), _np(d["W"])
    b, R = _np(d["b"]) if bias else None, _np(d["R"]) if res else None
    Z, Y = L.forward(X, W, b, act, R)
    zerr = (X.shape[1] + 2) * STEP * (np.abs(X) @ np.abs(W).T + (np.abs(b) if bias else 0)) + 1e-30
    yerr = 1.13 * zerr + (2.0 ** -19 * np.maximum(1, np.abs(Z)) if act else 0) + 2 * STEP * np.abs(Y)
    _within(f.Y, Y, yerr + 2.0 ** -8 * (np.abs(Y) + yerr), "Y")
    if isinstance(f.Z, api.Ckpt8):
        held = api.ckpt8_unpack(f.Z)
        s = np.exp2(f.Z.scales.cpu().numpy().astype(np.float64) - 127)[:, :(Z.shape[1] + 31) // 32]
        half = np.repeat(s / 2, 32, axis=1)[:, :Z.shape[1]]
        _within(held, Z, half + zerr, "Z8")
        top = np.zeros((Z.shape[0], s.shape[1] * 32))
        top[:, :Z.shape[1]] = np.abs(Z)
        slack = np.zeros_like(top)
        slack[:, :Z.shape[1]] = zerr
        top, slack = top.reshape(Z.shape[0], -1, 32), slack.reshape(Z.shape[0], -1, 32)
        # the scale is the smallest that holds the block
        assert (top.max(-1) - slack.max(-1) <= 127 * s).all()
        assert ((top.max(-1) + slack.max(-1) >= 127 * s / 2) | (s == 2.0 ** -126)).all()
    elif f.Z is not None:
        _within(f.Z, Z, zerr + 2.0 ** -8 * (np.abs(Z) + zerr), "Z")


def _check_bwd(d, g, act, x, z, fp32):
    X = _np(api.ckpt8_unpack(x) if isinstance(x, api.Ckpt8) else x)
    Z = None if act == 0 else _np(api.ckpt8_unpack(z) if isinstance(z, api.Ckpt8) else z)
    dY, W = _np(d["dY"]), _np(d["W"])
    dZ, dX, dW, db = L.backward(dY, X, W, Z, act)
    n, cout = dY.shape
    serr = 2.0 ** -19 * np.abs(dY) * np.maximum(1, np.abs(Z)) if act else np.zeros_like(dY)
    derr = serr + (2.0 ** -8 * np.abs(dZ) if act else 0)
    out = 0 if fp32 else 2.0 ** -8
    ex = derr @ np.abs(W) + cout * STEP * (np.abs(dZ) @ np.abs(W))
    ew = derr.T @ np.abs(X) + n * STEP * (np.abs(dZ).T @ np.abs(X))
    eb = serr.sum(0) + n * STEP * np.abs(dZ).sum(0)
    if g.dX is not None:
        _within(g.dX, dX, ex + 2.0 ** -8 * (np.abs(dX) + ex) + 1e-30, "dX")
    if g.dW is not None:
        _within(g.dW, dW, ew + out * (np.abs(dW) + ew) + 1e-30, "dW")
    if g.db is not None:
        _within(g.db, db, eb + out * (np.abs(db) + eb) + 1e-30, "db")


SIZES = [(1, 8, 8), (1, 1024, 512), (2, 200, 72), (7, 64, 264), (16, 512, 128), (17, 520, 136), (33, 1000, 40),
         (127, 72, 128), (128, 128, 256), (129, 264, 320), (300, 64, 1288), (1003, 328, 712), (2049, 192, 192)]


@pytest.mark.parametrize("n,cin,cout", SIZES)
@pytest.mark.parametrize("act", ACTS)
def test_forward(n, cin, cout, act):
    d = _inputs(n, cin, cout)
    for save in (None, "bf16", "ckpt8"):
        f = api.linear_fwd(d["X"], d["W"], d["b"], act, d["R"], save)
        assert api.workspace_status(f.ws) == 0
        _check_fwd(d, f, act)
    f = api.linear_fwd(d["X"], d["W"], None, act)
    _check_fwd(d, f, act, bias=False, res=False)


@pytest.mark.parametrize("n,cin,cout", SIZES)
@pytest.mark.parametrize("x8", [False, True])
@pytest.mark.parametrize("act,z8", [(api.ACT_NONE, False), (api.ACT_RELU, True), (api.ACT_SILU, False), (api.ACT_GELU, True),
                                    (api.ACT_GELU, False)])
def test_backward(n, cin, cout, x8, act, z8):
    d = _inputs(n, cin, cout)
    x = api.ckpt8_pack(d["X"]) if x8 else d["X"]
    z = None if act == 0 else api.ckpt8_pack(d["Z"]) if z8 else d["Z"]
    for fp32 in (False, True):
        g = api.linear_bwd(d["dY"], x, d["W"], z, act, grad_fp32=fp32)
        assert api.workspace_status(g.ws) == 0
        _check_bwd(d, g, act, x, z, fp32)


@pytest.mark.parametrize("n,cin,cout", [(20000, 1024, 1024), (9000, 256, 2056), (9001, 712, 1000), (70000, 264, 256)])
def test_large(n, cin, cout):
    """Several waves of the largest tiles, against float64 on the GPU: relative
    to the norm, one bf16 rounding of uniform relative error (2^-9 to 2^-8 at
    most: 2^-8 / sqrt(3) in the mean square), two where dZ is rounded too."""
    d = _inputs(n, cin, cout)
    rms = 2.0 ** -8 / 3 ** 0.5
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())  # noqa: E731
    f = api.linear_fwd(d["X"], d["W"], d["b"], api.ACT_GELU, d["R"], "ckpt8")
    z = d["X"].double() @ d["W"].double().t() + d["b"].double()
    y = torch.nn.functional.gelu(z, approximate="tanh") + d["R"].double()
    assert rel(f.Y, y) < rms
    x8 = api.ckpt8_pack(d["X"])
    for x in (d["X"], x8):
        xd = (api.ckpt8_unpack(x) if x is x8 else x).double()
        g = api.linear_bwd(d["dY"], x, d["W"], grad_fp32=True)
        dyd = d["dY"].double()
        # fp32 sums in short chains: 16 stages of at most 2^-23 of the running sum each, and their joining
        assert rel(g.dW, dyd.t() @ xd) < 16 * STEP
        assert rel(g.db, dyd.sum(0)) < 16 * STEP
        assert rel(g.dX, dyd @ d["W"].double()) < rms
        zd = api.ckpt8_unpack(f.Z).double().requires_grad_()
        dz, = torch.autograd.grad(torch.nn.functional.gelu(zd, approximate="tanh"), zd, dyd)
        g = api.linear_bwd(d["dY"], x, d["W"], f.Z, api.ACT_GELU)
        assert api.workspace_status(g.ws) == 0
        assert rel(g.dW, dz.t() @ xd) < 1.42 * rms
        assert rel(g.dX, dz @ d["W"].double()) < 1.42 * rms
        assert rel(g.db, dz.sum(0)) < rms


@pytest.mark.parametrize("n,cin,cout", [(20000, 1024, 1024), (9001, 712, 1000), (9001, 264, 2056), (50, 72, 136)])
@pytest.mark.parametrize("fp32", [False, True])
def test_checkpointed_weight_gradient_is_the_restored_ones(n, cin, cout, fp32):
    """The checkpoint's values are exact in bf16, so converting codes on the way
    to the tensor cores and restoring the tensor first give the same bits."""
    d = _inputs(n, cin, cout)
    x8 = api.ckpt8_pack(d["X"])
    a = api.linear_bwd(d["dY"], x8, None, need=("dW",), grad_fp32=fp32)
    b = api.linear_bwd(d["dY"], api.ckpt8_unpack(x8), None, need=("dW",), grad_fp32=fp32)
    assert torch.equal(a.dW, b.dW)


@pytest.mark.parametrize("n,cin,cout", [(20000, 128, 512), (20000, 256, 776), (12000, 520, 1032), (6000, 1024, 2048)])
def test_epilogues_of_the_pair_tiles(n, cin, cout):
    """Short contractions take the wide epilogue, long ones the narrow: every
    combination of what it does, at the rows of the first and last tiles."""
    d = _inputs(n, cin, cout)
    rows = torch.cat([torch.arange(300), torch.arange(n - 300, n)]).cuda()
    part = {k: v[rows].contiguous() if k in ("X", "R") else v for k, v in d.items()}
    for act in (api.ACT_NONE, api.ACT_RELU, api.ACT_GELU):
        for bias in (False, True):
            for res in (False, True):
                for save in (None, "bf16", "ckpt8"):
                    f = api.linear_fwd(d["X"], d["W"], d["b"] if bias else None, act, d["R"] if res else None, save)
                    assert api.workspace_status(f.ws) == 0
                    z = f.Z
                    if save == "bf16":
                        z = f.Z[rows]
                    elif save == "ckpt8":
                        z = api.Ckpt8(f.Z.codes[rows].contiguous(), f.Z.scales[rows].contiguous(), cout)
                    _check_fwd(part, api.LinearResult(f.Y[rows], z, f.ws), act, bias, res)


def test_gradients_against_differences():
    """<dY, Y> moved along a direction of X, W or bias, in float64 of the oracle,
    against the kernel's gradient along that direction: a central difference of
    step h is exact to h^2 (1e-6 of order-one third derivatives, summed), the
    gradients' own rounding is bounded per value as above."""
    n, cin, cout = 37, 64, 48
    d = _inputs(n, cin, cout, seed=5)
    act = api.ACT_GELU
    f = api.linear_fwd(d["X"], d["W"], d["b"], act, save="bf16")
    g = api.linear_bwd(d["dY"], d["X"], d["W"], f.Z, act, grad_fp32=True)
    X, W, b, dY = (_np(d[k]) for k in ("X", "W", "b", "dY"))
    loss = lambda X, W, b: (dY * L.forward(X, W, b, act)[1]).sum()  # noqa: E731
    Z = L.forward(X, W, b, act)[0]
    # Z is saved in bf16: the slope moves by at most 1.13 2^-8 |Z| (second derivative at most 1.13), dZ by 2^-8 of itself
    dz_err = np.abs(dY) * 1.13 * 2.0 ** -8 * np.abs(Z) + 2.0 ** -8 * np.abs(dY) * 1.13
    r = np.random.default_rng(0)
    h = 1e-3
    for i, (got, err) in enumerate(((g.dX, dz_err @ np.abs(W)), (g.dW, dz_err.T @ np.abs(X)), (g.db, dz_err.sum(0)))):
        v = r.normal(size=got.shape)
        a = [X, W, b]
        up, dn = list(a), list(a)
        up[i], dn[i] = a[i] + h * v, a[i] - h * v
        diff = (loss(*up) - loss(*dn)) / (2 * h)
        got64 = _np(got)
        tol = (np.abs(v) * (err + 2.0 ** -8 * np.abs(got64))).sum() + 1e-6 * np.abs(dY).sum() * np.abs(v).max() ** 3
        assert abs(diff - (got64 * v).sum()) <= tol


def test_needs_and_buffers():
    d = _inputs(130, 136, 72)
    full = api.linear_bwd(d["dY"], d["X"], d["W"], d["Z"], api.ACT_SILU)
    for need in (("dX",), ("dW",), ("db",), ("dW", "db")):
        g = api.linear_bwd(d["dY"], d["X"] if "dW" in need else None, d["W"] if "dX" in need else None, d["Z"], api.ACT_SILU,
                           need=need)
        for k in ("dX", "dW", "db"):
            assert (getattr(g, k) is None) == (k not in need)
            if k in need:
                assert torch.equal(getattr(g, k), getattr(full, k))
    out = tuple(torch.empty_like(t) for t in (full.dX, full.dW, full.db))
    ws = torch.empty(api.linear_workspace_size(130, 136, 72, api.ACT_SILU, True), dtype=torch.uint8, device="cuda")
    g = api.linear_bwd(d["dY"], d["X"], d["W"], d["Z"], api.ACT_SILU, out=out, ws=ws)
    assert g.dX is out[0] and g.ws is ws
    assert all(torch.equal(a, b) for a, b in zip(out, (full.dX, full.dW, full.db)))


def test_strided_rows_in_place_residual_and_what_lies_around():
    n, cin, cout = 45, 136, 264
    d = _inputs(n, cin, cout)
    want = api.linear_fwd(d["X"], d["W"], d["b"], api.ACT_SILU, d["R"])
    g = _gen(9)
    big_x = _rand(g, n + 2, cin + 72)
    big_x[1:n + 1, 8:8 + cin] = d["X"]
    room = torch.full((n + 3, cout + 40), 5.0, dtype=torch.bfloat16, device="cuda")
    y = room[1:n + 1, 16:16 + cout]
    y.copy_(d["R"])
    f = api.linear_fwd(big_x[1:n + 1, 8:8 + cin], d["W"], d["b"], api.ACT_SILU, residual=y, Y=y)
    assert f.Y is y and torch.equal(y, want.Y)
    room[1:n + 1, 16:16 + cout] = 5.0
    assert (room == 5).all()
    # strided dY, X and Z
    ref = api.linear_bwd(d["dY"], d["X"], d["W"], d["Z"], api.ACT_GELU)
    wide = _rand(g, n, 2 * cout)
    wide[:, :cout], wide[:, cout:] = d["dY"], d["Z"]
    got = api.linear_bwd(wide[:, :cout], big_x[1:n + 1, 8:8 + cin], d["W"], wide[:, cout:], api.ACT_GELU)
    for k in ("dX", "dW", "db"):
        assert torch.equal(getattr(ref, k), getattr(got, k))


@pytest.mark.parametrize("n", [0, 1])
def test_no_tokens_and_one(n):
    d = _inputs(max(n, 1), 64, 128)
    X, dY, Z = d["X"][:n], d["dY"][:n], d["Z"][:n]
    f = api.linear_fwd(X, d["W"], d["b"], api.ACT_GELU, save="ckpt8")
    g = api.linear_bwd(dY, X, d["W"], Z, api.ACT_GELU)
    torch.cuda.synchronize()
    assert f.Y.shape == (n, 128) and g.dX.shape == (n, 64)
    if n == 0:
        assert (g.dW == 0).all() and (g.db == 0).all()


def test_two_calls_give_the_same_bits():
    d = _inputs(3000, 520, 776)
    x8, z8 = api.ckpt8_pack(d["X"]), api.ckpt8_pack(d["Z"])
    a = api.linear_bwd(d["dY"], x8, d["W"], z8, api.ACT_GELU, grad_fp32=False)
    b = api.linear_bwd(d["dY"], x8, d["W"], z8, api.ACT_GELU, grad_fp32=False)
    c = api.linear_bwd(d["dY"], api.ckpt8_unpack(x8), d["W"], api.ckpt8_unpack(z8), api.ACT_GELU, grad_fp32=False)
    for k in ("dX", "dW", "db"):
        assert torch.equal(getattr(a, k), getattr(b, k))
        # the checkpoint's values are exact in bf16: restoring them first changes nothing
        assert torch.equal(getattr(a, k), getattr(c, k))


def test_streams_and_graph():
    d = _inputs(700, 264, 512)
    want_f = api.linear_fwd(d["X"], d["W"], d["b"], api.ACT_GELU, d["R"], "ckpt8")
    want_g = api.linear_bwd(d["dY"], d["X"], d["W"], want_f.Z, api.ACT_GELU)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for s in (s1, s2):                            # two calls at once, each with its own buffers
        with torch.cuda.stream(s):
            f = api.linear_fwd(d["X"], d["W"], d["b"], api.ACT_GELU, d["R"], "ckpt8")
            outs.append((f, api.linear_bwd(d["dY"], d["X"], d["W"], f.Z, api.ACT_GELU)))
    torch.cuda.synchronize()
    for f, g in outs:
        assert torch.equal(f.Y, want_f.Y) and all(torch.equal(getattr(g, k), getattr(want_g, k)) for k in ("dX", "dW", "db"))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f = api.linear_fwd(d["X"], d["W"], d["b"], api.ACT_GELU, d["R"], "ckpt8")
        g = api.linear_bwd(d["dY"], d["X"], d["W"], f.Z, api.ACT_GELU)
    for k in ("X", "dY"):
        d[k].copy_(_rand(_gen(11), *d[k].shape))
    graph.replay()
    torch.cuda.synchronize()
    want_f = api.linear_fwd(d["X"], d["W"], d["b"], api.ACT_GELU, d["R"], "ckpt8")
    want_g = api.linear_bwd(d["dY"], d["X"], d["W"], want_f.Z, api.ACT_GELU)
    assert torch.equal(f.Y, want_f.Y) and all(torch.equal(getattr(g, k), getattr(want_g, k)) for k in ("dX", "dW", "db"))


def test_two_graphs_replayed_in_turn_and_at_once():
    """Two captured training steps, each with its own buffers, replayed on two
    streams at once give what eager calls give."""
    runs = []
    for seed in (31, 32):
        d = _inputs(2300, 520, 640, seed=seed)

        def step(d=d):
            x8 = api.ckpt8_pack(d["X"])
            f = api.linear_fwd(d["X"], d["W"], d["b"], api.ACT_GELU, d["R"], "ckpt8")
            return f, api.linear_bwd(d["dY"], x8, d["W"], f.Z, api.ACT_GELU)

        want = step()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = step()
        runs.append((g, got, want, d))              # a graph does not keep its inputs
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    for _ in range(3):
        for (g, _, _, _), s in zip(runs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for _, (f, b), (wf, wb), _ in runs:
        assert api.workspace_status(f.ws) == 0 and api.workspace_status(b.ws) == 0
        assert torch.equal(f.Y, wf.Y) and all(torch.equal(getattr(b, k), getattr(wb, k)) for k in ("dX", "dW", "db"))


def test_a_workspace_is_used_again():
    """One workspace buffer for calls of different sizes, one after the other on a
    stream, whatever it held before; its status word starts clear in each."""
    ws = torch.full((api.linear_workspace_size(3000, 512, 512, api.ACT_GELU, True, x8=True),), 0xff, dtype=torch.uint8,
                    device="cuda")
    for n, cin, cout in ((3000, 512, 512), (5, 64, 72), (700, 264, 512)):
        d = _inputs(n, cin, cout)
        f = api.linear_fwd(d["X"], d["W"], d["b"], api.ACT_GELU, save="ckpt8", ws=ws)
        assert api.workspace_status(ws) == 0
        x8 = api.ckpt8_pack(d["X"])
        for need in (("dX", "dW", "db"), ("dX",), ("dW",), ("db",)):
            ws[:256] = 0xff
            g = api.linear_bwd(d["dY"], x8, d["W"], f.Z, api.ACT_GELU, need=need, ws=ws)
            assert api.workspace_status(ws) == 0
            want = api.linear_bwd(d["dY"], x8, d["W"], f.Z, api.ACT_GELU, need=need)
            assert all(torch.equal(getattr(g, k), getattr(want, k)) for k in need)


def test_non_finite_inputs_stay_in_their_rows():
    d = _inputs(70, 128, 192)
    X = d["X"].clone()
    X[3, 5], X[40, 0] = float("nan"), float("inf")
    f = api.linear_fwd(X, d["W"], d["b"], api.ACT_GELU, save="ckpt8")
    held = api.ckpt8_unpack(f.Z)
    clean = api.linear_fwd(d["X"], d["W"], d["b"], api.ACT_GELU, save="ckpt8")
    ok = torch.ones(70, dtype=torch.bool, device="cuda")
    ok[3] = ok[40] = False
    assert torch.equal(f.Y[ok], clean.Y[ok]) and torch.equal(held[ok], api.ckpt8_unpack(clean.Z)[ok])
    assert torch.isnan(f.Y[3]).all() and torch.isnan(held[3]).all()
    # a checkpoint that lost a block says so in every gradient it touches
    g = api.linear_bwd(d["dY"], d["X"], d["W"], f.Z, api.ACT_GELU)
    assert torch.isnan(g.dX[3]).all() and torch.isnan(g.db).all() and torch.isfinite(g.dX[ok]).all()


def test_activations_far_out():
    """Saturated activations and slopes are exact: 0 or z, 0 or 1."""
    z = torch.tensor([-3e38, -1e20, -200.0, -40.0, 40.0, 200.0, 1e20, 3e38], device="cuda").to(torch.bfloat16)
    W = torch.eye(8, device="cuda").to(torch.bfloat16)
    X = torch.diag(z.float()).to(torch.bfloat16)
    one = torch.ones(8, 8, dtype=torch.bfloat16, device="cuda")
    for act in (api.ACT_RELU, api.ACT_SILU, api.ACT_GELU):
        y = api.linear_fwd(X, W, act=act).Y.diagonal()
        assert torch.equal(y[4:], z[4:]) and (y[:4].abs() <= 1e-14).all()
        Z = z.expand(8, 8).contiguous()
        db = api.linear_bwd(one, X, W, Z, act, need=("db",), grad_fp32=True).db
        assert torch.equal(db[4:], torch.full((4,), 8.0, device="cuda")) and (db[:4].abs() <= 1e-12).all()


def test_offsets_past_32_bits():
    """2.2e9 outputs; the first and last rows against a call on those rows alone."""
    n, cin, cout = 540_680, 64, 4096
    d = dict(X=_rand(_gen(1), n, cin), W=_rand(_gen(2), cout, cin, s=0.125))
    f = api.linear_fwd(d["X"], d["W"], save="ckpt8")
    pick = torch.cat([torch.arange(300), torch.arange(n - 340, n)]).cuda()
    part = api.linear_fwd(d["X"][pick].contiguous(), d["W"], save="ckpt8")
    assert torch.equal(f.Y[pick], part.Y)
    assert torch.equal(f.Z.codes[pick], part.Z.codes) and torch.equal(f.Z.scales[pick], part.Z.scales)
    g = api.linear_bwd(f.Y, d["X"], d["W"], need=("dX",))
    dY, W = _np(part.Y), _np(d["W"])
    want, mag = dY @ W, np.abs(dY) @ np.abs(W)
    tol = cout * STEP * mag
    _within(g.dX[pick], want, tol + 2.0 ** -8 * (np.abs(want) + tol), "dX")


def test_layer_training_step_through_checkpoints():
    """The layer as it is trained: Q and K from the linear map, V from the fused
    projection, block-sparse attention, the output projection onto the residual
    stream; between forward and backward only 8-bit checkpoints of X, Q, K, V
    and O are kept.  The step's own checks: every piece equals the same call on
    the restored tensors, and the weight gradients match float64 products."""
    from dynamic_block_sparse_stats_b200.synth import WORKLOADS, make_inputs, make_projection
    w = WORKLOADS["small"]
    inp = make_inputs(w, "cuda", with_grad=True)
    X, Wv = make_projection(inp["V"])
    N, C, hd = X.shape[0], X.shape[1], w.heads * w.head_dim
    g = _gen(21)
    Wq, Wk, Wo = _rand(g, hd, C, s=C ** -0.5), _rand(g, hd, C, s=C ** -0.5), _rand(g, C, hd, s=hd ** -0.5)
    bo = _rand(g, C)
    p = api.params_for(w)
    shape = (N, w.heads, w.head_dim)
    Q = api.linear_fwd(X, Wq).Y.view(shape)
    K = api.linear_fwd(X, Wk).Y.view(shape)
    V, plan = api.project_v_plan(p, X, Wv, inp["a"])
    sel = api.select(p, plan, Q, K)
    fw = api.attn_fwd(p, plan, sel, Q, K, V)
    Y = api.linear_fwd(fw.O.flatten(1), Wo, bo, residual=X).Y
    held = {k: api.ckpt8_pack(t) for k, t in (("X", X), ("Q", Q.flatten(1)), ("K", K.flatten(1)), ("V", V.flatten(1)),
                                              ("O", fw.O.flatten(1)))}
    dY = _rand(g, N, C)
    out = api.linear_bwd(dY, held["O"], Wo, grad_fp32=True)
    Qr, Kr, Vr, Or = (api.ckpt8_unpack(held[k]).view(shape) for k in "QKVO")
    # the attention recomputes its own row sums from the restored operands
    re = api.attn_fwd(p, plan, sel, Qr, Kr, Vr)
    dQ, dK, dV = api.attn_bwd(p, plan, sel, Qr, Kr, Vr, re.O, out.dX.view(shape), re.lse, O_res=re.O_res,
                              deterministic=True)
    grads = [api.linear_bwd(t.flatten(1), held["X"], wt, grad_fp32=True) for t, wt in ((dQ, Wq), (dK, Wk), (dV, Wv))]
    torch.cuda.synchronize()
    for t in (fw.ws, re.ws, out.ws, plan.ws, *(x.ws for x in grads)):
        assert api.workspace_status(t) == _lib.PRISM_OK
    y = fw.O.flatten(1).double() @ Wo.double().t() + bo.double() + X.double()
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())  # noqa: E731
    assert rel(Y, y) < 2.0 ** -8
    Xr = api.ckpt8_unpack(held["X"]).double()
    assert rel(out.dW, dY.double().t() @ Or.flatten(1).double()) < 16 * STEP
    for t, gr in zip((dQ, dK, dV), grads):
        assert rel(gr.dW, t.flatten(1).double().t() @ Xr) < 16 * STEP
    # and the checkpoints move the gradients by no more than their rounding does: dWo sums N tokens' independent
    # errors of at most half a scale (2^-7 of a block's largest value) each
    exact = dY.double().t() @ fw.O.flatten(1).double()
    assert rel(out.dW, exact) < 0.05
