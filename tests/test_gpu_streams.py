"""Calls with an explicit stream: what they allocate belongs to that stream, and
is not given out again while the caller's stream may still use it."""
import pytest
import torch

from dynamic_block_sparse_stats_b200 import api
from dynamic_block_sparse_stats_b200.synth import WORKLOADS, make_bridge_output, make_inputs, make_projection

pytestmark = pytest.mark.gpu


def _owner(t):
    """The stream whose memory a tensor lies in."""
    at = t.data_ptr()
    return next(s["stream"] for s in torch.cuda.memory_snapshot() if s["address"] <= at < s["address"] + s["total_size"])


def _rand(seed, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)


def _linear(stream=None):
    X, W, b, dY = _rand(1, 600, 264), _rand(2, 328, 264) / 16, _rand(3, 328), _rand(4, 600, 328)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    x8 = api.ckpt8_pack(X, stream=stream)
    x = api.ckpt8_unpack(x8, stream=stream)
    f = api.linear_fwd(X, W, b, api.ACT_GELU, save="ckpt8", stream=stream)
    h = api.linear_fwd(X, W, b, api.ACT_GELU, save="bf16", stream=stream)
    g = api.linear_bwd(dY, x8, W, f.Z, api.ACT_GELU, stream=stream)
    # the inputs as well: they have to outlive the calls
    return (x8.codes, x8.scales, x, f.Y, f.Z.codes, f.Z.scales, h.Y, h.Z, g.dX, g.dW, g.db, f.ws, h.ws, g.ws), 3, (X, W, b, dY)


def _attention(stream=None):
    w = WORKLOADS["tiny_d128"]
    inp = make_inputs(w, "cuda", with_grad=True)
    hhat = make_bridge_output(inp["a"], 256)
    X, Wv = make_projection(inp["V"])
    p = api.params_for(w)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    a = api.a2v_norm(hhat, stream=stream)
    pl = api.plan(p, inp["V"], a, stream=stream)
    V, pv = api.project_v_plan(p, X, Wv, a, stream=stream)
    sel = api.select(p, pl, inp["Q"], inp["K"], cap=1, stream=stream)          # too small: grown by the call
    fw = api.attn_fwd(p, pl, sel, inp["Q"], inp["K"], inp["V"], stream=stream)
    d = api.attn_bwd(p, pl, sel, inp["Q"], inp["K"], inp["V"], fw.O, inp["dO"], fw.lse, O_res=fw.O_res, deterministic=True,
                     stream=stream)
    out = (a, pl.zone_shape, pl.perm, pl.inv_perm, V, pv.perm, sel.row_ptr, fw.O, fw.O_res, fw.lse, *d)
    return out + (pl.ws, pv.ws, sel.col, sel.row, sel.ws, fw.ws), 6, (inp, hhat, X, Wv, pl, pv, sel)


@pytest.mark.parametrize("path", [_linear, _attention])
def test_new_tensors_belong_to_the_calls_stream(path):
    want, rest, _keep = path()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got, _, _keep2 = path(s)
    s.synchronize()
    assert [_owner(t) for t in got] == [s.cuda_stream] * len(got)
    for u, v in zip(want[:-rest], got):
        assert torch.equal(u, v)


def test_a_workspace_is_not_given_out_while_its_call_may_run():
    X, W = _rand(1, 300, 64), _rand(2, 128, 64)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000_000)
    f = api.linear_fwd(X, W, stream=s)
    at = f.ws.data_ptr()
    del f
    mine = [torch.empty(256, dtype=torch.uint8, device="cuda") for _ in range(64)]
    assert not s.query()                             # the call has not begun
    assert at not in [t.data_ptr() for t in mine]
    s.synchronize()


def test_an_output_waits_for_the_callers_stream():
    X, W = _rand(1, 3000, 64), _rand(2, 1032, 64)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    f = api.linear_fwd(X, W, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(200_000_000)
    kept = f.Y.clone()                               # the caller's stream reads Y, later
    at, want = f.Y.data_ptr(), api.linear_fwd(X, W, stream=s).Y
    del f
    again = [api.linear_fwd(X, W, stream=s).Y for _ in range(4)]
    assert not torch.cuda.current_stream().query()
    assert at not in [t.data_ptr() for t in again]
    torch.cuda.synchronize()
    assert torch.equal(kept, want)


def test_buffers_of_the_caller_are_used_as_they_are():
    X, W = _rand(1, 300, 64), _rand(2, 128, 64)
    Y, ws = torch.empty(300, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(256, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    f = api.linear_fwd(X, W, Y=Y, ws=ws, stream=s)
    s.synchronize()
    assert f.Y is Y and f.ws is ws and torch.equal(Y, api.linear_fwd(X, W).Y)


def test_an_explicit_stream_inside_a_capture():
    X, W = _rand(1, 300, 64), _rand(2, 128, 64)
    want = api.linear_fwd(X, W, save="ckpt8")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        f = api.linear_fwd(X, W, save="ckpt8", stream=side)
        torch.cuda.current_stream().wait_stream(side)
        y = f.Y * 1
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want.Y) and torch.equal(f.Z.codes, want.Z.codes)
