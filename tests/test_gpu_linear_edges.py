"""What lies at the edges of the linear map's calls: the padding of a saved
checkpoint and the buffers around it."""
import pytest
import torch

from dynamic_block_sparse_stats_b200 import _lib, api

pytestmark = pytest.mark.gpu


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rand(g, *shape, s=1.0):
    return (s * torch.randn(*shape, generator=g, device="cuda")).to(torch.bfloat16)


def _framed(n, width, byte):
    """A checkpoint filled with `byte`, between two more rows of it."""
    ld = (width + 127) // 128 * 128
    codes = torch.full((n + 2, ld), byte, dtype=torch.uint8, device="cuda").view(torch.int8)
    scales = torch.full((n + 2, ld // 32), byte, dtype=torch.uint8, device="cuda")
    return codes, scales, api.Ckpt8(codes[1:n + 1], scales[1:n + 1], width)


# `out` ends 8..64 channels past a multiple of 128 (and elsewhere), at sizes of
# every kernel: few tokens, the split contraction, single and pair tiles
@pytest.mark.parametrize("n,cin,cout", [(129, 264, 320), (300, 64, 1288), (512, 1024, 192), (2049, 192, 192), (200, 1024, 64),
                                        (65, 64, 8), (77, 520, 136), (1, 64, 8), (16, 512, 136), (33, 1000, 40),
                                        (129, 264, 328), (1003, 328, 712), (5000, 264, 1288), (20000, 256, 776),
                                        (20000, 1024, 1032)])
def test_a_saved_checkpoint_is_written_whole(n, cin, cout):
    """Codes at channels past `out` are 0 whatever the buffer held, the blocks that
    exist are the same, and nothing is written outside the rows."""
    g = _gen(n + cout)
    X, W, b = _rand(g, n, cin), _rand(g, cout, cin, s=cin ** -0.5), _rand(g, cout)
    seen = []
    for byte in (0x55, 0xAA):
        codes, scales, z = _framed(n, cout, byte)
        f = api.linear_fwd(X, W, b, api.ACT_GELU, save="ckpt8", Z=z)
        assert api.workspace_status(f.ws) == 0 and f.Z is z
        assert (z.codes[:, cout:] == 0).all()
        for frame in (codes.view(torch.uint8), scales):
            assert (frame[0] == byte).all() and (frame[-1] == byte).all()
        seen.append((z.codes, z.scales))
    assert torch.equal(seen[0][0], seen[1][0]) and torch.equal(seen[0][1], seen[1][1])
    assert torch.equal(api.ckpt8_unpack(z), api.ckpt8_unpack(api.linear_fwd(X, W, b, api.ACT_GELU, save="ckpt8").Z))


@pytest.mark.parametrize("cin,cout", [(8, 8), (40, 72), (72, 136), (200, 200)])
def test_ragged_tiles_of_the_split_kernel_again_and_again(cin, cout):
    """Outputs that end inside a tile, in rows and columns: lanes with nothing to
    store meet the others at the kernel's last barrier, call after call."""
    g = _gen(cin)
    n = 1500
    X, W, dY = _rand(g, n, cin), _rand(g, cout, cin), _rand(g, n, cout)
    first = None
    for _ in range(40):
        f = api.linear_fwd(X[:131], W, save="ckpt8")
        b = api.linear_bwd(dY, X, W, grad_fp32=True)
        got = (f.Y, f.Z.codes, b.dX, b.dW, b.db)
        first = first or got
        assert api.workspace_status(f.ws) == 0 and api.workspace_status(b.ws) == 0
        assert all(torch.equal(u, v) for u, v in zip(first, got))
    # exact products, n additions of at most 2^-23 of the running magnitude each
    a, x = dY.double().t(), X.double()
    assert ((first[3] - a @ x).abs() <= n * 2.0 ** -23 * (a.abs() @ x.abs())).all()


def test_an_output_on_an_operand_is_refused_and_changes_nothing():
    """The input's buffer as dX's, with dW asked for: dW would read dX as X."""
    n, c = 300, 128
    g = _gen(3)
    X, W, dY, Z = _rand(g, n, c), _rand(g, c, c), _rand(g, n, c), _rand(g, n, c)
    kept = X.clone()
    for call in (lambda: api.linear_bwd(dY, X, W, out=(X, None, None)),
                 lambda: api.linear_bwd(dY, X, W, Z, api.ACT_GELU, out=(Z, None, None)),
                 lambda: api.linear_bwd(dY, X, W, out=(None, W, None)),
                 lambda: api.linear_fwd(X, W, save="bf16", Z=X),
                 lambda: api.linear_fwd(X[:c], W, Y=W),
                 lambda: api.linear_fwd(X[1:], W, residual=X[1:], Y=X[:-1])):
        with pytest.raises(_lib.PrismError, match="overlaps"):
            call()
    torch.cuda.synchronize()
    assert torch.equal(X, kept)


def test_outputs_beside_operands_in_one_buffer():
    """Column slices of one buffer share no memory; X's place is free for dX where
    dW is not asked for; a residual is added in place in a slice."""
    n, cin, cout = 700, 136, 264
    g = _gen(4)
    X, W, b, R, dY = _rand(g, n, cin), _rand(g, cout, cin), _rand(g, cout), _rand(g, n, cout), _rand(g, n, cout)
    want = api.linear_fwd(X, W, b, api.ACT_SILU, R).Y
    room = torch.zeros(n, cin + cout + 8, dtype=torch.bfloat16, device="cuda")
    room[:, :cin], room[:, cin:cin + cout] = X, R
    x, y = room[:, :cin], room[:, cin:cin + cout]
    assert torch.equal(api.linear_fwd(x, W, b, api.ACT_SILU, y, Y=y).Y, want)
    assert torch.equal(x, X) and (room[:, cin + cout:] == 0).all()
    grads = api.linear_bwd(dY, X, W)
    place = X.clone()
    got = api.linear_bwd(dY, place, W, need=("dX", "db"), out=(place, None, None))
    assert got.dX is place and torch.equal(place, grads.dX) and torch.equal(got.db, grads.db)


@pytest.mark.parametrize("own_stream", [False, True])
def test_a_large_workspace_is_given_back_with_the_call(own_stream):
    """dZ, the partial sums and a restored X do not outlive the call; the status does."""
    n, cin, cout = 20000, 264, 2056
    g = _gen(8)
    X, W, dY, Z = _rand(g, n, cin), _rand(g, cout, cin), _rand(g, n, cout), _rand(g, n, cout)
    x8 = api.ckpt8_pack(X)
    want = api.linear_bwd(dY, x8, W, Z, api.ACT_GELU,
                          ws=torch.empty(api.linear_workspace_size(n, cin, cout, api.ACT_GELU, True, True), dtype=torch.uint8,
                                         device="cuda"))
    assert want.ws.numel() > 2 * n * cout
    stream = torch.cuda.Stream() if own_stream else None
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    got = api.linear_bwd(dY, x8, W, Z, api.ACT_GELU, stream=stream)
    held = torch.cuda.memory_allocated() - before
    grads = sum(t.numel() * t.element_size() for t in (got.dX, got.dW, got.db))
    # the allocator gives a tensor up to 1 MiB more than asked for (a block's rest below that is not
    # split off): three gradients and the header; the workspace is 82 MB and more
    assert held <= grads + (4 << 20)
    torch.cuda.synchronize()
    assert api.workspace_status(got.ws) == _lib.PRISM_OK
    assert all(torch.equal(getattr(got, k), getattr(want, k)) for k in ("dX", "dW", "db"))
    small = api.linear_bwd(dY[:500], X[:500], W, Z[:500], api.ACT_GELU)
    assert small.ws.numel() > 256 and api.workspace_status(small.ws) == _lib.PRISM_OK


def test_the_status_of_a_large_call_in_a_graph():
    n, cin, cout = 20000, 264, 2056
    g = _gen(9)
    X, W, dY, Z = _rand(g, n, cin), _rand(g, cout, cin), _rand(g, n, cout), _rand(g, n, cout)
    want = api.linear_bwd(dY, X, W, Z, api.ACT_SILU)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = api.linear_bwd(dY, X, W, Z, api.ACT_SILU)
        later = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")    # may take the workspace's place
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert api.workspace_status(got.ws) == _lib.PRISM_OK and (later == 0).all()
        assert all(torch.equal(getattr(got, k), getattr(want, k)) for k in ("dX", "dW", "db"))
