"""GPU parity of prism_ckpt8_pack / prism_ckpt8_unpack with the float64
statement of the format: codes, scales and restored values are determined
exactly (power-of-two scales, ties to even), so every comparison is equality."""
import numpy as np
import pytest
import torch

from dynamic_block_sparse_stats_b200 import api
from oracle import linear_oracle as L

pytestmark = pytest.mark.gpu


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _check(x):
    c = api.ckpt8_pack(x)
    y = api.ckpt8_unpack(c)
    torch.cuda.synchronize()
    n, width = x.shape
    codes, scales = L.ckpt8_pack(x.float().cpu().numpy().astype(np.float64))
    got_s = c.scales.cpu().numpy()
    blocks = (width + 31) // 32
    assert np.array_equal(got_s[:, :blocks], scales[:, :blocks])
    assert np.array_equal(c.codes.cpu().numpy(), codes)
    want = L.ckpt8_unpack(codes, scales, width)
    assert np.array_equal(y.float().cpu().numpy().astype(np.float64), want, equal_nan=True)
    return c, y


@pytest.mark.parametrize("n,width,pad", [(1, 8, 0), (1, 1024, 0), (3, 40, 8), (7, 128, 0), (5, 136, 120), (33, 328, 696),
                                         (2, 4104, 0), (64, 1000, 24)])
def test_codes_scales_and_values(n, width, pad):
    g = _gen(n * 10007 + width)
    rows = torch.exp(4 * torch.randn(n, 1, generator=g, device="cuda"))
    x = (torch.randn(n, width + pad, generator=g, device="cuda") * rows).to(torch.bfloat16)
    _check(x[:, :width])


def test_borders_ties_and_extremes():
    """Blocks whose maximum sits at 127 and 127.5 times a power of two, halves
    that round to even, the largest finite values, subnormals, zeros of both
    signs."""
    rows = []
    for e in (-133, -127, -126, -120, -20, 0, 7, 100, 120, 121):
        for m in (127.0, 127.5, 126.5, 64.0, 63.5, 1.0):
            r = np.zeros(128)
            r[0] = m * 2.0 ** e
            r[1:32] = np.arange(-15, 16) / 2 * 2.0 ** e
            r[40] = -m * 2.0 ** e
            r[64] = -0.0
            rows.append(r)
    big = np.zeros(128)
    big[:4] = [3.3895313892515355e38, -3.3895313892515355e38, 1.0, 2.0 ** 127]
    rows.append(big)
    _check(torch.tensor(np.array(rows), dtype=torch.float64).to(torch.bfloat16).cuda())


def test_non_finite_blocks_restore_nan_and_leave_their_neighbours():
    x = torch.randn(6, 128, generator=_gen(3), device="cuda").to(torch.bfloat16)
    x[0, 5] = float("inf")
    x[1, 40] = float("-inf")
    x[2, 127] = float("nan")
    x[3, 31], x[3, 32] = float("nan"), float("inf")
    x[4, :] = float("nan")
    _, y = _check(x)
    y = y.float().cpu()
    for r, b in ((0, 0), (1, 1), (2, 3), (3, 0), (3, 1)):
        assert torch.isnan(y[r, 32 * b:32 * b + 32]).all()
    assert torch.isfinite(y[5]).all() and torch.isfinite(y[0, 32:]).all()


def test_the_error_is_at_most_half_a_scale():
    x = torch.randn(257, 520, generator=_gen(4), device="cuda").to(torch.bfloat16)
    c, y = _check(x)
    half = torch.ldexp(torch.ones_like(c.scales, dtype=torch.float64), c.scales.int() - 128)
    half = half.repeat_interleave(32, dim=1)[:, :520]
    assert ((y.double() - x.double()).abs() <= half).all()


def test_out_buffers_strided_rows_and_what_lies_behind_them():
    g = _gen(5)
    x = torch.randn(9, 264, generator=g, device="cuda").to(torch.bfloat16)
    c = api.alloc_ckpt8(9, 264, "cuda")
    assert api.ckpt8_pack(x, out=c) is c
    room = torch.full((11, 400), 7.0, dtype=torch.bfloat16, device="cuda")
    y = api.ckpt8_unpack(c, out=room[1:10, :264])
    torch.cuda.synchronize()
    assert torch.equal(y, api.ckpt8_unpack(api.ckpt8_pack(x)))
    assert (room[0] == 7).all() and (room[10] == 7).all() and (room[:, 264:] == 7).all()


def test_empty_and_streams_and_graph():
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    assert api.ckpt8_unpack(api.ckpt8_pack(e)).shape == (0, 64)
    x = torch.randn(300, 512, generator=_gen(6), device="cuda").to(torch.bfloat16)
    want = api.ckpt8_unpack(api.ckpt8_pack(x))
    c, y = api.alloc_ckpt8(300, 512, "cuda"), torch.empty_like(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    api.ckpt8_pack(x, out=c, stream=s)
    api.ckpt8_unpack(c, out=y, stream=s)
    s.synchronize()
    assert torch.equal(y, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.ckpt8_pack(x, out=c)
        api.ckpt8_unpack(c, out=y)
    x2 = torch.randn_like(x)
    x.copy_(x2)
    y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, api.ckpt8_unpack(api.ckpt8_pack(x2)))


def test_offsets_past_32_bits():
    """2.4e9 values: the last rows of the codes lie past 2^31 elements."""
    n, w = 600_000, 4000
    x = torch.empty(n, w, dtype=torch.bfloat16, device="cuda")
    x[:] = torch.randn(1, w, generator=_gen(7), device="cuda")
    x[-1] = torch.randn(w, generator=_gen(8), device="cuda")
    y = api.ckpt8_unpack(api.ckpt8_pack(x))
    torch.cuda.synchronize()
    pick = torch.tensor([0, n // 2, n - 2, n - 1], device="cuda")
    want = api.ckpt8_unpack(api.ckpt8_pack(x[pick]))
    assert torch.equal(y[pick], want)
