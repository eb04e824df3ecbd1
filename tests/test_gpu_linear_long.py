"""Weight gradients over very many tokens, with sums that keep their sign: the
tensor cores' accumulator truncates, so that one chain over all of them falls
short by more than the output's rounding.

Tolerance, relative to the value (all terms are positive): the output's rounding
2^-8 (bf16); a chain of at most 512 stages is 2048 instructions of 16 products,
each of which drops less than 2^-22 of the running sum, 2^-11; the chains' rounded
sums and the parts' add less than 2^-16.  In fp32, a chain of 8 stages: 2^-17, and
an addition a chain."""
import pytest
import torch

from dynamic_block_sparse_stats_b200 import api

pytestmark = pytest.mark.gpu


def _positive(seed, n, c):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.empty(n, c, dtype=torch.bfloat16, device="cuda")
    for at in range(0, n, 65536):
        m = min(65536, n - at)
        x[at:at + m] = torch.randn(m, c, generator=g, device="cuda").abs()
    return x


def _exact(dY, X, rows, cols):
    out = torch.zeros(len(rows), len(cols), dtype=torch.float64, device="cuda")
    for a, x in zip(dY.split(65536), X.split(65536)):
        out += a[:, rows].double().t() @ x[:, cols].double()
    return out


# the layer's largest grid, whole waves of pair tiles; the same from a checkpoint that is
# converted on the way (out < 2048); single tiles (out = 128); a split last wave alone
@pytest.mark.parametrize("n,cin,cout", [(860160, 1280, 4096), (860160, 4864, 1024), (80000, 18944, 128), (860160, 1024, 1024),
                                        (33000, 2056, 2568)])
def test_sums_of_one_sign(n, cin, cout):
    X, dY = _positive(1, n, cin), _positive(2, n, cout)
    rows = torch.cat([torch.arange(0, 40), torch.arange(cout - 40, cout)]).cuda()
    cols = torch.cat([torch.arange(0, 72), torch.arange(cin - 72, cin)]).cuda()
    x8 = api.ckpt8_pack(X)
    for x in (X, x8):
        want = _exact(dY, api.ckpt8_unpack(x) if x is x8 else X, rows, cols)
        for fp32, tol in ((False, 2.0 ** -8 + 2.0 ** -11 + 2.0 ** -16), (True, 2.0 ** -17 + n / 512 * 2.0 ** -24)):
            g = api.linear_bwd(dY, x, None, need=("dW",), grad_fp32=fp32)
            assert api.workspace_status(g.ws) == 0
            off = ((g.dW[rows][:, cols].double() - want).abs() / want).max()
            print(f"{'checkpoint' if x is x8 else 'bf16'} {'fp32' if fp32 else 'bf16'}: {float(off / tol):.3f} of the tolerance")
            assert off <= tol
            # and the same bits from the restored tensor
            if x is x8:
                same = api.linear_bwd(dY, api.ckpt8_unpack(x8), None, need=("dW",), grad_fp32=fp32)
                assert torch.equal(same.dW, g.dW)


@pytest.mark.parametrize("n,out", [(300, 64), (3000, 256), (9500, 512)])
def test_the_longest_contraction_of_the_forward_and_of_dx(n, out):
    """65536 channels, 1024 stages in one chain: 4096 instructions, 2^-10, and the
    output's rounding, as above."""
    wide = 65536
    X, W = _positive(3, n, wide), _positive(4, out, wide)
    tol = 2.0 ** -8 + 2.0 ** -10 + 2.0 ** -16
    rows = torch.cat([torch.arange(0, 64), torch.arange(n - 64, n)]).cuda()
    want = X[rows].double() @ W.double().t()
    for save in (None, "bf16"):
        f = api.linear_fwd(X, W, save=save)
        assert api.workspace_status(f.ws) == 0
        for got in (f.Y, f.Z) if save else (f.Y,):
            off = float(((got[rows].double() - want).abs() / want).max())
            print(f"forward: {off / tol:.3f} of the tolerance")
            assert off <= tol
    # dX of a map to 65536 channels: the same product
    g = api.linear_bwd(X, None, W.t().contiguous(), need=("dX",))
    assert api.workspace_status(g.ws) == 0
    assert float(((g.dX[rows].double() - want).abs() / want).max()) <= tol
