"""The checkpoint's stated error: at most half a scale, which is less than 1/127 of
the block's largest value unless the scale is the smallest there is."""
import numpy as np
import pytest

from oracle import linear_oracle as L


def _error(x):
    codes, scales = L.ckpt8_pack(x)
    return np.abs(L.ckpt8_unpack(codes, scales, x.shape[1]) - x), np.exp2(scales.astype(np.float64) - 127), scales


def test_a_block_past_one_part_in_128():
    x = np.zeros((1, 32))
    x[0, :2] = 63.75, 0.5                       # scale 1: 0.5 is a tie and becomes 0
    err, scale, _ = _error(x)
    assert scale[0, 0] == 1 and err[0, 1] == 0.5
    assert 63.75 / 128 < err[0, 1] < 63.75 / 127


@pytest.mark.parametrize("spread", [1.0, 30.0])
def test_less_than_one_part_in_127(spread):
    r = np.random.default_rng(int(spread))
    x = r.normal(size=(400, 128)) * np.exp(spread * r.normal(size=(400, 1)))
    x[:100, ::32] = (63.5 + 2.0 ** -18) * np.exp2(r.integers(-100, 100, size=(100, 1)).astype(np.float64))
    err, scale, byte = _error(x)
    err, top = err.reshape(400, 4, 32).max(-1), np.abs(x).reshape(400, 4, 32).max(-1)
    assert (err <= scale / 2).all()
    assert (err < top / 127)[byte > 1].all()


def test_the_smallest_scale_has_no_such_bound():
    x = np.zeros((1, 32))
    x[0, 0] = 2.0 ** -128
    err, _, byte = _error(x)
    assert byte[0, 0] == 1 and err[0, 0] == x[0, 0]
