"""Ended hypotheses whose totals lie at the ends of fp32's range."""
import numpy as np
import pytest

from test_beam_gpu import Step, dev_f32, tsd  # noqa: F401 (the fixture)
from gpu_util import to_dev_i32

pytestmark = pytest.mark.gpu

LOWEST = {True: -float(np.finfo(np.float32).max), False: -float.fromhex("0x1.fep127")}


@pytest.mark.parametrize("n", [1, 2, 5, 10, 59, 2 ** 31 - 1])
@pytest.mark.parametrize("alpha", [0.6, 1.0, 2.0, 0.01, -0.01, -0.6, 30.0])
@pytest.mark.parametrize("f32", [True, False])
def test_an_end_token_masked_with_the_lowest_number(tsd, f32, alpha, n):  # noqa: F811
    """It is a candidate where there are few others, and its total over the penalty a number if that is one: two
    roundings to 32 bits, the total's and the quotient's, 2^-25 for the penalty's power and alpha times 2^-28 for the
    logarithm in it; below the smallest normal number four roundings more, of 2^-150."""
    s = Step(tsd, 2, 2, 3, f32, 0, alpha=alpha)
    x = np.full((2, 2, 3), -np.inf)
    x[..., 0], x[..., 1] = LOWEST[f32], 3.0
    s.fill(x)
    s.scores.copy_(dev_f32([[-0.5, -np.inf], [-np.inf, -2.0]]))
    s.lengths.copy_(to_dev_i32([n, n]))
    s.run()
    got = s.get()
    assert got[0][:, 0].tolist() == [1, 1] and got[1][:, 0].tolist() == [0, 3]
    log_penalty = alpha * np.log((5 + n) / 6)
    total = np.float64(LOWEST[f32])  # the others' parts of it are far below its rounding
    with np.errstate(over="ignore"):
        want = total / np.exp(log_penalty)
    largest = float(np.finfo(np.float32).max)
    relative = (3 + abs(alpha) / 16) * 2.0 ** -24
    assert (got[3][:, 1] == -np.inf).all()
    if want < -largest * (1 + relative):
        assert (got[3][:, 0] == -np.inf).all()
    elif want > -largest * (1 - relative):
        assert (np.abs(got[3][:, 0] - want) <= relative * abs(want) + 2.0 ** -148).all(), (got[3], want)
        assert got[4][:, 0].tolist() == [0, 3] and got[5][:, 0].tolist() == [n, n]
    assert tsd.attn_get_device_status() == tsd.ATTN_OK


@pytest.mark.parametrize("total", [-1.2e38, -2.0 ** 126, -2.0 ** 100, -1e20, -1.0, -1e-20, -2.0 ** -100, 1e30, 2.9e38])
def test_totals_of_every_size(tsd, total):  # noqa: F811
    """A beam that ends for certain: its total is its score (at most two roundings and the penalty's)."""
    for n, alpha in ((10, 0.6), (4, 1.0), (30, -0.3), (7, 2.0)):
        s = Step(tsd, 1, 1, 2, True, 0, alpha=alpha)
        s.fill(np.array([[[0.0, -np.inf]]]))
        s.scores.copy_(dev_f32([[total]]))
        s.lengths.copy_(to_dev_i32([n]))
        s.run()
        got = s.get()
        want = float(np.float32(total)) / ((5 + n) / 6) ** alpha
        if abs(want) < 3.4e38:
            assert abs(got[3][0, 0] - want) <= 4 * 2.0 ** -24 * abs(want), (n, alpha, got[3], want)
            assert got[4][0, 0] == 0 and got[5][0, 0] == n
