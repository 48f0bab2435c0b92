"""A step of beam search where logits differ by less than totals hold, with nothing left out of the comparison."""
import math

import numpy as np
import pytest

import pages_util as pu
from test_beam_gpu import Step, dev_f32, tolerance, tsd  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu


def flat(parents, tokens, b, K, V):
    """The chosen pairs' places in their sentence."""
    return [(int(p) - b * K) * V + int(t) for p, t in zip(parents[b], tokens[b])]


@pytest.mark.parametrize("end", [1, -1])
@pytest.mark.parametrize("K", [1, 16])
@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("V,pad", [(129, 0), (200, 0), (200, 1), (2000, 0), (2001, 0), (9000, 3), (40000, 0)])
def test_different_logits_with_one_total(tsd, V, pad, f32, K, end):  # noqa: F811
    """Logits v 10^-25: all totals are -2.5 - log V in 48 bits (the logits reach 2^-67, a total's last bit is
    2^-46 and more), so that the lowest places are the best."""
    B = 2
    s = Step(tsd, B, K, V, f32, end, pad=pad)
    s.fill(np.broadcast_to(np.arange(V) * 1e-25, (B, K, V)))
    s.scores.copy_(dev_f32(np.full((B, K), -2.5)))
    s.run()
    tokens, parents, new, ended, rows, _ = s.get()
    want = [at for at in range(2 * K if end >= 0 else K) if at % V != end][:K]
    total = -2.5 - math.log(V)
    for b in range(B):
        assert flat(parents, tokens, b, K, V) == want
        assert (np.abs(new[b] - total) <= tolerance(total)).all()
        if end >= 0:  # the end token of the first beam is among the first 2 K places, no other beam's
            assert abs(ended[b, 0] - total) <= tolerance(total) + 2.0 ** -24 * abs(total)
            assert rows[b, 0] == b * K and (ended[b, 1:] == -np.inf).all()
    assert tsd.attn_get_device_status() == tsd.ATTN_OK


@pytest.mark.parametrize("K,V", [(1, 300), (4, 300), (4, 5000), (16, 700), (16, 2000)])
def test_some_ahead_of_many_with_one_total(tsd, K, V):  # noqa: F811
    """A few logits of 1 in the first row, at late places, and of the others all different with the same total."""
    s = Step(tsd, 1, K, V, True, -1)
    x = np.broadcast_to(2.0 ** -60 * (1 + np.arange(V) * 7919 % V * 2.0 ** -23), (1, K, V)).copy()
    few = sorted(V - 1 - 11 * j for j in range(max(K // 2, 1)))
    x[0, :, few] = 1
    assert len(np.unique(s.fill(x)[0, 0])) > 250
    s.scores.copy_(dev_f32(np.where(np.arange(K) == 0, -1.0, -30.0)[None]))
    s.run()
    tokens, parents, new = s.get()[:3]
    want = (few + [v for v in range(V) if v not in few])[:K]
    assert flat(parents, tokens, 0, K, V) == want and np.isfinite(new).all()


@pytest.mark.parametrize("K", [1, 5, 16])
@pytest.mark.parametrize("V", [150, 1000, 2000, 30000])
def test_totals_apart_by_their_last_bits(tsd, V, K):  # noqa: F811
    """Logits of 2^-41, whose totals (below 16) come out of three roundings of 2^-46 at most each: two of them that
    are further apart than 2^-43 are in their order, so that the j-th chosen logit is the j-th largest to 2^-43."""
    rng = np.random.default_rng(V + K)
    s = Step(tsd, 1, K, V, True, -1)
    x = s.fill(np.broadcast_to(2.0 ** -41 * rng.standard_normal(V), (1, K, V)))
    s.scores.copy_(dev_f32(np.full((1, K), -2.5)))
    s.run()
    tokens, parents, new = s.get()[:3]
    at = flat(parents, tokens, 0, K, V)
    assert len(set(at)) == K and np.isfinite(new).all()
    best = -np.sort(-x[0].ravel())[:K]
    assert (np.abs(x[0].ravel()[at] - best) <= 2.0 ** -43).all()


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("V,pad", [(700, 0), (5001, 0), (5000, 8), (40960, 0)])
def test_equal_logits_of_different_beams(tsd, f32, V, pad):  # noqa: F811
    """Whole numbers of three values, each beam its own: ties within a beam, log-sums that differ."""
    rng = np.random.default_rng(V)
    K = 4
    s = Step(tsd, 1, K, V, f32, V - 1, pad=pad)
    x = s.fill(rng.integers(0, 3, (1, K, V)).astype(float))
    s.scores.copy_(dev_f32(np.full((1, K), -2.5)))
    old = [t.cpu().numpy() for t in s.ended]
    tokens, parents, new, _, close = pu.select(x, np.full((1, K), -2.5), [1], V - 1, 0.6, old)
    assert not close
    s.run()
    got = s.get()
    assert np.array_equal(got[0], tokens) and np.array_equal(got[1], parents)
    assert (np.abs(got[2] - new) <= tolerance(new)).all()
