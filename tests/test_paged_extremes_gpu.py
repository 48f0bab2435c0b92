"""GPU tests of the paged cache at the ends of its numbers' ranges: infinite and
very large values, very large and very small queries and factors. The cases and
their 64-bit definitions are test_paged_gpu's and paged_util's."""
import numpy as np
import pytest

import synthetic

import paged_util as pu
from gpu_util import to_dev_bf16, to_host_f64
from test_paged_gpu import DecodeCase, dev, tsd  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


def set_rows(c, pool, b, position, column, value):
    """One column of one cached row, of every key head, in a copy of a bf16 pool."""
    page = c.case[5]
    pool[int(c.table[b, position // page]), :, position % page, column] = value


INFINITE_CASES = [
    # B, h, h_kv, n_q, d, page, lens, new_lens or None, causal; the positions are counted from the end
    (2, 8, 8, 1, 64, 16, [200, 40], None, True),                       # whole, eight warps' block
    (2, 8, 2, 1, 128, 16, [700, 3000], None, True),                    # split
    (2, 8, 2, 3, 64, 16, [90, 1700], [3, 2], True),                    # 12 query rows, a padded sequence
    (3, 28, 4, 4, 128, 32, [500, 1411, 64], [4, 1, 3], True),          # 28 query rows
    (80, 14, 2, 4, 64, 16, [9 + b for b in range(80)], None, True),    # wide tiles, whole
    (43, 28, 4, 4, 128, 16, [(411 * b) % 2500 for b in range(43)], None, False),  # wide tiles, split, no mask
]


@pytest.mark.parametrize("case", INFINITE_CASES, ids=lambda c: "B{}h{}kv{}q{}d{}x{}".format(*c[:5], max(c[6])))
def test_an_infinite_value_that_a_query_sees_is_infinite_in_its_output(tsd, case):
    """Column 3 holds +inf, column 4 -inf, column 5 one of each (no number), in the first row and
    near the end of each sequence; the other columns are as the definition has them."""
    B, h, h_kv, n_q, d, page, lens, new, causal = case
    c = DecodeCase(case, False, seed=40)
    pools = [p.clone() for p in c.pools]
    places = [[] for _ in range(B)]  # (position, column, value)
    for b, L in enumerate(lens):
        if L < 6:
            continue
        for position in {0, L // 2, L - 1}:
            places[b] += [(position, 3, np.inf), (position, 4, -np.inf)]
        places[b] += [(1, 5, np.inf), (2, 5, -np.inf)]
        for position, column, value in places[b]:
            set_rows(c, pools[1], b, position, column, value)
    clean = []
    for b, rows in enumerate(c.v_rows):
        rows = rows.copy()
        for position, column, _ in places[b]:
            rows[:, position, column] = 0
        clean.append(rows)
    got = to_host_f64(c.run(tsd, pools=pools))
    ref, mass, size = pu.decode(c.q, c.k_rows, clean, lens, c.new, causal, 1 / np.sqrt(d))
    want = ref.copy()
    for b, L in enumerate(lens):
        for t in range(c.new[b]):
            seen = min(L, L - c.new[b] + t + 1) if causal else L
            for position, column, value in places[b]:
                if position < seen:
                    with np.errstate(invalid="ignore"):
                        want[b, :, t, column] += value
    tol = pu.decode_tolerance(ref, mass, size, max(max(lens), 1), d)
    finite = np.isfinite(want)
    assert np.all(np.abs(got - ref)[finite] <= tol[finite])
    assert np.array_equal(got[~finite], want[~finite], equal_nan=True)
    assert tsd.attn_get_device_status() == tsd.ATTN_OK


@pytest.mark.parametrize("case", [
    (2, 4, 4, 1, 64, 16, [200, 37], None, True),
    (2, 8, 2, 2, 128, 16, [900, 2500], None, True),
    (3, 28, 4, 4, 64, 32, [500, 1411, 64], [4, 1, 3], True),
    (80, 14, 2, 4, 128, 16, [30 + b for b in range(80)], None, True),
], ids=lambda c: "B{}h{}kv{}q{}d{}x{}".format(*c[:5], max(c[6])))
@pytest.mark.parametrize("rise", [2.0, 7.4, 30.0])
def test_values_near_the_largest_bf16(tsd, case, rise):
    """Two thirds into each sequence a row has a logit that is `rise` powers of 2 above the other
    rows' and values near bf16's largest; the other rows' are a thousandth of that. No sum of
    weights of at most 1 times values passes fp32's range."""
    B, h, h_kv, n_q, d, page, lens, new, causal = case
    c = DecodeCase(case, False, seed=50)
    rng = np.random.default_rng(51)
    q = np.zeros((B, h, n_q, d))
    q[..., 0] = 1
    pools = [p.clone() for p in c.pools]
    k_rows, v_rows = [], []
    f64 = lambda x: synthetic.bf16_bits_to_f64(synthetic.f32_to_bf16_bits(np.asarray(x, dtype=np.float32)))
    for b, L in enumerate(lens):
        k, v = c.k_rows[b].copy(), f64(c.v_rows[b] * 3e34)
        k[..., 0] = f64(rng.uniform(-0.3, 0.3, k.shape[:2]))
        at = 2 * L // 3
        k[:, at, 0] = f64(rise)
        v[:, at] = f64(3.3e38 * rng.choice([-1.0, 1.0], (h_kv, d)) * rng.uniform(0.9, 1.0, (h_kv, d)))
        p = np.arange(L)
        place = c.table[b, p // page], slice(None), p % page
        for pool, rows in zip(pools, (k, v)):
            pool.view(c.torch.int16)[place] = dev(synthetic.f32_to_bf16_bits(
                rows.swapaxes(0, 1).astype(np.float32)).view(np.int16))
        k_rows.append(k)
        v_rows.append(v)
    scale = float(np.float32(np.log(2)))
    out = c.run(tsd, q=to_dev_bf16(synthetic.f32_to_bf16_bits(q.astype(np.float32))), pools=pools,
                scale=scale)
    c.check(tsd, out, k_rows, v_rows, q=q, scale=scale)


@pytest.mark.parametrize("d", [64, 128])
def test_4_bit_logits_of_zero_with_the_largest_queries(tsd, d):
    """Keys of zero against queries up to bf16's largest and a large factor: every logit is 0, and
    the output the mean of the values."""
    c = DecodeCase((2, 8, 2, 2, d, 16, [130, 1500], None, True), True, seed=60)
    c.factors = (2.0 ** 20, 0.03)
    pools = [c.torch.zeros_like(c.pools[0])] + c.pools[1:]
    q = np.where(np.arange(8)[None, :, None, None] % 2, 3.3e38, 1.0) * np.sign(c.q)
    bits = synthetic.f32_to_bf16_bits(q.astype(np.float32))
    out = c.run(tsd, q=to_dev_bf16(bits), pools=pools, scale=1.0)
    c.check(tsd, out, [np.zeros_like(k) for k in c.k_rows], q=synthetic.bf16_bits_to_f64(bits), scale=1.0)
