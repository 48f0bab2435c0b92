"""GPU parity of the paged key/value cache: appending with the rotation, the
4-bit form, and the decoding step's attention over either cache, against
plain 64-bit forms; then the operators together, as a decoding loop runs them."""
import numpy as np
import pytest

import synthetic

import paged_util as pu
from gpu_util import to_dev_bf16, to_dev_i32, to_host_f64

pytestmark = pytest.mark.gpu

SENTINEL = 0x5a  # what rows nobody writes hold


@pytest.fixture(scope="module")
def tsd():
    import torch
    from transformer_scaled_dot_gb300 import build as native_build
    native_build.build()
    import transformer_scaled_dot_gb300 as m
    m.library()
    torch.cuda.set_device(0)
    return m


def bf16(rng, *shape):
    """Normal values as bf16 bits, and in 64 bits."""
    bits = synthetic.f32_to_bf16_bits(rng.standard_normal(shape).astype(np.float32))
    return bits, synthetic.bf16_bits_to_f64(bits)


def dev(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x)).to("cuda")


# ------------------------------------------------------------------ append

APPEND_CASES = [
    # B, n_new, h, h_kv, d, page, kind, dim, past (rows before), new_lens or None
    (1, 1, 1, 1, 64, 16, 0, 0, [0], None),                    # the first token of all
    (3, 1, 8, 8, 64, 16, 1, 64, [0, 15, 16], None),           # either side of a page's end
    (2, 37, 4, 2, 64, 32, 1, 32, [5, 60], [37, 11]),          # half of each head, a padded sequence
    (4, 5, 6, 3, 128, 16, 2, 64, [3, 100, 31, 7], [5, 0, 1, 4]),
    (2, 9, 10, 5, 128, 64, 2, 128, [60, 2], None),
    (1, 150, 7, 1, 128, 256, 1, 128, [200], None),            # across a large page's end
    (2, 20, 33, 11, 64, 128, 1, 64, [1, 0], None),            # an odd number of heads
    (1, 3, 16, 16, 128, 16, 1, 96, [14], None),
    (5, 2, 40, 8, 128, 16, 0, 0, [0, 1, 2, 3, 4], [2, 1, 2, 0, 2]),
]


def append_case(tsd, case, q4, factors=(0.0113, 0.0071), layout="fused", k_out=True, x_f64=None,
                bad_pages=()):
    """Runs one append on seeded inputs; returns what was written and what the inputs were."""
    import torch
    B, n, h, h_kv, d, page, kind, dim, past, new = case
    rng = np.random.default_rng(sum(case[:8]) + 1000 * q4)
    heads = h + 2 * h_kv
    if x_f64 is None:
        x_bits, x = bf16(rng, B, n, heads, d)
    else:
        x_bits = synthetic.f32_to_bf16_bits(x_f64.astype(np.float32))
        x = synthetic.bf16_bits_to_f64(x_bits)
    new = [n] * B if new is None else new
    lens = [p + m for p, m in zip(past, new)]
    table, n_pages = pu.page_table(rng, lens, page)
    for b, i, value in bad_pages:
        table[b, i] = value
    rope = pu.rope_table(max(lens) + 3, dim) if kind else None
    shape = (n_pages, h_kv, page)
    if q4:
        pools = [torch.full(shape + (w,), SENTINEL, dtype=torch.uint8, device="cuda")
                 for w in (d // 2, d // 16, d // 2, d // 16)]
        args = (*pools, *factors)
        call = tsd.attn_cache_append_q4
    else:
        pools = [torch.full(shape + (d * 2,), SENTINEL, dtype=torch.uint8, device="cuda")
                 for _ in range(2)]
        args = tuple(pools)
        call = tsd.attn_cache_append
    if layout == "fused":    # [B, n, h + 2 h_kv, d]: a projection's output
        xd = to_dev_bf16(x_bits)
        q, k, v = xd, xd[:, :, h:], xd[:, :, h + h_kv:]
        strides = (n * heads * d, d, heads * d)
        q_strides = kv_strides = strides
    else:                    # [B, heads, n, d], each tensor its own
        q, k, v = (to_dev_bf16(x_bits[:, :, a:z].swapaxes(1, 2))
                   for a, z in ((0, h), (h, h + h_kv), (h + h_kv, heads)))
        q_strides, kv_strides = (h * n * d, n * d, d), (h_kv * n * d, n * d, d)
    q_out = torch.full((B, h, n, d * 2), SENTINEL, dtype=torch.uint8, device="cuda")
    ko = torch.full((B, h_kv, n, d * 2), SENTINEL, dtype=torch.uint8, device="cuda") if k_out else None
    call(q, *q_strides, k, v, *kv_strides, q_out, ko, *args, to_dev_i32(table), to_dev_i32(lens),
         to_dev_i32(new), None if rope is None else dev(rope), 0 if rope is None else len(rope), dim,
         kind, B, h, h_kv, n, d, n_pages, page, table.shape[1])
    torch.cuda.synchronize()
    view = lambda t: t.view(torch.bfloat16)
    return dict(x=x, rope=rope, table=table, lens=lens, new=new, n_pages=n_pages, q_out=view(q_out),
                k_out=None if ko is None else view(ko), pools=pools,
                status=tsd.attn_get_device_status())


def rotated(r, case, b, t):
    """The token's rotated queries and keys, its values, and their position, in 64 bits."""
    B, n, h, h_kv, d, page, kind, dim, past, _ = case
    p = r["lens"][b] - r["new"][b] + t
    x = r["x"][b, t]
    y = pu.rotate(x[:h + h_kv], p, r["rope"], kind, dim)
    return y[:h], y[h:], x[h + h_kv:], p


def rotation_tolerance(y, x, dim):
    """bf16's rounding (2^-8 of the value) after three 32-bit roundings of numbers no larger
    than twice the token's largest value."""
    return 2.0 ** -8 * np.abs(y) + (6 * 2.0 ** -24 * np.abs(x).max() if dim else 0)


@pytest.mark.parametrize("layout", ["fused", "heads"])
@pytest.mark.parametrize("case", APPEND_CASES, ids=lambda c: "B{}n{}h{}kv{}d{}p{}r{}x{}".format(*c[:8]))
def test_append_writes_the_rotated_rows_and_nothing_else(tsd, case, layout):
    B, n, h, h_kv, d, page, kind, dim, past, _ = case
    r = append_case(tsd, case, q4=False, layout=layout)
    assert r["status"] == tsd.ATTN_OK
    kc, vc = (to_host_f64(p.view(__import__("torch").bfloat16)) for p in r["pools"])
    raw = [p.cpu().numpy() for p in r["pools"]]
    q_out, k_out = to_host_f64(r["q_out"]), to_host_f64(r["k_out"])
    untouched = np.ones((r["n_pages"], page), dtype=bool)
    sentinel = to_host_f64(__import__("torch").full((2,), SENTINEL, dtype=__import__("torch").uint8)
                           .view(__import__("torch").bfloat16))[0]
    for b in range(B):
        for t in range(n):
            if t >= r["new"][b]:
                assert np.all(q_out[b, :, t] == sentinel) and np.all(k_out[b, :, t] == sentinel)
                continue
            q, k, v, p = rotated(r, case, b, t)
            tol = rotation_tolerance(q, r["x"][b, t], dim)
            assert np.all(np.abs(q_out[b, :, t] - q) <= tol)
            at, slot = r["table"][b, p // page], p % page
            untouched[at, slot] = False
            tol = rotation_tolerance(k, r["x"][b, t], dim)
            assert np.all(np.abs(kc[at, :, slot] - k) <= tol)
            assert np.array_equal(k_out[b, :, t], kc[at, :, slot])
            assert np.array_equal(vc[at, :, slot], v)
    for pool in raw:  # every slot that no token has is as it was
        assert np.all(pool.swapaxes(1, 2)[untouched] == SENTINEL)


def check_groups(codes, scales, want, error, factor):
    """codes [.., d/2], scales [.., d/16] against 64-bit values `want` [.., d] that the kernel
    has to within `error`: each number is one of the nearest its place has, allowing for that
    error (and 2^-22 of the quotient's own roundings)."""
    f = float(np.float32(factor))
    g = want.reshape(want.shape[:-1] + (-1, 16))
    s = pu.E4M3[scales]
    ideal = np.minimum(np.abs(g).max(-1) / (6 * f), 448.0)
    slack = np.broadcast_to(np.asarray(error) / (6 * f), ideal.shape) + ideal * 2.0 ** -22
    table = pu.E4M3[:0x7f]
    nearest = np.abs(ideal[..., None] - table).min(-1)
    assert np.all(np.abs(ideal - s) <= nearest + 2 * slack)
    y = np.where(s[..., None] > 0, g / np.maximum(s[..., None] * f, 1e-300), 0.0)
    slack = np.where(s > 0, np.asarray(error) / np.maximum(s * f, 1e-300), 0.0)[..., None] + np.abs(y) * 2.0 ** -22
    got = pu.code_values(codes).reshape(g.shape)
    y = np.clip(y, -6, 6)
    nearest = np.abs(y[..., None] - pu.E2M1).min(-1)
    assert np.all(np.abs(y - got) <= nearest + 2 * slack)
    return got * s[..., None] * f


@pytest.mark.parametrize("case", APPEND_CASES, ids=lambda c: "B{}n{}h{}kv{}d{}p{}r{}x{}".format(*c[:8]))
def test_append_q4_rounds_to_the_nearest_scale_and_codes(tsd, case):
    B, n, h, h_kv, d, page, kind, dim, past, _ = case
    factors = (0.0113, 0.0071)
    r = append_case(tsd, case, q4=True, factors=factors, layout="heads" if n % 2 else "fused")
    assert r["status"] == tsd.ATTN_OK
    pools = [p.cpu().numpy() for p in r["pools"]]
    q_out, k_out = to_host_f64(r["q_out"]), to_host_f64(r["k_out"])
    untouched = np.ones((r["n_pages"], page), dtype=bool)
    for b in range(B):
        for t in range(r["new"][b]):
            q, k, v, p = rotated(r, case, b, t)
            assert np.all(np.abs(q_out[b, :, t] - q) <= rotation_tolerance(q, r["x"][b, t], dim))
            assert np.all(np.abs(k_out[b, :, t] - k) <= rotation_tolerance(k, r["x"][b, t], dim))
            at, slot = r["table"][b, p // page], p % page
            untouched[at, slot] = False
            error = 6 * 2.0 ** -24 * np.abs(r["x"][b, t]).max() if dim else 0.0
            check_groups(pools[0][at, :, slot], pools[1][at, :, slot], k, error, factors[0])
            check_groups(pools[2][at, :, slot], pools[3][at, :, slot], v, 0.0, factors[1])
    for pool in pools:
        assert np.all(pool.swapaxes(1, 2)[untouched] == SENTINEL)


def test_append_q4_edges(tsd):
    """Zero groups, ties (to the even code), values over the largest, tiny ones, infinities, NaN."""
    case = (1, 1, 1, 1, 128, 16, 0, 0, [0], None)
    x = np.zeros((1, 1, 3, 128))
    k = x[0, 0, 1].reshape(8, 16)
    k[1] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5, -6]
    k[2, :2] = [2.0 ** 20, 3000.0]            # scale limited to 448
    k[3, :2] = [2.0 ** -20, -2.0 ** -21]      # scale rounds to 0
    k[4, :2] = [np.inf, 1]
    k[5, :2] = [np.nan, 1]
    k[6] = np.arange(16) * 9 / 8 / 4          # ties at a scale that is no power of two
    k[6, 15] = 6 * 9 / 8
    k[7, 0] = -np.inf
    with np.errstate(invalid="ignore"):
        r = append_case(tsd, case, q4=True, factors=(1.0, 1.0), x_f64=x)
    codes, scales = (p.cpu().numpy()[r["table"][0, 0], 0, 0] for p in r["pools"][:2])
    got = pu.code_values(codes).reshape(8, 16)
    assert list(scales) == [0, 0x38, 0x7e, 0, 0x7f, 0x7f, 0x39, 0x7f]
    assert np.all(got[[0, 3, 4, 5, 7]] == 0)
    assert np.array_equal(got[1], [6, 0, 1, 1, 2, 2, 4, 4, 0, -1, -1, -2, -2, -4, -4, -6])
    assert np.array_equal(got[2, :3], [6, 6, 0])
    assert np.array_equal(got[6, :9], [0, 0, 0.5, 1, 1, 1, 1.5, 2, 2])
    # the values' pool took the third head
    assert np.all(r["pools"][3].cpu().numpy()[r["table"][0, 0], 0, 0] == 0)


@pytest.mark.parametrize("q4", [False, True])
def test_append_leaves_out_tokens_without_a_page(tsd, q4):
    """A bad page index, a position past the table: reported, nothing written through it."""
    case = (3, 3, 2, 1, 64, 16, 1, 64, [14, 40, 2], None)
    r = append_case(tsd, case, q4, bad_pages=[(0, 1, 1 << 30), (1, 2, -7)])
    assert r["status"] == tsd.ATTN_ERR_DEVICE_INDEX
    assert tsd.attn_get_device_status() == tsd.ATTN_OK  # said once
    raw = r["pools"][0].cpu().numpy()
    written = (raw != SENTINEL).any(-1).any(1)          # [page, slot]
    want = np.zeros_like(written)
    want[r["table"][0, 0], 14:16] = True                # sequence 0: its third token's page is bad
    want[r["table"][2, 0], 2:5] = True                  # sequence 1: all three
    assert np.array_equal(written, want)


def test_append_skips_what_has_no_place(tsd):
    """More new tokens than rows: those at negative positions are not written. Positions past the
    rotation's table or the page table are, like bad pages, reported."""
    import torch
    B, n, h, h_kv, d, page = 3, 4, 1, 1, 64, 16
    x = torch.ones(B, n, 3, d, dtype=torch.bfloat16, device="cuda")
    pools = [torch.zeros(8, 1, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    table = to_dev_i32([[0, 1], [2, 3], [4, 5]])
    rope = dev(pu.rope_table(20, d))
    q_out = torch.zeros(B, h, n, d, dtype=torch.bfloat16, device="cuda")

    def call(lens, rope_rows):
        tsd.attn_cache_append(x, n * 3 * d, d, 3 * d, x[:, :, 1:], x[:, :, 2:], n * 3 * d, d, 3 * d,
                              q_out, None, *pools, table, to_dev_i32(lens), None, rope, rope_rows, d, 1,
                              B, h, h_kv, n, d, 8, page, 2)
        return tsd.attn_get_device_status()
    assert call([2, -3, 0], 20) == tsd.ATTN_OK
    v = pools[1][:, 0, :, 0].cpu().float().numpy()
    assert np.array_equal(np.argwhere(v), [[0, 0], [0, 1]])
    assert np.array_equal(q_out[:, 0, :, 0].float().cpu().numpy() != 0,
                          [[0, 0, 1, 1], [0, 0, 0, 0], [0, 0, 0, 0]])
    assert call([22, 4, 4], 20) == tsd.ATTN_ERR_DEVICE_INDEX  # rows 20, 21 have no angles
    v = pools[1][:, 0, :, 0].cpu().float().numpy()
    assert np.array_equal(np.argwhere(v[1]), [[2], [3]])
    assert call([4, 34, 2 ** 31 - 1], 20) == tsd.ATTN_ERR_DEVICE_INDEX  # past the page table


def test_append_in_place_and_without_queries(tsd):
    import torch
    B, n, h, h_kv, d, page = 2, 3, 4, 2, 64, 16
    rng = np.random.default_rng(5)
    bits, _ = bf16(rng, B, h, n, d)
    kv, _ = bf16(rng, 2, B, h_kv, n, d)
    rope = dev(pu.rope_table(16, d))
    table, lens = to_dev_i32([[1], [0]]), to_dev_i32([9, 3])
    run = lambda q, out, pools: tsd.attn_cache_append(
        q, h * n * d, n * d, d, *to_dev_bf16(kv), h_kv * n * d, n * d, d, out, None, *pools, table,
        lens, None, rope, 16, d, 2, B, h, h_kv, n, d, 2, page, 1)
    new_pools = lambda: [torch.zeros(2, h_kv, page, d, dtype=torch.bfloat16, device="cuda")
                         for _ in range(2)]
    a, b, c = new_pools(), new_pools(), new_pools()
    q = to_dev_bf16(bits)
    out = torch.empty_like(q)
    run(q, out, a)
    run(q, q, b)       # in place
    run(None, None, c)
    torch.cuda.synchronize()
    assert torch.equal(out, q)
    for x, y, z in zip(a, b, c):
        assert torch.equal(x, y) and torch.equal(x, z)
    assert tsd.attn_get_device_status() == tsd.ATTN_OK


def test_append_of_almost_only_padding(tsd):
    """The largest n_new: three tokens and 2^31 - 4 that are padding, which is never read."""
    import torch
    n, d, page, h_kv = 2 ** 31 - 1, 64, 16, 2
    rng = np.random.default_rng(17)
    bits, x = bf16(rng, 2, 3, h_kv, d)
    k, v = to_dev_bf16(bits)
    pools = [torch.zeros(2, h_kv, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    tsd.attn_cache_append(None, 0, 0, 0, k, v, 0, d, h_kv * d, None, None, *pools,
                          to_dev_i32([[1, 0]]), to_dev_i32([17]), to_dev_i32([3]), None, 0, 0, 0,
                          1, h_kv, h_kv, n, d, 2, page, 2)
    torch.cuda.synchronize()
    assert tsd.attn_get_device_status() == tsd.ATTN_OK
    for pool, rows in zip(pools, x):
        want = np.zeros((2, h_kv, page, d))
        want[1, :, 14], want[1, :, 15], want[0, :, 0] = rows  # positions 14, 15 and 16
        assert np.array_equal(to_host_f64(pool), want)


# ------------------------------------------------------------------ decode

DECODE_CASES = [
    # B, h, h_kv, n_q, d, page, lens, new_lens or None, causal
    (1, 1, 1, 1, 64, 16, [1], None, True),
    (1, 8, 8, 1, 64, 16, [200], None, True),
    (4, 8, 2, 1, 128, 16, [0, 1, 16, 17], None, True),               # an empty cache, pages' ends
    (3, 6, 3, 2, 64, 32, [63, 64, 65], None, True),
    (2, 12, 4, 3, 128, 16, [2, 700], None, True),                    # more new tokens than rows
    (5, 8, 1, 8, 64, 64, [8, 129, 500, 7, 64], [8, 3, 8, 0, 1], True),   # 64 rows of queries, padding
    (2, 28, 4, 4, 128, 128, [513, 300], [4, 2], True),               # 28 rows of queries
    (3, 5, 5, 1, 128, 256, [1000, 3, 257], None, True),
    (3, 16, 4, 3, 64, 16, [33, 100, 900], [3, 3, 1], False),         # no causal mask
    (2, 33, 11, 5, 64, 16, [77, 1500], None, False),
    (1, 64, 1, 8, 128, 16, [260], None, True),                       # 512 rows of queries
    (40, 4, 2, 1, 64, 16, [(37 * b) % 211 for b in range(40)], None, True),
    (1, 8, 2, 1, 128, 16, [5003], None, True),                       # one long sequence, split
    (2, 4, 1, 2, 64, 64, [9001, 1], None, True),
    (300, 2, 1, 1, 64, 16, [b % 19 for b in range(300)], None, True),  # more sequences than threads
    (70, 16, 8, 1, 64, 16, [(389 * b) % 1500 for b in range(70)], None, True),  # more pairs than blocks
    (400, 2, 2, 2, 128, 32, [5000] + [(7 * b) % 60 for b in range(399)], None, True),  # one long among short
    (1000, 1, 1, 1, 64, 64, [(b * b) % 97 for b in range(999)] + [2500], None, False),
    (3, 8, 8, 1, 128, 16, [1280, 1290, 4], None, True),              # just too long to be left whole
    (3, 8, 8, 1, 128, 16, [1264, 1250, 4], None, True),              # just short enough
    # wide query tiles (16 and 32 rows), whole and split, of both head sizes
    (33, 12, 4, 8, 64, 16, [(211 * b) % 2100 for b in range(33)], [b % 9 for b in range(33)], True),
    (3, 12, 4, 4, 128, 16, [1400, 5, 2000], None, True),
    (40, 28, 4, 4, 128, 32, [(97 * b) % 300 for b in range(40)], None, True),
    (42, 28, 4, 4, 128, 16, [(411 * b) % 1700 for b in range(42)], [4 - b % 5 for b in range(42)], True),
    (60, 18, 1, 2, 64, 16, [(31 * b) % 200 for b in range(60)], None, False),
    (5, 36, 2, 2, 64, 16, [1, 1500, 33, 700, 64], None, False),
]
decode_ids = lambda c: "B{}h{}kv{}q{}d{}p{}x{}".format(*c[:6], max(c[6]))


class DecodeCase:
    def __init__(self, case, q4, seed=0, spread=1.0):
        import torch
        self.case, self.q4 = case, q4
        B, h, h_kv, n_q, d, page, lens, new, causal = case
        rng = np.random.default_rng(seed + sum(case[:6]))
        self.new = [n_q] * B if new is None else new
        self.table, self.n_pages = pu.page_table(rng, lens, page)
        self.q_bits, self.q = bf16(rng, B, h, n_q, d)
        shape = (self.n_pages, h_kv, page)
        self.factors = (0.0625 * spread, 0.03)
        if q4:
            # codes of any value, scales from 2^-6 up to 2^5
            codes = [rng.integers(0, 256, shape + (d // 2,), dtype=np.uint8) for _ in range(2)]
            scales = [rng.integers(0x08, 0x60, shape + (d // 16,), dtype=np.uint8) for _ in range(2)]
            rows = [pu.dequantise(c, s, f) for c, s, f in zip(codes, scales, self.factors)]
            self.k_rows, self.v_rows = ([pu.gather(x, self.table[b], lens[b], page) for b in range(B)]
                                        for x in rows)
            # whatever no row uses holds NaN
            used = np.zeros((self.n_pages, page), dtype=bool)
            for b in range(B):
                p = np.arange(lens[b])
                used[self.table[b, p // page], p % page] = True
            for s in scales:
                s.swapaxes(1, 2)[~used] = 0x7f
            self.pools = [dev(codes[0]), dev(scales[0]), dev(codes[1]), dev(scales[1])]
        else:
            bits, rows = zip(*(bf16(rng, *shape, d) for _ in range(2)))
            self.k_rows, self.v_rows = ([pu.gather(x, self.table[b], lens[b], page) for b in range(B)]
                                        for x in rows)
            used = np.zeros((self.n_pages, page), dtype=bool)
            for b in range(B):
                p = np.arange(lens[b])
                used[self.table[b, p // page], p % page] = True
            for x in bits:
                x.swapaxes(1, 2)[~used] = 0x7fc0
            self.pools = [to_dev_bf16(x) for x in bits]
        self.dev = dict(q=to_dev_bf16(self.q_bits), table=to_dev_i32(self.table),
                        lens=to_dev_i32(lens), new=None if new is None else to_dev_i32(new))
        self.torch = torch

    def run(self, tsd, q=None, pools=None, workspace=None, out=None, stream=None, **change):
        B, h, h_kv, n_q, d, page, lens, new, causal = self.case
        a = {**self.dev, **change}
        wsb = tsd.attn_decode_paged_workspace_bytes(B, h, h_kv, n_q, d, page, self.table.shape[1])
        ws = self.torch.empty(wsb, dtype=self.torch.uint8, device="cuda") if workspace is None else workspace
        self.workspace = ws  # kept until the work is done
        if out is None:
            out = self.torch.full((B, h, n_q, d), float("nan"), dtype=self.torch.bfloat16, device="cuda")
        tail = (out, a["table"], a["lens"], a["new"], B, h, h_kv, n_q, d, self.n_pages, page,
                self.table.shape[1], 1 if causal else 0, a.get("scale", 0.0), ws, wsb, stream)
        q = a["q"] if q is None else q
        pools = self.pools if pools is None else pools
        if self.q4:
            tsd.attn_decode_paged_q4(q, *pools, *self.factors, *tail)
        else:
            tsd.attn_decode_paged(q, *pools, *tail)
        return out

    def check(self, tsd, out, k_rows=None, v_rows=None, q=None, scale=None, rows=slice(None)):
        B, h, h_kv, n_q, d, page, lens, new, causal = self.case
        self.torch.cuda.synchronize()
        got = to_host_f64(out)
        ref, mass, size = pu.decode(self.q if q is None else q, self.k_rows if k_rows is None else k_rows,
                                    self.v_rows if v_rows is None else v_rows, lens, self.new, causal,
                                    1 / np.sqrt(d) if scale is None else scale)
        got, ref, mass, size = got[rows], ref[rows], mass[rows], size[rows]
        assert np.all(np.isfinite(got))
        tol = pu.decode_tolerance(ref, mass, size, max(max(lens), 1), d)
        assert np.all(np.abs(got - ref) <= tol), float((np.abs(got - ref) / tol).max())
        assert np.all(got[mass == 0] == 0)


@pytest.mark.parametrize("q4", [False, True], ids=["bf16", "q4"])
@pytest.mark.parametrize("case", DECODE_CASES, ids=decode_ids)
def test_decode_matches_the_definition(tsd, case, q4):
    c = DecodeCase(case, q4)
    c.check(tsd, c.run(tsd))
    assert tsd.attn_get_device_status() == tsd.ATTN_OK


@pytest.mark.parametrize("q4", [False, True], ids=["bf16", "q4"])
def test_decode_with_peaked_and_with_flat_weights(tsd, q4):
    """A scale that leaves one row almost all the weight, and one that leaves all rows the same."""
    c = DecodeCase((2, 8, 2, 2, 64, 16, [300, 77], None, True), q4, seed=9)
    for scale in (3.0, 1e-6):
        c.check(tsd, c.run(tsd, scale=scale), scale=float(np.float32(scale)))


@pytest.mark.parametrize("d", [64, 128])
def test_decode_queries_of_any_size(tsd, d):
    """Query rows from 2^-60 to 2^60 in one call (a 4-bit cache's products are formed in f16)."""
    c = DecodeCase((1, 8, 2, 1, d, 16, [130], None, True), True, seed=3)
    factor = 2.0 ** np.array([-60, -30, -8, 0, 1, 8, 30, 60])
    q = c.q * factor[None, :, None, None]
    for i, f in enumerate(factor):
        scale = float(np.float32(0.1 / f))
        out = c.run(tsd, q=to_dev_bf16(synthetic.f32_to_bf16_bits(q.astype(np.float32))), scale=scale)
        ref, mass, size = pu.decode(q[:, i:i + 1], [c.k_rows[0][i // 4][None]], [c.v_rows[0][i // 4][None]],
                                    [130], [1], True, scale)
        c.torch.cuda.synchronize()
        got = to_host_f64(out)[:, i:i + 1]
        assert np.all(np.abs(got - ref) <= pu.decode_tolerance(ref, mass, size, 130, d))


@pytest.mark.parametrize("q4", [False, True], ids=["bf16", "q4"])
@pytest.mark.parametrize("case", [
    (2, 8, 4, 4, 64, 16, [37, 90], [4, 2], True),
    (2, 8, 4, 8, 128, 16, [37, 90], [8, 5], True),
    (2, 8, 4, 8, 64, 16, [37, 1500], [8, 5], True),                        # 16 query rows to a tile
    (2, 8, 4, 8, 128, 16, [37, 1500], [7, 8], True),
    (80, 14, 2, 4, 64, 16, [9 + b for b in range(80)], [1 + b % 4 for b in range(80)], True),   # 32
    (80, 14, 2, 4, 128, 16, [9 + b for b in range(80)], [1 + b % 4 for b in range(80)], True),
], ids=decode_ids)
def test_rows_that_a_query_does_not_see_do_not_reach_it(tsd, q4, case):
    """Infinities and NaN in a later token's key and value: earlier tokens' outputs are as
    without them; the token that sees them has no finite output to compare."""
    new = case[7]
    c = DecodeCase(case, q4, seed=4)
    pools = [p.clone() for p in c.pools]
    for b, L in enumerate(case[6]):
        at, slot = int(c.table[b, (L - 1) // 16]), (L - 1) % 16
        if q4:
            pools[1][at, :, slot] = 0x7f
            pools[3][at, :, slot] = 0x7f
        else:
            pools[0][at, :, slot, 3] = float("nan")
            pools[1][at, :, slot, 5] = float("inf")
            pools[1][at, :, slot, 6] = float("nan")
    got = to_host_f64(c.run(tsd, pools=pools))
    clean = to_host_f64(c.run(tsd))
    for b in range(case[0]):
        m = new[b]
        assert np.array_equal(got[b, :, :m - 1], clean[b, :, :m - 1])
        assert not np.any(np.isfinite(got[b, :, m - 1]).all(-1))
        assert np.all(got[b, :, m:] == 0)


@pytest.mark.parametrize("q4", [False, True], ids=["bf16", "q4"])
def test_decode_leaves_out_rows_without_a_page(tsd, q4):
    """Bad page indices: reported, and the rows take no part."""
    case = (2, 4, 2, 1, 64, 16, [70, 40], None, True)
    c = DecodeCase(case, q4, seed=6)
    table = c.table.copy()
    table[0, 2], table[1, 0] = c.n_pages, -5
    out = c.run(tsd, table=to_dev_i32(table))
    assert tsd.attn_get_device_status() == tsd.ATTN_ERR_DEVICE_INDEX
    keep = [np.r_[0:32, 48:70], np.r_[16:40]]
    c.case = case[:6] + ([54, 24],) + case[7:]
    c.check(tsd, out, [k[:, i] for k, i in zip(c.k_rows, keep)], [v[:, i] for v, i in zip(c.v_rows, keep)])


@pytest.mark.parametrize("lens", [[200, 200, 150], [1500, 1500, 1490]], ids=["whole", "split"])
@pytest.mark.parametrize("q4", [False, True], ids=["bf16", "q4"])
def test_sequences_that_share_pages(tsd, q4, lens):
    """A common beginning held once: the same page in several tables, and twice in one."""
    c = DecodeCase((3, 8, 2, 2, 64, 16, lens, None, True), q4, seed=31)
    table = c.table.copy()
    table[1, :-4], table[2, :8] = table[0, :-4], table[0, 0]
    c.k_rows, c.v_rows = list(c.k_rows), list(c.v_rows)
    for rows in (c.k_rows, c.v_rows):
        last = (lens[1] + 15) // 16
        shared = min(table.shape[1] - 4, last) * 16
        rows[1] = np.concatenate([rows[0][:, :shared], rows[1][:, shared:]], 1)
        rows[2] = np.concatenate([np.tile(rows[0][:, :16], (1, 8, 1)), rows[2][:, 128:]], 1)
    c.check(tsd, c.run(tsd, table=to_dev_i32(table)))
    assert tsd.attn_get_device_status() == tsd.ATTN_OK


@pytest.mark.parametrize("q4", [False, True], ids=["bf16", "q4"])
def test_decode_clamps_lengths(tsd, q4):
    """Lengths past the page table count as its rows; no lengths: all of them; negative: none."""
    case = (3, 4, 2, 2, 64, 16, [48, 48, 48], None, True)
    c = DecodeCase(case, q4, seed=7)
    c.table, full = np.ascontiguousarray(c.table[:, :3]), None
    c.dev["table"] = to_dev_i32(c.table)
    for lens in (None, to_dev_i32([48, 1000, 2 ** 31 - 1])):
        c.check(tsd, c.run(tsd, lens=lens))
    got = to_host_f64(c.run(tsd, lens=to_dev_i32([-1, 48, -(2 ** 31)]), new=to_dev_i32([9, 2, -4])))
    assert np.all(got[[0, 2]] == 0) and np.all(np.isfinite(got[1]))


@pytest.mark.parametrize("q4", [False, True], ids=["bf16", "q4"])
def test_decode_repeats_to_the_bit_and_on_other_streams(tsd, q4):
    """The same call again, with a workspace full of ones, on a stream of its own, two at once."""
    import torch
    c = DecodeCase((3, 8, 2, 1, 128, 16, [3000, 10, 900], None, True), q4, seed=8)
    first = c.run(tsd)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs, kept = [], []
    for i in range(6):
        with torch.cuda.stream(streams[i % 2]):
            ws = torch.full((c.workspace.numel(),), 255, dtype=torch.uint8, device="cuda")
            outs.append(c.run(tsd, workspace=ws, stream=None if i < 3 else streams[i % 2]))
            kept.append(ws)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o.view(torch.int16), first.view(torch.int16))


@pytest.mark.parametrize("q4", [False, True], ids=["bf16", "q4"])
def test_pools_past_32_bit_offsets(tsd, q4):
    """Pages whose elements lie past 2^32 (bf16) and 2^31 (4-bit codes) from the pool's start:
    the decoding step over them equals that over a small pool, and the append reaches them."""
    import torch
    h_kv, d, page, n_pages = 8, 128, 256, 20000 if q4 else 17000
    small = DecodeCase((2, 16, h_kv, 1, d, page, [700, 300], None, True), q4, seed=31)
    want = small.run(tsd)
    torch.cuda.synchronize()
    places = [n_pages - 1, 3, n_pages - 2, n_pages // 2 + 1, 0, n_pages - 7, n_pages - 9]
    used = sorted(set(int(x) for x in small.table.ravel() if x >= 0))
    move = {old: places[i] for i, old in enumerate(used)}
    big = []
    for pool in small.pools:
        t = torch.empty((n_pages,) + tuple(pool.shape[1:]), dtype=pool.dtype, device="cuda")
        for old, new in move.items():
            t[new].copy_(pool[old])
        big.append(t)
    assert big[0].numel() > (1 << 31 if q4 else 1 << 32)
    table = np.vectorize(lambda x: move.get(int(x), -1))(small.table).astype(np.int32)
    small.n_pages = n_pages
    got = small.run(tsd, pools=big, table=to_dev_i32(table))
    torch.cuda.synchronize()
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    # three new tokens on the last page
    x = torch.randn(1, 3, 3 * h_kv, d, device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    x = x.to(torch.bfloat16)
    tab, lens = to_dev_i32([[n_pages - 1]]), to_dev_i32([200])
    little = [torch.zeros((1,) + tuple(p.shape[1:]), dtype=p.dtype, device="cuda") for p in big]
    st = (9 * h_kv * d, d, 3 * h_kv * d)
    for pools, table, n in ((little, to_dev_i32([[0]]), 1), (big, tab, n_pages)):
        args = (x, *st, x[:, :, h_kv:], x[:, :, 2 * h_kv:], *st, torch.empty(1, h_kv, 3, d, dtype=x.dtype, device="cuda"),
                None, *pools)
        rest = (table, lens, None, None, 0, 0, 0, 1, h_kv, h_kv, 3, d, n, page, 1)
        if q4:
            tsd.attn_cache_append_q4(*args, 0.01, 0.01, *rest)
        else:
            tsd.attn_cache_append(*args, *rest)
    torch.cuda.synchronize()
    assert tsd.attn_get_device_status() == tsd.ATTN_OK
    for a, b in zip(little, big):
        assert torch.equal(a[0, :, 197:200].view(torch.uint8), b[n_pages - 1, :, 197:200].view(torch.uint8))


# ------------------------------------------------------------------ together

def together(tsd, q4, steps=6, n0=45):
    """A prompt through the projections, the append and causal attention, then one token at a
    time through the append and the paged decoding step, captured once and replayed."""
    import torch
    B, h, d, dm, page = 3, 4, 64, 128, 16
    rng = np.random.default_rng(11)
    total = n0 + steps
    x_bits, _ = bf16(rng, B, total, dm)
    w_bits = [bf16(rng, dm, h * d)[0] for _ in range(3)]
    x, w = to_dev_bf16(x_bits), [to_dev_bf16(b) for b in w_bits]
    w = [t * 0.125 for t in w]
    rope_np = pu.rope_table(total, d)
    rope = dev(rope_np)
    max_pages = -(-total // page)
    table_np = rng.permutation(B * max_pages).astype(np.int32).reshape(B, max_pages)
    table, n_pages = to_dev_i32(table_np), B * max_pages
    shape = (n_pages, h, page)
    factors = (0.01, 0.01)
    if q4:
        pools = [torch.zeros(shape + (n,), dtype=torch.uint8, device="cuda")
                 for n in (d // 2, d // 16, d // 2, d // 16)]
        append = lambda *a: tsd.attn_cache_append_q4(*a[:11], *pools, *factors, *a[11:])
        decode = lambda q, *a: tsd.attn_decode_paged_q4(q, *pools, *factors, *a)
    else:
        pools = [torch.zeros(shape + (d,), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        append = lambda *a: tsd.attn_cache_append(*a[:11], *pools, *a[11:])
        decode = lambda q, *a: tsd.attn_decode_paged(q, *pools, *a)
    new = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")

    def project_and_append(rows, n, lens):
        q, k, v = (new(B, n, h * d) for _ in range(3))
        tsd.mha_project_qkv(rows, rows, *w, q, k, v, B, n, n, dm, h, d, d)
        q_out, k_out = new(B, h, n, d), new(B, h, n, d)
        st = (n * h * d, d, h * d)
        append(q, *st, k, v, *st, q_out, k_out, table, lens, None, rope, total, d, 1, B, h, h, n, d,
               n_pages, page, max_pages)
        return q_out, k_out, q, k, v

    lens = to_dev_i32([n0] * B)
    q_out, k_out, q, k, v = project_and_append(x[:, :n0].contiguous(), n0, lens)
    prompt = new(B, h, n0, d)
    tsd.attn_forward_strided(q_out, h * n0 * d, n0 * d, d, k_out, h * n0 * d, n0 * d, d, v, n0 * h * d,
                             d, h * d, prompt, h * n0 * d, n0 * d, d, B, h, n0, n0, d, d,
                             tsd.ATTN_MASK_CAUSAL)
    qs, ks, vs = [[t.clone()] for t in (q, k, v)]
    wsb = tsd.attn_decode_paged_workspace_bytes(B, h, h, 1, d, page, max_pages)
    ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
    token, out = new(B, 1, dm), new(B, h, 1, d)

    def step():
        lens.add_(1)
        got = project_and_append(token, 1, lens)
        decode(got[0], out, table, lens, None, B, h, h, 1, d, n_pages, page, max_pages,
               tsd.ATTN_MASK_CAUSAL, 0.0, ws, wsb)
        return got
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # once before the capture
        token.copy_(x[:, n0:n0 + 1])
        step()
        lens.sub_(1)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    outs = []
    for i in range(steps):
        token.copy_(x[:, n0 + i:n0 + i + 1])
        graph.replay()
        outs.append(out.clone())
        for a, b in zip((qs, ks, vs), kept[2:]):
            a.append(b.clone())
    torch.cuda.synchronize()
    assert tsd.attn_get_device_status() == tsd.ATTN_OK
    assert lens.tolist() == [total] * B
    return dict(prompt=to_host_f64(prompt), steps=to_host_f64(torch.cat(outs, 2)), rope=rope_np,
                q=to_host_f64(torch.cat(qs, 1)), k=to_host_f64(torch.cat(ks, 1)),
                v=to_host_f64(torch.cat(vs, 1)), pools=pools, table=table_np, factors=factors,
                sizes=(B, h, d, n0, total, page))


@pytest.mark.parametrize("q4", [False, True], ids=["bf16", "q4"])
def test_prompt_and_decoding_steps_together(tsd, q4):
    r = together(tsd, q4)
    B, h, d, n0, total, page = r["sizes"]
    heads = lambda x: x.reshape(B, total, h, d).swapaxes(1, 2)
    q, k, v = (heads(r[n]) for n in "qkv")
    turn = lambda x: np.stack([pu.rotate(x[:, :, p], p, r["rope"], 1, d) for p in range(total)], 2)
    q, k = turn(q), turn(k)
    rounded = lambda x: synthetic.bf16_bits_to_f64(synthetic.f32_to_bf16_bits(x.astype(np.float32)))
    q, k = rounded(q), rounded(k)
    # the prompt: attn_forward on the rotated queries and keys
    causal = np.tril(np.ones((n0, n0), dtype=bool))
    x = np.where(causal, q[:, :, :n0] @ k[:, :, :n0].swapaxes(2, 3) / np.sqrt(d), -np.inf)
    p = np.exp(x - x.max(-1, keepdims=True))
    want = p / p.sum(-1, keepdims=True) @ v[:, :, :n0]
    # attn_forward rounds its weights to bf16 (2^-8) and its output likewise; the rotated bf16
    # queries and keys may be one rounding (2^-8) off the 64-bit ones here and there: twice that
    # of sum |q k| in the exponent
    size = np.abs(q[:, :, :n0]) @ np.abs(k[:, :, :n0]).swapaxes(2, 3) / np.sqrt(d)
    tol = (2.0 ** -7 + 2 * 2.0 ** -16 * size.max()) * (p / p.sum(-1, keepdims=True) @ np.abs(v[:, :, :n0])) + 1e-6
    assert np.all(np.abs(r["prompt"] - want) <= tol + 2.0 ** -8 * np.abs(want))
    # the steps, over what the cache holds
    if q4:
        pools = [t.cpu().numpy() for t in r["pools"]]
        kp, vp = (pu.dequantise(pools[2 * i], pools[2 * i + 1], r["factors"][i]) for i in (0, 1))
    else:
        kp, vp = (to_host_f64(t) for t in r["pools"])
    kr = [pu.gather(kp, r["table"][b], total, page) for b in range(B)]
    vr = [pu.gather(vp, r["table"][b], total, page) for b in range(B)]
    steps = total - n0
    for i in range(steps):
        n = n0 + i + 1
        one = q[:, :, n - 1:n]
        ref, mass, size = pu.decode(one, [a[:, :n] for a in kr], [a[:, :n] for a in vr], [n] * B, [1] * B,
                                    True, 1 / np.sqrt(d))
        # the query's bf16 rounding may fall the other way where it is near halfway: 2^-8 of
        # single features, 2^-16 of the logit's sum at most here
        tol = pu.decode_tolerance(ref, mass, size, n, d) + 2 * 2.0 ** -12 * size[..., None] * mass
        assert np.all(np.abs(r["steps"][:, :, i:i + 1] - ref) <= tol)
    # and what the cache holds is the rotated keys and the values
    for b in range(B):
        if not q4:
            assert np.array_equal(vr[b], v[b])
            assert np.all(np.abs(kr[b] - k[b]) <= 2.0 ** -7 * np.abs(k[b]) + 1e-6)
        else:
            for got, want in ((kr[b], k[b]), (vr[b], v[b])):
                top = np.abs(want).reshape(h, total, -1, 16).max(-1).repeat(16, -1)
                # half a step of the codes is a sixth of the largest at most, a scale is off by 2^-4
                assert np.all(np.abs(got - want) <= top * (1 / 6 + 1 / 16 + 2.0 ** -8))


@pytest.mark.parametrize("q4", [False, True], ids=["bf16", "q4"])
def test_graphs_that_share_a_workspace(tsd, q4):
    """Two captured decoding steps over one workspace, replayed in turn on one stream."""
    import torch
    cs = [DecodeCase((2, 8, 2, 1, 64, 16, lens, None, True), q4, seed=s)
          for s, lens in ((20, [700, 33]), (21, [64, 1200]))]
    wants = [c.run(tsd) for c in cs]
    torch.cuda.synchronize()
    size = max(c.workspace.numel() for c in cs)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    outs = [torch.zeros_like(w) for w in wants]
    graphs = []
    for c, o in zip(cs, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run(tsd, workspace=ws, out=o)
        graphs.append(g)
    for _ in range(20):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, wants):
        assert torch.equal(o.view(torch.int16), w.view(torch.int16))


def test_decode_equals_the_contiguous_cache(tsd):
    """attn_decode on the same rows, one query head to a key head: the two agree within the
    roundings of their outputs and weights."""
    import torch
    B, h, n_q, d, L, page = 2, 4, 3, 64, 320, 16
    c = DecodeCase((B, h, h, n_q, d, page, [L, 150], None, True), False, seed=12)
    flat = [torch.zeros(B, h, L, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for b, n in enumerate((L, 150)):
        for i, rows in enumerate((c.k_rows, c.v_rows)):
            flat[i][b, :, :n] = dev(rows[b]).to(torch.bfloat16)
    out = torch.empty(B, h, n_q, d, dtype=torch.bfloat16, device="cuda")
    wsb = tsd.attn_decode_workspace_bytes(B, h, n_q, L, d)
    ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
    tsd.attn_decode(c.dev["q"], *flat, out, B, h, n_q, L, d, d, c.dev["lens"], 0.0, ws, wsb)
    c.check(tsd, out)
    c.check(tsd, c.run(tsd))
