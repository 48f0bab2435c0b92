"""GPU tests of the paged cache's kernels in the variants that their launch
rules choose by size: the append of many tokens and of many heads, the
decoding step over long ranges, wide and narrow query tiles, and short
sequences under a wide page table. The cases are checked against the 64-bit
definitions of paged_util."""
import numpy as np
import pytest

import synthetic

import paged_util as pu
from gpu_util import to_dev_bf16, to_dev_i32, to_host_f64
from test_paged_gpu import (DecodeCase, bf16, check_groups, decode_ids, dev, rotation_tolerance,
                            tsd)  # noqa: F401 (tsd: a fixture)

pytestmark = pytest.mark.gpu

SENTINEL = 0x5a


# ------------------------------------------------------------------ append

def rotate_rows(x, positions, rope, kind, dim):
    """x [m, heads, d] in 64 bits, row i at positions[i]."""
    y = np.array(x)
    if kind == 0:
        return y
    c, s = (a[positions][:, None].astype(np.float64) for a in (rope[:, :dim // 2], rope[:, dim // 2:]))
    i, j = (slice(0, dim // 2), slice(dim // 2, dim)) if kind == pu.HALVES else \
        (slice(0, dim, 2), slice(1, dim, 2))
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., j] * c + x[..., i] * s
    return y


def check_append(tsd, case, q4, in_place=False, k_out=True, bad_pages=(), rope_rows=None):
    """One append on seeded inputs. in_place: queries [B, h, n, d] are their own output. bad_pages:
    (sequence, page of it, index). rope_rows: rows of the rotation's table, if not enough."""
    import torch
    B, n, h, h_kv, d, page, kind, dim, past, new = case
    rng = np.random.default_rng(sum(case[:8]) + 77)
    factors = (0.0113, 0.0071)
    new = [n] * B if new is None else new
    lens = [p + m for p, m in zip(past, new)]
    x_bits, x = bf16(rng, B, n, h + 2 * h_kv, d)
    table, n_pages = pu.page_table(rng, lens, page)
    for b, i, value in bad_pages:
        table[b, i] = value
    known = max(lens) + 1 if rope_rows is None else rope_rows
    rope = pu.rope_table(known, dim) if kind else None
    shape = (n_pages, h_kv, page)
    widths = (d // 2, d // 16, d // 2, d // 16) if q4 else (2 * d, 2 * d)
    pools = [torch.full(shape + (w,), SENTINEL, dtype=torch.uint8, device="cuda") for w in widths]
    xd = to_dev_bf16(x_bits)
    strides = (n * (h + 2 * h_kv) * d, d, (h + 2 * h_kv) * d)
    if in_place:
        q = to_dev_bf16(x_bits[:, :, :h].swapaxes(1, 2))
        q_strides, q_out = (h * n * d, n * d, d), q
    else:
        q, q_strides = xd, strides
        q_out = torch.full((B, h, n, 2 * d), SENTINEL, dtype=torch.uint8, device="cuda")
    ko = torch.full((B, h_kv, n, 2 * d), SENTINEL, dtype=torch.uint8, device="cuda") if k_out else None
    args = (q, *q_strides, xd[:, :, h:], xd[:, :, h + h_kv:], *strides, q_out, ko, *pools)
    rest = (to_dev_i32(table), to_dev_i32(lens), to_dev_i32(new), None if rope is None else dev(rope),
            0 if rope is None else known, dim, kind, B, h, h_kv, n, d, n_pages, page, table.shape[1])
    if q4:
        tsd.attn_cache_append_q4(*args, *factors, *rest)
    else:
        tsd.attn_cache_append(*args, *rest)
    torch.cuda.synchronize()
    status = tsd.attn_get_device_status()

    bits = lambda t: t.cpu().view(torch.uint8).reshape(t.shape[:-1] + (-1,)).numpy()
    f64 = lambda raw: synthetic.bf16_bits_to_f64(np.ascontiguousarray(raw).view(np.uint16))
    raw = [p.cpu().numpy() for p in pools]
    q_raw, k_raw = bits(q_out), None if ko is None else bits(ko)
    q_was = x_bits[:, :, :h].swapaxes(1, 2).copy().view(np.uint8) if in_place else SENTINEL
    q_was = np.broadcast_to(q_was, q_raw.shape)
    untouched = np.ones((n_pages, page), dtype=bool)
    left_out = False
    for b in range(B):
        t = np.arange(new[b])
        p = lens[b] - new[b] + t
        at = table[b, p // page]
        there = (at >= 0) & (at < n_pages) & ((p < known) if kind else True)
        left_out |= not there.all()
        skipped = np.r_[t[~there], np.arange(new[b], n)]
        assert np.array_equal(q_raw[b][:, skipped], q_was[b][:, skipped])
        if ko is not None:
            assert np.all(k_raw[b][:, skipped] == SENTINEL)
        t, p, at = t[there], p[there], at[there]
        if t.size == 0:
            continue
        slot = p % page
        untouched[at, slot] = False
        xs = x[b, t]
        turned = rotate_rows(xs[:, :h + h_kv], p, rope, kind, dim)
        top = np.abs(xs).max((1, 2), keepdims=True)
        tol = rotation_tolerance(turned, 1.0, 0) + (6 * 2.0 ** -24 * top if dim else 0)
        got_q = f64(q_raw[b][:, t].swapaxes(0, 1))
        assert np.all(np.abs(got_q - turned[:, :h]) <= tol[:, :h])
        if ko is not None:
            got_k = f64(k_raw[b][:, t].swapaxes(0, 1))
            assert np.all(np.abs(got_k - turned[:, h:]) <= tol[:, h:])
        if q4:
            error = 6 * 2.0 ** -24 * top if dim else 0.0
            check_groups(raw[0][at, :, slot], raw[1][at, :, slot], turned[:, h:], error, factors[0])
            check_groups(raw[2][at, :, slot], raw[3][at, :, slot], xs[:, h + h_kv:], 0.0, factors[1])
        else:
            assert np.all(np.abs(f64(raw[0][at, :, slot]) - turned[:, h:]) <= tol[:, h:])
            assert np.array_equal(f64(raw[1][at, :, slot]), xs[:, h + h_kv:])
    for pool in raw:
        assert np.all(pool.swapaxes(1, 2)[untouched] == SENTINEL)
    assert status == (tsd.ATTN_ERR_DEVICE_INDEX if left_out else tsd.ATTN_OK)


MANY_TOKENS = [
    # above 1520 tokens: two, three or four tokens to a block and three heads to a thread; the
    # first positions put pages' ends inside a block's tokens
    (2, 800, 6, 3, 64, 16, 1, 64, [5, 0], [800, 777]),
    (2, 811, 5, 5, 128, 16, 2, 128, [1, 30], [811, 640]),
    (3, 1100, 4, 2, 64, 32, 2, 32, [7, 31, 0], [1100, 3, 1099]),
    (3, 1101, 8, 1, 128, 64, 1, 64, [62, 3, 100], [1101, 1000, 0]),
    (4, 1203, 2, 2, 64, 16, 1, 64, [3, 14, 0, 9], [1203, 1, 1200, 703]),
    (4, 1203, 3, 1, 128, 128, 1, 96, [126, 2, 255, 0], None),
    (1600, 1, 4, 2, 128, 16, 1, 128, [(7 * b) % 50 for b in range(1600)], None),  # a token each
    (700, 7, 2, 1, 64, 16, 2, 64, [(5 * b) % 33 for b in range(700)], [b % 8 for b in range(700)]),
    (2, 800, 4, 4, 128, 16, 0, 0, [15, 1], None),
]
MANY_HEADS = [
    # a block's threads take a token's heads in two rounds: one head to a thread, then three
    (3, 2, 64, 16, 128, 16, 1, 128, [0, 15, 30], [2, 1, 2]),
    (2, 3, 128, 8, 64, 16, 2, 64, [14, 0], None),
    (16, 100, 88, 8, 128, 16, 1, 128, [b for b in range(16)], [100 if b == 3 else b for b in range(16)]),
    (16, 100, 184, 8, 64, 16, 2, 64, [b for b in range(16)], [100 if b == 5 else b for b in range(16)]),
]
append_ids = lambda c: "B{}n{}h{}kv{}d{}p{}r{}x{}".format(*c[:8])


@pytest.mark.parametrize("q4", [False, True], ids=["bf16", "q4"])
@pytest.mark.parametrize("case", MANY_TOKENS + MANY_HEADS, ids=append_ids)
def test_append_of_many_tokens_and_of_many_heads(tsd, case, q4):
    check_append(tsd, case, q4, in_place=case[1] % 2 == 1, k_out=case[2] != 5)


@pytest.mark.parametrize("q4", [False, True], ids=["bf16", "q4"])
@pytest.mark.parametrize("d", [64, 128])
def test_append_of_many_tokens_without_a_place(tsd, d, q4):
    """Bad pages between good ones, inside a block's tokens, and positions past the rotation's table."""
    case = (2, 1600, 4, 2, d, 16, 1, 64, [9, 2], [1600, 1501])
    check_append(tsd, case, q4, bad_pages=[(0, 0, -3), (0, 7, 1 << 30), (1, 50, -1), (1, 51, 100000)])
    check_append(tsd, case, q4, in_place=True, rope_rows=1202)


# ------------------------------------------------------------------ decode

def repeat(c, times):
    """The case's sequences `times` over on the same pages, every one with queries of its own."""
    B, *mid, lens, new, causal = c.case
    c.case = (B * times, *mid, list(lens) * times, None if new is None else list(new) * times, causal)
    h, h_kv, n_q, d, page = mid
    c.q_bits, c.q = bf16(np.random.default_rng(5), B * times, h, n_q, d)
    c.new = list(c.new) * times
    c.table = np.tile(c.table, (times, 1))
    c.k_rows, c.v_rows = list(c.k_rows) * times, list(c.v_rows) * times
    c.dev = dict(q=to_dev_bf16(c.q_bits), table=to_dev_i32(c.table), lens=to_dev_i32(c.case[6]),
                 new=None if new is None else to_dev_i32(c.case[7]))
    return c


def check_repeated(tsd, c, out, bases):
    """DecodeCase.check for a case of `bases` sequences repeated: all that share their rows at a time."""
    B, h, h_kv, n_q, d, page, lens, new, causal = c.case
    c.torch.cuda.synchronize()
    got, scale = to_host_f64(out), 1 / np.sqrt(d)
    assert np.all(np.isfinite(got))
    for b in range(bases):
        for t in range(n_q):
            if t >= c.new[b]:
                assert np.all(got[b::bases, :, t] == 0)
                continue
            n = lens[b] - c.new[b] + t + 1 if causal else lens[b]
            for head in range(h_kv):
                heads = slice(head * (h // h_kv), (head + 1) * (h // h_kv))
                q, k, v = c.q[b::bases, heads, t], c.k_rows[b][head, :n], c.v_rows[b][head, :n]
                w = q @ k.T * scale
                w = np.exp(w - w.max(-1, keepdims=True))
                w /= w.sum(-1, keepdims=True)
                ref, mass = w @ v, w @ np.abs(v) + 2.0 ** -25 * np.abs(v).sum(0)
                size = (np.abs(q) @ np.abs(k).T).max(-1) * scale
                tol = pu.decode_tolerance(ref, mass, size, max(lens), d)
                assert np.all(np.abs(got[b::bases, heads, t] - ref) <= tol)


def widen(c, max_pages):
    """The same sequences under a page table of `max_pages` entries each."""
    wide = np.full((c.table.shape[0], max_pages), -1, dtype=np.int32)
    wide[:, :c.table.shape[1]] = c.table
    c.table, c.dev["table"] = wide, to_dev_i32(wide)
    return c


LONG = [
    # as many pairs as make a block take sequences whole, of more than three times 2048 rows (a
    # warp looks up the places of 32 tiles, 2048 of the block's rows, at a time)
    ((3, 2, 2, 1, 64, 64, [7003, 6200, 2100], None, True), 240),
    ((3, 4, 2, 1, 128, 64, [6777, 9000, 4159], None, True), 200),
    ((2, 12, 2, 2, 64, 128, [6900, 6333], [1, 2], True), 240),           # 16 query rows to a tile
    ((2, 10, 1, 2, 128, 64, [6500, 4100], None, False), 330),            # 32
]


@pytest.mark.parametrize("q4", [False, True], ids=["bf16", "q4"])
@pytest.mark.parametrize("case,times", LONG, ids=["d64", "d128", "tile16", "tile32"])
def test_decode_over_long_ranges(tsd, case, times, q4):
    c = repeat(DecodeCase(case, q4, seed=70), times)
    check_repeated(tsd, c, c.run(tsd), case[0])
    assert tsd.attn_get_device_status() == tsd.ATTN_OK


@pytest.mark.parametrize("q4", [False, True], ids=["bf16", "q4"])
@pytest.mark.parametrize("d", [64, 128])
def test_bad_pages_far_into_a_range(tsd, d, q4):
    """Pages that are no pages in the second, third and fourth look-up of a warp's places."""
    case = (2, 2, 2, 1, d, 64, [7003, 8200], None, True)
    c = DecodeCase(case, q4, seed=71)
    gone = [{33, 40, 41, 66, 99, 100}, {0, 64, 65, 97, 127}]
    for b, pages in enumerate(gone):
        for i in pages:
            c.table[b, i] = -1 if i % 2 else c.n_pages + i
    keep = [np.array([p for p in range(L) if p // 64 not in g]) for L, g in zip(case[6], gone)]
    c.k_rows, c.v_rows = ([r[:, k] for r, k in zip(rows, keep)] for rows in (c.k_rows, c.v_rows))
    c = repeat(c, 240)
    out = c.run(tsd)
    assert tsd.attn_get_device_status() == tsd.ATTN_ERR_DEVICE_INDEX
    c.case = c.case[:6] + ([len(k) for k in keep] * 240,) + c.case[7:]
    check_repeated(tsd, c, out, 2)


TILES = [
    (43, 28, 4, 4, 64, 16, [(411 * b) % 2500 for b in range(43)], [4 - b % 5 for b in range(43)], True),  # 32, split
    (43, 28, 4, 4, 128, 16, [(411 * b) % 2500 for b in range(43)], None, False),
    (50, 12, 4, 4, 128, 16, [(29 * b) % 500 for b in range(50)], [1 + b % 4 for b in range(50)], True),   # 16, whole
    (50, 12, 4, 4, 64, 16, [(29 * b) % 500 for b in range(50)], None, True),
    (25, 28, 4, 4, 128, 32, [(61 * b) % 900 for b in range(25)], None, True),      # two tiles of 16, whole
    (25, 28, 4, 4, 64, 16, [(61 * b) % 900 for b in range(25)], None, False),
    (30, 9, 3, 3, 128, 16, [(61 * b) % 900 for b in range(30)], None, True),       # two of 8, four warps, whole
    (30, 9, 3, 3, 64, 16, [(61 * b) % 900 for b in range(30)], [b % 4 for b in range(30)], True),
]


@pytest.mark.parametrize("q4", [False, True], ids=["bf16", "q4"])
@pytest.mark.parametrize("case", TILES, ids=decode_ids)
def test_decode_with_every_query_tile(tsd, case, q4):
    c = DecodeCase(case, q4, seed=72)
    c.check(tsd, c.run(tsd))
    assert tsd.attn_get_device_status() == tsd.ATTN_OK


IDLE = [
    # less than a unit of work to a block, empty and padded sequences among the others
    (12, 8, 2, 1, 64, 16, [0, 100, 0, 0, 700, 33, 0, 900, 1, 0, 0, 64], None, True),
    (12, 8, 2, 2, 128, 16, [0, 100, 0, 0, 700, 33, 0, 900, 1, 0, 0, 64], [2, 0, 1, 0, 2, 1, 0, 2, 2, 2, 0, 1], True),
    (5, 28, 4, 4, 128, 32, [0, 0, 300, 0, 5], None, False),
    (70, 4, 1, 1, 64, 16, [90 if b in (3, 40, 69) else 0 for b in range(70)], None, True),
    (70, 4, 1, 1, 128, 16, [64 if b == 33 else 0 for b in range(70)], None, True),
    (3, 2, 2, 1, 128, 16, [0, 0, 0], None, True),
    (40, 2, 2, 8, 64, 16, [50] * 40, [0] * 40, True),
    (24, 32, 8, 1, 128, 16, [100 + 33 * b for b in range(24)], None, True),        # none empty
]


@pytest.mark.parametrize("q4", [False, True], ids=["bf16", "q4"])
@pytest.mark.parametrize("case", IDLE, ids=decode_ids)
def test_short_and_empty_sequences_under_a_wide_page_table(tsd, case, q4):
    c = widen(DecodeCase(case, q4, seed=73), 32768 // case[5])
    c.check(tsd, c.run(tsd))
    assert tsd.attn_get_device_status() == tsd.ATTN_OK
