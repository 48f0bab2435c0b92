"""The calls that keep a paged cache's pages, against plain forms of their definitions: tables,
counts and lists have to be equal, contents the same bytes."""
import numpy as np
import pytest

import pages_util as pu
from gpu_util import to_dev_i32

pytestmark = pytest.mark.gpu

GUARD = 777  # what entries nobody writes hold


@pytest.fixture(scope="module")
def tsd():
    import torch
    from transformer_scaled_dot_gb300 import build as native_build
    native_build.build()
    import transformer_scaled_dot_gb300 as m
    m.library()
    torch.cuda.set_device(0)
    return m


def ints(t):
    return t.cpu().numpy()


def ones(n=1):
    return to_dev_i32(np.full(n, GUARD))


def workspace(tsd, B, n_pages):
    import torch
    n = tsd.attn_cache_pages_workspace_bytes(B, n_pages)
    return torch.full((n,), 0xa5, dtype=torch.uint8, device="cuda"), n


def reserve(tsd, table, counts, lens, new, n_new, page, stream=None):
    """Runs a reserve on device arrays; (copies, n_copies, n_missing) as they came back."""
    B, max_pages = table.shape
    copies, n_copies, n_missing = to_dev_i32(np.full((B, 3), GUARD)), ones(), ones()
    ws, n = workspace(tsd, B, len(counts))
    tsd.attn_cache_reserve(table, counts, lens, new, copies, n_copies, n_missing, B, n_new, len(counts), page, max_pages,
                           ws, n, stream=stream)
    return ints(copies), int(n_copies), int(n_missing)


def check_state(plain, table, counts):
    assert np.array_equal(ints(table), np.array(plain.table))
    assert np.array_equal(ints(counts), np.array(plain.counts))
    assert plain.counts == list(np.bincount([p for r in plain.table for p in r if p >= 0], minlength=len(plain.counts)))


SHAPES = [
    # rows, max_pages, n_pages, page size
    (1, 1, 1, 16), (1, 1, 3, 256), (2, 3, 5, 16), (5, 33, 100, 32), (37, 9, 300, 16), (64, 70, 2500, 64),
    (300, 17, 4097, 128), (513, 40, 9000, 16), (3, 1500, 40000, 16),
]


@pytest.mark.parametrize("seed", range(3))
@pytest.mark.parametrize("shape", SHAPES)
def test_fork(tsd, shape, seed):
    B, max_pages, n_pages, page = shape
    rng = np.random.default_rng(100 * seed + B)
    table, counts = pu.state(rng, B, max_pages, n_pages, page)
    parents = rng.integers(-1, B, B) if seed else np.arange(B)
    if seed == 2:
        parents = np.where(rng.random(B) < 0.5, np.arange(B), parents)
    lens = rng.integers(0, 1000, B)
    plain = pu.Pages(table, counts, page)
    plain.fork(parents)
    t, c, l = to_dev_i32(table), to_dev_i32(counts), to_dev_i32(lens)
    tsd.attn_cache_fork(t, l, c, to_dev_i32(parents), B, n_pages, max_pages)
    assert tsd.attn_get_device_status() == tsd.ATTN_OK
    check_state(plain, t, c)
    assert np.array_equal(ints(l), np.where(parents >= 0, lens[parents], 0))


def test_fork_bad_parents_and_entries(tsd):
    table = np.array([[0, 1, -1], [2, 9, -1], [3, -5, 4]])  # a page past the pool, a negative entry
    counts = np.array([1, 1, 1, 1, 1, 0])
    t, c, l = to_dev_i32(table), to_dev_i32(counts), to_dev_i32([5, 6, 7])
    tsd.attn_cache_fork(t, l, c, to_dev_i32([3, -2, 0]), 3, 6, 3)
    assert tsd.attn_get_device_status() == tsd.ATTN_ERR_DEVICE_INDEX
    assert ints(t).tolist() == [[0, 1, -1], [2, 9, -1], [0, 1, -1]]
    assert ints(c).tolist() == [2, 2, 1, 0, 0, 0] and ints(l).tolist() == [5, 6, 5]
    tsd.attn_cache_fork(t, None, c, to_dev_i32([1, 1, 2]), 3, 6, 3)
    assert tsd.attn_get_device_status() == tsd.ATTN_ERR_DEVICE_INDEX  # page 9
    assert ints(t).tolist() == [[2, 9, -1], [2, 9, -1], [0, 1, -1]] and ints(c).tolist() == [1, 1, 2, 0, 0, 0]
    assert tsd.attn_get_device_status() == tsd.ATTN_OK


@pytest.mark.parametrize("B,max_pages", [(4096, 5), (32768, 2)])
def test_fork_many_rows(tsd, B, max_pages):
    """So many rows that a block has fewer columns, down to one."""
    rng = np.random.default_rng(B)
    n_pages = B * max_pages
    table = rng.permutation(n_pages).reshape(B, max_pages)
    parents = rng.integers(0, B, B)
    t, c = to_dev_i32(table), to_dev_i32(np.ones(n_pages))
    tsd.attn_cache_fork(t, None, c, to_dev_i32(parents), B, n_pages, max_pages)
    assert np.array_equal(ints(t), table[parents])
    assert np.array_equal(ints(c), np.bincount(table[parents].ravel(), minlength=n_pages))


@pytest.mark.parametrize("keep", ["none", "some", "all"])
@pytest.mark.parametrize("shape", SHAPES)
def test_release(tsd, shape, keep):
    B, max_pages, n_pages, page = shape
    rng = np.random.default_rng(B + max_pages)
    table, counts = pu.state(rng, B, max_pages, n_pages, page)
    lens = np.zeros(B, int) if keep == "none" else rng.integers(-1, max_pages * page + 2, B)
    plain = pu.Pages(table, counts, page)
    if keep != "all":
        plain.release(lens)
    t, c = to_dev_i32(table), to_dev_i32(counts)
    given = {"none": None, "some": to_dev_i32(lens), "all": to_dev_i32(np.full(B, 2 ** 31 - 1))}[keep]
    tsd.attn_cache_release(t, c, given, B, n_pages, page, max_pages)
    assert tsd.attn_get_device_status() == tsd.ATTN_OK
    check_state(plain, t, c)


def test_release_entries_out_of_range(tsd):
    t, c = to_dev_i32([[0, 7, -3, 1]]), to_dev_i32([1, 1, 0])
    tsd.attn_cache_release(t, c, to_dev_i32([16]), 1, 3, 16, 4)
    assert tsd.attn_get_device_status() == tsd.ATTN_ERR_DEVICE_INDEX
    assert ints(t).tolist() == [[0, -1, -1, -1]] and ints(c).tolist() == [1, 0, 0]


def grow(rng, plain, most):
    """Lengths with 0 .. most new tokens, on what the rows hold or a little off it, and how many are new."""
    lens, new, room = [], [], len(plain.table[0]) * plain.page
    for row in plain.table:
        held = sum(p >= 0 for p in row) * plain.page
        m = int(rng.integers(0, most + 1))
        lens.append(int(np.clip(held - rng.integers(0, plain.page + 1) + m, m, room)))
        new.append(m)
    return lens, new


@pytest.mark.parametrize("most", [1, 3, 40, 700])
@pytest.mark.parametrize("shape", SHAPES)
def test_reserve(tsd, shape, most):
    """Growing rows, some of whose pages are shared: with all, some and none of the sharers writing."""
    B, max_pages, n_pages, page = shape
    for seed in range(4):
        rng = np.random.default_rng(1000 * seed + B + most)
        table, counts = pu.state(rng, B, max_pages, n_pages, page, share=0.5)
        if seed > 1:  # rows that continue others whole
            plain = pu.Pages(table, counts, page)
            plain.fork(rng.integers(0, B, B) // 4 * 4 % B)
            table, counts = np.array(plain.table), np.array(plain.counts)
        plain = pu.Pages(table, counts, page)
        lens, new = grow(rng, plain, most)
        if seed == 3:  # rows of one parent write at the same place
            lens, new = [max(lens)] * B, [min(most, max(lens))] * B
        copies, missing = plain.reserve(lens, new)
        t, c = to_dev_i32(table), to_dev_i32(counts)
        got, n_copies, n_missing = reserve(tsd, t, c, to_dev_i32(lens), to_dev_i32(new), most, page)
        assert tsd.attn_get_device_status() == tsd.ATTN_OK
        assert (n_copies, n_missing) == (len(copies), missing)
        assert got[:n_copies].tolist() == [list(x) for x in copies] and (got[n_copies:] == GUARD).all()
        check_state(plain, t, c)


def test_reserve_keeps_one_of_the_sharers(tsd):
    """Three rows share a page that all of them write: the first keeps it. A fourth name that does
    not write it: everybody leaves."""
    for others in (0, 1):
        table = [[0, 1, -1], [0, 1, -1], [0, 1, -1], [0, 1 if others else -1, -1]]
        counts = [4, 3 + others, 0, 0, 0, 0]
        t, c = to_dev_i32(table), to_dev_i32(counts)
        copies, n, missing = reserve(tsd, t, c, to_dev_i32([21, 21, 21, 16]), to_dev_i32([1, 1, 1, 0]), 1, 16)
        if not others:
            assert ints(t).tolist() == [[0, 1, -1], [0, 2, -1], [0, 3, -1], [0, -1, -1]] and ints(c).tolist() == [4, 1, 1, 1, 0, 0]
            assert n == 2 and copies[:2].tolist() == [[1, 2, 4], [1, 3, 4]]
        else:
            assert ints(t).tolist() == [[0, 2, -1], [0, 3, -1], [0, 4, -1], [0, 1, -1]] and ints(c).tolist() == [4, 1, 1, 1, 1, 0]
            assert n == 3 and copies[:3].tolist() == [[1, 2, 4], [1, 3, 4], [1, 4, 4]]
        assert missing == 0


def test_reserve_without_new_lens_and_ends_of_ranges(tsd):
    """new_lens None: n_new for every row; lengths of zero, below it, negative, past the table."""
    table, counts = np.full((5, 4), -1), np.zeros(40)
    t, c = to_dev_i32(table), to_dev_i32(counts)
    lens = [0, 3, -4, 17, 64]
    copies, n, missing = reserve(tsd, t, c, to_dev_i32(lens), None, 5, 16)
    assert tsd.attn_get_device_status() == tsd.ATTN_OK and (n, missing) == (0, 0)
    # rows 3 and 4: the pages of positions 12 .. 16 and 59 .. 63
    assert ints(t).tolist() == [[-1] * 4, [0, -1, -1, -1], [-1] * 4, [1, 2, -1, -1], [-1, -1, -1, 3]]
    assert ints(c)[:5].tolist() == [1, 1, 1, 1, 0]
    reserve(tsd, t, c, to_dev_i32([0, 0, 0, 0, 66]), None, 5, 16)
    assert tsd.attn_get_device_status() == tsd.ATTN_ERR_DEVICE_INDEX
    assert ints(t)[4].tolist() == [-1, -1, -1, 3] and ints(c)[:5].tolist() == [1, 1, 1, 1, 0]
    reserve(tsd, t, c, to_dev_i32([2 ** 31 - 1] * 5), to_dev_i32([2 ** 31 - 1] * 5), 2 ** 31 - 1, 16)
    assert tsd.attn_get_device_status() == tsd.ATTN_ERR_DEVICE_INDEX
    assert (ints(t) >= 0).all()


def test_reserve_replaces_entries_out_of_range(tsd):
    t, c = to_dev_i32([[5, -9]]), to_dev_i32([1, 0, 0])
    copies, n, missing = reserve(tsd, t, c, to_dev_i32([20]), to_dev_i32([10]), 10, 16)
    assert tsd.attn_get_device_status() == tsd.ATTN_ERR_DEVICE_INDEX and (n, missing) == (0, 0)
    assert ints(t).tolist() == [[1, 2]] and ints(c).tolist() == [1, 1, 1]


@pytest.mark.parametrize("shape", [(4, 5, 12, 16), (64, 20, 700, 32), (700, 6, 1500, 16)])
def test_reserve_short_of_pages_changes_nothing(tsd, shape):
    B, max_pages, n_pages, page = shape
    rng = np.random.default_rng(B)
    table, counts = pu.state(rng, B, max_pages - 2, n_pages, page, share=0.5)
    table = np.concatenate([table, np.full((B, 2), -1)], 1)
    plain = pu.Pages(table, counts, page)
    plain.fork(rng.integers(0, B, B) // 4 * 4 % B)
    for p in range(n_pages):  # all but one page, of some other table
        if plain.counts[p] == 0 and 0 in plain.counts[p + 1:]:
            plain.counts[p] = 1
    table, counts = np.array(plain.table), np.array(plain.counts)
    lens, new = grow(rng, plain, page)
    copies, missing = plain.reserve(lens, new)
    assert missing > 0
    t, c = to_dev_i32(table), to_dev_i32(counts)
    got, n, n_missing = reserve(tsd, t, c, to_dev_i32(lens), to_dev_i32(new), page, page)
    assert (n, n_missing) == (0, missing) and (got == GUARD).all()
    assert np.array_equal(ints(t), table) and np.array_equal(ints(c), counts)


@pytest.mark.parametrize("n_pages", [1 << 12, (1 << 12) + 1, 100003, 1 << 20])
def test_reserve_from_large_pools(tsd, n_pages):
    """One to eight blocks of a cluster, pages at the pool's very end, every free page taken."""
    rng = np.random.default_rng(n_pages)
    counts = np.ones(n_pages, np.int32)
    free = np.sort(rng.choice(n_pages - 1, 300, replace=False))
    counts[free] = 0
    counts[-1] = 0
    table = np.full((7, 60), -1)
    t, c = to_dev_i32(table), to_dev_i32(counts)
    lens = [43 * 16] * 7  # 301 pages
    _, n, missing = reserve(tsd, t, c, to_dev_i32(lens), to_dev_i32(lens), 43 * 16, 16)
    assert (n, missing) == (0, 0)
    want = table.copy()
    want[:, :43] = np.append(free, n_pages - 1).reshape(7, 43)
    assert np.array_equal(ints(t), want) and (ints(c) == 1).all()


@pytest.mark.parametrize("B", [20000, 65535])
def test_reserve_many_rows(tsd, B):
    """More rows than a cluster has threads, pages shared four by four."""
    table = np.repeat(np.arange((B + 3) // 4), 4)[:B, None]
    counts = np.concatenate([np.bincount(table[:, 0]), np.zeros(B, int)])
    plain = pu.Pages(table, counts, 16)
    copies, missing = plain.reserve([9] * B, [2] * B)
    t, c = to_dev_i32(table), to_dev_i32(counts)
    got, n, n_missing = reserve(tsd, t, c, to_dev_i32([9] * B), None, 2, 16)
    assert (n, n_missing) == (len(copies), 0)
    assert np.array_equal(got[:n], np.array(copies))
    check_state(plain, t, c)


@pytest.mark.parametrize("apart", [True, False])
@pytest.mark.parametrize("max_copies", [0, 3, 1 << 20])
@pytest.mark.parametrize("shape", SHAPES + [(2, 4, 1 << 18, 16)])
def test_compact(tsd, shape, max_copies, apart):
    B, max_pages, n_pages, page = shape
    rng = np.random.default_rng(B + n_pages)
    table, counts = pu.state(rng, B, max_pages, n_pages, page)
    plain = pu.Pages(table, counts, page)
    room = min(max_copies, n_pages)
    copies, used = plain.compact(room)
    t, c = to_dev_i32(table), to_dev_i32(counts)
    t_out = to_dev_i32(np.full_like(table, GUARD)) if apart else t
    c_out = to_dev_i32(np.full_like(counts, GUARD)) if apart else c
    out, n_copies, n_used = to_dev_i32(np.full((max(room, 1), 3), GUARD)), ones(), ones()
    ws, n = workspace(tsd, B, n_pages)
    tsd.attn_cache_compact(t, c, t_out, c_out, out, n_copies, n_used, B, n_pages, page, max_pages, room, ws, n)
    assert tsd.attn_get_device_status() == tsd.ATTN_OK
    assert int(n_copies) == len(copies) and int(n_used) == used
    assert ints(out)[:len(copies)].tolist() == [list(x) for x in copies] and (ints(out)[len(copies):] == GUARD).all()
    check_state(plain, t_out, c_out)
    if apart:
        assert np.array_equal(ints(t), table) and np.array_equal(ints(c), counts)
    if room >= n_pages:
        assert (ints(c_out)[:used] > 0).all() and (ints(c_out)[used:] == 0).all()


def test_compact_without_rows_and_entries_out_of_range(tsd):
    ws, n = workspace(tsd, 1, 4)
    copies, n_copies, n_used = to_dev_i32(np.full((4, 3), GUARD)), ones(), ones()
    c, t = to_dev_i32([0, 2, 0, 1]), to_dev_i32([[3, 8, -2, 1]])
    tsd.attn_cache_compact(t, c, t, c, copies, n_copies, n_used, 0, 4, 16, 4, 4, ws, n)
    assert ints(c).tolist() == [1, 2, 0, 0] and ints(t).tolist() == [[3, 8, -2, 1]]
    c = to_dev_i32([0, 2, 0, 1])
    tsd.attn_cache_compact(t, c, t, c, copies, n_copies, n_used, 1, 4, 16, 4, 4, ws, n)
    assert tsd.attn_get_device_status() == tsd.ATTN_ERR_DEVICE_INDEX
    assert ints(t).tolist() == [[0, 8, -2, 1]] and int(n_used) == 2 and ints(copies)[0].tolist() == [3, 0, 16]


# ------------------------------------------------------------------ contents

def pools(rng, q4, layers, n_pages, h_kv, page, d, gap=0):
    """Pools of random bytes, `gap` rows behind each layer's."""
    import torch
    rows = n_pages * h_kv * page + gap
    widths = (d // 2, d // 16, d // 2, d // 16) if q4 else (2 * d, 2 * d)
    return [torch.from_numpy(rng.integers(0, 256, (layers, rows, w), dtype=np.uint8)).cuda() for w in widths]


def copied(pool, copies, n_pages, h_kv, page):
    out = ints(pool).copy()
    rows = out[:, :n_pages * h_kv * page].reshape(len(out), n_pages, h_kv, page, -1)
    for src, dst, n in copies:
        rows[:, dst, :, :n] = rows[:, src, :, :n]
    return out


def run_copy(tsd, q4, x, *args, **kw):
    (tsd.attn_cache_copy_q4 if q4 else tsd.attn_cache_copy)(*x, *args, **kw)


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("layers,n_pages,h_kv,page,d,gap", [
    (1, 2, 1, 16, 64, 0), (1, 40, 3, 16, 128, 0), (3, 25, 5, 32, 64, 16), (2, 12, 8, 64, 128, 48), (2, 5, 7, 256, 128, 0),
    (6, 30, 8, 16, 64, 0), (1, 4, 33, 128, 64, 0),
])
def test_copy(tsd, q4, layers, n_pages, h_kv, page, d, gap):
    """Whole pages and parts of pages of every size, layers with a gap between them."""
    rng = np.random.default_rng(n_pages + h_kv)
    x = pools(rng, q4, layers, n_pages, h_kv, page, d, gap)
    order, n = rng.permutation(n_pages), n_pages // 2
    rows = [page, 0, 1, page - 1, *rng.integers(1, page + 1, n)][:n]
    copies = list(zip(order[:n].tolist(), order[n:2 * n].tolist(), rows))
    want = [copied(p, copies, n_pages, h_kv, page) for p in x]
    listed = to_dev_i32(np.array(copies + [(0, 0, 16)] * 3))
    layer_rows = n_pages * h_kv * page + gap
    run_copy(tsd, q4, x, listed, to_dev_i32([n]), n + 3, layers, layer_rows, h_kv, d, n_pages, page)
    assert tsd.attn_get_device_status() == tsd.ATTN_OK
    for p, w in zip(x, want):
        assert np.array_equal(ints(p), w)


@pytest.mark.parametrize("q4", [False, True])
def test_copy_lists(tsd, q4):
    """No count: all; counts past the list or negative; numbers out of range are left out."""
    rng = np.random.default_rng(1)
    sizes = (2, 2 * 3 * 16 * 4, 3, 64, 8, 16)  # layers, layer_rows (8 pages of 3 heads), h_kv, d, pages, page size
    for copies, count, status, done in (
            ([(0, 1, 16), (2, 3, 5)], None, "OK", 2), ([(0, 1, 16), (2, 3, 5)], 1, "OK", 1), ([(0, 1, 16)], 0, "OK", 0),
            ([(0, 1, 16)], -3, "OK", 0), ([(0, 1, 16)], 2, "ERR_DEVICE_INDEX", 1),
            ([(-1, 1, 16), (0, 8, 16), (0, 2, 17), (0, 3, -1), (8, 4, 3), (5, 6, 7)], None, "ERR_DEVICE_INDEX", None)):
        x = pools(rng, q4, 2, 8, 3, 16, 64)
        want = [copied(p, copies[:done] if done is not None else copies[-1:], 8, 3, 16) for p in x]
        run_copy(tsd, q4, x, to_dev_i32(np.array(copies)), None if count is None else to_dev_i32([count]), len(copies), *sizes)
        assert tsd.attn_get_device_status() == getattr(tsd, "ATTN_" + status)
        for p, w in zip(x, want):
            assert np.array_equal(ints(p), w)


@pytest.mark.parametrize("copy", [(0, 1, -1), (0, 1, -2 ** 31), (-1, 1, 0), (0, 8, 0), (0, 8, 16)])
@pytest.mark.parametrize("n", [1, 600])
def test_copy_lists_of_nothing_to_copy(tsd, copy, n):
    """A number out of range is reported where no copy of the list has a row, too."""
    rng = np.random.default_rng(1)
    x = pools(rng, False, 1, 8, 3, 16, 64)
    want = [ints(p) for p in x]
    run_copy(tsd, False, x, to_dev_i32(np.array([(2, 3, 0)] * (n - 1) + [copy])), None, n, 1, 0, 3, 64, 8, 16)
    assert tsd.attn_get_device_status() == tsd.ATTN_ERR_DEVICE_INDEX
    for p, w in zip(x, want):
        assert np.array_equal(ints(p), w)


def test_copy_past_32_bit_offsets(tsd):
    """Pages on either side of 2^31 elements and 2^32 bytes of a pool, and a layer beyond them."""
    import torch
    h_kv, page, d, n_pages = 8, 64, 128, 40000  # 5.2 GB to a pool of bf16
    k = torch.zeros(2, n_pages, h_kv, page, d, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    far = [3, n_pages - 1, 33000, 32767, 16384]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(0)
    for x in (k, v):
        for p in far:
            x[:, p] = torch.randn(2, h_kv, page, d, generator=gen, device="cuda").to(torch.bfloat16)
    copies = [(3, n_pages - 2, 64), (n_pages - 1, 5, 64), (33000, 32768, 9), (32767, 6, 64), (16384, 39000, 33)]
    tsd.attn_cache_copy(k, v, to_dev_i32(np.array(copies)), None, 5, 2, n_pages * h_kv * page, h_kv, d, n_pages, page)
    assert tsd.attn_get_device_status() == tsd.ATTN_OK
    for x in (k, v):
        for src, dst, rows in copies:
            assert torch.equal(x[:, dst, :, :rows], x[:, src, :, :rows]) and not x[:, dst, :, rows:].any()
        assert int((x != 0).flatten(2).any(2).sum()) == 2 * (len(far) + len(copies))


def test_state_is_left_alone_around_it(tsd):
    """Nothing outside the arrays is written: calls on the middle of larger ones."""
    rng = np.random.default_rng(5)
    B, max_pages, n_pages, page = 11, 7, 60, 16
    table, counts = pu.state(rng, B, max_pages, n_pages, page)
    big_t, big_c = to_dev_i32(np.full((B + 2) * max_pages, GUARD)), to_dev_i32(np.full(n_pages + 14, GUARD))
    t, c = big_t[max_pages:-max_pages].view(B, max_pages), big_c[7:-7]
    t.copy_(to_dev_i32(table))
    c.copy_(to_dev_i32(counts))
    plain = pu.Pages(table, counts, page)
    parents = rng.integers(0, B, B)
    plain.fork(parents)
    lens, new = grow(rng, plain, 20)
    plain.reserve(lens, new)
    keep = rng.integers(0, 100, B)
    tsd.attn_cache_fork(t, None, c, to_dev_i32(parents), B, n_pages, max_pages)
    reserve(tsd, t, c, to_dev_i32(lens), to_dev_i32(new), 20, page)
    plain.release(keep)
    tsd.attn_cache_release(t, c, to_dev_i32(keep), B, n_pages, page, max_pages)
    check_state(plain, t, c)
    assert (ints(big_t)[:max_pages] == GUARD).all() and (ints(big_t)[-max_pages:] == GUARD).all()
    assert (ints(big_c)[:7] == GUARD).all() and (ints(big_c)[-7:] == GUARD).all()


def test_another_stream_and_a_graph(tsd):
    """A step of a group of beams on a side stream and captured: replays go on from the state they find."""
    import torch
    rng = np.random.default_rng(9)
    B, max_pages, n_pages, page, h_kv, d = 12, 8, 120, 16, 2, 64
    table, counts = pu.state(rng, B, max_pages - 4, n_pages, page)
    table = np.concatenate([table, np.full((B, 4), -1)], 1)
    x = pools(rng, False, 1, n_pages, h_kv, page, d)
    t, c, parents = to_dev_i32(table), to_dev_i32(counts), to_dev_i32(np.arange(B))
    lens, new = to_dev_i32(np.zeros(B)), to_dev_i32(np.ones(B))
    copies, n_copies, n_missing = to_dev_i32(np.full((B, 3), GUARD)), ones(), ones()
    ws, n = workspace(tsd, B, n_pages)

    def step(s):
        tsd.attn_cache_fork(t, None, c, parents, B, n_pages, max_pages, stream=s)
        tsd.attn_cache_reserve(t, c, lens, new, copies, n_copies, n_missing, B, 1, n_pages, page, max_pages, ws, n, stream=s)
        tsd.attn_cache_copy(*x, copies, n_copies, B, 1, 0, h_kv, d, n_pages, page, stream=s)

    plain = pu.Pages(table, counts, page)
    content = [ints(p).copy() for p in x]
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        step(side)
    for i in range(6):
        par = rng.integers(0, B, B)
        held = np.array([sum(p >= 0 for p in plain.table[q]) for q in par])
        ln = np.minimum(held * page + rng.integers(-6, 2, B), max_pages * page).clip(1)
        parents.copy_(to_dev_i32(par))
        lens.copy_(to_dev_i32(ln))
        torch.cuda.synchronize()
        if i % 2:
            graph.replay()
        else:
            step(side)
        torch.cuda.synchronize()
        plain.fork(par)
        listed, missing = plain.reserve(ln.tolist(), [1] * B)
        assert missing == 0 and int(n_copies) == len(listed)
        content = [copied(torch.from_numpy(p), listed, n_pages, h_kv, page) for p in content]
        check_state(plain, t, c)
        for p, w in zip(x, content):
            assert np.array_equal(ints(p), w)


@pytest.mark.parametrize("seed", range(12))
def test_random_calls_one_after_the_other(tsd, seed):
    """Forks, reserves, releases and compactions at random on one state, with their copies: tables and
    counts as the plain form's after every call, and every row's contents as when they were written."""
    import torch
    rng = np.random.default_rng(70 + seed)
    B, max_pages, page = int(rng.integers(1, 40)), int(rng.integers(1, 12)), int(rng.choice([16, 32, 64]))
    n_pages, h_kv, d, q4 = int(rng.integers(1, B * max_pages + 5)), int(rng.integers(1, 4)), 64, bool(seed % 2)
    plain = pu.Pages(np.full((B, max_pages), -1), np.zeros(n_pages), page)
    t, c = to_dev_i32(plain.table), to_dev_i32(plain.counts)
    x = pools(rng, q4, 2, n_pages, h_kv, page, d)
    held = np.zeros(B, int)      # rows of each sequence
    words = [[] for _ in range(B)]  # what was written into each row, as numbers
    serial = 1

    def row_of(b, p):
        return plain.table[b][p // page] * h_kv * page + p % page

    def moved(copies, n):
        listed = to_dev_i32(np.array([list(e) for e in copies] + [[0, 0, 1]]))
        run_copy(tsd, q4, x, listed, to_dev_i32([len(copies)]), len(copies) + 1, 2, n_pages * h_kv * page, h_kv, d, n_pages, page)

    for _ in range(30):
        what = rng.choice(["fork", "reserve", "reserve", "release", "compact"])
        if what == "fork":
            parents = rng.integers(-1, B, B) if rng.random() < 0.5 else np.arange(B) // 2 * 2
            plain.fork(parents)
            tsd.attn_cache_fork(t, None, c, to_dev_i32(parents), B, n_pages, max_pages)
            held = np.where(parents >= 0, held[parents], 0)
            words = [list(words[q]) if q >= 0 else [] for q in parents]
        elif what == "release":
            keep = np.where(rng.random(B) < 0.4, rng.integers(0, max_pages * page + 1, B), -1)
            keep = np.minimum(keep, held)
            plain.release(keep)
            tsd.attn_cache_release(t, c, to_dev_i32(keep), B, n_pages, page, max_pages)
            held = np.where(keep >= 0, keep, held)
            words = [w[:n] for w, n in zip(words, held)]
        elif what == "compact":
            most = int(rng.choice([1, 3, n_pages]))
            copies, used = plain.compact(most)
            out, n_copies, n_used = to_dev_i32(np.full((most, 3), GUARD)), ones(), ones()
            ws, n = workspace(tsd, B, n_pages)
            tsd.attn_cache_compact(t, c, t, c, out, n_copies, n_used, B, n_pages, page, max_pages, most, ws, n)
            assert (int(n_copies), int(n_used)) == (len(copies), used)
            assert ints(out)[:len(copies)].tolist() == [list(e) for e in copies]
            moved(copies, most)
        else:
            most = int(rng.choice([1, 1, 2, 30]))
            new = np.minimum(rng.integers(0, most + 1, B), max_pages * page - held)
            copies, missing = plain.reserve((held + new).tolist(), new.tolist())
            got, n, n_missing = reserve(tsd, t, c, to_dev_i32(held + new), to_dev_i32(new), most, page)
            assert (n, n_missing) == (len(copies), missing) and got[:n].tolist() == [list(e) for e in copies]
            if not missing:
                moved(copies, B)
                for b in range(B):  # the new tokens' rows, of every head and layer
                    for p in range(held[b], held[b] + new[b]):
                        words[b].append(serial % 251)
                        for pool in x:
                            pool[:, row_of(b, p):row_of(b, p) + (h_kv - 1) * page + 1:page] = serial % 251
                        serial += 1
                held = held + new
        check_state(plain, t, c)
    assert tsd.attn_get_device_status() == tsd.ATTN_OK
    for pool in x:
        rows = ints(pool)
        for b in range(B):
            for p, word in enumerate(words[b]):
                at = row_of(b, p)
                assert (rows[:, at:at + (h_kv - 1) * page + 1:page] == word).all(), (b, p)


def test_counts_that_do_not_fit_the_table(tsd):
    """A page twice in a row, counts too low and too high, negative ones: no access out of range, every
    entry a page or none, and what lies around the arrays as it was."""
    rng = np.random.default_rng(3)
    for seed in range(20):
        B, max_pages, n_pages = 40, 6, 60
        big_t, big_c = to_dev_i32(np.full(B * max_pages + 200, GUARD)), to_dev_i32(np.full(n_pages + 200, GUARD))
        t, c = big_t[100:-100].view(B, max_pages), big_c[100:-100]
        t.copy_(to_dev_i32(rng.integers(-1, n_pages, (B, max_pages)) if seed % 2 else rng.integers(-1, 8, (B, max_pages))))
        c.copy_(to_dev_i32(rng.integers(-2, 5, n_pages)))
        lens = rng.integers(0, max_pages * 16 + 1, B)
        new = [1, 40][seed % 4 // 2]
        reserve(tsd, t, c, to_dev_i32(lens), None, new, 16)
        assert ((ints(t) >= -1) & (ints(t) < n_pages)).all()
        tsd.attn_cache_fork(t, None, c, to_dev_i32(rng.integers(-1, B, B)), B, n_pages, max_pages)
        tsd.attn_cache_release(t, c, to_dev_i32(lens // 2), B, n_pages, 16, max_pages)
        assert ((ints(t) >= -1) & (ints(t) < n_pages)).all()
        for big in (big_t, big_c):
            assert (ints(big)[:100] == GUARD).all() and (ints(big)[-100:] == GUARD).all()
    assert tsd.attn_get_device_status() == tsd.ATTN_OK


FIRST_CALLS = """
import numpy as np, torch
import transformer_scaled_dot_gb300 as tsd
i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
n_pages, wsb = {n_pages}, tsd.attn_cache_pages_workspace_bytes(2, {n_pages})
table, counts, lens, parents = i32([[0, -1], [0, -1]]), torch.zeros(n_pages, dtype=torch.int32, device="cuda"), i32([17, 17]), i32([0, 0])
counts[0] = 2
copies, n, missing, ws = i32([[0, 0, 0]] * 4), i32([0]), i32([0]), torch.zeros(wsb, dtype=torch.uint8, device="cuda")
k, v = torch.randn(n_pages if n_pages < 99 else 99, 1, 16, 64, device="cuda").bfloat16(), torch.randn(99, 1, 16, 64, device="cuda").bfloat16()
x = torch.randn({B} * 2, 1000, device="cuda").bfloat16()
scores, tokens, rows = torch.zeros({B}, 2, device="cuda"), i32([[9, 9]] * {B}), i32([[9, 9]] * {B})
bsb = tsd.beam_select_workspace_bytes({B}, 2, 1000)
bws = torch.zeros(bsb, dtype=torch.uint8, device="cuda")
torch.cuda.synchronize()
with torch.cuda.graph(graph, stream=stream):
    tsd.attn_cache_fork(table, None, counts, parents, 2, n_pages, 2, stream=stream)
    tsd.attn_cache_reserve(table, counts, lens, None, copies, n, missing, 2, 1, n_pages, 16, 2, ws, wsb, stream=stream)
    tsd.attn_cache_copy(k, v, copies, n, 2, 1, 0, 1, 64, 99 if n_pages > 99 else n_pages, 16, stream=stream)
    tsd.attn_cache_release(table, counts, lens, 2, n_pages, 16, 2, stream=stream)
    tsd.attn_cache_compact(table, counts, table, counts, copies, n, missing, 2, n_pages, 16, 2, 4, ws, wsb, stream=stream)
    tsd.beam_select(x, 1000, scores, None, {B}, 2, 1000, -1, 0.0, tokens, rows, scores, None, None, None, bws, bsb, stream=stream)
assert (tokens == 9).all() and table.tolist() == [[0, -1], [0, -1]]
graph.replay()
torch.cuda.synchronize()
assert table.tolist() == [[0, 1], [0, 2]] and counts[:4].tolist() == [2, 1, 1, 0], (table, counts[:4])
assert (tokens >= 0).all() and (tokens != 9).any() and torch.isfinite(scores).all()
assert tsd.attn_get_device_status() == tsd.ATTN_OK
print("captured first")
"""


@pytest.mark.parametrize("n_pages,B", [(99, 1), (300000, 20)])
def test_first_calls_inside_a_capture(tsd, n_pages, B):
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS.format(n_pages=n_pages, B=B)], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stdout + r.stderr
