"""GPU tests of the paged cache at the ends of its sizes: the longest cache, the
most sequences, the most heads, and the library's first calls inside a capture."""
import os
import subprocess
import sys

import numpy as np
import pytest

import paged_util as pu
from gpu_util import to_dev_bf16, to_dev_i32, to_host_f64
from test_paged_gpu import bf16, dev, tsd  # noqa: F401 (tsd: a fixture)

pytestmark = pytest.mark.gpu


def call_decode(tsd, q4, q, pools, out, table, lens, B, h, h_kv, n_q, d, n_pages, page, max_pages):
    import torch
    wsb = tsd.attn_decode_paged_workspace_bytes(B, h, h_kv, n_q, d, page, max_pages)
    ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
    tail = (out, table, lens, None, B, h, h_kv, n_q, d, n_pages, page, max_pages, 1, 0.0, ws, wsb)
    if q4:
        tsd.attn_decode_paged_q4(q, *pools, 0.25, 0.5, *tail)
    else:
        tsd.attn_decode_paged(q, *pools, *tail)
    torch.cuda.synchronize()
    assert tsd.attn_get_device_status() == tsd.ATTN_OK


def make_pools(rng, q4, n_pages, h_kv, page, d):
    """Device pools and their 64-bit values [n_pages, h_kv, page, d]."""
    shape = (n_pages, h_kv, page)
    if not q4:
        bits, x = zip(*(bf16(rng, *shape, d) for _ in range(2)))
        return [to_dev_bf16(b) for b in bits], x
    codes = [rng.integers(0, 256, shape + (d // 2,), dtype=np.uint8) for _ in range(2)]
    scales = [rng.integers(0x30, 0x40, shape + (d // 16,), dtype=np.uint8) for _ in range(2)]
    x = [pu.dequantise(c, s, f) for c, s, f in zip(codes, scales, (0.25, 0.5))]
    return [dev(a) for pair in zip(codes, scales) for a in pair], x


@pytest.mark.parametrize("q4", [False, True], ids=["bf16", "q4"])
def test_the_longest_cache(tsd, q4):
    """2^30 rows of one sequence, a page of 256 rows again and again but for the last page: queries
    of 0 average all rows, of which the last row of the last page alone is seen by the second
    token only; and an append writes that row."""
    import torch
    d, page, max_pages = 64, 256, 1 << 22
    rng = np.random.default_rng(90)
    pools, (_, v) = make_pools(rng, q4, 2, 1, page, d)
    table = torch.zeros(1, max_pages, dtype=torch.int32, device="cuda")
    table[0, -1] = 1
    lens = to_dev_i32([1 << 30])
    q = torch.zeros(1, 2, 2, d, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q)
    call_decode(tsd, q4, q, pools, out, table, lens, 1, 2, 1, 2, d, 2, page, max_pages)
    n = float(1 << 30)
    total = v[0, 0].sum(0) * (max_pages - 1) + v[1, 0].sum(0)
    want = np.stack([(total - v[1, 0, -1]) / (n - 1), total / n])
    mass = np.abs(v).mean()
    # the rows of a warp are added up one product of 16 rows after the other, in 32 bits (cut off:
    # 2^-23 of the sum so far, at most n / 16 / 4 warps of mass over at least 152 blocks)
    steps = n / 16 / 4 / 152
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + steps * 2.0 ** -23) * 2 * mass
    got = to_host_f64(out)[0]
    assert np.all(np.abs(got - want) <= tol)
    # an append at the last position
    x_bits, x = bf16(rng, 1, 1, 2, d)
    xd = to_dev_bf16(x_bits)
    args = (None, 0, 0, 0, xd, xd[:, :, 1:], 2 * d, d, 2 * d, None, None, *pools)
    rest = (table, lens, None, None, 0, 0, 0, 1, 1, 1, 1, d, 2, page, max_pages)
    before = [p.clone() for p in pools]
    if q4:
        tsd.attn_cache_append_q4(*args, 0.25, 0.5, *rest)
    else:
        tsd.attn_cache_append(*args, *rest)
        torch.cuda.synchronize()
        assert np.array_equal(to_host_f64(pools[1])[1, 0, -1], x[0, 0, 1])
    torch.cuda.synchronize()
    assert tsd.attn_get_device_status() == tsd.ATTN_OK
    for a, b in zip(pools, before):
        changed = (a.view(torch.uint8) != b.view(torch.uint8)).any(-1).nonzero().tolist()
        assert changed == [[1, 0, page - 1]]


def check_short(got, q, k, v, table, lens, page, group):
    """Sequences of at most one page each, in one go: q [B, h, d], k, v [n_pages, h_kv, page, d]."""
    B, h, d = q.shape
    seen = np.arange(page) < np.asarray(lens)[:, None]
    for a in range(0, B, 4096):
        b = slice(a, min(a + 4096, B))
        kk, vv = (np.repeat(x[np.maximum(table[b, 0], 0)], group, 1) for x in (k, v))
        x = np.einsum("bhd,bhpd->bhp", q[b], kk) / np.sqrt(d)
        x = np.where(seen[b][:, None], x, -np.inf)
        top = x.max(-1, keepdims=True)
        w = np.exp(x - np.where(np.isfinite(top), top, 0))
        w /= np.maximum(w.sum(-1, keepdims=True), 1e-300)
        ref = np.einsum("bhp,bhpd->bhd", w, vv)
        mass = np.einsum("bhp,bhpd->bhd", w, np.abs(vv)) + 2.0 ** -25 * np.abs(vv).sum(2)
        size = np.einsum("bhd,bhpd->bhp", np.abs(q[b]), np.abs(kk)).max(-1) / np.sqrt(d)
        assert np.all(np.abs(got[b] - ref) <= pu.decode_tolerance(ref, mass, size, page, d))
        assert np.all(got[b][np.asarray(lens)[b] <= 0] == 0)


@pytest.mark.parametrize("max_pages", [1, 128], ids=["narrow", "wide"])
@pytest.mark.parametrize("q4", [False, True], ids=["bf16", "q4"])
def test_the_most_sequences(tsd, q4, max_pages):
    """65535 of them, of 0 to 16 rows each."""
    import torch
    B, h, h_kv, d, page, n_pages = 65535, 2, 1, 64, 16, 500
    rng = np.random.default_rng(91)
    pools, (k, v) = make_pools(rng, q4, n_pages, h_kv, page, d)
    table = np.full((B, max_pages), -1, dtype=np.int32)
    table[:, 0] = rng.integers(0, n_pages, B)
    lens = rng.integers(0, page + 1, B)
    q_bits, q = bf16(rng, B, h, 1, d)
    out = torch.full((B, h, 1, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    call_decode(tsd, q4, to_dev_bf16(q_bits), pools, out, to_dev_i32(table), to_dev_i32(lens), B, h, h_kv, 1,
                d, n_pages, page, max_pages)
    check_short(to_host_f64(out)[:, :, 0], q[:, :, 0], k, v, table, lens, page, h // h_kv)


@pytest.mark.parametrize("max_pages", [1, 128], ids=["narrow", "wide"])
@pytest.mark.parametrize("q4", [False, True], ids=["bf16", "q4"])
def test_the_most_heads(tsd, q4, max_pages):
    """65535 query heads, and as many key heads; the new row appended first."""
    import torch
    B, h, d, page = 1, 65535, 64, 16
    rng = np.random.default_rng(92)
    pools, (k, v) = make_pools(rng, q4, 1, h, page, d)
    table = np.full((B, max_pages), -1, dtype=np.int32)
    table[0, 0] = 0
    lens = [7]
    x_bits, x = bf16(rng, B, 1, 3 * h, d)
    xd = to_dev_bf16(x_bits)
    q_out = torch.empty(B, h, 1, d, dtype=torch.bfloat16, device="cuda")
    st = (3 * h * d, d, 3 * h * d)
    args = (xd, *st, xd[:, :, h:], xd[:, :, 2 * h:], *st, q_out, None, *pools)
    rest = (to_dev_i32(table), to_dev_i32(lens), None, None, 0, 0, 0, B, h, h, 1, d, 1, page, max_pages)
    if q4:
        tsd.attn_cache_append_q4(*args, 0.25, 0.5, *rest)
        raw = [p.cpu().numpy() for p in pools]
        k, v = (pu.dequantise(raw[2 * i], raw[2 * i + 1], f) for i, f in enumerate((0.25, 0.5)))
        for got, want in ((k, x[0, 0, h:2 * h]), (v, x[0, 0, 2 * h:])):
            # half a step of the codes is a sixth of the largest of 16 at most, a scale is off by
            # 2^-4 of it, or by half of e4m3's least step, times 6 and the factor, where it is small
            top = np.abs(want).reshape(h, 4, 16).max(-1).repeat(16, -1)
            assert np.all(np.abs(got[0, :, 6] - want) <= top * (1 / 6 + 1 / 16) + 6 * 0.5 * 2.0 ** -10)
    else:
        tsd.attn_cache_append(*args, *rest)
        k, v = (to_host_f64(p) for p in pools)
        assert np.array_equal(k[0, :, 6], x[0, 0, h:2 * h]) and np.array_equal(v[0, :, 6], x[0, 0, 2 * h:])
    assert np.array_equal(to_host_f64(q_out)[0, :, 0], x[0, 0, :h])
    out = torch.full((B, h, 1, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    call_decode(tsd, q4, q_out, pools, out, to_dev_i32(table), to_dev_i32(lens), B, h, h, 1, d, 1, page,
                max_pages)
    check_short(to_host_f64(out)[:, :, 0], x[:, 0, :h], k, v, table, lens, page, 1)


FIRST_CALLS = """
import torch
import transformer_scaled_dot_gb300 as tsd
x = torch.randn(2, 1, 12, 64, device="cuda").bfloat16()
table = torch.arange(256, dtype=torch.int32, device="cuda").view(2, 128)
lens = torch.tensor([900, 40], dtype=torch.int32, device="cuda")
bf = [torch.randn(256, 2, 16, 64, device="cuda").bfloat16() for _ in range(2)]
q4 = [torch.full((256, 2, 16, w), 0x39, dtype=torch.uint8, device="cuda") for w in (32, 4, 32, 4)]
kept = [[p.clone() for p in bf], [p.clone() for p in q4]]
q, out = (torch.zeros(2, 8, 1, 64, device="cuda").bfloat16() for _ in range(2))
out4 = out.clone()
st = (768, 64, 768)
size = tsd.attn_decode_paged_workspace_bytes(2, 8, 2, 1, 64, 16, 128)
ws = torch.empty(size, dtype=torch.uint8, device="cuda")
def step():
    kv = (x[:, :, 8:], x[:, :, 10:])
    sizes = (2, 8, 2, 1, 64, 256, 16, 128)
    tsd.attn_cache_append(x, *st, *kv, *st, q, None, *bf, table, lens, None, None, 0, 0, 0, *sizes)
    tsd.attn_decode_paged(q, *bf, out, table, lens, None, *sizes, 1, 0.0, ws, size)
    tsd.attn_cache_append_q4(x, *st, *kv, *st, q, None, *q4, 0.1, 0.1, table, lens, None, None, 0, 0, 0, *sizes)
    tsd.attn_decode_paged_q4(q, *q4, 0.1, 0.1, out4, table, lens, None, *sizes, 1, 0.0, ws, size)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    step()
for pools, old in zip((bf, q4), kept):
    assert all(torch.equal(a, b) for a, b in zip(pools, old))  # nothing ran yet
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in (out, out4, *bf, *q4)]
for pools, old in zip((bf, q4), kept):
    for a, b in zip(pools, old):
        a.copy_(b)
out.zero_(), out4.zero_()
step()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, (out, out4, *bf, *q4)))
assert out.float().abs().sum() > 0 and tsd.attn_get_device_status() == tsd.ATTN_OK
print("same")
"""


def test_first_calls_inside_a_capture(tsd):
    """A process whose first calls of the library are captured ones; replayed, they give what the
    same calls give outside a graph."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


def test_the_smallest_factor_over_the_longest_cache(tsd):
    """Values of 2^-100 under weights whose sum is near the largest that a 4-bit cache can have: the
    rows that a block begins with have logits 3.9 powers of 2 below all others, so that weights
    reach 2^14.9 times 2^30 rows. Every value is the same, and so is the output."""
    import torch
    d, page = 64, 256
    # rows for which 2^-100 over the sum, 2^11 (its logits' rise) rows, is 17.5 of fp32's least steps
    rows = int(2.0 ** 38 / 17.5 / 2.0 ** 3.9)
    max_pages = rows // page
    rows = max_pages * page
    codes = torch.zeros(2, 1, page, d // 2, dtype=torch.uint8, device="cuda")
    codes[1, :, :, 0] = 2  # a key's first column: 0 on page 0, 1 on page 1
    v_codes = torch.full_like(codes, 0x22)
    scales = torch.full((2, 1, page, d // 16), 0x38, dtype=torch.uint8, device="cuda")
    table = np.ones((1, max_pages), dtype=np.int32)
    blocks = 3 * torch.cuda.get_device_properties(0).multi_processor_count
    units = rows // 64 + 6  # of 64 rows, six standing for none
    for block in range(blocks):
        first = max(block * units // blocks - 6, 0) * 64 // page
        table[0, first:first + 2] = 0
    q = torch.zeros(1, 1, 1, d, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1
    out = torch.empty_like(q)
    wsb = tsd.attn_decode_paged_workspace_bytes(1, 1, 1, 1, d, page, max_pages)
    ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
    tsd.attn_decode_paged_q4(q, codes, scales, v_codes, scales, 1.0, 2.0 ** -100, out, to_dev_i32(table),
                             to_dev_i32([rows]), None, 1, 1, 1, 1, d, 2, page, max_pages, 0,
                             3.9 * np.log(2), ws, wsb)
    torch.cuda.synchronize()
    assert tsd.attn_get_device_status() == tsd.ATTN_OK
    got = to_host_f64(out).ravel() * 2.0 ** 100
    # bf16's rounding; a weight's to 11 bits; a warp's sums, one product of 16 rows after the other
    # in 32 bits (2^-23 of the sum so far, half of it on the average), in O and in the weights' own
    steps = rows / 16 / 4 / blocks
    assert np.all(np.abs(got - 1) <= 2.0 ** -8 + 2.0 ** -11 + 2 * steps * 2.0 ** -24), got
