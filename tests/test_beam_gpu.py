"""A step of beam search against a plain form in 64 bits, and beam searches over a paged cache."""
import math

import numpy as np
import pytest

import pages_util as pu
import synthetic
from gpu_util import to_dev_bf16, to_dev_i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tsd():
    import torch
    from transformer_scaled_dot_gb300 import build as native_build
    native_build.build()
    import transformer_scaled_dot_gb300 as m
    m.library()
    torch.cuda.set_device(0)
    return m


def dev_f32(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()


class Step:
    """Device arrays of one selection."""

    def __init__(self, tsd, B, K, V, f32, end, alpha=0.6, pad=0, offset=0):
        import torch
        self.tsd, self.B, self.K, self.V, self.f32, self.end, self.alpha = tsd, B, K, V, f32, end, alpha
        self.stride = V + pad
        self.buffer = torch.zeros(B * K * self.stride + offset, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
        self.x = self.buffer[offset:]
        self.scores, self.lengths = dev_f32(np.zeros((B, K))), to_dev_i32(np.ones(B))
        self.tokens, self.parents = to_dev_i32(np.full((B, K), -7)), to_dev_i32(np.full((B, K), -7))
        self.new_scores = dev_f32(np.full((B, K), np.nan))
        self.ended = [dev_f32(np.full((B, K), -np.inf)), to_dev_i32(np.full((B, K), -7)), to_dev_i32(np.full((B, K), -7))]
        self.bytes = tsd.beam_select_workspace_bytes(B, K, V)
        self.ws = torch.full((self.bytes,), 0xff, dtype=torch.uint8, device="cuda")  # NaN everywhere

    def fill(self, x):
        """x [B, K, V] values; what lies behind each row is +infinity. Returns them as the device has them, in 64 bits."""
        import torch
        full = np.full((self.B * self.K, self.stride), np.inf, np.float32)
        full[:, :self.V] = x.reshape(-1, self.V)
        if self.f32:
            self.x.copy_(torch.from_numpy(full.ravel()))
            return full[:, :self.V].astype(np.float64).reshape(x.shape)
        with np.errstate(invalid="ignore"):
            bits = torch.from_numpy(full).to(torch.bfloat16)
        self.x.copy_(bits.view(-1))
        return bits.double().numpy()[:, :self.V].reshape(x.shape)

    def run(self, stream=None):
        call = self.tsd.beam_select_f32 if self.f32 else self.tsd.beam_select
        call(self.x, self.stride, self.scores, self.lengths if self.end >= 0 else None, self.B, self.K, self.V, self.end,
             self.alpha, self.tokens, self.parents, self.new_scores, *(self.ended if self.end >= 0 else (None,) * 3),
             self.ws, self.bytes, stream=stream)

    def get(self):
        return [t.cpu().numpy() for t in (self.tokens, self.parents, self.new_scores, *self.ended)]


def logits(rng, B, K, V):
    """As a model gives them: most tokens unlikely, a few likely."""
    x = 2 * rng.standard_normal((B, K, V)) - 4
    for _ in range(5):
        at = rng.integers(0, V, (B, K))
        np.put_along_axis(x, at[..., None], 3 + 4 * rng.random((B, K, 1)), 2)
    return x


def tolerance(ref):
    """A total: half a step of 32 bits, 2^-24 of it; the log-sum's error, whose exponentials and
    tile sums are good to 2^-22 + 2^-23 + 10 2^-24 (ten additions from a lane to a tile) and whose joining
    adds 2^-22 + 2^-23 and a rounding: 2^-20 in all."""
    return 2.0 ** -24 * np.abs(ref) + 2.0 ** -20


def check(step, x, what=""):
    """Runs the step and compares it with the plain form; the sentences whose candidates are told
    apart by less than 32-bit sums resolve are left out, and few."""
    s = step
    scores, lengths = s.scores.cpu().numpy(), s.lengths.cpu().numpy()
    before = [t.cpu().numpy() for t in s.ended]
    tokens, parents, new, ended, close = pu.select(x, scores, lengths, s.end, s.alpha, before)
    s.run()
    got = s.get()
    assert len(close) <= max(1, s.B // 20), close
    for b in range(s.B):
        if b in close:
            continue
        assert np.array_equal(got[0][b], tokens[b]), (what, b)
        assert np.array_equal(got[1][b], parents[b]), (what, b)
        live = new[b] > -np.inf
        assert np.array_equal(got[2][b] > -np.inf, live) and not np.isnan(got[2][b]).any()
        assert (np.abs(got[2][b][live] - new[b][live]) <= tolerance(new[b][live])).all(), (what, b)
        if s.end >= 0:
            held = ended[0][b] > -np.inf
            assert np.array_equal(got[3][b] > -np.inf, held), (what, b)
            # the penalty divides total and error alike; it is at least 1 for n >= 1 and alpha >= 0
            scale = ((5 + max(int(lengths[b]), 1)) / 6) ** s.alpha
            assert (np.abs(got[3][b][held] - ended[0][b][held]) <= 2 * 2.0 ** -24 * np.abs(ended[0][b][held]) + 2.0 ** -20 / min(scale, 1)).all()
            assert np.array_equal(got[4][b], ended[1][b]) and np.array_equal(got[5][b], ended[2][b]), (what, b)
    return got


SHAPES = [
    # B, K, V, row padding, elements before the first row
    (1, 4, 32000, 0, 0), (3, 1, 1, 0, 0), (2, 1, 7, 0, 0), (2, 16, 2, 0, 0), (5, 3, 1023, 0, 0), (5, 3, 1024, 0, 0),
    (4, 5, 1025, 0, 0), (7, 4, 2049, 7, 0), (6, 4, 32003, 0, 0), (3, 8, 4096, 8, 8), (3, 8, 4096, 0, 1), (2, 16, 50257, 3, 5),
    (33, 2, 5000, 0, 0), (2, 13, 131072, 0, 0),
]


@pytest.mark.parametrize("end", [2, -1])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_step(tsd, shape, f32, end):
    B, K, V, pad, offset = shape
    end = min(end, V - 1)
    rng = np.random.default_rng(B + K + V)
    s = Step(tsd, B, K, V, f32, end, pad=pad, offset=offset)
    x = logits(rng, B, K, V)
    if end >= 0:
        x[:, :, end] += 9 * (rng.random((B, K)) < 0.5)
    x = s.fill(x)
    scores = -8 * rng.random((B, K))
    scores[::3, 1:] = -np.inf  # a sentence's start
    s.scores.copy_(dev_f32(scores))
    s.lengths.copy_(to_dev_i32(rng.integers(1, 60, B)))
    old = np.sort(np.where(rng.random((B, K)) < 0.5, -np.inf, -3 * rng.random((B, K))))[:, ::-1]
    s.ended[0].copy_(dev_f32(old))
    check(s, x)
    assert tsd.attn_get_device_status() == tsd.ATTN_OK


@pytest.mark.parametrize("f32", [False, True])
def test_largest_vocabulary(tsd, f32):
    """2^20 tokens of 16 beams: every thread holds as many tiles as there are."""
    rng = np.random.default_rng(3)
    s = Step(tsd, 1, 16, 1 << 20, f32, 5)
    x = s.fill(logits(rng, 1, 16, 1 << 20))
    s.scores.copy_(dev_f32(-6 * rng.random((1, 16))))
    check(s, x)


@pytest.mark.parametrize("kind", ["one group", "five groups", "few tokens", "all alike"])
def test_best_tokens_close_together(tsd, kind):
    """The likely tokens all in tiles that lie 8 (of 1024 tokens) apart in one beam, which is how the
    search for them is split: many more tiles pass its first look than have to."""
    rng = np.random.default_rng(6)
    K, V = 16, 1 << 20
    s = Step(tsd, 1, K, V, True, 3 * 1024)
    x = rng.standard_normal((1, K, V)).astype(np.float32) - 20
    tile = np.arange(V) // 1024
    if kind == "one group":
        x[0, 2, tile % 8 == 5] += 25
    elif kind == "five groups":
        x[0, 9, tile % 8 < 5] += 25
    elif kind == "few tokens":
        x[0, :] = -np.inf
        x[0, 3, (tile % 8 == 1) & (np.arange(V) % 1024 > 1021)] = 1 + rng.random(256)
    else:
        x[0, :] = 1.5
    s.scores.copy_(dev_f32(-2 - 1e-3 * np.arange(K)[None]))
    check(s, s.fill(x))


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("V,pad", [(700, 0), (5001, 0), (5000, 8), (40960, 0)])
def test_ties_go_to_the_lowest_place(tsd, f32, V, pad):
    """All logits the same, all beams the same; few different values; two beams alike."""
    rng = np.random.default_rng(V)
    K = 4
    s = Step(tsd, 3, K, V, f32, V - 1, pad=pad)
    x = np.zeros((3, K, V))
    x[1] = rng.integers(0, 3, (K, V))
    x[2] = np.round(4 * rng.standard_normal((1, V))) / 4
    s.fill(x)
    s.scores.copy_(dev_f32(np.full((3, K), -2.5)))
    s.run()
    tokens, parents, new, _, _ = [*s.get()[:3], None, None]
    for b in (0, 2):  # equal rows, whose sums are the same to the bit: flat order
        order = np.argsort(-np.tile(x[b, 0], K), kind="stable")
        order = [at for at in order if at % V != V - 1][:K]
        assert tokens[b].tolist() == [at % V for at in order] and parents[b].tolist() == [b * K + at // V for at in order]
    assert (tokens[1] >= 0).all() and np.isfinite(new).all()
    # within one beam, whatever the others are
    s.scores.copy_(dev_f32(np.where(np.arange(K) == 1, -1.0, -np.inf) * np.ones((3, 1))))
    check(s, s.fill(x), "one beam")


def test_tokens_that_are_never_chosen(tsd):
    """-infinity in most places, in all of a row, in all of a sentence; the type's lowest value is a number."""
    rng = np.random.default_rng(0)
    B, K, V = 6, 4, 3000
    s = Step(tsd, B, K, V, False, 2)
    x = logits(rng, B, K, V)
    x[0, :, 3:] = -np.inf                       # three tokens a beam
    x[1, 1] = -np.inf                           # a beam without any
    x[2] = -np.inf                              # nothing at all
    x[3, :, :] = -np.inf
    x[3, 2, 2999] = 1.0                         # one pair in all
    x[4, :, 10:] = -3.3895e38                   # the lowest number: weight 0, a candidate all the same
    x[4, :, :10] = -np.inf
    x[5, :, :2] = -np.inf
    x[5, :, 3:] = -np.inf                       # the end token only
    x = s.fill(x)
    s.scores.copy_(dev_f32(-3 * rng.random((B, K))))
    got = check(s, x)
    assert tsd.attn_get_device_status() == tsd.ATTN_OK
    assert (got[2][2] == -np.inf).all() and got[0][2].tolist() == [2] * 4 and got[1][2].tolist() == [8, 9, 10, 11]
    assert got[0][3].tolist() == [2999, 2, 2, 2] and got[1][3, 0] == 14
    assert (got[2][5] == -np.inf).all() and (got[3][5] > -np.inf).all()


@pytest.mark.parametrize("f32", [False, True])
def test_rows_that_are_no_numbers(tsd, f32):
    """A NaN or +infinity anywhere in a row, or in a score, takes the beam out and is reported; the
    others go on. A dead beam's logits are not looked at."""
    rng = np.random.default_rng(1)
    B, K, V = 5, 3, 2500
    s = Step(tsd, B, K, V, f32, -1)
    x = logits(rng, B, K, V)
    x[0, 1, 2499] = np.nan
    x[1, 0, 0] = np.inf
    x[2, 2, 1500:] = np.nan
    scores = -3 * rng.random((B, K))
    scores[3, 1] = np.nan
    scores[4, 0] = np.inf
    s.scores.copy_(dev_f32(scores))
    x = s.fill(x)
    check(s, x)
    assert tsd.attn_get_device_status() == tsd.ATTN_ERR_DEVICE_VALUE
    assert tsd.attn_get_device_status() == tsd.ATTN_OK
    x[:, 1:] = np.nan
    s.fill(x)
    s.scores.copy_(dev_f32(np.where(np.arange(K) == 0, -1.0, -np.inf) * np.ones((B, 1))))
    x[1, 0, 0] = 0.0
    x = s.fill(x)
    check(s, x)
    assert tsd.attn_get_device_status() == tsd.ATTN_OK


def test_far_values(tsd):
    """Logits and scores of very different sizes: totals in 64 bits, no overflow."""
    rng = np.random.default_rng(2)
    B, K, V = 4, 4, 4000
    s = Step(tsd, B, K, V, True, 7)
    x = rng.standard_normal((B, K, V))
    x[0] *= 1e30
    x[1] *= 100
    x[2] = x[2] * 1e-3 + 1000
    x[3] -= 3e38
    scores = -np.array([1, 1e4, 500, 1e-3])[:, None] * (1 + rng.random((B, K)))
    s.scores.copy_(dev_f32(scores))
    check(s, s.fill(x))


@pytest.mark.parametrize("alpha", [0.0, 0.6, 1.0, -0.5])
def test_ended_hypotheses(tsd, alpha):
    """The ended list over several steps, lengths of zero and below, equal scores, a NaN among the earlier ones."""
    rng = np.random.default_rng(7)
    B, K, V = 16, 5, 600
    s = Step(tsd, B, K, V, False, 0, alpha=alpha)
    for step in range(4):
        x = logits(rng, B, K, V)
        x[..., 0] += 8 * rng.random((B, K))
        x = s.fill(x)
        s.scores.copy_(dev_f32(-4 * rng.random((B, K))))
        s.lengths.copy_(to_dev_i32(np.where(np.arange(B) % 5 == 4, 0, rng.integers(1, 9, B))))
        check(s, x, step)
    # equal ended scores: the earlier one first, and places in order
    s = Step(tsd, 1, 3, 8, True, 0, alpha=0.0)
    x = np.full((1, 3, 8), -np.inf)
    x[..., 0] = 0  # each beam ends for certain: its total is its score
    s.fill(x)
    s.scores.copy_(dev_f32([[-2, -1, -2]]))
    s.ended[0].copy_(dev_f32([[-2, np.nan, -1]]))
    s.ended[1].copy_(to_dev_i32([[70, 71, 72]]))
    s.ended[2].copy_(to_dev_i32([[80, 81, 82]]))
    s.run()
    got = s.get()
    assert got[3].tolist() == [[-1, -1, -2]] and got[4].tolist() == [[72, 1, 70]] and got[5].tolist() == [[82, 1, 80]]


@pytest.mark.parametrize("alpha", [1e6, -1e12, 3e38])
def test_one_token_has_no_penalty(tsd, alpha):
    """(6 / 6)^alpha is 1 whatever alpha is; with more tokens the score is 0 or is none."""
    s = Step(tsd, 2, 2, 8, True, 0, alpha=alpha)
    x = np.full((2, 2, 8), -np.inf)
    x[..., 0] = 0  # each beam ends for certain: its total is its score
    s.fill(x)
    s.scores.copy_(dev_f32([[-3, -1.5], [-2, -4]]))
    s.lengths.copy_(to_dev_i32([1, 2]))
    s.run()
    got = s.get()
    assert got[3].tolist() == [[-1.5, -3], [0, 0] if alpha > 0 else [-np.inf, -np.inf]]
    assert got[4].tolist() == [[1, 0], [2, 3] if alpha > 0 else [-7, -7]]


@pytest.mark.parametrize("B,V", [(1, v) for v in (17, 33, 96, 120, 128, 129, 300, 1000, 1024, 2000, 4100)]
                         + [(30, v) for v in (33, 96, 128, 129, 1000, 2000, 4100)]
                         + [(60, v) for v in (40, 129, 300, 2000, 4000)] + [(170, 96), (170, 1100), (310, 128), (310, 200)])
@pytest.mark.parametrize("K", [7, 16])
def test_few_tiles(tsd, B, K, V):
    """One block, two, four and eight to a sentence, and two launches; fewer tiles than candidates: beams
    alike, one far ahead of the others (all candidates in its row), equal rows."""
    rng = np.random.default_rng(100 * B + 10 * K + V)
    s = Step(tsd, B, K, V, bool((B + V) % 2), 2, pad=V % 3)
    x = logits(rng, B, K, V)
    x[B // 2:, :, :] = np.round(x[B // 2:, :1, :])  # equal rows, many equal logits
    x = s.fill(x)
    kind = np.arange(B)[:, None] % 3
    scores = np.where(kind == 0, -rng.random((B, K)), np.where(kind == 1, -40.0 * np.arange(K), -0.137 * np.arange(K)))
    s.scores.copy_(dev_f32(scores))
    s.lengths.copy_(to_dev_i32(rng.integers(1, 30, B)))
    check(s, x)


@pytest.mark.parametrize("seed", range(40))
def test_random_shapes(tsd, seed):
    """Sizes, alignments, ranges of logits, dead beams and forbidden tokens at random."""
    rng = np.random.default_rng(500 + seed)
    B, K = int(rng.integers(1, 24)), int(rng.integers(1, 17))
    V = int(np.exp(rng.uniform(0, np.log(9000))))
    f32, end = bool(rng.integers(0, 2)), int(rng.integers(-1, V))
    s = Step(tsd, B, K, V, f32, end, alpha=float(rng.uniform(-1, 2)), pad=int(rng.choice([0, 0, 1, 5, 8])),
             offset=int(rng.choice([0, 0, 1, 3, 8])))
    x = float(rng.choice([0.1, 1, 3, 30, 400])) * logits(rng, B, K, V)
    x[rng.random(x.shape) < rng.choice([0, 0, 0.3, 0.95])] = -np.inf
    if end >= 0:
        x[..., end] = np.where(rng.random((B, K)) < 0.4, x.max(-1), x[..., end])
    x = s.fill(x)
    s.scores.copy_(dev_f32(np.where(rng.random((B, K)) < 0.2, -np.inf, -rng.choice([0.5, 20]) * rng.random((B, K)))))
    s.lengths.copy_(to_dev_i32(rng.integers(0, 400, B)))
    s.ended[0].copy_(dev_f32(np.where(rng.random((B, K)) < 0.5, -np.inf, -4 * rng.random((B, K)))))
    check(s, x, seed)
    assert tsd.attn_get_device_status() == tsd.ATTN_OK


@pytest.mark.parametrize("f32", [False, True])
def test_few_and_many_sentences_choose_alike(tsd, f32):
    """A sentence's choice is the same to the bit in a call of its own (one launch), in one of eight, and in one of nine (two)."""
    rng = np.random.default_rng(8)
    K, V = 4, 32768
    x, scores = logits(rng, 9, K, V), -5 * rng.random((9, K))
    got = []
    for B, at in ((9, 0), (8, 1), (1, 5)):
        s = Step(tsd, B, K, V, f32, 2)
        s.fill(x[at:at + B])
        s.scores.copy_(dev_f32(scores[at:at + B]))
        s.run()
        out = s.get()
        out[1] = out[1] % K
        out[4] = np.where(out[3] > -np.inf, out[4] % K, -1)
        got.append([a[5 - at] for a in out])
    for other in got[1:]:
        for a, b in zip(got[0], other):
            assert np.array_equal(a, b)


def test_two_streams_at_once(tsd):
    """Calls on two streams with workspaces of their own, in turn without waiting, choose as alone."""
    import torch
    rng = np.random.default_rng(12)
    steps, want = [], []
    for B, V in ((20, 32003), (3, 9000)):
        s = Step(tsd, B, 4, V, False, -1)
        s.fill(logits(rng, B, 4, V))
        s.scores.copy_(dev_f32(-5 * rng.random((B, 4))))
        s.run()
        want.append(s.get()[:3])
        steps.append((s, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for s, stream in steps:
            s.run(stream)
    torch.cuda.synchronize()
    for (s, _), w in zip(steps, want):
        for a, b in zip(s.get()[:3], w):
            assert np.array_equal(a, b)


def test_in_place_and_repeated(tsd):
    """new_scores may be the scores; the same call gives the same bits, on another stream too, and in a graph."""
    import torch
    rng = np.random.default_rng(4)
    B, K, V = 40, 4, 32003
    s = Step(tsd, B, K, V, False, -1)
    s.fill(logits(rng, B, K, V))
    scores = dev_f32(-5 * rng.random((B, K)))
    s.scores.copy_(scores)
    s.run()
    want = s.get()[:3]
    side = torch.cuda.Stream()
    s.new_scores = s.scores
    torch.cuda.synchronize()
    s.run(side)
    torch.cuda.synchronize()
    for a, b in zip(s.get()[:3], want):
        assert np.array_equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        s.run(side)
    for _ in range(3):
        s.scores.copy_(scores)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(s.get()[:3], want):
            assert np.array_equal(a, b)


# ------------------------------------------------------------------ a search over a paged cache

def tiny_model(rng, vocab, h, h_kv, d):
    """One attention layer as a language model: bf16 tables of query, key and value by token, and of logits by attention output."""
    def bits(*shape):
        return synthetic.f32_to_bf16_bits(rng.standard_normal(shape).astype(np.float32))
    q, k, v = bits(vocab, h, d), bits(vocab, h_kv, d), bits(vocab, h_kv, d)
    return q, k, v, (rng.standard_normal((h * d, vocab)) / math.sqrt(d)).astype(np.float32)


@pytest.mark.parametrize("q4", [False, True])
def test_beam_search_over_a_paged_cache(tsd, q4):
    """Selection, fork, reserve, copy, append and decode, step after step on the device: every beam's
    attention has to be that of its own tokens, which are followed here by the parents, in a cache where
    every hypothesis is stored by itself; and the end finds all pages free again."""
    import torch
    rng = np.random.default_rng(11 + q4)
    B, K, vocab, h, h_kv, d, page, steps, prompt = 3, 4, 50, 4, 2, 64, 16, 40, 13
    n, max_pages = B * K, 5
    n_pages = n * max_pages
    q, k, v, out_w = tiny_model(rng, vocab, h, h_kv, d)
    qd, kd, vd, wd = to_dev_bf16(q), to_dev_bf16(k), to_dev_bf16(v), dev_f32(out_w)
    # two caches: the searched one, and one whose rows are written anew from the tokens
    def pool():
        widths = (d // 2, d // 16, d // 2, d // 16) if q4 else (2 * d, 2 * d)
        return [torch.zeros(n_pages, h_kv, page, w, dtype=torch.uint8, device="cuda") for w in widths]
    mine, plain = pool(), pool()
    more = (0.02, 0.02) if q4 else ()
    append, decode = (tsd.attn_cache_append_q4, tsd.attn_decode_paged_q4) if q4 else (tsd.attn_cache_append, tsd.attn_decode_paged)
    table, counts = to_dev_i32(np.full((n, max_pages), -1)), to_dev_i32(np.zeros(n_pages))
    own_table = to_dev_i32(np.arange(n_pages).reshape(n, max_pages))
    lens = to_dev_i32(np.zeros(n))
    copies, n_copies, n_missing = to_dev_i32(np.zeros((n, 3))), to_dev_i32([0]), to_dev_i32([0])
    wsb = tsd.attn_cache_pages_workspace_bytes(n, n_pages)
    ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
    dsb = tsd.attn_decode_paged_workspace_bytes(n, h, h_kv, 1, d, page, max_pages)
    dws = torch.empty(dsb, dtype=torch.uint8, device="cuda")
    s = Step(tsd, B, K, vocab, True, 0)
    s.scores.copy_(dev_f32(np.where(np.arange(K) == 0, 0.0, -np.inf) * np.ones((B, 1))))

    def write(pools, tab, tokens, m):
        """Appends tokens [n, m] at the rows' ends."""
        kv = (m * h_kv * d, d, h_kv * d)
        append(None, 0, 0, 0, kd[tokens], vd[tokens], *kv, None, None, *pools, *more, tab, lens, None, None, 0, 0,
               tsd.ATTN_ROPE_NONE, n, h, h_kv, m, d, n_pages, page, max_pages)

    def attend(pools, tab, tokens):
        out = torch.empty(n, h, 1, d, dtype=torch.bfloat16, device="cuda")
        decode(qd[tokens].view(n, h, 1, d).contiguous(), *pools, *more, out, tab, lens, None, n, h, h_kv, 1, d, n_pages, page,
               max_pages, tsd.ATTN_MASK_CAUSAL, 0.0, dws, dsb)
        return out

    def reserve(m):
        lens.add_(m)
        tsd.attn_cache_reserve(table, counts, lens, None, copies, n_copies, n_missing, n, m, n_pages, page, max_pages, ws, wsb)
        run = tsd.attn_cache_copy_q4 if q4 else tsd.attn_cache_copy
        run(*mine, copies, n_copies, n, 1, 0, h_kv, d, n_pages, page)

    # prompts into every sentence's first row, the other beams share it
    prompts = torch.from_numpy(np.repeat(rng.integers(1, vocab, (B, prompt)), K, 0)).cuda()
    reserve(prompt)
    write(mine, table, prompts, prompt)
    write(plain, own_table, prompts, prompt)
    first = to_dev_i32(np.arange(n) // K * K)
    tsd.attn_cache_fork(table, None, counts, first, n, n_pages, max_pages)
    assert int((counts > 0).sum()) == B
    history = prompts
    token = prompts[:, -1]
    moved = 0
    for step in range(steps):
        got = attend(mine, table, token)
        ref = attend(plain, own_table, token)
        assert torch.equal(got, ref), step  # the same rows, split in the same way
        x = got.float().view(n, h * d) @ wd
        s.x.copy_(x.view(-1))
        s.lengths.copy_(to_dev_i32(np.full(B, step + 1)))
        want = pu.select(x.double().cpu().numpy().reshape(B, K, vocab), s.scores.cpu().numpy(), s.lengths.cpu().numpy(), 0, 0.6,
                         [t.cpu().numpy() for t in s.ended])
        s.run()
        if not want[4]:
            assert np.array_equal(s.tokens.cpu().numpy(), want[0]) and np.array_equal(s.parents.cpu().numpy(), want[1])
            assert np.array_equal(s.ended[1].cpu().numpy(), want[3][1])
        s.scores.copy_(s.new_scores)
        token = s.tokens.view(-1).long()
        parents = s.parents.view(-1)
        history = torch.cat([history[parents.long()], token[:, None]], 1)
        tsd.attn_cache_fork(table, lens, counts, parents, n, n_pages, max_pages)
        reserve(1)
        assert int(n_missing) == 0
        moved += int(n_copies)
        write(mine, table, token[:, None], 1)
        write(plain, own_table, history, history.shape[1])
        t = table.cpu().numpy()
        assert np.array_equal(counts.cpu().numpy(), np.bincount(t[t >= 0], minlength=n_pages))
    assert moved > 0
    # fewer pages than hypotheses stored by themselves would take
    assert int((counts > 0).sum()) < n * -(-(prompt + steps) // page)
    # compacted, the cache attends the same
    used = int((counts > 0).sum())
    moves, n_used = to_dev_i32(np.zeros((n_pages, 3))), to_dev_i32([0])
    tsd.attn_cache_compact(table, counts, table, counts, moves, n_copies, n_used, n, n_pages, page, max_pages, n_pages, ws, wsb)
    (tsd.attn_cache_copy_q4 if q4 else tsd.attn_cache_copy)(*mine, moves, n_copies, n_pages, 1, 0, h_kv, d, n_pages, page)
    assert int(n_used) == used and int(table.max()) == used - 1
    assert torch.equal(attend(mine, table, token), attend(plain, own_table, token))
    # speculated tokens taken back, then everything
    tsd.attn_cache_release(table, counts, lens - 20, n, n_pages, page, max_pages)
    t = table.cpu().numpy()
    assert np.array_equal(counts.cpu().numpy(), np.bincount(t[t >= 0], minlength=n_pages))
    assert ((t >= 0).sum(1) == -(-(prompt + steps - 20) // page)).all()
    tsd.attn_cache_release(table, counts, None, n, n_pages, page, max_pages)
    assert (counts == 0).all() and (table == -1).all()
    assert tsd.attn_get_device_status() == tsd.ATTN_OK
