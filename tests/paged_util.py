"""Plain 64-bit forms of the paged cache's operators for the tests, written
from the definitions in the header, and the pools and tables that they use."""
import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])
# e4m3: 0x7f and 0xff are NaN, there are no infinities
E4M3 = np.array([s * (m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
                 for s in (1, -1) for e in range(16) for m in range(8)])
E4M3[0x7f] = E4M3[0xff] = np.nan

HALVES, PAIRS = 1, 2


def rope_table(rows, dim, base=10000.0):
    angle = np.arange(rows)[:, None] * base ** (-np.arange(0, dim, 2) / dim)
    return np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)


def rotate(x, position, rope, kind, dim):
    """x [.., d] in 64 bits at one position."""
    y = np.array(x, dtype=np.float64)
    if kind == 0:
        return y
    c, s = rope[position, :dim // 2].astype(np.float64), rope[position, dim // 2:].astype(np.float64)
    i, j = (slice(0, dim // 2), slice(dim // 2, dim)) if kind == HALVES else \
        (slice(0, dim, 2), slice(1, dim, 2))
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., j] * c + x[..., i] * s
    return y


def page_table(rng, lens, page_size, spare=2, extra_pages=1):
    """(table [B, max_pages] with -1 past each sequence's last page, n_pages), pages in random order."""
    used = [-(-int(max(n, 0)) // page_size) for n in lens]
    max_pages = max(max(used), 1) + extra_pages
    n_pages = sum(used) + spare
    order = rng.permutation(n_pages)
    table = np.full((len(lens), max_pages), -1, dtype=np.int32)
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = order[at:at + u]
        at += u
    return table, n_pages


def gather(pool, table, length, page_size):
    """Rows 0 .. length - 1 of one sequence: pool [n_pages, h_kv, page_size, w] -> [h_kv, length, w]."""
    pages = table[:-(-length // page_size)]
    rows = pool[pages].swapaxes(0, 1).reshape(pool.shape[1], -1, pool.shape[-1])
    return rows[:, :length]


def code_values(codes):
    """[.., w] bytes -> [.., 2 w] values of the codes in 64 bits."""
    return np.stack([E2M1[codes & 15], E2M1[codes >> 4]], -1).reshape(codes.shape[:-1] + (-1,))


def dequantise(codes, scales, factor):
    return code_values(codes) * np.repeat(E4M3[scales], 16, -1) * float(np.float32(factor))


def decode(q, k_rows, v_rows, lens, new_lens, causal, scale):
    """q [B, h, n_q, d]; k_rows, v_rows: per sequence [h_kv, L, d]. Returns the output,
    sum p |v| (what an error of the weights is relative to) with 2^-25 sum |v| added to it (below
    which a weight's error is absolute), and the largest sum |q k| scale."""
    B, h, n_q, d = q.shape
    out, mass, size = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape[:3])
    for b in range(B):
        L, m = int(lens[b]), int(new_lens[b])
        group = h // k_rows[b].shape[0]
        for t in range(m):
            n = min(L, L - m + t + 1) if causal else L
            if n <= 0:
                continue
            for i in range(h):
                k, v = k_rows[b][i // group][:n], v_rows[b][i // group][:n]
                x = k @ q[b, i, t] * scale
                w = np.exp(x - x.max())
                w /= w.sum()
                out[b, i, t] = w @ v
                mass[b, i, t] = w @ np.abs(v) + 2.0 ** -25 * np.abs(v).sum(0)
                size[b, i, t] = (np.abs(k) @ np.abs(q[b, i, t])).max() * scale
    return out, mass, size


def decode_tolerance(ref, mass, size, n, d):
    """Largest |error| of an output element. The output's rounding to bf16: 2^-8 of the value.
    The weights: rounded to 11 bits or more (2^-11 each, and their sum is taken before the
    rounding); the 4-bit cache's are numbers of f16 taken times 2^11 or more, so that
    those under 2^-25 (2^-14, the least with 11 bits, over 2^11) of the largest are off by up to
    half of f16's least step, 2^-25 / 2^11 = 2^-36 = 2^-11 2^-25; their exponents' error, twice the logit's (2 (d + 4) 2^-24 of sum |q k|, in 32
    bits), and 2^-21 of the exponential itself; sums of n terms in 32 bits, n 2^-24."""
    weights = 2.0 ** -11 + 2 * (d + 4) * 2.0 ** -24 * size[..., None] + 2.0 ** -21 + n * 2.0 ** -24
    return 2.0 ** -8 * np.abs(ref) + 1.01 * weights * mass + 1e-30
