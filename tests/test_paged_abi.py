"""The paged cache's entry points refuse invalid arguments on the host before
any launch (CPU only; nothing here reaches the CUDA runtime)."""
import numpy as np
import pytest

import transformer_scaled_dot_gb300 as tsd
from transformer_scaled_dot_gb300 import build as native_build

import paged_util as pu

FAKE = 1 << 20  # 16-byte aligned, never dereferenced
OK, INVALID, UNSUPPORTED = tsd.ATTN_OK, tsd.ATTN_ERR_INVALID, tsd.ATTN_ERR_UNSUPPORTED

SIZES = dict(B=2, h=8, h_kv=2, n=1, d=64, n_pages=9, page_size=16, max_pages=4)
APPEND = dict(q=FAKE, q_sb=512, q_sh=64, q_sr=512, k=FAKE, v=FAKE, kv_sb=128, kv_sh=64, kv_sr=128,
              q_out=FAKE, k_out=None, k_cache=FAKE, v_cache=FAKE, table=FAKE, lens=FAKE, new=None,
              rope=FAKE, rope_rows=64, rope_dim=64, rope_kind=1, **SIZES, stream=None)
APPEND_Q4 = {}
for _k, _v in APPEND.items():
    APPEND_Q4[_k] = _v
    if _k == "k_cache":
        APPEND_Q4["k_scales"] = FAKE
    if _k == "v_cache":
        APPEND_Q4 |= {"v_scales": FAKE, "k_factor": 1.0, "v_factor": 1.0}
DECODE = dict(q=FAKE, k_cache=FAKE, v_cache=FAKE, out=FAKE, table=FAKE, lens=FAKE, new=None, **SIZES,
              mask=1, scale=0.0, ws=FAKE, ws_bytes=1 << 40, stream=None)
DECODE_Q4 = dict(q=FAKE, k_cache=FAKE, k_scales=FAKE, v_cache=FAKE, v_scales=FAKE, k_factor=1.0,
                 v_factor=1.0, out=FAKE, table=FAKE, lens=FAKE, new=None, **SIZES, mask=1, scale=0.0,
                 ws=FAKE, ws_bytes=1 << 40, stream=None)
CALLS = {"attn_cache_append": APPEND, "attn_cache_append_q4": APPEND_Q4,
         "attn_decode_paged": DECODE, "attn_decode_paged_q4": DECODE_Q4}

COMMON = [
    (dict(B=-1), INVALID), (dict(B=65536), INVALID), (dict(h=-8), INVALID),
    (dict(h_kv=0), INVALID), (dict(h_kv=3), INVALID),            # 8 heads over 3
    (dict(h=65536, h_kv=65536), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(d=256), UNSUPPORTED),
    (dict(n_pages=0), INVALID), (dict(max_pages=0), INVALID), (dict(page_size=0), INVALID),
    (dict(page_size=24), INVALID),                               # not a power of two
    (dict(page_size=8), UNSUPPORTED), (dict(page_size=512), UNSUPPORTED),
    (dict(max_pages=(1 << 26) + 1), UNSUPPORTED),                # more than 2^30 rows
    (dict(n_pages=(1 << 31) - 1, page_size=256, max_pages=1), UNSUPPORTED),  # 2^40 rows in the pool
    (dict(table=None), INVALID), (dict(table=FAKE + 2), INVALID), (dict(lens=FAKE + 1), INVALID),
    (dict(new=FAKE + 2), INVALID), (dict(q=FAKE + 8), INVALID),
    (dict(k_cache=None), INVALID), (dict(v_cache=None), INVALID), (dict(k_cache=FAKE + 4), INVALID),
    (dict(B=0), OK),
]
ONLY_APPEND = [
    (dict(n=-1), INVALID), (dict(n=0), OK), (dict(lens=None), INVALID),
    (dict(q=None), INVALID), (dict(q_out=None), INVALID),        # one without the other
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(v=FAKE + 8), INVALID),
    (dict(q_sh=60), INVALID), (dict(kv_sr=-64), INVALID), (dict(kv_sb=4), INVALID),
    (dict(rope_kind=3), INVALID), (dict(rope_kind=-1), INVALID), (dict(rope=None), INVALID),
    (dict(rope=FAKE + 4), INVALID), (dict(rope_rows=0), INVALID), (dict(rope_dim=0), INVALID),
    (dict(rope_dim=128), INVALID), (dict(rope_dim=33), INVALID), (dict(rope_dim=48), UNSUPPORTED),
    (dict(k_out=FAKE + 2), INVALID), (dict(B=40000, n=60000), INVALID),
]
ONLY_DECODE = [
    (dict(B=65535, h=65528, h_kv=8), INVALID),                   # 2^32 rows of queries
    (dict(B=60000, h=4096, h_kv=4096, page_size=256, max_pages=1 << 22), UNSUPPORTED),  # 2^52 units
    (dict(n=0), INVALID), (dict(n=9), UNSUPPORTED), (dict(q=None), INVALID), (dict(out=None), INVALID),
    (dict(out=FAKE + 2), INVALID), (dict(mask=2), INVALID), (dict(mask=4), INVALID),
    (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(ws=None), INVALID),
    (dict(ws=FAKE + 8), INVALID), (dict(ws_bytes=0), INVALID), (dict(h=0), OK),
    (dict(scale=3e38), INVALID),                                 # times log2(e): infinite
    (dict(scale=2e38, h=0), OK),
]
ONLY_Q4 = [
    (dict(k_scales=None), INVALID), (dict(v_scales=FAKE + 2), INVALID), (dict(k_factor=0.0), INVALID),
    (dict(v_factor=-1.0), INVALID), (dict(v_factor=float("inf")), INVALID),
    (dict(k_factor=float("nan")), INVALID), (dict(k_factor=1e-38), INVALID),
]
ONLY_DECODE_Q4 = [
    (dict(scale=1e10, k_factor=2.0 ** 100), INVALID),            # their product is infinite
    (dict(scale=1e8, k_factor=2.0 ** 100, h=0), OK),
]
CASES = [(name, change, expect) for name in CALLS
         for change, expect in COMMON + (ONLY_APPEND if "append" in name else ONLY_DECODE) +
         (ONLY_Q4 if "q4" in name else []) +
         (ONLY_DECODE_Q4 if name == "attn_decode_paged_q4" else [])]


@pytest.fixture(scope="module")
def lib():
    native_build.build()
    return tsd.library()


@pytest.mark.parametrize("name,change,expect", CASES, ids=lambda x: str(x).replace(" ", ""))
def test_paged_calls_refuse_bad_arguments(lib, name, change, expect):
    assert set(change) <= set(CALLS[name])
    assert getattr(lib, name)(*{**CALLS[name], **change}.values()) == expect


def test_paged_workspace_bytes(lib):
    f = tsd.attn_decode_paged_workspace_bytes
    assert f(2, 8, 2, 1, 64, 16, 4) > 0
    assert f(1, 8, 8, 8, 128, 256, 1 << 22) > 0
    for bad in ((-1, 8, 2, 1, 64, 16, 4), (2, 8, 3, 1, 64, 16, 4), (2, 8, 2, 0, 64, 16, 4),
                (2, 8, 2, 9, 64, 16, 4), (2, 8, 2, 1, 96, 16, 4), (2, 8, 2, 1, 64, 17, 4),
                (2, 8, 2, 1, 64, 16, 0)):
        assert f(*bad) == 0
    # a call with the bytes that the query names passes the check, one byte fewer does not
    need = f(2, 8, 2, 1, 64, 16, 4)
    assert lib.attn_decode_paged(*{**DECODE, "ws_bytes": need - 1}.values()) == INVALID


def test_device_index_status_string(lib):
    assert tsd.attn_status_string(tsd.ATTN_ERR_DEVICE_INDEX) == "ATTN_ERR_DEVICE_INDEX"


# ------------------------------------------------------------ the plain forms' own pins
def test_plain_code_tables():
    assert np.array_equal(pu.code_values(np.array([0x21, 0xf9], dtype=np.uint8)), [0.5, 1, -0.5, -6])
    assert pu.E4M3[0x38] == 1.0 and pu.E4M3[0x7e] == 448.0 and pu.E4M3[1] == 2.0 ** -9
    assert pu.E4M3[0xb8] == -1.0 and np.isnan(pu.E4M3[0x7f])


def test_plain_rotation_keeps_lengths_and_depends_on_distance_only():
    rng = np.random.default_rng(0)
    rope = pu.rope_table(300, 64)
    for kind in (pu.HALVES, pu.PAIRS):
        q, k = rng.standard_normal(64), rng.standard_normal(64)
        f = lambda x, p: pu.rotate(x, p, rope, kind, 64)
        # the table's fp32 cosines and sines leave a relative error of 2^-24 each
        assert abs(np.linalg.norm(f(q, 250)) - np.linalg.norm(q)) < 1e-6
        assert abs(f(q, 30) @ f(k, 10) - f(q, 220) @ f(k, 200)) < 1e-5
        assert np.array_equal(f(q, 0), q)


def test_plain_decode_of_equal_keys_is_the_mean_of_the_seen_rows():
    v = np.arange(10.0).reshape(1, 5, 2)
    out, _, _ = pu.decode(np.ones((1, 1, 2, 2)), [np.ones((1, 5, 2))], [v], [5], [2], True, 1.0)
    assert np.allclose(out[0, 0, 1], v[0].mean(0)) and np.allclose(out[0, 0, 0], v[0, :4].mean(0))
