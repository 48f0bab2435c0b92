"""The calls that keep a paged cache's pages, and the beam selection, refuse invalid arguments on
the host before any launch (CPU only; nothing here reaches the CUDA runtime)."""
import pytest

import transformer_scaled_dot_gb300 as tsd
from transformer_scaled_dot_gb300 import build as native_build

FAKE = 1 << 20  # 16-byte aligned, never dereferenced
OK, INVALID, UNSUPPORTED = tsd.ATTN_OK, tsd.ATTN_ERR_INVALID, tsd.ATTN_ERR_UNSUPPORTED

FORK = dict(table=FAKE, lens=None, counts=FAKE, parents=FAKE, B=2, n_pages=9, max_pages=4, stream=None)
RELEASE = dict(table=FAKE, counts=FAKE, keep=None, B=2, n_pages=9, page_size=16, max_pages=4, stream=None)
RESERVE = dict(table=FAKE, counts=FAKE, lens=FAKE, new=None, copies=FAKE, n_copies=FAKE, n_missing=FAKE, B=2, n_new=1,
               n_pages=9, page_size=16, max_pages=4, ws=FAKE, ws_bytes=1 << 20, stream=None)
COMPACT = dict(table=FAKE, counts=FAKE, table_out=FAKE, counts_out=FAKE, copies=FAKE, n_copies=FAKE, n_used=FAKE, B=2,
               n_pages=9, page_size=16, max_pages=4, max_copies=4, ws=FAKE, ws_bytes=1 << 20, stream=None)
COPY = dict(k=FAKE, v=FAKE, copies=FAKE, n_copies=None, max_copies=3, n_layers=2, layer_rows=9 * 2 * 16, h_kv=2, d=64,
            n_pages=9, page_size=16, stream=None)
COPY_Q4 = dict(k=FAKE, k_scales=FAKE, v=FAKE, v_scales=FAKE, **{k: v for k, v in COPY.items() if k not in ("k", "v")})
BEAM = dict(logits=FAKE, row_stride=100, scores=FAKE, lengths=FAKE, B=2, beams=4, vocab=100, end=2, alpha=0.6, tokens=FAKE,
            parents=FAKE, new_scores=FAKE, ended_scores=FAKE, ended_rows=FAKE, ended_lengths=FAKE, ws=FAKE,
            ws_bytes=1 << 20, stream=None)
CALLS = {"attn_cache_fork": FORK, "attn_cache_release": RELEASE, "attn_cache_reserve": RESERVE,
         "attn_cache_compact": COMPACT, "attn_cache_copy": COPY, "attn_cache_copy_q4": COPY_Q4, "beam_select": BEAM,
         "beam_select_f32": BEAM}

TABLES = [
    (dict(B=-1), INVALID), (dict(B=65536), INVALID), (dict(n_pages=0), INVALID), (dict(max_pages=0), INVALID),
    (dict(n_pages=(1 << 30) + 1), UNSUPPORTED), (dict(max_pages=(1 << 26) + 1), UNSUPPORTED),
    (dict(table=None), INVALID), (dict(table=FAKE + 2), INVALID), (dict(counts=None), INVALID),
    (dict(counts=FAKE + 1), INVALID),
]
SIZED = [(dict(page_size=0), INVALID), (dict(page_size=48), INVALID), (dict(page_size=8), UNSUPPORTED),
         (dict(page_size=512), UNSUPPORTED)]
REFUSED = {
    "attn_cache_fork": TABLES + [(dict(parents=None), INVALID), (dict(parents=FAKE + 2), INVALID),
                                 (dict(lens=FAKE + 2), INVALID), (dict(B=32769), UNSUPPORTED), (dict(B=0), OK)],
    "attn_cache_release": TABLES + SIZED + [(dict(keep=FAKE + 2), INVALID), (dict(B=0), OK)],
    "attn_cache_reserve": TABLES + SIZED + [
        (dict(lens=None), INVALID), (dict(lens=FAKE + 2), INVALID), (dict(new=FAKE + 1), INVALID), (dict(n_new=-1), INVALID),
        (dict(copies=None), INVALID), (dict(n_copies=None), INVALID), (dict(n_missing=None), INVALID),
        (dict(copies=FAKE + 2), INVALID), (dict(ws=None), INVALID), (dict(ws=FAKE + 8), INVALID), (dict(ws_bytes=71), INVALID),
        (dict(B=0), OK)],
    "attn_cache_compact": TABLES + SIZED + [
        (dict(max_copies=-1), INVALID), (dict(table_out=None), INVALID), (dict(counts_out=None), INVALID),
        (dict(copies=None), INVALID), (dict(n_copies=FAKE + 2), INVALID), (dict(n_used=None), INVALID), (dict(ws=None), INVALID),
        (dict(ws_bytes=71), INVALID)],
    "attn_cache_copy": [
        (dict(k=None), INVALID), (dict(v=FAKE + 8), INVALID), (dict(copies=None), INVALID), (dict(copies=FAKE + 2), INVALID),
        (dict(n_copies=FAKE + 1), INVALID), (dict(max_copies=-1), INVALID), (dict(n_layers=-1), INVALID),
        (dict(n_layers=65536), INVALID), (dict(layer_rows=9 * 2 * 16 - 16), INVALID), (dict(layer_rows=9 * 2 * 16 + 8), INVALID),
        (dict(layer_rows=1 << 60), INVALID), (dict(h_kv=0), INVALID), (dict(d=96), UNSUPPORTED), (dict(n_pages=0), INVALID),
        (dict(page_size=48), INVALID), (dict(page_size=8), UNSUPPORTED),
        (dict(h_kv=32768, page_size=256, d=128), UNSUPPORTED),  # pages of 2 GB
        (dict(max_copies=0), OK), (dict(n_layers=0), OK), (dict(n_layers=1, layer_rows=0, max_copies=0), OK)],
    "beam_select": [
        (dict(B=-1), INVALID), (dict(beams=0), INVALID), (dict(beams=17), UNSUPPORTED), (dict(vocab=0), INVALID),
        (dict(vocab=(1 << 20) + 1, row_stride=1 << 21), UNSUPPORTED), (dict(B=1 << 29), UNSUPPORTED),
        (dict(B=1 << 20, beams=16, vocab=1 << 20, row_stride=1 << 20), UNSUPPORTED), (dict(row_stride=99), INVALID),
        (dict(row_stride=1 << 60), INVALID), (dict(end=-2), INVALID), (dict(alpha=float("nan")), INVALID),
        (dict(alpha=float("inf")), INVALID), (dict(logits=None), INVALID), (dict(logits=FAKE + 1), INVALID),
        (dict(scores=None), INVALID), (dict(scores=FAKE + 2), INVALID), (dict(tokens=None), INVALID), (dict(parents=None), INVALID),
        (dict(new_scores=None), INVALID), (dict(lengths=None), INVALID), (dict(ended_scores=None), INVALID),
        (dict(ended_rows=FAKE + 2), INVALID), (dict(ended_lengths=None), INVALID), (dict(ws=None), INVALID),
        (dict(ws=FAKE + 8), INVALID), (dict(ws_bytes=63), INVALID), (dict(B=0), OK),
        (dict(B=0, end=-1, lengths=None, ended_scores=None, ended_rows=None, ended_lengths=None), OK)],
}
REFUSED["attn_cache_copy_q4"] = REFUSED["attn_cache_copy"] + [(dict(k_scales=None), INVALID), (dict(v_scales=FAKE + 4), INVALID)]
REFUSED["beam_select_f32"] = REFUSED["beam_select"] + [(dict(logits=FAKE + 2), INVALID)]


@pytest.fixture(scope="module")
def lib():
    native_build.build()
    return tsd.library()


@pytest.mark.parametrize("name", CALLS)
def test_refusals(lib, name):
    for change, status in REFUSED[name]:
        assert set(change) <= set(CALLS[name])
        args = {**CALLS[name], **change}
        assert getattr(lib, name)(*args.values()) == status, (name, change)


def test_workspace_sizes(lib):
    assert tsd.attn_cache_pages_workspace_bytes(2, 9) >= 72
    assert tsd.attn_cache_pages_workspace_bytes(65535, 1 << 30) >= 1 << 33
    for bad in ((-1, 9), (65536, 9), (2, 0), (2, (1 << 30) + 1)):
        assert tsd.attn_cache_pages_workspace_bytes(*bad) == 0
    assert tsd.beam_select_workspace_bytes(2, 4, 1025) >= 2 * 4 * 2 * 8
    for bad in ((-1, 4, 100), (2, 0, 100), (2, 17, 100), (2, 4, 0), (2, 4, (1 << 20) + 1), (1 << 20, 16, 1 << 20)):
        assert tsd.beam_select_workspace_bytes(*bad) == 0


def test_status_string(lib):
    assert tsd.attn_status_string(tsd.ATTN_ERR_DEVICE_VALUE) == "ATTN_ERR_DEVICE_VALUE"


def test_binding_raises(lib):
    with pytest.raises(tsd.AttnError):
        tsd.attn_cache_fork(None, None, None, None, 1, 1, 1, stream=0)
    with pytest.raises(tsd.AttnError):
        tsd.beam_select(None, 10, None, None, 1, 1, 10, -1, 0.0, None, None, None, stream=0)
