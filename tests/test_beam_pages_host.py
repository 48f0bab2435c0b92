"""What the host decides about a beam selection and the cache's pages, and what their sources keep to (CPU only)."""
import os
import re

import pytest

import transformer_scaled_dot_gb300 as tsd
from test_cache_pages_abi import BEAM, RESERVE, lib  # noqa: F401 (the fixture)

CSRC = os.path.join(os.path.dirname(os.path.abspath(tsd.__file__)), "csrc")


@pytest.mark.parametrize("name", ["beam_select.cu", "cache_pages.cu", "cache_copy.cu", "cache_append.cu", "attn_paged.cu"])
def test_no_loads_through_the_read_only_path(name):
    """These kernels begin while the launch before them, which may write what they read (beam_select the parents,
    fork the lengths), still runs. The read-only path is for memory that nobody writes in a kernel's life: neither
    its loads nor pointers that allow the compiler to use them."""
    with open(os.path.join(CSRC, name), encoding="utf-8") as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert "griddep_wait" in code
    assert not re.search(r"\b__ldg\b|ld\.global(\.\w+)*\.nc|\b__restrict__\b", code)


@pytest.mark.parametrize("name", ["beam_select", "beam_select_f32"])
def test_alpha_is_ignored_without_an_end_token(lib, name):  # noqa: F811
    for alpha in (float("nan"), float("inf"), -float("inf"), 1e300):
        args = {**BEAM, "B": 0, "end": -1, "alpha": alpha}
        assert getattr(lib, name)(*args.values()) == tsd.ATTN_OK, alpha
        assert getattr(lib, name)(*{**args, "end": 2}.values()) == tsd.ATTN_ERR_INVALID, alpha


def test_reserve_refuses_more_places_than_it_has_numbers_for(lib):  # noqa: F811
    """2^31 of them, of which each names itself where several name one page."""
    sizes = {**RESERVE, "n_pages": 1 << 20, "ws_bytes": 1 << 24}
    for B, max_pages, n_new in ((65535, 1 << 16, 1 << 20), (65535, 32769, 2 ** 31 - 1), (32769, 1 << 16, 65535 * 16 - 14),
                                (33, 1 << 26, 2 ** 31 - 1)):
        args = {**sizes, "B": B, "max_pages": max_pages, "n_new": n_new}
        assert lib.attn_cache_reserve(*args.values()) == tsd.ATTN_ERR_UNSUPPORTED, (B, max_pages, n_new)
    args = {**sizes, "B": 0, "max_pages": 1 << 26, "n_new": 2 ** 31 - 1}
    assert lib.attn_cache_reserve(*args.values()) == tsd.ATTN_OK
