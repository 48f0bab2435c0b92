"""What the paged cache's binding and entry points take on the host (CPU only;
nothing here reaches the CUDA runtime)."""
import pytest

import transformer_scaled_dot_gb300 as tsd

from test_paged_abi import APPEND, APPEND_Q4, FAKE, OK, lib  # noqa: F401 (lib: a fixture)


@pytest.mark.parametrize("name,call", [("attn_cache_append", APPEND), ("attn_cache_append_q4", APPEND_Q4)])
def test_without_a_rotation_its_arguments_are_ignored(lib, name, call):
    for rope, rows, dim in ((None, 0, 0), (FAKE + 4, -1, 33), (FAKE, 5, 1000)):
        change = dict(B=0, rope=rope, rope_rows=rows, rope_dim=dim, rope_kind=tsd.ATTN_ROPE_NONE)
        assert getattr(lib, name)(*{**call, **change}.values()) == OK
