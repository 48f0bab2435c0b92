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


def test_addresses_of_everything_that_the_binding_takes():
    """Tensors, arrays and plain addresses; a plain address costs no more than a tensor's (each
    call converts up to ten)."""
    import timeit

    import numpy as np
    import torch
    tensor, array = torch.zeros(4), np.zeros(4)
    assert tsd._ptr(None) is None and tsd._ptr(FAKE) == FAKE
    assert tsd._ptr(tensor) == tensor.data_ptr() and tsd._ptr(array) == array.ctypes.data
    cost = lambda x: min(timeit.repeat(lambda: tsd._ptr(x), number=20000, repeat=7))
    assert cost(FAKE) <= cost(tensor)
