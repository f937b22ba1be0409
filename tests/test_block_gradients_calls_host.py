"""Calls of the operators that train what stands around the experts that are refused on the host for more than one
argument's sake."""
import ctypes

import pytest

from test_block_gradients_host import check, combine, m  # noqa: F401

VP = ctypes.c_void_p
# combine(): T = 4, K = 64, topk = 4: grad_out 512 bytes at 0x10000, routes 2048 at 0x20000, ids 64 at 0x30000,
# weights 64 at 0x40000


@pytest.mark.parametrize("kw,code", [
    (dict(do=VP(0x20000)), "ARG"), (dict(do=VP(0x20000 + 2032)), "ARG"), (dict(do=VP(0x20000 - 2032)), "ARG"),
    (dict(do=VP(0x10000)), "ARG"), (dict(do=VP(0x10000 + 496)), "ARG"), (dict(do=VP(0x30000 - 16)), "ARG"),
    (dict(do=VP(0x40000)), "ARG"), (dict(dw=VP(0x40000)), "ARG"), (dict(dw=VP(0x40000 + 60)), "ARG"),
    (dict(dw=VP(0x30000 - 60)), "ARG"), (dict(dw=VP(0x10000 + 508)), "ARG"), (dict(dw=VP(0x20000 + 1024)), "ARG"),
    (dict(dw=VP(0x20000 + 1024), do=None), "ARG"), (dict(dw=VP(0x30000), ids=None, T=0), "OK"),
])
def test_combination_outputs_over_inputs_are_refused(m, kw, code):
    check(m, combine(m, **kw), code)
