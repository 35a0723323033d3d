"""Outputs that overlap inputs are refused on the host (no GPU). Only calls that are refused are made here: the
addresses are never dereferenced."""
import ctypes

import pytest

from sparse_mixture_experts_gate_b200 import binding as B
from sparse_mixture_experts_gate_b200 import build

P = 0x100000


@pytest.fixture(scope="module")
def L():
    build.build()
    return B.lib()


@pytest.mark.parametrize("dtype,es", [("fp32", 4), ("bf16", 2)])
def test_gradient_into_its_logits(L, dtype, es):
    c = B.moe_route_config_default()
    c.dtype = B.MOE_DTYPE[dtype]
    row = 8 * es

    def call(at, ld, gld, T):
        return L.moe_route_backward(ctypes.byref(c), P >> 4, P, ld, P >> 4, T, P + at, gld, None)

    for at, ld, gld, T in ((0, 8, 8, 4), (0, 8, 8, 1), (es, 8, 8, 1), (-es, 8, 8, 1), (3 * row, 8, 8, 4), (-3 * row, 8, 8, 4),
                           (7 * es, 16, 16, 3), (15 * es, 16, 16, 3), (-5 * 16 * es - es, 16, 16, 6), (8 * es, 16, 20, 3),
                           (-9 * es, 16, 9, 3), (4 * row, 8, 100, 5), (-100 * es + es, 100, 100, 2)):
        assert call(at, ld, gld, T) == B.MOE_ERR_INVALID_ARG, (at, ld, gld, T)
        assert b"overlap" in L.moe_last_error()
