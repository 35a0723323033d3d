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


def test_copies_into_the_workspace_of_rows_quantised_once(L):
    """3 rows of 64: 36 bytes each in the workspace, 9 copies of 32 bytes of codes, one scale tile."""
    def call(codes, scales, rows=9):
        return L.moe_mx_quantize_once(0, P >> 4, 0, 64, 3, 64, P >> 4, rows, 0, codes, scales, P, 3 * 36, None)

    far = P + (1 << 16)
    for codes, scales in ((P, far), (P + 96, far), (P - 272, far), (far, P), (far, P + 96), (far, P - 496)):
        assert call(codes, scales) == B.MOE_ERR_INVALID_ARG, (codes, scales)
        assert b"overlap" in L.moe_last_error()
    assert call(P, P, rows=0) == B.MOE_OK
