"""Host-side rules of the operators around the projection, without a GPU."""
import ctypes
import math

import pytest

from scatter_gemm_b200 import lora
from scatter_gemm_b200.build import build


@pytest.fixture(scope="module")
def L():
    build()
    return lora.lib()


@pytest.mark.parametrize("tok,most", [(1, 94080), (8, 11648), (9, 9472), (16, 5248)])
def test_w4_copies_rows_that_shared_memory_does_not_hold(L, tok, most):
    assert L.lora_w4_copies_x(tok, most) == 0 and L.lora_w4_copies_x(tok, most + 1) == 1
    assert L.lora_w4_copies_x(17, 1) == 1
    assert L.lora_w4_copies_x(0, 100000) == L.lora_w4_copies_x(-1, 9) == L.lora_w4_copies_x(3, 0) == 0


@pytest.mark.parametrize("which", ["k_scale", "v_scale"])
@pytest.mark.parametrize("scale,want", [(1e-39, 1), (2.0 ** -149, 1), (2.0 ** -128, 1),
                                        (2.0 ** -127, 0), (3e38, 0), (0.0, 1), (math.nan, 1)])
def test_rope_scales_need_a_finite_reciprocal(L, which, scale, want):
    # no tokens: nothing to do once the arguments are accepted
    scales = dict(k_scale=1.0, v_scale=1.0)
    scales[which] = scale
    off, st = (ctypes.c_int32 * 4)(0, 64, 128, 192), (ctypes.c_int64 * 3)(64, 64, 64)
    p = 0x10000
    got = L.lora_rope_append(p, 192, off, 64, 64, p, 0, 1, None, p, 10, 0, None, None, 0.0, 1e-6, p,
                             64, p, st, p, st, 4, 8, 0, scales["k_scale"], scales["v_scale"], p, 8,
                             0, 0, None)
    assert got == want
