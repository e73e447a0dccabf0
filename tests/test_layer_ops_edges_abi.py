"""Host-side rules of the operators around the projection, without a GPU."""
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
