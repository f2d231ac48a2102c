"""Widths beyond the ABI's 32 bits are refused, not cut to their low bits (no GPU)."""
import pytest

from mixture_experts_layer_schedule_gb300 import _lib


@pytest.mark.parametrize("wide", [2 ** 31, 2 ** 32 + 256, -2 ** 32 + 256, 2 ** 40 + 64])
def test_widths_past_32_bits(wide):
    for call in (lambda: _lib.ffn_problem(4, wide, 128), lambda: _lib.ffn_problem(4, 128, wide),
                 lambda: _lib.fp4_problem(4, wide, 64), lambda: _lib.fp4_problem(4, 64, wide)):
        with pytest.raises(ValueError, match="outside 32 bits"):
            call()


def test_token_counts_have_64_bits():
    assert _lib.ffn_problem(2 ** 31, 128, 128).N == 2 ** 31 and _lib.fp4_problem(2 ** 33, 64, 64).M == 2 ** 33
