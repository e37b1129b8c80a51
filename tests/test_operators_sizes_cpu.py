"""Sizes that do not fit the C ABI's 32 bits are refused by the Python layer, not cut."""
import pytest

from latent_moe_layer_route_gb300 import binding as B
from latent_moe_layer_route_gb300 import build


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


@pytest.mark.parametrize("H", [(1 << 32) + 256, 1 << 31, -1, 0, B.KLT_BLOCK_NORM_MAX_H + 1])
def test_block_norm_of_a_width_that_no_call_takes(H):
    with pytest.raises(B.KltError) as e:
        B.BlockNorm(H)
    assert e.value.code in (B.KLT_ERR_INVALID_ARG, B.KLT_ERR_UNSUPPORTED)


def test_block_norm_of_the_widest_rows():
    assert B.BlockNorm(B.KLT_BLOCK_NORM_MAX_H).H == B.KLT_BLOCK_NORM_MAX_H
