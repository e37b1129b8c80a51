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


@pytest.mark.parametrize("name", ["H", "gamma_post", "gamma_pre"])
def test_block_norm_keeps_what_it_was_made_with(name):
    """A call reads the weights by the address they had at creation: other tensors are another
    layer's, and giving them to this one must not free the ones it reads."""
    layer = B.BlockNorm(256)
    before = getattr(layer, name)
    with pytest.raises(AttributeError):
        setattr(layer, name, None)
    assert getattr(layer, name) is before
