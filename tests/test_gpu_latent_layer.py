"""Latent attention: calls without tokens or keys."""
import math

import pytest
import torch

from latent_moe_layer_route_gb300 import binding as B
from test_gpu_latent import _lib, layer, randn  # noqa: F401

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


# ---------------------------------------------------------------- nothing to do

def test_no_tokens_and_no_keys():
    at = layer(5, 128, 32)
    q = torch.empty(0, 5, 160, dtype=torch.bfloat16, device="cuda")
    cache = randn(1, 3, 64, 160).cuda()
    out, lse = at.attend(q, cache, i32([[0], [1]]), i32([5, 6]), i32([0, 0, 0]))
    assert out.shape == (0, 5, 128) and lse.shape == (0, 5)
    before = cache.clone()
    rows, turned = at.append(torch.empty(0, 160, dtype=torch.bfloat16, device="cuda"),
                             torch.empty(0, dtype=torch.int64, device="cuda"),
                             torch.empty(0, dtype=torch.int64, device="cuda"), cache,
                             q=torch.empty(0, 5, 32, dtype=torch.bfloat16, device="cuda"))
    assert rows is None and turned.shape == (0, 5, 32) and torch.equal(cache, before)
    empty = torch.empty(0, 5, 128, dtype=torch.bfloat16, device="cuda")
    kr = torch.empty(0, 32, dtype=torch.bfloat16, device="cuda")
    for causal in (True, False):
        out, lse = at.prefill(randn(2, 3, 5, 160).cuda(), empty, empty, kr, i32([0, 1, 3]),
                              i32([0, 0, 0]), causal=causal)
        assert bool((out == 0).all()) and bool((lse == -math.inf).all())
    assert at.status() == B.KLT_OK
