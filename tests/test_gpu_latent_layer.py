"""Latent attention: rows that are not finite, and calls without tokens or keys."""
import math

import pytest
import torch

import latent_util as U
from latent_moe_layer_route_gb300 import binding as B
from test_gpu_latent import NAN, _lib, layer, paged, randn, starts  # noqa: F401

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


# ---------------------------------------------------------------- rows that are not finite

@pytest.mark.parametrize("bad", [NAN, math.inf])
@pytest.mark.parametrize("columns", [slice(0, 192), slice(128, 192), slice(5, 6)])
def test_queries_that_see_a_row_that_is_not_finite(bad, columns):
    """They are not finite, however little of the row is; other sequences' are as ever; queries of the
    same sequence that do not see it may be either."""
    lens, counts, at_row = [130, 90, 200], [3, 7, 2], 86  # the second sequence's 4th to 7th query
    at, cu = layer(16), starts(counts)
    cache, table, seqs = paged(21, lens, 64, 192)
    q = randn(22, cu[-1], 16, 192)
    want, wl, ob, lb = U.attend(q, seqs, list(zip(cu, cu[1:])), 128, 192 ** -0.5)
    cache[int(table[1, at_row // 64]), at_row % 64, columns] = bad
    out, lse = (t.cpu() for t in at.attend(q.cuda(), cache.cuda(), table.cuda(), i32(lens), i32(cu)))
    keep = list(range(cu[1])) + list(range(cu[2], cu[3]))
    U.check(lse[keep], wl[keep], lb[keep], "lse")
    U.check(out[keep], want[keep], ob[keep], "out")
    sees = slice(cu[1] + at_row - (lens[1] - counts[1]), cu[2])
    assert sees.stop - sees.start == 4
    # an infinite score of either sign is a weight of nan or of zero, by the query's sign
    touched = ~out[sees].isfinite().all(-1) | ~lse[sees].isfinite()
    assert bool(touched.all())


@pytest.mark.parametrize("bad", [NAN, math.inf])
@pytest.mark.parametrize("part", ["k", "v", "k_rope"])
def test_expanded_queries_that_see_a_row_that_is_not_finite(part, bad):
    lens, at_row = [100, 300, 70], 137
    cu = starts(lens)
    at = layer(3)
    q, kv, kr = randn(1, cu[-1], 3, 192), randn(2, cu[-1], 3, 256), randn(3, cu[-1], 64)
    want, wl, ob, lb = U.prefill(q, kv[..., :128], kv[..., 128:], kr, cu, cu, 192 ** -0.5, True)
    g = dict(k=kv[..., :128].cuda(), v=kv[..., 128:].cuda(), k_rope=kr.cuda())
    g[part][cu[1] + at_row] = bad
    out, lse = (t.cpu() for t in at.prefill(q.cuda(), g["k"], g["v"], g["k_rope"], i32(cu), i32(cu)))
    keep = list(range(cu[1])) + list(range(cu[2], cu[3]))
    U.check(lse[keep], wl[keep], lb[keep], "lse")
    U.check(out[keep], want[keep], ob[keep], "out")
    touched = ~out[cu[1] + at_row:cu[2]].isfinite().all(-1)
    if part == "v" or math.isnan(bad):
        assert bool(touched.all())
    else:  # the sum of a row's infinite products has either sign, or none: nan
        s = torch.einsum("thd,hd->th", q[cu[1] + at_row:cu[2], :, :128].float(),
                         g["k"][cu[1] + at_row].cpu().float()) + torch.einsum(
            "thd,d->th", q[cu[1] + at_row:cu[2], :, 128:].float(),
            g["k_rope"][cu[1] + at_row].cpu().float())
        assert bool(touched[s != -math.inf].all())


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
