"""The expanded form's pairs of CTAs (klt_latent_prefill): what one of them hands to the other."""
import math

import pytest
import torch

import latent_util as U
from latent_moe_layer_route_gb300 import binding as B
from test_gpu_latent import NAN, _lib, layer, randn, starts  # noqa: F401

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


@pytest.mark.parametrize("bad", [NAN, math.inf])
@pytest.mark.parametrize("value", [64, 128])
def test_values_behind_a_sequence_have_no_effect(value, bad):
    """Behind every second sequence lies one that is not finite: it is cleared in the memory of both
    CTAs, half of its columns each, before the products of either read it."""
    keys = [1, 40, 130, 7, 255, 60, 127, 3, 129, 90, 383, 130, 520, 9, 65, 200]
    heads, cu = 24, starts(keys)
    at = layer(heads, 128, 16, 64, value)
    q, kv, kr = (randn(s, cu[-1], *n) for s, n in ((1, (heads, 80)), (2, (heads, 64 + value)),
                                                   (3, (16,))))
    keep = torch.cat([torch.arange(cu[b], cu[b + 1]) for b in range(0, len(keys), 2)])
    want, wl, ob, lb = U.prefill(q, kv[..., :64], kv[..., 64:], kr, cu, cu, 80 ** -0.5, True)
    g, gr = kv.cuda(), kr.cuda()
    for b in range(1, len(keys), 2):
        g[cu[b]:cu[b + 1]], gr[cu[b]:cu[b + 1]] = bad, bad
    args = [q.cuda(), g[..., :64], g[..., 64:], gr, i32(cu), i32(cu)]
    first = [t[keep.cuda()] for t in at.prefill(*args)]
    U.check(first[1], wl[keep], lb[keep], "lse")
    U.check(first[0], want[keep], ob[keep], "out")
    for _ in range(20):
        got = at.prefill(*args)
        assert all(torch.equal(t[keep.cuda()], f) for t, f in zip(got, first))
    assert at.status() == B.KLT_OK


def gives_up(queries, keys, heads, stall):
    """A launch whose copies stop after `stall` tiles, and others right behind it."""
    cu_q, cu_k = starts(queries), starts(keys)

    def operands(seed):
        kv = randn(seed, cu_k[-1], heads, 128).cuda()
        return [randn(seed + 1, cu_q[-1], heads, 80).cuda(), kv[..., :64], kv[..., 64:],
                randn(seed + 2, cu_k[-1], 16).cuda(), i32(cu_q), i32(cu_k)]

    bad, ok = (layer(heads, 128, 16, 64, 64) for _ in range(2))
    lost, args = operands(1), operands(4)
    want = [t.clone() for t in ok.prefill(*args)]
    torch.cuda.synchronize()
    bad.prefill(*lost, debug=B.KltLatentDebug(stall_after_tiles=stall, timeout_ms=5))
    got = [ok.prefill(*args) for _ in range(3)]
    torch.cuda.synchronize()
    assert bad.status() == B.KLT_ERR_DEVICE_TIMEOUT
    assert ok.status() == B.KLT_OK
    for g in got:
        assert all(torch.equal(x, y) for x, y in zip(g, want))
    bad.close()


@pytest.mark.parametrize("stall", [1, 2, 3, 4, 5, 6])
def test_waits_that_run_out_at_different_places(stall):
    """The second CTA's copies stop a tile behind the first one's, within a unit, at its ragged last
    tile (whose values are signalled to each CTA alone) or with the next unit's queries: all have
    landed when the pair ends, so nothing is left to the launches right behind it."""
    gives_up([40, 300, 129, 400], [130, 300, 257, 100], 90, stall)


@pytest.mark.parametrize("stall", [1, 2, 3])
def test_waits_that_run_out_between_units(stall):
    """Units of one tile of keys: a pair gives up while its CTAs ask for the next one, and one of them
    may not know that an answer is on its way."""
    gives_up([20, 100, 256, 60], [20, 128, 100, 90], 130, stall)
