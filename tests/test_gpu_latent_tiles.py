"""How the absorbed form (klt_latent_attend) lays out its work: row tiles of a sequence one by one, and
two side by side, in batches that the rule for them takes for what they are and in others; groups of
their own for every item, and equal shares of all tiles."""
import pytest
import torch

import latent_util as U
from latent_moe_layer_route_gb300 import binding as B_
from test_gpu_latent import _lib, layer, randn, run_attend  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,counts", [
    (64, [2] + [1] * 31),               # one sequence has a second tile
    (64, [4, 1, 1, 2] * 8),             # two queries on average: alike by count alone
    (64, [2] * 32), (64, [3] * 12), (72, [1] * 32), (72, [2, 0] * 16), (192, [1] * 32),
    (100, [1, 2, 1] * 10), (128, [1, 3, 0, 2] * 8), (256, [1] * 20), (40, [4, 2, 3] * 6)])
@pytest.mark.parametrize("many", [1, 4])
def test_row_tiles_of_a_sequence(heads, counts, many):
    counts = counts * many  # fewer items than CTAs, and more
    lens = [(67 * i) % 401 for i in range(len(counts))]
    run_attend(heads, lens, counts, seed=len(counts), rope=32)


def spread(kind, B):
    """Lengths of B sequences."""
    return {"alike": [640] * B, "short": [(41 * i) % 130 for i in range(B)],
            "ragged": [(977 * i) % 1300 for i in range(B)],
            "one long": [9000] + [(67 * i) % 300 for i in range(B - 1)],
            "last long": [(67 * i) % 300 for i in range(B - 1)] + [9000]}[kind]


@pytest.mark.parametrize("kind", ["alike", "short", "ragged", "one long", "last long"])
@pytest.mark.parametrize("heads,B", [(6, 22), (6, 60), (6, 110), (6, 151), (130, 10), (130, 37),
                                     (128, 11), (128, 40), (128, 75), (128, 400), (6, 400)])
def test_shares_of_the_work(heads, B, kind):
    """Groups of their own for every item, or equal shares of all tiles, as the lengths have it."""
    run_attend(heads, spread(kind, B), [1] * B, seed=B, rope=16)


@pytest.mark.parametrize("heads,B", [(6, 110), (128, 40), (6, 15)])
def test_shares_change_between_replays(heads, B):
    """One graph for lengths of every kind: what the second kernel joins follows them."""
    at, most = layer(heads, rope=16), 9000
    cache, page_ids = randn(1, 150, 64, 144).cuda(), torch.arange(141, dtype=torch.int32)
    table = torch.stack([(page_ids + 7 * b) % 150 for b in range(B)])
    rows = [cache.cpu()[table[b].long()].flatten(0, 1) for b in range(B)]
    q, lens = randn(2, B, heads, 144), torch.zeros(B, dtype=torch.int32, device="cuda")
    args = [q.cuda(), cache, table.cuda(), lens]
    at.attend(*args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = at.attend(*args)
    for kind in ("alike", "one long", "short", "ragged", "last long", "alike"):
        have = spread(kind, B)
        assert max(have) <= most
        lens.copy_(torch.tensor(have, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        want, wl, ob, lb = U.attend(q, [r[:n] for r, n in zip(rows, have)],
                                    [(b, b + 1) for b in range(B)], 128, 144 ** -0.5)
        U.check(lse, wl, lb, f"lse {kind}")
        U.check(out, want, ob, f"out {kind}")
    assert at.status() == B_.KLT_OK
