"""Latent attention's calls in the layouts in which a layer chains them, a decoding step replayed from
a graph, rows that are not finite, and calls without tokens or keys."""
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


# ---------------------------------------------------------------- nothing given, nothing to do

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float64])
def test_what_is_allocated_here_whatever_the_default_type(dtype):
    at, cache = layer(4), randn(1, 3, 64, 192).cuda()
    q, kv, kr = randn(2, 2, 4, 192).cuda(), randn(3, 5, 4, 256).cuda(), randn(4, 5, 64).cuda()
    table, lens, cu_q, cu_k = i32([[0], [1]]), i32([5, 6]), i32([0, 1, 2]), i32([0, 2, 5])

    def calls():
        return (at.attend(q, cache, table, lens) + at.attend(q, cache, table, lens, cu_q) +
                at.prefill(q, kv[..., :128], kv[..., 128:], kr, cu_q, cu_k) +
                at.append(kr.new_ones(2, 192), cu_k[:2].long(), q=q[..., 128:]))

    want, before = calls(), torch.get_default_dtype()
    torch.set_default_dtype(dtype)
    try:
        got = calls()
    finally:
        torch.set_default_dtype(before)
    assert all(a.dtype == b.dtype and torch.equal(a, b) for a, b in zip(got, want))


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


# ---------------------------------------------------------------- in a row

H, R, D, N, PAGE = 6, 256, 64, 128, 16


class Chain:
    """A layer's buffers: queries [N + D], absorbed queries [R + D] whose position parts the append
    writes, dense rows whose position parts the expanded form reads where they lie."""

    def __init__(self):
        self.at = layer(H, R, D, N, N, PAGE)
        self.pages = torch.tensor([[5, 0, 7, 2, 6], [3, 9, 1, 8, 4]])
        self.cache = torch.full((10, PAGE, R + D), NAN, dtype=torch.bfloat16, device="cuda")

    def slots(self, b, positions):
        return self.pages[b, positions // PAGE] * PAGE + positions % PAGE

    def rows(self, b, n):
        return self.cache.view(-1, R + D)[self.slots(b, torch.arange(n)).cuda()].cpu()


def _check_append(c, kv, q, positions, got_rows, got_q):
    want = U.rows_of(kv, R, positions, c.at.freq, None, 1e-6, "halves")
    size = want.abs()
    size[:, R:] = kv[:, R:].double().abs().amax(1, keepdim=True) * 2
    U.check(got_rows, want, U.HALF_STEP * want.abs() + 2.0 ** -19 * size + 1e-30, "rows")
    want = U.rotate(q.double(), positions, c.at.freq, "halves")
    U.check(got_q, want, U.HALF_STEP * want.abs() +
            2.0 ** -18 * q.double().abs().amax(-1, keepdim=True), "queries")


def test_a_prompt_without_copies_between_calls():
    c, lens = Chain(), [75, 33]
    T, cu = sum(lens), starts(lens)
    kv, q, up = randn(1, T, R + D), randn(2, T, H, N + D), randn(3, T, H, R)
    positions = torch.cat([torch.arange(n) for n in lens])
    slots = torch.cat([c.slots(b, torch.arange(n)) for b, n in enumerate(lens)])
    absorbed = torch.full((T, H, R + D), NAN, dtype=torch.bfloat16, device="cuda")
    absorbed[..., :R] = up.cuda()
    rows = torch.empty(T, R + D, dtype=torch.bfloat16, device="cuda")
    c.at.append(kv.cuda(), positions.cuda(), slots.cuda(), c.cache, kv_out=rows,
                q=q.cuda()[..., N:], q_out=absorbed[..., R:])
    _check_append(c, kv, q[..., N:], positions, rows, absorbed[..., R:])
    assert torch.equal(absorbed[..., :R].cpu(), up)
    assert torch.equal(c.cache.view(-1, R + D)[slots.cuda()], rows)
    out, lse = c.at.attend(absorbed, c.cache, c.pages.int().cuda(), i32(lens), i32(cu))
    want, wl, ob, lb = U.attend(absorbed.cpu(), [c.rows(b, n) for b, n in enumerate(lens)],
                                list(zip(cu, cu[1:])), R, (N + D) ** -0.5)
    U.check(lse, wl, lb, "absorbed: lse")
    U.check(out, want, ob, "absorbed")
    turned = q.cuda()
    turned[..., N:] = absorbed[..., R:]
    k, v = randn(4, T, H, N), randn(5, T, H, N)
    out, lse = c.at.prefill(turned, k.cuda(), v.cuda(), rows[:, R:], i32(cu), i32(cu))
    want, wl, ob, lb = U.prefill(turned.cpu(), k, v, rows[:, R:].cpu(), cu, cu, (N + D) ** -0.5, True)
    U.check(lse, wl, lb, "expanded: lse")
    U.check(out, want, ob, "expanded")
    assert c.at.status() == B.KLT_OK


def test_decoding_steps_replayed():
    """Append and absorbed attention of two sequences in one graph, replayed token after token; the
    second sequence stops growing half-way (its slot is none)."""
    c = Chain()
    kv = torch.zeros(2, R + D, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(2, H, D, dtype=torch.bfloat16, device="cuda")
    absorbed = torch.zeros(2, H, R + D, dtype=torch.bfloat16, device="cuda")
    positions, slots = (torch.full((2,), v, device="cuda") for v in (0, -1))
    lens, table = i32([0, 0]), c.pages.int().cuda()
    out = torch.empty(2, H, R, dtype=torch.bfloat16, device="cuda")
    lse, ws = torch.empty(2, H, device="cuda"), c.at.workspace(2)

    def step():
        c.at.append(kv, positions, slots, c.cache, q=q, q_out=absorbed[..., R:])
        c.at.attend(absorbed, c.cache, table, lens, out=out, lse=lse, workspace=ws)

    step()
    torch.cuda.synchronize()
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    have = [0, 0]
    for t in range(70):
        grows = [True, t < 33]
        new = [randn(100 * t + i, 2, *n) for i, n in enumerate(((R + D,), (H, D), (H, R)))]
        kv.copy_(new[0])
        q.copy_(new[1])
        absorbed[..., :R].copy_(new[2])
        at = [n if g else n - 1 for n, g in zip(have, grows)]
        positions.copy_(torch.tensor(at))
        slots.copy_(torch.tensor([int(c.slots(b, torch.tensor(at[b]))) if grows[b] else -1
                                  for b in range(2)]))
        have = [n + g for n, g in zip(have, grows)]
        lens.copy_(torch.tensor(have, dtype=torch.int32))
        before = c.rows(1, have[1])
        graph.replay()
        torch.cuda.synchronize()
        if not grows[1]:
            assert torch.equal(c.rows(1, have[1]), before)
        seqs = [c.rows(b, n) for b, n in enumerate(have)]
        _check_append(c, new[0][:1], new[1][:1], torch.tensor(at[:1]), seqs[0][-1:],
                      absorbed[:1, :, R:])
        want, wl, ob, lb = U.attend(absorbed.cpu(), seqs, [(0, 1), (1, 2)], R, (N + D) ** -0.5)
        U.check(lse, wl, lb, f"lse {t}")
        U.check(out, want, ob, f"out {t}")
    assert c.at.status() == B.KLT_OK
