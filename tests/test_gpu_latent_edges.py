"""klt_latent_* on the GPU: layouts, batches that take other ways through the kernels, streams and
graphs, what a call leaves to the next one when its waits run out, and the operators in a row."""
import math

import numpy as np
import pytest
import torch

import latent_util as U
from latent_moe_layer_route_gb300 import binding as B
from oracle.codecs import e4m3_decode
from test_gpu_latent import (NAN, _lib, layer, paged, randn, run_attend,  # noqa: F401
                             run_prefill, starts)

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


class Attend:
    """A call's operands and its reference."""

    def __init__(self, heads, lens, counts, latent=128, rope=64, page=64, seed=0, cu=True):
        self.heads, self.latent, self.lens = heads, latent, lens
        self.at = layer(heads, latent, rope, page=page)
        cache, table, seqs = paged(seed, lens, page, latent + rope)
        cu_q = starts(counts)
        self.q = randn(seed + 1, cu_q[-1], heads, latent + rope)
        self.ref = U.attend(self.q, seqs, list(zip(cu_q, cu_q[1:])), latent, (128 + rope) ** -0.5)
        self.gpu = [self.q.cuda(), cache.cuda(), table.cuda(), i32(lens), i32(cu_q) if cu else None]

    def __call__(self, **kw):
        return self.at.attend(*self.gpu, **kw)

    def check(self, out, lse):
        want, wl, ob, lb = self.ref
        U.check(lse, wl, lb, "lse")
        U.check(out, want, ob, "out")


class Prefill:
    def __init__(self, heads, queries, keys, causal=True, seed=0):
        self.at, self.causal = layer(heads), causal
        cu_q, cu_k = starts(queries), starts(keys)
        self.q = randn(seed, cu_q[-1], heads, 192)
        kv, kr = randn(seed + 1, cu_k[-1], heads, 256), randn(seed + 2, cu_k[-1], 64)
        self.ref = U.prefill(self.q, kv[..., :128], kv[..., 128:], kr, cu_q, cu_k, 192 ** -0.5,
                             causal)
        g = kv.cuda()
        self.gpu = [self.q.cuda(), g[..., :128], g[..., 128:], kr.cuda(), i32(cu_q), i32(cu_k)]

    def __call__(self, **kw):
        return self.at.prefill(*self.gpu, causal=self.causal, **kw)

    check = Attend.check


# ---------------------------------------------------------------- other ways through the kernels

def test_attend_one_query_a_sequence_without_starts():
    c = Attend(16, [70, 1, 300, 64], [1] * 4, cu=False)
    c.check(*c())


@pytest.mark.parametrize("heads", [8, 100])
def test_attend_more_sequences_than_groups(heads):
    """Shares of the tiles of all sequences in a row, which begin and end inside of items; with 100
    heads two row tiles side by side."""
    lens = [(37 * i) % 331 for i in range(210)]
    run_attend(heads, lens, [1 + (i % 7 == 0) for i in range(210)], seed=3)


def test_attend_more_sequences_than_threads():
    lens = [(53 * i) % 97 for i in range(900)]
    run_attend(4, lens, [i % 3 for i in range(900)], seed=4, rope=16)


@pytest.mark.parametrize("length,heads", [(64 * 152 + 1, 4), (64 * 600, 2), (64 * 40 + 7, 70)])
def test_attend_many_parts(length, heads):
    run_attend(heads, [length, 5], [1, 2], seed=length, rope=16)


def test_attend_parts_where_some_rows_see_nothing():
    """A long run of queries: the last tiles of keys are behind the first queries' own."""
    run_attend(2, [64 * 30], [64 * 30], seed=8, rope=16)


@pytest.mark.parametrize("heads", [1, 3, 16, 24, 64])
@pytest.mark.parametrize("layout", ["heads first", "padded heads", "padded tokens", "one token"])
def test_attend_query_layouts(heads, layout):
    """Bulk copies of packed rows, of a token's heads, and copies by threads."""
    T = 1 if layout == "one token" else 5
    c = Attend(heads, [200] * T, [1] * T, latent=256, rope=32, seed=heads)
    W = 288
    if layout == "heads first":
        wide = c.q.transpose(0, 1).contiguous().cuda().transpose(0, 1)
    elif layout == "padded tokens":
        wide = torch.full((T, heads * W + 16), NAN, dtype=torch.bfloat16, device="cuda")
        wide = wide[:, :heads * W].unflatten(1, (heads, W))
        wide.copy_(c.q)
    else:
        wide = torch.full((T, heads, W + 24), NAN, dtype=torch.bfloat16, device="cuda")[..., :W]
        wide.copy_(c.q)
    c.gpu[0] = wide
    out = torch.empty(heads, T, 256 + 8, dtype=torch.bfloat16, device="cuda")
    out = out.transpose(0, 1)[..., :256]
    _, lse = c(out=out)
    c.check(out, lse)


def test_attend_cache_strides():
    """One layer of a cache that interleaves layers in a page, rows padded."""
    c = Attend(20, [100, 33, 250], [1, 2, 1], seed=12)
    cache = c.gpu[1]
    pages, page, W = cache.shape
    wide = torch.full((pages, 3, page, W + 8), NAN, dtype=torch.bfloat16, device="cuda")
    wide[:, 1, :, :W] = cache
    c.gpu[1] = wide[:, 1, :, :W]
    c.check(*c())


def test_attend_lengths_and_pages_outside():
    """Lengths beyond the table are cut to it, negative ones to 0; pages outside of the cache read
    as rows of zeros."""
    at = layer(8)
    cache, table, seqs = paged(5, [128, 100, 128], 64, 192)
    table[2, 1] = cache.shape[0] + 7
    table[1, 0] = -3
    zeros = torch.zeros(64, 192, dtype=torch.bfloat16)
    seqs = [seqs[0], torch.cat([zeros, seqs[1][64:]]), torch.cat([seqs[2][:64], zeros]),
            torch.zeros(0, 192, dtype=torch.bfloat16)]
    table = torch.cat([table, torch.zeros(1, 2, dtype=torch.int32)])
    q = randn(6, 4, 8, 192)
    out, lse = at.attend(q.cuda(), cache.cuda(), table.cuda(), i32([2 ** 31 - 1, 100, 128, -5]))
    want, wl, ob, lb = U.attend(q, seqs, [(i, i + 1) for i in range(4)], 128, 192 ** -0.5)
    U.check(lse, wl, lb, "lse")
    U.check(out, want, ob, "out")


def test_attend_without_a_cache():
    at = layer(8)
    out, lse = at.attend(randn(1, 2, 8, 192).cuda(),
                         torch.empty(0, 64, 192, dtype=torch.bfloat16, device="cuda"),
                         torch.empty(2, 0, dtype=torch.int32, device="cuda"), i32([5, 0]))
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())


def test_rows_beyond_32_bits_of_elements():
    """A cache of more than 2^31 elements; the pages in use are its first and last ones."""
    pages = 2 ** 31 // (64 * 192) + 20
    cache = torch.empty(pages, 64, 192, dtype=torch.bfloat16, device="cuda")
    at = layer(4)
    ids = [pages - 1, 0, pages - 2]
    rows = torch.cat([randn(3, 150, 128), randn(4, 150, 64)], 1)
    slots = torch.tensor([ids[i // 64] * 64 + i % 64 for i in range(150)])
    positions = torch.arange(150)
    at.append(rows.cuda(), positions.cuda(), slots.cuda(), cache)
    want = U.rows_of(rows, 128, positions, at.freq, None, 1e-6, "halves").bfloat16()
    got = torch.cat([cache[i] for i in ids])[:150].cpu()
    U.check(got, want.double(), U.HALF_STEP * 2 * want.double().abs() + 1e-5, "rows")
    q = randn(5, 1, 4, 192)
    out, lse = at.attend(q.cuda(), cache, i32([ids]), i32([150]))
    want, wl, ob, lb = U.attend(q, [got], [(0, 1)], 128, 192 ** -0.5)
    U.check(lse, wl, lb, "lse")
    U.check(out, want, ob, "out")


@pytest.mark.parametrize("bad", [NAN, math.inf])
def test_rows_that_are_not_finite_stay_in_their_sequence(bad):
    c = Attend(16, [130, 90, 200], [1, 2, 1], seed=21)
    table, cache = c.gpu[2], c.gpu[1]
    cache[int(table[1, 0]), 3] = bad
    out, lse = c()
    want, wl, ob, lb = (t.clone() for t in c.ref)
    for t in (want, wl):
        t[1:3] = NAN
    keep = [0, 3]
    U.check(out.cpu()[keep], want[keep], ob[keep], "out")
    U.check(lse.cpu()[keep], wl[keep], lb[keep], "lse")
    assert not bool(out[1:3].isfinite().all())
    p = Prefill(3, [100, 70, 300], [100, 70, 300], seed=22)
    for t in p.gpu[1:4]:
        t[100 + 5] = bad
    out, lse = p()
    want, wl, ob, lb = p.ref
    keep = list(range(100)) + list(range(170, 470))
    U.check(out.cpu()[keep], want[keep], ob[keep], "out")
    U.check(lse.cpu()[keep], wl[keep], lb[keep], "lse")


def test_prefill_layouts():
    """Heads first, keys and values apart, padded rows."""
    p = Prefill(5, [140, 3], [140, 260], seed=31)
    q, k, v, kr = p.gpu[:4]
    p.gpu[0] = q.transpose(0, 1).contiguous().transpose(0, 1)
    wide = torch.full((5, 400, 136), NAN, dtype=torch.bfloat16, device="cuda")
    p.gpu[1] = wide.transpose(0, 1)[..., :128].copy_(k)
    p.gpu[2] = v.contiguous()
    p.gpu[3] = torch.full((400, 72), NAN, dtype=torch.bfloat16, device="cuda")[:, :64].copy_(kr)
    out = torch.empty(5, 143, 136, dtype=torch.bfloat16, device="cuda").transpose(0, 1)[..., :128]
    _, lse = p(out=out)
    p.check(out, lse)


def test_prefill_many_sequences():
    lens = [(29 * i) % 71 for i in range(150)]
    run_prefill(2, lens, [n + i % 5 for i, n in enumerate(lens)], nope=64, rope=16, value=64,
                seed=41)


def test_append_in_place_and_without_a_cache():
    at = layer(24, 256, 32, gamma=randn(1, 256).abs() + 0.5)
    kv, q = randn(2, 9, 288), randn(3, 9, 24, 160)
    positions = torch.arange(9) * 1000
    g = q.cuda()
    kv_out, q_out = at.append(kv.cuda(), positions.cuda(), q=g[..., 128:], q_out=g[..., 128:])
    assert q_out.data_ptr() == g[..., 128:].data_ptr()
    want = U.rotate(q[..., 128:].double(), positions, at.freq, "halves")
    size = q[..., 128:].double().abs().amax(-1, keepdim=True)
    U.check(g[..., 128:], want, U.HALF_STEP * want.abs() + 2.0 ** -18 * size, "queries")
    assert torch.equal(g[..., :128].cpu(), q[..., :128])
    only = at.append(kv.cuda(), positions.cuda())
    assert only[1] is None and torch.equal(only[0], kv_out)


def test_append_rows_that_are_not_finite():
    at = layer(2)
    kv = randn(5, 4, 192)
    kv[1, 3], kv[2, 150] = NAN, math.inf
    out, _ = at.append(kv.cuda(), torch.arange(4).cuda())
    out = out.cpu().float()
    assert bool(out[0].isfinite().all()) and bool(out[3].isfinite().all())
    assert bool(out[1, :128].isnan().all()) and bool(out[1, 128:].isfinite().all())
    assert bool(out[2, :128].isfinite().all()) and not bool(out[2, 128:].isfinite().all())


# ---------------------------------------------------------------- repeated calls

def test_same_bits_whatever_the_workspace_held():
    c = Attend(40, [3000, 700, 64], [1, 2, 1], seed=51)
    ws = c.at.workspace(3, 4)
    first = None
    for fill in (0x00, 0xFF, 0x7F):
        ws.fill_(fill)
        got = c(workspace=ws)
        c.check(*got)
        first = first or [t.clone() for t in got]
        assert all(torch.equal(a, b) for a, b in zip(got, first))


@pytest.mark.parametrize("op", ["attend", "prefill"])
def test_captured_calls(op):
    """Two graphs with workspaces of their own, replayed in turn and after their inputs changed."""
    make = (lambda s: Attend(16, [300, 65, 1000], [1, 2, 1], seed=s)) if op == "attend" else \
        (lambda s: Prefill(3, [200, 65], [300, 65], seed=s))
    a, b, other = make(1), make(2), make(3)
    graphs, outs = [], []
    for c in (a, b):
        c.check(*c())
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(c())
        graphs.append(g)
    for _ in range(2):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    a.check(*outs[0])
    b.check(*outs[1])
    for dst, src in zip(a.gpu, other.gpu):
        dst.copy_(src)
    graphs[0].replay()
    torch.cuda.synchronize()
    other.check(*outs[0])
    b.check(*outs[1])
    assert a.at.status() == b.at.status() == B.KLT_OK


def test_lengths_change_between_replays():
    """The shares follow the lengths on the device: from one part to many."""
    c = Attend(16, [6000, 6000], [1, 1], seed=61)
    g = torch.cuda.CUDAGraph()
    c()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        out, lse = c()
    rows = []
    for b in range(2):
        ids = c.gpu[2][b].long()
        rows.append(c.gpu[1][ids].flatten(0, 1).cpu())
    for lens in ([1, 0], [6000, 10], [64, 65], [3000, 5999], [0, 0]):
        c.gpu[3].copy_(i32(lens))
        g.replay()
        torch.cuda.synchronize()
        want, wl, ob, lb = U.attend(c.q, [r[:n] for r, n in zip(rows, lens)], [(0, 1), (1, 2)], 128,
                                    192 ** -0.5)
        U.check(lse, wl, lb, f"lse {lens}")
        U.check(out, want, ob, f"out {lens}")


def test_two_streams_at_once():
    """Calls on two streams, each with a workspace of its own, and both kinds of attention."""
    a, b = Attend(64, [9000], [1], rope=16, seed=71), Prefill(8, [700], [700], seed=72)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    a.check(*a())
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for s, c in ((streams[0], a), (streams[1], a), (streams[0], b), (streams[1], b)):
            with torch.cuda.stream(s):
                got.append((c, c()))
    torch.cuda.synchronize()
    for c, r in got:
        c.check(*r)
    given = a(stream=streams[0].cuda_stream)  # from another stream's point of view
    streams[0].synchronize()
    a.check(*given)
    assert a.at.status() == b.at.status() == B.KLT_OK


@pytest.mark.parametrize("stall", [1, 2, 3, 5])
@pytest.mark.parametrize("op", ["attend", "attend flat", "prefill"])
def test_waits_that_run_out(op, stall):
    """A launch whose copies stop gives up within its bounds, says so, and leaves nothing to the
    launches right behind it."""
    if op == "attend":
        bad, ok = (Attend(16, [64 * 152 * 7], [1], rope=16, seed=s) for s in (81, 82))
    elif op == "attend flat":
        lens = [300 + i for i in range(320)]
        bad, ok = (Attend(8, lens, [1] * 320, rope=16, seed=s) for s in (81, 82))
    else:
        bad, ok = (Prefill(2, [900, 30], [900, 130], seed=s) for s in (81, 82))
    want = [t.clone() for t in ok()]
    ok.check(*want)
    torch.cuda.synchronize()
    bad(debug=B.KltLatentDebug(stall_after_tiles=stall, timeout_ms=5))
    got = [ok() for _ in range(3)]
    torch.cuda.synchronize()
    assert bad.at.status() == B.KLT_ERR_DEVICE_TIMEOUT
    assert ok.at.status() == B.KLT_OK
    for g in got:
        assert all(torch.equal(x, y) for x, y in zip(g, want))
    bad.at.close()


def test_bounds_of_waits_grow_with_a_sequence():
    """Waits that last for all keys of a sequence do not run out for its length alone: the queries'
    copies of a group's second item, and threads of the expanded form without queries."""
    dbg = B.KltLatentDebug(timeout_ms=1)
    at, length = layer(64, 512, 64), 1 << 17  # 2048 tiles of some 1.4 us
    cache = randn(91, 8, 64, 576).cuda()
    args = [randn(92, 160, 64, 576).cuda(), cache, i32([[i % 8 for i in range(length // 64)]]),
            i32([length]), i32([0, 160])]
    want = [t.clone() for t in at.attend(*args)]
    got = at.attend(*args, debug=dbg)
    torch.cuda.synchronize()
    assert at.status() == B.KLT_OK and all(torch.equal(x, y) for x, y in zip(got, want))
    at, length = layer(1, nope=64, value=64), 1 << 20  # 8192 tiles of some 0.5 us
    row = randn(93, 1 << 14, 1, 64).cuda().repeat(length >> 14, 1, 1)
    args = [randn(94, 1, 1, 128).cuda(), row, row, row[:, 0], i32([0, 1]), i32([0, length])]
    want = [t.clone() for t in at.prefill(*args)]
    got = at.prefill(*args, debug=dbg)
    torch.cuda.synchronize()
    assert at.status() == B.KLT_OK and all(torch.equal(x, y) for x, y in zip(got, want))


# ---------------------------------------------------------------- refusals

def test_binding_refuses(lib=None):
    at = layer(4)
    q, cache = randn(1, 2, 4, 192).cuda(), randn(2, 3, 64, 192).cuda()
    table, lens = i32([[0], [1]]), i32([5, 6])
    assert at.attend(q, cache, table, lens)[0].shape == (2, 4, 128)
    for args in ((q[:, :3], cache, table, lens), (q[..., :184], cache, table, lens),
                 (q, cache[:, :32], table, lens), (q, cache, table[:1], lens),
                 (q, cache, table, lens[:1]), (q, cache, table, lens, i32([0, 1])),
                 (q.transpose(1, 2).contiguous().transpose(1, 2), cache, table, lens),
                 (q.cpu(), cache, table, lens)):
        with pytest.raises(ValueError):
            at.attend(*args)
    for args in ((q.float(), cache, table, lens), (q, cache, table.long(), lens),
                 (q, cache, table, lens.float())):
        with pytest.raises(TypeError):
            at.attend(*args)
    with pytest.raises(B.KltError) as e:
        at.attend(q, cache, table, lens, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.code == B.KLT_ERR_INVALID_ARG
    with pytest.raises(B.KltError) as e:
        at.attend(torch.empty(2, 4, 196, dtype=torch.bfloat16, device="cuda")[..., 4:], cache, table,
                  lens)
    assert e.value.code == B.KLT_ERR_ALIGN
    kv, pos = randn(3, 2, 192).cuda(), torch.arange(2).cuda()
    with pytest.raises(TypeError):
        at.append(kv, pos.int())
    with pytest.raises(ValueError):
        at.append(kv, pos[:1])
    with pytest.raises(B.KltError):
        at.append(kv, pos, None, cache)
    k, v, kr = randn(4, 5, 4, 128).cuda(), randn(5, 5, 4, 128).cuda(), randn(6, 5, 64).cuda()
    cu_q, cu_k = i32([0, 2]), i32([0, 5])
    assert at.prefill(q, k, v, kr, cu_q, cu_k)[1].shape == (2, 4)
    for args in ((q, k[:, :3], v, kr, cu_q, cu_k), (q, k, v[:4], kr, cu_q, cu_k),
                 (q, k, v, kr[:, :32], cu_q, cu_k), (q, k, v, kr, cu_q, i32([0, 5, 5]))):
        with pytest.raises(ValueError):
            at.prefill(*args)
    with pytest.raises(B.KltError):
        at.prefill(q, k[:1].expand(5, 4, 128), v, kr, cu_q, cu_k)


# ---------------------------------------------------------------- in a row

def _fp8(rng, N, K):
    codes = (rng.integers(0x20, 0x4A, (N, K)) | rng.integers(0, 2, (N, K)) << 7).astype(np.uint8)
    scales = (rng.uniform(0.5, 1.5, (-(-N // 128), -(-K // 128))) / K ** 0.5).astype(np.float32)
    w = e4m3_decode(codes) * np.repeat(np.repeat(scales, 128, 0), 128, 1)[:N, :K]
    return torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), torch.from_numpy(w)


def test_the_attention_of_a_layer():
    """A prompt and then a decoded token through one layer's attention: norm to codes, the FP8
    projections, append, attention in expanded form for the prompt and in absorbed form for both.
    Each stage is checked against float64 from what the stage before left; the two forms of the
    prompt's attention agree within what the roundings of their operands allow."""
    H, hid, R, D, N, V, page, T = 6, 512, 256, 64, 128, 128, 16, 75
    rng = np.random.default_rng(7)
    gen = torch.Generator().manual_seed(8)
    gamma = (torch.rand(R, generator=gen) + 0.5).bfloat16()
    at = layer(H, R, D, N, V, page, gamma=gamma)
    down_q, down_s, down = _fp8(rng, R + D, hid)
    query_q, query_s, _ = _fp8(rng, H * (N + D), hid)
    norm = B.BlockNorm(hid, gamma_pre=torch.ones(hid, dtype=torch.bfloat16, device="cuda"))
    to_kv, to_q = B.Fp8Linear(down_q, down_s), B.Fp8Linear(query_q, query_s)
    w_uk = (torch.randn(H, N, R, generator=gen) / R ** 0.5).bfloat16()
    w_uv = (torch.randn(H, V, R, generator=gen) / R ** 0.5).bfloat16()
    cache = torch.full((8, page, R + D), NAN, dtype=torch.bfloat16, device="cuda")
    pages = torch.tensor([5, 0, 7, 2, 6])
    table = pages[None].int().cuda()
    scale = (N + D) ** -0.5

    def step(h, first):
        """Cache, queries and dense rows of tokens first .. of the sequence."""
        n = h.shape[0]
        positions = torch.arange(first, first + n)
        slots = pages[positions // page] * page + positions % page
        xq, xs = B.fp8_codes(n, hid, "cuda"), torch.empty(n, hid // 128, device="cuda")
        norm(h.cuda(), q=xq, s=xs)
        kv, q = to_kv(xq, xs), to_q(xq, xs).unflatten(1, (H, N + D))
        rows, q_rope = at.append(kv, positions.cuda(), slots.cuda(), cache,
                                 kv_out=torch.empty_like(kv), q=q[..., N:], q_out=q[..., N:])
        torch.cuda.synchronize()
        want = U.rows_of(kv.cpu(), R, positions, at.freq, gamma, 1e-6, "halves")
        size = want.abs()
        size[:, R:] = kv[:, R:].cpu().double().abs().amax(1, keepdim=True) * 2
        U.check(rows, want, U.HALF_STEP * want.abs() + 2.0 ** -19 * size + 1e-30, "rows")
        assert torch.equal(cache.view(-1, R + D)[slots.cuda()], rows)
        return rows, q

    def absorbed(q):
        up = torch.einsum("thn,hnr->thr", q[..., :N].float(), w_uk.cuda().float()).bfloat16()
        return torch.cat([up, q[..., N:]], -1).contiguous()

    h = torch.randn(T, hid, generator=gen).bfloat16()
    rows, q = step(h, 0)
    k = torch.einsum("tr,hnr->thn", rows[:, :R].float(), w_uk.cuda().float()).bfloat16()
    v = torch.einsum("tr,hvr->thv", rows[:, :R].float(), w_uv.cuda().float()).bfloat16()
    out, lse = at.prefill(q.contiguous(), k, v, rows[:, R:].contiguous(), i32([0, T]), i32([0, T]))
    want, wl, ob, lb = U.prefill(q.cpu(), k.cpu(), v.cpu(), rows[:, R:].cpu(), [0, T], [0, T], scale,
                                 True)
    U.check(lse, wl, lb, "prompt, expanded: lse")
    U.check(out, want, ob, "prompt, expanded")

    qa = absorbed(q)
    oa, la = at.attend(qa, cache, table, i32([T]), i32([0, T]))
    want, wl, ob, lb = U.attend(qa.cpu(), [rows.cpu()], [(0, T)], R, scale)
    U.check(la, wl, lb, "prompt, absorbed: lse")
    U.check(oa, want, ob, "prompt, absorbed")
    # the forms: scores differ by the roundings of k (expanded) and of the absorbed queries
    g = scale * U.HALF_STEP * (
        torch.einsum("thn,khn->thk", q[..., :N].cpu().double().abs(), k.cpu().double().abs()) +
        torch.einsum("thr,kr->thk", qa[..., :R].cpu().double().abs(),
                     rows[:, :R].cpu().double().abs())).amax(-1)
    U.check(la, lse.cpu().double(), 1.01 * g + 2 * lb, "the two forms' lse")
    mixed = torch.einsum("thr,hvr->thv", oa.float(), w_uv.cuda().float())
    err = (mixed - out.float()).norm() / out.float().norm()
    assert float(err) < 0.02, err  # a few bf16 roundings of 2^-8 and weights off by e^g - 1

    row, q = step(torch.randn(1, hid, generator=gen).bfloat16(), T)
    qa = absorbed(q)
    oa, la = at.attend(qa, cache, table, i32([T + 1]))
    want, wl, ob, lb = U.attend(qa.cpu(), [torch.cat([rows, row]).cpu()], [(0, 1)], R, scale)
    U.check(la, wl, lb, "token: lse")
    U.check(oa, want, ob, "token")
    assert at.status() == to_kv.status() == to_q.status() == B.KLT_OK
