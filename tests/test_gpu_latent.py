"""Latent attention on the GPU (klt_latent_append, klt_latent_attend, klt_latent_prefill) against
float64, within bounds derived in latent_util."""
import math

import pytest
import torch

import latent_util as U
from latent_moe_layer_route_gb300 import binding as B
from latent_moe_layer_route_gb300 import build

pytestmark = pytest.mark.gpu
NAN = math.nan


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    B.load_library()


def layer(heads, latent=128, rope=64, nope=128, value=128, page=64, gamma=None, **kw):
    freq = (10000.0 ** (-torch.arange(0, rope, 2, dtype=torch.float64) / rope)).float()
    at = B.LatentAttention(heads, latent, rope, nope, value, page, inv_freq=freq.cuda(),
                           gamma=None if gamma is None else gamma.cuda(), **kw)
    at.freq = freq
    return at


def randn(seed, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


# ---------------------------------------------------------------- append

@pytest.mark.parametrize("T,heads,latent,rope,page,dtype,pairs,gamma", [
    (1, 1, 128, 16, 16, torch.bfloat16, "halves", True),
    (1, 16, 512, 64, 64, torch.bfloat16, "halves", True),
    (5, 3, 384, 48, 32, torch.float32, "neighbours", True),
    (33, 128, 256, 32, 1024, torch.bfloat16, "neighbours", False),
    (70, 40, 512, 64, 16, torch.float32, "halves", False),
    (19, 256, 128, 48, 128, torch.bfloat16, "halves", True),
    # two tokens to a block, the last one alone
    (1601, 36, 128, 64, 32, torch.bfloat16, "halves", True),
    (1512, 65, 256, 48, 16, torch.float32, "neighbours", False)])
def test_append(T, heads, latent, rope, page, dtype, pairs, gamma):
    g = randn(1, latent).abs() + 0.5 if gamma else None
    at = layer(heads, latent, rope, page=page, gamma=g, pairs=pairs)
    W = latent + rope
    wide = randn(2, T, W + 24, dtype=dtype)
    wide[0] *= 1e-6  # a row whose norm eps decides
    kv = wide[:, 8:8 + W]
    gen = torch.Generator().manual_seed(3)
    positions = torch.randint(0, 2_000_000, (T,), generator=gen)
    positions[-1] = 2 ** 31
    pages = -(-T // page) + 1
    slots = torch.randperm(pages * page, generator=gen)[:T]
    outside = [-1, pages * page, -(2 ** 62), 2 ** 62]
    for i, s in zip(range(1, T, 7), outside):
        slots[i] = s
    before = randn(4, pages, page, W)
    cache = before.cuda()
    q = randn(5, T, heads, 96 + rope)
    kv_out, q_out = at.append(wide.cuda()[:, 8:8 + W], positions.cuda(), slots.cuda(), cache,
                              kv_out=torch.empty(T, W, dtype=torch.bfloat16, device="cuda"),
                              q=q.cuda()[..., 96:])
    torch.cuda.synchronize()
    want = U.rows_of(kv, latent, positions, at.freq, g, 1e-6, pairs)
    # the row's sum of squares and its root in fp32; a turned pair's two products and angle
    size = want.abs()
    size[:, latent:] = kv[:, latent:].double().abs().amax(1, keepdim=True) * 2
    bound = U.HALF_STEP * want.abs() + 2.0 ** -19 * size + 1e-37
    U.check(kv_out, want, bound, "dense rows")
    flat = before.double().view(-1, W).clone()
    limit = torch.zeros_like(flat)
    for t, s in enumerate(slots.tolist()):
        if 0 <= s < pages * page:
            flat[s], limit[s] = want[t], bound[t]
    U.check(cache.view(-1, W), flat, limit, "cache")
    qr = q[..., 96:].double()
    want = U.rotate(qr, positions, at.freq, pairs)
    U.check(q_out, want, U.HALF_STEP * want.abs() + 2.0 ** -19 * 2 *
            qr.abs().amax(-1, keepdim=True), "queries")


# ---------------------------------------------------------------- attend

def paged(seed, lens, page, width, spare=3):
    """A cache whose unused rows are nan, its table, and each sequence's rows."""
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    gen = torch.Generator().manual_seed(seed)
    order = torch.randperm(pages, generator=gen)
    cache = torch.full((pages, page, width), NAN, dtype=torch.bfloat16)
    table = torch.full((len(lens), max(max(need), 1)), 2 ** 30, dtype=torch.int32)
    seqs, at = [], 0
    for b, n in enumerate(lens):
        rows = torch.randn(n, width, generator=gen).bfloat16()
        ids = order[at:at + need[b]]
        at += need[b]
        table[b, :need[b]] = ids.int()
        for i, page_id in enumerate(ids.tolist()):
            part = rows[i * page:(i + 1) * page]
            cache[page_id, :len(part)] = part
        seqs.append(rows)
    return cache, table, seqs


def starts(counts):
    out = [0]
    for n in counts:
        out.append(out[-1] + n)
    return out


def run_attend(heads, lens, counts, latent=128, rope=64, page=64, seed=0, spread=1.0, extra=0,
               at=None):
    W = latent + rope
    at = at or layer(heads, latent, rope, page=page)
    cache, table, seqs = paged(seed, lens, page, W)
    cu = starts(counts)
    T = cu[-1] + extra
    q = (randn(seed + 1, T, heads, W).float() * spread).bfloat16()
    out = torch.full((T, heads, latent), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, heads), 7.0, device="cuda")
    at.attend(q.cuda(), cache.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
              torch.tensor(cu, dtype=torch.int32).cuda(), out=out, lse=lse)
    torch.cuda.synchronize()
    assert at.status() == B.KLT_OK
    want, wl, ob, lb = U.attend(q, seqs, list(zip(cu, cu[1:])), latent, (128 + rope) ** -0.5)
    want[cu[-1]:], wl[cu[-1]:] = 7.0, 7.0  # rows behind the last sequence
    U.check(lse, wl, lb, "lse")
    U.check(out, want, ob, "out")


@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 513])
def test_attend_lengths(length):
    run_attend(16, [length], [1], seed=length)


@pytest.mark.parametrize("heads", [1, 2, 7, 8, 16, 31, 32, 33, 63, 64, 65, 100, 128, 129, 256])
def test_attend_heads(heads):
    run_attend(heads, [70, 131], [1, 1], seed=heads)


@pytest.mark.parametrize("latent", [128, 256, 384, 512])
@pytest.mark.parametrize("rope", [16, 32, 48, 64])
def test_attend_widths(latent, rope):
    run_attend(20, [100, 3, 190], [1, 1, 1], latent, rope, seed=latent + rope)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256, 1024])
def test_attend_pages(page):
    run_attend(16, [page - 1, page, page + 1, 2 * page + 5, 1], [1] * 5, page=page, seed=page)


@pytest.mark.parametrize("heads,lens,counts", [
    (16, [5, 100, 64, 200], [2, 4, 1, 3]),
    (40, [66, 129], [3, 2]),
    (128, [70, 65], [2, 5]),
    (3, [200, 70], [100, 70]),          # many queries, down to the first token
    (64, [1, 2, 3, 130], [1, 2, 3, 4]),
    (8, [3, 100], [9, 4]),              # queries before the first token see nothing
    (5, [0, 20, 0, 40], [1, 2, 3, 0]),  # empty sequences, and one without queries
    (5, [0, 0], [1, 1])])
def test_attend_several_queries(heads, lens, counts):
    run_attend(heads, lens, counts, seed=sum(lens), extra=3)


@pytest.mark.parametrize("spread", [0.0, 1e-3, 8.0, 60.0])
def test_attend_score_ranges(spread):
    run_attend(16, [300, 65], [1, 2], seed=5, spread=spread)


# ---------------------------------------------------------------- prefill

def run_prefill(heads, queries, keys, causal=True, nope=128, rope=64, value=128, seed=0, extra=0,
                spread=1.0):
    at = layer(heads, 128, rope, nope, value)
    cu_q, cu_k = starts(queries), starts(keys)
    T, S = cu_q[-1] + extra, cu_k[-1] + extra
    q = (randn(seed, T, heads, nope + rope).float() * spread).bfloat16()
    kv = randn(seed + 1, S, heads, nope + value)
    kr = randn(seed + 2, S, rope)
    kv[cu_k[-1]:], kr[cu_k[-1]:] = NAN, NAN  # behind the last sequence
    out = torch.full((T, heads, value), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, heads), 7.0, device="cuda")
    g = kv.cuda()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    at.prefill(q.cuda(), g[..., :nope], g[..., nope:], kr.cuda(), i32(cu_q), i32(cu_k),
               causal=causal, out=out, lse=lse)
    torch.cuda.synchronize()
    assert at.status() == B.KLT_OK
    want, wl, ob, lb = U.prefill(q, kv[..., :nope], kv[..., nope:], kr, cu_q, cu_k,
                                 (nope + rope) ** -0.5, causal)
    want[cu_q[-1]:], wl[cu_q[-1]:] = 7.0, 7.0
    U.check(lse, wl, lb, "lse")
    U.check(out, want, ob, "out")


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n", [1, 2, 63, 64, 127, 128, 129, 255, 256, 257, 400])
def test_prefill_lengths(n, causal):
    run_prefill(2, [n], [n], causal, seed=n)


@pytest.mark.parametrize("nope,rope,value", [(64, 16, 64), (64, 64, 128), (128, 32, 64),
                                             (128, 48, 128), (64, 32, 64)])
def test_prefill_widths(nope, rope, value):
    run_prefill(3, [130, 70], [130, 300], nope=nope, rope=rope, value=value, seed=nope + rope)


@pytest.mark.parametrize("heads,queries,keys,causal", [
    (1, [1, 5, 130], [1, 300, 131], True), (5, [3, 0, 200, 1], [3, 10, 450, 700], True),
    (2, [20, 300], [5, 129], True),     # more queries than keys: some see nothing
    (2, [20, 30], [0, 60], True), (2, [20, 30], [0, 60], False), (3, [7], [0], True),
    (4, [140, 1, 1, 257], [1, 140, 257, 600], False), (2, [129] * 40, [200] * 40, True)])
def test_prefill_sequences(heads, queries, keys, causal):
    run_prefill(heads, queries, keys, causal, seed=sum(keys), extra=5)


@pytest.mark.parametrize("spread", [0.0, 8.0, 60.0])
def test_prefill_score_ranges(spread):
    run_prefill(2, [260, 40], [300, 40], seed=9, spread=spread)


@pytest.mark.parametrize("value", [64, 128])
@pytest.mark.parametrize("n,m,causal", [
    (1, 1, True), (1, 129, True), (1, 256, True), (200, 257, True), (256, 384, True),
    (256, 385, False), (129, 640, True), (40, 900, False), (255, 1300, True)])
def test_prefill_few_queries(n, m, causal, value):
    """One tile of queries: its tiles of keys are shared out between two groups, an even or odd
    number of them, whose last one is either's."""
    run_prefill(3, [n, n], [m, m], causal, value=value, seed=n + m)


def test_prefill_few_queries_score_ranges():
    for spread in (0.0, 8.0, 60.0):
        run_prefill(2, [70, 200], [700, 1100], seed=10, spread=spread)


def test_prefill_groups_of_heads():
    """Keys and values of 16 heads and more fill half of L2: heads are taken by groups."""
    run_prefill(19, [260, 3, 40], [300, 9000, 40], nope=64, rope=16, seed=11)


def test_prefill_many_units():
    """More units than pairs of CTAs, short and long ones, ragged ends in every stage of the ring:
    a pair takes over many units, and its copies run ahead of its products."""
    lens = [1, 700, 130, 40, 515, 129, 3, 260, 90, 1030, 5, 384]
    run_prefill(40, lens, [n + 3 * i for i, n in enumerate(lens)], nope=64, rope=16, value=64,
                seed=77)
