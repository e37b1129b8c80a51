"""What is measured of latent attention: the step that fills the paged cache of latent rows, and
attention over it in its absorbed and in its expanded form.

    append   a token's latent row [c | r]: RMSNorm of c (latent width) times gamma, r (the part
             that carries the position) rotated by its position's angles; stored in the token's
             slot of the cache and in a dense copy, and the queries' position parts rotated too
    attend   queries in the latent space against the rows of a sequence's pages: the row is the
             key, its latent part the value; a sequence's new tokens are its last ones
    prefill  keys and values of every head, the keys' position part shared by the heads; packed
             sequences, a sequence's queries being its last tokens

With `own` false `run` computes them by elementary torch operations in 32 bits (the angles in
64), with `own` true by the framework's calls.
"""
import math
import random

import torch

own = False

EPS = 1e-6
NOPE = VALUE = 128
GAP = 2  # pages of the cache that belong to no sequence


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a decode batch's new tokens, far into their sequences
        dict(name="append_t16", op="append", T=16, heads=64, latent=512, rope=64, page=64,
             kv="bf16", pairs="halves", far=100000, holes=False),
        # an odd batch padded for a fixed launch: some tokens have no slot; an fp32 projection
        dict(name="append_t1003_ragged", op="append", T=1003, heads=40, latent=256, rope=32,
             page=16, kv="f32", pairs="neighbours", far=1000000, holes=True),
        # a prefill batch: nothing but memory traffic
        dict(name="append_t8192", op="append", T=8192, heads=64, latent=512, rope=64, page=64,
             kv="bf16", pairs="halves", far=8192, holes=False),
        # one short sequence, few heads: pure latency
        dict(name="attend_one", op="attend", B=1, heads=16, latent=512, rope=64, page=64, q=1,
             len=77, ragged=False),
        # one sequence of great length
        dict(name="attend_long", op="attend", B=1, heads=64, latent=512, rope=64, page=64, q=1,
             len=130001, ragged=False),
        # an ordinary decode batch of ragged lengths
        dict(name="attend_b32", op="attend", B=32, heads=64, latent=512, rope=64, page=64, q=1,
             len=8192, ragged=True),
        # up to four proposed tokens a sequence, a smaller latent, small pages, odd sizes
        dict(name="attend_b17_spec", op="attend", B=17, heads=40, latent=256, rope=32, page=16,
             q=4, len=3001, ragged=True),
        # a large decode batch with every head
        dict(name="attend_b128_h128", op="attend", B=128, heads=128, latent=512, rope=64,
             page=64, q=1, len=4096, ragged=True),
        # a few short prompts
        dict(name="prefill_short", op="prefill", B=3, heads=16, rope=64, q=65, ctx=0,
             causal=True, ragged=True),
        # a batch of prompts of ragged lengths
        dict(name="prefill_b12_ragged", op="prefill", B=12, heads=40, rope=64, q=2500, ctx=0,
             causal=True, ragged=True),
        # the next chunk of two long prompts
        dict(name="prefill_chunk", op="prefill", B=2, heads=32, rope=64, q=1024, ctx=15360,
             causal=True, ragged=False),
        # one long prompt with many heads: tensor work
        dict(name="prefill_8192", op="prefill", B=1, heads=64, rope=64, q=8192, ctx=0,
             causal=True, ragged=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "prefill"])
    heads = rng.choice([16, 32, 64, 128, rng.randint(1, 128)])
    rope = rng.choice([64, 64, 32, 48, 16])
    latent = rng.choice([512, 512, 384, 256, 128])
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        T = _log(rng, 1, 8192)
        return dict(op=op, T=T, heads=min(heads, 64 * 8192 // T), latent=latent, rope=rope,
                    page=page, kv=rng.choice(["bf16", "f32"]),
                    pairs=rng.choice(["halves", "neighbours"]), far=_log(rng, 8192, 1000000),
                    holes=rng.random() < 0.5)
    if op == "attend":
        while True:
            B, n, length = _log(rng, 1, 128), rng.choice([1, 1, 2, 4]), _log(rng, 16, 131072)
            if B * length <= 1 << 18 and B * length * heads * n <= 1 << 25:
                break
        return dict(op=op, B=B, heads=heads, latent=latent, rope=rope, page=page, q=n,
                    len=length, ragged=B > 1 and rng.random() < 0.7)
    while True:
        B, n = _log(rng, 1, 16), _log(rng, 1, 8192)
        ctx = rng.choice([0, _log(rng, 1, 16384)])
        if B * heads * n * (n + ctx) <= 64 * 8192 * 4096 and B * (n + ctx) * heads <= 1 << 20:
            break
    return dict(op=op, B=B, heads=heads, rope=rope, q=n, ctx=ctx, causal=rng.random() < 0.8,
                ragged=B > 1 and rng.random() < 0.7)


def _lengths(case):
    """Keys and queries of every sequence: the longest has the case's sizes, the others of a
    ragged batch anything from one token on."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    queries, keys = [], []
    for b in range(case["B"]):
        full = b == case["B"] // 2 or not case["ragged"]
        n = case["q"] if full else rng.randint(1, case["q"])
        if case["op"] == "attend":
            k = case["len"] if full else rng.randint(min(n, case["len"]), case["len"])
            n = min(n, k)
        else:
            k = n + (case["ctx"] if full else rng.randint(0, case["ctx"]))
        queries.append(n)
        keys.append(k)
    return queries, keys


def _pairs_of(case):
    """(query, key) pairs of one head that the masks leave."""
    queries, keys = _lengths(case)
    if case["op"] == "prefill" and not case["causal"]:
        return sum(n * k for n, k in zip(queries, keys))
    return sum(n * k - n * (n - 1) // 2 for n, k in zip(queries, keys))


# ---------------------------------------------------------------- inputs

def _ceil(a, b):
    return -(-a // b)


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _starts(lengths):
    out = [0]
    for n in lengths:
        out.append(out[-1] + n)
    return torch.tensor(out, dtype=torch.int32).cuda()


def _latent_rows(gen, rows, latent, rope):
    """Rows as a cache holds them: a normed part, a few of its channels larger, and a rotated
    part."""
    out = torch.empty(rows, latent + rope, dtype=torch.bfloat16, device="cuda")
    channel = torch.rand(latent, generator=gen, device="cuda")
    gain = torch.where(channel < 0.02, 4.0, 1.0)
    for lo in range(0, rows, 1 << 16):
        n = min(1 << 16, rows - lo)
        v = _randn(gen, n, latent + rope)
        v[:, :latent] *= gain
        out[lo:lo + n] = v
    return out


def _layer(case, st, latent=512, page=64, pairs="halves", gamma=None):
    from latent_moe_layer_route_gb300 import binding
    return binding.LatentAttention(
        case["heads"], latent=latent, rope=case["rope"], nope=NOPE, value=VALUE, page=page,
        inv_freq=st["inv_freq"], gamma=gamma, scale=st["scale"], eps=EPS, pairs=pairs)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, H, D = case["op"], case["heads"], case["rope"]
    st = dict(case=dict(case), scale=1.0 / math.sqrt(NOPE + D))
    st["inv_freq"] = (10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float().cuda()
    if op == "append":
        T, R, page = case["T"], case["latent"], case["page"]
        # the latent rows are the last columns of a wider projection's output
        wide = _randn(gen, T, 64 + R + D) * torch.exp(_randn(gen, T, 1) * 0.5)
        st["kv"] = (wide if case["kv"] == "f32" else wide.bfloat16())[:, 64:]
        st["gamma"] = (torch.rand(R, generator=gen, device="cuda") + 0.5).bfloat16()
        st["positions"] = torch.randint(0, case["far"], (T,), generator=gen, device="cuda")
        pages = _ceil(T, page) + GAP
        slots = torch.randperm(pages * page, generator=gen, device="cuda")[:T]
        if case["holes"]:  # padding; the first token is a real one
            hole = torch.rand(T, generator=gen, device="cuda") < 0.1
            hole[0] = False
            slots = torch.where(hole, -1, slots)
        st["slots"] = slots
        st["cache"] = _latent_rows(gen, pages * page, R, D).view(pages, page, R + D)
        st["queries"] = _randn(gen, T, H, NOPE + D).bfloat16()
        st["kv_out"] = torch.empty(T, R + D, dtype=torch.bfloat16, device="cuda")
        st["q_out"] = torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda")
        if own:
            st["layer"] = _layer(case, st, R, page, case["pairs"], st["gamma"])
        return st
    queries, keys = _lengths(case)
    T = sum(queries)
    st["cu_q"] = _starts(queries)
    st["lse"] = torch.empty(T, H, device="cuda")
    sharp = torch.exp(_randn(gen, 1, H, 1) * 0.3)  # heads differ in how far they spread
    if op == "attend":
        R, page = case["latent"], case["page"]
        st["seq_lens"] = torch.tensor(keys, dtype=torch.int32).cuda()
        used = [_ceil(k, page) for k in keys]
        pages = sum(used) + GAP
        order = torch.randperm(pages, generator=gen, device="cuda").int()
        table = torch.zeros(case["B"], max(used), dtype=torch.int32, device="cuda")
        lo = 0
        for b, n in enumerate(used):
            table[b, :n] = order[lo:lo + n]
            lo += n
        st["block_table"] = table
        st["cache"] = _latent_rows(gen, pages * page, R, D).view(pages, page, R + D)
        st["q"] = (_randn(gen, T, H, R + D) * sharp).bfloat16()
        st["out"] = torch.empty(T, H, R, dtype=torch.bfloat16, device="cuda")
        if own:
            st["layer"] = _layer(case, st, R, page)
            st["workspace"] = st["layer"].workspace(case["B"], T)
        return st
    S = sum(keys)
    st["cu_k"] = _starts(keys)
    st["q"] = (_randn(gen, T, H, NOPE + D) * sharp).bfloat16()
    # keys and values of a head side by side, as their projection leaves them
    st["kv"] = torch.empty(S, H, NOPE + VALUE, dtype=torch.bfloat16, device="cuda")
    for lo in range(0, S, 8192):
        n = min(8192, S - lo)
        st["kv"][lo:lo + n] = _randn(gen, n, H, NOPE + VALUE)
    st["k_rope"] = _randn(gen, S, D).bfloat16()
    st["out"] = torch.empty(T, H, VALUE, dtype=torch.bfloat16, device="cuda")
    if own:
        st["layer"] = _layer(case, st)
    return st


# ---------------------------------------------------------------- plain forms (32 bits)

def _rotate(v, positions, inv_freq, pairs):
    """fp32 v [T, ..., D] rotated by its tokens' angles."""
    angle = positions.double()[:, None] * inv_freq.double()
    shape = (-1,) + (1,) * (v.dim() - 2) + (inv_freq.shape[0],)
    c, s = torch.cos(angle).float().view(shape), torch.sin(angle).float().view(shape)
    half = v.shape[-1] // 2
    if pairs == "halves":
        a, b = v[..., :half], v[..., half:]
        return torch.cat([a * c - b * s, b * c + a * s], dim=-1)
    a, b = v[..., 0::2], v[..., 1::2]
    return torch.stack([a * c - b * s, b * c + a * s], dim=-1).flatten(-2)


def _plain_append(st):
    case = st["case"]
    R, pairs = case["latent"], case["pairs"]
    c = st["kv"][:, :R].float()
    c = c * torch.rsqrt(c.square().mean(dim=-1, keepdim=True) + EPS) * st["gamma"].float()
    r = _rotate(st["kv"][:, R:].float(), st["positions"], st["inv_freq"], pairs)
    rows = torch.cat([c, r], dim=-1).bfloat16()
    # a token without a slot writes the first token's row once more
    slots = st["slots"]
    there = slots >= 0
    flat = st["cache"].view(-1, rows.shape[1])
    flat[torch.where(there, slots, slots[0])] = torch.where(there[:, None], rows, rows[0])
    q = _rotate(st["queries"][..., NOPE:].float(), st["positions"], st["inv_freq"], pairs)
    return {"cache": st["cache"], "kv": rows, "q": q.bfloat16()}


def _softmax(s, allowed):
    """Weights and log-sum-exp of scores s along the last axis where `allowed`."""
    s = s.masked_fill(~allowed, -math.inf)
    m = s.amax(dim=-1, keepdim=True)
    p = torch.exp(s - m)
    total = p.sum(dim=-1, keepdim=True)
    return p / total, (m + torch.log(total)).squeeze(-1)


def _plain_attend(st):
    case = st["case"]
    R, page, H = case["latent"], case["page"], case["heads"]
    T, B, n = st["q"].shape[0], case["B"], case["q"]
    # queries of each sequence, one behind the other, padded to the most that one has
    first = st["cu_q"][:-1].long()
    count = st["cu_q"][1:].long() - first
    token = torch.arange(n, device="cuda")[None]
    q = st["q"][(first[:, None] + token).clamp(max=T - 1)].float()
    rows = st["cache"][st["block_table"].long()].flatten(1, 2)[:, :case["len"]].float()
    s = q.flatten(1, 2) @ rows.transpose(1, 2) * st["scale"]
    last = st["seq_lens"].long()[:, None] - count[:, None] + token
    allowed = torch.arange(rows.shape[1], device="cuda") <= last[..., None]
    p, lse = _softmax(s.view(B, n, H, -1), allowed[:, :, None])
    out = (p.flatten(1, 2) @ rows[..., :R]).view(B, n, H, R)
    # back to the tokens
    at = torch.arange(T, device="cuda")
    seq = torch.searchsorted(st["cu_q"][1:].long(), at, right=True)
    at = at - first[seq]
    return {"out": out[seq, at].bfloat16(), "lse": lse[seq, at]}


def _plain_prefill(st):
    case = st["case"]
    H = case["heads"]
    queries, keys = _lengths(case)
    out, lses = [], []
    t = k0 = 0
    for n, k in zip(queries, keys):
        q = st["q"][t:t + n].float().transpose(0, 1)
        kv = st["kv"][k0:k0 + k].float().transpose(0, 1)
        kr = st["k_rope"][k0:k0 + k].float()
        allowed = torch.ones(n, k, dtype=torch.bool, device="cuda")
        if case["causal"]:
            allowed = torch.arange(k, device="cuda") <= \
                torch.arange(k - n, k, device="cuda")[:, None]
        outs, ls = [], []
        step = max(1, (1 << 29) // (n * k))  # heads at a time
        for h in range(0, H, step):
            qh, kvh = q[h:h + step], kv[h:h + step]
            s = qh[..., :NOPE] @ kvh[..., :NOPE].transpose(1, 2)
            s = (s + qh[..., NOPE:] @ kr.t()) * st["scale"]
            p, lse = _softmax(s, allowed)
            outs.append(p @ kvh[..., NOPE:])
            ls.append(lse)
        out.append(torch.cat(outs).transpose(0, 1))
        lses.append(torch.cat(ls).t())
        t, k0 = t + n, k0 + k
    return {"out": torch.cat(out).bfloat16(), "lse": torch.cat(lses)}


# ---------------------------------------------------------------- the framework's calls

def _own(st):
    op, layer = st["case"]["op"], st["layer"]
    if op == "append":
        kv, q = layer.append(st["kv"], st["positions"], st["slots"], st["cache"],
                             kv_out=st["kv_out"], q=st["queries"][..., NOPE:],
                             q_out=st["q_out"])
        return {"cache": st["cache"], "kv": kv, "q": q}
    if op == "attend":
        out, lse = layer.attend(st["q"], st["cache"], st["block_table"], st["seq_lens"],
                                st["cu_q"], out=st["out"], lse=st["lse"],
                                workspace=st["workspace"])
    else:
        out, lse = layer.prefill(st["q"], st["kv"][..., :NOPE], st["kv"][..., NOPE:],
                                 st["k_rope"], st["cu_q"], st["cu_k"],
                                 causal=st["case"]["causal"], out=st["out"], lse=st["lse"])
    return {"out": out, "lse": lse}


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "attend": _plain_attend,
            "prefill": _plain_prefill}[state["case"]["op"]](state)


# ---------------------------------------------------------------- what it cannot do without

def work(case):
    H, D = case["heads"], case["rope"]
    if case["op"] == "append":
        T, width = case["T"], case["latent"] + D
        row = width * ((2 if case["kv"] == "bf16" else 4) + 2 + 2)
        return dict(bytes=T * (row + 2 * 2 * H * D + 16) + 2 * case["latent"] + 2 * D,
                    flops=T * (4 * case["latent"] + 3 * D * (H + 1)))
    queries, keys = _lengths(case)
    T, S = sum(queries), sum(keys)
    if case["op"] == "attend":
        R = case["latent"]
        table = 4 * sum(_ceil(k, case["page"]) for k in keys)
        return dict(bytes=2 * S * (R + D) + T * H * (2 * (2 * R + D) + 4) + table +
                    8 * case["B"], flops=2 * H * (2 * R + D) * _pairs_of(case))
    return dict(bytes=2 * (T * H * (NOPE + D + VALUE) + S * (H * (NOPE + VALUE) + D)) +
                4 * T * H + 8 * case["B"],
                flops=2 * H * (NOPE + D + VALUE) * _pairs_of(case))


# ---------------------------------------------------------------- the definition in 64 bits

def _exact_rotate(v, positions, inv_freq, pairs):
    """The pairs as complex numbers, times the unit number of their angle."""
    half = v.shape[-1] // 2
    z = torch.complex(v[..., :half], v[..., half:]) if pairs == "halves" else \
        torch.view_as_complex(v.reshape(*v.shape[:-1], half, 2).contiguous())
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       torch.outer(positions.double(), inv_freq.double()))
    z = z * (turn if v.dim() == 2 else turn[:, None])
    if pairs == "halves":
        return torch.cat([z.real, z.imag], dim=-1)
    return torch.view_as_real(z).reshape(v.shape)


def _exact_rows(s, v):
    """Softmax of the scores s [n, k] (minus infinity where masked) times v [k, d]."""
    lse = torch.logsumexp(s, dim=1)
    return torch.exp(s - lse[:, None]) @ v, lse


def exact(case, seed):
    st = prepare(case, seed)
    op, H = case["op"], case["heads"]
    if op == "append":
        R, pairs = case["latent"], case["pairs"]
        c = st["kv"][:, :R].double()
        c = c / torch.sqrt((c * c).sum(1, keepdim=True) / R + EPS) * st["gamma"].double()
        r = _exact_rotate(st["kv"][:, R:].double(), st["positions"], st["inv_freq"], pairs)
        rows = torch.cat([c, r], dim=1)
        cache = st["cache"].double().flatten(0, 1)
        kept = st["slots"] >= 0
        cache[st["slots"][kept]] = rows[kept]
        q = _exact_rotate(st["queries"][..., NOPE:].double(), st["positions"], st["inv_freq"],
                          pairs)
        return {"cache": cache.view(st["cache"].shape), "kv": rows, "q": q}
    queries, keys = _lengths(case)
    T, width = st["q"].shape[0], st["out"].shape[2]
    out = torch.empty(T, H, width, dtype=torch.float64, device="cuda")
    lse = torch.empty(T, H, dtype=torch.float64, device="cuda")
    t = k0 = 0
    for b, (n, k) in enumerate(zip(queries, keys)):
        # the keys that a query does not see lie behind it
        behind = torch.arange(k, device="cuda")[None] - \
            torch.arange(k - n, k, device="cuda")[:, None] > 0
        if op == "attend":
            pages = st["block_table"][b, :_ceil(k, case["page"])].long()
            rows = st["cache"][pages].flatten(0, 1)[:k].double()
            for i in range(n):
                s = st["scale"] * (st["q"][t + i].double() @ rows.t())
                s[:, behind[i]] = -math.inf
                out[t + i], lse[t + i] = _exact_rows(s, rows[:, :case["latent"]])
        else:
            kr = st["k_rope"][k0:k0 + k].double()
            for h in range(H):
                key = torch.cat([st["kv"][k0:k0 + k, h, :NOPE].double(), kr], dim=1)
                s = st["scale"] * (st["q"][t:t + n, h].double() @ key.t())
                if case["causal"]:
                    s.masked_fill_(behind, -math.inf)
                out[t:t + n, h], lse[t:t + n, h] = _exact_rows(
                    s, st["kv"][k0:k0 + k, h, NOPE:].double())
        t, k0 = t + n, k0 + k
    return {"out": out, "lse": lse}
