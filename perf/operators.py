"""What is measured of the operators around the mixture-of-experts tail: the norms before and
after a block, the e4m3 activation quantiser and the FP8 linear layer with block scales.

    h', n   = the join of two blocks: u = RMSNorm(y) gamma_post, h' = a h + b gate u,
              n = RMSNorm(h') gamma_pre, as bf16 and/or as e4m3 codes with a scale per 128
    q, s    = e4m3 codes and fp32 scales (amax / 448) of a tensor per row and 128 columns
    out     = x W^T of e4m3 operands, x with a scale per row and 128 columns, W with a scale
              per 128 x 128 block; as bf16 or fp32, or through SwiGLU to e4m3 and scales

With `own` false `run` computes them by elementary torch operations in 32 bits, with `own`
true by the framework's calls.
"""
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
GROUP = 128
EPS = 1e-6


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one token between two decoder blocks of the full width: pure latency
        dict(name="join_m1", op="join", M=1, H=7168, h="bf16", post=True, gate="none",
             sigmoid=False, out="bf16", pad=0),
        # a decode batch entering an FP8 layer, the residual stream kept in fp32
        dict(name="join_m16_fp8", op="join", M=16, H=7168, h="f32", post=True,
             gate="channel", sigmoid=False, out="fp8", pad=0),
        # a batch of odd size and width in a padded buffer, a sigmoid gate for each token
        dict(name="join_m1021_ragged", op="join", M=1021, H=2901, h="bf16", post=True,
             gate="token", sigmoid=True, out="both", pad=11),
        # a prefill batch: nothing but memory traffic
        dict(name="join_m8192_fp8", op="join", M=8192, H=7168, h="bf16", post=True,
             gate="channel", sigmoid=False, out="fp8", pad=0),
        # a decode batch's latent input
        dict(name="quant_m16", op="quant", M=16, K=3584, x="bf16", pad=0),
        # a prefill batch's hidden state
        dict(name="quant_m8192", op="quant", M=8192, K=7168, x="bf16", pad=0),
        # one token through a down projection
        dict(name="linear_m1", op="linear", M=1, N=7168, K=2048, act="none", out="bf16"),
        # a decode batch through the gate and up projections of a dense layer
        dict(name="linear_m16_swiglu", op="linear", M=16, N=4096, K=7168, act="swiglu",
             out="fp8"),
        # a larger decode batch through a square projection
        dict(name="linear_m128", op="linear", M=128, N=7168, K=7168, act="none", out="bf16"),
        # odd sizes in every direction, and an fp32 result (logits)
        dict(name="linear_m777_ragged", op="linear", M=777, N=1003, K=2090, act="none",
             out="f32"),
        # prefill, latent width to hidden width
        dict(name="linear_m4096", op="linear", M=4096, N=7168, K=3584, act="none",
             out="bf16"),
        # prefill through the gate and up projections
        dict(name="linear_m8192_swiglu", op="linear", M=8192, N=4096, K=7168, act="swiglu",
             out="fp8"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["join", "quant", "linear", "linear"])
    M = _log(rng, 1, 8192)
    if op == "join":
        H = rng.choice([128 * rng.randint(2, 64), 8 * rng.randint(32, 1024),
                        rng.randint(256, 8192)])
        return dict(op=op, M=M, H=H, h=rng.choice(["bf16", "f32"]),
                    post=rng.random() < 0.7,
                    gate=rng.choice(["none", "channel", "token", "full"]),
                    sigmoid=rng.random() < 0.5, out=rng.choice(["bf16", "fp8", "both"]),
                    pad=rng.choice([0, 0, 8, 5]))
    if op == "quant":
        K = rng.choice([128 * rng.randint(1, 64), rng.randint(128, 8192)])
        return dict(op=op, M=M, K=K, x=rng.choice(["bf16", "f32"]),
                    pad=rng.choice([0, 0, 8, 5]))
    swiglu = rng.random() < 0.5
    while True:
        N = 256 * rng.randint(1, 32) if swiglu else \
            rng.choice([128 * rng.randint(1, 64), _log(rng, 64, 8192)])
        K = rng.choice([128 * rng.randint(1, 64), _log(rng, 64, 8192)])
        if M * N * K <= 8192 * 4096 * 7168:  # no more work than the largest listed case
            break
    out = rng.choice(["fp8", "bf16"]) if swiglu else rng.choice(["bf16", "f32"])
    return dict(op=op, M=M, N=N, K=K, act="swiglu" if swiglu else "none", out=out)


# ---------------------------------------------------------------- inputs

def _ceil(a, b):
    return -(-a // b)


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _rows(gen, M, C, dtype, pad=0):
    """[M, C] activations: normal values, a few channels larger by an order, each row at a
    scale of its own; a view of a wider buffer where `pad` is not 0."""
    v = torch.randn(M, C + pad, generator=gen, device="cuda")
    channel = torch.rand(C + pad, generator=gen, device="cuda")
    v *= torch.where(channel < 0.02, 8.0, 1.0)
    v *= torch.exp(torch.randn(M, 1, generator=gen, device="cuda") * 0.5)
    return v.to(dtype)[:, :C]


def _quantized(v):
    """e4m3 codes and fp32 scales of v per row and 128 columns, in memory whose rows start on
    16 bytes."""
    M, K = v.shape
    q, s = _quant(v.float())
    wide = torch.zeros(M, _ceil(K, 16) * 16, dtype=torch.uint8, device=v.device)
    wide[:, :K] = q.view(torch.uint8)
    return wide.view(E4M3)[:, :K], s


def _weights(gen, N, K):
    """e4m3 codes [N, K] and fp32 scales of 128 x 128 blocks of normal weights, whose blocks
    differ in size."""
    nb, kb = _ceil(N, GROUP), _ceil(K, GROUP)
    w = torch.randn(nb * GROUP, kb * GROUP, generator=gen, device="cuda") / math.sqrt(K)
    w = w.view(nb, GROUP, kb, GROUP)
    w *= torch.exp(torch.randn(nb, 1, kb, 1, generator=gen, device="cuda") * 0.3)
    s = w.abs().amax(dim=(1, 3)) / E4M3_MAX
    q = (w / s[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3)
    q = q.view(torch.uint8).reshape(nb * GROUP, kb * GROUP)[:N, :K].contiguous()
    return q.view(E4M3), s


def _codes(M, C):
    """An empty e4m3 tensor [M, C] whose rows start on 16 bytes."""
    return torch.empty(M, _ceil(C, 16) * 16, dtype=torch.uint8, device="cuda").view(E4M3)[:, :C]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, M = case["op"], case["M"]
    st = dict(case=dict(case))
    if op == "join":
        H, pad = case["H"], case["pad"]
        st["h"] = _rows(gen, M, H, _dtype(case["h"]), pad)
        st["y"] = _rows(gen, M, H, torch.bfloat16, pad)
        st["gamma_post"] = (torch.rand(H, generator=gen, device="cuda") + 0.5).bfloat16() \
            if case["post"] else None
        st["gamma_pre"] = (torch.rand(H, generator=gen, device="cuda") + 0.5).bfloat16()
        shape = {"none": None, "channel": (1, H), "token": (M, 1), "full": (M, H)}[case["gate"]]
        st["gate"] = None if shape is None else \
            torch.randn(shape, generator=gen, device="cuda").bfloat16()
        st["res_scale"], st["branch_scale"] = 0.75, 1.25
        st["h_out"] = torch.empty(M, H, dtype=_dtype(case["h"]), device="cuda")
        st["n"] = torch.empty(M, H, dtype=torch.bfloat16, device="cuda") \
            if case["out"] != "fp8" else None
        st["q"] = _codes(M, H) if case["out"] != "bf16" else None
        st["s"] = torch.empty(M, _ceil(H, GROUP), device="cuda") \
            if case["out"] != "bf16" else None
        if own:
            from latent_moe_layer_route_gb300 import binding
            st["layer"] = binding.BlockNorm(
                H, gamma_post=st["gamma_post"], gamma_pre=st["gamma_pre"], eps=EPS,
                res_scale=st["res_scale"], branch_scale=st["branch_scale"],
                gate_sigmoid=case["sigmoid"])
    elif op == "quant":
        st["x"] = _rows(gen, M, case["K"], _dtype(case["x"]), case["pad"])
        st["q"] = _codes(M, case["K"])
        st["s"] = torch.empty(M, _ceil(case["K"], GROUP), device="cuda")
    else:
        N, K = case["N"], case["K"]
        st["xq"], st["xs"] = _quantized(_rows(gen, M, K, torch.float32))
        st["wq"], st["ws"] = _weights(gen, N, K)
        width = N // 2 if case["act"] == "swiglu" else N
        st["out"] = _codes(M, width) if case["out"] == "fp8" else \
            torch.empty(M, width, dtype=_dtype(case["out"]), device="cuda")
        st["out_s"] = torch.empty(M, _ceil(width, GROUP), device="cuda") \
            if case["out"] == "fp8" else None
        if own:
            from latent_moe_layer_route_gb300 import binding
            st["layer"] = binding.Fp8Linear(st["wq"], st["ws"], act=case["act"],
                                            out=case["out"])
    return st


# ---------------------------------------------------------------- plain forms (32 bits)

def _quant(v):
    """e4m3 codes and fp32 scales of fp32 v [M, C] per row and 128 columns: scale amax / 448
    (1 where that is 0), codes of the fp32 quotient, saturating."""
    M, C = v.shape
    groups = _ceil(C, GROUP)
    g = torch.nn.functional.pad(v, (0, groups * GROUP - C)).view(M, groups, GROUP)
    s = g.abs().amax(dim=-1) / E4M3_MAX
    s = torch.where(s == 0, torch.ones_like(s), s)
    q = (g / s[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3)
    return q.view(torch.uint8).reshape(M, groups * GROUP)[:, :C].contiguous().view(E4M3), s


def _rms(v, gamma):
    r = torch.rsqrt(v.square().mean(dim=-1, keepdim=True) + EPS)
    return v * r * gamma.float()


def _plain_join(st):
    case = st["case"]
    u = st["y"].float()
    if st["gamma_post"] is not None:
        u = _rms(u, st["gamma_post"])
    if st["gate"] is not None:
        gate = st["gate"].float()
        u = u * (1.0 / (1.0 + torch.exp(-gate)) if case["sigmoid"] else gate)
    h = st["h"].float() * st["res_scale"] + u * st["branch_scale"]
    n = _rms(h, st["gamma_pre"])
    got = {"h": h.to(st["h"].dtype)}
    if case["out"] != "fp8":
        got["n"] = n.bfloat16()
    if case["out"] != "bf16":
        got["q"], got["s"] = _quant(n)
    return got


def _plain_linear(st):
    case = st["case"]
    M, K = st["xq"].shape
    N = st["wq"].shape[0]
    x = st["xq"].float() * st["xs"].repeat_interleave(GROUP, 1)[:, :K]
    w = st["wq"].float() * st["ws"].repeat_interleave(GROUP, 0)[:N].repeat_interleave(
        GROUP, 1)[:, :K]
    v = x @ w.t()
    if case["act"] == "swiglu":
        g, u = v[:, :N // 2], v[:, N // 2:]
        v = g / (1.0 + torch.exp(-g)) * u
    if case["out"] == "fp8":
        q, s = _quant(v)
        return {"q": q, "s": s}
    return {"out": v.to(_dtype(case["out"]))}


def _plain(st):
    op = st["case"]["op"]
    if op == "join":
        return _plain_join(st)
    if op == "quant":
        q, s = _quant(st["x"].float())
        return {"q": q, "s": s}
    return _plain_linear(st)


# ---------------------------------------------------------------- the framework's calls

def _own(st):
    case = st["case"]
    if case["op"] == "join":
        st["layer"](st["h"], st["y"], st["gate"], h_out=st["h_out"], n=st["n"], q=st["q"],
                    s=st["s"])
        got = {"h": st["h_out"]}
        if case["out"] != "fp8":
            got["n"] = st["n"]
        if case["out"] != "bf16":
            got["q"], got["s"] = st["q"], st["s"]
        return got
    if case["op"] == "quant":
        from latent_moe_layer_route_gb300 import binding
        q, s = binding.quantize_fp8(st["x"], st["q"], st["s"])
        return {"q": q, "s": s}
    if case["out"] == "fp8":
        q, s = st["layer"](st["xq"], st["xs"], st["out"], st["out_s"])
        return {"q": q, "s": s}
    return {"out": st["layer"](st["xq"], st["xs"], st["out"])}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- what it cannot do without

def work(case):
    M = case["M"]
    if case["op"] == "join":
        H = case["H"]
        hb = 2 if case["h"] == "bf16" else 4
        out = (2 * H if case["out"] != "fp8" else 0) + \
            (H + 4 * _ceil(H, GROUP) if case["out"] != "bf16" else 0)
        gate = {"none": 0, "channel": 2 * H, "token": 2 * M, "full": 2 * M * H}[case["gate"]]
        return dict(bytes=M * (2 * H + 2 * hb * H + out) + gate +
                    2 * H * (2 if case["post"] else 1), flops=12 * M * H)
    if case["op"] == "quant":
        K = case["K"]
        return dict(bytes=M * (K * (2 if case["x"] == "bf16" else 4) + K +
                               4 * _ceil(K, GROUP)), flops=4 * M * K)
    N, K = case["N"], case["K"]
    width = N // 2 if case["act"] == "swiglu" else N
    out = width + 4 * _ceil(width, GROUP) if case["out"] == "fp8" else \
        width * (2 if case["out"] == "bf16" else 4)
    kb = _ceil(K, GROUP)
    return dict(bytes=M * (K + 4 * kb) + N * K + 4 * _ceil(N, GROUP) * kb + M * out,
                flops=2 * M * N * K)


# ---------------------------------------------------------------- the definition in 64 bits

def _e4m3_value(v):
    """The e4m3 value nearest to 64-bit v, ties to even, saturating: steps of 2^(e - 3) in
    the binade e, never below 2^-9."""
    mag = v.abs()
    _, ex = torch.frexp(mag)
    step = torch.ldexp(torch.ones_like(v), (ex - 1).clamp(min=-6) - 3)
    return torch.sign(v) * (torch.round(mag / step) * step).clamp(max=E4M3_MAX)


def _exact_codes(v):
    M, C = v.shape
    out, scales = torch.empty_like(v), []
    for lo in range(0, C, GROUP):
        g = v[:, lo:lo + GROUP]
        s = g.abs().max(dim=1).values / 448
        s = torch.where(s.float() == 0, torch.ones_like(s), s)
        out[:, lo:lo + GROUP] = _e4m3_value(g / s.float().double()[:, None])
        scales.append(s)
    return out, torch.stack(scales, dim=1)


def _exact_norm(v, gamma):
    return v / torch.sqrt((v * v).sum(1) / v.shape[1] + EPS)[:, None] * gamma.double()


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "quant":
        q, s = _exact_codes(st["x"].double())
        return {"q": q, "s": s}
    if case["op"] == "join":
        u = st["y"].double()
        if st["gamma_post"] is not None:
            u = _exact_norm(u, st["gamma_post"])
        if st["gate"] is not None:
            gate = st["gate"].double()
            u = u * (torch.sigmoid(gate) if case["sigmoid"] else gate)
        h = st["res_scale"] * st["h"].double() + st["branch_scale"] * u
        n = _exact_norm(h, st["gamma_pre"])
        got = {"h": h}
        if case["out"] != "fp8":
            got["n"] = n
        if case["out"] != "bf16":
            got["q"], got["s"] = _exact_codes(n)
        return got
    # the matrix product block by block: each 128 columns of K, scaled as their blocks say
    M, N, K = case["M"], case["N"], case["K"]
    v = torch.zeros(M, N, dtype=torch.float64, device="cuda")
    for b, lo in enumerate(range(0, K, GROUP)):
        x = st["xq"][:, lo:lo + GROUP].double() * st["xs"][:, b].double()[:, None]
        rows = torch.arange(N, device="cuda") // GROUP
        w = st["wq"][:, lo:lo + GROUP].double() * st["ws"][rows, b].double()[:, None]
        v.addmm_(x, w.t())
    if case["act"] == "swiglu":
        g, u = v[:, :N // 2], v[:, N // 2:]
        v = g * torch.sigmoid(g) * u
    if case["out"] == "fp8":
        q, s = _exact_codes(v)
        return {"q": q, "s": s}
    return {"out": v}
