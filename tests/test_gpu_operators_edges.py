"""klt_quantize, klt_block_norm and klt_linear_* on the GPU: the ends of their ranges, and what a
call leaves to the next one when its waits run out."""
import threading
import time

import numpy as np
import pytest
import torch

import parity_util as PU
from latent_moe_layer_route_gb300 import binding as B
from latent_moe_layer_route_gb300 import configs, inputs
from test_gpu_operators import EPS, Lin, _lib, _same  # noqa: F401  (_lib: the module's fixture)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- waits that run out

@pytest.mark.parametrize("tile,split,act,out", [
    (16, 2, "swiglu", "fp8"), (16, 8, "swiglu", "fp8"), (32, 4, "none", "bf16"),
    (64, 8, "swiglu", "bf16"), (64, 2, "none", "f32"), (128, 2, "none", "bf16"),
    (128, 4, "none", "f32")])
@pytest.mark.parametrize("stall", [1, 3])
def test_narrow_parts_that_come_late(tile, split, act, out, stall):
    """The CTAs of a cluster give up and still store their parts into one another's memory; the
    launches right behind them, which take over that memory, have the right results."""
    bad, ok = (Lin(130, 512, 128 * 40, act, out, seed=s) for s in (2, 3))
    form = dict(force_tile=tile, force_split=split)
    want = ok.layer(ok.xq, ok.xs, debug=B.KltLinearDebug(**form))
    ok.check(want)
    torch.cuda.synchronize()
    bad.layer(bad.xq, bad.xs, debug=B.KltLinearDebug(stall_after_kblocks=stall, timeout_ms=5, **form))
    got = [ok.layer(ok.xq, ok.xs, debug=B.KltLinearDebug(**form)) for _ in range(4)]
    torch.cuda.synchronize()
    assert bad.layer.status() == B.KLT_ERR_DEVICE_TIMEOUT
    pick = (lambda g: g) if out == "fp8" else (lambda g: (g,))
    for g in got:
        assert all(_same(a, b) for a, b in zip(pick(g), pick(want)))
    bad.layer.close()
    ok.close()


@pytest.mark.parametrize("act,out", [("none", "f32"), ("swiglu", "fp8")])
@pytest.mark.parametrize("M,N,split,stall", [
    (600, 512, 1, 1), (600, 512, 1, 4), (600, 512, 1, 7),  # before, at and after the stages' reuse
    (600, 512, 2, 1), (600, 512, 2, 4),  # parts of 4 and 5 k-blocks: the second one stops
    (2600, 2048, 1, 12)])  # in the second tile of the pairs that have one
def test_wide_pairs_that_give_up(M, N, split, stall, act, out):
    """The same for the CTA pairs of the token-major kernel."""
    bad, ok = (Lin(M, N, 128 * 9, act, out, seed=s) for s in (2, 3))
    form = dict(force_tile=256, force_split=split)
    want = ok.layer(ok.xq, ok.xs, debug=B.KltLinearDebug(**form))
    ok.check(want)
    torch.cuda.synchronize()
    bad.layer(bad.xq, bad.xs, debug=B.KltLinearDebug(stall_after_kblocks=stall, timeout_ms=5, **form))
    got = [ok.layer(ok.xq, ok.xs, debug=B.KltLinearDebug(**form)) for _ in range(4)]
    torch.cuda.synchronize()
    assert bad.layer.status() == B.KLT_ERR_DEVICE_TIMEOUT
    pick = (lambda g: g) if out == "fp8" else (lambda g: (g,))
    for g in got:
        assert all(_same(a, b) for a, b in zip(pick(g), pick(want)))
    bad.layer.close()
    ok.close()


@pytest.mark.parametrize("tile", [16, 256])
def test_the_bound_of_a_wait_does_not_count_the_launch_before(tile):
    """A launch that outlasts the next one's bound on its waits and leaves SMs free for it: one tile
    of 8192 k-blocks, some 3 ms, before a layer whose waits are bounded by 1 ms."""
    K = 1 << 20
    codes = torch.randint(0x30, 0x38, (256, K), dtype=torch.uint8, device="cuda")
    x = torch.randint(0x30, 0x38, (200, K), dtype=torch.uint8, device="cuda")
    slow = B.Fp8Linear(codes, torch.ones(2, K // 128, device="cuda"), out="f32")
    xs = torch.ones(200, K // 128, device="cuda")
    c = Lin(100, 256, 640, "none", "f32")
    dbg = B.KltLinearDebug(force_tile=tile, force_split=1, timeout_ms=1)
    c.check(c.layer(c.xq, c.xs, debug=dbg))
    torch.cuda.synchronize()
    out = torch.empty(200, 256, device="cuda")
    first, last = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    first.record()
    slow(x, xs, out, debug=B.KltLinearDebug(force_tile=256, force_split=1))
    last.record()
    torch.cuda.synchronize()
    assert first.elapsed_time(last) > 1.5  # ms
    for _ in range(3):
        slow(x, xs, out, debug=B.KltLinearDebug(force_tile=256, force_split=1))
        got = c.layer(c.xq, c.xs, debug=dbg)
        torch.cuda.synchronize()
        assert c.layer.status() == B.KLT_OK
        c.check(got)
    slow.close()
    c.close()


# ---------------------------------------------------------------- streams

def _late_writer(nbytes):
    """Memory of `nbytes` that torch may hand out again on the current stream, on which work that
    writes it is still queued."""
    torch.empty(64, dtype=torch.uint8, device="cuda").fill_(0)  # loads the kernel
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    blocks = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in nbytes]
    torch.cuda._sleep(100_000_000)  # some 50 ms
    for b in blocks:
        b.fill_(0x55)


@pytest.mark.parametrize("op", ["quantize", "norm", "linear", "linear_codes", "tail", "hidden"])
def test_outputs_of_a_call_on_a_given_stream(op):
    """What a call with `stream` allocates belongs to that stream: not to the current one, where
    work that still uses it may be queued."""
    M, H = 2048, 8192
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((M, H), device="cuda", generator=g).bfloat16()
    close = lambda: None  # noqa: E731
    if op == "quantize":
        sizes, call = (M * H, M * H // 32), lambda **k: B.quantize_fp8(x, **k)
    elif op == "norm":
        sizes, layer = (2 * M * H, 2 * M * H), B.BlockNorm(H, res_scale=0.5)
        call = lambda **k: layer(x, x, **k)[:2]  # noqa: E731
    elif op.startswith("linear"):
        act, out, N = ("swiglu", "fp8", 8192) if op == "linear_codes" else ("none", "f32", 4096)
        c = Lin(M, N, 256, act, out)
        sizes = (M * N // 2, M * N // 64) if out == "fp8" else (M * N * 4,)
        call, close = (lambda **k: c.layer(c.xq, c.xs, **k)), c.close
    else:
        cfg = configs.SMALL.with_(M=3000, E=8, topk=3, seed=41)
        act, w = inputs.make_inputs(cfg)
        w.update(inputs.make_projection_weights(cfg))
        tail = B.LatentMoETail(cfg, PU.to_cuda(w), flags=B.KLT_FLAG_DETERMINISTIC)
        a = PU.to_cuda(act)
        sizes, close = (2 * cfg.M * cfg.H,), tail.close
        call = (lambda **k: tail.forward(a["x"], a["z"], a["logits"], **k)) if op == "tail" else \
            (lambda **k: tail.forward_hidden(a["x"], **k))
    outs = lambda r: r if isinstance(r, tuple) else (r,)  # noqa: E731
    want = [t.clone() for t in outs(call())]
    side = torch.cuda.Stream()
    _late_writer(sizes)
    got = outs(call(stream=side.cuda_stream))
    torch.cuda.synchronize()
    assert all(_same(a, b) for a, b in zip(got, want))
    got = outs(call(stream=0))  # the default stream
    torch.cuda.synchronize()
    assert all(_same(a, b) for a, b in zip(got, want))
    close()


@pytest.mark.parametrize("op", ["quantize", "norm", "linear"])
def test_other_threads_run_while_a_launch_waits(op):
    """A call that waits for room in the stream's queue does not stop Python's other threads."""
    c = Lin(4, 256, 256, "none", "f32")
    x = torch.zeros((4, 256), device="cuda")
    layer, n = B.BlockNorm(256), torch.empty((4, 256), device="cuda", dtype=torch.bfloat16)
    q, s = B.fp8_codes(4, 256, "cuda"), torch.empty((4, 2), device="cuda")
    out = torch.empty((4, 256), device="cuda")
    call = {"quantize": lambda: B.quantize_fp8(x, q, s), "norm": lambda: layer(x, n=n),
            "linear": lambda: c.layer(c.xq, c.xs, out)}[op]
    for _ in range(3):
        call()
    torch.cuda._sleep(1)
    torch.cuda.synchronize()
    stop, gaps = threading.Event(), []

    def tick():
        last = time.perf_counter()
        while not stop.is_set():
            time.sleep(0.001)
            now = time.perf_counter()
            gaps.append(now - last)
            last = now

    clock = threading.Thread(target=tick)
    clock.start()
    torch.cuda._sleep(1_000_000_000)  # some 0.5 s
    slowest = 0.0
    for _ in range(4000):
        t0 = time.perf_counter()
        call()
        slowest = max(slowest, time.perf_counter() - t0)
    torch.cuda.synchronize()
    stop.set()
    clock.join()
    c.close()
    assert slowest > 0.2  # a call did wait
    assert max(gaps) < slowest / 2


# ---------------------------------------------------------------- sigmoid gates

@pytest.mark.parametrize("gate", ["channel", "token", "full", "strided"])
@pytest.mark.parametrize("M,H,pad", [(3, 256, 0), (5, 301, 0), (200, 8192, 0), (1400, 1001, 0),
                                     (1300, 6144, 0), (200, 8192, 8)])
@pytest.mark.parametrize("gd", [torch.bfloat16, torch.float32])
def test_sigmoid_gates_that_are_no_numbers(M, H, pad, gate, gd):
    """A gate of NaN gives NaN, an infinite one 0 or 1, whichever kernel takes the row."""
    shape = {"channel": (1, H), "token": (M, 1), "full": (M, H), "strided": (M, 2 * H)}[gate]
    g = torch.zeros(shape, device="cuda", dtype=gd)
    if gate == "strided":
        g = g[:, ::2]
    rows, cols = g.shape
    for i, v in enumerate((float("nan"), float("inf"), -float("inf"))):
        g[i % rows, (3 + 5 * i) % cols] = v
    h = torch.zeros((M, H + pad), device="cuda")[:, :H]
    y = torch.ones((M, H + pad), device="cuda", dtype=torch.bfloat16)[:, :H]
    out = torch.empty((M, H), device="cuda")
    B.BlockNorm(H, gate_sigmoid=True)(h, y, g, h_out=out)
    torch.testing.assert_close(out, torch.sigmoid(g.float()).expand(M, H), rtol=1e-6, atol=0,
                               equal_nan=True)


@pytest.mark.parametrize("gate", ["channel", "token", "full", "strided"])
@pytest.mark.parametrize("M,H,pad", [(3, 256, 0), (5, 301, 0), (200, 8192, 0), (1400, 1001, 0),
                                     (1300, 6144, 0), (200, 8192, 8)])
def test_sigmoid_gates_over_their_range(M, H, pad, gate):
    """u sigmoid(g) of u = 1 into an fp32 stream.  An exponential within 2 ulp (4 EPS) and a
    reciprocal within 1 (2 EPS), an addition, a product of the two and a multiply-add: 9 EPS of the
    value, with one more for the product with u; where e^g is subnormal, its steps of 2^-149 too."""
    shape = {"channel": (1, H), "token": (M, 1), "full": (M, H), "strided": (M, 2 * H)}[gate]
    rng = np.random.default_rng([7, M, H, pad])
    g = torch.from_numpy(rng.uniform(-104, 104, shape).astype(np.float32)).cuda()
    if gate == "strided":
        g = g[:, ::2]
    h = torch.zeros((M, H + pad), device="cuda")[:, :H]
    y = torch.ones((M, H + pad), device="cuda", dtype=torch.bfloat16)[:, :H]
    out = torch.empty((M, H + pad), device="cuda")[:, :H]
    B.BlockNorm(H, gate_sigmoid=True)(h, y, g, h_out=out)
    want = torch.sigmoid(g.double()).expand(M, H)
    assert ((out.double() - want).abs() <= 10 * EPS * want + 2.0 ** -148).all()


# ---------------------------------------------------------------- SwiGLU

def _swiglu_of_scales(g, u_over_g, tile):
    """silu(g) u of gates g and up values u = g * u_over_g: codes of 1, so that a product is its
    scale.  Returns (bf16 outputs, codes, scales); all 128 columns of a row are equal."""
    M = len(g)
    one = torch.zeros((256, 128), dtype=torch.uint8, device="cuda")
    one[:, 0] = 0x38
    xq = torch.zeros((M, 128), dtype=torch.uint8, device="cuda")
    xq[:, 0] = 0x38
    xs = torch.from_numpy(np.asarray(g, dtype=np.float32)).cuda()[:, None]
    ws = torch.tensor([[1.0], [u_over_g]], device="cuda")
    dbg = B.KltLinearDebug(force_tile=tile)
    out = B.Fp8Linear(one, ws, "swiglu", "bf16")(xq, xs, debug=dbg)
    q, s = B.Fp8Linear(one, ws, "swiglu", "fp8")(xq, xs, debug=dbg)
    assert (out.view(torch.int16) == out.view(torch.int16)[:, :1]).all()
    return out[:, 0].double().cpu().numpy(), q[:, 0].cpu(), s[:, 0].double().cpu().numpy()


@pytest.mark.parametrize("tile", [16, 32, 64, 256])
def test_swiglu_of_gates_far_below_zero(tile):
    """silu runs to 0 there: nothing is left of it, whatever the up value, and a group of it is
    zeros with a scale of 1; of an infinite gate the definition is NaN."""
    far = np.array([-200.0, -600.0, -1e4, -1e10, -1e30, -3e38])
    out, q, s = _swiglu_of_scales(np.concatenate([far, [-np.inf, np.nan, 1e4]]), 1.0, tile)
    n = len(far)
    assert (out[:n] == 0).all() and (s[:n] == 1).all()
    assert (q[:n].view(torch.uint8) & 0x7F == 0).all()
    assert np.isnan(out[n:n + 2]).all() and not np.isfinite(s[n:n + 2]).any()
    assert abs(out[-1] / 1e8 - 1) <= 2.0 ** -8 and abs(s[-1] * 448 / 1e8 - 1) <= 4 * EPS


@pytest.mark.parametrize("tile", [16, 32, 64, 256])
def test_swiglu_over_the_gates_range(tile):
    """The scale of a group of equal values is their magnitude over 448, in fp32: an exponential
    within 2 ulp (4 EPS), a reciprocal within 1 (2 EPS), an addition, three products, the division
    by 448 and its inputs' own products with their scales (exact here): 12 EPS, and the steps of
    2^-149 of a subnormal e^g times |g u| / 448, and of the scale itself."""
    rng = np.random.default_rng([8, tile])
    g = np.concatenate([rng.uniform(-104, 104, 900), rng.uniform(-20, 5, 900)]).astype(np.float32)
    out, q, s = _swiglu_of_scales(g, 0.5, tile)
    g = g.astype(np.float64)
    want = np.abs(g / (1 + np.exp(-g)) * g * 0.5) / 448
    err = 12 * EPS * want + 2.0 ** -148 * (g * g * 0.5 / 448 + 1)
    zero = want + err < 2.0 ** -148  # the scale of nothing is 1
    assert ((np.abs(s - want) <= err) | (zero & (s == 1))).all()


# ---------------------------------------------------------------- sizes beyond 32 bits

def test_a_layers_sizes_are_not_cut_to_32_bits():
    """2^32 + 256 rows of weights are more than a layer takes; cut to 32 bits they would be 256."""
    N = (1 << 32) + 256
    w = torch.zeros((N, 1), dtype=torch.uint8, device="cuda")
    s = torch.ones((N // 128, 1), device="cuda")
    with pytest.raises(B.KltError) as e:
        B.Fp8Linear(w, s)
    assert e.value.code == B.KLT_ERR_UNSUPPORTED
