"""klt_quantize, klt_block_norm and klt_linear_* on the GPU: the ends of their ranges, and what a
call leaves to the next one when its waits run out."""
import numpy as np
import pytest
import torch

from latent_moe_layer_route_gb300 import binding as B
from test_gpu_operators import Lin, _lib, _same  # noqa: F401  (_lib: the module's fixture)

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
