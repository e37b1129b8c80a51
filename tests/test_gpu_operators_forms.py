"""klt_quantize, klt_block_norm and klt_linear_* on the GPU: every kernel form at the sizes that
bring it out (several tiles for a CTA pair, several stagings of scales, two column sets of a thread),
the forms that are chosen by themselves, and rows whose offsets pass 32 bits.

Tolerances are those of test_gpu_operators."""
import numpy as np
import pytest
import torch

from latent_moe_layer_route_gb300 import binding as B
from test_gpu_operators import (BF16, EPS, F32, HALF, Lin, _cuda, _f64, _gen, _lib,  # noqa: F401
                                _norm_ref, _same, test_block_norm as block_norm_case)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- block norms

@pytest.mark.parametrize("case", [
    # aligned rows, two sets of 16 columns a thread: long bf16 rows ...
    (1300, 5120, BF16, BF16, "c", BF16, False, True, True, "hqs", 0),
    (1300, 4224, BF16, BF16, None, BF16, False, True, True, "hnqs", 0),
    (1300, 8192, BF16, BF16, "c", F32, True, True, True, "hnqs", 0),
    (1300, 8192, BF16, BF16, "c", BF16, True, True, True, "hnqs", 16),
    (1300, 4224, BF16, BF16, "t", BF16, True, False, False, "hnqs", 0),
    (1300, 6144, BF16, None, None, BF16, False, False, True, "nqs", 0),
    # ... and rows of more than 8192
    (160, 12800, BF16, BF16, "f", BF16, True, True, True, "hnqs", 0),
    (160, 12800, F32, BF16, "c", BF16, False, True, True, "hqs", 0),
    (160, 16384, F32, BF16, "t", F32, True, True, True, "hnqs", 0),
    (160, 8320, F32, None, None, BF16, False, False, True, "hnqs", 0),
    (160, 16384, BF16, BF16, None, BF16, False, True, True, "hn", 0),
    # long fp32 rows, and long bf16 rows with a gate of their own: one set
    (1300, 7168, F32, BF16, "c", BF16, True, True, True, "hnqs", 0),
    (1300, 7168, BF16, BF16, "f", BF16, True, True, True, "hnqs", 0),
    # rows on 16 bytes, not 32: two and four groups per half warp
    (1300, 2944, BF16, BF16, "c", BF16, True, True, True, "hnqs", 8),
    (1300, 5120, BF16, BF16, "f", BF16, False, True, True, "hnqs", 8),
    (1300, 5120, F32, BF16, "t", BF16, True, True, True, "hnqs", 4),
    # rows of any start, two sets of columns
    (200, 12001, F32, BF16, "c", BF16, True, True, True, "hnqs", 1),
    (200, 16383, BF16, BF16, "f", BF16, True, True, True, "hnqs", 0),
    # a block output or gate in fp32, and strided gates, in many rows of any start
    (1300, 2901, BF16, F32, "f", F32, True, True, True, "hnqs", 3),
    (1300, 5001, F32, F32, "x", BF16, False, True, True, "hnqs", 0),
    (300, 16383, F32, F32, "c", F32, True, True, True, "hnqs", 0),
], ids=lambda c: f"{c[0]}x{c[1]}-{c[4]}-{c[9]}-{c[10]}")
def test_block_norm_forms(case):
    block_norm_case(case)


@pytest.mark.parametrize("M,H", [(37, 1024), (1300, 5120), (1021, 1003)])
def test_block_norm_codes_are_those_of_n(M, H):
    """The codes times their scales are the unrounded n to half a code's step, and n in bf16 to
    half a step of its own more."""
    rng = _gen(3, M, H)
    h, y = _cuda(rng.standard_normal((M, H)), F32), _cuda(rng.standard_normal((M, H)), BF16)
    g = _cuda(rng.uniform(0.5, 1.5, H), BF16)
    G = -(-H // 128)
    n, q, s = torch.empty_like(y), B.fp8_codes(M, H, "cuda"), torch.empty((M, G), device="cuda")
    B.BlockNorm(H, g, g)(h, y, n=n, q=q, s=s)
    sr = np.repeat(s.cpu().numpy().astype(np.float64), 128, 1)[:, :H]
    back, n = _f64(q.contiguous()) * sr, _f64(n)
    exact = np.abs(n) * (1 + 2 * HALF[BF16])  # of the unrounded n, at most
    assert (np.abs(back - n) <= np.maximum(2.0 ** -4 * exact, 2.0 ** -10 * sr) +
            HALF[BF16] * exact + 80 * EPS * exact).all()


# ---------------------------------------------------------------- linear

@pytest.mark.parametrize("tile,act,out", [(t, "none", "f32") for t in (16, 32, 64, 128)] +
                         [(t, "swiglu", o) for t in (16, 32, 64) for o in ("fp8", "bf16")])
@pytest.mark.parametrize("split", [1, 2])
def test_linear_restages_scales(tile, act, out, split):
    """More k-blocks per part than scales are staged at once (16, 32 for tiles of 128)."""
    c = Lin(tile + 9, 256, 128 * (70 if tile == 128 else 37) + 16, act, out)
    c.check(c.layer(c.xq, c.xs, debug=B.KltLinearDebug(force_tile=tile, force_split=split)))
    c.close()


@pytest.mark.parametrize("M,N,K,act,out", [
    (2600, 4096, 256, "swiglu", "fp8"), (2600, 4096, 640, "swiglu", "bf16"),
    (2600, 4608, 130, "swiglu", "fp8"), (2600, 2100, 300, "none", "f32"),
    (5000, 2304, 512, "none", "bf16")])
@pytest.mark.parametrize("pad", [0, 16, 3])
def test_linear_wide_several_tiles_of_a_pair(M, N, K, act, out, pad):
    """More tiles than CTA pairs: the boxes, the group maxima and the scales of one tile follow
    those of another.  Rows on 16 bytes and not; nothing between them is written."""
    c = Lin(M, N, K, act, out)
    W = c.ref.shape[1]
    dt = {"bf16": BF16, "f32": F32, "fp8": torch.uint8}[out]
    base = torch.full((M + 1, W + pad), 77, dtype=dt, device="cuda")
    o_s = torch.full((M + 1, W // 128), -3.0, device="cuda") if out == "fp8" else None
    got = c.layer(c.xq, c.xs, base[:M, :W], None if o_s is None else o_s[:M],
                  debug=B.KltLinearDebug(force_tile=256, force_split=1))
    c.check(got)
    assert (base[M:] == 77).all() and (base[:, W:] == 77).all()
    assert o_s is None or (o_s[M:] == -3).all()
    c.close()


@pytest.mark.parametrize("M,N,K,act,out", [
    (300, 2048, 1500, "none", "bf16"), (777, 1003, 2090, "none", "f32"),
    (640, 1024, 4096, "swiglu", "fp8"), (1500, 200, 3000, "none", "f32"),
    (3000, 512, 1000, "swiglu", "bf16"), (4097, 384, 384, "none", "bf16"),
    (2048, 2560, 640, "swiglu", "fp8")])
def test_linear_forms_that_are_chosen(M, N, K, act, out):
    c = Lin(M, N, K, act, out)
    tile = c.layer.tile(M)
    got = c.layer(c.xq, c.xs)
    c.check(got)
    forced = c.layer(c.xq, c.xs, debug=B.KltLinearDebug(force_tile=tile % 1000,
                                                        force_split=tile // 1000))
    pick = (lambda g: g) if out == "fp8" else (lambda g: (g,))
    assert all(_same(a, b) for a, b in zip(pick(got), pick(forced)))
    c.close()


# ---------------------------------------------------------------- offsets beyond 32 bits

def _far(t, ld):
    """The same values in rows `ld` elements apart."""
    wide = torch.empty(((t.shape[0] - 1) * ld + t.shape[1],), dtype=t.dtype, device="cuda")
    v = wide.as_strided(t.shape, (ld, 1))
    v.copy_(t)
    return v


@pytest.mark.parametrize("M,K,ld", [(40, 300, 1 << 27), (4100, 300, (1 << 20) + 1),
                                    (20000, 256, 1 << 18), (4100, 1280, 1 << 20)])
def test_quantize_far_rows(M, K, ld):
    assert (M - 1) * ld > 1 << 32
    x = _cuda(_gen(31, M, K).standard_normal((M, K)), BF16)
    q, s = B.quantize_fp8(x)
    far = _far(torch.zeros((M, K), dtype=torch.uint8, device="cuda"), ld)
    _, s2 = B.quantize_fp8(_far(x, ld), far)
    assert torch.equal(far, q.view(torch.uint8)) and _same(s2, s)


@pytest.mark.parametrize("M,H,ld", [(40, 1000, 1 << 27), (40, 1024, 1 << 27),
                                    (4200, 1000, (1 << 20) + 2), (4200, 1024, 1 << 20),
                                    (4200, 4352, 1 << 20)])
def test_block_norm_far_rows(M, H, ld):
    assert (M - 1) * ld > 1 << 32
    rng = _gen(32, M, H)
    h, y, gate = (_cuda(rng.standard_normal((M, H)), BF16) for _ in range(3))
    g = _cuda(rng.uniform(0.5, 1.5, H), BF16)
    layer = B.BlockNorm(H, g, g, gate_sigmoid=True)
    outs = dict(h_out=torch.zeros_like(h), n=torch.zeros_like(h),
                q=torch.zeros((M, H), dtype=torch.uint8, device="cuda"))
    far = {k: _far(v, ld) for k, v in outs.items()}
    s, s2 = (torch.zeros((M, -(-H // 128)), device="cuda") for _ in range(2))
    layer(h, y, gate, s=s, **outs)
    layer(_far(h, ld), _far(y, ld), _far(gate, ld), s=s2, **far)
    assert all(_same(far[k], outs[k]) for k in outs) and _same(s, s2)


@pytest.mark.parametrize("tile", [16, 64, 256])
@pytest.mark.parametrize("act,out,N,more", [("none", "f32", 300, 0), ("none", "bf16", 256, 1),
                                            ("swiglu", "fp8", 512, 0), ("swiglu", "fp8", 512, 3)])
def test_linear_far_rows(tile, act, out, N, more):
    M, K, ld = 4200, 200, 1 << 20
    c = Lin(M, N, K, act, out)
    dbg = B.KltLinearDebug(force_tile=tile)
    pick = (lambda g: g) if out == "fp8" else (lambda g: (g,))
    want = pick(c.layer(c.xq, c.xs, debug=dbg))
    far = _far(torch.zeros_like(want[0]), ld + more)
    got = pick(c.layer(_far(c.xq, ld), c.xs, far, debug=dbg))
    assert all(_same(a, b) for a, b in zip(got, want))
    c.close()
