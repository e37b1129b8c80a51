"""klt_quantize, klt_block_norm and klt_linear_* on the GPU against plain 64-bit forms.

Tolerances (EPS = 2^-24, half a step of fp32; HALF[t] half a step of an output type):
  * quantiser: bit for bit (its definition is in fp32 and has no sums);
  * norms: a sum of H squares in fp32, all positive, taken as at most 32 terms per thread and
    two trees of 5 levels, then division, square root and reciprocal: under 50 EPS relative
    on the sum, half of that on its root, so 40 EPS covers a norm with its two products; the
    gate's exponential (2 ulp) and division stay in the same 40 EPS;
  * linear: per 128 columns the tensor core's fp32 sum, then one product with the scale
    (itself rounded) and KB additions: (KB + 24) EPS of sum |x w|;
  * SwiGLU of values off by e: |silu'| < 1.1, so 1.1 |u| e_g + |silu(g)| e_u + 16 EPS |v|;
  * e4m3 codes: half a step, 2^-4 of the value, or 2^-10 scales where codes are subnormal.
"""
import numpy as np
import pytest
import torch

from latent_moe_layer_route_gb300 import binding as B
from latent_moe_layer_route_gb300 import build, configs, inputs
from oracle import model as T
from oracle.codecs import e4m3_decode, e4m3_encode
import parity_util as PU

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    B.load_library()


def _gen(*seed):
    return np.random.default_rng(seed)


def _cuda(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda().to(dtype)


def _padded(t, pad):
    """The same values in rows `pad` elements further apart; the gaps hold NaN (zero codes)."""
    M, C = t.shape
    wide = torch.zeros((M, C + pad), dtype=t.dtype, device=t.device)
    if t.dtype in (BF16, F32):
        wide.fill_(float("nan"))
    wide[:, :C] = t
    return wide[:, :C]


def _f64(t):
    return t.cpu().to(torch.float64).numpy() if t.dtype in (BF16, F32) else \
        e4m3_decode(t.cpu().view(torch.uint8).numpy())


def _bits(t):
    return t.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def _same(a, b):
    return torch.equal(_bits(a), _bits(b))


def _offset_rows(M, C, dtype, pad, off, fill):
    """Rows that start `off` elements into their buffer and end `pad` before the next one."""
    base = torch.full((off + M * (C + pad) + 16,), fill, device="cuda",
                      dtype=torch.uint8 if dtype is None else dtype)
    return base.as_strided((M, C), (C + pad, 1), off), base


def _untouched(view, base, fill):
    rest = base.clone()
    rest.as_strided(view.shape, view.stride(), view.storage_offset()).fill_(fill)
    return bool((rest == fill).all())


# ---------------------------------------------------------------- quantiser

def _quant_ref(x32):
    """codes and scales of fp32 x by the definition, in fp32 (one rounding per operation)."""
    M, K = x32.shape
    G = -(-K // 128)
    codes = np.zeros((M, K), dtype=np.uint8)
    scales = np.zeros((M, G), dtype=np.float32)
    for g in range(G):
        v = x32[:, g * 128:(g + 1) * 128]
        s = (np.abs(v).max(axis=1) / np.float32(448.0)).astype(np.float32)
        s = np.where(s == 0, np.float32(1), s)
        scales[:, g] = s
        codes[:, g * 128:(g + 1) * 128] = e4m3_encode((v / s[:, None]).astype(np.float32))
    return codes, scales


@pytest.mark.parametrize("M,K,dtype,pad", [
    (700, 7168, F32, 0), (3001, 2048, BF16, 16), (3000, 2048, BF16, 8), (1, 128, BF16, 0), (1, 1, BF16, 0), (3, 127, F32, 0), (5, 129, BF16, 3), (16, 3584, BF16, 0),
    (7, 1000, F32, 8), (33, 136, BF16, 8), (2, 8, F32, 1), (700, 7168, BF16, 0),
    (300, 4099, F32, 5)])
def test_quantize(M, K, dtype, pad):
    rng = _gen(1, M, K)
    x = rng.standard_normal((M, K)) * np.exp(2 * rng.standard_normal((M, 1)))
    x[:, rng.integers(0, K)] *= 30
    xt = _padded(_cuda(x, dtype), pad)
    q = _padded(torch.zeros((M, K), dtype=torch.uint8, device="cuda"), 8 + pad)
    q._base.fill_(0xA5)
    s = torch.full((M, -(-K // 128)), -1.0, device="cuda")
    B.quantize_fp8(xt, q, s)
    codes, scales = _quant_ref(xt.cpu().float().numpy())
    np.testing.assert_array_equal(s.cpu().numpy(), scales)
    np.testing.assert_array_equal(q.cpu().numpy(), codes)
    assert (q._base[:, K:] == 0xA5).all()
    q2, s2 = B.quantize_fp8(xt)  # outputs allocated by the call
    assert torch.equal(q2.view(torch.uint8), q) and torch.equal(s2, s)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,K,pad", [(5000, 5, 0), (2100, 129, 1), (300, 2901, 0),
                                     (1100, 500, 3), (40, 16383, 2), (33, 128 * 128, 5)])
def test_quantize_rows_of_any_start(M, K, pad, dtype):
    rng = _gen(22, M, K, pad)
    x, _ = _offset_rows(M, K, dtype, pad, 3, float("nan"))
    x.copy_(torch.from_numpy(rng.standard_normal((M, K)) * np.exp(rng.standard_normal((M, 1)))))
    codes, scales = _quant_ref(x.cpu().float().numpy())
    for off in (0, 5, 16):
        q, base = _offset_rows(M, K, None, (off - K) % 16 if off == 16 else pad, off, 0xA5)
        s = torch.full((M, -(-K // 128)), -1.0, device="cuda")
        B.quantize_fp8(x, q, s)
        np.testing.assert_array_equal(s.cpu().numpy(), scales)
        np.testing.assert_array_equal(q.cpu().numpy(), codes)
        assert _untouched(q, base, 0xA5)


def test_quantize_extreme_groups():
    """Groups of zeros, tiny, huge, infinite and NaN values: each on its own."""
    x = np.ones((2, 128 * 8), dtype=np.float32)
    x[:, 0:128] = 0.0
    x[:, 128:256] = -0.0
    x[0, 256:384] = 1e-38   # the scale is subnormal
    x[0, 260] = -3e-39
    x[1, 256:384] = 1e-44   # the scale rounds to zero
    x[:, 384:512] = 3.3e38
    x[0, 400] = -1.1e38
    x[0, 520] = np.inf
    x[0, 700] = np.nan
    x[1, 800] = -np.inf
    xt = torch.from_numpy(x).cuda()
    q, s = B.quantize_fp8(xt)
    codes, scales = _quant_ref(np.nan_to_num(x, nan=1, posinf=1, neginf=1))
    bad = np.zeros((2, 8), dtype=bool)
    bad[0, 4] = bad[0, 5] = bad[1, 6] = True
    sc = s.cpu().numpy()
    assert not np.isfinite(sc[bad]).any()
    np.testing.assert_array_equal(sc[~bad], scales[~bad])
    back = _f64(q) * np.repeat(sc.astype(np.float64), 128, axis=1)
    wide = np.repeat(bad, 128, axis=1)
    assert np.isnan(back[wide]).all()
    np.testing.assert_array_equal(q.view(torch.uint8).cpu().numpy()[~wide], codes[~wide])


def test_quantize_is_the_tails_latent_quantisation():
    cfg = configs.SMALL.with_(M=9, seed=31)
    act, w = inputs.make_inputs(cfg)
    tail = B.LatentMoETail(cfg, PU.to_cuda(w))
    run = PU.Run(tail, PU.to_cuda(act), cfg)
    tail.close()
    q, s = B.quantize_fp8(act["z"].cuda())
    assert torch.equal(q.view(torch.uint8), run.zq) and torch.equal(s, run.zs)


# ---------------------------------------------------------------- block norms

def _norm_ref(h, y, gate, gpost, gpre, eps, a, b, sigmoid):
    """(h', its error scale, n, its error scale) in 64 bits."""
    H = h.shape[1]
    if y is None:
        h2 = a * h
        e = EPS * np.abs(h2)
    else:
        u = y if gpost is None else y / np.sqrt((y * y).sum(1, keepdims=True) / H + eps) * gpost
        if gate is not None:
            u = u * (1 / (1 + np.exp(-gate)) if sigmoid else gate)
        h2 = a * h + b * u
        e = 40 * EPS * (np.abs(a * h) + np.abs(b * u))
    if gpre is None:
        return h2, e, h2, e
    r = 1 / np.sqrt((h2 * h2).sum(1, keepdims=True) / H + eps)
    n = h2 * r * gpre
    # h' enters its own norm: each value's error, and the row's relative error in the root
    row = np.sqrt((e * e).sum(1, keepdims=True) / H) * r
    return h2, e, n, e * r * np.abs(gpre) + (40 * EPS + row) * np.abs(n)


CASES = [  # M, H, h dtype, y dtype, gate shape, gate dtype, sigmoid, post, pre, outputs, pad
    (1, 7168, BF16, BF16, None, BF16, False, True, True, "hn", 0),
    (16, 7168, F32, BF16, "c", BF16, False, True, True, "hqs", 0),
    (5, 129, BF16, F32, "t", F32, True, True, True, "hnqs", 3),
    (3, 1, F32, F32, "f", BF16, True, True, True, "hnqs", 0),
    (4, 7, BF16, BF16, None, BF16, False, False, True, "hnqs", 1),
    (9, 2901, BF16, BF16, "t", BF16, True, True, True, "hnqs", 11),
    (2, 8200, F32, BF16, "f", F32, False, True, True, "hnqs", 0),
    (2, 16384, BF16, BF16, "c", F32, True, True, True, "hnqs", 0),
    (3, 16383, F32, F32, "f", BF16, False, True, True, "hnqs", 2),
    (330, 512, BF16, BF16, "f", BF16, True, True, False, "hnqs", 0),
    (700, 7168, BF16, BF16, "c", BF16, False, True, True, "hqs", 0),
    (6, 640, F32, None, None, BF16, False, False, True, "nqs", 8),
    (6, 640, BF16, None, None, BF16, False, False, False, "hn", 0),
    (2, 256, BF16, BF16, "x", BF16, False, False, True, "n", 0),
    # many rows: persistent blocks
    (700, 1024, F32, BF16, "f", BF16, True, True, True, "hnqs", 0),
    (613, 1152, BF16, BF16, "t", F32, True, True, True, "hnqs", 128),
    (1300, 2048, F32, BF16, "x", BF16, False, True, True, "hnqs", 0),
    (650, 8192, F32, BF16, "c", F32, True, False, True, "hnqs", 0),
    (650, 1280, BF16, None, None, BF16, False, False, True, "nqs", 0),
    (650, 1024, BF16, BF16, "f", BF16, False, True, False, "hqs", 0),
    (620, 1408, F32, BF16, None, BF16, False, False, False, "hnqs", 0),
    (650, 1024, BF16, F32, "f", F32, True, True, True, "hnqs", 16),
    # fp32 block outputs and gates in aligned rows
    (9, 2048, F32, F32, "c", BF16, True, True, True, "hnqs", 0),
    (1300, 2560, BF16, F32, None, BF16, False, True, True, "hnqs", 0),
    (1300, 2560, F32, BF16, "f", F32, True, True, True, "hnqs", 8),
    (3, 16384, BF16, F32, "t", F32, True, True, True, "hnqs", 8),
    (3, 12800, F32, F32, "f", F32, False, True, True, "hnqs", 0),
    (1300, 640, BF16, F32, "x", F32, True, True, True, "hnqs", 0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}x{c[1]}-{c[4]}-{c[9]}-{c[10]}")
def test_block_norm(case):
    M, H, hd, yd, gs, gd, sig, post, pre, outs, pad = case
    rng = _gen(2, M, H)
    h = _padded(_cuda(rng.standard_normal((M, H)) * 3, hd), pad)
    y = None if yd is None else _padded(
        _cuda(rng.standard_normal((M, H)) * np.exp(rng.standard_normal((M, 1))), yd), pad)
    shape = {None: None, "c": (H,), "t": (M, 1), "f": (M, H), "x": (M, 2 * H)}[gs]
    gate = None if shape is None else _cuda(rng.standard_normal(shape), gd)
    if gs == "x":
        gate = gate[:, ::2]  # strided columns
    gpost = _cuda(rng.uniform(0.5, 1.5, H), BF16) if post else None
    gpre = _cuda(rng.uniform(0.5, 1.5, H), BF16) if pre else None
    a, b, eps = 0.75, 1.25, 1e-6
    layer = B.BlockNorm(H, gpost, gpre, eps, a, b, sig)
    out = {}
    if "h" in outs:
        out["h_out"] = _padded(torch.zeros((M, H), dtype=hd, device="cuda"), pad)
    if "n" in outs:
        out["n"] = _padded(torch.zeros((M, H), dtype=BF16, device="cuda"), pad)
    if "q" in outs:
        out["q"] = _padded(torch.zeros((M, H), dtype=torch.uint8, device="cuda"), pad)
        out["s"] = torch.full((M, -(-H // 128)), -1.0, device="cuda")
    layer(h, y, gate, **out)
    torch.cuda.synchronize()
    opt = lambda t: None if t is None else _f64(t)  # noqa: E731
    h2, eh, n, en = _norm_ref(_f64(h), opt(y), opt(gate), opt(gpost), opt(gpre),
                              float(np.float32(eps)), a, b, sig)
    if "h" in outs:
        assert (np.abs(_f64(out["h_out"]) - h2) <= HALF[hd] * np.abs(h2) + 1.01 * eh).all()
        assert pad == 0 or torch.isnan(out["h_out"]._base[:, H:]).all()
    if "n" in outs:
        assert (np.abs(_f64(out["n"]) - n) <= HALF[BF16] * np.abs(n) + 1.01 * en).all()
        assert pad == 0 or torch.isnan(out["n"]._base[:, H:]).all()
    if "q" in outs:
        s = out["s"].cpu().numpy().astype(np.float64)
        G = s.shape[1]
        wide = np.zeros((M, G * 128))
        wide[:, :H] = np.abs(n)
        amax = wide.reshape(M, G, 128).max(2)
        eamax = np.zeros((M, G * 128))
        eamax[:, :H] = en
        eamax = eamax.reshape(M, G, 128).max(2)
        ref_s = np.where(amax == 0, 1.0, amax / 448)
        assert (np.abs(s - ref_s) <= 1.01 * (eamax / 448 + EPS * ref_s)).all()
        sr = np.repeat(s, 128, axis=1)[:, :H]
        err = np.abs(_f64(out["q"]) * sr - n)
        assert (err <= 1.01 * np.maximum(2.0 ** -4 * np.abs(n), 2.0 ** -10 * sr) + 1.1 * en).all()
        assert pad == 0 or (out["q"]._base[:, H:] == 0).all()


def test_block_norm_in_place_and_allocating():
    rng = _gen(3)
    M, H = 37, 1024
    h, y = _cuda(rng.standard_normal((M, H)), F32), _cuda(rng.standard_normal((M, H)), BF16)
    g = _cuda(rng.uniform(0.5, 1.5, H), BF16)
    layer = B.BlockNorm(H, g, g)
    h1, n1, q1, s1 = layer(h, y)
    assert q1 is None and s1 is None and h1.dtype == F32 and n1.dtype == BF16
    h2, y2 = h.clone(), y.clone()
    layer(h2, y2, h_out=h2, n=y2)  # the stream and the block's output overwritten
    assert _same(h2, h1) and _same(y2, n1)
    # the quantised output is the quantiser's, of the unrounded n: within a bf16 rounding
    q, s = B.fp8_codes(M, H, "cuda"), torch.empty((M, H // 128), device="cuda")
    layer(h, y, q=q, s=s)
    qn, sn = B.quantize_fp8(n1)
    assert (s / sn - 1).abs().max() <= 2.0 ** -8 + 4 * EPS
    # entering a block without a block before it
    _, n0, _, _ = layer(h)
    ref = _norm_ref(_f64(h), None, None, None, _f64(g), float(np.float32(1e-6)), 1.0, 1.0, False)
    assert (np.abs(_f64(n0) - ref[2]) <= HALF[BF16] * np.abs(ref[2]) + 1.01 * ref[3]).all()


@pytest.mark.parametrize("M,H", [(40, 333), (300, 1029), (2000, 512), (1400, 1029)])
def test_block_norm_chain_in_place(M, H):
    """A residual stream updated in place by many calls in a row, whose rows share cache lines
    (odd widths): launches overlap, and each sees what the one before wrote."""
    rng = _gen(9, M, H)
    g = _cuda(rng.uniform(0.5, 1.5, H), BF16)
    y = _cuda(rng.standard_normal((M, H)), BF16)
    layer = B.BlockNorm(H, g, g, res_scale=0.9, branch_scale=0.7)

    def chain(sync):
        h, n = _cuda(_gen(10).standard_normal((M, H)), BF16), y.clone()
        for _ in range(60):
            layer(h, n, h_out=h, n=n)
            if sync:
                torch.cuda.synchronize()
        return h, n

    want = chain(True)
    for _ in range(3):
        got = chain(False)
        assert _same(got[0], want[0]) and _same(got[1], want[1])


@pytest.mark.parametrize("hd", [BF16, F32])
@pytest.mark.parametrize("M,H,pad", [
    (600, 500, 0), (2100, 129, 1), (70000, 5, 0), (600, 517, 3), (9, 4099, 0), (7, 4616, 8),
    (5, 8200, 7), (3, 12001, 0), (2, 16384, 5), (130, 2560, 8),
    # many values
    (2700, 517, 3), (300000, 5, 0), (11000, 129, 1), (2700, 500, 0), (350, 4099, 0),
    (300, 4616, 8), (170, 8200, 7), (120, 12001, 0), (90, 16383, 2), (530, 2560, 5)])
def test_block_norm_rows_of_any_start(M, H, pad, hd):
    """Every tensor's rows start on another element, and nothing around them is written."""
    rng = _gen(21, M, H, pad)

    def given(shape, dtype, off):
        v, _ = _offset_rows(*shape, dtype, pad, off, 7.0)
        v.copy_(torch.from_numpy(rng.standard_normal(shape)))
        return v

    h, y = given((M, H), hd, 1), given((M, H), BF16, 3)
    gate = given((M, H), BF16, 5)
    gpost, gpre = given((1, H), BF16, 1)[0], given((1, H), BF16, 2)[0]
    h2, h2_base = _offset_rows(M, H, hd, pad, 3, 7.0)
    n, n_base = _offset_rows(M, H, BF16, pad, 6, 7.0)
    q, q_base = _offset_rows(M, H, None, pad, 5, 0xA5)
    s = torch.full((M, -(-H // 128)), -1.0, device="cuda")
    layer = B.BlockNorm(H, gpost, gpre, 1e-6, 0.75, 1.25, True)
    layer(h, y, gate, h_out=h2, n=n, q=q, s=s)
    ref = _norm_ref(_f64(h), _f64(y), _f64(gate), _f64(gpost), _f64(gpre),
                    float(np.float32(1e-6)), 0.75, 1.25, True)
    assert (np.abs(_f64(h2) - ref[0]) <= HALF[hd] * np.abs(ref[0]) + 1.01 * ref[1]).all()
    assert (np.abs(_f64(n) - ref[2]) <= HALF[BF16] * np.abs(ref[2]) + 1.01 * ref[3]).all()
    sr = np.repeat(s.cpu().numpy().astype(np.float64), 128, axis=1)[:, :H]
    codes = q.contiguous().view(torch.float8_e4m3fn)
    err = np.abs(_f64(codes) * sr - ref[2])
    assert (err <= 1.01 * np.maximum(2.0 ** -4 * np.abs(ref[2]), 2.0 ** -10 * sr)
            + 1.1 * ref[3]).all()
    assert _untouched(h2, h2_base, 7.0) and _untouched(n, n_base, 7.0)
    assert _untouched(q, q_base, 0xA5)
    # in place, the same bits
    layer(h, y, gate, h_out=h, n=y)
    assert _same(h, h2) and _same(y, n)


def test_block_norm_zero_and_non_finite_rows():
    M, H = 4, 384
    h = torch.zeros((M, H), device="cuda")
    y = torch.zeros((M, H), device="cuda", dtype=BF16)
    y[1] = 1.0
    y[2, 5] = float("inf")
    h[3, 7] = float("nan")
    q, s = B.fp8_codes(M, H, "cuda"), torch.empty((M, 3), device="cuda")
    g = torch.ones(H, device="cuda", dtype=BF16)
    h2, n = torch.empty_like(h), torch.empty_like(y)
    B.BlockNorm(H, g, g)(h, y, h_out=h2, n=n, q=q, s=s)
    assert (h2[0] == 0).all() and (n[0] == 0).all() and (s[0] == 1).all()
    assert (q.view(torch.uint8)[0] & 0x7F == 0).all()
    assert torch.isfinite(n[1]).all() and torch.isfinite(s[1]).all()
    assert torch.isnan(n[2, 5]) and torch.isnan(n[3]).all() and torch.isnan(s[3]).all()
    assert B.BlockNorm(H)(h[:0], y[:0])[1].shape == (0, H)


def test_block_norm_refusals():
    h = torch.zeros((4, 256), device="cuda", dtype=BF16)
    f = h.float()
    g = torch.ones(256, device="cuda", dtype=BF16)
    n = B.BlockNorm(256, g, g)
    with pytest.raises(TypeError):
        n(h.half())
    with pytest.raises(TypeError):
        n(h, h, h_out=f)
    with pytest.raises(ValueError):
        n(h[:, :128], h)
    with pytest.raises(ValueError):
        n(h, h.t().contiguous().t())
    with pytest.raises(ValueError):
        n(h, None, g)
    with pytest.raises(ValueError):
        n(h, h.cpu())
    for shape in ((3, 256), (4, 128), (4,), (1, 4, 256)):
        with pytest.raises(ValueError):
            n(h, h, torch.zeros(shape, device="cuda", dtype=BF16))
    with pytest.raises(B.KltError):
        n(h, h, q=B.fp8_codes(4, 256, "cuda"))  # codes without scales
    with pytest.raises(B.KltError):
        n(h, h, n=torch.zeros((1, 256), device="cuda", dtype=BF16).expand(4, 256))
    with pytest.raises(ValueError):
        B.BlockNorm(256, g.float())


# ---------------------------------------------------------------- linear

def _codes_of(v, G0, G1):
    """e4m3 codes and fp32 scales of v in blocks of G0 x G1."""
    R, C = v.shape
    rb, cb = -(-R // G0), -(-C // G1)
    wide = np.zeros((rb * G0, cb * G1), dtype=np.float32)
    wide[:R, :C] = v
    t = wide.reshape(rb, G0, cb, G1)
    s = (np.abs(t).max(axis=(1, 3)) / 448).astype(np.float32)
    s = np.where(s == 0, np.float32(1), s)
    q = e4m3_encode(t / s[:, None, :, None]).reshape(rb * G0, cb * G1)[:R, :C]
    return np.ascontiguousarray(q), s


class Lin:
    """A random layer, its inputs, and its 64-bit result with error scales."""

    def __init__(self, M, N, K, act, out, seed=0):
        rng = _gen(4, M, N, K, seed)
        self.M, self.N, self.K, self.act, self.out = M, N, K, act, out
        x = rng.standard_normal((M, K)) * np.exp(rng.standard_normal((M, 1)))
        w = rng.standard_normal((N, K)) * np.exp(0.5 * rng.standard_normal((N, 1))) / K ** 0.5
        xq, xs = _codes_of(x, 1, 128)
        wq, ws = _codes_of(w, 128, 128)
        self.xq = B.fp8_codes(M, K, "cuda").view(torch.uint8)
        self.xq.copy_(torch.from_numpy(xq))
        self.xs = torch.from_numpy(xs).cuda()
        self.wq, self.ws = torch.from_numpy(wq).cuda(), torch.from_numpy(ws).cuda()
        xd = torch.from_numpy(e4m3_decode(xq) * np.repeat(xs.astype(np.float64), 128, 1)[:, :K])
        wd = torch.from_numpy(e4m3_decode(wq) * np.repeat(np.repeat(
            ws.astype(np.float64), 128, 0), 128, 1)[:N, :K])
        v = (xd @ wd.t()).numpy()
        e = (-(-K // 128) + 24) * EPS * (xd.abs() @ wd.abs().t()).numpy()
        if act == "swiglu":
            g, u, eg, eu = v[:, :N // 2], v[:, N // 2:], e[:, :N // 2], e[:, N // 2:]
            silu = g / (1 + np.exp(-g))
            v = silu * u
            e = 1.1 * np.abs(u) * eg + np.abs(silu) * eu + 1.1 * eg * eu + 16 * EPS * np.abs(v)
        self.ref, self.err = v, e
        self.layer = B.Fp8Linear(self.wq, self.ws, act, out)

    def check(self, got, rows=None):
        ref, err = (self.ref, self.err) if rows is None else (self.ref[rows], self.err[rows])
        if self.out == "fp8":
            q, s = got
            s = s.cpu().numpy().astype(np.float64)
            M, W = ref.shape
            amax = np.abs(ref).reshape(M, W // 128, 128).max(2)
            eamax = err.reshape(M, W // 128, 128).max(2)
            assert (np.abs(s - amax / 448) <= 1.01 * eamax / 448 + 2 * EPS * amax / 448).all()
            sr = np.repeat(s, 128, axis=1)
            off = np.abs(_f64(q) * sr - ref)
            assert (off <= 1.01 * np.maximum(2.0 ** -4 * np.abs(ref), 2.0 ** -10 * sr) +
                    1.1 * err).all()
        else:
            half = HALF[BF16 if self.out == "bf16" else F32]
            off = np.abs(_f64(got) - ref)
            assert (off <= half * np.abs(ref) + 1.01 * err).all(), \
                (off / (half * np.abs(ref) + 1.01 * err)).max()

    def close(self):
        assert self.layer.status() == B.KLT_OK
        self.layer.close()


@pytest.mark.parametrize("M,N,K,act,out", [
    (1, 128, 128, "none", "bf16"), (1, 1, 1, "none", "f32"), (1, 7168, 2048, "none", "bf16"),
    (3, 256, 256, "swiglu", "fp8"), (16, 512, 640, "swiglu", "bf16"), (16, 129, 127, "none", "f32"),
    (17, 384, 1000, "none", "bf16"), (33, 512, 896, "swiglu", "fp8"), (40, 1003, 2090, "none", "f32"),
    (64, 256, 1536, "none", "bf16"), (100, 513, 333, "none", "bf16"), (128, 640, 512, "none", "f32"),
    (129, 512, 130, "swiglu", "fp8"), (200, 300, 520, "none", "bf16")])
def test_linear(M, N, K, act, out):
    c = Lin(M, N, K, act, out)
    c.check(c.layer(c.xq, c.xs))
    c.close()


@pytest.mark.parametrize("tile,act,out", [(t, "none", "bf16") for t in (16, 32, 64, 128)] +
                         [(t, "swiglu", "fp8") for t in (16, 32, 64)])
@pytest.mark.parametrize("split", [1, 2, 4, 8])
def test_linear_every_narrow_form(tile, split, act, out):
    c = Lin(75, 512, 1100, act, out)  # a ragged last tile, 9 k-blocks in uneven parts
    c.check(c.layer(c.xq, c.xs, debug=B.KltLinearDebug(force_tile=tile, force_split=split)))
    c.close()


def test_linear_many_kblocks_narrow():
    """More k-blocks per part than scales are staged at once."""
    c = Lin(18, 128, 128 * 45 + 16, "none", "f32")
    for split in (1, 2):
        c.check(c.layer(c.xq, c.xs, debug=B.KltLinearDebug(force_tile=16, force_split=split)))
    c.close()


@pytest.mark.parametrize("M,N,K,act,out", [
    (256, 256, 128, "none", "bf16"), (300, 256, 256, "swiglu", "fp8"), (1, 1, 1, "none", "f32"),
    (129, 300, 2090, "none", "f32"), (513, 1003, 900, "none", "bf16"), (700, 768, 1024, "swiglu", "bf16"),
    (2100, 2560, 384, "none", "bf16"), (1500, 2048, 512, "swiglu", "fp8"), (257, 129, 127, "none", "bf16")])
def test_linear_wide(M, N, K, act, out):
    c = Lin(M, N, K, act, out)
    c.check(c.layer(c.xq, c.xs, debug=B.KltLinearDebug(force_tile=256)))
    c.close()


@pytest.mark.parametrize("M,N,K,act,out", [
    (1, 256, 512, "none", "bf16"), (300, 256, 640, "swiglu", "fp8"), (129, 300, 2090, "none", "f32"),
    (256, 129, 1030, "none", "bf16"), (700, 768, 1024, "swiglu", "bf16"), (513, 1003, 900, "none", "f32"),
    (2100, 2560, 384, "none", "bf16")])
def test_linear_wide_split(M, N, K, act, out):
    """A tile's K shared by two CTA pairs, evenly and not, also with more tiles than fit."""
    c = Lin(M, N, K, act, out)
    dbg = B.KltLinearDebug(force_tile=256, force_split=2)
    got = c.layer(c.xq, c.xs, debug=dbg)
    c.check(got)
    again = c.layer(c.xq, c.xs, debug=dbg)
    for a, b in zip(*((g if out == "fp8" else (g,)) for g in (got, again))):
        assert _same(a, b)
    c.close()


@pytest.mark.parametrize("tile,M", [(16, 9), (64, 70), (256, 300)])
def test_linear_strides_and_untouched_rows(tile, M):
    """Inputs and outputs in wider buffers; what lies outside the result stays."""
    for act, out, N in (("none", "bf16", 200), ("none", "f32", 131), ("swiglu", "fp8", 512)):
        c = Lin(M, N, 320, act, out)
        xq = _padded(c.xq, 48)
        W = c.ref.shape[1]
        dt = {"bf16": BF16, "f32": F32, "fp8": torch.uint8}[out]
        for pad in (3, 16):
            base = torch.full((M + 2, W + pad), 77, dtype=dt, device="cuda")
            o = base[:M, :W]
            o_s = torch.full((M + 1, W // 128), -3.0, device="cuda") if out == "fp8" else None
            got = c.layer(xq, c.xs, o, None if o_s is None else o_s[:M],
                          debug=B.KltLinearDebug(force_tile=tile))
            c.check(got)
            assert (base[M:] == 77).all() and (base[:, W:] == 77).all()
            assert o_s is None or (o_s[M:] == -3).all()
        c.close()


def test_linear_rows_do_not_depend_on_the_batch():
    """A row's result is the same bits alone and in a batch of the same kernel, and a batch's
    the same bits every time."""
    c = Lin(300, 384, 1536, "none", "f32")
    for tile, split in ((32, 4), (256, 1), (256, 2)):
        dbg = B.KltLinearDebug(force_tile=tile, force_split=split)
        full = c.layer(c.xq, c.xs, debug=dbg)
        for _ in range(5):
            assert _same(c.layer(c.xq, c.xs, debug=dbg), full)
        assert _same(c.layer(c.xq[:7], c.xs[:7], debug=dbg), full[:7])
    c.close()


def test_linear_zero_and_non_finite():
    c = Lin(40, 256, 256, "none", "f32")
    xs = c.xs.clone()
    xs[3, 1] = float("inf")
    xq = c.xq.clone()
    xq[5, 200] = 0x7F  # NaN code
    xq[6] = 0
    for tile in (16, 256):
        got = c.layer(xq, xs, debug=B.KltLinearDebug(force_tile=tile)).cpu()
        assert not torch.isfinite(got[3]).any() and torch.isnan(got[5]).all()
        assert (got[6] == 0).all()
        rows = [r for r in range(40) if r not in (3, 5, 6)]
        c.check(got[rows], rows)
    assert c.layer(xq[:0], xs[:0]).shape == (0, 256)
    c.close()


def test_linear_refusals():
    c = Lin(8, 256, 200, "swiglu", "fp8")
    f = c.layer
    with pytest.raises(TypeError):
        f(c.xq.float(), c.xs)
    with pytest.raises(ValueError):
        f(c.xq[:, :128], c.xs)
    with pytest.raises(ValueError):
        f(c.xq, c.xs[:4])
    with pytest.raises(ValueError):
        f(c.xq, c.xs.cpu())
    with pytest.raises(B.KltError) as e:  # rows 200 bytes apart
        f(c.xq.contiguous(), c.xs)
    assert e.value.code == B.KLT_ERR_ALIGN
    with pytest.raises(B.KltError) as e:
        f(_padded(c.xq, 24)[:, :200], c.xs, torch.empty(16, 64, dtype=torch.uint8, device="cuda")
          .as_strided((8, 128), (64, 1)))
    assert e.value.code == B.KLT_ERR_INVALID_ARG
    for dbg, code in ((dict(force_tile=128), B.KLT_ERR_UNSUPPORTED),
                      (dict(force_tile=48), B.KLT_ERR_INVALID_ARG),
                      (dict(force_tile=256, force_split=4), B.KLT_ERR_UNSUPPORTED),
                      (dict(force_split=4), B.KLT_ERR_UNSUPPORTED),  # 2 k-blocks
                      (dict(force_split=3), B.KLT_ERR_INVALID_ARG),
                      (dict(timeout_ms=-1), B.KLT_ERR_INVALID_ARG)):
        with pytest.raises(B.KltError) as e:
            f(c.xq, c.xs, debug=B.KltLinearDebug(**dbg))
        assert e.value.code == code, dbg
    with pytest.raises(ValueError):
        B.Fp8Linear(c.wq, c.ws[:1])
    with pytest.raises(ValueError):
        B.Fp8Linear(c.wq, c.ws, act="gelu")
    with pytest.raises(B.KltError):
        B.Fp8Linear(c.wq[:128].contiguous(), c.ws[:1], act="swiglu", out="fp8")
    c.close()
    with pytest.raises(B.KltError):
        f(c.xq, c.xs)


@pytest.mark.parametrize("tile,split", [(16, 1), (32, 2), (256, 1), (256, 2)])
def test_linear_bounded_wait_expires(tile, split):
    """The copies stop after one k-block: the waits on their data run out, every CTA returns
    and the handle reports it; another handle is not affected."""
    c = Lin(20, 256, 1280, "swiglu", "fp8")
    ok = Lin(20, 256, 1280, "swiglu", "fp8", seed=1)
    c.layer(c.xq, c.xs, debug=B.KltLinearDebug(stall_after_kblocks=1, timeout_ms=20,
                                               force_tile=tile, force_split=split))
    torch.cuda.synchronize()
    assert c.layer.status() == B.KLT_ERR_DEVICE_TIMEOUT
    c.layer.close()
    ok.check(ok.layer(ok.xq, ok.xs))
    ok.close()


# ---------------------------------------------------------------- together

def _dense_block(M, H, I, seed):
    """The operators of a dense FP8 layer between two norms, its weights and its input."""
    rng = _gen(5, seed)
    w13, s13 = _codes_of(rng.standard_normal((2 * I, H)) / H ** 0.5, 128, 128)
    w2, s2 = _codes_of(rng.standard_normal((H, I)) / I ** 0.5, 128, 128)
    cu = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    gam = [_cuda(rng.uniform(0.5, 1.5, H), BF16) for _ in range(3)]
    up = B.Fp8Linear(cu(w13), cu(s13), "swiglu", "fp8")
    down = B.Fp8Linear(cu(w2), cu(s2))
    enter = B.BlockNorm(H, gamma_pre=gam[0])
    leave = B.BlockNorm(H, gamma_post=gam[1], gamma_pre=gam[2], res_scale=0.9,
                        branch_scale=0.5)
    h = _cuda(rng.standard_normal((M, H)), BF16)
    gate = _cuda(rng.standard_normal(H), BF16)
    q, s = B.fp8_codes(M, H, "cuda"), torch.empty((M, H // 128), device="cuda")
    a, a_s = B.fp8_codes(M, I, "cuda"), torch.empty((M, I // 128), device="cuda")
    y = torch.empty((M, H), dtype=BF16, device="cuda")
    h2, n = torch.empty_like(h), torch.empty_like(h)

    def run():
        enter(h, q=q, s=s)
        up(q, s, a, a_s)
        down(a, a_s, y)
        leave(h, y, gate, h_out=h2, n=n)

    def reference():
        """In 64 bits, each stage from the GPU's own e4m3 input to it (codes next to a border
        may differ), so a stage is held to its own error."""
        deq = lambda c, sc, g0: e4m3_decode(c) * np.repeat(np.repeat(  # noqa: E731
            sc.astype(np.float64), g0, 0), 128, 1)
        num = lambda t: t.cpu().view(torch.uint8).numpy()  # noqa: E731
        x = deq(num(q), s.cpu().numpy(), 1)
        v = x @ deq(w13, s13, 128).T
        act = v[:, :I] / (1 + np.exp(-v[:, :I])) * v[:, I:]
        ad = deq(num(a), a_s.cpu().numpy(), 1)
        yr = ad @ deq(w2, s2, 128).T
        ref = _norm_ref(_f64(h), _f64(y), _f64(gate), _f64(gam[1]), _f64(gam[2]),
                        float(np.float32(1e-6)), float(np.float32(0.9)), 0.5, False)
        n0 = _norm_ref(_f64(h), None, None, None, _f64(gam[0]), float(np.float32(1e-6)), 1, 1,
                       False)[2]
        return x, n0, ad, act, yr, ref

    return dict(run=run, reference=reference, q=q, s=s, a=a, a_s=a_s, y=y, h2=h2, n=n, h=h,
                layers=(up, down))


def _check_block(b):
    x, n0, ad, act, yr, ref = b["reference"]()
    # e4m3 of a value: at most half a step, 2^-4, of it, or half a subnormal step of the scale
    for got, want, s in ((x, n0, b["s"]), (ad, act, b["a_s"])):
        sr = np.repeat(s.cpu().numpy().astype(np.float64), 128, 1)
        assert (np.abs(got - want) <= 1.01 * np.maximum(2.0 ** -4 * np.abs(want),
                                                        2.0 ** -10 * sr) + 1e-5 * sr * 448).all()
    rms = np.sqrt((yr ** 2).mean())
    assert (np.abs(_f64(b["y"]) - yr) <= 2.0 ** -8 * np.abs(yr) + 1e-5 * rms).all()
    for got, r, e in ((b["h2"], ref[0], ref[1]), (b["n"], ref[2], ref[3])):
        assert (np.abs(_f64(got) - r) <= 2.0 ** -8 * np.abs(r) + 1.01 * e).all()


@pytest.mark.parametrize("M", [1, 16, 100, 600])
def test_dense_layer(M):
    b = _dense_block(M, 1024, 512, M)
    b["run"]()
    torch.cuda.synchronize()
    _check_block(b)
    assert all(f.status() == B.KLT_OK for f in b["layers"])


@pytest.mark.parametrize("M", [4, 300])
def test_dense_layer_captured(M):
    """Two captured graphs of the same layer objects, replayed on new inputs and in turn with
    an eager run, give the eager run's bits."""
    b = _dense_block(M, 512, 256, 50 + M)
    b["run"]()
    side = torch.cuda.Stream()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            b["run"]()
        graphs.append(g)
    for i in range(3):
        b["h"].copy_(torch.randn(b["h"].shape, device="cuda") * (i + 1))
        b["run"]()
        want = [b[k].clone() for k in ("h2", "n", "y", "a_s")]
        for g in graphs:
            for k in ("h2", "n", "y", "a_s"):
                b[k].zero_()
            g.replay()
            assert all(_same(b[k], w) for k, w in zip(("h2", "n", "y", "a_s"), want))


def test_dense_layer_back_to_back_on_two_streams():
    """Many layers queued without a wait, each reading what the one before wrote, on two
    streams that share the layer objects: the same bits as one at a time."""
    H, I = 512, 256
    b = _dense_block(24, H, I, 77)
    up, down = b["layers"]
    g = torch.ones(H, device="cuda", dtype=BF16)
    norm = B.BlockNorm(H, g, g, res_scale=0.5, branch_scale=0.5)

    def chain(h0, sync):
        h = h0.clone()
        q, s = B.quantize_fp8(h)
        for _ in range(30):
            a, a_s = up(q, s)
            y = down(a, a_s)
            norm(h, y, h_out=h, q=q, s=s)
            if sync:
                torch.cuda.synchronize()
        return h, q

    starts = [torch.randn((24, H), device="cuda").to(BF16) for _ in range(2)]
    want = [chain(h, True) for h in starts]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for st, h in zip(streams, starts):
            with torch.cuda.stream(st):
                got.append(chain(h, False))
        torch.cuda.synchronize()
        for a, w in zip(got, want):
            assert _same(a[0], w[0]) and torch.equal(a[1].view(torch.uint8),
                                                     w[1].view(torch.uint8))


def test_moe_block_between_norms():
    """Norm, the tail from the hidden state, then gate, residual and the next norm, against
    the oracle's tail on the GPU's own bf16 norm."""
    cfg = configs.SMALL.with_(M=12, E=8, topk=3, seed=13)
    w = inputs.make_weights(cfg)
    w.update(inputs.make_projection_weights(cfg))
    rng = _gen(6)
    H = cfg.H
    h = _cuda(rng.standard_normal((cfg.M, H)), BF16)
    gam = [_cuda(rng.uniform(0.5, 1.5, H), BF16) for _ in range(3)]
    tail = B.LatentMoETail(cfg, PU.to_cuda(w), max_tokens=cfg.M)
    enter = B.BlockNorm(H, gamma_pre=gam[0])
    leave = B.BlockNorm(H, gam[1], gam[2], branch_scale=0.5, gate_sigmoid=True)
    gate = _cuda(rng.standard_normal((cfg.M, 1)), F32)
    for _ in range(3):  # launches overlap from one call to the next
        _, n, _, _ = enter(h)
        y = tail.forward_hidden(n)
        h2, n2, _, _ = leave(h, y, gate)
    torch.cuda.synchronize()
    assert tail.status() == B.KLT_OK
    tail.close()
    z, lg = T.latent_inputs(n.cpu(), w["w_lat"], w["w_gate"])
    o = T.tail({"x": n.cpu(), "z": torch.from_numpy(z).to(BF16),
                "logits": torch.from_numpy(lg).float()}, w, cfg)
    PU.assert_output_close(_f64(y), o["out"])
    ref = _norm_ref(_f64(h), _f64(y), _f64(gate), _f64(gam[1]), _f64(gam[2]),
                    float(np.float32(1e-6)), 1.0, 0.5, True)
    for got, r, e in ((h2, ref[0], ref[1]), (n2, ref[2], ref[3])):
        assert (np.abs(_f64(got) - r) <= 2.0 ** -8 * np.abs(r) + 1.01 * e).all()
