"""Host-side argument checks of klt_quantize, klt_block_norm and klt_linear_*: every refusal
comes before anything touches a device, so fake pointers never leave the host.  The binding's
own checks run on CPU tensors, which it refuses."""
import ctypes

import pytest
import torch

from latent_moe_layer_route_gb300 import binding as B
from latent_moe_layer_route_gb300 import build

PTR = 0x10000


@pytest.fixture(scope="module")
def lib():
    build.build()
    return B.load_library()


def _quant(lib, x=PTR, dtype=B.KLT_DT_BF16, ld_x=256, M=4, K=256, q=PTR, ld_q=256, s=PTR):
    return lib.klt_quantize(x, dtype, ld_x, M, K, q, ld_q, s, None)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), B.KLT_ERR_INVALID_ARG), (dict(K=0), B.KLT_ERR_INVALID_ARG),
    (dict(x=None), B.KLT_ERR_INVALID_ARG), (dict(q=None), B.KLT_ERR_INVALID_ARG),
    (dict(s=None), B.KLT_ERR_INVALID_ARG), (dict(ld_q=255), B.KLT_ERR_INVALID_ARG),
    (dict(ld_x=-256), B.KLT_ERR_INVALID_ARG), (dict(dtype=2), B.KLT_ERR_UNSUPPORTED),
    (dict(dtype=9), B.KLT_ERR_UNSUPPORTED), (dict(x=PTR + 1), B.KLT_ERR_ALIGN),
    (dict(M=1, K=2 ** 28 + 1, ld_q=2 ** 29), B.KLT_ERR_UNSUPPORTED),
    (dict(x=PTR + 2, dtype=B.KLT_DT_F32), B.KLT_ERR_ALIGN), (dict(s=PTR + 2), B.KLT_ERR_ALIGN),
    (dict(M=0, x=None), B.KLT_OK)])
def test_quantize_arguments(lib, kw, code):
    assert _quant(lib, **kw) == code


def _norm(lib, **kw):
    a = dict(M=4, H=256, h_dtype=0, y_dtype=0, gate_dtype=0, gate_sigmoid=0, eps=1e-6,
             res_scale=1.0, branch_scale=1.0, h=PTR, y=PTR, n=PTR, ld_h=256, ld_y=256,
             ld_n=256)
    a.update(kw)
    return lib.klt_block_norm(ctypes.byref(B.KltBlockNormArgs(**a)), None)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), B.KLT_ERR_INVALID_ARG), (dict(H=0), B.KLT_ERR_INVALID_ARG),
    (dict(eps=-1.0), B.KLT_ERR_INVALID_ARG), (dict(eps=float("nan")), B.KLT_ERR_INVALID_ARG),
    (dict(h=None), B.KLT_ERR_INVALID_ARG), (dict(n=None), B.KLT_ERR_INVALID_ARG),
    (dict(q=PTR), B.KLT_ERR_INVALID_ARG), (dict(s=PTR), B.KLT_ERR_INVALID_ARG),
    (dict(y=None, gate=PTR), B.KLT_ERR_INVALID_ARG),
    (dict(y=None, gamma_post=PTR), B.KLT_ERR_INVALID_ARG),
    (dict(ld_n=255), B.KLT_ERR_INVALID_ARG), (dict(ld_h=-1), B.KLT_ERR_INVALID_ARG),
    (dict(h_out=PTR, ld_h_out=128), B.KLT_ERR_INVALID_ARG),
    (dict(q=PTR, s=PTR, ld_q=255), B.KLT_ERR_INVALID_ARG),
    (dict(H=B.KLT_BLOCK_NORM_MAX_H + 1, ld_n=1 << 20), B.KLT_ERR_UNSUPPORTED),
    (dict(h_dtype=2), B.KLT_ERR_UNSUPPORTED), (dict(y_dtype=-1), B.KLT_ERR_UNSUPPORTED),
    (dict(gate_dtype=5), B.KLT_ERR_UNSUPPORTED),
    (dict(h=PTR + 1), B.KLT_ERR_ALIGN), (dict(h=PTR + 2, h_dtype=1), B.KLT_ERR_ALIGN),
    (dict(gamma_pre=PTR + 1), B.KLT_ERR_ALIGN), (dict(n=PTR + 1), B.KLT_ERR_ALIGN),
    (dict(M=0, h=None), B.KLT_OK)])
def test_block_norm_arguments(lib, kw, code):
    assert _norm(lib, **kw) == code


def test_block_norm_null(lib):
    assert lib.klt_block_norm(None, None) == B.KLT_ERR_INVALID_ARG


def _create(lib, N=256, K=256, act=0, out=0, w=PTR, ws=PTR):
    h = ctypes.c_void_p()
    rc = lib.klt_linear_create(ctypes.byref(B.KltLinearDims(N, K, act, out)), w, ws,
                               ctypes.byref(h))
    assert not h.value
    return rc


@pytest.mark.parametrize("kw,code", [
    (dict(N=0), B.KLT_ERR_INVALID_ARG), (dict(K=0), B.KLT_ERR_INVALID_ARG),
    (dict(w=None), B.KLT_ERR_INVALID_ARG), (dict(ws=None), B.KLT_ERR_INVALID_ARG),
    (dict(N=(1 << 20) + 1), B.KLT_ERR_UNSUPPORTED), (dict(N=1 << 20, K=1 << 20), B.KLT_ERR_UNSUPPORTED),
    (dict(act=2), B.KLT_ERR_UNSUPPORTED), (dict(act=1, N=384), B.KLT_ERR_UNSUPPORTED),
    (dict(act=1, out=1), B.KLT_ERR_UNSUPPORTED), (dict(act=0, out=2), B.KLT_ERR_UNSUPPORTED),
    (dict(out=7), B.KLT_ERR_UNSUPPORTED), (dict(ws=PTR + 2), B.KLT_ERR_ALIGN)])
def test_linear_create_arguments(lib, kw, code):
    assert _create(lib, **kw) == code


def test_linear_null(lib):
    h = ctypes.c_void_p()
    assert lib.klt_linear_create(None, PTR, PTR, ctypes.byref(h)) == B.KLT_ERR_INVALID_ARG
    assert lib.klt_linear_create(ctypes.byref(B.KltLinearDims(256, 256, 0, 0)), PTR, PTR,
                                 None) == B.KLT_ERR_INVALID_ARG
    assert lib.klt_linear_forward(None, PTR, 256, PTR, 4, PTR, 256, None, None, None) == \
        B.KLT_ERR_INVALID_ARG
    assert lib.klt_linear_status(None) == B.KLT_ERR_INVALID_ARG
    assert lib.klt_linear_tile(None, 4) == -B.KLT_ERR_INVALID_ARG
    assert lib.klt_linear_destroy(None) == B.KLT_OK


def test_binding_refuses_host_tensors(lib):
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        B.quantize_fp8(x)
    with pytest.raises(ValueError):
        B.BlockNorm(256)(x)
    with pytest.raises(ValueError):
        B.BlockNorm(256, gamma_pre=torch.ones(256, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        B.Fp8Linear(torch.zeros(256, 256, dtype=torch.uint8), torch.ones(2, 2))


def test_binding_refuses_what_is_no_strided_tensor(lib):
    class Lookalike:
        dtype, shape = torch.bfloat16, (4, 256)

    q, s = torch.zeros(4, 256, dtype=torch.uint8), torch.zeros(4, 2)
    for x in (None, 3, [1.0], Lookalike()):
        with pytest.raises(TypeError):
            B.quantize_fp8(x, q, s)
    with pytest.raises(TypeError):
        B.quantize_fp8(torch.zeros(4, 256, dtype=torch.float16), q, s)
    with pytest.raises(ValueError):
        B.quantize_fp8(torch.zeros(4, 256).to_sparse(), q, s)
    with pytest.raises(ValueError):
        B.quantize_fp8(torch.zeros(4, 256, device="meta"), q, s)


def test_fp8_codes_rows_start_on_16_bytes():
    q = B.fp8_codes(3, 130, "cpu")
    assert q.shape == (3, 130) and q.stride() == (144, 1) and q.dtype == torch.float8_e4m3fn
