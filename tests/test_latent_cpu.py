"""Host-side argument checks of klt_latent_*: every refusal comes before anything touches a device,
so fake pointers never leave the host.  A handle cannot be made without a device; the checks of a
call come before its first use, so a zeroed block of memory with the layer's sizes stands in for
one."""
import ctypes

import pytest
import torch

from latent_moe_layer_route_gb300 import binding as B
from latent_moe_layer_route_gb300 import build

PTR = 0x10000
INVALID, UNSUPPORTED, ALIGN = B.KLT_ERR_INVALID_ARG, B.KLT_ERR_UNSUPPORTED, B.KLT_ERR_ALIGN


@pytest.fixture(scope="module")
def lib():
    build.build()
    return B.load_library()


DIMS = dict(heads=4, latent=128, rope=64, nope=128, value=128, page=64, pairs=0, eps=1e-6,
            scale=0.1)


def _create(lib, inv_freq=PTR, gamma=PTR, **kw):
    d = B.KltLatentDims(**dict(DIMS, **kw))
    h = ctypes.c_void_p()
    rc = lib.klt_latent_create(ctypes.byref(d), inv_freq, gamma, ctypes.byref(h))
    assert not h.value
    return rc


@pytest.mark.parametrize("kw,code", [
    (dict(heads=0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(inv_freq=None), INVALID),
    (dict(heads=257), UNSUPPORTED), (dict(latent=64), UNSUPPORTED), (dict(latent=192), UNSUPPORTED),
    (dict(latent=640), UNSUPPORTED), (dict(rope=0), UNSUPPORTED), (dict(rope=24), UNSUPPORTED),
    (dict(rope=80), UNSUPPORTED), (dict(nope=96), UNSUPPORTED), (dict(value=192), UNSUPPORTED),
    (dict(page=8), UNSUPPORTED), (dict(page=48), UNSUPPORTED), (dict(page=2048), UNSUPPORTED),
    (dict(pairs=2), UNSUPPORTED), (dict(inv_freq=PTR + 2), ALIGN), (dict(gamma=PTR + 1), ALIGN)])
def test_create_arguments(lib, kw, code):
    assert _create(lib, **kw) == code


def test_null(lib):
    h, n = ctypes.c_void_p(), ctypes.c_uint64()
    assert lib.klt_latent_create(None, PTR, PTR, ctypes.byref(h)) == INVALID
    assert lib.klt_latent_create(ctypes.byref(B.KltLatentDims(**DIMS)), PTR, PTR, None) == INVALID
    assert lib.klt_latent_append(None, ctypes.byref(B.KltLatentAppendArgs()), None) == INVALID
    assert lib.klt_latent_attend(None, ctypes.byref(B.KltLatentAttendArgs()), None, None) == INVALID
    assert lib.klt_latent_prefill(None, ctypes.byref(B.KltLatentPrefillArgs()), None, None) == INVALID
    assert lib.klt_latent_workspace(None, 1, 1, ctypes.byref(n)) == INVALID
    assert lib.klt_latent_status(None) == INVALID
    assert lib.klt_latent_destroy(None) == B.KLT_OK


@pytest.fixture(scope="module")
def handle():
    """The handle begins with its klt_latent_dims; its device (-1) is no current one, so a call
    whose arguments are all right is refused for that at the latest."""
    memory = (ctypes.c_uint8 * 256)()
    d = B.KltLatentDims(**DIMS)
    ctypes.memmove(memory, ctypes.byref(d), ctypes.sizeof(d))
    fields = (ctypes.c_int32 * 3).from_buffer(memory, ctypes.sizeof(d))
    fields[0], fields[1], fields[2] = -1, 152, 6  # device, SMs, log2 of the page
    return memory


def _append(lib, handle, **kw):
    a = dict(T=3, kv_dtype=0, kv=PTR, positions=PTR, slots=PTR, cache=PTR, kv_out=PTR, q=PTR,
             q_out=PTR, pages=5, ld_kv=192, page_stride=64 * 192, row_stride=192, ld_kv_out=192,
             q_token=4 * 64, q_head=64, q_out_token=4 * 64, q_out_head=64)
    a.update(kw)
    return lib.klt_latent_append(ctypes.addressof(handle),
                                 ctypes.byref(B.KltLatentAppendArgs(**a)), None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), INVALID), (dict(kv=None), INVALID), (dict(positions=None), INVALID),
    (dict(slots=None), INVALID), (dict(cache=None), INVALID), (dict(q=None), INVALID),
    (dict(q_out=None), INVALID), (dict(pages=-1), INVALID), (dict(ld_kv=-8), INVALID),
    (dict(cache=None, slots=None, kv_out=None, q=None, q_out=None), INVALID),
    (dict(page_stride=64 * 192 - 8), INVALID), (dict(row_stride=184), INVALID),
    (dict(ld_kv_out=184), INVALID), (dict(q_out_head=56), INVALID),
    (dict(q_out_token=4 * 64 - 8), INVALID), (dict(q_out_token=64, q_out_head=2 * 64), INVALID),
    (dict(kv_dtype=2), UNSUPPORTED), (dict(kv_dtype=-1), UNSUPPORTED),
    (dict(pages=1 << 26), UNSUPPORTED),
    (dict(kv=PTR + 8), ALIGN), (dict(cache=PTR + 2), ALIGN), (dict(kv_out=PTR + 4), ALIGN),
    (dict(q=PTR + 8), ALIGN), (dict(q_out=PTR + 8), ALIGN), (dict(positions=PTR + 4), ALIGN),
    (dict(slots=PTR + 4), ALIGN), (dict(ld_kv=196), ALIGN), (dict(ld_kv=194, kv_dtype=1), ALIGN),
    (dict(page_stride=64 * 192 + 4), ALIGN), (dict(row_stride=196, page_stride=1 << 20), ALIGN),
    (dict(q_token=4 * 64 + 4), ALIGN), (dict(q_head=68), ALIGN),
    (dict(q_out_token=4 * 64 + 4), ALIGN), (dict(T=0, kv=None), B.KLT_OK)])
def test_append_arguments(lib, handle, kw, code):
    assert _append(lib, handle, **kw) == code


def _bytes(lib, handle):
    n = ctypes.c_uint64()
    assert lib.klt_latent_workspace(ctypes.addressof(handle), 2, 3, ctypes.byref(n)) == B.KLT_OK
    return n.value


def _attend(lib, handle, dbg=None, **kw):
    a = dict(B=2, T=3, max_pages=7, q=PTR, cache=PTR, block_table=PTR, seq_lens=PTR, cu_q=PTR,
             out=PTR, lse=PTR, workspace=PTR, workspace_bytes=_bytes(lib, handle), pages=5,
             q_token=4 * 192, q_head=192, page_stride=64 * 192, row_stride=192, ld_table=7,
             out_token=4 * 128, out_head=128)
    a.update(kw)
    return lib.klt_latent_attend(ctypes.addressof(handle),
                                 ctypes.byref(B.KltLatentAttendArgs(**a)),
                                 ctypes.byref(dbg) if dbg is not None else None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), INVALID), (dict(T=-1), INVALID), (dict(max_pages=-1), INVALID),
    (dict(pages=-1), INVALID), (dict(q=None), INVALID), (dict(cache=None), INVALID),
    (dict(block_table=None), INVALID), (dict(seq_lens=None), INVALID), (dict(out=None), INVALID),
    (dict(workspace=None), INVALID), (dict(cu_q=None), INVALID), (dict(q_token=-8), INVALID),
    (dict(ld_table=6), INVALID), (dict(row_stride=184), INVALID),
    (dict(page_stride=64 * 192 - 8), INVALID), (dict(out_head=120), INVALID),
    (dict(out_token=4 * 128 - 8), INVALID), (dict(workspace_bytes=16), INVALID),
    (dict(pages=1 << 25), UNSUPPORTED), (dict(max_pages=1 << 25, ld_table=1 << 25), UNSUPPORTED),
    (dict(T=1 << 29), UNSUPPORTED), (dict(page_stride=1 << 38), UNSUPPORTED),
    (dict(q_token=1 << 38), UNSUPPORTED),
    (dict(q=PTR + 8), ALIGN), (dict(cache=PTR + 8), ALIGN), (dict(out=PTR + 8), ALIGN),
    (dict(workspace=PTR + 8), ALIGN), (dict(lse=PTR + 2), ALIGN), (dict(block_table=PTR + 2), ALIGN),
    (dict(seq_lens=PTR + 1), ALIGN), (dict(cu_q=PTR + 2), ALIGN), (dict(q_token=772), ALIGN),
    (dict(q_head=196), ALIGN), (dict(row_stride=196, page_stride=1 << 20), ALIGN),
    (dict(out_token=516), ALIGN), (dict(T=0, q=None), B.KLT_OK)])
def test_attend_arguments(lib, handle, kw, code):
    assert _attend(lib, handle, **kw) == code


def _prefill(lib, handle, dbg=None, **kw):
    a = dict(B=2, T=3, S=5, causal=1, q=PTR, k=PTR, v=PTR, k_rope=PTR, cu_q=PTR, cu_k=PTR, out=PTR,
             lse=PTR, q_token=4 * 192, q_head=192, k_token=4 * 256, k_head=256, v_token=4 * 256,
             v_head=256, ld_k_rope=64, out_token=4 * 128, out_head=128)
    a.update(kw)
    return lib.klt_latent_prefill(ctypes.addressof(handle),
                                  ctypes.byref(B.KltLatentPrefillArgs(**a)),
                                  ctypes.byref(dbg) if dbg is not None else None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), INVALID), (dict(T=-1), INVALID), (dict(S=-1), INVALID), (dict(q=None), INVALID),
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k_rope=None), INVALID),
    (dict(cu_q=None), INVALID), (dict(cu_k=None), INVALID), (dict(out=None), INVALID),
    (dict(q_token=-8), INVALID), (dict(k_head=0), INVALID), (dict(v_token=0), INVALID),
    (dict(ld_k_rope=0), INVALID), (dict(q_head=0), INVALID), (dict(out_head=120), INVALID),
    (dict(out_token=4 * 128 - 8), INVALID), (dict(T=1 << 29), UNSUPPORTED),
    (dict(k_token=1 << 38), UNSUPPORTED),
    (dict(q=PTR + 8), ALIGN), (dict(k=PTR + 8), ALIGN), (dict(v=PTR + 8), ALIGN),
    (dict(k_rope=PTR + 8), ALIGN), (dict(out=PTR + 8), ALIGN), (dict(lse=PTR + 2), ALIGN),
    (dict(cu_q=PTR + 2), ALIGN), (dict(cu_k=PTR + 2), ALIGN), (dict(q_head=196), ALIGN),
    (dict(k_token=1028), ALIGN), (dict(v_head=260), ALIGN), (dict(ld_k_rope=68), ALIGN),
    (dict(out_token=516), ALIGN), (dict(T=0, q=None), B.KLT_OK)])
def test_prefill_arguments(lib, handle, kw, code):
    assert _prefill(lib, handle, **kw) == code


@pytest.mark.parametrize("n", [2**31 - 1, 2**31 - 4096])
def test_sizes_leave_room_to_round_up(lib, handle, n):
    """Rows are counted in 32 bits, rounded up to whole tiles."""
    assert _prefill(lib, handle, S=n) == UNSUPPORTED
    assert _prefill(lib, handle, T=n // 4 + 1) == UNSUPPORTED
    assert _attend(lib, handle, T=n // 4 + 1) == UNSUPPORTED
    assert _attend(lib, handle, pages=n // 64 + 1) == UNSUPPORTED


@pytest.mark.parametrize("dbg", [dict(stall_after_tiles=-1), dict(timeout_ms=-1)])
def test_debug_arguments(lib, handle, dbg):
    dbg = B.KltLatentDebug(**dbg)
    assert _attend(lib, handle, dbg) == INVALID
    assert _prefill(lib, handle, dbg) == INVALID


def test_workspace_arguments(lib, handle):
    n = ctypes.c_uint64()
    h = ctypes.addressof(handle)
    assert lib.klt_latent_workspace(h, 0, 1, ctypes.byref(n)) == INVALID
    assert lib.klt_latent_workspace(h, 1, -1, ctypes.byref(n)) == INVALID
    assert lib.klt_latent_workspace(h, 1, 1, None) == INVALID


def test_binding_refuses_what_is_no_cuda_tensor(lib):
    freq = torch.ones(32)
    with pytest.raises(ValueError):
        B.LatentAttention(4, inv_freq=freq)
    with pytest.raises(ValueError):
        B.LatentAttention(4, inv_freq=freq, pairs="thirds")
    with pytest.raises(B.KltError):
        B.LatentAttention(1 << 40, inv_freq=freq)
