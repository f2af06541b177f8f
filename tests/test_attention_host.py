"""Refusals of the paged-cache and attention entry points: host validation
returns the documented status before anything is launched, and the binding
refuses tensors that do not fit.  No GPU is needed."""
import ctypes

import numpy as np
import pytest
import torch

from bit_weight_quantized_nvq_b200 import capi

lib = capi.lib()
_keep = []


def p(off=0, nbytes=4096):
    # host buffers stand in for device pointers: validation never reads them
    buf = np.zeros(nbytes + 64, np.uint8)
    _keep.append(buf)
    return buf.ctypes.data + (-buf.ctypes.data % 16) + off


def cache(**kw):
    c = dict(k_codes=p(), k_scales=p(), v_codes=p(), v_scales=p(), n_pages=4, n_kv_heads=2, page_size=16, head_dim=64)
    c.update(kw)
    return capi.KVCache(**c)


OK, ARG, SHAPE, ALIGN, WS = (capi.NVQ_OK, capi.NVQ_ERR_INVALID_ARG, capi.NVQ_ERR_BAD_SHAPE,
                             capi.NVQ_ERR_MISALIGNED, capi.NVQ_ERR_WORKSPACE)

CACHES = [(dict(k_codes=None), ARG), (dict(v_scales=None), ARG), (dict(n_pages=0), ARG), (dict(n_kv_heads=-1), ARG),
          (dict(page_size=0), ARG), (dict(page_size=24), SHAPE), (dict(page_size=1 << 17), SHAPE),
          (dict(head_dim=96), SHAPE), (dict(head_dim=32), SHAPE), (dict(n_pages=1 << 32), SHAPE),
          (dict(n_kv_heads=1 << 17), SHAPE), (dict(n_pages=1 << 30, page_size=64), SHAPE),
          (dict(k_codes=p(8)), ALIGN), (dict(v_scales=p(4)), ALIGN)]

# rows of 2 heads x 64
KV = dict(k=p(), k_stride=128, v=p(), v_stride=128, dtype=1, cu=p(), lens=p(), table=p(), B=2, cols=3, rows=5)
BAD_KV = [(dict(k=None), ARG), (dict(v=None), ARG), (dict(cu=None), ARG), (dict(lens=None), ARG), (dict(table=None), ARG),
          (dict(B=-1), ARG), (dict(rows=-1), ARG), (dict(cols=-1), ARG), (dict(dtype=3), ARG), (dict(dtype=-1), ARG),
          (dict(k_stride=127), SHAPE), (dict(v_stride=64), SHAPE), (dict(rows=1 << 31), SHAPE), (dict(cols=1 << 31), SHAPE),
          (dict(k_stride=132), ALIGN), (dict(v_stride=130, dtype=0), ALIGN), (dict(k=p(8)), ALIGN), (dict(v=p(2)), ALIGN)]


def kv(fn, c, **kw):
    a = dict(KV, **kw)
    return fn(ctypes.byref(c) if c is not None else None, a["k"], a["k_stride"], a["v"], a["v_stride"], a["dtype"], a["cu"],
              a["lens"], a["table"], a["B"], a["cols"], a["rows"], None)


@pytest.mark.parametrize("fn", [lib.nvq_kv_write, lib.nvq_kv_read])
def test_cache_rows_are_refused(fn):
    assert kv(fn, None) == ARG
    for c, st in CACHES:
        assert kv(fn, cache(**c)) == st, c
    for a, st in BAD_KV:
        assert kv(fn, cache(), **a) == st, a
    for a in (dict(B=0), dict(rows=0), dict(rows=0, k=None, v=None, cu=None)):
        assert kv(fn, cache(), **a) == OK, a


DEC = dict(q=p(), q_stride=256, dtype=1, lens=p(), table=p(), B=2, cols=3, heads=4, scale=0.1, out=p(), out_stride=256,
           counters=p(), ws=p(), nbytes=1 << 40)
BAD_DEC = [(dict(q=None), ARG), (dict(out=None), ARG), (dict(lens=None), ARG), (dict(table=None), ARG), (dict(counters=None), ARG),
           (dict(B=-1), ARG), (dict(cols=-1), ARG), (dict(dtype=7), ARG), (dict(heads=0), ARG), (dict(heads=-4), ARG),
           (dict(scale=0.0), ARG), (dict(scale=-1.0), ARG), (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG),
           (dict(heads=5), SHAPE), (dict(heads=1 << 17), SHAPE), (dict(B=1 << 17), SHAPE), (dict(cols=1 << 28), SHAPE),
           (dict(B=1 << 15, cols=1 << 20), SHAPE), (dict(q_stride=1 << 38), SHAPE),
           (dict(q_stride=255), SHAPE), (dict(out_stride=0), SHAPE), (dict(q_stride=260), ALIGN), (dict(q=p(8)), ALIGN),
           (dict(out=p(4)), ALIGN), (dict(ws=p(8)), ALIGN), (dict(ws=None), WS), (dict(nbytes=0), WS)]


def dec(c, **kw):
    a = dict(DEC, **kw)
    return lib.nvq_attn_decode(ctypes.byref(c) if c is not None else None, a["q"], a["q_stride"], a["dtype"], a["lens"], a["table"],
                               a["B"], a["cols"], a["heads"], a["scale"], a["out"], a["out_stride"], a["counters"], a["ws"],
                               a["nbytes"], None)


def test_decode_is_refused():
    assert dec(None) == ARG
    for c, st in CACHES:
        assert dec(cache(**c)) == st, c
    for a, st in BAD_DEC:
        assert dec(cache(), **a) == st, a
    assert dec(cache(), B=0) == OK
    size = lib.nvq_attn_decode_workspace_size
    assert size(2, 4, 2, 64) > 0 and size(0, 4, 2, 64) == 0 and size(2, 5, 2, 64) == 0 and size(2, 4, 2, 80) == 0


PRE = dict(q=p(), qs=256, k=p(), ks=128, v=p(), vs=128, dtype=1, cu_q=p(), cu_k=p(), B=2, tq=5, tk=6, heads=4, kv=2, dim=64,
           scale=0.1, out=p(), os=256)
BAD_PRE = [(dict(q=None), ARG), (dict(k=None), ARG), (dict(v=None), ARG), (dict(out=None), ARG), (dict(cu_q=None), ARG),
           (dict(cu_k=None), ARG), (dict(B=-1), ARG), (dict(tq=-1), ARG), (dict(tk=-1), ARG), (dict(dtype=0), ARG), (dict(dtype=5), ARG),
           (dict(heads=0), ARG), (dict(kv=0), ARG), (dict(scale=0.0), ARG), (dict(scale=float("nan")), ARG),
           (dict(heads=3), SHAPE), (dict(dim=256), SHAPE), (dict(dim=0), SHAPE), (dict(B=1 << 17), SHAPE), (dict(tq=1 << 31), SHAPE),
           (dict(tk=1 << 31), SHAPE), (dict(qs=255), SHAPE), (dict(ks=64), SHAPE), (dict(vs=64), SHAPE), (dict(os=128), SHAPE),
           (dict(qs=1 << 39), SHAPE), (dict(tq=1 << 29, heads=1 << 14, kv=1, qs=1 << 20, os=1 << 20), SHAPE),
           (dict(qs=260), ALIGN), (dict(ks=132), ALIGN), (dict(vs=132), ALIGN), (dict(os=260), ALIGN), (dict(q=p(8)), ALIGN),
           (dict(k=p(2)), ALIGN), (dict(v=p(4)), ALIGN), (dict(out=p(8)), ALIGN)]


def pre(**kw):
    a = dict(PRE, **kw)
    return lib.nvq_attn_prefill(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["dtype"], a["cu_q"], a["cu_k"], a["B"], a["tq"],
                                a["tk"], a["heads"], a["kv"], a["dim"], a["scale"], 1, a["out"], a["os"], None)


def test_prefill_is_refused():
    for a, st in BAD_PRE:
        assert pre(**a) == st, a
    assert pre(B=0) == OK and pre(tq=0) == OK


@pytest.mark.parametrize("call", [lambda **a: dec(cache(), **a), pre])
def test_scales_whose_factors_would_overflow_are_refused(call):
    """Up to 2^64; B = 0 returns before anything is launched."""
    for scale in (float("inf"), 3e38, float(np.nextafter(np.float32(2.0 ** 64), np.float32(np.inf))), -0.1, 0.0):
        assert call(scale=scale) == ARG and call(scale=scale, B=0) == ARG, scale
    for scale in (2.0 ** 64, 1.0, 1e-38):
        assert call(scale=scale, B=0) == OK, scale


# --- the binding, on CPU tensors: every check is made before the library is called

def cpu_cache(pages=4, heads=2, page=16, dim=64):
    return capi.kv_cache(pages, heads, page, dim, device="cpu")


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_binding_refuses_tensors_that_do_not_fit():
    c = cpu_cache()
    k = torch.zeros(5, 2, 64, dtype=torch.float16)
    good = (i32(3), i32(2), i32(2, 3))
    for bad in ((k[:, :1], k), (k, k[:4]), (k, k.float()), (k.transpose(0, 1), k), (k[..., ::2], k), (k[..., :32], k), (k, k.to("meta"))):
        with pytest.raises((ValueError, TypeError)):
            capi.kv_write(c, *bad, *good)
    for cu, lens, table in ((i32(2), i32(2), i32(2, 3)), (i32(3), i32(2), i32(3, 3)), (i32(3).long(), i32(2), i32(2, 3)),
                            (i32(3), i32(2).float(), i32(2, 3)), (i32(3), i32(2), i32(2, 6)[:, ::2])):
        with pytest.raises((ValueError, TypeError)):
            capi.kv_write(c, k, k, cu, lens, table)
        with pytest.raises((ValueError, TypeError)):
            capi.kv_read(c, cu, lens, table, 5)
    with pytest.raises(TypeError):
        capi.kv_write(c, k.int(), k.int(), *good)
    with pytest.raises(ValueError):
        capi.kv_read(c, *good, 5, k=torch.zeros(4, 2, 64, dtype=torch.float16))
    for broken in ((c[0].float(),) + c[1:], (c[0], c[1].float()) + c[2:], (c[0], c[1][:2]) + c[2:], (c[0], c[1], c[2][:2], c[3][:2])):
        with pytest.raises(ValueError):
            capi.kv_write(broken, k, k, *good)
    q = torch.zeros(2, 4, 64)
    for args in ((q[:1], i32(2), i32(2, 3), i32(8)), (q, i32(2), i32(2, 3), i32(7)), (q, i32(2), i32(2, 3), i32(8).long()),
                 (q[..., :32], i32(2), i32(2, 3), i32(8)), (q, i32(2), i32(1, 3), i32(8))):
        with pytest.raises(ValueError):
            capi.attn_decode(c, *args)
    with pytest.raises(ValueError):
        capi.attn_decode(c, q, i32(2), i32(2, 3), i32(8), out=q.half())
    x = torch.zeros(5, 4, 64, dtype=torch.float16)
    for args in ((x, k, k[:4], i32(3)), (x, k, k.bfloat16(), i32(3)), (x, k, k, i32(3), i32(4)), (x, k, k, i32(3).long()),
                 (x, k[..., :32], k, i32(3))):
        with pytest.raises(ValueError):
            capi.attn_prefill(*args)
    with pytest.raises(ValueError):
        capi.attn_prefill(x, k, k, i32(3), out=torch.zeros(4, 4, 64, dtype=torch.float16))


def test_binding_refuses_a_workspace_elsewhere_or_with_gaps():
    """The pointer and the size of a workspace stand for memory of the call's
    device without gaps; anything else is refused before the library is called."""
    c, q = cpu_cache(), torch.zeros(2, 4, 64)
    space = torch.zeros(1 << 20, dtype=torch.uint8)
    for bad in (space[::2], space.view(1024, 1024).t(), torch.zeros(1 << 20, dtype=torch.uint8, device="meta")):
        with pytest.raises(ValueError, match="workspace"):
            capi.attn_decode(c, q, i32(2), i32(2, 3), i32(8), workspace=bad)
    with pytest.raises(ValueError, match="CUDA"):            # what is wrong here is the whole call's device
        capi.attn_decode(c, q, i32(2), i32(2, 3), i32(8), workspace=space)


def test_the_stalled_wait_is_refused_without_a_place_or_a_limit():
    for limit, at, st in ((10, p(), ARG), (2 * 10 ** 9, p(), ARG), (10 ** 6, None, ARG), (10 ** 6, p(4), ALIGN)):
        for moving in (0, 1):
            assert lib.nvq_debug_stalled_attn_wait(limit, moving, at, None) == st
