"""Refusals of the 8-bit KV cache's calls.  Every case returns its status before any CUDA call, so no GPU is
needed: the fake, aligned addresses below are never dereferenced."""
import ctypes as C

import pytest
import torch

FAKE = C.c_void_p(1 << 20)
MIS = C.c_void_p((1 << 20) + 8)  # not 16-byte aligned
ODD = C.c_void_p((1 << 20) + 2)  # not 4-byte aligned


def _p(xkv, **kw):
    base = dict(batch=2, n_kv_heads=2, head_dim=64, block=16, capacity=256)
    base.update(kw)
    return xkv.kv8_params(**base)


def _c(xkv, **kw):
    base = dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, weight=FAKE, ids=FAKE)
    base.update(kw)
    return xkv.KV8Pointers(**base)


BAD_PARAMS = [(dict(batch=0), 1), (dict(n_kv_heads=0), 1), (dict(head_dim=0), 1), (dict(block=0), 1), (dict(capacity=8), 1),
              (dict(capacity=250), 1), (dict(capacity=0), 1), (dict(capacity=-16), 1), (dict(head_dim=40), 2),
              (dict(head_dim=272), 2), (dict(block=4), 2), (dict(block=24, capacity=240), 2), (dict(block=256), 2),
              (dict(capacity=1 << 31), 2), (dict(batch=1 << 20, capacity=1 << 20), 2)]


@pytest.mark.parametrize("bad,status", BAD_PARAMS)
def test_sizes(xkv, bad, status):
    p, c, n = _p(xkv, **bad), _c(xkv), C.c_size_t(0)
    lib = xkv.lib
    assert lib.xkv_kv8_workspace_size(p, 4, C.byref(n)) == status
    assert lib.xkv_kv8_append(p, c, FAKE, None, 1, xkv.XKV_BF16, FAKE, FAKE, 4096, 4096, None) == status
    assert lib.xkv_kv8_attention_decode(p, c, FAKE, 4, xkv.XKV_BF16, FAKE, FAKE, 0, FAKE, 1 << 40, None) == status
    assert lib.xkv_kv8_evict(p, c, FAKE, 4, 1, 1, C.c_void_p(1 << 24), None) == status


def test_query_heads_and_workspace(xkv):
    p, n = _p(xkv), C.c_size_t(0)
    f = xkv.lib.xkv_kv8_workspace_size
    assert f(p, 32, C.byref(n)) == xkv.XKV_OK and n.value > 0
    assert f(p, 3, C.byref(n)) == f(p, 0, C.byref(n)) == f(p, -2, C.byref(n)) == xkv.XKV_ERR_INVALID_ARG
    assert f(p, 4, None) == f(None, 4, C.byref(n)) == xkv.XKV_ERR_INVALID_ARG
    assert f(p, 34, C.byref(n)) == xkv.XKV_ERR_UNSUPPORTED  # 17 query heads to a KV head
    assert f(p, 4, C.byref(n)) == xkv.XKV_OK
    g = xkv.lib.xkv_kv8_attention_decode
    for ws, size in ((None, n.value), (FAKE, n.value - 1), (MIS, n.value)):
        assert g(p, _c(xkv), FAKE, 4, xkv.XKV_BF16, FAKE, FAKE, 0, ws, size, None) == xkv.XKV_ERR_WORKSPACE


@pytest.mark.parametrize("bad", [dict(k=None), dict(v=None), dict(k_scale=None), dict(v_scale=None), dict(k=MIS),
                                 dict(v=MIS), dict(k_scale=ODD), dict(v_scale=ODD), dict(weight=ODD), dict(ids=ODD)])
def test_cache_pointers(xkv, bad):
    p, c = _p(xkv), _c(xkv, **bad)
    lib, inv = xkv.lib, xkv.XKV_ERR_INVALID_ARG
    assert lib.xkv_kv8_append(p, c, FAKE, None, 1, xkv.XKV_BF16, FAKE, FAKE, 128, 128, None) == inv
    assert lib.xkv_kv8_attention_decode(p, c, FAKE, 4, xkv.XKV_BF16, FAKE, FAKE, 0, FAKE, 1 << 40, None) == inv
    assert lib.xkv_kv8_evict(p, c, FAKE, 4, 1, 1, C.c_void_p(1 << 24), None) == inv


def test_append_arguments(xkv):
    p, c, f = _p(xkv), _c(xkv), xkv.lib.xkv_kv8_append
    ok = dict(lens=FAKE, counts=None, n=4, dt=xkv.XKV_BF16, k=FAKE, v=FAKE, ld=128, bs=512)

    def call(**kw):
        a = {**ok, **kw}
        return f(p, c, a["lens"], a["counts"], a["n"], a["dt"], a["k"], a["v"], a["ld"], a["bs"], None)

    assert call(n=0) == xkv.XKV_OK  # nothing to do, nothing launched
    for bad in (dict(lens=None), dict(lens=ODD), dict(counts=ODD), dict(n=-1), dict(n=257), dict(dt=2), dict(k=None),
                dict(v=None), dict(k=MIS), dict(v=MIS), dict(ld=120), dict(ld=132), dict(bs=-8), dict(bs=516),
                dict(dt=xkv.XKV_F32, ld=130)):
        assert call(**bad) == xkv.XKV_ERR_INVALID_ARG, bad


def test_append_of_no_rows_needs_no_address(xkv):
    # an empty tensor has none
    f = xkv.lib.xkv_kv8_append
    assert f(_p(xkv), _c(xkv), FAKE, None, 0, xkv.XKV_BF16, None, None, 128, 0, None) == xkv.XKV_OK
    assert f(_p(xkv), _c(xkv), None, None, 0, xkv.XKV_BF16, None, None, 128, 0, None) == xkv.XKV_ERR_INVALID_ARG
    assert f(_p(xkv), _c(xkv), FAKE, None, 1, xkv.XKV_BF16, FAKE, None, 128, 0, None) == xkv.XKV_ERR_INVALID_ARG


def test_attention_and_eviction_arguments(xkv):
    p, c, inv = _p(xkv), _c(xkv), xkv.XKV_ERR_INVALID_ARG
    f = xkv.lib.xkv_kv8_attention_decode
    for lens, dt, q, out in ((None, 1, FAKE, FAKE), (ODD, 1, FAKE, FAKE), (FAKE, 2, FAKE, FAKE), (FAKE, 1, None, FAKE),
                             (FAKE, 1, FAKE, None), (FAKE, 1, MIS, FAKE), (FAKE, 1, FAKE, MIS)):
        assert f(p, c, lens, 4, dt, q, out, 0, FAKE, 1 << 40, None) == inv
    assert f(p, _c(xkv, weight=None), FAKE, 4, 1, FAKE, FAKE, 1, FAKE, 1 << 40, None) == inv  # nothing to add to
    g, far = xkv.lib.xkv_kv8_evict, C.c_void_p(1 << 24)
    for budget, sink, recent in ((0, 0, 0), (4, 0, 0), (4, -1, 1), (4, 3, 2), (0, 0, 1), (2, 2 ** 31 - 1, 2 ** 31 - 1)):
        assert g(p, c, FAKE, budget, sink, recent, far, None) == inv, (budget, sink, recent)
    for lens, out in ((None, far), (FAKE, None), (ODD, far), (FAKE, ODD), (FAKE, FAKE),
                      (FAKE, C.c_void_p((1 << 20) + 4))):  # lens_out over lens
        assert g(p, c, lens, 4, 1, 1, out, None) == inv
    for gone in ("weight", "ids"):
        assert g(p, _c(xkv, **{gone: None}), FAKE, 4, 1, 1, far, None) == inv
    assert g(_p(xkv, block=8, capacity=8 * 131073), c, FAKE, 4, 1, 1, far, None) == xkv.XKV_ERR_UNSUPPORTED
    assert g(_p(xkv, batch=1 << 28, n_kv_heads=1, block=8, capacity=8), c, FAKE, 1, 0, 1, C.c_void_p(1 << 40),
             None) == xkv.XKV_ERR_UNSUPPORTED


def test_binding_checks_the_cache_tensors(xkv):
    f8, rows, nblk = torch.float8_e4m3fn, (2, 2, 256, 64), (2, 2, 16)
    k = torch.zeros(rows, dtype=torch.uint8).view(f8)
    s = torch.ones(nblk)
    with pytest.raises(ValueError):
        xkv.KV8Cache(k, k, s, s)  # host memory
    for bad in ((k.view(torch.uint8), k, s, s), (k, k[:, :, :128], s, s), (k, k, s[:, :1], s), (k, k, s, s[..., :8]),
                (k, k, s.double(), s), (k, k, s, s, None, torch.zeros(nblk)), (k, k, torch.ones((2, 2, 15)), s)):
        with pytest.raises(ValueError):
            xkv.KV8Cache(*bad)


def test_replaced_tensors_are_the_ones_that_calls_take(xkv, monkeypatch):
    import copy
    monkeypatch.setattr(xkv, "_ptr", lambda t: None if t is None else t.data_ptr())  # host tensors will do here
    f8, rows, nblk = torch.float8_e4m3fn, (2, 2, 256, 64), (2, 2, 16)
    new = {"k": lambda: torch.zeros(rows, dtype=torch.uint8).view(f8), "v": lambda: torch.zeros(rows, dtype=torch.uint8).view(f8),
           "k_scale": lambda: torch.ones(nblk), "v_scale": lambda: torch.ones(nblk), "weight": lambda: torch.zeros(nblk),
           "ids": lambda: torch.zeros(nblk, dtype=torch.int32)}
    c = xkv.KV8Cache(**{x: f() for x, f in new.items()})
    other = copy.copy(c)
    before = {x: getattr(c.pointers, x) for x in new}
    for x, f in new.items():
        t = f()
        setattr(c, x, t)
        assert getattr(c, x) is t and getattr(c.pointers, x) == t.data_ptr() != before[x]
        assert getattr(other.pointers, x) == before[x] == getattr(other, x).data_ptr()
    c.weight = None
    assert c.weight is None and c.pointers.weight is None and c.pointers.ids == c.ids.data_ptr()
    held = {x: getattr(c.pointers, x) for x in new}
    for x, bad in (("k", c.k[:1]), ("k", c.k.view(torch.uint8)), ("v", c.v[..., :32]), ("k_scale", c.k_scale[..., :8]),
                   ("v_scale", c.v_scale.double()), ("ids", torch.zeros(nblk)), ("weight", c.k_scale[:1])):
        kept = getattr(c, x)
        with pytest.raises(ValueError):
            setattr(c, x, bad)
        assert getattr(c, x) is kept and {y: getattr(c.pointers, y) for y in new} == held
