"""The cache's and the attention's entry points on the host, no GPU needed:
what they refuse before any CUDA call, the workspace's size, and the binding's
checks of shapes and types."""
import ctypes

import pytest
import torch

import elementwise_row_rmsnorm_gb300 as gbe
from elementwise_row_rmsnorm_gb300.binding import _KvCacheStruct

OK, NULL_, SHAPE, DTYPE, ALIAS, ALIGN, SCALE, WORKSPACE = 0, 1, 2, 3, 8, 9, 13, 14


@pytest.fixture(scope="module")
def L():
    gbe.build()
    return gbe.lib()


def _cache(**kw):
    """A description with made-up, well separated addresses; nothing is read through them."""
    f = dict(k=1 << 40, v=1 << 41, k_scale=None, v_scale=None, n_pages=10, Hkv=2, page_size=16, D=64, page_stride=None,
             dtype=1)
    f.update(kw)
    if f["page_stride"] is None:
        f["page_stride"] = f["Hkv"] * f["page_size"] * f["D"]
    return _KvCacheStruct(**f)


def _rows(L, fn, c, T=4, k=1 << 42, ks=128, v=1 << 43, vs=128, slots=1 << 44, bad=None, dtype=1):
    p = None if c is None else ctypes.addressof(c)
    return getattr(L, fn)(k, ks, v, vs, slots, T, p, bad, dtype, None)


@pytest.mark.parametrize("fn", ["gbe_kv_write", "gbe_kv_read"])
def test_cache_descriptions_that_are_refused(L, fn):
    assert _rows(L, fn, None) == NULL_
    assert _rows(L, fn, _cache(dtype=0)) == DTYPE          # an f32 cache with bf16 rows
    assert _rows(L, fn, _cache(dtype=3)) == DTYPE
    assert _rows(L, fn, _cache(), dtype=2) == DTYPE
    for bad in (dict(D=0), dict(D=7), dict(D=60), dict(D=264), dict(Hkv=0), dict(Hkv=4097), dict(page_size=0),
                dict(page_size=(1 << 20) + 1), dict(n_pages=-1), dict(n_pages=1 << 28), dict(page_stride=2040),
                dict(page_stride=1 << 62)):
        assert _rows(L, fn, _cache(**bad), ks=1 << 20, vs=1 << 20) == SHAPE, bad
    assert _rows(L, fn, _cache(page_stride=2052)) == ALIGN  # pages off the grid of 8 elements
    assert _rows(L, fn, _cache(k=(1 << 40) + 2)) == ALIGN
    assert _rows(L, fn, _cache(k=None)) == NULL_
    assert _rows(L, fn, _cache(dtype=2)) == NULL_           # no scales
    assert _rows(L, fn, _cache(), ks=127) == SHAPE          # tokens closer than Hkv * D
    assert _rows(L, fn, _cache(), T=-1) == SHAPE
    assert _rows(L, fn, _cache(), T=(1 << 29) + 1) == SHAPE
    assert _rows(L, fn, _cache(), T=0) == OK
    assert _rows(L, fn, _cache(), k=(1 << 42) + 1) == ALIGN
    assert _rows(L, fn, _cache(), slots=(1 << 44) + 2) == ALIGN
    assert _rows(L, fn, _cache(), slots=None) == NULL_
    assert _rows(L, fn, _cache(), bad=(1 << 45) + 1) == ALIGN


@pytest.mark.parametrize("fn", ["gbe_kv_write", "gbe_kv_read"])
def test_overlaps_that_are_refused(L, fn):
    assert _rows(L, fn, _cache(), k=1 << 40) == ALIAS               # rows within the cache
    # slots inside the cache: refused where the cache is written (a read gets as far as the driver, which knows no
    # such memory)
    assert (_rows(L, fn, _cache(), slots=(1 << 40) + 64) == ALIAS) == (fn == "gbe_kv_write")
    assert _rows(L, fn, _cache(), bad=(1 << 41) + 64) == ALIAS
    if fn == "gbe_kv_write":
        assert _rows(L, fn, _cache(v=(1 << 40) + 2048)) == ALIAS    # v's pages inside k's
        assert _rows(L, fn, _cache(dtype=2, k_scale=1 << 46, v_scale=(1 << 46) + 10)) == ALIAS
    else:
        assert _rows(L, fn, _cache(), v=(1 << 42) + 128) == ALIAS   # v's rows inside k's
        assert _rows(L, fn, _cache(), slots=(1 << 42) + 8) == ALIAS


def _decode(L, c=None, q=1 << 42, qs=256, out=1 << 43, os_=256, B=3, Hq=4, table=1 << 44, pages=8, lens=1 << 45,
            scale=0.1, ws=1 << 46, room=1 << 40, dtype=1):
    c = _cache() if c is None else c
    return L.gbe_attn_decode(q, qs, out, os_, B, Hq, ctypes.addressof(c), table, pages, lens, scale, ws, room, dtype,
                             None)


def test_decode_refusals(L):
    assert _decode(L, dtype=2) == DTYPE and _decode(L, dtype=0) == DTYPE
    assert _decode(L, Hq=3) == SHAPE and _decode(L, Hq=0) == SHAPE and _decode(L, Hq=1) == SHAPE
    assert _decode(L, Hq=65538, qs=1 << 40, os_=1 << 40) == SHAPE
    assert _decode(L, B=-1) == SHAPE and _decode(L, B=(1 << 20) + 1) == SHAPE
    assert _decode(L, pages=-1) == SHAPE and _decode(L, pages=(1 << 26) + 1) == SHAPE
    assert _decode(L, qs=255) == SHAPE and _decode(L, os_=255) == SHAPE
    assert _decode(L, scale=float("nan")) == SCALE and _decode(L, scale=float("inf")) == SCALE
    assert _decode(L, B=0) == OK
    need = L.gbe_attn_decode_workspace(3, 4, 2, 64, 16, 8)
    long = L.gbe_attn_decode_workspace(3, 4, 2, 64, 16, 1000)
    assert long > 0 and long >= need
    assert _decode(L, pages=1000, room=long - 1) == WORKSPACE
    assert _decode(L, pages=1000, room=-1) == WORKSPACE
    assert _decode(L, pages=1000, ws=None) == NULL_
    assert _decode(L, pages=1000, ws=(1 << 46) + 8) == ALIGN
    assert _decode(L, lens=None) == NULL_ and _decode(L, table=None) == NULL_ and _decode(L, q=None) == NULL_
    assert _decode(L, out=1 << 42) == ALIAS                 # out == q
    assert _decode(L, out=1 << 40) == ALIAS                 # out inside the cache
    assert _decode(L, pages=1000, ws=(1 << 45)) == ALIAS    # the workspace over lens
    assert _decode(L, lens=(1 << 45) + 2) == ALIGN


def test_workspace_sizes(L):
    W = L.gbe_attn_decode_workspace
    assert W(1, 32, 8, 128, 64, 1) == 0                     # one chunk: nothing to join
    assert W(0, 32, 8, 128, 64, 1000) == 0
    a = W(1, 32, 8, 128, 64, 1000)
    assert a > 0 and W(5, 32, 8, 128, 64, 1000) == 5 * a
    for bad in ((-1, 32, 8, 128, 64, 10), (1, 33, 8, 128, 64, 10), (1, 32, 0, 128, 64, 10), (1, 32, 8, 100, 64, 10),
                (1, 32, 8, 128, 0, 10), (1, 32, 8, 128, 64, -1), (1, 32, 8, 128, 64, 1 << 25)):
        assert W(*bad) == -1, bad
    with pytest.raises(ValueError):
        c = gbe.KvCache.__new__(gbe.KvCache)
        c.shape = (1, 3, 16, 64)
        gbe.attn_decode_workspace(1, 4, c, 10)


def _prompt(L, q=1 << 40, qs=256, k=1 << 41, ks=128, v=1 << 42, vs=128, out=1 << 43, os_=256, starts=1 << 44, n=2, T=50,
            Hq=4, H=2, D=64, scale=0.1, dtype=1):
    return L.gbe_attn_prompt(q, qs, k, ks, v, vs, out, os_, starts, n, T, Hq, H, D, scale, dtype, None)


def test_prompt_refusals(L):
    assert _prompt(L, dtype=2) == DTYPE
    for bad in (dict(n=-1), dict(T=-1), dict(T=(1 << 28) + 1), dict(Hq=3), dict(H=0), dict(Hq=0), dict(D=4), dict(D=257),
                dict(D=0), dict(D=264), dict(qs=255), dict(ks=127), dict(vs=127), dict(os_=255), dict(n=(1 << 24) + 1)):
        assert _prompt(L, **bad) == SHAPE, bad
    assert _prompt(L, scale=float("nan")) == SCALE and _prompt(L, scale=-float("inf")) == SCALE
    assert _prompt(L, T=0) == OK and _prompt(L, n=0) == OK
    assert _prompt(L, q=None) == NULL_ and _prompt(L, starts=None) == NULL_
    assert _prompt(L, k=(1 << 41) + 1) == ALIGN and _prompt(L, starts=(1 << 44) + 1) == ALIGN
    assert _prompt(L, out=1 << 40) == ALIAS                 # out == q
    assert _prompt(L, out=(1 << 41) + 64) == ALIAS
    assert _prompt(L, starts=(1 << 43) + 8) == ALIAS


def test_status_strings():
    for st in (SCALE, WORKSPACE):
        assert gbe.status_string(st) != "unknown status"


def test_binding_checks():
    """Shapes and types that the binding refuses before it calls the library."""
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    f8 = torch.zeros(4, 2, 16, 64, dtype=torch.float8_e4m3fn)
    s = torch.zeros(4, 2, 16, dtype=torch.uint8)
    for args in ((k, k[:3]), (k[0], k[0]), (k.half(), k.half()), (k, k.float()), (f8, f8), (f8, f8, s, s[:3]), (k, k, s, s),
                 (k.transpose(1, 2), k.transpose(1, 2)), (f8, f8, s.int(), s.int()), (k, k)):  # the last: not on a GPU
        with pytest.raises(ValueError):
            gbe.KvCache(*args)
    q = torch.zeros(5, 4, 64)
    with pytest.raises(ValueError):
        gbe.gbe_attn_prompt(q, q[:, :2], q[:4, :2], q, torch.zeros(2, dtype=torch.int32), 1.0)
    with pytest.raises(ValueError):
        gbe.gbe_attn_prompt(q, q[:, :2], q[:, :2], q, torch.zeros(2), 1.0)
    with pytest.raises(ValueError):
        gbe.gbe_attn_prompt(q, q[:, :2], q[:, :2], q, torch.zeros(2, dtype=torch.int32), 1.0)  # not on a GPU


def test_a_caches_tensors_cannot_be_exchanged():
    """The description that the library reads was made of the tensors given."""
    for name in ("k", "v", "k_scale", "v_scale"):
        with pytest.raises(AttributeError):
            setattr(gbe.KvCache.__new__(gbe.KvCache), name, torch.zeros(1))
