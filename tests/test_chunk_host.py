"""The entry points for new tokens behind a cached prefix and for windows, on
the host, no GPU needed: what they refuse before any CUDA call, workspaces'
sizes, and the binding's checks of shapes and types."""
import ctypes

import pytest
import torch

import elementwise_row_rmsnorm_gb300 as gbe
from elementwise_row_rmsnorm_gb300.binding import _KvCacheStruct

OK, NULL_, SHAPE, DTYPE, LAYOUT, ROTARY, ALIAS, ALIGN, SCALE, WORKSPACE = 0, 1, 2, 3, 4, 6, 8, 9, 13, 14


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


def _append(L, c=None, q=1 << 42, qo=1 << 43, qs=256, Hq=4, k=1 << 44, ks=128, v=1 << 45, vs=128, pos=1 << 46,
            slots=3 << 46, T=4, r=64, om=1 << 47, table=None, n=0, mu=1.0, layout=0, bad=None, dtype=1, null=False):
    c = _cache() if c is None else c
    return L.gbe_rope_kv_write(q, qo, qs, Hq, k, ks, v, vs, pos, slots, T, r, om, table, n, mu, layout,
                               None if null else ctypes.addressof(c), bad, dtype, None)


def test_append_refusals(L):
    assert _append(L, null=True) == NULL_
    assert _append(L, dtype=2) == DTYPE and _append(L, _cache(dtype=0)) == DTYPE
    assert _append(L, layout=2) == LAYOUT
    for bad in (dict(D=60), dict(D=264), dict(Hkv=0), dict(page_size=0), dict(n_pages=-1)):
        assert _append(L, _cache(**bad), ks=1 << 20, vs=1 << 20, qs=1 << 20) == SHAPE, bad
    for bad in (dict(T=-1), dict(T=(1 << 27) + 1), dict(Hq=-1), dict(Hq=65537), dict(qs=255), dict(ks=127), dict(vs=127),
                dict(table=1 << 48, n=-1)):
        assert _append(L, **bad) == SHAPE, bad
    for bad in (dict(r=63), dict(r=66), dict(r=-2), dict(mu=float("inf")), dict(mu=float("nan"))):
        assert _append(L, **bad) == ROTARY, bad
    assert _append(L, T=0) == OK
    for name in ("q", "qo", "k", "v", "pos", "slots", "om"):
        assert _append(L, **{name: None}) == NULL_, name
    assert _append(L, _cache(dtype=2)) == NULL_             # no scales
    for name, at in (("q", 1 << 42), ("qo", 1 << 43), ("k", 1 << 44), ("v", 1 << 45), ("pos", 1 << 46), ("slots", 3 << 46),
                     ("om", 1 << 47)):
        assert _append(L, **{name: at + 1}) == ALIGN, name
    assert _append(L, table=(1 << 48) + 4, n=3) == ALIGN and _append(L, bad=(1 << 48) + 2) == ALIGN


def test_append_overlaps(L):
    assert _append(L, qo=(1 << 42) + 512) == ALIAS          # part of q
    assert _append(L, qo=1 << 44) == ALIAS and _append(L, qo=1 << 45) == ALIAS
    assert _append(L, qo=1 << 40) == ALIAS and _append(L, k=1 << 40) == ALIAS and _append(L, q=1 << 41) == ALIAS
    assert _append(L, pos=1 << 43) == ALIAS and _append(L, slots=1 << 40) == ALIAS and _append(L, om=1 << 41) == ALIAS
    assert _append(L, bad=1 << 46) == ALIAS and _append(L, bad=1 << 40) == ALIAS
    assert _append(L, _cache(v=(1 << 40) + 2048)) == ALIAS  # v's pages inside k's
    # columns of one buffer are no overlap (the driver, asked next, knows no such memory)
    wide = dict(qs=512, ks=512, vs=512, q=1 << 42, qo=1 << 42, k=(1 << 42) + 512, v=(1 << 42) + 768)
    assert _append(L, **wide) not in (ALIAS, SHAPE, OK)


def _chunk(L, c=None, q=1 << 42, qs=256, out=1 << 43, os_=256, starts=1 << 44, n=3, T=20, Hq=4, table=1 << 45, pages=8,
           lens=1 << 46, window=0, sinks=0, scale=0.1, ws=1 << 47, room=1 << 40, dtype=1):
    c = _cache() if c is None else c
    return L.gbe_attn_chunk(q, qs, out, os_, starts, n, T, Hq, ctypes.addressof(c), table, pages, lens, window, sinks,
                            scale, ws, room, dtype, None)


def test_chunk_refusals(L):
    assert _chunk(L, dtype=2) == DTYPE and _chunk(L, dtype=0) == DTYPE
    for bad in (dict(Hq=3), dict(Hq=0), dict(Hq=1), dict(n=-1), dict(n=(1 << 24) + 1), dict(T=-1), dict(T=(1 << 28) + 1),
                dict(pages=-1), dict(pages=(1 << 26) + 1), dict(qs=255), dict(os_=255), dict(window=-1), dict(sinks=-1),
                dict(Hq=65538, qs=1 << 40, os_=1 << 40), dict(T=1 << 28, Hq=1024, qs=1 << 17, os_=1 << 17)):
        assert _chunk(L, **bad) == SHAPE, bad
    assert _chunk(L, scale=float("nan")) == SCALE and _chunk(L, scale=float("inf")) == SCALE
    assert _chunk(L, T=0) == OK and _chunk(L, n=0) == OK
    long = L.gbe_attn_chunk_workspace(3, 20, 4, 2, 64, 16, 1000, 0, 0)
    assert long > 0 and _chunk(L, pages=1000, room=long - 1) == WORKSPACE and _chunk(L, pages=1000, room=-1) == WORKSPACE
    assert _chunk(L, pages=1000, ws=None) == NULL_ and _chunk(L, pages=1000, ws=(1 << 47) + 8) == ALIGN
    for name in ("q", "out", "starts", "table", "lens"):
        assert _chunk(L, **{name: None}) == NULL_, name
    for name, at in (("q", 42), ("out", 43), ("starts", 44), ("table", 45), ("lens", 46)):
        assert _chunk(L, **{name: (1 << at) + 1}) == ALIGN, name
    for at in (42, 40, 41, 44, 45, 46):
        assert _chunk(L, out=1 << at) == ALIAS, at
        assert _chunk(L, pages=1000, ws=1 << at) == ALIAS, at
    assert _chunk(L, pages=1000, ws=1 << 43) == ALIAS


def test_chunk_workspace_sizes(L):
    W = L.gbe_attn_chunk_workspace
    assert W(1, 64, 32, 8, 128, 64, 16, 0, 0) == 0          # 1024 keys: no splits
    assert W(0, 64, 32, 8, 128, 64, 2048, 0, 0) == 0 and W(4, 0, 32, 8, 128, 64, 2048, 0, 0) == 0
    assert W(1, 64, 32, 8, 128, 64, 2048, 512, 4) == 0      # a window as narrow
    one = W(1, 1, 32, 8, 128, 64, 2048, 0, 0)
    assert one > 0 and W(1, 2, 32, 8, 128, 64, 2048, 0, 0) == 2 * one
    # never more than a few rounds of CTAs of 256 rows leave for a sequence, however long its chunk
    assert W(1, 1 << 20, 32, 8, 128, 64, 1 << 14, 0, 0) <= 8 * 152 * 256 * 130 * 4
    for bad in ((-1, 1, 32, 8, 128, 64, 10, 0, 0), (1, -1, 32, 8, 128, 64, 10, 0, 0), (1, 1, 33, 8, 128, 64, 10, 0, 0),
                (1, 1, 32, 8, 100, 64, 10, 0, 0), (1, 1, 32, 8, 128, 0, 10, 0, 0), (1, 1, 32, 8, 128, 64, 1 << 25, 0, 0),
                (1, 1, 32, 8, 128, 64, 10, -1, 0), (1, 1, 32, 8, 128, 64, 10, 1, -1)):
        assert W(*bad) == -1, bad
    with pytest.raises(ValueError):
        c = gbe.KvCache.__new__(gbe.KvCache)
        c.shape = (1, 3, 16, 64)
        gbe.attn_chunk_workspace(1, 5, 4, c, 10)


def test_window_refusals(L):
    c = _cache()

    def decode(window, sinks, pages=8, room=1 << 40):
        return L.gbe_attn_decode_window(1 << 42, 256, 1 << 43, 256, 3, 4, ctypes.addressof(c), 1 << 44, pages, 1 << 45,
                                        window, sinks, 0.1, 1 << 46, room, 1, None)

    def prompt(window, sinks, out=1 << 43):
        return L.gbe_attn_prompt_window(1 << 40, 256, 1 << 41, 128, 1 << 42, 128, out, 256, 1 << 44, 2, 50, 4, 2, 64,
                                        window, sinks, 0.1, 1, None)

    for f in (decode, prompt):
        assert f(-1, 0) == SHAPE and f(5, -1) == SHAPE
        # any window and any number of sinks are taken (the driver, asked next, knows no such memory)
        for window, sinks in ((0, 0), (1, 0), (1 << 62, 1 << 62)):
            assert f(window, sinks) not in (SHAPE, OK)
    assert prompt(5, 0, out=1 << 41) == ALIAS
    W = L.gbe_attn_decode_window_workspace
    assert W(3, 4, 2, 64, 16, 1000, 0, 0) == L.gbe_attn_decode_workspace(3, 4, 2, 64, 16, 1000)
    assert W(3, 4, 2, 64, 16, 1000, 100, 4) == 0
    assert 0 < W(3, 4, 2, 64, 16, 1000, 1000, 4) < W(3, 4, 2, 64, 16, 1000, 0, 0)
    assert W(3, 4, 2, 64, 16, 1000, 1 << 62, 1 << 62) == W(3, 4, 2, 64, 16, 1000, 0, 0)
    assert W(3, 4, 2, 64, 16, 1000, -1, 0) == -1
    assert decode(1000, 4, 1000, W(3, 4, 2, 64, 16, 1000, 1000, 4) - 1) == WORKSPACE


Q, K = torch.zeros(5, 4, 64), torch.zeros(5, 2, 64)
ODD = torch.zeros(5, 64, 4).transpose(1, 2)      # [5, 4, 64] whose entries are not contiguous
ODD_K = torch.zeros(5, 64, 2).transpose(1, 2)
I5, OM, STARTS = torch.zeros(5, dtype=torch.int32), torch.zeros(32), torch.tensor([0, 5], dtype=torch.int32)
TABLE = torch.zeros(5, 1, dtype=torch.int32)


def _shape():
    c = gbe.KvCache.__new__(gbe.KvCache)  # a cache as far as its shape
    c.shape = (3, 2, 16, 64)
    c.desc = b""
    return c


CALLS = {
    "rope_kv_write a": lambda: gbe.gbe_rope_kv_write(Q, Q, ODD_K, ODD_K, I5, I5, _shape(), OM, 64),
    "rope_kv_write b": lambda: gbe.gbe_rope_kv_write(Q, Q, Q, Q, I5, I5, _shape(), OM, 64),
    "rope_kv_write c": lambda: gbe.gbe_rope_kv_write(Q, Q, K, K, I5, I5[:4], _shape(), OM, 64),
    "attn_chunk a": lambda: gbe.gbe_attn_chunk(ODD, ODD, _shape(), STARTS, TABLE[:1], I5[:1], 0.1),
    "attn_chunk b": lambda: gbe.gbe_attn_chunk(Q, Q[:4], _shape(), STARTS, TABLE[:1], I5[:1], 0.1),
    "attn_chunk c": lambda: gbe.gbe_attn_chunk(Q, Q, _shape(), STARTS, TABLE[:1], I5[:2], 0.1),
    "attn_chunk d": lambda: gbe.gbe_attn_chunk(Q, Q, _shape(), STARTS, TABLE, I5[:1], 0.1),
    "attn_chunk e": lambda: gbe.gbe_attn_chunk(Q, Q, _shape(), STARTS, TABLE[:1], I5[:1].long(), 0.1),
    "attn_chunk f": lambda: gbe.gbe_attn_chunk(Q, Q, _shape(), STARTS.long(), TABLE[:1], I5[:1], 0.1),
    "attn_decode_window a": lambda: gbe.gbe_attn_decode_window(ODD, ODD, _shape(), TABLE, I5, 4, 0, 0.1),
    "attn_decode_window b": lambda: gbe.gbe_attn_decode_window(Q, Q, _shape(), TABLE[:4], I5, 4, 0, 0.1),
    "attn_prompt_window a": lambda: gbe.gbe_attn_prompt_window(Q, K, ODD_K, Q, STARTS, 4, 0, 0.1),
    "attn_prompt_window b": lambda: gbe.gbe_attn_prompt_window(Q, K, K[:4], Q, STARTS, 4, 0, 0.1),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_binding_names_the_call(name):
    with pytest.raises(ValueError, match=f"^{name.split()[0]}: "):
        CALLS[name]()


def test_binding_wants_device_memory():
    """Shapes that fit, on the CPU."""
    for call in (lambda: gbe.gbe_attn_chunk(Q, Q, _shape(), STARTS, TABLE[:1], I5[:1], 0.1),
                 lambda: gbe.gbe_attn_decode_window(Q, Q, _shape(), TABLE, I5, 4, 0, 0.1),
                 lambda: gbe.gbe_attn_prompt_window(Q, K, K, Q, STARTS, 4, 0, 0.1),
                 lambda: gbe.gbe_rope_kv_write(Q, Q, K, K, I5, I5, _shape(), OM, 64)):
        with pytest.raises(ValueError, match="on the CUDA device"):
            call()
