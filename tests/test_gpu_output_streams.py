"""The calls that allocate their outputs, given a stream: the memory comes from
that stream's pool and not from the current one's, where queued work may still
use it, and it goes back to its pool only when the current stream, which may
read the result, is done with it as well."""
import pytest
import torch

import elementwise_row_rmsnorm_gb300 as gbe

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
T, Hq, H, D, P = 2048, 16, 8, 128, 64


def _rand(*shape, dtype=BF, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _decode():
    cache = gbe.kv_cache(T // P, H, P, D)
    cache.k.copy_(_rand(*cache.shape, seed=2))
    cache.v.copy_(_rand(*cache.shape, seed=3))
    q, table, lens = _rand(4, Hq, D), torch.arange(T // P, dtype=torch.int32, device="cuda").repeat(4, 1), _i32([T] * 4)
    return lambda s: gbe.attn_decode(q, cache, table, lens, stream=s)


def _read():
    cache = gbe.kv_cache(T // P, H, P, D)
    cache.k.copy_(_rand(*cache.shape, seed=2))
    cache.v.copy_(_rand(*cache.shape, seed=3))
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    return lambda s: gbe.kv_read(cache, slots, stream=s)


def _prompt():
    q, k, v, starts = _rand(T, Hq, D), _rand(T, H, D, seed=2), _rand(T, H, D, seed=3), _i32([0, 700, T])
    return lambda s: gbe.attn_prompt(q, k, v, starts, stream=s)


def _simple(name):
    x, w, y = _rand(T, Hq * D), _rand(Hq * D, seed=2), _rand(T, Hq * D, seed=3)
    om = torch.rand(D // 2, device="cuda")
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    u = torch.rand(T, device="cuda")
    return {
        "rmsnorm": lambda s: gbe.rmsnorm(x, w, stream=s),
        "layernorm": lambda s: gbe.layernorm(x, w, w, stream=s),
        "add_rmsnorm": lambda s: gbe.add_rmsnorm(x, y, w, stream=s),
        "rope": lambda s: gbe.rope(x.view(T, Hq, D), pos, om, D, stream=s),
        "rope_cos_sin": lambda s: gbe.rope_cos_sin(om, D, T, stream=s),
        "silu_mul": lambda s: gbe.silu_mul(x, y, stream=s),
        "add": lambda s: gbe.add(x, y, stream=s),
        "embedding": lambda s: gbe.embedding(x, pos, stream=s),
        "argmax": lambda s: gbe.argmax(x, stream=s),
        "sample": lambda s: gbe.sample(x, u, "temperature", stream=s),
        "sample_seeded": lambda s: gbe.sample_seeded(x, "temperature", 7, stream=s),
        "pcg64_uniforms": lambda s: gbe.pcg64_uniforms(1 << 20, 7, stream=s),
    }[name]


SIMPLE = ["rmsnorm", "layernorm", "add_rmsnorm", "rope", "rope_cos_sin", "silu_mul", "add", "embedding", "argmax", "sample",
          "sample_seeded", "pcg64_uniforms"]


def _make(name):
    return {"attn_decode": _decode, "kv_read": _read, "attn_prompt": _prompt}.get(name, lambda: _simple(name))()


def _outputs(got):
    return got if isinstance(got, tuple) else (got,)


@pytest.mark.parametrize("name", ["attn_decode", "kv_read", "attn_prompt"] + SIMPLE)
@pytest.mark.parametrize("as_handle", [False, True])
def test_outputs_come_from_the_pool_of_the_stream_given(name, as_handle):
    call = _make(name)
    want = [x.clone() for x in _outputs(call(None))]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    # blocks of the outputs' sizes, free on the current stream, and on it alone
    free = [torch.empty_like(x) for x in want for _ in range(2)]
    mine = {x.data_ptr() for x in free}
    del free
    got = _outputs(call(side.cuda_stream if as_handle else side))
    torch.cuda.synchronize()
    assert not mine & {x.data_ptr() for x in got}, "memory that the current stream's queued work may still use"
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", ["attn_decode", "kv_read", "attn_prompt", "rmsnorm", "argmax"])
def test_outputs_go_back_when_the_current_stream_is_done_with_them(name):
    call = _make(name)
    side = torch.cuda.Stream()
    big = torch.zeros(1 << 28, device="cuda")
    like = [(x.shape, x.dtype) for x in _outputs(call(None))]
    with torch.cuda.stream(side):  # blocks to spare, so that nothing below asks the driver for memory
        spare = [torch.empty(s, dtype=t, device="cuda") for s, t in like for _ in range(3)]
    del spare
    torch.cuda.synchronize()
    got = _outputs(call(side))
    torch.cuda.synchronize()
    for _ in range(50):
        big.add_(1.0)  # the current stream is busy, as with a reader of the outputs
    where = {x.data_ptr() for x in got}
    del got
    with torch.cuda.stream(side):
        new = [torch.empty(s, dtype=t, device="cuda") for s, t in like]
    assert not torch.cuda.current_stream().query(), "the current stream was to be busy still"
    assert not where & {x.data_ptr() for x in new}
    torch.cuda.synchronize()


def test_the_default_streams_handle():
    """0 names the legacy default stream: the current one here."""
    call = _make("attn_decode")
    want = call(None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert torch.equal(call(0), want)
    with torch.cuda.stream(side):
        free = torch.empty_like(want)
        mine = free.data_ptr()
        del free
        got = call(0)
        torch.cuda.synchronize()
        assert got.data_ptr() != mine and torch.equal(got, want)


@pytest.mark.parametrize("name", ["attn_decode", "kv_read", "attn_prompt", "rmsnorm"])
@pytest.mark.parametrize("forked", [True, False])
def test_calls_with_a_stream_may_be_captured(name, forked):
    """On a stream forked from the capturing one, and on that one itself; replayed beside other work."""
    call = _make(name)
    want = [x.clone() for x in _outputs(call(None))]
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        s = side if forked else here
        if forked:
            side.wait_stream(here)
        dropped = call(s)
        del dropped
        got = _outputs(call(s))
        if forked:
            here.wait_stream(side)
        sums = [x.float().sum() for x in got]
    for _ in range(3):
        graph.replay()
        other = call(side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(torch.equal(a, b) for a, b in zip(_outputs(other), want))
        assert all(torch.equal(a, b.float().sum()) for a, b in zip(sums, want))
    del got, sums, graph
    torch.cuda.synchronize()
