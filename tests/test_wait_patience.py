"""When a wait of a tensor-core kernel's CTA gives up: ten seconds after it began
or after the last sign of work, whichever is later.  The rule itself, compiled
here; and on the GPU a call in which some warps work for longer than that."""
import ctypes
import os
import subprocess

import pytest
import torch

import elementwise_row_rmsnorm_gb300 as gbe
from chunk_ref import i32, rand
from elementwise_row_rmsnorm_gb300 import _build

RULE = """
#include "patience.h"
// the first of n looks at which the wait gives up; -1: it does not
extern "C" int gives_up(const uint32_t* now, const int* state, int n, long long blocks) {
    gbe::Patience p;
    for (int i = 0; i < n; ++i)
        if (p.over(now[i], state[i], blocks < 0 ? gbe::kPatience : gbe::patience_for(blocks))) return i;
    return -1;
}
"""
SECOND = 10 ** 9 / 2 ** 20  # ticks


@pytest.fixture(scope="module")
def gives_up(tmp_path_factory):
    at = tmp_path_factory.mktemp("rule")
    (at / "rule.cpp").write_text(RULE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", _build.CSRC, "-o", str(at / "rule.so"),
                    str(at / "rule.cpp")], check=True)
    f = ctypes.CDLL(str(at / "rule.so")).gives_up
    f.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong]

    def call(start, seconds, state, blocks=-1):
        """The second, of looks every quarter of one, at which the wait gives up; state(second)."""
        n = 4 * seconds
        now = (ctypes.c_uint32 * n)(*[int(start + x * SECOND / 4) & 0xFFFFFFFF for x in range(n)])
        at = f(now, (ctypes.c_int * n)(*[state(x / 4) for x in range(n)]), n, blocks)
        return None if at < 0 else at / 4
    return call


STARTS = [1, 10 ** 6, 2 ** 31 - 3000, 2 ** 32 - 3000, 2 ** 32 - 1]  # (32 bits wrap around)


@pytest.mark.parametrize("start", STARTS)
def test_ten_seconds(gives_up, start):
    assert 9.75 <= gives_up(start, 100, lambda t: 0) <= 10.25


@pytest.mark.parametrize("start", STARTS)
def test_long_work_does_not_count(gives_up, start):
    assert gives_up(start, 3600, lambda t: -1) is None                     # an hour of it
    assert gives_up(start, 3600, lambda t: -(t % 9 < 1)) is None           # a second of it, eight without
    assert gives_up(start, 3600, lambda t: -3 * (t % 9 < 1)) is None
    assert 109.5 <= gives_up(start, 3600, lambda t: -2 * (t < 100)) <= 110.25, "ten seconds after its end"


def test_a_long_list_is_waited_for(gives_up):
    for blocks, least in ((0, 10), (1000, 10), (1 << 23, 3 * (1 << 23) * 1e-6 + 10)):
        at = gives_up(7, 400, lambda t: 0, blocks)
        assert least - 0.5 <= at <= 200, (blocks, at)


@pytest.mark.gpu
def test_rows_computed_again_for_longer_than_that():
    """One sequence of n keys whose list is not split (there are too many kv heads for that), most of its pages the same
    one.  The last key's v is infinite, which 127 of 128 rows do not see: a warp computes 32 of them again, key by key,
    while the CTA's others wait."""
    P, H, D, m, n = 64, 640, 8, 128, 15 << 16  # (13 s)
    k, v = (rand((1, H, P, D), torch.bfloat16, s).repeat(2, 1, 1, 1) for s in (1, 2))
    cache = gbe.KvCache(k, v)
    cache.v[1, 0, P - 1] = float("inf")
    table = torch.zeros(1, n // P, dtype=torch.int32, device="cuda")
    table[0, -1] = 1
    q = rand((m, H, D), torch.bfloat16, 3)
    out = gbe.attn_chunk(q, cache, i32([0, m]), table, i32([n]), 0.3)
    # every key's logit and v occur as often as their row of a page is seen
    p = torch.arange(n - m, n, device="cuda", dtype=torch.float64)
    r = torch.arange(P, device="cuda", dtype=torch.float64)
    seen = ((p[:, None] - r) / P).floor() + 1
    K, V = k[0].double(), v[0].double()
    w = seen.log()[None] + torch.einsum("mhd,hpd->hmp", q.double(), K) * 0.3
    w = w.softmax(-1)
    want = torch.einsum("hmp,hpd->mhd", w, V)
    # n sums in f32 of weights and products, weights of 8 bits, the result rounded once
    tol = torch.einsum("hmp,hpd->mhd", w, V.abs()) * (2 * n * 2.0 ** -24 + 2.0 ** -8 + 1e-5) + want.abs() * 2.0 ** -8
    assert bool((out[-1, 0] == float("inf")).all())
    want[-1, 0], out[-1, 0] = 0.0, 0.0
    assert bool(out.isfinite().all())
    assert bool(((out.double() - want).abs() <= tol).all())
