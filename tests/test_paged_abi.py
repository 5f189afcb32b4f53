"""The paged decode path's entry points without a GPU: they reject bad arguments on the host,
before anything is enqueued."""

import ctypes

import pytest
import torch

import long_context_hs2_b200 as hs2
from long_context_hs2_b200 import build as hs2_build


@pytest.fixture(scope="module")
def lib():
    hs2_build.build()
    return hs2.load_library()


def cache(**kw):
    a = dict(k=16, v=16, ks=None, vs=None, weight=None, table=16, lens=16, n_pages=8, page=16,
             max_pages=4)
    a.update(kw)
    return hs2.hs2_paged_cache(hs2.hs2_kv_cache(a["k"], a["v"], a["ks"], a["vs"]), a["weight"],
                               a["table"], a["lens"], a["n_pages"], a["page"], a["max_pages"])


BAD_CACHES = [
    (dict(k=None), 1), (dict(v=8), 1), (dict(table=None), 1), (dict(lens=2), 1),
    (dict(weight=2), 1), (dict(n_pages=0), 1), (dict(page=0), 1), (dict(max_pages=0), 1),
    (dict(page=24), 2), (dict(n_pages=1 << 28, page=16), 2), (dict(max_pages=1 << 27), 2),
]


def test_rmsnorm_rejects(lib):
    f = lib.hs2_add_rmsnorm
    ok = [16, 16, 16, 4, 256, 1e-6, 16, 16, 16, 16, None]

    def call(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return f(*a)

    assert call(_0=None) == 1 and call(_0=8) == 1 and call(_2=None) == 1 and call(_1=8) == 1
    assert call(_3=0) == 1 and call(_4=0) == 1 and call(_5=-1.0) == 1
    assert call(_5=float("nan")) == 1 and call(_5=float("inf")) == 1
    assert call(_6=None, _7=None, _8=None, _9=None) == 1      # no output
    assert call(_8=None) == 1 and call(_9=None) == 1          # codes without scales, and back
    assert call(_6=8) == 1 and call(_7=8) == 1 and call(_8=8) == 1 and call(_9=2) == 1
    assert call(_4=24) == 2 and call(_4=32768 + 16) == 2 and call(_3=1 << 31) == 2


def test_fp8_gemm_rejects(lib):
    f = lib.hs2_fp8_gemm
    ok = [16, 16, 4, 16, 16, 8, 64, 16, None]
    for i in (0, 1, 3, 4, 7):
        assert f(*(ok[:i] + [None] + ok[i + 1:])) == 1
        assert f(*(ok[:i] + [2] + ok[i + 1:])) == 1
    for i in (2, 5, 6):
        assert f(*(ok[:i] + [0] + ok[i + 1:])) == 1
    assert f(*(ok[:6] + [72] + ok[7:])) == 2
    assert f(*(ok[:2] + [1 << 31] + ok[3:])) == 2


def test_append_rejects(lib):
    def call(c=None, K=16, V=16, ld=64, n=4, start=None, B=4, heads=1, D=64, dt=0):
        c = cache() if c is None else c
        return lib.hs2_paged_append(K, V, ld, n, start, ctypes.byref(c), B, heads, D, dt, None)

    for kw, st in BAD_CACHES:
        assert call(cache(**kw)) == st, kw
    assert call(K=None) == 1 and call(V=8) == 1 and call(n=0) == 1 and call(start=2) == 1
    assert call(ld=32) == 1 and call(ld=68) == 1 and call(n=5) == 1 and call(B=0) == 1
    assert call(heads=0) == 1 and call(dt=2) == 1 and call(dt=1) == 1    # E4M3 without scales
    assert call(D=96, ld=96) == 2 and call(B=65536, n=65536) == 2


def test_attn_rejects(lib):
    def call(c=None, Q=16, B=2, H=8, heads=1, D=64, scale=0.1, dt=0, O=16, lse=None, acc=0,
             ws=16, n=1 << 40):
        c = cache() if c is None else c
        return lib.hs2_paged_attn(Q, ctypes.byref(c), B, H, heads, D, scale, dt, O, lse, acc, ws,
                                  n, None)

    for kw, st in BAD_CACHES:
        assert call(cache(**kw)) == st, kw
    assert call(Q=None) == 1 and call(O=8) == 1 and call(lse=2) == 1
    assert call(scale=float("inf")) == 1 and call(H=9, heads=2) == 1 and call(H=0) == 1
    assert call(acc=1) == 1                                    # no weights to add to
    assert call(H=33) == 2 and call(D=80) == 2
    assert call(ws=None) == 4 and call(n=16) == 4
    w = lib.hs2_paged_attn_workspace
    assert w(2, 8, 1, 64) > 0 and w(2, 9, 2, 64) == 0 and w(2, 33, 1, 64) == 0
    assert w(0, 8, 1, 64) == 0 and w(2, 8, 1, 96) == 0 and w(65536, 8, 1, 64) == 0


def test_evict_rejects(lib):
    def call(c=None, B=2, heads=1, D=64, dt=0, topk=8, window=4, dst=None, dmax=0, kept=16,
             new_len=16):
        c = cache(weight=16) if c is None else c
        return lib.hs2_paged_evict(ctypes.byref(c), B, heads, D, dt, topk, window, dst, dmax,
                                   kept, new_len, None)

    for kw, st in BAD_CACHES:
        assert call(cache(**dict(dict(weight=16), **kw))) == st, kw
    assert call(cache()) == 1                                  # no weights
    assert call(kept=None) == 1 and call(new_len=2) == 1 and call(topk=-1) == 1
    assert call(window=0) == 1 and call(dst=2, dmax=4) == 1
    assert call(dst=16, dmax=0) == 1                           # 12 survivors need a page
    assert call(dst=16, dmax=3, topk=60) == 1                  # 64 need four
    assert call(topk=1 << 24) == 2


def test_binding_checks_tensors(lib):
    # on the CPU: not on the current device
    t = torch.zeros(64, dtype=torch.bfloat16)
    with pytest.raises(hs2.Hs2Error):
        hs2.hs2_add_rmsnorm(t, None, t, 1, 64, 1e-6, t, stream=0)
    with pytest.raises(hs2.Hs2Error):
        hs2.paged_cache(torch.zeros(2, 16, 1, 64), torch.zeros(2, 16, 1, 64),
                        torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    # rows that are not `ld` apart, or too few
    rows = torch.zeros(4, 64, dtype=torch.bfloat16)
    for bad in (rows[:, ::2], rows[:3], rows):
        with pytest.raises(hs2.Hs2Error):
            hs2.hs2_paged_append(bad, bad, 128, 4, None, cache(), 4, 1, 64, 0, stream=0)
