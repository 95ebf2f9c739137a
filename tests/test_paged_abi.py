"""C-ABI checks of the rotation and paged-cache calls that need no GPU: bad
host-side arguments are rejected before anything is launched."""

import ctypes as C

import pytest

import sparse_attention_csa_gb300 as csa
from sparse_attention_csa_gb300 import build as csa_build

P, NUL = C.c_void_p(0x10000), None


@pytest.fixture(scope="module")
def L():
    csa_build.build()
    return csa.lib()


def caller(fn, base):
    def call(**kw):
        assert set(kw) <= set(base), kw
        return fn(*{**base, **kw}.values())
    return call


def test_rope_freqs_rejects(L):
    call = caller(L.csa_rope_freqs, dict(n=64, theta=1e4, factor=1.0, orig=0, fast=32.0, slow=1.0,
                                         out=P, stream=NUL))
    assert call(out=NUL) == 1
    assert call(n=0) == call(n=63) == call(n=-2) == call(orig=-1) == 2
    assert call(theta=1.0) == call(theta=float("nan")) == call(theta=float("inf")) == 3
    assert call(factor=0.5) == call(factor=float("nan")) == 3
    assert call(orig=10, slow=0.0) == call(orig=10, fast=0.5) == 3
    assert call(orig=10, fast=float("inf")) == 3


def test_rope_rejects(L):
    call = caller(L.csa_rope, dict(
        x=P, dtype=0, xs=1024, pos=P, cu=NUL, batch=0, ps=1, freq=P, T=4, H=2, D=512, off=448, n=64,
        layout=0, ms=C.c_float(1.0), inv=0, out=C.c_void_p(0x1000000), outs=1024, stream=NUL))
    for k in ("x", "out", "freq", "pos"):
        assert call(**{k: NUL}) == 1, k
    assert call(T=-1) == call(H=0) == call(D=0) == call(batch=-1) == 2
    assert call(n=0) == call(n=7) == call(off=449) == call(off=-1) == call(n=514, off=0) == 2
    assert call(xs=1023) == call(outs=1023) == 2
    assert call(off=2 ** 31 - 1) == 2
    assert call(dtype=2) == call(layout=2) == 3
    assert call(D=2048, n=1026, off=0, xs=4096, outs=4096) == 3
    assert call(x=C.c_void_p(0x10001)) == 3
    assert call(dtype=1, x=C.c_void_p(0x10002)) == 3
    assert call(out=C.c_void_p(0x10000 + 512)) == 3   # overlapping
    assert call(out=P, outs=2048) == 3                # in place, another stride
    assert call(T=0) == 0


def test_append_rejects(L):
    call = caller(L.csa_cache_append, dict(
        rows=P, dtype=0, rs=512, seq=P, pos=P, pages=P, batch=2, maxp=4, nump=8, page=16, T=3,
        width=512, freq=P, off=448, n=64, layout=0, ms=C.c_float(1.0), ps=1, cache=P, stream=NUL))
    for k in ("rows", "pos", "pages", "cache", "freq"):
        assert call(**{k: NUL}) == 1, k
    assert call(T=-1) == call(batch=-1) == call(maxp=-1) == call(nump=-1) == 2
    assert call(page=0) == call(width=0) == call(rs=511) == 2
    assert call(n=-2) == call(n=3) == call(off=450) == 2
    assert call(seq=NUL) == 2  # three rows, two sequences
    assert call(dtype=5) == call(layout=-1) == 3
    assert call(rows=C.c_void_p(0x10001)) == call(cache=C.c_void_p(0x10001)) == 3
    assert call(T=0) == 0


def test_indexer_rejects(L):
    need = L.csa_indexer_topk_paged_workspace_size(3, 64, 4, 64, 8)
    assert need >= 3 * 64 * 4
    assert L.csa_indexer_topk_paged_workspace_size(0, 64, 4, 64, 8) == 0
    assert L.csa_indexer_topk_paged_workspace_size(1 << 20, 1 << 30, 64, 128, 8) >= 1 << 52
    call = caller(L.csa_indexer_topk_paged, dict(
        q=P, k=P, w=P, pages=P, seq=P, pos=P, batch=2, T=3, Hi=4, Di=64, nump=8, page=16, maxp=4,
        r=4, topk=8, idx=P, val=NUL, ws=P, wsb=need, stream=NUL))
    for k in ("q", "k", "w", "pages", "pos", "idx"):
        assert call(**{k: NUL}) == 1, k
    assert call(T=-1) == call(topk=0) == call(page=0) == call(nump=-1) == call(maxp=-1) == 2
    assert call(maxp=2 ** 20, page=2 ** 12) == 2
    assert call(seq=NUL) == 2
    assert call(Di=96) == call(Hi=0) == call(Hi=65) == call(r=1) == call(T=65536) == 3
    assert call(q=C.c_void_p(0x10008)) == call(k=C.c_void_p(0x10008)) == 3
    assert call(ws=NUL) == call(wsb=need - 1) == call(ws=C.c_void_p(0x10010)) == 4
    assert call(T=0) == 0


def test_mla_rejects(L):
    need = L.csa_sparse_mla_paged_workspace_size(3, 4)
    assert need > 0 and L.csa_sparse_mla_paged_workspace_size(0, 4) == 0
    call = caller(L.csa_sparse_mla_paged, dict(
        q=P, ori=P, cmp=P, idx=P, op=P, cp=P, seq=P, pos=P, batch=2, T=3, H=4, D=512, on=8, ops=16,
        om=4, cn=8, cps=16, cm=4, topk=8, sinks=P, scale=C.c_float(0.04), r=4, wl=127, wr=0, out=P,
        lse=P, ret=1, ws=P, wsb=need, stream=NUL))
    for k in ("q", "ori", "op", "cp", "pos", "out", "lse"):
        assert call(**{k: NUL}) == 1, k
    assert call(T=-1) == call(H=0) == call(wl=-1) == call(ops=0) == call(cps=0) == call(topk=0) == 2
    assert call(on=-1) == call(om=-1) == call(cn=-1) == call(cm=-1) == call(batch=-1) == 2
    assert call(om=2 ** 20, ops=2 ** 12) == call(cm=2 ** 20, cps=2 ** 12) == 2
    assert call(seq=NUL) == 2
    assert call(D=576) == call(H=65) == call(wr=1) == call(r=1) == 3
    assert call(wl=2 ** 27) == call(topk=2 ** 27 + 1) == call(idx=NUL, cm=2 ** 14, cps=2 ** 14) == 3
    for k in ("q", "ori", "cmp", "out"):
        assert call(**{k: C.c_void_p(0x10008)}) == 3, k
    assert call(ws=NUL) == call(wsb=need - 1) == call(ws=C.c_void_p(0x10010)) == 4
    assert call(T=0) == 0
