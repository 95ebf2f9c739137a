"""Checks of the calls around 4-bit rows and eviction that need no GPU: bad
host-side arguments are rejected before anything is launched, by the library
and by the binding; and the plain forms' own format."""

import ctypes as C

import numpy as np
import pytest
import torch

import sparse_attention_csa_gb300 as csa
from tests import _q4_ref as Q
from tests.test_paged_abi import L, NUL, P, caller  # noqa: F401
from tests.test_paged_sources import kernels, test_nothing_is_read_before_the_wait as waits_first

FAR = C.c_void_p(0x10000000)


def test_append_rejects(L):  # noqa: F811
    call = caller(L.csa_cache_append_q4, dict(
        rows=P, dtype=0, rs=512, seq=P, pos=P, pages=P, batch=2, maxp=4, nump=8, page=16, T=3,
        width=512, freq=P, off=448, n=64, layout=0, ms=C.c_float(1.0), ps=1, cache=P, stream=NUL))
    for k in ("rows", "pos", "pages", "cache", "freq"):
        assert call(**{k: NUL}) == 1, k
    assert call(T=-1) == call(batch=-1) == call(maxp=-1) == call(nump=-1) == 2
    assert call(page=0) == call(width=0) == call(rs=511) == 2
    assert call(n=-2) == call(n=3) == call(off=450) == 2
    assert call(seq=NUL) == 2
    assert call(dtype=5) == call(layout=-1) == call(width=576, off=512, rs=576) == 3
    assert call(off=447) == call(off=446, n=66) == call(off=0) == 3  # rotary dims held in 4 bits
    assert call(rows=C.c_void_p(0x10001)) == call(cache=C.c_void_p(0x10008)) == 3
    assert call(T=0) == 0


def test_read_rejects(L):  # noqa: F811
    call = caller(L.csa_cache_read_q4, dict(cache=P, pages=P, seq=P, pos=P, batch=2, maxp=4, nump=8,
                                            page=16, T=3, out=P, stream=NUL))
    for k in ("cache", "pages", "pos", "out"):
        assert call(**{k: NUL}) == 1, k
    assert call(T=-1) == call(batch=-1) == call(maxp=-1) == call(nump=-1) == call(page=0) == 2
    assert call(seq=NUL) == 2
    assert call(cache=C.c_void_p(0x10008)) == call(out=C.c_void_p(0x10008)) == 3
    assert call(T=0) == 0


def test_attention_rejects(L):  # noqa: F811
    need = L.csa_sparse_mla_paged_workspace_size(3, 4)
    call = caller(L.csa_sparse_mla_paged_q4, dict(
        q=P, ori=P, cmp=P, idx=P, op=P, cp=P, seq=P, pos=P, batch=2, T=3, H=4, D=512, on=8, ops=16,
        om=4, cn=8, cps=16, cm=4, topk=8, sinks=P, scale=C.c_float(0.04), r=4, wl=127, wr=0, out=P,
        lse=P, ret=1, ws=P, wsb=need, stream=NUL))
    for k in ("q", "ori", "op", "cp", "pos", "out", "lse"):
        assert call(**{k: NUL}) == 1, k
    assert call(T=-1) == call(H=0) == call(wl=-1) == call(ops=0) == call(cps=0) == call(topk=0) == 2
    assert call(on=-1) == call(om=-1) == call(cn=-1) == call(cm=-1) == call(batch=-1) == 2
    assert call(om=2 ** 20, ops=2 ** 12) == call(cm=2 ** 20, cps=2 ** 12) == call(seq=NUL) == 2
    assert call(D=576) == call(H=65) == call(wr=1) == call(r=1) == 3
    assert call(wl=2 ** 27) == call(topk=2 ** 27 + 1) == call(idx=NUL, cm=2 ** 14, cps=2 ** 14) == 3
    for k in ("q", "ori", "cmp", "out"):
        assert call(**{k: C.c_void_p(0x10008)}) == 3, k
    assert call(ws=NUL) == call(wsb=need - 1) == call(ws=C.c_void_p(0x10010)) == 4
    assert call(T=0) == 0


def test_mass_rejects(L):  # noqa: F811
    need = L.csa_attn_mass_paged_workspace_size(3, 8)
    assert need >= 3 * 8 * 4 and L.csa_attn_mass_paged_workspace_size(0, 8) == 0
    assert L.csa_attn_mass_paged_workspace_size(65535, 1 << 27) >= 65535 << 29
    call = caller(L.csa_attn_mass_paged, dict(
        q=P, lse=P, cmp=P, fmt=1, idx=P, pages=P, seq=P, pos=P, batch=2, T=3, H=4, D=512, nump=8,
        page=16, maxp=4, topk=8, scale=C.c_float(0.04), r=4, mass=P, out=FAR, ws=P, wsb=need,
        stream=NUL))
    for k in ("q", "lse", "cmp", "pages", "pos", "out"):
        assert call(**{k: NUL}) == 1, k
    assert call(T=-1) == call(H=0) == call(page=0) == call(nump=-1) == call(maxp=-1) == 2
    assert call(batch=-1) == call(topk=0) == call(seq=NUL) == call(maxp=2 ** 20, page=2 ** 12) == 2
    assert call(D=576) == call(H=65) == call(r=1) == call(T=65536) == call(batch=65536) == 3
    assert call(fmt=2) == call(fmt=-1) == call(topk=2 ** 27 + 1) == 3
    assert call(idx=NUL, maxp=2 ** 14, page=2 ** 14) == 3
    for k in ("q", "cmp"):
        assert call(**{k: C.c_void_p(0x10008)}) == 3, k
    assert call(mass=C.c_void_p(0x10002)) == call(out=C.c_void_p(0x10000002)) == 3
    assert call(out=C.c_void_p(0x10000 + 4)) == call(mass=C.c_void_p(0x10000000 + 508)) == 3
    assert call(ws=NUL) == call(wsb=need - 1) == call(ws=C.c_void_p(0x10010)) == 4
    assert call(batch=0) == call(maxp=0) == call(T=0, out=P) == 0
    assert call(cmp=NUL, ws=NUL) == 1 and call(cmp=NUL, nump=0, ws=NUL) == 4  # an empty pool


def test_evict_rejects(L):  # noqa: F811
    call = caller(L.csa_cache_evict, dict(
        mass=P, pages=P, rows=P, batch=2, maxp=4, page=16, keep=2, first=0, last=0,
        out=FAR, freed=C.c_void_p(0x20000000), n=P, stream=NUL))
    for k in ("mass", "pages", "rows", "out"):
        assert call(**{k: NUL}) == 1, k
    assert call(batch=-1) == call(maxp=-1) == call(page=0) == call(keep=-1) == 2
    assert call(first=-1) == call(last=-1) == call(maxp=2 ** 14, page=2 ** 18) == 2
    assert call(maxp=24577) == call(mass=C.c_void_p(0x10002)) == 3
    assert call(out=C.c_void_p(0x10000 + 4)) == call(freed=P) == call(freed=FAR) == 3
    assert call(freed=C.c_void_p(0x10000000 + 28)) == call(freed=C.c_void_p(0x10000 - 4)) == 3
    assert call(batch=0) == 0


def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_binding_refuses_cpu_tensors_and_wrong_kinds():
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    with pytest.raises(TypeError):
        csa.csa_cache_append_q4(bf(2, 512), i32(2), i32(2), i32(2, 3), u8(4, 16, 384))
    with pytest.raises(TypeError):
        csa.csa_cache_read_q4(u8(4, 16, 384), i32(2, 3), i32(2), i32(2), out=bf(2, 512))
    with pytest.raises(ValueError):
        csa.csa_cache_read_q4(u8(16, 384), i32(2, 3), i32(2), i32(2))
    with pytest.raises(TypeError):
        csa.csa_sparse_mla_paged_q4(bf(2, 4, 512), bf(4, 16, 512), u8(4, 16, 384), None, i32(2, 3),
                                    i32(2, 3), i32(2), i32(2), None, 0.05, 4, 127)
    with pytest.raises(TypeError):
        csa.csa_attn_mass_paged(bf(2, 4, 512), torch.zeros(2, 4), u8(4, 16, 384), None, i32(2, 3),
                                i32(2), i32(2), torch.zeros(2, 48), 0.05, 4, out=torch.zeros(2, 48))
    with pytest.raises(TypeError):
        csa.csa_cache_evict(torch.zeros(2, 48), i32(2, 3), i32(2), 1, out=i32(2, 3))
    with pytest.raises(TypeError):
        csa.csa_cache_evict(None, i32(2, 3), i32(2), 1)


def test_plain_format_round_trips():
    """The definition used by the tests: held values are held again as they
    are, and a value is off by at most half a step of its group's codes."""
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((20, 512)) * np.exp(rng.standard_normal((20, 1)))).astype(np.float32)
    b = Q.pack(x.astype(np.float64))
    y = Q.unpack(b)
    again = y.copy()
    assert np.array_equal(Q.unpack(Q.pack(again))[:, 448:], y[:, 448:])
    g, h = x[:, :448].reshape(20, 28, 16), y[:, :448].reshape(20, 28, 16)
    top = np.abs(g).max(2, keepdims=True)
    # the widest step (4 to 6) is a third of the scale's 6, the scale off by 2^-4
    assert (np.abs(g - h) <= top / 6 * (1 + 2.0 ** -4) + top * 2.0 ** -4).all()
    assert np.abs(h[np.abs(g) == top]).min() > 0


@pytest.mark.parametrize("name,expected", [
    ("cache_q4.cu", {"cache_append_q4_kernel", "cache_read_q4_kernel"}),
    ("attn_mass.cu", {"attn_weight_kernel", "attn_mass_all_kernel", "attn_mass_list_kernel"}),
    ("cache_evict.cu", {"cache_evict_kernel"}),
])
def test_nothing_is_read_before_the_wait(name, expected):
    """As in the paged kernels: what a launch that starts early touches lies
    behind its wait for the kernels before it."""
    waits_first(name, expected)
    for kernel in expected:
        body = kernels(name)[kernel]
        ahead = body[:body.index("grid_dependency_wait();")]
        for touch in ("token_slots(", "find_row(", "a.rows[", "a.pages[", "table["):
            assert touch not in ahead, f"{kernel}: {touch} before the wait"


def test_waits_of_whole_warps_are_voted():
    """A warp's lanes go on alike after a wait of the weight kernel: every one
    outside the thread that issues MMAs is voted on."""
    body = kernels("attn_mass.cu")["attn_weight_kernel"]
    one_lane = body[body.index("if (lane == 0) {\n                constexpr"):body.index("__syncwarp();\n        } else if")]
    import re
    rest = body.replace(one_lane, "")
    waits = [" ".join(x.split()) for x in re.split(r"[;{}]", rest) if "cx.wait(" in x]
    assert len(waits) == 6
    for x in waits:
        assert "__all_sync(0xffffffffu, cx.wait(" in x, x
