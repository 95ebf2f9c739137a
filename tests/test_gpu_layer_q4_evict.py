"""GPU tests of a layer continued over compressed rows held in 4 bits, weighed
and given back, as a server uses the calls together: prompt rows appended, steps
that add up the weight of their rows, eviction, and steps over what is left;
each against the 64-bit forms. And the same step captured into a graph."""

import numpy as np
import pytest
import torch

import sparse_attention_csa_gb300 as csa
from sparse_attention_csa_gb300.pipeline import PagedLayerCache, csa_layer_decode, csa_layer_evict
from tests import _paged_ref as R
from tests import _q4_ref as Q

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean_error_word():
    yield
    torch.cuda.synchronize()
    assert csa.csa_device_error() == (0, 0)


def i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


class Layer:
    def __init__(self, lens, H, room=40, bits=4, ratio=4, page=16, Hi=8, Di=64, seed=0):
        self.gen = g = torch.Generator().manual_seed(seed)
        self.lens, self.H, self.ratio, self.page, self.Hi, self.Di = lens, H, ratio, page, Hi, Di
        ends = [n + room for n in lens]
        self.ori_t, no = R.pool_rows(ends, page, seed=seed)
        self.cmp_t, nc = R.pool_rows([n // ratio for n in ends], page, seed=seed + 1)
        cmp = (torch.zeros((nc, page, 384), dtype=torch.uint8) if bits == 4
               else torch.zeros((nc, page, 512), dtype=torch.bfloat16))
        self.cache = PagedLayerCache(
            ori=torch.randn((no, page, 512), generator=g).bfloat16().cuda(), ori_pages=i32(self.ori_t),
            cmp=cmp.cuda(), cmp_pages=i32(self.cmp_t),
            k_idx=R.grid(g, (nc, page, Di), 0.5, torch.bfloat16).cuda(),
            mass=torch.zeros((len(lens), self.cmp_t.shape[1] * page), device="cuda"))
        self.sinks = torch.randn((H,), generator=g).cuda()
        # every compressed row there will be (fp32, as the compressor leaves it)
        seq = np.repeat(np.arange(len(lens)), [n // ratio for n in ends])
        pos = np.concatenate([np.arange(n // ratio) for n in ends])
        rows = torch.randn((len(seq), 512), generator=g)
        inv = csa.csa_rope_freqs(64)
        put = csa.csa_cache_append_q4 if bits == 4 else csa.csa_cache_append
        put(rows.cuda(), i32(seq), i32(pos), self.cache.cmp_pages, self.cache.cmp, inv_freq=inv,
            pos_stride=ratio)
        self.scale = R.inv_sqrt(512)

    def values(self):
        return Q.held(self.cache.cmp) if self.cache.cmp.dtype == torch.uint8 else self.cache.cmp

    def tokens(self, T):
        g = self.gen
        return dict(q=torch.randn((T, self.H, 512), generator=g).bfloat16().cuda(),
                    kv=torch.randn((T, 512), generator=g).bfloat16().cuda(),
                    q_idx=R.grid(g, (T, self.Hi, self.Di), 0.5, torch.bfloat16).cuda(),
                    w=R.grid(g, (T, self.Hi), 0.125, torch.float32).cuda())

    def step(self, t, seq, pos, indexer, topk, **kw):
        return csa_layer_decode(t["q"], t["kv"], self.cache, i32(seq), i32(pos), self.sinks, self.scale,
                                self.ratio, 31, q_idx=t["q_idx"] if indexer else None, w=t["w"],
                                topk=topk if indexer else 0, return_softmax_lse=True, **kw)

    def check(self, t, res, seq, pos, mass_before, indexer, topk):
        table = self.cache.cmp_pages.cpu().numpy()
        idx = None
        if indexer:
            idx = res.topk_idx.cpu().numpy()
            for k, (b, p) in enumerate(zip(seq, pos)):  # the best of the rows that are left
                live = [j for j in range((p + 1) // self.ratio) if R.slot(table, self.page, b, j)]
                rows, keys = R.gather(self.cache.k_idx, table, self.page, b, live)
                s = np.maximum(keys @ R.f64(t["q_idx"])[k].T, 0.0) @ R.f64(t["w"])[k]
                best = sorted(np.asarray(rows)[np.argsort(-s, kind="stable")[:topk]])
                got = [j for j in idx[k] if j >= 0 and R.slot(table, self.page, b, j)]
                assert got == best
        want, wlse, tol, ltol = R.attention(t["q"], self.cache.ori, self.values(), idx, self.ori_t, table,
                                            seq, pos, self.sinks, self.scale, self.ratio, 31)
        R.check(res.out, want, tol, "out")
        R.check(res.lse, wlse, ltol, "lse")
        mass, mtol = Q.mass(t["q"], res.lse, self.values(), idx, table, seq, pos, mass_before,
                            self.scale, self.ratio)
        R.check(self.cache.mass, mass, mtol, "mass")


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("indexer", [True, False])
def test_steps_eviction_and_steps_after(indexer, bits):
    lens, topk = [1500, 333, 70], 60
    L = Layer(lens, H=12, bits=bits, seed=bits)
    for step in range(5):
        seq = [0, 0, 1, 1, 2, 2]
        pos = [n + 2 * step + k for n in lens for k in (0, 1)]
        t, before = L.tokens(6), L.cache.mass.clone()
        res = L.step(t, seq, pos, indexer, topk)
        L.check(t, res, seq, pos, before, indexer, topk)
        if step == 2:
            rows = [(n + 2 * step + 2) // 4 for n in lens]
            table, mass = L.cache.cmp_pages.cpu().numpy(), L.cache.mass.cpu().numpy()
            freed, n_freed = csa_layer_evict(L.cache, i32(rows), 8, keep_first=4, keep_last=20)
            want = Q.evict(mass, table, rows, L.page, 8, 4, 20)
            assert np.array_equal(L.cache.cmp_pages.cpu().numpy(), want[0])
            assert np.array_equal(freed.cpu().numpy(), want[1])
            assert n_freed.tolist() == want[2].tolist() and want[2][0] > 0 and want[2][2] == 0
            # what is given back may be used by others at once
            gone = [p for r in want[1] for p in r if p >= 0]
            L.cache.cmp[gone] = 0x7F if bits == 4 else float("nan")
            if bits == 4:  # NaN scales: a row that is still read would show
                assert torch.isnan(Q.held(L.cache.cmp[gone])).any()


def test_step_captured_into_a_graph():
    lens = [900, 120]
    L = Layer(lens, H=16, seed=5)
    t = L.tokens(2)
    seq, pos = i32([0, 1]), i32([n + 3 for n in lens])
    args = (t["q"], t["kv"], L.cache, seq, pos, L.sinks, L.scale, 4, 31)
    kw = dict(q_idx=t["q_idx"], w=t["w"], topk=40, return_softmax_lse=True)
    first = csa_layer_decode(*args, **kw)
    mass = L.cache.mass.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        res = csa_layer_decode(*args, **kw)
    for _ in range(3):
        L.cache.mass.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(res.out, first.out) and torch.equal(res.topk_idx, first.topk_idx)
        assert torch.equal(L.cache.mass, mass)


def test_without_a_weight_nothing_else_changes():
    """A cache without `mass`: the step as it was, no LSE unless asked for."""
    L = Layer([500], H=8, seed=6)
    t = L.tokens(1)
    L.cache.mass = None
    res = csa_layer_decode(t["q"], t["kv"], L.cache, None, i32([500]), L.sinks, L.scale, 4, 31)
    assert res.lse is None and res.topk_idx is None
    want = R.attention(t["q"], L.cache.ori, L.values(), None, L.ori_t, L.cmp_t, [0], [500], L.sinks,
                       L.scale, 4, 31)
    R.check(res.out, want[0], want[2], "out")


def test_calls_on_a_stream_of_their_own():
    """Each call on a stream that is not the current one, results made by the
    call: as on the current stream."""
    L = Layer([700, 90], H=8, seed=7)
    t = L.tokens(2)
    seq, pos = i32([0, 1]), i32([701, 91])
    args = (t["q"], L.cache.ori, L.cache.cmp, None, L.cache.ori_pages, L.cache.cmp_pages, seq, pos,
            L.sinks, L.scale, 4, 31)
    out, lse = csa.csa_sparse_mla_paged_q4(*args, return_softmax_lse=True)
    margs = (t["q"], lse, L.cache.cmp, None, L.cache.cmp_pages, seq, pos, None, L.scale, 4)
    mass = csa.csa_attn_mass_paged(*margs)
    eargs = (mass, L.cache.cmp_pages, i32([175, 22]), 5)
    gone = csa.csa_cache_evict(*eargs)
    back = csa.csa_cache_read_q4(L.cache.cmp, L.cache.cmp_pages, seq, i32([9, 3]))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    o2, l2 = csa.csa_sparse_mla_paged_q4(*args, return_softmax_lse=True, stream=s)
    m2 = csa.csa_attn_mass_paged(*margs, stream=s)
    g2 = csa.csa_cache_evict(*eargs, stream=s)
    b2 = csa.csa_cache_read_q4(L.cache.cmp, L.cache.cmp_pages, seq, i32([9, 3]), stream=s)
    s.synchronize()
    assert torch.equal(o2, out) and torch.equal(l2, lse) and torch.equal(m2, mass) and torch.equal(b2, back)
    assert all(torch.equal(x, y) for x, y in zip(g2, gone))


def test_written_tensors_count_as_changed_in_place():
    L = Layer([300], H=8, seed=8)
    t = L.tokens(1)
    pos = i32([300])
    for name, call in {
        "cmp": lambda: csa.csa_cache_append_q4(torch.zeros((1, 512), device="cuda"), None, i32([2]),
                                               L.cache.cmp_pages, L.cache.cmp),
        "mass": lambda: csa.csa_attn_mass_paged(t["q"], torch.zeros((1, 8), device="cuda"), L.cache.cmp, None,
                                                L.cache.cmp_pages, None, pos, L.cache.mass, 0.04, 4,
                                                out=L.cache.mass),
        "cmp_pages": lambda: csa.csa_cache_evict(L.cache.mass, L.cache.cmp_pages, i32([75]), 9,
                                                 out=L.cache.cmp_pages),
    }.items():
        x = getattr(L.cache, name)
        v = x._version
        call()
        assert x._version > v, name
