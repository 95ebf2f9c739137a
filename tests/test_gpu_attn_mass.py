"""GPU tests of the attention weight that cached rows received, against the
64-bit form."""

import math

import numpy as np
import pytest
import torch

import sparse_attention_csa_gb300 as csa
from tests import _paged_ref as R
from tests import _q4_ref as Q
from tests.test_gpu_mla_q4 import Q4Case, i32
from tests.test_gpu_paged_timeout import sweep

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean_error_word():
    yield
    csa.csa_set_wait_limit_ns(0)
    torch.cuda.synchronize()
    assert csa.csa_device_error() == (0, 0)


class Mass:
    """A case's attention (its lse) and the weight its rows received."""

    def __init__(self, *args, bits=4, **kw):
        self.c = c = Q4Case(*args, **kw)
        _, self.lse = c.call()
        self.rows = c.cmp4 if bits == 4 else c.cmp
        gen = torch.Generator().manual_seed(5)
        self.base = torch.rand((c.cmp_table.shape[0], c.cmp_table.shape[1] * c.cmp.shape[1]),
                               generator=gen).cuda()

    def args(self, mass):
        c = self.c
        return (c.q, self.lse, self.rows, None if c.idx is None else i32(c.idx), i32(c.cmp_table),
                i32(c.seq), i32(c.pos), mass, c.scale, c.ratio)

    def call(self, mass="base", **kw):
        return csa.csa_attn_mass_paged(*self.args(self.base if isinstance(mass, str) else mass), **kw)

    def ref(self, base="base"):
        c = self.c
        return Q.mass(c.q, self.lse, c.cmp, c.idx, c.cmp_table, c.seq, c.pos,
                      self.base if isinstance(base, str) else base, c.scale, c.ratio)

    def check(self, mass="base", **kw):
        got = self.call(mass, **kw)
        want, tol = self.ref(mass)
        R.check(got, want, tol, "mass")
        return got


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("H", [1, 4, 33, 64])
@pytest.mark.parametrize("mode", ["list", "all"])
@pytest.mark.parametrize("lens,page,new", [
    ([1], 64, 1), ([700], 64, 1), ([1, 2, 3, 4, 5, 63, 64, 65, 130, 257], 16, 1),
    ([900, 33, 128], 40, 2), ([300, 1000, 5], 7, 4), ([2100], 128, 3),
])
def test_against_formula(bits, H, mode, lens, page, new):
    lens = [max(n, new) for n in lens]
    Mass(lens, H, mode, topk=50, page=page, new=new, seed=H + page, bits=bits).check()


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("mode,ratio,lens,new", [
    ("all", 2, [9000], 1), ("all", 4, [20000, 31, 4097], 2), ("all", 128, [40000, 700, 130, 12000], 1),
    ("list", 4, [30000, 100, 2047, 2048, 5000], 3),
])
def test_long_rows(bits, mode, ratio, lens, new):
    Mass([max(n, new) for n in lens], 64, mode, topk=512, ratio=ratio, cmp_page=48, new=new,
         seed=ratio, bits=bits).check()


@pytest.mark.parametrize("n_seq,new,mode", [(200, 1, "list"), (47, 4, "all"), (330, 2, "list"),
                                            (3, 120, "list"), (2, 300, "all")])
def test_many_tokens(n_seq, new, mode):
    rng = np.random.default_rng(n_seq)
    lens = rng.integers(new, 1500, n_seq)
    Mass(lens.tolist(), 8, mode, topk=96, new=new, page=32, seed=n_seq).check()


@pytest.mark.parametrize("mode", ["list", "all"])
def test_in_place_and_from_nothing(mode):
    m = Mass([500, 3000, 60], 16, mode, topk=40, new=2, seed=3)
    want = m.call()
    fresh = m.call(None)
    assert torch.equal(fresh, m.call(torch.zeros_like(m.base)))
    R.check(fresh, *m.ref(None), "from nothing")
    mine = m.base.clone()
    assert csa.csa_attn_mass_paged(*m.args(mine), out=mine) is mine and torch.equal(mine, want)
    # rows that received nothing keep their bits, whatever they are
    got = fresh != 0
    odd = torch.where(got, m.base, torch.full_like(m.base, math.nan))
    odd[:, ::2] = torch.where(got[:, ::2], odd[:, ::2], torch.full_like(odd[:, ::2], -0.0))
    bits = odd.view(torch.int32).clone()
    csa.csa_attn_mass_paged(*m.args(odd), out=odd)
    assert torch.equal(odd.view(torch.int32)[~got], bits[~got])
    assert torch.equal(odd[got], want[got])


def test_lists_with_what_they_may_hold():
    """Entries repeated (each counts), out of order, negative, not visible."""
    m = Mass([400, 400, 10, 3], 8, "list", topk=24, seed=7)
    c = m.c
    rng = np.random.default_rng(8)
    for t in range(4):
        nv = (int(c.pos[t]) + 1) // 4
        row = rng.integers(-3, nv + 5, 24)
        row[rng.integers(0, 24, 4)] = 2 ** 31 - 1
        row[5] = row[6] = row[7] = 0
        c.idx[t] = row
    _, m.lse = c.call()
    m.check()
    a = m.call()
    for _ in range(3):
        assert torch.equal(a, m.call())
    c.idx[:] = -1
    assert torch.equal(m.call(), m.base)


def test_padding_and_sequences_in_any_order():
    m = Mass([500, 80, 900], 16, "all", seq=[0, 5, 1, -9, 2, 0, 2, 0], seed=5,
             pos=[499, -1, 79, -3, 899, 10, 2, 498])
    m.check()
    m.c.seq[2] = 3
    m.call()
    assert csa.csa_device_error()[0] == 6
    m.c.pos[:] = -1
    assert torch.equal(m.call(), m.base)


def test_heads_without_lse_and_values_not_finite():
    m = Mass([300, 200], 8, "all", page=16, seed=6)
    m.lse[0, 3] = -math.inf
    m.check()
    b = int(m.c.seq[0])
    m.lse[0, 4] = math.nan        # this token's weights count as 0
    got = m.call()
    assert torch.equal(got[b], m.base[b]) and not got.isnan().any()
    m.lse[0, 4] = -300.0          # not this attention's
    got = m.call() - m.base
    assert (got[b] <= 8.001).all() and got.isfinite().all()


@pytest.mark.parametrize("mode", ["list", "all"])
def test_evicted_and_absent_pages(mode):
    m = Mass([3000, 900], 24, mode, topk=200, page=16, seed=9)
    t = m.c.cmp_table
    t[(np.random.default_rng(1).random(t.shape) < 0.4) & (t >= 0)] = Q.EVICTED
    m.check()
    t[0, :10] = -1
    got = m.call()
    assert csa.csa_device_error()[0] == 6
    R.check(got, *m.ref(), "mass")


def test_no_tokens_and_no_rows():
    m = Mass([300], 8, "all", seed=6)
    c = m.c
    e = lambda *s, dt=torch.bfloat16: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
    got = csa.csa_attn_mass_paged(e(0, 8, 512), e(0, 8, dt=torch.float32), m.rows, None, i32(c.cmp_table),
                                  i32([]), i32([]), m.base, c.scale, 4)
    assert torch.equal(got, m.base)
    got = csa.csa_attn_mass_paged(c.q, m.lse, m.rows[:0], None, i32(np.zeros((1, 0))), i32(c.seq),
                                  i32(c.pos), None, c.scale, 4)
    assert got.shape == (1, 0)


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("tokens", [3, 40, 700])
def test_waits_that_give_up(tokens, bits):
    rng = np.random.default_rng(tokens)
    n = 40000 if tokens == 3 else 1500
    m = Mass([n], 16, "all", seq=np.zeros(tokens, int), pos=rng.integers(0, n, tokens), seed=13, bits=bits)
    args = m.args(m.base)
    want = csa.csa_attn_mass_paged(*args)
    sweep(lambda: csa.csa_attn_mass_paged(*args), 14)
    assert torch.equal(csa.csa_attn_mass_paged(*args), want)


def test_captured_and_replayed():
    m = Mass([5000, 77], 64, "list", topk=512, seed=20)
    args, out = m.args(m.base), torch.empty_like(m.base)
    want = m.call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        csa.csa_attn_mass_paged(*args, out=out)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_offsets_beyond_32_bits():
    m = Mass([600], 32, "all", page=128, seed=30)
    want = m.ref()
    m.rows = torch.cat([torch.zeros((90000, 128, 384), dtype=torch.uint8, device="cuda"), m.rows])
    t = m.c.cmp_table
    m.c.cmp_table = t + np.where(t >= 0, 90000, 0).astype(np.int32)
    R.check(m.call(), *want, "mass")


@pytest.mark.parametrize("mode", ["list", "all"])
def test_wide_table_and_empty_pool(mode):
    """A table much wider than its sequences, and one without any page."""
    m = Mass([900, 50], 8, mode, topk=100, page=64, seed=31)
    t = m.c.cmp_table
    wide = np.full((2, 5000), -1, np.int32)
    wide[:, :t.shape[1]] = t
    m.c.cmp_table = wide
    m.base = torch.rand((2, 5000 * 64), generator=torch.Generator().manual_seed(1)).cuda()
    m.check()
    m.c.cmp_table[:] = -1
    m.rows = m.rows[:0]
    got = m.call()
    assert csa.csa_device_error()[0] == 6
    assert torch.equal(got, m.base)


def test_two_graphs_at_once_with_workspaces_of_their_own():
    ms = [Mass([5000, 77], 64, "list", topk=512, seed=40 + i, bits=b) for i, b in enumerate((4, 16))]
    want = [m.call() for m in ms]
    graphs = []
    for m in ms:
        args, out = m.args(m.base), torch.empty_like(m.base)
        ws = torch.empty(csa.csa_attn_mass_paged_workspace_size(2, 512), dtype=torch.uint8, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=torch.cuda.Stream()):
            csa.csa_attn_mass_paged(*args, out=out, workspace=ws)
        graphs.append((g, args, ws, out))
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(20):
        for (g, *_), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for (_, _, _, out), w in zip(graphs, want):
        assert torch.equal(out, w)


@pytest.mark.parametrize("bits", [4, 16])
def test_more_tokens_than_threads(bits):
    """More tokens than one pass over them holds, few of each sequence."""
    rng = np.random.default_rng(50)
    lens = rng.integers(5, 400, 650)
    Mass(lens.tolist(), 4, "list", topk=20, new=2, page=16, seed=51, bits=bits).check()
