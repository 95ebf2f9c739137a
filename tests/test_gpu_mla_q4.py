"""GPU tests of the paged sparse MLA attention over compressed rows held in 4
bits: against the 64-bit form over the held values, which are exact in bf16."""

import math

import numpy as np
import pytest
import torch

import sparse_attention_csa_gb300 as csa
from tests import _paged_ref as R
from tests import _q4_ref as Q
from tests.test_gpu_paged_mla import Case, i32
from tests.test_gpu_paged_timeout import sweep

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean_error_word():
    yield
    csa.csa_set_wait_limit_ns(0)
    torch.cuda.synchronize()
    assert csa.csa_device_error() == (0, 0)


class Q4Case(Case):
    """A Case whose compressed rows are held in 4 bits: `cmp4`; `cmp` are
    their values."""

    def __init__(self, *args, **kw):
        super().__init__(*args, **kw)
        self.cmp4 = None
        if self.cmp is not None:
            gen = torch.Generator().manual_seed(kw.get("seed", 0) + 77)
            self.cmp4 = Q.random_cache(gen, *self.cmp.shape[:2])
            self.cmp = Q.held(self.cmp4).cuda()
            self.cmp4 = self.cmp4.cuda()

    def args(self):
        return (self.q, self.ori, self.cmp4, None if self.idx is None else i32(self.idx),
                i32(self.ori_table), None if self.cmp is None else i32(self.cmp_table), i32(self.seq),
                i32(self.pos), self.sinks, self.scale, self.ratio, self.win_left)

    def call(self, **kw):
        return csa.csa_sparse_mla_paged_q4(*self.args(), return_softmax_lse=True, **kw)


@pytest.mark.parametrize("H", [1, 4, 33, 64])
@pytest.mark.parametrize("mode", ["list", "all", "window"])
@pytest.mark.parametrize("lens,page,win_left,new", [
    ([1], 64, 127, 1), ([700], 64, 127, 1), ([1, 2, 3, 4, 5, 63, 64, 65, 130, 257], 16, 127, 1),
    ([900, 33, 128], 40, 0, 2), ([300, 1000, 5], 7, 299, 4), ([2100], 128, 1023, 3),
])
def test_against_formula(H, mode, lens, page, win_left, new):
    lens = [max(n, new) for n in lens]
    Q4Case(lens, H, mode, topk=50, page=page, win_left=win_left, new=new, seed=H + page).check()


@pytest.mark.parametrize("sinks", [False, True])
@pytest.mark.parametrize("mode,ratio,lens", [
    ("all", 2, [9000]), ("all", 4, [20000, 31, 4097]), ("all", 128, [40000, 700, 130, 12000]),
    ("list", 4, [30000, 100, 2047, 2048, 5000]),
])
def test_split_rows(mode, ratio, lens, sinks):
    """Rows spread over many CTAs and joined."""
    Q4Case(lens, 64, mode, topk=512, ratio=ratio, cmp_page=48, sinks=sinks, seed=ratio).check()


@pytest.mark.parametrize("n_seq,new", [(200, 1), (47, 4), (330, 2)])
def test_many_tokens(n_seq, new):
    """More tokens than SMs, ragged."""
    rng = np.random.default_rng(n_seq)
    lens = rng.integers(new, 1500, n_seq)
    Q4Case(lens.tolist(), 8, "list", topk=96, new=new, page=32, seed=n_seq).check()


def test_peaked_scores():
    for seed, s in [(1, 8.0), (2, 30.0), (3, 200.0)]:
        Q4Case([6000, 513, 40], 64, "all", ratio=4, seed=seed, scale_q=s).check()


def test_repeats_bit_for_bit():
    c = Q4Case([7000, 100, 3000], 64, "list", topk=512, new=2, seed=4)
    a, la = c.call()
    ws = torch.full((csa.csa_sparse_mla_paged_workspace_size(6, 64),), 255, dtype=torch.uint8,
                    device="cuda")
    for _ in range(3):
        b, lb = c.call(workspace=ws)
        assert torch.equal(a, b) and torch.equal(la, lb)


def test_padding_and_lists():
    c = Q4Case([500, 80, 900], 16, "list", seq=[0, 5, 1, -9, 2, 0], pos=[499, -1, 79, -3, 899, 10],
               seed=5)
    out, lse = c.check()
    assert out[1].abs().max() == 0 and out[3].abs().max() == 0 and torch.isinf(lse[[1, 3]]).all()
    c = Q4Case([400, 400, 10, 3], 8, "list", topk=24, seed=7)
    rng = np.random.default_rng(8)
    for t in range(4):
        nv = (int(c.pos[t]) + 1) // 4
        row = rng.integers(-3, nv + 5, 24)
        row[rng.integers(0, 24, 4)] = 2 ** 31 - 1
        c.idx[t] = row
    c.check()
    c.idx[:] = -1
    c.check()
    c.idx[:, -1] = 0
    c.check()


@pytest.mark.parametrize("mode", ["list", "all"])
def test_evicted_and_absent_pages(mode):
    """Evicted pages are left out silently, by both forms; absent ones are
    recorded."""
    c = Q4Case([3000, 900], 24, mode, topk=200, page=16, ratio=4, seed=9)
    rng = np.random.default_rng(10)
    gone = rng.random(c.cmp_table.shape) < 0.4
    c.cmp_table[gone & (c.cmp_table >= 0)] = Q.EVICTED
    c.check()
    bf = Case.call(c)
    want, wlse, tol, ltol = c.ref()
    R.check(bf[0], want, tol)
    R.check(bf[1], wlse, ltol)
    c.cmp_table[0, :10] = 10 ** 6
    c.call()
    assert csa.csa_device_error()[0] == 6


def test_not_finite():
    """A NaN group of a row that a token sees makes that token's output NaN;
    rows that no token sees may hold anything; a NaN sink its head's."""
    c = Q4Case([700, 300], 8, "all", page=16, ratio=4, seed=12)
    vis = 700 // 4
    seen = np.zeros(c.cmp4.shape[:2], bool)
    for b, n in enumerate((700, 300)):
        for r in range(n // 4):
            seen[R.slot(c.cmp_table, 16, b, r)] = True
    c.cmp4[torch.from_numpy(~seen).cuda()] = 0x7F
    c.check()
    page, at = R.slot(c.cmp_table, 16, 0, vis - 1)
    c.cmp4[page, at, 224 + 5] = 0x7F
    out, lse = c.call()
    assert out[c.seq.tolist().index(0)].isnan().any(1).all() and lse[c.seq.tolist().index(0)].isnan().all()
    assert not out[c.seq.tolist().index(1)].isnan().any()
    c.cmp4[page, at, 224 + 5] = 0x38
    c.sinks[3] = math.nan
    out, lse = c.call()
    assert lse[:, 3].isnan().all() and not lse[:, :3].isnan().any() and out[:, 3].isnan().all()


@pytest.mark.parametrize("tokens", [3, 40, 700])
def test_waits_that_give_up(tokens):
    rng = np.random.default_rng(tokens)
    n = 20000 if tokens == 3 else 1500
    c = Q4Case([n], 16, "all", seq=np.zeros(tokens, int), pos=rng.integers(0, n, tokens), seed=13,
               win_left=300)
    args = c.args()
    want = csa.csa_sparse_mla_paged_q4(*args, return_softmax_lse=True)
    assert sweep(lambda: csa.csa_sparse_mla_paged_q4(*args), 12)
    got = csa.csa_sparse_mla_paged_q4(*args, return_softmax_lse=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_two_graphs_at_once_with_workspaces_of_their_own():
    cases = [Q4Case([5000, 77], 64, "list", topk=512, seed=20 + i) for i in range(2)]
    res = [c.call() for c in cases]
    graphs, outs = [], []
    for c in cases:
        args = c.args()
        ws = torch.empty(csa.csa_sparse_mla_paged_workspace_size(2, 64), dtype=torch.uint8, device="cuda")
        out, lse = torch.empty_like(res[0][0]), torch.empty_like(res[0][1])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=torch.cuda.Stream()):
            csa.csa_sparse_mla_paged_q4(*args, return_softmax_lse=True, workspace=ws, out=out, lse=lse)
        graphs.append((g, args, ws))
        outs.append((out, lse))
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(20):
        for (g, *_), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for (o, l), (wo, wl) in zip(outs, res):
        assert torch.equal(o, wo) and torch.equal(l, wl)


def test_offsets_beyond_32_bits():
    """Compressed pages behind 2^32 bytes of the pool, and behind 2^31 rows'
    worth of table."""
    c = Q4Case([600], 32, "all", page=128, ratio=4, seed=30)
    c.cmp4 = torch.cat([torch.zeros((90000, 128, 384), dtype=torch.uint8, device="cuda"), c.cmp4])
    want = c.ref()
    c.cmp_table = c.cmp_table + np.where(c.cmp_table >= 0, 90000, 0).astype(np.int32)
    out, lse = c.call()
    R.check(out, want[0], want[2])
    R.check(lse, want[1], want[3])
