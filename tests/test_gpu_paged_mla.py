"""GPU tests of the paged sparse MLA attention: against the 64-bit form, and
chained with the append and the indexer against the packed forward's oracle."""

import math

import numpy as np
import pytest
import torch

import oracle
import sparse_attention_csa_gb300 as csa
from tests import _paged_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean_error_word():
    yield
    torch.cuda.synchronize()
    assert csa.csa_device_error() == (0, 0)


def i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


class Case:
    """Sequences of the given lengths with `new` tokens each at their ends."""

    def __init__(self, lens, H, mode, topk=16, ratio=4, win_left=127, page=64, cmp_page=None,
                 new=1, sinks=True, seed=0, scale_q=1.0, pos=None, seq=None):
        gen = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.ratio, self.win_left, self.scale = ratio, win_left, R.inv_sqrt(512)
        cmp_page = cmp_page or page
        if seq is None:
            seq = np.repeat(np.arange(len(lens)), new)
            pos = np.concatenate([np.arange(n - new, n) for n in lens])
            perm = rng.permutation(len(seq))
            seq, pos = seq[perm], pos[perm]
        self.seq, self.pos = np.asarray(seq), np.asarray(pos)
        T = len(self.seq)
        low = [int(min([max(0, p - win_left) for s, p in zip(self.seq, self.pos)
                        if s == b and p >= 0] or [n])) for b, n in enumerate(lens)]
        self.ori_table, total = R.pool_rows(lens, page, seed=seed, keep_from=low)
        self.ori = torch.randn((total, page, 512), generator=gen).bfloat16().cuda()
        self.q = (scale_q * torch.randn((T, H, 512), generator=gen)).bfloat16().cuda()
        self.sinks = torch.randn((H,), generator=gen).cuda() if sinks else None
        self.cmp = self.cmp_table = self.idx = None
        if mode != "window":
            vis = [n // ratio for n in lens]
            self.cmp_table, total = R.pool_rows(vis, cmp_page, seed=seed + 1)
            self.cmp = torch.randn((total, cmp_page, 512), generator=gen).bfloat16().cuda()
        if mode == "list":
            self.idx = np.full((T, topk), -1, np.int32)
            for t in range(T):
                nv = (int(self.pos[t]) + 1) // ratio
                k = min(nv, topk)
                if k > 0:
                    self.idx[t, :k] = np.sort(rng.choice(nv, k, replace=False))

    def call(self, **kw):
        return csa.csa_sparse_mla_paged(
            self.q, self.ori, self.cmp, None if self.idx is None else i32(self.idx),
            i32(self.ori_table), None if self.cmp is None else i32(self.cmp_table), i32(self.seq),
            i32(self.pos), self.sinks, self.scale, self.ratio, self.win_left,
            return_softmax_lse=True, **kw)

    def ref(self):
        return R.attention(self.q, self.ori, self.cmp, self.idx, self.ori_table, self.cmp_table,
                           self.seq, self.pos, self.sinks, self.scale, self.ratio, self.win_left)

    def check(self, **kw):
        out, lse = self.call(**kw)
        want, wlse, tol, ltol = self.ref()
        R.check(out, want, tol, "out")
        R.check(lse, wlse, ltol, "lse")
        return out, lse


@pytest.mark.parametrize("H", [1, 4, 33, 64])
@pytest.mark.parametrize("mode", ["list", "all", "window"])
@pytest.mark.parametrize("lens,page,win_left,new", [
    ([1], 64, 127, 1), ([700], 64, 127, 1), ([1, 2, 3, 4, 5, 63, 64, 65, 130, 257], 16, 127, 1),
    ([900, 33, 128], 40, 0, 2), ([300, 1000, 5], 7, 299, 4), ([2100], 128, 1023, 3),
])
def test_against_formula(H, mode, lens, page, win_left, new):
    lens = [max(n, new) for n in lens]
    Case(lens, H, mode, topk=50, page=page, win_left=win_left, new=new, seed=H + page).check()


@pytest.mark.parametrize("sinks", [False, True])
@pytest.mark.parametrize("mode,ratio,lens", [
    ("all", 2, [9000]), ("all", 4, [20000, 31, 4097]), ("all", 128, [40000, 700, 130, 12000]),
    ("list", 4, [30000, 100, 2047, 2048, 5000]),
])
def test_split_rows(mode, ratio, lens, sinks):
    """Rows spread over many CTAs and joined."""
    Case(lens, 64, mode, topk=512, ratio=ratio, cmp_page=48, sinks=sinks, seed=ratio).check()


@pytest.mark.parametrize("n_seq,new", [(200, 1), (47, 4), (330, 2)])
def test_many_tokens(n_seq, new):
    """More tokens than SMs, ragged."""
    rng = np.random.default_rng(n_seq)
    lens = rng.integers(new, 1500, n_seq)
    Case(lens.tolist(), 8, "list", topk=96, new=new, page=32, seed=n_seq).check()


def test_peaked_scores():
    """Large logits: single keys dominate, the maximum moves between tiles and
    between the parts of a row."""
    for seed, s in [(1, 8.0), (2, 30.0), (3, 200.0)]:
        Case([6000, 513, 40], 64, "all", ratio=4, seed=seed, scale_q=s).check()


def test_repeats_bit_for_bit():
    c = Case([7000, 100, 3000], 64, "list", topk=512, new=2, seed=4)
    a, la = c.call()
    ws = torch.full((csa.csa_sparse_mla_paged_workspace_size(6, 64),), 255, dtype=torch.uint8,
                    device="cuda")  # whatever the workspace holds
    for _ in range(3):
        b, lb = c.call(workspace=ws)
        assert torch.equal(a, b) and torch.equal(la, lb)


def test_padding_slots():
    """Padding slots: out 0, lse -inf, whatever their sequence number; the
    others as without them."""
    c = Case([500, 80, 900], 16, "list", seq=[0, 5, 1, -9, 2, 0], pos=[499, -1, 79, -3, 899, 10],
             seed=5)
    out, lse = c.check()
    assert out[1].abs().max() == 0 and out[3].abs().max() == 0
    assert torch.isinf(lse[[1, 3]]).all()
    only = Case([500], 4, "window", seq=[0, 0], pos=[-1, -1], seed=6)
    out, lse = only.check()
    assert out.abs().max() == 0


def test_lists():
    """Entries out of order, repeated, negative, not visible, absent in the
    middle; rows with no entry left."""
    c = Case([400, 400, 10, 3], 8, "list", topk=24, seed=7)
    rng = np.random.default_rng(8)
    for t in range(4):
        nv = (int(c.pos[t]) + 1) // 4
        row = rng.integers(-3, nv + 5, 24)
        row[rng.integers(0, 24, 4)] = 2 ** 31 - 1
        c.idx[t] = row
    c.check()
    c.idx[:] = -1
    c.check()
    c.idx[:, -1] = 0  # a single entry at the end
    c.check()


def test_absent_pages():
    """Needed pages that are absent are left out and reported; a token that
    loses every row keeps only its sink."""
    c = Case([300, 300], 8, "all", page=16, ratio=4, seed=9)
    c.ori_table[0, 18] = -1
    c.cmp_table[1, 2] = 10 ** 6  # outside the pool
    keep = c.cmp_table.copy()
    keep[1, 2] = -1
    c.cmp_table, bad = keep, c.cmp_table
    want = c.ref()
    c.cmp_table = bad
    out, lse = c.call()
    assert csa.csa_device_error()[0] == 6
    R.check(out, want[0], want[2])
    R.check(lse, want[1], want[3])
    lone = Case([40], 8, "window", page=64, seed=10)
    lone.ori_table[:] = -1
    out, lse = lone.call()
    assert csa.csa_device_error()[0] == 6
    assert out.abs().max() == 0
    assert (lse[0] - lone.sinks).abs().max() <= 8 * R.U32 * (lone.sinks.abs().max() + 1)
    lone.sinks = None
    out, lse = lone.call()
    assert csa.csa_device_error()[0] == 6
    assert out.abs().max() == 0 and (lse == -math.inf).all()
    # a sequence outside the batch: padding, reported
    lone.seq[:] = 1
    out, lse = lone.call()
    assert csa.csa_device_error()[0] == 6
    assert out.abs().max() == 0 and (lse == -math.inf).all()


def test_nan_in_unseen_slots():
    """Rows no token sees (past a sequence's end in its last page, other
    pages) may hold anything."""
    for mode in ("list", "all", "window"):
        c = Case([70, 300, 9], 16, mode, page=64, cmp_page=16, topk=8, seed=11)
        out, lse = c.check()
        seen = np.zeros(c.ori.shape[:2], bool)
        for b, p in zip(c.seq, c.pos):
            for r in range(max(0, p - c.win_left), p + 1):
                seen[R.slot(c.ori_table, 64, b, r)] = True
        c.ori[torch.from_numpy(~seen).cuda()] = math.nan
        if c.cmp is not None:
            seen = np.zeros(c.cmp.shape[:2], bool)
            for t, (b, p) in enumerate(zip(c.seq, c.pos)):
                nv = (p + 1) // 4
                for r in (range(nv) if c.idx is None else [j for j in c.idx[t] if 0 <= j < nv]):
                    seen[R.slot(c.cmp_table, 16, b, r)] = True
            c.cmp[torch.from_numpy(~seen).cuda()] = math.nan
        o2, l2 = c.call()
        assert torch.equal(out, o2) and torch.equal(lse, l2)


def test_beyond_32_bit_offsets():
    """A compressed pool of more than 2^31 elements, pages at its end."""
    pages, page = 65600, 64
    c = Case([2000], 64, "list", topk=300, page=page, seed=12)
    small, table = c.cmp, c.cmp_table
    big = torch.empty((pages, page, 512), dtype=torch.bfloat16, device="cuda")
    n = small.shape[0]
    big[pages - n:] = small
    big[:n] = math.nan
    want = c.call()
    c.cmp, c.cmp_table = big, np.where(table >= 0, table + pages - n, -1)
    got = c.call()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_graph_and_streams():
    """Captured and replayed with new inputs; two calls at once on two streams
    with workspaces of their own."""
    c = Case([5000, 77, 900], 64, "list", topk=512, seed=13)
    d = Case([3000, 770, 90], 64, "list", topk=512, seed=14)
    want_c, want_d = c.call(), d.call()
    args = [c.q.clone(), i32(c.idx), i32(c.ori_table), i32(c.cmp_table), i32(c.seq), i32(c.pos)]
    out, lse = torch.empty_like(c.q), torch.empty((3, 64), device="cuda")
    ws = torch.empty(csa.csa_sparse_mla_paged_workspace_size(3, 64), dtype=torch.uint8, device="cuda")

    def step():
        csa.csa_sparse_mla_paged(args[0], c.ori, c.cmp, args[1], args[2], args[3], args[4], args[5],
                                 c.sinks, c.scale, c.ratio, c.win_left, return_softmax_lse=True,
                                 workspace=ws, out=out, lse=lse)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        out.zero_()
        g.replay()
        assert torch.equal(out, want_c[0]) and torch.equal(lse, want_c[1])
    args[0].copy_(-c.q)
    g.replay()
    neg = Case([5000, 77, 900], 64, "list", topk=512, seed=13)
    neg.q = -c.q
    assert torch.equal(out, neg.call()[0])
    s2 = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        with torch.cuda.stream(s):
            a = c.call(stream=s)
        with torch.cuda.stream(s2):
            b = d.call(stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(a[0], want_c[0]) and torch.equal(b[0], want_d[0])


def test_refusals():
    c = Case([100], 4, "list", topk=8, seed=15)

    def code(**kw):
        a = dict(q=c.q, ori=c.ori, cmp=c.cmp, idx=i32(c.idx), ot=i32(c.ori_table),
                 ct=i32(c.cmp_table), seq=i32(c.seq), pos=i32(c.pos), sinks=c.sinks, r=4, wl=127, wr=0,
                 ws=None)
        a.update(kw)
        with pytest.raises(csa.CsaError) as e:
            csa.csa_sparse_mla_paged(a["q"], a["ori"], a["cmp"], a["idx"], a["ot"], a["ct"], a["seq"],
                                     a["pos"], a["sinks"], 0.04, a["r"], a["wl"], a["wr"],
                                     workspace=a["ws"])
        return e.value.code

    assert code(r=1) == 3
    assert code(wr=1) == 3
    assert code(wl=-1) == 2
    assert code(ws=torch.empty(1024, dtype=torch.uint8, device="cuda")) == 4
    many = torch.zeros((2, 4, 512), dtype=torch.bfloat16, device="cuda")
    assert code(q=many, seq=None, pos=i32([1, 1]), cmp=None, idx=None) == 2
    wide = torch.zeros((1, 65, 512), dtype=torch.bfloat16, device="cuda")
    assert code(q=wide, sinks=None) == 3
    with pytest.raises(ValueError):
        code(ct=i32(np.zeros((2, 3))))
    with pytest.raises(ValueError):
        code(seq=i32([0, 0]))
    with pytest.raises(ValueError):
        code(sinks=torch.zeros(3, device="cuda"))
    with pytest.raises(TypeError):
        code(pos=c.q)


def test_empty_call():
    c = Case([100], 4, "window", seed=16)
    out, lse = csa.csa_sparse_mla_paged(c.q[:0], c.ori, None, None, i32(c.ori_table), None, None,
                                        i32([]), c.sinks, 0.04, 4, 127, return_softmax_lse=True)
    assert out.shape == (0, 4, 512) and lse.shape == (0, 4)


@pytest.mark.parametrize("mode", ["list", "all"])
def test_token_by_token_against_packed_oracle(mode):
    """Two sequences continued token by token: rows appended, the indexer's
    choice attended, equal to the packed forward's oracle at every position."""
    ratio, topk, win_left, H, Hi, Di = 4, 8, 15, 4, 4, 64
    lens, prompt, page = [75, 41], [61, 2], 16
    gen = torch.Generator().manual_seed(21)
    kv = [torch.randn((n, 512), generator=gen).bfloat16() for n in lens]
    cmp = [torch.randn((n // ratio, 512), generator=gen).bfloat16() for n in lens]
    ki = [R.grid(gen, (n // ratio, Di), 0.5, torch.bfloat16) for n in lens]
    q = [torch.randn((n, H, 512), generator=gen).bfloat16() for n in lens]
    qi = [R.grid(gen, (n, Hi, Di), 0.5, torch.bfloat16) for n in lens]
    w = [R.grid(gen, (n, Hi), 0.125, torch.float32) for n in lens]
    sinks = torch.randn((H,), generator=gen)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    cuc = oracle.compress_cu_seqlens(cu, ratio)
    idx, *_ = oracle.indexer_topk(torch.cat(qi), torch.cat(ki), torch.cat(w), int(cu[-1]), cu, cuc,
                                  ratio, topk)
    rows = idx if mode == "list" else None
    want, wlse = oracle.sparse_mla_fwd(torch.cat(q), torch.cat(kv), torch.cat(cmp), rows, cu, cuc,
                                       int(cu[-1]), sinks, R.inv_sqrt(512), ratio, win_left)
    ot, no = R.pool_rows(lens, page, seed=1)
    ct, nc = R.pool_rows([n // ratio for n in lens], page, seed=2)
    ori = torch.zeros((no, page, 512), dtype=torch.bfloat16, device="cuda")
    cmpc = torch.zeros((nc, page, 512), dtype=torch.bfloat16, device="cuda")
    kic = torch.zeros((nc, page, Di), dtype=torch.bfloat16, device="cuda")
    ot, ct = i32(ot), i32(ct)

    def append(cache, table, parts, b, lo, hi):
        if hi > lo:
            csa.csa_cache_append(parts[b][lo:hi].cuda(), i32([b] * (hi - lo)), i32(range(lo, hi)),
                                 table, cache)

    for b in range(2):
        append(ori, ot, kv, b, 0, prompt[b])
        append(cmpc, ct, cmp, b, 0, prompt[b] // ratio)
        append(kic, ct, ki, b, 0, prompt[b] // ratio)
    for step in range(14):
        pos = [p + step if p + step < n else -1 for p, n in zip(prompt, lens)]
        for b, p in enumerate(pos):
            if p >= 0:
                append(ori, ot, kv, b, p, p + 1)
                if (p + 1) % ratio == 0:
                    append(cmpc, ct, cmp, b, p // ratio, p // ratio + 1)
                    append(kic, ct, ki, b, p // ratio, p // ratio + 1)
        take = lambda parts: torch.stack([x[max(p, 0)] for x, p in zip(parts, pos)]).cuda()
        sel = None
        if mode == "list":
            sel, _ = csa.csa_indexer_topk_paged(take(qi), kic, take(w), ct, None, i32(pos), ratio, topk)
            for b, p in enumerate(pos):
                if p >= 0:
                    r = idx[cu[b] + p]
                    assert np.array_equal(sel[b].cpu().numpy(), np.where(r >= 0, r - cuc[b], -1))
        out, lse = csa.csa_sparse_mla_paged(take(q), ori, cmpc, sel, ot, ct, None, i32(pos),
                                            sinks.cuda(), R.inv_sqrt(512), ratio, win_left,
                                            return_softmax_lse=True)
        for b, p in enumerate(pos):
            if p >= 0:
                # weights round to bf16 once (2^-8 of sum p |v|, |v| < 4.8 here) and out once
                d = np.abs(R.f64(out[b]) - want[cu[b] + p])
                assert d.max() <= 2e-2 and d.mean() <= 2e-3
                assert np.abs(R.f64(lse[b]) - wlse[cu[b] + p]).max() <= 1e-3
