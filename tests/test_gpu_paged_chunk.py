"""GPU tests of a chunk of a prompt over the paged caches: many new tokens of
a sequence in one call, with 64 heads and compressed rows, through the calls and
through the layer step; and the same rows through the packed forward."""

import numpy as np
import pytest
import torch

import sparse_attention_csa_gb300 as csa
from sparse_attention_csa_gb300.pipeline import csa_layer_decode
from tests import _paged_ref as R
from tests.test_gpu_layer_decode import Layer, freqs
from tests.test_gpu_paged_mla import Case, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean_error_word():
    yield
    torch.cuda.synchronize()
    assert csa.csa_device_error() == (0, 0)


@pytest.mark.parametrize("mode", ["list", "all"])
@pytest.mark.parametrize("lens,new", [([1500], 700), ([900, 333], 300)])
def test_chunk_against_formula(mode, lens, new):
    c = Case(lens, 64, mode, topk=64, ratio=4, new=new, seed=new)
    out, lse = c.call()
    some = np.linspace(0, len(c.seq) - 1, 60).astype(int)  # in the order of the call: shuffled
    idx = None if c.idx is None else c.idx[some]
    want, wlse, tol, ltol = R.attention(c.q[torch.from_numpy(some).cuda()], c.ori, c.cmp, idx, c.ori_table,
                                        c.cmp_table, c.seq[some], c.pos[some], c.sinks, c.scale, c.ratio,
                                        c.win_left)
    some = torch.from_numpy(some).cuda()
    R.check(out[some], want, tol, "out")
    R.check(lse[some], wlse, ltol, "lse")


@pytest.mark.parametrize("mode", ["list", "all"])
def test_chunk_against_the_packed_forward(mode):
    """A whole prompt in one paged call and in the packed call: each rounds its
    weights to bf16 (2^-8 of the sum of weighted magnitudes) and its output."""
    n, H, ratio, topk, win_left, page = 1030, 64, 4, 48, 127, 64
    gen = torch.Generator().manual_seed(9)
    q = torch.randn((n, H, 512), generator=gen).bfloat16().cuda()
    kv = torch.randn((n, 512), generator=gen).bfloat16().cuda()
    cmp = torch.randn((n // ratio, 512), generator=gen).bfloat16().cuda()
    sinks, scale = torch.randn((H,), generator=gen).cuda(), R.inv_sqrt(512)
    cu = i32([0, n])
    cuc = csa.csa_compress_cu_seqlens(cu, ratio)
    idx = None
    if mode == "list":
        idx = torch.full((n, topk), -1, dtype=torch.int32)
        rng = np.random.default_rng(3)
        for t in range(n):
            nv = (t + 1) // ratio
            k = min(nv, topk)
            idx[t, :k] = torch.from_numpy(np.sort(rng.choice(nv, k, replace=False)).astype(np.int32)) if k else 0
        idx = idx.cuda()
    want, wlse = csa.csa_sparse_mla_fwd(q, kv, cmp, idx, cu, cu, cuc, sinks, scale, ratio, win_left,
                                        return_softmax_lse=True)
    ot, no = R.pool_rows([n], page, seed=1)
    ct, nc = R.pool_rows([n // ratio], page, seed=2)
    ori = torch.zeros((no, page, 512), dtype=torch.bfloat16, device="cuda")
    cmpc = torch.zeros((nc, page, 512), dtype=torch.bfloat16, device="cuda")
    zero = lambda k: torch.zeros(k, dtype=torch.int32, device="cuda")
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    csa.csa_cache_append(kv, zero(n), pos, i32(ot), ori)
    csa.csa_cache_append(cmp, zero(n // ratio), pos[:n // ratio], i32(ct), cmpc)
    out, lse = csa.csa_sparse_mla_paged(q, ori, cmpc, idx, i32(ot), i32(ct), zero(n), pos, sinks, scale, ratio,
                                        win_left, return_softmax_lse=True)
    # |v| stays below 6 and the weights sum to at most 1: both sides' weights
    # 2 * 2^-8 * E|v| (E over the weights, below 6), both outputs 2 * 2^-8 |out|
    assert kv.abs().max() < 6 and cmp.abs().max() < 6
    d = (out.double() - want.double()).abs()
    assert (d <= 2 * R.U16 * 6 + 2 * R.U16 * want.double().abs()).all()
    assert d.mean() <= 2 * R.U16 * want.double().abs().mean()
    assert (lse - wlse).abs().max() <= 1e-4  # 2^-22 (|l| + 4) and 512 rounded products a side, |l| < 10


def test_chunk_through_the_layer_step():
    """Rows appended and attended in one step of 260 tokens, rotated, the
    indexer's choice; each token as in a step of its own."""
    lens, topk, win_left = [800, 500], 24, 63
    A, B = Layer(lens, H=64, seed=5), Layer(lens, H=64, seed=5)
    inv = torch.from_numpy(freqs(64)).cuda()
    t = A.tokens(260)
    seq = np.array([0] * 130 + [1] * 130)
    pos = np.concatenate([np.arange(600, 730), np.arange(300, 430)])
    kw = dict(inv_freq=inv, turn_back=True, topk=topk, return_softmax_lse=True)

    def step(L, pick):
        at = torch.from_numpy(pick).cuda()
        return csa_layer_decode(t["q"][at], t["kv"][at], L.cache, i32(seq[pick]), i32(pos[pick]), L.sinks,
                                R.inv_sqrt(512), L.ratio, win_left, q_idx=t["q_idx"][at], w=t["w"][at], **kw)

    whole = step(A, np.arange(260))
    for k in range(130):
        pick = np.array([k, 130 + k])
        one = step(B, pick)
        at = torch.from_numpy(pick).cuda()
        assert torch.equal(one.topk_idx, whole.topk_idx[at])
        # the split over CTAs differs: sums in another order, weights rounded
        # against other maxima (2^-8 of magnitudes below 6 on either side), and
        # the output rounded, turned (by at most sqrt 2) and rounded again
        d = (one.out.double() - whole.out[at].double()).abs()
        assert (d <= 2 * R.U16 * 6 * 1.5).all()
        assert (one.lse - whole.lse[at]).abs().max() <= 1e-4
    assert torch.equal(A.cache.ori, B.cache.ori)
