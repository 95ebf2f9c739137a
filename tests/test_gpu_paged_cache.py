"""GPU tests of the paged row append and the paged indexer against their
64-bit forms: odd widths and pages, strides, padding, absent pages, ties."""

import numpy as np
import pytest
import torch

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


def freqs(n, theta=10000.0):
    return theta ** (-2.0 * np.arange(n // 2) / n)


# ------------------------------------------------------------------- append
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("width,n,off,half,page,extra", [
    (512, 64, 448, False, 64, 0), (512, 64, 448, True, 16, 512), (128, 64, 0, False, 1, 8),
    (512, 0, 0, False, 48, 0), (64, 32, 32, True, 7, 4), (33, 6, 20, False, 5, 0),
    (96, 96, 0, True, 33, 1), (1, 0, 0, False, 3, 2), (1024, 1024, 0, False, 2, 0),
])
@pytest.mark.parametrize("counts", [[1], [3, 0, 1], [40, 129, 7, 1, 65]])
def test_append(dtype, width, n, off, half, page, extra, counts):
    gen = torch.Generator().manual_seed(width + page)
    start = [5 * b for b in range(len(counts))]
    lens = [s + c for s, c in zip(start, counts)]
    table, total = R.pool_rows(lens, page, seed=page)
    seq = np.repeat(np.arange(len(counts)), counts)
    pos = np.concatenate([np.arange(s, s + c) for s, c in zip(start, counts)])
    perm = np.random.default_rng(1).permutation(len(seq))  # any order
    seq, pos = seq[perm], pos[perm]
    T = len(seq)
    wide = torch.randn((T, width + extra), generator=gen).to(dtype).cuda()
    rows = wide[:, extra:]
    cache = torch.randn((total, page, width), generator=gen).bfloat16().cuda()
    before = cache.clone()
    f = freqs(n) if n else None
    out = csa.csa_cache_append(rows, i32(seq), i32(pos), i32(table), cache,
                               inv_freq=None if f is None else torch.from_numpy(f).cuda(),
                               rope_offset=off, layout="half" if half else "interleaved",
                               pos_stride=4, mscale=1.0)
    assert out is cache
    x = R.f64(rows)[:, None]
    want, mag = R.rope(x, pos * 4, f, off, half) if n else (x, np.zeros_like(x))
    tol = R.rope_tol(want, mag, True)
    if dtype == torch.bfloat16:
        keep = np.ones(width, bool)
        keep[off:off + n] = False
        tol[..., keep] = 0.0  # copied
    mask = torch.ones((total, page), dtype=torch.bool)
    got = np.zeros((T, 1, width))
    for t in range(T):
        p, r = R.slot(table, page, seq[t], pos[t])
        got[t, 0] = R.f64(cache[p, r])
        mask[p, r] = False
    R.check(torch.from_numpy(got), want, tol)
    assert torch.equal(cache[mask.cuda()], before[mask.cuda()])  # every other slot as it was


def test_append_padding_and_absent():
    """Padding rows write nothing and report nothing; absent pages, pages
    outside the pool and sequences outside the batch are skipped and reported."""
    cache = torch.zeros((4, 8, 128), dtype=torch.bfloat16, device="cuda")
    rows = torch.ones((6, 128), dtype=torch.bfloat16, device="cuda")
    table = i32([[0, 1], [2, -1]])
    csa.csa_cache_append(rows, i32([0, 0, 1, 99, -5, 1]), i32([0, -1, 3, -1, -7, 7]), table, cache)
    assert csa.csa_device_error() == (0, 0)
    hit = cache[..., 0].float().cpu().numpy()
    assert hit.sum() == 3 and hit[0, 0] == hit[2, 3] == hit[2, 7] == 1
    for seq, pos, tab in [(1, 9, table), (0, 16, table), (2, 0, table), (-1, 0, table),
                          (0, 2 ** 31 - 1, table), (0, 0, i32([[4, 1], [2, 0]])),
                          (0, 0, i32([[-3, 1], [2, 0]]))]:
        before = cache.clone()
        csa.csa_cache_append(rows[:1], i32([seq]), i32([pos]), tab, cache)
        assert csa.csa_device_error()[0] == 6, (seq, pos)
        assert torch.equal(cache, before)
    # row t belongs to sequence t
    csa.csa_cache_append(2 * rows[:2], None, i32([1, 2]), table, cache)
    hit = cache[..., 0].float().cpu().numpy()
    assert hit[0, 1] == 2 and hit[2, 2] == 2


def test_append_beyond_32_bit_offsets():
    """A pool of more than 2^31 elements: slots at its end."""
    pages, page = 65600, 64
    cache = torch.empty((pages, page, 512), dtype=torch.bfloat16, device="cuda")
    cache[0], cache[-1] = 0.0, 0.0
    rows = torch.randn((64, 512), device="cuda").bfloat16()
    csa.csa_cache_append(rows, i32([0] * 64), i32(range(64)), i32([[pages - 1]]), cache)
    assert torch.equal(cache[-1], rows) and cache[0].float().abs().max() == 0


# ------------------------------------------------------------------ indexer
def indexer_case(lens, H, D, page, ratio, seed=0, new=1, step=0.5):
    """Values on a coarse grid: the scores are exact in fp32 (products are
    multiples of step^2 / 8; the sums stay below 2^24 of them), so rows and
    values have to be equal, ties included."""
    gen = torch.Generator().manual_seed(seed)
    vis = [n // ratio for n in lens]
    table, total = R.pool_rows(vis, page, seed=seed)
    cache = R.grid(gen, (total, page, D), step, torch.bfloat16).cuda()
    seq = np.repeat(np.arange(len(lens)), new)
    pos = np.concatenate([np.arange(n - new, n) for n in lens])
    perm = np.random.default_rng(seed).permutation(len(seq))
    seq, pos = seq[perm], pos[perm]
    T = len(seq)
    q = R.grid(gen, (T, H, D), step, torch.bfloat16).cuda()
    w = R.grid(gen, (T, H), 0.125, torch.float32).cuda()
    return q, cache, w, table, seq, pos


@pytest.mark.parametrize("values", [False, True])
@pytest.mark.parametrize("H,D", [(64, 128), (64, 64), (1, 128), (3, 64), (31, 128), (16, 64)])
@pytest.mark.parametrize("lens,page,ratio,topk,new", [
    ([1, 2, 3, 4, 5, 8], 16, 4, 3, 1), ([2600, 513, 700, 40], 64, 4, 128, 1),
    ([5000, 4999, 31], 40, 2, 512, 3), ([1029], 1, 8, 1, 2), ([4200], 128, 2, 2048, 1),
    ([900, 900], 7, 4, 17, 4),
])
def test_indexer(H, D, lens, page, ratio, topk, new, values):
    lens = [max(n, new) for n in lens]
    q, cache, w, table, seq, pos = indexer_case(lens, H, D, page, ratio, seed=H + topk, new=new)
    idx, val = csa.csa_indexer_topk_paged(q, cache, w, i32(table), i32(seq), i32(pos), ratio, topk,
                                          return_value=values)
    want, wval = R.indexer(q, cache, w, table, seq, pos, ratio, topk)
    assert np.array_equal(idx.cpu().numpy(), want)
    if values:
        assert np.array_equal(val.cpu().numpy().astype(np.float64), wval)
    else:
        assert val is None


@pytest.mark.parametrize("n,topk", [(140000, 512), (66000, 1024), (33000, 16), (40000, 5000)])
def test_indexer_long(n, topk):
    """Long rows, one to a few tokens, many equal scores (a coarse grid)."""
    q, cache, w, table, seq, pos = indexer_case([n, 90, n // 3], 16, 64, 64, 2, seed=n, step=1.0)
    idx, val = csa.csa_indexer_topk_paged(q, cache, w, i32(table), i32(seq), i32(pos), 2, topk,
                                          return_value=True)
    want, wval = R.indexer(q, cache, w, table, seq, pos, 2, topk)
    assert np.array_equal(idx.cpu().numpy(), want)
    assert np.array_equal(val.cpu().numpy().astype(np.float64), wval)


@pytest.mark.parametrize("n", [2000, 30000, 100000])
def test_indexer_all_equal(n):
    """Every score equal, of either sign or zero: the first rows win."""
    q, cache, w, table, seq, pos = indexer_case([n], 4, 64, 32, 2, seed=1)
    cache[:] = 1.0
    for s in (1.0, -1.0, 0.0):
        w[:] = s
        q[:] = 1.0
        idx, val = csa.csa_indexer_topk_paged(q, cache, w, i32(table), i32(seq), i32(pos), 2, 100,
                                              return_value=True)
        assert idx.cpu().tolist() == [list(range(100))]
        assert (val == s * 256.0).all()


def test_indexer_normal_values():
    """Unrounded normal inputs: rows equal unless scores at the border are
    within the fp32 error of the sums (64 heads x 128 products)."""
    gen = torch.Generator().manual_seed(3)
    table, total = R.pool_rows([3000], 64)
    cache = torch.randn((total, 64, 128), generator=gen).bfloat16().cuda()
    q = torch.randn((1, 64, 128), generator=gen).bfloat16().cuda()
    w = torch.randn((1, 64), generator=gen).cuda()
    pos = [11999]
    idx, val = csa.csa_indexer_topk_paged(q, cache, w, i32(table), None, i32(pos), 4, 512,
                                          return_value=True)
    all_idx, all_val = R.indexer(q, cache, w, table, [0], pos, 4, 3000)
    s = all_val[0]
    got = idx.cpu().numpy()[0]
    tol = (128 + 64) * R.U32 * (np.abs(R.f64(w[0])) @
                                (np.abs(R.f64(q[0])) @ np.abs(R.f64(cache).reshape(-1, 128)).T)).max()
    assert np.abs(val.cpu().numpy()[0] - s[got]).max() <= tol
    kth = np.sort(s)[-512]
    assert (s[got] >= kth - 2 * tol).all() and (np.diff(got) > 0).all()
    must = set(np.nonzero(s > kth + 2 * tol)[0])
    assert must <= set(got.tolist())


def test_indexer_padding_and_absent():
    q, cache, w, table, seq, pos = indexer_case([600, 600, 600], 8, 64, 16, 4, seed=9)
    seq, pos = np.array([0, 77, 2]), np.array([599, -1, 1])
    idx, val = csa.csa_indexer_topk_paged(q, cache, w, i32(table), i32(seq), i32(pos), 4, 64,
                                          return_value=True)
    want, wval = R.indexer(q, cache, w, table, seq, pos, 4, 64)
    assert np.array_equal(idx.cpu().numpy(), want)
    assert np.array_equal(val.cpu().numpy().astype(np.float64), wval)
    assert (idx[1:] == -1).all()
    assert csa.csa_device_error() == (0, 0)
    # an absent page is reported and its rows rank last
    holes = table.copy()
    holes[0, 3] = -1
    idx, _ = csa.csa_indexer_topk_paged(q, cache, w, i32(holes), i32(seq), i32(pos), 4, 64)
    assert csa.csa_device_error()[0] == 6
    got = idx[0].cpu().numpy()
    assert not ((got >= 48) & (got < 64)).any() and (np.diff(got) > 0).all()
    # positions past what the table can hold: its rows, reported
    idx, _ = csa.csa_indexer_topk_paged(q[:1], cache, w[:1], i32(table[:1]), None, i32([10 ** 6]), 4,
                                        200)
    assert csa.csa_device_error()[0] == 6
    # a sequence outside the batch: padding, reported
    idx, _ = csa.csa_indexer_topk_paged(q[:1], cache, w[:1], i32(table), i32([3]), i32([9]), 4, 2)
    assert csa.csa_device_error()[0] == 6 and (idx == -1).all()
    # no pages at all
    idx, _ = csa.csa_indexer_topk_paged(q[:1], cache[:0], w[:1], i32(np.zeros((1, 0))), None, i32([2]),
                                        4, 2)
    assert (idx == -1).all()


def test_indexer_refusals():
    q, cache, w, table, seq, pos = indexer_case([64, 64], 4, 64, 16, 4)
    args = (q, cache, w, i32(table), i32(seq), i32(pos))

    def code(*a, **k):
        with pytest.raises(csa.CsaError) as e:
            csa.csa_indexer_topk_paged(*a, **k)
        return e.value.code

    assert code(*args, 1, 8) == 3
    assert code(*args, 4, 0) == 2
    assert code(q, cache, w, i32(table[:1]), None, i32(pos), 4, 8) == 2  # two tokens, one sequence
    small = torch.empty(256, dtype=torch.uint8, device="cuda")
    assert code(*args, 4, 8, workspace=small) == 4
    with pytest.raises(ValueError):
        csa.csa_indexer_topk_paged(q, cache[..., :32], w, i32(table), i32(seq), i32(pos), 4, 8)
    with pytest.raises(ValueError):
        csa.csa_indexer_topk_paged(q, cache, w[:1], i32(table), i32(seq), i32(pos), 4, 8)
    with pytest.raises(ValueError):
        csa.csa_indexer_topk_paged(*args, 4, 8, out=torch.empty((2, 7), dtype=torch.int32,
                                                                device="cuda"))
