"""GPU tests of the paged indexer over tables much wider than their rows, and
with scores that are not exact in fp32."""

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


@pytest.mark.parametrize("n", [130, 600, 3000, 20000])
@pytest.mark.parametrize("values", [False, True])
def test_indexer_table_much_wider_than_its_rows(n, values):
    """A table for 70,000 rows of sequences that hold far fewer: the same rows
    as with a table that fits."""
    gen = torch.Generator().manual_seed(n)
    table, total = R.pool_rows([n, n // 2], 64, seed=2)
    cache = R.grid(gen, (total, 64, 64), 1.0, torch.bfloat16).cuda()
    q = R.grid(gen, (3, 8, 64), 1.0, torch.bfloat16).cuda()
    w = R.grid(gen, (3, 8), 0.25, torch.float32).cuda()
    wide = np.full((2, 1094), -1, np.int32)
    wide[:, :table.shape[1]] = table
    seq, pos = i32([0, 1, 0]), i32([4 * n - 1, 2 * n - 1, 2 * n])
    tight = csa.csa_indexer_topk_paged(q, cache, w, i32(table), seq, pos, 4, 100, return_value=values)
    got = csa.csa_indexer_topk_paged(q, cache, w, i32(wide), seq, pos, 4, 100, return_value=values)
    want, wval = R.indexer(q, cache, w, table, [0, 1, 0], [4 * n - 1, 2 * n - 1, 2 * n], 4, 100)
    assert np.array_equal(got[0].cpu().numpy(), want) and torch.equal(got[0], tight[0])
    if values:
        assert np.array_equal(R.f64(got[1]), wval)


@pytest.mark.parametrize("n,H,D,topk", [(700, 64, 64, 17), (9000, 8, 128, 512), (40000, 16, 64, 1024),
                                        (70000, 64, 128, 512)])
def test_indexer_unrounded_scores(n, H, D, topk):
    """Normal inputs, two tokens: rows equal unless scores at the border are
    within the fp32 error of the sums (D products, H terms)."""
    gen = torch.Generator().manual_seed(n)
    table, total = R.pool_rows([n], 64, seed=3)
    cache = torch.randn((total, 64, D), generator=gen).bfloat16().cuda()
    q = torch.randn((2, H, D), generator=gen).bfloat16().cuda()
    w = torch.randn((2, H), generator=gen).cuda()
    pos = [4 * n - 1, 3 * n]
    idx, val = csa.csa_indexer_topk_paged(q, cache, w, i32(table), i32([0, 0]), i32(pos), 4, topk,
                                          return_value=True)
    for t, p in enumerate(pos):
        rows = (p + 1) // 4
        _, k = R.gather(cache, table, 64, 0, range(rows))
        s = np.maximum(k @ R.f64(q[t]).T, 0.0) @ R.f64(w[t])
        got = idx[t].cpu().numpy()
        tol = (D + H) * R.U32 * (np.abs(R.f64(w[t])) @ (np.abs(R.f64(q[t])) @ np.abs(k).T)).max()
        assert np.abs(R.f64(val[t]) - s[got]).max() <= tol
        kth = np.sort(s)[-topk]
        assert (s[got] >= kth - 2 * tol).all() and (np.diff(got) > 0).all()
        assert set(np.nonzero(s > kth + 2 * tol)[0]) <= set(got.tolist())
