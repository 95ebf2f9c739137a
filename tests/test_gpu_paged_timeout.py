"""GPU tests of waits of the paged kernels that give up anywhere in their
pipelines: limits from the shortest to about a launch's length, so that some
waits of a launch (of a warp, even) end well and others do not. Every launch
ends, says whether it gave up, and the calls after it are right."""

import numpy as np
import pytest
import torch

import sparse_attention_csa_gb300 as csa
from tests import _paged_ref as R

pytestmark = pytest.mark.gpu

CSA_OK, CSA_ERR_TIMEOUT = 0, 7
LIMITS_NS = [1, 50, 200, 500, 1000, 2000, 3000, 5000, 8000, 12000, 20000]


@pytest.fixture(autouse=True)
def default_limit_again():
    yield
    csa.csa_set_wait_limit_ns(0)
    torch.cuda.synchronize()
    assert csa.csa_device_error() == (0, 0)


def i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


def sweep(call, kernel):
    """`call` under every limit a few times; True when some launch gave up."""
    torch.cuda.synchronize()
    gave_up = False
    try:
        for limit in LIMITS_NS:
            csa.csa_set_wait_limit_ns(limit)
            for _ in range(6):
                call()
                status, word = csa.csa_device_error()
                assert status in (CSA_OK, CSA_ERR_TIMEOUT)
                if status == CSA_ERR_TIMEOUT:
                    assert (word >> 24) == 2 and ((word >> 16) & 0xFF) == kernel
                    gave_up = True
    finally:
        csa.csa_set_wait_limit_ns(0)
    return gave_up


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("tokens", [3, 40, 700])
def test_indexer(tokens, dim):
    """Few long rows, several tokens in a CTA's run, more than one scan of them."""
    gen = torch.Generator().manual_seed(tokens)
    n = 20000 if tokens == 3 else 1500
    table, total = R.pool_rows([n], 64)
    cache = R.grid(gen, (total, 64, dim), 0.5, torch.bfloat16).cuda()
    q = R.grid(gen, (tokens, 32, dim), 0.5, torch.bfloat16).cuda()
    w = R.grid(gen, (tokens, 32), 0.125, torch.float32).cuda()
    pos = i32(np.random.default_rng(tokens).integers(0, 4 * n, tokens))
    args = (q, cache, w, i32(table), torch.zeros_like(pos), pos, 4, 64)
    want = csa.csa_indexer_topk_paged(*args, return_value=True)
    assert sweep(lambda: csa.csa_indexer_topk_paged(*args), 11)
    got = csa.csa_indexer_topk_paged(*args, return_value=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("tokens", [3, 40, 700])
def test_attention(tokens):
    gen = torch.Generator().manual_seed(tokens)
    n = 20000 if tokens == 3 else 1500
    table, total = R.pool_rows([n], 64)
    ori = torch.randn((total, 64, 512), generator=gen).bfloat16().cuda()
    q = torch.randn((tokens, 16, 512), generator=gen).bfloat16().cuda()
    pos = i32(np.random.default_rng(tokens).integers(0, n, tokens))
    args = (q, ori, None, None, i32(table), None, torch.zeros_like(pos), pos, None, 0.04, 1, n - 1)
    want = csa.csa_sparse_mla_paged(*args, return_softmax_lse=True)
    assert sweep(lambda: csa.csa_sparse_mla_paged(*args), 12)
    got = csa.csa_sparse_mla_paged(*args, return_softmax_lse=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
