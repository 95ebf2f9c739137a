"""GPU tests of the rotation and the append at the largest sizes they take."""

import numpy as np
import pytest
import torch

import sparse_attention_csa_gb300 as csa
from tests import _paged_ref as R

pytestmark = pytest.mark.gpu

MOST = 2 ** 31 - 1


@pytest.fixture(autouse=True)
def clean_error_word():
    yield
    torch.cuda.synchronize()
    assert csa.csa_device_error() == (0, 0)
    torch.cuda.empty_cache()


def test_rotation_of_the_most_tokens():
    """2^31 - 1 tokens of one pair each (8.6 GB), in place: the first, the last
    and some between turned by their own positions."""
    x = torch.ones((MOST, 2), dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, MOST], dtype=torch.int32, device="cuda")
    f = torch.tensor([2.0 ** -29], dtype=torch.float64, device="cuda")
    csa.csa_rope(x, None, f, cu_seqlens=cu, out=x)
    pos = np.array([0, 1, 2 ** 29, 2 ** 30 + 12345, MOST - 200, MOST - 1])
    want, mag = R.rope(np.ones((len(pos), 1, 2)), pos, [2.0 ** -29], 0, False)
    R.check(x[torch.from_numpy(pos).cuda()], want[:, 0], R.rope_tol(want, mag, True)[:, 0])


def test_append_of_the_most_rows():
    """2^31 - 1 rows of one value each (4.3 GB), one page each."""
    rows = torch.empty((MOST, 1), dtype=torch.bfloat16, device="cuda")
    rows.view(-1).copy_(torch.arange(MOST, dtype=torch.int32, device="cuda") % 251)
    cache = torch.zeros((1, MOST, 1), dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(MOST, dtype=torch.int32, device="cuda")
    seq = torch.zeros((1,), dtype=torch.int32, device="cuda").expand(MOST).contiguous()
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    csa.csa_cache_append(rows, seq, pos, table, cache)
    assert torch.equal(cache.view(-1), rows.view(-1))
