"""GPU tests of the rotation and the append at the largest sizes they take, and
of how exact the factors of far positions are."""

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


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("inverse", [False, True])
def test_factors_are_exact_to_fp32(layout, inverse):
    """The pair (1, 0) turns into (cos, sin). sincospif is off by one unit at
    most (2^-24), the rest of the angle rounds once more (2^-25), and the bits
    of the angle that are left out, the frequency's own rounding and the 64-bit
    formula's are together below 2^-29."""
    T, n = 100000, 64
    pos = np.random.default_rng(7).integers(0, 1 << 20, T).astype(np.int32)
    f = 10000.0 ** (-2.0 * np.arange(n // 2) / n)
    x = torch.zeros((T, 1, n), device="cuda")
    first = slice(0, n // 2) if layout == "half" else slice(0, n, 2)
    second = slice(n // 2, n) if layout == "half" else slice(1, n, 2)
    x[..., first] = 1.0
    y = R.f64(csa.csa_rope(x, torch.from_numpy(pos).cuda(), torch.from_numpy(f).cuda(), layout=layout,
                           inverse=inverse))[:, 0]
    angle = pos[:, None].astype(np.float64) * f * (-1.0 if inverse else 1.0)
    bound = 2.0 ** -24 + 2.0 ** -25 + 2.0 ** -29
    assert np.abs(y[:, first] - np.cos(angle)).max() <= bound
    assert np.abs(y[:, second] - np.sin(angle)).max() <= bound
