"""GPU tests of the mark for an evicted page in a table of window rows, whose
pages are not given back by weight: it is an absent page there, recorded as any
other, in both forms of the paged attention."""

import numpy as np
import pytest
import torch

import sparse_attention_csa_gb300 as csa
from tests import _paged_ref as R
from tests import _q4_ref as Q
from tests.test_gpu_mla_q4 import Q4Case
from tests.test_gpu_paged_mla import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean_error_word():
    yield
    torch.cuda.synchronize()
    assert csa.csa_device_error() == (0, 0)


@pytest.mark.parametrize("kind,mode", [(Case, "window"), (Case, "list"), (Q4Case, "window"), (Q4Case, "all")])
def test_recorded_and_left_out(kind, mode):
    c = kind([700, 300], 16, mode, topk=40, page=16, win_left=127, seed=3)
    c.check()
    assert csa.csa_device_error() == (0, 0)
    c.ori_table[0, 700 // 16 - 2] = Q.EVICTED
    out, lse = c.call()
    status, word = csa.csa_device_error()
    assert status == 6 and (word >> 16) & 0xFF == 12
    want, wlse, tol, ltol = c.ref()
    R.check(out, want, tol)
    R.check(lse, wlse, ltol)


@pytest.mark.parametrize("kind", [Case, Q4Case])
def test_not_recorded_where_no_token_looks(kind):
    """Behind the window, and in the compressed rows' table."""
    c = kind([2000], 8, "all", page=16, win_left=127, seed=4)
    c.ori_table[0, :100] = Q.EVICTED
    c.cmp_table[0, 3:9] = Q.EVICTED
    c.check()
    assert csa.csa_device_error() == (0, 0)


def test_one_kind_beside_the_other():
    """An evicted page of either table in the same call: one is recorded."""
    c = Q4Case([900], 8, "all", page=16, win_left=300, seed=5)
    c.cmp_table[0, 2] = Q.EVICTED
    c.check()
    assert csa.csa_device_error() == (0, 0)
    c.ori_table[0, 50] = Q.EVICTED
    out, lse = c.call()
    assert csa.csa_device_error()[0] == 6
    want, wlse, tol, ltol = c.ref()
    R.check(out, want, tol)
    assert np.isfinite(R.f64(lse)).all()
