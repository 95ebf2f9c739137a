"""GPU tests of the paged attention over 4-bit rows with numbers of tokens
beside those that one scan of their tiles holds, beside bf16 rows of the same
values. (That a scan's sum stays in 32 bits with every token at its largest is
asserted where the kernel is compiled: a run of it would take hours.)"""

import numpy as np
import pytest
import torch

import sparse_attention_csa_gb300 as csa
from tests import _paged_ref as R
from tests.test_gpu_mla_q4 import Q4Case
from tests.test_gpu_paged_mla import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean_error_word():
    yield
    torch.cuda.synchronize()
    assert csa.csa_device_error() == (0, 0)


@pytest.mark.parametrize("tokens", [383, 384, 385, 639, 640, 641, 768, 769, 1300])
def test_numbers_of_tokens(tokens):
    rng = np.random.default_rng(tokens)
    n_seq = 6
    lens = rng.integers(200, 1500, n_seq)
    seq = rng.integers(0, n_seq, tokens)
    pos = np.where(rng.random(tokens) < 0.1, -1, rng.integers(0, lens[seq]))
    c = Q4Case(lens.tolist(), 4, "all", page=32, seq=seq, pos=pos, seed=tokens)
    out, lse = c.check()
    bf, blse = Case.call(c)
    want, wlse, tol, ltol = c.ref()
    R.check(bf, want, tol)
    R.check(blse, wlse, ltol)
