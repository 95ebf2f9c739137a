"""GPU tests of waits of the attention-weight kernel that give up: under short
limits some launch does, says so, and the calls after it are right."""

import numpy as np
import pytest
import torch

import sparse_attention_csa_gb300 as csa
from tests.test_gpu_attn_mass import Mass
from tests.test_gpu_paged_timeout import sweep

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean_error_word():
    yield
    csa.csa_set_wait_limit_ns(0)
    torch.cuda.synchronize()
    assert csa.csa_device_error() == (0, 0)


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("tokens,mode", [(3, "all"), (40, "all"), (700, "all"), (40, "list")])
def test_some_launch_gives_up(tokens, mode, bits):
    rng = np.random.default_rng(tokens)
    n = 200000 if tokens == 3 else 6000
    pos = rng.integers(n // 2, n, tokens)
    m = Mass([n], 16, mode, topk=512, seq=np.zeros(tokens, int), pos=pos, seed=13, bits=bits)
    args = m.args(m.base)
    want = csa.csa_attn_mass_paged(*args)
    assert sweep(lambda: csa.csa_attn_mass_paged(*args), 14)
    assert torch.equal(csa.csa_attn_mass_paged(*args), want)
