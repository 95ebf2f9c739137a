"""GPU tests of the rotation and the paged calls beside autograd: what they
write in place, and the rotation inside a differentiable function."""

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


def test_rotation_in_place_is_seen():
    """A backward whose saved tensor was turned in place since is refused."""
    a = torch.randn((8, 2, 64), device="cuda", requires_grad=True)
    x = a * 2.0
    z = x.square().sum()  # saves x
    csa.csa_rope(x.detach(), i32(range(8)), csa.csa_rope_freqs(64), out=x.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        z.backward()


def test_everything_written_counts_as_changed():
    """Each tensor of the caller's that a call writes, and no other."""
    f, pos, seq, table = csa.csa_rope_freqs(64), i32([3, 1]), i32([0, 0]), i32([[0]])
    x = torch.randn((2, 4, 512), device="cuda").bfloat16()
    cache = torch.randn((1, 16, 512), device="cuda").bfloat16()
    keys = torch.randn((1, 16, 64), device="cuda").bfloat16()
    qi, w = torch.randn((2, 4, 64), device="cuda").bfloat16(), torch.randn((2, 4), device="cuda")
    out, lse = torch.empty_like(x), torch.empty((2, 4), device="cuda")
    idx, val = torch.empty((2, 3), dtype=torch.int32, device="cuda"), torch.empty((2, 3), device="cuda")
    everything = [f, pos, seq, table, x, cache, keys, qi, w, out, lse, idx, val]

    def changed(call):
        before = [t._version for t in everything]
        call()
        return [t for t, v in zip(everything, before) if t._version != v]

    def same(got, want):
        return len(got) == len(want) and all(any(g is t for g in got) for t in want)

    assert same(changed(lambda: csa.csa_rope(x, pos, f)), [])
    assert same(changed(lambda: csa.csa_rope(x, pos, f, out=out)), [out])
    assert same(changed(lambda: csa.csa_rope(x, pos, f, out=x)), [x])
    assert same(changed(lambda: csa.csa_rope_freqs(64, out=f)), [f])
    assert same(changed(lambda: csa.csa_cache_append(x[:, 0], seq, pos, table, cache)), [cache])
    ix = (qi, keys, w, table, seq, pos, 2, 3)
    assert same(changed(lambda: csa.csa_indexer_topk_paged(*ix)), [])
    assert same(changed(lambda: csa.csa_indexer_topk_paged(*ix, return_value=True, out=idx, out_val=val)),
                [idx, val])
    at = (x, cache, None, None, table, None, seq, pos, None, 0.04, 1, 15)
    assert same(changed(lambda: csa.csa_sparse_mla_paged(*at)), [])
    assert same(changed(lambda: csa.csa_sparse_mla_paged(*at, return_softmax_lse=True, out=out, lse=lse)),
                [out, lse])
    with torch.inference_mode():  # tensors without a version
        y = torch.randn((2, 4, 512), device="cuda").bfloat16()
        assert csa.csa_rope(y, pos, f, out=y) is y


class Turn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, pos, f):
        ctx.save_for_backward(pos, f)
        return csa.csa_rope(x, pos, f)

    @staticmethod
    def backward(ctx, g):
        pos, f = ctx.saved_tensors
        return csa.csa_rope(g.contiguous(), pos, f, inverse=True), None, None


def test_gradient_of_a_user_function():
    """The rotation and its inverse as forward and backward of a function:
    the gradient of a weighted sum against the 64-bit transpose."""
    gen = torch.Generator().manual_seed(0)
    x = torch.randn((20, 3, 64), generator=gen).cuda().requires_grad_()
    g = torch.randn((20, 3, 64), generator=gen).cuda()
    pos, f = i32(np.arange(20) * 991), csa.csa_rope_freqs(64)
    (Turn.apply(x, pos, f) * g).sum().backward()
    want, mag = R.rope(R.f64(g), pos.cpu().numpy(), R.f64(f), 0, False, inverse=True)
    R.check(x.grad, want, R.rope_tol(want, mag, False))
