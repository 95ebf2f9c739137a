"""GPU tests of attention weights far below 1: a row's weight is that of the
formula to 32 bits, however small, whatever number of tokens the call has."""

import numpy as np
import pytest
import torch

import sparse_attention_csa_gb300 as csa
from tests import _paged_ref as R
from tests import _q4_ref as Q
from tests.test_gpu_attn_mass import Mass
from tests.test_gpu_mla_q4 import i32

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean_error_word():
    yield
    torch.cuda.synchronize()
    assert csa.csa_device_error() == (0, 0)


def step(T, topk):
    """Weights are rounded to multiples of this (csa.h)."""
    lg = lambda n: int(np.ceil(np.log2(max(n, 1))))  # noqa: E731
    return 2.0 ** (2 * lg(T) + lg(topk) - 119)


def bound(m, T):
    """(weights of the formula, tolerance), without a term that does not scale
    with them but half a step a weight: Q.mass's, less its 2^-40 a weight. With
    d as there, w a row's weight from a token: w (2 d + 64 * 2^-24) + step / 2;
    the two words of a row's sum, their sum and the total round by 2^-24 each."""
    c = m.c
    out = np.zeros(tuple(m.base.shape))
    err = np.zeros_like(out)
    q, lse = R.f64(c.q), R.f64(m.lse)
    s = step(T, 1 if c.idx is None else c.idx.shape[1])
    for t in range(len(c.seq)):
        if c.pos[t] < 0:
            continue
        b, nv = int(c.seq[t]), (int(c.pos[t]) + 1) // c.ratio
        want = range(nv) if c.idx is None else [int(j) for j in c.idx[t] if 0 <= j < nv]
        rows, keys = R.gather(c.cmp, c.cmp_table, c.cmp.shape[1], b, want)
        if not len(rows):
            continue
        logit = c.scale * (q[t] @ keys.T)
        l = lse[t][:, None]
        w = np.exp(logit - l)
        d = 512 * R.U32 * c.scale * (np.abs(q[t]) @ np.abs(keys).T)
        d = d + 2.0 ** -22 * (np.abs(logit) + np.abs(l) + 4.0)
        np.add.at(out[b], rows, w.sum(0))
        np.add.at(err[b], rows, (w * (2 * d + 64 * R.U32)).sum(0) + s / 2)
    return out, err + 4 * R.U32 * out


def among(m, T):
    """The case's tokens among T, the others padding."""
    c = m.c
    n = len(c.seq)
    at = np.sort(np.random.default_rng(T).choice(T, n, replace=False))
    dev = torch.from_numpy(at).cuda()
    q = torch.zeros((T,) + tuple(c.q.shape[1:]), dtype=torch.bfloat16, device="cuda")
    q[dev] = c.q
    lse = torch.zeros((T, c.q.shape[1]), device="cuda")
    lse[dev] = m.lse
    seq, pos = np.zeros(T, np.int32), np.full(T, -1, np.int32)
    seq[at], pos[at] = c.seq, c.pos
    idx = None
    if c.idx is not None:
        idx = np.full((T, c.idx.shape[1]), -1, np.int32)
        idx[at] = c.idx
    return lambda mass, **kw: csa.csa_attn_mass_paged(
        q, lse, m.rows, None if idx is None else i32(idx), i32(c.cmp_table), i32(seq), i32(pos), mass,
        c.scale, c.ratio, **kw)


# weights are 2^-down of the attention's; heads few, so that T tokens of q stay small
@pytest.mark.parametrize("mode", ["list", "all"])
@pytest.mark.parametrize("T,down", [(7, 0), (7, 20), (7, 45), (7, 62), (4096, 0), (4096, 20), (4096, 45),
                                    (65535, 0), (65535, 30), (65535, 40)])
def test_weights_of_any_size(T, down, mode):
    m = Mass([500, 1300, 60], 4, mode, topk=48, page=32, new=2, seed=T % 1000 + down)
    m.lse += down * float(np.log(2.0))
    call = among(m, T)
    got = call(None)
    want, tol = bound(m, T)
    R.check(got, want, tol, "mass")
    assert (R.f64(got) > 0).sum() == (want > 0).sum()  # none is lost
    assert (tol <= 2.0 ** -8 * want).all()            # and the bound is a relative one
    mine = torch.zeros_like(got)
    assert call(mine, out=mine) is mine and torch.equal(mine, got)
    assert torch.equal(call(None), got)


@pytest.mark.parametrize("mode", ["list", "all"])
def test_many_small_weights_add_up(mode):
    """Every token of many gives a row less than any one step of their sum's
    size would hold."""
    T = 4096
    m = Mass([40], 1, mode, topk=8, page=8, seq=np.zeros(T, int), pos=np.full(T, 39), seed=9)
    m.lse += 45 * float(np.log(2.0))
    got = m.call(None)
    want, tol = bound(m, T)
    R.check(got, want, tol, "mass")
    assert (tol <= 2.0 ** -8 * want).all() and (want > 0).any()


def test_large_and_small_weights_of_one_row():
    """One token's weight of some 1 and another's far below it, in either
    order, and a list that repeats a small one."""
    m = Mass([200], 2, "list", topk=40, page=16, seq=[0, 0], pos=[199, 199], seed=11)
    m.c.idx[:] = np.arange(40)
    m.c.idx[1, 20:] = 3
    m.lse[0] += 50 * float(np.log(2.0))
    m.lse[1] += 5 * float(np.log(2.0))
    want, tol = bound(m, 2)
    R.check(m.call(None), want, tol, "mass")
    assert (tol <= 2.0 ** -8 * want).all()
    a = m.call(None)
    for _ in range(3):
        assert torch.equal(m.call(None), a)
