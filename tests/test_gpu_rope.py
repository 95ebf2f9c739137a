"""GPU tests of the rotation: against the 64-bit formula over types, layouts,
odd sizes, strides and far positions; its transpose; its refusals."""

import math

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


def freqs(n, theta=10000.0):
    return theta ** (-2.0 * np.arange(n // 2) / n)


def make(T, H, D, dtype, seed=0, stride=None):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn((T, H, D), generator=gen).to(dtype).cuda()
    if stride:
        wide = torch.randn((T, stride), generator=gen).to(dtype).cuda()
        view = wide[:, stride - H * D:].view(T, H, D)
        view.copy_(x)
        return view
    return x


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("T,H,D,n,off", [
    (1, 1, 512, 64, 448), (1, 64, 512, 64, 448), (3, 5, 512, 64, 0), (37, 64, 128, 64, 64),
    (700, 1, 512, 64, 448), (129, 3, 96, 32, 32), (5, 7, 33, 6, 3), (2, 2, 2, 2, 0),
    (1000, 4, 64, 64, 0), (11, 1, 1024, 1024, 0), (9, 2, 100, 10, 90),
])
def test_formula(dtype, layout, inverse, T, H, D, n, off):
    x = make(T, H, D, dtype, seed=T + D)
    pos = torch.from_numpy(np.random.default_rng(T).integers(0, 1 << 20, T).astype(np.int32)).cuda()
    f = freqs(n)
    y = csa.csa_rope(x, pos, torch.from_numpy(f).cuda(), rope_offset=off, layout=layout,
                     inverse=inverse)
    want, mag = R.rope(R.f64(x), pos.cpu().numpy(), f, off, layout == "half", 1.0, inverse)
    R.check(y, want, R.rope_tol(want, mag, dtype == torch.bfloat16))
    rest = np.ones(D, bool)
    rest[off:off + n] = False
    assert torch.equal(y[..., torch.from_numpy(rest)], x[..., torch.from_numpy(rest)])


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("stride", [None, 3 * 128 + 8, 3 * 128 + 1])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_in_place_and_strides(layout, stride, dtype):
    """In place only the rotary dims change; rows of a wider matrix (aligned or
    not) give what contiguous rows give, and the columns beside them stay."""
    x = make(50, 3, 128, dtype, seed=3, stride=stride)
    pos = torch.arange(100, 150, dtype=torch.int32).cuda()
    f = torch.from_numpy(freqs(64)).cuda()
    want = csa.csa_rope(x.contiguous(), pos, f, rope_offset=32, layout=layout, mscale=1.25)
    base = x._base.clone() if stride else None
    got = csa.csa_rope(x, pos, f, rope_offset=32, layout=layout, mscale=1.25, out=x)
    assert got.data_ptr() == x.data_ptr() and torch.equal(got, want)
    if stride:
        assert torch.equal(x._base[:, :stride - 384], base[:, :stride - 384])


def test_far_positions_and_pos_stride():
    pos = torch.tensor([0, 1, -1, -77, 2 ** 31 - 1, -2 ** 31, 1234567], dtype=torch.int32).cuda()
    x = make(7, 2, 64, torch.float32, seed=5)
    f = freqs(64)
    y = csa.csa_rope(x, pos, torch.from_numpy(f).cuda())
    want, mag = R.rope(R.f64(x), pos.cpu().numpy(), f, 0, False)
    # past 2^21 positions the 64-bit product itself rounds: p f 2^-52 radians
    far = np.abs(pos.cpu().numpy().astype(np.float64))[:, None, None] * 2.0 ** -50
    R.check(y, want, R.rope_tol(want, mag, False) + far * mag)
    y4 = csa.csa_rope(x, torch.arange(7, dtype=torch.int32).cuda(), torch.from_numpy(f).cuda(),
                      pos_stride=128)
    y1 = csa.csa_rope(x, 128 * torch.arange(7, dtype=torch.int32).cuda(), torch.from_numpy(f).cuda())
    assert torch.equal(y4, y1)


def test_packed_positions():
    """cu_seqlens: a token's position is its place in its sequence (empty
    sequences included); an uncovered token is reported."""
    lens = [5, 0, 17, 1]
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)).cuda()
    pos = torch.tensor(np.concatenate([np.arange(n) for n in lens]).astype(np.int32)).cuda()
    x = make(23, 4, 64, torch.bfloat16)
    f = torch.from_numpy(freqs(32)).cuda()
    got = csa.csa_rope(x, None, f, cu_seqlens=cu, pos_stride=4)
    assert torch.equal(got, csa.csa_rope(x, 4 * pos, f))
    csa.csa_rope(make(25, 4, 64, torch.bfloat16), None, f, cu_seqlens=cu)
    assert csa.csa_device_error()[0] == 6


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_inverse_is_the_transpose(layout):
    """<g, R x> = <R^T g, x>: the inverse is the backward (with mscale too),
    and it matches differences of the forward."""
    x, g = make(40, 8, 192, torch.float32, 1), make(40, 8, 192, torch.float32, 2)
    pos = torch.arange(40, dtype=torch.int32).cuda() * 977
    f = torch.from_numpy(freqs(128)).cuda()
    kw = dict(rope_offset=64, layout=layout, mscale=0.75)
    y = csa.csa_rope(x, pos, f, **kw)
    gx = csa.csa_rope(g, pos, f, inverse=True, **kw)
    a, b = (R.f64(g) * R.f64(y)).sum(), (R.f64(gx) * R.f64(x)).sum()
    mag = (np.abs(R.f64(g)) * np.abs(R.f64(x))).sum() * 2
    assert abs(a - b) <= 2.0 ** -20 * mag
    # d <g, y> / d x[t, h, e] by a difference (y is linear in x: any step)
    for t, h, e in [(0, 0, 64), (7, 3, 70), (39, 7, 191), (20, 1, 10)]:
        x2 = x.clone()
        x2[t, h, e] += 4.0
        d = ((R.f64(csa.csa_rope(x2, pos, f, **kw)) - R.f64(y)) * R.f64(g)).sum() / 4.0
        row = 8.0 * (np.abs(R.f64(x2[t, h])).max() + 4.0) * np.abs(R.f64(g[t, h])).max()
        assert abs(d - float(gx[t, h, e])) <= 2.0 ** -20 * row


def test_empty():
    f = torch.from_numpy(freqs(64)).cuda()
    x = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    assert csa.csa_rope(x, torch.empty(0, dtype=torch.int32, device="cuda"), f).shape == (0, 4, 64)


def test_long_grid():
    """More tokens than one block each, positions of every token its own."""
    T = 70001
    x = make(T, 1, 64, torch.float32)
    pos = torch.arange(T, dtype=torch.int32).cuda()
    f = freqs(64)
    y = csa.csa_rope(x, pos, torch.from_numpy(f).cuda())
    want, mag = R.rope(R.f64(x), np.arange(T), f, 0, False)
    R.check(y, want, R.rope_tol(want, mag, False))


@pytest.mark.parametrize("rope_dim,theta,factor,orig,fast,slow", [
    (64, 10000.0, 1.0, 0, 32, 1), (64, 10000.0, 8.0, 0, 32, 1), (64, 10000.0, 16.0, 65536, 32, 1),
    (128, 160000.0, 40.0, 4096, 32, 1), (2, 500.0, 4.0, 2048, 32, 1), (6, 1e6, 2.5, 100, 8, 8),
])
def test_freqs(rope_dim, theta, factor, orig, fast, slow):
    got = R.f64(csa.csa_rope_freqs(rope_dim, theta, factor, orig, fast, slow))
    i = np.arange(rope_dim // 2)
    f = theta ** (-2.0 * i / rope_dim)
    want = f / factor
    if orig:
        d = lambda b: rope_dim * math.log(orig / (2 * math.pi * b)) / (2 * math.log(theta))
        lo, hi = max(math.floor(d(fast)), 0), min(math.ceil(d(slow)), rope_dim - 1)
        g = np.clip((i - lo) / max(hi - lo, 1e-3), 0, 1)
        want = f / factor * g + f * (1 - g)
    np.testing.assert_allclose(got, want, rtol=2.0 ** -46)


def test_refusals():
    f = torch.from_numpy(freqs(64)).cuda()
    x = make(8, 2, 64, torch.bfloat16)
    pos = torch.arange(8, dtype=torch.int32).cuda()

    def code(fn):
        with pytest.raises(csa.CsaError) as e:
            fn()
        return e.value.code

    assert code(lambda: csa.csa_rope(x, pos, f, rope_offset=1)) == 2
    assert code(lambda: csa.csa_rope(x, pos, f, rope_offset=-2)) == 2
    assert code(lambda: csa.csa_rope(x, None, f)) == 1
    buf = torch.zeros(4096, dtype=torch.bfloat16, device="cuda")
    a, b = buf[:1024].view(8, 2, 64), buf[64:1088].view(8, 2, 64)
    assert code(lambda: csa.csa_rope(a, pos, f, out=b)) == 3  # overlapping
    wide = torch.zeros((8, 256), dtype=torch.bfloat16, device="cuda")
    left, right = wide[:, :128].view(8, 2, 64), wide[:, 128:].view(8, 2, 64)
    csa.csa_rope(left, pos, f, out=right)  # beside it, same rows: fine
    for bad in (x.half(), x.cpu()):
        with pytest.raises(TypeError):
            csa.csa_rope(bad, pos, f)
    with pytest.raises(ValueError):
        csa.csa_rope(x.transpose(0, 1), pos[:2], f)
    with pytest.raises(ValueError):
        csa.csa_rope(x, pos[:7], f)
    with pytest.raises(ValueError):
        csa.csa_rope(x, pos, f, layout="other")
    with pytest.raises(TypeError):
        csa.csa_rope(x, pos, f.float())
    with pytest.raises(TypeError):
        csa.csa_rope(x, pos, f, out=torch.empty_like(x, dtype=torch.float32))
