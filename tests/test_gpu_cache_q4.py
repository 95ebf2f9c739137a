"""Append to and read from a paged cache that holds rows in 4 bits, against the
format's definition in 64 bits: bytes have to be equal."""

import numpy as np
import pytest
import torch

import sparse_attention_csa_gb300 as csa
from tests import _paged_ref as ref
from tests import _q4_ref as q4

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


def clean():
    torch.cuda.synchronize()
    st, word = csa.csa_device_error()
    assert st == 0, hex(word)


def odd_rows(n, dtype, seed=0):
    """Rows with what a quantiser can get wrong."""
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn((n, 512), generator=gen) * torch.exp(2 * torch.randn((n, 1), generator=gen))
    if n >= 8:
        x[0] = 0.0
        x[1, :16], x[1, 16:32] = -0.0, 2.0 ** -130          # zero group, subnormal values
        # multiples of a quarter of the scale: ties. top 6 * 2^k -> scale 2^k
        x[2, :448] = torch.randint(-24, 25, (448,), generator=gen) * 0.25
        x[2, ::16] = 6.0
        x[3] *= 1e-37                                       # near the smallest exponent
        x[4] = x[4].clamp(-3, 3) * 1e38                     # near the largest
        x[5, 100], x[5, 200], x[5, 300] = float("nan"), float("inf"), -float("inf")
        x[6, 16:32] *= 2.0 ** -18                           # small groups beside large ones
        x[6, 32:48] *= 2.0 ** -14
        x[7] = 1e-4 * x[7] + 3.0
    return x.to(dtype)


def layout(lengths, page, seed=1):
    table, total = ref.pool_rows(lengths, page, seed=seed)
    seq = np.repeat(np.arange(len(lengths)), lengths)
    pos = np.concatenate([np.arange(n) for n in lengths])
    return table, total, seq, pos


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lengths,page,extra", [([9], 16, 0), ([33, 1, 70], 16, 24), ([11, 8], 7, 1),
                                                ([1], 1, 0), ([130, 70, 33, 64], 64, 512)])
def test_bytes(dtype, lengths, page, extra):
    table, total, seq, pos = layout(lengths, page)
    n = len(seq)
    wide = torch.zeros((n, 512 + extra), dtype=dtype)
    wide[:, extra:] = odd_rows(n, dtype)
    rows = wide.cuda()[:, extra:]
    cache = torch.full((total, page, 384), 0xA5, dtype=torch.uint8).cuda()
    csa.csa_cache_append_q4(rows, i32(seq), i32(pos), i32(table), cache)
    back = csa.csa_cache_read_q4(cache, i32(table), i32(seq), i32(pos))
    clean()
    want = np.full((total, page, 384), 0xA5, np.uint8)
    want[table[seq, pos // page], pos % page] = q4.pack(ref.f64(wide[:, extra:]))
    got = cache.cpu().numpy()
    if not np.array_equal(got, want):
        at = np.argwhere(got != want)
        raise AssertionError(f"{len(at)} bytes differ, first {at[0]}: {got[tuple(at[0])]:#x} for "
                             f"{want[tuple(at[0])]:#x}")
    values = q4.unpack(want[table[seq, pos // page], pos % page])
    assert np.array_equal(ref.f64(back), values, equal_nan=True)


def test_every_code_and_scale_reads_as_its_value():
    """All 16 codes under all 127 scales and several powers of two."""
    n = 28 * 5
    b = np.zeros((n, 384), np.uint8)
    for r in range(n):
        for g in range(28):
            b[r, 224 + g] = (28 * r + g) % 128
        words = np.zeros(56, np.uint32)
        for w in range(56):
            for k in range(8):
                words[w] |= np.uint32(((8 * (w % 2) + k + r) % 16) << (4 * k))
        b[r, :224] = words.astype("<u4").view(np.uint8)
        b[r, 252] = [27, 100, 127, 150, 227][r // 28]
    cache = torch.from_numpy(b).view(1, n, 384).cuda()
    out = csa.csa_cache_read_q4(cache, i32([[0]]), i32(np.zeros(n)), i32(np.arange(n)))
    clean()
    assert np.array_equal(ref.f64(out), q4.unpack(b), equal_nan=True)


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("rope_dim,offset,dtype", [(64, None, torch.float32), (32, None, torch.bfloat16),
                                                   (2, 449, torch.bfloat16), (18, 470, torch.float32),
                                                   (64, 448, torch.bfloat16)])
def test_rotation(half, rope_dim, offset, dtype):
    """Codes come from the row as it is, rotary dims as csa_cache_append leaves
    them, bit for bit, and within its bound of the 64-bit rotation."""
    n, page = 41, 16
    layout_name = "half" if half else "interleaved"
    x = odd_rows(n, dtype, seed=3)
    x[4] = x[5] = 1.0
    table, total, seq, pos = layout([n], page)
    pos_rows = np.arange(n)
    freq = 10000.0 ** (-2.0 * np.arange(rope_dim // 2) / rope_dim)
    kw = dict(inv_freq=torch.from_numpy(freq).cuda(), rope_offset=offset, layout=layout_name,
              mscale=1.25, pos_stride=1000)
    cache = torch.zeros((total, page, 384), dtype=torch.uint8).cuda()
    plain = torch.zeros((total, page, 512), dtype=torch.bfloat16).cuda()
    csa.csa_cache_append_q4(x.cuda(), i32(seq), i32(pos_rows), i32(table), cache, **kw)
    csa.csa_cache_append(x.cuda(), i32(seq), i32(pos_rows), i32(table), plain, **kw)
    got = csa.csa_cache_read_q4(cache, i32(table), i32(seq), i32(pos_rows))
    clean()
    at = (table[0][pos_rows // page], pos_rows % page)
    assert torch.equal(got[:, 448:].cpu(), plain.cpu()[at[0], at[1], 448:])
    assert np.array_equal(ref.f64(got[:, :448]), q4.unpack(q4.pack(ref.f64(x)))[:, :448])
    y, mag = ref.rope(ref.f64(x)[:, None, :], pos_rows * 1000, freq,
                      512 - rope_dim if offset is None else offset, half, mscale=1.25)
    # bf16 numbers below 2^-126 are 2^-133 apart: rounding there is off by half
    # of that whatever the value, which the bound relative to it leaves out
    tol = ref.rope_tol(y, mag, True)[:, 0, 448:] + 2.0 ** -134
    ref.check(got[:, 448:], y[:, 0, 448:], tol, "rotary dims")


def test_padding_absent_and_evicted_rows():
    page = 8
    table = np.array([[2, -1, q4.EVICTED, 0], [1, 99, 3, -1]], np.int32)
    cache = torch.full((4, page, 384), 7, dtype=torch.uint8).cuda()
    x = odd_rows(6, torch.float32, seed=5)
    seq, pos = [0, 1, 0, 1, 1, 0], [3, 0, -1, 17, -5, 25]
    csa.csa_cache_append_q4(x.cuda(), i32(seq), i32(pos), i32(table), cache)
    clean()
    want = np.full((4, page, 384), 7, np.uint8)
    packed = q4.pack(ref.f64(x))
    for r, (b, p) in enumerate(zip(seq, pos)):
        if p >= 0:
            want[table[b, p // page], p % page] = packed[r]
    assert np.array_equal(cache.cpu().numpy(), want)
    # reading an evicted page records nothing, writing to one does
    out = csa.csa_cache_read_q4(cache, i32(table), i32([0, 0, 0]), i32([3, 20, -4]))
    clean()
    assert np.array_equal(ref.f64(out)[0], q4.unpack(packed[:1])[0]) and not out[1:].any()
    for b, p in ((0, 20), (0, 9), (1, 9), (1, 32), (2, 0), (-1, 0)):
        before = cache.clone()
        csa.csa_cache_append_q4(x[:1].cuda(), i32([b]), i32([p]), i32(table), cache)
        assert csa.csa_device_error()[0] == 6, (b, p)
        assert torch.equal(cache, before)
        out = csa.csa_cache_read_q4(cache, i32(table), i32([b]), i32([p]))
        assert csa.csa_device_error()[0] == (0 if (b, p) == (0, 20) else 6), (b, p)
        assert not out.any()


def test_rows_are_sequences_without_row_seq_and_nothing_is_nothing():
    cache = torch.zeros((3, 4, 384), dtype=torch.uint8).cuda()
    table = i32([[0], [1], [2]])
    x = odd_rows(3, torch.bfloat16)
    csa.csa_cache_append_q4(x.cuda(), None, i32([0, 1, 2]), table, cache)
    out = csa.csa_cache_read_q4(cache, table, None, i32([0, 1, 2]))
    clean()
    assert np.array_equal(ref.f64(out), q4.unpack(q4.pack(ref.f64(x))))
    empty = torch.empty((0, 512), dtype=torch.bfloat16).cuda()
    csa.csa_cache_append_q4(empty, i32([]), i32([]), table, cache)
    assert csa.csa_cache_read_q4(cache, table, i32([]), i32([])).shape == (0, 512)
    clean()


def test_captured_and_replayed_on_another_stream():
    table, total, seq, pos = layout([50, 9], 16)
    n = len(seq)
    x = odd_rows(n, torch.float32, seed=9).cuda()
    cache = torch.zeros((total, 16, 384), dtype=torch.uint8).cuda()
    out = torch.empty((n, 512), dtype=torch.bfloat16).cuda()
    args = (i32(seq), i32(pos), i32(table))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        csa.csa_cache_append_q4(x, *args, cache)
        csa.csa_cache_read_q4(cache, args[2], args[0], args[1], out=out)
    for seed in (10, 11):
        x.copy_(odd_rows(n, torch.float32, seed=seed))
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(ref.f64(out), q4.unpack(q4.pack(ref.f64(x))), equal_nan=True)
    clean()


def test_offsets_beyond_32_bits():
    """Pages behind 2^32 bytes of the pool."""
    page, pages = 128, 90000                                 # 4.4 GB
    cache = torch.empty((pages, page, 384), dtype=torch.uint8, device="cuda")
    cache[-1] = 0
    table = i32([[pages - 1]])
    x = odd_rows(20, torch.float32, seed=12)
    seq, pos = i32(np.zeros(20)), i32(np.arange(20) + 100)
    csa.csa_cache_append_q4(x.cuda(), seq, pos, table, cache)
    out = csa.csa_cache_read_q4(cache, table, seq, pos)
    clean()
    assert np.array_equal(ref.f64(out), q4.unpack(q4.pack(ref.f64(x))), equal_nan=True)
    assert np.array_equal(cache[-1, 100:120].cpu().numpy(), q4.pack(ref.f64(x)))
