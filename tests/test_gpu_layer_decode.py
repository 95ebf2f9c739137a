"""GPU tests of whole decode steps: a layer continued token by token, with the
rotation, against the 64-bit forms; the step captured into a CUDA graph; the
paged kernels' timeout path; calls across a device reset; many tokens, long
runs and shared pages."""

import os
import subprocess
import sys
import textwrap

import numpy as np
import pytest
import torch

import sparse_attention_csa_gb300 as csa
from sparse_attention_csa_gb300 import build as csa_build
from sparse_attention_csa_gb300.pipeline import PagedLayerCache, csa_layer_decode
from tests import _paged_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean_error_word():
    yield
    torch.cuda.synchronize()
    assert csa.csa_device_error() == (0, 0)


def i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


def freqs(n, theta=10000.0):
    return theta ** (-2.0 * np.arange(n // 2) / n)


class Layer:
    """Sequences with a cached prefix and room for more; compressed rows cached
    to the end (a token only sees those that are complete)."""

    def __init__(self, lens, H, Hi=8, Di=64, ratio=4, page=32, seed=0):
        gen = torch.Generator().manual_seed(seed)
        self.lens, self.ratio, self.page, self.H = lens, ratio, page, H
        self.ori_t, no = R.pool_rows(lens, page, seed=seed)
        self.cmp_t, nc = R.pool_rows([n // ratio for n in lens], page, seed=seed + 1)
        self.cache = PagedLayerCache(
            ori=torch.randn((no, page, 512), generator=gen).bfloat16().cuda(), ori_pages=i32(self.ori_t),
            cmp=torch.randn((nc, page, 512), generator=gen).bfloat16().cuda(), cmp_pages=i32(self.cmp_t),
            k_idx=R.grid(gen, (nc, page, Di), 0.5, torch.bfloat16).cuda())
        self.sinks = torch.randn((H,), generator=gen).cuda()
        self.gen, self.Hi, self.Di = gen, Hi, Di

    def tokens(self, T):
        g = self.gen
        return dict(q=torch.randn((T, self.H, 512), generator=g).bfloat16().cuda(),
                    kv=torch.randn((T, 512), generator=g).bfloat16().cuda(),
                    q_idx=R.grid(g, (T, self.Hi, self.Di), 0.5, torch.bfloat16).cuda(),
                    w=R.grid(g, (T, self.Hi), 0.125, torch.float32).cuda())


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("indexer", [True, False])
def test_steps_with_rotation(layout, indexer):
    """Three steps of two drafted tokens each (one slot padding): appended rows,
    chosen rows, attention and the output turned back."""
    lens, topk, win_left, n = [300, 90, 41], 20, 31, 64
    L = Layer(lens, H=6)
    f = freqs(n)
    inv = torch.from_numpy(f).cuda()
    half = layout == "half"
    for step in range(3):
        seq = [0, 0, 1, 1, 2, 2]
        pos = [200 + 2 * step, 201 + 2 * step, 60 + 2 * step, 61 + 2 * step, 30 + step, -1]
        t = L.tokens(6)
        before = R.f64(L.cache.ori)
        res = csa_layer_decode(t["q"], t["kv"], L.cache, i32(seq), i32(pos), L.sinks, R.inv_sqrt(512),
                               L.ratio, win_left, inv_freq=inv, rope_layout=layout, turn_back=True,
                               q_idx=t["q_idx"] if indexer else None, w=t["w"], topk=topk,
                               return_softmax_lse=True)
        # the cache now holds the rotated rows, each rounded once
        want, mag = R.rope(R.f64(t["kv"])[:, None], pos, f, 448, half)
        for b, p, row, m in zip(seq, pos, want[:, 0], mag[:, 0]):
            if p >= 0:
                pg, r = R.slot(L.ori_t, L.page, b, p)
                R.check(L.cache.ori[pg, r], row, R.rope_tol(row, m, True), "row")
                before[pg, r] = R.f64(L.cache.ori[pg, r])
        assert np.array_equal(R.f64(L.cache.ori), before)
        idx = None
        if indexer:
            idx, _ = R.indexer(t["q_idx"], L.cache.k_idx, t["w"], L.cmp_t, seq, pos, L.ratio, topk)
            assert np.array_equal(res.topk_idx.cpu().numpy(), idx)
        # the attention's inputs as the kernel has them: q rounded after its turn
        q = csa.csa_rope(t["q"], i32(pos), inv, layout=layout)
        out, lse, tol, ltol = R.attention(q, L.cache.ori, L.cache.cmp, idx, L.ori_t, L.cmp_t, seq, pos,
                                          L.sinks, R.inv_sqrt(512), L.ratio, win_left)
        R.check(res.lse, lse, ltol, "lse")
        # the output is rounded, turned back, and its rotary dims rounded again
        back, mag = R.rope(out, pos, f, 448, half, inverse=True)
        both = tol.copy()
        nn = 2 * len(f)
        part = tol[..., 448:448 + nn]
        pair = part + (np.concatenate([part[..., nn // 2:], part[..., :nn // 2]], -1) if half else
                       part.reshape(*part.shape[:-1], nn // 2, 2)[..., ::-1].reshape(part.shape))
        both[..., 448:448 + nn] = pair
        extra = R.rope_tol(back, mag, True)
        extra[..., :448] = 0
        R.check(res.out, back, (both + extra) * (1 + R.U16), "out")


def test_step_in_a_graph():
    """The whole step captured once and replayed for a run of tokens, the
    positions advanced on the device: equal to eager calls, bit by bit."""
    lens, topk = [200, 333], 16
    inv = torch.from_numpy(freqs(64)).cuda()
    A, B = Layer(lens, H=8, seed=3), Layer(lens, H=8, seed=3)
    toks = [A.tokens(2) for _ in range(4)]
    seq, start = i32([0, 1]), i32([150, 300])
    kw = dict(inv_freq=inv, turn_back=True, topk=topk, return_softmax_lse=True)

    def eager(L, t, pos):
        return csa_layer_decode(t["q"], t["kv"], L.cache, seq, pos, L.sinks, 0.04, L.ratio, 63,
                                q_idx=t["q_idx"], w=t["w"], **kw)

    want = [eager(A, t, start + k) for k, t in enumerate(toks)]
    buf = {k: v.clone() for k, v in toks[0].items()}
    pos = start.clone()
    ws = (torch.empty(csa.csa_indexer_topk_paged_workspace_size(
        2, B.cmp_t.shape[1] * B.page, B.Hi, B.Di, topk), dtype=torch.uint8, device="cuda"),
        torch.empty(csa.csa_sparse_mla_paged_workspace_size(2, 8), dtype=torch.uint8, device="cuda"))

    def step():
        r = csa_layer_decode(buf["q"], buf["kv"], B.cache, seq, pos, B.sinks, 0.04, B.ratio, 63,
                             q_idx=buf["q_idx"], w=buf["w"], indexer_workspace=ws[0],
                             attention_workspace=ws[1], **kw)
        pos.add_(1)
        return r

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    pos.copy_(start)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        res = step()
    pos.copy_(start)
    B.cache.ori.copy_(Layer(lens, H=8, seed=3).cache.ori)
    for k, t in enumerate(toks):
        for name in buf:
            buf[name].copy_(t[name])
        g.replay()
        assert torch.equal(res.topk_idx, want[k].topk_idx)
        assert torch.equal(res.out, want[k].out) and torch.equal(res.lse, want[k].lse)
    assert torch.equal(A.cache.ori, B.cache.ori)


@pytest.mark.parametrize("T", [400, 12000])
def test_many_short_tokens(T):
    """More tokens than a scan's threads, more than 64 in a CTA's run, padding
    among them: every output is its own token's."""
    rng = np.random.default_rng(T)
    lens = [40, 7, 64, 100]
    table, total = R.pool_rows(lens, 16)
    gen = torch.Generator().manual_seed(T)
    ori = torch.randn((total, 16, 512), generator=gen).bfloat16().cuda()
    seq = rng.integers(0, 4, T)
    pos = np.array([rng.integers(-2, lens[b]) for b in seq])
    q1 = torch.randn((8, 3, 512), generator=gen).bfloat16()
    pick = rng.integers(0, 8, T)
    q = q1[torch.from_numpy(pick)].cuda()
    out, lse = csa.csa_sparse_mla_paged(q, ori, None, None, i32(table), None, i32(seq), i32(pos), None,
                                        0.05, 1, 50, return_softmax_lse=True)
    # each distinct (sequence, position, query) once through the 64-bit form
    keys = {}
    for t in range(T):
        keys.setdefault((seq[t], max(pos[t], -1), pick[t]), []).append(t)
    some = list(keys)[:300]
    want, wlse, tol, ltol = R.attention(torch.stack([q1[k[2]] for k in some]), ori, None, None, table, None,
                                        [k[0] for k in some], [k[1] for k in some], None, 0.05, 1, 50)
    for i, k in enumerate(some):
        ts = torch.tensor(keys[k]).cuda()
        R.check(out[ts[0]], want[i], tol[i])
        R.check(lse[ts[0]], wlse[i], ltol[i])
    for k, ts in keys.items():  # equal tokens: equal up to where their tiles were cut
        ts = torch.tensor(ts).cuda()
        d = (out[ts].float() - out[ts[0]].float()).abs().amax()
        assert d <= 2 * R.U16 * 8


@pytest.mark.parametrize("short", [60, 300])
def test_one_very_long_row_among_short(short):
    """A row of 700,000 keys (its table repeats a few pages) beside many short
    ones: runs of more than 64 tokens in one CTA, a token over most CTAs."""
    page, uniq, reps = 64, 40, 273
    gen = torch.Generator().manual_seed(5)
    ori = torch.randn((uniq + 2, page, 512), generator=gen).bfloat16().cuda()
    table = np.full((2, uniq * reps), -1, np.int32)
    table[0] = np.tile(np.arange(uniq), reps)
    table[1, 0] = uniq
    rows = uniq * reps * page
    T = short + 1
    seq = np.array([1] * short + [0])
    pos = np.array([i % page for i in range(short)] + [rows - 1])
    q = torch.randn((T, 2, 512), generator=gen).bfloat16().cuda()
    out, lse = csa.csa_sparse_mla_paged(q, ori, None, None, i32(table), None, i32(seq), i32(pos), None,
                                        R.inv_sqrt(512), 1, rows - 1, return_softmax_lse=True)
    want, wlse, tol, ltol = R.attention(q[:short], ori, None, None, table, None, seq[:short],
                                        pos[:short], None, R.inv_sqrt(512), 1, rows - 1)
    R.check(out[:short], want, tol)
    R.check(lse[:short], wlse, ltol)
    # every distinct row counts `reps` times
    keys = R.f64(ori[:uniq]).reshape(-1, 512)
    logit = R.inv_sqrt(512) * R.f64(q[-1]) @ keys.T
    m = logit.max(1, keepdims=True)
    e = np.exp(logit - m)
    prob = e / e.sum(1, keepdims=True)
    spread = prob @ np.abs(keys)
    # rounded weights (2^-8), 11,000 tiles' fp32 sums (each rounds by 2^-24) and
    # the logits' own error (512 * 2^-24 * 0.044 sum |q||k| < 1e-3, twice)
    bound = (R.U16 + 11000 * R.U32 + 2e-3) * spread + R.U16 * np.abs(prob @ keys)
    R.check(out[-1], prob @ keys, bound)
    R.check(lse[-1], m[:, 0] + np.log(reps * e.sum(1)), 2e-3)


def test_indexer_streams_and_shared_pages():
    """Two calls at once on two streams with workspaces of their own; sequences
    that share pages."""
    gen = torch.Generator().manual_seed(6)
    table, total = R.pool_rows([9000], 64)
    table = np.repeat(table, 3, 0)  # three sequences, one set of rows
    cache = R.grid(gen, (total, 64, 128), 0.5, torch.bfloat16).cuda()
    q = R.grid(gen, (3, 64, 128), 0.5, torch.bfloat16).cuda()
    w = R.grid(gen, (3, 64), 0.125, torch.float32).cuda()
    pos = [35999, 20000, 4095]
    want, _ = R.indexer(q, cache, w, table, [0, 1, 2], pos, 4, 512)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for s in (s1, s2):
            with torch.cuda.stream(s):
                got.append(csa.csa_indexer_topk_paged(q, cache, w, i32(table), None, i32(pos), 4, 512)[0])
    torch.cuda.synchronize()
    for g in got:
        assert np.array_equal(g.cpu().numpy(), want)


def test_timeout_path():
    """A wait limit of a microsecond makes the paged kernels' waits give up:
    recorded, the launch ends, and the next calls are right."""
    L = Layer([20000, 500], H=64, Hi=64, Di=128, seed=7)
    t = L.tokens(2)
    args = (t["q"], t["kv"], L.cache, None, i32([19999, 400]), L.sinks, 0.04, L.ratio, 127)
    kw = dict(q_idx=t["q_idx"], w=t["w"], topk=512)
    want = csa_layer_decode(*args, **kw)
    torch.cuda.synchronize()
    csa.csa_set_wait_limit_ns(1)
    try:
        csa.csa_sparse_mla_paged(t["q"], L.cache.ori, L.cache.cmp, None, L.cache.ori_pages,
                                 L.cache.cmp_pages, None, i32([19999, 400]), L.sinks, 0.04, 4, 127)
        assert csa.csa_device_error()[0] == 7
        csa.csa_indexer_topk_paged(t["q_idx"], L.cache.k_idx, t["w"], L.cache.cmp_pages, None,
                                   i32([19999, 400]), 4, 512)
        assert csa.csa_device_error()[0] == 7
    finally:
        csa.csa_set_wait_limit_ns(0)
    again = csa_layer_decode(*args, **kw)
    assert torch.equal(again.topk_idx, want.topk_idx) and torch.equal(again.out, want.out)


RESET = textwrap.dedent('''
    import ctypes as C, sys
    import numpy as np
    lib = C.CDLL(sys.argv[1])
    rt = C.CDLL("libcudart.so.13")
    vp, i32 = C.c_void_p, C.c_int32
    rt.cudaMalloc.argtypes = [C.POINTER(vp), C.c_size_t]
    rt.cudaMemcpy.argtypes = [vp, vp, C.c_size_t, C.c_int]
    lib.csa_sparse_mla_paged_workspace_size.restype = C.c_size_t
    lib.csa_sparse_mla_paged.argtypes = [vp] * 8 + [i32] * 11 + [vp, C.c_float, i32, i32, i32, vp, vp, i32, vp,
                                                                 C.c_size_t, vp]
    rng = np.random.default_rng(0)
    q = (rng.standard_normal((1, 4, 512)).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    kv = (rng.standard_normal((2, 64, 512)).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    pages, pos = np.array([[1, 0]], np.int32), np.array([100], np.int32)
    for round_ in range(2):
        def dev(a):
            p = vp()
            assert rt.cudaMalloc(C.byref(p), a.nbytes) == 0
            assert rt.cudaMemcpy(p, a.ctypes.data, a.nbytes, 1) == 0
            return p
        size = lib.csa_sparse_mla_paged_workspace_size(1, 4)
        ws, out = dev(np.zeros(size, np.uint8)), dev(np.zeros_like(q))
        rc = lib.csa_sparse_mla_paged(dev(q), dev(kv), None, None, dev(pages), None, None, dev(pos), 1, 1, 4,
                                      512, 2, 64, 2, 0, 0, 0, 0, None, 0.05, 1, 127, 0, out, None, 0, ws, size,
                                      None)
        assert rc == 0, rc
        word = i32(-1)
        assert lib.csa_device_error(None, C.byref(word)) == 0 and word.value == 0
        got = np.empty_like(q)
        assert rt.cudaMemcpy(got.ctypes.data, out, got.nbytes, 2) == 0
        print(got.astype(np.uint32).sum(), int(got[0, 3, 511]), flush=True)
        if round_ == 0:
            assert rt.cudaDeviceReset() == 0
''')


def test_paged_calls_after_device_reset():
    res = subprocess.run([sys.executable, "-c", RESET, csa_build.build()], capture_output=True, text=True,
                         timeout=300, env=dict(os.environ))
    assert res.returncode == 0, res.stderr[-2000:]
    a, b = res.stdout.strip().splitlines()
    assert a == b and a.split()[0] != "0"
