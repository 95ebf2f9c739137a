"""GPU tests of the order of the paged calls against the work around them:
inputs written right before a call, results on other streams."""

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


class Rows:
    """Three sequences' indexer rows, and tokens that move over them."""

    def __init__(self, n, topk=32, seed=0):
        gen = torch.Generator().manual_seed(seed)
        table, total = R.pool_rows([n, n, n], 64, seed=seed)
        self.table, self.topk = i32(table), topk
        self.cache = R.grid(gen, (total, 64, 64), 0.5, torch.bfloat16).cuda()
        self.q = R.grid(gen, (3, 8, 64), 0.5, torch.bfloat16).cuda()
        self.w = R.grid(gen, (3, 8), 0.125, torch.float32).cuda()

    def call(self, seq, pos, **kw):
        return csa.csa_indexer_topk_paged(self.q, self.cache, self.w, self.table, seq, pos, 4, self.topk, **kw)


@pytest.mark.parametrize("n", [300, 12000, 40000])
def test_indexer_sees_positions_written_right_before(n):
    """Positions and sequence numbers changed by a kernel between calls, also in
    a graph: each call answers for what stands there when its turn comes."""
    c = Rows(n)
    steps = 24
    rng = np.random.default_rng(n)
    all_seq = i32(rng.integers(0, 3, (steps, 3)))
    all_pos = i32(rng.integers(-1, 4 * n, (steps, 3)))
    want = []
    for k in range(steps):
        torch.cuda.synchronize()
        want.append(c.call(all_seq[k].clone(), all_pos[k].clone(), return_value=True))
        torch.cuda.synchronize()
    seq, pos = torch.zeros_like(all_seq[0]), torch.zeros_like(all_pos[0])
    ws = torch.empty(csa.csa_indexer_topk_paged_workspace_size(3, c.table.shape[1] * 64, 8, 64, c.topk),
                     dtype=torch.uint8, device="cuda")
    outs = [(torch.empty((3, c.topk), dtype=torch.int32, device="cuda"),
             torch.empty((3, c.topk), device="cuda")) for _ in range(steps)]

    def run():
        for k in range(steps):
            seq.copy_(all_seq[k])
            pos.copy_(all_pos[k])
            c.call(seq, pos, return_value=True, workspace=ws, out=outs[k][0], out_val=outs[k][1])

    def same():
        torch.cuda.synchronize()
        return all(torch.equal(a, b) and torch.equal(x, y) for (a, x), (b, y) in zip(want, outs))

    run()
    assert same()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for a, x in outs:
        a.zero_()
        x.zero_()
    g.replay()
    assert same()


def busy_blocks(shapes_dtypes, value):
    """Frees blocks of these sizes that the current stream goes on writing for
    a while: what the allocator would hand out next to the current stream."""
    blocks = [torch.empty(s, dtype=d, device="cuda") for s, d in shapes_dtypes]
    torch.cuda._sleep(200_000_000)
    for b in blocks:
        b.fill_(value)


@pytest.mark.parametrize("raw", [False, True])
def test_results_belong_to_the_calls_stream(raw):
    """With `stream=` naming a stream that is not the current one, results that
    the call makes itself are not memory which work pending on the current
    stream still writes."""
    side = torch.cuda.Stream()
    stream = side.cuda_stream if raw else side
    gen = torch.Generator().manual_seed(3)
    c = Rows(3000)
    seq, pos = i32([0, 1, 2]), i32([11999, 5000, 700])
    x = torch.randn((64, 8, 512), generator=gen).bfloat16().cuda()
    xpos, inv = torch.arange(64, dtype=torch.int32).cuda(), csa.csa_rope_freqs(64)
    ori = torch.randn((40, 64, 512), generator=gen).bfloat16().cuda()
    table, none, late = i32(np.arange(40)[None]), torch.zeros_like(xpos), xpos + 2000
    calls = [
        (lambda **k: (csa.csa_rope(x, xpos, inv, **k),), [((64, 8, 512), torch.bfloat16)]),
        (lambda **k: (csa.csa_rope_freqs(4096, 5e5, **k),), [((2048,), torch.float64)]),
        (lambda **k: c.call(seq, pos, return_value=True, **k),
         [((3, 32), torch.int32), ((3, 32), torch.float32)]),
        (lambda **k: csa.csa_sparse_mla_paged(x, ori, None, None, table, None, none, late, None, 0.04, 1, 127,
                                              return_softmax_lse=True, **k),
         [((64, 8, 512), torch.bfloat16), ((64, 8), torch.float32)]),
    ]
    for call, made in calls:
        want = [w.clone() for w in call() if w is not None]
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        busy_blocks(made, 7)
        got = call(stream=stream)
        side.synchronize()
        with torch.cuda.stream(side):
            early = [g.clone() for g in got]
        torch.cuda.synchronize()
        for w, e, g in zip(want, early, got):
            assert torch.equal(w, e) and torch.equal(w, g)


def test_ways_to_name_a_stream_and_a_device():
    """The default stream by its handle 0, as an object, or left out; a device
    by its number."""
    want = csa.csa_rope_freqs(64)
    for stream in (0, torch.cuda.default_stream(), torch.cuda.current_stream().cuda_stream, None):
        for device in (None, 0, "cuda", torch.device("cuda:0")):
            got = csa.csa_rope_freqs(64, device=device, stream=stream)
            torch.cuda.synchronize()
            assert got.device == want.device and torch.equal(got, want)
    with pytest.raises(TypeError):
        csa.csa_rope_freqs(64, device="cpu")
    c, seq, pos = Rows(300), i32([0, 1, 2]), i32([1199, 5, 700])
    idx = [c.call(seq, pos, stream=s)[0] for s in (None, 0, torch.cuda.default_stream())]
    torch.cuda.synchronize()
    assert torch.equal(idx[0], idx[1]) and torch.equal(idx[0], idx[2])
