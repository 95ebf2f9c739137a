"""Timed cases of the paged-serving operators: the rotation, the paged row
append, the paged lightning indexer and the paged sparse MLA attention.

``run`` computes a case in its plain form (elementary torch operations in 32
bits, 64 for angles) or, when ``own`` is true, with the library's calls.
``exact`` computes the same outputs from the definitions in 64 bits.

Shapes are those of the library's layers: 512-wide shared rows, 64 heads,
indexer 64 x 128, 512 selected rows, window 128, ratios 4 and 128.
"""

import math

import torch

own = False

_GOLD = 0.6180339887498949


def _lengths(case):
    """Context length of each sequence, new tokens included: spread over
    [lo, hi] by the golden ratio, the same for every seed."""
    lo, hi, n = case["lo"], case["hi"], case["seqs"]
    if n == 1:
        return [max(hi, case["new"])]
    return [max(case["new"], lo + int((hi - lo) * (((b + 1) * _GOLD) % 1.0))) for b in range(n)]


def listed():
    rope = {"op": "rope", "heads": 64, "dim": 512, "rope_dim": 64, "offset": 448, "half": False,
            "fp32": False, "inverse": False, "span": 1 << 20}
    append = {"op": "append", "dim": 512, "rope_dim": 64, "offset": 448, "half": False,
              "fp32": False, "page": 64, "extra": 0, "pos_stride": 1}
    indexer = {"op": "indexer", "new": 1, "heads": 64, "dim": 128, "ratio": 4, "topk": 512,
               "page": 64, "values": False}
    attn = {"op": "attention", "new": 1, "heads": 64, "window": 128, "mode": "list", "topk": 512,
            "ratio": 4, "page": 64}
    return [
        # queries of one decode step of 64 sequences, far positions
        dict(rope, name="rope_decode64", tokens=64),
        # queries of a long prompt
        dict(rope, name="rope_prefill8k", tokens=8192),
        # fp32 query gradients of the indexer, half layout, backward; odd length
        dict(rope, name="rope_grad_f32", tokens=4099, heads=64, dim=128, rope_dim=64, offset=64,
             half=True, fp32=True, inverse=True),
        # one new row for each of 128 sequences
        dict(append, name="append_decode128", seqs=128, new=1, lo=1000, hi=60000),
        # the rows of 16 prompts at once, taken out of a wider projection
        dict(append, name="append_prefill16k", seqs=16, new=1023, lo=1023, hi=9000, extra=512),
        # compressed rows as the compressor leaves them (fp32), position 4 j
        dict(append, name="append_compressed", seqs=5, new=1601, lo=1601, hi=9000, fp32=True,
             pos_stride=4, page=32),
        # one user with a 128k-token context, the scores wanted too
        dict(indexer, name="indexer_one_128k", seqs=1, lo=131072, hi=131072, values=True),
        # a full batch of ragged contexts
        dict(indexer, name="indexer_batch64", seqs=64, lo=4096, hi=65536),
        # one user: the smallest attention call
        dict(attn, name="attention_one", seqs=1, lo=131072, hi=131072),
        # a full batch, 512 selected rows each
        dict(attn, name="attention_batch64", seqs=64, lo=4096, hi=65536),
        # two drafted tokens beside the new one, odd batch, compressor-only layer
        dict(attn, name="attention_drafts_hca", seqs=27, new=3, mode="all", ratio=128, lo=2000,
             hi=131072),
        # few long ragged contexts, every compressed row attended
        dict(attn, name="attention_dense_long", seqs=6, mode="all", lo=30000, hi=262144,
             page=128),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "indexer", "attention"])
    if op == "rope":
        dim = rng.choice([64, 96, 128, 192, 512])
        rope_dim = rng.choice([d for d in (32, 64, 128) if d <= dim])
        heads = rng.choice([1, 3, 8, 16, 31, 64])
        tokens = _log_int(rng, 1, 16384)
        while tokens * heads * dim > 8192 * 64 * 512 // 2:
            tokens = max(1, tokens // 2)
        return {"op": op, "tokens": tokens, "heads": heads, "dim": dim, "rope_dim": rope_dim,
                "offset": rng.choice([0, dim - rope_dim]), "half": rng.random() < 0.5,
                "fp32": rng.random() < 0.4, "inverse": rng.random() < 0.5,
                "span": _log_int(rng, 16, 1 << 20)}
    if op == "append":
        dim = rng.choice([64, 128, 512])
        rope_dim = rng.choice([0, 32, 64])
        seqs = _log_int(rng, 1, 256)
        new = _log_int(rng, 1, max(1, 16384 // seqs))
        return {"op": op, "seqs": seqs, "new": new, "lo": new, "hi": new + _log_int(rng, 1, 8192),
                "dim": dim, "rope_dim": rope_dim, "offset": rng.choice([0, dim - rope_dim]),
                "half": rng.random() < 0.5, "fp32": rng.random() < 0.4,
                "page": rng.choice([16, 32, 48, 64, 128]), "extra": rng.choice([0, 0, 64, 520]),
                "pos_stride": rng.choice([1, 4, 128])}
    seqs = _log_int(rng, 1, 96)
    new = rng.choice([1, 1, 1, 2, 4])
    heads = rng.choice([4, 8, 16, 31, 64, 64])
    page = rng.choice([16, 40, 64, 128])
    if op == "indexer":
        ratio = rng.choice([2, 4, 8])
        hi = min(_log_int(rng, 64, 262144), 4194304 // (seqs * new))
        return {"op": op, "seqs": seqs, "new": new, "heads": heads,
                "dim": rng.choice([64, 128]), "lo": max(new, hi // rng.choice([1, 2, 16])),
                "hi": hi, "ratio": ratio, "topk": rng.choice([1, 17, 64, 256, 512, 1024]),
                "page": page, "values": False}
    mode = rng.choice(["list", "list", "all", "window"])
    ratio = rng.choice([4, 4, 128])
    most = 131072 * ratio if mode == "all" else 2097152
    hi = min(_log_int(rng, 16, 262144), max(64, most // (seqs * new)))
    return {"op": op, "seqs": seqs, "new": new, "heads": heads,
            "window": rng.choice([16, 128, 128, 300, 1024]), "mode": mode,
            "topk": rng.choice([8, 100, 512, 1024]), "ratio": ratio,
            "lo": max(new, hi // rng.choice([1, 2, 16])), "hi": hi, "page": page}


# ------------------------------------------------------------------- inputs
def _normal(gen, shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _grid(gen, shape, step, dtype):
    """Normal values rounded to multiples of `step`: low-precision activations,
    whose weighted sums are exact in 32 bits."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    return (torch.round(x / step) * step).to(dtype)


def _inv_freq(rope_dim, theta=10000.0):
    i = torch.arange(rope_dim // 2, dtype=torch.float64)
    return (theta ** (-2.0 * i / rope_dim)).cuda()


def _tables(rows, first, page, gen):
    """Page table [seqs, pages] (int32) for sequences holding `rows` rows each,
    pages before the one of row `first` released (-1), physical pages in
    random order; and the number of physical pages."""
    n = [-(-r // page) for r in rows]
    lo = [min(f // page, k) for f, k in zip(first, n)]
    used = sum(k - s for k, s in zip(n, lo))
    total = used + 3
    perm = torch.randperm(total, generator=gen, device="cuda").cpu().tolist()
    table = [[-1] * max(1, max(n, default=1)) for _ in rows]
    at = 0
    for b in range(len(rows)):
        for p in range(lo[b], n[b]):
            table[b][p] = perm[at]
            at += 1
    return torch.tensor(table, dtype=torch.int32, device="cuda"), total


def _new_tokens(case):
    lens = _lengths(case)
    seq, pos = [], []
    for b, n in enumerate(lens):
        for k in range(case["new"]):
            seq.append(b)
            pos.append(n - case["new"] + k)
    return lens, seq, pos


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    i32 = dict(dtype=torch.int32, device="cuda")
    st = {"case": dict(case)}
    if case["op"] == "rope":
        shape = (case["tokens"], case["heads"], case["dim"])
        dt = torch.float32 if case["fp32"] else torch.bfloat16
        st["x"] = _normal(gen, shape, dt)
        st["positions"] = torch.randint(0, case["span"], (case["tokens"],), generator=gen, **i32)
        st["inv_freq"] = _inv_freq(case["rope_dim"])
        st["out"] = torch.empty_like(st["x"])
        return st
    lens, seq, pos = _new_tokens(case)
    T = len(seq)
    st["q_seq"], st["q_pos"] = torch.tensor(seq, **i32), torch.tensor(pos, **i32)
    if case["op"] == "append":
        wide = case["dim"] + case["extra"]
        dt = torch.float32 if case["fp32"] else torch.bfloat16
        st["wide"] = _normal(gen, (T, wide), dt)
        st["rows"] = st["wide"][:, wide - case["dim"]:]
        first = [n - case["new"] for n in lens]
        st["pages"], total = _tables(lens, first, case["page"], gen)
        st["cache"] = _normal(gen, (total, case["page"], case["dim"]))
        st["inv_freq"] = _inv_freq(case["rope_dim"]) if case["rope_dim"] else None
        return st
    vis = [n // case["ratio"] for n in lens]
    if case["op"] == "indexer":
        hi, di = case["heads"], case["dim"]
        st["pages"], total = _tables(vis, [0] * len(vis), case["page"], gen)
        st["cache"] = _grid(gen, (total, case["page"], di), 0.5, torch.bfloat16)
        st["q"] = _grid(gen, (T, hi, di), 0.5, torch.bfloat16)
        st["w"] = _grid(gen, (T, hi), 0.125, torch.float32)
        st["idx"] = torch.empty((T, case["topk"]), **i32)
        st["val"] = torch.empty((T, case["topk"]), dtype=torch.float32, device="cuda")
        if own:
            import sparse_attention_csa_gb300 as csa
            st["ws"] = torch.empty(csa.csa_indexer_topk_paged_workspace_size(
                T, st["pages"].shape[1] * case["page"], hi, di, case["topk"]),
                dtype=torch.uint8, device="cuda")
        return st
    H, W = case["heads"], case["window"]
    first = [max(0, n - case["new"] - W + 1) for n in lens]
    st["ori_pages"], total = _tables(lens, first, case["page"], gen)
    st["ori"] = _normal(gen, (total, case["page"], 512))
    st["q"] = _normal(gen, (T, H, 512))
    st["sinks"] = _normal(gen, (H,), torch.float32)
    st["scale"] = 1.0 / math.sqrt(512.0)
    st["cmp"] = st["cmp_pages"] = st["idx"] = None
    if case["mode"] != "window":
        st["cmp_pages"], total = _tables(vis, [0] * len(vis), case["page"], gen)
        st["cmp"] = _normal(gen, (total, case["page"], 512))
    if case["mode"] == "list":
        idx = torch.full((T, case["topk"]), -1, **i32)
        for t in range(T):
            nv = (pos[t] + 1) // case["ratio"]
            k = min(nv, case["topk"])
            if k:
                perm = torch.randperm(nv, generator=gen, device="cuda")[:k]
                idx[t, :k] = torch.sort(perm).values.to(torch.int32)
        st["idx"] = idx
    st["out"] = torch.empty_like(st["q"])
    st["lse"] = torch.empty((T, H), dtype=torch.float32, device="cuda")
    if own:
        import sparse_attention_csa_gb300 as csa
        st["ws"] = torch.empty(csa.csa_sparse_mla_paged_workspace_size(T, H),
                               dtype=torch.uint8, device="cuda")
    return st


# --------------------------------------------------------------------- runs
def _cos_sin(positions, inv_freq, inverse):
    """fp32 cos and sin [T, n/2] of positions * inv_freq, the angle in 64 bits."""
    ang = positions.double()[:, None] * inv_freq[None, :]
    if inverse:
        ang = -ang
    return torch.cos(ang).float(), torch.sin(ang).float()


def _rotate(x, cos, sin, offset, half):
    """fp32 copy of x [T, H, D] with its rotary part turned."""
    y = x.float()
    if y.data_ptr() == x.data_ptr():
        y = y.clone()
    n = 2 * cos.shape[1]
    part = y[..., offset:offset + n]
    if half:
        a, b = part[..., :n // 2].clone(), part[..., n // 2:].clone()
    else:
        a, b = part[..., 0::2].clone(), part[..., 1::2].clone()
    c, s = cos[:, None, :], sin[:, None, :]
    ra, rb = a * c - b * s, b * c + a * s
    if half:
        part[..., :n // 2], part[..., n // 2:] = ra, rb
    else:
        part[..., 0::2], part[..., 1::2] = ra, rb
    return y


def _physical(table, seq, row, page):
    """Row of the pool (or -1) of each logical row [T, K] of sequences seq [T]."""
    ok = (row >= 0) & (row < table.shape[1] * page)
    r = torch.where(ok, row, torch.zeros_like(row)).long()
    p = table[seq.long()[:, None], r // page].long()
    return torch.where(ok & (p >= 0), p * page + r % page, torch.full_like(p, -1))


def _plain_indexer(st):
    c = st["case"]
    pages, page, k = st["pages"], c["page"], st["cache"].view(-1, c["dim"])
    T, cap, topk = st["q"].shape[0], pages.shape[1] * page, c["topk"]
    out, vals = [], []
    step = max(1, (1 << 28) // (cap * c["dim"] * 4))
    for t0 in range(0, T, step):
        sl = slice(t0, min(T, t0 + step))
        j = torch.arange(cap, device="cuda")[None, :].expand(sl.stop - t0, cap)
        nv = torch.div(st["q_pos"][sl] + 1, c["ratio"], rounding_mode="floor").long()
        phys = _physical(pages, st["q_seq"][sl], j, page)
        ok = (j < nv[:, None]) & (phys >= 0)
        rows = k[phys.clamp(min=0)].float()                                   # [g, cap, Di]
        dots = torch.bmm(st["q"][sl].float(), rows.transpose(1, 2))           # [g, Hi, cap]
        s = (torch.clamp(dots, min=0) * st["w"][sl][:, :, None]).sum(1)
        s = torch.where(ok, s, torch.full_like(s, -math.inf))
        order = torch.sort(s, dim=1, descending=True, stable=True).indices[:, :topk]
        if order.shape[1] < topk:
            more = order.new_full((order.shape[0], topk - order.shape[1]), cap)
            order = torch.cat([order, more], 1)
        keep = torch.where(order < nv[:, None], order, torch.full_like(order, cap))
        keep = torch.sort(keep, dim=1).values
        out.append(torch.where(keep < cap, keep, torch.full_like(keep, -1)).int())
        if c["values"]:
            v = torch.gather(s, 1, keep.clamp(max=cap - 1))
            vals.append(torch.where(keep < cap, v, torch.full_like(v, -math.inf)))
    return (torch.cat(out), torch.cat(vals)) if c["values"] else torch.cat(out)


def _plain_attention(st):
    c = st["case"]
    W, page = c["window"], c["page"]
    T, H = st["q"].shape[:2]
    ori = st["ori"].view(-1, 512)
    K = 0
    if st["cmp"] is not None:
        K = c["topk"] if st["idx"] is not None else st["cmp_pages"].shape[1] * page
    step = max(1, (1 << 30) // ((W + K) * 512 * 4))
    outs, lses = [], []
    for t0 in range(0, T, step):
        sl = slice(t0, min(T, t0 + step))
        g = sl.stop - t0
        pos, seq = st["q_pos"][sl].long(), st["q_seq"][sl]
        win = pos[:, None] - (W - 1) + torch.arange(W, device="cuda")[None, :]
        phys = _physical(st["ori_pages"], seq, win, page)
        ok, keys = phys >= 0, ori[phys.clamp(min=0)].float()
        if K:
            j = (st["idx"][sl].long() if st["idx"] is not None
                 else torch.arange(K, device="cuda")[None, :].expand(g, K))
            nv = torch.div(pos + 1, c["ratio"], rounding_mode="floor")
            cp = _physical(st["cmp_pages"], seq, j, page)
            ok = torch.cat([ok, (cp >= 0) & (j < nv[:, None])], 1)
            keys = torch.cat([keys, st["cmp"].view(-1, 512)[cp.clamp(min=0)].float()], 1)
        logit = torch.bmm(st["q"][sl].float(), keys.transpose(1, 2)) * st["scale"]
        logit = torch.where(ok[:, None, :], logit, torch.full_like(logit, -math.inf))
        m = torch.maximum(logit.amax(2), st["sinks"][None, :])
        p = torch.exp(logit - m[:, :, None])
        z = p.sum(2) + torch.exp(st["sinks"][None, :] - m)
        outs.append((torch.bmm(p, keys) / z[:, :, None]).bfloat16())
        lses.append(m + torch.log(z))
    return torch.cat(outs), torch.cat(lses)


def run(state):
    st, c = state, state["case"]
    layout = "half" if c.get("half") else "interleaved"
    if own:
        import sparse_attention_csa_gb300 as csa
        if c["op"] == "rope":
            return csa.csa_rope(st["x"], st["positions"], st["inv_freq"], rope_offset=c["offset"],
                                layout=layout, inverse=c["inverse"], out=st["out"])
        if c["op"] == "append":
            return csa.csa_cache_append(st["rows"], st["q_seq"], st["q_pos"], st["pages"],
                                        st["cache"], inv_freq=st["inv_freq"],
                                        rope_offset=c["offset"], layout=layout,
                                        pos_stride=c["pos_stride"])
        if c["op"] == "indexer":
            idx, val = csa.csa_indexer_topk_paged(
                st["q"], st["cache"], st["w"], st["pages"], st["q_seq"], st["q_pos"], c["ratio"],
                c["topk"], return_value=c["values"], workspace=st["ws"], out=st["idx"],
                out_val=st["val"] if c["values"] else None)
            return (idx, val) if c["values"] else idx
        return csa.csa_sparse_mla_paged(st["q"], st["ori"], st["cmp"], st["idx"], st["ori_pages"],
                                        st["cmp_pages"], st["q_seq"], st["q_pos"], st["sinks"],
                                        st["scale"], c["ratio"], c["window"] - 1,
                                        return_softmax_lse=True, workspace=st["ws"],
                                        out=st["out"], lse=st["lse"])
    if c["op"] == "rope":
        cos, sin = _cos_sin(st["positions"], st["inv_freq"], c["inverse"])
        return _rotate(st["x"], cos, sin, c["offset"], c["half"]).to(st["x"].dtype)
    if c["op"] == "append":
        y = st["rows"].float()
        if st["inv_freq"] is not None:
            cos, sin = _cos_sin(st["q_pos"].long() * c["pos_stride"], st["inv_freq"], False)
            y = _rotate(st["rows"][:, None, :], cos, sin, c["offset"], c["half"])[:, 0]
        slot = _physical(st["pages"], st["q_seq"], st["q_pos"][:, None], c["page"])[:, 0]
        st["cache"].view(-1, c["dim"])[slot] = y.bfloat16()
        return st["cache"]
    if c["op"] == "indexer":
        return _plain_indexer(st)
    return _plain_attention(st)


# -------------------------------------------------------------------- exact
def _exact_turn(x, theta, offset, half):
    """x [T, H, D] fp64 turned by theta [T, n/2] as complex products."""
    n = 2 * theta.shape[1]
    first = torch.arange(n // 2, device=x.device) + offset if half else \
        2 * torch.arange(n // 2, device=x.device) + offset
    second = first + (n // 2 if half else 1)
    z = torch.complex(x[..., first], x[..., second])
    z = z * torch.polar(torch.ones_like(theta), theta)[:, None, :]
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        theta = st["positions"].double()[:, None] * st["inv_freq"]
        return _exact_turn(st["x"].double(), -theta if case["inverse"] else theta, case["offset"],
                           case["half"])
    page = case["page"]
    seqs, poss = st["q_seq"].tolist(), st["q_pos"].tolist()
    if case["op"] == "append":
        rows = st["rows"].double()
        if st["inv_freq"] is not None:
            theta = (st["q_pos"].double() * case["pos_stride"])[:, None] * st["inv_freq"]
            rows = _exact_turn(rows[:, None], theta, case["offset"], case["half"])[:, 0]
        cache, table = st["cache"].double(), st["pages"].tolist()
        p = torch.tensor([table[b][n // page] for b, n in zip(seqs, poss)], device="cuda")
        cache[p, torch.tensor([n % page for n in poss], device="cuda")] = rows
        return cache

    def gather(pool, table, b, lo, hi):
        """Rows [lo, hi) of sequence b in 64 bits."""
        first, last = lo // page, max(lo // page, -(-hi // page))
        got = pool[table[b, first:last].long()].double().flatten(0, 1)
        return got[lo - first * page:hi - first * page]

    if case["op"] == "indexer":
        want = torch.full((len(seqs), case["topk"]), -1, dtype=torch.int32, device="cuda")
        score = torch.full(want.shape, -math.inf, dtype=torch.float64, device="cuda")
        for t, (b, n) in enumerate(zip(seqs, poss)):
            nv = (n + 1) // case["ratio"]
            if nv == 0:
                continue
            k = gather(st["cache"], st["pages"], b, 0, nv)
            s = torch.relu(k @ st["q"][t].double().T) @ st["w"][t].double()
            best = torch.argsort(s, descending=True, stable=True)[:case["topk"]]
            best = torch.sort(best).values
            want[t, :best.numel()], score[t, :best.numel()] = best.int(), s[best]
        return (want, score) if case["values"] else want
    outs, lses = [], []
    for t, (b, n) in enumerate(zip(seqs, poss)):
        keys = gather(st["ori"], st["ori_pages"], b, max(0, n - case["window"] + 1), n + 1)
        nv = (n + 1) // case["ratio"]
        if st["cmp"] is not None and nv:
            rows = gather(st["cmp"], st["cmp_pages"], b, 0, nv)
            if st["idx"] is not None:
                rows = rows[st["idx"][t][st["idx"][t] >= 0].long()]
            keys = torch.cat([keys, rows])
        logit = st["q"][t].double() @ keys.T * st["scale"]
        full = torch.cat([logit, st["sinks"].double()[:, None]], 1)
        prob = torch.softmax(full, 1)[:, :-1]
        outs.append(prob @ keys)
        lses.append(torch.logsumexp(full, 1))
    return torch.stack(outs), torch.stack(lses)


# --------------------------------------------------------------------- work
def work(case):
    """Bytes and operations of one pass: inputs read once, outputs written once."""
    if case["op"] == "rope":
        n = case["tokens"] * case["heads"]
        return {"bytes": 2 * n * case["dim"] * (4 if case["fp32"] else 2) + 4 * case["tokens"],
                "flops": 3 * n * case["rope_dim"]}
    lens, seq, pos = _new_tokens(case)
    T = len(seq)
    if case["op"] == "append":
        return {"bytes": T * (case["dim"] * (6 if case["fp32"] else 4) + 12),
                "flops": 3 * T * case["rope_dim"]}
    nv = [(p + 1) // case["ratio"] for p in pos]
    if case["op"] == "indexer":
        hd = case["heads"] * case["dim"]
        rows = sum(n // case["ratio"] for n in lens)
        each = hd * 2 + case["heads"] * 4 + case["topk"] * (8 if case["values"] else 4)
        return {"bytes": rows * case["dim"] * 2 + T * each,
                "flops": sum(nv) * 2 * hd}
    W, new, H = case["window"], case["new"], case["heads"]
    win = sum(min(W + new - 1, n) for n in lens)
    keys = [min(W, p + 1) for p in pos]
    rows = 0
    if case["mode"] == "all":
        rows = sum(n // case["ratio"] for n in lens)
        keys = [k + n for k, n in zip(keys, nv)]
    elif case["mode"] == "list":
        # rows that several tokens of a sequence select are read once
        sel = [min(n, case["topk"]) for n in nv]
        rows = sum(min(n // case["ratio"], sum(sel[b * new:(b + 1) * new]))
                   for b, n in enumerate(lens))
        keys = [k + n for k, n in zip(keys, sel)]
    return {"bytes": (win + rows) * 1024 + T * H * (2 * 1024 + 4)
            + (T * case["topk"] * 4 if case["mode"] == "list" else 0),
            "flops": 4 * 512 * H * sum(keys)}
