"""Timed cases of the calls around compressed rows held in 4 bits and their
eviction: append to and read from a 4-bit paged cache, the paged sparse MLA
attention over it, the attention weight that cached rows received, and the
pages to give back by it.

``run`` computes a case in its plain form (elementary torch operations in 32
bits, 64 for angles and long sums) or, when ``own`` is true, with the library's
calls. ``exact`` computes the same outputs from the definitions in 64 bits.

A row of 512 dims takes 384 bytes: dims 0-447 as codes of 4 bits (sign, two
exponent bits, one of mantissa) in 28 groups of 16 that share an e4m3 scale,
one power of two for the whole row, and dims 448-511 (the rotary ones) in bf16.
"""

import math

import torch

own = False

_GOLD = 0.6180339887498949
_MID = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)       # between neighbouring code values
_VALUE = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
_EVICTED = -2 ** 31


def _lengths(case):
    """Context length of each sequence, new tokens included: spread over
    [lo, hi] by the golden ratio, the same for every seed."""
    lo, hi, n = case["lo"], case["hi"], case["seqs"]
    if n == 1:
        return [max(hi, case.get("new", 1))]
    return [max(case.get("new", 1), lo + int((hi - lo) * (((b + 1) * _GOLD) % 1.0)))
            for b in range(n)]


def listed():
    append = {"op": "append", "new": 1, "fp32": True, "rope_dim": 64, "half": False, "page": 64,
              "extra": 0, "pos_stride": 4}
    read = {"op": "read", "page": 64}
    attn = {"op": "attention", "new": 1, "heads": 64, "window": 128, "mode": "list", "topk": 512,
            "ratio": 4, "page": 64}
    mass = {"op": "mass", "new": 1, "heads": 64, "mode": "list", "topk": 512, "ratio": 4,
            "page": 64, "bits": 4}
    evict = {"op": "evict", "page": 64, "first": 64, "last": 256}
    return [
        # the row that every fourth decode step of 128 sequences completes, as
        # the compressor leaves it (fp32), written and read back
        dict(append, name="append_decode128", seqs=128, lo=250, hi=15000),
        # the compressed rows of 16 prompts, taken out of a wider projection
        dict(append, name="append_prefill16k", seqs=16, new=1023, lo=1023, hi=9000, fp32=False,
             extra=512),
        # a few rows looked at by a debugging tool or moved to another page
        dict(read, name="read_few", seqs=7, new=3, lo=100, hi=5000),
        # the cached prefixes of five sequences, for a packed forward over them
        dict(read, name="read_prefix", seqs=5, new=8191, lo=8191, hi=8500, page=128),
        # one user with a 128k-token context: the smallest attention call
        dict(attn, name="attention_one", seqs=1, lo=131072, hi=131072),
        # a full batch, 512 selected rows each
        dict(attn, name="attention_batch64", seqs=64, lo=4096, hi=65536),
        # few long ragged contexts, every compressed row attended
        dict(attn, name="attention_dense_long", seqs=6, mode="all", lo=30000, hi=262144, page=128),
        # the weight that one user's selected rows received
        dict(mass, name="mass_one", seqs=1, lo=131072, hi=131072),
        # the same for a batch with two drafted tokens beside each new one, over bf16 rows
        dict(mass, name="mass_drafts_bf16", seqs=27, new=3, lo=4096, hi=65536, bits=16),
        # every compressed row of few long contexts
        dict(mass, name="mass_dense_long", seqs=6, mode="all", lo=30000, hi=262144, page=128),
        # one long sequence gives back three quarters of its pages
        dict(evict, name="evict_one", seqs=1, lo=32768, hi=32768, keep=128),
        # a batch of sequences held to one budget, some below it
        dict(evict, name="evict_batch64", seqs=64, lo=1000, hi=65536, keep=256),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "read", "attention", "mass", "attention", "mass", "evict"])
    seqs = _log_int(rng, 1, 96)
    page = rng.choice([16, 40, 64, 128])
    if op in ("append", "read"):
        new = _log_int(rng, 1, max(1, 16384 // seqs))
        case = {"op": op, "seqs": seqs, "new": new, "lo": new, "hi": new + _log_int(rng, 1, 8192),
                "page": page}
        if op == "append":
            case.update(fp32=rng.random() < 0.5, rope_dim=rng.choice([0, 32, 64, 64]),
                        half=rng.random() < 0.5, extra=rng.choice([0, 0, 64, 520]),
                        pos_stride=rng.choice([1, 4, 128]))
        return case
    if op == "evict":
        hi = min(_log_int(rng, 16, 262144), 4194304 // seqs)
        return {"op": op, "seqs": seqs, "lo": max(1, hi // rng.choice([1, 2, 16])), "hi": hi,
                "page": page, "first": rng.choice([0, 1, 64]), "last": rng.choice([0, 1, 100, 512]),
                "keep": _log_int(rng, 1, max(2, hi // page))}
    new = rng.choice([1, 1, 1, 2, 4])
    mode = rng.choice(["list", "list", "all"])
    ratio = rng.choice([4, 4, 128])
    most = 131072 * ratio if mode == "all" else 2097152
    hi = min(_log_int(rng, 16, 262144), max(64, most // (seqs * new)))
    case = {"op": op, "seqs": seqs, "new": new, "heads": rng.choice([4, 8, 16, 31, 64, 64]),
            "mode": mode, "topk": rng.choice([8, 100, 512, 1024]), "ratio": ratio,
            "lo": max(new, hi // rng.choice([1, 2, 16])), "hi": hi, "page": page}
    if op == "attention":
        case["window"] = rng.choice([16, 128, 128, 300, 1024])
    else:
        case["bits"] = rng.choice([4, 4, 16])
    return case


# --------------------------------------------------------------- 4-bit rows
def _pack(x):
    """fp32 rows [N, 512] as bytes [N, 384]."""
    n = x.shape[0]
    g = x[:, :448].reshape(n, 28, 16)
    fine = torch.isfinite(g)
    top = torch.where(fine, g.abs(), torch.zeros_like(g)).amax(2)                 # [N, 28]
    unit = top.amax(1) / 6.0
    e = torch.clamp(torch.frexp(unit).exponent - 8, -100, 100)                    # unit in [1, 2) 2^(e + 7)
    e = torch.where(unit > 0, e, torch.full_like(e, -100))
    row = torch.ldexp(torch.ones_like(unit), e)[:, None]
    s8 = torch.clamp(torch.ldexp(top / 6.0, -e[:, None]), max=448.0).to(torch.float8_e4m3fn)
    scale = s8.float() * row
    mag = g.abs()
    code = torch.zeros(g.shape, dtype=torch.int32, device=x.device)
    for i, mid in enumerate(_MID):  # a tie goes to the even code
        edge = (mid * scale)[:, :, None]
        code += ((mag >= edge) if i % 2 else (mag > edge)).int()
    code = torch.where((scale > 0)[:, :, None] & fine, code, torch.zeros_like(code))
    code = code | (torch.signbit(g).int() << 3)
    # 8 dims a word: the low half holds dims 0, 2, 4, 6, the high half 1, 3, 5, 7
    c = code.reshape(n, 56, 4, 2)
    shift = torch.tensor([0, 4, 8, 12], dtype=torch.int32, device=x.device)
    half = (c << shift[None, None, :, None]).sum(2, dtype=torch.int32)            # [N, 56, 2]
    halves = torch.stack([half & 255, half >> 8], 3).to(torch.uint8)              # [N, 56, 2, 2]
    out = torch.zeros((n, 384), dtype=torch.uint8, device=x.device)
    out[:, :224] = halves.reshape(n, 224)
    bad = ~fine.all(2)
    out[:, 224:252] = torch.where(bad, torch.full_like(s8.view(torch.uint8), 0x7F), s8.view(torch.uint8))
    out[:, 252] = (e + 127).to(torch.uint8)
    out[:, 256:] = x[:, 448:].bfloat16().contiguous().view(torch.uint8)
    return out


def _unpack(b):
    """bytes [..., 384] as fp32 rows [..., 512]."""
    lead = b.shape[:-1]
    word = b[..., :224].reshape(*lead, 56, 2, 2).int()
    half = word[..., 0] | (word[..., 1] << 8)                                     # [..., 56, 2]
    shift = torch.tensor([0, 4, 8, 12], dtype=torch.int32, device=b.device)
    code = (half[..., None, :] >> shift[:, None]) & 15                            # [..., 56, 4, 2]
    value = torch.tensor(_VALUE + tuple(-v for v in _VALUE), device=b.device)[code.long()]
    scale = b[..., 224:252].contiguous().view(torch.float8_e4m3fn).float()
    row = torch.ldexp(torch.ones(lead, device=b.device), b[..., 252].int() - 127)
    low = value.reshape(*lead, 28, 16) * (scale * row[..., None])[..., None]
    high = b[..., 256:].contiguous().view(torch.bfloat16).float()
    return torch.cat([low.reshape(*lead, 448), high], -1)


# ------------------------------------------------------------------- inputs
def _normal(gen, shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _rows(gen, n):
    """Rows as a compressor leaves them: normal, dims of different spread."""
    x = torch.randn((n, 512), generator=gen, device="cuda")
    return x * (0.25 + 2.0 * torch.rand((1, 512), generator=gen, device="cuda"))


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
    page = case["page"]
    if case["op"] == "evict":
        lens = _lengths(case)
        st["pages"], _ = _tables(lens, [0] * len(lens), page, gen)
        st["rows"] = torch.tensor(lens, **i32)
        st["mass"] = torch.exp(2.0 * torch.randn((len(lens), st["pages"].shape[1] * page),
                                                 generator=gen, device="cuda"))
        st["out"] = torch.empty_like(st["pages"])
        st["freed"] = torch.empty_like(st["pages"])
        st["n_freed"] = torch.empty((len(lens),), **i32)
        return st
    lens, seq, pos = _new_tokens(case)
    T = len(seq)
    st["q_seq"], st["q_pos"] = torch.tensor(seq, **i32), torch.tensor(pos, **i32)
    if case["op"] in ("append", "read"):
        first = [n - case["new"] for n in lens]
        st["pages"], total = _tables(lens, first, page, gen)
        st["cache"] = _pack(_rows(gen, total * page)).view(total, page, 384)
        st["out"] = torch.empty((T, 512), dtype=torch.bfloat16, device="cuda")
        if case["op"] == "append":
            wide = torch.empty((T, 512 + case["extra"]), device="cuda",
                               dtype=torch.float32 if case["fp32"] else torch.bfloat16)
            wide.normal_(generator=gen)
            wide[:, case["extra"]:] = _rows(gen, T).to(wide.dtype)
            st["wide"], st["new"] = wide, wide[:, case["extra"]:]
            st["inv_freq"] = _inv_freq(case["rope_dim"]) if case["rope_dim"] else None
        return st
    H = case["heads"]
    vis = [n // case["ratio"] for n in lens]
    st["cmp_pages"], total = _tables(vis, [0] * len(vis), page, gen)
    rows = _rows(gen, total * page)
    st["cmp"] = (_pack(rows).view(total, page, 384) if case.get("bits", 4) == 4
                 else rows.bfloat16().view(total, page, 512))
    del rows
    st["q"] = _normal(gen, (T, H, 512))
    st["scale"] = 0.75 / math.sqrt(512.0)
    st["idx"] = None
    if case["mode"] == "list":
        idx = torch.full((T, case["topk"]), -1, **i32)
        for t in range(T):
            nv = (pos[t] + 1) // case["ratio"]
            k = min(nv, case["topk"])
            if k:
                perm = torch.randperm(nv, generator=gen, device="cuda")[:k]
                idx[t, :k] = torch.sort(perm).values.to(torch.int32)
        st["idx"] = idx
    if case["op"] == "attention":
        W = case["window"]
        first = [max(0, n - case["new"] - W + 1) for n in lens]
        st["ori_pages"], total = _tables(lens, first, page, gen)
        st["ori"] = _normal(gen, (total, page, 512))
        st["sinks"] = _normal(gen, (H,), torch.float32)
        st["out"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty((T, H), dtype=torch.float32, device="cuda")
        st["ws"] = torch.empty((48 << 20,), dtype=torch.uint8, device="cuda")
        return st
    # log-sum-exp as the attention leaves it: the rows at hand, and a window
    # that took about as much
    ok, _, keys = _keys(st)
    logit = torch.bmm(st["q"].float(), keys.transpose(1, 2)) * st["scale"]
    logit = torch.where(ok[:, None, :], logit, torch.full_like(logit, -math.inf))
    st["lse"] = torch.logaddexp(torch.logsumexp(logit, 2),
                                torch.randn((T, H), generator=gen, device="cuda") + 4.0)
    shape = (len(lens), st["cmp_pages"].shape[1] * page)
    st["mass"] = torch.rand(shape, generator=gen, device="cuda") * 4.0
    st["new_mass"] = torch.empty(shape, device="cuda")
    slots = case["topk"] if case["mode"] == "list" else shape[1]
    st["ws"] = torch.empty(((slots + 256) * T * 4 + 4096,), dtype=torch.uint8, device="cuda")
    return st


# --------------------------------------------------------------------- runs
def _cos_sin(positions, inv_freq):
    """fp32 cos and sin [T, n/2] of positions * inv_freq, the angle in 64 bits."""
    ang = positions.double()[:, None] * inv_freq[None, :]
    return torch.cos(ang).float(), torch.sin(ang).float()


def _rotate(x, cos, sin, half):
    """fp32 copy of x [T, 512] with its last 2 * cos.shape[1] dims turned."""
    y = x.float().clone()
    n = 2 * cos.shape[1]
    part = y[:, 512 - n:]
    if half:
        a, b = part[:, :n // 2].clone(), part[:, n // 2:].clone()
        part[:, :n // 2], part[:, n // 2:] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = part[:, 0::2].clone(), part[:, 1::2].clone()
        part[:, 0::2], part[:, 1::2] = a * cos - b * sin, b * cos + a * sin
    return y


def _physical(table, seq, row, page):
    """Row of the pool (or -1) of each logical row [T, K] of sequences seq [T]."""
    ok = (row >= 0) & (row < table.shape[1] * page)
    r = torch.where(ok, row, torch.zeros_like(row)).long()
    p = table[seq.long()[:, None], r // page].long()
    return torch.where(ok & (p >= 0), p * page + r % page, torch.full_like(p, -1))


def _keys(st):
    """Compressed rows of every token: (present [T, K], row numbers, values)."""
    c, T = st["case"], st["q"].shape[0]
    cap = st["cmp_pages"].shape[1] * c["page"]
    j = (st["idx"].long() if st["idx"] is not None
         else torch.arange(cap, device="cuda")[None, :].expand(T, cap))
    nv = torch.div(st["q_pos"].long() + 1, c["ratio"], rounding_mode="floor")
    phys = _physical(st["cmp_pages"], st["q_seq"], j, c["page"])
    flat = st["cmp"].reshape(-1, st["cmp"].shape[2])[phys.clamp(min=0)]
    return (phys >= 0) & (j < nv[:, None]), j, _unpack(flat) if flat.dtype == torch.uint8 else flat.float()


def _plain_attention(st):
    c = st["case"]
    W = c["window"]
    pos = st["q_pos"].long()
    win = pos[:, None] - (W - 1) + torch.arange(W, device="cuda")[None, :]
    phys = _physical(st["ori_pages"], st["q_seq"], win, c["page"])
    ok, _, keys = _keys(st)
    ok = torch.cat([phys >= 0, ok], 1)
    keys = torch.cat([st["ori"].view(-1, 512)[phys.clamp(min=0)].float(), keys], 1)
    logit = torch.bmm(st["q"].float(), keys.transpose(1, 2)) * st["scale"]
    logit = torch.where(ok[:, None, :], logit, torch.full_like(logit, -math.inf))
    m = torch.maximum(logit.amax(2), st["sinks"][None, :])
    p = torch.exp(logit - m[:, :, None])
    z = p.sum(2) + torch.exp(st["sinks"][None, :] - m)
    return (torch.bmm(p, keys) / z[:, :, None]).bfloat16(), m + torch.log(z)


def _plain_mass(st):
    ok, j, keys = _keys(st)
    logit = torch.bmm(st["q"].float(), keys.transpose(1, 2)) * st["scale"]
    w = torch.where(ok, torch.exp(logit - st["lse"][:, :, None]).sum(1), 0.0)
    cap = st["mass"].shape[1]
    at = st["q_seq"].long()[:, None] * cap + torch.where(ok, j, torch.zeros_like(j))
    total = st["mass"].double().flatten()
    total.index_add_(0, at.flatten(), w.double().flatten())
    return total.float().view_as(st["mass"])


def _plain_evict(st):
    c = st["case"]
    page, pages, rows = c["page"], st["pages"], st["rows"].long()
    B, P = pages.shape
    used = (torch.arange(P * page, device="cuda")[None, :] < rows[:, None])
    total = torch.where(used, st["mass"].double(), 0.0).view(B, P, page).sum(2)
    p = torch.arange(P, device="cuda")[None, :]
    held = (p * page < rows[:, None]) & (pages >= 0)
    safe = (p * page < c["first"]) | ((p + 1) * page > (rows - c["last"]).clamp(min=0)[:, None])
    free = held & ~safe
    room = (c["keep"] - (held & safe).sum(1)).clamp(min=0)
    order = torch.sort(torch.where(free, total, -math.inf), dim=1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(1, order, p.expand(B, P).contiguous())
    gone = free & (rank >= room[:, None])
    first = torch.sort(torch.where(gone, p, P), dim=1).values
    freed = torch.gather(pages, 1, first.clamp(max=P - 1))
    return (torch.where(gone, _EVICTED, pages).int(), torch.where(first < P, freed, -1).int(),
            gone.sum(1).int())


def run(state):
    st, c = state, state["case"]
    layout = "half" if c.get("half") else "interleaved"
    if own:
        import sparse_attention_csa_gb300 as csa
        if c["op"] == "append":
            csa.csa_cache_append_q4(st["new"], st["q_seq"], st["q_pos"], st["pages"], st["cache"],
                                    inv_freq=st["inv_freq"], layout=layout,
                                    pos_stride=c["pos_stride"])
        if c["op"] in ("append", "read"):
            return csa.csa_cache_read_q4(st["cache"], st["pages"], st["q_seq"], st["q_pos"],
                                         out=st["out"])
        if c["op"] == "attention":
            return csa.csa_sparse_mla_paged_q4(
                st["q"], st["ori"], st["cmp"], st["idx"], st["ori_pages"], st["cmp_pages"],
                st["q_seq"], st["q_pos"], st["sinks"], st["scale"], c["ratio"], c["window"] - 1,
                return_softmax_lse=True, workspace=st["ws"], out=st["out"], lse=st["lse"])
        if c["op"] == "mass":
            return csa.csa_attn_mass_paged(
                st["q"], st["lse"], st["cmp"], st["idx"], st["cmp_pages"], st["q_seq"], st["q_pos"],
                st["mass"], st["scale"], c["ratio"], out=st["new_mass"], workspace=st["ws"])
        return csa.csa_cache_evict(st["mass"], st["pages"], st["rows"], c["keep"],
                                   keep_first=c["first"], keep_last=c["last"], out=st["out"],
                                   freed=st["freed"], n_freed=st["n_freed"])
    if c["op"] in ("append", "read"):
        slot = _physical(st["pages"], st["q_seq"], st["q_pos"][:, None], c["page"])[:, 0]
        if c["op"] == "append":
            y = st["new"].float()
            if st["inv_freq"] is not None:
                y = _rotate(y, *_cos_sin(st["q_pos"].long() * c["pos_stride"], st["inv_freq"]),
                            c["half"])
            st["cache"].view(-1, 384)[slot] = _pack(y)
        return _unpack(st["cache"].view(-1, 384)[slot]).bfloat16()
    if c["op"] == "attention":
        return _plain_attention(st)
    if c["op"] == "mass":
        return _plain_mass(st)
    return _plain_evict(st)


# -------------------------------------------------------------------- exact
def _exact_value(b):
    """bytes [N, 384] as fp64 rows: byte by byte, from the format's words."""
    n = b.shape[0]
    y = torch.empty((n, 512), dtype=torch.float64, device=b.device)
    d = torch.arange(448, device=b.device)
    inner = d % 8
    nibble = inner // 2 + 4 * (inner % 2)
    raw = b[:, (d // 8) * 4 + nibble // 2].int()
    code = torch.where(nibble % 2 == 1, raw >> 4, raw & 15)
    mag = code & 7
    value = torch.where(mag < 2, mag.double() * 0.5,
                        (1.0 + 0.5 * (mag & 1).double()) * torch.exp2((mag // 2 - 1).double()))
    s = b[:, 224:252].int()
    scale = torch.where(s < 8, (s & 7).double() * 2.0 ** -9,
                        (1.0 + (s & 7).double() / 8.0) * torch.exp2(((s >> 3) - 7).double()))
    scale = scale * torch.exp2(b[:, 252].double() - 127.0)[:, None]
    y[:, :448] = torch.where(code >= 8, -value, value) * scale[:, d // 16]
    top = (b[:, 256::2].int() | (b[:, 257::2].int() << 8)) << 16
    y[:, 448:] = top.view(torch.float32).double()
    return y


def _exact_rounded(x):
    """fp64 rows [N, 512] with dims 0-447 at the values they are held as."""
    n = x.shape[0]
    g = x[:, :448].reshape(n, 28, 16)
    top = g.abs().amax(2)
    unit = top.amax(1, keepdim=True) / 6.0
    row = torch.exp2(torch.floor(torch.log2(unit.clamp(min=1e-300))) - 7.0).clamp(2.0 ** -100, 2.0 ** 100)
    r = top / 6.0 / row
    step = torch.exp2(torch.floor(torch.log2(r.clamp(min=2.0 ** -6))) - 3.0)
    scale = (torch.round(r / step) * step * row)[:, :, None]
    z = g.abs() / scale.clamp(min=1e-300)
    fine = torch.where(z < 2.0, 0.5, torch.where(z < 4.0, 1.0, 2.0))
    held = torch.round(z / fine) * fine
    held = torch.where(scale > 0, torch.clamp(held, max=6.0) * scale, 0.0)
    return torch.cat([(torch.sign(g) * held).reshape(n, 448), x[:, 448:]], 1)


def exact(case, seed):
    if case["op"] == "evict":
        return None
    st = prepare(case, seed)
    page = case["page"]
    seqs, poss = st["q_seq"].tolist(), st["q_pos"].tolist()
    if case["op"] in ("append", "read"):
        if case["op"] == "append":
            x = st["new"].double()
            if st["inv_freq"] is not None:
                n = case["rope_dim"]
                theta = (st["q_pos"].double() * case["pos_stride"])[:, None] * st["inv_freq"]
                at = torch.arange(n // 2, device="cuda")
                first = 512 - n + (at if case["half"] else 2 * at)
                second = first + (n // 2 if case["half"] else 1)
                z = torch.complex(x[:, first], x[:, second]) * torch.polar(torch.ones_like(theta), theta)
                x[:, first], x[:, second] = z.real, z.imag
            return _exact_rounded(x)
        table = st["pages"].tolist()
        p = torch.tensor([table[b][n // page] for b, n in zip(seqs, poss)], device="cuda")
        return _exact_value(st["cache"][p, torch.tensor([n % page for n in poss], device="cuda")])

    def gather(pool, table, b, lo, hi):
        """Rows [lo, hi) of sequence b in 64 bits."""
        first, last = lo // page, max(lo // page, -(-hi // page))
        got = pool[table[b, first:last].long()].flatten(0, 1)[lo - first * page:hi - first * page]
        return _exact_value(got) if got.dtype == torch.uint8 else got.double()

    outs, lses = [], []
    mass = st["mass"].double() if case["op"] == "mass" else None
    for t, (b, n) in enumerate(zip(seqs, poss)):
        nv = (n + 1) // case["ratio"]
        j = (torch.arange(nv, device="cuda") if st["idx"] is None
             else st["idx"][t][st["idx"][t] >= 0].long())
        rows = gather(st["cmp"], st["cmp_pages"], b, 0, nv)[j]
        if mass is not None:
            logit = st["q"][t].double() @ rows.T * st["scale"]
            mass[b, j] += torch.exp(logit - st["lse"][t].double()[:, None]).sum(0)
            continue
        keys = torch.cat([gather(st["ori"], st["ori_pages"], b, max(0, n - case["window"] + 1), n + 1),
                          rows])
        logit = st["q"][t].double() @ keys.T * st["scale"]
        full = torch.cat([logit, st["sinks"].double()[:, None]], 1)
        outs.append(torch.softmax(full, 1)[:, :-1] @ keys)
        lses.append(torch.logsumexp(full, 1))
    return mass if mass is not None else (torch.stack(outs), torch.stack(lses))


# --------------------------------------------------------------------- work
def work(case):
    """Bytes and operations of one pass: inputs read once, outputs written once."""
    if case["op"] == "evict":
        lens = _lengths(case)
        P = -(-max(lens) // case["page"])
        return {"bytes": 4 * sum(lens) + len(lens) * (12 * P + 8), "flops": sum(lens)}
    lens, seq, pos = _new_tokens(case)
    T = len(seq)
    if case["op"] == "read":
        return {"bytes": T * (384 + 1024 + 12), "flops": T * 512}
    if case["op"] == "append":
        # the row is read, held and given back
        return {"bytes": T * (512 * (4 if case["fp32"] else 2) + 384 + 1024 + 12),
                "flops": T * (10 * 448 + 3 * case["rope_dim"])}
    new, H = case["new"], case["heads"]
    nv = [(p + 1) // case["ratio"] for p in pos]
    if case["mode"] == "all":
        keys = list(nv)
        rows = sum(n // case["ratio"] for n in lens)
    else:
        # rows that several tokens of a sequence select are read once
        keys = [min(n, case["topk"]) for n in nv]
        rows = sum(min(n // case["ratio"], sum(keys[b * new:(b + 1) * new]))
                   for b, n in enumerate(lens))
    listed_bytes = T * case["topk"] * 4 if case["mode"] == "list" else 0
    if case["op"] == "mass":
        cap = -(-max(n // case["ratio"] for n in lens) // case["page"]) * case["page"]
        return {"bytes": rows * (384 if case["bits"] == 4 else 1024) + T * H * (1024 + 4)
                + listed_bytes + 8 * len(lens) * max(cap, case["page"]),
                "flops": 2 * 512 * H * sum(keys)}
    W = case["window"]
    win = sum(min(W + new - 1, n) for n in lens)
    keys = [k + min(W, p + 1) for k, p in zip(keys, pos)]
    return {"bytes": win * 1024 + rows * 384 + T * H * (2 * 1024 + 4) + listed_bytes,
            "flops": 4 * 512 * H * sum(keys)}
