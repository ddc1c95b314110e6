"""The serving operators around the packed, paged KV cache: what is measured, and their plain forms.

Three operators a serving loop calls next to the decode step:

* ``tables``: block tables and slot maps from request lengths (``page_tables``);
* ``prompt``: causal attention of packed prompts, grouped heads (``prompt_attention``);
* ``tree``: attention of drafted tokens (a tree, or a chain) over the paged, packed cache
  (``tree_attention``).

With ``own`` false, ``run`` computes them with elementary torch operations in 32 bits; with ``own``
true it makes the calls of ``kv_cache_vector_11_b200``.
"""

import math
import random

import numpy as np
import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
MASK64 = (1 << 64) - 1
HALF = {"bf16": torch.bfloat16, "f16": torch.float16}
ROT_SEED = 1000


def _tq():
    import kv_cache_vector_11_b200 as tq
    return tq


# ---------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------

def listed():
    return [
        # -- block tables and slot maps --
        # a decode step of 256 requests of up to 128K tokens in 256-token pages (the paged benchmark's
        # page size): one new token each, the call that every step makes
        dict(name="tables decode 256", op="tables", batch=256, page=256, ctx_hi=131072, new_lo=1, new_hi=1,
             pad=0, mix=1),
        # the drafted trees of 33 requests in 16-token pages, the token rows padded to a captured size
        dict(name="tables drafts 33", op="tables", batch=33, page=16, ctx_hi=4096, new_lo=1, new_hi=64,
             pad=321, mix=2),
        # admission of 512 fresh prompts of up to 4096 tokens
        dict(name="tables prompts 512", op="tables", batch=512, page=64, ctx_hi=0, new_lo=1, new_hi=4096,
             pad=0, mix=3),
        # -- attention over whole prompts --
        # three short prompts of a small model in fp16: latency counts
        dict(name="prompt short f16", op="prompt", batch=3, hq=8, hkv=2, d=64, q_lo=1, q_hi=130, k_more=0,
             dtype="f16", mix=4),
        # a packed batch of ragged prompts at the benchmark's head layout (32 query heads, 8 KV heads)
        dict(name="prompt packed bf16", op="prompt", batch=16, hq=32, hkv=8, d=128, q_lo=64, q_hi=2048,
             k_more=0, dtype="bf16", mix=5),
        # one long prompt
        dict(name="prompt 8192 bf16", op="prompt", batch=1, hq=32, hkv=8, d=128, q_lo=8192, q_hi=8192,
             k_more=0, dtype="bf16", mix=6),
        # later chunks of prompts: fewer queries than keys, wide heads, three query heads to a KV head
        dict(name="prompt chunks d256", op="prompt", batch=5, hq=12, hkv=4, d=256, q_lo=33, q_hi=1024,
             k_more=2000, dtype="bf16", mix=7),
        # -- attention of drafted tokens over the packed cache --
        # one request, a small draft, a short cache: latency counts
        dict(name="tree small f16", op="tree", batch=1, hq=8, hkv=2, d=64, page=16, kb=4, vb=2, rot="haar",
             n_lo=5, n_hi=5, len_lo=300, len_hi=300, chain=False, dtype="f16", mix=8),
        # 16 requests with trees of up to 32 nodes over 3-bit caches of up to 32K tokens
        dict(name="tree 16 x 32K", op="tree", batch=16, hq=32, hkv=8, d=128, page=64, kb=3, vb=3, rot="wht",
             n_lo=8, n_hi=32, len_lo=2048, len_hi=32768, chain=False, dtype="bf16", mix=9),
        # single tokens of 64 requests whose lengths differ: a ragged decode step
        dict(name="tree single tokens", op="tree", batch=64, hq=32, hkv=8, d=128, page=128, kb=4, vb=3,
             rot="wht", n_lo=1, n_hi=1, len_lo=1, len_hi=32768, chain=True, dtype="bf16", mix=10),
        # the 128K decode workload's cache (4-bit keys, 3-bit values) with 64-node trees: the largest
        dict(name="tree 8 x 128K", op="tree", batch=8, hq=32, hkv=8, d=128, page=256, kb=4, vb=3, rot="wht",
             n_lo=64, n_hi=64, len_lo=131072, len_hi=131072, chain=False, dtype="bf16", mix=11),
        # wide heads, eight query heads to a KV head, deep trees
        dict(name="tree d256 group 8", op="tree", batch=4, hq=16, hkv=2, d=256, page=32, kb=4, vb=4,
             rot="wht", n_lo=60, n_hi=250, len_lo=1000, len_hi=9000, chain=False, dtype="f16", mix=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    mix = rng.randrange(100, 1 << 30)
    op = rng.choice(["tables", "prompt", "tree"])
    if op == "tables":
        new_hi = _log(rng, 1, 4096)
        return dict(op=op, batch=_log(rng, 1, 512), page=1 << rng.randrange(4, 9),
                    ctx_hi=rng.choice([0, _log(rng, 1, 131072)]), new_lo=rng.choice([0, 1]), new_hi=new_hi,
                    pad=rng.choice([0, rng.randrange(1, 500)]), mix=mix)
    hkv = rng.choice([1, 2, 4, 8])
    d = rng.choice([64, 128, 256])
    dtype = rng.choice(["bf16", "f16"])
    if op == "prompt":
        hq = hkv * rng.choice([1, 2, 3, 4])
        batch = _log(rng, 1, 24)
        return dict(op=op, batch=batch, hq=hq, hkv=hkv, d=d, q_lo=1, q_hi=_log(rng, 2, 6000 // math.isqrt(batch)),
                    k_more=rng.choice([0, 0, _log(rng, 1, 2000)]), dtype=dtype, mix=mix)
    group = rng.choice([1, 2, 4, 7, 8])
    batch = _log(rng, 1, 48)
    n_hi = rng.choice([1, _log(rng, 2, 64), _log(rng, 2, 256)])
    hi = _log(rng, 2 * n_hi, max(2 * n_hi + 1, 262144 // (batch * hkv)))
    return dict(op=op, batch=batch, hq=group * hkv, hkv=hkv, d=d, page=1 << rng.randrange(4, 9),
                kb=rng.choice([2, 3, 4]), vb=rng.choice([2, 3, 4]), rot=rng.choice(["wht", "haar"]), n_lo=1,
                n_hi=n_hi, len_lo=n_hi, len_hi=max(hi, n_hi), chain=rng.choice([False, True]), dtype=dtype, mix=mix)


def _lens(rng, n, lo, hi):
    """n lengths spread over the logarithm of [lo, hi] (0 counts as below 1)."""
    if hi <= 0:
        return [0] * n
    out = [_log(rng, max(lo, 1), hi) for _ in range(n)]
    if lo == 0:
        out = [0 if rng.random() < 0.2 else x for x in out]
    return out


def _shape(case):
    """The lengths of a case: a function of the case alone (the seed only changes values)."""
    rng = random.Random(case["mix"])
    if case["op"] == "tables":
        ctx = _lens(rng, case["batch"], 0, case["ctx_hi"])
        new = _lens(rng, case["batch"], case["new_lo"], case["new_hi"])
        return ctx, new
    if case["op"] == "prompt":
        q = _lens(rng, case["batch"], case["q_lo"], case["q_hi"])
        k = [x + (rng.randrange(case["k_more"] + 1) if case["k_more"] else 0) for x in q]
        return q, k
    n = _lens(rng, case["batch"], case["n_lo"], case["n_hi"])
    ln = [max(a, b) for a, b in zip(_lens(rng, case["batch"], case["len_lo"], case["len_hi"]), n)]
    return n, ln


def _pages_of(tokens, page):
    return -(-tokens // page)


def work(case):
    a, b = _shape(case)
    if case["op"] == "tables":
        n = sum(b)
        rows = n + case["pad"]
        fresh = sum(_pages_of(x + y, case["page"]) - _pages_of(x, case["page"]) for x, y in zip(a, b))
        held = sum(1 for x, y in zip(a, b) if x % case["page"] and y)
        # lengths in; slots (8 bytes), positions, offsets and totals out; pages from the free list into
        # the table; the entries of the last pages already held
        return {"bytes": 8 * len(a) + 12 * rows + 4 * (len(a) + 1) + 4 * len(a) + 8 * fresh + 4 * held, "flops": 0}
    if case["op"] == "prompt":
        pairs = sum(x * y - x * (x - 1) // 2 for x, y in zip(a, b))
        elems = sum(a) * 2 * case["hq"] + sum(b) * 2 * case["hkv"]
        return {"bytes": 2 * case["d"] * elems, "flops": 4 * case["d"] * case["hq"] * pairs}
    d, rows = case["d"], sum(a)
    row_bytes = d * (case["kb"] + case["vb"]) // 8 + 2 * (d // 32) * 2
    pairs = sum(x * (y - x) + (x * (x + 1) // 2 if case["chain"] else x * x) for x, y in zip(a, b))
    table = sum(_pages_of(y, case["page"]) for y in b)
    mask = 0 if case["chain"] else rows * 8 * _words(case)
    return {"bytes": sum(b) * case["hkv"] * row_bytes + rows * case["hq"] * d * 4 + 4 * table + mask,
            "flops": 4 * d * case["hq"] * pairs}


# ---------------------------------------------------------------------------------------------
# The cache format, as the library documents it
# ---------------------------------------------------------------------------------------------

def _splitmix(seed, n):
    out, state = [], seed & MASK64
    for _ in range(n):
        state = (state + 0x9E3779B97F4A7C15) & MASK64
        z = state
        z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & MASK64
        z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & MASK64
        out.append(z ^ (z >> 31))
    return out


def _rotation(kind, d):
    """The dense rotation of a seed, float64 [d, d]."""
    if kind == "wht":
        s = np.array([-1.0 if z >> 63 else 1.0 for z in _splitmix(ROT_SEED, 2 * d)])
        h = np.array([[1.0]])
        while h.shape[0] < d:
            h = np.block([[h, h], [h, -h]])
        return s[:d, None] * h * s[None, d:] / math.sqrt(d)
    u = np.array([(z >> 11) * 2.0 ** -53 for z in _splitmix(ROT_SEED, d * d)])
    r, t = np.sqrt(-2.0 * np.log(1.0 - u[0::2])), 2.0 * np.pi * u[1::2]
    g = np.stack([r * np.cos(t), r * np.sin(t)], 1).reshape(d, d)
    q, r = np.linalg.qr(g)
    q = q * np.sign(np.diag(r))[None, :]
    if np.linalg.slogdet(q)[0] < 0:
        q[:, 0] = -q[:, 0]
    return q


# Lloyd-Max levels of a coordinate of a unit 32-vector, as binary16 (the positive half)
LEVELS = {
    2: [0.07977294921875, 0.263427734375],
    3: [0.0428466796875, 0.1317138671875, 0.232421875, 0.3662109375],
    4: [0.0223236083984375, 0.06744384765625, 0.1138916015625, 0.1629638671875, 0.2161865234375,
        0.276611328125, 0.349853515625, 0.453369140625],
}


def _levels(bits):
    return np.array([-x for x in reversed(LEVELS[bits])] + LEVELS[bits], dtype=np.float32)


def _packed_rows(gen, n, d, bits, scale):
    """n cache rows of normally distributed values in the rotated frame: packed codes int32 and
    fp16 norms (as int16 bits)."""
    lv = torch.from_numpy(_levels(bits)).to(DEV)
    bound = (lv[1:] + lv[:-1]) / 2
    codes = torch.empty((n, d // 32 * bits), dtype=torch.int32, device=DEV)
    norms = torch.empty((n, d // 32), dtype=torch.float16, device=DEV)
    pos = torch.arange(32, device=DEV) * bits
    word, sh = pos // 32, pos % 32
    for r0 in range(0, n, 1 << 19):
        m = min(n - r0, 1 << 19)
        y = torch.randn((m, d // 32, 32), generator=gen, device=DEV) * scale
        nrm = y.norm(dim=-1, keepdim=True)
        c = torch.bucketize(y / nrm.clamp_min(1e-30), bound).to(torch.int64)
        words = torch.zeros((m, d // 32, bits + 1), dtype=torch.int64, device=DEV)
        words.index_add_(2, word, (c << sh) & 0xFFFFFFFF)
        words.index_add_(2, word + 1, (c << sh) >> 32)
        w = words[..., :bits]
        codes[r0:r0 + m] = torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32).reshape(m, -1)
        norms[r0:r0 + m] = nrm[..., 0].to(torch.float16)
    return codes, norms.view(torch.int16)


def _dequantize(codes, norms, bits, dtype=torch.float32):
    """Rows [..., words] and [..., blocks] -> values [..., d] in the rotated frame."""
    lv = torch.from_numpy(_levels(bits)).to(codes.device, dtype)
    nb = norms.shape[-1]
    w = codes.reshape(*codes.shape[:-1], nb, bits).long() & 0xFFFFFFFF
    w = torch.cat([w, torch.zeros_like(w[..., :1])], -1)
    w = w[..., :-1] | w[..., 1:] << 32                                # each word with the next one above it
    pos = torch.arange(32, device=codes.device) * bits
    idx = (w[..., pos // 32] >> pos % 32) & ((1 << bits) - 1)
    x = lv[idx] * norms.view(torch.float16).to(dtype).unsqueeze(-1)
    return x.reshape(*norms.shape[:-1], nb * 32)


# ---------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------

def _words(case):
    return -(-case["n_hi"] // 64)


def _ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device=DEV)


def _starts(lens):
    return _ints([0] + list(np.cumsum(lens)))


def _tree_mask(rng, n, words):
    """Ancestor bits of a random tree of n nodes (each node's parent comes before it): the bits of a
    row are the node and its ancestors, 64 to a word."""
    rows = []
    for i in range(n):
        parent = rng.randrange(max(-1, i - 8), i) if i else -1
        rows.append((rows[parent] if parent >= 0 else 0) | 1 << i)
    words_of = [[r >> 64 * w & MASK64 for w in range(words)] for r in rows]
    return [[x - (1 << 64) if x >> 63 else x for x in r] for r in words_of]


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    a, b = _shape(case)
    s = dict(case=case, op=case["op"])
    if case["op"] == "tables":
        P = case["page"]
        held = [_pages_of(x, P) for x in a]
        total = [_pages_of(x + y, P) for x, y in zip(a, b)]
        n_pages = sum(total) + 7
        perm = torch.randperm(n_pages, generator=gen, device=DEV).to(torch.int32)
        table = torch.full((case["batch"], max(max(total), 1)), -1, dtype=torch.int32, device=DEV)
        col = torch.arange(table.shape[1], device=DEV)
        own_pages = col[None, :] < _ints(held)[:, None]
        table[own_pages] = perm[:sum(held)]
        n_slots = sum(b) + case["pad"]
        s.update(ctx=_ints(a), new=_ints(b), table=table, free=perm[sum(held):].contiguous(), n_pages=n_pages, page=P,
                 n_slots=n_slots)
        if own:
            s["out"] = dict(cu_new=torch.empty(case["batch"] + 1, dtype=torch.int32, device=DEV),
                            total_lens=torch.empty(case["batch"], dtype=torch.int32, device=DEV),
                            slots=torch.empty(n_slots, dtype=torch.int64, device=DEV),
                            positions=torch.empty(n_slots, dtype=torch.int32, device=DEV),
                            n_taken=torch.empty(1, dtype=torch.int32, device=DEV))
        return s
    dt, d, hq, hkv = HALF[case["dtype"]], case["d"], case["hq"], case["hkv"]
    if case["op"] == "prompt":
        def rows(n, h):
            return torch.randn((n, h, d), generator=gen, device=DEV).to(dt)
        s.update(q=rows(sum(a), hq), k=rows(sum(b), hkv), v=rows(sum(b), hkv), cu_q=_starts(a),
                 cu_k=_starts(b), max_q=max(a), max_k=max(b))
        if a == b:
            s["cu_k"] = s["cu_q"]
        return s
    # drafted tokens: pages in random order, keys and values of unit variance, queries of twice that (peaked and
    # flat heads side by side)
    P = case["page"]
    rng = random.Random(seed)
    per = [_pages_of(x, P) for x in b]
    n_pages = sum(per) + 3
    perm = torch.randperm(n_pages, generator=gen, device=DEV).to(torch.int32)
    table = torch.zeros((case["batch"], max(per)), dtype=torch.int32, device=DEV)
    table[torch.arange(max(per), device=DEV)[None, :] < _ints(per)[:, None]] = perm[:sum(per)]
    pages = {}
    for name, bits in (("k", case["kb"]), ("v", case["vb"])):
        c, n = _packed_rows(gen, n_pages * hkv * P, d, bits, 1.0)
        pages[name + "_codes"] = c.view(n_pages, hkv, P, -1)
        pages[name + "_norms"] = n.view(n_pages, hkv, P, -1)
    heat = torch.linspace(0.5, 2.0, hq, device=DEV)[None, :, None]
    q = (torch.randn((sum(a), hq, d), generator=gen, device=DEV) * heat).to(dt)
    mask = None
    if not case["chain"]:
        w = _words(case)
        mask = _ints([r for n in a for r in _tree_mask(rng, n, w)], torch.int64).view(sum(a), w)
    R = _rotation(case["rot"], d)
    s.update(q=q, pages=pages, table=table, cu=_starts(a), lens=_ints(b), max_n=max(a), max_len=max(b), mask=mask,
             page=P, R32=torch.from_numpy(R).to(DEV, torch.float32), kc=_levels(case["kb"]), vc=_levels(case["vb"]))
    if own:
        tq = _tq()
        s["rot"] = tq.Rotation(case["rot"], d, d, ROT_SEED)
        s["ws"] = torch.empty(tq.tree_workspace_size(case["batch"], sum(a), max(a), hq, hkv, max(b), d),
                              dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------

def run(s):
    if own:
        return _run_own(s)
    return {"tables": _plain_tables, "prompt": _plain_prompt, "tree": _plain_tree}[s["op"]](s)


def _run_own(s):
    tq = _tq()
    c = s["case"]
    if s["op"] == "tables":
        out = tq.page_tables(s["ctx"], s["new"], s["page"], s["n_pages"], s["free"], s["table"], s["n_slots"],
                             out=s["out"])
        return dict(out, block_table=s["table"])
    if s["op"] == "prompt":
        return tq.prompt_attention(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"])
    return tq.tree_attention(s["rot"], c["kb"], c["vb"], s["kc"], s["vc"], s["q"], s["cu"], s["lens"], s["pages"],
                             s["table"], s["page"], s["max_n"], s["max_len"], tree_mask=s["mask"],
                             workspace=s["ws"])


def _plain_tables(s):
    ctx, new, P, n_slots = s["ctx"].long(), s["new"].long(), s["page"], s["n_slots"]
    batch, cols = s["table"].shape
    held, want = (ctx + P - 1) // P, (ctx + new + P - 1) // P
    need = want - held
    base = need.cumsum(0) - need
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device=new.device), new.cumsum(0)])
    # the table: column j of request b is a page it held, or the (base + j - held)-th free page
    j = torch.arange(cols, device=new.device)[None, :]
    pick = (base[:, None] + j - held[:, None]).clamp(0, s["free"].numel() - 1)
    fresh = (j >= held[:, None]) & (j < want[:, None])
    table = torch.where(fresh, s["free"][pick], s["table"])
    # the slot map: token i belongs to the request whose range holds i
    i = torch.arange(n_slots, device=new.device)
    b = (torch.searchsorted(cu, i, right=True) - 1).clamp(0, batch - 1)
    pos = ctx[b] + i - cu[b]
    live = i < cu[batch]
    page = table.long()[b, (pos // P).clamp(0, cols - 1)]
    slots = torch.where(live, page * P + pos % P, -1)
    return dict(cu_new=cu.int(), total_lens=(ctx + new).int(), slots=slots,
                positions=torch.where(live, pos, -1).int(), n_taken=need.sum().reshape(1).int(), block_table=table)


def _padded(x, starts, longest):
    """Packed rows [total, ...] -> [batch, longest, ...] (rows past a sequence repeat some row)."""
    at = starts[:-1].long()[:, None] + torch.arange(longest, device=x.device)[None, :]
    return x[at.clamp(max=x.shape[0] - 1)]


def _unpadded(x, starts, total):
    """The inverse: [batch, longest, ...] -> [total, ...]."""
    i = torch.arange(total, device=x.device)
    b = torch.searchsorted(starts[1:].long(), i, right=True)
    return x[b, i - starts.long()[b]]


def _attend(q, k, v, allowed, scale):
    """q [B, N, Hq, d], k and v [B, L, Hkv, d], allowed [B, N, L] -> [B, N, Hq, d]; a row that may
    attend nothing is zero."""
    B, N, hq, d = q.shape
    hkv = k.shape[2]
    q = q.reshape(B, N, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(B, hkv, -1, d)
    p = (q @ k.permute(0, 2, 3, 1)).mul_(scale).view(B, hkv, hq // hkv, N, -1)
    p.masked_fill_(~allowed[:, None, None], -math.inf)
    top = p.amax(-1, keepdim=True)
    p.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = p.view(B, hkv, -1, p.shape[-1]) @ v.permute(0, 2, 1, 3)
    o = o.view(B, hkv, hq // hkv, N, d) / torch.where(total == 0, 1.0, total)
    return o.permute(0, 3, 1, 2, 4).reshape(B, N, hq, d)


def _plain_prompt(s):
    q = _padded(s["q"].float(), s["cu_q"], s["max_q"])
    k, v = (_padded(s[n].float(), s["cu_k"], s["max_k"]) for n in "kv")
    nq, nk = (s[n][1:] - s[n][:-1] for n in ("cu_q", "cu_k"))
    i = torch.arange(s["max_q"], device=q.device)[None, :, None]
    j = torch.arange(s["max_k"], device=q.device)[None, None, :]
    allowed = (j < nk[:, None, None]) & (j <= i + (nk - nq)[:, None, None])
    o = _attend(q, k, v, allowed, s["case"]["d"] ** -0.5)
    return _unpadded(o, s["cu_q"], s["q"].shape[0]).to(s["q"].dtype)


def _plain_tree(s):
    c, P, L = s["case"], s["page"], s["max_len"]
    q = _padded(s["q"].float() @ s["R32"].T, s["cu"], s["max_n"])
    t = torch.arange(L, device=q.device)
    page = s["table"].long()[:, t // P]                                    # [B, L]

    def cache(name, bits):
        at = (page, slice(None), (t % P).expand_as(page))
        return _dequantize(s["pages"][name + "_codes"][at], s["pages"][name + "_norms"][at], bits)

    k, v = cache("k", c["kb"]), cache("v", c["vb"])                        # [B, L, Hkv, d]
    n = s["cu"][1:] - s["cu"][:-1]
    node = t[None, :] - (s["lens"] - n)[:, None]                           # [B, L]: the drafted token at t
    i = torch.arange(s["max_n"], device=q.device)
    if s["mask"] is None:
        sees = node[:, None, :] <= i[None, :, None]
    else:
        words = _padded(s["mask"], s["cu"], s["max_n"])                    # [B, N, W]
        bit = node.clamp(0, 64 * words.shape[2] - 1)
        w = words.gather(2, (bit // 64)[:, None, :].expand(-1, s["max_n"], -1))
        sees = (node[:, None, :] < 0) | ((w >> (bit % 64)[:, None, :]) & 1).bool()
    allowed = sees & (t[None, None, :] < s["lens"][:, None, None])
    o = _attend(q, k, v, allowed, c["d"] ** -0.5) @ s["R32"]
    return _unpadded(o, s["cu"], s["q"].shape[0]).to(s["q"].dtype)


# ---------------------------------------------------------------------------------------------
# The definitions in 64 bits, one sequence and one head at a time
# ---------------------------------------------------------------------------------------------

def _exact_head(q, k, v, allowed, scale):
    """softmax over the allowed keys of one head: q [N, d], k and v [L, d], allowed [N, L], all float64."""
    out = torch.empty((q.shape[0], v.shape[1]), dtype=torch.float64, device=q.device)
    for r in range(0, q.shape[0], 1024):
        x = torch.where(allowed[r:r + 1024], q[r:r + 1024] @ k.T * scale, -math.inf)
        out[r:r + 1024] = torch.nan_to_num(torch.softmax(x, dim=1)) @ v
    return out


def _exact_rows(codes, norms, bits):
    """Rows of packed codes [n, words] and fp16 norms [n, blocks], bit by bit -> float64 [n, d]."""
    n, nb = norms.shape
    stream = (codes.view(n, nb, bits, 1) >> torch.arange(32, device=codes.device)) & 1
    index = (stream.reshape(n, nb, 32, bits) << torch.arange(bits, device=codes.device)).sum(-1)
    values = torch.from_numpy(_levels(bits).astype(np.float64)).to(codes.device)[index]
    return (values * norms.view(torch.float16).double()[:, :, None]).view(n, -1)


def exact(case, seed):
    global own
    if case["op"] == "tables":
        return None
    was, own = own, False
    s = prepare(case, seed)
    own = was
    a, b = _shape(case)
    group, scale = case["hq"] // case["hkv"], 1.0 / math.sqrt(case["d"])
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    R = torch.from_numpy(_rotation(case["rot"], case["d"])).to(DEV) if case["op"] == "tree" else None
    q0 = k0 = 0
    for n, (nq, nk) in enumerate(zip(a, b)):
        i = torch.arange(nq, device=DEV)[:, None]
        j = torch.arange(nk, device=DEV)[None, :]
        if case["op"] == "prompt" or case["chain"]:
            allowed = j <= i + nk - nq
        else:
            bits = s["mask"][q0:q0 + nq].cpu().tolist()
            tail = [[bool(row[m // 64] >> (m % 64) & 1) for m in range(nq)] for row in bits]
            allowed = torch.ones((nq, nk), dtype=torch.bool, device=DEV)
            allowed[:, nk - nq:] = torch.tensor(tail, device=DEV)
        for h in range(case["hkv"]):
            if case["op"] == "prompt":
                k, v = (s[x][k0:k0 + nk, h].double() for x in "kv")
            else:
                P = case["page"]
                at = s["table"][n].long()[torch.arange(nk, device=DEV) // P]
                off = torch.arange(nk, device=DEV) % P
                k, v = (_exact_rows(s["pages"][x + "_codes"][at, h, off], s["pages"][x + "_norms"][at, h, off],
                                    case[x + "b"]) for x in "kv")
            for g in range(h * group, h * group + group):
                q = s["q"][q0:q0 + nq, g].double()
                if R is None:
                    out[q0:q0 + nq, g] = _exact_head(q, k, v, allowed, scale)
                else:
                    out[q0:q0 + nq, g] = _exact_head(q @ R.T, k, v, allowed, scale) @ R
        q0, k0 = q0 + nq, k0 + nk
    return out
