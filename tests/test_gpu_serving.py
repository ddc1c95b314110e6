"""GPU parity of the serving entry points against oracle/serving.py: page
tables, paged quantization, prompt attention, attention of drafted tokens, and a
run of them together.  Bounds: tests/serving.py."""

import numpy as np
import pytest

import workloads as W
from oracle import quant as oq
from oracle import serving as osv
from tests import parity as P
from tests import serving as S

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def tq():
    import kv_cache_vector_11_b200 as lib
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    return lib


TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def f64(t):
    return t.detach().cpu().double().numpy()


# -- page tables ------------------------------------------------------------------------------

def _tables(tq, ctx, new, page, n_pages, free, table, n_slots, positions=True):
    t = i32(table)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = {"cu_new": torch.full((len(ctx) + 1,), -7, dtype=torch.int32, device="cuda"),
           "total_lens": torch.full((len(ctx),), -7, dtype=torch.int32, device="cuda"),
           "slots": torch.full((n_slots,), -7, dtype=torch.int64, device="cuda"),
           "n_taken": torch.full((1,), -7, dtype=torch.int32, device="cuda")}
    if positions:
        out["positions"] = torch.full((n_slots,), -7, dtype=torch.int32, device="cuda")
    got = tq.page_tables(i32(ctx), i32(new), page, n_pages, i32(free), t, n_slots, out=out, status=status)
    ref = osv.page_tables(ctx, new, page, n_pages, free, np.asarray(table), n_slots)
    got = dict(got, block_table=t)
    for name, v in got.items():
        assert np.array_equal(v.cpu().numpy(), ref[name]), name
    want = (tq.STATUS_NO_PAGES if ref["no_pages"] else 0) | (tq.STATUS_BAD_PAGE if ref["bad_page"] else 0)
    assert int(status) == want
    return ref


@pytest.mark.parametrize("batch,page,ctx_hi,new_hi,pad", [
    (1, 16, 0, 1, 0), (1, 256, 5000, 5000, 3), (7, 16, 100, 40, 0), (33, 64, 0, 300, 129), (512, 16, 300, 2, 5),
    (513, 32, 64, 9, 0), (1500, 16, 40, 20, 1), (3, 65536, 200000, 70000, 0)])
def test_page_tables(tq, batch, page, ctx_hi, new_hi, pad):
    rng = np.random.default_rng(batch * page + new_hi)
    ctx = rng.integers(0, ctx_hi + 1, batch)
    new = rng.integers(0, new_hi + 1, batch)
    held, want = -(-ctx // page), -(-(ctx + new) // page)
    n_pages = int(want.sum()) + 5
    perm = rng.permutation(n_pages)
    table = np.full((batch, int(want.max()) + 1), -1, dtype=np.int32)
    at = 0
    for b in range(batch):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
    ref = _tables(tq, ctx, new, page, n_pages, perm[at:], table, int(new.sum()) + pad)
    assert not ref["no_pages"] and not ref["bad_page"]


def test_page_tables_refusals_on_the_device(tq):
    rng = np.random.default_rng(0)
    full = np.full((6, 3), -1)
    # the free list runs out in the middle; a later request needs no page
    table = full.copy()
    table[4, 0] = 2
    ref = _tables(tq, [0, 0, 0, 0, 5, 0], [16, 20, 33, 1, 3, 0], 16, 9, [0, 1, 3, 4], table, 80)
    assert ref["no_pages"] and ref["total_lens"].tolist() == [16, 20, 0, 0, 8, 0]
    # a row of the table is too short; the slot map is too short for the last one
    _tables(tq, [0, 0, 0, 0, 0, 0], [16, 60, 5, 0, 7, 9], 16, 9, [0, 1, 3, 4, 5, 6, 7, 8], full, 90)
    # no free list, no slots, negative lengths
    _tables(tq, [-3, 16, 0, 0, 0, 0], [-1, 0, -5, 0, 0, 0], 16, 9, [], np.where(full < 0, 1, 1), 4)
    _tables(tq, [0] * 6, [1] * 6, 16, 9, [0, 1, 3, 4, 5, 6, 7], full, 0)
    # pages outside the storage, held and free
    table = full.copy()
    table[0, 0], table[1, 0], table[2, 0] = -1, 9, 8
    ref = _tables(tq, [3, 3, 3, 0, 0, 0], [2, 2, 2, 2, 2, 2], 16, 9, [12, -4, 3], table, 12)
    assert ref["bad_page"] and not ref["no_pages"]
    # lengths whose sum passes 2^31
    _tables(tq, [2**31 - 1, 0], [1, 3], 65536, 9, [1, 2, 3], np.full((2, 40000), 1), 6, positions=False)
    _tables(tq, [0, 0, 0], [2**31 - 1, 2**31 - 1, 3], 16, 9, [1, 2, 3], np.full((3, 4), -1), 6)


def test_page_tables_replayed_with_other_lengths(tq):
    """A captured call reads the lengths of the replay."""
    page, n_slots = 16, 40
    ctx, new, table = i32([0, 0]), i32([0, 0]), i32(np.full((2, 4), -1))
    free = i32([4, 2, 0, 1, 3])
    out = tq.page_tables(ctx, new, page, 5, free, table, n_slots)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tq.page_tables(ctx, new, page, 5, free, table, n_slots, out=out)
    held = np.full((2, 4), -1)
    for c, n in (([0, 0], [17, 20]), ([0, 0], [1, 39]), ([0, 0], [0, 16])):
        ctx.copy_(i32(c)), new.copy_(i32(n)), table.copy_(i32(held))
        g.replay()
        torch.cuda.synchronize()
        ref = osv.page_tables(c, n, page, 5, free.cpu().numpy(), held, n_slots)
        for name, v in dict(out, block_table=table).items():
            assert np.array_equal(v.cpu().numpy(), ref[name]), (name, c, n)


# -- paged quantization -----------------------------------------------------------------------

@pytest.mark.parametrize("kind,d,bits,dtype", [("wht", 64, 4, "bf16"), ("wht", 128, 3, "bf16"), ("haar", 128, 2, "bf16"),
                                               ("wht", 256, 4, "bf16"), ("haar", 256, 3, "bf16"), ("wht", 128, 4, "f32"),
                                               ("haar", 64, 3, "f32"), ("haar", 64, 3, "bf16")])
@pytest.mark.parametrize("n_tokens,heads,page", [(1, 1, 16), (301, 3, 32)])
def test_quantize_paged_equals_quantize_and_scatter(tq, kind, d, bits, dtype, n_tokens, heads, page):
    rng = np.random.default_rng(d + bits + n_tokens)
    rot = tq.Rotation(kind, d, d, W.SEED_ROT)
    c, t = tq.build_codebook(bits)
    x = torch.from_numpy(rng.standard_normal((n_tokens, heads, d))).to("cuda", TYPES[dtype])
    n_pages = -(-n_tokens // page) + 2
    slots = rng.permutation(n_pages * page)[:n_tokens].astype(np.int64)
    bad = n_tokens > 1
    if bad:
        slots[::7] = -1
        slots[3] = n_pages * page              # one past the storage
        slots[4] = 2**40
    w, nb = tq.code_words_per_row(bits, 32, d), d // 32
    codes = torch.full((n_pages, heads, page, w), 0x5A5A5A5A, dtype=torch.int32, device="cuda")
    norms = torch.full((n_pages, heads, page, nb), 0x1234, dtype=torch.int16, device="cuda")
    want_c, want_n = codes.clone(), norms.clone()
    flat = tq.quantize_kv(rot, bits, c, t, x.view(-1, d))
    keep = np.nonzero((slots >= 0) & (slots < n_pages * page))[0]
    pg, off = torch.from_numpy(slots[keep] // page).cuda(), torch.from_numpy(slots[keep] % page).cuda()
    k = torch.from_numpy(keep).cuda()
    want_c[pg, :, off] = flat["codes"].view(n_tokens, heads, w)[k]
    want_n[pg, :, off] = flat["norms"].view(n_tokens, heads, nb)[k]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    tq.quantize_kv_paged(rot, bits, c, t, x, torch.from_numpy(slots).cuda(), codes, norms, page, status=status)
    assert torch.equal(codes, want_c) and torch.equal(norms, want_n)
    assert int(status) == (tq.STATUS_BAD_PAGE if bad else 0)


# -- prompt attention -------------------------------------------------------------------------

def _prompt(tq, lens_q, lens_k, hq, hk, d, dtype, seed=0, pad=0, amp=1.0, fused=False, scale=0.0, edit=None):
    rng = np.random.default_rng(seed + d + sum(lens_q))
    cu_q, cu_k = np.cumsum([0] + list(lens_q)), np.cumsum([0] + list(lens_k))
    nq, nk = int(cu_q[-1]), int(cu_k[-1])

    def rows(n, h):
        return torch.from_numpy(rng.standard_normal((n, h, d)) * amp).to(TYPES[dtype])
    if fused:
        assert lens_q == lens_k
        qkv = rows(nq + pad, hq + 2 * hk).cuda()
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    else:
        q, k, v = rows(nq + pad, hq).cuda(), rows(nk + pad, hk).cuda(), rows(nk + pad, hk).cuda()
    if edit is not None:
        edit(q, k, v)
    out = torch.full((nq + pad, hq, d), 7.0, dtype=TYPES[dtype], device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    same = list(lens_q) == list(lens_k)
    got = tq.prompt_attention(q, k, v, i32(cu_q), None if same else i32(cu_k), out=out, scale=scale, status=status)
    assert got is out and int(status) == 0
    ref, absum, sq = osv.prompt_attention(f64(q)[:nq], f64(k)[:nk], f64(v)[:nk], cu_q, cu_k, scale or None)
    g = f64(out)
    assert np.all(g[nq:] == 7.0), "rows behind the last sequence were written"
    g = g[:nq]
    assert np.array_equal(np.isnan(g), np.isnan(ref)) and np.array_equal(np.isinf(g), np.isinf(ref))
    fine = np.isfinite(ref)
    assert np.array_equal(np.sign(g[np.isinf(ref)]), np.sign(ref[np.isinf(ref)]))
    bound = S.prompt_bound(ref, absum, sq, dtype, d, max(lens_k))
    with np.errstate(invalid="ignore"):
        over = np.abs(g - ref) / bound
    assert over[fine].size == 0 or np.max(over[fine]) <= 1.0, f"{np.max(over[fine]):.3f} of the bound"
    return g, ref


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hq,hk", [(4, 2), (3, 1), (2, 2)])
def test_prompt_lengths(tq, d, dtype, hq, hk):
    lens = [1, 127, 0, 128, 129, 2, 300]
    _prompt(tq, lens, lens, hq, hk, d, dtype, pad=5)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_prompt_chunks_and_empty_rows(tq, d):
    # fewer queries than keys, equal, more (rows that attend nothing), none at all
    _prompt(tq, [1, 5, 130, 70, 3, 0, 9], [400, 261, 130, 3, 0, 50, 137], 4, 2, d, "bf16")


def test_prompt_single_queries_and_groups(tq):
    _prompt(tq, [1] * 40, [1 + 13 * i for i in range(40)], 8, 1, 128, "bf16")
    _prompt(tq, [1], [1], 1, 1, 64, "f16")
    _prompt(tq, [33], [33], 14, 2, 64, "f16")


def test_prompt_long(tq):
    _prompt(tq, [1500], [1500], 2, 1, 128, "bf16")
    _prompt(tq, [700], [1333], 2, 2, 64, "f16")


def test_prompt_strided_rows(tq):
    _prompt(tq, [200, 77], [200, 77], 4, 2, 128, "bf16", fused=True, pad=3)
    _prompt(tq, [65, 1], [65, 1], 4, 4, 64, "f16", fused=True)


def test_prompt_large_scores_and_scale(tq):
    _prompt(tq, [150, 300], [150, 300], 2, 1, 128, "bf16", amp=6.0)
    _prompt(tq, [150], [150], 2, 1, 128, "bf16", scale=0.5)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_prompt_masked_values_do_not_leak(tq, d):
    """NaN and infinities at keys that a query may not attend (later keys of its
    sequence, other sequences, padding) leave its output alone; the queries that
    attend them get what the arithmetic gives."""
    lens = [140, 60, 200]

    def edit(q, k, v):
        v[100, 0, 3] = float("nan")            # seen by queries 100 .. 139 of the first sequence
        v[130, 0, 5] = float("inf")
        v[131, 0, 5] = float("-inf")
        v[139, 0, d - 1] = float("-inf")
        v[200:, 0, :] = float("inf")           # the whole third sequence
        v[200:230, 0, :] = 1.0
        v[-2:] = float("nan")                  # padding
        k[-2:] = float("nan")
        q[-2:] = float("nan")
    g, ref = _prompt(tq, lens, lens, 2, 1, d, "bf16", pad=2, edit=edit)
    assert np.isfinite(ref[:100]).all() and np.isfinite(ref[140:230]).all()


def test_prompt_masked_keys_do_not_leak(tq):
    def edit(q, k, v):
        k[150, 0, 0] = float("nan")
        k[170, 0, :] = float("inf")
    _prompt(tq, [160, 40], [160, 40], 2, 1, 128, "bf16", edit=edit)


def test_prompt_offsets_outside_the_arrays_are_clamped(tq):
    q = torch.randn((50, 2, 64), device="cuda").half()
    out = torch.full_like(q, 7.0)
    tq.prompt_attention(q, q, q, i32([-5, 30, 90]), out=out)
    ok, _, _ = osv.prompt_attention(f64(q), f64(q), f64(q), [0, 30, 50], [0, 30, 50])
    assert np.abs(f64(out) - ok).max() < 0.01
    tq.prompt_attention(q, q, q, i32([0, 40, 10, 50]), out=out)      # decreasing: any output, no fault
    torch.cuda.synchronize()


def test_prompt_graph_stream_and_lengths_of_the_replay(tq):
    q, k, v = (torch.randn((300, h, 128), device="cuda").bfloat16() for h in (4, 2, 2))
    cu = i32([0, 100, 300])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(q)
    tq.prompt_attention(q, k, v, cu, out=out, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    replay = torch.zeros_like(q)
    with torch.cuda.graph(g):
        tq.prompt_attention(q, k, v, cu, out=replay)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, replay)
    cu.copy_(i32([0, 260, 290]))
    g.replay()
    assert torch.equal(replay[:290], tq.prompt_attention(q, k, v, cu)[:290])


@pytest.mark.parametrize("batch", [33, 128, 129, 400, 900])
def test_prompt_many_sequences(tq, batch):
    rng = np.random.default_rng(batch)
    lens = rng.integers(0, 9, batch).tolist()
    lens[batch // 2] = 300
    _prompt(tq, lens, lens, 2, 1, 64, "bf16", pad=4)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_prompt_runs_agree_bit_for_bit(tq, d):
    """Every wait of the kernel names a phase of its barrier by parity only; a wait
    that answers a phase too early shows as an output that changes from run to run
    (with other work in between, so that the timing changes)."""
    g = torch.Generator(device="cuda").manual_seed(d)
    for lens, hq, hk in (([1500], 2, 1), ([1, 127, 0, 128, 129, 2, 300], 3, 1), ([700, 40], 2, 2)):
        n = sum(lens)
        q, k, v = (torch.randn((n, h, d), generator=g, device="cuda").bfloat16() for h in (hq, hk, hk))
        cu = i32(np.cumsum([0] + lens))
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        first = tq.prompt_attention(q, k, v, cu, status=status)
        for _ in range(25):
            torch.randn(1 << 20, device="cuda")
            assert torch.equal(tq.prompt_attention(q, k, v, cu, status=status), first)
        assert int(status) == 0


def test_prompt_and_tree_on_two_streams_at_once(tq):
    rng = np.random.default_rng(11)
    d, page = 128, 32
    table, n_pages = S.page_tables_for(rng, [2000, 700], page)
    pages = S.cache_to(S.random_cache(rng, n_pages, 2, page, d, 4, 3), "cuda")
    rot = tq.Rotation("wht", d, d, W.SEED_ROT)
    kc, vc = tq.build_codebook(4)[0], tq.build_codebook(3)[0]
    q, k = (torch.randn((900, h, d), device="cuda").bfloat16() for h in (8, 2))
    cu_p, cu_t, lens, tab = i32([0, 800, 900]), i32([0, 40, 60]), i32([2000, 700]), i32(table)

    def tree(ws, stream=None):
        return tq.tree_attention(rot, 4, 3, kc, vc, q[:60], cu_t, lens, pages, tab, page, 40, 2000, workspace=ws, stream=stream)
    need = tq.tree_workspace_size(2, 60, 40, 8, 2, 2000, d)
    ws = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(2)]
    want_p, want_t = tq.prompt_attention(q, k, k, cu_p), tree(ws[0])
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        with torch.cuda.stream(streams[0]):
            got.append((tq.prompt_attention(q, k, k, cu_p), want_p))
        for i in (0, 1):
            with torch.cuda.stream(streams[1 + i]):
                got.append((tree(ws[i]), want_t))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in got)


def test_memory_of_a_call_is_kept_for_the_stream_it_runs_on(tq):
    """stream= another than the current one, workspace and outputs left to the call: what is allocated
    after the call, while that stream is still busy, does not get its memory."""
    rng = np.random.default_rng(12)
    d, page = 128, 32
    table, n_pages = S.page_tables_for(rng, [2000, 700], page)
    pages = S.cache_to(S.random_cache(rng, n_pages, 2, page, d, 4, 3), "cuda")
    rot = tq.Rotation("wht", d, d, W.SEED_ROT)
    kc, vc = tq.build_codebook(4)[0], tq.build_codebook(3)[0]
    q = torch.randn((60, 8, d), device="cuda").bfloat16()
    cu, lens, tab = i32([0, 40, 60]), i32([2000, 700]), i32(table)
    need = tq.tree_workspace_size(2, 60, 40, 8, 2, 2000, d)

    def tree(**kw):
        return tq.tree_attention(rot, 4, 3, kc, vc, q, cu, lens, pages, tab, page, 40, 2000, **kw)
    want = tree()
    side, x = torch.cuda.Stream(), torch.randn((4096, 4096), device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            x = x @ x * 1e-2
    got = tree(stream=side)
    later = [torch.full((need,), 0x3C, dtype=torch.uint8, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    assert torch.equal(got, want) and all(bool((t == 0x3C).all()) for t in later)


# -- drafted tokens over the cache ------------------------------------------------------------

def _tree(tq, nodes, lens, hq, hk, d, kb, vb, page, dtype="bf16", kind="wht", chain=False, seed=0, masks=None, scale=0.0,
          amp=1.0, pad=0, max_nodes=None, max_len=None, edit=None, l2=True):
    rng = np.random.default_rng(seed + d + sum(nodes) + sum(lens))
    table, n_pages = S.page_tables_for(rng, lens, page)
    pages = S.random_cache(rng, n_pages, hk, page, d, kb, vb)
    cu = np.cumsum([0] + list(nodes))
    rows = int(cu[-1])
    q = torch.from_numpy(rng.standard_normal((rows + pad, hq, d)) * amp).to("cuda", TYPES[dtype])
    if pad:
        q[rows:] = float("nan")
    max_nodes = max_nodes or max(max(nodes), 1)
    words = -(-max_nodes // 64)
    if not chain and masks is None:
        masks = [S.random_tree(rng, n) for n in nodes]
    mask = None
    if not chain:
        mask = np.zeros((rows + pad, words), dtype=np.int64)
        mask[:rows] = S.mask_words(masks, words)
        mask = torch.from_numpy(mask).cuda()
    if edit is not None:
        edit(pages, table)
    kc, vc = tq.build_codebook(kb)[0], tq.build_codebook(vb)[0]
    rot = tq.Rotation(kind, d, d, W.SEED_ROT)
    out = torch.full((rows + pad, hq, d), 7.0, dtype=TYPES[dtype], device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    max_len = max_len if max_len is not None else max(lens)
    need = tq.tree_workspace_size(len(lens), rows + pad, max_nodes, hq, hk, max_len, d)
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")     # NaN everywhere
    tq.tree_attention(rot, kb, vb, kc, vc, q, i32(cu), i32(lens), S.cache_to(pages, "cuda"), i32(table), page, max_nodes,
                      max_len, tree_mask=mask, scale=scale, out=out, workspace=ws[:need], status=status)
    torch.cuda.synchronize()
    assert int(status) == 0 and bool((ws[need:] == 0xFF).all()), "wrote past the workspace"
    q64 = f64(q)[:rows]
    ref, absum, sq = osv.tree_attention(q64, P.oracle_rotation(kind, d, W.SEED_ROT), cu, lens, masks if not chain else None,
                                        pages, table, page, kc, vc, kb, vb, scale or None)
    g = f64(out)
    assert np.all(g[rows:] == 7.0), "padding rows were written"
    g = g[:rows]
    bad = ~np.isfinite(ref).all(axis=-1)
    assert np.array_equal(bad, ~np.isfinite(g).all(axis=-1))
    if (~bad).any():
        err = np.linalg.norm(g - ref, axis=-1)[~bad]
        bound = S.tree_bound(ref, absum, sq, dtype, d, max(lens))[~bad]
        assert np.max(err / bound) <= 1.0, f"{np.max(err / bound):.3f} of the bound"
        if l2:
            nrm = np.linalg.norm(ref, axis=-1)[~bad]
            seen = nrm > 0
            rel = err[seen] / nrm[seen]
            assert rel.size == 0 or rel.max() <= P.DECODE_TOL + S.HALF_STEP[dtype]
    return g, ref


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kb,vb", [(4, 3), (3, 2), (2, 4)])
@pytest.mark.parametrize("kind", ["wht", "haar"])
def test_tree_types_and_bits(tq, d, kb, vb, kind):
    _tree(tq, [5, 1, 17], [300, 40, 129], 4, 2, d, kb, vb, 16, kind=kind)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("chain", [False, True])
def test_tree_query_types(tq, dtype, chain):
    _tree(tq, [7, 3], [200, 65], 8, 2, 128, 4, 3, 32, dtype=dtype, chain=chain, pad=3)


@pytest.mark.parametrize("hq,hk", [(1, 1), (2, 2), (7, 1), (8, 1), (9, 3), (16, 1), (40, 2)])
def test_tree_head_groups(tq, hq, hk):
    _tree(tq, [9, 20], [150, 270], hq, hk, 64, 4, 4, 64)


@pytest.mark.parametrize("n", [1, 16, 63, 64, 65, 128, 200, 256])
def test_tree_node_counts(tq, n):
    _tree(tq, [n, 2], [n + 77, 140], 4, 1, 64, 3, 3, 16)


@pytest.mark.parametrize("page", [16, 32, 128, 256, 1024])
def test_tree_pages_and_lengths(tq, page):
    lens = [1, 15, 16, 17, 127, 128, 129, 255, 256, 257, 511, 700, 0]
    nodes = [min(2, x) for x in lens]
    _tree(tq, nodes, lens, 4, 2, 128, 4, 3, page)
    _tree(tq, [1] * 12 + [0], lens, 4, 2, 128, 4, 3, page, chain=True)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kind", ["wht", "haar"])
def test_tree_more_rows_than_one_merge_wave(tq, d, kind):
    """1896 rows: merged 32 to a block, fewer than 8 rows an SM 8 to a block."""
    _tree(tq, [200, 37], [400, 90], 8, 2, d, 4, 3, 32, kind=kind, pad=1)


def test_tree_long_and_ragged(tq):
    _tree(tq, [4, 1, 30], [5000, 3, 1777], 4, 2, 128, 4, 3, 64)
    _tree(tq, [3], [20000], 2, 1, 64, 2, 2, 256)


def test_tree_many_requests(tq):
    rng = np.random.default_rng(1)
    lens = rng.integers(1, 400, 150).tolist()
    _tree(tq, [1] * 150, lens, 2, 2, 64, 4, 4, 32, chain=True)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kb,vb", [(4, 3), (3, 4), (2, 2), (4, 4), (3, 3), (2, 4)])
@pytest.mark.parametrize("dtype,kind", [("bf16", "wht"), ("f32", "haar")])
def test_tree_few_rows(tq, d, kb, vb, dtype, kind):
    """At most 8 rows share a key tile: a kernel of its own."""
    _tree(tq, [1, 2, 0, 1, 2], [300, 17, 5, 1, 1999], 8, 2, d, kb, vb, 16, dtype=dtype, kind=kind)
    _tree(tq, [1] * 6, [128, 16, 15, 129, 3000, 7], 7, 1, d, kb, vb, 64, chain=True, dtype=dtype, pad=2)


def test_tree_few_rows_masks_and_bad_norms(tq):
    masks = [[0b00001, 0, 0b00100, 0b11111, 0b00011], [0b01, 0b10]]
    g, ref = _tree(tq, [5, 2], [5, 60], 1, 1, 128, 4, 3, 16, masks=masks)
    assert np.all(g[1] == 0)

    def edit(pages, table):
        page = pages["v_norms"].shape[2]
        for name, t, what in (("k_norms", 61, "nan"), ("v_norms", 30, "inf")):
            pages[name][table[0, t // page], 0, t % page, 2] = np.float16(what)
            pages[name][table[0, 63 // page], 1, 64 % page:] = np.float16("nan")
    g, ref = _tree(tq, [4], [64], 2, 2, 128, 4, 3, 32, masks=[[0b0001, 0b0011, 0b0101, 0b1011]], edit=edit)
    assert np.isnan(g).all()          # token 30 of head 0 and the second page of head 1 are every node's

    def drafted(pages, table):
        page = pages["v_norms"].shape[2]
        pages["v_norms"][table[0, 61 // page], :, 61 % page, 0] = np.float16("inf")
    g, ref = _tree(tq, [4], [64], 2, 2, 64, 3, 2, 16, masks=[[0b0001, 0b0011, 0b0101, 0b1011]], edit=drafted)
    assert np.isfinite(g[[0, 2]]).all() and not np.isfinite(g[[1, 3]]).any()


def test_tree_few_rows_long_and_many(tq):
    rng = np.random.default_rng(8)
    lens = [int(x) for x in rng.integers(0, 700, 300)] + [20000]
    _tree(tq, [min(1, x) for x in lens], lens, 4, 1, 64, 4, 3, 64, chain=True)


def test_tree_more_requests_than_a_search_step(tq):
    rng = np.random.default_rng(5)
    nodes = rng.integers(0, 3, 1100).tolist()
    lens = [int(x) + n for x, n in zip(rng.integers(0, 40, 1100), nodes)]
    _tree(tq, nodes, lens, 2, 1, 64, 3, 2, 16, chain=True, pad=2)


@pytest.mark.parametrize("d,hq,hk,nodes", [(128, 8, 2, [40, 3, 64, 1, 33]), (64, 16, 1, [17, 8, 9, 256, 1]), (256, 4, 1, [70, 2, 32, 33, 1])])
def test_tree_row_tiles_of_every_filling(tq, d, hq, hk, nodes):
    # requests with one, two and more row tiles side by side, some of one row
    lens = [n + x for n, x in zip(nodes, (500, 0, 130, 64, 1000))]
    _tree(tq, nodes, lens, hq, hk, d, 4, 3, 32)


@pytest.mark.parametrize("bits", [2, 3, 4])
def test_tree_any_ascending_centroids(tq, bits):
    """The library's codebooks are symmetric; the call asks for ascending ones only."""
    rng = np.random.default_rng(bits)
    d, page, n = 128, 16, 90
    c = np.sort(rng.uniform(-0.5, 0.6, 1 << bits)).astype(np.float16).astype(np.float32)
    table, n_pages = S.page_tables_for(rng, [n], page)
    pages = S.random_cache(rng, n_pages, 1, page, d, bits, bits)
    q = torch.randn((3, 4, d), device="cuda").half()
    rot = tq.Rotation("wht", d, d, W.SEED_ROT)
    out = tq.tree_attention(rot, bits, bits, c, c, q, i32([0, 3]), i32([n]), S.cache_to(pages, "cuda"), i32(table), page, 3, n)
    ref, absum, sq = osv.tree_attention(f64(q), P.oracle_rotation("wht", d, W.SEED_ROT), [0, 3], [n], None, pages, table, page,
                                        c, c, bits, bits)
    assert np.all(np.linalg.norm(f64(out) - ref, axis=-1) <= S.tree_bound(ref, absum, sq, "f16", d, n))


@pytest.mark.parametrize("amp", [1e-12, 1e12])
def test_tree_query_magnitudes(tq, amp):
    """Rows of any fp32 magnitude: the products see them scaled to one."""
    _tree(tq, [5], [150], 4, 2, 128, 4, 3, 16, dtype="f32", amp=amp, scale=0.1 / amp, l2=False)


def test_tree_masks_that_leave_rows_empty(tq):
    # no cache before the nodes, and rows whose mask is empty, is not the node itself, or is full
    masks = [[0b0001, 0, 0b1000, 0b1111], [0, 0b01]]
    g, ref = _tree(tq, [4, 2], [4, 60], 4, 2, 128, 4, 3, 16, masks=masks)
    assert np.all(g[1] == 0) and np.all(ref[1] == 0)
    # bits past the nodes do not count
    _tree(tq, [2], [40], 2, 1, 64, 4, 4, 16, masks=[[(1 << 64) - 1, 0b10 | 1 << 63]], max_nodes=64)


def test_tree_more_nodes_than_tokens(tq):
    # nodes of which the first are not cached: they have no token to attend
    rng = np.random.default_rng(2)
    d, page = 64, 16
    table, n_pages = S.page_tables_for(rng, [3], page)
    pages = S.random_cache(rng, n_pages, 1, page, d, 4, 4)
    kc = tq.build_codebook(4)[0]
    rot = tq.Rotation("wht", d, d, W.SEED_ROT)
    q = torch.randn((5, 1, d), device="cuda").bfloat16()
    out = tq.tree_attention(rot, 4, 4, kc, kc, q, i32([0, 5]), i32([3]), S.cache_to(pages, "cuda"), i32(table), page, 5, 3)
    # node i is token i - 2: nodes 0 and 1 attend nothing, nodes 2 .. 4 the tokens 0 .. i - 2
    ref, _, _ = osv.tree_attention(f64(q)[2:], P.oracle_rotation("wht", d, W.SEED_ROT), [0, 3], [3], None, pages, table,
                                   page, kc, kc, 4, 4)
    g = f64(out)
    assert np.all(g[:2] == 0)
    assert np.linalg.norm(g[2:] - ref) <= (P.DECODE_TOL + 2.0**-8) * np.linalg.norm(ref)


def test_tree_larger_limits_than_lengths(tq):
    _tree(tq, [3, 1], [100, 30], 4, 2, 64, 4, 3, 32, max_nodes=200, max_len=100)


def test_tree_scale_and_peaked_scores(tq):
    _tree(tq, [5], [300], 4, 2, 128, 4, 3, 16, scale=0.25)
    _tree(tq, [5], [300], 4, 2, 128, 4, 3, 16, amp=12.0, l2=False)


def test_tree_nonfinite_norms_stay_with_their_readers(tq):
    """A drafted token with a NaN norm reaches only the nodes that attend it; what
    lies in a page behind the last token reaches none."""
    masks = [[0b0001, 0b0011, 0b0101, 0b1011]]

    def edit(pages, table):
        page = pages["v_norms"].shape[2]
        for name in ("k_norms", "v_norms"):
            t = 61                                    # node 1 of tokens 60 .. 63
            pages[name][table[0, t // page], :, t % page, 1] = np.float16("nan" if name == "k_norms" else "inf")
    g, ref = _tree(tq, [4], [64], 4, 2, 128, 4, 3, 16, masks=masks, edit=edit)
    assert np.isfinite(g[[0, 2]]).all() and not np.isfinite(g[[1, 3]]).any()

    def behind(pages, table):
        page = pages["v_norms"].shape[2]
        for name in ("k_norms", "v_norms"):
            pages[name][table[0, 50 // page], :, 50 % page:] = np.float16("nan")
    _tree(tq, [2], [50], 2, 2, 64, 4, 4, 64, edit=behind)


def test_tree_pages_outside_the_storage_are_clamped(tq):
    rng = np.random.default_rng(3)
    pages = S.cache_to(S.random_cache(rng, 4, 1, 16, 64, 4, 4), "cuda")
    kc = tq.build_codebook(4)[0]
    rot = tq.Rotation("wht", 64, 64, W.SEED_ROT)
    q = torch.randn((2, 1, 64), device="cuda").bfloat16()
    a, b = (tq.tree_attention(rot, 4, 4, kc, kc, q, i32([0, 2]), i32([60]), pages, i32([t]), 16, 2, 64)
            for t in ([-9, 2**31 - 1, 1, 99], [0, 3, 1, 3]))
    assert torch.equal(a, b)
    # lengths past max_len, offsets past the rows
    c, e = (tq.tree_attention(rot, 4, 4, kc, kc, q, i32(cu), i32([n]), pages, i32([[0, 3, 1, 3]]), 16, 2, 64)
            for cu, n in (([0, 2], 64), ([-4, 90], 5000)))
    assert torch.equal(c, e)


def test_tree_captured_twice_and_replayed(tq):
    """Two captured calls with workspaces of their own, replayed on two streams with other lengths."""
    rng = np.random.default_rng(4)
    lens0, page, d = [900, 300], 32, 128
    table, n_pages = S.page_tables_for(rng, [1024, 1024], page)
    pages = S.cache_to(S.random_cache(rng, n_pages, 2, page, d, 4, 3), "cuda")
    kc, vc = tq.build_codebook(4)[0], tq.build_codebook(3)[0]
    rot = tq.Rotation("wht", d, d, W.SEED_ROT)
    q = torch.randn((10, 8, d), device="cuda").bfloat16()
    cu, lens = i32([0, 4, 10]), i32(lens0)

    def call(**kw):
        return tq.tree_attention(rot, 4, 3, kc, vc, q, cu, lens, pages, i32_table, page, 8, 1024, **kw)
    i32_table = i32(table)
    call()
    graphs, outs = [], []
    for _ in range(2):
        ws = torch.empty(tq.tree_workspace_size(2, 10, 8, 8, 2, 1024, d), dtype=torch.uint8, device="cuda")
        out = torch.zeros_like(q)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(out=out, workspace=ws)
        graphs.append((g, ws))
        outs.append(out)
    for new in ([900, 300], [17, 1024], [6, 4]):
        lens.copy_(i32(new))
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        for _ in range(3):
            for (g, _), s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        want = call()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want), new


@pytest.mark.parametrize("d,hq", [(128, 8), (128, 4), (256, 8), (64, 8)])
def test_tree_runs_agree_bit_for_bit(tq, d, hq):
    rng = np.random.default_rng(d + hq)
    page, lens = 64, [3000, 129, 900]
    table, n_pages = S.page_tables_for(rng, lens, page)
    pages = S.cache_to(S.random_cache(rng, n_pages, 2, page, d, 4, 3), "cuda")
    kc, vc = tq.build_codebook(4)[0], tq.build_codebook(3)[0]
    rot = tq.Rotation("wht", d, d, W.SEED_ROT)
    q = torch.randn((95, hq, d), device="cuda").bfloat16()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(tq.tree_workspace_size(3, 95, 64, hq, 2, 3000, d), dtype=torch.uint8, device="cuda")

    def call():
        return tq.tree_attention(rot, 4, 3, kc, vc, q, i32([0, 30, 31, 95]), i32(lens), pages, i32(table), page, 64, 3000,
                                 workspace=ws, status=status)
    first = call()
    for _ in range(25):
        torch.randn(1 << 20, device="cuda")
        assert torch.equal(call(), first)
    assert int(status) == 0


def test_tree_is_deterministic(tq):
    a = _tree(tq, [20, 3], [3000, 2000], 8, 2, 128, 4, 3, 64)[0]
    b = _tree(tq, [20, 3], [3000, 2000], 8, 2, 128, 4, 3, 64)[0]
    assert np.array_equal(a, b)


# -- together ---------------------------------------------------------------------------------

def test_prompt_draft_accept_and_decode(tq):
    """A serving run: admit prompts, attend and store them, draft a tree, accept a
    branch by storing its rows again, take a single-token step; and the same
    cache read by decode_append_paged."""
    rng = np.random.default_rng(9)
    d, hq, hk, page, kb, vb = 128, 8, 2, 16, 4, 3
    prompts = [45, 130]
    batch, n_pages, max_pages = 2, 40, 16
    rot = tq.Rotation("wht", d, d, W.SEED_ROT)
    rot64 = P.oracle_rotation("wht", d, W.SEED_ROT)
    (kc, kt), (vc, vt) = tq.build_codebook(kb), tq.build_codebook(vb)
    pages = S.cache_to(S.random_cache(rng, n_pages, hk, page, d, kb, vb), "cuda")
    table = i32(np.full((batch, max_pages), -1))
    free = i32(rng.permutation(n_pages))

    def rows(n, h):
        return torch.from_numpy(rng.standard_normal((n, h, d))).to("cuda", torch.bfloat16)

    def store(k, v, slots):
        tq.quantize_kv_paged(rot, kb, kc, kt, k, slots, pages["k_codes"], pages["k_norms"], page)
        tq.quantize_kv_paged(rot, vb, vc, vt, v, slots, pages["v_codes"], pages["v_norms"], page)

    # prompts
    n = sum(prompts)
    q, k, v = rows(n, hq), rows(n, hk), rows(n, hk)
    t = tq.page_tables(i32([0, 0]), i32(prompts), page, n_pages, free, table, n)
    out = tq.prompt_attention(q, k, v, t["cu_new"])
    store(k, v, t["slots"])
    ref, absum, sq = osv.prompt_attention(f64(q), f64(k), f64(v), t["cu_new"].cpu().numpy(), t["cu_new"].cpu().numpy())
    assert np.all(np.abs(f64(out) - ref) <= S.prompt_bound(ref, absum, sq, "bf16", d, max(prompts)))
    free = free[int(t["n_taken"]):].contiguous()

    def cache_np():
        return {x: (p.cpu().numpy().view(np.uint32) if "codes" in x else p.cpu().numpy().view(np.float16))
                for x, p in pages.items()}

    def check(got, q, cu, lens, masks):
        ref, absum, sq = osv.tree_attention(f64(q), rot64, cu, lens, masks, cache_np(), table.cpu().numpy(), page, kc, vc,
                                            kb, vb)
        assert np.all(np.linalg.norm(f64(got) - ref, axis=-1) <= S.tree_bound(ref, absum, sq, "bf16", d, max(lens)))

    # drafts
    drafts = [6, 3]
    masks = [S.random_tree(rng, x) for x in drafts]
    masks[0] = [0b1, 0b11, 0b101, 0b1011, 0b10101, 0b110101]        # 0 -> 1 -> 3, 0 -> 2 -> 4 -> 5
    q, k, v = rows(9, hq), rows(9, hk), rows(9, hk)
    t = tq.page_tables(t["total_lens"], i32(drafts), page, n_pages, free, table, 12)     # 3 rows of padding
    pad = torch.zeros((3, hk, d), dtype=torch.bfloat16, device="cuda")
    store(torch.cat([k, pad]), torch.cat([v, pad]), t["slots"])
    free = free[int(t["n_taken"]):].contiguous()
    got = tq.tree_attention(rot, kb, vb, kc, vc, q, t["cu_new"], t["total_lens"], pages, table, page, 6, 256,
                            tree_mask=torch.from_numpy(S.mask_words(masks, 1)).cuda())
    check(got, q, t["cu_new"].cpu().numpy(), [x + y for x, y in zip(prompts, drafts)], masks)

    # accept the branch 0, 2, 4, 5 of request 0 and node 0 of request 1: their rows
    # again, at the slots that follow the prompt
    accepted = [[0, 2, 4, 5], [0]]
    slots = torch.full((9,), -1, dtype=torch.int64, device="cuda")
    for path, start in zip(accepted, (0, 6)):
        for i, node in enumerate(path):
            slots[start + node] = t["slots"][start + i]
    store(k, v, slots)
    lens = [x + len(a) for x, a in zip(prompts, accepted)]

    # one token each
    q, k1, v1 = rows(2, hq), rows(2, hk), rows(2, hk)
    t = tq.page_tables(i32(lens), i32([1, 1]), page, n_pages, free, table, 2)
    store(k1, v1, t["slots"])
    got = tq.tree_attention(rot, kb, vb, kc, vc, q, t["cu_new"], t["total_lens"], pages, table, page, 1, 256)
    check(got, q, [0, 1, 2], [x + 1 for x in lens], None)

    # the accepted branch attends like a chain of the same tokens
    flat = oq.quantize(f64(k)[2, 0][None], rot64, kc, kt, kb, 32)["words"][0]
    at = prompts[0] + 1                                              # node 2 is the second accepted token
    pg = int(table[0, at // page])
    assert np.array_equal(cache_np()["k_codes"][pg, 0, at % page], flat)

    # the decode step of equal lengths reads the same cache (request 0 alone)
    ctx = lens[0] + 1
    one = tq.decode_append_paged(rot, kb, vb, (kc, kt), (vc, vt), q[:1], k1[:1], v1[:1], pages, table[:1].contiguous(), hk,
                                 ctx, page)
    assert np.linalg.norm(f64(one)[0] - f64(got)[0]) <= (2 * P.DECODE_TOL + 2.0**-8) * np.linalg.norm(f64(one)[0])
