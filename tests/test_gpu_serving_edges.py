"""GPU tests of the serving entry points at the edges of what they accept: inputs
that are not finite, more nodes or tokens than a call allows for, the largest and
smallest magnitudes, calls on another stream.  Bounds: tests/serving.py."""

import numpy as np
import pytest

import workloads as W
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


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def f64(t):
    return t.detach().cpu().double().numpy()


class Tree:
    """Inputs of a tree_attention call over a random cache; ``call`` makes it."""

    def __init__(self, tq, nodes, lens, hq, hk, d, page=16, kb=4, vb=3, kind="wht", dtype=torch.bfloat16, seed=0,
                 norms=None):
        rng = np.random.default_rng(seed + d + sum(nodes) + sum(lens))
        self.tq, self.page, self.kb, self.vb, self.kind, self.d = tq, page, kb, vb, kind, d
        self.lens, self.cu = list(lens), np.cumsum([0] + list(nodes))
        self.rows, self.hq, self.hk = int(self.cu[-1]), hq, hk
        self.table, n_pages = S.page_tables_for(rng, lens, page)
        self.cache = S.random_cache(rng, n_pages, hk, page, d, kb, vb)
        if norms is not None:
            for name in ("k_norms", "v_norms"):
                self.cache[name] = (self.cache[name].astype(np.float64) * norms).astype(np.float16)
        self.pages = S.cache_to(self.cache, "cuda")
        self.q = torch.from_numpy(rng.standard_normal((self.rows, hq, d))).to("cuda", dtype)
        self.kc, self.vc = tq.build_codebook(kb)[0], tq.build_codebook(vb)[0]
        self.rot = tq.Rotation(kind, d, d, W.SEED_ROT)

    def call(self, max_nodes, max_len=None, q=None, cu=None, lens=None, mask=None, out=None, **kw):
        q = self.q if q is None else q
        out = torch.full_like(q, 7.0) if out is None else out
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.tq.tree_attention(self.rot, self.kb, self.vb, self.kc, self.vc, q, i32(self.cu if cu is None else cu),
                               i32(self.lens if lens is None else lens), self.pages, i32(self.table), self.page,
                               max_nodes, max(self.lens) if max_len is None else max_len, tree_mask=mask, out=out,
                               status=status, **kw)
        torch.cuda.synchronize()
        return out, int(status)

    def reference(self, q=None, masks=None, scale=None):
        return osv.tree_attention(f64(self.q if q is None else q), P.oracle_rotation(self.kind, self.d, W.SEED_ROT), self.cu,
                                  self.lens, masks, self.cache, self.table, self.page, self.kc, self.vc, self.kb, self.vb,
                                  scale)


# The four kernels by (nodes of a request, query heads, KV heads, head_dim): few rows
# (single tokens, 8 rows), one row tile, two row tiles, wide heads.
KERNELS = {"single": (1, 4, 2, 128), "few": (4, 4, 2, 64), "one tile": (9, 8, 2, 128), "two tiles": (70, 8, 2, 64),
           "wide": (9, 8, 2, 256)}


# -- queries that are not finite --------------------------------------------------------------

@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("length", [0, 40, 90, 700])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_tree_nonfinite_queries_stay_in_their_rows(tq, kernel, length, value):
    """A NaN or infinite query makes its own row NaN, in every kernel and at every
    length (its scores are NaN or of both signs), and leaves the others as they were."""
    n, hq, hk, d = KERNELS[kernel]
    lens = [n + length, n + 3]
    t = Tree(tq, [n, n], lens, hq, hk, d)
    want, _ = t.call(n)
    q = t.q.clone()
    q[n - 1, 1, d - 1] = value
    q[n, hq - 1, 0] = value
    got, status = t.call(n, q=q)
    hit = torch.zeros((t.rows, hq), dtype=torch.bool, device="cuda")
    hit[n - 1, 1] = hit[n, hq - 1] = True
    assert status == 0 and bool(torch.isfinite(want).all())
    assert bool(torch.isnan(got[hit]).all()), "a row of NaN scores came out finite"
    assert torch.equal(got[~hit], want[~hit])


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_prompt_nonfinite_queries_stay_in_their_rows(tq, d, value):
    g = torch.Generator(device="cuda").manual_seed(d)
    lens = [1, 40, 300]
    q, k, v = (torch.randn((sum(lens), h, d), generator=g, device="cuda").bfloat16() for h in (4, 2, 2))
    cu = i32(np.cumsum([0] + lens))
    want = tq.prompt_attention(q, k, v, cu)
    hit = torch.zeros((sum(lens), 4), dtype=torch.bool, device="cuda")
    for row, head in ((0, 2), (17, 1), (40, 3), (341 - 1, 0)):
        q[row, head] = value * torch.sign(q[row, head])      # (scores of both signs)
        hit[row, head] = True
    got = tq.prompt_attention(q, k, v, cu)
    assert bool(torch.isnan(got[hit]).all()) and torch.equal(got[~hit], want[~hit])


# -- prompt keys whose score is -infinity -----------------------------------------------------

@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("far", [False, True])
def test_prompt_first_score_minus_infinity(tq, d, far):
    """A key with a score of -infinity has weight 0, also where a value that is not
    finite, at a key that the row does not attend, has the rows computed on the CUDA cores."""
    g = torch.Generator(device="cuda").manual_seed(d)
    n = 150
    q, k, v = (torch.randn((n, h, d), generator=g, device="cuda").bfloat16() for h in (2, 1, 1))
    q[..., 0] = q[..., 0].abs() + 0.5
    k[0, 0, 0] = float("-inf")
    if far:
        v[100, 0, 3] = float("nan")
    got = f64(tq.prompt_attention(q, k, v, i32([0, n])))
    seen = 100 if far else n
    ref, absum, sq = osv.prompt_attention(f64(q)[1:seen], f64(k)[1:seen], f64(v)[1:seen], [0, seen - 1], [0, seen - 1])
    assert np.isnan(got[0]).all()                             # attends nothing else
    assert np.isfinite(got[1:seen]).all(), "a weight of 0 made a row NaN"
    assert np.all(np.abs(got[1:seen] - ref) <= S.prompt_bound(ref, absum, sq, "bf16", d, n))
    assert not far or np.isnan(got[100:, :, 3]).all() and np.isfinite(got[100:, :, 4:]).all()


# -- more nodes and tokens than the call allows for -------------------------------------------

@pytest.mark.parametrize("kernel,limit", [("few", 3), ("few", 1), ("one tile", 8), ("one tile", 2), ("two tiles", 64),
                                          ("two tiles", 17), ("wide", 5), ("wide", 1)])
@pytest.mark.parametrize("masked", [False, True])
def test_tree_more_nodes_than_max_nodes(tq, kernel, limit, masked):
    """Nodes from max_nodes on are left out; those kept attend what they attend in a
    call that allows for all of them, and the status says that some were left out."""
    n, hq, hk, d = KERNELS[kernel]
    rng = np.random.default_rng(n + limit)
    t = Tree(tq, [n, limit], [n + 80, limit + 3], hq, hk, d)
    masks = [S.random_tree(rng, n), S.random_tree(rng, limit)]
    mask = torch.from_numpy(S.mask_words(masks, -(-n // 64))).cuda() if masked else None
    got, status = t.call(limit, mask=mask)
    ref, absum, sq = t.reference(masks=masks if masked else None)
    kept = np.r_[0:limit, n:n + limit]
    g = f64(got)
    assert np.all(np.linalg.norm(g - ref, axis=-1)[kept] <= S.tree_bound(ref, absum, sq, "bf16", d, max(t.lens))[kept])
    assert np.all(g[limit:n] == 7.0), "rows of nodes that were left out were written"
    assert status == tq.STATUS_LIMIT
    assert t.call(n, mask=mask)[1] == 0


@pytest.mark.parametrize("kernel", KERNELS)
def test_tree_limits_are_reported(tq, kernel):
    n, hq, hk, d = KERNELS[kernel]
    t = Tree(tq, [n, n], [n + 80, n + 3], hq, hk, d)
    assert t.call(n)[1] == 0 and t.call(n, max_len=n + 82)[1] == 0
    assert t.call(n, max_len=n + 79)[1] == tq.STATUS_LIMIT
    for cu in ([-1, n, 2 * n], [0, n, 2 * n + 1], [0, n, n - 1]):
        assert t.call(n, cu=cu)[1] == tq.STATUS_LIMIT
    assert t.call(n, lens=[n + 80, -1])[1] == tq.STATUS_LIMIT
    assert t.call(n, cu=[0, n, n])[1] == 0 and t.call(n, lens=[n + 80, 0])[1] == 0


def test_tree_replayed_past_its_limits(tq):
    """A captured step whose lengths outgrow what it was captured for says so."""
    t = Tree(tq, [4, 4], [60, 64], 8, 2, 128)
    cu, lens, status = i32([0, 4, 8]), i32([60, 64]), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(tq.tree_workspace_size(2, 8, 4, 8, 2, 64, 128), dtype=torch.uint8, device="cuda")
    out, table = torch.zeros_like(t.q), i32(t.table)

    def call():
        tq.tree_attention(t.rot, t.kb, t.vb, t.kc, t.vc, t.q, cu, lens, t.pages, table, t.page, 4, 64, out=out,
                          workspace=ws, status=status)
    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for new_cu, new_lens, past in (([0, 4, 8], [50, 10], False), ([0, 5, 8], [50, 10], True), ([0, 4, 8], [50, 65], True),
                                   ([0, 3, 6], [64, 64], False)):
        cu.copy_(i32(new_cu)), lens.copy_(i32(new_lens)), status.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert int(status) == (tq.STATUS_LIMIT if past else 0), (new_cu, new_lens)


# -- magnitudes -------------------------------------------------------------------------------

@pytest.mark.parametrize("kernel", KERNELS)
def test_tree_rotated_queries_at_the_end_of_fp32(tq, kernel):
    """Finite rows whose largest rotated coordinate lies in [2^127, 2^128) (dense
    rotation: the Walsh-Hadamard sums would overflow)."""
    n, hq, hk, d = KERNELS[kernel]
    t = Tree(tq, [n], [n + 90], hq, hk, d, kind="haar", dtype=torch.float32)
    rng = np.random.default_rng(d)
    y = rng.standard_normal((t.rows, hq, d)) * 2.0**120
    y[..., d // 3] = 1.5 * 2.0**127
    q = torch.from_numpy((y @ P.oracle_rotation("haar", d, W.SEED_ROT)).astype(np.float32)).cuda()
    scale = float(np.float32(0.1 * 2.0**-126))
    assert bool(torch.isfinite(q).all()) and scale > 0
    got, status = t.call(n, q=q, scale=scale)
    ref, absum, sq = t.reference(q=q, scale=scale)
    assert status == 0
    assert np.all(np.linalg.norm(f64(got) - ref, axis=-1) <= S.tree_bound(ref, absum, sq, "f32", d, max(t.lens)))


@pytest.mark.parametrize("kernel", KERNELS)
def test_tree_zero_queries_with_a_small_scale(tq, kernel):
    """Scores of 0 at a scale whose product with a row's factor would underflow: the
    mean of the values that the row attends."""
    n, hq, hk, d = KERNELS[kernel]
    t = Tree(tq, [n], [n + 90], hq, hk, d, dtype=torch.float32)
    t.q.zero_()
    got, status = t.call(n, scale=1e-10)
    ref, absum, sq = t.reference(scale=1e-10)
    assert status == 0
    assert np.all(np.linalg.norm(f64(got) - ref, axis=-1) <= S.tree_bound(ref, absum, sq, "f32", d, max(t.lens)))


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("size", [1e-2, 1e-4, 1e-6])
def test_tree_small_norms(tq, kernel, size):
    """Dequantized values in fp16's subnormal range are rounded to a multiple of
    2^-24: off by 2^-25 each, so by 2^-25 sqrt(d) a value row and by as much times
    |q| and the scale a score, where S.tree_bound has 2^-11 of the value instead of
    its absolute term for these.  Weights below 2^-21 of a row's largest are off by
    2^-32 of it."""
    n, hq, hk, d = KERNELS[kernel]
    t = Tree(tq, [n, n], [n + 90, n + 300], hq, hk, d, dtype=torch.float32, norms=size)
    got, status = t.call(n)
    ref, absum, sq = t.reference()
    row = 2.0**-25 * np.sqrt(d)
    es = row * np.linalg.norm(f64(t.q), axis=-1) / np.sqrt(d)
    longest = float(np.max(np.abs(t.cache["v_norms"].astype(np.float64)))) * np.sqrt(d / 32)
    bound = S.tree_bound(ref, absum, sq, "f32", d, max(t.lens)) - 1e-6
    bound = bound + row + np.expm1(2 * es) * absum + max(t.lens) * 2.0**-32 * longest
    assert status == 0
    assert np.all(np.linalg.norm(f64(got) - ref, axis=-1) <= bound)


# -- calls on another stream ------------------------------------------------------------------

def _busy(x, n=20):
    for _ in range(n):
        x = x @ x * 1e-2
    return x


def _stream_calls(tq):
    """The calls that allocate what they are not given, each with the size in bytes
    of what it allocates: name -> (call(stream), sizes)."""
    t = Tree(tq, [40, 20], [2000, 700], 8, 2, 128, page=32)
    q, k = (torch.randn((900, h, 128), device="cuda").bfloat16() for h in (8, 2))
    cu_t, lens, table, cu_p = i32(t.cu), i32(t.lens), i32(t.table), i32([0, 800, 900])
    need = tq.tree_workspace_size(2, 60, 40, 8, 2, 2000, 128)
    free, new = i32(np.arange(400)), i32([3000, 2000])
    zero, tab = i32([0, 0]), i32(np.full((2, 200), -1))

    def tree(stream):
        return [tq.tree_attention(t.rot, t.kb, t.vb, t.kc, t.vc, t.q, cu_t, lens, t.pages, table, 32, 40, 2000,
                                  stream=stream)]

    def prompt(stream):
        return [tq.prompt_attention(q, k, k, cu_p, stream=stream)]

    def tables(stream):
        return list(tq.page_tables(zero, new, 16, 400, free, tab, 5000, stream=stream).values())
    return {"tree": (tree, [need, 2 * t.q.numel()]), "prompt": (prompt, [2 * q.numel()]),
            "tables": (tables, [40000, 20000, 12, 8, 4])}


@pytest.mark.parametrize("which", ["tree", "prompt", "tables"])
def test_memory_of_a_call_is_not_in_use_on_the_current_stream(tq, which):
    """stream= another than the current one, outputs and workspace left to the call:
    blocks that the current stream gave back, with work on them still queued there,
    are not among what the call writes."""
    call, sizes = _stream_calls(tq)[which]
    want = call(None)
    side, x = torch.cuda.Stream(), torch.randn((4096, 4096), device="cuda")
    torch.cuda.synchronize()
    before = [torch.full((n,), 0x3C, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
    _busy(x)
    copies = [t.clone() for t in before]              # queued behind the products
    del before
    got = call(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(bool((t == 0x3C).all()) for t in copies)


@pytest.mark.parametrize("which", ["tree", "prompt", "tables"])
def test_outputs_of_a_call_are_kept_for_the_current_stream(tq, which):
    """The same outputs, given back while the current stream has still to read them,
    are not among what a later call on that stream writes."""
    call, _ = _stream_calls(tq)[which]
    want = call(None)
    side, x = torch.cuda.Stream(), torch.randn((4096, 4096), device="cuda")
    torch.cuda.synchronize()
    got = call(side)
    torch.cuda.current_stream().wait_stream(side)
    _busy(x)
    copies = [t.clone() for t in got]
    sizes = [t.numel() * t.element_size() for t in got]
    del got
    with torch.cuda.stream(side):
        later = [torch.full((n,), 0x3C, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(copies, want)) and len(later) == 3 * len(sizes)


# -- prompt offsets past the arrays -----------------------------------------------------------

@pytest.mark.parametrize("batch", [1, 40, 200])
@pytest.mark.parametrize("d", [64, 256])
def test_prompt_rows_past_the_arrays_leave_the_others(tq, batch, d):
    """Offsets of a last sequence that end behind the arrays (a captured call replayed
    with larger ones): its rows that are there attend what they attend in full arrays,
    as far as it is there."""
    rng = np.random.default_rng(batch + d)
    cu = np.cumsum([0] + [3] * (batch - 1) + [150])
    total, first = int(cu[-1]), int(cu[-2])
    q, k, v = (torch.from_numpy(rng.standard_normal((total, h, d))).to("cuda", torch.bfloat16) for h in (4, 2, 2))
    ref, absum, sq = osv.prompt_attention(f64(q), f64(k), f64(v), cu, cu)
    for rows, keys in ((total, total), (total - 60, total), (total, total - 30), (total - 60, total - 30),
                       (total - 150, total)):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = f64(tq.prompt_attention(q[:rows], k[:keys], v[:keys], i32(cu), i32(cu), status=status))
        # (a call with no rows launches nothing)
        assert int(status) == (0 if rows == 0 or rows == keys == total else tq.STATUS_LIMIT)
        want, scale = ref[:rows].copy(), absum[:rows].copy()
        for h in range(4):                                # the rows some of whose keys are missing
            if rows > keys:
                every = np.ones((rows - keys, keys - first), dtype=bool)
                want[keys:, h], scale[keys:, h], _ = osv.attend(f64(q)[keys:rows, h], f64(k)[first:keys, h // 2],
                                                                f64(v)[first:keys, h // 2], every, d**-0.5)
        assert np.all(np.abs(got - want) <= S.prompt_bound(want, scale, sq[:rows], "bf16", d, 150))


def test_prompt_offsets_past_the_arrays_are_reported(tq):
    q = torch.randn((50, 2, 64), device="cuda").half()
    for cu, cu_k in (([-1, 30, 50], None), ([0, 30, 51], None), ([0, 40, 10, 50], None), ([0, 30, 50], [-2, 30, 50]),
                     ([0, 30, 50], [0, 31, 30]), ([0, 30, 50], [0, 30, 60]), ([0] * 300 + [51], None)):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        tq.prompt_attention(q, q, q, i32(cu), None if cu_k is None else i32(cu_k), status=status)
        assert int(status) == tq.STATUS_LIMIT, (cu, cu_k)
    for cu in ([0, 30, 50], [2, 2, 40], [0] * 300 + [50], [50, 50]):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        tq.prompt_attention(q, q, q, i32(cu), status=status)
        assert int(status) == 0, cu


# -- more of what the calls allow -------------------------------------------------------------

@pytest.mark.parametrize("kernel", KERNELS)
def test_tree_in_place(tq, kernel):
    """out may be q: the queries are read before the first output is written."""
    n, hq, hk, d = KERNELS[kernel]
    t = Tree(tq, [n, n], [n + 90, n + 700], hq, hk, d)
    want, _ = t.call(n)
    q = t.q.clone()
    got, status = t.call(n, q=q, out=q)
    assert status == 0 and got is q and torch.equal(got, want)


def test_tree_wide_groups_and_many_requests(tq):
    t = Tree(tq, [40, 3], [300, 170], 64, 1, 64)
    got, status = t.call(40)
    ref, absum, sq = t.reference()
    assert status == 0 and np.all(np.linalg.norm(f64(got) - ref, axis=-1) <= S.tree_bound(ref, absum, sq, "bf16", 64, 300))
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 60, 3000).tolist()
    t = Tree(tq, [min(1, x) for x in lens], lens, 2, 2, 64)
    got, status = t.call(1)
    ref, absum, sq = t.reference()
    assert status == 0 and np.all(np.linalg.norm(f64(got) - ref, axis=-1) <= S.tree_bound(ref, absum, sq, "bf16", 64, 60))


@pytest.mark.parametrize("group", [33, 37, 48, 64])
def test_prompt_wide_groups(tq, group):
    """Groups whose heads do not fit one row tile, a prime one among them."""
    rng = np.random.default_rng(group)
    q, k, v = (torch.from_numpy(rng.standard_normal((70, h, 64))).to("cuda", torch.bfloat16) for h in (group, 1, 1))
    cu = [0, 1, 70]
    got = f64(tq.prompt_attention(q, k, v, i32(cu)))
    ref, absum, sq = osv.prompt_attention(f64(q), f64(k), f64(v), cu, cu)
    assert np.all(np.abs(got - ref) <= S.prompt_bound(ref, absum, sq, "bf16", 64, 69))


def test_page_tables_largest_batch(tq):
    rng = np.random.default_rng(6)
    batch, page = 16384, 16
    ctx, new = rng.integers(0, 50, batch), rng.integers(0, 9, batch)
    held, want = -(-ctx // page), -(-(ctx + new) // page)
    n_pages = int(want.sum())
    perm = rng.permutation(n_pages)
    table = np.full((batch, 4), -1, dtype=np.int32)
    table[np.arange(4)[None, :] < held[:, None]] = perm[:held.sum()]
    free, n_slots = perm[held.sum():], int(new.sum()) + 3
    t = i32(table)
    out = tq.page_tables(i32(ctx), i32(new), page, n_pages, i32(free), t, n_slots)
    ref = osv.page_tables(ctx, new, page, n_pages, free, table, n_slots)
    for name, x in dict(out, block_table=t).items():
        assert np.array_equal(x.cpu().numpy(), ref[name]), name


def test_calls_without_tokens(tq):
    t = Tree(tq, [0, 0], [30, 0], 4, 2, 64)
    assert t.call(1)[1] == 0                                   # no rows
    q = torch.zeros((5, 4, 64), device="cuda").bfloat16()
    out, status = t.call(1, q=q)                               # rows of padding only
    assert status == 0 and bool((out == 7.0).all())
    none = torch.empty((0, 4, 64), device="cuda").bfloat16()
    assert tq.prompt_attention(none, none, none, i32([0, 0])).shape == none.shape
    got = tq.prompt_attention(q, none, none, i32([0, 5]), i32([0, 0]))
    assert bool((got == 0).all())                              # queries without a key
    kc, kt = tq.build_codebook(4)
    before = {k: v.clone() for k, v in t.pages.items()}
    tq.quantize_kv_paged(t.rot, 4, kc, kt, none[:, :2].contiguous(), torch.empty(0, dtype=torch.int64, device="cuda"),
                         t.pages["k_codes"], t.pages["k_norms"], t.page)
    assert all(torch.equal(before[k], v) for k, v in t.pages.items())


@pytest.mark.parametrize("kernel", KERNELS)
def test_offsets_past_32_bits_in_the_cache(tq, kernel):
    """Rows whose codes lie more than 2^32 bytes into the page storage are stored
    and read as in a small one."""
    n, hq, hk, d = KERNELS[kernel]
    page, bits, lens = 256, 4, [600, 300]
    per = [-(-x // page) for x in lens]
    small, wide = sum(per), (2**32 + 2**28) // (hk * page * d * bits // 8)
    rng = np.random.default_rng(d)
    rot = tq.Rotation("wht", d, d, W.SEED_ROT)
    kc, kt = tq.build_codebook(bits)
    rows = torch.from_numpy(rng.standard_normal((2, sum(lens), hk, d))).to("cuda", torch.bfloat16)
    q = torch.from_numpy(rng.standard_normal((2 * n, hq, d))).to("cuda", torch.bfloat16)
    out = []
    for n_pages in (small, wide):
        pages = {}
        for name in "kv":
            pages[name + "_codes"] = torch.zeros((n_pages, hk, page, d * bits // 32), dtype=torch.int32, device="cuda")
            pages[name + "_norms"] = torch.zeros((n_pages, hk, page, d // 32), dtype=torch.int16, device="cuda")
        ids = np.arange(n_pages - small, n_pages)
        table = np.zeros((2, max(per)), dtype=np.int64)
        table[0, :per[0]], table[1, :per[1]] = ids[:per[0]], ids[per[0]:]
        t = [np.arange(x) for x in lens]
        slots = np.concatenate([table[b][t[b] // page] * page + t[b] % page for b in range(2)])
        for i, name in enumerate("kv"):
            tq.quantize_kv_paged(rot, bits, kc, kt, rows[i], torch.from_numpy(slots).cuda(), pages[name + "_codes"],
                                 pages[name + "_norms"], page)
        out.append(tq.tree_attention(rot, bits, bits, kc, kc, q, i32([0, n, 2 * n]), i32(lens), pages, i32(table), page, n,
                                     max(lens)))
        del pages
    assert torch.equal(out[0], out[1]) and float(out[0].abs().max()) > 0


@pytest.mark.parametrize("d", [128, 256])
def test_prompt_offsets_past_32_bits(tq, d):
    """Rows that lie more than 2^32 elements into a fused projection."""
    heads, total, n = (16, 8, 8), 2**32 // (32 * d) + 700, 300
    qkv = torch.zeros((total, sum(heads), d), dtype=torch.bfloat16, device="cuda")
    qkv[-n:] = torch.randn((n, sum(heads), d), device="cuda").bfloat16()
    out = torch.zeros((total, heads[0], d), dtype=torch.bfloat16, device="cuda")
    q, k, v = qkv[:, :16], qkv[:, 16:24], qkv[:, 24:]
    tq.prompt_attention(q, k, v, i32([total - n, total - 100, total]), out=out)
    want = tq.prompt_attention(q[-n:], k[-n:], v[-n:], i32([0, n - 100, n]))
    assert torch.equal(out[-n:], want) and not bool(out[:-n].any())


def test_a_captured_step_replayed_with_other_lengths(tq):
    """Tables, stores and drafted-token attention of a step in one graph, rows padded to
    its size: every replay gives what the calls give for its lengths."""
    rng = np.random.default_rng(8)
    d, hq, hk, page, n_pages, rows = 128, 8, 2, 16, 64, 12
    rot = tq.Rotation("wht", d, d, W.SEED_ROT)
    (kc, kt), (vc, vt) = tq.build_codebook(4), tq.build_codebook(3)
    start = S.cache_to(S.random_cache(rng, n_pages, hk, page, d, 4, 3), "cuda")
    perm = rng.permutation(n_pages)
    first = np.full((2, 16), -1, dtype=np.int32)
    first[0, :10], first[1, :10] = perm[:10], perm[10:20]
    free = i32(perm[20:])
    ctx, new, table = i32([0, 0]), i32([0, 0]), i32(first)
    pages = {k: v.clone() for k, v in start.items()}
    q, k, v = (torch.from_numpy(rng.standard_normal((rows, h, d))).to("cuda", torch.bfloat16) for h in (hq, hk, hk))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def step(table, pages, out):
        t = tq.page_tables(ctx, new, page, n_pages, free, table, rows, status=status)
        tq.quantize_kv_paged(rot, 4, kc, kt, k, t["slots"], pages["k_codes"], pages["k_norms"], page, status=status)
        tq.quantize_kv_paged(rot, 3, vc, vt, v, t["slots"], pages["v_codes"], pages["v_norms"], page, status=status)
        return tq.tree_attention(rot, 4, 3, kc, vc, q, t["cu_new"], t["total_lens"], pages, table, page, 8, 256, out=out,
                                 status=status)
    out = torch.zeros_like(q)
    step(table, pages, out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(table, pages, out)
    for c, n in (([150, 33], [8, 4]), ([16, 160], [1, 1]), ([0, 159], [3, 0]), ([47, 48], [2, 7])):
        ctx.copy_(i32(c)), new.copy_(i32(n)), table.copy_(i32(first)), out.fill_(7.0)
        for name in pages:
            pages[name].copy_(start[name])
        g.replay()
        fresh = {name: x.clone() for name, x in start.items()}
        want = step(i32(first), fresh, torch.full_like(q, 7.0))
        torch.cuda.synchronize()
        assert int(status) == 0 and torch.equal(out, want), (c, n)
        assert all(torch.equal(pages[name], fresh[name]) for name in pages)
        assert bool((out[sum(n):] == 7.0).all()) and bool((out[:sum(n)] != 7.0).any())
