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
