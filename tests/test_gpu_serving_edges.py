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
