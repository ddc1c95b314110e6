"""Pins of oracle/serving.py: hand examples, invariants and the flat oracle."""

import numpy as np
from scipy.special import softmax

from oracle import attention, codebook, paged, quant, rotation, serving


def test_page_tables_hand_example():
    # page 4: request 0 holds 3 tokens (1 page) and gets 2 (a new page); request
    # 1 is new with 5 (2 pages); request 2 gets nothing
    table = np.array([[9, -1, -1], [-1, -1, -1], [7, 8, -1]])
    r = serving.page_tables([3, 0, 8], [2, 5, 0], 4, 12, [5, 6, 2, 1], table, 9)
    assert r["block_table"].tolist() == [[9, 5, -1], [6, 2, -1], [7, 8, -1]]
    assert r["cu_new"].tolist() == [0, 2, 7, 7]
    assert r["total_lens"].tolist() == [5, 5, 8]
    assert r["slots"].tolist() == [39, 20, 24, 25, 26, 27, 8, -1, -1]
    assert r["positions"].tolist() == [3, 4, 0, 1, 2, 3, 4, -1, -1]
    assert r["n_taken"].tolist() == [3] and not r["no_pages"] and not r["bad_page"]


def test_page_tables_refused_requests_take_nothing():
    # the list runs out at request 1; request 2 needs no page and is placed
    table = np.array([[-1, -1], [-1, -1], [3, -1]])
    r = serving.page_tables([0, 0, 1], [4, 8, 2], 4, 8, [1, 2], table, 14)
    assert r["total_lens"].tolist() == [4, 0, 3] and r["n_taken"].tolist() == [1] and r["no_pages"]
    assert r["slots"].tolist() == [4, 5, 6, 7] + [-1] * 8 + [13, 14]
    # a row that is too short does not use up the list
    r = serving.page_tables([0, 0], [12, 4], 4, 8, [1], np.full((2, 2), -1), 16)
    assert r["total_lens"].tolist() == [0, 4] and r["slots"][12:].tolist() == [4, 5, 6, 7]


def test_prompt_attention_is_softmax_attention():
    rng = np.random.default_rng(3)
    q, k, v = (rng.standard_normal((9, h, 8)) for h in (4, 2, 2))
    cu = [0, 4, 4, 9]
    out, absum, _ = serving.prompt_attention(q, k, v, cu, cu)
    for b in range(3):
        r = slice(cu[b], cu[b + 1])
        for h in range(4):
            s = q[r, h] @ k[r, h // 2].T / np.sqrt(8)
            s = np.where(np.tril(np.ones_like(s)) > 0, s, -np.inf)
            if s.size:
                assert np.allclose(out[r, h], softmax(s, axis=1) @ v[r, h // 2], rtol=0, atol=1e-13)
    assert np.all(absum >= np.abs(out) - 1e-15)


def test_chunks_equal_the_whole_prompt():
    rng = np.random.default_rng(4)
    q, k, v = (rng.standard_normal((11, 1, 8)) for _ in range(3))
    whole, _, _ = serving.prompt_attention(q, k, v, [0, 11], [0, 11])
    tail, _, _ = serving.prompt_attention(q[6:], k, v, [0, 5], [0, 11])
    assert np.allclose(whole[6:], tail, rtol=0, atol=1e-13)
    none, _, _ = serving.prompt_attention(q[:3], k[:1], v[:1], [0, 3], [0, 1])
    assert np.all(none[:2] == 0) and np.allclose(none[2], v[0])


def _cache(rng, n_pages, n_kv, page, d, kb, vb):
    pages = {}
    for name, bits in (("k", kb), ("v", vb)):
        idx = rng.integers(0, 1 << bits, (n_pages * n_kv * page, d))
        pages[name + "_codes"] = quant.pack(idx, bits, 32).reshape(n_pages, n_kv, page, -1)
        pages[name + "_norms"] = rng.uniform(0.5, 8, (n_pages, n_kv, page, d // 32)).astype(np.float16)
    return pages


def test_single_nodes_equal_the_flat_decode():
    rng = np.random.default_rng(5)
    d, n_kv, n_q, page, length = 64, 2, 4, 16, 37
    pages = _cache(rng, 8, n_kv, page, d, 4, 3)
    table = rng.permutation(8)[:6].reshape(2, 3)
    kc, vc = codebook.stored_table(4, 32)[0], codebook.stored_table(3, 32)[0]
    rot = rotation.rotation("wht", d, 1000)
    q = rng.standard_normal((2, n_q, d))
    out, _, _ = serving.tree_attention(q, rot, [0, 1, 2], [length] * 2, None, pages, table, page, kc, vc, 4, 3)
    flat = {}
    for name, bits in (("k", 4), ("v", 3)):
        w = pages[name + "_codes"].shape[-1]
        codes = paged.gather(pages[name + "_codes"].reshape(-1, w), table, page, n_kv, 2, length)
        flat[name] = quant.unpack(codes, bits, 32, d)
        flat[name + "n"] = paged.gather(pages[name + "_norms"].reshape(-1, d // 32), table, page, n_kv, 2, length)
    ref = attention.decode(q, rot, flat["k"], flat["kn"], kc, flat["v"], flat["vn"], vc, 32, n_kv, length)
    assert np.allclose(out, ref, rtol=0, atol=1e-12)


def test_a_branch_equals_its_path_alone():
    """A node of a tree equals the last node of a chain of its ancestors."""
    rng = np.random.default_rng(6)
    d, page, ctx = 64, 16, 20
    pages = _cache(rng, 4, 1, page, d, 4, 4)
    table = np.array([[2, 0, 3, 1]])
    kc = codebook.stored_table(4, 32)[0]
    rot = rotation.rotation("haar", d, 1000)
    q = rng.standard_normal((5, 2, d))
    parents = [-1, 0, 0, 1, 2]                     # 0 -> {1 -> 3, 2 -> 4}
    masks = []
    for i, p in enumerate(parents):
        masks.append((masks[p] if p >= 0 else 0) | 1 << i)
    tree, _, _ = serving.tree_attention(q, rot, [0, 5], [ctx + 5], [masks], pages, table, page, kc, kc, 4, 4)
    # the path 0, 2, 4 moved to the end of a cache of its own
    flat = {n: v[table[0]].transpose(0, 2, 1, 3).reshape(4 * page, 1, -1) for n, v in pages.items()}
    keep = list(range(ctx)) + [ctx, ctx + 2, ctx + 4]
    alone = {n: np.zeros_like(v) for n, v in pages.items()}
    for n in flat:
        for t, s in enumerate(keep):
            alone[n][t // page, 0, t % page] = flat[n][s, 0]
    chain, _, _ = serving.tree_attention(q[[0, 2, 4]], rot, [0, 3], [ctx + 3], None, alone, np.arange(4)[None], page,
                                         kc, kc, 4, 4)
    assert np.allclose(tree[[0, 2, 4]], chain, rtol=0, atol=1e-12)


def test_rows_that_attend_nothing_are_zero():
    rng = np.random.default_rng(7)
    out, absum, sq = serving.attend(rng.standard_normal((2, 4)), np.full((3, 4), np.nan), np.full((3, 4), np.nan),
                                    np.zeros((2, 3), dtype=bool), 1.0)
    assert np.all(out == 0) and np.all(absum == 0) and np.all(sq == 0)
