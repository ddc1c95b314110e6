"""Serving around the paged cache: page tables, prompt attention, drafted tokens.

TEST INFRASTRUCTURE (oracle).  Not imported by the product path.

The pages name the KV-cache allocation and softmax(Q K^T / sqrt(d)) V ("Google
TurboQuant deep dive", section 4.3) and nothing of a serving loop; the readings
are the library's own:

* requests take pages from the front of a free list in request order; a request
  that cannot be placed takes none;
* a sequence with fewer queries than keys asks about its last positions;
* drafted tokens lie in the cache after the tokens they extend, and a bit mask
  says which of them a node attends.

Besides each output the attention functions return, per output value, a bound
scale ``absum`` = sum_t p_t |v_t| and the spread ``sq`` = max_t sum |q k_t|, from
which the tests derive their rounding bounds.
"""

import numpy as np

from . import quant


def page_tables(ctx, new, page, n_pages, free, table, n_slots):
    """Sequential statement of tq_page_tables.  Returns a dict with the outputs,
    the updated ``block_table`` and ``no_pages`` / ``bad_page``."""
    table = np.array(table, copy=True)
    batch, max_pages = table.shape
    cu, total, taken = [0], [], 0
    wanted = 0                      # pages wanted so far, placed or not
    slots = np.full(n_slots, -1, dtype=np.int64)
    pos = np.full(n_slots, -1, dtype=np.int32)
    no_pages = bad_page = False
    for b in range(batch):
        c, n = max(int(ctx[b]), 0), max(int(new[b]), 0)
        start = cu[-1]
        cu.append(start + n)
        held, want = -(-c // page), -(-(c + n) // page)
        ok = want <= max_pages and start + n <= n_slots and c + n < 2**31
        need = want - held if ok else 0
        if ok and need and wanted + need > len(free):
            ok = False
        first = wanted
        wanted += need
        if not ok:
            no_pages = True
            total.append(c)
            continue
        taken += need
        total.append(c + n)
        for j in range(held, want):
            table[b, j] = free[first + j - held]
        for i in range(n):
            p = int(table[b, (c + i) // page])
            pos[start + i] = c + i
            if 0 <= p < n_pages:
                slots[start + i] = p * page + (c + i) % page
            else:
                bad_page = True
    cap = 2**31 - 1
    return {"cu_new": np.array([min(x, cap) for x in cu], dtype=np.int32),
            "total_lens": np.array(total, dtype=np.int32), "slots": slots, "positions": pos,
            "n_taken": np.array([taken], dtype=np.int32), "block_table": table,
            "no_pages": no_pages, "bad_page": bad_page}


def attend(q, k, v, allowed, scale):
    """One head: q [N, d], k and v [L, d], allowed bool [N, L], float64.  Returns
    (out, absum, sq); a row that may attend nothing is zero.  Keys a row may
    not attend are never multiplied."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    out = np.zeros((q.shape[0], v.shape[1]))
    absum = np.zeros_like(out)
    sq = np.zeros(q.shape[0])
    for i in range(q.shape[0]):
        at = np.nonzero(allowed[i])[0]
        if at.size == 0:
            continue
        with np.errstate(invalid="ignore"):
            s = k[at] @ q[i] * scale
            p = np.exp(s - s.max())
            p /= p.sum()
            out[i] = p @ v[at]
            absum[i] = p @ np.abs(v[at])
            sq[i] = np.max(np.abs(k[at]) @ np.abs(q[i])) * scale
    return out, absum, sq


def causal(nq, nk):
    """allowed[i, j] = j <= i + nk - nq."""
    return np.arange(nk)[None, :] <= np.arange(nq)[:, None] + nk - nq


def prompt_attention(q, k, v, cu_q, cu_k, scale=None):
    """Packed sequences: q [total_q, Hq, d], k and v [total_k, Hkv, d]."""
    group = q.shape[1] // k.shape[1]
    if scale is None:
        scale = 1.0 / np.sqrt(q.shape[2])
    out, absum = np.zeros(q.shape), np.zeros(q.shape)
    sq = np.zeros(q.shape[:2])
    for b in range(len(cu_q) - 1):
        rq, rk = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        ok = causal(rq.stop - rq.start, rk.stop - rk.start)
        for h in range(q.shape[1]):
            out[rq, h], absum[rq, h], sq[rq, h] = attend(q[rq, h], k[rk, h // group], v[rk, h // group], ok, scale)
    return out, absum, sq


def tree_allowed(n, length, mask):
    """allowed [n, length] of n nodes at the end of ``length`` cached tokens;
    mask: list of n Python ints (bit j = node j), or None for a chain."""
    first = length - n
    ok = np.zeros((n, length), dtype=bool)
    for i in range(n):
        for t in range(length):
            j = t - first
            ok[i, t] = j < 0 or (j <= i if mask is None else bool((mask[i] >> int(j)) & 1))
    return ok


def tree_attention(q, rot, cu, lens, masks, pages, table, page, kc, vc, kbits, vbits, scale=None):
    """q [rows, Hq, d]; pages: dict of uint32 codes [pages, Hkv, page, W] and fp16
    norms; masks: one list per request, or None.  Returns (out, absum, sq) with
    absum and sq of the rotated frame (absum [rows, Hq] = sum_t p |v_hat_t|_2)."""
    rot = np.asarray(rot, dtype=np.float64)
    rows, n_q, d = q.shape
    n_kv = pages["k_codes"].shape[1]
    if scale is None:
        scale = 1.0 / np.sqrt(d)
    out, absum, sq = np.zeros(q.shape), np.zeros((rows, n_q)), np.zeros((rows, n_q))
    for b in range(len(lens)):
        r, length = slice(cu[b], cu[b + 1]), int(lens[b])
        n = r.stop - r.start
        if n == 0:
            continue
        ok = tree_allowed(n, length, None if masks is None else masks[b])
        t = np.arange(length)
        pg = np.asarray(table[b])[t // page].astype(np.int64)
        for hk in range(n_kv):
            hat = {}
            for name, bits, c in (("k", kbits, kc), ("v", vbits, vc)):
                codes = pages[name + "_codes"][pg, hk, t % page]
                idx = quant.unpack(codes, bits, 32, d)
                hat[name] = quant.dequantize_rotated(idx, pages[name + "_norms"][pg, hk, t % page], c, 32)
            for h in range(hk * (n_q // n_kv), (hk + 1) * (n_q // n_kv)):
                qr = np.asarray(q[r, h], dtype=np.float64) @ rot.T
                o, _, sq[r, h] = attend(qr, hat["k"], hat["v"], ok, scale)
                norms = np.linalg.norm(hat["v"], axis=1)
                absum[r, h] = attend(qr, hat["k"], norms[:, None], ok, scale)[0][:, 0]
                out[r, h] = o @ rot
    return out, absum, sq
