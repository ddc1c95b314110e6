"""Helpers of the serving tests: inputs and the rounding bounds.

Bounds.  u = half a step of a type relative to the value (bf16 2^-8, fp16 2^-11,
fp32 2^-24).  A score is off by at most es = e_op * sq, where sq = scale * max_t
sum_i |q_i k_ti| and e_op the relative error of one product's operands plus the
d additions of the fp32 sum (each at most 2^-23, a truncated addition).  A weight
exp(s - m) is then off by a factor within exp(es) (its maximum by as much again,
which cancels in the quotient), the exponential itself by 2^-21, and it enters the
second product rounded to the operand type (u).  The divisor has the same
errors without the rounding.  So
    |out - ref| <= (u_p + u_v + exp(2 es) - 1 + 2^-20 + n 2^-23) * sum_t p_t |v_t| + u_out |ref|
with u_p, u_v the roundings of the weights and of the values and n 2^-23 for the
sums over n keys."""

import numpy as np

HALF_STEP = {"bf16": 2.0**-8, "f16": 2.0**-11, "f32": 2.0**-24}


def prompt_bound(out, absum, sq, dtype, d, n_keys):
    u = HALF_STEP[dtype]
    es = (d * 2.0**-23) * sq[..., None]
    return (u + np.expm1(2 * es) + 2.0**-20 + n_keys * 2.0**-23) * absum + u * np.abs(out) + 1e-30 + 2.0**-25 * (dtype == "f16")


def tree_bound(ref, absum, sq, dtype, d, n_keys):
    """Rotated queries and dequantized keys are rounded to fp16 (relative 2^-11
    each: 2^-10 of every product), so are the weights and the values.  absum is
    sum_t p |v_t|_2, and an orthogonal rotation back keeps 2-norms, so the bound
    is on the 2-norm of a row's error."""
    es = (2.0**-10 + (d + 8) * 2.0**-23) * sq
    e = 2.0**-11 + 2.0**-11 + np.expm1(2 * es) + 2.0**-20 + n_keys * 2.0**-23
    return e * absum + (HALF_STEP[dtype] + 2.0**-18) * np.linalg.norm(ref, axis=-1) + 1e-6


def random_tree(rng, n):
    """Ancestor bits (Python ints) of a random tree of n nodes."""
    masks = []
    for i in range(n):
        parent = int(rng.integers(max(-1, i - 6), i)) if i else -1
        masks.append((masks[parent] if parent >= 0 else 0) | 1 << i)
    return masks


def mask_words(masks, words):
    """int64 [rows, words] of lists of Python ints."""
    flat = [m for per in masks for m in per]
    out = np.zeros((len(flat), words), dtype=np.uint64)
    for r, m in enumerate(flat):
        for w in range(words):
            out[r, w] = (m >> (64 * w)) & ((1 << 64) - 1)
    return out.view(np.int64)


def page_tables_for(rng, lens, page, spare=3):
    """(table int32 [B, max_pages], n_pages) with the pages in random order."""
    per = [-(-x // page) for x in lens]
    n_pages = sum(per) + spare
    perm = rng.permutation(n_pages)
    table = np.zeros((len(lens), max(max(per), 1)), dtype=np.int32)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, n_pages


def random_cache(rng, n_pages, n_kv, page, d, kb, vb, scale=1.0):
    """Page storage with codes of every value and norms of rows of deviation ``scale``."""
    pages = {}
    for name, bits in (("k", kb), ("v", vb)):
        words = rng.integers(0, 2**32, (n_pages, n_kv, page, d * bits // 32), dtype=np.uint64).astype(np.uint32)
        pages[name + "_codes"] = words
        pages[name + "_norms"] = (scale * rng.uniform(0.3, 3.0, (n_pages, n_kv, page, d // 32))).astype(np.float16)
    return pages


def cache_to(pages, device):
    import torch
    return {n: torch.from_numpy(v.view(np.int32 if v.dtype == np.uint32 else np.int16)).to(device)
            for n, v in pages.items()}
