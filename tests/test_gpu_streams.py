"""GPU tests of calls on another stream than the current one (stream=) that
allocate their outputs and workspaces themselves: quantize, logits, decode,
append + decode, search."""

import numpy as np
import pytest

import workloads as W
from tests import serving as S

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def tq():
    import kv_cache_vector_11_b200 as lib
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    return lib


def _calls(tq):
    """name -> (call(stream) -> list of outputs, bytes of what it allocates)."""
    batch, hk, hq, ctx, d, kb, vb, page = 2, 2, 8, 4096, 128, 4, 3, 64
    g = torch.Generator(device="cuda").manual_seed(1)

    def rows(*shape):
        return torch.randn(shape, generator=g, device="cuda").bfloat16()
    rot = tq.Rotation("wht", d, d, W.SEED_ROT)
    qjl = tq.Rotation("gauss", 128, d, W.SEED_ROT + 1)
    (kc, kt), (vc, vt) = tq.build_codebook(kb), tq.build_codebook(vb)
    x, q = rows(batch * hk * ctx, d), rows(batch, hq, d)
    k, v = (tq.quantize_kv(rot, b, c, t, x) for b, c, t in ((kb, kc, kt), (vb, vc, vt)))
    rng = np.random.default_rng(1)
    table, n_pages = S.page_tables_for(rng, [ctx] * batch, page)
    pages = S.cache_to(S.random_cache(rng, n_pages, hk, page, d, kb, vb), "cuda")
    table = torch.from_numpy(table).cuda()
    new = rows(batch, hk, d)
    need = tq.decode_workspace_size(batch, hq, hk, ctx, d)
    out = 4 * batch * hq * d

    def quantize(stream):
        return list(tq.quantize_kv(rot, kb, kc, kt, x, qjl=qjl, stream=stream).values())

    def logits(stream):
        return [tq.attn_logits(rot, kb, kc, q, k["codes"], k["norms"], hk, ctx, stream=stream)]

    def decode(stream):
        return [tq.decode_attention(rot, kb, vb, kc, vc, q, k["codes"], k["norms"], v["codes"], v["norms"], hk, ctx,
                                    stream=stream)]

    def append(stream):
        return [tq.decode_append_paged(rot, kb, vb, (kc, kt), (vc, vt), q, new, new, pages, table, hk, ctx, page,
                                       stream=stream)]

    def search(stream):
        return list(tq.search_topk(rot, kb, kc, q[0], k["codes"], k["norms"], 5, stream=stream))
    n = x.shape[0]
    return {"quantize": (quantize, [64 * n, 8 * n, 16 * n, 2 * n]), "logits": (logits, [4 * batch * hq * ctx]),
            "decode": (decode, [need, out]), "append": (append, [need, out]),
            "search": (search, [tq.search_workspace_size(hq, n, d, 5), 4 * hq * 5])}


NAMES = ["quantize", "logits", "decode", "append", "search"]


def _busy(x, n=20):
    for _ in range(n):
        x = x @ x * 1e-2


@pytest.mark.parametrize("which", NAMES)
def test_memory_of_a_call_is_its_own(tq, which):
    """Blocks that the current stream gave back in front of the call, with work on them
    still queued, are not among what it writes; nor does what is allocated behind it,
    while its stream is still busy, get its memory."""
    call, sizes = _calls(tq)[which]
    want = [t.clone() for t in call(None)]
    side, x = torch.cuda.Stream(), torch.randn((4096, 4096), device="cuda")
    torch.cuda.synchronize()
    before = [torch.full((n,), 0x3C, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
    _busy(x)
    copies = [t.clone() for t in before]
    del before
    got = call(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and all(bool((t == 0x3C).all()) for t in copies)
    with torch.cuda.stream(side):
        _busy(x)
    got = call(side)
    later = [torch.full((n,), 0x3C, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and all(bool((t == 0x3C).all()) for t in later)


@pytest.mark.parametrize("which", NAMES)
def test_outputs_of_a_call_are_kept_for_the_current_stream(tq, which):
    call, _ = _calls(tq)[which]
    want = [t.clone() for t in call(None)]
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
