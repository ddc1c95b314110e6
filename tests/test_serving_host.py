"""CPU tests of the serving entry points: every refusal comes before a launch
(fake device pointers are never dereferenced), and the Python layer refuses
tensors whose type, shape or layout the kernels would misread."""

import ctypes

import numpy as np
import pytest

import kv_cache_vector_11_b200 as tq
from kv_cache_vector_11_b200 import _lib

torch = pytest.importorskip("torch")

FAKE = 1 << 20
OK, INVALID, UNSUPPORTED = 0, 1, 2
L = _lib._lib


@pytest.fixture(scope="module")
def rot():
    return tq.Rotation("wht", 128, 128, 1000)


def tables(ctx=FAKE, new=FAKE, batch=4, page=16, n_pages=8, free=FAKE, n_free=8, table=FAKE, max_pages=4, cu=FAKE,
           total=FAKE + 4096, slots=FAKE, pos=FAKE, n_slots=16, taken=FAKE, status=None):
    return L.tq_page_tables(ctx, new, batch, page, n_pages, free, n_free, table, max_pages, cu, total, slots, pos,
                            n_slots, taken, status, None)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), INVALID), (dict(batch=16385), UNSUPPORTED), (dict(page=24), UNSUPPORTED),
    (dict(page=8), UNSUPPORTED), (dict(page=1 << 17), UNSUPPORTED), (dict(n_pages=0), INVALID),
    (dict(max_pages=0), INVALID), (dict(n_free=-1), INVALID), (dict(n_slots=-1), INVALID), (dict(ctx=None), INVALID),
    (dict(new=None), INVALID), (dict(table=None), INVALID), (dict(cu=None), INVALID), (dict(total=None), INVALID),
    (dict(taken=None), INVALID), (dict(free=None), INVALID), (dict(slots=None), INVALID),
    (dict(total=FAKE), INVALID), (dict(slots=FAKE + 4), INVALID), (dict(cu=FAKE + 2), INVALID),
])
def test_page_tables_refusals(kw, code):
    assert tables(**kw) == code and tq.TQError(code, "x").args


@pytest.mark.parametrize("alias", ["ctx", "new"])
def test_page_tables_refuses_outputs_over_the_lengths(alias):
    apart = dict(ctx=FAKE, new=FAKE + 1024, cu=FAKE + 2048, total=FAKE + 4096)
    assert tables(**dict(apart, free=None)) == INVALID and "free_pages" in L.tq_last_error().decode()
    for out in ("cu", "total"):
        assert tables(**dict(apart, **{out: apart[alias]}, free=None)) == INVALID
        assert "input" in L.tq_last_error().decode()


def paged(rot, bits=4, block=32, x=FAKE, dtype=1, n=4, heads=2, d=128, slots=FAKE, page=16, n_pages=8, codes=FAKE,
          norms=FAKE, c=None, t=None):
    kc, kt = tq.build_codebook(max(bits, 1), 32)
    return L.tq_quantize_kv_paged(rot.handle, bits, block, kc.ctypes.data, kt.ctypes.data, x, dtype, n, heads, d, slots,
                                  page, n_pages, codes, norms, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(bits=1), UNSUPPORTED), (dict(block=64), UNSUPPORTED), (dict(dtype=2), INVALID), (dict(n=-1), INVALID),
    (dict(heads=0), INVALID), (dict(n=1 << 30, heads=4), UNSUPPORTED), (dict(d=64), INVALID),
    (dict(page=17), UNSUPPORTED), (dict(n_pages=0), INVALID), (dict(x=None), INVALID), (dict(slots=None), INVALID),
    (dict(codes=None), INVALID), (dict(norms=None), INVALID), (dict(x=FAKE + 8), INVALID),
    (dict(slots=FAKE + 4), INVALID), (dict(norms=FAKE + 8), INVALID), (dict(n=0, x=None), OK),
])
def test_quantize_paged_refusals(rot, kw, code):
    assert paged(rot, **kw) == code


def prompt(q=FAKE, k=FAKE, v=FAKE, dtype=1, cu_q=FAKE, cu_k=None, batch=2, tq_=8, tk=8, hq=4, hk=2, d=128, qs=512,
           ks=256, vs=256, scale=0.0, out=FAKE + 4096):
    return L.tq_prompt_attention(q, k, v, dtype, cu_q, cu_k, batch, tq_, tk, hq, hk, d, qs, ks, vs, scale, out, None,
                                 None)


@pytest.mark.parametrize("kw,code", [
    (dict(d=96), UNSUPPORTED), (dict(dtype=0), UNSUPPORTED), (dict(dtype=7), UNSUPPORTED), (dict(hq=3), INVALID),
    (dict(hk=0), INVALID), (dict(batch=0), INVALID), (dict(tq_=-1), INVALID), (dict(tq_=1 << 31), UNSUPPORTED),
    (dict(qs=511), INVALID), (dict(qs=504), INVALID), (dict(ks=248), INVALID), (dict(vs=260), INVALID),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(out=None), INVALID), (dict(cu_q=None), INVALID),
    (dict(q=FAKE + 8), INVALID), (dict(out=FAKE + 8), INVALID), (dict(cu_k=FAKE + 2), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(tq_=0, q=None), OK),
    (dict(out=FAKE), INVALID), (dict(tq_=2**31 - 200), UNSUPPORTED), (dict(tk=2**31 - 200, cu_k=FAKE), UNSUPPORTED),
    (dict(batch=2**31 - 1, hq=4, hk=4, ks=512, vs=512), UNSUPPORTED),
])
def test_prompt_refusals(kw, code):
    assert prompt(**kw) == code


def tree(rot, kb=4, vb=3, block=32, q=FAKE, dtype=1, cu=FAKE, batch=2, rows=8, nodes=4, lens=FAKE, max_len=64,
         mask=FAKE, words=1, hq=4, hk=2, d=128, page=16, n_pages=8, table=FAKE, max_pages=4, kc=FAKE, kn=FAKE, vc=FAKE,
         vn=FAKE, scale=0.0, out=FAKE, ws=FAKE, ws_bytes=1 << 40):
    c = [tq.build_codebook(max(b, 1), 32)[0] for b in (kb, vb)]
    return L.tq_tree_attention(rot.handle, kb, vb, block, c[0].ctypes.data, c[1].ctypes.data, q, dtype, cu, batch, rows,
                               nodes, lens, max_len, mask, words, hq, hk, d, page, n_pages, table, max_pages, kc, kn, vc,
                               vn, scale, out, ws, ws_bytes, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(kb=1), UNSUPPORTED), (dict(vb=1), UNSUPPORTED), (dict(block=64), UNSUPPORTED), (dict(dtype=3), INVALID),
    (dict(d=64), INVALID), (dict(batch=0), INVALID), (dict(rows=-1), INVALID), (dict(nodes=0), INVALID),
    (dict(nodes=257, words=5), INVALID), (dict(nodes=65, words=1), INVALID), (dict(hq=5), INVALID),
    (dict(hk=0), INVALID), (dict(page=20), UNSUPPORTED), (dict(n_pages=0), INVALID), (dict(max_len=65), INVALID),
    (dict(q=None), INVALID), (dict(cu=None), INVALID), (dict(lens=None), INVALID), (dict(table=None), INVALID),
    (dict(kc=None), INVALID), (dict(vn=None), INVALID), (dict(out=None), INVALID), (dict(ws=None), INVALID),
    (dict(ws_bytes=0), INVALID), (dict(ws=FAKE + 128), INVALID), (dict(q=FAKE + 8), INVALID),
    (dict(vc=FAKE + 4), INVALID), (dict(mask=FAKE + 4), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(rows=0, q=None), OK), (dict(max_len=2**31 - 200, max_pages=2**30), INVALID),
    (dict(n_pages=2**16, hk=1, page=65536), UNSUPPORTED), (dict(n_pages=2**31 - 1, hk=4, hq=4), UNSUPPORTED),
])
def test_tree_refusals(rot, kw, code):
    assert tree(rot, **kw) == code


def test_tree_workspace_is_zero_for_refused_sizes_and_monotone():
    size = tq.tree_workspace_size
    assert size(0, 8, 4, 4, 2, 64, 128) == 0 and size(2, 8, 257, 4, 2, 64, 128) == 0
    assert size(2, 8, 4, 5, 2, 64, 128) == 0 and size(2, 8, 4, 4, 2, 64, 96) == 0
    small = size(2, 8, 4, 4, 2, 64, 128)
    assert small > 0
    assert size(2, 8, 4, 4, 2, 4096, 128) >= small and size(2, 16, 8, 4, 2, 64, 128) >= small


def _i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_python_refuses_misread_tensors(rot):
    q = torch.zeros((4, 4, 128), dtype=torch.bfloat16)
    k = torch.zeros((4, 2, 128), dtype=torch.bfloat16)
    cu = _i32(3)
    for bad in (dict(cu_q=cu.long()), dict(q=q.half()), dict(k=k[:, :, ::2]), dict(v=k[:3]), dict(cu_k=_i32(4)),
                dict(out=q.float()), dict(out=q.transpose(0, 1).contiguous().transpose(0, 1))):
        kw = dict(q=q, k=k, v=k, cu_q=cu)
        kw.update(bad)
        with pytest.raises(ValueError):
            tq.prompt_attention(kw.pop("q"), kw.pop("k"), kw.pop("v"), kw.pop("cu_q"), **kw)
    with pytest.raises(ValueError):                     # another number of keys needs offsets of its own
        tq.prompt_attention(q, torch.zeros((5, 2, 128), dtype=torch.bfloat16),
                            torch.zeros((5, 2, 128), dtype=torch.bfloat16), cu)
    for bad in (dict(ctx=_i32(2).long()), dict(new=_i32(3)), dict(table=_i32(3, 2)), dict(table=_i32(2, 4)[:, ::2])):
        kw = dict(ctx=_i32(2), new=_i32(2), table=_i32(2, 2))
        kw.update(bad)
        with pytest.raises(ValueError):
            tq.page_tables(kw["ctx"], kw["new"], 16, 4, _i32(4), kw["table"], 8)
    x = torch.zeros((4, 2, 128), dtype=torch.bfloat16)
    kc, kt = tq.build_codebook(4)
    slots, codes, norms = torch.zeros(4, dtype=torch.int64), _i32(3, 2, 16, 16), torch.zeros((3, 2, 16, 4), dtype=torch.int16)
    for bad in (dict(slots=slots.int()), dict(codes=_i32(3, 2, 16, 12)), dict(norms=norms.half()), dict(x=x[:, :1]),
                dict(codes=_i32(3, 1, 16, 16))):
        kw = dict(x=x, slots=slots, codes=codes, norms=norms)
        kw.update(bad)
        with pytest.raises(ValueError):
            tq.quantize_kv_paged(rot, 4, kc, kt, kw["x"], kw["slots"], kw["codes"], kw["norms"], 16)
    pages = dict(k_codes=codes, k_norms=norms, v_codes=_i32(3, 2, 16, 12), v_norms=norms)
    mask = torch.zeros((4, 1), dtype=torch.int64)
    for bad in (dict(cu=_i32(2)), dict(lens=_i32(2).long()), dict(mask=mask.int()), dict(mask=mask[:3]),
                dict(pages=dict(pages, v_codes=codes)), dict(q=q[:, ::2]), dict(table=_i32(3, 4))):
        kw = dict(q=q, cu=_i32(3), lens=_i32(2), pages=pages, table=_i32(2, 4), mask=mask)
        kw.update(bad)
        with pytest.raises(ValueError):
            tq.tree_attention(rot, 4, 3, kc, tq.build_codebook(3)[0], kw["q"], kw["cu"], kw["lens"], kw["pages"],
                              kw["table"], 16, 2, 64, tree_mask=kw["mask"])


def _quantize_call(rot, bits, c, t, **kw):
    x = torch.zeros((4, 2, 128), dtype=torch.bfloat16)
    codes, norms = _i32(3, 2, 16, 4 * bits), torch.zeros((3, 2, 16, 4), dtype=torch.int16)
    tq.quantize_kv_paged(rot, bits, c, t, x, torch.zeros(4, dtype=torch.int64), codes, norms, 16, **kw)


def _tree_call(rot, kb, vb, kc, vc, **kw):
    norms = torch.zeros((3, 2, 16, 4), dtype=torch.int16)
    pages = dict(k_codes=_i32(3, 2, 16, 4 * kb), k_norms=norms, v_codes=_i32(3, 2, 16, 4 * vb), v_norms=norms)
    q = torch.zeros((4, 4, 128), dtype=torch.bfloat16)
    kw.setdefault("workspace", torch.zeros(256, dtype=torch.uint8))
    tq.tree_attention(rot, kb, vb, kc, vc, q, _i32(3), _i32(2), pages, _i32(2, 4), 16, 2, 64, **kw)


def test_python_refuses_codebooks_of_another_width(rot):
    """The library reads 2^bits centroids and 2^bits - 1 boundaries; a shorter array
    is refused (tensors on the CPU are too, but by another message)."""
    books = {b: tq.build_codebook(b) for b in (2, 3, 4)}
    for bits in (2, 3, 4):
        c, t = books[bits]
        for other in books:
            if other == bits:
                continue
            with pytest.raises(ValueError, match="centroids"):
                _quantize_call(rot, bits, books[other][0], t)
            with pytest.raises(ValueError, match="boundaries"):
                _quantize_call(rot, bits, c, books[other][1])
            with pytest.raises(ValueError, match="k_centroids"):
                _tree_call(rot, bits, 3, books[other][0], books[3][0])
            with pytest.raises(ValueError, match="v_centroids"):
                _tree_call(rot, 4, bits, books[4][0], books[other][0])
        with pytest.raises(ValueError, match="not on a CUDA device"):
            _quantize_call(rot, bits, c, t)
        with pytest.raises(ValueError, match="not on a CUDA device"):
            _tree_call(rot, bits, bits, list(c), c.astype(np.float64))


@pytest.mark.parametrize("status", [torch.zeros(1, dtype=torch.int32, device="meta"), torch.zeros(1, dtype=torch.int64),
                                    torch.zeros(1), torch.zeros(0, dtype=torch.int32)])
def test_python_refuses_a_status_that_the_kernels_cannot_write(rot, status):
    """A status word on another device would be a write to an address of that device."""
    (kc, kt), (vc, _) = tq.build_codebook(4), tq.build_codebook(3)
    q = torch.zeros((4, 2, 128), dtype=torch.bfloat16)
    for call in (lambda: tq.page_tables(_i32(2), _i32(2), 16, 4, _i32(4), _i32(2, 2), 8, status=status),
                 lambda: _quantize_call(rot, 4, kc, kt, status=status),
                 lambda: tq.prompt_attention(q, q, q, _i32(3), status=status),
                 lambda: _tree_call(rot, 4, 3, kc, vc, status=status)):
        with pytest.raises(ValueError, match="status"):
            call()


@pytest.mark.parametrize("workspace", [torch.zeros(1 << 20, dtype=torch.uint8, device="meta"),
                                       torch.zeros(1 << 20, dtype=torch.uint8)[::2]])
def test_python_refuses_a_workspace_on_another_device(rot, workspace):
    kc, vc = tq.build_codebook(4)[0], tq.build_codebook(3)[0]
    with pytest.raises(ValueError, match="workspace"):
        _tree_call(rot, 4, 3, kc, vc, workspace=workspace)


def test_python_refusals_name_the_tensor(rot):
    """What test_python_refuses_misread_tensors refuses, by message: tensors on the CPU
    raise ValueError at the latest, whatever else is wrong with them."""
    q, k = (torch.zeros((4, h, 128), dtype=torch.bfloat16) for h in (4, 2))
    cu = _i32(3)

    def refused(match, call, **bad):
        with pytest.raises(ValueError, match=match):
            call(**bad)

    def prompt_(q=q, k=k, v=k, cu_q=cu, **kw):
        tq.prompt_attention(q, k, v, cu_q, **kw)
    refused("not on a CUDA device", prompt_)
    refused("^cu_q:", prompt_, cu_q=cu.long())
    refused("^cu_q:", prompt_, cu_q=_i32(6)[::2])
    refused("^k:", prompt_, q=q.half())
    refused("^q:", prompt_, q=torch.zeros((4, 128, 4), dtype=torch.bfloat16).transpose(1, 2))
    refused("^k:", prompt_, k=k[:, :, ::2])
    refused("^v:", prompt_, v=k[:3])
    refused("^v:", prompt_, v=q)
    refused("^cu_k:", prompt_, cu_k=_i32(4))
    refused("^out:", prompt_, out=q.float())
    refused("^out:", prompt_, out=q.transpose(0, 1).contiguous().transpose(0, 1))
    refused("^cu_k is needed", prompt_, k=torch.zeros((5, 2, 128), dtype=torch.bfloat16),
            v=torch.zeros((5, 2, 128), dtype=torch.bfloat16))

    def tables_(ctx=_i32(2), new=_i32(2), free=_i32(4), table=_i32(2, 2), n_slots=8, **kw):
        tq.page_tables(ctx, new, 16, 4, free, table, n_slots, **kw)
    out = dict(cu_new=_i32(3), total_lens=_i32(2), slots=torch.zeros(8, dtype=torch.int64), positions=_i32(8), n_taken=_i32(1))
    refused("not on a CUDA device", tables_)
    refused("not on a CUDA device", tables_, out=out)
    refused("^ctx_lens:", tables_, ctx=_i32(2).long())
    refused("^new_lens:", tables_, new=_i32(3))
    refused("^free_pages:", tables_, free=_i32(8)[::2])
    refused("^block_table:", tables_, table=_i32(3, 2))
    refused("^block_table:", tables_, table=_i32(2, 4)[:, ::2])
    for name, wrong in (("cu_new", _i32(2)), ("total_lens", _i32(3)), ("slots", _i32(8)), ("positions", _i32(7)),
                        ("n_taken", torch.zeros(1))):
        refused(f"^{name}:", tables_, out=dict(out, **{name: wrong}))

    (kc, kt), vc = tq.build_codebook(4), tq.build_codebook(3)[0]
    slots, codes, norms = torch.zeros(4, dtype=torch.int64), _i32(3, 2, 16, 16), torch.zeros((3, 2, 16, 4), dtype=torch.int16)

    def paged_(x=k, slots=slots, codes=codes, norms=norms):
        tq.quantize_kv_paged(rot, 4, kc, kt, x, slots, codes, norms, 16)
    refused("not on a CUDA device", paged_)
    refused("^slots:", paged_, slots=slots.int())
    refused("^slots:", paged_, slots=slots[:3])
    refused("^codes:", paged_, codes=_i32(3, 2, 16, 12))
    refused("^codes:", paged_, codes=_i32(3, 1, 16, 16))
    refused("^norms:", paged_, norms=norms.half())
    refused("^norms:", paged_, norms=norms[:2])
    refused("^x:", paged_, x=q[:, ::2])

    pages = dict(k_codes=codes, k_norms=norms, v_codes=_i32(3, 2, 16, 12), v_norms=norms)
    mask, ws = torch.zeros((4, 1), dtype=torch.int64), torch.zeros(256, dtype=torch.uint8)

    def tree_(q=q, cu=_i32(3), lens=_i32(2), pages=pages, table=_i32(2, 4), mask=mask, **kw):
        tq.tree_attention(rot, 4, 3, kc, vc, q, cu, lens, pages, table, 16, 2, 64, tree_mask=mask, workspace=ws, **kw)
    refused("not on a CUDA device", tree_)
    refused("^cu_nodes:", tree_, cu=_i32(2))
    refused("^lens:", tree_, lens=_i32(2).long())
    refused("^tree_mask:", tree_, mask=mask.int())
    refused("^tree_mask:", tree_, mask=mask[:3])
    refused("^tree_mask:", tree_, mask=mask[:, 0])
    refused("^block_table:", tree_, table=_i32(3, 4))
    refused("^q and out:", tree_, q=q[:, ::2])
    refused("^q and out:", tree_, out=q.half())
    for name in pages:
        refused(f"^{name}:", tree_, pages=dict(pages, **{name: _i32(3, 2, 16, 5)}))


def test_python_refuses_a_rotation_of_another_device(rot):
    """A dense rotation's matrix lies on the device that it was made on."""
    class Dense:
        handle, device = rot.handle, 3
    (kc, kt), vc = tq.build_codebook(4), tq.build_codebook(3)[0]
    assert rot.device is None
    with pytest.raises(ValueError, match="^rotation: made on cuda:3"):
        _quantize_call(Dense, 4, kc, kt)
    with pytest.raises(ValueError, match="^rotation: made on cuda:3"):
        _tree_call(Dense, 4, 3, kc, vc)
