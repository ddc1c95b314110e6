"""ctypes binding of libtq.so (argument marshalling only)."""

import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libtq.so")

if not os.path.exists(_LIB_PATH):
    raise ImportError(
        f"{_LIB_PATH} is missing: build it with `python kv_cache_vector_11_b200/build.py` "
        "(there is no CPU fallback)")

_lib = ctypes.CDLL(_LIB_PATH)

FORMAT_VERSION = 1
STATUS_NORM_SATURATED = 1
STATUS_NONFINITE = 2
STATUS_TIMEOUT = 4
STATUS_NO_PAGES = 8
STATUS_BAD_PAGE = 16
STATUS_LIMIT = 32
FMT_NORM_F32 = 1
FMT_NORM_CORRECTED = 2
FMT_GROUPED = 4

ROT_KINDS = {"wht": 0, "haar": 1, "gauss": 2}
DTYPES = {"f32": 0, "bf16": 1, "f16": 2}

_c = ctypes
_vp = _c.c_void_p
_i32 = _c.c_int32
_i64 = _c.c_int64
_u64 = _c.c_uint64

_SIGS = {
    "tq_rotation_generate": (_i32, [_i32, _i32, _i32, _u64, _vp]),
    "tq_make_rotation": (_i32, [_i32, _i32, _i32, _u64, _c.POINTER(_vp)]),
    "tq_free_rotation": (None, [_vp]),
    "tq_rotation_copy_host": (_i32, [_vp, _vp]),
    "tq_rotation_info": (_i32, [_vp, _vp, _vp, _vp, _vp]),
    "tq_build_codebook": (_i32, [_i32, _i32, _vp, _vp]),
    "tq_code_words_per_row": (_i64, [_i32, _i32, _i32]),
    "tq_quantize_kv": (_i32, [_vp, _i32, _i32, _vp, _vp, _vp, _vp, _i32, _i64, _i32,
                               _vp, _vp, _vp, _vp, _vp, _vp]),
    "tq_quantize_kv_ex": (_i32, [_vp, _i32, _i32, _vp, _vp, _vp, _vp, _i32, _i64, _i32, _c.c_uint32,
                                  _vp, _vp, _vp, _vp, _vp, _vp]),
    "tq_attn_logits_ex": (_i32, [_vp, _i32, _i32, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i64,
                                  _i32, _c.c_uint32, _vp, _vp, _vp, _vp, _vp, _vp]),
    "tq_decode_attention_ex": (_i32, [_vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _i32, _i32, _i32,
                                       _i32, _i64, _i32, _c.c_uint32, _vp, _vp, _vp, _vp, _vp, _vp,
                                       _c.c_float, _vp, _vp, _c.c_size_t, _vp]),
    "tq_attn_logits": (_i32, [_vp, _i32, _i32, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i64,
                               _i32, _vp, _vp, _vp, _vp, _vp, _vp]),
    "tq_decode_workspace_size": (_c.c_size_t, [_i32, _i32, _i32, _i64, _i32]),
    "tq_decode_attention": (_i32, [_vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _i32, _i32, _i32,
                                    _i32, _i64, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _c.c_float,
                                    _vp, _vp, _c.c_size_t, _vp]),
    "tq_decode_attention_static": (_i32, [_vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _i32, _i32,
                                           _i32, _i32, _i64, _i32, _vp, _vp, _vp, _vp, _vp, _vp,
                                           _c.c_float, _vp, _vp]),
    "tq_decode_append_paged": (_i32, [_vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _i32, _vp,
                                       _vp, _i32, _i32, _i32, _i32, _i64, _i32, _i32, _i32, _vp,
                                       _i32, _vp, _vp, _vp, _vp, _c.c_float, _vp, _vp, _c.c_size_t,
                                       _vp, _vp]),
    "tq_search_workspace_size": (_c.c_size_t, [_i32, _i64, _i32, _i32]),
    "tq_search_topk": (_i32, [_vp, _i32, _i32, _vp, _vp, _i32, _i32, _i32, _vp, _vp, _i64, _i32,
                              _vp, _vp, _vp, _c.c_size_t, _vp]),
    "tq_page_tables": (_i32, [_vp, _vp, _i32, _i32, _i32, _vp, _i32, _vp, _i32, _vp, _vp, _vp, _vp,
                              _i32, _vp, _vp, _vp]),
    "tq_quantize_kv_paged": (_i32, [_vp, _i32, _i32, _vp, _vp, _vp, _i32, _i64, _i32, _i32, _vp,
                                    _i32, _i32, _vp, _vp, _vp, _vp]),
    "tq_prompt_attention": (_i32, [_vp, _vp, _vp, _i32, _vp, _vp, _i32, _i64, _i64, _i32, _i32, _i32,
                                   _i64, _i64, _i64, _c.c_float, _vp, _vp, _vp]),
    "tq_tree_workspace_size": (_c.c_size_t, [_i32, _i32, _i32, _i32, _i32, _i64, _i32]),
    "tq_tree_attention": (_i32, [_vp, _i32, _i32, _i32, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32,
                                 _vp, _i64, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _vp, _i32,
                                 _vp, _vp, _vp, _vp, _c.c_float, _vp, _vp, _c.c_size_t, _vp, _vp]),
    "tq_status_string": (_c.c_char_p, [_i32]),
    "tq_last_error": (_c.c_char_p, []),
}

for _name, (_res, _args) in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args


def lib_path():
    return _LIB_PATH


def exported_symbols():
    """Names of the C entry points this binding uses (all declared in tq.h)."""
    return sorted(_SIGS)


class TQError(RuntimeError):
    def __init__(self, status, where):
        reason = _lib.tq_last_error().decode()
        super().__init__(f"{where}: {_lib.tq_status_string(status).decode()} ({reason})")
        self.status = status


def _check(status, where):
    if status != 0:
        raise TQError(status, where)


def _ptr(t):
    """Device or host pointer of a torch tensor / numpy array (None -> NULL)."""
    if t is None:
        return None
    if isinstance(t, np.ndarray):
        return t.ctypes.data
    return t.data_ptr()


def _stream_ptr(stream, device):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return stream.cuda_stream


def _on(device):
    """Make ``device`` the current CUDA device for the C call: the library
    resolves per-device state (SM count, shared-memory limits, the static
    scratch address) through the current device."""
    import torch
    return torch.cuda.device(device)


def _empty(shape, dtype, device, stream, returned=True):
    """Memory that a call on ``stream`` allocates itself.  It comes from that
    stream's own blocks: one that the current stream gave back may still be read
    or written there, by work which ``stream`` does not wait for.  What the call
    returns is used on the current stream, and not given out again before that
    stream is done with it."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if returned:
        t.record_stream(torch.cuda.current_stream(device))
    return t


def rotation_generate(kind, rows, cols, seed):
    """Dense float64 matrix of a seeded rotation / projection (host only)."""
    out = np.empty((rows, cols), dtype=np.float64)
    _check(_lib.tq_rotation_generate(ROT_KINDS[kind], rows, cols, seed, out.ctypes.data),
           "tq_rotation_generate")
    return out


def build_codebook(bits, block=32):
    """(centroids fp32 [2^bits], boundaries fp32 [2^bits - 1]) (host only)."""
    c = np.empty(1 << bits, dtype=np.float32)
    t = np.empty((1 << bits) - 1, dtype=np.float32)
    _check(_lib.tq_build_codebook(bits, block, c.ctypes.data, t.ctypes.data), "tq_build_codebook")
    return c, t


def code_words_per_row(bits, block, head_dim):
    return int(_lib.tq_code_words_per_row(bits, block, head_dim))


class Rotation:
    """Owning wrapper of a tq_rotation handle on the current CUDA device."""

    def __init__(self, kind, rows, cols, seed):
        h = _vp()
        _check(_lib.tq_make_rotation(ROT_KINDS[kind], rows, cols, seed, _c.byref(h)),
               "tq_make_rotation")
        self._h = h
        self.kind, self.rows, self.cols, self.seed = kind, rows, cols, seed
        self.device = None                              # of the matrix; a WHT has none on the device
        if kind != "wht":
            import torch
            self.device = torch.cuda.current_device()

    @property
    def handle(self):
        return self._h

    def matrix(self):
        out = np.empty((self.rows, self.cols), dtype=np.float64)
        _check(_lib.tq_rotation_copy_host(self._h, out.ctypes.data), "tq_rotation_copy_host")
        return out

    def info(self):
        kind, rows, cols, seed = _i32(), _i32(), _i32(), _u64()
        _check(_lib.tq_rotation_info(self._h, _c.byref(kind), _c.byref(rows), _c.byref(cols),
                                     _c.byref(seed)), "tq_rotation_info")
        return kind.value, rows.value, cols.value, seed.value

    def close(self):
        if getattr(self, "_h", None):
            _lib.tq_free_rotation(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _dtype_code(t):
    import torch
    if t.dtype == torch.bfloat16:
        return DTYPES["bf16"]
    if t.dtype == torch.float32:
        return DTYPES["f32"]
    raise TypeError(f"unsupported dtype {t.dtype}")


def _format(norm_f32, norm_correction, grouped=False):
    return ((FMT_NORM_F32 if norm_f32 else 0) | (FMT_NORM_CORRECTED if norm_correction else 0) |
            (FMT_GROUPED if grouped else 0))


def quantize_kv(rot, bits, centroids, boundaries, x, qjl=None, block=32, out=None,
                status=None, stream=None, norm_f32=False, norm_correction=False, grouped=False):
    """Quantize rows x [n_rows, head_dim] (bf16 or fp32, CUDA) with ``rot``.

    Returns dict(codes=uint32-as-int32 [n, W], norms=fp16 bits as int16 (fp32
    with ``norm_f32``) [n, d/block], and, with ``qjl``, signs [n, m/32], rnorm
    [n]).  ``out`` may supply those tensors to write into.  ``centroids`` and
    ``boundaries`` are the codebook of ``block``.  ``grouped`` writes the codes
    in the lane-grouped row order (TQ_FMT_GROUPED: value caches, bf16, d = 128).
    """
    import torch
    n, d = x.shape
    w = max(code_words_per_row(bits, block, d), 0)   # -1 for an unsupported block: the call rejects it
    dev = x.device
    if out is None:
        out = {"codes": _empty((n, w), torch.int32, dev, stream),
               "norms": _empty((n, max(d // block, 0)), torch.float32 if norm_f32 else torch.int16, dev, stream)}
        if qjl is not None:
            out["signs"] = _empty((n, qjl.rows // 32), torch.int32, dev, stream)
            out["rnorm"] = _empty((n,), torch.int16, dev, stream)
    c = np.ascontiguousarray(centroids, dtype=np.float32)
    t = np.ascontiguousarray(boundaries, dtype=np.float32)
    with _on(dev):
        _check(_lib.tq_quantize_kv_ex(
            rot.handle, bits, block, c.ctypes.data, t.ctypes.data,
            qjl.handle if qjl is not None else None,
            _ptr(x), _dtype_code(x), n, d, _format(norm_f32, norm_correction, grouped),
            _ptr(out["codes"]), _ptr(out["norms"]), _ptr(out.get("signs")), _ptr(out.get("rnorm")),
            _ptr(status), _stream_ptr(stream, dev)), "tq_quantize_kv_ex")
    return out


def attn_logits(rot, k_bits, k_centroids, q, k_codes, k_norms, n_kv_heads, ctx, qjl=None,
                qjl_signs=None, qjl_rnorm=None, block=32, logits=None, stream=None,
                norm_f32=False):
    """Raw scores [batch, n_q_heads, ctx] (fp32, CUDA) of q [batch, n_q_heads, d]."""
    import torch
    batch, n_q, d = q.shape
    if logits is None:
        logits = _empty((batch, n_q, ctx), torch.float32, q.device, stream)
    c = np.ascontiguousarray(k_centroids, dtype=np.float32)
    with _on(q.device):
        _check(_lib.tq_attn_logits_ex(
            rot.handle, k_bits, block, c.ctypes.data, qjl.handle if qjl is not None else None,
            _ptr(q), _dtype_code(q), batch, n_q, n_kv_heads, ctx, d, _format(norm_f32, False),
            _ptr(k_codes), _ptr(k_norms), _ptr(qjl_signs), _ptr(qjl_rnorm), _ptr(logits),
            _stream_ptr(stream, q.device)), "tq_attn_logits_ex")
    return logits


def decode_workspace_size(batch, n_q_heads, n_kv_heads, ctx, head_dim):
    return int(_lib.tq_decode_workspace_size(batch, n_q_heads, n_kv_heads, ctx, head_dim))


def decode_attention(rot, k_bits, v_bits, k_centroids, v_centroids, q, k_codes, k_norms,
                     v_codes, v_norms, n_kv_heads, ctx, qjl=None, qjl_signs=None,
                     qjl_rnorm=None, scale=0.0, block=32, out=None, workspace=None,
                     stream=None, norm_f32=False, v_grouped=False):
    """Decode output [batch, n_q_heads, d] (fp32, CUDA).  ``v_grouped``: the
    value codes are in the lane-grouped row order (TQ_FMT_GROUPED)."""
    import torch
    batch, n_q, d = q.shape
    if out is None:
        out = _empty((batch, n_q, d), torch.float32, q.device, stream)
    with _on(q.device):
        need = decode_workspace_size(batch, n_q, n_kv_heads, ctx, d)
        if workspace is None:
            workspace = _empty((max(need, 16),), torch.uint8, q.device, stream, returned=False)
        kc = np.ascontiguousarray(k_centroids, dtype=np.float32)
        vc = np.ascontiguousarray(v_centroids, dtype=np.float32)
        _check(_lib.tq_decode_attention_ex(
            rot.handle, k_bits, v_bits, block, kc.ctypes.data, vc.ctypes.data,
            qjl.handle if qjl is not None else None,
            _ptr(q), _dtype_code(q), batch, n_q, n_kv_heads, ctx, d,
            _format(norm_f32, False, v_grouped),
            _ptr(k_codes), _ptr(k_norms), _ptr(qjl_signs), _ptr(qjl_rnorm),
            _ptr(v_codes), _ptr(v_norms), float(scale), _ptr(out),
            _ptr(workspace), workspace.numel() * workspace.element_size(),
            _stream_ptr(stream, q.device)), "tq_decode_attention_ex")
    return out


DECODE_STATIC_SCRATCH_BYTES = 16 << 20


def decode_attention_static(rot, k_bits, v_bits, k_centroids, v_centroids, q, k_codes, k_norms,
                            v_codes, v_norms, n_kv_heads, ctx, qjl=None, qjl_signs=None,
                            qjl_rnorm=None, scale=0.0, block=32, out=None, stream=None):
    """``decode_attention`` without a workspace, for callers that cannot
    allocate device memory on the call path (engine plugins that must not
    allocate while enqueueing, servers that hand out memory only from a
    pre-reserved arena, loops that must avoid cudaMalloc's implicit device
    synchronisation).  The split partials live in a fixed 16 MiB array inside
    the library; larger shapes raise TQError.  Calls that overlap on the GPU
    share that array and race, so issue them on one stream.  ``out`` may be
    passed in so the call itself allocates nothing."""
    import torch
    batch, n_q, d = q.shape
    if out is None:
        out = _empty((batch, n_q, d), torch.float32, q.device, stream)
    kc = np.ascontiguousarray(k_centroids, dtype=np.float32)
    vc = np.ascontiguousarray(v_centroids, dtype=np.float32)
    with _on(q.device):
        _check(_lib.tq_decode_attention_static(
            rot.handle, k_bits, v_bits, block, kc.ctypes.data, vc.ctypes.data,
            qjl.handle if qjl is not None else None,
            _ptr(q), _dtype_code(q), batch, n_q, n_kv_heads, ctx, d,
            _ptr(k_codes), _ptr(k_norms), _ptr(qjl_signs), _ptr(qjl_rnorm),
            _ptr(v_codes), _ptr(v_norms), float(scale), _ptr(out),
            _stream_ptr(stream, q.device)), "tq_decode_attention_static")
    return out


def search_workspace_size(n_queries, n_db, head_dim, k):
    return int(_lib.tq_search_workspace_size(n_queries, n_db, head_dim, k))


def search_topk(rot, bits, centroids, q, db_codes, db_norms, k, block=32, workspace=None,
                stream=None):
    """Top-k maximum-inner-product search of queries q [n_q, head_dim] (bf16
    or fp32, CUDA) over packed database rows; returns (scores fp32 [n_q, k],
    rows int32 [n_q, k])."""
    import torch
    n_q, d = q.shape
    n_db = db_codes.shape[0]
    scores = _empty((n_q, k), torch.float32, q.device, stream)
    rows = _empty((n_q, k), torch.int32, q.device, stream)
    c = np.ascontiguousarray(centroids, dtype=np.float32)
    with _on(q.device):
        need = search_workspace_size(n_q, n_db, d, k)
        if workspace is None:
            workspace = _empty((max(need, 256),), torch.uint8, q.device, stream, returned=False)
        _check(_lib.tq_search_topk(
            rot.handle, bits, block, c.ctypes.data, _ptr(q), _dtype_code(q), n_q, d,
            _ptr(db_codes), _ptr(db_norms), n_db, k, _ptr(scores), _ptr(rows), _ptr(workspace),
            workspace.numel() * workspace.element_size(), _stream_ptr(stream, q.device)),
            "tq_search_topk")
    return scores, rows


def decode_append_paged(rot, k_bits, v_bits, k_codebook, v_codebook, q, k_new, v_new, pages,
                        block_table, n_kv_heads, ctx, page_size, scale=0.0, out=None,
                        workspace=None, status=None, stream=None):
    """One decode step that first appends the step's token: k_new / v_new
    [batch, n_kv_heads, head_dim] are quantized into token ctx - 1 of the paged
    cache ``pages`` (dict of k_codes, k_norms, v_codes, v_norms, each
    [n_pages, n_kv_heads, page_size, ...] on the device) through
    ``block_table`` (int32 [batch, max_pages]); returns the attention output
    [batch, n_q_heads, head_dim] over tokens 0 .. ctx - 1.  ``k_codebook`` and
    ``v_codebook`` are (centroids, boundaries) pairs."""
    import torch
    batch, n_q, d = q.shape
    if out is None:
        out = _empty((batch, n_q, d), torch.float32, q.device, stream)
    kc = np.ascontiguousarray(k_codebook[0], dtype=np.float32)
    kt = np.ascontiguousarray(k_codebook[1], dtype=np.float32)
    vc = np.ascontiguousarray(v_codebook[0], dtype=np.float32)
    vt = np.ascontiguousarray(v_codebook[1], dtype=np.float32)
    n_pages = pages["k_codes"].shape[0]
    with _on(q.device):
        need = decode_workspace_size(batch, n_q, n_kv_heads, ctx, d)
        if workspace is None:
            workspace = _empty((max(need, 16),), torch.uint8, q.device, stream, returned=False)
        _check(_lib.tq_decode_append_paged(
            rot.handle, k_bits, v_bits, 32, kc.ctypes.data, kt.ctypes.data, vc.ctypes.data,
            vt.ctypes.data, _ptr(q), _dtype_code(q), _ptr(k_new), _ptr(v_new), _dtype_code(k_new),
            batch, n_q, n_kv_heads, ctx, d, page_size, n_pages, _ptr(block_table),
            block_table.shape[1], _ptr(pages["k_codes"]), _ptr(pages["k_norms"]),
            _ptr(pages["v_codes"]), _ptr(pages["v_norms"]), float(scale), _ptr(out),
            _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(status),
            _stream_ptr(stream, q.device)), "tq_decode_append_paged")
    return out


def _require(ok, what):
    if not ok:
        raise ValueError(what)


def _dtype_code16(t):
    """As _dtype_code, and fp16 (prompt and tree attention)."""
    import torch
    return DTYPES["f16"] if t.dtype == torch.float16 else _dtype_code(t)


def _ints(t, n, name, device, kind):
    """Pointer of a contiguous integer array of n entries on ``device`` (the
    kernels read it without further checks).  Here and below a message is put
    together only where it is raised (the strings of calls that pass were 4 of
    the 10 us that prompt_attention's checks took)."""
    if not (t.dtype is kind and t.numel() == n and t.is_contiguous() and t.device == device):
        raise ValueError(f"{name}: contiguous {kind} of {n} entries on {device}")
    return t.data_ptr()


def _rotation(rot, device):
    """Handle of a rotation whose matrix, if it has one, lies on ``device``."""
    if rot.device is not None and rot.device != device.index:
        raise ValueError(f"rotation: made on cuda:{rot.device}, used on {device}")
    return rot.handle


def _status_ptr(t, device):
    """Pointer of the status word (None: none is kept)."""
    import torch
    if t is None:
        return None
    if not (t.device == device and t.dtype in (torch.int32, torch.uint32) and t.numel() > 0):
        raise ValueError(f"status: int32 of at least one entry on {device}")
    return t.data_ptr()


def _page_part(t, name, kind, shape, device):
    """Pointer of one array of the page storage, [page][kv head][token][..]."""
    if not (t.shape == shape and t.dtype is kind and t.is_contiguous() and t.device == device):
        raise ValueError(f"{name}: contiguous {kind} {list(shape)} on {device}")
    return t.data_ptr()


def _host_floats(x, n, name):
    """The n values of x as fp32 in a bytes object, which ctypes passes as a
    pointer (0.3 us; an array's address by ``ndarray.ctypes`` takes several times
    that).  The library reads n of them whatever x holds."""
    b = np.ascontiguousarray(x, dtype=np.float32).tobytes()
    if len(b) != 4 * n:
        raise ValueError(f"{name}: {n} values, not {len(b) // 4}")
    return b


def _stream_of(device):
    """Handle of the current stream of a CUDA device.  Read without building a
    Stream object (2 us of a call that takes 12) where torch offers that."""
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(device.index) if raw is not None else torch.cuda.current_stream(device).cuda_stream


def _launch(fn, where, device, stream, *args):
    """fn(*args, stream) with ``device`` current (as _on; a serving step makes
    many short calls, so nothing is switched that is current already)."""
    import torch
    if device.type != "cuda":
        raise ValueError(f"{where}: tensors on {device}, not on a CUDA device")
    handle = _stream_of(device) if stream is None else stream.cuda_stream
    if torch.cuda.current_device() == device.index:
        status = fn(*args, handle)
    else:
        with torch.cuda.device(device):
            status = fn(*args, handle)
    if status != 0:
        raise TQError(status, where)


def page_tables(ctx_lens, new_lens, page_size, n_pages, free_pages, block_table, n_slots, out=None,
                status=None, stream=None):
    """Block tables and slot maps from request lengths: request b holds
    ctx_lens[b] tokens and gets new_lens[b] more (int32 [batch], CUDA).  Pages
    come from the front of ``free_pages`` (int32 [n_free]) in request order and
    are written into ``block_table`` (int32 [batch, max_pages]) in place.

    Returns dict(cu_new int32 [batch + 1], total_lens int32 [batch], slots
    int64 [n_slots], positions int32 [n_slots], n_taken int32 [1]); slots and
    positions are -1 past the last token and for requests that were not placed
    (STATUS_NO_PAGES in ``status``).  ``out`` may supply those tensors."""
    import torch
    dev = ctx_lens.device
    batch = ctx_lens.shape[0]
    if out is None:
        out = {"cu_new": _empty((batch + 1,), torch.int32, dev, stream),
               "total_lens": _empty((batch,), torch.int32, dev, stream),
               "slots": _empty((n_slots,), torch.int64, dev, stream),
               "positions": _empty((n_slots,), torch.int32, dev, stream),
               "n_taken": _empty((1,), torch.int32, dev, stream)}
    i32 = torch.int32
    _require(block_table.dim() == 2 and block_table.shape[0] == batch, "block_table: [batch, max_pages]")
    n_free, max_pages = free_pages.numel(), block_table.shape[1]
    positions = out.get("positions")
    args = (_ints(ctx_lens, batch, "ctx_lens", dev, i32), _ints(new_lens, batch, "new_lens", dev, i32), batch,
            page_size, n_pages, _ints(free_pages, n_free, "free_pages", dev, i32), n_free,
            _ints(block_table, batch * max_pages, "block_table", dev, i32), max_pages,
            _ints(out["cu_new"], batch + 1, "cu_new", dev, i32),
            _ints(out["total_lens"], batch, "total_lens", dev, i32),
            _ints(out["slots"], n_slots, "slots", dev, torch.int64),
            None if positions is None else _ints(positions, n_slots, "positions", dev, i32), n_slots,
            _ints(out["n_taken"], 1, "n_taken", dev, i32), _status_ptr(status, dev))
    _launch(_lib.tq_page_tables, "tq_page_tables", dev, stream, *args)
    return out


def quantize_kv_paged(rot, bits, centroids, boundaries, x, slots, codes, norms, page_size, block=32,
                      status=None, stream=None):
    """Quantize rows x [n_tokens, n_kv_heads, head_dim] (bf16 or fp32, CUDA)
    into page storage: token i goes to ``slots[i]`` (int64, as page_tables
    returns them; negative = not stored) of ``codes`` int32 [n_pages,
    n_kv_heads, page_size, W] and ``norms`` int16 [n_pages, n_kv_heads,
    page_size, head_dim / 32].  Same bits as ``quantize_kv``."""
    import torch
    n, heads, d = x.shape
    dev = x.device
    n_pages = codes.shape[0]
    w = d * bits // 32                                  # (the library refuses other blocks and widths)
    _require(x.is_contiguous(), "x: contiguous [n_tokens, n_kv_heads, head_dim]")
    slots_p = _ints(slots, n, "slots", dev, torch.int64)
    codes_p = _page_part(codes, "codes", torch.int32, (n_pages, heads, page_size, w), dev)
    norms_p = _page_part(norms, "norms", torch.int16, (n_pages, heads, page_size, d // 32), dev)
    _launch(_lib.tq_quantize_kv_paged, "tq_quantize_kv_paged", dev, stream, _rotation(rot, dev), bits, block,
            _host_floats(centroids, 1 << bits, "centroids"), _host_floats(boundaries, (1 << bits) - 1, "boundaries"),
            x.data_ptr(), _dtype_code(x), n, heads, d,
            slots_p, page_size, n_pages, codes_p, norms_p, _status_ptr(status, dev))


def prompt_attention(q, k, v, cu_q, cu_k=None, scale=0.0, out=None, status=None, stream=None):
    """Causal attention of packed sequences: q [total_q, n_q_heads, head_dim],
    k and v [total_k, n_kv_heads, head_dim] (bf16 or fp16, CUDA; the tokens may
    be strided, as slices of a fused projection are), offsets cu_q and cu_k
    int32 [batch + 1] (cu_k defaults to cu_q).  With fewer queries than keys
    the queries are the last ones.  Returns out, of q's type and shape; rows
    past cu_q[batch] are left as they are.  Offsets past the arrays are cut there
    and set STATUS_LIMIT in ``status``."""
    import torch
    total_q, n_q, d = q.shape
    total_k, n_kv, _ = k.shape
    dev = q.device
    if out is None:
        out = _empty((total_q, n_q, d), q.dtype, dev, stream)
    kind = q.dtype
    strides = []
    for name, t, n, h in (("q", q, total_q, n_q), ("k", k, total_k, n_kv), ("v", v, total_k, n_kv)):
        st = t.stride()
        if not (t.shape == (n, h, d) and t.dtype is kind and t.device == dev and st[2] == 1 and
                (h == 1 or st[1] == d)):
            raise ValueError(f"{name}: [{n}, {h}, {d}] rows of q's type, contiguous within a token")
        strides.append(st[0] if n > 1 else h * d)
    _require(out.shape == q.shape and out.dtype is kind and out.is_contiguous() and out.device == dev,
             "out: contiguous, of q's shape and type")
    batch = cu_q.numel() - 1
    cu_q_p = _ints(cu_q, batch + 1, "cu_q", dev, torch.int32)
    cu_k_p = None
    if cu_k is not None:
        cu_k_p = _ints(cu_k, batch + 1, "cu_k", dev, torch.int32)
    else:
        _require(total_k == total_q, "cu_k is needed where k has another length than q")
    _launch(_lib.tq_prompt_attention, "tq_prompt_attention", dev, stream, q.data_ptr(), k.data_ptr(), v.data_ptr(),
            _dtype_code16(q), cu_q_p, cu_k_p, batch, total_q, total_k, n_q, n_kv, d, *strides, float(scale),
            out.data_ptr(), _status_ptr(status, dev))
    return out


def tree_workspace_size(batch, n_rows, max_nodes, n_q_heads, n_kv_heads, max_len, head_dim):
    return int(_lib.tq_tree_workspace_size(batch, n_rows, max_nodes, n_q_heads, n_kv_heads, max_len,
                                           head_dim))


def tree_attention(rot, k_bits, v_bits, k_centroids, v_centroids, q, cu_nodes, lens, pages,
                   block_table, page_size, max_nodes, max_len, tree_mask=None, scale=0.0, block=32,
                   out=None, workspace=None, status=None, stream=None):
    """Attention of each request's newest tokens over its paged cache: q
    [n_rows, n_q_heads, head_dim] (bf16, fp16 or fp32, CUDA) holds request b's
    nodes at rows cu_nodes[b] .. (int32 [batch + 1]), the cached tokens
    lens[b] - n .. lens[b] - 1 of its ``lens[b]`` (int32 [batch], at most
    ``max_len``).  Node i attends all tokens before the nodes and the nodes
    whose bits are set in ``tree_mask`` (int64 [n_rows, words], 64 nodes to a
    word); without a mask the nodes 0 .. i.  ``pages`` and ``block_table`` as
    in decode_append_paged.  Returns out, of q's type and shape.

    The lengths stay on the device, so the host does not see them exceed the
    call's sizes: rows of nodes from ``max_nodes`` on are left as they were,
    lengths are cut at ``max_len``, and STATUS_LIMIT is set in ``status``."""
    import torch
    n_rows, n_q, d = q.shape
    dev = q.device
    batch = lens.shape[0]
    if out is None:
        out = _empty((n_rows, n_q, d), q.dtype, dev, stream)
    _require(q.is_contiguous() and out.shape == q.shape and out.dtype == q.dtype and
             out.is_contiguous() and out.device == dev, "q and out: contiguous, same shape and type")
    cu_p = _ints(cu_nodes, batch + 1, "cu_nodes", dev, torch.int32)
    lens_p = _ints(lens, batch, "lens", dev, torch.int32)
    _require(block_table.dim() == 2 and block_table.shape[0] == batch, "block_table: [batch, max_pages]")
    max_pages = block_table.shape[1]
    table_p = _ints(block_table, batch * max_pages, "block_table", dev, torch.int32)
    n_pages, n_kv = pages["k_codes"].shape[:2]
    # (the library refuses other blocks and widths)
    storage = [_page_part(pages[name], name, kind, (n_pages, n_kv, page_size, w), dev)
               for name, kind, w in (("k_codes", torch.int32, d * k_bits // 32), ("k_norms", torch.int16, d // 32),
                                     ("v_codes", torch.int32, d * v_bits // 32), ("v_norms", torch.int16, d // 32))]
    words, mask_p = 0, None
    if tree_mask is not None:
        _require(tree_mask.dim() == 2, "tree_mask: [n_rows, words]")
        words = tree_mask.shape[1]
        mask_p = _ints(tree_mask, n_rows * words, "tree_mask", dev, torch.int64)
    if workspace is None:
        with _on(dev):
            need = tree_workspace_size(batch, n_rows, max_nodes, n_q, n_kv, max_len, d)
        workspace = _empty((max(need, 256),), torch.uint8, dev, stream, returned=False)
    _require(workspace.device == dev and workspace.is_contiguous(), "workspace: contiguous, on q's device")
    _launch(_lib.tq_tree_attention, "tq_tree_attention", dev, stream, _rotation(rot, dev), k_bits, v_bits, block,
            _host_floats(k_centroids, 1 << k_bits, "k_centroids"), _host_floats(v_centroids, 1 << v_bits, "v_centroids"),
            q.data_ptr(), _dtype_code16(q), cu_p, batch, n_rows, max_nodes, lens_p, max_len, mask_p, words, n_q, n_kv, d,
            page_size, n_pages, table_p, max_pages, *storage, float(scale), out.data_ptr(), workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), _status_ptr(status, dev))
    return out
