"""Paged key / value cache: the pool and batch descriptors and the operators
over them (``qwen2_paged_*`` of ``include/qwen2.h``).

    pool = q2.PagedKV.zeros(n_pages, 64, n_kv_head, head_dim, q2.KV_INT8)
    batch = q2.PagedBatch(q_start, kv_len, pages, max_q)     # int32 CUDA tensors
    q = q2.paged_write(pool, batch, k, v, q=q, q_dtype=torch.bfloat16, rope=table)
    o = q2.paged_attention(pool, batch, q)

Argument marshalling only; every check that needs a value in device memory is
the kernels' own and is reported through ``PagedBatch.check``.  Calls do not
synchronise and may be captured into a CUDA graph: a replay reads the batch's
tensors anew.  Outputs and workspaces come from torch's allocator on the
stream of the call; threads may share a pool and a batch.
"""
from __future__ import annotations

import ctypes
from threading import get_ident as _thread

import numpy as np

KV_F16 = 0
KV_BF16 = 1
KV_INT8 = 2
KV_E4M3 = 3

ROPE_PLAIN = 0
ROPE_LINEAR = 1
ROPE_YARN = 2

_P, _I32, _I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64


class _Rows(ctypes.Structure):
    _fields_ = [("data", _P), ("dtype", _I32), ("row_stride", _I64), ("head_stride", _I64)]


class _PagedKV(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("k_scale", _P), ("v_scale", _P), ("format", _I32), ("n_pages", _I32),
                ("page_size", _I32), ("n_kv_head", _I32), ("head_dim", _I32), ("page_stride", _I64),
                ("token_stride", _I64), ("head_stride", _I64)]


class _PagedBatch(ctypes.Structure):
    _fields_ = [("n_seq", _I32), ("n_rows", _I32), ("max_q", _I32), ("max_pages", _I32), ("pages_stride", _I64),
                ("q_start", _P), ("kv_len", _P), ("pages", _P), ("guard", _P)]


class _WriteOpts(ctypes.Structure):
    _fields_ = [("q_norm", _P), ("k_norm", _P), ("norm_eps", ctypes.c_float), ("rope", _P), ("rope_rows", _I32),
                ("rotary_dim", _I32), ("interleaved", _I32)]


class _RopeScaling(ctypes.Structure):
    _fields_ = [("kind", _I32), ("factor", ctypes.c_double), ("original_rows", _I32),
                ("beta_fast", ctypes.c_double), ("beta_slow", ctypes.c_double)]


_bound = None


def _lib():
    global _bound
    if _bound is None:
        from . import lib
        L = lib()
        L.qwen2_rope_table.argtypes = [_I32, _I32, ctypes.c_double, _P, _P]
        L.qwen2_paged_write.argtypes = [_P, _P, _P, _I32, _P, _P, _P, _P, _P]
        L.qwen2_paged_read.argtypes = [_P, _P, _P, _I32, _P, _P, _P]
        L.qwen2_paged_attention.argtypes = [_P, _P, _I32, _P, _P, _P, ctypes.c_float, _I32, _P, _I64, _P]
        for f in (L.qwen2_rope_table, L.qwen2_paged_write, L.qwen2_paged_read, L.qwen2_paged_attention):
            f.restype = ctypes.c_int
        L.qwen2_paged_attention_workspace.argtypes = [_P, _P, _I32]
        L.qwen2_paged_attention_workspace.restype = _I64
        _bound = L
    return _bound


def _check(rc: int):
    if rc:
        from . import Qwen2Error
        raise Qwen2Error(rc, _lib().qwen2_last_error(None).decode())


_dtypes = {}     # torch dtype -> QWEN2_DTYPE_*
_formats = {}    # torch dtype -> QWEN2_KV_*
_t = None        # torch, once it is needed


def _types():
    global _t, _raw_stream, _capturing
    if _t is None:
        import torch
        _formats.update({torch.float16: KV_F16, torch.bfloat16: KV_BF16, torch.int8: KV_INT8,
                         torch.float8_e4m3fn: KV_E4M3})
        _dtypes.update({torch.float32: 0, torch.float16: 1, torch.bfloat16: 2})
        # The current stream's pointer, without building a Stream object for it.
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda index: torch.cuda.current_stream(index).cuda_stream)
        _capturing = torch.cuda.is_current_stream_capturing
        _t = torch
    return _t


def rope_table(rows: int, rotary_dim: int, theta: float = 1e6, kind: int = ROPE_PLAIN, factor: float = 1.0,
               original_rows: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0) -> np.ndarray:
    """(cos, sin) of position * theta^(-2i / rotary_dim), computed in double:
    f32 [rows, rotary_dim / 2, 2], host memory.  ``kind`` ROPE_LINEAR divides
    every angle by ``factor``; ROPE_YARN divides the slow dims' angles and
    scales the table (``original_rows``: the context trained at)."""
    out = np.empty((max(int(rows), 0), max(int(rotary_dim), 0) // 2, 2), dtype=np.float32)
    s = _RopeScaling(kind, factor, original_rows, beta_fast, beta_slow)
    _check(_lib().qwen2_rope_table(rows, rotary_dim, theta, ctypes.addressof(s), out.ctypes.data))
    return out


class PagedKV:
    """A pool of pages.  ``k``, ``v``: [n_pages, page_size, n_kv_head, head_dim]
    CUDA tensors (f16, bf16, int8 or float8_e4m3fn) of equal strides, the last
    dim contiguous; head-major pages are a permuted view.  ``k_scale``,
    ``v_scale`` (8-bit pools): f32 [n_pages, n_kv_head, page_size], contiguous."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        _types()
        if k.dim() != 4 or v.shape != k.shape:
            raise ValueError("k and v must be [n_pages, page_size, n_kv_head, head_dim]")
        if k.dtype not in _formats or v.dtype != k.dtype:
            raise ValueError(f"pages of {k.dtype} / {v.dtype} are not supported")
        if not (k.is_cuda and v.device == k.device):
            raise ValueError("k and v must be on one CUDA device")
        if v.stride() != k.stride() or k.stride(3) != 1:
            raise ValueError("k and v must have the same strides and contiguous heads")
        self.format = _formats[k.dtype]
        if self.format in (KV_INT8, KV_E4M3):
            want = (k.shape[0], k.shape[2], k.shape[1])
            for s in (k_scale, v_scale):
                if s is None or tuple(s.shape) != want or s.dtype != _t.float32 or \
                        s.device != k.device or not s.is_contiguous():
                    raise ValueError("8-bit pages need contiguous f32 scales [n_pages, n_kv_head, page_size]")
        else:
            k_scale = v_scale = None
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.device = k.device
        self.n_pages, self.page_size, self.n_kv_head, self.head_dim = k.shape
        self._c = _PagedKV(k.data_ptr(), v.data_ptr(), k_scale.data_ptr() if k_scale is not None else None,
                           v_scale.data_ptr() if v_scale is not None else None, self.format, self.n_pages,
                           self.page_size, self.n_kv_head, self.head_dim, *k.stride()[:3])
        self._at = ctypes.addressof(self._c)
        self._index = k.device.index

    @classmethod
    def zeros(cls, n_pages: int, page_size: int, n_kv_head: int, head_dim: int, format: int, device="cuda"):
        """A pool of zeroed, head-major pages."""
        torch = _types()
        dtype = next(d for d, f in _formats.items() if f == format)
        k, v = (torch.zeros((n_pages, n_kv_head, page_size, head_dim), dtype=torch.int8 if dtype.itemsize == 1 else dtype,
                            device=device).view(dtype).permute(0, 2, 1, 3) for _ in range(2))
        ks = vs = None
        if dtype.itemsize == 1:
            ks, vs = (torch.ones((n_pages, n_kv_head, page_size), dtype=torch.float32, device=device) for _ in range(2))
        return cls(k, v, ks, vs)


class PagedBatch:
    """The new rows of a batch and its pages, int32 CUDA tensors: ``q_start``
    [n_seq + 1] (row r of sequence s: q_start[s] <= r < q_start[s + 1]),
    ``kv_len`` [n_seq] (positions in the cache, the new rows included) and
    ``pages`` [n_seq, max_pages].  ``max_q``: an upper bound on the rows of one
    sequence.  The tensors are read by every call (and every graph replay)
    anew and may be changed in place between them."""

    def __init__(self, q_start, kv_len, pages, max_q: int):
        torch = _types()
        n = kv_len.shape[0] if kv_len.dim() == 1 else -1
        if n < 1 or tuple(q_start.shape) != (n + 1,) or pages.dim() != 2 or pages.shape[0] != n or pages.shape[1] < 1:
            raise ValueError("q_start must be [n_seq + 1], kv_len [n_seq] and pages [n_seq, max_pages]")
        for t in (q_start, kv_len, pages):
            if t.dtype != torch.int32 or not t.is_cuda or t.device != kv_len.device or t.stride(-1) != 1:
                raise ValueError("q_start, kv_len and pages must be int32 CUDA tensors, contiguous in their last dim")
        if n > 1 and pages.stride(0) < pages.shape[1]:
            raise ValueError("the rows of pages overlap")
        self.q_start, self.kv_len, self.pages = q_start, kv_len, pages
        self.device = kv_len.device
        self.n_seq, self.max_q = n, int(max_q)
        self.guard = torch.zeros(1, dtype=torch.int32, device=self.device)
        stride = max(pages.stride(0), pages.shape[1])
        self._c = _PagedBatch(n, 0, self.max_q, pages.shape[1], stride, q_start.data_ptr(), kv_len.data_ptr(),
                              pages.data_ptr(), self.guard.data_ptr())
        self._at = ctypes.addressof(self._c)
        self._space = {}      # workspace bytes by shapes
        self._buffers = {}    # workspaces by stream and thread

    def _with_rows(self, rows: int):
        """The batch's descriptor for a call with ``rows`` rows: the call's own,
        since calls from several threads may share the batch."""
        c = _PagedBatch.from_buffer_copy(self._c)
        c.n_rows = rows
        return c

    def check(self):
        """Synchronises, and raises Qwen2Error (QWEN2_E_DEVICE_GUARD) if a
        value in the batch's tensors was bad in any call since the last check."""
        from . import QWEN2_E_DEVICE_GUARD, Qwen2Error
        code = int(self.guard.item())
        if code:
            self.guard.zero_()
            names = {1: "position outside the pages or the rotation table", 3: "bad q_start", 4: "bounded wait timed out",
                     5: "page id outside the pool"}
            raise Qwen2Error(QWEN2_E_DEVICE_GUARD, f"device guard {code}: {names.get(code, 'unknown')}")


def _rows(t, name: str, heads, hd: int, rows, device):
    """The descriptor of a [rows, heads, head_dim] tensor (rows, heads: None for any)."""
    shape = t.shape
    if len(shape) != 3 or shape[2] != hd or (heads is not None and shape[1] != heads) or \
            (rows is not None and shape[0] != rows):
        raise ValueError(f"{name} must be [{'rows' if rows is None else rows}, {'heads' if heads is None else heads}, {hd}], "
                         f"not {list(shape)}")
    dt = _dtypes.get(t.dtype)
    if dt is None:
        raise ValueError(f"{name}: {t.dtype} is not supported")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    rs, hs, es = t.stride()
    if es != 1:
        raise ValueError(f"{name}: heads must be contiguous")
    return _Rows(t.data_ptr(), dt, rs, hs)


class _Call:
    """The stream of a call: the pool's device current and, where the caller
    names a stream, that stream current, so that outputs and workspaces are
    allocated for it."""

    def __init__(self, kv, batch, stream):
        if batch.device != kv.device:
            raise ValueError("the pool and the batch are on different devices")
        if stream is not None and stream.device != kv.device:
            raise ValueError("the stream belongs to another device")
        self.guard = _t.cuda.stream(stream) if stream is not None else _t.cuda.device(kv.device)

    def __enter__(self):
        self.guard.__enter__()

    def __exit__(self, *exc):
        return self.guard.__exit__(*exc)


def _plain(kv, batch, stream):
    """Whether a call needs no change of stream or device."""
    return stream is None and batch.device == kv.device and _t.cuda.current_device() == kv._index


def _f32(t, name: str, shape, device):
    if t.dtype != _t.float32 or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous f32 tensor of shape {list(shape)} on {device}")
    return t.data_ptr()


def paged_write(kv: PagedKV, batch: PagedBatch, k, v, q=None, q_out=None, q_dtype=None, q_norm=None, k_norm=None,
                norm_eps: float = 1e-6, rope=None, interleaved: bool = False, stream=None):
    """Store the batch's ``k``, ``v`` rows ([rows, n_kv_head, head_dim], f32 /
    f16 / bf16) in their pages, and return the finished queries of ``q``
    ([rows, n_head, head_dim]; None without).  ``q_norm`` / ``k_norm`` (f32
    [head_dim]): RMSNorm of every head; ``rope`` (f32 [positions, rotary_dim /
    2, 2], see rope_table): rotation of the leading rotary_dim dims of q and k
    at each row's position, dims paired (i, i + rotary_dim / 2) or, if
    ``interleaved``, (2i, 2i + 1).  Queries come in ``q_dtype`` (default: the
    pages' type if 16-bit, else q's if 16-bit, else f16)."""
    if not _plain(kv, batch, stream):
        with _Call(kv, batch, stream):
            return paged_write(kv, batch, k, v, q, q_out, q_dtype, q_norm, k_norm, norm_eps, rope, interleaved)
    dev, hd = kv.device, kv.head_dim
    rk = _rows(k, "k", kv.n_kv_head, hd, None, dev)
    rows = k.shape[0]
    rv = _rows(v, "v", kv.n_kv_head, hd, rows, dev)
    n_head, pq, po = 0, None, None
    if q is not None:
        rq = _rows(q, "q", None, hd, rows, dev)
        n_head = q.shape[1]
        if q_out is None:
            dt = q_dtype or (kv.k.dtype if kv.format <= KV_BF16 else q.dtype if q.dtype != _t.float32 else _t.float16)
            q_out = _t.empty((rows, n_head, hd), dtype=dt, device=dev)
        ro = _rows(q_out, "q_out", n_head, hd, rows, dev)
        pq, po = ctypes.addressof(rq), ctypes.addressof(ro)
    elif q_out is not None or q_norm is not None:
        raise ValueError("q_out and q_norm need q")
    po_opts = None
    if q_norm is not None or k_norm is not None or rope is not None:
        o = _WriteOpts(None, None, norm_eps, None, 0, 0, 0)
        if q_norm is not None:
            o.q_norm = _f32(q_norm, "q_norm", (hd,), dev)
        if k_norm is not None:
            o.k_norm = _f32(k_norm, "k_norm", (hd,), dev)
        if rope is not None:
            shape = rope.shape
            if len(shape) != 3 or shape[2] != 2:
                raise ValueError("rope must be [positions, rotary_dim / 2, 2]")
            o.rope = _f32(rope, "rope", shape, dev)
            o.rope_rows, o.rotary_dim, o.interleaved = shape[0], 2 * shape[1], int(interleaved)
        po_opts = ctypes.addressof(o)
    b = batch._with_rows(rows)
    rc = _lib().qwen2_paged_write(kv._at, ctypes.addressof(b), po_opts, n_head, pq, po, ctypes.addressof(rk), ctypes.addressof(rv),
                                  _raw_stream(kv._index))
    if rc:
        _check(rc)
    return q_out


def paged_read(kv: PagedKV, batch: PagedBatch, out_start, n_rows: int, dtype=None, k_out=None, v_out=None, stream=None):
    """Read the sequences' positions back as rows: position p of sequence s is
    row out_start[s] + p of (k, v), [n_rows, n_kv_head, head_dim] in ``dtype``
    (f32, f16 or bf16; default f32).  ``out_start``: int32 CUDA tensor
    [n_seq + 1]; rows outside the sequences are left as they were."""
    if not _plain(kv, batch, stream):
        with _Call(kv, batch, stream):
            return paged_read(kv, batch, out_start, n_rows, dtype, k_out, v_out)
    dev, heads, hd = kv.device, kv.n_kv_head, kv.head_dim
    if out_start.shape != (batch.n_seq + 1,) or out_start.dtype != _t.int32 or out_start.device != dev or \
            not out_start.is_contiguous():
        raise ValueError("out_start must be a contiguous int32 tensor [n_seq + 1] on the pool's device")
    if (k_out is None) != (v_out is None):
        raise ValueError("k_out and v_out go together")
    if k_out is None:
        k_out = _t.empty((n_rows, heads, hd), dtype=dtype or _t.float32, device=dev)
        v_out = _t.empty((n_rows, heads, hd), dtype=dtype or _t.float32, device=dev)
    rk, rv = _rows(k_out, "k_out", heads, hd, None, dev), _rows(v_out, "v_out", heads, hd, None, dev)
    if k_out.shape[0] < n_rows or v_out.shape[0] < n_rows:
        raise ValueError("k_out and v_out need n_rows rows")
    rc = _lib().qwen2_paged_read(kv._at, batch._at, out_start.data_ptr(), n_rows, ctypes.addressof(rk),
                                 ctypes.addressof(rv), _raw_stream(kv._index))
    if rc:
        _check(rc)
    return k_out, v_out


def _workspace(kv, batch, n_head, stream):
    """The batch's workspace on a stream, where one thread's calls come one after
    another (two threads' launches may alternate there, so each has its own); a
    call that is captured gets a new one, since its graph may be replayed beside
    anything."""
    key = (kv.n_kv_head, kv.head_dim, n_head)
    need = batch._space.get(key)
    if need is None:
        need = batch._space[key] = paged_attention_workspace(kv, batch, n_head)
    if _capturing():
        return _t.empty(need, dtype=_t.uint8, device=kv.device), need
    at = (stream, _thread())
    w = batch._buffers.get(at)
    if w is None or w.numel() < need:
        w = batch._buffers[at] = _t.empty(need, dtype=_t.uint8, device=kv.device)
    return w, need


def paged_attention(kv: PagedKV, batch: PagedBatch, q, out=None, scale=None, causal: bool = True,
                    return_lse: bool = False, workspace=None, stream=None):
    """Attention of the batch's rows ``q`` ([rows, n_head, head_dim], f16 or
    bf16, the pages' type where they are 16-bit) over its pages; row i of a
    sequence with n rows sees positions <= kv_len - n + i (``causal``) or all
    of them.  Returns o like q, with ``return_lse`` also f32 [rows, n_head]:
    the log of the sum of exp(scale q.k), -inf for a row without keys (whose o
    is 0).  ``scale``: default head_dim^-1/2.  ``workspace``: a uint8 CUDA
    tensor of ``paged_attention_workspace`` bytes (default: the batch keeps one
    for each stream and thread that use it; a captured call has its own)."""
    if not _plain(kv, batch, stream):
        with _Call(kv, batch, stream):
            return paged_attention(kv, batch, q, out, scale, causal, return_lse, workspace)
    dev, hd = kv.device, kv.head_dim
    rq = _rows(q, "q", None, hd, None, dev)
    shape = q.shape
    rows, n_head = shape[0], shape[1]
    if out is None:
        out = _t.empty_like(q)
    ro = _rows(out, "out", n_head, hd, rows, dev)
    lse = _t.empty((rows, n_head), dtype=_t.float32, device=dev) if return_lse else None
    b = batch._with_rows(rows)
    stream = _raw_stream(kv._index)
    if workspace is None:
        workspace, need = _workspace(kv, batch, n_head, stream)
    else:
        if workspace.dtype != _t.uint8 or workspace.device != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous uint8 tensor on the pool's device")
        need = workspace.numel()
    rc = _lib().qwen2_paged_attention(kv._at, ctypes.addressof(b), n_head, ctypes.addressof(rq), ctypes.addressof(ro),
                                      lse.data_ptr() if return_lse else None,
                                      hd ** -0.5 if scale is None else scale, int(causal), workspace.data_ptr(), need, stream)
    if rc:
        _check(rc)
    return (out, lse) if return_lse else out


def paged_attention_workspace(kv: PagedKV, batch: PagedBatch, n_head: int) -> int:
    """Workspace bytes of paged_attention for these shapes."""
    with _t.cuda.device(kv.device):
        need = _lib().qwen2_paged_attention_workspace(kv._at, batch._at, n_head)
    if need < 0:
        from . import QWEN2_E_ARG, Qwen2Error
        raise Qwen2Error(QWEN2_E_ARG, _lib().qwen2_last_error(None).decode())
    return need
