"""The paged cache entry points without a GPU: refusals come before any CUDA
call, and the rotation table is host code."""
import ctypes
import math
import os

import numpy as np
import pytest

q2 = pytest.importorskip("qwen2_decoder_forward_gb300")
from qwen2_decoder_forward_gb300 import paged  # noqa: E402

FAKE = 1 << 20     # a non-null, 256-byte aligned address that is never read


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(q2.LIB_PATH):
        from qwen2_decoder_forward_gb300 import build
        build.build()
    return paged._lib()


def _kv(**over):
    f = dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, format=0, n_pages=4, page_size=16, n_kv_head=2, head_dim=64,
             page_stride=2048, token_stride=64, head_stride=1024)
    f.update(over)
    return paged._PagedKV(**f)


def _batch(**over):
    f = dict(n_seq=2, n_rows=3, max_q=2, max_pages=2, pages_stride=2, q_start=FAKE, kv_len=FAKE, pages=FAKE, guard=None)
    f.update(over)
    return paged._PagedBatch(**f)


def _rows(**over):
    f = dict(data=FAKE, dtype=1, row_stride=128, head_stride=64)
    f.update(over)
    return paged._Rows(**f)


def _at(s):
    return None if s is None else ctypes.addressof(s)


KV_BAD = [
    (dict(format=4), q2.QWEN2_E_UNSUPPORTED), (dict(format=-1), q2.QWEN2_E_UNSUPPORTED),
    (dict(head_dim=96), q2.QWEN2_E_UNSUPPORTED), (dict(page_size=24), q2.QWEN2_E_UNSUPPORTED),
    (dict(page_size=8), q2.QWEN2_E_UNSUPPORTED), (dict(page_size=512), q2.QWEN2_E_UNSUPPORTED),
    (dict(n_pages=0), q2.QWEN2_E_ARG), (dict(n_kv_head=0), q2.QWEN2_E_ARG), (dict(k=None), q2.QWEN2_E_ARG),
    (dict(v=FAKE + 8), q2.QWEN2_E_ARG), (dict(token_stride=68), q2.QWEN2_E_ARG), (dict(page_stride=-2048), q2.QWEN2_E_ARG),
    (dict(format=2, k_scale=None), q2.QWEN2_E_ARG), (dict(format=3, v_scale=FAKE + 4), q2.QWEN2_E_ARG),
]
BATCH_BAD = [
    (dict(n_seq=0), q2.QWEN2_E_ARG), (dict(n_seq=4097), q2.QWEN2_E_ARG), (dict(kv_len=None), q2.QWEN2_E_ARG),
    (dict(pages=None), q2.QWEN2_E_ARG), (dict(max_pages=0), q2.QWEN2_E_ARG), (dict(pages_stride=1), q2.QWEN2_E_ARG),
    (dict(max_pages=1 << 27, pages_stride=1 << 27), q2.QWEN2_E_UNSUPPORTED),
]
ROW_BATCH_BAD = [(dict(q_start=None), q2.QWEN2_E_ARG), (dict(n_rows=-1), q2.QWEN2_E_ARG), (dict(max_q=-1), q2.QWEN2_E_ARG)]
ROWS_BAD = [(dict(data=None), q2.QWEN2_E_ARG), (dict(dtype=3), q2.QWEN2_E_UNSUPPORTED), (dict(row_stride=65), q2.QWEN2_E_ARG),
            (dict(head_stride=-64), q2.QWEN2_E_ARG), (dict(data=FAKE + 2), q2.QWEN2_E_ARG)]


def _refused(L, rc, code):
    assert rc == code
    assert L.qwen2_last_error(None)


@pytest.mark.parametrize("over,code", KV_BAD)
def test_bad_pools_are_refused_everywhere(L, over, code):
    kv, b, r = _kv(**over), _batch(), _rows()
    _refused(L, L.qwen2_paged_write(_at(kv), _at(b), None, 0, None, None, _at(r), _at(r), None), code)
    _refused(L, L.qwen2_paged_read(_at(kv), _at(b), FAKE, 3, _at(r), _at(r), None), code)
    _refused(L, L.qwen2_paged_attention(_at(kv), _at(b), 4, _at(r), _at(r), None, 1.0, 1, FAKE, 1 << 30, None), code)
    assert L.qwen2_paged_attention_workspace(_at(kv), _at(b), 4) == -1


@pytest.mark.parametrize("over,code", BATCH_BAD + ROW_BATCH_BAD)
def test_bad_batches_are_refused_everywhere(L, over, code):
    kv, b, r = _kv(), _batch(**over), _rows()
    _refused(L, L.qwen2_paged_write(_at(kv), _at(b), None, 0, None, None, _at(r), _at(r), None), code)
    _refused(L, L.qwen2_paged_attention(_at(kv), _at(b), 4, _at(r), _at(r), None, 1.0, 1, FAKE, 1 << 30, None), code)
    if (over, code) in BATCH_BAD:
        _refused(L, L.qwen2_paged_read(_at(kv), _at(b), FAKE, 3, _at(r), _at(r), None), code)


@pytest.mark.parametrize("over,code", ROWS_BAD)
def test_bad_rows_are_refused(L, over, code):
    kv, b, r, bad = _kv(), _batch(), _rows(), _rows(**over)
    for k, v in ((bad, r), (r, bad)):
        _refused(L, L.qwen2_paged_write(_at(kv), _at(b), None, 0, None, None, _at(k), _at(v), None), code)
        _refused(L, L.qwen2_paged_read(_at(kv), _at(b), FAKE, 3, _at(k), _at(v), None), code)
    for q, o in ((bad, r), (r, bad)):
        _refused(L, L.qwen2_paged_attention(_at(kv), _at(b), 4, _at(q), _at(o), None, 1.0, 1, FAKE, 1 << 30, None), code)
        _refused(L, L.qwen2_paged_write(_at(kv), _at(b), None, 4, _at(q), _at(o), _at(r), _at(r), None), code)


def test_null_descriptors_are_refused(L):
    kv, b, r = _kv(), _batch(), _rows()
    arg = q2.QWEN2_E_ARG
    _refused(L, L.qwen2_paged_write(None, _at(b), None, 0, None, None, _at(r), _at(r), None), arg)
    _refused(L, L.qwen2_paged_write(_at(kv), None, None, 0, None, None, _at(r), _at(r), None), arg)
    _refused(L, L.qwen2_paged_write(_at(kv), _at(b), None, 0, None, None, None, _at(r), None), arg)
    _refused(L, L.qwen2_paged_write(_at(kv), _at(b), None, 4, _at(r), None, _at(r), _at(r), None), arg)
    _refused(L, L.qwen2_paged_read(_at(kv), _at(b), None, 3, _at(r), _at(r), None), arg)
    _refused(L, L.qwen2_paged_attention(_at(kv), _at(b), 4, None, _at(r), None, 1.0, 1, FAKE, 1 << 30, None), arg)


def test_write_options_are_checked(L):
    kv, b, r = _kv(), _batch(), _rows()

    def rc(dtype=1, **f):
        o, v = paged._WriteOpts(**f), _rows(dtype=dtype)
        return L.qwen2_paged_write(_at(kv), _at(b), _at(o), 0, None, None, _at(r), _at(v), None)
    _refused(L, rc(rope=FAKE, rope_rows=8, rotary_dim=24), q2.QWEN2_E_UNSUPPORTED)
    _refused(L, rc(rope=FAKE, rope_rows=8, rotary_dim=80), q2.QWEN2_E_UNSUPPORTED)
    _refused(L, rc(rope=FAKE, rope_rows=0, rotary_dim=64), q2.QWEN2_E_ARG)
    _refused(L, rc(rope=FAKE + 8, rope_rows=8, rotary_dim=64), q2.QWEN2_E_ARG)
    _refused(L, rc(k_norm=FAKE, norm_eps=-1.0), q2.QWEN2_E_ARG)
    _refused(L, rc(k_norm=FAKE, norm_eps=float("nan")), q2.QWEN2_E_ARG)
    _refused(L, rc(k_norm=FAKE + 4), q2.QWEN2_E_ARG)
    _refused(L, rc(dtype=2), q2.QWEN2_E_ARG)                        # k f16, v bf16
    out32 = _rows(dtype=0)
    _refused(L, L.qwen2_paged_write(_at(kv), _at(b), None, 4, _at(r), _at(out32), _at(r), _at(r), None),
             q2.QWEN2_E_UNSUPPORTED)


def test_attention_types_heads_and_scale_are_checked(L):
    b, r = _batch(), _rows()

    def rc(kv=None, n_head=4, q=r, out=r, scale=1.0, batch=b):
        kv = kv or _kv()
        return L.qwen2_paged_attention(_at(kv), _at(batch), n_head, _at(q), _at(out), None, scale, 1, FAKE,
                                       1 << 30, None)
    _refused(L, rc(n_head=5), q2.QWEN2_E_ARG)
    _refused(L, rc(n_head=0), q2.QWEN2_E_ARG)
    _refused(L, rc(n_head=2 * 65), q2.QWEN2_E_UNSUPPORTED)
    _refused(L, rc(n_head=4, batch=_batch(n_rows=1 << 30)), q2.QWEN2_E_UNSUPPORTED)
    _refused(L, rc(q=_rows(dtype=2), out=_rows(dtype=2)), q2.QWEN2_E_UNSUPPORTED)     # bf16 over f16 pages
    _refused(L, rc(kv=_kv(format=1)), q2.QWEN2_E_UNSUPPORTED)                         # f16 over bf16 pages
    _refused(L, rc(kv=_kv(format=2), q=_rows(dtype=0), out=_rows(dtype=0)), q2.QWEN2_E_UNSUPPORTED)
    _refused(L, rc(out=_rows(dtype=2)), q2.QWEN2_E_UNSUPPORTED)
    for bad in (float("nan"), float("inf")):
        _refused(L, rc(scale=bad), q2.QWEN2_E_ARG)


def test_calls_without_rows_launch_nothing(L):
    kv, r = _kv(), _rows()
    b = _batch(n_rows=0)
    assert L.qwen2_paged_write(_at(kv), _at(b), None, 0, None, None, _at(r), _at(r), None) == 0
    assert L.qwen2_paged_read(_at(kv), _at(b), FAKE, 0, _at(r), _at(r), None) == 0
    assert L.qwen2_paged_attention(_at(kv), _at(b), 4, _at(r), _at(r), None, 1.0, 1, None, 0, None) == 0


# ---- the rotation table -----------------------------------------------------


def _angles(rows, dim, theta):
    return np.arange(rows)[:, None] * theta ** (-2.0 * np.arange(dim // 2) / dim)


@pytest.mark.parametrize("rows,dim,theta", [(1, 16, 1e4), (300, 64, 1e6), (40000, 32, 1e6)])
def test_plain_and_linear_tables(L, rows, dim, theta):
    a = _angles(rows, dim, theta)
    # One rounding to f32, and the 64-bit angle's own error: half a step of
    # position * theta_i, at most 40000 * 2^-53.
    tol = np.finfo(np.float32).eps / 2 + rows * 2.0 ** -50
    t = q2.rope_table(rows, dim, theta)
    assert t.shape == (rows, dim // 2, 2) and t.dtype == np.float32
    np.testing.assert_allclose(t[..., 0], np.cos(a), rtol=0, atol=tol)
    np.testing.assert_allclose(t[..., 1], np.sin(a), rtol=0, atol=tol)
    t = q2.rope_table(rows, dim, theta, kind=q2.ROPE_LINEAR, factor=4.0)
    np.testing.assert_allclose(t[..., 0], np.cos(a / 4), rtol=0, atol=tol)
    np.testing.assert_allclose(t[..., 1], np.sin(a / 4), rtol=0, atol=tol)


def test_yarn_table_keeps_fast_dims_and_divides_slow_ones(L):
    rows, dim, theta, factor, trained = 2000, 128, 1e6, 4.0, 32768
    t = q2.rope_table(rows, dim, theta, kind=q2.ROPE_YARN, factor=factor, original_rows=trained).astype(np.float64)
    gain = 0.1 * math.log(factor) + 1
    i = np.arange(dim // 2)
    turns = trained * theta ** (-2.0 * i / dim) / (2 * math.pi)     # full turns within the trained length
    a = _angles(rows, dim, theta)
    tol = gain * (np.finfo(np.float32).eps / 2) + rows * 2.0 ** -50
    # The ramp's ends are rounded outwards to whole dims, so dims within one
    # of an end may already be on it.
    fast, slow = i < np.argmax(turns < 32) - 1, i > np.argmax(turns < 1) + 1
    assert fast.sum() > 4 and slow.sum() > 4
    np.testing.assert_allclose(t[:, fast, 0], gain * np.cos(a[:, fast]), rtol=0, atol=tol)
    np.testing.assert_allclose(t[:, slow, 1], gain * np.sin(a[:, slow] / factor), rtol=0, atol=tol)
    # Between, the frequency falls monotonically from one to the other.
    inv = np.arctan2(t[1, :, 1], t[1, :, 0]) / theta ** (-2.0 * i / dim)
    assert np.all(np.diff(inv) <= 1e-6) and abs(inv[0] - 1) < 1e-6 and abs(inv[-1] - 1 / factor) < 1e-5


def test_yarn_with_factor_one_is_plain(L):
    np.testing.assert_array_equal(q2.rope_table(64, 64, 1e6, kind=q2.ROPE_YARN, factor=1.0, original_rows=512),
                                  q2.rope_table(64, 64, 1e6))


@pytest.mark.parametrize("args,kw", [((0, 64), {}), ((4, 63), {}), ((4, 64, -1.0), {}), ((4, 64), dict(kind=7)),
                                     ((4, 64), dict(kind=1, factor=0.5)), ((4, 64), dict(kind=2, factor=2.0)),
                                     ((4, 64), dict(kind=2, factor=2.0, original_rows=64, beta_fast=1.0, beta_slow=2.0)),
                                     ((4, 64, float("inf")), {}), ((4, 64), dict(kind=1, factor=float("nan")))])
def test_bad_tables_are_refused(L, args, kw):
    with pytest.raises(q2.Qwen2Error):
        q2.rope_table(*args, **kw)


# ---- the binding's own checks (CPU tensors are refused before any call) -----


def test_binding_refuses_host_tensors_and_bad_shapes():
    torch = pytest.importorskip("torch")
    k = torch.zeros((2, 16, 2, 64), dtype=torch.float16)
    with pytest.raises(ValueError):
        q2.PagedKV(k, k)
    with pytest.raises(ValueError):
        q2.PagedKV(k[0], k[0])
    with pytest.raises(ValueError):
        q2.PagedKV(k.float(), k.float())
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        q2.PagedBatch(i, i[:2], torch.zeros((2, 4), dtype=torch.int32), 1)
    with pytest.raises(ValueError):
        q2.PagedBatch(i, i, torch.zeros((3, 4), dtype=torch.int32), 1)
