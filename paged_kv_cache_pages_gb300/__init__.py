"""Python binding of libpagedattn.so: ubatch-aligned paged attention on GB300.

Argument marshalling only: every step runs in the library's CUDA kernels.
Tensors are torch CUDA tensors (float16 for K/V/Q/out, int32 tables, int64
slot mapping); the current torch stream is passed to each call.  The library
must have been built (``paged_kv_cache_pages_gb300.build.build()`` or
``__graft_entry__.build()``); importing without it raises ImportError -- there
is no fallback.

Entry points mirror include/paged_attn.h:
  batch_build     a step's tables, token lists and slots from request lengths, pages taken
                  from a reference-counted pool on the device
  expand_ubatch   per-token page-table / kv_len expansion + slot mapping
  kv_append       reshape-and-cache into the paged pool
  copy_pages      page copy of a copy-on-write fork
  masked_decode / masked_prefill   the unified-span baseline (masked attention over a
                  shared span) on the split-KV and on the tcgen05 path
  kv_append_fp8 / decode_fp8 / prefill_fp8 / forward_fp8   FP8 (E4M3) KV pages with
                  per-row scales
  plan / prefill / decode / run / forward   the attention itself
  plan_diff / diff_run / diff_forward       differential attention over the same pages
  plan_window / window_run / window_forward attention to the last positions, with sinks
  validate, read_error, set_prefill_min_run, workspace_size
  PagePool        host page allocator with reference-counted sharing
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpagedattn.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with "
                      "`python paged_kv_cache_pages_gb300/build.py` (needs nvcc)")

_lib = ctypes.CDLL(LIB_PATH)

PA_OK, PA_EINVAL, PA_EUNSUPPORTED, PA_EWORKSPACE = 0, -1, -2, -3
PA_ELAUNCH, PA_EDEVICE, PA_EALIGN, PA_ENOSPACE = -4, -5, -6, -7
PA_ERR_PAGE_RANGE, PA_ERR_KV_RANGE, PA_ERR_SLOT_RANGE = 0x1, 0x2, 0x4
PA_ERR_TIMEOUT, PA_ERR_SEQ_RANGE = 0x8, 0x10
PA_ERR_NO_SPACE, PA_ERR_REFCOUNT, PA_ERR_PLAN = 0x20, 0x40, 0x80

_vp, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t

_ATTN_ARGS = [_vp, _vp, _vp, _vp, _i, _vp, _i, _i, _i, _i, _i, _i, _f, _vp, _vp, _sz, _vp]
_SIGS = {
    "paged_attn_strerror": ([_i], ctypes.c_char_p),
    "paged_attn_version": ([], _i),
    "paged_expand_ubatch": ([_vp, _i, _i, _vp, _vp, _i, _i, _vp, _vp, _vp, _vp, _vp], _i),
    "paged_batch_build": ([_vp, _i, _i, _vp, _vp, _vp, _i, _i, _i] + [_vp] * 9, _i),
    "paged_kv_append": ([_vp, _vp, _vp, _i, _vp, _vp, _i, _i, _i, _i, _vp, _vp], _i),
    "paged_attn_workspace_size": ([_i, _i, _i, _i], _sz),
    "paged_attn_plan": ([_vp, _i, _vp, _i, _i, _i, _i, _i, _vp, _sz, _vp], _i),
    "paged_attn_prefill": (_ATTN_ARGS, _i),
    "paged_attn_decode": (_ATTN_ARGS, _i),
    "paged_attn_run": (_ATTN_ARGS, _i),
    "paged_attn_forward": (_ATTN_ARGS, _i),
    "paged_attn_validate": ([_vp, _i, _vp, _i, _i, _i, _vp, _vp], _i),
    "paged_attn_read_error": ([_vp, ctypes.POINTER(_i), _vp], _i),
    "paged_attn_set_prefill_min_run": ([_i], _i),
    "paged_attn_set_decode_wait_limit": ([ctypes.c_ulonglong], ctypes.c_ulonglong),
    "pa_pool_create": ([_i], _vp),
    "pa_pool_destroy": ([_vp], None),
    "pa_pool_num_free": ([_vp], _i),
    "pa_pool_alloc": ([_vp, _i, _vp], _i),
    "pa_pool_share": ([_vp, _vp, _i], _i),
    "pa_pool_release": ([_vp, _vp, _i], _i),
    "pa_pool_refcount": ([_vp, ctypes.c_int32], _i),
    "pa_pool_fork": ([_vp, _vp, _i, _i, _vp, _vp, _vp], _i),
    "paged_copy_pages": ([_vp, _vp, _i, _vp, _vp, _i, _i, _i, _i, _vp, _vp], _i),
    "paged_kv_append_fp8": ([_vp, _vp, _vp, _i, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp, _vp],
                            _i),
    "paged_attn_decode_fp8": ([_vp, _vp, _vp, _vp, _vp, _vp, _i, _vp, _i, _i, _i, _i, _i, _i,
                               ctypes.c_float, _vp, _vp, _sz, _vp], _i),
    "paged_attn_prefill_fp8": ([_vp, _vp, _vp, _vp, _vp, _vp, _i, _vp, _i, _i, _i, _i, _i, _i,
                                ctypes.c_float, _vp, _vp, _sz, _vp], _i),
    "paged_attn_forward_fp8": ([_vp, _vp, _vp, _vp, _vp, _vp, _i, _vp, _i, _i, _i, _i, _i, _i,
                                ctypes.c_float, _vp, _vp, _sz, _vp], _i),
    "paged_attn_plan_decode": ([_vp, _i, _vp, _i, _i, _i, _i, _i, _vp, _sz, _vp], _i),
    "paged_attn_masked_decode": ([_vp, _vp, _vp, _vp, _i, _vp, _i, _i, _i, _i, _i, _i,
                                  ctypes.c_float, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp], _i),
    "paged_attn_decode_append": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _vp, _i, _i, _i, _i, _i,
                                  _i, ctypes.c_float, _vp, _vp, _sz, _vp], _i),
    "paged_attn_plan_prefill": ([_vp, _i, _vp, _i, _i, _i, _i, _i, _vp, _sz, _vp], _i),
    "paged_attn_masked_prefill": ([_vp, _vp, _vp, _vp, _i, _vp, _i, _i, _i, _i, _i, _i,
                                   ctypes.c_float, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp], _i),
    "paged_attn_diff_workspace_size": ([_i, _i, _i, _i], _sz),
    "paged_attn_plan_diff": ([_vp, _i, _vp, _i, _i, _i, _i, _i, _vp, _sz, _vp], _i),
    "paged_attn_diff_run": (_ATTN_ARGS[:13] + [_vp, _vp, _f, _f] + _ATTN_ARGS[13:], _i),
    "paged_attn_diff_forward": (_ATTN_ARGS[:13] + [_vp, _vp, _f, _f] + _ATTN_ARGS[13:], _i),
    "paged_attn_window_workspace_size": ([_i, _i, _i, _i], _sz),
    "paged_attn_plan_window": ([_vp, _i, _vp, _i, _i, _i, _i, _i, _i, _vp, _sz, _vp], _i),
    "paged_attn_window_run": (_ATTN_ARGS[:13] + [_vp] + _ATTN_ARGS[13:], _i),
    "paged_attn_window_forward": (_ATTN_ARGS[:13] + [_i, _vp] + _ATTN_ARGS[13:], _i),
}
for _name, (_args, _res) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.argtypes = _args
    _fn.restype = _res


class PagedAttnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {strerror(status)} (status {status})")


def lib() -> ctypes.CDLL:
    """The loaded ctypes library (raw C-ABI access)."""
    return _lib


def strerror(status: int) -> str:
    return _lib.paged_attn_strerror(int(status)).decode()


def version() -> int:
    return int(_lib.paged_attn_version())


def _check(status: int, where: str):
    if status != PA_OK:
        raise PagedAttnError(status, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _raw_stream(stream, device):
    """The stream's handle; the device's current stream without building its Python object
    (3 us of a call)."""
    return torch._C._cuda_getCurrentRawStream(device.index) if stream is None \
        else stream.cuda_stream


def _used_on(stream, *made):
    """Buffers made here for a call on another stream than the current one stay allocated
    until that stream is past the call."""
    if stream is not None:
        for t in made:
            t.record_stream(stream)


def _int32(n):
    """`n` held to int32 (ctypes would wrap it): "all" from the largest on, refused below 1."""
    return max(min(int(n), 2 ** 31 - 1), -1)


def _req(t, dtype, name):
    if not (t.is_cuda and t.dtype == dtype and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor")


def _req_on(t, dtype, shape, device, name):
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.device != device \
            or device.type != "cuda":
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on "
                         "one CUDA device")


def _req_all(device, *wanted):
    """_req_on of every (tensor, dtype, shape, name), in one pass where all are as wanted (a
    call for each tensor was a third of a call's time)."""
    for t, dtype, shape, name in wanted:
        if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() \
                or t.device != device:
            _req_on(t, dtype, shape, device, name)
    if device.type != "cuda":
        _req_on(*wanted[0][:3], device, wanted[0][3])


def _call(fn_name, fn, device, args):
    """fn(*args, the device's current stream) with `device` as the current one (launches and
    the SM count go by it)."""
    if device.index == torch.cuda.current_device():
        status = fn(*args)
    else:
        with torch.cuda.device(device):
            status = fn(*args)
    if status != PA_OK:
        raise PagedAttnError(status, fn_name)


def workspace_size(T: int, Hq: int, Hkv: int, d: int) -> int:
    return int(_lib.paged_attn_workspace_size(T, Hq, Hkv, d))


def window_workspace_size(T: int, Hq: int, Hkv: int, d: int) -> int:
    return int(_lib.paged_attn_window_workspace_size(T, Hq, Hkv, d))


def new_workspace(T: int, Hq: int, Hkv: int, d: int, device=None) -> torch.Tensor:
    """Workspace of every call for these shapes but the differential ones (new_diff_workspace)."""
    n = max(workspace_size(T, Hq, Hkv, d), window_workspace_size(T, Hq, Hkv, d))
    if n == 0:
        raise PagedAttnError(PA_EUNSUPPORTED, "workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def expand_ubatch(seq_page_table, tok_seq, tok_pos, P, out=None, err=None, stream=None):
    """Per-token expansion -> (tok_page_table, tok_kv_len, slot_mapping)."""
    _req(seq_page_table, torch.int32, "seq_page_table")
    _req(tok_seq, torch.int32, "tok_seq")
    _req(tok_pos, torch.int32, "tok_pos")
    n_seq, max_pages = seq_page_table.shape
    T = tok_seq.shape[0]
    dev = seq_page_table.device
    if out is None:
        out = (torch.empty((T, max_pages), dtype=torch.int32, device=dev),
               torch.empty(T, dtype=torch.int32, device=dev),
               torch.empty(T, dtype=torch.int64, device=dev))
    tpt, kv, slot = out
    _check(_lib.paged_expand_ubatch(_ptr(seq_page_table), n_seq, max_pages, _ptr(tok_seq),
                                    _ptr(tok_pos), T, P, _ptr(tpt), _ptr(kv), _ptr(slot),
                                    _ptr(err), _stream(stream)), "paged_expand_ubatch")
    return tpt, kv, slot


class Batch(NamedTuple):
    """What batch_build leaves: first token of each request [n_seq + 1], each request's
    length after the step [n_seq], and the tokens' lists and tables [T]."""
    q_start: torch.Tensor
    seq_len: torch.Tensor
    tok_seq: torch.Tensor
    tok_pos: torch.Tensor
    tok_page_table: torch.Tensor
    tok_kv_len: torch.Tensor
    slot_mapping: torch.Tensor


def new_batch(n_seq: int, max_pages: int, T: int, device=None) -> Batch:
    """Output buffers of batch_build for up to T tokens of n_seq requests."""
    dev = device or "cuda"

    def i32(*shape):
        return torch.empty(shape, dtype=torch.int32, device=dev)
    return Batch(i32(n_seq + 1), i32(n_seq), i32(T), i32(T), i32(T, max_pages), i32(T),
                 torch.empty(T, dtype=torch.int64, device=dev))


def batch_build(seq_page_table, seq_len, new_len, page_ref, P, T, out=None, err=None,
                stream=None) -> Batch:
    """One serving step's tables from request lengths (see paged_batch_build): requests with
    new_len < 0 give their pages back, the longest prefix of the others that fits T tokens and
    the free pages is admitted, and its tokens' lists are written.  seq_page_table and
    page_ref are updated in place."""
    n_seq, max_pages = seq_page_table.shape
    dev, i32, num_pages = seq_page_table.device, torch.int32, page_ref.numel()
    _req_all(dev, (seq_page_table, i32, (n_seq, max_pages), "seq_page_table"),
             (seq_len, i32, (n_seq,), "seq_len"), (new_len, i32, (n_seq,), "new_len"),
             (page_ref, i32, (num_pages,), "page_ref"))
    if out is None:
        out = new_batch(n_seq, max_pages, T, dev)
        _used_on(stream, *out)
    else:
        _req_all(dev, (out[0], i32, (n_seq + 1,), "q_start"),
                 (out[1], i32, (n_seq,), "seq_len (out)"), (out[2], i32, (T,), "tok_seq"),
                 (out[3], i32, (T,), "tok_pos"),
                 (out[4], i32, (T, max_pages), "tok_page_table"),
                 (out[5], i32, (T,), "tok_kv_len"), (out[6], torch.int64, (T,), "slot_mapping"))
    if err is not None:
        _req_on(err, torch.int32, (err.numel(),), dev, "err")
    q_start, seq_len_out, tok_seq, tok_pos, tok_page_table, tok_kv_len, slot_mapping = out
    _call("paged_batch_build", _lib.paged_batch_build, dev,
          (seq_page_table.data_ptr(), n_seq, max_pages, seq_len.data_ptr(), new_len.data_ptr(),
           page_ref.data_ptr(), num_pages, P, T, q_start.data_ptr(), seq_len_out.data_ptr(),
           tok_seq.data_ptr(), tok_pos.data_ptr(), tok_page_table.data_ptr(),
           tok_kv_len.data_ptr(), slot_mapping.data_ptr(), None if err is None else err.data_ptr(),
           _raw_stream(stream, dev)))
    return out


def kv_append(k, v, slot_mapping, k_pages, v_pages, err=None, stream=None):
    """reshape-and-cache: write k/v [T][Hkv][d] into the pool at slot_mapping."""
    for t, n in ((k, "k"), (v, "v"), (k_pages, "k_pages"), (v_pages, "v_pages")):
        _req(t, torch.float16, n)
    _req(slot_mapping, torch.int64, "slot_mapping")
    N, Hkv, P, d = k_pages.shape
    T = slot_mapping.shape[0]
    _check(_lib.paged_kv_append(_ptr(k), _ptr(v), _ptr(slot_mapping), T, _ptr(k_pages),
                                _ptr(v_pages), N, Hkv, P, d, _ptr(err), _stream(stream)),
           "paged_kv_append")


def plan_decode(tok_page_table, tok_kv_len, Hq, Hkv, P, d, workspace, stream=None):
    """plan with every token on the split-KV path (for masked_decode / decode_fp8)."""
    _req(tok_page_table, torch.int32, "tok_page_table")
    _req(tok_kv_len, torch.int32, "tok_kv_len")
    T, max_pages = tok_page_table.shape
    _check(_lib.paged_attn_plan_decode(_ptr(tok_page_table), max_pages, _ptr(tok_kv_len), T, Hq,
                                       Hkv, P, d, _ptr(workspace), workspace.numel(),
                                       _stream(stream)), "paged_attn_plan_decode")


def plan_prefill(tok_page_table, tok_kv_len, Hq, Hkv, P, d, workspace, stream=None):
    """plan with every token in a tensor-core tile (for masked_prefill)."""
    _req(tok_page_table, torch.int32, "tok_page_table")
    _req(tok_kv_len, torch.int32, "tok_kv_len")
    T, max_pages = tok_page_table.shape
    _check(_lib.paged_attn_plan_prefill(_ptr(tok_page_table), max_pages, _ptr(tok_kv_len), T, Hq,
                                        Hkv, P, d, _ptr(workspace), workspace.numel(),
                                        _stream(stream)), "paged_attn_plan_prefill")


def masked_decode(q, k_pages, v_pages, tok_page_table, tok_kv_len, scale, cell_seq, cell_pos,
                  tok_seq, tok_pos, out, workspace, stream=None):
    """Unified-span baseline: split-KV attention of every token over its row, keeping
    only the slots whose cell belongs to the token's sequence at a position up to its
    own.  Runs on a plan from plan_decode."""
    return _masked("paged_attn_masked_decode", q, k_pages, v_pages, tok_page_table, tok_kv_len,
                   scale, cell_seq, cell_pos, tok_seq, tok_pos, out, workspace, stream)


def masked_prefill(q, k_pages, v_pages, tok_page_table, tok_kv_len, scale, cell_seq, cell_pos,
                   tok_seq, tok_pos, out, workspace, stream=None):
    """The same masked attention on the tcgen05 prefill tiles (the unified-span
    baseline of prefill).  Runs on a plan from plan_prefill."""
    return _masked("paged_attn_masked_prefill", q, k_pages, v_pages, tok_page_table, tok_kv_len,
                   scale, cell_seq, cell_pos, tok_seq, tok_pos, out, workspace, stream)


def _masked(fn_name, q, k_pages, v_pages, tok_page_table, tok_kv_len, scale, cell_seq, cell_pos,
            tok_seq, tok_pos, out, workspace, stream):
    for t, n in ((q, "q"), (k_pages, "k_pages"), (v_pages, "v_pages"), (out, "out")):
        _req(t, torch.float16, n)
    for t, n in ((tok_page_table, "tok_page_table"), (tok_kv_len, "tok_kv_len"),
                 (cell_seq, "cell_seq"), (cell_pos, "cell_pos"), (tok_seq, "tok_seq"),
                 (tok_pos, "tok_pos")):
        _req(t, torch.int32, n)
    T, Hq, d = q.shape
    N, Hkv, P, _ = k_pages.shape
    max_pages = tok_page_table.shape[1]
    _check(getattr(_lib, fn_name)(
        _ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(tok_page_table), max_pages, _ptr(tok_kv_len),
        T, Hq, Hkv, P, d, N, float(scale), _ptr(cell_seq), _ptr(cell_pos), _ptr(tok_seq),
        _ptr(tok_pos), _ptr(out), _ptr(workspace), workspace.numel(), _stream(stream)), fn_name)
    return out


def new_fp8_pool(num_pages, Hkv, P, d, device=None):
    """Empty FP8 pool: (k8 [N][Hkv][P][d] uint8, v8t [N][Hkv][d][P] uint8,
    k_scale, v_scale [N][Hkv][P] float32)."""
    dev = device or "cuda"
    return (torch.zeros((num_pages, Hkv, P, d), dtype=torch.uint8, device=dev),
            torch.zeros((num_pages, Hkv, d, P), dtype=torch.uint8, device=dev),
            torch.ones((num_pages, Hkv, P), dtype=torch.float32, device=dev),
            torch.ones((num_pages, Hkv, P), dtype=torch.float32, device=dev))


def kv_append_fp8(k, v, slot_mapping, k8, v8t, k_scale, v_scale, err=None, stream=None):
    """Quantising reshape-and-cache into FP8 pages (E4M3 codes, one scale per row)."""
    _req(k, torch.float16, "k")
    _req(v, torch.float16, "v")
    _req(slot_mapping, torch.int64, "slot_mapping")
    for t, n in ((k8, "k8"), (v8t, "v8t")):
        _req(t, torch.uint8, n)
    for t, n in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        _req(t, torch.float32, n)
    N, Hkv, P, d = k8.shape
    _check(_lib.paged_kv_append_fp8(_ptr(k), _ptr(v), _ptr(slot_mapping), slot_mapping.shape[0],
                                    _ptr(k8), _ptr(v8t), _ptr(k_scale), _ptr(v_scale), N, Hkv, P,
                                    d, _ptr(err), _stream(stream)), "paged_kv_append_fp8")


def _attn_fp8(name, q, k8, v8t, k_scale, v_scale, tok_page_table, tok_kv_len, scale, out,
              workspace, stream):
    _req(q, torch.float16, "q")
    _req(tok_page_table, torch.int32, "tok_page_table")
    _req(tok_kv_len, torch.int32, "tok_kv_len")
    T, Hq, d = q.shape
    N, Hkv, P, _ = k8.shape
    if out is None:
        out = torch.empty_like(q)
    _req(out, torch.float16, "out")
    if workspace is None:
        workspace = new_workspace(T, Hq, Hkv, d, q.device)
    _check(getattr(_lib, name)(
        _ptr(q), _ptr(k8), _ptr(v8t), _ptr(k_scale), _ptr(v_scale), _ptr(tok_page_table),
        tok_page_table.shape[1], _ptr(tok_kv_len), T, Hq, Hkv, P, d, N, float(scale), _ptr(out),
        _ptr(workspace), workspace.numel(), _stream(stream)), name)
    return out


def decode_fp8(q, k8, v8t, k_scale, v_scale, tok_page_table, tok_kv_len, scale, out, workspace,
               stream=None):
    """Split-KV decode attention over FP8 pages (on a plan from plan_decode or plan)."""
    return _attn_fp8("paged_attn_decode_fp8", q, k8, v8t, k_scale, v_scale, tok_page_table,
                     tok_kv_len, scale, out, workspace, stream)


def prefill_fp8(q, k8, v8t, k_scale, v_scale, tok_page_table, tok_kv_len, scale, out, workspace,
                stream=None):
    """Tensor-core prefill tiles over FP8 pages (on a plan from plan or plan_prefill)."""
    return _attn_fp8("paged_attn_prefill_fp8", q, k8, v8t, k_scale, v_scale, tok_page_table,
                     tok_kv_len, scale, out, workspace, stream)


def forward_fp8(q, k8, v8t, k_scale, v_scale, tok_page_table, tok_kv_len, scale, out=None,
                workspace=None, stream=None):
    """Plan + prefill + decode for one ubatch over FP8 pages; returns out [T][Hq][d]."""
    return _attn_fp8("paged_attn_forward_fp8", q, k8, v8t, k_scale, v_scale, tok_page_table,
                     tok_kv_len, scale, out, workspace, stream)


def copy_pages(src, dst, k_pages, v_pages, err=None, stream=None):
    """Page copy of a copy-on-write fork: page dst[i] <- page src[i] in both pools."""
    _req(src, torch.int32, "src")
    _req(dst, torch.int32, "dst")
    _req(k_pages, torch.float16, "k_pages")
    _req(v_pages, torch.float16, "v_pages")
    if src.shape != dst.shape:
        raise ValueError("src and dst must have the same length")
    N, Hkv, P, d = k_pages.shape
    _check(_lib.paged_copy_pages(_ptr(src), _ptr(dst), src.shape[0], _ptr(k_pages), _ptr(v_pages),
                                 N, Hkv, P, d, _ptr(err), _stream(stream)), "paged_copy_pages")


def plan(tok_page_table, tok_kv_len, Hq, Hkv, P, d, workspace, stream=None):
    _req(tok_page_table, torch.int32, "tok_page_table")
    _req(tok_kv_len, torch.int32, "tok_kv_len")
    T, max_pages = tok_page_table.shape
    _check(_lib.paged_attn_plan(_ptr(tok_page_table), max_pages, _ptr(tok_kv_len), T, Hq, Hkv, P,
                                d, _ptr(workspace), workspace.numel(), _stream(stream)),
           "paged_attn_plan")


def _attn(fn_name, q, k_pages, v_pages, tok_page_table, tok_kv_len, scale, out, workspace,
          stream):
    for t, n in ((q, "q"), (k_pages, "k_pages"), (v_pages, "v_pages")):
        _req(t, torch.float16, n)
    _req(tok_page_table, torch.int32, "tok_page_table")
    _req(tok_kv_len, torch.int32, "tok_kv_len")
    T, Hq, d = q.shape
    N, Hkv, P, d2 = k_pages.shape
    if d2 != d:
        raise ValueError("head_dim of q and k_pages differ")
    max_pages = tok_page_table.shape[1]
    if out is None:
        out = torch.empty_like(q)
    _req(out, torch.float16, "out")
    if workspace is None:
        workspace = new_workspace(T, Hq, Hkv, d, q.device)
    st = getattr(_lib, fn_name)(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(tok_page_table),
                                max_pages, _ptr(tok_kv_len), T, Hq, Hkv, P, d, N, float(scale),
                                _ptr(out), _ptr(workspace), workspace.numel(), _stream(stream))
    _check(st, fn_name)
    return out


def forward(q, k_pages, v_pages, tok_page_table, tok_kv_len, scale, out=None, workspace=None,
            stream=None):
    """Plan + prefill + decode for one ubatch; returns out [T][Hq][d] float16."""
    return _attn("paged_attn_forward", q, k_pages, v_pages, tok_page_table, tok_kv_len, scale,
                 out, workspace, stream)


def run(q, k_pages, v_pages, tok_page_table, tok_kv_len, scale, out=None, workspace=None,
        stream=None):
    """Prefill + decode of an already planned ubatch."""
    return _attn("paged_attn_run", q, k_pages, v_pages, tok_page_table, tok_kv_len, scale, out,
                 workspace, stream)


def prefill(q, k_pages, v_pages, tok_page_table, tok_kv_len, scale, out, workspace, stream=None):
    return _attn("paged_attn_prefill", q, k_pages, v_pages, tok_page_table, tok_kv_len, scale, out,
                 workspace, stream)


def decode(q, k_pages, v_pages, tok_page_table, tok_kv_len, scale, out, workspace, stream=None):
    return _attn("paged_attn_decode", q, k_pages, v_pages, tok_page_table, tok_kv_len, scale, out,
                 workspace, stream)


def decode_append(q, k_new, v_new, slot_mapping, k_pages, v_pages, tok_page_table, tok_kv_len,
                  scale, out, workspace, stream=None):
    """decode with the decode tokens' K/V append fused into the same launch (f16 pages):
    equals kv_append(k_new, v_new, slot_mapping, ...) then decode(...)."""
    for t, n in ((q, "q"), (k_new, "k_new"), (v_new, "v_new"), (k_pages, "k_pages"),
                 (v_pages, "v_pages"), (out, "out")):
        _req(t, torch.float16, n)
    _req(slot_mapping, torch.int64, "slot_mapping")
    _req(tok_page_table, torch.int32, "tok_page_table")
    _req(tok_kv_len, torch.int32, "tok_kv_len")
    T, Hq, d = q.shape
    N, Hkv, P, _ = k_pages.shape
    _check(_lib.paged_attn_decode_append(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(slot_mapping), _ptr(k_pages), _ptr(v_pages),
        _ptr(tok_page_table), tok_page_table.shape[1], _ptr(tok_kv_len), T, Hq, Hkv, P, d, N,
        float(scale), _ptr(out), _ptr(workspace), workspace.numel(), _stream(stream)),
        "paged_attn_decode_append")
    return out


def diff_workspace_size(T: int, Hq: int, Hkv: int, d: int) -> int:
    return int(_lib.paged_attn_diff_workspace_size(T, Hq, Hkv, d))


def new_diff_workspace(T: int, Hq: int, Hkv: int, d: int, device=None) -> torch.Tensor:
    """Workspace of the differential attention (plan_diff, diff_run, diff_forward)."""
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        n = diff_workspace_size(T, Hq, Hkv, d)
        if n == 0:
            raise PagedAttnError(PA_EUNSUPPORTED, "diff_workspace_size")
        return torch.empty(n, dtype=torch.uint8, device="cuda")


def _plan(fn_name, tok_page_table, tok_kv_len, Hq, Hkv, P, d, window, workspace, stream):
    dev = tok_page_table.device
    T, max_pages = tok_page_table.shape
    _req_on(tok_page_table, torch.int32, (T, max_pages), dev, "tok_page_table")
    _req_on(tok_kv_len, torch.int32, (T,), dev, "tok_kv_len")
    _req_on(workspace, torch.uint8, (workspace.numel(),), dev, "workspace")
    _call(fn_name, getattr(_lib, fn_name), dev,
          (tok_page_table.data_ptr(), max_pages, tok_kv_len.data_ptr(), T, Hq, Hkv, P, d, *window,
           workspace.data_ptr(), workspace.numel(), _raw_stream(stream, dev)))


def plan_diff(tok_page_table, tok_kv_len, Hq, Hkv, P, d, workspace, stream=None):
    """plan for diff_run (workspace from new_diff_workspace)."""
    _plan("paged_attn_plan_diff", tok_page_table, tok_kv_len, Hq, Hkv, P, d, (), workspace, stream)


def plan_window(tok_page_table, tok_kv_len, Hq, Hkv, P, d, window, workspace, stream=None):
    """plan for window_run: every token attends to its last `window` positions."""
    _plan("paged_attn_plan_window", tok_page_table, tok_kv_len, Hq, Hkv, P, d, (_int32(window),),
          workspace, stream)


def _attn_on(fn_name, q, k_pages, v_pages, tok_page_table, tok_kv_len, scale, extra, vectors, out,
             workspace, new_ws, stream):
    """Checks and marshals an attention call whose own arguments (`extra`) stand between the
    scale and the output; `vectors`: its float32 tensors, as (tensor or None, length, name)."""
    dev = q.device
    T, Hq, d = q.shape
    N, Hkv, P, _ = k_pages.shape
    max_pages = tok_page_table.shape[1]
    f16, i32 = torch.float16, torch.int32
    _req_all(dev, (q, f16, (T, Hq, d), "q"), (k_pages, f16, (N, Hkv, P, d), "k_pages"),
             (v_pages, f16, (N, Hkv, P, d), "v_pages"),
             (tok_page_table, i32, (T, max_pages), "tok_page_table"),
             (tok_kv_len, i32, (T,), "tok_kv_len"))
    for t, n, name in vectors:
        if t is not None:
            _req_on(t, torch.float32, (n,), dev, name)
    if out is None:
        out = torch.empty_like(q)
        _used_on(stream, out)
    else:
        _req_on(out, torch.float16, (T, Hq, d), dev, "out")
    if workspace is None:
        workspace = new_ws(T, Hq, Hkv, d, dev)
        _used_on(stream, workspace)
    else:
        _req_on(workspace, torch.uint8, (workspace.numel(),), dev, "workspace")
    _call(fn_name, getattr(_lib, fn_name), dev,
          (q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), tok_page_table.data_ptr(),
           max_pages, tok_kv_len.data_ptr(), T, Hq, Hkv, P, d, N, scale, *extra, out.data_ptr(),
           workspace.data_ptr(), workspace.numel(), _raw_stream(stream, dev)))
    return out


def _diff(fn_name, q, k_pages, v_pages, tok_page_table, tok_kv_len, scale, lam, norm_weight, eps,
          out_scale, out, workspace, stream):
    if lam is None:
        raise ValueError("lam (the weight of each head's second map) is required")
    return _attn_on(
        fn_name, q, k_pages, v_pages, tok_page_table, tok_kv_len, scale,
        (lam.data_ptr(), None if norm_weight is None else norm_weight.data_ptr(), eps, out_scale),
        ((lam, q.shape[1], "lam"), (norm_weight, q.shape[2], "norm_weight")), out, workspace,
        new_diff_workspace, stream)


def diff_run(q, k_pages, v_pages, tok_page_table, tok_kv_len, scale, lam, norm_weight=None,
             eps=1e-5, out_scale=1.0, out=None, workspace=None, stream=None):
    """Differential attention on a plan from plan_diff.  q rows are (q1 | q2) and cached K rows
    (k1 | k2), halves of d / 2: out = norm(softmax(q1 k1) V - lam softmax(q2 k2) V) * out_scale,
    the norm (norm_weight [d]) over each head's d values; None: no norm."""
    if workspace is None:
        raise ValueError("diff_run needs the workspace that plan_diff planned in")
    return _diff("paged_attn_diff_run", q, k_pages, v_pages, tok_page_table, tok_kv_len, scale,
                 lam, norm_weight, eps, out_scale, out, workspace, stream)


def diff_forward(q, k_pages, v_pages, tok_page_table, tok_kv_len, scale, lam, norm_weight=None,
                 eps=1e-5, out_scale=1.0, out=None, workspace=None, stream=None):
    """plan_diff then diff_run for one ubatch; returns out [T][Hq][d] float16."""
    return _diff("paged_attn_diff_forward", q, k_pages, v_pages, tok_page_table, tok_kv_len, scale,
                 lam, norm_weight, eps, out_scale, out, workspace, stream)


def window_run(q, k_pages, v_pages, tok_page_table, tok_kv_len, scale, sink=None, out=None,
               workspace=None, stream=None):
    """Attention to the last positions of each token (the window of the plan, made by
    plan_window); sink [Hq]: a logit per query head that joins the softmax with no value."""
    if workspace is None:
        raise ValueError("window_run needs the workspace that plan_window planned in")
    return _attn_on("paged_attn_window_run", q, k_pages, v_pages, tok_page_table, tok_kv_len,
                    scale, (None if sink is None else sink.data_ptr(),),
                    ((sink, q.shape[1], "sink"),), out, workspace, None, stream)


def window_forward(q, k_pages, v_pages, tok_page_table, tok_kv_len, scale, window, sink=None,
                   out=None, workspace=None, stream=None):
    """plan_window then window_run for one ubatch; returns out [T][Hq][d] float16."""
    return _attn_on("paged_attn_window_forward", q, k_pages, v_pages, tok_page_table, tok_kv_len,
                    scale, (_int32(window), None if sink is None else sink.data_ptr()),
                    ((sink, q.shape[1], "sink"),), out, workspace, new_workspace, stream)


def validate(tok_page_table, tok_kv_len, P, num_pages, err, stream=None):
    T, max_pages = tok_page_table.shape
    _check(_lib.paged_attn_validate(_ptr(tok_page_table), max_pages, _ptr(tok_kv_len), T, P,
                                    num_pages, _ptr(err), _stream(stream)), "paged_attn_validate")


def read_error(workspace, stream=None) -> int:
    """Synchronise and return the workspace's device error word (PA_ERR_* bits)."""
    v = ctypes.c_int(0)
    st = _lib.paged_attn_read_error(_ptr(workspace), ctypes.byref(v), _stream(stream))
    if st not in (PA_OK, PA_EDEVICE):
        raise PagedAttnError(st, "paged_attn_read_error")
    return int(v.value)


def set_decode_wait_limit(ns: int) -> int:
    """Limit (ns) of the split-KV decode kernel's bounded waits (0: the 2 s default).
    Returns the previous value."""
    return int(_lib.paged_attn_set_decode_wait_limit(int(ns)))


def set_prefill_min_run(n: int) -> int:
    """Shortest same-row run sent to the tensor-core prefill path; returns the old value."""
    return int(_lib.paged_attn_set_prefill_min_run(int(n)))


class PagePool:
    """Host page allocator (native): lowest-id-first free list, reference counts."""

    def __init__(self, num_pages: int):
        self._h = _lib.pa_pool_create(int(num_pages))
        if not self._h:
            raise PagedAttnError(PA_EINVAL, "pa_pool_create")
        self.num_pages = int(num_pages)

    def __del__(self):
        h = getattr(self, "_h", None)
        if h:
            _lib.pa_pool_destroy(h)
            self._h = None

    @property
    def num_free(self) -> int:
        return int(_lib.pa_pool_num_free(self._h))

    def alloc(self, n: int):
        buf = (ctypes.c_int32 * max(n, 1))()
        st = _lib.pa_pool_alloc(self._h, int(n), buf)
        if st < 0:
            raise PagedAttnError(st, "pa_pool_alloc")
        return [int(buf[i]) for i in range(n)]

    def share(self, pages):
        buf = (ctypes.c_int32 * max(len(pages), 1))(*pages)
        _check(_lib.pa_pool_share(self._h, buf, len(pages)), "pa_pool_share")

    def release(self, pages):
        buf = (ctypes.c_int32 * max(len(pages), 1))(*pages)
        _check(_lib.pa_pool_release(self._h, buf, len(pages)), "pa_pool_release")

    def refcount(self, page: int) -> int:
        return int(_lib.pa_pool_refcount(self._h, int(page)))

    def fork(self, pages, n_tokens: int, P: int):
        """Copy-on-write fork of a sequence holding n_tokens tokens in `pages`.
        Returns (child pages, (src, dst) page pair to copy, or None)."""
        n = (int(n_tokens) + P - 1) // P
        buf = (ctypes.c_int32 * max(n, 1))(*pages[:n])
        out = (ctypes.c_int32 * max(n, 1))()
        cs, cd = ctypes.c_int32(-1), ctypes.c_int32(-1)
        st = _lib.pa_pool_fork(self._h, buf, int(n_tokens), int(P), out, ctypes.byref(cs),
                               ctypes.byref(cd))
        if st < 0:
            raise PagedAttnError(st, "pa_pool_fork")
        return [int(out[i]) for i in range(n)], ((int(cs.value), int(cd.value)) if st else None)
