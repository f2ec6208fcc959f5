"""ctypes binding of the serving operators of libm3.so (include/m3_ops.h),
under the same names.

Argument marshalling only: shapes, types, devices and layouts are checked
here, numbers and alignment in the library.  Tensors are torch tensors of one
GPU; the work goes to `stream`, by default the current stream of that GPU.
Outputs are the caller's tensors.  There is no CPU fallback.
"""
from __future__ import annotations

import ctypes as C

import torch

from .m3 import M3_EINVAL, M3_KV_BF16, M3_KV_F16, M3Error, _check, lib

EXPORTED = ("m3_kv_map", "m3_kv_store", "m3_attn_prompt", "m3_attn_prefix_workspace",
            "m3_attn_prefix", "m3_logit_rules", "m3_ops_sync_status")

M3_LOGITS_F32, M3_LOGITS_BF16, M3_LOGITS_F16 = 0, 1, 2

_KV = {torch.bfloat16: M3_KV_BF16, torch.float16: M3_KV_F16}
_LOGITS = {torch.float32: M3_LOGITS_F32, torch.bfloat16: M3_LOGITS_BF16,
           torch.float16: M3_LOGITS_F16}
_I32, _I64, _F32 = torch.int32, torch.int64, torch.float32


def _setup():
    vp, i32, i64, f32 = C.c_void_p, C.c_int, C.c_int64, C.c_float
    lib.m3_kv_map.argtypes = [i32, vp, vp, vp, i32, vp, vp, i32, i64, i32, i32, i32, i32, vp, vp,
                              vp, vp, vp, vp, vp]
    lib.m3_kv_store.argtypes = [i32, i32, i32, i32, vp, i64, i64, vp, i64, i64, vp, vp, i32, i32,
                                vp]
    lib.m3_attn_prompt.argtypes = [i32, i32, i32, i32, i32, i32, i32, vp, i64, i64, vp, i64, i64,
                                   vp, i64, i64, vp, vp, f32, vp, i64, i64, vp, vp]
    lib.m3_attn_prefix_workspace.argtypes = [i32] * 7
    lib.m3_attn_prefix.argtypes = [i32, i32, i32, i32, i32, vp, i64, i64, vp, i32, i32, vp, i32,
                                   i32, vp, i32, i64, vp, f32, vp, i64, i64, vp, vp, i64, vp]
    lib.m3_logit_rules.argtypes = [i32, i32, i32, vp, i64, vp, i64, vp, i32, i64, vp, vp, vp, vp,
                                   vp, vp, i32, vp, i32, vp, vp]
    lib.m3_ops_sync_status.argtypes = [vp]
    for n in EXPORTED:
        getattr(lib, n).restype = C.c_int
    lib.m3_attn_prefix_workspace.restype = C.c_int64


_setup()


def _refuse(what: str):
    raise M3Error(M3_EINVAL, what)


def _arr(name: str, t, dtype, shape, dev):
    """The address of a contiguous tensor of this type, shape and device (None: null)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.device != dev:
        _refuse(f"{name}: a contiguous {dtype} tensor of shape {tuple(shape)} on {dev} is wanted")
    return t.data_ptr()


def _call(fn, dev, stream, *args) -> None:
    if dev.type != "cuda":
        _refuse("the tensors have to be on a GPU")
    if stream is not None and stream.device != dev:
        _refuse("the stream belongs to another device")
    if dev.index == torch.cuda.current_device():
        rc = fn(*args, torch.cuda.current_stream(dev).cuda_stream if stream is None
                else stream.cuda_stream)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, torch.cuda.current_stream(dev).cuda_stream if stream is None
                    else stream.cuda_stream)
    if rc:
        _check(rc)


def _heads(name: str, t, n, dtype, dev):
    """(address, row stride, head stride) of a [n, heads, D] tensor with D contiguous."""
    if t.dtype is not dtype or t.device != dev or t.dim() != 3 or t.shape[0] != n:
        _refuse(f"{name}: a {dtype} tensor [{n}, heads, D] on {dev} is wanted")
    a, b, c = t.stride()
    if c != 1 and t.shape[2] > 1:
        _refuse(f"{name}: the last dimension has to be contiguous")
    return t.data_ptr(), a, b


def m3_kv_map(fresh, cached, free_pages, table, page: int, n_pages: int, cu, positions, slots,
              seqs, lens, taken, start: int = 0, free_at=None, stream=None) -> None:
    """Page tables and slot maps from the requests' lengths (see m3_ops.h).
    table int32 [requests, max_pages], rows may be strided; in and out."""
    dev = fresh.device
    n = fresh.numel()
    if table.dtype is not _I32 or table.dim() != 2 or table.shape[0] != n or \
            table.device != dev or (table.stride(1) != 1 and table.shape[1] > 1):
        _refuse("table: an int32 tensor [requests, max_pages] with contiguous rows is wanted")
    nt = slots.numel()
    _call(lib.m3_kv_map, dev, stream, n, _arr("fresh", fresh, _I32, (n,), dev),
          _arr("cached", cached, _I32, (n,), dev),
          _arr("free_pages", free_pages, _I32, (free_pages.numel(),), dev), free_pages.numel(),
          _arr("free_at", free_at, _I32, (1,), dev), table.data_ptr(), table.shape[1],
          table.stride(0), page, n_pages, start, nt, _arr("cu", cu, _I32, (n + 1,), dev),
          _arr("positions", positions, _I32, (nt,), dev), _arr("slots", slots, _I64, (nt,), dev),
          _arr("seqs", seqs, _I32, (nt,), dev), _arr("lens", lens, _I32, (n,), dev),
          _arr("taken", taken, _I32, (1,), dev))


def _pool(pool, dtype, dev):
    if pool.dtype is not dtype or pool.dim() != 5 or pool.shape[1] != 2 or \
            not pool.is_contiguous() or pool.device != dev:
        _refuse(f"pool: a contiguous {dtype} tensor [pages, 2, kv heads, page, D] is wanted")
    return pool.data_ptr()


def _kv_type(t):
    if t.dtype not in _KV:
        _refuse("the type has to be bfloat16 or float16")
    return _KV[t.dtype]


def m3_kv_store(k, v, slots, pool, stream=None) -> None:
    """k, v [tokens, kv heads, D] into the pool's slots (see m3_ops.h)."""
    dev, n = k.device, slots.numel()
    dt = _kv_type(k)
    p = _pool(pool, k.dtype, dev)
    n_pages, _, hk, page, d = pool.shape
    ka, kt, kh = _heads("k", k, n, k.dtype, dev)
    va, vt, vh = _heads("v", v, n, k.dtype, dev)
    if k.shape[1:] != (hk, d) or v.shape[1:] != (hk, d):
        _refuse("k, v and the pool differ in heads or D")
    _call(lib.m3_kv_store, dev, stream, dt, n, hk, d, ka, kt, kh, va, vt, vh,
          _arr("slots", slots, _I64, (n,), dev), p, n_pages, page)


def m3_attn_prompt(q, k, v, cu_q, out, lse=None, cu_k=None, scale: float | None = None,
                   stream=None) -> None:
    """Causal attention over packed sequences (see m3_ops.h): q, out [n_q, heads, D],
    k, v [n_k, kv heads, D], lse float32 [n_q, heads]; scale: by default D^-0.5."""
    dev, dt = q.device, _kv_type(q)
    n_q, n_k = q.shape[0], k.shape[0]
    qa, qt, qh = _heads("q", q, n_q, q.dtype, dev)
    ka, kt, kh = _heads("k", k, n_k, q.dtype, dev)
    va, vt, vh = _heads("v", v, n_k, q.dtype, dev)
    oa, ot, oh = _heads("out", out, n_q, q.dtype, dev)
    _, hq, d = q.shape
    hk = k.shape[1]
    if k.shape[2] != d or v.shape[1:] != (hk, d) or out.shape[1:] != (hq, d):
        _refuse("q, k, v and out differ in heads or D")
    ns = cu_q.numel() - 1
    _call(lib.m3_attn_prompt, dev, stream, dt, ns, n_q, n_k, hq, hk, d, qa, qt, qh, ka, kt, kh,
          va, vt, vh, _arr("cu_q", cu_q, _I32, (ns + 1,), dev),
          _arr("cu_k", cu_k, _I32, (ns + 1,), dev), d ** -0.5 if scale is None else scale, oa, ot,
          oh, _arr("lse", lse, _F32, (n_q, hq), dev))


def m3_attn_prefix_workspace(n_rows: int, heads: int, kv_heads: int, d: int, prefix_pages: int,
                             page: int, max_pages: int) -> int:
    """Bytes of workspace of such an m3_attn_prefix call (see m3_ops.h)."""
    return lib.m3_attn_prefix_workspace(n_rows, heads, kv_heads, d, prefix_pages, page, max_pages)


def m3_attn_prefix(q, pool, prefix_pages, prefix_len: int, table, lens, out, lse=None,
                   scale: float | None = None, workspace=None, stream=None) -> None:
    """One-token attention of rows that share a prefix (see m3_ops.h): q, out
    [rows, heads, D], pool [pages, 2, kv heads, page, D], table int32 [rows, max_pages];
    workspace: a uint8 tensor, by default a new one."""
    dev, dt, n = q.device, _kv_type(q), q.shape[0]
    qa, qr, qh = _heads("q", q, n, q.dtype, dev)
    oa, orow, oh = _heads("out", out, n, q.dtype, dev)
    p = _pool(pool, q.dtype, dev)
    _, hq, d = q.shape
    n_pages, _, hk, page, pd = pool.shape
    if pd != d or out.shape[1:] != (hq, d):
        _refuse("q, the pool and out differ in heads or D")
    if table.dtype is not _I32 or table.dim() != 2 or table.shape[0] != n or \
            table.device != dev or (table.stride(1) != 1 and table.shape[1] > 1):
        _refuse("table: an int32 tensor [rows, max_pages] with contiguous rows is wanted")
    npp, mp = prefix_pages.numel(), table.shape[1]
    if workspace is None:
        size = lib.m3_attn_prefix_workspace(n, hq, hk, d, npp, page, mp)
        workspace = torch.empty(size, dtype=torch.uint8, device=dev)
        if stream is not None:
            workspace.record_stream(stream)
    elif workspace.device != dev or not workspace.is_contiguous():
        _refuse(f"workspace: a contiguous tensor on {dev} is wanted")
    _call(lib.m3_attn_prefix, dev, stream, dt, n, hq, hk, d, qa, qr, qh, p, n_pages, page,
          _arr("prefix_pages", prefix_pages, _I32, (npp,), dev), npp, prefix_len,
          table.data_ptr(), mp, table.stride(0), _arr("lens", lens, _I32, (n,), dev),
          d ** -0.5 if scale is None else scale, oa, orow, oh,
          _arr("lse", lse, _F32, (n, hq), dev), workspace.data_ptr(),
          workspace.numel() * workspace.element_size())


def m3_logit_rules(logits, out, history=None, hist_len=None, repetition=None, frequency=None,
                   presence=None, bias_ids=None, bias=None, mask=None, mask_row=None,
                   stream=None) -> None:
    """Penalties, biases and grammar masks (see m3_ops.h) on logits [rows, vocab]
    (rows may be strided); out: another such tensor, or logits itself.  history int32
    [rows, n], bias_ids int32 and bias float32 [rows, n], mask int32 [masks, words]."""
    dev = logits.device
    if logits.dtype not in _LOGITS or logits.dim() != 2:
        _refuse("logits: a float32, bfloat16 or float16 tensor [rows, vocab] is wanted")
    r, n = logits.shape
    if out.dtype is not logits.dtype or out.shape != logits.shape or out.device != dev:
        _refuse("out has to be like logits")
    if n > 1 and (logits.stride(1) != 1 or out.stride(1) != 1):
        _refuse("logits and out: rows have to be contiguous")
    nh = ldh = 0
    ha = None
    if history is not None:
        if history.dtype is not _I32 or history.dim() != 2 or history.shape[0] != r or \
                history.device != dev or (history.stride(1) != 1 and history.shape[1] > 1):
            _refuse("history: an int32 tensor [rows, n] with contiguous rows is wanted")
        ha, nh, ldh = history.data_ptr(), history.shape[1], history.stride(0)
    if (bias_ids is None) != (bias is None):
        _refuse("bias_ids and bias come together")
    nb = 0 if bias is None else bias.shape[-1]
    nm = 0
    if mask is not None:
        nm = mask.shape[0]
    _call(lib.m3_logit_rules, dev, stream, _LOGITS[logits.dtype], r, n, logits.data_ptr(),
          logits.stride(0), out.data_ptr(), out.stride(0), ha, nh, ldh,
          _arr("hist_len", hist_len, _I32, (r,), dev),
          _arr("repetition", repetition, _F32, (r,), dev),
          _arr("frequency", frequency, _F32, (r,), dev),
          _arr("presence", presence, _F32, (r,), dev),
          _arr("bias_ids", bias_ids, _I32, (r, nb), dev), _arr("bias", bias, _F32, (r, nb), dev),
          nb, _arr("mask", mask, _I32, (nm, (n + 31) // 32), dev), nm,
          _arr("mask_row", mask_row, _I32, (r,), dev))


def m3_ops_sync_status(stream=None) -> None:
    """Wait for the stream and raise what a kernel of these calls recorded (see m3_ops.h)."""
    st = torch.cuda.current_stream() if stream is None else stream
    with torch.cuda.device(st.device):
        _check(lib.m3_ops_sync_status(st.cuda_stream))
