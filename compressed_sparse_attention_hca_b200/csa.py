"""Thin ctypes binding of libcsa_b200 (include/csa.h): argument marshalling only.

Every function takes torch tensors that already live on the CUDA device,
passes their data pointers and the current CUDA stream to the C ABI, and
returns the output tensors.  All arithmetic runs in the library's kernels;
there is no CPU fallback: if the shared library is missing or a call fails,
an exception is raised.
"""
from __future__ import annotations

import ctypes
import os
import re

import torch

F32, BF16, KV_FP8MIX, IDX_NVFP4 = 0, 1, 2, 3
_STATUS = {0: "CSA_OK", 1: "CSA_ERR_INVALID_ARG", 2: "CSA_ERR_UNSUPPORTED", 3: "CSA_ERR_CUDA",
           4: "CSA_ERR_TIMEOUT"}

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libcsa_b200.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "csa.h")
_lib = None


class CsaError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__(f"{_STATUS.get(status, status)}: {msg}")
        self.status = status


def header_functions():
    """Names of the functions declared in include/csa.h."""
    src = open(HEADER).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    return sorted(set(re.findall(r"\b(csa_\w+|hca_\w+)\s*\(", src)))


def load():
    """Load libcsa_b200.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: run `python -m compressed_sparse_attention_hca_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P, i32, i64, sz, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    sigs = {
        "csa_last_error": (ctypes.c_char_p, []),
        "csa_version": (i32, []),
        "csa_last_launch_count": (i32, []),
        "csa_check_device_status": (i32, []),
        "csa_row_bytes": (i64, [i32, i32]),
        "csa_nvfp4_key_scale_bytes": (i64, [i64, i32]),
        "csa_compress": (i32, [P, P, P, P, P, P, i32, i64, i64, i64, i64, i64, i32, i32, i32, P, P,
                               i64, i64, i32, P]),
        "csa_rmsnorm_rope": (i32, [P, P, i64, i32, P, f32, P, i32, i32, i32, ctypes.c_double, i32, i32, P]),
        "csa_index_topk_workspace_size": (sz, [i32, i32, i64, i32, i32, i32, i32]),
        "csa_index_topk_plan": (i32, [i32, i32, i64, i32, i32, i32, i32, P]),
        "csa_compress_index_topk": (i32, [ctypes.POINTER(CompressJob), ctypes.POINTER(CompressJob),
                                          P, P, P, P, P, P, i32, i32, i64, i32, i32, i32, i32, i32,
                                          P, P, P, sz, P]),
        "csa_index_topk": (i32, [P, P, P, P, P, P, i32, i32, i64, i32, i32, i32, i32, i32, P, P, P,
                                 sz, P]),
        "csa_sparse_mqa_workspace_size": (sz, [i32, i32, i32, i32, i32, i32, i32, i32]),
        "csa_sparse_mqa": (i32, [P, i32, P, i64, P, i32, P, i64, P, P, i32, i32, P, f32, i32, i32,
                                 i32, i32, i32, P, P, sz, P]),
        "hca_dense_mqa_workspace_size": (sz, [i32, i32, i32, i32, i64, i32, i32, i32]),
        "hca_dense_mqa": (i32, [P, i32, P, i64, P, i64, P, P, i32, i32, P, f32, i32, i32, i32, i32,
                                i32, P, P, sz, P]),
        "csa_mqa_workspace_size": (sz, [i32, i32, i32, i32, i64, i32, i32, ctypes.POINTER(MqaOptions)]),
        "csa_sparse_mqa_ex": (i32, [P, i32, P, i64, P, i32, P, i64, P, P, i32, i32, P, f32, i32, i32,
                                    i32, i32, i32, P, P, sz, ctypes.POINTER(MqaOptions), P]),
        "hca_dense_mqa_ex": (i32, [P, i32, P, i64, P, i64, P, P, i32, i32, P, f32, i32, i32, i32, i32,
                                   i32, P, P, sz, ctypes.POINTER(MqaOptions), P]),
        "csa_compress_ex": (i32, [ctypes.POINTER(CompressJob), i32, P]),
        "csa_index_topk_paged": (i32, [P, P, P, P, P, ctypes.POINTER(Pages), P, i32, i32, i64, i32, i32, i32, i32,
                                       i32, P, P, P, sz, P]),
        "csa_grouped_out_proj_workspace_size": (sz, [i32, i32, i32, i32, i32, i32]),
        "csa_grouped_out_proj_plan": (i32, [i32, i32, i32, i32, i32, i32, P]),
        "csa_grouped_out_proj": (i32, [P, P, P, P, i32, i32, i32, i32, i32, i32, P, sz, P]),
        "csa_page_plan": (i32, [P, P, i32, i32, P, i32, P, P, P, i64, P, i32, P, P]),
        "csa_quant_nvfp4": (i32, [P, i64, i32, i64, i32, f32, P, i64, P, i64, i32, P, P, P, P]),
        "csa_nvfp4_linear_workspace_size": (sz, [i32, i32, i32]),
        "csa_nvfp4_linear": (i32, [P, P, P, P, f32, P, i32, i32, i32, i32, P, sz, P]),
        "csa_tree_mqa_workspace_size": (sz, [i32, i32, i32, i32, i64, i32, i32, ctypes.POINTER(MqaOptions)]),
        "csa_tree_mqa": (i32, [P, i32, P, i64, P, i32, P, i64, P, P, i32, P, P, P, P, i32, i32, P, f32, i32, i32,
                               i32, i32, i32, P, P, sz, ctypes.POINTER(MqaOptions), P]),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    _lib = lib
    return lib


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _check(status):
    if status != 0:
        raise CsaError(status, load().csa_last_error().decode())


def _dt_of(t):
    return F32 if t.dtype == torch.float32 else BF16


def check_device_status():
    """Synchronises the device; raises CsaError if a kernel wait timed out."""
    _check(load().csa_check_device_status())


def last_launch_count():
    """Kernels launched by this thread's last library call."""
    return int(load().csa_last_launch_count())


def row_bytes(dt, dim):
    return int(load().csa_row_bytes(dt, dim))


def nvfp4_key_scale_bytes(n_rows, dim):
    """Bytes of one request's blocked NVFP4 key-scale array."""
    return int(load().csa_nvfp4_key_scale_bytes(n_rows, dim))


def _need_cuda(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("all tensors must be contiguous CUDA tensors")


# The current device and the raw handle of its current stream: the public calls
# build objects that take longer than a small kernel.
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_current_stream = (getattr(torch._C, "_cuda_getCurrentRawStream", None) or
                   (lambda dev: torch.cuda.current_stream(dev).cuda_stream))
_F32, _BF16, _I32, _I64, _U8 = torch.float32, torch.bfloat16, torch.int32, torch.int64, torch.uint8


def _need(dev, dtype, what, ts):
    """All tensors contiguous, of `dtype` and on device `dev` (the current one,
    which the call launches on)."""
    for t in ts:
        if t is not None:
            if t.get_device() != dev or not t.is_contiguous():
                raise ValueError("all tensors must be contiguous and on the current CUDA device")
            if t.dtype is not dtype:
                raise ValueError(f"{what} must be {dtype}")


def _device_of(t):
    """The current device, which must be the tensor's (so CUDA is in use)."""
    dev = t.get_device()
    if dev < 0 or dev != _current_device():
        raise ValueError("all tensors must be contiguous and on the current CUDA device")
    return dev


# ------------------------------------------------------------------ paged cache

class Pages(ctypes.Structure):
    """csa_pages_t: the block table of a paged cache."""
    _fields_ = [("table", ctypes.c_void_p), ("max_pages", ctypes.c_int32), ("page_entries", ctypes.c_int32),
                ("n_pages", ctypes.c_int64)]


def pages(table, page_entries, n_pages):
    """A block table: table [batch, max_pages] int32 (CUDA) of pool pages of
    page_entries rows each; n_pages pages in the pool."""
    _need_cuda(table)
    if table.dtype != torch.int32 or table.dim() != 2:
        raise ValueError("table must be a [batch, max_pages] int32 tensor")
    p = Pages(table=table.data_ptr(), max_pages=table.shape[1], page_entries=page_entries, n_pages=n_pages)
    p._keep = table  # the struct holds a raw pointer: keep the tensor alive with it
    return p


class SlotMap(ctypes.Structure):
    """csa_slot_map_t: pool rows of a step's new rows in one paged cache, as
    the tensors row_start [batch + 1] int64, slots and sf_slots [capacity]
    int32 (sf_slots None when not asked for)."""
    _fields_ = [("_m", ctypes.c_int32), ("_capacity", ctypes.c_int64), ("_row_start", ctypes.c_void_p),
                ("_slots", ctypes.c_void_p), ("_sf_slots", ctypes.c_void_p)]


def slot_map(m, batch, capacity, *, scales=False, row_start=None, slots=None, sf_slots=None, device="cuda"):
    """A SlotMap for caches of one row per m tokens, for page_plan() to fill;
    its tensors are allocated when not given (sf_slots only with scales)."""
    if row_start is None:
        row_start = torch.empty(batch + 1, dtype=torch.int64, device=device)
    if slots is None:
        slots = torch.empty(capacity, dtype=torch.int32, device=device)
    if sf_slots is None and scales:
        sf_slots = torch.empty(capacity, dtype=torch.int32, device=device)
    _need_cuda(row_start, slots, sf_slots)
    if row_start.dtype is not _I64 or slots.dtype is not _I32 or (sf_slots is not None and sf_slots.dtype is not _I32):
        raise ValueError("row_start must be int64, slots and sf_slots int32")
    if row_start.numel() < batch + 1 or slots.numel() < capacity or (sf_slots is not None and
                                                                      sf_slots.numel() < capacity):
        raise ValueError("row_start needs batch + 1 places, slots and sf_slots capacity")
    s = SlotMap(m, capacity, row_start.data_ptr(), slots.data_ptr(), sf_slots.data_ptr() if sf_slots is not None
                else None)
    s.row_start, s.slots, s.sf_slots, s.batch = row_start, slots, sf_slots, batch
    s.device = slots.get_device()
    if row_start.get_device() != s.device or (sf_slots is not None and sf_slots.get_device() != s.device):
        raise ValueError("row_start, slots and sf_slots must be on one device")
    return s


def page_plan(len_before, len_after, page_tokens, table, free_list, free_count, *, maps=(), info=None,
              free_count_out=None):
    """Block tables and slot maps of a step: requests change from len_before to
    len_after tokens ([batch] int64), pages of page_tokens tokens are taken
    from and given back to the stack free_list [n_pages] int32 (free_count [1]
    int32, updated in place unless free_count_out is given), table [batch,
    max_pages] int32 and the SlotMaps `maps` (slot_map()) are filled.  Returns
    info [4] int32: pages taken, given back, not to be had, and the call's
    counter (info given by the caller must start as zeros)."""
    if info is None:
        info = torch.zeros(4, dtype=_I32, device=table.device)
    out = free_count if free_count_out is None else free_count_out
    dev = _device_of(table)
    _need(dev, _I64, "lengths", (len_before, len_after))
    _need(dev, _I32, "table, free_list, free_count and info", (table, free_list, free_count, out, info))
    batch = len_before.numel()
    if table.dim() != 2 or table.shape[0] != batch or len_after.numel() != batch or info.numel() < 4:
        raise ValueError("table must be [batch, max_pages], the lengths [batch] and info [4]")
    if free_count.numel() < 1 or out.numel() < 1:
        raise ValueError("free_count must hold a number")
    for m in maps:
        if m.batch != batch or m.device != dev:
            raise ValueError("every slot map must be made for this batch, on the current CUDA device")
    n = len(maps)
    each = ctypes.byref(maps[0]) if n == 1 else (SlotMap * n)(*maps) if n else None
    _check((_lib or load()).csa_page_plan(
        len_before.data_ptr(), len_after.data_ptr(), batch, page_tokens, table.data_ptr(), table.shape[1],
        free_list.data_ptr(), free_count.data_ptr(), out.data_ptr(), free_list.numel(),
        each, n, info.data_ptr(), _current_stream(dev)))
    return info


# ------------------------------------------------------------------ NVFP4 rows

def quant_nvfp4(x, *, x_scale=1.0, blocked=True, rows=None, sf_rows=None, codes=None, sf=None, values=None):
    """Rows of x [..., dim] (F32 or BF16; a 2-D x may have a row stride) to
    NVFP4: codes [rows, dim/2] uint8 and their E4M3 scales, in the blocked
    layout (keys; operands of nvfp4_linear) or row-major [rows, dim/16]
    (queries of index_topk).  rows / sf_rows [n] int32: the place of each row
    in `codes` and of its scales in `sf` (a SlotMap's slots and sf_slots; -1
    skips a row), which must then be given; values [n, dim] bf16: also the
    values the codes stand for.  Returns codes, sf."""
    dim = x.shape[-1]
    n = x.numel() // dim if dim else 0
    stride = dim
    dev = _device_of(x)
    if not x.is_contiguous():
        if x.dim() != 2 or x.stride(1) != 1:
            raise ValueError("x must be contiguous, or rows of it")
        stride = x.stride(0)
    if x.dtype is not _F32 and x.dtype is not _BF16:
        raise ValueError("x must be float32 or bfloat16")
    if dim <= 0 or dim % 64:
        raise ValueError("dim must be a positive multiple of 64")
    if (rows is not None or sf_rows is not None) and (codes is None or sf is None):
        raise ValueError("rows and sf_rows need the codes and sf they point into")
    if codes is None:
        codes = torch.empty(*x.shape[:-1], dim // 2, device=x.device, dtype=torch.uint8)
    if sf is None:
        sf = (torch.zeros(nvfp4_key_scale_bytes(n, dim), device=x.device, dtype=torch.uint8) if blocked else
              torch.empty(*x.shape[:-1], dim // 16, device=x.device, dtype=torch.uint8))
    _need(dev, _U8, "codes and sf", (codes, sf))
    _need(dev, _I32, "rows and sf_rows", (rows, sf_rows))
    _need(dev, _BF16, "values", (values,))
    if (rows is not None and rows.numel() < n) or (sf_rows is not None and sf_rows.numel() < n):
        raise ValueError("rows and sf_rows need a place for every row of x")
    if values is not None and values.numel() < n * dim:
        raise ValueError("values must be [n, dim]")
    sf_n = sf.numel() // (dim // 64 * 512) * 128 if blocked else sf.numel() // (dim // 16)
    _check((_lib or load()).csa_quant_nvfp4(
        x.data_ptr(), n, dim, stride, _dt_of(x), x_scale, codes.data_ptr(), codes.numel() // (dim // 2), sf.data_ptr(),
        sf_n, 1 if blocked else 0, rows.data_ptr() if rows is not None else None,
        sf_rows.data_ptr() if sf_rows is not None else None, values.data_ptr() if values is not None else None,
        _current_stream(dev)))
    return codes, sf


def nvfp4_linear_workspace_size(T, k, n):
    return int(load().csa_nvfp4_linear_workspace_size(T, k, n))


def nvfp4_linear(X, X_sf, W, W_sf, *, alpha=1.0, out=None, out_dt=BF16, ws=None):
    """Y [T, n] = alpha X W^T of NVFP4 matrices X [T, k/2] codes and W [n, k/2]
    codes, each with blocked scales (quant_nvfp4()).  ws: a workspace of
    nvfp4_linear_workspace_size bytes; a fresh one is made when not given."""
    if X.dim() != 2 or W.dim() != 2 or W.shape[1] != X.shape[1]:
        raise ValueError("X must be [T, k/2] and W [n, k/2]")
    T, n = X.shape[0], W.shape[0]
    k = 2 * X.shape[1]
    if ws is None:
        ws = torch.empty(nvfp4_linear_workspace_size(T, k, n), device=X.device, dtype=_U8)
    if out is None:
        out = torch.empty(T, n, device=X.device, dtype=torch.float32 if out_dt == F32 else torch.bfloat16)
    dev = _device_of(X)
    _need(dev, _U8, "codes, scales and ws", (X, X_sf, W, W_sf, ws))
    _need(dev, out.dtype, "out", (out,))
    if out.shape != (T, n) or (out.dtype is not _F32 and out.dtype is not _BF16):
        raise ValueError("out must be [T, n] float32 or bfloat16")
    strip = k // 64 * 512
    if X_sf.numel() < (T + 127) // 128 * strip or W_sf.numel() < (n + 127) // 128 * strip:
        raise ValueError("X_sf and W_sf must be the blocked scales of X and W")
    _check((_lib or load()).csa_nvfp4_linear(
        X.data_ptr(), X_sf.data_ptr(), W.data_ptr(), W_sf.data_ptr(), alpha, out.data_ptr(), _dt_of(out), T, k, n,
        ws.data_ptr(), ws.numel(), _current_stream(dev)))
    return out


# --------------------------------------------------------------------- compress

def compress(Ca, Za, Ba, m, Cb=None, Zb=None, Bb=None, *, tok0=0, e0=0, n_out=None, out_dt=None,
             out=None, out_sf=None, out_row0=0, n_tok=None):
    """Token-level compressor.  Ca/Za [batch, rows, dim] (F32 or BF16), Ba [m, dim] fp32.

    Entry e0 + j of request b goes to row out_row0 + j of out[b] (out:
    [batch, rows, ...]; NVFP4 out_sf: the blocked key scales [batch,
    nvfp4_key_scale_bytes(rows, dim)]; allocated when not given).  Returns out
    (and out_sf for NVFP4)."""
    _need_cuda(Ca, Za, Ba, Cb, Zb, Bb)
    batch, rows, dim = Ca.shape
    n_tok = rows if n_tok is None else n_tok
    in_dt = _dt_of(Ca)
    out_dt = in_dt if out_dt is None else out_dt
    if n_out is None:
        n_out = (tok0 + n_tok) // m - e0
    if out is None:
        stride = n_out + out_row0
        if out_dt in (F32, BF16):
            out = torch.empty(batch, stride, dim, device=Ca.device,
                              dtype=torch.float32 if out_dt == F32 else torch.bfloat16)
        else:
            out = torch.empty(batch, stride, row_bytes(out_dt, dim), device=Ca.device, dtype=torch.uint8)
        if out_dt == IDX_NVFP4:
            out_sf = torch.zeros(batch, nvfp4_key_scale_bytes(stride, dim), device=Ca.device, dtype=torch.uint8)
    _need_cuda(out, out_sf)
    stride = out.shape[1]
    if out_dt == IDX_NVFP4 and out_sf.numel() < batch * nvfp4_key_scale_bytes(stride, dim):
        raise ValueError("out_sf smaller than the blocked key-scale arrays of the cache")
    _check(load().csa_compress(_ptr(Ca), _ptr(Cb), _ptr(Za), _ptr(Zb), _ptr(Ba), _ptr(Bb), batch, n_tok,
                               tok0, rows, e0, n_out, dim, m, in_dt, _ptr(out), _ptr(out_sf), stride,
                               out_row0, out_dt, _stream()))
    return (out, out_sf) if out_dt == IDX_NVFP4 else out


# ------------------------------------------------------ normalisation + partial RoPE

def rmsnorm_rope(x, pos, *, g=None, eps=1e-6, rows_per_pos=1, pos_sign=1, rope_dims=64, base=10000.0,
                 out=None, out_dt=None):
    """RMSNorm (when g is given) and RoPE of the last rope_dims dims of every
    row (last axis) of x; row r uses pos[r // rows_per_pos] (pos int64,
    flattened).  out defaults to a new tensor of out_dt (x's dtype); out=x
    works in place."""
    _need_cuda(x, pos, g, out)
    dim = x.shape[-1]
    n_rows = x.numel() // dim
    in_dt = _dt_of(x)
    out_dt = in_dt if out_dt is None else out_dt
    if out is None:
        out = torch.empty(x.shape, device=x.device, dtype=torch.float32 if out_dt == F32 else torch.bfloat16)
    _check(load().csa_rmsnorm_rope(_ptr(x), _ptr(out), n_rows, dim, _ptr(g), eps, _ptr(pos), rows_per_pos,
                                   pos_sign, rope_dims, base, in_dt, out_dt, _stream()))
    return out


# ------------------------------------------------------------------- index top-k

def index_topk_workspace_size(batch, n_q, n_entries, k, n_heads, dim, dt):
    return int(load().csa_index_topk_workspace_size(batch, n_q, n_entries, k, n_heads, dim, dt))


def index_topk_plan(batch, n_q, n_entries, k, n_heads, dim, dt):
    """How csa_index_topk splits a call of this shape on the current device:
    dict(slice_len, n_slices, coop, tensor_core, ring_stages, tiles_per_stage)."""
    out = (ctypes.c_int32 * 6)()
    _check(load().csa_index_topk_plan(batch, n_q, n_entries, k, n_heads, dim, dt, ctypes.cast(out, ctypes.c_void_p)))
    keys = ("slice_len", "n_slices", "coop", "tensor_core", "ring_stages", "tiles_per_stage")
    return dict(zip(keys, [int(v) for v in out]))


def index_topk(qI, wI, KI, q_pos, m, k, *, dt=None, qI_sf=None, KI_sf=None, n_heads=None,
               scores=False, idx_out=None, ws=None, key_pages=None, n_entries=None):
    """Lightning indexer + top-k.  qI [B, T, H, d] (or NVFP4 codes [B, T, H, d/2]),
    wI [B, T, H] fp32, KI [B, E, d] (codes [B, E, d/2]), q_pos [B, T] int64.
    Paged keys: key_pages a Pages (pages()), KI / KI_sf the pool, n_entries = E.

    Returns idx [B, T, k] int32 (and the score tensor when scores=True)."""
    _need_cuda(qI, wI, KI, q_pos, qI_sf, KI_sf)
    if dt is None:
        dt = IDX_NVFP4 if qI.dtype == torch.uint8 else _dt_of(qI)
    B, T, H = wI.shape
    if key_pages is not None and n_entries is None:
        raise ValueError("paged keys need n_entries (logical keys per request)")
    E = KI.shape[1] if n_entries is None else n_entries
    dim = qI.shape[-1] * (2 if dt == IDX_NVFP4 else 1)
    dev = qI.device
    if idx_out is None:
        idx_out = torch.empty(B, T, k, device=dev, dtype=torch.int32)
    sc = None
    if scores:
        sc = torch.empty(B, T, E, device=dev, dtype=torch.float32 if dt == F32 else torch.bfloat16)
    need = index_topk_workspace_size(B, T, E, k, H, dim, dt)
    if ws is None or ws.numel() < need:
        ws = torch.zeros(need, device=dev, dtype=torch.uint8)  # zero before first use
    _check(load().csa_index_topk_paged(_ptr(qI), _ptr(qI_sf), _ptr(wI), _ptr(KI), _ptr(KI_sf),
                                       ctypes.byref(key_pages) if key_pages is not None else None, _ptr(q_pos),
                                       B, T, E, m, H, dim, k, dt, _ptr(idx_out), _ptr(sc), _ptr(ws),
                                       ws.numel(), _stream()))
    return (idx_out, sc) if scores else idx_out


class CompressJob(ctypes.Structure):
    """csa_compress_job_t: one compressor call's arguments (see compress())."""
    _fields_ = [("Ca", ctypes.c_void_p), ("Cb", ctypes.c_void_p), ("Za", ctypes.c_void_p), ("Zb", ctypes.c_void_p),
                ("Ba", ctypes.c_void_p), ("Bb", ctypes.c_void_p), ("n_tok", ctypes.c_int64),
                ("tok0", ctypes.c_int64), ("in_batch_stride", ctypes.c_int64), ("e0", ctypes.c_int64),
                ("n_out", ctypes.c_int64), ("dim", ctypes.c_int32), ("m", ctypes.c_int32), ("in_dt", ctypes.c_int32),
                ("out", ctypes.c_void_p), ("out_sf", ctypes.c_void_p), ("out_batch_stride", ctypes.c_int64),
                ("out_row0", ctypes.c_int64), ("out_dt", ctypes.c_int32), ("out_pages", ctypes.POINTER(Pages)),
                ("norm_g", ctypes.c_void_p), ("norm_eps", ctypes.c_float), ("rope_dims", ctypes.c_int32),
                ("rope_base", ctypes.c_double), ("pos_stride", ctypes.c_int64), ("pos_offset", ctypes.c_int64)]


def compress_job(Ca, Za, Ba, m, Cb=None, Zb=None, Bb=None, *, tok0, e0, n_out, out, out_dt, out_sf=None,
                 out_row0=None, n_tok=None, out_pages=None, norm_g=None, norm_eps=1e-6, rope_dims=0,
                 rope_base=10000.0, pos_stride=None, pos_offset=None):
    """A compressor call's arguments as a CompressJob (entries e0.. written to
    rows out_row0.. of `out`, out_row0 defaulting to e0; with out_pages (a
    Pages) `out` / `out_sf` are the pool and rows are logical rows).  norm_g /
    rope_dims: RMSNorm and RoPE of each entry before it is stored, entry i at
    position pos_stride * i + pos_offset (default m * i + m - 1)."""
    _need_cuda(Ca, Za, Ba, Cb, Zb, Bb, out, out_sf, norm_g)
    batch, rows, dim = Ca.shape
    job = CompressJob(
        Ca=Ca.data_ptr(), Cb=Cb.data_ptr() if Cb is not None else None, Za=Za.data_ptr(),
        Zb=Zb.data_ptr() if Zb is not None else None, Ba=Ba.data_ptr(), Bb=Bb.data_ptr() if Bb is not None else None,
        n_tok=rows if n_tok is None else n_tok, tok0=tok0, in_batch_stride=rows, e0=e0, n_out=n_out, dim=dim, m=m,
        in_dt=_dt_of(Ca), out=out.data_ptr(), out_sf=out_sf.data_ptr() if out_sf is not None else None,
        out_batch_stride=out.shape[1], out_row0=e0 if out_row0 is None else out_row0, out_dt=out_dt,
        out_pages=ctypes.pointer(out_pages) if out_pages is not None else None,
        norm_g=norm_g.data_ptr() if norm_g is not None else None, norm_eps=norm_eps, rope_dims=rope_dims,
        rope_base=rope_base, pos_stride=m if pos_stride is None else pos_stride,
        pos_offset=m - 1 if pos_offset is None else pos_offset)
    job._keep = (out_pages, norm_g)  # the struct holds raw pointers: keep what they point to alive with it
    return job


def compress_ex(job, batch):
    """Runs one CompressJob (compress_job()) on `batch` requests."""
    _check(load().csa_compress_ex(ctypes.byref(job), batch, _stream()))


def compress_index_topk(keys_job, qI, wI, KI, q_pos, m, k, *, extra_job=None, dt=None, qI_sf=None, KI_sf=None,
                        idx_out=None, ws=None, scores=False, n_entries=None):
    """Run the compressor job `keys_job` (index keys into KI / KI_sf) and, if
    given, `extra_job` (e.g. the KV cache), then index + top-k over KI: one
    launch when the tensor-core indexer takes the shape.  Returns idx
    [B, T, k] int32 (and the score tensor when scores=True)."""
    _need_cuda(qI, wI, KI, q_pos, qI_sf, KI_sf)
    if dt is None:
        dt = IDX_NVFP4 if qI.dtype == torch.uint8 else _dt_of(qI)
    B, T, H = wI.shape
    if keys_job.out_pages and n_entries is None:
        raise ValueError("a paged key cache needs n_entries (logical keys per request)")
    E = KI.shape[1] if n_entries is None else n_entries
    dim = qI.shape[-1] * (2 if dt == IDX_NVFP4 else 1)
    dev = qI.device
    if idx_out is None:
        idx_out = torch.empty(B, T, k, device=dev, dtype=torch.int32)
    sc = None
    if scores:
        sc = torch.empty(B, T, E, device=dev, dtype=torch.float32 if dt == F32 else torch.bfloat16)
    need = index_topk_workspace_size(B, T, E, k, H, dim, dt)
    if ws is None or ws.numel() < need:
        ws = torch.zeros(need, device=dev, dtype=torch.uint8)  # zero before first use
    _check(load().csa_compress_index_topk(ctypes.byref(keys_job),
                                          ctypes.byref(extra_job) if extra_job is not None else None,
                                          _ptr(qI), _ptr(qI_sf), _ptr(wI), _ptr(KI), _ptr(KI_sf), _ptr(q_pos), B, T,
                                          E, m, H, dim, k, dt, _ptr(idx_out), _ptr(sc), _ptr(ws), ws.numel(),
                                          _stream()))
    return (idx_out, sc) if scores else idx_out


# -------------------------------------------------------------------- attention

class MqaOptions(ctypes.Structure):
    """csa_mqa_options_t: fixed split count (batch-invariant decode), query
    RMSNorm weights and eps, RoPE dims of the query (at q_pos) and of the
    output (at -q_pos), RoPE base, block table of a paged entry cache."""
    _fields_ = [("splits", ctypes.c_int32), ("q_norm_g", ctypes.c_void_p), ("q_norm_eps", ctypes.c_float),
                ("q_rope_dims", ctypes.c_int32), ("out_rope_dims", ctypes.c_int32), ("rope_base", ctypes.c_double),
                ("entry_pages", ctypes.POINTER(Pages)), ("compress", ctypes.POINTER(CompressJob))]


def mqa_options(*, splits=0, q_norm_g=None, q_norm_eps=1e-6, q_rope_dims=0, out_rope_dims=0, rope_base=10000.0,
                entry_pages=None, compress=None):
    """Options of the attention calls; entry_pages: a Pages (pages()) when
    `entries` is the pool of a paged cache; compress: a CompressJob
    (compress_job()) launched before the entries are attended."""
    _need_cuda(q_norm_g)
    o = MqaOptions(splits=splits, q_norm_g=q_norm_g.data_ptr() if q_norm_g is not None else None,
                   q_norm_eps=q_norm_eps, q_rope_dims=q_rope_dims, out_rope_dims=out_rope_dims,
                   rope_base=rope_base, entry_pages=ctypes.pointer(entry_pages) if entry_pages is not None else None,
                   compress=ctypes.pointer(compress) if compress is not None else None)
    o._keep = (q_norm_g, entry_pages, compress)  # raw pointers: keep what they point to alive with the struct
    return o


def _n_entries(entries, n_entries, options):
    if options is not None and options.entry_pages:
        if n_entries is None:
            raise ValueError("a paged call needs n_entries (logical entries per request)")
        return n_entries
    return entries.shape[1] if n_entries is None else n_entries


def _opt_ref(options):
    return ctypes.byref(options) if options is not None else None


def mqa_workspace_size(batch, n_q, n_heads, dim, rows_per_query, q_dt, kv_dt, options=None):
    return int(load().csa_mqa_workspace_size(batch, n_q, n_heads, dim, rows_per_query, q_dt, kv_dt,
                                             _opt_ref(options)))


def _kv_dt(entries, kv_dt):
    if kv_dt is not None:
        return kv_dt
    return KV_FP8MIX if entries.dtype == torch.uint8 else _dt_of(entries)


def sparse_mqa_workspace_size(batch, n_q, n_heads, dim, k, window, q_dt, kv_dt):
    return int(load().csa_sparse_mqa_workspace_size(batch, n_q, n_heads, dim, k, window, q_dt, kv_dt))


def hca_dense_mqa_workspace_size(batch, n_q, n_heads, dim, n_entries, window, q_dt, kv_dt):
    return int(load().hca_dense_mqa_workspace_size(batch, n_q, n_heads, dim, n_entries, window, q_dt,
                                                   kv_dt))


def sparse_mqa(Q, entries, idx, win, win_start, q_pos, window, m, sink, scale, *, kv_dt=None, O=None,
               ws=None, options=None, n_entries=None):
    """CSA shared-KV MQA.  Q [B, T, H, c]; entries [B, E, row] (paged: the
    pool, with n_entries = E); idx [B, T, k] int32; win [B, Lw, row];
    win_start [B] int64; q_pos [B, T] int64; sink [H] fp32.
    options: an MqaOptions (mqa_options()) or None."""
    _need_cuda(Q, entries, idx, win, win_start, q_pos, sink)
    B, T, H, c = Q.shape
    kv_dt = _kv_dt(entries, kv_dt)
    q_dt = _dt_of(Q)
    k = idx.shape[-1]
    if O is None:
        O = torch.empty_like(Q)
    need = mqa_workspace_size(B, T, H, c, k + window, q_dt, kv_dt, options)
    if ws is None or ws.numel() < need:
        ws = torch.empty(need, device=Q.device, dtype=torch.uint8)
    _check(load().csa_sparse_mqa_ex(_ptr(Q), q_dt, _ptr(entries), _n_entries(entries, n_entries, options), _ptr(idx),
                                    k, _ptr(win),
                                    win.shape[1], _ptr(win_start), _ptr(q_pos), window, m, _ptr(sink),
                                    float(scale), B, T, H, c, kv_dt, _ptr(O), _ptr(ws), ws.numel(),
                                    _opt_ref(options), _stream()))
    return O


def hca_dense_mqa(Q, entries, win, win_start, q_pos, window, m, sink, scale, *, kv_dt=None, O=None,
                  ws=None, options=None, n_entries=None):
    """HCA dense shared-KV MQA over every visible entry plus the window
    (paged: entries is the pool, n_entries the logical entries)."""
    _need_cuda(Q, entries, win, win_start, q_pos, sink)
    B, T, H, c = Q.shape
    kv_dt = _kv_dt(entries, kv_dt)
    q_dt = _dt_of(Q)
    if O is None:
        O = torch.empty_like(Q)
    E = _n_entries(entries, n_entries, options)
    need = mqa_workspace_size(B, T, H, c, E + window, q_dt, kv_dt, options)
    if ws is None or ws.numel() < need:
        ws = torch.zeros(need, device=Q.device, dtype=torch.uint8)
    _check(load().hca_dense_mqa_ex(_ptr(Q), q_dt, _ptr(entries), E, _ptr(win), win.shape[1],
                                   _ptr(win_start), _ptr(q_pos), window, m, _ptr(sink), float(scale), B, T,
                                   H, c, kv_dt, _ptr(O), _ptr(ws), ws.numel(), _opt_ref(options), _stream()))
    return O


def tree_mqa_workspace_size(batch, n_q, n_heads, dim, rows_per_query, q_dt, kv_dt, options=None):
    return int(load().csa_tree_mqa_workspace_size(batch, n_q, n_heads, dim, rows_per_query, q_dt, kv_dt,
                                                  _opt_ref(options)))


def tree_mqa(Q, entries, win, win_start, draft, tree_mask, ctx_len, q_pos, window, m, sink, scale, *, idx=None,
             n_nodes=None, kv_dt=None, O=None, ws=None, options=None, n_entries=None):
    """Attention of a tree of drafted tokens.  Q [B, T, H, c]: T nodes per
    request; draft [B, D, row] their KV rows (and speculative entries);
    tree_mask [B, T, ceil(D / 32)] int32: bit j of a node's words says that it
    attends drafted row j; ctx_len [B] int64 committed tokens; q_pos [B, T]
    int64; n_nodes [B] int32 or None; idx [B, T, k] int32 selected entries or
    None for all; the rest as in sparse_mqa().  draft and tree_mask may be
    None when nothing is drafted."""
    dev = _device_of(Q)
    _need(dev, Q.dtype, "Q", (Q,))
    _need(dev, entries.dtype, "win and draft", (entries, win, draft))
    _need(dev, _I64, "win_start, ctx_len and q_pos", (win_start, ctx_len, q_pos))
    _need(dev, _I32, "tree_mask, idx and n_nodes", (tree_mask, idx, n_nodes))
    _need(dev, _F32, "sink", (sink,))
    B, T, H, c = Q.shape
    kv_dt = _kv_dt(entries, kv_dt)
    q_dt = _dt_of(Q)
    k = idx.shape[-1] if idx is not None else 0
    D = draft.shape[1] if draft is not None else 0
    E = _n_entries(entries, n_entries, options)
    if Q.dtype is not _F32 and Q.dtype is not _BF16:
        raise ValueError("Q must be float32 or bfloat16")
    if O is None:
        O = torch.empty_like(Q)
    elif O.shape != Q.shape:
        raise ValueError("O must be like Q")
    else:
        _need(dev, Q.dtype, "O", (O,))
    row = c if kv_dt != KV_FP8MIX else row_bytes(kv_dt, c)
    norm_g, table, _ = getattr(options, "_keep", (None, None, None))  # as mqa_options() was given them
    pg = options.entry_pages.contents if options is not None and options.entry_pages else None
    if (win.shape != (B, win.shape[1], row) or win_start.numel() != B or entries.shape[-1] != row or
            (pg is None and entries.shape != (B, E, row))):
        raise ValueError("entries must be [B, E, row] (or a pool of rows), win [B, n, row] and win_start [B]")
    if pg is not None and (entries.numel() < pg.n_pages * pg.page_entries * row or
                           (table is not None and table._keep.shape[0] < B)):
        raise ValueError("entries must be a pool of n_pages * page_entries rows and its table have a row per request")
    if norm_g is not None and (norm_g.dtype is not _F32 or norm_g.numel() != c):
        raise ValueError("q_norm_g must be float32 [c]")
    if D and (tree_mask is None or tree_mask.shape != (B, T, (D + 31) // 32) or draft.shape != (B, D, row)):
        raise ValueError("draft must be [B, D, row] and tree_mask [B, T, ceil(D / 32)]")
    if (ctx_len.numel() != B or q_pos.shape != (B, T) or sink.numel() != H or
            (idx is not None and idx.shape != (B, T, k)) or (n_nodes is not None and n_nodes.numel() != B)):
        raise ValueError("ctx_len and n_nodes must be [B], q_pos [B, T], idx [B, T, k], sink [H]")
    if ws is None:
        need = tree_mqa_workspace_size(B, T, H, c, (k if idx is not None else E) + window + D, q_dt, kv_dt, options)
        ws = torch.empty(need, device=Q.device, dtype=_U8)
    else:
        _need(dev, _U8, "ws", (ws,))
    _check((_lib or load()).csa_tree_mqa(
        Q.data_ptr(), q_dt, entries.data_ptr(), E, idx.data_ptr() if idx is not None else None, k, win.data_ptr(),
        win.shape[1], win_start.data_ptr(), draft.data_ptr() if D else None, D, tree_mask.data_ptr() if D else None,
        ctx_len.data_ptr(), q_pos.data_ptr(), n_nodes.data_ptr() if n_nodes is not None else None, window, m,
        sink.data_ptr(), scale, B, T, H, c, kv_dt, O.data_ptr(), ws.data_ptr(), ws.numel(), _opt_ref(options),
        _current_stream(dev)))
    return O


# ------------------------------------------------------ grouped output projection

def grouped_out_proj_workspace_size(T, n_h, c, g, d_g, d):
    return int(load().csa_grouped_out_proj_workspace_size(T, n_h, c, g, d_g, d))


def grouped_out_proj_plan(T, n_h, c, g, d_g, d):
    """How csa_grouped_out_proj divides a call of this shape: per projection
    (group, then output) the tokens per CTA, K slices per tile and CTAs."""
    out = (ctypes.c_int32 * 6)()
    _check(load().csa_grouped_out_proj_plan(T, n_h, c, g, d_g, d, ctypes.cast(out, ctypes.c_void_p)))
    v = [int(x) for x in out]
    keys = ("tokens_per_cta", "splits", "ctas")
    return {"group": dict(zip(keys, v[:3])), "output": dict(zip(keys, v[3:]))}


def grouped_out_proj(O, Wg, Wo, *, out=None, ws=None):
    """Grouped output projection.  O [T, n_h, c] bf16, Wg [g, n_h/g * c, d_g]
    bf16, Wo [g * d_g, d] bf16 -> Y [T, d] bf16.  ws: a workspace of
    grouped_out_proj_workspace_size bytes whose counters are zero (a fresh
    zeroed one is made when not given; every call leaves it zero)."""
    _need_cuda(O, Wg, Wo, out, ws)
    T, n_h, c = O.shape
    g, _, d_g = Wg.shape
    d = Wo.shape[1]
    if Wg.shape[1] * g != n_h * c or Wo.shape[0] != g * d_g:
        raise ValueError("Wg must be [g, n_h/g * c, d_g] and Wo [g * d_g, d]")
    if out is None:
        out = torch.empty(T, d, device=O.device, dtype=torch.bfloat16)
    need = grouped_out_proj_workspace_size(T, n_h, c, g, d_g, d)
    if ws is None:
        ws = torch.zeros(need, device=O.device, dtype=torch.uint8)
    _check(load().csa_grouped_out_proj(_ptr(O), _ptr(Wg), _ptr(Wo), _ptr(out), T, n_h, c, g, d_g, d, _ptr(ws),
                                       ws.numel() * ws.element_size(), _stream()))
    return out
