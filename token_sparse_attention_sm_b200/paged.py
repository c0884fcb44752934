"""Paged caches: block tables and slot maps of a ragged batch, the append of
new rows by slot, and the attention of new tokens over their paged caches
(CLSA article, section CLSAの仕組み: the self-decoder whose cache the decode
step routes over is such an attention).

A cache is K, V [num_pages, Hkv, page_size, d]; sequence b's token j is row
j % page_size of page block_table[b, j // page_size].  A dense cache
[B,Hkv,n_cap,d] is the paged cache of B pages with block_table[b, 0] = b, so
these calls also fill and read the caches of ``decode_step``.

A serving step is ``paged_plan`` once, then per layer ``paged_append`` and
``paged_attn`` with what it returned::

    p = sd.paged_plan(new_lens, lens, table, free_pages, free_count, 64, T, num_pages)
    sd.paged_append(K, V, k_new, v_new, p["slots"])
    out, lse = sd.paged_attn(q, K, V, table, p["q_start"], p["kv_lens"], max_new=n)
    lens, free_count = p["kv_lens"], p["free_left"]

Without ``ws`` a call uses a workspace kept for its device and stream, which
host threads may share: the kernels of one call are enqueued together.  Inside
a stream capture it takes one from the graph's own memory instead, so two
captured graphs share scratch only if they share a memory pool, and then they
must not overlap.  Calls given one Workspace are ordered by the caller, and a
capture needs it to be large enough already.  ``check`` reads the device status
(and synchronises); a capture needs check=False.  What calls with check=False
and the replays of a graph report is read later, with ``paged_status`` where
they had no ``ws``, else with ``read_device_status(ws)``.
"""
from __future__ import annotations

import ctypes
import functools
import importlib.util
import threading

import torch

from . import (DTYPE_CODES, SparseDecodeError, Workspace, _check, _need_result, lib_path, load,
               read_device_status)

_HEADER = 4096  # workspace bytes of the calls that only report a status
_TIMEOUT = 7  # SPARSE_ERR_TIMEOUT
_stream_ws: dict = {}
_I32, _F32 = torch.int32, torch.float32


class _PagedShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("B", "T", "Hq", "Hkv", "d", "dtype", "page_size", "num_pages", "max_blocks",
                 "max_new")]


@functools.lru_cache(maxsize=None)
def _entry(name: str):
    """A C entry point of the loaded library, called with Python's global lock
    held: an attention is up to three kernels over one schedule and its
    partials, and threads that share a stream must not mix those of two calls
    (the compiled calls hold the lock too)."""
    load()
    fn = getattr(_gil_library(), name)
    like = getattr(load(), name)
    fn.restype, fn.argtypes = like.restype, like.argtypes
    return fn


@functools.lru_cache(maxsize=None)
def _gil_library():
    return ctypes.PyDLL(lib_path())


@functools.lru_cache(maxsize=512)
def _shape(B, T, Hq, Hkv, d, dtype, page_size, num_pages, max_blocks, max_new=0):
    """The C shape of these sizes, by reference (read only by the library)."""
    if dtype not in DTYPE_CODES:
        raise TypeError(f"unsupported dtype {dtype}")
    sizes = (B, T, Hq, Hkv, d, DTYPE_CODES[dtype], page_size, num_pages, max_blocks, max_new)
    # ctypes would cut them to 32 bits without a word
    if not all(-1 << 31 <= x < 1 << 31 for x in sizes):
        raise ValueError("sizes must fit 32 bits")
    return ctypes.byref(_PagedShape(*sizes))


@functools.lru_cache(maxsize=512)
def _attn_plan(*sizes):
    """The C shape of an attention call and the workspace bytes it needs."""
    n = ctypes.c_size_t(0)
    sh = _shape(*sizes)
    _check(load().sparse_paged_workspace_size(sh, ctypes.byref(n)), "paged_attn")
    return sh, int(n.value)


@functools.lru_cache(maxsize=None)
def _calls():
    """The compiled form of the calls (csrc/binding/paged_calls.cpp), given the
    library's entry points."""
    from .build import CALLS, calls_current
    if not calls_current():
        raise RuntimeError(f"not built: {CALLS} is missing or was built for another torch or "
                           "Python (run `python -m token_sparse_attention_sm_b200.build`)")
    spec = importlib.util.spec_from_file_location("_paged_calls", CALLS)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    lib = load()
    m.bind(*(ctypes.cast(getattr(lib, f"sparse_paged_{n}"), ctypes.c_void_p).value
             for n in ("workspace_size", "plan", "append", "attn")))
    return m


def _plain(t):
    """(compiled calls, workspace, stream) when a call on t's device may take
    the compiled form: that device is current, nothing is being captured and
    the stream has a workspace; else None."""
    dev = t.get_device()
    if dev < 0 or dev != torch.cuda.current_device() or torch._C._cuda_isCurrentStreamCapturing():
        return None
    stream = torch._C._cuda_getCurrentRawStream(dev)
    ws = _stream_ws.get((dev, stream))
    return None if ws is None else (_calls(), ws, stream)


def _one_device(t, *ts) -> int:
    """The index of the device that all given tensors are on."""
    dev = t.get_device()
    for x in ts:
        if x is not None and x.get_device() != dev:
            break
    else:
        if dev >= 0:
            return dev
    if any(x is not None and not x.is_cuda for x in (t, *ts)):
        raise ValueError("all tensors must be CUDA tensors")
    raise ValueError("all tensors must be on one device")


def _kept(dev: int, stream: int) -> Workspace:
    """The workspace kept for a device's stream.  Its lock goes from its growth
    to the call that uses it, for threads that share the stream; the compiled
    calls, which read ``buf`` and launch without a break, need none."""
    ws = _stream_ws.get((dev, stream))
    if ws is None:
        ws = Workspace(f"cuda:{dev}")
        ws.lock, ws.key = threading.RLock(), (dev, stream)
        ws.get(_HEADER)  # whoever finds it finds a buffer
        ws = _stream_ws.setdefault((dev, stream), ws)
    return ws


def _launch(what: str, args, ws: Workspace | None, dev: int, nbytes: int, check: bool):
    """One C call sparse_<what>(*args, workspace of nbytes, stream) on the
    current device and stream, then its status."""
    call = _entry(f"sparse_{what}")
    stream = torch._C._cuda_getCurrentRawStream(dev)
    capturing = torch._C._cuda_isCurrentStreamCapturing()
    if ws is None and not capturing:
        ws = _kept(dev, stream)
        with ws.lock:
            buf = ws.get(nbytes)
            rc = call(*args, buf.data_ptr(), buf.numel(), stream)
        return _finish(rc, what, ws, check)
    if capturing and check:
        raise ValueError("check=True synchronises: give check=False inside a stream capture")
    if ws is None:
        status = _static_status(dev)
        if nbytes <= _HEADER:
            return _finish(call(*args, status, _HEADER, stream), what, None, check)
        # only the header has to start at zero: the graph clears it
        buf = torch.empty(nbytes, dtype=torch.uint8, device=f"cuda:{dev}")
        buf[:_HEADER].zero_()
        return _finish(_entry(f"sparse_{what}_status")(*args, buf.data_ptr(), nbytes, status,
                                                       stream), what, None, check)
    if ws.device.index not in (None, dev):
        raise ValueError(f"workspace on {ws.device}, tensors on cuda:{dev}")
    if capturing:
        if ws.buf is None or ws.buf.numel() < nbytes:
            raise ValueError("a workspace cannot grow inside a stream capture: "
                             f"get({nbytes}) before it")
        # the graph keeps this address, also when ws grows later
        ws.kept = getattr(ws, "kept", []) + [ws.buf]
    buf = ws.get(nbytes)
    return _finish(call(*args, buf.data_ptr(), buf.numel(), stream), what, ws, check)


def _finish(rc: int, what: str, ws, check: bool):
    if rc:
        _check(rc, what)
    if check:
        try:
            read_device_status(ws)
        except SparseDecodeError as e:
            _drop_after(e.status, ws)
            raise


def _drop_after(status: int, ws: Workspace | None):
    """A wait that ran out leaves counters that are not zero: the next call
    without ``ws`` gets a new workspace."""
    key = getattr(ws, "key", None)  # None: not a kept one
    if status == _TIMEOUT and key is not None and _stream_ws.get(key) is ws:
        del _stream_ws[key]


@functools.lru_cache(maxsize=None)
def _static_status(dev: int) -> int:
    """The address of the library's status area on the current device: a
    captured call without ``ws`` reports there, since its scratch is the graph's."""
    at = ctypes.c_void_p(0)
    _check(_entry("sparse_paged_static_status")(ctypes.byref(at)), "paged status")
    return at.value


def paged_status(raise_on_error: bool = True) -> int:
    """Synchronise the current stream and read (and reset) the device status of
    the paged calls made without ``ws``: those on this stream, and those captured
    on this device, whose replays should be over (what one in flight reports may
    be missed).  Raises SparseDecodeError unless it is SPARSE_OK; else returns it."""
    if torch._C._cuda_isCurrentStreamCapturing():
        raise ValueError("reading the status synchronises: not inside a stream capture")
    dev = torch.cuda.current_device()
    stream = torch._C._cuda_getCurrentRawStream(dev)
    ws = _stream_ws.get((dev, stream))
    rc, seen = 0, 0
    words = [(None, _static_status(dev))]
    if ws is not None:
        words.append((ws, ws.buf.data_ptr()))
    for w, at in words:
        flags = ctypes.c_uint32(0)
        one = load().sparse_read_device_status(at, stream, ctypes.byref(flags))
        _drop_after(one, w)
        rc, seen = one or rc, seen | flags.value
    if raise_on_error:
        _check(rc, f"device status (flags=0x{seen:x})")
    return rc


def paged_release() -> None:
    """Free the workspaces kept for the paged calls without ``ws`` (one per
    device and stream, up to 80 MB once it has served a large chunk).  Later
    calls make new ones; conditions that nobody has read are dropped."""
    _stream_ws.clear()


def _rows(t, name: str, heads: int, d: int) -> int:
    """The elements between the token rows of t [T,heads,d]; its heads and
    elements must be dense."""
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != d:
        raise ValueError(f"{name} must be [T,{heads},{d}], got {tuple(t.shape)}")
    st = t.stride()
    if st[2] != 1 or (heads > 1 and st[1] != d):
        raise ValueError(f"the rows of {name} must be contiguous")
    if t.shape[0] < 2:
        return heads * d
    if st[0] < heads * d or st[0] * t.element_size() % 16:
        raise ValueError(f"the rows of {name} must be distinct and a multiple of 16 bytes apart")
    return st[0]


def _need_int32(t, shape, name: str):
    if t.dtype is not _I32 or t.shape != shape or not t.is_contiguous():
        _need_result(t, shape, _I32, name)


def _cache_dims(K, V):
    if K.dim() != 4 or V.shape != K.shape or V.dtype != K.dtype:
        raise ValueError("K and V must be [num_pages,Hkv,page_size,d] of one shape and dtype")
    if not (K.is_contiguous() and V.is_contiguous()):
        raise ValueError("K and V must be contiguous")
    return K.shape


def paged_workspace_bytes(B, T, Hq, Hkv, d, dtype, page_size, num_pages, max_blocks,
                          max_new: int | None = None) -> int:
    """Bytes that paged_attn needs of a workspace for these sizes."""
    return _attn_plan(B, T, Hq, Hkv, d, dtype, page_size, num_pages, max_blocks, max_new or 0)[1]


def paged_plan(new_lens, lens, block_table, free_pages, free_count, page_size: int,
               num_tokens: int, num_pages: int, ws: Workspace | None = None, check: bool = True,
               kv_lens=None, q_start=None, positions=None, slots=None, free_left=None):
    """The block tables and slot map of one batch step, on the device from the
    requests' lengths (sparse_paged_plan).

    new_lens, lens [B] int32: new and already cached tokens of every sequence;
    block_table [B,max_blocks] int32, updated in place; free_pages [F] int32
    and free_count [1] int32: the free list, pages taken from its end;
    num_tokens: rows of the packed tensors (at least the new tokens).  Returns
    dict(kv_lens [B], q_start [B+1], positions [T], slots [T], free_left [1]),
    all int32; kv_lens may be lens and free_left free_count to update them in
    place.  A batch that does not fit raises (SPARSE_ERR_CAPACITY) and takes
    nothing."""
    if ws is None and q_start is None and positions is None and slots is None:
        plain = _plain(new_lens)
        if plain is not None:
            calls, w, stream = plain
            r = calls.plan(w, stream, new_lens, lens, block_table, free_pages, free_count,
                           int(page_size), int(num_tokens), int(num_pages), kv_lens, free_left)
            if type(r) is tuple:
                _finish(0, "paged_plan", w, check)
                return {"kv_lens": r[0], "q_start": r[1], "positions": r[2], "slots": r[3],
                        "free_left": r[4]}
            if r is not None:
                _check(r, "paged_plan")
    dev = _one_device(new_lens, lens, block_table, free_pages, free_count, kv_lens, q_start,
                      positions, slots, free_left)
    if new_lens.dim() != 1 or block_table.dim() != 2 or free_pages.dim() != 1:
        raise ValueError("new_lens must be [B], block_table [B,max_blocks], free_pages [F]")
    B, T, F = new_lens.shape[0], int(num_tokens), free_pages.shape[0]
    blocks = block_table.shape[1]
    if T < 0:
        raise ValueError("num_tokens must not be negative")
    _need_int32(new_lens, (B,), "new_lens")
    _need_int32(lens, (B,), "lens")
    _need_int32(block_table, (B, blocks), "block_table")
    _need_int32(free_pages, (F,), "free_pages")
    _need_int32(free_count, (1,), "free_count")
    sizes = (T, T, B, B + 1, 1)
    res = [positions, slots, kv_lens, q_start, free_left]
    for t, n, name in zip(res, sizes, ("positions", "slots", "kv_lens", "q_start", "free_left")):
        if t is not None:
            _need_int32(t, (n,), name)
    sh = _shape(B, T, 1, 1, 64, _F32, int(page_size), int(num_pages), blocks)
    # before the results are allocated
    _check(_entry("sparse_paged_workspace_size")(sh, ctypes.byref(ctypes.c_size_t(0))),
           "paged_plan")
    if torch.cuda.current_device() != dev:
        with torch.cuda.device(dev):
            return paged_plan(new_lens, lens, block_table, free_pages, free_count, page_size,
                              num_tokens, num_pages, ws, check, kv_lens, q_start, positions, slots,
                              free_left)
    # one allocation for the results that were not given
    want = [n for t, n in zip(res, sizes) if t is None]
    if want:
        new = iter(torch.empty(sum(want), dtype=_I32, device=new_lens.device).split(want))
        res = [next(new) if t is None else t for t in res]
    positions, slots, kv_lens, q_start, free_left = res
    _launch("paged_plan", (
        sh, new_lens.data_ptr(), lens.data_ptr(), block_table.data_ptr(), free_pages.data_ptr(), F,
        free_count.data_ptr(), kv_lens.data_ptr(), q_start.data_ptr(), positions.data_ptr(),
        slots.data_ptr(), free_left.data_ptr()), ws, dev, _HEADER, check)
    return {"kv_lens": kv_lens, "q_start": q_start, "positions": positions, "slots": slots,
            "free_left": free_left}


def paged_append(K, V, k_new, v_new, slots, ws: Workspace | None = None, check: bool = True):
    """Write the new tokens' rows k_new, v_new [T,Hkv,d] (column ranges of
    wider rows are fine) to their slots [T] int32 of the paged caches K, V
    [num_pages,Hkv,page_size,d]; rows with slot -1 are skipped, the other slots
    are distinct, and no row is both read and written."""
    if ws is None:
        plain = _plain(K)
        if plain is not None:
            calls, w, stream = plain
            r = calls.append(w, stream, K, V, k_new, v_new, slots)
            if r is not None:
                return _finish(r, "paged_append", w, check)
    dev = _one_device(K, V, k_new, v_new, slots)
    pages, Hkv, page, d = _cache_dims(K, V)
    if not (k_new.dtype == v_new.dtype == K.dtype):
        raise ValueError("K, V, k_new and v_new must share a dtype")
    ks, vs = _rows(k_new, "k_new", Hkv, d), _rows(v_new, "v_new", Hkv, d)
    T = k_new.shape[0]
    if v_new.shape[0] != T:
        raise ValueError("k_new and v_new must have the same rows")
    _need_int32(slots, (T,), "slots")
    sh = _shape(1, T, Hkv, Hkv, d, K.dtype, page, pages, 1)
    if T == 0:
        return
    if torch.cuda.current_device() != dev:
        with torch.cuda.device(dev):
            return paged_append(K, V, k_new, v_new, slots, ws, check)
    _launch("paged_append", (
        sh, K.data_ptr(), V.data_ptr(), k_new.data_ptr(), ks, v_new.data_ptr(), vs,
        slots.data_ptr()), ws, dev, _HEADER, check)


def paged_attn(q, K, V, block_table, q_start, kv_lens, window: int = 0, sinks: int = 0,
               max_new: int | None = None, ws: Workspace | None = None, check: bool = True,
               return_lse: bool = True, out=None, lse=None):
    """Attention of new tokens over their sequences' paged caches, themselves
    included (sparse_paged_attn).

    q [T,Hq,d]: the packed new tokens, sequence b's in rows q_start[b] to
    q_start[b+1] - 1 (q_start [B+1], kv_lens [B] int32: what paged_plan
    returned); row i stands at position p = kv_lens[b] - new tokens + i and
    sees tokens j <= p, under ``window`` >= 1 only those with j > p - window
    or j < ``sinks``.  max_new: the most new tokens one sequence has (1 for a
    decode step).  Up to 16 rows per KV head, max_new * Hq / Hkv, take the kernels
    for few rows, which are faster there and keep 16 bits of a bf16 call's
    weights (8 in the others); left out, it stands for T.  Returns
    (out [T,Hq,d], lse [T,Hq] or None); rows behind the last sequence are not
    written.  ``out`` and ``lse`` overlap no other tensor of the call."""
    if ws is None:
        plain = _plain(q)
        if plain is not None and (max_new is None or max_new >= 1):
            calls, w, stream = plain
            r = calls.attn(w, stream, q, K, V, block_table, q_start, kv_lens, int(window),
                           int(sinks), int(max_new or 0), return_lse, out, lse)
            if type(r) is tuple:
                _finish(0, "paged_attn", w, check)
                return r
            if r is not None:
                _check(r, "paged_attn")
    dev = _one_device(q, K, V, block_table, q_start, kv_lens, out, lse)
    pages, Hkv, page, d = _cache_dims(K, V)
    if q.dim() != 3 or q.dtype != K.dtype:
        raise ValueError("q must be [T,Hq,d] of the cache's dtype")
    T, Hq = q.shape[0], q.shape[1]
    qs = _rows(q, "q", Hq, d)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B,max_blocks]")
    B, blocks = block_table.shape
    _need_int32(block_table, (B, blocks), "block_table")
    _need_int32(q_start, (B + 1,), "q_start")
    _need_int32(kv_lens, (B,), "kv_lens")
    if out is not None:
        _need_result(out, (T, Hq, d), q.dtype, "out")
    if lse is not None:
        _need_result(lse, (T, Hq), _F32, "lse")
    window, sinks = int(window), int(sinks)
    if not (0 <= window < 1 << 31 and 0 <= sinks < 1 << 31):
        raise ValueError("window and sinks must not be negative")
    if max_new is not None and int(max_new) < 1:
        raise ValueError("max_new must be at least 1")
    sh, nbytes = _attn_plan(B, T, Hq, Hkv, d, K.dtype, page, pages, blocks, int(max_new or 0))
    if torch.cuda.current_device() != dev:
        with torch.cuda.device(dev):
            return paged_attn(q, K, V, block_table, q_start, kv_lens, window, sinks, max_new, ws,
                              check, return_lse, out, lse)
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    if lse is None and return_lse:
        lse = torch.empty((T, Hq), dtype=_F32, device=q.device)
    if T == 0:
        return out, lse
    _launch("paged_attn", (
        sh, q.data_ptr(), qs, K.data_ptr(), V.data_ptr(), block_table.data_ptr(),
        q_start.data_ptr(), kv_lens.data_ptr(), window, sinks, out.data_ptr(),
        None if lse is None else lse.data_ptr()), ws, dev, nbytes, check)
    return out, lse
