"""Python binding of libcmr_kv8 (include/cmr_kv8.h): a paged KV cache held in 8 bits.

The rotation that writes it (rotate_qk_kv8), the attention that reads it
(attend_kv8) and the upkeep of its pages (kv8_extend, kv8_fork, kv8_free,
kv8_compact).  As in the binding of libcmr, every step runs in the library's CUDA
kernels; this module checks tensor dtypes, devices and shapes, allocates outputs
and workspaces with torch when the caller does not pass them, and forwards raw
pointers and the current CUDA stream.  There is no fallback.

The cache is a pool of pages of P tokens, torch.float8_e4m3fn [L, pages, hk, P, D]
for K and V, with a float32 power of two [L, pages, hk] to each page and head; a
row of page_table, int32 [rows, max_pages], lists one sequence's pages in order
(-1 behind the last), and page_refs, int32 [pages], counts the rows that hold a
page (0: free).
"""
import ctypes
import os
from typing import Optional, Sequence, Tuple

import torch

from .cmr import CMR_OK, _stream_ptr

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libcmr_kv8.so")

CMR_DEVICE_PAGES_FULL = 8
CMR_DEVICE_BAD_SCALE = 16
STATUS_TEXT = {1: "CMR_EINVAL: invalid argument", 2: "CMR_ECUDA: CUDA runtime error",
               3: "CMR_EUNSUPPORTED: shape outside this build's limits"}
PAGE_TOKENS = (16, 32, 64, 128)
HEAD_DIMS = (64, 128, 256)

_p, _i, _l, _d, _z = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_double,
                      ctypes.c_size_t)
_POOL = [_p, _p, _p, _p]
# name -> (restype, argtypes); mirrors include/cmr_kv8.h
SIGNATURES = {
    "cmr_kv8_rotate_qk": (ctypes.c_int, [_p, _p, _p, _p, _i, _p, _p, _p, _l, _i, _i, _i, _i, _d,
                                         ctypes.POINTER(_i), _i] + _POOL
                          + [_i, _i, _p, _i, _i, _p, _p, _p]),
    "cmr_kv8_attend": (ctypes.c_int, [_p, _p, _p, _i, _p, _l, _i, _i, _i, _i, _d] + _POOL
                       + [_i, _i, _p, _i, _i, _p, _p, _z, _p, _p]),
    "cmr_kv8_attend_workspace_bytes": (_z, [_i, _l, _i, _i, _i, _i]),
    "cmr_kv8_extend": (ctypes.c_int, [_p, _i, _i, _p, _i, _i, _p, _p, _i, _p, _z, _p, _p]),
    "cmr_kv8_fork": (ctypes.c_int, _POOL + [_i, _i, _i, _i, _i, _p, _i, _i, _p, _p, _p, _p, _i,
                                            _p, _z, _p, _p]),
    "cmr_kv8_free": (ctypes.c_int, [_p, _i, _i, _p, _i, _p, _i, _p, _z, _p, _p]),
    "cmr_kv8_compact": (ctypes.c_int, _POOL + [_i, _i, _i, _i, _i, _p, _i, _i, _p, _p, _z, _p,
                                               _p]),
    "cmr_kv8_pages_workspace_bytes": (_z, [_i, _i, _i]),
    "cmr_kv8_last_attend_kernel": (ctypes.c_char_p, []),
    "cmr_kv8_last_error_message": (ctypes.c_char_p, []),
}

_lib = None


class Kv8Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = lib().cmr_kv8_last_error_message().decode()
        super().__init__(f"{where}: {STATUS_TEXT.get(status, 'unknown cmr_status')} -- {msg}")


def lib() -> ctypes.CDLL:
    """The loaded libcmr_kv8.so with its signatures set; raises if it was not built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"{LIB_PATH} is missing: build it with `python -m vlm_decoder_positional_b200.build`"
                " (there is no CPU fallback)")
        l = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(l, name)
            f.restype = res
            f.argtypes = args
        _lib = l
    return _lib


def _check(status: int, where: str):
    if status != CMR_OK:
        raise Kv8Error(status, where)


def _want(t, name: str, dtype: torch.dtype, dev: Optional[torch.device], shape=None):
    """t's data pointer, after the checks (shape: a tuple, None for any size in a place)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dev is not None and t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and (t.dim() != len(shape) or any(
            w is not None and w != s for w, s in zip(shape, t.shape))):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    return t.data_ptr()


def _maybe(t, name, dtype, dev, shape=None):
    return None if t is None else _want(t, name, dtype, dev, shape)


def _pool(k_pages, v_pages, k_scales, v_scales, dev):
    """Pointers of the pool, and (L, pages, hk, P, D)."""
    kp = _want(k_pages, "k_pages", torch.float8_e4m3fn, dev, (None,) * 5)
    shape = tuple(k_pages.shape)
    return (kp, _want(v_pages, "v_pages", torch.float8_e4m3fn, dev, shape),
            _want(k_scales, "k_scales", torch.float32, dev, shape[:3]),
            _want(v_scales, "v_scales", torch.float32, dev, shape[:3])), shape


def _heads(t, name, dev, n=None, L=None, D=None):
    """(pointer, (L, N, H, D)) of bf16 [L, N, H, D] or [N, H, D]."""
    p = _want(t, name, torch.bfloat16, dev)
    s = tuple(t.shape)
    s = (1,) + s if len(s) == 3 else s
    if len(s) != 4:
        raise ValueError(f"{name} must be [L, N, H, D] or [N, H, D]")
    if (n is not None and s[1] != n) or (L is not None and s[0] != L) or \
            (D is not None and s[3] != D):
        raise ValueError(f"{name} shape {s} does not match L={L}, N={n}, D={D}")
    return p, s


def _batch(cu_seqlens, pos_offset, slot, n, seqs, dev):
    """(num_seqs, pointers of cu_seqlens, pos_offset and slot)."""
    if cu_seqlens is None:
        b = n
    else:
        b = cu_seqlens.numel() - 1
        if b < 0:
            raise ValueError("cu_seqlens needs num_seqs + 1 entries")
    if seqs is not None and seqs != b:
        raise ValueError(f"start and amount hold {seqs} sequences, the batch {b}")
    return b, _maybe(cu_seqlens, "cu_seqlens", torch.int32, dev, (b + 1,)), \
        _maybe(pos_offset, "pos_offset", torch.int32, dev, (b,)), \
        _maybe(slot, "slot", torch.int32, dev, (b,))


def _workspace(workspace, need, dev):
    """(tensor, pointer, bytes): the caller's, or a new one."""
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    elif not workspace.is_cuda or workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous CUDA tensor on {dev}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def rotate_qk_kv8(q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor,
                  start: torch.Tensor, amount: torch.Tensor, k_pages: torch.Tensor,
                  v_pages: torch.Tensor, k_scales: torch.Tensor, v_scales: torch.Tensor,
                  page_table: torch.Tensor, cu_seqlens: Optional[torch.Tensor] = None,
                  pos_offset: Optional[torch.Tensor] = None,
                  slot: Optional[torch.Tensor] = None, theta: float = 1e7,
                  sections: Sequence[int] = (11, 11, 10), rot_dim: int = 64,
                  device_status: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None) -> Optional[torch.Tensor]:
    """cmr_kv8_rotate_qk: rotate q in place and write the rotated k rows and the v rows
    into the paged 8-bit cache.  cu_seqlens=None means one token per sequence (a
    decode step); slot gives each sequence's row of page_table (default: its
    own number).  Returns q."""
    kp, (L, n, hk, D) = _heads(k, "k", None)
    dev = k.device
    vp = _heads(v, "v", dev)
    if vp[1] != (L, n, hk, D):
        raise ValueError("v must have the shape of k")
    qp, hq = None, 0
    if q is not None:
        qp, qs = _heads(q, "q", dev, n, L, D)
        hq = qs[2]
    pool, (pl, pages, phk, P, pd) = _pool(k_pages, v_pages, k_scales, v_scales, dev)
    if (pl, phk, pd) != (L, hk, D):
        raise ValueError(f"k_pages must be [L, pages, hk, P, D] = [{L}, pages, {hk}, P, {D}]")
    table = _want(page_table, "page_table", torch.int32, dev, (None, None))
    b, cu, off, sl = _batch(cu_seqlens, pos_offset, slot, n, start.numel(), dev)
    sp = _want(start, "start", torch.int32, dev, (b,))
    ap = _want(amount, "amount", torch.int32, dev, (b,))
    st = _maybe(device_status, "device_status", torch.int32, dev)
    sec = (_i * 3)(*[int(x) for x in sections])
    if n == 0 or L == 0:
        return q
    with torch.cuda.device(dev):
        _check(lib().cmr_kv8_rotate_qk(
            qp if hq else None, kp, vp[0], cu, b, off, sp, ap, n, L, hq, hk, D, float(theta), sec,
            int(rot_dim), *pool, pages, P, table, page_table.shape[0], page_table.shape[1], sl, st,
            _stream_ptr(dev, stream)), "cmr_kv8_rotate_qk")
    return q


def attend_kv8_workspace_bytes(num_seqs: int, n_tokens: int, num_layers: int, hq: int, hk: int,
                               head_dim: int) -> int:
    """Workspace bytes of attend_kv8 for these sizes on the current device."""
    return int(lib().cmr_kv8_attend_workspace_bytes(int(num_seqs), int(n_tokens),
                                                    int(num_layers), int(hq), int(hk),
                                                    int(head_dim)))


def attend_kv8(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
               k_scales: torch.Tensor, v_scales: torch.Tensor, page_table: torch.Tensor,
               cu_seqlens: Optional[torch.Tensor] = None,
               pos_offset: Optional[torch.Tensor] = None, slot: Optional[torch.Tensor] = None,
               scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None,
               device_status: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """cmr_kv8_attend: causal attention of q, bf16 [L, N, hq, D] (or [N, hq, D]), over
    the paged 8-bit cache; the token at absolute index p sees indices 0 .. p.
    scale defaults to 1 / sqrt(D).  workspace: a CUDA tensor of
    attend_kv8_workspace_bytes (allocated when None).  Returns out, like q."""
    qp, (L, n, hq, D) = _heads(q, "q", None)
    dev = q.device
    pool, (pl, pages, hk, P, pd) = _pool(k_pages, v_pages, k_scales, v_scales, dev)
    if (pl, pd) != (L, D):
        raise ValueError(f"k_pages must be [L, pages, hk, P, D] = [{L}, pages, hk, P, {D}]")
    table = _want(page_table, "page_table", torch.int32, dev, (None, None))
    b, cu, off, sl = _batch(cu_seqlens, pos_offset, slot, n, None, dev)
    if out is None:
        out = torch.empty_like(q)
    op = _want(out, "out", torch.bfloat16, dev, tuple(q.shape))
    st = _maybe(device_status, "device_status", torch.int32, dev)
    if n == 0 or L == 0:
        return out
    with torch.cuda.device(dev):
        # a new workspace belongs to the stream that runs the call
        with torch.cuda.stream(stream):
            ws, wp, wb = _workspace(workspace, lib().cmr_kv8_attend_workspace_bytes(
                b, n, L, hq, hk, D), dev)
        _check(lib().cmr_kv8_attend(
            qp, op, cu, b, off, n, L, hq, hk, D, D ** -0.5 if scale is None else float(scale),
            *pool, pages, P, table, page_table.shape[0], page_table.shape[1], sl, wp, wb, st,
            _stream_ptr(dev, stream)), "cmr_kv8_attend")
    return out


def last_attend_kernel() -> str:
    """Name of the kernel this thread's last attend_kv8 launched ('' before any)."""
    return lib().cmr_kv8_last_attend_kernel().decode()


def kv8_pages_workspace_bytes(table_rows: int, num_pages: int, n: int = 0) -> int:
    """Workspace bytes of the page calls for a table, a pool and n entries."""
    return int(lib().cmr_kv8_pages_workspace_bytes(int(table_rows), int(num_pages), int(n)))


def _pages_state(page_table, page_refs):
    t = _want(page_table, "page_table", torch.int32, None, (None, None))
    return t, _want(page_refs, "page_refs", torch.int32, page_table.device, (None,)), \
        page_table.device


def _pages_call(name, dev, before, after, rows, pages, n, workspace, device_status, stream):
    st = _maybe(device_status, "device_status", torch.int32, dev)
    l = lib()
    with torch.cuda.device(dev):
        with torch.cuda.stream(stream):
            ws, wp, wb = _workspace(workspace, l.cmr_kv8_pages_workspace_bytes(rows, pages, n),
                                    dev)
        _check(getattr(l, name)(*before, *after, wp, wb, st, _stream_ptr(dev, stream)), name)


def kv8_extend(page_table: torch.Tensor, page_refs: torch.Tensor, slots: torch.Tensor,
               lens: torch.Tensor, page_tokens: int, workspace: Optional[torch.Tensor] = None,
               device_status: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """cmr_kv8_extend: give rows slots the pages that they lack to hold lens tokens.
    Returns page_table."""
    t, r, dev = _pages_state(page_table, page_refs)
    n = slots.numel()
    s = _want(slots, "slots", torch.int32, dev, (n,))
    ln = _want(lens, "lens", torch.int32, dev, (n,))
    if n:
        rows, cols = page_table.shape
        _pages_call("cmr_kv8_extend", dev, (t, rows, cols, r, page_refs.numel(),
                                            int(page_tokens)), (s, ln, n), rows,
                    page_refs.numel(), n, workspace, device_status, stream)
    return page_table


def kv8_fork(k_pages: torch.Tensor, v_pages: torch.Tensor, k_scales: torch.Tensor,
             v_scales: torch.Tensor, page_table: torch.Tensor, page_refs: torch.Tensor,
             src: torch.Tensor, dst: torch.Tensor, lens: torch.Tensor,
             workspace: Optional[torch.Tensor] = None,
             device_status: Optional[torch.Tensor] = None,
             stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """cmr_kv8_fork: make the empty rows dst hold the first lens tokens of rows src,
    whole pages shared and the rest copied.  Returns page_table."""
    t, r, dev = _pages_state(page_table, page_refs)
    pool, (L, pages, hk, P, D) = _pool(k_pages, v_pages, k_scales, v_scales, dev)
    if pages != page_refs.numel():
        raise ValueError(f"page_refs counts {page_refs.numel()} pages, the pool holds {pages}")
    n = src.numel()
    s = _want(src, "src", torch.int32, dev, (n,))
    d = _want(dst, "dst", torch.int32, dev, (n,))
    ln = _want(lens, "lens", torch.int32, dev, (n,))
    if n:
        rows, cols = page_table.shape
        _pages_call("cmr_kv8_fork", dev, pool + (L, hk, D, pages, P, t, rows, cols, r),
                    (s, d, ln, n), rows, pages, n, workspace, device_status, stream)
    return page_table


def kv8_free(page_table: torch.Tensor, page_refs: torch.Tensor, slots: torch.Tensor,
             workspace: Optional[torch.Tensor] = None,
             device_status: Optional[torch.Tensor] = None,
             stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """cmr_kv8_free: empty rows slots, one holder less for each of their pages.
    Returns page_table."""
    t, r, dev = _pages_state(page_table, page_refs)
    n = slots.numel()
    s = _want(slots, "slots", torch.int32, dev, (n,))
    if n:
        rows, cols = page_table.shape
        _pages_call("cmr_kv8_free", dev, (t, rows, cols, r, page_refs.numel()), (s, n), rows,
                    page_refs.numel(), n, workspace, device_status, stream)
    return page_table


def kv8_compact(k_pages: torch.Tensor, v_pages: torch.Tensor, k_scales: torch.Tensor,
                v_scales: torch.Tensor, page_table: torch.Tensor, page_refs: torch.Tensor,
                workspace: Optional[torch.Tensor] = None,
                device_status: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """cmr_kv8_compact: move pages so that those in use are the pool's first.
    Returns page_table."""
    t, r, dev = _pages_state(page_table, page_refs)
    pool, (L, pages, hk, P, D) = _pool(k_pages, v_pages, k_scales, v_scales, dev)
    if pages != page_refs.numel():
        raise ValueError(f"page_refs counts {page_refs.numel()} pages, the pool holds {pages}")
    rows, cols = page_table.shape
    _pages_call("cmr_kv8_compact", dev, pool + (L, hk, D, pages, P, t, rows, cols, r), (), rows,
                pages, 0, workspace, device_status, stream)
    return page_table
