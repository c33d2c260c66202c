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
import functools
import os
import struct
from typing import Optional, Sequence, Tuple

import torch

from .cmr import CMR_OK

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

# cmr_kv8_call's numbers, and the packing of their words: the arguments in one array cost
# half of what ctypes takes for each of them.  The tensors are known to be on the device.
_KNOWN_ADDRESSES = 256
_CALLS = {"cmr_kv8_rotate_qk": (0, struct.Struct("=13qd14q")),
          "cmr_kv8_attend": (1, struct.Struct("=10qd14q")),
          "cmr_kv8_extend": (2, struct.Struct("=13q")), "cmr_kv8_fork": (3, struct.Struct("=21q")),
          "cmr_kv8_free": (4, struct.Struct("=9q")), "cmr_kv8_compact": (5, struct.Struct("=17q"))}
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
    "cmr_kv8_free": (ctypes.c_int, [_p, _i, _i, _p, _i, _p, _i, _p, _p]),
    "cmr_kv8_compact": (ctypes.c_int, _POOL + [_i, _i, _i, _i, _i, _p, _i, _i, _p, _p, _z, _p,
                                               _p]),
    "cmr_kv8_pages_workspace_bytes": (_z, [_i, _i, _i]),
    "cmr_kv8_call": (ctypes.c_int, [_i, ctypes.c_char_p, _i]),
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


# The checks below take a decode step's dozen tensors, which cost as much host time as its
# launch: the good case is told by few comparisons, and `ix` is the device's index.

def _raw_stream(ix: int, stream: Optional[torch.cuda.Stream]) -> int:
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(ix)


def _want(t, name: str, dtype: torch.dtype, ix: Optional[int], shape=None) -> int:
    """t's data pointer, after the checks (shape: a tuple, None for any size in a place)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if ix is not None and t.get_device() != ix:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{ix}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and (t.dim() != len(shape) or any(
            w is not None and w != s for w, s in zip(shape, t.shape))):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    return t.data_ptr()


def _ptr(t, name: str, dtype: torch.dtype, ix: int, shape: Tuple[int, ...]) -> int:
    """_want for a known shape."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == ix and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    return _want(t, name, dtype, ix, shape)


def _ints(t, name: str, ix: int, n: int) -> int:
    """_want for n int32 values."""
    try:
        if t.dtype is torch.int32 and t.dim() == 1 and t.numel() == n and \
                t.get_device() == ix and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    return _want(t, name, torch.int32, ix, (n,))


def _status(t, ix):
    return 0 if t is None else _want(t, "device_status", torch.int32, ix)


def _pool(k_pages, v_pages, k_scales, v_scales, ix):
    """Pointers of the pool, and (L, pages, hk, P, D)."""
    kp = _want(k_pages, "k_pages", torch.float8_e4m3fn, ix)
    shape = k_pages.shape
    if len(shape) != 5:
        raise ValueError(f"k_pages must be [L, pages, hk, P, D], got {list(shape)}")
    heads = shape[:3]
    return (kp, _ptr(v_pages, "v_pages", torch.float8_e4m3fn, ix, shape),
            _ptr(k_scales, "k_scales", torch.float32, ix, heads),
            _ptr(v_scales, "v_scales", torch.float32, ix, heads)), shape


def _heads(t, name, ix, n=None, L=None, D=None):
    """(pointer, (L, N, H, D)) of bf16 [L, N, H, D] or [N, H, D]."""
    p = _want(t, name, torch.bfloat16, ix)
    s = t.shape
    if len(s) == 3:
        s = (1, *s)
    if len(s) != 4:
        raise ValueError(f"{name} must be [L, N, H, D] or [N, H, D]")
    if n is not None and (s[1] != n or s[0] != L or s[3] != D):
        raise ValueError(f"{name} shape {tuple(s)} does not match L={L}, N={n}, D={D}")
    return p, s


def _table(page_table, ix):
    """(pointer, rows, columns) of page_table."""
    p = _want(page_table, "page_table", torch.int32, ix)
    if page_table.dim() != 2:
        raise ValueError("page_table must be [rows, max_pages]")
    rows, cols = page_table.shape
    return p, rows, cols


def _batch(cu_seqlens, pos_offset, slot, n, ix):
    """(num_seqs, pointers of cu_seqlens, pos_offset and slot)."""
    if cu_seqlens is None:
        b, cu = n, 0
    else:
        cu = _want(cu_seqlens, "cu_seqlens", torch.int32, ix)
        b = cu_seqlens.numel() - 1
        if b < 0 or cu_seqlens.dim() != 1:
            raise ValueError("cu_seqlens needs num_seqs + 1 entries")
    return b, cu, 0 if pos_offset is None else _ints(pos_offset, "pos_offset", ix, b), \
        0 if slot is None else _ints(slot, "slot", ix, b)


def _workspace(workspace, need, dev, stream):
    """(tensor, pointer, bytes): the caller's, or a new one that belongs to the stream
    that runs the call."""
    if workspace is None:
        if need == 0:
            return None, 0, 0
        if stream is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        else:
            with torch.cuda.stream(stream):
                workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        return workspace, workspace.data_ptr(), need
    if not workspace.is_cuda or workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous CUDA tensor on {dev}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


@functools.lru_cache(maxsize=64)
def _sections(t, h, w):
    """(array, address) of the three counts."""
    a = (_i * 3)(t, h, w)
    return a, ctypes.addressof(a)


def _call(name: str, ix: int, *args):
    """The C function on device ix, as the current one."""
    number, words = _CALLS[name]
    try:
        packed = words.pack(*args)
    except struct.error as e:
        raise TypeError(f"{name}: an argument is not a number of its kind ({e})") from None
    f = (_lib or lib()).cmr_kv8_call
    number += _KNOWN_ADDRESSES
    if torch._C._cuda_getDevice() == ix:
        status = f(number, packed, len(packed) // 8)
    else:
        with torch.cuda.device(ix):
            status = f(number, packed, len(packed) // 8)
    if status != CMR_OK:
        raise Kv8Error(status, name)


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
    ix = k.get_device()
    vp = _ptr(v, "v", torch.bfloat16, ix, k.shape)
    qp, hq = 0, 0
    if q is not None:
        qp, qs = _heads(q, "q", ix, n, L, D)
        hq = qs[2]
    pool, (pl, pages, phk, P, pd) = _pool(k_pages, v_pages, k_scales, v_scales, ix)
    if (pl, phk, pd) != (L, hk, D):
        raise ValueError(f"k_pages must be [L, pages, hk, P, D] = [{L}, pages, {hk}, P, {D}]")
    table, rows, cols = _table(page_table, ix)
    b, cu, off, sl = _batch(cu_seqlens, pos_offset, slot, n, ix)
    sp = _ints(start, "start", ix, b)
    ap = _ints(amount, "amount", ix, b)
    st = _status(device_status, ix)
    if n and L:
        _call("cmr_kv8_rotate_qk", ix, qp if hq else 0, kp, vp, cu, b, off, sp, ap, n, L, hq, hk, D,
              theta, _sections(*sections)[1], rot_dim, *pool, pages, P, table, rows, cols, sl, st,
              _raw_stream(ix, stream))
    return q


@functools.lru_cache(maxsize=1024)
def _attend_bytes(index, *sizes):
    with torch.cuda.device(index):
        return lib().cmr_kv8_attend_workspace_bytes(*sizes)


def attend_kv8_workspace_bytes(num_seqs: int, n_tokens: int, num_layers: int, hq: int, hk: int,
                               head_dim: int, device: Optional[torch.device] = None) -> int:
    """Workspace bytes of attend_kv8 for these sizes on a device (default: the current)."""
    index = None if device is None else torch.device(device).index
    if not torch.cuda.is_available():  # sizes that leave nothing to do need no device
        return lib().cmr_kv8_attend_workspace_bytes(num_seqs, n_tokens, num_layers, hq, hk, head_dim)
    return _attend_bytes(torch.cuda.current_device() if index is None else index, num_seqs,
                         n_tokens, num_layers, hq, hk, head_dim)


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
    ix = q.get_device()
    pool, (pl, pages, hk, P, pd) = _pool(k_pages, v_pages, k_scales, v_scales, ix)
    if (pl, pd) != (L, D):
        raise ValueError(f"k_pages must be [L, pages, hk, P, D] = [{L}, pages, hk, P, {D}]")
    table, rows, cols = _table(page_table, ix)
    b, cu, off, sl = _batch(cu_seqlens, pos_offset, slot, n, ix)
    if out is not None:
        op = _ptr(out, "out", torch.bfloat16, ix, q.shape)
    else:
        if stream is None:
            out = torch.empty_like(q)
        else:
            with torch.cuda.stream(stream):
                out = torch.empty_like(q)
        op = out.data_ptr()
    st = _status(device_status, ix)
    if n and L:
        ws, wp, wb = _workspace(workspace, _attend_bytes(ix, b, n, L, hq, hk, D)
                                if workspace is None else 0, q.device, stream)
        _call("cmr_kv8_attend", ix, qp, op, cu, b, off, n, L, hq, hk, D,
              D ** -0.5 if scale is None else scale, *pool, pages, P, table, rows, cols, sl, wp,
              wb, st, _raw_stream(ix, stream))
    return out


def last_attend_kernel() -> str:
    """Name of the kernel this thread's last attend_kv8 launched ('' before any)."""
    return lib().cmr_kv8_last_attend_kernel().decode()


@functools.lru_cache(maxsize=1024)
def kv8_pages_workspace_bytes(table_rows: int, num_pages: int, n: int = 0) -> int:
    """Workspace bytes of the page calls for a table, a pool and n entries."""
    return lib().cmr_kv8_pages_workspace_bytes(table_rows, num_pages, n)


def _pages_state(page_table, page_refs, *pool):
    """(device index, pointers and shape of the pool, pointer of the table, rows, columns,
    pointer of the counts, pages)."""
    t, rows, cols = _table(page_table, None)
    ix = page_table.get_device()
    if not pool:
        r = _want(page_refs, "page_refs", torch.int32, ix, (None,))
        return ix, (), None, t, rows, cols, r, page_refs.numel()
    ptrs, shape = _pool(*pool, ix)
    r = _ints(page_refs, "page_refs", ix, shape[1])
    return ix, ptrs, shape, t, rows, cols, r, shape[1]


def _pages_call(name, table, before, after, rows, pages, n, workspace, device_status, stream):
    ix = table.get_device()
    st = _status(device_status, ix)
    ws, wp, wb = _workspace(workspace, kv8_pages_workspace_bytes(rows, pages, n)
                            if workspace is None else 0, table.device, stream)
    _call(name, ix, *before, *after, wp, wb, st, _raw_stream(ix, stream))


def kv8_extend(page_table: torch.Tensor, page_refs: torch.Tensor, slots: torch.Tensor,
               lens: torch.Tensor, page_tokens: int, workspace: Optional[torch.Tensor] = None,
               device_status: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """cmr_kv8_extend: give rows slots the pages that they lack to hold lens tokens.
    Returns page_table."""
    ix, _, _, t, rows, cols, r, pages = _pages_state(page_table, page_refs)
    n = slots.numel()
    s = _ints(slots, "slots", ix, n)
    ln = _ints(lens, "lens", ix, n)
    if n:
        _pages_call("cmr_kv8_extend", page_table, (t, rows, cols, r, pages, page_tokens), (s, ln, n),
                    rows, pages, n, workspace, device_status, stream)
    return page_table


def kv8_fork(k_pages: torch.Tensor, v_pages: torch.Tensor, k_scales: torch.Tensor,
             v_scales: torch.Tensor, page_table: torch.Tensor, page_refs: torch.Tensor,
             src: torch.Tensor, dst: torch.Tensor, lens: torch.Tensor,
             workspace: Optional[torch.Tensor] = None,
             device_status: Optional[torch.Tensor] = None,
             stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """cmr_kv8_fork: make the empty rows dst hold the first lens tokens of rows src,
    whole pages shared and the rest copied.  Returns page_table."""
    ix, pool, (L, _, hk, P, D), t, rows, cols, r, pages = _pages_state(
        page_table, page_refs, k_pages, v_pages, k_scales, v_scales)
    n = src.numel()
    s = _ints(src, "src", ix, n)
    d = _ints(dst, "dst", ix, n)
    ln = _ints(lens, "lens", ix, n)
    if n:
        _pages_call("cmr_kv8_fork", page_table, pool + (L, hk, D, pages, P, t, rows, cols, r),
                    (s, d, ln, n), rows, pages, n, workspace, device_status, stream)
    return page_table


def kv8_free(page_table: torch.Tensor, page_refs: torch.Tensor, slots: torch.Tensor,
             device_status: Optional[torch.Tensor] = None,
             stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """cmr_kv8_free: empty rows slots, one holder less for each of their pages.
    Returns page_table."""
    ix, _, _, t, rows, cols, r, pages = _pages_state(page_table, page_refs)
    n = slots.numel()
    s = _ints(slots, "slots", ix, n)
    if n:
        _call("cmr_kv8_free", ix, t, rows, cols, r, pages, s, n, _status(device_status, ix),
              _raw_stream(ix, stream))
    return page_table


def kv8_compact(k_pages: torch.Tensor, v_pages: torch.Tensor, k_scales: torch.Tensor,
                v_scales: torch.Tensor, page_table: torch.Tensor, page_refs: torch.Tensor,
                workspace: Optional[torch.Tensor] = None,
                device_status: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """cmr_kv8_compact: move pages so that those in use are the pool's first.
    Returns page_table."""
    ix, pool, (L, _, hk, P, D), t, rows, cols, r, pages = _pages_state(
        page_table, page_refs, k_pages, v_pages, k_scales, v_scales)
    if L:
        _pages_call("cmr_kv8_compact", page_table, pool + (L, hk, D, pages, P, t, rows, cols, r), (),
                    rows, pages, 0, workspace, device_status, stream)
    return page_table
