"""ctypes binding of the decoder cache of include/had.h (argument marshalling only).

The cache holds, per token and key-value head, the d signs of the key and the
value in 4 bits with a scale and a zero point, in pages that a table assigns
to sequences.  A step of a decoder, with ``lens`` tokens cached so far::

    src, dst = had_cache_reserve(table, lens, refs, page, grow)  # room, pages of its own
    had_cache_copy_pages(cache, src, dst)                        # shared last pages
    had_cache_append(k, v, sigma_k, cache, table, lens)          # per layer, as the next
    lens += grow
    out = had_cache_attention(q, sigma_q, cache, table, lens, N, tau)

One table serves the pools of all layers.  As in ``had``, each function has
the name of its C entry point and does no arithmetic of its own: it checks
tensors, allocates missing outputs, passes pointers and the stream, and raises
``HadError`` on a non-OK status.  Work goes to the current stream of the
tensors' device, or to ``stream``; outputs are allocated on that same stream.
No call synchronizes, so what only the device can see (a page that is not
there, a pool that is full) is reported in ``dev_status``.
"""
import contextlib
import ctypes

import torch

from . import had as _had
from .had import HAD_BF16, HAD_F32, HadError  # noqa: F401  (HadError: for callers)

HAD_ERR_NO_PAGES = 7

HAD_OP_CACHE_ATTENTION = 13
HAD_OP_CACHE_APPEND = 14
HAD_OP_CACHE_READ = 15
HAD_OP_CACHE_FORK = 16
HAD_OP_CACHE_RESERVE = 17
HAD_OP_CACHE_FREE = 18
HAD_OP_CACHE_EVICT = 19
HAD_OP_CACHE_COMPACT = 20
HAD_OP_CACHE_COPY_PAGES = 21


class _Pool(ctypes.Structure):
    _fields_ = [("kbits", ctypes.c_void_p), ("vcodes", ctypes.c_void_p),
                ("vscale", ctypes.c_void_p), ("pages", ctypes.c_int), ("heads", ctypes.c_int),
                ("page", ctypes.c_int), ("d", ctypes.c_int)]


def _declare(lib):
    vp, i32, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    pool = ctypes.POINTER(_Pool)
    sig = {
        "had_cache_append": [vp, vp, i32, vp, pool, vp, i32, vp, vp, i32, i32, vp, vp],
        "had_cache_read": [pool, vp, i32, vp, vp, i32, i32, vp, vp, vp, vp],
        "had_cache_attention": [vp, i32, vp, pool, vp, i32, vp, vp, i32, i32, i32, i32, f32, i32,
                                i32, vp, vp, vp],
        "had_cache_fork": [vp, vp, vp, i32, i32, i32, i32, vp, vp, i32, vp, vp],
        "had_cache_reserve": [vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, vp],
        "had_cache_free": [vp, vp, vp, i32, i32, i32, vp, i32, vp, vp],
        "had_cache_evict": [vp, vp, vp, i32, i32, i32, i32, i32, i32, vp, vp],
        "had_cache_compact": [vp, vp, i32, i32, i32, vp, vp, vp, vp, vp],
        "had_cache_copy_pages": [pool, vp, vp, i32, vp, vp],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    return lib


_lib = _declare(_had._lib)
_INT, _F32, _BF16 = torch.int32, torch.float32, torch.bfloat16
_Tensor = torch.Tensor


def _dev(t, name, dtype, ndim, device=None):
    """``t`` as a contiguous CUDA tensor of this type and number of dimensions."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the HAD library has no CPU path)")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got {t.dim()}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the other tensors on {device}")
    return t


def _shaped(t, name, dtype, shape, device):
    """The address of ``t``, a contiguous CUDA tensor of this type and shape."""
    # a step of a decoder makes these checks dozens of times: one expression
    # when all is well (0.4 us), the reasons otherwise
    if not (isinstance(t, _Tensor) and t.shape == shape and t.dtype is dtype and
            t.is_contiguous() and t.device == device and t.is_cuda):
        _dev(t, name, dtype, len(shape), device)
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


def _ints(t, name, n, device):
    """The address of an int32 vector of n entries."""
    return _shaped(t, name, _INT, (n,), device)


def _opt(t, name, n, device):
    return None if t is None else _shaped(t, name, _INT, (n,), device)


# Handles without the Python objects around them (2 us of a call each).
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


class _on:
    """The device and stream of a call: makes the tensors' device and the given
    stream current for the call where they are not, and gives the stream's
    handle."""
    __slots__ = ("stack", "handle")

    def __init__(self, device, stream):
        self.stack = None
        if stream is not None or _current_device() != device.index:
            if stream is not None and stream.device != device:
                raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
            self.stack = contextlib.ExitStack()
            self.stack.enter_context(torch.cuda.device(device))
            if stream is not None:
                self.stack.enter_context(torch.cuda.stream(stream))
        self.handle = _raw_stream(device.index)

    def __enter__(self):
        return self.handle

    def __exit__(self, *exc):
        if self.stack is not None:
            self.stack.close()
        return False


def _int(x, name):
    """A whole number that the C ABI's int holds (ctypes would cut it silently)."""
    if not -2 ** 31 <= x < 2 ** 31:
        raise ValueError(f"{name} must fit 32 bits, got {x}")
    return x


def _check(status, where):
    if status:
        raise HadError(status, where)


class Cache:
    """A pool of pages: kbits [pages, heads, page, d/32] int32, vcodes
    [pages, heads, page, d/2] uint8, vscale [pages, heads, page, 2] bfloat16.
    Holds the tensors; a program keeps one per layer."""

    __slots__ = ("kbits", "vcodes", "vscale", "pages", "heads", "page", "d", "device", "_pool")

    def __init__(self, kbits, vcodes, vscale):
        pages, heads, page, words = _dev(kbits, "kbits", _INT, 4).shape
        self.kbits, self.vcodes, self.vscale, self.device = kbits, vcodes, vscale, kbits.device
        self.pages, self.heads, self.page, self.d = pages, heads, page, 32 * words
        self._pool = _Pool(kbits.data_ptr(),
                           _shaped(vcodes, "vcodes", torch.uint8, (pages, heads, page, 16 * words),
                                   self.device),
                           _shaped(vscale, "vscale", _BF16, (pages, heads, page, 2), self.device),
                           pages, heads, page, 32 * words)

    @classmethod
    def empty(cls, pages, heads, page, d, device="cuda"):
        """A pool of zeroed pages."""
        if d not in (64, 128):
            raise ValueError(f"d must be 64 or 128, got {d}")
        if page not in (16, 32, 64, 128, 256):
            raise ValueError(f"page must be 16, 32, 64, 128 or 256, got {page}")
        return cls(torch.zeros(pages, heads, page, d // 32, dtype=_INT, device=device),
                   torch.zeros(pages, heads, page, d // 2, dtype=torch.uint8, device=device),
                   torch.zeros(pages, heads, page, 2, dtype=torch.bfloat16, device=device))


def empty_books(seqs, max_pages, pages, device="cuda"):
    """table [seqs, max_pages], lens [seqs] and refs [pages] of empty sequences."""
    return (torch.full((seqs, max_pages), -1, dtype=_INT, device=device),
            torch.zeros(seqs, dtype=_INT, device=device),
            torch.zeros(pages, dtype=_INT, device=device))


_CODES = {_BF16: HAD_BF16, _F32: HAD_F32}


def _dtype_code(t, name):
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be bfloat16 or float32, got {t.dtype}")
    return code


def _of(cache):
    if not isinstance(cache, Cache):
        raise TypeError("cache must be a Cache")
    return cache


def _table(table, B, dev):
    """The address and the row length of the table of B sequences."""
    width = table.shape[-1] if isinstance(table, _Tensor) and table.dim() == 2 else 0
    return _shaped(table, "table", _INT, (B, width), dev), width


def had_cache_append(k, v, sigma_k, cache, table, start, counts=None, dev_status=None,
                     stream=None):
    """Write tokens k, v [B, heads, T, d] of table rows [B, max_pages] from position start[b] on;
    of row b the first counts[b] (default: all T)."""
    dev = _of(cache).device
    B, H, T, d = shape = _dev(k, "k", None, 4, dev).shape
    if H != cache.heads or d != cache.d:
        raise ValueError(f"k must be [B, {cache.heads}, T, {cache.d}], got {tuple(shape)}")
    args = (k.data_ptr(), _shaped(v, "v", k.dtype, shape, dev), _dtype_code(k, "k"),
            _shaped(sigma_k, "sigma_k", _F32, (H,), dev), cache._pool, *_table(table, B, dev),
            _ints(start, "start", B, dev), _opt(counts, "counts", B, dev), B, T,
            _opt(dev_status, "dev_status", 1, dev))
    with _on(dev, stream) as s:
        _check(_lib.had_cache_append(*args, s), "had_cache_append")


def had_cache_read(cache, table, start, T, counts=None, bits=None, values=None, dev_status=None,
                   stream=None):
    """Tokens start[b] .. start[b] + counts[b] - 1 (default: T of them); returns
    (bits [B, heads, T, d/32] int32, values [B, heads, T, d] float32), zeros behind the count."""
    dev = _of(cache).device
    B = _dev(table, "table", _INT, 2, dev).shape[0]
    args = (cache._pool, *_table(table, B, dev), _ints(start, "start", B, dev),
            _opt(counts, "counts", B, dev), B, _int(T, "T"))
    p_status = _opt(dev_status, "dev_status", 1, dev)
    like_bits, like_values = (B, cache.heads, T, cache.d // 32), (B, cache.heads, T, cache.d)
    with _on(dev, stream) as s:
        if bits is None:
            bits = torch.empty(like_bits, dtype=_INT, device=dev)
        if values is None:
            values = torch.empty(like_values, dtype=_F32, device=dev)
        _check(_lib.had_cache_read(*args, _shaped(bits, "bits", _INT, like_bits, dev),
                                   _shaped(values, "values", _F32, like_values, dev), p_status, s),
               "had_cache_read")
    return bits, values


def had_cache_attention(q, sigma_q, cache, table, lens, N, tau, window=0, sinks=0, counts=None,
                        out=None, dev_status=None, stream=None):
    """Attention of the newest tokens q [B, Hq, T, d] (of which counts[b], default all) to the
    lens[b] cached ones: the N best visible keys, within `window` positions and the first
    `sinks` tokens if window > 0; returns out [B, Hq, T, d] float32."""
    dev = _of(cache).device
    B, Hq, T, d = shape = _dev(q, "q", None, 4, dev).shape
    if d != cache.d:
        raise ValueError(f"q must be [B, Hq, T, {cache.d}], got {tuple(shape)}")
    args = (q.data_ptr(), _dtype_code(q, "q"), _shaped(sigma_q, "sigma_q", _F32, (Hq,), dev),
            cache._pool, *_table(table, B, dev), _ints(lens, "lens", B, dev),
            _opt(counts, "counts", B, dev), B, Hq, T, _int(N, "N"), tau, _int(window, "window"),
            _int(sinks, "sinks"))
    p_status = _opt(dev_status, "dev_status", 1, dev)
    with _on(dev, stream) as s:
        if out is None:
            out = torch.empty_like(q, dtype=_F32)
        _check(_lib.had_cache_attention(*args, _shaped(out, "out", _F32, shape, dev), p_status, s),
               "had_cache_attention")
    return out


def _books(table, lens, refs):
    """Device of a call on the books, and (table, lens, refs, S, max_pages, pages); without
    lens where a call has none."""
    S, width = _dev(table, "table", _INT, 2).shape
    dev = table.device
    P = _dev(refs, "refs", _INT, 1, dev).shape[0]
    if lens is None:
        return dev, (table.data_ptr(), refs.data_ptr(), S, width, P)
    return dev, (table.data_ptr(), _ints(lens, "lens", S, dev), refs.data_ptr(), S, width, P)


def had_cache_fork(table, lens, refs, page, src, dst, dev_status=None, stream=None):
    """Sequence dst[i] continues as a copy of sequence src[i], for all i at once; in place."""
    dev, books = _books(table, lens, refs)
    n = _dev(src, "src", _INT, 1, dev).shape[0]
    args = (*books, _int(page, "page"), src.data_ptr(), _ints(dst, "dst", n, dev), n,
            _opt(dev_status, "dev_status", 1, dev))
    with _on(dev, stream) as s:
        _check(_lib.had_cache_fork(*args, s), "had_cache_fork")


def had_cache_reserve(table, lens, refs, page, grow, src=None, dst=None, dev_status=None,
                      stream=None):
    """Room for grow[s] more tokens of every sequence, in place; returns (src [S], dst [S]) int32,
    the shared last pages to be copied (-1: none) with had_cache_copy_pages."""
    dev, books = _books(table, lens, refs)
    S = lens.shape[0]
    args = (*books, _int(page, "page"), _ints(grow, "grow", S, dev))
    p_status = _opt(dev_status, "dev_status", 1, dev)
    with _on(dev, stream) as s:
        src = torch.empty_like(lens) if src is None else src
        dst = torch.empty_like(lens) if dst is None else dst
        _check(_lib.had_cache_reserve(*args, _ints(src, "src", S, dev), _ints(dst, "dst", S, dev),
                                      p_status, s), "had_cache_reserve")
    return src, dst


def had_cache_free(table, lens, refs, seqs, dev_status=None, stream=None):
    """The sequences listed in seqs [n] let their pages go and become empty; in place."""
    dev, books = _books(table, lens, refs)
    n = _dev(seqs, "seqs", _INT, 1, dev).shape[0]
    args = (*books, seqs.data_ptr(), n, _opt(dev_status, "dev_status", 1, dev))
    with _on(dev, stream) as s:
        _check(_lib.had_cache_free(*args, s), "had_cache_free")


def had_cache_evict(table, lens, refs, page, window, sinks=0, dev_status=None, stream=None):
    """Every sequence lets go of the pages that lie wholly in [sinks, lens - window); in place."""
    dev, books = _books(table, lens, refs)
    args = (*books, _int(page, "page"), _int(window, "window"), _int(sinks, "sinks"),
            _opt(dev_status, "dev_status", 1, dev))
    with _on(dev, stream) as s:
        _check(_lib.had_cache_evict(*args, s), "had_cache_evict")


def had_cache_compact(table, refs, src=None, dst=None, live=None, dev_status=None, stream=None):
    """Renames the used pages to 0 .. live - 1, in place; returns (src [pages], dst [pages],
    live [1]) int32, the pages to be copied (-1: none) with had_cache_copy_pages."""
    dev, books = _books(table, None, refs)
    P = refs.shape[0]
    p_status = _opt(dev_status, "dev_status", 1, dev)
    with _on(dev, stream) as s:
        src = torch.empty_like(refs) if src is None else src
        dst = torch.empty_like(refs) if dst is None else dst
        live = torch.empty(1, dtype=_INT, device=dev) if live is None else live
        _check(_lib.had_cache_compact(*books, _ints(src, "src", P, dev), _ints(dst, "dst", P, dev),
                                      _ints(live, "live", 1, dev), p_status, s),
               "had_cache_compact")
    return src, dst, live


def had_cache_copy_pages(cache, src, dst, dev_status=None, stream=None):
    """Copies page src[i] to page dst[i] of the pool; pairs with a negative index are skipped."""
    dev = _of(cache).device
    n = _dev(src, "src", _INT, 1, dev).shape[0]
    args = (cache._pool, src.data_ptr(), _ints(dst, "dst", n, dev), n,
            _opt(dev_status, "dev_status", 1, dev))
    with _on(dev, stream) as s:
        _check(_lib.had_cache_copy_pages(*args, s), "had_cache_copy_pages")
