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
_INT = torch.int32


def _dev(t, name, dtype, ndim, device=None):
    """``t`` as a contiguous CUDA tensor of this type and number of dimensions."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    # a decode step makes these checks dozens of times: one test when all is well
    if t.is_cuda and t.is_contiguous() and t.dim() == ndim and \
            (dtype is None or t.dtype is dtype) and (device is None or t.device == device):
        return t
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the HAD library has no CPU path)")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got {t.dim()}")
    raise ValueError(f"{name} is on {t.device}, the other tensors on {device}")


def _ints(t, name, n, device):
    """An int32 vector of n entries; its address."""
    _dev(t, name, _INT, 1, device)
    if t.numel() != n:
        raise ValueError(f"{name} must have {n} entries, got {t.numel()}")
    return t.data_ptr()


def _opt(t, name, n, device):
    return None if t is None else _ints(t, name, n, device)


def _shaped(t, name, dtype, shape, device):
    _dev(t, name, dtype, len(shape), device)
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    return t


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

    def __init__(self, kbits, vcodes, vscale):
        _dev(kbits, "kbits", _INT, 4)
        _dev(vcodes, "vcodes", torch.uint8, 4, kbits.device)
        _dev(vscale, "vscale", torch.bfloat16, 4, kbits.device)
        pages, heads, page, words = kbits.shape
        if vcodes.shape != (pages, heads, page, 16 * words) or vscale.shape != (pages, heads, page, 2):
            raise ValueError("kbits, vcodes and vscale must be [pages, heads, page, d/32], "
                             f"[.., d/2] and [.., 2], got {tuple(kbits.shape)}, "
                             f"{tuple(vcodes.shape)} and {tuple(vscale.shape)}")
        self.kbits, self.vcodes, self.vscale = kbits, vcodes, vscale
        self.pages, self.heads, self.page, self.d = pages, heads, page, 32 * words
        self.device = kbits.device
        self._pool = _Pool(kbits.data_ptr(), vcodes.data_ptr(), vscale.data_ptr(), pages, heads,
                           page, self.d)
        self._ref = ctypes.byref(self._pool)

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


def _dtype_code(t, name):
    if t.dtype == torch.bfloat16:
        return HAD_BF16
    if t.dtype == torch.float32:
        return HAD_F32
    raise TypeError(f"{name} must be bfloat16 or float32, got {t.dtype}")


def _of(cache):
    if not isinstance(cache, Cache):
        raise TypeError("cache must be a Cache")
    return cache


def had_cache_append(k, v, sigma_k, cache, table, start, counts=None, dev_status=None,
                     stream=None):
    """Write tokens k, v [B, heads, T, d] of table rows [B, max_pages] from position start[b] on;
    of row b the first counts[b] (default: all T)."""
    dev = _of(cache).device
    B, H, T, d = _dev(k, "k", None, 4, dev).shape
    if H != cache.heads or d != cache.d:
        raise ValueError(f"k must be [B, {cache.heads}, T, {cache.d}], got {tuple(k.shape)}")
    _shaped(v, "v", k.dtype, (B, H, T, d), dev)
    _shaped(sigma_k, "sigma_k", torch.float32, (H,), dev)
    width = _rows(table, B, dev)
    p_start, p_counts = _ints(start, "start", B, dev), _opt(counts, "counts", B, dev)
    p_status = _opt(dev_status, "dev_status", 1, dev)
    with _on(dev, stream) as s:
        _check(_lib.had_cache_append(k.data_ptr(), v.data_ptr(), _dtype_code(k, "k"),
                                     sigma_k.data_ptr(), cache._ref, table.data_ptr(), width,
                                     p_start, p_counts, B, T, p_status, s), "had_cache_append")


def had_cache_read(cache, table, start, T, counts=None, bits=None, values=None, dev_status=None,
                   stream=None):
    """Tokens start[b] .. start[b] + counts[b] - 1 (default: T of them); returns
    (bits [B, heads, T, d/32] int32, values [B, heads, T, d] float32), zeros behind the count."""
    dev = _of(cache).device
    B = _dev(table, "table", _INT, 2, dev).shape[0]
    width = _rows(table, B, dev)
    p_start, p_counts = _ints(start, "start", B, dev), _opt(counts, "counts", B, dev)
    p_status = _opt(dev_status, "dev_status", 1, dev)
    with _on(dev, stream) as s:
        if bits is None:
            bits = torch.empty((B, cache.heads, T, cache.d // 32), dtype=_INT, device=dev)
        if values is None:
            values = torch.empty((B, cache.heads, T, cache.d), dtype=torch.float32, device=dev)
        _shaped(bits, "bits", _INT, (B, cache.heads, T, cache.d // 32), dev)
        _shaped(values, "values", torch.float32, (B, cache.heads, T, cache.d), dev)
        _check(_lib.had_cache_read(cache._ref, table.data_ptr(), width, p_start, p_counts, B, T,
                                   bits.data_ptr(), values.data_ptr(), p_status, s),
               "had_cache_read")
    return bits, values


def had_cache_attention(q, sigma_q, cache, table, lens, N, tau, window=0, sinks=0, counts=None,
                        out=None, dev_status=None, stream=None):
    """Attention of the newest tokens q [B, Hq, T, d] (of which counts[b], default all) to the
    lens[b] cached ones: the N best visible keys, within `window` positions and the first
    `sinks` tokens if window > 0; returns out [B, Hq, T, d] float32."""
    dev = _of(cache).device
    B, Hq, T, d = _dev(q, "q", None, 4, dev).shape
    if d != cache.d:
        raise ValueError(f"q must be [B, Hq, T, {cache.d}], got {tuple(q.shape)}")
    _shaped(sigma_q, "sigma_q", torch.float32, (Hq,), dev)
    width = _rows(table, B, dev)
    p_lens, p_counts = _ints(lens, "lens", B, dev), _opt(counts, "counts", B, dev)
    p_status = _opt(dev_status, "dev_status", 1, dev)
    with _on(dev, stream) as s:
        if out is None:
            out = torch.empty((B, Hq, T, d), dtype=torch.float32, device=dev)
        else:
            _shaped(out, "out", torch.float32, (B, Hq, T, d), dev)
        _check(_lib.had_cache_attention(q.data_ptr(), _dtype_code(q, "q"), sigma_q.data_ptr(),
                                        cache._ref, table.data_ptr(), width, p_lens, p_counts, B,
                                        Hq, T, _int(N, "N"), tau, _int(window, "window"),
                                        _int(sinks, "sinks"), out.data_ptr(), p_status, s),
               "had_cache_attention")
    return out


def _rows(table, B, dev):
    """Entries of a row of the table of B sequences."""
    _dev(table, "table", _INT, 2, dev)
    if table.shape[0] != B:
        raise ValueError(f"table must have {B} rows, got {table.shape[0]}")
    return table.shape[1]


def _books(table, lens, refs):
    """Device, S, max_pages and pages of the books of a call."""
    dev = _dev(table, "table", _INT, 2).device
    S, width = table.shape
    if lens is not None:
        _ints(lens, "lens", S, dev)
    _dev(refs, "refs", _INT, 1, dev)
    return dev, S, width, refs.numel()


def had_cache_fork(table, lens, refs, page, src, dst, dev_status=None, stream=None):
    """Sequence dst[i] continues as a copy of sequence src[i], for all i at once; in place."""
    dev, S, width, P = _books(table, lens, refs)
    n = _dev(src, "src", _INT, 1, dev).numel()
    p_dst = _ints(dst, "dst", n, dev)
    p_status = _opt(dev_status, "dev_status", 1, dev)
    with _on(dev, stream) as s:
        _check(_lib.had_cache_fork(table.data_ptr(), lens.data_ptr(), refs.data_ptr(), S, width,
                                   P, _int(page, "page"), src.data_ptr(), p_dst, n, p_status, s),
               "had_cache_fork")


def had_cache_reserve(table, lens, refs, page, grow, src=None, dst=None, dev_status=None,
                      stream=None):
    """Room for grow[s] more tokens of every sequence, in place; returns (src [S], dst [S]) int32,
    the shared last pages to be copied (-1: none) with had_cache_copy_pages."""
    dev, S, width, P = _books(table, lens, refs)
    p_grow = _ints(grow, "grow", S, dev)
    p_status = _opt(dev_status, "dev_status", 1, dev)
    with _on(dev, stream) as s:
        src = torch.empty(S, dtype=_INT, device=dev) if src is None else src
        dst = torch.empty(S, dtype=_INT, device=dev) if dst is None else dst
        _check(_lib.had_cache_reserve(table.data_ptr(), lens.data_ptr(), refs.data_ptr(), S,
                                      width, P, _int(page, "page"), p_grow, _ints(src, "src", S, dev),
                                      _ints(dst, "dst", S, dev), p_status, s),
               "had_cache_reserve")
    return src, dst


def had_cache_free(table, lens, refs, seqs, dev_status=None, stream=None):
    """The sequences listed in seqs [n] let their pages go and become empty; in place."""
    dev, S, width, P = _books(table, lens, refs)
    n = _dev(seqs, "seqs", _INT, 1, dev).numel()
    p_status = _opt(dev_status, "dev_status", 1, dev)
    with _on(dev, stream) as s:
        _check(_lib.had_cache_free(table.data_ptr(), lens.data_ptr(), refs.data_ptr(), S, width,
                                   P, seqs.data_ptr(), n, p_status, s), "had_cache_free")


def had_cache_evict(table, lens, refs, page, window, sinks=0, dev_status=None, stream=None):
    """Every sequence lets go of the pages that lie wholly in [sinks, lens - window); in place."""
    dev, S, width, P = _books(table, lens, refs)
    p_status = _opt(dev_status, "dev_status", 1, dev)
    with _on(dev, stream) as s:
        _check(_lib.had_cache_evict(table.data_ptr(), lens.data_ptr(), refs.data_ptr(), S, width,
                                    P, _int(page, "page"), _int(window, "window"),
                                    _int(sinks, "sinks"), p_status, s), "had_cache_evict")


def had_cache_compact(table, refs, src=None, dst=None, live=None, dev_status=None, stream=None):
    """Renames the used pages to 0 .. live - 1, in place; returns (src [pages], dst [pages],
    live [1]) int32, the pages to be copied (-1: none) with had_cache_copy_pages."""
    dev, S, width, P = _books(table, None, refs)
    p_status = _opt(dev_status, "dev_status", 1, dev)
    with _on(dev, stream) as s:
        src = torch.empty(P, dtype=_INT, device=dev) if src is None else src
        dst = torch.empty(P, dtype=_INT, device=dev) if dst is None else dst
        live = torch.empty(1, dtype=_INT, device=dev) if live is None else live
        _check(_lib.had_cache_compact(table.data_ptr(), refs.data_ptr(), S, width, P,
                                      _ints(src, "src", P, dev), _ints(dst, "dst", P, dev),
                                      _ints(live, "live", 1, dev), p_status, s),
               "had_cache_compact")
    return src, dst, live


def had_cache_copy_pages(cache, src, dst, dev_status=None, stream=None):
    """Copies page src[i] to page dst[i] of the pool; pairs with a negative index are skipped."""
    dev = _of(cache).device
    n = _dev(src, "src", _INT, 1, dev).numel()
    p_dst = _ints(dst, "dst", n, dev)
    p_status = _opt(dev_status, "dev_status", 1, dev)
    with _on(dev, stream) as s:
        _check(_lib.had_cache_copy_pages(cache._ref, src.data_ptr(), p_dst, n, p_status, s),
               "had_cache_copy_pages")
