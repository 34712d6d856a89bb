"""Binding of the decoder cache of include/had.h (argument marshalling only).

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
``HadError`` on a non-OK status.  The checks run in ``_cache.so``
(csrc/had_cache_bind.cpp): a step makes several of these calls, and through
ctypes each took longer than its kernel.  Work goes to the current stream of the
tensors' device, or to ``stream``; outputs are allocated on that same stream.
No call synchronizes, so what only the device can see (a page that is not
there, a pool that is full) is reported in ``dev_status``.
"""
import contextlib
import os

import torch

from . import had  # noqa: F401  (loads libhad.so, which _cache.so is linked to)
from .had import HadError  # noqa: F401

if not os.path.exists(os.path.join(os.path.dirname(os.path.abspath(__file__)), "_cache.so")):
    raise ImportError("_cache.so is missing: build it with `python -m "
                      "sparse_attention_sigma_b200.build`")
from . import _cache as _native  # noqa: E402

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


def _on(stream):
    """The given stream, and its device, made current for a call."""
    if not isinstance(stream, torch.cuda.Stream):
        raise TypeError("stream must be a torch.cuda.Stream")
    return torch.cuda.stream(stream)


def _check(status, where):
    if status:
        raise HadError(status, where)


def _same_device(stream, tensor):
    if isinstance(tensor, torch.Tensor) and tensor.is_cuda and stream.device != tensor.device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {tensor.device}")


def _call(function, where, args, stream, tensor):
    """Outputs of a native call on the given stream, or on the current one of the tensors'
    device."""
    if stream is None:
        result = function(*args)
    else:
        with _on(stream):
            _same_device(stream, tensor)
            result = function(*args)
    if type(result) is int:
        _check(result, where)
        return None
    _check(result[0], where)
    return result[1:]


class Cache:
    """A pool of pages: kbits [pages, heads, page, d/32] int32, vcodes
    [pages, heads, page, d/2] uint8, vscale [pages, heads, page, 2] bfloat16.
    Holds the tensors; a program keeps one per layer, and makes another for other tensors."""
    __slots__ = ("_tensors", "pages", "heads", "page", "d", "_pool")

    def __init__(self, kbits, vcodes, vscale):
        self._pool, self.pages, self.heads, self.page, self.d = _native.pool(kbits, vcodes, vscale)
        self._tensors = kbits, vcodes, vscale

    @property
    def kbits(self):
        return self._tensors[0]

    @property
    def vcodes(self):
        return self._tensors[1]

    @property
    def vscale(self):
        return self._tensors[2]

    @property
    def device(self):
        return self.kbits.device

    @classmethod
    def empty(cls, pages, heads, page, d, device="cuda"):
        """A pool of zeroed pages."""
        if d not in (64, 128):
            raise ValueError(f"d must be 64 or 128, got {d}")
        if page not in (16, 32, 64, 128, 256):
            raise ValueError(f"page must be 16, 32, 64, 128 or 256, got {page}")
        return cls(torch.zeros(pages, heads, page, d // 32, dtype=torch.int32, device=device),
                   torch.zeros(pages, heads, page, d // 2, dtype=torch.uint8, device=device),
                   torch.zeros(pages, heads, page, 2, dtype=torch.bfloat16, device=device))


def _of(cache):
    if not isinstance(cache, Cache):
        raise TypeError("cache must be a Cache")
    return cache._pool


def empty_books(seqs, max_pages, pages, device="cuda"):
    """table [seqs, max_pages], lens [seqs] and refs [pages] of empty sequences."""
    return (torch.full((seqs, max_pages), -1, dtype=torch.int32, device=device),
            torch.zeros(seqs, dtype=torch.int32, device=device),
            torch.zeros(pages, dtype=torch.int32, device=device))


def had_cache_append(k, v, sigma_k, cache, table, start, counts=None, dev_status=None,
                     stream=None):
    """Write tokens k, v [B, heads, T, d] of table rows [B, max_pages] from position start[b] on;
    of row b the first counts[b] (default: all T)."""
    _call(_native.append, "had_cache_append",
          (_of(cache), k, v, sigma_k, table, start, counts, dev_status), stream, k)


def had_cache_read(cache, table, start, T, counts=None, bits=None, values=None, dev_status=None,
                   stream=None):
    """Tokens start[b] .. start[b] + counts[b] - 1 (default: T of them); returns
    (bits [B, heads, T, d/32] int32, values [B, heads, T, d] float32), zeros behind the count."""
    return _call(_native.read, "had_cache_read",
                 (_of(cache), table, start, T, counts, bits, values, dev_status), stream, table)


def had_cache_attention(q, sigma_q, cache, table, lens, N, tau, window=0, sinks=0, counts=None,
                        out=None, dev_status=None, stream=None, max_len=0):
    """Attention of the newest tokens q [B, Hq, T, d] (of which counts[b], default all) to the
    lens[b] cached ones: the N best visible keys, within `window` positions and the first
    `sinks` tokens if window > 0; returns out [B, Hq, T, d] float32.  max_len: what lens is
    expected not to pass, a hint that speeds up many long sequences."""
    return _call(_native.attention, "had_cache_attention",
                 (_of(cache), q, sigma_q, table, lens, N, tau, window, sinks, counts, out,
                  dev_status, max_len), stream, q)[0]


def had_cache_fork(table, lens, refs, page, src, dst, dev_status=None, stream=None):
    """Sequence dst[i] continues as a copy of sequence src[i], for all i at once; in place."""
    _call(_native.fork, "had_cache_fork", (table, lens, refs, page, src, dst, dev_status), stream,
          table)


def had_cache_reserve(table, lens, refs, page, grow, src=None, dst=None, dev_status=None,
                      stream=None):
    """Room for grow[s] more tokens of every sequence, in place; returns (src [S], dst [S]) int32,
    the shared last pages to be copied (-1: none) with had_cache_copy_pages.  lens may have gone
    back since the last call: pages behind it are kept unless another sequence names them too."""
    return _call(_native.reserve, "had_cache_reserve",
                 (table, lens, refs, page, grow, src, dst, dev_status), stream, table)


def had_cache_free(table, lens, refs, seqs, dev_status=None, stream=None):
    """The sequences listed in seqs [n] let their pages go and become empty; in place."""
    _call(_native.free, "had_cache_free", (table, lens, refs, seqs, dev_status), stream, table)


def had_cache_evict(table, lens, refs, page, window, sinks=0, dev_status=None, stream=None):
    """Every sequence lets go of the pages that lie wholly in [sinks, lens - window); in place."""
    _call(_native.evict, "had_cache_evict", (table, lens, refs, page, window, sinks, dev_status),
          stream, table)


def had_cache_compact(table, refs, src=None, dst=None, live=None, dev_status=None, stream=None):
    """Renames the used pages to 0 .. live - 1, in place; returns (src [pages], dst [pages],
    live [1]) int32, the pages to be copied (-1: none) with had_cache_copy_pages."""
    return _call(_native.compact, "had_cache_compact", (table, refs, src, dst, live, dev_status),
                 stream, table)


def had_cache_copy_pages(cache, src, dst, dev_status=None, stream=None):
    """Copies page src[i] to page dst[i] of the pool; pairs with a negative index are skipped."""
    _call(_native.copy_pages, "had_cache_copy_pages", (_of(cache), src, dst, dev_status), stream,
          src)
