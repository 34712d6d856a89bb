"""The decoder cache without a GPU: refusals of the C ABI and of the binding,
and the pins of its oracle."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle
from oracle import cache as ocache
from sparse_attention_sigma_b200 import build as _build

_build.build()                      # the library loads without a GPU
from sparse_attention_sigma_b200 import cache  # noqa: E402

FAKE = 4096                         # never dereferenced: the checks fail first
OK, INVALID, UNSUPPORTED = 0, 1, 2


class PoolStruct(ctypes.Structure):
    """had_cache_t"""
    _fields_ = [("kbits", ctypes.c_void_p), ("vcodes", ctypes.c_void_p),
                ("vscale", ctypes.c_void_p), ("pages", ctypes.c_int), ("heads", ctypes.c_int),
                ("page", ctypes.c_int), ("d", ctypes.c_int)]


def _library():
    lib = ctypes.CDLL(_build.LIB)
    vp, i32, f32, pl = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.POINTER(PoolStruct)
    for name, args in {
            "had_cache_append": [vp, vp, i32, vp, pl, vp, i32, vp, vp, i32, i32, vp, vp],
            "had_cache_read": [pl, vp, i32, vp, vp, i32, i32, vp, vp, vp, vp],
            "had_cache_attention": [vp, i32, vp, pl, vp, i32, vp, vp, i32, i32, i32, i32, f32, i32,
                                    i32, i32, vp, vp, vp],
            "had_cache_fork": [vp, vp, vp, i32, i32, i32, i32, vp, vp, i32, vp, vp],
            "had_cache_reserve": [vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, vp],
            "had_cache_free": [vp, vp, vp, i32, i32, i32, vp, i32, vp, vp],
            "had_cache_evict": [vp, vp, vp, i32, i32, i32, i32, i32, i32, vp, vp],
            "had_cache_compact": [vp, vp, i32, i32, i32, vp, vp, vp, vp, vp],
            "had_cache_copy_pages": [pl, vp, vp, i32, vp, vp]}.items():
        getattr(lib, name).argtypes = args
        getattr(lib, name).restype = ctypes.c_int
    return lib


lib = _library()


def pool(pages=8, heads=2, page=16, d=64, kbits=FAKE, vcodes=FAKE, vscale=FAKE):
    return ctypes.byref(PoolStruct(kbits, vcodes, vscale, pages, heads, page, d))


def call(name, ok, **changes):
    args = dict(ok, **changes)
    return getattr(lib, name)(*args.values())


APPEND = dict(k=FAKE, v=FAKE, dt=0, sigma=FAKE, pool=pool(), table=FAKE, width=4, start=FAKE,
              counts=None, B=1, T=1, status=None, stream=None)
READ = dict(pool=pool(), table=FAKE, width=4, start=FAKE, counts=None, B=1, T=1, bits=FAKE,
            values=FAKE, status=None, stream=None)
ATTEND = dict(q=FAKE, dt=0, sigma=FAKE, pool=pool(), table=FAKE, width=4, lens=FAKE, counts=None,
              B=1, Hq=2, T=1, N=4, tau=0.1, window=0, sinks=0, max_len=0, out=FAKE, status=None,
              stream=None)
FORK = dict(table=FAKE, lens=FAKE, refs=FAKE, S=4, width=4, pages=8, page=16, src=FAKE, dst=FAKE,
            n=1, status=None, stream=None)
RESERVE = dict(table=FAKE, lens=FAKE, refs=FAKE, S=4, width=4, pages=8, page=16, grow=FAKE,
               src=FAKE, dst=FAKE, status=None, stream=None)
FREE = dict(table=FAKE, lens=FAKE, refs=FAKE, S=4, width=4, pages=8, seqs=FAKE, n=1, status=None,
            stream=None)
EVICT = dict(table=FAKE, lens=FAKE, refs=FAKE, S=4, width=4, pages=8, page=16, window=8, sinks=0,
             status=None, stream=None)
COMPACT = dict(table=FAKE, refs=FAKE, S=4, width=4, pages=8, src=FAKE, dst=FAKE, live=FAKE,
               status=None, stream=None)
COPY = dict(pool=pool(), src=FAKE, dst=FAKE, n=1, status=None, stream=None)

POOLS = [(dict(pool=None), INVALID), (dict(pool=pool(d=96)), UNSUPPORTED),
         (dict(pool=pool(page=24)), UNSUPPORTED), (dict(pool=pool(page=512)), UNSUPPORTED),
         (dict(pool=pool(pages=0)), INVALID), (dict(pool=pool(heads=0)), INVALID),
         (dict(pool=pool(kbits=None)), INVALID), (dict(pool=pool(vcodes=4100)), INVALID),
         (dict(pool=pool(vscale=None)), INVALID),
         (dict(pool=pool(pages=2 ** 31 - 1, heads=2 ** 16)), UNSUPPORTED)]
TABLES = [(dict(table=None), INVALID), (dict(table=4098), INVALID), (dict(width=0), INVALID),
          (dict(width=2 ** 27), UNSUPPORTED)]
BOOKS = TABLES[:3] + [(dict(refs=None), INVALID), (dict(S=0), INVALID), (dict(pages=0), INVALID),
                      (dict(pages=2 ** 31 - 1), UNSUPPORTED)]
PAGES = [(dict(page=0), UNSUPPORTED), (dict(page=1), UNSUPPORTED), (dict(page=48), UNSUPPORTED)]

REFUSALS = {
    "had_cache_append": (APPEND, POOLS + TABLES + [
        (dict(dt=2), INVALID), (dict(k=None), INVALID), (dict(v=4100), INVALID),
        (dict(sigma=None), INVALID), (dict(start=None), INVALID), (dict(counts=4097), INVALID),
        (dict(B=0), INVALID), (dict(T=0), INVALID), (dict(B=2 ** 16, T=2 ** 16), UNSUPPORTED),
        (dict(status=4097), INVALID)]),
    "had_cache_read": (READ, POOLS + TABLES + [
        (dict(bits=None, values=None), INVALID), (dict(values=4100), INVALID),
        (dict(start=None), INVALID), (dict(T=0), INVALID)]),
    "had_cache_attention": (ATTEND, POOLS + TABLES + [
        (dict(dt=5), INVALID), (dict(q=None), INVALID), (dict(q=4104), INVALID),
        (dict(out=None), INVALID), (dict(lens=None), INVALID), (dict(sigma=None), INVALID),
        (dict(Hq=3), INVALID), (dict(Hq=0), INVALID), (dict(N=0), INVALID),
        (dict(tau=-0.5), INVALID), (dict(tau=float("nan")), INVALID),
        (dict(tau=float("inf")), INVALID), (dict(window=-1), INVALID), (dict(sinks=-1), INVALID),
        (dict(max_len=-1), INVALID),
        (dict(T=0), INVALID), (dict(B=2 ** 15, T=2 ** 16), UNSUPPORTED)]),
    "had_cache_fork": (FORK, BOOKS + PAGES + [
        (dict(lens=None), INVALID), (dict(src=None), INVALID), (dict(dst=4098), INVALID),
        (dict(n=-1), INVALID), (dict(n=5), INVALID), (dict(S=8193), UNSUPPORTED)]),
    "had_cache_reserve": (RESERVE, BOOKS + PAGES + [
        (dict(lens=None), INVALID), (dict(grow=None), INVALID), (dict(src=None), INVALID),
        (dict(S=8193), UNSUPPORTED)]),
    "had_cache_free": (FREE, BOOKS + [(dict(seqs=None), INVALID), (dict(n=-1), INVALID)]),
    "had_cache_evict": (EVICT, BOOKS + PAGES + [(dict(window=0), INVALID),
                                                (dict(sinks=-1), INVALID)]),
    "had_cache_compact": (COMPACT, BOOKS + [(dict(live=None), INVALID), (dict(src=None), INVALID)]),
    "had_cache_copy_pages": (COPY, POOLS + [(dict(src=None), INVALID), (dict(n=-1), INVALID)]),
}


@pytest.mark.parametrize("name", sorted(REFUSALS))
def test_arguments_are_refused_before_any_cuda_call(name):
    ok, cases = REFUSALS[name]
    for changes, want in cases:
        assert call(name, ok, **changes) == want, changes


def test_empty_lists_are_no_work():
    assert call("had_cache_fork", FORK, n=0, src=None, dst=None) == OK
    assert call("had_cache_free", FREE, n=0, seqs=None) == OK
    assert call("had_cache_copy_pages", COPY, n=0, src=None, dst=None) == OK


def test_status_launches_and_workspaces():
    from sparse_attention_sigma_b200 import had
    assert had.had_status_string(cache.HAD_ERR_NO_PAGES) == "HAD_ERR_NO_PAGES"
    for op in range(cache.HAD_OP_CACHE_ATTENTION, cache.HAD_OP_CACHE_COPY_PAGES + 1):
        assert had.had_workspace_bytes(op, 1, 1, 1, 64, 1) == 0
        assert had.had_launch_count(op, 1, 1, 1, 64, 1) == 1


# --------------------------------------------------------------- the binding

I = torch.int32
K = torch.zeros(1, 2, 3, 64)
TABLE, VEC, REFS = torch.zeros(1, 4, dtype=I), torch.zeros(1, dtype=I), torch.zeros(8, dtype=I)


CALLS = {
    "Cache": lambda: cache.Cache(*[torch.zeros(1, 1, 16, 2, dtype=I)] * 3),
    "had_cache_fork": lambda: cache.had_cache_fork(TABLE, VEC, REFS, 16, VEC, VEC),
    "had_cache_reserve": lambda: cache.had_cache_reserve(TABLE, VEC, REFS, 16, VEC),
    "had_cache_free": lambda: cache.had_cache_free(TABLE, VEC, REFS, VEC),
    "had_cache_evict": lambda: cache.had_cache_evict(TABLE, VEC, REFS, 16, 8),
    "had_cache_compact": lambda: cache.had_cache_compact(TABLE, REFS),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_host_tensors_are_refused(name):
    with pytest.raises(ValueError, match="no CPU path"):
        CALLS[name]()


# a Cache holds device tensors, so these can only be reached with one: on a host
# they refuse whatever else they are given
NEED_A_CACHE = {
    "had_cache_append": lambda c: cache.had_cache_append(K, K, torch.ones(2), c, TABLE, VEC),
    "had_cache_read": lambda c: cache.had_cache_read(c, TABLE, VEC, 3),
    "had_cache_attention": lambda c: cache.had_cache_attention(K, torch.ones(2), c, TABLE, VEC, 2,
                                                               0.1),
    "had_cache_copy_pages": lambda c: cache.had_cache_copy_pages(c, VEC, VEC),
}


@pytest.mark.parametrize("name", sorted(NEED_A_CACHE))
def test_what_is_no_cache_is_refused(name):
    for c in (None, K, object()):
        with pytest.raises(TypeError, match="Cache"):
            NEED_A_CACHE[name](c)


def test_every_wrapper_is_covered():
    public = {n for n in dir(cache) if n.startswith("had_") and callable(getattr(cache, n))}
    assert public <= set(CALLS) | set(NEED_A_CACHE), public


def test_wrong_objects_are_refused():
    with pytest.raises(TypeError, match="torch.Tensor"):
        cache.had_cache_compact([[0]], REFS)
    with pytest.raises(TypeError, match="torch.Tensor"):
        cache.Cache(None, None, None)
    with pytest.raises(TypeError, match="stream"):
        cache.had_cache_compact(TABLE, REFS, stream=3)


def test_cache_empty_refuses_sizes_the_library_lacks():
    with pytest.raises(ValueError, match="d must be"):
        cache.Cache.empty(4, 1, 16, 96)
    with pytest.raises(ValueError, match="page must be"):
        cache.Cache.empty(4, 1, 24, 64)


# ---------------------------------------------------------- pins of the oracle

def test_bf16_rounding_is_directed():
    g = np.random.default_rng(3)
    x = np.concatenate([g.standard_normal(200), [0.0, 1.0, -1.0, 1e-40, -1e-40, 255.5, -255.5]])
    x = x.astype(np.float32)
    lo, hi = ocache.bf16_round(x, -1), ocache.bf16_round(x, +1)
    near = torch.from_numpy(x).bfloat16().float().numpy()
    assert (lo <= x).all() and (hi >= x).all()
    assert ((near == lo) | (near == hi)).all()
    for r in (lo, hi):
        assert not (r.view(np.uint32) & 0xFFFF).any()
    exact = lo == hi
    assert (x[exact] == lo[exact]).all()
    # neighbours: nothing of bf16 lies between
    gap = np.abs((lo[~exact].view(np.int32) >> 16) - (hi[~exact].view(np.int32) >> 16))
    assert (gap == 1).all()


def test_quantised_values_lie_within_half_a_step():
    g = np.random.default_rng(5)
    v = (g.standard_normal((64, 64)) * 10.0 ** g.integers(-6, 7, (64, 1))).astype(np.float32)
    code, s, z = ocache.quantise(v)
    assert code.min() == 0 and code.max() == 15
    for r in range(8):
        for e in range(64):
            got = Fraction(float(s[r])) * int(code[r, e]) + Fraction(float(z[r]))
            step = Fraction(float(s[r]))
            # half a step, and the two roundings of (v - z) / s: 2^-23 of at most 16 steps
            assert abs(got - Fraction(float(v[r, e]))) <= step / 2 + 16 * step / 2 ** 23


@pytest.mark.parametrize("row,codes,scale,zero", [
    (np.full(64, 0.5), 0, 0.0, 0.5),
    (np.full(64, -0.0), 0, 0.0, 0.0),
    (np.arange(64) % 16, np.arange(64) % 16, 1.0, 0.0),
    (-(np.arange(64) % 16.0), 15 - np.arange(64) % 16, 1.0, -15.0),
])
def test_quantise_closed_forms(row, codes, scale, zero):
    c, s, z = ocache.quantise(row[None].astype(np.float32))
    assert (c[0] == codes).all() and s[0] == scale and z[0] == zero


@pytest.mark.parametrize("poison", [np.nan, np.inf, -np.inf, 3.4e38])
def test_quantise_marks_rows_it_cannot_hold(poison):
    v = np.zeros((2, 64), np.float32)
    v[0, 7], v[0, 8] = poison, -3.4e38 if poison == np.float64(3.4e38) else 0
    c, s, z = ocache.quantise(v)
    assert np.isnan(s[0]) and np.isnan(z[0]) and not c.any() and s[1] == z[1] == 0


def test_attend_is_the_causal_oracle_on_a_whole_sequence():
    g = np.random.default_rng(7)
    n, d, N, tau = 40, 64, 9, 0.125
    sq, sk = (np.where(g.random((1, 1, n, d)) < 0.5, -1, 1).astype(np.int8) for _ in range(2))
    codes, s, z = ocache.quantise(g.standard_normal((n, d)).astype(np.float32))
    v = (codes * s[:, None].astype(np.float64) + z[:, None]).astype(np.float32)
    idx, _, _, out = oracle.attention_causal_rows(sq, sk, v[None, None], tau, N, range(n))
    for i in range(n):
        o, kept, _ = ocache.attend(sq[0, 0, i], sk[0, 0], codes, s, z, N, tau, 0, 0, i)
        assert (kept == idx[i][idx[i] >= 0]).all()
        np.testing.assert_allclose(o, out[i], rtol=1e-5, atol=1e-6)


def test_attend_under_a_window_is_a_masked_softmax():
    g = np.random.default_rng(9)
    n, d, W, S = 50, 64, 11, 3
    sq = np.where(g.random(d) < 0.5, -1, 1)
    sk = np.where(g.random((n, d)) < 0.5, -1, 1)
    codes, s, z = ocache.quantise(g.standard_normal((n, d)).astype(np.float32))
    v = codes * s[:, None].astype(np.float64) + z[:, None]
    logit = torch.tensor(0.1 * (sk @ sq))
    for i in (0, 2, 10, 11, 13, 14, 49):
        mask = torch.tensor([j <= i and (j > i - W or j < S) for j in range(n)])
        want = torch.softmax(logit.masked_fill(~mask, -torch.inf), 0).numpy() @ v
        o, kept, _ = ocache.attend(sq, sk, codes, s, z, n, 0.1, W, S, i)
        assert kept.size == mask.sum()
        np.testing.assert_allclose(o, want, atol=1e-12)
    o, kept, _ = ocache.attend(sq, sk, codes, s, z, 4, 0.1, W, S, -1)
    assert not o.any() and kept.size == 0


def test_books_by_hand():
    # pages of 16: sequence 0 holds 20 tokens in pages 3 and 1, sequence 1 nothing
    b = ocache.Books([[3, 1, -1, -1], [-1] * 4], [20, 0], [0, 1, 0, 1, 0, 0], 16)
    b.fork([0], [1])
    assert b.table == [[3, 1, -1, -1]] * 2 and b.lens == [20, 20] and b.refs == [0, 2, 0, 2, 0, 0]
    # both grow into a third page; the first gets a copy of page 1, the second keeps it
    assert b.reserve([13, 20]) == ([1, -1], [0, -1])
    assert b.table == [[3, 0, 2, -1], [3, 1, 4, -1]] and b.refs == [1, 1, 1, 2, 1, 0]
    assert b.reserve([13, 20]) == ([-1, -1], [-1, -1])          # the room is there
    assert b.reserve([40, 40]) is None                          # one page is left, two are wanted
    assert b.refs == [1, 1, 1, 2, 1, 0]
    b.lens = [33, 40]
    b.evict(8, 4)                                               # 16 .. 24 and 16 .. 31 unseen
    assert b.table == [[3, 0, 2, -1], [3, -1, 4, -1]] and b.refs == [1, 0, 1, 2, 1, 0]
    b.evict(1, 0)
    assert b.table == [[-1, -1, 2, -1], [-1, -1, 4, -1]] and b.refs == [0, 0, 1, 0, 1, 0]
    assert b.compact() == ([2, 4, -1, -1, -1, -1], [0, 1, -1, -1, -1, -1], 2)
    assert b.table == [[-1, -1, 0, -1], [-1, -1, 1, -1]] and b.refs == [1, 1, 0, 0, 0, 0]
    b.free([1, 1])
    assert b.table[1] == [-1] * 4 and b.lens == [33, 0] and b.refs == [1, 0, 0, 0, 0, 0]


def test_books_by_hand_where_a_length_was_lowered():
    # 20 tokens in pages 0 and 1, forked; the copy goes back to 16 tokens and on by 4: page 1,
    # behind its length, is the other one's too
    b = ocache.Books([[0, 1, -1], [-1] * 3], [20, 0], [1, 1, 0, 0, 0], 16)
    b.fork([0], [1])
    b.lens[1] = 16
    assert b.reserve([0, 4]) == ([-1, -1], [-1, -1])
    assert b.table == [[0, 1, -1], [0, 2, -1]] and b.refs == [2, 1, 1, 0, 0]
    # both go back to 10 tokens and on: page 0 is copied for the first, and kept by the last
    b.lens = [10, 10]
    assert b.reserve([1, 1]) == ([0, -1], [3, -1])
    assert b.table == [[3, 1, -1], [0, 2, -1]] and b.refs == [1, 1, 1, 1, 0]
    # three hold page 1 behind their lengths: whoever grows over it lets it go
    b = ocache.Books([[0, 1], [2, 1], [3, 1]], [16, 16, 16], [1, 3, 1, 1, 0, 0, 0], 16)
    assert b.reserve([1, 0, 5]) == ([-1] * 3, [-1] * 3)
    assert b.table == [[0, 4], [2, 1], [3, 5]] and b.refs == [1, 1, 1, 1, 1, 1, 0]
    # a page that all let go is free for the next call
    b = ocache.Books([[0, 1], [2, 1]], [16, 16], [1, 2, 1, 0, 0], 16)
    assert b.reserve([1, 1]) == ([-1] * 2, [-1] * 2)
    assert b.table == [[0, 3], [2, 4]] and b.refs == [1, 0, 1, 1, 1]
    assert ocache.Books([[0, 1], [2, 1]], [16, 16], [1, 2, 1, 0], 16).reserve([1, 1]) is None


def test_books_by_hand_where_entries_are_missing_behind_the_length():
    # a sequence whose first pages were let go starts again: the holes are filled where they are
    b = ocache.Books([[-1, -1, 4, -1, 2]], [70], [0, 0, 1, 0, 1, 0, 0], 16)
    b.lens = [0]
    assert b.reserve([80]) == ([-1], [-1])
    assert b.table == [[0, 1, 4, 3, 2]] and b.refs == [1, 1, 1, 1, 1, 0, 0]


def test_quantise_marks_rows_whose_largest_code_would_overflow():
    v = np.full((3, 64), 3.30e38, np.float32)
    v[:, 0] = 3.4028235e38, 3.35e38, 3.30e38
    c, s, z = ocache.quantise(v)
    assert np.isnan(s[0]) and np.isnan(z[0]) and not c[0].any()
    assert np.isfinite(s[1:]).all() and np.isfinite(c[1:] * s[1:, None] + z[1:, None]).all()
