"""The decoder cache on the GPU against its 64-bit oracle.

Bits, codes, scales and books have to be equal.  Attention is compared within
    |err| <= (kept / 4 + 64) 2^-23 sum p (|c s| + |z|)
per element: p carries at most 64 units of 2^-23 (the argument of exp up to 23
in size and rounded once, exp to 2 units, a sum of at most 129 levels, one
division), the products and the sum over at most a quarter of the kept tokens
in one running fp32 value (four or more partial sums) the rest.  Where values
are whole numbers and all weights equal, a wrong kept token shows as a whole
count (test_kept_sets).
"""
import math

import numpy as np
import pytest
import torch

import oracle
from oracle import cache as ocache

pytestmark = pytest.mark.gpu
I = torch.int32
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def cache():
    from sparse_attention_sigma_b200 import cache as _cache
    return _cache


def ints(x):
    return torch.tensor(x, dtype=I, device="cuda")


def status():
    return torch.zeros(1, dtype=I, device="cuda")


def flags(st):
    return int(st.item())


INVALID, BAD_SIGMA, NO_PAGES = 1 << 1, 1 << 5, 1 << 7


class Filled:
    """A pool and books of sequences of the given lengths, filled by had_cache_append, and the
    oracle's view of the same tokens."""

    def __init__(self, cache, lens, H, d, page, dtype=BF16, seed=0, values=None, same_keys=False,
                 spare=2):
        g = torch.Generator().manual_seed(seed)
        B, T = len(lens), max(max(lens), 1)
        self.d, self.page, self.lens = d, page, lens
        self.k = torch.randn(B, H, T, d, generator=g).to(dtype)
        if same_keys:
            self.k[:, :, 1:] = self.k[:, :, :1]
        v = torch.randn(B, H, T, d, generator=g) if values is None else values(B, H, T, d)
        self.v = v.to(dtype)
        self.sigma = 0.5 + torch.rand(H, generator=g)
        width = -(-T // page) + 1
        need = [-(-n // page) for n in lens]
        order = torch.randperm(sum(need) + spare, generator=g).to(I)
        self.table = torch.full((B, width), -1, dtype=I)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.refs = torch.zeros(order.numel(), dtype=I)
        self.refs[order[:at].long()] = 1
        self.table, self.refs = self.table.cuda(), self.refs.cuda()
        self.cache = cache.Cache.empty(order.numel(), H, page, d)
        # what was there before shows wherever a kernel reads a place it should not
        self.cache.kbits.fill_(-1)
        self.cache.vcodes.fill_(255)
        self.cache.vscale.fill_(float("nan"))
        st = status()
        cache.had_cache_append(self.k.cuda(), self.v.cuda(), self.sigma.cuda(), self.cache,
                               self.table, ints([0] * B), counts=ints(lens), dev_status=st)
        assert flags(st) == 0
        self.sk = np.where(self.k.float().numpy() / self.sigma.numpy()[None, :, None, None] < 0,
                           -1, 1)
        self.codes, self.scale, self.zero = ocache.quantise(self.v.float().numpy())

    def rows(self, q, sigma_q, lens, counts, N, tau, window, sinks):
        """(out, bound) of the oracle for queries q [B, Hq, T, d]."""
        B, Hq, T, d = q.shape
        G = Hq // self.sk.shape[1]
        sq = np.where(q.float().numpy() / sigma_q.numpy()[None, :, None, None] < 0, -1, 1)
        out, bound = np.zeros(q.shape), np.zeros(q.shape)
        for b in range(B):
            for h in range(Hq):
                for t in range(counts[b]):
                    o, kept, size = ocache.attend(
                        sq[b, h, t], self.sk[b, h // G], self.codes[b, h // G],
                        self.scale[b, h // G], self.zero[b, h // G], N, np.float32(tau), window,
                        sinks, lens[b] - counts[b] + t)
                    out[b, h, t] = o
                    bound[b, h, t] = (kept.size / 4 + 64) * 2.0 ** -23 * size
        return out, bound


def queries(B, Hq, T, d, dtype, seed=99):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(B, Hq, T, d, generator=g).to(dtype), 0.5 + torch.rand(Hq, generator=g)


# ------------------------------------------------------------- append and read

@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,page,T,start,counts", [
    (1, 1, 16, 1, [0], None),
    (3, 2, 16, 1, [15, 16, 33], None),
    (3, 5, 32, 77, [5, 0, 31], [77, 0, 3]),
    (2, 3, 256, 300, [255, 1], [300, 299]),
    (2, 1, 64, 129, [0, 64], None),
])
def test_append_and_read_back(cache, dtype, d, B, H, page, T, start, counts):
    g = torch.Generator().manual_seed(T + d)
    k, v = (torch.randn(B, H, T, d, generator=g).to(dtype) for _ in range(2))
    sigma = 0.5 + torch.rand(H, generator=g)
    width = max(-(-(s + T) // page) for s in start)
    table = torch.randperm(B * width, generator=g).to(I).reshape(B, width).cuda()
    c = cache.Cache.empty(B * width, H, page, d)
    c.vscale.fill_(7.0)
    st = status()
    cnt = None if counts is None else ints(counts)
    cache.had_cache_append(k.cuda(), v.cuda(), sigma.cuda(), c, table, ints(start), counts=cnt,
                           dev_status=st)
    bits, values = cache.had_cache_read(c, table, ints(start), T, counts=cnt, dev_status=st)
    assert flags(st) == 0
    real = np.arange(T)[None] < np.array(counts or [T] * B)[:, None]
    signs = np.where(k.float().numpy() / sigma.numpy()[None, :, None, None] < 0, -1, 1)
    want = np.where(real[:, None, :, None], oracle.pack(signs).view(np.int32), 0)
    assert np.array_equal(bits.cpu().numpy(), want)
    code, s, z = ocache.quantise(v.float().numpy())
    exact = code * s[..., None].astype(np.float64) + z[..., None]     # 4 + 8 bits and a bf16: exact
    exact = np.where(real[:, None, :, None], exact, 0).astype(np.float32)
    assert np.array_equal(values.cpu().numpy(), exact)
    # nothing but the written places changed
    touched = torch.zeros(B * width, page, dtype=torch.bool)
    for b in range(B):
        for t in range(T):
            if real[b, t]:
                touched[table[b, (start[b] + t) // page].item(), (start[b] + t) % page] = True
    rest = ~touched[:, None, :].expand(-1, H, -1).cuda()
    assert not c.kbits[rest].any() and not c.vcodes[rest].any()
    assert (c.vscale[rest] == 7.0).all()


def test_append_of_special_rows(cache):
    """Constants, signed zeros, tiny and huge ranges, NaN and infinities; signs of -0, NaN and a
    quotient that underflows."""
    d = 64
    v = torch.zeros(1, 1, 12, d)
    v[0, 0, 1] = -0.0
    v[0, 0, 2] = 0.1
    v[0, 0, 3] = torch.linspace(-1e-40, 1e-40, d)
    v[0, 0, 4] = torch.linspace(-1.6e38, 1.6e38, d)
    v[0, 0, 5] = torch.linspace(-3.0e38, 3.0e38, d)             # the range passes fp32
    v[0, 0, 6, 3] = float("nan")
    v[0, 0, 7, 63] = float("inf")
    v[0, 0, 8, 0] = -float("inf")
    v[0, 0, 9] = torch.arange(d) * 2.0 ** -149
    v[0, 0, 10] = 1.0 + torch.arange(d) * 2.0 ** -23
    v[0, 0, 11] = -3.4e38                                        # no bf16 at or below it
    k = torch.zeros(1, 1, 12, d)
    k[0, 0, 0] = -0.0
    k[0, 0, 1] = float("nan")
    k[0, 0, 2] = -1e-45
    k[0, 0, 3] = -float("inf")
    c = cache.Cache.empty(1, 1, 16, d)
    st = status()
    cache.had_cache_append(k.cuda(), v.cuda(), torch.full((1,), 4.0, device="cuda"), c, ints([[0]]),
                           ints([0]), dev_status=st)
    code, s, z = ocache.quantise(v.numpy())
    got = c.vcodes.cpu().numpy()[0, 0, :12]
    assert np.array_equal(np.stack([got & 15, got >> 4], -1).reshape(12, d), code[0, 0])
    got = c.vscale.float().cpu().numpy()[0, 0, :12]
    assert np.array_equal(got[:, 0], s[0, 0], equal_nan=True)
    assert np.array_equal(got[:, 1], z[0, 0], equal_nan=True)
    assert np.isnan(s[0, 0, [5, 6, 7, 8, 11]]).all() and np.isfinite(s[0, 0, [0, 1, 2, 3, 4, 9, 10]]).all()
    assert c.kbits[0, 0, :4].cpu().tolist() == [[0, 0], [0, 0], [0, 0], [-1, -1]]
    assert flags(st) == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
def test_codes_of_many_rows_are_those_of_the_ieee_quotient(cache, dtype, d):
    """Quotients beside and on a half: rows of few bits, of whole multiples of half a step, of any
    magnitude down to subnormal scales."""
    g = torch.Generator().manual_seed(d)
    T = 16384
    v = torch.randn(1, 1, T, d, generator=g)
    kind = torch.arange(T)[:, None] % 4
    v = torch.where(kind == 1, (v * 8).round() / 8, v)
    half = torch.randint(0, 31, (T, d), generator=g) * 0.5
    half[:, 0], half[:, 1] = 0, 15
    v = torch.where(kind == 2, half * (1 + torch.randint(0, 128, (T, 1), generator=g) / 128), v)
    v = torch.where(kind == 3, v * 2.0 ** torch.randint(-148, 120, (T, 1), generator=g), v).to(dtype)
    c = cache.Cache.empty(T // 256, 1, 256, d)
    st = status()
    cache.had_cache_append(v.cuda(), v.cuda(), torch.ones(1, device="cuda"), c,
                           torch.arange(T // 256, dtype=I, device="cuda")[None], ints([0]),
                           dev_status=st)
    code, s, z = ocache.quantise(v.float().numpy()[0, 0])
    got = c.vcodes.cpu().numpy().reshape(T, d // 2)
    assert np.array_equal(np.stack([got & 15, got >> 4], -1).reshape(T, d), code)
    got = c.vscale.float().cpu().numpy().reshape(T, 2)
    assert np.array_equal(got[:, 0], s, equal_nan=True) and np.array_equal(got[:, 1], z, equal_nan=True)
    assert flags(st) == 0


def test_append_flags_what_it_cannot_place(cache):
    k = torch.randn(4, 1, 2, 64, device="cuda")
    c = cache.Cache.empty(2, 1, 16, 64)
    table = ints([[0, -1], [1, 2], [1, 1], [0, 1]])
    for start, counts, sigma, want in (
            ([15, 0, 0, 0], [2, 0, 0, 0], 1.0, INVALID),         # behind the sequence's pages
            ([0, 15, 0, 0], [0, 2, 0, 0], 1.0, INVALID),         # a page the pool lacks
            ([0, 0, 31, 0], [0, 0, 2, 0], 1.0, INVALID),         # behind the table
            ([0, 0, 0, -1], [0, 0, 0, 2], 1.0, INVALID),
            ([0, 0, 0, 0], [3, 0, 0, 0], 1.0, INVALID),          # more than T
            ([0, 0, 0, 0], [-1, 0, 0, 0], 1.0, INVALID),
            ([0, 0, 0, 0], [0, 0, 0, 0], 1.0, 0),
            ([0, 0, 0, 0], [0, 0, 0, 2], 0.0, BAD_SIGMA)):
        st = status()
        cache.had_cache_append(k, k, torch.full((1,), sigma, device="cuda"), c, table, ints(start),
                               counts=ints(counts), dev_status=st)
        assert flags(st) == want, (start, counts)
        if sigma:
            st = status()
            cache.had_cache_read(c, table, ints(start), 2, counts=ints(counts), dev_status=st)
            assert flags(st) == want


# ------------------------------------------------------------------- attention

ATTEND = [
    # lens, Hq, Hkv, d, page, T, counts, N, window, sinks, dtype
    ([1], 1, 1, 64, 16, 1, None, 1, 0, 0, BF16),
    ([128], 2, 2, 64, 16, 1, None, 16, 0, 0, F32),
    ([33, 0, 17], 4, 2, 128, 16, 1, None, 5, 0, 0, BF16),
    ([300, 299, 1], 5, 1, 64, 32, 1, None, 1000, 0, 0, F32),
    ([700], 6, 1, 128, 64, 1, None, 100, 0, 0, BF16),
    ([1030, 515], 16, 2, 64, 128, 1, None, 64, 0, 0, BF16),
    ([2500], 3, 3, 64, 256, 1, None, 2499, 0, 0, F32),
    ([600, 40, 39], 8, 8, 128, 64, 1, None, 50, 40, 4, BF16),
    ([100], 1, 1, 64, 16, 1, None, 3, 1, 0, F32),
    ([100], 1, 1, 64, 16, 1, None, 3, 1, 33, F32),
    ([70, 200], 2, 1, 64, 32, 1, None, 500, 64, 300, BF16),
    ([50, 3, 0, 5], 4, 2, 64, 16, 5, [5, 4, 0, 5], 7, 0, 0, F32),
    ([2, 1], 2, 2, 128, 16, 4, None, 3, 0, 0, BF16),             # more queries than tokens
    ([65], 3, 1, 64, 64, 65, None, 9, 0, 0, BF16),
    ([200, 130], 4, 2, 128, 32, 37, [37, 20], 300, 0, 0, F32),
    ([333], 10, 2, 64, 32, 60, None, 20, 31, 5, BF16),
    ([260], 7, 1, 64, 128, 33, None, 16, 100, 0, F32),
    ([150], 11, 1, 128, 16, 3, None, 33, 20, 1, BF16),
]


@pytest.mark.parametrize("case", ATTEND, ids=lambda c: "-".join(map(str, c[:-1])).replace(" ", ""))
def test_attention(cache, case):
    lens, Hq, H, d, page, T, counts, N, window, sinks, dtype = case
    f = Filled(cache, lens, H, d, page, dtype, seed=sum(lens) + d)
    q, sigma_q = queries(len(lens), Hq, T, d, dtype)
    tau = 1 / math.sqrt(d)
    st = status()
    out = cache.had_cache_attention(q.cuda(), sigma_q.cuda(), f.cache, f.table, ints(lens), N, tau,
                                    window=window, sinks=sinks,
                                    counts=None if counts is None else ints(counts), dev_status=st)
    assert flags(st) == 0
    want, bound = f.rows(q, sigma_q, lens, counts or [T] * len(lens), N, tau, window, sinks)
    err = np.abs(out.cpu().numpy() - want)
    assert (err <= bound).all(), (err - bound).max()


def _marks(B, H, T, d):
    """Values of which element e is 15 where token j has j mod d = e, else 0: codes 15 and 0,
    scale 1, zero point 0."""
    v = torch.zeros(B, H, T, d)
    j = torch.arange(T)
    v[:, :, j, j % d] = 15.0
    return v


@pytest.mark.parametrize("lens,G,T,N,window,sinks,same", [
    ([100], 1, 1, 50, 0, 0, True),               # one level: ties only, the lowest indices win
    ([1000], 4, 1, 333, 0, 0, True),
    ([5000], 3, 1, 1234, 0, 0, True),
    ([5000], 8, 1, 777, 0, 0, False),
    ([900, 31], 2, 9, 200, 0, 0, False),
    ([900, 310], 4, 50, 100, 333, 7, True),
    ([20000], 1, 1, 9000, 0, 0, False),
    ([9000], 5, 2, 4000, 6000, 100, False),
])
@pytest.mark.parametrize("d", [64, 128])
def test_kept_sets(cache, d, lens, G, T, N, window, sinks, same):
    """With tau 0 every kept token weighs 1 / n, so n out[e] counts the kept tokens of each
    residue: exact sets, ties included."""
    f = Filled(cache, lens, 1, d, 64, F32, seed=G + N, values=_marks, same_keys=same)
    q, sigma_q = queries(len(lens), G, T, d, F32)
    st = status()
    out = cache.had_cache_attention(q.cuda(), sigma_q.cuda(), f.cache, f.table, ints(lens), N, 0.0,
                                    window=window, sinks=sinks, dev_status=st).cpu().numpy()
    assert flags(st) == 0
    sq = np.where(q.numpy() / sigma_q.numpy()[None, :, None, None] < 0, -1, 1)
    for b, n in enumerate(lens):
        for h in range(G):
            for t in range(T):
                _, kept, _ = ocache.attend(sq[b, h, t], f.sk[b, 0], f.codes[b, 0], f.scale[b, 0],
                                           f.zero[b, 0], N, 0.0, window, sinks, n - T + t)
                count = np.bincount(kept % d, minlength=d)
                got = out[b, h, t] * kept.size / 15
                assert np.array_equal(np.rint(got), count)
                assert np.abs(got - count).max() < 0.01


@pytest.mark.parametrize("d,n,G,T,N,window", [
    (64, 45000, 1, 1, 700, 0),                   # a CTA's slice passes its shared memory
    (128, 23000, 8, 1, 5000, 0),
    (64, 46000, 3, 1, 46000, 44000),
])
def test_long_contexts(cache, d, n, G, T, N, window):
    f = Filled(cache, [n, n // 2], 1, d, 256, BF16, seed=n)
    q, sigma_q = queries(2, G, T, d, BF16)
    st = status()
    out = cache.had_cache_attention(q.cuda(), sigma_q.cuda(), f.cache, f.table, ints(f.lens), N,
                                    0.1, window=window, sinks=5, dev_status=st)
    assert flags(st) == 0
    want, bound = f.rows(q, sigma_q, f.lens, [T, T], N, 0.1, window, 5)
    assert (np.abs(out.cpu().numpy() - want) <= bound).all()


@pytest.mark.parametrize("longest", [513, 600, 1040, 1100, 2064, 2784])
@pytest.mark.parametrize("G,d", [(1, 64), (7, 128)])
def test_lengths_about_what_a_cta_holds(cache, longest, G, d):
    """A launch for the longest sequence splits it over CTAs that hold little more than their part;
    shorter sequences beside it use fewer of them."""
    lens = [longest, 512, 500, 400, 385, 384, 383, 300, 257, 256, longest // 2, longest // 2 + 1]
    f = Filled(cache, lens, 1, d, 16, BF16, seed=longest)
    q, sigma_q = queries(len(lens), G, 1, d, BF16)
    st = status()
    table = f.table[:, :-(-longest // 16)].contiguous()
    out = cache.had_cache_attention(q.cuda(), sigma_q.cuda(), f.cache, table, ints(lens), 200, 0.1,
                                    dev_status=st)
    assert flags(st) == 0
    want, bound = f.rows(q, sigma_q, lens, [1] * len(lens), 200, 0.1, 0, 0)
    assert (np.abs(out.cpu().numpy() - want) <= bound).all()


@pytest.mark.parametrize("lens,H,G,T,d,N,window", [
    ([2100, 0, 700, 1], 2, 2, 1, 64, 90, 0), ([5000, 300], 1, 3, 2, 128, 400, 0),
    ([6000, 900, 37], 2, 8, 1, 128, 100, 0), ([3000, 12000], 1, 1, 1, 64, 5000, 0),
    ([3000, 250], 1, 4, 9, 64, 50, 2000)])
def test_tables_much_wider_than_their_sequences(cache, lens, H, G, T, d, N, window):
    """The launch is made for as many keys as a table row may hold, the work for those that are
    there."""
    f = Filled(cache, lens, H, d, 16, BF16, seed=sum(lens))
    q, sigma_q = queries(len(lens), H * G, T, d, BF16)
    want, bound = f.rows(q, sigma_q, lens, [T] * len(lens), N, 0.1, window, 4)
    for width in (1000, 70000):
        table = torch.full((len(lens), width), -1, dtype=I, device="cuda")
        table[:, :f.table.shape[1]] = f.table
        st = status()
        for max_len in (0, max(lens), 1, 2 ** 31 - 1):           # a hint, right or wrong
            out = cache.had_cache_attention(q.cuda(), sigma_q.cuda(), f.cache, table, ints(lens),
                                            N, 0.1, window=window, sinks=4, dev_status=st,
                                            max_len=max_len)
            assert flags(st) == 0
            assert (np.abs(out.cpu().numpy() - want) <= bound).all()


@pytest.mark.parametrize("B,H,G,T,d,n,window", [
    (16, 16, 1, 80, 64, 90, 0), (35, 61, 3, 1, 128, 50, 20), (16, 17, 2, 32, 128, 70, 33),
    (40, 53, 1, 3, 64, 40, 0)])
def test_many_short_tiles(cache, B, H, G, T, d, n, window):
    """More tiles than the card has places for warps."""
    g = np.random.default_rng(B)
    lens = [int(x) for x in g.integers(0, n, B)]
    lens[0] = n
    f = Filled(cache, lens, H, d, 32, BF16, seed=B)
    q, sigma_q = queries(B, G * H, T, d, BF16)
    st = status()
    out = cache.had_cache_attention(q.cuda(), sigma_q.cuda(), f.cache, f.table, ints(lens), 11, 0.1,
                                    window=window, sinks=3, dev_status=st).cpu().numpy()
    assert flags(st) == 0
    # (every seventh head: the oracle goes row by row)
    for h in range(0, G * H, 7):
        sq = np.where(q[:, h].float().numpy() / sigma_q[h].item() < 0, -1, 1)
        for b in range(B):
            for t in range(T):
                o, kept, size = ocache.attend(
                    sq[b, t], f.sk[b, h // G], f.codes[b, h // G], f.scale[b, h // G],
                    f.zero[b, h // G], 11, np.float32(0.1), window, 3, lens[b] - T + t)
                err = np.abs(out[b, h, t] - o)
                assert (err <= (kept.size / 4 + 64) * 2.0 ** -23 * size).all()


def test_pools_beyond_32_bit_offsets(cache):
    """The last pages of a pool of 5 GB: byte offsets of codes and bits pass 2^32."""
    page, H, d, n = 256, 8, 128, 700
    P = 2 ** 32 // (page * H * d // 2) + 300
    make = lambda *s, dtype: torch.empty(*s, dtype=dtype, device="cuda")      # noqa: E731
    c = cache.Cache(make(P, H, page, d // 32, dtype=I), make(P, H, page, d // 2, dtype=torch.uint8),
                    make(P, H, page, 2, dtype=BF16))
    f = Filled(cache, [n], H, d, page, BF16, seed=1)
    table = ints([[P - 1, P - 200, P - 7]])
    st = status()
    cache.had_cache_append(f.k.cuda(), f.v.cuda(), f.sigma.cuda(), c, table, ints([0]), dev_status=st)
    got, want = (cache.had_cache_read(x, t, ints([0]), n, dev_status=st)
                 for x, t in ((c, table), (f.cache, f.table)))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    q, sigma_q = (x.cuda() for x in queries(1, 16, 1, d, BF16))
    args = ints([n]), 100, 0.1
    want = cache.had_cache_attention(q, sigma_q, f.cache, f.table, *args, dev_status=st)
    assert torch.equal(want, cache.had_cache_attention(q, sigma_q, c, table, *args, dev_status=st))
    cache.had_cache_copy_pages(c, table[0], ints([3, 1, 0]), dev_status=st)
    assert torch.equal(want, cache.had_cache_attention(q, sigma_q, c, ints([[3, 1, 0]]), *args,
                                                       dev_status=st))
    assert flags(st) == 0


def test_values_of_any_size_keep_their_weight(cache):
    """Tokens whose scales differ by 60 orders of magnitude: each output element is as exact as
    its own sum allows."""
    def values(B, H, T, d):
        g = torch.Generator().manual_seed(4)
        return torch.randn(B, H, T, d, generator=g) * 10.0 ** torch.randint(-30, 31, (B, H, T, 1),
                                                                             generator=g)
    f = Filled(cache, [400], 2, 64, 32, F32, values=values)
    q, sigma_q = queries(1, 4, 1, 64, F32)
    out = cache.had_cache_attention(q.cuda(), sigma_q.cuda(), f.cache, f.table, ints([400]), 60, 0.5)
    want, bound = f.rows(q, sigma_q, [400], [1], 60, 0.5, 0, 0)
    assert (np.abs(out.cpu().numpy() - want) <= bound).all()


@pytest.mark.parametrize("tau", [0.0, 3.0, 1e30])
def test_temperatures(cache, tau):
    f = Filled(cache, [300], 1, 64, 16, F32)
    q, sigma_q = queries(1, 2, 1, 64, F32)
    out = cache.had_cache_attention(q.cuda(), sigma_q.cuda(), f.cache, f.table, ints([300]), 40, tau)
    want, bound = f.rows(q, sigma_q, [300], [1], 40, tau, 0, 0)
    # exp's argument reaches 128 tau: its rounding is 128 tau 2^-24 relative where it matters
    assert (np.abs(out.cpu().numpy() - want) <= bound * (1 + min(tau, 10.0))).all()


def test_rows_that_keep_an_unholdable_value_are_nan_and_no_others(cache):
    def values(B, H, T, d):
        v = torch.ones(B, H, T, d)
        v[0, 0, 10, 5] = float("nan")
        return v
    f = Filled(cache, [64], 2, 64, 16, F32, values=values)
    q, sigma_q = queries(1, 4, 64, 64, F32)
    out = cache.had_cache_attention(q.cuda(), sigma_q.cuda(), f.cache, f.table, ints([64]), 8, 0.1)
    want, _ = f.rows(q, sigma_q, [64], [64], 8, 0.1, 0, 0)
    got = out.cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.isnan(got).any() and not np.isnan(got[:, 2:]).any()
    assert np.abs(got[~np.isnan(got)][np.nonzero(got[~np.isnan(got)])] - 1).max() < 1e-5


def test_attention_flags_bad_books(cache):
    f = Filled(cache, [100, 100], 1, 64, 16, F32)
    q, sigma_q = queries(2, 1, 2, 64, F32)
    args = q.cuda(), sigma_q.cuda(), f.cache

    def run(table, lens, counts=None, sigma=None):
        st = status()
        out = cache.had_cache_attention(args[0], args[1] if sigma is None else sigma, args[2],
                                        table, ints(lens), 5, 0.1, dev_status=st,
                                        counts=None if counts is None else ints(counts))
        return flags(st), out

    clean = run(f.table, [100, 100])
    assert clean[0] == 0
    for page in (-1, -7, f.cache.pages, 2 ** 31 - 1):
        t = f.table.clone()
        t[0, 3] = page
        flag, out = run(t, [100, 100])
        assert flag == INVALID and torch.equal(out[1], clean[1][1])
    for lens, counts in (([-1, 100], None), ([f.table.shape[1] * 16 + 1, 100], None),
                         ([100, 100], [3, 2]), ([100, 100], [-1, 2])):
        flag, out = run(f.table, lens, counts)
        assert flag == INVALID and not out[0].any() and torch.equal(out[1], clean[1][1])
    flag, _ = run(f.table, [100, 100], sigma=torch.full((1,), -1.0, device="cuda"))
    assert flag == BAD_SIGMA


def test_padded_rows_are_zero_and_evicted_pages_are_not_read(cache):
    """Under a window the pages before it may be gone; rows behind a count get zeros."""
    W, S, n = 40, 5, 400
    f = Filled(cache, [n], 2, 64, 16, BF16)
    q, sigma_q = queries(1, 4, 3, 64, BF16)
    run = lambda table, st: cache.had_cache_attention(                    # noqa: E731
        q[:, :, :2].contiguous().cuda(), sigma_q.cuda(), f.cache, table, ints([n]), 16, 0.1,
        window=W, sinks=S, counts=ints([1]), dev_status=st)
    st = status()
    before = run(f.table, st)
    table = f.table.clone()
    cache.had_cache_evict(table, ints([n]), f.refs, 16, W, S)
    assert (table == -1).sum() > (f.table == -1).sum() + 10
    after = run(table, st)
    assert flags(st) == 0 and torch.equal(before, after)
    assert not after[:, :, 1].any() and after[:, :, 0].any()


# --------------------------------------------------------------- pages' books

def _same_books(table, lens, refs, b):
    t, n, r = b.arrays()
    assert np.array_equal(table.cpu().numpy(), t)
    assert np.array_equal(lens.cpu().numpy(), n)
    assert np.array_equal(refs.cpu().numpy(), r)


@pytest.mark.parametrize("S,width,P,page,seed", [
    (1, 3, 5, 16, 0), (5, 9, 40, 16, 1), (7, 5, 30, 256, 2), (64, 40, 1500, 64, 3),
    (33, 70, 900, 32, 4), (3, 1, 3, 128, 5)])
def test_books_through_a_run(cache, S, width, P, page, seed):
    """Forks, growth, eviction, departures and compactions in turn, as a beam server has them."""
    g = np.random.default_rng(seed)
    table, lens, refs = cache.empty_books(S, width, P)
    b = ocache.Books(table, lens, refs, page)
    st = status()
    full = 0
    for step in range(30):
        grow = g.integers(0, max(2, width * page // 6), S) * (g.random(S) < 0.7)
        grow = np.minimum(grow, width * page - np.array(b.lens))
        src, dst = cache.had_cache_reserve(table, lens, refs, page, ints(grow.tolist()),
                                           dev_status=st)
        want = b.reserve(grow.tolist())
        if want is None:
            assert flags(st) == NO_PAGES
            st.zero_()
            full += 1
            want = [-1] * S, [-1] * S
        else:
            lens += ints(grow.tolist())
            b.lens = [n + int(x) for n, x in zip(b.lens, grow)]
        assert src.tolist() == want[0] and dst.tolist() == want[1]
        _same_books(table, lens, refs, b)
        n = int(g.integers(0, S + 1))
        to = g.permutation(S)[:n]
        frm = g.integers(0, S, n)
        cache.had_cache_fork(table, lens, refs, page, ints(frm.tolist()), ints(to.tolist()),
                             dev_status=st)
        b.fork(frm.tolist(), to.tolist())
        _same_books(table, lens, refs, b)
        if step % 3 == 1:
            W, sinks = int(g.integers(1, width * page)), int(g.integers(0, 2 * page))
            cache.had_cache_evict(table, lens, refs, page, W, sinks, dev_status=st)
            b.evict(W, sinks)
        if step % 4 == 2 or full:
            full = 0
            gone = g.integers(0, S, S // 2 + 1)                   # some listed twice
            cache.had_cache_free(table, lens, refs, ints(gone.tolist()), dev_status=st)
            b.free(gone.tolist())
            _same_books(table, lens, refs, b)
            src, dst, live = cache.had_cache_compact(table, refs, dev_status=st)
            want = b.compact()
            assert (src.tolist(), dst.tolist(), live.item()) == want
        _same_books(table, lens, refs, b)
        assert flags(st) == 0
        counted = np.bincount(table[table >= 0].cpu().numpy(), minlength=P)
        assert np.array_equal(counted, refs.cpu().numpy())


@pytest.mark.parametrize("S,width,P", [(3000, 20, 70001), (8192, 7, 60000)])
def test_books_of_a_large_pool(cache, S, width, P):
    """More pages and sequences than one pass of a CTA over them covers, up to the most there may
    be."""
    page = 16
    g = np.random.default_rng(11)
    table, lens, refs = cache.empty_books(S, width, P)
    b = ocache.Books(table, lens, refs, page)
    grow = g.integers(0, width * page - 40, S)
    cache.had_cache_reserve(table, lens, refs, page, ints(grow.tolist()))
    b.reserve(grow.tolist())
    lens += ints(grow.tolist())
    b.lens = grow.tolist()
    to = g.permutation(S)[:S // 2]
    frm = g.integers(0, S, to.size)
    cache.had_cache_fork(table, lens, refs, page, ints(frm.tolist()), ints(to.tolist()))
    b.fork(frm.tolist(), to.tolist())
    _same_books(table, lens, refs, b)
    src, dst = cache.had_cache_reserve(table, lens, refs, page, ints([1] * S))
    assert (src.tolist(), dst.tolist()) == b.reserve([1] * S)
    _same_books(table, lens, refs, b)
    gone = list(range(0, S, 3))
    cache.had_cache_free(table, lens, refs, ints(gone))
    b.free(gone)
    src, dst, live = cache.had_cache_compact(table, refs)
    assert (src.tolist(), dst.tolist(), live.item()) == b.compact()
    _same_books(table, lens, refs, b)


def test_books_refuse_and_stay_as_they_were(cache):
    page = 16
    table, lens, refs = ints([[0, 1, -1], [2, -1, -1]]), ints([20, 10]), ints([1, 1, 1, 0])
    start = [x.clone() for x in (table, lens, refs)]

    def unchanged(want, st):
        assert flags(st) == want
        assert all(torch.equal(a, x) for a, x in zip(start, (table, lens, refs)))
        st.zero_()

    st = status()
    for grow, want in (([40, 0], INVALID), ([-1, 1], INVALID), ([13, 20], NO_PAGES)):
        src, dst = cache.had_cache_reserve(table, lens, refs, page, ints(grow), dev_status=st)
        assert src.tolist() == dst.tolist() == [-1, -1]
        unchanged(want, st)
    for src, dst in (([0, 0], [1, 1]), ([2], [0]), ([0], [-1]), ([-1], [0]), ([0], [2])):
        cache.had_cache_fork(table, lens, refs, page, ints(src), ints(dst), dev_status=st)
        unchanged(INVALID, st)
    bad = lens.clone()
    bad[0] = 49
    cache.had_cache_fork(table, bad, refs, page, ints([0]), ints([1]), dev_status=st)
    unchanged(INVALID, st)
    src, dst = cache.had_cache_reserve(table, bad, refs, page, ints([0, 0]), dev_status=st)
    unchanged(INVALID, st)
    # the last page is not there
    hole = ints([[0, -1, -1], [2, -1, -1]])
    cache.had_cache_reserve(hole, lens, refs, page, ints([1, 0]), dev_status=st)
    assert hole.tolist() == [[0, -1, -1], [2, -1, -1]]
    unchanged(INVALID, st)
    cache.had_cache_free(table, lens, refs, ints([-1, 2]), dev_status=st)
    unchanged(INVALID, st)
    # names that are no pages are dropped by free and stay in compact
    wild = ints([[9, 1, -1], [2, -1, -1]])
    cache.had_cache_compact(wild, refs.clone(), dev_status=st)
    assert flags(st) == INVALID and wild.tolist() == [[9, 1, -1], [2, -1, -1]]
    st.zero_()
    r = refs.clone()
    cache.had_cache_free(wild, lens.clone(), r, ints([0]), dev_status=st)
    assert flags(st) == INVALID and r.tolist() == [1, 0, 1, 0] and wild[0].tolist() == [-1] * 3


@pytest.mark.parametrize("d,page,H", [(64, 16, 1), (128, 64, 3), (64, 256, 2)])
def test_copy_pages(cache, d, page, H):
    P = 40
    c = cache.Cache.empty(P, H, page, d)
    g = torch.Generator(device="cuda").manual_seed(1)
    for a in (c.kbits, c.vcodes, c.vscale.view(torch.int16)):
        a.copy_(torch.randint(-2 ** 15, 2 ** 15, a.shape, generator=g, device="cuda"))
    raw = [a.view(torch.uint8).reshape(P, -1).clone() for a in (c.kbits, c.vcodes, c.vscale)]
    src = [0, 3, 3, -1, 7, P, 9, -1] + [11] * 9
    dst = [20, 21, 22, 23, -1, 24, P, -1] + list(range(30, 39))
    st = status()
    cache.had_cache_copy_pages(c, ints(src), ints(dst), dev_status=st)
    assert flags(st) == INVALID
    want = [r.clone() for r in raw]
    for s, t in zip(src, dst):
        if 0 <= s < P and 0 <= t < P:
            for r, w in zip(raw, want):
                w[t] = r[s]
    for a, w in zip((c.kbits, c.vcodes, c.vscale), want):
        assert torch.equal(a.view(torch.uint8).reshape(P, -1), w)


# ------------------------------------------------------------- used together

def _decode(cache, steps, stream=None):
    """Two sequences of a prompt, forked into four that go on, d 64, window and sinks."""
    B, H, G, d, page, N, W, S = 4, 2, 3, 64, 16, 12, 48, 4
    g = torch.Generator().manual_seed(2)
    table, lens, refs = cache.empty_books(B, 10, 60)
    c = cache.Cache.empty(60, H, page, d)
    sk, sq = (0.5 + torch.rand(H, generator=g)).cuda(), (0.5 + torch.rand(G * H, generator=g)).cuda()
    hist_k = [torch.zeros(H, 0, d) for _ in range(B)]
    hist_v = [torch.zeros(H, 0, d) for _ in range(B)]
    st = status()

    def step(T, counts, Nq):
        k, v = (torch.randn(B, H, T, d, generator=g) for _ in range(2))
        q = torch.randn(B, G * H, T, d, generator=g)
        grow = ints(counts)
        src, dst = cache.had_cache_reserve(table, lens, refs, page, grow, dev_status=st,
                                           stream=stream)
        cache.had_cache_copy_pages(c, src, dst, dev_status=st, stream=stream)
        cache.had_cache_append(k.cuda(), v.cuda(), sk, c, table, lens, counts=grow, dev_status=st,
                               stream=stream)
        lens.add_(grow)
        out = cache.had_cache_attention(q.cuda(), sq, c, table, lens, Nq, 0.125, window=W, sinks=S,
                                        counts=grow, dev_status=st, stream=stream)
        cache.had_cache_evict(table, lens, refs, page, W, S, dev_status=st, stream=stream)
        worst = 0.0
        for b, n in enumerate(counts):
            hist_k[b] = torch.cat([hist_k[b], k[b, :, :n]], 1)
            hist_v[b] = torch.cat([hist_v[b], v[b, :, :n]], 1)
            code, s, z = ocache.quantise(hist_v[b].numpy())
            for h in range(G * H):
                signs = np.where(hist_k[b][h // G].numpy() / sk[h // G].item() < 0, -1, 1)
                for t in range(n):
                    row = np.where(q[b, h, t].numpy() / sq[h].item() < 0, -1, 1)
                    o, kept, size = ocache.attend(row, signs, code[h // G], s[h // G], z[h // G],
                                                  Nq, np.float32(0.125), W, S,
                                                  hist_k[b].shape[1] - n + t)
                    err = np.abs(out[b, h, t].cpu().numpy() - o)
                    worst = max(worst, (err / ((kept.size / 4 + 64) * 2.0 ** -23 * size)).max())
        assert worst <= 1 and flags(st) == 0

    step(70, [70, 33, 0, 0], 20)
    src, dst = [0, 1], [2, 3]
    cache.had_cache_fork(table, lens, refs, page, ints(src), ints(dst), dev_status=st, stream=stream)
    for s, t in zip(src, dst):
        hist_k[t], hist_v[t] = hist_k[s], hist_v[s]
    for i in range(steps):
        step(1, [1] * B, N)
        if i % 3 == 1:
            order = [1, 0, 0, 3] if i % 2 else [2, 1, 2, 0]
            cache.had_cache_fork(table, lens, refs, page, ints(order), ints(range(B)), dev_status=st,
                                 stream=stream)
            hist_k[:], hist_v[:] = [hist_k[o] for o in order], [hist_v[o] for o in order]
        if i == 5:
            cache.had_cache_free(table, lens, refs, ints([3]), dev_status=st, stream=stream)
            hist_k[3] = hist_v[3] = torch.zeros(H, 0, d)
            src, dst, live = cache.had_cache_compact(table, refs, dev_status=st, stream=stream)
            cache.had_cache_copy_pages(c, src, dst, dev_status=st, stream=stream)
            assert live.item() == torch.unique(table[table >= 0]).numel()
    step(4, [4, 3, 1, 0], N)
    counted = np.bincount(table[table >= 0].cpu().numpy(), minlength=60)
    assert np.array_equal(counted, refs.cpu().numpy())


def test_decoding_with_forks_growth_eviction_and_compaction(cache):
    _decode(cache, 12)


def test_calls_go_to_the_given_stream(cache):
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        _decode(cache, 4, stream=s)


def test_a_chunked_prompt_is_the_causal_forward(cache):
    """A prompt in three chunks through the cache against had_attention_causal_fwd on the values
    that the cache holds, within that call's tolerance."""
    from sparse_attention_sigma_b200 import had
    B, H, n, d, N, tau = 2, 3, 300, 64, 40, 0.125
    f = Filled(cache, [n] * B, H, d, 64, F32, seed=8)
    q, sigma_q = queries(B, H, n, d, F32)
    _, values = cache.had_cache_read(f.cache, f.table, ints([0] * B), n)
    want = had.had_attention_causal_fwd(q.cuda(), f.k.cuda(), values, sigma_q.cuda(),
                                        f.sigma.cuda(), N, tau)
    at = 0
    for chunk in (100, 1, 199):
        out = cache.had_cache_attention(q[:, :, at:at + chunk].contiguous().cuda(), sigma_q.cuda(),
                                        f.cache, f.table, ints([at + chunk] * B), N, tau)
        assert (out - want[:, :, at:at + chunk]).abs().max() <= 2e-3
        at += chunk


def test_a_captured_step_replays_on_new_contents(cache):
    """reserve, copy, append and attend in one graph: replays go on where the books stand, two
    graphs of the same shapes side by side."""
    H, G, d, page, N = 2, 2, 64, 16, 9
    runs = []
    for seed in (0, 1):
        f = Filled(cache, [30, 47], H, d, page, F32, seed=seed, spare=20)
        lens, grow = ints(f.lens), ints([1, 1])
        table = torch.full((2, 8), -1, dtype=I, device="cuda")
        table[:, :f.table.shape[1]] = f.table
        k, v = (torch.zeros(2, H, 1, d, device="cuda") for _ in range(2))
        q, sq = torch.zeros(2, G * H, 1, d, device="cuda"), torch.ones(G * H, device="cuda")
        sk = f.sigma.cuda()
        st = status()

        def step():
            src, dst = cache.had_cache_reserve(table, lens, f.refs, page, grow, dev_status=st)
            cache.had_cache_copy_pages(f.cache, src, dst, dev_status=st)
            cache.had_cache_append(k, v, sk, f.cache, table, lens, dev_status=st)
            lens.add_(grow)
            return cache.had_cache_attention(q, sq, f.cache, table, lens, N, 0.125, dev_status=st)

        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        runs.append((f, graph, k, v, q, out, st, lens, [f.k, f.v], (table, grow, sq, sk)))
    g = torch.Generator().manual_seed(5)
    for _ in range(20):
        for f, graph, k, v, q, out, st, lens, hist, _ in runs:
            for x in (k, v, q):
                x.copy_(torch.randn(x.shape, generator=g))
            graph.replay()
            if hist[0].shape[2] < lens.max().item():
                hist[:] = [torch.cat([h, torch.zeros(2, H, 1, d)], 2) for h in hist]
            for b, n in enumerate(lens.tolist()):
                hist[0][b, :, n - 1], hist[1][b, :, n - 1] = k[b, :, 0].cpu(), v[b, :, 0].cpu()
            assert flags(st) == 0
            f.sk = np.where(hist[0].numpy() / f.sigma.numpy()[None, :, None, None] < 0, -1, 1)
            f.codes, f.scale, f.zero = ocache.quantise(hist[1].numpy())
            want, bound = f.rows(q.cpu(), torch.ones(G * H), lens.tolist(), [1, 1], N, 0.125, 0, 0)
            assert (np.abs(out.cpu().numpy() - want) <= bound).all()


def test_results_do_not_depend_on_the_run(cache):
    f = Filled(cache, [3000, 2000], 2, 128, 64, BF16)
    q, sigma_q = queries(2, 8, 2, 128, BF16)
    run = lambda: cache.had_cache_attention(q.cuda(), sigma_q.cuda(), f.cache, f.table,  # noqa: E731
                                            ints([3000, 2000]), 500, 0.1)
    first = run()
    assert all(torch.equal(first, run()) for _ in range(5))


def test_refusals_of_the_binding(cache):
    f = Filled(cache, [20], 2, 64, 16, F32)
    q, s = torch.zeros(1, 4, 1, 64, device="cuda"), torch.ones(4, device="cuda")
    ok = dict(q=q, sigma_q=s, cache=f.cache, table=f.table, lens=ints([20]), N=4, tau=0.1)
    cache.had_cache_attention(**ok)
    for change, error in (
            (dict(q=q.half()), TypeError), (dict(q=q.transpose(1, 2)), ValueError),
            (dict(q=q[..., :32].contiguous()), ValueError), (dict(q=q[0]), ValueError),
            (dict(sigma_q=s[:2]), ValueError), (dict(sigma_q=s.double()), TypeError),
            (dict(table=f.table.long()), TypeError), (dict(table=f.table[0]), ValueError),
            (dict(table=f.table.repeat(2, 1)), ValueError), (dict(lens=ints([20, 20])), ValueError),
            (dict(lens=torch.tensor([20], device="cuda")), TypeError),
            (dict(counts=ints([1, 1])), ValueError), (dict(N=0), cache.HadError),
            (dict(tau=-1.0), cache.HadError), (dict(window=-1), cache.HadError),
            (dict(window=2 ** 31), ValueError), (dict(sinks=-1), cache.HadError),
            (dict(max_len=-1), cache.HadError),
            (dict(out=torch.zeros(1, 4, 1, 64)), ValueError), (dict(cache=f.cache.kbits), TypeError),
            (dict(q=q[:, :3].contiguous(), sigma_q=s[:3]), cache.HadError),
            (dict(dev_status=torch.zeros(2, dtype=I, device="cuda")), ValueError)):
        with pytest.raises(error):
            cache.had_cache_attention(**dict(ok, **change))
    for name in ("q", "sigma_q", "table", "lens"):              # a host tensor among the others
        with pytest.raises(ValueError, match="no CPU path"):
            cache.had_cache_attention(**dict(ok, **{name: ok[name].cpu()}))
    for change in (dict(N=2 ** 31), dict(N=-2 ** 31 - 1), dict(window=2 ** 32 + 4), dict(sinks=2 ** 70)):
        with pytest.raises(ValueError, match="32 bits"):
            cache.had_cache_attention(**dict(ok, **change))
    for change in (dict(N=4.5), dict(tau="x"), dict(N=None)):
        with pytest.raises(TypeError):
            cache.had_cache_attention(**dict(ok, **change))
    k = torch.zeros(1, 2, 1, 64, device="cuda")
    with pytest.raises(ValueError):
        cache.had_cache_append(k[:, :1].contiguous(), k, s[:2], f.cache, f.table, ints([0]))
    with pytest.raises(TypeError):
        cache.had_cache_append(k, k.bfloat16(), s[:2], f.cache, f.table, ints([0]))
    with pytest.raises(ValueError):
        cache.Cache(f.cache.kbits, f.cache.vcodes[:, :1].contiguous(), f.cache.vscale)
    with pytest.raises(cache.HadError):
        cache.had_cache_read(f.cache, f.table, ints([0]), 0)


# ------------------------------------------- slices that pass a CTA's memory

def _grown(size):
    """Values of unit noise times size(j, n) at token j of n."""
    def values(B, H, T, d):
        g = torch.Generator().manual_seed(T + d)
        return torch.randn(B, H, T, d, generator=g) * size(torch.arange(T, dtype=torch.float64), T)[:, None]
    return values


SIZES = {
    "grow": lambda j, n: 10.0 ** (6 * j / n),
    "fall": lambda j, n: 10.0 ** (-6 * j / n),
    "last_grow": lambda j, n: torch.where(j < 0.85 * n, 0.2, 1.2),
    "step": lambda j, n: 8.0 ** torch.floor(5 * j / n),
    "swing": lambda j, n: 10.0 ** (8 * torch.sin(j / n * 40)),
}


# 300 tiles or more with one CTA each, which holds 5120 keys in tiles of four
# rows and 2560 in tiles of eight: every instance of the path with segments
@pytest.mark.parametrize("B,G,T,n", [(300, 1, 1, 11000), (1, 3, 800, 6000)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", sorted(SIZES))
def test_values_that_change_size_between_segments(cache, d, B, G, T, n, size):
    """What was summed in earlier segments follows the row's scale in the later ones.  (Sequences
    of one prompt share its pages; the oracle goes through every 37th row.)"""
    f = Filled(cache, [n], 1, d, 64, F32, seed=n + d, values=_grown(SIZES[size]))
    table = f.table.repeat(B, 1)
    lens = [n - 17 * b for b in range(B)]
    q, sigma_q = queries(B, G, T, d, F32)
    for N, tau in ((n, 0.0), (n, 0.1), (400, 0.1)):
        st = status()
        out = cache.had_cache_attention(q.cuda(), sigma_q.cuda(), f.cache, table, ints(lens), N, tau,
                                        dev_status=st).cpu().numpy().reshape(-1, d)
        assert flags(st) == 0
        sq = np.where(q.numpy() / sigma_q.numpy()[None, :, None, None] < 0, -1, 1).reshape(-1, d)
        for r in range(0, B * G * T, 37):
            o, kept, bound = ocache.attend(sq[r], f.sk[0, 0], f.codes[0, 0], f.scale[0, 0],
                                           f.zero[0, 0], N, np.float32(tau), 0, 0,
                                           lens[r // (G * T)] - T + r % T)
            assert (np.abs(out[r] - o) <= (kept.size / 4 + 64) * 2.0 ** -23 * bound).all(), (N, tau, r)


@pytest.mark.parametrize("B,G,T,n", [(300, 1, 1, 11000), (1, 3, 800, 6000)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("same", [True, False])
def test_kept_sets_over_several_segments(cache, d, B, G, T, n, same):
    """As test_kept_sets: counts of the kept tokens of each residue, ties across segments."""
    f = Filled(cache, [n], 1, d, 64, F32, seed=n, values=_marks, same_keys=same)
    lens = [n - 17 * b for b in range(B)]
    q, sigma_q = queries(B, G, T, d, F32)
    sq = np.where(q.numpy() / sigma_q.numpy()[None, :, None, None] < 0, -1, 1).reshape(-1, d)
    for N in (100, 3001):
        st = status()
        out = cache.had_cache_attention(q.cuda(), sigma_q.cuda(), f.cache, f.table.repeat(B, 1),
                                        ints(lens), N, 0.0, dev_status=st).cpu().numpy().reshape(-1, d)
        assert flags(st) == 0
        for r in range(0, B * G * T, 37):
            _, kept, _ = ocache.attend(sq[r], f.sk[0, 0], f.codes[0, 0], f.scale[0, 0], f.zero[0, 0],
                                       N, 0.0, 0, 0, lens[r // (G * T)] - T + r % T)
            count = np.bincount(kept % d, minlength=d)
            got = out[r] * kept.size / 15
            assert np.array_equal(np.rint(got), count) and np.abs(got - count).max() < 0.01


@pytest.mark.parametrize("B,G,T,n", [(300, 1, 1, 11000), (1, 3, 800, 6000)])
@pytest.mark.parametrize("d", [64, 128])
def test_an_unholdable_value_in_a_later_segment(cache, d, B, G, T, n):
    def values(b, h, t, e):
        v = torch.ones(b, h, t, e)
        v[0, 0, n - 200 - 17 * (B - 1), 5] = float("nan")
        return v
    f = Filled(cache, [n], 1, d, 64, F32, seed=n, values=values)
    lens = [n - 17 * b for b in range(B)]
    q, sigma_q = queries(B, G, T, d, F32)
    sq = np.where(q.numpy() / sigma_q.numpy()[None, :, None, None] < 0, -1, 1).reshape(-1, d)
    out = cache.had_cache_attention(q.cuda(), sigma_q.cuda(), f.cache, f.table.repeat(B, 1),
                                    ints(lens), n // 2, 0.1).cpu().numpy().reshape(-1, d)
    nans = 0
    for r in range(0, B * G * T, 7):
        o, kept, bound = ocache.attend(sq[r], f.sk[0, 0], f.codes[0, 0], f.scale[0, 0], f.zero[0, 0],
                                       n // 2, np.float32(0.1), 0, 0, lens[r // (G * T)] - T + r % T)
        assert np.array_equal(np.isnan(out[r]), np.isnan(o))
        nans += np.isnan(o).any()
        if not np.isnan(o).any():
            assert (np.abs(out[r] - o) <= (kept.size / 4 + 64) * 2.0 ** -23 * bound).all()
    assert 0 < nans < B * G * T / 7


def _lowered(cache, S, width, P, page, seed, evict):
    """Forks, lengths that go back and growth in turn, against the oracle."""
    g = np.random.default_rng(seed)
    table, lens, refs = cache.empty_books(S, width, P)
    b = ocache.Books(table, lens, refs, page)
    st = status()
    exchanged = gone = 0
    for step in range(40):
        before = np.array(b.table), np.array(b.refs)
        grow = g.integers(0, max(2, width * page // 3), S) * (g.random(S) < 0.7)
        grow = np.minimum(grow, width * page - np.array(b.lens))
        src, dst = cache.had_cache_reserve(table, lens, refs, page, ints(grow.tolist()), dev_status=st)
        want = b.reserve(grow.tolist())
        if want is None:
            assert flags(st) == NO_PAGES
            st.zero_()
            want = [-1] * S, [-1] * S
            all_gone = g.integers(0, S, S // 2 + 1)
            cache.had_cache_free(table, lens, refs, ints(all_gone.tolist()), dev_status=st)
            b.free(all_gone.tolist())
        else:
            lens += ints(grow.tolist())
            b.lens = [n + int(x) for n, x in zip(b.lens, grow)]
            now = np.array(b.table)
            changed = (before[0] >= 0) & (now != before[0])
            exchanged += int(changed.sum()) - sum(x >= 0 for x in want[0])
            gone += int(((before[1] > 0) & (np.array(b.refs) == 0)).sum())
        assert src.tolist() == want[0] and dst.tolist() == want[1]
        _same_books(table, lens, refs, b)
        n = int(g.integers(0, S + 1))
        to, frm = g.permutation(S)[:n], g.integers(0, S, n)
        cache.had_cache_fork(table, lens, refs, page, ints(frm.tolist()), ints(to.tolist()),
                             dev_status=st)
        b.fork(frm.tolist(), to.tolist())
        if evict and step % 2:
            W = int(g.integers(1, width * page))
            cache.had_cache_evict(table, lens, refs, page, W, 0, dev_status=st)
            b.evict(W, 0)
        # some go back, to any length that still has its last page
        for s in np.flatnonzero(g.random(S) < 0.5):
            n = int(g.integers(0, b.lens[s] + 1))
            if n % page and b.table[s][n // page] < 0:
                n = 0
            b.lens[s] = n
        lens.copy_(ints(b.lens))
        _same_books(table, lens, refs, b)
        assert flags(st) == 0
        counted = np.bincount(table[table >= 0].cpu().numpy(), minlength=P)
        assert np.array_equal(counted, refs.cpu().numpy())
    return exchanged, gone


LOWERED = [(2, 4, 12, 16, 0), (5, 9, 60, 16, 1), (9, 40, 300, 32, 2), (64, 40, 2000, 64, 3),
           (33, 70, 1500, 16, 4), (700, 12, 7000, 16, 5)]


@pytest.mark.parametrize("S,width,P,page,seed", LOWERED)
def test_books_where_lengths_go_back_after_forks(cache, S, width, P, page, seed):
    """Pages behind a length that another sequence reads are exchanged, never written."""
    exchanged, gone = _lowered(cache, S, width, P, page, seed, False)
    assert exchanged >= 10 and gone > 0      # the run does what it is for


def test_a_sequence_that_went_back_after_a_fork_leaves_the_other_as_it_was(cache):
    H, d, page = 2, 64, 16
    f = Filled(cache, [70], H, d, page, F32, spare=12)
    table = torch.full((2, 8), -1, dtype=I, device="cuda")
    table[:1, :f.table.shape[1]] = f.table
    lens, st = ints([70, 0]), status()
    cache.had_cache_fork(table, lens, f.refs, page, ints([0]), ints([1]), dev_status=st)
    before = cache.had_cache_read(f.cache, table[:1], ints([0]), 70, dev_status=st)
    k, v = torch.randn(2, H, 60, d, device="cuda"), torch.randn(2, H, 60, d, device="cuda")
    for back in (48, 37, 16, 0):
        lens[1] = back
        grow = ints([0, 50])
        src, dst = cache.had_cache_reserve(table, lens, f.refs, page, grow, dev_status=st)
        cache.had_cache_copy_pages(f.cache, src, dst, dev_status=st)
        cache.had_cache_append(k, v, f.sigma.cuda(), f.cache, table, lens, counts=grow, dev_status=st)
        lens += grow
        after = cache.had_cache_read(f.cache, table[:1], ints([0]), 70, dev_status=st)
        assert flags(st) == 0
        assert torch.equal(before[0], after[0]) and torch.equal(before[1], after[1])
        # the other one has the common tokens and its own
        bits, values = cache.had_cache_read(f.cache, table[1:], ints([0]), back + 50, dev_status=st)
        assert torch.equal(bits[:, :, :back], before[0][:, :, :back])
        assert torch.equal(values[:, :, :back], before[1][:, :, :back])
        code, s, z = ocache.quantise(v[1:, :, :50].cpu().numpy())
        own = (code * s[..., None].astype(np.float64) + z[..., None]).astype(np.float32)
        assert np.array_equal(values[:, :, back:].cpu().numpy(), own)
        counted = np.bincount(table[table >= 0].cpu().numpy(), minlength=f.refs.numel())
        assert np.array_equal(counted, f.refs.cpu().numpy())


@pytest.mark.parametrize("S,width,P,page,seed", LOWERED)
def test_books_where_lengths_go_back_over_evicted_pages(cache, S, width, P, page, seed):
    """Entries behind a length may be missing before others that are there."""
    _lowered(cache, S, width, P, page, seed, True)


def test_a_sequence_that_starts_again_over_evicted_pages(cache):
    page, st = 16, status()
    table, lens, refs = ints([[-1, -1, 4, -1, 2]]), ints([0]), ints([0, 0, 1, 0, 1, 0, 0])
    src, dst = cache.had_cache_reserve(table, lens, refs, page, ints([80]), dev_status=st)
    assert flags(st) == 0 and src.tolist() == dst.tolist() == [-1]
    assert table.tolist() == [[0, 1, 4, 3, 2]] and refs.tolist() == [1, 1, 1, 1, 1, 0, 0]


@pytest.mark.parametrize("G,d,n", [(1, 64, 31), (1, 128, 400), (3, 64, 400), (4, 128, 3000)])
def test_large_values_of_keys_that_weigh_little(cache, G, d, n):
    """Scales that make up for the weights: every kept token adds as much to the first row.  exp's
    argument goes up to 65, in place of the 23 of the bound, so that takes three times its units."""
    tau = 2.0
    f = Filled(cache, [n], 1, d, 64, F32, seed=n)
    q, sigma_q = queries(1, G, 1, d, F32)
    sq = np.where(q.numpy() / sigma_q.numpy()[None, :, None, None] < 0, -1, 1)
    logit = tau * (f.sk[0, 0] @ sq[0, 0, 0])
    size = torch.from_numpy(np.exp(np.minimum(logit.max() - logit, 64.0)))
    v = (torch.randn(1, 1, n, d, generator=torch.Generator().manual_seed(3)) * size[:, None]).float()
    f = Filled(cache, [n], 1, d, 64, F32, seed=n, values=lambda *_: v)
    st = status()
    out = cache.had_cache_attention(q.cuda(), sigma_q.cuda(), f.cache, f.table, ints([n]), n, tau,
                                    dev_status=st)
    assert flags(st) == 0
    want, bound = f.rows(q, sigma_q, [n], [1], n, tau, 0, 0)
    assert (np.abs(out.cpu().numpy() - want) <= 3 * bound).all()


@pytest.mark.parametrize("ratio", [24, 30, 36, 40, 90])
@pytest.mark.parametrize("at", [5, 20])
@pytest.mark.parametrize("d", [64, 128])
def test_one_huge_value_that_weighs_next_to_nothing(cache, d, at, ratio):
    """31 tokens equal to the query and one opposite to it, of weight e^-69 = 1e-30, whose scale is
    2^ratio times theirs."""
    n = 32
    f = Filled(cache, [n], 1, d, 32, F32, same_keys=True)
    k = f.k.clone()
    k[:, :, at] = -k[:, :, at]
    v = torch.randn(1, 1, n, d, generator=torch.Generator().manual_seed(1))
    v[:, :, at] *= 2.0 ** ratio
    st, tau = status(), 34.5 / d
    cache.had_cache_append(k.cuda(), v.cuda(), f.sigma.cuda(), f.cache, f.table, ints([0]), dev_status=st)
    out = cache.had_cache_attention(f.k[:, :, :1].contiguous().cuda(), f.sigma.cuda(), f.cache, f.table,
                                    ints([n]), n, tau, dev_status=st)
    assert flags(st) == 0
    f.sk[:, :, at] *= -1
    f.codes, f.scale, f.zero = ocache.quantise(v.numpy())
    want, bound = f.rows(f.k[:, :, :1], f.sigma, [n], [1], n, tau, 0, 0)
    assert (np.abs(out.cpu().numpy() - want) <= bound).all()


@pytest.mark.parametrize("d", [64, 128])
def test_scales_of_either_sign(cache, d):
    """A pool that append did not write: c s + z with negative and zero scales of any size."""
    n = 500
    f = Filled(cache, [n], 2, d, 16, F32, seed=6)
    g = torch.Generator().manual_seed(7)
    scale = torch.randn(f.cache.vscale.shape, generator=g)
    scale = scale * 10.0 ** torch.randint(-20, 21, scale.shape[:3] + (1,), generator=g)
    scale[torch.rand(scale.shape[:3], generator=g) < 0.1, 0] = 0.0
    f.cache.vscale.copy_(scale)
    pages = f.table[0, :-(-n // 16)].cpu().long()
    sz = scale.bfloat16().double()[pages].permute(1, 0, 2, 3).reshape(2, -1, 2)[:, :n].numpy()
    f.scale, f.zero = sz[None, ..., 0], sz[None, ..., 1]
    q, sigma_q = queries(1, 6, 1, d, F32)
    for N in (20, n):
        st = status()
        out = cache.had_cache_attention(q.cuda(), sigma_q.cuda(), f.cache, f.table, ints([n]), N, 0.1,
                                        dev_status=st)
        assert flags(st) == 0
        want, _ = f.rows(q, sigma_q, [n], [1], N, 0.1, 0, 0)
        # what is summed is p (c - 8) s and p (z + 8 s): 16 steps and z at most
        codes, f.codes = f.codes, np.full_like(f.codes, 16)
        _, bound = f.rows(q, sigma_q, [n], [1], N, 0.1, 0, 0)
        f.codes = codes
        assert (np.abs(out.cpu().numpy() - want) <= bound).all()


def _library():
    """The C ABI itself: ctypes lets go of Python's lock during a call."""
    import ctypes
    from sparse_attention_sigma_b200 import build
    lib = ctypes.CDLL(build.LIB)
    vp, i32 = ctypes.c_void_p, ctypes.c_int
    lib.had_cache_attention.argtypes = ([vp, i32, vp, vp, vp, i32, vp, vp, i32, i32, i32, i32,
                                         ctypes.c_float, i32, i32, i32, vp, vp, vp])
    lib.had_cache_read.argtypes = [vp, vp, i32, vp, vp, i32, i32, vp, vp, vp, vp]
    lib.had_cache_reserve.argtypes = [vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, vp]
    return lib


class _PoolStruct:
    """had_cache_t of a Cache, as ctypes passes it."""
    def __new__(cls, c):
        import ctypes

        class had_cache_t(ctypes.Structure):
            _fields_ = [(n, ctypes.c_void_p) for n in ("kbits", "vcodes", "vscale")] + [
                (n, ctypes.c_int) for n in ("pages", "heads", "page", "d")]
        return ctypes.pointer(had_cache_t(c.kbits.data_ptr(), c.vcodes.data_ptr(), c.vscale.data_ptr(),
                                          c.pages, c.heads, c.page, c.d))


def test_host_threads_that_call_at_once(cache):
    """Two threads whose calls take different amounts of shared memory of the same kernels."""
    import threading
    lib = _library()
    H, G, d, page = 2, 2, 128, 16
    f = Filled(cache, [1500], H, d, page, F32)
    pool = _PoolStruct(f.cache)
    q, sigma_q = (x.cuda() for x in queries(1, G * H, 1, d, F32))
    lens, bad = ints([1500]), []
    want = cache.had_cache_attention(q, sigma_q, f.cache, f.table, lens, 50, 0.1)
    calls, keep = [], []
    for width, S in ((1200, 1800), (2500, 8192)):               # 40 and 50 KB, 29 and 131 KB
        table = torch.full((1, width), -1, dtype=I, device="cuda")
        table[:, :f.table.shape[1]] = f.table
        out, s = torch.zeros_like(want), torch.cuda.Stream()
        books = cache.empty_books(S, 1, 10) + tuple(torch.zeros(S, dtype=I, device="cuda") for _ in "gsd")
        keep.append((table, books, s, out))
        t, n, r, grow, src, dst = (x.data_ptr() for x in books)
        calls.append((
            (q.data_ptr(), 1, sigma_q.data_ptr(), pool, table.data_ptr(), width, lens.data_ptr(), None, 1,
             G * H, 1, 50, 0.1, 0, 0, 0, out.data_ptr(), None, s.cuda_stream),
            (t, n, r, S, 1, 10, page, grow, src, dst, None, s.cuda_stream)))
    torch.cuda.synchronize()

    def work(attention, reserve):
        for _ in range(400):
            bad.extend(x for x in [lib.had_cache_attention(*attention) for _ in range(10)] if x)
            bad.extend(x for x in [lib.had_cache_reserve(*reserve) for _ in range(10)] if x)

    threads = [threading.Thread(target=work, args=c) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not bad, (len(bad), bad[:5])
    for _, _, _, out in keep:
        assert torch.allclose(out, want, rtol=1e-5, atol=1e-5)


def test_more_than_2_to_30_rows(cache):
    """Rows of a read whose threads, eight each, pass 2^32: 4 M sequences that share one page."""
    page, d, B = 256, 64, 2 ** 22 + 5
    f = Filled(cache, [page], 1, d, page, F32, spare=0)
    table = f.table[:, :1].repeat(B, 1)
    start, st = torch.zeros(B, dtype=I, device="cuda"), status()
    bits = torch.full((B, page, d // 32), 0x5a5a5a5a, dtype=I, device="cuda")
    assert _library().had_cache_read(_PoolStruct(f.cache), table.data_ptr(), 1, start.data_ptr(), None, B,
                                     page, bits.data_ptr(), None, st.data_ptr(),
                                     torch.cuda.current_stream().cuda_stream) == 0
    want = cache.had_cache_read(f.cache, f.table, ints([0]), page)[0][0, 0]
    assert flags(st) == 0
    for b in range(0, B, 1 << 19):
        assert (bits[b:b + (1 << 19)] == want).all()


@pytest.mark.parametrize("d", [64, 128])
def test_queries_equal_and_opposite_to_keys(cache, d):
    """Distances 0 and d in each place of a word of four: each query is a token or its opposite."""
    n, T = 40, 8
    f = Filled(cache, [n], 1, d, 16, F32, seed=3)
    at = torch.tensor([0, 7, 15, 16, 31, 1, 20, 30])
    q = f.k[:, :, at].contiguous()
    for N in (1, n):
        st = status()
        for sign in (1, -1):
            out = cache.had_cache_attention((sign * q).cuda(), f.sigma.cuda(), f.cache, f.table, ints([n]),
                                            N, 0.1, dev_status=st)
            want, bound = f.rows(sign * q, f.sigma, [n], [T], N, 0.1, 0, 0)
            assert (np.abs(out.cpu().numpy() - want) <= bound).all()
        assert flags(st) == 0


def test_a_cache_whose_tensors_get_other_storage(cache):
    """A call reads the tensors as they are: other storage of the same shape, or a refusal."""
    f = Filled(cache, [112], 2, 64, 16, F32)
    q, sigma_q = (x.cuda() for x in queries(1, 2, 1, 64, F32))
    run = lambda c: cache.had_cache_attention(q, sigma_q, c, f.table, ints([112]), 9, 0.1)  # noqa: E731
    other = [f.cache.kbits.flip(1), f.cache.vcodes.flip(1), f.cache.vscale.flip(1)]
    want = run(cache.Cache(*other))
    assert not torch.equal(run(f.cache), want)
    for name, t in zip(("kbits", "vcodes", "vscale"), other):
        with pytest.raises(AttributeError):
            setattr(f.cache, name, t)
        getattr(f.cache, name).data = t
    assert torch.equal(run(f.cache), want)
    f.cache.vcodes.data = other[1][:-1]
    with pytest.raises(ValueError, match="any more"):
        run(f.cache)
    f.cache.vcodes.data = other[1].transpose(0, 1)
    with pytest.raises(ValueError, match="any more"):
        cache.had_cache_copy_pages(f.cache, ints([0]), ints([1]))
    f.cache.vcodes.data = other[1].cpu()
    with pytest.raises(ValueError, match="any more"):
        cache.had_cache_read(f.cache, f.table, ints([0]), 1)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_whose_largest_code_would_overflow(cache, dtype, d):
    """Rows up to the largest number of bf16, where 15 s + z may pass fp32: marked, never infinite."""
    T, most = 256, torch.finfo(BF16).max
    g = torch.Generator().manual_seed(d)
    low = most * 10.0 ** torch.linspace(-3, 0, T, dtype=torch.float64)[:, None]
    v = low + (most - low) * torch.rand(1, 1, T, d, generator=g, dtype=torch.float64)
    v[..., 3], v[..., 5] = most, low[:, 0]
    v = v.clamp(max=most).to(dtype)
    c = cache.Cache.empty(1, 1, 256, d)
    st = status()
    cache.had_cache_append(v.cuda(), v.cuda(), torch.ones(1, device="cuda"), c, ints([[0]]), ints([0]),
                           dev_status=st)
    values = cache.had_cache_read(c, ints([[0]]), ints([0]), T, dev_status=st)[1].cpu().numpy()
    code, s, z = ocache.quantise(v.float().numpy())
    assert 0 < np.isnan(s).sum() < T and not np.isinf(values).any()
    exact = (code * s[..., None].astype(np.float64) + z[..., None]).astype(np.float32)
    assert np.array_equal(values, exact, equal_nan=True)
    assert flags(st) == 0
