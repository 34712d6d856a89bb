"""The cache operators of binarized attention: cases, plain forms and exact values.

A cache of a decoder that attends with binarized keys holds, for every token
and key-value head, the d signs of the key (1 bit each) and the value in 4
bits with a scale and a zero point (bf16).  Tokens lie in pages; a table row
per sequence lists its pages.  The operators write tokens into pages, read
them back, attend to them (top-N of the Hamming logits, optionally within a
sliding window and a few first tokens), and keep the pages' books.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _attend(name, B, Hq, Hkv, d, page, T, len_min, len_max, N, window=0, sinks=0, dtype="bf16"):
    return dict(name=name, kind="attend", B=B, Hq=Hq, Hkv=Hkv, d=d, page=page, T=T,
                len_min=len_min, len_max=len_max, N=N, window=window, sinks=sinks, dtype=dtype)


def _append(name, B, Hkv, d, page, T, ragged, dtype="bf16"):
    return dict(name=name, kind="append", B=B, Hkv=Hkv, d=d, page=page, T=T, ragged=ragged,
                dtype=dtype)


def _pages(name, kind, S, Hkv, d, page, len_min, len_max, moves=0, window=0, sinks=0):
    return dict(name=name, kind=kind, S=S, Hkv=Hkv, d=d, page=page, len_min=len_min,
                len_max=len_max, moves=moves, window=window, sinks=sinks)


def listed():
    return [
        # one sequence of the tiny workload's size generating one token: pure latency
        _attend("decode_tiny", 1, 2, 2, 64, 16, 1, 128, 128, 16, dtype="f32"),
        # a batch of short answers, every query head with its own keys
        _attend("decode_short", 32, 12, 12, 64, 16, 1, 33, 512, 64),
        # the long workload's context, four query heads to a key head, ragged
        _attend("decode_long", 16, 16, 4, 64, 64, 1, 1000, 4096, 512),
        # very long contexts, d 128: the largest cache read
        _attend("decode_vlong", 16, 32, 8, 128, 64, 1, 15000, 16384, 2048),
        # a window and four first tokens over contexts far longer than the window; all visible kept
        _attend("decode_window", 32, 32, 8, 128, 64, 1, 4097, 16384, 1028, window=1024, sinks=4),
        # a draft of up to five tokens checked at once; padded batch, an empty sequence, odd sizes
        _attend("draft_ragged", 7, 12, 3, 64, 32, 5, 0, 2777, 100),
        # a chunk of a prompt against what is cached before it, window and first tokens
        _attend("chunk_window", 4, 16, 4, 64, 64, 512, 2048, 4096, 64, window=512, sinks=4),
        # one new token of each sequence of a batch into the cache
        _append("append_step", 32, 12, 64, 16, 1, False),
        # whole prompts into the cache, ragged, d 128
        _append("append_prompt", 2, 8, 128, 64, 16384, True),
        # a beam step: parents forked, room made with copies of shared last pages, window evicted
        _pages("pages_beam", "beam", 64, 8, 128, 64, 500, 4096, window=1024, sinks=4),
        # copying many pages of one pool at once
        _pages("pages_copy", "copy", 64, 8, 128, 64, 2000, 4096, moves=1501),
        # half of the sequences leave and the pool closes its holes
        _pages("pages_compact", "compact", 64, 8, 128, 64, 1000, 4096),
    ]


def draw(rng):
    def logu(a, b):
        return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))

    case = _drawn(rng, logu)
    del case["name"]
    return case


def _drawn(rng, logu):
    kind = rng.choice(["attend"] * 6 + ["append"] * 2 + ["beam", "copy", "compact"])
    d = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128, 256])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind == "attend":
        Hkv = rng.choice([1, 2, 3, 4, 8])
        G = rng.choice([1, 1, 2, 3, 4, 5, 8])
        T = rng.choice([1, 1, 1, 2, 3, logu(4, 300)])
        len_max = logu(T, 16384)
        # the (query, key) pairs and the cached tokens of a case stay below the largest listed one's
        most = min((1 << 23) // (len_max * Hkv * G * T), (1 << 21) // (len_max * Hkv))
        if most < 1:
            len_max = max(T, (1 << 23) // (Hkv * G * T))
            most = 1
        B = rng.randint(1, max(1, min(32, most)))
        window, sinks = rng.choice([(0, 0), (0, 0), (logu(1, 2048), rng.choice([0, 1, 4, 33]))])
        N = logu(1, max(1, len_max // rng.choice([1, 2, 8])))
        return _attend(None, B, Hkv * G, Hkv, d, page, T, rng.randint(0, len_max), len_max, N,
                       window, sinks, dtype)
    if kind == "append":
        T = rng.choice([1, logu(2, 8192)])
        Hkv = rng.choice([1, 3, 4, 8, 12])
        B = rng.randint(1, max(1, min(32, (1 << 17) // (T * Hkv))))
        return _append(None, B, Hkv, d, page, T, rng.random() < 0.5, dtype)
    Hkv = rng.choice([1, 2, 5, 8])
    S = rng.randint(2, 64)
    len_max = logu(2, 4096)
    return _pages(None, kind, S, Hkv, d, page, rng.randint(1, len_max), len_max,
                  moves=logu(1, max(1, (1 << 19) // (page * Hkv))) if kind == "copy" else 0,
                  window=rng.choice([0, logu(1, 1024)]), sinks=rng.choice([0, 4]))


# ------------------------------------------------------------------ sizes of a case

def _ceil(a, b):
    return -(-a // b)


def _lengths(case, count):
    """Lengths of the sequences: spread over [len_min, len_max], the first the longest."""
    lo, hi = case["len_min"], case["len_max"]
    return [hi - (b * 2654435761 % 1000003) % (hi - lo + 1) if b else hi for b in range(count)]


def _counts(case):
    """New tokens of each sequence (of T): ragged where T > 1 in a ragged batch; never above the length."""
    T = case["T"]
    return [T - (b * 7) % 3 if T > 2 and b else T for b in range(case["B"])]


def _append_plan(case):
    """First position and number of the new tokens of each sequence."""
    T, page = case["T"], case["page"]
    start = [(b * 37) % (2 * page) for b in range(case["B"])]
    count = [T - (b * T) // (2 * case["B"]) if case["ragged"] else T for b in range(case["B"])]
    return start, count


def _token_bytes(d):
    return d // 8 + d // 2 + 4


def work(case):
    d = case["d"]
    if case["kind"] == "attend":
        esize = 2 if case["dtype"] == "bf16" else 4
        nbytes = flops = 0
        for L, c in zip(_lengths(case, case["B"]), _counts(case)):
            pairs = kept = 0
            seen, most = 0, 0
            W, S = case["window"], case["sinks"]
            for t in range(c):
                i = L - c + t
                if i < 0:
                    continue
                vis = i + 1 if W <= 0 else min(i + 1, W) + min(S, max(0, i + 1 - W))
                pairs += vis
                kept += min(case["N"], vis)
                most = max(most, min(case["N"], vis))
                # keys seen by any row: the last row's and, under a window, one more per row before it
                seen = vis if W <= 0 else min(i + 1, vis + t)
            nbytes += case["Hkv"] * (seen * d // 8 + most * (d // 2 + 4))
            nbytes += case["Hq"] * c * d * (esize + 4)
            flops += case["Hq"] * 2 * d * (pairs + kept)
        return {"bytes": nbytes, "flops": flops}
    if case["kind"] == "append":
        esize = 2 if case["dtype"] == "bf16" else 4
        tokens = sum(_append_plan(case)[1]) * case["Hkv"]
        # K and V read, the cache's form written; then read back as bits and fp32
        return {"bytes": tokens * (2 * d * esize + 2 * _token_bytes(d) + d // 8 + 4 * d),
                "flops": tokens * 8 * d}
    lens = _lengths(case, case["S"])
    page_bytes = case["page"] * case["Hkv"] * _token_bytes(d)
    if case["kind"] == "copy":
        return {"bytes": 2 * case["moves"] * page_bytes, "flops": 0}
    if case["kind"] == "beam":
        forks = case["S"] // 2
        table = sum(_ceil(n, case["page"]) for n in lens) * 4
        return {"bytes": 2 * forks * page_bytes + 4 * table, "flops": 0}
    left = sum(_ceil(n, case["page"]) for n in lens[1::2])
    return {"bytes": 2 * (left // 2) * page_bytes + 8 * left, "flops": 0}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed * 1000003 + 17)


def _signal(g, heads, tokens, d, w):
    """Keys or queries with a shared low-rank signal and unit noise: heavy-tailed logits."""
    u = torch.randn(heads, tokens, w.shape[1], generator=g, device="cuda")
    return u @ w / math.sqrt(w.shape[1]) + torch.randn(heads, tokens, d, generator=g, device="cuda")


class _Pool:
    """The three arrays of a pool of pages."""

    def __init__(self, pages, heads, page, d):
        self.kbits = torch.zeros(pages, heads, page, d // 32, dtype=torch.int32, device="cuda")
        self.vcodes = torch.zeros(pages, heads, page, d // 2, dtype=torch.uint8, device="cuda")
        self.vscale = torch.zeros(pages, heads, page, 2, dtype=torch.bfloat16, device="cuda")

    def arrays(self):
        return self.kbits, self.vcodes, self.vscale

    def raw(self):
        """The arrays as whole numbers: what moving pages has to keep bit for bit."""
        return self.kbits, self.vcodes, self.vscale.view(torch.int16)


def _tables(lens, page, width, spare, g):
    """Table rows of sequences of these lengths over pages in a random order, and the pages' counts."""
    need = [_ceil(n, page) for n in lens]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    refs[order[:at].long()] = 1
    return table, refs


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = _gen(seed)
    d, page, Hkv = case["d"], case["page"], case["Hkv"]
    if case["kind"] == "attend":
        B, Hq, T = case["B"], case["Hq"], case["T"]
        dt = DT[case["dtype"]]
        lens, counts = _lengths(case, B), _counts(case)
        table, refs = _tables(lens, page, _ceil(max(max(lens), 1), page), 3, g)
        pool = _Pool(refs.numel(), Hkv, page, d)
        w = torch.randn(Hkv, 32, d, generator=g, device="cuda")
        sigma = 1.4 + 0.1 * torch.rand(Hkv, generator=g, device="cuda")
        for b, n in enumerate(lens):
            if n:
                k = _signal(g, Hkv, n, d, w).to(dt)
                v = torch.randn(Hkv, n, d, generator=g, device="cuda").to(dt)
                _plain_append(k[None], v[None], sigma, pool, table[b:b + 1], _i32([0]), _i32([n]))
        q = _signal(g, Hkv, B * T * (Hq // Hkv), d, w).reshape(Hq, B, T, d).transpose(0, 1)
        return dict(case=case, pool=pool, table=table, lens=_i32(lens), counts=_i32(counts),
                    q=q.to(dt).contiguous(),
                    sigma_q=1.4 + 0.1 * torch.rand(Hq, generator=g, device="cuda"),
                    N=case["N"], tau=1.0 / math.sqrt(d), window=case["window"],
                    sinks=case["sinks"])
    if case["kind"] == "append":
        B, T = case["B"], case["T"]
        dt = DT[case["dtype"]]
        start, count = _append_plan(case)
        lens = [s + c for s, c in zip(start, count)]
        table, refs = _tables(lens, page, _ceil(max(lens), page), 1, g)
        pool = _Pool(refs.numel(), Hkv, page, d)
        k = torch.randn(B, Hkv, T, d, generator=g, device="cuda").to(dt)
        v = torch.randn(B, Hkv, T, d, generator=g, device="cuda")
        # a few channels of values run larger than the rest, as they do in practice
        v = (v * (1 + 4 * (torch.arange(d, device="cuda") % 23 == 0))).to(dt)
        return dict(case=case, pool=pool, table=table, start=_i32(start), count=_i32(count), k=k,
                    v=v, sigma_k=0.9 + 0.2 * torch.rand(Hkv, generator=g, device="cuda"))
    S = case["S"]
    lens = _lengths(case, S)
    width = _ceil(case["len_max"], page) + 2
    spare = 2 * S + 2 * case["moves"]
    table, refs = _tables(lens, page, width, spare, g)
    pool = _Pool(refs.numel(), Hkv, page, d)
    for a in pool.arrays():
        raw = a.view(torch.int32)
        raw.copy_(torch.randint(-2 ** 31, 2 ** 31, raw.shape, generator=g, device="cuda"))
        if a.dtype == torch.bfloat16:
            a.copy_(torch.rand(a.shape, generator=g, device="cuda"))
    st = dict(case=case, pool=pool, table=table, refs=refs, lens=_i32(lens))
    if case["kind"] == "copy":
        free = torch.nonzero(refs == 0).flatten()
        used = torch.nonzero(refs).flatten()
        m = min(case["moves"], free.numel())
        pick = torch.randint(0, used.numel(), (m,), generator=g, device="cuda")
        st["src"] = used[pick].to(torch.int32)
        perm = torch.randperm(free.numel(), generator=g, device="cuda")[:m]
        st["dst"] = free[perm].to(torch.int32)
    elif case["kind"] == "beam":
        # every group of sequences goes on from some of its members
        parent = torch.randint(0, S, (S,), generator=g, device="cuda")
        parent = torch.where(torch.arange(S, device="cuda") % 2 == 0,
                             torch.arange(S, device="cuda"), parent)
        st["src"] = parent.to(torch.int32)
        st["dst"] = torch.arange(S, dtype=torch.int32, device="cuda")
        st["grow"] = torch.ones(S, dtype=torch.int32, device="cuda")
    else:
        st["leave"] = torch.arange(0, S, 2, dtype=torch.int32, device="cuda")
    return st


# ------------------------------------------------------------------ plain forms

def _slots(pool, table, b, pos):
    """Page and slot of positions `pos` of the sequences of table rows b."""
    page = pool.kbits.shape[2]
    return table[b, pos // page].long(), pos % page


def _new_tokens(start, count, T):
    """Sequence, index and position of every new token of a padded batch, as flat lists."""
    b, t = torch.nonzero(torch.arange(T, device="cuda") < count[:, None], as_tuple=True)
    return b, t, start[b] + t


def _bits(neg):
    """Packed signs of a boolean [..., d]: bit k of word w is element 32 w + k."""
    w = neg.reshape(*neg.shape[:-1], -1, 32).long()
    word = (w << torch.arange(32, device=neg.device)).sum(-1)
    return torch.where(word >= 2 ** 31, word - 2 ** 32, word).to(torch.int32)


def _bf16_down(x):
    """Largest bf16 not above the fp32 x."""
    raw = x.contiguous().view(torch.int32)
    cut = raw & -65536
    cut = torch.where((raw < 0) & (cut != raw), cut + 65536, cut)
    return cut.view(torch.float32)


def _plain_quantise(v):
    """4-bit codes of the rows of v, with scale and zero point as (bf16-valued) fp32."""
    v = v.float()
    zero = _bf16_down(v.amin(-1) + 0.0)
    span = v.amax(-1) - zero
    # a quotient by a tensor is the IEEE division (by a scalar, a product with its reciprocal)
    scale = -_bf16_down(-(span / torch.full_like(span, 15.0)))
    code = ((v - zero[..., None]) / scale[..., None]).round().clamp(0, 15)
    code = torch.where(scale[..., None] > 0, code, torch.zeros_like(code))
    return code.to(torch.int32), scale + 0.0, zero


def _plain_append(k, v, sigma, pool, table, start, count):
    neg = (k.float() / sigma[None, :, None, None]) < 0
    b, t, pos = _new_tokens(start, count, k.shape[2])
    p, slot = _slots(pool, table, b, pos)
    code, scale, zero = _plain_quantise(v[b, :, t])
    pool.kbits[p, :, slot] = _bits(neg[b, :, t])
    pool.vcodes[p, :, slot] = (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8)
    pool.vscale[p, :, slot] = torch.stack([scale, zero], -1).to(torch.bfloat16)


def _plain_values(pool, p, slot):
    """Values of cached tokens, fp32 [..., heads, d] for pages and slots [...]."""
    byte = pool.vcodes[p, :, slot]
    code = torch.stack([byte & 15, byte >> 4], -1).flatten(-2)
    sz = pool.vscale[p, :, slot].float()
    return code * sz[..., :1] + sz[..., 1:]


def _plain_read(pool, table, start, count, T):
    H, d = pool.kbits.shape[1], pool.vcodes.shape[3] * 2
    B = table.shape[0]
    bits = torch.zeros(B, H, T, d // 32, dtype=torch.int32, device="cuda")
    vals = torch.zeros(B, H, T, d, device="cuda")
    b, t, pos = _new_tokens(start, count, T)
    p, slot = _slots(pool, table, b, pos)
    bits[b, :, t] = pool.kbits[p, :, slot]
    vals[b, :, t] = _plain_values(pool, p, slot)
    return bits, vals


def _plain_attend(st):
    pool, table, q, lens = st["pool"], st["table"], st["q"], st["lens"].long()
    B, Hq, T, d = q.shape
    Hkv = pool.kbits.shape[1]
    G = Hq // Hkv
    L = table.shape[1] * pool.kbits.shape[2]
    j = torch.arange(L, device="cuda")
    p, slot = _slots(pool, table.clamp(min=0), torch.arange(B, device="cuda")[:, None],
                     j.expand(B, L))
    word = pool.kbits[p, :, slot].transpose(1, 2)
    sk = 1.0 - 2.0 * ((word[..., None] >> torch.arange(32, device="cuda")) & 1).flatten(-2)
    sq = 1.0 - 2.0 * ((q.float() / st["sigma_q"][None, :, None, None]) < 0).float()
    s = sq.reshape(B, Hkv, G * T, d) @ sk.transpose(2, 3)
    # position of token t of a sequence; tokens past its count see nothing
    t = torch.arange(T, device="cuda")
    pos = torch.where(t < st["counts"][:, None], (lens - st["counts"])[:, None] + t, -1)[..., None]
    vis = j <= pos
    if st["window"] > 0:
        vis &= (j > pos - st["window"]) | (j < st["sinks"])
    vis = vis.repeat(1, G, 1)[:, None]
    h = torch.where(vis, (d - s) * 0.5, d + 1.0).to(torch.uint8)
    n = vis.sum(-1, keepdim=True).clamp(max=st["N"])
    last = h.sort(-1).values.gather(-1, (n - 1).clamp(min=0).expand(B, Hkv, G * T, 1))
    less = vis & (h < last)
    tie = vis & (h == last)
    keep = less | (tie & (tie.cumsum(-1) <= n - less.sum(-1, keepdim=True)))
    best = torch.where(vis, s, -float(d)).amax(-1, keepdim=True)
    w = torch.exp(st["tau"] * (s - best)) * keep
    z = w.sum(-1, keepdim=True)
    # pages behind a sequence hold what earlier tokens left: their weights are 0, their values cut
    seen = (j < lens[:, None])[..., None, None]
    value = torch.where(seen, _plain_values(pool, p, slot), 0.0).transpose(1, 2)
    return ((w @ value) / torch.where(z > 0, z, 1.0)).reshape(B, Hq, T, d)


def _plain_fork(table, lens, refs, page, src, dst):
    s, t = src.long(), dst.long()
    new_len, old = lens[s], table[t]
    # pages that were reserved behind the source's tokens stay the source's own
    held = torch.arange(table.shape[1], device="cuda")[None] * page < new_len[:, None]
    new = torch.where(held, table[s], -1)
    refs.index_add_(0, new[new >= 0].long(), torch.ones_like(new[new >= 0]))
    refs.index_add_(0, old[old >= 0].long(), -torch.ones_like(old[old >= 0]))
    table[t] = new
    lens[t] = new_len


def _plain_reserve(table, lens, refs, page, grow):
    S, width = table.shape
    have = (lens + page - 1) // page
    want = torch.where(grow > 0, (lens + grow + page - 1) // page, have)
    last = (lens // page).clamp(max=width - 1).long()
    shared = table.gather(1, last[:, None])[:, 0]
    part = (grow > 0) & (lens % page != 0)
    earlier = ((shared[None] == shared[:, None]) & part[None]).tril(-1).sum(1)
    copy = part & (refs[shared.clamp(min=0).long()] - earlier > 1)
    idx = torch.arange(width, device="cuda")[None]
    need = (idx >= have[:, None]) & (idx < want[:, None]) & (table < 0)
    need |= copy[:, None] & (idx == last[:, None])
    where = torch.nonzero(need)
    page_of = torch.nonzero(refs == 0).flatten()[:where.shape[0]].to(torch.int32)
    refs[page_of.long()] = 1
    table[where[:, 0], where[:, 1]] = page_of
    refs.index_add_(0, shared[copy].long(), -torch.ones_like(shared[copy]))
    fresh = table.gather(1, last[:, None])[:, 0]
    none = torch.full_like(shared, -1)
    return torch.where(copy, shared, none), torch.where(copy, fresh, none)


def _plain_drop(table, refs, gone):
    pages = table[gone]
    pages = pages[pages >= 0]
    refs.index_add_(0, pages.long(), -torch.ones_like(pages))
    table[gone] = -1


def _plain_free(table, lens, refs, seqs):
    gone = torch.zeros_like(table, dtype=torch.bool)
    gone[seqs.long()] = True
    _plain_drop(table, refs, gone)
    lens[seqs.long()] = 0


def _plain_evict(table, lens, refs, page, window, sinks):
    first = torch.arange(table.shape[1], device="cuda")[None] * page
    _plain_drop(table, refs, (first >= sinks) & (first + page <= lens[:, None] - window))


def _plain_compact(table, refs):
    P = refs.numel()
    used = refs > 0
    live = int(used.sum())
    hole = torch.nonzero(~used[:live]).flatten()
    far = torch.nonzero(used[live:]).flatten() + live
    to = torch.arange(P, device="cuda")
    to[far] = hole
    refs[hole] = refs[far]
    refs[far] = 0
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()].to(torch.int32), table))
    src = torch.full((P,), -1, dtype=torch.int32, device="cuda")
    dst = src.clone()
    src[:far.numel()], dst[:far.numel()] = far.to(torch.int32), hole.to(torch.int32)
    return src, dst, _i32([live])


def _plain_copy(pool, src, dst):
    m = (src >= 0) & (dst >= 0)
    s, t = src[m].long(), dst[m].long()
    for a in pool.arrays():
        a[t] = a[s]


# ------------------------------------------------------------------ one pass

def run(st):
    if own:
        return _run_own(st)
    case, pool = st["case"], st["pool"]
    if case["kind"] == "attend":
        return _plain_attend(st)
    if case["kind"] == "append":
        _plain_append(st["k"], st["v"], st["sigma_k"], pool, st["table"], st["start"], st["count"])
        return _plain_read(pool, st["table"], st["start"], st["count"], case["T"])
    if case["kind"] == "copy":
        _plain_copy(pool, st["src"], st["dst"])
        return pool.raw()
    table, lens, refs = st["table"].clone(), st["lens"].clone(), st["refs"].clone()
    if case["kind"] == "beam":
        _plain_fork(table, lens, refs, case["page"], st["src"], st["dst"])
        src, dst = _plain_reserve(table, lens, refs, case["page"], st["grow"])
        _plain_copy(pool, src, dst)
        if case["window"] > 0:
            _plain_evict(table, lens, refs, case["page"], case["window"], case["sinks"])
        return (table, lens, refs, src, dst) + pool.raw()
    _plain_free(table, lens, refs, st["leave"])
    src, dst, live = _plain_compact(table, refs)
    _plain_copy(pool, src, dst)
    return (table, lens, refs, src, dst, live) + pool.raw()


def _run_own(st):
    from sparse_attention_sigma_b200 import cache
    case, pool = st["case"], cache.Cache(*st["pool"].arrays())
    if case["kind"] == "attend":
        return cache.had_cache_attention(st["q"], st["sigma_q"], pool, st["table"], st["lens"],
                                         st["N"], st["tau"], window=st["window"],
                                         sinks=st["sinks"], counts=st["counts"])
    if case["kind"] == "append":
        cache.had_cache_append(st["k"], st["v"], st["sigma_k"], pool, st["table"], st["start"],
                               counts=st["count"])
        return cache.had_cache_read(pool, st["table"], st["start"], case["T"], counts=st["count"])
    if case["kind"] == "copy":
        cache.had_cache_copy_pages(pool, st["src"], st["dst"])
        return st["pool"].raw()
    table, lens, refs = st["table"].clone(), st["lens"].clone(), st["refs"].clone()
    if case["kind"] == "beam":
        cache.had_cache_fork(table, lens, refs, case["page"], st["src"], st["dst"])
        src, dst = cache.had_cache_reserve(table, lens, refs, case["page"], st["grow"])
        cache.had_cache_copy_pages(pool, src, dst)
        if case["window"] > 0:
            cache.had_cache_evict(table, lens, refs, case["page"], case["window"], case["sinks"])
        return (table, lens, refs, src, dst) + st["pool"].raw()
    cache.had_cache_free(table, lens, refs, st["leave"])
    src, dst, live = cache.had_cache_compact(table, refs)
    cache.had_cache_copy_pages(pool, src, dst)
    return (table, lens, refs, src, dst, live) + st["pool"].raw()


# ------------------------------------------------------------------ exact values

def _exact_rows(st, b, L, c):
    """Signs and values in 64 bits of the L cached tokens of sequence b, by walking its pages."""
    pool, page = st["pool"], st["case"]["page"]
    ids = st["table"][b, :_ceil(L, page)].tolist()
    words = torch.cat([pool.kbits[i] for i in ids], 1)[:, :L].long() & 0xFFFFFFFF
    code = torch.cat([pool.vcodes[i] for i in ids], 1)[:, :L]
    sz = torch.cat([pool.vscale[i] for i in ids], 1)[:, :L].double()
    H, _, half = code.shape
    value = torch.empty(H, L, 2 * half, dtype=torch.float64, device="cuda")
    value[..., 0::2] = (code % 16).double() * sz[..., :1] + sz[..., 1:]
    value[..., 1::2] = (code // 16).double() * sz[..., :1] + sz[..., 1:]
    sign = torch.empty_like(value)
    for k in range(2 * half):
        sign[..., k] = 1 - 2 * ((words[..., k // 32] >> (k % 32)) % 2).double()
    return sign, value


def exact(case, seed):
    if case["kind"] == "attend":
        st = prepare(case, seed)
        q, d, G = st["q"], case["d"], case["Hq"] // case["Hkv"]
        out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
        # an fp32 quotient is negative wherever the operands' signs differ and it does not underflow
        sq = torch.where(q.double() / st["sigma_q"].double()[None, :, None, None] < -2.0 ** -150,
                         -1.0, 1.0).double()
        for b, (L, c) in enumerate(zip(_lengths(case, case["B"]), _counts(case))):
            if L == 0:
                continue
            sign, value = _exact_rows(st, b, L, c)
            j = torch.arange(L, device="cuda")
            for h in range(case["Hq"]):
                s = sq[b, h, :c] @ sign[h // G].T
                for t0 in range(0, c, 64):
                    rows = torch.arange(t0, min(t0 + 64, c), device="cuda")
                    i = (L - c + rows)[:, None]
                    seen = (j <= i) & ((j > i - case["window"]) | (j < case["sinks"])
                                       if case["window"] > 0 else j <= i)
                    # one order of all keys of a row: the logit first, the lower index within it
                    rank = torch.where(seen, s[rows] * (L + 1) - j, -math.inf)
                    order = rank.argsort(-1, descending=True)[:, :case["N"]]
                    logit = torch.where(seen.gather(1, order), st["tau"] * s[rows].gather(1, order),
                                        -math.inf)
                    some = seen.any(-1)
                    p = torch.softmax(logit[some], -1)
                    out[b, h, rows[some]] = torch.einsum("rn,rnd->rd", p, value[h // G][order[some]])
        return out
    if case["kind"] == "append":
        st = prepare(case, seed)
        start, count = _append_plan(case)
        vals = np.zeros((case["B"], case["Hkv"], case["T"], case["d"]))
        for b, c in enumerate(count):
            v = st["v"][b, :, :c].float().cpu().numpy()
            # the definition's own steps are fp32: the extremes, the quotient by 15, the quotient by the scale
            lo, hi = v.min(-1, keepdims=True), v.max(-1, keepdims=True)
            zero = _directed(lo, -1)
            scale = _directed((hi - zero) / np.float32(15), +1)
            safe = np.where(scale > 0, scale, np.float32(1))
            code = np.where(scale > 0, np.clip(np.rint((v - zero) / safe), 0, 15), 0)
            vals[b, :, :c] = code.astype(np.float64) * scale.astype(np.float64) + zero
        return None, vals
    return None     # pages move whole: every output is a whole number


def _directed(x, way):
    """Nearest bf16 value not below (way +1) or not above (way -1) the fp32 x, by the neighbours of a cut."""
    cut = (np.ascontiguousarray(x).view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32)
    beyond = ((np.ascontiguousarray(cut).view(np.uint32) >> 16) + 1).astype(np.uint32)
    beyond = np.ascontiguousarray(beyond << np.uint32(16)).view(np.float32)
    miss = (cut < x) if way > 0 else (cut > x)
    return np.where(miss, beyond, cut)
